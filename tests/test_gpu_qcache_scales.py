"""Values of unlike magnitude in one sequence, in the paged cache's attention: what a row sees is held to the bound of
its own largest product of weight and value scale, however large the values of places are that it does not see or
gives no weight; and elements that are zero in every heavy place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


SIZES = [(2, 2), (10, 4), (34, 2)]          # nodes and group: few rows; 40 and 68, for the tensor-core kernel


def floor(t, group):
    return 2.0 ** -20 if t * group <= 32 else None


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", SIZES)
@pytest.mark.parametrize("spread", [2.0 ** 12, 2.0 ** 30, 2.0 ** 40, 2.0 ** 90])
def test_large_values_of_places_that_rows_do_not_see(fmt, kind, t, group, spread):
    import qcache_cases as qc
    lens = [1201, 50]
    K = [qc.rows((n + t, 1, 64), 1) for n in lens]
    V = [qc.rows((n + t, 1, 64), 2) * 2.0 ** -3 for n in lens]
    for v, n in zip(V, lens):
        v[n] *= spread                       # the first node: seen by itself only
    sees = np.broadcast_to(np.eye(t, dtype=bool), (2, t, t)).copy()
    case = qc.Case(fmt, 64, 1, 32, K, V, lens, None, t, 1201)
    q = qc.rows((2, t, group, 64), 3, qc.TYPES[kind][0])
    out, lse = case.call(q, sees)
    skip = {(0, 0), (1, 0)} if kind == "fp16" else ()       # their own values are beyond fp16
    case.check(q, out, lse, sees, skip=skip, floor=floor(t, group))


@pytest.mark.parametrize("fmt", ["int8", "e2m1"])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", SIZES)
@pytest.mark.parametrize("where", ["first", "middle", "last", "all over"])
@pytest.mark.parametrize("bits", [24, 34, 45])
def test_large_values_that_have_no_weight(fmt, kind, t, group, where, bits):
    """Places of weight exp(-60) or so have values 2^bits times the others'."""
    import qcache_cases as qc
    n = 1301
    k, v = qc.rows((n + t, 1, 64), 4) * 0.3, qc.rows((n + t, 1, 64), 5) * 2.0 ** -8
    far = {"first": [0, 1], "middle": [640, 700], "last": [n - 1], "all over": list(range(5, n, 97))}[where]
    k[..., 0] = 10.0
    k[far, :, 0] = -50.0
    v[far] *= 2.0 ** bits
    case = qc.Case(fmt, 64, 1, 64, [k], [v], [n], None, t)
    q = qc.rows((1, t, group, 64), 6, qc.TYPES[kind][0]) * 0.5
    q[..., 0] = 8.0
    out, lse = case.call(q)
    case.check(q, out, lse, floor=floor(t, group))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", SIZES)
@pytest.mark.parametrize("bits", [10, 30, 60])
def test_the_heaviest_place_holds_least(kind, t, group, bits):
    """Scores rise along the prefix in steps and values fall, so that references and units move apart."""
    import qcache_cases as qc
    n = 2000
    step = torch.arange(n + t, device="cuda") // 100
    k, v = qc.rows((n + t, 1, 64), 7) * 0.2, qc.rows((n + t, 1, 64), 8)
    k[..., 0] = (step.float() * 5)[:, None]
    v *= torch.exp2(-step.float() * bits / 20)[:, None, None]
    case = qc.Case("int8", 64, 1, 16, [k], [v], [n], None, t)
    q = qc.rows((1, t, group, 64), 9, qc.TYPES[kind][0]) * 0.5
    q[..., 0] = 8.0
    out, lse = case.call(q)
    case.check(q, out, lse, floor=floor(t, group))


@pytest.mark.parametrize("t,group", SIZES)
@pytest.mark.parametrize("fmt", ["int8", "e2m1"])
def test_an_element_that_is_zero_in_the_heavy_places(fmt, t, group):
    """The bound that the header states holds for it: lighter weights may be off by 2^-29 of the heaviest product."""
    import qcache_cases as qc
    n = 1500
    k, v = qc.rows((n + t, 1, 64), 10) * 0.2, qc.rows((n + t, 1, 64), 11)
    k[..., 0] = 0.0
    k[::50, :, 0] = 12.0
    v[::50, :, 7] = 0.0
    case = qc.Case(fmt, 64, 1, 16, [k], [v], [n], None, t)
    for scale in (0.125, 0.5, 1.0, 1.5):
        q = qc.rows((1, t, group, 64), 12, torch.bfloat16) * 0.2
        q[..., 0] = 1.5
        out, lse = case.call(q, scale=scale)
        case.check(q, out, lse, scale=scale, floor=floor(t, group))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("scale", [0.75, 1.0, 1.25])
def test_light_places_beside_settled_heavy_ones(fmt, scale):
    """bf16 outputs of few rows: one channel is zero in all heavy places and large in the light ones, whose weights reach
    below fp16's. What is lost is within 2^-20 of the row's largest element a light place, as the header states."""
    import qcache_cases as qc
    n, t, group = 900, 1, 4
    k, v = torch.zeros((n + t, 1, 64), device="cuda"), qc.rows((n + t, 1, 64), 13)
    k[:100, :, 0] = 12.0 + torch.rand(100, 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    k[100:, :, 0] = torch.linspace(-2.0, 2.0, n + t - 100, device="cuda")[:, None]
    v[:100, :, 7], v[100:, :, 7] = 0.0, 100.0
    case = qc.Case(fmt, 64, 1, 16, [k], [v], [n], None, t)
    q = torch.zeros((1, t, group, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0
    out, _ = case.call(q, scale=scale)
    got = qc.host(out)[0, 0, 0]
    s = 2 * scale * case.K[0][:, 0, 0]
    p = np.exp(s - s.max())
    p /= p.sum()
    want, weight = p @ case.V[0][:, 0], p @ np.abs(case.V[0][:, 0])
    e = 2 * scale * 72 * qc.U * np.abs(case.K[0][:, 0, 0]).max() + 4 * qc.U * np.abs(s).max()
    tol = (2.0 ** -11 + 4 * e + 2.0 ** -20) * weight + qc.half_ulp(want, 8)
    assert (np.abs(got - want) <= tol + (n + t) * 2.0 ** -20 * np.abs(want).max()).all()
    others = np.arange(64) != 7
    assert (np.abs(got - want) <= tol + (n + t) * 2.0 ** -34 * np.abs(want).max())[others].all()


@pytest.mark.parametrize("t,group", [(2, 2), (40, 1)])
@pytest.mark.parametrize("low", [-28, -33, -36])
def test_small_elements_of_a_bf16_query(t, group, low):
    """Keys are zero where the query is largest: what counts is 2^low of it. Elements from 2^-30 on are exact, smaller
    ones to a step of 2^-37 of the power of two below the largest, as the header states."""
    import qcache_cases as qc
    n = 1100
    k = qc.rows((n + t, 1, 64), 14)
    k[..., 0] = 0.0
    case = qc.Case("int8", 64, 1, 16, [k], [qc.rows((n + t, 1, 64), 15)], [n], None, t)
    q = (qc.rows((1, t, group, 64), 16) * 2.0 ** low).to(torch.bfloat16)
    q[..., 0] = 1.5
    out, lse = case.call(q, scale=2.0 ** -low / 8)
    top = np.exp2(np.floor(np.log2(np.abs(qc.host(q)).max(-1, keepdims=True))))
    held = np.rint(qc.host(q) / (top * 2.0 ** -37)) * (top * 2.0 ** -37)
    if low == -28:
        assert (np.abs(held - qc.host(q)) <= np.where(np.abs(qc.host(q)) < top * 2.0 ** -30, top * 2.0 ** -38, 0)).all()
    case.check(torch.from_numpy(held).cuda(), out, lse, scale=2.0 ** -low / 8)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", SIZES)
@pytest.mark.parametrize("size", [0, -80, 60])
def test_log_sums_do_not_hang_on_the_values(kind, t, group, size):
    """Rows that see zeros only, beside nodes that do not (0), and caches of very small and very large values: the
    log-sum is as exact as that of any other."""
    import qcache_cases as qc
    lens = [5, 0, 1100]
    K = [qc.rows((n + t, 1, 64), 17) * 0.1 for n in lens]
    V = [qc.rows((n + t, 1, 64), 18) * 2.0 ** size for n in lens]
    sees = np.broadcast_to(np.eye(t, dtype=bool), (3, t, t)).copy()
    if size == 0:
        for n, v in zip(lens, V):
            v[:n + t - 1] = 0
        sees[:, 0, t - 1] = False
    case = qc.Case("e4m3", 64, 1, 64, K, V, lens, None, t, 1100)
    q = qc.rows((3, t, group, 64), 19, qc.TYPES[kind][0]) * 0.1
    out, lse = case.call(q, sees, 0.02)
    if kind == "fp16" and size:                              # outputs beyond fp16: the log-sums alone
        for b, n in enumerate(lens):
            for i in range(t):
                seen = [*range(n), n + i]
                s = 0.02 * (qc.host(q)[b, i] @ case.K[b][seen, 0].T)
                want = np.log(np.exp(s).sum(-1))
                e = 0.02 * 72 * qc.U * (np.abs(qc.host(q)[b, i]) @ np.abs(case.K[b][seen, 0]).T).max() + 4 * qc.U * np.abs(s).max()
                assert (np.abs(qc.host(lse)[b, i] - want) <= e + qc.U * np.abs(want) + (len(seen) / 4 + 64) * qc.U).all()
    else:
        case.check(q, out, lse, sees, 0.02, floor=floor(t, group))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("d,page,group", [(64, 16, 3), (128, 16, 1), (128, 64, 3), (64, 256, 8), (128, 256, 8)])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_rows_taken_again(fmt, d, page, group, kind):
    """Few rows, all but the first node's far below the unit: within one run of tiles and over several, under a tree, over
    absent pages, several heads."""
    import qcache_cases as qc
    t, lens = 5, [3001, 20, 0, 27]
    K = [qc.rows((n + t, 2, d), 20 + i) for i, n in enumerate(lens)]
    V = [qc.rows((n + t, 2, d), 30 + i) * 2.0 ** -3 for i, n in enumerate(lens)]
    for v, n in zip(V, lens):
        v[n, 1] *= 2.0 ** 70
    sees = np.broadcast_to(np.tril(np.ones((t, t), bool)), (4, t, t)).copy()
    sees[:, 1:, 0] = False
    sees[2, 3] = False
    case = qc.Case(fmt, d, 2, page, K, V, lens, [5, 4, 5, 5], t, 3001)
    q = qc.rows((4, t, 2 * group, d), 40, qc.TYPES[kind][0])
    skip = {(b, 0) for b in range(4)} if kind == "fp16" else ()
    out, lse = case.call(q, sees)
    case.check(q, out, lse, sees, skip=skip, floor=2.0 ** -20)
    table, gone = case.table.copy(), [3, 7]
    table[0, gone] = [-1, len(case.pages)]
    out, lse = case.call(q, sees, table=table)
    import random_access_kv_gb300 as fq
    assert fq.qc_status(case.ctx) == fq.QC_FLAG_RANGE
    keep = ~np.isin(np.arange(3001 + t) // page, gone)
    case.K[0], case.V[0], case.lens[0] = case.K[0][keep], case.V[0][keep], int(keep[:3001].sum())
    case.check(q, out, lse, sees, skip=skip, floor=2.0 ** -20)
