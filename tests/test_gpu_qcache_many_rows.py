"""The paged cache's attention of more than 32 query rows per key/value head over bounds of 1,024 places and more, which
the tensor-core kernel takes: formats, types, page sizes, one and two row tiles, lengths around its tiles of 128,
masks, absent pages, references that move, streams and graphs; and the bits that weights keep, in both kernels."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402

FMTS = ["int8", "e4m3", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def random_tree(n_seq, t, seed):
    r = np.random.default_rng([seed, t])
    return np.tril(np.ones((t, t), bool))[None] & ((r.random((n_seq, t, t)) < 0.6) | np.eye(t, dtype=bool))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_formats_pages_and_types(fmt, d, page, kind):
    import qcache_cases as qc
    t, group = 9, 4                                         # 36 rows: one row tile
    case = qc.random_case(fmt, d, 2, page, [1024 - t, 300, 0], [t, 4, t], t, seed=page)
    case.run(qc.rows((3, t, 2 * group, d), 1, qc.TYPES[kind][0]), random_tree(3, t, page))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", [(33, 1), (17, 8), (65, 4), (5, 64)])
def test_rows_and_row_tiles(fmt, kind, t, group):            # 33, 136, 260, 320 rows: the last row tiles are not full
    import qcache_cases as qc
    d = 64 if t % 4 == 1 else 128
    case = qc.random_case(fmt, d, 1, 64, [1100, 0, 129], [t, t, (t + 1) // 2], t, seed=t)
    case.run(qc.rows((3, t, group, d), 2, qc.TYPES[kind][0]), random_tree(3, t, t))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [36, 130])
def test_lengths_around_a_tile(d, t):
    import qcache_cases as qc
    lens = [0, 1, 91, 92, 93, 127, 128, 129, 255, 256, 257, 383]
    case = qc.random_case("e4m3", d, 1, 16, lens, [t - i for i in range(len(lens))], t, 1024, seed=d)
    case.run(qc.rows((len(lens), t, 1, d), 3, torch.float16))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t", [36, 140])
def test_many_sequences_several_jobs_to_a_unit(kind, t):
    import qcache_cases as qc
    r = np.random.default_rng(t)
    lens = r.integers(0, 400, 70)
    lens[[3, 11]] = 0
    nodes = r.integers(0, t + 1, 70)
    case = qc.random_case("int8", 64, 4, 32, lens.tolist(), nodes.tolist(), t, 1024)
    q = qc.rows((70, t, 4, 64), 4, qc.TYPES[kind][0])
    out, lse = case.call(q)
    assert fq.qc_status(case.ctx) == 0
    case.check(q, out, lse, heads=[0, 3])


@pytest.mark.parametrize("t", [300, 1000])
def test_a_prompts_chunk(t):
    import qcache_cases as qc
    case = qc.random_case("int8", 64, 1, 64, [300, 0], [t, t - 7], t, 1024)
    q = qc.rows((2, t, 1, 64), 5, torch.bfloat16)
    out, lse = case.call(q)
    case.check(q, out, lse, skip={(b, i) for b in range(2) for i in range(t) if i % 7 and i not in (t - 8, t - 7, t - 1)})


@pytest.mark.parametrize("fmt,kind,d,t", [("e2m1", "fp16", 128, 1), ("e2m1", "bf16", 64, 40), ("e4m3", "fp16", 64, 6), ("e4m3", "fp16", 128, 40),
                                          ("e2m1", "fp16", 64, 40)])
def test_long_prefixes(fmt, kind, d, t):
    import qcache_cases as qc
    case = qc.random_case(fmt, d, 1, 64, [20011, 777], None, t, seed=6)
    q = qc.rows((2, t, 4, d), 6, qc.TYPES[kind][0])
    out, lse = case.call(q)
    case.check(q, out, lse, heads=[0, 3], skip={(b, i) for b in range(2) for i in range(3, t - 3)})


@pytest.mark.parametrize("t", [40, 140])
def test_rows_that_see_nothing(t):
    import qcache_cases as qc
    sees = np.zeros((3, t, t), bool)
    sees[0, 1, 0] = True
    sees[1, :, t - 1] = True
    for fmt, kind, lens, nodes in (("int8", "fp16", [0, 0, 40], [t, t, t]), ("e2m1", "bf16", [0, 0, 0], [0, 0, 0])):
        case = qc.random_case(fmt, 64, 1, 16, lens, nodes, t, 1024)
        case.run(qc.rows((3, t, 2, 64), 7, qc.TYPES[kind][0]), sees)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [3.0, -0.5, 0.0])
def test_peaked_negative_and_flat_scores(fmt, kind, scale):
    import qcache_cases as qc
    t = 40
    case = qc.random_case(fmt, 64, 1, 16, [1257, 90], None, t, seed=8)
    case.run(qc.rows((2, t, 2, 64), 8, qc.TYPES[kind][0]), scale=scale)


@pytest.mark.parametrize("rise", [1.0, 2.5, 3.5, 6.0])
def test_references_that_move(rise):
    """Scores rise by `rise` (base 2) every half tile of 64 places."""
    import qcache_cases as qc
    n, t = 2001, 40
    k = qc.rows((n + t, 1, 64), 9) * 0.05
    k[..., 0] = (torch.arange(n + t, device="cuda") // 64 * rise * float(np.log(2)))[:, None]
    for kind in ("fp16", "bf16"):
        case = qc.Case("e4m3", 64, 1, 32, [k], [qc.rows((n + t, 1, 64), 10)], [n], None, t)
        q = qc.rows((1, t, 2, 64), 11, qc.TYPES[kind][0]) * 0.05
        q[..., 0] = 1.0
        case.run(q, scale=1.0)


@pytest.mark.parametrize("q_scale", [2.0 ** 60, 2.0 ** -60])
def test_bf16_queries_beyond_fp16(q_scale):
    import qcache_cases as qc
    t = 40
    case = qc.random_case("e2m1", 128, 1, 32, [1100, 33], None, t, seed=12)
    case.run(qc.rows((2, t, 4, 128), 12, torch.bfloat16) * q_scale, scale=0.09 / q_scale)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_pages_that_do_not_exist_and_lengths_beyond_the_bound(fmt, page):
    import qcache_cases as qc
    t, d, n = 40, 64, 1100
    case = qc.random_case(fmt, d, 1, page, [n, n], None, t, seed=page)
    q = qc.rows((2, t, 1, d), 13, torch.float16)
    good = case.call(q)
    assert fq.qc_status(case.ctx) == 0
    case.check(q, *good)
    table = case.table.copy()
    gone = [1, 2, n // page // 2]
    table[1, gone] = [-1, len(case.pages), 2 ** 31 - 1]
    out, lse = case.call(q, table=table)
    assert fq.qc_status(case.ctx) == fq.QC_FLAG_RANGE
    assert torch.equal(out[0], good[0][0]) and torch.equal(lse[0], good[1][0])
    places = np.arange(n + t)
    keep = ~np.isin(places // page, gone)
    case.K[1], case.V[1], case.lens[1] = case.K[1][keep], case.V[1][keep], int(keep[:n].sum())
    case.check(q, out, lse)
    case = qc.random_case(fmt, d, 1, page, [n, 5], None, t, seed=page)
    good = case.call(q)
    out, lse = case.call(q, lens=[n + 1, 5])                  # clamped
    assert fq.qc_status(case.ctx) == fq.QC_FLAG_RANGE and torch.equal(out, good[0]) and torch.equal(lse, good[1])
    out, lse = case.call(q, lens=[n, -1])
    assert fq.qc_status(case.ctx) == fq.QC_FLAG_RANGE and torch.equal(out[0], good[0][0]) and torch.isfinite(out).all()


def test_strides_stream_and_counts():
    import qcache_cases as qc
    t, hq = 40, 4
    case = qc.random_case("e4m3", 64, 2, 16, [1037, 5], None, t, 1100)
    wide = qc.rows((2, hq + 3, t, 64), 14, torch.float16)
    q = wide[:, :hq].transpose(1, 2)                          # heads outermost, inside a wider row
    out, lse = case.call(q, counts=False, stream=torch.cuda.Stream())
    assert fq.qc_status(case.ctx) == 0
    case.check(q, out, lse)
    one = qc.rows((1, t, 1, 64), 15, torch.float16).expand(2, t, hq, 64)      # one query for all
    out, lse = case.call(one)
    case.check(one, out, lse)


@pytest.mark.parametrize("t", [1, 40])
def test_calls_in_a_graph(t):
    """A write and an attention, captured once and replayed over other inputs."""
    import qcache_cases as qc
    n = 1200
    case = qc.random_case("int8", 64, 1, 16, [n], None, t)
    q, k, v = (torch.zeros((1, t, 2, 64), dtype=torch.float16, device="cuda"), *(torch.zeros((t, 1, 64), device="cuda") for _ in range(2)))
    at = np.arange(n, n + t)
    slots = torch.from_numpy(case.table[0][at // 16].astype(np.int64) * 16 + at % 16).cuda()
    out, lse = torch.empty_like(q), torch.empty((1, t, 2), device="cuda")
    args = (torch.from_numpy(case.table).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), None, None, 0.125, n, out, lse,
            fq.alloc_attend_workspace(case.ctx, 1, t, 2, n))

    def step():
        fq.qc_write(case.ctx, k, v, slots, case.pages)
        fq.qc_attend(case.ctx, case.pages, q, *args)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.copy_(qc.rows(tuple(q.shape), 20 + i, torch.float16))
        k.copy_(qc.rows(tuple(k.shape), 30 + i))
        v.copy_(qc.rows(tuple(v.shape), 40 + i))
        graph.replay()
        torch.cuda.synchronize()
        held = torch.empty_like(k), torch.empty_like(v)
        fq.qc_read(case.ctx, case.pages, slots, *held)
        for have, new in zip((case.K, case.V), held):
            have[0][n:] = qc.host(new)
        case.check(q, out, lse)
    assert fq.qc_status(case.ctx) == 0


@pytest.mark.slow
def test_byte_offsets_beyond_32_bits():
    import qcache_cases as qc
    ctx, n, t = qc.context("e2m1", 128, 8, 64), 1100, 40
    each = -(-(n + t) // 64)
    n_pages = (5 << 30) // fq.qc_page_bytes(ctx)
    pages = torch.empty((n_pages, fq.qc_page_bytes(ctx)), dtype=torch.uint8, device="cuda")
    k, v, q = qc.rows((n + t, 8, 128), 15), qc.rows((n + t, 8, 128), 16), qc.rows((1, t, 8, 128), 17, torch.float16)
    at, got = torch.arange(n + t, device="cuda"), []
    for which in (n_pages - each + torch.arange(each, device="cuda"), torch.randperm(each, device="cuda")):
        fq.qc_write(ctx, k, v, which[at // 64] * 64 + at % 64, pages)
        out = torch.empty_like(q)
        fq.qc_attend(ctx, pages, q, which.int()[None].contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"), None, None, 0.09, n,
                     out, None, fq.alloc_attend_workspace(ctx, 1, t, 8, n))
        got.append(out)
    assert fq.qc_status(ctx) == 0
    assert torch.equal(got[0], got[1]) and got[0].abs().max() > 0


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t", [1, 40])
def test_bits_of_the_weights(kind, t):
    """Three values of equal weights that cancel, of sizes whose roundings do not: what is left of the sum shows the
    bits that the weights keep (an fp16 output's come in two halves)."""
    import qcache_cases as qc
    r = np.random.default_rng(1)
    d, n_seq = 64, 12
    V, K = [], []
    for b in range(n_seq):
        base = r.standard_normal((1, d))
        a, c = r.uniform(1, 2, 2)
        v = np.zeros((3 + t, 1, d))
        v[0], v[1], v[2] = base * a, base * c, -base * (a + c)
        V.append(torch.from_numpy(v.astype(np.float32)).cuda())
        K.append(torch.zeros((3 + t, 1, d), device="cuda"))
        K[-1][3:] = -100.0                                   # the nodes themselves weigh nothing
    case = qc.Case("int8", d, 1, 16, K, V, [3] * n_seq, None, t, 1100)
    q = torch.ones((n_seq, t, 1, d), dtype=qc.TYPES[kind][0], device="cuda")
    out, lse = case.call(q)
    case.check(q, out, lse)
    if kind == "fp16":
        assert qc.host(out).__abs__().max() < 2.0 ** -16
