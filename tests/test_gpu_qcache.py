"""The quantised paged cache on the GPU (include/qcache.h) against the oracle in 64 bits: head norm with
position rotation, write (every byte of the pages), read, and attention of drafted tokens over formats,
page sizes, head layouts, lengths, masks, strides and streams; the refusals of each call.

Tolerances, with u = 2^-24 the float32 unit roundoff:
* norm_rope: the mean square of d <= 128 elements is eight fused steps and at most four butterfly adds
  (12 u, halved by the root), plus rsqrt (2 ulp = 4 u), eps (u), two products (2 u); the rotation adds
  two products and a sum (2 u) of |a| + |b|. 16 u (|a| + |b|) bounds it, plus half an ulp of the type.
* write: equal bytes. read: one float32 product, rounded to the type: equal.
* attend: a score is off by e = scale (d + 8) u sum|q k| + 4 u |s| (products of codes are exact; sums of
  d terms, three scalings). A weight is off by 2^-11 (rounding to float16) + 2 e + 2^-21 (exponential and
  the running rescale, up to 16 times). out = sum p v / sum p: within (2^-11 + 4 e + 2^-20) sum p|v| / sum p
  plus half an ulp of the type. lse: e + u |lse| + (n / 4 + 64) u for sums of n weights in parts.
"""
import numpy as np
import pytest

from oracle import qcache as oq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402

U = 2.0 ** -24
TYPES = {"fp16": (torch.float16, 11), "bf16": (torch.bfloat16, 8), "fp32": (torch.float32, 24)}
FMTS = ["int8", "e4m3", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


_CTX = {}


def context(fmt="int8", d=64, heads=2, page=16):
    key = (fmt, d, heads, page)
    if key not in _CTX:
        _CTX[key] = fq.qc_create(*key)
    return _CTX[key]


def half_ulp(x, bits):
    """Half the spacing of a type of `bits` significant bits at |x| (fp16's least spacing 2^-24 included)."""
    a = np.maximum(np.abs(x), 2.0 ** -14 if bits == 11 else 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(a)) - bits) * 1.0001


def rows(shape, seed, dtype):
    r = np.random.default_rng([seed, *shape])
    x = r.standard_normal(shape) * np.exp(r.uniform(-1, 1, (*shape[:-1], 1))) * np.exp(r.uniform(-1, 1, shape[-1]))
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def host(t):
    return t.double().cpu().numpy()


# ---- norm_rope --------------------------------------------------------------------------------

def rope_table(most, rot, seed=0):
    a = np.random.default_rng(seed).uniform(-3, 3, (most, rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def check_norm_rope(got, x, w, eps, pos, table, rot, inter, bits):
    x, w = host(x), None if w is None else host(w)
    want = oq.norm_rope(x, w, eps, pos, None if table is None else host(table), rot, inter)
    size = np.abs(oq.norm_rope(x, w, eps, pos, None, 0, inter))
    pair = size.copy()
    half = rot // 2
    first = np.arange(half) * 2 if inter else np.arange(half)
    second = first + (1 if inter else half)
    pair[..., first] = pair[..., second] = size[..., first] + size[..., second]
    err = np.abs(host(got) - want)
    tol = 16 * U * pair + half_ulp(np.abs(want) + 16 * U * pair, bits)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 32, True), (64, 48, False), (128, 128, False), (128, 96, False),
                                         (128, 64, True), (128, 128, True), (128, 0, False), (64, 16, False)])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (3, 5, 2), (131, 12, 12)])
def test_norm_rope(kind, d, rot, inter, n, hq, hk):
    dtype, bits = TYPES[kind]
    ctx = context(d=d)
    x = rows((n, hq + 2 * hk, d), 1, dtype)                 # queries, keys and values in one row
    q, k = x[:, :hq], x[:, hq:hq + hk]
    wq, wk = rows((d,), 2, torch.float32), rows((d,), 3, torch.float32)
    table = rope_table(50, rot) if rot else None
    pos = np.random.default_rng(n).integers(0, 50, n)
    qo, ko = torch.empty((n, hq, d), dtype=dtype, device="cuda"), torch.empty((n, hk, d), dtype=dtype, device="cuda")
    fq.qc_norm_rope(ctx, q, k, wq, wk, 1e-5, torch.from_numpy(pos).cuda(), table, rot, inter, qo, ko)
    check_norm_rope(qo, q, wq, 1e-5, pos, table, rot, inter, bits)
    check_norm_rope(ko, k, wk, 1e-5, pos, table, rot, inter, bits)
    # in place, the rotation alone for the keys: the same numbers for the queries, the values untouched
    before = x.clone()
    fq.qc_norm_rope(ctx, q, k, wq, None, 1e-5, torch.from_numpy(pos).cuda(), table, rot, inter, q, k)
    assert torch.equal(q, qo) and torch.equal(x[:, hq + hk:], before[:, hq + hk:])
    check_norm_rope(k, before[:, hq:hq + hk], None, 1e-5, pos, table, rot, inter, bits)
    assert fq.qc_status(ctx) == 0


def test_norm_rope_many_rows_one_input_and_broadcast_heads():
    ctx, n = context(d=128), 6001
    q = rows((n, 1, 128), 4, torch.bfloat16).expand(n, 9, 128)          # head stride 0
    out = torch.empty((n, 9, 128), dtype=torch.bfloat16, device="cuda")
    pos, table, w = np.arange(n) % 77, rope_table(77, 128), rows((128,), 5, torch.float32)
    fq.qc_norm_rope(ctx, q, None, w, None, 0.0, torch.from_numpy(pos).cuda(), table, 128, False, out, None)
    check_norm_rope(out[::97], q[::97], w, 0.0, pos[::97], table, 128, False, 8)
    assert torch.equal(out[:, 0], out[:, 8])


def test_norm_rope_positions_out_of_the_table_and_zero_rows():
    ctx = context(d=64)
    x = rows((5, 3, 64), 6, torch.float16)
    x[1] = 0
    out = torch.full_like(x, 7)
    pos = torch.tensor([-1, 0, 10, 2 ** 40, 9], device="cuda")
    w = rows((64,), 5, torch.float32)
    fq.qc_norm_rope(ctx, None, x, None, w, 1e-6, pos, rope_table(10, 64), 64, True, None, out)
    assert fq.qc_status(ctx) == fq.QC_FLAG_RANGE and fq.qc_status(ctx) == 0
    assert (out[[0, 1, 2, 3]] == 0).all() and (out[4] != 0).any()


# ---- write and read ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,heads,page,n", [(64, 1, 16, 1), (64, 3, 32, 50), (128, 2, 64, 77), (128, 5, 16, 33), (64, 2, 256, 300)])
def test_write_every_byte_and_read(fmt, kind, d, heads, page, n):
    dtype, _ = TYPES[kind]
    ctx = context(fmt, d, heads, page)
    n_pages = n // page + 3
    r = np.random.default_rng([n, d])
    slots = r.permutation(n_pages * page)[:n].astype(np.int64)
    if n > 5:
        slots[[2, 4]] = -1
    x = rows((n, 2 * heads, d), 7, dtype)
    k, v = x[:, 0::2], x[:, 1::2]                              # interleaved heads: strides of their own
    v[0, 0, 3:9] = 0
    want = np.full((n_pages, oq.page_bytes(fmt, d, heads, page)), 0xA5, dtype=np.uint8)
    assert fq.qc_page_bytes(ctx) == want.shape[1]
    pages = torch.from_numpy(want).cuda()
    fq.qc_write(ctx, k, v, torch.from_numpy(slots).cuda(), pages)
    oq.pack(want, slots, k.float().cpu().numpy(), v.float().cpu().numpy(), fmt, page)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    order = r.permutation(n)
    for out_kind in TYPES:
        odt = TYPES[out_kind][0]
        ko, vo = (torch.full((n, heads, d), 3.0, dtype=odt, device="cuda") for _ in range(2))
        fq.qc_read(ctx, pages, torch.from_numpy(slots[order]).cuda(), ko, vo)
        for got, x in ((ko, k), (vo, v)):
            held = oq.values(*oq.quantise(x.float().cpu().numpy()[order], fmt), fmt)
            held[slots[order] == -1] = 0
            # code times scale is exact in 64 bits: one rounding to float32, one to the type
            assert torch.equal(got.cpu(), torch.from_numpy(held.astype(np.float32)).to(odt)), out_kind
    only = torch.empty((n, heads, d), dtype=dtype, device="cuda")
    fq.qc_read(ctx, pages, torch.from_numpy(slots).cuda(), None, only)
    both = torch.empty_like(only)
    fq.qc_read(ctx, pages, torch.from_numpy(slots).cuda(), torch.empty_like(only), both)
    assert torch.equal(only, both) and fq.qc_status(ctx) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", TYPES)
def test_write_and_read_of_many_rows_at_any_allowed_alignment(fmt, kind):
    d, heads, page, n = 128, 2, 64, 20011                       # enough for several rows to a lane group
    dtype, _ = TYPES[kind]
    ctx = context(fmt, d, heads, page)
    n_pages = n // page + 2
    r = np.random.default_rng(n)
    slots = r.permutation(n_pages * page)[:n].astype(np.int64)
    some = 16 // torch.empty((), dtype=dtype).element_size()    # 16 bytes: off the 32 of a whole store
    x = rows((1, some + n * heads * d), 31, dtype)[0, some:].view(n, heads, d)
    want = np.zeros((n_pages, oq.page_bytes(fmt, d, heads, page)), dtype=np.uint8)
    pages = torch.from_numpy(want).cuda()
    fq.qc_write(ctx, x, x, torch.from_numpy(slots).cuda(), pages)
    xs = x.float().cpu().numpy()
    oq.pack(want, slots, xs, xs, fmt, page)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    held = torch.from_numpy(oq.values(*oq.quantise(xs, fmt), fmt).astype(np.float32)).to(dtype)
    room = torch.full((2 * some + n * heads * d,), 3.0, dtype=dtype, device="cuda")
    off, whole = room[some:-some].view(n, heads, d), torch.empty((n, heads, d), dtype=dtype, device="cuda")
    assert off.data_ptr() % 32 == 16 and whole.data_ptr() % 32 == 0
    fq.qc_read(ctx, pages, torch.from_numpy(slots).cuda(), off, whole)
    assert torch.equal(off.cpu(), held) and torch.equal(whole.cpu(), held)
    assert (room[:some] == 3).all() and (room[-some:] == 3).all() and fq.qc_status(ctx) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_write_edge_rows(fmt):
    ctx = context(fmt, 64, 1, 16)
    x = rows((12, 1, 64), 8, torch.float32)
    x[0] = 0
    x[1] = x[1] * 2.0 ** -110
    x[2, 0, 3] = float("nan")
    x[3, 0, 63] = float("-inf")
    x[4] = torch.linspace(-3.4028234e38, 3.4028234e38, 64)
    x[5] = torch.arange(64) - 32.0
    x[6, 0] = torch.arange(64) / 4 - 8
    x[6, 0, 0] = 127.0 if fmt == "int8" else 448.0 if fmt == "e4m3" else 2688.0     # exact units: ties
    x[7, 0, 1:] = 0
    x[8, 0, 16:] *= 2.0 ** -20                                                      # blocks below the least scale
    x[9] = 2.0 ** -100
    slots = np.arange(12, dtype=np.int64)
    want = np.zeros((1, oq.page_bytes(fmt, 64, 1, 16)), dtype=np.uint8)
    pages = torch.from_numpy(want).cuda()
    fq.qc_write(ctx, x, x, torch.from_numpy(slots).cuda(), pages)
    assert fq.qc_status(ctx) == fq.QC_FLAG_NONFINITE
    oq.pack(want, slots, x.cpu().numpy(), x.cpu().numpy(), fmt, 16)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)


def test_slots_out_of_range_are_skipped_or_read_as_zeros():
    ctx = context("e4m3", 64, 2, 16)
    pages = fq.alloc_pages(ctx, 2)
    x = rows((6, 2, 64), 9, torch.float16)
    slots = torch.tensor([0, 32, -2, 31, -1, 2 ** 40], device="cuda")
    fq.qc_write(ctx, x, x, slots, pages)
    assert fq.qc_status(ctx) == fq.QC_FLAG_RANGE
    out = torch.full_like(x, 5)
    fq.qc_read(ctx, pages, slots, out, None)
    assert fq.qc_status(ctx) == fq.QC_FLAG_RANGE
    assert (out[[1, 2, 4, 5]] == 0).all() and (out[[0, 3]] != 0).any(-1).all()
    fq.qc_read(ctx, pages, slots[[0, 4]], out[:2], None)
    assert fq.qc_status(ctx) == 0


# ---- attend -----------------------------------------------------------------------------------

def tree_words(sees):
    n_seq, t, _ = sees.shape
    bits = np.zeros((n_seq, t, -(-t // 32) * 32), dtype=np.uint64)
    bits[..., :t] = sees
    w = (bits.reshape(n_seq, t, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32)).cuda()


def run_attend(fmt, kind, d, heads, group, page, lens, nodes, t, seed=0, tree=True, use_nodes=True, scale=None, sees=None,
               slack=0, q_layout="flat", stream=None, q_scale=1.0, sample=None):
    """A cache of dirty pages (every byte 0xFF: NaN scales) with only the places of lens + nodes written."""
    dtype, bits = TYPES[kind]
    ctx = context(fmt, d, heads, page)
    r = np.random.default_rng([seed, d, heads, t, len(lens)])
    n_seq, hq = len(lens), heads * group
    nodes = list(nodes) if use_nodes else [t] * n_seq
    max_len = max(lens) + slack
    each = -(-(max_len + t) // page)
    n_pages = n_seq * each + 2
    table = r.permutation(n_pages)[:n_seq * each].reshape(n_seq, each).astype(np.int32)
    pages = torch.full((n_pages, fq.qc_page_bytes(ctx)), 0xFF, dtype=torch.uint8, device="cuda")
    K, V = [], []
    for b in range(n_seq):
        n = lens[b] + nodes[b]
        at = np.arange(n)
        slots = torch.from_numpy(table[b][at // page].astype(np.int64) * page + at % page).cuda()
        k, v = rows((n, heads, d), 10 * seed + b, torch.float32), rows((n, heads, d), 500 + 10 * seed + b, torch.float32)
        if n:
            fq.qc_write(ctx, k, v, slots, pages)
            ko, vo = torch.empty_like(k), torch.empty_like(v)
            fq.qc_read(ctx, pages, slots, ko, vo)
            k, v = ko, vo
        K.append(host(k))
        V.append(host(v))
    if q_layout == "packed":                                   # queries inside a wider row, heads outermost
        wide = rows((n_seq, hq + 3, t, d), seed + 77, dtype) * q_scale
        q = wide[:, :hq].transpose(1, 2)
    else:
        q = rows((n_seq, t, hq, d), seed + 77, dtype) * q_scale
    if sees is None:
        sees = np.tril(np.ones((t, t), bool))[None].repeat(n_seq, 0)
        if tree:
            sees &= (r.random((n_seq, t, t)) < 0.6) | np.eye(t, dtype=bool)
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = torch.full((n_seq, t, hq, d), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((n_seq, t, hq), 9.0, dtype=torch.float32, device="cuda")
    ws = fq.alloc_attend_workspace(ctx, n_seq, t, hq, max_len)
    ws.fill_(0xFF)
    args = (ctx, pages, q, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.tensor(nodes, dtype=torch.int32, device="cuda") if use_nodes else None,
            tree_words(sees) if tree else None, scale, max_len)
    torch.cuda.synchronize()
    fq.qc_attend(*args, out, lse, ws, stream)
    torch.cuda.synchronize()
    assert fq.qc_status(ctx) == 0
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    fq.qc_attend(*args, again, lse2, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call gives the same bits"
    fq.qc_attend(*args, again.zero_(), None, ws)
    assert torch.equal(out, again)
    got, glse, qh = host(out), host(lse), host(q)
    heads_seen = range(hq) if sample is None else sample
    qs = qh[:, :, list(heads_seen)]
    worst = 0.0
    for j, h in enumerate(heads_seen):
        kv = h // group
        want, wl, weight = oq.attend(qs[:, :, j:j + 1], [x[:, kv:kv + 1] for x in K], [x[:, kv:kv + 1] for x in V], lens, nodes,
                                     sees, scale)
        for b in range(n_seq):
            n = lens[b] + nodes[b]
            if not n:
                assert (got[b, :, h] == 0).all() and np.isneginf(glse[b, :, h]).all()
                continue
            mags = np.abs(qs[b, :, j]) @ np.abs(K[b][:, kv]).T                           # [t, n]: sum |q k|
            s = np.abs(qs[b, :, j] @ K[b][:, kv].T).max(-1)
            e = (abs(scale) * ((d + 8) * U * mags.max(-1) + 4 * U * s))
            tol = (2.0 ** -11 + 4 * e + 2.0 ** -20)[:, None] * weight[b, :, 0] + half_ulp(want[b, :, 0], bits)
            err = np.abs(got[b, :, h] - want[b, :, 0])
            assert (err <= tol).all(), (b, h, (err / tol).max())
            worst = max(worst, (err / tol).max())
            fin = np.isfinite(wl[b, :, 0])
            np.testing.assert_array_equal(np.isfinite(glse[b, :, h]), fin)
            assert (glse[b, ~fin, h] == -np.inf).all() and (got[b, ~fin, h] == 0).all()
            tol = e + U * np.abs(np.where(fin, wl[b, :, 0], 0)) + (n / 4 + 64) * U
            assert (np.abs(glse[b, fin, h] - wl[b, fin, 0]) <= tol[fin]).all(), (b, h)
    return worst


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_attend_single_token(fmt, d, kind):
    run_attend(fmt, kind, d, 2, 1, 16, [0, 1, 14, 15, 16, 63, 64, 200], [1] * 8, 1, tree=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attend_pages(fmt, d, page):
    run_attend(fmt, "fp16", d, 2, 2, page, [page - 1, 3 * page, 2 * page + 5, 0], [4, 1, 3, 2], 4, seed=page)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads,group,t", [(1, 1, 2), (1, 4, 16), (2, 3, 5), (1, 8, 17), (2, 8, 4), (1, 5, 33), (1, 4, 64),
                                           (2, 12, 7), (1, 1, 130), (1, 8, 65), (1, 64, 3)])
def test_attend_groups_and_nodes(fmt, heads, group, t):
    d = 128 if t % 2 else 64
    run_attend(fmt, "bf16" if group % 2 else "fp16", d, heads, group, 32, [130, 0, 31], [t, max(1, t - 1), (t + 1) // 2], t, seed=t)


@pytest.mark.parametrize("d,group,t", [(64, 1, 1), (128, 4, 1), (128, 8, 9), (64, 8, 40), (128, 4, 64)])
def test_attend_long_prefix_is_split(d, group, t):
    run_attend("int8", "bf16", d, 1, group, 64, [20011, 777], [t, t], t, seed=3, sample=[0, group - 1])


@pytest.mark.parametrize("layout", ["flat", "packed"])
def test_attend_causal_chain_without_tree_or_counts(layout):
    run_attend("e4m3", "fp16", 64, 2, 4, 16, [37, 5], None, 6, tree=False, use_nodes=False, q_layout=layout, slack=100)


@pytest.mark.parametrize("t", [5, 40])
def test_attend_rows_that_see_nothing(t):
    sees = np.zeros((3, t, t), bool)
    sees[0, 1, 0] = True
    sees[1, :, t - 1] = True                       # places later than the node's own
    run_attend("int8", "fp16", 128, 1, 4, 16, [0, 0, 40], [t, t, t], t, sees=sees)
    run_attend("e2m1", "bf16", 64, 1, 4, 16, [0, 0, 0], [0, 0, 0], t, sees=sees)


@pytest.mark.parametrize("t", [1, 40])
@pytest.mark.parametrize("scale", [3.0, -0.5, 0.0])
def test_attend_peaked_negative_and_flat_scores(scale, t):
    run_attend("int8", "fp16", 64, 1, 2, 16, [257, 90], [t, t], t, scale=scale, seed=5)


@pytest.mark.parametrize("t", [1, 40])
@pytest.mark.parametrize("q_scale", [2.0 ** 60, 2.0 ** -60])
def test_attend_bf16_queries_beyond_fp16(q_scale, t):
    run_attend("e2m1", "bf16", 128, 1, 4, 32, [100, 33], [t, t], t, q_scale=q_scale, scale=0.09 / q_scale, seed=6)


@pytest.mark.parametrize("t", [1, 40])
def test_attend_on_another_stream(t):
    s = torch.cuda.Stream()
    run_attend("e4m3", "bf16", 128, 2, 2, 64, [500, 10], [t, t], t, stream=s, seed=8)


@pytest.mark.parametrize("t", [1, 40])
def test_attend_values_of_unlike_scales(t):
    """The heaviest places hold zero or tiny values: what the others give must not be lost beside them."""
    ctx, n = context("int8", 64, 1, 16), 200
    k = torch.zeros((n + t, 1, 64), device="cuda")
    k[:, 0, 0] = 1.0
    k[5, 0, 0] = k[n - 1, 0, 0] = 12.0                        # weights e^11 times the others'
    v = rows((n + t, 1, 64), 11, torch.float32)
    v[5], v[n - 1] = 0, v[n - 1] * 2.0 ** -30
    pages = fq.alloc_pages(ctx, -(-(n + t) // 16))
    slots = torch.arange(n + t, device="cuda")
    fq.qc_write(ctx, k, v, slots, pages)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    fq.qc_read(ctx, pages, slots, kk, vv)
    q = torch.zeros((1, t, 1, 64), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    out = torch.empty_like(q)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    table = torch.arange(len(pages), dtype=torch.int32, device="cuda")[None]
    sees = np.eye(t, dtype=bool)[None]
    fq.qc_attend(ctx, pages, q, table, lens, None, tree_words(sees), 1.0, n, out, None, fq.alloc_attend_workspace(ctx, 1, t, 1, n))
    want, _, weight = oq.attend(host(q), [host(kk)], [host(vv)], [n], [t], sees, 1.0)
    # beside the usual bound, a weight below 2^-24 of the largest p |v| may vanish
    tol = 2.0 ** -10 * weight + half_ulp(want, 11) + 2.0 ** -24
    assert (np.abs(host(out) - want) <= tol).all()


def test_attend_flags_bad_pages_lengths_and_counts():
    ctx = context("int8", 64, 1, 16)
    pages = fq.alloc_pages(ctx, 4)
    k, v = rows((64, 1, 64), 12, torch.float16), rows((64, 1, 64), 13, torch.float16)
    fq.qc_write(ctx, k, v, torch.arange(64, device="cuda"), pages)
    q = rows((1, 1, 1, 64), 14, torch.float16)
    ws = fq.alloc_attend_workspace(ctx, 1, 1, 1, 63)

    def call(table, length, nodes=1):
        out = torch.empty_like(q)
        fq.qc_attend(ctx, pages, q, torch.tensor([table], dtype=torch.int32, device="cuda"),
                     torch.tensor([length], dtype=torch.int32, device="cuda"),
                     torch.tensor([nodes], dtype=torch.int32, device="cuda"), None, 0.1, 63, out, None, ws)
        return out, fq.qc_status(ctx)

    good, flag = call([0, 1, 2, 3], 63)
    assert flag == 0
    out, flag = call([0, 7, 2, -1], 63)                       # tokens of pages 7 and -1 are not seen
    assert flag == fq.QC_FLAG_RANGE
    keep = torch.cat([k[:16], k[32:48]]), torch.cat([v[:16], v[32:48]])
    held = [oq.values(*oq.quantise(x.float().cpu().numpy(), "int8"), "int8") for x in keep]
    want, _, _ = oq.attend(host(q), [held[0]], [held[1]], [31], [1], np.ones((1, 1, 1), bool), 0.1)
    np.testing.assert_allclose(host(out), want, atol=2e-3)
    out, flag = call([0, 1, 2, 3], 64)                        # clamped to max_len
    assert flag == fq.QC_FLAG_RANGE and torch.equal(out, good)
    out, flag = call([0, 1, 2, 3], -5)
    assert flag == fq.QC_FLAG_RANGE and torch.isfinite(out).all()
    out, flag = call([0, 1, 2, 3], 63, 2)
    assert flag == fq.QC_FLAG_RANGE and torch.equal(out, good)
    out, flag = call([0, 1, 2, 3], 63, -1)
    assert flag == fq.QC_FLAG_RANGE and (out == 0).all()


@pytest.mark.slow
@pytest.mark.parametrize("t", [1, 64])
def test_attend_beyond_four_gigabytes(t):
    """Pages whose byte offsets pass 32 bits."""
    ctx = context("int8", 128, 8, 64)
    n_pages = (5 << 30) // fq.qc_page_bytes(ctx)
    pages = torch.empty((n_pages, fq.qc_page_bytes(ctx)), dtype=torch.uint8, device="cuda")
    far = n_pages - 3 + torch.arange(3, device="cuda")
    n = 150
    at = torch.arange(n, device="cuda")
    k, v = rows((n, 8, 128), 15, torch.float32), rows((n, 8, 128), 16, torch.float32)
    q = rows((1, t, 8, 128), 17, torch.bfloat16)
    got = []
    for which in (far, torch.tensor([2, 0, 1], device="cuda")):
        slots = which[at // 64] * 64 + at % 64
        fq.qc_write(ctx, k, v, slots, pages)
        back = torch.empty_like(k)
        fq.qc_read(ctx, pages, slots, None, back)
        out = torch.empty_like(q)
        fq.qc_attend(ctx, pages, q, which.int()[None].contiguous(), torch.tensor([n - t], dtype=torch.int32, device="cuda"), None,
                     None, 0.09, n - t, out, None, fq.alloc_attend_workspace(ctx, 1, t, 8, n - t))
        got.append((back, out))
    assert fq.qc_status(ctx) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[0][1].abs().max() > 0


# ---- refusals ---------------------------------------------------------------------------------

def test_norm_rope_refusals():
    ctx = context(d=64)
    x = rows((4, 2, 64), 1, torch.float16)
    o, w, pos, tab = torch.zeros_like(x), torch.ones(64, device="cuda"), torch.arange(4, device="cuda"), rope_table(9, 64)

    def call(q=x, k=None, w=w, eps=1e-6, pos=pos, tab=tab, rot=64, out=o):
        fq.qc_norm_rope(ctx, q, k, w, None, eps, pos, tab, rot, False, out, None)

    call()
    o.zero_()
    for bad in (dict(q=None), dict(q=x[:, :, :32]), dict(q=x.double()), dict(q=x.cpu()), dict(out=o[:3]), dict(out=o.float()),
                dict(q=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(w=w.half()), dict(w=w[:32]), dict(pos=pos.int()),
                dict(pos=pos[:2]), dict(tab=tab[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(rot=8, tab=rope_table(9, 8)), dict(rot=80, tab=rope_table(9, 80))):
        with pytest.raises(fq.FQError) as e:
            call(**bad)
        assert e.value.code == 1
    wide = rows((4, 2, 72), 1, torch.float16)
    for q in (wide[:, :, 4:68], rows((4, 2, 68), 1, torch.float16)[:, :, :64]):
        with pytest.raises(fq.FQError) as e:
            call(q=q)
        assert e.value.code == 4
    torch.cuda.synchronize()
    assert (o == 0).all()
    call(q=x[:0], pos=pos[:0], out=o[:0])                     # nothing to do


def test_write_and_read_refusals():
    ctx = context("int8", 64, 2, 16)
    x, slots, pages = rows((4, 2, 64), 1, torch.float16), torch.arange(4, device="cuda"), fq.alloc_pages(context("int8", 64, 2, 16), 2)
    for args in ((x[:, :1], x, slots, pages), (x, x[:3], slots, pages), (x, x.float(), slots, pages), (x.double(), x.double(), slots, pages),
                 (x, x, slots.int(), pages), (x, x, slots[:2], pages), (x, x, slots, pages[:, :-16]), (x, x, slots, pages.cpu())):
        with pytest.raises((ValueError, TypeError)):
            fq.qc_write(ctx, *args)
        with pytest.raises((ValueError, TypeError)):
            k, v, s, p = args
            fq.qc_read(ctx, p, s, k, v)
    with pytest.raises(ValueError):
        fq.qc_read(ctx, pages, slots, torch.empty((4, 2, 128), dtype=torch.float16, device="cuda")[:, :, ::2], None)
    buf = torch.zeros(2 * pages.numel() + 16, dtype=torch.uint8, device="cuda")
    off = buf[8:8 + pages.numel()].view_as(pages)
    for call in (lambda: fq.qc_write(ctx, x, x, slots, off), lambda: fq.qc_read(ctx, off, slots, torch.empty_like(x), None)):
        with pytest.raises(fq.FQError) as e:
            call()
        assert e.value.code == 4
    torch.cuda.synchronize()
    assert (pages == 0).all() and (buf == 0).all()
    fq.qc_write(ctx, x[:0], x[:0], slots[:0], pages)
    fq.qc_read(ctx, pages, slots[:0], x[:0].contiguous(), None)


def test_attend_refusals():
    ctx = context("int8", 64, 2, 16)
    pages = fq.alloc_pages(ctx, 4)
    i32 = dict(dtype=torch.int32, device="cuda")
    base = dict(pages=pages, q=rows((2, 3, 4, 64), 1, torch.float16), table=torch.zeros((2, 2), **i32), lens=torch.full((2,), 9, **i32),
                nodes=None, tree=torch.zeros((2, 3, 1), **i32), scale=0.1, max_len=20, out=torch.zeros((2, 3, 4, 64), dtype=torch.float16,
                                                                                                       device="cuda"),
                lse=torch.zeros((2, 3, 4), device="cuda"), workspace=fq.alloc_attend_workspace(ctx, 2, 3, 4, 20))

    def call(**kw):
        fq.qc_attend(ctx, *{**base, **kw}.values())

    for bad in (dict(q=base["q"][..., :32]), dict(q=base["q"][0]), dict(q=base["q"].float(), out=base["out"].double()),
                dict(out=base["out"].bfloat16()), dict(out=base["out"][:, :2]), dict(table=base["table"].long()),
                dict(table=base["table"][:1]), dict(lens=base["lens"][:1]), dict(lens=base["lens"].cpu()), dict(nodes=base["lens"].long()),
                dict(tree=torch.zeros((2, 3, 2), **i32)), dict(lse=base["lse"].half()), dict(workspace=base["workspace"].float()),
                dict(pages=pages[:, :-16].contiguous())):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    q3 = rows((2, 3, 3, 64), 1, torch.float16)                # three query heads over two
    for bad in (dict(scale=float("inf")), dict(scale=float("nan")), dict(max_len=30), dict(max_len=-1),
                dict(q=q3, out=torch.zeros_like(q3), lse=None), dict(q=base["q"].float(), out=base["out"].float()),
                dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        if "workspace" in bad and fq.qc_attend_workspace(ctx, 2, 3, 4, 20) == 0:
            continue
        with pytest.raises(fq.FQError) as e:
            call(**bad)
        assert e.value.code == 1, bad
    torch.cuda.synchronize()
    assert (base["out"] == 0).all()
    for args in ((-1, 1, 4, 8), (1, 0, 4, 8), (1, 1025, 4, 8), (1, 1, 5, 8), (1, 1, 256, 8), (1, 1, 4, -1), (70000, 1, 4, 8)):
        with pytest.raises(fq.FQError):
            fq.qc_attend_workspace(ctx, *args)


def test_create_refusals_and_lifetime():
    for args in (("int8", 96, 1, 16), ("int8", 64, 0, 16), ("int8", 64, 2000, 16), ("int8", 64, 1, 24), ("int8", 64, 1, 8),
                 ("int8", 64, 1, 512)):
        with pytest.raises(fq.FQError) as e:
            fq.qc_create(*args)
        assert e.value.code == 1
    with pytest.raises(ValueError):
        fq.qc_create("int4", 64, 1, 16)
    with pytest.raises(fq.FQError) as e:
        fq.qc_create("int8", 64, 1, 16, 99)
    assert e.value.code == 5
    ctx = fq.qc_create("e2m1", 128, 3, 32)
    fq.qc_destroy(ctx)
    with pytest.raises(fq.FQError):
        fq.qc_page_bytes(ctx)
