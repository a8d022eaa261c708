"""The serving step's operators with as many sequences, and as large a vocabulary, as they take."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402

MOST = 65535


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("share", [1.0, 0.01])
def test_plan_write_and_attend_as_many_sequences_as_there_may_be(share):
    # one token of most sequences, or of a few with long runs of sequences between them that have none, over 0 to 15 cached ones
    r = np.random.default_rng(int(100 * share))
    lens, news = r.integers(0, 16, MOST), (r.random(MOST) < share).astype(np.int64)
    n, d, page = int(news.sum()), 64, 16
    ctx = fq.qc_create("e4m3", d, 1, page)
    pages = fq.alloc_pages(ctx, MOST)
    free, i64 = i32(r.permutation(MOST)), dict(dtype=torch.int64, device="cuda")

    def plan(ln, nw, table, taken):
        rows = int(np.sum(nw))
        starts, slots, pos = i32(np.zeros(MOST + 1)), torch.empty(rows, **i64), torch.empty(rows, **i64)
        took = torch.empty(1, **i64)
        fq.qc_plan(ctx, i32(ln), i32(nw), free, taken, table, starts, slots, pos, took)
        return starts, slots, pos, took

    table = torch.full((MOST, 1), -1, dtype=torch.int32, device="cuda")
    _, slots, pos, took = plan(np.zeros(MOST), lens, table, torch.zeros(1, **i64))           # the cached tokens
    owner = np.repeat(np.arange(MOST), lens)
    place = np.concatenate([np.arange(x) for x in lens])
    page_of = np.where(lens > 0, np.cumsum(lens > 0) - 1, -1)
    want = free.cpu().numpy()[page_of[owner]] * page + place
    assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(pos.cpu().numpy(), place) and int(took) == (lens > 0).sum()
    gen = torch.Generator(device="cuda").manual_seed(1)
    old = [torch.randn((len(want), 1, d), generator=gen, device="cuda") for _ in range(2)]
    fq.qc_write(ctx, *old, slots, pages)
    starts, slots, pos, took = plan(lens, news, table, took)
    new = [torch.randn((n, 1, d), generator=gen, device="cuda") for _ in range(2)]
    fq.qc_write(ctx, *new, slots, pages)
    q = torch.randn((n, 2, d), generator=gen, device="cuda").half()
    out, lse = torch.empty_like(q), torch.empty((n, 2), device="cuda")
    ws = fq.alloc_chunk_workspace(ctx, MOST, n, 2, 15, 1)
    fq.qc_attend_chunk(ctx, pages, q, starts, table, i32(lens), None, None, 0.125, 0.0, 0, 15, 1, out, lse, ws)
    assert fq.qc_status(ctx) == 0
    who = torch.from_numpy(np.flatnonzero(news)).cuda()
    at = table[who, 0].long()[:, None] * page + torch.arange(page, device="cuda")
    K, V = (torch.empty((n * page, 1, d), dtype=torch.float32, device="cuda") for _ in range(2))
    fq.qc_read(ctx, pages, at.reshape(-1), K, V)
    seen = (torch.arange(page, device="cuda")[None] <= i32(lens)[who][:, None])[:, None]
    K, V = (torch.where(seen[:, 0, :, None], x.view(n, page, d).double(), 0) for x in (K, V))
    s = torch.where(seen, 0.125 * torch.einsum("nhd,npd->nhp", q.double(), K), -torch.inf)
    p = torch.softmax(s, -1)
    right = torch.einsum("nhp,npd->nhd", p, V)
    # float32 scores of 64 products (their sizes sum to less than 100), weights of 22 bits, float16's rounding
    size = torch.einsum("nhp,npd->nhd", p, V.abs())
    assert ((out.double() - right).abs() <= 2.0 ** -11 * right.abs() + 2.0 ** -25 + 1e-4 * size).all()
    assert ((lse.double() - torch.logsumexp(s, -1)).abs() <= 1e-4).all()
    ctx.close()


def test_verify_as_many_sequences_as_there_may_be():
    r = np.random.default_rng(2)
    ctx = fq.qc_create("int8", 64, 1, 16)
    # probabilities of whole sixteenths, so that every sum is exact
    p, q = r.multinomial(16, [0.25] * 4, (MOST, 2)) / 16, r.multinomial(16, [0.25] * 4, (MOST, 1)) / 16
    tokens, u = r.integers(0, 4, (MOST, 1)), r.integers(0, 2 ** 20, (MOST, 2)) / 2 ** 20
    path, out, came = i32(np.full((MOST, 1), -9)), i32(np.full((MOST, 2), -9)), i32(np.full(MOST, -9))
    pd, qd, ud = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (p, q, u))
    fq.qc_verify(ctx, pd, qd, i32(tokens), None, None, ud, path, out, came)
    assert fq.qc_status(ctx) == 0
    row, x = np.arange(MOST), tokens[:, 0]
    ok = u[:, 0] * q[row, 0, x] < p[row, 0, x]
    left = np.maximum(p[:, 0] - q[:, 0], 0)
    left[left.sum(-1) == 0] = p[left.sum(-1) == 0, 0]
    w = np.where(ok[:, None], p[:, 1], left)
    last = (np.cumsum(w, -1) > (u[:, 1] * w.sum(-1))[:, None]).argmax(-1)
    assert np.array_equal(came.cpu().numpy(), ok) and np.array_equal(path[:, 0].cpu().numpy(), np.where(ok, 0, -1))
    want = np.where(ok[:, None], np.stack([x, last], 1), np.stack([last, np.full(MOST, -1)], 1))
    assert np.array_equal(out.cpu().numpy(), want)
    ctx.close()


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("off", [0, 1])
def test_verify_the_largest_vocabulary(kind, off):
    # whole multiples of 2^-24: every sum is exact. The token is rejected, and half of the vocabulary is left
    vocab, ctx = 2 ** 24, fq.qc_create("int8", 64, 1, 16)
    dtype = getattr(torch, kind)
    p = torch.full((1, 2, vocab + off), 2.0 ** -24, dtype=dtype, device="cuda")[..., off:]
    q = torch.zeros((1, 1, vocab + off), dtype=dtype, device="cuda")[..., off:]
    q[..., :vocab // 2] = 2.0 ** -23
    path, out, came = i32([[-9]]), i32([[-9, -9]]), i32([-9])
    for u, want in (([0.75, 0.25], 2 ** 23 + 2 ** 21), ([0.75, 0.0], 2 ** 23), ([0.75, 1 - 2.0 ** -24], vocab - 1)):
        fq.qc_verify(ctx, p, q, i32([[5]]), None, None, torch.tensor([u], device="cuda"), path, out, came)
        assert int(came) == 0 and out.tolist() == [[want, -1]], u
    fq.qc_verify(ctx, p, q, i32([[5]]), None, None, torch.tensor([[0.25, 0.5]], device="cuda"), path, out, came)
    assert int(came) == 1 and out.tolist() == [[5, 2 ** 23]]
    assert fq.qc_status(ctx) == 0
    ctx.close()
