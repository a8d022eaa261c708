"""Pins of the quantised cache's oracle on the CPU: the code tables, rounding, error bounds, the page
layout and attention, each against something stated another way."""
import numpy as np
import pytest

from oracle import attention as oat
from oracle import qcache as oq

FMTS = ["int8", "e4m3", "e2m1"]


def test_code_tables():
    torch = pytest.importorskip("torch")
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oq.E4M3, want)
    assert oq.E4M3[-1] == 448 and (np.diff(oq.E4M3) > 0).all() and (np.diff(oq.E2M1) > 0).all()
    y = torch.from_numpy(np.random.default_rng(0).uniform(0, 460, 20000).astype(np.float32)).clamp(max=448)
    np.testing.assert_array_equal(oq.nearest(oq.E4M3, y.numpy()), y.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_nearest_takes_ties_to_even_codes():
    mid = (oq.E2M1[1:] + oq.E2M1[:-1]) / 2
    i = oq.nearest(oq.E2M1, mid)
    assert (i % 2 == 0).all() and (np.abs(oq.E2M1[i] - mid) == np.diff(oq.E2M1) / 2).all()
    np.testing.assert_array_equal(oq.nearest(oq.E2M1, [100.0, 0.0]), [7, 0])


@pytest.mark.parametrize("fmt", FMTS)
def test_round_trip_error(fmt):
    # int8: half a step of A / 127. e4m3: 2^-4 of the value, or half the least code. e2m1: a code is off by
    # at most 1/4 of its value or 1/4 (6 -> 5 is the widest: 1/6), the block scale by 2^-4 of itself,
    # which lets a block's largest value clip by as much.
    r = np.random.default_rng(3)
    x = (r.standard_normal((50, 3, 64)) * np.exp(r.uniform(-3, 3, (50, 3, 1)))).astype(np.float32)
    got = oq.values(*oq.quantise(x, fmt), fmt)
    A = np.abs(x).max(-1, keepdims=True).astype(np.float64)
    err = np.abs(got - x)
    if fmt == "int8":
        assert (err <= A / 254 * 1.0001).all()
    elif fmt == "e4m3":
        assert (err <= np.maximum(np.abs(x) / 16, A / 448 / 1024) * 1.0001).all()
    else:
        a = np.abs(x).reshape(50, 3, 4, 16).max(-1, keepdims=True).repeat(16, -1).reshape(x.shape)
        assert (err <= (a / 6 * 1.07 + A / 2688 * 2.0 ** -8)).all()
    np.testing.assert_allclose(np.abs(got).max(-1, keepdims=True), A, rtol=0.07)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_hold_zeros(fmt):
    x = np.zeros((4, 1, 64), dtype=np.float32)
    x[1, 0, 5] = 2.0 ** -101
    x[2, 0, 7] = np.nan
    x[3, 0, 9] = np.inf
    codes, scale, block = oq.quantise(x, fmt)
    assert (scale == 0).all() and (oq.values(codes, scale, block, fmt) == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_pages_hold_every_byte_once(fmt, d):
    page, heads, n_pages = 16, 2, 2
    pages = np.full((n_pages, oq.page_bytes(fmt, d, heads, page)), 0xEE, dtype=np.uint8)
    r = np.random.default_rng(1)
    slots = r.permutation(n_pages * page)
    k = r.standard_normal((len(slots), heads, d)).astype(np.float32)
    oq.pack(pages, slots, k, 0 * k, fmt, page)
    # values are zero, so every byte of theirs is; the keys' bytes are where read_row finds them
    rb = d // 2 if fmt == "e2m1" else d
    part = pages.shape[1] // heads
    for i in (0, 5, 31):
        p, t = divmod(int(slots[i]), page)
        for h in range(heads):
            raw = []
            for byte in range(t * rb, t * rb + rb):
                line, piece, inner = byte // 128, byte // 16 % 8, byte % 16
                raw.append(pages[p, h * part + line * 128 + (piece ^ (line % 8)) * 16 + inner])
            codes = oq.quantise(k[i, h], fmt)[0]
            if fmt == "e2m1":
                got = np.stack([np.array(raw) & 15, np.array(raw) >> 4], -1).ravel()
                np.testing.assert_array_equal(got, codes)
            else:
                np.testing.assert_array_equal(np.array(raw), codes & 255)
    for h in range(heads):
        assert (pages[:, h * part + page * rb:h * part + 2 * page * rb] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_is_a_rotation_of_the_normed_row(interleaved):
    r = np.random.default_rng(2)
    x, w = r.standard_normal((5, 3, 64)), r.uniform(0.5, 2, 64)
    pos, angle = np.array([0, 3, 9, 9, 1]), r.uniform(-3, 3, (10, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    y = oq.norm_rope(x, w, 0.0, pos, table, 32, interleaved)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True)) * w
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(n, axis=-1))
    np.testing.assert_allclose(y[..., 32:], n[..., 32:])
    # the same position turns two rows alike: their inner product stays; an opposite table undoes it
    np.testing.assert_allclose((y[2] * y[3]).sum(), (n[2] * n[3]).sum())
    back = oq.norm_rope(y, None, 0.0, pos, np.concatenate([np.cos(angle), -np.sin(angle)], 1), 32, interleaved)
    np.testing.assert_allclose(back, n, atol=1e-12)


def test_attend_against_the_codec_oracle_and_masks():
    r = np.random.default_rng(4)
    lens, nodes, hq, heads, d = [7, 0], [3, 2], 4, 2, 16
    K = [r.standard_normal((a + b, heads, d)) for a, b in zip(lens, nodes)]
    V = [r.standard_normal((a + b, heads, d)) for a, b in zip(lens, nodes)]
    q = r.standard_normal((2, 3, hq, d))
    sees = np.zeros((2, 3, 3), bool)
    sees[0] = np.tril(np.ones((3, 3), bool))
    sees[1, 1, 0] = True
    out, lse, _ = oq.attend(q, K, V, lens, nodes, sees, 0.3)
    for h in range(hq):
        want = oat.softmax_attention(q[0, 2, h], K[0][:, h // 2], V[0][:, h // 2], 0.3)
        np.testing.assert_allclose(out[0, 2, h], want)
        np.testing.assert_allclose(out[1, 1, h], V[1][0, h // 2])           # one place seen: its value
        np.testing.assert_allclose(lse[1, 1, h], 0.3 * q[1, 1, h] @ K[1][0, h // 2])
    assert (out[1, 0] == 0).all() and np.isneginf(lse[1, 0]).all()           # nothing seen
    assert (out[1, 2] == 0).all() and np.isneginf(lse[1, 2]).all()           # no such node
