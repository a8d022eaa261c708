"""Capped scores of the attention of chunks, place by place: small scores under a large cap keep their digits.

Bound, with u = 2^-24, of a score s = cap tanh(s0 / cap) against 64 bits. The dot product is off by |scale| (d + 8) u sum|q k|,
which capping does not enlarge. Where |s0| is below cap / 4 the rest is relative: five roundings up to the argument,
four of constants, one for the argument times them, three of the polynomial (6e-8 of its own included) and one of the last
product are 14 u |s| (16 here). From there on s is cap - 2 cap r with r = 1 / (1 + e^2a): an exponential of 2^-22.5 gives
2 cap r (1 - r) of that, cap 2^-23.5 at most; sum, reciprocal, constant and the last step 2 cap r (u + 2 u) + 2 u cap <= 5 u
cap; the argument's five roundings 5 u cap a sech^2 a <= 2.3 u cap: 9 u cap (12 here), whatever the score. A weight is
off by its score's error, by u (|s| + 160) for being taken with the logarithm of a value's scale and by 2^-19 (exponentials and
rescaling); the rest is as in tests/chunk_cases.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from oracle import qcache as oq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402

KINDS = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def check(case, q, out, lse, scale, cap, window=0, some=None):
    from chunk_cases import U, half_ulp, host
    d, group = q.shape[2], q.shape[1] // case.K[0].shape[1]
    bits = 11 if q.dtype is torch.float16 else 8
    rounding = 2.0 ** -22 if bits == 11 else 2.0 ** -11
    qh, got, glse, worst = host(q), host(out), host(lse), 0.0
    for row, (b, i) in enumerate((b, i) for b, t in enumerate(case.news) for i in range(t)):
        if some is not None and row not in some:
            continue
        lo, hi = oq.seen_by(case.lens[b] + i, case.lens[b] + case.news[b], 0, window)
        for h in range(q.shape[1]):
            k, v, x = case.K[b][lo:hi, h // group], case.V[b][lo:hi, h // group], qh[row, h]
            s0 = scale * (k @ x)
            s = cap * np.tanh(s0 / cap)
            e = abs(scale) * ((d + 8) * U * (np.abs(k) @ np.abs(x)) + (2.0 ** -38 * np.abs(x).max() * np.abs(k).sum(-1) if bits == 8 else 0))
            e = e + np.where(np.abs(s0) < 0.2499 * cap, 16 * U * np.abs(s), 12 * U * cap)
            w = e + U * (np.abs(s).max() + 160) + 2.0 ** -19
            p, m = np.exp(s - s.max()), len(s)
            p = p / p.sum()
            want, size = p @ v, p @ np.abs(v)
            tol = (p * w) @ np.abs(v) + (p @ w + rounding + (m / 4 + 64) * U) * size + half_ulp(want, bits)
            tol = tol + m * 2.0 ** -29 * 1.1 * (p * np.abs(v).max(-1)).max()
            err = np.abs(got[row, h] - want)
            assert (err <= tol).all(), ("out", b, i, h, (err / tol).max())
            worst = max(worst, (err / tol).max())
            wl = s.max() + np.log(np.exp(s - s.max()).sum())
            # to first order by the weights' errors, and U |s|, U 160 for the reference
            bound = p @ e + U * (np.abs(s).max() + 160) + U * abs(wl) + (m / 4 + 64) * U
            assert abs(glse[row, h] - wl) <= bound, ("lse", b, i, h, abs(glse[row, h] - wl) / bound)
    return worst


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("cap", [2.0 ** -20, 0.5, 5.0, 30.0, 1e3, 1e6, 2.0 ** 40])
def test_capped_scores(fmt, kind, cap):
    import chunk_cases as cc
    case = cc.Case(fmt, 64, 2, 64, [200, 0, 900], [40, 130, 1])
    q = cc.rows((171, 4, 64), 1, KINDS[kind])
    some = {0, 7, 39, 40, 41, 100, 169, 170}
    for scale in (0.125, 1.0, 6.0):
        out, lse = case.call(q, cap=cap, scale=scale)
        assert fq.qc_status(case.ctx) == 0
        check(case, q, out, lse, scale, cap, some=some)
        if cap >= 1e6:                                        # what an absolute bound would let through
            for wrong in (torch.zeros_like(out), out * 1.02):
                with pytest.raises(AssertionError):
                    check(case, q, wrong, lse, scale, cap, some=some)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_cap_far_above_the_scores_does_nothing(fmt, kind, d):
    # tanh(a) / a is 1 - 2^-80 or nearer: what a call without a cap gives is right for this one, too
    import chunk_cases as cc
    case = cc.Case(fmt, d, 1, 32, [300, 5], [70, 1])
    q = cc.rows((71, 3, d), 2, KINDS[kind])
    for scale in (d ** -0.5, 2.0):
        (out, lse), (plain, lse0) = case.call(q, cap=2.0 ** 40, scale=scale), case.call(q, scale=scale)
        check(case, q, out, lse, scale, 2.0 ** 40, some={0, 33, 69, 70})
        check(case, q, plain, lse0, scale, 2.0 ** 40, some={0, 33, 69, 70})


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_scores_around_a_quarter_of_the_cap(kind):
    # where one form ends and the other begins, and far above, in one tile: a head's keys grow along the places
    import chunk_cases as cc
    n, d = 640, 64
    K = torch.zeros((n, 1, d), device="cuda")
    K[:, 0, 0] = torch.linspace(-6, 6, n, device="cuda")
    case = cc.Case("int8", d, 1, 64, [500], [140], K=[K])
    q = torch.zeros((140, 2, d), dtype=KINDS[kind], device="cuda")
    q[:, :, 0] = 1.0
    for cap in (4.0, 1.0, 20.0):
        out, lse = case.call(q, cap=cap, scale=0.5, window=600)
        check(case, q, out, lse, 0.5, cap, window=600, some={0, 99, 139})
