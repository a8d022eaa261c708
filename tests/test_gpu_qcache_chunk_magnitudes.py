"""Attention of chunks over value rows of any magnitude that the cache holds, 2^-98 to 2^124, alone and side by side: the sums of
weights do not hang on it. Against the oracle in 64 bits at the tolerance of tests/chunk_cases.py (whose 160 u counts the
logarithm of a value's scale, 141 at most)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402

LOW, HIGH = -98, 124


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def exponents(how, n, r):
    """log2 of the value rows' magnitude; -inf: a row of zeros."""
    if how == "rising":
        return np.linspace(LOW, HIGH, n)
    if how == "falling":
        return np.linspace(HIGH, LOW, n)
    if how == "random":
        return r.uniform(LOW, HIGH, n)
    if how == "tiles":                                         # every second tile of places
        return np.where(np.arange(n) // 128 % 2, -90.0, 60.0)
    if how == "few":                                           # ordinary ones, and a few that are not, and zeros
        e = np.zeros(n)
        e[r.integers(0, n, 4)] = (43.0, 50.0, 110.0, HIGH)
        e[r.integers(0, n, 20)] = -np.inf
        return e
    if how == "last huge" or how == "first huge":              # one huge row, the first to be taken or the last
        e = r.uniform(-20, 5, n)
        e[n - 1 if how == "last huge" else 0] = 100
        return e
    return np.full(n, float(how))


def make(fmt, d, lens, news, how, scores, seed):
    """Keys of which element 0 decides the score: equal ones, spread ones, or such that weight times value is alike all over."""
    import chunk_cases as cc
    K, V = [], []
    for b, n in enumerate(x + y for x, y in zip(lens, news)):
        r = np.random.default_rng([seed, b])
        e = exponents(how, n, r)
        k, v = 0.01 * r.standard_normal((n, 1, d)), r.standard_normal((n, 1, d)) * np.exp2(np.minimum(e, HIGH))[:, None, None]
        if scores == "spread":
            k[:, 0, 0] += 15.0 * r.standard_normal(n)
        elif scores == "against":
            k[:, 0, 0] -= np.log(2.0) * np.where(np.isfinite(e), e, 0)
        K.append(torch.from_numpy(k.astype(np.float32)).cuda())
        V.append(torch.from_numpy(np.clip(v, -2.0 ** 126, 2.0 ** 126).astype(np.float32)).cuda())
    return cc.Case(fmt, d, 1, 64, lens, news, K=K, V=V)


def queries(n, hq, d, dtype=torch.bfloat16):
    import chunk_cases as cc
    q = 0.02 * cc.rows((n, hq, d), 3, torch.float32)
    q[:, :, 0] = torch.linspace(0.5, 1.0, hq, device="cuda")
    return q.to(dtype)


HOW = ["-98", "-60", "43", "46", "80", "100", "124", "rising", "falling", "random", "tiles", "few", "last huge", "first huge"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("scores", ["equal", "spread", "against"])
def test_one_token_a_tile_to_a_unit(how, scores):
    # 24 tiles, each of them a part of its own
    make("int8", 64, [2999], [1], how, scores, 1).run(queries(1, 2, 64), scale=1.0)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("scores", ["equal", "spread", "against"])
def test_tokens_of_sequences_that_share_units(how, scores):
    # 240 tiles over the pairs of CTAs: both softmax groups at one row tile, and parts
    case = make("e4m3", 128, [2999] * 10, [1] * 10, how, scores, 2)
    case.run(queries(10, 4, 128), scale=1.0, some={0, 3, 9})


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("how", HOW)
def test_chunks(fmt, how):
    case = make(fmt, 64, [700, 0], [300, 150], how, "spread", 3)
    case.run(queries(450, 2, 64), scale=1.0, some={0, 1, 150, 299, 300, 301, 449})


@pytest.mark.parametrize("how", ["random", "few", "rising"])
@pytest.mark.parametrize("kw", [dict(window=200), dict(cap=30.0), dict(slopes=[0.05, 0.01]), dict(prefix=[900, 20])])
def test_masks_caps_and_biases(how, kw):
    case = make("int8", 64, [700, 0], [300, 150], how, "equal", 4)
    case.run(queries(450, 2, 64), scale=1.0, some={0, 1, 150, 299, 300, 301, 449}, **kw)


@pytest.mark.parametrize("how", ["-98", "-60", "rising", "random", "tiles"])
def test_float16_outputs(how):
    # what float16 holds of the outputs: exponents up to 10
    import chunk_cases as cc
    lens, news, K, V = [1400, 3], [200, 1], [], []
    for b, n in enumerate(x + y for x, y in zip(lens, news)):
        r = np.random.default_rng([5, b])
        e = np.minimum(exponents(how, n, r), 10)
        K.append(torch.from_numpy(r.standard_normal((n, 1, 64)).astype(np.float32)).cuda())
        V.append(torch.from_numpy((r.standard_normal((n, 1, 64)) * np.exp2(e)[:, None, None]).astype(np.float32)).cuda())
    case = cc.Case("int8", 64, 1, 64, lens, news, K=K, V=V)
    case.run(queries(201, 2, 64, torch.float16), scale=1.0, some={0, 77, 199, 200})


def test_odd_queries_and_absent_pages_beside_huge_values():
    case = make("int8", 64, [600], [140], "random", "equal", 6)
    q = queries(140, 4, 64)
    table = case.table.copy()
    table[0, 2], missing = -1, [np.r_[128:192]]
    case.run(q, scale=1.0, table=table, missing=missing, flags=fq.QC_FLAG_RANGE, some={0, 70, 139})
    good, glse = case.call(q, scale=1.0)
    bad = q.clone()
    bad[1, 0, 5], bad[1, 1, 0], bad[1, 3, 63] = float("nan"), float("inf"), -float("inf")
    out, lse = case.call(bad, scale=1.0)
    hit = torch.zeros((140, 4), dtype=torch.bool, device="cuda")
    hit[1, [0, 1, 3]] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], glse[~hit])
