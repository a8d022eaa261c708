"""Attention of chunks over tens of thousands of places, where many units' parts are joined: single tokens, drafts and prompts'
chunks, with and without windows, biases and prefixes, against the oracle in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402,F401
from random_access_kv_gb300 import build as fbuild  # noqa: E402

KINDS = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("fmt,kind", [("int8", "bf16"), ("e4m3", "fp16"), ("e2m1", "bf16")])
@pytest.mark.parametrize("lens,news", [([40000], [1]), ([33333], [700]), ([60001, 17, 25000, 0], [1, 1, 5, 300]), ([20000] * 3, [257, 4, 512])])
def test_long_contexts(fmt, kind, lens, news):
    import chunk_cases as cc
    case = cc.Case(fmt, 64, 1, 128, lens, news)
    n = sum(news)
    q = cc.rows((n, 2, 64), 1, KINDS[kind])
    some = {0, n // 2, max(0, n - 301), n - 1}
    case.run(q, some=some)
    case.run(q, some=some, slopes=[2.0 ** -12, 2.0 ** -8], window=15000)
    case.run(q, some=some, prefix=[a + t // 2 for a, t in zip(lens, news)], cap=20.0)


def test_many_sequences_over_long_contexts():
    import chunk_cases as cc
    r = np.random.default_rng(4)
    lens, news = r.integers(1000, 20000, 24).tolist(), [1] * 20 + [2, 3, 4, 5]
    case = cc.Case("int8", 64, 1, 64, lens, news)
    case.run(cc.rows((34, 4, 64), 2, torch.bfloat16), some={0, 7, 19, 20, 27, 33})
