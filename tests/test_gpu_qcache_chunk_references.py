"""Attention of chunks where the rows' references move: ahead of need and in need within one tile, in one row of a warp or in
several, against the oracle in 64 bits at the tolerance of tests/chunk_cases.py."""
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


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("news", [1, 200])
def test_two_moves_in_a_tile(kind, d, half, news):
    # tiles are taken from the last to the first. In tile 2 head 0's scores rise by 5 (its products pass 2^9, and its
    # reference moves at the next tile's start), in a half of tile 1 head 1's, and head 2's after both, by 20 (they pass
    # the limit). Both are rows of one warp
    import chunk_cases as cc
    n, r = 512, np.random.default_rng(d + half)
    K = 0.02 * r.standard_normal((n, 1, d))
    K[256:384, 0, 0] += 5.0
    K[256:384, 0, 2] += 5.0
    at = 128 + 64 * half
    K[at:at + 64, 0, 1] += 20.0
    K[at:at + 64, 0, 2] += 25.0
    K = torch.from_numpy(K.astype(np.float32)).cuda()
    case = cc.Case("int8", d, 1, 64, [n - news], [news], K=[K])
    q = torch.zeros((news, 4, d), dtype=KINDS[kind], device="cuda")
    for h in range(3):
        q[:, h, h] = 1.0
    q[:, 3] = cc.rows((news, d), 5, KINDS[kind])
    case.run(q, scale=1.0)
