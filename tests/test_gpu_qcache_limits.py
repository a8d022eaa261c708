"""Sizes past what the paged cache's calls take are refused as bad arguments, before any launch. (The tensors are
broadcast: no memory of that size is held.)"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import _binding as fb  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def test_more_rows_than_a_call_takes():
    ctx = fq.qc_create("int8", 64, 1024, 16)
    pages = fq.alloc_pages(ctx, 1)
    x = torch.zeros((1, 1024, 64), dtype=torch.float16, device="cuda")
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    L, n = fb.lib(), 2 ** 38
    at = x.data_ptr()
    assert L.qc_write(ctx, 0, n, at, 0, 64, at, 0, 64, slot.data_ptr(), pages.data_ptr(), 1, None) == fb.FQ_EINVAL
    assert L.qc_read(ctx, 0, n, slot.data_ptr(), pages.data_ptr(), 1, at, at, None) == fb.FQ_EINVAL
    assert L.qc_norm_rope(ctx, 0, n, at, 1, 0, 64, None, None, 0, 0, 0, None, 0.0, None, None, 0, 0, 0, at, 0, 64, None, 0, 0,
                          None) == fb.FQ_EINVAL
    torch.cuda.synchronize()
    assert fq.qc_status(ctx) == 0
    fq.qc_destroy(ctx)
