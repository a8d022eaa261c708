"""The paged cache's C ABI without a GPU: null contexts and the host-side checks that come before any device work."""
import ctypes

import pytest

from random_access_kv_gb300 import _binding as fb
from random_access_kv_gb300 import build as fbuild


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fb.lib()


def test_null_context(L):
    assert L.qc_page_bytes(None) == -1
    assert L.qc_attend_workspace(None, 1, 1, 1, 1) == -1
    assert L.qc_norm_rope(None, 0, 1, None, 1, 0, 0, None, None, 0, 0, 0, None, 0.0, None, None, 0, 0, 0, None, 0, 0, None, 0, 0,
                          None) == fb.FQ_EINVAL
    assert L.qc_write(None, 0, 1, None, 0, 0, None, 0, 0, None, None, 1, None) == fb.FQ_EINVAL
    assert L.qc_read(None, 0, 1, None, None, 1, None, None, None) == fb.FQ_EINVAL
    assert L.qc_attend(None, 0, 1, 1, 1, None, 0, 0, 0, None, 0, None, None, None, None, 1, 1.0, 1, None, None, None, 0,
                       None) == fb.FQ_EINVAL
    assert L.qc_status(None, None, None) == fb.FQ_EINVAL
    L.qc_destroy(None)


@pytest.mark.parametrize("fmt,d,heads,page", [(-1, 64, 1, 16), (3, 64, 1, 16), (0, 96, 1, 16), (0, 64, 0, 16), (0, 64, 1025, 16),
                                              (0, 64, 1, 8), (0, 64, 1, 48), (0, 64, 1, 512)])
def test_create_rejects_unsupported_geometry(L, fmt, d, heads, page):
    h = ctypes.c_void_p()
    assert L.qc_create(ctypes.byref(h), fmt, d, heads, page, 0) == fb.FQ_EINVAL and not h.value
    assert L.qc_create(None, 0, 64, 1, 16, 0) == fb.FQ_EINVAL


def test_create_without_gpu_reports_no_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(fb.FQError) as e:
        fb.qc_create("int8", 64, 2, 16)
    assert e.value.code == fb.FQ_ENODEV
