"""The paged cache's operators together, as examples/draft_step.py runs them: every format steps through, sequences
grow by what is accepted, and a moved row keeps its values (a row read from the cache and written back is held
to within one rounding of its scale)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
def test_draft_steps(fmt):
    import draft_step
    lens, out, lse = draft_step.run(fmt, steps=3, sequences=3)
    assert ((lens > 300) & (lens <= 300 + 3 * 4)).all()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and out.abs().max() > 0
    again, out2, lse2 = draft_step.run(fmt, steps=3, sequences=3)
    assert torch.equal(lens, again) and torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
def test_rows_moved_within_the_cache(fmt):
    # a row's codes are those of its own values: read as float32 and written again, each value moves by at most
    # two roundings of float32 (the scale found anew, and the product)
    ctx = fq.qc_create(fmt, 128, 2, 16)
    pages = fq.alloc_pages(ctx, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((20, 2, 128), generator=g, device="cuda") for _ in range(2))
    a, b = torch.arange(20, device="cuda"), 30 + torch.arange(20, device="cuda")
    fq.qc_write(ctx, k, v, a, pages)
    held = [torch.empty_like(k) for _ in range(2)]
    fq.qc_read(ctx, pages, a, *held)
    fq.qc_write(ctx, *held, b, pages)
    moved = [torch.empty_like(k) for _ in range(2)]
    fq.qc_read(ctx, pages, b, *moved)
    assert fq.qc_status(ctx) == 0
    for x, y in zip(held, moved):
        assert ((x - y).abs() <= 2 * 2.0 ** -23 * x.abs()).all()
    ctx.close()
