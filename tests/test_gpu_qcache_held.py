"""qc_plan where free pages run out and requests say what they hold, against the oracle (pinned by
tests/test_oracle_qcache_held.py): a page that was wanting is not held, and a second try asks for it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from oracle import qcache as oq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402
from test_oracle_qcache_held import CASES, tables, width_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def both(page, lens, news, held, free, table):
    """The kernel's and the oracle's plan are equal; returns the oracle's table, slots and held."""
    ctx = fq.qc_create("int8", 64, 1, page)
    n = sum(news)
    now = list(held)
    want = oq.plan(lens, news, free, 0, table, n, page, now)
    t, starts, held_out = i32(table), i32(np.zeros(len(lens) + 1)), i32(np.full(len(lens), -9))
    slots, pos = (torch.full((n,), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    took = torch.full((1,), -9, dtype=torch.int64, device="cuda")
    fq.qc_plan(ctx, i32(lens), i32(news), i32(free), torch.zeros_like(took), t, starts, slots, pos, took, i32(held), held_out)
    flags = fq.qc_status(ctx)
    for got, w in ((t, want[0]), (starts, want[1]), (slots, want[2]), (pos, want[3]), (held_out, now)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert int(took) == want[4] and flags == (fq.QC_FLAG_PAGES if want[5] else 0) and not want[6]
    ctx.close()
    return want[0], want[2], now


@pytest.mark.parametrize("page,lens,news,held,n_free", CASES)
def test_pages_run_out_and_come_in(page, lens, news, held, n_free):
    table = tables(lens, held, width_of(page, lens, news))
    table, slots, now = both(page, lens, news, held, np.arange(n_free), table)
    assert (slots == -1).any()
    table, slots, now = both(page, lens, news, now, np.arange(n_free, n_free + 2), table)     # some come in
    table, slots, now = both(page, lens, news, now, np.arange(n_free + 2, 500), table)        # and the rest
    assert (slots >= 0).all()


def test_many_requests_that_run_out():
    r = np.random.default_rng(0)
    lens, news = r.integers(0, 100, 3000).tolist(), r.integers(0, 40, 3000).tolist()
    held = [-(-a // 16) + int(x) for a, x in zip(lens, r.integers(0, 2, 3000))]
    table = tables(lens, held, 10)
    for n_free in (0, 1, 777, 2000):
        both(16, lens, news, held, np.arange(n_free), table)
