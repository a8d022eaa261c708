"""A workspace of the paged cache's attention serves every call of up to the sizes that it was asked for."""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("d,heads", [(64, 1), (64, 8), (128, 8), (128, 1)])
def test_smaller_calls_want_no_more(fmt, d, heads):
    ctx = fq.qc_create(fmt, d, heads, 32)
    seqs, nodes, groups = (0, 1, 2, 8, 33, 300), (1, 5, 8, 16, 24, 25, 31, 32, 33, 64, 65, 130, 300), (1, 2, 4, 16)
    lens = (0, 1, 100, 900, 990, 991, 992, 1000, 1022, 1023, 1024, 5000, 16384, 100000)
    want = {}
    for s, n, g, m in itertools.product(range(len(seqs)), range(len(nodes)), range(len(groups)), range(len(lens))):
        b = want[s, n, g, m] = fq.qc_attend_workspace(ctx, seqs[s], nodes[n], groups[g] * heads, lens[m])
        for i in range(4):                                   # one step less in each size
            at = [s, n, g, m]
            at[i] -= 1
            if at[i] >= 0:
                assert want[tuple(at)] <= b, (seqs[s], nodes[n], groups[g], lens[m], i)
    fq.qc_destroy(ctx)


@pytest.mark.parametrize("d", [64, 128])
def test_one_workspace_serves_both_kernels(d):
    import qcache_cases as qc
    heads, group = 2, 4
    sizes = [(2, 40, [1500, 900]), (2, 6, [1500, 900]), (2, 8, [1500, 3]), (2, 9, [1014, 20]), (2, 9, [1015, 20]), (1, 40, [900]), (1, 1, [1500]),
             (1, 1, [0])]
    ws = None
    for i, (n_seq, t, lens) in enumerate(sizes):
        case = qc.random_case("int8", d, heads, 16, lens, None, t, seed=i)
        if ws is None:
            ws = fq.alloc_attend_workspace(case.ctx, n_seq, t, heads * group, case.max_len)
        q = qc.rows((n_seq, t, heads * group, d), i, torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((n_seq, t, heads * group), device="cuda")
        fq.qc_attend(case.ctx, case.pages, q, torch.from_numpy(case.table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), None,
                     None, d ** -0.5, case.max_len, out, lse, ws)
        case.check(q, out, lse)
    assert fq.qc_status(case.ctx) == 0
