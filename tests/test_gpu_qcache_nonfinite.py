"""Queries that are not finite, in the paged cache's attention: a row with a NaN or an infinity that sees a place gives NaN
and a log-sum of NaN, however its work is divided; one that sees nothing, or whose node is not there, gives zeros and
minus infinity; the other rows are as they are without it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# few rows (up to 32 per key/value head) and many, from 1,024 places on; within one run of tiles and over several
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("t,group", [(3, 2), (12, 4), (34, 4)])
@pytest.mark.parametrize("lens", [[20, 0], [3001, 0]], ids=["whole", "split"])
def test_queries_that_are_not_finite(kind, t, group, lens):
    import qcache_cases as qc
    heads, d = 2, 64
    case = qc.random_case("int8", d, heads, 32, lens, [t - 1, t], t, 3001)
    q = qc.rows((2, t, heads * group, d), 3, qc.TYPES[kind][0])
    sees = qc.chain(2, t)
    sees[1, 0] = False                                   # a row that sees nothing
    poison = [(0, 0, 0, 5, "nan"), (0, 1, 1, 0, "inf"), (0, 1, 3, 63, "-inf"), (1, 1, 2, 8, "inf"), (1, 2, 0, 1, "nan"),
              (0, t - 1, 1, 2, "nan"), (1, 0, 0, 0, "inf")]       # the last two: no such node, nothing seen
    for b, i, h, j, what in poison:
        q[b, i, h, j] = float(what)
    out, lse = case.call(q, sees)
    assert fq.qc_status(case.ctx) == 0
    for b, i, h, _, what in poison[:5]:
        assert torch.isnan(out[b, i, h]).all() and torch.isnan(lse[b, i, h]), (b, i, h, what)
    for b, i, h, _, what in poison[5:]:
        assert (out[b, i, h] == 0).all() and lse[b, i, h] == -np.inf, (b, i, h, what)
    clean = q.clone()
    for b, i, h, _, _ in poison:
        clean[b, i, h] = 0
    hit = {(b, i, h) for b, i, h, _, _ in poison}
    for h in range(heads * group):
        skip = {(b, i) for b, i, g in hit if g == h}
        case.check(clean, out, lse, sees, heads=[h], skip=skip)


@pytest.mark.parametrize("t", [2, 40])
def test_scores_beyond_float32_are_not_silent(t):
    import qcache_cases as qc
    K = [torch.full((1100 + t, 1, 64), 2.0 ** 60, device="cuda")]
    V = [qc.rows((1100 + t, 1, 64), 4)]
    case = qc.Case("e4m3", 64, 1, 16, K, V, [1100], None, t)
    q = torch.full((1, t, 1, 64), 2.0 ** 70, dtype=torch.bfloat16, device="cuda")
    q[:, 0] = 0
    out, lse = case.call(q, scale=1.0)
    assert torch.isnan(out[:, 1:]).all() and torch.isnan(lse[:, 1:]).all()
    case.check(q, out, lse, scale=1.0, skip={(0, i) for i in range(1, t)})
