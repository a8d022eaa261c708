"""qc_verify where probabilities are no probabilities: rows that sum to far more or far less than 1, and what a sum past float32's
range gives. Against the oracle's exact fractions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import random_access_kv_gb300 as fq  # noqa: E402
from oracle import qcache as oq  # noqa: E402
from random_access_kv_gb300 import build as fbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    fbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def call(p, q, tokens, u):
    n_seq, t, vocab = q.shape
    ctx = fq.qc_create("int8", 64, 1, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    path, out, came = (torch.full(s, -9, **i32) for s in ((n_seq, t), (n_seq, t + 1), (n_seq,)))
    # all nodes are the prefix' children: one after the other is asked
    fq.qc_verify(ctx, p, q, torch.tensor(tokens, **i32), torch.full((n_seq, t), -1, **i32), None, u, path, out, came)
    flags = fq.qc_status(ctx)
    ctx.close()
    return path, out, came, flags


@pytest.mark.parametrize("up", [-140, -120, -60, 0, 60, 120])
@pytest.mark.parametrize("vocab", [5, 257, 4000])
def test_rows_of_any_sum(up, vocab):
    n_seq, t = 6, 3
    r = np.random.default_rng([vocab, up + 200])
    p, q = (torch.from_numpy((r.dirichlet(np.ones(vocab), (n_seq, n)) * 2.0 ** up).astype(np.float32)).cuda() for n in (t + 1, t))
    if up > 0:
        q = q * 2.0 ** -up                                    # so that not everything is rejected
    tokens, u = r.integers(0, vocab, (n_seq, t)), torch.from_numpy(r.random((n_seq, t + 1)).astype(np.float32)).cuda()
    path, out, came, flags = call(p, q, tokens, u)
    assert flags == 0
    for b in range(n_seq):
        stand, last = oq.verify(p[b].double().cpu().numpy(), q[b].double().cpu().numpy(), tokens[b], [-1] * t, t, u[b].tolist())
        assert int(came[b]) == len(stand) and path[b, :len(stand)].tolist() == stand
        assert out[b, :len(stand) + 1].tolist() == [tokens[b][c] for c in stand] + [last]


def test_a_sum_past_the_range_is_told():
    p = torch.full((1, 2, 40), 3e38, device="cuda")
    q = torch.full((1, 1, 40), 1e38, device="cuda")
    path, out, came, flags = call(p, q, [[3]], torch.tensor([[0.5, 0.5]], device="cuda"))
    assert int(came) == 1 and path.tolist() == [[0]] and out[0, 0] == 3      # 0.5 * 1e38 < 3e38: accepted
    assert int(out[0, 1]) == -1 and flags == fq.QC_FLAG_RANGE                 # the row after it cannot be drawn from
