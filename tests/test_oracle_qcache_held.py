"""The oracle's plan where free pages run out and requests say what they hold: a page that was wanting is not held, and is asked
for again. The cases are run on the GPU by tests/test_gpu_qcache_held.py."""
import numpy as np
import pytest

from oracle import qcache as oq

# page, lens, news, held, free pages of the first try
CASES = [
    (16, [20, 33, 0, 16, 5, 40], [40, 3, 20, 1, 1, 40], [2, 5, 0, 1, 1, 3], 4),
    (16, [0, 0, 0], [16, 33, 5], [0, 0, 0], 0),
    (16, [0, 0, 0], [16, 33, 5], [0, 0, 0], 2),
    (32, [31, 64, 7], [200, 1, 26], [1, 2, 1], 6),
    (64, [100] * 40, [1 + 70 * (b % 3) for b in range(40)], [2 + b % 2 for b in range(40)], 11),
]


def tables(lens, held, width):
    """Each request's held pages are its own, the rest of its row is -1."""
    table = np.full((len(lens), width), -1, np.int64)
    table[:] = np.where(np.arange(width) < np.array(held)[:, None], 1000 + np.arange(len(lens) * width).reshape(-1, width), -1)
    return table


def width_of(page, lens, news):
    return max(-(-(a + b) // page) for a, b in zip(lens, news))


@pytest.mark.parametrize("page,lens,news,held,n_free", CASES)
def test_what_was_wanting_is_not_held(page, lens, news, held, n_free):
    table = tables(lens, held, width_of(page, lens, news))
    first = list(held)
    got, starts, slots, pos, taken, lack, odd = oq.plan(lens, news, np.arange(n_free), 0, table, sum(news), page, first)
    assert lack and not odd and taken == n_free and sum(first) - sum(held) == n_free
    for b, n in enumerate(first):
        assert (got[b, :n] >= 0).all()                        # what is held is there
        assert (got[b, n:] == -1).all()
    # a second try of the same step with all that is wanting gets it, and no page twice
    again = list(first)
    want, starts2, slots2, _, taken2, lack, odd = oq.plan(lens, news, np.arange(n_free, 1000), 0, got, sum(news), page, again)
    assert not lack and not odd and np.array_equal(starts, starts2)
    assert (slots2 >= 0).all() and len(set(slots2.tolist())) == len(slots2)
    assert all(n == max(h, -(-(a + t) // page)) for n, h, a, t in zip(again, held, lens, news))
    pages = np.concatenate([want[b, :n] for b, n in enumerate(again)])
    assert len(set(pages.tolist())) == len(pages)
    # tokens that had a slot in the first try keep it
    assert np.array_equal(slots2[slots >= 0], slots[slots >= 0])
