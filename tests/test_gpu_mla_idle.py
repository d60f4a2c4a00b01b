"""Requests that a step adds nothing to need no row, page or slot: they are
served, whatever room the others lack."""
import pytest

from oracle import attention as A

CASES = [([0, 5, 9], [3, 0, 0], 16, [[1], [2], [3]], [7, 8], 2, 2),           # behind rows that are not there
         ([40, 5], [0, 1], 16, [[1, 2], [3, 4]], [7], 1, 4),                  # as long as its table, and longer
         ([4, 0, 2], [0, 20, 0], 4, [[1], [2], [3]], [], 0, 30)]              # behind a request that finds no page
FAILED = [1, 0, 1]


@pytest.mark.parametrize("case,failed", zip(CASES, FAILED))
def test_oracle(case, failed):
    old, new, page, table, free, n_free, N = case
    got = A.pages_extend(old, new, page, table, free, n_free, N)
    assert got[3] == failed
    assert got[1] == [a + b if b and not failed else a for a, b in zip(old, new)]


@pytest.mark.gpu
@pytest.mark.parametrize("case,failed", zip(CASES, FAILED))
@pytest.mark.parametrize("more", [0, 5000])
def test_kernel(case, failed, more):
    """Alone, and with more idle requests than one block places (two launches)."""
    from test_gpu_mla_decode import extend
    old, new, page, table, free, n_free, N = case
    old, new, table = old + [3] * more, new + [0] * more, table + [[5] * len(table[0])] * more
    got = extend(old, new, page, table, free, n_free, N)
    assert got[3] == failed
    assert tuple(got) == tuple(A.pages_extend(old, new, page, table, free, n_free, N))
