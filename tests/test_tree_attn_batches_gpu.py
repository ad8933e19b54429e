"""A row of gdr_tree_attn beside other rows: where its item is cut over blocks follows from all rows' units, so
its bits may change with the batch, but alone and beside any others it stays within the bound of the float64
form, and the same call always gives the same bits."""
import pytest
import torch

from tests.test_tree_attn_gpu import _case, _check, _run

pytestmark = pytest.mark.gpu


def _rows(c, rows):
    """The case of these rows alone (the pages stay as they are)."""
    return {n: t[rows] if n in ("q", "table", "ctx", "lengths", "see") else t for n, t in c.items()}


@pytest.mark.parametrize("D,N", [(64, 9), (128, 9), (128, 70), (256, 9)])
def test_a_row_alone_and_beside_others(D, N):
    c = _case(5, N, 8, 2, D, 32, [700, 64, 1500, 3, 5000], "tree", seed=D + N)
    whole = _run(c)
    _check(c, *whole)
    for rows in ([0], [2, 0], [0, 1, 2, 3], [4, 3, 2, 1, 0]):
        part = _rows(c, rows)
        got = _run(part)
        _check(part, *got)
        again = _run(part)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
