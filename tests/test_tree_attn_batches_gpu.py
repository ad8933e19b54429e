"""A row of gdr_tree_attn beside other rows: where its item is cut over blocks follows from all rows' units, so
its bits may change with the batch, but alone and beside any others it stays within the bound of the float64
form, and the same call always gives the same bits."""
import math

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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx", [70, 640, 9000])   # a tile of both; tiles of their own, each a part; an item cut over many blocks
def test_a_seen_infinity_of_vanishing_weight(ctx, D):
    """A node's V holds infinities and a nan; its weight against the context's is below the smallest float."""
    c = _case(1, 4, 4, 2, D, 64, [ctx], "tree", seed=D)
    c["see"][0] = torch.eye(4, dtype=torch.bool)
    c["see"][0, 3, 2] = True
    at = ctx + torch.arange(4)
    pages = c["table"][0].long()[at // 64]
    c["q"][:] = 8
    c["k"][pages, at % 64] = -8                       # the nodes' scores: -64 D^1/2, at most -512
    c["v"][pages[2], at[2] % 64, :, 5] = math.inf
    c["v"][pages[2], at[2] % 64, :, 6] = -math.inf
    c["v"][pages[2], at[2] % 64, :, 37] = math.nan
    o, lse = _run(c)
    rows = torch.tensor([2, 3])
    assert (o[0, rows, :, 5] == math.inf).all() and (o[0, rows, :, 6] == -math.inf).all() and torch.isnan(o[0, rows, :, 37]).all()
    rest = torch.ones(D, dtype=torch.bool)
    rest[[5, 6, 37]] = False
    assert torch.isfinite(o[0, :2]).all() and torch.isfinite(o[..., rest]).all() and torch.isfinite(lse).all()
