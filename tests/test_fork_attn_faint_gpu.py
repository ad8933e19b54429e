"""gdr_fork_attn: what is not finite in a seen position reaches the output however small its weight, where the weight is a
product of small ones (a warp's part among the row's own positions, and these beside the shared ones)."""
import math

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("M", [4, 64])              # (short rows in one kernel, or the shared positions by themselves)
@pytest.mark.parametrize("N,G", [(1, 1), (1, 8), (1, 16), (3, 5), (2, 16), (8, 8), (5, 16)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_that_vanish_as_a_product(D, N, G, M, bad):
    """Scores (natural logarithms): 0 in the shared positions, -70 in the first of the own ones and in the nodes, -150 in the
    others: e^-70 and e^-80 are floats, e^-150 is not."""
    page, B, own = 64, 3, 128
    pages = 1 + B * (own // page + 1)
    table = torch.full((B, M), -1, dtype=torch.int32)
    table[:, 0] = 0
    table[:, 1:4] = torch.arange(1, pages, dtype=torch.int32).view(B, 3)
    k = torch.zeros(pages, page, 1, D)
    k[1:, ..., 0] = -150
    k[1::3, :16, :, 0] = -70
    k[3::3, :N, :, 0] = -70                          # (the nodes)
    v = torch.randn(pages, page, 1, D, generator=torch.Generator().manual_seed(D + N))
    q = torch.zeros(B, N, G, D)
    q[..., 0] = 1
    places = {0: (0, 5), 1: (4, 20), 2: (8, 50)}     # row b's: a shared position (all rows see it), own ones of small weight
    for b, (pg, at) in places.items():
        v[pg, at, 0, 7 + b] = bad
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    bf = lambda t: t.cuda().bfloat16()   # noqa: E731
    o = gdr.gdr_fork_attn(bf(q), bf(k), bf(v), table.cuda(), i32([page + own] * B), i32([0, B]), i32([page]), scale=1.0)
    gdr.gdr_sync_status()
    want = torch.zeros(B, D, dtype=torch.bool)
    want[:, 7] = True
    want[1, 8] = want[2, 9] = True
    assert torch.equal(~torch.isfinite(o).cpu(), want[:, None, None].expand(B, N, G, D))
