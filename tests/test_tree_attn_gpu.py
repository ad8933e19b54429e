"""gdr_tree_attn against float64 over the seen positions alone.

Tolerances: a softmax weight is rounded to bf16 (2^-8 relative), its score is off by at most
(D + 8) 2^-22 of E = max_j scale sum |q k| (float32 sums in the tensor core, which may drop rather than
round) and the exponential by 2^-21; the same score error sits in the sum l. So o is off by at most
(2^-8 + 2 e) A + 2^-8 |o| with A = sum p |v| and e = (D + 8) 2^-22 E + 2^-19, and lse by
e + 2^-22 (1 + |lse| + E)."""
import math

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def _pack(see):
    B, N, _ = see.shape
    W = (N + 63) // 64
    full = torch.zeros(B, N, W * 64, dtype=torch.int64)
    full[..., :N] = see.long()
    return (full.view(B, N, W, 64) << torch.arange(64)).sum(-1)


def _see(kind, B, N, g):
    i = torch.arange(N)
    if kind == "chain":
        return (i[None, :] <= i[:, None]).expand(B, N, N).clone()
    if kind == "random":   # any mask at all, rows that see nothing among them
        see = torch.rand(B, N, N, generator=g) < 0.4
        see[:, ::3] = False
        return see
    see = torch.zeros(B, N, N, dtype=torch.bool)
    for b in range(B):
        for n in range(N):
            if n:
                see[b, n] = see[b, int(torch.randint(max(0, n - 5), n, (1,), generator=g))]
            see[b, n, n] = True
    return see


def _case(B, N, Hq, Hk, D, page, ctx, kind, seed=0, lengths=None, spare=2, qs=1.5, M=None):
    g = torch.Generator().manual_seed(seed)
    ctx = torch.tensor([ctx[b % len(ctx)] for b in range(B)], dtype=torch.int32)
    lengths = torch.tensor([N] * B if lengths is None else [lengths[b % len(lengths)] for b in range(B)], dtype=torch.int32)
    need = [-(-(int(c) + N) // page) for c in ctx]
    P, M = sum(need) + spare, M or max(need)
    order = torch.randperm(P, generator=g).int()
    table = torch.full((B, M), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = (qs * torch.randn(B, N, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(P, page, Hk, D, generator=g).bfloat16() for _ in "kv")
    return dict(q=q, k=k, v=v, table=table, ctx=ctx, lengths=lengths, see=_see(kind, B, N, g), kind=kind, scale=D ** -0.5)


def _run(c, with_lengths=True, mask=None):
    d = {n: c[n].cuda() for n in ("q", "k", "v", "table", "ctx", "lengths")}
    if mask is None and c["kind"] != "chain":
        mask = _pack(c["see"]).cuda()
    o, lse = gdr.gdr_tree_attn(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["lengths"] if with_lengths else None, mask,
                               scale=c["scale"], want_lse=True)
    gdr.gdr_sync_status()
    return o.double().cpu(), lse.double().cpu()


def _check(c, o, lse):
    D = c["q"].shape[-1]
    wo, wl, A, E = ref.tree_attn(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["lengths"], c["see"], c["scale"])
    e = (D + 8) * 2.0 ** -22 * E + 2.0 ** -19
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (o[empty] == 0).all()
    off = (o - wo).abs() - ((2.0 ** -8 + 2 * e[..., None]) * A + 2.0 ** -8 * wo.abs())
    assert torch.isfinite(o).all() and off.max() <= 0, f"o off by {off.max():.3e} over the bound"
    loff = (lse - wl).abs() - (e + 2.0 ** -22 * (1 + wl.abs() + E))
    assert loff[~empty].numel() == 0 or loff[~empty].max() <= 0, f"lse off by {loff[~empty].max():.3e} over the bound"


CASES = [
    (1, 1, 1, 1, 128, 64, [0]), (1, 1, 4, 2, 128, 64, [130]), (2, 1, 8, 1, 64, 16, [1, 127]), (1, 1, 16, 2, 256, 32, [300]),
    (3, 2, 6, 2, 128, 16, [0, 128, 15]), (2, 17, 5, 1, 64, 128, [200, 3]), (4, 13, 8, 4, 128, 64, [64, 63, 65, 1000]),
    (2, 64, 8, 2, 128, 32, [500, 0]), (2, 65, 3, 1, 256, 64, [31, 129]), (1, 100, 6, 3, 64, 16, [77]),
    (2, 130, 8, 1, 128, 128, [250, 6]), (1, 7, 128, 1, 128, 64, [150]), (1, 3, 40, 8, 256, 128, [1100]),
]


@pytest.mark.parametrize("kind", ["chain", "tree", "random"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, kind):
    c = _case(*case, kind, seed=sum(case[:6]))
    _check(c, *_run(c))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_ragged_lengths(kind, D):
    """Rows of no nodes, one, some, all; padded nodes give 0 and -inf."""
    c = _case(6, 20, 4, 2, D, 16, [100, 0, 300, 5, 700, 64], kind, seed=D, lengths=[0, 1, 20, 7, 13, 19])
    _check(c, *_run(c))


def test_many_rows():
    """More rows than threads of a block, and more items than blocks."""
    c = _case(500, 2, 4, 2, 64, 16, [0, 40, 3, 129, 17], "tree", seed=3, lengths=[2, 1, 0, 2])
    _check(c, *_run(c))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_long_context_is_split_over_blocks(D, page):
    c = _case(1, 3, 4, 2, D, page, [30011], "tree", seed=5)
    _check(c, *_run(c))


@pytest.mark.parametrize("B,N,Hq,Hk,D,seed", [(40, 2, 5, 5, 64, 0), (40, 2, 5, 5, 64, 1), (40, 1, 10, 5, 128, 2), (7, 2, 6, 3, 128, 3),
                                              (31, 1, 5, 5, 256, 4), (9, 20, 10, 1, 64, 5), (60, 70, 6, 3, 64, 6)])
def test_shares_begin_anywhere(B, N, Hq, Hk, D, seed):
    """Items of all lengths, more and fewer than blocks: shares begin and end inside items, at their ends and
    between them."""
    g = torch.Generator().manual_seed(seed)
    most = 2500 if N < 20 else 900
    ctx = (most * torch.rand(B, generator=g) ** 2).int().tolist()
    c = _case(B, N, Hq, Hk, D, 16, ctx, "tree", seed=seed, lengths=[N, N, max(1, N // 2)])
    _check(c, *_run(c))


def test_chain_of_many_nodes_is_a_prefill():
    c = _case(2, 300, 4, 2, 128, 64, [0, 77], "chain", seed=6, lengths=[300, 211])
    _check(c, *_run(c))


def test_rising_scores():
    """The maximum grows at every tile, far past the reference's slack, and once falls."""
    for D in (64, 128, 256):
        c = _case(1, 5, 4, 1, D, 16, [1500], "tree", seed=7)
        at = torch.arange(1505)
        size = (0.02 * at).clamp(max=25)
        size[700:900] = 0.1
        pages = c["table"][0].long()[at // 16]
        c["k"][pages, at % 16] = (c["q"][0, 0, 0].float() / 4 * size[:, None, None] / 8).bfloat16()
        _check(c, *_run(c))


def test_large_scores():
    c = _case(2, 9, 8, 2, 128, 32, [400, 130], "tree", seed=8, qs=40.0)
    _check(c, *_run(c))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_places_do_not_matter(D, bad):
    """Free pages, positions past a row's nodes and nodes that a row does not see hold nan, inf or the
    type's lowest values; rows that see none of them are untouched, bit for bit."""
    c = _case(3, 12, 4, 2, D, 16, [0, 50, 200], "tree", seed=9, lengths=[12, 5, 9])
    c["see"][:, 1:] &= ~torch.tensor([j == 3 for j in range(12)])   # node 3 is seen by itself and row 0's node 0 alone
    c["see"][:, 3, 3] = True
    clean_o, clean_lse = _run(c)
    _check(c, clean_o, clean_lse)
    used = torch.zeros(c["k"].shape[:2], dtype=torch.bool)
    for b in range(3):
        at = torch.arange(int(c["ctx"][b] + c["lengths"][b]))
        used[c["table"][b].long()[at // 16], at % 16] = True
        e = int(c["ctx"][b]) + 3
        used[int(c["table"][b, e // 16]), e % 16] = False            # node 3
    c["k"][~used], c["v"][~used] = bad, bad
    o, lse = _run(c)
    rows = ~c["see"][..., 3] | (torch.arange(12) >= c["lengths"][:, None])
    assert torch.equal(o[rows], clean_o[rows]) and torch.equal(lse[rows], clean_lse[rows])


@pytest.mark.parametrize("long", [False, True])
def test_seen_infinities_reach_their_rows(long):
    """A node's V holds +inf, -inf and nan: exactly the rows that see it get them (also in a part of an
    item that several blocks share)."""
    c = _case(1, 6, 4, 2, 128, 64, [9000 if long else 70], "tree", seed=10)
    c["see"][0] = torch.eye(6, dtype=torch.bool)
    c["see"][0, 4, 2] = c["see"][0, 5, 2] = c["see"][0, 5, 3] = True
    at = int(c["ctx"][0]) + torch.arange(6)
    pages = c["table"][0].long()[at // 64]
    c["v"][pages[2], at[2] % 64, :, 5] = math.inf
    c["v"][pages[2], at[2] % 64, 1, 70] = math.nan
    c["v"][pages[3], at[3] % 64, :, 5] = -math.inf
    o, _ = _run(c)
    want, _, _, _ = ref.tree_attn(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["lengths"], c["see"], c["scale"])
    assert torch.equal(torch.isnan(o), torch.isnan(want)) and torch.equal(torch.isinf(o), torch.isinf(want))
    assert torch.equal(o[torch.isinf(o)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    assert (o[fine] - want[fine]).abs().max() < 0.05


def test_results_do_not_depend_on_the_batch_or_the_run():
    c = _case(3, 9, 8, 2, 128, 32, [700, 64, 1500], "tree", seed=11)
    a, la = _run(c)
    b, lb = _run(c)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_rows_and_pages():
    c = _case(4, 3, 4, 2, 128, 16, [40, 40, 40, 40], "tree", seed=12)
    good, _ = _run(c)
    c["ctx"][1], c["lengths"][2] = 1000, 4
    c["table"][3, 1] = 10 ** 6
    d = {n: c[n].cuda() for n in ("q", "k", "v", "table", "ctx", "lengths")}
    o, lse = gdr.gdr_tree_attn(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["lengths"], _pack(c["see"]).cuda(), want_lse=True)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    assert torch.allclose(o[0].double().cpu(), good[0], atol=0.02)
    assert (o[1:3] == 0).all() and (lse[1:3] == -math.inf).all() and torch.isfinite(o[3].float()).all()
    c["table"][3, 1] = -1
    gdr.gdr_tree_attn(d["q"], d["k"], d["v"], c["table"].cuda(), d["ctx"], d["lengths"], _pack(c["see"]).cuda())
    with pytest.raises(gdr.GdrError):
        gdr.gdr_sync_status()


def test_pages_past_32_bits():
    """The row's pages are the pool's last, past 2^32 bytes."""
    P, page, Hk, D = 66000, 16, 16, 128
    c = _case(1, 3, 32, Hk, D, page, [37], "tree", seed=13)
    n = c["table"].shape[1]
    k = torch.empty(P, page, Hk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[P - n:], v[P - n:] = c["k"][c["table"][0].long()].cuda(), c["v"][c["table"][0].long()].cuda()
    table = torch.arange(P - n, P, dtype=torch.int32, device="cuda")[None]
    o, lse = gdr.gdr_tree_attn(c["q"].cuda(), k, v, table, c["ctx"].cuda(), None, _pack(c["see"]).cuda(), want_lse=True)
    gdr.gdr_sync_status()
    _check(c, o.double().cpu(), lse.double().cpu())


def test_on_another_stream_and_in_a_graph():
    c = _case(2, 5, 8, 2, 128, 64, [900, 33], "tree", seed=14)
    want, _ = _run(c)
    d = {n: c[n].cuda() for n in ("q", "k", "v", "table", "ctx", "lengths")}
    mask, o = _pack(c["see"]).cuda(), torch.empty_like(d["q"])
    ws = torch.empty(gdr.tree_attn_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    call = lambda: gdr.gdr_tree_attn(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["lengths"], mask, o=o, ws=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(o.double().cpu(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    o.zero_()
    d["ctx"][1] = 20   # the graph reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    c["ctx"][1] = 20
    assert torch.equal(o.double().cpu(), _run(c)[0])


def test_waits_that_run_out_are_reported():
    c = _case(2, 5, 8, 2, 128, 64, [900, 33], "tree", seed=15)
    want, _ = _run(c)
    d = {n: c[n].cuda() for n in ("q", "k", "v", "table", "ctx", "lengths")}
    gdr.debug_set_wait_budget(0)
    try:
        gdr.gdr_tree_attn(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["lengths"], _pack(c["see"]).cuda())
        with pytest.raises(gdr.GdrError) as e:
            gdr.gdr_sync_status()
        assert e.value.status == gdr.GDR_ERR_TIMEOUT
    finally:
        gdr.debug_set_wait_budget(-1)
    assert torch.equal(_run(c)[0], want)
