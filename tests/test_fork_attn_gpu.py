"""gdr_fork_attn against float64 over the seen positions alone, row by row.

Tolerances as for gdr_tree_attn: a softmax weight is rounded to bf16 (2^-8 relative), its score is off by at most
(D + 8) 2^-22 of E = max_j scale sum |q k| and the exponential by 2^-21; the same score error sits in the sum. The
two parts' weights add less than 2^-20 of A = sum p |v|. So o is off by at most (2^-8 + 2 e) A + 2^-8 |o| with
e = (D + 8) 2^-22 E + 2^-19, and lse by e + 2^-22 (1 + |lse| + E)."""
import math

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


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
    see = torch.rand(B, N, N, generator=g) < 0.4   # any mask at all, nodes that see no node among them
    see[:, ::3] = False
    return see


def _case(first, shared, own, N, Hq, Hk, D, page, kind="chain", seed=0, lengths=None, qs=1.5):
    """first, shared: the groups; own: own positions of the rows, by turns."""
    g = torch.Generator().manual_seed(seed)
    B = max(first[-1], 1)
    group = [next((t for t in range(len(shared)) if first[t] <= b < first[t + 1]), -1) for b in range(B)]
    sh = [shared[t] if t >= 0 else 0 for t in group]
    own = [own[b % len(own)] for b in range(B)]
    ctx = torch.tensor([s + o for s, o in zip(sh, own)], dtype=I32)
    lengths = torch.tensor([N] * B if lengths is None else [lengths[b % len(lengths)] for b in range(B)], dtype=I32)
    need = [-(-(o + N) // page) for o in own]
    P, M = sum(shared) // page + sum(need) + 2, max(s // page + n for s, n in zip(sh, need))
    order = torch.randperm(P, generator=g).int().tolist()
    trunk = [[order.pop() for _ in range(s // page)] for s in shared]
    table = torch.full((B, M), -1, dtype=I32)
    for b in range(B):
        row = (trunk[group[b]] if group[b] >= 0 else []) + [order.pop() for _ in range(need[b])]
        table[b, :len(row)] = torch.tensor(row, dtype=I32)
    q = (qs * torch.randn(B, N, Hq, D, generator=g)).bfloat16()
    k, v = (torch.randn(P, page, Hk, D, generator=g).bfloat16() for _ in "kv")
    return dict(q=q, k=k, v=v, table=table, ctx=ctx, lengths=lengths, see=_see(kind, B, N, g), kind=kind, scale=D ** -0.5,
                first=torch.tensor(first, dtype=I32), shared=torch.tensor(shared, dtype=I32))


def _args(c):
    d = {n: c[n].cuda() for n in ("q", "k", "v", "table", "ctx", "first", "shared", "lengths")}
    return (*d.values(), _pack(c["see"]).cuda() if c["kind"] != "chain" else None, c["scale"])


def _run(c):
    o, lse = gdr.gdr_fork_attn(*_args(c), want_lse=True)
    gdr.gdr_sync_status()
    return o.double().cpu(), lse.double().cpu()


def _check(c, o=None, lse=None):
    if o is None:
        o, lse = _run(c)
    D = c["q"].shape[-1]
    wo, wl, A, E = ref.tree_attn(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["lengths"], c["see"], c["scale"])
    e = (D + 8) * 2.0 ** -22 * E + 2.0 ** -19
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (o[empty] == 0).all()
    off = (o - wo).abs() - ((2.0 ** -8 + 2 * e[..., None]) * A + 2.0 ** -8 * wo.abs())
    assert torch.isfinite(o).all() and off.max() <= 0, f"o off by {off.max():.3e} over the bound"
    loff = (lse - wl).abs() - (e + 2.0 ** -22 * (1 + wl.abs() + E))
    assert loff[~empty].numel() == 0 or loff[~empty].max() <= 0, f"lse off by {loff[~empty].max():.3e} over the bound"


CASES = [   # first, shared, own, N, Hq, Hk, D, page
    ([0, 1], [64], [0], 1, 1, 1, 128, 64), ([0, 3], [128], [0, 1, 63], 1, 4, 2, 128, 64), ([0, 2, 5], [16, 304], [5, 0, 130], 1, 8, 1, 64, 16),
    ([0, 4], [96], [33, 7], 2, 6, 2, 128, 32), ([0, 1, 1, 3], [128, 256, 0], [10], 3, 16, 2, 256, 128), ([0, 7, 9], [512, 64], [64, 3], 1, 5, 5, 64, 64),
    ([2, 6], [256], [100, 17], 1, 8, 2, 128, 64), ([0, 3], [1040], [15], 5, 12, 4, 256, 16), ([0, 2, 4], [64, 192], [70, 1], 17, 8, 4, 128, 32),
    ([0, 2], [128], [20], 64, 8, 2, 128, 64), ([0, 3], [320], [9, 40], 65, 4, 1, 64, 32), ([0, 2], [64], [130], 30, 6, 1, 256, 64),
    ([0, 2], [384], [3], 2, 128, 1, 128, 128), ([0, 40], [192], [2, 30], 1, 16, 1, 128, 64),
]


@pytest.mark.parametrize("kind", ["chain", "random"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, kind):
    _check(_case(*case, kind, seed=case[0][-1] + case[6]))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["chain", "random"])
def test_ragged_lengths(kind, D):
    """Rows of no nodes, one, some, all; padded nodes give 0 and -inf."""
    _check(_case([0, 2, 6], [96, 320], [100, 0, 300, 5, 700, 64], 20, 4, 2, D, 16, kind, seed=D, lengths=[0, 1, 20, 7, 13, 19]))


def test_more_groups_than_blocks_and_rows_than_threads():
    first = [b * 3 for b in range(201)]
    _check(_case(first, [16 * (t % 5) for t in range(200)], [0, 40, 3, 129, 17], 2, 4, 2, 64, 16, seed=3, lengths=[2, 1, 0, 2]))


@pytest.mark.parametrize("T", [31, 32, 33, 64, 65, 1025])
def test_many_groups(T):
    """Groups of no rows, one and some, rows before and behind all of them."""
    first = [1]
    for t in range(T):
        first.append(first[-1] + (0, 1, 1, 0, 0, 2, 0)[t % 7])
    rows = _case(first, [16 * (t % 3) for t in range(T)], [0, 5, 21], 1, 2, 1, 64, 16, seed=T)
    tail = {n: torch.cat([rows[n], rows[n][:1]]) for n in ("q", "ctx", "lengths", "table", "see")}   # (row 0 is in no group either)
    _check({**rows, **tail})


@pytest.mark.parametrize("D,page,B,N", [(64, 16, 3, 1), (128, 64, 2, 3), (256, 128, 2, 2), (128, 32, 40, 8)])
def test_long_trunk_is_split_over_blocks(D, page, B, N):
    _check(_case([0, B], [20096], [77, 1], N, 4, 2 if B < 10 else 1, D, page, seed=5))


def test_long_own_part():
    _check(_case([0, 2], [64], [9001, 40], 2, 4, 2, 128, 16, seed=6))


def test_same_as_tree_attention():
    """With nothing shared, and beside gdr_tree_attn on the same rows."""
    c = _case([0, 0], [0], [1], 3, 8, 2, 128, 64, seed=8)
    c2 = _case([0, 5], [640], [33, 200], 3, 8, 2, 128, 64, seed=9)
    for x in (c, c2):
        a = _args(x)
        o1, l1 = gdr.gdr_fork_attn(*a, want_lse=True)
        o2, l2 = gdr.gdr_tree_attn(a[0], a[1], a[2], a[3], a[4], a[7], a[8], x["scale"], want_lse=True)
        gdr.gdr_sync_status()
        # two roundings of each weight (2^-8 of |v| < 6) and of each result
        assert (o1.double() - o2.double()).abs().max() <= 2 * 2.0 ** -8 * 6 and (l1 - l2).abs().max() < 1e-4


def test_rising_and_far_scores():
    """The shared part's scores far above or below the own ones: the smaller weight vanishes."""
    for D in (64, 128, 256):
        for sign in (1.0, -1.0):
            c = _case([0, 2], [256], [120], 2, 4, 1, D, 32, seed=10)
            c["q"] = torch.ones_like(c["q"])
            c["k"][:] = 0.0
            at = c["table"][:, :8].long().unique()
            c["k"][at] = sign * 16 * 128.0 / D
            c["k"][at, 5] = sign * 17 * 128.0 / D
            _check(c)


def test_unseen_places_do_not_matter():
    """inf and nan behind the rows' ends, in other rows' pages and at unseen nodes."""
    for D in (64, 128, 256):
        c = _case([0, 3], [96], [40, 0, 13], 9, 6, 2, D, 32, "random", seed=11, lengths=[9, 5, 0])
        clean_o, clean_l = _run(c)
        k, v = c["k"].clone(), c["v"].clone()
        used = torch.zeros(k.shape[:2], dtype=torch.bool)
        for b in range(3):
            for pos in range(int(c["ctx"][b]) + int(c["lengths"][b])):
                used[c["table"][b, pos // 32].long(), pos % 32] = True
        k[~used], v[~used] = float("nan"), float("inf")
        # a node that nobody sees
        c["see"][:, :, 4] = False
        clean = _run(c)
        for b in (0,):
            pos = int(c["ctx"][b]) + 4
            k[c["table"][b, pos // 32].long(), pos % 32] = float("inf")
            v[c["table"][b, pos // 32].long(), pos % 32] = float("nan")
        c["k"], c["v"] = k, v
        o, l = _run(c)
        assert torch.equal(o, clean[0]) and torch.equal(l, clean[1])
        del clean_o, clean_l


def test_seen_infinities_reach_the_output():
    c = _case([0, 2], [64], [20], 3, 4, 2, 128, 32, seed=12)
    pos = int(c["ctx"][0]) + 1                      # node 1 of row 0: nodes 1 and 2 see it
    c["v"][c["table"][0, pos // 32].long(), pos % 32, 0, 7] = float("inf")
    c["v"][c["table"][1, 0].long(), 3, 1, 9] = float("-inf")   # a shared position: everyone sees it
    o, _ = _run(c)
    assert torch.isinf(o[0, 1:, :2, 7]).all() and torch.isfinite(o[0, 0, :, 7]).all() and torch.isfinite(o[1, :, :, 7]).all()
    assert torch.isinf(o[:, :, 2:, 9]).all() and torch.isfinite(o[:, :, :2, 9]).all()


def _refused(c, rows, **change):
    want = _run(c)
    for k, v in change.items():
        c[k] = v
    o, lse = gdr.gdr_fork_attn(*_args(c), want_lse=True)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    o, lse = o.double().cpu(), lse.double().cpu()
    for b in range(c["q"].shape[0]):
        if b in rows:
            assert (o[b] == 0).all() and (lse[b] == -math.inf).all(), b
        else:
            assert torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b]), b


def test_refusals_on_the_device():
    make = lambda: _case([0, 2, 4], [64, 128], [20, 33], 2, 4, 2, 128, 32, seed=13)   # noqa: E731
    t = lambda *x: torch.tensor(x, dtype=I32)   # noqa: E731
    _refused(make(), [0, 1, 2, 3], first=t(0, 3, 2))
    _refused(make(), [0, 1], shared=t(48, 128))
    _refused(make(), [0, 1], shared=t(-32, 128))
    _refused(make(), [2, 3], shared=t(64, 1 << 20))
    _refused(make(), [2, 3], shared=t(64, 192))        # beyond the rows' contexts
    _refused(make(), [1], lengths=t(2, 3, 2, 2))
    _refused(make(), [0], ctx=t(1 << 30, 97, 148, 161))
    _refused(make(), [2], ctx=t(84, 97, 100, 161))     # below what its group shares
    c = make()
    _refused(c, [2, 3], first=t(0, 2, 5))              # a group that leaves the rows


def test_pages_out_of_range_are_read_as_zeros():
    for at, rows in ((1, [0, 1]), (3, [0])):           # a shared page (of the first row's table), an own one
        c = _case([0, 2, 4], [64, 128], [50, 33], 2, 4, 2, 128, 32, seed=14)
        want = _run(c)
        c["table"][0, at] = 10 ** 6
        o, lse = gdr.gdr_fork_attn(*_args(c), want_lse=True)
        with pytest.raises(gdr.GdrError):
            gdr.gdr_sync_status()
        o = o.double().cpu()
        assert torch.isfinite(o).all()
        for b in range(4):
            assert torch.equal(o[b], want[0][b]) == (b not in rows), b


def test_only_the_first_rows_table_counts_for_what_is_shared():
    c = _case([0, 3], [128], [9], 1, 4, 2, 128, 32, seed=15)
    want = _run(c)
    c["table"][1:, :4] = -1
    assert all(torch.equal(a, b) for a, b in zip(want, _run(c)))


def test_same_bits_other_stream_and_replay():
    c = _case([0, 9, 12], [2048, 512], [50, 333, 4], 3, 8, 2, 128, 64, seed=16)
    a = _args(c)
    o, lse = gdr.gdr_fork_attn(*a, want_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for kw in (dict(), dict(stream=s)):
        o2, l2 = gdr.gdr_fork_attn(*a, want_lse=True, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    ws = torch.empty(gdr.fork_attn_workspace_bytes(12, 3, 8, 128), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, l3 = gdr.gdr_fork_attn(*a, want_lse=True, ws=ws)
    for k in (1.0, 0.5):
        a[0].mul_(k)
        g.replay()
        torch.cuda.synchronize()
        got = o3.clone(), l3.clone()
        o4, l4 = gdr.gdr_fork_attn(*a, want_lse=True)
        gdr.gdr_sync_status()
        assert torch.equal(got[0], o4) and torch.equal(got[1], l4)


def _wide(c):
    """The same with a table of many more pages than the rows have."""
    B, M = c["table"].shape
    return {**c, "table": torch.cat([c["table"], torch.full((B, 2048 // c["k"].shape[1]), -1, dtype=I32)], 1)}


@pytest.mark.parametrize("kind", ["chain", "random"])
@pytest.mark.parametrize("case", [c for c in CASES if c[3] * c[4] // c[5] <= 64])
def test_wide_tables(case, kind):
    """Short rows are attended at once where the table says that they are short, in parts where it does not."""
    c = _case(*case, kind, seed=case[0][-1] + case[6])
    _check(c)
    _check(_wide(c))


@pytest.mark.parametrize("wide", [False, True])
def test_refusals_of_short_rows(wide):
    make = lambda: (_wide if wide else dict)(_case([0, 2, 2, 4], [64, 0, 128], [20, 33], 2, 4, 2, 64, 32, seed=13))   # noqa: E731
    t = lambda *x: torch.tensor(x, dtype=I32)   # noqa: E731
    _refused(make(), [0, 1, 2, 3], first=t(0, 3, 2, 4))
    _refused(make(), [0, 1], shared=t(48, 0, 128))
    _refused(make(), [], shared=t(64, 48, 128))        # of a group without rows
    _refused(make(), [2], ctx=t(84, 97, 100, 161))
    _refused(make(), [3], lengths=t(2, 2, 2, 3))
    c = make()
    _refused(c, [2, 3], first=t(0, 2, 2, 5))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["chain", "random"])
@pytest.mark.parametrize("B,N,Hq,Hk", [(5, 2, 4, 1), (240, 1, 6, 2), (238, 2, 8, 2), (160, 8, 3, 3), (479, 3, 2, 1)])
def test_few_query_rows(B, N, Hq, Hk, kind, D):
    """Up to eight query rows a key head, of few rows and of many, which are shared out otherwise."""
    c = _case([1, B // 3, B - 2], [64, 192], [0, 5, 31, 32, 33, 64, 130, 300], N, Hq, Hk, D, 16 if N == 2 else 64, kind, seed=B + D,
              lengths=[N, max(1, N - 1), N, N, 0])
    _check(c)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,wide", [(3, False), (3, True), (160, False)])
@pytest.mark.parametrize("Hq", [12, 24, 48, 96])
def test_few_query_rows_and_what_is_not_finite(Hq, B, wide, D):
    c = _case([0, B // 3, B], [96, 32], [40, 0, 13], 2, Hq, 3, D, 32, "random", seed=21 + D, lengths=[2, 1, 0, 2])
    c = _wide(c) if wide else c
    c["see"][:, :, :] = torch.tensor([[True, False], [True, False]])   # nobody sees node 1
    want = _run(c)
    _check(c, *want)
    used = torch.zeros(c["k"].shape[:2], dtype=torch.bool)
    for b in range(B):
        for pos in range(int(c["ctx"][b]) + min(1, int(c["lengths"][b]))):
            used[c["table"][b, pos // 32].long(), pos % 32] = True
    c["k"][~used], c["v"][~used] = float("nan"), float("inf")
    assert all(torch.equal(a, b) for a, b in zip(want, _run(c)))
    # seen ones reach the output, however small their weight: of a node, of the own part, of the shared part
    for x in ("node", "own", "shared"):
        d = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in c.items()}
        pos = {"node": int(d["ctx"][0]), "own": int(d["ctx"][0]) - 3, "shared": 5}[x]
        page = d["table"][0, pos // 32].long()
        d["v"][page, pos % 32, 1, 7] = float("-inf")
        d["k"][page, pos % 32, 1] = 0.0
        d["q"][0] *= 30.0                        # (the weight of a score of 0 vanishes)
        o, _ = _run(d)
        inside = torch.zeros_like(o, dtype=torch.bool)
        rows = range(B // 3) if x == "shared" else [0]
        for b in rows:
            inside[b, :int(d["lengths"][b]), Hq // 3:2 * Hq // 3, 7] = True
        assert not torch.isfinite(o[inside]).any() and torch.isfinite(o[~inside]).all(), x


def test_pages_beyond_32_bit_offsets():
    """Pools of more than 2^32 elements: the same bits as from a small one, in every form of the call."""
    page, D = 128, 256
    pool_pages = (1 << 32) // (page * D) + 70
    pools = [torch.empty(pool_pages, page, 1, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for B, N, Hq, wide in ((3, 2, 4, False), (3, 2, 4, True), (2, 3, 6, False), (2, 20, 4, False)):
        c = _case([0, B], [128], [30, 100], N, Hq, 1, D, page, "random", seed=B + N)
        c = _wide(c) if wide else c
        P = c["k"].shape[0]
        pos = int(c["ctx"][0])
        c["v"][c["table"][0, pos // page].long(), pos % page, 0, 5] = float("inf")   # (read again by the rows that see it)
        a = _args(c)
        want = gdr.gdr_fork_attn(*a, want_lse=True)
        for pool, x in zip(pools, (a[1], a[2])):
            pool[pool_pages - P:] = x
        table = torch.where(a[3] >= 0, a[3] + (pool_pages - P), a[3]).int()
        got = gdr.gdr_fork_attn(a[0], pools[0], pools[1], table, *a[4:], want_lse=True)
        gdr.gdr_sync_status()
        assert all(torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else I32), y.view(torch.int16 if y.dtype == torch.bfloat16 else I32))
                   for x, y in zip(want, got))
