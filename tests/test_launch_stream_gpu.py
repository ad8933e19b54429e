"""Calls on a stream that is not the current one: the workspace and the outputs that a call allocates are of
the launch stream's memory, so that nobody is given them before the call's kernels have run."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr

pytestmark = pytest.mark.gpu


def _randn(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _attn(seed):
    """Few rows of long contexts: every item is cut over many blocks, whose parts lie in the workspace."""
    B, N, Hq, Hk, D, page, M = 2, 5, 8, 2, 128, 64, 160
    table = torch.randperm(B * M, generator=torch.Generator().manual_seed(seed)).int().view(B, M).cuda()
    a = (_randn(seed, B, N, Hq, D), _randn(seed + 1, B * M, page, Hk, D), _randn(seed + 2, B * M, page, Hk, D), table,
         _i([M * page - 7, 9000]))
    return lambda **kw: gdr.gdr_tree_attn(*a, want_lse=True, **kw)


def _grad(seed):
    B, N, Hq, Hk, D = 2, 400, 8, 2, 128
    f32 = torch.float32
    a = (_randn(seed, B, N, Hq, D), _randn(seed + 1, B, N, Hk, D), _randn(seed + 2, D, dtype=f32), _randn(seed + 3, D, dtype=f32),
         torch.logspace(0, -4, 32, dtype=torch.float64, device="cuda"), torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N),
         _randn(seed + 4, B, N, Hq, D), _randn(seed + 5, B, N, Hk, D))
    return lambda **kw: gdr.gdr_qk_norm_rope_backward(*a, **kw)


def _cache(seed):
    """Rows forked from row 0 and given pages: the lists of new pages lie in the workspace."""
    F, M, page, P = 60, 12, 16, 1000
    k = _randn(seed, 2, P, page, 2, 64)
    table = torch.full((F + 1, M), -1, dtype=torch.int32, device="cuda")
    table[0, :4] = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:4].int()
    ctx, refs = _i([50] + [0] * F), torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[table[0, :4].long()] = 1
    src, dst = _i([0] * F), torch.arange(1, F + 1, dtype=torch.int32, device="cuda")

    def call(**kw):
        mine = [t.clone() for t in (k, k, table, ctx, refs)]
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        gdr.gdr_cache_fork(*mine, src, dst, **kw)
        gdr.gdr_cache_reserve(*mine[2:], dst, 100, page, **kw)
        return mine
    return call


def _segments():
    return {s["address"]: s["stream"] for s in torch.cuda.memory_snapshot()}


def _taken_for(call, s):
    """The streams of the memory segments that a call on stream s adds, its results dropped at once."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = _segments()
    call(stream=s)
    after = _segments()
    s.synchronize()
    return {stream for at, stream in after.items() if at not in before}


@pytest.mark.parametrize("make", [_attn, _grad])
def test_memory_is_of_the_launch_stream(make):
    call, s = make(1), torch.cuda.Stream()
    call()   # (what the library sets up at its first call)
    s.wait_stream(torch.cuda.current_stream())
    assert _taken_for(call, s) == {s.cuda_stream}
    gdr.gdr_sync_status()


@pytest.mark.parametrize("make", [_attn, _grad, _cache])
def test_calls_on_two_streams_keep_apart(make):
    """Calls of two streams in flight at once, while the current stream takes and overwrites memory."""
    calls = [make(10), make(20)]
    want = [call() for call in calls]
    gdr.gdr_sync_status()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for s, call, out in zip(streams, calls, got):
            out.append(call(stream=s))
            for n in (1 << 12, 1 << 20, gdr.tree_attn_workspace_bytes(128)):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    gdr.gdr_sync_status()
    for out, one in zip(got, want):
        for each in out:
            assert all(torch.equal(a, b) for a, b in zip(each, one))


def test_dropped_outputs_are_not_overwritten_while_they_are_read():
    """The current stream reads an output that is dropped before the read has run; the launch stream's next
    call is not given its memory."""
    a, b, s = _attn(30), _attn(40), torch.cuda.Stream()
    want = a()[0].clone()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        o, lse = a(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(2_000_000)   # (cycles: the read below waits a millisecond)
        kept = o.clone()
        del o, lse
        b(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
    gdr.gdr_sync_status()
