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


def _delta_inputs(seed, B=2, L=700, Hk=2, Hv=4, D=128, dtype=torch.bfloat16):
    f32 = torch.float32
    return (_randn(seed, B, L, Hk, D, dtype=dtype), _randn(seed + 1, B, L, Hk, D, dtype=dtype), _randn(seed + 2, B, L, Hv, D, dtype=dtype),
            -_randn(seed + 3, B, L, Hv, dtype=f32).abs(), torch.sigmoid(_randn(seed + 4, B, L, Hv, dtype=f32)))


def _prefill(seed):
    a = _delta_inputs(seed)
    return lambda **kw: gdr.gdr_chunk_fwd(*a, **kw)


def _delta_forks(seed):
    a = _delta_inputs(seed, B=40, L=16)
    trunk, idx = _randn(seed + 5, 3, 4, 128, 128, dtype=torch.float32), torch.arange(40, device="cuda") % 3
    return lambda **kw: gdr.gdr_fork_fwd(*a, trunk, idx, **kw)


def _delta_decode(seed):
    a, states = _delta_inputs(seed, L=1), _randn(seed + 5, 2, 4, 128, 128, dtype=torch.float32)

    def call(**kw):
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        return (gdr.gdr_decode_step(*a, states.clone(), **kw),)
    return call


def _delta_grad(seed):
    a, dO = _delta_inputs(seed), _randn(seed + 6, 2, 700, 4, 128)
    return lambda **kw: gdr.gdr_backward_chunked(*a, None, dO, want_dS0=False, **kw)[:5]


def _delta_grad_f32(seed):
    a, dO = _delta_inputs(seed, L=90, dtype=torch.float32), _randn(seed + 6, 2, 90, 4, 128, dtype=torch.float32)
    return lambda **kw: gdr.gdr_backward(*a, None, dO, want_dS0=False, **kw)[:5]


def _prologue_inputs(seed, B=2, L=300, Hk=2, Hv=4):
    f32 = torch.float32
    return (_randn(seed, B, L, (2 * Hk + Hv) * 128), _randn(seed + 1, (2 * Hk + Hv) * 128, 4, dtype=f32), _randn(seed + 2, B, L, Hv, dtype=f32),
            _randn(seed + 3, B, L, Hv, dtype=f32), _randn(seed + 4, Hv, dtype=f32), _randn(seed + 5, Hv, dtype=f32), Hk, Hv)


def _prologue(seed):
    a = _prologue_inputs(seed)
    return lambda **kw: gdr.gdr_prologue(*a, **kw)


def _fused_prologue(seed):
    a = _prologue_inputs(seed)
    return lambda **kw: gdr.gdr_chunk_fwd_prologue(*a, **kw)


def _gated(seed):
    x, z, w = _randn(seed, 3000, 128), _randn(seed + 1, 3000, 128), _randn(seed + 2, 128, dtype=torch.float32)
    return lambda **kw: (gdr.gdr_gated_rmsnorm(x, z, w, **kw),)


def _prefill_gated(seed):
    a, z, w = _delta_inputs(seed), _randn(seed + 6, 2, 700, 4, 128), _randn(seed + 7, 128, dtype=torch.float32)
    return lambda **kw: gdr.gdr_chunk_fwd_gated(*a, None, z, w, 1e-6, **kw)


def _prefill_save(seed):
    a = _delta_inputs(seed)
    return lambda **kw: gdr.gdr_chunk_fwd_save(*a, **kw)[:2]


DELTA = [_prefill, _delta_forks, _delta_grad, _delta_grad_f32, _prologue, _fused_prologue, _gated, _prefill_gated, _prefill_save]


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


@pytest.mark.parametrize("make", [_attn, _grad] + DELTA)
def test_memory_is_of_the_launch_stream(make):
    call, s = make(1), torch.cuda.Stream()
    call()   # (what the library sets up at its first call)
    s.wait_stream(torch.cuda.current_stream())
    assert _taken_for(call, s) == {s.cuda_stream}
    gdr.gdr_sync_status()


@pytest.mark.parametrize("make", [_attn, _grad, _cache, _delta_decode] + DELTA)
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
