"""The operators of a fork batch's step on other streams, two at once, and captured side by side."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests.test_fork_attn_gpu import _args, _case
from tests.test_launch_stream_gpu import _randn, _taken_for

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _fork(seed):
    a = _args(_case([0, 20, 31], [4096, 1024], [70, 400, 3], 2, 8, 2, 128, 64, seed=seed))
    return lambda **kw: gdr.gdr_fork_attn(*a, want_lse=True, **kw)


def _sample(seed):
    x = _randn(seed, 40, 30000, dtype=F32) * 3
    t, u = torch.full((40,), 0.9, device="cuda"), torch.rand(40, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    p = torch.full((40,), 0.95, device="cuda")
    return lambda **kw: gdr.gdr_sample(x, t, u, None, p, want_probs=True, **kw)


def _norm_inputs(seed, rows=700, C=1024):
    return dict(h=_randn(seed, rows, C), y=_randn(seed + 1, rows, C), pre_w=_randn(seed + 2, C, dtype=F32), post_w=_randn(seed + 3, C, dtype=F32),
                gate=_randn(seed + 4, rows, C), scale=_randn(seed + 5, C, dtype=F32))


def _norm(seed):
    a = _norm_inputs(seed)
    return lambda **kw: gdr.gdr_block_norm(**a, **kw)


def _grad(seed):
    a, dn, dh = _norm_inputs(seed), _randn(seed + 6, 700, 1024), _randn(seed + 7, 700, 1024, dtype=F32)
    return lambda **kw: gdr.gdr_block_norm_backward(**a, dn=dn, dh_out=dh, **kw)


MAKE = [_fork, _sample, _norm, _grad]


@pytest.mark.parametrize("make", MAKE)
def test_memory_is_of_the_launch_stream(make):
    call, s = make(1), torch.cuda.Stream()
    call()
    s.wait_stream(torch.cuda.current_stream())
    assert _taken_for(call, s) == {s.cuda_stream}
    gdr.gdr_sync_status()


@pytest.mark.parametrize("make", MAKE)
def test_calls_on_two_streams_keep_apart(make):
    calls = [make(10), make(20)]
    want = [call() for call in calls]
    gdr.gdr_sync_status()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for s, call, out in zip(streams, calls, got):
            out.append(call(stream=s))
            for n in (1 << 12, 1 << 20, 1 << 25):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    gdr.gdr_sync_status()
    for out, one in zip(got, want):
        for each in out:
            assert all(torch.equal(a, b) for a, b in zip(each, one))


@pytest.mark.parametrize("make", MAKE)
def test_two_captured_graphs(make):
    """Each graph has its own workspace and outputs: replays one after the other, each over the other's."""
    calls, graphs, outs = [make(30), make(40)], [], []
    want = [[t.clone() for t in call()] for call in calls]
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for out, one in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, one))
    gdr.gdr_sync_status()


def test_a_wait_that_runs_out_is_reported():
    """With no time to wait the attention gives up with an error; the next call runs as ever."""
    call = _fork(50)
    want = call()
    gdr.gdr_sync_status()
    gdr.debug_set_wait_budget(0)
    try:
        call()
        with pytest.raises(gdr.GdrError) as e:
            gdr.gdr_sync_status()
        assert e.value.status == gdr.GDR_ERR_TIMEOUT
    finally:
        gdr.debug_set_wait_budget(-1)
    assert all(torch.equal(a, b) for a, b in zip(want, call()))
    gdr.gdr_sync_status()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,N,Hq,Hk,shared", [(3, 1, 4, 1, 128), (31, 1, 8, 2, 4096), (240, 2, 8, 2, 2048), (20, 3, 8, 2, 4096), (12, 8, 8, 2, 4096), (12, 40, 8, 2, 4096)])
def test_waits_that_run_out_in_every_form(B, N, Hq, Hk, shared, D):
    a = _args(_case([0, B], [shared], [200, 400, 3], N, Hq, Hk, D, 16, seed=60 + B))
    want = gdr.gdr_fork_attn(*a, want_lse=True)
    gdr.gdr_sync_status()
    gdr.debug_set_wait_budget(0)
    try:
        gdr.gdr_fork_attn(*a, want_lse=True)
        with pytest.raises(gdr.GdrError) as e:
            gdr.gdr_sync_status()
        assert e.value.status == gdr.GDR_ERR_TIMEOUT
    finally:
        gdr.debug_set_wait_budget(-1)
    got = gdr.gdr_fork_attn(*a, want_lse=True)
    gdr.gdr_sync_status()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
