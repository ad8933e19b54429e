"""Refusals of the operators of a fork batch's step: by the library on the host and before any CUDA call, by the compiled
binding, and every pair of overlapping arrays (no GPU needed: addresses and tensors have no memory)."""
import ctypes

import pytest
import torch

from gated_deltanet_rule_gb300 import build as gbuild
from gated_deltanet_rule_gb300 import gdr
from tests.test_serve_binding import BF16, F32, I64, U8, Odd, T

INV, UNS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED
BIG = 1 << 34


def A(n):
    """An address far from every other one, 16-byte aligned; never dereferenced."""
    return ctypes.c_void_p(n << 40)


def off(n, by=4):
    return ctypes.c_void_p((n << 40) + by)


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


def msg(L):
    return L.gdr_last_error_message().decode()


# ---- the library ---------------------------------------------------------------------------------
def _fork(L, q=A(1), k=A(2), v=A(3), table=A(4), ctx=A(5), lengths=A(6), mask=A(7), first=A(8), shared=A(9), scale=0.1, o=A(10),
          lse=A(11), B=4, N=3, Hq=4, Hk=2, D=128, P=9, page=16, M=8, T=2, dt=1, ws=A(12), n=BIG):
    return L.gdr_fork_attn(q, k, v, table, ctx, lengths, mask, first, shared, scale, o, lse, B, N, Hq, Hk, D, P, page, M, T, dt,
                           ws, n, None)


def test_fork_attn(L):
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(ctx=None), dict(first=None), dict(shared=None),
               dict(o=None), dict(ws=None), dict(B=0), dict(N=0), dict(Hq=3), dict(T=0), dict(T=-1), dict(P=0), dict(M=0), dict(dt=7),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=off(1)), dict(o=off(10, 8)), dict(first=off(8, 2)),
               dict(shared=off(9, 1)), dict(ctx=off(5, 2)), dict(mask=off(7)), dict(lse=off(11, 2)), dict(ws=off(12)), dict(o=A(1)),
               dict(lse=A(8)), dict(ws=A(9))):
        assert _fork(L, **kw) == INV, kw
    need = L.gdr_fork_attn_workspace_bytes(4, 3, 4, 128)
    assert need > 0 and _fork(L, n=need - 1) == INV and "workspace" in msg(L)
    for kw in (dict(D=96), dict(page=48), dict(page=256), dict(dt=0), dict(Hq=258, Hk=2), dict(B=65536), dict(T=65536),
               dict(N=1 << 16, Hq=128, Hk=1, B=1), dict(M=1 << 28), dict(B=1 << 13, N=1 << 13)):
        assert _fork(L, **kw) == UNS, kw
    for a in ((0, 3, 4, 128), (4, 0, 4, 128), (4, 3, 0, 128), (4, 3, 4, 100), (1 << 13, 1 << 13, 4, 128)):
        assert L.gdr_fork_attn_workspace_bytes(*a) == 0


def _sample(L, logits=A(1), stride=1000, t=A(2), u=A(3), k=A(4), p=A(5), m=A(6), token=A(7), probs=A(8), R=4, V=1000, dt=0):
    return L.gdr_sample(logits, stride, t, u, k, p, m, token, probs, R, V, dt, None)


def test_sample(L):
    for kw in (dict(logits=None), dict(t=None), dict(u=None), dict(token=None), dict(token=None, u=None, probs=None), dict(R=0), dict(V=0),
               dict(dt=5), dict(stride=999), dict(stride=-1000), dict(stride=(1 << 32) + 1), dict(logits=off(1, 2)), dict(t=off(2, 2)),
               dict(token=off(7, 1)), dict(probs=off(8, 2)), dict(probs=A(1)), dict(token=A(3)), dict(token=A(8))):
        assert _sample(L, **kw) == INV, kw
    for kw in (dict(V=(1 << 18) + 1, stride=1 << 19), dict(V=(1 << 18) - 7, stride=(1 << 18) + 1), dict(V=(1 << 18) - 7, stride=1 << 18, logits=off(1)),
               dict(R=(1 << 24) + 1)):
        assert _sample(L, **kw) == UNS, kw
    assert _sample(L, dt=1, logits=off(1, 1)) == INV


def _norm(L, h=A(1), y=A(2), gate=A(3), post=A(4), scale=A(5), pre=A(6), eps=1e-6, ho=A(7), no=A(8), rows=5, C=64, yr=64, gr=64, dt=1):
    return L.gdr_block_norm(h, y, gate, post, scale, pre, eps, ho, no, rows, C, yr, gr, dt, None)


def test_block_norm(L):
    for kw in (dict(h=None), dict(y=None), dict(pre=None), dict(ho=None), dict(no=None), dict(rows=0), dict(C=0), dict(C=-8), dict(dt=3),
               dict(eps=-1.0), dict(eps=float("nan")), dict(yr=56), dict(yr=68), dict(gr=63), dict(gr=1 << 23), dict(h=off(1)),
               dict(gate=off(3, 8)), dict(pre=off(6)), dict(ho=off(7)), dict(no=A(7)), dict(no=A(1)), dict(ho=off(1, 16)), dict(ho=A(2)), dict(no=A(4))):
        assert _norm(L, **kw) == INV, kw
    for kw in (dict(C=60, yr=64), dict(C=16392, yr=16392, gr=16392), dict(rows=(1 << 40) + 1)):
        assert _norm(L, **kw) == UNS, kw
    assert _norm(L, ho=A(1), no=off(1, 16)) == INV   # (in place, and the other output over it)


def _grad(L, h=A(1), y=A(2), gate=A(3), post=A(4), scale=A(5), pre=A(6), dho=A(7), dn=A(8), eps=1e-6, dh=A(9), dy=A(10), dg=A(11), dpre=A(12),
          dpost=A(13), dscale=A(14), rows=5, C=64, yr=64, gr=64, dt=1, ws=A(15), n=BIG):
    return L.gdr_block_norm_backward(h, y, gate, post, scale, pre, dho, dn, eps, dh, dy, dg, dpre, dpost, dscale, rows, C, yr, gr, dt, ws, n,
                                     None)


def test_block_norm_backward(L):
    for kw in (dict(dn=None), dict(dh=None), dict(dy=None), dict(dpre=None), dict(dg=None), dict(dpost=None), dict(dscale=None), dict(gate=None),
               dict(post=None), dict(scale=None), dict(ws=None), dict(dho=off(7)), dict(dy=off(10, 8)), dict(ws=off(15)), dict(dh=off(7, 16)),
               dict(dh=A(1)), dict(dy=A(2)), dict(dg=A(3)), dict(dpost=A(12)), dict(ws=A(9)), dict(dy=A(8))):
        assert _grad(L, **kw) == INV, kw
    need = L.gdr_block_norm_backward_workspace_bytes(64)
    assert need > 0 and _grad(L, n=need - 1) == INV and "workspace" in msg(L)
    assert [L.gdr_block_norm_backward_workspace_bytes(c) for c in (0, 4, 60, -8, 16392)] == [0] * 5
    assert _grad(L, C=60) == UNS


# each call: (arguments in order, the arrays among them; written ones; pairs that may be one array)
CALLS = {
    "gdr_fork_attn": ("q k_pages v_pages table ctx lengths mask first shared".split() + [0.1] + "o lse".split()
                      + [4, 3, 4, 2, 128, 9, 16, 8, 2, 1, "ws", BIG, None], "o lse ws", ()),
    "gdr_sample": (["logits", 1000] + "temperature u top_k top_p min_p token probs".split() + [4, 1000, 0, None], "token probs", ()),
    "gdr_block_norm": ("h y gate post_w scale pre_w".split() + [1e-6] + "h_out n_out".split() + [5, 64, 64, 64, 1, None], "h_out n_out",
                       (("h_out", "h"),)),
    "gdr_block_norm_backward": ("h y gate post_w scale pre_w dh_out dn".split() + [1e-6] + "dh dy dgate dpre_w dpost_w dscale".split()
                                + [5, 64, 64, 64, 1, "ws", BIG, None], "dh dy dgate dpre_w dpost_w dscale ws", (("dh", "dh_out"),)),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_written_array_keeps_apart(L, name):
    args, written, same = CALLS[name]
    arrays = [a for a in args if isinstance(a, str)]
    for out in written.split():
        for other in arrays:
            if other == out:
                continue
            for shift in (0, 16):
                if shift == 0 and (out, other) in same:
                    continue
                at = {a: ctypes.c_void_p((n + 1) << 40) for n, a in enumerate(arrays)}
                at[out] = ctypes.c_void_p(at[other].value + (shift if other not in ("first", "shared", "ctx", "lengths", "temperature", "u",
                                                                                    "top_k", "top_p", "min_p", "token") else 0))
                st = getattr(L, name)(*[at[a] if isinstance(a, str) else a for a in args])
                assert st == INV and "overlaps" in msg(L), (out, other)


# ---- the binding ---------------------------------------------------------------------------------
def _b_fork(**kw):
    a = dict(q=T((4, 3, 4, 128), BF16), k_pages=T((9, 16, 2, 128), BF16), v_pages=T((9, 16, 2, 128), BF16), table=T((4, 8)), ctx=T((4,)),
             first=T((3,)), shared=T((2,)), lengths=T((4,)), mask=T((4, 3, 1), I64), o=T((4, 3, 4, 128), BF16), lse=T((4, 3, 4), F32),
             ws=T((1 << 28,), U8))
    return gdr.gdr_fork_attn, {**a, **kw}


def _b_sample(**kw):
    a = dict(logits=T((4, 50), F32), temperature=T((4,), F32), u=T((4,), F32), top_k=T((4,)), top_p=T((4,), F32), min_p=T((4,), F32),
             token=T((4,)), probs=T((4, 50), F32))
    return gdr.gdr_sample, {**a, **kw}


def _b_norm(**kw):
    a = dict(h=T((2, 5, 64), BF16), y=T((2, 5, 64), BF16), pre_w=T((64,), F32), post_w=T((64,), F32), gate=T((2, 5, 64), BF16),
             scale=T((64,), F32), h_out=T((2, 5, 64), BF16), n_out=T((2, 5, 64), BF16))
    return gdr.gdr_block_norm, {**a, **kw}


def _b_grad(**kw):
    a = _b_norm()[1]
    del a["h_out"], a["n_out"]
    a.update(dn=T((2, 5, 64), BF16), dh_out=T((2, 5, 64), F32), dh=T((2, 5, 64), F32), ws=T((1 << 24,), U8))
    return gdr.gdr_block_norm_backward, {**a, **kw}


MAKE = [_b_fork, _b_sample, _b_norm, _b_grad]


def _refused(make, match, error=ValueError, **kw):
    gbuild.build()
    fn, a = make(**kw)
    with pytest.raises(error, match=match):
        fn(**a)


@pytest.mark.parametrize("make", MAKE)
def test_tensors_of_two_devices_or_none(make):
    for name, t in make()[1].items():
        if isinstance(t, torch.Tensor):
            _refused(make, "device of the other tensors", **{name: T(tuple(t.shape), t.dtype, "cuda:1")})
            _refused(make, "must be a CUDA tensor", **{name: T(tuple(t.shape), t.dtype, "cpu")})


@pytest.mark.parametrize("make", MAKE)
def test_types_and_shapes(make):
    for name, t in make()[1].items():
        if not isinstance(t, torch.Tensor) or name == "ws":
            continue
        _refused(make, None, (ValueError, TypeError), **{name: T(tuple(t.shape), torch.float16)})
        _refused(make, None, **{name: T((*t.shape, 2), t.dtype)})
        if name not in ("logits", "h", "shared"):
            _refused(make, None, **{name: T((t.shape[0] + 1, *t.shape[1:]), t.dtype)})


def test_layouts():
    _refused(_b_sample, "last dimension", logits=T((4, 50), F32, strides=(100, 2)))
    _refused(_b_sample, "drawn with u", u=None)
    _refused(_b_norm, "last dimension", y=T((2, 5, 64), BF16, strides=(640, 128, 2)))
    _refused(_b_norm, "one stride", gate=T((2, 5, 64), BF16, strides=(1000, 128, 1)))
    for shape, strides in (((2, 64), (0, 1)), ((2, 5, 64), (0, 0, 1)), ((2, 5, 64), (64, 0, 1)), ((2, 5, 64), (0, 64, 1))):   # expanded rows
        for name in ("y", "gate"):
            like = {n: T(shape, BF16) for n in ("h", "y", "gate", "h_out", "n_out")}
            _refused(_b_norm, "one stride", **{**like, name: T(shape, BF16, strides=strides)})
    _refused(_b_norm, "contiguous", h=T((2, 5, 64), BF16, strides=(640, 128, 1)))
    _refused(_b_fork, "wrong shape", first=T((4,)))
    _refused(_b_fork, r"\[T\]", shared=T((2, 1)))
    _refused(_b_fork, "neither true nor false", ArithmeticError, want_lse=Odd(), lse=None)
    _refused(_b_sample, "neither true nor false", ArithmeticError, want_probs=Odd(), probs=None)
    for make in (_b_fork, _b_grad):
        for strides in ((0,), (2,)):
            _refused(make, "ws must be contiguous", ws=T((1 << 28,), U8, strides=strides))


def test_what_does_not_fit_in_32_bits():
    big = 2 ** 32
    _refused(_b_sample, "32 bits", logits=T((4, big + 50), F32))
    _refused(_b_norm, "32 bits", h=T((2, big + 64), BF16), y=T((2, big + 64), BF16))
    _refused(_b_fork, "32 bits", table=T((4, big + 8)))
    _refused(_b_fork, "32 bits", shared=T((big + 2,)), first=T((big + 3,)))
