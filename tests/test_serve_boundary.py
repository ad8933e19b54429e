"""Refusals of the attention-layer operators, on the host and before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from gated_deltanet_rule_gb300 import build as gbuild
from gated_deltanet_rule_gb300 import gdr

INV, UNS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED


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


def _rope(L, q=A(1), k=A(2), qw=A(3), kw=A(4), inv=A(5), pos=A(6), eps=1e-6, qo=A(7), ko=A(8), B=2, N=3, Hq=4, Hk=2, D=128,
          R=64, qt=512, qh=128, kt=256, kh=128, dt=1):
    return L.gdr_qk_norm_rope(q, k, qw, kw, inv, pos, eps, 0, qo, ko, B, N, Hq, Hk, D, R, qt, qh, kt, kh, dt, None)


def test_norm_rope(L):
    for kw in (dict(q=None), dict(inv=None), dict(ko=None), dict(B=0), dict(N=0), dict(Hq=3), dict(dt=9), dict(R=8), dict(R=144),
               dict(R=-16), dict(eps=-1.0), dict(eps=float("nan")), dict(qt=4), dict(kh=-128), dict(q=off(1)), dict(qo=off(7)),
               dict(inv=off(5)), dict(pos=off(6, 2)), dict(qo=A(1)), dict(ko=off(2, 16)), dict(ko=A(7))):
        assert _rope(L, **kw) == INV, kw
    assert _rope(L, D=96) == UNS and "D=96" in msg(L)
    assert _rope(L, B=1 << 13, N=1 << 13) == UNS
    assert _rope(L, qt=2, dt=0) == INV


def _append(L, v=A(9), qo=A(7), kp=A(10), vp=A(11), table=A(12), ctx=A(13), lengths=None, P=10, page=64, M=4, q=A(1), vt=256):
    return L.gdr_qk_norm_rope_append(q, A(2), v, A(3), A(4), A(5), A(6), 1e-6, 0, qo, kp, vp, table, ctx, lengths, P, page, M,
                                     2, 3, 4, 2, 128, 64, 512, 128, 256, 128, vt, 128, 1, None)


def test_append(L):
    for kw in (dict(v=None), dict(kp=None), dict(table=None), dict(ctx=None), dict(P=0), dict(M=0), dict(kp=off(10)),
               dict(table=off(12, 2)), dict(lengths=off(14, 1)), dict(kp=A(11)), dict(vp=A(9)), dict(qo=A(10)), dict(vt=3)):
        assert _append(L, **kw) == INV, kw
    assert _append(L, page=48) == UNS and _append(L, page=256) == UNS
    assert _append(L, M=1 << 26) == UNS


def _back(L, dqo=A(7), dko=A(8), dq=A(9), dk=A(10), dqw=A(11), dkw=A(12), ws=A(13), n=1 << 30, D=128):
    return L.gdr_qk_norm_rope_backward(A(1), A(2), A(3), A(4), A(5), A(6), dqo, dko, 1e-6, 0, dq, dk, dqw, dkw, 2, 3, 4, 2, D, 64,
                                       512, 128, 256, 128, 1, ws, n, None)


def test_norm_rope_backward(L):
    need = L.gdr_qk_norm_rope_backward_workspace_bytes(128)
    assert need > 0 and L.gdr_qk_norm_rope_backward_workspace_bytes(100) == 0
    for kw in (dict(dqo=None), dict(dk=None), dict(dkw=None), dict(ws=None), dict(n=need - 1), dict(dq=off(9)), dict(dq=A(7)),
               dict(dk=A(9)), dict(dqw=A(3)), dict(ws=A(10))):
        assert _back(L, **kw) == INV, kw
    assert "workspace" in (_back(L, n=need - 1) and msg(L))
    assert _back(L, D=32) == UNS


def _attn(L, q=A(1), k=A(2), v=A(3), table=A(4), ctx=A(5), mask=A(6), scale=0.1, o=A(7), lse=A(8), B=2, N=4, Hq=4, Hk=2, D=128,
          P=9, page=16, M=4, dt=1, ws=A(9), n=1 << 34):
    return L.gdr_tree_attn(q, k, v, table, ctx, None, mask, scale, o, lse, B, N, Hq, Hk, D, P, page, M, dt, ws, n, None)


def test_tree_attn(L):
    need = L.gdr_tree_attn_workspace_bytes(128)
    assert need > 0 and L.gdr_tree_attn_workspace_bytes(80) == 0
    for kw in (dict(q=None), dict(v=None), dict(table=None), dict(o=None), dict(N=0), dict(Hq=5), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(k=off(2)), dict(mask=off(6)), dict(lse=off(8, 2)),
               dict(ws=None), dict(n=need - 1), dict(o=A(1)), dict(lse=A(7)), dict(o=A(3)), dict(ws=off(2, 64)), dict(P=0)):
        assert _attn(L, **kw) == INV, kw
    for kw in (dict(D=32), dict(dt=0), dict(page=48), dict(Hq=258, Hk=2), dict(B=70000)):
        assert _attn(L, **kw) == UNS, kw


def _verify(L, tokens=A(1), p=A(2), q=A(3), path=A(4), nxt=A(5), B=2, N=4, V=100, dt=0, u=A(7)):
    return L.gdr_verify_draft(tokens, A(8), A(9), p, q, u, A(10), path, A(11), nxt, B, N, V, dt, None)


def test_verify(L):
    for kw in (dict(tokens=None), dict(p=None), dict(path=None), dict(nxt=None), dict(B=0), dict(N=0), dict(V=0), dict(dt=3),
               dict(u=off(7, 2)), dict(p=off(2, 2)), dict(q=off(3, 1), dt=1), dict(path=A(1)), dict(nxt=A(2))):
        assert _verify(L, **kw) == INV, kw
    assert _verify(L, N=1025) == UNS and _verify(L, V=1 << 30) == UNS


def test_cache_calls(L):
    W = 1 << 30

    def reserve(table=A(1), refs=A(3), rows=A(4), extra=3, F=2, M=4, P=9, page=16, ws=A(5), n=W):
        return L.gdr_cache_reserve(table, A(2), refs, rows, extra, F, 8, M, P, page, ws, n, None)

    def fork(k=A(6), v=A(7), src=A(8), layers=2, rb=256, ws=A(5), n=W, P=9, page=16, F=2):
        return L.gdr_cache_fork(k, v, A(1), A(2), A(3), src, A(4), F, 8, 4, layers, P, page, rb, ws, n, None)

    def compact(k=A(6), v=A(7), path=A(8), new=A(9), W=6, rb=256, page=16, B=2, ctx=A(2)):
        return L.gdr_cache_compact(k, v, A(1), ctx, path, A(4), new, B, W, 4, 2, 9, page, rb, None)

    need = L.gdr_cache_workspace_bytes(2, 4)
    assert need > 0 and L.gdr_cache_workspace_bytes(0, 4) == 0
    for kw in (dict(table=None), dict(refs=None), dict(rows=off(4, 2)), dict(extra=-1), dict(F=0), dict(M=0), dict(P=0),
               dict(ws=None), dict(n=need - 1), dict(ws=off(5))):
        assert reserve(**kw) == INV, kw
    assert reserve(page=24) == UNS and reserve(F=1 << 21) == UNS
    for kw in (dict(k=None), dict(v=off(7)), dict(src=None), dict(layers=0), dict(rb=24), dict(rb=0), dict(v=A(6)),
               dict(n=need - 1)):
        assert fork(**kw) == INV, kw
    assert fork(page=1) == UNS and fork(layers=20000) == UNS
    assert L.gdr_cache_free(A(1), None, A(3), A(4), 2, 8, 4, 9, None) == INV
    assert L.gdr_cache_free(A(1), A(2), A(3), A(4), 2, 0, 4, 9, None) == INV
    for kw in (dict(k=None), dict(path=None), dict(new=None), dict(W=0), dict(B=0), dict(rb=8), dict(new=A(2)), dict(v=off(6, 64)),
               dict(path=off(8, 1))):
        assert compact(**kw) == INV, kw
    assert compact(W=2049) == UNS and compact(page=8) == UNS


def test_bindings_refuse_cpu_tensors_and_shapes():
    q = torch.zeros(1, 2, 4, 128)
    with pytest.raises(ValueError):
        gdr.gdr_qk_norm_rope(q, q, q[0, 0, 0], q[0, 0, 0], torch.zeros(4).double(), torch.zeros(1, 2, dtype=torch.int32))
    i = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdr.gdr_verify_draft(i, i, i[0], torch.zeros(2, 2, 5), None, torch.zeros(2, 2), torch.zeros(2))
    with pytest.raises(ValueError):
        gdr.gdr_cache_free(i, i[0], i[0], i[0])
