"""gdr_verify_draft against a float64 walk of the tree: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def _tree(rng, B, N, width):
    par = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            par[b, i] = i - 1 if width == 1 else max(0, i - 1 - rng.integers(0, 2 * width))
    return par


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _make(B, N, V, width, seed, drawn=True, close=0.7):
    rng = np.random.default_rng(seed)
    logits = 2 * rng.standard_normal((B, N, V))
    p, q = _softmax(logits), _softmax(logits + close * rng.standard_normal((B, N, V)))
    par = _tree(rng, B, N, width)
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            row = q[b, par[b, i]].astype(np.float64)
            if drawn:
                tok[b, i] = rng.choice(V, p=row / row.sum())
            else:
                nth = int((par[b, 1:i] == par[b, i]).sum())
                tok[b, i] = np.argsort(-row)[min(nth, V - 1)]
    u = rng.random((B, N), dtype=np.float32)
    un = rng.random(B, dtype=np.float32)
    n = rng.integers(max(1, N // 2), N + 1, B).astype(np.int32)
    return tok, par, n, p, (q if drawn else None), u, un


def _run(tok, par, n, p, q, u, un, dtype=torch.float32):
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    P = d(p).to(dtype)
    Q = None if q is None else d(q).to(dtype)
    out = gdr.gdr_verify_draft(d(tok), d(par), d(n), P, Q, d(u), d(un))
    return [x.cpu().numpy() for x in out], P.float().cpu().numpy(), None if Q is None else Q.float().cpu().numpy()


def _check(case, dtype=torch.float32):
    tok, par, n, p, q, u, un = case
    (path, count, nxt), p, q = _run(*case, dtype=dtype)
    gdr.gdr_sync_status()
    for b in range(p.shape[0]):
        want, token = ref.verify_row(tok[b], par[b], int(n[b]), p[b], None if q is None else q[b], u[b], un[b])
        assert list(path[b]) == want + [-1] * (p.shape[1] - len(want)), b
        assert count[b] == len(want) and nxt[b] == token, (b, nxt[b], token)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,N,V,width", [(1, 1, 1, 1), (2, 2, 3, 1), (7, 6, 33, 1), (20, 12, 257, 3), (5, 40, 1000, 2),
                                         (3, 9, 5003, 4), (2, 5, 70001, 3), (1, 6, 32000, 1)])
def test_against_float64(B, N, V, width, drawn, dtype):
    _check(_make(B, N, V, width, B + N + V + width, drawn), dtype)


def test_many_refusals():
    """Drafts from a distribution far from the target's: most siblings are refused."""
    _check(_make(40, 17, 300, 8, 3, close=4.0))


def test_draft_equal_to_target_is_always_accepted():
    tok, par, n, p, q, u, un = _make(6, 8, 500, 1, 4)
    u[:] = np.float32(1 - 2.0 ** -24)
    (path, count, _), _, _ = _run(tok, par, n, p, p, u, un)
    for b in range(6):
        assert count[b] == n[b] and list(path[b, :count[b]]) == list(range(n[b]))
    _check((tok, par, n, p, p, u, un))


def test_corner_rows():
    """Repeated given tokens, an empty residual, an empty distribution, NaN and negative entries, u_next
    at both ends, length 0, the last token alone."""
    B, N, V = 8, 5, 130
    tok, par, n, p, _, u, un = _make(B, N, V, 4, 5, drawn=False)
    par[:, 1:] = 0                      # four siblings
    n[:] = N
    tok[0, 1:] = 7                      # the same token four times
    u[0] = np.float32(0.999)
    p[1, 0] = 0
    p[1, 0, 9] = 1                      # one token has everything, and it is accepted
    tok[1, 2] = 9
    p[2] = 0                            # nothing at all
    p[3, :, ::2], p[3, :, 1] = np.nan, -1
    un[4], un[5] = 0, np.float32(1 - 2.0 ** -24)
    u[4:6] = np.float32(0.9999)
    n[6] = 0
    p[7] = 0
    p[7, :, V - 1] = 1
    tok[7, 1:] = 3
    _check((tok, par, n, p, None, u, un))
    q = np.where(p > 0, p, 0).astype(np.float32)
    q[1, 0] = 1.0 / V
    _check((tok, par, n, p, q, u, un))


def test_empty_residual_keeps_the_state():
    """q covers p everywhere: nothing is left of p - q, so refusals change nothing and p is sampled."""
    tok, par, n, p, q, u, un = _make(4, 4, 100, 3, 6)
    p = (0.5 * q).astype(np.float32)
    par[:, 1:] = 0
    n[:] = 4
    u[:] = np.float32(0.9)
    _check((tok, par, n, p, q, u, un))


def test_invalid_nodes_are_no_candidates():
    tok, par, n, p, q, u, un = _make(3, 6, 50, 1, 7)
    n[:] = 6
    tok[0, 1], tok[1, 2], par[2, 1] = 50, -1, 4
    u[:] = 0
    (path, count, nxt), _, _ = _run(tok, par, n, p, q, u, un)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    assert list(count) == [1, 2, 1] and list(path[1]) == [0, 1, -1, -1, -1, -1]
    assert all(0 <= t < 50 for t in nxt)


def test_bad_length_leaves_the_row():
    tok, par, n, p, q, u, un = _make(2, 4, 50, 1, 8)
    n[:] = [5, 4]
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    path = torch.full((2, 4), 77, dtype=torch.int32, device="cuda")
    count, nxt = torch.full((2,), 77, dtype=torch.int32, device="cuda"), torch.full((2,), 77, dtype=torch.int32, device="cuda")
    gdr.gdr_verify_draft(d(tok), d(par), d(n), d(p), d(q), d(u), d(un), path, count, nxt)
    with pytest.raises(gdr.GdrError):
        gdr.gdr_sync_status()
    assert (path[0] == 77).all() and count[0] == 77 and nxt[0] == 77 and count[1] >= 1


def test_first_token_follows_the_target():
    """Two drafts drawn from q, then the residual: the first token emitted has the target's
    distribution (60,000 rows; each share within five standard deviations)."""
    B, V = 60000, 5
    rng = np.random.default_rng(11)
    p = np.array([0.4, 0.3, 0.05, 0.05, 0.2], np.float32)
    q = np.array([0.1, 0.2, 0.3, 0.35, 0.05], np.float32)
    tok = np.stack([np.zeros(B), rng.choice(V, B, p=q / q.sum(dtype=np.float64)),
                    rng.choice(V, B, p=q / q.sum(dtype=np.float64))], 1).astype(np.int32)
    par = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
    (path, count, nxt), _, _ = _run(tok, par, np.full(B, 3, np.int32), np.tile(p, (B, 3, 1)), np.tile(q, (B, 3, 1)),
                                    rng.random((B, 3), dtype=np.float32), rng.random(B, dtype=np.float32))
    gdr.gdr_sync_status()
    first = np.where(count > 1, tok[np.arange(B), np.maximum(path[:, 1], 0)], nxt)
    share = np.bincount(first, minlength=V) / B
    assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B)).all(), share


def test_offsets_past_32_bits():
    """The deepest node's rows lie past 2^32 bytes and 2^31 elements."""
    N, V = 24, 100_000_000
    p = torch.zeros(1, N, V, device="cuda")
    tok = torch.arange(N, dtype=torch.int32, device="cuda")[None] + V - 100
    par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda")[None]
    for i in range(N):
        p[0, i, V - 100 + i + 1] = 1
    u = torch.full((1, N), 0.5, device="cuda")
    path, count, nxt = gdr.gdr_verify_draft(tok, par, torch.tensor([N], dtype=torch.int32, device="cuda"), p, None, u, u[:, 0].contiguous())
    gdr.gdr_sync_status()
    assert count.item() == N and nxt.item() == V - 100 + N and path[0].tolist() == list(range(N))
