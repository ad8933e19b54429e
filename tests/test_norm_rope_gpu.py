"""gdr_qk_norm_rope, its form that leaves k and v in pages, and its gradient, against float64.

Tolerances: a lane adds 16 squares and the head log2(D/16) more, so the mean of squares is off by at most
20 roundings of 2^-24, its root by 10; with the products, the angle (2^-32 turn and one rounding) and the
turn's three operations an output is off by less than 32 x 2^-24 of the magnitudes it is formed from,
plus half a step of its type. A gradient chains two such sums: 64 x 2^-24 of its magnitudes. A weight
gradient adds at most 100 terms in sequence and then in trees: 128 x 2^-24 of the sum of magnitudes."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _make(B, N, Hq, Hk, D, R, dtype, seed, fused=False, far=False):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(B, N, Hq + 2 * Hk, D, generator=g)).to(dtype)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    qw, kw = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    pos = torch.randint(0, 2 ** 31 - 1 if far else 5000, (B, N), generator=g, dtype=torch.int32)
    xd = x.cuda()
    dq, dk, dv = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hk], xd[:, :, Hq + Hk:]
    if not fused:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    return (q, k, v, qw, kw, inv, pos), (dq, dk, dv, qw.cuda(), kw.cuda(), inv.cuda(), pos.cuda())


def _within(got, want, scale, dtype, steps=32):
    got = got.double().cpu()
    tol = steps * 2.0 ** -24 * scale + HALF[dtype] * want.abs()
    off = (got - want).abs() - tol
    assert torch.isfinite(got).all() and off.max() <= 0, f"off by {off.max():.3e} over the bound"


CASES = [(1, 1, 1, 1, 64, 64), (2, 5, 4, 2, 128, 128), (3, 7, 5, 1, 256, 64), (1, 33, 16, 4, 128, 0),
         (2, 3, 6, 3, 64, 48), (1, 130, 3, 3, 256, 256), (4, 1, 15, 5, 128, 16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, dtype, interleaved):
    c, d = _make(*case, dtype, sum(case), fused=case[0] % 2 == 0)
    q_out, k_out = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:], eps=1e-6, interleaved=interleaved)
    gdr.gdr_sync_status()
    for out, x, w in ((q_out, c[0], c[3]), (k_out, c[1], c[4])):
        _within(out, *ref.norm_rope(x, w, c[6], c[5], 1e-6, interleaved), dtype)


def test_far_positions_and_negative():
    c, d = _make(2, 40, 2, 1, 128, 128, torch.float32, 5, far=True)
    c[6][1] = -c[6][1]
    d[6].copy_(c[6])
    q_out, _ = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    # the reference's own angle: float64 leaves pos 2^-53 of an angle up to 2^31
    want, scale = ref.norm_rope(c[0], c[3], c[6], c[5], 1e-6, False)
    _within(q_out, want, scale * (1 + 2.0 ** 31 * 2.0 ** -53 / (32 * 2.0 ** -24)), torch.float32)


def test_zero_rows_and_large_values():
    c, d = _make(1, 4, 2, 1, 128, 128, torch.bfloat16, 6)
    d[0][0, 1] = 0
    c[0][0, 1] = 0
    d[0][0, 2] *= 1e15
    c[0][0, 2] = d[0][0, 2].cpu()
    q_out, _ = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    assert (q_out[0, 1] == 0).all()
    _within(q_out, *ref.norm_rope(c[0], c[3], c[6], c[5], 1e-6, False), torch.bfloat16)


def test_many_tokens():
    c, d = _make(1, 9000, 8, 2, 128, 64, torch.bfloat16, 7)
    q_out, k_out = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    _within(q_out, *ref.norm_rope(c[0], c[3], c[6], c[5], 1e-6, False), torch.bfloat16)
    _within(k_out, *ref.norm_rope(c[1], c[4], c[6], c[5], 1e-6, False), torch.bfloat16)


def _pages(B, M, page, Hk, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    P = B * M + 2
    table = torch.randperm(P, generator=g)[:B * M].int().view(B, M)
    k = torch.randn(P, page, Hk, D, generator=g).to(dtype)
    return table, k, (k.float() + 1).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,page,D", [(1, 1, 16, 64), (3, 5, 16, 128), (2, 70, 32, 256), (5, 3, 128, 128), (2, 9, 64, 64)])
def test_append(B, N, page, D, dtype):
    c, d = _make(B, N, 6, 2, D, 32, dtype, B + N, fused=True)
    M = 100 // page + 2
    table, kp, vp = _pages(B, M, page, 2, D, dtype, 3)
    ctx = torch.tensor([(17 * b) % (M * page - N + 1) for b in range(B)], dtype=torch.int32)
    lengths = torch.tensor([max(0, N - 2 * b) for b in range(B)], dtype=torch.int32)
    kd, vd = kp.cuda(), vp.cuda()
    q_out = gdr.gdr_qk_norm_rope_append(*d, kd, vd, table.cuda(), ctx.cuda(), lengths.cuda())
    gdr.gdr_sync_status()
    dense_q, dense_k = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    assert torch.equal(q_out, dense_q)
    for b in range(B):
        for i in range(int(lengths[b])):
            e, o = int(table[b, (ctx[b] + i) // page]), int(ctx[b] + i) % page
            kp[e, o], vp[e, o] = dense_k[b, i].cpu(), c[2][b, i]
    assert torch.equal(kd.cpu(), kp) and torch.equal(vd.cpu(), vp)   # and nothing else was written


def test_append_bad_rows_write_nothing():
    c, d = _make(4, 3, 2, 1, 64, 32, torch.bfloat16, 9)
    table, kp, vp = _pages(4, 2, 16, 1, 64, torch.bfloat16, 4)
    ctx = torch.tensor([2, 30, -1, 5], dtype=torch.int32)        # row 1 leaves its table, row 2 is negative
    lengths = torch.tensor([3, 3, 3, 4], dtype=torch.int32)      # row 3: more than N
    table[0, 0] = 99                                             # row 0: a page that is none
    kd, vd = kp.cuda(), vp.cuda()
    gdr.gdr_qk_norm_rope_append(*d, kd, vd, table.cuda(), ctx.cuda(), lengths.cuda())
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    assert torch.equal(kd.cpu(), kp) and torch.equal(vd.cpu(), vp)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_gradient(case, dtype, interleaved):
    c, d = _make(*case, dtype, 50 + sum(case), fused=case[0] % 2 == 0)
    g = torch.Generator().manual_seed(1)
    dqo, dko = (torch.randn(t.shape, generator=g).to(dtype) for t in (c[0], c[1]))
    dq, dk, dqw, dkw = gdr.gdr_qk_norm_rope_backward(d[0], d[1], *d[3:], dqo.cuda(), dko.cuda(), interleaved=interleaved)
    gdr.gdr_sync_status()
    for dx, dw, x, w, do in ((dq, dqw, c[0], c[3], dqo), (dk, dkw, c[1], c[4], dko)):
        wx, ww, sx, sw = ref.norm_rope_grad(x, w, c[6], c[5], 1e-6, interleaved, do)
        _within(dx, wx, sx, torch.float32, 64)
        _within(dw, ww, sw, torch.float32, 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    c, d = _make(1, 6, 4, 2, 128, 64, torch.float32, 77)
    g = torch.Generator().manual_seed(2)
    dqo, dko = torch.randn(c[0].shape, generator=g), torch.randn(c[1].shape, generator=g)
    got = gdr.gdr_qk_norm_rope_backward(d[0], d[1], *d[3:], dqo.cuda(), dko.cuda(), interleaved=interleaved)

    def loss(q, k, qw, kw):
        a, _ = ref.norm_rope(q, qw, c[6], c[5], 1e-6, interleaved)
        b, _ = ref.norm_rope(k, kw, c[6], c[5], 1e-6, interleaved)
        return float((a * dqo.double()).sum() + (b * dko.double()).sum())

    base = [c[0].double(), c[1].double(), c[3].double(), c[4].double()]
    for n in range(4):
        way = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = list(base), list(base)
        up[n], down[n] = base[n] + h * way, base[n] - h * way
        diff = (loss(*up) - loss(*down)) / (2 * h)
        dot = float((got[n].double().cpu() * way).sum())
        size = float((got[n].double().cpu().abs() * way.abs()).sum())
        assert abs(diff - dot) <= 1e-5 * size + 1e-6


def test_gradient_is_deterministic_and_sums_many_rows():
    c, d = _make(3, 700, 8, 2, 128, 128, torch.bfloat16, 8)
    g = torch.Generator().manual_seed(3)
    dqo, dko = (torch.randn(t.shape, generator=g).bfloat16() for t in (c[0], c[1]))
    one = gdr.gdr_qk_norm_rope_backward(d[0], d[1], *d[3:], dqo.cuda(), dko.cuda())
    two = gdr.gdr_qk_norm_rope_backward(d[0], d[1], *d[3:], dqo.cuda(), dko.cuda())
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    _, ww, _, sw = ref.norm_rope_grad(c[0], c[3], c[6], c[5], 1e-6, False, dqo)
    _within(one[2], ww, sw, torch.float32, 128)


def test_on_another_stream():
    c, d = _make(2, 50, 4, 2, 128, 128, torch.bfloat16, 10)
    want = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = gdr.gdr_qk_norm_rope(d[0], d[1], *d[3:])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
