"""gdr_block_norm and its gradient against float64.

Tolerances, in steps of u = 2^-24. A row's sum of squares adds at most 32 terms a lane and 9 levels of sums, so a root
mean square is off by at most 22 u, with rsqrtf's 2 ulp 26 u. A sigmoid's exponent is rounded (|gate| < 8: 12 u) and
exp and division add 4 u. With the products x is off by less than 64 u of its terms' magnitudes A, a norm of x by 64 u of
those and of how much A exceeds x. A gradient is a product of at most four such factors: 256 u of its magnitudes; a
weight's gradient adds at most 64 rows in sequence and then in trees: 512 u. Outputs of a smaller type add half a step."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import fork_ref as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def _make(shape, dtype, seed, gate=True, post=True, scale=True, fused=False):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]
    h = (2 * torch.randn(*shape, generator=g)).to(dtype)
    both = torch.randn(*shape[:-1], 2 * C, generator=g).to(dtype)
    w = lambda mean: mean + 0.2 * torch.randn(C, generator=g)   # noqa: E731
    c = dict(h=h, y=both[..., :C], pre_w=w(1.0), post_w=w(1.0) if post else None, gate=both[..., C:] if gate else None,
             scale=w(0.5) if scale else None)
    both_d = both.cuda()
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    if fused:
        d["y"], d["gate"] = both_d[..., :C], both_d[..., C:] if gate else None
    else:
        d["y"], d["gate"] = d["y"].contiguous(), d["gate"].contiguous() if gate else None
    return c, d, (torch.randn(*shape, generator=g).to(dtype), torch.randn(*shape, generator=g))


def _within(got, want, mag, steps, what):
    tol = steps * U * mag + HALF[got.dtype] * want.abs()
    got = got.double().cpu()
    off = (got - want).abs() - tol
    assert torch.isfinite(got).all() and off.max() <= 0, f"{what}: off by {off.max():.3e} over the bound"


SHAPES = [(1, 8), (3, 16), (2, 5, 120), (7, 136), (33, 256), (5, 1000), (400, 512), (9, 4096), (6, 4104), (5, 8192), (3, 12000), (4, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    for seed, more in enumerate([dict(), dict(gate=False, fused=True), dict(post=False), dict(scale=False, fused=True),
                                 dict(gate=False, post=False, scale=False)]):
        c, d, _ = _make(shape, dtype, seed, **more)
        x, n = gdr.gdr_block_norm(**d, eps=1e-6)
        wx, wn, mx, mn = ref.block_norm(**c, eps=1e-6)
        _within(x, wx, mx, 64, (more, "x"))
        _within(n, wn, mn, 128, (more, "n"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(shape, dtype):
    for seed, more in enumerate([dict(), dict(gate=False, fused=True), dict(post=False), dict(scale=False, fused=True),
                                 dict(gate=False, post=False, scale=False)]):
        c, d, (dn, dh_out) = _make(shape, dtype, seed + 10, **more)
        dh_out = None if seed == 2 else dh_out
        got = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=None if dh_out is None else dh_out.cuda(), eps=1e-6)
        want, mag = ref.block_norm_grad(**c, eps=1e-6, dn=dn, dh_out=dh_out)
        for name, t in zip(("dh", "dy", "dgate", "dpre_w", "dpost_w", "dscale"), got):
            assert (t is None) == (name not in want), name
            if t is not None:
                _within(t, want[name], mag[name], 512 if name in ("dpre_w", "dpost_w", "dscale") else 256, (more, name))


def test_gradient_against_differences():
    """A directional derivative of sum(x a) + sum(n b), by central differences of the definition in float64."""
    c, d, (dn, dh_out) = _make((11, 72), torch.float32, 3)
    got = dict(zip(("h", "y", "gate", "pre_w", "post_w", "scale"),
                   gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda(), eps=1e-6)))
    g = torch.Generator().manual_seed(4)
    for name, grad in got.items():
        v = torch.randn(c[name].shape, generator=g, dtype=torch.float64)

        def loss(t):
            x, n, _, _ = ref.block_norm(**{**{k: a.double() for k, a in c.items()}, name: c[name].double() + t * v}, eps=1e-6)
            return float((x * dh_out.double()).sum() + (n * dn.double()).sum())
        e = 1e-5
        slope = (loss(e) - loss(-e)) / (2 * e)
        terms = grad.double().cpu() * v
        # differences: e^2 of the third derivative (1e-10 of terms of order 1) and 2^-52 / e of the losses' sums
        assert abs(float(terms.sum()) - slope) <= 256 * U * float(terms.abs().sum()) + 1e-7 * (1 + float(terms.abs().sum())), name


def test_residual_in_place_and_gradient_in_place():
    c, d, (dn, dh_out) = _make((50, 640), torch.bfloat16, 5)
    x, n = gdr.gdr_block_norm(**d)
    h = d["h"].clone()
    x2, n2 = gdr.gdr_block_norm(**{**d, "h": h}, h_out=h)
    assert x2.data_ptr() == h.data_ptr() and torch.equal(x, h) and torch.equal(n, n2)
    one = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda())
    run = dh_out.cuda()
    two = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=run, dh=run)
    assert two[0].data_ptr() == run.data_ptr() and all(torch.equal(a, b) for a, b in zip(one, two))


def test_zero_rows_and_a_sum_that_cancels():
    c, d, (dn, dh_out) = _make((6, 256), torch.float32, 6, gate=False, post=False, scale=False)
    for t in (c, d):
        t["h"][0], t["y"][0] = 0, 0
        t["h"][1] = -t["y"][1]             # x is 0
        t["h"][2] = -t["y"][2] * (1 + 2.0 ** -20)
    x, n = gdr.gdr_block_norm(**d)
    assert (x[:2] == 0).all() and (n[:2] == 0).all()
    wx, wn, mx, mn = ref.block_norm(**c, eps=1e-6)
    _within(x, wx, mx, 64, "x")
    got = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda())
    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_many_rows_and_the_same_bits():
    c, d, (dn, dh_out) = _make((5000, 256), torch.bfloat16, 7)
    x, n = gdr.gdr_block_norm(**d)
    wx, wn, mx, mn = ref.block_norm(**c, eps=1e-6)
    _within(x, wx, mx, 64, "x")
    _within(n, wn, mn, 128, "n")
    one = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda())
    two = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda())
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    want, mag = ref.block_norm_grad(**c, eps=1e-6, dn=dn, dh_out=dh_out)
    for name, t in zip(("dh", "dy", "dgate", "dpre_w", "dpost_w", "dscale"), one):
        _within(t, want[name], mag[name], 512 if name in ("dpre_w", "dpost_w", "dscale") else 256, name)


def test_captured_and_replayed():
    c, d, (dn, dh_out) = _make((64, 512), torch.bfloat16, 8)
    dn, dh_out = dn.cuda(), dh_out.cuda()
    ws = torch.empty(gdr.block_norm_backward_workspace_bytes(512), dtype=torch.uint8, device="cuda")
    run = lambda: (*gdr.gdr_block_norm(**d), *gdr.gdr_block_norm_backward(**d, dn=dn, dh_out=dh_out, ws=ws))   # noqa: E731
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for k in (2.0, -0.5):
        d["h"].mul_(k)
        dn.mul_(k)
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, run()))
