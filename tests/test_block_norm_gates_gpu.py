"""gdr_block_norm_backward with gates far from zero, where sigmoid(gate) or its distance from 1 is small.

Tolerances as in test_block_norm_gpu.py, in steps of u = 2^-24: 256 u of a gradient's magnitudes. dgate's magnitude has the
factor g (1 - g) itself. With |gate| <= 30 the exponent gate log2(e) is below 43.3 and off by half a last place (2^-19 = 32 u) and by
the constant's rounding (43.3 x 0.5 u), times ln 2: 38 u of g or 1 - g, the exponential and the division 4 u more: 64 u on
top of what smaller gates take."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import fork_ref as ref
from tests.test_block_norm_gpu import _make, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 16), (40, 1000), (9, 2560), (5, 4096), (6, 8192), (3, 16384)])
@pytest.mark.parametrize("more", [dict(), dict(post=False), dict(scale=False, fused=True)])
def test_gradients_at_large_gates(more, shape, dtype):
    c, d, (dn, dh_out) = _make(shape, dtype, 31, **more)
    far = 30 * torch.linspace(-1, 1, c["gate"].numel(), dtype=torch.float64)
    gate = far[torch.randperm(far.numel(), generator=torch.Generator().manual_seed(3))].reshape(shape).to(dtype)
    c["gate"] = gate
    d["gate"] = d["gate"].copy_(gate)
    got = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda(), eps=1e-6)
    want, mag = ref.block_norm_grad(**c, eps=1e-6, dn=dn, dh_out=dh_out)
    gate = gate.double()
    for t in (want, mag):   # 1 - g as such: the difference has lost a thousandth of it in float64, too
        t["dgate"] = t["dgate"] * torch.sigmoid(-gate) / (1 - torch.sigmoid(gate) if t is want else 1)
    for name, t in zip(("dh", "dy", "dgate", "dpre_w", "dpost_w", "dscale"), got):
        if t is not None:
            _within(t, want[name], mag[name], 576 if name in ("dpre_w", "dpost_w", "dscale") else 320, name)


def test_gates_at_the_ends():
    """Gates at which nothing or everything passes: gradients are finite, and dgate vanishes."""
    for dtype in (torch.bfloat16, torch.float32):
        c, d, (dn, dh_out) = _make((4, 256), dtype, 33)
        ends = torch.tensor([float("inf"), -float("inf"), 200.0, -200.0, torch.finfo(dtype).max, torch.finfo(dtype).min, 0.0, -0.0])
        d["gate"] = ends.to(dtype).repeat(32).expand(4, 256).contiguous().cuda()
        dh, dy, dgate, *_ = gdr.gdr_block_norm_backward(**d, dn=dn.cuda(), dh_out=dh_out.cuda())
        assert torch.isfinite(dh).all() and torch.isfinite(dy).all()
        assert (dgate.view(4, 32, 8)[..., :6] == 0).all() and (dgate.view(4, 32, 8)[..., 6:] != 0).any()
