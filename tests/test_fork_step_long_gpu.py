"""Arrays of more than 2^32 elements: the last rows of gdr_block_norm, its gradient and gdr_sample are those of the same rows
alone, bit by bit (float32 logits: up to the total's rounding, 3 x 2^-24)."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _room(gib):
    if torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() < (gib << 30):
        pytest.skip("not enough memory")


def _some(n, C, seed, dtype=BF16):
    return torch.randn(n, C, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def test_block_norm():
    _room(150)
    C, few = 8192, 700
    rows = (1 << 32) // C + 100
    h = torch.zeros(rows, C, dtype=BF16, device="cuda")
    both = torch.zeros(rows, 2 * C, dtype=BF16, device="cuda")     # y and gate are slices of one projection
    h[-few:], both[-few:] = _some(few, C, 1), _some(few, 2 * C, 2)
    w = [_some(1, C, 3 + i, F32)[0] for i in range(3)]
    a = dict(h=h, y=both[:, :C], pre_w=w[0], post_w=w[1], gate=both[:, C:], scale=w[2])
    one = {k: v[-few:] if v.dim() == 2 else v for k, v in a.items()}
    for x, y in zip(gdr.gdr_block_norm(**a), gdr.gdr_block_norm(**one)):
        assert torch.equal(x[-few:], y) and not x[:-few].any()
    del x, y
    dn = torch.zeros(rows, C, dtype=BF16, device="cuda")
    dn[-few:] = _some(few, C, 9)
    got, want = gdr.gdr_block_norm_backward(**a, dn=dn), gdr.gdr_block_norm_backward(**one, dn=dn[-few:].contiguous())
    gdr.gdr_sync_status()
    for i in range(3):   # dh, dy, dgate
        assert torch.equal(got[i][-few:], want[i]) and not got[i][:1000].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sample(dtype):
    _room(120)
    V, few = 100001, 40
    R = (1 << 32) // V + 50
    x = torch.zeros(R, V + 3, dtype=dtype, device="cuda")[:, 1:V + 1]
    x[-few:] = 3 * _some(few, V, 5, dtype)
    T, u, k = torch.full((R,), 0.8, device="cuda"), torch.linspace(0, 0.999, R, device="cuda"), torch.full((R,), 50, dtype=torch.int32, device="cuda")
    token, probs = gdr.gdr_sample(x, T, u, k, want_probs=True)
    t1, p1 = gdr.gdr_sample(x[-few:], T[-few:], u[-few:], k[-few:], want_probs=True)
    gdr.gdr_sync_status()
    assert torch.equal(token[-few:], t1)
    assert ((probs[-few:] - p1).abs() <= (0 if dtype == BF16 else 3 * 2.0 ** -24) * p1).all()
    assert int(token[0]) == 0 and int(token[-few - 1]) == 49 and int((probs[-few - 1] > 0).sum()) == 50
