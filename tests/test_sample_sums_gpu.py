"""gdr_sample where sums come close to its borders.

Tolerances as in test_sample_gpu.py: running sums are off by at most 2^-36 of the total and 2^-41 a token."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests.test_sample_gpu import _call, _check, _logits, _params

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _last_kept(x, ps):
    """For each p the least and greatest index that may be the last kept one (x: a row's logits, T = 1)."""
    x = x.double().cpu().numpy()
    order = np.argsort(-x, kind="stable")
    w = np.exp(x[order] - x.max())
    before, total = np.cumsum(w) - w, w.sum()
    off = (2.0 ** -36 + len(x) * 2.0 ** -41) * total
    last = np.maximum.accumulate(order)
    want = ps.astype(np.float64) * total
    return [last[np.maximum(np.searchsorted(before, want + o, side="left"), 1) - 1] for o in (-off, off)]


@pytest.mark.parametrize("V,R,rows", [(2003, 1 << 17, 16), (33001, 1 << 14, 24)])
def test_very_many_values_of_top_p(V, R, rows):
    """Consecutive values of p over one row: wherever the border lies among the partial sums, the filter holds. With u = 1 the
    token is the last kept one; the last index is the row's lowest logit, which all these p leave out."""
    g = np.random.default_rng(V)
    T, u = torch.ones(R, device="cuda"), torch.ones(R, device="cuda")
    for seed in range(rows):
        x = _logits(1, V, F32, 100 + seed)[0]
        x[-1] = x.min() - 1e-3
        p0 = np.float32(g.uniform(0.5, 0.95))
        ps = (p0 + np.arange(R, dtype=np.float32) * np.float32(2.0 ** -24)).astype(np.float32)
        token, _ = gdr.gdr_sample(x.expand(R, V).contiguous(), T, u, None, torch.from_numpy(ps).cuda())
        gdr.gdr_sync_status()
        token, (lo, hi) = token.cpu().numpy(), _last_kept(x, ps)
        off = np.nonzero((token < lo) | (token > hi))[0]
        assert len(off) == 0, (seed, len(off), [(float(ps[i]), int(token[i]), int(lo[i]), int(hi[i])) for i in off[:3]])


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 70001, 200002])
@pytest.mark.parametrize("filters", [dict(), dict(top_k=150000), dict(top_k=1000), dict(min_p=1e-30)])
def test_weights_below_half_a_unit_are_not_drawn(at, filters, dtype):
    """One token has all the weight that counts; the others' e^-29 is 0.28 units of 2^-40 each and 2^16 units together."""
    R, V = 6, 200003
    x = torch.full((R, V), -29.0, device="cuda")
    if dtype == F32:
        x[1::2] -= torch.arange(V, device="cuda") * 1e-6
    x[:, at] = 0
    u = torch.tensor([0.0, 0.0, 1.0, 1.0, 2.0 ** -30, 1 - 2.0 ** -24], device="cuda")
    kw = {k: torch.full((R,), v, dtype=torch.int32 if k == "top_k" else F32, device="cuda") for k, v in filters.items()}
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    gdr.gdr_sample(x.to(dtype), torch.ones(R, device="cuda"), u, token=token, **kw)
    gdr.gdr_sync_status()
    assert token.tolist() == [at] * R


@pytest.mark.parametrize("T", [0.25, 1.0])
def test_draws_among_weights_around_the_unit(T):
    """A row's tail of weights between 2^-43 and 2^-37 of the largest: u at either end draws what has weight."""
    V = 150001
    x = (-27.75 + 2.0 * torch.randn(8, V, generator=torch.Generator().manual_seed(5))).cuda() * T
    x[:, 75000] = 0
    u = [0.0, 2.0 ** -31, 2.0 ** -24, 0.25, 0.75, 1 - 2.0 ** -23, 1 - 2.0 ** -24, 1.0]
    for y in (x, x.bfloat16()):
        _check(y, [T] * 8, u)
        _check(y, [T] * 8, u, k=[100000] * 8)
        _check(y, [T] * 8, u, p=[1 - 2.0 ** -24] * 8)


@pytest.mark.parametrize("value,below,top,steps,behind", [(0.0, -0.5, 25.375, 9, 94970), (-0.0, -0.5, 25.375, 9, 94970), (128.0, 126.5, 153.0, 4, 121072)])
def test_top_p_ends_where_a_bin_of_several_values_ends(value, below, top, steps, behind):
    """bf16 logits whose border lies next to the end of a bin that holds more than one value (around zero, above 127): each
    weight of 10.5 units is rounded for itself, and 1 - p, some steps of 2^-24, is a little less than the mass behind the bin."""
    n = 100000
    x = torch.full((1, n + behind + 1), below, device="cuda")
    x[0, 1:n + 1] = value
    x[0, 0] = top
    y = x.bfloat16()
    assert torch.equal(y.float(), x)
    _check(y, [(top - value) / 25.375], [0.5], p=[1 - steps * 2.0 ** -24])


@pytest.mark.parametrize("filters", ["none", "k", "p", "kp", "min_p"])
def test_bf16_rows_have_the_same_bits_in_any_batch(filters):
    """Sums of bf16 rows are of whole numbers: tokens and probabilities do not depend on how many blocks share a row."""
    V = 60011
    x = _logits(4, V, torch.bfloat16, 21)
    x[1] *= 50
    x[2] *= 2.0 ** -7
    a = _params(4, 22)
    kw = {}
    if "k" in filters:
        kw["k"] = [40, 30000, 30000, 2000]
    if filters in ("p", "kp"):
        kw["p"] = [0.9, 0.7, 0.6, 0.999]
    if filters == "min_p":
        kw["m"] = [0.05, 1e-4, 0.9, 0.01]
    T = [a["T"][0], 20.0, 0.01, a["T"][3]]
    one = None
    for times in (1, 3, 10, 18, 40, 100):
        token, probs = _call(x.repeat(times, 1), T * times, a["u"] * times, **{k: v * times for k, v in kw.items()})
        one = one or (token[:4], probs[:4])
        for i in range(times):
            assert (token[4 * i:4 * i + 4] == one[0]).all() and (probs[4 * i:4 * i + 4] == one[1]).all(), (times, i)


@pytest.mark.parametrize("T", [1e36, 1e38, float("inf")])
@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_min_p_with_a_temperature_above_the_largest(T, dtype):
    """Temperatures above 1e36 count as 1e36 for every filter: e^-100 is below 1e-3."""
    x = torch.tensor([[3e38, 2e38, 2.98e38, -1e38]], device="cuda").to(dtype)
    _, probs = _call(x, [T], None, m=[1e-3])
    w = np.exp((x.double().cpu().numpy()[0] - float(x[0, 0])) / float(np.float32(1e36)))
    want = np.where(w >= 1e-3, w, 0) / w[w >= 1e-3].sum()
    assert (np.abs(probs[0] - want) <= 5 * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_what_has_no_weight_has_no_probability(dtype):
    """Probabilities are 0, not the smallest float, beside a logit of +inf and far below the largest one; what a float32 can
    still show is there."""
    x = torch.zeros(4, 64, device="cuda")
    x[0, 5] = float("inf")
    x[1] = -1000.0
    x[1, 7] = 3.0
    x[2] = 2e4
    x[2, 9] = 3e4
    x[3] = -100.0
    x[3, 11] = 0.0
    token, probs = _call(x.to(dtype), [1.0] * 4, [0.999] * 4)
    assert token.tolist() == [5, 7, 9, 11]
    assert [int((q > 0).sum()) for q in probs] == [1, 1, 1, 64]
    assert np.abs(probs[3][0] - np.exp(-100.0)) <= 2.0 ** -149


@pytest.mark.parametrize("T", [1.5e-30, 1e-33, 1e-40])
@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_temperatures_below_the_smallest(T, dtype):
    """Temperatures below 1.5e-30, but for 0, count as that for every filter."""
    x = torch.tensor([[0.0, -1e-30, -1e-29, -1e-33, -1.0]] * 3, device="cuda").to(dtype)
    least = float(np.float32(1.5e-30))
    w = np.exp(x[0].double().cpu().numpy() / least)
    _, probs = _call(x, [T, T, 0.0], None, m=[0.25, 0.9, 0.9])
    for r, m in enumerate((0.25, 0.9)):
        want = np.where(w >= m, w, 0) / w[w >= m].sum()
        assert (np.abs(probs[r] - want) <= 5 * 2.0 ** -24 * want).all()
    assert probs[2].tolist() == [1, 0, 0, 0, 0]
