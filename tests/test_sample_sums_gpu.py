"""gdr_sample where sums come close to its borders.

Tolerances as in test_sample_gpu.py: running sums are off by at most 2^-36 of the total and 2^-41 a token."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests.test_sample_gpu import _logits

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
