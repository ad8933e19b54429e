"""gdr_sample against float64.

Tolerances. A weight is off by at most 2^-37 of itself (the pair of its exponent holds 2^-39, the polynomial
2^-44, the table 2^-48) and rounded to 2^-41 of the largest weight, so running sums are off by at most
2^-36 of the total and 2^-41 a token: a border within that distance of u may fall to either side. With p next to 1 more than
one token may lie within it: what is behind the border has 1 - p of the total, at p = 1 - 2^-24 spread over thousands of tokens
of less than 2^-30 each, and the sums of 30011 tokens may be off by 2^-36 + 30011 x 2^-41 > 2^-27. Each of these tokens is then
p's border for sums that are off by less. What equals a border
of top-p by arithmetic (equal logits) has to come out exactly. Probabilities are a float (2^-24), times an inverse (2^-24
for the total as a float, 2^-24 for the division), rounded (2^-24): 5 x 2^-24 with the weight's own rounding, and
the smallest float where they vanish."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import fork_ref as ref

pytestmark = pytest.mark.gpu


def _t(x, dtype):
    return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")


def _call(logits, T, u=None, k=None, p=None, m=None, probs=True):
    token, pr = gdr.gdr_sample(logits, _t(T, torch.float32), _t(u, torch.float32), _t(k, torch.int32), _t(p, torch.float32),
                               _t(m, torch.float32), want_probs=probs)
    gdr.gdr_sync_status()
    return None if token is None else token.cpu().numpy(), None if pr is None else pr.double().cpu().numpy()


def _check(logits, T, u=None, k=None, p=None, m=None):
    token, probs = _call(logits, T, u, k, p, m)
    x = logits.double().cpu().numpy()
    f32 = lambda v: float(np.float32(v))   # noqa: E731
    for r in range(x.shape[0]):
        V = x.shape[1]
        off = 2.0 ** -36 + V * 2.0 ** -41
        args = (f32(T[r]), 0 if k is None else k[r], 1.0 if p is None else f32(p[r]), 0.0 if m is None else f32(m[r]))
        w = ref.weights(x[r], args[0])
        sets = [ref.kept(x[r], *args, off=o) for o in (0.0, -off, off)]
        got = probs[r] > 0
        near = [s for s in sets if not (got & ~s).any() and not (s & ~got & (w > 1e-30)).any()]
        if not near:   # the first tokens of the order, and no fewer and no more than both ends of that distance leave
            order = np.lexsort((np.arange(V), -x[r]))
            first = np.zeros(V, dtype=bool)
            first[order[:int(got.sum())]] = True
            if (first == got).all() and not (sets[1] & ~got).any() and not (got & ~sets[2]).any():
                near = [got]
        assert near, (r, args, int(got.sum()), [int(s.sum()) for s in sets])
        left = np.where(near[0], w, 0.0)
        want = left / left.sum() if left.sum() > 0 else left
        tol = 5 * 2.0 ** -24 * want + 2.0 ** -149
        assert (np.abs(probs[r] - want) <= tol).all(), (r, args, np.max(np.abs(probs[r] - want) - tol))
        if u is not None:
            may = ref.drawn(left, min(f32(u[r]), 1.0), off * left.sum())
            assert int(token[r]) in may, (r, args, int(token[r]), sorted(may)[:5])
    return token, probs


def _logits(R, V, dtype, seed, scale=3.0):
    return (scale * torch.randn(R, V, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _params(R, seed):
    g = np.random.default_rng(seed)
    return dict(T=list(g.choice([0.3, 0.7, 1.0, 1.6], R)), u=list(g.random(R).astype(np.float32)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 255, 1000, 4099, 32000, 100003, 262136])
def test_sizes(V, dtype):
    R = 5 if V < 50000 else 2
    a = _params(R, V)
    x = _logits(R, V, dtype, V)
    _check(x, a["T"], a["u"])
    g = np.random.default_rng(V + 1)
    k, p, m = g.integers(1, 80, R).tolist(), g.uniform(0.3, 0.99, R).tolist(), g.uniform(0, 0.2, R).tolist()
    _check(x, a["T"], a["u"], k=k)
    _check(x, a["T"], a["u"], p=p)
    _check(x, a["T"], a["u"], m=m)
    _check(x, a["T"], a["u"], k=k, p=p, m=m)


def test_largest_vocabulary_in_aligned_rows():
    a = _params(2, 3)
    _check(_logits(2, 1 << 18, torch.float32, 3), a["T"], a["u"], k=[0, 5000], p=[0.9, 0.8])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [1, 3, 40, 160, 400])
def test_rows(R, dtype):
    """Every split of rows over blocks, and rows of their own filters."""
    g = np.random.default_rng(R)
    a = _params(R, R)
    _check(_logits(R, 3001, dtype, R), a["T"], a["u"], k=g.integers(0, 4000, R).tolist(), p=g.choice([0.0, 0.2, 0.9, 0.999, 1.0], R).tolist(),
           m=g.choice([0.0, 1e-6, 0.05, 1.0], R).tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits_go_to_the_lowest_index(dtype):
    x = torch.zeros(6, 1000, dtype=dtype, device="cuda")
    x[1] = -7.25
    x[2, ::2] = 1.0
    x[3] = 3e38
    x[4] = torch.finfo(dtype).min
    x[5, ::2] = -0.0
    want = [(100, 0), (250, 0), (7, None), (999, 0), (1000, 0), (10, 0)]
    _, probs = _call(x, [1.0] * 6, None, k=[n for n, _ in want])
    for r, (n, _) in enumerate(want):
        where = np.nonzero(probs[r] > 0)[0]
        assert where.tolist() == (list(range(0, 2 * n, 2)) if r == 2 else list(range(n))), r
        np.testing.assert_allclose(probs[r][where], 1 / n, rtol=2.0 ** -21)
    # half of the mass of equal tokens is half of the tokens, no more
    _, probs = _call(x[:2], [1.0, 0.37], None, p=[0.5, 0.25])
    assert [int((q > 0).sum()) for q in probs] == [500, 250]
    assert (probs[0][:500] > 0).all() and (probs[1][:250] > 0).all()


def test_borders_of_u():
    x = _logits(1, 5000, torch.float32, 9).expand(6, 5000).contiguous()
    last = np.nextafter(np.float32(1), np.float32(0))
    token, _ = _check(x, [1.0] * 6, [0.0, 1e-30, 0.5, last, 1.0, 3.0], p=[0.7] * 6)
    keep = np.nonzero(ref.kept(x[0].double().cpu().numpy(), 1.0, 0, float(np.float32(0.7))))[0]
    assert token[0] == keep[0] and token[4] == token[5] == keep[-1]


def test_masked_infinite_and_nan_logits():
    inf = float("inf")
    x = _logits(8, 777, torch.float32, 2)
    x[0] = -inf
    x[1] = float("nan")
    x[2, 5:] = -inf
    x[3, 100], x[3, 300] = inf, inf
    x[4, ::3] = float("nan")
    x[5] = torch.finfo(torch.float32).min
    x[6, :] = torch.finfo(torch.float32).min
    x[6, 42] = 1.5
    x[7, 1:] = -inf
    u = [0.3, 0.3, 0.9, 0.6, 0.7, 0.25, 0.5, 0.99]
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        for more in (dict(), dict(k=[3] * 8), dict(p=[0.8] * 8), dict(m=[0.1] * 8), dict(k=[700] * 8, p=[0.9] * 8, m=[1e-3] * 8)):
            token, _ = _check(y, [0.8] * 8, u, **more)
            assert token[0] == -1 and token[1] == -1 and token[6] == 42 and token[7] == 0
    token, _ = _check(x, [0.0] * 8, u)
    assert token[3] == 100 and token[5] == 0


@pytest.mark.parametrize("T", [1e-30, 1e-4, 0.01, 0.05, 30.0, 1e6, float("inf")])
def test_extreme_temperatures(T):
    x = _logits(4, 3000, torch.float32, 4)
    x[1] += 40
    x[2] *= 1e-3
    x[3, 1] = x[3].max() * (1 + 2.0 ** -22)
    u = [0.1, 0.5, 0.9, 0.7]
    _check(x, [T] * 4, u)
    _check(x, [T] * 4, u, k=[10, 100, 1000, 2], p=[0.5, 0.9, 0.99, 0.6])


def test_greedy_takes_the_first_largest():
    x = _logits(3, 4000, torch.bfloat16, 8)
    x[0, 17] = x[0, 900] = 50
    token, probs = _check(x, [0.0] * 3, [0.1, 0.5, 0.9], k=[0, 7, 1], p=[0.5, 1.0, 0.1], m=[0.0, 0.5, 1.0])
    assert token[0] == 17 and (probs.max(1) == 1).all()


def test_slices_of_wider_rows():
    """Rows that begin at any element."""
    for dtype in (torch.float32, torch.bfloat16):
        wide = _logits(9, 1237, dtype, 6)
        for at in (0, 1, 3):
            view = wide[:, at:at + 1200]
            a = _params(9, at)
            k = [0, 1, 2, 30, 1199, 1200, 5, 6, 7]
            _check(view, a["T"], a["u"], k=k, p=[0.9] * 9)
            one, _ = _call(view, a["T"], a["u"], k=k)
            two, _ = _call(view.contiguous(), a["T"], a["u"], k=k)
            assert (one == two).all()


def test_rows_out_of_range_stay_untouched():
    x = _logits(6, 500, torch.float32, 1)
    token, probs = torch.full((6,), -7, dtype=torch.int32, device="cuda"), torch.full((6, 500), -3.0, device="cuda")
    f = torch.float32
    gdr.gdr_sample(x, _t([1.0, -1.0, float("nan"), 1.0, 1.0, 1.0], f), _t([0.5] * 6, f), _t([0, 0, 0, -2, 0, 0], torch.int32),
                   _t([1.0, 1.0, 1.0, 1.0, 1.5, 1.0], f), _t([0.0, 0.0, 0.0, 0.0, 0.0, -0.1], f), token, probs)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    assert token[0] >= 0 and (token[1:] == -7).all() and (probs[1:] == -3).all() and abs(float(probs[0].sum()) - 1) < 1e-4


def test_tokens_and_probabilities_alone_and_the_same_bits():
    x = _logits(20, 9000, torch.bfloat16, 5)
    a = _params(20, 5)
    p = [0.95] * 20
    t1, _ = _call(x, a["T"], a["u"], p=p, probs=False)
    t2, q2 = _call(x, a["T"], a["u"], p=p)
    _, q3 = _call(x, a["T"], None, p=p)
    assert (t1 == t2).all() and (q2 == q3).all()


def test_frequencies():
    """Uniform numbers at equal steps draw each token as often as its probability says, to one draw."""
    n = 4096
    x = _logits(1, 12, torch.float32, 3, scale=1.0).expand(n, 12).contiguous()
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    token, probs = _call(x, [0.9] * n, u.tolist(), k=[7] * n)
    got = np.bincount(token, minlength=12)
    assert (np.abs(got - probs[0] * n) <= 1.0).all()


def test_captured_and_replayed():
    x = _logits(30, 5000, torch.float32, 7)
    T, u, p = torch.full((30,), 0.8, device="cuda"), torch.rand(30, device="cuda"), torch.full((30,), 0.9, device="cuda")
    token, probs = torch.empty(30, dtype=torch.int32, device="cuda"), torch.empty(30, 5000, device="cuda")
    run = lambda: gdr.gdr_sample(x, T, u, None, p, None, token, probs)   # noqa: E731
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (1, 2):
        x.copy_(_logits(30, 5000, torch.float32, 70 + seed))
        u.copy_(torch.rand(30, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        t1, p1 = token.clone(), probs.clone()
        run()
        assert torch.equal(t1, token) and torch.equal(p1, probs)
    gdr.gdr_sync_status()


@pytest.mark.parametrize("filters", ["none", "k", "p", "kp", "min_p"])
@pytest.mark.parametrize("shift,scale", [(0, 1e-3), (0, 0.02), (0, 1.0), (0, 60.0), (0, 400.0), (-120, 5.0), (-130, 0.5), (126, 1.0), (300, 100.0)])
def test_bf16_logits_of_every_size(shift, scale, filters):
    """Values that are counted one by one, those around zero and the large ones, on either side of the border."""
    R, V = 6, 20011
    x = (_logits(R, V, torch.float32, 11, scale=1.0) * scale + shift).bfloat16()
    x[0, ::3] = 0.0
    x[1, ::5] = -0.0
    x[2, 7::11] = float("-inf")
    a = _params(R, 11)
    T = [t * max(scale, 0.01) for t in a["T"]]
    kw = dict(k=[0, 10000, 13500, 40, 20000, 9000]) if filters in ("k", "kp") else {}
    if filters in ("p", "kp"):
        kw["p"] = [0.5, 0.7, 0.99, 0.9, 0.75, 0.6]
    if filters == "min_p":
        kw["m"] = [0.3, 0.5, 0.01, 1e-6, 0.9, 0.1]
    _check(x, T, a["u"], **kw)


@pytest.mark.parametrize("T", [0.05, 0.2, 0.45, 0.8])
@pytest.mark.parametrize("up", [3.0, 9.0, 25.0])
def test_borders_far_below_the_largest(up, T):
    """Some likely tokens, and borders among those that have next to no weight."""
    R, V = 10, 30011
    x = _logits(R, V, torch.float32, 17, scale=2.0)
    x[:, 5:17] += up
    x[2, 100:200] = x[2, 99]                           # equal ones there
    ks = [11, 13, 40, 400, 2000, 29000, 0, 0, 0, 30]
    ps = [1.0, 1.0, 0.999, 1.0, 1.0, 1.0, 1 - 2.0 ** -20, 1 - 2.0 ** -24, 0.5, 1 - 2.0 ** -24]
    _check(x, [T] * R, _params(R, 17)["u"], k=ks, p=ps)
    _check(x, [T] * R, _params(R, 18)["u"], k=ks)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(10, 60011), (20, 33001), (25, 60011), (30, 33001), (40, 60011), (60, 33001), (76, 20011), (2, 131072)])
def test_rows_of_any_number_of_blocks(R, V, dtype):
    """From one to eight blocks a row, powers of two and others."""
    g = np.random.default_rng(R)
    a = _params(R, R + 1)
    _check(_logits(R, V, dtype, R), a["T"], a["u"], k=g.integers(0, 200, R).tolist(), p=g.choice([0.5, 0.9, 0.99, 1.0], R).tolist())
    _check(_logits(R, V, dtype, R), a["T"], a["u"], p=g.choice([0.3, 0.9, 0.999], R).tolist(), m=g.choice([0.0, 0.05], R).tolist())
