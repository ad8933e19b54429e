"""gdr_cache_reserve, _fork, _free and _compact against lists: everything equal, nothing else written."""
import numpy as np
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def _pool(ctx, rows, M, page, layers=2, Hk=2, D=64, spare=6, seed=0, dtype=torch.bfloat16, extra=0):
    """Rows 0 .. len(ctx)-1 hold ctx positions (and pages for `extra` more), the rest nothing."""
    rng = np.random.default_rng(seed)
    need = [-(-(c + extra) // page) for c in ctx]
    P = sum(need) + spare
    order = rng.permutation(P)
    table = torch.full((rows, M), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.from_numpy(order[at:at + n].astype(np.int32))
        at += n
    lens = torch.zeros(rows, dtype=torch.int32)
    lens[:len(ctx)] = torch.tensor(ctx, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    k = torch.randn(layers, P, page, Hk, D, generator=torch.Generator().manual_seed(seed)).to(dtype)
    v = (k.float() * 2 + 1).to(dtype)
    host = (k, v, table, lens, refs)
    return ref.Pool(*host), [t.cuda() for t in host]


def _same(pool, d):
    gdr.gdr_sync_status()
    assert d[2].tolist() == pool.table
    assert d[3].tolist() == pool.ctx
    assert d[4].tolist() == pool.refs
    assert torch.equal(d[0].cpu(), pool.k) and torch.equal(d[1].cpu(), pool.v)


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,ctx", [(16, [1]), (16, [16, 33]), (32, [0, 5, 64]), (64, [200, 129]), (128, [128, 1000, 77])])
def test_fork_again_and_free(page, ctx, dtype):
    F, T = 7, len(ctx)
    pool, d = _pool(ctx, T + F, 1000 // page + 2, page, spare=F + 3, seed=page, dtype=dtype)
    rng = np.random.default_rng(1)
    src = rng.integers(0, T, F)
    dst = T + rng.permutation(F)
    for _ in range(2):   # the second fork gives the first one's pages back
        gdr.gdr_cache_fork(*d, _i(src), _i(dst))
        pool.fork(src, dst)
        _same(pool, d)
    gdr.gdr_cache_free(*d[2:], _i(dst[:4]))
    for r in dst[:4]:
        pool.release(r)
    _same(pool, d)


def test_fork_of_a_fork_keeps_counts():
    pool, d = _pool([100], 6, 8, 16, spare=8)
    for src, dst in (([0, 0], [1, 2]), ([1, 2], [3, 4]), ([4], [1])):
        gdr.gdr_cache_fork(*d, _i(src), _i(dst))
        pool.fork(src, dst)
        _same(pool, d)
    gdr.gdr_cache_free(*d[2:], _i([0, 1, 2, 3, 4]))
    for r in range(5):
        pool.release(r)
    _same(pool, d)
    assert d[4].sum() == 0


def test_reserve():
    pool, d = _pool([1, 16, 40, 0], 5, 10, 16, spare=20)
    for rows, extra in (([2, 0], 1), ([0, 1, 2, 3, 4], 30), ([1], 0), ([3], 130)):
        gdr.gdr_cache_reserve(*d[2:], _i(rows), extra, 16)
        pool.reserve(rows, extra)
        _same(pool, d)


def test_reserve_refuses_a_gap():
    """A page behind an empty entry would be overwritten: the row is left alone, the others are served."""
    pool, d = _pool([40, 20], 2, 8, 16)
    d[2][0, 5] = 0   # (row 0 holds entries 0 .. 2)
    want = d[2].clone()
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_cache_reserve(*d[2:], _i([0, 1]), 60, 16)
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    pool.reserve([1], 60)
    assert d[2][0].tolist() == want[0].tolist() and d[2][1].tolist() == pool.table[1]


@pytest.mark.parametrize("extra", [10, 30, 60])   # the new pages end before the page behind the gap, at it, past it
def test_reserve_never_fills_around_a_gap(extra):
    pool, d = _pool([40], 2, 8, 16)
    d[2][0, 4] = 0   # (row 0 holds entries 0 .. 2)
    want = d[2].clone(), d[4].clone()
    gdr.gdr_cache_reserve(*d[2:], _i([0]), extra, 16)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    assert torch.equal(d[2], want[0]) and torch.equal(d[4], want[1])


def test_many_rows_and_pages():
    """More rows than one block's threads, more pages than one pass of the search."""
    F = 1500
    pool, d = _pool([70] * 3, 3 + F, 6, 16, layers=1, Hk=1, spare=9000, seed=3)
    src, dst = [f % 3 for f in range(F)], list(range(3, 3 + F))
    gdr.gdr_cache_fork(*d, _i(src), _i(dst))
    pool.fork(src, dst)
    _same(pool, d)
    gdr.gdr_cache_reserve(*d[2:], _i(dst), 20, 16)
    pool.reserve(dst, 20)
    _same(pool, d)


def test_out_of_pages():
    pool, d = _pool([20], 6, 4, 16, spare=2)
    gdr.gdr_cache_fork(*d, _i([0, 0, 0]), _i([1, 2, 3]))
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_NO_PAGES
    pool.fork([0, 0, 0], [1, 2, 3])
    _same(pool, d)                      # two forks done, the third left empty
    gdr.gdr_cache_reserve(*d[2:], _i([0]), 40, 16)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_NO_PAGES
    _same(pool, d)
    # a fork that needs no new page still goes through
    pool, d = _pool([32], 3, 4, 16, spare=0)
    gdr.gdr_cache_fork(*d, _i([0]), _i([1]))
    pool.fork([0], [1])
    _same(pool, d)


def test_bad_rows_are_left_alone():
    pool, d = _pool([20, 30, 40], 6, 4, 16, spare=9)
    d[2][2, 1] = 1000                   # row 2 holds a page that is none
    pool.table[2][1] = 1000

    def refused(call, *a):
        call(*a)
        with pytest.raises(gdr.GdrError) as e:
            gdr.gdr_sync_status()
        assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX

    refused(gdr.gdr_cache_fork, *d, _i([0, 9, 2, -1]), _i([3, 4, 4, 5]))
    pool.fork([0], [3])
    _same(pool, d)
    refused(gdr.gdr_cache_fork, *d, _i([1, 1, 4]), _i([4, 4, 77]))      # listed twice; a source that is listed
    pool.fork([1], [4])
    _same(pool, d)
    refused(gdr.gdr_cache_fork, *d, _i([1, 1]), _i([5, 5]))
    pool.fork([1], [5])
    _same(pool, d)
    refused(gdr.gdr_cache_free, *d[2:], _i([5, 5, -3]))
    pool.release(5)
    _same(pool, d)
    refused(gdr.gdr_cache_reserve, *d[2:], _i([0, 0, 6]), 20, 16)
    pool.reserve([0], 20)
    _same(pool, d)
    refused(gdr.gdr_cache_reserve, *d[2:], _i([1]), 50, 16)             # past the table's end
    _same(pool, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,W,D", [(16, 1, 64), (16, 40, 64), (64, 9, 128), (128, 33, 256), (32, 300, 64)])
def test_compact(page, W, D, dtype):
    ctx = [0, 1, page - 1, page, 3 * page + 5]
    pool, d = _pool(ctx, 5, (3 * page + 5 + W) // page + 1, page, layers=3, D=D, spare=1, seed=W, dtype=dtype, extra=W)
    rng = np.random.default_rng(W)
    path, n = np.full((5, W), -1, np.int32), []
    for b in range(5):
        keep = np.nonzero(rng.random(W) < (0.5 if b else 2))[0]
        path[b, :len(keep)] = keep
        n.append(len(keep))
    n[4], path[4] = min(n[4], 1), path[4]
    new = gdr.gdr_cache_compact(*d[:4], _i(path), _i(n))
    want = pool.compact(path.tolist(), n)
    assert new.tolist() == want
    _same(pool, d)


def test_compact_refuses_bad_paths():
    W = 6
    ctx = [10] * 7
    pool, d = _pool(ctx, 7, 1, 16, extra=W)
    path = [[0, 2, 2, -1, -1, -1], [1, 0, 2, 3, 4, 5], [-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 6], [0, 3, 5, -1, -1, -1],
            [0, 3, 5, -1, -1, -1], [2, 4, -1, -1, -1, -1]]
    n = [3, 2, 2, 6, 3, 7, 2]
    d[2][4, 0] = -1
    pool.table[4][0] = -1
    new = gdr.gdr_cache_compact(*d[:4], _i(path), _i(n))
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX
    good = ref.Pool(*[t.cpu() for t in d])
    good.k, good.v = pool.k, pool.v
    for b in range(6):
        n[b] = 0
    want = good.compact(path, n)
    assert new.tolist() == want
    assert torch.equal(d[0].cpu(), good.k) and torch.equal(d[1].cpu(), good.v)


def test_compact_past_32_bits():
    """The last page of a layer lies past 2^32 bytes."""
    P, page, Hk, D = 70000, 16, 16, 128
    k = torch.zeros(1, P, page, Hk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, P - 1, 3], v[0, P - 1, 3] = 1, 2
    new = gdr.gdr_cache_compact(k, v, _i([[P - 1]]), _i([1]), _i([[0, 2]]), _i([2]))
    gdr.gdr_sync_status()
    assert new.item() == 3
    assert (k[0, P - 1, 2] == 1).all() and (v[0, P - 1, 2] == 2).all() and k.float().sum() == 2 * Hk * D
