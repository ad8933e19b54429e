"""Page tables longer than a block, and tables that hold what they should not: refused rows are untouched, the
others are served."""
import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests.test_cache_gpu import _i, _pool, _same

pytestmark = pytest.mark.gpu


def _refused(call, *a):
    call(*a)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_DEVICE_INDEX


@pytest.mark.parametrize("held", [0, 1, 255, 256, 257, 511, 512, 513, 700])
def test_reserve_in_long_tables(held):
    M, page = 700, 16
    pool, d = _pool([held * page, 40, 1], 4, M, page, layers=1, Hk=1, spare=1500)
    for extra in (0, 1, 40, 300 * page):
        rows = [r for r in (0, 1, 2, 3) if pool.ctx[r] + extra <= M * page]
        gdr.gdr_cache_reserve(*d[2:], _i(rows), extra, page)
        pool.reserve(rows, extra)
        _same(pool, d)


@pytest.mark.parametrize("extra", [0, 9, 5000])
@pytest.mark.parametrize("at", [4, 200, 255, 256, 257, 300, 511, 512, 1024, 1999])
def test_reserve_refuses_a_page_behind_an_empty_entry_wherever_it_lies(at, extra):
    pool, d = _pool([40, 0, 300 * 16, 40], 4, 2000, 16, layers=1, Hk=1, spare=700)   # rows 0, 1 and 3 hold 3, 0 and 3 pages
    d[2][:2, at] = 7
    for r in (0, 1):
        pool.table[r][at] = 7
    _refused(gdr.gdr_cache_reserve, *d[2:], _i([0, 1, 2, 3]), extra, 16)
    pool.reserve([2, 3], extra)
    _same(pool, d)


@pytest.mark.parametrize("entry", ["P", 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 2, 3, 299])
def test_reserve_refuses_a_page_out_of_range(at, entry):
    """Among the pages that the context needs, and behind them."""
    pool, d = _pool([300 * 16, 40], 2, 600, 16, layers=1, Hk=1, spare=50)
    d[3][0] = pool.ctx[0] = 40   # (300 pages held, 3 of them filled)
    d[2][0, at] = pool.table[0][at] = len(pool.refs) if entry == "P" else entry
    for extra in (0, 500):
        _refused(gdr.gdr_cache_reserve, *d[2:], _i([0, 1]), extra, 16)
        pool.reserve([1], extra)
        _same(pool, d)


@pytest.mark.parametrize("entry", ["P", 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 2, 3, 400])
def test_free_refuses_a_page_out_of_range(at, entry):
    """A page that is none cannot be given back: the row is left as it is."""
    pool, d = _pool([40, 100, 0], 4, 500, 16, layers=1, Hk=1)
    d[2][0, at] = pool.table[0][at] = len(pool.refs) if entry == "P" else entry
    _refused(gdr.gdr_cache_free, *d[2:], _i([0, 1, 2]))
    pool.release(1)
    pool.release(2)
    _same(pool, d)


@pytest.mark.parametrize("entry", ["P", 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 2, 3, 400])
def test_fork_refuses_a_row_that_holds_a_page_out_of_range(at, entry):
    pool, d = _pool([40, 100, 60], 5, 500, 16, layers=1, Hk=1)
    d[2][2, at] = pool.table[2][at] = len(pool.refs) if entry == "P" else entry
    _refused(gdr.gdr_cache_fork, *d, _i([0, 0, 1]), _i([2, 3, 4]))
    pool.fork([0, 1], [3, 4])
    _same(pool, d)


def test_as_many_pages_as_32_bits_count():
    """The search for free pages ends where the counts do, past every page in use."""
    P = 2 ** 31 - 1
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    table, ctx = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), _i([0, 0])
    gdr.gdr_cache_reserve(table, ctx, refs, _i([0]), 10, 16)
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_sync_status()
    assert e.value.status == gdr.GDR_ERR_NO_PAGES and (table == -1).all()
    refs[P - 2:] = 0
    gdr.gdr_cache_reserve(table, ctx, refs, _i([1]), 20, 16)
    gdr.gdr_sync_status()
    assert table.tolist() == [[-1] * 4, [P - 2, P - 1, -1, -1]] and (refs[P - 3:] == 1).all()
