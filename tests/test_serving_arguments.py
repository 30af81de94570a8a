"""Arguments of the serving calls that the checks must not let pass in silence; all but the last
test on the CPU, where no kernel runs."""
import ctypes

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_abi_serving import INVALID, OK, P, append, cache

PAGES = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
LENS = torch.ones(3, dtype=torch.int32)


def _fields(table, n=3):
    return fa._cache(PAGES, PAGES.clone(), table, LENS[:n], n, 2, 64, torch.bfloat16)


def test_a_block_table_whose_rows_overlap_is_refused():
    """The library takes rows at least a row's length apart; one row seen as many is not that."""
    table = torch.arange(4, dtype=torch.int32)
    for shared in (table.expand(3, 4), table[:1].expand(3, 1), torch.arange(9, dtype=torch.int32).as_strided((3, 4), (2, 1))):
        with pytest.raises(ValueError, match="block_table"):
            _fields(shared)


def test_block_tables_that_are_taken():
    """(row stride, entries): one row of any stride, rows cut from wider ones, tables without entries."""
    wide = torch.zeros(3, 9, dtype=torch.int32)
    assert _fields(wide)[8:10] == (9, 9)
    assert _fields(wide[:, :4])[8:10] == (9, 4)
    assert _fields(wide[:, :1])[8:10] == (9, 1)
    assert _fields(wide[:1, :4], 1)[8:10] == (4, 4)
    assert _fields(wide[0, :4].expand(1, 4), 1)[8:10] == (4, 4)
    assert _fields(wide[:, :0])[9] == 0
    assert _fields(torch.zeros(3, 0, dtype=torch.int32))[9] == 0


def test_keys_are_written_without_query_heads():
    """Without queries the number of their heads does not matter; with some it must."""
    c = lambda **kw: cache(v_cache=P + 4096, **kw)        # noqa: E731
    assert append(c(), q=None, q_out=None, H=0, k=None) == INVALID        # the keys are looked at
    assert append(c(kv_lens=None), q=None, q_out=None, H=0) == INVALID
    assert append(c(), q=None, q_out=None, H=3, k=None) == INVALID        # nor is their grouping
    assert append(c(), H=0) == INVALID                                    # queries of no head
    assert append(c(), q=None, q_out=None, H=0, Hkv=0) == OK
    assert append(c(), q=None, q_out=None, H=0, T=0) == OK
    assert append(c(), q=None, q_out=None, H=-1) == INVALID


def test_a_workspace_counts_the_memory_it_has():
    """One byte seen as many is no workspace of many bytes."""
    w = torch.empty(64, dtype=torch.int32)
    assert fa._workspace_bytes(w) == 256
    for bad in (w[:1].expand(1 << 20), w[::2]):
        with pytest.raises(ValueError, match="workspace"):
            fa._workspace_bytes(bad)


@pytest.mark.gpu
def test_keys_without_queries_reach_the_cache():
    """The library's call with no query heads at all writes what the call with queries does."""
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((2, 2, 3, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    want, got = (tuple(torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)) for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2)
    lens = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    fa.append_paged(k, v, *want, table, lens, q=k)
    st3 = ctypes.c_int64 * 3
    c = fa.FaPagedCache(*(x.data_ptr() for x in got), 2 * 16 * 64, 16 * 64, 64, 4, 16, table.data_ptr(), 2, 2, lens.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert fa.lib.fa_append_paged(c, k.data_ptr(), st3(*k.stride()[:3]), v.data_ptr(), st3(*v.stride()[:3]), None, st3(), None,
                                  2, 0, 2, 3, 64, None, None, 0, 0, 1.0, fa.FA_BF16, stream) == OK
    assert fa.check_device_status() == 0
    assert bool(got[0].any()) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
