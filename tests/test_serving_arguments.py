"""Arguments of the serving calls that the checks must not let pass in silence (CPU only: no kernel
runs)."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa

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
