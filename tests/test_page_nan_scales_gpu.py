"""A page whose value scale is NaN shows in every row that sees one of its keys, however small the key's
probability and whatever shares its tile."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from page_reference import STORES
from test_paged_gpu import _i32

pytestmark = pytest.mark.gpu


def _call(store, d, H, T, length, nan_page, pages=None, slope=60.0, **kw):
    """One sequence in pages of 16 tokens, one key head: O, NaN the value scale of page nan_page."""
    g = torch.Generator(device="cuda").manual_seed(length + d)
    n = -(-length // 16)
    kc, vc = (torch.randint(-60, 61, (n, 1, 16, d), generator=g, device="cuda").to(STORES[store]) for _ in range(2))
    ks, vs = (torch.full((n, 1), 2.0 ** -6, device="cuda") for _ in range(2))
    vs[nan_page] = float("nan")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    q = torch.randn((1, H, T, d), generator=g, device="cuda").to(torch.bfloat16)
    pages = None if pages is None else _i32([[pages]])
    o, lse = fa.forward_paged(q, kc, vc, table, _i32([length]), k_scales=ks, v_scales=vs, pages=pages,
                              alibi_slopes=torch.full((H,), slope, device="cuda"), **kw)
    assert fa.check_device_status() == 0
    assert bool(torch.isfinite(lse).all())
    return o


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 2), (24, 1), (8, 5)])
def test_keys_without_weight_show(store, d, H, T):
    """The bias takes 60 from a score for each place: 16 places away nothing is left of a probability (e^-960)."""
    for length in (2000, 1998, 33, 41, 64, 200):        # whole tiles, and tiles that the last key ends
        n = -(-length // 16)
        for page in {0, 1, n // 2, max(0, n - 3), n - 2}:
            assert bool(torch.isnan(_call(store, d, H, T, length, page)).all()), (length, page)


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 2), (24, 1)])
def test_beside_entries_that_are_no_pages(store, d, H, T):
    for length in (2000, 90):
        last = -(-length // 16) - 1
        for pages in ([1, last], [1, -1, last, -1], [-1, 1, -1, -1, -1, last], [last, 1, -1]):
            if len(pages) <= last + 1:
                assert bool(torch.isnan(_call(store, d, H, T, length, 1, pages)).all()), (length, pages)
                assert bool(torch.isfinite(_call(store, d, H, T, length, 2, pages)).all())


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 8])
def test_rows_before_the_page_stay(store, d, H):
    """Drafted tokens at places 30 to 34, and page 2 begins at 32."""
    o = _call(store, d, H, 5, 35, 2)
    assert bool(torch.isfinite(o[:, :, :2]).all()) and bool(torch.isnan(o[:, :, 2:]).all())
