"""What is not a number in a paged cache or a query shows in every row that sees it, and in no other."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_paged_gpu import _cache, _i32

pytestmark = pytest.mark.gpu
NAN = float("nan")

# a CTA for each segment; many CTAs for one sequence (over 64 parts); both kinds in a call
LENS = [[300], [40, 3, 260], [40000], [5000, 300, 0, 17]]


def _case(lens, T, d, seed=0):
    kc, vc, table, g = _cache(lens, 2, 16, d, "bf16", seed, fill=NAN)
    q = torch.randn((len(lens), 4, T, d), generator=g, device="cuda").to(torch.bfloat16)
    return q, kc, vc, table, _i32(lens)


def _compare(got, want, poisoned):
    """Rows of `poisoned` [B, H, T] are NaN throughout, all others what they were."""
    assert fa.check_device_status() == 0
    (o, lse), (o0, lse0) = got, want
    assert bool(torch.isnan(o[poisoned]).all()) and bool(torch.isnan(lse[poisoned]).all())
    assert torch.equal(o[~poisoned], o0[~poisoned]) and torch.equal(lse[~poisoned], lse0[~poisoned])


@pytest.mark.parametrize("d,cap", [(64, 20.0), (128, 0.0)])
@pytest.mark.parametrize("lens", LENS)
def test_a_query(lens, cap, d):
    q, kc, vc, table, n = _case(lens, 2, d)
    want = fa.forward_paged(q, kc, vc, table, n, softcap=cap)
    q2 = q.clone()
    q2[0, 1, 0, 5] = NAN
    q2[-1, 2, 1] = NAN
    poisoned = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    poisoned[0, 1, 0] = poisoned[-1, 2, 1] = True
    _compare(fa.forward_paged(q2, kc, vc, table, n, softcap=cap), want, poisoned)


@pytest.mark.parametrize("d,cap", [(64, 20.0), (128, 0.0)])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("first,count", [(0, 1), (7, 1), (0, 32), (-2, 1), (-1, 1), (0, None)])
def test_keys(lens, first, count, cap, d):
    """One key, a whole tile of keys, the keys that only the last token sees, all keys."""
    q, kc, vc, table, n = _case(lens, 2, d)
    want = fa.forward_paged(q, kc, vc, table, n, softcap=cap)
    b, length = 0, lens[0]
    at = torch.arange(length, device="cuda")
    at = at[first % length:][:count]
    k2 = kc.clone()
    k2[table[b].long()[at // 16], 1, at % 16] = NAN
    poisoned = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    for t in range(2):
        poisoned[b, 2:, t] = bool((at <= length - 2 + t).any())
    _compare(fa.forward_paged(q, k2, vc, table, n, softcap=cap), want, poisoned)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("first,bad", [(0, NAN), (20, float("inf")), (-1, float("inf"))])
def test_values(lens, first, bad, d):
    """A value that is not finite shows in its column alone; an infinite one stays infinite."""
    q, kc, vc, table, n = _case(lens, 1, d)
    o0, lse0 = fa.forward_paged(q, kc, vc, table, n)
    at = first % lens[0]
    v2 = vc.clone()
    v2[table[0, at // 16].long(), 1, at % 16, 3] = bad
    o, lse = fa.forward_paged(q, kc, v2, table, n)
    assert fa.check_device_status() == 0
    assert torch.equal(lse, lse0)
    hit = torch.zeros(o.shape, dtype=torch.bool, device="cuda")
    hit[0, 2:, :, 3] = True
    assert bool(torch.isnan(o[hit]).all() if bad != bad else (o[hit] == bad).all())
    assert torch.equal(o[~hit], o0[~hit])
