"""Bounds of pages' keys against the keys themselves: under scales that a caller wrote, and as the pages hold them."""
import numpy as np
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from page_reference import STORES
from test_paged_gpu import TYPES, _i32

pytestmark = pytest.mark.gpu


def _near(dtype, rng, n):
    """Scales of the bounds, and for each a value next to a whole number of it, from below or above, whose fp32
    product with the scale's fp32 reciprocal lies on the whole number or beyond it."""
    scales, values = [], []
    while len(scales) < n:
        x = np.float32(torch.tensor(rng.uniform(1.0, 60.0)).to(TYPES[dtype]).float().item())
        k = int(rng.integers(1, 64))            # no larger scale is needed
        unit = np.float32(x / np.float32(k))
        for _ in range(3):
            unit = np.nextafter(unit, np.float32(0.0) if rng.random() < 0.5 else np.float32(1e9))
            there = np.float32(x * (np.float32(1.0) / unit))
            exact = float(x) / float(unit)
            if exact != k and abs(exact - k) < 1e-4 and (np.floor(there) != np.floor(exact) or np.ceil(there) != np.ceil(exact)):
                scales.append(unit)
                values.append(x)
                break
    return scales, values


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("T", [1, 70])
def test_any_scale_of_the_callers(dtype, turned, T):
    """The page held a token, bounds of 0 and a scale that is no power of two: the bounds hold in exact arithmetic, and are
    the tightest whole numbers that do."""
    rng = np.random.default_rng(5)
    scales, values = _near(dtype, rng, 64)
    n, page, d = len(scales), 128, 64
    kc, vc = (torch.zeros((n, 1, page, d), dtype=TYPES[dtype], device="cuda") for _ in range(2))
    kb = torch.zeros((n, 1, 2, d), dtype=torch.int8, device="cuda")
    bs = torch.tensor(scales, device="cuda")[:, None].contiguous()
    x = torch.tensor(values, device="cuda").to(TYPES[dtype])
    k = torch.zeros((n, 1, T, d), dtype=TYPES[dtype], device="cuda")
    k[:, 0, T // 2, 20], k[:, 0, T // 3, 41] = x, -x
    assert bool((x.abs().float() <= 127 * bs[:, 0]).all())
    # turned by angles of 0
    inv_freq = torch.zeros(8, dtype=torch.float64, device="cuda") if turned else None
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    fa.append_paged(k, k, kc, vc, table, _i32([T + 1] * n), inv_freq=inv_freq, k_bounds=kb, bound_scales=bs)
    assert fa.check_device_status() == 0
    assert bs[:, 0].tolist() == [float(s) for s in scales]
    quotient = x.double().cpu() / torch.tensor([float(s) for s in scales], dtype=torch.float64)
    assert torch.equal(kb[:, 0, 1, 20].double().cpu(), torch.ceil(quotient))
    assert torch.equal(kb[:, 0, 0, 41].double().cpu(), torch.floor(-quotient))
    lo, hi = (kb[:, 0, i].double() * bs.double() for i in (0, 1))
    keys = k[:, 0].double()
    assert bool((keys.amin(1) >= lo).all()) and bool((keys.amax(1) <= hi).all())


@pytest.mark.parametrize("turned", [False, True])
def test_a_callers_scale_that_grows(turned):
    """Earlier bounds go from a scale that is no power of two to a larger one that is: down and up, exactly."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, page, d = 500, 16, 64
    kc, vc = (torch.zeros((n, 1, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lo = torch.randint(-127, 1, (n, 1, 1, d), generator=g, device="cuda")
    hi = torch.randint(0, 128, (n, 1, 1, d), generator=g, device="cuda")
    kb = torch.cat((lo, hi), 2).to(torch.int8).contiguous()
    was = kb.double()
    # scales next to fractions of the power of two that comes, so that products lie next to whole numbers
    part = torch.randint(1, 64, (n, 1), generator=g, device="cuda").double() / 64
    old = torch.where(torch.rand((n, 1), generator=g, device="cuda") < 0.5, part * (1 - 2.0 ** -24), part * (1 + 2.0 ** -23)).float()
    bs = old.clone()
    k = torch.zeros((n, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    k[..., 7] = 127.0                                     # 127 codes of 1: the scale becomes 1
    k[..., 9] = -127.0
    fa.append_paged(k, k, kc, vc, torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(), _i32([2] * n),
                    inv_freq=torch.zeros(8, dtype=torch.float64, device="cuda") if turned else None, k_bounds=kb, bound_scales=bs)
    grew = bs[:, 0] != old[:, 0]
    assert fa.check_device_status() == 0 and bool((bs[grew] == 1.0).all()) and bool((old[~grew] >= 1.0).all())
    exact = was * old.double()[..., None, None]           # 31 bits: exact in 64
    want = torch.stack((torch.floor(exact[:, :, 0]).clamp(max=0), torch.ceil(exact[:, :, 1]).clamp(min=0)), 2)
    want[:, :, 1, 7], want[:, :, 0, 9] = 127, -127
    assert torch.equal(kb[grew].double(), want[grew])


@pytest.mark.parametrize("store", ["16", "int8", "e4m3"])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_as_the_pages_hold_them(store, turned, d):
    """Keys of 16-bit and int8 pages lie within their bounds as they are stored.  Those of e4m3 pages may lie outside by their
    rounding: half a step, 2^-4 of the value, and where a code is below the normal range 2^-10 of the scale, each time that it
    is rounded; scales at least double when they grow, so 2^-9 of the last one in all.  Then no key of a page that is not
    chosen has a larger product with the rounded query than the scores of those that are, but for that."""
    g = torch.Generator(device="cuda").manual_seed(d)
    page, length, K = 16, 600, 9
    n = -(-length // page)
    kind = torch.bfloat16 if store == "16" else STORES[store]
    kc, vc = (torch.zeros((n, 1, page, d), dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (None if store == "16" else torch.zeros((n, 1), device="cuda") for _ in range(2))
    kb, bs = torch.zeros((n, 1, 2, d), dtype=torch.int8, device="cuda"), torch.zeros((n, 1), device="cuda")
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None]
    k = (torch.randn((1, 1, length, d), generator=g, device="cuda") * torch.exp(torch.randn((1, 1, length, 1), generator=g, device="cuda"))).to(torch.bfloat16)
    inv_freq = fa.rotary_frequencies(32)[0] if turned else None
    cuts = [0, 1, 2, 9, 311, 312, 330, 331, 333, 340, 600]      # pages written in one go and token by token: scales that grow
    for begin, end in zip(cuts, cuts[1:]):
        fa.append_paged(k[:, :, begin:end], k[:, :, begin:end], kc, vc, table, _i32([end]), inv_freq=inv_freq, k_scales=ks, v_scales=vs,
                        k_bounds=kb, bound_scales=bs)
    at = table[0].long()
    held = kc[at, 0].double() * (1.0 if ks is None else ks[at].double()[..., None])
    there = (torch.arange(n * page, device="cuda") < length).reshape(n, page, 1)
    lo, hi = (kb[at, 0, i].double() * bs[at].double() for i in (0, 1))
    # the value before its rounding is within 1 / (1 - 2^-4) of the code's
    excess = torch.zeros_like(held) if store != "e4m3" else 2.0 ** -4 / (1 - 2.0 ** -4) * held.abs() + 2.0 ** -9 * ks[at].double()[..., None]
    outside = torch.maximum(lo[:, None] - held, held - hi[:, None]).masked_fill(~there, 0.0)
    assert bool((outside <= excess).all())
    assert bool((outside > 0.0).any()) == (store == "e4m3")
    q = torch.randn((1, 1, 1, d), generator=g, device="cuda").to(torch.bfloat16)
    pages = fa.select_pages(q, kb, bs, table, _i32([length]), K, page, first=0, last=0)[0, 0].long()
    assert fa.check_device_status() == 0 and bool((pages >= 0).all())
    unit = 2.0 ** np.ceil(np.log2(float(q.abs().max()) / 127.0))
    rounded = torch.round(q[0, 0, 0].double() / unit)
    scores = torch.maximum(rounded * lo, rounded * hi).sum(-1)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[pages] = False
    products = ((held * rounded).sum(-1) - (excess * rounded.abs()).sum(-1)).masked_fill(~there[..., 0], -float("inf"))
    assert float(products[rest].max()) <= float(scores[pages].min())
