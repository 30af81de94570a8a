"""Attention over 8-bit pages whose value scales lie far apart: a page of large values that a row gives no weight
takes no precision from the others.

The bound is page_reference.py's, but for what is rounded below fp16's normal range: a row's products p vs are
rounded in units of the largest of them (or of one not larger), so that part is 2^-25 max_j (p_j vs_j) sum |e_j|.
The unit's exponent is a difference of two fp32 numbers and is applied twice, to products and outputs, by exponentials
with errors of 2^-22: with the score scales here |log2| of it stays below 256, 2 (2^-22 + 256 V) sum p |v| in all.
"""
import math

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from page_reference import STORES
from scored_reference import V, assert_within, scores, softmax
from test_paged_gpu import TYPES, _i32

pytestmark = pytest.mark.gpu


def _check(q, kc, vc, ks, vs, length, o, lse, slope, pages=None, page=16):
    B, H, T, d = q.shape
    Hkv = kc.shape[1]
    scale = 1 / math.sqrt(d)
    qpos = length - T + torch.arange(T, device="cuda")
    for g in range(Hkv):
        which = torch.arange(-(-length // page), device="cuda") if pages is None else pages[0, g].long()
        which = which[which >= 0]
        kpos = (which[:, None] * page + torch.arange(page, device="cuda")).flatten()
        there = kpos < length
        c, e = (x[which, g].reshape(-1, d)[there].double() for x in (kc, vc))
        k1, v1 = (x[which, g].double().repeat_interleave(page)[there][:, None] for x in (ks, vs))
        kpos = kpos[there]
        allowed = kpos[None, :] <= qpos[:, None]
        dist = (qpos[:, None] - kpos[None, :]).abs().double()
        for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
            x = q[0, h].double()
            s, _, err = scores(x, k1 * c, allowed, dist, scale, 0.0, slope)
            err = err + (4 * V * (x @ (k1 * c).T * scale).abs() +
                         scale * 2.0 ** -39 * x.abs().amax(-1, keepdim=True) * (k1 * c).abs().sum(-1)[None, :]).masked_fill(~allowed, 0.0)
            p, want_lse = softmax(s)
            f = 2 * (err.amax(-1, keepdim=True) + 2.0 ** -22)
            want, size = p @ (v1 * e), p @ (v1 * e).abs()
            u = torch.finfo(q.dtype).eps / 2
            tol = u * want.abs() + (2.0 ** -11 + f + 2 * (2.0 ** -22 + 256 * V)) * size
            tol = tol + 2.0 ** -25 * (p * v1.T).amax(-1, keepdim=True) * (allowed.double() @ e.abs())
            if q.dtype == torch.float16:
                tol = tol + 2.0 ** -25
            assert_within(f"O {h}", o[0, h], want, tol)
            assert_within(f"LSE {h}", lse[0, h], want_lse, f[:, 0] / 2 + 4 * V * (1 + want_lse.abs()))


def _inputs(store, d, dtype, H, Hkv, T, length, g):
    n = -(-length // 16)
    kc, vc = (torch.randint(-60, 61, (n, Hkv, 16, d), generator=g, device="cuda").to(STORES[store]) for _ in range(2))
    ks, vs = (2.0 ** -6 * torch.exp(torch.randn((n, Hkv), generator=g, device="cuda")).clamp(0.25, 4.0) for _ in range(2))
    q = torch.randn((1, H, T, d), generator=g, device="cuda").to(TYPES[dtype])
    return kc, vc, ks, vs, torch.arange(n, dtype=torch.int32, device="cuda")[None], q


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,T", [(4, 1, 1), (2, 2, 3), (24, 1, 1), (8, 1, 5)])
def test_large_values_without_weight(store, dtype, d, H, Hkv, T):
    """A bias of 0.5 a place takes e^-70 and more from the pages whose scales are 2^20 to 2^60 times the others'."""
    g = torch.Generator(device="cuda").manual_seed(d + H)
    for length, large, up in ((300, [0], 2.0 ** 20), (300, [3], 2.0 ** 40), (2100, [0, 1, 60, 90], 2.0 ** 60), (190, [0], 2.0 ** 24)):
        kc, vc, ks, vs, table, q = _inputs(store, d, dtype, H, Hkv, T, length, g)
        vs[large] *= up
        pages = torch.tensor([large + list(range(max(large) + 1, table.shape[1]))], device="cuda").repeat(Hkv, 1)
        for chosen in (None, pages.to(torch.int32)[None].contiguous(), pages.flip(1).to(torch.int32)[None].contiguous()):
            o, lse = fa.forward_paged(q, kc, vc, table, _i32([length]), k_scales=ks, v_scales=vs, pages=chosen,
                                      alibi_slopes=torch.full((H,), 0.5, device="cuda"))
            assert fa.check_device_status() == 0
            _check(q, kc, vc, ks, vs, length, o, lse, 0.5, chosen)


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,T", [(4, 1), (24, 1), (8, 5)])
def test_scales_of_all_sizes(store, d, H, T):
    """Scales from 2^-60 to 2^30, and none at all, in any order: rows of each page's weight."""
    g = torch.Generator(device="cuda").manual_seed(d + H)
    for length, slope in ((300, 0.0), (300, 0.2), (1500, 0.05), (33, 0.0)):
        kc, vc, ks, vs, table, q = _inputs(store, d, "fp16", H, 1, T, length, g)
        vs *= torch.exp2(torch.randint(-60, 10, vs.shape, generator=g, device="cuda").float())
        vs[1] = 0.0
        o, lse = fa.forward_paged(q, kc, vc, table, _i32([length]), k_scales=ks, v_scales=vs,
                                  alibi_slopes=torch.full((H,), slope, device="cuda") if slope else None)
        assert fa.check_device_status() == 0
        _check(q, kc, vc, ks, vs, length, o, lse, slope)


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("H", [4, 24])
def test_values_of_no_size_at_the_heaviest_key(store, H):
    """The last page has scale 0 and all the weight, others little (or, underflowing, none): 0 and no NaN."""
    g = torch.Generator(device="cuda").manual_seed(H)
    for slope in (0.5, 30.0):
        kc, vc, ks, vs, table, q = _inputs(store, 128, "bf16", H, 1, 1, 304, g)
        vs[-1] = 0.0
        o, lse = fa.forward_paged(q, kc, vc, table, _i32([304]), k_scales=ks, v_scales=vs, alibi_slopes=torch.full((H,), slope, device="cuda"))
        _check(q, kc, vc, ks, vs, 304, o, lse, slope)
        assert slope < 1.0 or not bool(o.any())


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,T", [(4, 1), (24, 1), (8, 5)])
def test_the_smallest_and_the_largest_scales(store, d, H, T):
    """All values as small as scales from 2^-100 on make them (and somewhat smaller), or as large as they may be: sums of P (up
    to 2^8) times values run in fp32 before they are divided, so 2^8 times 1500 keys times 2^8 codes of scales up to 2^98
    stays below 2^128.  (Scales of 2^114 do not.)"""
    g = torch.Generator(device="cuda").manual_seed(d + H)
    for shift in (2.0 ** -90, 2.0 ** -94, 2.0 ** -106, 2.0 ** 100):     # of scales around 2^-6
        for length, slope in ((300, 0.0), (1500, 0.1), (33, 0.0)):
            kc, vc, ks, vs, table, q = _inputs(store, d, "bf16", H, 1, T, length, g)
            vs *= shift
            o, lse = fa.forward_paged(q, kc, vc, table, _i32([length]), k_scales=ks, v_scales=vs,
                                      alibi_slopes=torch.full((H,), slope, device="cuda") if slope else None)
            assert fa.check_device_status() == 0
            _check(q, kc, vc, ks, vs, length, o, lse, slope)
