"""8-bit pages on the GPU: their write (scales, codes, key bounds) and attention over them, all pages or chosen
ones, against 64-bit formulas (bounds derived in page_reference.py)."""
import math

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from page_reference import LARGEST, STORES, grid, head_forward8, power
from scored_reference import assert_within, head_forward
from test_paged_gpu import TYPES, _cache, _i32, _slopes
from test_rotary_gpu import _turn

pytestmark = pytest.mark.gpu


def _coded(x, store, g, any_scale=True):
    """Pages [n, Hkv, page, d] in 8 bits, with scales that differ from page to page."""
    x = x.float() * torch.exp(torch.randn(x.shape[:2], generator=g, device="cuda"))[..., None, None]
    scale = x.abs().amax((-1, -2)) / LARGEST[store] * (1.0 if not any_scale else 1.03)
    y = x / scale[..., None, None]
    return (torch.round(y) if store == "int8" else y).to(STORES[store]), scale


def _cache8(lens, Hkv, page, d, dtype, store, seed):
    """A cache of random pages; codes that no sequence holds are the store's worst (NaN for e4m3), scales of
    unused pages NaN."""
    kc, vc, table, g = _cache(lens, Hkv, page, d, dtype, seed)
    used = torch.zeros((kc.shape[0], page), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            used[table[b, i].item(), : min(page, n - i * page)] = True
    out = []
    for c in (kc, vc):
        code, scale = _coded(c, store, g)
        raw = code.view(torch.uint8)
        raw.masked_fill_(~used[:, None, :, None], 0x7f)
        scale = torch.where(used.any(-1)[:, None], scale, float("nan"))
        out += [code, scale]
    return out[0], out[2], out[1], out[3], table, g


def _check(q, kc, vc, ks, vs, table, lens, o, lse, cap=0.0, slopes=None, q_lens=None, scale=None, pages=None):
    B, H, T, d = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    for b, n in enumerate(lens):
        new = T if q_lens is None else min(max(q_lens[b], 0), T)
        qpos = n - new + torch.arange(T, device="cuda")
        exists = (torch.arange(T, device="cuda") < new)[:, None]
        for g in range(Hkv):
            total = -(-n // page)
            if pages is None:
                which = torch.arange(total, device="cuda")
            else:
                which = pages[b, g, : min(total, pages.shape[2])].long()
                which = which[(which >= 0) & (which < total)]
            kpos = (which[:, None] * page + torch.arange(page, device="cuda")).flatten()
            there = kpos < n
            kpos = kpos[there]
            at = table[b].long()[which]
            c, e = (x[at, g].reshape(-1, d)[there].double() for x in (kc, vc))
            k1, v1 = (torch.ones((kpos.numel(), 1), dtype=torch.float64, device="cuda") if x is None else
                      x[at, g].double().repeat_interleave(page)[there][:, None] for x in (ks, vs))
            allowed = (kpos[None, :] <= qpos[:, None]) & exists
            dist = (qpos[:, None] - kpos[None, :]).abs().double()
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                slope = 0.0 if slopes is None else float(slopes[h])
                if ks is None:
                    u = torch.finfo(q.dtype).eps / 2
                    ref = head_forward(q[b, h].double(), c, e, allowed, dist, scale, cap, slope, u,
                                       2.0 ** -25 if q.dtype == torch.float16 else 0.0)
                else:
                    ref = head_forward8(q[b, h].double(), c, e, k1, v1, allowed, dist, scale, cap, slope, q.dtype)
                assert_within(f"O {b} {h}", o[b, h], ref[0], ref[2])
                assert_within(f"LSE {b} {h}", lse[b, h], ref[1], ref[3])


def _run(lens, H, Hkv, T, page, d, dtype, store, cap=0.0, alibi=False, q_lens=None, scale=None, seed=0, picks=0):
    if store == "16":
        kc, vc, table, g = _cache(lens, Hkv, page, d, dtype, seed, fill=float("nan"))
        ks = vs = None
    else:
        kc, vc, ks, vs, table, g = _cache8(lens, Hkv, page, d, dtype, store, seed)
    q = (torch.randn((len(lens), H, T, d), generator=g, device="cuda") * 2).to(TYPES[dtype])
    q *= torch.exp2(torch.randint(-3, 3, (len(lens), H, T, 1), generator=g, device="cuda")).to(TYPES[dtype]) / 8
    slopes = _slopes(H) if alibi else None
    pages = None
    if picks:
        pages = torch.full((len(lens), Hkv, picks), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            total = -(-n // page)
            for h in range(Hkv):
                some = torch.randperm(total, generator=g, device="cuda")[: min(picks, total)]
                pages[b, h, : some.numel()] = some.to(torch.int32)          # any order
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), softcap=cap, alibi_slopes=slopes, scale=scale,
                              q_lens=None if q_lens is None else _i32(q_lens), k_scales=ks, v_scales=vs, pages=pages)
    assert fa.check_device_status() == 0
    _check(q, kc, vc, ks, vs, table, lens, o, lse, cap, slopes, q_lens, scale, pages)


SHAPES = [([1], 1, 1, 1, 16), ([0], 4, 2, 1, 16), ([17], 8, 8, 1, 16), ([0, 1, 15, 16, 17, 0, 33, 0], 8, 2, 1, 16),
          ([500, 3, 1290], 4, 1, 1, 48), ([129, 64, 128], 16, 1, 1, 64), ([20, 9], 24, 1, 1, 32),
          ([5000], 4, 2, 1, 256), ([37, 700], 6, 2, 3, 32), ([4, 2, 0, 260], 8, 1, 5, 16), ([100], 40, 1, 2, 16),
          ([3000, 0, 17], 17, 1, 1, 32), ([33, 2, 900], 8, 1, 7, 16), ([4000], 32, 1, 1, 64)]


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,Hkv,T,page", SHAPES)
def test_lengths_heads_and_pages(store, dtype, d, lens, H, Hkv, T, page):
    _run(lens, H, Hkv, T, page, d, dtype, store, seed=sum(lens) + H)


@pytest.mark.parametrize("store,dtype", [("int8", "bf16"), ("e4m3", "fp16"), ("16", "bf16"), ("16", "fp16")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,Hkv,T,page", SHAPES)
@pytest.mark.parametrize("picks", [1, 5, 70])
def test_chosen_pages(store, dtype, d, lens, H, Hkv, T, page, picks):
    _run(lens, H, Hkv, T, page, d, dtype, store, seed=sum(lens) + H, picks=picks)


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("cap,alibi,scale", [(30.0, False, None), (0.0, True, None), (5.0, True, 0.5), (1e-3, False, None)])
def test_scores(store, cap, alibi, scale):
    _run([1, 250, 0, 3000], 8, 2, 2, 64, 128, "bf16", store, cap=cap, alibi=alibi, scale=scale, seed=3)
    _run([1, 250, 0, 3000], 4, 4, 1, 16, 64, "fp16", store, cap=cap, alibi=alibi, scale=scale, seed=4)
    _run([1, 250, 0, 3000], 4, 4, 3, 16, 64, "fp16", store, cap=cap, alibi=alibi, scale=scale, seed=5, picks=9)
    _run([1, 250, 0, 3000], 4, 4, 3, 48, 128, "bf16", "16", cap=cap, alibi=alibi, scale=scale, seed=5, picks=9)


def test_ragged_new_tokens():
    for store in ("int8", "e4m3"):
        for picks in (0, 4):
            _run([40, 3, 900, 0, 7], 4, 2, 6, 16, 64, "bf16", store, q_lens=[6, 2, 0, 6, 9], alibi=True, seed=5, picks=picks)
            _run([40, 3, 900, 0, 7, 2100], 16, 2, 5, 16, 128, "fp16", store, q_lens=[5, 2, 0, 5, 9, 3], cap=20.0, seed=6,
                 picks=picks)


def test_lists_with_gaps_and_strangers():
    """-1 and pages that the sequence does not have see nothing, wherever they stand; nothing chosen gives 0."""
    lens, page = [300, 70], 16
    kc, vc, ks, vs, table, g = _cache8(lens, 2, page, 64, "bf16", "int8", 7)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    pages = _i32([[[3, -1, 18, 7, -1], [-1, -1, -1, -1, -1]], [[19, 4, 2 ** 31 - 1, -2 ** 31, 0], [5, 0, -1, 1, 2]]])
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs, pages=pages)
    assert fa.check_device_status() == 0
    _check(q, kc, vc, ks, vs, table, lens, o, lse, pages=pages)
    assert not bool(o[0, 2:].any()) and bool(torch.isinf(lse[0, 2:]).all())


def test_all_pages_chosen_are_all_pages():
    lens, page = [2000, 33, 1], 16
    kc, vc, ks, vs, table, g = _cache8(lens, 2, page, 128, "bf16", "e4m3", 8)
    q = torch.randn((3, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    pages = torch.arange(table.shape[1], dtype=torch.int32, device="cuda").expand(3, 2, -1).contiguous()
    want = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs)
    got = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs, pages=pages)
    _check(q, kc, vc, ks, vs, table, lens, *got)
    assert torch.equal(want[0], got[0])


def test_ranges_of_queries_and_scales():
    """Queries and scales near the ends of their types' ranges; scales of a page far apart from the next one's."""
    lens, page, d = [200, 65], 16, 64
    kc, vc, ks, vs, table, g = _cache8(lens, 2, page, d, "bf16", "int8", 9)
    q = torch.randn((2, 4, 2, d), generator=g, device="cuda")
    for qs, kscale, vscale in ((2.0 ** 100, 2.0 ** -100, 1.0), (2.0 ** -100, 2.0 ** 90, 2.0 ** 60), (1.0, 1.0, 2.0 ** -60)):
        q2, k2, v2 = (q * qs).to(torch.bfloat16), ks * kscale, vs * vscale
        o, lse = fa.forward_paged(q2, kc, vc, table, _i32(lens), k_scales=k2, v_scales=v2)
        _check(q2, kc, vc, k2, v2, table, lens, o, lse)
    far = vs * torch.exp2(torch.randint(-30, 12, vs.shape, generator=g, device="cuda").float())
    q2 = q.to(torch.bfloat16)
    o, lse = fa.forward_paged(q2, kc, vc, table, _i32(lens), k_scales=ks, v_scales=far)
    _check(q2, kc, vc, ks, far, table, lens, o, lse)
    far[table[0, 2].item(), 1] = 0.0
    ks[table[0, 3].item(), 0] = 0.0
    o, lse = fa.forward_paged(q2, kc, vc, table, _i32(lens), k_scales=ks, v_scales=far)
    _check(q2, kc, vc, ks, far, table, lens, o, lse)


def test_nan_scales_show_where_their_page_is_seen():
    lens, page = [100, 40], 16
    for store in ("int8", "e4m3"):
        kc, vc, ks, vs, table, g = _cache8(lens, 2, page, 64, "bf16", store, 10)
        q = torch.randn((2, 4, 3, 64), generator=g, device="cuda").to(torch.bfloat16)
        want = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs)
        for scales in (ks, vs):
            at = table[0, 6].item()                     # tokens 96 to 99: rows 0 to 2 stand at 97 to 99
            was = scales[at, 1].clone()
            scales[at, 1] = float("nan")
            o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs)
            scales[at, 1] = was
            assert bool(torch.isnan(o[0, 2:]).all()) and bool(torch.isnan(lse[0, 2:]).all()) == (scales is ks)
            assert torch.equal(o[0, :2], want[0][0, :2]) and torch.equal(o[1], want[0][1])
        lens2 = [98, 40]                                # rows stand at 95, 96, 97: the first does not see the page
        for scales in (ks, vs):
            at = table[0, 6].item()
            was = scales[at, 1].clone()
            scales[at, 1] = float("nan")
            o, _ = fa.forward_paged(q, kc, vc, table, _i32(lens2), k_scales=ks, v_scales=vs)
            scales[at, 1] = was
            assert bool(torch.isfinite(o[0, 2:, 0]).all()) and bool(torch.isnan(o[0, 2:, 1:]).all())
        q[1, 0, 0, 5] = float("nan")
        o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), k_scales=ks, v_scales=vs)
        assert bool(torch.isnan(o[1, 0, 0]).all()) and bool(torch.isfinite(o[1, 0, 1:]).all()) and bool(torch.isfinite(o[1, 1:]).all())


def test_same_bits_layouts_graphs_streams_and_workspaces():
    lens = [3000, 5, 800]
    kc, vc, ks, vs, table, g = _cache8(lens, 2, 32, 128, "bf16", "e4m3", 8)
    q = torch.randn((3, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    n = _i32(lens)
    pages = torch.stack([torch.randperm(max(1, -(-x // 32)), generator=g, device="cuda")[torch.arange(20, device="cuda") % max(1, -(-x // 32))]
                         for x in lens]).to(torch.int32)[:, None].repeat(1, 2, 1)
    for extra in ({}, dict(pages=pages)):
        kw = dict(k_scales=ks, v_scales=vs, **extra)
        want = fa.forward_paged(q, kc, vc, table, n, **kw)
        for _ in range(3):
            got = fa.forward_paged(q, kc, vc, table, n, **kw)
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        both = torch.stack((kc.view(torch.uint8), vc.view(torch.uint8)), 1).transpose(2, 3).contiguous().view(kc.dtype)
        got = fa.forward_paged(q, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), table, n, **kw)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        ws = torch.full((fa.forward_paged_workspace_size(3, 8, 2, 1, 128, table.shape[1] * 32),), 255, dtype=torch.uint8, device="cuda")
        graphs = []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                out = fa.forward_paged(q, kc, vc, table, n, workspace=ws, **kw)
            graphs.append((gr, out))
        for _ in range(3):
            for gr, out in graphs:
                out[0].zero_()
                gr.replay()
                assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = [fa.forward_paged(q, kc, vc, table, n, stream=s, **kw) for s in (side, None, side)]
        torch.cuda.synchronize()
        assert all(torch.equal(x[0], want[0]) for x in got)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("store", ["int8", "e4m3"])
def test_short_sequences_in_wide_tables(store, d):
    """Few tiles, shared by all blocks of a call that is sized for many: blocks whose share holds no tile, or one."""
    for n in (1, 16, 33, 64, 65, 150, 160, 200, 330, 500):
        for T, lens in ((1, [n]), (2, [n, 0, 1, n])):
            kc, vc, ks, vs, table, g = _cache8(lens, 2, 16, d, "bf16", store, n)
            wide = torch.full((len(lens), 70), -1, dtype=torch.int32, device="cuda")
            wide[:, : table.shape[1]] = table
            q = torch.randn((len(lens), 4, T, d), generator=g, device="cuda").to(torch.bfloat16)
            ws = torch.randint(0, 256, (fa.forward_paged_workspace_size(len(lens), 4, 2, T, d, 70 * 16),), generator=g, device="cuda", dtype=torch.uint8)
            for _ in range(2):                           # and with what the call left
                o, lse = fa.forward_paged(q, kc, vc, wide, _i32(lens), k_scales=ks, v_scales=vs, workspace=ws)
                _check(q, kc, vc, ks, vs, table, lens, o, lse)
    assert fa.check_device_status() == 0


def test_one_workspace_for_calls_of_different_kinds():
    """16-bit, 8-bit and chosen pages in turn, captured and replayed in another order."""
    lens = [3000, 700]
    kc, vc, ks, vs, table, g = _cache8(lens, 2, 16, 128, "bf16", "int8", 12)
    k16, v16 = ((c.float() * s.nan_to_num()[..., None, None]).to(torch.bfloat16) for c, s in ((kc, ks), (vc, vs)))
    q = torch.randn((2, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    n = _i32(lens)
    pages = torch.arange(40, dtype=torch.int32, device="cuda").expand(2, 2, 40).contiguous()
    ws = torch.randint(0, 256, (fa.forward_paged_workspace_size(2, 8, 2, 1, 128, table.shape[1] * 16),), generator=g, device="cuda", dtype=torch.uint8)
    calls = [lambda w: fa.forward_paged(q, k16, v16, table, n, workspace=w),
             lambda w: fa.forward_paged(q, kc, vc, table, n, k_scales=ks, v_scales=vs, workspace=w),
             lambda w: fa.forward_paged(q, kc, vc, table, n, k_scales=ks, v_scales=vs, pages=pages, workspace=w),
             lambda w: fa.forward_paged(q, k16, v16, table, n, pages=pages, workspace=w)]
    want = [c(None) for c in calls]
    graphs = []
    for c in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = c(ws)
        graphs.append((gr, out))
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (1, 1, 3, 3), (2, 0, 2, 1)):
        for i in order:
            graphs[i][0].replay()
            assert torch.equal(graphs[i][1][0], want[i][0]) and torch.equal(graphs[i][1][1], want[i][1])
            got = calls[(i + 1) % 4](ws)
            assert torch.equal(got[0], want[(i + 1) % 4][0])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes."""
    pages = (1 << 32) // (8 * 64 * 128) + 40
    kc, vc = (torch.empty((pages, 8, 64, 128), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, 8), 0.02, device="cuda") for _ in range(2))
    at = torch.tensor([pages - 1, 3, pages - 20, 0], device="cuda")
    for c in (kc, vc):
        c[at] = torch.randint(-127, 128, (4, 8, 64, 128), dtype=torch.int8, device="cuda")
    table = at.to(torch.int32).repeat(2, 1).contiguous()
    q = torch.randn((2, 8, 1, 128), device="cuda").to(torch.bfloat16)
    lens = _i32([250, 130])
    o, lse = fa.forward_paged(q, kc, vc, table, lens, k_scales=ks, v_scales=vs)
    _check(q, kc, vc, ks, vs, table, [250, 130], o, lse)
    k, v = (torch.randn((2, 8, 1, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    table[1] = _i32([5, pages - 3, pages - 7, 9])
    bounds, unit = torch.zeros((pages, 8, 2, 128), dtype=torch.int8, device="cuda"), torch.zeros((pages, 8), device="cuda")
    fa.append_paged(k, v, kc, vc, table, _i32([193, 129]), k_scales=ks, v_scales=vs, k_bounds=bounds, bound_scales=unit)
    for b, page in ((0, 0), (1, pages - 7)):
        for name, x, c, sc in (("k", k, kc, ks), ("v", v, vc, vs)):
            two = torch.tensor([power(float(y.abs().max()), 127.0) for y in x[b, :, 0]], device="cuda")
            assert torch.equal(sc[page], two)
            assert torch.equal(c[page, :, 0].float(), torch.round(x[b, :, 0].float() / two[:, None]))
        assert torch.equal(bounds[page, :, 0].float(), torch.floor(k[b, :, 0].float() / unit[page][:, None]))
    assert fa.check_device_status() == 0


# ---- writing -------------------------------------------------------------------------------------

class Pages:
    """Pages written one call after another, as the definition has it, in 64 bits."""

    def __init__(self, k, v, ks, vs, bounds, unit, store):
        self.c = [None if x is None else x.double().cpu() for x in (k, v, ks, vs, bounds, unit)]
        self.store = store

    def write(self, table, lens, new, k, v):
        kc, vc, ks, vs, bounds, unit = self.c
        page = kc.shape[2]
        for b, n in enumerate(lens):
            begin = n - new[b]
            for p in range(max(begin, 0) // page, -(-n // page) if new[b] else 0):
                first, end = max(begin, 0, p * page), min(n, (p + 1) * page)
                at, kept = int(table[b, p]), first - p * page
                for g in range(kc.shape[1]):
                    for x, c, sc in ((k, kc, ks), (v, vc, vs)):
                        x = x[b, g, first - begin: end - begin].double().cpu()
                        top = float(x.abs().max())
                        if self.store != "16":
                            need = power(top, LARGEST[self.store])
                            was = float(sc[at, g])
                            now = max(was, need) if kept else need
                            if kept and now > was:
                                c[at, g, :kept] = grid(c[at, g, :kept] * (was / now), self.store)
                            sc[at, g] = now
                            c[at, g, kept: end - p * page] = grid(x / now, self.store)
                        else:
                            c[at, g, kept: end - p * page] = x
                        if c is kc and bounds is not None:
                            need = power(top, 127.0)
                            was = float(unit[at, g])
                            now = max(was, need) if kept else need
                            lo, hi = torch.floor(x.amin(0) / now), torch.ceil(x.amax(0) / now)
                            if kept:
                                lo = torch.minimum(lo, torch.floor(bounds[at, g, 0] * (was / now)))
                                hi = torch.maximum(hi, torch.ceil(bounds[at, g, 1] * (was / now)))
                            bounds[at, g, 0], bounds[at, g, 1], unit[at, g] = lo, hi, now

    def check(self, *got):
        for name, x, y in zip(("k", "v", "k_scales", "v_scales", "bounds", "bound_scales"), got, self.c):
            if x is not None:
                x = x.double().cpu()
                same = (x == y) | (torch.isnan(x) & torch.isnan(y))
                assert bool(same.all()), (name, int((~same).sum()), x[~same][:5], y[~same][:5])


def _stores(n, Hkv, page, d, dtype, store, bounds):
    kind = TYPES[dtype] if store == "16" else STORES[store]
    kc, vc = (torch.zeros((n, Hkv, page, d), dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (None if store == "16" else torch.full((n, Hkv), 8.0, device="cuda") for _ in range(2))
    kb = torch.full((n, Hkv, 2, d), 99, dtype=torch.int8, device="cuda") if bounds else None
    bs = torch.full((n, Hkv), 2.0 ** 30, device="cuda") if bounds else None
    return kc, vc, ks, vs, kb, bs


@pytest.mark.parametrize("store,bounds", [("int8", False), ("int8", True), ("e4m3", False), ("e4m3", True), ("16", True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,page,T", [(64, 16, 1), (128, 48, 3), (64, 64, 200), (128, 64, 150), (128, 256, 300), (64, 32, 17),
                                      (128, 16, 9), (64, 512, 700)])
def test_append_is_exact(store, bounds, dtype, d, page, T):
    """Several writes to the same pages: later tokens larger and smaller than the ones before."""
    Hkv, B = 3, 4
    g = torch.Generator(device="cuda").manual_seed(T + d)
    width = -(-4 * (T + 3) // page) + 1
    kc, vc, ks, vs, kb, bs = state = _stores(B * width + 2, Hkv, page, d, dtype, store, bounds)
    ref = Pages(*state, store)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).reshape(B, width)
    lens = [0, 3, 0, 0]
    for size, new in ((1.0, [T, T, 0, min(T, 2)]), (0.01, [1, T, T, T]), (30.0, [T // 2 + 1, 0, T, 1]), (1e-3, [1, 1, 1, 1])):
        lens = [a + b for a, b in zip(lens, new)]
        kv = (torch.randn((B, T, 2 * Hkv, d), generator=g, device="cuda") * size *
              torch.exp2(torch.randint(-3, 3, (B, T, 2 * Hkv, 1), generator=g, device="cuda"))).to(TYPES[dtype])
        k, v = (x.transpose(1, 2) for x in kv.split(Hkv, 2))
        assert fa.append_paged(k, v, kc, vc, table, _i32(lens), q_lens=_i32(new), k_scales=ks, v_scales=vs, k_bounds=kb,
                               bound_scales=bs) is None
        assert fa.check_device_status() == 0
        ref.write(table, lens, new, k, v)
        ref.check(*state)


@pytest.mark.parametrize("store,bounds", [("int8", True), ("e4m3", True), ("e4m3", False), ("16", True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,page,T,lens,new", [
    (64, 64, 16, 1, [1, 30, 0], [1, 1, 0]), (128, 32, 48, 5, [5, 30, 700], [5, 2, 0]), (128, 128, 64, 150, [150, 30, 700], [150, 7, 140]),
    (64, 16, 128, 300, [300, 2, 310], [300, 9, 300])])
def test_append_turns_keys_and_queries(store, bounds, interleaved, d, rot, page, T, lens, new):
    """A code is off by half a step of its own and by the rotation's error; the scale is that of the turned keys."""
    Hkv, H, B = 2, 6, 3
    g = torch.Generator(device="cuda").manual_seed(T + d)
    width = -(-max(lens) // page)
    kc, vc, ks, vs, kb, bs = _stores(B * width, Hkv, page, d, "bf16", store, bounds)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).reshape(B, width)
    qkv = torch.randn((B, T, H + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], 2))
    inv_freq = fa.rotary_frequencies(rot)[0]
    q2 = fa.append_paged(k, v, kc, vc, table, _i32(lens), q=q, q_lens=_i32(new), inv_freq=inv_freq, interleaved=interleaved,
                         mscale=1.1, k_scales=ks, v_scales=vs, k_bounds=kb, bound_scales=bs)
    assert fa.check_device_status() == 0
    plain = fa.append_paged(k, v, *(torch.zeros((B * width, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)),
                            table, _i32(lens), q=q, q_lens=_i32(new), inv_freq=inv_freq, interleaved=interleaved, mscale=1.1)
    assert torch.equal(q2, plain)
    half_step = {"int8": lambda y: torch.full_like(y, 0.5), "e4m3": lambda y: 2.0 ** -4 * y.abs() + 2.0 ** -10}
    for b, n in enumerate(lens):
        c = min(new[b], T)
        pos = n - c + torch.arange(T, device="cuda")
        there = (torch.arange(T, device="cuda") < c) & (pos >= 0)
        p = pos[there]
        if p.numel() == 0:
            continue
        ref, size = _turn(k[b:b + 1][:, :, there], p, inv_freq, interleaved, 1.1)
        err = (6e-7 * size)[0]
        for x, e, cache, scales in ((ref[0], err, kc, ks), (v[b][:, there].double(), 0.0, vc, vs)):
            got = cache[table[b].long()[p // page], :, p % page].double().transpose(0, 1)
            if store == "16":
                assert bool(((got - x).abs() <= 2.0 ** -8 * x.abs() * 1.01 + e).all())
                continue
            unit = scales[table[b].long()[p // page]].double().T[..., None]
            assert bool(((got - x / unit).abs() <= half_step[store](x / unit) + e / unit).all())
            for i in p.div(page, rounding_mode="floor").unique().tolist():
                for h in range(Hkv):
                    top = float(x[h][p // page == i].abs().max())
                    # a page that held tokens keeps its scale, the 8 of _stores, until a larger one is needed
                    was = 8.0 if i * page < int(p[0]) else 0.0
                    assert float(scales[table[b, i].long(), h]) in (max(was, power(top * (1 - 2e-6), LARGEST[store])),
                                                                    max(was, power(top * (1 + 2e-6), LARGEST[store])))
        if bounds:
            for i in p.div(page, rounding_mode="floor").unique().tolist():
                at, here = table[b, i].long(), p // page == i
                unit = bs[at].double()[:, None]
                lo, hi = kb[at].double().unbind(1)
                x, slack = ref[0][:, here], err[:, here].amax(1) + (2.0 ** -8 * ref[0][:, here].abs().amax(1) if store == "16" else 0.0)
                mn, mx = x.amin(1), x.amax(1)
                assert bool(((lo * unit <= mn + slack) & (hi * unit >= mx - slack)).all())
                if i * page >= int(p[0]):               # no bounds of earlier tokens among them
                    assert bool(((lo * unit >= mn - slack - unit) & (hi * unit <= mx + slack + unit)).all())


def test_extreme_values_and_zeros():
    g = torch.Generator(device="cuda").manual_seed(1)
    for store in ("int8", "e4m3"):
        for dtype, sizes in (("bf16", (0.0, 2.0 ** -133, 2.0 ** -110, 1.0, 2.0 ** 127)), ("fp16", (0.0, 2.0 ** -24, 2.0 ** -14, 30000.0))):
            for size in sizes:
                state = _stores(4, 2, 16, 64, dtype, store, True)
                ref = Pages(*state, store)
                kc, vc, ks, vs, kb, bs = state
                table = _i32([[2, 0], [1, 3]])
                k, v = ((torch.rand((2, 2, 20, 64), generator=g, device="cuda") * 2 - 1).mul(size).to(TYPES[dtype]) for _ in range(2))
                fa.append_paged(k, v, kc, vc, table, _i32([20, 20]), q_lens=_i32([20, 9]), k_scales=ks, v_scales=vs, k_bounds=kb, bound_scales=bs)
                ref.write(table, [20, 20], [20, 9], k, v)
                # the second sequence's first page keeps what it held: its scale is the caller's 8
                ref.check(*state)


def test_what_is_not_finite_shows_until_the_page_begins_anew():
    for store in ("int8", "e4m3"):
        for bad in (float("nan"), float("inf"), -float("inf")):
            kc, vc, ks, vs, kb, bs = _stores(3, 2, 16, 64, "bf16", store, True)
            table, one = _i32([[1, 2]]), torch.ones((1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
            kw = dict(k_scales=ks, v_scales=vs, k_bounds=kb, bound_scales=bs)
            fa.append_paged(one, one, kc, vc, table, _i32([1]), **kw)
            broken = one.clone()
            broken[0, 1, 0, 9] = bad
            fa.append_paged(broken, one, kc, vc, table, _i32([2]), **kw)
            assert bool(torch.isnan(ks[1, 1])) and bool(torch.isnan(bs[1, 1])) and bool(torch.isfinite(ks[1, 0]))
            assert bool(torch.isfinite(vs[1]).all())
            fa.append_paged(one, one, kc, vc, table, _i32([3]), **kw)
            assert bool(torch.isnan(ks[1, 1])) and not bool(torch.isnan(kc.float()).any())
            o, lse = fa.forward_paged(one, kc, vc, table, _i32([3]), k_scales=ks, v_scales=vs)
            assert bool(torch.isnan(o[0, 1]).all()) and bool(torch.isfinite(o[0, 0]).all())
            fa.append_paged(one, one, kc, vc, table, _i32([1]), **kw)
            assert bool(torch.isfinite(ks[1]).all()) and bool(torch.isfinite(bs[1]).all())


def test_nothing_else_is_written():
    """Pages without new tokens, slots behind the last one, padding and places below 0."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for T in (2, 40):
        kc, vc, ks, vs, kb, bs = state = _stores(12, 2, 16, 64, "bf16", "int8", True)
        for c in (kc, vc):
            c.copy_(torch.randint(-127, 128, c.shape, generator=g, device="cuda"))
        before = [x.clone() for x in state]
        table = _i32([[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]])
        k, v = (torch.randn((4, 2, T, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        lens, new = [17, 1, 0, 20], [1, 2, 1, 0]
        fa.append_paged(k, v, kc, vc, table, _i32(lens), q_lens=_i32(new), k_scales=ks, v_scales=vs, k_bounds=kb, bound_scales=bs)
        assert fa.check_device_status() == 0
        assert torch.equal(kc[1, :, 1:], before[0][1, :, 1:]) and torch.equal(vc[3, :, 1:], before[1][3, :, 1:])
        for x, y in zip(state, before):
            assert not torch.equal(x[1], y[1]) and not torch.equal(x[3], y[3])
            x[1], x[3] = y[1], y[3]
            assert torch.equal(x, y)


def test_bad_pages_and_lengths_are_reported():
    kc, vc, ks, vs, table, g = _cache8([100, 50], 2, 16, 64, "bf16", "int8", 3)
    kb, bs = torch.zeros((kc.shape[0], 2, 2, 64), dtype=torch.int8, device="cuda"), torch.ones((kc.shape[0], 2), device="cuda")
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    k, v = q[:, :2].contiguous(), q[:, 2:].contiguous()
    n = _i32([100, 50])
    kw = dict(k_scales=ks, v_scales=vs)
    pages = _i32([[[0, 1, 2, 3], [6, 5, 1, 0]], [[0, 1, 2, 3], [3, 2, 1, 0]]])
    want = [fa.forward_paged(q, kc, vc, table, n, pages=p, **kw)[0] for p in (None, pages)]
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 3] = bad                                     # tokens 48, 49 of the second sequence
        for p, w in zip((None, pages), want):
            o, _ = fa.forward_paged(q, kc, vc, t, n, pages=p, **kw)
            assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
            assert torch.equal(o[0], w[0])
        state = [x.clone() for x in (kc, vc, ks, vs, kb, bs)]
        fa.append_paged(k, v, state[0], state[1], t, n, k_scales=state[2], v_scales=state[3], k_bounds=state[4], bound_scales=state[5])
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
        at = table[0, 6].item()
        for x, y in zip(state, (kc, vc, ks, vs, kb, bs)):
            if x.dtype == torch.float32:
                x, y = x.nan_to_num(nan=-1.0), y.nan_to_num(nan=-1.0)
            x[at] = y[at]
            assert torch.equal(x, y)                      # the second sequence wrote nothing
        fa.select_pages(q, kb, bs, t, n, 2, 16)
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
    long = _i32([100, table.shape[1] * 16 + 1])
    for p, w in zip((None, pages), want):
        o, lse = fa.forward_paged(q, kc, vc, table, long, pages=p, **kw)
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(o[0], w[0]) and not bool(o[1].any()) and bool(torch.isinf(lse[1]).all())
    fa.append_paged(k, v, kc, vc, table, long, **kw)
    assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
    assert bool((fa.select_pages(q, kb, bs, table, long, 2, 16)[1] == -1).all())
    assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG


def test_refusals():
    kc, vc, ks, vs, table, g = _cache8([100, 50], 2, 16, 64, "bf16", "int8", 3)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    n, kw = _i32([100, 50]), dict(k_scales=ks, v_scales=vs)
    with pytest.raises(ValueError, match="k_scales"):
        fa.forward_paged(q, kc, vc, table, n)
    with pytest.raises(ValueError, match="v_scales"):
        fa.forward_paged(q, kc, vc, table, n, k_scales=ks)
    with pytest.raises(ValueError, match="k_scales"):
        fa.forward_paged(q, kc, vc, table, n, k_scales=ks.double(), v_scales=vs)
    with pytest.raises(ValueError, match="v_scales"):
        fa.forward_paged(q, kc, vc, table, n, k_scales=ks, v_scales=vs.T)
    with pytest.raises(ValueError, match="CUDA"):
        fa.forward_paged(q, kc, vc, table, n, k_scales=ks.cpu(), v_scales=vs)
    with pytest.raises(ValueError, match="must be torch.int8"):
        fa.forward_paged(q, kc, vc.view(torch.float8_e4m3fn), table, n, **kw)
    with pytest.raises(ValueError, match="no scales"):
        fa.forward_paged(q, kc.bfloat16(), vc.bfloat16(), table, n, **kw)
    with pytest.raises(ValueError, match="k_cache"):
        fa.forward_paged(q, kc.half(), vc.half(), table, n)
    for bad in (torch.zeros((2, 2, 0)), torch.zeros((2, 4, 3)), torch.zeros((2, 2))):
        with pytest.raises(ValueError, match="pages"):
            fa.forward_paged(q, kc, vc, table, n, pages=bad.int().cuda(), **kw)
    with pytest.raises(ValueError, match="pages"):
        fa.forward_paged(q, kc, vc, table, n, pages=torch.zeros((2, 2, 3), device="cuda"), **kw)
    with pytest.raises(ValueError, match="k_bounds"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, k_bounds=torch.zeros((3, 2, 2, 64), dtype=torch.int8, device="cuda"), bound_scales=ks, **kw)
    kb = torch.zeros((kc.shape[0], 2, 2, 64), dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError, match="bound_scales"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, k_bounds=kb, **kw)
    with pytest.raises(ValueError, match="without k_bounds"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, bound_scales=ks, **kw)
    with pytest.raises(ValueError, match="overlap"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, k_scales=ks, v_scales=ks)
    with pytest.raises(ValueError, match="overlap"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, k_bounds=kb, bound_scales=vs, **kw)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, kc, table, n, **kw)
