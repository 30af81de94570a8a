"""The paged cache on the GPU: writing new tokens (keys and queries rotated), and attention of the new
tokens over the pages, against 64-bit formulas (bounds derived in scored_reference.py)."""
import math

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from scored_reference import assert_within, head_forward
from test_rotary_gpu import _check as check_turned

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(lens, Hkv, page, d, dtype, seed=0, fill=None, spare=3):
    """Pages in shuffled order; what no sequence uses is `fill` (NaN, say)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need, default=0))), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.randn((total, Hkv, page, d), generator=g, device="cuda").to(TYPES[dtype]) for _ in range(2))
    at = 0
    used = torch.zeros((total, page), dtype=torch.bool, device="cuda")
    for b, (n, w) in enumerate(zip(lens, need)):
        table[b, :w] = order[at:at + w]
        at += w
        for i in range(w):
            used[table[b, i].item(), : min(page, n - i * page)] = True
    if fill is not None:
        for c in (kc, vc):
            c.masked_fill_(~used[:, None, :, None], fill)
    return kc, vc, table, g


def _slopes(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _check(q, kc, vc, table, lens, o, lse, cap=0.0, slopes=None, q_lens=None, scale=None):
    B, H, T, d = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    for b, n in enumerate(lens):
        new = T if q_lens is None else min(max(q_lens[b], 0), T)
        pages = table[b, : -(-n // page)].long()
        kpos = torch.arange(n, device="cuda")
        qpos = n - new + torch.arange(T, device="cuda")
        exists = (torch.arange(T, device="cuda") < new)[:, None]
        allowed = (kpos[None, :] <= qpos[:, None]) & exists
        dist = (qpos[:, None] - kpos[None, :]).abs().double()
        for h in range(H):
            g = h // (H // Hkv)
            k, v = (c[pages, g].reshape(-1, d)[:n].double() for c in (kc, vc))
            ro, rl, ot, lt = head_forward(q[b, h].double(), k, v, allowed, dist, scale, cap,
                                          0.0 if slopes is None else float(slopes[h]), u,
                                          2.0 ** -25 if q.dtype == torch.float16 else 0.0)
            assert_within(f"O {b} {h}", o[b, h], ro, ot)
            assert_within(f"LSE {b} {h}", lse[b, h], rl, lt)


def _run(lens, H, Hkv, T, page, d, dtype, cap=0.0, alibi=False, q_lens=None, scale=None, seed=0):
    kc, vc, table, g = _cache(lens, Hkv, page, d, dtype, seed, fill=float("nan"))
    q = (torch.randn((len(lens), H, T, d), generator=g, device="cuda") * 2).to(TYPES[dtype])
    slopes = _slopes(H) if alibi else None
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), softcap=cap, alibi_slopes=slopes, scale=scale,
                              q_lens=None if q_lens is None else _i32(q_lens))
    assert fa.check_device_status() == 0
    _check(q, kc, vc, table, lens, o, lse, cap, slopes, q_lens, scale)
    return q, kc, vc, table, o, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,Hkv,T,page", [
    ([1], 1, 1, 1, 16), ([0], 4, 2, 1, 16), ([17], 8, 8, 1, 16), ([0, 1, 15, 16, 17, 0, 33, 0], 8, 2, 1, 16),
    ([500, 3, 1290], 4, 1, 1, 48), ([129, 64, 128], 16, 1, 1, 64), ([20, 9], 24, 1, 1, 32),
    ([5000], 4, 2, 1, 256), ([37, 700], 6, 2, 3, 32), ([4, 2, 0, 260], 8, 1, 5, 16), ([100], 40, 1, 2, 16),
    ([3000, 0, 17], 17, 1, 1, 32), ([33, 2, 900], 8, 1, 7, 16), ([4000], 32, 1, 1, 64)])
def test_lengths_heads_and_pages(dtype, d, lens, H, Hkv, T, page):
    _run(lens, H, Hkv, T, page, d, dtype, seed=sum(lens) + H)


@pytest.mark.parametrize("cap,alibi,scale", [(30.0, False, None), (0.0, True, None), (5.0, True, 0.5), (1e-3, False, None),
                                             (1e6, False, None)])
def test_scores(cap, alibi, scale):
    _run([1, 250, 0, 3000], 8, 2, 2, 64, 128, "bf16", cap=cap, alibi=alibi, scale=scale, seed=3)
    _run([1, 250, 0, 3000], 4, 4, 1, 16, 64, "fp16", cap=cap, alibi=alibi, scale=scale, seed=4)


def test_ragged_new_tokens():
    _run([40, 3, 900, 0, 7], 4, 2, 6, 16, 64, "bf16", q_lens=[6, 2, 0, 6, 9], alibi=True, seed=5)
    _run([40, 3, 900, 0, 7, 2100], 16, 2, 5, 16, 128, "bf16", q_lens=[5, 2, 0, 5, 9, 3], cap=20.0, alibi=True, seed=6)


def test_many_sequences():
    """More sequences than a warp scans at once, most of them short, one long."""
    lens = [(7 * i) % 61 for i in range(200)] + [9000]
    _run(lens, 4, 2, 1, 16, 64, "bf16", seed=6)


def test_same_bits_every_time_and_any_layout():
    lens = [3000, 5, 800]
    kc, vc, table, g = _cache(lens, 2, 32, 128, "bf16", 8, fill=float("inf"))
    q = torch.randn((3, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens))
    for _ in range(3):
        o2, lse2 = fa.forward_paged(q, kc, vc, table, _i32(lens))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # pages with keys and values in turn, tokens before heads
    both = torch.stack((kc, vc), 1).transpose(2, 3).contiguous()          # [pages, 2, page, Hkv, d]
    k2, v2 = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    wide = torch.full((3, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    o2, lse2 = fa.forward_paged(q, k2, v2, wide[:, : table.shape[1]], _i32(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa.check_device_status() == 0


def test_shared_pages_and_offsets_past_32_bits():
    """Two sequences over the same pages; a cache of more than 2^31 values."""
    pages = (1 << 31) // (8 * 64 * 128) + 40
    kc, vc = (torch.empty((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = torch.tensor([pages - 1, 3, pages - 20, 0], device="cuda")
    for c in (kc, vc):
        c[at] = torch.randn((4, 8, 64, 128), device="cuda").to(torch.bfloat16)
    table = at.to(torch.int32).repeat(2, 1).contiguous()
    q = torch.randn((2, 8, 1, 128), device="cuda").to(torch.bfloat16)
    o, lse = fa.forward_paged(q, kc, vc, table, _i32([250, 130]))
    _check(q, kc, vc, table, [250, 130], o, lse)
    assert fa.check_device_status() == 0


def test_captured_call_follows_the_lengths():
    """A captured decode step replays with the lengths the device holds then; two graphs have their
    own workspaces."""
    lens = [300, 40]
    kc, vc, table, g = _cache([600, 600], 2, 16, 64, "bf16", 9)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    n = _i32(lens)
    fa.forward_paged(q, kc, vc, table, n)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = fa.forward_paged(q, kc, vc, table, n)
        graphs.append((gr, out))
    for new in ([300, 40], [600, 0], [1, 599]):
        n.copy_(_i32(new))
        for gr, _ in graphs:
            gr.replay()
        want = fa.forward_paged(q, kc, vc, table, n)
        for _, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        _check(q, kc, vc, table, new, *want)


@pytest.mark.parametrize("fill", [0, 255, None])
def test_workspaces_hold_anything(fill):
    """What a workspace holds on entry does not matter; calls and two captured graphs may share one."""
    lens = [5000, 300]
    kc, vc, table, g = _cache(lens, 2, 16, 64, "bf16", 11)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    n = _i32(lens)
    want = fa.forward_paged(q, kc, vc, table, n)
    need = fa.forward_paged_workspace_size(2, 4, 2, 1, 64, table.shape[1] * 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for i in range(5):
        if i != 2:                                # once: what the last call left
            ws.random_(0, 256) if fill is None else ws.fill_(fill)
        got = fa.forward_paged(q, kc, vc, table, n, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = fa.forward_paged(q, kc, vc, table, n, workspace=ws)
        graphs.append((gr, out))
    for _ in range(3):
        for gr, out in graphs:
            out[0].zero_()
            gr.replay()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once():
    lens = [4000, 1000]
    kc, vc, table, g = _cache(lens, 4, 64, 128, "bf16", 10)
    qs = [torch.randn((2, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [fa.forward_paged(q, kc, vc, table, _i32(lens)) for q in qs]
    n = _i32(lens)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [fa.forward_paged(q, kc, vc, table, n, stream=s) for q, s in zip(qs, side)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- writing -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (128, 128), (64, 0)])
@pytest.mark.parametrize("lens,new,T,page", [([1], None, 1, 16), ([20, 16, 0, 33], None, 1, 16),
                                             ([100, 7, 63, 64], [37, 0, 40, 5], 40, 48),
                                             ([300, 2], [300, 9], 300, 64)])
def test_append(dtype, interleaved, d, rot, lens, new, T, page):
    Hkv, H, B = 2, 6, len(lens)
    kc, vc, table, g = _cache(lens, Hkv, page, d, dtype, T + d)
    k0, v0 = kc.clone(), vc.clone()
    # projections leave [B, T, heads, d]; q, k, v cut from one tensor
    qkv = torch.randn((B, T, H + 2 * Hkv, d), generator=g, device="cuda").to(TYPES[dtype])
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], 2))
    inv_freq = fa.rotary_frequencies(rot)[0] if rot else None
    q2 = fa.append_paged(k, v, kc, vc, table, _i32(lens), q=q, q_lens=None if new is None else _i32(new),
                         inv_freq=inv_freq, interleaved=interleaved, mscale=1.1)
    assert fa.check_device_status() == 0
    turn = inv_freq if rot else torch.zeros(0, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        c = T if new is None else min(new[b], T)
        pos = n - c + torch.arange(T, device="cuda")
        there = (torch.arange(T, device="cuda") < c) & (pos >= 0)
        assert not bool(q2[b][:, ~there].any())
        p = pos[there]
        if p.numel() == 0:
            continue
        pages = table[b].long()[p // page]
        check_turned(q2[b:b + 1][:, :, there], q[b:b + 1][:, :, there], p, turn, interleaved, 1.1)
        got = kc[pages, :, p % page].transpose(0, 1)[None]
        check_turned(got, k[b:b + 1][:, :, there], p, turn, interleaved, 1.1)
        assert torch.equal(vc[pages, :, p % page].transpose(0, 1), v[b][:, there])
        for now, old in ((kc, k0), (vc, v0)):          # nothing else is written
            old[pages, :, p % page] = now[pages, :, p % page]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_without_queries_and_in_place():
    kc, vc, table, g = _cache([30, 5], 2, 16, 64, "bf16", 1)
    k, v = (torch.randn((2, 2, 1, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    inv_freq, _ = fa.rotary_frequencies(64)
    n = _i32([30, 5])
    k1, v1 = kc.clone(), vc.clone()
    assert fa.append_paged(k, v, kc, vc, table, n, inv_freq=inv_freq) is None
    q2 = fa.append_paged(k, v, k1, v1, table, n, q=q, inv_freq=inv_freq)
    assert torch.equal(kc, k1) and torch.equal(vc, v1)
    assert fa.append_paged(k, v, k1, v1, table, n, q=q, inv_freq=inv_freq, q_out=q) is q
    assert torch.equal(q, q2)


def test_nothing_to_do():
    """Empty batches, no new tokens, tables without entries."""
    kc, vc, table, g = _cache([16], 2, 16, 64, "bf16", 1)
    q = torch.zeros((0, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.forward_paged(q, kc, vc, table[:0], _i32([]))
    assert o.shape == q.shape and lse.shape == (0, 4, 1)
    assert fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table[:0], _i32([]), q=q).shape == q.shape
    q = torch.zeros((1, 4, 0, 64), dtype=torch.bfloat16, device="cuda")
    assert fa.forward_paged(q, kc, vc, table, _i32([16]))[0].shape == q.shape
    q = torch.ones((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.forward_paged(q, kc, vc, table[:, :0], _i32([0]))
    assert not bool(o.any()) and bool(torch.isinf(lse).all())
    assert fa.check_device_status() == 0
    fa.forward_paged(q, kc, vc, table[:, :0], _i32([1]))
    assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG


def test_a_decoder_reads_what_it_wrote():
    """Prompt, then tokens one by one and drafted together: every step's attention over the cache
    equals attention over all keys so far."""
    H, Hkv, d, page, B = 4, 2, 64, 16, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.full((20, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.randperm(20, generator=g, device="cuda").to(torch.int32).reshape(B, 10)
    inv_freq, _ = fa.rotary_frequencies(32)
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    all_k, all_v = ([torch.zeros((Hkv, 0, d), device="cuda", dtype=torch.bfloat16) for _ in range(B)] for _ in range(2))
    for T, counts in ((50, [50, 31]), (1, [1, 1]), (1, [1, 1]), (4, [4, 2]), (1, [1, 1])):
        q, k, v = (torch.randn((B, h, T, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv))
        new = _i32(counts)
        n += new
        q2 = fa.append_paged(k, v, kc, vc, table, n, q=q, q_lens=new, inv_freq=inv_freq)
        o, lse = fa.forward_paged(q2, kc, vc, table, n, q_lens=new, softcap=20.0)
        assert fa.check_device_status() == 0
        for b in range(B):
            pos = (n[b] - new[b] + torch.arange(T, device="cuda")).to(torch.int32)
            kr = fa.rotary(k[b], pos, inv_freq)
            all_k[b] = torch.cat((all_k[b], kr[:, : counts[b]]), 1)
            all_v[b] = torch.cat((all_v[b], v[b][:, : counts[b]]), 1)
            allowed = torch.arange(int(n[b]), device="cuda")[None, :] <= pos[:, None]
            allowed &= (torch.arange(T, device="cuda") < counts[b])[:, None]
            for h in range(H):
                ro, rl, ot, lt = head_forward(fa.rotary(q[b], pos, inv_freq)[h].double(), all_k[b][h // 2].double(),
                                              all_v[b][h // 2].double(), allowed, allowed.double(), d ** -0.5, 20.0, 0.0,
                                              2.0 ** -8)
                assert_within("O", o[b, h], ro, ot)
                assert_within("LSE", lse[b, h], rl, lt)


# ---- refusals ------------------------------------------------------------------------------------

def test_bad_pages_and_lengths_are_reported():
    """Table entries and lengths outside their contract are not followed; the status tells."""
    kc, vc, table, g = _cache([100, 50], 2, 16, 64, "bf16", 3)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    k, v = q[:, :2].contiguous(), q[:, 2:].contiguous()
    n = _i32([100, 50])
    want, _ = fa.forward_paged(q, kc, vc, table, n)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 3] = bad                                     # tokens 48, 49 of the second sequence
        o, _ = fa.forward_paged(q, kc, vc, t, n)
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(o[0], want[0])
        k1, v1 = kc.clone(), vc.clone()
        fa.append_paged(k, v, k1, v1, t, n)
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
        page, slot = int(table[0, 99 // 16]), 99 % 16
        assert torch.equal(k1[page, :, slot], k[0, :, 0])
        k1[page, :, slot] = kc[page, :, slot]
        assert torch.equal(k1, kc)                        # the second sequence wrote nothing
    long = _i32([100, table.shape[1] * 16 + 1])
    o, lse = fa.forward_paged(q, kc, vc, table, long)
    assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
    assert torch.equal(o[0], want[0]) and not bool(o[1].any()) and bool(torch.isinf(lse[1]).all())
    fa.append_paged(k, v, kc, vc, table, long)
    assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
    o, lse = fa.forward_paged(q, kc, vc, table, _i32([100, -5]))
    assert fa.check_device_status() == 0 and not bool(o[1].any())


def test_refusals():
    kc, vc, table, g = _cache([100, 50], 2, 16, 64, "bf16", 3)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    n = _i32([100, 50])
    with pytest.raises(ValueError, match="contiguous bf16"):
        fa.forward_paged(q.float(), kc, vc, table, n)
    with pytest.raises(ValueError, match="contiguous bf16"):
        fa.forward_paged(q.transpose(0, 1), kc, vc, table, n)
    with pytest.raises(ValueError, match="same shape and strides"):
        fa.forward_paged(q, kc, vc.transpose(1, 2).contiguous().transpose(1, 2), table, n)
    with pytest.raises(ValueError, match="block_table"):
        fa.forward_paged(q, kc, vc, table.long(), n)
    with pytest.raises(ValueError, match="kv_lens"):
        fa.forward_paged(q, kc, vc, table, n[:1])
    with pytest.raises(ValueError, match="dividing"):
        fa.forward_paged(q[:, :3].contiguous(), kc, vc, table, n)
    with pytest.raises(ValueError, match="alibi_slopes"):
        fa.forward_paged(q, kc, vc, table, n, alibi_slopes=_slopes(3))
    with pytest.raises(ValueError, match="overlap"):
        fa.forward_paged(q, kc, vc, table, n, o=q)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.forward_paged(q, kc, vc, table, n, softcap=-1.0)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.forward_paged(q, kc, vc, table, n, softcap=float("inf"))
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.forward_paged(q, kc, vc, table, n, scale=0.0)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        wide = torch.zeros((2, 40), dtype=torch.int32, device="cuda")
        fa.forward_paged(q, kc, vc, wide, n, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.forward_paged(q, kc[:, :, :8], vc[:, :, :8], table, n)          # pages of 8 tokens
    with pytest.raises(ValueError, match="q_out"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n, q_out=q)
    with pytest.raises(ValueError, match="overlap"):
        fa.append_paged(q[:, :2].contiguous(), q[:, 2:], kc, vc, table, n, q=q.clone(), q_out=q)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):                   # pages that share memory
        fa.append_paged(q[:, :2], q[:, 2:], kc[:1].expand(5, 2, 16, 64), vc[:1].expand(5, 2, 16, 64), table, n)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):                   # keys and values in one place
        fa.append_paged(q[:, :2], q[:, 2:], kc, kc, table, n)
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.append_paged(q[:, :2], q[:, 2:], kc, vc, table, n,
                        inv_freq=torch.ones(40, dtype=torch.float64, device="cuda"))
