"""The choice of pages by the bounds of their keys, and pages assigned from lengths, on the GPU against plain
Python; a decoder that does all of it, step by step."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from page_reference import STORES, assign, choose, head_forward8, page_scores
from scored_reference import assert_within
from test_paged_gpu import TYPES, _i32

pytestmark = pytest.mark.gpu


def _bounds(n, Hkv, d, g, ties=False):
    lo = torch.randint(-127, 1, (n, Hkv, d), generator=g, device="cuda")
    hi = torch.randint(0, 128, (n, Hkv, d), generator=g, device="cuda")
    if ties:                                            # few different pages
        which = torch.randint(0, 3, (n,), generator=g, device="cuda")
        lo, hi = lo[:3][which], hi[:3][which]
    unit = torch.exp2(torch.randint(-7, -5, (n, Hkv), generator=g, device="cuda").float())
    unit = torch.ones_like(unit) if ties else unit
    return torch.stack((lo, hi), 2).to(torch.int8).contiguous(), unit


def _table(lens, page, g):
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, w in enumerate(need):
        table[b, :w] = order[at:at + w]
        at += w
    return table, total


def _want(q, bounds, unit, table, lens, K, page, first, last, q_lens=None):
    B, H, T, d = q.shape
    Hkv = bounds.shape[1]
    out = torch.full((B, Hkv, K), -1, dtype=torch.int32)
    bounds, unit = bounds.double().cpu(), unit.double().cpu()
    for b, n in enumerate(lens):
        new = T if q_lens is None else min(max(q_lens[b], 0), T)
        total = -(-n // page)
        if new == 0 or total == 0:
            continue
        at = table[b, :total].long().cpu()
        for g in range(Hkv):
            rows = q[b, g * (H // Hkv):(g + 1) * (H // Hkv), :new].reshape(-1, d)
            best = page_scores(rows, bounds[at, g, 0], bounds[at, g, 1], unit[at, g]) if total > K else [0.0] * total
            chosen = choose(best, total, K, first, last)
            out[b, g, : len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,Hkv,T,page,K,first,last", [
    ([1], 1, 1, 1, 16, 1, 1, 1), ([0, 5], 4, 2, 1, 16, 3, 0, 0), ([1000, 17, 160, 161], 4, 1, 1, 16, 10, 1, 1),
    ([900, 333], 8, 2, 3, 16, 7, 0, 0), ([5000], 8, 8, 1, 16, 100, 2, 3), ([2000, 700], 40, 2, 1, 16, 9, 1, 0),
    ([3000], 6, 1, 7, 32, 33, 0, 2), ([70000, 12], 2, 1, 1, 16, 200, 1, 1), ([600], 2, 2, 1, 16, 4, 3, 3),
    ([640], 2, 2, 1, 16, 39, 0, 0), ([4096], 64, 2, 2, 256, 5, 1, 1), ([160000, 5], 4, 1, 5, 16, 300, 1, 1), ([20000] * 3, 2, 2, 1, 16, 900, 0, 7),
    ([786000], 1, 1, 1, 16, 1000, 500, 400), ([1600], 2, 1, 1, 16, 40, 60, 60)])
def test_the_highest_scores_are_chosen(dtype, d, lens, H, Hkv, T, page, K, first, last):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + K)
    table, n = _table(lens, page, g)
    for ties in (False, True):
        bounds, unit = _bounds(n, Hkv, d, g, ties)
        q = torch.randn((len(lens), H, T, d), generator=g, device="cuda").to(TYPES[dtype])
        got = fa.select_pages(q, bounds, unit, table, _i32(lens), K, page, first=first, last=last)
        assert fa.check_device_status() == 0
        assert torch.equal(got, _want(q, bounds, unit, table, lens, K, page, first, last))


def test_ragged_new_tokens_and_ranges_of_queries():
    g = torch.Generator(device="cuda").manual_seed(5)
    lens, new = [400, 900, 33, 700, 64], [3, 0, 5, 1, 9]
    table, n = _table(lens, 16, g)
    bounds, unit = _bounds(n, 2, 64, g)
    for size in (1.0, 2.0 ** -120, 2.0 ** 100, 0.0):
        q = (torch.randn((5, 6, 5, 64), generator=g, device="cuda") * size).to(torch.bfloat16)
        got = fa.select_pages(q, bounds, unit, table, _i32(lens), 6, 16, q_lens=_i32(new))
        assert torch.equal(got, _want(q, bounds, unit, table, lens, 6, 16, 1, 1, new))
    assert bool((got[1] == -1).all())


def test_nan_bounds_come_first_and_nan_queries_have_no_say():
    g = torch.Generator(device="cuda").manual_seed(6)
    table, n = _table([1600], 16, g)
    bounds, unit = _bounds(n, 1, 64, g)
    q = torch.randn((1, 4, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
    want = fa.select_pages(q[:, 1:].contiguous(), bounds, unit, table, _i32([1600]), 9, 16)
    q[0, 0, 0, 3] = float("nan")
    assert torch.equal(fa.select_pages(q, bounds, unit, table, _i32([1600]), 9, 16), want)
    unit[table[0, 57].item()] = float("nan")
    got = fa.select_pages(q, bounds, unit, table, _i32([1600]), 9, 16)[0, 0].tolist()
    assert 57 in got and 0 in got and 99 in got and len(set(got) - set(want[0, 0].tolist())) <= 1


def test_nan_queries_have_no_say_next_to_other_blocks_of_rows():
    """24 rows of a key head are scored 16 and 8 at a time: all of the first, or of the second ones, are NaN."""
    g = torch.Generator(device="cuda").manual_seed(16)
    for length in (1600, 12000):                          # scored by the block that chooses, and before it
        table, n = _table([length], 16, g)
        bounds, unit = _bounds(n, 1, 64, g)
        q = torch.randn((1, 24, 1, 64), generator=g, device="cuda").to(torch.bfloat16)
        for nan, rest in ((slice(0, 16), slice(16, 24)), (slice(16, 24), slice(0, 16))):
            x = q.clone()
            x[0, nan, 0, 5] = float("nan")
            want = fa.select_pages(q[:, rest].contiguous(), bounds, unit, table, _i32([length]), 9, 16)
            assert torch.equal(fa.select_pages(x, bounds, unit, table, _i32([length]), 9, 16), want)
        q[..., 7] = float("inf")                          # none has a say: the lower numbers
        got = fa.select_pages(q, bounds, unit, table, _i32([length]), 9, 16)[0, 0].tolist()
        assert got == [*range(8), -(-length // 16) - 1]


def test_given_lists_without_new_tokens_are_emptied():
    g = torch.Generator(device="cuda").manual_seed(17)
    table, n = _table([1600, 20], 16, g)
    bounds, unit = _bounds(n, 2, 64, g)
    pages = torch.full((2, 2, 5), 7, dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 4, 0, 64), dtype=torch.float16, device="cuda")
    assert fa.select_pages(q, bounds, unit, table, _i32([1600, 20]), 5, 16, pages=pages) is pages
    assert bool((pages == -1).all())


def test_bounds_hold_for_every_key():
    """A page's score is no less than the product of the rounded query with any of its keys, so the page of the
    highest product of one query is always chosen when its score is alone above the others'."""
    g = torch.Generator(device="cuda").manual_seed(7)
    page, d = 16, 64
    kc, vc = (torch.zeros((40, 1, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb, bs = torch.zeros((40, 1, 2, d), dtype=torch.int8, device="cuda"), torch.zeros((40, 1), device="cuda")
    table = torch.randperm(40, generator=g, device="cuda").to(torch.int32)[None]
    k = torch.randn((1, 1, 600, d), generator=g, device="cuda").to(torch.bfloat16)
    for begin, end in ((0, 311), (311, 312), (312, 600)):
        fa.append_paged(k[:, :, begin:end], k[:, :, begin:end], kc, vc, table, _i32([end]), k_bounds=kb, bound_scales=bs)
    lo, hi = (kb[table[0].long(), 0, i].double() * bs[table[0].long()].double() for i in (0, 1))
    for p in range(38):
        keys = k[0, 0, p * page: (p + 1) * page].double()
        assert bool(((keys >= lo[p]) & (keys <= hi[p])).all())
    assert fa.check_device_status() == 0


def test_choice_in_a_graph_on_streams_and_with_given_memory():
    g = torch.Generator(device="cuda").manual_seed(8)
    lens = [4000, 100]
    table, n = _table([4000, 4000], 16, g)
    bounds, unit = _bounds(n, 2, 128, g)
    q = torch.randn((2, 8, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    nl = _i32(lens)
    table = torch.cat((table, torch.full((2, 300), -1, dtype=torch.int32, device="cuda")), 1)     # room to grow
    ws = torch.full((fa.select_pages_workspace_size(2, 2, 550, 20),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    out = torch.empty((2, 2, 20), dtype=torch.int32, device="cuda")
    fa.select_pages(q, bounds, unit, table, nl, 20, 16)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        assert fa.select_pages(q, bounds, unit, table, nl, 20, 16, pages=out, workspace=ws) is out
    for new in ([4000, 100], [1, 4000], [0, 321]):
        nl.copy_(_i32(new))
        gr.replay()
        assert torch.equal(out, _want(q, bounds, unit, table, new, 20, 16, 1, 1))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [fa.select_pages(q, bounds, unit, table, nl, 20, 16, stream=s) for s in (side, None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, out) for x in got)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,T,long", [
    (20, 8, 2, 1, 9600), (20, 8, 2, 4, 8300), (13, 3, 3, 17, 12000),     # scored on all SMs first: 8, 16 and more rows
    (160, 4, 4, 1, 8400), (80, 16, 8, 6, 8200),                            # many slices: a block scores and chooses
    (38, 2, 1, 1, 9000), (39, 2, 1, 1, 9000), (19, 12, 2, 2, 33000)])       # the most that are chosen from where they are scored
def test_slices_of_many_numbers(d, B, H, Hkv, T, long):
    g = torch.Generator(device="cuda").manual_seed(B + H + T)
    lens = [long if b % 37 == 1 else 16 * (b % 40) + b % 7 for b in range(B)]
    table, n = _table(lens, 16, g)
    bounds, unit = _bounds(n, Hkv, d, g, ties=B % 2 == 1)
    q = torch.randn((B, H, T, d), generator=g, device="cuda").to(torch.float16)
    got = fa.select_pages(q, bounds, unit, table, _i32(lens), 11, 16)
    assert torch.equal(got, _want(q, bounds, unit, table, lens, 11, 16, 1, 1))


def test_captured_choices_share_a_workspace():
    """Two captured calls and calls between them count in the same words."""
    g = torch.Generator(device="cuda").manual_seed(18)
    table, n = _table([12000, 9000], 16, g)
    bounds, unit = _bounds(n, 2, 64, g)
    q = [torch.randn((2, 8, T, 64), generator=g, device="cuda").to(torch.bfloat16) for T in (1, 5)]
    nl = _i32([12000, 9000])
    ws = torch.randint(0, 256, (fa.select_pages_workspace_size(2, 2, 750, 20),), generator=g, device="cuda", dtype=torch.uint8)
    out = [torch.empty((2, 2, 20), dtype=torch.int32, device="cuda") for _ in q]
    graphs = []
    for x, y in zip(q, out):
        fa.select_pages(x, bounds, unit, table, nl, 20, 16, pages=y, workspace=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fa.select_pages(x, bounds, unit, table, nl, 20, 16, pages=y, workspace=ws)
    for lens in ([12000, 9000], [8200, 12], [11999, 8999], [12000, 9000]):
        nl.copy_(_i32(lens))
        want = [_want(x, bounds, unit, table, lens, 20, 16, 1, 1) for x in q]
        for order in ((0, 1), (1, 0), (1, 1)):
            for y in out:
                y.fill_(-5)
            for i in order:
                graphs[i].replay()
            for i in set(order):
                assert torch.equal(out[i], want[i])
            assert torch.equal(fa.select_pages(q[0], bounds, unit, table, nl, 20, 16, workspace=ws), want[0])


def test_choice_refusals():
    g = torch.Generator(device="cuda").manual_seed(8)
    table, n = _table([400], 16, g)
    bounds, unit = _bounds(n, 2, 64, g)
    q, nl = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda"), _i32([400])
    call = lambda q=q, b=bounds, u=unit, t=table, n=nl, K=4, page=16, **kw: fa.select_pages(q, b, u, t, n, K, page, **kw)  # noqa: E731
    assert call().shape == (1, 2, 4)
    for match, kw in (("contiguous bf16", dict(q=q.float())), ("dividing", dict(q=q[:, :3].contiguous())), ("k_bounds", dict(b=bounds.float())),
                      ("k_bounds", dict(b=bounds[:, :, :1].contiguous())), ("bound_scales", dict(u=unit.half())), ("kv_lens", dict(n=nl.long())),
                      ("block_table", dict(t=table.long())), ("n_select", dict(K=0)), ("CUDA", dict(u=unit.cpu())),
                      ("pages", dict(pages=torch.zeros((1, 2, 5), dtype=torch.int32, device="cuda")))):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    for match, kw in (("INVALID_ARG", dict(first=-1)), ("UNSUPPORTED", dict(page=24)), ("INVALID_ARG", dict(page=0))):
        with pytest.raises(fa.FaError, match=match):
            call(**kw)
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        call(t=torch.zeros((1, 49153), dtype=torch.int32, device="cuda"))


# ---- pages from lengths --------------------------------------------------------------------------

def _state(old, page, width, free, g, extra=5):
    held = [-(-n // page) for n in old]
    n = sum(held) + free + extra
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    table = [[-7] * width for _ in old]
    at = 0
    for b, h in enumerate(held):
        table[b][:h] = order[at:at + h]
        at += h
    first = int(torch.randint(0, n, (1,), generator=g, device="cuda"))
    ring = [-9] * n
    for i in range(free):
        ring[(first + i) % n] = order[at + i]
    return table, ring, [first, free]


@pytest.mark.parametrize("old,new,page,T", [
    ([0], [1], 16, 1), ([0], [0], 16, 0), ([16], [17], 16, 3), ([15, 16, 0, 31], [16, 17, 1, 40], 16, 4), ([100, 50, 0], [0, 50, 300], 32, 300),
    ([100, 50, 7], [3, 0, 0], 16, 2), ([4096, 0], [4097, 4096], 4096, 5000), (list(range(1500)), [n + 1 for n in range(1500)], 16, 1),
    ([(7 * i) % 90 for i in range(1300)], [(11 * i) % 90 for i in range(1300)], 16, 20), ([5] * 33, [5 + i * 300 for i in range(33)], 48, 9600)])
def test_pages_are_assigned(old, new, page, T):
    g = torch.Generator(device="cuda").manual_seed(sum(new) + T)
    width = max(-(-n // page) for n in old + new) + 2
    grow = sum(max(0, -(-y // page) + -x // page) for x, y in zip(old, new))
    for extra, over in ((0, False), (9, False), (9, True)):
        table, ring, state = _state(old, page, width, grow + extra, g)
        t, r, s, n = _i32(table), _i32(ring), _i32(state), _i32(old)
        outs = dict(lens=n, state=s) if over else {}       # written over the inputs
        lens, q_lens, slots, positions, state2 = fa.assign_pages(t, n, _i32(new), r, s, page, T, **outs)
        assert fa.check_device_status() == 0
        want_slots, want_pos, want_state = assign(table, old, new, ring, state, page, T)
        assert t.tolist() == table and r.tolist() == ring and state2.tolist() == want_state and (over or s.tolist() == state)
        assert lens.tolist() == new and q_lens.tolist() == [max(0, y - x) for x, y in zip(old, new)]
        assert slots.dtype == torch.int64 and slots.tolist() == want_slots and positions.tolist() == want_pos


def test_all_or_nothing():
    g = torch.Generator(device="cuda").manual_seed(3)
    old, new = [16, 40, 30], [48, 0, 33]
    for free, new, state in ((2, new, None), (9, [48, 0, -1], None), (9, [48, 0, 16 * 8 + 1], None), (9, new, [-1, 9]), (9, new, [99, 9]),
                             (9, new, [0, 99]), (9, new, [0, -1])):
        table, ring, st = _state(old, 16, 8, free, g)
        t, r, s = _i32(table), _i32(ring), _i32(state or st)
        lens, q_lens, slots, positions, state2 = fa.assign_pages(t, _i32(old), _i32(new), r, s, 16, 3)
        assert fa.check_device_status() == fa.FA_ERR_INVALID_ARG
        assert t.tolist() == table and r.tolist() == ring and torch.equal(s, state2)
        assert lens.tolist() == old and not bool(q_lens.any())
        assert bool((slots == -1).all()) and bool((positions == -1).all())


def test_growing_in_place_in_a_graph():
    """One captured step that grows every sequence, its outputs written over its inputs; more tokens than
    one block places."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, page, T = 6, 16, 2000
    table, ring, state = _state([0] * B, page, 800, 2400, g)
    t, r, s = _i32(table), _i32(ring), _i32(state)
    lens, want = _i32([0] * B), _i32([0] * B)
    q_lens, slots, positions = _i32([0] * B), torch.zeros((B, T), dtype=torch.int64, device="cuda"), torch.zeros((B, T), dtype=torch.int32, device="cuda")
    out = dict(lens=lens, q_lens=q_lens, slots=slots, positions=positions, state=s)
    fa.assign_pages(t, lens, want, r, s, page, T, **out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fa.assign_pages(t, lens, want, r, s, page, T, **out)
    now = [0] * B
    for new in ([2000, 1, 300, 0, 17, 999], [2001, 2, 0, 16, 17, 1800], [0] * B, [3000] * B, [0, 5, 6, 7, 8, 9]):
        want.copy_(_i32(new))
        gr.replay()
        want_slots, want_pos, state = assign(table, now, new, ring, state, page, T)
        now = new
        assert fa.check_device_status() == 0
        assert lens.tolist() == new and s.tolist() == state and t.tolist() == table and r.tolist() == ring
        assert slots.tolist() == want_slots and positions.tolist() == want_pos


def test_assignment_refusals():
    t, n, r, s = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), _i32([0, 0]), _i32([0, 1, 2]), _i32([0, 3])
    for match, args in (("block_table", (t.long(), n, n, r, s)), ("new_lens", (t, n, n[:1], r, s)), ("free_state", (t, n, n, r, r)),
                        ("free_pages", (t, n, n, r.long(), s)), ("CUDA", (t, n, n, r.cpu(), s)), ("rows", (t[:1].expand(2, 3), n, n, r, s))):
        with pytest.raises(ValueError, match=match):
            fa.assign_pages(*args, 16, 1)
    with pytest.raises(ValueError, match="max_new"):
        fa.assign_pages(t, n, n, r, s, 16, -1)
    with pytest.raises(ValueError, match="overlap"):
        fa.assign_pages(t, n, _i32([1, 1]), r, s, 16, 1, q_lens=n)
    with pytest.raises(ValueError, match="overlap"):
        fa.assign_pages(t, n, _i32([1, 1]), r, s, 16, 1, state=r[:2])
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.assign_pages(t, n, n, r, s, 24, 1)
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.assign_pages(t, n, n, r[:0], s, 16, 1)


# ---- together ------------------------------------------------------------------------------------

@pytest.mark.parametrize("store,d,rot", [("int8", 64, 32), ("e4m3", 128, 128)])
def test_a_decoder_over_small_caches(store, d, rot):
    """Prompts, tokens and drafts, a sequence that ends and another that takes its place: pages assigned, tokens
    written, pages chosen, attention over them; each step's result is attention over the chosen pages' values,
    and these are the keys and values to the store's precision."""
    H, Hkv, page, B, K = 4, 2, 16, 3, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    n_pages = 40
    kc, vc = (torch.zeros((n_pages, Hkv, page, d), dtype=STORES[store], device="cuda") for _ in range(2))
    ks, vs, bs = (torch.zeros((n_pages, Hkv), device="cuda") for _ in range(3))
    kb = torch.zeros((n_pages, Hkv, 2, d), dtype=torch.int8, device="cuda")
    table = torch.zeros((B, 14), dtype=torch.int32, device="cuda")
    ring, state, lens = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32), _i32([7, n_pages]), _i32([0] * B)
    inv_freq, _ = fa.rotary_frequencies(rot)
    all_k, all_v = ([torch.zeros((Hkv, 0, d), device="cuda") for _ in range(B)] for _ in range(2))
    now = [0] * B
    for T, new in ((150, [150, 31, 0]), (1, [151, 32, 0]), (4, [155, 34, 0]), (1, [156, 0, 0]), (60, [157, 0, 60]), (1, [158, 1, 61]), (1, [159, 2, 62])):
        lens, q_lens, slots, positions, state = fa.assign_pages(table, lens, _i32(new), ring, state, page, T)
        q, k, v = (torch.randn((B, h, T, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv))
        q2 = fa.append_paged(k, v, kc, vc, table, lens, q=q, q_lens=q_lens, inv_freq=inv_freq, k_scales=ks, v_scales=vs, k_bounds=kb,
                             bound_scales=bs)
        pages = fa.select_pages(q2, kb, bs, table, lens, K, page, q_lens=q_lens)
        o, lse = fa.forward_paged(q2, kc, vc, table, lens, q_lens=q_lens, k_scales=ks, v_scales=vs, pages=pages)
        assert fa.check_device_status() == 0
        assert torch.equal(pages, _want(q2, kb, bs, table, new, K, page, 1, 1, q_lens.tolist()))
        turned = fa.rotary(k.float(), positions.clamp(min=0), inv_freq)
        for b, n in enumerate(new):
            count = max(0, n - now[b])
            if n < now[b]:
                all_k[b], all_v[b] = all_k[b][:, :n], all_v[b][:, :n]
            all_k[b], all_v[b] = torch.cat((all_k[b], turned[b, :, :count]), 1), torch.cat((all_v[b], v[b, :, :count].float()), 1)
            # the slots say where the tokens are
            at = slots[b, :count]
            for cache, scales, x in ((kc, ks, turned), (vc, vs, v.float())):
                got = cache.float()[at // page, :, at % page] * scales[at // page][..., None]
                step = scales[at // page][..., None]
                # half a step of a code: 2^-4 of an e4m3 value, or 2^-10 below its normal range
                tol = 0.5 * step if store == "int8" else 2.0 ** -4 * x[b, :, :count].transpose(0, 1).abs() + 2.0 ** -10 * step
                assert bool(((got - x[b, :, :count].transpose(0, 1)).abs() <= tol * 1.0001 + 1e-6).all())
            for h in range(H):
                if count == 0:
                    continue
                which = pages[b, h // 2][pages[b, h // 2] >= 0].long()
                kpos = (which[:, None] * page + torch.arange(page, device="cuda")).flatten()
                there = kpos < n
                place = table[b].long()[which]
                c, e = (x[place, h // 2].reshape(-1, d)[there].double() for x in (kc, vc))
                k1, v1 = (x[place, h // 2].double().repeat_interleave(page)[there][:, None] for x in (ks, vs))
                kpos = kpos[there]
                qpos = n - count + torch.arange(count, device="cuda")
                ref = head_forward8(q2[b, h, :count].double(), c, e, k1, v1, kpos[None, :] <= qpos[:, None],
                                    (qpos[:, None] - kpos).double(), d ** -0.5, 0.0, 0.0, torch.bfloat16)
                assert_within("O", o[b, h, :count], ref[0], ref[2])
                assert_within("LSE", lse[b, h, :count], ref[1], ref[3])
                # values of the cache are those of the keys: at most two roundings of a code apart
                for scale, code, mine in ((k1, c, all_k[b][h // 2]), (v1, e, all_v[b][h // 2])):
                    x = mine[kpos].double()
                    tol = scale if store == "int8" else 2.0 ** -3 * x.abs() + 2.0 ** -9 * scale
                    assert bool(((code * scale - x).abs() <= tol * 1.0001 + 1e-6).all())
        now = new
