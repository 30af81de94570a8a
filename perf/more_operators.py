"""Cases and plain forms of the operators that serve long contexts from small caches: what each one
computes, in elementary torch operations, and the calls that a program makes of the library's kernels.

Four operators, one after another in a decoding step: pages assigned to sequences as they grow, with
the places of their new tokens; the write of those tokens into 8-bit pages with a scale for each page
and head, bounds of each page's keys kept on the way; the choice of the pages whose bounds promise the
highest scores; and attention over 8-bit pages, all of them or the chosen ones.

``own`` selects the library's kernels; otherwise ``run`` computes the plain form.
"""
import math
import random
import zlib

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_LARGEST = {"int8": 127.0, "e4m3": 448.0}


# ---- the cases -----------------------------------------------------------------------------------

def _attend(name, B, H, Hkv, T, d, page, dtype, store, lo, hi, picks=0, softcap=0.0, alibi=False):
    c = dict(kind="attend", B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, store=store, lo=lo, hi=hi,
             picks=picks, softcap=softcap, alibi=alibi)
    return dict(c, name=name) if name else c


def _append(name, B, H, Hkv, T, d, page, dtype, store, hi, rot, interleaved, ragged, bounds):
    c = dict(kind="append", B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, store=store, hi=hi, rot=rot,
             interleaved=interleaved, ragged=ragged, bounds=bounds)
    return dict(c, name=name) if name else c


def _select(name, B, H, Hkv, T, d, page, dtype, lo, hi, picks, first, last):
    c = dict(kind="select", B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, lo=lo, hi=hi, picks=picks,
             first=first, last=last)
    return dict(c, name=name) if name else c


def _assign(name, B, T, page, hi, release):
    c = dict(kind="assign", B=B, T=T, page=page, hi=hi, release=release)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for one user, short cache: latency
        _attend("attend-b1-short", 1, 32, 8, 1, 128, 16, "bf16", "e4m3", 200, 200),
        # a serving batch of unequal lengths, capped scores
        _attend("attend-b64-ragged", 64, 32, 8, 1, 128, 64, "bf16", "int8", 1, 8192, softcap=50.0),
        # few users, very long contexts, the whole cache read
        _attend("attend-b2-128k", 2, 32, 8, 1, 128, 64, "bf16", "e4m3", 100000, 131072),
        # drafted tokens checked in one call, biased scores, one key head per query head
        _attend("attend-draft5-d64", 16, 16, 16, 5, 64, 48, "fp16", "int8", 5, 4000, alibi=True),
        # long contexts of which each key head reads the 64 pages chosen for it
        _attend("attend-picked-64k", 8, 32, 8, 1, 128, 64, "bf16", "int8", 40000, 65536, picks=64),
        # chosen pages of a 16-bit cache, two drafted tokens, short sequences among them
        _attend("attend-picked-16bit", 3, 24, 4, 2, 64, 32, "fp16", "16", 1, 20000, picks=33),
        # the cache write of a decoding batch, keys and queries rotated in the same call
        _append("append-b64-token", 64, 32, 8, 1, 128, 64, "bf16", "e4m3", 2048, 128, False, False, False),
        # the cache write of a ragged batch of prompts, key bounds kept (positions by distance bias)
        _append("append-prompts", 4, 32, 8, 4096, 128, 64, "bf16", "int8", 8192, 0, False, True, True),
        # the choice of pages for a decoding batch of unequal lengths
        _select("select-b64-ragged", 64, 32, 8, 1, 128, 64, "bf16", 1, 8192, 32, 1, 2),
        # the choice of a few among thousands of small pages, three drafted tokens
        _select("select-b2-128k", 2, 32, 8, 3, 128, 16, "bf16", 100000, 131072, 256, 1, 4),
        # a decoding batch grows by one token each
        _assign("assign-b256-token", 256, 1, 64, 8192, False),
        # prompts of many lengths come, other sequences end
        _assign("assign-prompts", 40, 4096, 16, 16384, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "picked", "append", "append", "select", "assign"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 8])
    H = Hkv * rng.choice([1, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind in ("attend", "picked"):
        hi = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(128, 131072 // hi)))
        picks = _log(rng, 1, 100) if kind == "picked" else 0
        store = rng.choice(["int8", "e4m3", "16"] if picks else ["int8", "e4m3"])
        return _attend(None, B, H, Hkv, rng.choice([1, 1, 1, 2, 7]), d, page, dtype, store, rng.randint(0, hi), hi,
                       picks, softcap=rng.choice([0.0, 0.0, 30.0]), alibi=rng.random() < 0.3)
    if kind == "append":
        T = _log(rng, 1, 2048) if rng.random() < 0.5 else 1
        bounds = rng.random() < 0.5
        # what is rotated is a rounded number before it is rounded to 8 bits: whole numbers of two
        # computations may then differ, so integers come of keys as they are
        store = rng.choice(["int8", "e4m3", "16"] if bounds else ["int8", "e4m3"])
        rot = 0 if bounds or store == "int8" else rng.choice([0, 16, 32, d])
        return _append(None, _log(rng, 1, max(1, min(128, 8192 // T))), H, Hkv, T, d, page, dtype, store,
                       T + _log(rng, 1, 2048), rot, rng.random() < 0.5, rng.random() < 0.5, bounds)
    if kind == "select":
        hi = _log(rng, 40 * page, 65536)                 # the longest sequence has pages to choose from
        B = _log(rng, 1, max(1, min(64, 131072 // hi)))
        first, last = rng.choice([0, 1, 2]), rng.choice([0, 1, 3])
        return _select(None, B, H, Hkv, rng.choice([1, 1, 2, 5]), d, page, dtype, rng.randint(0, hi), hi,
                       first + last + _log(rng, 4, min(200, hi // page - 10)), first, last)
    T = _log(rng, 1, 4096) if rng.random() < 0.5 else 1
    return _assign(None, _log(rng, 1, max(1, min(600, 160000 // T))), T, page, T + _log(rng, 1, 12000), rng.random() < 0.5)


# ---- the inputs ----------------------------------------------------------------------------------

def _lengths(case, n, lo, hi, salt):
    """n lengths in [lo, hi] that belong to the case itself, so that its work is known."""
    keys = ("kind", "B", "T", "hi", "page", "picks")
    r = random.Random(zlib.crc32(repr([salt] + [case.get(k) for k in keys]).encode()))
    return [r.randint(lo, hi) for _ in range(n)]


def _cache_lens(case):
    """Tokens of each sequence, the new ones included."""
    lens = _lengths(case, case["B"], case["lo"], case["hi"], 1)
    lens[-1] = case["hi"]
    return lens


def _append_lens(case):
    """(tokens in the cache, the new ones included; new tokens) of each sequence."""
    new = _lengths(case, case["B"] - 1, 0, case["T"], 2) + [case["T"]] if case["ragged"] else [case["T"]] * case["B"]
    old = _lengths(case, case["B"], 0, case["hi"] - case["T"], 3)
    return [a + b for a, b in zip(old, new)], new


def _assign_lens(case):
    """(tokens before, tokens after) of each sequence; some end, and some of them are prompts."""
    r = random.Random(zlib.crc32(repr([4] + [case[k] for k in ("B", "T", "hi", "page")]).encode()))
    old, new = [], []
    for b in range(case["B"]):
        a = r.randint(0, case["hi"] - case["T"])
        if case["release"] and b % 3 == 1:
            n = r.choice([0, 0, a // 2])                 # ended, or drafts taken back
        elif case["T"] > 1:
            n = a + r.randint(0, case["T"])
        else:
            n = a + 1
        old.append(a)
        new.append(n)
    return old, new


def _pages(n, page):
    return -(-n // page)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(_TYPES[dtype])


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, lens, page):
    """A table of pages in shuffled order, and the pages in all; unused entries name page 0."""
    need = [_pages(n, page) for n in lens]
    width, used = max(1, max(need)), sum(need)
    order = torch.randperm(used + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[at] = order[:used]
    return table, used + 1


def _stored(x, store):
    """Values [pages, heads, page, d] in 8 bits, each page and head by its largest, and the scales; the
    largest value of a page differs from page to page."""
    scale = x.abs().amax((-1, -2)) / _LARGEST[store]
    y = x / scale[..., None, None]
    return (torch.round(y) if store == "int8" else y.clamp(-448.0, 448.0)).to(_TYPES[store]), scale


def _cache(g, case, pages, spread=True):
    """A cache's keys or values and their scales (16-bit ones have none)."""
    x = torch.randn((pages, case["Hkv"], case["page"], case["d"]), generator=g, device="cuda")
    if case["store"] == "16":
        return x.to(_TYPES[case["dtype"]]), None
    if spread:
        x *= torch.exp(0.5 * torch.randn((pages, case["Hkv"], 1, 1), generator=g, device="cuda")).clamp(max=4.0)
    return _stored(x, case["store"])


def _choice(g, case, lens):
    """Pages chosen for each sequence and key head, ascending, the last page among them; -1 behind."""
    B, Hkv, K = case["B"], case["Hkv"], case["picks"]
    n = torch.tensor([_pages(x, case["page"]) for x in lens], device="cuda")[:, None, None]
    W = max(1, int(n.max()))
    at = torch.arange(W, device="cuda")
    key = torch.rand((B, Hkv, W), generator=g, device="cuda")
    key = torch.where(at == n - 1, 2.0, torch.where(at < n, key, -1.0))
    value, place = torch.topk(key, min(K, W))
    place = torch.where(value >= 0.0, place, W).sort(-1).values
    out = torch.full((B, Hkv, K), -1, dtype=torch.int32, device="cuda")
    out[..., : place.shape[-1]] = torch.where(place < W, place, -1).to(torch.int32)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    B, page = case["B"], case["page"]
    if case["kind"] == "assign":
        old, new = _assign_lens(case)
        held, want = ([_pages(n, page) for n in x] for x in (old, new))
        grown = sum(max(0, w - h) for h, w in zip(held, want))
        used, spare = sum(held), grown + 37
        s["block_table"] = torch.zeros((B, _pages(case["hi"], page)), dtype=torch.int32, device="cuda")
        order = torch.randperm(used + spare, generator=g, device="cuda").to(torch.int32)
        at = torch.arange(s["block_table"].shape[1], device="cuda")[None, :] < torch.tensor(held, device="cuda")[:, None]
        s["block_table"][at] = order[:used]
        # the free pages lie in a ring, from some place on
        begin = int(torch.randint(0, used + spare, (1,), generator=g, device="cuda"))
        s["free_pages"] = torch.full((used + spare,), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][(begin + torch.arange(spare, device="cuda")) % (used + spare)] = order[used:]
        s["free_state"] = _int32([begin, spare])
        s["old"], s["new"] = _int32(old), _int32(new)
        return s
    H, Hkv, T, d, dtype = (case[k] for k in ("H", "Hkv", "T", "d", "dtype"))
    if case["kind"] == "append":
        lens, new = _append_lens(case)
        s["block_table"], n_pages = _table(g, lens, page)
        s["k_cache"], s["k_scales"] = _cache(g, case, n_pages)
        s["v_cache"], s["v_scales"] = _cache(g, case, n_pages)
        if case["store"] != "16":                       # as earlier writes left them: powers of two
            for n in ("k_scales", "v_scales"):
                s[n] = _two(torch.ceil(torch.log2(s[n])))
        s["k_bounds"] = s["bound_scales"] = None
        if case["bounds"]:
            lo = torch.randint(-127, 1, (n_pages, Hkv, 1, d), generator=g, device="cuda", dtype=torch.int8)
            hi = torch.randint(0, 128, (n_pages, Hkv, 1, d), generator=g, device="cuda", dtype=torch.int8)
            s["k_bounds"] = torch.cat((lo, hi), 2).contiguous()
            s["bound_scales"] = _two(torch.randint(-7, -3, (n_pages, Hkv), generator=g, device="cuda"))
        s["kv_lens"], s["q_lens"] = _int32(lens), _int32(new)
        # the projections' outputs: [B, T, heads, d], seen as [B, heads, T, d]
        s["k"], s["v"] = (_normal(g, (B, T, Hkv, d), dtype).transpose(1, 2) for _ in range(2))
        s["q"] = _normal(g, (B, T, H, d), dtype).transpose(1, 2) if case["rot"] else None
        i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = torch.pow(10000.0, -i / case["rot"]) if case["rot"] else None
        return s
    lens = _cache_lens(case)
    s["kv_lens"] = _int32(lens)
    s["q"] = _normal(g, (B, H, T, d), dtype, 2.0)
    s["block_table"], n_pages = _table(g, lens, page)
    if case["kind"] == "select":
        # bounds of keys with a page-wide part and a part of their own
        mid = torch.randn((n_pages, Hkv, d), generator=g, device="cuda")
        half = 1.5 * torch.rand((n_pages, Hkv, d), generator=g, device="cuda") + 0.2
        s["bound_scales"] = _two(torch.ceil(torch.log2((mid.abs() + half).amax(-1) / 127.0)))
        unit = s["bound_scales"][..., None]
        s["k_bounds"] = torch.stack((torch.floor((mid - half) / unit), torch.ceil((mid + half) / unit)), 2).to(torch.int8)
        return s
    s["k_cache"], s["k_scales"] = _cache(g, case, n_pages)
    s["v_cache"], s["v_scales"] = _cache(g, case, n_pages)
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if case["alibi"] else None
    s["pages"] = _choice(g, case, lens) if case["picks"] else None
    return s


# ---- one pass ------------------------------------------------------------------------------------
#
# A cache's 8-bit codes and its scales come back as they are held: their products are the values.

def run(s):
    if own:
        return _run_own(s)
    return {"attend": _plain_attend, "append": _plain_append, "select": _plain_select,
            "assign": _plain_assign}[s["kind"]](s)


def _run_own(s):
    import exact_io_aware_23_gb300 as fa
    if s["kind"] == "attend":
        o, lse = fa.forward_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                  softcap=s["softcap"], alibi_slopes=s["slopes"], k_scales=s["k_scales"],
                                  v_scales=s["v_scales"], pages=s["pages"])
        return dict(o=o, lse=lse)
    if s["kind"] == "append":
        q = fa.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                            q=s["q"], q_lens=s["q_lens"], inv_freq=s["inv_freq"], interleaved=s["interleaved"],
                            k_scales=s["k_scales"], v_scales=s["v_scales"], k_bounds=s["k_bounds"],
                            bound_scales=s["bound_scales"])
        return dict(q=q, **_written(s))
    if s["kind"] == "select":
        return dict(pages=fa.select_pages(s["q"], s["k_bounds"], s["bound_scales"], s["block_table"], s["kv_lens"],
                                          s["picks"], s["page"], first=s["first"], last=s["last"]))
    lens, q_lens, slots, positions, state = fa.assign_pages(s["block_table"], s["old"], s["new"], s["free_pages"],
                                                            s["free_state"], s["page"], s["T"])
    return dict(lens=lens, q_lens=q_lens, slots=slots, positions=positions, state=state, table=s["block_table"],
                free=s["free_pages"])


def _written(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales", "k_bounds", "bound_scales")}


# ---- plain forms: 32-bit arithmetic, rounded once at the end --------------------------------------

def _values(cache, scales):
    return cache.float() if scales is None else cache.float() * scales[..., None, None]


def _plain_attend(s):
    B, H, Hkv, T, d, page = (s[n] for n in ("B", "H", "Hkv", "T", "d", "page"))
    G = H // Hkv
    lens = s["kv_lens"].long()
    table = s["block_table"].long()
    off = torch.arange(page, device="cuda")
    if s["pages"] is None:
        at = torch.arange(table.shape[1] * page, device="cuda").expand(B, 1, -1)         # places of the keys
        take = lambda c, sc: _values(c[table], None if sc is None else sc[table]).permute(0, 2, 1, 3, 4)  # noqa: E731
    else:
        pages = s["pages"].long()
        at = torch.where(pages[..., None] >= 0, pages[..., None] * page + off, table.shape[1] * page).reshape(B, Hkv, -1)
        where = torch.gather(table[:, None, :].expand(B, Hkv, -1), 2, pages.clamp(0, table.shape[1] - 1))
        head = torch.arange(Hkv, device="cuda")[None, :, None]
        take = lambda c, sc: _values(c[where, head], None if sc is None else sc[where, head])  # noqa: E731
    k, v = (take(s[n + "_cache"], s[n + "_scales"]).reshape(B, Hkv, 1, -1, d) for n in "kv")
    there = at < lens[:, None, None]
    v = torch.where(there[:, :, None, :, None], v, 0.0)
    q = s["q"].float().reshape(B, Hkv, G, T, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    del k
    if s["softcap"] > 0.0:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    pos = lens[:, None] - T + torch.arange(T, device="cuda")[None, :]                    # the new tokens' places
    dist = pos[:, None, None, :, None] - at[:, :, None, None, :]
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(Hkv, G, 1, 1) * dist.float()
    x = torch.where((dist >= 0) & there[:, :, None, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0.0, 1.0, l)
    lse = torch.where(l == 0.0, -math.inf, m + torch.log(l))
    return dict(o=o.reshape(B, H, T, d).to(s["q"].dtype), lse=lse.reshape(B, H, T))


def _plain_turn(x, positions, inv_freq, interleaved):
    """x [B, heads, T, d] with pair i of each head turned by position * inv_freq[i]."""
    half = inv_freq.numel()
    angle = (positions.double()[..., None] * inv_freq).unsqueeze(1)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = x.float()
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, rest), -1)


def _power(amax, largest):
    """The smallest power of two, at least 2^-100, that ``largest`` of reaches amax."""
    m, e = torch.frexp(amax)                             # amax = m 2^e, m in [0.5, 1)
    ml, el = math.frexp(largest)
    return _two(torch.where(amax > 0.0, e - el + (m > ml).int(), -100).clamp(min=-100))


def _two(e):
    """2^e in fp32 for e in [-126, 127], by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _round8(y, store):
    return torch.round(y).to(torch.int8) if store == "int8" else y.to(torch.float8_e4m3fn)


def _plain_append(s):
    B, Hkv, T, d, page, store = (s[n] for n in ("B", "Hkv", "T", "d", "page", "store"))
    lens, new = s["kv_lens"].long(), s["q_lens"].long()
    t = torch.arange(T, device="cuda")
    begin = lens - new
    pos = begin[:, None] + t                                                             # [B, T]
    there = t[None, :] < new[:, None]
    q, k = s["q"], s["k"].float()
    if q is not None:
        q = _plain_turn(q, pos, s["inv_freq"], s["interleaved"]).to(q.dtype)
        q = torch.where(there[:, None, :, None], q, torch.zeros((), dtype=q.dtype, device="cuda"))
        k = _plain_turn(k, pos, s["inv_freq"], s["interleaved"])
    # the pages that get tokens: P of each sequence at most, from page `lead` on
    P = (T + page - 2) // page + 1
    lead = begin // page
    b, at = torch.nonzero(there, as_tuple=True)
    off = pos[b, at] - lead[b] * page
    fresh = torch.zeros((B, P * page), dtype=torch.bool, device="cuda")
    fresh[b, off] = True
    fresh = fresh.reshape(B, P, page)
    pb, pp = torch.nonzero(fresh.any(-1), as_tuple=True)
    place = s["block_table"].long()[pb, lead[pb] + pp]                                   # their places in the cache
    kept = (begin[pb] - (lead[pb] + pp) * page).clamp(min=0)                             # tokens that were there
    old = (kept > 0)[:, None]
    slot = torch.arange(page, device="cuda")
    is_new, is_old = (m[:, None, :, None] for m in (fresh[pb, pp], slot < kept[:, None]))

    def spread(x):
        y = torch.zeros((B, P * page, Hkv, d), dtype=x.dtype, device="cuda")
        y[b, off] = x[b, :, at]
        return y.reshape(B, P, page, Hkv, d)[pb, pp].transpose(1, 2)                     # [pages, Hkv, page, d]

    for name, x in (("k", k), ("v", s["v"].float())):
        x = spread(x)
        cache, scales = s[name + "_cache"], s[name + "_scales"]
        raw = cache.view(torch.int16 if store == "16" else torch.uint8)
        if store == "16":
            x = x.to(cache.dtype)
            raw[place] = torch.where(is_new, x.view(torch.int16), raw[place])
            x = x.float()
        else:
            was = scales[place]
            scale = torch.maximum(torch.where(old, was, 0.0), _power(x.abs().amax((-1, -2)), _LARGEST[store]))
            scales[place] = scale
            again = cache.view(torch.uint8)[place].view(cache.dtype).float() * (was / scale)[..., None, None]
            again = _round8(torch.where(is_old, again, 0.0), store).view(torch.uint8)
            first = _round8(x * (1.0 / scale)[..., None, None], store).view(torch.uint8)
            raw[place] = torch.where(is_new, first, torch.where(is_old, again, raw[place]))
        if name == "k" and s["bounds"]:
            was = s["bound_scales"][place]
            unit = torch.maximum(torch.where(old, was, 0.0), _power(x.abs().amax((-1, -2)), 127.0))
            lo = torch.floor(torch.where(is_new, x, math.inf).amin(2) / unit[..., None])
            hi = torch.ceil(torch.where(is_new, x, -math.inf).amax(2) / unit[..., None])
            ratio = (was / unit)[..., None]
            bounds = s["k_bounds"][place].float()
            lo = torch.where(old[..., None], torch.minimum(lo, torch.floor(bounds[:, :, 0] * ratio)), lo)
            hi = torch.where(old[..., None], torch.maximum(hi, torch.ceil(bounds[:, :, 1] * ratio)), hi)
            s["k_bounds"][place] = torch.stack((lo, hi), 2).to(torch.int8)
            s["bound_scales"][place] = unit
    return dict(q=q, **_written(s))


def _plain_select(s):
    B, H, Hkv, T, d, page, K = (s[n] for n in ("B", "H", "Hkv", "T", "d", "page", "picks"))
    table = s["block_table"].long()
    W = table.shape[1]
    q = s["q"].float()
    unit = _power(q.abs().amax(-1), 127.0)
    q = torch.round(q / unit[..., None]).reshape(B, Hkv, -1, d)
    q = torch.cat((q.clamp(max=0.0), q.clamp(min=0.0)), -1)                              # meet the lower and the upper bounds
    bounds = s["k_bounds"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, W, 2 * d).float()
    x = torch.matmul(q.double(), bounds.double().transpose(-1, -2)).float()              # whole numbers below 2^24
    x = x * unit.reshape(B, Hkv, -1, 1) * s["bound_scales"][table].transpose(1, 2)[:, :, None, :]
    x = x.amax(2)                                                                        # [B, Hkv, W]
    n = ((s["kv_lens"].long() + page - 1) // page)[:, None, None]
    at = torch.arange(W, device="cuda")
    x = torch.where((at < s["first"]) | (at >= n - s["last"]), math.inf, x)
    x = torch.where(at < n, x, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :K]
    order = torch.where(order < n, order, W).sort(-1).values
    out = torch.full((B, Hkv, K), -1, dtype=torch.int32, device="cuda")
    out[..., : order.shape[-1]] = torch.where(order < W, order, -1).to(torch.int32)
    return dict(pages=out)


def _plain_assign(s):
    page, T = s["page"], s["T"]
    old, new, table, ring = s["old"].long(), s["new"].long(), s["block_table"], s["free_pages"]
    n, W = ring.numel(), table.shape[1]
    held, want = (old + page - 1) // page, (new + page - 1) // page
    grow, less = (want - held).clamp(min=0), (held - want).clamp(min=0)
    first, count = s["free_state"].long()
    j = torch.arange(W, device="cuda")
    comes = (j >= held[:, None]) & (j < want[:, None])
    goes = (j >= want[:, None]) & (j < held[:, None])
    taken = (first + (grow.cumsum(0) - grow)[:, None] + j - held[:, None]) % n
    given = (first + count + (less.cumsum(0) - less)[:, None] + j - want[:, None]) % n
    table.copy_(torch.where(comes, ring[taken], table))
    ring[given[goes]] = table[goes]
    state = torch.stack(((first + grow.sum()) % n, count - grow.sum() + less.sum())).to(torch.int32)
    t = torch.arange(T, device="cuda")
    q_lens = (new - old).clamp(min=0)
    there = t < q_lens[:, None]
    pos = torch.where(there, old[:, None] + t, -1)
    at = torch.gather(table.long(), 1, (pos // page).clamp(0, W - 1))
    slots = torch.where(there, at * page + pos % page, -1)
    return dict(lens=s["new"].clone(), q_lens=q_lens.to(torch.int32), slots=slots, positions=pos.to(torch.int32),
                state=state, table=table, free=ring)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    page = case["page"]
    if case["kind"] == "assign":
        old, new = _assign_lens(case)
        moved = sum(abs(_pages(a, page) - _pages(b, page)) for a, b in zip(old, new))
        # lengths and states; a table entry and a free page for each one moved; places of the new tokens
        return dict(bytes=16 * case["B"] + 16 + 8 * moved + 12 * case["B"] * case["T"], flops=0)
    H, Hkv, T, d = (case[n] for n in ("H", "Hkv", "T", "d"))
    if case["kind"] == "append":
        lens, new = _append_lens(case)
        pages = sum(_pages(a, page) - (a - b) // page for a, b in zip(lens, new) if b)
        rows, size = sum(new), 2 if case["store"] == "16" else 1
        # keys and values read and written, queries too; a scale (and bounds) of each page written
        return dict(bytes=rows * 2 * Hkv * d * (2 + size) + (4 * rows * H * d if case["rot"] else 0)
                    + pages * Hkv * (8 * (size == 1) + (2 * d + 4) * case["bounds"]),
                    flops=3 * rows * (H + Hkv) * case["rot"] + 4 * rows * Hkv * d)
    lens = _cache_lens(case)
    pages = [_pages(n, page) for n in lens]
    if case["kind"] == "select":
        read = sum(n for n in pages if n > case["picks"])                  # few pages are chosen without a look
        return dict(bytes=read * Hkv * (2 * d + 4) + 2 * case["B"] * H * T * d + 4 * case["B"] * Hkv * case["picks"],
                    flops=4 * read * H * T * d)
    size = 2 if case["store"] == "16" else 1
    if case["picks"]:
        keys = sum(n if p <= case["picks"] else (case["picks"] - 1) * page + n - (p - 1) * page for n, p in zip(lens, pages))
        read = sum(min(p, case["picks"]) for p in pages)
    else:
        keys, read = sum(lens), sum(pages)
    rows = case["B"] * T * H
    return dict(bytes=2 * keys * Hkv * d * size + 8 * read * Hkv * (size == 1) + 4 * read * Hkv * (case["picks"] > 0)
                + 4 * rows * d + 4 * rows, flops=4 * keys * T * H * d)


# ---- the definitions in 64 bits, one sequence and head after another -------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "select": _exact_select,
            "assign": _exact_assign}[case["kind"]](s, case)


def _exact_attend(s, case):
    B, H, Hkv, T, d, page = (case[n] for n in ("B", "H", "Hkv", "T", "d", "page"))
    if B * H > 4096:
        return None
    o = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_cache_lens(case)):
        if n == 0:
            continue
        qpos = n - T + torch.arange(T, device="cuda")
        for g in range(Hkv):
            which = torch.arange(_pages(n, page), device="cuda") if s["pages"] is None else s["pages"][b, g]
            which = which[which >= 0].long()
            kpos = (which[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
            at = s["block_table"][b].long()[which]
            k, v = (s[c + "_cache"][at, g].double() for c in "kv")
            if s["k_scales"] is not None:
                k, v = k * s["k_scales"][at, g, None, None].double(), v * s["v_scales"][at, g, None, None].double()
            k, v, kpos = k.reshape(-1, d)[kpos < n], v.reshape(-1, d)[kpos < n], kpos[kpos < n]
            heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            x = s["q"][b, heads].double() @ k.T / math.sqrt(d)
            if s["softcap"] > 0.0:
                x = s["softcap"] * torch.tanh(x / s["softcap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][heads, None, None].double() * (qpos[:, None] - kpos[None, :])
            x = x.masked_fill(kpos[None, :] > qpos[:, None], -math.inf)
            total = torch.logsumexp(x, -1)
            lse[b, heads] = total
            o[b, heads] = torch.exp(x - torch.where(torch.isinf(total), 0.0, total)[..., None]) @ v
    return dict(o=o, lse=lse)


def _exact_turn(x, pos, inv_freq, interleaved):
    """x [heads, N, d] as complex pairs times exp(i * angle)."""
    half = inv_freq.numel()
    r = x[..., : 2 * half].double()
    pairs = r.unflatten(-1, (half, 2)) if interleaved else r.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.ones((pos.numel(), half), device="cuda", dtype=torch.float64), pos.double()[:, None] * inv_freq)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., 2 * half:].double()), -1)


def _exact_grid(y, store):
    """The nearest values that the store holds, ties to the even one."""
    if store == "int8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_append(s, case):
    """Floating outputs only (queries; 8-bit floats and scales): whole numbers are compared as such."""
    page, store = case["page"], case["store"]
    q = None if s["q"] is None else torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    out = {n: None if s[n] is None else s[n].double() for n in ("k_cache", "v_cache", "k_scales", "v_scales", "bound_scales")}
    reach = lambda top, largest: 2.0 ** max(-100, math.ceil(math.log2(top / largest))) if top > 0.0 else 2.0 ** -100  # noqa: E731
    for b, (n, new) in enumerate(zip(*_append_lens(case))):
        pos = torch.arange(n - new, n, device="cuda")
        k, v = s["k"][b, :, :new].double(), s["v"][b, :, :new].double()
        if q is not None and new:
            k = _exact_turn(s["k"][b, :, :new], pos, s["inv_freq"], s["interleaved"])
            q[b, :, :new] = _exact_turn(s["q"][b, :, :new], pos, s["inv_freq"], s["interleaved"])
        for p in range((n - new) // page, _pages(n, page) if new else 0):
            first, end = max(n - new, p * page), min(n, (p + 1) * page)
            at, kept = int(s["block_table"][b, p]), first - p * page
            for name, x in (("k", k), ("v", v)):
                x = x[:, first - (n - new): end - (n - new)]
                top = x.abs().amax((1, 2)).tolist()
                cache, scales = out[name + "_cache"], out[name + "_scales"]
                if store == "16":
                    cache[at, :, kept: end - p * page] = x
                else:
                    was = scales[at].clone()
                    need = torch.tensor([reach(y, _LARGEST[store]) for y in top], dtype=torch.float64, device="cuda")
                    scales[at] = torch.maximum(was, need) if kept else need
                    unit = scales[at][:, None, None]
                    cache[at, :, :kept] = _exact_grid(cache[at, :, :kept] * was[:, None, None] / unit, store)
                    cache[at, :, kept: end - p * page] = _exact_grid(x / unit, store)
                if name == "k" and case["bounds"]:
                    need = torch.tensor([reach(y, 127.0) for y in top], dtype=torch.float64, device="cuda")
                    out["bound_scales"][at] = torch.maximum(out["bound_scales"][at], need) if kept else need
    if store == "int8":
        out["k_cache"] = out["v_cache"] = None
    return dict(q=q, k_bounds=None, **out)


def _exact_select(s, case):
    H, Hkv, page, K = (case[n] for n in ("H", "Hkv", "page", "picks"))
    G = H // Hkv
    out = torch.full((case["B"], Hkv, K), -1, dtype=torch.int32, device="cuda")
    if case["B"] * Hkv > 1024:
        return None
    for b, length in enumerate(_cache_lens(case)):
        n = _pages(length, page)
        at = s["block_table"][b, :n].long()
        for g in range(Hkv):
            q = s["q"][b, g * G:(g + 1) * G].reshape(-1, case["d"]).double()
            top = q.abs().amax(-1, keepdim=True)
            unit = torch.exp2(torch.ceil(torch.log2(top / 127.0)).clamp(min=-100.0))
            q = torch.round(q / unit)
            lo, hi = s["k_bounds"][at, g].double().unbind(1)
            best = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
            for r in range(q.shape[0]):
                best = torch.maximum(best, torch.maximum(q[r] * lo, q[r] * hi).sum(-1) * unit[r])
            best = (best * s["bound_scales"][at, g].double()).tolist()
            forced = lambda p: p < case["first"] or p >= n - case["last"]  # noqa: E731
            chosen = sorted(sorted(range(n), key=lambda p: (not forced(p), 0.0 if forced(p) else -best[p], p))[:K])
            out[b, g, : len(chosen)] = _int32(chosen)
    return dict(pages=out)


def _exact_assign(s, case):
    page, T = case["page"], case["T"]
    table, ring = s["block_table"].tolist(), s["free_pages"].tolist()
    first, count = s["free_state"].tolist()
    n, taken, given = len(ring), 0, 0
    old, new = _assign_lens(case)
    slots, positions = ([[-1] * T for _ in old] for _ in range(2))
    for b, (x, y) in enumerate(zip(old, new)):
        for p in range(_pages(x, page), _pages(y, page)):
            table[b][p] = ring[(first + taken) % n]
            taken += 1
        for t in range(max(0, min(T, y - x))):
            positions[b][t] = x + t
            slots[b][t] = table[b][(x + t) // page] * page + (x + t) % page
    for b, (x, y) in enumerate(zip(old, new)):
        for p in range(_pages(y, page), _pages(x, page)):
            ring[(first + count + given) % n] = table[b][p]
            given += 1
    return dict(lens=_int32(new), q_lens=_int32([max(0, y - x) for x, y in zip(old, new)]),
                slots=torch.tensor(slots, device="cuda"), positions=_int32(positions),
                state=_int32([(first + taken) % n, count - taken + given]), table=_int32(table), free=_int32(ring))
