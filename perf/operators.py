"""Cases and plain forms of the language-model operators: what each one computes, in elementary
torch operations, and the calls that a program makes of the library's own kernels.

Four operators, used together by one decoder: attention whose scores are capped by a tanh, get a
bias linear in distance, or see a prefix or only their own document (training: forward and
backward); rotary positions (forward and backward); the step that rotates new tokens and writes
their keys and values into a paged cache; and attention of the new tokens over that cache.

``own`` selects the library's kernels; otherwise ``run`` computes the plain form.
"""
import math
import random
import zlib

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- the cases -----------------------------------------------------------------------------------

def _scored(name, B, H, Hkv, N, d, dtype, causal=True, softcap=0.0, alibi=False, prefix=False,
            padded=False, docs=0):
    c = dict(kind="scored", B=B, H=H, Hkv=Hkv, N=N, d=d, dtype=dtype, causal=causal, softcap=softcap,
             alibi=alibi, prefix=prefix, padded=padded, docs=docs)
    return dict(c, name=name) if name else c


def _paged(name, B, H, Hkv, T, d, page, dtype, lo, hi, softcap=0.0, alibi=False):
    c = dict(kind="paged", B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, lo=lo, hi=hi,
             softcap=softcap, alibi=alibi)
    return dict(c, name=name) if name else c


def _append(name, B, H, Hkv, T, d, page, dtype, hi, rot, interleaved, ragged):
    c = dict(kind="append", B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype, hi=hi, rot=rot,
             interleaved=interleaved, ragged=ragged)
    return dict(c, name=name) if name else c


def _rotary(name, B, H, N, d, dtype, rot, interleaved, start, stretch, strided):
    c = dict(kind="rotary", B=B, H=H, N=N, d=d, dtype=dtype, rot=rot, interleaved=interleaved,
             start=start, stretch=stretch, strided=strided)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a training step of one layer with capped scores and grouped heads at the longest context
        _scored("scored-8k-cap-gqa", 1, 16, 4, 8192, 128, "bf16", softcap=50.0),
        # the small decoder shape of the benchmark, with a distance bias in place of positions
        _scored("scored-1k-alibi-d64", 8, 12, 12, 1024, 64, "fp16", alibi=True),
        # an encoder batch with padded sequences: capped and biased in both directions
        _scored("scored-pad-both-d64", 4, 16, 16, 511, 64, "bf16", causal=False, softcap=30.0,
                alibi=True, padded=True),
        # documents packed into one row of tokens, each with a prompt that sees itself whole
        _scored("scored-docs-prefix", 1, 8, 2, 6145, 128, "bf16", softcap=30.0, prefix=True, docs=11),
        # one token for one user, short cache: latency
        _paged("paged-b1-short", 1, 32, 8, 1, 128, 16, "bf16", 200, 200),
        # a serving batch of unequal lengths
        _paged("paged-b64-ragged", 64, 32, 8, 1, 128, 64, "bf16", 1, 8192, softcap=50.0),
        # few users, very long contexts: the cache is split over its length
        _paged("paged-b2-128k", 2, 32, 8, 1, 128, 256, "bf16", 100000, 131072),
        # drafted tokens checked in one call, biased scores, one key head per query head
        _paged("paged-draft5-d64", 16, 16, 16, 5, 64, 32, "fp16", 5, 4000, alibi=True),
        # the cache write of a decoding batch, queries rotated in the same call
        _append("append-b64-token", 64, 32, 8, 1, 128, 64, "bf16", 2048, 128, False, False),
        # the cache write of a ragged batch of prompts, a part of each head rotated
        _append("append-prompts", 4, 32, 8, 4096, 128, 64, "bf16", 8192, 64, True, True),
        # a training step's queries, strided as the projection leaves them, forward and backward
        _rotary("rotary-train-16k", 2, 32, 16384, 128, "bf16", 128, False, 0, 1.0, True),
        # positions far into a context stretched eightfold, a quarter of the head, 32-bit values
        _rotary("rotary-far-fp32", 3, 12, 333, 64, "fp32", 16, True, 1000000, 8.0, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scored", "scored", "paged", "paged", "append", "rotary"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "scored":
        Hkv = rng.choice([1, 2, 4])
        H = Hkv * rng.choice([1, 2, 4])
        causal = rng.random() < 0.7
        docs = rng.randint(1, 20) if rng.random() < 0.4 else 0
        N = _log(rng, 2, 6000) if not docs else _log(rng, 40, 6000)
        B = 1 if docs else max(1, min(8, _log(rng, 1, 8), 6000 // N))
        mods = rng.choice([(30.0, False), (0.0, True), (50.0, True), (20.0, False)])
        return _scored(None, B, H, Hkv, N, d, dtype, causal=causal, softcap=mods[0], alibi=mods[1],
                       prefix=causal and rng.random() < 0.4, padded=not docs and rng.random() < 0.3,
                       docs=docs)
    if kind == "paged":
        Hkv = rng.choice([1, 2, 8])
        H = Hkv * rng.choice([1, 3, 4, 8])
        hi = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(128, 131072 // hi)))
        return _paged(None, B, H, Hkv, rng.choice([1, 1, 1, 2, 7]), d, rng.choice([16, 32, 48, 64, 128, 256]),
                      dtype, rng.randint(0, hi), hi, softcap=rng.choice([0.0, 0.0, 30.0]),
                      alibi=rng.random() < 0.3)
    if kind == "append":
        Hkv = rng.choice([1, 2, 8])
        T = _log(rng, 1, 2048) if rng.random() < 0.5 else 1
        return _append(None, _log(rng, 1, max(1, min(128, 8192 // T))), Hkv * rng.choice([1, 3, 4]), Hkv, T,
                       d, rng.choice([16, 32, 48, 64, 256]), dtype, T + _log(rng, 1, 2048),
                       rng.choice([16, 32, d // 2, d]), rng.random() < 0.5, rng.random() < 0.5)
    return _rotary(None, rng.randint(1, 4), rng.choice([1, 3, 8, 20]), _log(rng, 1, 8192), d,
                   rng.choice(["bf16", "fp16", "fp32"]), rng.choice([16, 32, d // 2, d]),
                   rng.random() < 0.5, rng.choice([0, 17, 100000, 1000000]), rng.choice([1.0, 4.0]),
                   rng.random() < 0.5)


# ---- the inputs ----------------------------------------------------------------------------------

def _lengths(case, n, lo, hi, salt):
    """n lengths in [lo, hi] that belong to the case itself, so that its work is known."""
    keys = ("kind", "B", "N", "T", "hi", "docs", "page")
    r = random.Random(zlib.crc32(repr([salt] + [case.get(k) for k in keys]).encode()))
    return [r.randint(lo, hi) for _ in range(n)]


def _documents(case):
    """Lengths of the packed documents."""
    cuts = sorted(_lengths(case, case["docs"] - 1, 0, case["N"], 1))
    ends = cuts + [case["N"]]
    return [b - a for a, b in zip([0] + cuts, ends)]


def _scored_rows(case):
    """(rows, valid keys, prefix) of each sequence or document."""
    if case["docs"]:
        rows = _documents(case)
        keys = rows
    else:
        rows = [case["N"]] * case["B"]
        keys = _lengths(case, case["B"] - 1, 0, case["N"], 2) + [case["N"]] if case["padded"] else rows
    prefix = _lengths(case, len(rows), 0, max(1, case["N"] // (2 * max(1, case["docs"]))), 3) if case["prefix"] else [0] * len(rows)
    return rows, keys, prefix


def _paged_lens(case):
    lens = _lengths(case, case["B"], case.get("lo", case["T"]), case["hi"], 4)
    lens[-1] = case["hi"]
    return lens


def _append_lens(case):
    """(tokens in the cache, the new ones included; new tokens) of each sequence."""
    new = _lengths(case, case["B"], 0, case["T"], 5) if case["ragged"] else [case["T"]] * case["B"]
    old = _lengths(case, case["B"], 0, case["hi"] - case["T"], 6)
    return [a + b for a, b in zip(old, new)], new


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(_TYPES[dtype])


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _slopes(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _cache(g, case, lens):
    """Key and value pages, and a table of them in shuffled order; unused entries name page 0."""
    B, page, Hkv, d = case["B"], case["page"], case["Hkv"], case["d"]
    need = [-(-n // page) for n in lens]
    width, used = max(1, max(need)), sum(need)
    order = torch.randperm(used + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[at] = order[:used]
    shape = (used + 1, Hkv, page, d)
    return _normal(g, shape, case["dtype"]), _normal(g, shape, case["dtype"]), table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    B, H, d = case["B"], case["H"], case["d"]
    if case["kind"] == "scored":
        rows, keys, prefix = _scored_rows(case)
        lead = () if case["docs"] else (B,)
        s["q"] = _normal(g, lead + (H, case["N"], d), case["dtype"], 2.0)
        s["k"] = _normal(g, lead + (case["Hkv"], case["N"], d), case["dtype"])
        s["v"] = _normal(g, lead + (case["Hkv"], case["N"], d), case["dtype"])
        s["do"] = _normal(g, lead + (H, case["N"], d), case["dtype"])
        s["slopes"] = _slopes(H) if case["alibi"] else None
        s["prefix_lens"] = _int32(prefix) if case["prefix"] else None
        s["kv_lens"] = _int32(keys) if case["padded"] else None
        if case["docs"]:
            s["max_seqlen"] = max(rows)
            s["cu_seqlens"] = _int32([sum(rows[:i]) for i in range(len(rows) + 1)])
    elif case["kind"] == "paged":
        lens = _paged_lens(case)
        s["k_cache"], s["v_cache"], s["block_table"] = _cache(g, case, lens)
        s["kv_lens"] = _int32(lens)
        s["q"] = _normal(g, (B, H, case["T"], d), case["dtype"], 2.0)
        s["slopes"] = _slopes(H) if case["alibi"] else None
    elif case["kind"] == "append":
        lens, new = _append_lens(case)
        s["k_cache"], s["v_cache"], s["block_table"] = _cache(g, case, lens)
        s["kv_lens"], s["q_lens"] = _int32(lens), _int32(new)
        # the projections' outputs: [B, T, heads, d], seen as [B, heads, T, d]
        s["q"], s["k"], s["v"] = (_normal(g, (B, case["T"], h, d), case["dtype"]).transpose(1, 2)
                                  for h in (H, case["Hkv"], case["Hkv"]))
        s["inv_freq"] = _frequencies(case["rot"], 1.0)
    else:
        shape = (B, case["N"], H, d) if case["strided"] else (B, H, case["N"], d)
        s["x"], s["dy"] = _normal(g, shape, case["dtype"]), _normal(g, (B, H, case["N"], d), case["dtype"])
        if case["strided"]:
            s["x"] = s["x"].transpose(1, 2)
        s["positions"] = torch.arange(case["N"], device="cuda", dtype=torch.int32) + case["start"]
        s["inv_freq"] = _frequencies(case["rot"], case["stretch"])
        s["mscale"] = 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0
    return s


def _frequencies(rot, stretch):
    """Radians per position of each pair, positions squeezed by ``stretch``."""
    i = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64)
    return torch.pow(torch.tensor(10000.0, device="cuda", dtype=torch.float64), -i / rot) / stretch


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"scored": _plain_scored, "paged": _plain_paged, "append": _plain_append,
            "rotary": _plain_rotary}[s["kind"]](s)


def _run_own(s):
    import exact_io_aware_23_gb300 as fa
    if s["kind"] == "scored":
        mods = dict(causal=s["causal"], softcap=s["softcap"], alibi_slopes=s["slopes"],
                    prefix_lens=s["prefix_lens"])
        if s["docs"]:
            o, lse = fa.forward_varlen(s["q"], s["k"], s["v"], s["cu_seqlens"], s["max_seqlen"], **mods)
            dq, dk, dv = fa.backward_varlen(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu_seqlens"],
                                            s["max_seqlen"], **mods)
        else:
            o, lse = fa.forward(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"], **mods)
            dq, dk, dv = fa.backward(s["q"], s["k"], s["v"], o, lse, s["do"], kv_lens=s["kv_lens"], **mods)
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    if s["kind"] == "paged":
        o, lse = fa.forward_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                  softcap=s["softcap"], alibi_slopes=s["slopes"])
        return dict(o=o, lse=lse)
    if s["kind"] == "append":
        q = fa.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                            q=s["q"], q_lens=s["q_lens"], inv_freq=s["inv_freq"],
                            interleaved=s["interleaved"])
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    rot = dict(interleaved=s["interleaved"], mscale=s["mscale"])
    return dict(y=fa.rotary(s["x"], s["positions"], s["inv_freq"], **rot),
                dx=fa.rotary_backward(s["dy"], s["positions"], s["inv_freq"], **rot))


# ---- plain forms: 32-bit arithmetic, rounded once at the end --------------------------------------

def _plain_masks(s):
    """allowed [B or 1, 1, 1, N, N] and the distance i - j [N, N] of a scored state."""
    N = s["N"]
    n = torch.arange(N, device="cuda")
    if s["docs"]:
        cu = s["cu_seqlens"].long()
        doc = torch.searchsorted(cu[1:], n, right=True)              # a token's document
        pos = n - cu[doc]
        allowed = (doc[:, None] == doc[None, :])[None]
        prefix = None if s["prefix_lens"] is None else s["prefix_lens"].long()[doc][None, None, :]
    else:
        pos = n
        allowed = torch.ones((1, N, N), dtype=torch.bool, device="cuda")
        if s["kv_lens"] is not None:
            allowed = allowed & (n[None, None, :] < s["kv_lens"].long()[:, None, None])
        prefix = None if s["prefix_lens"] is None else s["prefix_lens"].long()[:, None, None]
    if s["causal"]:
        seen = (pos[None, :] <= pos[:, None])[None]
        if prefix is not None:
            seen = seen | (pos < prefix)
        allowed = allowed & seen
    return allowed[:, None, None], pos[:, None] - pos[None, :]


def _plain_scored(s):
    Hkv, G, N, d = s["Hkv"], s["H"] // s["Hkv"], s["N"], s["d"]
    out = s["q"].dtype
    scale = 1.0 / math.sqrt(d)
    q, do = (s[n].float().reshape(-1, Hkv, G, N, d) for n in ("q", "do"))
    k, v = (s[n].float().reshape(-1, Hkv, 1, N, d) for n in ("k", "v"))
    allowed, dist = _plain_masks(s)
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    slope = 1.0
    if s["softcap"] > 0.0:
        t = torch.tanh(x / s["softcap"])
        x, slope = t * s["softcap"], 1.0 - t * t
        del t
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(Hkv, G, 1, 1) * dist.abs().float()
    x = torch.where(allowed, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m0)
    del x
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0.0, 1.0, l)
    lse = torch.where(l == 0.0, -math.inf, m0 + torch.log(l))
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * slope * scale
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    shape, kshape = s["q"].shape, s["k"].shape
    return dict(o=o.reshape(shape).to(out), lse=lse.reshape(shape[:-1]), dq=dq.reshape(shape).to(out),
                dk=dk.reshape(kshape).to(out), dv=dv.reshape(kshape).to(out))


def _plain_paged(s):
    B, H, Hkv, T, d = s["B"], s["H"], s["Hkv"], s["T"], s["d"]
    G = H // Hkv
    lens = s["kv_lens"].long()
    L = s["block_table"].shape[1] * s["page"]
    at = torch.arange(L, device="cuda")
    table = s["block_table"].long()
    k, v = (s[n][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, L, d).float() for n in ("k_cache", "v_cache"))
    there = at[None, :] < lens[:, None]
    v = torch.where(there[:, None, None, :, None], v, 0.0)
    q = s["q"].float().reshape(B, Hkv, G, T, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    if s["softcap"] > 0.0:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    pos = lens[:, None] - T + torch.arange(T, device="cuda")[None, :]           # the new tokens' places
    dist = pos[:, None, None, :, None] - at
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(Hkv, G, 1, 1) * dist.float()
    x = torch.where((dist >= 0) & there[:, None, None, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0.0, 1.0, l)
    lse = torch.where(l == 0.0, -math.inf, m + torch.log(l))
    return dict(o=o.reshape(B, H, T, d).to(s["q"].dtype), lse=lse.reshape(B, H, T))


def _plain_turn(x, positions, inv_freq, interleaved, mscale, back=False):
    """x [.., heads, N, d] with pair i of each head turned by position * inv_freq[i]."""
    half = inv_freq.numel()
    angle = positions.double()[..., None] * inv_freq
    cos, sin = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    cos, sin = (t.unsqueeze(-3) for t in (cos, -sin if back else sin))          # every head alike
    x = x.float()
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, rest), -1)


def _plain_append(s):
    T, page = s["T"], s["page"]
    lens, new = s["kv_lens"].long(), s["q_lens"].long()
    t = torch.arange(T, device="cuda")
    pos = (lens - new)[:, None] + t                                              # [B, T]
    there = t[None, :] < new[:, None]
    q, k = (_plain_turn(s[n], pos, s["inv_freq"], s["interleaved"], 1.0).to(s["q"].dtype) for n in ("q", "k"))
    q = torch.where(there[:, None, :, None], q, torch.zeros((), dtype=q.dtype, device="cuda"))
    b, at = torch.nonzero(there, as_tuple=True)
    p = pos[b, at]
    rows = s["block_table"].long()[b, p // page]
    s["k_cache"][rows, :, p % page] = k[b, :, at]
    s["v_cache"][rows, :, p % page] = s["v"][b, :, at]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_rotary(s):
    out = s["x"].dtype
    y = _plain_turn(s["x"], s["positions"], s["inv_freq"], s["interleaved"], s["mscale"])
    dx = _plain_turn(s["dy"], s["positions"], s["inv_freq"], s["interleaved"], s["mscale"], back=True)
    return dict(y=y.to(out).contiguous(), dx=dx.to(out).contiguous())


# ---- what a pass cannot do without ---------------------------------------------------------------

def _pairs(case):
    """Query-key pairs that a scored case's masks leave, over sequences, for one head."""
    total = 0
    for rows, keys, prefix in zip(*_scored_rows(case)):
        keys = min(keys, rows)
        if not case["causal"]:
            total += rows * keys
            continue
        f = min(prefix, keys)                       # every row sees at least the prefix
        total += rows * f + sum(min(i + 1, keys) - f for i in range(f, rows))
    return total


def work(case):
    H, Hkv, d = case["H"], case.get("Hkv", case["H"]), case["d"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] == "scored":
        # q, k, v, do read; o, dq, dk, dv and the row statistic written; two products forward, five back
        rows = case["B"] * case["N"]
        return dict(bytes=rows * (4 * H + 4 * Hkv) * d * size + 4 * rows * H,
                    flops=14 * _pairs(case) * H * d)
    if case["kind"] == "paged":
        keys, rows = sum(_paged_lens(case)), case["B"] * case["T"] * H
        return dict(bytes=2 * keys * Hkv * d * size + 2 * rows * d * size + 4 * rows, flops=4 * keys * case["T"] * H * d)
    if case["kind"] == "append":
        new = sum(_append_lens(case)[1])
        return dict(bytes=2 * new * (H + 2 * Hkv) * d * size, flops=3 * new * (H + Hkv) * case["rot"])
    n = case["B"] * H * case["N"]
    return dict(bytes=4 * n * d * size, flops=2 * 3 * n * case["rot"])


# ---- the definitions in 64 bits, row by row ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"scored": _exact_scored, "paged": _exact_paged, "append": _exact_append,
            "rotary": _exact_rotary}[case["kind"]](s, case)


def _exact_scores(s, h, q, k, qpos, kpos):
    """Scores of one head in 64 bits, and their derivative by the scaled product."""
    x = q @ k.T / math.sqrt(s["d"])
    dx = torch.ones_like(x)
    if s["softcap"] > 0.0:
        t = torch.tanh(x / s["softcap"])
        x, dx = s["softcap"] * t, 1.0 / torch.cosh(x / s["softcap"]) ** 2
    if s["slopes"] is not None:
        x = x - s["slopes"][h].double() * (qpos[:, None] - kpos[None, :]).abs()
    return x, dx


def _exact_softmax(x):
    """Row probabilities and log of the sum; rows without a key give zeros and -inf."""
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p, lse


def _exact_scored(s, case):
    H, Hkv, N, d = (case[n] for n in ("H", "Hkv", "N", "d"))
    rows, keys, prefix = _scored_rows(case)
    if sum(n * n for n in rows) * H > 3e9:
        return None
    q, do = (s[n].reshape(-1, H, N, d) for n in ("q", "do"))
    k, v = (s[n].reshape(-1, Hkv, N, d) for n in ("k", "v"))
    o, dq, dk, dv = (torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (q, q, k, k))
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    begin = 0
    for i, (n, nk, f) in enumerate(zip(rows, keys, prefix)):
        b, at = (0, slice(begin, begin + n)) if case["docs"] else (i, slice(0, n))
        begin += n
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        hidden = (pos[None, :] >= nk).expand(n, n)
        if case["causal"]:
            hidden = hidden | ((pos[None, :] > pos[:, None]) & (pos[None, :] >= f))
        for h in range(H):
            g = h // (H // Hkv)
            qh, kh, vh, gh = q[b, h, at].double(), k[b, g, at].double(), v[b, g, at].double(), do[b, h, at].double()
            x, dx = _exact_scores(s, h, qh, kh, pos, pos)
            p, lse[b, h, at] = _exact_softmax(x.masked_fill(hidden, -math.inf))
            o[b, h, at] = p @ vh
            dp = gh @ vh.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * dx / math.sqrt(d)
            dq[b, h, at] = ds @ kh
            dk[b, g, at] += ds.T @ qh
            dv[b, g, at] += p.T @ gh
    shape = s["q"].shape
    return dict(o=o.reshape(shape), lse=lse.reshape(shape[:-1]), dq=dq.reshape(shape),
                dk=dk.reshape(s["k"].shape), dv=dv.reshape(s["v"].shape))


def _exact_paged(s, case):
    B, H, Hkv, T, d, page = (case[n] for n in ("B", "H", "Hkv", "T", "d", "page"))
    o = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_paged_lens(case)):
        if n == 0:
            continue
        pages = s["block_table"][b, : -(-n // page)].long()
        kpos = torch.arange(n, device="cuda")
        qpos = n - T + torch.arange(T, device="cuda")
        for g in range(Hkv):
            k, v = (s[c][pages, g].reshape(-1, d)[:n].double() for c in ("k_cache", "v_cache"))
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                x, _ = _exact_scores(s, h, s["q"][b, h].double(), k, qpos, kpos)
                p, lse[b, h] = _exact_softmax(x.masked_fill(kpos[None, :] > qpos[:, None], -math.inf))
                o[b, h] = p @ v
    return dict(o=o, lse=lse)


def _exact_turn(x, pos, inv_freq, interleaved, mscale, sign):
    """x [.., N, d] as complex pairs times mscale * exp(i * sign * angle)."""
    half = inv_freq.numel()
    r = x[..., : 2 * half].double()
    pairs = r.unflatten(-1, (half, 2)) if interleaved else r.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(inv_freq, mscale).expand(pos.numel(), half), sign * pos.double()[:, None] * inv_freq)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., 2 * half:].double()), -1)


def _exact_append(s, case):
    page = case["page"]
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b, (n, new) in enumerate(zip(*_append_lens(case))):
        if new == 0:
            continue
        pos = torch.arange(n - new, n, device="cuda")
        at = s["block_table"][b].long()[pos // page]
        q[b, :, :new] = _exact_turn(s["q"][b, :, :new], pos, s["inv_freq"], s["interleaved"], 1.0, 1)
        kc[at, :, pos % page] = _exact_turn(s["k"][b, :, :new], pos, s["inv_freq"], s["interleaved"], 1.0, 1).transpose(0, 1)
        vc[at, :, pos % page] = s["v"][b, :, :new].transpose(0, 1).double()
    return dict(q=q, k_cache=kc, v_cache=vc)


def _exact_rotary(s, case):
    turn = lambda x, sign: _exact_turn(x, s["positions"], s["inv_freq"], s["interleaved"], s["mscale"], sign)  # noqa: E731
    return dict(y=turn(s["x"], 1), dx=turn(s["dy"], -1))
