"""Host-side argument checks of the rotary and paged-cache calls: the documented status before any
CUDA call (CPU only: no kernel runs)."""
import ctypes
import os
import re

import pytest
import torch

import exact_io_aware_23_gb300 as fa

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000                        # aligned, never dereferenced: every call below returns early
S3 = ctypes.c_int64 * 3
DENSE = S3(1 << 20, 1 << 13, 64)


def rotary(fn, x=P, xs=DENSE, y=P, ys=DENSE, B=1, H=2, N=8, d=64, pos=P, ps=0, inv=P, rot=64, mscale=1.0, dtype=0):
    return fn(x, xs, y, ys, B, H, N, d, pos, ps, inv, rot, 0, mscale, dtype, None)


@pytest.mark.parametrize("fn", [fa.lib.fa_rotary, fa.lib.fa_rotary_backward])
def test_rotary_argument_checks(fn):
    assert rotary(fn, d=96) == UNSUPPORTED
    assert rotary(fn, dtype=9) == UNSUPPORTED
    assert rotary(fn, rot=24) == UNSUPPORTED
    assert rotary(fn, rot=80) == UNSUPPORTED              # more than the head
    assert rotary(fn, rot=-16) == INVALID
    assert rotary(fn, B=-1) == INVALID
    assert rotary(fn, B=65536) == UNSUPPORTED
    assert rotary(fn, B=60000, H=60000, N=60000) == UNSUPPORTED
    assert rotary(fn, inv=None) == INVALID
    assert rotary(fn, mscale=float("nan")) == INVALID
    assert rotary(fn, x=None) == INVALID
    assert rotary(fn, y=P + 8) == INVALID
    assert rotary(fn, pos=None) == INVALID
    assert rotary(fn, ps=-1) == INVALID
    assert rotary(fn, xs=S3(1 << 20, 1 << 13, 68)) == INVALID          # rows off the 16-byte grid
    assert rotary(fn, ys=S3(1 << 20, 4, 64)) == INVALID
    assert rotary(fn, ys=S3(0, 32, 64)) == INVALID        # heads that overlap
    assert rotary(fn, B=2, ys=S3(0, 1 << 13, 64)) == INVALID
    for empty in (dict(B=0), dict(H=0), dict(N=0)):
        assert rotary(fn, x=None, pos=None, **empty) == OK


def cache(**kw):
    c = dict(k_cache=P, v_cache=P, page_stride=1 << 12, head_stride=1 << 10, token_stride=64, n_pages=4,
             page_size=16, block_table=P, table_stride=3, max_pages=3, kv_lens=P)
    c.update(kw)
    return ctypes.byref(fa.FaPagedCache(*[c[n] for n, _ in fa.FaPagedCache._fields_]))


BAD_CACHES = [(dict(k_cache=None), INVALID), (dict(v_cache=P + 8), INVALID), (dict(page_size=0), INVALID),
              (dict(page_size=24), UNSUPPORTED), (dict(page_size=8192), UNSUPPORTED), (dict(n_pages=-1), INVALID), (dict(token_stride=65), INVALID),
              (dict(head_stride=4), INVALID), (dict(page_stride=4), INVALID), (dict(block_table=None), INVALID),
              (dict(kv_lens=None), INVALID), (dict(table_stride=2), INVALID), (dict(max_pages=-1), INVALID)]


def append(c=None, k=P, ks=DENSE, v=P, q=P, qs=DENSE, q_out=P, B=2, H=4, Hkv=2, T=1, d=64, inv=P, rot=64, dtype=0, q_lens=None):
    return fa.lib.fa_append_paged(cache() if c is None else c, k, ks, v, DENSE, q, qs, q_out, B, H, Hkv, T, d, q_lens, inv,
                                  rot, 0, 1.0, dtype, None)


def test_append_argument_checks():
    for kw, status in BAD_CACHES:
        assert append(cache(**kw)) == status, kw
    assert append(dtype=1) == UNSUPPORTED                 # the cache is 16 bits
    assert append() == INVALID                            # keys and values in one place
    assert append(cache(v_cache=P + 4096, page_stride=0)) == INVALID
    assert append(cache(v_cache=P + 4096, token_stride=32)) == INVALID
    assert append(Hkv=3) == UNSUPPORTED
    assert append(B=0, c=cache(kv_lens=None)) == OK
    assert append(Hkv=0) == INVALID
    assert append(d=80) == UNSUPPORTED
    assert append(rot=40) == UNSUPPORTED
    assert append(inv=None) == INVALID
    assert append(k=None) == INVALID
    assert append(v=P + 2) == INVALID
    assert append(q_out=None) == INVALID
    assert append(q=P + 4) == INVALID
    assert append(ks=S3(1 << 20, 12, 64)) == INVALID
    assert append(q_lens=P + 1) == INVALID
    assert append(T=0, k=None) == OK
    assert append(B=0, k=None) == OK


def paged(c=None, q=P, o=P, lse=P, B=2, H=4, Hkv=2, T=1, d=64, scale=0.125, mod=None, dtype=0, w=P, wsb=None):
    wsb = fa.forward_paged_workspace_size(2, 4, 2, 1, 64, 1600) if wsb is None else wsb
    return fa.lib.fa_forward_paged(q, cache(max_pages=100, table_stride=100) if c is None else c, o, lse, B, H, Hkv, T, d, scale, None,
                                   None if mod is None else ctypes.byref(mod), dtype, w, wsb, None)


def test_paged_attention_argument_checks():
    for kw, status in BAD_CACHES:
        assert paged(cache(**kw)) == status, kw
    ws = fa.forward_paged_workspace_size(2, 4, 2, 1, 64, 1600)
    assert ws % 256 == 0 and ws > 0
    assert fa.forward_paged_workspace_size(2, 4, 2, 1, 128, 1600) > ws
    assert fa.forward_paged_workspace_size(0, 4, 2, 1, 64, 1600) == 0
    assert fa.forward_paged_workspace_size(2, 4, 3, 1, 64, 1600) == 0
    assert fa.forward_paged_workspace_size(2, 4, 2, 1, 64, 512) == 0       # a CTA each: none needed
    assert fa.forward_paged_workspace_size(9999, 4, 2, 1, 64, 512) == ws   # too many for that
    many = cache(max_pages=1 << 20, table_stride=1 << 20, page_size=4096)
    assert paged(many, B=60000, H=4, Hkv=4) == UNSUPPORTED                 # more tiles than 31 bits count
    assert paged(dtype=1) == UNSUPPORTED
    assert paged(d=96) == UNSUPPORTED
    assert paged(Hkv=3) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert paged(scale=bad) == INVALID
    assert paged(q=None) == INVALID
    assert paged(o=P + 8) == INVALID
    assert paged(lse=None) == INVALID
    assert paged(w=None) == INVALID
    assert paged(w=P + 16) == INVALID
    assert paged(wsb=ws - 256) == INVALID
    for bad in (-1.0, float("nan"), float("inf")):
        assert paged(mod=fa.FaScoreMod(bad, None, None)) == INVALID
    assert paged(mod=fa.FaScoreMod(0.0, None, P)) == UNSUPPORTED       # no prefix over a cache
    assert paged(mod=fa.FaScoreMod(0.0, P + 2, None)) == INVALID
    assert paged(T=0, q=None) == OK
    assert paged(B=0, q=None) == OK


def test_host_tensors_are_refused():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    pos = torch.arange(8, dtype=torch.int32)
    inv, _ = fa.rotary_frequencies(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.rotary(x, pos, inv)
    table, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    pages = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.append_paged(x, x, pages, pages.clone(), table, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.forward_paged(x, pages, pages.clone(), table, n)


def test_scored_argument_checks():
    """The score arguments are checked with the plain calls' own checks, and before any launch."""
    ws = fa.backward_deterministic_workspace_size(2, 8, 100)

    def fwd(mod, dtype=0, H=8, Hkv=2, N=128, d=64, scale=0.125, q=P):
        return fa.lib.fa_forward_scored(q, P, P, P, P, 2, H, Hkv, N, d, scale, 1, dtype, None, mod, None)

    def bwd(mod, dtype=0, H=8, Hkv=2, N=100, d=64, scale=0.125, q=P, w=P, wsb=ws):
        return fa.lib.fa_backward_scored(q, P, P, P, P, P, P, P, P, 2, H, Hkv, N, d, scale, 1, dtype, None, mod, w, wsb, None)

    def fwd_v(mod, dtype=0, H=8, Hkv=2, N=100, d=64, scale=0.125, q=P):
        return fa.lib.fa_forward_varlen_scored(q, P, P, P, P, P, 3, N, N, H, Hkv, d, scale, 1, dtype, mod, None)

    def bwd_v(mod, dtype=0, H=8, Hkv=2, N=100, d=64, scale=0.125, q=P, w=P, wsb=ws):
        return fa.lib.fa_backward_varlen_scored(q, P, P, P, P, P, P, P, P, P, 3, N, N, H, Hkv, d, scale, 1, dtype, mod, w,
                                                wsb, None)
    good = fa.FaScoreMod(30.0, P, P)
    for call in (fwd, bwd, fwd_v, bwd_v):
        assert call(None) == INVALID
        for bad in (-1.0, float("nan"), float("inf")):
            assert call(fa.FaScoreMod(bad, None, None)) == INVALID
        assert call(fa.FaScoreMod(0.0, P + 2, None)) == INVALID
        assert call(fa.FaScoreMod(0.0, None, P + 1)) == INVALID
        assert call(fa.FaScoreMod(1e-41, None, None)) == UNSUPPORTED       # 1 / softcap beyond fp32
        assert call(good, dtype=1) == UNSUPPORTED
        assert call(good, d=96) == UNSUPPORTED
        assert call(good, Hkv=3) == UNSUPPORTED
        assert call(good, scale=0.0) == INVALID
        assert call(good, q=None) == INVALID
        assert call(good, N=0) == OK
    for call in (bwd, bwd_v):
        assert call(good, w=None) == INVALID
        assert call(good, w=P + 16) == INVALID
    assert bwd(good, wsb=ws - 4) == INVALID


def test_packed_calls():
    """One structure in place of the arguments: the same checks, and the layouts of the header."""
    for fn in (fa.lib.fa_forward_scored_packed, fa.lib.fa_backward_scored_packed, fa.lib.fa_rotary_packed,
               fa.lib.fa_rotary_backward_packed, fa.lib.fa_append_paged_packed, fa.lib.fa_forward_paged_packed):
        assert fn(None) == INVALID
    header = open(os.path.join(os.path.dirname(fa.LIB_PATH), os.pardir, "include", "fa.h")).read()
    size = {"int": 4, "float": 4, "fa_paged_cache": ctypes.sizeof(fa.FaPagedCache)}      # others: 8
    for name, packed in (("fa_scored_call", fa._SCORED), ("fa_rotary_call", fa._ROTARY),
                         ("fa_append_paged_call", fa._APPEND), ("fa_forward_paged_call", fa._PAGED)):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", header).group(1)
        total = 0
        for field in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";")[:-1]:
            kind = field.split()[1 if field.split()[0] == "const" else 0]
            for one in field.split(","):
                n = int((re.findall(r"\[(\d+)\]", one) or [1])[0])
                total += n * (8 if "*" in one else size.get(kind, 8))
        assert packed.size == (total + 7) // 8 * 8, name

    rot = dict(x=P, y=P, pos=P, inv=P, xs=(1 << 16, 1 << 13, 64), ys=(1 << 16, 1 << 13, 64), B=1, H=2, N=8, d=64, rot=0)
    def rotary_packed(**kw):
        c = dict(rot, **kw)
        return fa.lib.fa_rotary_packed(fa._ROTARY.pack(c["x"], c["y"], c["pos"], c["inv"], 0, *c["xs"], *c["ys"], 0,
                                                       c["B"], c["H"], c["N"], c["d"], c["rot"], 0, 0, 1.0))
    assert rotary_packed(N=0) == OK
    assert rotary_packed(x=0) == INVALID
    assert rotary_packed(d=80) == UNSUPPORTED
    assert rotary_packed(rot=40) == UNSUPPORTED
    assert rotary_packed(ys=(0, 32, 64)) == INVALID

    def scored_packed(fn, q=P, kv_lens=0, cu=0, B=1, N=64, d=64, scale=0.1, softcap=30.0, ws=1 << 20):
        return fn(fa._SCORED.pack(q, P, P, P, P, P, P, P, P, kv_lens, cu, 0, 0, P, ws, 0, B, 2, 2, N, 128, d, 1, 0,
                                  scale, softcap))
    for fn in (fa.lib.fa_forward_scored_packed, fa.lib.fa_backward_scored_packed):
        assert scored_packed(fn, N=0) == OK
        assert scored_packed(fn, cu=P, B=0) == OK
        assert scored_packed(fn, cu=P, kv_lens=P) == INVALID
        assert scored_packed(fn, q=0) == INVALID
        assert scored_packed(fn, softcap=-1.0) == INVALID
        assert scored_packed(fn, scale=0.0) == INVALID
        assert scored_packed(fn, d=80) == UNSUPPORTED
    assert scored_packed(fa.lib.fa_backward_scored_packed, ws=0) == INVALID

    c = (P, P + 4096, 4096, 1024, 64, 4, 16, P, 8, 8, P)
    def append_packed(B=1, d=64, k=P, q=0):
        return fa.lib.fa_append_paged_packed(fa._APPEND.pack(*c, k, P, q, 0, 0, 0, 0, *(1 << 16, 1 << 13, 64) * 3,
                                                             B, 2, 2, 1, d, 0, 0, 0, 1.0))
    assert append_packed(B=0) == OK
    assert append_packed(k=0) == INVALID
    assert append_packed(q=P) == INVALID                  # queries without a place for them
    assert append_packed(d=80) == UNSUPPORTED

    def paged_packed(B=1, d=64, q=P, scale=0.1, softcap=0.0):
        return fa.lib.fa_forward_paged_packed(fa._PAGED.pack(*c, q, P, P, 0, 0, 0, 0, 0, B, 2, 2, 1, d, 0, scale, softcap))
    assert paged_packed(B=0) == OK
    assert paged_packed(q=0) == INVALID
    assert paged_packed(scale=0.0) == INVALID
    assert paged_packed(softcap=float("inf")) == INVALID
    assert paged_packed(d=80) == UNSUPPORTED
