"""Host-side argument checks of the calls on 8-bit and chosen pages, of the choice itself and of the pages'
assignment: the documented status before any CUDA call (CPU only: no kernel runs)."""
import ctypes
import os
import re

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_abi_serving import BAD_CACHES, DENSE, INVALID, OK, P, S3, UNSUPPORTED, cache

Q = P + (1 << 20)


def store(**kw):
    c = dict(format=2, k_scales=P, v_scales=Q, k_bounds=None, bound_scales=None)
    c.update(kw)
    return ctypes.byref(fa.FaPageStore(*[c[n] for n, _ in fa.FaPageStore._fields_]))


BAD_STORES = [(dict(format=3), UNSUPPORTED), (dict(format=-1), UNSUPPORTED), (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID),
              (dict(k_scales=P + 2), INVALID), (dict(v_scales=P + 1, format=1), INVALID)]
BAD_BOUNDS = [(dict(k_bounds=P + 8, bound_scales=P), INVALID), (dict(k_bounds=P), INVALID), (dict(k_bounds=P, bound_scales=P + 2), INVALID)]


def append(c=None, s=None, k=P, ks=DENSE, q=None, B=2, H=4, Hkv=2, T=1, d=64, dtype=0):
    return fa.lib.fa_append_paged_store(cache(v_cache=P + 4096) if c is None else c, store() if s is None else s, k, ks, P, DENSE, q, DENSE, None,
                                        B, H, Hkv, T, d, None, None, 0, 0, 1.0, dtype, None)


def test_append_checks():
    for kw, status in BAD_CACHES:
        assert append(cache(**{"v_cache": P + 4096, **kw})) == status, kw
    for kw, status in BAD_STORES + BAD_BOUNDS:
        assert append(s=store(**kw)) == status, kw
    assert append(s=store(v_scales=P)) == INVALID                          # one place for both scales
    assert append(s=store(k_bounds=P, bound_scales=P)) == INVALID
    assert append(cache(v_cache=P + 4096, token_stride=72)) == INVALID     # rows of 8-bit values off the 16-byte grid
    assert append(cache(v_cache=P + 4096, head_stride=8)) == INVALID
    assert append(cache()) == INVALID                                      # keys and values in one place
    assert append(k=None) == INVALID
    assert append(q=P) == INVALID                                          # queries without a place for them
    assert append(dtype=1) == UNSUPPORTED
    assert append(q=P, Hkv=3) == UNSUPPORTED
    assert append(d=96) == UNSUPPORTED
    assert append(B=0, s=store(format=9)) == OK
    assert append(T=0, k=None) == OK


def forward(c=None, s=None, pages=None, n=0, q=P, B=2, H=4, Hkv=2, T=1, d=64, dtype=0, w=P, wsb=None, mod=None):
    wsb = fa.forward_paged_workspace_size(2, 4, 2, 1, 64, 1600) if wsb is None else wsb
    return fa.lib.fa_forward_paged_store(q, cache(max_pages=100, table_stride=100) if c is None else c, store() if s is None else s, pages, n, P, P,
                                         B, H, Hkv, T, d, 0.125, None, mod, dtype, w, wsb, None)


def test_forward_checks():
    for kw, status in BAD_CACHES:
        assert forward(cache(**kw)) == status, kw
    for kw, status in BAD_STORES:
        assert forward(s=store(**kw)) == status, kw
    assert forward(cache(max_pages=100, table_stride=100, token_stride=72)) == INVALID
    assert forward(w=None) == INVALID
    assert forward(wsb=256) == INVALID
    assert forward(pages=P, n=0, w=None) == INVALID
    assert forward(pages=P, n=-1, w=None) == INVALID
    assert forward(pages=P + 2, n=4, w=None) == INVALID
    assert forward(pages=P, n=99, w=None) == INVALID                       # 1584 keys: a workspace is needed
    assert forward(pages=P, n=99, wsb=256) == INVALID
    many = cache(max_pages=1 << 20, table_stride=1 << 20, page_size=4096)
    assert forward(many, B=60000, H=4, Hkv=4) == UNSUPPORTED               # more tiles than 31 bits count
    long = cache(max_pages=1 << 19, table_stride=1 << 19, page_size=4096)
    assert forward(long, pages=P, n=4) == UNSUPPORTED                      # places that mark keys which do not exist
    assert forward(q=None) == INVALID
    assert forward(dtype=1) == UNSUPPORTED
    assert forward(mod=ctypes.byref(fa.FaScoreMod(-1.0, None, None))) == INVALID
    assert forward(B=0, s=store(format=9)) == OK


def select(c=None, s=None, q=P, pages=P, B=2, H=4, Hkv=2, T=1, d=64, n=4, first=1, last=1, dtype=0, w=P, wsb=1 << 20):
    return fa.lib.fa_select_pages(q, cache(max_pages=100, table_stride=100, k_cache=None, v_cache=None) if c is None else c,
                                  store(k_bounds=P, bound_scales=P) if s is None else s, pages, B, H, Hkv, T, d, None, n, first, last, dtype, w, wsb, None)


def test_select_checks():
    assert fa.select_pages_workspace_size(2, 2, 1000, 10) == 16128         # 16000 bytes, in steps of 256
    assert fa.select_pages_workspace_size(2, 2, 512, 10) == 0              # few pages,
    assert fa.select_pages_workspace_size(400, 2, 1000, 10) == 0           # many sequences,
    assert fa.select_pages_workspace_size(2, 2, 1000, 1000) == 0           # no choice
    assert fa.select_pages_workspace_size(0, 2, 1000, 10) == 0
    wide = cache(max_pages=1000, table_stride=1000, k_cache=None, v_cache=None)
    assert select(wide, w=None) == INVALID
    assert select(wide, w=P + 16) == INVALID
    assert select(wide, wsb=16000) == INVALID
    for kw, status in BAD_CACHES:
        if "k_cache" not in kw and "v_cache" not in kw and not any("stride" in n and n != "table_stride" for n in kw):
            assert select(cache(**kw)) == status, kw
    for kw, status in BAD_BOUNDS + [(dict(), INVALID)]:
        assert select(s=store(**kw)) == status, kw
    assert fa.lib.fa_select_pages(P, cache(), None, P, 2, 4, 2, 1, 64, None, 4, 1, 1, 0, P, 1 << 20, None) == INVALID
    assert select(q=None) == INVALID
    assert select(q=P + 8) == INVALID
    assert select(pages=None) == INVALID
    assert select(n=-1) == INVALID
    assert select(first=-1) == INVALID
    assert select(last=-2) == INVALID
    assert select(dtype=1) == UNSUPPORTED
    assert select(Hkv=3) == UNSUPPORTED
    assert select(cache(max_pages=49153, table_stride=49153)) == UNSUPPORTED
    assert select(n=0, q=None) == OK
    assert select(B=0, q=None) == OK


def assign(table=P, stride=8, B=2, width=8, page=16, old=P, new=P, ring=P, n=4, state=P, state2=P, lens=P, q_lens=P, slots=P, pos=P, T=1):
    return fa.lib.fa_assign_pages(table, stride, B, width, page, old, new, ring, n, state, state2, lens, q_lens, slots, pos, T, None)


def test_assign_checks():
    for kw in (dict(table=None), dict(table=P + 2), dict(stride=7), dict(B=-1), dict(width=-1), dict(page=0), dict(old=None), dict(new=P + 1),
               dict(ring=None), dict(n=0), dict(n=-1), dict(state=None), dict(state2=None), dict(lens=None), dict(q_lens=None), dict(slots=None),
               dict(slots=P + 4), dict(pos=None), dict(T=-1)):
        assert assign(**kw) == INVALID, kw
    for kw in (dict(page=24), dict(page=8192), dict(B=65536), dict(B=60000, T=60000)):
        assert assign(**kw) == UNSUPPORTED, kw


def test_packed_layouts():
    for fn in (fa.lib.fa_select_pages_packed, fa.lib.fa_assign_pages_packed):
        assert fn(None) == INVALID
    assert fa.lib.fa_append_paged_store_packed(None) == INVALID
    assert fa.lib.fa_forward_paged_store_packed(None) == INVALID
    header = open(os.path.join(os.path.dirname(fa.LIB_PATH), os.pardir, "include", "fa.h")).read()
    size = {"int": 4, "float": 4, "fa_paged_cache": ctypes.sizeof(fa.FaPagedCache), "fa_page_store": ctypes.sizeof(fa.FaPageStore),
            "fa_append_paged_call": fa._APPEND.size, "fa_forward_paged_call": fa._PAGED.size}
    for name, packed in (("fa_select_pages_call", fa._SELECT), ("fa_assign_pages_call", fa._ASSIGN),
                         ("fa_append_paged_store_call", fa._APPEND_STORE), ("fa_forward_paged_store_call", fa._PAGED_STORE)):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", header).group(1)
        total = 0
        for field in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";")[:-1]:
            kind = field.split()[1 if field.split()[0] == "const" else 0]
            total += sum(8 if "*" in one else size.get(kind, 8) for one in field.split(","))
        assert packed.size == (total + 7) // 8 * 8, name


def test_host_tensors_are_refused():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    table, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.select_pages(q, torch.zeros(2, 2, 2, 64, dtype=torch.int8), torch.zeros(2, 2), table, n, 1, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.assign_pages(table, n, n, n, n, 16)


def test_assign_sizes_that_end_behind_31_bits():
    for T in (2 ** 31 - 1, 2 ** 31 - 2047, 2 ** 31 - 4096):
        assert assign(B=1, T=T) == UNSUPPORTED
    assert assign(B=1, T=2 ** 31 - 4097, slots=None) == INVALID           # of a size that is looked at


def test_lists_that_end_behind_31_bits():
    for n in (2 ** 31 - 1, 2 ** 31 - 4096):
        assert select(n=n) == UNSUPPORTED
    assert select(n=2 ** 31 - 4097, q=None) == INVALID                     # of a length that is looked at
