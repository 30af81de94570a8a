"""Scored attention on the GPU: scores capped by a tanh, lowered by a bias linear in distance, prefix
and document masks, forward and backward, against 64-bit formulas (bounds in scored_reference.py)."""
import math

import pytest
import torch

import exact_io_aware_23_gb300 as fa
from scored_reference import assert_within, head_backward, head_forward

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _slopes(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _inputs(lead, H, Hkv, N, d, dtype, seed, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h, m=1.0: (torch.randn(lead + (h, N, d), generator=g, device="cuda") * m).to(TYPES[dtype])  # noqa: E731
    return r(H, q_scale), r(Hkv), r(Hkv), r(H)


def _check_sequence(t, out, at, n, nk, prefix, causal, cap, slopes, scale, dtype, b=None):
    """Compares one sequence (rows `at` of batch b, or of the packed axis) with the formulas."""
    q, k, v, do = t
    o, lse, dq, dk, dv = out
    pick = (lambda x, h: x[h, at]) if b is None else (lambda x, h: x[b, h, at])
    H, Hkv, u = q.shape[-3], k.shape[-3], torch.finfo(q.dtype).eps / 2
    pos = torch.arange(n, device="cuda")
    allowed = (pos[None, :] < nk).expand(n, n)
    if causal:
        allowed = allowed & ((pos[None, :] <= pos[:, None]) | (pos[None, :] < prefix))
    dist = (pos[:, None] - pos[None, :]).abs().double()
    tiny = TINY[dtype]
    for g in range(Hkv):
        sums = [0.0, 0.0, 0.0, 0.0]
        kk, vv = (torch.where((pos < nk)[:, None], pick(x, g).double(), 0.0) for x in (k, v))
        for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
            slope = 0.0 if slopes is None else float(slopes[h])
            ro, rl, ot, lt = head_forward(pick(q, h).double(), kk, vv, allowed, dist, scale, cap, slope, u, tiny)
            assert_within(f"O {b} {h}", pick(o, h), ro, ot)
            assert_within(f"LSE {b} {h}", pick(lse, h), rl, lt)
            rq, rk, rv, qt, kt, vt = head_backward(pick(q, h).double(), kk, vv, pick(do, h).double(), allowed, dist, scale, cap, slope, u, tiny)
            # P is rebuilt from the fp32 LSE: its error is one of P's, relative
            assert_within(f"dQ {b} {h}", pick(dq, h), rq, qt)
            for i, x in enumerate((rk, rv, kt, vt)):
                sums[i] = sums[i] + x
        assert_within(f"dK {b} {g}", pick(dk, g), sums[0], sums[2])
        assert_within(f"dV {b} {g}", pick(dv, g), sums[1], sums[3])


def _batch(B, H, Hkv, N, d, dtype="bf16", causal=True, cap=0.0, alibi=False, prefix=None, kv=None, scale=None,
           seed=0, q_scale=2.0, fill=float("nan")):
    t = _inputs((B,), H, Hkv, N, d, dtype, seed, q_scale)
    if kv is not None:                            # what lies behind the valid keys
        for b, n in enumerate(kv):
            t[1][b, :, max(n, 0):] = fill
            t[2][b, :, max(n, 0):] = fill
    mods = dict(causal=causal, softcap=cap, alibi_slopes=_slopes(H) if alibi else None, scale=scale,
                prefix_lens=None if prefix is None else _i32(prefix), kv_lens=None if kv is None else _i32(kv))
    q, k, v, do = t
    o, lse = fa.forward(q, k, v, **mods)
    dq, dk, dv = fa.backward(q, k, v, o, lse, do, **mods)
    assert fa.check_device_status() == 0
    for b in range(B):
        _check_sequence(t, (o, lse, dq, dk, dv), slice(0, N), N, N if kv is None else max(0, min(N, kv[b])),
                        0 if prefix is None else prefix[b], causal, cap, mods["alibi_slopes"],
                        d ** -0.5 if scale is None else scale, dtype, b)
    return t, (o, lse, dq, dk, dv), mods


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp16"), (128, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", [1, 2, 127, 129, 300, 640])
@pytest.mark.parametrize("cap,alibi", [(20.0, False), (0.0, True), (50.0, True)])
def test_lengths(N, d, dtype, causal, cap, alibi):
    _batch(1, 2, 2, N, d, dtype, causal, cap, alibi, seed=N + d)


@pytest.mark.parametrize("cap,q_scale", [(0.5, 2.0), (3.0, 2.0), (1e-3, 1.0), (1e4, 2.0), (1e30, 2.0)])
def test_caps_far_below_and_above_the_scores(cap, q_scale):
    """The exponential form, its mixture with the polynomial between tiles, and caps that do nothing."""
    _batch(1, 2, 1, 400, 128, "bf16", True, cap, True, seed=3, q_scale=q_scale)
    _batch(1, 2, 1, 400, 64, "fp16", False, cap, False, seed=4, q_scale=q_scale)


@pytest.mark.parametrize("H,Hkv", [(4, 2), (6, 1), (3, 3)])
@pytest.mark.parametrize("causal", [False, True])
def test_grouped_heads_and_padding(H, Hkv, causal):
    """Padded keys hold NaN and infinities; a sequence of no keys; lengths outside [0, N]."""
    _batch(5, H, Hkv, 260, 64, "bf16", causal, 30.0, True, kv=[260, 0, 1, 129, 200], seed=5)
    _batch(2, H, Hkv, 260, 128, "fp16", causal, 30.0, False, kv=[-3, 255], seed=6, fill=float("inf"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [None, [513, 40, 513, 300, 0, 513]])
def test_prefixes(d, kv):
    _batch(6, 2, 1, 513, d, "bf16", True, 0.0, True, prefix=[0, 100, 256, 513, 20, 129], kv=kv, seed=7)
    _batch(6, 2, 1, 513, d, "fp16", True, 25.0, False, prefix=[1, 128, 385, 900, -4, 512], kv=kv, seed=8)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,spare", [([300, 0, 1, 129, 517, 128, 64], 70), ([1], 0), ([1000], 200), ([5, 3, 2], 1)])
def test_documents(lens, spare, causal, d, dtype):
    """Packed documents; what lies behind the last one is NaN and is left as it was."""
    H, Hkv, total = 4, 2, sum(lens) + spare
    t = _inputs((), H, Hkv, total, d, dtype, 9)
    for x in t:
        x[:, sum(lens):] = float("nan")
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    prefix = [(37 * (i + 1)) % (n + 5) for i, n in enumerate(lens)]
    mods = dict(causal=causal, softcap=30.0, alibi_slopes=_slopes(H), prefix_lens=_i32(prefix))
    q, k, v, do = t
    o, lse = fa.forward_varlen(q, k, v, _i32(cu), max(lens), **mods)
    dq, dk, dv = fa.backward_varlen(q, k, v, o, lse, do, _i32(cu), max(lens), **mods)
    assert fa.check_device_status() == 0
    for a, n, f in zip(cu, lens, prefix):
        if n > 0:
            _check_sequence(t, (o, lse, dq, dk, dv), slice(a, a + n), n, n, f, causal, 30.0, mods["alibi_slopes"],
                            d ** -0.5, dtype)


def test_a_document_with_nan_stays_alone():
    lens = [200, 90, 150]
    t = _inputs((), 2, 1, 440, 128, "bf16", 10)
    mods = dict(causal=True, softcap=30.0)
    cu = _i32([0, 200, 290, 440])

    def run(t):
        q, k, v, do = t
        o, lse = fa.forward_varlen(q, k, v, cu, 200, **mods)
        return (o, lse) + fa.backward_varlen(q, k, v, o, lse, do, cu, 200, **mods)
    want = run(t)
    for x in t:
        x[:, 200:290] = float("nan")
    got = run(t)
    for a, b in zip(got, want):
        assert torch.equal(a[:, :200], b[:, :200]) and torch.equal(a[:, 290:], b[:, 290:])
    assert bool(torch.isnan(got[0][:, 200:290]).all())


def test_documents_equal_separate_sequences():
    lens = [400, 129, 0, 1000, 77]
    t = _inputs((), 4, 2, sum(lens), 128, "bf16", 11)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    prefix = [30, 129, 0, 700, 1]
    mods = dict(causal=True, softcap=50.0, alibi_slopes=_slopes(4))
    q, k, v, do = t
    o, lse = fa.forward_varlen(q, k, v, _i32(cu), 1000, prefix_lens=_i32(prefix), **mods)
    got = fa.backward_varlen(q, k, v, o, lse, do, _i32(cu), 1000, prefix_lens=_i32(prefix), **mods)
    for a, n, f in zip(cu, lens, prefix):
        if n == 0:
            continue
        q1, k1, v1, do1 = (x[None, :, a:a + n].contiguous() for x in t)
        o1, l1 = fa.forward(q1, k1, v1, prefix_lens=_i32([f]), **mods)
        g1 = fa.backward(q1, k1, v1, o1, l1, do1, prefix_lens=_i32([f]), **mods)
        assert torch.equal(o[:, a:a + n], o1[0]) and torch.equal(lse[:, a:a + n], l1[0])
        for x, y in zip(got, g1):
            assert torch.equal(x[:, a:a + n], y[0])


def test_nothing_set_is_plain_attention_and_bits_repeat():
    q, k, v, do = _inputs((2,), 4, 2, 700, 128, "bf16", 12)
    o, lse = fa.forward(q, k, v, causal=True)
    mod = fa.FaScoreMod(0.0, None, None)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    st = fa.lib.fa_forward_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), lse2.data_ptr(), 2, 4, 2, 700,
                                  128, 128 ** -0.5, 1, fa.FA_BF16, None, mod, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    none = _i32([0, 0])                           # an empty prefix changes the variant, not the function
    o2, lse2 = fa.forward(q, k, v, causal=True, prefix_lens=none)
    u = 2.0 ** -8
    assert bool(((o2.double() - o.double()).abs() <= 2 * u * o.double().abs() + 2 * u).all())
    first = fa.backward(q, k, v, o, lse, do, causal=True, softcap=30.0)
    for _ in range(3):
        for a, b in zip(fa.backward(q, k, v, o, lse, do, causal=True, softcap=30.0), first):
            assert torch.equal(a, b)


def test_long_rows():
    """Every tile position of a long causal row against the formulas, forward and backward."""
    _batch(1, 1, 1, 4100, 128, "bf16", True, 50.0, True, prefix=[900], seed=13)


def test_captured_step_on_a_side_stream():
    q, k, v, do = _inputs((1,), 2, 2, 300, 64, "bf16", 14)
    prefix = _i32([10])
    mods = dict(causal=True, softcap=30.0, prefix_lens=prefix)

    def step():
        o, lse = fa.forward(q, k, v, **mods)
        return (o, lse) + fa.backward(q, k, v, o, lse, do, **mods)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in (10, 200):
        prefix.fill_(n)
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    want = fa.forward(q, k, v, **mods)
    torch.cuda.synchronize()
    got = fa.forward(q, k, v, stream=side, **mods)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    q, k, v, do = _inputs((1,), 4, 2, 130, 64, "bf16", 15)
    mask = torch.ones((2, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="no block mask"):
        fa.forward(q, k, v, softcap=10.0, block_mask=mask)
    with pytest.raises(ValueError, match="no block mask"):
        fa.forward(q, k, v, softcap=10.0, dropout_p=0.1)
    o, lse = fa.forward(q, k, v, softcap=10.0)
    with pytest.raises(ValueError, match="fused"):
        fa.backward(q, k, v, o, lse, do, softcap=10.0, fused=True)
    wide = torch.empty((*lse.shape[:2], 2 * lse.shape[2]), device="cuda")
    with pytest.raises(ValueError, match="lse"):
        fa.backward(q, k, v, o, wide[:, :, ::2], do, softcap=10.0)
    with pytest.raises(ValueError, match="lse"):
        fa.forward(q, k, v, softcap=10.0, lse=wide[:, :, ::2])
    with pytest.raises(ValueError, match="o must be"):
        fa.forward(q, k, v, softcap=10.0, o=o[:, :2])
    for name in ("dq", "dk", "dv"):
        with pytest.raises(ValueError, match=name):
            fa.backward(q, k, v, o, lse, do, softcap=10.0, **{name: torch.empty_like(q).float()})
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.backward(q, k, v, o, lse, do, softcap=10.0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="alibi_slopes"):
        fa.forward(q, k, v, alibi_slopes=_slopes(2))
    with pytest.raises(ValueError, match="alibi_slopes"):
        fa.forward(q, k, v, alibi_slopes=_slopes(4).double())
    with pytest.raises(ValueError, match="prefix_lens"):
        fa.forward(q, k, v, causal=True, prefix_lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="prefix_lens"):
        fa.forward(q, k, v, causal=True, prefix_lens=_i32([1, 2]))
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(fa.FaError, match="INVALID_ARG"):
            fa.forward(q, k, v, softcap=bad)
        with pytest.raises(fa.FaError, match="INVALID_ARG"):
            fa.backward(q, k, v, o, lse, do, softcap=bad)
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.forward(q, k, v, softcap=1e-42)
    f = [x.float() for x in (q, q[:, :4], q[:, :4])]
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.forward(*f, softcap=10.0)
