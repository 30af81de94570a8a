"""Distance biases on the GPU whose slopes are negative or of both signs, against 64-bit formulas.  The
bounds of scored_reference.py take a slope by its size: `_signed_scores` gives a negative one that
error too."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
import scored_reference
from scored_reference import V
from test_paged_gpu import _cache, _check as check_paged
from test_scored_gpu import _check_sequence, _i32, _inputs

pytestmark = pytest.mark.gpu
_scores = scored_reference.scores


def _signed_scores(q, k, allowed, dist, scale, cap, slope, *rest):
    """Scores with their error bound, whose term of the bias is 4 v |slope| |i - j|."""
    s, c, e = _scores(q, k, allowed, dist, scale, cap, slope, *rest)
    if slope < 0.0:
        e = e + torch.where(allowed, 8 * V * -slope * dist, 0.0)
    return s, c, e


@pytest.fixture(autouse=True)
def _bounds(monkeypatch):
    monkeypatch.setattr(scored_reference, "scores", _signed_scores)


def _slopes(values):
    return torch.tensor(values, dtype=torch.float32, device="cuda")


def _batch(B, N, d, dtype, causal, cap, slopes, prefix=None, kv=None, seed=0, Hkv=2):
    t = _inputs((B,), len(slopes), Hkv, N, d, dtype, seed)
    mods = dict(causal=causal, softcap=cap, alibi_slopes=_slopes(slopes),
                prefix_lens=None if prefix is None else _i32(prefix), kv_lens=None if kv is None else _i32(kv))
    q, k, v, do = t
    o, lse = fa.forward(q, k, v, **mods)
    out = (o, lse) + fa.backward(q, k, v, o, lse, do, **mods)
    assert fa.check_device_status() == 0
    for b in range(B):
        _check_sequence(t, out, slice(0, N), N, N if kv is None else kv[b], 0 if prefix is None else prefix[b], causal,
                        cap, mods["alibi_slopes"], d ** -0.5, dtype, b)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("N,causal,prefix", [(1, False, None), (200, False, None), (517, False, None), (300, True, None),
                                             (400, True, [290, 17])])
def test_signs(N, causal, prefix, cap, d, dtype):
    """Tiles on either side of the diagonal and across it, within one row of scores."""
    _batch(2, N, d, dtype, causal, cap, [-0.5, 0.25, 0.0, -0.01], prefix=prefix, seed=N + d)


def test_signs_where_two_blocks_share_an_sm():
    """d = 64 with more pairs of tiles than SMs runs the forward with 64-key tiles."""
    _batch(20, 300, 64, "bf16", False, 0.0, [-0.5, 0.25, -0.02, 0.1], kv=[300 - 13 * i for i in range(20)], seed=1)
    _batch(20, 300, 64, "bf16", True, 20.0, [-0.5, 0.25, -0.02, 0.1], prefix=[15 * i for i in range(20)], seed=2)


@pytest.mark.parametrize("causal", [False, True])
def test_signs_in_documents(causal):
    lens, H = [300, 0, 1, 129, 70], 4
    t = _inputs((), H, 2, sum(lens), 128, "bf16", 3)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    prefix = [200, 0, 1, 129, 3]
    mods = dict(causal=causal, softcap=30.0, alibi_slopes=_slopes([-0.5, 0.25, -0.02, 0.1]), prefix_lens=_i32(prefix))
    q, k, v, do = t
    o, lse = fa.forward_varlen(q, k, v, _i32(cu), max(lens), **mods)
    out = (o, lse) + fa.backward_varlen(q, k, v, o, lse, do, _i32(cu), max(lens), **mods)
    assert fa.check_device_status() == 0
    for a, n, f in zip(cu, lens, prefix):
        if n > 0:
            _check_sequence(t, out, slice(a, a + n), n, n, f, causal, 30.0, mods["alibi_slopes"], 128 ** -0.5, "bf16")


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T", [1, 5])
def test_signs_over_a_paged_cache(T, cap):
    lens = [5, 250, 0, 3000]
    kc, vc, table, g = _cache(lens, 2, 32, 64, "bf16", T, fill=float("nan"))
    q = (torch.randn((4, 4, T, 64), generator=g, device="cuda") * 2).to(torch.bfloat16)
    slopes = _slopes([-0.5, 0.25, -0.02, 0.1])
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), softcap=cap, alibi_slopes=slopes)
    assert fa.check_device_status() == 0
    check_paged(q, kc, vc, table, lens, o, lse, cap, slopes)
