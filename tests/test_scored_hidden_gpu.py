"""Scores that a mask hides do not enter a result, not even through the form of the tanh, which a warp
chooses for the scores that one of its rows sees: the same bits whatever the hidden ones would be."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_scored_gpu import _i32, _inputs

pytestmark = pytest.mark.gpu


def _step(t, **mods):
    q, k, v, do = t
    o, lse = fa.forward(q, k, v, softcap=30.0, **mods)
    return (o, lse) + fa.backward(q, k, v, o, lse, do, softcap=30.0, **mods)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("alibi", [False, True])
def test_padded_keys(d, dtype, causal, alibi):
    """Keys behind a sequence's valid ones."""
    kv = [40, 200, 129, 1]
    t = _inputs((4,), 2, 1, 260, d, dtype, 1)
    mods = dict(causal=causal, kv_lens=_i32(kv),
                alibi_slopes=torch.tensor([0.1, 0.01], device="cuda") if alibi else None)
    want = None
    for fill in (0.0, 3000.0, float("inf"), float("nan")):
        for b, n in enumerate(kv):
            t[1][b, :, n:] = fill
            t[2][b, :, n:] = fill
        got = _step(t, **mods)
        want = got if want is None else want
        for name, a, b in zip(("O", "LSE", "dQ", "dK", "dV"), got, want):
            assert torch.equal(a, b), (name, fill)
    assert fa.check_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_later_keys(dtype):
    """Keys that all of a warp's 32 queries come before."""
    t = _inputs((1,), 2, 1, 256, 128, dtype, 2)
    want = _step(t, causal=True)
    t[1][:, :, 32:] *= 60.0
    got = _step(t, causal=True)
    for name, a, b in zip(("O", "LSE", "dQ"), got, want):
        assert torch.equal(a[:, :, :32], b[:, :, :32]), name


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_earlier_queries(dtype):
    """Queries that all of a warp's 32 keys come after."""
    t = _inputs((1,), 2, 1, 256, 128, dtype, 3)
    want = _step(t, causal=True)
    t[0][:, :, :32] *= 60.0
    got = _step(t, causal=True)
    for name, a, b in zip(("dK", "dV"), got[3:], want[3:]):
        assert torch.equal(a[:, :, 32:64], b[:, :, 32:64]), name
