"""The backward at d = 64, whose warps may be a tile apart: some take the tanh's polynomial, some its
exponential form, some see nothing of a tile.  Wherever they stand, gradients are the formulas' and
have the same bits on every call."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_scored_gpu import _check_sequence, _i32, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,G", [([0, 19, 211, 1], 4), ([400, 33, 130], 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_documents(lens, G, dtype):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    mods = dict(causal=True, softcap=5.0, scale=0.3)
    for seed in range(100):
        t = _inputs((), G, 1, sum(lens), 64, dtype, seed)
        q, k, v, do = t
        o, lse = fa.forward_varlen(q, k, v, _i32(cu), max(lens), **mods)
        runs = [fa.backward_varlen(q, k, v, o, lse, do, _i32(cu), max(lens), **mods) for _ in range(5)]
        for other in runs[1:]:
            for name, a, b in zip(("dQ", "dK", "dV"), runs[0], other):
                assert torch.equal(a, b), (name, seed)
        if seed < 5:
            for a, n in zip(cu, lens):
                if n > 0:
                    _check_sequence(t, (o, lse) + runs[0], slice(a, a + n), n, n, 0, True, 5.0, None, 0.3, dtype)
    assert fa.check_device_status() == 0


@pytest.mark.parametrize("mods", [dict(), dict(softcap=5.0), dict(dropout_p=0.2, seed=3)])
def test_batches(mods):
    """Plain scores, capped ones and dropout, batched."""
    q, k, v, do = _inputs((6,), 4, 2, 500, 64, "bf16", 1)
    o, lse = fa.forward(q, k, v, causal=True, **mods)
    want = fa.backward(q, k, v, o, lse, do, causal=True, **mods)
    for _ in range(100):
        for name, a, b in zip(("dQ", "dK", "dV"), fa.backward(q, k, v, o, lse, do, causal=True, **mods), want):
            assert torch.equal(a, b), name
