"""Scored calls on another stream with key lengths that have to be copied first (strided, or on the
host): the stream waits for the copy, and its memory is not given away while the kernels read it."""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from test_scored_gpu import _i32, _inputs

pytestmark = pytest.mark.gpu
MODS = dict(causal=True, softcap=30.0)


@pytest.mark.parametrize("where", ["strided", "host"])
@pytest.mark.parametrize("given", [False, True])
def test_copied_lengths(where, given):
    B, H, N, d = 16, 4, 2048, 128
    q, k, v, do = _inputs((B,), H, 2, N, d, "bf16", 1)
    lens = [N - 97 * i for i in range(B)]
    o0, lse0 = fa.forward(q, k, v, kv_lens=_i32(lens), **MODS)
    want = (o0, lse0) + fa.backward(q, k, v, o0, lse0, do, kv_lens=_i32(lens), **MODS)
    fwd = dict(o=torch.empty_like(q), lse=torch.empty_like(lse0)) if given else {}
    bwd = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               workspace=torch.empty(fa.backward_workspace_size(B, H, N, d), dtype=torch.uint8, device="cuda")) if given else {}
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    wide = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        wide.zero_()
        for _ in range(5):
            busy = (busy @ busy).clamp_(-1.0, 1.0)       # the current stream is busy for some milliseconds
        wide[:, 0] = torch.tensor(lens, dtype=torch.int32).cuda(non_blocking=True)
        kv = wide[:, 0] if where == "strided" else torch.tensor(lens, dtype=torch.int32)
        o, lse = fa.forward(q, k, v, kv_lens=kv, stream=side, **fwd, **MODS)
        taken = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(4)]     # memory given back, if any
        grads = fa.backward(q, k, v, o, lse, do, kv_lens=kv, stream=side, **bwd, **MODS)
        taken += [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for name, a, b in zip(("O", "LSE", "dQ", "dK", "dV"), (o, lse) + grads, want):
            assert torch.equal(a, b), name
        del taken
