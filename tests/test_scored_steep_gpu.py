"""Distance biases on the GPU so steep that each query keeps its own key alone.

Slopes in the thousands leave each query its own key: neighbours weigh exp(-1000) at most, the
scores themselves staying below 40.  So P is 1 there and 0 elsewhere, O_i = v_i, dV_i sums the
group's dO_i, and LSE_i = s_ii, which the bias, 0 at the key itself, leaves as it is.  A score is
off by (d + 4) v scale sum_c |q_c k_c| + 4 v |s| whatever the slope, and LSE by 4 v (1 + |LSE|) more;
P, rebuilt from it, by those errors relative, and by its rounding u to the operands' type.
"""
import pytest
import torch

import exact_io_aware_23_gb300 as fa
from scored_reference import V, assert_within
from test_paged_gpu import _cache
from test_scored_gpu import _i32, _inputs

pytestmark = pytest.mark.gpu
SLOPES = [1000.0, 20000.0, 3000.0, 1e5]


def _score_error(q, k, scale):
    return (q.shape[-1] + 4) * V * scale * (q.abs() * k.abs()).sum(-1) + 4 * V * (q * k).sum(-1).abs() * scale


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,N", [(1, 1), (1, 300), (20, 290)])
def test_steep_slopes(B, N, causal, d, dtype):
    H, Hkv = 4, 2
    q, k, v, do = _inputs((B,), H, Hkv, N, d, dtype, N)
    mods = dict(causal=causal, alibi_slopes=torch.tensor(SLOPES, device="cuda"))
    o, lse = fa.forward(q, k, v, **mods)
    dv = fa.backward(q, k, v, o, lse, do, **mods)[2]
    assert fa.check_device_status() == 0
    u, tiny = torch.finfo(q.dtype).eps / 2, 2.0 ** -25 if dtype == "fp16" else 0.0
    qd, dod = q.double(), do.double()
    kd, vd = (t.double().repeat_interleave(H // Hkv, 1) for t in (k, v))
    assert_within("O", o, vd, 2 * u * vd.abs() + tiny)
    want = (qd * kd).sum(-1) * d ** -0.5
    err = _score_error(qd, kd, d ** -0.5) + 4 * V * (1 + want.abs())
    assert_within("LSE", lse, want, err)
    off = (2 * err + 4 * V)[..., None] + u                  # of P: by its score and by LSE; its rounding
    group = lambda t: t.reshape(B, Hkv, H // Hkv, N, -1).sum(2)     # noqa: E731
    assert_within("dV", dv, group(dod), u * group(dod).abs() + group(off * dod.abs()) + tiny)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_steep_slopes_over_a_paged_cache(d, dtype):
    lens, T = [3, 40, 700, 5000], 3
    kc, vc, table, g = _cache(lens, 2, 16, d, dtype, 4, fill=float("nan"))
    q = (torch.randn((4, 4, T, d), generator=g, device="cuda") * 2).to(kc.dtype)
    o, lse = fa.forward_paged(q, kc, vc, table, _i32(lens), alibi_slopes=torch.tensor(SLOPES, device="cuda"))
    assert fa.check_device_status() == 0
    u, tiny = torch.finfo(q.dtype).eps / 2, 2.0 ** -25 if dtype == "fp16" else 0.0
    for b, n in enumerate(lens):
        at = torch.arange(n - T, n, device="cuda")
        page = table[b].long()[at // 16]
        kd, vd = (c[page, :, at % 16].transpose(0, 1).double().repeat_interleave(2, 0) for c in (kc, vc))
        qd = q[b].double()
        assert_within("O", o[b], vd, 2 * u * vd.abs() + tiny)
        want = (qd * kd).sum(-1) * d ** -0.5
        assert_within("LSE", lse[b], want, _score_error(qd, kd, d ** -0.5) + 4 * V * (1 + want.abs()))
