"""Rotary positions on the GPU: fa_rotary, its gradient, and the frequencies for stretched contexts,
against complex rotation in 64 bits.

The bound: the angle is off by at most pi 2^-24 (its conversion to fp32) + 2^-29, the sine and cosine
by an ulp more (2^-23), their product with mscale and the two products and sum by half an ulp each,
4 2^-24 in all; together below 6e-7 of mscale (|a| + |b|).  Then one rounding to the output's type."""
import math

import pytest
import torch

import exact_io_aware_23_gb300 as fa

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _turn(x, pos, inv_freq, interleaved, mscale, sign=1):
    """x [B, H, N, d] turned in 64 bits, and |a| + |b| of each value's pair."""
    half = inv_freq.numel()
    r = x[..., : 2 * half].double()
    pairs = r.unflatten(-1, (half, 2)) if interleaved else r.unflatten(-1, (2, half)).transpose(-1, -2)
    w = sign * pos.double()[..., None] * inv_freq
    w = w[:, None] if w.dim() == 3 else w
    a, b = pairs[..., 0], pairs[..., 1]
    y = torch.stack((a * w.cos() - b * w.sin(), a * w.sin() + b * w.cos()), -1) * mscale
    size = pairs.abs().sum(-1, keepdim=True).expand_as(pairs)
    back = (lambda t: t.flatten(-2)) if interleaved else (lambda t: t.transpose(-1, -2).flatten(-2))
    rest = x[..., 2 * half:].double()
    return torch.cat((back(y), rest), -1), torch.cat((back(size) * abs(mscale), torch.zeros_like(rest)), -1)


def _check(got, x, pos, inv_freq, interleaved, mscale, sign=1):
    ref, size = _turn(x, pos, inv_freq, interleaved, mscale, sign)
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + 6e-7 * size
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25                       # half a step of the subnormal numbers
    assert bool(((got.double() - ref).abs() <= tol).all())
    rest = 2 * inv_freq.numel()
    assert torch.equal(got[..., rest:], x[..., rest:])


def _x(B, H, N, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((B, H, N, d), generator=g, device="cuda").to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,d,rot", [(1, 1, 1, 64, 64), (2, 3, 77, 64, 16), (3, 5, 33, 128, 96),
                                         (2, 40, 300, 128, 128), (1, 2, 5000, 128, 48)])
def test_forward_and_gradient(dtype, interleaved, B, H, N, d, rot):
    inv_freq, _ = fa.rotary_frequencies(rot)
    x = _x(B, H, N, d, dtype, seed=N + rot)
    pos = torch.randint(0, 1 << 20, (B, N), dtype=torch.int32, device="cuda")
    y = fa.rotary(x, pos, inv_freq, interleaved=interleaved, mscale=1.25)
    _check(y, x, pos, inv_freq, interleaved, 1.25)
    dx = fa.rotary_backward(x, pos, inv_freq, interleaved=interleaved, mscale=1.25)
    _check(dx, x, pos, inv_freq, interleaved, 1.25, sign=-1)
    assert fa.check_device_status() == 0


def test_gradient_against_differences():
    """The map is linear: <rotary(x), dy> = <x, rotary_backward(dy)>, and a difference of any size
    is the map of the difference."""
    inv_freq, _ = fa.rotary_frequencies(64)
    x, e, dy = (_x(2, 3, 50, 128, "fp32", seed=s) for s in (1, 2, 3))
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 977
    f = lambda t: fa.rotary(t, pos, inv_freq, mscale=0.9).double()                # noqa: E731
    dx = fa.rotary_backward(dy, pos, inv_freq, mscale=0.9).double()
    slope = ((f(x + e) - f(x)) * dy.double()).sum()
    size = float(e.abs().double().sum() * 2) + float(x.abs().double().sum()) * 4
    assert abs(float(slope - ((x + e).double() - x.double()).mul(dx).sum())) <= 2e-6 * size * float(dy.abs().max())


@pytest.mark.parametrize("pos", [0, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7])
def test_far_positions(pos):
    inv_freq = torch.tensor([1.0, 0.7, 1e-4, 3e-9, 0.0, -0.3, 2.0 ** -60, 5.0], dtype=torch.float64, device="cuda")
    x = _x(1, 2, 3, 64, "fp32")
    p = torch.full((3,), pos, dtype=torch.int32, device="cuda")
    # the reference's own product of position and frequency is off by 2^-53 of up to 2^33.4
    _check(fa.rotary(x, p, inv_freq), x, p, inv_freq, False, 1.0)


def test_strides_and_in_place():
    inv_freq, _ = fa.rotary_frequencies(64)
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    qkv = _x(2, 70, 3 * 5, 64, "bf16").reshape(2, 70, 15, 64)
    for part in range(3):
        x = qkv[:, :, part * 5:(part + 1) * 5].transpose(1, 2)
        y = fa.rotary(x, pos, inv_freq)
        assert y.is_contiguous()
        assert torch.equal(y, fa.rotary(x.contiguous(), pos, inv_freq))
    before = qkv.clone()
    x = qkv[:, :, 5:10].transpose(1, 2)
    y = fa.rotary(x, pos, inv_freq)
    assert fa.rotary(x, pos, inv_freq, out=x) is x
    assert torch.equal(x, y)
    assert torch.equal(qkv[:, :, :5], before[:, :, :5]) and torch.equal(qkv[:, :, 10:], before[:, :, 10:])
    wide = _x(1, 1, 70, 64, "bf16").expand(2, 4, 70, 64)                # one head seen as many
    assert torch.equal(fa.rotary(wide, pos, inv_freq), fa.rotary(wide.contiguous(), pos, inv_freq))
    packed = _x(1, 4, 70, 128, "fp16")[0]
    assert torch.equal(fa.rotary(packed, pos, inv_freq), fa.rotary(packed[None], pos, inv_freq)[0])


def test_many_tokens_past_32_bit_offsets():
    """2^31 values and more: offsets pass 32 bits."""
    N = (1 << 24) + 5
    inv_freq, _ = fa.rotary_frequencies(128)
    x = torch.randn((1, 1, N, 128), device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    y = fa.rotary(x, pos, inv_freq)
    for at in (slice(0, 3), slice(N // 2, N // 2 + 3), slice(N - 3, N)):
        _check(y[:, :, at], x[:, :, at], pos[at], inv_freq, False, 1.0)


def test_empty_and_copy():
    inv_freq, _ = fa.rotary_frequencies(64)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert fa.rotary(_x(2, 3, 0, 64, "bf16"), pos, inv_freq).shape == (2, 3, 0, 64)
    x = _x(2, 3, 9, 64, "bf16")
    none = torch.zeros(0, dtype=torch.float64, device="cuda")
    assert torch.equal(fa.rotary(x, torch.arange(9, dtype=torch.int32, device="cuda"), none), x)


def test_memory_the_current_stream_still_reads():
    """The output of a call on another stream may lie in memory that was given back on the current
    one, whose kernels still read it."""
    inv_freq, _ = fa.rotary_frequencies(128)
    x = _x(1, 8, 4096, 128, "bf16")
    pos = torch.arange(4096, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    old = x.clone()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        busy = (busy @ busy).clamp_(-1.0, 1.0)          # some milliseconds
    kept = old.clone()
    del old
    y = fa.rotary(x, pos, inv_freq, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, x)
    assert torch.equal(y, fa.rotary(x, pos, inv_freq))


def test_captured_and_on_another_stream():
    inv_freq, _ = fa.rotary_frequencies(128)
    x = _x(1, 8, 256, 128, "bf16")
    pos = torch.arange(256, dtype=torch.int32, device="cuda")
    want = fa.rotary(x, pos, inv_freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = fa.rotary(x, pos, inv_freq, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.rotary(x, pos, inv_freq, out=out)
    pos += 3
    g.replay()
    assert torch.equal(out, fa.rotary(x, pos, inv_freq))


def test_refusals():
    inv_freq, _ = fa.rotary_frequencies(64)
    x = _x(1, 2, 8, 64, "bf16")
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="positions"):
        fa.rotary(x, pos.long(), inv_freq)
    with pytest.raises(ValueError, match="positions"):
        fa.rotary(x, pos[:7], inv_freq)
    with pytest.raises(ValueError, match="float64"):
        fa.rotary(x, pos, inv_freq.float())
    with pytest.raises(ValueError, match="adjoin"):
        fa.rotary(x.transpose(-1, -2).contiguous().transpose(-1, -2), pos, inv_freq)
    with pytest.raises(ValueError, match="overlap"):
        buf = _x(1, 2, 9, 64, "bf16")
        fa.rotary(buf[:, :, :8], pos, inv_freq, out=buf[:, :, 1:])
    for shared in (x[:, :1].clone().expand(1, 2, 8, 64), torch.zeros_like(x).as_strided((1, 2, 8, 64), (1024, 512, 32, 1))):
        with pytest.raises(fa.FaError, match="INVALID_ARG"):          # written elements that share memory
            fa.rotary(x, pos, inv_freq, out=shared)
    with pytest.raises(ValueError, match="dtype"):
        fa.rotary(x.double(), pos, inv_freq)
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.rotary(x, pos, inv_freq[:12])                              # 24 values: not a multiple of 16
    with pytest.raises(fa.FaError, match="UNSUPPORTED"):
        fa.rotary(x[..., :32].contiguous(), pos, inv_freq[:8])         # d = 32
    with pytest.raises(fa.FaError, match="INVALID_ARG"):
        fa.rotary(_x(1, 2, 8, 72, "bf16")[..., 4:68], pos, inv_freq)   # rows off the 16-byte grid


def test_frequencies():
    plain, m = fa.rotary_frequencies(128, 10000.0, device="cpu")
    assert m == 1.0 and plain.dtype == torch.float64
    assert torch.allclose(plain, 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128), rtol=1e-15)
    linear, _ = fa.rotary_frequencies(128, factor=4.0, device="cpu")
    assert torch.allclose(linear, plain / 4, rtol=1e-15)
    ntk, _ = fa.rotary_frequencies(128, factor=4.0, method="ntk", device="cpu")
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / (plain[-1] / 4)) - 1) < 1e-12
    ramp, m = fa.rotary_frequencies(128, factor=4.0, method="ramp", trained_len=4096, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(ramp[turns > 32], plain[turns > 32])
    assert torch.allclose(ramp[turns < 1], plain[turns < 1] / 4, rtol=1e-15)
    assert bool((ramp <= plain).all()) and bool((ramp >= plain / 4 * (1 - 1e-15)).all())
    assert abs(m - (0.1 * math.log(4.0) + 1)) < 1e-15
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, factor=0.5),
                dict(rotary_dim=64, base=0.0), dict(rotary_dim=64, method="?"), dict(rotary_dim=64, method="ramp")):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(**bad)
