"""Attention with capped and biased scores in 64 bits, head by head, and bounds on what a kernel may
differ by that takes 16-bit operands, adds in 32 bits and rounds its probabilities (and dS) and its
outputs once to the operands' type.

A rounding to type t is off by at most half a step, u = finfo(t).eps / 2 relative to the value; one
fp32 operation by v = 2^-24.  The bounds, for one row i with probabilities p, and e_ij the largest
error of a score:

  e_ij  : d products added in fp32, in any order, (d + 4) v scale sum_c |q_c k_c|.  The cap by its
          polynomial, where no score of the head exceeds 0.4 of the cap, is off by 6 2^-24 of itself
          (its own 9.9e-8, Horner's steps, the scaled coefficients, the product with cap): 2^-21 |s|;
          by the exponential, errors of 2^-22 in 1 / (1 + exp 2x) times 2 cap: 2^-20 cap in all.
          The bf16 backward's polynomial is off by 6.3e-6 of the score itself: 2^-17 |s| in all.  The
          bias 4 v slope |i - j| more, 4 v |s_ij| for the conversion to base 2.
  p     : relative error 2 (max_j e_ij + 2^-22) =: f_i  (numerator and normaliser)
  O     : u |O| + (u + f_i) sum_j p_j |v_j|
  LSE   : max_j e_ij + 2^-22 + 4 v (1 + |LSE|)
  dV    : u |dV| + sum_i (u + f_i) p_ij |dO_i|
  dS_ij : = p (dP - D) c, c = the cap's derivative.  dP adds d products: (d + 2) v sum |dO_c V_c|;
          D = sum_j p dP takes that error and f_i of each term, and one v for each of its fp32
          additions in turn; c = 1 - tanh^2 is off by
          twice the tanh's error, absolutely, and by 2 c e_ij / cap through its argument;
          then one rounding u:
          (u + f_i + 2 e_ij / cap) |dS| + p |dP - D| 2^-20 + p c (the errors of dP and D)
  dQ,dK : u |.| + scale sum of the above times |K| or |Q|; products added in fp32 stay below
          f's slack.

fp16 has no relative precision below 2^-14: half a step there is 2^-25 whatever the value, so a
rounding of x to fp16 is off by max(u |x|, 2^-25) <= u |x| + tiny.  That holds for each rounded
probability (the kernels' are relative to a maximum no larger than the row's, so their sum is at
least 1 and the normalised error no larger), each dS and each output:
  O     : + tiny (1 + sum over the row's keys of |v_j|)
  dV    : + tiny (1 + sum |dO_i|);  dQ : + tiny (1 + scale sum |K_j|);  dK : + tiny (1 + scale sum |Q_i|)
Each is asserted element by element.
"""
import math

import torch

V = 2.0 ** -24


def scores(q, k, allowed, dist, scale, cap, slope, poly=2.0 ** -21):
    """(s, c, e): masked scores, the cap's derivative, the error bound of s."""
    x = q @ k.T * scale
    e = (q.shape[-1] + 4) * V * scale * (q.abs() @ k.abs().T)
    c = torch.ones_like(x)
    if cap > 0.0:
        t = torch.tanh(x / cap)
        fits = x.numel() == 0 or float(x.abs().max()) <= 0.4 * cap
        x, c = cap * t, 1.0 - t * t
        e = e + poly * x.abs() + (0.0 if fits else 2.0 ** -20 * cap)
    if slope != 0.0:
        x = x - slope * dist
        e = e + 4 * V * slope * dist
    e = e + 4 * V * x.abs()
    return x.masked_fill(~allowed, -math.inf), c, e.masked_fill(~allowed, 0.0)


def softmax(s):
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p, lse


def head_forward(q, k, v, allowed, dist, scale, cap, slope, u, tiny=0.0):
    """O, LSE of one head and the bounds of both (64-bit inputs)."""
    s, _, e = scores(q, k, allowed, dist, scale, cap, slope)
    p, lse = softmax(s)
    f = 2 * (e.amax(-1, keepdim=True) + 2.0 ** -22) if s.shape[-1] else torch.zeros_like(lse)[:, None]
    o = p @ v
    o_tol = u * o.abs() + (u + f) * (p @ v.abs()) + tiny * (1 + allowed.double() @ v.abs())
    lse_tol = f[:, 0] / 2 + 4 * V * (1 + lse.abs().nan_to_num(posinf=0.0))
    return o, lse, o_tol, lse_tol


def head_backward(q, k, v, do, allowed, dist, scale, cap, slope, u, tiny=0.0):
    """dQ, dK, dV of one head and their bounds."""
    # bf16 (u = 2^-8) or finer; the derivative 1 - tanh^2 takes twice the tanh's error
    poly = 2.0 ** -17 if u > 2.0 ** -10 else 2.0 ** -21
    s, c, e = scores(q, k, allowed, dist, scale, cap, slope, poly)
    p, _ = softmax(s)
    f = 2 * (e.amax(-1, keepdim=True) + 2.0 ** -22)
    d = q.shape[-1]
    dp = do @ v.T
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - delta) * c
    dp_err = (d + 2) * V * (do.abs() @ v.abs().T)
    # each of the 128-key tiles adds to two pairs of sums 32 times in turn
    dp_err = dp_err + (p * ((f + 34 * V * max(1, s.shape[-1] // 128)) * dp.abs() + dp_err)).sum(-1, keepdim=True)
    ds_tol = (u + f + (2 * e / cap if cap > 0.0 else 0.0)) * ds.abs() + p * c * dp_err
    if cap > 0.0:
        ds_tol = ds_tol + p * (dp - delta).abs() * 2 * max(poly, 2.0 ** -21)
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    a = allowed.double()
    return (dq, dk, dv, u * dq.abs() + scale * ds_tol @ k.abs() + tiny * (1 + scale * a @ k.abs()),
            u * dk.abs() + scale * ds_tol.T @ q.abs() + tiny * (1 + scale * a.T @ q.abs()),
            u * dv.abs() + ((u + f) * p).T @ do.abs() + tiny * (1 + a.T @ do.abs()))


def assert_within(name, got, ref, tol):
    got = got.double()
    assert torch.equal(torch.isinf(got), torch.isinf(ref)), f"{name}: infinities differ"
    fine = ~torch.isinf(ref)
    assert bool(torch.isfinite(got[fine]).all()), f"{name}: not finite"
    over = ((got - ref).abs() - tol)[fine]
    # gradients that vanish in exact arithmetic keep the rounding of their terms: the bound has it
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1e-30, (name, worst, float((got - ref).abs()[fine].max()))
