"""8-bit pages, key bounds, the choice of pages and their assignment in plain Python and 64 bits, and bounds
on what a kernel's attention over 8-bit pages may differ by.

The bounds for one row, next to those of scored_reference.py (v = 2^-24), with k = ks c and v = vs e the
values that codes and scales stand for:

  e_ij  : three more roundings of the score's products with scales (3 v |x|, 4 taken), and of a bf16 query's
          values below 2^-28 of the row's largest, which lose up to 2^-39 of that: scale 2^-39 max |q| sum |k|
  O     : p vs / u is rounded to fp16, off by half a step, 2^-11 of it, or 2^-25 (below fp16's normal
          range) in units of u, at most the largest vs that the row's pages have; its own two roundings
          in fp32 are within f's slack.  u_out |O| + (2^-11 + f) sum p |v| + 2^-25 max vs sum |e|, and
          half a step of fp16's subnormal outputs
"""
import math

import torch

from scored_reference import V, scores, softmax

LARGEST = {"int8": 127.0, "e4m3": 448.0}
STORES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def power(amax, largest):
    """The smallest power of two, at least 2^-100, that `largest` of reaches amax."""
    if not amax > 0.0:
        return 2.0 ** -100
    e = math.frexp(amax / largest)[1] - 2                   # amax / largest is in [2^(e + 1), 2^(e + 2)), about
    while largest * 2.0 ** e < amax:
        e += 1
    return 2.0 ** max(e, -100)


def grid(y, store):
    """The nearest values that the store holds (64 bits), ties to the even one."""
    if store == "int8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def head_forward8(q, c, e, ks, vs, allowed, dist, scale, cap, slope, dtype):
    """O, LSE of one head over keys ks c and values vs e (64-bit inputs; ks, vs a column), and their bounds."""
    k, v = ks * c, vs * e
    s, _, err = scores(q, k, allowed, dist, scale, cap, slope)
    x = (q @ k.T * scale).abs()
    top = q.abs().amax(-1, keepdim=True)
    err = err + (4 * V * x + scale * 2.0 ** -39 * top * k.abs().sum(-1)[None, :]).masked_fill(~allowed, 0.0)
    p, lse = softmax(s)
    f = 2 * (err.amax(-1, keepdim=True) + 2.0 ** -22) if s.shape[-1] else torch.zeros_like(lse)[:, None]
    o = p @ v
    u = torch.finfo(dtype).eps / 2
    unit = float(vs.max()) if vs.numel() else 0.0
    tol = u * o.abs() + (2.0 ** -11 + f) * (p @ v.abs()) + 2.0 ** -25 * unit * (allowed.double() @ e.abs())
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return o, lse, tol, f[:, 0] / 2 + 4 * V * (1 + lse.abs().nan_to_num(posinf=0.0))


def choose(best, n, n_select, first, last):
    """The pages chosen of n by their scores: a list."""
    forced = [p < first or p >= n - last for p in range(n)]
    order = sorted(range(n), key=lambda p: (not forced[p], 0.0 if forced[p] else -best[p], p))
    return sorted(order[:n_select])


def page_scores(q, lo, hi, unit):
    """Scores of pages (lo, hi [pages, d], unit [pages]) for the rows q [rows, d]."""
    best = None
    for row in q.double().cpu():
        two = power(float(row.abs().max()), 127.0)
        c = torch.round(row / two)
        s = torch.maximum(c * lo, c * hi).sum(-1) * two * unit
        best = s if best is None else torch.maximum(best, s)
    return best.tolist()


def assign(table, old, new, ring, state, page, T):
    """assign_pages on lists, in place for the table and the ring."""
    first, count = state
    n, taken, given = len(ring), 0, 0
    pages = lambda x: -(-x // page)  # noqa: E731
    for b, (x, y) in enumerate(zip(old, new)):
        for j in range(pages(x), pages(y)):
            table[b][j] = ring[(first + taken) % n]
            taken += 1
    for b, (x, y) in enumerate(zip(old, new)):
        for j in range(pages(y), pages(x)):
            ring[(first + count + given) % n] = table[b][j]
            given += 1
    slots, positions = ([[-1] * T for _ in old] for _ in range(2))
    for b, (x, y) in enumerate(zip(old, new)):
        for t in range(max(0, min(T, y - x))):
            positions[b][t] = x + t
            slots[b][t] = table[b][(x + t) // page] * page + (x + t) % page
    return slots, positions, [(first + taken) % n, count - taken + given]
