"""The 64-bit formulas that the scored kernels are held to: their gradients against differences of
their forward, and the tanh polynomial's error (CPU only)."""
import math
import os
import re

import pytest
import torch

from scored_reference import head_backward, head_forward

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cap,slope,causal", [(1.5, 0.0, True), (0.0, 0.3, False), (4.0, 0.1, True)])
def test_gradients_against_differences(cap, slope, causal):
    g = torch.Generator().manual_seed(1)
    n, d = 7, 5
    q, k, v, do = (torch.randn((n, d), generator=g, dtype=torch.float64) for _ in range(4))
    i = torch.arange(n)
    allowed = (i[None, :] <= i[:, None]) if causal else torch.ones((n, n), dtype=torch.bool)
    allowed = allowed & (i[None, :] != 3)
    allowed[2] = False                                   # a row that sees nothing
    dist = (i[:, None] - i[None, :]).abs().double()
    f = lambda q, k, v: head_forward(q, k, v, allowed, dist, 0.7, cap, slope, 0.0)[0]     # noqa: E731
    grads = head_backward(q, k, v, do, allowed, dist, 0.7, cap, slope, 0.0)[:3]
    for x, dx in zip((q, k, v), grads):
        for at in [(0, 0), (2, 1), (3, 2), (5, 4), (6, 3)]:
            h = 1e-5
            keep = float(x[at])
            x[at] = keep + h
            up = (f(q, k, v) * do).sum()
            x[at] = keep - h
            down = (f(q, k, v) * do).sum()
            x[at] = keep
            # central differences: h^2 times a third derivative of order 10, and 1e-16 / h rounding
            assert abs(float((up - down) / (2 * h) - dx[at])) <= 1e-7


def test_tanh_polynomial():
    text = open(os.path.join(ROOT, "exact_io_aware_23_gb300", "csrc", "fa_score.cuh")).read()
    body = re.search(r"kTanhPoly\[4\] = \{(.*?)\};", text, re.S).group(1)
    c = [float(x) for x in body.replace("\n", " ").split(",")]
    x = torch.linspace(-0.4, 0.4, 200001, dtype=torch.float64)
    t = x * sum(a * x ** (2 * i) for i, a in enumerate(c))
    ref = torch.tanh(x)
    fine = ref != 0
    assert float(((t - ref)[fine] / ref[fine]).abs().max()) < 9.9e-8
    assert math.isclose(c[0], 1.0, abs_tol=9.9e-8)
    body = re.search(r"kTanhLow\[3\] = \{(.*?)\};", text, re.S).group(1)       # the bf16 backward's
    c = [float(v) for v in body.split(",")]
    t = x * sum(a * x ** (2 * i) for i, a in enumerate(c))
    assert float(((t - ref)[fine] / ref[fine]).abs().max()) < 6.3e-6
