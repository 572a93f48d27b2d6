"""The polynomial behind the activation's normal distribution (csrc/zero_act.hip),
with the coefficients read from there, against the complementary error function."""
import math
import os
import re

import pytest
import torch

from sharded_mixed_precision_step_amd import _build

pytestmark = pytest.mark.cpu


def _coefficients():
    """Highest power first."""
    with open(os.path.join(_build.CSRC, "zero_act.hip"), encoding="utf-8") as f:
        text = f.read()
    first = re.search(r"float m = ([-\d.e]+)f;", text)
    rest = re.findall(r"m = __builtin_fmaf\(m, t, ([-\d.e]+)f\);", text)
    assert first and len(rest) == 9
    return [float(c) for c in (first.group(1), *rest)]


def test_the_fit():
    """Phi(-x) = exp(-x^2 / 2) t P(t), t = 1 / (1 + x / 4): in 64 bits to 6e-8 of the value,
    from 0 to where it leaves fp32's normal range."""
    x = torch.linspace(0, 13, 1 << 18, dtype=torch.float64)
    t = 1 / (1 + x / 4)
    m = torch.zeros_like(x)
    for c in _coefficients():
        m = m * t + torch.tensor(c, dtype=torch.float32).double()
    want = 0.5 * torch.special.erfc(x * math.sqrt(0.5))
    err = (torch.exp(-0.5 * x * x) * t * m / want - 1).abs()
    assert float(err.max()) < 6e-8
    # What an error of t makes of the value, d log(t P(t)) / d log t.  With R(x) = Phi(-x)
    # exp(x^2 / 2) that is -(4 + x) R' / R, R' = x R - 1 / sqrt(2 pi): 4 sqrt(2 / pi) =
    # 3.19 at 0, and less behind.
    p = t * m
    growth = (p[1:].log() - p[:-1].log()) / (t[1:].log() - t[:-1].log())
    assert float(growth.abs().max()) < 4 * math.sqrt(2 / math.pi) + 1e-3
