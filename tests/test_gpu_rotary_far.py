"""Rotary angles of far positions, slow pairs included, against angles in 80 decimal digits.

The stated bound: |pos| (theta 2^-47 + 2^-62) plus 2^-26 of a turn (2^-23.3) off the angle; the
sine and cosine of it and the fp32 result add less than 2^-22."""
from decimal import Decimal, localcontext

import numpy as np
import pytest

from gpu_common import dev_tensor, to_np

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596")


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _theta(rot, base, scaling, factor, orig, slow, fast):
    b, f = Decimal(base), Decimal(factor)
    if scaling == "NTK":
        b *= (f.ln() * rot / (rot - 2)).exp()
    th = [(-Decimal(2 * i) / rot * b.ln()).exp() for i in range(rot // 2)]
    if scaling == "LINEAR":
        th = [t / f for t in th]
    if scaling == "BY_PARTS":
        w = [min(Decimal(1), max(Decimal(0), (orig * t / TWO_PI - slow) / (fast - slow))) for t in th]
        th = [t * ((1 - v) / f + v) for t, v in zip(th, w)]
    return th


@pytest.mark.parametrize("scaling", ["PLAIN", "LINEAR", "NTK", "BY_PARTS"])
@pytest.mark.parametrize("base,factor", [(10000.0, 8.0), (500000.0, 2.0), (1000000.0, 1.0)])
def test_slow_pairs_at_far_positions(hm, scaling, base, factor):
    import torch
    rot, orig, slow, fast = 128, 4096, 1, 32
    x = np.zeros((1, 1, 1, rot))
    x[..., :rot // 2] = 1.0                     # half layout: (1, 0) becomes (cos, sin)
    for pos in (12345, (1 << 31) - 1, 1 << 40, -(1 << 45) - 7, (1 << 50) + 3, 1 << 57):
        t = dev_tensor(x, "f32")
        hm.hm_rotary(hm.rotary_args(t, None, t, None, base=base, scaling=getattr(hm, "HM_ROTARY_" + scaling),
                                    factor=factor, orig_len=orig, beta_slow=slow, beta_fast=fast,
                                    positions=torch.tensor([[pos]], device="cuda")))
        with localcontext() as c:
            c.prec = 80
            th = _theta(rot, base, scaling, factor, orig, slow, fast)
            ang = np.array([float((pos * v) % TWO_PI) for v in th])
            tol = np.array([float(abs(pos) * (v / 2 ** 47 + Decimal(1) / 2 ** 62)) for v in th])
        tol += 2 * np.pi * 2.0 ** -26 + 2.0 ** -22
        got = to_np(t).ravel()
        assert np.all(np.abs(got[:rot // 2] - np.cos(ang)) <= tol), pos
        assert np.all(np.abs(got[rot // 2:] - np.sin(ang)) <= tol), pos
        assert tol.min() < 0.2      # the slow pairs' angles mean something at every one of them
