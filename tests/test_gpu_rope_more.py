"""saw_rope_table where its arithmetic is least exact.

The bound of a value, factor a: the angle's fraction of a turn is cut to 2^-32
turns (1.5e-9 rad); its distance from the nearest quarter turn, at most pi / 4,
is rounded to binary32, multiplied by a rounded 2 pi 2^-32 and rounded again: 3
* 2^-24 * pi / 4 = 1.4e-7 rad, which moves a cosine there by at most 0.71 of it
and a sine by at most 3 * 2^-24 * x cos x, 1.0e-7 either way.  The series: the
last step rounds by 2^-25, the square of the angle and the sum before it by 2^-26
or less each, and what is left out is below 2^-29: 5e-8 together.  The factor and
the product with it: 2^-24 of the value, 6e-8.  All: 2.1e-7 < 2^-22, times a.
The frequency is a binary64: a relative 2^-52 of it moves the angle of position
p by p w 2^-52 radians, which counts beyond some 10^7 positions.
"""
import math

import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f", [0.25, 1.0, 4.0])
def test_yarn_factor_on_the_values(f):
    """0.1 ln(factor) + 1 for longer contexts, 1 otherwise: the first row's cosines, at angle 0, are that factor."""
    t = torch.empty(4, 64, device="cuda")
    saw.saw_rope_table(t, 1e4, saw.SAW_ROPE_YARN, f, 2048)
    want = max(1.0, 0.1 * math.log(f) + 1)
    assert np.abs(t[0, :32].cpu().numpy() - want).max() <= 2.0 ** -22 * want
    assert (t[0, 32:] == 0).all()


@pytest.mark.parametrize("base,att", [(1e4, 0.0), (1.0625, 1.3), (5e5, 0.75)])
def test_values_over_many_angles(base, att):
    """A million positions of eight pairs, every quarter and its ends."""
    n, r = 1 << 20, 16
    t = torch.empty(n, r, device="cuda")
    saw.saw_rope_table(t, base, att_scale=att)
    w = base ** (-2.0 * np.arange(r // 2) / r)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * torch.from_numpy(w).cuda()
    want = (att or 1.0) * torch.cat((a.cos(), a.sin()), 1)
    # (both sides' frequency and the reference's angle: a few 2^-52 of it)
    bound = (att or 1.0) * (2.0 ** -22 + 8 * 2.0 ** -53 * float(a.max()))
    assert (t.double() - want).abs().max().item() <= bound
