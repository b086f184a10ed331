"""saw_rope_table and saw_rope_append beyond the serving shapes."""
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
