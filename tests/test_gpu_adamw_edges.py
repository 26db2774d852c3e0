"""AdamW, 8-bit moments and clipping at the ends of what the formats and the
calls hold, against the fp64 oracle."""
import numpy as np
import pytest
from test_gpu_adamw import U, Flat, _dt, _np

from gpu_env import context
from oracle import adamw as oa

pytestmark = pytest.mark.gpu

def test_factor_is_rounded_once():
    """Norms that are whole numbers of 5 are exact; the factor is the fp32 value nearest to 1 / (norm + 1e-6)."""
    import torch
    ctx = context()
    got = []
    for c in range(1, 101):
        norm, factor = ctx.clip_grads([torch.tensor([3.0 * c, 4.0 * c], device="cuda")], 1.0, apply=False)
        assert float(norm) == 5.0 * c
        got.append(float(factor))
    want = np.float32(1.0 / (5.0 * np.arange(1, 101) + 1e-6))
    np.testing.assert_array_equal(np.float32(got), want)
