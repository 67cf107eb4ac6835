"""Calls of the rotary, paged-cache and tree entry points as users make them: gradients through rope, strides of
dimensions of size one, a mask shared by all nodes, contexts far past the table, workspaces, values near fp32's end."""
import math

import numpy as np
import pytest
import torch

import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, check_tree, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rotary_coefficients():
    """cos and sin of an angle that is exact modulo a turn: folded to an eighth of a turn, its fp32 form is off by at
    most 2^-25 of pi/4 (2.4e-8), and sincospif by one ulp of its result."""
    D, T = 256, 4096
    g = gen(650)
    turns = torch.randint(-2**62, 2**62, (D // 2,), generator=g)
    pos = torch.randint(0, 2**40, (T,), generator=g)
    x = torch.zeros(T, 1, D)
    x[..., :D // 2] = 1.0
    y, _ = rq.rope(x.to(DEV), None, pos.to(DEV), turns.to(DEV))
    p, w = pos.numpy().astype(np.uint64)[:, None], turns.numpy().astype(np.uint64)[None, :]
    phase = p * w                                                # wraps modulo one turn
    whole = phase >> np.uint64(61)                               # eighths, so that the rest keeps 53 bits
    rest = (phase & np.uint64(2**61 - 1)).astype(np.float64) * (2 * math.pi * 2.0**-64)
    eighth = whole.astype(np.float64) * (math.pi / 4)
    cos = np.cos(eighth) * np.cos(rest) - np.sin(eighth) * np.sin(rest)
    sin = np.sin(eighth) * np.cos(rest) + np.cos(eighth) * np.sin(rest)
    got = y[:, 0].cpu().double().numpy()
    ulp = lambda v: np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-12))) - 23)
    for have, want, other in ((got[:, :D // 2], cos, sin), (got[:, D // 2:], sin, cos)):
        err = np.abs(have - want)
        assert (err <= 2.4e-8 * np.abs(other) + ulp(want) + 1e-15).all(), float((err - 2.4e-8 * np.abs(other) - ulp(want)).max())
