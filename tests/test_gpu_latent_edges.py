"""Latent attention at the edges of its arguments: scales, strides and orders, rows that see nothing beside
values that are not finite. Against the 64-bit forms of tests/_latent.py, with its tolerances."""
import math

import pytest
import torch

from test_gpu_latent import Attend, Prefill, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("scale", [1e-37, 1e-38, 1e-42])
@pytest.mark.parametrize("lens,top", [([700, 1, 0, 64], 0), ([30000, 7], 0), ([900] * 200, 300)])
def test_attend_scales_down_to_subnormal(fmt, scale, lens, top):
    """Scores of almost nothing: the softmax is a mean, lse the logarithm of the count."""
    a = Attend(lens, 16, 64, fmt, top=top, req=[0] * len(lens) if top else None, seed=17)
    a.scale = scale
    a.check()


@pytest.mark.parametrize("scale", [1e-38, 1e-42])
def test_prefill_scales_down_to_subnormal(scale):
    p = Prefill([300, 7], [500, 7], 2, seed=18)
    p.scale = scale
    p.check()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_prefill_rows_without_keys_beside_values_that_are_not_finite(bad):
    """More queries than keys: the first rows see none, in a tile whose other rows see a NaN or infinite value."""
    p = Prefill([200, 40], [150, 30], 2, seed=16)
    p.v[3], p.v[160] = bad, bad
    out, lse = p.run()
    assert int(p.st) == 0
    for rows in (slice(0, 50), slice(200, 210)):
        assert not out[rows].any() and bool(torch.isneginf(lse[rows]).all())
