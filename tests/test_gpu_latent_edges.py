"""Latent attention at the edges of its arguments: scales, strides and orders, rows that see nothing beside
values that are not finite. Against the 64-bit forms of tests/_latent.py, with its tolerances."""
import ctypes
import math

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import latent
from test_gpu_latent import DEV, Attend, Prefill, _lib  # noqa: F401

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


@pytest.mark.parametrize("lens,fmt", [([30000, 500], "bf16"), ([700], "bf16"), ([30000, 500], "mxfp4")])
@pytest.mark.parametrize("step", [0, 8])
def test_attend_one_head_with_any_head_stride(lens, fmt, step):
    a = Attend(lens, 1, 64, fmt, seed=19)
    want, want_lse = a.check()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    args = latent.AttendArgs(a.cache.args, a.q.data_ptr(), a.q.stride(0), step, len(lens), 1, a.table.data_ptr(), a.table.shape[0],
                             a.table.shape[1], None, a.lens.data_ptr(), None, 0, 0, a.scale, out.data_ptr(), lse.data_ptr(), None)
    assert latent.load().csa_latent_attend(ctypes.byref(args), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("top", [0, 200])
@pytest.mark.parametrize("heads", [20, 100])
def test_attend_head_major_queries(fmt, top, heads):
    for lens in ([500, 129, 0], [20000, 3000, 64]):
        a = Attend(lens, heads, 64, fmt, top=top, seed=20)
        want = a.run()
        a.q = a.q.transpose(0, 1).contiguous().transpose(0, 1)
        assert a.q.stride(1) > a.q.stride(0)
        out, lse = a.check()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_prefill_head_major():
    p = Prefill([300, 1, 64], [500, 90, 64], 3, seed=21)
    want = p.run()
    p.q, p.kn, p.v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (p.q, p.kn, p.v))
    assert p.q.stride(1) > p.q.stride(0) and p.v.stride(1) > p.v.stride(0)
    out, lse = p.check()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
