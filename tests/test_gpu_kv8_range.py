"""Attention over the FP8 cache where ranges are wide: scales at both ends, one key far above many, long
caches, and what stands in places that a query does not see."""
import numpy as np
import pytest
import torch

import ref8
import ref8_bound
from gpu_helpers import npy
from test_gpu_kv8 import Pair, heads

pytestmark = pytest.mark.gpu


def attend(sb, p, q, causal=False, window=0, sinks=0, scale=None, nan=None):
    """Attention over p's cache against FP64. nan: truth values of out that have to be NaN, the others are
    compared."""
    B, n, Hq, D = q.shape
    out = torch.full_like(q, 9.0)
    lse = torch.full((B, Hq, n), 9.0, device="cuda")
    ws = sb.AttnWorkspace(B, Hq, n, D)
    sb.kv8_attention(q, p.gpu, out, lse, scale=scale, causal=causal, window=window, sinks=sinks, ws=ws)
    sb.check(ws)
    ref, rl, tol, ltol = ref8_bound.attention(p.ref, ref8.f64(q), [n] * B, D ** -0.5 if scale is None else scale, causal,
                                              window, sinks)
    got, gl = ref8.f64(out), npy(lse).astype(np.float64)
    if nan is not None:
        assert np.array_equal(np.isnan(got), nan), np.argwhere(np.isnan(got) != nan)[:5]
        got = np.where(nan, ref, got)
    d = np.abs(got - ref)
    assert (d <= tol).all(), (float(np.nanmax(d / tol)), np.argwhere(~(d <= tol))[:5])
    dead = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), dead)
    e = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, rl))
    assert (e <= ltol).all(), float((e / np.maximum(ltol, 1e-300)).max())
    return ref, tol


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("power", [-130, -126, -123, -119, -112])
def test_values_of_the_smallest_scales(sbg, n, D, power):
    """Exponent byte 0 stands for 2^-127, and its codes need not be zero."""
    p = Pair(sbg, 1, 2, 512, D)
    p.store(heads(1, 450, 2, D, 1), heads(1, 450, 2, D, 2, 2.0 ** power))
    if power < -122:
        assert not npy(p.gpu.v_exp)[:, :, :7].any() and npy(p.gpu.v_codes)[:, :, :450].any()
    attend(sbg, p, heads(1, n, 2, D, 3))
    attend(sbg, p, heads(1, n, 2, D, 3), causal=True, window=100, sinks=3)


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("power", [100, 117])
def test_values_of_the_largest_scales(sbg, n, power):
    p = Pair(sbg, 1, 2, 512, 64)
    p.store(heads(1, 450, 2, 64, 1), heads(1, 450, 2, 64, 2, 2.0 ** power))
    attend(sbg, p, heads(1, n, 2, 64, 3))
