"""The GELU of the FP8 linear layer over its whole range, the negative tail included."""
import numpy as np
import pytest
import torch

import ref8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 8, 20, 300, 20000])
def test_gelu_keeps_its_relative_precision(sbg, M):
    """The bias alone carries the argument (X is zero), so it is exact. y = v / (1 + 2^(-2 log2(e) u)): u is four
    FP32 roundings from exact, so the exponent a is off by |a| 2^-22, exp2 and the reciprocal by 2^-21
    together, the rest by 2^-22: |a| 2^-22 + 2^-20 of the value; a reciprocal below 2^-126 is zero, which is off by
    2^-126 |v| at most."""
    N = 1024
    v = torch.linspace(-12.0, 6.0, N - 4).tolist() + [0.0, -30.0, 30.0, -1e30]
    bias = torch.tensor(v, dtype=torch.bfloat16, device="cuda")
    X, W = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda"), torch.randn(N, 64, device="cuda").to(torch.bfloat16)
    ws = sbg.Workspace(1, 1)
    w, a = sbg.WeightFp8(W, bias, ws), sbg.Fp8Tensor(M, 64)
    b = ref8.f64(bias)
    arg = 2 * np.log2(np.e) * np.sqrt(2 / np.pi) * (b + 0.044715 * b ** 3)
    with np.errstate(over="ignore"):
        ref = b / (1 + np.exp2(-arg))
    rel = np.minimum(np.abs(arg), 200.0) * 2.0 ** -22 + 2.0 ** -20
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        Y = torch.empty(M, N, dtype=dt, device="cuda")
        sbg.linear_fp8(X, a, w, Y, epilogue=sbg.EPI_GELU, ws=ws)
        sbg.check(ws)
        d = np.abs(ref8.f64(Y) - ref[None])
        tol = np.abs(ref) * (rel + half) + np.abs(b) * 2.0 ** -126
        assert (d <= tol).all(), (float(np.nanmax(d / tol)), b[np.argmax((d / np.maximum(tol, 1e-300)).max(0))])
