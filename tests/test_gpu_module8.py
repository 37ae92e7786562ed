"""The 8-bit operators as one attention module, under the Temporal Delta Cache: q/k/v projection, store,
attention, output projection, module record."""
import numpy as np
import pytest
import torch

import ref8
from gpu_helpers import rel_fro

pytestmark = pytest.mark.gpu


def test_attention_module_of_a_denoising_step(sbg):
    text, frames, H, D = 30, 200, 3, 64
    M, C = text + frames, H * D
    g = torch.Generator().manual_seed(1)

    def weight(n, k):
        return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).cuda()

    Wqkv, Wo = weight(3 * C, C), weight(C, C)
    ws, aws = sbg.Workspace(M, C), sbg.AttnWorkspace(1, H, M, D)
    wqkv, wo = sbg.WeightFp8(Wqkv), sbg.WeightFp8(Wo)
    a, b = sbg.Fp8Tensor(M, C), sbg.Fp8Tensor(M, C)
    cache = sbg.KvCache8(1, H, 256, D)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv = torch.empty(M, 3 * C, dtype=torch.bfloat16, device="cuda")
    o, y = (torch.empty(M, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last, stats, state = torch.zeros_like(y), sbg.alloc_stats(), sbg.alloc_state()
    prec = torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg, rule = sbg.config(tdc_thresh=10.0), sbg.Rule(1.0, 0.0, 0.1)
    x0 = torch.randn(M, C, generator=g)
    for step in range(4):
        x = (x0 + 0.05 * step * torch.randn(M, C, generator=g)).to(torch.bfloat16).cuda()
        before = y.clone()
        sbg.module_decide(state, cfg, [rule], [prec])
        sbg.linear_fp8(x, a, wqkv, qkv, prec=prec, ws=ws)
        q, k, v = qkv.view(1, M, 3, H, D).unbind(2)
        sbg.kv8_store(k, v, cache, start=zero, prec=prec, ws=aws)
        sbg.kv8_attention(q, cache, o.view(1, M, H, D), prec=prec, ws=aws)
        sbg.linear_fp8(o, b, wo, y, prec=prec, ws=ws)
        sbg.module_record(y, x, last, prec, stats, state, ws)
        sbg.check(ws)
        sbg.check(aws)
        if step >= 2:  # the module's output barely changed: every kernel of the step wrote nothing
            assert int(prec.item()) == sbg.SKIP and torch.equal(y, before)
            continue
        # FP64 from the definitions, each stage on the kernel's own rounded input
        def linear(t, W):
            return ref8.encode_rows(ref8.f64(t))[2] @ ref8.encode_rows(ref8.f64(W))[2].T
        assert rel_fro(ref8.f64(qkv), linear(x, Wqkv)) < 2.0 ** -8
        ref = ref8.Cache(1, H, 256, D)
        ref.store(ref8.f64(k), ref8.f64(v))
        want, _, tol, _ = ref8.attention(ref, ref8.f64(q), [M], D ** -0.5)
        assert (np.abs(ref8.f64(o).reshape(want.shape) - want) <= tol).all()
        assert rel_fro(ref8.f64(y), linear(o, Wo)) < 2.0 ** -8
        # and the module's error against full precision stays that of 3-bit mantissas
        X = ref8.f64(x)
        f = (X @ ref8.f64(Wqkv).T).reshape(M, 3, H, D)
        s = np.einsum("ihd,jhd->hij", f[:, 0], f[:, 1]) * D ** -0.5
        p = np.exp(s - s.max(2, keepdims=True))
        full = np.einsum("hij,jhd->ihd", p / p.sum(2, keepdims=True), f[:, 2]).reshape(M, C) @ ref8.f64(Wo).T
        assert rel_fro(ref8.f64(y), full) < 0.12
