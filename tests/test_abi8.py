"""Host-side validation of the 8-bit entry points (no GPU: every case fails before any CUDA call)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sb():
    from video_diffusion_mixed_b200 import build
    build.build()
    from video_diffusion_mixed_b200 import sixbit
    sixbit.lib()
    return sixbit


def P(a):
    return ctypes.c_void_p(a)


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def test_sf_bytes(sb):
    f = sb.lib().sb_fp8_sf_bytes
    assert f(1, 64) == 512 and f(128, 512) == 512 and f(129, 576) == 2048 and f(17776, 1920) == 139 * 4 * 512
    assert f(-1, 64) == -1 and f(1, -64) == -1


def test_encode_and_linear(sb):
    L = sb.lib()
    a, ws = sb.Fp8(0x1000, 0x2000, 4, 128), P(0x9000)
    enc = lambda X, M, K, t, w=ws: L.sb_fp8_encode(X, M, K, None, t and ctypes.byref(t), w, None)  # noqa: E731
    assert enc(None, 4, 128, a) == sb.SB_EINVAL
    assert enc(P(0x100), 4, 128, None) == sb.SB_EINVAL
    assert enc(P(0x100), 4, 128, a, None) == sb.SB_EINVAL
    assert enc(P(0x108), 4, 128, a) == sb.SB_EALIGN
    assert enc(P(0x100), 0, 128, a) == sb.SB_ESHAPE
    assert enc(P(0x100), (1 << 30) + 1, 128, a) == sb.SB_ESHAPE
    assert enc(P(0x100), 4, 96, a) == sb.SB_EUNSUPPORTED
    assert enc(P(0x100), 4, 16448, a) == sb.SB_EUNSUPPORTED
    assert enc(P(0x100), 5, 128, a) == sb.SB_ESHAPE
    assert enc(P(0x100), 4, 128, sb.Fp8(0x1000, 0, 4, 128)) == sb.SB_EINVAL
    assert enc(P(0x100), 4, 128, sb.Fp8(0x1004, 0x2000, 4, 128)) == sb.SB_EALIGN
    assert L.sb_fp8_encode(P(0x100), 4, 128, P(0x102), ctypes.byref(a), ws, None) == sb.SB_EALIGN

    w = sb.WeightFp8C(None, sb.Fp8(0x3000, 0x4000, 64, 128), 64, 128)
    lin = lambda M=4, t=a, wt=w, epi=0, out=0, Y=P(0x5000), X=P(0x100): L.sb_linear_fp8(  # noqa: E731
        X, ctypes.byref(t), None, ctypes.byref(wt), epi, out, Y, M, ws, None)
    assert lin(Y=None) == sb.SB_EINVAL
    assert lin(epi=2) == sb.SB_EINVAL
    assert lin(out=2) == sb.SB_EINVAL
    assert lin(M=0) == sb.SB_ESHAPE
    assert lin(M=5) == sb.SB_ESHAPE
    assert lin(Y=P(0x5004)) == sb.SB_EALIGN
    assert lin(X=P(0x101)) == sb.SB_EALIGN
    assert lin(wt=sb.WeightFp8C(P(0x8), sb.Fp8(0x3000, 0x4000, 64, 128), 64, 128)) == sb.SB_EALIGN
    assert lin(wt=sb.WeightFp8C(None, sb.Fp8(0x3000, 0x4000, 48, 128), 48, 128)) == sb.SB_EUNSUPPORTED
    assert lin(wt=sb.WeightFp8C(None, sb.Fp8(0x3000, 0x4000, 64, 64), 64, 128)) == sb.SB_ESHAPE
    c = sb.WeightFp8C()
    c.w = sb.Fp8(0x3000, 0x4000, 40, 128)
    assert L.sb_prepare_weight_fp8(P(0x100), None, 40, 128, ctypes.byref(c), ws, None) == sb.SB_EUNSUPPORTED
    c.w = sb.Fp8(0x3000, 0x4000, 32, 128)
    assert L.sb_prepare_weight_fp8(P(0x100), P(0x8), 32, 128, ctypes.byref(c), ws, None) == sb.SB_EALIGN
    assert L.sb_prepare_weight_fp8(P(0x100), None, 64, 128, ctypes.byref(c), ws, None) == sb.SB_ESHAPE


def cache(sb, **kw):
    f = dict(k_codes=0x1000, v_codes=0x2000, k_exp=0x3000, v_exp=0x4000, lens=0x5000, batch=2, heads=4, capacity=128,
             dim=64)
    f.update(kw)
    return sb.Kv8(*f.values())


BAD_CACHES = [(dict(v_codes=None), "SB_EINVAL"), (dict(lens=None), "SB_EINVAL"), (dict(k_exp=0x3004), "SB_EALIGN"),
              (dict(dim=96), "SB_EUNSUPPORTED"), (dict(dim=0), "SB_EUNSUPPORTED"), (dict(batch=0), "SB_ESHAPE"),
              (dict(heads=20000), "SB_ESHAPE"), (dict(capacity=100), "SB_ESHAPE"), (dict(capacity=0), "SB_ESHAPE"),
              (dict(batch=16384, heads=16384), "SB_ESHAPE"), (dict(batch=256, heads=4, capacity=1 << 30), "SB_ESHAPE")]


def test_store(sb):
    L = sb.lib()
    s = strides(1024, 256, 64)

    def store(c=None, k=P(0x100), v=P(0x200), ks=s, vs=s, n=4, start=None, counts=None, ws=P(0x9000), prec=None):
        c = c or cache(sb)
        return L.sb_kv8_store(k, ks, v, vs, n, ctypes.byref(c), start, counts, prec, ws, None)
    for kw, status in BAD_CACHES:
        assert store(cache(sb, **kw)) == getattr(sb, status), kw
    assert store(k=None) == sb.SB_EINVAL and store(ks=None) == sb.SB_EINVAL and store(ws=None) == sb.SB_EINVAL
    assert store(v=P(0x204)) == sb.SB_EALIGN
    assert store(n=0) == sb.SB_ESHAPE and store(n=129) == sb.SB_ESHAPE
    assert store(ks=strides(1024, 4, 64)) == sb.SB_EALIGN and store(vs=strides(-8, 256, 64)) == sb.SB_EALIGN
    assert store(vs=strides(1 << 60, 256, 64)) == sb.SB_ESHAPE
    assert store(start=P(0x6)) == sb.SB_EALIGN and store(prec=P(0x2)) == sb.SB_EALIGN


def test_attention(sb):
    L = sb.lib()
    s = strides(1024, 256, 64)
    need = ctypes.c_size_t(0)
    assert L.sb_kv8_workspace_size(2, 4, 3, 64, ctypes.byref(need)) == sb.SB_OK and need.value >= 256

    def attn(c=None, q=P(0x100), qs=s, n=3, hq=4, scale=1.0, causal=0, window=0, sinks=0, ql=None, out=P(0x200), os=s,
             lse=None, ws=P(0x9000), size=1 << 40):
        c, o = c or cache(sb), sb.Attn(scale, causal, window, sinks)
        return L.sb_kv8_attention(q, qs, n, hq, ctypes.byref(c), ctypes.byref(o), ql, out, os, lse, None, ws, size,
                                  None)
    for kw, status in BAD_CACHES:
        assert attn(cache(sb, **kw)) == getattr(sb, status), kw
    assert attn(q=None) == sb.SB_EINVAL and attn(os=None) == sb.SB_EINVAL and attn(ws=None) == sb.SB_EINVAL
    assert attn(hq=6) == sb.SB_ESHAPE and attn(hq=0) == sb.SB_ESHAPE and attn(n=0) == sb.SB_ESHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attn(scale=scale) == sb.SB_EINVAL
    assert attn(window=-1) == sb.SB_EINVAL and attn(sinks=4) == sb.SB_EINVAL and attn(window=4, sinks=-1) == sb.SB_EINVAL
    assert attn(out=P(0x204)) == sb.SB_EALIGN and attn(lse=P(0x204)) == sb.SB_EALIGN and attn(ql=P(0x6)) == sb.SB_EALIGN
    assert attn(qs=strides(1024, 256, 60)) == sb.SB_EALIGN
    assert attn(size=need.value - 1) == sb.SB_ESHAPE
    for bad in ((0, 4, 1, 64), (1, 0, 1, 64), (1, 1, 0, 64)):
        assert L.sb_kv8_workspace_size(*bad, ctypes.byref(need)) == sb.SB_ESHAPE
    assert L.sb_kv8_workspace_size(1, 1, 1, 80, ctypes.byref(need)) == sb.SB_EUNSUPPORTED
    assert L.sb_kv8_workspace_size(1, 1, 1, 64, None) == sb.SB_EINVAL


def test_binding_refuses_host_tensors(sb):
    """Tensors that are not on a CUDA device never reach the library."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(sb.SixbitError) as e:
        sb.WeightFp8(x)
    assert e.value.status == sb.SB_EINVAL
    with pytest.raises(sb.SixbitError):
        sb.KvCache8(1, 1, 64, 64, device="cpu")


def test_reference_grid():
    """The test reference's E4M3 grid and encoder against torch's own float8 type."""
    import numpy as np
    import ref8
    every = np.arange(256, dtype=np.uint8)
    fine = every[(every & 127) != 127]
    want = torch.from_numpy(fine).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref8.value_of(fine), want)
    assert np.array_equal(ref8.code_of(want), fine)
    x = torch.randn(4000, generator=torch.Generator().manual_seed(1)) * torch.tensor([0.001, 0.1, 3, 100]).repeat(1000)
    x = x.clamp(-448, 448)
    assert np.array_equal(ref8.nearest_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    for a, e in ((448.0, 0), (449.0, 1), (1.75, -8), (1.76, -7), (0.0, -127), (2.0 ** -133, -127), (3.38e38, 120)):
        assert ref8.exponent(a) == e
