"""GPU parity of the FP8 linear layer (sb_fp8_encode, sb_prepare_weight_fp8, sb_linear_fp8): codes and
scales bit for bit, products against FP64."""
import numpy as np
import pytest
import torch

import ref8
from gpu_helpers import npy

pytestmark = pytest.mark.gpu


def rows(M, K, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    if kind == "outliers":
        x[:, torch.randperm(K, generator=g)[:max(K // 100, 1)]] *= 40
    elif kind == "wide":  # a different magnitude in every block, subnormal bf16 to 2^100
        nb = -(-K // 128)
        s = torch.randint(-133, 100, (M, nb), generator=g).double().exp2()
        x = (x.double() * s.repeat_interleave(128, 1)[:, :K]).float()
    elif kind == "edges":  # largest values on, just below and just above 448 * 2^e; zero blocks
        nb = -(-K // 128)
        top = torch.tensor([448.0, 446.0, 450.0, 0.0, 1.75, 1.7578125, 1.0, 3.5])
        x = x.clamp(-1, 1)
        for i in range(nb):
            t = top[torch.randint(0, 8, (M,), generator=g)]
            blk = x[:, i * 128:(i + 1) * 128]
            blk *= t[:, None]
            blk[:, 5] = t
    return x.to(torch.bfloat16).cuda()


ENC = [(1, 64), (3, 128), (130, 192), (128, 512), (257, 576), (33, 1920), (1000, 7680)]


@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "edges"])
@pytest.mark.parametrize("M,K", ENC)
def test_encode_bitexact(sbg, M, K, kind):
    X = rows(M, K, 1, kind)
    a = sbg.Fp8Tensor(M, K)
    a.sf.fill_(0xEE)
    ws = sbg.Workspace(1, 1)
    sbg.fp8_encode(X, a, ws)
    sbg.check(ws)
    codes, ex, _ = ref8.encode_rows(ref8.f64(X))
    x = ref8.f64(X)
    codes = np.where(np.signbit(x), codes | 128, codes)  # the sign of a value that rounds to zero
    assert np.array_equal(npy(a.codes), codes)
    assert np.array_equal(npy(a.exponents()), ex)
    full = sbg.Fp8Tensor(-(-M // 128) * 128, -(-K // 512) * 512)  # padding rows and blocks hold zero
    full.sf.copy_(a.sf)
    pad = npy(full.exponents())
    assert not pad[M:].any() and not pad[:, ex.shape[1]:].any()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_encode_reports_nonfinite(sbg, bad):
    X = rows(70, 256, 2)
    X[69, 200] = bad
    a, ws = sbg.Fp8Tensor(70, 256), sbg.Workspace(1, 1)
    sbg.fp8_encode(X, a, ws)
    with pytest.raises(sbg.SixbitError) as e:
        sbg.check(ws)
    assert e.value.status == sbg.SB_ENONFINITE
    sbg.check(ws)


class Layer:
    def __init__(self, sb, M, N, K, seed=0, kind="outliers", bias=True):
        self.X, self.W = rows(M, K, seed, kind), (rows(N, K, seed + 1).float() * 0.05).to(torch.bfloat16)
        self.bias = rows(1, N, seed + 2).view(N) if bias else None
        self.ws = sb.Workspace(1, 1)
        self.w = sb.WeightFp8(self.W, self.bias, self.ws)
        self.a = sb.Fp8Tensor(M, K)

    def reference(self, gelu=False):
        """FP64 output and the FP32 kernel's error bound: exact products; sums of 32 products a step,
        each step off by at most 2^-22 of the sum of magnitudes so far (an adder that truncates), the
        split of K adding at most 16 more; bias one rounding; GELU: slope below 1.13 and the hardware
        tanh's 2^-10.9 of half the value."""
        _, _, x = ref8.encode_rows(ref8.f64(self.X))
        _, _, w = ref8.encode_rows(ref8.f64(self.W))
        y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        tol = mag * (x.shape[1] / 32 + 16) * 2.0 ** -22
        if self.bias is not None:
            y = y + ref8.f64(self.bias)[None]
            tol = tol + np.abs(y) * 2.0 ** -23
        if gelu:
            tol = 1.13 * tol + np.abs(y) * (2.0 ** -11.9 + 2.0 ** -20)
            y = ref8.gelu(y)
        return y, tol + 1e-30


SHAPES = [(1, 32, 64), (1, 1920, 1920), (2, 96, 320), (7, 160, 1024), (8, 7680, 640), (9, 256, 256), (16, 416, 1984),
          (17, 1920, 512), (31, 64, 8192), (33, 384, 128), (64, 128, 1920), (65, 5760, 192), (128, 1920, 576), (129, 32, 704), (226, 1920, 1920),
          (255, 224, 448), (300, 512, 1088), (513, 768, 384), (1350, 1920, 640), (700, 3840, 1344)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("gelu", [False, True], ids=["linear", "gelu"])
def test_linear(sbg, M, N, K, gelu):
    L = Layer(sbg, M, N, K, seed=3, bias=not (M % 2 and K % 128))
    ref, tol = L.reference(gelu)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((M + 2, N), 7.0, dtype=dt, device="cuda")
        Y = buf[1:M + 1]
        if Y.data_ptr() % 16:
            continue
        sbg.linear_fp8(L.X, L.a, L.w, Y, epilogue=sbg.EPI_GELU if gelu else sbg.EPI_NONE, ws=L.ws)
        sbg.check(L.ws)
        got = ref8.f64(Y)
        t = tol + (np.abs(ref) + tol) * 2.0 ** -8 if dt == torch.bfloat16 else tol
        assert (np.abs(got - ref) <= t).all(), float((np.abs(got - ref) / t).max())
        assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
    codes, ex, _ = ref8.encode_rows(ref8.f64(L.X))  # X's codes are in `a`, whatever the path
    assert np.array_equal(npy(L.a.codes) & 127, codes & 127) and np.array_equal(npy(L.a.exponents()), ex)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_scales_of_every_magnitude(sbg, M):
    """Blocks of 2^-60 .. 2^60 in X and W: the products' scales leave no block behind."""
    N, K = 128, 1024
    L = Layer(sbg, M, N, K, seed=5, bias=False)
    g = torch.Generator().manual_seed(9)
    s = torch.randint(-50, 50, (1, 8), generator=g).float().exp2().repeat_interleave(128, 1).cuda()
    L.X = (L.X.float() * s).to(torch.bfloat16)
    L.W = (L.W.float() / s).to(torch.bfloat16)
    L.w = sbg.WeightFp8(L.W, None, L.ws)
    Y = torch.empty(M, N, device="cuda")
    sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
    sbg.check(L.ws)
    ref, tol = L.reference()
    assert (np.abs(ref8.f64(Y) - ref) <= tol).all()


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_encoded_operand_serves_several_layers(sbg, M):
    """X None multiplies the codes in `a`: the same bits as encoding within the call."""
    L = Layer(sbg, M, 256, 640, seed=7)
    Y, Z = (torch.empty(M, 256, device="cuda") for _ in range(2))
    sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
    b = sbg.Fp8Tensor(M, 640)
    sbg.fp8_encode(L.X, b, L.ws)
    sbg.linear_fp8(None, b, L.w, Z, ws=L.ws)
    sbg.check(L.ws)
    assert torch.equal(Y, Z)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_skip_flag_writes_nothing(sbg, M):
    L = Layer(sbg, M, 64, 128, seed=8)
    prec = torch.tensor([sbg.SKIP], dtype=torch.int32, device="cuda")
    Y = torch.full((M, 64), 5.0, device="cuda")
    L.a.codes.fill_(3)
    L.a.sf.fill_(9)
    sbg.fp8_encode(L.X, L.a, L.ws, prec=prec)
    sbg.linear_fp8(L.X, L.a, L.w, Y, prec=prec, ws=L.ws)
    sbg.check(L.ws)
    assert (Y == 5).all() and (L.a.codes == 3).all() and (L.a.sf == 9).all()
    prec.fill_(sbg.NVFP4)  # any other value computes
    sbg.linear_fp8(L.X, L.a, L.w, Y, prec=prec, ws=L.ws)
    sbg.check(L.ws)
    assert (Y != 5).any()


@pytest.mark.parametrize("M", [1, 24, 300])
def test_captured_and_replayed_on_new_inputs(sbg, M):
    L = Layer(sbg, M, 192, 384, seed=10)
    Y = torch.empty(M, 192, dtype=torch.bfloat16, device="cuda")
    sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
    for seed in (20, 21):
        L.X.copy_(rows(M, 384, seed, "outliers"))
        g.replay()
        torch.cuda.synchronize()
        got = Y.clone()
        sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
        sbg.check(L.ws)
        assert torch.equal(got, Y)


def test_other_stream(sbg):
    L = Layer(sbg, 200, 256, 512, seed=12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y, Z = (torch.empty(200, 256, device="cuda") for _ in range(2))
    with torch.cuda.stream(s):
        sbg.linear_fp8(L.X, L.a, L.w, Y, ws=L.ws)
    s.synchronize()
    sbg.linear_fp8(L.X, L.a, L.w, Z, ws=L.ws)
    sbg.check(L.ws)
    assert torch.equal(Y, Z)


@pytest.mark.parametrize("N,K,gelu", [(7680, 1920, True), (1920, 7680, False), (1920, 1920, False)])
def test_full_video_sampled(sbg, N, K, gelu):
    """17776 tokens: several tiles for every CTA pair, sampled rows against FP64."""
    M = 17776
    L = Layer(sbg, M, N, K, seed=13)
    Y = torch.empty(M, N, device="cuda")
    Yb = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    epi = sbg.EPI_GELU if gelu else sbg.EPI_NONE
    sbg.linear_fp8(L.X, L.a, L.w, Y, epilogue=epi, ws=L.ws)
    sbg.linear_fp8(None, L.a, L.w, Yb, epilogue=epi, ws=L.ws)
    sbg.check(L.ws)
    assert torch.equal(Yb, Y.to(torch.bfloat16))
    idx = torch.arange(0, M, 181, device="cuda")
    L.X = L.X[idx]
    ref, tol = L.reference(gelu)
    assert (np.abs(ref8.f64(Y[idx]) - ref) <= tol).all()
