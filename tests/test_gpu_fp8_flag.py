"""The FP8 linear layer behind a precision flag that the stream changes right after it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 8, 200, 6000])
def test_flag_changed_right_behind_a_skipped_call(sbg, M):
    """Skipped and computed calls in turn, the flag rewritten between them without a wait: a skipped call's first
    launch has ended, too, when the flag changes, so nothing of it is written."""
    g = torch.Generator().manual_seed(M)
    X = [torch.randn(M, 512, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    W = (torch.randn(256, 512, generator=g) * 0.05).to(torch.bfloat16).cuda()
    ws = sbg.Workspace(1, 1)
    w, a, b = sbg.WeightFp8(W, None, ws), sbg.Fp8Tensor(M, 512), sbg.Fp8Tensor(M, 512)
    want, Y = torch.empty(M, 256, device="cuda"), torch.empty(M, 256, device="cuda")
    sbg.linear_fp8(X[0], a, w, want, ws=ws)
    codes = a.codes.clone()
    prec = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(200):
        prec.fill_(sbg.NVFP4)
        sbg.linear_fp8(X[0], a, w, Y, prec=prec, ws=ws)
        prec.fill_(sbg.SKIP)
        sbg.linear_fp8(X[1], a, w, Y, prec=prec, ws=ws)
        prec.fill_(sbg.NVFP4)
        sbg.linear_fp8(X[1], b, w, torch.empty_like(Y), prec=prec, ws=ws)
    sbg.check(ws)
    assert torch.equal(Y, want) and torch.equal(a.codes, codes)
