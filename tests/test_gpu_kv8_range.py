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


def refer(p):
    """The reference takes over what the GPU's cache holds."""
    g, r = p.gpu, p.ref
    r.codes[0], r.codes[1], r.exps[0], r.exps[1] = npy(g.k_codes), npy(g.v_codes), npy(g.k_exp), npy(g.v_exp)
    r.lens[:] = npy(g.lens)


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


def stepped(p, scales, scores, seed, blank=()):
    """Blocks of 64 tokens whose values have these scales (log2) and whose keys these scores (in nats, for a
    query of 8 in channel 0 at D = 64); a block in `blank` holds zeros in channels 32 and up."""
    m = len(scales) * 64
    k, v = heads(1, m, 1, 64, seed).float() * 0.3, heads(1, m, 1, 64, seed + 1).float()
    k[..., 0] = torch.tensor(scores, dtype=torch.float32, device="cuda").repeat_interleave(64)[None, :, None]
    v *= torch.tensor(scales, dtype=torch.float64, device="cuda").exp2().repeat_interleave(64)[None, :, None, None].float()
    for b in blank:
        v[:, 64 * b:64 * b + 64, :, 32:] = 0
    p.store(k.to(torch.bfloat16), v.to(torch.bfloat16))
    return m


@pytest.mark.parametrize("n", [1, 20, 200])
def test_blocks_of_different_scale_each_by_its_weight(sbg, n):
    """Values 2^20 larger in blocks that get no weight: the others keep their precision."""
    p = Pair(sbg, 1, 1, 512, 64)
    stepped(p, [0, -20, 10, 20, -20, 5, -3, 0], [0, 0, -60, -60, 0, -60, 0, 0], 3)
    q = heads(1, n, 1, 64, 5)
    q[..., 0] = 8.0
    ref, tol = attend(sbg, p, q)
    assert np.median(tol / np.abs(ref)) < 0.02


WIDE = {"small above large": ([60, -60], [0, 110]), "large above small": ([-60, 60], [110, 0]),
        "far apart, equal": ([-100, 20, -100], [0, 0, 0]), "falling": ([100, 50, 0, -50, -100], [0, 50, 100, 150, 200]),
        "rising": ([-100, -50, 0, 50, 100], [200, 150, 100, 50, 0]), "alternating": ([90, -90] * 4, [-150, 10] * 4),
        "sum of the small": ([0, -120, 0, -120], [0, 80, 1, 81]), "ends": ([117, -126], [-180, 3])}


@pytest.mark.parametrize("n", [1, 20, 200])
@pytest.mark.parametrize("case", list(WIDE))
def test_scales_further_apart_than_the_sums_range(sbg, n, case):
    """Blocks whose scales differ by up to 2^243, scores that undo it: the sum and the output each keep
    their precision."""
    scales, scores = WIDE[case]
    p = Pair(sbg, 1, 1, 512, 64)
    stepped(p, scales, scores, 11)
    q = heads(1, n, 1, 64, 5)
    q[..., 0] = 8.0
    attend(sbg, p, q)
    attend(sbg, p, q, causal=True)


@pytest.mark.parametrize("n", [1, 20, 200])
def test_small_blocks_under_large_ones(sbg, n):
    """Equal scores, a block 2^12 to 2^24 larger that holds zeros in half the channels: what the others keep there."""
    for gap in (12, 20, 24):
        p = Pair(sbg, 1, 1, 512, 64)
        stepped(p, [0, gap, 0, 0], [0, 0, 0, 0], 17, blank=(1,))
        q = heads(1, n, 1, 64, 5)
        q[..., 0] = 8.0
        ref, tol = attend(sbg, p, q)
        assert gap == 24 or np.median(tol[..., 32:] / np.abs(ref[..., 32:])) < 0.1  # at 2^-24 a half step is 2^-8 a key


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("nats", [14, 18, 22])
def test_one_key_far_above_a_long_cache(sbg, n, D, nats):
    """A first key that takes nearly all the weight and holds zeros: the output is what the other 131070 add up to."""
    held = 131071
    p = Pair(sbg, 1, 1, held + 1, D)
    k, v = heads(1, held, 1, D, 1, 0.05), torch.ones(1, held, 1, D, dtype=torch.bfloat16, device="cuda")
    v[..., ::3] = 3.0
    k[..., 0] = 0
    k[:, 0, :, 0], v[:, 0] = nats, 0
    p.store(k, v)
    q = heads(1, n, 1, D, 5)
    q[..., 0] = 8.0
    ref, tol = attend(sbg, p, q, scale=0.125)
    if nats <= 18:  # the bound itself says something: 19.3 nats, the most of these rows, are 2^-27.8, and 2^-32 of that is 0.06
        assert (tol < 0.1 * np.abs(ref)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,H", [(1, 2, 2), (3, 4, 1), (40, 1, 1)])
def test_whole_long_cache(sbg, n, Hq, H, D):
    p = Pair(sbg, 1, H, 131072, D)
    p.fill([131071], seed=31)
    attend(sbg, p, heads(1, n, Hq, D, 33))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,held,first", [(5, 130, 128), (16, 200, 192), (300, 448, 256), (384, 448, 320)])
@pytest.mark.parametrize("power", [40, 70, 110])
def test_later_tokens_leave_earlier_rows_alone(sbg, n, held, first, D, power):
    """Causal: values of any size behind a query's position change nothing for it."""
    p = Pair(sbg, 1, 2, 512, D)
    k, v = heads(1, held, 2, D, 1), heads(1, held, 2, D, 2).float()
    v[:, first:] *= 2.0 ** power
    p.store(k, v.to(torch.bfloat16))
    attend(sbg, p, heads(1, n, 2, D, 3), causal=True)


@pytest.mark.parametrize("n", [5, 16, 300])
def test_tokens_behind_the_window_leave_later_rows_alone(sbg, n):
    p = Pair(sbg, 1, 2, 512, 64)
    k, v = heads(1, 500, 2, 64, 1), heads(1, 500, 2, 64, 2).float()
    v[:, :448] *= torch.tensor([2.0 ** 90, 1.0, 2.0 ** -80, 2.0 ** 70, 1.0, 2.0 ** 100, 1.0],
                               device="cuda").repeat_interleave(64)[None, :, None, None]
    p.store(k, v.to(torch.bfloat16))
    for window, sinks in ((1, 0), (40, 0), (100, 3), (200, 70)):
        attend(sbg, p, heads(1, n, 2, 64, 3), causal=True, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,held,at", [(5, 130, 128), (16, 200, 193), (300, 448, 256), (300, 448, 300), (384, 448, 64)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_nonfinite_value_reaches_only_what_sees_it(sbg, n, held, at, D, bad):
    """Causal and windowed: a stored Inf (the code of its block's largest value) or NaN changes its own channel of
    the rows that see it and nothing else."""
    p = Pair(sbg, 1, 2, 512, D)
    k, v = heads(1, held, 2, D, 1), heads(1, held, 2, D, 2)
    v[0, at, 1, 7] = bad
    sbg.kv8_store(k, v, p.gpu, ws=p.ws)
    with pytest.raises(sbg.SixbitError):
        sbg.check(p.ws)
    refer(p)
    nan = p.ref.codes[1] & 0x7f == 0x7f
    nan[:, :, held:] = False
    assert nan.sum() == (1 if bad != bad else 0)
    p.ref.codes[1][nan] = 0
    if bad == bad:  # 448 * 2^120 is past FP32: rows that see it may overflow, keep it below
        p.gpu.v_exp[0, 1, at // 64] = 200
        p.ref.exps[1][0, 1, at // 64] = 200
    q = heads(1, n, 4, D, 3)
    for window, sinks in ((0, 0), (60, 2)):
        mark = None
        if bad != bad:
            mark = np.zeros((1, n, 4, D), bool)
            see = ref8.visible(held, n, True, window, sinks)[:, at]
            mark[0, see, 2:, 7] = True
        attend(sbg, p, q, causal=True, window=window, sinks=sinks, nan=mark)


def test_a_nonfinite_key_reaches_only_what_sees_it(sbg):
    for n, held, at in ((5, 130, 128), (300, 448, 300)):
        p = Pair(sbg, 1, 1, 512, 64)
        k, v = heads(1, held, 1, 64, 1), heads(1, held, 1, 64, 2)
        k[0, at, 0, 7] = float("nan")
        sbg.kv8_store(k, v, p.gpu, ws=p.ws)
        refer(p)
        nan = p.ref.codes[0] & 0x7f == 0x7f
        p.ref.codes[0][nan] = 0
        q = heads(1, n, 1, 64, 3)
        out = torch.empty_like(q)
        ws = sbg.AttnWorkspace(1, 1, n, 64)
        sbg.kv8_attention(q, p.gpu, out, causal=True, ws=ws)
        sbg.check(ws)
        ref, _, tol, _ = ref8_bound.attention(p.ref, ref8.f64(q), [n], 0.125, True)
        got, sees = ref8.f64(out), ref8.visible(held, n, True, 0, 0)[:, at]
        assert np.isnan(got[0, sees]).all()
        assert (np.abs(got - ref)[0, ~sees] <= tol[0, ~sees]).all()


def test_one_workspace_for_a_prompt_and_its_tokens(sbg):
    """Sized for the longest prompt of the largest batch: shorter prompts, single tokens and smaller batches fit."""
    ws = sbg.AttnWorkspace(2, 32, 9000, 64)
    for B, n, Hq, H in ((2, 9000, 32, 2), (2, 700, 8, 2), (1, 40, 32, 1), (2, 1, 32, 2), (1, 3, 4, 4)):
        p = Pair(sbg, B, H, 9024, 64)
        p.fill([9000] + [5000] * (B - 1), seed=9)
        q = heads(B, n, Hq, 64, 10)
        out, own = torch.empty_like(q), torch.empty_like(q)
        sbg.kv8_attention(q, p.gpu, out, causal=True, ws=ws)
        sbg.check(ws)
        sbg.kv8_attention(q, p.gpu, own, causal=True, ws=sbg.AttnWorkspace(B, Hq, n, 64))
        assert torch.equal(out, own)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 8, 40, 150])
def test_wide_scales_and_nan_over_parts_of_a_long_cache(sbg, n, D):
    """Long caches, whose keys are read in parts that are joined: blocks 2^200 apart, zeros among them, shared key heads,
    and a NaN at a position that only the last query sees."""
    held = [8100, 700]
    p = Pair(sbg, 2, 2, 8192, D)
    k, v = heads(2, 8100, 2, D, 1), heads(2, 8100, 2, D, 2).float()
    v[0, 4096:4160] *= 2.0 ** 100
    v[0, 6400:6464] *= 2.0 ** -100
    v[0, 2048:2944] = 0
    v[1, 64:128] *= 2.0 ** -90
    v = v.to(torch.bfloat16)
    p.store(k, v, counts=held)
    q = heads(2, n, 4, D, 3)
    attend(sbg, p, q, causal=True)
    attend(sbg, p, q, causal=True, window=2500, sinks=5)
    v[0, 8099, 1, 9] = float("nan")
    sbg.kv8_store(k, v, p.gpu, start=torch.zeros(2, dtype=torch.int32, device="cuda"),
                  counts=torch.tensor(held, dtype=torch.int32, device="cuda"), ws=p.ws)
    with pytest.raises(sbg.SixbitError):
        sbg.check(p.ws)
    refer(p)
    p.ref.codes[1][0, 1, 8099, 9] = 0
    mark = np.zeros((2, n, 4, D), bool)
    mark[0, n - 1, 2:, 9] = True
    attend(sbg, p, q, causal=True, nan=mark)


@pytest.mark.parametrize("n", [1, 200])
def test_rows_computed_apart_in_a_replayed_graph(sbg, n):
    p = Pair(sbg, 1, 1, 512, 64)
    stepped(p, [0, -100, 0, 90], [0, 0, 0, 0], 11)
    q = heads(1, n, 1, 64, 5)
    out, want, ws = torch.empty_like(q), torch.empty_like(q), sbg.AttnWorkspace(1, 1, n, 64)
    sbg.kv8_attention(q, p.gpu, want, causal=True, ws=ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sbg.kv8_attention(q, p.gpu, out, causal=True, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        sbg.check(ws)
        assert torch.equal(out, want)
    attend(sbg, p, q, causal=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 20, 300])
def test_blocks_of_zeros(sbg, n, D):
    """First, in between, last and with nearly all the weight: zeros count in the sum and in nothing else."""
    for zeros, nats in (([0], 0), ([1, 2], 30), ([0, 3, 6], 60), ([6], 110), ([0, 1, 2, 3, 4, 5, 6], 0)):
        p = Pair(sbg, 1, 1, 512, D)
        k, v = heads(1, 440, 1, D, 7, 0.3), heads(1, 440, 1, D, 8)
        k[..., 0] = 0
        for b in zeros:
            v[:, 64 * b:64 * b + 64] = 0
            k[:, 64 * b:64 * b + 64, :, 0] = nats
        p.store(k, v)
        q = heads(1, n, 1, D, 9, 0.5)
        q[..., 0] = 8.0
        attend(sbg, p, q, causal=True, scale=0.125)
        attend(sbg, p, q, causal=True, window=130, sinks=2, scale=0.125)
