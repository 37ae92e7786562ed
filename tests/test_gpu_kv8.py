"""GPU parity of the FP8 key/value cache and of the attention that reads it."""
import numpy as np
import pytest
import torch

import ref8
from gpu_helpers import npy

pytestmark = pytest.mark.gpu


def heads(B, n, H, D, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, n, H, D, generator=g) * scale
    x[..., :: D // 4] *= 6
    return x.to(torch.bfloat16).cuda()


class Pair:
    """A cache on the GPU and its reference, filled by the same stores; unused memory holds NaN codes
    and the largest exponents."""

    def __init__(self, sb, B, H, cap, D):
        self.sb, self.B, self.H, self.D = sb, B, H, D
        self.gpu, self.ref = sb.KvCache8(B, H, cap, D), ref8.Cache(B, H, cap, D)
        for t in (self.gpu.k_codes, self.gpu.v_codes, self.gpu.k_exp, self.gpu.v_exp):
            t.fill_(0xFF)
        self.ref.codes[:] = 0xFF
        self.ref.exps[:] = 0xFF
        self.ws = sb.Workspace(1, 1)

    def store(self, k, v, start=None, counts=None, check=True):
        dev = [None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda") for t in (start, counts)]
        self.sb.kv8_store(k, v, self.gpu, start=dev[0], counts=dev[1], ws=self.ws)
        if check:
            self.sb.check(self.ws)
        self.ref.store(ref8.f64(k), ref8.f64(v), start, counts)

    def fill(self, lens, seed=0, vscale=1.0):
        n = max(max(lens), 1)
        self.store(heads(self.B, n, self.H, self.D, seed), heads(self.B, n, self.H, self.D, seed + 1, vscale),
                   counts=lens)

    def same(self):
        g, r = self.gpu, self.ref
        assert np.array_equal(npy(g.lens), r.lens)
        assert np.array_equal(npy(g.k_exp), r.exps[0]) and np.array_equal(npy(g.v_exp), r.exps[1])
        assert np.array_equal(npy(g.k_codes), r.codes[0]) and np.array_equal(npy(g.v_codes), r.codes[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 130, 320])
def test_store_prompt_then_tokens(sbg, n, D):
    p = Pair(sbg, 2, 3, 448, D)
    p.store(heads(2, n, 3, D, 1), heads(2, n, 3, D, 2))
    p.same()
    for i in range(3):  # single tokens, each larger: the block's earlier codes are rounded again
        p.store(heads(2, 1, 3, D, 3 + i, 4.0 ** i), heads(2, 1, 3, D, 9 + i, 8.0 ** i))
        p.same()
    p.store(heads(2, 70, 3, D, 30, 0.01), heads(2, 70, 3, D, 31, 100.0))
    p.same()


def test_store_ragged_positions_and_strides(sbg):
    """Sequences at different places and of different counts, keys and values inside one projection."""
    B, H, D, n = 4, 5, 64, 100
    p = Pair(sbg, B, H, 512, D)
    p.fill([100, 64, 1, 0], seed=4)
    x = torch.stack([heads(B, n, H, D, 7), heads(B, n, H, D, 8, 3.0)], 2)  # [B][n][2][H][D]
    p.store(x[:, :, 0], x[:, :, 1], start=[37, 64, 0, 0], counts=[100, 1, 64, 0])
    p.same()
    y = heads(B, H, n, D, 11).transpose(1, 2)  # head-major rows
    p.store(y, y, counts=[7, 100, 0, 63])
    p.same()
    one = heads(1, n, H, D, 12).expand(B, n, H, D)  # one sequence for all of the batch
    p.store(one, one, start=[0, 3, 64, 63])
    p.same()


def test_store_values(sbg):
    """Zeros (exponent 0), subnormals, the largest bf16 values and -0.0."""
    p = Pair(sbg, 1, 2, 128, 64)
    z = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    p.store(z, -z)
    p.same()
    tiny = (heads(1, 3, 2, 64, 1).float() * 2.0 ** -133).to(torch.bfloat16)
    big = torch.full_like(z, 3.3895e38)
    p.store(tiny, big)
    p.same()
    p.store(heads(1, 2, 2, 64, 2), tiny[:, :2])
    p.same()


def test_store_refuses_on_the_device(sbg):
    """Positions past what is held, counts or ends out of range: that sequence keeps everything, the
    others are stored, and the error is reported once."""
    for bad in (dict(start=[5, 11], counts=[2, 2]), dict(start=[5, -1], counts=[2, 2]),
                dict(start=[5, 4], counts=[2, 5]), dict(start=[5, 4], counts=[2, -1])):
        p = Pair(sbg, 2, 2, 64, 64)
        p.fill([10, 10])
        p.store(heads(2, 4, 2, 64, 3), heads(2, 4, 2, 64, 4), check=False, **bad)
        with pytest.raises(sbg.SixbitError) as e:
            sbg.check(p.ws)
        assert e.value.status == sbg.SB_ESHAPE
        p.same()
        sbg.check(p.ws)
    p = Pair(sbg, 2, 2, 64, 64)
    p.fill([64, 60])
    p.store(heads(2, 4, 2, 64, 3), heads(2, 4, 2, 64, 4), check=False)
    with pytest.raises(sbg.SixbitError):
        sbg.check(p.ws)
    p.same()
    assert npy(p.gpu.lens).tolist() == [64, 64]


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_store_reports_nonfinite(sbg, bad):
    p = Pair(sbg, 1, 1, 64, 64)
    k = heads(1, 3, 1, 64, 1)
    k[0, 2, 0, 63] = bad
    sbg.kv8_store(k, heads(1, 3, 1, 64, 2), p.gpu, ws=p.ws)
    with pytest.raises(sbg.SixbitError) as e:
        sbg.check(p.ws)
    assert e.value.status == sbg.SB_ENONFINITE


def test_skip_flag_writes_nothing(sbg):
    p = Pair(sbg, 1, 2, 128, 64)
    p.fill([70])
    prec = torch.tensor([sbg.SKIP], dtype=torch.int32, device="cuda")
    sbg.kv8_store(heads(1, 9, 2, 64, 5), heads(1, 9, 2, 64, 6), p.gpu, prec=prec, ws=p.ws)
    p.same()
    for n in (1, 40, 300):
        q, out = heads(1, n, 2, 64, 7), torch.full((1, n, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        ws = sbg.AttnWorkspace(1, 2, n, 64)
        sbg.kv8_attention(q, p.gpu, out, prec=prec, ws=ws)
        sbg.check(ws)
        assert (out == 3).all()


# ---- attention ----

def attend(sb, p, n, Hq, causal=False, window=0, sinks=0, nqs=None, seed=50, scale=None, qscale=1.0, q=None, out=None):
    B, D = p.B, p.D
    q = heads(B, n, Hq, D, seed, qscale) if q is None else q
    out = torch.full((B, n, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    out.fill_(9.0)
    lse = torch.full((B, Hq, n), 9.0, device="cuda")
    ws = sb.AttnWorkspace(B, Hq, n, D)
    ql = None if nqs is None else torch.tensor(nqs, dtype=torch.int32, device="cuda")
    sb.kv8_attention(q, p.gpu, out, lse, scale=scale, causal=causal, window=window, sinks=sinks, q_lens=ql, ws=ws)
    sb.check(ws)
    nqs = [n] * B if nqs is None else nqs
    ref, rl, tol, ltol = ref8.attention(p.ref, ref8.f64(q), nqs, D ** -0.5 if scale is None else scale, causal, window, sinks)
    got, gl = ref8.f64(out), npy(lse).astype(np.float64)
    for b in range(B):
        r = nqs[b]
        assert (got[b, r:] == 9).all() and (gl[b, :, r:] == 9).all()
        d = np.abs(got[b, :r] - ref[b, :r])
        assert (d <= tol[b, :r]).all(), (b, float(np.nanmax(d / tol[b, :r])), np.argwhere(~(d <= tol[b, :r]))[:3])
        dead = np.isneginf(rl[b, :, :r])
        assert (np.isneginf(gl[b, :, :r]) == dead).all()
        e = np.abs(np.where(dead, 0, gl[b, :, :r]) - np.where(dead, 0, rl[b, :, :r]))
        assert (e <= ltol[b, :, :r]).all(), float((e / ltol[b, :, :r]).max())
    return out, lse


LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 511, 1000]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (4, 1), (10, 2), (16, 1)])
def test_one_token(sbg, Hq, H, D):
    p = Pair(sbg, len(LENS), H, 1024, D)
    p.fill(LENS, seed=3, vscale=2.0)
    attend(sbg, p, 1, Hq)
    attend(sbg, p, 1, Hq, causal=True, window=70, sinks=3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 5, 8, 17, 33, 128, 129, 256, 300])
@pytest.mark.parametrize("Hq,H", [(2, 2), (6, 2), (8, 1)])
def test_many_tokens(sbg, n, Hq, H, D):
    p = Pair(sbg, 5, H, 640, D)
    p.fill([0, 1, 129, 300, 577], seed=5)
    attend(sbg, p, n, Hq)
    attend(sbg, p, n, Hq, causal=True)  # more queries than tokens held: the first ones see nothing


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40, 260])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (64, 64), (65, 1), (100, 130), (200, 700), (5000, 4)])
def test_window_and_sinks(sbg, n, window, sinks, D):
    p = Pair(sbg, 3, 2, 640, D)
    p.fill([70, 333, 600], seed=6)
    attend(sbg, p, n, 4, causal=True, window=window, sinks=sinks)
    attend(sbg, p, n, 4, causal=False, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,nqs", [(7, [7, 0, 3]), (50, [1, 50, 0]), (300, [299, 128, 1]), (257, [257, 129, 256])])
def test_ragged_queries(sbg, n, nqs, D):
    p = Pair(sbg, 3, 2, 512, D)
    p.fill([400, 511, 130], seed=7)
    attend(sbg, p, n, 6, causal=True, nqs=nqs)
    attend(sbg, p, n, 6, causal=False, nqs=nqs)


@pytest.mark.parametrize("n", [1, 30, 270])
def test_strided_queries_and_outputs(sbg, n):
    B, H, D = 2, 3, 64
    p = Pair(sbg, B, H, 256, D)
    p.fill([200, 256], seed=8)
    qkv = heads(B, n, 3 * H, D, 60)
    big = torch.full((B, H, n + 3, D), 1.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, :, 2:n + 2].transpose(1, 2)
    attend(sbg, p, n, H, q=qkv[:, :, H:2 * H], out=out)
    assert (big[:, :, :2] == 1).all() and (big[:, :, n + 2:] == 1).all()


@pytest.mark.parametrize("n", [1, 20, 200])
@pytest.mark.parametrize("qscale", [2.0 ** -40, 1e-3, 12.0, 2.0 ** 20])
def test_query_magnitudes(sbg, n, qscale):
    """Flat and one-hot softmax; the scale parameter brings far queries back."""
    p = Pair(sbg, 1, 2, 512, 64)
    p.fill([450], seed=9)
    attend(sbg, p, n, 2, qscale=qscale, scale=0.125 if qscale < 100 else 0.125 / qscale)


@pytest.mark.parametrize("n", [1, 20, 200])
def test_blocks_of_very_different_scale(sbg, n):
    """Values whose blocks differ by 2^40: weights of small blocks keep their precision when the large
    ones get no weight, and the running maximum follows."""
    p = Pair(sbg, 1, 1, 512, 64)
    k, v = heads(1, 512, 1, 64, 3), heads(1, 512, 1, 64, 4)
    s = torch.tensor([0, -20, 10, 20, -20, 5, -3, 0]).float().exp2().repeat_interleave(64).view(1, 512, 1, 1).cuda()
    v = (v.float() * s).to(torch.bfloat16)
    hide = ((s > 2).float() * -60.0)  # the large blocks are far below in score
    k = k.float() * 0.3
    k[..., 0] = 0.0
    k[..., 1:2] = hide
    p.store(k.to(torch.bfloat16), v)
    q = heads(1, n, 1, 64, 5)
    q[..., 1] = 8.0
    attend(sbg, p, n, 1, q=q)


def test_nan_query_stays_in_its_row(sbg):
    p = Pair(sbg, 1, 2, 128, 64)
    p.fill([100], seed=2)
    for n in (2, 40, 200):
        q = heads(1, n, 2, 64, 3)
        clean, _ = attend(sbg, p, n, 2, q=q)
        bad = q.clone()
        bad[0, 1, 1, 7] = float("nan")
        out = torch.empty_like(q)
        ws = sbg.AttnWorkspace(1, 2, n, 64)
        sbg.kv8_attention(bad, p.gpu, out, ws=ws)
        sbg.check(ws)
        keep = torch.ones(1, n, 2, dtype=torch.bool, device="cuda")
        keep[0, 1, 1] = False
        assert torch.equal(out[keep], clean[keep])
        assert torch.isnan(out[0, 1, 1]).all()


def test_lengths_out_of_range_are_clamped_and_reported(sbg):
    for n in (1, 40, 200):
        p = Pair(sbg, 2, 1, 64, 64)
        p.fill([64, 30], seed=2)
        q = heads(2, n, 1, 64, 3)
        good, _ = attend(sbg, p, n, 1, q=q)
        for field, bad in (("lens", 5000), ("q", n + 5), ("q", -3), ("lens", -2)):
            p.gpu.lens.copy_(torch.tensor([64, 30], dtype=torch.int32))
            ql = torch.tensor([n, n], dtype=torch.int32, device="cuda")
            (p.gpu.lens if field == "lens" else ql)[0] = bad
            out = torch.full_like(q, 9.0)
            ws = sbg.AttnWorkspace(2, 1, n, 64)
            sbg.kv8_attention(q, p.gpu, out, q_lens=ql, ws=ws)
            with pytest.raises(sbg.SixbitError) as e:
                sbg.check(ws)
            assert e.value.status == sbg.SB_ESHAPE
            assert torch.equal(out[1], good[1])
            if bad > 0:
                assert torch.equal(out[0], good[0])
            else:
                assert (out[0] == (9 if field == "q" else 0)).all()


@pytest.mark.parametrize("n", [1, 40, 300])
def test_captured_and_replayed(sbg, n):
    """A stream's step in a graph: store at the device's lengths, then attend; every replay moves on."""
    B, H, D, cap = 2, 2, 64, 1984
    p = Pair(sbg, B, H, cap, D)
    p.fill([50, 7], seed=1)
    k, v, q = heads(B, n, H, D, 2), heads(B, n, H, D, 3), heads(B, n, H, D, 4)
    out = torch.empty_like(q)
    ws = sbg.AttnWorkspace(B, H, n, D)
    lens0 = p.gpu.lens.clone()
    sbg.kv8_store(k, v, p.gpu, ws=ws)
    sbg.kv8_attention(q, p.gpu, out, causal=True, ws=ws)
    torch.cuda.synchronize()
    p.gpu.lens.copy_(lens0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sbg.kv8_store(k, v, p.gpu, ws=ws)
        sbg.kv8_attention(q, p.gpu, out, causal=True, ws=ws)
    # the warm-up's tokens were dropped, but their block exponents may have risen: refill the reference
    p.ref.codes[0], p.ref.codes[1] = npy(p.gpu.k_codes), npy(p.gpu.v_codes)
    p.ref.exps[0], p.ref.exps[1] = npy(p.gpu.k_exp), npy(p.gpu.v_exp)
    for i in range(3):
        k.copy_(heads(B, n, H, D, 70 + i, 1.0 + i))
        v.copy_(heads(B, n, H, D, 80 + i))
        q.copy_(heads(B, n, H, D, 90 + i))
        g.replay()
        sbg.check(ws)
        p.ref.store(ref8.f64(k), ref8.f64(v))
        p.same()
        ref, _, tol, _ = ref8.attention(p.ref, ref8.f64(q), [n] * B, D ** -0.5, True)
        assert (np.abs(ref8.f64(out) - ref) <= tol).all()


def test_two_streams_with_their_own_workspaces(sbg):
    p = Pair(sbg, 1, 2, 1024, 64)
    p.fill([1000], seed=3)
    for n in (1, 300):
        qs = [heads(1, n, 4, 64, s) for s in (1, 2)]
        want = [attend(sbg, p, n, 4, q=q)[0].clone() for q in qs]
        streams, outs = [torch.cuda.Stream() for _ in qs], [torch.empty_like(q) for q in qs]
        wss = [sbg.AttnWorkspace(1, 4, n, 64) for _ in qs]
        torch.cuda.synchronize()
        for _ in range(5):
            for s, q, o, ws in zip(streams, qs, outs, wss):
                with torch.cuda.stream(s):
                    sbg.kv8_attention(q, p.gpu, o, ws=ws)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_same_result_twice(sbg):
    p = Pair(sbg, 2, 2, 4096, 128)
    p.fill([4000, 77], seed=3)
    for n in (1, 5, 130):
        a, la = attend(sbg, p, n, 8, seed=4)
        a, la = a.clone(), la.clone()
        b, lb = attend(sbg, p, n, 8, seed=4)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("D,cap", [(128, 1 << 25), (64, 1 << 26)])
def test_offsets_past_32_bits(sbg, D, cap):
    """A cache of more than 2^32 bytes for keys: the last tokens of the last head."""
    n = cap - 3
    cache = sbg.KvCache8(1, 2, cap, D)
    cache.lens.fill_(n - 40)
    k, v = heads(1, 40, 2, D, 1), heads(1, 40, 2, D, 2)
    ws = sbg.AttnWorkspace(1, 2, 1, D)
    sbg.kv8_store(k, v, cache, ws=ws)
    small = Pair(sbg, 1, 2, 128, D)
    off = (n - 40) % 64  # the same place inside a block
    if off:
        z = torch.zeros(1, off, 2, D, dtype=torch.bfloat16, device="cuda")
        small.store(z, z)
    small.store(k, v)
    first = (n - 40) // 64 * 64
    held = small.gpu.k_codes[:, :, off:off + 40]
    assert torch.equal(cache.k_codes[:, :, n - 40:n], held)
    for nq in (1, 40):
        q = heads(1, nq, 2, D, 3)
        a, b = torch.empty_like(q), torch.empty_like(q)
        ws2 = sbg.AttnWorkspace(1, 2, nq, D)
        sbg.kv8_attention(q, cache, a, window=40, ws=ws2)
        sbg.kv8_attention(q, small.gpu, b, window=40, ws=ws2)
        sbg.check(ws2)
        d = (a.float() - b.float()).abs()
        assert (d <= 2.0 ** -7 * b.float().abs() + 2.0 ** -9).all() and first % 64 == 0
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("B,H,Hq,D", [(33, 1, 1, 64), (70, 2, 4, 64), (70, 2, 2, 128), (300, 4, 4, 64), (1200, 1, 3, 64)])
@pytest.mark.parametrize("n", [1, 3])
def test_many_sequences_of_mixed_lengths(sbg, B, H, Hq, D, n):
    """More sequences than a warp has lanes, among them empty ones and ones without queries; from 1184
    heads on a block takes a whole head."""
    g = torch.Generator().manual_seed(B)
    lens = [int(x) for x in torch.randint(0, 300, (B,), generator=g)]
    lens[0], lens[B // 2], lens[-1] = 0, 383, 1
    p = Pair(sbg, B, H, 384, D)
    p.fill(lens, seed=3)
    attend(sbg, p, n, Hq, causal=True)
    attend(sbg, p, n, Hq, nqs=[b % (n + 1) for b in range(B)], window=50, sinks=2)
    attend(sbg, p, n, Hq, nqs=[0] * B)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,H", [(17, 1, 1), (40, 4, 2), (150, 2, 2)])
def test_parts_of_long_caches(sbg, n, Hq, H, D):
    """Few row tiles over long caches: the keys are split and the parts joined, some of them empty."""
    p = Pair(sbg, 3, H, 8192, D)
    p.fill([8100, 600, 3], seed=12)
    attend(sbg, p, n, Hq, causal=True)
    attend(sbg, p, n, Hq, nqs=[n, n - 5, 1])
    attend(sbg, p, n, Hq, causal=True, window=900, sinks=130)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("power", [-126, -118, -100, 100])
def test_query_rows_at_the_ends_of_the_range(sbg, n, power):
    """Rows near the smallest and the largest bf16 values, brought back by the scale: the power of two
    that a row is multiplied with and the one that takes it back are the same."""
    p = Pair(sbg, 1, 1, 256, 64)
    p.fill([200], seed=9)
    attend(sbg, p, n, 1, qscale=2.0 ** power, scale=0.125 * 2.0 ** -power)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_nan_in_the_cache_stays_in_its_head(sbg, n):
    """A stored NaN is reported; other heads and sequences, and tiles that no query sees, are not touched by it."""
    k, v = heads(2, 400, 2, 64, 21), heads(2, 400, 2, 64, 22)
    q = heads(2, n, 2, 64, 23)

    def run(v, **kw):
        p = Pair(sbg, 2, 2, 512, 64)
        sbg.kv8_store(k, v, p.gpu, ws=p.ws)
        out = torch.empty_like(q)
        ws = sbg.AttnWorkspace(2, 2, n, 64)
        sbg.kv8_attention(q, p.gpu, out, ws=ws, **kw)
        sbg.check(ws)
        return out, p.ws

    bad = v.clone()
    bad[1, 10, 0, 5] = float("nan")
    clean, _ = run(v)
    got, ws = run(bad)
    with pytest.raises(sbg.SixbitError) as e:
        sbg.check(ws)
    assert e.value.status == sbg.SB_ENONFINITE
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, :, 1], clean[1, :, 1])
    assert torch.isnan(got[1, :, 0]).any(-1).all()
    assert torch.equal(run(bad, window=200)[0], run(v, window=200)[0])  # the block of token 10 ends at 64
