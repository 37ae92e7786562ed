"""The 8-bit operators from their definitions, in numpy FP64 (no code shared with the library)."""
import numpy as np

TOKENS = 64
BLOCK = 128


def f64(t):
    """A torch tensor's values in FP64 (bf16, fp32)."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def nearest_e4m3(v):
    """v on the E4M3 grid: 3 mantissa bits, smallest normal 2^-6, ties to even, saturating at 448."""
    v = np.asarray(v, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.clip(np.rint(v / step) * step, -448, 448)


def code_of(v):
    """The E4M3 byte of a value on the grid (v may be -0.0)."""
    m = np.abs(v)
    e = np.floor(np.log2(np.maximum(m, 2.0 ** -6)))
    sub = m < 2.0 ** -6
    byte = np.where(sub, m * 512, (e + 7) * 8 + (m / np.exp2(e) - 1) * 8).astype(np.int64)
    return np.where(np.signbit(v), byte | 128, byte).astype(np.uint8)


def value_of(code):
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where(c & 128, -v, v)


def exponent(amax):
    """Smallest integer e >= -127 with amax <= 448 * 2^e; -127 for 0."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(amax / 448)) - 1, -200.0)
    for _ in range(3):
        e = np.where(amax > 448 * np.exp2(e), e + 1, e)
    return np.maximum(e, -127).astype(np.int64)


def encode_rows(x):
    """(codes [R][K], exponent bytes [R][nb], values [R][K]) of FP64 rows in blocks of 128 channels."""
    R, K = x.shape
    nb = -(-K // BLOCK)
    codes, vals = np.zeros((R, K), np.uint8), np.zeros((R, K))
    ex = np.zeros((R, nb), np.uint8)
    for i in range(nb):
        sl = slice(i * BLOCK, min((i + 1) * BLOCK, K))
        e = exponent(np.abs(x[:, sl]).max(1))
        g = nearest_e4m3(x[:, sl] * np.exp2(-e[:, None].astype(np.float64)))
        codes[:, sl], vals[:, sl], ex[:, i] = code_of(g), g * np.exp2(e[:, None].astype(np.float64)), e + 127
    return codes, ex, vals


def gelu(v):
    return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))


class Cache:
    """A key/value cache of FP64 code values and exponents: store() follows the definition token by
    token block."""

    def __init__(self, batch, heads, capacity, dim):
        self.codes = np.zeros((2, batch, heads, capacity, dim), np.uint8)
        self.exps = np.zeros((2, batch, heads, capacity // TOKENS), np.uint8)
        self.lens = np.zeros(batch, np.int64)

    def store(self, k, v, start=None, counts=None):
        B, n = k.shape[:2]
        cap = self.codes.shape[3]
        for b in range(B):
            p = int(self.lens[b] if start is None else start[b])
            c = int(n if counts is None else counts[b])
            if not (0 <= p <= self.lens[b] and 0 <= c <= n and p + c <= cap):
                continue
            for w, x in enumerate((k, v)):
                lo = p
                while lo < p + c:
                    blk = lo // TOKENS
                    hi = min((blk + 1) * TOKENS, p + c)
                    part = np.moveaxis(x[b, lo - p:hi - p], 0, 1)  # [H][tokens][D]
                    e = exponent(np.abs(part).max((1, 2)))
                    codes = self.codes[w, b]
                    if lo > blk * TOKENS:
                        old = self.exps[w, b, :, blk].astype(np.int64) - 127
                        e = np.maximum(e, old)
                        held = value_of(codes[:, blk * TOKENS:lo]) * np.exp2((old - e).astype(np.float64))[:, None, None]
                        codes[:, blk * TOKENS:lo] = code_of(np.copysign(nearest_e4m3(held), held))
                    g = part * np.exp2(-e.astype(np.float64))[:, None, None]
                    codes[:, lo:hi] = code_of(np.copysign(nearest_e4m3(g), g))
                    self.exps[w, b, :, blk] = e + 127
                    lo = hi
            self.lens[b] = p + c

    def values(self, w, b, h):
        n = int(self.lens[b])
        unit = np.exp2(self.exps[w, b, h].astype(np.float64) - 127).repeat(TOKENS)[:n, None]
        return value_of(self.codes[w, b, h, :n]) * unit


def visible(n, nq, causal, window, sinks):
    j = np.arange(n)[None]
    p = (n - nq + np.arange(nq) if causal else np.full(nq, n - 1))[:, None]
    see = j <= p
    if window:
        see &= (p - j < window) | (j < sinks)
    return see


def attention(cache, q, nqs, scale, causal=False, window=0, sinks=0):
    """FP64 (out, lse, bound of out, bound of lse); q [B][n][Hq][D] FP64. The bounds are those of a
    kernel that keeps sums in FP32, rounds softmax weights to fp16 and the output to bf16:
      scores    every product is exact, D of them are summed in FP32 (2^-22 of the sum of magnitudes a
                step allows for truncating adders), then one scaling and exp2 (each 2^-22 of the score
                in powers of two): err_s absolute, a relative error of each weight;
      weights   2^-11 (fp16, half a step), and 2^-25 of the row's largest weight at the subnormal end,
                for as many keys as there are;
      sums      n terms in FP32, 2^-22 relative a chunk of 32: below 2^-12 for the lengths tested;
      output    2^-8 of the value (bf16, half a step of 2^-7)."""
    B, n, Hq, D = q.shape
    H = cache.codes.shape[2]
    out, lse = np.zeros(q.shape), np.full((B, Hq, n), -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros((B, Hq, n))
    for b in range(B):
        see = visible(int(cache.lens[b]), int(nqs[b]), causal, window, sinks)
        for h in range(Hq):
            k, v = cache.values(0, b, h // (Hq // H)), cache.values(1, b, h // (Hq // H))
            r = int(nqs[b])
            x = np.where(see, q[b, :r, h] @ k.T * scale, -np.inf)
            mag = np.where(see, np.abs(q[b, :r, h]) @ np.abs(k).T * scale, 0.0)
            if x.shape[1] == 0 or r == 0:
                continue
            top = x.max(1, keepdims=True)
            live = np.isfinite(top[:, 0])
            w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            tot = w.sum(1, keepdims=True)
            tot1 = np.where(tot > 0, tot, 1)
            out[b, :r, h] = w @ v / tot1
            with np.errstate(divide="ignore"):
                lse[b, h, :r] = np.where(live, top[:, 0] + np.log(tot[:, 0]), -np.inf)
            # the score error matters where the weight does: weights beyond 2^-40 of the largest are lost
            near = see & (x > top - 28)
            err = np.where(near, mag, 0.0).max(1) * (D / 16) * 2.0 ** -22 + np.where(near, np.abs(x), 0).max(1, initial=0) * 2.0 ** -21 + 2.0 ** -20
            a = w @ np.abs(v) / tot1
            vmax = np.abs(v).max(0)[None] if len(v) else 0.0
            tol[b, :r, h] = (2.0 ** -8 * np.abs(out[b, :r, h]) + (2.0 ** -11 + 2.0 ** -12 + 2 * err[:, None]) * a
                             + 2.0 ** -25 * see.sum(1)[:, None] * vmax / tot1 + 1e-30)
            ltol[b, h, :r] = err + 2.0 ** -12 * 0.01 + np.abs(np.where(live, lse[b, h, :r], 0.0)) * 2.0 ** -22
    return out, lse, tol, ltol
