"""Attention over the 8-bit cache in FP64, with error bounds that count each key by its own weight: what a
key that gets no weight holds, and how long the cache is, loosens nothing."""
import numpy as np

from ref8 import TOKENS, value_of, visible


def attention(cache, q, nqs, scale, causal=False, window=0, sinks=0, gain=32):
    """(out, lse, bound of out, bound of lse) of q [B][n][Hq][D] FP64 over a ref8.Cache. Rows that see nothing
    give 0 and -inf. The bounds are those of this arithmetic, per key j with weight p_j (sum 1):

      e_j  relative error of a weight: products are exact, D of them are summed in FP32 by adders that may
           truncate (D / 16 steps of 2^-22 of the sum of magnitudes), the score is scaled once and its
           exponent is rounded with the block's own (2^-21 of both, in nats), exp2 adds 2^-20; times 1.1
           for what is of second order;
      2^-11  the weight in fp16, half a step; and `sub`: weights times their block's scale are rounded relative
           to the row's largest such product P, so one below 2^-gain P may be lost whole, and one below
           2^(11 - gain) P is off by at most 2^-gain P. A block of zeros has no scale of its own; it stands with
           at most 2^-64 of the largest, because sums of weights are held within 2^64 of one another;
      2^-12  FP32 sums: at most 1024 steps into one accumulator, 2^-22 each;
      2^-8   the bf16 output, half a step, and 2^-133 below its normal range.

    The row sum has FP32 weights, so its error is sum p_j e_j + 2^-12 of itself at most."""
    B, n, Hq, D = q.shape
    H = cache.codes.shape[2]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, ltol = np.full((B, Hq, n), -np.inf), np.zeros((B, Hq, n))
    for b in range(B):
        r, held = int(nqs[b]), int(cache.lens[b])
        if r == 0 or held == 0:
            continue
        see = visible(held, r, causal, window, sinks)
        for h in range(Hq):
            kh = h // (Hq // H)
            k, v = cache.values(0, b, kh), cache.values(1, b, kh)
            ev = (cache.exps[1, b, kh].astype(np.float64) - 127).repeat(TOKENS)[:held][None]
            code = np.abs(value_of(cache.codes[1, b, kh, :held]))
            x = np.where(see, q[b, :r, h] @ k.T * scale, -np.inf)
            top = x.max(1, keepdims=True)
            live = np.isfinite(top)
            top = np.where(live, top, 0.0)
            w = np.exp(x - top)
            tot = w.sum(1, keepdims=True)
            tot1 = np.where(tot > 0, tot, 1.0)
            p = w / tot1
            mag = np.abs(q[b, :r, h]) @ np.abs(k).T * scale
            xs = np.where(see, np.abs(x), 0.0)
            e = 1.1 * (mag * (D / 16) * 2.0 ** -22 + (xs + np.log(2) * np.abs(ev)) * 2.0 ** -21 + 2.0 ** -20)
            e = np.where(p > 0, e, 0.0)
            out[b, :r, h] = p @ v
            lse[b, h, :r] = np.where(live, top + np.log(tot1), -np.inf)[:, 0]
            zeros = ~(np.add.reduceat(code.sum(1), np.arange(0, held, TOKENS)) > 0).repeat(TOKENS)[:held][None]
            scale2 = np.where(zeros, np.maximum(ev, ev.max() - 64), ev)
            prod = np.where(see, (x - top) / np.log(2) + scale2, -np.inf)  # log2 of weight times scale
            P = prod.max(1, keepdims=True)
            lost = see & (prod < P - gain)
            part = see & ~lost & (prod < P - gain + 11)
            Pt = np.exp2(np.where(live, P, 0.0) - gain) / tot1
            err = (p * e).sum(1, keepdims=True)
            tol[b, :r, h] = (2.0 ** -8 * np.abs(out[b, :r, h]) + (p * (e + 2.0 ** -11 + 2.0 ** -12)) @ np.abs(v)
                             + np.abs(out[b, :r, h]) * (err + 2.0 ** -12)
                             + np.where(lost, p, 0.0) @ np.abs(v) + Pt * (part.astype(np.float64) @ code) + 2.0 ** -133)
            ltol[b, h, :r] = np.where(live, err + 2.0 ** -12 * 0.01 + (np.where(live, np.abs(top), 0.0) + np.log(tot1)
                                      + np.log(2) * np.abs(ev).max()) * 2.0 ** -21, 0.0)[:, 0]
    return out, lse, tol, ltol
