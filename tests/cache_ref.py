"""Plain CPU implementation of the 4-bit K/V cache and of attention over it.

The stored values follow include/fa.h step by step in numpy float32 (the
header fixes that precision for the division); attention is in float64 and
comes with bounds on the rounding errors of the library's kernels:

  * P s, the weight of a group's codes, is rounded to f16: half a step is
    2^-11 of the value (2^-25 absolute below f16's normal range, where the
    largest weight of the row is at least 1), on codes 0 .. 15;
  * a score is a sum of d products in fp32 (one rounding each, at most 2^-23
    with the chopped adds of a matrix unit) of |q| (lo + 15 s), scaled; an
    absolute error e of a score is a relative error of about e of p, and the
    approximate exponential adds 2^-21;
  * the result is rounded to the output's type: half a step, eps / 2.

With more than 64 query rows a K/V head there is another kernel, for some of the
sizes, and the bound is the larger one. In it V and P are f16 operands of the tensor
cores: half a step is 2^-11 of each value (of V, scaled by a power of two to below 2^8
a tile of keys, 2^-25 below f16's normal range, so 2^-32 of the tile's largest; of P,
whose largest is at least 1, 2^-25). K is the middle of a group, lo + 8 s, and
s (u - 8), which is exact but below f16's normal range (2^-31 of the tile's largest);
the middle and the sums of q that it meets have two f16 terms each, 2^-21 of the
product in all.
"""
import numpy as np
import torch

GROUP = 32


def quantise(x):
    """(u, s, lo) of 16-bit rows x [..., d]: int64 codes and float32 s, lo [..., d / 32]."""
    dt = x.dtype
    y = x.float().numpy().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = y.min(-1), y.max(-1)
        s32 = (hi - lo) / np.float32(15)
        s = torch.from_numpy(s32).to(dt).float().numpy()
        bad = ~np.isfinite(y).all(-1) | ~np.isfinite(s)
        safe = np.where((s > 0) & ~bad, s, np.float32(1))
        u = np.minimum(np.rint((y - lo[..., None]) / safe[..., None]), np.float32(15))
    u = np.where(((s > 0) & ~bad)[..., None], u, 0).astype(np.int64)
    nan = np.float32(np.nan)
    return u, np.where(bad, nan, s), np.where(bad, nan, lo)


def stands_for(x):
    """float64 values that the cache stands for after 16-bit rows x were written."""
    u, s, lo = quantise(x)
    y = lo.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * u
    return y.reshape(x.shape)


def read_back(x):
    """What cache_read returns: lo + s u in fp32 (s u is exact), rounded to the type."""
    u, s, lo = quantise(x)
    y = lo[..., None] + s[..., None] * u.astype(np.float32)
    return torch.from_numpy(y.astype(np.float32).reshape(x.shape)).to(x.dtype)


def attend(q, k, v, n, causal, scale, out_eps):
    """Attention of one sequence and the error bounds of its outputs.

    q: 16-bit [Hq, Nq, d] of which rows i < n are the last n tokens; k, v: the
    16-bit rows [Hk, len, d] as they were written. Returns float64 O, LSE and
    the bounds on |O - computed|, |LSE - computed|.
    """
    Hq, Nq, d = q.shape
    Hk, L, _ = k.shape
    f16_operands = Hq // Hk * Nq > 64  # possibly
    O, lse = np.zeros((Hq, Nq, d)), np.full((Hq, Nq), -np.inf)
    tO, tl = np.zeros((Hq, Nq, d)), np.zeros((Hq, Nq))
    for h in range(Hk):
        kd, vd = stands_for(k[h]), stands_for(v[h])
        _, ks, klo = quantise(k[h])
        _, vs, vlo = quantise(v[h])
        kmag = np.repeat(np.abs(klo) + 15 * ks, GROUP, -1).astype(np.float64)
        vstep = 15 * np.repeat(vs, GROUP, -1).astype(np.float64)
        for hq in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
            qd = q[hq].double().numpy()
            for i in range(min(n, Nq)):
                m = min(L, max(L - n + i + 1, 0)) if causal else L
                if m == 0:
                    continue
                z = scale * (kd[:m] @ qd[i])
                e = scale * 2.0 ** -23 * (d + 8) * (kmag[:m] @ np.abs(qd[i]))
                top = z.max()
                p = np.exp(z - top)
                l = p.sum()
                p /= l
                O[hq, i] = p @ vd[:m]
                lse[hq, i] = top + np.log(l)
                rel = 2 * e.max() + 2.0 ** -20 + m * 2.0 ** -24  # of p / l
                w = (p[:, None] * vstep[:m])
                tO[hq, i] = (2.0 ** -11 * w.sum(0) + m * 2.0 ** -25 * w.max() +
                             2 * rel * (p @ (np.abs(vd[:m]) + 2 * vstep[:m])))
                if f16_operands:
                    av = np.abs(vd[:m])
                    ek = scale * ((2.0 ** -21 * kmag[:m] + 2.0 ** -30 * kmag[:m].max()) @
                                  np.abs(qd[i])).max()
                    rel += 2 * ek
                    tl[hq, i] = ek
                    tO[hq, i] = np.maximum(
                        tO[hq, i],
                        2 * 2.0 ** -11 * (p @ av) + m * 2.0 ** -24 * p.max() * av.max() +
                        2.0 ** -32 * av.max() + 2 * rel * (p @ av))
                tO[hq, i] += out_eps / 2 * (np.abs(O[hq, i]) + tO[hq, i])
                tl[hq, i] += e.max() + 2.0 ** -20 + m * 2.0 ** -24 + 2.0 ** -22 * abs(lse[hq, i])
    return O, lse, tO, tl
