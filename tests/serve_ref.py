"""Plain 64-bit forms of the 4-bit matrices and of sampling, for the tests (numpy, row by row)."""

import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 512.0 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def nearest(x, grid):
    """Members of a grid of magnitudes nearest to x; of two as near, the one at an even place; at most the last."""
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    i = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.copysign(grid[i], x)


def fp4(x, fmt):
    """(values, scales times factors [R, blocks], row factors) of x [R, K], by the formats' definition; NaN blocks."""
    x = x.detach().cpu().double().numpy()
    R, K = x.shape
    B = BLOCK[fmt]
    nb = -(-K // B)
    v = np.zeros((R, nb * B))
    v[:, :K] = x
    v = v.reshape(R, nb, B)
    top = np.abs(v).max(2)
    bad = ~np.isfinite(v).all(2)
    top = np.where(bad, 0.0, top)
    f = np.ones(R)
    if fmt == "nvfp4":
        for r in range(R):
            m = top[r].max()
            if m > 0:
                e = math.floor(math.log2(m / 2688.0)) - 1
                while m > 2688.0 * 2.0 ** e:
                    e += 1
                f[r] = 2.0 ** max(e, -100)
        scale = nearest(top / f[:, None] / 6.0, E4M3) * f[:, None]
    else:
        scale = np.empty_like(top)
        for i, m in np.ndenumerate(top):
            scale[i] = 2.0 ** max(-127, math.frexp(m)[1] - 3) if m > 0 else 2.0 ** -127
    scale = np.abs(scale)
    q = nearest(np.where(bad[..., None], 0.0, v) / np.where(scale == 0, 1.0, scale)[..., None], E2M1)
    out = q * scale[..., None]
    out[bad] = np.nan
    return out.reshape(R, -1)[:, :K], np.where(bad, np.nan, scale), f


def row_distribution(z, T=1.0, k=0, p=1.0, mp=0.0):
    """(kept mask, masses) of one row of logits, by sorting."""
    z = z.detach().cpu().double().numpy()
    z = np.where(z <= -1e29, -np.inf, z)
    T, k, p, mp = float(T), int(k), float(p), float(mp)
    if T == 0.0:
        T, k = 1.0, 1
    top = z.max()
    kept = z > -np.inf
    if top == -np.inf:
        return kept, np.zeros_like(z)
    with np.errstate(over="ignore"):
        w = np.exp((z - top) / T)
    order = np.lexsort((np.arange(z.size), -z))
    n = int(kept.sum())
    if 0 < k < n:
        kept[order[k:]] = False
        n = k
    if p < 1.0:
        ws = w[order[:n]]
        before = np.cumsum(ws) - ws
        out = before >= p * ws.sum()
        out[0] = False
        kept[order[:n][out]] = False
    if mp > 0.0:
        kept &= z - top >= T * math.log(mp)
    return kept, w


def row_sample(z, u, **how):
    """(token, its log-probability, how near the draw came to a token's border, in parts of the mass)."""
    kept, w = row_distribution(z, **how)
    if not kept.any():
        return -1, -math.inf, 1.0
    c = np.cumsum(np.where(kept, w, 0.0))
    t = int(np.searchsorted(c, float(u) * c[-1], side="right"))
    return t, math.log(w[t] / c[-1]), float(np.abs(c / c[-1] - float(u)).min())


def row_logprobs(z, T=1.0, **how):
    kept, w = row_distribution(z, T=T, **how)
    out = np.full(w.shape, -np.inf)
    if kept.any():
        zz = z.detach().cpu().double().numpy()
        out[kept] = (zz[kept] - zz[kept].max()) / (float(T) or 1.0) - math.log(w[kept].sum())
    return out


def settings(kind, n, g):
    """temperature, top_k, top_p, min_p vectors of n entries on the generator's device (None where unused)."""
    dev = g.device

    def uni(lo, hi):
        return torch.rand(n, generator=g, device=dev) * (hi - lo) + lo

    k = torch.randint(1, 60, (n,), generator=g, device=dev, dtype=torch.int32)
    return {"none": (None, None, None, None), "t": (uni(0.3, 2.0), None, None, None), "k": (None, k, None, None),
            "p": (uni(0.5, 1.5), None, uni(0.05, 0.999), None), "kp": (uni(0.5, 1.5), k, uni(0.05, 0.999), None),
            "minp": (uni(0.5, 1.5), None, None, uni(0.001, 0.5)),
            "all": (uni(0.5, 1.5), k, uni(0.5, 0.999), uni(0.001, 0.1)),
            "greedy": (torch.zeros(n, device=dev), k, uni(0.05, 0.999), uni(0.001, 0.5))}[kind]
