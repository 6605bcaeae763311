"""Sampling at the ends of its settings' ranges, and next to the borders of heavy tokens."""

import math

import numpy as np
import pytest
import torch

import serve_ref as ref
from speculative_decoding_head_gb300.binding import Sampler
from test_gpu_sample import check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("k", [None, 5, 2000])  # a search for masses, a short list, both searches
@pytest.mark.parametrize("V", [3, 700, 40000, 800001])
def test_negative_zero_is_zero(V, k, dtype):
    """top-p, u, min-p and the temperature may be -0."""
    N = 6
    z = torch.empty(N, V, device="cuda").normal_(0.0, 2.0, generator=gen(V)).to(dtype)
    full = lambda v, t=F32: torch.full((N,), v, device="cuda", dtype=t)  # noqa: E731
    s, zero, minus = Sampler(N, V), full(0.0), -full(0.0)
    assert (minus.view(torch.int32) == -2 ** 31).all()
    kk = None if k is None else full(k, torch.int32)

    def both(u, **how):
        out = {"token": full(-7, torch.int32), "logp": full(9.0)}
        return (*s.sample(z, u, top_k=kk, out=out, **how).values(), s.logprobs(z, top_k=kk, **how))

    u = torch.rand(N, generator=gen(1), device="cuda")
    p = full(0.9)
    for want, got in ((both(zero), both(minus)), (both(zero, top_p=p), both(minus, top_p=p)),
                      (both(u, top_p=zero), both(u, top_p=minus)), (both(zero, top_p=zero), both(minus, top_p=minus)),
                      (both(u, min_p=zero), both(u, min_p=minus)), (both(u, temperature=zero), both(u, temperature=minus))):
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert (got[0] >= 0).all()
    top = z.float().max(1)[0]
    tok, logp, lp = both(u, top_p=minus)  # the first token of the largest logit alone
    first = (z.float() == top[:, None]).float().argmax(1)
    assert torch.equal(tok.long(), first) and (logp == 0).all() and (torch.isfinite(lp).sum(1) == 1).all()
    assert s.device_status() == 0


def test_temperatures_that_count_as_the_least():
    """Above 0 and below 1e-30 a temperature is 1e-30; 0 alone is greedy."""
    V, N = 3000, 6
    z = torch.linspace(0, 4e-29, V, device="cuda").repeat(N, 1)
    z[1:] += torch.empty(N - 1, V, device="cuda").normal_(0.0, 1e-30, generator=gen(2))
    u = torch.rand(N, generator=gen(3), device="cuda")
    full = lambda v, t=F32: torch.full((N,), v, device="cuda", dtype=t)  # noqa: E731
    s = Sampler(N, V)
    for how in ((None, None, None), (None, full(0.9), None), (full(40, torch.int32), full(0.8), None), (None, None, full(0.3))):
        check(z, (full(1e-30), *how), u)
        kw = dict(zip(("top_k", "top_p", "min_p"), how))
        want = (*s.sample(z, u, temperature=full(1e-30), **kw).values(), s.logprobs(z, temperature=full(1e-30), **kw))
        for T in (1e-31, 1e-38, 2.0 ** -149):
            got = (*s.sample(z, u, temperature=full(T), **kw).values(), s.logprobs(z, temperature=full(T), **kw))
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        greedy = s.sample(z, u, temperature=full(0.0), **kw)
        assert torch.equal(greedy["token"].long(), z.argmax(1)) and (greedy["logp"] == 0).all()
    assert s.device_status() == 0


def beside(border, tol):
    """The largest fp32 numbers at or below border - tol and the least ones at or above border + tol (float64 arrays)."""
    lo, hi = (border - tol).astype(np.float32), (border + tol).astype(np.float32)
    lo = np.where(lo > border - tol, np.nextafter(lo, np.float32(0)), lo)
    hi = np.where(hi < border + tol, np.nextafter(hi, np.float32(1)), hi)
    return lo, hi


# A token's mass is off by 2^-26.5 of itself at the most: with w = r ln(2) / 32 < 2^-4.9 the two roundings of r
# are off by 2^-29.5 each, the two last ones of the polynomial, of its product with the table's entry and of the entry by
# 2^-28.9 each, the whole number by 2^-31. So a border at a share b of the mass, between tokens that are off to different
# sides, is off by b (1 - b) 2^-25.5, and by some units of 2^-46 of the maximum's mass. (fp32 settings lie 2^-24 apart.)
def tolerance(b):
    return b * (1 - b) * 2.0 ** -25.5 + 2.0 ** -40


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heavy,each", [(2, 1), (3, 1), (3, 300), (2, 5000)])  # some values, the tokens that have each
def test_borders_of_heavy_tokens(heavy, each, dtype):
    """u and top-p on both sides of a border of few heavy tokens, and of many that share few logits (and so their errors)."""
    N = 4096 if each == 1 else 256
    V, g = heavy * each, gen(heavy * each)
    z = torch.empty(N, heavy, device="cuda").normal_(0.0, 1.5, generator=g).to(dtype)
    T = torch.rand(N, generator=g, device="cuda") * 1.7 + 0.3
    zz, t = z.double().cpu().numpy(), T.double().cpu().numpy()
    w = np.exp((zz - zz.max(1, keepdims=True)) / t[:, None])
    z = z.repeat_interleave(each, 1)  # the tokens of one value are neighbours
    w = np.repeat(w, each, 1)
    c = np.cumsum(w, 1)
    S, rows = c[:, -1:], np.arange(N)
    s = Sampler(N, V)
    for at in (np.full(N, (V - 1) // 2), np.full(N, V - 2), np.random.default_rng(V).integers(0, V - 1, N)):
        b = (c / S)[rows, at]
        for u, side in zip(beside(b, tolerance(b)), (0, 1)):
            # the token that 64 bits draw: far from a border of theirs but for this one's
            x = u.astype(np.float64)
            clear = np.abs(c / S - x[:, None]) >= (tolerance(c / S) * (np.arange(V) != at[:, None]))
            fine = clear.all(1) & (x >= 0) & (x < 1)
            want = (c <= x[:, None] * S).sum(1)
            # u lies on the side that is meant, but where a token beside the border has less than u's own step
            assert fine.sum() > N // 2 and (want[fine] == at[fine] + side).mean() > 0.9
            got = s.sample(z, torch.from_numpy(np.where(fine, u, 0.5).astype(np.float32)).cuda(), temperature=T)["token"]
            assert np.array_equal(got.cpu().numpy()[fine], want[fine])
    # top-p: a token is kept while what comes before it is less than p of the mass
    order = np.argsort(-w, 1, kind="stable")
    ws = np.take_along_axis(w, order, 1)
    c = np.cumsum(ws, 1)
    for at in (np.zeros(N, int), np.full(N, (V - 1) // 2), np.full(N, V - 2)):
        b = (c / S)[rows, at]
        for p in beside(b, tolerance(b)):
            x = p.astype(np.float64)
            clear = np.abs(c / S - x[:, None]) >= (tolerance(c / S) * (np.arange(V) != at[:, None]))
            fine = clear.all(1) & (x > 0) & (x < 1)
            want = ((c - ws) < x[:, None] * S).sum(1)
            got = s.logprobs(z, temperature=T, top_p=torch.from_numpy(np.where(fine, p, 0.5).astype(np.float32)).cuda())
            assert np.array_equal(torch.isfinite(got).sum(1).cpu().numpy()[fine], want[fine])
