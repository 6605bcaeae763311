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
