"""Sampling at the ends of its settings' ranges, and next to the borders of heavy tokens."""

import math

import numpy as np
import pytest
import torch

import serve_ref as ref
from speculative_decoding_head_gb300.binding import Sampler

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
