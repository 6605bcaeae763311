"""Rounds of a head server with vocabularies of any size, and with requests that cannot be verified."""

import numpy as np
import pytest
import torch

import oracle
from parity import compare_verify, gpu_np
from speculative_decoding_head_gb300.serve_head import Chain, HeadServer

pytestmark = pytest.mark.gpu


def server(B, gamma, V, H, r, seed=0, dtype=torch.float32, mode="static"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    chain = Chain(V, H, g, sharp=0.6)
    W1 = torch.empty(V, r, device="cuda").normal_(0.0, 0.05, generator=g).to(dtype)
    W2 = torch.empty(r, V, device="cuda").normal_(0.0, 0.05, generator=g).to(dtype)
    w = torch.empty(H + r, device="cuda").normal_(0.0, 0.05, generator=g)
    sps = torch.full((1 + B * (gamma + 1),), 400.0, dtype=torch.float64, device="cuda")
    return chain, HeadServer(B, gamma, chain.W_out, W1, W2, w, mode=mode), sps, g


@pytest.mark.parametrize("V", [4099, 50257, 4102, 997])
def test_vocabularies_of_any_size(V):
    """With W1 and W2 in fp32 (bf16 ones want a multiple of 8)."""
    B, gamma, H, r = 6, 3, 100, 48
    chain, s, sps, g = server(B, gamma, V, H, r, seed=V)
    p = torch.full((B,), 0.9, device="cuda")
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    for rnd in range(2):
        d = s.draft(chain.draft_hidden(anchor, gamma, 0.5), anchor, sps, 5, rnd)
        v = s.verify(chain.target_hidden(anchor, d), anchor, d, 5, rnd, top_p=p)
        assert s.device_status() == 0
        ro = d["row_off"].cpu().numpy()
        o = oracle.verify(s.Q[:ro[-1]].cpu().numpy(), ro, d["lengths"].cpu().numpy(), anchor.cpu().numpy(),
                          d["tokens"].cpu().numpy(), s.U.view(B, gamma, V).cpu().numpy(), s.W1.cpu().numpy(),
                          s.W2.cpu().numpy(), 5, rnd)
        compare_verify(gpu_np(v), o, range(B)).check_rate()
        anchor = v["next_anchor"]


# the draft's two paths, and each of the verify's sweeps
@pytest.mark.parametrize("V,dtype", [(4096, torch.bfloat16), (16384, torch.bfloat16), (4099, torch.float32)])
@pytest.mark.parametrize("mode", ["static", "compact"])
@pytest.mark.parametrize("bad", ["temperature", "hidden"])
def test_a_round_with_a_request_that_cannot_be_verified(bad, mode, V, dtype):
    """The status says so, the anchors that come out are ids of the vocabulary all the same (what a caller looks up
    next), and after a reset rounds are what they were."""
    B, gamma = 8, 3
    chain, s, sps, g = server(B, gamma, V, 128, 64, seed=2, dtype=dtype, mode=mode)
    T = torch.full((B,), 0.8, device="cuda")
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    h = chain.draft_hidden(anchor, gamma, 0.5)
    d = s.draft(h, anchor, sps, 1, 0)
    ht = chain.target_hidden(anchor, d)
    want = {k: t.clone() for k, t in (*d.items(), *s.verify(ht, anchor, d, 1, 0, temperature=T).items())}
    assert s.device_status() == 0
    broken, hb = T.clone(), ht.clone()
    if bad == "temperature":
        broken[3] = float("nan")
    else:
        hb[int(d["row_off"][3]):int(d["row_off"][4])] = float("nan")
    junk = [torch.full((B,), 123456789, device="cuda", dtype=torch.int32) for _ in range(8)]
    del junk  # what new outputs of this size are likely made of
    for _ in range(2):  # and in a round after it, without a reset
        v = s.verify(hb, anchor, d, 1, 0, temperature=broken)
        assert s.device_status() != 0
        assert ((v["next_anchor"] >= 0) & (v["next_anchor"] < V)).all()
        assert ((v["n_acc"] >= -1) & (v["n_acc"] <= gamma)).all() and int(v["n_acc"][3]) == -1
    s.reset()
    assert s.device_status() == 0
    d = s.draft(h, anchor, sps, 1, 0)
    got = {**d, **s.verify(ht, anchor, d, 1, 0, temperature=T)}
    assert s.device_status() == 0 and all(torch.equal(got[k], want[k]) for k in want)
