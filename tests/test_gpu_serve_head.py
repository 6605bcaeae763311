"""Rounds with a 4-bit output layer and sampling settings, the operators together as they are used."""

import numpy as np
import pytest
import torch

import oracle
import serve_ref as ref
from parity import compare_verify, gpu_np
from speculative_decoding_head_gb300.binding import DsparkError, Sampler, Workspace
from speculative_decoding_head_gb300.serve_head import Chain, HeadServer
from speculative_decoding_head_gb300.workloads import bf16_bits

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def server(B, gamma, V, H, r, fmt="nvfp4", seed=0, mode="static"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    chain = Chain(V, H, g, sharp=0.6)
    W1 = torch.empty(V, r, device="cuda").normal_(0.0, 0.05, generator=g).to(BF16)
    W2 = torch.empty(r, V, device="cuda").normal_(0.0, 0.05, generator=g).to(BF16)
    w = torch.empty(H + r, device="cuda").normal_(0.0, 0.05, generator=g)
    sps = torch.full((1 + B * (gamma + 1),), 400.0, dtype=torch.float64, device="cuda")
    return chain, HeadServer(B, gamma, chain.W_out, W1, W2, w, fmt=fmt, mode=mode), sps, g


@pytest.mark.parametrize("V", [4104, 8192, 16384])  # three of the verify's sweeps
@pytest.mark.parametrize("kind", ["none", "k", "p", "all", "greedy"])
def test_rounds_against_the_oracle(kind, V):
    B, gamma, H, r = 12, 3, 256, 64
    chain, s, sps, g = server(B, gamma, V, H, r, "nvfp4" if V != 8192 else "mxfp4", seed=V,
                              mode="compact" if V == 8192 else "static")
    how = dict(zip(("temperature", "top_k", "top_p", "min_p"), ref.settings(kind, B, g)))
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    for rnd in range(3):
        d = s.draft(chain.draft_hidden(anchor, gamma, 0.5), anchor, sps, 5, rnd)
        ht = chain.target_hidden(anchor, d)
        v = s.verify(ht, anchor, d, 5, rnd, **how)
        torch.cuda.synchronize()
        assert s.device_status() == 0
        # U and P are the products of what the 4 bits stand for: |error| at most 2^-20 of the terms' magnitudes
        Wv = s.layer.lookup(dtype=torch.float32).double()
        Hv = s.hidden.lookup(dtype=torch.float32).double()
        assert ((s.U.double() - Hv @ Wv.t()).abs() <= 2.0 ** -20 * (Hv.abs() @ Wv.abs().t()) + 1e-30).all()
        ro, L = d["row_off"].cpu().numpy(), d["lengths"].cpu().numpy()
        Q, P = s.Q[:ro[-1]].cpu(), s.P[:ro[-1]].cpu()
        for b in (0, B - 1):
            one = {a: float(t[b]) for a, t in zip(("T", "k", "p", "mp"), how.values()) if t is not None}
            for n in range(ro[b], ro[b + 1]):
                assert np.array_equal(np.isfinite(ref.row_logprobs(P[n], **one)), np.isfinite(Q[n].numpy()))
        o = oracle.verify(Q.numpy(), ro, L, anchor.cpu().numpy(), d["tokens"].cpu().numpy(),
                          s.U.view(B, gamma, V).cpu().numpy(), bf16_bits(s.W1).cpu().numpy().view(np.uint16),
                          bf16_bits(s.W2).cpu().numpy().view(np.uint16), 5, rnd)
        compare_verify(gpu_np(v), o, range(B)).check_rate()
        # what was emitted is kept in its row
        n_acc, nxt, tok = v["n_acc"].cpu().numpy(), v["next_anchor"].cpu().numpy(), d["tokens"].cpu().numpy()
        for b in range(B):
            for j in range(n_acc[b]):
                assert np.isfinite(Q[ro[b] + j, tok[b, j]])
            assert np.isfinite(Q[ro[b] + n_acc[b], nxt[b]])
        anchor = v["next_anchor"]


def test_without_settings_a_round_is_the_plain_one():
    B, gamma, V = 24, 4, 8192
    chain, s, sps, g = server(B, gamma, V, 256, 64)
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    d = s.draft(chain.draft_hidden(anchor, gamma, 0.5), anchor, sps, 1, 0)
    v = s.verify(chain.target_hidden(anchor, d), anchor, d, 1, 0)
    plain = s.ws.verify(s.P, d["row_off"], d["lengths"], anchor, d["tokens"], d["pd_tok"], d["lse"], s.U, s.W1, s.W2, 1, 0)
    ro = d["row_off"].cpu().numpy()
    o = oracle.verify(s.P[:ro[-1]].cpu().numpy(), ro, d["lengths"].cpu().numpy(), anchor.cpu().numpy(),
                      d["tokens"].cpu().numpy(), s.U.view(B, gamma, V).cpu().numpy(), bf16_bits(s.W1).cpu().numpy().view(np.uint16),
                      bf16_bits(s.W2).cpu().numpy().view(np.uint16), 1, 0)
    close = np.minimum(o["acc_margin"], o["smp_margin"]) < oracle.MARGIN
    assert (((v["n_acc"] == plain["n_acc"]) & (v["next_anchor"] == plain["next_anchor"])).cpu().numpy() | close).all()


def test_hidden_states_behind_the_last_row_are_not_looked_at():
    B, gamma, V = 24, 4, 8192
    chain, s, sps, g = server(B, gamma, V, 256, 64, mode="compact")
    sps = 400.0 / (1.0 + 0.2 * torch.arange(sps.numel(), dtype=torch.float64, device="cuda"))  # short lengths pay
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    d = s.draft(chain.draft_hidden(anchor, gamma, 0.5), anchor, sps, 1, 0)
    ht, last = chain.target_hidden(anchor, d), int(d["row_off"][B])
    assert last < B * (gamma + 1)
    want = {k: t.clone() for k, t in s.verify(ht, anchor, d, 1, 0).items()}
    ht[last:] = float("nan")
    got = s.verify(ht, anchor, d, 1, 0)
    assert s.device_status() == 0
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_emitted_tokens_follow_the_settings():
    """The first token of a round has the processed distribution whatever the draft: chi-squared over the
    kept tokens of one row (at most 20, so 19 degrees of freedom; the value 80 has a probability below 1e-8)."""
    B, V, r, rounds = 4096, 256, 16, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty(V, device="cuda").normal_(0.0, 2.0, generator=g)
    u = z + torch.empty(V, device="cuda").normal_(0.0, 1.0, generator=g)
    W1, W2 = torch.zeros(V, r, device="cuda"), torch.zeros(r, V, device="cuda")
    ws = Workspace(B, 1, V, r, 0, "f32", "static")
    U = u.expand(B, 1, V).contiguous()
    how = dict(temperature=torch.full((B,), 0.9, device="cuda"), top_k=torch.full((B,), 20, device="cuda", dtype=torch.int32),
               top_p=torch.full((B,), 0.85, device="cuda"))
    anchor = torch.zeros(B, dtype=torch.int32, device="cuda")
    s = Sampler(2 * B, V, requests=B)
    one = torch.ones(1, device="cuda")
    sps = torch.full((1 + 2 * B,), 400.0, dtype=torch.float64, device="cuda")
    seen = torch.zeros(V, dtype=torch.int64, device="cuda")
    P = z.expand(2 * B, V).contiguous()
    for rnd in range(rounds):
        d = ws.draft(U, W1, W2, anchor, torch.empty(B, 1, 0, device="cuda"), torch.zeros(r, device="cuda"), one, 7, rnd)
        p = ws.plan(d["conf"], sps)
        Q = s.logprobs(P, row_off=p["row_off"], **how)
        v = ws.verify(Q, p["row_off"], p["lengths"], anchor, d["tokens"], d["pd_tok"], d["lse"], U, W1, W2, 7, rnd)
        first = torch.where(v["n_acc"] > 0, d["tokens"][:, 0], v["next_anchor"])
        seen += torch.bincount(first.long(), minlength=V)
    assert ws.device_status() == 0 and s.device_status() == 0
    kept, w = ref.row_distribution(z, T=float(how["temperature"][0]), k=20, p=float(how["top_p"][0]))
    want = np.where(kept, w, 0.0) / w[kept].sum() * B * rounds
    have = seen.double().cpu().numpy()
    assert have[~kept].sum() == 0 and kept.sum() > 3
    assert ((have[kept] - want[kept]) ** 2 / want[kept]).sum() < 80


def test_a_finite_fill_verifies_the_same():
    B, gamma, V = 16, 3, 4104
    chain, s, sps, g = server(B, gamma, V, 128, 64, seed=9)
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.full((B,), 0.8, device="cuda")
    d = s.draft(chain.draft_hidden(anchor, gamma, 0.5), anchor, sps, 1, 0)
    v = s.verify(chain.target_hidden(anchor, d), anchor, d, 1, 0, top_p=p)
    Q = s.sampler.logprobs(s.P, row_off=d["row_off"], top_p=p, fill=-1e30)
    v2 = s.ws.verify(Q, d["row_off"], d["lengths"], anchor, d["tokens"], d["pd_tok"], d["lse"], s.U, s.W1, s.W2, 1, 0)
    assert torch.equal(v["n_acc"], v2["n_acc"]) and torch.equal(v["next_anchor"], v2["next_anchor"])


def test_a_round_in_a_graph():
    B, gamma, V = 8, 3, 4096
    chain, s, sps, g = server(B, gamma, V, 256, 64, seed=4)
    anchor = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.full((B,), 0.9, device="cuda")
    h = chain.draft_hidden(anchor, gamma, 0.5)
    d = s.draft(h, anchor, sps, 1, 0)
    ht = chain.target_hidden(anchor, d)
    v = s.verify(ht, anchor, d, 1, 0, top_p=p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        d2 = s.draft(h, anchor, sps, 1, 0)
        v2 = s.verify(ht, anchor, d2, 1, 0, top_p=p)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d2["tokens"], d["tokens"])
    assert torch.equal(v2["n_acc"], v["n_acc"]) and torch.equal(v2["next_anchor"], v["next_anchor"])


def test_shapes_that_do_not_fit():
    t = torch.zeros
    with pytest.raises(DsparkError):
        HeadServer(2, 2, t(64, 32, device="cuda"), t(63, 16, device="cuda"), t(16, 64, device="cuda"), t(48, device="cuda"))
    with pytest.raises(DsparkError):
        HeadServer(2, 2, t(64, 32, device="cuda"), t(64, 16, device="cuda"), t(16, 64, device="cuda"), t(47, device="cuda"))
