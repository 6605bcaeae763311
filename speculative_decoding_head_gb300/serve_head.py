"""Serving the head: rounds whose output layer is held in 4 bits and whose
target draws with its users' settings.

The output matrix [V, H] is brought into 4 bits once (``Fp4Matrix``). A round
makes the parallel logits U of the draft's hidden states, drafts
and plans (``Workspace``), makes the target's logits of the packed verify rows with the same
layer, turns them into the distribution that temperature, top-k, top-p and
min-p make of them (``Sampler.logprobs``, a request's settings for its rows by the
plan's offsets), and verifies against that: what a round emits is what ``Sampler.sample``
would have drawn, row after row. No step waits for the host.

``python -m speculative_decoding_head_gb300.serve_head`` serves a synthetic
chain of tokens and prints what the rounds emit.
"""

from __future__ import annotations

import argparse
import math
from typing import Dict, Optional

import torch

from .binding import DsparkError, Fp4Matrix, Sampler, Workspace


class HeadServer:
    """Rounds of B requests and gamma positions over an output layer ``W_out``
    [V, H] (bf16 or fp32; kept in 4 bits, format ``fmt``), with the Markov head's W1 [V, r] and W2 [r, V] and the
    confidence head's w [H + r] and T [gamma] (1 if None). They are all on one CUDA device, where the rounds run on
    its current stream, whichever device is current."""

    def __init__(self, B: int, gamma: int, W_out: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, w: torch.Tensor,
                 T: Optional[torch.Tensor] = None, mode: str = "static", fmt: str = "nvfp4"):
        V, H = W_out.shape
        if W1.shape[0] != V or W2.shape != (W1.shape[1], V) or w.shape != (H + W1.shape[1],):
            raise DsparkError(f"W1 {list(W1.shape)}, W2 {list(W2.shape)} and w {list(w.shape)} do not fit W_out {[V, H]}")
        dev, f32 = W_out.device, torch.float32
        if dev.type != "cuda":
            raise DsparkError(f"W_out must be on a CUDA device, got {dev}")
        self.device = dev
        self.B, self.gamma, self.V, self.H, self.mode = B, gamma, V, H, mode
        self._here(W1=W1, W2=W2, w=w)
        if T is not None:
            self._here(T=T)
            self._long("T", T, gamma)
        self.W1, self.W2, self.w = W1, W2, w
        self.T = torch.ones(gamma, dtype=f32, device=dev) if T is None else T
        with torch.cuda.device(dev):  # a workspace belongs to the current device, and so do its calls
            self.ws = Workspace(B, gamma, V, W1.shape[1], H, "bf16" if W1.dtype == torch.bfloat16 else "f32", mode)
        self.layer = Fp4Matrix(V, H, fmt, device=dev).quantise(W_out)
        self.hidden, self.rows = (Fp4Matrix(n, H, fmt, device=dev) for n in (B * gamma, B * (gamma + 1)))
        self.sampler = Sampler(B * (gamma + 1), V, requests=B, device=dev)
        self.U = torch.empty(B * gamma, V, dtype=f32, device=dev)
        self.P, self.Q = (torch.empty(B * (gamma + 1), V, dtype=f32, device=dev) for _ in range(2))

    def _here(self, **tensors: torch.Tensor) -> None:
        """Refuses tensors of another device: the workspace takes their addresses as they are."""
        for name, t in tensors.items():
            if t.device != self.device:
                raise DsparkError(f"{name} on {t.device}, the server on {self.device}")

    @staticmethod
    def _long(name: str, t: torch.Tensor, n: int) -> None:
        """Refuses a vector of another length: the workspace reads as many values as its shape says."""
        if t.shape != (n,):
            raise DsparkError(f"{name} must be [{n}], got {list(t.shape)}")

    def draft(self, h: torch.Tensor, anchor: torch.Tensor, sps: torch.Tensor, seed: int, rnd: int) -> Dict[str, torch.Tensor]:
        """Drafts and plans from the draft's hidden states h [B, gamma, H]:
        ``Workspace.draft``'s and ``Workspace.plan``'s outputs."""
        self._here(h=h, anchor=anchor, sps=sps)
        self._long("anchor", anchor, self.B)
        if self.mode != "static":  # a static plan does not look at it
            self._long("sps", sps, 1 + self.B * (self.gamma + 1))
        with torch.cuda.device(self.device):
            self.layer.linear(self.hidden.quantise(h.view(-1, self.H)), out=self.U)
            out = self.ws.new_draft_outputs(self.device)
            out["tokens"].zero_()  # ids of the vocabulary, whatever becomes of the draft
            d = self.ws.draft(self.U, self.W1, self.W2, anchor, h.float().contiguous(), self.w, self.T, seed, rnd, out=out)
            return {**d, **self.ws.plan(d["conf"], sps)}

    def verify(self, ht: torch.Tensor, anchor: torch.Tensor, d: Dict[str, torch.Tensor], seed: int, rnd: int,
               **settings) -> Dict[str, torch.Tensor]:
        """Verifies the last draft against the target's hidden states ht [B (gamma + 1), H], packed by the plan's
        row_off (rows past its last are not looked at), under ``Sampler``'s settings, an entry per request:
        ``Workspace.verify``'s outputs. One request that cannot be verified (a setting out of range, hidden states that
        are not finite) ends the round: ``device_status`` tells of it, and the outputs mean nothing until ``reset``, but
        for that next_anchor holds no id outside of the vocabulary."""
        self._here(ht=ht, anchor=anchor, **{k: d[k] for k in ("row_off", "lengths", "tokens", "pd_tok", "lse")})
        self._long("anchor", anchor, self.B)
        with torch.cuda.device(self.device):
            self.layer.linear(self.rows.quantise(ht, count=d["row_off"][self.B :]), out=self.P)
            self.sampler.logprobs(self.P, row_off=d["row_off"], out=self.Q, **settings)
            out = {"n_acc": torch.full((self.B,), -1, dtype=torch.int32, device=self.device), "next_anchor": anchor.clone()}
            return self.ws.verify(self.Q, d["row_off"], d["lengths"], anchor, d["tokens"], d["pd_tok"], d["lse"], self.U,
                                  self.W1, self.W2, seed, rnd, out=out)

    def _parts(self):
        return (self.layer, self.hidden, self.rows, self.sampler, self.ws)

    def device_status(self) -> int:
        """The first device error of any of the rounds' calls (synchronises)."""
        with torch.cuda.device(self.device):
            return next((s for s in (o.device_status() for o in self._parts()) if s), 0)

    def reset(self) -> None:
        """Clears the device errors, so that rounds go on (and the lagged planner's history)."""
        with torch.cuda.device(self.device):
            for o in self._parts():
                o.reset()


class Chain:
    """A synthetic model: the hidden state after a token points to its
    successor's row of the output layer, the draft's with noise."""

    def __init__(self, V: int, H: int, g: torch.Generator, sharp: float = 1.0):
        self.g, dev = g, g.device
        self.W_out = torch.empty(V, H, device=dev).normal_(0.0, 1.0, generator=g).to(torch.bfloat16)
        self.successor = torch.randperm(V, generator=g, device=dev)
        self.sharp = sharp

    def after(self, x: torch.Tensor, noise: float = 0.0) -> torch.Tensor:
        h = self.W_out[self.successor[x]].float() * (self.sharp * 12.0 / self.W_out.shape[1])
        return (h + noise * torch.empty_like(h).normal_(0.0, 12.0 / self.W_out.shape[1], generator=self.g)).to(torch.bfloat16)

    def draft_hidden(self, anchor: torch.Tensor, gamma: int, noise: float) -> torch.Tensor:
        x, out = anchor.long(), []
        for _ in range(gamma):
            out.append(self.after(x, noise))
            x = self.successor[x]
        return torch.stack(out, 1)

    def target_hidden(self, anchor: torch.Tensor, d: Dict[str, torch.Tensor]) -> torch.Tensor:
        """Hidden states of the packed rows: row row_off[b] + j is after x_j (x_0 the anchor)."""
        x = torch.cat([anchor[:, None], d["tokens"]], 1)
        B, R = x.shape
        n = torch.arange(B * R, device=x.device, dtype=torch.int32)
        b = (torch.searchsorted(d["row_off"], n, right=True) - 1).clamp(0, B - 1)
        j = (n - d["row_off"][b]).clamp(0, R - 1).long()
        return self.after(x[b, j].long())


def main():
    ap = argparse.ArgumentParser(description="Serve a synthetic chain with a 4-bit output layer and sampling settings.")
    for name, value in (("batch", 32), ("gamma", 5), ("vocab", 32000), ("hidden", 1024), ("rank", 64), ("rounds", 50),
                        ("top-k", 0), ("seed", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    for name, value in (("temperature", 0.8), ("top-p", 0.95), ("min-p", 0.0), ("noise", 0.5)):
        ap.add_argument(f"--{name}", type=float, default=value)
    ap.add_argument("--format", choices=["nvfp4", "mxfp4"], default="nvfp4")
    a = ap.parse_args()
    for name, low, high in (("batch", 1, 4096), ("gamma", 1, 32), ("vocab", 1, 1 << 24), ("hidden", 1, 65536), ("rank", 1, 1024),
                            ("rounds", 1, math.inf), ("temperature", 0, 3e38), ("top-p", 0, 1), ("min-p", 0, 1), ("noise", 0, 3e38)):
        if not low <= getattr(a, name.replace("-", "_")) <= high:
            ap.error(f"--{name} must be {f'from {low} to {high:g}' if high < 3e38 else f'at least {low} and finite'}")
    g = torch.Generator(device="cuda").manual_seed(a.seed)
    chain = Chain(a.vocab, a.hidden, g)
    W1 = torch.empty(a.vocab, a.rank, device="cuda").normal_(0.0, 0.02, generator=g).to(torch.bfloat16)
    W2 = torch.empty(a.rank, a.vocab, device="cuda").normal_(0.0, 0.02, generator=g).to(torch.bfloat16)
    w = torch.empty(a.hidden + a.rank, device="cuda").normal_(0.0, 0.05, generator=g)
    s = HeadServer(a.batch, a.gamma, chain.W_out, W1, W2, w, fmt=a.format)
    sps = torch.full((1 + a.batch * (a.gamma + 1),), 400.0, dtype=torch.float64, device="cuda")
    full = lambda v, t=torch.float32: torch.full((a.batch,), v, dtype=t, device="cuda")  # noqa: E731
    settings = dict(temperature=full(a.temperature), top_k=full(a.top_k, torch.int32), top_p=full(a.top_p),
                    min_p=full(a.min_p))
    anchor = torch.randint(0, a.vocab, (a.batch,), generator=g, device="cuda", dtype=torch.int32)
    emitted = torch.zeros((), dtype=torch.int64, device="cuda")
    for rnd in range(a.rounds):
        d = s.draft(chain.draft_hidden(anchor, a.gamma, a.noise), anchor, sps, a.seed, rnd)
        v = s.verify(chain.target_hidden(anchor, d), anchor, d, a.seed, rnd, **settings)
        anchor = v["next_anchor"]
        emitted += v["n_acc"].sum() + a.batch
    if s.device_status():
        raise SystemExit(f"device status {s.device_status()}")
    print(f"{a.rounds} rounds of {a.batch} requests: {int(emitted) / (a.rounds * a.batch):.2f} tokens a request and round")


if __name__ == "__main__":
    main()
