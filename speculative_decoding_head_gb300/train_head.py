"""Training the Markov head's W1 and W2 on the cross entropy of eq. (9).

This is one term of the objective: ``Workspace.train_loss`` reports all three,
weighted, and the other two have no gradients here.

One step over a teacher-forced batch (B blocks of gamma positions): the rows
W1[x_prev] (``Embedding.lookup``), the loss of z = U + W1[x_prev] W2 against
the reference tokens (``LinearCE.forward``), the gradients of
(1/B) sum exp(-k / tau) ce, eq. (12)'s weights (``LinearCE.grad``), the
gradient of W1 by token (``Embedding.grad``), both gradients clipped together
(``GradClip``), and a step of plain gradient descent on fp32 copies. The logits
[B gamma, V] are never stored; the weights it trains are the ones that
``Workspace.draft`` takes.

``python -m speculative_decoding_head_gb300.train_head`` trains a head on
synthetic text (a random bigram chain) and prints the loss.
"""

from __future__ import annotations

import argparse

import torch

from .binding import DsparkError, Embedding, GradClip, LinearCE


class HeadTrainer:
    """W1 [V, r] and W2 [r, V] in training, V a multiple of 8; ``W1`` and ``W2`` are the bf16 weights."""

    def __init__(self, B: int, gamma: int, V: int, r: int, lr: float = 1.0, tau: float = 4.0, max_norm: float = 1.0,
                 w_std: float = 0.02, seed: int = 0, device="cuda"):
        if V % 8:
            raise DsparkError(f"V must be a multiple of 8, as for a draft with bf16 weights, got {V}")
        g = torch.Generator(device=device).manual_seed(seed)
        self.B, self.gamma, self.lr, self.max_norm = B, gamma, lr, max_norm
        n, bf16 = B * gamma, torch.bfloat16
        self.master = [torch.empty(V, r, device=device).normal_(0.0, w_std, generator=g),
                       torch.empty(r, V, device=device).normal_(0.0, w_std, generator=g)]
        self.W1, self.W2 = (m.to(bf16) for m in self.master)
        self.rows = torch.empty(n, -(-r // 8) * 8, dtype=bf16, device=device)[:, :r]  # LinearCE wants rows on 16 bytes
        self.dW1 = torch.empty(V, r, dtype=bf16, device=device)
        self.ce = LinearCE(n, r, V, layout="kv", device=device)
        self.out = self.ce.new_outputs()
        self.emb = Embedding(n, V, r, device=device)
        self.clip = GradClip([self.dW1, self.out["dW"]])
        self.weight = torch.exp(-torch.arange(gamma, device=device) / tau).repeat(B)

    def step(self, U: torch.Tensor, anchor: torch.Tensor, xstar: torch.Tensor):
        """One step on U [B, gamma, V] fp32, anchor [B] and xstar [B, gamma]
        int32 (-1: no token there, and none drafted from). Returns that
        loss before the step and the gradients' norm, on the device. A norm that
        is not finite leaves the weights as they are (and sets the status)."""
        prev = torch.cat([anchor[:, None], xstar[:, :-1]], 1).reshape(-1)
        # a position whose previous token is missing has no row of W1: it is left out
        target = torch.where(prev >= 0, xstar.reshape(-1), torch.full_like(prev, -1))
        U = U.view(self.B * self.gamma, -1)
        X = self.emb.lookup(self.W1, prev, out=self.rows)
        self.ce.forward(X, self.W2, target, U=U, out=self.out)
        self.ce.grad(X, self.W2, target, self.out["lse"], wt=self.weight, scale=1.0 / self.B, U=U, out=self.out)
        self.emb.grad(self.out["dX"], prev, out=self.dW1)
        norm = self.clip.clip(self.max_norm).clone()
        skip = ~torch.isfinite(norm)  # the clip has left such gradients as they are
        for m, w, d in zip(self.master, (self.W1, self.W2), (self.dW1, self.out["dW"])):
            m.add_(d.masked_fill_(skip, 0.0), alpha=-self.lr)
            w.copy_(m)
        return (self.out["loss"] * self.weight).sum() / self.B, norm

    def device_status(self) -> int:
        """The first device error of any of the step's calls (synchronises)."""
        return next((s for s in (o.device_status() for o in (self.ce, self.emb, self.clip)) if s), 0)


def bigram_batch(B: int, gamma: int, V: int, successor: torch.Tensor, g: torch.Generator, p: float = 0.8):
    """Blocks of a chain that moves from a token to its successor with probability p, else anywhere."""
    dev = successor.device
    x = [torch.randint(0, V, (B,), generator=g, device=dev)]
    for _ in range(gamma):
        jump = torch.randint(0, V, (B,), generator=g, device=dev)
        x.append(torch.where(torch.rand(B, generator=g, device=dev) < p, successor[x[-1]], jump))
    return x[0].int(), torch.stack(x[1:], 1).int()


def main():
    ap = argparse.ArgumentParser(description="Train a Markov head on a synthetic bigram chain.")
    for name, value in (("batch", 128), ("gamma", 5), ("vocab", 4096), ("rank", 64), ("steps", 200), ("seed", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--lr", type=float, default=20.0)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(a.seed)
    successor = torch.randperm(a.vocab, generator=g, device="cuda")
    t = HeadTrainer(a.batch, a.gamma, a.vocab, a.rank, lr=a.lr, w_std=0.1, seed=a.seed)
    for i in range(a.steps):
        anchor, xstar = bigram_batch(a.batch, a.gamma, a.vocab, successor, g)
        U = torch.empty(a.batch, a.gamma, a.vocab, device="cuda").normal_(0.0, 0.5, generator=g)
        loss, norm = t.step(U, anchor, xstar)
        if i % 20 == 0 or i == a.steps - 1:
            print(f"step {i}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}")
    if t.device_status():
        raise SystemExit(f"device status {t.device_status()}")


if __name__ == "__main__":
    main()
