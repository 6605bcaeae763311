"""The head's training step: the operators together, against the objective and against torch in 64 bits."""

import numpy as np
import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import LinearCE, Workspace
from speculative_decoding_head_gb300.train_head import HeadTrainer, bigram_batch
from speculative_decoding_head_gb300.workloads import Workload, make_loss_inputs

from parity import to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_cross_entropy_is_the_objectives():
    """dspark_train_loss's ce of a batch equals the linear cross entropy of
    X = W1[x_prev], W = W2, U. Each is within its own derived bound of the
    formula (the objective's 5e-5 + 2e-6 |ce|; here twice the error of an
    accumulation over r = 128, 2^-23 * 30 * 16, and of the sum's log)."""
    wl = Workload("train_ce", B=12, gamma=5, V=5000, r=128, H=0, wdtype="bf16", mode="static", seed=23, u_std=2.0,
                  w_std=0.05)
    dev = to_device(make_loss_inputs(wl))
    ws = Workspace.for_workload(wl)
    ref = ws.train_loss(dev["U"], dev["W1"], dev["W2"], dev["anchor"], dev["xstar"], dev["P"], dev["conf"], 4.0)
    prev = torch.cat([dev["anchor"][:, None], dev["xstar"][:, :-1]], 1).reshape(-1)
    n = wl.B * wl.gamma
    ce = LinearCE(n, wl.r, wl.V, layout="kv")
    out = ce.forward(dev["W1"][prev.long()], dev["W2"], dev["xstar"].reshape(-1), U=dev["U"].view(n, wl.V))
    a, b = out["loss"].cpu().numpy().astype(np.float64), ref["ce"].reshape(-1).cpu().numpy().astype(np.float64)
    tol = 5e-5 + 2e-6 * np.abs(b) + 2 * (2.0 ** -23 * 30 * 16 + 2.0 ** -20 + 2.0 ** -22 * 20)
    assert (np.abs(a - b) <= tol).all(), np.abs(a - b).max()


def test_step_against_64_bits():
    """One step's loss, gradients' norm and new weights against torch in 64
    bits. The gradients are bf16 (2^-8 relative each, and G's rounding under
    them, the sum of absolute terms at most a few times the entry's size), so
    the weights' change agrees in the 2-norm to 2^-7."""
    B, gamma, V, r = 16, 4, 3000, 64
    t = HeadTrainer(B, gamma, V, r, lr=2.0, max_norm=0.1, w_std=0.1)
    g = torch.Generator(device="cuda").manual_seed(1)
    anchor, xstar = bigram_batch(B, gamma, V, torch.randperm(V, generator=g, device="cuda"), g)
    xstar[3, 1:] = -1                                    # a short block
    U = torch.randn(B, gamma, V, generator=g, device="cuda")
    W = [w.double().requires_grad_() for w in (t.W1, t.W2)]
    before = [m.clone() for m in t.master]
    loss, norm = t.step(U, anchor, xstar)
    assert t.device_status() == 0
    prev = torch.cat([anchor[:, None], xstar[:, :-1]], 1).long()
    live = (prev >= 0) & (xstar >= 0)
    z = U.double() + W[0][prev.clamp(min=0)] @ W[1]
    ce = torch.logsumexp(z, -1) - z.gather(-1, xstar.clamp(min=0).long()[..., None])[..., 0]
    ref = (ce * live * torch.exp(-torch.arange(gamma, device="cuda") / 4.0)).sum() / B
    ref.backward()
    ref = float(ref.detach())
    assert abs(float(loss) - ref) <= 1e-5 * ref
    total = float(sum((w.grad ** 2).sum() for w in W)) ** 0.5
    assert abs(float(norm) - total) <= 2.0 ** -7 * total
    scale = min(1.0, 0.1 / total)
    for m, m0, w in zip(t.master, before, W):
        want = -2.0 * scale * w.grad
        assert float((m.double() - m0.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())


def test_training_lowers_the_loss_and_the_head_drafts():
    """Two hundred steps on a bigram chain: the loss falls below that of a head that knows nothing, and the draft takes the weights."""
    B, gamma, V, r = 64, 5, 1024, 64
    t = HeadTrainer(B, gamma, V, r, lr=20.0, w_std=0.1)
    g = torch.Generator(device="cuda").manual_seed(2)
    successor = torch.randperm(V, generator=g, device="cuda")
    losses = []
    for _ in range(200):
        anchor, xstar = bigram_batch(B, gamma, V, successor, g)
        losses.append(float(t.step(torch.zeros(B, gamma, V, device="cuda"), anchor, xstar)[0]))
    assert t.device_status() == 0
    assert losses[-1] < 0.8 * losses[0], (losses[0], losses[-1])
    ws = Workspace(B, gamma, V, r, 0, wdtype="bf16", mode="static")
    d = ws.draft(torch.zeros(B, gamma, V, device="cuda"), t.W1, t.W2, anchor, None,
                 torch.zeros(r, device="cuda"), torch.ones(gamma, device="cuda"), 0, 0)
    torch.cuda.synchronize()
    assert ws.device_status() == 0
    prev = torch.cat([anchor[:, None], d["tokens"][:, :-1]], 1).long()
    follow = float((d["tokens"].long() == successor[prev]).float().mean())
    assert follow > 20.0 / V, follow
