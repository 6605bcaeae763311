"""The training step on gradients that are not finite and at ranks off multiples of 8."""

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import DsparkError
from speculative_decoding_head_gb300.train_head import HeadTrainer, bigram_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_whose_gradients_are_not_finite_changes_no_weight(bad):
    B, gamma, V, r = 8, 4, 1000, 32
    t = HeadTrainer(B, gamma, V, r, lr=2.0, w_std=0.1)
    g = torch.Generator(device="cuda").manual_seed(3)
    anchor, xstar = bigram_batch(B, gamma, V, torch.randperm(V, generator=g, device="cuda"), g)
    U = torch.randn(B, gamma, V, generator=g, device="cuda")
    U[2, 1, 17] = bad
    keep = [x.clone() for x in (*t.master, t.W1, t.W2)]
    _, norm = t.step(U, anchor, xstar)
    assert not torch.isfinite(norm) and t.device_status() == 4       # DSPARK_ENUMERIC
    assert all(torch.equal(a, b) for a, b in zip((*t.master, t.W1, t.W2), keep))
    U[2, 1, 17] = 0.0                                                # the next step goes on from there
    _, norm = t.step(U, anchor, xstar)
    assert torch.isfinite(norm) and all(torch.isfinite(m).all() for m in t.master)
    assert not torch.equal(t.master[1], keep[1])


@pytest.mark.parametrize("r", [1, 20, 33])
def test_ranks_that_are_no_multiple_of_8(r):
    """The gradients' norm and the step against 64 bits, as for whole ranks."""
    B, gamma, V = 8, 3, 1000
    t = HeadTrainer(B, gamma, V, r, lr=1.0, max_norm=0.1, w_std=0.3)
    g = torch.Generator(device="cuda").manual_seed(4)
    anchor, xstar = bigram_batch(B, gamma, V, torch.randperm(V, generator=g, device="cuda"), g)
    U = torch.randn(B, gamma, V, generator=g, device="cuda")
    W = [w.double().requires_grad_() for w in (t.W1, t.W2)]
    before = [m.clone() for m in t.master]
    loss, norm = t.step(U, anchor, xstar)
    assert t.device_status() == 0
    prev = torch.cat([anchor[:, None], xstar[:, :-1]], 1).long()
    z = U.double() + W[0][prev] @ W[1]
    ce = torch.logsumexp(z, -1) - z.gather(-1, xstar.long()[..., None])[..., 0]
    ref = (ce * torch.exp(-torch.arange(gamma, device="cuda") / 4.0)).sum() / B
    ref.backward()
    total = float(sum((w.grad ** 2).sum() for w in W)) ** 0.5
    assert abs(float(loss) - float(ref.detach())) <= 1e-5 * float(ref.detach())
    assert abs(float(norm) - total) <= 2.0 ** -7 * total
    for m, m0, w in zip(t.master, before, W):
        want = -min(1.0, 0.1 / total) * w.grad
        assert float((m.double() - m0.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())


def test_vocabularies_the_draft_does_not_take_are_refused():
    with pytest.raises(DsparkError):
        HeadTrainer(4, 3, 1001, 16)
