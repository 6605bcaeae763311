"""The training step on gradients that are not finite."""

import pytest
import torch

from speculative_decoding_head_gb300 import build
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
