"""What the bindings of the 4-bit matrices and of sampling refuse on the host.

Runs without a GPU: nothing is launched."""

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import DsparkError, Embedding, Fp4Matrix, LinearCE, Sampler


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("make", [lambda d: Fp4Matrix(4, 64, device=d), lambda d: Sampler(4, 64, device=d),
                                  lambda d: Sampler(4, 64, requests=2, device=d), lambda d: Embedding(4, 64, 16, device=d),
                                  lambda d: LinearCE(4, 16, 64, device=d)])
def test_objects_off_the_gpu_are_refused(make):
    """Their calls would take a CPU tensor's address for one of the object's device."""
    for device in ("cpu", torch.device("cpu")):
        with pytest.raises(DsparkError):
            make(device)
