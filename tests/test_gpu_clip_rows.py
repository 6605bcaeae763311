"""Clipping of lists with empty tensors.

Tolerances are those of test_gpu_clip.py.
"""

import ctypes as C

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import load

from test_gpu_clip import NORM_TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_an_empty_tensors_pointers_are_not_looked_at():
    x = torch.full((9,), 4.0, device="cuda")
    norm, st = torch.zeros((), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lib = load()
    scratch = torch.empty(lib.dspark_clip_grads_scratch_bytes(3), dtype=torch.uint8, device="cuda")
    ptrs = (C.c_void_p * 3)(None, x.data_ptr(), 7)       # no address, and one on no boundary
    code = lib.dspark_clip_grads(3, ptrs, ptrs, (C.c_int64 * 3)(0, 9, 0), (C.c_int32 * 3)(1, 0, 0), 6.0, norm.data_ptr(),
                                 scratch.data_ptr(), st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert code == 0 and float(norm) == 12.0 and int(st) == 0
    assert ((x.double() - 2.0).abs() <= 2.0 * (NORM_TOL + 2.0 ** -23)).all()
