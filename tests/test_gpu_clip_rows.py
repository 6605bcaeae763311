"""Clipping of lists with empty tensors and of matrices whose rows lie apart.

Tolerances are those of test_gpu_clip.py.
"""

import ctypes as C
import math

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import GradClip, LinearCE, load

from test_gpu_clip import BF16, F32, NORM_TOL, UNIT, _check, _make, _norm

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


def _padded(rows, cols, ld, dtype, g, shift=0):
    """A matrix of rows `ld` apart inside a buffer of NaN."""
    flat = torch.full((rows * ld + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    t = flat[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    return flat, t


ROWS = [(1, 5, 8, 0), (3, 1, 4, 0), (7, 9, 16, 0), (50, 300, 304, 0), (257, 100, 101, 0), (40, 64, 72, 3), (3, 16384, 16392, 0),
        (5, 40003, 40008, 0), (2, 16385, 16385 + 7, 0), (4099, 3, 8, 0), (20000, 33, 40, 0), (3, 0, 8, 0), (0, 4, 8, 0)]


@pytest.mark.parametrize("rows,cols,ld,shift", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [True, False])
def test_matrices_of_padded_rows(rows, cols, ld, shift, dtype, in_place):
    """Matrices whose rows lie apart, beside contiguous tensors: what lies between the rows is neither read nor written."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    flat, a = _padded(rows, cols, ld, dtype, g, shift)
    other = _make([1000, 7], [F32, BF16])
    ts = [other[0], a, other[1]]
    gap = torch.isnan(flat)
    for max_norm in (0.5, 1e9):
        flat2, o = (flat, a) if in_place else _padded(rows, cols, ld + 8, dtype, g)
        gap2 = gap if in_place else torch.ones_like(flat2, dtype=torch.bool)
        if not in_place:
            gap2[:rows * (ld + 8)].view(rows, ld + 8)[:, :cols] = False
            flat2[gap2] = 5.0
        before = [t.double() for t in ts]
        norm = math.sqrt(sum(float((t ** 2).sum()) for t in before))
        coef = min(1.0, max_norm / (norm + 1e-6))
        outs = [torch.full_like(other[0], 3.0), o, torch.full_like(other[1], 3.0)]
        op = GradClip(ts, None if in_place else outs)
        got = op.clip(max_norm)
        assert op.device_status() == 0 and abs(float(got) - norm) <= NORM_TOL * norm
        for t, r in zip(op.outs, before):
            r = r * coef
            assert ((t.double() - r).abs() <= (NORM_TOL + 2.0 ** -23 + UNIT[t.dtype]) * 1.001 * r.abs() + 1e-44).all()
        assert (torch.isnan(flat2[gap2]) if in_place else flat2[gap2] == 5.0).all()


@pytest.mark.parametrize("layout,N,K,V", [("vk", 40, 20, 301), ("kv", 40, 16, 301), ("vk", 9, 4100, 999)])
def test_the_cross_entropys_gradients_are_taken(layout, N, K, V):
    """dX and dW of any size, as new_outputs makes them."""
    g = torch.Generator(device="cuda").manual_seed(6)
    op = LinearCE(N, K, V, layout)
    out = op.new_outputs()
    for k in ("dX", "dW"):
        out[k].copy_(torch.randn(out[k].shape, generator=g, device="cuda"))
    norm = _norm([out["dX"], out["dW"]])
    want = [out[k].double() / (norm + 1e-6) for k in ("dX", "dW")]
    assert abs(float(GradClip([out["dX"], out["dW"]]).clip(1.0)) - norm) <= NORM_TOL * norm
    for k, w in zip(("dX", "dW"), want):
        assert ((out[k].double() - w).abs() <= (NORM_TOL + 2.0 ** -23 + UNIT[BF16]) * 1.001 * w.abs()).all()


def test_many_padded_matrices_and_not_finite():
    g = torch.Generator(device="cuda").manual_seed(7)
    ts = [_padded(3 + i % 5, 10 + i, 16 + i, [BF16, F32][i % 2], g)[1] for i in range(600)]
    _check(ts, 2.0)
    ts[333][1, 2] = math.nan
    op = GradClip(ts)
    assert math.isnan(float(op.clip(1.0))) and op.device_status() == 4


def test_rows_past_32_bits():
    rows, ld = 70001, 32768
    buf = torch.zeros(rows, ld, dtype=BF16, device="cuda")
    x = buf[:, :5]
    x[0, 0], x[rows - 1, 4], buf[65537, 5] = 3.0, 4.0, 100.0
    op = GradClip([x])
    assert abs(float(op.clip(2.5)) - 5.0) <= 5.0 * NORM_TOL and op.device_status() == 0
    assert float(x[0, 0]) == 1.5 and float(x[rows - 1, 4]) == 2.0 and float(buf[65537, 5]) == 100.0
