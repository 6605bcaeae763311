"""The 4-bit product's row factors at magnitudes far apart."""

import pytest
import torch

from speculative_decoding_head_gb300.binding import Fp4Matrix
from test_gpu_fp4 import check_product, values

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("a,b", [(1e36, 1e-30), (1e-30, 1e36), (3e37, 1e-28), (1e12, 1e15), (1e-16, 1e-18), (1e-30, 1e20)])
@pytest.mark.parametrize("N,K,V", [(5, 2048, 300), (300, 512, 129)])
def test_large_rows_and_small_ones(N, K, V, a, b):
    """Factors that are far from 1 on one side and far below it on the other: a sum times one of them alone may lie
    past fp32's range where the product does not."""
    x4 = Fp4Matrix(N, K).quantise(values((N, K), F32, seed=N).clamp(-5, 5) * a)
    w4 = Fp4Matrix(V, K).quantise(values((V, K), F32, seed=V).clamp(-5, 5) * b)
    for dtype in (F32, BF16):
        y = w4.linear(x4, dtype=dtype)
        assert y.isfinite().all()
        check_product(x4, w4, y)
    same = Fp4Matrix(N, K).quantise(torch.full((N, K), a, device="cuda"))
    ones = Fp4Matrix(V, K).quantise(torch.full((V, K), b, device="cuda"))
    y = ones.linear(same)
    check_product(same, ones, y)
    assert y.isfinite().all() and (y > 0).all()


def test_rows_of_all_magnitudes():
    """A row of each power of four from 2^-120 to 2^120 against each: where the product lies in fp32's range it is
    right, past it infinite, and a sum of 0 is 0 whatever the factors are."""
    K = 64
    e = torch.arange(-120, 121, 2, device="cuda").double()
    base = values((1, K), F32, seed=3).clamp(-5, 5).double()
    m4 = Fp4Matrix(e.numel(), K).quantise((base * torch.exp2(e)[:, None]).float())
    y = m4.linear(m4).double()
    X = m4.lookup(dtype=F32).double()
    want = X @ X.t()
    size = X.abs() @ X.abs().t()
    inside = size < 2.0 ** 127
    # the tensor cores' sum as in check_product, and half a step of the result, which may be a subnormal
    tol = 12 * 2.0 ** -23 * size + 2.0 ** -24 * want.abs() + 2.0 ** -150
    assert ((y - want).abs() <= tol)[inside].all()
    assert y[want > 2.0 ** 129].isposinf().all()
    half = torch.zeros(2, K, device="cuda")
    half[0, :32], half[1, 32:] = 2.0 ** 120, 2.0 ** 120
    z4 = Fp4Matrix(2, K).quantise(half)
    y = z4.linear(z4)
    assert float(y[0, 1]) == 0 and float(y[1, 0]) == 0 and y.diag().isposinf().all()
