"""The 4-bit product's limit on tiles, refused on the host before any CUDA call."""

import ctypes as C

import pytest

from speculative_decoding_head_gb300 import binding, build

EUNSUPPORTED = 5
OK = 256  # never dereferenced


@pytest.mark.parametrize("N,V", [(1 << 24, 1 << 24), ((1 << 22) + 1, 1 << 24), (1 << 24, (1 << 22) + 1)])
@pytest.mark.parametrize("type", [0, 1])
@pytest.mark.parametrize("U", [None, OK])
def test_products_of_more_than_2_to_30_tiles(N, V, type, U):
    build.build()
    m = binding.Fp4Data(OK, OK, OK)
    x, w = binding.Fp4Dims(N, 64, 0), binding.Fp4Dims(V, 64, 0)
    assert -(-N // 256) * -(-V // 256) > 1 << 30
    assert binding.load().dspark_fp4_linear(C.byref(x), C.byref(m), C.byref(w), C.byref(m), U, V, 512, type, V, OK,
                                            None) == EUNSUPPORTED
