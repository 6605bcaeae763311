"""Matrices in microscaled 4-bit floating point against their definition in 64 bits.

Quantisation and lookup are exact: every value is compared for equality. The product's terms
are exact and summed in fp32 by the tensor cores, which cut a running sum off to 24 bits or
so; the tolerance counts one unit in the last place (2^-23 of the sum of magnitudes) for
every 16 terms and 8 more for the joins, then the output's own rounding (half a step)."""

import math

import numpy as np
import pytest
import torch

import serve_ref as ref
from speculative_decoding_head_gb300.binding import DsparkError, Fp4Matrix

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FMTS = ("nvfp4", "mxfp4")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def values(shape, dtype, seed=0, std=1.0):
    x = torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen(seed))
    x[:, ::7] *= 5
    return x.to(dtype)


def same(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.array_equal(got[fine], want[fine]), int((got[fine] != want[fine]).sum())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,K", [(1, 1), (3, 16), (5, 33), (2, 64), (130, 256), (128, 257), (300, 1000), (7, 2048),
                                 (5, 2064), (2, 5120), (1, 32768), (1, 65535)])
def test_quantised_values_are_the_nearest(R, K, fmt, dtype):
    x = values((R, K), dtype, seed=R + K)
    m = Fp4Matrix(R, K, fmt).quantise(x)
    want, _, f = ref.fp4(x, fmt)
    same(m.lookup(dtype=F32), want)
    same(m.lookup(dtype=BF16), want)
    if fmt == "nvfp4":
        assert np.array_equal(m.rowf[:R].cpu().double().numpy(), f)
    assert m.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_layout_of_codes_and_scales(fmt):
    R, K = 200, 300
    x = values((R, K), BF16, seed=1)
    m = Fp4Matrix(R, K, fmt).quantise(x)
    want, scale, f = ref.fp4(x, fmt)
    B, ld = ref.BLOCK[fmt], (K + 31) // 32 * 16
    codes = m.codes.cpu().numpy().reshape(R, ld)
    nib = np.stack([codes & 15, codes >> 4], 2).reshape(R, -1)
    val = np.where(nib & 8, -1.0, 1.0) * ref.E2M1[nib & 7]
    assert not val[:, K:].any()
    raw = m.scales.cpu().numpy()
    nb = 256 // B
    for r in (0, 1, 31, 32, 127, 128, 199):
        for b in range(-(-K // B)):
            at = ((r // 128) * 2 + b // nb) * 128 * nb + b % nb // 4 * 512 + r % 128 % 32 * 16 + r % 128 // 32 * 4 + b % 4
            s = ref.E4M3[raw[at]] * f[r] if fmt == "nvfp4" else 2.0 ** (int(raw[at]) - 127)
            assert s == scale[r, b]
            assert np.array_equal(val[r, b * B:min(K, b * B + B)] * s, want[r, b * B:b * B + B])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", FMTS)
def test_borders_between_two_numbers(fmt, dtype):
    """Quotients on each border of the 4-bit numbers and of the scales, and one step to either side."""
    rows = []
    for s in (1.0, 1.125, 1.375, 1.875, 3.0 * 2.0 ** -5):
        row = [6.0 * s]
        for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            t = torch.tensor([b * s], dtype=dtype)
            step = t * torch.finfo(dtype).eps
            row += [float(t), float(t + step), float(t - step / 2), -float(t), -float(t + step), -float(t - step / 2)]
        rows.append(row[:32] + row[:1] * 0 + [0.0] * (64 - len(row[:32])))
        rows.append([6.0 * s] + row[32:] + [0.0] * (63 - len(row[32:])))
    # a block's largest magnitude at a border between two scales, beside a row's largest value
    for e in range(8):
        for mid in (8.5, 9.5, 12.5, 15.5):
            t = torch.tensor([6.0 * mid * 2.0 ** -e], dtype=dtype)
            near = [float(t), float(t * (1 + torch.finfo(dtype).eps)), float(t * (1 - torch.finfo(dtype).eps / 2))]
            for v in near:
                rows.append([2688.0] + [0.0] * 31 + [v, v / 3, -v / 5] + [0.0] * 29)
    x = torch.tensor(rows, device="cuda").to(dtype)
    m = Fp4Matrix(*x.shape, fmt).quantise(x)
    same(m.lookup(dtype=F32), ref.fp4(x, fmt)[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_zeros_and_extreme_magnitudes(fmt):
    x = torch.zeros(10, 100, device="cuda")
    x[1] = 3.4e38
    x[2] = 1e-44
    x[3, :50] = 2.0 ** -126
    x[4, 0], x[4, 1:] = 1e20, 1e-20
    x[5] = -0.0
    x[6] = torch.finfo(F32).tiny * torch.arange(100, device="cuda")
    x[7, ::16] = 2688.0
    x[8] = 2.0 ** torch.arange(-50, 50, device="cuda").float()
    m = Fp4Matrix(10, 100, fmt).quantise(x)
    want = ref.fp4(x, fmt)[0]
    same(m.lookup(dtype=F32), want.astype(np.float32).astype(np.float64))
    assert m.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", FMTS)
def test_blocks_that_are_not_finite(fmt, dtype):
    x = values((4, 128), dtype, seed=3)
    x[0, 5], x[1, 40], x[2, 100] = float("nan"), float("inf"), float("-inf")
    m = Fp4Matrix(4, 128, fmt).quantise(x)
    same(m.lookup(dtype=F32), ref.fp4(x, fmt)[0])
    assert m.device_status() == 4
    m.reset()
    assert m.device_status() == 0
    # the rows' products are NaN, the others are not
    w = Fp4Matrix(9, 128, fmt).quantise(values((9, 128), dtype, seed=4))
    y = w.linear(m)
    assert y[:3].isnan().all() and y[3].isfinite().all()


def test_strides_and_alignment():
    for fmt in FMTS:
        big = values((40, 333), F32, seed=5)
        for dtype in (BF16, F32):
            for view in (big.to(dtype)[:, 1:300], big.to(dtype)[::2, 3:300], big.to(dtype)[3:, :256]):
                m = Fp4Matrix(*view.shape, fmt).quantise(view)
                want = ref.fp4(view, fmt)[0]
                out = torch.full((view.shape[0], 400), 7.0, device="cuda", dtype=dtype)
                m.lookup(out=out[:, 5:5 + view.shape[1]])
                same(out[:, 5:5 + view.shape[1]], want)
                assert (out[:, :5] == 7).all() and (out[:, 5 + view.shape[1]:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [40, 256, 5376])  # several rows a CTA, one, and one of many threads
@pytest.mark.parametrize("count", [-1, 0, 1, 129, 200, 1 << 30])
def test_rows_behind_the_last_are_not_read(count, K, dtype, fmt):
    R = 200
    x = values((R, K), dtype, seed=count & 255)
    n = min(max(count, 0), R)
    x[n:] = math.nan
    m = Fp4Matrix(R, K, fmt)
    m.codes.fill_(255)
    m.scales.fill_(255)
    m.rowf.fill_(math.nan)
    m.quantise(x, count=torch.tensor([count], dtype=torch.int32, device="cuda"))
    full = Fp4Matrix(R, K, fmt).quantise(torch.where(torch.arange(R, device="cuda")[:, None] < n, x, 0).to(dtype))
    assert m.device_status() == 0
    assert torch.equal(m.codes, full.codes) and torch.equal(m.scales, full.scales)
    assert torch.equal(m.lookup(), full.lookup()) and (m.lookup()[n:] == 0).all()
    if fmt == "nvfp4":
        assert torch.equal(m.rowf[:R], full.rowf[:R])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("V,D,N", [(1, 16, 3), (300, 256, 1000), (1000, 100, 77), (129280, 33, 500)])
def test_rows_by_token(V, D, N, fmt):
    x = values((V, D), BF16, seed=6, std=0.02)
    m = Fp4Matrix(V, D, fmt).quantise(x)
    idx = torch.randint(0, V, (N,), generator=gen(7), device="cuda", dtype=torch.int32)
    idx[::5] = -1
    every = m.lookup(dtype=F32)
    want = torch.where((idx >= 0)[:, None], every[idx.clamp(min=0).long()], torch.zeros(1, device="cuda"))
    assert torch.equal(m.lookup(idx, dtype=F32), want)
    assert torch.equal(m.lookup(idx, dtype=BF16), want.to(BF16))
    assert m.device_status() == 0
    idx[1] = V
    assert not m.lookup(idx)[1].any()
    assert m.device_status() == 6
    assert m.lookup(idx[:0]).shape == (0, D)


def check_product(x4, w4, y, U=None):
    X, W = x4.lookup(dtype=F32).double(), w4.lookup(dtype=F32).double()
    want = X @ W.t()
    size = X.abs() @ W.abs().t()
    K = X.shape[1]
    tol = (-(-K // 16) + 8) * 2.0 ** -23 * size
    if U is not None:
        want = want + U.double()
        tol = tol + 2.0 ** -24 * want.abs()
    tol = tol + torch.finfo(y.dtype).eps / 2 * want.abs() + 1e-30
    worst = ((y.double() - want).abs() / tol).max()
    assert worst <= 1.0, float(worst)


SHAPES = [(1, 1, 1), (1, 64, 128), (2, 64, 200), (16, 128, 128), (3, 31, 100), (17, 100, 129), (100, 256, 384),
          (128, 320, 1000), (129, 300, 257), (200, 1000, 130), (224, 512, 500), (225, 512, 500), (240, 96, 700),
          (256, 4096, 300), (257, 160, 1000), (640, 256, 4104), (700, 777, 1001), (5, 5120, 2000), (1030, 600, 129)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K,V", SHAPES)
def test_product(N, K, V, fmt):
    x4 = Fp4Matrix(N, K, fmt).quantise(values((N, K), BF16, seed=N))
    w4 = Fp4Matrix(V, K, fmt).quantise(values((V, K), BF16, seed=V, std=0.05))
    check_product(x4, w4, w4.linear(x4))
    check_product(x4, w4, w4.linear(x4, dtype=BF16))
    U = torch.empty(N, V, device="cuda").normal_(0.0, 2.0, generator=gen(9))
    check_product(x4, w4, w4.linear(x4, U=U), U)
    check_product(x4, w4, w4.linear(x4, U=U, dtype=BF16), U)
    V0 = U.clone()
    check_product(x4, w4, w4.linear(x4, U=V0, out=V0), U)  # added in place
    assert w4.device_status() == 0 and x4.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_product_into_strided_rows(fmt):
    N, K, V = 33, 200, 301
    x4 = Fp4Matrix(N, K, fmt).quantise(values((N, K), F32, seed=1))
    w4 = Fp4Matrix(V, K, fmt).quantise(values((V, K), F32, seed=2))
    for dtype in (F32, BF16):
        for off, ld in ((0, 304), (1, 310), (2, 333)):
            big = torch.full((N, ld + 3), 7.0, dtype=dtype, device="cuda")
            Ub = torch.empty(N, ld + 1, device="cuda").normal_(generator=gen(3))
            y, U = big[:, off:off + V], Ub[:, 1:1 + V]
            check_product(x4, w4, w4.linear(x4, U=U, out=y), U)
            assert (big[:, :off] == 7).all() and (big[:, off + V:] == 7).all()


def test_many_tiles_and_persistent_ctas():
    """More tiles than SMs at every width of a tile, so that both accumulators and the ring of stages go round."""
    for N, V in ((8, 40000), (250, 40000), (600, 20000)):
        x4 = Fp4Matrix(N, 520).quantise(values((N, 520), BF16, seed=N))
        w4 = Fp4Matrix(V, 520).quantise(values((V, 520), BF16, seed=V, std=0.05))
        y = w4.linear(x4)
        check_product(x4, w4, y)
        for _ in range(3):
            assert torch.equal(w4.linear(x4), y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K,V", [(5, 100, 700), (601, 64, 20011)])  # of the second a pair has several tiles
def test_logits_of_any_alignment_are_added(N, K, V, fmt):
    """The sum is one rounding of the product's fp32 result, however U's and Y's rows lie."""
    x4 = Fp4Matrix(N, K, fmt).quantise(values((N, K), F32, seed=1))
    w4 = Fp4Matrix(V, K, fmt).quantise(values((V, K), F32, seed=2))
    z = w4.linear(x4)
    even = -(-V // 8) * 8
    for ldu, offu in ((even, 0), (even, 1), (even + 1, 0), (even + 5, 3)):
        U = torch.empty(N, ldu + 4, device="cuda").normal_(generator=gen(ldu + offu))[:, offu:offu + V]
        U = U.as_strided((N, V), (ldu, 1), offu) if ldu >= V + offu else U
        want = z + U
        for ldy, offy in ((even, 0), (even + 8, 1), (even + 1, 0)):
            for dtype in (F32, BF16):
                big = torch.full((N, ldy + 8), 7.0, dtype=dtype, device="cuda")
                y = big[:, offy:offy + V]
                assert torch.equal(w4.linear(x4, U=U, out=y), want.to(dtype))
                assert (big[:, :offy] == 7).all() and (big[:, offy + V:] == 7).all()
        inplace = torch.empty(N, ldu + 4, device="cuda")[:, offu:offu + V]
        inplace.copy_(U)
        assert torch.equal(w4.linear(x4, U=inplace, out=inplace), want)


def test_offsets_past_32_bits():
    N, K, V = 16700, 64, 129280
    x4 = Fp4Matrix(N, K).quantise(values((N, K), BF16, seed=1))
    w4 = Fp4Matrix(V, K).quantise(values((V, K), BF16, seed=2))
    y = w4.linear(x4, dtype=BF16)
    last = Fp4Matrix(5, K).quantise(values((N, K), BF16, seed=1)[-5:])
    assert torch.equal(w4.linear(last, dtype=BF16), y[-5:])


def test_streams_and_graphs():
    N, K, V = 48, 512, 3000
    x, w = values((N, K), BF16, seed=1), values((V, K), BF16, seed=2)
    x4, w4 = Fp4Matrix(N, K), Fp4Matrix(V, K).quantise(w)
    want = w4.linear(x4.quantise(x)).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.linear(x4.quantise(x, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.linear(x4.quantise(x), out=out)
    x.copy_(values((N, K), BF16, seed=8))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, w4.linear(x4.quantise(x)))
    assert not torch.equal(out, want)


def test_refusals():
    with pytest.raises(DsparkError):
        Fp4Matrix(4, 0)
    with pytest.raises(DsparkError):
        Fp4Matrix(4, 65537)
    with pytest.raises(DsparkError):
        Fp4Matrix(4, 64, "fp4")
    a, b, c = Fp4Matrix(4, 64), Fp4Matrix(6, 64, "mxfp4"), Fp4Matrix(6, 32)
    x = torch.zeros(4, 64, device="cuda")
    for bad in (x.half(), x[:, :32], x.t(), x.cpu()):
        with pytest.raises(DsparkError):
            a.quantise(bad)
    for other in (b, c):
        with pytest.raises(DsparkError):
            other.linear(a)
    a.quantise(x)
    w = Fp4Matrix(6, 64).quantise(torch.zeros(6, 64, device="cuda"))
    with pytest.raises(DsparkError):
        w.linear(a, out=torch.empty(4, 7, device="cuda"))
    with pytest.raises(DsparkError):
        w.linear(a, U=torch.empty(4, 6, device="cuda", dtype=BF16))
    with pytest.raises(DsparkError):
        a.lookup(torch.zeros(2, dtype=torch.int64, device="cuda"))
    for count in (torch.zeros(2, device="cuda", dtype=torch.int32), torch.zeros(1, device="cuda"),
                  torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(DsparkError):
            a.quantise(x, count=count)
    flat = x[:1].expand(4, 64)  # rows that overlap
    with pytest.raises(DsparkError):
        a.quantise(flat)
    with pytest.raises(DsparkError):
        a.lookup(out=flat)
    with pytest.raises(DsparkError):
        w.linear(a, out=torch.empty(1, 6, device="cuda").expand(4, 6))
    with pytest.raises(DsparkError):
        w.linear(a, U=torch.empty(1, 6, device="cuda").expand(4, 6))
    assert Fp4Matrix(0, 64).quantise(torch.zeros(0, 64, device="cuda")).rows == 0
    assert w.linear(Fp4Matrix(0, 64)).shape == (0, 6)
