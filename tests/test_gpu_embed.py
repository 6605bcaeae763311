"""Embedding rows and the table's gradient on the GPU against the formulas in 64 bits.

Tolerances. A looked-up value is one fp32 product (2^-24 relative) rounded to
the table's type (bf16: 2^-8 relative, fp32: exact). A gradient entry is a
sum of fp32 values in a fixed grouping (32 rows, up to 8 groups of them, then
runs of 256 rows): at most n additions deep, so its error is at most
2^-24 * min(n, 32 + 8 + n / 256 + 4) * sum |dout| * |scale| with n the token's
rows, plus the product with the scale, the addition to base (2^-24 relative
each) and the rounding to the gradient's type.
"""

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import DsparkError, Embedding

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
UNIT = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _mat(rows, cols, ld, dtype, g, shift=0):
    """[rows, cols] with leading dimension ld, `shift` values past an aligned address, NaN in between."""
    flat = torch.full((rows * ld + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    t = flat[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    return t


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,V,D,lde,ldo,shift", [
    (1, 1, 1, 1, 1, 0), (6, 1024, 16, 16, 80, 0), (5, 7, 3, 3, 5, 1), (33, 100, 257, 264, 257, 0),
    (1000, 513, 256, 256, 256, 0), (130, 50, 1000, 1000, 1008, 8), (67, 31, 5120, 5120, 5376, 0), (9, 20, 300, 301, 303, 3),
])
def test_lookup(dtype, N, V, D, lde, ldo, shift):
    g = _gen(N + D)
    E = _mat(V, D, lde, dtype, g, shift)
    idx = torch.randint(-1, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    full = torch.full((N * ldo + shift,), 5.0, dtype=dtype, device="cuda")
    out = full[shift:].view(N, ldo)[:, :D]
    op = Embedding(N, V, D)
    got = op.lookup(E, idx, scale=1.7, out=out)
    assert op.device_status() == 0 and got is out
    ref = torch.where((idx >= 0)[:, None], E[idx.clamp(min=0).long()].double() * float(torch.tensor(1.7)), 0.0)
    assert ((got.double() - ref).abs() <= (2.0 ** -24 + UNIT[dtype]) * 1.001 * ref.abs()).all()
    assert (full[:shift] == 5.0).all() and (full[shift:].view(N, ldo)[:, D:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [8191, 8193, 20002])
@pytest.mark.parametrize("D,ld,shift", [(1, 1, 0), (9, 11, 1), (16, 16, 0), (17, 24, 8), (64, 64, 0), (65, 65, 0),
                                        (128, 128, 0), (129, 136, 0)])
def test_lookup_of_many_short_rows(dtype, N, D, ld, shift):
    g = _gen(N + D)
    E = _mat(700, D, ld, dtype, g, shift)
    idx = torch.randint(-1, 700, (N,), generator=g, device="cuda", dtype=torch.int32)
    full = torch.full((N * ld + shift,), 5.0, dtype=dtype, device="cuda")
    op = Embedding(N, 700, D)
    got = op.lookup(E, idx, scale=0.5, out=full[shift:].view(N, ld)[:, :D])
    assert op.device_status() == 0
    # a product with 0.5 is exact
    assert torch.equal(got, torch.where((idx >= 0)[:, None], E[idx.clamp(min=0).long()] * 0.5, 0.0))
    assert (full[:shift] == 5.0).all() and (full[shift:].view(N, ld)[:, D:] == 5.0).all()


def _grad_ref(dout, idx, V, scale, base):
    D = dout.shape[1]
    ref = torch.zeros(V, D, dtype=F64, device="cuda")
    mag = torch.zeros(V, D, dtype=F64, device="cuda")
    has = idx >= 0
    i = idx[has].long()
    ref.index_add_(0, i, dout[has].double())
    mag.index_add_(0, i, dout[has].double().abs())
    n = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, i, torch.ones(i.numel(), dtype=F64, device="cuda"))
    s = float(torch.tensor(scale, dtype=F32))
    ref, mag = ref * s, mag * abs(s)
    depth = torch.minimum(n, 44 + n / 256)[:, None]
    tol = 2.0 ** -24 * depth * mag + 2.0 ** -23 * ref.abs()
    if base is not None:
        ref = ref + base.double()
        tol = tol + 2.0 ** -24 * ref.abs()
    return ref, tol, n


def _check_grad(N, V, D, tin, tout, idx, scale=0.75, ldd=None, ldo=None, shift=0, with_base=False, in_place=False, seed=1):
    g = _gen(seed)
    dout = _mat(N, D, ldd or D, tin, g, shift)
    out = _mat(V, D, ldo or D, tout, g, shift)
    base = _mat(V, D, ldo or D, tout, g, shift) if with_base else None
    if in_place:
        base = out
    ref, tol, n = _grad_ref(dout, idx, V, scale, base)
    before = out.clone()
    op = Embedding(N, V, D)
    got = op.grad(dout, idx, scale=scale, base=base, out=out)
    assert op.device_status() == 0
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all() and (err <= tol + UNIT[tout] * 1.001 * ref.abs()).all(), float(err.max())
    none = n == 0
    if in_place:
        assert torch.equal(got[none], before[none])
    elif base is not None:
        assert torch.equal(got[none], base[none])
    else:
        assert (got[none] == 0).all()
    return op, got, dout


def _idx(N, V, kind, seed=2):
    g = _gen(seed)
    if kind == "uniform":
        return torch.randint(-1, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "one":                       # every row the same token
        return torch.full((N,), V // 2, dtype=torch.int32, device="cuda")
    if kind == "none":
        return torch.full((N,), -1, dtype=torch.int32, device="cuda")
    if kind == "ends":                      # the first and the last token alone
        return torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, 0, V - 1).int()
    u = torch.rand(N, generator=g, device="cuda", dtype=F64)      # frequencies falling as 1 / rank, low tokens first
    return (torch.exp(u * torch.log(torch.tensor(float(V + 1)))) - 1).long().clamp(0, V - 1).int()


@pytest.mark.parametrize("kind", ["uniform", "one", "none", "ends", "zipf"])
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (6, 1024, 16), (255, 33, 40), (256, 1000, 256), (257, 70, 264),
                                   (1000, 1025, 300), (8192, 300, 64), (8193, 40000, 72), (40000, 5000, 24)])
def test_gradient(N, V, D, kind):
    _check_grad(N, V, D, BF16, BF16, _idx(N, V, kind))


@pytest.mark.parametrize("tin,tout", [(BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("ldd,ldo,shift", [(None, None, 0), (133, 131, 0), (136, 136, 8), (135, 136, 3)])
def test_gradient_types_and_layouts(tin, tout, ldd, ldo, shift):
    for N, kind in ((700, "zipf"), (9000, "zipf"), (3, "uniform")):
        _check_grad(N, 900, 130, tin, tout, _idx(N, 900, kind), ldd=ldd, ldo=ldo, shift=shift)


@pytest.mark.parametrize("tin,tout", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_added(tin, tout, in_place):
    for N, V, D in ((600, 300, 200), (10000, 700, 333), (4, 50, 8)):
        _check_grad(N, V, D, tin, tout, _idx(N, V, "zipf"), with_base=not in_place, in_place=in_place)


def test_large_vocabulary_and_three_digits():
    _check_grad(20000, 1 << 21, 8, F32, F32, _idx(20000, 1 << 21, "uniform"))
    _check_grad(500, 129280, 16, BF16, BF16, _idx(500, 129280, "uniform"))


@pytest.mark.parametrize("N", [4096, 4097, 16385, 32768, 32769, 70000, 262144, 262145, 530000])
@pytest.mark.parametrize("V", [2, 1025, (1 << 20) + 1])
def test_lengths_about_the_sorts_bounds(N, V):
    """Sizes on both sides of where the sort's form changes, of one to three digits."""
    for kind in ("uniform", "zipf"):
        _check_grad(N, V, 3, F32, F32, _idx(N, V, kind))


def test_offsets_past_32_bits():
    """A table whose rows lie more than 2^31 values apart from end to end."""
    V, D = 70001, 32768
    E = torch.empty(V, D, dtype=BF16, device="cuda")
    E[0], E[V - 1], E[65537] = 1.0, 2.0, 3.0
    idx = torch.tensor([V - 1, 0, 65537, V - 1], dtype=torch.int32, device="cuda")
    op = Embedding(4, V, D)
    out = op.lookup(E, idx)
    assert (out[0] == 2).all() and (out[1] == 1).all() and (out[2] == 3).all() and (out[3] == 2).all()
    E.fill_(float("nan"))
    op.grad(out, idx, out=E)
    assert (E[V - 1] == 4).all() and (E[0] == 1).all() and (E[65537] == 3).all() and (E[65536] == 0).all()
    assert not torch.isnan(E[::1000].float()).any()


def test_no_rows():
    op = Embedding(0, 20, 16)
    idx = torch.empty(0, dtype=torch.int32, device="cuda")
    assert op.lookup(torch.zeros(20, 16, device="cuda"), idx).shape == (0, 16)
    out = torch.full((20, 16), 7.0, device="cuda")
    op.grad(torch.empty(0, 16, device="cuda"), idx, out=out)
    assert (out == 0).all()
    out.fill_(7.0)
    op.grad(torch.empty(0, 16, device="cuda"), idx, base=out, out=out)
    assert (out == 7).all()


def test_tokens_out_of_range_are_reported():
    g = _gen(3)
    for N in (40, 9000):
        idx = torch.randint(0, 100, (N,), generator=g, device="cuda", dtype=torch.int32)
        clean = idx.clone()
        for at, bad in ((3, 100), (N - 1, -2), (17, 2 ** 31 - 1), (20, -2 ** 31)):
            idx[at], clean[at] = bad, -1
        dout, E = torch.randn(N, 40, generator=g, device="cuda"), torch.randn(100, 40, generator=g, device="cuda")
        op = Embedding(N, 100, 40)
        got = op.lookup(E, idx)
        assert op.device_status() == 6      # DSPARK_ERANGE
        op.reset()
        assert torch.equal(got, op.lookup(E, clean)) and op.device_status() == 0
        got = op.grad(dout, idx)
        assert op.device_status() == 6
        op.reset()
        assert torch.equal(got, op.grad(dout, clean)) and op.device_status() == 0


def test_same_result_each_time_and_on_another_stream():
    idx = _idx(30000, 2000, "zipf")
    op, first, dout = _check_grad(30000, 2000, 136, BF16, F32, idx)
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(first)
        side.wait_stream(torch.cuda.current_stream())
        op.grad(dout, idx, scale=0.75, out=out, stream=side)
        side.synchronize()
        assert torch.equal(out, first)


def test_gradient_against_differences():
    """sum(R * lookup(E)) is linear in E: its change along a direction is the gradient's product with it."""
    g = _gen(8)
    N, V, D = 300, 50, 24
    grid = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float() / 8  # noqa: E731
    E, R, d = grid(V, D), grid(N, D), grid(V, D)
    idx = _idx(N, V, "uniform")
    op = Embedding(N, V, D)
    total = lambda T: float((op.lookup(T, idx, scale=0.5).double() * R.double()).sum())  # noqa: E731
    grad = op.grad(R, idx, scale=0.5)
    # every value lies on a grid that fp32 sums hold exactly
    assert (total(E + d) - total(E - d)) / 2 == float((grad.double() * d.double()).sum())


def test_refusals():
    op = Embedding(10, 20, 16)
    E, idx = torch.zeros(20, 16, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda")
    dout = torch.zeros(10, 16, device="cuda")
    for bad in (lambda: op.lookup(E.half(), idx), lambda: op.lookup(E[:19], idx), lambda: op.lookup(E, idx.long()),
                lambda: op.lookup(E, idx[:9]), lambda: op.lookup(E.cpu(), idx), lambda: op.lookup(E.t().contiguous().t(), idx),
                lambda: op.lookup(E, idx, out=torch.zeros(10, 16, device="cuda", dtype=BF16)),
                lambda: op.lookup(E, idx, out=torch.zeros(10, 15, device="cuda")),
                lambda: op.grad(dout.double(), idx), lambda: op.grad(dout[:9], idx), lambda: op.grad(dout, idx.float()),
                lambda: op.grad(dout, idx, base=torch.zeros(20, 16, device="cuda", dtype=BF16), out=E),
                lambda: op.grad(dout, idx, out=torch.zeros(21, 16, device="cuda"))):
        with pytest.raises(DsparkError):
            bad()
    for dims in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (2 ** 24 + 1, 8, 8), (8, 2 ** 24 + 1, 8), (8, 8, 2 ** 20 + 1)):
        with pytest.raises(DsparkError):
            Embedding(*dims)
