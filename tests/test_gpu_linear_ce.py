"""The linear cross entropy and its gradients on the GPU against the formulas in 64 bits.

Tolerances, from the arithmetic. z is a sum of K exact products of bf16 values
in a tensor-core accumulator of 24 bits, a rounding of at most one unit
(2^-23 of the partial sum) per 16 terms and a few for U and the last
exponent's argument: |z error| <= 2^-23 * zmax * (K/16 + 8) with zmax the
largest partial sum's magnitude, taken as max|U| + max over (n, v) of sum_k
|x w|. lse is a maximum plus the log of a sum of exponentials with relative
error 2^-21 each (ex2.approx and the products before it): |lse error| <= that
+ 2^-20 + 2^-22 |lse|. The loss is lse - z: twice that. An entry of G =
w (p - [v = t]) has p's relative error (the z and lse errors, 2^-21) and one
rounding to bf16 (8 significant bits: 2^-8 relative); the products add exact terms in fp32 (2^-23
per 16 terms); the result is rounded to bf16 once more. So an entry of dX or
dW is off by at most 2^-8 |entry| + (2^-8 + e) * scale * sum |w| (p + [v = t])
|factor|, e the relative error of p plus the accumulation's.
"""

import math

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import DsparkError, LinearCE

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _mat(rows, cols, pad, std, dtype, g):
    """[rows, cols] with padded rows, the padding NaN: nothing may read it."""
    ld = -(-cols // 8) * 8 + pad
    t = torch.full((rows, ld), float("nan"), dtype=dtype, device="cuda")
    t[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda") * std
    return t[:, :cols]


def _inputs(N, K, V, layout="vk", U=False, pad=0, ignored=0.0, seed=3, wstd=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wstd = 2.0 / math.sqrt(K) if wstd is None else wstd
    X = _mat(N, K, pad, 1.0, BF16, g)
    W = _mat(*((V, K) if layout == "vk" else (K, V)), pad, wstd, BF16, g)
    Um = _mat(N, V, pad, 2.0, F32, g) if U else None
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    if ignored:
        t[torch.rand(N, generator=g, device="cuda") < ignored] = -1
    wt = torch.rand(N, generator=g, device="cuda") + 0.25
    return X, W, Um, t, wt


def _reference(X, W, U, t, wt, scale, layout):
    Xd, Wd = X.double(), W.double()
    Wd = Wd.t() if layout == "kv" else Wd           # [V, K]
    z = Xd @ Wd.t()
    zmax = float((Xd.abs() @ Wd.abs().t()).max())
    if U is not None:
        z = z + U.double()
        zmax += float(U[torch.isfinite(U)].abs().max()) if torch.isfinite(U).any() else 0.0
    lse = torch.logsumexp(z, 1)
    live = (t >= 0) & torch.isfinite(lse)
    t0 = t.clamp(min=0).long()
    zt = z.gather(1, t0[:, None])[:, 0]
    loss = torch.where(t >= 0, lse - zt, torch.zeros_like(lse))
    loss = torch.where((t >= 0) & (lse == -math.inf), torch.full_like(lse, math.inf), loss)
    w = (wt.double() if wt is not None else torch.ones_like(lse)) * live
    p = torch.where(live[:, None], torch.exp(z - torch.where(live, lse, torch.zeros_like(lse))[:, None]),
                    torch.zeros_like(z))
    hot = torch.zeros_like(z)
    hot[torch.arange(z.shape[0], device=z.device), t0] = 1.0
    G, Ga = w[:, None] * (p - hot), w[:, None].abs() * (p + hot)
    dX, dW = scale * (G @ Wd), scale * (G.t() @ Xd)
    aX, aW = abs(scale) * (Ga @ Wd.abs()), abs(scale) * (Ga.t() @ Xd.abs())
    if layout == "kv":
        dW, aW = dW.t(), aW.t()
    K, N, V = X.shape[1], X.shape[0], z.shape[1]
    ez = 2.0 ** -23 * zmax * (K / 16 + 8)
    el = ez + 2.0 ** -20 + 2.0 ** -22 * lse.abs()
    ep = float(ez + el[torch.isfinite(el)].max() if torch.isfinite(el).any() else ez) + 2.0 ** -20
    tol = {"lse": el, "loss": 2 * el,
           "dX": 2.0 ** -8 * 1.01 * dX.abs() + (2.0 ** -8 * 1.01 + ep + 2.0 ** -23 * (V / 16 + 64)) * aX + 1e-30,
           "dW": 2.0 ** -8 * 1.01 * dW.abs() + (2.0 ** -8 * 1.01 + ep + 2.0 ** -23 * (N / 16 + 64)) * aW + 1e-30}
    return {"loss": loss, "lse": lse, "dX": dX, "dW": dW}, tol


def _close(got, ref, tol, what):
    got = got.double()
    inf = torch.isinf(ref)
    assert (got[inf] == ref[inf]).all(), what
    d = (got - ref)[~inf].abs()
    assert torch.isfinite(d).all() and (d <= tol[~inf]).all(), (what, float(d.max()), float((d / tol[~inf]).max()))


def _check(X, W, U, t, wt, scale, layout, op=None, dx=True, dw=True):
    N, K = X.shape
    V = W.shape[0] if layout == "vk" else W.shape[1]
    op = op or LinearCE(N, K, V, layout)
    out = op.new_outputs(dx, dw)
    op.forward(X, W, t, U=U, out=out)
    assert op.device_status() == 0
    op.grad(X, W, t, out["lse"], wt=wt, scale=scale, U=U, out=out)
    assert op.device_status() == 0
    ref, tol = _reference(X, W, U, t, wt, scale, layout)
    for k in out:
        _close(out[k], ref[k], tol[k], k)
    return op, out


SHAPES = [
    # N, K, V, layout, U, pad, ignored
    (1, 1, 1, "vk", False, 0, 0.0),
    (1, 8, 5, "kv", True, 0, 0.0),
    (2, 3, 7, "vk", True, 8, 0.0),
    (6, 80, 1024, "vk", False, 0, 0.0),          # the tiny round's sizes
    (6, 16, 1024, "kv", True, 0, 0.0),
    (33, 64, 129, "vk", False, 0, 0.2),
    (127, 65, 255, "kv", False, 8, 0.0),
    (128, 256, 256, "vk", True, 0, 0.0),
    (129, 257, 257, "kv", True, 16, 0.5),
    (257, 100, 1001, "vk", False, 24, 0.1),
    (300, 192, 4104, "kv", True, 0, 0.0),
    (640, 256, 8200, "kv", True, 0, 0.0),
    (65, 1300, 515, "vk", False, 0, 0.0),
    (511, 320, 2500, "vk", False, 0, 0.0),
    (1025, 40, 300, "kv", False, 0, 0.0),
]


@pytest.mark.parametrize("N,K,V,layout,U,pad,ignored", SHAPES)
def test_values_and_gradients(N, K, V, layout, U, pad, ignored):
    X, W, Um, t, wt = _inputs(N, K, V, layout, U, pad, ignored)
    _check(X, W, Um, t, wt, 1.0 / N, layout)


def test_vocabulary_in_pieces():
    """N V large enough that G takes several pieces, the last one ragged, in both layouts."""
    for layout in ("vk", "kv"):
        X, W, U, t, wt = _inputs(4100, 72, 50001, layout, False, 0, 0.1)
        _check(X, W, U, t, wt, 0.5, layout)


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("N,K,V,U,pad,ignored", [
    (1, 16, 4097, True, 0, 0.0), (1, 700, 40000, False, 0, 0.0), (31, 264, 4100, True, 8, 0.1), (32, 65, 5000, False, 0, 0.3),
    (33, 1030, 4353, True, 0, 0.0), (63, 128, 24001, True, 8, 0.1), (64, 80, 33000, False, 0, 0.1), (65, 80, 33000, True, 0, 0.0),
    (7, 72, 3840, True, 0, 0.0), (7, 72, 3841, True, 0, 0.0),
])
def test_few_rows(N, K, V, U, pad, ignored, layout):
    """Up to 64 rows: the logits' product has tokens as its rows."""
    X, W, Um, t, wt = _inputs(N, K, V, layout, U, pad, ignored)
    _check(X, W, Um, t, wt, 0.5, layout)


@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_masks_with_few_rows(layout):
    V = 60000                       # several tiles to a warp
    X, W, U, t, wt = _inputs(40, 64, V, layout, True)
    U, t = U.clone(), t.clone()
    t[0], t[1], t[2], t[3], t[4], t[5], t[6] = 1, 30000, 59999, 500, 7, -1, 100
    U[0, ::2] = -math.inf
    U[1, :30000] = -math.inf        # whole tiles at the start
    U[2, :59999] = -math.inf        # the last token alone
    U[3, 500] = -math.inf           # the target
    U[4] = -math.inf                # nothing left
    U[5] = -math.inf
    U[6, 256:] = torch.finfo(F32).min
    U[7] = -1e30
    op = LinearCE(40, 64, V, layout)
    out = op.forward(X, W, t, U=U, out=op.new_outputs())
    op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, U=U, out=out)
    assert op.device_status() == 0
    masked = torch.where(U <= -1e30, torch.full_like(U, -math.inf), U)
    ref, tol = _reference(X, W, masked, t, wt, 1.0, layout)
    for k in out:
        _close(out[k], ref[k], tol[k], k)
    for dead in (4, 7):
        assert out["lse"][dead] == -math.inf and out["loss"][dead] == math.inf and (out["dX"][dead] == 0).all()
    assert out["lse"][5] == -math.inf and out["loss"][5] == 0 and (out["dX"][5] == 0).all()
    assert out["loss"][3] == math.inf
    for bad in (V, -2):             # a target out of range: reported, the row left out
        t[9] = bad
        got = op.forward(X, W, t, U=U, out=op.new_outputs())
        assert op.device_status() == 6
        op.reset()
        op.grad(X, W, t, got["lse"], wt=wt, U=U, out=got)
        assert op.device_status() == 6
        op.reset()
        assert got["loss"][9] == 0 and (got["dX"][9] == 0).all()


@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_whole_tiles_summed_over_pieces(layout):
    """dX has tiles for most of the grid, so that each is summed in place from piece to piece."""
    X, W, U, t, wt = _inputs(4100, 1000, 40003, layout, False, 0, 0.1)
    _check(X, W, U, t, wt, 1.0, layout)


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("N,K,V,U,pad,ignored", [
    (1500, 1001, 7003, False, 0, 0.1),     # ragged in every size, parts of tiles shared by pairs of CTAs
    (1030, 1300, 9000, True, 8, 0.0),
    (3000, 2100, 40003, False, 0, 0.2),    # many tiles, the second piece narrower than the first
])
def test_long_products(N, K, V, U, pad, ignored, layout):
    """N K V of 1e10 and more: dX or dW is made transposed, X's transpose is an operand."""
    X, W, Um, t, wt = _inputs(N, K, V, layout, U, pad, ignored)
    _check(X, W, Um, t, wt, 0.25, layout)


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("N,K,V,U", [
    (9, 200, 4800, True),                       # logits in tiles of 64 columns,
    (300, 130, 2561, True), (20, 72, 9473, False),   # of 128,
    (300, 130, 5121, True), (20, 72, 9729, False),   # of 256
    (70, 200, 4800, True), (65, 72, 9473, False), (129, 72, 9729, True),
    (33, 1025, 1100, True),                     # few tiles of a longer contraction
    (130, 260, 40001, False),                   # dX on some of the pairs, dW on the others
])
def test_widths_of_tiles(N, K, V, U, layout):
    X, W, Um, t, wt = _inputs(N, K, V, layout, U, 0, 0.1)
    _check(X, W, Um, t, wt, 1.0, layout)


@pytest.mark.parametrize("dx,dw", [(True, False), (False, True)])
@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_one_gradient_alone(dx, dw, layout):
    X, W, U, t, wt = _inputs(200, 136, 3000, layout, True)
    _check(X, W, U, t, None, 2.0, layout, dx=dx, dw=dw)


def test_large_logits():
    """Logits in the hundreds: the running maximum keeps the exponentials in range."""
    X, W, U, t, wt = _inputs(70, 64, 900, wstd=8.0)
    _check(X, W, U, t, wt, 1.0, "vk")


def test_masks():
    """-inf on single tokens, on a target, on all tokens of a row, on a whole tile; the type's lowest value as a mask."""
    X, W, U, t, wt = _inputs(40, 64, 1000, "vk", True)
    U = U.clone()
    t = t.clone()
    t[3], t[4], t[5], t[6], t[7], t[9] = 500, 10, 20, -1, 999, 600
    U[0, ::2] = -math.inf
    t[0] = 1
    U[1, :256] = -math.inf          # the first tile's columns
    t[1] = 300
    U[2, 1:] = -math.inf            # one token left, the target
    t[2] = 0
    U[3, 500] = -math.inf           # the target masked: loss +inf
    U[5] = -math.inf                # nothing left
    U[6] = -math.inf                # nothing left, and no target
    U[7, :999] = torch.finfo(F32).min
    U[8] = -1e30                    # a mask's value throughout: nothing left
    U[9, 256:512] = -math.inf
    U[10, int(t[10])] = torch.finfo(F32).min    # a target masked by the lowest value: loss +inf
    op = LinearCE(40, 64, 1000)
    out = op.forward(X, W, t, U=U, out=op.new_outputs())
    op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, U=U, out=out)
    assert op.device_status() == 0
    masked = torch.where(U <= -1e30, torch.full_like(U, -math.inf), U)
    ref, tol = _reference(X, W, masked, t, wt, 1.0, "vk")
    for k in out:
        _close(out[k], ref[k], tol[k], k)
    for dead in (5, 8):
        assert out["lse"][dead] == -math.inf and out["loss"][dead] == math.inf and (out["dX"][dead] == 0).all()
    assert out["lse"][6] == -math.inf and out["loss"][6] == 0 and (out["dX"][6] == 0).all()
    assert out["loss"][3] == math.inf and out["loss"][10] == math.inf


def test_nan_and_infinity_stay_in_their_row():
    X, W, U, t, wt = _inputs(30, 64, 700, "vk", True)
    U = U.clone()
    U[4, 17], U[5, 300], t[6] = math.nan, math.inf, -1
    U[6, 3] = math.nan              # a row left out keeps its NaN out of the gradients
    op = LinearCE(30, 64, 700)
    out = op.forward(X, W, t, U=U, out=op.new_outputs(dw=False))
    op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, U=U, out=out)
    for bad in (4, 5):
        assert torch.isnan(out["lse"][bad]) and torch.isnan(out["loss"][bad]) and torch.isnan(out["dX"][bad]).all()
    assert out["loss"][6] == 0 and (out["dX"][6] == 0).all()
    good = [i for i in range(30) if i not in (4, 5, 6)]
    ref, tol = _reference(X[good], W, U[good], t[good], wt[good], 1.0, "vk")
    for k in out:
        _close(out[k][good], ref[k], tol[k], k)


def test_targets_out_of_range_are_reported():
    X, W, U, t, wt = _inputs(20, 64, 700)
    for bad in (700, -2, 2 ** 31 - 1, -2 ** 31):
        t2 = t.clone()
        t2[3] = bad
        op = LinearCE(20, 64, 700)
        out = op.forward(X, W, t2, out=op.new_outputs())
        assert op.device_status() == 6       # DSPARK_ERANGE
        op.reset()
        op.grad(X, W, t2, out["lse"], wt=wt, out=out)
        assert op.device_status() == 6
        op.reset()
        t2[3] = -1
        ref = op.forward(X, W, t2, out=op.new_outputs())
        assert op.device_status() == 0
        op.grad(X, W, t2, ref["lse"], wt=wt, out=ref)
        for k in out:
            assert torch.equal(out[k], ref[k]), k


def test_no_rows_and_all_rows_left_out():
    W = torch.randn(50, 16, device="cuda").bfloat16()
    op = LinearCE(0, 16, 50)
    out = op.new_outputs()
    out["dW"].fill_(7.0)
    X, t = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    op.forward(X, W, t, out=out)
    op.grad(X, W, t, out["lse"], out=out)
    assert (out["dW"] == 0).all()
    X, W, U, t, wt = _inputs(70, 16, 50)
    t.fill_(-1)
    op = LinearCE(70, 16, 50)
    out = op.forward(X, W, t, out=op.new_outputs())
    op.grad(X, W, t, out["lse"], wt=wt, out=out)
    assert (out["loss"] == 0).all() and (out["dX"] == 0).all() and (out["dW"] == 0).all()
    assert torch.isfinite(out["lse"]).all()


def test_padding_of_the_outputs_is_left_alone():
    for layout, N, K, V in (("vk", 70, 50, 300), ("kv", 70, 50, 301), ("vk", 2050, 1250, 5003), ("kv", 2050, 1250, 5003)):
        X, W, U, t, wt = _inputs(N, K, V, layout)
        op = LinearCE(N, K, V, layout)
        out = op.new_outputs(False, False)
        k64, v64 = -(-K // 64) * 64, -(-V // 64) * 64
        full = {"dX": torch.full((N, k64), 9.0, dtype=BF16, device="cuda"),
                "dW": torch.full((V, k64) if layout == "vk" else (K, v64), 9.0, dtype=BF16, device="cuda")}
        cols = {"dX": K, "dW": K if layout == "vk" else V}
        for k in full:
            out[k] = full[k][:, :cols[k]]
        _, plain = _check(X, W, U, t, wt, 1.0, layout)
        op.forward(X, W, t, out=out)
        op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, out=out)
        for k in full:
            assert (full[k][:, cols[k]:] == 9.0).all(), k
            assert torch.equal(full[k][:, :cols[k]], plain[k]), k


def test_same_result_each_time_and_on_another_stream():
    X, W, U, t, wt = _inputs(300, 96, 5000, "kv", True)
    op, first = _check(X, W, U, t, wt, 1.0, "kv")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = op.new_outputs()
        side.wait_stream(torch.cuda.current_stream())
        op.forward(X, W, t, U=U, out=out, stream=side)
        op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, U=U, out=out, stream=side)
        side.synchronize()
        for k in out:
            assert torch.equal(out[k], first[k]), k


def test_captured_in_a_graph():
    X, W, U, t, wt = _inputs(100, 64, 2000)
    op, first = _check(X, W, U, t, wt, 1.0, "vk")
    out = op.new_outputs()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(X, W, t, out=out)
        op.grad(X, W, t, out["lse"], wt=wt, scale=1.0, out=out)
    for k in out:
        out[k].zero_()
    g.replay()
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k], first[k]), k


def test_gradient_against_differences():
    """The loss along a direction, by central differences of the kernel's own
    losses. X, W and the step lie on a grid that bf16 holds exactly. The
    difference's error is a sixth of the third derivative, and the third
    cumulant of a row's logits' change over its tokens is at most
    r^3 / (6 sqrt 3), r its range; the losses add their own tolerance, the
    gradient its own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    N, K, V, step = 24, 40, 500, 2.0 ** -4

    def grid(*shape):
        return torch.randint(-32, 33, shape, generator=g, device="cuda").float() * step

    X, W = grid(N, K).bfloat16(), (grid(V, K) / 4).bfloat16()
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    wt = torch.rand(N, generator=g, device="cuda") + 0.5
    op, out = _check(X, W, None, t, wt, 1.0, "vk")
    _, tol = _reference(X, W, None, t, wt, 1.0, "vk")

    def total(a, b):
        return float((op.forward(a, b, t)["loss"].double() * wt.double()).sum())

    loss_tol = float((tol["loss"] * wt.double()).sum())
    for which in ("dX", "dW"):
        M = X if which == "dX" else W
        unit = step if which == "dX" else step / 4
        sign = torch.where(torch.rand(M.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        d = torch.where(torch.rand(M.shape, generator=g, device="cuda") < 0.05, unit * sign, torch.zeros_like(sign))
        hi, lo = (M.float() + d).bfloat16(), (M.float() - d).bfloat16()
        assert torch.equal(hi.float() - M.float(), d) and torch.equal(M.float() - lo.float(), d)
        if which == "dX":
            diff = (total(hi, W) - total(lo, W)) / 2
            dz = d.double() @ W.double().t()
        else:
            diff = (total(X, hi) - total(X, lo)) / 2
            dz = X.double() @ d.double().t()
        r = dz.amax(1) - dz.amin(1)
        third = float((wt.double() * r ** 3).sum()) / (36 * math.sqrt(3))
        along = float((out[which].double() * d.double()).sum())
        along_tol = float((tol[which] * d.abs().double()).sum())
        assert abs(diff - along) <= third + loss_tol + along_tol, (which, diff, along, third, loss_tol, along_tol)


def test_offsets_past_32_bits():
    """W and dW of 2.2e9 values, U rows 2^31 values apart from end to end; the reference in pieces of the vocabulary."""
    N, K, V = 2000, 8, 1_100_003
    g = torch.Generator(device="cuda").manual_seed(9)
    U = torch.randn(N, -(-V // 4) * 4, generator=g, device="cuda")[:, :V]
    X = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    W = torch.randn(V, K, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    t[N - 1] = V - 1
    rows = [0, 7, N - 2, N - 1]
    op = LinearCE(N, K, V)
    out = op.forward(X, W, t, U=U, out=op.new_outputs(dw=False))
    op.grad(X, W, t, out["lse"], scale=1.0, U=U, out=out)
    assert op.device_status() == 0
    ref, tol = _reference(X[rows], W, U[rows], t[rows], None, 1.0, "vk")
    for k in out:
        _close(out[k][rows], ref[k], tol[k], k)
    del U, out, op
    N, K, V = 24, 2048, 1_100_003
    X = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    W = torch.empty(V, K, dtype=BF16, device="cuda").normal_(0.0, 0.03, generator=g)
    t = torch.randint(V - 200, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    op = LinearCE(N, K, V)
    out = op.forward(X, W, t, out=op.new_outputs(dx=False))
    op.grad(X, W, t, out["lse"], scale=1.0, out=out)
    assert op.device_status() == 0
    z = torch.cat([X.double() @ W[a:a + 100_000].double().t() for a in range(0, V, 100_000)], 1)
    lse = torch.logsumexp(z, 1)
    zmax = 2.0 * float(z.abs().max()) + 0.03 * K        # the partial sums' magnitude: sum |x w| <= 0.03 K on average
    ez = 2.0 ** -23 * zmax * (K / 16 + 8)
    el = ez + 2.0 ** -20 + 2.0 ** -22 * lse.abs()
    _close(out["lse"], lse, el, "lse")
    a = V - 300                                          # the last rows of dW, the targets among them
    p = torch.exp(z[:, a:] - lse[:, None])
    hot = torch.zeros_like(p)
    hot[torch.arange(N, device="cuda"), t.long() - a] = 1.0
    ref = (p - hot).t() @ X.double()
    mag = (p + hot).t() @ X.double().abs()
    tol = 2.0 ** -8 * 1.01 * ref.abs() + (2.0 ** -8 * 1.01 + float(ez + el.max()) + 2.0 ** -20 + 2.0 ** -23 * 66) * mag
    _close(out["dW"][a:], ref, tol + 1e-30, "dW")


def test_refusals():
    X, W, U, t, wt = _inputs(20, 64, 300, "vk", True)
    op = LinearCE(20, 64, 300)
    out = op.forward(X, W, t, out=op.new_outputs())
    bad = [
        dict(X=X.float()), dict(W=W.float()), dict(U=U.bfloat16()), dict(target=t.long()),
        dict(X=X[:19]), dict(W=W[:, :32]), dict(U=U[:, :299]), dict(target=t[:19]),
        dict(X=X.t().contiguous().t()), dict(X=X.cpu()),
        dict(X=torch.zeros(20, 65, dtype=BF16, device="cuda")[:, :64]),      # row stride not a multiple of 8
        dict(X=torch.zeros(20, 72, dtype=BF16, device="cuda")[:, 1:65]),     # rows not on 16 bytes
        dict(U=torch.zeros(20, 301, device="cuda")[:, :300]),
    ]
    for change in bad:
        a = {**dict(X=X, W=W, target=t, U=U), **change}
        with pytest.raises(DsparkError):
            op.forward(a["X"], a["W"], a["target"], U=a["U"])
        with pytest.raises(DsparkError):
            op.grad(a["X"], a["W"], a["target"], out["lse"], U=a["U"], out=op.new_outputs())
    with pytest.raises(DsparkError):
        op.grad(X, W, t, out["lse"].double())
    with pytest.raises(DsparkError):
        op.grad(X, W, t, out["lse"], wt=wt[:5])
    with pytest.raises(DsparkError):
        op.grad(X, W, t, out["lse"], out={"loss": out["loss"]})              # no gradient asked for
    for dims in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (2 ** 20 + 1, 8, 8), (8, 65537, 8), (8, 8, 2 ** 24 + 1)):
        with pytest.raises(DsparkError):
            LinearCE(*dims)
    with pytest.raises(DsparkError):
        LinearCE(8, 8, 8, layout="kk")
