"""The gradients' norm and clipping on the GPU against the formulas in 64 bits.

Tolerances. Squares of at most 32 values are summed in fp32 in four chains (8
fused steps and two additions: 10 * 2^-24 relative, all terms positive), the
rest in fp64; the root halves that, and the norm is rounded to fp32:
|error| <= 2^-20 relative. The factor is fp32 (2^-24) and carries the norm's
error; a scaled value is one fp32 product rounded to its type.
"""

import math

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import DsparkError, GradClip

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
UNIT = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
NORM_TOL = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _make(sizes, kinds, std=1.0, shift=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        flat = torch.full((n + shift + 3,), float("nan"), dtype=kinds[i % len(kinds)], device="cuda")
        t = flat[shift:shift + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * std)
        out.append(t)
    return out


def _norm(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def _check(ts, max_norm, in_place=False):
    norm = _norm(ts)
    coef = min(1.0, max_norm / (norm + 1e-6))
    ref = [t.double() * coef for t in ts]
    outs = None if in_place else [torch.full_like(t, 3.0) for t in ts]
    op = GradClip(ts, outs)
    got = op.clip(max_norm)
    assert op.device_status() == 0
    assert abs(float(got) - norm) <= NORM_TOL * norm, (float(got), norm)
    for t, r in zip(op.outs, ref):
        d = (t.double() - r).abs()
        assert (d <= (NORM_TOL + 2.0 ** -23 + UNIT[t.dtype]) * 1.001 * r.abs() + 1e-44).all(), float(d.max())
    return op


SIZES = [[1], [7, 8, 9], [0, 5, 0], [32768, 32767, 32769, 1], [100003, 3, 64], [4096] * 40]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("kinds", [[BF16], [F32], [BF16, F32]])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_norm_and_scaling(sizes, kinds, shift):
    for max_norm in (0.5, 1e6):
        _check(_make(sizes, kinds, shift=shift), max_norm)
        _check(_make(sizes, kinds, shift=shift), max_norm, in_place=True)


@pytest.mark.parametrize("count", [31, 32, 33, 511, 512, 513, 1200])
def test_many_tensors(count):
    _check(_make([1 + (i * 37) % 900 for i in range(count)], [BF16, F32]), 2.0)


def test_large_list():
    _check(_make([30_000_001, 20_000_000, 5], [F32, BF16]), 1.0)


def test_a_tensor_past_32_bits():
    n = 2 ** 31 + 11
    x = torch.zeros(n, dtype=BF16, device="cuda")
    x[0], x[2 ** 31 - 1], x[n - 1] = 3.0, 4.0, 12.0
    op = GradClip([x])
    assert abs(float(op.clip(6.5)) - 13.0) <= 13.0 * NORM_TOL and op.device_status() == 0
    assert float(x[0]) == 1.5 and float(x[2 ** 31 - 1]) == 2.0 and float(x[n - 1]) == 6.0
    assert int(torch.count_nonzero(x[:2 ** 30])) == 1


def test_within_the_norm_nothing_changes():
    ts = _make([1000, 333], [BF16, F32])
    keep = [t.clone() for t in ts]
    _check(ts, 1e9, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    op = _check(ts, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(op.outs, keep))


def test_zero_and_empty():
    for ts in ([torch.zeros(100, device="cuda")], [torch.zeros(0, device="cuda")], []):
        op = GradClip(ts, [torch.ones_like(t) for t in ts])
        assert float(op.clip(1.0)) == 0.0 and op.device_status() == 0
        assert all((o == 0).all() for o in op.outs)
    ts = _make([100], [F32])
    op = GradClip(ts)
    op.clip(0.0)                                   # a largest norm of zero
    assert (ts[0] == 0).all()


@pytest.mark.parametrize("std", [1e-30, 1e-20, 1e-16, 1e15, 1e19, 1e30])
@pytest.mark.parametrize("kinds", [[BF16], [F32]])
def test_squares_out_of_range(std, kinds):
    """Values whose squares overflow or vanish in fp32; a small share among ordinary ones too."""
    _check(_make([5000, 17], kinds, std=std), math.inf)
    mixed = _make([5000], kinds, std=std) + _make([40], kinds, std=1.0, seed=2)
    mixed.append(torch.cat([mixed[0][:100], mixed[1]]))
    _check(mixed, math.inf)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(bad):
    for kinds in ([BF16], [F32]):
        ts = _make([100, 70000], kinds)
        ts[1][65432] = bad
        keep = [t.clone() for t in ts]
        op = GradClip(ts)
        norm = float(op.clip(1.0))
        assert not math.isfinite(norm) and op.device_status() == 4      # DSPARK_ENUMERIC
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(ts, keep))
        op.reset()
        ts[1][65432] = 0.0
        assert math.isfinite(float(op.clip(1.0))) and op.device_status() == 0


def test_same_result_each_time_and_on_another_stream():
    ts = _make([200_000, 70_001], [BF16, F32])
    op = _check(ts, 1.0)
    first, norm = [o.clone() for o in op.outs], float(op.norm)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in op.outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        op.clip(1.0, stream=side)
        side.synchronize()
        assert float(op.norm) == norm and all(torch.equal(a, b) for a, b in zip(op.outs, first))


def test_refusals():
    x = torch.zeros(10, device="cuda")
    for bad in (lambda: GradClip([x.half()]), lambda: GradClip([x.cpu()]), lambda: GradClip([x[::2]]),
                lambda: GradClip([x], []), lambda: GradClip([x], [x[:5]]), lambda: GradClip([x], [x.bfloat16()]),
                lambda: GradClip([x]).clip(-1.0), lambda: GradClip([x]).clip(math.nan)):
        with pytest.raises(DsparkError):
            bad()
