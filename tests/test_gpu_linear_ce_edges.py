"""The linear cross entropy where it can go wrong: rows left out, batches without rows, early starts, pieces, long sums.

Tolerances are those of test_gpu_linear_ce.py where nothing else is said.
"""

import ctypes as C
import math
import subprocess

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import LinearCE

from test_gpu_linear_ce import BF16, F64, _check, _close, _inputs, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("N,K,V", [(40, 70, 1000), (40, 64, 5000), (300, 136, 3000), (1500, 1001, 7003), (4100, 72, 50001)])
def test_rows_left_out_hold_anything(N, K, V, layout):
    """NaN and infinities in rows of X and U that are left out (no target, or
    one out of range) reach no entry of dW; nor does a row with every token masked."""
    X, W, U, t, wt = _inputs(N, K, V, layout, True, 8, 0.1)
    t[0] = t[N - 1] = -1
    t[1], t[2] = V, 3
    U[2] = -math.inf
    dead = torch.nonzero((t < 0) | (t >= V))[:, 0]
    clean = X.clone()
    clean[dead] = 0.0
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        X[dead[i::3], i::2] = bad
    U[dead[::2], ::3] = math.nan
    op = LinearCE(N, K, V, layout)
    out = op.forward(X, W, t, U=U, out=op.new_outputs())
    op.grad(X, W, t, out["lse"], wt=wt, scale=0.5, U=U, out=out)
    assert op.device_status() == 6              # the target out of range
    t[1] = -1
    U[dead] = 0.0
    ref, tol = _reference(clean, W, U, t, wt, 0.5, layout)
    assert (out["loss"][dead] == 0).all() and (out["dX"][dead] == 0).all()
    for k in ("dX", "dW"):
        _close(out[k], ref[k], tol[k], k)
    alone = op.new_outputs(dx=False)
    op.grad(X, W, t, out["lse"], wt=wt, scale=0.5, U=U, out=alone)
    assert torch.equal(alone["dW"], out["dW"])


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("dx,dw", [(True, False), (False, True)])
def test_no_rows_and_one_gradient(dx, dw, layout):
    """A batch without rows is allowed whichever gradient is asked for (an empty dX has no address)."""
    op = LinearCE(0, 16, 50, layout)
    out = op.new_outputs(dx, dw)
    if dw:
        out["dW"].fill_(7.0)
    X, t = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    W = torch.randn(*op.w_shape, device="cuda").bfloat16() if layout == "vk" else (
        torch.randn(16, 56, device="cuda").bfloat16()[:, :50])
    op.grad(X, W, t, out["lse"], out=out)
    assert op.device_status() == 0
    if dw:
        assert (out["dW"] == 0).all()


LATE = r"""
#include <cuda_runtime.h>
#include <stdint.h>
// Lets the kernel that follows start at once, then takes ms milliseconds and copies n pieces.
__global__ void late(const uint4* src, uint4* dst, int n, unsigned long long ms) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 1000000; ++i) {
    __nanosleep(1000);
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > ms * 1000000ull) break;
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int run_late(const void* src, void* dst, int n, int ms, void* stream) {
  late<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint4*>(src), static_cast<uint4*>(dst), n,
                                                         ms);
  return cudaGetLastError();
}
"""


@pytest.mark.parametrize("N,K,V,layout", [(6, 80, 1024, "vk"), (6, 80, 5000, "vk"), (300, 64, 2000, "kv"),
                                          (1500, 1000, 7000, "vk")])
def test_behind_a_long_kernel_that_lets_it_start(N, K, V, layout, tmp_path_factory):
    """A kernel that lets its dependents start early and then runs 0.6 s, longer
    than any wait of the operator's own may last, delays a call and no more."""
    at = tmp_path_factory.getbasetemp() / "late.so"
    if not at.exists():
        src = at.with_suffix(".cu")
        src.write_text(LATE)
        subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", str(at), str(src)], check=True)
    late = C.CDLL(str(at)).run_late
    late.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]
    X, W, _, t, wt = _inputs(N, K, V, layout)
    op, first = _check(X, W, None, t, wt, 1.0, layout)
    keep = X.contiguous().clone()
    X2 = torch.zeros_like(keep)                  # K is a multiple of 8: rows on 16 bytes without padding
    out = op.new_outputs()
    stream = torch.cuda.current_stream().cuda_stream

    def delay():
        X2.zero_()
        assert late(keep.data_ptr(), X2.data_ptr(), keep.numel() // 8, 600, stream) == 0

    delay()
    op.forward(X2, W, t, out=out)
    delay()
    op.grad(X2, W, t, out["lse"], wt=wt, scale=1.0, out=out)
    assert op.device_status() == 0
    for k in first:
        assert torch.equal(out[k], first[k]), k


def _launches(op, *a, **kw):
    """Kernels of one gradient call (the nodes of a graph that records it)."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        op.grad(*a, **kw)
    n = C.c_size_t(0)
    assert C.CDLL("libcudart.so.13").cudaGraphGetNodes(C.c_void_p(g.raw_cuda_graph()), None, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("layout", ["vk", "kv"])
@pytest.mark.parametrize("N,K,V,U", [(64, 16, 600003, True), (33, 24, 1100003, False)])
def test_few_rows_and_pieces(N, K, V, U, layout):
    """Tokens as rows of the logits' product, the vocabulary in two pieces:
    targets at both sides of where the second begins, and at the ends."""
    X, W, Um, t, wt = _inputs(N, K, V, layout, U, 0, 0.1)
    half = -(-(-(-V // 2)) // 256) * 256
    t[:8] = torch.tensor([half - 1, half, half + 1, half - 257, half + 255, 0, V - 1, -1], dtype=torch.int32)
    op, out = _check(X, W, Um, t, wt, 1.0, layout)
    # a launch that makes G alone, one a piece, and at most the transpose and a join
    assert 3 <= _launches(op, X, W, t, out["lse"], wt=wt, U=Um, out=out) <= 5
    one = LinearCE(N, K, 10000, layout)
    w = W[:10000] if layout == "vk" else W[:, :10000]
    u = Um[:, :10000] if U else None
    assert _launches(one, X, w, t % 10000, out["lse"], wt=wt, U=u, out=one.new_outputs()) < _launches(
        op, X, W, t, out["lse"], wt=wt, U=Um, out=out)


@pytest.mark.parametrize("layout", ["vk", "kv"])
def test_long_contraction_and_pieces(layout):
    """K of 1024 and more and several pieces, the last one narrower, with targets about their edge."""
    N, K, V = 4100, 1030, 40003
    X, W, _, t, wt = _inputs(N, K, V, layout, False, 0, 0.1)
    half = -(-(-(-V // 2)) // 256) * 256
    t[:4] = torch.tensor([half - 1, half, 0, V - 1], dtype=torch.int32)
    op, out = _check(X, W, None, t, wt, 1.0, layout)
    assert _launches(op, X, W, t, out["lse"], wt=wt, out=out) >= 4     # the transpose, G alone, a launch a piece


@pytest.mark.parametrize("layout,U", [("vk", False), ("vk", True), ("kv", False)])
@pytest.mark.parametrize("N,K", [(192, 4096), (128, 16384), (48, 4096)])
def test_what_the_accumulator_cuts_off_is_made_up_for(N, K, layout, U):
    """The mean over rows of lse's signed error. Cut once per 16 terms, a sum of n
    steps that grows evenly loses 0.36 2^-23 (n + 1) / 2 of itself, so that
    uncorrected lse is off by that times E_p[x w] (the logit's product part). At
    least half of it has to be made up for: a factor left out, twice as large,
    applied to U too or of the wrong sign is off by all of it or more. Beside it
    there is lse's own rounding, of mean zero over the rows: 2^-24 |lse|."""
    V = 8192
    X, W, Um, t, _ = _inputs(N, K, V, layout, U)
    lse = LinearCE(N, K, V, layout).forward(X, W, t, U=Um)["lse"].double()
    dot = X.double() @ (W.double().t() if layout == "vk" else W.double())
    z = dot + Um.double() if U else dot
    ref = torch.logsumexp(z, 1)
    shift = 0.36 * 2.0 ** -23 * (K / 16 + 1) / 2 * float((torch.softmax(z, 1) * dot).sum(1).mean())
    mean = float((lse - ref).mean())
    print(f"shift {shift:.3e}, mean error {mean:.3e}")
    assert abs(mean) <= 0.5 * shift + 2.0 ** -24 * float(ref.abs().mean()), (mean, shift)


@pytest.mark.parametrize("K", [4096, 65536])
def test_logits_that_do_not_grow_evenly(K):
    """The correction at its worst. Row 0's terms all come last (its sums are
    cut once or twice): off by the whole factor. Row 1 grows to +-A and comes back to a
    small rest: off by what is cut on the way, one unit of A per 16 terms at most."""
    V = 1024
    g = torch.Generator(device="cuda").manual_seed(11)
    X = torch.zeros(2, K, dtype=BF16, device="cuda")
    X[0, K - 16:] = torch.randn(16, generator=g, device="cuda").bfloat16()
    X[1] = 1.0
    X[1, K // 2:] = -1.0
    W = torch.empty(V, K, dtype=BF16, device="cuda")
    W[:, :K // 2] = (torch.rand(V, K // 2, generator=g, device="cuda") * 0.25).bfloat16()
    W[:, K // 2:] = W[:, :K // 2]
    W[:, K - 16:] += torch.randn(V, 16, generator=g, device="cuda").bfloat16()
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = LinearCE(2, K, V).forward(X, W, t)
    z = X.double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    peak = float((X.double()[1, :K // 2] @ W.double()[:, :K // 2].t()).max())
    step = 2.0 ** -23
    bound = torch.tensor([0.36 * step * (K / 16 + 1) / 2 * float(z[0].abs().max()) + 4 * step * float(z[0].abs().max()),
                          step * peak * (K / 16 + 8)], device="cuda", dtype=F64)
    err = (out["lse"].double() - lse).abs()
    print(f"K {K}: lse error {err.tolist()}, bound {bound.tolist()}")
    assert (err <= bound + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all(), (err, bound)
