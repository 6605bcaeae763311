"""What the training operators' calls make when they are given another stream."""

import pytest
import torch

from speculative_decoding_head_gb300 import build
from speculative_decoding_head_gb300.binding import Embedding, GradClip, LinearCE

from test_gpu_embed import _gen, _idx
from test_gpu_linear_ce import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_what_an_embedding_makes_belongs_to_its_stream():
    """Scratch and results that a call on another stream makes come from that
    stream's memory: a block just freed on the current stream, whose work may still be going on there, is not taken."""
    N, V, D = 3000, 5000, 64
    idx, g = _idx(N, V, "zipf"), _gen(4)
    dout = torch.randn(N, D, generator=g, device="cuda")
    op = Embedding(N, V, D)
    want = op.grad(dout, idx)
    rows = op.lookup(want, idx)
    side = torch.cuda.Stream()
    op = Embedding(N, V, D)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (op._bytes, 4 * V * D, 4 * N * D)]
    blocks = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in freed]
    del freed
    got = op.grad(dout, idx, stream=side)
    got2 = op.lookup(got, idx, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, rows)
    for t in (op.scratch, got, got2):
        assert not any(a <= t.data_ptr() < b for a, b in blocks)


def test_what_a_cross_entropy_makes_belongs_to_its_stream():
    """Results that a call on another stream makes come from that stream's
    memory, not from a block just freed on the current one."""
    N, K, V = 3000, 64, 900
    X, W, _, t, wt = _inputs(N, K, V)
    op, first = _check(X, W, None, t, wt, 1.0, "vk")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (4 * N, 4 * N, 2 * N * K, 2 * V * K)]
    blocks = [(x.data_ptr(), x.data_ptr() + x.numel()) for x in freed]
    del freed
    got = op.forward(X, W, t, stream=side)
    grads = op.grad(X, W, t, got["lse"], wt=wt, scale=1.0, stream=side)
    side.synchronize()
    for x, ref in ((got["loss"], first["loss"]), (got["lse"], first["lse"]), (grads["dX"], first["dX"]),
                   (grads["dW"], first["dW"])):
        assert torch.equal(x, ref) and not any(a <= x.data_ptr() < b for a, b in blocks)


@pytest.mark.parametrize("given", [True, False])
def test_an_objects_memory_outlives_its_streams_work(given):
    """An object dropped while another stream still works with its buffers: their
    memory does not go to the stream that it was made on before that work has ended."""
    N, V, D = 3000, 5000, 64
    idx, g = _idx(N, V, "zipf"), _gen(4)
    dout, out = torch.randn(N, D, generator=g, device="cuda"), torch.empty(V, D, device="cuda")
    X, W, _, t, wt = _inputs(N, D, V)
    side = torch.cuda.Stream()
    ops = [Embedding(N, V, D), LinearCE(N, D, V), GradClip([dout])]
    grads = ops[1].new_outputs()
    ops[0].grad(dout, idx, out=out)             # its scratch is made on the current stream
    ops[1].forward(X, W, t, out=grads)
    ops[1].grad(X, W, t, grads["lse"], wt=wt, out=grads)    # every kernel is loaded now: loading one waits for the device
    ops[2].clip(1e9)
    sizes = [op.scratch.numel() for op in ops]
    blocks = [(op.scratch.data_ptr(), op.scratch.data_ptr() + op.scratch.numel()) for op in ops]
    torch.cuda.synchronize()
    kw = {"stream": side} if given else {}
    with torch.cuda.stream(None if given else side):
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)      # a fifth of a second
        ops[0].grad(dout, idx, out=out, **kw)
        ops[1].grad(X, W, t, grads["lse"], wt=wt, out=grads, **kw)
        ops[2].clip(1e9, **kw)
    del ops
    made = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not side.query()                     # else the machine was too slow for this test to say anything
    for m in made:
        assert not any(a <= m.data_ptr() < b for a, b in blocks)
    side.synchronize()
