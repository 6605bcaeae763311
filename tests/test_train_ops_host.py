"""What the training operators' binding does on the host, on stand-ins for tensors of several devices.

Runs without a GPU: nothing is launched.
"""

import ctypes as C

import pytest
import torch

from speculative_decoding_head_gb300 import binding, build
from speculative_decoding_head_gb300.binding import DsparkError

ZERO, ONE = torch.device("cuda", 0), torch.device("cuda", 1)


class Stand:
    """What the binding looks at of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = shape, dtype, device
        self.streams = []

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (*self.shape[1:], 1)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        self.streams.append(stream)


class FakeLib:
    """Records which device was current at each call."""

    def __init__(self, current):
        self.current, self.calls = current, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current[-1], args[-1]))
            return 0
        return call


class FakeStream:
    def __init__(self, device, address):
        self.device, self.cuda_stream = device, address


@pytest.fixture
def devices(monkeypatch):
    """Device 0 is current; torch's ways to the current device and streams answer for two devices."""
    current = [0]

    class On:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(binding, "_current_device", lambda: current[-1])
    monkeypatch.setattr(binding, "_current_stream", lambda index: 1000 + index)
    monkeypatch.setattr(binding.torch.cuda, "device", On)
    monkeypatch.setattr(binding.torch.cuda, "current_stream", lambda d: FakeStream(torch.device(d), 1000 + d.index))
    return current


def _object(cls, current, device, **fields):
    op = object.__new__(cls)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(binding.torch, "zeros", lambda n, dtype, device: Stand((n,), dtype, device))
        binding._TrainOp.__init__(op, device)
    op.lib, op.scratch = FakeLib(current), Stand((64,), torch.uint8, device)
    for k, v in fields.items():
        setattr(op, k, v)
    return op


def _lce(current, device):
    dims = binding.LceDims(8, 16, 32, 0)
    return _object(binding.LinearCE, current, device, N=8, K=16, V=32, layout="vk", _dims=dims, _pdims=C.byref(dims))


def _lce_tensors(device):
    bf, f, i = torch.bfloat16, torch.float32, torch.int32
    return {"X": Stand((8, 16), bf, device), "W": Stand((32, 16), bf, device), "target": Stand((8,), i, device),
            "lse": Stand((8,), f, device), "wt": Stand((8,), f, device), "U": Stand((8, 32), f, device),
            "out": {"loss": Stand((8,), f, device), "lse": Stand((8,), f, device), "dX": Stand((8, 16), bf, device),
                    "dW": Stand((32, 16), bf, device)}}


def test_calls_run_on_the_objects_device(devices):
    ce, t = _lce(devices, ONE), _lce_tensors(ONE)
    ce.forward(t["X"], t["W"], t["target"], U=t["U"], out=t["out"])
    ce.grad(**t)
    emb = _object(binding.Embedding, devices, ONE, N=8, V=32, D=16, _bytes=64)
    E, idx, rows = (Stand((32, 16), torch.float32, ONE), Stand((8,), torch.int32, ONE), Stand((8, 16), torch.float32, ONE))
    emb.lookup(E, idx, out=rows)
    emb.grad(rows, idx, out=E)
    clip = _object(binding.GradClip, devices, ONE, count=0, _in=None, _out=None, _shape=(None,), _types=None,
                   norm=Stand((), torch.float32, ONE))
    clip._f = clip.lib.dspark_clip_grads
    clip.clip(1.0)
    calls = ce.lib.calls + emb.lib.calls + clip.lib.calls
    assert len(calls) == 5
    # device 1 was current at each launch, the stream was device 1's, and device 0 is current again
    assert all(device == 1 and stream == 1001 for _, device, stream in calls) and devices == [0]
    here = _lce(devices, ZERO)
    t = _lce_tensors(ZERO)
    here.forward(t["X"], t["W"], t["target"], out=t["out"])
    assert here.lib.calls[0][1:] == (0, 1000)


@pytest.mark.parametrize("name", ["X", "W", "target", "lse", "wt", "U", "dX", "dW"])
def test_tensors_of_another_device_are_refused(devices, name):
    ce, t, other = _lce(devices, ONE), _lce_tensors(ONE), _lce_tensors(ZERO)
    if name in t:
        t[name] = other[name]
    else:
        t["out"][name] = other["out"][name]
    with pytest.raises(DsparkError):
        ce.grad(**t)
    assert not ce.lib.calls


def test_embedding_tensors_of_another_device_are_refused(devices):
    def args(**at):
        f = torch.float32
        return {k: Stand(s, f if k != "idx" else torch.int32, at.get(k, ONE))
                for k, s in (("E", (32, 16)), ("idx", (8,)), ("out", (8, 16)))}

    emb = _object(binding.Embedding, devices, ONE, N=8, V=32, D=16, _bytes=64)
    for name in ("E", "idx", "out"):
        with pytest.raises(DsparkError):
            emb.lookup(**args(**{name: ZERO}))
        a = args(**{name: ZERO})
        with pytest.raises(DsparkError):
            emb.grad(a["out"], a["idx"], out=a["E"])
        a = args()
        with pytest.raises(DsparkError):
            emb.grad(a["out"], a["idx"], base=Stand((32, 16), torch.float32, ZERO), out=a["E"])
    assert not emb.lib.calls


def test_gradients_on_two_devices_are_refused(monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: None)
    a, b = (Stand((4,), torch.float32, d) for d in (ZERO, ONE))
    with pytest.raises(DsparkError):
        binding.GradClip([a, b])
    with pytest.raises(DsparkError):
        binding.GradClip([a], [b])


def test_streams_of_another_device_are_refused(devices):
    ce, t = _lce(devices, ONE), _lce_tensors(ONE)
    with pytest.raises(DsparkError):
        ce.forward(t["X"], t["W"], t["target"], out=t["out"], stream=FakeStream(ZERO, 77))
    assert not ce.lib.calls
    ce.forward(t["X"], t["W"], t["target"], out=t["out"], stream=FakeStream(ONE, 77))
    assert ce.lib.calls[0][1:] == (1, 77) and len(ce.scratch.streams) == len(ce.status.streams) == 1


def test_clip_rows_arguments():
    build.build()
    lib, ok = binding.load(), C.c_void_p(256)     # never dereferenced: the checks come first

    def clip(n=1, ptr=256, out=256, rows=3, cols=10, ldi=16, ldo=16, type=0, max_norm=1.0, **kw):
        a = {**dict(norm=ok, scratch=ok, st=ok), **kw}
        arr = lambda t, v: (t * 1)(v)  # noqa: E731
        return lib.dspark_clip_grads_rows(n, arr(C.c_void_p, ptr), arr(C.c_void_p, out), arr(C.c_int64, rows),
                                          arr(C.c_int64, cols), arr(C.c_int64, ldi), arr(C.c_int64, ldo),
                                          arr(C.c_int32, type), max_norm, a["norm"], a["scratch"], a["st"], None)

    for kw in (dict(n=-1), dict(ptr=None), dict(out=None), dict(ptr=258), dict(ptr=257, type=1), dict(rows=-1),
               dict(cols=-1), dict(ldi=9), dict(ldo=9), dict(ldi=-16), dict(ldi=24), dict(out=512, ldo=(1 << 44) + 1),
               dict(rows=1 << 40, cols=32, ldi=32, ldo=32), dict(rows=(1 << 44) + 1, cols=0), dict(type=2),
               dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(scratch=None), dict(st=None),
               dict(scratch=C.c_void_p(260))):
        assert clip(**kw) == 1, kw
    assert lib.dspark_clip_grads_rows(1, *([None] * 7), 1.0, ok, ok, ok, None) == 1


def test_what_clip_takes_for_a_matrix():
    """Contiguous tensors of any shape, and matrices whose rows are contiguous."""
    lay = lambda t: binding.GradClip._layout(t, None, "t")  # noqa: E731

    class Cuda(torch.Tensor):       # a CPU tensor that answers as a CUDA one
        is_cuda = True

    def of(*shape):
        return torch.zeros(*shape).as_subclass(Cuda)

    assert lay(of(3, 4, 5)) is None and lay(of(7)) is None and lay(of(0, 5)) is None and lay(of(6, 8)[:1, :3]) is None
    assert lay(of(6, 8)[:, :5]) == 8 and lay(of(6, 8)[:, 7:]) == 8 and lay(of(6, 8)[::2]) == 16
    for bad in (of(9)[::2], of(3, 4).t(), of(3, 4, 5)[:, :, :2], of(1, 5).expand(4, 5), of(4, 6)[:, ::2]):
        with pytest.raises(DsparkError):
            lay(bad)
    with pytest.raises(DsparkError):
        lay(torch.zeros(6, 8)[:, :5])


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (6, 80, 1024), (64, 256, 151936), (65, 64, 4000), (640, 256, 129280), (1001, 4100, 50257),
                                   (4096, 5376, 129280), (16384, 256, 129280), (32768, 256, 129280), (1 << 20, 64, 50257),
                                   (64, 16, 600003), (300000, 8, 300), (5, 65536, 2000)])
def test_scratch_is_what_the_header_says(N, K, V, layout):
    """The sizes that include/dspark.h gives, and no more than their roundings beside them."""
    build.build()
    got = binding.load().dspark_linear_ce_scratch_bytes(C.byref(binding.LceDims(N, K, V, layout, 0, 0, 0, 0, 0)))
    up = lambda x, m: -(-x // m) * m  # noqa: E731
    forward = N * max(16 * -(-V // 256), 9728) + 4 * N
    piece = min(2 * N * up(V, 64), max(1 << 30, 2 * N * 2048))
    gradient = 2 * piece + 2 * max(N * up(K, 8), K * up(N, 8)) + 4 * max(up(N, 32) * K, up(K, 32) * N) + 80_000_000
    assert 0 < got <= max(forward, gradient) + 8 * 256, (got, forward, gradient)
