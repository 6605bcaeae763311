"""What a head server does on the host with several devices, on stand-ins for tensors and for the operators.

Runs without a GPU: nothing is launched."""

import types

import pytest
import torch

from speculative_decoding_head_gb300 import serve_head
from speculative_decoding_head_gb300.binding import DsparkError

ZERO, ONE = torch.device("cuda", 0), torch.device("cuda", 1)
B, GAMMA, V, H, R = 4, 3, 64, 32, 16


class Stand:
    """What a server looks at of a tensor."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device

    def view(self, *shape):
        return self

    def float(self):
        return self

    def contiguous(self):
        return self

    def clone(self):
        return self

    def zero_(self):
        self.zeroed = True
        return self

    def __getitem__(self, _):
        return self


@pytest.fixture
def devices(monkeypatch):
    """Device 0 is current. Returns the current devices' stack and what was current at each call of an operator."""
    current, calls = [0], []

    class On:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()

    class Op:
        """A workspace follows the current device; the other operators have a device of their own."""

        def __init__(self, *args, device=None, **kw):
            self.device = device
            calls.append(("new", current[-1] if device is None else device.index))

        def __getattr__(self, name):
            def call(*args, **kw):
                calls.append((name, current[-1] if self.device is None else self.device.index))
                where = torch.device("cuda", calls[-1][1])
                if name == "quantise":
                    return self
                if name == "device_status":
                    return 0
                if kw.get("out") is not None and name == "draft":
                    return kw["out"]
                keys = {"plan": ("lengths", "row_off"), "verify": ("n_acc", "next_anchor")}
                return {k: Stand((B,), torch.int32, where) for k in keys.get(name, ("tokens", "pd_tok", "lse", "conf"))}
            return call

    def make(*shape, dtype=None, device=None):
        return Stand(shape, dtype, torch.device("cuda", current[-1]) if device is None else torch.device(device))

    fake = types.SimpleNamespace(**{k: getattr(torch, k) for k in ("float32", "int32", "bfloat16", "device")})
    fake.empty = fake.ones = fake.zeros = make
    fake.full = lambda shape, _, dtype=None, device=None: make(*shape, dtype=dtype, device=device)
    fake.cuda = types.SimpleNamespace(device=On)
    monkeypatch.setattr(serve_head, "torch", fake)
    for name in ("Workspace", "Fp4Matrix", "Sampler"):
        monkeypatch.setattr(serve_head, name, Op)
    return current, calls


def tensors(device, **other):
    f32, i32 = torch.float32, torch.int32
    at = lambda name, shape, dtype: Stand(shape, dtype, other.get(name, device))  # noqa: E731
    return dict(W_out=at("W_out", (V, H), f32), W1=at("W1", (V, R), f32), W2=at("W2", (R, V), f32),
                w=at("w", (H + R,), f32), T=at("T", (GAMMA,), f32)), dict(
        h=at("h", (B, GAMMA, H), f32), ht=at("ht", (B * (GAMMA + 1), H), f32), anchor=at("anchor", (B,), i32),
        sps=at("sps", (1 + B * (GAMMA + 1),), torch.float64))


@pytest.mark.parametrize("device", [ZERO, ONE])
def test_a_server_runs_on_its_own_device(devices, device):
    current, calls = devices
    weights, ins = tensors(device)
    s = serve_head.HeadServer(B, GAMMA, **weights)
    d = s.draft(ins["h"], ins["anchor"], ins["sps"], 0, 0)
    s.verify(ins["ht"], ins["anchor"], d, 0, 0)
    s.device_status()
    assert current == [0]
    names = {name for name, _ in calls}
    assert {"new", "draft", "plan", "verify", "linear", "logprobs", "device_status"} <= names
    assert {where for _, where in calls} == {device.index}, calls


@pytest.mark.parametrize("name", ["W1", "W2", "w", "T"])
def test_weights_of_another_device_are_refused(devices, name):
    weights, _ = tensors(ONE, **{name: ZERO})
    with pytest.raises(DsparkError):
        serve_head.HeadServer(B, GAMMA, **weights)
    assert not devices[1]


def test_a_server_off_the_gpu_is_refused(devices):
    weights, _ = tensors(torch.device("cpu"))
    with pytest.raises(DsparkError):
        serve_head.HeadServer(B, GAMMA, **weights)
    assert not devices[1]


@pytest.mark.parametrize("name", ["h", "ht", "anchor", "sps", "tokens", "lengths", "row_off", "pd_tok", "lse"])
def test_a_rounds_tensors_of_another_device_are_refused(devices, name):
    calls = devices[1]
    weights, ins = tensors(ONE)
    s = serve_head.HeadServer(B, GAMMA, **weights)
    d = s.draft(ins["h"], ins["anchor"], ins["sps"], 0, 0)
    calls.clear()
    _, bad = tensors(ONE, **{name: ZERO})
    if name in d:
        d[name] = Stand((B,), torch.int32, ZERO)
    if name in ("h", "anchor", "sps"):
        with pytest.raises(DsparkError):
            s.draft(bad["h"], bad["anchor"], bad["sps"], 0, 1)
    if name not in ("h", "sps"):
        with pytest.raises(DsparkError):
            s.verify(bad["ht"], bad["anchor"], d, 0, 1)
    assert not calls


@pytest.mark.parametrize("mode", ["static", "compact"])
def test_vectors_of_another_length_are_refused(devices, mode):
    """The workspace takes as many values from an address as its shape says."""
    calls = devices[1]
    weights, ins = tensors(ONE)
    for n in (GAMMA - 1, GAMMA + 1):
        with pytest.raises(DsparkError):
            serve_head.HeadServer(B, GAMMA, **{**weights, "T": Stand((n,), torch.float32, ONE)}, mode=mode)
    assert not calls
    s = serve_head.HeadServer(B, GAMMA, **weights, mode=mode)
    d = s.draft(ins["h"], ins["anchor"], ins["sps"], 0, 0)
    calls.clear()
    for n in (B - 1, B + 1):
        short = Stand((n,), torch.int32, ONE)
        with pytest.raises(DsparkError):
            s.draft(ins["h"], short, ins["sps"], 0, 1)
        with pytest.raises(DsparkError):
            s.verify(ins["ht"], short, d, 0, 1)
    sps = Stand((B * (GAMMA + 1),), torch.float64, ONE)
    if mode == "compact":
        with pytest.raises(DsparkError):
            s.draft(ins["h"], ins["anchor"], sps, 0, 1)
        assert not calls
    else:  # not looked at
        s.draft(ins["h"], ins["anchor"], sps, 0, 1)


@pytest.mark.parametrize("args", ["--temperature -1", "--temperature nan", "--temperature inf", "--top-p 1.5", "--top-p -0.1",
                                  "--top-p nan", "--min-p 2", "--min-p -1", "--batch 0", "--gamma 0", "--rounds 0",
                                  "--noise -1", "--hidden 0"])
def test_the_command_refuses_settings_out_of_range(args, monkeypatch, capsys):
    """Before anything runs: a round with such a setting has no next tokens to go on from."""
    monkeypatch.setattr("sys.argv", ["serve_head", *args.split()])
    with pytest.raises(SystemExit) as e:
        serve_head.main()
    assert e.value.code == 2 and args.split()[0] in capsys.readouterr().err


def test_a_drafts_tokens_are_ids_before_it_writes_them(devices):
    """A draft that ends with a device error leaves tokens as they were: what a caller looks up next, so not memory as
    it was."""
    weights, ins = tensors(ONE)
    s = serve_head.HeadServer(B, GAMMA, **weights)
    assert s.draft(ins["h"], ins["anchor"], ins["sps"], 0, 0)["tokens"].zeroed
