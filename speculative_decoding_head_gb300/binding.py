"""Python binding of libdspark.so (ctypes; argument marshalling only).

Every step of a round runs in the library's CUDA kernels. PyTorch supplies
device memory and the current stream. If the library has not been built the
binding raises; there is no CPU fallback.
"""

from __future__ import annotations

import ctypes as C
import os
import threading
from typing import Dict, Optional, Sequence

import torch

from .build import LIB_PATH

MODES = {"static": 0, "compact": 1, "lagged": 2}
WDTYPES = {"f32": 0, "bf16": 1}
LAYOUTS = {"vk": 0, "kv": 1}
FP4_FORMATS = {"nvfp4": 0, "mxfp4": 1}

SYMBOLS = [
    "dspark_ws_create", "dspark_ws_destroy", "dspark_ws_reset", "dspark_last_error",
    "dspark_status_string", "dspark_last_launch_count", "dspark_path",
    "dspark_markov_draft", "dspark_plan", "dspark_verify", "dspark_round", "dspark_ws_set_path",
    "dspark_sts_fit", "dspark_sts_scratch_bytes", "dspark_train_loss", "dspark_train_loss_scratch_bytes",
    "dspark_rnn_draft", "dspark_rnn_draft_scratch_bytes", "dspark_verify_rnn",
    "dspark_pctree_scratch_bytes", "dspark_pctree_build", "dspark_pctree_verify",
    "dspark_ws_set_shard", "dspark_plan_shard",
    "dspark_linear_ce", "dspark_linear_ce_grad", "dspark_linear_ce_scratch_bytes",
    "dspark_embed", "dspark_embed_grad", "dspark_embed_grad_scratch_bytes",
    "dspark_clip_grads", "dspark_clip_grads_rows", "dspark_clip_grads_scratch_bytes",
    "dspark_fp4_code_bytes", "dspark_fp4_scale_bytes", "dspark_fp4_quant", "dspark_fp4_rows", "dspark_fp4_linear",
    "dspark_sample", "dspark_sample_logprobs",
]


class DsparkError(RuntimeError):
    pass


class Dims(C.Structure):
    _fields_ = [("B", C.c_int), ("gamma", C.c_int), ("V", C.c_int), ("r", C.c_int), ("H", C.c_int),
                ("wdtype", C.c_int), ("mode", C.c_int), ("lag", C.c_int)]


class LceDims(C.Structure):
    _fields_ = [("N", C.c_int), ("K", C.c_int), ("V", C.c_int), ("layout", C.c_int), ("ldx", C.c_int64),
                ("ldw", C.c_int64), ("ldu", C.c_int64), ("lddx", C.c_int64), ("lddw", C.c_int64)]


class Fp4Dims(C.Structure):
    _fields_ = [("rows", C.c_int), ("K", C.c_int), ("format", C.c_int)]


class Fp4Data(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rowf", C.c_void_p)]


class SampleArgs(C.Structure):
    _fields_ = [("N", C.c_int), ("V", C.c_int), ("requests", C.c_int), ("type", C.c_int), ("ldz", C.c_int64),
                ("row_off", C.c_void_p), ("temperature", C.c_void_p), ("top_k", C.c_void_p), ("top_p", C.c_void_p),
                ("min_p", C.c_void_p)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return LIB_PATH


def load() -> C.CDLL:
    """Load libdspark.so (built by __graft_entry__.build() or build.py)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise DsparkError(f"libdspark.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        lib = C.CDLL(LIB_PATH)
        P, i32, u64 = C.c_void_p, C.c_int, C.c_uint64
        lib.dspark_ws_create.argtypes = [C.POINTER(Dims), C.POINTER(P)]
        lib.dspark_ws_create.restype = i32
        lib.dspark_ws_destroy.argtypes = [P]
        lib.dspark_ws_destroy.restype = None
        lib.dspark_ws_reset.argtypes = [P, P]
        lib.dspark_ws_reset.restype = i32
        lib.dspark_last_error.argtypes = [P, C.POINTER(i32)]
        lib.dspark_last_error.restype = i32
        lib.dspark_status_string.argtypes = [i32]
        lib.dspark_status_string.restype = C.c_char_p
        lib.dspark_last_launch_count.argtypes = [P]
        lib.dspark_last_launch_count.restype = i32
        lib.dspark_path.argtypes = [P]
        lib.dspark_path.restype = C.c_char_p
        lib.dspark_ws_set_path.argtypes = [P, C.c_char_p]
        lib.dspark_ws_set_path.restype = i32
        lib.dspark_markov_draft.argtypes = [P, P, P, P, P, P, P, P, u64, u64, P, P, P, P, P]
        lib.dspark_markov_draft.restype = i32
        lib.dspark_plan.argtypes = [P, P, P, P, P, P]
        lib.dspark_plan.restype = i32
        lib.dspark_verify.argtypes = [P, P, P, P, P, P, P, P, P, P, P, u64, u64, P, P, P]
        lib.dspark_verify.restype = i32
        lib.dspark_round.argtypes = [P] * 10 + [u64, u64] + [P] * 9
        lib.dspark_round.restype = i32
        lib.dspark_sts_fit.argtypes = [P, P, i32, i32, P, i32, i32, P, P, P, P, P]
        lib.dspark_sts_fit.restype = i32
        lib.dspark_sts_scratch_bytes.argtypes = [i32, i32]
        lib.dspark_sts_scratch_bytes.restype = C.c_size_t
        lib.dspark_train_loss.argtypes = [P] * 8 + [C.c_double] + [P] * 6
        lib.dspark_train_loss.restype = i32
        lib.dspark_train_loss_scratch_bytes.argtypes = [P]
        lib.dspark_train_loss_scratch_bytes.restype = C.c_size_t
        lib.dspark_rnn_draft.argtypes = [P] * 9 + [u64, u64] + [P] * 7
        lib.dspark_rnn_draft.restype = i32
        lib.dspark_verify_rnn.argtypes = [P] * 11 + [u64, u64] + [P] * 3
        lib.dspark_verify_rnn.restype = i32
        lib.dspark_rnn_draft_scratch_bytes.argtypes = [P]
        lib.dspark_rnn_draft_scratch_bytes.restype = C.c_size_t
        lib.dspark_pctree_scratch_bytes.argtypes = [P, i32, i32]
        lib.dspark_pctree_scratch_bytes.restype = C.c_size_t
        lib.dspark_pctree_build.argtypes = [P] * 5 + [i32, i32] + [P] * 7
        lib.dspark_pctree_build.restype = i32
        lib.dspark_pctree_verify.argtypes = [P] * 4 + [i32, u64, u64] + [P] * 4
        lib.dspark_pctree_verify.restype = i32
        lib.dspark_ws_set_shard.argtypes = [P, i32]
        lib.dspark_ws_set_shard.restype = i32
        lib.dspark_plan_shard.argtypes = [P, P, P, i32, i32, P, P, P, P, P]
        lib.dspark_plan_shard.restype = i32
        lib.dspark_linear_ce.argtypes = [C.POINTER(LceDims)] + [P] * 9
        lib.dspark_linear_ce.restype = i32
        lib.dspark_linear_ce_grad.argtypes = [C.POINTER(LceDims)] + [P] * 6 + [C.c_float] + [P] * 5
        lib.dspark_linear_ce_grad.restype = i32
        lib.dspark_linear_ce_scratch_bytes.argtypes = [C.POINTER(LceDims)]
        lib.dspark_linear_ce_scratch_bytes.restype = C.c_size_t
        i64, f = C.c_int64, C.c_float
        lib.dspark_embed.argtypes = [P, i32, i64, i32, i32, P, i32, f, P, i64, P, P]
        lib.dspark_embed.restype = i32
        lib.dspark_embed_grad.argtypes = [P, i32, i64, P, i32, i32, i32, f, P, i64, P, i32, i64, P, P, P]
        lib.dspark_embed_grad.restype = i32
        lib.dspark_embed_grad_scratch_bytes.argtypes = [i32, i32, i32]
        lib.dspark_embed_grad_scratch_bytes.restype = C.c_size_t
        lib.dspark_clip_grads.argtypes = [i32, P, P, P, P, f, P, P, P, P]
        lib.dspark_clip_grads.restype = i32
        lib.dspark_clip_grads_rows.argtypes = [i32] + [P] * 7 + [f] + [P] * 4
        lib.dspark_clip_grads_rows.restype = i32
        lib.dspark_clip_grads_scratch_bytes.argtypes = [i32]
        lib.dspark_clip_grads_scratch_bytes.restype = C.c_size_t
        D4, M4 = C.POINTER(Fp4Dims), C.POINTER(Fp4Data)
        for name in ("dspark_fp4_code_bytes", "dspark_fp4_scale_bytes"):
            getattr(lib, name).argtypes = [D4]
            getattr(lib, name).restype = C.c_size_t
        lib.dspark_fp4_quant.argtypes = [D4, P, i32, i64, P, M4, P, P]
        lib.dspark_fp4_quant.restype = i32
        lib.dspark_fp4_rows.argtypes = [D4, M4, P, i32, P, i32, i64, P, P]
        lib.dspark_fp4_rows.restype = i32
        lib.dspark_fp4_linear.argtypes = [D4, M4, D4, M4, P, i64, P, i32, i64, P, P]
        lib.dspark_fp4_linear.restype = i32
        lib.dspark_sample.argtypes = [C.POINTER(SampleArgs), P, P, P, P, P, P]
        lib.dspark_sample.restype = i32
        lib.dspark_sample_logprobs.argtypes = [C.POINTER(SampleArgs), P, f, P, i64, P, P]
        lib.dspark_sample_logprobs.restype = i32
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().dspark_status_string(int(code)).decode()


def _check(code: int, what: str) -> None:
    if code != 0:
        raise DsparkError(f"{what}: {status_string(code)} ({code})")


def _ptr(t: Optional[torch.Tensor], dtype=None, name="") -> C.c_void_p:
    if t is None:
        return C.c_void_p(0)
    if not t.is_cuda:
        raise DsparkError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise DsparkError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise DsparkError(f"{name} must be {dtype}, got {t.dtype}")
    return C.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return 1
    if t.dtype == torch.float32:
        return 0
    raise DsparkError(f"{name} must be bf16 or fp32, got {t.dtype}")


def _rows(t: torch.Tensor, rows: int, cols: int, dtype, name: str, device: int):
    """Address and leading dimension of a matrix on CUDA device ``device`` whose rows are contiguous."""
    if t.dtype != dtype or t.get_device() != device or t.dim() != 2:
        raise DsparkError(f"{name} must be a matrix of {dtype} on cuda:{device}, got {list(t.shape)} {t.dtype} on "
                          f"{t.device}")
    r, c = t.shape
    if r != rows or c != cols:
        raise DsparkError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    ld, step = t.stride()
    if step != 1 and c > 1:
        raise DsparkError(f"{name} must have contiguous rows")
    return t.data_ptr(), (ld if r > 1 else -(-c // 8) * 8)


def _vec(t: Optional[torch.Tensor], n: int, dtype, name: str, device: int):
    """Address of a contiguous vector of n values on CUDA device ``device`` (None: no vector)."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        raise DsparkError(f"{name} must be a contiguous vector [{n}] of {dtype} on cuda:{device}, got {list(t.shape)} "
                          f"{t.dtype} on {t.device}")
    return t.data_ptr()


# torch's own short ways to the current device and a device's current stream, where it has them
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def sts_fit(raw: torch.Tensor, cstar: torch.Tensor, Tgrid: torch.Tensor, M: int = 15, stream=None):
    """Sequential temperature scaling (``dspark_sts_fit``): raw and cstar are
    [N, gamma] fp32 CUDA tensors, Tgrid [G] fp32. Returns (T [gamma] fp32,
    ece [gamma] fp64, device status [1] int32), all on the device."""
    lib = load()
    f32 = torch.float32
    if raw.dim() != 2 or cstar.shape != raw.shape:
        raise DsparkError("raw and cstar must be [N, gamma] of the same shape")
    N, g = raw.shape
    G = Tgrid.numel()
    dev = raw.device
    scratch = torch.empty(int(lib.dspark_sts_scratch_bytes(N, G)), dtype=torch.uint8, device=dev)
    T = torch.empty(g, dtype=f32, device=dev)
    ece = torch.empty(g, dtype=torch.float64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    code = lib.dspark_sts_fit(_ptr(raw, f32, "raw"), _ptr(cstar, f32, "cstar"), N, g, _ptr(Tgrid, f32, "Tgrid"), G,
                              int(M), _ptr(T, f32, "T"), _ptr(ece, torch.float64, "ece"), _ptr(scratch, None, "scratch"),
                              _ptr(status, torch.int32, "status"), _stream(stream))
    _check(code, "dspark_sts_fit")
    return T, ece, status


class Workspace:
    """One DSpark workspace: the library's scratch arena for a fixed shape."""

    def __init__(self, B: int, gamma: int, V: int, r: int, H: int, wdtype: str = "bf16",
                 mode: str = "compact", lag: int = 2, path: Optional[str] = None):
        self.lib = load()
        self.dims = Dims(B, gamma, V, r, H, WDTYPES[wdtype], MODES[mode], lag if mode == "lagged" else 0)
        self.wdtype = torch.bfloat16 if wdtype == "bf16" else torch.float32
        self._h = C.c_void_p()
        _check(self.lib.dspark_ws_create(C.byref(self.dims), C.byref(self._h)), "dspark_ws_create")
        if path is not None:
            self.set_path(path)

    @classmethod
    def for_workload(cls, wl, path: Optional[str] = None) -> "Workspace":
        return cls(wl.B, wl.gamma, wl.V, wl.r, wl.H, wl.wdtype, wl.mode, wl.lag or 2, path)

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            self.lib.dspark_ws_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------ state
    @property
    def handle(self) -> C.c_void_p:
        return self._h

    @property
    def path(self) -> str:
        return self.lib.dspark_path(self._h).decode()

    def set_path(self, path: str) -> None:
        _check(self.lib.dspark_ws_set_path(self._h, path.encode()), "dspark_ws_set_path")

    @property
    def last_launches(self) -> int:
        return int(self.lib.dspark_last_launch_count(self._h))

    def reset(self, stream=None) -> None:
        _check(self.lib.dspark_ws_reset(self._h, _stream(stream)), "dspark_ws_reset")

    def device_status(self) -> int:
        v = C.c_int(0)
        _check(self.lib.dspark_last_error(self._h, C.byref(v)), "dspark_last_error")
        return int(v.value)

    # ------------------------------------------------------------ outputs
    def new_draft_outputs(self, device="cuda") -> Dict[str, torch.Tensor]:
        B, g = self.dims.B, self.dims.gamma
        return {"tokens": torch.empty((B, g), dtype=torch.int32, device=device),
                "pd_tok": torch.empty((B, g), dtype=torch.float32, device=device),
                "lse": torch.empty((B, g), dtype=torch.float32, device=device),
                "conf": torch.empty((B, g), dtype=torch.float32, device=device)}

    def new_plan_outputs(self, device="cuda") -> Dict[str, torch.Tensor]:
        B = self.dims.B
        return {"lengths": torch.empty(B, dtype=torch.int32, device=device),
                "row_off": torch.empty(B + 1, dtype=torch.int32, device=device)}

    def new_verify_outputs(self, device="cuda") -> Dict[str, torch.Tensor]:
        B = self.dims.B
        return {"n_acc": torch.empty(B, dtype=torch.int32, device=device),
                "next_anchor": torch.empty(B, dtype=torch.int32, device=device)}

    # ------------------------------------------------------------ calls
    def draft(self, U, W1, W2, anchor, h, w, T, seed: int, rnd: int, out=None, stream=None):
        out = out or self.new_draft_outputs(U.device)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_markov_draft(
            self._h, _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"), _ptr(W2, self.wdtype, "W2"),
            _ptr(anchor, i32, "anchor"), _ptr(h, f32, "h") if self.dims.H > 0 else C.c_void_p(0),
            _ptr(w, f32, "w"), _ptr(T, f32, "T"), int(seed), int(rnd),
            _ptr(out["tokens"], i32, "tokens"), _ptr(out["pd_tok"], f32, "pd_tok"),
            _ptr(out["lse"], f32, "lse"), _ptr(out["conf"], f32, "conf"), _stream(stream))
        _check(code, "dspark_markov_draft")
        return out

    def plan(self, conf, sps, out=None, stream=None):
        out = out or self.new_plan_outputs(conf.device)
        code = self.lib.dspark_plan(self._h, _ptr(conf, torch.float32, "conf"),
                                    _ptr(sps, torch.float64, "sps"),
                                    _ptr(out["lengths"], torch.int32, "lengths"),
                                    _ptr(out["row_off"], torch.int32, "row_off"), _stream(stream))
        _check(code, "dspark_plan")
        return out

    def set_shard(self, b_offset: int):
        """This workspace holds requests b_offset .. b_offset + B - 1 of a
        batch split across devices (``dspark_ws_set_shard``)."""
        _check(self.lib.dspark_ws_set_shard(self._h, int(b_offset)), "dspark_ws_set_shard")

    def plan_shard(self, conf, sps, b_begin: int, b_count: int, out=None, stream=None):
        """Plan the whole batch (this workspace's B) from the gathered
        confidences and keep requests b_begin .. b_begin + b_count - 1
        (``dspark_plan_shard``). ``out`` gains lengths_local [b_count] and
        row_off_local [b_count + 1]."""
        dev = conf.device
        out = out or self.new_plan_outputs(dev)
        if "lengths_local" not in out:
            out["lengths_local"] = torch.zeros(b_count, dtype=torch.int32, device=dev)
            out["row_off_local"] = torch.zeros(b_count + 1, dtype=torch.int32, device=dev)
        i32 = torch.int32
        code = self.lib.dspark_plan_shard(self._h, _ptr(conf, torch.float32, "conf"),
                                          _ptr(sps, torch.float64, "sps"), int(b_begin), int(b_count),
                                          _ptr(out["lengths"], i32, "lengths"), _ptr(out["row_off"], i32, "row_off"),
                                          _ptr(out["lengths_local"], i32, "lengths_local"),
                                          _ptr(out["row_off_local"], i32, "row_off_local"), _stream(stream))
        _check(code, "dspark_plan_shard")
        return out

    def verify(self, P, row_off, lengths, anchor, tokens, pd_tok, lse, U, W1, W2, seed: int, rnd: int,
               out=None, stream=None):
        out = out or self.new_verify_outputs(P.device)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_verify(
            self._h, _ptr(P, f32, "P"), _ptr(row_off, i32, "row_off"), _ptr(lengths, i32, "lengths"),
            _ptr(anchor, i32, "anchor"), _ptr(tokens, i32, "tokens"), _ptr(pd_tok, f32, "pd_tok"),
            _ptr(lse, f32, "lse"), _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"),
            _ptr(W2, self.wdtype, "W2"), int(seed), int(rnd), _ptr(out["n_acc"], i32, "n_acc"),
            _ptr(out["next_anchor"], i32, "next_anchor"), _stream(stream))
        _check(code, "dspark_verify")
        return out

    def rnn_draft(self, U, W1, W2, Wr, anchor, h, w, T, seed: int, rnd: int, out=None, stream=None):
        """Draft tail with the RNN head (``dspark_rnn_draft``): as ``draft``,
        plus Wr [3, r, 2r + H]; ``out`` also holds ovec [B, gamma, r] fp32."""
        if out is None:
            out = self.new_draft_outputs(U.device)
            B, g, r = self.dims.B, self.dims.gamma, self.dims.r
            out["ovec"] = torch.empty(B, g, r, dtype=torch.float32, device=U.device)
            out["scratch"] = torch.empty(int(self.lib.dspark_rnn_draft_scratch_bytes(self._h)), dtype=torch.uint8,
                                         device=U.device)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_rnn_draft(
            self._h, _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"), _ptr(W2, self.wdtype, "W2"),
            _ptr(Wr, self.wdtype, "Wr"), _ptr(anchor, i32, "anchor"),
            _ptr(h, f32, "h") if self.dims.H > 0 else C.c_void_p(0), _ptr(w, f32, "w"), _ptr(T, f32, "T"),
            int(seed), int(rnd), _ptr(out["tokens"], i32, "tokens"), _ptr(out["pd_tok"], f32, "pd_tok"),
            _ptr(out["lse"], f32, "lse"), _ptr(out["conf"], f32, "conf"), _ptr(out["ovec"], f32, "ovec"),
            _ptr(out["scratch"], None, "scratch"), _stream(stream))
        _check(code, "dspark_rnn_draft")
        return out

    def pctree_build(self, U, W1, W2, anchor, c: int, N: int, out=None, stream=None):
        """PCTree's draft tree (``dspark_pctree_build``): tok, par, dep [B, N+1]
        int32, lp [B, N+1] fp32, n_nodes [B] int32."""
        B = self.dims.B
        if out is None:
            dev = U.device
            nbytes = int(self.lib.dspark_pctree_scratch_bytes(self._h, int(c), int(N)))
            if nbytes == 0:
                raise DsparkError(f"dspark_pctree_build: unsupported c={c}, N={N}")
            out = {k: torch.empty(B, N + 1, dtype=torch.int32, device=dev) for k in ("tok", "par", "dep")}
            out["lp"] = torch.empty(B, N + 1, dtype=torch.float32, device=dev)
            out["n_nodes"] = torch.empty(B, dtype=torch.int32, device=dev)
            out["scratch"] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_pctree_build(
            self._h, _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"), _ptr(W2, self.wdtype, "W2"),
            _ptr(anchor, i32, "anchor"), int(c), int(N), _ptr(out["tok"], i32, "tok"), _ptr(out["par"], i32, "par"),
            _ptr(out["dep"], i32, "dep"), _ptr(out["lp"], f32, "lp"), _ptr(out["n_nodes"], i32, "n_nodes"),
            _ptr(out["scratch"], None, "scratch"), _stream(stream))
        _check(code, "dspark_pctree_build")
        return out

    def pctree_verify(self, P, tok, par, N: int, seed: int, rnd: int, out=None, stream=None):
        """PCTree's lossless tree verify (``dspark_pctree_verify``): P [B, N+1, V]
        fp32. Returns path [B, gamma+1], n_acc [B], next_anchor [B] (int32)."""
        B, g = self.dims.B, self.dims.gamma
        if out is None:
            dev = P.device
            out = {"path": torch.empty(B, g + 1, dtype=torch.int32, device=dev),
                   "n_acc": torch.empty(B, dtype=torch.int32, device=dev),
                   "next_anchor": torch.empty(B, dtype=torch.int32, device=dev)}
        i32 = torch.int32
        code = self.lib.dspark_pctree_verify(
            self._h, _ptr(P, torch.float32, "P"), _ptr(tok, i32, "tok"), _ptr(par, i32, "par"), int(N), int(seed),
            int(rnd), _ptr(out["path"], i32, "path"), _ptr(out["n_acc"], i32, "n_acc"),
            _ptr(out["next_anchor"], i32, "next_anchor"), _stream(stream))
        _check(code, "dspark_pctree_verify")
        return out

    def verify_rnn(self, P, row_off, lengths, anchor, tokens, pd_tok, lse, U, ovec, W2, seed: int, rnd: int,
                   out=None, stream=None):
        """Verify of RNN-head drafts (``dspark_verify_rnn``): p_d of a rejected
        position from U + o W2 with ovec [B, gamma, r] fp32."""
        out = out or self.new_verify_outputs(P.device)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_verify_rnn(
            self._h, _ptr(P, f32, "P"), _ptr(row_off, i32, "row_off"), _ptr(lengths, i32, "lengths"),
            _ptr(anchor, i32, "anchor"), _ptr(tokens, i32, "tokens"), _ptr(pd_tok, f32, "pd_tok"),
            _ptr(lse, f32, "lse"), _ptr(U, f32, "U"), _ptr(ovec, f32, "ovec"), _ptr(W2, self.wdtype, "W2"),
            int(seed), int(rnd), _ptr(out["n_acc"], i32, "n_acc"), _ptr(out["next_anchor"], i32, "next_anchor"),
            _stream(stream))
        _check(code, "dspark_verify_rnn")
        return out

    def new_loss_outputs(self, device="cuda") -> Dict[str, torch.Tensor]:
        B, g = self.dims.B, self.dims.gamma
        return {"ce": torch.empty(B, g, dtype=torch.float32, device=device),
                "l1": torch.empty(B, g, dtype=torch.float32, device=device),
                "bce": torch.empty(B, g, dtype=torch.float32, device=device),
                "loss": torch.empty(1, dtype=torch.float64, device=device),
                "scratch": torch.empty(int(self.lib.dspark_train_loss_scratch_bytes(self._h)), dtype=torch.uint8,
                                       device=device)}

    def train_loss(self, U, W1, W2, anchor, xstar, P, conf, tau: float, out=None, stream=None):
        """Teacher-forced training objective (``dspark_train_loss``): U and P
        [B, gamma, V] fp32, xstar and conf [B, gamma]; per-position ce, l1,
        bce and the scalar loss stay on the device."""
        out = out or self.new_loss_outputs(U.device)
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_train_loss(
            self._h, _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"), _ptr(W2, self.wdtype, "W2"),
            _ptr(anchor, i32, "anchor"), _ptr(xstar, i32, "xstar"), _ptr(P, f32, "P"), _ptr(conf, f32, "conf"),
            float(tau), _ptr(out["ce"], f32, "ce"), _ptr(out["l1"], f32, "l1"), _ptr(out["bce"], f32, "bce"),
            _ptr(out["loss"], torch.float64, "loss"), _ptr(out["scratch"], None, "scratch"), _stream(stream))
        _check(code, "dspark_train_loss")
        return out

    def round(self, U, W1, W2, anchor, h, w, T, sps, P, seed: int, rnd: int, out=None, stream=None):
        """draft -> plan -> verify on P packed for this round's lengths."""
        if out is None:
            out = {**self.new_draft_outputs(U.device), **self.new_plan_outputs(U.device),
                   **self.new_verify_outputs(U.device)}
        f32, i32 = torch.float32, torch.int32
        code = self.lib.dspark_round(
            self._h, _ptr(U, f32, "U"), _ptr(W1, self.wdtype, "W1"), _ptr(W2, self.wdtype, "W2"),
            _ptr(anchor, i32, "anchor"), _ptr(h, f32, "h") if self.dims.H > 0 else C.c_void_p(0),
            _ptr(w, f32, "w"), _ptr(T, f32, "T"), _ptr(sps, torch.float64, "sps"), _ptr(P, f32, "P"),
            int(seed), int(rnd), _ptr(out["tokens"], i32, "tokens"), _ptr(out["pd_tok"], f32, "pd_tok"),
            _ptr(out["lse"], f32, "lse"), _ptr(out["conf"], f32, "conf"),
            _ptr(out["lengths"], i32, "lengths"), _ptr(out["row_off"], i32, "row_off"),
            _ptr(out["n_acc"], i32, "n_acc"), _ptr(out["next_anchor"], i32, "next_anchor"),
            _stream(stream))
        _check(code, "dspark_round")
        return out


class _TrainOp:
    """What the objects of the operators without a workspace share (training the
    head, matrices in 4 bits, sampling). A call takes tensors of the
    object's device and runs there, whichever device is current. Memory that it makes
    belongs to the stream it runs on; the object's own buffers (``_buffers``) are
    noted with every stream that a call uses, so that their memory is not given
    away while that stream's work on them goes on."""

    def __init__(self, device):
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._index, self._device = self.status.get_device(), self.status.device
        if self._index < 0:
            raise DsparkError(f"the object must be on a CUDA device, got {self._device}")
        self._streams = set()

    def _buffers(self):
        return (self.scratch, self.status)

    def _call(self, f, *args) -> int:
        if _current_device() == self._index:
            return f(*args)
        with torch.cuda.device(self._index):
            return f(*args)

    def _on(self, stream) -> int:
        """Address of the stream that a call runs on (the current one if None)."""
        raw = _current_stream(self._index) if stream is None else stream.cuda_stream
        if raw not in self._streams:
            stream = torch.cuda.current_stream(self.status.device) if stream is None else stream
            if stream.device != self.status.device:
                raise DsparkError(f"the stream belongs to {stream.device}, the object to {self.status.device}")
            self._streams.add(raw)
            for t in self._buffers():
                t.record_stream(stream)
        return raw

    def _new(self, shape, dtype, stream):
        """A new tensor on the object's device, of the stream that a call runs on."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self._device)

    def device_status(self) -> int:
        """The first device error since the last reset (synchronises)."""
        return int(self.status.item())

    def reset(self) -> None:
        self.status.zero_()


class LinearCE(_TrainOp):
    """Softmax cross entropy of z = X W (+ U) over the vocabulary, with its
    gradients and without keeping z (``dspark_linear_ce``,
    ``dspark_linear_ce_grad``), for N rows of K features and V tokens. Holds
    the calls' scratch and status word; calls that share one object must be
    ordered on one stream.

    X [N, K] and W ([V, K] for layout "vk", [K, V] for "kv") are bf16 with
    contiguous rows whose stride is a multiple of 8; U [N, V] fp32 (row stride
    a multiple of 4) or None; target [N] int32, -1 for a row left out."""

    def __init__(self, N: int, K: int, V: int, layout: str = "vk", device="cuda"):
        self.lib = load()
        if layout not in LAYOUTS:
            raise DsparkError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
        self.N, self.K, self.V, self.layout = int(N), int(K), int(V), layout
        self._dims = LceDims(self.N, self.K, self.V, LAYOUTS[layout], 0, 0, 0, 0, 0)
        self._pdims = C.byref(self._dims)
        nbytes = int(self.lib.dspark_linear_ce_scratch_bytes(self._pdims))
        if nbytes == 0:
            raise DsparkError(f"dspark_linear_ce: unsupported N={N}, K={K}, V={V}")
        self.scratch = torch.empty(nbytes, dtype=torch.uint8, device=device)
        super().__init__(device)

    @property
    def w_shape(self):
        return (self.V, self.K) if self.layout == "vk" else (self.K, self.V)

    def new_outputs(self, dx: bool = True, dw: bool = True) -> Dict[str, torch.Tensor]:
        """loss and lse [N] fp32; dX [N, K] and dW (W's shape) bf16 where wanted,
        their rows padded to a multiple of 8 in memory."""
        dev = self.scratch.device

        def mat(rows, cols):
            return torch.empty(rows, -(-cols // 8) * 8, dtype=torch.bfloat16, device=dev)[:, :cols]

        out = {k: torch.empty(self.N, dtype=torch.float32, device=dev) for k in ("loss", "lse")}
        if dx:
            out["dX"] = mat(self.N, self.K)
        if dw:
            out["dW"] = mat(*self.w_shape)
        return out

    def _inputs(self, X, W, target, U):
        dev, d = self._index, self._dims
        px, d.ldx = _rows(X, self.N, self.K, torch.bfloat16, "X", dev)
        pw, d.ldw = _rows(W, *self.w_shape, torch.bfloat16, "W", dev)
        pu = None
        if U is not None:
            pu, d.ldu = _rows(U, self.N, self.V, torch.float32, "U", dev)
        return px, pw, pu, _vec(target, self.N, torch.int32, "target", dev)

    def forward(self, X, W, target, U=None, out=None, stream=None):
        """loss and lse of every row."""
        if out is None:
            with torch.cuda.stream(stream):
                out = self.new_outputs(False, False)
        ins = self._inputs(X, W, target, U)
        f32, dev = torch.float32, self._index
        pl, ps = _vec(out["loss"], self.N, f32, "loss", dev), _vec(out["lse"], self.N, f32, "lse", dev)
        code = self._call(self.lib.dspark_linear_ce, self._pdims, *ins, pl, ps, self.scratch.data_ptr(),
                          self.status.data_ptr(), self._on(stream))
        _check(code, "dspark_linear_ce")
        return out

    def grad(self, X, W, target, lse, wt=None, scale: float = 1.0, U=None, out=None, stream=None):
        """Gradients of scale * sum_n wt[n] loss[n] with lse from ``forward``,
        into out["dX"] and out["dW"] (the ones that ``out`` has)."""
        if out is None:
            with torch.cuda.stream(stream):
                out = self.new_outputs()
        ins = self._inputs(X, W, target, U)
        f32, bf16, dev = torch.float32, torch.bfloat16, self._index
        px = pw = None
        if out.get("dX") is not None:
            px, self._dims.lddx = _rows(out["dX"], self.N, self.K, bf16, "dX", dev)
        if out.get("dW") is not None:
            pw, self._dims.lddw = _rows(out["dW"], *self.w_shape, bf16, "dW", dev)
        ps, pt = _vec(lse, self.N, f32, "lse", dev), _vec(wt, self.N, f32, "wt", dev)
        code = self._call(self.lib.dspark_linear_ce_grad, self._pdims, *ins, ps, pt, scale, px, pw,
                          self.scratch.data_ptr(), self.status.data_ptr(), self._on(stream))
        _check(code, "dspark_linear_ce_grad")
        return out


class Embedding(_TrainOp):
    """Rows of a table [V, D] looked up for N tokens and scaled
    (``dspark_embed``), and the table's gradient (``dspark_embed_grad``).
    Holds the gradient's scratch (made at its first call) and a status word; calls that share one
    object must be ordered on one stream. Matrices are bf16 or fp32 with contiguous
    rows; idx [N] int32, -1 for a row without a token."""

    def __init__(self, N: int, V: int, D: int, device="cuda"):
        self.lib = load()
        self.N, self.V, self.D = int(N), int(V), int(D)
        self._bytes = int(self.lib.dspark_embed_grad_scratch_bytes(self.N, self.V, self.D))
        if self._bytes == 0:
            raise DsparkError(f"dspark_embed: unsupported N={N}, V={V}, D={D}")
        self.scratch: Optional[torch.Tensor] = None
        super().__init__(device)

    def _buffers(self):
        return (self.status,) if self.scratch is None else (self.scratch, self.status)

    def _mat(self, t, rows, dtype, name):
        return _rows(t, rows, self.D, dtype, name, self._index)

    def lookup(self, E, idx, scale: float = 1.0, out=None, stream=None):
        """scale * E[idx] as [N, D] in E's type (into ``out`` if given)."""
        code = _dtype_code(E, "E")
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty(self.N, self.D, dtype=E.dtype, device=E.device)
        pe, lde = self._mat(E, self.V, E.dtype, "E")
        po, ldo = self._mat(out, self.N, E.dtype, "out")
        pi = _vec(idx, self.N, torch.int32, "idx", self._index)
        r = self._call(self.lib.dspark_embed, pe, code, lde, self.V, self.D, pi, self.N, scale, po, ldo,
                       self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_embed")
        return out

    def grad(self, dout, idx, scale: float = 1.0, base=None, out=None, stream=None):
        """base + scale * the rows of ``dout`` [N, D] summed per token, as
        [V, D] into ``out`` (dout's type if not given). ``base`` has out's type;
        it may be ``out`` itself."""
        code = _dtype_code(dout, "dout")
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty(self.V, self.D, dtype=dout.dtype if base is None else base.dtype, device=dout.device)
        if self.scratch is None:
            with torch.cuda.stream(stream):
                self.scratch = torch.empty(self._bytes, dtype=torch.uint8, device=self.status.device)
            self._streams.clear()
        pd, ldd = self._mat(dout, self.N, dout.dtype, "dout")
        po, ldo = self._mat(out, self.V, out.dtype, "out")
        pb, ldb = (None, self.D) if base is None else self._mat(base, self.V, out.dtype, "base")
        pi = _vec(idx, self.N, torch.int32, "idx", self._index)
        r = self._call(self.lib.dspark_embed_grad, pd, code, ldd, pi, self.N, self.V, self.D, scale, pb, ldb, po,
                       _dtype_code(out, "out"), ldo, self.scratch.data_ptr(), self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_embed_grad")
        return out


class GradClip(_TrainOp):
    """The 2-norm over a list of gradient tensors and their scaling to a largest
    norm (``dspark_clip_grads``), in place or into ``outs``. The object keeps
    the list (and the scratch and status word): make it for the gradient buffers
    that a training loop reuses. Tensors are bf16 or fp32 and contiguous, or
    matrices with contiguous rows (``dspark_clip_grads_rows``)."""

    def __init__(self, grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self.lib = load()
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise DsparkError(f"{len(self.grads)} gradients, {len(self.outs)} outputs")
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            self._layout(g, None, f"grads[{i}]")
            self._layout(o, g.dtype, f"outs[{i}]")
            if g.device != self.grads[0].device or o.device != g.device:
                raise DsparkError(f"grads[{i}] on {g.device}, outs[{i}] on {o.device}: all must be on one device")
            if o.shape != g.shape:
                raise DsparkError(f"outs[{i}] must be {list(g.shape)}, got {list(o.shape)}")
        n = self.count = len(self.grads)
        self._in = (C.c_void_p * max(n, 1))(*[g.data_ptr() for g in self.grads])
        self._out = (C.c_void_p * max(n, 1))(*[o.data_ptr() for o in self.outs])
        i64 = C.c_int64 * max(n, 1)
        if all(t.is_contiguous() for t in (*self.grads, *self.outs)):
            self._f, self._shape = self.lib.dspark_clip_grads, (i64(*[g.numel() for g in self.grads]),)
        else:
            lay = [(self._layout(g, None, ""), self._layout(o, None, "")) for g, o in zip(self.grads, self.outs)]
            # a matrix's rows, unless both of a pair are contiguous: those are one row
            flat = [a is None and b is None for a, b in lay]
            shape = [(1, g.numel()) if f else tuple(g.shape) for f, g in zip(flat, self.grads)]
            ld = [[c if x is None else x for x, (_, c) in zip(side, shape)] for side in zip(*lay)]
            self._f = self.lib.dspark_clip_grads_rows
            self._shape = (i64(*[r for r, _ in shape]), i64(*[c for _, c in shape]), i64(*ld[0]), i64(*ld[1]))
        self._types = (C.c_int32 * max(n, 1))(*[_dtype_code(g, f"grads[{i}]") for i, g in enumerate(self.grads)])
        device = self.grads[0].device if n else "cuda"
        self.scratch = torch.empty(int(self.lib.dspark_clip_grads_scratch_bytes(n)), dtype=torch.uint8, device=device)
        self.norm = torch.zeros((), dtype=torch.float32, device=device)
        super().__init__(device)

    @staticmethod
    def _layout(t: torch.Tensor, dtype, name: str) -> Optional[int]:
        """None for a contiguous tensor, the leading dimension of a matrix with contiguous rows; others are refused."""
        if t.is_contiguous() or t.dim() != 2 or t.stride(0) < t.shape[1] or (t.stride(1) != 1 and t.shape[1] > 1):
            _ptr(t, dtype, name)
            return None
        _ptr(t[0], dtype, name)
        return t.stride(0)

    def _buffers(self):
        return (self.scratch, self.norm, self.status)

    def clip(self, max_norm: float, stream=None) -> torch.Tensor:
        """Scale the gradients; returns their norm before that (a device fp32 scalar)."""
        code = self._call(self._f, self.count, self._in, self._out, *self._shape, self._types, max_norm,
                          self.norm.data_ptr(), self.scratch.data_ptr(), self.status.data_ptr(), self._on(stream))
        _check(code, "dspark_clip_grads")
        return self.norm


class Fp4Matrix(_TrainOp):
    """A matrix of ``rows`` rows of K values held in microscaled 4-bit floating
    point, "nvfp4" (blocks of 16, e4m3 scales, a power of two per row) or "mxfp4"
    (blocks of 32, power-of-two scales): an output layer [V, K], a table W1 [V, r], or the rows
    that go through a layer. Holds the codes, their scales, the rows' factors and a
    status word; calls that share one object must be ordered on one stream."""

    def __init__(self, rows: int, K: int, fmt: str = "nvfp4", device="cuda"):
        self.lib = load()
        if fmt not in FP4_FORMATS:
            raise DsparkError(f"fmt must be one of {sorted(FP4_FORMATS)}, got {fmt!r}")
        self.rows, self.K, self.fmt = int(rows), int(K), fmt
        self._dims = Fp4Dims(self.rows, self.K, FP4_FORMATS[fmt])
        self._pdims = C.byref(self._dims)
        codes, scales = (int(f(self._pdims)) for f in (self.lib.dspark_fp4_code_bytes, self.lib.dspark_fp4_scale_bytes))
        if codes == 0 or scales == 0:
            raise DsparkError(f"dspark_fp4: unsupported rows={rows}, K={K}")
        self.codes = torch.empty(codes, dtype=torch.uint8, device=device)
        self.scales = torch.empty(scales, dtype=torch.uint8, device=device)
        self.rowf = torch.empty(max(1, -(-self.rows // 128)) * 128, dtype=torch.float32, device=device)
        self._data = Fp4Data(self.codes.data_ptr(), self.scales.data_ptr(), self.rowf.data_ptr())
        self._pdata = C.byref(self._data)
        super().__init__(device)

    def _buffers(self):
        return (self.codes, self.scales, self.rowf, self.status)

    def quantise(self, X: torch.Tensor, count: Optional[torch.Tensor] = None, stream=None) -> "Fp4Matrix":
        """Takes X [rows, K] (bf16 or fp32, contiguous rows) into the matrix (``dspark_fp4_quant``); returns it.
        Rows from ``count`` [1] int32 on (a packed batch's end, on the device) are not read and become zeros."""
        code = _dtype_code(X, "X")
        px, ldx = _rows(X, self.rows, self.K, X.dtype, "X", self._index)
        pc = _vec(count, 1, torch.int32, "count", self._index)
        r = self._call(self.lib.dspark_fp4_quant, self._pdims, px, code, ldx, pc, self._pdata,
                       self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_fp4_quant")
        return self

    def lookup(self, idx: Optional[torch.Tensor] = None, dtype=torch.bfloat16, out=None, stream=None):
        """The values of rows idx [N] int32 (-1: zeros), or of all rows, as
        [N, K] bf16 or fp32 (``dspark_fp4_rows``)."""
        n = self.rows if idx is None else idx.numel()
        if out is None:
            out = self._new((n, self.K), dtype, stream)
            po, ldo = out.data_ptr(), self.K
        else:
            po, ldo = _rows(out, n, self.K, out.dtype, "out", self._index)
        code = _dtype_code(out, "out")
        pi = _vec(idx, n, torch.int32, "idx", self._index)
        r = self._call(self.lib.dspark_fp4_rows, self._pdims, self._pdata, pi, n, po, code, ldo,
                       self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_fp4_rows")
        return out

    def linear(self, X: "Fp4Matrix", U: Optional[torch.Tensor] = None, dtype=torch.float32, out=None, stream=None):
        """X W^T (+ U) as [N, rows] for this matrix W and X of the same format
        and K (``dspark_fp4_linear``): fp32 or bf16, U [N, rows] fp32 (it may be ``out``)."""
        if X._index != self._index:
            raise DsparkError(f"X on {X.status.device}, the matrix on {self.status.device}")
        if X.fmt != self.fmt or X.K != self.K:
            raise DsparkError(f"X holds {X.fmt} rows of {X.K}, the matrix {self.fmt} rows of {self.K}")
        if out is None:
            out = self._new((X.rows, self.rows), dtype, stream)
        code = _dtype_code(out, "out")
        po, ldo = _rows(out, X.rows, self.rows, out.dtype, "out", self._index)
        pu, ldu = (None, 0) if U is None else _rows(U, X.rows, self.rows, torch.float32, "U", self._index)
        X._on(stream)
        r = self._call(self.lib.dspark_fp4_linear, X._pdims, X._pdata, self._pdims, self._pdata, pu, ldu,
                       po, code, ldo, self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_fp4_linear")
        return out


class Sampler(_TrainOp):
    """Draws from up to N rows of V logits with temperature, top-k, top-p and min-p
    (``dspark_sample``), and the distribution that they make of the rows
    (``dspark_sample_logprobs``). The settings are device vectors (temperature (0: greedy, below 1e-30: 1e-30), top_p and
    min_p fp32, top_k int32; None: off), an entry per row, or per request where
    ``row_off`` [requests + 1] int32 says which rows belong to whom. Holds a status
    word; calls that share one object must be ordered on one stream."""

    def __init__(self, N: int, V: int, requests: Optional[int] = None, device="cuda"):
        self.lib = load()
        self.N, self.V, self.requests = int(N), int(V), None if requests is None else int(requests)
        if not (0 <= self.N <= 1 << 24 and 1 <= self.V <= 1 << 24 and (requests is None or self.requests >= 1)):
            raise DsparkError(f"dspark_sample: unsupported N={N}, V={V}, requests={requests}")
        self._args = SampleArgs(self.N, self.V, self.requests or 0)
        self._pargs = C.byref(self._args)
        super().__init__(device)

    def _buffers(self):
        return (self.status,)

    def _set(self, Z, row_off, temperature, top_k, top_p, min_p) -> int:
        """Takes a call's inputs into the argument block; returns the address of the logits."""
        dev, f32, i32, a = self._index, torch.float32, torch.int32, self._args
        a.type = _dtype_code(Z, "Z")
        pz, a.ldz = _rows(Z, self.N, self.V, Z.dtype, "Z", dev)
        n = self.N
        if row_off is None:
            a.row_off = None
        elif self.requests is None:
            raise DsparkError("row_off needs a Sampler made with requests")
        else:
            n = self.requests
            a.row_off = _vec(row_off, n + 1, i32, "row_off", dev)
        a.temperature = _vec(temperature, n, f32, "temperature", dev)
        a.top_k = _vec(top_k, n, i32, "top_k", dev)
        a.top_p = _vec(top_p, n, f32, "top_p", dev)
        a.min_p = _vec(min_p, n, f32, "min_p", dev)
        return pz

    def sample(self, Z, u, temperature=None, top_k=None, top_p=None, min_p=None, row_off=None, out=None, stream=None):
        """token [N] int32 and logp [N] fp32 drawn with u [N] fp32 in [0, 1);
        rows that ``row_off`` gives to no request are left as they are."""
        made = out is None
        if made:
            out = {"token": self._new((self.N,), torch.int32, stream), "logp": self._new((self.N,), torch.float32, stream)}
        dev, f32 = self._index, torch.float32
        pz = self._set(Z, row_off, temperature, top_k, top_p, min_p)
        pu = _vec(u, self.N, f32, "u", dev)
        if made:
            pt, pl = out["token"].data_ptr(), out["logp"].data_ptr()
        else:
            pt, pl = _vec(out["token"], self.N, torch.int32, "token", dev), _vec(out.get("logp"), self.N, f32, "logp", dev)
        r = self._call(self.lib.dspark_sample, self._pargs, pz, pu, pt, pl, self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_sample")
        return out

    def logprobs(self, Z, temperature=None, top_k=None, top_p=None, min_p=None, row_off=None,
                 fill: float = float("-inf"), out=None, stream=None):
        """[N, V] fp32: the log-probabilities that ``sample`` draws with, ``fill`` where a token is left out."""
        if out is None:
            out = self._new((self.N, self.V), torch.float32, stream)
        pz = self._set(Z, row_off, temperature, top_k, top_p, min_p)
        po, ldo = _rows(out, self.N, self.V, torch.float32, "out", self._index)
        r = self._call(self.lib.dspark_sample_logprobs, self._pargs, pz, fill, po, ldo,
                       self.status.data_ptr(), self._on(stream))
        _check(r, "dspark_sample_logprobs")
        return out
