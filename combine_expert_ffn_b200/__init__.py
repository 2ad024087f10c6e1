"""Python binding of libmoe, the B200 (sm_100a) MoE-layer forward library.

Argument marshalling only: every function below forwards torch tensors'
device pointers and the current CUDA stream to the C entry point of the same
name in ``include/moe.h`` and raises :class:`MoeError` on a nonzero status.
All arithmetic happens in the library's CUDA kernels; there is no CPU or
PyTorch fallback.  If ``libmoe.so`` is missing the import fails -- build it
with ``python combine_expert_ffn_b200/build.py``.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: run `python combine_expert_ffn_b200/build.py`")

_lib = C.CDLL(LIB_PATH)

STATUS = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
    3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_TIMEOUT",
    6: "MOE_ERR_DEVICE_FAULT", 7: "MOE_ERR_NO_DEVICE",
}
MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_WORKSPACE_TOO_SMALL, \
    MOE_ERR_CUDA, MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_DEVICE_FAULT, MOE_ERR_NO_DEVICE = range(8)

EXPORTS = ("moe_check_config", "moe_workspace_size", "moe_status_string", "moe_launch_count",
           "moe_read_device_status", "moe_last_device_status", "moe_clear_device_status",
           "moe_route", "moe_route_select",
           "moe_dispatch", "moe_expert_ffn", "moe_combine", "moe_forward",
           "moe_selftest_bounded_wait", "moe_dispatch_noalloc", "moe_route_hash",
           "moe_bias_update", "moe_expert_ffn_gather", "moe_dispatch_fp8",
           "moe_expert_ffn_fp8", "moe_permute", "moe_ep_workspace_size", "moe_ep_plan",
           "moe_ep_dispatch", "moe_ep_expert_ffn", "moe_ep_combine", "moe_ep_dispatch_fp8",
           "moe_ep_expert_ffn_fp8", "moe_ep_token_plan", "moe_ep_token_base",
           "moe_ep_dispatch_dedup", "moe_ep_fanout", "moe_ep_dispatch_dedup_fp8",
           "moe_ep_fanout_fp8", "moe_ep_combine_plan", "moe_ep_dispatch_dedup_plan",
           "moe_ep_precombine", "moe_ep_combine_dedup", "moe_ipc_get_handle",
           "moe_ipc_open_handle", "moe_ipc_close_handle", "moe_packed_weights_size",
           "moe_pack_weights", "moe_expert_ffn_packed", "moe_forward_packed",
           "moe_balance_loss", "moe_route_backward", "moe_combine_backward",
           "moe_int8_workspace_size", "moe_quantize_weights_int8", "moe_dispatch_int8",
           "moe_expert_ffn_int8", "moe_forward_int8")

MOE_ROUTER_SIGMOID, MOE_ROUTER_SQRT_SOFTPLUS, MOE_ROUTER_HASH = 0, 1, 2
MOE_PAYLOAD_BF16, MOE_PAYLOAD_FP8 = 0, 1


class MoeConfig(C.Structure):
    """Mirror of ``moe_config``."""
    _fields_ = [(n, C.c_int32) for n in
                ("T", "d", "E", "G", "K", "M", "d_ff", "n_shared", "d_ff_shared", "router",
                 "payload")]

    @classmethod
    def of(cls, shape, router=None, payload=None) -> "MoeConfig":
        """From any object with the nine size attributes (e.g. ``synth.MoeShape``);
        router and payload from the arguments, else the object's, else the defaults
        (sigmoid router, bf16 payload)."""
        if router is None:
            router = getattr(shape, "router", MOE_ROUTER_SIGMOID)
        if payload is None:
            payload = getattr(shape, "payload", MOE_PAYLOAD_BF16)
        return cls(*(int(getattr(shape, n)) for n, _ in cls._fields_[:-2]), int(router),
                   int(payload))

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class Int8Weights(C.Structure):
    """Mirror of ``moe_int8_weights`` that keeps the tensors it points to.

    ``Int8Weights(w_gate=..., w_gate_scale=..., ...)`` takes int8 codes and fp32 scales of the
    header's layouts (the ``ws_`` ones only for a layer with shared experts); they become
    attributes of ``tensors``.  ``quantize_weights_int8`` makes one from bf16 weights.
    """
    _codes = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")
    _fields_ = [(n, C.c_void_p) for n in _codes] + [(n + "_scale", C.c_void_p) for n in _codes]

    def __init__(self, **tensors):
        names = {n for n, _ in self._fields_}
        for n, t in tensors.items():
            if n not in names:
                raise TypeError(f"Int8Weights: no field {n!r}")
            if t is not None and (t.dtype != (torch.int8 if n in self._codes else torch.float32)
                                  or not t.is_contiguous()):
                raise TypeError(f"Int8Weights: {n} must be a contiguous tensor of int8 codes or "
                                "fp32 scales")
        super().__init__(**{n: None if t is None else t.data_ptr() for n, t in tensors.items()})
        self.tensors = dict(tensors)

    def check(self, fn, c):
        """Raises MoeError unless every tensor given has the size of configuration ``c`` and lies
        on the current GPU.  A passed configuration is remembered: the tensors never change."""
        key = (c.d, c.E, c.d_ff, c.n_shared, c.d_ff_shared)
        if key == self.__dict__.get("_checked") and self._device == torch.cuda.current_device():
            return
        k = _Call(fn, c)
        up, up_s = c.d_ff, c.n_shared * c.d_ff_shared
        sizes = {"w_gate": c.E * up * c.d, "w_up": c.E * up * c.d, "w_down": c.E * up * c.d,
                 "w_gate_scale": c.E * up, "w_up_scale": c.E * up, "w_down_scale": c.E * c.d,
                 "ws_gate": up_s * c.d, "ws_up": up_s * c.d, "ws_down": up_s * c.d,
                 "ws_gate_scale": up_s, "ws_up_scale": up_s, "ws_down_scale": c.d}
        for n, t in self.tensors.items():
            if t is not None and (c.n_shared > 0 or not n.startswith("ws_")):
                k.t(t, t.dtype, sizes[n])
        self._checked, self._device = key, k.dev


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({moe_status_string(status)})")


_P, _S, _I64 = C.c_void_p, C.c_size_t, C.c_int64
_CP = C.POINTER(MoeConfig)
_sig = {
    "moe_check_config": (C.c_int, [_CP]),
    "moe_workspace_size": (_S, [_CP]),
    "moe_status_string": (C.c_char_p, [C.c_int]),
    "moe_launch_count": (C.c_uint64, []),
    "moe_read_device_status": (C.c_int, [_P, _P, _P]),
    "moe_last_device_status": (C.c_int, [_P, _P]),
    "moe_clear_device_status": (C.c_int, [_P, _P]),
    "moe_route": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_route_select": (C.c_int, [_CP, _P, _P, _P, _P, _P]),
    "moe_dispatch": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_expert_ffn": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_combine": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P]),
    "moe_forward": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                              _P, _P, _P, _P, _P, _S, _P]),
    "moe_route_hash": (C.c_int, [_CP, _P, _P, _P, _P]),
    "moe_permute": (C.c_int, [_CP, _P, _P, _P, _P]),
    "moe_ep_workspace_size": (_S, [_CP, C.c_int32]),
    "moe_ep_plan": (C.c_int, [_CP, C.c_int32, C.c_int32, _P, _P, _P, _P]),
    "moe_ep_dispatch": (C.c_int, [_CP, C.c_int32, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_ep_expert_ffn": (C.c_int, [_CP, C.c_int32, C.c_int32, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _P, _P, _S, _P]),
    "moe_ep_combine": (C.c_int, [_CP, C.c_int32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_ep_token_plan": (C.c_int, [_CP, C.c_int32, _P, _P, _P, _P]),
    "moe_ep_token_base": (C.c_int, [_CP, C.c_int32, C.c_int32, _P, _P, _P]),
    "moe_ep_dispatch_dedup": (C.c_int, [_CP, C.c_int32] + [_P] * 11),
    "moe_ep_fanout": (C.c_int, [_CP, C.c_int32] + [_P] * 6),
    "moe_ep_dispatch_dedup_fp8": (C.c_int, [_CP, C.c_int32] + [_P] * 12),
    "moe_ep_fanout_fp8": (C.c_int, [_CP, C.c_int32] + [_P] * 8),
    "moe_ep_combine_plan": (C.c_int, [_CP, C.c_int32] + [_P] * 12),
    "moe_ep_dispatch_dedup_plan": (C.c_int, [_CP, C.c_int32] + [_P] * 15),
    "moe_ep_precombine": (C.c_int, [_CP, C.c_int32] + [_P] * 8),
    "moe_ep_combine_dedup": (C.c_int, [_CP, C.c_int32] + [_P] * 8),
    "moe_ep_dispatch_fp8": (C.c_int, [_CP, C.c_int32, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_ep_expert_ffn_fp8": (C.c_int, [_CP, C.c_int32, C.c_int32, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_ipc_get_handle": (C.c_int, [_P, _P]),
    "moe_ipc_open_handle": (C.c_int, [_P, _P]),
    "moe_ipc_close_handle": (C.c_int, [_P]),
    "moe_dispatch_fp8": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_expert_ffn_fp8": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S,
                                     _P]),
    "moe_expert_ffn_gather": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S,
                                        _P]),
    "moe_bias_update": (C.c_int, [_CP, _P, C.c_float, _P, _P]),
    "moe_selftest_bounded_wait": (C.c_int, [_I64, _P, _P]),
    "moe_dispatch_noalloc": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_packed_weights_size": (_S, [_CP]),
    "moe_pack_weights": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_expert_ffn_packed": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_forward_packed": (C.c_int, [_CP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _P, _S, _P]),
}
_WP = C.POINTER(Int8Weights)
_F32, _I32 = C.c_float, C.c_int32
_sig |= {
    "moe_balance_loss": (C.c_int, [_CP, _P, _P, _P, _I32, _F32, _P, _P, _P, _P, _S, _P]),
    "moe_route_backward": (C.c_int, [_CP, _P, _P, _P, _P, _I32, _P, _P, _F32, _P, _P, _P]),
    "moe_combine_backward": (C.c_int, [_CP] + [_P] * 7),
    "moe_int8_workspace_size": (_S, [_CP]),
    "moe_quantize_weights_int8": (C.c_int, [_CP] + [_P] * 6 + [_WP, _P]),
    "moe_dispatch_int8": (C.c_int, [_CP] + [_P] * 11 + [_S, _P]),
    "moe_expert_ffn_int8": (C.c_int, [_CP, _P, _P, _P, _WP, _P, _P, _P, _P, _S, _P]),
    "moe_forward_int8": (C.c_int, [_CP] + [_P] * 5 + [_WP] + [_P] * 8 + [_S, _P]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _cfg(cfg):
    return C.byref(cfg if isinstance(cfg, MoeConfig) else MoeConfig.of(cfg))


def _ok(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st)


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


class _Call:
    """One call of an entry point that checks its tensors: ``c`` the configuration, ``stream(s)``
    the stream's handle, ``t(tensor, dtype, numel)`` the device pointer of a tensor that has this
    dtype, is contiguous, holds at least ``numel`` elements and lies on the current GPU (None and
    raw device pointers pass as they are; anything else raises MoeError).  The current device is
    asked for once, and only where there is a tensor on a GPU."""
    __slots__ = ("fn", "c", "dev")

    def __init__(self, fn, cfg):
        self.fn = fn
        self.c = cfg if isinstance(cfg, MoeConfig) else MoeConfig.of(cfg)
        self.dev = None

    def t(self, t, dtype, numel):
        if t is None or isinstance(t, int):
            return t
        if t.dtype is dtype and t.numel() >= numel and t.is_contiguous():
            dev = t.get_device()  # -1 on the host
            if dev == self.dev:
                return t.data_ptr()
            if dev >= 0 and self.dev is None and dev == torch.cuda.current_device():
                self.dev = dev
                return t.data_ptr()
        raise MoeError(self.fn, MOE_ERR_INVALID_ARG)

    def weights(self, w):
        """A reference to an Int8Weights whose tensors fit the configuration; None passes."""
        if w is None:
            return None
        if not isinstance(w, Int8Weights):
            raise MoeError(self.fn, MOE_ERR_INVALID_ARG)
        w.check(self.fn, self.c)
        return C.byref(w)

    def ws(self, ws):
        """(device pointer, bytes) of a workspace tensor."""
        if ws is None:
            return None, 0
        if ws.get_device() != torch.cuda.current_device():
            raise MoeError(self.fn, MOE_ERR_INVALID_ARG)
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def sequences(self, seq_offsets):
        """(device pointer, number of sequences) of a seq_offsets argument."""
        if seq_offsets is None:
            return None, 1
        n = seq_offsets.numel() - 1
        if n < 0:
            raise MoeError(self.fn, MOE_ERR_INVALID_ARG)
        return self.t(seq_offsets, torch.int32, 1), n

    def stream(self, stream):
        if stream is None and self.dev is not None:
            return _raw_stream(self.dev)
        return _stream(stream)


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the handle without a Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream


# ----------------------------------------------------------------- queries
def moe_check_config(cfg) -> int:
    return _lib.moe_check_config(_cfg(cfg))


def moe_workspace_size(cfg) -> int:
    return _lib.moe_workspace_size(_cfg(cfg))


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def moe_launch_count() -> int:
    return _lib.moe_launch_count()


def alloc_workspace(cfg, device="cuda") -> torch.Tensor:
    """Device workspace of moe_workspace_size(cfg) bytes (torch blocks are 512-byte aligned)."""
    n = moe_workspace_size(cfg)
    if n == 0:
        raise MoeError("moe_workspace_size", moe_check_config(cfg) or MOE_ERR_UNSUPPORTED_SHAPE)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_read_device_status(ws, stream=None) -> int:
    out = C.c_int32(-1)
    _ok("moe_read_device_status", _lib.moe_read_device_status(_ptr(ws), C.byref(out), _stream(stream)))
    return out.value


def moe_last_device_status(ws, stream=None) -> int:
    """The device status word (synchronises the stream); host-side read errors as codes."""
    return int(_lib.moe_last_device_status(_ptr(ws), _stream(stream)))


def moe_clear_device_status(ws, stream=None) -> None:
    _ok("moe_clear_device_status", _lib.moe_clear_device_status(_ptr(ws), _stream(stream)))


# ----------------------------------------------------------------- stages
def moe_route(cfg, x, router_w, logit_offset, bias, topk_idx, topk_w, scores=None, ws=None,
              stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_route", _lib.moe_route(_cfg(cfg), _ptr(x), _ptr(router_w), _ptr(logit_offset),
                                    _ptr(bias), _ptr(topk_idx), _ptr(topk_w), _ptr(scores), wp, wn,
                                    _stream(stream)))


def moe_route_hash(cfg, token_ids, topk_idx, topk_w, stream=None) -> None:
    _ok("moe_route_hash", _lib.moe_route_hash(_cfg(cfg), _ptr(token_ids), _ptr(topk_idx),
                                              _ptr(topk_w), _stream(stream)))


def moe_bias_update(cfg, counts, gamma, bias, stream=None) -> None:
    _ok("moe_bias_update", _lib.moe_bias_update(_cfg(cfg), _ptr(counts), C.c_float(gamma),
                                                _ptr(bias), _stream(stream)))


def moe_route_select(cfg, scores, bias, topk_idx, topk_w, stream=None) -> None:
    _ok("moe_route_select", _lib.moe_route_select(_cfg(cfg), _ptr(scores), _ptr(bias),
                                                  _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


def moe_dispatch(cfg, x, topk_idx, counts, offsets, send, send_tok, perm_token, inv_perm, x_perm,
                 ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_dispatch", _lib.moe_dispatch(_cfg(cfg), _ptr(x), _ptr(topk_idx), _ptr(counts),
                                          _ptr(offsets), _ptr(send), _ptr(send_tok),
                                          _ptr(perm_token), _ptr(inv_perm), _ptr(x_perm), wp, wn,
                                          _stream(stream)))


def moe_expert_ffn(cfg, x_perm, offsets, w_gate, w_up, w_down, y_perm, x, ws_gate, ws_up, ws_down,
                   y_shared, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_expert_ffn", _lib.moe_expert_ffn(_cfg(cfg), _ptr(x_perm), _ptr(offsets), _ptr(w_gate),
                                              _ptr(w_up), _ptr(w_down), _ptr(y_perm), _ptr(x),
                                              _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down),
                                              _ptr(y_shared), wp, wn, _stream(stream)))


def moe_expert_ffn_gather(cfg, x, perm_token, offsets, w_gate, w_up, w_down, y_perm, ws_gate,
                          ws_up, ws_down, y_shared, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_expert_ffn_gather",
        _lib.moe_expert_ffn_gather(_cfg(cfg), _ptr(x), _ptr(perm_token), _ptr(offsets),
                                   _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y_perm),
                                   _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(y_shared), wp,
                                   wn, _stream(stream)))


def moe_permute(cfg, x, inv_perm, x_perm, stream=None) -> None:
    _ok("moe_permute", _lib.moe_permute(_cfg(cfg), _ptr(x), _ptr(inv_perm), _ptr(x_perm),
                                        _stream(stream)))


# ----------------------------------------------------------------- the router's training side
def moe_balance_loss(cfg, scores, topk_idx, seq_offsets, alpha, counts, prob, loss, ws,
                     stream=None) -> None:
    """Per-sequence balance loss, counts and mean affinities (seq_offsets None: one sequence)."""
    k = _Call("moe_balance_loss", cfg)
    c, t, f32, i32 = k.c, k.t, torch.float32, torch.int32
    seq, n = k.sequences(seq_offsets)
    _ok(k.fn, _lib.moe_balance_loss(
        C.byref(c), t(scores, f32, c.T * c.E), t(topk_idx, i32, c.T * c.K), seq, n, alpha,
        t(counts, i32, n * c.E), t(prob, f32, n * c.E), t(loss, f32, n), *k.ws(ws),
        k.stream(stream)))


def moe_route_backward(cfg, scores, topk_idx, d_topk_w, seq_offsets, counts, d_loss, alpha,
                       d_logits, device_status=None, stream=None) -> None:
    """Gradient of the gates (d_topk_w, or None) and of the balance loss (d_loss, or None) with
    respect to the router's logits."""
    k = _Call("moe_route_backward", cfg)
    c, t, f32, i32 = k.c, k.t, torch.float32, torch.int32
    seq, n = k.sequences(seq_offsets) if d_loss is not None else (None, 1)
    _ok(k.fn, _lib.moe_route_backward(
        C.byref(c), t(scores, f32, c.T * c.E), t(topk_idx, i32, c.T * c.K),
        t(d_topk_w, f32, c.T * c.K), seq, n, t(counts, i32, n * c.E), t(d_loss, f32, n), alpha,
        t(d_logits, f32, c.T * c.E), t(device_status, i32, 1), k.stream(stream)))


def moe_combine_backward(cfg, d_out, y_perm, inv_perm, topk_w, d_y_perm, d_topk_w,
                         stream=None) -> None:
    k = _Call("moe_combine_backward", cfg)
    c, t, f32, bf16 = k.c, k.t, torch.float32, torch.bfloat16
    rows = c.T * c.K
    _ok(k.fn, _lib.moe_combine_backward(
        C.byref(c), t(d_out, bf16, c.T * c.d), t(y_perm, bf16, rows * c.d),
        t(inv_perm, torch.int32, rows), t(topk_w, f32, rows), t(d_y_perm, bf16, rows * c.d),
        t(d_topk_w, f32, rows), k.stream(stream)))


# ----------------------------------------------------------------- experts in int8
def moe_int8_workspace_size(cfg) -> int:
    return _lib.moe_int8_workspace_size(_cfg(cfg))


def alloc_int8_workspace(cfg, device="cuda") -> torch.Tensor:
    """Device workspace of moe_int8_workspace_size(cfg) bytes; serves every entry point."""
    n = moe_int8_workspace_size(cfg)
    if n == 0:
        raise MoeError("moe_int8_workspace_size",
                       moe_check_config(cfg) or MOE_ERR_UNSUPPORTED_SHAPE)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_quantize_weights_int8(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, weights,
                              stream=None) -> None:
    k = _Call("moe_quantize_weights_int8", cfg)
    c = k.c
    w8 = k.weights(weights)
    n, ns = c.E * c.d_ff * c.d, c.n_shared * c.d_ff_shared * c.d
    ptrs = [k.t(w, torch.bfloat16, n) for w in (w_gate, w_up, w_down)]
    ptrs += [k.t(w, torch.bfloat16, ns) for w in (ws_gate, ws_up, ws_down)]
    _ok(k.fn, _lib.moe_quantize_weights_int8(C.byref(c), *ptrs, w8, k.stream(stream)))


def quantize_weights_int8(cfg, w_gate, w_up, w_down, ws_gate=None, ws_up=None, ws_down=None,
                          stream=None) -> Int8Weights:
    """Allocates codes and scales for the bf16 weights and fills them with
    moe_quantize_weights_int8.  (On a stream that is not the current one, the caller orders the
    allocation before it.)"""
    c = cfg if isinstance(cfg, MoeConfig) else MoeConfig.of(cfg)
    dev = w_gate.device
    ns, ffs = c.n_shared, c.d_ff_shared
    shapes = {"w_gate": (c.E, c.d_ff, c.d), "w_up": (c.E, c.d_ff, c.d), "w_down": (c.E, c.d, c.d_ff)}
    scales = {"w_gate": (c.E, c.d_ff), "w_up": (c.E, c.d_ff), "w_down": (c.E, c.d)}
    if ns > 0:
        shapes |= {"ws_gate": (ns, ffs, c.d), "ws_up": (ns, ffs, c.d), "ws_down": (ns, c.d, ffs)}
        scales |= {"ws_gate": (ns, ffs), "ws_up": (ns, ffs), "ws_down": (c.d,)}
    t = {n: torch.empty(s, dtype=torch.int8, device=dev) for n, s in shapes.items()}
    t |= {n + "_scale": torch.empty(s, dtype=torch.float32, device=dev) for n, s in scales.items()}
    w = Int8Weights(**t)
    moe_quantize_weights_int8(c, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, w, stream)
    return w


def moe_dispatch_int8(cfg, x, topk_idx, counts, offsets, send, send_tok, perm_token, inv_perm,
                      x_perm_q, x_scale, ws, stream=None) -> None:
    k = _Call("moe_dispatch_int8", cfg)
    c, t, i32 = k.c, k.t, torch.int32
    rows, groups = c.T * c.K, c.G * c.G
    _ok(k.fn, _lib.moe_dispatch_int8(
        C.byref(c), t(x, torch.bfloat16, c.T * c.d), t(topk_idx, i32, rows), t(counts, i32, c.E),
        t(offsets, i32, c.E + 1), t(send, i32, groups), t(send_tok, i32, groups),
        t(perm_token, i32, rows), t(inv_perm, i32, rows), t(x_perm_q, torch.int8, rows * c.d),
        t(x_scale, torch.float32, rows), *k.ws(ws), k.stream(stream)))


def moe_expert_ffn_int8(cfg, x_perm_q, x_scale, offsets, weights, y_perm, x, y_shared, ws,
                        stream=None) -> None:
    """weights: Int8Weights."""
    k = _Call("moe_expert_ffn_int8", cfg)
    c, t, bf16 = k.c, k.t, torch.bfloat16
    rows = c.T * c.K
    w8 = k.weights(weights)
    _ok(k.fn, _lib.moe_expert_ffn_int8(
        C.byref(c), t(x_perm_q, torch.int8, rows * c.d), t(x_scale, torch.float32, rows),
        t(offsets, torch.int32, c.E + 1), w8, t(y_perm, bf16, rows * c.d),
        t(x, bf16, c.T * c.d), t(y_shared, bf16, c.T * c.d), *k.ws(ws), k.stream(stream)))


def moe_forward_int8(cfg, x, router_w, logit_offset, bias, weights, out, topk_idx=None,
                     topk_w=None, counts=None, offsets=None, send=None, send_tok=None, ws=None,
                     stream=None, token_ids=None) -> None:
    """weights: Int8Weights; ws: alloc_int8_workspace(cfg)."""
    k = _Call("moe_forward_int8", cfg)
    c, t, i32, f32 = k.c, k.t, torch.int32, torch.float32
    rows, groups = c.T * c.K, c.G * c.G
    w8 = k.weights(weights)
    _ok(k.fn, _lib.moe_forward_int8(
        C.byref(c), t(x, torch.bfloat16, c.T * c.d), t(router_w, f32, c.E * c.d),
        t(logit_offset, f32, c.E), t(bias, f32, c.E), t(token_ids, torch.int64, c.T),
        w8, t(out, torch.bfloat16, c.T * c.d), t(topk_idx, i32, rows),
        t(topk_w, f32, rows), t(counts, i32, c.E), t(offsets, i32, c.E + 1),
        t(send, i32, groups), t(send_tok, i32, groups), *k.ws(ws), k.stream(stream)))


# ----------------------------------------------------------------- expert parallelism
def moe_ep_workspace_size(cfg, world) -> int:
    return _lib.moe_ep_workspace_size(_cfg(cfg), int(world))


def moe_ep_plan(cfg, world, rank, counts_all, base, local_offsets, stream=None) -> None:
    _ok("moe_ep_plan", _lib.moe_ep_plan(_cfg(cfg), int(world), int(rank), _ptr(counts_all),
                                        _ptr(base), _ptr(local_offsets), _stream(stream)))


def moe_ep_dispatch(cfg, world, x, topk_idx, offsets, inv_perm, base, recv_x_ptrs,
                    device_status=None, stream=None) -> None:
    """recv_x_ptrs: device int64 tensor of `world` device pointers."""
    _ok("moe_ep_dispatch",
        _lib.moe_ep_dispatch(_cfg(cfg), int(world), _ptr(x), _ptr(topk_idx), _ptr(offsets),
                             _ptr(inv_perm), _ptr(base), _ptr(recv_x_ptrs), _ptr(device_status),
                             _stream(stream)))


def moe_ep_expert_ffn(cfg, world, rank, recv_x, local_offsets, w_gate, w_up, w_down, recv_y, x,
                      ws_gate, ws_up, ws_down, y_shared, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_ep_expert_ffn",
        _lib.moe_ep_expert_ffn(_cfg(cfg), int(world), int(rank), _ptr(recv_x),
                               _ptr(local_offsets), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                               _ptr(recv_y), _ptr(x), _ptr(ws_gate), _ptr(ws_up),
                               _ptr(ws_down), _ptr(y_shared), wp, wn, _stream(stream)))


def moe_ep_token_plan(cfg, world, topk_idx, tok_slot, tok_counts, stream=None) -> None:
    _ok("moe_ep_token_plan",
        _lib.moe_ep_token_plan(_cfg(cfg), int(world), _ptr(topk_idx), _ptr(tok_slot),
                               _ptr(tok_counts), _stream(stream)))


def moe_ep_token_base(cfg, world, rank, tok_counts_all, tok_base, stream=None) -> None:
    _ok("moe_ep_token_base",
        _lib.moe_ep_token_base(_cfg(cfg), int(world), int(rank), _ptr(tok_counts_all),
                               _ptr(tok_base), _stream(stream)))


def moe_ep_dispatch_dedup(cfg, world, x, topk_idx, offsets, inv_perm, base, tok_slot, tok_base,
                          recv_tok_ptrs, recv_idx_ptrs, device_status=None, stream=None) -> None:
    """recv_tok_ptrs / recv_idx_ptrs: device int64 tensors of `world` device pointers."""
    _ok("moe_ep_dispatch_dedup",
        _lib.moe_ep_dispatch_dedup(_cfg(cfg), int(world), _ptr(x), _ptr(topk_idx), _ptr(offsets),
                                   _ptr(inv_perm), _ptr(base), _ptr(tok_slot), _ptr(tok_base),
                                   _ptr(recv_tok_ptrs), _ptr(recv_idx_ptrs), _ptr(device_status),
                                   _stream(stream)))


def moe_ep_fanout(cfg, world, recv_tok, recv_idx, local_offsets, recv_x, device_status=None,
                  stream=None) -> None:
    _ok("moe_ep_fanout",
        _lib.moe_ep_fanout(_cfg(cfg), int(world), _ptr(recv_tok), _ptr(recv_idx),
                           _ptr(local_offsets), _ptr(recv_x), _ptr(device_status),
                           _stream(stream)))


def moe_ep_dispatch_dedup_fp8(cfg, world, x, topk_idx, offsets, inv_perm, base, tok_slot,
                              tok_base, recv_tq_ptrs, recv_ts_ptrs, recv_idx_ptrs,
                              device_status=None, stream=None) -> None:
    _ok("moe_ep_dispatch_dedup_fp8",
        _lib.moe_ep_dispatch_dedup_fp8(_cfg(cfg), int(world), _ptr(x), _ptr(topk_idx),
                                       _ptr(offsets), _ptr(inv_perm), _ptr(base), _ptr(tok_slot),
                                       _ptr(tok_base), _ptr(recv_tq_ptrs), _ptr(recv_ts_ptrs),
                                       _ptr(recv_idx_ptrs), _ptr(device_status), _stream(stream)))


def moe_ep_fanout_fp8(cfg, world, recv_tq, recv_ts, recv_idx, local_offsets, recv_q, recv_scale,
                      device_status=None, stream=None) -> None:
    _ok("moe_ep_fanout_fp8",
        _lib.moe_ep_fanout_fp8(_cfg(cfg), int(world), _ptr(recv_tq), _ptr(recv_ts),
                               _ptr(recv_idx), _ptr(local_offsets), _ptr(recv_q),
                               _ptr(recv_scale), _ptr(device_status), _stream(stream)))


def moe_ep_combine_plan(cfg, world, topk_idx, topk_w, offsets, inv_perm, base, tok_slot, tok_base,
                        list_ptrs, lw_ptrs, lcnt_ptrs, device_status=None, stream=None) -> None:
    _ok("moe_ep_combine_plan",
        _lib.moe_ep_combine_plan(_cfg(cfg), int(world), _ptr(topk_idx), _ptr(topk_w),
                                 _ptr(offsets), _ptr(inv_perm), _ptr(base), _ptr(tok_slot),
                                 _ptr(tok_base), _ptr(list_ptrs), _ptr(lw_ptrs), _ptr(lcnt_ptrs),
                                 _ptr(device_status), _stream(stream)))


def moe_ep_dispatch_dedup_plan(cfg, world, x, topk_idx, topk_w, offsets, inv_perm, base,
                               tok_slot, tok_base, recv_tok_ptrs, recv_idx_ptrs, list_ptrs,
                               lw_ptrs, lcnt_ptrs, device_status=None, stream=None) -> None:
    """moe_ep_dispatch_dedup + moe_ep_combine_plan in one launch (same outputs)."""
    _ok("moe_ep_dispatch_dedup_plan",
        _lib.moe_ep_dispatch_dedup_plan(_cfg(cfg), int(world), _ptr(x), _ptr(topk_idx),
                                        _ptr(topk_w), _ptr(offsets), _ptr(inv_perm), _ptr(base),
                                        _ptr(tok_slot), _ptr(tok_base), _ptr(recv_tok_ptrs),
                                        _ptr(recv_idx_ptrs), _ptr(list_ptrs), _ptr(lw_ptrs),
                                        _ptr(lcnt_ptrs), _ptr(device_status), _stream(stream)))


def moe_ep_precombine(cfg, world, recv_y, lst, lw, lcnt, tok_base, partial, device_status=None,
                      stream=None) -> None:
    _ok("moe_ep_precombine",
        _lib.moe_ep_precombine(_cfg(cfg), int(world), _ptr(recv_y), _ptr(lst), _ptr(lw),
                               _ptr(lcnt), _ptr(tok_base), _ptr(partial), _ptr(device_status),
                               _stream(stream)))


def moe_ep_combine_dedup(cfg, world, topk_idx, tok_slot, tok_base, partial_ptrs, y_shared, out,
                         device_status=None, stream=None) -> None:
    _ok("moe_ep_combine_dedup",
        _lib.moe_ep_combine_dedup(_cfg(cfg), int(world), _ptr(topk_idx), _ptr(tok_slot),
                                  _ptr(tok_base), _ptr(partial_ptrs), _ptr(y_shared), _ptr(out),
                                  _ptr(device_status), _stream(stream)))


def moe_ep_dispatch_fp8(cfg, world, x, topk_idx, offsets, inv_perm, base, recv_q_ptrs,
                        recv_scale_ptrs, device_status=None, stream=None) -> None:
    """recv_q_ptrs / recv_scale_ptrs: device int64 tensors of `world` device pointers."""
    _ok("moe_ep_dispatch_fp8",
        _lib.moe_ep_dispatch_fp8(_cfg(cfg), int(world), _ptr(x), _ptr(topk_idx), _ptr(offsets),
                                 _ptr(inv_perm), _ptr(base), _ptr(recv_q_ptrs),
                                 _ptr(recv_scale_ptrs), _ptr(device_status), _stream(stream)))


def moe_ep_expert_ffn_fp8(cfg, world, rank, recv_q, recv_scale, local_offsets, w_gate, w_up,
                          w_down, recv_y, x, ws_gate, ws_up, ws_down, y_shared, ws,
                          stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_ep_expert_ffn_fp8",
        _lib.moe_ep_expert_ffn_fp8(_cfg(cfg), int(world), int(rank), _ptr(recv_q),
                                   _ptr(recv_scale), _ptr(local_offsets), _ptr(w_gate),
                                   _ptr(w_up), _ptr(w_down), _ptr(recv_y), _ptr(x),
                                   _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(y_shared), wp,
                                   wn, _stream(stream)))


def moe_ep_combine(cfg, world, topk_idx, topk_w, offsets, inv_perm, base, recv_y_ptrs, y_shared,
                   out, device_status=None, stream=None) -> None:
    _ok("moe_ep_combine",
        _lib.moe_ep_combine(_cfg(cfg), int(world), _ptr(topk_idx), _ptr(topk_w), _ptr(offsets),
                            _ptr(inv_perm), _ptr(base), _ptr(recv_y_ptrs), _ptr(y_shared),
                            _ptr(out), _ptr(device_status), _stream(stream)))


MOE_IPC_HANDLE_BYTES = 72


def moe_ipc_get_handle(t) -> bytes:
    h = (C.c_char * MOE_IPC_HANDLE_BYTES)()
    _ok("moe_ipc_get_handle", _lib.moe_ipc_get_handle(_ptr(t), C.cast(h, C.c_void_p)))
    return bytes(h)


def moe_ipc_open_handle(handle: bytes) -> int:
    buf = (C.c_char * MOE_IPC_HANDLE_BYTES).from_buffer_copy(handle)
    p = C.c_void_p()
    _ok("moe_ipc_open_handle", _lib.moe_ipc_open_handle(C.cast(buf, C.c_void_p), C.byref(p)))
    return p.value


def moe_ipc_close_handle(ptr: int) -> None:
    _ok("moe_ipc_close_handle", _lib.moe_ipc_close_handle(C.c_void_p(ptr)))


def moe_dispatch_fp8(cfg, x, topk_idx, counts, offsets, send, send_tok, perm_token, inv_perm,
                     x_perm_q, x_scale, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_dispatch_fp8",
        _lib.moe_dispatch_fp8(_cfg(cfg), _ptr(x), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                              _ptr(send), _ptr(send_tok), _ptr(perm_token), _ptr(inv_perm),
                              _ptr(x_perm_q), _ptr(x_scale), wp, wn, _stream(stream)))


def moe_expert_ffn_fp8(cfg, x_perm_q, x_scale, offsets, w_gate, w_up, w_down, y_perm, x, ws_gate,
                       ws_up, ws_down, y_shared, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_expert_ffn_fp8",
        _lib.moe_expert_ffn_fp8(_cfg(cfg), _ptr(x_perm_q), _ptr(x_scale), _ptr(offsets),
                                _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y_perm), _ptr(x),
                                _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(y_shared), wp, wn,
                                _stream(stream)))


def moe_combine(cfg, y_perm, inv_perm, topk_w, y_shared, out, stream=None) -> None:
    _ok("moe_combine", _lib.moe_combine(_cfg(cfg), _ptr(y_perm), _ptr(inv_perm), _ptr(topk_w),
                                        _ptr(y_shared), _ptr(out), _stream(stream)))


def moe_forward(cfg, x, router_w, logit_offset, bias, w_gate, w_up, w_down, ws_gate, ws_up,
                ws_down, out, topk_idx=None, topk_w=None, counts=None, offsets=None, send=None,
                send_tok=None, ws=None, stream=None, token_ids=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_forward", _lib.moe_forward(_cfg(cfg), _ptr(x), _ptr(router_w), _ptr(logit_offset),
                                        _ptr(bias), _ptr(token_ids), _ptr(w_gate), _ptr(w_up),
                                        _ptr(w_down),
                                        _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(out),
                                        _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                                        _ptr(send), _ptr(send_tok), wp, wn, _stream(stream)))


def moe_packed_weights_size(cfg) -> int:
    return int(_lib.moe_packed_weights_size(_cfg(cfg)))


def moe_pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed,
                     stream=None) -> None:
    _ok("moe_pack_weights", _lib.moe_pack_weights(_cfg(cfg), _ptr(w_gate), _ptr(w_up),
                                                  _ptr(w_down), _ptr(ws_gate), _ptr(ws_up),
                                                  _ptr(ws_down), _ptr(packed), _stream(stream)))


def pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, device="cuda",
                 stream=None):
    """Allocates the packed-weight buffer (uint8) and fills it with moe_pack_weights."""
    n = moe_packed_weights_size(cfg)
    if n == 0:
        raise MoeError("moe_packed_weights_size", MOE_ERR_UNSUPPORTED_SHAPE)
    packed = torch.empty(n, dtype=torch.uint8, device=device)
    moe_pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed, stream)
    return packed


def moe_expert_ffn_packed(cfg, x_perm, offsets, packed, y_perm, x, y_shared, ws,
                          stream=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_expert_ffn_packed",
        _lib.moe_expert_ffn_packed(_cfg(cfg), _ptr(x_perm), _ptr(offsets), _ptr(packed),
                                   _ptr(y_perm), _ptr(x), _ptr(y_shared), wp, wn,
                                   _stream(stream)))


def moe_forward_packed(cfg, x, router_w, logit_offset, bias, packed, out, topk_idx=None,
                       topk_w=None, counts=None, offsets=None, send=None, send_tok=None, ws=None,
                       stream=None, token_ids=None) -> None:
    wp, wn = _ws(ws)
    _ok("moe_forward_packed",
        _lib.moe_forward_packed(_cfg(cfg), _ptr(x), _ptr(router_w), _ptr(logit_offset),
                                _ptr(bias), _ptr(token_ids), _ptr(packed), _ptr(out),
                                _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                                _ptr(send), _ptr(send_tok), wp, wn, _stream(stream)))


def moe_selftest_bounded_wait(timeout_ns, ws, stream=None) -> None:
    _ok("moe_selftest_bounded_wait",
        _lib.moe_selftest_bounded_wait(int(timeout_ns), _ptr(ws), _stream(stream)))


def moe_dispatch_noalloc(cfg, x, topk_idx, counts, offsets, send, send_tok, perm_token, inv_perm,
                         x_perm, device_status=None, stream=None) -> None:
    """moe_dispatch with its scratch in the library's static device array (no workspace)."""
    _ok("moe_dispatch_noalloc",
        _lib.moe_dispatch_noalloc(_cfg(cfg), _ptr(x), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                  _ptr(send), _ptr(send_tok), _ptr(perm_token), _ptr(inv_perm),
                                  _ptr(x_perm), _ptr(device_status), _stream(stream)))


# ----------------------------------------------------------------- convenience
def forward_outputs(cfg, device="cuda"):
    """Allocates the outputs of moe_forward (out, topk_idx, topk_w, counts, offsets, send, send_tok)."""
    c = cfg if isinstance(cfg, MoeConfig) else MoeConfig.of(cfg)
    return {
        "out": torch.empty(c.T, c.d, dtype=torch.bfloat16, device=device),
        "topk_idx": torch.empty(c.T, c.K, dtype=torch.int32, device=device),
        "topk_w": torch.empty(c.T, c.K, dtype=torch.float32, device=device),
        "counts": torch.empty(c.E, dtype=torch.int32, device=device),
        "offsets": torch.empty(c.E + 1, dtype=torch.int32, device=device),
        "send": torch.empty(c.G, c.G, dtype=torch.int32, device=device),
        "send_tok": torch.empty(c.G, c.G, dtype=torch.int32, device=device),
    }
