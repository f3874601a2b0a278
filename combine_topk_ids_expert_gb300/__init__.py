"""GB300-native MoE expert-parallel token dispatch and combine.

A thin binding over libep_gb300.so (the C ABI of include/ep.h). Every step of
the dispatch/combine path runs in the library's CUDA kernels; this module only
marshals arguments. PyTorch supplies device memory (the workspace and the
caller's tensors) and streams.

Module-level functions carry the C names (``ep_dispatch``, ``ep_combine``,
...) and take a buffer handle and torch tensors. ``Buffer`` wraps them for
everyday use and returns torch views into the workspace::

    buf = Buffer(num_max_tokens_per_rank=8192, hidden=7168, num_experts=256,
                 num_ranks=8, topk=8, dtype=torch.bfloat16)
    d = buf.dispatch(x_TD, topk_scores_TK, topk_expert_ids_TK, num_tokens_per_rank=8192)
    y = experts(d.recv_x)                    # [R, S, D], rows past each rank's total undefined
    out_TD = buf.combine(y, topk_scores_TK)  # [T, D]
"""
from __future__ import annotations

import contextlib
import ctypes as C
from dataclasses import dataclass
from functools import cached_property

import torch

from . import _abi
from ._abi import (EP_ACT_GELU, EP_ACT_SILU, EP_BF16, EP_DEVERR_BAD_ID, EP_DEVERR_DEBUG_STRAY, EP_DEVERR_DEBUG_UNWRITTEN,
                   EP_DEVERR_ROW_OOB, EP_DEVERR_TIMEOUT, EP_F32, EP_FP4_MX, EP_FP4_NV,
                   EP_NOALLOC_SCRATCH_BYTES, EP_SCORE_SIGMOID, EP_SCORE_SOFTMAX,
                   EP_LAYOUT_PACKED, EP_LAYOUT_STRIDED, EP_PERMUTE_BULK, EP_PERMUTE_DEFAULT,
                   EP_PERMUTE_VEC, EpBufferInfo, EpConfig, EpDedupOut, EpDispatchOut, EpError,
                   EpFp4, EpLayout, EpW4, check)

__all__ = [
    "Buffer", "Layout", "DispatchResult", "EpConfig", "EpError",
    "ep_buffer_required_bytes", "ep_buffer_init", "ep_buffer_destroy", "ep_dispatch_layout",
    "ep_dispatch", "ep_dispatch_permute", "ep_combine", "ep_combine_backward",
    "ep_dispatch_backward", "ep_dispatch_dedup", "ep_dedup_expand", "ep_expert_gemm",
    "ep_expert_glu", "ep_expert_glu_backward", "ep_expert_gemm_backward",
    "ep_expert_gemv_w4", "ep_expert_glu_w4", "W4", "EpW4",
    "route", "route_backward", "quantize_fp4", "tile_fp4_scales", "untile_fp4_scales", "FP4",
    "ep_route", "ep_route_backward", "ep_fp4_scale_bytes", "ep_quantize_fp4", "ep_dequantize_fp4",
    "ep_dispatch_fp4", "ep_expert_gemm_fp4", "ep_expert_glu_fp4", "EpFp4",
    "ep_moe_layer", "ep_moe_layer_fp4", "ep_moe_layer_workspace_bytes", "EP_SCORE_SOFTMAX", "EP_SCORE_SIGMOID", "EP_FP4_MX", "EP_FP4_NV",
    "ep_get_device_error", "DedupResult",
    "ep_buffer_query", "ep_dispatch_layout_noalloc", "ep_dispatch_layout_noalloc_scratch_bytes",
    "EP_NOALLOC_SCRATCH_BYTES", "ep_pattern_probe", "ep_pad_tokens", "group_num_tokens_per_rank",
    "ep_derive_max_tokens_pretrain",
    "ep_derive_max_tokens_inference", "ep_validate_max_tokens", "ep_status_string",
    "EP_BF16", "EP_F32", "EP_PERMUTE_DEFAULT", "EP_PERMUTE_VEC", "EP_PERMUTE_BULK",
    "EP_LAYOUT_STRIDED", "EP_LAYOUT_PACKED", "EP_ACT_SILU", "EP_ACT_GELU",
    "EP_DEVERR_BAD_ID", "EP_DEVERR_ROW_OOB", "EP_DEVERR_TIMEOUT", "EP_DEVERR_DEBUG_UNWRITTEN",
    "EP_DEVERR_DEBUG_STRAY", "library_path",
]

_TORCH_TO_EP = {torch.bfloat16: EP_BF16, torch.float32: EP_F32}
_ACTS = {"silu": EP_ACT_SILU, "gelu": EP_ACT_GELU}
_SCORES = {"softmax": EP_SCORE_SOFTMAX, "sigmoid": EP_SCORE_SIGMOID}
_FP4_FORMATS = {"mx": EP_FP4_MX, "nv": EP_FP4_NV}
_FP4_BLOCK = {"mx": 32, "nv": 16}
_EP_TO_TORCH = {EP_BF16: torch.bfloat16, EP_F32: torch.float32}


def library_path() -> str:
    return _abi.LIB_PATH


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


_lib = _abi.lib

# The current stream's handle without a Stream object around it: 0.2 against 3 us, of
# calls that take about 10.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty_on(device: torch.device, shape: tuple, dtype: torch.dtype, stream,
              kept: bool = True) -> torch.Tensor:
    """Memory for what a call's kernels write on `stream`: from that stream's own pool, so
    that what used it before is done by then in stream order, and dropping it hands it on
    only behind those kernels. kept: the caller gets it, and may drop it while the current
    stream still works on it; that work is waited for too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    here = torch.cuda.current_stream(device)
    if stream == here:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if kept:
        t.record_stream(here)
    return t


_HERE = contextlib.nullcontext()


def _on_device_of(first: torch.Tensor, *others: torch.Tensor | None):
    """A context in which `first`'s device is the current one, checked to be the others' too."""
    dev = first.get_device()      # -1 on the host
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected all tensors on {first.device}, got one on {t.device}")
    return _HERE if dev == _current_device() else torch.cuda.device(first.device)


def _check_dtype(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# ---------------------------------------------------------------------------
# C-named functions (one call each)
# ---------------------------------------------------------------------------

def ep_buffer_required_bytes(cfg: EpConfig) -> int:
    return int(_abi.lib().ep_buffer_required_bytes(C.byref(cfg)))


def ep_buffer_init(cfg: EpConfig, workspace: torch.Tensor) -> C.c_void_p:
    h = C.c_void_p()
    check(_abi.lib().ep_buffer_init(C.byref(cfg), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), C.byref(h)),
          "ep_buffer_init")
    return h


def ep_buffer_destroy(handle) -> None:
    check(_abi.lib().ep_buffer_destroy(handle), "ep_buffer_destroy")


def ep_dispatch_layout(handle, topk_expert_ids_TK: torch.Tensor, num_tokens: int,
                       num_tokens_per_rank: int, stream=None,
                       host_tokens_per_expert: torch.Tensor | None = None) -> EpLayout:
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    host = None
    if host_tokens_per_expert is not None:
        _check_dtype(host_tokens_per_expert, torch.int32, "host_tokens_per_expert")
        if host_tokens_per_expert.is_cuda or not host_tokens_per_expert.is_contiguous():
            raise ValueError("host_tokens_per_expert must be a contiguous CPU tensor")
        host = host_tokens_per_expert.data_ptr()
    out = EpLayout()
    check(_abi.lib().ep_dispatch_layout(handle, _ptr(topk_expert_ids_TK), num_tokens,
                                        num_tokens_per_rank, _stream(stream), C.byref(out), host),
          "ep_dispatch_layout")
    return out


def ep_dispatch(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                topk_expert_ids_TK: torch.Tensor, num_tokens: int, num_tokens_per_rank: int,
                stream=None) -> EpDispatchOut:
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    out = EpDispatchOut()
    check(_abi.lib().ep_dispatch(handle, _ptr(x_TD), _ptr(topk_scores_TK),
                                 _ptr(topk_expert_ids_TK), num_tokens, num_tokens_per_rank,
                                 _stream(stream), C.byref(out)), "ep_dispatch")
    return out


def ep_dispatch_permute(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                        stream=None) -> EpDispatchOut:
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    out = EpDispatchOut()
    check(_abi.lib().ep_dispatch_permute(handle, _ptr(x_TD), _ptr(topk_scores_TK),
                                         _stream(stream), C.byref(out)), "ep_dispatch_permute")
    return out


def ep_combine(handle, y_recv: torch.Tensor, topk_scores_TK: torch.Tensor, num_tokens: int,
               out_TD: torch.Tensor, out_dtype: int, stream=None) -> None:
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    check(_abi.lib().ep_combine(handle, _ptr(y_recv), _ptr(topk_scores_TK), num_tokens,
                                _ptr(out_TD), out_dtype, _stream(stream)), "ep_combine")


def ep_combine_backward(handle, grad_out_TD: torch.Tensor, y_recv: torch.Tensor | None,
                        topk_scores_TK: torch.Tensor, num_tokens: int, grad_y_recv: torch.Tensor,
                        grad_scores_TK: torch.Tensor | None = None, stream=None) -> None:
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    if grad_scores_TK is not None:
        _check_dtype(grad_scores_TK, torch.float32, "grad_scores_TK")
    check(_abi.lib().ep_combine_backward(handle, _ptr(grad_out_TD), _ptr(y_recv),
                                         _ptr(topk_scores_TK), num_tokens, _ptr(grad_y_recv),
                                         _ptr(grad_scores_TK), _stream(stream)),
          "ep_combine_backward")


def ep_dispatch_backward(handle, grad_recv_x: torch.Tensor,
                         grad_recv_scores: torch.Tensor | None, num_tokens: int,
                         grad_x_TD: torch.Tensor, grad_x_dtype: int,
                         grad_scores_TK: torch.Tensor | None = None, stream=None) -> None:
    for name, t in (("grad_recv_scores", grad_recv_scores), ("grad_scores_TK", grad_scores_TK)):
        if t is not None:
            _check_dtype(t, torch.float32, name)
    check(_abi.lib().ep_dispatch_backward(handle, _ptr(grad_recv_x), _ptr(grad_recv_scores),
                                          num_tokens, _ptr(grad_x_TD), grad_x_dtype,
                                          _ptr(grad_scores_TK), _stream(stream)),
          "ep_dispatch_backward")


def ep_dispatch_dedup(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                      topk_expert_ids_TK: torch.Tensor, num_tokens: int, num_tokens_per_rank: int,
                      stream=None) -> EpDedupOut:
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    out = EpDedupOut()
    check(_abi.lib().ep_dispatch_dedup(handle, _ptr(x_TD), _ptr(topk_scores_TK),
                                       _ptr(topk_expert_ids_TK), num_tokens, num_tokens_per_rank,
                                       _stream(stream), C.byref(out)), "ep_dispatch_dedup")
    return out


def ep_dedup_expand(handle, topk_expert_ids_TK: torch.Tensor, y_recv: torch.Tensor,
                    stream=None) -> None:
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    check(_abi.lib().ep_dedup_expand(handle, _ptr(topk_expert_ids_TK), _ptr(y_recv),
                                     _stream(stream)), "ep_dedup_expand")


def ep_expert_gemm(handle, x_recv: torch.Tensor, weights: torch.Tensor, din: int, dout: int,
                   y_recv: torch.Tensor, stream=None) -> None:
    for name, t in (("x_recv", x_recv), ("weights", weights), ("y_recv", y_recv)):
        _check_dtype(t, torch.bfloat16, name)
    check(_abi.lib().ep_expert_gemm(handle, _ptr(x_recv), _ptr(weights), din, dout, _ptr(y_recv),
                                    _stream(stream)), "ep_expert_gemm")


def ep_expert_glu(handle, x_recv: torch.Tensor, w_gate_up: torch.Tensor, din: int, dff: int,
                  act: int, gate_up: torch.Tensor | None, h: torch.Tensor, stream=None) -> None:
    for name, t in (("x_recv", x_recv), ("w_gate_up", w_gate_up), ("gate_up", gate_up), ("h", h)):
        if t is not None:
            _check_dtype(t, torch.bfloat16, name)
    check(_abi.lib().ep_expert_glu(handle, _ptr(x_recv), _ptr(w_gate_up), din, dff, act,
                                   _ptr(gate_up), _ptr(h), _stream(stream)), "ep_expert_glu")


def ep_expert_glu_backward(handle, grad_y: torch.Tensor, w_down: torch.Tensor,
                           gate_up: torch.Tensor, dff: int, dout: int, act: int,
                           grad_gate_up: torch.Tensor, stream=None) -> None:
    for name, t in (("grad_y", grad_y), ("w_down", w_down), ("gate_up", gate_up),
                    ("grad_gate_up", grad_gate_up)):
        _check_dtype(t, torch.bfloat16, name)
    check(_abi.lib().ep_expert_glu_backward(handle, _ptr(grad_y), _ptr(w_down), _ptr(gate_up),
                                            dff, dout, act, _ptr(grad_gate_up), _stream(stream)),
          "ep_expert_glu_backward")


def ep_expert_gemm_backward(handle, grad_y: torch.Tensor, x_recv: torch.Tensor | None,
                            weights: torch.Tensor | None, din: int, dout: int,
                            grad_x: torch.Tensor | None = None,
                            grad_weights: torch.Tensor | None = None, accumulate: bool = False,
                            stream=None) -> None:
    """grad_weights may be bfloat16 or float32."""
    for name, t in (("grad_y", grad_y), ("x_recv", x_recv), ("weights", weights),
                    ("grad_x", grad_x)):
        if t is not None:
            _check_dtype(t, torch.bfloat16, name)
    w_dtype = EP_BF16
    if grad_weights is not None:
        if grad_weights.dtype not in _TORCH_TO_EP:
            raise TypeError(f"grad_weights must be bfloat16 or float32, got {grad_weights.dtype}")
        w_dtype = _TORCH_TO_EP[grad_weights.dtype]
    check(_abi.lib().ep_expert_gemm_backward(handle, _ptr(grad_y), _ptr(x_recv), _ptr(weights),
                                             din, dout, _ptr(grad_x), _ptr(grad_weights), w_dtype,
                                             int(accumulate), _stream(stream)),
          "ep_expert_gemm_backward")


@dataclass(frozen=True)
class W4:
    """The experts' 4-bit weights [E, rows, din] with group scales: w = (code - zero) * scale.
    A group is din / scales.shape[-1] consecutive elements: 32, 64 or 128."""
    codes: torch.Tensor               # [E, rows, din / 2] uint8, element 2j in byte j's low nibble
    scales: torch.Tensor              # [E, rows, din / group] bfloat16 or float32
    zeros: torch.Tensor | None = None   # [E, rows, din / group] uint8 (0..15); None: 8 everywhere

    def __post_init__(self):
        c, s, z = self.codes, self.scales, self.zeros
        _check_dtype(c, torch.uint8, "codes")
        if s.dtype not in _TORCH_TO_EP:
            raise TypeError(f"scales must be bfloat16 or float32, got {s.dtype}")
        if c.dim() != 3 or s.dim() != 3 or c.shape[:2] != s.shape[:2] or not s.shape[2] \
                or 2 * c.shape[2] % s.shape[2]:
            raise ValueError(f"codes [E, rows, din / 2] and scales [E, rows, din / group] do not "
                             f"fit: {tuple(c.shape)}, {tuple(s.shape)}")
        if z is not None:
            _check_dtype(z, torch.uint8, "zeros")
            if z.shape != s.shape:
                raise ValueError(f"zeros must be shaped as scales, got {tuple(z.shape)}")
        object.__setattr__(self, "_checked", self._form())

    def _form(self) -> tuple:
        c, s, z = self.codes, self.scales, self.zeros
        return c.shape, c.dtype, s.shape, s.dtype, None if z is None else (z.shape, z.dtype)

    @cached_property
    def din(self) -> int:
        return 2 * self.codes.shape[2]

    @cached_property
    def rows(self) -> int:
        return self.codes.shape[1]

    @cached_property
    def group(self) -> int:
        return self.din // self.scales.shape[2]

    def _struct(self) -> EpW4:
        """The C struct of one call. The fields cannot be set again, but a tensor's storage can
        be swapped under it (t.data = ..., set_, a module's move to another device and back):
        addresses, device and layout are taken anew each time."""
        if self._form() != self._checked:
            raise ValueError("the tensors of this W4 changed their shapes or types since it was "
                             "made: make another one of them")
        return EpW4(_ptr(self.codes), _ptr(self.scales), _ptr(self.zeros),
                    _TORCH_TO_EP[self.scales.dtype], self.group)


def ep_expert_gemv_w4(handle, x_recv: torch.Tensor, weights: W4, din: int, dout: int,
                      y_recv: torch.Tensor, stream=None) -> None:
    for name, t in (("x_recv", x_recv), ("y_recv", y_recv)):
        _check_dtype(t, torch.bfloat16, name)
    check(_abi.lib().ep_expert_gemv_w4(handle, _ptr(x_recv), C.byref(weights._struct()), din, dout,
                                       _ptr(y_recv), _stream(stream)), "ep_expert_gemv_w4")


def ep_expert_glu_w4(handle, x_recv: torch.Tensor, weights: W4, din: int, dff: int, act: int,
                     h: torch.Tensor, stream=None) -> None:
    for name, t in (("x_recv", x_recv), ("h", h)):
        _check_dtype(t, torch.bfloat16, name)
    check(_abi.lib().ep_expert_glu_w4(handle, _ptr(x_recv), C.byref(weights._struct()), din, dff,
                                      act, _ptr(h), _stream(stream)), "ep_expert_glu_w4")


# -- the router ------------------------------------------------------------------

def ep_route(logits_TE: torch.Tensor, select_TE: torch.Tensor | None, topk: int, score: int,
             normalize: bool, scale: float, topk_expert_ids_TK: torch.Tensor,
             topk_scores_TK: torch.Tensor, stream=None) -> None:
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    T, E = logits_TE.shape
    check(_abi.lib().ep_route(_ptr(logits_TE), _TORCH_TO_EP[logits_TE.dtype], _ptr(select_TE), T, E,
                              topk, score, int(normalize), scale, _ptr(topk_expert_ids_TK),
                              _ptr(topk_scores_TK), _stream(stream)), "ep_route")


def ep_route_backward(grad_scores_TK: torch.Tensor, logits_TE: torch.Tensor,
                      topk_expert_ids_TK: torch.Tensor, score: int, normalize: bool, scale: float,
                      grad_logits_TE: torch.Tensor, stream=None) -> None:
    T, E = logits_TE.shape
    check(_abi.lib().ep_route_backward(_ptr(grad_scores_TK), _ptr(logits_TE),
                                       _TORCH_TO_EP[logits_TE.dtype], _ptr(topk_expert_ids_TK), T, E,
                                       topk_expert_ids_TK.shape[1], score, int(normalize), scale,
                                       _ptr(grad_logits_TE), _stream(stream)), "ep_route_backward")


def _check_logits(logits: torch.Tensor, score: str) -> int:
    if logits.dtype not in _TORCH_TO_EP:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got {tuple(logits.shape)}")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _SCORES[score]


def route(logits_TE: torch.Tensor, topk: int, score: str = "softmax", normalize: bool = True,
          select: torch.Tensor | None = None, scale: float = 1.0, stream=None):
    """(topk_expert_ids_TK int32, topk_scores_TK fp32), as dispatch takes them: of each token the
    topk experts with the largest `select` (fp32 [T, E]; the logits unless given: biased, masked
    with -inf where a token may not go or does not exist), ties to the lowest index. Scores are
    scale times the softmax or the sigmoids of the logits, shared out over the chosen ones if
    normalize. A slot without an expert has id -1 and score 0."""
    kind = _check_logits(logits_TE, score)
    T, E = logits_TE.shape
    if not 1 <= topk <= E:
        raise ValueError(f"topk must be in 1..{E}, got {topk}")
    if select is not None:
        _check_dtype(select, torch.float32, "select")
        if select.shape != logits_TE.shape:
            raise ValueError(f"select must be shaped as logits, got {tuple(select.shape)}")
    with _on_device_of(logits_TE, select):
        ids = _empty_on(logits_TE.device, (T, topk), torch.int32, stream)
        scores = _empty_on(logits_TE.device, (T, topk), torch.float32, stream)
        ep_route(logits_TE, select, topk, kind, normalize, scale, ids, scores, stream)
    return ids, scores


def route_backward(grad_scores_TK: torch.Tensor, logits_TE: torch.Tensor,
                   topk_expert_ids_TK: torch.Tensor, score: str = "softmax",
                   normalize: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """The gradient of the logits (their type) from that of route's scores, fp32, which
    Buffer.combine_backward returns."""
    kind = _check_logits(logits_TE, score)
    ids = topk_expert_ids_TK
    _check_dtype(ids, torch.int32, "topk_expert_ids_TK")
    _check_dtype(grad_scores_TK, torch.float32, "grad_scores_TK")
    if ids.dim() != 2 or ids.shape[0] != logits_TE.shape[0] or grad_scores_TK.shape != ids.shape:
        raise ValueError(f"ids and grad_scores must be [{logits_TE.shape[0]}, topk], got "
                         f"{tuple(ids.shape)} and {tuple(grad_scores_TK.shape)}")
    with _on_device_of(logits_TE, ids, grad_scores_TK):
        grad = _empty_on(logits_TE.device, tuple(logits_TE.shape), logits_TE.dtype, stream)
        ep_route_backward(grad_scores_TK, logits_TE, ids, kind, normalize, scale, grad, stream)
    return grad


# -- microscaled 4-bit floating point ----------------------------------------------

def ep_fp4_scale_bytes(rows: int, cols: int, format: int) -> int:
    return int(_abi.lib().ep_fp4_scale_bytes(rows, cols, format))


def _fp4_tiles(rows: int, cols: int, format: str) -> tuple:
    """Shape of the scales of [rows, cols]."""
    return (rows + 127) // 128, cols // (4 * _FP4_BLOCK[format]), 32, 4, 4


def tile_fp4_scales(scales: torch.Tensor) -> torch.Tensor:
    """Block scales (uint8) of one row after the other, [..., rows, cols / block], in the tiles
    that FP4 holds."""
    _check_dtype(scales, torch.uint8, "scales")
    blocks = scales.shape[-1]
    if scales.dim() < 2 or not blocks or blocks % 4:
        raise ValueError(f"scales must be [..., rows, blocks] with 4 blocks or a multiple, got "
                         f"{tuple(scales.shape)}")
    flat = scales.reshape(-1, blocks)
    flat = torch.nn.functional.pad(flat, (0, 0, 0, -flat.shape[0] % 128))
    return flat.view(-1, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def untile_fp4_scales(scales: torch.Tensor, rows: int) -> torch.Tensor:
    """The reverse: [rows, cols / block]."""
    g, kt = scales.shape[:2]
    return scales.permute(0, 3, 2, 1, 4).reshape(128 * g, 4 * kt)[:rows]


@dataclass(frozen=True)
class FP4:
    """A matrix [..., rows, cols] in microscaled 4-bit floating point: weights [E, rows, cols]
    with rows a multiple of 128, receive rows, or any other. quantize_fp4 makes one."""
    codes: torch.Tensor                # [..., rows, cols / 2] uint8, element 2j in byte j's low nibble
    scales: torch.Tensor               # [ceil(all rows / 128), cols / (4 block), 32, 4, 4] uint8
    format: str                        # "mx" (blocks of 32, ue8m0) or "nv" (16, ue4m3)
    tensor_scale: torch.Tensor | None = None   # nv: fp32, one number for each matrix

    def __post_init__(self):
        c, s, g = self.codes, self.scales, self.tensor_scale
        if self.format not in _FP4_FORMATS:
            raise ValueError(f"format must be one of {sorted(_FP4_FORMATS)}, got {self.format!r}")
        _check_dtype(c, torch.uint8, "codes")
        _check_dtype(s, torch.uint8, "scales")
        if c.dim() < 2 or not c.shape[-1] or c.shape[-1] % 64:
            raise ValueError(f"codes must be [..., rows, cols / 2] with cols a multiple of 128, "
                             f"got {tuple(c.shape)}")
        want = _fp4_tiles(self.rows, self.cols, self.format)
        if tuple(s.shape) != want:
            raise ValueError(f"scales must be {list(want)} (tile_fp4_scales), got {list(s.shape)}")
        if g is not None:
            _check_dtype(g, torch.float32, "tensor_scale")
            if self.format != "nv":
                raise ValueError("only nv has a tensor_scale")
            if g.numel() != self.matrices:
                raise ValueError(f"tensor_scale must hold {self.matrices} numbers, got "
                                 f"{tuple(g.shape)}")
        object.__setattr__(self, "_checked", self._form())

    @classmethod
    def _of(cls, codes: torch.Tensor, scales: torch.Tensor, format: str, rows: int, cols: int) -> FP4:
        """Of tensors that the package has just made: nothing to check."""
        q = object.__new__(cls)
        q.__dict__.update(codes=codes, scales=scales, format=format, tensor_scale=None, rows=rows,
                          cols=cols)
        q.__dict__["_checked"] = q._form()
        return q

    def _form(self) -> tuple:
        c, s, g = self.codes, self.scales, self.tensor_scale
        return c.shape, c.dtype, s.shape, s.dtype, None if g is None else (g.shape, g.dtype)

    @cached_property
    def cols(self) -> int:
        return 2 * self.codes.shape[-1]

    @cached_property
    def rows(self) -> int:
        """All rows, of every matrix."""
        return self.codes.numel() // self.codes.shape[-1]

    @cached_property
    def matrices(self) -> int:
        n = 1
        for d in self.codes.shape[:-2]:
            n *= d
        return n

    def _struct(self) -> EpFp4:
        """The C struct of one call, addresses taken anew each time (as W4's)."""
        if self._form() != self._checked:
            raise ValueError("the tensors of this FP4 changed their shapes or types since it was "
                             "made: make another one of them")
        g = self.tensor_scale
        dev = self.codes.get_device()
        if self.scales.get_device() != dev or (g is not None and g.get_device() != dev):
            raise ValueError("the tensors of this FP4 are on several devices")
        return EpFp4(_ptr(self.codes), _ptr(self.scales), _ptr(g), _FP4_FORMATS[self.format])

    def dequantize(self, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """The values, [..., rows, cols] in bfloat16 (rounded) or float32."""
        if dtype not in _TORCH_TO_EP:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        with _on_device_of(self.codes):
            lead = self.codes.shape[:-1]
            out = _empty_on(self.codes.device, (*lead, self.cols), dtype, stream)
            check(_lib().ep_dequantize_fp4(C.byref(self._struct()), self.rows, self.cols,
                                           max(1, lead[-1]), _ptr(out), _TORCH_TO_EP[dtype],
                                           _stream(stream)), "ep_dequantize_fp4")
        return out


def ep_quantize_fp4(x: torch.Tensor, out: FP4, stream=None) -> None:
    _check_dtype(x, torch.bfloat16, "x")
    if x.shape != (*out.codes.shape[:-1], out.cols):
        raise ValueError(f"x must be {[*out.codes.shape[:-1], out.cols]}, got {list(x.shape)}")
    check(_abi.lib().ep_quantize_fp4(_ptr(x), out.rows, out.cols, max(1, out.codes.shape[-2]),
                                     C.byref(out._struct()), _stream(stream)), "ep_quantize_fp4")


def ep_dequantize_fp4(q: FP4, out: torch.Tensor, stream=None) -> None:
    if out.dtype not in _TORCH_TO_EP:
        raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
    if out.shape != (*q.codes.shape[:-1], q.cols):
        raise ValueError(f"out must be {[*q.codes.shape[:-1], q.cols]}, got {list(out.shape)}")
    check(_abi.lib().ep_dequantize_fp4(C.byref(q._struct()), q.rows, q.cols,
                                       max(1, q.codes.shape[-2]), _ptr(out),
                                       _TORCH_TO_EP[out.dtype], _stream(stream)),
          "ep_dequantize_fp4")


def quantize_fp4(x: torch.Tensor, format: str = "nv", tensor_scale: torch.Tensor | None = None,
                 stream=None) -> FP4:
    """x [..., rows, cols] (bf16, cols a multiple of 128) in microscaled 4-bit floating point.
    tensor_scale (nv only): fp32, one number for each matrix, by which the block scales are
    measured; amax / (6 * 448) of the matrix uses their whole range."""
    _check_dtype(x, torch.bfloat16, "x")
    if format not in _FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(_FP4_FORMATS)}, got {format!r}")
    if x.dim() < 2 or not x.shape[-1] or x.shape[-1] % 128:
        raise ValueError(f"x must be [..., rows, cols] with cols a multiple of 128, got "
                         f"{tuple(x.shape)}")
    with _on_device_of(x, tensor_scale):
        cols = x.shape[-1]
        lead = x.shape[:-1]
        rows = x.numel() // cols
        codes = _empty_on(x.device, (*lead, cols // 2), torch.uint8, stream)
        scales = _empty_on(x.device, _fp4_tiles(rows, cols, format), torch.uint8, stream)
        if tensor_scale is None:
            q = FP4._of(codes, scales, format, rows, cols)
        else:
            q = FP4(codes, scales, format, tensor_scale)
        check(_lib().ep_quantize_fp4(_ptr(x), rows, cols, max(1, lead[-1]), C.byref(q._struct()),
                                     _stream(stream)), "ep_quantize_fp4")
    return q


def ep_dispatch_fp4(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                    topk_expert_ids_TK: torch.Tensor, num_tokens: int, num_tokens_per_rank: int,
                    rows: FP4, stream=None) -> EpDispatchOut:
    _check_dtype(x_TD, torch.bfloat16, "x_TD")
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    out = EpDispatchOut()
    check(_abi.lib().ep_dispatch_fp4(handle, _ptr(x_TD), _ptr(topk_scores_TK),
                                     _ptr(topk_expert_ids_TK), num_tokens, num_tokens_per_rank,
                                     C.byref(rows._struct()), _stream(stream), C.byref(out)),
          "ep_dispatch_fp4")
    return out


def ep_expert_gemm_fp4(handle, x_recv: FP4, weights: FP4, din: int, dout: int,
                       y_recv: torch.Tensor, stream=None) -> None:
    _check_dtype(y_recv, torch.bfloat16, "y_recv")
    check(_abi.lib().ep_expert_gemm_fp4(handle, C.byref(x_recv._struct()),
                                        C.byref(weights._struct()), din, dout, _ptr(y_recv),
                                        _stream(stream)), "ep_expert_gemm_fp4")


def ep_expert_glu_fp4(handle, x_recv: FP4, w_gate_up: FP4, din: int, dff: int, act: int,
                      h: torch.Tensor | FP4, stream=None) -> None:
    """h: bfloat16 rows, or an FP4 that receives them quantised."""
    if not isinstance(h, FP4):
        _check_dtype(h, torch.bfloat16, "h")
    check(_abi.lib().ep_expert_glu_fp4(handle, C.byref(x_recv._struct()),
                                       C.byref(w_gate_up._struct()), din, dff, act,
                                       None if isinstance(h, FP4) else _ptr(h),
                                       C.byref(h._struct()) if isinstance(h, FP4) else None,
                                       _stream(stream)), "ep_expert_glu_fp4")


# -- a whole layer for a few tokens ---------------------------------------------------

def ep_moe_layer_workspace_bytes(handle, num_tokens: int, dff: int) -> int:
    return int(_abi.lib().ep_moe_layer_workspace_bytes(handle, num_tokens, dff))


def _moe_layer(call: str, handle, x_TD, topk_scores_TK, topk_expert_ids_TK, num_tokens, w_gate_up,
               w_down, dff, act, out_TD, workspace, stream) -> None:
    _check_dtype(x_TD, torch.bfloat16, "x_TD")
    _check_dtype(topk_scores_TK, torch.float32, "topk_scores_TK")
    _check_dtype(topk_expert_ids_TK, torch.int32, "topk_expert_ids_TK")
    if out_TD.dtype not in _TORCH_TO_EP:
        raise TypeError(f"out must be bfloat16 or float32, got {out_TD.dtype}")
    check(getattr(_abi.lib(), call)(
        handle, _ptr(x_TD), _ptr(topk_scores_TK), _ptr(topk_expert_ids_TK), num_tokens, w_gate_up,
        w_down, dff, act, _ptr(out_TD), _TORCH_TO_EP[out_TD.dtype], _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), call)


def ep_moe_layer(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                 topk_expert_ids_TK: torch.Tensor, num_tokens: int, w_gate_up: torch.Tensor,
                 w_down: torch.Tensor, dff: int, act: int, out_TD: torch.Tensor,
                 workspace: torch.Tensor, stream=None) -> None:
    for name, t in (("w_gate_up", w_gate_up), ("w_down", w_down)):
        _check_dtype(t, torch.bfloat16, name)
    _moe_layer("ep_moe_layer", handle, x_TD, topk_scores_TK, topk_expert_ids_TK, num_tokens,
               _ptr(w_gate_up), _ptr(w_down), dff, act, out_TD, workspace, stream)


def ep_moe_layer_fp4(handle, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                     topk_expert_ids_TK: torch.Tensor, num_tokens: int, w_gate_up: FP4,
                     w_down: FP4, dff: int, act: int, out_TD: torch.Tensor,
                     workspace: torch.Tensor, stream=None) -> None:
    _moe_layer("ep_moe_layer_fp4", handle, x_TD, topk_scores_TK, topk_expert_ids_TK, num_tokens,
               C.byref(w_gate_up._struct()), C.byref(w_down._struct()), dff, act, out_TD, workspace,
               stream)


def ep_get_device_error(handle, stream=None) -> int:
    v = C.c_uint32(0)
    check(_abi.lib().ep_get_device_error(handle, _stream(stream), C.byref(v)),
          "ep_get_device_error")
    return int(v.value)


def ep_buffer_query(handle) -> EpBufferInfo:
    info = EpBufferInfo()
    check(_abi.lib().ep_buffer_query(handle, C.byref(info)), "ep_buffer_query")
    return info


def ep_dispatch_layout_noalloc(topk_expert_ids_TK: torch.Tensor, num_tokens: int,
                               num_tokens_per_rank: int, topk: int, num_experts: int,
                               num_ranks: int, tokens_per_expert: torch.Tensor,
                               expert_offset: torch.Tensor, rows_per_rank: torch.Tensor,
                               rank_prefix: torch.Tensor, tokens_in_rank: torch.Tensor,
                               pos: torch.Tensor, error_flags: torch.Tensor | None = None,
                               stream=None) -> None:
    """The layout without a buffer, for callers that cannot allocate device
    memory: the caller supplies every output tensor (int32, on one CUDA device);
    the library uses its own fixed device scratch and allocates nothing. The
    tensors' sizes are checked here, since the C call only sees pointers: ids
    and pos hold num_tokens * topk entries, the per-expert outputs num_experts,
    the per-rank outputs num_ranks, error_flags (optional) one word."""
    T, K, E, R = int(num_tokens), int(topk), int(num_experts), int(num_ranks)
    if T < 0 or int(num_tokens_per_rank) < T:
        raise ValueError(f"need 0 <= num_tokens ({T}) <= num_tokens_per_rank "
                         f"({num_tokens_per_rank})")
    tensors = [("topk_expert_ids_TK", topk_expert_ids_TK, T * K),
               ("tokens_per_expert", tokens_per_expert, E), ("expert_offset", expert_offset, E),
               ("rows_per_rank", rows_per_rank, R), ("rank_prefix", rank_prefix, R),
               ("tokens_in_rank", tokens_in_rank, R), ("pos", pos, T * K)]
    if error_flags is not None:
        tensors.append(("error_flags", error_flags, 1))
    device = topk_expert_ids_TK.device
    if not topk_expert_ids_TK.is_cuda:
        raise ValueError("topk_expert_ids_TK must be a CUDA tensor")
    for name, t, n in tensors:
        if name != "error_flags":
            _check_dtype(t, torch.int32, name)
        elif t.dtype not in (torch.int32, torch.uint32) or not t.is_cuda or not t.is_contiguous():
            raise TypeError("error_flags must be a contiguous 4-byte integer CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, topk_expert_ids_TK on {device}")
        if t.numel() < n:
            raise ValueError(f"{name} has {t.numel()} elements, the call needs {n}")
    with torch.cuda.device(device):     # the device whose scratch the call uses
        check(_abi.lib().ep_dispatch_layout_noalloc(
            _ptr(topk_expert_ids_TK), T, num_tokens_per_rank, K, E, R, _ptr(tokens_per_expert),
            _ptr(expert_offset), _ptr(rows_per_rank), _ptr(rank_prefix), _ptr(tokens_in_rank),
            _ptr(pos), _ptr(error_flags), _stream(stream)), "ep_dispatch_layout_noalloc")


def ep_dispatch_layout_noalloc_scratch_bytes(num_tokens: int, topk: int, num_experts: int,
                                             num_ranks: int) -> int:
    """Bytes of the fixed device scratch that ep_dispatch_layout_noalloc needs for
    these sizes (host arithmetic only); accepted when <= EP_NOALLOC_SCRATCH_BYTES."""
    return int(_abi.lib().ep_dispatch_layout_noalloc_scratch_bytes(num_tokens, topk,
                                                                   num_experts, num_ranks))


def ep_pattern_probe(pattern: int, src: torch.Tensor | None, dst: torch.Tensor, rows: int,
                     row_bytes: int, fan: int = 1, stream=None) -> None:
    """Measurement aid: one of the hot path's HBM access patterns (EP_PATTERN_*)
    on `rows` rows of row_bytes, alone in a kernel. Sizes are checked here:
    FANOUT writes fan*rows rows, GATHER reads fan*rows rows, READ writes one
    16-byte word per row."""
    n_src = rows * row_bytes * (fan if pattern == _abi.EP_PATTERN_GATHER else 1)
    n_dst = (rows * 16 if pattern == _abi.EP_PATTERN_READ
             else rows * row_bytes * (fan if pattern == _abi.EP_PATTERN_FANOUT else 1))
    if pattern != _abi.EP_PATTERN_WRITE and (src is None or src.numel() * src.element_size() < n_src):
        raise ValueError(f"src must hold {n_src} bytes")
    if dst.numel() * dst.element_size() < n_dst:
        raise ValueError(f"dst must hold {n_dst} bytes")
    check(_abi.lib().ep_pattern_probe(pattern, _ptr(src), _ptr(dst), rows, row_bytes, fan,
                                      _stream(stream)), "ep_pattern_probe")


def ep_pad_tokens(n: int) -> int:
    return int(_abi.lib().ep_pad_tokens(n))


def group_num_tokens_per_rank(num_local_tokens: int, group=None) -> int:
    """num_tokens_per_rank for one expert-parallel group: the largest token count
    of its ranks ("fix(moe): equalize and align per-rank token counts for HybridEP
    dispatch", section "Fix": every rank pads to the EP-group max; dispatch then
    rounds it up to a multiple of 4, as ep_pad_tokens shows). One all-reduce (MAX)
    over the torch.distributed `group`, on a CUDA tensor under NCCL and a host
    tensor otherwise; without an initialised process group, the local count.
    Host logic on host integers: nothing here reads device memory."""
    import torch.distributed as dist
    n = int(num_local_tokens)
    if n < 0:
        raise ValueError(f"num_local_tokens must be >= 0, got {n}")
    if not (dist.is_available() and dist.is_initialized()):
        return n
    nccl = dist.get_backend(group) == "nccl"
    dev = torch.device("cuda", torch.cuda.current_device()) if nccl else torch.device("cpu")
    t = torch.tensor([n], dtype=torch.int64, device=dev)
    dist.all_reduce(t, op=dist.ReduceOp.MAX, group=group)
    return int(t.item())


def ep_derive_max_tokens_pretrain(local_batch_size: int, seq_len: int, cp: int, tp: int) -> int:
    return int(_abi.lib().ep_derive_max_tokens_pretrain(local_batch_size, seq_len, cp, tp))


def ep_derive_max_tokens_inference(max_num_batched_tokens: int, cp: int, tp: int) -> int:
    return int(_abi.lib().ep_derive_max_tokens_inference(max_num_batched_tokens, cp, tp))


def ep_validate_max_tokens(configured: int, derived: int) -> int:
    return int(_abi.lib().ep_validate_max_tokens(configured, derived))


def ep_status_string(status: int) -> str:
    return _abi.lib().ep_status_string(status).decode()


# ---------------------------------------------------------------------------
# Buffer: workspace ownership plus torch views of the results
# ---------------------------------------------------------------------------

@dataclass
class Layout:
    tokens_per_expert: torch.Tensor   # [E] int32
    expert_offset: torch.Tensor       # [E] int32
    rows_per_rank: torch.Tensor       # [R] int32
    rank_prefix: torch.Tensor         # [R] int32, inclusive
    tokens_in_rank: torch.Tensor      # [R] int32
    pos: torch.Tensor                 # [T, K] int32
    num_tokens: int
    padded_tokens: int
    rank_stride: int
    packed: bool


@dataclass
class DispatchResult:
    recv_x: torch.Tensor              # [R, S, D] (strided) or [R*S, D] (packed)
    recv_scores: torch.Tensor         # [R, S] or [R*S] fp32
    recv_src: torch.Tensor            # [R, S] or [R*S] int32
    layout: Layout


class _OfWorkspace:
    """Fields that are views of a buffer's workspace, each made when it is first asked for: nine
    of them cost more than a small call's kernels take."""

    @classmethod
    def _with(cls, space: _Space, views: dict, **fields):
        """views: name: (address, type, shape)."""
        o = object.__new__(cls)
        o.__dict__.update(fields)
        o.__dict__["_space"] = space
        o.__dict__["_views"] = views
        return o

    def __getattr__(self, name: str):
        view = self.__dict__.get("_views", {}).get(name)
        if view is None:
            raise AttributeError(f"{type(self).__name__!r} object has no attribute {name!r}")
        t = self.__dict__[name] = self._space.view(*view)
        return t


class _Space:
    """A workspace, and what it is as elements of the types that were asked for."""

    def __init__(self, workspace: torch.Tensor):
        self.workspace, self.base, self.typed = workspace, workspace.data_ptr(), {}

    def view(self, ptr: int, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
        base = self.typed.get(dtype)
        if base is None:
            base = self.typed[dtype] = self.workspace.view(dtype)
        strides, n = [], 1
        for s in reversed(shape):
            strides.append(n)
            n *= s
        return base.as_strided(shape, strides[::-1],
                               base.storage_offset() + (ptr - self.base) // base.element_size())


class _WorkspaceLayout(_OfWorkspace, Layout):
    pass


class _WorkspaceResult(_OfWorkspace, DispatchResult):
    pass


@dataclass
class DedupResult:
    recv_x: torch.Tensor              # [R, P, D]: one row per distinct (token, rank)
    recv_tok_src: torch.Tensor        # [R, P] int32 source token
    recv_topk_idx: torch.Tensor       # [R, P, K] int32 local expert index or -1
    recv_topk_w: torch.Tensor         # [R, P, K] fp32 score or 0
    tok_pos: torch.Tensor             # [T, R] int32 row of (t, r) or -1
    layout: Layout                    # tokens_in_rank[r] = rank r's rows


class Buffer:
    """A dispatcher buffer: one workspace sized from num_max_tokens_per_rank,
    reused by every call (no allocation after construction).

    stream: where a call's kernels run, the current stream by default. On another one, the
    caller sees to it that inputs are complete in its order and stay until it is done with
    them; what the call returns is complete in its order and may be dropped at any time."""

    def __init__(self, num_max_tokens_per_rank: int, hidden: int, num_experts: int,
                 num_ranks: int, topk: int, dtype: torch.dtype = torch.bfloat16,
                 num_sms: int = 0, permute_impl: int = EP_PERMUTE_DEFAULT, device=None,
                 layout: str = "strided"):
        if dtype not in _TORCH_TO_EP:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        mode = {"strided": EP_LAYOUT_STRIDED, "packed": EP_LAYOUT_PACKED}[layout]
        self.cfg = EpConfig(num_max_tokens_per_rank, hidden, num_experts, num_ranks, topk,
                            _TORCH_TO_EP[dtype], num_sms, permute_impl, mode)
        self.packed = mode == EP_LAYOUT_PACKED
        nbytes = ep_buffer_required_bytes(self.cfg)
        if nbytes == 0:
            raise EpError(_abi.EP_ERR_INVALID_ARG, "ep_buffer_required_bytes")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.device = dev
        self.dtype = dtype
        self.E, self.R, self.K, self.D = num_experts, num_ranks, topk, hidden
        with torch.cuda.device(dev):
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            self.handle = ep_buffer_init(self.cfg, self.workspace)
        self._space = _Space(self.workspace)
        self._layer_bytes: dict = {}
        self._stride: int | None = None        # of the last call's receive layout

    # -- views -------------------------------------------------------------
    def _view(self, ptr: int, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
        return self._space.view(ptr, dtype, shape)

    def _layout(self, L: EpLayout) -> Layout:
        T, E, R, K = L.num_tokens, self.E, self.R, self.K
        self._stride = L.rank_stride
        i32 = torch.int32
        return _WorkspaceLayout._with(
            self._space,
            {"tokens_per_expert": (L.tokens_per_expert, i32, (E,)),
             "expert_offset": (L.expert_offset, i32, (E,)),
             "rows_per_rank": (L.rows_per_rank, i32, (R,)),
             "rank_prefix": (L.rank_prefix, i32, (R,)),
             "tokens_in_rank": (L.tokens_in_rank, i32, (R,)),
             "pos": (L.pos, i32, (T, K))},
            num_tokens=T, padded_tokens=L.padded_tokens, rank_stride=L.rank_stride,
            packed=bool(L.packed))

    def _dispatch_result(self, d: EpDispatchOut, recv_x: FP4 | None = None) -> DispatchResult:
        S = d.layout.rank_stride
        self._stride = S
        lead = (self.R * S,) if self.packed else (self.R, S)
        views = {"recv_scores": (d.recv_scores, torch.float32, lead),
                 "recv_src": (d.recv_src, torch.int32, lead)}
        layout = self._layout(d.layout)
        if recv_x is None:
            views["recv_x"] = d.recv_x, self.dtype, lead + (self.D,)
            return _WorkspaceResult._with(self._space, views, layout=layout)
        return _WorkspaceResult._with(self._space, views, recv_x=recv_x, layout=layout)

    # -- memory of results -----------------------------------------------------
    def _empty(self, shape: tuple, dtype: torch.dtype, stream, kept: bool = True) -> torch.Tensor:
        """Memory on the buffer's device for what a call's kernels write on `stream` (_empty_on)."""
        return _empty_on(self.device, shape, dtype, stream, kept)

    def _new_rows(self, width: int, stream, dtype: torch.dtype = torch.bfloat16,
                  kept: bool = True) -> torch.Tensor:
        """Memory for rows of the last call's receive layout."""
        S = self._last_stride()
        lead = (self.R * S,) if self.packed else (self.R, S)
        return self._empty(lead + (width,), dtype, stream, kept)

    # -- calls -------------------------------------------------------------
    def dispatch_layout(self, topk_expert_ids_TK: torch.Tensor, num_tokens_per_rank: int,
                        stream=None, host_counts: bool = False):
        """Layout only. With host_counts=True also returns the per-expert
        counts as a CPU tensor (synchronises; refused while capturing)."""
        host = torch.empty(self.E, dtype=torch.int32) if host_counts else None
        L = ep_dispatch_layout(self.handle, topk_expert_ids_TK, topk_expert_ids_TK.shape[0],
                               num_tokens_per_rank, stream, host)
        lay = self._layout(L)
        return (lay, host) if host_counts else lay

    def dispatch(self, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                 topk_expert_ids_TK: torch.Tensor, num_tokens_per_rank: int | None = None,
                 stream=None) -> DispatchResult:
        _check_dtype(x_TD, self.dtype, "x_TD")
        T = x_TD.shape[0]
        N = T if num_tokens_per_rank is None else num_tokens_per_rank
        d = ep_dispatch(self.handle, x_TD, topk_scores_TK, topk_expert_ids_TK, T, N, stream)
        return self._dispatch_result(d)

    def dispatch_permute(self, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                         stream=None) -> DispatchResult:
        _check_dtype(x_TD, self.dtype, "x_TD")
        return self._dispatch_result(ep_dispatch_permute(self.handle, x_TD, topk_scores_TK,
                                                         stream))

    def combine(self, y_recv: torch.Tensor, topk_scores_TK: torch.Tensor,
                out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                stream=None) -> torch.Tensor:
        _check_dtype(y_recv, self.dtype, "y_recv")
        T = topk_scores_TK.shape[0]
        if out is None:
            od = self.dtype if out_dtype is None else out_dtype
            out = self._empty((T, self.D), od, stream)
        if out.dtype not in _TORCH_TO_EP:
            raise TypeError(f"out dtype must be bfloat16 or float32, got {out.dtype}")
        ep_combine(self.handle, y_recv, topk_scores_TK, T, out, _TORCH_TO_EP[out.dtype], stream)
        return out

    def combine_backward(self, grad_out: torch.Tensor, y_recv: torch.Tensor | None,
                         topk_scores_TK: torch.Tensor, grad_y: torch.Tensor | None = None,
                         want_scores: bool = True, stream=None):
        """(grad_y [R, S, D], grad_scores [T, K] or None) for the last dispatch.
        grad_y rows that no pair references are left as they were."""
        _check_dtype(grad_out, self.dtype, "grad_out")
        T = topk_scores_TK.shape[0]
        if grad_y is None:
            grad_y = self._new_rows(self.D, stream, self.dtype)
        gs = self._empty((T, self.K), torch.float32, stream) if want_scores else None
        ep_combine_backward(self.handle, grad_out, y_recv, topk_scores_TK, T, grad_y, gs, stream)
        return grad_y, gs

    def dispatch_backward(self, grad_recv_x: torch.Tensor, num_tokens: int,
                          grad_recv_scores: torch.Tensor | None = None,
                          out_dtype: torch.dtype | None = None, stream=None):
        """(grad_x [T, D], grad_scores [T, K] or None) for the last dispatch."""
        _check_dtype(grad_recv_x, self.dtype, "grad_recv_x")
        od = self.dtype if out_dtype is None else out_dtype
        gx = self._empty((num_tokens, self.D), od, stream)
        gs = None
        if grad_recv_scores is not None:
            gs = self._empty((num_tokens, self.K), torch.float32, stream)
        ep_dispatch_backward(self.handle, grad_recv_x, grad_recv_scores, num_tokens, gx,
                             _TORCH_TO_EP[od], gs, stream)
        return gx, gs

    def dispatch_dedup(self, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                       topk_expert_ids_TK: torch.Tensor, num_tokens_per_rank: int | None = None,
                       stream=None) -> DedupResult:
        """One receive row per distinct (token, rank)."""
        _check_dtype(x_TD, self.dtype, "x_TD")
        T = x_TD.shape[0]
        N = T if num_tokens_per_rank is None else num_tokens_per_rank
        d = ep_dispatch_dedup(self.handle, x_TD, topk_scores_TK, topk_expert_ids_TK, T, N, stream)
        P, R, K = d.rows_per_rank_stride, self.R, self.K
        lay = self._layout(d.layout)
        return DedupResult(
            recv_x=self._view(d.recv_x, self.dtype, (R, P, self.D)),
            recv_tok_src=self._view(d.recv_tok_src, torch.int32, (R, P)),
            recv_topk_idx=self._view(d.recv_topk_idx, torch.int32, (R, P, K)),
            recv_topk_w=self._view(d.recv_topk_w, torch.float32, (R, P, K)),
            tok_pos=self._view(d.tok_pos, torch.int32, (T, R)),
            layout=lay)

    def dedup_expand(self, topk_expert_ids_TK: torch.Tensor, y_recv: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
        """The receiver's expansion of the last dedupe dispatch into per-expert rows
        (a tensor shaped like a dispatch's recv_x), ready for combine."""
        if y_recv is None:
            y_recv = self._new_rows(self.D, stream, self.dtype)
        ep_dedup_expand(self.handle, topk_expert_ids_TK, y_recv, stream)
        return y_recv

    def expert_gemm(self, x_recv: torch.Tensor, weights: torch.Tensor,
                    y_recv: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y = x * W_e^T over each expert's receive rows (weights [E, dout, din]),
        from the counts of the last dispatch on this buffer. Returns y_recv with
        the receive layout's leading shape and dout columns."""
        E, dout, din = weights.shape
        if E != self.E:
            raise ValueError(f"weights must have {self.E} experts, got {E}")
        if x_recv.shape[-1] != din:
            raise ValueError(f"x_recv has {x_recv.shape[-1]} columns, weights expect {din}")
        if y_recv is None:
            y_recv = self._new_rows(dout, stream)
        ep_expert_gemm(self.handle, x_recv, weights, din, dout, y_recv, stream)
        return y_recv

    # -- the experts' gated feed-forward block ---------------------------------
    def _rows(self, t: torch.Tensor, name: str, width: int) -> torch.Tensor:
        """t, checked to be rows of the last call's receive layout, `width` columns wide."""
        n = self.R * self._last_stride()
        if t.dim() < 2 or t.shape[-1] != width or t.numel() != n * width:
            raise ValueError(f"{name} must hold the receive layout's {n} rows of {width} "
                             f"columns, got {tuple(t.shape)}")
        return t

    def _out_rows(self, t: torch.Tensor | None, name: str, width: int, stream) -> torch.Tensor:
        return self._new_rows(width, stream) if t is None else self._rows(t, name, width)

    def _weights(self, w: torch.Tensor, name: str, rows: int | None,
                 cols: int | None) -> tuple[int, int]:
        """(rows, columns) of w, checked to be [E, rows, cols] (None: any number)."""
        shape = tuple(w.shape)
        if len(shape) != 3 or shape[0] != self.E or (rows is not None and rows != shape[1]) \
                or (cols is not None and cols != shape[2]):
            want = [self.E, *("any" if n is None else n for n in (rows, cols))]
            raise ValueError(f"{name} must be {want}, got {list(shape)}")
        return shape[1], shape[2]

    @staticmethod
    def _activation(act: str) -> int:
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
        return _ACTS[act]

    def expert_glu(self, x_recv: torch.Tensor, w_gate_up: torch.Tensor, act: str = "silu",
                   gate_up: torch.Tensor | None = None, h: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
        """h = act(x Wg^T) * (x Wu^T) over each expert's receive rows, one kernel.
        w_gate_up is [E, 2 dff, din], gate rows first. gate_up, if given, receives the
        pre-activations for the backward pass. Returns h in the receive layout."""
        dff2, din = self._weights(w_gate_up, "w_gate_up", None, None)
        if dff2 % 2:
            raise ValueError(f"w_gate_up must hold gate and up rows, got {dff2} rows")
        dff = dff2 // 2
        self._rows(x_recv, "x_recv", din)
        if gate_up is not None:
            self._rows(gate_up, "gate_up", dff2)
        h = self._out_rows(h, "h", dff, stream)
        ep_expert_glu(self.handle, x_recv, w_gate_up, din, dff, self._activation(act), gate_up, h,
                      stream)
        return h

    def expert_ffn(self, x_recv: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                   act: str = "silu", save: bool = False, stream=None):
        """The experts' gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T, with
        w_gate_up [E, 2 dff, din] (gate rows first) and w_down [E, dout, dff]: two kernels,
        ready for combine. save=True returns (y, h, gate_up), what expert_ffn_backward needs."""
        dff2, _ = self._weights(w_gate_up, "w_gate_up", None, None)
        self._weights(w_down, "w_down", None, dff2 // 2)
        gate_up = self._new_rows(dff2, stream) if save else None
        h = self._new_rows(dff2 // 2, stream, kept=save)
        self.expert_glu(x_recv, w_gate_up, act, gate_up, h, stream)
        y = self.expert_gemm(h, w_down, stream=stream)
        return (y, h, gate_up) if save else y

    def expert_gemm_backward(self, grad_y: torch.Tensor, x_recv: torch.Tensor | None,
                             weights: torch.Tensor | None, want_x: bool = True,
                             want_weights: bool = True, grad_x: torch.Tensor | None = None,
                             grad_weights: torch.Tensor | None = None, accumulate: bool = False,
                             stream=None):
        """(grad_x, grad_weights) of expert_gemm, None for one that is not wanted.
        grad_weights may be a bfloat16 or float32 tensor [E, dout, din]; accumulate=True
        adds to it (gradient accumulation over micro-batches)."""
        if not want_x and not want_weights:
            raise ValueError("neither gradient is wanted: want_x or want_weights")
        if want_x and weights is None:
            raise ValueError("grad_x needs weights (or want_x=False)")
        if want_weights and x_recv is None:
            raise ValueError("grad_weights needs x_recv (or want_weights=False)")
        dout = grad_y.shape[-1]
        if want_x:
            _, din = self._weights(weights, "weights", dout, None)
        else:
            din = x_recv.shape[-1]
        self._rows(grad_y, "grad_y", dout)
        if want_weights:
            self._rows(x_recv, "x_recv", din)
            if grad_weights is None:
                if accumulate:
                    raise ValueError("accumulate=True needs grad_weights")
                grad_weights = self._empty((self.E, dout, din), torch.bfloat16, stream)
            self._weights(grad_weights, "grad_weights", dout, din)
        grad_x = self._out_rows(grad_x, "grad_x", din, stream) if want_x else None
        grad_weights = grad_weights if want_weights else None
        ep_expert_gemm_backward(self.handle, grad_y, x_recv if want_weights else None,
                                weights if want_x else None, din, dout, grad_x, grad_weights,
                                accumulate, stream)
        return grad_x, grad_weights

    def expert_glu_backward(self, grad_y: torch.Tensor, w_down: torch.Tensor,
                            gate_up: torch.Tensor, act: str = "silu",
                            grad_gate_up: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
        """The gradient of the pre-activations [.., 2 dff] from the gradient of y, through
        w_down [E, dout, dff] and the activation, one kernel."""
        dout, dff = self._weights(w_down, "w_down", None, None)
        self._rows(grad_y, "grad_y", dout)
        self._rows(gate_up, "gate_up", 2 * dff)
        grad_gate_up = self._out_rows(grad_gate_up, "grad_gate_up", 2 * dff, stream)
        ep_expert_glu_backward(self.handle, grad_y, w_down, gate_up, dff, dout,
                               self._activation(act), grad_gate_up, stream)
        return grad_gate_up

    def expert_ffn_backward(self, grad_y: torch.Tensor, x_recv: torch.Tensor,
                            w_gate_up: torch.Tensor, w_down: torch.Tensor,
                            gate_up: torch.Tensor, h: torch.Tensor, act: str = "silu",
                            grad_w_gate_up: torch.Tensor | None = None,
                            grad_w_down: torch.Tensor | None = None, accumulate: bool = False,
                            stream=None):
        """(grad_x, grad_w_gate_up, grad_w_down) of expert_ffn, from the gate_up and h that
        expert_ffn(..., save=True) returned. The weight gradients may be given as bfloat16
        or float32 tensors, with accumulate=True to add to them."""
        grad_gate_up = self._new_rows(gate_up.shape[-1], stream, kept=False)
        self.expert_glu_backward(grad_y, w_down, gate_up, act, grad_gate_up, stream)
        _, grad_w_down = self.expert_gemm_backward(grad_y, h, w_down, want_x=False,
                                                   grad_weights=grad_w_down,
                                                   accumulate=accumulate, stream=stream)
        grad_x, grad_w_gate_up = self.expert_gemm_backward(grad_gate_up, x_recv, w_gate_up,
                                                           grad_weights=grad_w_gate_up,
                                                           accumulate=accumulate, stream=stream)
        return grad_x, grad_w_gate_up, grad_w_down

    # -- the same block on 4-bit weights ----------------------------------------
    def expert_gemv_w4(self, x_recv: torch.Tensor, weights: W4,
                       y_recv: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y = x W_e^T over each expert's receive rows with 4-bit weights, for the few rows
        per expert of a decode batch."""
        self._weights(weights.codes, "weights.codes", None, None)
        self._rows(x_recv, "x_recv", weights.din)
        y_recv = self._out_rows(y_recv, "y_recv", weights.rows, stream)
        ep_expert_gemv_w4(self.handle, x_recv, weights, weights.din, weights.rows, y_recv, stream)
        return y_recv

    def expert_glu_w4(self, x_recv: torch.Tensor, w_gate_up: W4, act: str = "silu",
                      h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """expert_glu with 4-bit weights of 2 dff rows per expert, gate rows first."""
        self._weights(w_gate_up.codes, "w_gate_up.codes", None, None)
        if w_gate_up.rows % 2:
            raise ValueError(f"w_gate_up must hold gate and up rows, got {w_gate_up.rows} rows")
        dff = w_gate_up.rows // 2
        self._rows(x_recv, "x_recv", w_gate_up.din)
        h = self._out_rows(h, "h", dff, stream)
        ep_expert_glu_w4(self.handle, x_recv, w_gate_up, w_gate_up.din, dff,
                         self._activation(act), h, stream)
        return h

    def expert_ffn_w4(self, x_recv: torch.Tensor, w_gate_up: W4, w_down: W4, act: str = "silu",
                      y_recv: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """expert_ffn with 4-bit weights: two kernels, ready for combine."""
        if w_down.din * 2 != w_gate_up.rows:
            raise ValueError(f"w_down takes {w_down.din} columns, w_gate_up gives "
                             f"{w_gate_up.rows // 2}")
        h = self.expert_glu_w4(x_recv, w_gate_up, act,
                               self._new_rows(w_down.din, stream, kept=False), stream)
        return self.expert_gemv_w4(h, w_down, y_recv, stream)

    def _here(self, *tensors: torch.Tensor | None):
        """A context in which the buffer's device is the current one, with `tensors` on it."""
        return _on_device_of(self.workspace, *tensors)

    # -- the same block in 4-bit floating point ----------------------------------
    def dispatch_fp4(self, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                     topk_expert_ids_TK: torch.Tensor, num_tokens_per_rank: int | None = None,
                     format: str = "nv", tensor_scale: torch.Tensor | None = None,
                     stream=None) -> DispatchResult:
        """dispatch whose receive rows are quantised on the way: recv_x is an FP4 of
        [R * S, D] rows (rows past each rank's total undefined), in memory of its own."""
        T = x_TD.shape[0]
        if x_TD.shape != (T, self.D) or topk_expert_ids_TK.shape != (T, self.K) or \
                topk_scores_TK.shape != (T, self.K):
            raise ValueError(f"x, scores and ids must be [T, {self.D}], [T, {self.K}] and "
                             f"[T, {self.K}], got {tuple(x_TD.shape)}, "
                             f"{tuple(topk_scores_TK.shape)}, {tuple(topk_expert_ids_TK.shape)}")
        if format not in _FP4_FORMATS:
            raise ValueError(f"format must be one of {sorted(_FP4_FORMATS)}, got {format!r}")
        if self.D % 128:
            raise ValueError(f"4-bit rows need a hidden size that is a multiple of 128, got {self.D}")
        N = T if num_tokens_per_rank is None else num_tokens_per_rank
        if not T <= N <= self.cfg.num_max_tokens_per_rank:
            raise EpError(_abi.EP_ERR_CAPACITY if N >= T else _abi.EP_ERR_INVALID_ARG,
                          "ep_dispatch_fp4")
        with self._here(x_TD, topk_scores_TK, topk_expert_ids_TK, tensor_scale):
            q = self._fp4_rows(self.R * ep_pad_tokens(N) * self.K, self.D, format, tensor_scale,
                               stream)
            d = ep_dispatch_fp4(self.handle, x_TD, topk_scores_TK, topk_expert_ids_TK, T, N, q,
                                stream)
        return self._dispatch_result(d, q)

    def _fp4_rows(self, rows: int, cols: int, format: str, tensor_scale, stream,
                  kept: bool = True) -> FP4:
        if tensor_scale is None:
            return FP4._of(self._empty((rows, cols // 2), torch.uint8, stream, kept),
                           self._empty(_fp4_tiles(rows, cols, format), torch.uint8, stream, kept),
                           format, rows, cols)
        return FP4(self._empty((rows, cols // 2), torch.uint8, stream, kept),
                   self._empty(_fp4_tiles(rows, cols, format), torch.uint8, stream, kept), format,
                   tensor_scale)

    def _rows_fp4(self, x: FP4, name: str, width: int) -> FP4:
        """x, checked to be rows of the last call's receive layout, `width` columns wide."""
        n = self.R * self._last_stride()
        if x.cols != width or x.rows != n or (x.tensor_scale is not None
                                              and x.tensor_scale.numel() != 1):
            raise ValueError(f"{name} must hold the receive layout's {n} rows of {width} columns "
                             f"(with one tensor_scale), got {x.rows} of {x.cols}")
        return x

    def _weights_fp4(self, w: FP4, name: str, x_recv: FP4) -> int:
        """Rows of each expert's w, checked to be [E, rows, any] in the rows' format."""
        for n, q in ((name, w), ("x_recv", x_recv)):
            if not isinstance(q, FP4):
                raise TypeError(f"{n} must be an FP4, got {type(q).__name__}")
        n, _ = self._weights(w.codes, name + ".codes", None, None)
        if w.format != x_recv.format:
            raise ValueError(f"{name} is {w.format}, the rows are {x_recv.format}")
        if n % 128:
            raise ValueError(f"{name} must hold a multiple of 128 rows for each expert, got {n}")
        return n

    def expert_gemm_fp4(self, x_recv: FP4, weights: FP4, y_recv: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
        """y = x W_e^T over each expert's receive rows (dispatch_fp4's recv_x) with weights
        [E, dout, din], both in 4 bits; y in bf16."""
        dout = self._weights_fp4(weights, "weights", x_recv)
        self._rows_fp4(x_recv, "x_recv", weights.cols)
        with self._here(x_recv.codes, weights.codes, y_recv):
            y_recv = self._out_rows(y_recv, "y_recv", dout, stream)
            ep_expert_gemm_fp4(self.handle, x_recv, weights, weights.cols, dout, y_recv, stream)
        return y_recv

    def expert_glu_fp4(self, x_recv: FP4, w_gate_up: FP4, act: str = "silu",
                       h: torch.Tensor | FP4 | None = None, quantize: bool = False,
                       h_scale: torch.Tensor | None = None, stream=None):
        """h = act(x Wg^T) * (x Wu^T) over each expert's receive rows, both in 4 bits: in bf16,
        or, with quantize, as an FP4 of the same format (h_scale: its tensor_scale). A given h
        says by itself which."""
        if h is not None and (h_scale is not None or (quantize and not isinstance(h, FP4))):
            raise ValueError("a given h is a bfloat16 tensor, or an FP4 with its own tensor_scale: "
                             "quantize and h_scale are for one that is made")
        if h_scale is not None and not quantize:
            raise ValueError("h_scale needs quantize=True")
        rows = self._weights_fp4(w_gate_up, "w_gate_up", x_recv)
        if rows % 256:
            raise ValueError(f"w_gate_up must hold gate and up rows, 128 of each or a multiple, "
                             f"got {rows} rows")
        dff = rows // 2
        self._rows_fp4(x_recv, "x_recv", w_gate_up.cols)
        if h is None and quantize:
            h = self._fp4_rows(self.R * self._last_stride(), dff, x_recv.format, h_scale, stream)
        elif isinstance(h, FP4):
            self._rows_fp4(h, "h", dff)
            if h.format != x_recv.format:
                raise ValueError(f"h is {h.format}, the rows are {x_recv.format}")
        else:
            h = self._out_rows(h, "h", dff, stream)
        with self._here(x_recv.codes, w_gate_up.codes, h.codes if isinstance(h, FP4) else h):
            ep_expert_glu_fp4(self.handle, x_recv, w_gate_up, w_gate_up.cols, dff,
                              self._activation(act), h, stream)
        return h

    def expert_ffn_fp4(self, x_recv: FP4, w_gate_up: FP4, w_down: FP4, act: str = "silu",
                       h_scale: torch.Tensor | None = None, y_recv: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
        """expert_ffn with rows, weights and what is between them in 4 bits: two kernels, y in
        bf16, ready for combine."""
        dff = self._weights_fp4(w_gate_up, "w_gate_up", x_recv) // 2
        if w_down.cols != dff:
            raise ValueError(f"w_down takes {w_down.cols} columns, w_gate_up gives {dff}")
        h = self._fp4_rows(self.R * self._last_stride(), dff, x_recv.format, h_scale, stream,
                           kept=False)
        self.expert_glu_fp4(x_recv, w_gate_up, act, h, stream=stream)
        return self.expert_gemm_fp4(h, w_down, y_recv, stream)

    # -- the whole layer for a few tokens ------------------------------------------
    def moe_layer(self, x_TD: torch.Tensor, topk_scores_TK: torch.Tensor,
                  topk_expert_ids_TK: torch.Tensor, w_gate_up, w_down, act: str = "silu",
                  out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  stream=None) -> torch.Tensor:
        """dispatch, the experts' gated block and combine in two kernels, for at most 64 tokens
        and 512 (token, k) pairs: weights w_gate_up [E, 2 dff, D] and w_down [E, D, dff], bf16
        tensors or FP4 (activations within 2^-22 of their block's largest: include/ep.h). Leaves
        the last dispatch's layout and receive rows alone."""
        fp4 = isinstance(w_gate_up, FP4)
        if fp4 != isinstance(w_down, FP4):
            raise TypeError("w_gate_up and w_down must both be tensors or both FP4")
        if fp4:
            if w_gate_up.format != w_down.format:
                raise ValueError(f"w_gate_up is {w_gate_up.format}, w_down {w_down.format}")
            shapes = [(*w.codes.shape[:-1], w.cols) for w in (w_gate_up, w_down)]
        else:
            shapes = [tuple(w_gate_up.shape), tuple(w_down.shape)]
        dff = shapes[1][-1]
        if shapes != [(self.E, 2 * dff, self.D), (self.E, self.D, dff)]:
            raise ValueError(f"weights must be [{self.E}, 2 dff, {self.D}] and [{self.E}, {self.D}, "
                             f"dff], got {shapes}")
        T = x_TD.shape[0]
        if x_TD.shape != (T, self.D) or topk_expert_ids_TK.shape != (T, self.K) or \
                topk_scores_TK.shape != (T, self.K):
            raise ValueError(f"x, scores and ids must be [T, {self.D}], [T, {self.K}] and "
                             f"[T, {self.K}], got {tuple(x_TD.shape)}, "
                             f"{tuple(topk_scores_TK.shape)}, {tuple(topk_expert_ids_TK.shape)}")
        kind = self._activation(act)
        if out is not None and out.shape != (T, self.D):
            raise ValueError(f"out must be {[T, self.D]}, got {list(out.shape)}")
        nbytes = self._layer_bytes.get((T, dff))
        if nbytes is None:
            nbytes = self._layer_bytes[T, dff] = ep_moe_layer_workspace_bytes(self.handle, T, dff)
        if nbytes == 0:
            raise EpError(_abi.EP_ERR_CAPACITY if T > min(64, self.cfg.num_max_tokens_per_rank)
                          or T * self.K > 512 else _abi.EP_ERR_INVALID_ARG, "ep_moe_layer")
        with self._here(x_TD, topk_scores_TK, topk_expert_ids_TK, out,
                        *((w_gate_up.codes, w_down.codes) if fp4 else (w_gate_up, w_down))):
            if out is None:
                out = self._empty((T, self.D), torch.bfloat16 if out_dtype is None else out_dtype,
                                  stream)
            work = self._empty((nbytes,), torch.uint8, stream, kept=False)
            (ep_moe_layer_fp4 if fp4 else ep_moe_layer)(
                self.handle, x_TD, topk_scores_TK, topk_expert_ids_TK, T, w_gate_up, w_down, dff,
                kind, out, work, stream)
        return out

    def _last_stride(self) -> int:
        if self._stride is None:
            raise EpError(_abi.EP_ERR_NO_LAYOUT, "receive rows of a buffer without a dispatch")
        return self._stride

    def device_error(self, stream=None) -> int:
        return ep_get_device_error(self.handle, stream)

    def info(self) -> dict:
        i = ep_buffer_query(self.handle)
        return {f: getattr(i, f) for f, _ in EpBufferInfo._fields_}

    def close(self) -> None:
        if getattr(self, "handle", None) is not None:
            ep_buffer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
