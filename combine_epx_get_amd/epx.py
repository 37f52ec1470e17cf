"""Thin ctypes binding over libepx.so (the C ABI in include/epx.h).

Argument marshalling only: tensors are checked for dtype, shape, device and
contiguity, and their data pointers and the current HIP stream are passed to
the library. Every step of dispatch and combine runs in the library's HIP
kernels; there is no fallback of any kind. Importing this module fails when
the library has not been built (``python -m combine_epx_get_amd.build``).

PyTorch serves as the device allocator and stream provider only.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional

import torch

# The release library, or the one EPX_LIBRARY names (e.g. the bounds-checked
# libepx_checked.so built beside it).
_LIB_PATH = os.environ.get("EPX_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                          "libepx.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built; run `python -m combine_epx_get_amd.build`")
_lib = ctypes.CDLL(_LIB_PATH)

MODE_PER_EXPERT = 0
MODE_HOST_RELAY = 1
BF16 = 0
FP8_E4M3 = 1
F32 = 2
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
ACT_NONE = 0
ACT_SWIGLU = 1

STATUS = {0: "EPX_OK", 1: "EPX_ERR_ARG", 2: "EPX_ERR_INDEX", 3: "EPX_ERR_CAPACITY", 4: "EPX_ERR_DEVICE",
          5: "EPX_ERR_SCRATCH"}

LAYOUT_FIELDS = ["expert_count", "expert_offset", "rank_rows", "rank_tokens", "rank_offset",
                 "host_tokens", "host_offset", "slot", "row_token", "relay_slot", "relay_token",
                 "fanout_expert", "fanout_rank_mask", "relay_dst_rank", "totals", "group_offset",
                 "workspace"]
RELAY_FIELDS = ("relay_slot", "relay_token", "fanout_expert", "fanout_rank_mask")


class epx_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_tokens", "topk", "num_experts", "num_ranks", "num_hosts", "my_rank", "mode",
                 "num_groups")]


class epx_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYOUT_FIELDS]


class epx_expert_rows(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("row_offset", ctypes.c_void_p), ("row_count", ctypes.c_void_p)]


_P = ctypes.c_void_p
_lib.epx_layout_sizes.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(ctypes.c_int64)]
_lib.epx_get_layout.argtypes = [ctypes.POINTER(epx_problem), _P, ctypes.POINTER(epx_layout), _P]
_lib.epx_dispatch.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P,
                              ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int64, _P]
_lib.epx_combine.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P,
                             ctypes.c_int64, _P, ctypes.c_int32, _P, _P]
_lib.epx_read_error.argtypes = [ctypes.POINTER(epx_layout), ctypes.POINTER(ctypes.c_int32), _P]
_lib.epx_f32_to_e4m3.argtypes = [_P, _P, ctypes.c_int64, _P]
_lib.epx_relay_fanout.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P, _P,
                                  ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int64, _P]
_lib.epx_combine_relay_partials.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P,
                                            ctypes.c_int64, _P, ctypes.c_int32, ctypes.c_int32, _P,
                                            ctypes.c_int64, _P]
_lib.epx_combine_relay_finish.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P,
                                          ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P]
_lib.epx_layout_dispatch.argtypes = [ctypes.POINTER(epx_problem), _P, ctypes.POINTER(epx_layout), _P,
                                     ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int64, _P]
_lib.epx_layout_dispatch_noalloc.argtypes = [ctypes.POINTER(epx_problem), _P, ctypes.POINTER(epx_layout), _P,
                                             ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int64, _P]
_lib.epx_dispatch_group.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), ctypes.c_int32,
                                    _P, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int64, _P]
_lib.epx_combine_group.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), ctypes.c_int32,
                                   _P, ctypes.c_int64, _P, ctypes.c_int32, _P, _P, _P]
_lib.epx_plan_swaps.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int32,
                                _P, _P, _P, _P, _P, _P]
_I32 = ctypes.c_int32
_lib.epx_route.argtypes = [ctypes.POINTER(epx_problem), _P, _I32, _I32, _P, _I32, ctypes.c_float, _P, _P, _P]
_lib.epx_route_backward.argtypes = [ctypes.POINTER(epx_problem), _P, _I32, _I32, _I32, ctypes.c_float, _P, _P,
                                    _P, _P]
_lib.epx_combine_backward.argtypes = [ctypes.POINTER(epx_problem), ctypes.POINTER(epx_layout), _P, _P,
                                      ctypes.c_int64, _P, _I32, _P, _P, _P]
_lib.epx_expert_gemm.argtypes = [ctypes.POINTER(epx_expert_rows), _P, _P, _I32, _I32, _I32, _P, _P, _P]
_lib.epx_expert_gemm_dgrad.argtypes = [ctypes.POINTER(epx_expert_rows), _P, _P, _I32, _I32, _I32, _P, _P, _P]
_lib.epx_expert_gemm_wgrad.argtypes = [ctypes.POINTER(epx_expert_rows), _P, _P, _I32, _I32, _I32, _I32, _P, _P]
_lib.epx_mxfp4_quantize.argtypes = [_P, ctypes.c_int64, _I32, _P, _P, _P]
_lib.epx_mxfp4_dequantize.argtypes = [_P, _P, ctypes.c_int64, _I32, _P, _P]
_lib.epx_expert_gemm_mxfp4.argtypes = [ctypes.POINTER(epx_expert_rows), _P, _P, _P, _P, _I32, _I32, _I32, _I32,
                                       _P, _P, _P]
_ROWS = ctypes.POINTER(epx_expert_rows)
for _f in ("epx_int8_quantize", "epx_mxint8_quantize"):
    getattr(_lib, _f).argtypes = [_P, ctypes.c_int64, _I32, _P, _P, _P]
for _f in ("epx_int8_dequantize", "epx_mxint8_dequantize"):
    getattr(_lib, _f).argtypes = [_P, _P, ctypes.c_int64, _I32, _P, _P]
_lib.epx_expert_gemm_int8.argtypes = [_ROWS, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P]
_lib.epx_expert_gemm_keep8.argtypes = [_ROWS, _P, _P, _I32, _I32, _P, _P, _P, _P]
_lib.epx_expert_gemm_dgrad_kept8.argtypes = [_ROWS, _P, _P, _I32, _I32, _P, _P, _P, _P, _P]
_lib.epx_expert_gemm_wgrad_kept8.argtypes = [_ROWS, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]
_lib.epx_time_next_call.argtypes = [_P, _P]
_lib.epx_checked_violations.argtypes = [ctypes.POINTER(ctypes.c_int64), _P]
_lib.epx_status_string.argtypes = [ctypes.c_int]
_lib.epx_status_string.restype = ctypes.c_char_p
for _f in ("epx_layout_sizes", "epx_get_layout", "epx_dispatch", "epx_combine", "epx_read_error",
           "epx_f32_to_e4m3", "epx_relay_fanout", "epx_combine_relay_partials",
           "epx_combine_relay_finish", "epx_plan_swaps", "epx_dispatch_group", "epx_combine_group",
           "epx_layout_dispatch", "epx_time_next_call", "epx_layout_dispatch_noalloc",
           "epx_checked_violations", "epx_route", "epx_route_backward", "epx_combine_backward",
           "epx_expert_gemm", "epx_expert_gemm_dgrad", "epx_expert_gemm_wgrad", "epx_mxfp4_quantize",
           "epx_mxfp4_dequantize", "epx_expert_gemm_mxfp4", "epx_int8_quantize", "epx_int8_dequantize",
           "epx_mxint8_quantize", "epx_mxint8_dequantize", "epx_expert_gemm_int8", "epx_expert_gemm_keep8",
           "epx_expert_gemm_dgrad_kept8", "epx_expert_gemm_wgrad_kept8"):
    getattr(_lib, _f).restype = ctypes.c_int
_lib.epx_abi_version.restype = ctypes.c_int32
NARRAYS = len(LAYOUT_FIELDS)


class EpxError(RuntimeError):
    def __init__(self, code: int, call: str):
        msg = _lib.epx_status_string(code).decode()
        super().__init__(f"{call}: {STATUS.get(code, code)} ({msg})")
        self.code = code


def _check(code: int, call: str) -> None:
    if code != 0:
        raise EpxError(code, call)


def abi_version() -> int:
    return int(_lib.epx_abi_version())


def make_problem(num_tokens: int, topk: int, num_experts: int, num_ranks: int, num_hosts: int,
                 my_rank: int = 0, mode: int = MODE_PER_EXPERT, num_groups: int = 1) -> epx_problem:
    return epx_problem(num_tokens, topk, num_experts, num_ranks, num_hosts, my_rank, mode, num_groups)


def epx_layout_sizes(problem: epx_problem) -> List[int]:
    sizes = (ctypes.c_int64 * NARRAYS)()
    _check(_lib.epx_layout_sizes(ctypes.byref(problem), sizes), "epx_layout_sizes")
    return list(sizes)


class Layout:
    """Device arrays of one layout (torch tensors) and the matching C struct."""

    def __init__(self, problem: epx_problem, device="cuda"):
        sizes = epx_layout_sizes(problem)
        relay = problem.mode == MODE_HOST_RELAY
        self.problem = problem
        self.tensors: Dict[str, torch.Tensor] = {}
        ptrs = []
        for name, n in zip(LAYOUT_FIELDS, sizes):
            if name in RELAY_FIELDS and not relay:
                ptrs.append(None)
                continue
            t = torch.empty(max(int(n), 1), dtype=torch.int32, device=device)
            self.tensors[name] = t
            ptrs.append(t.data_ptr())
        self.struct = epx_layout(*ptrs)
        self.sizes = dict(zip(LAYOUT_FIELDS, sizes))

    def __getitem__(self, name: str) -> torch.Tensor:
        return self.tensors[name][: self.sizes[name]]


# The current stream's raw handle: torch's own accessor costs about 0.1 us
# per call against about 3 us for torch.cuda.current_stream() (measured on
# MI355X), which is a third of a decode-sized call's host time.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# The same for the current device (0.1 us against 0.2), once a CUDA tensor exists.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, name: str, ndim: Optional[int] = None) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: need {ndim} dimensions, got {tuple(t.shape)}")


def epx_get_layout(problem: epx_problem, topk_idx: torch.Tensor, layout: Layout, stream=None) -> None:
    _need(topk_idx, torch.int32, "topk_idx", 2)
    if tuple(topk_idx.shape) != (problem.num_tokens, problem.topk):
        raise ValueError(f"topk_idx shape {tuple(topk_idx.shape)} != (T, k)")
    _check(_lib.epx_get_layout(ctypes.byref(problem), topk_idx.data_ptr(), ctypes.byref(layout.struct),
                               _stream(stream)), "epx_get_layout")


def _dispatch_args(problem, x, out_dtype, recv, recv_scales):
    _need(x, torch.bfloat16, "x", 2)
    if x.shape[0] != problem.num_tokens:
        raise ValueError("x: first dimension must be num_tokens")
    hidden = x.shape[1]
    if out_dtype == BF16:
        _need(recv, torch.bfloat16, "recv", 2)
        scales_ptr = None
    else:
        _need(recv, torch.uint8, "recv", 2)
        _need(recv_scales, torch.float32, "recv_scales", 2)
        if recv_scales.shape != (recv.shape[0], hidden // 128):
            raise ValueError("recv_scales: need [capacity_rows, hidden/128]")
        scales_ptr = recv_scales.data_ptr()
    if recv.shape[1] != hidden:
        raise ValueError("recv: second dimension must be hidden")
    return hidden, scales_ptr


def epx_dispatch(problem: epx_problem, layout: Layout, x: torch.Tensor, out_dtype: int,
                 recv: torch.Tensor, recv_scales: Optional[torch.Tensor] = None, stream=None) -> None:
    hidden, scales_ptr = _dispatch_args(problem, x, out_dtype, recv, recv_scales)
    _check(_lib.epx_dispatch(ctypes.byref(problem), ctypes.byref(layout.struct), x.data_ptr(), hidden,
                             out_dtype, recv.data_ptr(), scales_ptr, recv.shape[0], _stream(stream)),
           "epx_dispatch")


def epx_layout_dispatch(problem: epx_problem, topk_idx: torch.Tensor, layout: Layout, x: torch.Tensor,
                        out_dtype: int, recv: torch.Tensor, recv_scales: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """epx_get_layout then epx_dispatch in one call: one launch for decode-sized
    batches, the row assignment and the copies in one launch for larger ones."""
    _need(topk_idx, torch.int32, "topk_idx", 2)
    if tuple(topk_idx.shape) != (problem.num_tokens, problem.topk):
        raise ValueError(f"topk_idx shape {tuple(topk_idx.shape)} != (T, k)")
    hidden, scales_ptr = _dispatch_args(problem, x, out_dtype, recv, recv_scales)
    _check(_lib.epx_layout_dispatch(ctypes.byref(problem), topk_idx.data_ptr(), ctypes.byref(layout.struct),
                                    x.data_ptr(), hidden, out_dtype, recv.data_ptr(), scales_ptr,
                                    recv.shape[0], _stream(stream)),
           "epx_layout_dispatch")


def epx_layout_dispatch_noalloc(problem: epx_problem, topk_idx: torch.Tensor, layout, x: torch.Tensor,
                                out_dtype: int, recv: torch.Tensor, recv_scales: Optional[torch.Tensor] = None,
                                stream=None) -> None:
    """epx_layout_dispatch with the library's static scratch in place of the
    layout's workspace. `layout` is a Layout or an epx_layout struct (its
    workspace may be NULL)."""
    _need(topk_idx, torch.int32, "topk_idx", 2)
    if tuple(topk_idx.shape) != (problem.num_tokens, problem.topk):
        raise ValueError(f"topk_idx shape {tuple(topk_idx.shape)} != (T, k)")
    hidden, scales_ptr = _dispatch_args(problem, x, out_dtype, recv, recv_scales)
    struct = layout.struct if isinstance(layout, Layout) else layout
    _check(_lib.epx_layout_dispatch_noalloc(ctypes.byref(problem), topk_idx.data_ptr(), ctypes.byref(struct),
                                            x.data_ptr(), hidden, out_dtype, recv.data_ptr(), scales_ptr,
                                            recv.shape[0], _stream(stream)),
           "epx_layout_dispatch_noalloc")


def epx_dispatch_group(problem: epx_problem, layout: Layout, group: int, x: torch.Tensor, out_dtype: int,
                       recv: torch.Tensor, recv_scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """Dispatch of one expert group's rows (recv is the whole [T*k, ...] buffer)."""
    hidden, scales_ptr = _dispatch_args(problem, x, out_dtype, recv, recv_scales)
    _check(_lib.epx_dispatch_group(ctypes.byref(problem), ctypes.byref(layout.struct), group, x.data_ptr(),
                                   hidden, out_dtype, recv.data_ptr(), scales_ptr, recv.shape[0],
                                   _stream(stream)),
           "epx_dispatch_group")


def epx_combine(problem: epx_problem, layout: Layout, y: torch.Tensor, topk_weights: torch.Tensor,
                out: torch.Tensor, stream=None) -> None:
    _need(y, torch.bfloat16, "y", 2)
    _need(topk_weights, torch.float32, "topk_weights", 2)
    _need(out, torch.bfloat16, "out", 2)
    if tuple(topk_weights.shape) != (problem.num_tokens, problem.topk):
        raise ValueError("topk_weights: need [T, k]")
    if tuple(out.shape) != (problem.num_tokens, y.shape[1]):
        raise ValueError("out: need [T, hidden]")
    _check(_lib.epx_combine(ctypes.byref(problem), ctypes.byref(layout.struct), y.data_ptr(), y.shape[0],
                            topk_weights.data_ptr(), y.shape[1], out.data_ptr(), _stream(stream)),
           "epx_combine")


def epx_combine_group(problem: epx_problem, layout: Layout, group: int, y: torch.Tensor,
                      topk_weights: torch.Tensor, carry: Optional[torch.Tensor], out: torch.Tensor,
                      stream=None) -> None:
    """One expert group's combine; call for groups 0..m-1 in order on one
    float32 [T, hidden] carry."""
    _need(y, torch.bfloat16, "y", 2)
    _need(topk_weights, torch.float32, "topk_weights", 2)
    _need(out, torch.bfloat16, "out", 2)
    if tuple(topk_weights.shape) != (problem.num_tokens, problem.topk):
        raise ValueError("topk_weights: need [T, k]")
    if tuple(out.shape) != (problem.num_tokens, y.shape[1]):
        raise ValueError("out: need [T, hidden]")
    if carry is not None:
        _need(carry, torch.float32, "carry", 2)
        if tuple(carry.shape) != tuple(out.shape):
            raise ValueError("carry: need [T, hidden]")
    _check(_lib.epx_combine_group(ctypes.byref(problem), ctypes.byref(layout.struct), group, y.data_ptr(),
                                  y.shape[0], topk_weights.data_ptr(), y.shape[1],
                                  carry.data_ptr() if carry is not None else None, out.data_ptr(),
                                  _stream(stream)),
           "epx_combine_group")


def epx_read_error(layout: Layout, stream=None) -> int:
    """Synchronising read of the layout's bad-id count (0 = all ids valid)."""
    bad = ctypes.c_int32(0)
    code = _lib.epx_read_error(ctypes.byref(layout.struct), ctypes.byref(bad), _stream(stream))
    if code not in (0, 2):
        _check(code, "epx_read_error")
    return int(bad.value)


def epx_time_next_call(start_event: Optional[int], stop_event: Optional[int]) -> None:
    """Bind two raw hipEvent_t handles to the kernels of the next library call
    from this thread (start: its first kernel's start, stop: its last kernel's
    end); None, None disarms."""
    _check(_lib.epx_time_next_call(start_event, stop_event), "epx_time_next_call")


def epx_checked_violations(stream=None) -> int:
    """Bounds-checked library only: accesses its checks skipped since the last
    call (synchronises the stream and resets the count)."""
    n = ctypes.c_int64(-1)
    _check(_lib.epx_checked_violations(ctypes.byref(n), _stream(stream)), "epx_checked_violations")
    return int(n.value)


def epx_f32_to_e4m3(inp: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    _need(inp, torch.float32, "in")
    _need(out, torch.uint8, "out")
    if inp.numel() != out.numel():
        raise ValueError("in/out sizes differ")
    _check(_lib.epx_f32_to_e4m3(inp.data_ptr(), out.data_ptr(), inp.numel(), _stream(stream)),
           "epx_f32_to_e4m3")


def epx_relay_fanout(problem: epx_problem, layout: Layout, relay_rows: torch.Tensor, recv: torch.Tensor,
                     relay_scales: Optional[torch.Tensor] = None, recv_scales: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Relay rows -> per-expert rows (bf16 rows, or fp8 codes with scales)."""
    fp8 = relay_rows.dtype == torch.uint8
    _need(relay_rows, torch.uint8 if fp8 else torch.bfloat16, "relay_rows", 2)
    _need(recv, relay_rows.dtype, "recv", 2)
    hidden = relay_rows.shape[1]
    if recv.shape[1] != hidden:
        raise ValueError("recv: hidden differs from relay_rows")
    if fp8:
        _need(relay_scales, torch.float32, "relay_scales", 2)
        _need(recv_scales, torch.float32, "recv_scales", 2)
        # the kernel reads relay_scales[r] for relay rows r and writes
        # recv_scales[o] for per-expert rows o: one scale per 128 channels
        if tuple(relay_scales.shape) != (relay_rows.shape[0], hidden // 128):
            raise ValueError("relay_scales: need [relay_rows, hidden/128]")
        if tuple(recv_scales.shape) != (recv.shape[0], hidden // 128):
            raise ValueError("recv_scales: need [capacity_rows, hidden/128]")
    _check(_lib.epx_relay_fanout(ctypes.byref(problem), ctypes.byref(layout.struct), relay_rows.data_ptr(),
                                 relay_scales.data_ptr() if fp8 else None, relay_rows.shape[0], hidden,
                                 FP8_E4M3 if fp8 else BF16, recv.data_ptr(),
                                 recv_scales.data_ptr() if fp8 else None, recv.shape[0], _stream(stream)),
           "epx_relay_fanout")


def epx_combine_relay_partials(problem: epx_problem, layout: Layout, y: torch.Tensor,
                               topk_weights: torch.Tensor, partials: torch.Tensor, stream=None) -> None:
    """Per relay row fp32 (float32 tensor) or bf16 (bfloat16 tensor) partial sums."""
    _need(y, torch.bfloat16, "y", 2)
    _need(topk_weights, torch.float32, "topk_weights", 2)
    if partials.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("partials: float32 or bfloat16")
    _need(partials, partials.dtype, "partials", 2)
    if partials.shape[1] != y.shape[1]:
        raise ValueError("partials: hidden differs from y")
    pd = F32 if partials.dtype == torch.float32 else BF16
    _check(_lib.epx_combine_relay_partials(ctypes.byref(problem), ctypes.byref(layout.struct), y.data_ptr(),
                                           y.shape[0], topk_weights.data_ptr(), y.shape[1], pd,
                                           partials.data_ptr(), partials.shape[0], _stream(stream)),
           "epx_combine_relay_partials")


def epx_combine_relay_finish(problem: epx_problem, layout: Layout, partials: torch.Tensor,
                             out: torch.Tensor, stream=None) -> None:
    if partials.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("partials: float32 or bfloat16")
    _need(partials, partials.dtype, "partials", 2)
    _need(out, torch.bfloat16, "out", 2)
    if tuple(out.shape) != (problem.num_tokens, partials.shape[1]):
        raise ValueError("out: need [T, hidden]")
    pd = F32 if partials.dtype == torch.float32 else BF16
    _check(_lib.epx_combine_relay_finish(ctypes.byref(problem), ctypes.byref(layout.struct),
                                         partials.data_ptr(), partials.shape[0], pd, partials.shape[1],
                                         out.data_ptr(), _stream(stream)),
           "epx_combine_relay_finish")


def epx_plan_swaps(num_experts: int, num_ranks: int, num_hosts: int, expert_count: torch.Tensor,
                   slot_expert: torch.Tensor, tau: int, out: Optional[dict] = None, stream=None) -> dict:
    """Per-step intra-host expert swaps. Returns (and fills, if given) the
    int32 tensors slot_expert [E], load_before [R], load_after [R],
    swaps [H * (R/H)//2, 7] and host_bad [H]."""
    E, R, H = num_experts, num_ranks, num_hosts
    _need(expert_count, torch.int32, "expert_count", 1)
    _need(slot_expert, torch.int32, "slot_expert", 1)
    if expert_count.numel() < E or slot_expert.numel() != E:
        raise ValueError("expert_count needs >= E entries, slot_expert exactly E")
    npair = H * ((R // H) // 2) if H > 0 and R % H == 0 else 0
    shapes = {"slot_expert": (E,), "load_before": (R,), "load_after": (R,), "swaps": (npair, 7),
              "host_bad": (H,)}
    if out is None:
        out = {n: torch.empty(sh, dtype=torch.int32, device=slot_expert.device) for n, sh in shapes.items()}
    for n, sh in shapes.items():
        _need(out[n], torch.int32, n)
        if tuple(out[n].shape) != sh:
            raise ValueError(f"{n}: need shape {sh}")
    _check(_lib.epx_plan_swaps(E, R, H, expert_count.data_ptr(), slot_expert.data_ptr(), tau,
                               out["slot_expert"].data_ptr(), out["load_before"].data_ptr(),
                               out["load_after"].data_ptr(), out["swaps"].data_ptr() if npair else None,
                               out["host_bad"].data_ptr(), _stream(stream)),
           "epx_plan_swaps")
    return out


_LOGITS = {torch.bfloat16: BF16, torch.float32: F32}


def _device(t, name: str) -> int:
    """The index of the current device, which the tensors of a call have to be
    on: the calls launch there, and pointers of another one would be read across."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: need a CUDA tensor")
    dev = _current_device()
    if t.get_device() != dev:
        raise ValueError(f"{name}: on device {t.get_device()}, the current device is {dev}")
    return dev


def _ptr(t, dtype, name: str, shape: tuple, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on the device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:   # no tensor
        pass
    _need(t, dtype, name, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name}: need shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name}: on device {t.get_device()}, the current device is {dev}")


def _columns(t, dtype, name: str) -> int:
    """Columns of a tensor of two dimensions (whose shape _ptr checks)."""
    try:
        _, n = t.shape
    except (AttributeError, ValueError):
        _need(t, dtype, name, 2)
        raise ValueError(f"{name}: need 2 dimensions") from None
    return n


def _rows_device(rows) -> int:
    """As _device, for row ranges (CUDA tensors, checked when they were made)."""
    dev = _current_device()
    if rows.device != dev:
        raise ValueError(f"rows: on device {rows.device}, the current device is {dev}")
    return dev


def _launch_stream(stream, dev: int) -> int:
    if stream is None and _raw_current_stream is not None:
        return _raw_current_stream(dev)
    return _stream(stream)


def _logits_dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _LOGITS:
        raise ValueError(f"{name}: bfloat16 or float32")
    return _LOGITS[t.dtype]


def epx_route(problem: epx_problem, logits: torch.Tensor, score: int, topk_idx: torch.Tensor,
              topk_weights: torch.Tensor, bias: Optional[torch.Tensor] = None, renormalize: bool = True,
              scale: float = 1.0, stream=None) -> None:
    """Router: the k experts of every token and their weights, from logits [T, E]."""
    code, dev = _logits_dtype(logits, "logits"), _device(logits, "logits")
    T, E, k = problem.num_tokens, problem.num_experts, problem.topk
    _check(_lib.epx_route(ctypes.byref(problem), _ptr(logits, logits.dtype, "logits", (T, E), dev), code, score,
                          _ptr(bias, torch.float32, "bias", (E,), dev) if bias is not None else None,
                          int(bool(renormalize)), scale, _ptr(topk_idx, torch.int32, "topk_idx", (T, k), dev),
                          _ptr(topk_weights, torch.float32, "topk_weights", (T, k), dev),
                          _launch_stream(stream, dev)), "epx_route")


def epx_route_backward(problem: epx_problem, logits: torch.Tensor, score: int, topk_idx: torch.Tensor,
                       dweights: torch.Tensor, dlogits: torch.Tensor, renormalize: bool = True,
                       scale: float = 1.0, stream=None) -> None:
    """Gradient of epx_route's weights: dlogits [T, E] from dweights [T, k]."""
    code, dev = _logits_dtype(logits, "logits"), _device(logits, "logits")
    T, E, k = problem.num_tokens, problem.num_experts, problem.topk
    _check(_lib.epx_route_backward(ctypes.byref(problem), _ptr(logits, logits.dtype, "logits", (T, E), dev), code,
                                   score, int(bool(renormalize)), scale,
                                   _ptr(topk_idx, torch.int32, "topk_idx", (T, k), dev),
                                   _ptr(dweights, torch.float32, "dweights", (T, k), dev),
                                   _ptr(dlogits, logits.dtype, "dlogits", (T, E), dev),
                                   _launch_stream(stream, dev)), "epx_route_backward")


def epx_combine_backward(problem: epx_problem, layout: Layout, dout: torch.Tensor, y: Optional[torch.Tensor],
                         topk_weights: torch.Tensor, dy: torch.Tensor,
                         dweights: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradient of epx_combine: dy (rows of y) and, if given, dweights [T, k]
    (without it y is not read and may be None)."""
    dev = _device(dy, "dy")
    _need(dy, torch.bfloat16, "dy", 2)
    T, k = problem.num_tokens, problem.topk
    y_rows, hidden = dy.shape
    _check(_lib.epx_combine_backward(ctypes.byref(problem), ctypes.byref(layout.struct),
                                     _ptr(dout, torch.bfloat16, "dout", (T, hidden), dev),
                                     _ptr(y, torch.bfloat16, "y", (y_rows, hidden), dev)
                                     if dweights is not None else None, y_rows,
                                     _ptr(topk_weights, torch.float32, "topk_weights", (T, k), dev), hidden,
                                     dy.data_ptr(),
                                     _ptr(dweights, torch.float32, "dweights", (T, k), dev)
                                     if dweights is not None else None, _launch_stream(stream, dev)),
           "epx_combine_backward")


class ExpertRows:
    """Row ranges of the experts on this GPU (device tensors) and the matching C struct."""

    def __init__(self, row_offset: torch.Tensor, row_count: torch.Tensor, num_rows: int):
        _need(row_offset, torch.int32, "row_offset", 1)
        _need(row_count, torch.int32, "row_count", 1)
        if row_offset.numel() < row_count.numel() or row_offset.device != row_count.device:
            raise ValueError("row_offset: need an entry for every expert of row_count, on its device")
        if not 0 <= num_rows <= (1 << 31) - 4096:
            raise ValueError("num_rows: need 0 <= num_rows <= 2^31 - 4096")
        self.row_offset, self.row_count = row_offset, row_count
        self.num_experts, self.num_rows, self.device = row_count.numel(), int(num_rows), row_count.get_device()
        self.struct = epx_expert_rows(self.num_experts, self.num_rows, row_offset.data_ptr(), row_count.data_ptr())


def expert_rows(row_offset: torch.Tensor, row_count: torch.Tensor, num_rows: int) -> ExpertRows:
    """Rows [row_offset[e], row_offset[e] + row_count[e]) for each expert e, in
    buffers of num_rows rows. A layout's arrays serve as they are:
    expert_rows(L["expert_offset"], L["expert_count"], T * k)."""
    return ExpertRows(row_offset, row_count, num_rows)


def epx_expert_gemm(rows: ExpertRows, x: torch.Tensor, w: torch.Tensor, out: torch.Tensor, act: int = ACT_NONE,
                    preact: Optional[torch.Tensor] = None, stream=None) -> None:
    """out[r] = act(x[r] @ w[e].T) for the rows r of every expert e. With
    ACT_SWIGLU w is [n, 2 * width, inner] (gate rows, then up rows) and preact,
    if given, receives the product before the activation."""
    dev, bf16 = _rows_device(rows), torch.bfloat16
    width, inner, R = _columns(out, bf16, "out"), _columns(x, bf16, "x"), rows.num_rows
    wide = 2 * width if act == ACT_SWIGLU else width
    _check(_lib.epx_expert_gemm(ctypes.byref(rows.struct), _ptr(x, bf16, "x", (R, inner), dev),
                                _ptr(w, bf16, "w", (rows.num_experts, wide, inner), dev), width, inner, act,
                                _ptr(preact, bf16, "preact", (R, wide), dev) if preact is not None else None,
                                _ptr(out, bf16, "out", (R, width), dev), _launch_stream(stream, dev)),
           "epx_expert_gemm")


def epx_expert_gemm_dgrad(rows: ExpertRows, dy: torch.Tensor, w: torch.Tensor, dx: torch.Tensor,
                          input_act: int = ACT_NONE, preact: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx[r] = dy[r] @ w[e]; with input_act=ACT_SWIGLU (the product's input was
    the gated activation of preact) dx is the gradient of preact."""
    dev, bf16 = _rows_device(rows), torch.bfloat16
    try:
        n, width, inner = w.shape
    except (AttributeError, ValueError):
        _need(w, bf16, "w", 3)
        raise ValueError("w: need 3 dimensions") from None
    R = rows.num_rows
    wide = 2 * inner if input_act == ACT_SWIGLU else inner
    _check(_lib.epx_expert_gemm_dgrad(ctypes.byref(rows.struct), _ptr(dy, bf16, "dy", (R, width), dev),
                                      _ptr(w, bf16, "w", (rows.num_experts, width, inner), dev), width, inner,
                                      input_act,
                                      _ptr(preact, bf16, "preact", (R, wide), dev) if preact is not None else None,
                                      _ptr(dx, bf16, "dx", (R, wide), dev), _launch_stream(stream, dev)),
           "epx_expert_gemm_dgrad")


def epx_expert_gemm_wgrad(rows: ExpertRows, dy: torch.Tensor, x: torch.Tensor, dw: torch.Tensor,
                          accumulate: bool = False, stream=None) -> None:
    """dw[e] = dy[r].T @ x[r] summed over the rows of every expert e; bfloat16
    or float32, the latter also added to what dw holds."""
    code, dev, bf16 = _logits_dtype(dw, "dw"), _rows_device(rows), torch.bfloat16
    if dw.dim() != 3:
        raise ValueError(f"dw: need 3 dimensions, got {tuple(dw.shape)}")
    n, width, inner = dw.shape
    R = rows.num_rows
    _check(_lib.epx_expert_gemm_wgrad(ctypes.byref(rows.struct), _ptr(dy, bf16, "dy", (R, width), dev),
                                      _ptr(x, bf16, "x", (R, inner), dev), width, inner, code,
                                      int(bool(accumulate)),
                                      _ptr(dw, dw.dtype, "dw", (rows.num_experts, width, inner), dev),
                                      _launch_stream(stream, dev)), "epx_expert_gemm_wgrad")


def _mxfp4_args(values, codes, scales, name):
    """(rows, inner, addresses, device); rows are the product of all dimensions but the last."""
    dev = _device(values, name)
    _need(values, torch.bfloat16, name)
    if values.dim() < 2:
        raise ValueError(f"{name}: need at least 2 dimensions")
    inner, lead = values.shape[-1], tuple(values.shape[:-1])
    if inner == 0 or inner % 32:
        raise ValueError(f"{name}: the last dimension must be a multiple of 32")
    return (values.numel() // inner, inner, values.data_ptr(),
            _ptr(codes, torch.uint8, "codes", lead + (inner // 2,), dev),
            _ptr(scales, torch.uint8, "scales", lead + (inner // 32,), dev), dev)


def epx_mxfp4_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """bf16 rows [..., inner] to 4-bit codes [..., inner/2] and scale bytes [..., inner/32]."""
    num_rows, inner, px, pc, ps, dev = _mxfp4_args(x, codes, scales, "x")
    _check(_lib.epx_mxfp4_quantize(px, num_rows, inner, pc, ps, _launch_stream(stream, dev)), "epx_mxfp4_quantize")


def epx_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """The bf16 values that 4-bit codes and scale bytes stand for."""
    num_rows, inner, po, pc, ps, dev = _mxfp4_args(out, codes, scales, "out")
    _check(_lib.epx_mxfp4_dequantize(pc, ps, num_rows, inner, po, _launch_stream(stream, dev)),
           "epx_mxfp4_dequantize")


def epx_expert_gemm_mxfp4(rows: ExpertRows, x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor,
                          w_scales: torch.Tensor, out: torch.Tensor, act: int = ACT_NONE,
                          out_scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """epx_expert_gemm for fp8 rows (codes and a float32 scale per 128 channels,
    as epx_dispatch writes them) and 4-bit weights. out is bfloat16, or uint8
    codes with out_scales [rows, width/128]."""
    dev, u8, f32 = _rows_device(rows), torch.uint8, torch.float32
    fp8 = isinstance(out, torch.Tensor) and out.dtype is u8
    rtype = u8 if fp8 else torch.bfloat16
    if out_scales is not None and not fp8:
        raise ValueError("out_scales: only with uint8 rows out")
    width, inner, R, n = _columns(out, rtype, "out"), _columns(x, u8, "x"), rows.num_rows, rows.num_experts
    wide = 2 * width if act == ACT_SWIGLU else width
    _check(_lib.epx_expert_gemm_mxfp4(ctypes.byref(rows.struct), _ptr(x, u8, "x", (R, inner), dev),
                                      _ptr(x_scales, f32, "x_scales", (R, inner // 128), dev),
                                      _ptr(w, u8, "w", (n, wide, inner // 2), dev),
                                      _ptr(w_scales, u8, "w_scales", (n, wide, inner // 32), dev), width, inner, act,
                                      FP8_E4M3 if fp8 else BF16, _ptr(out, rtype, "out", (R, width), dev),
                                      _ptr(out_scales, f32, "out_scales", (R, width // 128), dev) if fp8 else None,
                                      _launch_stream(stream, dev)), "epx_expert_gemm_mxfp4")


def _rows8_args(values, codes, scales, name, unit, scale_dtype):
    """(rows, inner, addresses, device); rows are the product of all dimensions but the last."""
    try:
        shape, dev = values.shape, values.get_device()
        lead, inner = shape[:-1], shape[-1]
        # the usual call, in as few steps as tell it (these calls are short)
        if (len(shape) > 1 and inner and inner % unit == 0 and values.dtype is torch.bfloat16
                and codes.dtype is torch.int8 and scales.dtype is scale_dtype and codes.shape == shape
                and scales.shape == (lead if unit == 16 else lead + (inner // 32,))
                and dev >= 0 and dev == codes.get_device() == scales.get_device() == _current_device()
                and values.is_contiguous() and codes.is_contiguous() and scales.is_contiguous()):
            return values.numel() // inner, inner, values.data_ptr(), codes.data_ptr(), scales.data_ptr(), dev
    except (AttributeError, IndexError):   # no tensor, or one without dimensions
        pass
    dev = _device(values, name)
    _need(values, torch.bfloat16, name)
    if values.dim() < 2:
        raise ValueError(f"{name}: need at least 2 dimensions")
    inner, lead = values.shape[-1], tuple(values.shape[:-1])
    if inner == 0 or inner % unit:
        raise ValueError(f"{name}: the last dimension must be a multiple of {unit}")
    return (values.numel() // inner, inner, values.data_ptr(), _ptr(codes, torch.int8, "codes", lead + (inner,), dev),
            _ptr(scales, scale_dtype, "scales", lead if unit == 16 else lead + (inner // 32,), dev), dev)


def epx_int8_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """bf16 rows [..., inner] to int8 codes [..., inner] and a float32 scale a row [...]."""
    num_rows, inner, px, pc, ps, dev = _rows8_args(x, codes, scales, "x", 16, torch.float32)
    _check(_lib.epx_int8_quantize(px, num_rows, inner, pc, ps, _launch_stream(stream, dev)), "epx_int8_quantize")


def epx_int8_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """bf16(code * scale) of int8 rows."""
    num_rows, inner, po, pc, ps, dev = _rows8_args(out, codes, scales, "out", 16, torch.float32)
    _check(_lib.epx_int8_dequantize(pc, ps, num_rows, inner, po, _launch_stream(stream, dev)), "epx_int8_dequantize")


def epx_mxint8_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """bf16 rows [..., inner] to int8 codes [..., inner] and a scale byte per 32 values [..., inner/32]."""
    num_rows, inner, px, pc, ps, dev = _rows8_args(x, codes, scales, "x", 32, torch.uint8)
    _check(_lib.epx_mxint8_quantize(px, num_rows, inner, pc, ps, _launch_stream(stream, dev)), "epx_mxint8_quantize")


def epx_mxint8_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """The bf16 values that int8 codes and scale bytes stand for (exact)."""
    num_rows, inner, po, pc, ps, dev = _rows8_args(out, codes, scales, "out", 32, torch.uint8)
    _check(_lib.epx_mxint8_dequantize(pc, ps, num_rows, inner, po, _launch_stream(stream, dev)),
           "epx_mxint8_dequantize")


def _kept_ptrs(codes, scales, name: str, R: int, columns: int, dev: int):
    """Addresses of [R, columns] activations kept in 8 bits, and of their scale bytes."""
    if columns % 32:
        raise ValueError(f"{name}_codes: the last dimension must be a multiple of 32")
    return (_ptr(codes, torch.int8, name + "_codes", (R, columns), dev),
            _ptr(scales, torch.uint8, name + "_scales", (R, columns // 32), dev))


def epx_expert_gemm_int8(rows: ExpertRows, x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor,
                         w_scales: torch.Tensor, out: torch.Tensor, act: int = ACT_NONE,
                         preact_codes: Optional[torch.Tensor] = None, preact_scales: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """epx_expert_gemm for int8 rows (a float32 scale each, as epx_int8_quantize
    writes them) and int8 weights [n, width or 2 * width, inner] with a scale
    per column of the product. With ACT_SWIGLU preact_codes and preact_scales, if
    given, receive the product before the activation in 8 bits."""
    dev, i8, f32 = _rows_device(rows), torch.int8, torch.float32
    width, inner, R, n = _columns(out, torch.bfloat16, "out"), _columns(x, i8, "x"), rows.num_rows, rows.num_experts
    wide = 2 * width if act == ACT_SWIGLU else width
    pc, ps = None, None
    if preact_codes is not None or preact_scales is not None:
        pc, ps = _kept_ptrs(preact_codes, preact_scales, "preact", R, wide, dev)
    _check(_lib.epx_expert_gemm_int8(ctypes.byref(rows.struct), _ptr(x, i8, "x", (R, inner), dev),
                                     _ptr(x_scales, f32, "x_scales", (R,), dev),
                                     _ptr(w, i8, "w", (n, wide, inner), dev),
                                     _ptr(w_scales, f32, "w_scales", (n, wide), dev), width, inner, act, pc, ps,
                                     _ptr(out, torch.bfloat16, "out", (R, width), dev), _launch_stream(stream, dev)),
           "epx_expert_gemm_int8")


def epx_expert_gemm_keep8(rows: ExpertRows, x: torch.Tensor, w: torch.Tensor, out: torch.Tensor,
                          preact_codes: torch.Tensor, preact_scales: torch.Tensor, stream=None) -> None:
    """epx_expert_gemm with ACT_SWIGLU that keeps the product before the
    activation in 8 bits (as epx_mxint8_quantize keeps rows)."""
    dev, bf16 = _rows_device(rows), torch.bfloat16
    width, inner, R = _columns(out, bf16, "out"), _columns(x, bf16, "x"), rows.num_rows
    pc, ps = _kept_ptrs(preact_codes, preact_scales, "preact", R, 2 * width, dev)
    _check(_lib.epx_expert_gemm_keep8(ctypes.byref(rows.struct), _ptr(x, bf16, "x", (R, inner), dev),
                                      _ptr(w, bf16, "w", (rows.num_experts, 2 * width, inner), dev), width, inner, pc,
                                      ps, _ptr(out, bf16, "out", (R, width), dev), _launch_stream(stream, dev)),
           "epx_expert_gemm_keep8")


def epx_expert_gemm_dgrad_kept8(rows: ExpertRows, dy: torch.Tensor, w: torch.Tensor, preact_codes: torch.Tensor,
                                preact_scales: torch.Tensor, dx: torch.Tensor, act_out: Optional[torch.Tensor] = None,
                                stream=None) -> None:
    """epx_expert_gemm_dgrad with input_act=ACT_SWIGLU and pre-activations kept
    in 8 bits; act_out, if given, receives the activation of the kept values."""
    dev, bf16 = _rows_device(rows), torch.bfloat16
    try:
        n, width, inner = w.shape
    except (AttributeError, ValueError):
        _need(w, bf16, "w", 3)
        raise ValueError("w: need 3 dimensions") from None
    R = rows.num_rows
    pc, ps = _kept_ptrs(preact_codes, preact_scales, "preact", R, 2 * inner, dev)
    _check(_lib.epx_expert_gemm_dgrad_kept8(ctypes.byref(rows.struct), _ptr(dy, bf16, "dy", (R, width), dev),
                                            _ptr(w, bf16, "w", (rows.num_experts, width, inner), dev), width, inner, pc,
                                            ps,
                                            _ptr(act_out, bf16, "act_out", (R, inner), dev)
                                            if act_out is not None else None,
                                            _ptr(dx, bf16, "dx", (R, 2 * inner), dev), _launch_stream(stream, dev)),
           "epx_expert_gemm_dgrad_kept8")


def epx_expert_gemm_wgrad_kept8(rows: ExpertRows, dy: torch.Tensor, x_codes: torch.Tensor, x_scales: torch.Tensor,
                                dw: torch.Tensor, accumulate: bool = False, stream=None) -> None:
    """epx_expert_gemm_wgrad for rows x kept in 8 bits by epx_mxint8_quantize."""
    code, dev, bf16 = _logits_dtype(dw, "dw"), _rows_device(rows), torch.bfloat16
    if dw.dim() != 3:
        raise ValueError(f"dw: need 3 dimensions, got {tuple(dw.shape)}")
    n, width, inner = dw.shape
    R = rows.num_rows
    pc, ps = _kept_ptrs(x_codes, x_scales, "x", R, inner, dev)
    _check(_lib.epx_expert_gemm_wgrad_kept8(ctypes.byref(rows.struct), _ptr(dy, bf16, "dy", (R, width), dev), pc, ps,
                                            width, inner, code, int(bool(accumulate)),
                                            _ptr(dw, dw.dtype, "dw", (rows.num_experts, width, inner), dev),
                                            _launch_stream(stream, dev)), "epx_expert_gemm_wgrad_kept8")


def relay_capacity(problem: epx_problem) -> int:
    return problem.num_tokens * min(problem.topk, problem.num_hosts)
