"""ctypes binding of libmoe_route.so (include/moe_route.h, include/moe_layer.h, include/moe_block.h),
with the C names.

Argument marshalling only: torch tensors supply device memory and the current HIP stream, and
every step runs in the library's HIP kernels. If the library is not built, loading fails with an
ImportError; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_route.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOPK = 64
MOE_NOALLOC_SCRATCH_BYTES = 16 << 20
MOE_MAX_SEQS = 65536
MOE_MATMUL_MAX_K = 131056
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
ACT_CODES = {"none": MOE_ACT_NONE, "swiglu": MOE_ACT_SWIGLU}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
SCORE_CODES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_MAX_GROUPS = 64
MOE_MAT_NONE, MOE_MAT_SWIGLU, MOE_MAT_RELU, MOE_MAT_SILU, MOE_MAT_GELU = range(5)
MAT_ACT_CODES = {"none": MOE_MAT_NONE, "swiglu": MOE_MAT_SWIGLU, "relu": MOE_MAT_RELU,
                 "silu": MOE_MAT_SILU, "gelu": MOE_MAT_GELU}
MOE_MAT_MAX_SIZE = 4194304

DTYPE_CODES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8_e4m3": MOE_FP8_E4M3}
TORCH_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8_e4m3": torch.uint8}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {moe_status_str(status)}")
        self.status = status


class moe_dispatch_out_t(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "recv", "recv_scales", "expert_counts", "expert_offsets", "rank_counts", "rank_offsets",
        "token_row", "row_token")]


_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        lib.moe_status_str.argtypes = [I]
        lib.moe_status_str.restype = ctypes.c_char_p
        lib.moe_route_topk.argtypes = [P, I, I, I, P, P, P]
        lib.moe_dispatch_workspace_bytes.argtypes = [I, I, I]
        lib.moe_dispatch_workspace_bytes.restype = Z
        lib.moe_dispatch_layout.argtypes = [P, I, I, I, I, P, P, Z, P]
        lib.moe_dispatch_pack.argtypes = [P, I, I, I, I, P, I, P, P, P]
        lib.moe_dispatch.argtypes = [P, I, I, I, P, I, I, I, I, P, P, Z, P]
        lib.moe_route_dispatch.argtypes = [P, P, I, I, I, I, I, I, I, P, P, P, P, Z, P]
        lib.moe_route_dispatch_noalloc.argtypes = [P, P, I, I, I, I, I, I, I, P, P, P, P]
        lib.moe_combine.argtypes = [P, I, I, I, I, P, P, P, I, P]
        lib.moe_ep_capacity.argtypes = [I, I, I, I]
        lib.moe_ep_capacity.restype = ctypes.c_int64
        lib.moe_ep_send.argtypes = [P, I, I, I, P, I, I, I, I, I, I, P, P, P, P, Z, P]
        lib.moe_ep_recv.argtypes = [P, I, I, I, I, I, I, I, P, P, P, P, P, P]
        lib.moe_ep_return.argtypes = [P, I, I, I, I, I, I, P, P, P, P]
        lib.moe_ep_combine.argtypes = [P, I, I, I, I, P, P, I, P, I, P]
        lib.moe_ep_partial_rows.argtypes = [P, I, I, I, I, I, I, I, P, P, P]
        lib.moe_ep_reduce_workspace_bytes.argtypes = [I, I]
        lib.moe_ep_reduce_workspace_bytes.restype = Z
        lib.moe_ep_reduce.argtypes = [P, I, I, I, I, I, I, I, P, I, I, P, P, P, P, I, P, P, Z, P]
        lib.moe_ep_combine_reduced.argtypes = [P, I, I, I, I, P, I, P, I, P]
        lib.moe_check_topk.argtypes = [P, I, I, I, P, P]
        F = ctypes.c_float
        lib.moe_balance_workspace_bytes.argtypes = [I, I, I]
        lib.moe_balance_workspace_bytes.restype = Z
        lib.moe_balance_loss.argtypes = [P, P, P, I, I, I, I, F, P, P, P, P, P, Z, P]
        lib.moe_route_grad.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, F, P, P]
        lib.moe_quant_rows.argtypes = [P, I, I, I, P, P, P, P]
        lib.moe_expert_matmul_i8.argtypes = [P, P, I, P, P, P, P, I, I, I, I, I, P, I, P]
        lib.moe_route_scored.argtypes = [P, P, I, I, I, I, I, I, I, I, F, P, P, P]
        lib.moe_route_scored_grad.argtypes = [P, P, P, P, I, I, I, I, I, F, P, P]
        lib.moe_bias_update.argtypes = [P, P, I, I, F, P, P]
        lib.moe_combine_grad.argtypes = [P, I, P, I, P, P, I, I, I, P, P, P]
        lib.moe_expert_matmul_workspace_bytes.argtypes = [I, I, I, I]
        lib.moe_expert_matmul_workspace_bytes.restype = Z
        lib.moe_expert_matmul.argtypes = [P, I, P, P, P, P, I, I, I, I, I, P, P, P, I, P, Z, P]
        lib.moe_matmul_grad_workspace_bytes.argtypes = [I, I, I, I]
        lib.moe_matmul_grad_workspace_bytes.restype = Z
        lib.moe_expert_matmul_grad.argtypes = [P, P, I, P, P, P, I, I, I, I, I, P, P, I, P, I, P, P, Z,
                                               P]
        for fn in ("moe_route_scored", "moe_route_scored_grad", "moe_bias_update", "moe_combine_grad",
                   "moe_expert_matmul", "moe_expert_matmul_grad", "moe_balance_loss", "moe_route_grad", "moe_quant_rows", "moe_expert_matmul_i8",
                   "moe_route_topk", "moe_dispatch_layout", "moe_dispatch_pack", "moe_dispatch",
                   "moe_route_dispatch", "moe_route_dispatch_noalloc", "moe_combine", "moe_ep_send",
                   "moe_ep_recv", "moe_ep_return", "moe_ep_combine", "moe_ep_partial_rows", "moe_ep_reduce",
                   "moe_ep_combine_reduced", "moe_check_topk"):
            getattr(lib, fn).restype = I
        _lib = lib
    return _lib


def moe_status_str(status: int) -> str:
    return load().moe_status_str(status).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor, fp8_ok: bool = False) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if fp8_ok and t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_FP8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def moe_route_topk(logits: torch.Tensor, k: int, topk_idx: Optional[torch.Tensor] = None,
                   topk_w: Optional[torch.Tensor] = None, stream=None):
    """Top-k expert ids (int32 [T,k]) and renormalised softmax weights (fp32 [T,k])."""
    T, E = logits.shape
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    assert logits.dtype == torch.float32 and logits.is_contiguous()
    _check("moe_route_topk", load().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx),
                                                   _ptr(topk_w), _stream(stream)))
    return topk_idx, topk_w


def moe_check_topk(topk_idx: torch.Tensor, E: int, counts: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Device int32 [2]: slots with an id outside [0, E), in-range slots repeating an earlier slot
    of their token. Enqueued on the stream; read it after the stream has finished."""
    T, k = topk_idx.shape
    if counts is None:
        counts = torch.empty(2, dtype=torch.int32, device=topk_idx.device)
    assert topk_idx.dtype == torch.int32 and topk_idx.is_contiguous()
    _check("moe_check_topk", load().moe_check_topk(_ptr(topk_idx), T, k, E, _ptr(counts),
                                                   _stream(stream)))
    return counts


def _debug_check_ids(fn: str, topk_idx: torch.Tensor, E: int, stream) -> None:
    """With MOE_ROUTE_DEBUG=1, check caller-given ids on the GPU before they are dispatched and
    raise ValueError naming what is wrong (this waits for the stream)."""
    if os.environ.get("MOE_ROUTE_DEBUG", "0") != "1":
        return
    counts = moe_check_topk(topk_idx, E, stream=stream)
    bad, rep = (int(v) for v in counts.cpu().tolist())
    if bad or rep:
        raise ValueError(f"{fn}: {bad} expert ids outside [0, {E}) and {rep} repeated within a "
                         f"token (MOE_ROUTE_DEBUG=1)")


def moe_dispatch_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(load().moe_dispatch_workspace_bytes(T, E, k))


@dataclass
class DispatchBuffers:
    """Caller-owned dispatch outputs (device tensors)."""
    recv: Optional[torch.Tensor]
    recv_scales: Optional[torch.Tensor]
    expert_counts: torch.Tensor
    expert_offsets: torch.Tensor
    rank_counts: torch.Tensor
    rank_offsets: torch.Tensor
    token_row: torch.Tensor
    row_token: torch.Tensor

    def as_struct(self) -> moe_dispatch_out_t:
        s = moe_dispatch_out_t()
        for name, _ in moe_dispatch_out_t._fields_:
            t = getattr(self, name)
            setattr(s, name, None if t is None else t.data_ptr())
        return s


def alloc_dispatch_out(T: int, H: int, E: int, k: int, N: int, payload: Optional[str],
                       device="cuda") -> DispatchBuffers:
    """Allocate the outputs of one dispatch (payload None: layout outputs only)."""
    R = T * k
    i32 = dict(dtype=torch.int32, device=device)
    recv = None if payload is None else torch.empty((R, H), dtype=TORCH_DTYPES[payload],
                                                    device=device)
    scales = (torch.empty((R, H // 128), dtype=torch.float32, device=device)
              if payload == "fp8_e4m3" else None)
    return DispatchBuffers(recv, scales, torch.empty(E, **i32), torch.empty(E + 1, **i32),
                           torch.empty(N, **i32), torch.empty(N + 1, **i32),
                           torch.empty(R, **i32), torch.empty(R, **i32))


def alloc_workspace(T: int, E: int, k: int, device="cuda") -> torch.Tensor:
    n = max(moe_dispatch_workspace_bytes(T, E, k), 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_dispatch_layout(topk_idx: torch.Tensor, E: int, n_ranks: int, out: DispatchBuffers,
                        workspace: torch.Tensor, stream=None) -> DispatchBuffers:
    T, k = topk_idx.shape
    _debug_check_ids("moe_dispatch_layout", topk_idx, E, stream)
    st = out.as_struct()
    _check("moe_dispatch_layout", load().moe_dispatch_layout(
        _ptr(topk_idx), T, k, E, n_ranks, ctypes.byref(st), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def moe_dispatch_pack(x: torch.Tensor, k: int, token_row: torch.Tensor, recv: torch.Tensor,
                      recv_scales: Optional[torch.Tensor] = None, stream=None):
    T, H = x.shape
    pd = _dtype_code(recv, fp8_ok=True)
    _check("moe_dispatch_pack", load().moe_dispatch_pack(
        _ptr(x), _dtype_code(x), T, H, k, _ptr(token_row), pd, _ptr(recv), _ptr(recv_scales),
        _stream(stream)))
    return recv, recv_scales


def moe_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, E: int, n_ranks: int,
                 out: DispatchBuffers, workspace: torch.Tensor, stream=None) -> DispatchBuffers:
    T, H = x.shape
    k = topk_idx.shape[1]
    _debug_check_ids("moe_dispatch", topk_idx, E, stream)
    st = out.as_struct()
    _check("moe_dispatch", load().moe_dispatch(
        _ptr(x), _dtype_code(x), T, H, _ptr(topk_idx), k, E, n_ranks,
        _dtype_code(out.recv, fp8_ok=True), ctypes.byref(st), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def moe_route_dispatch(logits: torch.Tensor, x: torch.Tensor, k: int, n_ranks: int,
                       out: DispatchBuffers, workspace: torch.Tensor,
                       topk_idx: Optional[torch.Tensor] = None,
                       topk_w: Optional[torch.Tensor] = None, stream=None):
    """Route (top-k ids and weights) and dispatch in one call; returns (topk_idx, topk_w, out)."""
    T, E = logits.shape
    H = x.shape[1]
    assert logits.dtype == torch.float32 and logits.is_contiguous() and x.shape[0] == T
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    st = out.as_struct()
    _check("moe_route_dispatch", load().moe_route_dispatch(
        _ptr(logits), _ptr(x), _dtype_code(x), T, H, E, k, n_ranks,
        _dtype_code(out.recv, fp8_ok=True), _ptr(topk_idx), _ptr(topk_w), ctypes.byref(st),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return topk_idx, topk_w, out


def moe_route_dispatch_noalloc(logits: torch.Tensor, x: torch.Tensor, k: int, n_ranks: int,
                               out: DispatchBuffers, topk_idx: Optional[torch.Tensor] = None,
                               topk_w: Optional[torch.Tensor] = None, stream=None):
    """moe_route_dispatch with the library's fixed device scratch instead of a workspace (the
    call allocates no device memory); returns (topk_idx, topk_w, out)."""
    T, E = logits.shape
    H = x.shape[1]
    assert logits.dtype == torch.float32 and logits.is_contiguous() and x.shape[0] == T
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    st = out.as_struct()
    _check("moe_route_dispatch_noalloc", load().moe_route_dispatch_noalloc(
        _ptr(logits), _ptr(x), _dtype_code(x), T, H, E, k, n_ranks,
        _dtype_code(out.recv, fp8_ok=True), _ptr(topk_idx), _ptr(topk_w), ctypes.byref(st),
        _stream(stream)))
    return topk_idx, topk_w, out


def moe_combine(y: torch.Tensor, token_row: torch.Tensor, topk_w: torch.Tensor,
                out: torch.Tensor, stream=None) -> torch.Tensor:
    T, k = topk_w.shape
    H = y.shape[1]
    _check("moe_combine", load().moe_combine(
        _ptr(y), _dtype_code(y), T, H, k, _ptr(token_row), _ptr(topk_w), _ptr(out),
        _dtype_code(out), _stream(stream)))
    return out


# ------------------------------------------------------------------------------------------------
# Expert parallelism over S sources and N ranks on one GPU (see include/moe_route.h).

def moe_ep_capacity(T: int, E: int, k: int, n_ranks: int) -> int:
    return int(load().moe_ep_capacity(T, E, k, n_ranks))


def moe_ep_send(x: torch.Tensor, topk_idx: torch.Tensor, E: int, n_ranks: int, source: int,
                n_sources: int, cap: int, regions: torch.Tensor, region_counts: torch.Tensor,
                send_row: torch.Tensor, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Sender half of dispatch for one source; fills its regions, counts and send_row."""
    T, H = x.shape
    k = topk_idx.shape[1]
    _debug_check_ids("moe_ep_send", topk_idx, E, stream)
    _check("moe_ep_send", load().moe_ep_send(
        _ptr(x), _dtype_code(x), T, H, _ptr(topk_idx), k, E, n_ranks, source, n_sources, cap,
        _ptr(regions), _ptr(region_counts), _ptr(send_row), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return send_row


def moe_ep_recv(regions: torch.Tensor, E: int, n_ranks: int, rank: int, n_sources: int, cap: int,
                region_counts: torch.Tensor, grouped: torch.Tensor, expert_counts: torch.Tensor,
                expert_offsets: torch.Tensor, grouped_src: torch.Tensor, stream=None):
    """Receiver half of dispatch for one rank: grouped rows, counts, offsets, source rows."""
    H = regions.shape[1]
    _check("moe_ep_recv", load().moe_ep_recv(
        _ptr(regions), _dtype_code(regions), H, E, n_ranks, rank, n_sources, cap,
        _ptr(region_counts), _ptr(grouped), _ptr(expert_counts), _ptr(expert_offsets),
        _ptr(grouped_src), _stream(stream)))
    return grouped


def moe_ep_return(y_grouped: torch.Tensor, E: int, n_ranks: int, n_sources: int, cap: int,
                  grouped_src: torch.Tensor, expert_offsets: torch.Tensor, returns: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """Receiver half of combine: expert outputs back to their region rows."""
    H = y_grouped.shape[1]
    _check("moe_ep_return", load().moe_ep_return(
        _ptr(y_grouped), _dtype_code(y_grouped), H, E, n_ranks, n_sources, cap, _ptr(grouped_src),
        _ptr(expert_offsets), _ptr(returns), _stream(stream)))
    return returns


def moe_ep_combine(returns: torch.Tensor, send_row: torch.Tensor, topk_w: torch.Tensor,
                   out: torch.Tensor, stream=None) -> torch.Tensor:
    """Sender half of combine for one source: weighted sum over its returned rows."""
    T, k = topk_w.shape
    H = returns.shape[1]
    _check("moe_ep_combine", load().moe_ep_combine(
        _ptr(returns), _dtype_code(returns), T, H, k, _ptr(send_row), _ptr(topk_w),
        returns.shape[0], _ptr(out), _dtype_code(out), _stream(stream)))
    return out


def moe_ep_partial_rows(topk_idx: torch.Tensor, E: int, n_ranks: int, source: int,
                        n_sources: int, pcap: int, part_row: torch.Tensor,
                        part_counts: torch.Tensor, stream=None) -> torch.Tensor:
    """Partial-row layout of one source: part_row [T, N], part_counts column `source`."""
    T, k = topk_idx.shape
    _check("moe_ep_partial_rows", load().moe_ep_partial_rows(
        _ptr(topk_idx), T, k, E, n_ranks, source, n_sources, pcap, _ptr(part_row),
        _ptr(part_counts), _stream(stream)))
    return part_row


def moe_ep_reduce(y_grouped: torch.Tensor, E: int, n_ranks: int, rank: int, n_sources: int,
                  cap: int, grouped_src: torch.Tensor, topk_idx: torch.Tensor,
                  topk_w: torch.Tensor, send_row: torch.Tensor, part_row: torch.Tensor, pcap: int,
                  partials: torch.Tensor, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Expert side of the pre-reduced combine for one rank (source tables stacked)."""
    H = y_grouped.shape[1]
    TT, k = topk_idx.shape
    _check("moe_ep_reduce", load().moe_ep_reduce(
        _ptr(y_grouped), _dtype_code(y_grouped), H, E, n_ranks, rank, n_sources, cap,
        _ptr(grouped_src), TT // n_sources, k, _ptr(topk_idx), _ptr(topk_w), _ptr(send_row),
        _ptr(part_row), pcap, _ptr(partials), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return partials


def moe_ep_reduce_workspace(n_sources: int, cap: int, device="cuda") -> torch.Tensor:
    n = max(int(load().moe_ep_reduce_workspace_bytes(n_sources, cap)), 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_ep_combine_reduced(partials: torch.Tensor, part_row: torch.Tensor, out: torch.Tensor,
                           stream=None) -> torch.Tensor:
    """Source side of the pre-reduced combine: a token's partial rows added in rank order."""
    T, N = part_row.shape
    H = partials.shape[1]
    _check("moe_ep_combine_reduced", load().moe_ep_combine_reduced(
        _ptr(partials), _dtype_code(partials), T, H, N, _ptr(part_row), partials.shape[0],
        _ptr(out), _dtype_code(out), _stream(stream)))
    return out


# ------------------------------------------------------------------------------------------------
# Router training and the experts' product in 8-bit integers (see include/moe_layer.h). These calls
# check every tensor (device, type, shape, density) before the library sees its pointer, and run
# on the device of their tensors whichever one is current.

def _arg(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """Address of a tensor that is what the call needs; raises what is wrong with it otherwise.
    `dtype`: one, or a tuple to choose from."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.device == device and
            (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)) and
            t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor is needed, got {type(t).__name__}")
    dtypes = dtype if type(dtype) is tuple else (dtype,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, needs {' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, needs {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the call is on {device}")
    raise ValueError(f"{name}: not contiguous")


def _opt(name: str, t: Optional[torch.Tensor], dtype, shape, device) -> Optional[int]:
    return None if t is None else _arg(name, t, dtype, shape, device)


_MOST = 2 ** 31 - 1                   # the library's sizes are int32; ctypes would pass on low bits


def _too_large(name: str, *sizes: int) -> None:
    raise ValueError(f"{name}: size {max(sizes)}, needs at most {_MOST}")


def _matrix(name: str, t: torch.Tensor):
    """Device, rows and columns of a call, from its main input."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{name}: a 2-d tensor is needed")
    rows, cols = t.shape
    if rows > _MOST or cols > _MOST:
        _too_large(name, rows, cols)
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, needs a GPU")
    return t.device, rows, cols


def _empty(shape, dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory for a call on `stream`, from that stream's pool: what was freed on another stream may
    still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = (torch.cuda.ExternalStream(raw, device=device) if raw
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_MASKS = (torch.bool, torch.uint8)
_WIDE = (torch.bfloat16, torch.float32)


def _enqueue(fn: str, device: torch.device, stream, *args) -> None:
    """Call a library function on `device`, on `stream` or the device's current stream. (The raw
    calls below cost a tenth of torch.cuda.current_stream() and torch.cuda.device(), which took
    more host time than the launch.)"""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == device.index:
        status = getattr(_lib or load(), fn)(*args, raw)
    else:
        with torch.cuda.device(device):
            status = getattr(_lib or load(), fn)(*args, raw)
    if status != MOE_OK:
        raise MoeError(fn, status)


@functools.lru_cache(maxsize=1024)
def moe_balance_workspace_bytes(T: int, E: int, n_seqs: int = 1) -> int:
    if max(T, E, n_seqs) > _MOST:
        _too_large("T, E, n_seqs", T, E, n_seqs)
    return int(load().moe_balance_workspace_bytes(T, E, n_seqs))


def alloc_balance_workspace(T: int, E: int, n_seqs: int = 1, device="cuda") -> torch.Tensor:
    n = max(moe_balance_workspace_bytes(T, E, n_seqs), 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, alpha: float, n_seqs: int = 1,
                     token_mask: Optional[torch.Tensor] = None,
                     loss: Optional[torch.Tensor] = None,
                     expert_counts: Optional[torch.Tensor] = None,
                     prob_sums: Optional[torch.Tensor] = None,
                     seq_tokens: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Balance loss of the router; returns (loss [1], expert_counts [S,E], prob_sums [S,E],
    seq_tokens [S]). token_mask [T] bool or uint8: False marks padding. Without a workspace one
    is allocated for the call."""
    dev, T, E = _matrix("logits", logits)
    k = topk_idx.shape[-1]
    n_seqs = int(n_seqs)
    if k > _MOST or n_seqs > _MOST:
        _too_large("topk_idx" if k > _MOST else "n_seqs", k, n_seqs)
    if n_seqs < 1 or T % n_seqs:
        raise ValueError(f"n_seqs: {n_seqs} sequences do not divide {T} tokens")
    if loss is None:
        loss = _empty((1,), torch.float32, dev, stream)
    if expert_counts is None:
        expert_counts = _empty((n_seqs, E), torch.int32, dev, stream)
    if prob_sums is None:
        prob_sums = _empty((n_seqs, E), torch.float32, dev, stream)
    if seq_tokens is None:
        seq_tokens = _empty((n_seqs,), torch.int32, dev, stream)
    if workspace is None:
        workspace = _empty((max(moe_balance_workspace_bytes(T, E, n_seqs), 1),), torch.uint8, dev,
                           stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: needs contiguous memory on {dev}")
    _enqueue("moe_balance_loss", dev, stream,
             _arg("logits", logits, torch.float32, (T, E), dev),
             _arg("topk_idx", topk_idx, torch.int32, (T, k), dev),
             _opt("token_mask", token_mask, _MASKS, (T,), dev), T, E, k, n_seqs, float(alpha),
             _arg("loss", loss, torch.float32, (1,), dev),
             _arg("expert_counts", expert_counts, torch.int32, (n_seqs, E), dev),
             _arg("prob_sums", prob_sums, torch.float32, (n_seqs, E), dev),
             _arg("seq_tokens", seq_tokens, torch.int32, (n_seqs,), dev),
             workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return loss, expert_counts, prob_sums, seq_tokens


def moe_route_grad(logits: torch.Tensor, topk_idx: torch.Tensor,
                   topk_w: Optional[torch.Tensor] = None, dtopk_w: Optional[torch.Tensor] = None,
                   token_mask: Optional[torch.Tensor] = None,
                   expert_counts: Optional[torch.Tensor] = None,
                   seq_tokens: Optional[torch.Tensor] = None,
                   dloss: Optional[torch.Tensor] = None, alpha: float = 0.0, n_seqs: int = 1,
                   dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the router's logits [T,E]: of the balance loss (given expert_counts and
    seq_tokens), of the routing weights (given topk_w and dtopk_w), or their sum."""
    dev, T, E = _matrix("logits", logits)
    k = topk_idx.shape[-1]
    n_seqs = int(n_seqs)
    if k > _MOST or n_seqs > _MOST:
        _too_large("topk_idx" if k > _MOST else "n_seqs", k, n_seqs)
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, dev, stream)
    _enqueue("moe_route_grad", dev, stream,
             _arg("logits", logits, torch.float32, (T, E), dev),
             _arg("topk_idx", topk_idx, torch.int32, (T, k), dev),
             _opt("topk_w", topk_w, torch.float32, (T, k), dev),
             _opt("dtopk_w", dtopk_w, torch.float32, (T, k), dev),
             _opt("token_mask", token_mask, _MASKS, (T,), dev),
             _opt("expert_counts", expert_counts, torch.int32, (n_seqs, E), dev),
             _opt("seq_tokens", seq_tokens, torch.int32, (n_seqs,), dev),
             _opt("dloss", dloss, torch.float32, (1,), dev), T, E, k, n_seqs, float(alpha),
             _arg("dlogits", dlogits, torch.float32, (T, E), dev))
    return dlogits


def moe_quant_rows(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None, n_rows: Optional[torch.Tensor] = None,
                   stream=None):
    """8-bit rows: (q int8 [R,H], scale fp32 [R]) with x about q * scale. n_rows (int32 [1] on
    the device): only the first n_rows rows are quantised."""
    dev, R, H = _matrix("x", x)
    if q is None:
        q = _empty((R, H), torch.int8, dev, stream)
    if scale is None:
        scale = _empty((R,), torch.float32, dev, stream)
    _enqueue("moe_quant_rows", dev, stream, _arg("x", x, _WIDE, (R, H), dev), _dtype_code(x), R, H,
             _opt("n_rows", n_rows, torch.int32, (1,), dev), _arg("q", q, torch.int8, (R, H), dev),
             _arg("scale", scale, torch.float32, (R,), dev))
    return q, scale


def moe_expert_matmul_i8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor,
                         w_scale: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None,
                         row_token: Optional[torch.Tensor] = None, act: str = "none",
                         out: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The experts' product of 8-bit rows a [A,K] (scale [A]) with 8-bit weights w [E,N,K] (scale
    [E,N]; act "swiglu": [E,2N,K], gate channels first); returns out [R,N] in out's type or
    out_dtype. Row r of expert e (expert_offsets [E+1]) reads row row_token[r] of a, or row r
    without row_token. Without expert_offsets E must be 1: a plain product."""
    dev, A, K = _matrix("a", a)
    if act not in ACT_CODES:
        raise ValueError(f"act: {act!r}, needs one of {sorted(ACT_CODES)}")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w: a 3-d tensor is needed")
    E, n_w, _ = w.shape
    if E > _MOST or n_w > _MOST:
        _too_large("w", E, n_w)
    if act == "swiglu" and n_w % 2:
        raise ValueError(f"w: {n_w} channels do not split into gate and up")
    N = n_w // 2 if act == "swiglu" else n_w
    R = A if row_token is None else row_token.numel()
    if R > _MOST:
        _too_large("row_token", R)
    if out is None:
        out = _empty((R, N), out_dtype, dev, stream)
    _enqueue("moe_expert_matmul_i8", dev, stream, _arg("a", a, torch.int8, (A, K), dev),
             _arg("a_scale", a_scale, torch.float32, (A,), dev), A,
             _opt("row_token", row_token, torch.int32, (R,), dev),
             _arg("w", w, torch.int8, (E, n_w, K), dev),
             _arg("w_scale", w_scale, torch.float32, (E, n_w), dev),
             _opt("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev), R, E, N, K,
             ACT_CODES[act], _arg("out", out, _WIDE, (R, N), dev), _dtype_code(out))
    return out


# ------------------------------------------------------------------------------------------------
# Scored routing, the experts' product in bf16, and their gradients (see include/moe_block.h), with
# the same checks.

def moe_route_scored(logits: torch.Tensor, k: int, score: str = "softmax",
                     bias: Optional[torch.Tensor] = None, n_groups: int = 1, topk_groups: int = 1,
                     group_top: int = 2, renormalize: bool = True, scale: float = 1.0,
                     topk_idx: Optional[torch.Tensor] = None,
                     topk_w: Optional[torch.Tensor] = None, stream=None):
    """Scored routing of logits [T,E]: (expert ids int32 [T,k], weights fp32 [T,k]). Scores are
    "softmax" or "sigmoid"; bias [E] takes part in the choice only; with n_groups > 1 the experts of
    the topk_groups groups with the largest sums of their group_top best are chosen from. Weights are
    the chosen scores, over their sum if renormalize, times scale."""
    dev, T, E = _matrix("logits", logits)
    if score not in SCORE_CODES:
        raise ValueError(f"score: {score!r}, needs one of {sorted(SCORE_CODES)}")
    k, n_groups, topk_groups, group_top = int(k), int(n_groups), int(topk_groups), int(group_top)
    if max(k, n_groups, topk_groups, group_top) > _MOST or min(k, n_groups, topk_groups, group_top) < 0:
        raise ValueError(f"k, n_groups, topk_groups, group_top: {k}, {n_groups}, {topk_groups}, "
                         f"{group_top}")
    if topk_idx is None:
        topk_idx = _empty((T, k), torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _empty((T, k), torch.float32, dev, stream)
    _enqueue("moe_route_scored", dev, stream, _arg("logits", logits, torch.float32, (T, E), dev),
             _opt("bias", bias, torch.float32, (E,), dev), T, E, k, SCORE_CODES[score], n_groups,
             topk_groups, group_top, int(bool(renormalize)), float(scale),
             _arg("topk_idx", topk_idx, torch.int32, (T, k), dev),
             _arg("topk_w", topk_w, torch.float32, (T, k), dev))
    return topk_idx, topk_w


def moe_route_scored_grad(logits: torch.Tensor, topk_idx: torch.Tensor, dtopk_w: torch.Tensor,
                          score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                          add: Optional[torch.Tensor] = None,
                          dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits [T,E] through the weights of moe_route_scored, plus add [T,E] (which may
    be dlogits itself)."""
    dev, T, E = _matrix("logits", logits)
    if score not in SCORE_CODES:
        raise ValueError(f"score: {score!r}, needs one of {sorted(SCORE_CODES)}")
    k = topk_idx.shape[-1]
    if k > _MOST:
        _too_large("topk_idx", k)
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, dev, stream)
    _enqueue("moe_route_scored_grad", dev, stream,
             _arg("logits", logits, torch.float32, (T, E), dev),
             _arg("topk_idx", topk_idx, torch.int32, (T, k), dev),
             _arg("dtopk_w", dtopk_w, torch.float32, (T, k), dev),
             _opt("add", add, torch.float32, (T, E), dev), T, E, k, SCORE_CODES[score],
             int(bool(renormalize)), float(scale),
             _arg("dlogits", dlogits, torch.float32, (T, E), dev))
    return dlogits


def moe_bias_update(bias: torch.Tensor, expert_counts: torch.Tensor, rate: float,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Balance biases [L,E] (or [E]) after a step: plus rate where an expert's count is below its
    layer's mean, minus rate where it is above. out may be bias itself."""
    if not isinstance(bias, torch.Tensor) or bias.dim() not in (1, 2):
        raise TypeError("bias: a 1-d or 2-d tensor is needed")
    dev, L, E = _matrix("bias", bias if bias.dim() == 2 else bias[None])
    if out is None:
        out = _empty(bias.shape, torch.float32, dev, stream)
    _enqueue("moe_bias_update", dev, stream, _arg("bias", bias, torch.float32, bias.shape, dev),
             _arg("expert_counts", expert_counts, torch.int32, bias.shape, dev), L, E, float(rate),
             _arg("out", out, torch.float32, bias.shape, dev))
    return out


def _wanted(want, names) -> tuple:
    """What a call is to compute: one of the names, or several of them."""
    want = (want,) if isinstance(want, str) else tuple(want)
    if not want or len(set(want)) != len(want) or not set(want) <= set(names):
        raise ValueError(f"want: {want!r}, needs some of {', '.join(map(repr, names))}, each once")
    return want


def moe_combine_grad(dout: torch.Tensor, y: Optional[torch.Tensor], token_row: torch.Tensor,
                     topk_w: torch.Tensor, dy: Optional[torch.Tensor] = None,
                     dtopk_w: Optional[torch.Tensor] = None, stream=None, want=None):
    """Gradient of moe_combine from dout [T,H]: (dy [T*k,H], dtopk_w [T,k]). `want` names those to
    compute, "dy" or "dtopk_w"; the other is None. By default both, or without y only dy (in its own
    type, bf16 if it is not given)."""
    dev, T, H = _matrix("dout", dout)
    k = topk_w.shape[-1]
    if k > _MOST or T * k > _MOST:
        _too_large("topk_w", k, T * k)
    with_dy, with_dw = True, y is not None
    if want is not None:
        want = _wanted(want, ("dy", "dtopk_w"))
        with_dy, with_dw = "dy" in want, "dtopk_w" in want
    if y is None and (with_dw or dtopk_w is not None):
        raise ValueError("dtopk_w: needs y")
    wide = y if y is not None else dy
    y_dtype = torch.bfloat16 if wide is None else wide.dtype
    if dy is None:
        dy = _empty((T * k, H), y_dtype, dev, stream) if with_dy else None
    elif not with_dy:
        raise ValueError("dy: given, and not in want")
    if dtopk_w is None:
        dtopk_w = _empty((T, k), torch.float32, dev, stream) if with_dw else None
    elif not with_dw:
        raise ValueError("dtopk_w: given, and not in want")
    _enqueue("moe_combine_grad", dev, stream, _arg("dout", dout, _WIDE, (T, H), dev),
             _dtype_code(dout), _opt("y", y, _WIDE, (T * k, H), dev), _dtype_code(y if dy is None else dy),
             _arg("token_row", token_row, torch.int32, (T * k,), dev),
             _arg("topk_w", topk_w, torch.float32, (T, k), dev), T, H, k,
             _opt("dy", dy, y_dtype, (T * k, H), dev),
             _opt("dtopk_w", dtopk_w, torch.float32, (T, k), dev))
    return dy, dtopk_w


def _product_sizes(w: torch.Tensor, act: str, R: int):
    if act not in MAT_ACT_CODES:
        raise ValueError(f"act: {act!r}, needs one of {sorted(MAT_ACT_CODES)}")
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w: a 3-d tensor is needed")
    if R > _MOST:
        _too_large("row_token", R)
    E, n_w, K = w.shape
    if max(E, n_w, K) > _MOST:
        _too_large("w", E, n_w, K)
    return E, n_w, K


@functools.lru_cache(maxsize=1024)
def moe_expert_matmul_workspace_bytes(R: int, E: int, channels: int, K: int) -> int:
    if max(R, E, channels, K) > _MOST:
        _too_large("R, E, channels, K", R, E, channels, K)
    return int(load().moe_expert_matmul_workspace_bytes(R, E, channels, K))


def alloc_expert_matmul_workspace(R: int, E: int, channels: int, K: int, device="cuda") -> torch.Tensor:
    n = max(moe_expert_matmul_workspace_bytes(R, E, channels, K), 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_expert_matmul(a: torch.Tensor, w: torch.Tensor,
                      expert_offsets: Optional[torch.Tensor] = None,
                      row_token: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, act: str = "none",
                      residual: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' product of bf16 rows a [A,K] with bf16 weights w [E,N,K] (act "swiglu": [E,2N,K],
    gate channels first): act(a w^T + bias) + residual, out [R,N] in out's type or out_dtype. act is
    "none", "relu", "silu", "gelu" (tanh form) or "swiglu"; bias [E,N or 2N] fp32; residual [R,N] in
    out's type, it may be out; pre [R,N or 2N] bf16 gets the sums before the activation. Row r of expert
    e (expert_offsets [E+1]) reads row row_token[r] of a, or row r without row_token. Without
    expert_offsets E must be 1: a plain product. Sizes that need a workspace and get none have one
    allocated for the call."""
    dev, A, K = _matrix("a", a)
    R = A if row_token is None else row_token.numel()
    E, n_w, _ = _product_sizes(w, act, R)
    if act == "swiglu" and n_w % 2:
        raise ValueError(f"w: {n_w} channels do not split into gate and up")
    N = n_w // 2 if act == "swiglu" else n_w
    if out is None:
        out = _empty((R, N), out_dtype, dev, stream)
    if workspace is None:
        need = moe_expert_matmul_workspace_bytes(R, E, n_w, K)
        workspace = _empty((need,), torch.uint8, dev, stream) if need else None
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: needs contiguous memory on {dev}")
    _enqueue("moe_expert_matmul", dev, stream, _arg("a", a, torch.bfloat16, (A, K), dev), A,
             _opt("row_token", row_token, torch.int32, (R,), dev),
             _arg("w", w, torch.bfloat16, (E, n_w, K), dev),
             _opt("bias", bias, torch.float32, (E, n_w), dev),
             _opt("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev), R, E, N, K,
             MAT_ACT_CODES[act], _opt("residual", residual, out.dtype, (R, N), dev),
             _opt("pre", pre, torch.bfloat16, (R, n_w), dev),
             _arg("out", out, _WIDE, (R, N), dev), _dtype_code(out),
             None if workspace is None else workspace.data_ptr(),
             0 if workspace is None else workspace.numel() * workspace.element_size())
    return out


@functools.lru_cache(maxsize=1024)
def moe_matmul_grad_workspace_bytes(R: int, E: int, N: int, K: int) -> int:
    if max(R, E, N, K) > _MOST:
        _too_large("R, E, N, K", R, E, N, K)
    return int(load().moe_matmul_grad_workspace_bytes(R, E, N, K))


def alloc_matmul_grad_workspace(R: int, E: int, N: int, K: int, device="cuda") -> torch.Tensor:
    n = max(moe_matmul_grad_workspace_bytes(R, E, N, K), 1)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_expert_matmul_grad(dy: torch.Tensor, a: Optional[torch.Tensor], w: torch.Tensor,
                           expert_offsets: Optional[torch.Tensor] = None, want=("da", "dw"),
                           row_token: Optional[torch.Tensor] = None, act: str = "none",
                           pre: Optional[torch.Tensor] = None, da: Optional[torch.Tensor] = None,
                           dw: Optional[torch.Tensor] = None,
                           dbias: Optional[torch.Tensor] = None,
                           da_dtype: torch.dtype = torch.bfloat16,
                           dw_dtype: torch.dtype = torch.float32,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the product a w^T + bias from dy [R,N] bf16: a tuple of those that `want` names, in
    its order. "da" [R,K], one row for each row of dy (with row_token, moe_combine with weights of one
    adds up a token's); "dw" [E,N,K]; "dbias" [E,N] fp32. With an activation, a was act(pre) and da is
    the gradient of pre ([R,K]; "swiglu": pre and da [R,2K]). a may be None if only "da" is wanted and
    row_token is not given. Without a workspace one is allocated for the call."""
    dev, R, N = _matrix("dy", dy)
    E, _, K = _product_sizes(w, act, R)
    want = _wanted(want, ("da", "dw", "dbias"))
    if a is None and ("dw" in want or row_token is not None):
        raise ValueError("a: needed for 'dw', and with row_token")
    A = R if a is None else _matrix("a", a)[1]
    if "da" in want:
        n_a = 2 * K if act == "swiglu" else K
        if act != "none" and pre is None:
            raise ValueError(f"pre: needed for act {act!r}")
        if da is None:
            da = _empty((R, n_a), da_dtype, dev, stream)
        _arg("da", da, _WIDE, (R, n_a), dev)
        _opt("pre", pre, torch.bfloat16, (R, n_a), dev)
    else:
        da = None
    if "dw" in want:
        if dw is None:
            dw = _empty((E, N, K), dw_dtype, dev, stream)
        _arg("dw", dw, _WIDE, (E, N, K), dev)
    else:
        dw = None
    if "dbias" in want:
        if dbias is None:
            dbias = _empty((E, N), torch.float32, dev, stream)
        _arg("dbias", dbias, torch.float32, (E, N), dev)
    else:
        dbias = None
    if workspace is None:
        workspace = _empty((max(moe_matmul_grad_workspace_bytes(R, E, N, K), 1),), torch.uint8, dev,
                           stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: needs contiguous memory on {dev}")
    address = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    code = lambda t: MOE_F32 if t is None else _dtype_code(t)  # noqa: E731
    _enqueue("moe_expert_matmul_grad", dev, stream, _arg("dy", dy, torch.bfloat16, (R, N), dev),
             _opt("a", a, torch.bfloat16, (A, K), dev), A,
             _opt("row_token", row_token, torch.int32, (R,), dev),
             _arg("w", w, torch.bfloat16, (E, N, K), dev),
             _opt("expert_offsets", expert_offsets, torch.int32, (E + 1,), dev), R, E, N, K,
             MAT_ACT_CODES[act], address(pre), address(da), code(da), address(dw), code(dw),
             address(dbias), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    got = {"da": da, "dw": dw, "dbias": dbias}
    return tuple(got[name] for name in want)
