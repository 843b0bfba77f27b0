"""Python binding of the MI355X expert-parallel routing library (include/ep.h).

Argument marshalling only: each function checks dtypes, devices, shapes and
contiguity of PyTorch tensors, then calls the C entry point of the same name
in ``libcombine_ep_prepare_amd.so`` with raw device pointers and the current
HIP stream. Every step of the computation runs in the library's kernels.
There is no fallback: if the library is missing, importing the binding
raises.

The five routing ops follow the per-step calls of "Expert Parallelism: common C API
+ NCCL EP backend" (section "Per-step (allocation-free, CUDA-graph
capturable)"): prepare, dispatch, combine, dispatch_bwd and combine_bwd. The
experts' own work between dispatch and combine stands beside them: the grouped
linear, its backward and its 4-bit form, and the gated activation with its
backward; the norm in front of a layer, and the linear and activation in 8 bits
with scales; and the whole layer for a few tokens.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcombine_ep_prepare_amd.so")

EP_OK = 0
EP_ERR_NULL = 1
EP_ERR_SHAPE = 2
EP_ERR_ALIGN = 3
EP_ERR_HANDLE_SIZE = 4
EP_ERR_CAPACITY = 5
EP_ERR_DEVICE = 6
EP_ERR_HIP = 7
EP_ERR_SCRATCH = 8
EP_ERR_WORKSPACE = 9
PREPARE_STATIC_SCRATCH_BYTES = 4 << 20

STATUS_BAD_EXPERT = 1
STATUS_OVERFLOW = 2
STATUS_LAYOUT = 4

DTYPE_BF16 = 0
DTYPE_FP16 = 1
DTYPE_FP32 = 2
LAYOUT_NO_PAD_FILL = 1
LAYOUT_ZERO_TAIL = 4

SCALE_BLOCK = 128          # values of a row to one scale, in 8 bits
MAX_NORM_FEATURES = 16384
MAX_LAYER_ROUTES = 1024
E4M3 = torch.float8_e4m3fn  # the type of 8-bit values

# payload type code -> torch dtype of the rows
TORCH_DTYPE = {DTYPE_BF16: torch.bfloat16, DTYPE_FP16: torch.float16,
               DTYPE_FP32: torch.float32}
_CODE_OF = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32,
            "bf16": DTYPE_BF16, "fp16": DTYPE_FP16, "fp32": DTYPE_FP32}

ENTRY_POINTS = ("ep_recv_capacity_worst", "ep_handle_mem_size", "ep_handle_regions",
                "ep_prepare", "ep_prepare_static", "ep_dispatch",
                "ep_combine", "ep_dispatch_bwd", "ep_combine_bwd", "ep_combine_weighted",
                "ep_combine_weighted_bwd", "ep_grouped_linear", "ep_grouped_linear_bwd",
                "ep_grouped_linear_quant", "ep_swiglu", "ep_swiglu_bwd", "ep_rms_norm",
                "ep_rms_norm_bwd", "ep_rms_norm_bwd_workspace", "ep_swiglu_scaled",
                "ep_grouped_linear_scaled", "ep_expert_layer", "ep_expert_layer_workspace",
                "ep_read_status", "ep_status_str")


class Layout(C.Structure):
    """ep_layout_t. ``dtype`` is the payload type (a torch dtype, "bf16",
    "fp16", "fp32" or a DTYPE_* code); ``fill_pads=False`` sets
    LAYOUT_NO_PAD_FILL; ``zero_tail=True`` sets LAYOUT_ZERO_TAIL
    (expert-major outputs also get zeros in the rows past the live total)."""
    _fields_ = [("num_tokens", C.c_int64), ("topk", C.c_int32), ("num_experts", C.c_int32),
                ("alignment", C.c_int32), ("dtype", C.c_uint16), ("flags", C.c_uint16),
                ("hidden", C.c_int64), ("recv_capacity", C.c_int64)]

    def __init__(self, num_tokens, topk, num_experts, alignment, hidden, recv_capacity,
                 dtype=DTYPE_BF16, fill_pads=True, zero_tail=False):
        code = dtype if isinstance(dtype, int) else _CODE_OF[dtype]
        flags = (0 if fill_pads else LAYOUT_NO_PAD_FILL) | (LAYOUT_ZERO_TAIL if zero_tail else 0)
        super().__init__(num_tokens, topk, num_experts, alignment, code, flags, hidden,
                         recv_capacity)

    @property
    def payload_dtype(self) -> torch.dtype:
        """torch dtype of the payload rows (bfloat16 for an unknown code)."""
        return TORCH_DTYPE.get(self.dtype, torch.bfloat16)

    @property
    def T(self):
        return self.num_tokens

    @property
    def K(self):
        return self.topk

    @property
    def E(self):
        return self.num_experts

    @property
    def A(self):
        return self.alignment

    @property
    def H(self):
        return self.hidden

    @property
    def cap(self):
        return self.recv_capacity


class HandleRegions(C.Structure):
    """ep_handle_regions_t: byte offsets of the routing maps in a handle."""
    _fields_ = [("status", C.c_size_t), ("counts", C.c_size_t), ("offsets", C.c_size_t),
                ("slot", C.c_size_t), ("row_src", C.c_size_t), ("bytes", C.c_size_t),
                ("runs", C.c_size_t), ("maps_bytes", C.c_size_t),
                ("stream_live", C.c_size_t), ("run_units", C.c_size_t),
                ("run_list_entries", C.c_size_t)]


class EpError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_str(code)} (ep_status_t {code})")
        self.code = code


def _load_library(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
            "g.build()'` (hipcc, gfx950)")
    lib = C.CDLL(path)
    i64, i32, vp, sz = C.c_int64, C.c_int32, C.c_void_p, C.c_size_t
    lp = C.POINTER(Layout)
    lib.ep_recv_capacity_worst.argtypes = [i64, i32, i32, i32]
    lib.ep_recv_capacity_worst.restype = i64
    lib.ep_handle_mem_size.argtypes = [lp]
    lib.ep_handle_mem_size.restype = sz
    lib.ep_handle_regions.argtypes = [lp, C.POINTER(HandleRegions)]
    lib.ep_handle_regions.restype = C.c_int
    lib.ep_prepare.argtypes = [lp, vp, vp, vp, vp, sz, vp]
    lib.ep_prepare_static.argtypes = [lp, vp, vp, vp, vp, sz, vp]
    lib.ep_dispatch.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp]
    lib.ep_combine.argtypes = [lp, vp, sz, vp, vp, vp]
    lib.ep_dispatch_bwd.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp]
    lib.ep_combine_bwd.argtypes = [lp, vp, sz, vp, vp, vp]
    lib.ep_combine_weighted.argtypes = [lp, vp, sz, vp, vp, vp, vp]
    lib.ep_combine_weighted_bwd.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp, vp]
    lib.ep_read_status.argtypes = [vp, C.POINTER(C.c_uint32), vp]
    lib.ep_grouped_linear.argtypes = [lp, vp, sz, vp, vp, vp, i64, vp]
    lib.ep_grouped_linear_bwd.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp, i64, vp]
    lib.ep_grouped_linear_quant.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp, i64, i32, vp]
    lib.ep_swiglu.argtypes = [lp, vp, sz, vp, vp, vp]
    lib.ep_swiglu_bwd.argtypes = [lp, vp, sz, vp, vp, vp, vp]
    lib.ep_rms_norm.argtypes = [lp, vp, vp, vp, C.c_float, vp, vp, vp, vp, vp]
    lib.ep_rms_norm_bwd_workspace.argtypes = [lp]
    lib.ep_rms_norm_bwd_workspace.restype = sz
    lib.ep_rms_norm_bwd.argtypes = [lp, vp, vp, vp, vp, C.c_float, vp, vp, vp, sz, vp]
    lib.ep_swiglu_scaled.argtypes = [lp, vp, sz, vp, vp, vp, vp]
    lib.ep_grouped_linear_scaled.argtypes = [lp, vp, sz, vp, vp, vp, vp, vp, i64, vp]
    lib.ep_expert_layer_workspace.argtypes = [lp, i64]
    lib.ep_expert_layer_workspace.restype = sz
    lib.ep_expert_layer.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, sz, vp]
    for name in ("ep_prepare", "ep_prepare_static", "ep_dispatch", "ep_combine",
                 "ep_dispatch_bwd",
                 "ep_combine_bwd", "ep_combine_weighted", "ep_combine_weighted_bwd",
                 "ep_grouped_linear", "ep_grouped_linear_bwd", "ep_grouped_linear_quant",
                 "ep_swiglu", "ep_swiglu_bwd", "ep_rms_norm", "ep_rms_norm_bwd",
                 "ep_swiglu_scaled", "ep_grouped_linear_scaled", "ep_expert_layer",
                 "ep_read_status"):
        getattr(lib, name).restype = C.c_int
    lib.ep_status_str.argtypes = [C.c_int]
    lib.ep_status_str.restype = C.c_char_p
    return lib


lib = _load_library()


def status_str(code: int) -> str:
    return lib.ep_status_str(code).decode()


def _check(code: int, what: str):
    if code != EP_OK:
        raise EpError(code, what)


def recv_capacity_worst(T: int, K: int, E: int, A: int) -> int:
    return int(lib.ep_recv_capacity_worst(T, K, E, A))


def handle_mem_size(layout: Layout) -> int:
    return int(lib.ep_handle_mem_size(C.byref(layout)))


def handle_regions(layout: Layout) -> HandleRegions:
    out = HandleRegions()
    _check(lib.ep_handle_regions(C.byref(layout), C.byref(out)), "ep_handle_regions")
    return out


def handle_maps(layout: Layout, handle: torch.Tensor) -> dict:
    """Views of the routing maps inside a prepared handle (no copy)."""
    r = handle_regions(layout)

    def view(off, n, dtype):
        return handle[off:off + 4 * n].view(dtype)

    return {
        "status": view(r.status, 1, torch.int32),
        "counts": view(r.counts, layout.E, torch.int32),
        "offsets": view(r.offsets, layout.E + 1, torch.int32),
        "slot": view(r.slot, layout.T * layout.K, torch.int32),
        "row_src": view(r.row_src, layout.cap, torch.int32),
        "runs": view(r.runs, 8 * 2 * r.run_list_entries, torch.int32).view(8, -1, 2),
        "stream_live": view(r.stream_live, 8, torch.int32),
        "run_units": view(r.run_units, 1, torch.int32),
    }


# The checks below run for every tensor of every call, and the small calls of
# decoding take about as long on the host as on the GPU: plain ints for
# pointers (the argument types convert them), one query each for a tensor's
# device and the current one, the latter without torch.cuda's check that there
# is a context: a tensor on a GPU has one.

def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _need(t: Optional[torch.Tensor], name: str, dtype, shape=None, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    device = t.get_device()
    if device < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}; the library runs on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_all(required, optional=()):
    """_need for several (tensor, name, dtype, shape), those of `optional` perhaps
    None: one query for the current device, and what is amiss said by _need."""
    current = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else 0
    for t, name, dtype, shape in required:
        if (t is None or t.dtype is not dtype or t.get_device() != current
                or not t.is_contiguous() or t.shape != shape):
            _need(t, name, dtype, shape)
    for t, name, dtype, shape in optional:
        if t is not None and (t.dtype is not dtype or t.get_device() != current
                              or not t.is_contiguous() or t.shape != shape):
            _need(t, name, dtype, shape)


def _both(name_a: str, a, name_b: str, b):
    if (a is None) != (b is None):
        raise ValueError(f"{name_a} and {name_b} go together")


def _out_features(weight: torch.Tensor) -> int:
    if weight.dim() != 3:
        raise ValueError(f"weight must have shape (E, N, H), got {tuple(weight.shape)}")
    return weight.shape[1]


def new_handle(layout: Layout, device=None) -> torch.Tensor:
    """Allocate the caller-owned handle memory for ``layout`` (uint8 tensor)."""
    n = handle_mem_size(layout)
    if n == 0:
        raise ValueError("invalid layout")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def prepare(layout: Layout, topk_idx: torch.Tensor, token_counts: torch.Tensor,
            handle: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None,
            stream=None):
    _need(topk_idx, "topk_idx", torch.int64, (layout.T, layout.K))
    _need(token_counts, "token_counts", torch.int32, (layout.E,))
    _need(expert_offsets, "expert_offsets", torch.int32, (layout.E + 1,), allow_none=True)
    _need(handle, "handle", torch.uint8)
    _check(lib.ep_prepare(C.byref(layout), _ptr(topk_idx), _ptr(token_counts),
                          _ptr(expert_offsets), _ptr(handle), handle.numel(),
                          _stream(stream)), "ep_prepare")


def prepare_static(layout: Layout, topk_idx: torch.Tensor, token_counts: torch.Tensor,
                   handle: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None,
                   stream=None):
    """prepare with its scratch in the library's static device array: the
    handle needs only ``handle_regions(layout).maps_bytes`` bytes. Calls that
    overlap on one device race."""
    _need(topk_idx, "topk_idx", torch.int64, (layout.T, layout.K))
    _need(token_counts, "token_counts", torch.int32, (layout.E,))
    _need(expert_offsets, "expert_offsets", torch.int32, (layout.E + 1,), allow_none=True)
    _need(handle, "handle", torch.uint8)
    _check(lib.ep_prepare_static(C.byref(layout), _ptr(topk_idx), _ptr(token_counts),
                                 _ptr(expert_offsets), _ptr(handle), handle.numel(),
                                 _stream(stream)), "ep_prepare_static")


def dispatch(layout: Layout, handle: torch.Tensor, tokens: torch.Tensor,
             topk_weights: Optional[torch.Tensor], recv_tokens: torch.Tensor,
             recv_topk_weights: Optional[torch.Tensor] = None, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(tokens, "tokens", layout.payload_dtype, (layout.T, layout.H))
    _need(topk_weights, "topk_weights", torch.float32, (layout.T, layout.K), allow_none=True)
    _need(recv_tokens, "recv_tokens", layout.payload_dtype, (layout.cap, layout.H))
    _need(recv_topk_weights, "recv_topk_weights", torch.float32, (layout.cap,),
          allow_none=True)
    _check(lib.ep_dispatch(C.byref(layout), _ptr(handle), handle.numel(), _ptr(tokens),
                           _ptr(topk_weights), _ptr(recv_tokens), _ptr(recv_topk_weights),
                           _stream(stream)), "ep_dispatch")


def combine(layout: Layout, handle: torch.Tensor, expert_out: torch.Tensor,
            result: torch.Tensor, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(expert_out, "expert_out", layout.payload_dtype, (layout.cap, layout.H))
    _need(result, "result", layout.payload_dtype, (layout.T, layout.H))
    _check(lib.ep_combine(C.byref(layout), _ptr(handle), handle.numel(), _ptr(expert_out),
                          _ptr(result), _stream(stream)), "ep_combine")


def dispatch_bwd(layout: Layout, handle: torch.Tensor, grad: torch.Tensor,
                 g_recv_topk_weights: Optional[torch.Tensor], grad_tokens: torch.Tensor,
                 grad_topk_weights: Optional[torch.Tensor] = None, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(grad, "grad", layout.payload_dtype, (layout.cap, layout.H))
    _need(g_recv_topk_weights, "g_recv_topk_weights", torch.float32, (layout.cap,),
          allow_none=True)
    _need(grad_tokens, "grad_tokens", layout.payload_dtype, (layout.T, layout.H))
    _need(grad_topk_weights, "grad_topk_weights", torch.float32, (layout.T, layout.K),
          allow_none=True)
    _check(lib.ep_dispatch_bwd(C.byref(layout), _ptr(handle), handle.numel(), _ptr(grad),
                               _ptr(g_recv_topk_weights), _ptr(grad_tokens),
                               _ptr(grad_topk_weights), _stream(stream)), "ep_dispatch_bwd")


def combine_bwd(layout: Layout, handle: torch.Tensor, grad: torch.Tensor,
                grad_expert_out: torch.Tensor, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(grad, "grad", layout.payload_dtype, (layout.T, layout.H))
    _need(grad_expert_out, "grad_expert_out", layout.payload_dtype, (layout.cap, layout.H))
    _check(lib.ep_combine_bwd(C.byref(layout), _ptr(handle), handle.numel(), _ptr(grad),
                              _ptr(grad_expert_out), _stream(stream)), "ep_combine_bwd")


def combine_weighted(layout: Layout, handle: torch.Tensor, expert_out: torch.Tensor,
                     recv_topk_weights: torch.Tensor, result: torch.Tensor, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(expert_out, "expert_out", layout.payload_dtype, (layout.cap, layout.H))
    _need(recv_topk_weights, "recv_topk_weights", torch.float32, (layout.cap,))
    _need(result, "result", layout.payload_dtype, (layout.T, layout.H))
    _check(lib.ep_combine_weighted(C.byref(layout), _ptr(handle), handle.numel(),
                                   _ptr(expert_out), _ptr(recv_topk_weights), _ptr(result),
                                   _stream(stream)), "ep_combine_weighted")


def combine_weighted_bwd(layout: Layout, handle: torch.Tensor, grad: torch.Tensor,
                         expert_out: Optional[torch.Tensor], recv_topk_weights: torch.Tensor,
                         grad_expert_out: torch.Tensor,
                         grad_recv_topk_weights: Optional[torch.Tensor] = None, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(grad, "grad", layout.payload_dtype, (layout.T, layout.H))
    _need(expert_out, "expert_out", layout.payload_dtype, (layout.cap, layout.H), allow_none=True)
    _need(recv_topk_weights, "recv_topk_weights", torch.float32, (layout.cap,))
    _need(grad_expert_out, "grad_expert_out", layout.payload_dtype, (layout.cap, layout.H))
    _need(grad_recv_topk_weights, "grad_recv_topk_weights", torch.float32, (layout.cap,),
          allow_none=True)
    _check(lib.ep_combine_weighted_bwd(C.byref(layout), _ptr(handle), handle.numel(),
                                       _ptr(grad), _ptr(expert_out), _ptr(recv_topk_weights),
                                       _ptr(grad_expert_out), _ptr(grad_recv_topk_weights),
                                       _stream(stream)), "ep_combine_weighted_bwd")


def grouped_linear(layout: Layout, handle: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                   out: torch.Tensor, stream=None):
    """out [cap,N] = each live row of x [cap,H] through its expert's weight [E,N,H]."""
    N = _out_features(weight)
    _need(handle, "handle", torch.uint8)
    _need(x, "x", layout.payload_dtype, (layout.cap, layout.H))
    _need(weight, "weight", layout.payload_dtype, (layout.E, N, layout.H))
    _need(out, "out", layout.payload_dtype, (layout.cap, N))
    _check(lib.ep_grouped_linear(C.byref(layout), _ptr(handle), handle.numel(), _ptr(x),
                                 _ptr(weight), _ptr(out), N, _stream(stream)),
           "ep_grouped_linear")


def grouped_linear_bwd(layout: Layout, handle: torch.Tensor, grad: torch.Tensor,
                       x: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                       grad_x: Optional[torch.Tensor] = None,
                       grad_weight: Optional[torch.Tensor] = None, stream=None):
    """The gradients of ``grouped_linear``; an output that is None is skipped,
    and so is the operand that only it needs (weight for grad_x, x for
    grad_weight)."""
    if grad.dim() != 2:
        raise ValueError(f"grad must have two dimensions, got {tuple(grad.shape)}")
    N = grad.shape[1]
    _need(handle, "handle", torch.uint8)
    _need(grad, "grad", layout.payload_dtype, (layout.cap, N))
    _need(x, "x", layout.payload_dtype, (layout.cap, layout.H), allow_none=grad_weight is None)
    _need(weight, "weight", layout.payload_dtype, (layout.E, N, layout.H),
          allow_none=grad_x is None)
    _need(grad_x, "grad_x", layout.payload_dtype, (layout.cap, layout.H), allow_none=True)
    _need(grad_weight, "grad_weight", layout.payload_dtype, (layout.E, N, layout.H),
          allow_none=True)
    _check(lib.ep_grouped_linear_bwd(C.byref(layout), _ptr(handle), handle.numel(), _ptr(grad),
                                     _ptr(x), _ptr(weight), _ptr(grad_x), _ptr(grad_weight), N,
                                     _stream(stream)), "ep_grouped_linear_bwd")


def grouped_linear_quant(layout: Layout, handle: torch.Tensor, x: torch.Tensor,
                         qweight: torch.Tensor, scales: torch.Tensor,
                         zeros: Optional[torch.Tensor], out: torch.Tensor, stream=None):
    """``grouped_linear`` with 4-bit weights: qweight uint8 [E,N,H/2] (the low
    four bits are the even input), scales [E,N,H/G] of the payload type, zeros
    uint8 [E,N,H/G] or None for 8; the group size G follows from the shapes."""
    if scales.dim() != 3 or scales.shape[2] < 1 or layout.H % scales.shape[2] != 0:
        raise ValueError(f"scales must have shape (E, N, H / group), got {tuple(scales.shape)}")
    N, groups = scales.shape[1], scales.shape[2]
    _need(handle, "handle", torch.uint8)
    _need(x, "x", layout.payload_dtype, (layout.cap, layout.H))
    _need(qweight, "qweight", torch.uint8, (layout.E, N, layout.H // 2))
    _need(scales, "scales", layout.payload_dtype, (layout.E, N, groups))
    _need(zeros, "zeros", torch.uint8, (layout.E, N, groups), allow_none=True)
    _need(out, "out", layout.payload_dtype, (layout.cap, N))
    _check(lib.ep_grouped_linear_quant(C.byref(layout), _ptr(handle), handle.numel(), _ptr(x),
                                       _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out), N,
                                       layout.H // groups, _stream(stream)),
           "ep_grouped_linear_quant")


def swiglu(layout: Layout, handle: torch.Tensor, gate_up: torch.Tensor, out: torch.Tensor,
           stream=None):
    """out [cap,H] = silu(gate) * up of each live row, gate and up the halves
    of gate_up [cap,2H]."""
    _need(handle, "handle", torch.uint8)
    _need(gate_up, "gate_up", layout.payload_dtype, (layout.cap, 2 * layout.H))
    _need(out, "out", layout.payload_dtype, (layout.cap, layout.H))
    _check(lib.ep_swiglu(C.byref(layout), _ptr(handle), handle.numel(), _ptr(gate_up),
                         _ptr(out), _stream(stream)), "ep_swiglu")


def swiglu_bwd(layout: Layout, handle: torch.Tensor, grad: torch.Tensor,
               gate_up: torch.Tensor, grad_gate_up: torch.Tensor, stream=None):
    _need(handle, "handle", torch.uint8)
    _need(grad, "grad", layout.payload_dtype, (layout.cap, layout.H))
    _need(gate_up, "gate_up", layout.payload_dtype, (layout.cap, 2 * layout.H))
    _need(grad_gate_up, "grad_gate_up", layout.payload_dtype, (layout.cap, 2 * layout.H))
    _check(lib.ep_swiglu_bwd(C.byref(layout), _ptr(handle), handle.numel(), _ptr(grad),
                             _ptr(gate_up), _ptr(grad_gate_up), _stream(stream)),
           "ep_swiglu_bwd")


def scale_columns(hidden: int) -> int:
    """Scales that a row of ``hidden`` 8-bit values has room for."""
    return (hidden + 1023) // 1024 * 8


def _scale_blocks(n: int) -> int:
    return (n + SCALE_BLOCK - 1) // SCALE_BLOCK


def rms_norm(layout: Layout, x: torch.Tensor, weight: torch.Tensor, eps: float,
             out: Optional[torch.Tensor] = None, out_q: Optional[torch.Tensor] = None,
             out_scales: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None,
             sum_out: Optional[torch.Tensor] = None, stream=None):
    """The norm of x [T,H] (with a residual: of sum_out = x + residual) times
    weight [H], into out [T,H], or in 8 bits into out_q with out_scales
    [T, scale_columns(H)], or both. sum_out may be residual (or x) itself."""
    T, H, dtype = layout.num_tokens, layout.hidden, layout.payload_dtype
    if out is None and out_q is None:
        raise ValueError("out or out_q is required")
    _both("out_q", out_q, "out_scales", out_scales)
    _both("residual", residual, "sum_out", sum_out)
    rows = (T, H)
    _need_all(((x, "x", dtype, rows), (weight, "weight", dtype, (H,))),
              ((out, "out", dtype, rows), (out_q, "out_q", E4M3, rows),
               (out_scales, "out_scales", torch.float32, (T, scale_columns(H))),
               (residual, "residual", dtype, rows), (sum_out, "sum_out", dtype, rows)))
    _check(lib.ep_rms_norm(C.byref(layout), _ptr(x), _ptr(residual), _ptr(weight), eps,
                           _ptr(sum_out), _ptr(out), _ptr(out_q), _ptr(out_scales),
                           _stream(stream)), "ep_rms_norm")


def new_rms_norm_bwd_workspace(layout: Layout, device=None) -> torch.Tensor:
    """The workspace of ``rms_norm_bwd`` for ``layout`` (uint8 tensor)."""
    n = int(lib.ep_rms_norm_bwd_workspace(C.byref(layout)))
    if n == 0:
        raise ValueError("invalid layout")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def rms_norm_bwd(layout: Layout, grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                 eps: float, grad_x: torch.Tensor, grad_weight: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 grad_sum: Optional[torch.Tensor] = None, stream=None):
    """The gradients of ``rms_norm``'s out with respect to what the norm was of
    (x, or sum_out with a residual) and the weight; grad_sum is a gradient of
    sum_out that is added to the first. A grad_weight that is None is skipped, and
    needs no workspace."""
    H, dtype = layout.hidden, layout.payload_dtype
    rows = (layout.num_tokens, H)
    if grad_weight is not None:
        _need(workspace, "workspace", torch.uint8)
    _need_all(((grad, "grad", dtype, rows), (x, "x", dtype, rows),
               (weight, "weight", dtype, (H,)), (grad_x, "grad_x", dtype, rows)),
              ((grad_weight, "grad_weight", dtype, (H,)), (grad_sum, "grad_sum", dtype, rows)))
    _check(lib.ep_rms_norm_bwd(C.byref(layout), _ptr(grad), _ptr(grad_sum), _ptr(x),
                               _ptr(weight), eps, _ptr(grad_x), _ptr(grad_weight),
                               _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               _stream(stream)), "ep_rms_norm_bwd")


def swiglu_scaled(layout: Layout, handle: torch.Tensor, gate_up: torch.Tensor,
                  out_q: torch.Tensor, out_scales: torch.Tensor, stream=None):
    """``swiglu`` with its result in 8 bits: out_q [cap,H] and out_scales
    [cap, scale_columns(H)]."""
    cap, H = layout.recv_capacity, layout.hidden
    _need(handle, "handle", torch.uint8)
    _need_all(((gate_up, "gate_up", layout.payload_dtype, (cap, 2 * H)),
               (out_q, "out_q", E4M3, (cap, H)),
               (out_scales, "out_scales", torch.float32, (cap, scale_columns(H)))))
    _check(lib.ep_swiglu_scaled(C.byref(layout), _ptr(handle), handle.numel(), _ptr(gate_up),
                                _ptr(out_q), _ptr(out_scales), _stream(stream)),
           "ep_swiglu_scaled")


def grouped_linear_scaled(layout: Layout, handle: torch.Tensor, x: torch.Tensor,
                          x_scales: torch.Tensor, weight: torch.Tensor,
                          weight_scales: torch.Tensor, out: torch.Tensor, stream=None):
    """``grouped_linear`` of 8-bit operands: x [cap,H] with x_scales
    [cap, scale_columns(H)], weight [E,N,H] with weight_scales
    [E, ceil(N/128), ceil(H/128)]; out [cap,N] of the layout's payload type."""
    N, E, H, cap = _out_features(weight), layout.num_experts, layout.hidden, layout.recv_capacity
    _need(handle, "handle", torch.uint8)
    _need_all(((x, "x", E4M3, (cap, H)),
               (x_scales, "x_scales", torch.float32, (cap, scale_columns(H))),
               (weight, "weight", E4M3, (E, N, H)),
               (weight_scales, "weight_scales", torch.float32,
                (E, _scale_blocks(N), _scale_blocks(H))),
               (out, "out", layout.payload_dtype, (cap, N))))
    _check(lib.ep_grouped_linear_scaled(C.byref(layout), _ptr(handle), handle.numel(), _ptr(x),
                                        _ptr(x_scales), _ptr(weight), _ptr(weight_scales),
                                        _ptr(out), N, _stream(stream)),
           "ep_grouped_linear_scaled")


def new_expert_layer_workspace(layout: Layout, inner: int, device=None) -> torch.Tensor:
    """The workspace of ``expert_layer`` for ``layout`` and ``inner`` features
    between the products (uint8 tensor)."""
    n = int(lib.ep_expert_layer_workspace(C.byref(layout), inner))
    if n == 0:
        raise ValueError("invalid layout or inner")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def expert_layer(layout: Layout, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                 tokens: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor,
                 result: torch.Tensor, workspace: torch.Tensor,
                 gate_up_scales: Optional[torch.Tensor] = None,
                 down_scales: Optional[torch.Tensor] = None, stream=None):
    """A whole expert layer for a few tokens (T * K up to MAX_LAYER_ROUTES),
    without a handle: result [T,H] = each token's routes, weighted, through
    gate_up [E,2I,H], the gated activation and down [E,H,I]. Weights of the
    payload type, or in 8 bits with both scales."""
    if down.dim() != 3:
        raise ValueError(f"down must have shape (E, H, I), got {tuple(down.shape)}")
    T, K, E, H = layout.num_tokens, layout.topk, layout.num_experts, layout.hidden
    inner, dtype = down.shape[2], layout.payload_dtype
    _both("gate_up_scales", gate_up_scales, "down_scales", down_scales)
    weights = dtype if gate_up_scales is None else E4M3
    _need(workspace, "workspace", torch.uint8)
    _need_all(((topk_idx, "topk_idx", torch.int64, (T, K)),
               (topk_weights, "topk_weights", torch.float32, (T, K)),
               (tokens, "tokens", dtype, (T, H)),
               (gate_up, "gate_up", weights, (E, 2 * inner, H)),
               (down, "down", weights, (E, H, inner)), (result, "result", dtype, (T, H))),
              ((gate_up_scales, "gate_up_scales", torch.float32,
                (E, _scale_blocks(2 * inner), _scale_blocks(H))),
               (down_scales, "down_scales", torch.float32,
                (E, _scale_blocks(H), _scale_blocks(inner)))))
    _check(lib.ep_expert_layer(C.byref(layout), _ptr(topk_idx), _ptr(topk_weights),
                               _ptr(tokens), _ptr(gate_up), _ptr(gate_up_scales), _ptr(down),
                               _ptr(down_scales), _ptr(result), inner, _ptr(workspace),
                               workspace.numel(), _stream(stream)), "ep_expert_layer")


def read_status(handle: torch.Tensor, stream=None) -> int:
    """Status word of the handle (waits for the stream)."""
    _need(handle, "handle", torch.uint8)
    out = C.c_uint32(0)
    _check(lib.ep_read_status(_ptr(handle), C.byref(out), _stream(stream)), "ep_read_status")
    return int(out.value)
