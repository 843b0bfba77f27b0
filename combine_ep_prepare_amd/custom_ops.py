"""The routing ops as ``torch.library`` custom ops, with autograd and fake
(meta) implementations, so that they can sit inside a ``torch.compile``
graph and be captured in a CUDA/HIP graph.

"[PyTorch] Expert Parallelism: PyTorch wrapper + autograd ops with symm-mem
zero-copy" (sections "Summary" and "Public Python API") registers dispatch and
combine as ``torch.library.custom_op`` with ``mutates_args`` and autograd
support; this module does the same for the one-GPU library. Every op
allocates its outputs with PyTorch and calls the C entry point of the same
name; nothing is computed here.

A layout travels as a list of ints ``[T, K, E, A, H, recv_capacity, dtype,
flags]`` (``layout_list``); the handle is the uint8 device tensor that
``prepare`` fills (declared mutated by prepare, read by the others). The
experts' ops take the routing's layout and use the row length of the tensor
that they are given in place of its H.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch
from torch import Tensor

from . import (DTYPE_BF16, E4M3, LAYOUT_NO_PAD_FILL, LAYOUT_ZERO_TAIL, TORCH_DTYPE, Layout,
               combine as _combine,
               combine_bwd as _combine_bwd, combine_weighted as _combine_weighted,
               combine_weighted_bwd as _combine_weighted_bwd, dispatch as _dispatch,
               dispatch_bwd as _dispatch_bwd, expert_layer as _expert_layer,
               grouped_linear as _grouped_linear, grouped_linear_bwd as _grouped_linear_bwd,
               grouped_linear_quant as _grouped_linear_quant,
               grouped_linear_scaled as _grouped_linear_scaled, new_expert_layer_workspace,
               new_rms_norm_bwd_workspace, prepare as _prepare, rms_norm as _rms_norm,
               rms_norm_bwd as _rms_norm_bwd, scale_columns, swiglu as _swiglu,
               swiglu_bwd as _swiglu_bwd, swiglu_scaled as _swiglu_scaled)

NS = "ep_mi355x"


def layout_list(layout: Layout) -> List[int]:
    return [int(layout.num_tokens), int(layout.topk), int(layout.num_experts),
            int(layout.alignment), int(layout.hidden), int(layout.recv_capacity),
            int(layout.dtype), int(layout.flags)]


def _layout(ll: Sequence[int], zero_tail: bool = False) -> Layout:
    """The layout of a list; ``zero_tail`` adds LAYOUT_ZERO_TAIL, which every
    op below that allocates an expert-major output sets, so that its rows past
    the live total are zeros rather than uninitialised memory."""
    T, K, E, A, H, cap, dt, flags = ll
    return Layout(T, K, E, A, H, cap, dtype=dt, fill_pads=not (flags & LAYOUT_NO_PAD_FILL),
                  zero_tail=zero_tail or bool(flags & LAYOUT_ZERO_TAIL))


def _pdtype(ll: Sequence[int]) -> torch.dtype:
    return TORCH_DTYPE.get(ll[6], TORCH_DTYPE[DTYPE_BF16])


# --------------------------------------------------------------------------
# prepare
# --------------------------------------------------------------------------

@torch.library.custom_op(f"{NS}::prepare", mutates_args=("handle",))
def prepare(topk_idx: Tensor, handle: Tensor, layout: List[int]) -> Tuple[Tensor, Tensor]:
    """(token_counts int32 [E], expert_offsets int32 [E+1]); fills ``handle``."""
    L = _layout(layout)
    counts = torch.empty(L.E, dtype=torch.int32, device=topk_idx.device)
    offsets = torch.empty(L.E + 1, dtype=torch.int32, device=topk_idx.device)
    _prepare(L, topk_idx, counts, handle, offsets)
    return counts, offsets


@prepare.register_fake
def _(topk_idx, handle, layout):
    E = layout[2]
    return (topk_idx.new_empty((E,), dtype=torch.int32),
            topk_idx.new_empty((E + 1,), dtype=torch.int32))


# --------------------------------------------------------------------------
# dispatch and its backward
# --------------------------------------------------------------------------

@torch.library.custom_op(f"{NS}::dispatch", mutates_args=())
def dispatch(tokens: Tensor, topk_weights: Tensor, handle: Tensor,
             layout: List[int]) -> Tuple[Tensor, Tensor]:
    """(recv_tokens [cap,H], recv_topk_weights fp32 [cap]); rows past the live
    total are zeros."""
    L = _layout(layout, zero_tail=True)
    recv = torch.empty(L.cap, L.H, dtype=tokens.dtype, device=tokens.device)
    recv_w = torch.empty(L.cap, dtype=torch.float32, device=tokens.device)
    _dispatch(L, handle, tokens, topk_weights, recv, recv_w)
    return recv, recv_w


@dispatch.register_fake
def _(tokens, topk_weights, handle, layout):
    cap, H = layout[5], layout[4]
    return tokens.new_empty((cap, H)), tokens.new_empty((cap,), dtype=torch.float32)


@torch.library.custom_op(f"{NS}::dispatch_bwd", mutates_args=())
def dispatch_bwd(grad: Tensor, g_recv_topk_weights: Optional[Tensor], handle: Tensor,
                 layout: List[int]) -> Tuple[Tensor, Tensor]:
    """(grad_tokens [T,H], grad_topk_weights fp32 [T,K]); a None weight
    gradient gives zero weight gradients."""
    L = _layout(layout)
    gt = torch.empty(L.T, L.H, dtype=grad.dtype, device=grad.device)
    gw = torch.empty(L.T, L.K, dtype=torch.float32, device=grad.device)
    _dispatch_bwd(L, handle, grad, g_recv_topk_weights, gt, gw)
    return gt, gw


@dispatch_bwd.register_fake
def _(grad, g_recv_topk_weights, handle, layout):
    T, K, H = layout[0], layout[1], layout[4]
    return grad.new_empty((T, H)), grad.new_empty((T, K), dtype=torch.float32)


def _dispatch_setup(ctx, inputs, output):
    _, _, handle, layout = inputs
    ctx.save_for_backward(handle)
    ctx.layout = layout


def _dispatch_backward(ctx, g_recv, g_recv_w):
    (handle,) = ctx.saved_tensors
    layout = ctx.layout
    if g_recv is None:
        g_recv = torch.zeros(layout[5], layout[4], dtype=_pdtype(layout), device=handle.device)
    gt, gw = dispatch_bwd(g_recv.contiguous(),
                          None if g_recv_w is None else g_recv_w.contiguous(), handle, layout)
    return gt, gw, None, None


dispatch.register_autograd(_dispatch_backward, setup_context=_dispatch_setup)


# --------------------------------------------------------------------------
# combine and its backward
# --------------------------------------------------------------------------

@torch.library.custom_op(f"{NS}::combine", mutates_args=())
def combine(expert_out: Tensor, handle: Tensor, layout: List[int]) -> Tensor:
    """Unweighted sum of each token's received rows, [T,H]."""
    L = _layout(layout)
    out = torch.empty(L.T, L.H, dtype=expert_out.dtype, device=expert_out.device)
    _combine(L, handle, expert_out, out)
    return out


@combine.register_fake
def _(expert_out, handle, layout):
    return expert_out.new_empty((layout[0], layout[4]))


@torch.library.custom_op(f"{NS}::combine_bwd", mutates_args=())
def combine_bwd(grad: Tensor, handle: Tensor, layout: List[int]) -> Tensor:
    """grad_expert_out [cap,H]: each live row takes its token's gradient; pad
    rows zero (unless the layout skips the pad fill); rows past the live total
    zero (combine never reads them)."""
    L = _layout(layout, zero_tail=True)
    out = torch.empty(L.cap, L.H, dtype=grad.dtype, device=grad.device)
    _combine_bwd(L, handle, grad, out)
    return out


@combine_bwd.register_fake
def _(grad, handle, layout):
    return grad.new_empty((layout[5], layout[4]))


def _combine_setup(ctx, inputs, output):
    _, handle, layout = inputs
    ctx.save_for_backward(handle)
    ctx.layout = layout


def _combine_backward(ctx, g):
    (handle,) = ctx.saved_tensors
    return combine_bwd(g.contiguous(), handle, ctx.layout), None, None


combine.register_autograd(_combine_backward, setup_context=_combine_setup)


# --------------------------------------------------------------------------
# weighted combine and its backward
# --------------------------------------------------------------------------

@torch.library.custom_op(f"{NS}::combine_weighted", mutates_args=())
def combine_weighted(expert_out: Tensor, recv_topk_weights: Tensor, handle: Tensor,
                     layout: List[int]) -> Tensor:
    """Sum of each token's received rows, each scaled by its received weight."""
    L = _layout(layout)
    out = torch.empty(L.T, L.H, dtype=expert_out.dtype, device=expert_out.device)
    _combine_weighted(L, handle, expert_out, recv_topk_weights, out)
    return out


@combine_weighted.register_fake
def _(expert_out, recv_topk_weights, handle, layout):
    return expert_out.new_empty((layout[0], layout[4]))


@torch.library.custom_op(f"{NS}::combine_weighted_bwd", mutates_args=())
def combine_weighted_bwd(grad: Tensor, expert_out: Tensor, recv_topk_weights: Tensor,
                         handle: Tensor, layout: List[int]) -> Tuple[Tensor, Tensor]:
    """(grad_expert_out [cap,H], grad_recv_topk_weights fp32 [cap]); rows past
    the live total zero in both."""
    L = _layout(layout, zero_tail=True)
    gr = torch.empty(L.cap, L.H, dtype=grad.dtype, device=grad.device)
    gw = torch.empty(L.cap, dtype=torch.float32, device=grad.device)
    _combine_weighted_bwd(L, handle, grad, expert_out, recv_topk_weights, gr, gw)
    return gr, gw


@combine_weighted_bwd.register_fake
def _(grad, expert_out, recv_topk_weights, handle, layout):
    cap, H = layout[5], layout[4]
    return grad.new_empty((cap, H)), grad.new_empty((cap,), dtype=torch.float32)


def _cw_setup(ctx, inputs, output):
    expert_out, recv_topk_weights, handle, layout = inputs
    ctx.save_for_backward(expert_out, recv_topk_weights, handle)
    ctx.layout = layout


def _cw_backward(ctx, g):
    expert_out, w, handle = ctx.saved_tensors
    gr, gw = combine_weighted_bwd(g.contiguous(), expert_out, w, handle, ctx.layout)
    return gr, gw, None, None


combine_weighted.register_autograd(_cw_backward, setup_context=_cw_setup)


# --------------------------------------------------------------------------
# the experts' products and activation
# --------------------------------------------------------------------------

def _rows_layout(ll: Sequence[int], hidden: int) -> Layout:
    return _layout([*ll[:4], hidden, *ll[5:]], zero_tail=True)


@torch.library.custom_op(f"{NS}::grouped_linear", mutates_args=())
def grouped_linear(x: Tensor, weight: Tensor, handle: Tensor, layout: List[int]) -> Tensor:
    """Each live row of x [cap,H] through its expert's weight [E,N,H]: [cap,N]."""
    out = torch.empty(x.shape[0], weight.shape[1], dtype=x.dtype, device=x.device)
    _grouped_linear(_rows_layout(layout, x.shape[1]), handle, x, weight, out)
    return out


@grouped_linear.register_fake
def _(x, weight, handle, layout):
    return x.new_empty((x.shape[0], weight.shape[1]))


@torch.library.custom_op(f"{NS}::grouped_linear_bwd", mutates_args=())
def grouped_linear_bwd(grad: Tensor, x: Tensor, weight: Tensor, handle: Tensor,
                       layout: List[int]) -> Tuple[Tensor, Tensor]:
    """(grad_x [cap,H], grad_weight [E,N,H])."""
    gx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    gw = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device)
    _grouped_linear_bwd(_rows_layout(layout, x.shape[1]), handle, grad, x, weight, gx, gw)
    return gx, gw


@grouped_linear_bwd.register_fake
def _(grad, x, weight, handle, layout):
    return x.new_empty(x.shape), weight.new_empty(weight.shape)


# The two gradients one by one, for a backward that is asked for one of them.

@torch.library.custom_op(f"{NS}::grouped_linear_grad_x", mutates_args=())
def grouped_linear_grad_x(grad: Tensor, weight: Tensor, handle: Tensor,
                          layout: List[int]) -> Tensor:
    """grad_x [cap,H] alone."""
    gx = torch.empty(grad.shape[0], weight.shape[2], dtype=grad.dtype, device=grad.device)
    _grouped_linear_bwd(_rows_layout(layout, weight.shape[2]), handle, grad, None, weight, gx,
                        None)
    return gx


@grouped_linear_grad_x.register_fake
def _(grad, weight, handle, layout):
    return grad.new_empty((grad.shape[0], weight.shape[2]))


@torch.library.custom_op(f"{NS}::grouped_linear_grad_weight", mutates_args=())
def grouped_linear_grad_weight(grad: Tensor, x: Tensor, handle: Tensor,
                               layout: List[int]) -> Tensor:
    """grad_weight [E,N,H] alone."""
    gw = torch.empty(layout[2], grad.shape[1], x.shape[1], dtype=grad.dtype, device=grad.device)
    _grouped_linear_bwd(_rows_layout(layout, x.shape[1]), handle, grad, x, None, None, gw)
    return gw


@grouped_linear_grad_weight.register_fake
def _(grad, x, handle, layout):
    return grad.new_empty((layout[2], grad.shape[1], x.shape[1]))


def _linear_setup(ctx, inputs, output):
    x, weight, handle, layout = inputs
    ctx.save_for_backward(x, weight, handle)
    ctx.layout = layout


def _linear_backward(ctx, g):
    x, weight, handle = ctx.saved_tensors
    g, gx, gw = g.contiguous(), None, None
    want_x, want_w = ctx.needs_input_grad[:2]
    if want_x and want_w:
        gx, gw = grouped_linear_bwd(g, x, weight, handle, ctx.layout)
    elif want_x:
        gx = grouped_linear_grad_x(g, weight, handle, ctx.layout)
    elif want_w:
        gw = grouped_linear_grad_weight(g, x, handle, ctx.layout)
    return gx, gw, None, None


grouped_linear.register_autograd(_linear_backward, setup_context=_linear_setup)


@torch.library.custom_op(f"{NS}::grouped_linear_quant", mutates_args=())
def grouped_linear_quant(x: Tensor, qweight: Tensor, scales: Tensor, zeros: Optional[Tensor],
                         handle: Tensor, layout: List[int]) -> Tensor:
    """``grouped_linear`` with 4-bit weights; no autograd."""
    out = torch.empty(x.shape[0], scales.shape[1], dtype=x.dtype, device=x.device)
    _grouped_linear_quant(_rows_layout(layout, x.shape[1]), handle, x, qweight, scales, zeros,
                          out)
    return out


@grouped_linear_quant.register_fake
def _(x, qweight, scales, zeros, handle, layout):
    return x.new_empty((x.shape[0], scales.shape[1]))


@torch.library.custom_op(f"{NS}::swiglu", mutates_args=())
def swiglu(gate_up: Tensor, handle: Tensor, layout: List[int]) -> Tensor:
    """silu(gate) * up of each live row of gate_up [cap,2I]: [cap,I]."""
    hidden = gate_up.shape[1] // 2
    out = torch.empty(gate_up.shape[0], hidden, dtype=gate_up.dtype, device=gate_up.device)
    _swiglu(_rows_layout(layout, hidden), handle, gate_up, out)
    return out


@swiglu.register_fake
def _(gate_up, handle, layout):
    return gate_up.new_empty((gate_up.shape[0], gate_up.shape[1] // 2))


@torch.library.custom_op(f"{NS}::swiglu_bwd", mutates_args=())
def swiglu_bwd(grad: Tensor, gate_up: Tensor, handle: Tensor, layout: List[int]) -> Tensor:
    """The gradient of gate_up [cap,2I]."""
    out = torch.empty(gate_up.shape, dtype=gate_up.dtype, device=gate_up.device)
    _swiglu_bwd(_rows_layout(layout, gate_up.shape[1] // 2), handle, grad, gate_up, out)
    return out


@swiglu_bwd.register_fake
def _(grad, gate_up, handle, layout):
    return gate_up.new_empty(gate_up.shape)


def _swiglu_setup(ctx, inputs, output):
    gate_up, handle, layout = inputs
    ctx.save_for_backward(gate_up, handle)
    ctx.layout = layout


def _swiglu_backward(ctx, g):
    gate_up, handle = ctx.saved_tensors
    return swiglu_bwd(g.contiguous(), gate_up, handle, ctx.layout), None, None


swiglu.register_autograd(_swiglu_backward, setup_context=_swiglu_setup)


# --------------------------------------------------------------------------
# the norm in front of a layer, the ops in 8 bits, the layer for a few tokens
# --------------------------------------------------------------------------

def _norm_layout(x: Tensor) -> Layout:
    return Layout(x.shape[0], 1, 1, 1, x.shape[1], 0, dtype=x.dtype)


@torch.library.custom_op(f"{NS}::rms_norm", mutates_args=())
def rms_norm(x: Tensor, weight: Tensor, eps: float) -> Tensor:
    """The norm of the rows of x [T,H] times weight [H]."""
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _rms_norm(_norm_layout(x), x, weight, eps, out=out)
    return out


@rms_norm.register_fake
def _(x, weight, eps):
    return x.new_empty(x.shape)


@torch.library.custom_op(f"{NS}::add_rms_norm", mutates_args=())
def add_rms_norm(x: Tensor, residual: Tensor, weight: Tensor,
                 eps: float) -> Tuple[Tensor, Tensor]:
    """(the norm of x + residual times weight, x + residual)."""
    out, total = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    _rms_norm(_norm_layout(x), x, weight, eps, out=out, residual=residual, sum_out=total)
    return out, total


@add_rms_norm.register_fake
def _(x, residual, weight, eps):
    return x.new_empty(x.shape), x.new_empty(x.shape)


@torch.library.custom_op(f"{NS}::rms_norm_bwd", mutates_args=())
def rms_norm_bwd(grad: Tensor, x: Tensor, weight: Tensor, eps: float,
                 grad_sum: Optional[Tensor]) -> Tuple[Tensor, Tensor]:
    """The gradients of what the norm was of and of the weight."""
    L = _norm_layout(x)
    gx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    gw = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device)
    _rms_norm_bwd(L, grad, x, weight, eps, gx, gw, new_rms_norm_bwd_workspace(L, x.device),
                  grad_sum)
    return gx, gw


@rms_norm_bwd.register_fake
def _(grad, x, weight, eps, grad_sum):
    return x.new_empty(x.shape), weight.new_empty(weight.shape)


# The first alone, for a backward that is not asked for the weight's.

@torch.library.custom_op(f"{NS}::rms_norm_grad_x", mutates_args=())
def rms_norm_grad_x(grad: Tensor, x: Tensor, weight: Tensor, eps: float,
                    grad_sum: Optional[Tensor]) -> Tensor:
    """The gradient of what the norm was of alone."""
    gx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _rms_norm_bwd(_norm_layout(x), grad, x, weight, eps, gx, grad_sum=grad_sum)
    return gx


@rms_norm_grad_x.register_fake
def _(grad, x, weight, eps, grad_sum):
    return x.new_empty(x.shape)


def _norm_gradients(ctx, want_w, g, g_sum):
    x, weight = ctx.saved_tensors
    if want_w:
        return rms_norm_bwd(g.contiguous(), x, weight, ctx.eps, g_sum)
    return rms_norm_grad_x(g.contiguous(), x, weight, ctx.eps, g_sum), None


def _norm_setup(ctx, inputs, output):
    x, weight, ctx.eps = inputs
    ctx.save_for_backward(x, weight)


def _norm_backward(ctx, g):
    gx, gw = _norm_gradients(ctx, ctx.needs_input_grad[1], g, None)
    return gx, gw, None


rms_norm.register_autograd(_norm_backward, setup_context=_norm_setup)


def _add_norm_setup(ctx, inputs, output):
    ctx.eps = inputs[3]
    ctx.save_for_backward(output[1], inputs[2])


def _add_norm_backward(ctx, g, g_sum):
    gx, gw = _norm_gradients(ctx, ctx.needs_input_grad[2], g, g_sum.contiguous())
    return gx, gx, gw, None


add_rms_norm.register_autograd(_add_norm_backward, setup_context=_add_norm_setup)


@torch.library.custom_op(f"{NS}::rms_norm_scaled", mutates_args=())
def rms_norm_scaled(x: Tensor, weight: Tensor, eps: float) -> Tuple[Tensor, Tensor]:
    """``rms_norm`` in 8 bits: (e4m3 [T,H], scales [T, scale_columns(H)]); no autograd,
    like the ops below."""
    q = torch.empty(x.shape, dtype=E4M3, device=x.device)
    scales = torch.empty(x.shape[0], scale_columns(x.shape[1]), dtype=torch.float32,
                         device=x.device)
    _rms_norm(_norm_layout(x), x, weight, eps, out_q=q, out_scales=scales)
    return q, scales


@rms_norm_scaled.register_fake
def _(x, weight, eps):
    return (x.new_empty(x.shape, dtype=E4M3),
            x.new_empty((x.shape[0], scale_columns(x.shape[1])), dtype=torch.float32))


@torch.library.custom_op(f"{NS}::add_rms_norm_scaled", mutates_args=())
def add_rms_norm_scaled(x: Tensor, residual: Tensor, weight: Tensor,
                        eps: float) -> Tuple[Tensor, Tensor, Tensor]:
    """(e4m3, scales, x + residual)."""
    q = torch.empty(x.shape, dtype=E4M3, device=x.device)
    scales = torch.empty(x.shape[0], scale_columns(x.shape[1]), dtype=torch.float32,
                         device=x.device)
    total = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _rms_norm(_norm_layout(x), x, weight, eps, out_q=q, out_scales=scales, residual=residual,
              sum_out=total)
    return q, scales, total


@add_rms_norm_scaled.register_fake
def _(x, residual, weight, eps):
    return (x.new_empty(x.shape, dtype=E4M3),
            x.new_empty((x.shape[0], scale_columns(x.shape[1])), dtype=torch.float32),
            x.new_empty(x.shape))


@torch.library.custom_op(f"{NS}::swiglu_scaled", mutates_args=())
def swiglu_scaled(gate_up: Tensor, handle: Tensor, layout: List[int]) -> Tuple[Tensor, Tensor]:
    """``swiglu`` in 8 bits: (e4m3 [cap,I], scales [cap, scale_columns(I)])."""
    hidden = gate_up.shape[1] // 2
    q = torch.empty(gate_up.shape[0], hidden, dtype=E4M3, device=gate_up.device)
    scales = torch.empty(gate_up.shape[0], scale_columns(hidden), dtype=torch.float32,
                         device=gate_up.device)
    _swiglu_scaled(_rows_layout(layout, hidden), handle, gate_up, q, scales)
    return q, scales


@swiglu_scaled.register_fake
def _(gate_up, handle, layout):
    cap, hidden = gate_up.shape[0], gate_up.shape[1] // 2
    return (gate_up.new_empty((cap, hidden), dtype=E4M3),
            gate_up.new_empty((cap, scale_columns(hidden)), dtype=torch.float32))


@torch.library.custom_op(f"{NS}::grouped_linear_scaled", mutates_args=())
def grouped_linear_scaled(x: Tensor, x_scales: Tensor, weight: Tensor, weight_scales: Tensor,
                          handle: Tensor, layout: List[int]) -> Tensor:
    """``grouped_linear`` of 8-bit operands, a result of the layout's payload type."""
    out = torch.empty(x.shape[0], weight.shape[1], dtype=_pdtype(layout), device=x.device)
    _grouped_linear_scaled(_rows_layout(layout, x.shape[1]), handle, x, x_scales, weight,
                           weight_scales, out)
    return out


@grouped_linear_scaled.register_fake
def _(x, x_scales, weight, weight_scales, handle, layout):
    return x.new_empty((x.shape[0], weight.shape[1]), dtype=_pdtype(layout))


@torch.library.custom_op(f"{NS}::expert_layer", mutates_args=())
def expert_layer(tokens: Tensor, topk_idx: Tensor, topk_weights: Tensor, gate_up: Tensor,
                 down: Tensor, gate_up_scales: Optional[Tensor],
                 down_scales: Optional[Tensor]) -> Tensor:
    """A whole expert layer for a few tokens [T,H]."""
    out = torch.empty(tokens.shape, dtype=tokens.dtype, device=tokens.device)
    L = Layout(tokens.shape[0], topk_idx.shape[1], down.shape[0], 1, tokens.shape[1], 0,
               dtype=tokens.dtype)
    _expert_layer(L, topk_idx, topk_weights, tokens, gate_up, down, out,
                  new_expert_layer_workspace(L, down.shape[2], tokens.device), gate_up_scales,
                  down_scales)
    return out


@expert_layer.register_fake
def _(tokens, topk_idx, topk_weights, gate_up, down, gate_up_scales, down_scales):
    return tokens.new_empty(tokens.shape)
