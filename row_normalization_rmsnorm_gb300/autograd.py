"""torch.autograd Functions and nn.Modules over the C ABI.

The frozen-parameter rule of "perf(norm): skip dW/dB calculation when
parameters are frozen" (Key Changes): each backward asks
``ctx.needs_input_grad`` whether the weight (and the LayerNorm bias) need a
gradient and passes NULL for those that do not, so a frozen parameter gets
no workspace, no partial sums and no column reduction, only dx.  A call in
which nothing requires grad saves nothing for a backward.

All arithmetic runs in the library's kernels; this module allocates the
outputs (and the dW / dB workspace) with torch and marshals arguments.
Inputs may have any leading shape; the last dimension is normalised and
must be contiguous.  Forward-mode tangents are refused, and so are second
derivatives through the checkpointed forms and the block boundary.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B

# how a backward's saved rows may be kept: `checkpoint=` of the functions and
# modules below (None: in full)
CHECKPOINT_FORMATS = {None: B.NORM_SAVED_FULL, "e4m3": B.NORM_SAVED_E4M3, "int8": B.NORM_SAVED_INT8}


def _format(checkpoint):
    if checkpoint not in CHECKPOINT_FORMATS:
        raise ValueError(f"checkpoint must be one of {list(CHECKPOINT_FORMATS)}, got {checkpoint!r}")
    return CHECKPOINT_FORMATS[checkpoint]


def _ckpt_like(x2):
    return torch.empty(x2.shape[0], B.norm_ckpt_row_bytes(x2.shape[1]), dtype=torch.uint8, device=x2.device)


def _stat(x2):
    return torch.empty(x2.shape[0], dtype=torch.float32, device=x2.device)


def _kept(*tensors):
    """Whether a backward may follow a call on these tensors."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """A 2-D [rows, N] view with contiguous rows (copying only if needed)."""
    if t.dim() == 0:
        raise ValueError("expected at least one dimension")
    if t.dim() == 2 and t.is_contiguous():
        r = t
    else:
        if t.stride(-1) != 1:
            t = t.contiguous()
        try:
            r = t.view(-1, t.shape[-1])
        except RuntimeError:
            return t.contiguous().view(-1, t.shape[-1])
    rows, n = r.shape
    if rows == 0 or r.stride(0) >= n:
        return r
    # rows that share memory (a gradient expanded over the rows) are copied out;
    # the stride of a single row says nothing: it gets the row's length
    return r.contiguous() if rows > 1 else r.as_strided((1, n), (n, 1))


def _shaped(t, shape):
    return t if t.shape == shape else t.view(shape)


def _workspace(M, N, dw, db, device):
    nb = B.norm_bwd_workspace_bytes(M, N, dw, db)
    return torch.empty(nb, dtype=torch.uint8, device=device) if nb else None


class RMSNormFunction(torch.autograd.Function):
    """y = x * rstd * (w + offset), rstd = 1/sqrt(mean(x^2) + eps)."""

    @staticmethod
    def forward(ctx, x, w, eps=1e-6, offset=0.0, in_place=False):
        x2 = _rows(x)
        M, N = x2.shape
        y = torch.empty_like(x2)
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
        B.norm_rms_fwd(x2, w, y, rstd, offset, eps)
        ctx.eps, ctx.offset, ctx.in_place = eps, offset, in_place
        ctx.save_for_backward(x2, w, rstd)
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        x2, w, rstd = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_dx or need_dw):
            return None, None, None, None, None
        M, N = x2.shape
        dy2 = _rows(dy)
        # in place: dx overwrites the incoming gradient's own storage (when
        # its rows are that storage, not a copy), saving one M x N buffer
        own = ctx.in_place and dy2.data_ptr() == dy.data_ptr() and dy2.dtype == x2.dtype
        dx = dy2 if own else torch.empty_like(x2)
        dw = torch.empty_like(w) if need_dw else None
        B.norm_rms_bwd(dy2, x2, w, rstd, dx, dw, _workspace(M, N, need_dw, False, x2.device) if need_dw else None,
                       ctx.offset, ctx.eps)
        return (dx.view(dy.shape) if need_dx else None), dw, None, None, None


class LayerNormFunction(torch.autograd.Function):
    """y = (x - mean) * rstd * (w + offset) + b (b may be None)."""

    @staticmethod
    def forward(ctx, x, w, b=None, eps=1e-6, offset=0.0):
        x2 = _rows(x)
        M, N = x2.shape
        y = torch.empty_like(x2)
        mean = torch.empty(M, dtype=torch.float32, device=x.device)
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
        B.norm_ln_fwd(x2, w, b, y, mean, rstd, offset, eps)
        ctx.eps, ctx.offset = eps, offset
        ctx.has_b = b is not None
        ctx.save_for_backward(x2, w, mean, rstd)
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        x2, w, mean, rstd = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        need_db = ctx.has_b and ctx.needs_input_grad[2]
        if not (need_dx or need_dw or need_db):
            return None, None, None, None, None
        M, N = x2.shape
        dy2 = _rows(dy)
        dx = torch.empty_like(x2)
        dw = torch.empty_like(w) if need_dw else None
        db = torch.empty_like(w) if need_db else None
        ws = _workspace(M, N, need_dw, need_db, x2.device) if (need_dw or need_db) else None
        B.norm_ln_bwd(dy2, x2, w, mean, rstd, dx, dw, db, ws, ctx.offset, ctx.eps)
        return (dx.view(dy.shape) if need_dx else None), dw, db, None, None


class FusedAddRMSNormFunction(torch.autograd.Function):
    """h = x + residual; y = RMSNorm(h) * (w + offset).  Returns (y, h)."""

    @staticmethod
    def forward(ctx, x, residual, w, eps=1e-6, offset=0.0, in_place=False):
        x2, r2 = _rows(x), _rows(residual)
        M, N = x2.shape
        y = torch.empty_like(x2)
        h = torch.empty_like(x2)
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
        B.norm_fused_add_rms_fwd(x2, r2, w, y, h, rstd, offset, eps)
        ctx.eps, ctx.offset, ctx.in_place = eps, offset, in_place
        ctx.save_for_backward(h, w, rstd)
        return y.view(x.shape), h.view(x.shape)

    @staticmethod
    def backward(ctx, dy, dh):
        h, w, rstd = ctx.saved_tensors
        need_x, need_r, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.needs_input_grad[2]
        if not (need_x or need_r or need_dw):
            return None, None, None, None, None, None
        M, N = h.shape
        if dy is None:
            dy = torch.zeros_like(h)
        dy2 = _rows(dy)
        dh2 = None if dh is None else _rows(dh)
        # in place: dx overwrites the residual stream's incoming gradient
        # (dh_out), whose value it already adds
        own = ctx.in_place and dh2 is not None and dh2.data_ptr() == dh.data_ptr() and dh2.dtype == h.dtype
        dx = dh2 if own else torch.empty_like(h)
        dw = torch.empty_like(w) if need_dw else None
        B.norm_fused_add_rms_bwd(dy2, dh2, h, w, rstd, dx, dw,
                                 _workspace(M, N, need_dw, False, h.device) if need_dw else None, ctx.offset, ctx.eps)
        # h = x + residual: one gradient serves both inputs
        g = dx.view(dy.shape)
        return (g if need_x else None), (g if need_r else None), dw, None, None, None


class RMSNormCkptFunction(torch.autograd.Function):
    """RMSNorm that keeps its input for the backward as an 8-bit checkpoint."""

    @staticmethod
    def forward(ctx, x, w, eps, offset, fmt):
        x2 = _rows(x)
        y, rstd, q = torch.empty_like(x2), _stat(x2), _ckpt_like(x2)
        B.norm_rms_fwd_ckpt(x2, w, y, rstd, q, fmt, offset, eps)
        ctx.offset, ctx.fmt = offset, fmt
        ctx.save_for_backward(q, w, rstd)
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, w, rstd = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        dy2 = _rows(dy)
        M, N = dy2.shape
        dx = torch.empty_like(dy2)
        dw = torch.empty_like(w) if need_dw else None
        B.norm_rms_bwd_ckpt(dy2, q, ctx.fmt, w, rstd, dx, dw,
                            _workspace(M, N, True, False, dy.device) if need_dw else None, ctx.offset)
        return (dx.view(dy.shape) if need_dx else None), dw, None, None, None


class LayerNormCkptFunction(torch.autograd.Function):
    """LayerNorm that keeps its input, less the row's mean, for the backward as
    an 8-bit checkpoint."""

    @staticmethod
    def forward(ctx, x, w, b, eps, offset, fmt):
        x2 = _rows(x)
        y, rstd, q = torch.empty_like(x2), _stat(x2), _ckpt_like(x2)
        B.norm_ln_fwd_ckpt(x2, w, b, y, None, rstd, q, fmt, offset, eps)
        ctx.offset, ctx.fmt, ctx.has_b = offset, fmt, b is not None
        ctx.save_for_backward(q, w, rstd)
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, w, rstd = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        need_db = ctx.has_b and ctx.needs_input_grad[2]
        dy2 = _rows(dy)
        M, N = dy2.shape
        dx = torch.empty_like(dy2)
        dw = torch.empty_like(w) if need_dw else None
        db = torch.empty_like(w) if need_db else None
        ws = _workspace(M, N, need_dw, need_db, dy.device) if (need_dw or need_db) else None
        B.norm_ln_bwd_ckpt(dy2, q, ctx.fmt, w, rstd, dx, dw, db, ws, ctx.offset)
        return (dx.view(dy.shape) if need_dx else None), dw, db, None, None, None


class FusedAddRMSNormCkptFunction(torch.autograd.Function):
    """FusedAddRMSNorm that keeps h for the backward as an 8-bit checkpoint:
    the residual stream itself is then free once its next reader is done."""

    @staticmethod
    def forward(ctx, x, residual, w, eps, offset, fmt):
        x2, r2 = _rows(x), _rows(residual)
        y, h, rstd, q = torch.empty_like(x2), torch.empty_like(x2), _stat(x2), _ckpt_like(x2)
        B.norm_fused_add_rms_fwd_ckpt(x2, r2, w, y, h, rstd, q, fmt, offset, eps)
        ctx.offset, ctx.fmt = offset, fmt
        ctx.save_for_backward(q, w, rstd)
        ctx.set_materialize_grads(False)
        ctx.shapes = x.shape, residual.shape
        return y.view(x.shape), h.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        q, w, rstd = ctx.saved_tensors
        need_x, need_r, need_dw = ctx.needs_input_grad[:3]
        if dy is None and dh is None:
            return (None,) * 6
        if dy is None:
            dy = torch.zeros_like(dh)
        dy2, dh2 = _rows(dy), None if dh is None else _rows(dh)
        M, N = dy2.shape
        dx = torch.empty_like(dy2)
        dw = torch.empty_like(w) if need_dw else None
        B.norm_fused_add_rms_bwd_ckpt(dy2, dh2, q, ctx.fmt, w, rstd, dx, dw,
                                      _workspace(M, N, True, False, dy.device) if need_dw else None, ctx.offset)
        # one gradient serves both inputs: as one tensor (two views of its memory
        # would each pass for the only one, and be added to in place)
        xs, rs = ctx.shapes
        dx = _shaped(dx, xs)
        dr = dx if xs == rs or not need_x else dx.clone()
        return (dx if need_x else None), (_shaped(dr, rs) if need_r else None), dw, None, None, None


def _gate_rows(gate, x, rows_per_gate):
    """A gate as ([N] or [rows, N], rows_per_gate): [N], [rows, N] with
    rows_per_gate, or x's shape with trailing row dimensions of 1 ([B, 1, N] for
    x [B, T, N]: one gate row per sequence)."""
    if gate is None or gate.dim() == 1:
        return gate, None
    if rows_per_gate is not None:
        return _rows(gate), rows_per_gate
    if gate.dim() != x.dim() or gate.shape[-1] != x.shape[-1]:
        raise ValueError(f"gate {tuple(gate.shape)} does not broadcast over x {tuple(x.shape)}")
    lead = x.dim() - 1
    p = max((d + 1 for d in range(lead) if gate.shape[d] != 1), default=0)
    if gate.shape[:p] != x.shape[:p]:
        raise ValueError(
            f"gate {tuple(gate.shape)} must have x's leading dimensions {tuple(x.shape)} up to trailing ones")
    R = 1
    for d in range(p, lead):
        R *= x.shape[d]
    return _rows(gate), max(1, R)


class BlockRMSNormFunction(torch.autograd.Function):
    """h = residual_scale * residual + block_scale * gate * RMSNorm(x; w_post);
    y = RMSNorm(h; w_pre).  Returns (y, h), y None without w_pre."""

    @staticmethod
    def forward(ctx, x, residual, w_post, w_pre, gate, rows_per_gate, residual_scale, block_scale, eps, offset, fmt,
                kept=True):
        x2, r2 = _rows(x), _rows(residual)
        g2, R = _gate_rows(gate, x, rows_per_gate)
        post, pre = w_post is not None, w_pre is not None
        if not kept:   # no backward follows; outputs that are no views may be written over
            y, h = (x2.new_empty(x.shape) if pre else None), x2.new_empty(x.shape)
            B.norm_block_rms_fwd(x2, r2, w_post, w_pre, _shaped(y, x2.shape) if pre else None, _shaped(h, x2.shape),
                                 gate=g2, rows_per_gate=R, residual_scale=residual_scale, block_scale=block_scale,
                                 offset=offset, eps=eps)
            return y, h
        y, h = (torch.empty_like(x2) if pre else None), torch.empty_like(x2)
        rs1, rs2 = (_stat(x2) if post else None), (_stat(x2) if pre else None)
        full = fmt == B.NORM_SAVED_FULL
        # x is needed for its norm's gradients and for the gate's; h for its norm's
        need_x = post or (gate is not None and gate.requires_grad)
        xq = _ckpt_like(x2) if need_x and not full else None
        hq = _ckpt_like(x2) if pre and not full else None
        B.norm_block_rms_fwd(x2, r2, w_post, w_pre, y, h, rs1, rs2, gate=g2, rows_per_gate=R, x_ckpt=xq, h_ckpt=hq,
                             ckpt_format=fmt if xq is not None or hq is not None else B.NORM_SAVED_FULL,
                             residual_scale=residual_scale, block_scale=block_scale, offset=offset, eps=eps)
        ctx.args = (R, residual_scale, block_scale, offset, fmt, x.shape, residual.shape)
        ctx.gate_shape = None if gate is None else gate.shape
        ctx.set_materialize_grads(False)
        ctx.save_for_backward((x2 if full else xq) if need_x else None, (h if full else hq) if pre else None, w_post,
                              w_pre, rs1, rs2, g2)
        return (_shaped(y, x.shape) if pre else None), _shaped(h, x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x2, h, w_post, w_pre, rs1, rs2, g2 = ctx.saved_tensors
        R, residual_scale, block_scale, offset, fmt, x_shape, r_shape = ctx.args
        need_x, need_r, need_post, need_pre, need_gate = ctx.needs_input_grad[:5]
        if dy is None and dh is None:
            return (None,) * 12
        if w_pre is not None and dy is None:
            dy = torch.zeros_like(dh)
        dy2, dh2 = (None if t is None else _rows(t) for t in (dy, dh))
        one = dy2 if dy2 is not None else dh2
        M, N = one.shape
        dx = torch.empty_like(one) if need_x else None
        dr = torch.empty_like(one) if need_r else None
        dw1 = torch.empty_like(w_post) if need_post else None
        dw2 = torch.empty_like(w_pre) if need_pre else None
        dg = torch.empty_like(g2) if need_gate else None
        rows = 0 if g2 is None else 1 if g2.dim() == 1 else g2.shape[0]
        nb = B.norm_block_bwd_workspace_bytes(M, N, rows, need_post, need_pre, need_gate)
        ws = torch.empty(nb, dtype=torch.uint8, device=one.device) if nb else None
        B.norm_block_rms_bwd(dy2, dh2, x2, h, w_post, w_pre, rs1, rs2, dx, dr, dw1, dw2, gate=g2, dgate=dg,
                             rows_per_gate=R, saved_format=fmt, workspace=ws, residual_scale=residual_scale,
                             block_scale=block_scale, offset=offset)
        return (None if dx is None else _shaped(dx, x_shape), None if dr is None else _shaped(dr, r_shape), dw1, dw2,
                None if dg is None else _shaped(dg, ctx.gate_shape), None, None, None, None, None, None, None)


def rms_norm(x, weight, eps=1e-6, offset=0.0, in_place=False, checkpoint=None):
    """in_place=True writes the input gradient over the incoming output
    gradient (the in-place backward of "fix(cutedsl): fuse Gemma RMSNorm
    weight offset in FP32", Testing Done); only for graphs in which nothing
    else reads that output gradient afterwards.  checkpoint="e4m3" or "int8"
    keeps x for the backward in 8 bits (not with in_place)."""
    fmt = _format(checkpoint)
    if fmt != B.NORM_SAVED_FULL:
        if in_place:
            raise ValueError("checkpoint does not go with in_place")
        if _kept(x, weight):
            return RMSNormCkptFunction.apply(x, weight, eps, offset, fmt)
    return RMSNormFunction.apply(x, weight, eps, offset, in_place)


def layer_norm(x, weight, bias=None, eps=1e-6, offset=0.0, checkpoint=None):
    """checkpoint="e4m3" or "int8" keeps x - mean for the backward in 8 bits."""
    fmt = _format(checkpoint)
    if fmt != B.NORM_SAVED_FULL and _kept(x, weight, bias):
        return LayerNormCkptFunction.apply(x, weight, bias, eps, offset, fmt)
    return LayerNormFunction.apply(x, weight, bias, eps, offset)


def fused_add_rms_norm(x, residual, weight, eps=1e-6, offset=0.0, in_place=False, checkpoint=None):
    """in_place=True writes the input gradient over the incoming gradient of
    the residual stream (h), which it contains; as for rms_norm, only where
    nothing else reads that gradient afterwards.  checkpoint="e4m3" or "int8"
    keeps h for the backward in 8 bits (not with in_place)."""
    fmt = _format(checkpoint)
    if fmt != B.NORM_SAVED_FULL:
        if in_place:
            raise ValueError("checkpoint does not go with in_place")
        if _kept(x, residual, weight):
            return FusedAddRMSNormCkptFunction.apply(x, residual, weight, eps, offset, fmt)
    return FusedAddRMSNormFunction.apply(x, residual, weight, eps, offset, in_place)


def block_rms_norm(x, residual, w_post=None, w_pre=None, gate=None, rows_per_gate=None, residual_scale=1.0,
                   block_scale=1.0, eps=1e-6, offset=0.0, checkpoint=None):
    """The norms before and after a block with its gate and scales:

        h = residual_scale * residual + block_scale * gate * RMSNorm(x; w_post)
        y = RMSNorm(h; w_pre)

    Returns (y, h).  w_post None: x itself; w_pre None: y is None.  gate: [N] (a
    scale per channel), x's shape with trailing row dimensions of 1 ([B, 1, N]:
    one row per sequence; x's shape: per token), or [rows, N] with
    rows_per_gate.  checkpoint="e4m3" or "int8" keeps x and h for the backward in
    8 bits."""
    # (always through the function: an input that carries a forward-mode tangent
    # need not require a gradient, and is refused there)
    return BlockRMSNormFunction.apply(x, residual, w_post, w_pre, gate, rows_per_gate, residual_scale, block_scale, eps,
                                      offset, _format(checkpoint), _kept(x, residual, w_post, w_pre, gate))


class RMSNorm(torch.nn.Module):
    """RMSNorm over the last dimension; offset=1 with zero-initialised weight
    is the Gemma form y = x * rstd * (1 + w)."""

    def __init__(self, hidden, eps=1e-6, offset=0.0, dtype=torch.bfloat16, device="cuda", in_place=False,
                 checkpoint=None):
        super().__init__()
        init = torch.zeros if offset else torch.ones
        self.weight = torch.nn.Parameter(init(hidden, dtype=dtype, device=device))
        self.eps, self.offset, self.in_place, self.checkpoint = eps, offset, in_place, checkpoint

    def forward(self, x):
        return rms_norm(x, self.weight, self.eps, self.offset, self.in_place, self.checkpoint)


class LayerNorm(torch.nn.Module):
    def __init__(self, hidden, eps=1e-6, bias=True, dtype=torch.bfloat16, device="cuda", checkpoint=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, dtype=dtype, device=device)) if bias else None
        self.eps, self.checkpoint = eps, checkpoint

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps, checkpoint=self.checkpoint)


class FusedAddRMSNorm(torch.nn.Module):
    """Returns (normalised, residual stream) for h = x + residual."""

    def __init__(self, hidden, eps=1e-6, offset=0.0, dtype=torch.bfloat16, device="cuda", in_place=False,
                 checkpoint=None):
        super().__init__()
        init = torch.zeros if offset else torch.ones
        self.weight = torch.nn.Parameter(init(hidden, dtype=dtype, device=device))
        self.eps, self.offset, self.in_place, self.checkpoint = eps, offset, in_place, checkpoint

    def forward(self, x, residual):
        return fused_add_rms_norm(x, residual, self.weight, self.eps, self.offset, self.in_place, self.checkpoint)


class BlockRMSNorm(torch.nn.Module):
    """The boundary between two blocks (see block_rms_norm): `post` and `pre`
    norms, a learned scale per channel (channel_scale: its initial value, None
    for none), or a gate passed to forward.  Returns (normalised, residual
    stream)."""

    def __init__(self, hidden, eps=1e-6, offset=0.0, post=True, pre=True, channel_scale=None, residual_scale=1.0,
                 block_scale=1.0, dtype=torch.bfloat16, device="cuda", checkpoint=None):
        super().__init__()
        init = torch.zeros if offset else torch.ones

        def weight(want):
            return torch.nn.Parameter(init(hidden, dtype=dtype, device=device)) if want else None

        self.weight_post, self.weight_pre = weight(post), weight(pre)
        self.channel_scale = None if channel_scale is None else torch.nn.Parameter(
            torch.full((hidden,), float(channel_scale), dtype=dtype, device=device))
        self.eps, self.offset, self.checkpoint = eps, offset, checkpoint
        self.residual_scale, self.block_scale = residual_scale, block_scale

    def forward(self, x, residual, gate=None, rows_per_gate=None):
        if gate is not None and self.channel_scale is not None:
            raise ValueError("a gate does not go with channel_scale")
        return block_rms_norm(x, residual, self.weight_post, self.weight_pre,
                              self.channel_scale if gate is None else gate, rows_per_gate, self.residual_scale,
                              self.block_scale, self.eps, self.offset, self.checkpoint)
