"""User-facing BackLite attention on the bl_attn C ABI.

``BLAttention(negl_prob)`` mirrors the module the "BackLite" README describes
(Usage, Forward signature): it is called as
``attn(query, key, value, scale=None, return_softmax_lse=False, tile_stats=None)``
on (batch, seq_len, heads, head_dim) bf16 tensors, with key/value carrying
``heads_k`` heads.  With negl_prob > 0 the forward records tile statistics
(allocating the buffer unless one is passed, README, Note) and the backward
builds the block-sparse mask from them before running the sparse backward
(How It Works, Phase 2).  With no statistics buffer passed, the forward
keeps only the tile weights d_ij the mask reads (the "Introducing BackLite"
post, Using Sparsity), reduced in its epilogue.  negl_prob = 0 records nothing and runs the dense
backward (Key properties).  ``BL_VERBOSE=1`` prints mask density per head
after each mask pass (README, Debugging, names the same kind of switch).
``causal=True`` (optionally with ``window=W``) gives decoder attention, with
the sliding windows of the "Introducing BackLite" post's Nanochat runs
(Training Nanochat).  ``BLAttention.varlen(q, k, v, cu_seqlens)`` runs the
same chain on a packed variable-length batch ([total, heads, head_dim]
tensors, host offsets cu_seqlens), each sequence attending only to itself.

Around it: ``BLRMSNorm`` and ``BLLayerNorm`` (norms with the residual's addition,
also as the attention's q/k norm), ``BLLinear8`` (linear layers whose products
run on 8-bit codes), ``BLDropout`` (dropout whose mask is never stored), ``Rotary`` (positions on several axes, such
as time, height and width), and activations kept in 8 bits until the backward
(``checkpoint="int8"`` or ``"e4m3"`` of the attention and the norm).

PyTorch only allocates memory and supplies the stream; all arithmetic runs in
libbl_attn.so.
"""
from __future__ import annotations

import math
import os

import torch
from torch.autograd.function import once_differentiable

from . import _lib, linear, ops


def default_tiles(n: int, d: int):
    """Tile sizes used when the caller does not choose: 128 x 128."""
    return 128, 128


class _BLAttnFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, negl_prob, block_q, block_k, tile_stats, causal, window,
                checkpoint=None, checkpoint_out=False, checkpoint_in_forward=False):
        B, n, H, d = q.shape
        Hk = k.shape[2]
        keep, (q, k, v) = _checkpoint_qkv((q, k, v), checkpoint, checkpoint_in_forward)
        shape = _lib.make_shape(B, n, H, Hk, d, block_q, block_k, causal, window)
        o = torch.empty_like(q)
        lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
        stats = logw = None
        if negl_prob > 0:
            T_r, T_c = _lib.tiles(shape)
            if tile_stats is None and _lib.fwd_tile_weights_supported(shape):
                # Only the T_r x T_c tile weights outlive the forward; the
                # statistics rows stay in a scratch freed on return.
                logw = torch.empty((B, H, T_r, T_c), dtype=torch.float32, device=q.device)
                ws = torch.empty(_lib.fwd_workspace_bytes(shape), dtype=torch.uint8,
                                 device=q.device)
                _lib.attn_fwd_tile_weights(shape, q, k, v, scale, o, lse, logw, workspace=ws)
            else:
                want = (B, H, T_c, T_r * block_q)
                stats = tile_stats if tile_stats is not None else torch.empty(
                    want, dtype=torch.float32, device=q.device)
        if logw is None:
            _lib.attn_fwd(shape, q, k, v, scale, o, lse, stats)
        _save_qkvo(ctx, keep, o, lse, checkpoint if checkpoint_out else None)
        ctx.stats, ctx.logw = stats, logw
        ctx.cfg = (shape, scale, negl_prob)
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    def backward(ctx, g_o, _g_lse):
        q, k, v, o, lse = _saved_qkvo(ctx)
        shape, scale, negl_prob = ctx.cfg
        g_o = g_o.contiguous()
        lists = None
        if ctx.stats is not None or ctx.logw is not None:
            lists = _lib.alloc_lists(shape, g_o.device)
            if ctx.logw is not None:
                _lib.mask_from_tile_weights(shape, ctx.logw, negl_prob, lists)
            else:
                _lib.mask_from_stats(shape, ctx.stats, lse, negl_prob, lists)
            if os.environ.get("BL_VERBOSE") == "1":
                m = lists["mask"].float()
                dens = m.mean(dim=(2, 3)).cpu()
                print(f"[bl_attn] mask density per (batch, head): {dens.tolist()} "
                      f"backward skip fraction {1.0 - float(m.mean()):.4f}")
        if isinstance(q, ops.Act8):
            return (*ops.attn_bwd_act8(shape, q, k, v, o, g_o, lse, scale, lists), *[None] * 10)
        g_q = torch.empty_like(q)
        g_k = torch.empty_like(k)
        g_v = torch.empty_like(v)
        ws = torch.empty(_lib.bwd_workspace_bytes(shape), dtype=torch.uint8, device=q.device)
        _lib.attn_bwd(shape, q, k, v, o, g_o, lse, scale, lists, g_q, g_k, g_v, ws)
        return (g_q, g_k, g_v, *[None] * 10)


def _checkpoint_qkv(qkv, checkpoint, in_forward):
    """What is kept of (q, k, v) for the backward, and what the forward reads: with
    ``checkpoint`` Act8s, one scale a (token, head), and ``in_forward`` their values."""
    if checkpoint is None:
        return qkv, qkv
    keep = [ops.act_save(t, checkpoint) for t in qkv]
    return keep, [ops.act_load(t) for t in keep] if in_forward else qkv


def _save_qkvo(ctx, keep, o, lse, o_format):
    """Saves q, k, v (tensors or Act8s), o (in 8 bits with ``o_format``) and lse."""
    keep = (*keep, o if o_format is None else ops.act_save(o, o_format))
    ctx.in8 = tuple(int(isinstance(t, ops.Act8)) for t in keep)
    flat = []
    for t in keep:
        flat += [t.codes, t.scales] if isinstance(t, ops.Act8) else [t]
    ctx.save_for_backward(*flat, lse)


def _saved_qkvo(ctx):
    *flat, lse = ctx.saved_tensors
    got, at = [], 0
    for in8 in ctx.in8:
        got.append(ops.Act8(flat[at], flat[at + 1], 0, torch.bfloat16) if in8 else flat[at])
        at += 1 + in8
    return (*got, lse)


class _BLAttnVarlenFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, vl, scale, negl_prob, checkpoint=None, checkpoint_out=False,
                checkpoint_in_forward=False):
        keep, (q, k, v) = _checkpoint_qkv((q, k, v), checkpoint, checkpoint_in_forward)
        o = torch.empty_like(q)
        lse = torch.empty(vl.sizes["lse"], dtype=torch.float32, device=q.device)
        stats = logw = None
        if negl_prob > 0 and _lib.fwd_tile_weights_supported_varlen(vl):
            logw = torch.empty(vl.sizes["mask"], dtype=torch.float32, device=q.device)
            ws = torch.empty(_lib.fwd_workspace_bytes_varlen(vl), dtype=torch.uint8,
                             device=q.device)
            _lib.attn_fwd_tile_weights_varlen(vl, q, k, v, scale, o, lse, logw, workspace=ws)
        else:
            if negl_prob > 0:
                stats = torch.empty(vl.sizes["tile_stats"], dtype=torch.float32,
                                    device=q.device)
            _lib.attn_fwd_varlen(vl, q, k, v, scale, o, lse, stats)
        _save_qkvo(ctx, keep, o, lse, checkpoint if checkpoint_out else None)
        ctx.stats, ctx.logw = stats, logw
        ctx.cfg = (vl, scale, negl_prob)
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    def backward(ctx, g_o, _g_lse):
        q, k, v, o, lse = _saved_qkvo(ctx)
        q, k, v, o = (ops.act_load(t) if isinstance(t, ops.Act8) else t for t in (q, k, v, o))
        vl, scale, negl_prob = ctx.cfg
        lists = None
        if ctx.stats is not None or ctx.logw is not None:
            lists = _lib.alloc_varlen_lists(vl, q.device)
            if ctx.logw is not None:
                _lib.mask_from_tile_weights_varlen(vl, ctx.logw, negl_prob, lists)
            else:
                _lib.mask_from_stats_varlen(vl, ctx.stats, lse, negl_prob, lists)
        g_q, g_k, g_v = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(vl.sizes["bwd_workspace_bytes"], dtype=torch.uint8, device=q.device)
        _lib.attn_bwd_varlen(vl, q, k, v, o, g_o.contiguous(), lse, scale, lists, g_q, g_k, g_v,
                             ws)
        return (g_q, g_k, g_v, *[None] * 6)


class _RopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, fixed, plan):
        ctx.save_for_backward(positions, fixed)
        ctx.plan = plan
        return ops.rope_with(q, k, positions, plan, fixed)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_q, g_k):
        positions, fixed = ctx.saved_tensors
        g_q, g_k = (g if g is None or g.stride(-1) == 1 else g.contiguous() for g in (g_q, g_k))
        return (*ops.rope_with(g_q, g_k, positions, ctx.plan, fixed, inverse=True), None, None, None)


class Rotary(torch.nn.Module):
    """Rotary positions with one to four axes: ``rotary(q, k, positions)``.  The
    arguments are those of ``ops.RopePlan``; ``positions`` as in ``ops.rope``
    (``ops.grid_positions(T, Y, X)`` gives a video grid's).  q and k may have any
    strides; without a contiguous last dim they are copied first."""

    def __init__(self, head_dim, sections, theta: float = 10000.0, layout: str = "half",
                 shared: bool = False, freqs=None, device=None):
        super().__init__()
        if device is None:
            device = "cuda" if torch.cuda.is_available() else "cpu"
        self.plan = ops.RopePlan(head_dim, sections, theta, layout, shared, freqs, device)
        # a buffer, so that the module moves between devices; the plan, which replicas
        # of the module share, keeps its own
        self.register_buffer("fixed", self.plan.fixed, persistent=False)

    def forward(self, q, k, positions):
        q, k = (t if t is None or t.stride(-1) == 1 else t.contiguous() for t in (q, k))
        return _RopeFn.apply(q, k, positions, self.fixed, self.plan)


class _RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, checkpoint, group):
        ctx.set_materialize_grads(False)
        y, h, rstd = ops.rms_norm_fwd(x, weight, eps, residual)
        ctx.in8 = (group, x.dtype) if checkpoint is not None else None
        if ctx.in8:
            h8 = ops.act_save(h, checkpoint, group)
            ctx.save_for_backward(h8.codes, h8.scales, rstd, weight)
        else:
            ctx.save_for_backward(h, rstd, weight)
        ctx.added = residual is not None
        return (y, h) if ctx.added else y

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y, g_h=None):
        *h, rstd, weight = ctx.saved_tensors
        if g_y is None:                    # only the stream behind the addition was used
            g_w = torch.zeros_like(weight) if ctx.needs_input_grad[1] else None
            return g_h, g_w, g_h, None, None, None
        h = ops.Act8(*h, *ctx.in8) if ctx.in8 else h[0].contiguous()
        g_x, g_w = ops.rms_norm_bwd(g_y.contiguous(), h, rstd, weight,
                                    None if g_h is None else g_h.contiguous(),
                                    need_g_w=ctx.needs_input_grad[1])
        return g_x, g_w, g_x if ctx.added else None, None, None, None


class BLRMSNorm(torch.nn.Module):
    """Root-mean-square norm over the last dim of ``cols`` elements.

    ``norm(x)`` gives y; ``norm(x, residual)`` adds first and gives (y, h) with
    h = x + residual, the stream that goes on.  ``checkpoint`` ("int8" or
    "e4m3") keeps h in 8 bits until the backward, one scale for every ``group``
    elements, and the backward reads the codes as they are."""

    def __init__(self, cols: int, eps: float = 1e-6, checkpoint: str | None = None,
                 group: int = 128, device=None, dtype=None):
        super().__init__()
        if not 1 <= cols <= _lib.NORM_MAX_COLS:
            raise ValueError(f"1 to {_lib.NORM_MAX_COLS} elements, got {cols}")
        _check_checkpoint(checkpoint)
        if group not in (0, 32, 64, 128):
            raise ValueError(f"group must be 0, 32, 64 or 128, got {group}")
        self.cols, self.eps, self.checkpoint, self.group = int(cols), float(eps), checkpoint, group
        self.weight = torch.nn.Parameter(torch.ones(cols, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        if x.shape[-1] != self.cols:
            raise ValueError(f"rows of {x.shape[-1]} elements, the norm has {self.cols}")
        x, residual = (t if t is None or ops.row_stride(t) is not None else t.contiguous()
                       for t in (x, residual))
        checkpoint = self.checkpoint if _wants_backward(x, self.weight, residual) else None
        return _RMSNormFn.apply(x, self.weight, residual, self.eps, checkpoint, self.group)


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps, checkpoint, group):
        ctx.set_materialize_grads(False)
        y, h, mean, rstd = linear.layer_norm_fwd(x, weight, bias, eps, residual)
        ctx.in8 = (group, x.dtype) if checkpoint is not None else None
        if ctx.in8:
            h8 = ops.act_save(h, checkpoint, group)
            ctx.save_for_backward(h8.codes, h8.scales, mean, rstd, weight)
        else:
            ctx.save_for_backward(h, mean, rstd, weight)
        ctx.added = residual is not None
        ctx.bias_type = None if bias is None else bias.dtype
        return (y, h) if ctx.added else y

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y, g_h=None):
        *h, mean, rstd, weight = ctx.saved_tensors
        _, need_w, need_b, *_ = ctx.needs_input_grad
        if g_y is None:                    # only the stream behind the addition was used
            cols = g_h.shape[-1]
            g_w = torch.zeros_like(weight) if need_w else None
            g_b = g_h.new_zeros(cols, dtype=ctx.bias_type) if need_b else None
            return g_h, g_w, g_b, g_h, None, None, None
        h = ops.Act8(*h, *ctx.in8) if ctx.in8 else h[0].contiguous()
        g_x, g_w, g_b = linear.layer_norm_bwd(g_y.contiguous(), h, mean, rstd, weight,
                                              None if g_h is None else g_h.contiguous(),
                                              need_g_w=need_w, need_g_b=need_b)
        if g_b is not None:
            g_b = g_b.to(ctx.bias_type)    # fp32 where there is no weight
        return g_x, g_w, g_b, g_x if ctx.added else None, None, None, None


class BLLayerNorm(torch.nn.Module):
    """Layer norm over the last dim of ``cols`` elements, with a weight and a ``bias``
    unless these are off (``affine=False`` turns both off).

    ``norm(x)`` gives y; ``norm(x, residual)`` adds first and gives (y, h) with
    h = x + residual, the stream that goes on.  ``checkpoint`` ("int8" or
    "e4m3") keeps h in 8 bits until the backward, one scale for every ``group``
    elements, and the backward reads the codes as they are."""

    def __init__(self, cols: int, eps: float = 1e-5, affine: bool = True, bias: bool = True,
                 checkpoint: str | None = None, group: int = 128, device=None, dtype=None):
        super().__init__()
        if not 1 <= cols <= _lib.NORM_MAX_COLS:
            raise ValueError(f"1 to {_lib.NORM_MAX_COLS} elements, got {cols}")
        _check_checkpoint(checkpoint)
        if group not in (0, 32, 64, 128):
            raise ValueError(f"group must be 0, 32, 64 or 128, got {group}")
        self.cols, self.eps, self.checkpoint, self.group = int(cols), float(eps), checkpoint, group
        self.weight = self.bias = None
        if affine:
            self.weight = torch.nn.Parameter(torch.ones(cols, device=device, dtype=dtype))
            if bias:
                self.bias = torch.nn.Parameter(torch.zeros(cols, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        if x.shape[-1] != self.cols:
            raise ValueError(f"rows of {x.shape[-1]} elements, the norm has {self.cols}")
        x, residual = (t if t is None or ops.row_stride(t) is not None else t.contiguous()
                       for t in (x, residual))
        wants = _wants_backward(x, self.weight, self.bias, residual)
        return _LayerNormFn.apply(x, self.weight, self.bias, residual, self.eps,
                                  self.checkpoint if wants else None, self.group)


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, used):
        ctx.save_for_backward(used)
        ctx.p, ctx.added = p, residual is not None
        return linear.dropout(x, p, used, residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y):
        used, = ctx.saved_tensors
        g_x = linear.dropout(g_y.contiguous(), ctx.p, used) if ctx.needs_input_grad[0] else None
        return g_x, g_y if ctx.added else None, None, None


class BLDropout(torch.nn.Module):
    """Dropout whose mask is a function of (seed, offset) and the element's place and is
    formed again in the backward.  ``drop(x)`` or ``drop(x, residual)``, which adds the
    residual behind it.  Every call in training takes the next offset of ``state``, an
    int64 tensor (seed, offset) on the device: a captured graph draws anew with every
    replay, and a saved state brings the same masks back.  ``seed`` None draws one.
    Out of training, and with p = 0, nothing is dropped.

    ``state`` moves with the module and is in its ``state_dict``, but it is none of its
    buffers: data-parallel wrappers send rank 0's buffers to all ranks with every forward,
    which would have all ranks drop the same places.  Ranks drop different ones where their
    seeds differ, and so do layers: a copy (``copy.deepcopy``) has the state of what it was
    copied from, and needs a seed of its own (``drop.state[0] = seed``) to drop others.

    ``used`` is a call's state drawn in advance, ``used = dropout_next(drop.state)``; the
    call then leaves ``state`` as it is.  A forward that the backward runs again
    (``torch.utils.checkpoint`` and its like) needs it, drawn outside of what is run again
    and passed in, so that both runs drop the same places:
    ``checkpoint(lambda x, used: drop(x, used=used), x, dropout_next(drop.state))``.
    Within a backward a call without it is refused, as its mask would be another one."""

    def __init__(self, p: float = 0.1, seed: int | None = None, device=None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must lie in [0, 1], got {p}")
        if device is None:
            device = "cuda" if torch.cuda.is_available() else "cpu"
        if seed is None:
            seed = int(torch.randint(2 ** 63 - 1, ()))
        self.p = float(p)
        self.state = torch.tensor([seed, 0], dtype=torch.int64, device=device)

    def _apply(self, fn, *args, **kwargs):
        super()._apply(fn, *args, **kwargs)
        self.state = fn(self.state)
        return self

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        destination[prefix + "state"] = self.state if keep_vars else self.state.detach()

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys,
                              unexpected_keys, error_msgs):
        name, unexpected = prefix + "state", []
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys,
                                      unexpected, error_msgs)
        unexpected_keys += [k for k in unexpected if k != name]
        state = state_dict.get(name)
        if state is None:
            if strict:
                missing_keys.append(name)
        elif state.dtype != torch.int64 or state.shape != (2,):
            error_msgs.append(f"{name} must be two int64, got {state.dtype} {tuple(state.shape)}")
        elif local_metadata.get("assign_to_params_buffers", False):
            self.state = state.detach()
        else:
            self.state.copy_(state)

    def forward(self, x, residual=None, used=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else x + residual
        if used is None:
            if torch._C._current_graph_task_id() != -1:
                raise RuntimeError(
                    "a forward that a backward runs again needs the state of its first run: "
                    "draw used = dropout_next(drop.state) outside and call drop(x, used=used)")
            used = linear.dropout_next(self.state)
        elif not isinstance(used, torch.Tensor):
            raise TypeError("used must be a tensor, the state that dropout_next gave")
        elif used.data_ptr() == self.state.data_ptr():
            raise ValueError("used is the state that goes on: pass dropout_next(drop.state)")
        x, residual = (t if t is None or ops.row_stride(t) is not None else t.contiguous()
                       for t in (x, residual))
        return _DropoutFn.apply(x, residual, self.p, used)


class _Linear8Fn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, w8, wants):
        need_x, need_w = wants and ctx.needs_input_grad[0], wants and ctx.needs_input_grad[1]
        if w8 is None:
            w8 = linear.weight_save(weight)
        x8, x_cols = linear.act_save_both(x, cols=need_w)
        if need_x or need_w:
            ctx.save_for_backward(*((w8.codes, w8.scales) if need_x else (None, None)),
                                  *((x_cols.codes, x_cols.scales) if need_w else (None, None)))
            ctx.types = x.dtype, weight.dtype
        return linear.matmul8(x8, w8, x.dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y):
        w_codes, w_scales, x_codes, x_scales = ctx.saved_tensors
        need_x, need_w, *_ = ctx.needs_input_grad
        x_type, w_type = ctx.types
        if ops.row_stride(g_y) is None:
            g_y = g_y.contiguous()
        g8, g_cols = linear.act_save_both(g_y, rows=need_x, cols=need_w)
        g_x = g_w = None
        if need_x:
            g_x = linear.matmul8_gx(g8, linear.Weight8(w_codes, w_scales, w_type), x_type)
        if need_w:
            g_w = linear.matmul8_gw(g_cols, linear.Cols8(x_codes, x_scales, x_type), w_type)
        return g_x, g_w, None, None


class BLLinear8(torch.nn.Module):
    """y = x w^T with a weight [out, in] kept in its own type and products on e4m3 codes:
    x and g_y with a scale for every 128 elements of a row (of a column of 128 tokens for
    the weight's gradient), w with one for every 128 x 128.  What waits for the backward
    are codes: a byte an element of x and of w.

    ``linear(x)``; x may also be an Act8 in e4m3 with groups of 128, such as a norm's
    8-bit output, where no backward is wanted.  ``w8``, the ``weight_save`` of the weight,
    spares a call its saving; it has to be that of the weight as it is."""

    def __init__(self, in_features: int, out_features: int, device=None, dtype=None):
        super().__init__()
        if in_features < 1 or out_features < 1:
            raise ValueError(f"at least one feature, got {in_features} and {out_features}")
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.weight = torch.nn.Parameter(
            torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x, w8=None):
        if w8 is not None and (not isinstance(w8, linear.Weight8) or
                               w8.codes.shape != self.weight.shape):
            raise ValueError(f"w8 must be the Weight8 of a weight {tuple(self.weight.shape)}")
        if isinstance(x, ops.Act8):
            if _wants_backward(self.weight):
                raise ValueError("codes carry no gradient: call with x, or without gradients")
            return linear.matmul8(x, linear.weight_save(self.weight) if w8 is None else w8)
        if x.shape[-1] != self.in_features:
            raise ValueError(f"rows of {x.shape[-1]} elements, the layer takes {self.in_features}")
        x = x if ops.row_stride(x) is not None else x.contiguous()
        return _Linear8Fn.apply(x, self.weight, w8, _wants_backward(x, self.weight))


def _wants_backward(*tensors):
    """Whether a backward can follow.  (Within an autograd function the grad mode is off.)"""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _check_checkpoint(checkpoint, out=False, in_forward=False):
    if checkpoint not in (None, "int8", "e4m3"):
        raise ValueError(f'checkpoint must be None, "int8" or "e4m3", got {checkpoint!r}')
    if (out or in_forward) and checkpoint is None:
        raise ValueError("checkpoint_out and checkpoint_in_forward need a checkpoint format")


class BLAttention(torch.nn.Module):
    """Attention whose backward skips the lightest tiles (negl_prob of the mass).

    ``q_norm`` and ``k_norm`` (``BLRMSNorm`` or ``BLLayerNorm`` of head_dim or of
    heads * head_dim elements) and then ``rotary`` (``Rotary``; the call takes ``positions``) are
    applied to the query and the key first.

    ``checkpoint`` ("int8" or "e4m3") keeps the q, k and v that the backward reads
    in 8 bits; ``checkpoint_out`` the output too, which by default stays in bf16,
    the type in which the layer behind usually keeps it anyway.  By default the
    forward stays exact and the gradients carry the rounding: the probabilities
    that the backward forms from the rounded q and k no longer sum to one against
    the exact log-sum-exp, which peaked attention amplifies.  With
    ``checkpoint_in_forward`` the forward reads the rounded q, k and v too: its
    output carries the rounding, and the gradients are exactly those of what it
    computed.  ``calibrate_negl_prob`` measures either."""

    def __init__(self, negl_prob: float = 0.05, block_q: int | None = None,
                 block_k: int | None = None, causal: bool = False, window: int = 0,
                 q_norm: BLRMSNorm | BLLayerNorm | None = None,
                 k_norm: BLRMSNorm | BLLayerNorm | None = None,
                 rotary: Rotary | None = None, checkpoint: str | None = None,
                 checkpoint_out: bool = False, checkpoint_in_forward: bool = False):
        super().__init__()
        _check_checkpoint(checkpoint, checkpoint_out, checkpoint_in_forward)
        if not (0.0 <= negl_prob < 1.0):
            raise ValueError("negl_prob must lie in [0, 1)")
        if window < 0 or (window and not causal):
            raise ValueError("a sliding window needs causal=True")
        self.negl_prob = float(negl_prob)
        self.block_q, self.block_k = block_q, block_k
        self.causal, self.window = bool(causal), int(window)
        self.q_norm, self.k_norm, self.rotary = q_norm, k_norm, rotary
        self.checkpoint, self.checkpoint_out = checkpoint, bool(checkpoint_out)
        self.checkpoint_in_forward = bool(checkpoint_in_forward)

    def _before(self, query, key, positions):
        """q/k norm and rotation of the query and the key."""
        if (positions is None) != (self.rotary is None):
            raise ValueError("positions go with a rotary module" if self.rotary is None else
                             "the rotary module needs positions")
        if self.q_norm is not None:
            query = _norm_heads(self.q_norm, query)
        if self.k_norm is not None:
            key = _norm_heads(self.k_norm, key)
        if self.rotary is not None:
            query, key = self.rotary(query, key, positions)
        return query, key

    def _checkpoints(self, *qkv):
        """(checkpoint, checkpoint_out, checkpoint_in_forward) of a call: nothing is kept
        where no backward can follow, but the forward still reads rounded tensors."""
        if _wants_backward(*qkv):
            return self.checkpoint, self.checkpoint_out, self.checkpoint_in_forward
        return self.checkpoint if self.checkpoint_in_forward else None, False, \
            self.checkpoint_in_forward

    def forward(self, query, key, value, scale=None, return_softmax_lse=False, tile_stats=None,
                positions=None):
        query, key = self._before(query, key, positions)
        d = query.shape[-1]
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        bq, bk = default_tiles(query.shape[1], d)
        bq = self.block_q or bq
        bk = self.block_k or bk
        q, k, v = (t.contiguous() for t in (query, key, value))
        o, lse = _BLAttnFn.apply(q, k, v, float(scale), self.negl_prob, bq, bk, tile_stats,
                                 int(self.causal), self.window, *self._checkpoints(q, k, v))
        return (o, lse) if return_softmax_lse else o

    def varlen(self, query, key, value, cu_seqlens, scale=None, return_softmax_lse=False,
               positions=None):
        """The same attention on a packed batch: query [total, H, d], key/value
        [total, Hk, d], cu_seqlens the nseq + 1 token offsets (a host sequence
        or CPU tensor).  Returns O [total, H, d] and, if asked, the flat LSE
        (per sequence a [H, n_s] block at offset H * cu_seqlens[s]).  ``positions``
        of a rotary module: [total, axes]."""
        query, key = self._before(query, key, positions)
        total, H, d = query.shape
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        bq, bk = default_tiles(total, d)
        vl = _lib.Varlen(cu_seqlens, H, key.shape[1], d, self.block_q or bq, self.block_k or bk,
                         int(self.causal), self.window)
        if vl.total != total:
            raise ValueError(f"cu_seqlens covers {vl.total} tokens, query has {total}")
        q, k, v = (t.contiguous() for t in (query, key, value))
        o, lse = _BLAttnVarlenFn.apply(q, k, v, vl, float(scale), self.negl_prob,
                                       *self._checkpoints(q, k, v))
        return (o, lse) if return_softmax_lse else o


def _norm_heads(norm, t):
    """A q/k norm over every head's own elements, or over all heads' together."""
    if norm.cols == t.shape[-1]:
        return norm(t)
    if norm.cols == t.shape[-1] * t.shape[-2]:
        return norm(t.flatten(-2)).view(t.shape)
    raise ValueError(f"a norm of {norm.cols} elements fits neither a head of {t.shape[-1]} nor "
                     f"{t.shape[-2]} of them")
