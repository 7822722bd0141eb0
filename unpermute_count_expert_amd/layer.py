"""Device-resident MoE expert layer over the C ABI.

Holds one GPU's local expert weights (fp8 e4m3 codes + 128x128 fp32 block
scales) and a workspace sized once for the largest chunk; forward() is one
moe_forward_chunked call on the current stream.

Every tensor is checked (dtype, contiguity, shape against the weights, one
device) before its pointer reaches the library: ids must be int32 (torch.topk
returns int64, which the kernels would read as pairs of int32), router
weights float32, tokens bf16 (or their int16 bits) of width K.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib


class MoeLayer:
    def __init__(self, w13: torch.Tensor, w13_s: torch.Tensor, w2: torch.Tensor, w2_s: torch.Tensor,
                 num_global_experts: int, expert_map: Optional[torch.Tensor] = None, align: int = 128):
        _lib.check_arg(w13, "w13", _lib.E4M3, (None, None, None))
        self.El, twoN, self.K = w13.shape
        if twoN % 256 or self.K % 128:
            raise ValueError(f"w13 has shape {tuple(w13.shape)}; expected (El, 2N, K) with N and K "
                             "multiples of 128")
        self.N = twoN // 2
        _lib.check_arg(w13_s, "w13_s", _lib.F32, (self.El, twoN // 128, self.K // 128))
        _lib.check_arg(w2, "w2", _lib.E4M3, (self.El, self.K, self.N))
        _lib.check_arg(w2_s, "w2_s", _lib.F32, (self.El, self.K // 128, self.N // 128))
        _lib.check_arg(expert_map, "expert_map", _lib.I32, (num_global_experts,), optional=True)
        devs = {t.device for t in (w13, w13_s, w2, w2_s, expert_map) if t is not None}
        if len(devs) != 1:
            raise ValueError(f"the weights are on several devices: {sorted(map(str, devs))}")
        self.device = devs.pop()
        self.w13, self.w13_s, self.w2, self.w2_s = w13, w13_s, w2, w2_s
        self.Eg = num_global_experts
        self.expert_map = expert_map
        self.align = align
        self._ws = None

    def problem(self, M: int, topk: int, chunk_size: int = 0, apply_on_input: int = 0):
        return _lib.problem(M, self.K, self.N, topk, self.Eg, self.El, self.align, apply_on_input,
                            chunk_size)

    def workspace(self, p) -> torch.Tensor:
        n = _lib.moe_forward_workspace_size(p)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        return self._ws

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                chunk_size: int = 0, apply_on_input: int = 0, out: Optional[torch.Tensor] = None,
                per_chunk_counts: Optional[torch.Tensor] = None) -> torch.Tensor:
        _lib.check_arg(x, "x", _lib.BF16, (None, self.K))
        _lib.check_arg(topk_ids, "topk_ids", _lib.I32, (x.shape[0], None))
        M, topk = topk_ids.shape
        p = self.problem(M, topk, chunk_size, apply_on_input)
        if out is None:
            out = torch.empty((M, self.K), dtype=torch.int16, device=x.device)  # bf16 bits
        _lib.check_forward_args(p, x, topk_ids, topk_weights, self.expert_map, self.w13, self.w13_s, self.w2,
                                self.w2_s, out, per_chunk_counts)
        _lib.check_device(x, topk_ids, topk_weights, out, per_chunk_counts, self.w13)
        ws = self.workspace(p)
        _lib.moe_forward_chunked(p, x, topk_ids, topk_weights, self.expert_map, self.w13, self.w13_s,
                                 self.w2, self.w2_s, out, ws, per_chunk_counts)
        return out


@dataclass
class SavedRows:
    """What MoeTrainLayer.backward needs of one forward call.  topk_weights is the caller's own tensor: it and the
    layer's weights stay as they are until then."""
    tokens: int
    topk_weights: torch.Tensor
    counts: torch.Tensor
    expert_offsets: torch.Tensor
    inv_perm: torch.Tensor
    a_perm: torch.Tensor
    h: torch.Tensor
    act: torch.Tensor
    y: torch.Tensor
    rows_hint: int


@dataclass
class SavedCheckpoint:
    """The same where the layer keeps a checkpoint: the tokens (the caller's own tensor, which stays as it is until
    then, or codes with their scales x_s) and the experts' gate and up rows (bf16, or codes with h_s)."""
    tokens: int
    topk_weights: torch.Tensor
    counts: torch.Tensor
    expert_offsets: torch.Tensor
    inv_perm: torch.Tensor
    x: torch.Tensor
    x_s: Optional[torch.Tensor]
    h: torch.Tensor
    h_s: Optional[torch.Tensor]
    rows_hint: int


class MoeTrainLayer:
    """One GPU's local experts in bf16, forward and backward.

    w13 [El, 2N, K] (gate rows, then up rows) and w2 [El, K, N] bf16.
    forward() returns the output and the rows that its backward() needs, so
    several forwards may run before their backwards; backward() returns the
    gradients of the tokens and of the router weights and adds those of the
    expert weights to the fp32 grad_w13 / grad_w2 (zero_grad() clears them);
    clip_gradients() scales them in place to a global norm.  Every step is a
    library call on the current stream.  N and K: multiples of 128.

    checkpoint: what a forward call keeps of its rows for backward().
      None    the permuted tokens, gate and up rows, activations and expert
              outputs in bf16, 4 K + 6 N bytes a row;
      "bf16"  gate and up rows, 4 N bytes a row, and the caller's tokens;
      "e4m3"  gate and up rows, 2 N bytes a row, and the tokens, K bytes
              each, in 8 bits with a scale byte for every 32 values.
    With a checkpoint the gate and up products and the activation are one
    kernel, as are the down product's gradient and the activation's, which
    recomputes the activations; the router weights' gradient comes from the
    down product's gradient instead of its outputs.  8 bits round what the
    gradients are taken at by up to 2^-4 of each value, or 2^-10 of its
    block's scale where that is more, so small values beside large ones among
    32 become 0; magnitudes past 3.29e38 become infinite.  The output is the
    same with either checkpoint.

    infer() is the forward pass alone: it keeps nothing.

    With gradients enabled and any of tokens, router weights and expert
    weights requiring them, forward()'s output carries a graph whose backward
    is backward(): the tokens and router weights get their gradients through
    autograd.  The expert weights' are in grad_w13 / grad_w2 alike (their own
    .grad stays as it is: it would hold a bf16 sum).
    """

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, num_global_experts: int,
                 expert_map: Optional[torch.Tensor] = None, align: int = 16, checkpoint: Optional[str] = None):
        if checkpoint not in (None, "bf16", "e4m3"):
            raise ValueError(f"checkpoint is {checkpoint!r}; expected None, 'bf16' or 'e4m3'")
        self.checkpoint = checkpoint
        bf = (torch.bfloat16,)
        _lib.check_arg(w13, "w13", bf, (None, None, None))
        self.El, twoN, self.K = w13.shape
        if twoN % 256 or self.K % 128:
            raise ValueError(f"w13 has shape {tuple(w13.shape)}; expected (El, 2N, K) with N and K "
                             "multiples of 128")
        self.N = twoN // 2
        _lib.check_arg(w2, "w2", bf, (self.El, self.K, self.N))
        _lib.check_arg(expert_map, "expert_map", _lib.I32, (num_global_experts,), optional=True)
        devs = {t.device for t in (w13, w2, expert_map) if t is not None}
        if len(devs) != 1:
            raise ValueError(f"the weights are on several devices: {sorted(map(str, devs))}")
        self.device = devs.pop()
        self.w13, self.w2 = w13, w2
        self.Eg = num_global_experts
        self.expert_map = expert_map
        self.align = align
        self.grad_w13 = torch.zeros(w13.shape, dtype=torch.float32, device=self.device)
        self.grad_w2 = torch.zeros(w2.shape, dtype=torch.float32, device=self.device)

    def _empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def zero_grad(self):
        self.grad_w13.zero_()
        self.grad_w2.zero_()

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor):
        """(out [M, K] bf16, the rows backward() needs)."""
        self._check_tokens(x, topk_ids, topk_weights)
        if torch.is_grad_enabled():
            weights = self.w13.requires_grad or self.w2.requires_grad
            if weights or x.requires_grad or topk_weights.requires_grad:
                return _Graph.apply(x, topk_weights, _anchor() if weights else None, topk_ids, self)
        return self._forward(x, topk_ids, topk_weights)

    def infer(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor) -> torch.Tensor:
        """The output [M, K] bf16 of a forward call with a checkpoint, none kept and no graph."""
        self._check_tokens(x, topk_ids, topk_weights)
        return self._gated_forward(x, topk_ids, topk_weights, None, None)[0]

    def _check_tokens(self, x, topk_ids, topk_weights):
        _lib.check_arg(x, "x", (torch.bfloat16,), (None, self.K))
        _lib.check_arg(topk_ids, "topk_ids", _lib.I32, (x.shape[0], None))
        _lib.check_arg(topk_weights, "topk_weights", _lib.F32, topk_ids.shape)
        _lib.check_device(x, topk_ids, topk_weights, self.w13)

    def _gated_forward(self, x, topk_ids, topk_weights, h, h_s):
        """(out, counts, expert_offsets, inv_perm, rows_hint), with gate and up rows kept in h and h_s if given."""
        M, topk = topk_ids.shape
        El, K, N, i32 = self.El, self.K, self.N, torch.int32
        cap = _lib.moe_max_rows(M, topk, El, self.align)
        hint = max(1, M * topk * El // self.Eg)
        counts, offsets, inv = (self._empty(*n, dtype=i32) for n in ((El,), (El + 1,), (M, topk)))
        a, act = self._empty(cap, K), self._empty(cap, N)
        ws = self._empty(_lib.moe_permute_workspace_size(M, topk, El), dtype=torch.uint8)
        _lib.moe_permute_bf16(x, topk_ids, self.expert_map, self.Eg, El, self.align, cap, a, counts, offsets, inv,
                              self._empty(cap, dtype=i32), ws)
        _lib.moe_grouped_gemm_bf16_silu_mul(a, self.w13, offsets, counts, act, h, h_s, hint)
        _lib.moe_grouped_gemm_bf16(act, self.w2, offsets, counts, a, hint)   # the experts' outputs, in the tokens' place
        out = self._empty(M, K)
        _lib.moe_unpermute_weight_reduce(a, inv, topk_weights, 0, out)
        return out, counts, offsets, inv, hint

    def _forward(self, x, topk_ids, topk_weights):
        M, topk = topk_ids.shape
        El, K, N, i32 = self.El, self.K, self.N, torch.int32
        cap = _lib.moe_max_rows(M, topk, El, self.align)
        if self.checkpoint is not None:
            h_s = x_s = None
            if self.checkpoint == "e4m3":
                u8, block = torch.uint8, _lib.CHECKPOINT_BLOCK
                h, h_s = self._empty(cap, 2 * N, dtype=u8), self._empty(cap, 2 * N // block, dtype=u8)
                kept, x_s = self._empty(M, K, dtype=u8), self._empty(M, K // block, dtype=u8)
                _lib.moe_checkpoint(x, kept, x_s)
            else:
                h, kept = self._empty(cap, 2 * N), x
            out, counts, offsets, inv, hint = self._gated_forward(x, topk_ids, topk_weights, h, h_s)
            return out, SavedCheckpoint(M, topk_weights, counts, offsets, inv, kept, x_s, h, h_s, hint)
        s = SavedRows(M, topk_weights, self._empty(El, dtype=i32), self._empty(El + 1, dtype=i32),
                      self._empty(M, topk, dtype=i32), self._empty(cap, K), self._empty(cap, 2 * N),
                      self._empty(cap, N), self._empty(cap, K), max(1, M * topk * El // self.Eg))
        ws = self._empty(_lib.moe_permute_workspace_size(M, topk, El), dtype=torch.uint8)
        _lib.moe_permute_bf16(x, topk_ids, self.expert_map, self.Eg, El, self.align, cap, s.a_perm, s.counts,
                              s.expert_offsets, s.inv_perm, self._empty(cap, dtype=i32), ws)
        seg = (s.expert_offsets, s.counts)
        _lib.moe_grouped_gemm_bf16(s.a_perm, self.w13, *seg, s.h, s.rows_hint)
        _lib.moe_silu_mul(s.h, N, s.act, *seg, El)
        _lib.moe_grouped_gemm_bf16(s.act, self.w2, *seg, s.y, s.rows_hint)
        out = self._empty(M, K)
        _lib.moe_unpermute_weight_reduce(s.y, s.inv_perm, topk_weights, 0, out)
        return out, s

    def backward(self, dout: torch.Tensor, s):
        """(dx [M, K] bf16, gradient of topk_weights [M, topk] fp32); adds to grad_w13 and grad_w2."""
        _lib.check_arg(dout, "dout", (torch.bfloat16,), (s.tokens, self.K))
        _lib.check_device(dout, self.w13)
        if isinstance(s, SavedCheckpoint):
            return self._backward_checkpoint(dout, s)
        El, N = self.El, self.N
        seg = (s.expert_offsets, s.counts)
        dy, dweights = torch.empty_like(s.y), torch.empty_like(s.topk_weights)
        _lib.moe_unpermute_weight_reduce_bwd(dout, s.y, s.inv_perm, s.topk_weights, dy, dweights)
        dact, dh = torch.empty_like(s.act), torch.empty_like(s.h)
        _lib.moe_grouped_gemm_bf16_dgrad(dy, self.w2, *seg, dact, s.rows_hint)
        _lib.moe_grouped_gemm_bf16_wgrad(dy, s.act, *seg, self.grad_w2, 1, s.rows_hint)
        _lib.moe_silu_mul_bwd(s.h, dact, N, dh, *seg, El)
        _lib.moe_grouped_gemm_bf16_wgrad(dh, s.a_perm, *seg, self.grad_w13, 1, s.rows_hint)
        da, dx = torch.empty_like(s.a_perm), torch.empty_like(dout)
        _lib.moe_grouped_gemm_bf16_dgrad(dh, self.w13, *seg, da, s.rows_hint)
        # a token's row was copied to each of its experts: its gradient is the plain sum of theirs
        _lib.moe_unpermute_weight_reduce(da, s.inv_perm, None, 1, dx)
        return dx, dweights

    def _backward_checkpoint(self, dout, s):
        K, N, f32 = self.K, self.N, torch.float32
        cap = s.h.shape[0]
        seg = (s.expert_offsets, s.counts)
        d, weights = self._empty(cap, K), self._empty(cap, dtype=f32)
        _lib.moe_permute_rows(dout, s.inv_perm, d, s.topk_weights, weights)
        dh, act, dots = self._empty(cap, 2 * N), self._empty(cap, N), self._empty(cap, -(-N // 64), dtype=f32)
        _lib.moe_grouped_gemm_bf16_dgrad_silu_mul(d, self.w2, *seg, s.h, dh, act, s.h_s, weights, dots, s.rows_hint)
        dweights = torch.empty_like(s.topk_weights)
        _lib.moe_topk_weights_bwd(dots, s.inv_perm, dweights)
        _lib.moe_grouped_gemm_bf16_wgrad(d, act, *seg, self.grad_w2, 1, s.rows_hint)   # act has the router weights
        a = self._empty(cap, K)
        if s.x_s is None:
            _lib.moe_permute_rows(s.x, s.inv_perm, a)
        else:
            _lib.moe_checkpoint_restore(s.x, s.x_s, a, s.inv_perm)
        _lib.moe_grouped_gemm_bf16_wgrad(dh, a, *seg, self.grad_w13, 1, s.rows_hint)
        dx = torch.empty_like(dout)
        _lib.moe_grouped_gemm_bf16_dgrad(dh, self.w13, *seg, d, s.rows_hint)   # d is read: its rows' gradients
        _lib.moe_unpermute_weight_reduce(d, s.inv_perm, None, 1, dx)
        return dx, dweights

    def clip_gradients(self, max_norm: float, extra=(), reduce=None) -> torch.Tensor:
        """Scales grad_w13, grad_w2 and the tensors of `extra` in place to a global 2-norm of at most max_norm
        and returns the norm before [1] fp32.  reduce(sumsq), if given, runs between the two steps on the
        float64 sum of squares [1]: ranks that hold other experts add theirs there."""
        grads = [self.grad_w13, self.grad_w2, *extra]
        sumsq, norm = self._empty(1, dtype=torch.float64), self._empty(1, dtype=torch.float32)
        _lib.moe_grad_sumsq(grads, sumsq, self._empty(_lib.moe_grad_workspace_size(len(grads)), dtype=torch.uint8))
        if reduce is not None:
            reduce(sumsq)
        _lib.moe_grad_clip(grads, None, sumsq, max_norm, norm)
        return norm


def _anchor() -> torch.Tensor:
    """What makes the output require a gradient for the expert weights.  They are no inputs of the graph, as nothing
    goes to their .grad; a new leaf a call also keeps graphs of one layer apart (a captured backward must share no
    leaf with an eager graph that lives)."""
    return torch.empty(0, requires_grad=True)


class _Graph(torch.autograd.Function):
    """MoeTrainLayer.forward and backward as one node.  What backward reads besides the rows is saved with its
    version, so that weights changed in between are an error."""

    @staticmethod
    def forward(ctx, x, topk_weights, anchor, topk_ids, layer):
        out, ctx.rows = layer._forward(x, topk_ids, topk_weights)
        ctx.layer = layer
        kept = (x,) if layer.checkpoint == "bf16" else ()
        ctx.save_for_backward(topk_weights, layer.w13.detach(), layer.w2.detach(), *kept)
        return out, ctx.rows

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _):
        ctx.saved_tensors   # the check of their versions
        dx, dweights = ctx.layer.backward(dout.contiguous(), ctx.rows)
        return dx, dweights, None, None, None
