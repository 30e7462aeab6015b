"""FP8GatedMLP: a gated feed-forward block on the library's FP8 path.

y = (act(x Wg^T) * (x Wu^T)) Wd^T under the DelayedScaling recipe with the
HYBRID format, as FP8Linear runs one linear: E4M3 for the input, the weights
and the hidden state, E5M2 for the gradients. Forward: the cast of x, both
projections with the gate in one launch (fp8_gated_fwd), the down projection.
Backward: the cast of dy, its way through the down projection and the gate in
one launch (fp8_gated_dgrad), dWd, then dx and dWg, dWu in one launch
(fp8_gated_bwd). Any number of tokens; up to FEW_TOKENS of them (serving)
stream the weights at the memory's rate. With a norm before it, the residual's
addition, the norm and the cast of its output are one launch (fp8_rmsnorm_fwd),
and so is their backward pass, the residual stream's gradient included. This file
only allocates the outputs through torch and passes pointers.
"""

from __future__ import annotations

import torch

from . import (AMAX_MAX, E4M3, E5M2, FEW_TOKENS, GELU_TANH, MAX_NORM_COLS, SILU, Meta, _stream,
               delayed_scaling_update, fp8_gated_bwd, fp8_gated_dgrad, fp8_gated_fwd, fp8_linear_bwd_rowmajor,
               fp8_linear_few, fp8_linear_fwd, fp8_quantize, fp8_rmsnorm_bwd, fp8_rmsnorm_bwd_workspace_bytes,
               fp8_rmsnorm_fwd)
from .linear import first_order, refuse_capture, watch_leaves

__all__ = ["FP8GatedMLP"]


def _rows16(rows: int, cols: int, dtype: torch.dtype, device) -> torch.Tensor:
    """[rows rounded up to 16, cols], the added rows zero: fp8_linear_fwd and
    fp8_linear_bwd_rowmajor take multiples of 16 tokens."""
    t = torch.empty(((rows + 15) // 16 * 16, cols), dtype=dtype, device=device)
    if t.shape[0] != rows:
        t[rows:].zero_()
    return t


class _CopyState:
    """Which state of a weight its copy is of, and when it is there. The weight's
    array is kept alive, so that another one under the same parameter (.data =
    ..., which leaves the version as it is) cannot have its address."""

    def __init__(self):
        self.version = self.array = self.event = None
        self.streams, self.wait = (), False  # those that the copy is there for; whether others wait for the event

    def __reduce__(self):  # a copy of the module casts its own
        return _CopyState, ()

    def note(self, w: torch.Tensor, cast: bool) -> None:
        """What has been enqueued on the current stream makes the copy w's: a cast,
        which only this module knows of, or a step, which its caller orders before
        the weight's uses."""
        self.version, self.array, self.wait = w._version, w.detach(), cast
        if w.is_cuda:
            self.streams = {_stream(None)}
            if cast:
                self.event = self.event or torch.cuda.Event()
                self.event.record()

    def forget(self) -> None:
        self.array = None

    def is_current(self, w: torch.Tensor) -> bool:
        a = self.array
        return a is not None and self.version == w._version and a.dtype == w.dtype and a.is_set_to(w)

    def use(self, copy: torch.Tensor) -> None:
        """The copy is about to be read on the current stream, which is not among
        `streams`: that one waits for its cast and keeps the array from being reused."""
        if not copy.is_cuda:
            return
        stream = torch.cuda.current_stream()
        if self.wait:
            stream.wait_event(self.event)
        copy.record_stream(stream)
        self.streams.add(stream.cuda_stream)


def _capturing(w: torch.Tensor) -> bool:
    return w.is_cuda and torch.cuda.is_current_stream_capturing()


def _rows(x: torch.Tensor, cols: int) -> torch.Tensor:
    """x as dense rows on a 16-byte boundary."""
    x2 = x.reshape(-1, cols)
    if x2.is_contiguous() and x2.data_ptr() % 16 == 0:
        return x2
    return x2.clone(memory_format=torch.contiguous_format)


def _codes_of(x2, residual, norm, eps, meta, X8):
    """The E4M3 codes of a linear's input in X8: of x2, or of the norm of x2 plus the
    residual, whose sum and rstd are returned (without a norm: None, None)."""
    if norm is None:
        fp8_quantize(x2, E4M3, meta.scale, X8, None, meta.cur_amax)
        return None, None
    rstd = torch.empty(x2.shape[0], dtype=torch.float32, device=x2.device)
    total = torch.empty_like(residual) if residual is not None else None
    fp8_rmsnorm_fwd(x2, norm, X8, rstd, eps=eps, residual=residual, total=total, y_scale=meta.scale, y_amax=meta.cur_amax)
    return total, rstd


def _norm_grads(dxn, total, dtotal, norm, rstd, x_dtype, need_norm, shape):
    """(dx, dresidual, dnorm) of _codes_of's norm from the gradient of its output and of
    the sum. Of one type, dx and dresidual are one tensor, as an addition's gradients
    are: two views of its memory would each be taken for a gradient of its own."""
    M, K = dxn.shape
    dresidual = torch.empty_like(total)
    dx = torch.empty((M, K), dtype=x_dtype, device=dxn.device) if x_dtype != total.dtype else None
    dnorm = workspace = None
    if need_norm:
        dnorm = torch.empty_like(norm)
        workspace = torch.empty(fp8_rmsnorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device=dxn.device)
    if dtotal is not None:
        dtotal = _rows(dtotal.to(total.dtype), K)
    fp8_rmsnorm_bwd(dxn, total, norm, rstd, dresidual, dnorm, workspace, dtotal=dtotal, dx=dx)
    dresidual = dresidual.reshape(shape)
    return dresidual if dx is None else dx.reshape(shape), dresidual, dnorm


def _check_norm_weight(norm, x, features: int) -> None:
    if norm is not None and (norm.shape != (features,) or norm.device != x.device):
        raise ValueError(f"norm must be ({features},) on {x.device}, got {tuple(norm.shape)} on {norm.device}")


def _check_norm(features: int, eps: float | None) -> None:
    if eps is not None and not (0.0 <= eps < float("inf") and features <= MAX_NORM_COLS):
        raise ValueError(f"a norm needs an eps >= 0 and at most {MAX_NORM_COLS} features")


def _check_input(x, residual, features, device, norm) -> None:
    if x.dim() == 0 or x.shape[-1] != features or x.device != device:
        raise ValueError(f"x must be [..., {features}] on {device}, got {tuple(x.shape)} on {x.device}")
    if residual is None:
        return
    if norm is None:
        raise ValueError("a residual needs the block's norm (norm_eps)")
    if residual.shape != x.shape or residual.device != x.device or residual.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"residual must be bf16 or fp32 {tuple(x.shape)} on {x.device}, got {residual.dtype} "
                         f"{tuple(residual.shape)} on {residual.device}")


class _FP8GatedMLPFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, norm, gate_up, down, mlp, keep):
        K, F = mlp.features, mlp.hidden
        x2 = _rows(x, K)
        M, dev = x2.shape[0], x.device
        gu8, d8 = mlp.weight_copies(keep)
        X8 = torch.empty((M, K), dtype=torch.uint8, device=dev)
        norm = norm.detach().contiguous() if norm is not None else None
        total, rstd = _codes_of(x2, _rows(residual, K) if residual is not None else None, norm, mlp.norm_eps, mlp.meta_x, X8)
        few = M <= FEW_TOKENS
        H8 = torch.empty((M, F), dtype=torch.uint8, device=dev) if few and not keep else _rows16(M, F, torch.uint8, dev)
        gu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if keep else None
        fp8_gated_fwd(X8, gu8, mlp.meta_x.scale_inv, mlp.meta_gate_up.scale_inv, H8[:M], act=mlp.act,
                      h_scale=mlp.meta_h.scale, h_amax=mlp.meta_h.cur_amax, gu=gu)
        y = torch.empty((M if few else H8.shape[0], K), dtype=x.dtype, device=dev)
        (fp8_linear_few if few else fp8_linear_fwd)(H8[:M] if few else H8, d8, mlp.meta_h.scale_inv,
                                                    mlp.meta_down.scale_inv, y)
        if total is not None:
            total = total.reshape(x.shape)
        if keep:
            # the codes were made with this step's scales: keep those for backward
            factors = torch.cat([mlp.meta_x.scale_inv, mlp.meta_gate_up.scale_inv, mlp.meta_h.scale_inv,
                                 mlp.meta_down.scale_inv])
            normed = None if norm is None else x2 if total is None else total
            ctx.save_for_backward(X8, gu, H8, gu8, d8, factors, normed, rstd, norm)
            ctx.mlp = mlp
            ctx.like = (x.shape, x.dtype, gate_up.dtype, down.dtype)
            watch_leaves(ctx)
            ctx.set_materialize_grads(False)
        y = y[:M].reshape(x.shape)
        return y if total is None else (y, total)

    @staticmethod
    def backward(ctx, dy, dtotal=None):
        refuse_capture(ctx)
        X8, gu, H8, gu8, d8, factors, normed, rstd, norm = ctx.saved_tensors
        mlp = ctx.mlp
        x_shape, x_dtype, gate_up_dtype, down_dtype = ctx.like
        need_x, need_residual, need_norm, need_gate_up, need_down = ctx.needs_input_grad[:5]
        K, F, M, dev = mlp.features, mlp.hidden, X8.shape[0], X8.device
        if dy is None:  # only the sum was used: its gradient is the residual's and x's, and may be differentiated again
            dx, dresidual = (dtotal.to(t) if n and dtotal is not None else None
                             for n, t in ((need_x, x_dtype), (need_residual, normed.dtype if normed is not None else x_dtype)))
            return dx, dresidual, None, None, None, None, None
        sinv_x, sinv_gu, sinv_h, sinv_d = factors[0:1], factors[1:2], factors[2:3], factors[3:4]
        dy2 = _rows(dy.to(x_dtype), K)
        md, mg = mlp.meta_dy, mlp.meta_dgu
        D8 = _rows16(M, K, torch.uint8, dev)
        fp8_quantize(dy2, E5M2, md.scale, D8[:M], None, md.cur_amax)
        dx = dresidual = dnorm = dgate_up = ddown = None
        if need_down:
            ddown = torch.empty((K, F), dtype=down_dtype, device=dev)
            fp8_linear_bwd_rowmajor(D8, None, H8, md.scale_inv, None, sinv_h, None, ddown, dw_nonfinite=mlp.dw_nonfinite)
        need_in = need_x or need_residual or need_norm
        if need_in or need_gate_up:
            G8 = torch.empty((M, 2 * F), dtype=torch.uint8, device=dev)
            fp8_gated_dgrad(D8[:M], d8, gu, md.scale_inv, sinv_d, mg.scale, G8, act=mlp.act, dgu_amax=mg.cur_amax)
            if need_in:
                dx = torch.empty((M, K), dtype=x_dtype, device=dev)
            if need_gate_up:
                dgate_up = torch.empty((2 * F, K), dtype=gate_up_dtype, device=dev)
            fp8_gated_bwd(None, None, X8, gu8, sinv_x, sinv_gu, None, mg.scale_inv, G8, dx, dgate_up, act=mlp.act,
                          dw_nonfinite=mlp.dw_nonfinite if dgate_up is not None else None)
        if need_in and norm is not None:
            dx, dresidual, dnorm = _norm_grads(dx, _rows(normed, K), dtotal, norm, rstd, x_dtype, need_norm, x_shape)
        elif dx is not None:
            dx = dx.reshape(x_shape)
        return *first_order(dx if need_x else None, dresidual if need_residual else None, dnorm, dgate_up, ddown), None, None


class _WeightCopies:
    """The E4M3 copies of a module's weights. The module gives _weights() (a tuple of
    (weight, meta)) and calls _make_copies() when it has them."""

    def _make_copies(self, device) -> None:
        weights = self._weights()
        # of each weight: the E4M3 copy, and what it is of
        self._copies = [torch.empty(w.shape, dtype=torch.uint8, device=device) for w, _ in weights]
        self._cast_of = [_CopyState() for _ in weights]
        self._in_a_graph = [False] * len(weights)  # a captured graph reads the copy's array
        self._trains_in_a_graph = False  # replays change the weights and their scales unseen

    def weight_copies(self, for_training: bool = False):
        """The weights' E4M3 copies under their metas' scales, cast if they are
        not current. A capture casts them in the graph, but for a pass without
        gradients in eval mode: that graph reads the current ones, which every
        later cast then writes in place."""
        weights = self._weights()
        capturing = _capturing(weights[0][0])
        here = _stream(None) if weights[0][0].is_cuda else None
        for i, (w, m) in enumerate(weights):
            w8, state = self._copies[i], self._cast_of[i]
            current = state.is_current(w)
            if capturing:
                current = current and not for_training and not self.training
                self._trains_in_a_graph = self._trains_in_a_graph or for_training
                self._in_a_graph[i] = self._in_a_graph[i] or current
            elif current and here not in state.streams:
                state.use(w8)
            if not current:
                if w.shape != w8.shape or w.device != w8.device:
                    raise ValueError(f"a weight must stay {tuple(w8.shape)} on {w8.device}, got {tuple(w.shape)} on "
                                     f"{w.device}")
                # a new array, as a backward pass may still hold the last one; but a
                # graph's stays (and a backward pass that holds it fails)
                if self._in_a_graph[i]:
                    torch.autograd.graph.increment_version(w8)
                else:
                    with torch.inference_mode(False):  # (an evaluation's copy serves training too)
                        w8 = self._copies[i] = torch.empty_like(w8)
                fp8_quantize(w.detach().contiguous(), E4M3, m.scale, w8, None, m.cur_amax)
                self._note(i, w, capturing, cast=True)
        return tuple(self._copies)

    def copies_for_step(self):
        """(weight, E4M3 copy, meta) for an optimizer that writes the copies; it
        calls copies_written() when it has."""
        return [(w, w8, m) for (w, m), w8 in zip(self._weights(), self._copies)]

    def copies_written(self, weights=None) -> None:
        """The copies of `weights` (all, if None) are of the weights as they are
        now; the others are as current as they were. A backward pass that still
        needs the ones before fails, as after any change in place."""
        capturing = _capturing(self._weights()[0][0])
        if capturing:
            self._trains_in_a_graph = True
        for i, (w, _) in enumerate(self._weights()):
            if weights is None or any(w is x for x in weights):
                torch.autograd.graph.increment_version(self._copies[i])
                self._note(i, w, capturing, cast=False)

    def _note(self, i: int, w: torch.Tensor, capturing: bool, cast: bool) -> None:
        # (what a capture records has not run, and what its replays do is not seen)
        if capturing or self._trains_in_a_graph:
            self._cast_of[i].forget()
        else:
            self._cast_of[i].note(w, cast)

    def weights_changed(self) -> None:
        """Cast the weights again before their next use: for changes that torch does
        not see, as through .data or a pointer; its own are noticed."""
        for state in self._cast_of:
            state.forget()

    def _apply(self, fn, *args, **kw):  # .to() and the like: the arrays before are let go
        self.weights_changed()
        return super()._apply(fn, *args, **kw)

    def update_scales(self) -> None:
        """Roll the amax histories and refresh the scales for the next step; the
        weights' copies, cast under the old ones, are not current after it."""
        delayed_scaling_update(self.metas(), self.algo, self.margin)
        if _capturing(self._weights()[0][0]):
            self._trains_in_a_graph = True
        self.weights_changed()


class FP8GatedMLP(_WeightCopies, torch.nn.Module):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T with FP8 GEMMs under delayed scaling.

    features and hidden must be multiples of 16. gate_up [2 hidden, features]
    holds Wg above Wu, down [features, hidden] Wd, in high precision; their E4M3
    copies are cast when they are not current. Call update_scales() once per
    training step, after backward; an optimizer that writes the copies itself
    (AdamW) does so after it. x is bf16 or fp32. In a CUDA graph the casts are
    part of the graph, unless it is captured in eval mode without gradients
    (serving): then it reads the copies that are current, and after a change of
    the weights weight_copies() casts them for its next replay. A captured backward
    pass is refused where torch would end the process: a pass of this library's modules
    with the same weights or inputs that was made before on the default stream still had
    its graph. What torch's own operations hold of a weight (a penalty on it, a view of it
    as the input) is not seen: drop their results before a capture, too.

    With norm_eps the block begins with a root-mean-square norm (weight: norm
    [features]) and takes part in a residual stream: block(x, residual) gives
    (MLP(norm(t)), t) with t = x + residual in the residual's type, both of which the
    next block takes; without a residual t is x.
    """

    def __init__(self, features: int, hidden: int, act: int = SILU, history_len: int = 16,
                 amax_compute_algo: int = AMAX_MAX, margin: int = 0, device="cuda", dtype: torch.dtype = torch.float32,
                 norm_eps: float | None = None):
        super().__init__()
        if features % 16 or hidden % 16:
            raise ValueError("FP8 linears need features and hidden divisible by 16")
        _check_norm(features, norm_eps)
        if act not in (SILU, GELU_TANH):
            raise ValueError(f"unknown activation {act}")
        self.features, self.hidden, self.act = features, hidden, act
        self.algo, self.margin = amax_compute_algo, margin

        def weight(rows, cols):
            bound = 1.0 / cols ** 0.5
            return torch.nn.Parameter(torch.empty((rows, cols), device=device, dtype=dtype).uniform_(-bound, bound))

        self.gate_up, self.down = weight(2 * hidden, features), weight(features, hidden)
        self.norm_eps = norm_eps
        self.norm = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype)) if norm_eps is not None else None
        self.meta_x, self.meta_gate_up = Meta(history_len, E4M3, device), Meta(history_len, E4M3, device)
        self.meta_h, self.meta_down = Meta(history_len, E4M3, device), Meta(history_len, E4M3, device)
        self.meta_dy, self.meta_dgu = Meta(history_len, E5M2, device), Meta(history_len, E5M2, device)
        # 1 once a weight gradient held an Inf or NaN, until its reader clears it
        # (AdamW finds the step's by its own pass over the gradients)
        self.dw_nonfinite = torch.zeros(1, dtype=torch.int32, device=device)
        self._make_copies(device)

    def metas(self):
        return [self.meta_x, self.meta_gate_up, self.meta_h, self.meta_down, self.meta_dy, self.meta_dgu]

    def _weights(self):
        return (self.gate_up, self.meta_gate_up), (self.down, self.meta_down)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        _check_input(x, residual, self.features, self._copies[0].device, self.norm)
        _check_norm_weight(self.norm, x, self.features)
        inputs = (x, residual, self.norm, self.gate_up, self.down)
        keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)
        out = _FP8GatedMLPFn.apply(*inputs, self, keep)
        return (out, x) if self.norm is not None and residual is None else out
