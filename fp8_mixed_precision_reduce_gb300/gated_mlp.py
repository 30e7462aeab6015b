"""FP8GatedMLP: a gated feed-forward block on the library's FP8 path.

y = (act(x Wg^T) * (x Wu^T)) Wd^T under the DelayedScaling recipe with the
HYBRID format, as FP8Linear runs one linear: E4M3 for the input, the weights
and the hidden state, E5M2 for the gradients. Forward: the cast of x, both
projections with the gate in one launch (fp8_gated_fwd), the down projection.
Backward: the cast of dy, its way through the down projection and the gate in
one launch (fp8_gated_dgrad), dWd, then dx and dWg, dWu in one launch
(fp8_gated_bwd). Any number of tokens; up to FEW_TOKENS of them (serving)
stream the weights at the memory's rate. This file only allocates the outputs
through torch and passes pointers.
"""

from __future__ import annotations

import torch

from . import (AMAX_MAX, E4M3, E5M2, FEW_TOKENS, GELU_TANH, SILU, Meta, _stream, delayed_scaling_update,
               fp8_gated_bwd, fp8_gated_dgrad, fp8_gated_fwd, fp8_linear_bwd_rowmajor, fp8_linear_few, fp8_linear_fwd,
               fp8_quantize)
from .linear import first_order

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


class _FP8GatedMLPFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_up, down, mlp, keep):
        K, F = mlp.features, mlp.hidden
        x2 = x.reshape(-1, K)
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        M, dev = x2.shape[0], x.device
        gu8, d8 = mlp.weight_copies(keep)
        X8 = torch.empty((M, K), dtype=torch.uint8, device=dev)
        fp8_quantize(x2, E4M3, mlp.meta_x.scale, X8, None, mlp.meta_x.cur_amax)
        few = M <= FEW_TOKENS
        H8 = torch.empty((M, F), dtype=torch.uint8, device=dev) if few and not keep else _rows16(M, F, torch.uint8, dev)
        gu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if keep else None
        fp8_gated_fwd(X8, gu8, mlp.meta_x.scale_inv, mlp.meta_gate_up.scale_inv, H8[:M], act=mlp.act,
                      h_scale=mlp.meta_h.scale, h_amax=mlp.meta_h.cur_amax, gu=gu)
        y = torch.empty((M if few else H8.shape[0], K), dtype=x.dtype, device=dev)
        (fp8_linear_few if few else fp8_linear_fwd)(H8[:M] if few else H8, d8, mlp.meta_h.scale_inv,
                                                    mlp.meta_down.scale_inv, y)
        if keep:
            # the codes were made with this step's scales: keep those for backward
            factors = torch.cat([mlp.meta_x.scale_inv, mlp.meta_gate_up.scale_inv, mlp.meta_h.scale_inv,
                                 mlp.meta_down.scale_inv])
            ctx.save_for_backward(X8, gu, H8, gu8, d8, factors)
            ctx.mlp = mlp
            ctx.like = (x.shape, x.dtype, gate_up.dtype, down.dtype)
        return y[:M].reshape(x.shape)

    @staticmethod
    def backward(ctx, dy):
        X8, gu, H8, gu8, d8, factors = ctx.saved_tensors
        mlp = ctx.mlp
        x_shape, x_dtype, gate_up_dtype, down_dtype = ctx.like
        K, F, M, dev = mlp.features, mlp.hidden, X8.shape[0], dy.device
        sinv_x, sinv_gu, sinv_h, sinv_d = factors[0:1], factors[1:2], factors[2:3], factors[3:4]
        dy2 = dy.reshape(-1, K).to(x_dtype)
        if not dy2.is_contiguous():
            dy2 = dy2.contiguous()
        md, mg = mlp.meta_dy, mlp.meta_dgu
        D8 = _rows16(M, K, torch.uint8, dev)
        fp8_quantize(dy2, E5M2, md.scale, D8[:M], None, md.cur_amax)
        dx = dgate_up = ddown = None
        if ctx.needs_input_grad[2]:
            ddown = torch.empty((K, F), dtype=down_dtype, device=dev)
            fp8_linear_bwd_rowmajor(D8, None, H8, md.scale_inv, None, sinv_h, None, ddown, dw_nonfinite=mlp.dw_nonfinite)
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            G8 = torch.empty((M, 2 * F), dtype=torch.uint8, device=dev)
            fp8_gated_dgrad(D8[:M], d8, gu, md.scale_inv, sinv_d, mg.scale, G8, act=mlp.act, dgu_amax=mg.cur_amax)
            if ctx.needs_input_grad[0]:
                dx = torch.empty((M, K), dtype=x_dtype, device=dev)
            if ctx.needs_input_grad[1]:
                dgate_up = torch.empty((2 * F, K), dtype=gate_up_dtype, device=dev)
            fp8_gated_bwd(None, None, X8, gu8, sinv_x, sinv_gu, None, mg.scale_inv, G8, dx, dgate_up, act=mlp.act,
                          dw_nonfinite=mlp.dw_nonfinite if dgate_up is not None else None)
        return *first_order(dx.reshape(x_shape) if dx is not None else None, dgate_up, ddown), None, None


class FP8GatedMLP(torch.nn.Module):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T with FP8 GEMMs under delayed scaling.

    features and hidden must be multiples of 16. gate_up [2 hidden, features]
    holds Wg above Wu, down [features, hidden] Wd, in high precision; their E4M3
    copies are cast when they are not current. Call update_scales() once per
    training step, after backward; an optimizer that writes the copies itself
    (AdamW) does so after it. x is bf16 or fp32. In a CUDA graph the casts are
    part of the graph, unless it is captured in eval mode without gradients
    (serving): then it reads the copies that are current, and after a change of
    the weights weight_copies() casts them for its next replay.
    """

    def __init__(self, features: int, hidden: int, act: int = SILU, history_len: int = 16,
                 amax_compute_algo: int = AMAX_MAX, margin: int = 0, device="cuda", dtype: torch.dtype = torch.float32):
        super().__init__()
        if features % 16 or hidden % 16:
            raise ValueError("FP8 linears need features and hidden divisible by 16")
        if act not in (SILU, GELU_TANH):
            raise ValueError(f"unknown activation {act}")
        self.features, self.hidden, self.act = features, hidden, act
        self.algo, self.margin = amax_compute_algo, margin

        def weight(rows, cols):
            bound = 1.0 / cols ** 0.5
            return torch.nn.Parameter(torch.empty((rows, cols), device=device, dtype=dtype).uniform_(-bound, bound))

        self.gate_up, self.down = weight(2 * hidden, features), weight(features, hidden)
        self.meta_x, self.meta_gate_up = Meta(history_len, E4M3, device), Meta(history_len, E4M3, device)
        self.meta_h, self.meta_down = Meta(history_len, E4M3, device), Meta(history_len, E4M3, device)
        self.meta_dy, self.meta_dgu = Meta(history_len, E5M2, device), Meta(history_len, E5M2, device)
        # 1 once a weight gradient held an Inf or NaN, until its reader clears it
        # (AdamW finds the step's by its own pass over the gradients)
        self.dw_nonfinite = torch.zeros(1, dtype=torch.int32, device=device)
        # of gate_up and of down: the E4M3 copy, and what it is of
        self._copies = [torch.empty(w.shape, dtype=torch.uint8, device=device) for w in (self.gate_up, self.down)]
        self._cast_of = [_CopyState(), _CopyState()]
        self._in_a_graph = [False, False]  # a captured graph reads the copy's array
        self._trains_in_a_graph = False  # replays change the weights and their scales unseen

    def metas(self):
        return [self.meta_x, self.meta_gate_up, self.meta_h, self.meta_down, self.meta_dy, self.meta_dgu]

    def _weights(self):
        return (self.gate_up, self.meta_gate_up), (self.down, self.meta_down)

    def weight_copies(self, for_training: bool = False):
        """The weights' E4M3 copies under their metas' scales, cast if they are
        not current. A capture casts them in the graph, but for a pass without
        gradients in eval mode: that graph reads the current ones, which every
        later cast then writes in place."""
        capturing = _capturing(self.gate_up)
        here = _stream(None) if self.gate_up.is_cuda else None
        for i, (w, m) in enumerate(self._weights()):
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
        capturing = _capturing(self.gate_up)
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

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() == 0 or x.shape[-1] != self.features or x.device != self._copies[0].device:
            raise ValueError(f"x must be [..., {self.features}] on {self._copies[0].device}, got {tuple(x.shape)} on "
                             f"{x.device}")
        keep = torch.is_grad_enabled() and (x.requires_grad or self.gate_up.requires_grad or self.down.requires_grad)
        return _FP8GatedMLPFn.apply(x, self.gate_up, self.down, self, keep)

    def update_scales(self) -> None:
        """Roll the amax histories and refresh the scales for the next step; the
        weights' copies, cast under the old ones, are not current after it."""
        delayed_scaling_update(self.metas(), self.algo, self.margin)
        if _capturing(self.gate_up):
            self._trains_in_a_graph = True
        self.weights_changed()
