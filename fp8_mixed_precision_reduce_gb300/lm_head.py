"""FP8LMHead: a language model's last layer on the library's FP8 path, from the
residual stream to log probabilities.

logits = n W^T with n = x, or the root-mean-square norm of x + residual, under the
DelayedScaling recipe with the HYBRID format as FP8Linear runs one linear; then the log
probabilities of given tokens and their entropy, or the most probable tokens
(mp_logprobs_fwd). Backward: the logits' gradient as E5M2 codes in one pass over the
logits (mp_logprobs_bwd), then dx and dW in one launch (fp8_linear_bwd_rowmajor). The
gradient of the logits is never stored in more than 8 bits.
"""

from __future__ import annotations

import torch

from . import (AMAX_MAX, E4M3, E5M2, FEW_TOKENS, MAX_TOP, Meta, fp8_linear_bwd_rowmajor, fp8_linear_few,
               fp8_linear_fwd, mp_logprobs_bwd, mp_logprobs_fwd)
from .gated_mlp import (_check_input, _check_norm, _check_norm_weight, _codes_of, _norm_grads, _rows, _rows16,
                        _WeightCopies)
from .linear import first_order, refuse_capture, watch_leaves

__all__ = ["FP8LMHead"]


def _logits_of(x, residual, norm, head, for_training: bool):
    """The logits' rows (head.logits_dtype, [tokens, vocabulary rounded up]), and what
    they were made of."""
    K = head.features
    x2 = _rows(x, K)
    M, dev = x2.shape[0], x.device
    (w8,) = head.weight_copies(for_training)
    few = M <= FEW_TOKENS
    X8 = torch.empty((M, K), dtype=torch.uint8, device=dev) if few and not for_training else _rows16(M, K, torch.uint8, dev)
    norm = norm.detach().contiguous() if norm is not None else None
    total, rstd = _codes_of(x2, _rows(residual, K) if residual is not None else None, norm, head.norm_eps, head.meta_x,
                            X8[:M])
    logits = torch.empty((M if few else X8.shape[0], w8.shape[0]), dtype=head.logits_dtype, device=dev)
    (fp8_linear_few if few else fp8_linear_fwd)(X8[:M] if few else X8, w8, head.meta_x.scale_inv, head.meta_weight.scale_inv,
                                                logits)
    return logits[:M], X8, w8, x2 if total is None else total, rstd, norm


class _FP8LMHeadFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, norm, weight, targets, head, with_entropy, keep):
        logits, X8, w8, normed, rstd, norm = _logits_of(x, residual, norm, head, keep)
        M, dev = logits.shape[0], x.device
        t = targets.reshape(-1)
        t = t if t.is_contiguous() else t.contiguous()
        logprob = torch.empty(targets.shape, dtype=torch.float32, device=dev)
        entropy = torch.empty_like(logprob) if with_entropy else None
        stats = torch.empty((M, 2), dtype=torch.float32, device=dev)
        mp_logprobs_fwd(logits, t, logprob.view(-1), stats, entropy=entropy.view(-1) if with_entropy else None,
                        vocab=head.vocab)
        if keep:
            factors = torch.cat([head.meta_x.scale_inv, head.meta_weight.scale_inv])
            ctx.save_for_backward(logits, X8, w8, t, stats, entropy, factors, normed if norm is not None else None, rstd, norm)
            ctx.head = head
            ctx.like = (x.shape, x.dtype, weight.dtype)
            ctx.set_materialize_grads(False)
            watch_leaves(ctx)
        return (logprob, entropy) if with_entropy else logprob

    @staticmethod
    def backward(ctx, dlogprob, dentropy=None):
        refuse_capture(ctx)
        logits, X8, w8, t, stats, entropy, factors, normed, rstd, norm = ctx.saved_tensors
        head = ctx.head
        x_shape, x_dtype, w_dtype = ctx.like
        need_x, need_residual, need_norm, need_weight = ctx.needs_input_grad[:4]
        if dlogprob is None and dentropy is None:
            return (None,) * 8
        M, K, dev = logits.shape[0], head.features, logits.device
        flat = lambda g: g.to(torch.float32).reshape(-1).contiguous()  # noqa: E731
        da = flat(dlogprob) if dlogprob is not None else torch.zeros(M, dtype=torch.float32, device=dev)
        db = flat(dentropy) if dentropy is not None else None
        md = head.meta_dlogits
        D8 = _rows16(M, logits.shape[1], torch.uint8, dev)
        mp_logprobs_bwd(logits, t, stats, da, D8[:M], entropy=entropy.reshape(-1) if db is not None else None, dentropy=db,
                        scale=md.scale, amax=md.cur_amax, vocab=head.vocab)
        need_in = need_x or need_residual or need_norm
        dx = torch.empty((D8.shape[0], K), dtype=x_dtype, device=dev) if need_in else None
        dw = torch.empty(w8.shape, dtype=w_dtype, device=dev) if need_weight else None
        if dx is not None or dw is not None:
            fp8_linear_bwd_rowmajor(D8, w8, X8, md.scale_inv, factors[1:2], factors[0:1], dx, dw,
                                    dw_nonfinite=head.dw_nonfinite if dw is not None else None)
        dresidual = dnorm = None
        if dx is not None:
            dx = dx[:M]
            if norm is not None:
                dx, dresidual, dnorm = _norm_grads(dx, normed, None, norm, rstd, x_dtype, need_norm, x_shape)
            else:
                dx = dx.reshape(x_shape)
        return *first_order(dx if need_x else None, dresidual if need_residual else None, dnorm, dw), None, None, None, None


class FP8LMHead(_WeightCopies, torch.nn.Module):
    """Log probabilities over a vocabulary, from x or from the norm of x + residual.

    features must be a multiple of 16; vocab is any (the weight has its rows rounded up
    to 16, the added ones without a token, zero and never changed by a gradient). The
    weight is kept in high precision with an E4M3 copy as FP8GatedMLP keeps its own;
    call update_scales() once per training step, after backward.

    head(x, targets) gives the log p of each target, with entropy=True (log p, entropy),
    fp32 in the targets' shape, differentiable; a target outside 0 .. vocab - 1 (a prompt's
    or padding's) has log p 0 and no gradient. head.top(x, k) gives the k most probable tokens and their log p.
    With norm_eps both take the residual stream: n = norm(x + residual).

    The logits are held in bf16, whatever x's type, until log p is taken from them in
    fp32: a logit of 16 to 32 is off by up to 2^-4, and top takes the lower token of two that
    bf16 makes equal. With logits_dtype=torch.float32 they are the product's own fp32, and
    take twice the memory.
    """

    def __init__(self, features: int, vocab: int, history_len: int = 16, amax_compute_algo: int = AMAX_MAX,
                 margin: int = 0, device="cuda", dtype: torch.dtype = torch.float32, norm_eps: float | None = None,
                 logits_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if logits_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("logits_dtype must be bf16 or fp32")
        if features % 16 or features < 16 or vocab < 1:
            raise ValueError("FP8 linears need features divisible by 16, and a vocabulary")
        _check_norm(features, norm_eps)
        self.features, self.vocab, self.logits_dtype = features, vocab, logits_dtype
        self.algo, self.margin = amax_compute_algo, margin
        bound = 1.0 / features ** 0.5
        weight = torch.empty(((vocab + 15) // 16 * 16, features), device=device, dtype=dtype).uniform_(-bound, bound)
        weight[vocab:].zero_()
        self.weight = torch.nn.Parameter(weight)
        self.norm_eps = norm_eps
        self.norm = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype)) if norm_eps is not None else None
        self.meta_x, self.meta_weight = Meta(history_len, E4M3, device), Meta(history_len, E4M3, device)
        self.meta_dlogits = Meta(history_len, E5M2, device)
        # 1 once a weight gradient held an Inf or NaN, until its reader clears it
        self.dw_nonfinite = torch.zeros(1, dtype=torch.int32, device=device)
        self._make_copies(device)

    def metas(self):
        return [self.meta_x, self.meta_weight, self.meta_dlogits]

    def _weights(self):
        return ((self.weight, self.meta_weight),)

    def _check(self, x, residual) -> None:
        _check_input(x, residual, self.features, self._copies[0].device, self.norm)
        _check_norm_weight(self.norm, x, self.features)

    def forward(self, x: torch.Tensor, targets: torch.Tensor, residual: torch.Tensor | None = None, entropy: bool = False):
        self._check(x, residual)
        if targets.shape != x.shape[:-1] or targets.dtype != torch.int64 or targets.device != x.device:
            raise ValueError(f"targets must be int64 {tuple(x.shape[:-1])} on {x.device}, got {targets.dtype} "
                             f"{tuple(targets.shape)} on {targets.device}")
        inputs = (x, residual, self.norm, self.weight)
        keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)
        return _FP8LMHeadFn.apply(*inputs, targets, self, entropy, keep)

    @torch.no_grad()
    def top(self, x: torch.Tensor, k: int = 1, residual: torch.Tensor | None = None):
        """(log p, tokens) of the k most probable tokens, [..., k] each, most probable
        first, of equal logits the lower token first."""
        self._check(x, residual)
        if not 1 <= k <= min(MAX_TOP, self.vocab):
            raise ValueError(f"k must lie in 1..{min(MAX_TOP, self.vocab)}, got {k}")
        logits, *_ = _logits_of(x, residual, self.norm, self, False)
        M, dev = logits.shape[0], x.device
        stats, logprob = (torch.empty((M, n), dtype=torch.float32, device=dev) for n in (2, k))
        tokens = torch.empty((M, k), dtype=torch.int64, device=dev)
        mp_logprobs_fwd(logits, None, None, stats, top_logprob=logprob, top_id=tokens, vocab=self.vocab)
        return logprob.reshape(*x.shape[:-1], k), tokens.reshape(*x.shape[:-1], k)
