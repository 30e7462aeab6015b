"""TokenEmbedding: a language model's first layer.

Rows of a table, scaled (mp_embedding_fwd), read from the weight or from its E4M3
copy, which AdamW writes as it does FP8GatedMLP's ([MP] "FP32 Master Copy of Weights",
"LLM) Mixed-Precision 개념 및 학습 방법 알아보기"); the dense gradient of the table from
the tokens in sorted order (mp_embedding_bwd), the same bits at every call.
"""

from __future__ import annotations

import torch

from . import (AMAX_MAX, E4M3, Meta, mp_embedding_bwd, mp_embedding_bwd_workspace_bytes, mp_embedding_fwd)
from .gated_mlp import _rows, _WeightCopies
from .linear import first_order, refuse_capture, watch_leaves

__all__ = ["TokenEmbedding"]


class _TokenEmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, module, keep):
        flat = ids.reshape(-1)
        flat = flat if flat.is_contiguous() else flat.contiguous()
        out = torch.empty((*ids.shape, module.features), dtype=module.out_dtype, device=ids.device)
        rows = out.view(-1, module.features)
        if module.fp8:
            (table,) = module.weight_copies(keep)
            mp_embedding_fwd(flat, table, rows, scale=module.scale, sinv=module.meta_weight.scale_inv)
        else:
            mp_embedding_fwd(flat, weight.detach().contiguous(), rows, scale=module.scale)
        if keep:
            ctx.save_for_backward(flat)
            ctx.like = (weight.shape, weight.dtype, module.scale)
            watch_leaves(ctx)
        return out

    @staticmethod
    def backward(ctx, dy):
        refuse_capture(ctx)
        (ids,) = ctx.saved_tensors
        (V, K), dtype, scale = ctx.like
        dy2 = _rows(dy, K)
        dtable = torch.empty((V, K), dtype=dtype, device=dy.device)
        workspace = torch.empty(mp_embedding_bwd_workspace_bytes(ids.shape[0], V, K), dtype=torch.uint8, device=dy.device)
        mp_embedding_bwd(ids, dy2, dtable, workspace, scale=scale)
        return None, *first_order(dtable), None, None


class TokenEmbedding(_WeightCopies, torch.nn.Module):
    """weight[ids] * scale, in out_dtype (bf16 or fp32).

    features must be a multiple of 16; ids are int64, and one outside 0 .. vocab - 1
    (padding) gives a row of zeros and no gradient. With fp8 the rows are read from the
    weight's E4M3 copy under delayed scaling, kept as FP8GatedMLP keeps its own: call
    update_scales() once per training step, after backward.
    """

    def __init__(self, vocab: int, features: int, scale: float = 1.0, fp8: bool = False, history_len: int = 16,
                 amax_compute_algo: int = AMAX_MAX, margin: int = 0, device="cuda", dtype: torch.dtype = torch.float32,
                 out_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if features % 16 or features < 16 or vocab < 1:
            raise ValueError("an embedding needs features divisible by 16, and a vocabulary")
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be bf16 or fp32")
        self.vocab, self.features, self.scale, self.fp8, self.out_dtype = vocab, features, float(scale), fp8, out_dtype
        self.algo, self.margin = amax_compute_algo, margin
        self.weight = torch.nn.Parameter(torch.randn((vocab, features), device=device, dtype=torch.float32).mul_(0.02).to(dtype))
        if fp8:
            self.meta_weight = Meta(history_len, E4M3, device)
            self._make_copies(device)

    def metas(self):
        return [self.meta_weight] if self.fp8 else []

    def _weights(self):
        return ((self.weight, self.meta_weight),) if self.fp8 else ()

    def weight_copies(self, for_training: bool = False):
        return super().weight_copies(for_training) if self.fp8 else ()

    def copies_for_step(self):
        return super().copies_for_step() if self.fp8 else []

    def copies_written(self, weights=None) -> None:
        if self.fp8:
            super().copies_written(weights)

    def weights_changed(self) -> None:
        if self.fp8:
            super().weights_changed()

    def update_scales(self) -> None:
        if self.fp8:
            super().update_scales()

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        w = self.weight
        if ids.dtype != torch.int64 or ids.device != w.device:
            raise ValueError(f"ids must be int64 on {w.device}, got {ids.dtype} on {ids.device}")
        if w.shape != (self.vocab, self.features):
            raise ValueError(f"weight must be {(self.vocab, self.features)}, got {tuple(w.shape)}")
        keep = torch.is_grad_enabled() and w.requires_grad
        return _TokenEmbeddingFn.apply(ids, w, self, keep)
