"""AdamW over a model's parameters in the library's many-tensor step.

One call of mp_grad_norm and one of mp_adamw_step per step, whatever the number
of parameters: the loss scale, the overflow skip, gradient clipping, the
decoupled decay, moments in fp32 or in 8-bit codes, and the E4M3 copies of the
weights that the next forward pass reads ([MP] "FP32 Master Copy of Weights" and
the dynamic loss-scale procedure, "LLM) Mixed-Precision 개념 및 학습 방법
알아보기"). This file keeps the state and passes pointers.
"""

from __future__ import annotations

import torch

from . import AdamWTensors, mp_adamw_step, mp_adamw_workspace_bytes, mp_grad_norm

__all__ = ["AdamW"]


class AdamW:
    """AdamW on fp32 parameters whose gradients are of the loss times
    ``loss_scale`` (a device tensor, adapted as the steps go).

    Parameters of two or more dimensions decay by ``weight_decay``, the others
    do not. ``state_bits`` 8 holds the moments of parameters of at least
    ``min_8bit_size`` elements in 8 bits, the others' in 32. ``modules``: those
    with ``copies_for_step()`` (FP8GatedMLP) get the E4M3 copies of those of
    their weights that are among ``params`` written by the step, under the
    scales of their metas: call update_scales() before step(). (Of a weight that
    several modules hold, the first one's copy; the others cast theirs.)
    """

    _SCALARS = ("loss_scale", "growth_tracker", "beta_pows", "seed")

    def __init__(self, params, lr: float, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 max_norm: float = 0.0, state_bits: int = 32, min_8bit_size: int = 4096, modules=(),
                 loss_scale: float = 65536.0, growth_interval: int = 2000, seed: int = 0):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 32 or 8")
        self.lr, self.betas, self.eps, self.max_norm = lr, betas, eps, max_norm
        self.growth_interval = growth_interval
        dev, f32 = self.params[0].device, torch.float32
        for p in self.params:
            if p.dtype != torch.float32 or not p.is_contiguous() or p.device != dev:
                raise ValueError("AdamW needs dense fp32 parameters on one device")
        spans = sorted((p.data_ptr(), p.data_ptr() + 4 * p.numel()) for p in self.params if p.numel() > 0)
        if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
            raise ValueError("AdamW was given a parameter, or a part of its memory, twice")
        self.modules = list(modules)
        self.state = []
        for p in self.params:
            n = p.numel()
            if state_bits == 8 and n >= min_8bit_size:
                blocks = (n + 255) // 256
                self.state.append(dict(exp_avg=torch.zeros(n, dtype=torch.int8, device=dev),
                                       exp_avg_sq=torch.zeros(n, dtype=torch.uint8, device=dev),
                                       exp_avg_scale=torch.zeros(blocks, dtype=f32, device=dev),
                                       exp_avg_sq_scale=torch.zeros(blocks, dtype=f32, device=dev)))
            else:
                self.state.append(dict(exp_avg=torch.zeros(n, dtype=f32, device=dev),
                                       exp_avg_sq=torch.zeros(n, dtype=f32, device=dev)))
        self.weight_decay = [weight_decay if p.dim() >= 2 else 0.0 for p in self.params]
        self.loss_scale = torch.full((1,), float(loss_scale), dtype=f32, device=dev)
        self.growth_tracker = torch.zeros(1, dtype=torch.int32, device=dev)
        self.found_inf = torch.zeros(1, dtype=torch.int32, device=dev)
        self.beta_pows = torch.ones(2, dtype=f32, device=dev)
        self.grad_norm = torch.zeros(1, dtype=f32, device=dev)
        self.seed = torch.full((1,), seed, dtype=torch.int32, device=dev)
        self.workspace = torch.zeros(mp_adamw_workspace_bytes() // 4, dtype=torch.int32, device=dev)
        self._plan, self._arrays = None, None

    def _copies(self):
        """What the step writes of the modules' copies: {id(weight): (copy, meta)},
        and each module's weights among them."""
        mine, copies, written = {id(p) for p in self.params}, {}, []
        for mod in self.modules:
            of = [x for x in mod.copies_for_step() if id(x[0]) in mine and id(x[0]) not in copies]
            copies.update((id(w), (c, m)) for w, c, m in of)
            written.append((mod, [w for w, _, _ in of]))
        return copies, written

    def _tensors(self, grads, copies) -> AdamWTensors:
        """The step's tensors, rebuilt when an array or a decay that they hold is another."""
        now = [p.data_ptr() for p in self.params] + list(self.weight_decay)
        now += [(c.data_ptr(), m.scale.data_ptr(), m.cur_amax.data_ptr()) for c, m in copies.values()]
        if self._plan is not None and now == self._arrays:
            self._plan.set_grads(grads)
            return self._plan
        plan = AdamWTensors()
        for p, g, s, decay in zip(self.params, grads, self.state, self.weight_decay):
            c, m = copies.get(id(p), (None, None))
            scaled = dict(copy=c, copy_scale=m.scale, copy_amax=m.cur_amax) if c is not None else {}
            plan.add(g, p.detach(), weight_decay=decay, **s, **scaled)
        self._plan, self._arrays = plan, now
        return plan

    def step(self) -> None:
        """One step from the parameters' .grad; nothing is read back to the host."""
        grads = []
        for i, p in enumerate(self.params):
            if p.grad is None:
                raise ValueError(f"parameter {i} has no gradient")
            if not p.is_contiguous():
                raise ValueError(f"parameter {i} is no longer dense")
            g = p.grad
            if not g.is_contiguous() or g.data_ptr() % 16:  # (the library reads dense rows of 16 bytes)
                g = g.clone(memory_format=torch.contiguous_format)
            grads.append(g)
        copies, written = self._copies()
        plan = self._tensors(grads, copies)
        mp_grad_norm(plan, self.grad_norm, self.found_inf, self.workspace)
        mp_adamw_step(plan, self.loss_scale, self.growth_tracker, self.found_inf, self.beta_pows, self.workspace,
                      lr=self.lr, beta1=self.betas[0], beta2=self.betas[1], eps=self.eps, seed=self.seed,
                      grad_norm=self.grad_norm if self.max_norm > 0 else None, max_norm=self.max_norm,
                      growth_interval=self.growth_interval)
        plan.release_grads()
        torch.autograd.graph.increment_version(self.params)
        for mod, weights in written:
            mod.copies_written(weights)

    def state_dict(self) -> dict:
        """Everything but the parameters that the next step depends on."""
        return dict(state=[{k: v.clone() for k, v in s.items()} for s in self.state],
                    scalars={k: getattr(self, k).clone() for k in self._SCALARS})

    def load_state_dict(self, saved: dict) -> None:
        if len(saved["state"]) != len(self.state):
            raise ValueError(f"{len(saved['state'])} saved states for {len(self.state)} parameters")
        scalars = {k: getattr(self, k) for k in self._SCALARS}
        pairs = [*zip(self.state, saved["state"]), (scalars, {k: saved["scalars"][k] for k in self._SCALARS})]
        for mine, s in pairs:
            if {k: (v.dtype, v.shape) for k, v in mine.items()} != {k: (v.dtype, v.shape) for k, v in s.items()}:
                raise ValueError("a saved state has other types or sizes than its parameter's")
        for mine, s in pairs:
            for k, v in s.items():
                mine[k].copy_(v)

    def zero_grad(self) -> None:
        for p in self.params:
            p.grad = None
