"""FP8GatedMLP and AdamW together: the block's output and gradients against the
same block in 64 bits, and the training example.

FP8 rounds each operand of a GEMM by at most 2^-4 (E4M3) or 2^-3 (E5M2) of
itself, independently from element to element, so a sum over many of them is
off by about (2^-4 / sqrt(3)) sqrt(1 + 1) = 5 % of its spread per GEMM of two
E4M3 operands in the 2-norm; the output sees two such GEMMs and h's rounding
(at most 10 %), a gradient up to three with one E5M2 operand each (at most 25 %).
What is checked here is the composition, so these rough bounds do: the kernels
have their own tests."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def reference(x, gate_up, down, act):
    F = gate_up.shape[0] // 2
    g, u = x @ gate_up[:F].T, x @ gate_up[F:].T
    a = torch.nn.functional.silu(g) if act == 0 else torch.nn.functional.gelu(g, approximate="tanh")
    return (a * u) @ down.T


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", [(1,), (5,), (3, 11), (64,), (65,), (2, 100), (1237,)])
def test_block_against_64_bits(cuda_lib, shape, act, dtype):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(1)
    mlp = FP8GatedMLP(272, 528, act=act)
    for step in range(2):  # the first step fills the histories, the second runs under their scales
        x = torch.randn((*shape, 272), device="cuda").to(dtype).requires_grad_(True)
        dy = (torch.randn((*shape, 272), device="cuda") * 1e-3).to(dtype)
        mlp.zero_grad(set_to_none=True)
        y = mlp(x)
        y.backward(dy)
        assert cuda_lib.fp8mp_check() == 0
        if step == 0:
            mlp.update_scales()
    xr = x.detach().double().requires_grad_(True)
    gur, dr = (w.detach().double().requires_grad_(True) for w in (mlp.gate_up, mlp.down))
    yr = reference(xr, gur, dr, act)
    yr.backward(dy.double())
    assert y.shape == x.shape and y.dtype == dtype
    assert relative(y, yr.detach()) < 0.10
    for got, want in ((x.grad, xr.grad), (mlp.gate_up.grad, gur.grad), (mlp.down.grad, dr.grad)):
        assert got.shape == want.shape and relative(got, want) < 0.25
    assert mlp.dw_nonfinite.item() == 0


def test_parts_without_gradients(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((40, 64), device="cuda", requires_grad=True)
    y = mlp(x)
    y.sum().backward()
    full = [x.grad, mlp.gate_up.grad, mlp.down.grad]
    mlp.gate_up.requires_grad_(False)
    mlp.down.requires_grad_(False)
    mlp.gate_up.grad = mlp.down.grad = None
    x.grad = None
    mlp(x).sum().backward()
    assert torch.equal(x.grad, full[0]) and mlp.gate_up.grad is None and mlp.down.grad is None
    with torch.no_grad():
        assert torch.equal(mlp(x), y)


def test_gradients_after_a_recast_use_their_own_copies(cuda_lib):
    """The scales and copies change between forward and backward: the backward
    pass still uses those of its forward."""
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(2)
    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((32, 64), device="cuda", requires_grad=True)
    y = mlp(x)
    y.sum().backward()
    want = x.grad.clone()
    x.grad = None
    y = mlp(x)
    # the weights' meta alone moves on: dy's and dgu's scales stay
    cuda_lib.delayed_scaling_update([mlp.meta_gate_up, mlp.meta_down], 0)
    mlp.weights_changed()
    mlp.weight_copies()
    y.sum().backward()
    assert torch.equal(x.grad, want)


def test_the_step_writes_what_a_cast_would(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(3)
    mlp = FP8GatedMLP(128, 256)
    opt = AdamW(mlp.parameters(), lr=1e-2, state_bits=8, modules=[mlp], loss_scale=1024.0)
    for _ in range(3):
        x = torch.randn((48, 128), device="cuda")
        opt.zero_grad()
        (mlp(x).pow(2).mean() * opt.loss_scale).sum().backward()
        mlp.update_scales()
        opt.step()
        assert opt.found_inf.item() == 0
        written = [c.clone() for c in mlp.weight_copies()]
        mlp.weights_changed()
        assert all(torch.equal(a, b) for a, b in zip(written, mlp.weight_copies()))
    assert opt.growth_tracker.item() == 3


def test_changed_weights_are_cast_again(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((32, 64), device="cuda")
    with torch.no_grad():
        y = mlp(x)
        first = mlp.weight_copies()
        assert mlp.weight_copies()[0] is first[0]  # cast once
        mlp.down.mul_(-1)
        assert torch.equal(mlp(x), -y)


def test_a_stale_backward_pass_fails(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    opt = AdamW(mlp.parameters(), lr=1e-2, modules=[mlp])
    y = mlp(torch.randn((32, 64), device="cuda"))
    y.sum().backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError):
        y.sum().backward()


@pytest.mark.parametrize("bits", [8, 32])
def test_saved_state_continues_the_run(cuda_lib, bits):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW

    torch.manual_seed(4)
    start = torch.randn((96, 64), device="cuda")
    grads = [torch.randn((96, 64), device="cuda") for _ in range(4)]

    def make():
        p = torch.nn.Parameter(start.clone())
        return p, AdamW([p], lr=1e-2, state_bits=bits, loss_scale=1.0)

    def steps(p, opt, gs):
        for g in gs:
            p.grad = g.clone()
            opt.step()

    p, opt = make()
    steps(p, opt, grads)
    q, other = make()
    steps(q, other, grads[:2])
    saved, weights = other.state_dict(), q.detach().clone()
    r, third = make()
    with torch.no_grad():
        r.copy_(weights)
    third.load_state_dict(saved)
    steps(r, third, grads[2:])
    assert torch.equal(p, r)
    with pytest.raises(ValueError):
        AdamW([p, r], lr=1.0).load_state_dict(saved)


def test_an_overflowing_step_is_skipped(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    opt = AdamW(mlp.parameters(), lr=1e-2, modules=[mlp], loss_scale=64.0)
    x = torch.randn((32, 64), device="cuda")
    x[3, 5] = float("nan")
    before = [p.detach().clone() for p in mlp.parameters()]
    (mlp(x).sum() * opt.loss_scale).sum().backward()
    opt.step()
    assert opt.found_inf.item() == 1 and opt.loss_scale.item() == 32.0
    assert all(torch.equal(a, b) for a, b in zip(before, mlp.parameters()))


def test_the_copies_after_a_skipped_step(cuda_lib):
    """update_scales changes the scales and the step that follows is skipped: the
    next forward pass is still the weights' own."""
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    opt = AdamW(mlp.parameters(), lr=1e-2, modules=[mlp])
    x = torch.randn((32, 64), device="cuda")
    (mlp(x).sum() * float("nan")).backward()  # (an infinite gradient saturates in its cast)
    mlp.update_scales()
    opt.step()
    assert opt.found_inf.item() == 1
    y = mlp(x)
    mlp.weights_changed()
    assert torch.equal(y, mlp(x)) and torch.isfinite(y).all()


@pytest.mark.parametrize("frozen", ["gate_up", "down"])
def test_a_frozen_weight_keeps_its_own_copy(cuda_lib, frozen):
    """update_scales changes a weight's scale and the step does not hold that
    weight: the next forward pass is that of a fresh cast."""
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(5)
    mlp = FP8GatedMLP(64, 96)
    getattr(mlp, frozen).requires_grad_(False)
    opt = AdamW([p for p in mlp.parameters() if p.requires_grad], lr=1e-2, modules=[mlp], loss_scale=64.0)
    x = torch.randn((32, 64), device="cuda")
    for _ in range(2):
        opt.zero_grad()
        (mlp(x).sum() * opt.loss_scale).sum().backward()
        mlp.update_scales()
        opt.step()
        y = mlp(x)
        mlp.weights_changed()
        assert torch.equal(y, mlp(x))


def test_replaced_weights_are_cast_again(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        y = mlp(x)
        for w in (mlp.gate_up, mlp.down):
            old = w.data
            w.data = -old
            z = mlp(x)
            w.data = old
            assert not torch.equal(z, y) and torch.equal(mlp(x), y)


def test_weights_of_any_strides(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        y = mlp(x)
        for w in (mlp.gate_up, mlp.down):
            w.data = w.data.t().contiguous().t()
            assert not w.is_contiguous() and torch.equal(mlp(x), y)


def test_weights_replaced_more_than_once(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        mlp(x)
        for w in (mlp.gate_up, mlp.down):
            for _ in range(2):  # the second may take the first's place in memory
                w.data = w.data * 0.5
            y = mlp(x)
            mlp.weights_changed()
            assert torch.equal(y, mlp(x))


def test_copies_cast_on_another_stream(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    side = torch.cuda.Stream()
    with torch.no_grad():
        mlp(x)
        mlp.gate_up.mul_(-1)
        mlp.down.mul_(-1)
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(400_000_000)
        here = mlp(x)  # casts the weights, after a fifth of a second
        with torch.cuda.stream(side):
            there = mlp(x)
        torch.cuda.synchronize()
    assert torch.equal(here, there)


def test_a_captured_cast_has_not_run(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        mlp(x)
        mlp.update_scales()
        want = mlp(x)
        mlp.weights_changed()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = mlp(x)
        assert torch.equal(mlp(x), want)
        graph.replay()
        assert torch.equal(y, want)
        mlp.down.mul_(-1)
        graph.replay()
        assert torch.equal(y, -want) and torch.equal(mlp(x), -want)


def test_a_graph_reads_the_copies_that_are_current(cuda_lib):
    """In eval mode it was captured without a cast: the next cast writes where it reads."""
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96).eval()
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        want = mlp(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = mlp(x)
        mlp.down.mul_(-1)
        assert torch.equal(mlp(x), -want)
        fill = [torch.full_like(c, 0x7F) for c in mlp.weight_copies() for _ in range(8)]  # freed arrays' places, if any
        graph.replay()
        assert torch.equal(y, -want) and len(fill) == 16


@pytest.mark.parametrize("optimizer", ["many-tensor", "torch"])
@pytest.mark.parametrize("warm_up", [0, 3])
def test_a_captured_training_step(cuda_lib, warm_up, optimizer):
    """Replays, with evaluations before and between them, are the steps."""
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(6)
    x = torch.randn((48, 64), device="cuda")
    start = FP8GatedMLP(64, 96).state_dict()

    def make():
        mlp = FP8GatedMLP(64, 96)
        mlp.load_state_dict(start)
        if optimizer == "torch":
            opt, loss_scale = torch.optim.SGD(mlp.parameters(), lr=1e-2), 1.0
        else:
            opt = AdamW(mlp.parameters(), lr=1e-2, modules=[mlp], loss_scale=64.0)
            loss_scale = opt.loss_scale

        def step():
            opt.zero_grad()
            (mlp(x).pow(2).mean() * loss_scale).sum().backward()
            mlp.update_scales()
            opt.step()

        def evaluate():
            with torch.no_grad():
                return mlp(x)

        return mlp, step, evaluate

    eager, eager_step, eager_evaluate = make()
    mlp, step, evaluate = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(warm_up):
            step()
        evaluate()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(warm_up):
        eager_step()
    assert torch.equal(evaluate(), eager_evaluate())
    for _ in range(3):
        graph.replay()
        eager_step()
        assert torch.equal(mlp.gate_up, eager.gate_up) and torch.equal(mlp.down, eager.down)
        assert torch.equal(evaluate(), eager_evaluate())


@pytest.mark.parametrize("kind", ["gated", "linear"])
def test_second_derivatives_are_refused(cuda_lib, kind):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
    from fp8_mixed_precision_reduce_gb300.linear import FP8Linear

    layer = FP8GatedMLP(64, 96) if kind == "gated" else FP8Linear(64, 64)
    x = torch.randn((16, 64), device="cuda", requires_grad=True)
    g, = torch.autograd.grad(layer(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (g.pow(2).sum() + x.sum()).backward()
    again, = torch.autograd.grad(layer(x).sum(), x)
    assert torch.equal(again, g) and not again.requires_grad


def test_training_after_an_evaluation_in_inference_mode(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((32, 64), device="cuda")
    with torch.inference_mode():
        y = mlp(x)
    z = mlp(x)
    z.sum().backward()
    assert torch.equal(y, z) and torch.isfinite(mlp.down.grad).all()


def test_copies_of_a_module(cuda_lib):
    import copy
    import io

    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn((5, 64), device="cuda")
    with torch.no_grad():
        y = mlp(x)
        other = copy.deepcopy(mlp)
        file = io.BytesIO()
        torch.save(mlp, file)
        file.seek(0)
        mlp.down.mul_(-1)
        assert torch.equal(mlp(x), -y) and torch.equal(other(x), y)
        assert torch.equal(torch.load(file, weights_only=False)(x), y)


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64), (1, 64), (2, 3, 64), (70, 64)])
def test_any_number_of_tokens(cuda_lib, shape):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    mlp = FP8GatedMLP(64, 96)
    x = torch.randn(shape, device="cuda", requires_grad=True)
    y = mlp(x)
    y.sum().backward()
    assert y.shape == x.shape == x.grad.shape
    assert torch.isfinite(mlp.gate_up.grad).all() and torch.isfinite(mlp.down.grad).all()
    if x.numel() == 0:
        assert (mlp.gate_up.grad == 0).all() and (mlp.down.grad == 0).all()


def test_a_replaced_weight_is_the_one_that_is_stepped(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW

    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    opt = AdamW([p], lr=0.5)
    p.grad = torch.ones_like(p)
    opt.step()
    old = p.data
    kept = old.clone()
    p.data = torch.full((300,), 7.0, device="cuda")
    p.grad = torch.ones_like(p)
    opt.step()
    assert torch.equal(old, kept) and (p < 7.0).all()


def test_a_changed_decay_applies_at_the_next_step(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW

    p = torch.nn.Parameter(torch.ones((4, 64), device="cuda"))
    opt = AdamW([p], lr=0.5, weight_decay=0.0, loss_scale=1.0)
    for decay, want in ((0.0, 1.0), (0.5, 0.75), (0.0, 0.75)):
        opt.weight_decay[0] = decay
        p.grad = torch.zeros_like(p)
        opt.step()
        assert (p == want).all()


def test_refusals(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    for bad in (dict(features=60, hidden=96), dict(features=64, hidden=90), dict(features=64, hidden=96, act=7)):
        with pytest.raises(ValueError):
            FP8GatedMLP(**bad)
    p = torch.nn.Parameter(torch.zeros(8, device="cuda"))
    for params, kw in (([], {}), ([p], dict(state_bits=16)),
                       ([torch.nn.Parameter(torch.zeros(8, device="cuda", dtype=torch.bfloat16))], {})):
        with pytest.raises(ValueError):
            AdamW(params, lr=1e-3, **kw)
    with pytest.raises(ValueError):
        AdamW([p], lr=1e-3).step()


def plain_training(example, features, hidden, tokens, steps, lr):
    """The example's training in fp32 torch operations with torch.optim.AdamW,
    from the same weights and inputs."""
    torch.manual_seed(0)
    teacher = [torch.randn(s, device="cuda") / s[1] ** 0.5 * 1.5
               for s in ((hidden, features), (hidden, features), (features, hidden))]
    block = example.Block(features, hidden)
    norm, gate_up, down = (torch.nn.Parameter(p.detach().clone()) for p in (block.norm, block.mlp.gate_up, block.mlp.down))
    opt = torch.optim.AdamW([dict(params=[norm], weight_decay=0.0), dict(params=[gate_up, down], weight_decay=0.01)],
                            lr=lr, betas=(0.9, 0.95), eps=1e-8)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, features), device="cuda")
        n = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
        target = x + (torch.nn.functional.silu(n @ teacher[0].T) * (n @ teacher[1].T)) @ teacher[2].T
        loss = (x + reference(n * norm, gate_up, down, 0) - target).pow(2).mean()
        opt.zero_grad()
        loss.backward()
        torch.nn.utils.clip_grad_norm_([norm, gate_up, down], 1.0)
        opt.step()
        losses.append(loss.item())
    return losses


@pytest.mark.parametrize("bits", [8, 32])
def test_training_example(cuda_lib, bits):
    """The example's loss falls as it does in fp32 from the same start: the drop
    over 150 steps within a tenth of fp32's."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_gated_mlp
    finally:
        sys.path.pop(0)
    sizes = dict(features=128, hidden=256, tokens=500, steps=150, lr=2e-3)
    losses, off = train_gated_mlp.run(**sizes, bits=bits, log=lambda s: None)
    plain = plain_training(train_gated_mlp, **sizes)
    mean = lambda v: sum(v[-10:]) / 10  # noqa: E731
    drop, want = losses[0] - mean(losses), plain[0] - mean(plain)
    assert want > 0 and abs(drop - want) <= 0.1 * want, (losses[0], mean(losses), plain[0], mean(plain))
    assert off < 0.05
