"""FP8GatedMLP, FP8Linear and AdamW around the library's calls, without a GPU:
on CPU tensors, with the calls they make replaced by plain torch operations."""

import gc
import weakref

import pytest
import torch

import fp8_mixed_precision_reduce_gb300 as fp8mp
from fp8_mixed_precision_reduce_gb300 import adamw, gated_mlp, linear


def cast(w, scale):
    return (w.detach().float() * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def plain_quantize(x, fmt, scale, out, out_t=None, amax=None, stream=None):
    out.copy_(cast(x, scale))
    amax.copy_(torch.maximum(amax, x.abs().max()))


def plain_update(metas, algo, margin=0, stream=None):
    for m in metas:
        if m.cur_amax.item() > 0:
            m.scale.copy_(fp8mp.FMT_MAX[m.fmt] / m.cur_amax)
            m.scale_inv.copy_(1 / m.scale)


def plain_step(plan, *scalars, lr, **kw):
    """w -= lr (grad + decay w), and the copies of a plan's rows."""
    rows = plan.c_array()
    for i, (grad, w, *_, copy, scale, amax) in enumerate(plan._keep):
        w.sub_(lr * (grad + rows[i].weight_decay * w))
        if copy is not None:
            copy.copy_(cast(w, scale))
            amax.copy_(torch.maximum(amax, w.abs().max()))


@pytest.fixture
def plain(monkeypatch):
    fp8mp.build()
    monkeypatch.setattr(gated_mlp, "fp8_quantize", plain_quantize)
    monkeypatch.setattr(gated_mlp, "delayed_scaling_update", plain_update)
    monkeypatch.setattr(adamw, "mp_grad_norm", lambda *a: None)
    monkeypatch.setattr(adamw, "mp_adamw_step", plain_step)


def block(seed=0):
    torch.manual_seed(seed)
    return gated_mlp.FP8GatedMLP(32, 48, device="cpu")


def step(opt, *modules):
    for p in opt.params:
        p.grad = torch.randn_like(p)
    for m in modules:
        m.update_scales()
    opt.step()


def copies_are_current(mlp):
    return all(torch.equal(c, cast(w, m.scale)) for c, w, m in zip(
        mlp.weight_copies(), (mlp.gate_up, mlp.down), (mlp.meta_gate_up, mlp.meta_down)))


# ------------------------------------- copies that a step writes, and others


@pytest.mark.parametrize("trained", ["gate_up", "down"])
@pytest.mark.parametrize("cast_before", [True, False])
def test_a_weight_the_step_does_not_hold(plain, trained, cast_before):
    mlp = block()
    opt = adamw.AdamW([getattr(mlp, trained)], lr=1e-2, modules=[mlp])
    for _ in range(3):
        if cast_before:
            mlp.weight_copies()
        step(opt, mlp)
        assert copies_are_current(mlp)


def test_what_the_step_wrote_is_not_cast_again(plain, monkeypatch):
    mlp = block()
    opt = adamw.AdamW([mlp.gate_up], lr=1e-2, modules=[mlp])
    mlp.weight_copies()
    step(opt, mlp)
    cast_weights = []
    monkeypatch.setattr(gated_mlp, "fp8_quantize", lambda x, *a: (cast_weights.append(x.shape), plain_quantize(x, *a)))
    mlp.weight_copies()
    assert cast_weights == [mlp.down.shape]


def test_two_optimizers_of_one_module(plain):
    mlp = block()
    first, second = (adamw.AdamW([w], lr=1e-2, modules=[mlp]) for w in (mlp.gate_up, mlp.down))
    mlp.weight_copies()
    for p in (mlp.gate_up, mlp.down):
        p.grad = torch.randn_like(p)
    mlp.update_scales()
    first.step()
    assert copies_are_current(mlp)
    second.step()
    assert copies_are_current(mlp)


def test_a_weight_of_two_modules(plain):
    a, b = block(1), block(2)
    b.down = a.down
    opt = adamw.AdamW([a.gate_up, a.down, b.gate_up], lr=1e-2, modules=[a, b])
    for _ in range(2):
        step(opt, a, b)
        a.meta_down.scale.mul_(2)  # (the modules' scales of the shared weight need not agree)
        a.weights_changed()
        step(opt)
        assert copies_are_current(a) and copies_are_current(b)


def test_a_parameter_that_was_replaced(plain):
    mlp = block()
    opt = adamw.AdamW(mlp.parameters(), lr=1e-2, modules=[mlp])
    step(opt, mlp)
    mlp.down = torch.nn.Parameter(torch.randn_like(mlp.down))
    step(opt, mlp)
    assert copies_are_current(mlp)


# ------------------------------------------------------------------- inputs


@pytest.mark.parametrize("shape", [(4, 16), (2, 64), (1, 31), (0, 16), (32, 4), ()])
def test_an_input_of_another_width_is_refused(shape):
    """Also one whose elements would fill rows of the block's width."""
    with pytest.raises(ValueError, match="32"):
        block()(torch.zeros(shape))


def test_an_input_on_another_device_is_refused():
    with pytest.raises(ValueError, match="meta"):
        block()(torch.zeros((4, 32), device="meta"))


@pytest.mark.parametrize("x", [torch.zeros((16, 16)), torch.zeros((16, 64)), torch.zeros(()),
                               torch.zeros((16, 32), device="meta")])
def test_a_linear_refuses_an_input_of_another_width_or_device(x):
    """(A weight's copy was laid out for the input's width.)"""
    with pytest.raises(ValueError, match="32"):
        linear.FP8Linear(32, 48, device="cpu")(x)


# ------------------------------------------------ what a kept plan was made of


def test_a_changed_decay_is_the_next_steps(plain):
    p = torch.nn.Parameter(torch.ones(4, 16))
    opt = adamw.AdamW([p], lr=0.5, weight_decay=0.0)
    for decay, want in ((0.0, 1.0), (0.5, 0.75), (0.0, 0.75)):
        opt.weight_decay[0] = decay
        p.grad = torch.zeros_like(p)
        opt.step()
        assert (p == want).all()


def test_a_replaced_amax_is_the_one_that_is_raised(plain):
    mlp = block()
    opt = adamw.AdamW(mlp.parameters(), lr=1e-2, modules=[mlp])
    step(opt)
    old = mlp.meta_down.cur_amax
    mlp.meta_down.cur_amax, kept = torch.zeros(1), old.clone()
    step(opt)
    assert torch.equal(old, kept) and mlp.meta_down.cur_amax.item() == mlp.down.abs().max().item()


# ------------------------------------------ weights that are not as they were


def test_a_transposed_weight_is_cast_as_it_reads(plain, monkeypatch):
    mlp = block()
    laid_out = []
    monkeypatch.setattr(gated_mlp, "fp8_quantize",
                        lambda x, *a: (laid_out.append(x.is_contiguous()), plain_quantize(x, *a)))
    for w in (mlp.gate_up, mlp.down):
        w.data = w.data.t().contiguous().t()
    assert copies_are_current(mlp) and all(laid_out)


def test_a_weight_of_another_shape_is_refused(plain):
    mlp = block()
    for w in (mlp.gate_up, mlp.down):
        kept = w.data
        for other in (torch.zeros((200, 32)), kept[:16], kept.reshape(-1)):
            w.data = other
            with pytest.raises(ValueError, match="weight"):
                mlp.weight_copies()
        w.data = kept
        mlp.weight_copies()
    mlp.down = torch.nn.Parameter(mlp.down.to("meta"))
    with pytest.raises(ValueError, match="weight"):
        mlp.weight_copies()


def test_a_weight_transposed_in_place_is_cast_again(plain):
    mlp = gated_mlp.FP8GatedMLP(32, 32, device="cpu")
    mlp.weight_copies()
    mlp.down.data = mlp.down.data.t()  # the same address and version
    assert copies_are_current(mlp)


def test_a_parameter_that_is_no_longer_dense_is_refused(plain):
    p = torch.nn.Parameter(torch.ones(16, 16))
    opt = adamw.AdamW([p], lr=1e-2)
    step(opt)
    p.data = p.data.t()
    with pytest.raises(ValueError, match="dense"):
        step(opt)


# ------------------------------------------------------------------- AdamW


def test_a_parameter_given_twice_is_refused():
    """(Two rows of one launch would update the same memory.)"""
    p = torch.nn.Parameter(torch.zeros(8, 8))
    q = torch.nn.Parameter(torch.zeros(8))
    with pytest.raises(ValueError, match="twice"):
        adamw.AdamW([p, q, p], lr=1e-3)
    tied = torch.nn.Parameter(p.data)
    with pytest.raises(ValueError, match="twice"):
        adamw.AdamW([p, q, tied], lr=1e-3)
    with pytest.raises(ValueError, match="twice"):
        adamw.AdamW([torch.nn.Parameter(p.data.view(-1)[16:48]), p], lr=1e-3)
    empty = [torch.nn.Parameter(torch.zeros(0)) for _ in range(2)]
    flat = torch.zeros(64)
    adamw.AdamW([*empty, *(torch.nn.Parameter(flat[i:i + 16]) for i in range(0, 64, 16))], lr=1e-3)


def test_a_state_that_does_not_fit_is_not_loaded_in_part():
    make = lambda *shapes: adamw.AdamW([torch.nn.Parameter(torch.ones(s)) for s in shapes], lr=1e-3)  # noqa: E731
    saved = make((8, 8), (4, 4)).state_dict()
    for s in saved["state"]:
        s["exp_avg"].fill_(3.0)
    for bad in (make((8, 8), (4, 5)), make((8, 8), (4, 4))):
        if bad.params[1].numel() == 16:
            saved["scalars"]["loss_scale"] = torch.ones(2)
        before = bad.state_dict()
        with pytest.raises(ValueError):
            bad.load_state_dict(saved)
        after = bad.state_dict()
        assert all(torch.equal(a[k], b[k]) for a, b in zip(before["state"], after["state"]) for k in a)
        assert all(torch.equal(v, after["scalars"][k]) for k, v in before["scalars"].items())


# ----------------------------------------------------------------- binding


def test_the_current_stream_without_torchs_raw_call(monkeypatch):
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        with monkeypatch.context() as m:
            m.delattr(torch._C, name, raising=False)
            assert fp8mp._stream(None) == 77
    assert fp8mp._stream(5) == 5 and fp8mp._stream(Stream()) == 77


def test_gradients_at_any_address(plain, monkeypatch):
    """Views into a flat buffer, after a tensor of odd size."""
    params = [torch.nn.Parameter(torch.zeros(n)) for n in (5, 7, 16)]
    flat = torch.arange(28.0)
    for p, g in zip(params, flat.split([5, 7, 16])):
        p.grad = g
    seen = []
    monkeypatch.setattr(adamw, "mp_grad_norm", lambda plan, *a: seen.extend(r.grad for r in plan.c_array()))
    adamw.AdamW(params, lr=1.0, weight_decay=0.0).step()
    assert all(address % 16 == 0 for address in seen) and len(seen) == 3
    assert torch.equal(torch.cat([p.detach() for p in params]), -flat)


def test_copies_cast_in_inference_mode_serve_training_too(plain):
    mlp = block()
    with torch.inference_mode():
        mlp.weight_copies()
    opt = adamw.AdamW(mlp.parameters(), lr=1e-2, modules=[mlp])
    assert not any(c.is_inference() for c in mlp.weight_copies())
    step(opt, mlp)
    assert copies_are_current(mlp)


def test_a_step_lets_its_gradients_go(plain):
    p = torch.nn.Parameter(torch.zeros(8, 8))
    opt = adamw.AdamW([p], lr=1e-2)
    for _ in range(2):
        p.grad = torch.ones(8, 8)
        grad = weakref.ref(p.grad)
        opt.step()
        opt.zero_grad()
        gc.collect()
        assert grad() is None


def test_a_plan_without_its_gradients_is_refused():
    plan = fp8mp.AdamWTensors()
    plan.add(torch.zeros(300))
    plan.release_grads()
    with pytest.raises(fp8mp.Fp8mpError, match="set_grads"):
        plan.c_array()
    g = torch.zeros(300)
    plan.set_grads([g])
    assert plan.c_array()[0].grad == g.data_ptr()


def test_a_linear_refuses_a_weight_or_bias_of_another_shape():
    x = torch.zeros((16, 32))
    for name, other in (("weight", torch.zeros((48, 64))), ("weight", torch.zeros((32, 32))), ("bias", torch.zeros(16))):
        layer = linear.FP8Linear(32, 48, device="cpu")
        getattr(layer, name).data = other
        with pytest.raises(ValueError, match=name):
            layer(x)
    layer = linear.FP8Linear(32, 48, device="cpu")
    layer.weight = torch.nn.Parameter(layer.weight.to("meta"))
    with pytest.raises(ValueError, match="weight"):
        layer(x)
