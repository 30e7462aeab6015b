"""What mp_grad_norm, mp_adamw_step and their binding refuse, without a GPU."""

import ctypes

import pytest
import torch

import fp8_mixed_precision_reduce_gb300 as fp8mp

P = 4096  # a fake, aligned address: validation fails before it is used


@pytest.fixture(scope="module")
def lib():
    fp8mp.build()
    return fp8mp.load()


def row(**kw):
    d = dict(grad=P, master=P, exp_avg=P, exp_avg_sq=P, n=100, grad_dtype=fp8mp.BF16, state_bits=32)
    d.update(kw)
    return fp8mp.fp8mp_adamw_tensor(**d)


def step(lib, rows, loss_scale=P, growth=P, found=P, pows=P, seed=P, norm=None, max_norm=0.0, b1=0.9, b2=0.95,
         eps=1e-8, interval=10, ws=P, ws_bytes=1 << 20):
    arr = (fp8mp.fp8mp_adamw_tensor * max(1, len(rows)))(*rows)
    return lib.mp_adamw_step(arr, len(rows), loss_scale, growth, found, pows, seed, norm, max_norm, 1e-3, b1, b2, eps,
                             0.5, 2.0, interval, ws, ws_bytes, None)


def test_struct_layout(lib):
    assert ctypes.sizeof(fp8mp.fp8mp_adamw_tensor) == 96
    assert fp8mp.fp8mp_adamw_tensor.n.offset == 72 and fp8mp.fp8mp_adamw_tensor.reserved.offset == 92
    assert fp8mp.mp_adamw_workspace_bytes() % 16 == 0


@pytest.mark.parametrize("kw,word", [
    (dict(grad=None), "grad"), (dict(grad=P + 2), "aligned"), (dict(master=None), "NULL"),
    (dict(exp_avg=P + 8), "aligned"), (dict(copy=P + 4), "aligned"), (dict(n=-1), "n = -1"),
    (dict(n=1 << 50), "n ="), (dict(grad_dtype=7), "grad_dtype"), (dict(state_bits=16), "state_bits"),
    (dict(reserved=1), "reserved"), (dict(state_bits=8), "scales"),
    (dict(state_bits=8, exp_avg_scale=P + 2, exp_avg_sq_scale=P), "misaligned"), (dict(copy_scale=P), "no copy"),
    (dict(copy=P, copy_amax=P), "no scale"), (dict(copy=P, copy_scale=P + 1), "misaligned"),
])
def test_bad_tensors(lib, kw, word):
    assert step(lib, [row(), row(**kw)]) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(loss_scale=None), "loss_scale"), (dict(growth=None), "growth"), (dict(found=None), "found_inf"),
    (dict(pows=None), "beta_pows"), (dict(norm=P), "max_norm"), (dict(b1=1.0), "betas"), (dict(b2=-0.1), "betas"),
    (dict(eps=0.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(interval=0), "growth_interval"),
    (dict(ws=None), "workspace"), (dict(ws_bytes=16), "workspace"), (dict(ws=P + 4), "aligned"),
])
def test_bad_arguments(lib, kw, word):
    assert step(lib, [row()], **kw) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


def test_8_bit_moments_need_a_seed(lib):
    eight = row(state_bits=8, exp_avg_scale=P, exp_avg_sq_scale=P)
    assert step(lib, [eight], seed=None) == fp8mp.ERR_INVALID
    assert "seed" in fp8mp.last_error()


def test_norm_arguments(lib):
    arr = (fp8mp.fp8mp_adamw_tensor * 1)(row())
    assert lib.mp_grad_norm(arr, -1, P, P, P, 1 << 20, None) == fp8mp.ERR_INVALID
    assert lib.mp_grad_norm(None, 1, P, P, P, 1 << 20, None) == fp8mp.ERR_INVALID
    assert lib.mp_grad_norm(arr, 1, None, P, P, 1 << 20, None) == fp8mp.ERR_INVALID
    assert lib.mp_grad_norm(arr, 1, P, None, P, 1 << 20, None) == fp8mp.ERR_INVALID
    assert lib.mp_grad_norm(arr, 1, P, P, P, 64, None) == fp8mp.ERR_INVALID
    many = (fp8mp.fp8mp_adamw_tensor * 3)(*[row(n=1 << 40)] * 3)
    assert lib.mp_grad_norm(many, 3, P, P, P, 1 << 20, None) == fp8mp.ERR_INVALID
    assert "too many" in fp8mp.last_error()


def test_binding_checks_shapes_and_types():
    z = torch.zeros
    plan = fp8mp.AdamWTensors()
    good = dict(grad=z(300), master=z(300), exp_avg=z(300), exp_avg_sq=z(300))
    plan.add(**good)
    assert len(plan) == 1
    codes = dict(exp_avg=z(300, dtype=torch.int8), exp_avg_sq=z(300, dtype=torch.uint8))
    plan.add(**{**good, **codes}, exp_avg_scale=z(2), exp_avg_sq_scale=z(2))
    for bad in (dict(master=z(299)), dict(master=z(300, dtype=torch.float64)), dict(exp_avg=None), codes,
                dict(exp_avg=z(300, dtype=torch.int8)), dict(grad=z(600)[::2]),
                dict(copy=z(300, dtype=torch.uint8)), dict(copy=z(300, dtype=torch.bfloat16), copy_scale=z(1)),
                {**codes, "exp_avg_scale": z(1), "exp_avg_sq_scale": z(2)}):
        with pytest.raises(fp8mp.Fp8mpError):
            fp8mp.AdamWTensors().add(**{**good, **bad})
    with pytest.raises(TypeError):
        fp8mp.AdamWTensors().add(**{**good, "grad": z(300, dtype=torch.float16)})
    with pytest.raises(fp8mp.Fp8mpError):
        plan.set_grads([z(300)])
    with pytest.raises(fp8mp.Fp8mpError):
        plan.set_grads([z(300), z(301)])


def test_a_refused_call_leaves_the_plan_as_it_was():
    z = torch.zeros
    plan = fp8mp.AdamWTensors()
    first, second = z(300), z(200)
    plan.add(first)
    for bad in (z(300, dtype=torch.float16), z(600)[::2]):
        with pytest.raises((TypeError, fp8mp.Fp8mpError)):
            plan.add(bad)
        assert len(plan) == 1
    plan.add(second)
    before = [(r.grad, r.grad_dtype, r.n) for r in plan.c_array()]
    assert before == [(first.data_ptr(), fp8mp.F32, 300), (second.data_ptr(), fp8mp.F32, 200)]
    for bad in (z(201), z(200, dtype=torch.float16), z(400)[::2]):
        with pytest.raises((TypeError, fp8mp.Fp8mpError)):
            plan.set_grads([z(300, dtype=torch.bfloat16), bad])
        assert [(r.grad, r.grad_dtype, r.n) for r in plan.c_array()] == before


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -126 * (1 - 2.0 ** -23), -1e-8])
def test_an_eps_without_a_reciprocal_is_refused(lib, eps):
    """The steps with 8-bit moments divide by flushing reciprocals: 0 / eps has to
    be 0 where a moment is."""
    assert step(lib, [row()], eps=eps) == fp8mp.ERR_INVALID
    assert "eps" in fp8mp.last_error(), fp8mp.last_error()
