"""FP8GatedMLP with its norm, FP8LMHead and TokenEmbedding without a GPU: what they
refuse, and their weights' copies, on CPU tensors with the casts in plain torch."""

import copy
import types

import pytest
import torch

import fp8_mixed_precision_reduce_gb300 as fp8mp
from fp8_mixed_precision_reduce_gb300 import adamw, embedding, gated_mlp, linear, lm_head
from test_lib_host_modules import cast, plain, step  # noqa: F401

I64 = torch.int64


def mlp(**kw):
    return gated_mlp.FP8GatedMLP(32, 48, device="cpu", norm_eps=1e-6, **kw)


def head(**kw):
    return lm_head.FP8LMHead(32, 50, device="cpu", **kw)


def table(**kw):
    return embedding.TokenEmbedding(50, 32, device="cpu", **kw)


@pytest.mark.parametrize("make", [
    lambda: gated_mlp.FP8GatedMLP(16400, 32, device="cpu", norm_eps=1e-6), lambda: gated_mlp.FP8GatedMLP(32, 32, device="cpu", norm_eps=-1.0),
    lambda: gated_mlp.FP8GatedMLP(32, 32, device="cpu", norm_eps=float("nan")), lambda: lm_head.FP8LMHead(24, 50, device="cpu"),
    lambda: lm_head.FP8LMHead(32, 0, device="cpu"), lambda: lm_head.FP8LMHead(32, 50, device="cpu", norm_eps=float("inf")),
    lambda: embedding.TokenEmbedding(50, 40, device="cpu"), lambda: embedding.TokenEmbedding(0, 32, device="cpu"),
    lambda: embedding.TokenEmbedding(50, 32, device="cpu", out_dtype=torch.float16)])
def test_sizes_that_no_kernel_takes(make):
    with pytest.raises(ValueError):
        make()


@pytest.mark.parametrize("make", [mlp, lambda: head(norm_eps=1e-6)])
def test_residuals_that_do_not_fit(make):
    m = make()
    call = (lambda x, r: m(x, r)) if isinstance(m, gated_mlp.FP8GatedMLP) else (lambda x, r: m(x, torch.zeros(4, dtype=I64), r))
    x = torch.zeros((4, 32))
    for r in (torch.zeros((3, 32)), torch.zeros((4, 32, 1)), torch.zeros((4, 32), dtype=torch.float16), torch.zeros((4, 32), device="meta")):
        with pytest.raises(ValueError, match="residual"):
            call(x, r)
    m.norm.data = torch.ones(16)
    with pytest.raises(ValueError, match="norm"):
        call(x, x)


def test_a_residual_needs_the_norm():
    x = torch.zeros((4, 32))
    with pytest.raises(ValueError, match="norm"):
        gated_mlp.FP8GatedMLP(32, 48, device="cpu")(x, x)
    with pytest.raises(ValueError, match="norm"):
        head()(x, torch.zeros(4, dtype=I64), x)


@pytest.mark.parametrize("x,t", [(torch.zeros(4, 16), torch.zeros(4, dtype=I64)), (torch.zeros(4, 32), torch.zeros(4)),
                                 (torch.zeros(4, 32), torch.zeros(5, dtype=I64)), (torch.zeros(4, 32), torch.zeros((4, 1), dtype=I64)),
                                 (torch.zeros(4, 32), torch.zeros(4, dtype=I64, device="meta"))])
def test_targets_that_do_not_fit(x, t):
    with pytest.raises(ValueError):
        head()(x, t)


@pytest.mark.parametrize("k", [0, -1, 33, 51])
def test_top_of_too_many(k):
    with pytest.raises(ValueError, match="k must"):
        head().top(torch.zeros(4, 32), k)
    with pytest.raises(ValueError, match="1..7"):
        lm_head.FP8LMHead(32, 7, device="cpu").top(torch.zeros(4, 32), 8)


@pytest.mark.parametrize("ids", [torch.zeros(3), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=I64, device="meta")])
def test_ids_that_do_not_fit(ids):
    with pytest.raises(ValueError, match="ids"):
        table()(ids)


def test_an_embedding_of_another_shape_is_refused():
    m = table()
    m.weight.data = torch.zeros((49, 32))
    with pytest.raises(ValueError, match="weight"):
        m(torch.zeros(3, dtype=I64))


def test_rows_are_dense_and_aligned():
    flat = torch.arange(200.0)
    for x in (flat[:64].view(2, 32), flat[1:65].view(2, 32), flat[:128].view(2, 64)[:, :32], flat[:64].view(32, 2).t(),
              flat[:32].expand(3, 32)):
        rows = gated_mlp._rows(x, 32)
        assert rows.is_contiguous() and rows.data_ptr() % 16 == 0 and torch.equal(rows, x.reshape(-1, 32))


def test_the_heads_added_rows_have_no_token():
    m = head()
    assert m.weight.shape == (64, 32) and (m.weight[50:] == 0).all() and (m.weight[:50] != 0).any(1).all()


def test_steps_write_the_copies(plain):  # noqa: F811
    torch.manual_seed(0)
    modules = [mlp(), head(norm_eps=1e-6), table(fp8=True), table()]
    params = [p for m in modules for p in m.parameters()]
    opt = adamw.AdamW(params, lr=1e-2, modules=modules)
    for _ in range(3):
        step(opt, *modules)
        for m in modules:
            for c, (w, meta) in zip(m.weight_copies(), m._weights()):
                assert torch.equal(c, cast(w, meta.scale))
    assert modules[3].weight_copies() == () and modules[3].metas() == []


def test_only_the_weights_have_copies(plain):  # noqa: F811
    """The norm's weight is read as it is."""
    assert len(mlp()._copies) == 2 and len(head(norm_eps=1e-6)._copies) == 1
    assert [n for n, _ in gated_mlp.FP8GatedMLP(32, 48, device="cpu").named_parameters()] == ["gate_up", "down"]


def test_a_copy_of_a_module_casts_its_own(plain):  # noqa: F811
    m = table(fp8=True)
    m.weight_copies()
    twin = copy.deepcopy(m)
    with torch.no_grad():
        twin.weight.mul_(-1)
    (mine,), (its,) = m.weight_copies(), twin.weight_copies()
    assert torch.equal(mine, cast(m.weight, m.meta_weight.scale)) and torch.equal(its, cast(twin.weight, twin.meta_weight.scale))


def test_a_weight_held_twice(plain):  # noqa: F811
    """An embedding and a head that share one weight."""
    h = lm_head.FP8LMHead(32, 64, device="cpu")
    e = embedding.TokenEmbedding(64, 32, device="cpu", fp8=True)
    e.weight = h.weight
    opt = adamw.AdamW([h.weight], lr=1e-2, modules=[h, e])
    for _ in range(2):
        step(opt, h, e)
        for m in (h, e):
            (c,), ((w, meta),) = m.weight_copies(), m._weights()
            assert torch.equal(c, cast(w, meta.scale))
    assert fp8mp.E4M3 == h.meta_weight.fmt


def test_logits_of_another_type_are_refused():
    for dtype in (torch.float16, torch.float64, None):
        with pytest.raises(ValueError, match="logits"):
            head(logits_dtype=dtype)
    assert head().logits_dtype is torch.bfloat16 and head(logits_dtype=torch.float32).logits_dtype is torch.float32


# ------------------------------- passes on the CPU, the kernels' outputs left as they are


@pytest.fixture
def no_kernels(plain, monkeypatch):  # noqa: F811
    nothing = lambda *a, **kw: None  # noqa: E731
    for mod in (gated_mlp, lm_head, embedding, linear):
        for name in dir(mod):
            if name.startswith(("fp8_", "mp_")) and callable(getattr(mod, name)) and not name.endswith("_bytes"):
                monkeypatch.setattr(mod, name, nothing)
    where = types.SimpleNamespace(stream=0, capturing=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: where.capturing)
    monkeypatch.setattr(linear, "_stream", lambda s: where.stream)
    return where


@pytest.mark.parametrize("x_dtype,r_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_the_streams_gradient_is_its_callers(no_kernels, x_dtype, r_dtype):
    """Where only the sum is used the block is an addition: the caller's gradient stays
    as it is, and has a derivative of its own."""
    m = mlp()
    x = torch.randn((4, 32)).to(x_dtype).requires_grad_(True)
    r = torch.randn((4, 32)).to(r_dtype).requires_grad_(True)
    g = torch.randn((4, 32)).to(r_dtype)
    dx, dr = torch.autograd.grad([m(x, r)[1]], [x, r], grad_outputs=[g], create_graph=True)
    assert not g.requires_grad and g.grad_fn is None
    assert torch.equal(dr, g) and torch.equal(dx, g.to(x_dtype)) and dx.dtype == x_dtype
    g.requires_grad_(True)
    dx, dr = torch.autograd.grad([m(x, r)[1]], [x, r], grad_outputs=[g], create_graph=True)
    v = torch.randn((4, 32)).bfloat16()
    (again,) = torch.autograd.grad([dx, dr], [g], grad_outputs=[v.to(x_dtype), v.to(r_dtype)])
    assert torch.equal(again, v.to(r_dtype) + v.to(r_dtype))


@pytest.fixture
def bf16_by_default():
    torch.set_default_dtype(torch.bfloat16)
    yield
    torch.set_default_dtype(torch.float32)


def test_top_under_another_default_type(no_kernels, bf16_by_default, monkeypatch):
    """What the kernels write in fp32 is fp32 whatever torch's default is."""
    seen = []
    monkeypatch.setattr(lm_head, "mp_logprobs_fwd", lambda logits, t, lp, stats, entropy=None, top_logprob=None, top_id=None, vocab=None:
                        seen.extend(x.dtype for x in (stats, lp, entropy, top_logprob) if x is not None))
    m = head(norm_eps=1e-6)
    logprob, ids = m.top(torch.zeros((4, 32)), 3, torch.zeros((4, 32)))
    with torch.no_grad():
        m(torch.zeros((4, 32)), torch.zeros(4, dtype=I64), torch.zeros((4, 32)), entropy=True)
    assert logprob.dtype is torch.float32 and ids.dtype is I64
    assert len(seen) == 5 and set(seen) == {torch.float32}


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_under_another_default_type(plain, bf16_by_default, bits):  # noqa: F811
    m = table(fp8=True)
    opt = adamw.AdamW(m.parameters(), lr=1e-2, state_bits=bits, min_8bit_size=1, modules=[m])
    for t in (opt.loss_scale, opt.beta_pows, opt.grad_norm):
        assert t.dtype is torch.float32
    step(opt, m)
    assert torch.equal(m.weight_copies()[0], cast(m.weight, m.meta_weight.scale))


def passes():
    """Of each module: a pass with its leaves."""
    lin, m, h, e = linear.FP8Linear(32, 32, device="cpu"), mlp(), head(norm_eps=1e-6), table()
    r = torch.zeros((16, 32))
    return [lambda x: lin(x), lambda x: m(x, r)[0], lambda x: h(x, torch.zeros(16, dtype=I64), r),
            lambda x: e(torch.zeros(16, dtype=I64)).float()]


@pytest.mark.parametrize("which", range(4))
def test_which_captured_backward_passes_are_refused(no_kernels, which):
    """A leaf's gradient is added up on the stream of the first pass that took it in, as
    long as any pass holds it: the default stream's cannot be captured."""
    where, run = no_kernels, passes()[which]
    x = torch.zeros((16, 32), requires_grad=True)

    def on(stream, capturing=False):
        where.stream, where.capturing = stream, capturing
        return run(x).sum()

    def refused(y):
        where.stream, where.capturing = 9, True
        try:
            y.backward()
        except RuntimeError as err:
            assert "eager pass" in str(err)
            return True
        return False

    eager = on(0)
    assert refused(on(9, True))
    side = on(5)
    assert refused(on(9, True))
    del eager  # (the leaf's node is still the first pass's)
    assert refused(on(9, True))
    captured = on(9, True)
    del side
    assert refused(captured)
    del captured
    assert not refused(on(9, True))
    side = on(5)
    eager = on(0)
    assert not refused(on(9, True))  # (an older pass than the default stream's made the node)
    del side
    assert not refused(on(9, True))
    del eager
    captured = on(9, True)
    eager = on(0)
    assert not refused(captured)
    del captured, eager
    with torch.no_grad():
        y = on(0)
    assert not refused(on(9, True)) and not y.requires_grad
    on(0).backward()
    assert not refused(on(9, True))


@pytest.mark.parametrize("first", range(3))
@pytest.mark.parametrize("second", range(3))
def test_a_leaf_of_two_modules(no_kernels, first, second):
    where, x = no_kernels, torch.zeros((16, 32), requires_grad=True)
    eager = passes()[first](x)
    where.stream, where.capturing = 9, True
    captured = passes()[second](x)
    with pytest.raises(RuntimeError, match="eager pass"):
        captured.sum().backward()
    del eager, captured
    passes()[second](x).sum().backward()


@pytest.mark.parametrize("shape", [(), (5,), (2, 3), (0,)])
def test_results_may_be_changed_in_place(no_kernels, shape):
    """As torch.nn.Embedding's and a loss's may: they are tensors of their own."""
    ids = torch.zeros(shape, dtype=I64)
    out = table(out_dtype=torch.float32)(ids)
    assert out.shape == (*shape, 32)
    out += 1
    out.sum().backward()
    for h, entropy in ((head(), False), (head(norm_eps=1e-6), True)):
        got = h(torch.zeros((*shape, 32)), ids, entropy=entropy)
        logprob = got[0] if entropy else got
        assert logprob.shape == shape and (not entropy or got[1].shape == shape)
        logprob *= 2
        logprob.sum().backward()
