"""FP8GatedMLP with its norm, FP8LMHead and TokenEmbedding together: values and
gradients against the same layers in 64 bits, streams, graphs, and the example.

The kernels have their own tests; what is checked here is the composition. Where a
GEMM's operands are rounded to FP8 the bounds are those of test_gpu_gated_mlp.py
(relative 2-norm: 5 % for each GEMM of two E4M3 operands, 10 % where an E5M2 operand
takes part); what does not pass through a GEMM is held to its own rounding."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


def norm64(t, w, eps):
    return t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps) * w


def mlp64(x, gate_up, down):
    F = gate_up.shape[0] // 2
    return (torch.nn.functional.silu(x @ gate_up[:F].T) * (x @ gate_up[F:].T)) @ down.T


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("x_dtype,r_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF), (BF, None), (F32, None)])
@pytest.mark.parametrize("shape", [(1,), (3, 11), (300,)])
def test_block_with_norm_against_64_bits(cuda_lib, shape, x_dtype, r_dtype):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(1)
    mlp = FP8GatedMLP(272, 528, norm_eps=1e-6)
    with torch.no_grad():
        mlp.norm.add_(torch.randn(272, device="cuda") * 0.1)
    for turn in range(2):  # the first pass fills the histories, the second runs under their scales
        x = torch.randn((*shape, 272), device="cuda").to(x_dtype).requires_grad_(True)
        r = (torch.randn((*shape, 272), device="cuda") * 3).to(r_dtype).requires_grad_(True) if r_dtype else None
        dy = (torch.randn((*shape, 272), device="cuda") * 1e-3).to(x_dtype)
        dt = (torch.randn((*shape, 272), device="cuda") * 1e-3).to(r_dtype or x_dtype)
        mlp.zero_grad(set_to_none=True)
        y, total = mlp(x, r)
        torch.autograd.backward([y, total], [dy, dt])
        assert cuda_lib.fp8mp_check() == 0
        if turn == 0:
            mlp.update_scales()
    leaves = [t.detach().double().requires_grad_(True) for t in (x, mlp.norm, mlp.gate_up, mlp.down)]
    rd = r.detach().double().requires_grad_(True) if r_dtype else None
    xd, nd, gd, dd = leaves
    td = xd + rd if r_dtype else xd
    yd = mlp64(norm64(td, nd, 1e-6), gd, dd)
    torch.autograd.backward([yd, td], [dy.double(), dt.double()])
    assert y.shape == total.shape == x.shape and y.dtype == x_dtype and total.dtype == (r_dtype or x_dtype)
    if r_dtype:
        assert torch.equal(total, (x.float() + r.float()).to(r_dtype))
    else:
        assert total is x
    assert relative(y, yd.detach()) < 0.10
    grads = [(x.grad, xd.grad), (mlp.norm.grad, nd.grad), (mlp.gate_up.grad, gd.grad), (mlp.down.grad, dd.grad)]
    if r_dtype:
        grads.append((r.grad, rd.grad))
        assert r.grad.dtype == r_dtype
    for got, want in grads:
        assert got.shape == want.shape and relative(got, want) < 0.25


def test_the_stream_alone(cuda_lib):
    """Gradients of the sum, or of y, alone."""
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP

    torch.manual_seed(2)
    mlp = FP8GatedMLP(64, 96, norm_eps=1e-6)
    x, r = (torch.randn((24, 64), device="cuda", requires_grad=True) for _ in range(2))
    g = torch.randn((24, 64), device="cuda")
    mlp(x, r)[1].backward(g)
    assert torch.equal(x.grad, g) and torch.equal(r.grad, g) and mlp.norm.grad is None
    x.grad = r.grad = None
    mlp(x, r)[0].backward(g)
    only = x.grad.clone()
    assert torch.equal(x.grad, r.grad) and mlp.norm.grad is not None
    x.grad = r.grad = None
    y, total = mlp(x, r)
    torch.autograd.backward([y, total], [g, g])
    assert torch.allclose(x.grad, only + g, rtol=1e-6, atol=1e-6)
    # parts without gradients
    for frozen in ([mlp.gate_up, mlp.down], [mlp.norm], [mlp.norm, mlp.gate_up, mlp.down]):
        for p in mlp.parameters():
            p.requires_grad_(not any(p is q for q in frozen))
            p.grad = None
        x.grad = None
        mlp(x, r.detach())[0].backward(g)
        assert torch.equal(x.grad, only) and all(p.grad is None for p in frozen)
    with torch.no_grad():
        y2, total2 = mlp(x, r)
        assert torch.equal(y2, y) and torch.equal(total2, total)


@pytest.mark.parametrize("shape", [(24, 64), (4, 6, 64)])
def test_gradients_of_x_and_the_residual_are_apart(cuda_lib, shape):
    """They are equal, but what accumulates into one is not the other's."""
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(9)
    g = torch.randn(shape, device="cuda")
    t = torch.randint(0, 30, shape[:-1], device="cuda")
    mlp, head = FP8GatedMLP(64, 96, norm_eps=1e-6), FP8LMHead(64, 30, norm_eps=1e-6)
    for out in (lambda x, r: (mlp(x, r)[0] * g).sum(), lambda x, r: (mlp(x, r)[1] * g).sum(), lambda x, r: head(x, t, r).sum()):
        x, r = (torch.randn(shape, device="cuda", requires_grad=True) for _ in range(2))
        out(x, r).backward()
        once = x.grad.clone()
        assert torch.equal(r.grad, once) and x.grad.data_ptr() != r.grad.data_ptr()
        out(x, r).backward()
        assert torch.equal(x.grad, 2 * once) and torch.equal(r.grad, 2 * once)
        x.grad = None
        out(x, x).backward()  # (x + x is another norm's input: the gradients add up)
        assert x.grad.shape == x.shape and torch.isfinite(x.grad).all()


def test_no_second_derivative(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    x = torch.randn((16, 64), device="cuda", requires_grad=True)
    r = torch.randn((16, 64), device="cuda", requires_grad=True)
    t = torch.zeros(16, dtype=torch.int64, device="cuda")
    e = TokenEmbedding(30, 64)
    for out, of in ((FP8GatedMLP(64, 96, norm_eps=1e-6)(x, r)[0], (x, r)), (FP8LMHead(64, 30)(x, t), (x,)),
                    (e(t).float(), (e.weight,))):
        grads = torch.autograd.grad(out.square().sum(), of, create_graph=True)
        with pytest.raises(RuntimeError, match="second"):
            sum(g.square().sum() for g in grads).backward()


@pytest.mark.parametrize("x_dtype,r_dtype", [(BF, None), (F32, None), (BF, F32)])
@pytest.mark.parametrize("tokens,vocab", [((1,), 17), ((2, 9), 1000), ((129,), 4096), ((333,), 5003)])
def test_head_against_64_bits(cuda_lib, tokens, vocab, x_dtype, r_dtype):
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(3)
    head = FP8LMHead(272, vocab, norm_eps=1e-6 if r_dtype else None)
    with torch.no_grad():
        head.weight.mul_(4)
    t = torch.randint(0, vocab, tokens, device="cuda")
    if t.numel() > 2:
        t.view(-1)[1] = -100
    for turn in range(2):
        x = torch.randn((*tokens, 272), device="cuda").to(x_dtype).requires_grad_(True)
        r = torch.randn((*tokens, 272), device="cuda").to(r_dtype).requires_grad_(True) if r_dtype else None
        da, db = torch.randn(tokens, device="cuda"), torch.randn(tokens, device="cuda") * 0.1
        head.zero_grad(set_to_none=True)
        logprob, entropy = head(x, t, r, entropy=True)
        torch.autograd.backward([logprob, entropy], [da, db])
        assert cuda_lib.fp8mp_check() == 0
        if turn == 0:
            head.update_scales()
    xd, wd = x.detach().double().requires_grad_(True), head.weight.detach()[:vocab].double().requires_grad_(True)
    n = xd
    if r_dtype:
        rd, nd = r.detach().double().requires_grad_(True), head.norm.detach().double().requires_grad_(True)
        n = norm64(xd + rd, nd, 1e-6)
    logits = n @ wd.T
    logp = torch.log_softmax(logits, -1)
    given = t >= 0
    at = torch.where(given, logp.gather(-1, t.clamp_min(0)[..., None])[..., 0], 0.0)
    H = -(logp.exp() * logp).sum(-1)
    # the logits' gradient saturates at the largest of the pass before (of one token whose
    # weight was a tenth of this pass's, a tenth is left): 57344 / scale
    (dlogits,) = torch.autograd.grad([at, H], logits, [da.double(), db.double()], retain_graph=True)
    most = 57344.0 / head.meta_dlogits.scale.item()
    logits.backward(dlogits.clamp(-most, most))
    assert logprob.shape == entropy.shape == t.shape and logprob.dtype == F32
    assert (logprob[~given] == 0).all()
    # the logits have a spread of 4 and 5 % of it as error, and log p one logit's and the sum's
    assert (logprob.double() - at.detach()).square().mean().sqrt().item() < 0.5
    assert (entropy.double() - H.detach()).square().mean().sqrt().item() < 0.5
    assert head.weight.grad.shape == head.weight.shape and not head.weight.grad[vocab:].any()
    grads = [(x.grad, xd.grad), (head.weight.grad[:vocab], wd.grad)]
    if r_dtype:
        grads += [(r.grad, rd.grad), (head.norm.grad, nd.grad)]
    for got, want in grads:
        assert relative(got, want) < 0.25
    assert head.dw_nonfinite.item() == 0


def test_head_is_its_kernels(cuda_lib):
    """The same calls by hand give the same bits."""
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(4)
    M, K, V = 48, 64, 500
    head = FP8LMHead(K, V)
    x = torch.randn((M, K), device="cuda", requires_grad=True)
    t = torch.randint(0, V, (M,), device="cuda")
    logprob, entropy = head(x, t, entropy=True)
    da = torch.randn(M, device="cuda")
    logprob.backward(da)
    X8 = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    (W8,) = head.weight_copies()
    one = torch.ones(1, device="cuda")
    cuda_lib.fp8_quantize(x.detach(), cuda_lib.E4M3, one, X8)
    logits = torch.empty((M, 512), dtype=BF, device="cuda")
    cuda_lib.fp8_linear_few(X8, W8, one, one, logits)
    stats, lp, H = torch.empty((M, 2), device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    cuda_lib.mp_logprobs_fwd(logits, t, lp, stats, entropy=H, vocab=V)
    assert torch.equal(lp, logprob) and torch.equal(H, entropy) and torch.equal(head(x, t), logprob)
    D8 = torch.empty((M, 512), dtype=torch.uint8, device="cuda")
    cuda_lib.mp_logprobs_bwd(logits, t, stats, da, D8, scale=one, vocab=V)
    dx, dw = torch.empty_like(x), torch.empty_like(head.weight)
    cuda_lib.fp8_linear_bwd_rowmajor(D8, W8, X8, one, one, one, dx, dw)
    assert torch.equal(dx, x.grad) and torch.equal(dw, head.weight.grad)
    top, ids = head.top(x, 5)
    want = torch.sort(logits[:, :V].float(), dim=1, descending=True, stable=True).indices[:, :5]
    assert torch.equal(ids, want)
    assert torch.allclose(top, torch.log_softmax(logits[:, :V].float(), 1).gather(1, want), atol=1e-5)


@pytest.mark.parametrize("tokens", [(), (1,), (128,), (3, 67), (300,)])
def test_top_of_any_number_of_tokens(cuda_lib, tokens):
    """As log p of the tokens that it gives, and as each token alone."""
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(10)
    head = FP8LMHead(64, 1003, norm_eps=1e-6)
    x, r = (torch.randn((*tokens, 64), device="cuda").to(BF) for _ in range(2))
    logprob, ids = head.top(x, 4, r)
    assert logprob.shape == ids.shape == (*tokens, 4) and ids.dtype == torch.int64
    for i in range(4):
        assert torch.allclose(head(x, ids[..., i].contiguous(), r).detach(), logprob[..., i], rtol=1e-5, atol=1e-5)
    if tokens:
        flat = lambda t: t.reshape(-1, 64)  # noqa: E731
        for m in (0, x.numel() // 64 - 1):
            _, alone = head.top(flat(x)[m], 1, flat(r)[m])
            assert alone[0] == ids.reshape(-1, 4)[m, 0]


def test_inputs_of_other_strides_and_broadcast_ones(cuda_lib):
    """The same values as dense tensors give the same bits; gradients gather where the
    strides say."""
    from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(11)
    mlp, head, e = FP8GatedMLP(64, 96, norm_eps=1e-6), FP8LMHead(64, 30, norm_eps=1e-6), TokenEmbedding(30, 64, out_dtype=F32)
    base = torch.randn(4 * 9 * 64 + 3, device="cuda", requires_grad=True)
    ids = torch.randint(0, 30, (9, 8), device="cuda").t()[::2]
    assert ids.shape == (4, 9) and not ids.is_contiguous()
    for shape, stride, offset in (((4, 9, 64), (576, 64, 1), 1), ((4, 9, 64), (64, 256, 1), 0), ((4, 9, 64), (0, 64, 1), 0),
                                  ((4, 9, 64), (9, 1, 36), 3)):
        x = base.as_strided(shape, stride, offset)
        dense = x.detach().contiguous().clone().requires_grad_(True)
        r = torch.randn(shape, device="cuda")
        y, total = mlp(x, r)
        y2, total2 = mlp(dense, r)
        assert torch.equal(y, y2) and torch.equal(total, total2)
        assert torch.equal(head(r, ids, x), head(r, ids.contiguous(), dense))
        base.grad = None
        y.sum().backward()
        y2.sum().backward()
        places = torch.arange(base.numel(), device="cuda").as_strided(shape, stride, offset).reshape(-1)
        want = torch.zeros_like(base).index_put_((places,), dense.grad.reshape(-1), accumulate=True)
        assert torch.allclose(base.grad, want, rtol=1e-5, atol=1e-6)
    out = e(ids)
    assert torch.equal(out, e(ids.contiguous()))
    out.backward(torch.ones(1, device="cuda").expand(4, 9, 64))
    count = torch.bincount(ids.reshape(-1), minlength=30).float()
    assert torch.equal(e.weight.grad, count[:, None].expand(30, 64))


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64)])
def test_no_tokens(cuda_lib, shape):
    from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    mlp, head = FP8GatedMLP(64, 96, norm_eps=1e-6), FP8LMHead(64, 30, norm_eps=1e-6)
    x, r = (torch.zeros(shape, device="cuda", requires_grad=True) for _ in range(2))
    y, total = mlp(x, r)
    logprob, entropy = head(y, torch.zeros(shape[:-1], dtype=torch.int64, device="cuda"), total, entropy=True)
    (logprob.sum() + entropy.sum()).backward()
    assert y.shape == total.shape == shape and logprob.shape == shape[:-1] and x.grad.shape == shape
    assert all((p.grad == 0).all() for m in (mlp, head) for p in m.parameters())
    assert head.top(x, 3, r)[1].shape == (*shape[:-1], 3) and cuda_lib.fp8mp_check() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype,out", [(F32, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("shape", [(), (1,), (4, 33), (0,), (2, 0)])
def test_embedding(cuda_lib, shape, dtype, out, fp8):
    from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding

    torch.manual_seed(5)
    e = TokenEmbedding(300, 48, scale=3.0, fp8=fp8, dtype=dtype, out_dtype=out)
    ids = torch.randint(-20, 320, shape, device="cuda")
    y = e(ids)
    inside = (ids >= 0) & (ids < 300)
    table = e.weight.detach().float()
    if fp8:
        table = (table * 1.0).clamp(-448, 448).to(torch.float8_e4m3fn).float()  # (the first scale is 1)
    want = torch.where(inside[..., None], table[ids.clamp(0, 299)] * 3.0, 0.0).to(out)
    assert torch.equal(y, want) and y.dtype == out and y.shape == (*shape, 48)
    dy = torch.randn_like(y)
    y.backward(dy)
    g = torch.zeros((300, 48), dtype=torch.float64, device="cuda")
    g.index_put_((ids[inside],), dy[inside].double() * 3.0, accumulate=True)
    assert e.weight.grad.dtype == dtype
    assert torch.allclose(e.weight.grad.double(), g, rtol=1e-2 if dtype == BF else 1e-5, atol=1e-5)
    assert cuda_lib.fp8mp_check() == 0


def test_embedding_and_head_of_one_weight(cuda_lib):
    from fp8_mixed_precision_reduce_gb300.adamw import AdamW
    from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(6)
    head = FP8LMHead(64, 256)
    e = TokenEmbedding(256, 64, fp8=True)
    e.weight = head.weight
    opt = AdamW([head.weight], lr=1e-3, modules=[head, e], loss_scale=1024.0)
    ids = torch.randint(0, 256, (100,), device="cuda")
    for _ in range(3):
        opt.zero_grad()
        (-head(e(ids), ids).mean() * opt.loss_scale).sum().backward()
        both = head.weight.grad.clone()
        head.weight.grad = None
        x = e(ids).detach()
        (-head(x, ids).mean() * opt.loss_scale).sum().backward()
        assert not torch.equal(both, head.weight.grad)  # (the lookup's part)
        head.weight.grad = both
        head.update_scales()
        e.update_scales()
        opt.step()
        for m in (head, e):
            ((w, meta),) = m._weights()
            want = (w.detach() * meta.scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(m.weight_copies()[0], want)
    assert opt.found_inf.item() == 0 and cuda_lib.fp8mp_check() == 0


def model(cuda_lib, seed=7):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_language_model as ex

    torch.manual_seed(seed)
    return ex.Model(500, 64, 96, 2)


def passes(m, ids):
    logprob, entropy = m(ids[:, :-1], ids[:, 1:], entropy=True)
    (-logprob.mean() - 0.01 * entropy.mean()).backward()
    return logprob, entropy


def test_a_model_on_another_stream(cuda_lib):
    m = model(cuda_lib)
    ids = torch.randint(0, 500, (8, 20), device="cuda")
    want = passes(m, ids)
    grads = [p.grad.clone() for p in m.parameters()]
    m.zero_grad(set_to_none=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = passes(m, ids)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(p.grad, g) for p, g in zip(m.parameters(), grads))


def test_serving_from_a_graph(cuda_lib):
    m = model(cuda_lib).eval()
    ids = torch.randint(0, 500, (5,), device="cuda")
    with torch.no_grad():
        m.top(ids, 3)  # (the weights are cast)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logprob, tokens = m.top(ids, 3)
        for seed in range(3):
            ids.copy_(torch.randint(-1, 500, (5,), device="cuda"))
            graph.replay()
            want = m.top(ids, 3)
            assert torch.equal(logprob, want[0]) and torch.equal(tokens, want[1])
        m.head.weight.mul_(-1)
        m.head.weight_copies()
        graph.replay()
        assert torch.equal(tokens, m.top(ids, 3)[1])


def test_a_training_pass_from_a_graph(cuda_lib):
    m = model(cuda_lib)
    ids = torch.randint(0, 500, (8, 20), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (as captures of a backward pass ask for)
        passes(m, ids)
    torch.cuda.current_stream().wait_stream(side)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logprob, _ = passes(m, ids)
    for seed in range(2):
        ids.copy_(torch.randint(0, 500, (8, 20), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [logprob.clone()] + [p.grad.clone() for p in m.parameters()]
        twin = model(cuda_lib)
        want = [passes(twin, ids)[0]] + [p.grad for p in twin.parameters()]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


CAPTURED_BESIDE_AN_EAGER_PASS = """
import torch
from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding
from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

e, head, mlp = TokenEmbedding(30, 64), FP8LMHead(64, 30, norm_eps=1e-6), FP8GatedMLP(64, 96, norm_eps=1e-6)
ids = torch.randint(0, 30, (8,), device="cuda")
r = torch.randn(8, 64, device="cuda")
for run, module in ((lambda: e(ids), e), (lambda: head(r, ids), head), (lambda: mlp(r)[0], mlp)):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run().float().sum().backward()
    torch.cuda.current_stream().wait_stream(side)
    module.zero_grad(set_to_none=True)
    eager = run()
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            run().float().sum().backward()
        print("captured")
    except RuntimeError as err:
        print("refused" if "eager pass" in str(err) else err)
    with torch.no_grad():
        y = run()
    del eager
    module.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run().float().sum().backward()
    graph.replay()
    got = [p.grad.clone() for p in module.parameters()]
    module.zero_grad(set_to_none=True)
    run().float().sum().backward()
    print("same" if all(torch.equal(a, p.grad) for a, p in zip(got, module.parameters())) else "other")
"""


def test_a_captured_backward_pass_beside_an_eager_graph_is_refused(cuda_lib):
    """In a process of its own: without the refusal it would end."""
    r = subprocess.run([sys.executable, "-c", CAPTURED_BESIDE_AN_EAGER_PASS], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["refused", "same"] * 3, r.stdout


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_runs(cuda_lib, bits):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_language_model as ex

    losses, good = ex.run(vocab=203, features=64, hidden=96, blocks=2, batch=8, length=15, steps=6, bits=bits, log=lambda s: None)
    assert len(losses) == 6 and all(0 < x < 50 for x in losses) and 0 <= good <= 1
    assert cuda_lib.fp8mp_check() == 0


def test_a_models_gradients_against_differences_of_scales(cuda_lib):
    """The gradient of the whole model's loss with respect to each norm's weight, scaled
    by (1 + h) and (1 - h): differences of the FP8 model are no use (its codes jump), so
    of the same model in 64 bits."""
    m = model(cuda_lib)
    ids = torch.randint(0, 500, (16, 33), device="cuda")
    for _ in range(2):
        m.zero_grad(set_to_none=True)
        logprob = m(ids[:, :-1], ids[:, 1:])
        (-logprob.mean() * 1024).backward()
        for f in m.fp8_modules():
            f.update_scales()

    def loss(factor):
        e = m.embedding
        x, r = e.weight.double()[ids[:, :-1]] * e.scale, None
        for b in m.blocks:
            t = x if r is None else x + r
            x, r = mlp64(norm64(t, b.norm.double() * factor, 1e-6), b.gate_up.double(), b.down.double()), t
        n = norm64(x + r, m.head.norm.double(), 1e-6)
        logp = torch.log_softmax(n @ m.head.weight.double()[:500].T, -1)
        return -logp.gather(-1, ids[:, 1:, None]).mean().item()

    with torch.no_grad():
        h = 1e-4
        want = (loss(1 + h) - loss(1 - h)) / (2 * h) * 1024
        got = sum((b.norm.grad.double() * b.norm.double()).sum().item() for b in m.blocks)
        size = sum((b.norm.grad.double() * b.norm.double()).norm().item() for b in m.blocks)
    assert abs(got - want) <= 0.25 * max(abs(want), size), (got, want)


@pytest.mark.parametrize("tokens", [(1,), (2, 9), (333,)])
@pytest.mark.parametrize("x_dtype", [BF, F32])
def test_head_with_logits_in_fp32(cuda_lib, tokens, x_dtype):
    """The same calls by hand with fp32 logits give the same bits; and of the product of
    the codes in 64 bits the logits are off by no more than fp32 sums are: 64 products of
    two 4-bit significands, exact, added with fewer than 64 roundings (of up to 2^-22 of the
    terms' sum, where the tensor core cuts), and two scales. log p moves by at most twice
    the largest error of a logit; x - m and its product with log2(e) round by 2^-24 of
    at most twice the largest logit each, the difference by 2^-24 of itself, and the 500 terms
    of S and their sum by less than 2^-22 a term."""
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    torch.manual_seed(12)
    K, V = 64, 500
    head = FP8LMHead(K, V, logits_dtype=F32)
    with torch.no_grad():
        head.weight.mul_(8)
    x = (torch.randn((*tokens, K), device="cuda") * 4).to(x_dtype).requires_grad_(True)
    t = torch.randint(0, V, tokens, device="cuda")
    logprob, entropy = head(x, t, entropy=True)
    da = torch.randn(tokens, device="cuda")
    logprob.backward(da)
    M, rows = x.numel() // K, (x.numel() // K + 15) // 16 * 16
    X8 = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
    (W8,) = head.weight_copies()
    one = torch.ones(1, device="cuda")
    cuda_lib.fp8_quantize(x.detach().reshape(M, K), cuda_lib.E4M3, one, X8[:M])
    logits = torch.empty((rows, 512), device="cuda")
    if M <= cuda_lib.FEW_TOKENS:
        cuda_lib.fp8_linear_few(X8[:M], W8, one, one, logits[:M])
    else:
        cuda_lib.fp8_linear_fwd(X8, W8, one, one, logits)
    logits = logits[:M]
    stats, lp, H = torch.empty((M, 2), device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    cuda_lib.mp_logprobs_fwd(logits, t.reshape(-1), lp, stats, entropy=H, vocab=V)
    assert torch.equal(lp, logprob.reshape(-1)) and torch.equal(H, entropy.reshape(-1))
    D8 = torch.zeros((rows, 512), dtype=torch.uint8, device="cuda")
    cuda_lib.mp_logprobs_bwd(logits, t.reshape(-1), stats, da.reshape(-1), D8[:M], scale=one, vocab=V)
    dx, dw = torch.empty((rows, K), dtype=x_dtype, device="cuda"), torch.empty_like(head.weight)
    cuda_lib.fp8_linear_bwd_rowmajor(D8, W8, X8, one, one, one, dx, dw)
    assert torch.equal(dx[:M].reshape(x.shape), x.grad) and torch.equal(dw, head.weight.grad)
    xd, wd = (c.view(torch.float8_e4m3fn).double() for c in (X8[:M], W8[:V]))
    exact, room = xd @ wd.T, 66 * 2.0 ** -22 * (xd.abs() @ wd.abs().T)
    logp = torch.log_softmax(exact, -1)
    want = logp.gather(1, t.reshape(-1, 1))[:, 0]
    worst = room.max(1).values  # log p is off by the target's logit and by a mean of all of them
    bound = 2 * worst + 2.0 ** -23 * (2 * exact.abs().max(1).values + want.abs() + 8) + 500 * 2.0 ** -22
    assert ((logprob.detach().reshape(-1).double() - want).abs() <= bound).all()
    assert cuda_lib.fp8mp_check() == 0


def test_top_of_logits_that_bf16_makes_equal(cuda_lib):
    """Logits of 17 and 17 + 2^-6: equal in bf16, where the lower token comes first."""
    from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

    for dtype, want in ((None, [3, 7]), (BF, [3, 7]), (F32, [7, 3])):
        head = FP8LMHead(32, 40, **({} if dtype is None else dict(logits_dtype=dtype)))
        with torch.no_grad():
            head.weight.zero_()
            head.weight[3, 0] = head.weight[7, 0] = 16.0
            head.weight[3, 1] = head.weight[7, 1] = 1.0
            head.weight[7, 2] = 2.0 ** -6
        x = torch.ones((3, 32), device="cuda")
        logprob, ids = head.top(x, 2)
        assert ids.tolist() == [want] * 3
        gap = logprob[:, 0] - logprob[:, 1]  # (of two values in (-1, -0.5), rounded by 2^-25 each)
        assert ((gap - (2.0 ** -6 if dtype is F32 else 0.0)).abs() <= 2.0 ** -24).all()


WHICH_CAPTURES_ARE_REFUSED = """
import torch
from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding
from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP
from fp8_mixed_precision_reduce_gb300.linear import FP8Linear
from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead

linear, e, head, mlp = FP8Linear(64, 64), TokenEmbedding(30, 64), FP8LMHead(64, 30, norm_eps=1e-6), FP8GatedMLP(64, 96, norm_eps=1e-6)
ids = torch.randint(0, 30, (16,), device="cuda")
r = torch.randn(16, 64, device="cuda")

def beside(run, stream):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        y = run()
    torch.cuda.current_stream().wait_stream(stream)
    return y

for run, module in ((lambda: linear(r), linear), (lambda: e(ids), e), (lambda: head(r, ids), head), (lambda: mlp(r)[0], mlp)):
    side = torch.cuda.Stream()

    def refused():
        module.zero_grad(set_to_none=True)
        try:
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                run().float().sum().backward()
        except RuntimeError as err:
            assert "eager pass" in str(err), err
            return True
        return False

    beside(run, side).float().sum().backward()
    eager = run()
    assert refused()
    later = beside(run, side)
    del eager  # (the leaves' nodes are still the first pass's)
    assert refused()
    del later
    older = beside(run, side)
    eager = run()
    module.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run().float().sum().backward()
    graph.replay()
    torch.cuda.synchronize()
    got = [p.grad.clone() for p in module.parameters()]
    del older, eager, graph
    module.zero_grad(set_to_none=True)
    run().float().sum().backward()
    assert all(torch.equal(a, p.grad) for a, p in zip(got, module.parameters()))
    print("ok")
"""


def test_which_captured_backward_passes_are_refused(cuda_lib):
    """In a process of its own: what should be refused would end it."""
    r = subprocess.run([sys.executable, "-c", WHICH_CAPTURES_ARE_REFUSED], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["ok"] * 4, r.stdout


def test_every_gradient_of_the_examples_model_against_64_bits(cuda_lib):
    """Embedding, two blocks and head in a training pass. The bounds are the sums of the
    parts' (5 % for each rounding to E4M3 or product of it, 10 % where an E5M2 operand takes
    part) over the longest way to a gradient: forward through the table's copy, four GEMMs
    and the head (30 %), backward through the head (10 %), two a block (40 %) and
    a weight's product (10 %). Less than 1, which no gradient of a wrong sign or of
    another input would be."""
    m = model(cuda_lib)
    ids = torch.randint(0, 500, (16, 33), device="cuda")
    for turn in range(2):  # the first pass fills the histories, the second runs under their scales
        m.zero_grad(set_to_none=True)
        logprob = m(ids[:, :-1], ids[:, 1:])
        (-logprob.mean() * 1024).backward()
        if turn == 0:
            for f in m.fp8_modules():
                f.update_scales()
    of = {n: p.detach().double().requires_grad_(True) for n, p in m.named_parameters()}
    x, r = of["embedding.weight"][ids[:, :-1]] * m.embedding.scale, None
    for i in range(len(m.blocks)):
        t = x if r is None else x + r
        x, r = mlp64(norm64(t, of[f"blocks.{i}.norm"], 1e-6), of[f"blocks.{i}.gate_up"], of[f"blocks.{i}.down"]), t
    logits = norm64(x + r, of["head.norm"], 1e-6) @ of["head.weight"][:500].T
    want = torch.log_softmax(logits, -1).gather(-1, ids[:, 1:, None])[..., 0]
    (-want.mean() * 1024).backward()
    assert relative(logprob.detach() - logprob.detach().mean(), (want - want.mean()).detach()) < 0.6
    worst = {n: relative(p.grad, of[n].grad) for n, p in m.named_parameters()}
    assert len(worst) == 9 and all(w < 0.9 for w in worst.values()), worst
