"""fp8_rmsnorm_fwd and fp8_rmsnorm_bwd against the formulas in 64 bits.

Tolerances. u = 2^-24. The sum of squares: a thread adds at most 16 pairs' squares one
after another, then 5 + 5 shuffles and one join of the pair's halves, all of one sign,
so it is good to 27 u; rstd takes half of that and four operations of its own: 18 u,
20 allowed. y has two products more.
Backward: each of n, g, g n is rounded once or twice; the mean has 27 u of the sum
of |g n|; the bounds below count them. Outputs add half a step of their type."""

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 16), (9, 16), (5, 272), (300, 1024), (3, 1040), (77, 2736), (2, 4096), (1237, 4096), (4, 8192), (3, 8208),
         (2, 16384), (0, 64), (700, 16384), (500, 6160), (6000, 1024), (11000, 272),
         (200, 11472), (4250, 3584), (4300, 3584), (4300, 5616), (700, 3600)]


def guarded(shape, dtype):
    """A tensor in the middle of a buffer, and a check that what surrounds it is as it was."""
    n = 1
    for d in shape:
        n *= d
    flat = torch.full((n + 128,), 77, dtype=dtype, device="cuda")

    def check():
        assert (flat[:64] == 77).all() and (flat[64 + n:] == 77).all()

    return flat[64:64 + n].view(shape), check


def inputs(M, K, x, t, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * M + K)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    channel = torch.exp(r(K))
    return (r(M, K) * 2).to(x), (r(M, K) * channel).to(t), 1 + 0.2 * r(K), r


def within(got, want, bound, what):
    bad = ((got.double() - want).abs() > bound) | ~torch.isfinite(got.double())
    assert not bad.any(), (what, int(bad.sum()), ((got.double() - want).abs() / bound)[bad].max().item())


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("x,t,y", [(BF, BF, "e4m3"), (BF, F32, BF), (F32, F32, F32), (F32, BF, "e4m3"), (BF, None, "e4m3"),
                                   (F32, None, BF)])
def test_forward(cuda_lib, M, K, x, t, y):
    xs, rs, w, _ = inputs(M, K, x, t or F32)
    w = w.to(BF) if K % 32 else w
    scale, amax = torch.tensor([20.0], device="cuda"), torch.full((1,), 1e-3, device="cuda")
    out, check = guarded((M, K), torch.uint8 if y == "e4m3" else y)
    rstd, check_r = guarded((M,), F32)
    total, check_t = guarded((M, K), t) if t else (None, lambda: None)
    cuda_lib.fp8_rmsnorm_fwd(xs, w, out, rstd, eps=1e-5, residual=rs if t else None, total=total,
                             y_scale=scale if y == "e4m3" else None, y_amax=amax)
    assert cuda_lib.fp8mp_check() == 0
    check(), check_r(), check_t()
    s = xs
    if t:
        s = (xs.float() + rs.float()).to(t)
        assert torch.equal(total, s)
    s = s.double()
    want_r = 1 / torch.sqrt(s.square().mean(1) + 1e-5)
    within(rstd, want_r, 20 * U * want_r, "rstd")
    want = s * want_r[:, None] * w.double()
    if y == "e4m3":
        v = (want * 20.0).clamp(-448, 448)
        within(out.view(torch.float8_e4m3fn).float(), v, (2.0 ** -4 + 24 * U) * v.abs() + 2.0 ** -10, "codes")
    else:
        within(out, want, (HALF[y] + 24 * U) * want.abs(), "y")
    most = max(1e-3, want.abs().max().item() if M else 0.0)
    assert abs(amax.item() - most) <= 24 * U * most


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dy,t,stream,dx", [(BF, BF, True, False), (BF, F32, True, True), (F32, F32, False, False),
                                            (F32, BF, False, True)])
@pytest.mark.parametrize("weight", [BF, F32])
def test_backward(cuda_lib, M, K, dy, t, stream, dx, weight):
    dys, ts, w, r = inputs(M, K, dy, t, 1)
    w = w.to(weight)
    rstd = (1 / torch.sqrt(ts.double().square().mean(1) + 1e-6)).float()
    dt = r(M, K).to(t) if stream else None
    dr, check = guarded((M, K), t)
    dxs, check_x = guarded((M, K), dy) if dx else (None, lambda: None)
    dw, check_w = guarded((K,), weight)
    ws, check_s = guarded((max(16, cuda_lib.fp8_rmsnorm_bwd_workspace_bytes(M, K)),), torch.uint8)
    cuda_lib.fp8_rmsnorm_bwd(dys, ts, w, rstd, dr, dw, ws, dtotal=dt, dx=dxs)
    assert cuda_lib.fp8mp_check() == 0
    check(), check_x(), check_w(), check_s()
    n = ts.double() * rstd.double()[:, None]
    g = dys.double() * w.double()
    c, ca = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    want = rstd.double()[:, None] * (g - n * c)
    slack = rstd.double()[:, None] * (4 * g.abs() + n.abs() * (40 * ca + 4 * c.abs())) * U
    if stream:
        want = want + dt.double()
    within(dr, want, HALF[t] * (want.abs() + slack) + slack + 2 * U * want.abs(), "dresidual")
    if dx:
        within(dxs, want, HALF[dy] * (want.abs() + slack) + slack + 2 * U * want.abs(), "dx")
    each = dys.double() * n
    loose = (M / 456 + 32) * U * each.abs().sum(0)
    within(dw, each.sum(0), HALF[weight] * (each.sum(0).abs() + loose) + loose, "dw")
    again = torch.empty_like(dw)
    cuda_lib.fp8_rmsnorm_bwd(dys, ts, w, rstd, torch.empty_like(dr), again, ws, dtotal=dt)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("K", [64, 2048])
def test_gradient_is_the_differences(cuda_lib, K):
    """The sum of y dy at t + h d and t - h d, in 64 bits, against the gradient along d."""
    M = 6
    _, t, w, r = inputs(M, K, F32, F32, 2)
    dy, d = r(M, K), r(M, K)
    rstd = (1 / torch.sqrt(t.double().square().mean(1) + 1e-6)).float()
    dr, dw = torch.empty_like(t), torch.empty_like(w)
    ws = torch.empty(cuda_lib.fp8_rmsnorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_rmsnorm_bwd(dy, t, w, rstd, dr, dw, ws)

    def f(s, v):
        return (s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * v * dy.double()).sum().item()

    h, e = 1e-5, r(K).double()
    td, wd = t.double(), w.double()
    by_t = (f(td + h * d.double(), wd) - f(td - h * d.double(), wd)) / (2 * h)
    by_w = (f(td, wd + h * e) - f(td, wd - h * e)) / (2 * h)
    # the differences are off by h^2 times a third derivative and 2^-53 f / h; both far below the kernel's rounding
    room = 1e-5
    assert abs(by_t - (dr.double() * d.double()).sum().item()) <= room * (dr.double() * d.double()).abs().sum().item()
    assert abs(by_w - (dw.double() * e).sum().item()) <= room * (dw.double() * e).abs().sum().item() + 1e-6


def test_in_place(cuda_lib):
    M, K = 37, 528
    x, r, w, rnd = inputs(M, K, BF, F32, 3)
    y, y2 = (torch.empty((M, K), dtype=BF, device="cuda") for _ in range(2))
    rstd, total = torch.empty(M, device="cuda"), torch.empty_like(r)
    cuda_lib.fp8_rmsnorm_fwd(x, w, y, rstd, residual=r, total=total)
    own = r.clone()
    cuda_lib.fp8_rmsnorm_fwd(x, w, y2, rstd, residual=own, total=own)
    assert torch.equal(own, total) and torch.equal(y, y2)
    dt = rnd(M, K)
    dr, own = torch.empty_like(dt), dt.clone()
    cuda_lib.fp8_rmsnorm_bwd(x, total, w, rstd, dr, dtotal=dt)
    cuda_lib.fp8_rmsnorm_bwd(x, total, w, rstd, own, dtotal=own)
    assert torch.equal(own, dr)


@pytest.mark.parametrize("K", [256, 4096])
def test_rows_of_zeros_nan_and_infinities(cuda_lib, K):
    """Each in its own row; the others are as without them."""
    M = 24
    x, _, w, _ = inputs(M, K, F32, F32, 4)
    y, rstd = torch.empty((M, K), device="cuda"), torch.empty(M, device="cuda")
    cuda_lib.fp8_rmsnorm_fwd(x, w, y, rstd)
    bad = x.clone()
    bad[3] = 0
    bad[5, K // 2] = float("nan")
    bad[7, 1] = float("inf")
    bad[9] = 1e30
    code, amax = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
    cuda_lib.fp8_rmsnorm_fwd(bad, w, y2, rstd2)
    cuda_lib.fp8_rmsnorm_fwd(bad, w, code, rstd2, y_scale=torch.ones(1, device="cuda"), y_amax=amax)
    others = [m for m in range(M) if m not in (3, 5, 7, 9)]
    assert torch.equal(y2[others], y[others]) and torch.equal(rstd2[others], rstd[others])
    assert (y2[3] == 0).all() and abs(rstd2[3].item() - 1000.0) < 1e-3 and (code[3] == 0).all()
    assert torch.isnan(y2[5]).all() and torch.isnan(rstd2[5]) and (code[5] == 0x7F).all()
    assert rstd2[7].item() == 0 and torch.isnan(y2[7, 1]) and (y2[7, 2:] == 0).all() and code[7, 1].item() == 0x7F
    assert rstd2[9].item() == 0 and (y2[9] == 0).all()
    assert amax.item() == y2[torch.isfinite(y2)].abs().max().item()


def test_gradient_rows_are_apart(cuda_lib):
    M, K = 20, 512
    dy, t, w, _ = inputs(M, K, F32, F32, 5)
    rstd = (1 / torch.sqrt(t.square().mean(1) + 1e-6)).contiguous()
    dr, dr2 = torch.empty_like(t), torch.empty_like(t)
    cuda_lib.fp8_rmsnorm_bwd(dy, t, w, rstd, dr)
    dy[11, 3] = float("nan")
    cuda_lib.fp8_rmsnorm_bwd(dy, t, w, rstd, dr2)
    others = [m for m in range(M) if m != 11]
    assert torch.equal(dr2[others], dr[others]) and torch.isnan(dr2[11]).all()


def test_more_than_2_31_elements(cuda_lib):
    M, K = 140000, 16384
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    tail = torch.randn((3, K), device="cuda").to(BF)
    x[-3:] = tail
    w = torch.ones(K, device="cuda")
    y, rstd = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
    one = torch.ones(1, device="cuda")
    cuda_lib.fp8_rmsnorm_fwd(x, w, y, rstd, y_scale=one)
    y2, rstd2 = torch.empty((3, K), dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    cuda_lib.fp8_rmsnorm_fwd(tail, w, y2, rstd2, y_scale=one)
    assert torch.equal(y[-3:], y2) and torch.equal(rstd[-3:], rstd2)
    dr = torch.empty_like(x)
    cuda_lib.fp8_rmsnorm_bwd(x, x, w, rstd, dr)
    dr2 = torch.empty_like(tail)
    cuda_lib.fp8_rmsnorm_bwd(tail, tail, w, rstd2, dr2)
    assert torch.equal(dr[-3:], dr2) and cuda_lib.fp8mp_check() == 0


def test_another_stream_and_a_graph(cuda_lib):
    M, K = 33, 1040
    x, r, w, _ = inputs(M, K, BF, BF, 6)
    scale, amax = torch.full((1,), 16.0, device="cuda"), torch.zeros(1, device="cuda")
    make = lambda: (torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda"),  # noqa: E731
                    torch.empty_like(r))
    y, rstd, total = make()
    cuda_lib.fp8_rmsnorm_fwd(x, w, y, rstd, residual=r, total=total, y_scale=scale, y_amax=amax)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, rstd2, total2 = make()
    with torch.cuda.stream(side):
        cuda_lib.fp8_rmsnorm_fwd(x, w, y2, rstd2, residual=r, total=total2, y_scale=scale, y_amax=amax)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2) and torch.equal(total, total2)
    y3, rstd3, total3 = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.fp8_rmsnorm_fwd(x, w, y3, rstd3, residual=r, total=total3, y_scale=scale, y_amax=amax)
    x.mul_(-1)
    cuda_lib.fp8_rmsnorm_fwd(x, w, y, rstd, residual=r, total=total, y_scale=scale, y_amax=amax)
    graph.replay()
    assert torch.equal(y, y3) and torch.equal(rstd, rstd3) and torch.equal(total, total3)
    assert cuda_lib.fp8mp_check() == 0
