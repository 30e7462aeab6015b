"""The gated feed-forward block (fp8_gated_fwd, fp8_gated_dgrad,
fp8_gated_bwd) against the formulas in 64 bits.

Error bounds, by the repository's bound for an FP8 GEMM before rounding
(1e-5 sum |a b|, fp32 accumulation) and the fast exp and quotient (the
logistic p is good to (4 + 1.2 |z|) 2^-23 of itself, z its argument):

* g and u: D = 1e-5 sum |x w| s + 2^-22 |.|;
* h = act(g) u: (1.13 Dg |u| + |act(g)| Du) + |h| (4 + 1.2 |z|) 2^-23 + 2^-22 |h|
  (1.13 bounds both activations' slopes);
* dh: D as above; dg = dh u act'(g): D |u act'| + |dh u| E + 2^-22 |dg| with E
  the error of act' = p + g p (1 - p) z': the logistic's relative error times
  (p + 2 |g p z'|), plus 2^-22 of each term and |g p z'| for 1 - p.

What is rounded to bf16 or FP8 after that must lie between the roundings of
the two ends of its interval.
"""

import numpy as np
import pytest
import torch

from gpu_util import E4M3, E5M2

pytestmark = pytest.mark.gpu
F8 = {E4M3: (torch.float8_e4m3fn, 448.0), E5M2: (torch.float8_e5m2, 57344.0)}
ACTS = {"silu": 0, "gelu": 1}


@pytest.fixture(params=["pair", "single"])
def engine(request, monkeypatch):
    """Both tile engines (the library reads FP8MP_GEMM_ENGINE per call)."""
    monkeypatch.setenv("FP8MP_GEMM_ENGINE", request.param)
    return request.param


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(shape, std, scale, fmt, g):
    dt, top = F8[fmt]
    x = torch.randn(shape, generator=g, device="cuda") * std * scale
    return x.clamp(-top, top).to(dt).view(torch.uint8), torch.tensor([1.0 / scale], device="cuda")


def wide(c, fmt):
    return c.view(F8[fmt][0]).to(torch.float64)


def cast(x, fmt):
    dt, top = F8[fmt]
    return x.float().clamp(-top, top).to(dt).to(torch.float64)


def logistic(g, act):
    if act == "silu":
        return torch.special.expit(g), torch.ones_like(g), g
    c = 2 * (2 / np.pi) ** 0.5
    z = c * (g + 0.044715 * g ** 3)
    return torch.special.expit(z), c * (1 + 3 * 0.044715 * g * g), z


def between(got, lo, hi, what):
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def forward_reference(x8, w8, s, act):
    """(g, Dg, u, Du, h, Dh)."""
    x, w = wide(x8, E4M3), wide(w8, E4M3)
    F = w.shape[0] // 2
    pre, size = (x @ w.T) * s, (x.abs() @ w.abs().T) * s
    D = 1e-5 * size + 2.0 ** -22 * pre.abs()
    g, u, Dg, Du = pre[:, :F], pre[:, F:], D[:, :F], D[:, F:]
    p, _, z = logistic(g, act)
    h = g * p * u
    Dh = 1.13 * Dg * u.abs() + (g * p).abs() * Du + h.abs() * ((4 + 1.2 * z.abs()) * 2.0 ** -23 + 2.0 ** -22)
    return g, Dg, u, Du, h, Dh


def run_forward(fp8mp, M, F, K, act, fp8, save, seed=0, start_amax=0.0):
    g = gen(seed + M * 7 + F * 3 + K)
    x8, sx = codes((M, K), 1.0, 64.0, E4M3, g)
    w8, sw = codes((2 * F, K), 1.5 / K ** 0.5, 32.0 * K ** 0.5, E4M3, g)
    h = torch.full((M, F), 0x22, dtype=torch.uint8, device="cuda") if fp8 else torch.full(
        (M, F), 7.0, dtype=torch.bfloat16, device="cuda")
    scale = torch.tensor([60.0], device="cuda") if fp8 else None
    amax = torch.tensor([start_amax], device="cuda")
    gu = torch.full((M, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda") if save else None
    fp8mp.fp8_gated_fwd(x8, w8, sx, sw, h, act=ACTS[act], h_scale=scale, h_amax=amax, gu=gu)
    assert fp8mp.fp8mp_check() == 0
    return x8, w8, (sx * sw).double().item(), h, scale, amax, gu


def check_forward(fp8mp, M, F, K, act, fp8, save, seed=0):
    x8, w8, s, h, scale, amax, gu = run_forward(fp8mp, M, F, K, act, fp8, save, seed)
    g, Dg, u, Du, y, Dy = forward_reference(x8, w8, s, act)
    if fp8:
        k = scale.double().item()
        between(wide(h, E4M3), cast((y - Dy) * k, E4M3), cast((y + Dy) * k, E4M3), "h")
    else:
        between(h.double(), (y - Dy).bfloat16().double(), (y + Dy).bfloat16().double(), "h")
    top = y.abs().max().item()
    assert abs(amax.item() - top) <= Dy.max().item() + 2.0 ** -23 * top
    if save:
        between(gu[:, :F].double(), (g - Dg).bfloat16().double(), (g + Dg).bfloat16().double(), "g")
        between(gu[:, F:].double(), (u - Du).bfloat16().double(), (u + Du).bfloat16().double(), "u")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("M,F,K", [(128, 128, 128), (256, 256, 256), (1, 16, 16), (3, 48, 16), (33, 112, 80),
                                   (127, 144, 272), (129, 272, 144), (300, 1040, 528), (511, 400, 1296),
                                   (1000, 2064, 768)])
def test_forward(cuda_lib, engine, M, F, K, act, fp8):
    check_forward(cuda_lib, M, F, K, act, fp8, True)
    check_forward(cuda_lib, M, F, K, act, fp8, False, seed=1)


@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 66, 80])
@pytest.mark.parametrize("F,K", [(2064, 768), (496, 4096), (80, 4112), (5504, 144)])
def test_forward_few_tokens(cuda_lib, M, F, K):
    check_forward(cuda_lib, M, F, K, "silu", True, M % 2 == 0)
    check_forward(cuda_lib, M, F, K, "gelu", False, M % 3 == 0)


def test_forward_large(cuda_lib):
    check_forward(cuda_lib, 4096, 3600, 1040, "silu", True, True)


def test_amax_is_raised(cuda_lib):
    *_, amax, _ = run_forward(cuda_lib, 40, 64, 64, "silu", True, False, start_amax=1e6)
    assert amax.item() == 1e6


def test_empty_forward(cuda_lib):
    u8, bf = torch.uint8, torch.bfloat16
    z = lambda *s, dtype=u8: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    one, amax = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    cuda_lib.fp8_gated_fwd(z(0, 64), z(64, 64), one, one, z(0, 32), h_scale=one)
    cuda_lib.fp8_gated_fwd(z(5, 64), z(0, 64), one, one, z(5, 0), h_scale=one)
    for h in (torch.full((5, 32), 3, dtype=u8, device="cuda"), torch.full((5, 32), 3.0, dtype=bf, device="cuda")):
        gu = torch.full((5, 64), 3.0, dtype=bf, device="cuda")
        cuda_lib.fp8_gated_fwd(z(5, 0), z(64, 0), one, one, h, h_scale=one if h.dtype == u8 else None, h_amax=amax,
                               gu=gu)
        assert (h == 0).all() and (gu == 0).all() and amax.item() == 0


@pytest.mark.parametrize("M", [7, 200])
def test_a_nan_row_stays_in_its_row(cuda_lib, M):
    g = gen(5)
    x8, sx = codes((M, 96), 1.0, 64.0, E4M3, g)
    w8, sw = codes((2 * 80, 96), 0.1, 400.0, E4M3, g)
    clean = torch.empty((M, 80), dtype=torch.uint8, device="cuda")
    a, b = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    k = torch.tensor([30.0], device="cuda")
    cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, clean, h_scale=k, h_amax=a)
    x8[3, 10] = 0x7F
    h = torch.empty_like(clean)
    cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, h, h_scale=k, h_amax=b)
    keep = torch.arange(M, device="cuda") != 3
    assert (h[3] == 0x7F).all() and torch.equal(h[keep], clean[keep])
    assert torch.isfinite(b).all() and b <= a


def test_saturating_preactivations(cuda_lib):
    """|g| up to 1e5: exp over- and underflows and h is still act(g) u."""
    x8 = torch.full((4, 64), 0x7E, dtype=torch.uint8, device="cuda")  # 448
    w8 = torch.full((64, 64), 0x38, dtype=torch.uint8, device="cuda")  # 1
    w8[8:16] = 0xB8  # gate rows 8-15: -1
    one = torch.ones(1, device="cuda")
    for act, a in ACTS.items():
        h = torch.empty((4, 32), dtype=torch.bfloat16, device="cuda")
        cuda_lib.fp8_gated_fwd(x8, w8, one, one, h, act=a)
        v = 448.0 * 64
        want = torch.full((32,), v * v, dtype=torch.float64)
        want[8:16] = 0
        assert torch.equal(h.double().cpu(), want.bfloat16().double().expand(4, 32))


# -------------------------------------------------------- a few tokens' linear


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 4096, 14336), (2, 48, 80), (5, 144, 4112), (16, 128, 128),
                                   (17, 2064, 768), (33, 6000, 1552), (64, 400, 2064), (64, 16, 16), (63, 30000, 144)])
def test_linear_few(cuda_lib, M, N, K, bias, y_dtype):
    g = gen(M + N + K)
    x8, sx = codes((M, K), 1.0, 64.0, E4M3, g)
    w8, sw = codes((N, K), 1.0 / K ** 0.5, 32.0 * K ** 0.5, E4M3, g)
    b = torch.randn(N, generator=g, device="cuda").to(bias) if bias is not None else None
    y = torch.full((M, N), 5.0, dtype=y_dtype, device="cuda")
    amax = torch.zeros(1, device="cuda")
    cuda_lib.fp8_linear_few(x8, w8, sx, sw, y, bias=b, y_amax=amax)
    assert cuda_lib.fp8mp_check() == 0
    s = (sx * sw).double().item()
    ref, size = (wide(x8, E4M3) @ wide(w8, E4M3).T) * s, (wide(x8, E4M3).abs() @ wide(w8, E4M3).abs().T) * s
    if b is not None:
        ref, size = ref + b.double(), size + b.double().abs()
    D = 1e-5 * size + 2.0 ** -22 * ref.abs()
    between(y.double(), (ref - D).to(y_dtype).double(), (ref + D).to(y_dtype).double(), "y")
    assert amax.item() == y.abs().max().item()
    again = torch.empty_like(y)
    for _ in range(5):
        cuda_lib.fp8_linear_few(x8, w8, sx, sw, again, bias=b)
        assert torch.equal(y, again)


@pytest.mark.parametrize("M", [65, 66, 80, 96, 127, 128])
@pytest.mark.parametrize("N,K", [(16, 16), (4096, 5632), (2048, 5632), (272, 14336), (20016, 144), (6000, 1552)])
def test_linear_few_of_more_tokens(cuda_lib, M, N, K):
    test_linear_few(cuda_lib, M, N, K, torch.bfloat16, torch.bfloat16)


def test_linear_few_equals_the_linear_where_both_run(cuda_lib):
    """Whole numbers whose sums are exact in fp32: the split changes nothing."""
    g = gen(8)
    x8 = torch.randint(0, 2, (32, 4096), generator=g, device="cuda", dtype=torch.uint8) * 0x38  # 0 or 1
    w8 = torch.randint(0, 2, (272, 4096), generator=g, device="cuda", dtype=torch.uint8) * 0x38 + 0
    one = torch.ones(1, device="cuda")
    a, b = torch.empty((32, 272), device="cuda"), torch.empty((32, 272), device="cuda")
    cuda_lib.fp8_linear_fwd(x8, w8, one, one, a)
    cuda_lib.fp8_linear_few(x8, w8, one, one, b)
    assert torch.equal(a, b) and a.max() > 100


def test_linear_few_of_nothing(cuda_lib):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    one, b = torch.ones(1, device="cuda"), torch.arange(32, device="cuda", dtype=torch.float32)
    cuda_lib.fp8_linear_few(z(0, 64), z(32, 64), one, one, torch.empty((0, 32), device="cuda"))
    y = torch.full((3, 32), 7.0, device="cuda")
    cuda_lib.fp8_linear_few(z(3, 0), z(32, 0), one, one, y, bias=b)
    assert torch.equal(y, b.expand(3, 32))
    assert cuda_lib.fp8mp_check() == 0


# ---------------------------------------------------------------- backward


def gate_reference(dh, Ddh, gu, act):
    F = gu.shape[1] // 2
    g, u = gu[:, :F].double(), gu[:, F:].double()
    p, dz, z = logistic(g, act)
    a, da = g * p, p + g * p * (1 - p) * dz
    rel = (4 + 1.2 * z.abs()) * 2.0 ** -23
    gpz = (g * p * dz).abs()
    Eda = rel * (p + 2 * gpz) + 2.0 ** -22 * (p + gpz) + gpz * 2.0 ** -22
    dg, du = dh * u * da, dh * a
    Dg = Ddh * (u * da).abs() + (dh * u).abs() * Eda + 2.0 ** -22 * dg.abs()
    Du = Ddh * a.abs() + du.abs() * (rel + 2.0 ** -22)
    return torch.cat([dg, du], 1), torch.cat([Dg, Du], 1)


def check_codes(dgu8, amax, dgu, D, scale):
    between(wide(dgu8, E5M2), cast((dgu - D) * scale, E5M2), cast((dgu + D) * scale, E5M2), "dgu8")
    top = dgu.abs().max().item()
    assert abs(amax.item() - top) <= D.max().item() + 2.0 ** -23 * top


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fmt", [E5M2, E4M3])
@pytest.mark.parametrize("M,F,N", [(128, 256, 128), (256, 256, 256), (1, 16, 16), (5, 48, 80), (33, 64, 272),
                                   (127, 144, 272), (129, 320, 144), (300, 1040, 528), (1000, 2064, 768)])
def test_dgrad(cuda_lib, engine, M, F, N, act, fmt):
    g = gen(M + F + N)
    dy8, sy = codes((M, N), 1e-3, 2.0 ** 20 if fmt == E5M2 else 2.0 ** 16, fmt, g)
    wd8, sw = codes((N, F), 0.05, 1000.0, E4M3, g)
    gu = (torch.randn((M, 2 * F), generator=g, device="cuda") * 2).to(torch.bfloat16)
    scale, amax = torch.tensor([2.0 ** 18], device="cuda"), torch.zeros(1, device="cuda")
    dgu8 = torch.full((M, 2 * F), 0x22, dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_gated_dgrad(dy8, wd8, gu, sy, sw, scale, dgu8, act=ACTS[act], dgu_amax=amax, dy_fmt=fmt)
    assert cuda_lib.fp8mp_check() == 0
    s = (sy * sw).double().item()
    a, b = wide(dy8, fmt), wide(wd8, E4M3)
    dh, size = (a @ b) * s, (a.abs() @ b.abs()) * s
    dgu, D = gate_reference(dh, 1e-5 * size + 2.0 ** -22 * dh.abs(), gu, act)
    check_codes(dgu8, amax, dgu, D, scale.item())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,F,K", [(1, 16, 16), (5, 48, 80), (17, 2064, 48), (127, 144, 272), (300, 1040, 528),
                                   (1237, 272, 1040)])
def test_backward(cuda_lib, engine, M, F, K, act, dtype):
    g = gen(M + F + K)
    x8, sx = codes((M, K), 1.0, 64.0, E4M3, g)
    w8, sw = codes((2 * F, K), 0.05, 1000.0, E4M3, g)
    gu = (torch.randn((M, 2 * F), generator=g, device="cuda") * 2).to(torch.bfloat16)
    dh = (torch.randn((M, F), generator=g, device="cuda") * 1e-3).to(dtype)
    scale, sinv = torch.tensor([2.0 ** 20], device="cuda"), torch.tensor([2.0 ** -20], device="cuda")
    amax, flag = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dgu8 = torch.full((M, 2 * F), 0x22, dtype=torch.uint8, device="cuda")
    dx = torch.full((M, K), 5.0, dtype=dtype, device="cuda")
    dw = torch.full((2 * F, K), 5.0, dtype=dtype, device="cuda")
    cuda_lib.fp8_gated_bwd(dh, gu, x8, w8, sx, sw, scale, sinv, dgu8, dx, dw, act=ACTS[act], dgu_amax=amax,
                           dw_nonfinite=flag)
    assert cuda_lib.fp8mp_check() == 0
    dgu, D = gate_reference(dh.double(), torch.zeros_like(dh, dtype=torch.float64), gu, act)
    check_codes(dgu8, amax, dgu, D, scale.item())
    d, x, w = wide(dgu8, E5M2), wide(x8, E4M3), wide(w8, E4M3)
    for got, a, b, s in ((dx, d, w, (sinv * sw)), (dw, d.T, x, (sinv * sx))):
        s = s.double().item()
        ref, size = (a @ b) * s, (a.abs() @ b.abs()) * s
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all()
    assert flag.item() == 0
    # the GEMMs alone, from codes that are there, and each gradient alone
    for want in ("both", "dx", "dw"):
        dx2 = torch.empty_like(dx) if want != "dw" else None
        dw2 = torch.empty_like(dw) if want != "dx" else None
        cuda_lib.fp8_gated_bwd(None, None, x8, w8, sx, sw, None, sinv, dgu8, dx2, dw2)
        assert dx2 is None or torch.equal(dx2, dx)
        assert dw2 is None or torch.equal(dw2, dw)


@pytest.mark.parametrize("M,F,K", [(1237, 2736, 1040), (300, 8192, 528), (16, 4096, 16), (2000, 5504, 256)])
def test_backward_of_few_long_tiles(cuda_lib, engine, M, F, K):
    """dX has few tiles with contractions of 2F, dW many of M: each tile of dX has
    SMs of its own, and each output equals its own launch's (in test_backward)."""
    test_backward(cuda_lib, engine, M, F, K, "silu", torch.bfloat16)


def test_backward_of_nothing(cuda_lib):
    u8, bf, one = torch.uint8, torch.bfloat16, torch.ones(1, device="cuda")
    e = lambda *s, dtype=u8: torch.ones(s, dtype=dtype, device="cuda")  # noqa: E731
    dw = e(64, 48, dtype=torch.float32)
    cuda_lib.fp8_gated_bwd(e(0, 32, dtype=bf), e(0, 64, dtype=bf), e(0, 48), e(64, 48), one, one, one, one, e(0, 64),
                           e(0, 48, dtype=bf), dw)
    assert (dw == 0).all()
    dgu8 = e(5, 64)
    cuda_lib.fp8_gated_dgrad(e(5, 0), e(0, 32), e(5, 64, dtype=bf), one, one, one, dgu8)
    assert (dgu8 == 0).all()
    cuda_lib.fp8_gated_dgrad(e(0, 16), e(16, 32), e(0, 64, dtype=bf), one, one, one, e(0, 64))
    assert cuda_lib.fp8mp_check() == 0


def test_backward_flags_a_nonfinite_weight_gradient(cuda_lib):
    g = gen(3)
    x8, sx = codes((40, 64), 1.0, 64.0, E4M3, g)
    w8, sw = codes((96, 64), 0.1, 400.0, E4M3, g)
    gu = torch.randn((40, 96), generator=g, device="cuda").to(torch.bfloat16)
    dh = torch.randn((40, 48), generator=g, device="cuda")
    dh[39, 47] = float("nan")
    one, flag, amax = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(
        1, device="cuda")
    dw, dgu8 = torch.empty((96, 64), device="cuda"), torch.empty((40, 96), dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_gated_bwd(dh, gu, x8, w8, sx, sw, one, one, dgu8, None, dw, dgu_amax=amax, dw_nonfinite=flag)
    assert flag.item() == 1 and torch.isfinite(amax).all()
    assert (dgu8[39, 47] == 0x7F) and (dgu8[39, 95] == 0x7F)
    nan = torch.isnan(dw)
    assert nan[47].all() and nan[95].all() and nan.sum() == 2 * 64


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_of_saturated_gates(cuda_lib, act, dtype):
    """|g| up to bf16's largest: act' is 1 or 0 there, and g^2 has no place in
    fp32. Everything is a power of two or saturates: no tolerance."""
    g = torch.tensor([2.0 ** e for e in (14, 30, 60, 63, 64, 70, 100, 127)], device="cuda")
    gu = torch.cat([g, -g, torch.full((16,), 0.5, device="cuda")]).to(torch.bfloat16).expand(5, 32).contiguous()
    dh = torch.full((5, 16), 2.0 ** -6, dtype=dtype, device="cuda")
    one = torch.ones(1, device="cuda")
    dgu8, amax = torch.empty((5, 32), dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    x8, w8 = (torch.zeros((n, 16), dtype=torch.uint8, device="cuda") for n in (5, 32))
    cuda_lib.fp8_gated_bwd(dh, gu, x8, w8, one, one, one, one, dgu8, None, None, act=ACTS[act], dgu_amax=amax)
    want = torch.zeros((5, 32), dtype=torch.float64, device="cuda")
    want[:, :8] = 2.0 ** -7
    want[:, 16:24] = (g.double() * 2.0 ** -6).clamp(max=57344.0)
    assert torch.equal(wide(dgu8, E5M2), want) and amax.item() == 2.0 ** 121


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(cuda_lib, act):
    """dg, du are the derivatives of the h that the forward pass returns, by
    central differences in 64 bits of the forward formula, at the gradient
    dh = 1: codes under a scale of 2^8, so to half a step of E5M2."""
    F, M = 64, 32
    gu = (torch.linspace(-9, 9, M * 2 * F, device="cuda")[torch.randperm(M * 2 * F, device="cuda", generator=gen(1))]
          ).reshape(M, 2 * F).to(torch.bfloat16)
    g, u = gu[:, :F].double(), gu[:, F:].double()
    f = lambda g, u: g * logistic(g, act)[0] * u  # noqa: E731
    step = 1e-5
    dg, du = (f(g + step, u) - f(g - step, u)) / (2 * step), (f(g, u + step) - f(g, u - step)) / (2 * step)
    one, scale = torch.ones(1, device="cuda"), torch.tensor([256.0], device="cuda")
    dgu8 = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda")
    x8, w8 = torch.zeros((M, 16), dtype=torch.uint8, device="cuda"), torch.zeros((2 * F, 16), dtype=torch.uint8,
                                                                                 device="cuda")
    cuda_lib.fp8_gated_bwd(torch.ones((M, F), device="cuda"), gu, x8, w8, one, one, scale, one, dgu8, None, None,
                           act=ACTS[act])
    got, want = wide(dgu8, E5M2) / 256, torch.cat([dg, du], 1)
    assert ((got - want).abs() <= want.abs() / 8 + 2.0 ** -17 / 256 + 1e-6).all()


# ------------------------------------------------------------------- other


def test_repeats_are_bitwise_equal(cuda_lib, engine):
    M, F, K = 700, 656, 528
    first = None
    for _ in range(20):
        *_, h, _, amax, gu = run_forward(cuda_lib, M, F, K, "silu", True, True)
        now = [h.clone(), amax.clone(), gu.clone()]
        g = gen(9)
        dy8, sy = codes((M, K), 1e-3, 2.0 ** 20, E5M2, g)
        wd8, sw = codes((K, F), 0.05, 1000.0, E4M3, g)
        dgu8 = torch.empty((M, 2 * F), dtype=torch.uint8, device="cuda")
        cuda_lib.fp8_gated_dgrad(dy8, wd8, gu, sy, sw, torch.tensor([2.0 ** 18], device="cuda"), dgu8)
        now.append(dgu8)
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_another_stream_and_a_graph(cuda_lib):
    g = gen(2)
    x8, sx = codes((200, 256), 1.0, 64.0, E4M3, g)
    w8, sw = codes((512, 256), 0.1, 400.0, E4M3, g)
    k = torch.tensor([30.0], device="cuda")
    out = [torch.zeros((200, 256), dtype=torch.uint8, device="cuda") for _ in range(3)]
    cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, out[0], h_scale=k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, out[1], h_scale=k)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, out[2], h_scale=k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


class Odd:
    """Arrays that start 16 bytes past a 32-byte boundary, with bytes around them
    that no call may write."""

    def __init__(self):
        self.rooms = []

    def empty(self, shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        room = torch.full((n + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
        at = 256 + (16 - (room.data_ptr() + 256)) % 32
        self.rooms.append((room, at, n))
        return room[at:at + n].view(dtype).view(shape)

    def of(self, x):
        y = self.empty(x.shape, x.dtype)
        y.copy_(x)
        return y

    def check(self):
        for room, at, n in self.rooms:
            assert room[at:at + n].data_ptr() % 32 == 16
            assert (room[:at] == 0x5A).all() and (room[at + n:] == 0x5A).all()


@pytest.mark.parametrize("M,F,K", [(1, 32, 16), (33, 272, 144), (64, 1024, 256), (127, 528, 80), (300, 2064, 272)])
def test_16_byte_alignment_and_nothing_past_the_ends(cuda_lib, engine, M, F, K):
    """Bit for bit what the same calls give on aligned arrays."""
    g = gen(M + F)
    u8, bf = torch.uint8, torch.bfloat16
    x8, sx = codes((M, K), 1.0, 64.0, E4M3, g)
    w8, sw = codes((2 * F, K), 0.2, 400.0, E4M3, g)
    dy8, sy = codes((M, K), 1e-3, 2.0 ** 20, E5M2, g)
    wd8, sd = codes((K, F), 0.05, 1000.0, E4M3, g)
    dh = torch.randn((M, F), generator=g, device="cuda").to(bf)
    bias = torch.randn((F,), generator=g, device="cuda")
    k = torch.tensor([30.0], device="cuda")
    odd = Odd()
    results = []
    for place, empty in ((lambda x: x, lambda s, d: torch.empty(s, dtype=d, device="cuda")), (odd.of, odd.empty)):
        x, w, dy, wd, d, b = (place(z) for z in (x8, w8, dy8, wd8, dh, bias))
        h, hb, gu = empty((M, F), u8), empty((M, F), bf), empty((M, 2 * F), bf)
        cuda_lib.fp8_gated_fwd(x, w, sx, sw, h, h_scale=k, gu=gu)
        cuda_lib.fp8_gated_fwd(x, w, sx, sw, hb, act=1)
        g1, g2 = empty((M, 2 * F), u8), empty((M, 2 * F), u8)
        cuda_lib.fp8_gated_dgrad(dy, wd, gu, sy, sd, k, g1)
        dx, dw = empty((M, K), bf), empty((2 * F, K), torch.float32)
        cuda_lib.fp8_gated_bwd(d, gu, x, w, sx, sw, k, sx, g2, dx, dw)
        got = [h, hb, gu, g1, g2, dx, dw]
        if M <= 128:
            for dtype in (bf, torch.float32):
                got.append(empty((M, F), dtype))
                cuda_lib.fp8_linear_few(x, w[:F], sx, sw, got[-1], bias=b)
        results.append(got)
    for a, b in zip(*results):
        assert torch.equal(a.view(u8), b.view(u8))
    odd.check()
    assert cuda_lib.fp8mp_check() == 0


@pytest.mark.slow
def test_offsets_past_32_bits(cuda_lib):
    """gu of 4.4e9 elements (8.8 GB), h of 2.2e9: the last rows are right."""
    M, F, K = 153000, 14336, 16
    g = gen(4)
    x8, sx = codes((M, K), 1.0, 64.0, E4M3, g)
    w8, sw = codes((2 * F, K), 0.4, 128.0, E4M3, g)
    k, amax = torch.tensor([30.0], device="cuda"), torch.zeros(1, device="cuda")
    h = torch.zeros((M, F), dtype=torch.uint8, device="cuda")
    gu = torch.zeros((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp8_gated_fwd(x8, w8, sx, sw, h, h_scale=k, h_amax=amax, gu=gu)
    tail = slice(M - 70, M)
    gg, Dg, u, Du, y, Dy = forward_reference(x8[tail].contiguous(), w8, (sx * sw).double().item(), "silu")
    between(wide(h[tail], E4M3), cast((y - Dy) * 30, E4M3), cast((y + Dy) * 30, E4M3), "h")
    between(gu[tail, F:].double(), (u - Du).bfloat16().double(), (u + Du).bfloat16().double(), "u")
    dh = torch.randn((70, F), generator=g, device="cuda").to(torch.bfloat16)
    big = torch.zeros((M, F), dtype=torch.bfloat16, device="cuda")
    big[tail] = dh
    scale, one = torch.tensor([256.0], device="cuda"), torch.ones(1, device="cuda")
    dgu8 = torch.zeros((M, 2 * F), dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_gated_bwd(big, gu, x8, w8, sx, sw, scale, one, dgu8, None, None, dgu_amax=amax)
    dgu, D = gate_reference(dh.double(), torch.zeros_like(dh, dtype=torch.float64), gu[tail], "silu")
    between(wide(dgu8[tail].contiguous(), E5M2), cast((dgu - D) * 256, E5M2), cast((dgu + D) * 256, E5M2), "dgu8")
    assert (dgu8[:1000] & 0x7F == 0).all()
    N = 16
    dy8, sy = codes((M, N), 1.0, 64.0, E5M2, g)
    wd8, sd = codes((N, F), 0.4, 128.0, E4M3, g)
    cuda_lib.fp8_gated_dgrad(dy8, wd8, gu, sy, sd, scale, dgu8, dgu_amax=amax)
    a, b, s = wide(dy8[tail].contiguous(), E5M2), wide(wd8, E4M3), (sy * sd).double().item()
    dh, size = (a @ b) * s, (a.abs() @ b.abs()) * s
    dgu, D = gate_reference(dh, 1e-5 * size + 2.0 ** -22 * dh.abs(), gu[tail], "silu")
    between(wide(dgu8[tail].contiguous(), E5M2), cast((dgu - D) * 256, E5M2), cast((dgu + D) * 256, E5M2), "dgu8")
    assert cuda_lib.fp8mp_check() == 0
