"""mp_logprobs_fwd and mp_logprobs_bwd against the formulas in 64 bits.

Tolerances. u = 2^-24, z = (x - m) log2(e). exp2's hardware approximation is good
to 4 u of the result, its argument to 2 u |z|, so a term of S is off by
(2 |z| ln 2 + 4) u of itself. Of a long row a thread
adds V / 1024 terms to each of four running sums (of a short one, of at most 16384
elements, V / 128: 128), whose rescaling (one product, as an exponential, at every larger
maximum) and 9 joins add (V / 1024 + 60) u at most (of a short one V / 128 + 60). log S adds two
roundings of |log S|, the subtractions those of their results. What is sum_v p_v |z_v| or
p_v z_v^2 there is taken from the 64-bit p."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LN2 = math.log(2.0)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def logits(M, V, dtype, seed=0, ld=None, masked=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed + M * 31 + V)
    x = torch.randn((M, ld or V), generator=g, device="cuda") * 3
    if masked:
        x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < masked, -INF)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    x[torch.arange(M), t] = torch.randn(M, generator=g, device="cuda") + 5
    t[torch.rand(M, generator=g, device="cuda") < 0.2] = -100
    return x.to(dtype), t


def forward(lib, x, t, k=0, entropy=True, vocab=None):
    M = x.shape[0]
    logprob, stats = torch.full((M,), 7.0, device="cuda"), torch.full((M, 2), 7.0, device="cuda")
    H = torch.full((M,), 7.0, device="cuda") if entropy else None
    top = torch.full((M, k), 7.0, device="cuda") if k else None
    ids = torch.full((M, k), -7, dtype=torch.int64, device="cuda") if k else None
    lib.mp_logprobs_fwd(x, t, logprob, stats, entropy=H, top_logprob=top, top_id=ids, vocab=vocab)
    assert lib.fp8mp_check() == 0
    return logprob, stats, H, top, ids


def reference(x):
    """log p, and the rounding (in u) that log S, and that the entropy, may have."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    d = x - m
    log_s = torch.log(torch.exp(d).sum(1, keepdim=True))
    logp = d - log_s
    p = torch.exp(logp)
    z = torch.where(p > 0, d, 0.0).abs() / LN2
    V = x.shape[1]
    adds = V / (128 if V <= 16384 else 1024) + 60
    of_s = (p * (2 * LN2 * z + 4)).sum(1) + adds + 4 * log_s[:, 0]
    of_h = of_s + LN2 * (p * z * (2 * LN2 * z + 8)).sum(1) + LN2 * (adds + 4) * (p * z).sum(1)
    return logp, d, log_s[:, 0], of_s, of_h


def ranked(x, k):
    """Largest first, of equal ones the lower index."""
    return torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :k]


SIZES = [(1, 1), (3, 2), (2, 7), (5, 50), (9, 1000), (4, 4097), (1, 50001), (333, 5003), (7, 128000), (40, 128000), (150, 33333),
         (5000, 515), (6000, 8001), (5001, 16385)]


@pytest.mark.parametrize("M,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("masked", [0.0, 0.7])
def test_forward(cuda_lib, M, V, dtype, masked):
    x, t = logits(M, V, dtype, masked=masked)
    k = min(V, 20)
    logp, d, log_s, of_s, of_h = reference(x)
    given = t >= 0
    at = logp.gather(1, t.clamp_min(0)[:, None])[:, 0]
    room = (of_s + 2 * d.gather(1, t.clamp_min(0)[:, None])[:, 0].abs() + 2) * U
    want = -(torch.exp(logp) * torch.where(logp > -INF, logp, 0.0)).sum(1)
    # with everything, with the entropy, with neither: short rows go another way without the top
    for kk, entropy in ((k, True), (0, True), (0, False)):
        logprob, stats, H, top, ids = forward(cuda_lib, x, t, kk, entropy)
        assert (logprob[~given] == 0).all()
        assert ((logprob.double() - at).abs() <= room)[given].all()
        assert torch.equal(stats[:, 0], x.float().amax(1))
        assert ((stats[:, 1].double() - log_s).abs() <= of_s * U).all()
        if entropy:
            assert ((H.double() - want).abs() <= of_h * U).all()
        if kk:
            best = ranked(x, k)
            assert torch.equal(ids, best)
            wanted, far = logp.gather(1, best), d.gather(1, best)
            assert torch.equal(torch.isinf(top), torch.isinf(wanted))
            fine = torch.isfinite(wanted)
            assert ((top.double() - wanted).abs() <= (of_s[:, None] + 2 * far.abs() + 2) * U)[fine].all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 2, 32])
def test_ties_go_to_the_lowest_index(cuda_lib, dtype, k):
    """Equal logits throughout, few values, few tokens allowed, a rising and a falling
    row, large ones in one thread's columns alone, both zeros."""
    V = 20011
    i = torch.arange(V, device="cuda", dtype=F32)
    rows = [torch.zeros(V, device="cuda"), (i % 3), torch.full((V,), -INF, device="cuda"), i / 64, -i / 64,
            torch.where((i // 8) % 512 == 5, 100 + i / 1000, i * 0), torch.where(i % 2 == 0, -0.0, 0.0),
            torch.where(i == V - 1, 1.0, 0.0), torch.where(i < 4, 1.0, 0.0), torch.full((V,), -3.3e38, device="cuda"),
            torch.where((i // 4) % 512 == 7, i, -i), torch.where((i > 9000) & (i < 12000), 5.0, -2.0)]
    x = torch.stack(rows)
    x[2, [17, 4000, 19999]] = torch.tensor([1.0, 2.0, 2.0], device="cuda")
    for part in (x.to(dtype), x.to(dtype)[:, :V // 16 * 16].contiguous()):
        for M in (len(rows), 400):  # (rows shared by several CTAs, and not)
            y = part.repeat((M + len(rows) - 1) // len(rows), 1)[:M].contiguous()
            *_, top, ids = forward(cuda_lib, y, torch.zeros(M, dtype=torch.int64, device="cuda"), k)
            assert torch.equal(ids, ranked(y, k))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [12, 48, 200, 400])
@pytest.mark.parametrize("offset", [0, 1])
def test_long_rows_over_any_number_of_ctas(cuda_lib, dtype, M, offset):
    """The selection of rows that 8, 4, 2 and 1 CTAs share: ties across them, all that is
    allowed in one's part, infinities and NaN there; off the 16-byte boundaries too."""
    V, k = 100003, 32
    i = torch.arange(V, device="cuda", dtype=F32)
    g = torch.Generator(device="cuda").manual_seed(21)
    rows = torch.stack([torch.zeros(V, device="cuda"), i % 7, torch.where(i == V - 1, 1.0, -INF), torch.where(i == 0, 1.0, -INF),
                        torch.where((i > 60000) & (i < 60040), i, -INF), torch.where(i % 12501 == 0, 3.0, -3e38),
                        -(i - 50000).abs() / 4096, torch.randn(V, generator=g, device="cuda"),
                        torch.where(i > V - 20, 2.0, 1.0), torch.where(i < 20, 2.0, 1.0),
                        torch.where(i % 2 == 0, -INF, -3e38), torch.randn(V, generator=g, device="cuda")])
    x = rows.repeat((M + 11) // 12, 1)[:M].to(dtype)
    room = torch.empty(M * V + offset, dtype=dtype, device="cuda")
    y = room[offset:].view(M, V).copy_(x)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    logprob, stats, H, top, ids = forward(cuda_lib, y, t, k)
    assert torch.equal(ids, ranked(x, k))
    logp, d, log_s, of_s, of_h = reference(x[:12])
    assert torch.equal(stats[:, 0], x.float().amax(1))
    want = -(torch.exp(logp) * torch.where(logp > -INF, logp, 0.0)).sum(1)
    assert ((stats[:12, 1].double() - log_s).abs() <= of_s * U).all() and ((H[:12].double() - want).abs() <= of_h * U).all()
    at, far = logp.gather(1, t[:12, None])[:, 0], d.gather(1, t[:12, None])[:, 0]
    fine = torch.isfinite(at)
    assert torch.equal(torch.isinf(logprob[:12]), ~fine)
    assert ((logprob[:12].double() - at).abs() <= (of_s + 2 * far.abs() + 2) * U)[fine].all()
    y[:, 99999] = float("nan")
    *_, top, ids = forward(cuda_lib, y, t, 2)
    x[:, 99999] = -INF
    best = ranked(x, 2)
    several = torch.isfinite(x.float()).sum(1) >= 2
    assert torch.isnan(top).all() and torch.equal(ids[several], best[several])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [11, 500])
def test_rows_of_infinities_nan_and_lowest_values(cuda_lib, dtype, M):
    V = 9001
    x, t = logits(M, V, dtype, seed=1)
    t.clamp_min_(0)
    low = torch.finfo(dtype).min
    good = forward(cuda_lib, x, t, 3)
    x[1] = -INF                     # nothing is allowed
    x[2] = low                      # nothing is allowed, by the type's lowest value
    x[3, 5000] = float("nan")
    x[4, 77] = INF
    x[5] = low
    x[5, t[5]] = 1.0                # one token is
    x[6] = -INF
    x[6, 8000] = 2.0
    x[7] = float("nan")
    x[8, :] = 3e38
    logprob, stats, H, top, ids = forward(cuda_lib, x, t, 3)
    others = [m for m in range(M) if m not in range(1, 9)]
    for a, b in zip((logprob, stats, H, top, ids), good):
        assert torch.equal(a[others], b[others])
    assert logprob[1].item() == -INF and H[1].item() == 0 and (stats[1] == -INF).all()
    assert (top[1] == -INF).all() and ids[1].tolist() == [0, 1, 2]
    for m in (2, 8):
        assert abs(logprob[m].item() + math.log(V)) < 1e-5 and abs(H[m].item() - math.log(V)) < 1e-5
        assert ids[m].tolist() == [0, 1, 2]
    for m in (3, 4, 7):
        assert torch.isnan(logprob[m]) and torch.isnan(H[m]) and torch.isnan(top[m]).all()
    assert ids[4, 0].item() == 77 and 5000 not in ids[3].tolist() and ids[7].tolist() == [0, 1, 2]
    assert logprob[5].item() == 0 and H[5].item() == 0 and ids[5, 0].item() == t[5].item()
    assert ids[6].tolist() == [8000, 0, 1] and top[6].tolist() == [0.0, -INF, -INF] and H[6].item() == 0
    # and their gradients
    a, b = torch.ones(M, device="cuda"), torch.ones(M, device="cuda")
    dx = torch.empty_like(x)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, dx, entropy=H, dentropy=b)
    assert cuda_lib.fp8mp_check() == 0
    assert (dx[1] == 0).all()
    uniform = -torch.full((V,), 1 / V, device="cuda", dtype=torch.float64)
    uniform[t[2]] += 1
    assert (dx[2].double() - uniform).abs().max().item() <= HALF[dtype] + 1e-6
    for m in (3, 4, 7):
        assert torch.isnan(dx[m]).all()
    assert dx[5].abs().max().item() <= 1e-6
    assert torch.isfinite(dx[others]).all()


BACK = [(1, 1), (3, 7), (5, 50), (9, 1008), (4, 4097), (2, 50001), (333, 5008), (7, 128000), (1300, 2064), (2001, 2047)]
MANY = [(4900, 2064), (4900, 4096), (4863, 4096), (4900, 1031)]  # a warp for each row, or a block


@pytest.mark.parametrize("M,V", BACK + MANY)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("codes", [False, True])
def test_backward(cuda_lib, M, V, dtype, entropy, codes):
    ld = (V + 15) // 16 * 16 if codes else V
    x, t = logits(M, V, dtype, seed=2, ld=ld, masked=0.3)
    x[:, V:] = float("nan")  # the padding is not looked at
    _, stats, H, *_ = forward(cuda_lib, x, t, vocab=V)
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randn(M, generator=g, device="cuda") * 100
    b = torch.randn(M, generator=g, device="cuda") * 10 if entropy else None
    a[:1], amax = 0.0, torch.zeros(1, device="cuda")
    scale = torch.tensor([256.0], device="cuda") if codes else None
    flat = torch.full((M * ld + 256,), 77, dtype=torch.uint8 if codes else dtype, device="cuda")
    dx = flat[128:128 + M * ld].view(M, ld)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, dx, entropy=H if entropy else None, dentropy=b, scale=scale, amax=amax,
                             vocab=V)
    assert cuda_lib.fp8mp_check() == 0
    assert (flat[:128] == 77).all() and (flat[128 + M * ld:] == 77).all()
    assert (dx[:, V:] == 0).all()
    logp = x[:, :V].double() - stats[:, :1].double() - stats[:, 1:].double()
    p, given = torch.exp(logp), t >= 0
    z = torch.where(p > 0, logp, 0.0).abs() / LN2
    aa = torch.where(given, a, 0.0).double()[:, None]
    tilt = torch.where(p > 0, logp, 0.0) + H.double()[:, None]
    bb = b.double()[:, None] if entropy else 0.0
    want = -p * (aa + bb * tilt)
    one = torch.zeros_like(want).scatter_(1, t.clamp_min(0)[:, None], aa)
    want = want + one
    slack = p * (aa.abs() + (bb.abs() * (z + H.double()[:, None] + 4) if entropy else 0.0)) * (2 * z + 16) * U
    slack = slack + 2 * U * one.abs() + 1e-37
    if codes:
        got, s = dx.view(torch.float8_e5m2).double()[:, :V], (want * 256.0).clamp(-57344, 57344)
        ok = (got - s).abs() <= 2.0 ** -3 * (s.abs() + 256 * slack) + 256 * slack + 2.0 ** -17
    else:
        ok = (dx[:, :V].double() - want).abs() <= HALF[dtype] * (want.abs() + slack) + slack
    assert ok.all(), (int((~ok).sum()), want[~ok][:4])
    most = want.abs().max().item()
    assert abs(amax.item() - most) <= slack.max().item() + 2 * U * most


def test_gradient_is_the_differences(cuda_lib):
    M, V = 4, 300
    x, t = logits(M, V, F32, seed=3)
    t.clamp_min_(0)
    g = torch.Generator(device="cuda").manual_seed(6)
    a, b = (torch.randn(M, generator=g, device="cuda") for _ in range(2))
    d = torch.randn((M, V), generator=g, device="cuda").double()
    _, stats, H, *_ = forward(cuda_lib, x, t)
    dx = torch.empty_like(x)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, dx, entropy=H, dentropy=b)

    def f(y):
        logp = y - torch.logsumexp(y, 1, keepdim=True)
        at = logp.gather(1, t[:, None])[:, 0]
        return (a.double() * at - b.double() * (torch.exp(logp) * logp).sum(1)).sum().item()

    h = 1e-5
    by = (f(x.double() + h * d) - f(x.double() - h * d)) / (2 * h)
    along = dx.double() * d
    assert abs(by - along.sum().item()) <= 1e-5 * along.abs().sum().item()


@pytest.mark.parametrize("dtype,V", [(BF, 5001), (F32, 2048)])
def test_the_gradient_in_place_of_the_logits(cuda_lib, dtype, V):
    M = 21
    x, t = logits(M, V, dtype, seed=4)
    _, stats, *_ = forward(cuda_lib, x, t)
    a = torch.randn(M, device="cuda")
    dx = torch.empty_like(x)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, dx)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, x)
    assert torch.equal(x, dx)


def test_rows_without_a_gradient_are_zero(cuda_lib):
    x, t = logits(6, 1000, BF, seed=5)
    t[:] = torch.tensor([3, -1, 1000, 2 ** 40, -2 ** 62, 999], device="cuda")
    logprob, stats, *_ = forward(cuda_lib, x, t)
    assert (logprob[1:5] == 0).all() and (logprob[[0, 5]] != 0).all()
    x[1] = float("nan")
    a = torch.ones(6, device="cuda")
    a[5] = 0
    dx = torch.full_like(x, 7)
    cuda_lib.mp_logprobs_bwd(x, t, stats, a, dx)
    assert (dx[1:] == 0).all() and (dx[0] != 0).any()


def test_odd_addresses(cuda_lib):
    """Logits that start between 16-byte boundaries."""
    V, M = 777, 5
    for dtype in (BF, F32):
        flat, t = logits(1, V * M + 9, dtype, seed=6)
        t = torch.arange(M, device="cuda")
        for off in range(9):
            x = flat[0, off:off + V * M].view(M, V)
            got, whole = forward(cuda_lib, x, t, 4), forward(cuda_lib, x.clone(), t, 4)
            for p, q in zip(got, whole):  # (another dealing of the columns to threads: other roundings)
                assert torch.allclose(p.double(), q.double(), rtol=1e-5, atol=1e-5)
            assert torch.equal(got[4], whole[4])
            out = torch.full_like(flat, 7)
            dx = out[0, off:off + V * M].view(M, V)
            ref = torch.empty((M, V), dtype=dtype, device="cuda")
            cuda_lib.mp_logprobs_bwd(x, t, got[1], torch.ones(M, device="cuda"), dx)
            cuda_lib.mp_logprobs_bwd(x.clone(), t, got[1], torch.ones(M, device="cuda"), ref)
            assert torch.equal(dx, ref) and (out[0, :off] == 7).all() and (out[0, off + V * M:] == 7).all()


def test_more_than_2_31_logits(cuda_lib):
    M, V = 17000, 128000
    x = torch.zeros((M, V), dtype=BF, device="cuda")
    tail, t = logits(2, V, BF, seed=7)
    x[-2:] = tail
    ts = torch.zeros(M, dtype=torch.int64, device="cuda")
    ts[-2:] = t
    logprob, stats, H, top, ids = forward(cuda_lib, x, ts, 2)
    want = forward(cuda_lib, tail, t, 2)
    assert torch.equal(ids[-2:], want[4]) and torch.allclose(logprob[-2:], want[0], rtol=1e-5, atol=1e-6)
    out = torch.empty((M, V), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    cuda_lib.mp_logprobs_bwd(x, ts, stats, torch.ones(M, device="cuda"), out, scale=one)
    small = torch.empty((2, V), dtype=torch.uint8, device="cuda")
    cuda_lib.mp_logprobs_bwd(tail, t, stats[-2:].contiguous(), torch.ones(2, device="cuda"), small, scale=one)
    assert torch.equal(out[-2:], small) and cuda_lib.fp8mp_check() == 0


def test_another_stream_and_a_graph(cuda_lib):
    x, t = logits(5, 30001, BF, seed=8)
    want = forward(cuda_lib, x, t, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = forward(cuda_lib, x, t, 8)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    bufs = [torch.empty_like(v) for v in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.mp_logprobs_fwd(x, t, bufs[0], bufs[1], entropy=bufs[2], top_logprob=bufs[3], top_id=bufs[4])
    x.copy_(x.flip(1))
    want = forward(cuda_lib, x, t, 8)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(want, bufs))
