"""mp_embedding_fwd bit for bit, mp_embedding_bwd against the formula in 64 bits.

Tolerance of the gradient: a row's c gradients are added in fp32, c - 1 additions
and at most as many joins of partial sums, each off by 2^-24 of a partial sum, which
is at most the sum of the absolute values; the scaling and the output's rounding add
2^-24 and half a step of the type."""

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def some_ids(M, V, seed, spread=1.0):
    """Ids of uneven frequency, some outside of the table."""
    g = rng(seed)
    r = torch.rand(M, generator=g, device="cuda", dtype=torch.float64) ** spread
    ids = (r * V).long().clamp_max(V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[ids]
    out = torch.rand(M, generator=g, device="cuda")
    ids[out < 0.05] = -1
    ids[out > 0.98] = V
    ids[(out > 0.97) & (out <= 0.98)] = 2 ** 40 + 3
    return ids


@pytest.mark.parametrize("M,V,K", [(1, 1, 16), (7, 5, 16), (33, 1000, 272), (1000, 77, 1040), (5000, 30000, 4096)])
@pytest.mark.parametrize("table,out", [("e4m3", BF), ("e4m3", F32), (BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_forward(cuda_lib, M, V, K, table, out):
    g = rng(M + V)
    w = torch.randn((V, K), generator=g, device="cuda")
    ids = some_ids(M, V, 1)
    sinv = None
    factor = torch.tensor(0.37, device="cuda")
    if table == "e4m3":
        codes = torch.randint(0, 256, (V, K), generator=g, device="cuda").to(torch.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x11
        sinv = torch.tensor([0.03], device="cuda")
        w, values, factor = codes, codes.view(torch.float8_e4m3fn).float(), sinv[0] * factor
    else:
        w = w.to(table)
        values = w.float()
    flat = torch.full((M * K + 64,), 77, dtype=out, device="cuda")
    got = flat[32:32 + M * K].view(M, K)
    cuda_lib.mp_embedding_fwd(ids, w, got, scale=0.37, sinv=sinv)
    assert cuda_lib.fp8mp_check() == 0
    inside = (ids >= 0) & (ids < V)
    want = torch.where(inside[:, None], values[ids.clamp(0, V - 1)] * factor, 0.0).to(out)
    assert torch.equal(got, want) and (flat[:32] == 77).all() and (flat[32 + M * K:] == 77).all()


def backward(lib, ids, dy, V, out, scale=1.0, fill=0xAB):
    M, K = dy.shape
    flat = torch.full((V * K + 64,), 77, dtype=out, device="cuda")
    n = lib.mp_embedding_bwd_workspace_bytes(M, V, K)
    ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
    got = flat[32:32 + V * K].view(V, K)
    lib.mp_embedding_bwd(ids, dy, got, ws[:n], scale=scale)
    assert lib.fp8mp_check() == 0
    assert (flat[:32] == 77).all() and (flat[32 + V * K:] == 77).all() and (ws[n:] == fill).all()
    return got


def hold(got, ids, dy, scale):
    V = got.shape[0]
    inside = (ids >= 0) & (ids < V)
    at, d = ids[inside], dy[inside].double()
    want = torch.zeros(got.shape, dtype=torch.float64, device="cuda").index_put_((at,), d, accumulate=True) * scale
    size = torch.zeros_like(want).index_put_((at,), d.abs(), accumulate=True) * abs(scale)
    count = torch.bincount(at, minlength=V).double()[:, None]
    room = (2 * count + 2) * U * size
    assert ((got.double() - want).abs() <= HALF[got.dtype] * (want.abs() + room) + room).all()
    assert (got[count[:, 0] == 0] == 0).all()


@pytest.mark.parametrize("M,V,K", [(1, 1, 16), (17, 3, 16), (77, 1000, 272), (1000, 77, 1040), (3000, 511, 48), (3000, 512, 64),
                                   (2500, 513, 64), (5000, 30000, 4096), (40000, 262144, 16), (70000, 300, 32), (0, 40, 16), (5000, 2 ** 21 + 5, 16),
                                   (16384, 262143, 16), (16385, 511, 16), (4096, 1023, 16), (4097, 1024, 16),
                                   (32768, 131071, 16), (32768, 131072, 16), (32769, 100, 16),
                                   (32, 9, 4112), (127, 40, 48), (128, 30000, 1040), (129, 40, 48), (128, 3, 16384),
                                   (0, 40, 2064), (300, 70, 4112), (4095, 600, 1040)])
@pytest.mark.parametrize("dy,out", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_backward(cuda_lib, M, V, K, dy, out):
    ids = some_ids(M, V, 2, spread=6.0)
    d = torch.randn((M, K), generator=rng(3), device="cuda").to(dy)
    got = backward(cuda_lib, ids, d, V, out, 1.75)
    hold(got, ids, d, 1.75)
    assert torch.equal(got, backward(cuda_lib, ids, d, V, out, 1.75, fill=0))


@pytest.mark.parametrize("ids", ["one", "none", "rising", "falling", "two", "edges"])
@pytest.mark.parametrize("M", [15, 16, 17, 127, 128, 129, 130, 131, 132, 133, 2049, 40000])
def test_runs(cuda_lib, ids, M):
    """One id throughout, none inside the table, all different, two that alternate,
    runs that end with the chunks."""
    V, K = 50000, 32
    i = torch.arange(M, device="cuda")
    ids = dict(one=torch.full_like(i, 4321), none=torch.where(i % 2 == 0, -5, V), rising=i, falling=V - 1 - i,
               two=i % 2 * 49999, edges=i // 16 * 7)[ids]
    d = torch.randn((M, K), generator=rng(4), device="cuda")
    got = backward(cuda_lib, ids, d, V, F32)
    hold(got, ids, d, 1.0)


def test_the_order_of_equal_ids_is_theirs(cuda_lib):
    """1e8 + 1 - 1e8: the sum depends on its order, which is the positions'."""
    ids = torch.tensor([3, 1, 3, 0, 3, 1], device="cuda")
    d = torch.zeros((6, 16), device="cuda")
    d[0], d[2], d[4] = 1e8, 1.0, -1e8
    d[1], d[5] = 2.0, 3.0
    got = backward(cuda_lib, ids, d, 5, F32)
    assert (got[3] == (torch.tensor(1e8) + 1 - 1e8).item()).all() and (got[1] == 5).all()


@pytest.mark.parametrize("M", [128, 129, 5000])
def test_the_order_of_equal_ids_among_others(cuda_lib, M):
    ids = torch.arange(M, device="cuda") + 10
    ids[[5, 60, M - 1]] = 3
    d = torch.zeros((M, 16), device="cuda")
    d[5], d[60], d[M - 1] = 1e8, 1.0, -1e8
    got = backward(cuda_lib, ids, d, 6000, F32)
    assert (got[3] == (torch.tensor(1e8) + 1 - 1e8).item()).all()


@pytest.mark.parametrize("M", [100, 200])
def test_gradient_of_a_table_of_many_rows(cuda_lib, M):
    """More rows than a block marks at a time, and more bytes than 2^32."""
    V, K = 40000003, 64
    ids = torch.randint(0, V, (M,), generator=rng(11), device="cuda")
    ids[0], ids[1], ids[2], ids[3] = V - 1, V - 1, 0, 131072
    d = torch.randint(1, 9, (M, K), generator=rng(12), device="cuda").to(BF)
    dt = torch.full((V, K), 9, dtype=BF, device="cuda")
    ws = torch.empty(cuda_lib.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    cuda_lib.mp_embedding_bwd(ids, d, dt, ws)
    rows, back = torch.unique(ids, return_inverse=True)
    want = torch.zeros((len(rows), K), device="cuda").index_put_((back,), d.float(), accumulate=True)
    assert torch.equal(dt[rows].float(), want) and cuda_lib.fp8mp_check() == 0
    assert int(dt.view(torch.int32).ne(0).any(1).sum()) == len(rows)


def test_nan_stays_in_its_row(cuda_lib):
    M, V, K = 300, 50, 64
    ids = some_ids(M, V, 5)
    d = torch.randn((M, K), generator=rng(6), device="cuda")
    good = backward(cuda_lib, ids, d, V, F32)
    m = int(torch.nonzero((ids >= 0) & (ids < V))[0])
    d[m, 9] = float("nan")
    d[ids < 0] = float("inf")  # (these have no row)
    got = backward(cuda_lib, ids, d, V, F32)
    same = torch.ones_like(got, dtype=torch.bool)
    same[ids[m], 9] = False
    assert torch.equal(got[same], good[same]) and torch.isnan(got[ids[m], 9])


def test_tables_past_2_32_bytes(cuda_lib):
    V, K = 300001, 8192
    codes = torch.zeros((V, K), dtype=torch.uint8, device="cuda")
    codes[-1] = 0x38  # 1.0
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    out = torch.empty((3, K), dtype=BF, device="cuda")
    cuda_lib.mp_embedding_fwd(ids, codes, out, sinv=torch.ones(1, device="cuda"))
    assert (out[[0, 2]] == 1).all() and (out[1] == 0).all()
    d = torch.ones((3, K), dtype=BF, device="cuda")
    dt = torch.full((V, K), 9, dtype=BF, device="cuda")
    ws = torch.empty(cuda_lib.mp_embedding_bwd_workspace_bytes(3, V, K), dtype=torch.uint8, device="cuda")
    cuda_lib.mp_embedding_bwd(ids, d, dt, ws)
    assert (dt[-1] == 2).all() and (dt[0] == 1).all() and not dt[1:-1].any() and cuda_lib.fp8mp_check() == 0


def test_another_stream_and_a_graph(cuda_lib):
    M, V, K = 500, 3000, 64
    ids = some_ids(M, V, 7)
    d = torch.randn((M, K), generator=rng(8), device="cuda").to(BF)
    want = backward(cuda_lib, ids, d, V, BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = backward(cuda_lib, ids, d, V, BF)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)
    ws = torch.empty(cuda_lib.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    dt = torch.empty((V, K), dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.mp_embedding_bwd(ids, d, dt, ws)
    for seed in (9, 10):
        ids.copy_(some_ids(M, V, seed))
        graph.replay()
        assert torch.equal(dt, backward(cuda_lib, ids, d, V, BF))
