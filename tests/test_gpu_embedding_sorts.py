"""The table's gradient past 4096 tokens: up to 32768 of them sorted in shared memory,
with the zeroing beside it, if key and position fit 32 bits together; else through global
memory. What test_gpu_embedding.py and test_gpu_lm_launch.py test of fewer tokens: runs of
equal ids, streams and graphs, first calls from several threads, what came before on the
stream; and tables of more rows than a block marks at a time.

The gradients are whole numbers (|dy| <= 8, a row's sum below 2^24), so results are exact
in fp32 whatever the order; a row of bf16 is rounded once."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
# (tokens, rows of the table): sorted by counting; in shared memory, least and most tokens,
# with the most rows that each allows; through global memory by rows, and by tokens
WAYS = [(4096, 60000), (4097, 60000), (8192, 2 ** 19 - 1), (16384, 2 ** 18 - 1), (32768, 2 ** 17 - 1),
        (8192, 2 ** 19), (16385, 2 ** 17), (32769, 60000)]


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def some(M, V, K, seed, dtype=F32):
    ids = torch.randint(-3, V + 3, (M,), generator=rng(seed), device="cuda")
    ids[: M // 8] = ids[M // 8]  # a long run among short ones
    return ids, torch.randint(-8, 9, (M, K), generator=rng(seed + 1), device="cuda").to(dtype)


def exact(ids, dy, V):
    inside = (ids >= 0) & (ids < V)
    return torch.zeros((V, dy.shape[1]), device="cuda").index_put_((ids[inside],), dy[inside].float(), accumulate=True)


def workspace(lib, M, V, K):
    return torch.empty(lib.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,V", WAYS)
@pytest.mark.parametrize("kind", ["one", "none", "rising", "falling", "two", "last"])
def test_runs(cuda_lib, kind, M, V):
    K = 32
    i = torch.arange(M, device="cuda")
    ids = dict(one=torch.full_like(i, 4321), none=torch.where(i % 2 == 0, -5, V), rising=i, falling=V - 1 - i,
               two=i % 2 * (V - 1), last=V - 1 - i // 16 * 7)[kind]
    dy = torch.randint(-8, 9, (M, K), generator=rng(M), device="cuda").float()
    got = torch.full((V, K), 7.0, device="cuda")
    cuda_lib.mp_embedding_bwd(ids, dy, got, workspace(cuda_lib, M, V, K))
    assert torch.equal(got, exact(ids, dy, V)) and cuda_lib.fp8mp_check() == 0


@pytest.mark.parametrize("M,V", WAYS)
def test_the_order_of_equal_ids(cuda_lib, M, V):
    """1e8 + 1 - 1e8 at three far positions: the sum depends on its order."""
    ids = torch.arange(M, device="cuda") + 10
    ids[[5, M // 2, M - 1]] = 3
    d = torch.zeros((M, 16), device="cuda")
    d[5], d[M // 2], d[M - 1] = 1e8, 1.0, -1e8
    got = torch.empty((V, 16), device="cuda")
    cuda_lib.mp_embedding_bwd(ids, d, got, workspace(cuda_lib, M, V, 16))
    assert (got[3] == (torch.tensor(1e8) + 1 - 1e8).item()).all() and cuda_lib.fp8mp_check() == 0


@pytest.mark.parametrize("M,V", WAYS)
def test_it_waits_for_its_inputs(cuda_lib, M, V):
    """The zeroing that starts beside the sort does not start beside what came before: a
    long kernel that still reads the last gradient, and others that write the ids and dy."""
    K = 16 * max(1, min(64, 2 ** 26 // V // 16))
    dt, kept = torch.zeros((V, K), dtype=BF, device="cuda"), torch.empty((V, K), dtype=BF, device="cuda")
    ws = workspace(cuda_lib, M, V, K)
    ids, dy = torch.empty(M, dtype=torch.int64, device="cuda"), torch.empty((M, K), dtype=BF, device="cuda")
    for turn in range(10):
        new_ids, new_dy = some(M, V, K, 100 * turn, BF)
        torch.cuda.synchronize()
        dt.fill_(turn + 1)
        kept.copy_(dt)                   # (reads what the call then overwrites)
        dy.copy_(new_dy)
        ids.copy_(new_ids)
        cuda_lib.mp_embedding_bwd(ids, dy, dt, ws)
        dy.fill_(float("nan"))           # (and this waits for the call)
        ids.fill_(0)
        assert (kept == turn + 1).all(), turn
        assert torch.equal(dt, exact(new_ids, new_dy, V).to(BF)), turn
    assert cuda_lib.fp8mp_check() == 0


@pytest.mark.parametrize("M,V", WAYS)
def test_another_stream_and_two_graphs(cuda_lib, M, V):
    """Two graphs of one workspace, replayed one after another on one stream."""
    K = 48
    a, b = ([*some(M, V, K, seed), torch.full((V, K), 5.0, device="cuda")] for seed in (1, 2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda_lib.mp_embedding_bwd(*a, workspace(cuda_lib, M, V, K))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a[2], exact(a[0], a[1], V))
    ws, graphs = workspace(cuda_lib, M, V, K), []
    for of in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            cuda_lib.mp_embedding_bwd(*of, ws)
    for turn in range(3):
        for of in (a, b):
            ids, dy = some(M, V, K, 50 + turn)
            of[0].copy_(ids.roll(turn))
            of[1].copy_(dy)
        graphs[0].replay()
        graphs[1].replay()
        for of in (a, b):
            assert torch.equal(of[2], exact(of[0], of[1], V)), turn
    assert cuda_lib.fp8mp_check() == 0


@pytest.mark.parametrize("M,V", [(5000, 40000003), (32769, 40000003), (4096, 40000003)])
def test_more_rows_than_a_block_marks(cuda_lib, M, V):
    """131579 rows a block or more where it marks 131072 at a time, the ids on both sides
    of a block's windows; more bytes than 2^32."""
    K = 64
    ids, d = some(M, V, K, 11, BF)
    part = torch.tensor([V * p // 304 for p in range(305)], device="cuda")
    edges = torch.cat([part[1:] - 1, part[:-1], part[:-1] + 131071, part[:-1] + 131072])
    ids[-len(edges):] = edges
    d = d.abs()
    d[:, 0] = 1  # (a row with a token is not zero)
    dt = torch.full((V, K), 9, dtype=BF, device="cuda")
    cuda_lib.mp_embedding_bwd(ids, d, dt, workspace(cuda_lib, M, V, K))
    inside = (ids >= 0) & (ids < V)
    rows, back = torch.unique(ids[inside], return_inverse=True)
    want = torch.zeros((len(rows), K), device="cuda").index_put_((back,), d[inside].float(), accumulate=True)
    assert torch.equal(dt[rows], want.to(BF)) and cuda_lib.fp8mp_check() == 0
    assert int(dt.view(torch.int32).ne(0).any(1).sum()) == len(rows)


CHILD = r"""
import sys, threading, torch
sys.path.insert(0, ROOT)
import fp8_mixed_precision_reduce_gb300 as f

K = 64
torch.cuda.init()

def run(stream, ins):
    out = []
    with torch.cuda.stream(stream):
        for ids, dy, V in ins:
            dt = torch.empty((V, K), device="cuda")
            ws = torch.empty(f.mp_embedding_bwd_workspace_bytes(len(ids), V, K), dtype=torch.uint8, device="cuda")
            f.mp_embedding_bwd(ids, dy, dt, ws)
            out.append(dt)
        stream.synchronize()
    return out

def inputs(i):
    g = torch.Generator(device="cuda").manual_seed(i)
    return [(torch.randint(-1, V, (M,), generator=g, device="cuda"), torch.randn((M, K), generator=g, device="cuda"), V)
            for M, V in ((16384, 5000 + i), (5000, 60000), (32768, 1000), (40000, 3000))]

ins = [inputs(i) for i in range(8)]
torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in range(8)]
out = [None] * 8
barrier = threading.Barrier(8)

def worker(i):
    barrier.wait()
    out[i] = run(streams[i], ins[i])

threads = [threading.Thread(target=worker, args=(i,)) for i in range(8)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert f.fp8mp_check() == 0
for i in range(8):
    assert all(torch.equal(a, b) for a, b in zip(out[i], run(torch.cuda.current_stream(), ins[i]))), i
print("threads ok")
"""


def test_first_calls_from_eight_threads():
    code = CHILD.replace("ROOT", repr(ROOT), 1)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "threads ok" in r.stdout


def test_without_programmatic_launch():
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_gpu_embedding_sorts.py", "-k",
           "waits or order or (test_runs and (two or last))"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8MP_PDL="0"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
