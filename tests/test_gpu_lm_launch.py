"""The norm, the log probabilities and the embedding: first calls from several host
threads at once, each on its own stream (per-device settings are made on first use), and
without programmatic launch, each in a fresh interpreter; one graph's replays among other
work; calls one after another that depend on each other."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, threading, torch
sys.path.insert(0, ROOT)
import fp8_mixed_precision_reduce_gb300 as f

M, K, V = 700, 1040, 5008
torch.cuda.init()

def inputs(i):
    g = torch.Generator(device="cuda").manual_seed(i)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return r(M, K).bfloat16(), r(M, K), 1 + 0.1 * r(K), r(M, V) * 3, torch.randint(-1, V, (M,), generator=g, device="cuda")

def run(stream, ins):
    x, res, w, logits, t = ins
    with torch.cuda.stream(stream):
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
        one, am = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
        y, rstd, tot = e(M, K, dtype=torch.uint8), e(M), e(M, K)
        f.fp8_rmsnorm_fwd(x, w, y, rstd, residual=res, total=tot, y_scale=one, y_amax=am)
        dr, dw, dx = e(M, K), e(K), e(M, K, dtype=torch.bfloat16)
        ws = e(f.fp8_rmsnorm_bwd_workspace_bytes(M, K), dtype=torch.uint8)
        f.fp8_rmsnorm_bwd(x, tot, w, rstd, dr, dw, ws, dtotal=res, dx=dx)
        lp, st, H, top, ids = e(M), e(M, 2), e(M), e(M, 5), e(M, 5, dtype=torch.int64)
        f.mp_logprobs_fwd(logits, t, lp, st, entropy=H, top_logprob=top, top_id=ids)
        d8 = e(M, V, dtype=torch.uint8)
        f.mp_logprobs_bwd(logits, t, st, lp, d8, entropy=H, dentropy=H, scale=one, amax=am)
        out = e(M, K)
        f.mp_embedding_fwd(t % V, logits[:, :K].contiguous(), out, scale=2.0)
        dt = e(V, K)
        ws2 = e(f.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8)
        f.mp_embedding_bwd(t, dx, dt, ws2)  # (dx comes from the norm's backward pass)
        stream.synchronize()
        return [y, rstd, tot, am, dr, dw, dx, lp, st, H, top, ids, d8, out, dt]

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
    ref = run(torch.cuda.current_stream(), ins[i])
    assert all(torch.equal(a, b) for a, b in zip(out[i], ref)), i
print("threads ok")
"""


def test_first_calls_from_eight_threads():
    code = CHILD.replace("ROOT", repr(ROOT), 1)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "threads ok" in r.stdout


def test_without_programmatic_launch():
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_gpu_norm.py",
           "tests/test_gpu_logprob.py", "tests/test_gpu_embedding.py", "-k",
           "(test_forward and (1237 or 4097 or 5003)) or (test_backward and (1237 or 5008 or 30000)) or test_runs or graph"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8MP_PDL="0"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout


def test_the_tables_gradient_waits_for_its_inputs(cuda_lib):
    """Its zeroing starts beside its sort, not beside what came before: a long kernel that
    still reads the last gradient, and one that still writes the ids and dy."""
    M, V, K = 4096, 60000, 1024
    dt = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(cuda_lib.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    for turn in range(20):
        g = torch.Generator(device="cuda").manual_seed(turn)
        ids = torch.empty(M, dtype=torch.int64, device="cuda")
        dy = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        new = torch.randint(0, V, (M,), generator=g, device="cuda")
        torch.cuda.synchronize()
        dt.fill_(turn + 1)
        read = dt.float().sum()          # (reads what the call then overwrites)
        dy.fill_(1.0)
        ids.copy_(new)
        cuda_lib.mp_embedding_bwd(ids, dy, dt, ws)
        after = dt.float().sum()
        assert read.item() == (turn + 1.0) * V * K and after.item() == float(M) * K, turn
        count = torch.bincount(new, minlength=V)
        assert torch.equal(dt[:, 0].float(), count.float()) and torch.equal(dt[:, -1], dt[:, 0])


def test_a_graph_among_other_calls(cuda_lib):
    """Replays of a captured call and eager calls on one stream, in turn."""
    M, V = 64, 30000
    x = torch.randn((M, V), device="cuda").bfloat16()
    t = torch.randint(0, V, (M,), device="cuda")
    a, st, d = torch.empty(M, device="cuda"), torch.empty((M, 2), device="cuda"), torch.empty_like(x)
    b, st2 = torch.empty(M, device="cuda"), torch.empty((M, 2), device="cuda")
    cuda_lib.mp_logprobs_fwd(x, t, a, st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.mp_logprobs_fwd(x, t, a, st)
        cuda_lib.mp_logprobs_bwd(x, t, st, a, d)
    for turn in range(10):
        x.copy_(torch.randn((M, V), device="cuda"))
        graph.replay()
        cuda_lib.mp_logprobs_fwd(x, t, b, st2)
        e = torch.empty_like(x)
        cuda_lib.mp_logprobs_bwd(x, t, st2, b, e)
        assert torch.equal(a, b) and torch.equal(d, e)
    assert cuda_lib.fp8mp_check() == 0
