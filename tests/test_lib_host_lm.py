"""What the norm, the log probabilities and the embedding and their binding refuse,
without a GPU."""

import pytest
import torch

import fp8_mixed_precision_reduce_gb300 as fp8mp

P = 1 << 12  # fake, aligned addresses, far apart: validation fails before one is used
Q, R, S = 1 << 30, 1 << 31, 1 << 32


@pytest.fixture(scope="module")
def lib():
    fp8mp.build()
    return fp8mp.load()


def refused(call, defaults, kw, word):
    a = dict(defaults)
    a.update(kw)
    assert call(*a.values(), None) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


NORM = dict(x=P, x_dtype=1, residual=None, total=None, t_dtype=1, M=5, K=48, w=P, w_dtype=0, eps=1e-6, scale=P, y=Q,
            y_dtype=1, amax=None, rstd=P)


@pytest.mark.parametrize("kw,word", [
    (dict(K=24), "multiple of 16"), (dict(K=16400), "16384"), (dict(M=-1), "outside"), (dict(M=1 << 31), "outside"),
    (dict(x_dtype=2), "x_dtype"), (dict(w_dtype=5), "w_dtype"), (dict(scale=None, y_dtype=7), "y_dtype"),
    (dict(residual=P), "together"), (dict(total=P), "together"), (dict(residual=R, total=S, t_dtype=3), "t_dtype"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(x=None), "x is NULL"),
    (dict(x=P + 8), "aligned"), (dict(w=None), "w is NULL"), (dict(w=P + 4), "aligned"), (dict(y=None), "y is NULL"),
    (dict(scale=P + 2), "scale"), (dict(amax=P + 1), "misaligned"), (dict(rstd=None), "rstd"), (dict(y=P), "overlap"),
    (dict(residual=R, total=R + 16), "in part"), (dict(residual=R, total=P), "overlap"),
    (dict(residual=Q, total=R), "y overlaps"), (dict(residual=R, total=Q + 64), "y overlaps")])
def test_norm_forward(lib, kw, word):
    refused(lib.fp8_rmsnorm_fwd, NORM, kw, word)


NORM_BWD = dict(dy=P, dy_dtype=1, dtotal=None, total=Q, t_dtype=1, rstd=P, M=5, K=48, w=P, w_dtype=0, dr=R, dx=None, dw=S,
                dw_dtype=0, ws=S + 4096, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,word", [
    (dict(K=8), "multiple of 16"), (dict(M=-2), "outside"), (dict(dy_dtype=2), "dy_dtype"), (dict(t_dtype=-1), "t_dtype"),
    (dict(w_dtype=2), "w_dtype"), (dict(dw_dtype=2), "dw_dtype"), (dict(dy=None), "dy is NULL"), (dict(total=Q + 2), "aligned"),
    (dict(dr=None), "dresidual"), (dict(rstd=P + 2), "misaligned"), (dict(dw=S + 4), "aligned"), (dict(ws=None), "workspace"),
    (dict(ws_bytes=191), "needed"), (dict(dtotal=R + 16), "in part"), (dict(dr=Q), "overlaps"), (dict(dr=P + 16), "overlaps"),
    (dict(dx=R), "dx"), (dict(dx=P), "dx"), (dict(dtotal=S + 65536, dx=S + 65536), "dx")])
def test_norm_backward(lib, kw, word):
    refused(lib.fp8_rmsnorm_bwd, NORM_BWD, kw, word)


LOGP = dict(x=P, dtype=1, M=3, V=100, ld=112, targets=P, logprob=P, stats=P, entropy=None, top=None, ids=None, k=0)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "x_dtype"), (dict(M=-1), "M = -1"), (dict(V=0), "V = 0"), (dict(V=113), "V = 113"),
    (dict(ld=1 << 31), "2^31"), (dict(M=1 << 30, ld=1 << 20), "too large"), (dict(x=None), "logits is NULL"), (dict(x=P + 1), "misaligned"),
    (dict(x=P + 2, dtype=0), "misaligned"), (dict(targets=None), "together"), (dict(logprob=None), "together"),
    (dict(targets=P + 4), "targets"), (dict(stats=None), "stats"), (dict(stats=P + 4), "stats"), (dict(entropy=P + 2), "entropy"),
    (dict(k=33), "top = 33"), (dict(k=-1), "top = -1"), (dict(k=8, V=7), "top = 8"), (dict(k=3, ids=P), "top_logprob"),
    (dict(k=3, top=P), "top_id"), (dict(k=3, top=P, ids=P + 4), "top_id")])
def test_logprobs_forward(lib, kw, word):
    refused(lib.mp_logprobs_fwd, LOGP, kw, word)


LOGP_BWD = dict(x=P, dtype=1, M=3, V=100, ld=112, targets=P, stats=P, da=P, entropy=None, db=None, scale=P, out=Q, amax=None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "x_dtype"), (dict(V=200), "V = 200"), (dict(entropy=P), "together"), (dict(db=P), "together"),
    (dict(ld=104), "multiple of 16"), (dict(x=P + 2), "aligned"), (dict(out=Q + 8), "aligned"), (dict(out=None), "dlogits"),
    (dict(out=P + 16), "overlap"), (dict(targets=None), "targets"), (dict(stats=P + 4), "stats"), (dict(da=None), "dlogprob"),
    (dict(scale=P + 1), "scale"), (dict(amax=P + 3), "amax"), (dict(scale=None, out=Q + 1), "misaligned"),
    (dict(scale=None, out=Q + 2), "modulo 16"), (dict(scale=None, out=P + 32), "in part")])
def test_logprobs_backward(lib, kw, word):
    refused(lib.mp_logprobs_bwd, LOGP_BWD, kw, word)


EMBED = dict(ids=P, M=3, table=P, dtype=1, V=10, K=32, sinv=None, scale=1.0, out=Q, out_dtype=1)


@pytest.mark.parametrize("kw,word", [
    (dict(M=-1), "M = -1"), (dict(V=-1), "V = -1"), (dict(V=1 << 31), "2^31"), (dict(M=1 << 29, K=1 << 16), "too large"), (dict(K=24), "multiple of 16"),
    (dict(ids=None), "ids"), (dict(ids=P + 4), "misaligned"), (dict(dtype=2), "table_dtype"), (dict(out_dtype=2), "out_dtype"),
    (dict(table=None), "table"), (dict(table=P + 8), "aligned"), (dict(out=None), "out is NULL"), (dict(sinv=P + 2), "sinv"),
    (dict(out=P + 16), "overlap")])
def test_embedding_forward(lib, kw, word):
    refused(lib.mp_embedding_fwd, EMBED, kw, word)


EMBED_BWD = dict(ids=P, M=3, dy=P, dy_dtype=1, V=10, K=32, scale=1.0, dt=Q, dt_dtype=0, ws=R, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,word", [
    (dict(M=1 << 30), "2^30 - 1"), (dict(K=-16), "K = -16"), (dict(ids=P + 2), "misaligned"), (dict(dy_dtype=2), "dy_dtype"),
    (dict(dt_dtype=9), "dtable_dtype"), (dict(dy=None), "dy is NULL"), (dict(dt=None), "dtable"), (dict(ws=R + 4), "aligned"),
    (dict(ws_bytes=100), "needed"), (dict(dt=P), "overlap")])
def test_embedding_backward(lib, kw, word):
    refused(lib.mp_embedding_bwd, EMBED_BWD, kw, word)


def test_workspaces(lib):
    assert lib.fp8_rmsnorm_bwd_workspace_bytes(5, 24) == -1 and lib.fp8_rmsnorm_bwd_workspace_bytes(-1, 16) == -1
    assert lib.fp8_rmsnorm_bwd_workspace_bytes(0, 64) == 0 and lib.fp8_rmsnorm_bwd_workspace_bytes(5, 2048) > 0
    assert lib.mp_embedding_bwd_workspace_bytes(5, 10, 24) == -1 and lib.mp_embedding_bwd_workspace_bytes(5, 10, 32) > 0


def test_nothing_to_do_needs_no_device(lib):
    empty = dict.fromkeys(("x", "w", "y", "scale", "rstd"))
    assert lib.fp8_rmsnorm_fwd(*{**NORM, **empty, "M": 0}.values(), None) == fp8mp.OK
    assert lib.fp8_rmsnorm_fwd(*{**NORM, **empty, "K": 0}.values(), None) == fp8mp.OK
    assert lib.fp8_rmsnorm_bwd(*{**NORM_BWD, "M": 0, "dw": None}.values(), None) == fp8mp.OK
    assert lib.mp_logprobs_fwd(*{**LOGP, "M": 0, "x": None, "stats": None}.values(), None) == fp8mp.OK
    assert lib.mp_logprobs_bwd(*{**LOGP_BWD, "M": 0, "x": None, "out": None}.values(), None) == fp8mp.OK
    assert lib.mp_embedding_fwd(*{**EMBED, "M": 0, "ids": None, "out": None}.values(), None) == fp8mp.OK
    assert lib.mp_embedding_bwd(*{**EMBED_BWD, "V": 0, "dt": None, "ws": None}.values(), None) == fp8mp.OK


BF, F32, U8, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64


def z(*s, dtype=F32):
    return torch.zeros(s, dtype=dtype)


def raises(f, *args, **kw):
    with pytest.raises(fp8mp.Fp8mpError) as e:
        f(*args, **kw)
    assert "current CUDA device" not in str(e.value)  # (which every call on the CPU ends with)


def test_tensors_off_the_gpu_are_refused():
    x, w, y, r = z(5, 32), z(32), z(5, 32), z(5)
    for device in ("cpu", "meta"):
        with pytest.raises(fp8mp.Fp8mpError, match="current CUDA device"):
            fp8mp.fp8_rmsnorm_fwd(*(t.to(device) for t in (x, w, y, r)))


def test_binding_checks_the_norms_tensors():
    f, one = fp8mp.fp8_rmsnorm_fwd, torch.ones(1)
    x, w, y, r = z(5, 32, dtype=BF), z(32), z(5, 32, dtype=BF), z(5)
    for args, kw in (((z(32, dtype=BF), w, y, r), {}), ((x.half(), w, y, r), {}), ((x, z(16), y, r), {}),
                     ((x, w, y, r), dict(y_scale=one)), ((x, w, y.to(U8), r), {}), ((x, w, y, z(4)), {}),
                     ((x, w, y, r.double()), {}), ((x, w, y, r), dict(residual=x)), ((x, w, y, r), dict(total=x)),
                     ((x, w, y, r), dict(residual=x, total=z(5, 32))), ((x.t(), w, y, r), {}),
                     ((x, w, y, r), dict(y_amax=z(2))), ((x, w, y, r), dict(y_amax=one.double()))):
        raises(f, *args, **kw)
    b, ws = fp8mp.fp8_rmsnorm_bwd, z(1 << 20, dtype=U8)
    for args, kw in (((x, x, w, r, z(5, 32)), {}), ((x, z(5, 16, dtype=BF), w, r, y), {}), ((x, x, w, r, y, z(32)), {}),
                     ((x, x, w, r, y, z(16), ws), {}), ((x, x, w, r, y, z(32), ws.float()), {}), ((x, x, w, r, y), dict(dtotal=z(5, 32))),
                     ((x, z(5, 32), w, r, z(5, 32)), dict(dx=z(5, 32)))):
        raises(b, *args, **kw)


def test_binding_checks_the_logits_tensors():
    f, x, t, r, st = fp8mp.mp_logprobs_fwd, z(3, 48, dtype=BF), z(3, dtype=I64), z(3), z(3, 2)
    for args, kw in (((x[0], t, r, st), {}), ((x.half(), t, r, st), {}), ((x[:, :40], t, r, st), {}),
                     ((x, t.int(), r, st), {}), ((x, t, None, st), {}), ((x, None, r, st), {}), ((x, t, r, z(3)), {}),
                     ((x, t, r, st), dict(vocab=49)), ((x, t, r, st), dict(vocab=0)), ((x, t, r, st), dict(entropy=z(2))),
                     ((x, t, r, st), dict(top_id=z(3, 4, dtype=I64))), ((x, t, r, st), dict(top_logprob=z(3, 4))),
                     ((x, t, r, st), dict(top_id=z(3, 4, dtype=I64), top_logprob=z(3, 5))),
                     ((x, t, r, st), dict(top_id=z(3, 40, dtype=I64), top_logprob=z(3, 40)))):
        raises(f, *args, **kw)
    b, one, d = fp8mp.mp_logprobs_bwd, torch.ones(1), z(3, 48, dtype=BF)
    for args, kw in (((x, t, st, r, d.float()), {}), ((x, t, st, r, d), dict(scale=one)), ((x, t, st, r, d.to(U8)), {}),
                     ((x, t, st, z(4), d), {}), ((x, t, st, r, d), dict(entropy=r)), ((x, t, st, r, d), dict(dentropy=r)),
                     ((x, t, st, r, d[:, :32]), {}), ((x, t, st, r, d), dict(amax=z(3)))):
        raises(b, *args, **kw)


def test_binding_checks_the_tables_tensors():
    f, ids, w, out = fp8mp.mp_embedding_fwd, z(4, dtype=I64), z(9, 32), z(4, 32)
    for args, kw in (((ids.int(), w, out), {}), ((ids[None], w, out), {}), ((ids, w, z(4, 16)), {}), ((ids, w.to(U8), out), {}),
                     ((ids, w, out), dict(sinv=torch.ones(1))), ((ids, w.half(), out), {}), ((ids, w, out.half()), {}),
                     ((ids, w.t().contiguous().t(), out), {})):
        raises(f, *args, **kw)
    b, ws = fp8mp.mp_embedding_bwd, z(1 << 20, dtype=U8)
    for args in ((ids, z(3, 32), w, ws), (ids, out, z(9, 16), ws), (ids, out, w[0], ws), (ids, out, w, ws.float())):
        raises(b, *args)
