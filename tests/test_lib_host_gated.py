"""What the gated feed-forward calls and their binding refuse, without a GPU."""

import pytest
import torch

import fp8_mixed_precision_reduce_gb300 as fp8mp

P = 4096  # a fake, aligned address: validation fails before it is used


@pytest.fixture(scope="module")
def lib():
    fp8mp.build()
    return fp8mp.load()


def fwd(lib, x8=P, w8=P, M=5, F=32, K=48, act=0, sx=P, sw=P, hs=P, h=P, amax=None, gu=None):
    return lib.fp8_gated_fwd(x8, w8, M, F, K, act, sx, sw, hs, h, amax, gu, None)


def dgrad(lib, dy8=P, wd8=P, gu=P, M=5, F=32, N=48, act=0, fmt=1, sy=P, sw=P, scale=P, out=P, amax=None):
    return lib.fp8_gated_dgrad(dy8, wd8, gu, M, F, N, act, fmt, sy, sw, scale, out, amax, None)


def bwd(lib, dh=P, dh_dtype=1, gu=P, x8=P, w8=P, M=5, F=32, K=48, act=0, sx=P, sw=P, scale=P, sinv=P, dgu8=P,
        amax=None, dx=P, dx_dtype=1, dw=1 << 20, dw_dtype=1, flag=None):
    return lib.fp8_gated_bwd(dh, dh_dtype, gu, x8, w8, M, F, K, act, sx, sw, scale, sinv, dgu8, amax, dx, dx_dtype, dw,
                             dw_dtype, flag, None)


BAD_SIZES = [(dict(F=40), "multiples of 16"), (dict(M=-1), "negative"), (dict(F=1 << 30), "too large"),
             (dict(act=2), "act")]


@pytest.mark.parametrize("kw,word", BAD_SIZES + [
    (dict(K=24), "multiples of 16"), (dict(h=None), "h is NULL"), (dict(h=P + 8), "aligned"), (dict(x8=None), "x8"),
    (dict(w8=P + 1), "aligned"), (dict(sx=None), "sinv_x"), (dict(sw=P + 2), "misaligned"), (dict(hs=P + 2), "h_scale"),
    (dict(gu=P + 2), "aligned"), (dict(amax=P + 1), "misaligned")])
def test_forward(lib, kw, word):
    assert fwd(lib, **kw) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


@pytest.mark.parametrize("kw,word", BAD_SIZES + [
    (dict(N=24), "multiples of 16"), (dict(gu=None), "gu"), (dict(out=None), "dgu8"), (dict(scale=None), "dgu_scale"),
    (dict(dy8=P + 4), "aligned"), (dict(wd8=None), "wd8"), (dict(fmt=2), "dy_fmt"), (dict(sy=None), "sinv_dy")])
def test_dgrad(lib, kw, word):
    assert dgrad(lib, **kw) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


@pytest.mark.parametrize("kw,word", BAD_SIZES + [
    (dict(K=24), "multiples of 16"), (dict(dh_dtype=3), "dh_dtype"), (dict(dx_dtype=3), "dx_dtype"),
    (dict(dw_dtype=3), "dw_dtype"), (dict(gu=None), "gu"), (dict(dgu8=None), "dgu8"), (dict(scale=None), "dgu_scale"),
    (dict(sinv=None), "dgu_sinv"), (dict(x8=None), "x8"), (dict(w8=None), "w8"), (dict(sx=None), "sinv_x"),
    (dict(sw=None), "sinv_w"), (dict(dw=P + 16), "overlap"), (dict(dh=P + 2), "aligned"),
    (dict(flag=P + 1), "misaligned")])
def test_backward(lib, kw, word):
    assert bwd(lib, **kw) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(M=129), "outside 0..128"), (dict(M=-1), "outside"), (dict(N=24), "multiples of 16"), (dict(K=8), "multiples of 16"),
    (dict(N=1 << 31), "2^30"), (dict(y=None), "y is NULL"), (dict(y_dtype=4), "y_dtype"), (dict(bias=P, bias_dtype=4), "bias_dtype"),
    (dict(x8=P + 1), "aligned"), (dict(w8=None), "w8"), (dict(sx=None), "sinv_x"), (dict(amax=P + 1), "misaligned")])
def test_linear_few(lib, kw, word):
    a = dict(x8=P, w8=P, M=5, N=32, K=48, sx=P, sw=P, bias=None, bias_dtype=0, y=P, y_dtype=1, amax=None)
    a.update(kw)
    assert lib.fp8_linear_few(*a.values(), None) == fp8mp.ERR_INVALID
    assert word in fp8mp.last_error(), fp8mp.last_error()


def test_nothing_to_do_needs_no_device(lib):
    assert fwd(lib, M=0, x8=None, h=None) == fp8mp.OK
    assert fwd(lib, F=0, w8=None, h=None) == fp8mp.OK
    assert dgrad(lib, M=0, dy8=None, out=None) == fp8mp.OK
    assert bwd(lib, M=0, dw=None, dx=None, dh=None) == fp8mp.OK


def test_binding_checks_shapes_and_types():
    u8, bf = torch.uint8, torch.bfloat16
    z = lambda *s, dtype=u8: torch.zeros(s, dtype=dtype)  # noqa: E731
    one = torch.ones(1)
    x8, w8 = z(5, 48), z(64, 48)
    for h, kw in ((z(5, 32, dtype=bf), dict(h_scale=one)), (z(5, 32), {}), (z(5, 48), dict(h_scale=one)),
                  (z(5, 32), dict(h_scale=one, gu=z(5, 32, dtype=bf))),
                  (z(5, 32), dict(h_scale=one, gu=z(5, 64, dtype=torch.float32)))):
        with pytest.raises(fp8mp.Fp8mpError):
            fp8mp.fp8_gated_fwd(x8, w8, one, one, h, **kw)
    with pytest.raises(fp8mp.Fp8mpError):
        fp8mp.fp8_gated_fwd(x8, z(64, 32), one, one, z(5, 32), h_scale=one)
    with pytest.raises(fp8mp.Fp8mpError):
        fp8mp.fp8_gated_dgrad(z(5, 48), z(48, 32), z(5, 32, dtype=bf), one, one, one, z(5, 64))
    with pytest.raises(fp8mp.Fp8mpError):
        fp8mp.fp8_gated_bwd(z(5, 32, dtype=bf), None, x8, w8, one, one, one, one, z(5, 64), None, None)
    with pytest.raises(fp8mp.Fp8mpError):
        fp8mp.fp8_gated_bwd(None, None, x8, w8, one, one, None, one, z(5, 64), z(5, 32, dtype=bf), None)
