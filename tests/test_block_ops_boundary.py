"""Argument checks of the operators around the mixers (ret_rms_norm,
ret_causal_conv, ret_selective_scan, ret_matvec_w4, ret_quantize_w4): every
refusal comes before any CUDA call, so none of this needs a GPU."""
import ctypes

import pytest
import torch

from retentive_network_scale_b200 import build as rbuild
from retentive_network_scale_b200 import retention as R

FAKE, ODD, MISALIGNED = 0x10000, 0x10001, 0x10008  # never dereferenced
S = R.STATUS_NAMES.index
F32, BF16, I8, E4M3 = R.RET_F32, R.RET_BF16, R.RET_I8, R.RET_E4M3


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return R.load_library()


def norm(lib, rows=4, d=64, xt=BF16, x=FAKE, ldx=64, w=FAKE, rt=BF16, r=None, ro=None, eps=1e-5,
         yt=BF16, y=FAKE, group=0, scales=None):
    return lib.ret_rms_norm(rows, d, xt, x, ldx, w, rt, r, ro, eps, yt, y, group, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "RET_ERR_SHAPE"), (dict(d=0), "RET_ERR_SHAPE"),
    (dict(d=R.RET_MAX_NORM_WIDTH + 1, ldx=1 << 20), "RET_ERR_SHAPE"), (dict(ldx=63), "RET_ERR_SHAPE"),
    (dict(group=32), "RET_ERR_SHAPE"), (dict(yt=I8, scales=FAKE, group=16), "RET_ERR_SHAPE"),
    (dict(yt=I8, scales=FAKE, group=128), "RET_ERR_SHAPE"),
    (dict(xt=I8), "RET_ERR_DTYPE"), (dict(yt=4), "RET_ERR_DTYPE"), (dict(rt=-1), "RET_ERR_DTYPE"),
    (dict(eps=-1.0), "RET_ERR_ARG"), (dict(eps=float("nan")), "RET_ERR_ARG"),
    (dict(x=None), "RET_ERR_NULL"), (dict(y=None), "RET_ERR_NULL"), (dict(yt=E4M3), "RET_ERR_NULL"),
    (dict(ro=FAKE), "RET_ERR_NULL"), (dict(x=ODD), "RET_ERR_ALIGN"), (dict(y=MISALIGNED), "RET_ERR_ALIGN"),
    (dict(r=MISALIGNED), "RET_ERR_ALIGN"),
])
def test_rms_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == S(status)


def conv(lib, B=2, L=4, D=8, W=4, t=BF16, x=FAKE, ldx=8, w=FAKE, bias=None, act=1, lengths=None,
         si=None, so=None, y=FAKE):
    return lib.ret_causal_conv(B, L, D, W, t, x, ldx, w, bias, act, lengths, si, so, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "RET_ERR_SHAPE"), (dict(L=-1), "RET_ERR_SHAPE"), (dict(D=0), "RET_ERR_SHAPE"),
    (dict(W=1), "RET_ERR_SHAPE"), (dict(W=R.RET_MAX_CONV_WIDTH + 1), "RET_ERR_SHAPE"),
    (dict(ldx=7), "RET_ERR_SHAPE"), (dict(t=I8), "RET_ERR_DTYPE"), (dict(act=2), "RET_ERR_ARG"),
    (dict(x=None), "RET_ERR_NULL"), (dict(y=None), "RET_ERR_NULL"), (dict(w=None), "RET_ERR_NULL"),
    (dict(x=ODD), "RET_ERR_ALIGN"), (dict(lengths=ODD), "RET_ERR_ALIGN"),
    (dict(so=MISALIGNED), "RET_ERR_ALIGN"),
])
def test_causal_conv_refusals(lib, kw, status):
    assert conv(lib, **kw) == S(status)


def scan(lib, u=FAKE, delta=FAKE, A=FAKE, bm=FAKE, cm=FAKE, z=None, lengths=None, si=None, so=None,
         y=FAKE, **kw):
    base = dict(B=2, L=4, D=8, N=16, G=2, dtype=BF16, softplus=1, ldu=8, ldd=8, ldz=8, ldb=32, ldc=32)
    base.update(kw)
    d = R.RetScanDesc(**base)
    return lib.ret_selective_scan(ctypes.byref(d), u, delta, None, A, bm, cm, None, z, lengths, si, so,
                                  y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "RET_ERR_SHAPE"), (dict(L=-1), "RET_ERR_SHAPE"), (dict(N=0), "RET_ERR_SHAPE"),
    (dict(N=R.RET_MAX_SCAN_STATES + 1, ldb=1 << 12, ldc=1 << 12), "RET_ERR_SHAPE"),
    (dict(G=3), "RET_ERR_SHAPE"), (dict(G=0), "RET_ERR_SHAPE"), (dict(ldu=7), "RET_ERR_SHAPE"),
    (dict(ldd=7), "RET_ERR_SHAPE"), (dict(ldz=7, z=FAKE), "RET_ERR_SHAPE"), (dict(ldb=31), "RET_ERR_SHAPE"),
    (dict(ldc=31), "RET_ERR_SHAPE"), (dict(dtype=E4M3), "RET_ERR_DTYPE"), (dict(softplus=2), "RET_ERR_ARG"),
    (dict(u=None), "RET_ERR_NULL"), (dict(delta=None), "RET_ERR_NULL"), (dict(A=None), "RET_ERR_NULL"),
    (dict(bm=None), "RET_ERR_NULL"), (dict(cm=None), "RET_ERR_NULL"), (dict(y=None), "RET_ERR_NULL"),
    (dict(u=ODD), "RET_ERR_ALIGN"), (dict(z=ODD), "RET_ERR_ALIGN"), (dict(si=MISALIGNED), "RET_ERR_ALIGN"),
    (dict(lengths=ODD), "RET_ERR_ALIGN"),
])
def test_selective_scan_refusals(lib, kw, status):
    assert scan(lib, **kw) == S(status)


def test_selective_scan_null_description(lib):
    assert lib.ret_selective_scan(None, *[FAKE] * 12, None) == S("RET_ERR_NULL")


def matvec(lib, M=2, N=8, K=128, group=128, xt=BF16, x=FAKE, ldx=128, xs=None, xg=0, wq=FAKE, s=FAKE,
           z=None, yt=BF16, y=FAKE):
    return lib.ret_matvec_w4(M, N, K, group, xt, x, ldx, xs, xg, wq, s, z, yt, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "RET_ERR_SHAPE"), (dict(M=R.RET_MAX_MATVEC_ROWS + 1), "RET_ERR_SHAPE"),
    (dict(N=-1), "RET_ERR_SHAPE"), (dict(N=R.RET_MAX_MATVEC_COLUMNS + 1), "RET_ERR_SHAPE"), (dict(K=0), "RET_ERR_SHAPE"), (dict(K=192, ldx=192), "RET_ERR_SHAPE"),
    (dict(group=16), "RET_ERR_SHAPE"), (dict(ldx=127), "RET_ERR_SHAPE"),
    (dict(xg=128), "RET_ERR_SHAPE"), (dict(xt=I8, xs=FAKE, xg=64), "RET_ERR_SHAPE"),
    (dict(xt=I8, xs=FAKE, xg=256), "RET_ERR_SHAPE"),
    (dict(xt=4), "RET_ERR_DTYPE"), (dict(yt=I8), "RET_ERR_DTYPE"),
    (dict(xt=E4M3), "RET_ERR_NULL"), (dict(x=None), "RET_ERR_NULL"), (dict(wq=None), "RET_ERR_NULL"),
    (dict(s=None), "RET_ERR_NULL"), (dict(y=None), "RET_ERR_NULL"),
    (dict(x=ODD), "RET_ERR_ALIGN"), (dict(wq=MISALIGNED), "RET_ERR_ALIGN"), (dict(z=ODD), "RET_ERR_ALIGN"),
])
def test_matvec_w4_refusals(lib, kw, status):
    assert matvec(lib, **kw) == S(status)


def test_quantize_w4_refusals(lib):
    f = lambda K=128, N=8, g=64, t=BF16, W=FAKE, ld=8, q=FAKE, s=FAKE, z=None: \
        lib.ret_quantize_w4(K, N, g, t, W, ld, q, s, z, None)  # noqa: E731
    assert f(K=96) == f(K=0) == f(N=-1) == f(g=48) == f(ld=7) == S("RET_ERR_SHAPE")
    assert f(t=I8) == S("RET_ERR_DTYPE")
    assert f(W=None) == f(q=None) == f(s=None) == S("RET_ERR_NULL")
    assert f(W=ODD) == f(q=MISALIGNED) == f(z=ODD) == S("RET_ERR_ALIGN")


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the refusal on a machine without sm_100")
def test_valid_calls_without_sm100_refuse(lib):
    # empty problems: valid arguments, nothing would be read
    for r in (norm(lib, rows=0), conv(lib, B=0), scan(lib, B=0), matvec(lib, M=0)):
        assert r == S("RET_ERR_UNSUPPORTED")


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(TypeError):
        R.ret_rms_norm(x, x)
    with pytest.raises(TypeError):
        R.ret_causal_conv(x, w, x)
    with pytest.raises(TypeError):
        R.ret_selective_scan(x, x, w, x, x, x)
    with pytest.raises(TypeError):
        R.ret_matvec_w4(x[0], x[0], x[0], x[0])
    with pytest.raises(TypeError):
        R.ret_quantize_w4(w, 32)
