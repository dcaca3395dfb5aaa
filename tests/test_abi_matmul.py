"""Host-side refusals of the INT8 and grouped-product entry points: every call here is rejected
before anything touches the GPU, or has nothing to do."""
import os

import pytest

import mixture_experts_layer_counting_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")

OK, INVAL, UNSUP, WS = moe.MOE_OK, moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED, moe.MOE_EWORKSPACE
F32, BF16 = moe.MOE_F32, moe.MOE_BF16
P = 1 << 20   # a 16-byte aligned stand-in for a pointer; never read


def status(fn, *args):
    try:
        fn(*args)
    except moe.MoeError as e:
        return e.status
    return OK


def test_int8_rows():
    q, d = moe.moe_quantize_int8, moe.moe_dequantize_int8
    assert status(q, P, BF16, -1, 8, P, P, 0) == INVAL and status(q, P, BF16, 4, 0, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_FP8_E4M3, 4, 8, P, P, 0) == UNSUP and status(d, P, P, 4, 8, P, moe.MOE_MXFP4, 0) == UNSUP
    for x, qq, sf in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P, P + 2)):
        assert status(q, x, BF16, 4, 8, qq, sf, 0) == INVAL
    assert status(q, P + 2, F32, 4, 8, P, P, 0) == INVAL
    assert status(d, P, P, 4, 8, P + 2, F32, 0) == INVAL and status(d, P, None, 4, 8, P, F32, 0) == INVAL
    assert status(q, None, BF16, 0, 8, None, None, 0) == OK and status(d, None, None, 0, 8, None, F32, 0) == OK


def test_int8_weights():
    q, d = moe.moe_quantize_int8_weights, moe.moe_dequantize_int8_weights
    assert status(q, P, BF16, -1, 8, 8, P, P, 0) == INVAL and status(q, P, BF16, 1, 8, -8, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_MXFP4, 1, 8, 8, P, P, 0) == UNSUP
    assert status(q, P, BF16, 1, 2 ** 20, 2 ** 20, P, P, 0) == UNSUP
    assert status(q, P, BF16, 2, 8, 8, None, P, 0) == INVAL and status(q, P + 1, BF16, 2, 8, 8, P, P, 0) == INVAL
    assert status(d, P, P, 2, 8, 8, P + 1, BF16, 0) == INVAL and status(d, P, P + 1, 2, 8, 8, P, BF16, 0) == INVAL
    for e, k, n in ((0, 8, 8), (2, 0, 8), (2, 8, 0)):
        assert status(q, None, F32, e, k, n, None, None, 0) == OK
        assert status(d, None, None, e, k, n, None, F32, 0) == OK


def test_int8_weights_of_an_empty_reduction_have_scales():
    """K = 0 has no codes, but N scales for each matrix: a pointer for them is checked like any other."""
    q = moe.moe_quantize_int8_weights
    for sf in (P + 1, P + 2):
        assert status(q, None, F32, 2, 0, 8, None, sf, 0) == INVAL
    assert status(q, None, F32, 2, 0, 0, None, P + 2, 0) == OK and status(q, None, F32, 0, 0, 8, None, P + 2, 0) == OK


def test_int8_weights_past_what_the_kernels_count():
    """Rows and columns are counted in 32 bits, up to a step past the last one."""
    q, d = moe.moe_quantize_int8_weights, moe.moe_dequantize_int8_weights
    top = 2 ** 30
    for k, n in ((top + 1, 1), (1, top + 1), (2 ** 31 - 1, 1), (1, 2 ** 31 - 1)):
        assert status(q, None, BF16, 1, k, n, None, None, 0) == UNSUP
        assert status(d, None, None, 1, k, n, None, BF16, 0) == UNSUP
    for k, n in ((top, 1), (1, top)):                     # the sizes are taken, the pointers are not
        assert status(q, None, BF16, 1, k, n, None, None, 0) == INVAL
        assert status(d, None, None, 1, k, n, None, BF16, 0) == INVAL


def test_matmul_int8():
    f = lambda x=P, xs=P, M=8, H=64, N=8, w=P, ws=P, y=P, out=BF16: status(  # noqa: E731
        moe.moe_matmul_int8, x, xs, M, H, N, w, ws, y, out, 0)
    assert f(M=-1) == INVAL and f(H=0) == INVAL and f(N=0) == INVAL
    assert f(H=24) == UNSUP and f(H=2 ** 17) == UNSUP and f(N=2 ** 20 + 1) == UNSUP and f(M=2 ** 30 + 1) == UNSUP
    assert f(M=2 ** 30, N=2 ** 20) == UNSUP and f(out=moe.MOE_MXFP4) == UNSUP
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=P + 8), dict(w=P + 8),
               dict(xs=P + 2), dict(ws=P + 2), dict(y=P + 1), dict(y=P + 2, out=F32)):
        assert f(**kw) == INVAL, kw
    assert f(M=0, x=None, xs=None, w=None, ws=None, y=None) == OK


def test_grouped_matmul_int8_and_gate_up():
    f = lambda x=P, xs=P, src=P, T=4, K=2, cu=P, M=8, E=4, H=64, N=8, w=P, ws=P, y=P, out=BF16: status(  # noqa: E731
        moe.moe_grouped_matmul_int8, x, xs, src, T, K, cu, M, E, H, N, w, ws, y, out, 0)
    g = lambda x=P, xs=P, src=P, T=4, K=2, cu=P, M=8, E=4, H=64, N=8, w=P, ws=P, y=P: status(  # noqa: E731
        moe.moe_ffn_gate_up_int8, x, xs, src, T, K, cu, M, E, H, N, w, P, ws, P, y, 0)
    for h in (f, g):
        assert h(M=-1) == INVAL and h(E=0) == INVAL and h(K=0) == INVAL and h(T=-1) == INVAL and h(N=0) == INVAL
        assert h(H=40) == UNSUP and h(E=1025) == UNSUP and h(H=2 ** 17) == UNSUP
        assert h(T=2 ** 25, H=64) == UNSUP                    # the gathered codes past 2 GiB
        assert h(M=2 ** 30, N=2 ** 20) == UNSUP
        for kw in (dict(x=None), dict(xs=None), dict(cu=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=P + 4),
                   dict(w=P + 4), dict(ws=P + 1), dict(y=P + 1), dict(cu=P + 2), dict(src=P + 2)):
            assert h(**kw) == INVAL, kw
        assert h(M=0, x=None, xs=None, w=None, ws=None, y=None) == OK
        assert h(M=0, src=None, T=0, K=0, x=None, xs=None, w=None, ws=None, y=None) == OK
    assert f(out=moe.MOE_FP8_E4M3) == UNSUP


def test_grouped_ffn_int8():
    n = moe.moe_grouped_ffn_int8_workspace_bytes(8, 48)
    assert n >= 8 * 48 * 3 + 32 and n % 256 == 0
    assert moe.moe_grouped_ffn_int8_workspace_bytes(8, 40) == 0 and moe.moe_grouped_ffn_int8_workspace_bytes(-1, 48) == 0
    f = lambda x=P, wd=P, sd=P, y=P, ws=P, nb=n, M=8, H=64, Hp=48, E=4, cu=P, su=P: status(  # noqa: E731
        moe.moe_grouped_ffn_int8, x, P, P, 4, 2, cu, M, E, H, Hp, P, P, wd, P, su, sd, y, ws, nb, 0)
    assert f(nb=n - 1) == WS and f(ws=None) == WS and f(ws=P + 8) == INVAL
    assert f(H=40) == UNSUP and f(Hp=40) == UNSUP and f(E=0) == INVAL
    for kw in (dict(x=None), dict(wd=None), dict(sd=None), dict(y=None), dict(cu=None), dict(wd=P + 8), dict(sd=P + 2),
               dict(y=P + 1), dict(su=P + 2), dict(x=P + 8)):
        assert f(**kw) == INVAL, kw
    assert f(M=0, ws=None, nb=0) == OK


def test_grouped_matmul():
    f = lambda x=P, act=BF16, src=P, T=4, K=2, cu=P, M=8, E=4, H=64, N=8, w=P, wgt=None, tr=0, y=P, out=BF16: status(  # noqa: E731
        moe.moe_grouped_matmul, x, act, src, T, K, cu, M, E, H, N, w, act if wgt is None else wgt, tr, y, out, 0)
    assert f(M=-1) == INVAL and f(E=0) == INVAL and f(H=0) == INVAL and f(N=0) == INVAL and f(tr=2) == INVAL
    assert f(K=0) == INVAL and f(T=-1) == INVAL
    assert f(wgt=F32) == UNSUP and f(act=F32) == UNSUP and f(act=moe.MOE_FP8_E4M3) == UNSUP and f(out=moe.MOE_MXFP4) == UNSUP
    assert f(E=1025) == UNSUP and f(H=2 ** 20 + 1) == UNSUP and f(N=2 ** 20 + 1) == UNSUP
    assert f(M=2 ** 30, N=2 ** 20) == UNSUP and f(T=2 ** 24) == UNSUP
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(cu=None), dict(x=P + 1), dict(w=P + 1), dict(y=P + 1),
               dict(cu=P + 1), dict(src=P + 1), dict(y=P + 2, out=F32), dict(x=P + 2, act=F32, out=F32)):
        assert f(**kw) == INVAL, kw
    assert f(M=0, x=None, w=None, y=None) == OK and f(M=0, src=None, T=0, K=0, x=None, w=None, y=None) == OK


def test_grouped_matmul_wgrad():
    f = lambda x=P, dy=P, dt=BF16, cu=P, M=8, E=4, H=64, N=8, dw=P, dwt=F32, acc=0: status(  # noqa: E731
        moe.moe_grouped_matmul_wgrad, x, dy, dt, cu, M, E, H, N, dw, dwt, acc, 0)
    assert f(M=-1) == INVAL and f(E=0) == INVAL and f(H=0) == INVAL and f(N=0) == INVAL and f(acc=2) == INVAL
    assert f(dt=F32, dwt=BF16) == UNSUP and f(dwt=BF16, acc=1) == UNSUP and f(dt=moe.MOE_MXFP4) == UNSUP
    assert f(dwt=moe.MOE_FP8_E4M3) == UNSUP and f(E=1025) == UNSUP and f(E=16, H=2 ** 20, N=2 ** 20) == UNSUP
    for kw in (dict(x=None), dict(dy=None), dict(cu=None), dict(dw=None), dict(x=P + 1), dict(dy=P + 1), dict(dw=P + 2),
               dict(cu=P + 2), dict(x=P + 2, dt=F32)):
        assert f(**kw) == INVAL, kw
