"""Host-side refusals of routing by scores and of the MXFP4 entry points: every call here is
rejected before anything touches the GPU, or has nothing to do."""
import os

import pytest

import mixture_experts_layer_counting_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")

OK, INVAL, UNSUP, WS = moe.MOE_OK, moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED, moe.MOE_EWORKSPACE
P = 1 << 20   # a 16-byte aligned stand-in for a pointer; never read


def status(fn, *args):
    try:
        fn(*args)
    except moe.MoeError as e:
        return e.status
    return OK


def route(T=4, E=16, K=2, score=moe.MOE_SCORE_SIGMOID, groups=4, topk_groups=2, group_top=2, renorm=1, scale=1.0):
    return moe.RouteDesc(T, E, K, score, groups, topk_groups, group_top, renorm, scale)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVAL), (dict(E=0), INVAL), (dict(K=0), INVAL), (dict(score=2), INVAL), (dict(groups=0), INVAL),
    (dict(groups=5), INVAL), (dict(topk_groups=0), INVAL), (dict(topk_groups=5), INVAL), (dict(group_top=0), INVAL),
    (dict(group_top=3), INVAL), (dict(groups=16, topk_groups=16), INVAL),      # group_top 2 of groups of 1
    (dict(K=9), INVAL),                                                      # more than the kept groups hold
    (dict(renorm=2), INVAL), (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL),
    (dict(E=64, K=33, groups=1, topk_groups=1), UNSUP), (dict(E=1028), UNSUP),
    (dict(E=260, groups=130), UNSUP)])
def test_route_scored_refusals(kw, want):
    d = route(**kw)
    assert status(moe.moe_route_scored, d, P, moe.MOE_F32, P, P, P, 0) == want
    assert status(moe.moe_route_scored_backward, d, P, moe.MOE_F32, P, P, P, 0) == want


def test_route_scored_buffers_and_formats():
    f, b = moe.moe_route_scored, moe.moe_route_scored_backward
    assert status(f, route(), None, moe.MOE_F32, None, P, P, 0) == INVAL
    assert status(f, route(), P, moe.MOE_F32, None, None, P, 0) == INVAL
    assert status(f, route(), P, moe.MOE_F32, None, P, None, 0) == INVAL
    assert status(f, route(), P, moe.MOE_FP8_E4M3, None, P, P, 0) == UNSUP
    assert status(b, route(), P, moe.MOE_MXFP4, P, P, P, 0) == UNSUP
    for args in ((None, P, P, P), (P, None, P, P), (P, P, None, P), (P, P, P, None)):
        assert status(b, route(), args[0], moe.MOE_F32, *args[1:], 0) == INVAL
    assert status(f, route(T=0), None, moe.MOE_F32, None, None, None, 0) == OK
    assert status(b, route(T=0), None, moe.MOE_BF16, None, None, None, 0) == OK


def test_mxfp4_rows_refusals():
    q, d = moe.moe_quantize_mxfp4, moe.moe_dequantize_mxfp4
    assert status(q, P, moe.MOE_BF16, -1, 64, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_BF16, 4, 0, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_BF16, 4, 48, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_FP8_E4M3, 4, 64, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_BF16, 2 ** 31 - 1, 2 ** 31 - 32, P, P, 0) == UNSUP
    assert status(q, None, moe.MOE_BF16, 4, 64, P, P, 0) == INVAL
    assert status(q, P + 8, moe.MOE_BF16, 4, 64, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_BF16, 4, 64, P + 2, P, 0) == INVAL
    assert status(q, None, moe.MOE_BF16, 0, 64, None, None, 0) == OK
    assert status(d, P, P, 4, 40, P, moe.MOE_F32, 0) == UNSUP
    assert status(d, P, P, 4, 64, P, moe.MOE_MXFP4, 0) == UNSUP
    assert status(d, P, P, 4, 64, P + 4, moe.MOE_F32, 0) == INVAL
    assert status(d, P, None, 4, 64, P, moe.MOE_F32, 0) == INVAL
    assert status(d, None, None, 0, 64, None, moe.MOE_F32, 0) == OK


def test_mxfp4_weights_refusals():
    q, d = moe.moe_quantize_mxfp4_weights, moe.moe_dequantize_mxfp4_weights
    S, D = moe.MOE_MXFP4, moe.MOE_MXFP4_PAIRED
    assert status(q, P, moe.MOE_BF16, -1, 64, 8, S, P, P, 0) == INVAL
    assert status(q, P, moe.MOE_BF16, 2, 48, 8, S, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_BF16, 2, 64, 8, D, P, P, 0) == UNSUP          # paired needs K % 128
    assert status(q, P, moe.MOE_BF16, 2, 128, 7, D, P, P, 0) == UNSUP         # and N % 2
    assert status(q, P, moe.MOE_BF16, 2, 128, 8, moe.MOE_BF16, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_MXFP4, 2, 128, 8, S, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_F32, 70000, 128, 8, S, P, P, 0) == UNSUP
    assert status(q, P, moe.MOE_F32, 2, 128, 8, S, P + 4, P, 0) == INVAL
    assert status(q, P, moe.MOE_F32, 2, 128, 8, S, P, None, 0) == INVAL
    assert status(q, None, moe.MOE_F32, 2, 128, 0, S, None, None, 0) == OK
    assert status(d, P, P, S, 2, 128, 8, P + 2, moe.MOE_BF16, 0) == INVAL
    assert status(d, P, P, D, 2, 128, 3, P, moe.MOE_BF16, 0) == UNSUP
    assert status(d, None, None, S, 0, 128, 8, None, moe.MOE_BF16, 0) == OK


def test_ffn_mxfp4_refusals():
    up = lambda x=P, xs=P, src=P, T=4, K=2, cu=P, M=8, E=4, H=256, Hp=128, wg=P, hq=P: status(  # noqa: E731
        moe.moe_ffn_gate_up_mxfp4, x, xs, src, T, K, cu, M, E, H, Hp, wg, P, P, P, hq, P, 0)
    assert up(M=-1) == INVAL and up(E=0) == INVAL and up(K=0) == INVAL and up(T=-1) == INVAL
    assert up(H=320) == UNSUP and up(Hp=64) == UNSUP and up(E=1025) == UNSUP
    assert up(H=128, T=2 ** 26) == UNSUP                       # the codes of x past 2 GiB
    assert up(H=2 ** 17, Hp=2 ** 15) == UNSUP                  # the codes of one matrix
    assert up(cu=None) == INVAL and up(x=None) == INVAL and up(xs=None) == INVAL and up(hq=None) == INVAL
    assert up(wg=P + 8) == INVAL and up(x=P + 4) == INVAL
    assert up(M=0, x=None, xs=None, wg=None, hq=None) == OK
    dn = lambda h=P, cu=P, M=8, E=4, H=256, Hp=128, y=P: status(  # noqa: E731
        moe.moe_ffn_down_mxfp4, h, P, cu, M, E, H, Hp, P, P, y, 0)
    assert dn(H=192) == UNSUP and dn(Hp=192) == UNSUP and dn(cu=None) == INVAL and dn(y=None) == INVAL
    assert dn(h=P + 8) == INVAL and dn(y=P + 2) == INVAL and dn(M=0, h=None, y=None) == OK
    n = moe.moe_grouped_ffn_mxfp4_workspace_bytes(8, 128)
    assert n >= 8 * 64 + 8 * 4 and moe.moe_grouped_ffn_mxfp4_workspace_bytes(8, 100) == 0
    gr = lambda ws=P, nb=n, y=P, wd=P, M=8: status(  # noqa: E731
        moe.moe_grouped_ffn_mxfp4, P, P, P, 4, 2, P, M, 4, 256, 128, P, P, wd, P, P, P, y, ws, nb, 0)
    assert gr(nb=n - 1) == WS and gr(ws=None) == WS and gr(y=None) == INVAL and gr(wd=P + 8) == INVAL
    assert gr(ws=P + 8) == INVAL and gr(M=0, ws=None, nb=0) == OK


def test_sizes_past_one_launch_are_refused():
    """A launch's threads along an axis are counted in 32 bits: larger sizes are refused, not cut."""
    d = route(T=2 ** 26)
    assert status(moe.moe_route_scored, d, P, moe.MOE_F32, P, P, P, 0) == UNSUP
    assert status(moe.moe_route_scored_backward, d, P, moe.MOE_F32, P, P, P, 0) == UNSUP
    for f, args in ((moe.moe_quantize_mxfp4, lambda r, c: (P, moe.MOE_BF16, r, c, P, P, 0)),
                    (moe.moe_dequantize_mxfp4, lambda r, c: (P, P, r, c, P, moe.MOE_BF16, 0))):
        assert status(f, *args(2 ** 30, 32)) == UNSUP            # 2^35 values
        assert status(f, *args(2 ** 20, 2 ** 15)) == UNSUP
    for n in (2 ** 30 + 2, 2 ** 31 - 2):                         # column numbers past 32 bits in a lane
        assert status(moe.moe_quantize_mxfp4_weights, P, moe.MOE_BF16, 1, 128, n, moe.MOE_MXFP4, P, P, 0) == UNSUP
        assert status(moe.moe_dequantize_mxfp4_weights, P, P, moe.MOE_MXFP4_PAIRED, 1, 128, n, P, moe.MOE_F32, 0) == UNSUP


def test_matrices_past_one_launch_are_refused():
    for k, n in ((2 ** 8, 2 ** 30), (2 ** 20, 2 ** 18), (2 ** 23, 2 ** 30)):  # 2^38 values and more in one matrix
        assert status(moe.moe_quantize_mxfp4_weights, P, moe.MOE_F32, 1, k, n, moe.MOE_MXFP4, P, P, 0) == UNSUP
        assert status(moe.moe_dequantize_mxfp4_weights, P, P, moe.MOE_MXFP4, 1, k, n, P, moe.MOE_F32, 0) == UNSUP
