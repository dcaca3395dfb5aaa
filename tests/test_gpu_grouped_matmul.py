"""Products of ragged expert groups and the gradient of their weights, against float64.

A sum of n products in fp32, in any order, errs by at most n 2^-24 of the sum of the products' magnitudes (the
products themselves are exact for bf16 and round once, inside the same bound, for fp32); an output in bf16
rounds once more, by 2^-8 of its value. Adding to what a gradient holds is one more fp32 rounding."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_counting_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FMT = {"f32": (moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, torch.bfloat16)}


def guarded(shape, dtype, fill, skip=0):
    """A tensor that starts `skip` elements into its memory, with 64 elements of `fill` behind it."""
    n = int(np.prod(shape))
    buf = torch.full((skip + n + 64,), fill, dtype=dtype, device=DEV)
    return buf[skip:skip + n].view(*shape), buf[skip + n:]


def values(g, shape, dtype, skip=0):
    t, _ = guarded(shape, dtype, 0, skip)
    t.copy_(torch.randn(*shape, generator=g).to(dtype))
    return t


def np64(t):
    return t.detach().double().cpu().numpy()


def offsets(counts):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return cu, torch.from_numpy(cu).to(DEV)


def by_expert(cu, x, w):
    """The products and the sums of their magnitudes."""
    y = np.zeros((x.shape[0], w.shape[2]))
    m = np.zeros_like(y)
    for e in range(len(cu) - 1):
        a, b = cu[e], cu[e + 1]
        if b > a:
            y[a:b], m[a:b] = x[a:b] @ w[e], np.abs(x[a:b]) @ np.abs(w[e])
    return y, m


SHAPES = [
    ((1,), 1, 1), ((3, 0, 2), 7, 5), ((0, 0, 0), 8, 8), ((5, 1, 0, 33), 40, 24), ((16, 16, 17), 64, 40), ((1,) * 9, 130, 33),
    ((130, 64, 0, 5), 72, 136), ((257, 255), 200, 264), ((40, 300, 0, 511), 256, 257), ((600,), 56, 520),
    ((2, 30, 31, 1), 1024, 192), ((0, 5, 0, 0, 9, 0), 3584, 48), ((8,) * 70, 128, 96), ((31, 250), 510, 65), ((512, 100), 512, 512),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts,H,N", SHAPES)
def test_product(counts, H, N, dtype, out, transposed, gather):
    g = torch.Generator().manual_seed(H + N + transposed)
    E, T, K = len(counts), 40, 3
    cu, cud = offsets(counts)
    rows, M = int(cu[-1]), int(cu[-1]) + 5
    dt = FMT[dtype][1]
    w = values(g, (E, N, H) if transposed else (E, H, N), dt)
    y, yg = guarded((M, N), FMT[out][1], 7.0)
    if gather:
        x = values(g, (T, H), dt)
        src = torch.randint(0, T * K, (M,), generator=g, dtype=torch.int32)
        src[2::11] = -1
        at = src[:rows].long()
        xr = np64(x)[(at // K).clamp(min=0).numpy()] * (at >= 0).numpy()[:, None]
        moe.moe_grouped_matmul(x, FMT[dtype][0], src.to(DEV), T, K, cud, M, E, H, N, w, FMT[dtype][0], transposed, y, FMT[out][0])
    else:
        x = values(g, (M, H), dt)
        xr = np64(x)[:rows]
        moe.moe_grouped_matmul(x, FMT[dtype][0], None, 0, 0, cud, M, E, H, N, w, FMT[dtype][0], transposed, y, FMT[out][0])
    torch.cuda.synchronize()
    wr = np64(w)
    ref, mag = by_expert(cu, xr, wr.transpose(0, 2, 1) if transposed else wr)
    tol = H * U * mag
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    got = np64(y)
    assert (np.abs(got[:rows] - ref) <= tol).all()
    assert (got[rows:] == 7.0).all() and bool((yg == 7.0).all())       # rows behind the groups stay


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts,H,N", SHAPES)
def test_weight_gradient(counts, H, N, dtype, out, accumulate):
    if accumulate and out == "bf16":
        pytest.skip("refused: gradients are added in fp32")
    g = torch.Generator().manual_seed(H + N)
    E = len(counts)
    cu, cud = offsets(counts)
    M = int(cu[-1]) + 5
    x, dy = values(g, (M, H), FMT[dtype][1]), values(g, (M, N), FMT[dtype][1])
    x[cu[-1]:] = float("nan")                                          # rows of no group take no part
    before = torch.randn(E, H, N, generator=g)
    dw, guard = guarded((E, H, N), FMT[out][1], 7.0)
    dw.copy_(before)
    moe.moe_grouped_matmul_wgrad(x, dy, FMT[dtype][0], cud, M, E, H, N, dw, FMT[out][0], accumulate)
    torch.cuda.synchronize()
    xr, dr = np64(x), np64(dy)
    ref, tol = np.zeros((E, H, N)), np.zeros((E, H, N))
    for e in range(E):
        a, b = cu[e], cu[e + 1]
        if b > a:
            ref[e], tol[e] = xr[a:b].T @ dr[a:b], (b - a) * U * (np.abs(xr[a:b]).T @ np.abs(dr[a:b]))
    if accumulate:
        ref = ref + before.double().numpy()
        tol = tol * (1 + U) + U * np.abs(ref)
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(np64(dw) - ref) <= tol).all()
    assert bool((guard == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [0, 1])
def test_gradients_against_differences(dtype, transposed):
    """d/ds of sum(y * dy) along random directions of x and of W: the product is bilinear, so a difference
    of whole steps is exact up to the sums' error."""
    g = torch.Generator().manual_seed(3)
    counts, H, N = (9, 0, 40, 3), 72, 24
    E, t, d = 4, FMT[dtype][1], FMT[dtype][0]
    cu, cud = offsets(counts)
    M = int(cu[-1])
    grid = lambda *s: (torch.randint(-8, 9, s, generator=g) / 4.0).to(t).to(DEV)  # noqa: E731  sums exact in fp32
    shape = (E, N, H) if transposed else (E, H, N)
    x, w, dy, vx, vw = grid(M, H), grid(*shape), grid(M, N), grid(M, H), grid(*shape)

    def y_of(x, w):
        y = torch.empty(M, N, device=DEV)
        o = y if dtype == "f32" else torch.empty(M, N, device=DEV)
        moe.moe_grouped_matmul(x, d, None, 0, 0, cud, M, E, H, N, w, d, transposed, o, moe.MOE_F32)
        return np64(o)

    dx = torch.empty(M, H, device=DEV)
    moe.moe_grouped_matmul(dy, d, None, 0, 0, cud, M, E, N, H, w, d, 1 - transposed, dx, moe.MOE_F32)
    dw = torch.empty(*shape, device=DEV)
    if transposed:
        moe.moe_grouped_matmul_wgrad(dy, x, d, cud, M, E, N, H, dw, moe.MOE_F32, 0)
    else:
        moe.moe_grouped_matmul_wgrad(x, dy, d, cud, M, E, H, N, dw, moe.MOE_F32, 0)
    torch.cuda.synchronize()
    base, dyn = y_of(x, w), np64(dy)
    # multiples of 1/16 below 2^20: every sum, and every shifted operand in bf16 (integers / 4 up to 4), is exact
    assert ((y_of(x + vx, w) - base) * dyn).sum() == (np64(dx) * np64(vx)).sum()
    assert ((y_of(x, w + vw) - base) * dyn).sum() == (np64(dw) * np64(vw)).sum()


@pytest.mark.parametrize("skip", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (3, 5, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_that_start_at_any_element(dtype, skip):
    g = torch.Generator().manual_seed(1)
    counts, H, N = (40, 0, 7, 129), 64, 48
    E, (d, t) = 4, FMT[dtype]
    cu, cud = offsets(counts)
    M = int(cu[-1])
    x, dy = values(g, (M, H), t, skip[0]), values(g, (M, N), t, skip[1])
    for transposed in (0, 1):
        w = values(g, (E, N, H) if transposed else (E, H, N), t, skip[1])
        y, yg = guarded((M, N), t, 7.0, skip[2])
        moe.moe_grouped_matmul(x, d, None, 0, 0, cud, M, E, H, N, w, d, transposed, y, d)
        torch.cuda.synchronize()
        wr = np64(w)
        ref, mag = by_expert(cu, np64(x), wr.transpose(0, 2, 1) if transposed else wr)
        tol = H * U * mag * (1 + 2.0 ** -8) + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(ref)
        assert (np.abs(np64(y) - ref) <= tol).all() and bool((yg == 7.0).all())
    dw, wg = guarded((E, H, N), torch.float32, 7.0, skip[2])
    moe.moe_grouped_matmul_wgrad(x, dy, d, cud, M, E, H, N, dw, moe.MOE_F32, 0)
    torch.cuda.synchronize()
    xr, dr = np64(x), np64(dy)
    for e in range(E):
        a, b = cu[e], cu[e + 1]
        tol = max(b - a, 1) * U * (np.abs(xr[a:b]).T @ np.abs(dr[a:b]))
        assert (np.abs(np64(dw)[e] - xr[a:b].T @ dr[a:b]) <= tol).all()
    assert bool((wg == 7.0).all())


def test_offsets_outside_the_rows_are_cut():
    """Entries below 0 or above M count as the nearer end, a descending pair as no rows."""
    M, H, N, E = 50, 64, 32, 5
    g = torch.Generator().manual_seed(2)
    x, w = values(g, (M, H), torch.bfloat16), values(g, (E, H, N), torch.bfloat16)
    cu = torch.tensor([-9, 20, 12, 40, 70, 1000], dtype=torch.int32, device=DEV)
    y, yg = guarded((M, N), torch.float32, 7.0)
    moe.moe_grouped_matmul(x, moe.MOE_BF16, None, 0, 0, cu, M, E, H, N, w, moe.MOE_BF16, 0, y, moe.MOE_F32)
    dw, wg = guarded((E, H, N), torch.float32, 7.0)
    dy = values(g, (M, N), torch.bfloat16)
    moe.moe_grouped_matmul_wgrad(x, dy, moe.MOE_BF16, cu, M, E, H, N, dw, moe.MOE_F32, 0)
    torch.cuda.synchronize()
    assert bool((yg == 7.0).all()) and bool((wg == 7.0).all())
    xr, wr, dr = np64(x), np64(w), np64(dy)
    for e, a, b in ((0, 0, 20), (3, 40, 50)):
        assert (np.abs(np64(dw)[e] - xr[a:b].T @ dr[a:b]) <= (b - a) * U * (np.abs(xr[a:b]).T @ np.abs(dr[a:b]))).all()
    # rows 12..19 belong to two of these groups; the others to one
    for e, a, b in ((0, 0, 12), (2, 20, 40), (3, 40, 50)):
        assert (np.abs(np64(y)[a:b] - xr[a:b] @ wr[e]) <= H * U * (np.abs(xr[a:b]) @ np.abs(wr[e]))).all()
    assert bool((dw[1] == 0).all()) and bool((dw[4] == 0).all())


def test_gradient_without_rows_is_zero():
    for dtype, out in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        dw, guard = guarded((3, 40, 24), FMT[out][1], 7.0)
        cu = torch.zeros(4, dtype=torch.int32, device=DEV)
        moe.moe_grouped_matmul_wgrad(None, None, FMT[dtype][0], cu, 0, 3, 40, 24, dw, FMT[out][0], 0)
        torch.cuda.synchronize()
        assert bool((dw == 0).all()) and bool((guard == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,N", [(72, 40), (200, 264), (65, 33)])
def test_what_lies_next_to_a_group_stays_out(dtype, H, N):
    """NaN in the next expert's rows and weights, and in the columns past a tile, reaches no one else."""
    g = torch.Generator().manual_seed(4)
    d, t = FMT[dtype]
    counts = (70, 9, 300)
    cu, cud = offsets(counts)
    M, E = int(cu[-1]), 3
    for transposed in (0, 1):
        x, dy = values(g, (M, H), t), values(g, (M, N), t)
        w = values(g, (E, N, H) if transposed else (E, H, N), t)
        x[70:79], w[1], dy[70:79] = float("nan"), float("inf"), float("nan")
        y = torch.empty(M, N, dtype=t, device=DEV)
        moe.moe_grouped_matmul(x, d, None, 0, 0, cud, M, E, H, N, w, d, transposed, y, d)
        dw = torch.empty(E, H, N, device=DEV)
        moe.moe_grouped_matmul_wgrad(x, dy, d, cud, M, E, H, N, dw, moe.MOE_F32, 0)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(y[:70].float()).all()) and bool(torch.isfinite(y[79:].float()).all())
        assert bool(torch.isnan(y[70:79].float()).all())
        assert bool(torch.isfinite(dw[0]).all()) and bool(torch.isfinite(dw[2]).all()) and bool(torch.isnan(dw[1]).all())
