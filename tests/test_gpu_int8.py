"""INT8 quantisation (bit for bit against the oracle) and the INT8 products.

The integer sums are exact, so a product differs from its definition by three fp32 roundings (conversion, row
scale, column scale): 3 * 2^-24 of its value, and the bf16 rounding of the output, 2^-8 of it. In
gate/up g and u carry those 3 * 2^-24; h = silu(g) u then lies within 1.1 delta_g |u| + |silu(g)| delta_u + 16 * 2^-24
|h| (|silu'| <= 1.1; silu by the hardware's exponential and reciprocal) before its rounding to bf16."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_counting_amd as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FMT = {"f32": (moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, torch.bfloat16)}
TINY = 2.0 ** -126   # results below the normal range keep an absolute error


def edge_rows(rng, R, C):
    """Rows of every kind: ordinary, huge, tiny, subnormal, zero, ties, with NaN or infinity."""
    x = rng.standard_normal((R, C)) * np.exp2(rng.integers(-40, 40, (R, 1)).astype(np.float64))
    kind = rng.integers(0, 10, R)
    x[kind == 1] = 0.0
    ties = rng.integers(-126, 127, (R, C)) + 0.5
    ties[:, 0] = 127.0
    ties *= np.exp2(rng.integers(-110, 100, (R, 1)).astype(np.float64))
    x[kind == 2] = ties[kind == 2]
    x[kind == 3] *= 2.0 ** -130
    x[kind == 4] = rng.choice([0.0, -0.0, 3e38, -1e38], (int((kind == 4).sum()), C))
    # next to a border: the odd multiples of half a scale, one fp32 step up or down
    near = ((rng.integers(-126, 127, (R, C)) + 0.5) * rng.uniform(0.5, 2.0, (R, 1)).astype(np.float32)).astype(np.float32)
    near = np.where(rng.random((R, C)) < 0.5, np.nextafter(near, np.float32(np.inf)), near)
    near[:, 0] = np.abs(near).max(axis=1) * 1.01
    x[kind == 5] = near[kind == 5]
    for k, v in ((6, np.nan), (7, np.inf), (8, -np.inf)):
        x[kind == k, rng.integers(0, C)] = v
    return x


def guarded(shape, dtype, fill):
    """A tensor with 64 elements of `fill` behind it."""
    n = int(np.prod(shape))
    buf = torch.full((n + 64,), fill, dtype=dtype, device=DEV)
    return buf[:n].view(*shape), buf[n:]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 7168), (3, 7), (70, 33), (37, 160), (65, 512), (129, 1000), (40, 1031),
                                 (33, 2048), (17, 4096), (19, 8192), (9, 8199), (5, 20011)])
def test_quantize_rows_and_back(R, C, dtype):
    x = edge_rows(np.random.default_rng(R + C), R, C)
    xt = torch.from_numpy(x.astype(np.float32)).to(FMT[dtype][1])
    q, qg = guarded((R, C), torch.int8, 0x55)
    sf, sg = guarded((R,), torch.float32, 9.0)
    moe.moe_quantize_int8(xt.to(DEV), FMT[dtype][0], R, C, q, sf)
    torch.cuda.synchronize()
    rq, rs = O.quantize_int8(xt.float().numpy())
    assert np.array_equal(sf.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert bool((qg == 0x55).all()) and bool((sg == 9.0).all())
    ref = torch.from_numpy(rq.astype(np.float32) * rs[:, None])
    for out in FMT:
        v, vg = guarded((R, C), FMT[out][1], 9.0)
        moe.moe_dequantize_int8(q, sf, R, C, v, FMT[out][0])
        torch.cuda.synchronize()
        assert np.array_equal(v.float().cpu().numpy(), ref.to(FMT[out][1]).float().numpy(), equal_nan=True)
        assert bool((vg == 9.0).all())


def test_quantize_rows_at_any_element():
    R, C = 37, 515
    for dtype in FMT:
        buf = torch.from_numpy(edge_rows(np.random.default_rng(5), 1, R * C + 1).astype(np.float32))[0]
        buf = torch.nan_to_num(buf, posinf=1.0, neginf=1.0).to(FMT[dtype][1]).to(DEV)
        x = buf[1:].view(R, C)
        qb = torch.empty(R * C + 3, dtype=torch.int8, device=DEV)
        q, sf = qb[3:].view(R, C), torch.empty(R, device=DEV)
        moe.moe_quantize_int8(x, FMT[dtype][0], R, C, q, sf)
        torch.cuda.synchronize()
        rq, rs = O.quantize_int8(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(sf.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (2, 64, 3), (3, 130, 5), (1, 96, 7), (2, 257, 65), (2, 256, 40), (3, 384, 66),
                                   (1, 1151, 301), (2, 512, 130), (1, 2048, 64)])
def test_quantize_weights_and_back(E, K, N, dtype):
    w = np.stack([edge_rows(np.random.default_rng(E * K + N + e), N, K).T for e in range(E)])
    wt = torch.from_numpy(w.astype(np.float32)).to(FMT[dtype][1]).contiguous()
    ref = [O.quantize_int8(m.T) for m in wt.float().numpy()]
    rq, rs = np.stack([r[0] for r in ref]), np.stack([r[1] for r in ref])
    q, qg = guarded((E, N, K), torch.int8, 0x55)
    sf, sg = guarded((E, N), torch.float32, 9.0)
    moe.moe_quantize_int8_weights(wt.to(DEV), FMT[dtype][0], E, K, N, q, sf)
    torch.cuda.synchronize()
    assert np.array_equal(sf.cpu().numpy(), rs, equal_nan=True) and np.array_equal(q.cpu().numpy(), rq)
    assert bool((qg == 0x55).all()) and bool((sg == 9.0).all())
    values = torch.from_numpy((rq.astype(np.float32) * rs[:, :, None]).transpose(0, 2, 1))
    for out in FMT:
        v, vg = guarded((E, K, N), FMT[out][1], 9.0)
        moe.moe_dequantize_int8_weights(q, sf, E, K, N, v, FMT[out][0])
        torch.cuda.synchronize()
        assert np.array_equal(v.float().cpu().numpy(), values.to(FMT[out][1]).float().numpy(), equal_nan=True)
        assert bool((vg == 9.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,N", [(1, 1), (3, 7), (2, 200)])
def test_weights_of_an_empty_reduction(E, N, dtype):
    """The largest magnitude of a column without values is 0: its scale is 1. Nothing else is read or written."""
    sf, sg = guarded((E, N), torch.float32, 9.0)
    moe.moe_quantize_int8_weights(None, FMT[dtype][0], E, 0, N, None, sf)
    moe.moe_dequantize_int8_weights(None, sf, E, 0, N, None, FMT[dtype][0])
    torch.cuda.synchronize()
    assert bool((sf == 1.0).all()) and bool((sg == 9.0).all())


# ----------------------------------------------------------------------------- products

class Groups:
    """Random codes and scales for the given rows per expert; `tail` rows behind the last group."""

    def __init__(self, counts, H, N, T=40, K=3, pad=(), tail=5, seed=0, mats=1):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.N, self.T, self.K = len(counts), H, N, T, K
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        self.M = self.rows + tail
        self.src = rng.integers(0, T * K, self.M).astype(np.int32)
        for r in pad:
            self.src[r] = -1
        self.x = rng.integers(-128, 128, (T, H)).astype(np.int8)
        self.xs = rng.uniform(0.5, 2.0, T).astype(np.float32) / 127
        self.w = [rng.integers(-128, 128, (self.E, N, H)).astype(np.int8) for _ in range(mats)]
        # products of a few units, where silu is neither linear nor flat
        self.ws = [(rng.uniform(0.5, 2.0, (self.E, N)) * 3 / (74 * np.sqrt(H))).astype(np.float32) for _ in range(mats)]
        self.dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
                    for k, v in dict(cu=self.cu, src=self.src, x=self.x, xs=self.xs).items()}
        self.wd = [torch.from_numpy(v).to(DEV) for v in self.w]
        self.wsd = [torch.from_numpy(v).to(DEV) for v in self.ws]

    def product(self, i, x, xs):
        """x [rows, H] codes in group order."""
        out = np.zeros((self.rows, self.w[i].shape[1]))
        for e in range(self.E):
            a, b = self.cu[e], self.cu[e + 1]
            if b > a:
                out[a:b] = (x[a:b].astype(np.float64) @ self.w[i][e].astype(np.float64).T) * self.ws[i][e].astype(np.float64)
        return out * xs[:, None].astype(np.float64)

    def gathered(self):
        at = self.src[:self.rows] // self.K
        live = self.src[:self.rows] >= 0
        return np.where(live[:, None], self.x[at], 0), np.where(live, self.xs[at], np.float32(0))


SHAPES = [
    ((1,), 16, 1), ((3, 0, 2), 48, 5), ((0, 0, 0), 64, 8), ((7, 1, 0, 33), 80, 24), ((16, 16, 17), 256, 40),
    ((1,) * 9, 528, 129), ((130, 64, 0, 5), 144, 136), ((257, 255), 400, 264), ((40, 300, 0, 511), 1024, 257),
    ((600,), 112, 520), ((2, 30, 31, 1), 2048, 384), ((0, 5, 0, 0, 9, 0), 7168, 48), ((8,) * 70, 256, 200),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,H,N", SHAPES)
def test_grouped_product(counts, H, N, out, gather):
    pad = tuple(range(2, sum(counts), 11)) if gather else ()
    c = Groups(counts, H, N, pad=pad, seed=H + N)
    y, yg = guarded((c.M, N), FMT[out][1], 7.0)
    if gather:
        x, xs = c.gathered()
        moe.moe_grouped_matmul_int8(c.dev["x"], c.dev["xs"], c.dev["src"], c.T, c.K, c.dev["cu"], c.M, c.E, H, N, c.wd[0],
                                    c.wsd[0], y, FMT[out][0])
    else:
        rng = np.random.default_rng(1)
        x = rng.integers(-128, 128, (c.M, H)).astype(np.int8)
        xs = rng.uniform(0.5, 2.0, c.M).astype(np.float32)
        moe.moe_grouped_matmul_int8(torch.from_numpy(x).to(DEV), torch.from_numpy(xs).to(DEV), None, 0, 0, c.dev["cu"], c.M,
                                    c.E, H, N, c.wd[0], c.wsd[0], y, FMT[out][0])
        x, xs = x[:c.rows], xs[:c.rows]
    torch.cuda.synchronize()
    ref = c.product(0, x, xs)
    got = y.double().cpu().numpy()
    tol = (3 * U + (2.0 ** -8 if out == "bf16" else 0)) * 1.01 * np.abs(ref)
    assert (np.abs(got[:c.rows] - ref) <= tol).all()
    assert (got[c.rows:] == 7.0).all() and bool((yg == 7.0).all())      # rows behind the groups stay


@pytest.mark.parametrize("M,H,N", [(1, 16, 1), (1, 7168, 2048), (2, 48, 7), (17, 4096, 96), (33, 256, 130), (64, 1040, 520),
                                   (300, 128, 300), (513, 784, 257), (1024, 512, 640)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_dense_product(M, H, N, out):
    rng = np.random.default_rng(M + H + N)
    x, w = rng.integers(-128, 128, (M, H)).astype(np.int8), rng.integers(-128, 128, (N, H)).astype(np.int8)
    xs, ws = rng.uniform(0.5, 2.0, M).astype(np.float32), rng.uniform(0.5, 2.0, N).astype(np.float32)
    y, yg = guarded((M, N), FMT[out][1], 7.0)
    moe.moe_matmul_int8(*[torch.from_numpy(v).to(DEV) for v in (x, xs)], M, H, N,
                        *[torch.from_numpy(v).to(DEV) for v in (w, ws)], y, FMT[out][0])
    torch.cuda.synchronize()
    ref = (x.astype(np.float64) @ w.T.astype(np.float64)) * xs[:, None].astype(np.float64) * ws.astype(np.float64)
    tol = (3 * U + (2.0 ** -8 if out == "bf16" else 0)) * 1.01 * np.abs(ref)
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all() and bool((yg == 7.0).all())


def test_the_largest_sum_fits():
    """All codes -128 at the longest reduction: 2^14 * 131056, just below 2^31."""
    for M in (3, 200):
        H, N = 2 ** 17 - 16, 130
        x = torch.full((M, H), -128, dtype=torch.int8, device=DEV)
        w = torch.full((N, H), -128, dtype=torch.int8, device=DEV)
        y = torch.empty(M, N, device=DEV)
        moe.moe_matmul_int8(x, torch.ones(M, device=DEV), M, H, N, w, torch.ones(N, device=DEV), y, moe.MOE_F32)
        torch.cuda.synchronize()
        assert bool((y == float(2 ** 14 * H)).all())          # 2^14 times a 17-bit number: exact in fp32


@pytest.mark.parametrize("M", [5, 200])
def test_scales_of_nan_zero_and_padding(M):
    """NaN rows and columns spread, rows of scale 0 and padding rows are zeros even against a NaN column."""
    H, N, E = 64, 72, 2
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.integers(-127, 128, (M, H)).astype(np.int8)).to(DEV)
    w = torch.from_numpy(rng.integers(-127, 128, (E, N, H)).astype(np.int8)).to(DEV)
    xs, ws = torch.ones(M, device=DEV), torch.ones(E, N, device=DEV)
    xs[1], xs[2], ws[:, 5] = float("nan"), 0.0, float("nan")
    src = torch.arange(M, dtype=torch.int32, device=DEV)
    src[3], src[4] = -1, M + 7                            # padding; a token that does not exist
    cu = torch.tensor([0, M - 1, M], dtype=torch.int32, device=DEV)
    y = torch.empty(M, N, device=DEV)
    moe.moe_grouped_matmul_int8(x, xs, src, M, 1, cu, M, E, H, N, w, ws, y, moe.MOE_F32)
    h = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_ffn_gate_up_int8(x, xs, src, M, 1, cu, M, E, H, N, w, w, ws, ws, h)
    torch.cuda.synchronize()
    for t in (y, h):
        t = t.float().cpu()
        assert bool(torch.isnan(t[1]).all()) and bool((t[2:5] == 0).all()) and bool(torch.isnan(t[0, 5]))
        assert bool(torch.isfinite(t[0, :5]).all())


@pytest.mark.parametrize("counts,H,Hp", [((3, 0, 2), 48, 16), ((7, 1, 0, 33), 80, 48), ((1,) * 9, 528, 144),
                                         ((130, 64, 0, 5), 144, 136), ((257, 255), 400, 272), ((300, 40), 1024, 130),
                                         ((0, 5, 0, 9), 7168, 64), ((2, 30, 31, 1), 2048, 384), ((8,) * 40, 256, 200)])
def test_gate_up(counts, H, Hp):
    c = Groups(counts, H, Hp, pad=tuple(range(2, sum(counts), 11)), seed=H + Hp, mats=2)
    h, hg = guarded((c.M, Hp), torch.bfloat16, 7.0)
    moe.moe_ffn_gate_up_int8(c.dev["x"], c.dev["xs"], c.dev["src"], c.T, c.K, c.dev["cu"], c.M, c.E, H, Hp, *c.wd, *c.wsd, h)
    torch.cuda.synchronize()
    x, xs = c.gathered()
    g, u = c.product(0, x, xs), c.product(1, x, xs)
    ref = O.silu(g) * u
    dg, du = 3.01 * U * np.abs(g), 3.01 * U * np.abs(u)
    tol = (1.1 * dg * np.abs(u) + np.abs(O.silu(g)) * du + 16 * U * np.abs(ref)) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ref)
    got = h.double().cpu().numpy()
    assert (np.abs(got[:c.rows] - ref) <= tol + TINY).all()
    assert (got[c.rows:] == 7.0).all() and bool((hg == 7.0).all())


@pytest.mark.parametrize("counts,H,Hp", [((3, 0, 2), 48, 16), ((7, 1, 0, 33), 80, 48), ((130, 64, 0, 5), 144, 144),
                                         ((257, 255), 400, 272), ((1, 0, 1, 1), 2048, 1024)])
def test_grouped_ffn(counts, H, Hp):
    """The halves against their own tests' references: h's codes from the stored h bit for bit, y from those codes."""
    c = Groups(counts, H, Hp, pad=(1,), seed=H + Hp, mats=2)
    rng = np.random.default_rng(9)
    wd = rng.integers(-127, 128, (c.E, H, Hp)).astype(np.int8)
    sd = rng.uniform(0.5, 2.0, (c.E, H)).astype(np.float32) / 127
    n = moe.moe_grouped_ffn_int8_workspace_bytes(c.M, Hp)
    ws, wg = guarded((n,), torch.uint8, 0x55)
    y, yg = guarded((c.M, H), torch.bfloat16, 7.0)
    moe.moe_grouped_ffn_int8(c.dev["x"], c.dev["xs"], c.dev["src"], c.T, c.K, c.dev["cu"], c.M, c.E, H, Hp, *c.wd,
                             torch.from_numpy(wd).to(DEV), *c.wsd, torch.from_numpy(sd).to(DEV), y, ws, n)
    h = torch.empty(c.M, Hp, dtype=torch.bfloat16, device=DEV)
    moe.moe_ffn_gate_up_int8(c.dev["x"], c.dev["xs"], c.dev["src"], c.T, c.K, c.dev["cu"], c.M, c.E, H, Hp, *c.wd, *c.wsd, h)
    torch.cuda.synchronize()
    hb = ws[:c.M * Hp * 2].view(torch.bfloat16).view(c.M, Hp)
    assert torch.equal(hb[:c.rows], h[:c.rows])
    o = (c.M * Hp * 2 + 255) // 256 * 256
    hq = ws[o:o + c.M * Hp].view(torch.int8).view(c.M, Hp).cpu().numpy()
    o += (c.M * Hp + 255) // 256 * 256
    hs = ws[o:o + c.M * 4].view(torch.float32).cpu().numpy()
    rq, rs = O.quantize_int8(h[:c.rows].float().cpu().numpy())
    assert np.array_equal(hq[:c.rows], rq) and np.array_equal(hs[:c.rows], rs)
    c.w, c.ws = [wd], [sd]
    ref = c.product(0, rq, rs)
    got = y.double().cpu().numpy()
    assert (np.abs(got[:c.rows] - ref) <= (3 * U + 2.0 ** -8) * 1.01 * np.abs(ref)).all()
    assert (got[c.rows:] == 7.0).all() and bool((yg == 7.0).all()) and bool((wg == 0x55).all())


@pytest.mark.parametrize("rows", [9, 400])
def test_padding_rows_of_the_ffn(rows):
    """Their h is zeros whatever the gate and up weights hold, and goes through the down product as a row of zeros: zeros, but
    NaN in a column of NaN scale. Rows beside them are not touched by it."""
    H, Hp, E, T = 64, 48, 2, 20
    g = torch.Generator(device=DEV).manual_seed(rows)
    code = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
    x, wg, wu, wd = code(T, H), code(E, Hp, H), code(E, Hp, H), code(E, H, Hp)
    xs, sg, su, sd = (torch.full(s, 0.01, device=DEV) for s in ((T,), (E, Hp), (E, Hp), (E, H)))
    src = torch.randint(0, T, (rows,), generator=g, device=DEV, dtype=torch.int32)
    src[1::4] = -1
    pad = (src < 0).cpu()
    cu = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    n = moe.moe_grouped_ffn_int8_workspace_bytes(rows, Hp)
    ws, y = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)

    def ffn():
        moe.moe_grouped_ffn_int8(x, xs, src, T, 1, cu, rows, E, H, Hp, wg, wu, wd, sg, su, sd, y, ws, n)
        torch.cuda.synchronize()
        return y.float().cpu()

    first = ffn()
    assert bool((first[pad] == 0).all()) and bool(torch.isfinite(first).all())
    sd[:, 5] = float("nan")
    out = ffn()
    assert bool(torch.isnan(out[:, 5]).all())
    keep = [c for c in range(H) if c != 5]
    assert torch.equal(out[:, keep], first[:, keep])
    sg[:, 3] = float("nan")                                # h of the other rows is NaN there, and their y everywhere
    out = ffn()
    assert bool((out[pad][:, keep] == 0).all()) and bool(torch.isnan(out[~pad]).all())
