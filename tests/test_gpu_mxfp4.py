"""MXFP4 quantisation (bit for bit against the oracle) and the FFN with both operands in MXFP4.

The products are exact in fp32 and their sums err by at most K 2^-24 of the sum of their
magnitudes, which bounds g, u and y elementwise (delta below). h = silu(g) u then lies within
delta_h = 1.1 delta_g |u| + |silu(g)| delta_u + 16 * 2^-24 |h| (|silu'| <= 1.1; silu by the hardware's
exponential and reciprocal). Rounding is monotone, so a stored h code must lie between the codes
of h - delta_h and h + delta_h, under a scale byte between those of the block's largest
magnitude -+ delta_h. y is checked against the product of the h that the device stored, plus the one bf16
rounding, 2^-8 of its value."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_counting_amd as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FMT = {"f32": (moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, torch.bfloat16)}


def edge_values(rng, R, C):
    """Blocks of every kind: ordinary, huge, tiny, subnormal, zero, ties, with NaN or infinity."""
    x = rng.standard_normal((R, C // 32, 32))
    x *= np.exp2(rng.integers(-30, 30, (R, C // 32, 1)).astype(np.float64))
    kind = rng.integers(0, 10, (R, C // 32))
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.25, 1.5, 1.75, 2.5, 3.5, 5.0, 5.5, 6.0, 7.5])
    x[kind == 1] = 0.0
    ties = rng.choice(grid, x.shape) * rng.choice([-1, 1], x.shape) * np.exp2(rng.integers(-100, 100, kind.shape)[..., None].astype(float))
    x[kind == 2] = ties[kind == 2]
    x[kind == 3] *= 2.0 ** -140
    x[kind == 4] = rng.choice([0.0, -0.0, 3e38, -1e38], x[kind == 4].shape)
    spot = rng.integers(0, 32, kind.shape)
    for k, v in ((5, np.nan), (6, np.inf), (7, -np.inf)):
        at = np.argwhere(kind == k)
        for r, b in at[: max(1, len(at) // 4)]:
            x[r, b, spot[r, b]] = v
    return x.reshape(R, C)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 32), (1, 7168), (3, 96), (37, 160), (256, 512), (501, 1120)])
def test_quantize_rows_and_back(R, C, dtype):
    x = edge_values(np.random.default_rng(R + C), R, C)
    xt = torch.from_numpy(x.astype(np.float32)).to(DEV).to(FMT[dtype][1])
    q = torch.full((R, C // 2), 0x55, dtype=torch.uint8, device=DEV)
    sf = torch.full((R, C // 32), 0x55, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4(xt, FMT[dtype][0], R, C, q, sf)
    torch.cuda.synchronize()
    rq, rsf = O.quantize_mxfp4(xt.float().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), rsf)
    # a negative value that rounds to zero keeps its sign in the code; both decode to zero
    assert np.array_equal(q.cpu().numpy(), rq)
    ref = O.decode_mxfp4_rows(rq, rsf)
    for out in FMT:
        v = torch.full((R, C), 9.0, dtype=FMT[out][1], device=DEV)
        moe.moe_dequantize_mxfp4(q, sf, R, C, v, FMT[out][0])
        torch.cuda.synchronize()
        assert np.array_equal(v.float().cpu().numpy().astype(np.float64), ref, equal_nan=True)


def test_quantize_every_bf16_value():
    """Each bf16 bit pattern next to a block maximum of its own scale and of larger ones."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).float()
    rows = []
    for mult in (1.0, 1.5, 3.0, 8.0):
        b = v.view(-1, 1).repeat(1, 32)
        b[:, 1:] = 0
        b[:, 1] = (v * mult).to(torch.bfloat16).float()
        rows.append(b)
    x = torch.cat(rows).to(torch.bfloat16).to(DEV)
    R = x.shape[0]
    q = torch.empty(R, 16, dtype=torch.uint8, device=DEV)
    sf = torch.empty(R, 1, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4(x, moe.MOE_BF16, R, 32, q, sf)
    torch.cuda.synchronize()
    rq, rsf = O.quantize_mxfp4(x.float().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), rsf) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,K,N", [(1, 32, 1), (2, 64, 3), (3, 128, 4), (1, 96, 7), (2, 160, 9), (2, 256, 40),
                                   (3, 384, 66), (1, 1152, 301), (2, 512, 130)])
def test_quantize_weights_and_back(E, K, N, dtype):
    w = np.stack([edge_values(np.random.default_rng(E * K + N + e), N, K).T for e in range(E)])
    wt = torch.from_numpy(w.astype(np.float32)).to(DEV).to(FMT[dtype][1]).contiguous()
    stored = wt.float().cpu().numpy()
    ref = [O.quantize_mxfp4(stored[e].T) for e in range(E)]
    rq = np.stack([r[0] for r in ref])
    rsf = np.stack([r[1].T for r in ref])
    q = torch.full((E, N, K // 2), 0x55, dtype=torch.uint8, device=DEV)
    sf = torch.full((E, K // 32, N), 0x55, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4_weights(wt, FMT[dtype][0], E, K, N, moe.MOE_MXFP4, q, sf)
    torch.cuda.synchronize()
    assert np.array_equal(sf.cpu().numpy(), rsf) and np.array_equal(q.cpu().numpy(), rq)
    values = np.stack([O.decode_mxfp4(rq[e], rsf[e]) for e in range(E)])
    layouts = [(moe.MOE_MXFP4, q)]
    if K % 128 == 0 and N % 2 == 0:
        packed = torch.empty_like(q)
        moe.moe_pack_mxfp4_pairs(q, packed, E, N, K)
        direct = torch.full_like(q, 0x55)
        sf2 = torch.full_like(sf, 0x55)
        moe.moe_quantize_mxfp4_weights(wt, FMT[dtype][0], E, K, N, moe.MOE_MXFP4_PAIRED, direct, sf2)
        torch.cuda.synchronize()
        assert torch.equal(direct, packed) and torch.equal(sf, sf2)
        layouts.append((moe.MOE_MXFP4_PAIRED, direct))
    for layout, codes in layouts:
        for out in FMT:
            v = torch.full((E, K, N), 9.0, dtype=FMT[out][1], device=DEV)
            moe.moe_dequantize_mxfp4_weights(codes, sf, layout, E, K, N, v, FMT[out][0])
            torch.cuda.synchronize()
            assert np.array_equal(v.float().cpu().numpy().astype(np.float64), values, equal_nan=True)


# ----------------------------------------------------------------------------- the FFN

def codes(rng, *shape):
    return rng.integers(0, 256, shape).astype(np.uint8)


def scales(rng, K, *shape):
    b = 127 + int(np.floor(np.log2(2.0 / np.sqrt(K)))) - 2
    return (b + rng.integers(-1, 2, shape)).astype(np.uint8)


class Case:
    """Random codes and scales for the given rows per expert."""

    def __init__(self, counts, H, Hp, T=40, K=3, pad=(), tail=5, seed=0):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.Hp, self.T, self.K = len(counts), H, Hp, T, K
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        self.M = self.rows + tail
        self.src = rng.integers(0, T * K, self.M).astype(np.int32)
        for r in pad:
            self.src[r] = -1
        self.x_q, self.x_sf = codes(rng, T, H // 2), (127 + rng.integers(-4, 3, (T, H // 32))).astype(np.uint8)
        E = self.E
        self.wg, self.wu, self.wd = codes(rng, E, Hp, H // 2), codes(rng, E, Hp, H // 2), codes(rng, E, H, Hp // 2)
        self.sg, self.su, self.sd = scales(rng, H, E, H // 32, Hp), scales(rng, H, E, H // 32, Hp), scales(rng, Hp, E, Hp // 32, H)

    def gpu(self):
        self.d = {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in vars(self).items()
                  if isinstance(v, np.ndarray)}
        return self

    def gate_up(self, gathered=True):
        d = self.d
        h_q = torch.full((self.M, self.Hp // 2), 0x33, dtype=torch.uint8, device=DEV)
        h_sf = torch.full((self.M, self.Hp // 32), 0x33, dtype=torch.uint8, device=DEV)
        if gathered:
            x_q, x_sf, src = d["x_q"], d["x_sf"], d["src"]
        else:
            tok = (d["src"].clamp(min=0) // self.K).long()
            x_q, x_sf, src = d["x_q"][tok].contiguous(), d["x_sf"][tok].contiguous(), None
            x_q[d["src"] < 0] = 0
        moe.moe_ffn_gate_up_mxfp4(x_q, x_sf, src, self.T, self.K, d["cu"], self.M, self.E, self.H, self.Hp, d["wg"],
                                  d["wu"], d["sg"], d["su"], h_q, h_sf)
        torch.cuda.synchronize()
        return h_q, h_sf

    def down(self, h_q, h_sf):
        d = self.d
        y = torch.full((self.M, self.H), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_ffn_down_mxfp4(h_q, h_sf, d["cu"], self.M, self.E, self.H, self.Hp, d["wd"], d["sd"], y)
        torch.cuda.synchronize()
        return y

    def grouped(self):
        d = self.d
        y = torch.full((self.M, self.H), 7.0, dtype=torch.bfloat16, device=DEV)
        n = moe.moe_grouped_ffn_mxfp4_workspace_bytes(self.M, self.Hp)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        moe.moe_grouped_ffn_mxfp4(d["x_q"], d["x_sf"], d["src"], self.T, self.K, d["cu"], self.M, self.E, self.H, self.Hp,
                                  d["wg"], d["wu"], d["wd"], d["sg"], d["su"], d["sd"], y, ws, n)
        torch.cuda.synchronize()
        return y

    def check_h(self, h_q, h_sf):
        h_q, h_sf = h_q.cpu().numpy(), h_sf.cpu().numpy()
        assert (h_q[self.rows:] == 0x33).all() and (h_sf[self.rows:] == 0x33).all()   # rows behind the last group
        x = O.decode_mxfp4_rows(self.x_q, self.x_sf)
        for e in range(self.E):
            lo, hi = self.cu[e], self.cu[e + 1]
            if lo == hi:
                continue
            src = self.src[lo:hi]
            xr = np.where((src >= 0)[:, None], x[np.maximum(src, 0) // self.K], 0.0)
            wg, wu = O.decode_mxfp4(self.wg[e], self.sg[e]), O.decode_mxfp4(self.wu[e], self.su[e])
            g, u = xr @ wg, xr @ wu
            dg, du = (np.abs(xr) @ np.abs(w) * self.H * U for w in (wg, wu))
            h = O.silu(g) * u
            dh = 1.1 * dg * np.abs(u) + (np.abs(O.silu(g)) + 1.1 * dg) * du + 16 * U * np.abs(h)
            shape = (hi - lo, self.Hp // 32, 32)
            byte = h_sf[lo:hi].astype(int)
            a, d = np.abs(h).reshape(shape), dh.reshape(shape)
            b_lo = O.mxfp4_scale_byte(np.maximum(a - d, 0).max(axis=2)).astype(int)
            b_hi = O.mxfp4_scale_byte((a + d).max(axis=2)).astype(int)
            assert ((b_lo <= byte) & (byte <= b_hi)).all(), f"expert {e}: scale bytes"
            X = np.exp2(byte - 127.0)[:, :, None]
            got = O.decode_mxfp4_rows(h_q[lo:hi], h_sf[lo:hi]).reshape(shape) / X
            low = O.decode_e2m1(O.round_e2m1((h - dh).reshape(shape) / X))
            high = O.decode_e2m1(O.round_e2m1((h + dh).reshape(shape) / X))
            bad = ~((low <= got) & (got <= high))
            assert not bad.any(), f"expert {e}: {bad.sum()} codes, first at {np.argwhere(bad)[0]}"

    def check_y(self, y, h_q, h_sf):
        y = y.float().cpu().numpy().astype(np.float64)
        assert (y[self.rows:] == 7.0).all()
        h = O.decode_mxfp4_rows(h_q.cpu().numpy()[:self.rows], h_sf.cpu().numpy()[:self.rows])
        for e in range(self.E):
            lo, hi = self.cu[e], self.cu[e + 1]
            wd = O.decode_mxfp4(self.wd[e], self.sd[e])
            ref = h[lo:hi] @ wd
            tol = np.abs(h[lo:hi]) @ np.abs(wd) * self.Hp * U + 2.0 ** -8 * np.abs(ref)
            assert (np.abs(y[lo:hi] - ref) <= tol).all(), f"expert {e}"

    def check(self):
        h = self.gate_up()
        self.check_h(*h)
        y = self.down(*h)
        self.check_y(y, *h)
        plain = self.gate_up(gathered=False)
        assert torch.equal(h[0], plain[0]) and torch.equal(h[1], plain[1])
        assert torch.equal(y.view(torch.int16), self.grouped().view(torch.int16))


SHAPES = [
    ([1], 128, 128, ()),
    ([0, 1, 0, 2], 256, 128, ()),
    ([5, 0, 31, 32, 33], 384, 256, (3, 9, 40)),
    ([16, 17, 15, 0, 1, 64, 65], 512, 384, ()),
    ([255, 256, 257, 0, 300], 256, 384, (0, 260, 1000)),
    ([700, 3, 129], 640, 128, ()),
    ([130, 190], 1152, 640, ()),
    ([40] * 12, 128, 256, tuple(range(0, 480, 7))),
]


@pytest.mark.parametrize("counts,H,Hp,pad", SHAPES, ids=lambda s: "_".join(map(str, s[:8])) if isinstance(s, (list, tuple)) else str(s))
def test_ffn_mxfp4(counts, H, Hp, pad):
    print(f"[case] rows {counts} H={H} Hp={Hp}", flush=True)
    Case(counts, H, Hp, pad=pad, seed=H + Hp).gpu().check()


def test_ffn_mxfp4_many_experts_few_rows():
    rng = np.random.default_rng(0)
    Case(list(rng.integers(0, 4, 200)), 256, 128, seed=1).gpu().check()


def test_ffn_mxfp4_no_rows():
    c = Case([0, 0, 0], 256, 128, tail=6).gpu()
    h = c.gate_up()
    y = c.down(*h)
    assert (h[0] == 0x33).all() and (h[1] == 0x33).all() and (y == 7.0).all()


def test_ffn_mxfp4_nan_scale_stays_in_its_row():
    """A row whose activations hold a NaN block gives NaN, its neighbours are untouched."""
    c = Case([20, 150], 384, 256, seed=9)
    clean = Case([20, 150], 384, 256, seed=9).gpu()
    t = int(c.src[4]) // c.K
    c.x_sf[t, 11] = 255
    c.x_q[t, 11 * 16:12 * 16] = 0
    c.gpu()
    h, h0 = c.gate_up(), clean.gate_up()
    y, y0 = c.down(*h), clean.down(*h0)
    hit = torch.from_numpy(c.src[:c.rows] // c.K == t).to(DEV)
    rest = ~hit
    assert (h[1][:c.rows][hit] == 255).all()
    assert torch.isnan(y[:c.rows][hit]).all()
    assert torch.equal(h[0][:c.rows][rest], h0[0][:c.rows][rest])
    assert torch.equal(y[:c.rows][rest].view(torch.int16), y0[:c.rows][rest].view(torch.int16))


@pytest.mark.parametrize("H,Hp", [(2048, 128), (1920, 256), (1152, 640), (128, 2304), (640, 1152)])
def test_ffn_mxfp4_several_tiles_per_block(H, Hp):
    """More tiles than CUs in one or both halves: a block goes on to its next tile while its stores are under
    way, after whole and partial row blocks and after reductions of one, two and more stages."""
    rng = np.random.default_rng(H)
    counts = [int(c) for c in rng.integers(0, 300, 60)]
    counts[:8] = [256, 32, 96, 128, 160, 255, 1, 0]
    print(f"[case] rows {counts[:12]}.. H={H} Hp={Hp}", flush=True)
    c = Case(counts, H, Hp, T=64, seed=Hp).gpu()
    c.check()
    h = c.gate_up()
    y = c.down(*h)
    for _ in range(3):
        again = c.gate_up()
        assert torch.equal(h[0], again[0]) and torch.equal(h[1], again[1])
        assert torch.equal(y.view(torch.int16), c.down(*again).view(torch.int16))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,K,N", [(3, 384, 1030), (2, 2176, 514), (1, 128, 4102), (2, 896, 1022), (5, 128, 2048), (1, 160, 2047),
                                   (9, 1152, 8)])
def test_quantize_weights_in_many_blocks(E, K, N, dtype):
    """Matrices of several blocks along either axis, rows that end on whole lines and rows that do not."""
    test_quantize_weights_and_back(E, K, N, dtype)


@pytest.mark.parametrize("counts,H,Hp", [([3, 5, 0, 2], 256, 128), ([40, 300, 0, 130], 384, 256), ([100, 20], 128, 128)])
def test_ffn_mxfp4_padding_rows_beside_nan_weights(counts, H, Hp):
    """A weight block that holds NaN (scale byte 255) reaches every row of its expert, but not the padding rows:
    their h is zeros in both kernels (few rows: streamed, many: tiles)."""
    rows = sum(counts)
    pad = tuple(range(1, rows, 3))
    c = Case(counts, H, Hp, pad=pad, seed=rows)
    clean = Case(counts, H, Hp, pad=pad, seed=rows).gpu()
    for w, s in ((c.wg, c.sg), (c.wu, c.su)):
        s[0, 1, 70] = 255
        w[0, 70, 16:32] = 0
    c.sg[1, 2, 33] = 255
    c.wg[1, 33, 32:48] = 0
    c.gpu()
    h, h0 = c.gate_up(), clean.gate_up()
    src = torch.from_numpy(c.src[:rows]).to(DEV)
    for q, sf in (h, h0):
        assert not q[:rows][src < 0].any() and not sf[:rows][src < 0].any()
    expert = torch.from_numpy(np.repeat(np.arange(len(counts)), counts)).to(DEV)
    live = src >= 0
    blocks = {0: [70 // 32], 1: [33 // 32]}
    for e in range(len(counts)):
        at = (expert == e) & live
        for b in range(Hp // 32):
            if b in blocks.get(e, ()):
                assert (h[1][:rows][at][:, b] == 255).all()
            else:
                assert torch.equal(h[1][:rows][at][:, b], h0[1][:rows][at][:, b])
    assert not torch.isnan(c.down(*h)[:rows][~live].float()).any()


# Uneven small batches, which stream in both halves: experts with several chunks of 16 rows (at most 8 rows per
# expert on average) or of 32 (more).
UNEVEN = [
    ([70, 0, 1, 0, 17, 0, 0, 3, 0, 0, 0, 0], 384, 128, (2, 69, 80)),
    ([100, 0, 33, 32, 1, 0, 0, 0, 0, 0, 0, 0], 512, 128, (0, 31, 99, 131)),
    ([0] * 7 + [64], 640, 256, ()),
    ([0] * 7 + [120], 1152, 128, (64, 65)),
    ([0, 0, 0, 40] + [0] * 60 + [1, 16, 17] + [0] * 80 + [50, 0, 0], 256, 128, (41, 123)),
]


@pytest.mark.parametrize("counts,H,Hp,pad", UNEVEN, ids=lambda s: "_".join(map(str, s[:5])) if isinstance(s, (list, tuple)) else str(s))
def test_ffn_mxfp4_uneven_small_batches(counts, H, Hp, pad):
    print(f"[case] rows {counts[:12]}.. H={H} Hp={Hp}", flush=True)
    Case(counts, H, Hp, pad=pad, seed=len(counts)).gpu().check()


@pytest.mark.parametrize("counts", [[9, 0, 3, 1], [0, 50, 3, 0, 0, 0]])
def test_ffn_mxfp4_nan_scale_stays_in_its_row_streamed(counts):
    rows = sum(counts)
    c = Case(counts, 384, 128, seed=4)
    clean = Case(counts, 384, 128, seed=4).gpu()
    t = int(c.src[5]) // c.K
    c.x_sf[t, 7] = 255
    c.x_q[t, 7 * 16:8 * 16] = 0
    c.gpu()
    h, h0 = c.gate_up(), clean.gate_up()
    y, y0 = c.down(*h), clean.down(*h0)
    hit = torch.from_numpy(c.src[:rows] // c.K == t).to(DEV)
    assert (h[1][:rows][hit] == 255).all() and torch.isnan(y[:rows][hit]).all()
    assert torch.equal(h[0][:rows][~hit], h0[0][:rows][~hit]) and torch.equal(h[1][:rows][~hit], h0[1][:rows][~hit])
    assert torch.equal(y[:rows][~hit].view(torch.int16), y0[:rows][~hit].view(torch.int16))


def median_us(call, calls=5, times=7):
    call()
    got = []
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            call()
        b.record()
        torch.cuda.synchronize()
        got.append(a.elapsed_time(b) * 1e3 / calls)
    return sorted(got)[times // 2]


def test_ffn_mxfp4_a_heavy_expert_does_not_serialise_a_small_batch():
    """2048 rows on one of 64 experts read one expert's weights, not 64: they may not take many times the evenly
    spread batch's time (one block per column panel took 54 times)."""
    H, Hp, E, M = 7168, 128, 64, 2048
    us = []
    for counts in ([M // E] * E, [0] * 40 + [M] + [0] * (E - 41)):
        c = Case(counts, H, Hp, T=M, K=1, tail=0).gpu()
        d = c.d
        h_q = torch.empty(M, Hp // 2, dtype=torch.uint8, device=DEV)
        h_sf = torch.empty(M, Hp // 32, dtype=torch.uint8, device=DEV)
        us.append(median_us(lambda: moe.moe_ffn_gate_up_mxfp4(d["x_q"], d["x_sf"], d["src"], M, 1, d["cu"], M, E, H, Hp, d["wg"],
                                                              d["wu"], d["sg"], d["su"], h_q, h_sf)))
    print(f"[time] even {us[0]:.1f} us, one expert {us[1]:.1f} us", flush=True)
    assert us[1] <= 6 * us[0]


@pytest.mark.parametrize("E,Hp", [(256, 128), (16, 2048)])
def test_ffn_mxfp4_fewer_rows_do_not_take_longer(E, Hp):
    """As many tiles as CUs, 16 and 17 rows per expert: whichever kernel takes them, one row less per expert may not
    cost more (streamed, the 16 took 1.6 times the 17's time)."""
    H, us = 7168, []
    for r in (16, 17):
        M = E * r
        c = Case([r] * E, H, Hp, T=M, K=1, tail=0).gpu()
        d = c.d
        h_q = torch.empty(M, Hp // 2, dtype=torch.uint8, device=DEV)
        h_sf = torch.empty(M, Hp // 32, dtype=torch.uint8, device=DEV)
        us.append(median_us(lambda: moe.moe_ffn_gate_up_mxfp4(d["x_q"], d["x_sf"], d["src"], M, 1, d["cu"], M, E, H, Hp, d["wg"],
                                                              d["wu"], d["sg"], d["su"], h_q, h_sf)))
    print(f"[time] 16 rows {us[0]:.1f} us, 17 rows {us[1]:.1f} us", flush=True)
    assert us[0] <= 1.25 * us[1]
