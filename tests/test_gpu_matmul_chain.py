"""The INT8 and grouped products as they are used: in chains with routing, permutation and combine, forwards and
backwards; captured into HIP graphs and replayed; on other streams; at offsets past 32 bits; and at
sizes that reach every kernel (many tiles, few tiles, whole and partial ones)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_counting_amd as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF16, F32 = moe.MOE_BF16, moe.MOE_F32
FMT = {"f32": (F32, torch.float32), "bf16": (BF16, torch.bfloat16)}


def i32(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device=DEV)


def u8(n):
    return torch.full((max(int(n), 1),), 0x55, dtype=torch.uint8, device=DEV)


def np64(t):
    return t.detach().double().cpu().numpy()


class Int8Layer:
    """route -> permute -> quantise -> INT8 experts -> combine, with a dense INT8 projection of the tokens added; every
    buffer allocated once."""

    def __init__(self, T, E, K, H, Hp, pad=1, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.T, self.E, self.K, self.H, self.Hp, self.pad = T, E, K, H, Hp, pad
        self.M = moe.moe_padded_capacity(T, E, K, pad)
        self.d = moe.RouteDesc(T, E, K, moe.MOE_SCORE_SIGMOID, 1, 1, 1, 1, 2.5)
        self.logits = torch.randn(T, E, generator=g, device=DEV)
        self.x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        self.wq, self.ws = [], []
        for e, k, n in ((E, H, Hp), (E, H, Hp), (E, Hp, H), (1, H, H)):
            w = torch.randn(e, k, n, generator=g, device=DEV) / k ** 0.5
            q, s = torch.empty(e, n, k, dtype=torch.int8, device=DEV), torch.empty(e, n, device=DEV)
            moe.moe_quantize_int8_weights(w, F32, e, k, n, q, s)
            self.wq.append(q)
            self.ws.append(s)
        self.idx, self.w = i32(T, K), torch.empty(T, K, device=DEV)
        self.counts, self.cu, self.pos, self.src = i32(E), i32(E + 1), i32(T, K), i32(self.M)
        self.nperm = moe.moe_permute_workspace_bytes(T, E, K)
        self.perm_ws = u8(self.nperm)
        self.x_q, self.x_sf = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        self.nws = moe.moe_grouped_ffn_int8_workspace_bytes(self.M, Hp)
        self.ffn_ws = u8(self.nws)
        self.y = torch.zeros(self.M, H, dtype=torch.bfloat16, device=DEV)
        self.dense = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        self.out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)

    def run(self, stream=None):
        T, E, K, H, Hp, M = self.T, self.E, self.K, self.H, self.Hp, self.M
        moe.moe_route_scored(self.d, self.logits, F32, None, self.idx, self.w, stream)
        moe.moe_permute_padded(None, None, BF16, self.idx, self.w, T, H, E, K, self.pad, self.counts, self.cu, self.pos,
                               self.src, None, None, None, self.perm_ws, self.nperm, stream)
        moe.moe_quantize_int8(self.x, BF16, T, H, self.x_q, self.x_sf, stream)
        moe.moe_grouped_ffn_int8(self.x_q, self.x_sf, self.src, T, K, self.cu, M, E, H, Hp, *self.wq[:3], *self.ws[:3], self.y,
                                 self.ffn_ws, self.nws, stream)
        moe.moe_matmul_int8(self.x_q, self.x_sf, T, H, H, self.wq[3], self.ws[3], self.dense, BF16, stream)
        moe.moe_combine_shared(self.y, BF16, self.pos, self.w, T, H, K, self.dense, self.out, BF16, stream)
        return self.out

    def check(self):
        """From the stored codes in float64. h is rounded to bf16 and to codes of 1 / 127 of its row's largest: where the sums of
        fp32 and of float64 fall on two sides of a border a code differs by one. The relative noise of g, u and
        silu, 20 * 2^-24, moves fewer than 1 in 1000 codes (a border every 2^-8 of a value), each by a
        step of about 1 / 30 of h's root mean square: below 0.2 % of y in the 2-norm; y, the dense part and out add
        2^-9 / sqrt(3) each."""
        x = O.decode_int8(self.x_q.cpu().numpy(), self.x_sf.cpu().numpy())
        idx, w = self.idx.cpu().numpy(), np64(self.w)
        q, s = [t.cpu().numpy() for t in self.wq], [t.cpu().numpy() for t in self.ws]
        val = lambda i, e: O.decode_int8(q[i][e], s[i][e]).T  # noqa: E731
        ref = x @ val(3, 0)
        for e in range(self.E):
            t, k = np.nonzero(idx == e)
            if not len(t):
                continue
            g = x[t] @ val(0, e)
            h = torch.from_numpy(O.silu(g) * (x[t] @ val(1, e))).to(torch.bfloat16).double().numpy()
            np.add.at(ref, t, w[t, k][:, None] * (O.decode_int8(*O.quantize_int8(h)) @ val(2, e)))
        assert np.linalg.norm(np64(self.out) - ref) <= (0.002 + 3 * 2.0 ** -9) * np.linalg.norm(ref)


@pytest.mark.parametrize("T,E,K,H,Hp,pad", [(1, 8, 2, 256, 128, 1), (37, 16, 4, 512, 144, 1), (300, 12, 3, 272, 240, 1),
                                            (37, 16, 4, 512, 144, 8), (700, 5, 2, 512, 256, 32)])
def test_int8_layer(T, E, K, H, Hp, pad):
    c = Int8Layer(T, E, K, H, Hp, pad, seed=T)
    first = c.run().clone()
    c.check()
    assert torch.equal(c.run(), first)             # the same bits again


def test_int8_layer_with_a_poisoned_workspace(monkeypatch):
    c = Int8Layer(45, 9, 2, 256, 128, 4, seed=3)
    first = c.run().clone()
    monkeypatch.setenv("MOE_DEBUG_POISON", "1")
    assert torch.equal(c.run(), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,N", [(64, 40), (65, 33), (512, 8)])
def test_a_layer_of_single_projections_and_its_gradients(dtype, H, N):
    """out[t] = sum_k w_tk x_t . W[e_tk], and the gradients of x and W, against autograd in float64."""
    T, E, K = 83, 7, 3
    d, dt = FMT[dtype]
    g = torch.Generator().manual_seed(H)
    x, w = torch.randn(T, H, generator=g).to(dt), (torch.randn(E, H, N, generator=g) / H ** 0.5).to(dt)
    dout = torch.randn(T, N, generator=g).to(dt)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    tw = torch.rand(T, K, generator=g)
    xd, wd, doutd, idxd, twd = (t.to(DEV) for t in (x, w, dout, idx, tw))
    M = T * K
    counts, cu, pos, src, row_w = i32(E), i32(E + 1), i32(T, K), i32(M), torch.empty(M, device=DEV)
    n = moe.moe_permute_workspace_bytes(T, E, K)
    xp = torch.empty(M, H, dtype=dt, device=DEV)
    moe.moe_permute(xd, None, d, idxd, twd, T, H, E, K, counts, cu, pos, src, row_w, xp, None, u8(n), n)
    y, yg = torch.empty(M, N, dtype=dt, device=DEV), torch.empty(M, N, dtype=dt, device=DEV)
    moe.moe_grouped_matmul(xp, d, None, 0, 0, cu, M, E, H, N, wd, d, 0, y, d)
    moe.moe_grouped_matmul(xd, d, src, T, K, cu, M, E, H, N, wd, d, 0, yg, d)
    out = torch.empty(T, N, dtype=torch.float32, device=DEV)
    moe.moe_combine(y, d, pos, twd, T, N, K, out, F32)
    # backward: the rows' gradients, then the product's two gradients, then the copies of a token
    dy = (doutd[(src // K).long()].float() * row_w[:, None]).to(dt)
    dx_rows, dw = torch.empty(M, H, dtype=dt, device=DEV), torch.empty(E, H, N, device=DEV)
    moe.moe_grouped_matmul(dy, d, None, 0, 0, cu, M, E, N, H, wd, d, 1, dx_rows, d)
    moe.moe_grouped_matmul_wgrad(xp, dy, d, cu, M, E, H, N, dw, F32, 0)
    dx = torch.empty(T, H, dtype=torch.float32, device=DEV)
    moe.moe_combine(dx_rows, d, pos, None, T, H, K, dx, F32)
    torch.cuda.synchronize()
    assert torch.equal(y, yg)                      # gathered rows are the permuted ones
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    ref = sum(tw[:, k, None].double() * torch.bmm(x64[:, None], w64[idx[:, k].long()])[:, 0] for k in range(K))
    gx, gw = torch.autograd.grad((ref * dout.double()).sum(), (x64, w64))
    # rows round to the format (y; dy, then dx_rows): 2^-8 each for bf16; sums of H, N and counts products
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    for got, want, terms in ((out, ref, H), (dx, gx, N), (dw, gw, M)):
        err = np.abs(np64(got) - want.detach().numpy()).max()
        assert err <= (2 * eps * K + terms * U) * float(want.detach().abs().max()) * 4, err


def test_graph_replays():
    """Everything captured once; each replay, with new inputs and eager calls in between, gives the eager bits."""
    T, E, K, H, Hp = 33, 8, 2, 256, 128
    c = Int8Layer(T, E, K, H, Hp, seed=1)
    M = c.M
    g = torch.Generator(device=DEV).manual_seed(5)
    wb = torch.randn(E, H, Hp, generator=g, device=DEV).bfloat16()
    xp, dy = torch.randn(M, H, generator=g, device=DEV).bfloat16(), torch.randn(M, Hp, generator=g, device=DEV).bfloat16()
    yb, dxb = torch.empty(M, Hp, dtype=torch.bfloat16, device=DEV), torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
    dw = torch.zeros(E, H, Hp, device=DEV)
    back = torch.empty(T, H, device=DEV)

    def step():
        c.run()
        moe.moe_grouped_matmul(c.x, BF16, c.src, T, K, c.cu, M, E, H, Hp, wb, BF16, 0, yb, BF16)
        moe.moe_grouped_matmul(dy, BF16, None, 0, 0, c.cu, M, E, Hp, H, wb, BF16, 1, dxb, BF16)
        moe.moe_grouped_matmul_wgrad(xp, dy, BF16, c.cu, M, E, H, Hp, dw, F32, 1)
        moe.moe_dequantize_int8(c.x_q, c.x_sf, T, H, back, F32)
        return [t.clone() for t in (c.out, yb, dxb, dw, back)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        for t in (c.x, c.logits, xp, dy, wb):
            t.copy_(torch.randn(*t.shape, generator=g, device=DEV))
        before = dw.clone()
        want = step()
        dw.copy_(before)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        torch.zeros(1 << 20, device=DEV).sum()


def test_two_streams_at_once():
    a, b = Int8Layer(64, 8, 2, 512, 256, seed=1), Int8Layer(64, 8, 2, 512, 256, seed=2)
    wa, wb = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(5):
        a.out.zero_()
        b.out.zero_()
        s1.wait_stream(torch.cuda.current_stream())
        s2.wait_stream(torch.cuda.current_stream())
        a.run(s1)                                   # an explicit stream
        with torch.cuda.stream(s2):
            b.run()                                 # the current one
        torch.cuda.current_stream().wait_stream(s1)
        torch.cuda.current_stream().wait_stream(s2)
        assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


# ----------------------------------------------------------------------------- every kernel

def draw_rows(g, counts, H, N, dt, transposed):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(cu[-1]) + 3
    E = len(counts)
    w = torch.randn(E, *((N, H) if transposed else (H, N)), generator=g, device=DEV).to(dt)
    return cu, torch.from_numpy(cu).to(DEV), M, E, torch.randn(M, H, generator=g, device=DEV).to(dt), w


def spread(E, rows, seed):
    """Ragged groups of about `rows`, some of them empty."""
    r = np.random.default_rng(seed)
    c = r.integers(rows // 2, rows + rows // 2 + 1, E)
    c[r.integers(0, E, max(1, E // 6))] = 0
    return [int(v) for v in c]


BIG = [
    (spread(8, 3000, 1), 24, 520), (spread(8, 3000, 2), 64, 520), (spread(8, 3000, 3), 200, 520), (spread(8, 3000, 4), 199, 517),
    (spread(128, 100, 5), 24, 520), (spread(128, 100, 6), 136, 513), (spread(128, 100, 7), 133, 520), (spread(60, 700, 8), 320, 40),
    (spread(300, 12, 9), 256, 136), ([5000], 256, 1100),
]


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,H,N", BIG)
def test_many_tiles(counts, H, N, dtype, transposed):
    g = torch.Generator(device=DEV).manual_seed(H)
    d, dt = FMT[dtype]
    cu, cud, M, E, x, w = draw_rows(g, counts, H, N, dt, transposed)
    y = torch.full((M, N), 7.0, dtype=dt, device=DEV)
    moe.moe_grouped_matmul(x, d, None, 0, 0, cud, M, E, H, N, w, d, transposed, y, d)
    xd = x.double()
    assert bool((y[cu[-1]:] == 7.0).all())
    for e in range(E):
        a, b = int(cu[e]), int(cu[e + 1])
        if a == b:
            continue
        m = w[e].double().t() if transposed else w[e].double()
        ref = xd[a:b] @ m
        tol = H * U * (xd[a:b].abs() @ m.abs())
        if dtype == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert bool(((y[a:b].double() - ref).abs() <= tol).all()), e


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,H,N", [(c, h // 16 * 16 + 16, n) for c, h, n in BIG])
def test_many_tiles_int8(counts, H, N, out):
    g = torch.Generator(device=DEV).manual_seed(H)
    cu, cud, M, E, _, _ = draw_rows(g, counts, 1, 1, torch.float32, 0)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
    x, w, w2 = code(M, H), code(E, N, H), code(E, N, H)
    xs, ws, ws2 = (torch.rand(*s, generator=g, device=DEV) * 0.01 + 0.001 for s in ((M,), (E, N), (E, N)))
    d, dt = FMT[out]
    y = torch.full((M, N), 7.0, dtype=dt, device=DEV)
    moe.moe_grouped_matmul_int8(x, xs, None, 0, 0, cud, M, E, H, N, w, ws, y, d)
    h = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_ffn_gate_up_int8(x, xs, None, 0, 0, cud, M, E, H, N, w, w2, ws, ws2, h)
    assert bool((y[cu[-1]:] == 7.0).all()) and bool((h[cu[-1]:] == 7.0).all())
    xd = x.double()
    for e in range(E):
        a, b = int(cu[e]), int(cu[e + 1])
        if a == b:
            continue
        s = xs[a:b, None].double()
        ref = (xd[a:b] @ w[e].double().t()) * s * ws[e].double()
        tol = (3 * U + (2.0 ** -8 if out == "bf16" else 0)) * 1.01 * ref.abs()
        assert bool(((y[a:b].double() - ref).abs() <= tol).all()), e
        up = (xd[a:b] @ w2[e].double().t()) * s * ws2[e].double()
        act = ref * torch.sigmoid(ref)
        hr = act * up
        tol = (1.1 * 3.01 * U * ref.abs() * up.abs() + act.abs() * 3.01 * U * up.abs() + 16 * U * hr.abs()) * (1 + 2.0 ** -7)
        assert bool(((h[a:b].double() - hr).abs() <= tol + 2.0 ** -8 * hr.abs() + 2.0 ** -126).all()), e


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("counts,H,N", [(spread(9, 200, 1), 1100, 1104), (spread(9, 200, 2), 1104, 1096), ([0] * 3 + [90] + [0] * 6, 1104, 1024),
                                        (spread(40, 60, 3), 48, 2048), (spread(40, 60, 4), 47, 2047), (spread(30, 40, 5), 2048, 24),
                                        ([64] * 9, 1024, 1280), ([3000], 520, 264), (spread(9, 200, 6), 1099, 1101)])
def test_many_tiles_of_the_weight_gradient(counts, H, N, dtype, out, accumulate):
    if accumulate and out == "bf16":
        pytest.skip("refused: gradients are added in fp32")
    g = torch.Generator(device=DEV).manual_seed(N)
    d, dt = FMT[dtype]
    cu, cud, M, E, x, _ = draw_rows(g, counts, H, 1, dt, 0)
    dy = torch.randn(M, N, generator=g, device=DEV).to(dt)
    before = torch.randn(E, H, N, generator=g, device=DEV)
    dw = before.to(FMT[out][1]).clone()
    moe.moe_grouped_matmul_wgrad(x, dy, d, cud, M, E, H, N, dw, FMT[out][0], accumulate)
    for e in range(E):
        a, b = int(cu[e]), int(cu[e + 1])
        xr, dr = x[a:b].double(), dy[a:b].double()
        ref = xr.t() @ dr if b > a else torch.zeros(H, N, dtype=torch.float64, device=DEV)
        tol = (b - a) * U * (xr.abs().t() @ dr.abs()) if b > a else torch.zeros_like(ref)
        if accumulate:
            ref = ref + before[e].double()
            tol = tol * (1 + U) + U * ref.abs()
        if out == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert bool(((dw[e].double() - ref).abs() <= tol).all()), e


# ----------------------------------------------------------------------------- gathered rows, every kernel
#
# The rows of a group lie anywhere among T tokens, fewer than there are rows; some are padding (-1) or name a token that does
# not exist. A gathered product is the one of the permuted rows bit for bit: the same kernel and the same order of sums.

GATHERED = [
    (spread(8, 3000, 1), 24, 520), (spread(8, 3000, 3), 200, 520), (spread(8, 3000, 4), 199, 517),   # many rows, odd sizes
    ([9000, 3, 0, 700, 1, 0, 129, 5000], 72, 520), ([9000, 3, 0, 700, 1, 0, 129, 5000], 71, 264),    # uneven groups
    ([900, 1, 7000], 136, 1032), ([900, 1, 7000], 65, 1031), ([30] * 3 + [4000], 64, 1160),
    (spread(128, 100, 5), 24, 520), (spread(128, 100, 6), 136, 513), (spread(128, 100, 7), 133, 520),
    (spread(60, 700, 8), 320, 40), (spread(60, 700, 9), 333, 33), ([130, 0, 70, 257], 1032, 72), ([130, 0, 70, 257], 1031, 71),
    (spread(300, 12, 9), 256, 136), ([5000], 256, 1100), ([33] * 40, 80, 200), ([2] * 90, 264, 104),
]


def draw_gather(g, rows, M, T, K):
    """row_src for M rows, and where each row lies (padding: -1)."""
    src = torch.randint(0, T * K, (M,), generator=g, device=DEV, dtype=torch.int32)
    src[2::11] = -1
    src[5::13] = torch.randint(T * K, T * K + 1000, (len(src[5::13]),), generator=g, device=DEV, dtype=torch.int32)
    src[rows:] = 2 ** 31 - 1                       # behind the last group: not looked at
    at = torch.where((src >= 0) & (src < T * K), src // K, -1).long()
    return src, at


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts,H,N", GATHERED)
def test_gathered_rows(counts, H, N, dtype, out, transposed):
    g = torch.Generator(device=DEV).manual_seed(H + N)
    d, dt = FMT[dtype]
    T, K = 301, 3
    cu, cud, M, E, _, w = draw_rows(g, counts, H, N, dt, transposed)
    rows = int(cu[-1])
    src, at = draw_gather(g, rows, M, T, K)
    x = torch.randn(T, H, generator=g, device=DEV).to(dt)
    permuted = x[at.clamp(min=0)] * (at >= 0)[:, None].to(dt)
    y, yp = (torch.full((M, N), 7.0, dtype=FMT[out][1], device=DEV) for _ in range(2))
    moe.moe_grouped_matmul(x, d, src, T, K, cud, M, E, H, N, w, d, transposed, y, FMT[out][0])
    moe.moe_grouped_matmul(permuted, d, None, 0, 0, cud, M, E, H, N, w, d, transposed, yp, FMT[out][0])
    assert torch.equal(y, yp) and bool((y[rows:] == 7.0).all())
    xd = permuted.double()
    for e in range(E):
        a, b = int(cu[e]), int(cu[e + 1])
        if a == b:
            continue
        m = w[e].double().t() if transposed else w[e].double()
        ref = xd[a:b] @ m
        tol = H * U * (xd[a:b].abs() @ m.abs())
        if out == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        assert bool(((y[a:b].double() - ref).abs() <= tol).all()), e


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,H,N", [(c, h // 16 * 16 + 16, n) for c, h, n in GATHERED])
def test_gathered_rows_int8(counts, H, N, out):
    g = torch.Generator(device=DEV).manual_seed(H + N)
    T, K = 301, 3
    cu, cud, M, E, _, _ = draw_rows(g, counts, 1, 1, torch.float32, 0)
    rows = int(cu[-1])
    src, at = draw_gather(g, rows, M, T, K)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
    x, w, w2 = code(T, H), code(E, N, H), code(E, N, H)
    xs, ws, ws2 = (torch.rand(*s, generator=g, device=DEV) * 0.01 + 0.001 for s in ((T,), (E, N), (E, N)))
    live = at >= 0
    xp, xsp = x[at.clamp(min=0)] * live[:, None].to(torch.int8), xs[at.clamp(min=0)] * live.float()
    d, dt = FMT[out]
    y, yp = (torch.full((M, N), 7.0, dtype=dt, device=DEV) for _ in range(2))
    h, hp = (torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_grouped_matmul_int8(x, xs, src, T, K, cud, M, E, H, N, w, ws, y, d)
    moe.moe_grouped_matmul_int8(xp, xsp, None, 0, 0, cud, M, E, H, N, w, ws, yp, d)
    moe.moe_ffn_gate_up_int8(x, xs, src, T, K, cud, M, E, H, N, w, w2, ws, ws2, h)
    moe.moe_ffn_gate_up_int8(xp, xsp, None, 0, 0, cud, M, E, H, N, w, w2, ws, ws2, hp)
    assert torch.equal(y, yp) and bool((y[rows:] == 7.0).all())
    assert torch.equal(h, hp) and bool((h[rows:] == 7.0).all())
    xd = xp.double()
    for e in range(E):
        a, b = int(cu[e]), int(cu[e + 1])
        if a == b:
            continue
        s = xsp[a:b, None].double()
        ref = (xd[a:b] @ w[e].double().t()) * s * ws[e].double()
        tol = (3 * U + (2.0 ** -8 if out == "bf16" else 0)) * 1.01 * ref.abs()
        assert bool(((y[a:b].double() - ref).abs() <= tol).all()), e
        up = (xd[a:b] @ w2[e].double().t()) * s * ws2[e].double()
        act = ref * torch.sigmoid(ref)
        hr = act * up
        tol = (1.1 * 3.01 * U * ref.abs() * up.abs() + act.abs() * 3.01 * U * up.abs() + 16 * U * hr.abs()) * (1 + 2.0 ** -7)
        assert bool(((h[a:b].double() - hr).abs() <= tol + 2.0 ** -8 * hr.abs() + 2.0 ** -126).all()), e
    # padding rows are zeros beside columns whose scale is NaN, the others of such a column NaN
    ws[:, 1::7], ws2[:, 2::7] = float("nan"), float("nan")
    moe.moe_grouped_matmul_int8(x, xs, src, T, K, cud, M, E, H, N, w, ws, y, d)
    moe.moe_ffn_gate_up_int8(x, xs, src, T, K, cud, M, E, H, N, w, w2, ws, ws2, h)
    for t in (y, h):
        assert bool((t[:rows][~live[:rows]] == 0).all()) and bool(torch.isnan(t[:rows][live[:rows]][:, 1::7]).all())
    assert bool(torch.isfinite(y[:rows, 0::7]).all()) and bool(torch.isfinite(h[:rows, 0::7]).all())


@pytest.mark.parametrize("T,E,K,H,Hp,pad", [(32, 52, 8, 512, 256, 1), (256, 52, 8, 272, 144, 1), (2000, 4, 2, 512, 512, 1),
                                            (8192, 4, 2, 256, 512, 32)])
def test_int8_layer_of_batches(T, E, K, H, Hp, pad):
    """Decode batches over many experts, and prefills whose gathered rows reach the larger tiles."""
    c = Int8Layer(T, E, K, H, Hp, pad, seed=T)
    first = c.run().clone()
    c.check()
    assert torch.equal(c.run(), first)


# ----------------------------------------------------------------------------- past 32 bits

def test_weights_past_4_gib():
    """The last expert's matrix begins beyond 2^32 bytes, for few rows and for many."""
    for rows in (3, 300):
        E, H, N = 150, 4096, 4096                  # bf16: 5.0 GB; INT8: 2.5 GB
        cu = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        cu[E] = rows
        g = torch.Generator(device=DEV).manual_seed(1)
        x = torch.randn(rows, H, generator=g, device=DEV).bfloat16()
        w = torch.zeros(E, H, N, dtype=torch.bfloat16, device=DEV)
        w[E - 1] = torch.randn(H, N, generator=g, device=DEV).bfloat16()
        y = torch.empty(rows, N, device=DEV)
        for t in (0, 1):
            moe.moe_grouped_matmul(x, BF16, None, 0, 0, cu, rows, E, H, N, w, BF16, t, y, F32)
            m = w[E - 1].double().t() if t else w[E - 1].double()
            assert bool(((y.double() - x.double() @ m).abs() <= H * U * (x.double().abs() @ m.abs())).all())
        dw = torch.full((E, H, N // 2), 3.0, device=DEV)   # 5.0 GB
        moe.moe_grouped_matmul_wgrad(x, x[:, :N // 2].contiguous(), BF16, cu, rows, E, H, N // 2, dw, F32, 0)
        ref = x.double().t() @ x[:, :N // 2].double()
        tol = rows * U * (x.double().abs().t() @ x[:, :N // 2].double().abs())
        assert bool(((dw[E - 1].double() - ref).abs() <= tol).all()) and bool((dw[:E - 1] == 0).all())


def test_int8_weights_past_4_gib():
    E, H, N = 300, 4096, 4096
    w = torch.zeros(E, H, N, dtype=torch.bfloat16, device=DEV)     # 10 GB
    g = torch.Generator(device=DEV).manual_seed(1)
    w[E - 1] = torch.randn(H, N, generator=g, device=DEV).bfloat16()
    q, s = torch.full((E, N, H), 5, dtype=torch.int8, device=DEV), torch.zeros(E, N, device=DEV)
    moe.moe_quantize_int8_weights(w, BF16, E, H, N, q, s)
    rq, rs = O.quantize_int8(w[E - 1].float().t().cpu().numpy())
    assert np.array_equal(q[E - 1].cpu().numpy(), rq) and np.array_equal(s[E - 1].cpu().numpy(), rs)
    assert bool((q[:E - 1] == 0).all()) and bool((s[:E - 1] == 1).all())
    moe.moe_dequantize_int8_weights(q, s, E, H, N, w, BF16)
    assert torch.equal(w[E - 1].cpu(), torch.from_numpy((rq * rs[:, None]).T).to(torch.bfloat16))
    for rows in (3, 300):
        cu = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        cu[E] = rows
        x = torch.randint(-127, 128, (rows, H), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
        y = torch.empty(rows, N, device=DEV)
        moe.moe_grouped_matmul_int8(x, torch.ones(rows, device=DEV), None, 0, 0, cu, rows, E, H, N, q, s, y, F32)
        ref = (x.double() @ q[E - 1].double().t()) * s[E - 1].double()
        assert bool(((y.double() - ref).abs() <= 3.01 * U * ref.abs()).all())


def test_rows_past_4_gib():
    """x, dy and y reach beyond 2^32 bytes; groups at both ends."""
    M, H, N = 300_000, 8192, 32
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.zeros(M, H, dtype=torch.bfloat16, device=DEV)
    x[-200:] = torch.randn(200, H, generator=g, device=DEV).bfloat16()
    cu = torch.tensor([0, 5, M - 150, M], dtype=torch.int32, device=DEV)
    w = torch.randn(3, H, N, generator=g, device=DEV).bfloat16()
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_matmul(x, BF16, None, 0, 0, cu, M, 3, H, N, w, BF16, 0, y, BF16)
    for a, b, e in ((M - 200, M - 150, 1), (M - 150, M, 2)):
        ref = x[a:b].double() @ w[e].double()
        tol = H * U * (x[a:b].double().abs() @ w[e].double().abs()) * 1.01 + 2.0 ** -8 * ref.abs()
        assert bool(((y[a:b].double() - ref).abs() <= tol).all())
    dy = torch.randn(M, N, generator=g, device=DEV).bfloat16()
    dw = torch.empty(3, H, N, device=DEV)
    moe.moe_grouped_matmul_wgrad(x, dy, BF16, cu, M, 3, H, N, dw, F32, 0)
    for a, b, e in ((M - 200, M - 150, 1), (M - 150, M, 2)):
        ref = x[a:b].double().t() @ dy[a:b].double()
        tol = (M if e == 1 else 150) * U * (x[a:b].double().abs().t() @ dy[a:b].double().abs())
        assert bool(((dw[e].double() - ref).abs() <= tol).all())
    # the other way round: a wide output
    wt = torch.randn(3, H, N, generator=g, device=DEV).bfloat16()
    moe.moe_grouped_matmul(dy, BF16, None, 0, 0, cu, M, 3, N, H, wt, BF16, 1, x, BF16)
    for a, b, e in ((0, 5, 0), (M - 170, M - 150, 1), (M - 150, M, 2)):
        m = wt[e].double().t()
        ref = dy[a:b].double() @ m
        tol = N * U * (dy[a:b].double().abs() @ m.abs()) * 1.01 + 2.0 ** -8 * ref.abs()
        assert bool(((x[a:b].double() - ref).abs() <= tol).all())


def test_quantised_rows_past_4_gib():
    R, C = 300_000, 16384                          # bf16: 9.8 GB, codes 4.9 GB
    x = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    x[-3:] = torch.randn(3, C, generator=g, device=DEV).bfloat16()
    q, s = torch.full((R, C), 5, dtype=torch.int8, device=DEV), torch.zeros(R, device=DEV)
    moe.moe_quantize_int8(x, BF16, R, C, q, s)
    rq, rs = O.quantize_int8(x[-3:].float().cpu().numpy())
    assert np.array_equal(q[-3:].cpu().numpy(), rq) and np.array_equal(s[-3:].cpu().numpy(), rs)
    assert bool((q[:1000] == 0).all()) and bool((s[:-3] == 1).all())
    moe.moe_dequantize_int8(q, s, R, C, x, BF16)
    assert torch.equal(x[-3:].cpu(), torch.from_numpy(rq * rs[:, None]).to(torch.bfloat16))
