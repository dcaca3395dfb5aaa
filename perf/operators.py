"""Routing by scores and the MXFP4 x MXFP4 expert FFN: inputs, one pass, and plain forms.

A case is one call (or the few calls that belong together) of a user's program:

* ``route``        scores -> top-k experts and their weights (``moe_route_scored``);
* ``route_train``  the same, then the gradient of the logits (``moe_route_scored_backward``);
* ``quant_rows``   activations to MXFP4 and back (``moe_quantize_mxfp4``, ``moe_dequantize_mxfp4``);
* ``quant_weights`` stacked expert weights to MXFP4 and back (``..._mxfp4_weights``);
* ``ffn``          the grouped SwiGLU expert FFN on MXFP4 rows and MXFP4 weights
  (``moe_grouped_ffn_mxfp4``).

``run`` calls the library where ``own`` is true and computes the plain torch form otherwise.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoded token of a 64-expert layer: latency
        dict(name="route_token", op="route", T=1, E=64, K=6, score="softmax", bias=False, groups=1,
             topk_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16", masked=False),
        # a prefill batch of the 384-expert layer, sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route_prefill", op="route", T=8192, E=384, K=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=False),
        # a training step's routing on the same layer
        dict(name="route_train_sigmoid", op="route_train", T=8192, E=384, K=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=False),
        # softmax scores kept unnormalised (a dense gradient), an odd padded batch, masked experts
        dict(name="route_train_softmax", op="route_train", T=4095, E=64, K=6, score="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, dtype="bf16", masked=True),
        # activations of one decoded token, and of a prefill batch
        dict(name="quant_token", op="quant_rows", R=1, C=7168, dtype="bf16"),
        dict(name="quant_prefill", op="quant_rows", R=8192, C=7168, dtype="bf16"),
        # loading weights: one projection of the 64-expert layer (fp32 master weights), and of an
        # expert-parallel rank's 52 slots
        dict(name="quant_weights_64", op="quant_weights", E=64, K=2048, N=1024, dtype="f32", paired=False),
        dict(name="quant_weights_52", op="quant_weights", E=52, K=7168, N=2048, dtype="bf16", paired=True),
        # one decoded token, a ragged middle-sized batch, the balanced rank at prefill, and the
        # whole 384-expert layer under skewed routing
        dict(name="ffn_token", op="ffn", T=1, E=52, K=8, H=7168, Hp=2048, skew=0.0),
        dict(name="ffn_64", op="ffn", T=4095, E=64, K=6, H=2048, Hp=1024, skew=0.0),
        dict(name="ffn_52", op="ffn", T=8192, E=52, K=8, H=7168, Hp=2048, skew=0.0),
        dict(name="ffn_384", op="ffn", T=8192, E=384, K=8, H=7168, Hp=2048, skew=0.2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route_train", "quant_rows", "quant_weights", "ffn", "ffn"])
    if op in ("route", "route_train"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = rng.randint(2, 384 // groups)
        E = groups * size
        topk_groups = rng.randint(1, groups)
        K = rng.randint(1, min(16, topk_groups * size))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, K=K, score=score, bias=rng.random() < 0.5,
                    groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.random() < 0.4)
    if op == "quant_rows":
        return dict(op=op, R=_log_int(rng, 1, 16384), C=32 * rng.randint(1, 256), dtype=rng.choice(["f32", "bf16"]))
    if op == "quant_weights":
        K, N = 128 * rng.randint(1, 56), 2 * rng.randint(1, 1024)
        return dict(op=op, E=_log_int(rng, 1, 52), K=K, N=N, dtype=rng.choice(["f32", "bf16"]),
                    paired=rng.random() < 0.5)
    H, Hp = 128 * rng.randint(2, 56), 128 * rng.randint(1, 16)
    E = rng.randint(1, 96)
    K = rng.randint(1, min(8, E))
    return dict(op=op, T=_log_int(rng, 1, 8192), E=E, K=K, H=H, Hp=Hp, skew=rng.choice([0.0, 0.3, 1.0]))


# ------------------------------------------------------------------------------- the inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


# The e2m1 magnitudes of the codes 0..7; bit 3 is the sign.
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _byte_table(dev, dtype):
    """[256, 2]: the values of a byte's low and high code."""
    half = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=dev)
    b = torch.arange(256, device=dev)
    return torch.stack([half[b & 15], half[b >> 4]], dim=1)


def _normal_codes(g, dev, shape):
    """Bytes of two codes each, drawn from 65536 pairs of block-scaled normal values."""
    # blocks of 32 normals scaled by their largest, as the format does: the codes' frequencies
    v = torch.randn(4096, 32, generator=g, device=dev)
    p = _code_of(v / _scale_of(v.abs().amax(dim=1, keepdim=True))).reshape(-1, 2)
    table = (p[:, 0] | (p[:, 1] << 4)).to(torch.uint8)
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.uint8, device=dev)
    step = 1 << 28
    for i in range(0, n, step):
        at = torch.randint(0, table.numel(), (min(step, n - i),), generator=g, device=dev, dtype=torch.int32)
        torch.index_select(table, 0, at, out=out[i:i + at.numel()])
    return out.view(shape)


def _scale_of(amax):
    """2^(floor(log2 amax) - 2), at least 2^-127 (an all-zero block: 2^-127)."""
    _, e = torch.frexp(amax)
    e = torch.where(amax > 0, e.to(torch.int32) - 3, torch.full_like(e, -127, dtype=torch.int32)).clamp(-127, 127)
    return torch.ldexp(torch.ones_like(amax), e)


def _code_of(v):
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    m = torch.clamp(torch.round(a / step) * step, max=6.0)
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.int32)
    return code | ((v < 0).to(torch.int32) << 3)


def _weight_scales(g, dev, E, K, N):
    # N(0, 1/K) weights: the largest of 32 is near 2.1 / sqrt(K), its exponent one of two
    b = 127 + math.floor(math.log2(2.1 / math.sqrt(K))) - 2
    return (b + torch.randint(0, 2, (E, K // 32, N), generator=g, device=dev, dtype=torch.int32)).to(torch.uint8)


def prepare(case, seed):
    dev = _device()
    g = _gen(dev, seed)
    s = {"case": case}
    if case["op"] in ("route", "route_train"):
        T, E, K = case["T"], case["E"], case["K"]
        l = torch.randn(T, E, generator=g, device=dev)
        if case["masked"]:
            # some experts switched off per token, written the three ways that programs write it,
            # and the padding rows of the batch switched off wholly
            u = torch.rand(T, E, generator=g, device=dev)
            low = torch.finfo(_DT[case["dtype"]]).min
            l = torch.where(u < 0.04, -math.inf, torch.where(u < 0.08, low, torch.where(u < 0.1, math.nan, l)))
            l[T - T // 16:] = -math.inf
        s["logits"] = l.to(_DT[case["dtype"]])
        spread = 0.1 if case["score"] == "sigmoid" else 0.3 / E
        s["bias"] = torch.randn(E, generator=g, device=dev) * spread if case["bias"] else None
        s["idx"] = torch.empty(T, K, dtype=torch.int32, device=dev)
        s["w"] = torch.empty(T, K, dtype=torch.float32, device=dev)
        if case["op"] == "route_train":
            s["d_w"] = torch.randn(T, K, generator=g, device=dev)
            s["d_logits"] = torch.empty(T, E, dtype=s["logits"].dtype, device=dev)
        return s
    if case["op"] == "quant_rows":
        R, C = case["R"], case["C"]
        s["x"] = torch.randn(R, C, generator=g, device=dev).to(_DT[case["dtype"]])
        s["q"] = torch.empty(R, C // 2, dtype=torch.uint8, device=dev)
        s["sf"] = torch.empty(R, C // 32, dtype=torch.uint8, device=dev)
        s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device=dev)
        return s
    if case["op"] == "quant_weights":
        E, K, N = case["E"], case["K"], case["N"]
        s["w"] = torch.empty(E, K, N, dtype=_DT[case["dtype"]], device=dev)
        for e in range(E):
            s["w"][e] = torch.randn(K, N, generator=g, device=dev) / math.sqrt(K)
        s["q"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
        s["sf"] = torch.empty(E, K // 32, N, dtype=torch.uint8, device=dev)
        s["values"] = torch.empty(E, K, N, dtype=torch.bfloat16, device=dev)
        return s
    T, E, K, H, Hp = (case[k] for k in ("T", "E", "K", "H", "Hp"))
    M = T * K
    x = torch.randn(T, H // 32, 32, generator=g, device=dev)
    X = _scale_of(x.abs().amax(dim=2, keepdim=True))
    c = _code_of(x / X).view(T, H // 2, 2)
    s["x_q"] = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)
    s["x_sf"] = (torch.frexp(X)[1].to(torch.int32) + 126).to(torch.uint8).view(T, H // 32)
    del x, X, c
    for name, k, n in (("gate", H, Hp), ("up", H, Hp), ("down", Hp, H)):
        s["w_" + name] = _normal_codes(g, dev, (E, n, k // 2))
        s["sf_" + name] = _weight_scales(g, dev, E, k, n)
    # the routing plan: copies grouped by expert, in the order of their flat index
    rank = torch.randperm(E, generator=g, device=dev).float()
    l = torch.randn(T, E, generator=g, device=dev) - case["skew"] * torch.log1p(rank)
    expert = torch.topk(l, K, dim=1).indices.reshape(-1)
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=E)
    s["row_src"] = order.to(torch.int32)
    s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), counts.cumsum(0)]).to(torch.int32)
    # for the plain form: the experts with rows, their largest group, each row's place there
    s["active"] = torch.nonzero(counts).view(-1)
    s["cap"] = int(counts.max())
    place = torch.zeros(E, dtype=torch.int64, device=dev)
    place[s["active"]] = torch.arange(s["active"].numel(), device=dev)
    by_row = expert[order]
    s["slot"] = place[by_row] * s["cap"] + torch.arange(M, device=dev) - s["cu"][by_row].long()
    s["y"] = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    s["ws"] = torch.empty(M * Hp // 2 + M * Hp // 32 + 4096, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "route":
        idx, w, _ = _plain_route(state)
        return idx, w
    if op == "route_train":
        return _plain_route_train(state)
    if op == "quant_rows":
        x = state["x"].float()
        return _plain_mx(x.view(x.shape[0], -1, 32), 2).view(x.shape).to(torch.bfloat16)
    if op == "quant_weights":
        w = state["w"].float()
        E, K, N = w.shape
        return _plain_mx(w.view(E, K // 32, 32, N), 2).view(E, K, N).to(torch.bfloat16)
    return _plain_ffn(state)


def _run_own(s):
    import mixture_experts_layer_counting_amd as moe
    c = s["case"]
    op = c["op"]
    dt = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16}
    if op in ("route", "route_train"):
        d = s.get("desc")
        if d is None:
            score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
            d = s["desc"] = moe.RouteDesc(c["T"], c["E"], c["K"], score, c["groups"], c["topk_groups"],
                                          c["group_top"], int(c["renorm"]), c["scale"])
        t = dt[c["dtype"]]
        moe.moe_route_scored(d, s["logits"], t, s["bias"], s["idx"], s["w"])
        if op == "route":
            return s["idx"], s["w"]
        moe.moe_route_scored_backward(d, s["logits"], t, s["idx"], s["d_w"], s["d_logits"])
        return s["idx"], s["w"], s["d_logits"]
    if op == "quant_rows":
        moe.moe_quantize_mxfp4(s["x"], dt[c["dtype"]], c["R"], c["C"], s["q"], s["sf"])
        moe.moe_dequantize_mxfp4(s["q"], s["sf"], c["R"], c["C"], s["values"], moe.MOE_BF16)
        return s["values"]
    if op == "quant_weights":
        layout = moe.MOE_MXFP4_PAIRED if c["paired"] else moe.MOE_MXFP4
        moe.moe_quantize_mxfp4_weights(s["w"], dt[c["dtype"]], c["E"], c["K"], c["N"], layout, s["q"], s["sf"])
        moe.moe_dequantize_mxfp4_weights(s["q"], s["sf"], layout, c["E"], c["K"], c["N"], s["values"],
                                         moe.MOE_BF16)
        return s["values"]
    M = c["T"] * c["K"]
    moe.moe_grouped_ffn_mxfp4(s["x_q"], s["x_sf"], s["row_src"], c["T"], c["K"], s["cu"], M, c["E"], c["H"],
                              c["Hp"], s["w_gate"], s["w_up"], s["w_down"], s["sf_gate"], s["sf_up"],
                              s["sf_down"], s["y"], s["ws"], s["ws"].numel())
    return s["y"]


# ------------------------------------------------------------------------------- plain forms


def _masked(l):
    """Experts that may not be picked: NaN, -inf or the type's lowest value."""
    return ~(l > torch.finfo(l.dtype).min)


def _plain_route(s):
    """Scores and picks in 64 bits (picks next to a border decide on the last digits)."""
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    off = _masked(s["logits"])
    l = torch.where(off, -math.inf, s["logits"].double())
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(dim=1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        total = p.sum(dim=1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    choice = torch.where(off, -math.inf, p + s["bias"].double()) if s["bias"] is not None else l
    if c["topk_groups"] < G:
        u = choice if s["bias"] is not None or c["group_top"] == 1 else torch.where(off, -math.inf, p)
        best = torch.sort(u.view(T, G, E // G), dim=2, descending=True).values[..., :c["group_top"]]
        none = best[..., 0] == -math.inf
        score = torch.where(best == -math.inf, 0.0, best).sum(dim=2)
        score = torch.where(none, -math.inf, score)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], choice.view(T, G, E // G), -math.inf).view(T, E)
    v, i = torch.sort(choice, dim=1, descending=True, stable=True)
    v, i = v[:, :K], i[:, :K]
    got = v > -math.inf
    w = torch.where(got, torch.gather(p, 1, i), 0.0)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(got, i, -1).to(torch.int32), (w * c["scale"]).float(), p


def _plain_route_train(s):
    c = s["case"]
    idx, w, p = _plain_route(s)
    p = p.float()
    got = idx >= 0
    i = idx.clamp(min=0).long()
    q = torch.where(got, torch.gather(p, 1, i), 0.0)
    d = torch.where(got, s["d_w"], 0.0)
    if c["renorm"]:
        total = q.sum(dim=1, keepdim=True)
        r = q / torch.where(total > 0, total, 1.0)
        v = r * (d - (d * r).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            v = v * (1.0 - q)
        out = torch.zeros_like(p).scatter_add_(1, i, torch.where(got, v, 0.0))
    elif c["score"] == "sigmoid":
        out = torch.zeros_like(p).scatter_add_(1, i, d * q * (1.0 - q))
    else:
        out = torch.zeros_like(p).scatter_add_(1, i, d * q) - p * (d * q).sum(dim=1, keepdim=True)
    return idx, w, (out * c["scale"]).to(s["logits"].dtype)


def _plain_mx(v, dim):
    """Values of blocks of 32 along `dim` after MXFP4: e2m1 to nearest even times a power of two."""
    X = _scale_of(v.abs().amax(dim=dim, keepdim=True))
    a = v / X
    m = a.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.clamp(torch.round(a / step) * step, -6.0, 6.0) * X


def _values(codes, scales, dtype):
    """codes [..., N, K/2], scales [..., K/32, N] -> values [..., N, K]."""
    *lead, N, half = codes.shape
    v = torch.index_select(_byte_table(codes.device, dtype), 0, codes.reshape(-1).int())
    v = v.view(*lead, N, half // 16, 32)
    X = torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), scales.int() - 127)
    return v.mul_(X.transpose(-1, -2).unsqueeze(-1)).view(*lead, N, 2 * half)


def _grouped(s, dtype, mx):
    """The grouped FFN over the experts that have rows, each group padded to the largest."""
    c = s["case"]
    K, H, Hp, cap = c["K"], c["H"], c["Hp"], s["cap"]
    act = s["active"]
    A = act.numel()

    def weight(name):
        q, sf = s["w_" + name], s["sf_" + name]
        if A < c["E"]:
            q, sf = q[act], sf[act]
        return _values(q, sf, dtype)

    x = _values(s["x_q"], s["x_sf"].t(), dtype)
    rows = torch.zeros(A * cap, H, dtype=dtype, device=x.device)
    rows[s["slot"]] = x[(s["row_src"] // K).long()]
    rows = rows.view(A, cap, H)
    w = weight("gate")
    gate = torch.bmm(rows, w.transpose(1, 2))
    del w
    h = gate / (1.0 + torch.exp(-gate))
    del gate
    w = weight("up")
    h = h * torch.bmm(rows, w.transpose(1, 2))
    del w, rows
    h = mx(h.view(A, cap, Hp // 32, 32), 3).view(A, cap, Hp)
    w = weight("down")
    y = torch.bmm(h, w.transpose(1, 2)).view(A * cap, H)
    return y[s["slot"]]


def _plain_ffn(s):
    return _grouped(s, torch.float32, _plain_mx).to(torch.bfloat16)


# ------------------------------------------------------------------------------- the work


def work(case):
    op = case["op"]
    if op in ("route", "route_train"):
        T, E, K = case["T"], case["E"], case["K"]
        b = 4 if case["dtype"] == "f32" else 2
        n = T * E * b + T * K * 8
        f = 10 * T * E
        if op == "route_train":
            n += T * E * b + T * K * 4
            f += 4 * T * E
        return {"bytes": n, "flops": f}
    if op in ("quant_rows", "quant_weights"):
        n = case["R"] * case["C"] if op == "quant_rows" else case["E"] * case["K"] * case["N"]
        b = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * b + n // 2 + n // 32 + n * 2, "flops": 4 * n}
    T, E, K, H, Hp = (case[k] for k in ("T", "E", "K", "H", "Hp"))
    M = T * K
    used = min(E, M)
    weights = used * 3 * H * Hp * 17 // 32
    return {"bytes": weights + T * H * 17 // 32 + M * H * 2, "flops": 6 * M * H * Hp}


# ------------------------------------------------------------------------------- in 64 bits


def _mx_exact(v, dim):
    """The format's definition: nearest of the 15 values, a tie to the even code."""
    v = v.double()
    amax = v.abs().amax(dim=dim, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    X = torch.exp2(torch.where(amax > 0, e - 2, -127.0).clamp(-127, 127))
    a = v / X
    m = a.abs()
    out = torch.zeros_like(a)
    for border, up, value in ((0.25, False, 0.5), (0.75, True, 1.0), (1.25, False, 1.5), (1.75, True, 2.0),
                              (2.5, False, 3.0), (3.5, True, 4.0), (5.0, False, 6.0)):
        out = torch.where((m >= border) if up else (m > border), value, out)
    return torch.copysign(out, a) * X


def _exact_route(s):
    """Picks one at a time by the largest remaining choice; gradient by autograd."""
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    raw = s["logits"].double()
    live = torch.isfinite(raw) & (s["logits"] != torch.finfo(s["logits"].dtype).min)
    x = torch.where(live, raw, 0.0).requires_grad_(True)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.where(live, x, -1e300)
        p = torch.softmax(p, dim=1)
    p = torch.where(live, p, 0.0)
    with torch.no_grad():
        choice = p + s["bias"].double() if s["bias"] is not None else raw.clone()
        choice = torch.where(live, choice, -math.inf)
        if c["topk_groups"] < G:
            u = choice if s["bias"] is not None or c["group_top"] == 1 else torch.where(live, p, -math.inf)
            u = u.view(T, G, E // G).clone()
            score = torch.full((T, G), -math.inf, dtype=torch.float64, device=x.device)
            for n in range(c["group_top"]):
                best, at = u.max(dim=2)
                score = torch.where(best > -math.inf, (best if n == 0 else score + best), score)
                u.scatter_(2, at[..., None], -math.inf)
            left = torch.ones(T, G, dtype=torch.bool, device=x.device)
            for _ in range(c["topk_groups"]):
                best = torch.where(left, score, -math.inf).amax(dim=1, keepdim=True)
                at = (left & (score == best)).to(torch.int8).argmax(dim=1, keepdim=True)
                left.scatter_(1, at, False)
            choice = torch.where(left[:, :, None], -math.inf, choice.view(T, G, E // G)).view(T, E)
        picks = []
        for _ in range(K):
            best = choice.amax(dim=1, keepdim=True)
            at = (choice == best).to(torch.int8).argmax(dim=1, keepdim=True)
            picks.append(torch.where(best > -math.inf, at, -1))
            choice.scatter_(1, at, -math.inf)
        i = torch.cat(picks, dim=1)
    got = i >= 0
    w = torch.where(got, torch.gather(p, 1, i.clamp(min=0)), 0.0)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = w * c["scale"]
    if c["op"] == "route":
        return i.to(torch.int32), w.detach()
    d = torch.where(got, s["d_w"].double(), 0.0)
    grad, = torch.autograd.grad((w * d).sum(), x)
    return i.to(torch.int32), w.detach(), torch.where(live, grad, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_train"):
        return _exact_route(s)
    if op == "quant_rows":
        x = s["x"]
        return _mx_exact(x.view(x.shape[0], -1, 32), 2).view(x.shape)
    if op == "quant_weights":
        E, K, N = s["w"].shape
        return torch.stack([_mx_exact(w.view(K // 32, 32, N), 1).view(K, N).to(torch.bfloat16) for w in s["w"]]).double()
    c = case
    # expert by expert, from the codes' values: rows of an expert as a matrix product in 64 bits
    half = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=s["x_q"].device)

    def values(q, sf):  # [N, K/2], [N, K/32]
        v = torch.stack([half[(q & 15).long()], half[(q >> 4).long()]], dim=2).view(q.shape[0], -1, 32)
        return (v * torch.exp2(sf.double() - 127)[:, :, None]).view(q.shape[0], -1)

    x = values(s["x_q"], s["x_sf"])
    y = torch.zeros(c["T"] * c["K"], c["H"], dtype=torch.float64, device=x.device)
    cu = s["cu"].tolist()
    for e in range(c["E"]):
        if cu[e + 1] == cu[e]:
            continue
        rows = x[(s["row_src"][cu[e]:cu[e + 1]] // c["K"]).long()]
        gate = rows @ values(s["w_gate"][e], s["sf_gate"][e].t()).t()
        up = rows @ values(s["w_up"][e], s["sf_up"][e].t()).t()
        h = gate * torch.sigmoid(gate) * up
        h = _mx_exact(h.view(h.shape[0], -1, 32), 2).view(h.shape)
        y[cu[e]:cu[e + 1]] = h @ values(s["w_down"][e], s["sf_down"][e].t()).t()
    return y
