"""Cases for the operators around the sparse-MoE layer: MXFP4 quantisation, the grouped MXFP4 x
MXFP4 product, the experts on MXFP4 activations, and the gradients of the router, the token
permutation and the combine.

`run` computes a case either in its plain form (elementary torch operations in 32 bits, rounded
once) or, with `own` set, through the library's entry points.  `exact` computes the same outputs
in 64 bits from the definitions.

Formats: MXFP4 is OCP Microscaling v1.0 -- E2M1 codes (two per byte, even element in the low
nibble) and one E8M0 scale byte per 32 consecutive elements of a row.  A block's scale is
2^(floor(log2 max|v|) - 2); its elements are v / scale rounded to nearest even and saturated at 6.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest quantisation: one decode batch of eight 4096-wide token rows
        {"name": "quantise_decode_rows", "op": "quantise", "rows": 8, "cols": 4096, "dtype": "bf16", "pad": 0},
        # weights of 24 experts of a 2816-wide layer turned into MXFP4 from an fp32 checkpoint whose rows
        # sit in a wider buffer (an odd number of rows, rows not contiguous)
        {"name": "quantise_weights_fp32", "op": "quantise", "rows": 33791, "cols": 2816, "dtype": "fp32", "pad": 64},
        # one new token: six of 256 experts, one row each (gate/up projection of a 4096-wide layer)
        {"name": "product_one_token", "op": "product", "groups": 256, "tokens": 1, "top_k": 6, "n": 4096, "k": 4096},
        # a long prompt through the same projection: 49152 sorted rows in 256 ragged groups
        {"name": "product_prefill", "op": "product", "groups": 256, "tokens": 8192, "top_k": 6, "n": 4096, "k": 4096},
        # the experts of a decode batch of eight tokens, from x to the sorted expert outputs
        {"name": "experts_decode", "op": "experts", "tokens": 8, "hidden": 4096, "ffn": 2048, "experts": 256, "top_k": 6, "shared": 0},
        # the experts of a prompt with a shared expert and a contraction (704) that is no power of two
        {"name": "experts_prefill_shared", "op": "experts", "tokens": 2049, "hidden": 2816, "ffn": 704, "experts": 128, "top_k": 8, "shared": 1},
        # gradient of the combine: a small batch, and a training batch with skewed routing
        {"name": "combine_grad_small", "op": "combine_grad", "tokens": 7, "hidden": 4096, "experts": 256, "top_k": 6, "shared": 0},
        {"name": "combine_grad_batch", "op": "combine_grad", "tokens": 4096, "hidden": 2048, "experts": 128, "top_k": 8, "shared": 0},
        # gradient of the permutation with the router's part: one token, and a batch with a shared expert
        {"name": "permute_grad_one_token", "op": "permute_grad", "tokens": 1, "hidden": 2048, "experts": 128, "top_k": 8, "shared": 0},
        {"name": "permute_grad_batch", "op": "permute_grad", "tokens": 8191, "hidden": 2816, "experts": 128, "top_k": 8, "shared": 1},
        # gradient of the router: a small batch, and a training batch with skewed routing
        {"name": "route_grad_small", "op": "route_grad", "tokens": 33, "hidden": 2048, "experts": 128, "top_k": 8, "shared": 0},
        {"name": "route_grad_batch", "op": "route_grad", "tokens": 8192, "hidden": 4096, "experts": 256, "top_k": 6, "shared": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "product", "experts", "combine_grad", "permute_grad", "route_grad"])
    if op == "quantise":
        return {"op": op, "rows": _log(rng, 1, 40000), "cols": 32 * _log(rng, 1, 128), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "pad": rng.choice([0, 0, 8, 64])}
    experts = _log(rng, 1, 256)
    top_k = rng.randint(1, min(8, experts))
    if op == "product":
        return {"op": op, "groups": experts, "tokens": _log(rng, 1, 4096), "top_k": top_k, "n": 8 * _log(rng, 2, 512), "k": 64 * _log(rng, 1, 64)}
    case = {"op": op, "tokens": _log(rng, 1, 4096), "hidden": 128 * _log(rng, 1, 32), "experts": experts, "top_k": top_k, "shared": rng.randint(0, 1)}
    if op == "experts":
        case["ffn"] = 64 * _log(rng, 1, 32)
        case["tokens"] = _log(rng, 1, 2048)
    if op == "route_grad":
        case["shared"] = 0
    return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _codes(g, *shape):
    """Random MXFP4 weights: every code equally likely, scales 2^-8 .. 2^-4."""
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(119, 124, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def _routing(g, tokens, experts, top_k, shared, skew):
    """Seeded logits (with a Zipf bias when skew) -> the routing and permutation that steps 1 and 2 leave behind."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    if skew:
        rank = 1 + torch.randperm(experts, generator=g, device="cuda")
        logits = logits - torch.log(rank.float())
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = top.indices[:, :top_k].contiguous()
    gates = torch.softmax(top.values[:, :top_k], dim=1).contiguous()
    groups = experts + shared
    flat = torch.cat([idx.reshape(-1), torch.full((tokens,), experts, device="cuda")]) if shared else idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(flat, minlength=groups)
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    active = torch.nonzero(counts).reshape(-1)
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return {"idx": i32(idx), "gates": gates, "offsets": i32(offsets), "sorted_flat": i32(order), "inv_pos": i32(inv),
            "active": active, "n_max": int(counts.max())}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantise":
        rows, cols, pad = case["rows"], case["cols"], case["pad"]
        # rows of different magnitudes, as the rows of a weight matrix or of token activations have
        mag = torch.exp2(torch.randn(rows, 1, generator=g, device="cuda") * 2 - 5)
        buf = (torch.randn(rows, cols + pad, generator=g, device="cuda") * mag).to(_DT[case["dtype"]])
        s["x"] = buf[:, :cols]
        return s
    if op == "product":
        T, G, k = case["tokens"], case["groups"], case["top_k"]
        s |= _routing(g, T, G, k, 0, False)
        a = _plain_mx4_codes(_normal(g, (T * k, case["k"])).float())
        s["a_codes"], s["a_scales"] = a
        s["w_codes"], s["w_scales"] = _codes(g, G, case["n"], case["k"])
        return s
    T, H, E, k, S = case["tokens"], case["hidden"], case["experts"], case["top_k"], case["shared"]
    s |= _routing(g, T, E, k, S, op != "experts")
    R = T * k + T * S
    if op == "experts":
        F = case["ffn"]
        s["x"] = _normal(g, (T, H))
        # group E, when there is one, is the shared expert: kept apart by the program, stacked here so that the plain form is one product
        s["w13"], s["w13_scale"] = _codes(g, E + S, 2 * F, H)
        s["w2"], s["w2_scale"] = _codes(g, E + S, H, F)
    elif op == "combine_grad":
        s["dy"] = _normal(g, (T, H), 0.01)
        s["o"] = _normal(g, (R, H))
    elif op == "permute_grad":
        s["dxs"] = _normal(g, (R, H), 0.01)
        s["dlogits"] = torch.randn(T, k, generator=g, device="cuda") * 0.01
        s["w_router"] = torch.randn(E, H, generator=g, device="cuda") * 0.02
    elif op == "route_grad":
        s["x"] = _normal(g, (T, H))
        s["dg"] = torch.randn(T, k, generator=g, device="cuda") * 0.1
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _pow2(e):
    """2^e for integer e in [-126, 127], from its bit pattern."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_blocks(x32):
    """(elements on the E2M1 grid [rows, blocks, 32], block exponents [rows, blocks])."""
    b = x32.reshape(x32.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.zeros_like(amax, dtype=torch.int32)).clamp(min=-127)
    v = b * _pow2(-e)[..., None]
    a = v.abs()
    q = torch.where(a < 2, torch.round(a * 2) * 0.5, torch.where(a < 4, torch.round(a), torch.round(a * 0.5) * 2)).clamp(max=6)
    return torch.copysign(q, v), e


def _plain_mx4(x32):
    """The values that x's MXFP4 codes stand for."""
    q, e = _plain_blocks(x32)
    return torch.ldexp(q, e[..., None]).reshape(x32.shape)


def _plain_mx4_codes(x32):
    q, e = _plain_blocks(x32)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).reshape(x32.shape[0], -1, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _table():
    m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    v = torch.cat([m, -m])
    byte = torch.arange(256, device="cuda")
    return torch.stack([v[byte & 15], v[byte >> 4]], 1)


def _plain_decode(codes, scales):
    v = torch.nn.functional.embedding(codes.to(torch.int32), _table())
    v = v.reshape(codes.shape[:-1] + (-1, 32))
    s = torch.exp2(scales.float() - 127)
    return v.mul_(s[..., None]).reshape(codes.shape[:-1] + (-1,))


def _plain_product(s, a, w_codes, w_scales):
    """a [R, K] fp32 rows sorted by group times their group's weights: one batched product over the groups that have rows."""
    active, n_max = s["active"], s["n_max"]
    start = s["offsets"][active].to(torch.int64)
    w = _plain_decode(w_codes[active], w_scales[active])
    rows = (start[:, None] + torch.arange(n_max, device="cuda")).clamp(max=a.shape[0] - 1)
    out = torch.bmm(a[rows], w.transpose(1, 2))
    r = torch.arange(a.shape[0], device="cuda")
    at = torch.searchsorted(start, r, right=True) - 1
    return out[at, r - start[at]]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantise":
        return _plain_mx4(s["x"].float()).to(s["x"].dtype)
    if op == "product":
        return _plain_product(s, _plain_decode(s["a_codes"], s["a_scales"]), s["w_codes"], s["w_scales"]).to(torch.bfloat16)
    T, k, S = c["tokens"], c["top_k"], c["shared"]
    flat = s["sorted_flat"].to(torch.int64)
    if op == "experts":
        token = torch.where(flat < T * k, flat // k, flat - T * k)
        x = _plain_mx4(s["x"].float())[token]
        gu = _plain_product(s, x, s["w13"], s["w13_scale"])
        gate, up = gu.chunk(2, 1)
        h = _plain_mx4(gate / (1 + torch.exp(-gate)) * up)
        return _plain_product(s, h, s["w2"], s["w2_scale"]).to(torch.bfloat16)
    if op == "route_grad":
        gates, dg = s["gates"], s["dg"]
        dl = gates * (dg - (gates * dg).sum(1, keepdim=True))
        dense = torch.zeros(T, c["experts"], device="cuda").scatter_(1, s["idx"].to(torch.int64), dl)
        return {"dlogits": dl, "dw_router": dense.t() @ s["x"].float(), "dbias": dense.sum(0)}
    pos = s["inv_pos"].to(torch.int64)
    routed, shared = pos[:T * k].reshape(T, k), pos[T * k:]
    if op == "combine_grad":
        dy = s["dy"].float()
        d_o = torch.empty_like(s["o"])
        d_o[routed] = (s["gates"][..., None] * dy[:, None]).to(torch.bfloat16)
        if S:
            d_o[shared] = s["dy"]
        return {"d_o_sorted": d_o, "d_topk_w": (s["o"][routed].float() * dy[:, None]).sum(-1)}
    dx = s["dxs"][routed].float().sum(1) + (s["dlogits"][..., None] * s["w_router"][s["idx"].to(torch.int64)]).sum(1)
    if S:
        dx = dx + s["dxs"][shared].float()
    return dx.to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls
_ws = None


def _workspace(F, nbytes):
    """The program's one scratch buffer: made once, larger when a call needs more."""
    global _ws
    if _ws is None or _ws.numel() < nbytes:
        _ws = torch.empty(max(nbytes, 4096), dtype=torch.uint8, device="cuda")
        F.ft_moe_workspace_init(_ws)
    return _ws


def _own(s):
    from expert_offload_serving_router_b200 import ftmoe as F
    c = s["case"]
    op = c["op"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "quantise":
        x, rows, cols = s["x"], c["rows"], c["cols"]
        codes, scales, values = new(rows, cols // 2, dtype=torch.uint8), new(rows, cols // 32, dtype=torch.uint8), new(rows, cols, dtype=x.dtype)
        dt = {"bf16": F.FT_T_BF16, "fp16": F.FT_T_FP16, "fp32": F.FT_T_FP32}[c["dtype"]]
        F.ft_mx4_quantize(rows, cols, dt, x, x.stride(0), codes, scales, values)
        return values
    if op == "product":
        G, R, n, k = c["groups"], c["tokens"] * c["top_k"], c["n"], c["k"]
        ws = _workspace(F, F.ft_mx4_product_workspace_bytes(G, R, n, k))
        out = new(R, n)
        F.ft_mx4_product(G, R, n, k, s["offsets"], s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], out, ws)
        return out
    T, H, E, k, S = c["tokens"], c["hidden"], c["experts"], c["top_k"], c["shared"]
    R = T * k + T * S
    if op == "experts":
        shape = F.make_shape(H, c["ffn"], E, k, S, F.FT_W_MXFP4)
        w = F.make_weights(s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], None,
                           *((s["w13"][E], s["w13_scale"][E], s["w2"][E], s["w2_scale"][E]) if S else ()))
        ws = _workspace(F, F.ft_moe_workspace_bytes(shape, T))
        o = new(R, H)
        F.ft_moe_experts_mx4(shape, T, w, s["x"], s["offsets"], s["inv_pos"], o, ws)
        return o
    shape = F.make_shape(H, 64, E, k, S)
    if op == "combine_grad":
        d_o, d_w = new(R, H), new(T, k, dtype=torch.float32)
        F.ft_moe_combine_backward(shape, T, s["dy"], s["o"], s["inv_pos"], s["gates"], d_o, d_w)
        return {"d_o_sorted": d_o, "d_topk_w": d_w}
    if op == "permute_grad":
        dx = new(T, H)
        F.ft_moe_permute_backward(shape, T, s["dxs"], s["inv_pos"], s["idx"], s["dlogits"], s["w_router"], dx)
        return dx
    ws = _workspace(F, F.ft_moe_workspace_bytes(shape, T))
    dl, dw, db = new(T, k, dtype=torch.float32), new(E, H, dtype=torch.float32), new(E, dtype=torch.float32)
    F.ft_moe_route_backward(shape, T, s["x"], s["idx"], s["gates"], s["dg"], s["offsets"], s["sorted_flat"], dl, dw, db, ws)
    return {"dlogits": dl, "dw_router": dw, "dbias": db}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    mx = 17 / 32          # bytes of one MXFP4 element with its share of the scale
    if op == "quantise":
        n, b = case["rows"] * case["cols"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": n * (2 * b + mx), "flops": 0}
    T, k = case["tokens"], case["top_k"]
    touched = lambda E: E * (1 - (1 - k / E) ** T)  # noqa: E731 -- groups with rows, expected
    if op == "product":
        R, n, K = T * k, case["n"], case["k"]
        return {"bytes": touched(case["groups"]) * n * K * mx + R * K * mx + R * n * 2, "flops": 2 * R * n * K}
    H, E, S = case["hidden"], case["experts"], case["shared"]
    R = T * k + T * S
    if op == "experts":
        F = case["ffn"]
        return {"bytes": (touched(E) + S) * 3 * F * H * mx + T * H * 2 + R * H * 2 + R * 4, "flops": 6 * R * F * H}
    if op == "combine_grad":
        return {"bytes": T * H * 2 + T * k * H * 2 + R * H * 2 + R * 4 + T * k * 8, "flops": 4 * R * H}
    if op == "permute_grad":
        return {"bytes": R * H * 2 + T * H * 2 + touched(E) * H * 4 + R * 4 + T * k * 8, "flops": (R + 2 * T * k) * H}
    return {"bytes": T * H * 2 + E * H * 4 + E * 4 + T * k * 20, "flops": 2 * T * k * H}


# ------------------------------------------------------------------ the definitions in 64 bits
_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _exact_mx4(v):
    """fp64 values -> the fp64 values of their MXFP4 form: nearest grid point by the midpoints, ties to the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    mids = torch.tensor(_MIDS, dtype=torch.float64, device=v.device)
    b = v.reshape(-1, 32)
    m = b.abs().max(1, keepdim=True).values
    scale = torch.where(m > 0, torch.exp2((torch.frexp(m).exponent - 3).double().clamp(min=-127)), torch.ones_like(m))
    a = (b / scale).abs()
    i = torch.bucketize(a, mids)
    tie = a == mids[i.clamp(max=6)]
    i = i + (tie & (i % 2 == 1) & (i < 7)).long()
    return (torch.sign(b) * grid[i] * scale).reshape(v.shape)


def _exact_decode(codes, scales):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=codes.device)
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).reshape(codes.shape[:-1] + (-1, 32))
    return (v * torch.exp2(scales.double() - 127)[..., None]).reshape(codes.shape[:-1] + (-1,))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _exact_mx4(s["x"].double())
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]
    if op == "product":
        a = _exact_decode(s["a_codes"], s["a_scales"])
        out = torch.empty(a.shape[0], case["n"], dtype=torch.float64, device=a.device)
        for e, lo, hi in spans:
            out[lo:hi] = a[lo:hi] @ _exact_decode(s["w_codes"][e], s["w_scales"][e]).t()
        return out
    T, k, S, H = case["tokens"], case["top_k"], case["shared"], case["hidden"]
    flat = s["sorted_flat"].long()
    token = torch.where(flat < T * k, flat // k, flat - T * k)
    if op == "experts":
        x = _exact_mx4(s["x"].double())
        out = torch.empty(flat.numel(), H, dtype=torch.float64, device=x.device)
        F = case["ffn"]
        for e, lo, hi in spans:
            r = x[token[lo:hi]] @ _exact_decode(s["w13"][e], s["w13_scale"][e]).t()
            h = _exact_mx4(r[:, :F] * torch.sigmoid(r[:, :F]) * r[:, F:])
            out[lo:hi] = h @ _exact_decode(s["w2"][e], s["w2_scale"][e]).t()
        return out
    gates = s["gates"].double()
    if op == "combine_grad":
        dy = s["dy"].double()
        weight = torch.cat([gates.reshape(-1), torch.ones(T * S, dtype=torch.float64, device=dy.device)])[flat]
        dot = (s["o"].double() * dy[token]).sum(1)
        d_w = torch.zeros(T * k + T * S, dtype=torch.float64, device=dy.device)
        d_w[flat] = dot
        return {"d_o_sorted": weight[:, None] * dy[token], "d_topk_w": d_w[:T * k].reshape(T, k)}
    if op == "permute_grad":
        dx = torch.zeros(T, H, dtype=torch.float64, device=flat.device)
        dx.index_add_(0, token, s["dxs"].double())
        for j in range(k):
            dx += s["dlogits"][:, j:j + 1].double() * s["w_router"].double()[s["idx"][:, j].long()]
        return dx
    # the softmax's Jacobian over the kept logits, diag(g) - g g^T, applied to the gates' gradient
    jac = torch.diag_embed(gates) - gates[:, :, None] * gates[:, None, :]
    dl = (jac @ s["dg"].double()[..., None])[..., 0]
    by_row = dl.reshape(-1)[flat]
    x = s["x"].double()
    dw = torch.zeros(case["experts"], H, dtype=torch.float64, device=x.device)
    db = torch.zeros(case["experts"], dtype=torch.float64, device=x.device)
    for e, lo, hi in spans:
        dw[e] = by_row[lo:hi] @ x[token[lo:hi]]
        db[e] = by_row[lo:hi].sum()
    return {"dlogits": dl, "dw_router": dw, "dbias": db}
