"""GPU parity of the MXFP4 quantiser, the grouped MXFP4 product and the experts on MXFP4 activations
against plain 64-bit forms.

Tolerances.  Codes, scales and dequantised values are exact.  A product's output is one fp32 sum of exact
products rounded to bf16: |out - exact| <= 2^-8 |exact| + sum_bound(K) sum|a w| (mx4_util).  The experts'
hidden values go through a second quantisation, which is a step function: with |h - h64| <= dh the
code is one of those between Q(h64 - dh) and Q(h64 + dh) (for a block whose largest element may fall on
either side of a power of two: of both scales), so sum |w2| times that interval is added."""
import numpy as np
import pytest

import mx4_util as M
from expert_offload_serving_router_b200 import ftmoe as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpu_util import ensure_built
    ensure_built()


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def new_ws(n=4096):
    import torch
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    F.ft_moe_workspace_init(ws)
    return ws


DT = {"bf16": F.FT_T_BF16, "fp16": F.FT_T_FP16, "fp32": F.FT_T_FP32}


def tdtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def run_quantize(x, dtype, cols, with_values=True):
    """x: CUDA tensor [rows, >= cols] view with unit column stride."""
    import torch
    rows = x.shape[0]
    codes = torch.full((rows + 1, cols // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 1, cols // 32), 0xCD, dtype=torch.uint8, device="cuda")
    vals = torch.full((rows + 1, cols), 7.0, dtype=x.dtype, device="cuda") if with_values else None
    F.ft_mx4_quantize(rows, cols, DT[dtype], x, x.stride(0), codes, scales, vals)
    torch.cuda.synchronize()
    # the row behind the last one stays as it was
    assert (codes[rows] == 0xAB).all() and (scales[rows] == 0xCD).all()
    assert vals is None or (vals[rows] == 7.0).all()
    return codes[:rows].cpu().numpy(), scales[:rows].cpu().numpy(), None if vals is None else vals[:rows].double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 32, 0, 0), (3, 64, 0, 0), (1, 4096, 0, 0), (257, 96, 8, 0),
                                                 (129, 704, 1, 0), (65, 2816, 3, 1), (1000, 160, 64, 8)])
def test_quantize_exact(dtype, rows, cols, pad, shift):
    """pad 1 and 3, shift 1: rows off 16-byte alignment."""
    import torch
    g = np.random.default_rng(rows * 7 + cols)
    x = g.standard_normal((rows, cols + pad)) * np.exp2(g.integers(-12, 6, size=(rows, 1)))
    t = torch.from_numpy(x).to(tdtype(dtype))
    buf = torch.zeros(rows * (cols + pad) + shift, dtype=tdtype(dtype), device="cuda")
    v = buf[shift:].view(rows, cols + pad)
    v.copy_(t)
    x = v[:, :cols]
    codes, scales, vals = run_quantize(x, dtype, cols)
    rc, rs = M.quantize(x.double().cpu().numpy())
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, M.pack(rc))
    assert np.array_equal(vals, M.values(rc, rs))
    c2, s2, _ = run_quantize(x, dtype, cols, with_values=False)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_borders_zeros_nans_extremes(dtype):
    import torch
    g = np.random.default_rng(5)
    info = torch.finfo(tdtype(dtype))
    pts = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    rows = [np.resize(np.concatenate([pts, -pts]), 32) * 2.0 ** e for e in (-8, 0, 3, 10)]
    rows += [np.zeros(32), -np.zeros(32)]
    for bad in (np.nan, np.inf, -np.inf):
        for at in (0, 13, 31):
            r = g.standard_normal(32)
            r[at] = bad
            rows.append(r)
    rows += [np.full(32, info.max), np.full(32, -info.max), np.full(32, info.tiny), np.full(32, info.smallest_normal / 4),
             np.where(np.arange(32) == 9, info.max, info.tiny)]
    x = torch.from_numpy(np.stack(rows)).to(tdtype(dtype)).cuda()
    codes, scales, vals = run_quantize(x, dtype, 32)
    rc, rs = M.quantize(x.double().cpu().numpy())
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, M.pack(rc))
    want = torch.from_numpy(M.values(rc, rs)).to(tdtype(dtype)).double().numpy()
    assert np.array_equal(vals, want, equal_nan=True)


# ------------------------------------------------------------------ product
def run_product(off, ac, asc, wc, ws_, n, k, rows=None, ws=None):
    import torch
    rows = ac.shape[0] if rows is None else rows
    out = torch.full((rows + 1, n), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = new_ws() if ws is None else ws
    F.ft_mx4_product(len(off) - 1, rows, n, k, cuda(off), cuda(ac), cuda(asc), cuda(wc), cuda(ws_), out, ws)
    F.ft_moe_check(ws)
    assert (out[rows] == 3.0).all()
    return out[:rows].double().cpu().numpy()


def product64(off, ac, asc, wc, ws_):
    a, out, mag = M.dequantize(ac, asc), None, None
    n = wc.shape[1]
    out = np.full((a.shape[0], n), 3.0)
    mag = np.zeros_like(out)
    for g in range(len(off) - 1):
        lo, hi = off[g], off[g + 1]
        if hi > lo:
            w = M.dequantize(wc[g], ws_[g])
            out[lo:hi] = a[lo:hi] @ w.T
            mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w).T
    return out, mag


def check_product(got, want, mag, k):
    tol = M.UB16 * np.abs(want) + M.sum_bound(k) * mag
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: {got[bad][:4]} {want[bad][:4]}"


def activations(g, rows, k):
    code, scale = M.quantize(g.standard_normal((rows, k)) * np.exp2(g.integers(-6, 4, size=(rows, 1))))
    return M.pack(code), scale


@pytest.mark.parametrize("groups,rows,n,k,skew", [
    (1, 1, 128, 64, 0), (1, 1, 8, 64, 0), (1, 3, 24, 128, 0), (1, 33, 136, 192, 0), (1, 224, 128, 256, 0),
    (1, 225, 256, 512, 0), (1, 700, 384, 704, 0), (2, 449, 128, 320, 0), (5, 97, 200, 768, 1.5), (8, 300, 128, 1024, 2),
    (8, 1, 640, 2816, 0), (256, 6, 256, 4096, 0), (256, 300, 128, 2048, 1), (256, 5000, 64, 256, 1), (3, 2500, 128, 8192, 0),
    # the 96-row tile and the pairs (odd counts of 128-row groups, ragged K, a group of one row among large ones)
    (16, 640, 1536, 320, 0), (9, 700, 2056, 768, 1), (1, 1999, 2176, 320, 0), (1, 4100, 2184, 1088, 0), (64, 6400, 2048, 192, 0.3),
    (5, 4500, 1160, 704, 2.5)])
def test_product(groups, rows, n, k, skew):
    g = np.random.default_rng(groups * 1000 + rows + n + k)
    off = M.random_offsets(g, groups, rows, skew)
    ac, asc = activations(g, rows, k)
    wc, ws_ = M.random_weights(g, groups, n, k)
    got = run_product(off, ac, asc, wc, ws_, n, k)
    want, mag = product64(off, ac, asc, wc, ws_)
    check_product(got, want, mag, k)


def test_product_integer_exact():
    """Sums of small integers have no rounding at all: every output is exact, whatever the order."""
    g = np.random.default_rng(1)
    rows, n, k = 37, 136, 448
    code = g.choice(np.array([0, 2, 4, 10, 12], dtype=np.uint8), size=(rows, k))     # 0, 1, 2, -1, -2
    wcode = g.choice(np.array([0, 2, 10], dtype=np.uint8), size=(2, n, k), p=[.8, .1, .1])
    one = lambda *s: np.full(s, 127, np.uint8)  # noqa: E731
    off = np.array([0, 20, 37], np.int32)
    args = (off, M.pack(code), one(rows, k // 32), M.pack(wcode), one(2, n, k // 32))
    got = run_product(*args, n, k)
    want, _ = product64(*args)
    assert np.abs(want).max() <= 256
    assert np.array_equal(got, want)


def test_product_scales_reach_their_blocks():
    """One nonzero 32-block at a time, each with a scale of its own: a scale byte applied to a neighbouring block
    or row changes the result by a power of two."""
    g = np.random.default_rng(2)
    k, n = 576, 144
    nb = k // 32
    rows = 2 * nb
    code = np.zeros((rows, k), np.uint8)
    asc = g.integers(110, 140, size=(rows, nb), dtype=np.uint8)
    for r in range(rows):
        code[r, 32 * (r % nb):32 * (r % nb) + 32] = 2                  # value 1
    wcode = np.full((1, n, k), 2, np.uint8)
    wsc = g.integers(110, 140, size=(1, n, nb), dtype=np.uint8)
    off = np.array([0, rows], np.int32)
    args = (off, M.pack(code), asc, M.pack(wcode), wsc)
    got = run_product(*args, n, k)
    want, _ = product64(*args)
    assert np.array_equal(got, want)                                  # 32 * 2^i: exact in bf16


def test_product_nan_scale_stays_in_its_row():
    g = np.random.default_rng(3)
    off = np.array([0, 10, 21], np.int32)
    ac, asc = activations(g, 21, 256)
    wc, ws_ = M.random_weights(g, 2, 128, 256)
    want, mag = product64(off, ac, asc, wc, ws_)
    asc2 = asc.copy()
    asc2[4, 3] = 255
    got = run_product(off, ac, asc2, wc, ws_, 128, 256)
    assert np.isnan(got[4]).all()
    keep = np.arange(21) != 4
    check_product(got[keep], want[keep], mag[keep], 256)


def test_product_rows_outside_the_groups_are_left():
    import torch
    g = np.random.default_rng(4)
    off = np.array([5, 12, 12, 30], np.int32)                         # rows 0..4 and 30.. belong to no group
    ac, asc = activations(g, 40, 128)
    wc, ws_ = M.random_weights(g, 3, 64, 128)
    got = run_product(off, ac, asc, wc, ws_, 64, 128)
    want, mag = product64(off, ac, asc, wc, ws_)
    assert (got[:5] == 3.0).all() and (got[30:] == 3.0).all()
    check_product(got[5:30], want[5:30], mag[5:30], 128)


@pytest.mark.parametrize("off", [[0, 9, 4, 20], [-3, 5, 9, 20], [0, 5, 9, 70], [0, 2 ** 31 - 1, -2 ** 31, 20]])
def test_product_bad_offsets_are_reported(off):
    """The kernel's own check: a table out of order or out of range is reported, nothing of it is followed."""
    import torch
    g = np.random.default_rng(4)
    ac, asc = activations(g, 20, 128)
    wc, ws_ = M.random_weights(g, 3, 64, 128)
    out = torch.full((40, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = new_ws()
    F.ft_mx4_product(3, 20, 64, 128, cuda(np.array(off, np.int32)), cuda(ac), cuda(asc), cuda(wc), cuda(ws_), out[:20], ws)
    with pytest.raises(F.FtError) as ei:
        F.ft_moe_check(ws)
    assert ei.value.status == F.FT_ERR_DEVICE_CHECK and "offsets" in str(ei.value)
    assert (out == 3.0).all()
    F.ft_moe_check(ws)


def test_product_unaligned_scales_and_repeat_is_identical():
    import torch
    g = np.random.default_rng(6)
    off = np.array([0, 100, 333], np.int32)
    ac, asc = activations(g, 333, 1024)
    wc, ws_ = M.random_weights(g, 2, 256, 1024)
    base = run_product(off, ac, asc, wc, ws_, 256, 1024)
    ws = new_ws()
    out = torch.empty(333, 256, dtype=torch.bfloat16, device="cuda")

    def off2(a):          # the same bytes two past a 256-byte boundary
        t = torch.empty(a.size + 2, dtype=torch.uint8, device="cuda")
        t[2:] = cuda(a.reshape(-1))
        return t[2:]
    for _ in range(2):
        F.ft_mx4_product(2, 333, 256, 1024, cuda(off), cuda(ac), off2(asc), cuda(wc), off2(ws_), out, ws)
        F.ft_moe_check(ws)
        assert np.array_equal(out.double().cpu().numpy(), base)


# ------------------------------------------------------------------ experts
def routing(g, T, E, k, S):
    import oracle
    idx = np.stack([g.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32)
    off, sf, inv = oracle.permute(idx, E, S)
    return idx, off, sf, inv


def layer_weights(g, E, S, H, Fd):
    w = {}
    w["w13"], w["w13_scale"] = M.random_weights(g, E, 2 * Fd, H)
    w["w2"], w["w2_scale"] = M.random_weights(g, E, H, Fd)
    if S:
        w["sw13"], w["sw13_scale"] = M.random_weights(g, 1, 2 * Fd, H)
        w["sw2"], w["sw2_scale"] = M.random_weights(g, 1, H, Fd)
    d = {k: cuda(v) for k, v in w.items()}
    p = d.get
    return w, d, F.make_weights(p("w13"), p("w13_scale"), p("w2"), p("w2_scale"), None, p("sw13"), p("sw13_scale"),
                                p("sw2"), p("sw2_scale"))


def q_interval(h, dh):
    """Largest distance from Q(h) that quantising any h' within dh of h (a whole row's blocks) can have."""
    lo, hi = h - dh, h + dh
    c, s = M.quantize(h)
    v = M.values(c, s)
    b = np.abs(h).reshape(s.shape + (32,))
    d = dh.reshape(s.shape + (32,))
    far = np.zeros_like(v)
    m_lo = np.maximum(b - d, 0).max(-1)
    m_hi = (b + d).max(-1)
    for m in (m_lo, m_hi):                                            # the block's scale at either end
        e = np.where(m > 0, np.maximum(np.frexp(np.where(m > 0, m, 1.0))[1] - 3, -127), 0)
        for x in (lo, hi):
            y = np.ldexp(x.reshape(s.shape + (32,)), -e[..., None])
            a = np.minimum(np.abs(y), 6)
            # the two grid points around a cover both roundings near a border
            up = M.GRID[np.searchsorted(M.GRID, a, side="left").clip(max=7)]
            dn = M.GRID[(np.searchsorted(M.GRID, a, side="right") - 1).clip(min=0)]
            r = np.where(a - dn <= up - a, dn, up)
            alt = np.where(a - dn == up - a, up, r)
            for z in (r, alt):
                q = np.ldexp(np.where(y < 0, -z, z), e[..., None]).reshape(v.shape)
                far = np.maximum(far, np.abs(q - v))
    return v, far


def experts64(w, off, tok, x, E, Fd, H):
    """fp64 o_sorted and its tolerance."""
    xc, xs = M.quantize(x)
    xq = M.values(xc, xs)
    R = len(tok)
    out, tol = np.zeros((R, H)), np.zeros((R, H))
    for g in range(len(off) - 1):
        lo, hi = off[g], off[g + 1]
        if hi == lo:
            continue
        if g < E:
            w13, w2 = M.dequantize(w["w13"][g], w["w13_scale"][g]), M.dequantize(w["w2"][g], w["w2_scale"][g])
        else:
            w13, w2 = M.dequantize(w["sw13"][0], w["sw13_scale"][0]), M.dequantize(w["sw2"][0], w["sw2_scale"][0])
        xr = xq[tok[lo:hi]]
        gu, mag = xr @ w13.T, np.abs(xr) @ np.abs(w13).T
        gate, up = gu[:, :Fd], gu[:, Fd:]
        d = M.sum_bound(H) * mag
        h = M.silu(gate) * up
        # |silu'| <= 1.1; expf, the division and the products are a few fp32 roundings
        dh = 1.1 * d[:, :Fd] * (np.abs(up) + d[:, Fd:]) + np.abs(M.silu(gate)) * d[:, Fd:] + 2.0 ** -20 * np.abs(h)
        hq, far = q_interval(h, dh)
        out[lo:hi] = hq @ w2.T
        tol[lo:hi] = M.UB16 * np.abs(out[lo:hi]) + far @ np.abs(w2).T * (1 + M.UB16) + M.sum_bound(Fd) * (np.abs(hq) @ np.abs(w2).T)
    return out, tol


@pytest.mark.parametrize("T,H,Fd,E,k,S", [(1, 128, 64, 1, 1, 0), (1, 256, 128, 8, 2, 1), (5, 512, 192, 16, 3, 0),
                                          (40, 384, 64, 8, 8, 1), (33, 1024, 704, 4, 2, 0), (300, 256, 128, 4, 2, 1),
                                          (700, 128, 320, 3, 1, 0), (64, 2816, 64, 128, 8, 1), (301, 128, 704, 32, 8, 1),
                                          (640, 256, 704, 32, 6, 1), (2000, 128, 1984, 4, 2, 0)])
def test_experts_mx4(T, H, Fd, E, k, S):
    import torch
    import oracle  # noqa: F401
    g = np.random.default_rng(T + H + Fd)
    idx, off, sf, inv = routing(g, T, E, k, S)
    w, d, weights = layer_weights(g, E, S, H, Fd)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16)
    shape = F.make_shape(H, Fd, E, k, S, F.FT_W_MXFP4)
    R = T * k + T * S
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    o = torch.full((R + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_experts_mx4(shape, T, weights, x.cuda(), cuda(off), cuda(inv), o, ws)
    F.ft_moe_check(ws)
    assert (o[R] == 3.0).all()
    tok = np.where(sf < T * k, sf // k, sf - T * k)
    want, tol = experts64(w, off, tok, x.double().numpy(), E, Fd, H)
    got = o[:R].double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside"
    # the tolerance is dominated by the bf16 rounding on nearly every element, not by the flips it allows
    assert np.median(tol / (np.abs(want) + 1e-9 * np.abs(want).max())) < 0.05


def test_experts_mx4_nan_token_stays_in_its_rows():
    import torch
    g = np.random.default_rng(11)
    T, H, Fd, E, k = 9, 256, 128, 4, 2
    idx, off, sf, inv = routing(g, T, E, k, 0)
    w, d, weights = layer_weights(g, E, 0, H, Fd)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    outs = []
    for bad in (False, True):
        if bad:
            x[3, 77] = float("nan")
        o = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
        F.ft_moe_experts_mx4(shape, T, weights, x, cuda(off), cuda(inv), o, ws)
        F.ft_moe_check(ws)
        outs.append(o.double().cpu().numpy())
    hit = np.isin(sf // k, [3])
    assert np.isnan(outs[1][hit]).all()
    assert np.array_equal(outs[0][~hit], outs[1][~hit])


@pytest.mark.parametrize("T,S", [(1, 0), (8, 1), (32, 0), (33, 1), (200, 0)])
def test_layer_forward_mx4_is_its_steps(T, S):
    """The layer call = route, permute, experts and combine called one by one, bit for bit."""
    import torch
    g = np.random.default_rng(T)
    H, Fd, E, k = 512, 192, 16, 4
    w, d, weights = layer_weights(g, E, S, H, Fd)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.02).cuda()
    shape = F.make_shape(H, Fd, E, k, S, F.FT_W_MXFP4)
    R = T * k + T * S
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    lg = torch.empty(T, E, device="cuda")
    F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, idx, lg, ws)
    F.ft_moe_check(ws)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    idx2, gw, off, sf, inv = i32(T, k), torch.empty(T, k, device="cuda"), i32(E + S + 1), i32(R), i32(R)
    o, y2 = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(y)
    F.ft_moe_route(shape, T, x, wr, None, idx2, gw, None, ws)
    F.ft_moe_permute(shape, T, idx2, x, off, sf, inv, None, ws)
    F.ft_moe_experts_mx4(shape, T, weights, x, off, inv, o, ws)
    F.ft_moe_combine(shape, T, o, inv, gw, y2)
    F.ft_moe_check(ws)
    assert torch.equal(idx, idx2)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    # and y follows the 64-bit combine of the experts' rows
    yr = (o.double()[inv[:T * k].long()].view(T, k, H) * gw.double()[..., None]).sum(1)
    if S:
        yr = yr + o.double()[inv[T * k:].long()]
    mag = (o.double()[inv[:T * k].long()].view(T, k, H) * gw.double()[..., None]).abs().sum(1) + yr.abs()
    assert ((y.double() - yr).abs() <= M.UB16 * yr.abs() + 16 * M.U32 * mag).all()


def test_quantized_weights_run_the_layer():
    """Weights quantised by ft_mx4_quantize are the layer's w13 / w2: the bf16-activation experts on them agree with
    the dequantised values, and the captured layer replays to the same bits on another stream."""
    import torch
    g = np.random.default_rng(21)
    T, H, Fd, E, k = 48, 256, 128, 8, 2
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    full = [torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16).cuda() * 0.05 for s in ((E * 2 * Fd, H), (E * H, Fd))]
    q = []
    for m in full:
        c = torch.empty(m.shape[0], m.shape[1] // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(m.shape[0], m.shape[1] // 32, dtype=torch.uint8, device="cuda")
        F.ft_mx4_quantize(m.shape[0], m.shape[1], F.FT_T_BF16, m, m.stride(0), c, s)
        q.append((c, s))
    weights = F.make_weights(q[0][0], q[0][1], q[1][0], q[1][1])
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.02).cuda()
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws)
    F.ft_moe_check(ws)
    first = y.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), first.view(torch.int16))
    # bf16 activations on the same weights: the two forms differ by the activations' 4-bit rounding only
    y16 = torch.empty_like(y)
    F.ft_moe_layer_forward(shape, T, x, wr, None, weights, y16, None, None, ws)
    F.ft_moe_check(ws)
    rel = ((y16.double() - first.double()).norm() / y16.double().norm()).item()
    # x and h each carry at most a quarter of their block's largest element as error; in the norm well under 1/2
    assert rel < 0.5


@pytest.mark.parametrize("groups,rows,n,k", [(256, 40, 1024, 2048), (16, 640, 1536, 2048), (8, 3000, 2048, 2048)])
def test_product_wait_timeout_is_reported_and_the_next_call_is_exact(groups, rows, n, k):
    """A bound shorter than any stage: the kernel gives up, reports it, and leaves the context usable."""
    import torch
    g = np.random.default_rng(31)
    off = M.random_offsets(g, groups, rows)
    ac, asc = activations(g, rows, k)
    wc, ws_ = M.random_weights(g, groups, n, k)
    base = run_product(off, ac, asc, wc, ws_, n, k)
    args = [cuda(off), cuda(ac), cuda(asc), cuda(wc), cuda(ws_)]
    ws = new_ws()
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    prev = F.ft_set_pipeline_wait_limit_ns(1)
    try:
        F.ft_mx4_product(groups, rows, n, k, *args, out, ws)
        with pytest.raises(F.FtError) as ei:
            F.ft_moe_check(ws)
    finally:
        F.ft_set_pipeline_wait_limit_ns(prev)
    assert ei.value.status == F.FT_ERR_DEVICE_CHECK and "timed out" in str(ei.value)
    F.ft_mx4_product(groups, rows, n, k, *args, out, ws)
    F.ft_moe_check(ws)
    assert np.array_equal(out.double().cpu().numpy(), base)


def test_experts_mx4_wait_timeout_is_reported_and_the_next_call_is_exact():
    import torch
    g = np.random.default_rng(32)
    T, H, Fd, E, k, S = 640, 512, 704, 32, 6, 1
    idx, off, sf, inv = routing(g, T, E, k, S)
    w, d, weights = layer_weights(g, E, S, H, Fd)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    shape = F.make_shape(H, Fd, E, k, S, F.FT_W_MXFP4)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    off, inv = cuda(off), cuda(inv)
    outs = []
    for limit in (0, 1, 0):
        o = torch.empty(T * (k + S), H, dtype=torch.bfloat16, device="cuda")
        prev = F.ft_set_pipeline_wait_limit_ns(limit)
        try:
            F.ft_moe_experts_mx4(shape, T, weights, x, off, inv, o, ws)
            if limit:
                with pytest.raises(F.FtError) as ei:
                    F.ft_moe_check(ws)
                assert ei.value.status == F.FT_ERR_DEVICE_CHECK
            else:
                F.ft_moe_check(ws)
        finally:
            F.ft_set_pipeline_wait_limit_ns(prev)
        outs.append(o)
    assert torch.equal(outs[0].view(torch.int16), outs[2].view(torch.int16))


def test_two_layers_on_two_streams_with_a_workspace_each():
    import torch
    g = np.random.default_rng(33)
    T, H, Fd, E, k = 200, 512, 256, 16, 4
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    runs = []
    for i in range(2):
        w, d, weights = layer_weights(g, E, 0, H, Fd)
        x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
        wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.02).cuda()
        ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
        y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws)
        F.ft_moe_check(ws)
        runs.append((x, wr, weights, ws, y, y.clone(), d))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (x, wr, weights, ws, y, want, d) in zip(streams, runs):
            F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws, stream=st)
    torch.cuda.synchronize()
    for x, wr, weights, ws, y, want, d in runs:
        F.ft_moe_check(ws)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
