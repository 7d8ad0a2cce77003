"""The MXFP4 calls at the ends of their ranges and behind other work: gates from subnormal results of SiLU to the largest
finite values, more tokens and tiles than one grid or table holds, matrices past 2^31 elements, calls one behind another
and captured behind other streams."""
import numpy as np
import pytest

import mx4_util as M
from expert_offload_serving_router_b200 import ftmoe as F
from test_gpu_mx4 import cuda, new_ws, q_interval

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpu_util import ensure_built
    ensure_built()


# per 32-element block of h: gates sign x {0.5 .. 6} x 2^e, all with up = 2^u
GATES = [(s, e, u) for s, e, u in [
    (-1, -3, 0), (1, -3, 0), (-1, 1, 0), (1, 1, 0), (-1, 4, 0), (1, 4, 0), (-1, 4, 100), (-1, 5, 120),
    (-1, 7, 0), (1, 7, 0), (-1, 13, 0), (1, 13, 0), (-1, 13, 120), (-1, 20, 0), (1, 20, 0), (-1, 20, 120),
    (-1, 27, 0), (-1, 30, 0), (-1, 31, 120), (-1, 33, 0), (1, 33, 0), (-1, 40, 0), (-1, 66, 120), (1, 66, 10),
    (-1, 100, 0), (1, 100, 0), (-1, 125, 0), (-1, 125, 120), (1, 125, -10), (1, 123, 0), (-1, 6, 90), (1, 6, 90)]]


@pytest.mark.parametrize("T", [1, 700, 4000])      # a tile of 32 rows, of 96, of a pair
def test_experts_mx4_gates_of_every_size(T):
    """x = (1, 0, ...) and one nonzero weight a row, so that every gate is exact; W2 = the identity, so that o is h's
    MXFP4 form.  h = silu(gate) up to a few fp32 roundings, 2^-20, and what the kernel flushes: below 2^-116."""
    import torch
    E, k, nb = 1, 1, len(GATES)
    Fd = 32 * nb
    H = Fd
    assert H % 128 == 0
    mag = np.resize(np.array([1, 2, 3, 4, 5, 6, 7], np.uint8), 32)          # codes of 0.5 1 1.5 2 3 4 6
    code13 = np.zeros((E, 2 * Fd, H), np.uint8)
    sc13 = np.full((E, 2 * Fd, H // 32), 127, np.uint8)
    gate, up = np.zeros(Fd), np.zeros(Fd)
    for b, (s, e, u) in enumerate(GATES):
        f = slice(32 * b, 32 * b + 32)
        code13[0, f, 0] = mag | (8 if s < 0 else 0)
        code13[0, Fd + 32 * b:Fd + 32 * b + 32, 0] = 2
        sc13[0, f, 0] = 127 + e
        sc13[0, Fd + 32 * b:Fd + 32 * b + 32, 0] = 127 + u
        gate[f] = s * M.GRID[mag] * 2.0 ** e
        up[f] = 2.0 ** u
    code2 = np.zeros((E, H, Fd), np.uint8)
    code2[0, np.arange(Fd), np.arange(Fd)] = 2
    d = [cuda(a) for a in (M.pack(code13), sc13, M.pack(code2), np.full((E, H, Fd // 32), 127, np.uint8))]
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    o = torch.full((T, H), 3.0, dtype=torch.bfloat16, device="cuda")
    off, inv = cuda(np.array([0, T], np.int32)), cuda(np.arange(T, dtype=np.int32))
    F.ft_moe_experts_mx4(shape, T, F.make_weights(*d), x, off, inv, o, ws)
    F.ft_moe_check(ws)
    with np.errstate(over="ignore"):
        h = (M.silu(gate) * up)[None]
    assert np.abs(h).max() < 3.4e38
    want, far = q_interval(h, 2.0 ** -20 * np.abs(h) + 2.0 ** -116)
    assert (far[0] <= 2.0 ** -114).mean() > 0.9                             # hardly any value near a rounding border
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} of {got.size} are not finite"
    bad = ~(np.abs(got - want) <= far + 2.0 ** -116)
    assert not bad.any(), f"first at {np.argwhere(bad)[0]}: {got[bad][:4]}"


# ------------------------------------------------------------------ one call behind another, no wait in between
def _consumer(g, wdtype, T, H, Fd, E, k):
    """ft_moe_experts on its GEMV path, with routing made beforehand: (x, call(o))."""
    import torch
    shape = F.make_shape(H, Fd, E, k, 0, wdtype)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    if wdtype == F.FT_W_MXFP4:
        q13, q2 = M.random_weights(g, E, 2 * Fd, H), M.random_weights(g, E, H, Fd)
        d = [cuda(a) for a in (*q13, *q2)]
        weights = F.make_weights(*d)
    else:
        d = [torch.from_numpy(g.standard_normal(s) * 0.05).to(torch.bfloat16).cuda() for s in ((E, 2 * Fd, H), (E, H, Fd))]
        weights = F.make_weights(d[0], None, d[1], None)
    idx = cuda(np.stack([g.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32))
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    off, sf, inv = i32(E + 1), i32(T * k), i32(T * k)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_permute(shape, T, idx, None, off, sf, inv, None, ws)
    F.ft_moe_check(ws)

    def call(o):
        F.ft_moe_experts(shape, T, weights, x, None, off, sf, o, ws)
    call.keep = (d, off, sf, inv, ws)
    return x, call


def _producer(g, kind, T, H, x):
    """A call that writes x [T, H] and lets the kernel behind it start before it is done."""
    import torch
    if kind == "product":
        K = 8192
        code, scale = M.quantize(g.standard_normal((T, K)))
        wc, wsc = M.random_weights(g, 1, H, K, lo=115, hi=119)
        a = [cuda(v) for v in (np.array([0, T], np.int32), M.pack(code), scale, wc, wsc)]
        ws = new_ws()
        return lambda: F.ft_mx4_product(1, T, H, K, *a, x, ws)
    E, k, Fd = 16, 4, 1024
    # x of a size that keeps the consumer's h inside the f16 range which MXFP4 GEMVs on bf16 activations document
    d = [cuda(a) for a in (*M.random_weights(g, E, 2 * Fd, H, lo=115, hi=119), *M.random_weights(g, E, H, Fd, lo=115, hi=119))]
    weights = F.make_weights(*d)
    z = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    if kind == "experts_mx4":
        shape = F.make_shape(H, Fd, E, 1, 0, F.FT_W_MXFP4)
        ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
        off, inv = np.zeros(E + 1, np.int32), cuda(np.arange(T, dtype=np.int32))
        off[1:] = T
        off = cuda(off)
        keep = (d, z, ws, off, inv)
        return lambda: keep and F.ft_moe_experts_mx4(shape, T, weights, z, off, inv, x, ws)
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.02).cuda()
    fn = {"layer": F.ft_moe_layer_forward, "layer_mx4": F.ft_moe_layer_forward_mx4}[kind]
    keep = (d,)
    return lambda: keep and fn(shape, T, z, wr, None, weights, x, None, None, ws)


@pytest.mark.parametrize("kind", ["product", "experts_mx4", "layer", "layer_mx4"])
@pytest.mark.parametrize("wdtype", [F.FT_W_BF16, F.FT_W_MXFP4])
@pytest.mark.parametrize("T", [1, 3])
def test_experts_read_what_the_call_before_them_wrote(T, wdtype, kind):
    """ft_moe_experts on x straight behind the call that writes x: the same bits as with a wait in between, each time with
    other contents in x before."""
    import torch
    g = np.random.default_rng(T + 10 * wdtype)
    H, Fd, E, k = 2048, 512, 8, 2
    x, experts = _consumer(g, wdtype, T, H, Fd, E, k)
    produce = _producer(g, kind, T, H, x)
    want = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    produce()
    torch.cuda.synchronize()
    experts(want)
    torch.cuda.synchronize()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    outs = [torch.empty_like(want) for _ in range(20)]
    for i, o in enumerate(outs):
        x.fill_(float(i + 1))
        produce()
        experts(o)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------ more tokens than a grid's second dimension holds
def _check_combine(y, o, inv, gw, T, k, S):
    """y against the 64-bit combine of the rows o: one bf16 rounding and k + S + 1 fp32 ones."""
    for lo in range(0, T, 16384):
        hi = min(T, lo + 16384)
        terms = o[inv[lo * k:hi * k].long()].double().view(hi - lo, k, -1) * gw[lo:hi].double()[..., None]
        want, mag = terms.sum(1), terms.abs().sum(1)
        if S:
            sh = o[inv[T * k + lo:T * k + hi].long()].double()
            want, mag = want + sh, mag + sh.abs()
        assert ((y[lo:hi].double() - want).abs() <= M.UB16 * want.abs() + 2 * (k + S + 1) * M.U32 * mag).all()


@pytest.mark.parametrize("T,H,k,S", [(65535, 128, 2, 1), (65536, 128, 2, 1), (70001, 128, 3, 0), (65537, 2176, 2, 0)])
def test_combine_beyond_65535_tokens(T, H, k, S):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(T)
    R = T * (k + S)
    o = torch.randn(R, H, device="cuda", generator=gen).to(torch.bfloat16)
    inv = torch.randperm(R, device="cuda", generator=gen).to(torch.int32)
    gw = torch.rand(T, k, device="cuda", generator=gen)
    y = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_combine(F.make_shape(H, 64, 8, k, S), T, o, inv, gw, y)
    torch.cuda.synchronize()
    assert (y[T] == 3.0).all()
    _check_combine(y[:T], o, inv, gw, T, k, S)


@pytest.mark.parametrize("T,S", [(65536, 1), (66001, 0)])
def test_layer_forward_mx4_beyond_65535_tokens(T, S):
    """The layer call = its steps bit for bit, and the combine of their rows in 64 bits."""
    import torch
    g = np.random.default_rng(T)
    H, Fd, E, k = 128, 64, 8, 2
    d = [cuda(a) for a in (*M.random_weights(g, E, 2 * Fd, H), *M.random_weights(g, E, H, Fd))]
    sh = [cuda(a) for a in (*M.random_weights(g, 1, 2 * Fd, H), *M.random_weights(g, 1, H, Fd))] if S else []
    weights = F.make_weights(*d, None, *sh)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.1).cuda()
    shape = F.make_shape(H, Fd, E, k, S, F.FT_W_MXFP4)
    R = T * (k + S)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    y = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws)
    F.ft_moe_check(ws)
    assert (y[T] == 3.0).all()
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, gw, off, sf, inv = i32(T, k), torch.empty(T, k, device="cuda"), i32(E + S + 1), i32(R), i32(R)
    o, y2 = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_route(shape, T, x, wr, None, idx, gw, None, ws)
    F.ft_moe_permute(shape, T, idx, None, off, sf, inv, None, ws)
    F.ft_moe_experts_mx4(shape, T, weights, x, off, inv, o, ws)
    F.ft_moe_combine(shape, T, o, inv, gw, y2)
    F.ft_moe_check(ws)
    assert torch.equal(y[:T].view(torch.int16), y2.view(torch.int16))
    _check_combine(y[:T], o, inv, gw, T, k, S)


def test_layer_forward_beyond_65535_tokens():
    """The bf16 layer on the same grid: its last tokens equal the same tokens in a call of their own, up to the order in
    which the router's K splits are added (their number goes by T)."""
    import torch
    g = np.random.default_rng(5)
    T, H, Fd, E, k = 65600, 128, 64, 8, 2
    d = [torch.from_numpy(g.standard_normal(s) * 0.1).to(torch.bfloat16).cuda() for s in ((E, 2 * Fd, H), (E, H, Fd))]
    weights = F.make_weights(d[0], None, d[1], None)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32) * 0.1).cuda()
    shape = F.make_shape(H, Fd, E, k)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    y, few = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(1000, H, dtype=torch.bfloat16, device="cuda")
    idx, idx2 = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(1000, k, dtype=torch.int32, device="cuda")
    F.ft_moe_layer_forward(shape, T, x, wr, None, weights, y, idx, None, ws)
    F.ft_moe_check(ws)
    F.ft_moe_layer_forward(shape, 1000, x[-1000:], wr, None, weights, few, idx2, None, ws)
    F.ft_moe_check(ws)
    same = (idx[-1000:] == idx2).all(1)
    assert same.float().mean() > 0.99                                # two logits may swap within their last bits
    diff = (y[-1000:].float() - few.float()).abs()[same]
    # gates a few fp32 roundings apart: at most a neighbouring bf16 value
    assert (diff <= 2 * M.UB16 * torch.maximum(y[-1000:].float().abs(), few.float().abs())[same] + 1e-6).all()


# ------------------------------------------------------------------ more tiles than a CTA works out ahead
def _decode(codes, scales):
    """Codes [..., cols / 2] and scale bytes [..., cols / 32] on the device -> fp64 values."""
    import torch
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


# 148 CTAs (74 pairs) take 258 tiles each: 256 of them from the table, the others decoded in the roles' loops
@pytest.mark.parametrize("sizes,n", [([1] * 256, 19072), ([60] * 256, 19072), ([10299, 10304, 10311], 35328)])
def test_product_more_tiles_than_the_table(sizes, n):
    import torch
    k, G, rows = 64, len(sizes), sum(sizes)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    byte = lambda *s, lo=0, hi=256: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    ac, asc = byte(rows, k // 2), byte(rows, k // 32, lo=120, hi=130)
    wc, wsc = byte(G, n, k // 2), byte(G, n, k // 32, lo=119, hi=124)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    out = torch.full((rows + 1, n), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = new_ws()
    F.ft_mx4_product(G, rows, n, k, cuda(off), ac, asc, wc, wsc, out, ws)
    F.ft_moe_check(ws)
    assert (out[rows] == 3.0).all()
    for g in range(G):
        w = _decode(wc[g], wsc[g])
        for lo in range(off[g], off[g + 1], 2048):
            hi = min(off[g + 1], lo + 2048)
            a = _decode(ac[lo:hi], asc[lo:hi])
            want = a @ w.t()
            tol = M.UB16 * want.abs() + M.sum_bound(k) * (a.abs() @ w.abs().t())
            assert ((out[lo:hi].double() - want).abs() <= tol).all(), (g, lo)


def test_quantize_beyond_2_31_elements():
    """The last rows of a matrix of 2.15e9 elements: as quantised on their own."""
    import torch
    rows, cols, n = 524800, 4096, 700
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:n].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    for lo in range(n, rows, n):
        x[lo:lo + n] = x[:min(n, rows - lo)]
    x[-n:] *= 3
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    vals = torch.empty_like(x)
    F.ft_mx4_quantize(rows, cols, F.FT_T_BF16, x, cols, codes, scales, vals)
    for at in (0, rows // 2, rows - n):
        c, s, v = torch.empty_like(codes[:n]), torch.empty_like(scales[:n]), torch.empty_like(vals[:n])
        F.ft_mx4_quantize(n, cols, F.FT_T_BF16, x[at:at + n], cols, c, s, v)
        assert torch.equal(c, codes[at:at + n]) and torch.equal(s, scales[at:at + n]) and torch.equal(v, vals[at:at + n])


@pytest.mark.parametrize("rows", [40, 3000])
@pytest.mark.parametrize("before", ["nothing", "memset", "another stream", "memset and another stream"])
def test_calls_captured_behind_other_work(before, rows):
    """The MXFP4 calls as programmatic dependents of what a capture may hold before them: the same bits as eagerly."""
    import torch
    g = np.random.default_rng(rows)
    H, Fd, E, k = 256, 128, 4, 2
    T = rows // 2
    d = [cuda(a) for a in (*M.random_weights(g, E, 2 * Fd, H), *M.random_weights(g, E, H, Fd))]
    weights = F.make_weights(*d)
    shape = F.make_shape(H, Fd, E, k, 0, F.FT_W_MXFP4)
    ws = new_ws(F.ft_moe_workspace_bytes(shape, T))
    src = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    x = torch.zeros_like(src)
    idx = np.stack([g.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    off, sf, inv = i32(E + 1), i32(T * k), i32(T * k)
    F.ft_moe_permute(shape, T, cuda(idx), None, off, sf, inv, None, ws)
    o = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    wr = torch.from_numpy(g.standard_normal((E, H)).astype(np.float32)).cuda()
    y = torch.empty_like(src)
    ac, asc = cuda(M.random_weights(g, rows, H)[0]), cuda(M.random_weights(g, rows, H)[1])
    out = torch.empty(rows, 2 * Fd, dtype=torch.bfloat16, device="cuda")
    goff = cuda(np.array([0, rows // 3, rows // 3, rows - 1, rows], np.int32))
    pad = torch.ones(1 << 20, device="cuda")
    ws_p = new_ws()
    calls = [
        lambda: F.ft_moe_experts_mx4(shape, T, weights, x, off, inv, o, ws),
        lambda: F.ft_mx4_product(E, rows, 2 * Fd, H, goff, ac, asc, d[0], d[1], out, ws_p),
        lambda: F.ft_moe_layer_forward_mx4(shape, T, x, wr, None, weights, y, None, None, ws),
    ]
    results = [o, out, y]
    for call, res in zip(calls, results):
        x.copy_(src)
        call()
        F.ft_moe_check(ws)
        F.ft_moe_check(ws_p)
        want = res.clone()
        res.zero_()
        x.zero_()
        st, side = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            if "stream" in before:
                side.wait_stream(st)
                with torch.cuda.stream(side):
                    pad.mul_(1.0)
                    x.copy_(src)
            if "memset" in before:
                pad.zero_()
            if "stream" in before:
                st.wait_stream(side)
            call()
        if "stream" not in before:
            x.copy_(src)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        F.ft_moe_check(ws)
        F.ft_moe_check(ws_p)
        assert torch.equal(res.view(torch.int16), want.view(torch.int16))
