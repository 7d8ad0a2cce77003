"""GPU parity of the gradients of the router, the permutation and the combine: against the formulas in 64 bits,
against differences of the 64-bit forward, and as one chain against automatic differentiation in 64 bits.

Tolerances count roundings: fp32 sums of n terms n * 2^-24 of the sum of absolute terms, one bf16 rounding 2^-8 of
the value."""
import numpy as np
import pytest

import mx4_util as M
from expert_offload_serving_router_b200 import ftmoe as F

pytestmark = pytest.mark.gpu

CASES = [(1, 128, 1, 1, 0), (1, 2048, 128, 8, 1), (3, 256, 4, 2, 1), (7, 4096, 256, 6, 0), (33, 512, 8, 8, 0),
         (100, 1152, 40, 5, 1), (513, 384, 5, 1, 0), (1500, 128, 16, 3, 1), (2049, 640, 128, 8, 0),
         (2100, 256, 7, 3, 1), (2301, 128, 256, 6, 1)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gpu_util import ensure_built
    ensure_built()


def setup(T, H, E, k, S, seed=0, skew=1.5, dup=False):
    """Seeded routing through the library's own permutation."""
    import torch
    g = np.random.default_rng(1000 * seed + T + H + E)
    p = np.exp(-skew * np.log1p(g.permutation(E)))
    p /= p.sum()
    p = 0.5 * p + 0.5 / E
    idx = np.stack([g.choice(E, size=k, replace=dup, p=p) for _ in range(T)]).astype(np.int32)
    gates = g.random((T, k)).astype(np.float32) + 0.05
    gates /= gates.sum(1, keepdims=True)
    shape = F.make_shape(H, 64, E, k, S)
    R = T * (k + S)
    ws = torch.empty(F.ft_moe_workspace_bytes(shape, T), dtype=torch.uint8, device="cuda")
    F.ft_moe_workspace_init(ws)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(shape=shape, T=T, H=H, E=E, k=k, S=S, R=R, g=g, ws=ws, idx=torch.from_numpy(idx).cuda(),
             gates=torch.from_numpy(gates).cuda(), off=i32(E + S + 1), sf=i32(R), inv=i32(R))
    F.ft_moe_permute(shape, T, s["idx"], None, s["off"], s["sf"], s["inv"], None, ws)
    F.ft_moe_check(ws)
    return s


def normal(s, *shape, std=1.0):
    import torch
    return torch.from_numpy(s["g"].standard_normal(shape) * std).to(torch.bfloat16).cuda()


def combine_backward(s, dy, o, want_o=True, want_w=True):
    import torch
    d_o = torch.full((s["R"] + 1, s["H"]), 3.0, dtype=torch.bfloat16, device="cuda") if want_o else None
    d_w = torch.full((s["T"] + 1, s["k"]), 3.0, device="cuda") if want_w else None
    F.ft_moe_combine_backward(s["shape"], s["T"], dy, o, s["inv"], s["gates"], d_o, d_w)
    torch.cuda.synchronize()
    assert d_o is None or (d_o[s["R"]] == 3.0).all()
    assert d_w is None or (d_w[s["T"]] == 3.0).all()
    return d_o[:s["R"]] if want_o else None, d_w[:s["T"]] if want_w else None


@pytest.mark.parametrize("T,H,E,k,S", CASES)
def test_combine_backward(T, H, E, k, S):
    import torch
    s = setup(T, H, E, k, S)
    dy, o = normal(s, T, H, std=0.1), normal(s, s["R"], H)
    d_o, d_w = combine_backward(s, dy, o)
    pos = s["inv"].long()
    routed = pos[:T * k].view(T, k)
    want = torch.empty_like(d_o)
    want[routed] = (s["gates"][..., None] * dy.float()[:, None]).to(torch.bfloat16)   # one fp32 product, one rounding: exact
    if S:
        want[pos[T * k:]] = dy
    assert torch.equal(d_o.view(torch.int16), want.view(torch.int16))
    terms = o.double()[routed] * dy.double()[:, None]
    assert ((d_w.double() - terms.sum(-1)).abs() <= H * M.U32 * terms.abs().sum(-1)).all()
    only_o, _ = combine_backward(s, dy, None, want_w=False)
    _, only_w = combine_backward(s, dy, o, want_o=False)
    assert torch.equal(only_o.view(torch.int16), d_o.view(torch.int16)) and torch.equal(only_w, d_w)


def permute_backward(s, dxs, dl=None, wr=None):
    import torch
    dx = torch.full((s["T"] + 1, s["H"]), 3.0, dtype=torch.bfloat16, device="cuda")
    F.ft_moe_permute_backward(s["shape"], s["T"], dxs, s["inv"], None if dl is None else s["idx"], dl, wr, dx)
    torch.cuda.synchronize()
    assert (dx[s["T"]] == 3.0).all()
    return dx[:s["T"]]


@pytest.mark.parametrize("router", [False, True])
@pytest.mark.parametrize("T,H,E,k,S", CASES)
def test_permute_backward(T, H, E, k, S, router):
    import torch
    s = setup(T, H, E, k, S)
    dxs = normal(s, s["R"], H)
    dl = wr = None
    pos = s["inv"].long()
    terms = dxs.double()[pos[:T * k]].view(T, k, H)
    if S:
        terms = torch.cat([terms, dxs.double()[pos[T * k:]][:, None]], 1)
    if router:
        dl = torch.from_numpy(s["g"].standard_normal((T, k)).astype(np.float32)).cuda()
        wr = torch.from_numpy(s["g"].standard_normal((E, H)).astype(np.float32)).cuda()
        terms = torch.cat([terms, dl.double()[..., None] * wr.double()[s["idx"].long()]], 1)
    dx = permute_backward(s, dxs, dl, wr)
    want = terms.sum(1)
    tol = M.UB16 * want.abs() + (terms.shape[1] + 1) * M.U32 * (1 + M.UB16) * terms.abs().sum(1)
    assert ((dx.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("T,H,E,k,S", [(4600, 4096, 256, 8, 1), (6900, 4096, 7, 5, 1), (16500, 1280, 33, 8, 0), (27400, 1024, 64, 6, 0),
                                       (164001, 128, 8, 8, 0)])
def test_permute_backward_rows_beyond_the_cache(T, H, E, k, S):
    """dx_sorted above 320 MB: the form with W_r's slice in shared memory; a few tokens of it alone (the other form) give
    the same bits."""
    import torch
    s = setup(T, H, E, k, S)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dxs = torch.randn(s["R"], H, device="cuda", generator=gen).to(torch.bfloat16)
    dl, wr = torch.randn(T, k, device="cuda", generator=gen), torch.randn(E, H, device="cuda", generator=gen)
    dx = permute_backward(s, dxs, dl, wr)
    pos = s["inv"].long()
    for lo in range(0, T, 20000):
        hi = min(T, lo + 20000)
        terms = dxs.double()[pos[lo * k:hi * k]].view(hi - lo, k, H)
        if S:
            terms = torch.cat([terms, dxs.double()[pos[T * k + lo:T * k + hi]][:, None]], 1)
        terms = torch.cat([terms, dl[lo:hi].double()[..., None] * wr.double()[s["idx"][lo:hi].long()]], 1)
        want, mag = terms.sum(1), terms.abs().sum(1)
        tol = M.UB16 * want.abs() + (terms.shape[1] + 1) * M.U32 * (1 + M.UB16) * mag
        assert ((dx[lo:hi].double() - want).abs() <= tol).all()
    n, at = 50, T - 57
    few = dict(s, T=n, shape=F.make_shape(H, 64, E, k, S))
    few["idx"] = s["idx"][at:at + n].contiguous()
    few["inv"] = torch.arange(n * (k + S), dtype=torch.int32, device="cuda")
    rows = torch.cat([pos[at * k:(at + n) * k]] + ([pos[T * k + at:T * k + at + n]] if S else []))
    alone = permute_backward(few, dxs[rows].contiguous(), dl[at:at + n].contiguous(), wr)
    assert torch.equal(alone.view(torch.int16), dx[at:at + n].view(torch.int16))


@pytest.mark.parametrize("H", [128, 384, 1024, 1280, 2816])
@pytest.mark.parametrize("T", [256, 257, 1025])
@pytest.mark.parametrize("k,S", [(1, 0), (2, 1), (3, 0), (5, 1), (6, 0), (7, 1)])
def test_combine_backward_warps_per_token(T, H, k, S):
    """Both sides of the bounds on tokens, columns and k that choose how many warps take a token and how many slots they hold."""
    import torch
    s = setup(T, H, 9, k, S)
    dy, o = normal(s, T, H, std=0.1), normal(s, s["R"], H)
    d_o, d_w = combine_backward(s, dy, o)
    pos = s["inv"].long()
    routed = pos[:T * k].view(T, k)
    want = torch.empty_like(d_o)
    want[routed] = (s["gates"][..., None] * dy.float()[:, None]).to(torch.bfloat16)
    if S:
        want[pos[T * k:]] = dy
    assert torch.equal(d_o.view(torch.int16), want.view(torch.int16))
    terms = o.double()[routed] * dy.double()[:, None]
    assert ((d_w.double() - terms.sum(-1)).abs() <= H * M.U32 * terms.abs().sum(-1)).all()


def route_backward(s, x, dg, want_w=True, want_b=True):
    import torch
    E, H, T, k = s["E"], s["H"], s["T"], s["k"]
    dl = torch.full((T + 1, k), 3.0, device="cuda")
    dw = torch.full((E + 1, H), 3.0, device="cuda") if want_w else None
    db = torch.full((E + 1,), 3.0, device="cuda") if want_b else None
    F.ft_moe_route_backward(s["shape"], T, x, s["idx"], s["gates"], dg, s["off"], s["sf"], dl, dw, db, s["ws"])
    F.ft_moe_check(s["ws"])
    assert (dl[T] == 3.0).all() and (dw is None or (dw[E] == 3.0).all()) and (db is None or db[E] == 3.0)
    return dl[:T], dw[:E] if want_w else None, db[:E] if want_b else None


def check_route_backward(s, x, dg, dl, dw, db):
    import torch
    E, k = s["E"], s["k"]
    gd, dd = s["gates"].double(), dg.double()
    sm = (gd * dd).sum(1, keepdim=True)
    want = gd * (dd - sm)
    # s: k products and sums; the difference and the last product round once each
    e_dl = (k + 3) * M.U32 * gd * (dd.abs() + (gd * dd).abs().sum(1, keepdim=True))
    assert ((dl.double() - want).abs() <= e_dl).all()
    onehot = torch.nn.functional.one_hot(s["idx"].long(), E).double()        # [T, k, E]
    dense, e_dense, mag = ((onehot * v[..., None]).sum(1) for v in (want, e_dl, want.abs()))
    n = onehot.sum((0, 1))                                                    # pairs per expert
    if dw is not None:
        xd = x.double()
        tol = e_dense.t() @ xd.abs() + (n[:, None] + 2) * M.U32 * (mag.t() @ xd.abs())
        assert ((dw.double() - dense.t() @ xd).abs() <= tol).all()
        assert (dw[n == 0] == 0).all()
    if db is not None:
        assert ((db.double() - dense.sum(0)).abs() <= e_dense.sum(0) + (n + 2) * M.U32 * mag.sum(0)).all()
        assert (db[n == 0] == 0).all()


@pytest.mark.parametrize("T,H,E,k,S", CASES)
def test_route_backward(T, H, E, k, S):
    import torch
    s = setup(T, H, E, k, S)
    x = normal(s, T, H)
    dg = torch.from_numpy(s["g"].standard_normal((T, k)).astype(np.float32)).cuda()
    dl, dw, db = route_backward(s, x, dg)
    check_route_backward(s, x, dg, dl, dw, db)
    dl2, dw2, _ = route_backward(s, x, dg, want_b=False)
    dl3, _, db3 = route_backward(s, None, dg, want_w=False)
    dl4, _, _ = route_backward(s, None, dg, want_w=False, want_b=False)
    assert torch.equal(dw2, dw) and torch.equal(db3, db)
    assert torch.equal(dl2, dl) and torch.equal(dl3, dl) and torch.equal(dl4, dl)


@pytest.mark.parametrize("T", [5, 700, 4000])
def test_route_backward_one_busy_expert_and_repeated_index(T):
    """Every pair of most tokens on the same expert (the same index twice in a token): one sum over many segments."""
    import torch
    s = setup(T, 256, 6, 5, 0, seed=3, skew=6.0, dup=True)
    x = normal(s, T, 256)
    dg = torch.from_numpy(s["g"].standard_normal((T, 5)).astype(np.float32)).cuda()
    check_route_backward(s, x, dg, *route_backward(s, x, dg))
    a, b = route_backward(s, x, dg), route_backward(s, x, dg)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    dy, o = normal(s, T, 256), normal(s, s["R"], 256)
    d_o, d_w = combine_backward(s, dy, o)
    terms = o.double()[s["inv"].long()].view(T, 5, 256) * dy.double()[:, None]
    assert ((d_w.double() - terms.sum(-1)).abs() <= 256 * M.U32 * terms.abs().sum(-1)).all()


def test_route_backward_no_tokens_gives_zeros():
    import torch
    shape = F.make_shape(256, 64, 8, 2)
    dw, db = torch.ones(8, 256, device="cuda"), torch.ones(8, device="cuda")
    F.ft_moe_route_backward(shape, 0, None, None, None, None, None, None, None, dw, db, None, 0)
    assert not dw.any() and not db.any()


def test_nan_and_inf_stay_where_they_are():
    import torch
    T, H, E, k = 20, 256, 8, 2
    s = setup(T, H, E, k, 1)
    dy, o = normal(s, T, H), normal(s, s["R"], H)
    dy[4, 9] = float("nan")
    o[s["inv"][7 * k].long(), 3] = float("inf")
    d_o, d_w = combine_backward(s, dy, o)
    assert torch.isnan(d_w[4]).all() and not torch.isfinite(d_w[7, 0])
    rest = torch.ones(T, k, dtype=torch.bool, device="cuda")
    rest[4] = False
    rest[7, 0] = False
    assert torch.isfinite(d_w[rest]).all()
    assert int(torch.isnan(d_o).sum()) == k + 1                 # one column of token 4's rows
    dxs = normal(s, s["R"], H)
    dxs[s["inv"][11 * k + 1].long(), 0] = float("nan")
    dx = permute_backward(s, dxs)
    assert int(torch.isnan(dx).sum()) == 1 and torch.isnan(dx[11, 0])


def test_dropped_pair_contributes_nothing():
    """A position outside [0, R) is the kernels' own bounds check."""
    import torch
    T, H, E, k = 6, 256, 4, 2
    s = setup(T, H, E, k, 0)
    dy, o, dxs = normal(s, T, H), normal(s, s["R"], H), normal(s, s["R"], H)
    d_o, d_w = combine_backward(s, dy, o)
    gone = int(s["inv"][2 * k + 1])
    for bad in (-1, s["R"], 2 ** 31 - 1):
        s["inv"][2 * k + 1] = bad
        d_o2, d_w2 = combine_backward(s, dy, o)
        assert d_w2[2, 1] == 0 and (d_o2[gone] == 3.0).all()
        keep = torch.arange(s["R"], device="cuda") != gone
        assert torch.equal(d_o2[keep], d_o[keep])
        dx = permute_backward(s, dxs)
        assert torch.equal(dx[2], dxs[int(s["inv"][2 * k])])


def test_differences_of_the_forward():
    """Directional derivatives of L = <dy, combine(o, softmax(kept logits))> and of the gather, from central differences of
    the 64-bit forward, against the kernels' gradients."""
    import torch
    T, H, E, k, S = 12, 256, 6, 3, 1
    s = setup(T, H, E, k, S, seed=9)
    g = torch.Generator().manual_seed(0)
    logits = torch.randn(T, k, generator=g, dtype=torch.float64).cuda()
    s["gates"] = torch.softmax(logits, 1).float()
    dy, o = normal(s, T, H), normal(s, s["R"], H)
    pos = s["inv"].long()

    def loss(lg, rows):
        y = (torch.softmax(lg, 1)[..., None] * rows[pos[:T * k]].view(T, k, H)).sum(1) + rows[pos[T * k:]]
        return float((y * dy.double()).sum())
    d_o, d_w = combine_backward(s, dy, o)
    dl, _, _ = route_backward(s, None, d_w, want_w=False, want_b=False)
    eps = 1e-5
    for i in range(4):
        v = torch.randn(T, k, generator=g, dtype=torch.float64).cuda()
        fd = (loss(logits + eps * v, o.double()) - loss(logits - eps * v, o.double())) / (2 * eps)
        an = float((dl.double() * v).sum())
        # the difference's own error is O(eps^2); gates in fp32 (2^-24) and H-term dots: a few 1e-6 of the terms' sizes
        assert abs(fd - an) <= 1e-5 * float((dl.double() * v).abs().sum()) + 1e-5 * float(dy.double().norm())
        u = torch.randn(s["R"], H, generator=g, dtype=torch.float64).cuda()
        fd = (loss(logits, o.double() + eps * u) - loss(logits, o.double() - eps * u)) / (2 * eps)
        an = float((d_o.double() * u).sum())
        assert abs(fd - an) <= 2 * M.UB16 * float((d_o.double() * u).abs().sum()) / np.sqrt(s["R"] * H) * 8 + 1e-5 * float(dy.double().norm())


@pytest.mark.parametrize("T,S", [(5, 0), (40, 1), (300, 1)])
def test_chain_against_automatic_differentiation(T, S):
    """route -> permute -> experts -> combine with MXFP4 fake-quantised activations (straight-through), backwards through
    the library: dx, dW_r and db against torch's automatic differentiation in 64 bits of the same formula.  The experts are a
    square matrix each, differentiated by the caller (torch), so every intermediate the kernels read is bf16."""
    import torch
    H, E, k = 256, 8, 3
    s = setup(T, H, E, k, S, seed=T)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr = (0.3 * torch.randn(E, H, generator=g)).cuda()
    bias = torch.randn(E, generator=g).cuda()
    dy = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    we = (torch.randn(E + S, H, H, generator=g) / 16).to(torch.bfloat16).cuda()
    ws, shape, R = s["ws"], s["shape"], s["R"]
    gates = torch.empty(T, k, device="cuda")
    F.ft_moe_route(shape, T, x, wr, bias, s["idx"], gates, None, ws)
    F.ft_moe_permute(shape, T, s["idx"], x, s["off"], s["sf"], s["inv"], None, ws)
    F.ft_moe_check(ws)
    s["gates"] = gates
    codes = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    xq = torch.empty_like(x)
    F.ft_mx4_quantize(T, H, F.FT_T_BF16, x, H, codes, scales, xq)
    sf = s["sf"].long()
    tok = torch.where(sf < T * k, sf // k, sf - T * k)
    grp = torch.where(sf < T * k, s["idx"].view(-1).long()[sf.clamp(max=T * k - 1)], torch.full_like(sf, E))
    o = torch.bmm(we[grp].float(), xq[tok].float()[..., None])[..., 0].to(torch.bfloat16)
    y = torch.empty_like(x)
    F.ft_moe_combine(shape, T, o, s["inv"], gates, y)
    d_o, d_w = combine_backward(s, dy, o)
    dxs = torch.bmm(we[grp].float().transpose(1, 2), d_o.float()[..., None])[..., 0].to(torch.bfloat16)
    dl, dw, db = route_backward(s, x, d_w)
    dx = permute_backward(s, dxs, dl, wr)
    # the same in 64 bits, the experts' output as the bf16 rows the kernels saw (its rounding is the caller's)
    x64 = x.double().requires_grad_()
    wr64, b64 = wr.double().requires_grad_(), bias.double().requires_grad_()
    lg = (x64 @ wr64.t() + b64).gather(1, s["idx"].long())
    g64 = torch.softmax(lg, 1)
    xq64 = x64 + (xq.double() - x64).detach()                           # straight-through
    o64 = torch.bmm(we.double()[grp], xq64[tok][..., None])[..., 0]
    o64 = o64 + (o.double() - o64).detach()
    pos = s["inv"].long()
    y64 = (g64[..., None] * o64[pos[:T * k]].view(T, k, H)).sum(1)
    if S:
        y64 = y64 + o64[pos[T * k:]]
    (y64 * dy.double()).sum().backward()
    # gates: fp32 softmax of fp32 logits, a few 1e-6; d_o, dxs and dx are bf16: three roundings of 2^-8 each in the norm
    assert ((y.double() - y64).norm() / y64.norm()).item() <= 2 * M.UB16
    assert ((dx.double() - x64.grad).norm() / x64.grad.norm()).item() <= 3 * M.UB16
    assert ((dw.double() - wr64.grad).norm() / wr64.grad.norm()).item() <= 2e-5
    assert ((db.double() - b64.grad).norm() / b64.grad.norm()).item() <= 2e-5


def test_backward_captured_in_a_graph():
    import torch
    s = setup(70, 512, 16, 4, 1)
    x, dy, o, dxs = normal(s, 70, 512), normal(s, 70, 512), normal(s, s["R"], 512), normal(s, s["R"], 512)
    wr = torch.randn(16, 512, device="cuda")
    d_o, d_w = torch.empty(s["R"], 512, dtype=torch.bfloat16, device="cuda"), torch.empty(70, 4, device="cuda")
    dl, dw, db, dx = torch.empty(70, 4, device="cuda"), torch.empty(16, 512, device="cuda"), torch.empty(16, device="cuda"), torch.empty_like(x)

    def step():
        F.ft_moe_combine_backward(s["shape"], 70, dy, o, s["inv"], s["gates"], d_o, d_w)
        F.ft_moe_route_backward(s["shape"], 70, x, s["idx"], s["gates"], d_w, s["off"], s["sf"], dl, dw, db, s["ws"])
        F.ft_moe_permute_backward(s["shape"], 70, dxs, s["inv"], s["idx"], dl, wr, dx)
    step()
    want = [t.clone() for t in (d_o, d_w, dl, dw, db, dx)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for t in (d_o, d_w, dl, dw, db, dx):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (d_o, d_w, dl, dw, db, dx)))


@pytest.mark.parametrize("k", [8, 6, 5])
def test_routing_arrays_off_their_alignment(k):
    """inv_pos, gates, experts and logit gradients are plain int32 / fp32 arrays: any 4-byte aligned address."""
    import torch
    T, H, E, S = 50, 512, 16, 1
    s = setup(T, H, E, k, S)
    dy, o, dxs = normal(s, T, H), normal(s, s["R"], H), normal(s, s["R"], H)
    wr = torch.randn(E, H, device="cuda")
    dl = torch.randn(T, k, device="cuda")
    d_o, d_w = combine_backward(s, dy, o)
    dx = permute_backward(s, dxs, dl, wr)

    def moved(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)
    for name in ("inv", "gates", "idx"):
        s[name] = moved(s[name])
    d_o2, d_w2 = combine_backward(s, dy, o)
    dx2 = permute_backward(s, dxs, moved(dl), wr)
    assert torch.equal(d_o.view(torch.int16), d_o2.view(torch.int16)) and torch.equal(d_w, d_w2)
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16))


@pytest.mark.parametrize("T,H,k", [(6, 256, 2), (300, 512, 4), (2000, 256, 3), (1100, 1280, 5)])     # 8, 4, 1 and 8 warps a token
def test_dropped_pair_has_no_gradient_where_dy_is_not_finite(T, H, k):
    import torch
    s = setup(T, H, 8, k, 1)
    dy, o = normal(s, T, H), normal(s, s["R"], H)
    dy[2, 5], dy[3, 7], dy[4, 11] = float("inf"), float("nan"), float("-inf")
    for t in (2, 3, 4, 5):
        s["inv"][t * k + 1] = -1
    _, d_w = combine_backward(s, dy, o)
    _, only = combine_backward(s, dy, o, want_o=False)
    assert torch.equal(d_w.view(torch.int32), only.view(torch.int32))
    assert (d_w[2:6, 1] == 0).all()
    assert not torch.isfinite(d_w[2:5, 0]).any()
    assert torch.isfinite(d_w[5:]).all() and torch.isfinite(d_w[:2]).all()


def test_dropped_pair_keeps_the_routers_part():
    """The router's part of dx goes by topk_idx and dlogits alone: a dropped pair's logit still moves the other gates."""
    import torch
    T, H, E, k = 6, 256, 4, 2
    s = setup(T, H, E, k, 0)
    dxs = normal(s, s["R"], H)
    dl, wr = torch.randn(T, k, device="cuda"), torch.randn(E, H, device="cuda")
    s["inv"][2 * k + 1] = -1
    dx = permute_backward(s, dxs, dl, wr)
    terms = torch.cat([dxs.double()[int(s["inv"][2 * k])][None], dl[2].double()[:, None] * wr.double()[s["idx"][2].long()]])
    want, mag = terms.sum(0), terms.abs().sum(0)
    assert ((dx[2].double() - want).abs() <= M.UB16 * want.abs() + 4 * M.U32 * (1 + M.UB16) * mag).all()
