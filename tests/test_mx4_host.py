"""Host-side checks of the MXFP4 and gradient entry points (no GPU): arguments are refused with the
documented status before any CUDA call, empty calls need no pointers, workspace sizes."""
import numpy as np
import pytest

import mx4_util as M
from expert_offload_serving_router_b200 import build as ftbuild
from expert_offload_serving_router_b200 import ftmoe as F

FAKE = 1 << 20     # 256-byte aligned non-null address; never dereferenced (validation fails first)
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    ftbuild.build()


def refused(code, fn, *args, **kw):
    with pytest.raises(F.FtError) as ei:
        fn(*args, stream=0, **kw)
    assert ei.value.status == code, ei.value
    return str(ei.value)


def test_quantize_refusals():
    q = F.ft_mx4_quantize
    ok = dict(rows=4, cols=64, dtype=F.FT_T_BF16, x=FAKE, x_stride=64, codes=FAKE, scales=FAKE, values=None)
    call = lambda code, **kw: refused(code, q, *{**ok, **kw}.values())  # noqa: E731
    call(F.FT_ERR_INVALID_ARG, rows=-1)
    call(F.FT_ERR_INVALID_ARG, cols=0)
    call(F.FT_ERR_UNSUPPORTED, cols=48)
    call(F.FT_ERR_INVALID_ARG, dtype=3)
    call(F.FT_ERR_INVALID_ARG, x=None)
    call(F.FT_ERR_INVALID_ARG, codes=None)
    call(F.FT_ERR_INVALID_ARG, scales=None)
    call(F.FT_ERR_INVALID_ARG, x=FAKE + 1)
    call(F.FT_ERR_INVALID_ARG, x=FAKE + 2, dtype=F.FT_T_FP32)
    call(F.FT_ERR_INVALID_ARG, codes=FAKE + 8)
    call(F.FT_ERR_INVALID_ARG, values=FAKE + 8)
    assert "x_stride" in call(F.FT_ERR_INVALID_ARG, x_stride=32)
    call(F.FT_ERR_UNSUPPORTED, rows=BIG)
    q(0, 64, F.FT_T_BF16, None, 64, None, None, None, stream=0)      # no rows: nothing to do, no pointers needed


def test_product_refusals():
    p = F.ft_mx4_product
    ok = dict(groups=2, rows=4, n=64, k=128, offsets=FAKE, a_codes=FAKE, a_scales=FAKE, w_codes=FAKE, w_scales=FAKE,
              out=FAKE, ws=FAKE, ws_bytes=BIG)
    call = lambda code, **kw: refused(code, p, *{**ok, **kw}.values())  # noqa: E731
    for bad in (dict(groups=0), dict(rows=-1), dict(n=0), dict(k=0)):
        call(F.FT_ERR_INVALID_ARG, **bad)
    for bad in (dict(groups=257), dict(k=96), dict(k=16448), dict(n=12), dict(rows=2 ** 31 - 1, n=1 << 20)):
        call(F.FT_ERR_UNSUPPORTED, **bad)
    for name in ("offsets", "a_codes", "a_scales", "w_codes", "w_scales", "out", "ws"):
        call(F.FT_ERR_INVALID_ARG, **{name: None})
    for bad in (dict(a_codes=FAKE + 8), dict(w_codes=FAKE + 8), dict(out=FAKE + 8), dict(a_scales=FAKE + 1),
                dict(w_scales=FAKE + 1), dict(ws=FAKE + 128)):
        call(F.FT_ERR_INVALID_ARG, **bad)
    call(F.FT_ERR_WORKSPACE, ws_bytes=64)
    assert F.ft_mx4_product_workspace_bytes(2, 4, 64, 128) >= 4096
    assert F.ft_mx4_product_workspace_bytes(2, 4, 64, 100) == 0
    p(2, 0, 64, 128, None, None, None, None, None, None, None, 0, stream=0)


def _layer_args(shape, **kw):
    w = F.make_weights(FAKE, FAKE, FAKE, FAKE)
    d = dict(shape=shape, T=4, weights=w, x=FAKE, offsets=FAKE, inv_pos=FAKE, o_sorted=FAKE, ws=FAKE, ws_bytes=BIG)
    return list({**d, **kw}.values())


def test_experts_mx4_refusals():
    mx = F.make_shape(256, 128, 8, 2, 0, F.FT_W_MXFP4)
    bf = F.make_shape(256, 128, 8, 2)
    e = F.ft_moe_experts_mx4
    refused(F.FT_ERR_UNSUPPORTED, e, *_layer_args(bf))                              # BF16 weights
    refused(F.FT_ERR_UNSUPPORTED, e, *_layer_args(mx, weights=F.make_weights(expert_ptrs=FAKE)))
    refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(mx, weights=F.make_weights(FAKE, None, FAKE, FAKE)))
    refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(mx, T=-1))
    for name in ("x", "offsets", "inv_pos", "o_sorted", "ws"):
        refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(mx, **{name: None}))
    refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(mx, x=FAKE + 2))
    refused(F.FT_ERR_WORKSPACE, e, *_layer_args(mx, ws_bytes=4096))
    refused(F.FT_ERR_UNSUPPORTED, e, *_layer_args(mx, T=2 ** 30))                   # T * k past 31 bits
    e(mx, 0, F.make_weights(), None, None, None, None, None, 0, stream=0)
    sh = F.make_shape(256, 128, 8, 2, 1, F.FT_W_MXFP4)
    refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(sh))                              # no shared weights
    w = F.make_weights(FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE + 1, FAKE, FAKE)
    refused(F.FT_ERR_INVALID_ARG, e, *_layer_args(sh, weights=w))


def test_layer_forward_mx4_refusals():
    mx = F.make_shape(256, 128, 8, 2, 0, F.FT_W_MXFP4)
    w = F.make_weights(FAKE, FAKE, FAKE, FAKE)
    f = F.ft_moe_layer_forward_mx4
    refused(F.FT_ERR_UNSUPPORTED, f, F.make_shape(256, 128, 8, 2), 4, FAKE, FAKE, None, w, FAKE, None, None, FAKE, BIG)
    refused(F.FT_ERR_INVALID_ARG, f, mx, 4, None, FAKE, None, w, FAKE, None, None, FAKE, BIG)
    refused(F.FT_ERR_INVALID_ARG, f, mx, 4, FAKE, FAKE + 4, None, w, FAKE, None, None, FAKE, BIG)
    refused(F.FT_ERR_WORKSPACE, f, mx, 4, FAKE, FAKE, None, w, FAKE, None, None, FAKE, 256)
    f(mx, 0, None, None, None, F.make_weights(), None, None, None, None, 0, stream=0)


def test_backward_refusals():
    s = F.make_shape(256, 64, 8, 2)
    c = F.ft_moe_combine_backward
    assert "neither" in refused(F.FT_ERR_INVALID_ARG, c, s, 4, FAKE, FAKE, FAKE, FAKE, None, None)
    refused(F.FT_ERR_INVALID_ARG, c, s, 4, FAKE, None, FAKE, FAKE, FAKE, FAKE)       # gates' gradient needs o_sorted
    refused(F.FT_ERR_INVALID_ARG, c, s, 4, None, FAKE, FAKE, FAKE, FAKE, FAKE)
    refused(F.FT_ERR_INVALID_ARG, c, s, 4, FAKE + 2, FAKE, FAKE, FAKE, FAKE, FAKE)
    refused(F.FT_ERR_INVALID_ARG, c, s, -1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    refused(F.FT_ERR_UNSUPPORTED, c, s, 2 ** 30, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    c(s, 0, None, None, None, None, FAKE, None, stream=0)
    p = F.ft_moe_permute_backward
    assert "together" in refused(F.FT_ERR_INVALID_ARG, p, s, 4, FAKE, FAKE, FAKE, None, FAKE, FAKE)
    refused(F.FT_ERR_INVALID_ARG, p, s, 4, None, FAKE, None, None, None, FAKE)
    refused(F.FT_ERR_INVALID_ARG, p, s, 4, FAKE, FAKE, FAKE, FAKE, FAKE + 4, FAKE)
    p(s, 0, None, None, None, None, None, None, stream=0)
    r = F.ft_moe_route_backward
    refused(F.FT_ERR_INVALID_ARG, r, s, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, BIG)
    refused(F.FT_ERR_INVALID_ARG, r, s, 4, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, BIG)
    refused(F.FT_ERR_INVALID_ARG, r, s, 4, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, BIG)
    refused(F.FT_ERR_INVALID_ARG, r, s, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 8, None, FAKE, BIG)
    refused(F.FT_ERR_WORKSPACE, r, s, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 256)
    r(s, 0, None, None, None, None, None, None, None, None, None, None, 0, stream=0)


def test_reference_quantizer_is_nearest_even_on_every_border():
    """The tests' own quantiser, pinned by hand: grid points stay, midpoints go to the even code, 6 saturates."""
    row = np.zeros((1, 32))
    pts = [0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9, -0.25, -0.75, -5, -0.0]
    row[0, :len(pts)] = pts
    code, scale = M.quantize(row)
    assert scale[0, 0] == 127
    got = M.values(code, scale)[0, :len(pts)]
    assert got.tolist() == [0, 0, 0.5, 1, 1, 1, 1.5, 2, 2, 2, 3, 4, 4, 4, 6, 6, 6, -0.0, -1, -4, -0.0]
    assert np.signbit(got[17]) and np.signbit(got[20])
    code, scale = M.quantize(np.full((1, 32), 2.0 ** -140))
    assert scale[0, 0] == 0 and not (code & 7).any()


class _Elsewhere:
    """Stands for a tensor on another device than the current one."""
    device = "cuda:1"

    def __init__(self, d):
        self.d = d

    def data_ptr(self):
        return FAKE

    def get_device(self):
        return self.d


@pytest.mark.parametrize("where", [1, -1])
def test_tensors_of_another_device_are_refused(monkeypatch, where):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, there = _Elsewhere(0), _Elsewhere(where)
    s = F.make_shape(256, 64, 8, 2)
    mx = F.make_shape(256, 128, 8, 2, 0, F.FT_W_MXFP4)
    w = F.make_weights(FAKE, FAKE, FAKE, FAKE)
    calls = [
        (F.ft_mx4_quantize, (4, 64, F.FT_T_BF16, here, 64, here, there, None)),
        (F.ft_mx4_product, (2, 4, 64, 128, here, here, here, there, here, here, here, BIG)),
        (F.ft_moe_experts_mx4, (mx, 4, w, here, here, there, here, here, BIG)),
        (F.ft_moe_layer_forward_mx4, (mx, 4, here, there, None, w, here, None, None, here, BIG)),
        (F.ft_moe_combine_backward, (s, 4, there, here, here, here, here, here)),
        (F.ft_moe_permute_backward, (s, 4, here, here, None, None, None, there)),
        (F.ft_moe_route_backward, (s, 4, here, here, here, there, here, here, here, here, here, here, BIG)),
    ]
    for fn, args in calls:
        assert "current" in refused(F.FT_ERR_INVALID_ARG, fn, *args)


@pytest.mark.parametrize("where", [1, -1])
@pytest.mark.parametrize("field", [0, 1, 2, 3, 5, 6, 7, 8])
def test_weights_on_another_device_are_refused(monkeypatch, where, field):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here = _Elsewhere(0)
    given = [here] * 4 + [None] + [here] * 4
    given[field] = _Elsewhere(where)
    w = F.make_weights(*given)
    mx = F.make_shape(256, 128, 8, 2, 1, F.FT_W_MXFP4)
    name = F.ft_moe_weights._fields_[field][0]
    for fn, args in ((F.ft_moe_experts_mx4, (mx, 4, w, here, here, here, here, here, BIG)),
                     (F.ft_moe_layer_forward_mx4, (mx, 4, here, here, None, w, here, None, None, here, BIG))):
        msg = refused(F.FT_ERR_INVALID_ARG, fn, *args)
        assert "current" in msg and name in msg
    # an address put in its place is the caller's own, as everywhere; the calls go on to their other checks
    setattr(w, name, FAKE + 1)
    assert "current" not in refused(F.FT_ERR_INVALID_ARG, F.ft_moe_experts_mx4, mx, 4, w, here, here, here, here, here, BIG)
