"""Refusals of the operators around the layer (CPU): the binding's checks and the C entry points' own, before any
CUDA call."""
import ctypes
import math

import pytest
import torch

from fine_grained_mixture_route_b200 import moe

BF, F32 = torch.bfloat16, torch.float32


def _m(rows, d, dtype=BF):
    return torch.zeros((rows, d), dtype=dtype)


def test_rmsnorm_refuses_before_any_call():
    x, w = _m(4, 64), torch.ones(64, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        moe.rmsnorm(x, w)
    for bad, what in ((dict(x=x.half()), "dtype"), (dict(x=x[:, ::2]), "contiguous"), (dict(x=x[0]), "matrix"),
                      (dict(weight=w.float()), "weight has dtype"), (dict(weight=torch.ones(63, dtype=BF)), "weight has shape"),
                      (dict(residual=_m(5, 64)), "residual has shape"), (dict(residual=_m(4, 64, F32)), "residual has dtype"),
                      (dict(fmt=7), "fmt"), (dict(out={"y": _m(4, 63)}), "out"), (dict(out={"rstd": torch.zeros(5)}), "out"),
                      (dict(fmt=moe.FMT_MXFP8, out={"scale": torch.zeros((4, 3), dtype=torch.uint8)}), "out")):
        args = dict(x=x, weight=w)
        args.update(bad)
        with pytest.raises((ValueError, TypeError), match=what):
            moe.rmsnorm(**args)
    with pytest.raises(TypeError):
        moe.rmsnorm([1.0], w)


def test_rmsnorm_backward_refuses_before_any_call():
    s, w, r = _m(4, 64), torch.ones(64, dtype=BF), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.rmsnorm_backward(s, s, w, r)
    for bad, what in ((dict(dy=_m(4, 63)), "dy has shape"), (dict(dy=_m(4, 64, F32)), "dy has dtype"),
                      (dict(rstd=torch.ones(5)), "rstd has shape"), (dict(rstd=torch.ones(4, dtype=BF)), "rstd has dtype"),
                      (dict(dsum=_m(3, 64)), "dsum has shape"), (dict(dx=_m(4, 64, F32)), "dx has dtype"),
                      (dict(dweight=torch.zeros(63)), "dweight has shape"), (dict(ws=torch.zeros(4)), "ws has dtype")):
        args = dict(dy=s, s=s, weight=w, rstd=r)
        args.update(bad)
        with pytest.raises((ValueError, TypeError), match=what):
            moe.rmsnorm_backward(**args)


def test_grad_lists_refused():
    ws = torch.zeros(1 << 14, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.grad_norm([torch.zeros(4)], ws)
    with pytest.raises(TypeError):
        moe.grad_norm([torch.zeros(4)], torch.zeros(4))
    for bad, what in (([torch.zeros(4).half()], "dtype"), ([torch.zeros((4, 4))[:, :2]], "contiguous"), ([3.0], "Tensor")):
        with pytest.raises((ValueError, TypeError), match=what):
            moe._tensor_list(bad, "tensors", torch.device("cpu"))
    t = torch.zeros(100)
    with pytest.raises(ValueError, match="overlap"):
        moe._no_overlap(moe._spans([t[:50], t[49:]]), "tensors")
    with pytest.raises(ValueError, match="overlap"):
        moe._no_overlap(moe._spans([t, t]), "tensors")          # the same gradient twice
    moe._no_overlap(moe._spans([t[:50], t[50:], t[:0]]), "tensors")


def test_clipping_refuses_what_overlaps():
    ws, t = torch.zeros(1 << 14, dtype=torch.uint8), torch.zeros(100)
    a, b, e = t[:40], t[40:80], t[:0]

    def clip(ts, out=None):
        return moe.clip_grads(ts, 1.0, ws, out=out)

    for ts in ([t, t], [t[:50], t[49:]], [a, b, t[79:81]], [b, a, t], [t[10:20], e, t[:11]], [t.view(torch.int32).view(torch.float32), t]):
        with pytest.raises(ValueError, match="overlap"):
            clip(ts)
    o = torch.zeros(100)
    for out in ([b, a],                                         # another gradient's place
                [a, t[39:79]],                                  # its own gradient, one element off, and the one before
                [t[1:41], o[:40]],                              # its own gradient, one element off
                [o[:40], o[39:79]], [o[:40], o[:40]], [a, a]):  # one another, or another output that is a gradient
        with pytest.raises(ValueError, match="overlap"):
            clip([a, b], out)
    for out in ([o[:40]], [o[:40], o[40:81]], [o[:40], o[40:80].bfloat16()]):
        with pytest.raises(ValueError, match="same shape and type"):
            clip([a, b], out)
    # allowed as far as the overlap goes: the gradients themselves, some of them, neighbours, empty ones anywhere
    for ts, out in (([a, b], None), ([a, b], [a, b]), ([a, b], [a, o[:40]]), ([a, b], [o[:40], o[40:80]]), ([e, a, e, b], None),
                    ([a, e, b], [a, t[20:20], t[80:].new_zeros(40)]), ([], None), ([], [])):
        with pytest.raises(ValueError, match="CUDA"):
            clip(ts, out)


def test_c_entry_points_return_errors():
    lib, INV, UNS, WS = moe.lib_handle(), moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
    p, odd = ctypes.c_void_p(1 << 40), ctypes.c_void_p((1 << 40) + 8)      # never dereferenced

    def norm(dtype=1, rows=4, d=64, x=p, res=None, w=p, eps=1e-6, s=None, y=p, fmt=0, codes=None, sc=None, rstd=None):
        return lib.moe_rmsnorm(dtype, rows, d, x, res, w, eps, s, y, fmt, codes, sc, rstd, None)

    assert norm(rows=0, x=None, y=None) == moe.MOE_OK
    for kw in (dict(dtype=2), dict(rows=-1), dict(d=0), dict(x=None), dict(w=None), dict(y=None), dict(res=p), dict(s=p),
               dict(fmt=3), dict(codes=p), dict(fmt=1, codes=p), dict(fmt=2, sc=p), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(x=odd), dict(y=odd), dict(w=odd), dict(fmt=1, codes=odd, sc=p)):
        assert norm(**kw) == INV, kw
    for kw in (dict(d=60), dict(d=16392), dict(rows=1 << 31), dict(dtype=0, fmt=1, codes=p, sc=p), dict(dtype=0, d=16385)):
        assert norm(**kw) == UNS, kw
    need = lib.moe_rmsnorm_backward_workspace_bytes
    assert need(1, 4, 64) >= 256 and need(1, 100000, 7168) >= 7168 * 4 and need(1, 4, 60) == 0 and need(5, 4, 64) == 0

    def bwd(dtype=1, rows=4, d=64, dy=p, s=p, w=p, r=p, ds=None, dx=p, dw=p, ws=p, n=1 << 30):
        return lib.moe_rmsnorm_backward(dtype, rows, d, dy, s, w, r, ds, dx, dw, ws, n, None)

    for kw in (dict(dy=None), dict(s=None), dict(w=None), dict(r=None), dict(dx=None), dict(dw=None), dict(ds=odd), dict(dx=odd)):
        assert bwd(**kw) == INV, kw
    for kw in (dict(ws=None), dict(n=16), dict(ws=odd)):
        assert bwd(**kw) == WS, kw
    assert bwd(d=60) == UNS

    T = lambda **k: (moe.MoeTensor * 1)(moe.MoeTensor(*[{**dict(data=1 << 40, numel=8, dtype=1), **k}[f]  # noqa: E731
                                                         for f in ("data", "numel", "dtype")]))
    n = lib.moe_grad_workspace_bytes()
    for t in (T(dtype=3), T(numel=-1), T(data=0), T(data=(1 << 40) + 1), T(data=(1 << 40) + 2, dtype=0)):
        assert lib.moe_grad_norm(t, 1, p, p, n, None) == INV
    assert lib.moe_grad_norm(T(numel=1 << 40), 1, p, p, n, None) == UNS
    assert lib.moe_grad_norm(T(), 70000, p, p, n, None) == UNS
    assert lib.moe_grad_norm(T(), 1, None, p, n, None) == INV and lib.moe_grad_norm(None, 1, p, p, n, None) == INV
    assert lib.moe_grad_norm(T(), 1, p, p, n - 1, None) == WS and lib.moe_grad_norm(T(), 1, p, None, n, None) == WS
    for m in (-1.0, math.nan):
        assert lib.moe_clip_grads(T(), None, 1, m, p, p, n, None) == INV
    assert lib.moe_clip_grads(T(), T(numel=9), 1, 1.0, p, p, n, None) == INV
    assert lib.moe_clip_grads(T(), T(dtype=0), 1, 1.0, p, p, n, None) == INV


def _shape(**kw):
    base = dict(T=4, d=128, n_experts=8, inter=64, top_k=2, n_shared=1, inter_shared=64, has_bias=1, dtype=moe.MOE_BF16,
                gate_mode=0, routed_fmt=moe.FMT_NATIVE)
    base.update(kw)
    return moe.MoeShape(*[base[f] for f, _ in moe.MoeShape._fields_])


def test_few_sizes_and_workspace():
    n = moe.few_workspace_bytes(_shape())
    assert n > 0 and moe.few_workspace_bytes(_shape(T=16)) > n and moe.few_workspace_bytes(_shape(T=0)) > 0
    assert moe.few_workspace_bytes(_shape(T=1)) < n             # one workspace for fewer tokens, too
    for bad in (dict(T=17), dict(d=32776), dict(d=132), dict(T=-1), dict(top_k=9), dict(dtype=moe.MOE_F32, d=130),
                dict(dtype=moe.MOE_F32, inter=66), dict(dtype=moe.MOE_F32, inter_shared=65),
                dict(routed_fmt=moe.FMT_MXFP8, d=136), dict(routed_fmt=moe.FMT_E4M3, dtype=moe.MOE_F32)):
        assert moe.few_workspace_bytes(_shape(**bad)) == 0, bad
        with pytest.raises(ValueError):
            moe.new_few_workspace(_shape(**bad), "cpu")
    assert moe.few_workspace_bytes(_shape(dtype=moe.MOE_F32, n_shared=0, inter_shared=65)) > 0


def test_few_c_entry_point_returns_errors():
    lib = moe.lib_handle()
    p, odd = ctypes.c_void_p(1 << 40), ctypes.c_void_p((1 << 40) + 8)
    w = lambda v=1 << 40, **k: moe.MoeWeights(**{**{n: v for n in ("w1", "b1", "w3", "b3", "w2", "b2")}, **k})  # noqa: E731

    def few(sh=None, x=p, c=p, R=None, S=None, out=p, ws=p, n=1 << 30, **kw):
        sh = _shape(**kw) if sh is None else sh
        return lib.moe_layer_forward_few(ctypes.byref(sh), x, c, None, ctypes.byref(w() if R is None else R),
                                         ctypes.byref(w()) if S is None else S, out, None, None, None, ws, n, None)

    assert few(T=0, x=None, out=None) == moe.MOE_OK
    for kw in (dict(x=None), dict(c=None), dict(out=None), dict(x=odd), dict(c=odd), dict(out=odd), dict(R=w((1 << 40) + 8)),
               dict(R=w(b1=None)), dict(R=w(s1=1 << 40, s3=1 << 40, s2=1 << 40)), dict(n_shared=0), dict(gate_mode=3)):
        assert few(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert few(S=ctypes.POINTER(moe.MoeWeights)()) == moe.MOE_ERR_INVALID_ARG
    for kw in (dict(T=17), dict(d=32776), dict(d=132), dict(dtype=moe.MOE_F32, d=130)):
        assert few(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    need = moe.few_workspace_bytes(_shape())
    for kw in (dict(ws=None), dict(ws=odd), dict(n=need - 1)):
        assert few(**kw) == moe.MOE_ERR_WORKSPACE, kw


def test_few_binding_refuses_before_any_call():
    from fine_grained_mixture_route_b200 import workloads as W
    cfg = W.scaled(W.CONFIGS["small"], T=4, d=64, n_experts=8, top_k=2, inter=32, inter_shared=32)
    L = W.make_layer(cfg, "cpu")
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 2, L["shared"])
    ws = torch.zeros(64, dtype=torch.uint8)

    def call(**kw):
        a = dict(L, ws=ws)
        a.update(kw)
        return moe.layer_forward_few(shape, a["x"], a["centroids"], a["routed"], a["shared"], a["ws"],
                                     **{k: v for k, v in kw.items() if k in ("out", "gate", "router_bias")})

    with pytest.raises(ValueError, match="CUDA"):
        call()
    for kw, what in ((dict(x=L["x"].float()), "x has dtype"), (dict(x=L["x"][:3]), "x holds"), (dict(ws=torch.zeros(8)), "ws"),
                     (dict(out=torch.zeros(4, 64)), "out"), (dict(gate=torch.zeros(7)), "gate"),
                     (dict(router_bias=torch.zeros(7)), "router_bias"),
                     (dict(routed=dict(L["routed"], w2=L["routed"]["w2"].float())), "routed.w2")):
        with pytest.raises(ValueError, match=what):
            call(**kw)


# ------------------------------------------------------------------------------ the layer on rows in 8 bits
def _q8_args(fmt="e4m3", T=4, d=64, E=4, I=32):
    s = {k: torch.zeros(v, dtype=torch.uint8) for k, v in (("w1", (E, I, d)), ("w3", (E, I, d)), ("w2", (E, d, I)))}
    if fmt == "e4m3":
        s.update(s1=torch.zeros(E, I), s3=torch.zeros(E, I), s2=torch.zeros(E, d))
    else:
        s.update(sf13=torch.zeros(moe.mx_scale_bytes(moe.MX_UP, E, I, d), dtype=torch.uint8),
                 sf2=torch.zeros(moe.mx_scale_bytes(moe.MX_DOWN, E, d, I), dtype=torch.uint8))
    x, c = _m(T, d), _m(E, d)
    shape = moe.shape_of(x, c, s, 2, None)
    scale = torch.zeros(T) if fmt == "e4m3" else torch.zeros((T, -(-d // 32)), dtype=torch.uint8)
    return dict(shape=shape, x=x, x_codes=torch.zeros((T, d), dtype=torch.uint8), x_scale=scale, centroids=c, routed=s,
                shared=None, ws=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
def test_quantized_layer_refuses_before_any_call(fmt):
    a = _q8_args(fmt)
    with pytest.raises(ValueError, match="CUDA"):
        moe.layer_forward_quantized(**a)
    for bad, what in ((dict(x_codes=None), "x_codes"), (dict(x_scale=None), "x_scale"),
                      (dict(x_codes=torch.zeros((4, 63), dtype=torch.uint8)), "x_codes holds"),
                      (dict(x_codes=_m(4, 64)), "x_codes has dtype"), (dict(x_scale=a["x_scale"][:3]), "x_scale holds"),
                      (dict(x_scale=torch.zeros((4, 2), dtype=torch.int8)), "x_scale has dtype"),
                      (dict(ws=torch.zeros(4)), "ws has dtype")):
        with pytest.raises((ValueError, TypeError), match=what):
            moe.layer_forward_quantized(**{**a, **bad})


def test_quantized_layer_needs_8_bit_experts():
    a = _q8_args()
    E, I, d = a["routed"]["w1"].shape
    native = {"w1": torch.zeros((E, I, d), dtype=BF), "w3": torch.zeros((E, I, d), dtype=BF), "w2": torch.zeros((E, d, I), dtype=BF)}
    shape = moe.shape_of(a["x"], a["centroids"], native, 2, None)
    with pytest.raises(ValueError, match="8-bit"):
        moe.layer_forward_quantized(**{**a, "shape": shape, "routed": native})


def test_quantized_layer_c_entry_point_returns_errors():
    lib, p, odd = moe.lib_handle(), ctypes.c_void_p(1 << 40), ctypes.c_void_p((1 << 40) + 8)      # never dereferenced

    def call(fmt=moe.FMT_E4M3, x=p, codes=p, scales=p, ws=p, T=4):
        sh = moe.make_shape(T, 64, 4, 32, 2, routed_fmt=fmt, has_bias=False)
        w = moe.MoeWeights(w1=p, w3=p, w2=p)
        if fmt == moe.FMT_E4M3:
            w.s1 = w.s3 = w.s2 = p
        elif fmt == moe.FMT_MXFP8:
            w.sf13 = w.sf2 = p
        return lib.moe_layer_forward_quantized(ctypes.byref(sh), x, codes, scales, p, None, ctypes.byref(w), None, p, None, None,
                                               None, ws, 1 << 30, None)

    assert call(T=0, x=None, codes=None, scales=None) == moe.MOE_OK
    for kw in (dict(codes=None), dict(scales=None), dict(codes=odd), dict(x=None), dict(scales=ctypes.c_void_p((1 << 40) + 2))):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(fmt=moe.FMT_NATIVE) == moe.MOE_ERR_UNSUPPORTED
    assert call(ws=None) == moe.MOE_ERR_WORKSPACE
