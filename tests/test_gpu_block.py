"""The operators around the layer together, as a transformer block runs them (B200): norm with 8-bit rows and the FP8
layer that reads them, norm and the few-token layer, and a training step's norm, layer, their backward and clipping."""
import pytest
import torch

from fine_grained_mixture_route_b200 import moe, quant
from fine_grained_mixture_route_b200 import workloads as W
from tests import block_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FMT = {"e4m3": moe.FMT_E4M3, "mxfp8": moe.FMT_MXFP8}


def _layer(T, d, E, I, k, Ks, fmt=None, seed=0, bias=True):
    cfg = W.LayerConfig("block", T, d, E, I, k, Ks, I if Ks else 0, bias, BF, "normal_inv_sqrt_d")
    L = W.make_layer(cfg, "cuda", seed)
    L["cfg"] = cfg
    if fmt:
        L["routed"] = quant.quantize_stack(L["routed"], fmt)
    return L


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
@pytest.mark.parametrize("T,d,Ks", [(1, 272, 0), (130, 1280, 1)])
def test_given_codes_are_the_layer_s_own(fmt, T, d, Ks):
    # what the layer would make of x itself, given: the same bits
    L = _layer(T, d, 16, 208, 4, Ks, fmt)
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 4, L["shared"])
    ws = moe.new_workspace(shape)
    want = moe.layer_forward(shape, L["x"], L["centroids"], L["routed"], L["shared"], ws)
    if fmt == "e4m3":
        codes, scale = moe.quantize_rows_e4m3(L["x"], ws)
    else:
        e = R.run_exponents(torch.nn.functional.pad(L["x"].double(), (0, -d % 32)).view(T, -1, 32).abs().amax(2))
        codes = (L["x"].double() * torch.pow(2.0, -e).repeat_interleave(32, 1)[:, :d]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        scale = (e + 127).to(torch.uint8)
    idx = torch.empty((T, 4), dtype=torch.int32, device="cuda")
    got = moe.layer_forward_quantized(shape, L["x"], codes, scale, L["centroids"], L["routed"], L["shared"], ws, idx=idx)
    assert torch.equal(got, want) and moe.check_device_error(ws) == 0
    # and they are what is read: with all codes zero the routed experts see a zero row
    zero = moe.layer_forward_quantized(shape, L["x"], torch.zeros_like(codes), scale, L["centroids"], L["routed"], L["shared"], ws)
    assert not torch.equal(zero, want)


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
def test_norm_feeds_the_fp8_layer(fmt):
    # norm with codes -> layer, against norm -> layer that quantises the rounded rows: they differ by the rounding of
    # single codes (a step of 2^-3 relative at most, and only where the two values lie on either side of a border)
    L = _layer(96, 1024, 16, 256, 4, 1, fmt)
    w = torch.ones(1024, dtype=BF, device="cuda")
    n = moe.rmsnorm(L["x"], w, residual=torch.flip(L["x"], [0]).contiguous(), fmt=FMT[fmt])
    shape = moe.shape_of(n["y"], L["centroids"], L["routed"], 4, L["shared"])
    ws = moe.new_workspace(shape)
    a = moe.layer_forward_quantized(shape, n["y"], n["codes"], n["scale"], L["centroids"], L["routed"], L["shared"], ws)
    b = moe.layer_forward(shape, n["y"], L["centroids"], L["routed"], L["shared"], ws)
    assert moe.check_device_error(ws) == 0 and _rel(a, b) <= 2.0 ** -4


def test_decode_block_captured():
    # norm -> few-token layer -> the next norm with the residual, one graph, replayed on new rows
    L = _layer(4, 512, 16, 128, 3, 1)
    x, w = L["x"].clone(), torch.full((512,), 1.25, dtype=BF, device="cuda")
    shape = moe.shape_of(x, L["centroids"], L["routed"], 3, L["shared"])
    ws = moe.new_few_workspace(shape)

    def block(ws):
        n = moe.rmsnorm(x, w)
        o = moe.layer_forward_few(shape, n["y"], L["centroids"], L["routed"], L["shared"], ws)
        return moe.rmsnorm(o, w, residual=x)

    block(ws)                                                   # warm, before the capture
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = block(ws)
    for seed in (5, 6):
        x.copy_(W.make_x(L["cfg"], "cuda", seed=seed))
        g.replay()
        want = block(moe.new_few_workspace(shape))
        assert all(torch.equal(got[k], want[k]) for k in ("y", "sum", "rstd"))
    assert moe.check_device_error(ws) == 0


def test_training_step():
    # s = x + r; y = norm(s); out = s + layer(y); loss = sum(out * G): gradients through the layer's own backward, the
    # norm's, and the clipping of all of them, against torch's autograd of the same formulas in fp32
    T, d, E, I, k = 64, 256, 16, 64, 2
    L = _layer(T, d, E, I, k, 1)
    r = W.make_x(L["cfg"], "cuda", seed=9)
    w = torch.linspace(0.5, 1.5, d, device="cuda").to(BF)
    G = W.make_x(L["cfg"], "cuda", seed=10)
    n = moe.rmsnorm(L["x"], w, residual=r)
    shape = moe.shape_of(n["y"], L["centroids"], L["routed"], k, L["shared"])
    ws = moe.new_workspace(shape)
    ctx, wsb = moe.new_train_buffers(shape)[:2]
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    moe.layer_forward_train(shape, n["y"], L["centroids"], L["routed"], L["shared"], ws, ctx)
    moe.layer_forward(shape, n["y"], L["centroids"], L["routed"], L["shared"], ws, idx=idx)
    gr = moe.layer_backward(shape, n["y"], L["centroids"], L["routed"], L["shared"], G, ctx, wsb)
    dx, dw = moe.rmsnorm_backward(gr["dx"], n["sum"], w, n["rstd"], dsum=G)

    # autograd: the picks are given, all else is differentiated
    s = n["sum"].float().requires_grad_()
    wf = w.float().requires_grad_()
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * wf
    P = {n_: {q: t.float().requires_grad_() for q, t in L[n_].items() if t is not None} for n_ in ("routed", "shared")}
    C = L["centroids"].float().requires_grad_()
    gate = torch.softmax(y @ C.T, 1).gather(1, idx.long())

    def expert(S, e, v):
        h = torch.nn.functional.silu(v @ S["w1"][e].T + S["b1"][e]) * (v @ S["w3"][e].T + S["b3"][e])
        return h @ S["w2"][e].T + S["b2"][e]

    out = s + expert(P["shared"], 0, y)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, gate[t, j, None] * expert(P["routed"], e, y[t]))
    (out * G.float()).sum().backward()
    # the layer's gradients are bf16 products of bf16 hidden rows (2^-8 each of several roundings): 2^-5 in the norm
    assert _rel(dx, s.grad) <= 2.0 ** -5 and _rel(dw, wf.grad) <= 2.0 ** -5
    tensors = moe.grad_tensors(gr) + [dw]
    before = [t.clone() for t in tensors]
    wsg = moe.new_grad_workspace()
    total = torch.stack([t.double().square().sum() for t in before]).sum().sqrt()
    norm = moe.clip_grads(tensors, float(total) / 4, wsg)
    assert abs(float(norm) - float(total)) <= 2.0 ** -22 * float(total)
    after = moe.grad_norm(tensors, wsg)
    assert abs(float(after) - float(total) / 4) <= 2.0 ** -8 * float(total) / 4
    ref = [C.grad] + [P[n_][q].grad for n_ in ("routed", "shared") for q in ("w1", "b1", "w3", "b3", "w2", "b2")] + [wf.grad]
    refn = torch.stack([t.double().square().sum() for t in ref]).sum().sqrt()
    assert abs(float(refn) / float(total) - 1.0) <= 2.0 ** -5
