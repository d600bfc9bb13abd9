"""The whole layer for a few tokens (moe.layer_forward_few) against the 64-bit definition (B200)."""
import math

import numpy as np
import pytest
import torch

from fine_grained_mixture_route_b200 import moe, quant
from fine_grained_mixture_route_b200 import workloads as W
from tests import block_ref as R
from tests import parity

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _case(T, d, E, I, k, Ks=0, Is=None, bias=True, dtype=BF, fmt=None, mode=0, seed=0):
    cfg = W.LayerConfig("few", T, d, E, I, k, Ks, (Is or I) if Ks else 0, bias, dtype, "normal_inv_sqrt_d")
    L = W.make_layer(cfg, "cuda", seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    for s in (L["routed"], L["shared"]):                       # hidden values of order one, whatever the sizes
        for n in ("w1", "w3", "w2") if s is not None else ():
            s[n].normal_(0.0, s[n].shape[-1] ** -0.5, generator=g)
        for n in ("b1", "b3", "b2") if s is not None and bias else ():
            s[n].normal_(0.0, 0.3, generator=g)
    if fmt:
        L["routed"] = quant.quantize_stack(L["routed"], fmt)
    L["router_bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if mode else None
    L["cfg"], L["mode"] = cfg, mode
    return L


def _run(L, ws=None, x=None, **kw):
    x = L["x"] if x is None else x
    shape = moe.shape_of(x, L["centroids"], L["routed"], L["cfg"].top_k, L["shared"], L["mode"])
    ws = moe.new_few_workspace(shape) if ws is None else ws
    T, k, E = shape.T, shape.top_k, shape.n_experts
    o = {"idx": torch.full((T, k), -7, dtype=torch.int32, device="cuda"), "gate": torch.full((T, k), 9.0, device="cuda"),
         "counts": torch.full((E,), -1, dtype=torch.int32, device="cuda")}
    o["out"] = moe.layer_forward_few(shape, x, L["centroids"], L["routed"], L["shared"], ws, router_bias=L["router_bias"],
                                     **o, **kw)
    o["ws"] = ws
    return o


def _check(L, o, x=None, tiny=0.0):
    x = L["x"] if x is None else x
    assert moe.check_device_error(o["ws"]) == 0
    idx, gate = o["idx"].cpu().numpy().astype(np.int64), o["gate"].cpu().numpy().astype(np.float64)
    bias = None if L["router_bias"] is None else parity.f64(L["router_bias"])
    parity.check_routing(idx, gate, parity.f64(x), parity.f64(L["centroids"]), L["cfg"].top_k, L["mode"], bias)
    assert np.array_equal(o["counts"].cpu().numpy(), np.bincount(idx.reshape(-1), minlength=L["cfg"].n_experts))
    ref, bound = R.few_layer(x, o["idx"], o["gate"], L["routed"], L["shared"], L["cfg"].n_shared)
    err = (o["out"].double() - ref).abs()
    tol = R.HALF[x.dtype] * (ref.abs() + bound) + bound + tiny
    assert (err <= tol).all(), float((err / tol).max())


SHAPES = [
    dict(T=1, d=64, E=4, I=32, k=1),
    dict(T=1, d=8, E=1, I=8, k=1),                              # the smallest
    dict(T=2, d=72, E=5, I=40, k=2, Ks=1),                      # odd multiples of 8
    dict(T=3, d=264, E=33, I=104, k=4, Ks=2, Is=200),           # shared experts of another width
    dict(T=8, d=1280, E=64, I=320, k=7, Ks=1),
    dict(T=9, d=1032, E=40, I=328, k=3, Ks=1),                  # two groups of tokens
    dict(T=16, d=2048, E=64, I=1408, k=6, Ks=2, bias=False),
    dict(T=16, d=512, E=2, I=256, k=2),                         # every expert meets every token
    dict(T=5, d=256, E=1024, I=64, k=32),                       # the most experts and picks
    dict(T=16, d=128, E=300, I=48, k=32, Ks=16, Is=24),         # the most of all
    dict(T=1, d=7168, E=16, I=2048, k=8, Ks=1),
    dict(T=4, d=4104, E=8, I=1032, k=2),                        # a stage's end inside a warp's columns
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_bf16(kw):
    L = _case(**kw)
    _check(L, _run(L))


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
@pytest.mark.parametrize("kw", [dict(T=1, d=64, E=4, I=32, k=1), dict(T=1, d=16, E=1, I=16, k=1),
                                dict(T=3, d=272, E=33, I=112, k=4, Ks=2, Is=200), dict(T=16, d=2064, E=12, I=400, k=6, Ks=1),
                                dict(T=8, d=1280, E=64, I=320, k=7, Ks=1, bias=False), dict(T=2, d=7168, E=8, I=2048, k=4),
                                dict(T=11, d=528, E=9, I=2320, k=3)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_fp8(kw, fmt):
    L = _case(fmt=fmt, **kw)
    _check(L, _run(L))


@pytest.mark.parametrize("kw", [dict(T=1, d=4, E=1, I=4, k=1), dict(T=7, d=256, E=16, I=64, k=4, Ks=1),
                                dict(T=16, d=516, E=9, I=132, k=3, Ks=2, Is=68), dict(T=2, d=1028, E=5, I=1100, k=2, bias=False)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_fp32(kw):
    L = _case(dtype=F32, **kw)
    _check(L, _run(L))


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("dtype,fmt", [(BF, None), (BF, "mxfp8"), (F32, None)])
def test_gate_modes_with_a_router_bias(mode, dtype, fmt):
    L = _case(T=6, d=256, E=24, I=64, k=4, Ks=1, dtype=dtype, fmt=fmt, mode=mode)
    _check(L, _run(L))


def test_agrees_with_the_layer():
    # the same layer: picks equal, outputs within the larger path's bf16 hidden rows
    L = _case(T=16, d=1024, E=32, I=256, k=4, Ks=1, seed=4)
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 4, L["shared"])
    ref = moe.layer_forward(shape, L["x"], L["centroids"], L["routed"], L["shared"], moe.new_workspace(shape))
    o = _run(L)
    assert float((o["out"].double() - ref.double()).norm() / ref.double().norm()) <= 2.0 ** -6


def test_equal_scores_go_to_the_lower_index():
    L = _case(T=3, d=64, E=40, I=32, k=5)
    L["centroids"][:] = L["centroids"][0]
    o = _run(L)
    assert o["idx"].tolist() == [[0, 1, 2, 3, 4]] * 3
    _check(L, o)


def test_picks_that_do_not_exist():
    L = _case(T=4, d=64, E=6, I=32, k=3, Ks=1, mode=1)
    L["router_bias"][:] = float("-inf")
    L["router_bias"][[1, 4]] = 0.0                              # two experts left for three picks
    o = _run(L)
    with pytest.raises(moe.MoeError) as e:
        moe.check_device_error(o["ws"])
    assert e.value.detail == 1
    idx = o["idx"].clone()
    assert set(idx[:, :2].reshape(-1).tolist()) == {1, 4} and (idx[:, 2] >= 6).all()
    idx[:, 2] = -1
    ref, bound = R.few_layer(L["x"], idx, o["gate"], L["routed"], L["shared"], 1)
    assert ((o["out"].double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + bound) + bound).all()
    x = L["x"].clone()                                          # one token's logits are NaN: the others keep their results
    L["router_bias"].zero_()
    want = _run(L)["out"]
    x[2, 5] = float("nan")
    o = _run(L, x=x)
    with pytest.raises(moe.MoeError):
        moe.check_device_error(o["ws"])
    assert torch.equal(o["out"][[0, 1, 3]], want[[0, 1, 3]]) and torch.isnan(o["out"][2]).all()
    # no shared expert and no pick left: zeros
    L = _case(T=2, d=64, E=3, I=32, k=1, mode=1)
    L["router_bias"][:] = float("-inf")
    o = _run(L)
    assert (o["out"] == 0).all() and (o["counts"] == 0).all()


def test_infinite_rows_stay_in_their_rows():
    L = _case(T=3, d=128, E=4, I=64, k=2, Ks=1)
    want = _run(L)["out"]
    L["routed"]["w2"][:, 7, 3] = float("inf")
    got = _run(L)["out"]
    keep = torch.arange(128, device="cuda") != 7
    assert torch.equal(got[:, keep], want[:, keep]) and not torch.isfinite(got[:, 7]).any()


@pytest.mark.parametrize("fmt", [None, "e4m3", "mxfp8"])
def test_an_infinite_expert_stays_with_the_tokens_that_picked_it(fmt):
    L = _case(T=6, d=256, E=24, I=64, k=2, Ks=1, fmt=fmt)
    o = _run(L)
    e = int(o["idx"][0, 0])
    hit = (o["idx"] == e).any(1)
    assert hit.any() and not hit.all()
    w = L["routed"]["w2"]
    if fmt:
        w[e] = 0x7F                                             # the code of NaN
    else:
        w[e] = float("inf")
    got = _run(L)["out"]
    assert torch.equal(got[~hit], o["out"][~hit]) and not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -40, 2.0 ** 20, 2.0 ** 60])
def test_fp8_rows_of_any_size(fmt, size):
    # rows of very different sizes, and hidden rows far outside fp16's range
    L = _case(T=5, d=272, E=8, I=48, k=3, fmt=fmt, bias=False)
    L["x"] *= torch.tensor([[1.0], [2.0 ** -30], [size], [2.0 ** -8], [0.0]], device="cuda", dtype=BF)
    L["centroids"].zero_()                                      # the same experts for all
    # h of a row of 2^-100 is near 2^-200, below fp32's normal numbers, and may be lost whole: 3 experts * 48 hidden
    # values of at most 2^-126 times weights below 1 are less than 2^-118
    _check(L, _run(L), tiny=2.0 ** -118)


def test_block_scales_of_the_smallest_byte():
    # w2 near 2^-121: every run's scale is 2^-127 (byte 0).  Results lie near bf16's smallest normal number, 2^-126,
    # below which its step is 2^-133: half of that on top
    L = _case(T=3, d=272, E=6, I=48, k=2, bias=False)
    L["routed"]["w2"] *= 2.0 ** -118
    L["routed"] = quant.quantize_stack(L["routed"], "mxfp8")
    sf2 = L["routed"]["sf2"]
    assert (sf2 == 0).any() and ((sf2 == 0) | (sf2 == 127)).all()
    o = _run(L)
    assert (o["out"] != 0).any()
    _check(L, o, tiny=2.0 ** -134)


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
def test_fp8_infinite_and_nan_inputs_stay_in_their_token(fmt):
    L = _case(T=5, d=272, E=8, I=48, k=3, fmt=fmt, bias=False)
    L["centroids"].zero_()
    want = _run(L)["out"]
    x = L["x"].clone()
    x[1, 7], x[3, 0] = float("inf"), float("nan")
    o = _run(L, x=x)                                            # 0 * infinity: NaN scores, no picks
    with pytest.raises(moe.MoeError):
        moe.check_device_error(o["ws"])
    assert torch.equal(o["out"][[0, 2, 4]], want[[0, 2, 4]])


def test_workspace_outputs_and_rows_around():
    L = _case(T=12, d=520, E=20, I=136, k=4, Ks=1)
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 4, L["shared"])
    n = moe.few_workspace_bytes(shape)
    whole = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = whole[256:256 + n]
    ws[:256] = 0
    big = torch.full((14, 520), 3.0, dtype=BF, device="cuda")
    first = None
    for T in (12, 1, 7, 12):                                    # one workspace for fewer tokens of the same layer, too
        s = moe.shape_of(L["x"][:T], L["centroids"], L["routed"], 4, L["shared"])
        big.fill_(3.0)
        moe.layer_forward_few(s, L["x"][:T], L["centroids"], L["routed"], L["shared"], ws, out=big[1:1 + T])
        assert (big[0] == 3).all() and (big[1 + T:] == 3).all()
        if T == 12:
            first = big.clone() if first is None else first
            assert torch.equal(first, big)                      # the same bits every time
    assert moe.check_device_error(ws) == 0
    assert (whole[:256] == 0x5A).all() and (whole[256 + n:] == 0x5A).all()


def test_captured_and_replayed_with_new_inputs():
    L = _case(T=4, d=512, E=16, I=128, k=3, Ks=1)
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 3, L["shared"])
    ws = moe.new_few_workspace(shape)
    x, out = L["x"].clone(), torch.empty_like(L["x"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        moe.layer_forward_few(shape, x, L["centroids"], L["routed"], L["shared"], ws, out=out)
    for seed in range(3):
        x.copy_(W.make_x(L["cfg"], "cuda", seed=50 + seed))
        g.replay()
        want = _run(L, x=x)["out"]                              # an eager call between two replays, its own workspace
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert moe.check_device_error(ws) == 0


def test_two_streams_with_their_own_workspaces():
    L = _case(T=2, d=1024, E=16, I=256, k=4, Ks=1)
    want = _run(L)["out"]
    streams = [torch.cuda.Stream() for _ in range(2)]
    shape = moe.shape_of(L["x"], L["centroids"], L["routed"], 4, L["shared"])
    wss = [moe.new_few_workspace(shape) for _ in streams]
    outs = [torch.empty_like(L["x"]) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, o in zip(streams, wss, outs):
            moe.layer_forward_few(shape, L["x"], L["centroids"], L["routed"], L["shared"], ws, out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(moe.check_device_error(ws) == 0 for ws in wss)


def test_no_tokens():
    L = _case(T=1, d=64, E=4, I=32, k=2)
    x = L["x"][:0]
    shape = moe.shape_of(x, L["centroids"], L["routed"], 2, None)
    out = moe.layer_forward_few(shape, x, L["centroids"], L["routed"], None, moe.new_few_workspace(shape))
    assert out.shape == (0, 64)


@pytest.mark.parametrize("kw", [dict(T=16, d=1024, E=1024, I=8, k=1), dict(T=16, d=2048, E=600, I=16, k=2, Ks=1, Is=8),
                                dict(T=1, d=1280, E=64, I=320, k=7, Ks=1)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_gates_of_blocks_without_a_routed_unit(kw):
    # fewer units of the up-projection than SMs, and many gates to compute: blocks that had none of them add b2 with
    # gates that nothing else made them wait for.  b2 dominates the result; other calls before each repeat leave other
    # gates in shared memory
    L = _case(**kw)
    L["routed"]["b2"].normal_(0.0, 30.0, generator=torch.Generator(device="cuda").manual_seed(3))
    other = _case(**dict(kw, T=max(1, kw["T"] // 2)), seed=8)
    o = _run(L)
    _check(L, o)
    first = o["out"].clone()
    for _ in range(20):
        _run(other)
        assert torch.equal(_run(L)["out"], first)


@pytest.mark.parametrize("where,fmt", [("routed", None), ("routed", "e4m3"), ("routed", "mxfp8"), ("shared", None), ("shared", "e4m3")])
@pytest.mark.parametrize("T,I", [(1, 16), (11, 1408)])
def test_hidden_values_that_nearly_cancel(where, fmt, T, I):
    # h0 = s (1 + 2^-18), h1 = s, w2 = (1, -1): the result is 2^-18 s, which hidden values of 16 bits lose whole.
    # h in fp32, or in two fp16 parts of 22 bits: two of them are off by 2 (4 * 2^-24 + 2^-23) with the roundings of b's
    # scales, and the two products' sum by 2 * 2^-23 if it truncates, in units of s: less than 2^-20
    L = _case(T=T, d=256, E=1, I=I, k=1, Ks=1, bias=False)
    for n in ("routed", "shared"):
        for w in ("w1", "w3", "w2"):
            L[n][w].zero_()
    L["x"].zero_()
    L["x"][:, 0], L["x"][:, 1] = 1.0, 2.0 ** -18
    i, j = I - 13, I - 5                                        # within one product of 16 columns
    w = L[where]
    w["w1"][0, [i, j], 0] = 1.0
    w["w3"][0, [i, j], 0] = 1.0
    w["w3"][0, i, 1] = 1.0
    w["w2"][0, :, i], w["w2"][0, :, j] = 1.0, -1.0
    if fmt:
        L["routed"] = quant.quantize_stack(L["routed"], fmt)
    o = _run(L)
    assert moe.check_device_error(o["ws"]) == 0
    ref, _ = R.few_layer(L["x"], o["idx"], o["gate"], L["routed"], L["shared"], 1)
    assert (ref > 0.7 * 2.0 ** -18).all()
    assert ((o["out"].double() - ref).abs() <= 2.0 ** -8 * ref + 2.0 ** -20).all()


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_infinite_hidden_values_stay_infinite(fmt):
    # a hidden value beyond fp32's range times finite weights: infinite where the weight is not 0, and NaN where it is
    L = _case(T=2, d=64, E=1, I=32, k=1, Ks=1, bias=False)
    for n in ("routed", "shared"):
        for w in ("w1", "w3", "w2"):
            L[n][w].zero_()
    L["x"][:] = 0
    L["x"][0, 0], L["x"][1, 0] = 2.0 ** 100, 1.0
    L["shared"]["w1"][0, 5, 0] = L["shared"]["w3"][0, 5, 0] = 1.0
    L["shared"]["w2"][0, :, 5] = torch.linspace(-1, 1, 64, device="cuda")
    L["shared"]["w2"][0, 9, 5] = 0.0
    if fmt:
        L["routed"] = quant.quantize_stack(L["routed"], fmt)
    out = _run(L)["out"].float()
    sign = torch.sign(L["shared"]["w2"][0, :, 5].float())
    keep = torch.arange(64, device="cuda") != 9
    assert torch.equal(out[0, keep], sign[keep] * float("inf")) and torch.isnan(out[0, 9])
    assert torch.isfinite(out[1]).all() and (out[1, keep] != 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
@pytest.mark.parametrize("largest,rel", [(m, r) for m in (1.0, 1.9921875, 2.0 ** -90) for r in (1.0, 1.25, 1.5, 1.9921875, 33.0, 2.0 ** 20)] +
                         [(2.0 ** -100, r) for r in (65.0, 2.0 ** 12, 2.0 ** 20)] +       # not below bf16's subnormal step, 2^-133
                         [(m, r) for m in (2.0 ** -112, 2.0 ** -118) for r in (2.0 ** 18, 7.0 * 2.0 ** 18, 2.0 ** 25)])
def test_small_values_beside_a_large_one(fmt, largest, rel):
    # x = (largest, v) with v at rel times the bound below which a value may be lost: h = silu(w v) * b3 with w near 2^-30 / v
    bound = 2.0 ** -39 * largest if largest >= 2.0 ** -112 else 2.0 ** -151
    v = float(torch.tensor(rel * bound, dtype=torch.float64).bfloat16())
    assert v > 0.0
    w = 2.0 ** (-30 - math.frexp(v)[1])
    L = _case(T=1, d=64, E=1, I=16, k=1)
    s = L["routed"]
    for n in ("w1", "w3", "w2", "b1", "b3", "b2"):
        s[n].zero_()
    L["x"].zero_()
    L["x"][0, 0], L["x"][0, 40] = largest, v
    s["w1"][0, 3, 40], s["b3"][0, 3], s["w2"][0, :, 3] = w, 1.0, 1.0
    assert torch.isfinite(s["w1"]).all()
    L["routed"] = quant.quantize_stack(s, fmt)
    o = _run(L)
    ref, _ = R.few_layer(L["x"], o["idx"], o["gate"], L["routed"], None, 0)
    # |silu'| is about 1/2 there; a bf16 result, and 2^-20 for the 22 bits of h and the scales' products
    assert ((o["out"].double() - ref).abs() <= 0.51 * w * bound + (2.0 ** -8 + 2.0 ** -20) * ref.abs()).all()


@pytest.mark.parametrize("fmt", [None, "mxfp8"])
def test_a_workspace_after_an_error(fmt):
    # barriers are counts of arrivals that only grow: whole rounds of them after a call that flagged an error, also once the
    # error word has been read, which clears that word alone
    L = _case(T=3, d=64, E=6, I=32, k=2, Ks=1, fmt=fmt)
    ws = _run(L)["ws"]
    want = _run(L, ws=ws)["out"]
    x = L["x"].clone()
    x[1] = float("nan")
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    for calls in (3, 5):
        _run(L, ws=ws, x=x)
        with pytest.raises(moe.MoeError):
            moe.check_device_error(ws)
        assert ws[64:88].view(torch.int64).tolist() == [calls * blocks, calls * blocks, calls * blocks if fmt else 0]
        o = _run(L, ws=ws)
        assert torch.equal(o["out"], want) and moe.check_device_error(ws) == 0


@pytest.mark.parametrize("fmt", [None, "e4m3", "mxfp8"])
@pytest.mark.parametrize("T", [2, 5, 11])
def test_experts_read_an_infinite_row(fmt, T):
    # sigmoid gates: every key of the infinite row is 1 + bias, so that experts are picked and read it.  All of its hidden
    # values are infinite, and w2's rows have one sign each: infinite results of that sign.  The other tokens keep their bits
    L = _case(T=T, d=272, E=8, I=48, k=3, Ks=1, bias=False, mode=2)
    L["centroids"][:, 7] = 2.0 ** -6
    sign = torch.where(torch.arange(272, device="cuda") % 3 == 0, -1.0, 1.0)
    for n in ("routed", "shared"):
        s = L[n]
        s["w1"][:, :, 7], s["w3"][:, :, 7] = 1.0, 1.0
        s["w2"].copy_((0.5 + s["w2"].float().abs().clamp(max=1.0)) * sign[None, :, None])
    if fmt:
        L["routed"] = quant.quantize_stack(L["routed"], fmt)
    want = _run(L)
    x = L["x"].clone()
    x[T - 1, 7] = float("inf")
    o = _run(L, x=x)
    assert moe.check_device_error(o["ws"]) == 0
    assert torch.equal(o["out"][:-1], want["out"][:-1]) and torch.equal(o["idx"][:-1], want["idx"][:-1])
    top = torch.sort(L["router_bias"], descending=True, stable=True).indices[:3]
    assert torch.equal(o["idx"][-1].long(), top) and ((o["gate"][-1] - 1 / 3).abs() <= 2.0 ** -22).all()
    assert torch.equal(o["out"][-1].float(), sign * float("inf"))
