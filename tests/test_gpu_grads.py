"""Gradient norm and clipping (moe.grad_norm, moe.clip_grads) against 64-bit sums (B200)."""
import math

import pytest
import torch

from fine_grained_mixture_route_b200 import moe

pytestmark = pytest.mark.gpu
# thread sums of 16 squares in fp32 (each term off by at most 16 * 2^-24), all else in 64 bits; the root halves
# that, and the result is rounded once to fp32
NORM_RTOL = 16 * 2.0 ** -25 + 2.0 ** -23


def _norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def _coef(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))


def _check_scaled(out, src, coef):
    for o, s in zip(out, src):
        want = s.double() * coef
        half = 2.0 ** -8 if s.dtype == torch.bfloat16 else 2.0 ** -24
        # the coefficient: the norm's error and its own two roundings
        assert ((o.double() - want).abs() <= (half + NORM_RTOL + 2.0 ** -22) * want.abs() + 1e-38).all()


def _tensors(sizes, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(torch.bfloat16 if i % 2 else torch.float32)
            for i, n in enumerate(sizes)]


LISTS = {"one": [1], "none": [], "empty": [0, 0], "odd": [1, 2, 3, 0, 7, 8, 9, 4097, 16385, 33333], "large": [5_000_003, 7, 3_000_001],
         "many": [17 + i for i in range(500)]}


@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name):
    ts = _tensors(LISTS[name])
    ws = moe.new_grad_workspace()
    n64 = _norm64(ts)
    norm = moe.grad_norm(ts, ws)
    assert norm.dtype == torch.float32 and norm.shape == () and abs(float(norm) - n64) <= NORM_RTOL * n64
    for max_norm in (0.3 * n64, 2 * n64, 0.0, math.inf):
        out = [torch.full_like(t, 7) for t in ts]
        got = moe.clip_grads(ts, max_norm, ws, out=out)
        assert torch.equal(got, norm)                          # the same sums, however it is asked for
        _check_scaled(out, ts, _coef(n64, max_norm))
        mine = [t.clone() for t in ts]
        moe.clip_grads(mine, max_norm, ws)
        assert all(torch.equal(a, b) for a, b in zip(mine, out))


def test_views_at_any_alignment():
    base = _tensors([4099, 70001, 70001])
    ts = [base[0][1:], base[1][3:-2], base[2][5:11], base[2][13:60000]]     # 4-, 2- and 4-byte aligned starts
    outs = [torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")[k:k + t.numel()]
            for k, t in zip((1, 3, 5, 1), ts)]                 # the last one aligned differently from its source
    keep = [b.clone() for b in base]
    ws = moe.new_grad_workspace()
    n64 = _norm64(ts)
    norm = moe.clip_grads(ts, 0.5 * n64, ws, out=outs)
    assert abs(float(norm) - n64) <= NORM_RTOL * n64
    _check_scaled(outs, ts, _coef(n64, 0.5 * n64))
    moe.clip_grads(ts, 0.5 * n64, ws)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))
    assert torch.equal(base[1][:3], keep[1][:3]) and torch.equal(base[1][-2:], keep[1][-2:])
    assert torch.equal(base[2][11:13], keep[2][11:13]) and torch.equal(base[2][60000:], keep[2][60000:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-35, 1e-22, 1e-12, 1e18, 1e30])
def test_sizes_whose_squares_leave_fp32(dtype, scale):
    t = (torch.randn(40000, device="cuda") * scale).to(dtype)
    t[:16000] = 0
    ws = moe.new_grad_workspace()
    n64 = _norm64([t])
    assert abs(float(moe.grad_norm([t], ws)) - n64) <= NORM_RTOL * n64


def test_infinite_and_nan_gradients():
    ws = moe.new_grad_workspace()
    t = torch.ones(1000, device="cuda").bfloat16()
    t[3] = float("inf")
    out = [torch.empty_like(t)]
    assert float(moe.clip_grads([t], 1.0, ws, out=out)) == math.inf
    assert torch.isnan(out[0][3]) and (out[0][:3] == 0).all() and (out[0][4:] == 0).all()
    t[5] = float("nan")
    assert math.isnan(float(moe.clip_grads([t], 1.0, ws, out=out))) and torch.isnan(out[0]).all()
    fine = torch.ones(10, device="cuda")
    assert float(moe.grad_norm([fine], ws)) == pytest.approx(math.sqrt(10), rel=1e-6)   # nothing kept from the call before


def test_not_clipped_is_not_written():
    t = torch.randn(100_000, device="cuda").bfloat16()
    bits = t.clone()
    moe.clip_grads([t], 1e9, moe.new_grad_workspace())
    assert torch.equal(t.view(torch.int16), bits.view(torch.int16))


def test_same_bits_every_time_and_captured():
    ts = _tensors([3_000_001, 1234, 777_777])
    ws = moe.new_grad_workspace()
    out = [torch.empty_like(t) for t in ts]
    norm = torch.empty((), device="cuda")
    want = moe.grad_norm(ts, ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        moe.clip_grads(ts, 0.25, ws, out=out, norm=norm)
    first = None
    for _ in range(3):
        norm.zero_()
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        first = [o.clone() for o in out] if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    _check_scaled(out, ts, _coef(_norm64(ts), 0.25))


def test_offsets_past_31_bits():
    t = torch.zeros((1 << 31) + 5, dtype=torch.bfloat16, device="cuda")
    t[-3:] = torch.tensor([3.0, 4.0, 12.0], device="cuda").bfloat16()
    ws = moe.new_grad_workspace()
    assert float(moe.clip_grads([t], 1.0, ws)) == 13.0
    _check_scaled([t[-3:]], [torch.tensor([3.0, 4.0, 12.0], device="cuda").bfloat16()], _coef(13.0, 1.0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_clipping_of_an_infinite_norm(dtype):
    ws = moe.new_grad_workspace()
    one = torch.ones(1000, device="cuda", dtype=dtype)          # an infinite gradient
    one[3] = float("inf")
    large = torch.full((1000,), 3e38, device="cuda", dtype=dtype)       # finite ones whose norm is beyond fp32
    for t in (one, large):
        mine, out = t.clone(), torch.zeros_like(t)
        assert float(moe.clip_grads([mine], math.inf, ws)) == math.inf and torch.equal(mine, t)
        assert float(moe.clip_grads([t], math.inf, ws, out=[out])) == math.inf and torch.equal(out, t)
    one[5] = float("nan")
    assert math.isnan(float(moe.clip_grads([one], math.inf, ws))) and torch.isnan(one).all()
    small = torch.zeros(10, device="cuda", dtype=dtype)
    assert float(moe.clip_grads([small], math.inf, ws)) == 0.0 and (small == 0).all()
