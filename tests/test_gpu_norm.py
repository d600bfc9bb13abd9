"""RMS norm (moe.rmsnorm, moe.rmsnorm_backward) against 64-bit plain forms (B200)."""
import pytest
import torch

from fine_grained_mixture_route_b200 import moe
from tests import block_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(rows, d, dtype, seed=0, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * d + rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = n(rows, d).to(dtype)
    res = (n(rows, d) * n(rows, 1).exp()).to(dtype) if residual else None
    if residual:
        res[:, ::5] *= 16                                       # channels far larger than the others
    return x, res, (1 + 0.2 * n(d)).to(dtype)


def _check_rows(o, x, res, w, eps, fmt):
    s, r, v = R.forward(x, res, w, eps)
    dt = x.dtype
    if res is not None:
        assert torch.equal(o["sum"], (x.float() + res.float()).to(dt))
        s = o["sum"].double()
        r = R.rms(s, eps)
        v = s * r[:, None] * w.double()
    else:
        assert o["sum"] is None
    assert ((o["rstd"].double() - r).abs() <= R.F32 * r).all()
    y = o["y"].double()
    half = R.HALF[dt]
    assert ((y - v).abs() <= (half + R.F32) * v.abs() + 1e-38).all()
    if fmt == moe.FMT_NATIVE:
        assert o["codes"] is None and o["scale"] is None
        return
    q = o["codes"].view(torch.float8_e4m3fn).double()
    if fmt == moe.FMT_E4M3:
        amax = v.abs().amax(1)
        sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        assert ((o["scale"].double() - sc).abs() <= 2 * R.F32 * sc).all()
        u = v / o["scale"].double()[:, None]
    else:
        rows, d = v.shape
        nr = -(-d // 32)
        p = torch.zeros((rows, nr * 32), dtype=torch.float64, device=v.device)
        p[:, :d] = v
        amax = p.view(rows, nr, 32).abs().amax(2)
        e = o["scale"].double() - 127.0
        lo, hi = R.run_exponents(amax * (1 - 2 * R.F32)), R.run_exponents(amax * (1 + 2 * R.F32))
        assert (((e == lo) | (e == hi))).all()                  # the two differ only next to a border
        u = v / torch.pow(2.0, e).repeat_interleave(32, 1)[:, :d]
    # normal codes: half a step relative; below 2^-6: half of the step 2^-9; above 448 by v's own error only
    assert ((q - u).abs() <= (2.0 ** -4 + 4 * R.F32) * u.abs() + 2.0 ** -10).all()
    assert (q.abs() <= 448).all()


@pytest.mark.parametrize("rows,d", [(1, 8), (1, 7168), (3, 264), (37, 1024), (700, 1032), (301, 2056), (600, 8),
                                    (1200, 248), (5, 16384), (400, 16384), (333, 7168)])
@pytest.mark.parametrize("fmt", [moe.FMT_NATIVE, moe.FMT_E4M3, moe.FMT_MXFP8])
@pytest.mark.parametrize("residual", [True, False])
def test_rows_bf16(rows, d, fmt, residual):
    x, res, w = _inputs(rows, d, torch.bfloat16, residual=residual)
    _check_rows(moe.rmsnorm(x, w, eps=EPS, residual=res, fmt=fmt), x, res, w, EPS, fmt)


@pytest.mark.parametrize("rows,d", [(1, 1), (7, 3), (500, 33), (2, 1023), (2, 16383), (700, 16383), (3, 4096), (900, 256),
                                    (350, 4100)])
def test_rows_fp32_of_any_width(rows, d):
    x, res, w = _inputs(rows, d, torch.float32)
    _check_rows(moe.rmsnorm(x, w, eps=EPS, residual=res), x, res, w, EPS, moe.FMT_NATIVE)


def test_fp32_rows_off_16_byte_alignment():
    base = torch.randn(9 * 64 + 1, device="cuda")
    x = base[1:].view(9, 64)
    w = torch.ones(64, device="cuda")
    _check_rows(moe.rmsnorm(x, w), x, None, w, 1e-6, moe.FMT_NATIVE)


def test_special_rows():
    d = 256
    x = torch.randn(6, d, device="cuda").bfloat16()
    x[0] = 0                                                   # a padded row
    x[1] = 1e-30                                               # squares below fp32's range
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4, :32] = 0                                              # a run of zeros
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    for fmt in (moe.FMT_NATIVE, moe.FMT_E4M3, moe.FMT_MXFP8):
        o = moe.rmsnorm(x, w, fmt=fmt)
        assert (o["y"][0] == 0).all() and torch.isfinite(o["y"][[0, 1, 4, 5]]).all()
        assert torch.isnan(o["y"][2, 5]) and (o["y"][2, :5] == 0).all()     # inf * 0, and the others over infinity
        assert torch.isnan(o["y"][3]).all()
        keep = [0, 1, 4, 5]
        part = {k: (None if v is None else v[keep]) for k, v in o.items()}
        _check_rows(part, x[keep], None, w, 1e-6, fmt)
        if fmt == moe.FMT_E4M3:
            assert o["scale"][0] == 1 and (o["codes"][0] == 0).all()
        if fmt == moe.FMT_MXFP8:
            assert (o["scale"][0] == 127).all() and o["scale"][4, 0] == 127


def test_rows_are_independent_and_in_place_sum():
    x, res, w = _inputs(400, 1536, torch.bfloat16)
    one = moe.rmsnorm(x, w, residual=res, fmt=moe.FMT_MXFP8)
    part = moe.rmsnorm(x[17:18].contiguous(), w, residual=res[17:18].contiguous(), fmt=moe.FMT_MXFP8)
    s = res.clone()
    inp = moe.rmsnorm(x, w, residual=s, fmt=moe.FMT_MXFP8, out={"sum": s})
    assert inp["sum"] is s
    for k in ("y", "sum", "codes", "scale", "rstd"):
        assert torch.equal(one[k], inp[k]), k
        # one row alone takes another split of the row over the threads: equal up to the sum's order
        assert ((one[k][17:18].double() - part[k].double()).abs() <= 2 * one[k][17:18].double().abs()).all()
    assert ((one["rstd"][17:18] - part["rstd"]).abs() <= 2 * R.F32 * part["rstd"]).all()


def test_offsets_past_31_bits():
    rows, d = 300_001, 7168                                    # 2.15e9 elements
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, d, device="cuda").bfloat16()
    x[-3:] = tail
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    o = moe.rmsnorm(x, w, fmt=moe.FMT_E4M3)
    last = {k: (None if v is None else v[-3:]) for k, v in o.items()}
    _check_rows(last, tail, None, w, 1e-6, moe.FMT_E4M3)
    assert (o["y"][-4] == 0).all() and o["scale"][-4] == 1


@pytest.mark.parametrize("rows,d,dtype", [(1, 8, torch.bfloat16), (5, 7168, torch.bfloat16), (1000, 2048, torch.bfloat16),
                                          (2500, 264, torch.bfloat16), (900, 7168, torch.bfloat16),
                                          (310, 16384, torch.bfloat16), (64, 1, torch.float32), (333, 35, torch.float32),
                                          (20, 16383, torch.float32), (600, 1028, torch.float32), (310, 8200, torch.float32),
                                          (2600, 64, torch.float32)])
@pytest.mark.parametrize("dsum", [True, False])
def test_backward(rows, d, dtype, dsum):
    s, ds, w = _inputs(rows, d, dtype, seed=1)
    dy = _inputs(rows, d, dtype, seed=2, residual=False)[0]
    ds = ds if dsum else None
    rstd = R.rms(s.double(), EPS).float()
    dx, dw = moe.rmsnorm_backward(dy, s, w, rstd, dsum=ds)
    ref, size, rw, rw_size = R.backward(dy, s, w, rstd, ds)
    assert ((dx.double() - ref).abs() <= R.HALF[dtype] * ref.abs() + 2 * R.F32 * size).all()
    # a column's sum: at most ceil(rows / blocks) additions in a thread, then 32 warps' partials and their tree
    n = rows + 64
    assert ((dw.double() - rw).abs() <= n * 2.0 ** -24 * rw_size + 1e-30).all()
    again = moe.rmsnorm_backward(dy, s, w, rstd, dsum=ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_against_differences():
    rows, d = 3, 40
    s, _, w = _inputs(rows, d, torch.float32, seed=3, residual=False)
    dy = torch.randn(rows, d, device="cuda")
    o = moe.rmsnorm(s, w, eps=EPS)
    dx, dw = moe.rmsnorm_backward(dy, s, w, o["rstd"])
    f = lambda a, b: float((R.forward(a, None, b, EPS)[2] * dy.double()).sum())  # noqa: E731
    h = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 39)):
        up, dn = s.double().clone(), s.double().clone()
        up[i, j] += h
        dn[i, j] -= h
        assert abs((f(up, w.double()) - f(dn, w.double())) / (2 * h) - float(dx[i, j])) <= 1e-4
    for j in (0, 39):
        up, dn = w.double().clone(), w.double().clone()
        up[j] += h
        dn[j] -= h
        assert abs((f(s.double(), up) - f(s.double(), dn)) / (2 * h) - float(dw[j])) <= 1e-4


def test_backward_in_place_and_empty():
    s, ds, w = _inputs(200, 512, torch.bfloat16)
    dy = torch.randn(200, 512, device="cuda").bfloat16()
    rstd = moe.rmsnorm(s, w)["rstd"]
    want = moe.rmsnorm_backward(dy, s, w, rstd, dsum=ds)
    buf = ds.clone()
    got = moe.rmsnorm_backward(dy, s, w, rstd, dsum=buf, dx=buf)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = torch.empty((0, 512), dtype=torch.bfloat16, device="cuda")
    dx, dw = moe.rmsnorm_backward(e, e, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 512) and (dw == 0).all()
    o = moe.rmsnorm(e, w, fmt=moe.FMT_MXFP8)
    assert o["y"].shape == (0, 512) and o["scale"].shape == (0, 16)


def test_captured_on_a_side_stream():
    x, res, w = _inputs(64, 1024, torch.bfloat16)
    want = moe.rmsnorm(x, w, residual=res, fmt=moe.FMT_E4M3)
    dwant = moe.rmsnorm_backward(x, want["sum"], w, want["rstd"], dsum=res)
    out = {k: (None if v is None else torch.empty_like(v)) for k, v in want.items()}
    dx, dw = torch.empty_like(x), torch.empty_like(dwant[1])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        moe.rmsnorm(x, w, residual=res, fmt=moe.FMT_E4M3, out=out)
        moe.rmsnorm_backward(x, out["sum"], w, out["rstd"], dsum=res, dx=dx, dweight=dw, ws=ws)
    for _ in range(2):
        for t in (*[v for v in out.values() if v is not None], dx, dw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
        assert torch.equal(dx, dwant[0]) and torch.equal(dw, dwant[1])


@pytest.mark.parametrize("rows", [1, 700])
def test_codes_between_two_steps_go_to_the_even_one(rows):
    # a row whose mean square is 1 exactly, with the largest value 49: scale 49 / 448 = 7 / 64, and 7 n / 2^j over it is
    # n * 2^(6 - j), with n odd and of 5 bits halfway between two codes.  Times the rounded reciprocal of 7 / 64 it is not
    d = 8192
    v = [49.0] + [s * 7 * n / 2.0 ** j for n in range(17, 32, 2) for j in (4, 5) for s in (1, -1)]
    left = d - sum(t * t for t in v)
    while left > 0:                                             # the rest: powers of two
        t = 1.0
        while t * t > left:
            t /= 2
        v.append(t)
        left -= t * t
    assert left == 0 and len(v) <= d
    x = torch.tensor(v + [0.0] * (d - len(v)), device="cuda").bfloat16()
    assert torch.equal(x.double().square().sum().cpu(), torch.tensor(float(d), dtype=torch.float64))
    o = moe.rmsnorm(x.repeat(rows, 1), torch.ones(d, device="cuda", dtype=torch.bfloat16), eps=0.0, fmt=moe.FMT_E4M3)
    assert (o["rstd"] == 1).all() and (o["scale"] == 7.0 / 64.0).all() and torch.equal(o["y"], x.repeat(rows, 1))
    want = (x.double() / (7.0 / 64.0)).float().to(torch.float8_e4m3fn).view(torch.uint8)      # to the nearest, ties to even
    assert torch.equal(o["codes"], want.repeat(rows, 1))
    codes, scale = moe.quantize_rows_e4m3(o["y"], torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(codes, o["codes"]) and torch.equal(scale, o["scale"])


@pytest.mark.parametrize("size", [1.0, 2.0 ** -30, 2.0 ** 30])
def test_codes_are_those_of_the_ieee_quotient(size):
    # 33 million values over their rows' scales, from the rstd and scale that the kernel returns, in the order of its products
    x = torch.randn(4096, 8192, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16() * size
    w = (torch.randn(8192, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * (1 if size == 1 else 2.0 ** -70)).bfloat16()
    o = moe.rmsnorm(x, w, eps=0.0, fmt=moe.FMT_E4M3)
    v = x.float() * o["rstd"][:, None] * w.float()
    assert torch.equal(o["y"], v.bfloat16())
    assert torch.equal((v / o["scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), o["codes"])


@pytest.mark.parametrize("rows", [2, 700])
@pytest.mark.parametrize("d", [64, 2048])
@pytest.mark.parametrize("s,w,eps", [(2.0 ** -100, 2.0 ** -60, 2.0 ** -100), (2.0 ** -80, 2.0 ** -75, 2.0 ** -80), (2.0 ** 55, 2.0 ** 75, 0.0),
                                     (2.0 ** -100, 1.0, 1e-6), (0.0, 1.0, 1e-6), (1.0, 0.0, 1e-6)])
def test_e4m3_scale_of_rows_whose_products_leave_fp32(rows, d, s, w, eps):
    # s * w lies outside fp32's range, s * rstd * w does not (and rows of zeros or tiny numbers, which look alike)
    x = (torch.randn(rows, d, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") * s).bfloat16()
    x[0] = torch.randn(d, device="cuda").bfloat16() if w >= 0.5 else x[0]       # an ordinary row among them
    _check_rows(moe.rmsnorm(x, torch.full((d,), w, device="cuda").bfloat16(), eps=eps, fmt=moe.FMT_E4M3), x, None,
                torch.full((d,), w, device="cuda").bfloat16(), eps, moe.FMT_E4M3)


@pytest.mark.parametrize("fmt", [moe.FMT_NATIVE, moe.FMT_E4M3, moe.FMT_MXFP8])
@pytest.mark.parametrize("d", [264, 1536, 7168])
def test_a_row_alone_is_the_row_among_others(fmt, d):
    # one row takes another split over the threads than 400 do: the sums' order differs, and with it rstd by 2 F32 at most.
    # Both results are then within half a step of values that far apart: a whole step of y, and of the codes' values
    x, res, w = _inputs(400, d, torch.bfloat16)
    all_ = moe.rmsnorm(x, w, residual=res, fmt=fmt)
    for i in (0, 17, 399):
        one = moe.rmsnorm(x[i:i + 1].clone(), w, residual=res[i:i + 1].clone(), fmt=fmt)
        assert torch.equal(one["sum"][0], all_["sum"][i])
        r = all_["rstd"][i].double()
        assert (one["rstd"][0].double() - r).abs() <= 2 * R.F32 * r
        v = (all_["sum"][i].double() * r * w.double()).abs()
        assert ((one["y"][0].double() - all_["y"][i].double()).abs() <= (2 * R.HALF[torch.bfloat16] + 4 * R.F32) * v).all()
        if fmt == moe.FMT_NATIVE:
            continue
        q = [o.view(torch.float8_e4m3fn).double() for o in (one["codes"][0], all_["codes"][i])]
        if fmt == moe.FMT_E4M3:
            s = [one["scale"][0].double(), all_["scale"][i].double()]
            assert (s[0] - s[1]).abs() <= 4 * R.F32 * s[1]
        else:
            e = [one["scale"][0].double() - 127, all_["scale"][i].double() - 127]
            assert ((e[0] - e[1]).abs() <= 1).all() and (e[0] != e[1]).sum() <= 1      # next to a border of the exponent only
            s = [torch.pow(2.0, k).repeat_interleave(32)[:d] for k in e]
        step = torch.maximum(*s) if fmt == moe.FMT_MXFP8 else s[1]
        assert ((q[0] * s[0] - q[1] * s[1]).abs() <= (2 * 2.0 ** -4 + 8 * R.F32) * v + 2 * 2.0 ** -10 * step).all()
