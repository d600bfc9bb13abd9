"""Plain 64-bit forms of the operators around the layer (tests only), and the bounds that rounding
gives: a rounding to type t is off by at most finfo(t).eps / 2 relative to the value."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# A row's fp32 sum of squares has at most 128 additions in one thread and 10 in the tree, each off by
# 2^-24, and the square root halves what they add up to: rstd is within 2^-17 with room for its own
# four roundings.  v = s * rstd * w adds two more.
F32 = 2.0 ** -17


def rms(s64, eps):
    return 1.0 / torch.sqrt((s64 * s64).mean(1) + eps)


def forward(x, residual, w, eps):
    """(s rounded to the rows' type, rstd, v) in 64 bits."""
    s = x.double() if residual is None else (x.double() + residual.double())
    s = s.to(x.dtype).double()            # fp32 holds the sum of two bf16 rows of like size exactly enough: one rounding
    r = rms(s, eps)
    return s, r, s * r[:, None] * w.double()


def backward(dy, s, w, rstd, dsum):
    s, dy, w, r = s.double(), dy.double(), w.double(), rstd.double()[:, None]
    xhat, g = s * r, dy * w
    m = (g * xhat).mean(1, keepdim=True)
    dx = r * (g - xhat * m)
    size = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, size, (dy * xhat).sum(0), (dy * xhat).abs().sum(0)


def run_exponents(amax):
    """Smallest e with amax <= 448 * 2^e by search, 0 for 0 (64 bits)."""
    e = torch.full_like(amax, -127.0)
    for k in range(-127, 128):
        e = torch.where(amax > 448.0 * 2.0 ** k, torch.full_like(e, float(min(k + 1, 127))), e)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def dense_stack(stack):
    """fp32 weights an expert stack stands for, per expert: {w1, w3, w2, b1, b3, b2} of expert e in 64 bits."""
    def mx(codes, sf, half_of, P):
        rows, K = codes.shape
        r, j = torch.arange(rows, device=codes.device)[:, None], torch.arange(-(-K // 32), device=codes.device)[None]
        blk = (r // P) * (-(-K // 128)) + j // 4
        at = blk * 1024 + half_of(r) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4
        e = sf[at].double() - 127
        return codes.view(torch.float8_e4m3fn).double() * torch.pow(2.0, e).repeat_interleave(32, 1)[:, :K]

    def get(e):
        o = {}
        for w, s in (("w1", "s1"), ("w3", "s3"), ("w2", "s2")):
            t = stack[w][e]
            if t.dtype != torch.uint8:
                o[w] = t.double()
            elif stack.get("sf13") is None:
                o[w] = t.view(torch.float8_e4m3fn).double() * stack[s][e].double()[:, None]
            elif w == "w2":
                o[w] = mx(t, stack["sf2"][e], lambda r: r // 128 % 2, 256)
            else:
                o[w] = mx(t, stack["sf13"][e], lambda r, h=int(w == "w3"): r * 0 + h, 128)
        for b in ("b1", "b3", "b2"):
            o[b] = None if stack.get(b) is None else stack[b][e].double()
        return o
    return get


# fp32 sums of up to 7168 products in 8 warps of MMAs: at most 7168 / 128 + 24 roundings of 2^-23 (an MMA may
# truncate) against the sum of absolute products, and the same for fp32 FMAs; h keeps 16 bits in two bf16 parts
SUM, H16 = 2.0 ** -16, 2.0 ** -16


def expert(w, x):
    """(y, bound on the fp32 kernel's error of y) of one expert for one row, 64 bits."""
    a, g = w["w1"] @ x, w["w3"] @ x
    ea, eg = SUM * (w["w1"].abs() @ x.abs()), SUM * (w["w3"].abs() @ x.abs())
    if w["b1"] is not None:
        a, g = a + w["b1"], g + w["b3"]
        ea, eg = ea + 2.0 ** -24 * a.abs(), eg + 2.0 ** -24 * g.abs()
    s = a * torch.sigmoid(a)
    h = s * g
    eh = 1.1 * ea * g.abs() + s.abs() * eg + H16 * h.abs()     # |silu'| <= 1.1
    y, ey = w["w2"] @ h, w["w2"].abs() @ (eh + SUM * h.abs())
    return (y, ey) if w["b2"] is None else (y + w["b2"], ey + 2.0 ** -24 * w["b2"].abs())


def few_layer(x, idx, gate, routed, shared, Ks):
    """(out, bound before the last rounding) for given picks (idx < 0: left out) and gates."""
    outs, errs = [], []
    R, S = dense_stack(routed), None if shared is None else dense_stack(shared)
    seen = {}
    for t in range(x.shape[0]):
        v = x[t].double()
        o, b = torch.zeros_like(v), torch.zeros_like(v)
        for k in range(Ks):
            y, e = expert(S(k), v)
            o, b = o + y, b + e
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e < 0:
                continue
            seen.setdefault(e, R(e))
            y, err = expert(seen[e], v)
            g = float(gate[t, j])
            o, b = o + g * y, b + g * err + 2.0 ** -22 * g * y.abs()
        outs.append(o)
        errs.append(b)
    return torch.stack(outs), torch.stack(errs)
