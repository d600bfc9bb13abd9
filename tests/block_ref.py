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
