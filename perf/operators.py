"""What surrounds the MoE layer in a transformer block, as measured work.

Four operators, each with its plain form (elementary torch operations in 32 bits, rounded once at the end) and
the call a user makes of the framework:

  norm       RMS norm of the residual stream before the layer, with the residual's addition and, for FP8 experts,
             the same rows in 8 bits with scales
  norm_bwd   its gradients
  few        the whole layer (router, routed and shared experts, combine) for 1 to 16 tokens
  grad_norm  the global norm over a training step's gradients
  clip       the same, and the gradients scaled down to a largest norm

Sizes are those of the framework's own layer configurations (tiny, small, mid, decode, prefill), or generic.
"""
import math

import torch

own = False

EPS = 1e-6
STD = 0.006                    # standard deviation of the layer's initial weights
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ the cases
def _norm(name, rows, d, dtype, fmt, residual):
    return dict(name=name, op="norm", rows=rows, d=d, dtype=dtype, fmt=fmt, residual=residual)


def _bwd(name, rows, d, dtype, dsum):
    return dict(name=name, op="norm_bwd", rows=rows, d=d, dtype=dtype, dsum=dsum)


def _few(name, T, d, E, I, k, Ks, bias, dtype="bf16", fmt="native", mode=0):
    return dict(name=name, op="few", T=T, d=d, E=E, I=I, k=k, Ks=Ks, bias=bias, dtype=dtype, fmt=fmt, mode=mode)


def _grads(name, op, layers, d, E, I, Ks, bias, dtype, ratio):
    return dict(name=name, op=op, layers=layers, d=d, E=E, I=I, Ks=Ks, bias=bias, dtype=dtype, ratio=ratio)


def listed():
    return [
        # one new token of a decode step in front of FP8 experts: latency only
        _norm("norm_token", 1, 7168, "bf16", "e4m3", True),
        # a ragged batch of plain rows, a width that is no multiple of 16 and no residual (a first or a final norm)
        _norm("norm_ragged", 999, 2056, "bf16", "none", False),
        # the prefill layer's rows, block-scaled codes beside the 16-bit rows
        _norm("norm_prefill", 16384, 7168, "bf16", "mxfp8", True),
        # the tiny layer's training step, 32 bits
        _bwd("bwd_tiny", 128, 256, "f32", False),
        # the prefill layer's training step, the gradient of the residual stream joining
        _bwd("bwd_prefill", 16384, 7168, "bf16", True),
        # the small layer, one token: launches and dependencies, hardly any bytes
        _few("few_small_1", 1, 1280, 64, 320, 7, 1, True),
        # the decode layer with all of its 256 experts, one user
        _few("few_decode_1", 1, 7168, 256, 2048, 8, 1, True),
        # the prefill layer's expert shape in the block-scaled format, four tokens (a drafted continuation)
        _few("few_mx_4", 4, 7168, 32, 2048, 8, 1, True, fmt="mxfp8"),
        # the mid layer, the largest batch of the kind: most experts are met, some by several tokens
        _few("few_mid_16", 16, 2048, 64, 1408, 6, 2, False),
        # four tiny layers' gradients: many small tensors
        _grads("clip_tiny", "clip", 4, 256, 16, 64, 1, True, "f32", 0.3),
        # the mid layer's gradients, norm alone (what is logged each step)
        _grads("grad_norm_mid", "grad_norm", 1, 2048, 64, 1408, 2, False, "bf16", 1.0),
        # the same gradients clipped
        _grads("clip_mid", "clip", 1, 2048, 64, 1408, 2, False, "bf16", 0.3),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _unnamed(c):
    c.pop("name")
    return c


def draw(rng):
    """One more case: sizes over the whole range of its operator, never more bytes than the largest listed case."""
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "few", "few", "few", "few", "grads", "grads"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = _log_int(rng, 64, 8192, 8)
        if dtype == "f32" and rng.random() < 0.5:
            d = max(1, d - rng.randint(1, 7))                   # odd widths exist in 32 bits only
        rows = _log_int(rng, 1, max(1, min(40000, 16384 * 7168 // (d * (2 if dtype == "f32" else 1)))))
        if op == "norm":
            return _unnamed(_norm("", rows, d, dtype, rng.choice(["none", "e4m3", "mxfp8"]) if dtype == "bf16" else "none",
                                  rng.random() < 0.7))
        return _unnamed(_bwd("", rows, d, dtype, rng.random() < 0.7))
    if op == "few":
        dtype = rng.choice(["bf16"] * 5 + ["f32"])
        fmt = rng.choice(["native", "native", "e4m3", "mxfp8"]) if dtype == "bf16" else "native"
        step = 16 if fmt != "native" else 8
        d = _log_int(rng, 64, 7168 if dtype == "bf16" else 1024, step)
        I = _log_int(rng, 32, 2048 if dtype == "bf16" else 512, step)
        E = _log_int(rng, 2, max(2, min(256, (4 << 30) // (6 * d * I))))
        k = rng.randint(1, min(8, E))
        T = rng.randint(1, 16) if rng.random() < 0.7 else 1
        while T > 1 and T * k * d * I * 12 > (12 << 30):        # the plain form gathers a matrix per pick
            T //= 2
        return _unnamed(_few("", T, d, E, I, k, rng.randint(0, 2), rng.random() < 0.5, dtype, fmt, rng.randint(0, 2)))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = _log_int(rng, 64, 2048, 8)
    I = _log_int(rng, 32, 1408, 8)
    E = _log_int(rng, 1, max(1, min(64, (64 * 2048 * 1408) // (d * I * (2 if dtype == "f32" else 1)))))
    return _unnamed(_grads("", rng.choice(["clip", "clip", "grad_norm"]), rng.randint(1, 3) if E * d * I < 1 << 24 else 1,
                           d, E, I, rng.randint(0, 2), rng.random() < 0.5, dtype, rng.choice([0.1, 0.7, 3.0])))


# ------------------------------------------------------------------------------------------ the inputs
class _Random:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, std, dtype, mean=0.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=self.g)


def _norm_rows(r, case, dt):
    """The residual stream: rows whose size varies, and a few channels much larger than the others."""
    s = r.normal((case["rows"], case["d"]), 1.0, dt)
    s *= (r.normal((case["rows"], 1), 0.5, torch.float32).exp()).to(dt)
    s[:, :: max(1, case["d"] // 5)] *= 16
    return s


def _e4m3_rows(w):
    """16-bit rows -> codes and one fp32 scale per row, as e4m3 expert stacks hold them."""
    amax = w.abs().amax(-1).float()
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (w.float() / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _run_exponents(amax):
    """The smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9), 0 for 0, within [-127, 127]."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8).clamp(-127, 127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _pad_to(t, dim, size, value):
    if t.shape[dim] == size:
        return t
    shape = list(t.shape)
    shape[dim] = size - t.shape[dim]
    return torch.cat([t, torch.full(shape, value, dtype=t.dtype, device=t.device)], dim)


def _mx_rows(w):
    """16-bit rows [..., K] -> codes and the byte e + 127 of each run of 32 inputs."""
    K = w.shape[-1]
    runs = -(-K // 32)
    v = _pad_to(w, w.dim() - 1, runs * 32, 0).unflatten(-1, (runs, 32))
    e = _run_exponents(v.abs().amax(-1).float())
    codes = torch.ldexp(v.float(), -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2)[..., :K].contiguous(), (e + 127).to(torch.uint8)


def _mx_tiles(sf):
    """Bytes [E, halves, groups * 128 rows, chunks * 4 runs] -> the documented 512-byte tiles of each half."""
    E, H, R, J = sf.shape
    t = sf.view(E, H, R // 128, 4, 32, J // 4, 4)                 # expert, half, group, r / 32, r % 32, chunk, run
    return t.permute(0, 2, 5, 1, 4, 3, 6).reshape(E, -1).contiguous()


def _mx_up(s1, s3):
    R, J = -(-s1.shape[1] // 128) * 128, -(-s1.shape[2] // 4) * 4
    return _mx_tiles(torch.stack([_pad_to(_pad_to(s, 1, R, 127), 2, J, 127) for s in (s1, s3)], 1))


def _mx_down(s2):
    R, J = -(-s2.shape[1] // 256) * 256, -(-s2.shape[2] // 4) * 4
    s = _pad_to(_pad_to(s2, 1, R, 127), 2, J, 127)
    return _mx_tiles(s.view(s.shape[0], R // 256, 2, 128, J).transpose(1, 2).reshape(s.shape[0], 2, R // 2, J))


def _stack(r, E, d, I, bias, dt):
    w13 = r.normal((2, E, I, d), STD, dt)                         # w1 and w3 as the halves of one buffer
    s = {"w1": w13[0], "w3": w13[1], "w2": r.normal((E, d, I), STD, dt), "b1": None, "b3": None, "b2": None}
    if bias:
        s.update(b1=r.normal((E, I), 0.1, dt), b3=r.normal((E, I), 0.1, dt), b2=r.normal((E, d), STD, dt))
    return s


def _quantised(s, fmt):
    q, runs = dict(s), {}
    codes13 = torch.empty(s["w1"].shape[:0] + (2,) + s["w1"].shape, dtype=torch.uint8, device="cuda")
    one = _e4m3_rows if fmt == "e4m3" else _mx_rows
    for w in ("w1", "w3", "w2"):
        parts = [one(s[w][e]) for e in range(s[w].shape[0])]      # an expert at a time: 32-bit copies are large
        codes = torch.stack([p[0] for p in parts])
        if w != "w2":
            codes13[0 if w == "w1" else 1] = codes
            codes = codes13[0 if w == "w1" else 1]
        q[w] = codes
        runs[w] = torch.stack([p[1] for p in parts])
    if fmt == "e4m3":
        q.update(s1=runs["w1"], s3=runs["w3"], s2=runs["w2"])
    else:
        q.update(sf13=_mx_up(runs["w1"], runs["w3"]), sf2=_mx_down(runs["w2"]))
    return q, runs


def prepare(case, seed):
    r = _Random(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"case": case}
    if op == "norm":
        st["weight"] = r.normal((case["d"],), 0.2, dt, mean=1.0)
        st["x"] = r.normal((case["rows"], case["d"]), 1.0, dt) if case["residual"] else _norm_rows(r, case, dt)
        st["residual"] = _norm_rows(r, case, dt) if case["residual"] else None
    elif op == "norm_bwd":
        st["weight"] = r.normal((case["d"],), 0.2, dt, mean=1.0)
        st["s"] = _norm_rows(r, case, dt)
        st["rstd"] = (st["s"].double().square().mean(1) + EPS).rsqrt().float()
        st["dy"] = r.normal((case["rows"], case["d"]), 1.0, dt)
        st["dsum"] = r.normal((case["rows"], case["d"]), 1.0, dt) if case["dsum"] else None
    elif op == "few":
        d, E, I = case["d"], case["E"], case["I"]
        st["x"] = r.normal((case["T"], d), 1.0, dt)
        st["centroids"] = r.normal((E, d), 1.0 / math.sqrt(d), dt)
        st["router_bias"] = r.normal((E,), 0.1, torch.float32) if case["mode"] else None
        st["routed"], st["runs"] = _stack(r, E, d, I, case["bias"], dt), None
        if case["fmt"] != "native":
            st["routed"], st["runs"] = _quantised(st["routed"], case["fmt"])
        st["shared"] = _stack(r, case["Ks"], d, I, case["bias"], dt) if case["Ks"] else None
        if own:
            from fine_grained_mixture_route_b200 import moe
            st["shape"] = moe.shape_of(st["x"], st["centroids"], st["routed"], case["k"], st["shared"], case["mode"])
            st["ws"] = moe.new_few_workspace(st["shape"])
    else:
        st["grads"] = []
        for _ in range(case["layers"]):
            d, scale = case["d"], float(torch.empty(1).uniform_(-9, -3, generator=torch.Generator().manual_seed(seed)).exp())
            st["grads"] += [r.normal((case["E"], d), scale, torch.float32), r.normal((d,), scale, torch.float32)]
            for E in (case["E"], case["Ks"]):
                if E:
                    s = _stack(r, E, d, case["I"], case["bias"], dt)
                    st["grads"] += [s[w].mul_(scale / STD) for w in ("w1", "w3", "w2", "b1", "b3", "b2") if s[w] is not None]
        total = math.sqrt(sum(float(g.float().square().sum(dtype=torch.float64)) for g in st["grads"]))
        st["max_norm"] = total * case["ratio"]
        st["out"] = [torch.empty_like(g) for g in st["grads"]] if op == "clip" else None
        if own:
            from fine_grained_mixture_route_b200 import moe
            st["ws"] = moe.new_grad_workspace()
    return st


# ------------------------------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        from fine_grained_mixture_route_b200 import moe
        if op == "norm":
            fmt = {"none": moe.FMT_NATIVE, "e4m3": moe.FMT_E4M3, "mxfp8": moe.FMT_MXFP8}[st["case"]["fmt"]]
            out = moe.rmsnorm(st["x"], st["weight"], eps=EPS, residual=st["residual"], fmt=fmt)
            if out["codes"] is not None:
                out["codes"] = out["codes"].view(torch.float8_e4m3fn)
            if fmt == moe.FMT_MXFP8:
                out["scale"] = out["scale"].view(torch.float8_e8m0fnu)
            return out
        if op == "norm_bwd":
            dx, dw = moe.rmsnorm_backward(st["dy"], st["s"], st["weight"], st["rstd"], dsum=st["dsum"])
            return {"dx": dx, "dweight": dw}
        if op == "few":
            gate = torch.empty((st["case"]["T"], st["case"]["k"]), dtype=torch.float32, device="cuda")
            out = moe.layer_forward_few(st["shape"], st["x"], st["centroids"], st["routed"], st["shared"], st["ws"],
                                        gate=gate, router_bias=st["router_bias"])
            return {"out": out, "gate": gate}
        if op == "grad_norm":
            return {"norm": moe.grad_norm(st["grads"], st["ws"])}
        norm = moe.clip_grads(st["grads"], st["max_norm"], st["ws"], out=st["out"])
        return {"norm": norm, "grads": st["out"]}
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_bwd":
        return _plain_norm_bwd(st)
    if op == "few":
        return _plain_few(st)
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt().float()
    if op == "grad_norm":
        return {"norm": norm}
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, "grads": [(g.float() * coef).to(g.dtype) for g in st["grads"]]}


def _plain_norm(st):
    x, w, fmt = st["x"], st["weight"], st["case"]["fmt"]
    s = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    f = s.float()
    rstd = (f.square().mean(1) + EPS).rsqrt()
    v = f * rstd[:, None] * w.float()
    out = {"y": v.to(x.dtype), "sum": None if st["residual"] is None else s, "rstd": rstd, "codes": None, "scale": None}
    if fmt == "e4m3":
        amax = v.abs().amax(1)
        out["scale"] = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        out["codes"] = (v / out["scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    elif fmt == "mxfp8":
        rows, d = v.shape
        runs = -(-d // 32)
        p = _pad_to(v, 1, runs * 32, 0.0).view(rows, runs, 32)
        e = _run_exponents(p.abs().amax(2))
        out["codes"] = torch.ldexp(p, -e[..., None]).view(rows, -1)[:, :d].to(torch.float8_e4m3fn)
        out["scale"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_norm_bwd(st):
    rstd = st["rstd"][:, None]
    xhat = st["s"].float() * rstd
    dy = st["dy"].float()
    g = dy * st["weight"].float()
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["s"].dtype), "dweight": (dy * xhat).sum(0)}


def _route(x, c, bias, k, mode):
    z = x.double() @ c.double().T                                  # picks next to a border: 64 bits
    b = torch.zeros_like(z[0]) if bias is None else bias.double()
    key = torch.sigmoid(z) + b if mode == 2 else z + b
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    if mode == 0:
        gate = torch.softmax(key, 1).gather(1, idx)
    elif mode == 1:
        gate = torch.softmax(top, 1)
    else:
        gate = torch.sigmoid(z).gather(1, idx)
        gate = gate / gate.sum(1, keepdim=True)
    return idx, gate.float()


def _picked(q, runs, name, idx, fmt):
    """The weight matrices of the given experts in 32 bits."""
    w = q[name][idx]
    if fmt == "native":
        return w.float()
    w = w.view(torch.float8_e4m3fn).float()
    s = runs[name][idx]
    if fmt == "e4m3":
        return w * s[..., None]
    s = torch.exp2(s.float() - 127.0)
    return w * s.repeat_interleave(32, -1)[..., : w.shape[-1]]


def _plain_few(st):
    c, x, q = st["case"], st["x"], st["routed"]
    idx, gate = _route(x, st["centroids"], st["router_bias"], c["k"], c["mode"])
    f = x.float()
    a = torch.matmul(_picked(q, st["runs"], "w1", idx, c["fmt"]), f[:, None, :, None])[..., 0]
    g = torch.matmul(_picked(q, st["runs"], "w3", idx, c["fmt"]), f[:, None, :, None])[..., 0]
    if c["bias"]:
        a, g = a + q["b1"][idx].float(), g + q["b3"][idx].float()
    h = a * torch.sigmoid(a) * g
    y = torch.matmul(_picked(q, st["runs"], "w2", idx, c["fmt"]), h[..., None])[..., 0]
    if c["bias"]:
        y = y + q["b2"][idx].float()
    out = (gate[..., None] * y).sum(1)
    if st["shared"] is not None:
        s = st["shared"]
        a, g = torch.matmul(f, s["w1"].float().mT), torch.matmul(f, s["w3"].float().mT)
        if c["bias"]:
            a, g = a + s["b1"][:, None].float(), g + s["b3"][:, None].float()
        y = torch.matmul(a * torch.sigmoid(a) * g, s["w2"].float().mT)
        if c["bias"]:
            y = y + s["b2"][:, None].float()
        out = out + y.sum(0)
    return {"out": out.to(x.dtype), "gate": gate}


# ------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, b = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        n = case["rows"] * case["d"]
        codes = 0 if case["fmt"] == "none" else n + (4 * case["rows"] if case["fmt"] == "e4m3" else n // 32)
        return {"bytes": n * b * (4 if case["residual"] else 2) + codes + case["d"] * b + 4 * case["rows"], "flops": 6.0 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["d"]
        return {"bytes": n * b * (4 if case["dsum"] else 3) + case["d"] * (b + 4) + 4 * case["rows"], "flops": 10.0 * n}
    if op == "few":
        T, d, E, I, k, Ks = (case[n] for n in ("T", "d", "E", "I", "k", "Ks"))
        met = E * (1.0 - (1.0 - k / E) ** T)                       # experts that some token picks, if all are as likely
        per = {"native": 1.0 * b, "e4m3": 1.0, "mxfp8": 1.0 + 1.0 / 32}[case["fmt"]]
        bias = (2 * I + d) * b if case["bias"] else 0
        scales = 4 * (2 * I + d) if case["fmt"] == "e4m3" else 0
        return {"bytes": met * (3 * d * I * per + bias + scales) + Ks * (3 * d * I * b + bias) + E * d * b + 2 * T * d * b,
                "flops": 2.0 * T * (3 * d * I * (k + Ks) + d * E)}
    n = {"f32": 0, "bf16": 0}
    n["f32"] += case["layers"] * (case["E"] * case["d"] + case["d"])
    n[case["dtype"]] += case["layers"] * (case["E"] + case["Ks"]) * (3 * case["d"] * case["I"] + (2 * case["I"] + case["d"] if case["bias"] else 0))
    return {"bytes": (4 * n["f32"] + 2 * n["bf16"]) * (2 if op == "clip" else 1), "flops": 3.0 * (n["f32"] + n["bf16"])}


# ------------------------------------------------------------------------------------------ the definitions in 64 bits
def _exact_route(x, c, bias, k, mode):
    z = (x.double()[:, None, :] * c.double()[None]).sum(2)
    b = 0.0 if bias is None else bias.double()
    key = (1.0 / (1.0 + torch.exp(-z)) if mode == 2 else z) + b
    idx, left = [], key.clone()
    for _ in range(k):
        i = left.argmax(1)
        idx.append(i)
        left.scatter_(1, i[:, None], -math.inf)
    idx = torch.stack(idx, 1)
    if mode == 0:
        e = torch.exp(key)
        gate = e.gather(1, idx) / e.sum(1, keepdim=True)
    else:
        p = torch.exp(key.gather(1, idx)) if mode == 1 else 1.0 / (1.0 + torch.exp(-z.gather(1, idx)))
        gate = p / p.sum(1, keepdim=True)
    return idx, gate


def _exact_matrix(st, name, e):
    """One routed expert's matrix in 64 bits, from its codes and scales where it is held in 8 bits."""
    w, fmt = st["routed"][name][e], st["case"]["fmt"]
    if fmt == "native":
        return w.double()
    v, s = w.view(torch.float8_e4m3fn).double(), st["runs"][name][e]
    if fmt == "e4m3":
        return v * s.double()[:, None]
    at = torch.arange(v.shape[1], device=v.device) // 32
    return v * torch.pow(2.0, s.double() - 127.0)[:, at]


def _exact_expert(x, w1, w3, w2, b1, b3, b2):
    a, g = w1 @ x, w3 @ x
    if b1 is not None:
        a, g = a + b1.double(), g + b3.double()
    y = w2 @ (a / (1.0 + torch.exp(-a)) * g)
    return y if b2 is None else y + b2.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # the sum is rounded to the rows' type before it is normalised: that rounding belongs to the definition
        full = st["x"].double() + (0.0 if st["residual"] is None else st["residual"].double())
        s = full.to(st["x"].dtype).double()
        rstd = 1.0 / torch.sqrt((s * s).sum(1) / case["d"] + EPS)
        v = s * rstd[:, None] * st["weight"].double()
        out = {"y": v, "sum": full if case["residual"] else None, "rstd": rstd, "codes": None, "scale": None}
        if case["fmt"] == "e4m3":                                  # the codes before their rounding
            top = v.abs().max(1).values
            out["scale"] = torch.where(top == 0, 1.0, top / 448.0)
            out["codes"] = v / out["scale"][:, None]
        elif case["fmt"] == "mxfp8":
            runs = -(-case["d"] // 32)
            at = torch.arange(case["d"], device=v.device) // 32
            top = torch.zeros((case["rows"], runs), dtype=torch.float64, device=v.device)
            top.scatter_reduce_(1, at[None].expand_as(v), v.abs(), "amax")
            e = torch.where(top > 0, torch.ceil(torch.log2(top / 448.0)), 0.0).clamp(-127, 127)
            out["codes"], out["scale"] = v / torch.pow(2.0, e)[:, at], torch.pow(2.0, e)
        return out
    if op == "norm_bwd":
        s, dy, w, r = st["s"].double(), st["dy"].double(), st["weight"].double(), st["rstd"].double()[:, None]
        dot = (dy * w * s).sum(1, keepdim=True)
        dx = r * dy * w - s * dot * r ** 3 / case["d"]
        return {"dx": dx if st["dsum"] is None else dx + st["dsum"].double(), "dweight": (dy * s * r).sum(0)}
    if op == "few":
        idx, gate = _exact_route(st["x"], st["centroids"], st["router_bias"], case["k"], case["mode"])
        rows, b = [], st["routed"]
        for t in range(case["T"]):
            x, y = st["x"][t].double(), torch.zeros(case["d"], dtype=torch.float64, device="cuda")
            for k in range(case["Ks"]):
                s = st["shared"]
                y += _exact_expert(x, *(s[n][k].double() for n in ("w1", "w3", "w2")),
                                   *(None if s[n] is None else s[n][k] for n in ("b1", "b3", "b2")))
            for j in range(case["k"]):
                e = int(idx[t, j])
                y += gate[t, j] * _exact_expert(x, *(_exact_matrix(st, n, e) for n in ("w1", "w3", "w2")),
                                                *(None if b[n] is None else b[n][e] for n in ("b1", "b3", "b2")))
            rows.append(y)
        return {"out": torch.stack(rows), "gate": gate}
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in st["grads"]))
    if op == "grad_norm":
        return {"norm": torch.tensor(norm, dtype=torch.float64)}
    coef = min(1.0, st["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [g.double() * coef for g in st["grads"]]}
