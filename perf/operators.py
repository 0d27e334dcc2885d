"""Measured cases of the decoder-block operators around the quantized linear layer.

Three operators, each in its plain form (elementary torch operations in 32 or
64 bits) and, where ``own`` is true, as calls of this library:

  norm     residual addition + RMS norm + per-token quantization
           (``qlinear_norm_quantize``);
  gemv     the quantized linear layer for 1 to 16 rows (``qlinear_gemv``);
  experts  the layer grouped by expert over ragged row segments
           (``qlinear_prepare_experts`` before, ``qlinear_grouped_gemm`` timed).

Widths come from the linear layers this repository quantizes (1920 / 5760 /
7680, 5120 / 13824 / 15360) and from generic expert widths (1408, 2048).
"""
import math

import numpy as np
import torch

own = False

EPS = float(np.float32(1e-6))
QMAX = {"f16": 127, "int8": 127, "f16_6": 31}   # activation formats that carry integer codes
LARGEST_NORM = 32760 * 5120
LARGEST_GEMV = 15360 * 5120
LARGEST_EXPERTS = 35552 * 7680 * 1920


def listed():
    return [
        # one decoded token between two layers: latency of one launch
        dict(name="norm 1 token", op="norm", m=1, k=1920, fmt="f16", hadamard=True, residual=True),
        # a ragged prompt without a residual branch, 6-bit codes
        dict(name="norm 333 tokens", op="norm", m=333, k=5120, fmt="f16_6", hadamard=True, residual=False),
        # the 2B-sized block's whole token count, int8 codes returned as the bf16 values they stand for
        dict(name="norm 17776 tokens", op="norm", m=17776, k=1920, fmt="int8", hadamard=True, residual=True),
        # the largest block: bf16 output for an unquantized consumer
        dict(name="norm 32760 tokens", op="norm", m=32760, k=5120, fmt="bf16", hadamard=False, residual=True),
        # one decoded token through the smallest layer
        dict(name="gemv 1x1920x1920", op="gemv", m=1, n=1920, k=1920, fmt="bf16", hadamard=True),
        # a batch of odd size through a long reduction, int8 codes
        dict(name="gemv 5x5120x13824", op="gemv", m=5, n=5120, k=13824, fmt="int8", hadamard=True),
        # the largest batch this form takes, codes of the f16 MMA's type
        dict(name="gemv 16x7680x1920", op="gemv", m=16, n=7680, k=1920, fmt="f16", hadamard=True),
        # one decoded token through the widest layer: weight bandwidth
        dict(name="gemv 1x15360x5120", op="gemv", m=1, n=15360, k=5120, fmt="bf16", hadamard=True),
        # one decoding step of 8 sequences, two experts each, picked out of the token's codes
        dict(name="experts decode", op="experts", e=64, used=64, t=16, n=1408, k=2048, gather=2, tail=0),
        # a small batch's second expert product: about 23 rows an expert, rows already in expert order
        dict(name="experts 1500 rows", op="experts", e=64, used=64, t=1500, n=2048, k=1408, gather=0, tail=12),
        # a prompt with idle experts and a long reduction
        dict(name="experts 6000 rows", op="experts", e=32, used=19, t=6000, n=1920, k=7680, gather=0, tail=7),
        # the 2B-sized block's tokens, two experts each
        dict(name="experts 35552 rows", op="experts", e=8, used=8, t=35552, n=7680, k=1920, gather=2, tail=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "experts"])
    had = rng.random() < 0.7
    if op == "norm":
        k = 128 * _log(rng, 1, 108)
        m = min(_log(rng, 1, 32760), LARGEST_NORM // k)
        fmt = rng.choice(["f16", "f16_6", "int8", "bf16"])
        return dict(op=op, m=m, k=k, fmt=fmt, hadamard=had and fmt != "bf16", residual=rng.random() < 0.7)
    if op == "gemv":
        k = 128 * _log(rng, 1, 108)
        n = min(16 * _log(rng, 1, 960), LARGEST_GEMV // k // 16 * 16)
        return dict(op=op, m=rng.randint(1, 16), n=n, k=k, fmt=rng.choice(["bf16", "int8", "f16", "f16_6"]), hadamard=had)
    e = _log(rng, 1, 64)
    used = rng.randint(max(1, e // 2), e)
    n, k = 16 * _log(rng, 1, 480), 128 * _log(rng, 1, 60)
    while e * n * k > 8 * 7680 * 1920:
        n, k = max(16, n // 32 * 16), max(128, k // 256 * 128)
    t = min(_log(rng, 1, 16384), max(1, LARGEST_EXPERTS // (4 * n * k)))
    return dict(op=op, e=e, used=used, t=t, n=n, k=k, gather=rng.choice([0, 1, 2, 4]), tail=rng.choice([0, 3, 40]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activations(m, k, gen):
    """N(0, 1) rows with about 1% of the channels 30 times as large."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    x *= torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 30.0, 1.0)
    return x.to(torch.bfloat16)


def _stage(h, s):
    """One butterfly stage of distance s: (a, b) -> (a + b, a - b)."""
    v = h.view(*h.shape[:-1], h.shape[-1] // (2 * s), 2, s)
    a, b = v[..., 0, :], v[..., 1, :]
    return torch.stack((a + b, a - b), dim=-2).view(h.shape)


def _rotate(x):
    """Rows times blockdiag(H_128): stages 1, 2, 4, ..., 64, each rounded to fp32."""
    return _stage(_stage(_stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16), 32), 64)


def _token_codes(z, qmax):
    """Per-row symmetric integer codes (fp32 values) and scales amax / qmax of fp32 rows."""
    amax = z.abs().amax(dim=-1)
    q = torch.full_like(amax, qmax)
    zero = amax == 0
    inv = torch.where(zero, amax, torch.div(q, amax))
    return torch.round(z * inv[:, None]), torch.where(zero, amax, torch.div(amax, q))


def _pack(w):
    """NVFP4 of fp32 rows [..., N, K]: codes [..., N, K/2], E4M3 scales [..., N, K/16], tensor scales [...]."""
    amax = w.abs().amax(dim=(-2, -1))
    g = torch.div(amax, torch.full_like(amax, 2688.0))
    b = w.view(*w.shape[:-1], w.shape[-1] // 16, 16)
    sf = torch.div(b.abs().amax(dim=-1), (6.0 * g)[..., None, None]).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = sf.float() * g[..., None, None]
    y = b * torch.where(den == 0, den, den.reciprocal())[..., None]
    a = y.abs()
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
         + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * (y < 0).byte()).view(w.shape)
    return dict(codes=c[..., 0::2] | (c[..., 1::2] << 4), sf=sf, g=g)


def _counts(case, gen):
    """Rows of each expert: ragged, summing to t, zero for the experts that are not used."""
    e, used, t = case["e"], case["used"], case["t"]
    alive = torch.randperm(e, generator=gen, device="cuda")[:used]
    p = torch.softmax(0.5 * torch.randn(used, generator=gen, device="cuda"), 0)
    ids = alive[torch.multinomial(p, t, replacement=True, generator=gen)]
    return torch.bincount(ids, minlength=e)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, k = case["op"], case["k"]
    s = dict(case=case, hadamard=case.get("hadamard", True), lut=torch.tensor(
        [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda"))
    if op == "norm":
        s["x"] = _activations(case["m"], k, gen)
        s["r"] = _activations(case["m"], k, gen) if case["residual"] else None
        s["gamma"] = (1 + 0.1 * torch.randn(k, generator=gen, device="cuda")).to(torch.bfloat16)
        return s
    n = case["n"]
    if op == "gemv":
        w = (0.02 * torch.randn(n, k, generator=gen, device="cuda")).to(torch.bfloat16)
        x = _activations(case["m"], k, gen)
        fmt = case["fmt"]
    else:
        w = (0.02 * torch.randn(case["e"], n, k, generator=gen, device="cuda")).to(torch.bfloat16)
        t, per = case["t"], case["gather"]
        counts = _counts(case, gen)
        s["cap"] = int(counts.max())
        s["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
        tokens = max(1, t // per) if per else t + case["tail"]
        s["rows"] = (torch.randint(0, tokens, (t + case["tail"],), generator=gen, device="cuda").to(torch.int32)
                     if per else None)
        x = _activations(tokens, k, gen)
        s["y"] = torch.full((t + case["tail"], n), 0.25, device="cuda").to(torch.bfloat16)
        fmt = "f16"
    if fmt == "bf16":
        s["a"], s["scales"] = x, None
    else:
        z = x.float()
        q, s["scales"] = _token_codes(_rotate(z) if s["hadamard"] else z, QMAX[fmt])
        s["a"] = q.to(torch.int8 if fmt == "int8" else torch.float16)
    if own:
        from bit_quantized_linear_block_b200 import qlinear as ql
        s["w"] = (ql.qlinear_prepare_weights(w, ql.QL_W_NVFP4, hadamard=s["hadamard"]) if op == "gemv"
                  else ql.qlinear_prepare_experts(w, hadamard=True))
        s["q"] = dict(codes=s["a"], scales=s["scales"])
    else:
        w = w.float()
        s["w"] = _pack(_rotate(w) if s["hadamard"] else w)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _weights(s):
    """fp32 E2M1 value times block scale of the packed weights (the tensor scale stays apart)."""
    c, sf = s["w"]["codes"], s["w"]["sf"].float()
    v = s["lut"][torch.stack((c & 15, c >> 4), dim=-1).long()]
    v = v.view(*sf.shape, 16) * sf[..., None]
    return v.view(*c.shape[:-1], 2 * c.shape[-1])


def _norm(s):
    case, x = s["case"], s["x"]
    h = (x.float() + s["r"].float()).to(torch.bfloat16) if s["r"] is not None else x
    mean = torch.div(h.double().square().sum(-1), torch.full((), float(case["k"]), dtype=torch.float64, device="cuda"))
    rstd = (mean + EPS).sqrt().reciprocal().float()
    y = (h.float() * rstd[:, None] * s["gamma"].float()).to(torch.bfloat16)
    out = dict(residual=h) if s["r"] is not None else {}
    if case["fmt"] == "bf16":
        return dict(out, codes=y)
    z = y.float()
    q, scales = _token_codes(_rotate(z) if s["hadamard"] else z, QMAX[case["fmt"]])
    if case["fmt"] == "int8":
        return dict(out, values=(q * scales[:, None]).to(torch.bfloat16))
    return dict(out, codes=q.to(torch.float16), scales=scales)


def _norm_own(s):
    from bit_quantized_linear_block_b200 import qlinear as ql
    case = s["case"]
    fmt = dict(f16=ql.QL_ACT_INT8_F16, f16_6=ql.QL_ACT_INT6_F16, int8=ql.QL_ROUTE_INT8, bf16=ql.QL_ROUTE_BF16)[case["fmt"]]
    q = ql.qlinear_norm_quantize(s["x"], s["gamma"], fmt, hadamard=s["hadamard"], residual=s["r"], eps=EPS)
    out = dict(residual=q["residual"]) if s["r"] is not None else {}
    if case["fmt"] == "bf16":
        return dict(out, codes=q["codes"])
    if case["fmt"] == "int8":
        return dict(out, values=(q["codes"].float() * q["scales"][:, None]).to(torch.bfloat16))
    return dict(out, codes=q["codes"], scales=q["scales"])


def _gemv(s):
    a = s["a"].float()
    if s["scales"] is None and s["hadamard"]:
        a = _rotate(a)
    alpha = s["w"]["g"] * (1 / 128 if s["hadamard"] else 1.0)
    y = a @ _weights(s).t() * alpha
    return (y if s["scales"] is None else y * s["scales"][:, None]).to(torch.bfloat16)


def _gemv_own(s):
    from bit_quantized_linear_block_b200 import qlinear as ql
    case = s["case"]
    fmt = dict(f16=ql.QL_ACT_INT8_F16, f16_6=ql.QL_ACT_INT6_F16, int8=ql.QL_ROUTE_INT8, bf16=ql.QL_ROUTE_BF16)[case["fmt"]]
    return ql.qlinear_gemv(fmt, s["q"], case["m"], s["w"])


def _experts(s):
    case, off, t = s["case"], s["offsets"].long(), s["case"]["t"]
    row = torch.arange(t, device="cuda")
    e = torch.searchsorted(off[1:], row, right=True)
    pos = row - off[e]
    src = row if s["rows"] is None else s["rows"][:t].long()
    a = torch.zeros(case["e"], s["cap"], case["k"], device="cuda")
    a[e, pos] = s["a"][src].float()
    z = torch.bmm(a, _weights(s).transpose(1, 2))
    s["y"][:t] = (z[e, pos] * (s["scales"][src] * s["w"]["g"][e] * (1 / 128))[:, None]).to(torch.bfloat16)
    return s["y"]


def _experts_own(s):
    from bit_quantized_linear_block_b200 import qlinear as ql
    return ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, s["q"], s["offsets"], s["w"], rows=s["rows"], Y=s["y"])


def run(state):
    op = state["case"]["op"]
    if own:
        return (_norm_own if op == "norm" else _gemv_own if op == "gemv" else _experts_own)(state)
    return (_norm if op == "norm" else _gemv if op == "gemv" else _experts)(state)


def work(case):
    op, k = case["op"], case["k"]
    if op == "norm":
        code = 1 if case["fmt"] == "int8" else 2
        per = 2 + code + (4 if case["residual"] else 0)
        values = case["m"] * k
        return dict(bytes=values * per + 2 * k + (0 if case["fmt"] == "bf16" else 4 * case["m"]),
                    flops=values * (6 + (7 if case["hadamard"] else 0)))
    n = case["n"]
    weight = n * k // 2 + n * k // 16 + 4
    if op == "gemv":
        m = case["m"]
        code = 1 if case["fmt"] == "int8" else 2
        return dict(bytes=weight + m * k * code + 2 * m * n + (0 if case["fmt"] == "bf16" else 4 * m), flops=2 * m * n * k)
    t, per = case["t"], case["gather"]
    tokens = min(t, max(1, t // per)) if per else t
    return dict(bytes=min(case["used"], t) * weight + tokens * (2 * k + 4) + 2 * t * n + 4 * (case["e"] + 1)
                + (4 * t if per else 0), flops=2 * t * n * k)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _h128():
    i = np.arange(128)
    odd = np.array([bin(v).count("1") & 1 for v in range(128)])
    return torch.from_numpy(np.where(odd[i[:, None] & i[None, :]], -1.0, 1.0)).cuda()


def _spin(z):
    return (z.view(-1, 128) @ _h128()).view(z.shape)


def _dense(w):
    """fp64 values of packed NVFP4 rows, from the formats' definitions."""
    c = torch.stack((w["codes"] & 15, w["codes"] >> 4), dim=-1).view(*w["codes"].shape[:-1], -1).long()
    mag, sign = c & 7, 1.0 - 2.0 * (c >> 3).double()
    ex, man = mag >> 1, (mag & 1).double()
    v = sign * torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2(ex.double() - 1))
    b = w["sf"].view(torch.uint8).long()
    ex, man = b >> 3, (b & 7).double()
    sf = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex.double() - 7))
    return v * sf.repeat_interleave(16, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(torch.bfloat16).double()
        y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * s["gamma"].double()
        y = y.to(torch.bfloat16)
        out = dict(residual=h) if s["r"] is not None else {}
        if case["fmt"] == "bf16":
            return dict(out, codes=y.double())
        z = _spin(y.double()) if case["hadamard"] else y.double()
        scales = z.abs().amax(-1) / QMAX[case["fmt"]]
        q = torch.round(z / scales.clamp(min=1e-300)[:, None])
        if case["fmt"] == "int8":
            return dict(out, values=q * scales[:, None])
        return dict(out, codes=q, scales=scales)
    if case["op"] == "gemv":
        a = s["a"].double()
        if s["scales"] is None and case["hadamard"]:
            a = _spin(a)
        y = a @ _dense(s["w"]).t() * s["w"]["g"].double() / (128 if case["hadamard"] else 1)
        return y if s["scales"] is None else y * s["scales"].double()[:, None]
    if 2.0 * case["t"] * case["n"] * case["k"] > 2e14:
        return None
    y, off = s["y"].double(), s["offsets"].tolist()
    for e in range(case["e"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            src = torch.arange(lo, hi, device="cuda") if s["rows"] is None else s["rows"][lo:hi].long()
            w = _dense({f: v[e] for f, v in s["w"].items()})
            y[lo:hi] = s["a"][src].double() @ w.t() * (s["scales"][src].double() * s["w"]["g"][e].double() / 128)[:, None]
    return y
