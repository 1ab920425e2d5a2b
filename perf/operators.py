"""Workloads of the operators around the tiled product, and their plain forms.

Three groups, as a transformer layer meets them:

  linear       C = act(A @ B + bias) + residual in one launch, with the value before the
               activation saved for the backward pass where training asks for it
  linear_grad  its gradients: dZ = dC * act'(Z), dA = dZ @ B^T, dB = A^T @ dZ and the
               bias gradient (the column sums of dZ)
  norm         H = X + residual, Y = H / rms(H) * weight, in 16 bits or in 8 bits (e4m3)
               with one scale per row
  norm_grad    the gradients of Y and of the residual stream with respect to X and weight
  scaled       the product of two e4m3 operands with one scale per row of A and per
               column of B, with the same epilogue as `linear`

`run` computes them with elementary torch operations in 32 bits, or, where `own` is set,
with tile_scheduling_amd.  Sizes: the repository's workload shapes (4096, 8192, 16384,
2048, 1000, 5000 x 12290) and generic ones around them.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
_SQRT_HALF = math.sqrt(0.5)
_TANH_C = math.sqrt(2.0 / math.pi)
_TANH_A = 0.044715

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")


def _linear(m, n, k, dtype, out, w, act, bias, residual, preact=False):
    return {"op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "out": out, "w": w, "act": act,
            "bias": bias, "residual": residual, "preact": preact}


def _grad(m, n, k, dtype, w, act):
    return {"op": "linear_grad", "m": m, "n": n, "k": k, "dtype": dtype, "w": w, "act": act}


def _norm(m, n, dtype, to, residual):
    return {"op": "norm", "m": m, "n": n, "dtype": dtype, "to": to, "residual": residual}


def _norm_grad(m, n, dtype, stream):
    return {"op": "norm_grad", "m": m, "n": n, "dtype": dtype, "stream": stream}


def _scaled(m, n, k, out, act, bias, residual):
    return {"op": "scaled", "m": m, "n": n, "k": k, "out": out, "act": act, "bias": bias, "residual": residual}


def listed():
    return [
        # one token through an output projection, added to the residual stream (latency)
        {"name": "linear_1x4096x4096", **_linear(1, 4096, 4096, "bf16", "bf16", "nk", "none", True, True)},
        # a small decoding batch through an up projection with odd sizes, weights stored [K][N]
        {"name": "linear_13x12290x1000", **_linear(13, 12290, 1000, "f16", "f16", "kn", "gelu", True, False)},
        # the ragged product of the benchmark with a 32-bit residual stream
        {"name": "linear_5000x12290x1000", **_linear(5000, 12290, 1000, "bf16", "f32", "kn", "gelu_tanh", True, True)},
        # a training step's up projection, the value before the activation saved
        {"name": "linear_4096x16384x4096", **_linear(4096, 16384, 4096, "bf16", "bf16", "nk", "gelu", True, False, True)},
        # the backward pass of a short batch of tokens (1000 rows: not a multiple of a tile)
        {"name": "linear_grad_1000x2048x512", **_grad(1000, 2048, 512, "f16", "kn", "silu")},
        # the backward pass of a training step
        {"name": "linear_grad_4096x8192x4096", **_grad(4096, 8192, 4096, "bf16", "nk", "gelu")},
        # one token's norm in front of an 8-bit product (latency)
        {"name": "norm_1x4096", **_norm(1, 4096, "bf16", "e4m3", True)},
        # a prompt's norm in front of an 8-bit product
        {"name": "norm_5000x8192", **_norm(5000, 8192, "bf16", "e4m3", True)},
        # the backward pass of a norm, with the gradient that comes along the residual stream
        {"name": "norm_grad_8192x4096", **_norm_grad(8192, 4096, "bf16", True)},
        # a decoding batch of four tokens with 8-bit weights
        {"name": "scaled_4x8192x8192", **_scaled(4, 8192, 8192, "bf16", "none", True, True)},
        # a ragged prompt with 8-bit weights whose rows are not a multiple of 16 bytes
        {"name": "scaled_5000x12290x1000", **_scaled(5000, 12290, 1000, "f16", "relu", True, False)},
        # a prompt's up projection in 8 bits
        {"name": "scaled_4096x16384x4096", **_scaled(4096, 16384, 4096, "bf16", "silu", True, False)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """Log-uniform; half of the sizes are rounded down to a multiple of 64 where there is one."""
    v = _log(rng, lo, hi)
    return v // 64 * 64 if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "norm", "norm_grad", "scaled", "scaled"))
    dtype = rng.choice(("f16", "bf16"))
    if op in ("norm", "norm_grad"):
        n = _size(rng, 16 if op == "norm_grad" else 1, 16384)
        m = _size(rng, 1, max(1, min(16384, (1 << 26) // n)))
        if op == "norm_grad":
            return _norm_grad(m, n, rng.choice(("f16", "bf16", "f32")), rng.random() < 0.5)
        dtype = rng.choice(("f16", "bf16", "f32"))
        return _norm(m, n, dtype, rng.choice((dtype, "e4m3")), rng.random() < 0.7)
    m, n, k = _size(rng, 1, 8192), _size(rng, 16, 16384), _size(rng, 16, 8192)
    most = 1 << (37 if op == "linear_grad" else 38)
    while m * n * k > most:
        m = max(1, m // 2)
    act = rng.choice(ACTS)
    if op == "linear_grad":
        return _grad(m, n, k, dtype, rng.choice(("nk", "kn")), act)
    if op == "scaled":
        return _scaled(m, n, k, rng.choice(("f16", "bf16", "f32")), act, rng.random() < 0.7, rng.random() < 0.5)
    return _linear(m, n, k, dtype, rng.choice((dtype, "f32")), rng.choice(("nk", "kn")), act, rng.random() < 0.7,
                   rng.random() < 0.5, rng.random() < 0.3)


def work(case):
    m, n, k = case["m"], case["n"], case.get("k", 0)
    if case["op"] == "linear":
        s, o = SIZE[case["dtype"]], SIZE[case["out"]]
        b = (m * k + k * n) * s + m * n * o * (1 + case["residual"] + case["preact"]) + n * s * case["bias"]
        return {"bytes": b, "flops": 2 * m * n * k}
    if case["op"] == "linear_grad":
        s = SIZE[case["dtype"]]
        return {"bytes": 2 * (m * k + k * n + m * n) * s + 4 * n, "flops": 4 * m * n * k}
    if case["op"] == "norm":
        s, o = SIZE[case["dtype"]], SIZE[case["to"]]
        b = m * n * (s * (3 if case["residual"] else 1) + o) + n * s + (4 * m if case["to"] == "e4m3" else 0)
        return {"bytes": b, "flops": 5 * m * n}
    if case["op"] == "norm_grad":
        s = SIZE[case["dtype"]]
        return {"bytes": m * n * s * (3 + case["stream"]) + 2 * n * s, "flops": 9 * m * n}
    o = SIZE[case["out"]]
    b = m * k + k * n + 4 * (m + n) + m * n * o * (1 + case["residual"]) + n * o * case["bias"]
    return {"bytes": b, "flops": 2 * m * n * k}


# ---- inputs ----------------------------------------------------------------------------


def _quantised(x):
    """e4m3 rows and their scales (the value is q * scale)."""
    scale = (x.abs().amax(dim=1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case)
    m, n, k = case["m"], case["n"], case.get("k", 0)
    if case["op"] in ("linear", "linear_grad"):
        dt = DT[case["dtype"]]
        s["a"] = normal(m, k).to(dt)
        # weights of variance 1 / k, stored [N][K] (a projection's weight matrix) or [K][N]
        w = (normal(n, k) if case["w"] == "nk" else normal(k, n)) * (1.0 / math.sqrt(k))
        s["weight"] = w.to(dt)
        s["b"] = s["weight"].t() if case["w"] == "nk" else s["weight"]
        if case["op"] == "linear":
            s["bias"] = normal(n).to(dt) if case["bias"] else None
            s["res"] = normal(m, n).to(DT[case["out"]]) if case["residual"] else None
        else:
            s["z"] = normal(m, n).to(dt)
            s["dc"] = normal(m, n).to(dt)
    elif case["op"] == "norm":
        dt = DT[case["dtype"]]
        s["x"] = normal(m, n).to(dt)
        s["res"] = normal(m, n).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * normal(n)).to(dt)
    elif case["op"] == "norm_grad":
        dt = DT[case["dtype"]]
        s["h"] = normal(m, n).to(dt)
        s["dy"] = normal(m, n).to(dt)
        s["dh"] = normal(m, n).to(dt) if case["stream"] else None
        s["weight"] = (1.0 + 0.1 * normal(n)).to(dt)
    else:
        s["qa"], s["sa"] = _quantised(normal(m, k))
        s["qb"], s["sb"] = _quantised(normal(n, k) * (1.0 / math.sqrt(k)))
        s["bias"] = normal(n).to(DT[case["out"]]) if case["bias"] else None
        s["res"] = normal(m, n).to(DT[case["out"]]) if case["residual"] else None
    return s


# ---- the plain forms ---------------------------------------------------------------------


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * _SQRT_HALF))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_TANH_C * (z + _TANH_A * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * _SQRT_HALF)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(_TANH_C * (z + _TANH_A * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _TANH_C * (1.0 + 3.0 * _TANH_A * z * z)
    if act == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return g * (1.0 + z * (1.0 - g))
    return torch.ones_like(z)


def _epilogue(z, s, dt):
    c = _act(z, s["act"])
    if s["res"] is not None:
        c = c + s["res"].float()
    return c.to(dt)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "linear":
        z = s["a"].float() @ s["b"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = {"c": _epilogue(z, s, DT[s["out"]])}
        if s["preact"]:
            out["preact"] = z.to(DT[s["out"]])
        return out
    if s["op"] == "linear_grad":
        dz = s["dc"].float() * _act_grad(s["z"].float(), s["act"])
        dt = DT[s["dtype"]]
        return {"da": (dz @ s["b"].float().t()).to(dt), "db": (s["a"].float().t() @ dz).to(dt), "dbias": dz.sum(0)}
    if s["op"] == "norm":
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
        out = {} if s["res"] is None else {"h": h.to(s["x"].dtype)}
        if s["to"] == "e4m3":
            out["scale"] = (y.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
            out["y"] = (y / out["scale"][:, None]).to(torch.float8_e4m3fn)
        else:
            out["y"] = y.to(DT[s["to"]])
        return out
    if s["op"] == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        g = dy * s["weight"].float()
        dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * (h * r)).sum(0).to(s["h"].dtype)}
    z = (s["qa"].float() @ s["qb"].float().t()) * s["sa"][:, None] * s["sb"][None, :]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    return {"c": _epilogue(z, s, DT[s["out"]])}


# ---- the framework's calls -------------------------------------------------------------------


def _run_own(s):
    import tile_scheduling_amd as ts

    if s["op"] == "linear":
        z = torch.empty(s["m"], s["n"], dtype=DT[s["out"]], device=s["a"].device) if s["preact"] else None
        c = ts.gemm_epilogue(s["a"], s["b"], bias=s["bias"], activation=s["act"], residual=s["res"], preact=z,
                             out_dtype=DT[s["out"]])
        return {"c": c} if z is None else {"c": c, "preact": z}
    if s["op"] == "linear_grad":
        da, db, dbias = ts.gemm_epilogue_backward(s["dc"], s["a"], s["b"], preact=s["z"], activation=s["act"])
        return {"da": da, "db": db, "dbias": dbias}
    if s["op"] == "norm":
        y, scale, h = ts.rmsnorm(s["x"], s["weight"], residual=s["res"], eps=EPS, out_dtype=DT[s["to"]])
        out = {"y": y}
        if scale is not None:
            out["scale"] = scale
        if s["res"] is not None:
            out["h"] = h
        return out
    if s["op"] == "norm_grad":
        dx, dw = ts.rmsnorm_backward(s["dy"], s["h"], s["weight"], eps=EPS, dh=s["dh"])
        return {"dx": dx, "dweight": dw}
    c = ts.gemm_scaled(s["qa"], s["qb"].t(), s["sa"], s["sb"], bias=s["bias"], activation=s["act"],
                       residual=s["res"], out_dtype=DT[s["out"]])
    return {"c": c}


# ---- the definitions in 64 bits --------------------------------------------------------------


def _phi(z):
    """The normal distribution function, with the tail that 1 + erf loses."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _gate(z, act):
    """act(z) = z * gate(z), and the gate's derivative."""
    if act == "relu":
        return (z > 0).double(), torch.zeros_like(z)
    if act == "gelu":
        return _phi(z), torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)
        g = torch.sigmoid(u)
        return g, g * torch.sigmoid(-u) * math.sqrt(8.0 / math.pi) * (1.0 + 0.134145 * z ** 2)
    if act == "silu":
        g = torch.sigmoid(z)
        return g, g * torch.sigmoid(-z)
    return torch.ones_like(z), torch.zeros_like(z)


def _product64(a, b):
    """a @ b in 64 bits, by blocks of rows to bound the memory."""
    return torch.cat([a[i:i + 2048].double() @ b.double() for i in range(0, a.shape[0], 2048)])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("linear", "scaled"):
        if case["op"] == "linear":
            z = _product64(s["a"], s["b"])
        else:
            z = _product64(s["qa"].float(), s["qb"].float().t())
            z = z * s["sa"].double()[:, None] * s["sb"].double()[None, :]
        if s["bias"] is not None:
            z = z + s["bias"].double()
        c = z * _gate(z, case["act"])[0]
        if s["res"] is not None:
            c = c + s["res"].double()
        return {"c": c, "preact": z} if case.get("preact") else {"c": c}
    if case["op"] == "linear_grad":
        z = s["z"].double()
        g, dg = _gate(z, case["act"])
        dz = s["dc"].double() * (g + z * dg)
        return {"da": _product64(dz, s["b"].t()), "db": _product64(s["a"].t(), dz), "dbias": dz.sum(0)}
    w = s["weight"].double()
    if case["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        y = w * h / torch.sqrt(h.square().sum(1, keepdim=True) / case["n"] + EPS)
        out = {} if s["res"] is None else {"h": h}
        if case["to"] == "e4m3":
            scale = torch.maximum(y.abs().amax(1) / E4M3_MAX, torch.full_like(y[:, 0], SCALE_MIN))
            return {**out, "y": y / scale[:, None], "scale": scale}
        return {**out, "y": y}
    h, dy = s["h"].double(), s["dy"].double()
    rms = torch.sqrt(h.square().sum(1, keepdim=True) / case["n"] + EPS)
    unit = h / rms
    dx = (w * dy - unit * ((w * dy * unit).sum(1, keepdim=True) / case["n"])) / rms
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dweight": (dy * unit).sum(0)}
