"""Workloads of the second set of operators around the tiled product, and their plain forms.

  layernorm       H = X + residual, Y = (H - mean) / sqrt(var + eps) * weight + bias, in 16
                  bits or in 8 bits (e4m3) with one scale per row
  layernorm_grad  the gradients with respect to X, weight and bias, from H as it was or from
                  H kept in 8 bits
  int8            the product of two int8 operands with one scale per row of A (token) and
                  per column of B (channel), with bias, activation and residual
  project8        a projection of 16-bit rows in 8 bits: rows (or their layer norm) rounded to
                  int8 with one scale a row, then the product above
  checkpoint      the value before an activation kept in 8 bits for the backward pass, and
                  what that makes of it: the activation's value again (an operand of the next
                  weight's gradient), dZ = dU * act'(Z) and the bias gradient
  linear_step     a linear layer's training step: U = act(X @ W + bias) with the value before
                  the activation kept in 8 bits by the product itself, and dX, dW, dbias from it

8 bits of a checkpoint: int8 values with one power of two for each 32 columns of a row.
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
EPS = 1e-5
E4M3_MAX = 448.0
INT8_MAX = 127.0
SCALE_MIN = 2.0 ** -100
_SQRT_HALF = math.sqrt(0.5)
_TANH_C = math.sqrt(2.0 / math.pi)
_TANH_A = 0.044715

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")


def _layernorm(m, n, dtype, to, residual):
    return {"op": "layernorm", "m": m, "n": n, "dtype": dtype, "to": to, "residual": residual}


def _layernorm_grad(m, n, dtype, stream, kept8):
    return {"op": "layernorm_grad", "m": m, "n": n, "dtype": dtype, "stream": stream, "kept8": kept8}


def _int8(m, n, k, out, act, bias, residual):
    return {"op": "int8", "m": m, "n": n, "k": k, "out": out, "act": act, "bias": bias, "residual": residual}


def _project8(m, n, k, dtype, norm, act, residual):
    return {"op": "project8", "m": m, "n": n, "k": k, "dtype": dtype, "norm": norm, "act": act, "residual": residual}


def _checkpoint(m, n, dtype, act):
    return {"op": "checkpoint", "m": m, "n": n, "dtype": dtype, "act": act}


def _linear_step(m, n, k, dtype, w, act):
    return {"op": "linear_step", "m": m, "n": n, "k": k, "dtype": dtype, "w": w, "act": act}


def listed():
    return [
        # one token's norm, added to the residual stream (latency)
        {"name": "layernorm_1x4096", **_layernorm(1, 4096, "bf16", "bf16", True)},
        # a prompt's norm in front of an 8-bit product
        {"name": "layernorm_5000x8192", **_layernorm(5000, 8192, "bf16", "e4m3", True)},
        # the backward pass of a short batch of tokens, its rows kept in 8 bits
        {"name": "layernorm_grad_1000x2048", **_layernorm_grad(1000, 2048, "f16", False, True)},
        # the backward pass of a training batch, with the gradient that comes along the residual stream
        {"name": "layernorm_grad_8192x4096", **_layernorm_grad(8192, 4096, "bf16", True, False)},
        # a ragged prompt with 8-bit weights whose rows are not a multiple of 16 bytes
        {"name": "int8_5000x12290x1000", **_int8(5000, 12290, 1000, "f16", "relu", True, False)},
        # a prompt's up projection in 8 bits
        {"name": "int8_4096x16384x4096", **_int8(4096, 16384, 4096, "bf16", "silu", True, False)},
        # one token through an output projection, added to the residual stream (latency)
        {"name": "project8_1x4096x4096", **_project8(1, 4096, 4096, "bf16", False, "none", True)},
        # a prompt's norm and up projection
        {"name": "project8_2048x8192x4096", **_project8(2048, 8192, 4096, "bf16", True, "gelu", False)},
        # the activation of a short batch of tokens (1000 rows: not a multiple of a tile)
        {"name": "checkpoint_1000x2048", **_checkpoint(1000, 2048, "f16", "silu")},
        # the activation of a training batch
        {"name": "checkpoint_4096x16384", **_checkpoint(4096, 16384, "bf16", "gelu")},
        # the training step of a small layer on a short batch
        {"name": "linear_step_1000x2048x512", **_linear_step(1000, 2048, 512, "f16", "kn", "silu")},
        # the training step of an up projection
        {"name": "linear_step_4096x8192x4096", **_linear_step(4096, 8192, 4096, "bf16", "nk", "gelu")},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """Log-uniform; half of the sizes are rounded down to a multiple of 64 where there is one."""
    v = _log(rng, lo, hi)
    return v // 64 * 64 if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("layernorm", "layernorm_grad", "int8", "int8", "project8", "checkpoint", "linear_step"))
    dtype = rng.choice(("f16", "bf16"))
    if op in ("layernorm", "layernorm_grad", "checkpoint"):
        n = _size(rng, 16 if op == "layernorm_grad" else 1, 16384)
        m = _size(rng, 1, max(1, min(16384, (1 << 26) // n)))
        dtype = rng.choice(("f16", "bf16", "f32"))
        if op == "layernorm":
            return _layernorm(m, n, dtype, rng.choice((dtype, "e4m3")), rng.random() < 0.7)
        if op == "layernorm_grad":
            return _layernorm_grad(m, n, dtype, rng.random() < 0.5, rng.random() < 0.5)
        return _checkpoint(m, n, dtype, rng.choice(ACTS[1:]))
    m, n, k = _size(rng, 1, 8192), _size(rng, 16, 16384), _size(rng, 16, 8192)
    most = 1 << (37 if op == "linear_step" else 38)
    while m * n * k > most:
        m = max(1, m // 2)
    if op == "linear_step":
        return _linear_step(m, n, k, dtype, rng.choice(("nk", "kn")), rng.choice(ACTS[1:]))
    act = rng.choice(ACTS)
    if op == "project8":
        return _project8(m, n, k, dtype, rng.random() < 0.5, act, rng.random() < 0.5)
    return _int8(m, n, k, rng.choice(("f16", "bf16", "f32")), act, rng.random() < 0.7, rng.random() < 0.5)


def _blocks(n):
    return -(-n // 32)


def work(case):
    m, n, k = case["m"], case["n"], case.get("k", 0)
    kept = m * _blocks(n) * 33   # a checkpoint's bytes
    if case["op"] == "layernorm":
        s, o = SIZE[case["dtype"]], SIZE[case["to"]]
        b = m * n * (s * (3 if case["residual"] else 1) + o) + 2 * n * s + (4 * m if case["to"] == "e4m3" else 0)
        return {"bytes": b, "flops": 8 * m * n}
    if case["op"] == "layernorm_grad":
        s = SIZE[case["dtype"]]
        b = m * n * s * (2 + case["stream"]) + (kept if case["kept8"] else m * n * s) + 3 * n * s
        return {"bytes": b, "flops": 14 * m * n}
    if case["op"] == "int8":
        o = SIZE[case["out"]]
        b = m * k + k * n + 4 * (m + n) + m * n * o * (1 + case["residual"]) + n * o * case["bias"]
        return {"bytes": b, "flops": 2 * m * n * k}
    if case["op"] == "project8":
        s = SIZE[case["dtype"]]
        b = m * k * s + k * n + 4 * n + m * n * s * (1 + case["residual"]) + (2 * k * s if case["norm"] else 0) + n * s
        return {"bytes": b, "flops": 2 * m * n * k}
    if case["op"] == "checkpoint":
        s = SIZE[case["dtype"]]
        return {"bytes": 4 * m * n * s + 2 * kept + 4 * n, "flops": 30 * m * n}
    s = SIZE[case["dtype"]]
    return {"bytes": 2 * (m * k + k * n + m * n) * s + 2 * kept + 2 * n * s, "flops": 6 * m * n * k}


# ---- inputs ----------------------------------------------------------------------------


def _codes(x):
    """int8 rows and their scales (the value is q * scale), for inputs that a program has as such."""
    scale = (x.abs().amax(dim=1) / INT8_MAX).clamp_min(SCALE_MIN)
    return (x / scale[:, None]).round().to(torch.int8), scale


def _pitch(n):
    """Bytes of a checkpoint's row: its values, 32 a block, then one exponent a block."""
    return -(-_blocks(n) * 33 // 64) * 64


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case)
    m, n, k = case["m"], case["n"], case.get("k", 0)
    dt = DT[case.get("dtype", "f32")]
    if case["op"] in ("layernorm", "layernorm_grad"):
        # rows with a mean of their own, of the size of their spread
        x = normal(m, n) + normal(m, 1)
        s["weight"] = (1.0 + 0.1 * normal(n)).to(dt)
        if case["op"] == "layernorm":
            s["x"] = x.to(dt)
            s["bias"] = (0.1 * normal(n)).to(dt)
            s["res"] = normal(m, n).to(dt) if case["residual"] else None
        else:
            if case["kept8"]:
                q, e = _to_blocks(x.to(dt).float())
                kept = torch.zeros(m, _pitch(n), dtype=torch.uint8, device=DEV)
                kept[:, :32 * _blocks(n)] = q.reshape(m, -1).to(torch.int8).view(torch.uint8)
                kept[:, 32 * _blocks(n):33 * _blocks(n)] = e.reshape(m, -1).to(torch.uint8)
                s["kept"] = kept
            else:
                s["h"] = x.to(dt)
            s["dy"] = normal(m, n).to(dt)
            s["dh"] = normal(m, n).to(dt) if case["stream"] else None
    elif case["op"] == "int8":
        s["qa"], s["sa"] = _codes(normal(m, k))
        s["qb"], s["sb"] = _codes(normal(n, k) * (1.0 / math.sqrt(k)))
        s["bias"] = normal(n).to(DT[case["out"]]) if case["bias"] else None
        s["res"] = normal(m, n).to(DT[case["out"]]) if case["residual"] else None
    elif case["op"] == "project8":
        s["x"] = normal(m, k).to(dt)
        s["qb"], s["sb"] = _codes(normal(n, k) * (1.0 / math.sqrt(k)))
        s["bias"] = normal(n).to(dt)
        s["res"] = normal(m, n).to(dt) if case["residual"] else None
        if case["norm"]:
            s["gain"] = (1.0 + 0.1 * normal(k)).to(dt)
            s["shift"] = (0.1 * normal(k)).to(dt)
    elif case["op"] == "checkpoint":
        s["z"] = normal(m, n).to(dt)
        s["du"] = normal(m, n).to(dt)
    else:
        s["x"] = normal(m, k).to(dt)
        # weights of variance 1 / k, stored [N][K] (a projection's weight matrix) or [K][N]
        w = (normal(n, k) if case["w"] == "nk" else normal(k, n)) * (1.0 / math.sqrt(k))
        s["weight"] = w.to(dt)
        s["wkn"] = s["weight"].t() if case["w"] == "nk" else s["weight"]
        s["bias"] = normal(n).to(dt)
        s["du"] = normal(m, n).to(dt)
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


def _to_blocks(x):
    """int8 values [m, blocks, 32] and biased exponents [m, blocks, 1] of fp32 rows: the power of
    two of a block is the least that brings its largest value to 127 or below, rounded."""
    m, n = x.shape
    pad = 32 * _blocks(n) - n
    if pad:
        x = torch.cat([x, x.new_zeros(m, pad)], dim=1)
    x = x.reshape(m, -1, 32)
    most = x.abs().amax(2, keepdim=True)
    # the exponent of 127.5 / 128 of the next power of two on counts as that power's own
    e = (((most.view(torch.int32) + 0x10000) >> 23) - 6).clamp_min(1)
    return (x * ((254 - e) << 23).view(torch.float32)).round(), e


def _from_blocks(q, e, n):
    x = q * (e << 23).view(torch.float32)
    return x.reshape(x.shape[0], -1)[:, :n]


def _kept(kept, n):
    """The rows that a checkpoint's bytes stand for."""
    b = _blocks(n)
    q = kept[:, :32 * b].view(torch.int8).float().reshape(-1, b, 32)
    return _from_blocks(q, kept[:, 32 * b:33 * b].to(torch.int32).reshape(-1, b, 1), n)


def _normalised(h, weight, bias):
    c = h - h.mean(1, keepdim=True)
    return c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * weight.float() + bias.float()


def _product8(qa, sa, s, dt):
    z = (qa @ s["qb"].float().t()) * sa[:, None] * s["sb"][None, :]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    c = _act(z, s["act"])
    if s["res"] is not None:
        c = c + s["res"].float()
    return c.to(dt)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "layernorm":
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        y = _normalised(h, s["weight"], s["bias"])
        out = {} if s["res"] is None else {"h": h.to(s["x"].dtype)}
        if s["to"] == "e4m3":
            out["scale"] = (y.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
            out["y"] = (y / out["scale"][:, None]).to(torch.float8_e4m3fn)
        else:
            out["y"] = y.to(DT[s["to"]])
        return out
    if s["op"] == "layernorm_grad":
        dt = s["dy"].dtype
        h, dy = (_kept(s["kept"], s["n"]) if s["kept8"] else s["h"].float()), s["dy"].float()
        c = h - h.mean(1, keepdim=True)
        r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        unit = c * r
        g = dy * s["weight"].float()
        dx = r * (g - g.mean(1, keepdim=True) - unit * (g * unit).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * unit).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}
    if s["op"] == "int8":
        return {"c": _product8(s["qa"].float(), s["sa"], s, DT[s["out"]])}
    if s["op"] == "project8":
        y = s["x"].float()
        if s["norm"]:
            y = _normalised(y, s["gain"], s["shift"])
        scale = (y.abs().amax(1) / INT8_MAX).clamp_min(SCALE_MIN)
        return {"c": _product8((y / scale[:, None]).round(), scale, s, s["x"].dtype)}
    if s["op"] == "checkpoint":
        z = _from_blocks(*_to_blocks(s["z"].float()), s["n"])
        dz = s["du"].float() * _act_grad(z, s["act"])
        dt = s["z"].dtype
        return {"u": _act(z, s["act"]).to(dt), "dz": dz.to(dt), "dbias": dz.sum(0)}
    dt = s["x"].dtype
    w = s["wkn"].float()
    z = s["x"].float() @ w + s["bias"].float()
    u = _act(z, s["act"]).to(dt)
    z = _from_blocks(*_to_blocks(z), s["n"])
    dz = s["du"].float() * _act_grad(z, s["act"])
    return {"u": u, "dx": (dz @ w.t()).to(dt), "dw": (s["x"].float().t() @ dz).to(dt), "dbias": dz.sum(0).to(dt)}


# ---- the framework's calls -------------------------------------------------------------------


def _run_own(s):
    import tile_scheduling_amd as ts

    if s["op"] == "layernorm":
        y, scale, h = ts.layernorm(s["x"], s["weight"], s["bias"], residual=s["res"], eps=EPS, out_dtype=DT[s["to"]])
        out = {"y": y}
        if scale is not None:
            out["scale"] = scale
        if s["res"] is not None:
            out["h"] = h
        return out
    if s["op"] == "layernorm_grad":
        h = ts.Checkpoint(s["kept"], s["n"]) if s["kept8"] else s["h"]
        dx, dw, db = ts.layernorm_backward(s["dy"], h, s["weight"], eps=EPS, dh=s["dh"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if s["op"] == "int8":
        c = ts.gemm_scaled(s["qa"], s["qb"].t(), s["sa"], s["sb"], bias=s["bias"], activation=s["act"],
                           residual=s["res"], out_dtype=DT[s["out"]])
        return {"c": c}
    if s["op"] == "project8":
        if s["norm"]:
            q, scale, _ = ts.layernorm(s["x"], s["gain"], s["shift"], eps=EPS, out_dtype=torch.int8)
        else:
            q, scale = ts.quantize_rows(s["x"], torch.int8)
        c = ts.gemm_scaled(q, s["qb"].t(), scale, s["sb"], bias=s["bias"], activation=s["act"], residual=s["res"],
                           out_dtype=s["x"].dtype)
        return {"c": c}
    if s["op"] == "checkpoint":
        kept = ts.checkpoint_pack(s["z"])
        u = torch.empty_like(s["z"])
        dz, db = ts.act_grad(s["du"], kept, s["act"], act_out=u)
        return {"u": u, "dz": dz, "dbias": db}
    kept = ts.Checkpoint.empty(s["m"], s["n"], s["x"].device)
    u = ts.gemm_epilogue(s["x"], s["wkn"], bias=s["bias"], activation=s["act"], preact=kept)
    dx, dw, db = ts.gemm_epilogue_backward(s["du"], s["x"], s["wkn"], preact=kept, activation=s["act"],
                                           dbias_dtype=s["x"].dtype)
    return {"u": u, "dx": dx, "dw": dw, "dbias": db}


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


def _kept64(z):
    """z rounded to 8 bits a value: steps of 2^e, e the least whole number for which the largest of
    32 neighbours in a row is at most 127 steps."""
    m, n = z.shape
    rows = torch.nn.functional.pad(z, (0, -n % 32)).unflatten(1, (-1, 32))
    most = rows.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.floor(torch.log2(most.clamp_min(2.0 ** -120))) - 6.0)
    step = torch.where(torch.round(most / step) > 127.0, 2.0 * step, step)
    return (torch.round(rows / step) * step).flatten(1)[:, :n]


def _norm64(h):
    """Rows less their mean over their deviation, and one over that deviation."""
    d = h - h.sum(1, keepdim=True) / h.shape[1]
    dev = torch.sqrt(d.square().sum(1, keepdim=True) / h.shape[1] + EPS)
    return d / dev, 1.0 / dev


def _finish64(z, s):
    if s["bias"] is not None:
        z = z + s["bias"].double()
    c = z * _gate(z, s["act"])[0]
    return c if s["res"] is None else c + s["res"].double()


def exact(case, seed):
    s = prepare(case, seed)
    n = case["n"]
    if case["op"] == "layernorm":
        h = s["x"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        y = _norm64(h)[0] * s["weight"].double() + s["bias"].double()
        out = {} if s["res"] is None else {"h": h}
        if case["to"] == "e4m3":
            scale = torch.maximum(y.abs().amax(1) / E4M3_MAX, torch.full_like(y[:, 0], SCALE_MIN))
            return {**out, "y": y / scale[:, None], "scale": scale}
        return {**out, "y": y}
    if case["op"] == "layernorm_grad":
        if case["kept8"]:
            b = _blocks(n)
            step = torch.exp2(s["kept"][:, 32 * b:33 * b].double() - 127.0)
            h = (s["kept"][:, :32 * b].view(torch.int8).double() * step.repeat_interleave(32, 1))[:, :n]
        else:
            h = s["h"].double()
        unit, r = _norm64(h)
        dy = s["dy"].double()
        g = s["weight"].double() * dy
        dx = r * (g - (g.sum(1, keepdim=True) + unit * (g * unit).sum(1, keepdim=True)) / n)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": (dy * unit).sum(0), "dbias": dy.sum(0)}
    if case["op"] == "int8":
        z = _product64(s["qa"], s["qb"].t()) * s["sa"].double()[:, None] * s["sb"].double()[None, :]
        return {"c": _finish64(z, s)}
    if case["op"] == "project8":
        y = s["x"].double()
        if case["norm"]:
            y = _norm64(y)[0] * s["gain"].double() + s["shift"].double()
        scale = torch.maximum(y.abs().amax(1) / INT8_MAX, torch.full_like(y[:, 0], SCALE_MIN))
        z = _product64(torch.round(y / scale[:, None]), s["qb"].t()) * scale[:, None] * s["sb"].double()[None, :]
        return {"c": _finish64(z, s)}
    if case["op"] == "checkpoint":
        z = _kept64(s["z"].double())
        g, dg = _gate(z, case["act"])
        dz = s["du"].double() * (g + z * dg)
        return {"u": z * g, "dz": dz, "dbias": dz.sum(0)}
    z = _product64(s["x"], s["wkn"]) + s["bias"].double()
    u = z * _gate(z, case["act"])[0]
    z = _kept64(z)
    g, dg = _gate(z, case["act"])
    dz = s["du"].double() * (g + z * dg)
    return {"u": u, "dx": _product64(dz, s["wkn"].t()), "dw": _product64(s["x"].t(), dz), "dbias": dz.sum(0)}
