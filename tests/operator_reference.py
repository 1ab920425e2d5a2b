"""The operators' definitions in 64 bits, and the error bounds of the kernels, for the tests.

A rounding to type t is off by at most HALF[t] relative to the value (half a step), plus
half of the smallest subnormal where the value is that small.  An fp32 sum of n terms is off
by at most n 2^-24 times the sum of their magnitudes, whatever its order.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24,
        torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149,
        torch.float8_e4m3fn: 2.0 ** -10}
U = 2.0 ** -24
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
# Evaluation of an activation or its slope in fp32, relative to |z| + 1: up to twelve
# roundings, two one-ulp transcendental instructions (2^-23 each) and the fitted tail
# (3.9e-7); the exponent's argument is rounded relative to its size, up to 2^7 before the
# exponential vanishes below what |z| + 1 sees.  Together less than 2e-6.
ACT_ERR = 2e-6
# Largest slope of the activations (gelu: 1.1290, gelu_tanh: 1.1290, silu: 1.0998), and
# of their slopes (gelu: 0.80, gelu_tanh: 0.80, silu: 0.5).
LIP, LIP_SLOPE = 1.13, 0.81


def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def act(z, name):
    if name == "relu":
        return z * (z > 0)
    if name == "gelu":
        return z * phi(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def rounded(x, dtype):
    """|error| of one rounding of x (64 bits) to dtype."""
    return HALF[dtype] * x.abs() + TINY[dtype]


def product(a, b, bias=None, scale_a=None, scale_b=None, eight=False):
    """z and its fp32 error bound, from 64-bit values of a and b.

    eight: the 8-bit matrix instruction (16-bit outputs of e4m3 operands).  It shifts the
    eight products of k = 8 i .. 8 i + 7 to the exponent of the largest and drops what lies
    below its 13th fraction bit: each of the eight loses less than 2^-13 of a power of two
    that is no larger than the largest product, so a group loses less than 2^-10 of its
    largest product.  (That 13 bits are kept is itself tested: test_scaled_group_precision.)
    """
    a, b = a.double().cpu(), b.double().cpu()
    z, s = a @ b, a.abs() @ b.abs()
    lost = 0.0
    if eight:
        for i in range(0, a.shape[1], 8):
            p = a[:, i:i + 8, None].abs() * b[None, i:i + 8].abs()
            lost = lost + 2.0 ** -10 * p.amax(1)
    if scale_a is not None:
        f = scale_a.double().cpu()[:, None] * scale_b.double().cpu()[None, :]
        z, s, lost = z * f, s * f, lost * f
    n = a.shape[1] + 4
    if bias is not None:
        z = z + bias.double().cpu()
        s = s + bias.double().cpu().abs()
    return z, n * U * s + lost


def forward(z, zerr, name, residual, dtype):
    """C and its error bound."""
    c = act(z, name)
    err = LIP * zerr + (ACT_ERR * (z.abs() + 1) if name not in ("none", "relu") else 0.0)
    if residual is not None:
        r = residual.double().cpu()
        c = c + r
        err = err + U * (c.abs() + err)
    return c, err + rounded(c.abs() + err, dtype)


def check(got, want, bound, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: "
                             f"{float(got[tuple(i)])!r} against {float(want[tuple(i)])!r}, "
                             f"bound {float(bound[tuple(i)] if torch.is_tensor(bound) else bound)!r}")


def gen(seed, device="cpu"):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    return normal


def padded(t, device, pad=0, offset=0, fill=float("nan")):
    """A view of t's values on `device` whose rows are `pad` elements longer in memory and which
    starts `offset` elements into its buffer; what lies around holds `fill`."""
    m, n = t.shape
    buf = torch.full((offset + m * (n + pad) + 16,), fill, dtype=torch.float32).to(t.dtype).to(device)
    v = buf[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    v.copy_(t)
    return v, buf
