"""Rows in 8 bits, from their definition, in 64 bits on the CPU."""
from __future__ import annotations

import torch


def steps(x):
    """Per block of 32 columns of x [M, N] (float64): the exponent byte and the step."""
    m, n = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -n % 32)).reshape(m, -1, 32)
    most = b.abs().amax(2)
    mant, ex = torch.frexp(torch.where(most.isfinite(), most, torch.zeros_like(most)))   # most = mant 2^ex, mant in [1/2, 1)
    e = torch.where(most > 0, ex - 7, torch.full_like(ex, -200))          # 64 to 128 steps
    e = torch.where(torch.round(torch.ldexp(most, -e)) > 127, e + 1, e).clamp_min(-126)
    byte = torch.where(most.isfinite(), e + 127, torch.full_like(e, 255))
    step = torch.where(most.isfinite(), torch.ldexp(torch.ones_like(most), e), torch.full_like(most, float("nan")))
    return b, byte.to(torch.uint8), step


def pack(x):
    """The bytes of each row of x: values, then exponents.  Blocks that stand for NaN: any values (0 here)."""
    b, byte, step = steps(x)
    q = torch.round(b / step[:, :, None]).nan_to_num(0.0, 0.0, 0.0).to(torch.int8)
    return torch.cat([q.reshape(x.shape[0], -1).view(torch.uint8), byte], dim=1)


def unpack(data, n):
    """The values (float64) of a Checkpoint's data."""
    data = data.cpu()
    b = -(-n // 32)
    e = data[:, 32 * b:33 * b].int()
    step = torch.where(e == 255, torch.tensor(float("nan"), dtype=torch.float64), torch.ldexp(torch.ones(()).double(), e - 127))
    q = data[:, :32 * b].contiguous().view(torch.int8).double().reshape(-1, b, 32)
    return (q * step[:, :, None]).reshape(data.shape[0], -1)[:, :n]


def check_bytes(kept, x, what=""):
    """Whether a Checkpoint holds x, bit for bit (the values of NaN blocks aside)."""
    want = pack(x)
    got = kept.data[:, :want.shape[1]].cpu()
    v = want.shape[1] // 33 * 32
    assert torch.equal(got[:, v:], want[:, v:]), what + ": exponents"
    bad = (want[:, v:] == 255).repeat_interleave(32, 1)
    assert torch.equal(got[:, :v].masked_fill(bad, 0), want[:, :v].masked_fill(bad, 0)), what + ": values"
