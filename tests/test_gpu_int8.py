"""Products of int8 operands with a scale per token and channel, and rows rounded to 8 bits, on the GPU."""
import pytest
import torch

import tests.operator_reference as R
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tile_scheduling_amd as ts
else:
    ts = None

H, B, F, I, Q = torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def codes(seed, *shape, lo=-127):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randint(lo, 128, shape, generator=g, dtype=torch.int8)


def sums(a, b):
    return (a.double() @ b.double())   # whole numbers below 2^53: exact


def expect(a, b, sa, sb, bias):
    """z and its error: the sum's one rounding, two scalings and the bias."""
    z = sums(a, b) * sa.double()[:, None] * sb.double()[None, :]
    s = z.abs()
    if bias is not None:
        z = z + bias.double()
    return z, R.U * (4 * s + 2 * z.abs())


SHAPES = [(1, 1, 1), (1, 128, 256), (4, 96, 48), (17, 130, 1000), (32, 33, 144), (31, 9000, 80), (129, 257, 144), (200, 300, 77), (33, 64, 2048),
          (60, 140, 4099), (300, 520, 1000), (512, 512, 384), (64, 300, 77), (100, 33, 1000), (128, 130, 2048), (40, 4100, 4096),
          (65, 8192, 130), (48, 5, 3)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [H, B, F])
def test_product(M, N, K, out):
    n = R.gen(M + N + K)
    a, b = codes(M + K, M, K), codes(N + K + 1, N, K)
    sa, sb = 0.01 * (1 + n(M).abs()), (1 + n(N).abs()) / K
    bias, res = n(N).to(out), n(M, N).to(out)
    for name, bi, r in (("none", None, None), ("gelu", bias, None), ("silu", bias, res), ("relu", None, res), ("gelu_tanh", bias, res)):
        say(M, N, K, out, name)
        pre = torch.empty(M, N, dtype=out, device="cuda")
        c = ts.gemm_scaled(a.cuda(), b.cuda().t(), sa.cuda(), sb.cuda(), bias=None if bi is None else bi.cuda(), activation=name,
                           residual=None if r is None else r.cuda(), preact=pre, out_dtype=out)
        z, zerr = expect(a, b.t(), sa, sb, bi)
        R.check(pre, z, zerr + R.rounded(z.abs() + zerr, out), "preact")
        want, err = R.forward(z, zerr, name, r, out)
        R.check(c, want, err, "C")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sums_are_exact(M, N, K):
    a, b = codes(1, M, K, lo=-128), codes(2, N, K, lo=-128)
    say(M, N, K)
    want = sums(a, b.t()).float()   # one rounding, none below 2^24
    assert torch.equal(ts.gemm_scaled(a.cuda(), b.cuda().t(), out_dtype=F).cpu(), want)


@pytest.mark.parametrize("M,N", [(2, 16), (40, 16), (200, 16), (100, 16)])
def test_largest_sums(M, N):
    K = (1 << 17) - 1
    a, b = torch.full((M, K), -128, dtype=I), torch.full((N, K), -128, dtype=I)
    b[1] = 127
    b[2, ::2] = 127
    say(M, N)
    want = sums(a[:1], b.t()).float().expand(M, N)
    assert torch.equal(ts.gemm_scaled(a.cuda(), b.cuda().t(), out_dtype=F).cpu(), want)


@pytest.mark.parametrize("tile", ["128x128x64", "256x256x64w8"])
@pytest.mark.parametrize("out", [H, B, F])
def test_every_schedule_gives_the_same_bits(tile, out):
    M, N, K = 700, 900, 1160
    n = R.gen(9)
    a, b, sa, sb = codes(3, M, K).cuda(), codes(4, N, K).cuda(), n(M).abs().cuda(), (n(N).abs() / K).cuda()
    res, bias = n(M, N).to(out).cuda(), n(N).cuda()
    want = None
    for kw in (dict(order="row_major", mode="tiled"), dict(order="grouped", group_m=2, mode="persistent", num_programs=7),
               dict(order="auto", mode="crosstile"), dict(order="row_major", mode="streamk", num_programs=11),
               dict(order="grouped", group_m=3, mode="streamk", num_programs=5)):
        say(tile, out, kw)
        c = ts.gemm_scaled(a, b.t(), sa, sb, bias=bias, activation="gelu", residual=res, out_dtype=out,
                           schedule=ts.Schedule(tile=tile, **kw))
        want = c if want is None else want
        assert torch.equal(c, want)   # the sums are exact, whatever their order
    z, zerr = expect(a.cpu(), b.cpu().t(), sa.cpu(), sb.cpu(), bias.cpu())
    R.check(c, *R.forward(z, zerr, "gelu", res, out), "C")


@pytest.mark.parametrize("out", [H, B, F])
@pytest.mark.parametrize("K,pad", [(272, 0), (333, 0), (400, 7)])
def test_every_epilogue_on_the_256_tile(K, pad, out):
    # tiles inside and on both edges, several a program
    M, N = 600, 1100
    n = R.gen(K)
    a, b = codes(11, M, K), codes(12, N, K)
    sa, sb = 0.01 * (1 + n(M).abs()), (1 + n(N).abs()) / K
    res = n(M, N).to(out)
    sched = ts.Schedule(order="auto", mode="auto", num_programs=3, tile="256x256x64w8")
    for name in R.ACTS:
        for bias in (None, n(N), n(N).to(out)):
            z, zerr = expect(a, b.t(), sa, sb, bias)
            for r in (None, res):
                say(K, pad, out, name, bias is not None, r is not None)
                cd, cb = R.padded(torch.zeros(M, N).to(out), "cuda", pad, pad, fill=3.0)
                rd = None if r is None else R.padded(r, "cuda", pad, pad)[0]
                c = ts.gemm_scaled(a.cuda(), b.cuda().t(), sa.cuda(), sb.cuda(), bias=None if bias is None else bias.cuda(),
                                   activation=name, residual=rd, out=cd, schedule=sched)
                R.check(c, *R.forward(z, zerr, name, r, out), "C")
                if r is not None:   # in the residual's place
                    rd2 = R.padded(r, "cuda", pad, pad)[0]
                    ts.gemm_scaled(a.cuda(), b.cuda().t(), sa.cuda(), sb.cuda(), bias=None if bias is None else bias.cuda(),
                                   activation=name, residual=rd2, out=rd2, schedule=sched)
                    assert torch.equal(rd2, c)
                cd.fill_(3.0)
                assert bool((cb == 3.0).all())
        # one scale alone, and preact beside C
        for s1, s2 in ((sa, None), (None, sb)):
            pre = torch.empty(M, N, dtype=out, device="cuda")
            c = ts.gemm_scaled(a.cuda(), b.cuda().t(), None if s1 is None else s1.cuda(), None if s2 is None else s2.cuda(),
                               activation=name, preact=pre, out_dtype=out, schedule=sched)
            d = ts.gemm_scaled(a.cuda(), b.cuda().t(), None if s1 is None else s1.cuda(), None if s2 is None else s2.cuda(),
                               activation=name, out_dtype=out, schedule=sched)
            assert torch.equal(c, d)
            z, zerr = expect(a, b.t(), torch.ones(M) if s1 is None else s1, torch.ones(N) if s2 is None else s2, None)
            fits = z.abs() < 6e4   # (fp16: without a scale the sums are larger than its values)
            over = torch.where(fits, zerr + R.rounded(z.abs() + zerr, out), torch.full_like(z, float("inf")))
            R.check(torch.where(fits.cuda(), pre.double(), torch.zeros((), dtype=torch.float64, device="cuda")),
                    torch.where(fits, z, torch.zeros_like(z)), over, "preact")


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (4, 4), (16, 16), (5, 3)])
@pytest.mark.parametrize("M,N,K", [(3, 40, 96), (60, 70, 200), (90, 5000, 130), (300, 140, 1000), (140, 300, 1004), (260, 8200, 196)])
def test_strides_and_guards(M, N, K, pad, offset):
    a, b = codes(5, M, K), codes(6, N, K)

    def inside(t):
        m, k = t.shape
        buf = torch.full((offset + m * (k + pad) + 16,), 77, dtype=I, device="cuda")
        v = buf[offset:offset + m * (k + pad)].view(m, k + pad)[:, :k]
        v.copy_(t)
        return v

    cd, cb = R.padded(torch.zeros(M, N), "cuda", pad, offset, fill=3.0)
    say(M, N, K, pad, offset)
    c = ts.gemm_scaled(inside(a), inside(b).t(), out=cd)
    assert torch.equal(c.cpu(), sums(a, b.t()).float())
    cd.fill_(3.0)
    assert bool((cb == 3.0).all())


def test_no_products_and_scales_that_are_not_finite():
    a, b = torch.zeros(40, 0, dtype=I, device="cuda"), torch.zeros(24, 0, dtype=I, device="cuda")
    bias = torch.arange(24.0, device="cuda")
    for m in (40, 5):
        assert torch.equal(ts.gemm_scaled(a[:m], b.t(), bias=bias, out_dtype=F), bias.expand(m, 24))
    for m in (3, 50):
        a, b = codes(7, m, 64).cuda(), codes(8, 20, 64).cuda()
        sa = torch.ones(m, device="cuda")
        sa[0], sa[1] = float("nan"), float("inf")
        c = ts.gemm_scaled(a, b.t(), sa, out_dtype=F)
        assert bool(c[0].isnan().all()) and not bool(c[1].isfinite().any()) and bool(c[2:].isfinite().all())


@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (5, 64), (300, 100), (700, 520), (1, 4096), (300, 2051), (6, 8192), (2, 16384),
                                 (3, 30000), (2, 65536), (2, 65537)])
@pytest.mark.parametrize("dtype", [H, B, F])
@pytest.mark.parametrize("to", [I, Q])
def test_quantize_rows(M, N, dtype, to):
    x = (R.gen(M * N)(M, N) * torch.exp2(4 * R.gen(M)(M, 1))).to(dtype)
    say(M, N, dtype, to)
    q, s = ts.quantize_rows(x.cuda(), to)
    top = 127.0 if to == I else 448.0
    # an exact maximum and one correctly rounded quotient
    scale = (x.float().abs().amax(1) / top).clamp_min(2.0 ** -100)
    assert torch.equal(s.cpu(), scale)
    fine = scale.isfinite()   # (a row of the fp16 matrices may hold an infinity; test_quantize_special_rows has those)
    assert bool(x[~fine].isinf().any(1).all())
    quotient = (x.double() / scale.double()[:, None])[fine]
    got = q.double().cpu()[fine]
    if to == I:
        # the quotient's fp32 rounding, at most 127 * 2^-24, and half a step
        assert bool(((got - quotient).abs() <= 0.5 + 127 * 2.0 ** -24).all())
        assert bool((got.abs().amax(1) == 127).all())
    else:
        R.check(got, quotient, 2.0 ** -4 * quotient.abs() * (1 + 2.0 ** -20) + 2.0 ** -10, "e4m3")


def test_quantize_special_rows():
    for N in (5, 200, 3000, 70000):
        x = R.gen(N)(5, N)
        x[0] = 0.0
        x[1, 2] = float("nan")
        x[2, 3] = float("inf")
        x[3] *= 1e-38
        x[4] = float("-inf")
        w = torch.ones(16, N, dtype=I, device="cuda")
        q, s = ts.quantize_rows(x.cuda())
        assert float(s[0]) == 2.0 ** -100 and bool((q[0] == 0).all()) and bool(s[1].isnan()) and bool(s[2].isinf())
        c = ts.gemm_scaled(q, w.t(), s, out_dtype=F)
        assert bool((c[0] == 0).all()) and bool(c[1].isnan().all()) and not bool(c[2].isfinite().any())
        assert bool((c[3] == 0).all()) and not bool(c[4].isfinite().any())
    q, s = ts.quantize_rows(torch.empty(3, 0, device="cuda"))
    assert q.shape == (3, 0) and bool((s == 2.0 ** -100).all())
    assert ts.quantize_rows(torch.empty(0, 8, device="cuda"))[0].shape == (0, 8)


@pytest.mark.parametrize("N", [1, 100, 520, 4096, 20000, 70000])
@pytest.mark.parametrize("dtype", [B, F])
def test_rmsnorm_to_int8(N, dtype):
    n = R.gen(N)
    x, r, w = n(7, N).to(dtype), n(7, N).to(dtype), (1 + 0.2 * n(N)).to(dtype)
    q, s, h = ts.rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), out_dtype=I)
    y, _, h0 = ts.rmsnorm(x.float().cuda(), w.float().cuda(), residual=r.float().cuda())   # the same sums, unrounded
    assert torch.equal(h, h0.to(dtype))
    y = y.cpu()
    scale = (y.abs().amax(1) / 127).clamp_min(2.0 ** -100)   # (a tensor on the GPU is multiplied by 1 / 127 instead)
    assert torch.equal(s.cpu(), scale)
    got, quotient = q.double().cpu(), y.double() / scale.double()[:, None]
    assert bool(((got - quotient).abs() <= 0.5 + 127 * 2.0 ** -24).all())


def test_block_in_8_bits_captured_and_on_two_streams():
    # norm, up projection, rows rounded, down projection onto the residual stream
    n = R.gen(41)
    M, D, E = 70, 264, 520
    x, r, g = n(M, D).to(B).cuda(), n(M, D).to(B).cuda(), torch.ones(D, dtype=B, device="cuda")
    w1, s1 = ts.quantize_rows((n(E, D) / D ** 0.5).to(B).cuda())
    w2, s2 = ts.quantize_rows((n(D, E) / E ** 0.5).to(B).cuda())

    def block():
        q, s, h = ts.layernorm(x, g, residual=r, out_dtype=I)
        u = ts.gemm_scaled(q, w1.t(), s, s1, activation="gelu", out_dtype=B)
        q2, t = ts.quantize_rows(u)
        return ts.gemm_scaled(q2, w2.t(), t, s2, residual=h, out_dtype=B), h

    want, h = block()
    # against the same block in 64 bits: two roundings to 127 steps, each of the size of a value's
    # share of its row's largest (below 4.5 deviations here): 4.5 / 127 / sqrt(12) = 1.0 % of a deviation
    # each for the rows and the weights, four in all, and bf16's; under 4 % of the block's deviation
    h64 = (x.double() + r.double()).cpu()
    y = (h64 - h64.mean(1, keepdim=True)) / torch.sqrt(h64.var(1, keepdim=True, unbiased=False) + 1e-5)
    n = R.gen(41)
    n(M, D), n(M, D)
    u = R.act(y @ (n(E, D) / D ** 0.5).to(B).double().t(), "gelu")
    c = u @ (n(D, E) / E ** 0.5).to(B).double().t()
    off = (want.double().cpu() - h.double().cpu()) - c
    assert float(off.norm() / c.norm()) < 0.04
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other, _ = block()
    side.synchronize()
    assert torch.equal(other, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        again, _ = block()
    for _ in range(3):
        again.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, want)
        block()


@pytest.mark.parametrize("N,K", [(300, 2048), (530, 2051), (1100, 4096), (1100, 4001)])
@pytest.mark.parametrize("out", [H, B, F])
def test_every_row_count_gives_the_same_bits(N, K, out):
    # a row's result does not depend on the rows beside it: one pass over B (up to 32, 64 or 128 rows), K split among
    # programs (from there on) and both tiles round every term alike
    M = 600
    n = R.gen(N + K)
    a, b, sa, sb = codes(21, M, K).cuda(), codes(22, N, K).cuda(), (0.01 * (1 + n(M).abs())).cuda(), ((1 + n(N).abs()) / K).cuda()
    bias, res = n(N).cuda(), n(M, N).to(out).cuda()
    tile = lambda t: ts.Schedule(order="auto", mode="auto", tile=t)
    for name, bi, r, s1, s2 in (("none", None, None, sa, sb), ("none", bias, None, sa, None), ("none", bias, res, None, sb),
                                ("relu", bias, res, sa, sb), ("gelu", bias, None, sa, sb), ("gelu", bias, res, sa, sb),
                                ("silu", bias, res, sa, sb), ("gelu_tanh", bias, res, sa, sb)):
        def product(rows, schedule=None, pre=None):
            return ts.gemm_scaled(a[:rows], b.t(), None if s1 is None else s1[:rows], s2, bias=bi, activation=name,
                                  residual=None if r is None else r[:rows], preact=pre, out_dtype=out, schedule=schedule)

        pre = torch.empty(M, N, dtype=out, device="cuda")
        want = product(M, tile("128x128x64"))
        say(N, K, out, name, r is not None)
        assert torch.equal(product(M, tile("256x256x64w8")), want) and torch.equal(product(M, tile("128x128x64"), pre), want)
        for rows in (1, 5, 17, 33, 64, 65, 128, 129, 200, 300):
            p = torch.empty(rows, N, dtype=out, device="cuda")
            assert torch.equal(product(rows), want[:rows]), rows
            assert torch.equal(product(rows, None, p), want[:rows]) and torch.equal(p, pre[:rows]), rows
