"""The product with a fused epilogue, its gradients and its 8-bit form on the GPU, against their
definitions in 64 bits (bounds derived in operator_reference)."""
import ctypes

import pytest
import torch

import tests.operator_reference as R
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tile_scheduling_amd as ts
else:
    ts = None

H, B, F, Q = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def operands(M, N, K, dtype, layout, seed, pad=0, offset=0):
    """A [M,K] and B [K,N] as views stored in `layout` ("nn", "nt", "tn", "tt"), with padding."""
    n = R.gen(seed)
    a, b = n(M, K).to(dtype), (n(K, N) / max(K, 1) ** 0.5).to(dtype)
    if layout[0] == "n":
        ad, _ = R.padded(a, "cuda", pad, offset)
    else:
        ad = R.padded(a.t().contiguous(), "cuda", pad, offset)[0].t()
    if layout[1] == "n":
        bd, _ = R.padded(b, "cuda", pad, offset)
    else:
        bd = R.padded(b.t().contiguous(), "cuda", pad, offset)[0].t()
    return a, b, ad, bd


SHAPES = [(1, 1, 1), (1, 64, 128), (3, 130, 72), (16, 100, 200), (17, 257, 64), (33, 64, 8), (128, 128, 64),
          (129, 131, 136), (130, 256, 1001), (257, 300, 65), (300, 96, 640), (64, 512, 0), (5, 1000, 1000)]


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_shapes_and_layouts(M, N, K, layout):
    for i, (dtype, out) in enumerate([(H, H), (B, F), (B, B), (H, F)]):
        name = R.ACTS[(M + N + i) % 5]
        n = R.gen(M * 7 + N + i)
        a, b, ad, bd = operands(M, N, K, dtype, layout, M + 3 * N + K + i)
        bias, res = n(N).to(dtype), n(M, N).to(out)
        pre = torch.empty(M, N, dtype=out, device="cuda")
        say(M, N, K, layout, dtype, out, name)
        c = ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=res.cuda(), preact=pre, out_dtype=out)
        z, zerr = R.product(a, b, bias)
        want, bound = R.forward(z, zerr, name, res, out)
        R.check(c, want, bound, "C")
        R.check(pre, z, zerr + R.rounded(z.abs() + zerr, out), "preact")


@pytest.mark.parametrize("layout", ["nn", "nt"])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 31), (16, 64), (70, 33), (257, 1000), (1000, 4200), (33000, 96), (40, 9000)])
def test_few_rows(N, K, layout):
    # one token to 32 rows: the one-pass kernels, and the tile kernels on the same call
    for i, M in enumerate((1, 2, 13, 16, 17, 32)):
        dtype, out = [(H, H), (B, F), (B, B), (H, F)][i % 4]
        name = R.ACTS[i % 5]
        n = R.gen(M + N + K)
        a, b, ad, bd = operands(M, N, K, dtype, layout, M * N + K, pad=i, offset=i)
        bias, res = n(N), n(M, N).to(out)
        rd, _ = R.padded(res, "cuda", 3, 1)
        pd, pbuf = R.padded(torch.zeros(M, N).to(out), "cuda", 2, 1, fill=7.0)
        cd, cbuf = R.padded(torch.zeros(M, N).to(out), "cuda", 5, 0, fill=7.0)
        say(M, N, K, layout, dtype, out, name)
        z, zerr = R.product(a, b, bias)
        want, bound = R.forward(z, zerr, name, res, out)
        for sched in (None, ts.Schedule(order="auto", mode="crosstile")):
            cd.zero_()
            pd.zero_()
            ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=rd, preact=pd, out=cd, schedule=sched)
            R.check(cd, want, bound, f"C {sched}")
            R.check(pd, z, zerr + R.rounded(z.abs() + zerr, out), f"preact {sched}")
        for buf, v in ((cbuf, cd), (pbuf, pd)):
            v.fill_(7.0)
            assert bool((buf == 7.0).all())
        zz = n(M, N).to(out)
        got = ts.gemm_dact(ad, bd, zz.cuda(), "gelu")
        p, perr = R.product(a, b)
        s = R.slope(zz.double(), "gelu")
        err = 1.2 * perr + R.ACT_ERR * (zz.double().abs() + 1) * p.abs()
        R.check(got, p * s, err + R.rounded((p * s).abs() + err, out), "dact")


@pytest.mark.parametrize("M", [1, 2, 7, 32, 33])
def test_outer_product(M):
    # K = 1: the one column of A is contiguous along M and along K
    for N in (1, 5, 70):
        n = R.gen(M + N)
        for dtype in (H, B):
            a, b = n(M, 1).to(dtype), n(1, N).to(dtype)
            for ad in (a.cuda(), a.t().contiguous().cuda().t()):
                for bd in (b.cuda(), b.t().contiguous().cuda().t()):
                    z, zerr = R.product(a, b)
                    want, bound = R.forward(z, zerr, "relu", None, F)
                    R.check(ts.gemm_epilogue(ad, bd, activation="relu", out_dtype=F), want, bound)


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("M,N,K", [(33, 64, 1024), (64, 129, 1031), (200, 7, 4100), (35, 1, 2048), (129, 260, 16384), (300, 516, 2051)])
def test_split_k(M, N, K, layout):
    # few tiles and a long K: the sums of parts of K joined by a second kernel; the same bits on
    # every run, nothing outside the views written, and a schedule's whole tiles agree
    for i, (dtype, out) in enumerate([(H, H), (B, F), (B, B)]):
        name = R.ACTS[(i + M) % 5]
        n = R.gen(M + N + K + i)
        a, b, ad, bd = operands(M, N, K, dtype, layout, M * N + K, pad=3 * i, offset=i)
        bias, res = n(N).to(dtype if i else F), n(M, N).to(out)
        rd, _ = R.padded(res, "cuda", 3, 1)
        pd, pbuf = R.padded(torch.zeros(M, N).to(out), "cuda", 2, 1, fill=7.0)
        cd, cbuf = R.padded(torch.zeros(M, N).to(out), "cuda", 5, 0, fill=7.0)
        say(M, N, K, layout, dtype, out, name)
        z, zerr = R.product(a, b, bias)
        want, bound = R.forward(z, zerr, name, res, out)
        first = None
        for sched in (None, None, ts.Schedule(order="auto", mode="crosstile")):
            cd.zero_()
            pd.zero_()
            ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=rd, preact=pd, out=cd, schedule=sched)
            R.check(cd, want, bound, f"C {sched}")
            R.check(pd, z, zerr + R.rounded(z.abs() + zerr, out), f"preact {sched}")
            first = cd.clone() if first is None else first
            assert sched is not None or torch.equal(first, cd)
        for buf, v in ((cbuf, cd), (pbuf, pd)):
            v.fill_(7.0)
            assert bool((buf == 7.0).all())
        cd.copy_(res)   # the residual in C's own memory
        ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=cd, out=cd)
        assert torch.equal(first, cd)
        zz = n(M, N).to(out)
        got = ts.gemm_dact(ad, bd, zz.cuda(), "silu")
        p, perr = R.product(a, b)
        sl = R.slope(zz.double(), "silu")
        err = 1.2 * perr + R.ACT_ERR * (zz.double().abs() + 1) * p.abs()
        R.check(got, p * sl, err + R.rounded((p * sl).abs() + err, out), "dact")


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (2, 2)])
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
def test_strides_and_alignment(layout, pad, offset):
    # rows with padding that holds NaN, odd starts; C, residual and preact with padding too
    for M, N, K in [(7, 66, 72), (140, 133, 200), (20, 35, 33)]:
        a, b, ad, bd = operands(M, N, K, B, layout, 5 + pad, pad, offset)
        n = R.gen(9)
        bias, res = n(N), n(M, N).to(B)
        rd, _ = R.padded(res, "cuda", pad, offset)
        cd, cbuf = R.padded(torch.zeros(M, N).to(B), "cuda", pad, offset, fill=7.0)
        pd, pbuf = R.padded(torch.zeros(M, N).to(B), "cuda", pad, offset, fill=7.0)
        say(layout, pad, offset, M, N, K)
        ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation="silu", residual=rd, preact=pd, out=cd)
        z, zerr = R.product(a, b, bias)
        want, bound = R.forward(z, zerr, "silu", res, B)
        R.check(cd, want, bound, "C")
        R.check(pd, z, zerr + R.rounded(z.abs() + zerr, B), "preact")
        for buf, v in ((cbuf, cd), (pbuf, pd)):   # nothing outside the view was written
            v.fill_(7.0)
            assert bool((buf == 7.0).all())


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("out", [B, F])
def test_gradient_epilogue(name, out):
    for M, N, K in [(5, 40, 64), (150, 260, 96), (257, 129, 33)]:
        a, b, ad, bd = operands(M, N, K, B, "nt", 11)
        z = (R.gen(3)(M, N) * 2).to(out)
        say(name, out, M, N, K)
        got = ts.gemm_dact(ad, bd, z.cuda(), name)
        p, perr = R.product(a, b)
        s = R.slope(z.double(), name)
        err = 1.2 * perr + R.ACT_ERR * (z.double().abs() + 1) * p.abs()
        R.check(got, p * s, err + R.rounded((p * s).abs() + err, out))


@pytest.mark.parametrize("tile", ["128x128x64", "256x256x64w8"])
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
def test_schedules_give_the_same_bits(tile, layout):
    M, N, K = 700, 1030, 456
    a, b, ad, bd = operands(M, N, K, H, layout, 21)
    res = R.gen(2)(M, N).to(H).cuda()
    kw = dict(bias=R.gen(4)(N).to(H).cuda(), activation="gelu", residual=res)
    ref = ts.gemm_epilogue(ad, bd, schedule=ts.Schedule(tile=tile), **kw)
    want, bound = R.forward(*R.product(a, b, kw["bias"]), "gelu", res, H)
    R.check(ref, want, bound)
    for mode, P in (("persistent", 3), ("crosstile", 5), ("auto", 0), ("persistent", 0)):
        for order, remap in (("grouped", True), ("auto", False)):
            s = ts.Schedule(order=order, group_m=2, mode=mode, num_programs=P, xcd_remap=remap, tile=tile)
            say(s.label())
            assert torch.equal(ref, ts.gemm_epilogue(ad, bd, schedule=s, **kw)), s.label()
    for P in (7, 13, 0):   # another order of summation along K: the bound, and the same bits twice
        s = ts.Schedule(order="grouped", group_m=4, mode="streamk", num_programs=P, tile=tile)
        say(s.label())
        x = ts.gemm_epilogue(ad, bd, schedule=s, **kw)
        R.check(x, want, bound, s.label())
        assert torch.equal(x, ts.gemm_epilogue(ad, bd, schedule=s, **kw))


def test_residual_in_place_and_two_outputs_of_one_product():
    M, N, K = 300, 520, 128
    a, b, ad, bd = operands(M, N, K, B, "nt", 31)
    res = R.gen(5)(M, N).to(B)
    c = res.cuda()
    out = ts.gemm_epilogue(ad, bd, residual=c, out=c)
    assert out.data_ptr() == c.data_ptr()
    assert torch.equal(c, ts.gemm_epilogue(ad, bd, residual=res.cuda()))


def test_infinities_and_nan():
    # a NaN or infinity in A reaches its own row only; act(-inf) as the formula says
    a, b, ad, bd = operands(40, 140, 96, B, "nt", 41)
    clean = ts.gemm_epilogue(ad, bd, activation="relu")
    ad[7, 3] = float("nan")
    ad[9, 5] = float("inf")
    c = ts.gemm_epilogue(ad, bd, activation="relu")
    assert bool(c[7].isnan().all())
    keep = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(c[keep], clean[keep])
    inf = (bd[5] > 0) & (bd[5] != 0)
    assert bool((c[9][inf] == float("inf")).all()) and bool((c[9][bd[5] < 0] == 0).all())


@pytest.mark.parametrize("dtype,layout", [(H, "nn"), (B, "nt")])
@pytest.mark.parametrize("M,N,K", [(1, 48, 32), (70, 200, 136), (333, 131, 77), (257, 512, 256)])
@pytest.mark.parametrize("name", ["none", "gelu", "silu"])
def test_backward(M, N, K, dtype, layout, name):
    a, b, ad, bd = operands(M, N, K, dtype, layout, 51)
    n = R.gen(6)
    dc, z = n(M, N).to(dtype), n(M, N).to(dtype)
    say(M, N, K, dtype, name)
    da, db, dbias = ts.gemm_epilogue_backward(dc.cuda(), ad, bd, preact=z.cuda(), activation=name)
    d64, s64 = dc.double(), R.slope(z.double(), name)
    dz = d64 * s64
    dzerr = R.ACT_ERR * (z.double().abs() + 1) * d64.abs() if name != "none" else torch.zeros_like(dz)
    R.check(dbias, dz.sum(0), dzerr.sum(0) + M * R.U * dz.abs().sum(0) + 1e-30, "dbias")
    zr = dzerr + R.rounded(dz.abs() + dzerr, dtype)    # dZ is an operand: rounded once
    for got, x, y, ex, ey, what in ((da, dz, b.double().t(), zr, None, "dA"), (db, a.double().t(), dz, None, zr, "dB")):
        want = x @ y
        err = (ex @ y.abs() if ex is not None else x.abs() @ ey) + (x.shape[1] + 4) * R.U * (x.abs() @ y.abs()) * 1.01
        R.check(got, want, err + R.rounded(want.abs() + err, dtype), what)
    assert da.dtype == dtype and db.dtype == dtype


def test_gradient_against_differences():
    # the 64-bit definition's central differences, through the whole chain, along random directions
    M, N, K = 24, 40, 32
    n = R.gen(61)
    a, b, bias, res, dc = n(M, K).to(H), (n(K, N) / 6).to(H), n(N), n(M, N).to(H), n(M, N).to(H)
    for name in R.ACTS[2:]:
        pre = torch.empty(M, N, dtype=F, device="cuda")
        ts.gemm_epilogue(a.cuda(), b.cuda(), bias=bias.cuda(), activation=name, residual=res.cuda().float(), preact=pre,
                         out_dtype=F)
        da, db, dbias = ts.gemm_epilogue_backward(dc.cuda().float(), a.cuda(), b.cuda(), preact=pre, activation=name)

        def loss(a, b, bias):
            return float((R.act(a @ b + bias, name) * dc.double()).sum())

        x = [a.double(), b.double(), bias.double()]
        for i, g in enumerate((da, db, dbias)):
            v = n(*x[i].shape).double()
            up, down = list(x), list(x)
            up[i], down[i] = x[i] + 1e-5 * v, x[i] - 1e-5 * v
            want = (loss(*up) - loss(*down)) / 2e-5
            # the gradients are rounded to fp16 (and dZ once more): 2 half steps of the sum's terms
            size = float((g.double().cpu().abs() * v.abs()).sum())
            assert abs(float((g.double().cpu() * v).sum()) - want) <= 3 * 2.0 ** -11 * size + 1e-6 * abs(want), (name, i)


@pytest.mark.parametrize("M,N", [(0, 8), (1, 1), (1, 300), (9, 7), (515, 1000), (64, 2051)])
def test_act_grad(M, N):
    for tin, tout, name in [(H, H, "gelu_tanh"), (B, B, "none"), (F, B, "silu"), (F, F, "relu"), (F, H, "gelu")]:
        n = R.gen(71)
        dc, z = n(M, N).to(tin), n(M, N).to(tin)
        say(M, N, tin, tout, name)
        dz, db = ts.act_grad(R.padded(dc, "cuda", 3, 1)[0] if M else dc.cuda(), z.cuda(), name, out_dtype=tout,
                             dbias_dtype=F)
        want = dc.double() * R.slope(z.double(), name)
        err = R.ACT_ERR * (z.double().abs() + 1) * dc.double().abs()
        R.check(dz, want, err + R.rounded(want.abs() + err, tout), "dz")
        R.check(db, want.sum(0), err.sum(0) + (M + 1) * R.U * want.abs().sum(0) + 1e-30, "dbias")
        assert torch.equal(db, ts.act_grad(dc.cuda(), z.cuda(), name, out_dtype=tout, dbias_dtype=F)[1])


def quantised(x):
    s = (x.abs().amax(1) / 448).clamp_min(2.0 ** -100)
    return (x / s[:, None]).to(Q), s


@pytest.mark.parametrize("out", [H, B, F])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 256), (4, 96, 48), (17, 130, 1000), (129, 257, 144),
                                   (300, 300, 33), (256, 512, 1024), (40, 64, 0), (16, 33000, 130), (32, 50, 9100),
                                   (2, 17, 0), (33, 200, 4200), (140, 130, 9001)])
def test_scaled(M, N, K, out):
    for name, pad in (("none", 0), ("silu", 16), ("gelu", 5)):
        n = R.gen(M + N + K)
        qa, sa = quantised(n(M, K)) if K else (n(M, K).to(Q), torch.ones(M))
        qb, sb = quantised(n(N, K)) if K else (n(N, K).to(Q), torch.ones(N))
        bias, res = n(N).to(out), n(M, N).to(out)
        pre = torch.empty(M, N, dtype=out, device="cuda")
        # the padding holds the largest value: any of it that is read shows
        ad, bd = (R.padded(q.float(), "cpu", pad, 0, fill=448.0)[0] for q in (qa, qb))
        ad, bd = (torch.empty_strided(v.shape, v.stride(), dtype=Q, device="cuda").copy_(v.to(Q)) for v in (ad, bd))
        say(M, N, K, out, name, pad)
        c = ts.gemm_scaled(ad, bd.t(), sa.cuda(), sb.cuda(), bias=bias.cuda(), activation=name, residual=res.cuda(),
                           preact=pre, out_dtype=out)
        z, zerr = R.product(qa.float(), qb.float().t(), bias, sa, sb, eight=out != F)
        want, bound = R.forward(z, zerr, name, res, out)
        R.check(c, want, bound, "C")
        R.check(pre, z, zerr + R.rounded(z.abs() + zerr, out), "preact")


def test_scaled_group_precision():
    # 2^16 + 2^t - 2^16 (the last by the bias): in one group of eight products exact while t is
    # at most 13 bits below 16; across groups, and with fp32 output (operands widened to
    # fp16), as far as fp32 holds the sum
    for k2, out, least in ((1, H, 3), (7, H, 3), (8, H, -7), (1, F, -7), (9, F, -7)):
        for t in range(least, 16):
            a, b = torch.zeros(1, 64), torch.zeros(1, 64)
            a[0, 0], b[0, 0] = 256.0, 256.0
            a[0, k2] = 2.0 ** max(min(t, 8), -9)
            b[0, k2] = 2.0 ** t / float(a[0, k2])
            c = ts.gemm_scaled(a.to(Q).cuda(), b.to(Q).cuda().t(), bias=torch.tensor([-65536.0]).cuda(), out_dtype=out)
            assert float(c[0, 0]) == 2.0 ** t, (k2, out, t)


def test_scaled_without_scales_is_exact_on_small_integers():
    n = R.gen(81)
    a, b = (n(200, 272) * 2).round().clamp(-4, 4), (n(140, 272) * 2).round().clamp(-4, 4)
    c = ts.gemm_scaled(a.to(Q).cuda(), b.to(Q).cuda().t(), out_dtype=F)
    assert torch.equal(c.cpu().double(), a.double() @ b.double().t())


def test_large_tile_and_ragged_large_product():
    # the 256 tile with edges in M, N and K, several tiles a program
    M, N, K = 1500, 3000, 520
    a, b, ad, bd = operands(M, N, K, B, "nt", 91)
    bias = R.gen(8)(N).to(B)
    sched = ts.Schedule(order="auto", mode="auto", tile="256x256x64w8", num_programs=16)
    c = ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation="gelu_tanh", out_dtype=F, schedule=sched)
    want, bound = R.forward(*R.product(a, b, bias), "gelu_tanh", None, F)
    R.check(c, want, bound)
    qa, sa = quantised(a.float())
    qb, sb = quantised(b.float().t().contiguous())
    c = ts.gemm_scaled(qa.cuda(), qb.cuda().t(), sa.cuda(), sb.cuda(), out_dtype=F, schedule=sched)
    z, zerr = R.product(qa.float(), qb.float().t(), None, sa, sb)
    R.check(c, z, zerr + R.rounded(z.abs() + zerr, F))


@pytest.mark.parametrize("pad,offset", [(60, 0), (3, 1)])
@pytest.mark.parametrize("dtype,out", [(B, B), (H, H), (B, F), (H, F)])
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
def test_every_epilogue_on_the_256_tile(layout, dtype, out, pad, offset):
    # tiles inside the matrix and on its edges, several a program; C, residual and preact with rows of
    # whole 128-byte lines (pad 60) and not; every activation with every use of a second matrix
    M, N, K = 600, 900, 200
    sched = ts.Schedule(order="auto", mode="auto", tile="256x256x64w8", num_programs=3)
    a, b, ad, bd = operands(M, N, K, dtype, layout, 77)
    n = R.gen(5)
    bias, res = n(N).to(dtype), n(M, N).to(out)
    z0, zerr0 = R.product(a, b)
    z1, zerr1 = R.product(a, b, bias)
    cd, cbuf = R.padded(res, "cuda", pad, offset, fill=7.0)
    pd, pbuf = R.padded(res, "cuda", pad, offset, fill=7.0)
    for name in R.ACTS:
        say(layout, dtype, out, pad, name)
        ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, out=cd, schedule=sched)
        want, bound = R.forward(z1, zerr1, name, None, out)
        R.check(cd, want, bound, f"{name}")
        pd.zero_()
        ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, preact=pd, out=cd, schedule=sched)
        R.check(cd, want, bound, f"{name} with preact")
        R.check(pd, z1, zerr1 + R.rounded(z1.abs() + zerr1, out), f"{name} preact")
        cd.copy_(res)   # in place
        ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=cd, out=cd, schedule=sched)
        want, bound = R.forward(z1, zerr1, name, res, out)
        R.check(cd, want, bound, f"{name} with residual")
        pd.zero_()
        rd = res.cuda()
        ts.gemm_epilogue(ad, bd, activation=name, residual=rd, preact=pd, out=cd, schedule=sched)
        want, bound = R.forward(z0, zerr0, name, res, out)
        R.check(cd, want, bound, f"{name} with both")
        R.check(pd, z0, zerr0 + R.rounded(z0.abs() + zerr0, out), f"{name} preact of both")
        pd.copy_(res)
        ts.gemm_dact(ad, bd, pd, name, out=pd, schedule=sched)   # in place
        sl = R.slope(res.double(), name)
        err = 1.2 * zerr0 + R.ACT_ERR * (res.double().abs() + 1) * z0.abs()
        R.check(pd, z0 * sl, err + R.rounded((z0 * sl).abs() + err, out), f"{name} gradient")
    for buf, v in ((cbuf, cd), (pbuf, pd)):   # nothing outside the views was written
        v.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_layer_forward_and_backward_together():
    # norm -> up projection with activation -> down projection with residual, and back
    M, D, E = 130, 192, 320
    n = R.gen(101)
    x, r0 = n(M, D).to(B), n(M, D).to(B)
    g, w1, b1 = (1 + 0.1 * n(D)).to(B), (n(E, D) / D ** 0.5).to(B), n(E).to(B)
    w2, b2, dy = (n(D, E) / E ** 0.5).to(B), n(D).to(B), n(M, D).to(B)
    cu = [t.cuda() for t in (x, r0, g, w1, b1, w2, b2, dy)]
    X, R0, G, W1, B1, W2, B2, DY = cu
    y, _, h = ts.rmsnorm(X, G, residual=R0)
    z = torch.empty(M, E, dtype=B, device="cuda")
    u = ts.gemm_epilogue(y, W1.t(), bias=B1, activation="gelu", preact=z)
    out = ts.gemm_epilogue(u, W2.t(), bias=B2, residual=h)
    du, dw2, db2 = ts.gemm_epilogue_backward(DY, u, W2.t())
    dyn, dw1, db1 = ts.gemm_epilogue_backward(du, y, W1.t(), preact=z, activation="gelu")
    dz = ts.gemm_dact(DY, W2, z, "gelu")   # the same dZ in one launch
    dx, dg = ts.rmsnorm_backward(dyn, h, G, dh=DY)

    P = [t.double().requires_grad_() for t in (x, r0, g, w1, b1, w2, b2)]
    hh = P[0] + P[1]
    yy = hh * torch.rsqrt((hh * hh).mean(1, keepdim=True) + 1e-6) * P[2]
    zz = yy @ P[3].t() + P[4]
    oo = R.act(zz, "gelu") @ P[5].t() + P[6] + hh
    grads = torch.autograd.grad(oo, P, dy.double())
    # bf16 intermediates: each of up to six roundings on a path is off by 2^-8 at most
    def near(got, want, what):
        got, want = got.double().cpu(), want.detach()
        assert float((got - want).norm() / want.norm()) <= 6 * 2.0 ** -8, what
    near(out, oo, "out")
    for got, i, what in ((dx, 0, "dx"), (dx, 1, "dresidual"), (dg, 2, "dgain"), (dw1.t(), 3, "dw1"), (db1, 4, "db1"),
                         (dw2.t(), 5, "dw2"), (db2, 6, "db2")):
        near(got, grads[i], what)
    near(dz, (dy.double() @ w2.double()) * R.slope(zz.detach(), "gelu"), "dz")
    # the 8-bit form of the same layer's forward pass: two e4m3 operands a product
    q, s, h8 = ts.rmsnorm(X, G, residual=R0, out_dtype=Q)
    qw1, sw1 = quantised(w1.float())
    u8 = ts.gemm_scaled(q, qw1.cuda().t(), s, sw1.cuda(), bias=B1, activation="gelu")
    assert torch.equal(h8, h)
    uu = R.act(zz.detach(), "gelu")
    assert float((u8.double().cpu() - uu).norm() / uu.norm()) <= 2 * 2.0 ** -4


def test_streams_and_captured_graph():
    # another stream than the default, and a graph replayed with eager work in between
    M, N, K = 200, 333, 77          # packed operands: the call's own workspace
    a, b, ad, bd = operands(M, N, K, B, "nt", 111)
    sk = ts.Schedule(mode="streamk", num_programs=5, tile="128x128x64")
    bias = R.gen(1)(N).to(B).cuda()
    ref = ts.gemm_epilogue(ad, bd, bias=bias, activation="silu")
    ref_sk = ts.gemm_epilogue(ad, bd, bias=bias, activation="silu", schedule=sk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ts.gemm_epilogue(ad, bd, bias=bias, activation="silu")
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = (ts.gemm_epilogue(ad, bd, bias=bias, activation="silu"),
                    ts.gemm_epilogue(ad, bd, bias=bias, activation="silu", schedule=sk),
                    *ts.gemm_epilogue_backward(ref, ad, bd, preact=ref, activation="silu"))
        graphs.append((gr, outs))
    eager = ts.gemm_epilogue_backward(ref, ad, bd, preact=ref, activation="silu")
    for i in range(3):
        for gr, outs in graphs:
            for o in outs:
                o.fill_(float("nan"))
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref_sk), i
            for x, y in zip(outs[2:], eager):
                assert torch.equal(x, y), i
        assert torch.equal(ts.gemm_epilogue(ad, bd, bias=bias, activation="silu"), ref)


def some(c, rows, cols):
    return c[rows][:, cols].double().cpu()


@pytest.mark.parametrize("which", ["output", "wide output", "few rows nt", "few rows nn", "scaled few rows", "operand", "split"])
def test_beyond_32_bits(which):
    # offsets past 2^32 bytes (and, of C, past 2^31 elements): some rows and columns, the last among them
    M, N, K, dtype, out = {"output": (66000, 33000, 24, B, B), "wide output": (33000, 33100, 40, H, F),
                           "few rows nt": (3, 270000, 8200, B, F), "few rows nn": (20, 270001, 8200, B, B),
                           "scaled few rows": (2, 530000, 8200, Q, B), "operand": (300, 600000, 4096, H, H),
                           "split": (40, 130, 17000000, B, F)}[which]
    if which == "split":
        K = (1 << 21) - 8   # the longest K of the direct loads' offsets
        M = 1100            # A: 4.6 GB
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def normal(r, c):
        t = torch.empty(r, c, dtype=dtype if dtype != Q else H, device="cuda").normal_(generator=g)
        return t.to(Q) if dtype == Q else t

    a = normal(M, K)
    bt = which in ("few rows nt", "scaled few rows", "operand", "split")
    b = normal(N, K).t() if bt else normal(K, N)
    say(which, M, N, K)
    rows = sorted({0, 1, M // 2, M - 2, M - 1} & set(range(M)))
    cols = sorted({0, 1, N // 2, N // 2 + 1, N - 2, N - 1})
    res = torch.empty(M, N, dtype=out, device="cuda").normal_(generator=g) if which.endswith("output") else None
    r = some(res, rows, cols) if res is not None else None
    if dtype == Q:
        c = ts.gemm_scaled(a, b, out_dtype=out, activation="relu")
    else:
        c = ts.gemm_epilogue(a, b, out_dtype=out, activation="relu", residual=res, out=res)
    ar, bc = a[rows].float(), b[:, cols].float()
    z, zerr = R.product(ar, bc, eight=dtype == Q)
    want, bound = R.forward(z, zerr, "relu", r, out)
    R.check(some(c, rows, cols), want, bound, which)
