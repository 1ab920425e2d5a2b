"""Rows in 8 bits on the GPU: packing bit for bit, the product that keeps its value before the activation,
and what the backward pass makes of them."""
import pytest
import torch

import tests.checkpoint_reference as K8
import tests.operator_reference as R
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import tile_scheduling_amd as ts
else:
    ts = None

H, B, F = torch.float16, torch.bfloat16, torch.float32
SHAPES = [(1, 1), (3, 7), (5, 31), (4, 32), (2, 33), (700, 64), (17, 100), (1, 4096), (300, 2051), (33, 16384), (2, 70001)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", [H, B, F])
def test_pack_and_unpack(M, N, dtype):
    n = R.gen(M + N)
    x = (n(M, N) * torch.exp2(8 * n(M, 1))).to(dtype)
    say(M, N, dtype)
    k = ts.checkpoint_pack(x.cuda())
    K8.check_bytes(k, x.double())
    want = K8.unpack(k.data, N)
    same = lambda t: torch.equal(t.isnan(), want.isnan()) and torch.equal(t.nan_to_num(0.0), want.nan_to_num(0.0))
    assert same(ts.checkpoint_unpack(k).cpu().double())
    assert same(ts.checkpoint_unpack(k, out_dtype=B).cpu().double())   # 8 significant bits
    step = K8.steps(x)[2].repeat_interleave(32, 1)[:, :N]
    assert torch.equal(step.isnan(), want.isnan())   # (blocks of the fp16 matrices may hold infinities)
    assert bool(((want - x.double()).abs() <= 0.5 * step)[~step.isnan()].all())


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("out", [H, B, F])
def test_unpack_with_activation(name, out):
    x = 3 * R.gen(5)(37, 200)
    k = ts.checkpoint_pack(x.cuda())
    z = K8.unpack(k.data, 200)
    c, err = R.forward(z, torch.zeros_like(z), name, None, out)
    R.check(ts.checkpoint_unpack(k, name, out_dtype=out), c, err, name)


def test_pack_borders():
    rows = []
    for e in (-130, -126, -7, 0, 6, 7, 120, 127):
        for m in (1.0, 127 / 64, 127.5 / 64 * (1 - 2 ** -24), 127.5 / 64, 127.5 / 64 * (1 + 2 ** -23), 2 - 2 ** -23):
            row = torch.zeros(64, dtype=torch.float64)
            row[:32] = torch.linspace(-1, 1, 32, dtype=torch.float64) * m * 2.0 ** min(e, 127)
            row[40] = -m * 2.0 ** e
            row[41] = 0.5 * 2.0 ** (e - 6)     # half a step: to even
            row[42] = 1.5 * 2.0 ** (e - 6)
            rows.append(row)
    x = torch.stack(rows).float()
    x = torch.cat([x, torch.zeros(2, 64), torch.full((1, 64), 2.0 ** -149), torch.full((1, 64), -(2.0 ** -127)),
                   torch.full((1, 64), 1.5 * 2.0 ** -127)])
    x = x[x.isfinite().all(1)]
    K8.check_bytes(ts.checkpoint_pack(x.cuda()), x.double())


def test_infinities_and_nan_stay_in_their_block():
    x = R.gen(3)(6, 100)
    x[0, 5] = float("inf")
    x[1, 40] = float("-inf")
    x[2, 99] = float("nan")
    x[3, :] = float("nan")
    k = ts.checkpoint_pack(x.cuda())
    K8.check_bytes(k, x.double())
    v = ts.checkpoint_unpack(k).cpu()
    bad = torch.nn.functional.pad(~x.isfinite(), (0, 28)).reshape(6, 4, 32).any(2).repeat_interleave(32, 1)[:, :100]
    assert torch.equal(v.isnan(), bad)


@pytest.mark.parametrize("pad,offset", [(1, 1), (3, 0), (8, 8)])
def test_strides_and_guards(pad, offset):
    for M, N in [(9, 65), (4, 1027)]:
        x = R.gen(N)(M, N).to(B)
        xd, _ = R.padded(x, "cuda", pad, offset)
        nb = -(-N // 32)
        buf = torch.full((M + 2, (33 * nb + 15) // 16 * 16 + 16 * pad), 201, dtype=torch.uint8, device="cuda")
        k = ts.checkpoint_pack(xd, ts.Checkpoint(buf[1:-1], N))
        K8.check_bytes(k, x.double())
        assert bool((buf[:, 33 * nb:] == 201).all()) and bool((buf[0] == 201).all()) and bool((buf[-1] == 201).all())
        yd, yb = R.padded(torch.zeros(M, N), "cuda", pad, offset, fill=3.0)
        ts.checkpoint_unpack(k, out=yd)
        assert torch.equal(yd.cpu().double(), K8.unpack(k.data, N))
        yd.fill_(3.0)
        assert bool((yb == 3.0).all())
        # a slice of rows is a checkpoint of those rows
        assert torch.equal(ts.checkpoint_unpack(ts.Checkpoint(k.data[2:4], N)).cpu().double(), K8.unpack(k.data, N)[2:4])


@pytest.mark.parametrize("M,N", [(0, 8), (1, 1), (1, 300), (9, 7), (515, 1000), (64, 2051)])
@pytest.mark.parametrize("name", R.ACTS)
def test_act_grad_from_checkpoint(M, N, name):
    n = R.gen(M + N)
    z, dc = n(M, N), n(M, N)
    say(M, N, name)
    k = ts.checkpoint_pack(z.cuda())
    z8 = ts.checkpoint_unpack(k)
    # the same arithmetic on the same values: the same bits
    u = torch.empty(M, N, device="cuda")
    dz, db = ts.act_grad(dc.cuda(), k, name, out=torch.empty(M, N, device="cuda"), act_out=u)
    dz0, db0 = ts.act_grad(dc.cuda(), z8, name, out=torch.empty(M, N, device="cuda"))
    assert torch.equal(dz, dz0) and torch.equal(db, db0)
    assert torch.equal(u, ts.checkpoint_unpack(k, name))
    for dtype in (H, B):
        dcd = dc.to(dtype).cuda()
        u = torch.empty(M, N, dtype=dtype, device="cuda")
        dz, db = ts.act_grad(dcd, k, name, act_out=u, dbias_dtype=dtype)
        zz = z8.cpu().double()
        want = dc.to(dtype).double() * R.slope(zz, name)
        err = (R.ACT_ERR * (zz.abs() + 1) if name not in ("none", "relu") else 0.0) * dc.to(dtype).double().abs() + R.U * want.abs()
        R.check(dz, want, err + R.rounded(want.abs() + err, dtype), "dz")
        c, cerr = R.forward(zz, torch.zeros_like(zz), name, None, dtype)
        R.check(u, c, cerr, "u")
        bound = (err + (M + 2) * R.U * want.abs()).sum(0)
        R.check(db, want.sum(0), bound + R.rounded(want.sum(0).abs() + bound, dtype), "dbias")


def test_act_grad_with_a_16_bit_preact_gives_the_value_too():
    n = R.gen(11)
    z, dc = n(100, 300).to(B), n(100, 300).to(B)
    zd, u = z.cuda(), torch.empty(100, 300, dtype=B, device="cuda")
    dz, db = ts.act_grad(dc.cuda(), zd, "gelu", act_out=u)
    dz0, db0 = ts.act_grad(dc.cuda(), zd, "gelu")
    assert torch.equal(dz, dz0) and torch.equal(db, db0)
    c, err = R.forward(z.double(), torch.zeros(100, 300).double(), "gelu", None, B)
    R.check(u, c, err, "u")
    # each output in an input's place: dZ on dC, the value on preact
    dcd = dc.cuda()
    d2, _ = ts.act_grad(dcd, zd, "gelu", out=dcd, act_out=zd)
    assert torch.equal(dcd, dz0) and torch.equal(zd, u)
    # only the value and the bias gradient of a plain layer
    dcd = dc.cuda()
    same, db = ts.act_grad(dcd, z.cuda(), "none", act_out=u)
    assert same is dcd and torch.equal(u.cpu(), z)


def stored(t, transposed):
    return t.t().contiguous().cuda().t() if transposed else t.cuda()


def limit(name):
    return 1.0 if name in ("none", "relu") else R.LIP


PRODUCTS = [(1, 1, 1, None), (3, 40, 96, None), (17, 70, 200, None), (32, 300, 72, None), (60, 70, 2048, None),
            (200, 140, 96, None), (300, 33, 1000, None), (129, 260, 264, "128x128x64"), (300, 516, 520, "256x256x64w8"),
            (512, 512, 256, "256x256x64w8"), (600, 1100, 272, "256x256x64w8")]


@pytest.mark.parametrize("M,N,K,tile", PRODUCTS)
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("dtype,out", [(H, H), (B, B), (B, F), (H, F)])
def test_product_keeps_its_preact(M, N, K, tile, layout, dtype, out):
    n = R.gen(M + N + K)
    a, b, bias, res = n(M, K).to(dtype), (n(K, N) / K ** 0.5).to(dtype), n(N).to(dtype), n(M, N).to(out)
    ad, bd = stored(a, layout[0] == "t"), stored(b, layout[1] == "t")
    sched = ts.Schedule(order="auto", mode="auto", tile=tile) if tile else None
    z, zerr = R.product(a, b, bias)
    for name, r in (("gelu", None), ("silu", res), ("relu", None), ("none", res)):
        say(M, N, K, tile, layout, dtype, out, name)
        k = ts.Checkpoint.empty(M, N)
        k.data.fill_(201)
        c = ts.gemm_epilogue(ad, bd, bias=bias.cuda(), activation=name, residual=None if r is None else r.cuda(),
                             preact=k, out_dtype=out, schedule=sched)
        c64, cerr = R.forward(z, zerr, name, r, out)
        R.check(c, c64, cerr, "C")
        nb = -(-N // 32)
        assert bool((k.data[:, 33 * nb:] == 201).all())
        v = K8.unpack(k.data, N)
        # the step: the least for the largest value of a block, which is off by zerr at most
        pad = lambda t: torch.nn.functional.pad(t, (0, -N % 32)).reshape(M, -1, 32).amax(2)
        most, off = pad(z.abs()), pad(zerr)
        step = torch.ldexp(torch.ones(M, nb).double(), k.data[:, 32 * nb:33 * nb].cpu().int() - 127)
        assert bool((127.5 * step > most - off).all()) and bool((127.5 * step / 2 <= most + off).all())
        wide = step.repeat_interleave(32, 1)[:, :N]
        R.check(v, z, 0.5 * wide + zerr, "kept")
        assert bool((k.data[:, N:32 * nb].cpu() == 0).all())   # columns behind N


@pytest.mark.parametrize("M,N,K,tile", PRODUCTS)
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("dtype", [H, B])
def test_product_keeps_what_it_would_have_written(M, N, K, tile, layout, dtype):
    # the value before the activation in fp32, packed, is what the product keeps by itself: the same sums
    n = R.gen(M + N + 3 * K)
    a, b, bias = n(M, K).to(dtype), (n(K, N) / K ** 0.5).to(dtype), n(N).to(dtype).cuda()
    ad, bd = stored(a, layout[0] == "t"), stored(b, layout[1] == "t")
    sched = ts.Schedule(order="auto", mode="auto", tile=tile) if tile else None
    say(M, N, K, tile, layout, dtype)
    z = torch.empty(M, N, device="cuda")
    c = ts.gemm_epilogue(ad, bd, bias=bias, activation="gelu", preact=z, out_dtype=F, schedule=sched)
    k = ts.Checkpoint.empty(M, N)
    c8 = ts.gemm_epilogue(ad, bd, bias=bias, activation="gelu", preact=k, out_dtype=F, schedule=sched)
    assert torch.equal(c, c8)
    K8.check_bytes(k, z.cpu().double())


@pytest.mark.parametrize("M,N,K,tile", PRODUCTS)
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("layout,dtype", [("nn", H), ("nt", B), ("tn", B), ("tt", H)])
def test_gradient_epilogue_from_checkpoint(M, N, K, tile, name, layout, dtype):
    n = R.gen(M * 5 + N + K)
    a, b, z = n(M, K).to(dtype), (n(K, N) / K ** 0.5).to(dtype), n(M, N)
    ad, bd = stored(a, layout[0] == "t"), stored(b, layout[1] == "t")
    sched = ts.Schedule(order="auto", mode="auto", tile=tile) if tile else None
    k = ts.checkpoint_pack(z.cuda())
    say(M, N, K, tile, name, layout, dtype)
    for out in (dtype, F):
        z8 = ts.checkpoint_unpack(k, out_dtype=out)
        c = ts.gemm_dact(ad, bd, k, name, out=torch.empty(M, N, dtype=out, device="cuda"), schedule=sched)
        d, derr = R.product(a, b)
        s = R.slope(K8.unpack(k.data, N), name)
        err = limit(name) * derr + (R.ACT_ERR * (z8.cpu().double().abs() + 1) if name not in ("none", "relu") else 0.0) * (d.abs() + derr)
        want = d * s
        err = err + R.U * want.abs()
        R.check(c, want, err + R.rounded(want.abs() + err, out), "C")
    assert ts.gemm_dact(ad, bd, k, name).dtype == dtype


def test_backward_from_checkpoints():
    # a linear layer whose input and value before the activation are kept in 8 bits
    n = R.gen(21)
    M, N, K = 200, 136, 264
    a, b, dc = n(M, K).to(B), (n(K, N) / K ** 0.5).to(B), n(M, N).to(B)
    z = n(M, N)
    ka, kz = ts.checkpoint_pack(a.cuda()), ts.checkpoint_pack(z.cuda())
    da, db, dbias = ts.gemm_epilogue_backward(dc.cuda(), ka, b.cuda(), preact=kz, activation="gelu")
    a8, z8 = ts.checkpoint_unpack(ka, out_dtype=B), ts.checkpoint_unpack(kz, out_dtype=B)
    da0, db0, dbias0 = ts.gemm_epilogue_backward(dc.cuda(), a8, b.cuda(), preact=z8, activation="gelu")
    assert torch.equal(da, da0) and torch.equal(db, db0) and torch.equal(dbias, dbias0)
    dx, dw = ts.rmsnorm_backward(dc.cuda(), kz, torch.ones(N, dtype=B, device="cuda"))
    dx0, dw0 = ts.rmsnorm_backward(dc.cuda(), z8, torch.ones(N, dtype=B, device="cuda"))
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_refusals_of_the_library():
    a, b = torch.zeros(512, 512, dtype=B, device="cuda"), torch.zeros(512, 512, dtype=B, device="cuda")
    k = ts.Checkpoint.empty(512, 512)
    for call in (lambda: ts.gemm_epilogue(a, b, preact=k, schedule=ts.Schedule(mode="streamk", num_programs=7)),
                 lambda: ts.gemm_scaled(a.to(torch.int8), b.to(torch.int8).t(), preact=k),
                 lambda: ts.checkpoint_unpack(k, out_dtype=torch.int8)):
        with pytest.raises(ts.TsError) as e:
            call()
        assert e.value.status in (ts.TS_ERR_UNSUPPORTED, ts.TS_ERR_INVALID_ARG) and "TS_" in str(e.value)
    with pytest.raises(ValueError, match="same GPU"):
        ts.checkpoint_pack(a, ts.Checkpoint.empty(512, 512, "cpu"))


def test_captured_graph_and_streams():
    n = R.gen(31)
    M, N, K = 300, 520, 264
    a, b, dc = n(M, K).to(B).cuda(), (n(K, N) / K ** 0.5).to(B).cuda(), n(M, N).to(B).cuda()
    k0 = ts.Checkpoint.empty(M, N)
    u0 = ts.gemm_epilogue(a, b, activation="gelu", preact=k0)
    g0 = ts.gemm_epilogue_backward(dc, a, b, preact=k0, activation="gelu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        k1 = ts.Checkpoint.empty(M, N)
        u1 = ts.gemm_epilogue(a, b, activation="gelu", preact=k1)
        g1 = ts.gemm_epilogue_backward(dc, a, b, preact=k1, activation="gelu")
    side.synchronize()
    nb = -(-N // 32)
    assert torch.equal(u0, u1) and torch.equal(k0.data[:, :33 * nb], k1.data[:, :33 * nb])
    assert all(torch.equal(x, y) for x, y in zip(g0, g1))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        k2 = ts.Checkpoint.empty(M, N)
        u2 = ts.gemm_epilogue(a, b, activation="gelu", preact=k2)
        g2 = ts.gemm_epilogue_backward(dc, a, b, preact=k2, activation="gelu")
        p2 = ts.checkpoint_pack(u2)
        v2 = ts.checkpoint_unpack(p2, "silu", out_dtype=B)
    want = ts.checkpoint_unpack(ts.checkpoint_pack(u0), "silu", out_dtype=B)
    for i in range(3):
        for t in (u2, v2, *g2):
            t.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(u2, u0) and torch.equal(v2, want) and all(torch.equal(x, y) for x, y in zip(g0, g2))
        ts.checkpoint_pack(a)


def test_beyond_32_bits():
    # more than 2^32 bytes in x and 2^32 bytes of values: the last rows
    M, N = 300005, 16000
    x = torch.empty(M, N, dtype=B, device="cuda").normal_()
    k = ts.checkpoint_pack(x)
    rows = [0, 1, M // 2, M - 2, M - 1]
    K8.check_bytes(ts.Checkpoint(k.data[rows].contiguous(), N), x[rows].double().cpu())
    y = ts.checkpoint_unpack(k, out=x)
    assert torch.equal(y[rows].double().cpu(), K8.unpack(k.data[rows], N))
    dz, _ = ts.act_grad(y, k, "relu", out=y, dbias=False)
    assert torch.equal(dz[rows].double().cpu(), K8.unpack(k.data[rows], N).clamp_min(0.0))


@pytest.mark.parametrize("dtype", [H, B, F])
@pytest.mark.parametrize("name", R.ACTS)
def test_largest_values_of_a_type(dtype, name):
    # from 255/256 of a power of two on a block's largest value is kept as that power, which the type does not hold
    # where it is its last: the value that is read still lies within half a step
    top, n = torch.finfo(dtype).max, R.gen(77)
    low = top if dtype == B else 2.0 ** (16 if dtype == H else 128) * 255 / 256
    x = n(9, 100).double()
    x[0, 3], x[1, 40], x[2], x[3] = top, -top, top, -top
    x[4], x[5] = torch.linspace(-1, 1, 100) * top, torch.linspace(1, -1, 100) * low
    x[6, 99], x[7, 0], x[8, 64:] = low, -low, torch.linspace(low, top, 36)
    x = x.to(dtype)
    dc = n(9, 100).to(dtype)
    assert bool(x.isfinite().all())
    k = ts.checkpoint_pack(x.cuda())
    K8.check_bytes(k, x.double())
    half = 0.5 * K8.steps(x)[2].repeat_interleave(32, 1)[:, :100]
    say(dtype, name)
    for out in (dtype, F):
        v = ts.checkpoint_unpack(k, out_dtype=out).cpu().double()
        assert bool(((v - x.double()).abs() <= half + R.rounded(v, dtype) * (out == H)).all())
    z = ts.checkpoint_unpack(k, out_dtype=dtype).cpu().double()
    want, err = R.forward(z, torch.zeros_like(z), name, None, dtype)
    R.check(ts.checkpoint_unpack(k, name, out_dtype=dtype), want, err, "value")
    u = torch.empty(9, 100, dtype=dtype, device="cuda")
    dz, _ = ts.act_grad(dc.cuda(), k, name, act_out=u, dbias=False)
    R.check(u, want, err, "u")
    s = R.slope(z, name)
    # the slopes of these values are 0 or 1, but for the block's small ones
    serr = R.ACT_ERR * (z.abs().clamp_max(64.0) + 1) if name not in ("none", "relu") else 0.0
    bound = (serr + R.U * s.abs()) * dc.double().abs()
    R.check(dz, dc.double() * s, bound + R.rounded((dc.double() * s).abs() + bound, dtype), "dz")
    # the products that read a checkpoint: few rows, tiles (rows repeated), K split
    eye = torch.eye(9).to(B if dtype == F else dtype)
    for rows, K, tile in ((9, 9, None), (180, 9, "128x128x64"), (612, 9, "256x256x64w8"), (180, 4096, None)):
        a = torch.zeros(rows, K, dtype=eye.dtype)
        a[:, :9] = eye.repeat(rows // 9, 1)
        b = torch.zeros(K, 100, dtype=eye.dtype)
        b[:9] = dc.to(eye.dtype)[:, :100]
        sched = ts.Schedule(order="auto", mode="auto", tile=tile) if tile else None
        kk = ts.Checkpoint(k.data.repeat(rows // 9, 1), 100)
        c = ts.gemm_dact(a.cuda(), b.cuda(), kk, name, out=torch.empty(rows, 100, device="cuda"), schedule=sched)
        d = b[:9].double().repeat(rows // 9, 1)
        zz, ss = z.repeat(rows // 9, 1), s.repeat(rows // 9, 1)
        serr = R.ACT_ERR * (zz.abs().clamp_max(64.0) + 1) if name not in ("none", "relu") else 0.0
        R.check(c, d * ss, (serr + 2 * R.U * ss.abs()) * d.abs() + R.TINY[F], f"gradient {rows} {K}")


def test_gradients_from_the_largest_values_of_fp16():
    g = torch.Generator().manual_seed(5)
    M, N, K = 40, 96, 64
    x = 65280.0 + 32.0 * torch.randint(0, 8, (M, N), generator=g)
    x = (x * (1 - 2 * torch.randint(0, 2, (M, N), generator=g))).to(H)
    n = R.gen(6)
    dy, w, b = n(M, N).to(H), (1 + 0.2 * n(N)).to(H), (n(N, K) / N).to(H)
    k = ts.checkpoint_pack(x.cuda())
    x8 = ts.checkpoint_unpack(k, out_dtype=H)
    assert bool(((x8.cpu().double() - x.double()).abs() <= 512.0).all())
    dx, dw = ts.rmsnorm_backward(dy.cuda(), k, w.cuda())
    dx0, dw0 = ts.rmsnorm_backward(dy.cuda(), x8, w.cuda())
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all()) and torch.equal(dx, dx0) and torch.equal(dw, dw0)
    assert all(bool(t.isfinite().all()) for t in ts.layernorm_backward(dy.cuda(), k, w.cuda()))
    dc = (1e-4 * n(M, K)).to(H)
    da, db, _ = ts.gemm_epilogue_backward(dc.cuda(), k, b.cuda(), dbias=False)
    want = x8.cpu().double().t() @ dc.double()
    err = (M + 4) * R.U * (x8.cpu().double().abs().t() @ dc.double().abs())
    R.check(db, want, err + R.rounded(want.abs() + err, H), "dB")


@pytest.mark.parametrize("M,N,K,tile", PRODUCTS)
@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("dtype", [H, B])
def test_16_bit_products_keep_the_same_bytes(M, N, K, tile, layout, dtype):
    # the straight forms of 16-bit C for each activation keep what the general form of fp32 C keeps
    n = R.gen(M + 2 * N + K)
    a, b, bias = n(M, K).to(dtype), (n(K, N) / K ** 0.5).to(dtype), n(N).to(dtype).cuda()
    ad, bd = stored(a, layout[0] == "t"), stored(b, layout[1] == "t")
    sched = ts.Schedule(order="auto", mode="auto", tile=tile) if tile else None
    nb = -(-N // 32)
    for name in R.ACTS:
        say(M, N, K, tile, layout, dtype, name)
        k, k32 = ts.Checkpoint.empty(M, N), ts.Checkpoint.empty(M, N)
        ts.gemm_epilogue(ad, bd, bias=bias, activation=name, preact=k, schedule=sched)
        ts.gemm_epilogue(ad, bd, bias=bias, activation=name, preact=k32, out_dtype=F, schedule=sched)
        assert torch.equal(k.data[:, :33 * nb], k32.data[:, :33 * nb])
