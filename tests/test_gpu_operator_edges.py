"""The operators around the product on the GPU at the edges of what their contract allows: empty
matrices, values at the ends of the types' ranges, infinities, calls that overlap in time.  Against
definitions in 64 bits (bounds derived in operator_reference)."""
import threading

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


@pytest.mark.parametrize("M", [1, 5, 40, 700])
def test_gradients_of_no_columns(M):
    # dC is M x 0: dA = dC @ B^T is zero, dB and dbias have no elements
    for dtype, name in ((H, "none"), (B, "gelu"), (H, "silu")):
        dc, z = torch.empty(M, 0, dtype=dtype, device="cuda"), torch.empty(M, 0, dtype=dtype, device="cuda")
        dz, db = ts.act_grad(dc, z, name, dbias_dtype=F)
        assert dz.shape == (M, 0) and db.shape == (0,)
        a, b = torch.ones(M, 7, dtype=dtype, device="cuda"), torch.empty(7, 0, dtype=dtype, device="cuda")
        da, dw, db = ts.gemm_epilogue_backward(dc, a, b, preact=z, activation=name)
        assert torch.equal(da, torch.zeros(M, 7, dtype=dtype, device="cuda"))
        assert dw.shape == (7, 0) and db.shape == (0,)


@pytest.mark.parametrize("M", [1, 17, 5000])
def test_norm_of_no_columns(M):
    # rows without elements: nothing to norm, and the least scale (2^-100) for the e4m3 form
    filled = [torch.full((max(M, 128),), 5.0, device="cuda") for _ in range(4)]   # what is freed here may come back as the scale
    del filled
    for dtype in (H, B, F):
        x = torch.empty(M, 0, dtype=dtype, device="cuda")
        for res in (None, torch.empty(M, 0, dtype=dtype, device="cuda")):
            y, scale, h = ts.rmsnorm(x, torch.empty(0, dtype=dtype, device="cuda"), residual=res)
            assert y.shape == (M, 0) and scale is None and h.shape == (M, 0)
            q, scale, h = ts.rmsnorm(x, residual=res, out_dtype=Q)
            assert q.shape == (M, 0) and h.shape == (M, 0)
            assert torch.equal(scale, torch.full((M,), 2.0 ** -100, device="cuda"))


@pytest.mark.parametrize("M,N", [(3, 7), (5, 64), (40, 520), (6, 4096), (9, 16384), (5, 20000), (3, 32776)])
@pytest.mark.parametrize("dtype", [B, F])
def test_norm_backward_far_from_unit_scale(M, N, dtype):
    # rows of every magnitude that the forward pass takes: r^3 is outside fp32's range for most of them,
    # dx is not
    n = R.gen(M + 5 * N)
    at = torch.tensor([1e15, 1e-14, 1e12, 1e17, 1e-17, 1.0, 1e-6, 1e9, 3e16] * 5)[:M]
    h = (n(M, N) * at[:, None]).to(dtype)
    # dy aligned with h in part, so that the mean is no small difference
    unit = h.double() / at[:, None].double()
    dy, w = (n(M, N) + unit.float()).to(dtype), (1 + 0.2 * n(N)).to(dtype)
    say(M, N, dtype)
    for eps in (1e-36, 0.0):
        dx, dw = ts.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=eps)
        h64, dy64, w64 = h.double(), dy.double(), w.double()
        r = 1.0 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + eps)
        g, u = w64 * dy64, h64 * r
        mean = (g * u).mean(1, keepdim=True)
        want = r * (g - u * mean)
        # r: (N/2 + 8) U; the mean's sum N U of its terms' magnitudes and r twice; then a few products
        rerr = (N / 2 + 8) * R.U
        merr = (g * u).abs().mean(1, keepdim=True) * ((N + 8) * R.U + 2 * rerr)
        err = (r * g).abs() * (rerr + 4 * R.U) + (r * u).abs() * (merr + (rerr + 4 * R.U) * mean.abs()) + 2 * R.U * want.abs()
        R.check(dx, want, err + R.rounded(want.abs() + err, dtype) + 2.0 ** -126, f"dx eps {eps}")
        wd = (dy64 * u).sum(0)
        derr = (dy64 * u).abs().sum(0) * ((M + 4) * R.U + rerr)
        R.check(dw, wd, derr + R.rounded(wd.abs() + derr, dtype), "dweight")


def infinite(M, N, K, dtype):
    """Operands whose product is infinite, of either sign, in rows 1 and 2 and finite elsewhere."""
    n = R.gen(M + N + K)
    a, b = n(M, K).to(dtype), (n(K, N) / max(K, 1) ** 0.5).to(dtype)
    a[1, 0] = float("inf")
    a[min(2, M - 1), K - 1] = float("-inf")
    return a, b


@pytest.mark.parametrize("layout", ["nn", "nt"])
@pytest.mark.parametrize("M,N,K,tile", [(3, 40, 96, None), (32, 300, 72, None), (60, 70, 2048, None), (200, 140, 96, None),
                                        (600, 520, 128, "256x256x64w8")])
@pytest.mark.parametrize("name", R.ACTS)
def test_infinite_products(M, N, K, tile, layout, name):
    # few rows, K split, the 128 and the 256 tile: act(+-inf) as the definition evaluates it, the other
    # rows untouched
    sched = None if tile is None else ts.Schedule(order="auto", mode="auto", tile=tile, num_programs=3)
    for dtype, out in ((H, H), (B, F)):
        a, b = infinite(M, N, K, dtype)
        ad, bd = a.cuda(), (b.cuda() if layout == "nn" else b.t().contiguous().cuda().t())
        say(M, N, K, tile, layout, name, dtype)
        z, zerr = R.product(a, b)
        _, bound = R.forward(z, zerr, name, None, out)
        want = z.clamp_min(0.0) if name == "relu" else R.act(z, name)
        finite = torch.isfinite(z)
        res = torch.ones(M, N, dtype=out, device="cuda")
        for residual in (None, res):
            add = 0.0 if residual is None else 1.0
            c = ts.gemm_epilogue(ad, bd, activation=name, residual=residual, out_dtype=out, schedule=sched).double().cpu()
            w = want + add
            same = (c == w) | (c.isnan() & w.isnan())
            assert bool(same[~finite].all()), (name, "infinite sums")
            off = (c - w).abs()[finite]
            assert bool((off <= (bound + 2 * R.U * (w.abs() + 1) + R.rounded(w.abs(), out))[finite]).all()), (name, "finite sums")


@pytest.mark.parametrize("name", R.ACTS)
def test_activation_of_every_magnitude(name):
    # z itself as the product with a unit matrix, from the smallest to the largest, and its ends
    mags = torch.tensor([10.0 ** e for e in range(-37, 39)] + [64.0, 88.0, 104.0, 128.0, 3.0e38, float("inf")])
    z = torch.cat([mags, -mags, torch.tensor([0.0, float("nan")])]).to(B)
    for M in (1, 40):
        c = ts.gemm_epilogue(torch.ones(M, 1, dtype=B, device="cuda"), z[None].cuda(), activation=name, out_dtype=F)
        z64 = z.double()
        want = (z64.clamp_min(0.0) if name == "relu" else R.act(z64, name)).expand(M, -1)
        got = c.double().cpu()
        nan = want.isnan()
        assert bool(got.isnan()[nan].all()), name
        inf = want.isinf()
        assert bool((got == want)[inf].all()), name
        rest = ~nan & ~inf
        size = z64.abs().expand(M, -1)
        # positive arguments: relative; negative ones leave a tail, absolutely small
        bound = R.ACT_ERR * torch.where(z64 > 0, size, (size + 1).clamp_max(300.0)) + 2.0 ** -126
        assert bool(((got - want).abs()[rest] <= bound[rest]).all()), name


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("dtype", [B, F])
def test_slopes_of_every_magnitude(name, dtype):
    # act' of any finite value is finite: act_grad, and the product's gradient form on each of its kernels
    mags = torch.tensor([10.0 ** e for e in range(-37, 39)] + [64.0, 88.0, 104.0, 128.0, 3.0e38])
    z = torch.cat([mags, -mags, torch.tensor([0.0])]).to(dtype)
    N = z.numel()
    want = R.slope(z.double(), name)
    # far out the definition's own 64-bit terms overflow to NaN: the limit there
    far = z.double().abs() > 1e6
    if name != "relu" and name != "none":
        want = torch.where(far, (z.double() > 0).double(), want)
    bound = R.ACT_ERR * (z.double().abs() + 1).clamp_max(300.0)
    dz, _ = ts.act_grad(torch.ones(9, N, dtype=dtype, device="cuda"), z.expand(9, N).contiguous().cuda(), name)
    R.check(dz, want.expand(9, N), (bound + R.rounded(want.abs() + bound, dtype)).expand(9, N), "act_grad")
    op = B if dtype == B else H
    for M, K, tile in ((4, 8, None), (40, 8, None), (40, 2048, None), (300, 64, "256x256x64w8")):
        reps = 1 if tile is None else 4
        zz = z.repeat(reps).expand(M, -1).contiguous().cuda()
        a = torch.zeros(M, K, dtype=op, device="cuda")
        a[:, 0] = 1.0
        b = torch.zeros(K, N * reps, dtype=op, device="cuda")
        b[0] = 1.0
        sched = None if tile is None else ts.Schedule(order="auto", mode="auto", tile=tile)
        say(name, dtype, M, K, tile)
        got = ts.gemm_dact(a, b, zz, name, schedule=sched)
        w, bo = want.repeat(reps).expand(M, -1), bound.repeat(reps).expand(M, -1)
        R.check(got, w, bo + R.rounded(w.abs() + bo, dtype), f"dact {M} {K}")


@pytest.mark.parametrize("M,K,sched", [(1, 64, None), (32, 64, None), (33, 64, None), (33, 2048, None), (200, 64, "128x128x64"),
                                       (300, 256, "256x256x64w8"), (300, 2048, "streamk")])
def test_scales_multiply_in_the_order_they_are_written(M, K, sched):
    # ((A @ B) * scale_a) * scale_b on every kernel: the scales' own product is outside fp32's range
    s = None
    if sched == "streamk":
        s = ts.Schedule(mode="streamk", num_programs=7, tile="128x128x64")
    elif sched:
        s = ts.Schedule(order="auto", mode="auto", tile=sched)
    N = 130 if sched != "256x256x64w8" else 520
    for ea, eb, va, vb in ((70, 60, 2.0 ** -9, 2.0 ** -9), (-100, -50, 256.0, 256.0), (100, -120, 1.0, 1.0)):
        a, b = torch.zeros(M, K), torch.zeros(N, K)
        a[:, 5], b[:, 5] = va, vb
        a[:, K - 1], b[:, K - 1] = va, vb
        want = ((2 * va * vb) * 2.0 ** ea) * 2.0 ** eb
        say(M, K, sched, ea, eb)
        c = ts.gemm_scaled(a.to(Q).cuda(), b.to(Q).cuda().t(), torch.full((M,), 2.0 ** ea, device="cuda"),
                           torch.full((N,), 2.0 ** eb, device="cuda"), out_dtype=F, schedule=s)
        assert bool((c.double() == want).all()), (ea, eb, float(c[0, 0]), want)


def test_stream_k_order_does_not_depend_on_earlier_calls():
    # the automatic order depends on the grid, and a stream-K grid on the number of K steps: a call with few
    # steps in front must not lend its order to one with many on the same tiles, where it would move the cuts
    # along K and with them the bits
    tile, P = "256x256x64w8", 72
    for nm, nn, short, long in ((3, 5, 2, 12), (4, 6, 2, 12), (5, 4, 2, 16)):
        M, N = 256 * nm, 256 * nn
        n = R.gen(nm)
        auto = ts.Schedule(order="auto", mode="streamk", num_programs=P, tile=tile)
        got = []
        for K in (64 * short, 64 * long):
            a, b = n(M, K).to(H).cuda(), (n(K, N) / K ** 0.5).to(H).cuda()
            q = ts.query(M, N, K, auto)
            fixed = ts.Schedule(order=("row_major", "grouped")[q["order"]], group_m=max(q["group_m"], 1), mode="streamk",
                                num_programs=P, xcd_remap=bool(q["xcd_remap"]), tile=tile)
            say(nm, nn, K, fixed.label())
            got.append((q["order"], q["group_m"], q["xcd_remap"]))
            assert torch.equal(ts.gemm_epilogue(a, b, out_dtype=F, schedule=auto), ts.gemm_epilogue(a, b, out_dtype=F, schedule=fixed))
        assert got[0] != got[1]   # the shapes are such that the choice differs


def test_outputs_that_would_overwrite_what_is_still_read():
    # dZ of 16 bits over an fp32 dC, y over h, another row stride in place: errors before any launch
    x, w = torch.ones(40, 40, dtype=B, device="cuda"), torch.ones(40, 40, dtype=B, device="cuda")
    dc = torch.ones(40, 40, dtype=F, device="cuda")
    for call in (lambda: ts.act_grad(dc, None, "none", out=dc.view(B)[:, :40]),
                 lambda: ts.rmsnorm(x, w[0], residual=w, h=x, out=x),
                 lambda: ts.rmsnorm(dc[:, :20], out=dc.view(-1)[:800].view(40, 20))):
        with pytest.raises(ts.TsError) as e:
            call()
        assert e.value.status == ts.TS_ERR_INVALID_ARG
    assert bool((x == 1).all()) and bool((w == 1).all()) and bool((dc == 1).all())


def test_output_on_an_operand_is_refused():
    x, w = torch.ones(40, 40, dtype=B, device="cuda"), torch.ones(40, 40, dtype=B, device="cuda")
    for out in (x, w):
        with pytest.raises(ValueError, match="operand"):
            ts.gemm_epilogue(x, w, out=out)
        with pytest.raises(ValueError, match="operand"):
            ts.gemm_epilogue(x, w.t(), out=out, activation="gelu")
        with pytest.raises(ValueError, match="operand"):
            ts.gemm_epilogue(x, w, preact=out, activation="gelu")
        assert ts.gemm_dact(x, w, out, "relu").shape == (40, 40)   # there it is only read
    assert bool((x == 1).all()) and bool((w == 1).all())
    # nothing to write: an operand of no elements may lie anywhere
    e = torch.empty(0, 40, dtype=B, device="cuda")
    assert ts.gemm_epilogue(e, w, out=e).shape == (0, 40)


def quantised(x):
    s = (x.abs().amax(1) / 448).clamp_min(2.0 ** -100)
    return (x / s[:, None]).to(Q), s


@pytest.mark.parametrize("out", [H, B, F])
@pytest.mark.parametrize("K,pad", [(272, 0), (272, 16), (333, 0), (400, 7)])
def test_every_epilogue_of_8_bit_products_on_the_256_tile(K, pad, out):
    # the 8-bit products (16-bit C) and the widened ones (fp32 C): tiles inside the matrix and on its
    # edges, several a program; rows that the loads take and rows that are packed
    M, N = 600, 900
    sched = ts.Schedule(order="auto", mode="auto", tile="256x256x64w8", num_programs=3)
    n = R.gen(K + pad)
    qa, sa = quantised(n(M, K))
    qb, sb = quantised(n(N, K) / K ** 0.5)
    ad, bd = (torch.full((q.shape[0], K + pad), 448.0).to(Q).cuda()[:, :K].copy_(q.cuda()) for q in (qa, qb))
    bias, res = n(N).to(out), n(M, N).to(out)
    z0, zerr0 = R.product(qa.float(), qb.float().t(), None, sa, sb, eight=out != F)
    z1, zerr1 = R.product(qa.float(), qb.float().t(), bias, sa, sb, eight=out != F)
    p0, perr0 = R.product(qa.float() * 2.0 ** -9, qb.float().t() * 2.0 ** -9, eight=out != F)
    cd, cbuf = R.padded(res, "cuda", 3, 1, fill=7.0)
    pd, pbuf = R.padded(res, "cuda", 3, 1, fill=7.0)
    sa, sb, bias, rd = sa.cuda(), sb.cuda(), bias.cuda(), res.cuda()
    for name in R.ACTS:
        say(K, pad, out, name)
        ts.gemm_scaled(ad, bd.t(), sa, sb, bias=bias, activation=name, out=cd, schedule=sched)
        want, bound = R.forward(z1, zerr1, name, None, out)
        R.check(cd, want, bound, name)
        pd.zero_()
        ts.gemm_scaled(ad, bd.t(), sa, sb, bias=bias, activation=name, preact=pd, out=cd, schedule=sched)
        R.check(cd, want, bound, f"{name} with preact")
        R.check(pd, z1, zerr1 + R.rounded(z1.abs() + zerr1, out), f"{name} preact")
        cd.copy_(res)   # in place
        ts.gemm_scaled(ad, bd.t(), sa, sb, bias=bias, activation=name, residual=cd, out=cd, schedule=sched)
        want, bound = R.forward(z1, zerr1, name, res, out)
        R.check(cd, want, bound, f"{name} with residual")
        pd.zero_()
        ts.gemm_scaled(ad, bd.t(), sa, sb, activation=name, residual=rd, preact=pd, out=cd, schedule=sched)
        want, bound = R.forward(z0, zerr0, name, res, out)
        R.check(cd, want, bound, f"{name} with both")
        R.check(pd, z0, zerr0 + R.rounded(z0.abs() + zerr0, out), f"{name} preact of both")
        # the gradient form has no scales; 2^-18 in all keeps its values in fp16
        pd.copy_(res)
        ones = torch.full((M,), 2.0 ** -9, device="cuda"), torch.full((N,), 2.0 ** -9, device="cuda")
        plain = ts.gemm_scaled(ad, bd.t(), *ones, out_dtype=out, schedule=sched)
        R.check(plain, p0, perr0 + R.rounded(p0.abs() + perr0, out), "powers of two as scales")
        if out != H:
            got = ts.gemm_dact(ad, bd.t(), pd, name, out=pd, schedule=sched)   # in place
            sl, p, perr = R.slope(res.double(), name), p0 * 2.0 ** 18, perr0 * 2.0 ** 18
            err = 1.2 * perr + R.ACT_ERR * (res.double().abs() + 1) * p.abs()
            R.check(got, p * sl, err + R.rounded((p * sl).abs() + err, out), f"{name} gradient")
    for buf, v in ((cbuf, cd), (pbuf, pd)):   # nothing outside the views was written
        v.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("tile", ["128x128x64", "256x256x64w8"])
@pytest.mark.parametrize("out", [H, B, F])
def test_8_bit_products_in_every_mode(tile, out):
    # whole tiles a program: the same bits in every mode; K cut in stream-K mode: the bound, the same bits twice
    M, N, K = 520, 700, 1000
    n = R.gen(12)
    qa, sa = quantised(n(M, K))
    qb, sb = quantised(n(N, K) / K ** 0.5)
    bias, res = n(N).to(out), n(M, N).to(out)
    want, bound = R.forward(*R.product(qa.float(), qb.float().t(), bias, sa, sb, eight=out != F), "gelu", res, out)
    qa, qb, sa, sb, bias, res = (t.cuda() for t in (qa, qb, sa, sb, bias, res))

    def run(**kw):
        say(tile, out, kw)
        return ts.gemm_scaled(qa, qb.t(), sa, sb, bias=bias, activation="gelu", residual=res, out_dtype=out,
                              schedule=ts.Schedule(tile=tile, **kw))

    ref = run()
    R.check(ref, want, bound, "tiled")
    for mode, P in (("persistent", 3), ("crosstile", 5), ("auto", 0)):
        assert torch.equal(ref, run(mode=mode, num_programs=P, order="grouped", group_m=2)), mode
    for P in (5, 7, 0):
        x = run(mode="streamk", num_programs=P, order="auto")
        R.check(x, want, bound, f"stream-K {P}")
        assert torch.equal(x, run(mode="streamk", num_programs=P, order="auto"))


def calls_of_every_kind():
    """Name -> a call whose outputs are a tuple of tensors: one for each kernel that takes a workspace,
    and the few-row and norm kernels."""
    n = R.gen(33)

    def dev(t):
        return t.cuda()

    a, b = dev(n(200, 77).to(B)), dev((n(333, 77) / 9).to(B)).t()              # packed
    s1, s2 = dev(n(60, 2048).to(H)), dev((n(2048, 130) / 45).to(H))            # K split
    x, w = dev(n(5, 1000).to(B)), dev((n(700, 1000) / 31).to(B)).t()           # few rows
    l1, l2 = dev(n(700, 512).to(B)), dev((n(900, 512) / 22).to(B)).t()         # tiles
    qa, sa = quantised(n(130, 500))
    qb, sb = quantised(n(260, 500))
    qa, sa, qb, sb = dev(qa), dev(sa), dev(qb).t(), dev(sb)
    h, dy, g = dev(n(300, 1032).to(B)), dev(n(300, 1032).to(B)), dev(n(1032).to(B))
    z, dc = dev(n(200, 333).to(B)), dev(n(200, 333).to(B))
    sk = ts.Schedule(mode="streamk", num_programs=7, tile="128x128x64")
    return {
        "packed": lambda: (ts.gemm_epilogue(a, b, activation="gelu"),),
        "split": lambda: (ts.gemm_epilogue(s1, s2, activation="silu", out_dtype=F),),
        "few rows": lambda: (ts.gemm_epilogue(x, w, activation="relu"),),
        "tiles": lambda: (ts.gemm_epilogue(l1, l2, activation="gelu_tanh"),),
        "stream-K": lambda: (ts.gemm_epilogue(l1, l2, activation="gelu", schedule=sk),),
        "8 bits": lambda: (ts.gemm_scaled(qa, qb, sa, sb, activation="silu"),),
        "backward": lambda: ts.gemm_epilogue_backward(dc, a, b, preact=z, activation="gelu"),
        "norm": lambda: tuple(ts.rmsnorm(h, g, residual=dy)[i] for i in (0, 2)),
        "norm backward": lambda: ts.rmsnorm_backward(dy, h, g, dh=dy),
    }


def same(got, want, what):
    assert len(got) == len(want)
    for x, y in zip(got, want):
        assert torch.equal(x, y), what


def test_two_streams_at_the_same_time():
    # the same calls in opposite orders on two streams that do not wait for one another, and a captured
    # run of them replayed on a third: each has workspaces of its own
    calls = calls_of_every_kind()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    graph, captured = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        for k, f in calls.items():
            captured[k] = f()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for turn in range(3):
        for outs in captured.values():
            for o in outs:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        got = [[], []]
        for i in range(4):
            with torch.cuda.stream(streams[2]):
                graph.replay()
            for k1, k2 in zip(calls, reversed(calls)):
                for s, k in ((0, k1), (1, k2)):
                    with torch.cuda.stream(streams[s]):
                        got[s].append((k, calls[k]()))
        torch.cuda.synchronize()
        for k, outs in got[0] + got[1] + list(captured.items()):
            same(outs, want[k], (turn, k))


def test_threads():
    # four threads, each on a stream of its own, the first calls of some of them being the process's first
    calls = calls_of_every_kind()
    names = list(calls)
    torch.cuda.synchronize()
    got, errors = [[] for _ in range(4)], []

    def work(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(3 * len(names)):
                    k = names[(i * (t + 1) + t) % len(names)]
                    got[t].append((k, calls[k]()))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (reported below, in the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
        assert not t.is_alive()
    assert not errors, errors
    want = {k: f() for k, f in calls.items()}
    for outs in got:
        assert len(outs) == 3 * len(names)
        for k, o in outs:
            same(o, want[k], k)


@pytest.mark.parametrize("N", [40, 512, 4096, 30000, 70000])
@pytest.mark.parametrize("dtype", [B, F])
def test_e4m3_is_the_quotient_rounded_once(N, dtype):
    # rows of +-1 with eps 0 have r = 1, so y is the weight itself: values next to the middle between two
    # e4m3 numbers times the scale, where a quotient off by one step of fp32 lands on the other side
    n = R.gen(N)
    x = torch.where(n(3, N) > 0, 1.0, -1.0).to(dtype)
    for i in range(8):
        most = float(n(1).abs() + 0.1) * 10.0 ** (2 * i - 8)
        scale = torch.tensor(most) / 448
        steps = torch.arange(0, 255, dtype=torch.uint8).view(Q).float()
        steps = steps[steps.isfinite() & (steps >= 0)].unique().double()
        middle = (steps[1:] + steps[:-1]) / 2 * float(scale)
        pick = torch.randint(0, len(middle), (N,), generator=torch.Generator().manual_seed(i))
        w = middle[pick].float()
        w = (w.view(torch.int32) + torch.randint(-2, 3, (N,), generator=torch.Generator().manual_seed(i + 50), dtype=torch.int32)).view(F)
        w[N // 2] = most
        q, s, _ = ts.rmsnorm(x.cuda(), w.cuda(), eps=0.0, out_dtype=Q)
        say(N, dtype, i)
        assert bool((s.cpu() == w.max() / 448).all())
        want = (w / s.cpu()[:, None] * x.float()).to(Q).float()   # division and rounding of IEEE 754
        assert torch.equal(q.float().cpu(), want), int((q.float().cpu() != want).sum())


def test_e4m3_of_rows_with_infinite_weights():
    w = torch.ones(100)
    w[7] = float("inf")
    q, s, _ = ts.rmsnorm(torch.ones(4, 100, device="cuda"), w.cuda(), out_dtype=Q)
    assert bool((s == float("inf")).all())
    q = q.float()
    assert bool(q[:, 7].isnan().all()) and bool((q[:, :7] == 0).all()) and bool((q[:, 8:] == 0).all())


def test_an_error_left_by_another_call_is_not_this_calls():
    # the caller's own failed HIP call leaves its error behind; the operators report their launches only
    import ctypes

    hip = ctypes.CDLL(next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line))
    calls = calls_of_every_kind()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    for k, f in calls.items():
        f()   # dropped: what the call below allocates is there already (torch would report the error otherwise)
        torch.cuda.synchronize()
        assert hip.hipSetDevice(4096) != 0   # no such device: an error, and nothing else
        try:
            got = f()
        finally:
            left = hip.hipGetLastError()
        assert left != 0, k                  # still there for the caller to see
        same(got, want[k], k)
