"""Layer norm with the residual's addition, its 8-bit outputs and its gradients on the GPU, against
their definitions in 64 bits."""
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

H, B, F, Q, I = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
U = R.U
SHAPES = [(1, 1), (3, 7), (5, 64), (300, 100), (2, 512), (700, 520), (1, 4096), (4, 2048), (300, 2051), (6, 8192),
          (2, 16384), (3, 30000), (2, 32769), (1, 131080)]


def stats(h, eps):
    """u, r, and the error of the kernels' u (absolute) and r (relative).

    Sums of N terms are off by N U of the terms' magnitudes.  The mean is off by e0 = (N + 2) U mean|h|; the
    differences from it are rounded once, their sum corrects the mean, so a centred value is off by
    its own roundings and by the error of that correction; the variance is a sum of squares of
    differences that may be e0 larger, its root halves the error.  (h itself: one rounding.)
    """
    N = h.shape[1]
    c = h - h.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    e0 = (N + 2) * U * h.abs().mean(1, keepdim=True)
    cerr = U * (h.abs() + 4 * c.abs()) + (N + 4) * U * (c.abs().mean(1, keepdim=True) + e0) + 2 * U * e0
    verr = (N + 8) * U * ((c * c).mean(1, keepdim=True) + 4 * e0 * e0) + 2 * (c * cerr).abs().mean(1, keepdim=True)
    rerr = 0.5 * verr * r * r + 6 * U
    return c * r, r, cerr * r + (c * r).abs() * (rerr + 2 * U), rerr


def forward(h, w, b, eps=1e-5):
    u, _, uerr, _ = stats(h, eps)
    y = u * w + b
    return y, uerr * w.abs() + 2 * U * ((u * w).abs() + y.abs())


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(B, B), (H, F), (F, F)])
def test_norm(M, N, dtype, wtype):
    n = R.gen(M + N)
    x, res = (n(M, N) + 2 * n(M, 1)).to(dtype), n(M, N).to(dtype)
    w, b = (1 + 0.2 * n(N)).to(wtype), (0.3 * n(N)).to(wtype)
    for residual in (None, res):
        say(M, N, dtype, residual is not None)
        rd = None if residual is None else residual.cuda()
        h64 = x.double() + (0 if residual is None else res.double())
        for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
            y, scale, h = ts.layernorm(x.cuda(), None if ww is None else ww.cuda(), None if bb is None else bb.cuda(), residual=rd)
            want, err = forward(h64, torch.ones(N).double() if ww is None else ww.double(),
                                torch.zeros(N).double() if bb is None else bb.double())
            R.check(y, want, err + R.rounded(want.abs() + err, dtype), "y")
            assert scale is None
        want, err = forward(h64, w.double(), b.double())
        if residual is not None:   # two 16-bit values add exactly or within one fp32 rounding
            R.check(h, h64, U * h64.abs() + R.rounded(h64.abs() * (1 + U), dtype), "h")
        keep = ts.Checkpoint.empty(M, N)
        for to, top in ((Q, 448.0), (I, 127.0)):
            q, s, h2 = ts.layernorm(x.cuda(), w.cuda(), b.cuda(), residual=rd, out_dtype=to, keep=keep)
            assert torch.equal(h2, h)
            amax, aerr = want.abs().amax(1), err.amax(1)
            R.check(s, (amax / top).clamp_min(2.0 ** -100), (aerr + 4 * U * amax) / top + 1e-37, "scale")
            v = q.double().cpu() * s.double().cpu()[:, None]
            step = s.double().cpu()[:, None]
            # half a step: relative to the value and at least 2^-10 of the scale, or of the scale itself
            half = 2.0 ** -4 * want.abs() + 2.0 ** -10 * step if to == Q else 0.5 * step + 127 * U * step
            R.check(v, want, half + 2 * err + 1e-30, str(to))
            # what is kept is the unrounded sum (one fp32 addition)
            K8.check_bytes(keep, (x.float() + (0 if residual is None else res.float())).double(), "keep")


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 8)])
def test_strides_in_place_and_guards(pad, offset):
    for M, N in [(9, 65), (4, 1027)]:
        n = R.gen(N)
        x, res, w, b = n(M, N).to(B), n(M, N).to(B), n(N).to(B), n(N).to(B)
        want = ts.layernorm(x.cuda(), w.cuda(), b.cuda(), residual=res.cuda())
        xd, xb = R.padded(x, "cuda", pad, offset, fill=3.0)
        rd, rb = R.padded(res, "cuda", pad, offset, fill=3.0)
        yd, yb = R.padded(torch.zeros(M, N).to(B), "cuda", pad, offset, fill=3.0)
        say(M, N, pad, offset)
        ts.layernorm(xd, w.cuda(), b.cuda(), residual=rd, out=yd, h=rd)   # h takes the residual's place
        assert torch.equal(yd, want[0]) and torch.equal(rd, want[2])
        for to in (Q, I):
            q0 = ts.layernorm(x.cuda(), w.cuda(), b.cuda(), residual=res.cuda(), out_dtype=to)
            qd = torch.full((M, N + pad), 1.0).to(to).cuda()
            q, s, _ = ts.layernorm(x.cuda(), w.cuda(), b.cuda(), residual=res.cuda(), out=qd[:, :N])
            assert torch.equal(q.float(), q0[0].float()) and torch.equal(s, q0[1])
            assert bool((qd[:, N:].float() == 1.0).all())
        for v, buf in ((rd, rb), (yd, yb)):
            v.fill_(3.0)
            assert bool((buf == 3.0).all())


@pytest.mark.parametrize("N", [5, 200, 3000, 40000])
def test_special_rows(N):
    x = R.gen(N)(7, N)
    x[0] = 0.0                       # no spread
    x[1] = 1234.5
    x[2, 2] = float("nan")
    x[3, 3] = float("inf")
    x[4] *= 1e-30                    # eps decides
    x[5] *= 1e15
    x[6] = x[6] + 4096.0             # a mean four thousand times the spread
    b = torch.full((N,), 0.25)
    y, _, _ = ts.layernorm(x.cuda(), bias=b.cuda())
    q, s, _ = ts.layernorm(x.cuda(), out_dtype=I)
    assert bool((y[0] == 0.25).all()) and bool((q[0] == 0).all()) and float(s[0]) == 2.0 ** -100
    want, err = forward(x.double(), torch.ones(N).double(), b.double())
    # a row without spread: the mean's rounding is all there is, and its square beside eps is nothing
    R.check(y[1], torch.full((N,), 0.25).double(), 0.25 * U + 1234.5 * U * 4 / 1e-5 ** 0.5, "constant row")
    assert bool(y[2].isnan().all()) and bool(s[2].isnan()) and bool(y[3].isnan().all()) and bool(s[3].isnan())
    R.check(y[4:], want[4:], err[4:] + R.rounded(want[4:].abs() + err[4:], F), "y")
    # the correction of the mean: well below what the mean's own rounding (2^-12 of a spread) would leave
    off = (y[6].double().cpu() - want[6]).abs().max()
    assert float(off) < 2.0 ** -11
    assert ts.layernorm(torch.empty(0, N, device="cuda"))[0].shape == (0, N)


@pytest.mark.parametrize("M", [1, 17])
def test_no_columns(M):
    x = torch.empty(M, 0, device="cuda")
    for to in (Q, I):
        q, s, _ = ts.layernorm(x, out_dtype=to)
        assert q.shape == (M, 0) and bool((s == 2.0 ** -100).all())
    dx, dw, db = ts.layernorm_backward(x, x, torch.empty(0, device="cuda"))
    assert dx.shape == (M, 0) and dw.shape == (0,) and db.shape == (0,)


GRADS = [(1, 1), (3, 7), (5, 64), (1100, 100), (40, 520), (1, 4096), (2100, 1030), (9, 8192), (3, 12000), (3, 16384),
         (5, 20000), (70, 16392), (2, 70001)]


def gradients(h, dy, w, dh, eps):
    """dx, dw, db and the errors of the kernels (before the last rounding)."""
    M, N = h.shape
    u, r, uerr, rerr = stats(h, eps)
    g = w * dy
    mean = lambda t: t.mean(1, keepdim=True)
    mg, mgu = mean(g), mean(g * u)
    want = r * (g - mg - u * mgu) + dh
    mgerr = (N + 4) * U * mean(g.abs())
    mguerr = (N + 8) * U * mean((g * u).abs()) + mean(g.abs() * uerr) + mgerr * mean(u.abs() + uerr) * (N + 4) * U
    err = (r * (g.abs() + mg.abs() + (u * mgu).abs()) * (rerr + 6 * U) + r * mgerr + r * uerr * (mgu.abs() + mguerr)
           + r * u.abs() * mguerr + 4 * U * (want.abs() + dh.abs()))
    dw, db = (dy * u).sum(0), dy.sum(0)
    dwerr = (dy.abs() * uerr).sum(0) + (M + 4) * U * (dy * u).abs().sum(0)
    return want, err, dw, dwerr, db, (M + 4) * U * dy.abs().sum(0)


@pytest.mark.parametrize("M,N", GRADS)
@pytest.mark.parametrize("dtype,wtype", [(B, B), (H, F), (F, F)])
def test_backward(M, N, dtype, wtype):
    n = R.gen(M * 3 + N)
    h, dy, dh = (n(M, N) + n(M, 1)).to(dtype), (n(M, N) + 0.5).to(dtype), n(M, N).to(dtype)
    w = (1 + 0.2 * n(N)).to(wtype)
    say(M, N, dtype, wtype)
    args = dict(eps=1e-3, dh=dh.cuda())
    dx, dw, db = ts.layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), **args)
    want, err, wd, derr, bd, berr = gradients(h.double(), dy.double(), w.double(), dh.double(), 1e-3)
    R.check(dx, want, err + R.rounded(want.abs() + err, dtype), "dx")
    R.check(dw, wd, derr + R.rounded(wd.abs() + derr, wtype), "dweight")
    R.check(db, bd, berr + R.rounded(bd.abs() + berr, wtype), "dbias")
    # the same bits twice, with fewer outputs and with dx in dy's place
    for kw in (dict(), dict(dweight=False), dict(dbias=False), dict(dweight=False, dbias=False)):
        d2, w2, b2 = ts.layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), **args, **kw)
        assert torch.equal(dx, d2) and (w2 is None or torch.equal(dw, w2)) and (b2 is None or torch.equal(db, b2))
        assert (w2 is None) == ("dweight" in kw) and (b2 is None) == ("dbias" in kw)
    dyc, dhc = dy.cuda(), dh.cuda()
    ts.layernorm_backward(dyc, h.cuda(), w.cuda(), eps=1e-3, dh=dhc, out=dyc)
    assert torch.equal(dyc, dx)
    ts.layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-3, dh=dhc, out=dhc)
    assert torch.equal(dhc, dx)
    d4, w4, b4 = ts.layernorm_backward(dy.cuda(), h.cuda(), eps=1e-3)
    assert w4 is None and b4.dtype == F
    want, err, _, _, bd, berr = gradients(h.double(), dy.double(), torch.ones(N).double(), torch.zeros(M, N).double(), 1e-3)
    R.check(d4, want, err + R.rounded(want.abs() + err, dtype), "dx without weight")
    R.check(b4, bd, berr + R.rounded(bd.abs() + berr, F), "dbias without weight")


@pytest.mark.parametrize("M,N", GRADS)
@pytest.mark.parametrize("dtype", [B, H, F])
def test_backward_from_checkpoint(M, N, dtype):
    n = R.gen(M + 7 * N)
    h, dy, dh = n(M, N) + n(M, 1), n(M, N).to(dtype), n(M, N).to(dtype)
    w = (1 + 0.2 * n(N)).to(dtype)
    k = ts.checkpoint_pack(h.cuda())
    if N % 32:   # what lies behind column N does not matter
        k.data[:, N:(N + 31) // 32 * 32] = 99
    say(M, N, dtype)
    dx, dw, db = ts.layernorm_backward(dy.cuda(), k, w.cuda(), eps=1e-3, dh=dh.cuda())
    want, err, wd, derr, bd, berr = gradients(K8.unpack(k.data, N), dy.double(), w.double(), dh.double(), 1e-3)
    R.check(dx, want, err + R.rounded(want.abs() + err, dtype), "dx")
    R.check(dw, wd, derr + R.rounded(wd.abs() + derr, dtype), "dweight")
    R.check(db, bd, berr + R.rounded(bd.abs() + berr, dtype), "dbias")
    if dtype != H:   # the values are exact in bf16 and fp32: the same bits
        d2 = ts.layernorm_backward(dy.cuda(), ts.checkpoint_unpack(k, out_dtype=dtype), w.cuda(), eps=1e-3, dh=dh.cuda())
        assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), d2))


@pytest.mark.parametrize("M,N", [(5, 64), (6, 4096), (9, 16384), (3, 32776)])
def test_backward_far_from_unit_scale(M, N):
    n = R.gen(M + N)
    for scale in (1e12, 1e-12):
        h, dy = n(M, N) * scale, n(M, N)
        dx, dw, db = ts.layernorm_backward(dy.cuda(), h.cuda(), torch.ones(N, device="cuda"), eps=0.0)
        want, err, wd, derr, _, _ = gradients(h.double(), dy.double(), torch.ones(N).double(), torch.zeros(M, N).double(), 0.0)
        R.check(dx, want, err + R.rounded(want.abs() + err, F), "dx")
        R.check(dw, wd, derr + R.rounded(wd.abs() + derr, F), "dweight")


def test_backward_against_differences_and_no_rows():
    n = R.gen(7)
    h, dy, w, b = n(6, 48), n(6, 48), 1 + 0.2 * n(48), n(48)
    dx, dw, db = ts.layernorm_backward(dy.cuda(), h.cuda(), w.cuda())

    def loss(h, w, b):
        return float(((stats(h, 1e-5)[0] * w + b) * dy.double()).sum())

    h64, w64, b64 = h.double(), w.double(), b.double()
    for g, x, f in ((dx, h64, lambda v: loss(v, w64, b64)), (dw, w64, lambda v: loss(h64, v, b64)), (db, b64, lambda v: loss(h64, w64, v))):
        v = n(*x.shape).double()
        want = (f(x + 1e-5 * v) - f(x - 1e-5 * v)) / 2e-5
        size = float((g.double().cpu().abs() * v.abs()).sum())
        assert abs(float((g.double().cpu() * v).sum()) - want) <= 200 * U * size + 1e-6 * abs(want)
    e = torch.empty(0, 48, device="cuda")
    dx, dw, db = ts.layernorm_backward(e, e, w.cuda())
    assert dx.shape == (0, 48) and bool((dw == 0).all()) and bool((db == 0).all())


def test_captured_graph_and_streams():
    n = R.gen(8)
    x, r, w, b = n(64, 1000).to(B).cuda(), n(64, 1000).to(B).cuda(), n(1000).to(B).cuda(), n(1000).to(B).cuda()

    def both():
        keep = ts.Checkpoint.empty(64, 1000)
        q, s, h = ts.layernorm(x, w, b, residual=r, out_dtype=I, keep=keep)
        return (q, s, h, *ts.layernorm_backward(x, keep, w, dh=r), *ts.layernorm_backward(x, h, w))

    eager = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(eager, other))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        again = both()
    for i in range(3):
        for t in again:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(eager, again))
        ts.layernorm(x, w)


def test_more_rows_than_a_launch_holds():
    # two columns: y = +-d / sqrt(d^2 + eps), d half their difference; 2^27 + 5 rows are more threads than one launch takes
    M = (1 << 27) + 5
    x = torch.empty(M, 2, dtype=H, device="cuda").uniform_(-2, 2)
    y, _, _ = ts.layernorm(x, eps=1.0)
    for i in range(0, M, 1 << 25):
        v = x[i:i + (1 << 25)].float()
        d = (v[:, :1] - v[:, 1:]) * 0.5
        want = torch.cat([d, -d], 1) * torch.rsqrt(d * d + 1.0)
        # two fp32 evaluations of up to 16 roundings of values up to 2, and half a step of fp16
        off = (y[i:i + (1 << 25)].float() - want).abs()
        assert bool((off <= want.abs() * 2.0 ** -11 + 64 * 2.0 ** -24 + 2.0 ** -25).all()), i


def test_beyond_32_bits():
    # more than 2^32 bytes, and 2^31 elements, in every matrix: the last rows
    M, N = 300005, 8000
    x = torch.empty(M, N, dtype=B, device="cuda").normal_()
    w = torch.empty(N, dtype=B, device="cuda").uniform_(0.5, 1.5)
    rows = [0, 1, M // 2, M - 2, M - 1]
    x64, w64 = x[rows].double().cpu(), w.double().cpu()
    k = ts.Checkpoint.empty(M, N)
    y, _, _ = ts.layernorm(x, w, keep=k)
    want, err = forward(x64, w64, 0.0)
    R.check(y[rows], want, err + R.rounded(want.abs() + err, B), "y")
    K8.check_bytes(ts.Checkpoint(k.data[rows].contiguous(), N), x64)
    dy = y[rows].double().cpu()
    for h, h64 in ((x, x64), (k, K8.unpack(k.data[rows], N))):
        dx, dw, db = ts.layernorm_backward(y, h, w, dh=y)
        full, err = gradients(h64, dy, w64, dy, 1e-5)[:2]
        R.check(dx[rows], full, err + R.rounded(full.abs() + err, B), "dx")
        assert torch.isfinite(dw.float()).all() and torch.isfinite(db.float()).all()
        del dx


def test_layer_forward_and_backward_together():
    # a feed-forward block whose norm and activation are kept in 8 bits, against the same block in 64 bits
    # whose backward pass starts from the kept values
    n = R.gen(51)
    M, D, E = 130, 264, 520
    x, r, g, b = n(M, D).to(B), n(M, D).to(B), (1 + 0.2 * n(D)).to(B), (0.1 * n(D)).to(B)
    w1, b1, w2 = (n(D, E) / D ** 0.5).to(B), n(E).to(B), (n(E, D) / E ** 0.5).to(B)
    do = n(M, D).to(B)
    c = lambda t: t.cuda()
    kh, kz = ts.Checkpoint.empty(M, D), ts.Checkpoint.empty(M, E)
    y, _, h = ts.layernorm(c(x), c(g), c(b), residual=c(r), keep=kh)
    u = ts.gemm_epilogue(y, c(w1), bias=c(b1), activation="gelu", preact=kz)
    o = ts.gemm_epilogue(u, c(w2), residual=h)
    # backward: u is formed again from kz, y from kh
    dub = ts.gemm_epilogue(c(do), c(w2).t())
    u2 = torch.empty(M, E, dtype=B, device="cuda")
    dz, db1 = ts.act_grad(dub, kz, "gelu", act_out=u2)
    dw2 = ts.gemm_epilogue(u2.t(), c(do))
    y2, _, _ = ts.layernorm(ts.checkpoint_unpack(kh, out_dtype=B), c(g), c(b))
    dy, dw1 = ts.gemm_epilogue(dz, c(w1).t()), ts.gemm_epilogue(y2.t(), dz)
    dx, dg, db = ts.layernorm_backward(dy, kh, c(g), dh=c(do))

    d = lambda t: t.double().cpu()
    h64 = d(x) + d(r)
    y64 = stats(h64, 1e-5)[0] * d(g) + d(b)
    z64 = y64 @ d(w1) + d(b1)
    o64 = R.act(z64, "gelu") @ d(w2) + h64
    hk, zk = K8.unpack(kh.data, D), K8.unpack(kz.data, E)
    yk = stats(hk, 1e-5)[0] * d(g) + d(b)
    du64 = d(do) @ d(w2).t()
    dz64 = du64 * R.slope(zk, "gelu")
    want = {"o": o64, "dz": dz64, "db1": dz64.sum(0), "dw2": R.act(zk, "gelu").t() @ d(do), "dw1": yk.t() @ dz64}
    dy64 = dz64 @ d(w1).t()
    full = gradients(hk, dy64, d(g), d(do), 1e-5)
    want.update(dx=full[0], dg=full[2], db=full[4])
    got = {"o": o, "dz": dz, "db1": db1, "dw2": dw2, "dw1": dw1, "dx": dx, "dg": dg, "db": db}
    for name, t in want.items():
        # chains of up to six roundings to bf16 (2^-8 at most, 2^-8 / sqrt(3) in the mean square), each carried on with a
        # factor of about one: under 2 % of the output's norm
        assert float((d(got[name]) - t).norm() / t.norm()) < 0.02, name


# Rows whose mean is thousands of deviations.  x - mean is exact there (the two are within a factor of two of each
# other), so what is left of the mean's rounding is the error of its correction, the mean of those differences.
# A sum here is at most DEEP additions deep: up to 40 of a thread's own, then the exchanges between threads.
DEEP = 64


def far_stats(h, eps):
    """As stats, for such rows; the mean is off by less than 2^-6 before its correction (DEEP roundings of 2^13)."""
    c = h - h.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    cerr = (DEEP + 4) * U * (c.abs() + c.abs().mean(1, keepdim=True) + 2.0 ** -6)
    rerr = (DEEP + 16) * U
    return c * r, r, cerr * r + (c * r).abs() * (rerr + 2 * U), rerr


def far_rows(M, N):
    n = R.gen(M + 5 * N)
    return n(M, N) + 4096.0 + 100.0 * n(M, 1), n


@pytest.mark.parametrize("N", [200, 3000, 16384, 40000])
def test_mean_far_from_zero(N):
    h, n = far_rows(32, N)
    w, b = 1 + 0.2 * n(N), 0.3 * n(N)
    y, _, _ = ts.layernorm(h.cuda(), w.cuda(), b.cuda())
    u, _, uerr, _ = far_stats(h.double(), 1e-5)
    want = u * w.double() + b.double()
    R.check(y, want, uerr * w.double().abs() + 3 * U * ((u * w.double()).abs() + want.abs()), "y")


@pytest.mark.parametrize("N", [200, 3000, 12000, 16384, 20000, 40000])
def test_backward_mean_far_from_zero(N):
    h, n = far_rows(16, N)
    u, r, uerr, rerr = far_stats(h.double(), 1e-5)
    w = 1 + 0.2 * n(N)
    # dy along u, so that mean(g u) is about one and u's error reaches dx
    dy = (u + 0.2 * n(16, N)).float()
    dx, dw, db = ts.layernorm_backward(dy.cuda(), h.cuda(), w.cuda())
    mean = lambda t: t.mean(1, keepdim=True)
    y64 = dy.double()
    g = w.double() * y64
    mg, mgu = mean(g), mean(g * u)
    want = r * (g - mg - u * mgu)
    mguerr = (2 * DEEP + 16) * U * (mean((g * u).abs()) + mean(g.abs()))
    err = (r * ((g.abs() + mg.abs() + (u * mgu).abs()) * (rerr + 6 * U) + DEEP * U * mean(g.abs()) + uerr * (mgu.abs() + mguerr)
                + (u.abs() + uerr) * mguerr) + 4 * U * want.abs())
    R.check(dx, want, err + R.rounded(want.abs() + err, F), "dx")
    wd, derr = (y64 * u).sum(0), (y64.abs() * uerr).sum(0) + 20 * U * (y64 * u).abs().sum(0)
    R.check(dw, wd, derr + R.rounded(wd.abs() + derr, F), "dweight")
    R.check(db, y64.sum(0), 20 * U * y64.abs().sum(0) + R.TINY[F], "dbias")
