"""The norm with the residual's addition, its e4m3 output and its gradients on the GPU,
against their definitions in 64 bits."""
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
EPS = 1e-6
SHAPES = [(1, 1), (3, 7), (5, 64), (300, 100), (2, 512), (700, 520), (1, 4096), (4, 2048), (300, 2051), (6, 8192),
          (2, 16384), (3, 30000), (2, 65536), (2, 65537), (1, 131080)]


def norm64(h, w, eps=EPS):
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * r * w, r


def y_error(y, N):
    # r: a sum of N squares (each rounding relative to the sum of magnitudes, which is the sum
    # itself), halved by the root, plus division, root and reciprocal; then two products
    return ((N / 2 + 8) * R.U) * y.abs()


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(B, B), (H, F), (F, F)])
def test_norm(M, N, dtype, wtype):
    n = R.gen(M + N)
    x, res = n(M, N).to(dtype), n(M, N).to(dtype)
    w = (1 + 0.2 * n(N)).to(wtype)
    for residual in (None, res):
        say(M, N, dtype, residual is not None)
        y, scale, h = ts.rmsnorm(x.cuda(), w.cuda(), residual=None if residual is None else residual.cuda())
        h64 = x.double() + (0 if residual is None else res.double())
        want, _ = norm64(h64, w.double())
        err = y_error(want, N) + (0 if residual is None else 2 * R.U) * want.abs()
        R.check(y, want, err + R.rounded(want.abs() + err, dtype), "y")
        assert scale is None
        if residual is not None:   # two 16-bit values add exactly or within one fp32 rounding
            R.check(h, h64, R.U * h64.abs() + R.rounded(h64.abs() * (1 + R.U), dtype), "h")
        q, s, h2 = ts.rmsnorm(x.cuda(), w.cuda(), residual=None if residual is None else residual.cuda(), out_dtype=Q)
        assert torch.equal(h2, h)
        amax = (want.abs() + 0).amax(1)
        R.check(s, (amax / 448).clamp_min(2.0 ** -100), (N / 2 + 16) * R.U * amax / 448 + 1e-37, "scale")
        v = q.double().cpu() * s.double().cpu()[:, None]
        # half a step of e4m3 relative to the value, or half the smallest step (2^-10 of the scale)
        bound = 2.0 ** -4 * want.abs() + 2.0 ** -10 * s.double().cpu()[:, None] + 2 * err + 1e-30
        R.check(v, want, bound, "e4m3")


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 8)])
def test_norm_strides_in_place_and_guards(pad, offset):
    for M, N in [(9, 65), (4, 1027)]:
        n = R.gen(N)
        x, res, w = n(M, N).to(B), n(M, N).to(B), n(N).to(B)
        want = ts.rmsnorm(x.cuda(), w.cuda(), residual=res.cuda())
        xd, xb = R.padded(x, "cuda", pad, offset, fill=3.0)
        rd, rb = R.padded(res, "cuda", pad, offset, fill=3.0)
        yd, yb = R.padded(torch.zeros(M, N).to(B), "cuda", pad, offset, fill=3.0)
        say(M, N, pad, offset)
        y, _, h = ts.rmsnorm(xd, w.cuda(), residual=rd, out=yd, h=rd)   # h takes the residual's place
        assert torch.equal(yd, want[0]) and torch.equal(rd, want[2])
        q0 = ts.rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), out_dtype=Q)
        qd = torch.full((M, N + pad), 1.0).to(Q).cuda()
        q, s, _ = ts.rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), out=qd[:, :N])
        assert torch.equal(q.float(), q0[0].float()) and torch.equal(s, q0[1])
        assert bool((qd[:, N:].float() == 1.0).all())
        for v, b in ((rd, rb), (yd, yb)):
            v.fill_(3.0)
            assert bool((b == 3.0).all())


@pytest.mark.parametrize("N", [5, 200, 3000, 70000])
def test_norm_special_rows(N):
    x = R.gen(N)(6, N)
    x[0] = 0.0                       # a row of zeros
    x[1, 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] *= 1e-30                    # eps decides
    x[4] *= 1e15
    y, _, _ = ts.rmsnorm(x.cuda())
    q, s, _ = ts.rmsnorm(x.cuda(), out_dtype=Q)
    assert bool((y[0] == 0).all()) and bool((q[0].float() == 0).all()) and float(s[0]) == 2.0 ** -100
    assert bool(y[1].isnan().all()) and bool(q[1].float().isnan().all()) and bool(s[1].isnan())
    assert bool(y[2, 3].isnan()) and bool((y[2, :3] == 0).all()) and bool(s[2].isnan())
    want, _ = norm64(x[3:].double(), torch.ones(N).double())
    R.check(y[3:], want, y_error(want, N) + R.rounded(want, F))
    # an empty matrix, and one of no rows
    assert ts.rmsnorm(torch.empty(0, N, device="cuda"))[0].shape == (0, N)


@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (5, 64), (1100, 100), (40, 520), (1, 4096), (2100, 1030), (9, 8192),
                                 (3, 16384), (5, 20000), (2, 32768), (70, 32776), (2, 70001)])
@pytest.mark.parametrize("dtype,wtype", [(B, B), (H, F), (F, F)])
def test_norm_backward(M, N, dtype, wtype):
    n = R.gen(M * 3 + N)
    h, dy, dh = n(M, N).to(dtype), n(M, N).to(dtype), n(M, N).to(dtype)
    w = (1 + 0.2 * n(N)).to(wtype)
    say(M, N, dtype, wtype)
    dx, dw = ts.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-3, dh=dh.cuda())
    h64, dy64, w64 = h.double(), dy.double(), w.double()
    y, r = norm64(h64, torch.ones(N).double(), 1e-3)
    g = w64 * dy64
    k = r ** 3 * (g * h64).mean(1, keepdim=True)
    want = r * g - h64 * k + dh.double()
    # r is off by (N/2 + 8) U relative; k by the sum's (N + 3 N/2 + 32) U of its terms' magnitudes
    rerr = (N / 2 + 8) * R.U
    kerr = r ** 3 * (g * h64).abs().mean(1, keepdim=True) * (2.5 * N + 40) * R.U
    err = (r * g).abs() * (rerr + 4 * R.U) + h64.abs() * (kerr + 4 * R.U * k.abs()) + 2 * R.U * (want.abs() + dh.double().abs())
    R.check(dx, want, err + R.rounded(want.abs() + err, dtype), "dx")
    wd = (dy64 * y).sum(0)
    derr = (dy64 * y).abs().sum(0) * ((M + 4) * R.U + rerr)
    R.check(dw, wd, derr + R.rounded(wd.abs() + derr, wtype), "dweight")
    # without the stream's gradient and without a weight; dx in dy's place; the same bits twice
    d2, w2 = ts.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-3, dh=dh.cuda())
    assert torch.equal(dx, d2) and torch.equal(dw, w2)
    dyc = dy.cuda()
    d3, w3 = ts.rmsnorm_backward(dyc, h.cuda(), w.cuda(), eps=1e-3, dh=dh.cuda(), out=dyc)
    assert torch.equal(dyc, dx) and torch.equal(w3, dw)
    d4, w4 = ts.rmsnorm_backward(dy.cuda(), h.cuda(), eps=1e-3)
    assert w4 is None
    k1 = r ** 3 * (dy64 * h64).mean(1, keepdim=True)
    want = r * dy64 - h64 * k1
    kerr = r ** 3 * (dy64 * h64).abs().mean(1, keepdim=True) * (2.5 * N + 40) * R.U
    err = (r * dy64).abs() * (rerr + 4 * R.U) + h64.abs() * (kerr + 4 * R.U * k1.abs()) + 2 * R.U * want.abs()
    R.check(d4, want, err + R.rounded(want.abs() + err, dtype), "dx without weight")


def test_norm_backward_against_differences_and_no_rows():
    n = R.gen(7)
    h, dy, w = n(6, 48), n(6, 48), 1 + 0.2 * n(48)
    dx, dw = ts.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda())

    def loss(h, w):
        return float((norm64(h, w)[0] * dy.double()).sum())

    for g, x, f in ((dx, h, lambda v: loss(v, w.double())), (dw, w, lambda v: loss(h.double(), v))):
        v = n(*x.shape).double()
        want = (f(x.double() + 1e-5 * v) - f(x.double() - 1e-5 * v)) / 2e-5
        size = float((g.double().cpu().abs() * v.abs()).sum())
        assert abs(float((g.double().cpu() * v).sum()) - want) <= 200 * R.U * size + 1e-6 * abs(want)
    dx, dw = ts.rmsnorm_backward(torch.empty(0, 48, device="cuda"), torch.empty(0, 48, device="cuda"), w.cuda())
    assert dx.shape == (0, 48) and bool((dw == 0).all())


def test_norm_captured_graph():
    n = R.gen(8)
    x, r, w = n(64, 1000).to(B).cuda(), n(64, 1000).to(B).cuda(), n(1000).to(B).cuda()
    eager = ts.rmsnorm(x, w, residual=r, out_dtype=Q)
    dx0, dw0 = ts.rmsnorm_backward(x, eager[2], w, dh=r)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        q, s, h = ts.rmsnorm(x, w, residual=r, out_dtype=Q)
        dx, dw = ts.rmsnorm_backward(x, h, w, dh=r)
    for i in range(3):
        for t in (s, h, dx, dw):
            t.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.float(), eager[0].float()) and torch.equal(s, eager[1]) and torch.equal(h, eager[2])
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
        ts.rmsnorm(x, w)


def test_norm_of_more_rows_than_a_launch_holds():
    # one column: y = x / sqrt(x^2 + eps) w; 2^27 + 5 rows are more threads than one launch takes
    M = (1 << 27) + 5
    x = torch.empty(M, 1, dtype=H, device="cuda").uniform_(-2, 2)
    w = torch.tensor([3.0], device="cuda")
    y, _, _ = ts.rmsnorm(x, w, eps=1.0)
    for i in range(0, M, 1 << 25):
        v = x[i:i + (1 << 25)].float()
        want = 3.0 * v * torch.rsqrt(v * v + 1.0)
        # two fp32 evaluations (each within 8 roundings of 2^-24) and half a step of fp16
        off = (y[i:i + (1 << 25)].float() - want).abs()
        assert bool((off <= want.abs() * (2.0 ** -11 + 16 * 2.0 ** -24) + 2.0 ** -25).all()), i


def test_beyond_32_bits():
    # more than 2^32 bytes, and 2^31 elements, in every matrix: the last rows
    M, N = 300005, 8000
    x = torch.empty(M, N, dtype=B, device="cuda").normal_()
    w = torch.empty(N, dtype=B, device="cuda").uniform_(0.5, 1.5)
    rows = [0, 1, M // 2, M - 2, M - 1]
    x64, w64 = x[rows].double().cpu(), w.double().cpu()
    y, _, _ = ts.rmsnorm(x, w)
    want, r = norm64(x64, w64)
    R.check(y[rows], want, y_error(want, N) + R.rounded(want.abs() * 1.01, B), "y")
    dy = y[rows].double().cpu()
    dx, dw = ts.rmsnorm_backward(y, x, w, dh=y, out=y)   # dy and dh are y itself
    k = r ** 3 * (w64 * dy * x64).mean(1, keepdim=True)
    full = r * w64 * dy - x64 * k + dy
    # the sums of N products in r and k (N 2^-24 each, r cubed), a few products, one rounding to bf16
    size = (r * w64 * dy).abs() + x64.abs() * r ** 3 * (w64 * dy * x64).abs().mean(1, keepdim=True) + dy.abs()
    err = (3 * N + 32) * R.U * size
    R.check(dx[rows], full, err + R.rounded(full.abs() + err, B), "dx")
    assert torch.isfinite(dw.float()).all()
