"""The operators around the product on the CPU: every refusal comes before any HIP call, and
valid calls reach the device check."""
import ctypes
import re

import pytest
import torch

import tile_scheduling_amd as ts

FAKE = 0x10000   # 256-byte aligned, never dereferenced: every call below ends before a launch
INV, UNS, ALI, DEV = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED, ts.TS_ERR_ALIGNMENT, ts.TS_ERR_NO_DEVICE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


def epilogue(M=64, N=64, K=64, a=FAKE, b=FAKE, c=FAKE, strides=(64, 1, 64, 1, 64, 1), ab=ts.TS_F16, ct=ts.TS_F16,
             epi=None, sched=None, ws=None, wb=0):
    e = ts._Epilogue(**epi) if epi is not None else None
    return ts._lib.ts_gemm_epilogue(a, b, c, M, N, K, *strides, ab, ct, ctypes.byref(e) if e is not None else None,
                                    ctypes.byref(sched._c()) if sched else None, None, ws, wb)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(K=-1), INV), (dict(M=1 << 32), UNS), (dict(ab=9), INV), (dict(ct=ts.TS_E4M3), UNS),
    (dict(ab=ts.TS_F32, ct=ts.TS_F32), UNS), (dict(ab=ts.TS_F16, ct=ts.TS_BF16), UNS),
    (dict(ab=ts.TS_E4M3, ct=ts.TS_BF16), UNS),                                    # B stored [K][N]
    (dict(ab=ts.TS_E4M3, ct=ts.TS_BF16, strides=(1, 64, 1, 64, 64, 1)), UNS),     # A stored [K][M]
    (dict(strides=(64, 2, 64, 1, 64, 1)), UNS), (dict(strides=(64, 1, 64, 2, 64, 1)), UNS),
    (dict(strides=(64, 1, 64, 1, 64, 2)), UNS), (dict(strides=(63, 1, 64, 1, 64, 1)), INV),
    (dict(strides=(0, 1, 64, 1, 64, 1)), INV), (dict(strides=(-64, 1, 64, 1, 64, 1)), INV),
    (dict(strides=(64, 1, 64, 1, 63, 1)), INV), (dict(c=0), INV), (dict(a=0), INV), (dict(b=0), INV),
    (dict(a=FAKE + 1), ALI), (dict(c=FAKE + 1), ALI), (dict(ct=ts.TS_F32, c=FAKE + 2), ALI),
    (dict(epi=dict(activation=5)), INV), (dict(epi=dict(activation=-1)), INV), (dict(epi=dict(grad=2)), INV),
    (dict(epi=dict(grad=1)), INV),                                                # no preact to read
    (dict(epi=dict(grad=1, preact=FAKE, stride_pm=64, residual=FAKE, stride_rm=64)), INV),
    (dict(epi=dict(grad=1, preact=FAKE, stride_pm=64, bias=FAKE, bias_dtype=1)), INV),
    (dict(epi=dict(bias=FAKE)), INV), (dict(epi=dict(bias=FAKE, bias_dtype=ts.TS_E4M3)), INV),
    (dict(epi=dict(residual=FAKE, stride_rm=63)), INV), (dict(epi=dict(preact=FAKE, stride_pm=0)), INV),
    (dict(c=FAKE + 256, epi=dict(preact=FAKE + 256, stride_pm=64)), INV),         # preact in C's place
    (dict(epi=dict(preact=FAKE + 512, stride_pm=64, residual=FAKE + 512, stride_rm=64)), INV),
    (dict(epi=dict(scale_a=FAKE)), INV),                                          # scales with 16-bit operands
    (dict(epi=dict(bias=FAKE + 1, bias_dtype=1)), ALI), (dict(epi=dict(residual=FAKE + 1, stride_rm=64)), ALI),
    (dict(ab=ts.TS_E4M3, ct=ts.TS_F32, strides=(64, 1, 1, 64, 64, 1), epi=dict(scale_b=FAKE + 2)), ALI),
    (dict(sched=ts.Schedule(tile="64x64x32")), UNS), (dict(sched=ts.Schedule(tile="256x256x64pp")), UNS),
    (dict(sched=ts.Schedule(order="grouped", group_m=0)), INV), (dict(sched=ts.Schedule(num_programs=-1)), INV),
    (dict(wb=-1), INV),
    (dict(K=65, strides=(65, 1, 64, 1, 64, 1)), INV),                             # packing without a workspace
    (dict(K=65, strides=(65, 1, 64, 1, 64, 1), ws=FAKE + 16, wb=1 << 30), INV),   # misaligned workspace
    (dict(K=1 << 23, strides=(1 << 23, 1, 64, 1, 64, 1)), UNS),                   # rows beyond the in-tile offsets
    (dict(M=512, N=512, K=512, strides=(512, 1, 512, 1, 512, 1),
          sched=ts.Schedule(mode="streamk", num_programs=7)), INV),               # stream-K without a workspace
])
def test_epilogue_refusals(kw, expect):
    got = epilogue(**kw)
    assert got == expect, (ts.status_string(got), kw)


def test_workspace_sizes():
    def need(M, N, K, strides, ab=ts.TS_F16, a=FAKE, b=FAKE, sched=None):
        return ts._lib.ts_gemm_epilogue_workspace(a, b, M, N, K, *strides, ab, ab if ab < 4 else 2,
                                                  ctypes.byref(sched._c()) if sched else None)

    up = lambda v: -(-v // 256) * 256
    assert need(100, 64, 64, (64, 1, 64, 1)) == 0
    assert need(100, 65, 64, (64, 1, 65, 1)) == up(64 * 144)              # odd rows of B: 65 -> 72 elements
    assert need(100, 64, 65, (65, 1, 64, 1)) == up(100 * 144)             # K = 65: A's rows padded to 72
    assert need(100, 64, 65, (65, 1, 1, 65)) == up(100 * 144) + up(64 * 144)
    assert need(100, 64, 65, (1, 100, 64, 1)) == 0                        # stored along M and N: any K
    assert need(100, 64, 64, (64, 1, 64, 1), a=FAKE + 2) == up(100 * 128)
    assert need(100, 64, 100, (100, 1, 1, 100), ab=ts.TS_E4M3) == up(100 * 112) + up(64 * 112)
    assert need(0, 64, 65, (65, 1, 64, 1)) == 0
    assert need(100, 64, 64, (32, 1, 64, 1)) == INV
    # K split among programs: fp32 sums of whole tiles in front of packed operands
    assert need(100, 64, 1024, (1024, 1, 64, 1)) == 2 * 128 * 128 * 4
    assert need(100, 64, 1024, (1025, 1, 64, 1)) == 2 * 128 * 128 * 4 + up(100 * 2048)
    assert need(130, 300, 16384, (16384, 1, 300, 1)) == 32 * 6 * 128 * 128 * 4
    assert need(32, 300, 16384, (16384, 1, 1, 16384)) == 0                # few rows, B [N][K]
    assert need(32, 300, 4088, (4088, 1, 300, 1)) == 0                    # and [K][N]
    assert need(32, 300, 4096, (4096, 1, 300, 1)) > 0 and need(16, 300, 4096, (4096, 1, 300, 1)) == 0
    assert need(100, 64, 1024, (1024, 1, 64, 1), sched=ts.Schedule(tile="128x128x64")) == 0
    sk = ts.Schedule(mode="streamk", num_programs=7, tile="128x128x64")
    assert need(512, 512, 512, (512, 1, 512, 1), sched=sk) == 256 + 7 * 128 * 128 * 4


def test_empty_outputs_are_no_ops():
    assert epilogue(M=0) == ts.TS_OK and epilogue(N=0, strides=(64, 1, 0, 1, 0, 1)) == ts.TS_OK
    assert ts._lib.ts_rmsnorm(None, None, None, None, None, None, 0, 8, 8, 8, 8, 8, 1, 1, 1, 1e-6, None) == ts.TS_OK
    assert ts._lib.ts_act_grad(None, None, None, None, 0, 8, 8, 8, 8, 1, 1, 3, 0, None, None, 0) == ts.TS_OK


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(strides=(64, 1, 1, 64, 64, 1)), dict(strides=(1, 64, 64, 1, 64, 1)), dict(strides=(1, 64, 1, 64, 64, 1)),
    dict(K=0), dict(M=1, strides=(0, 1, 64, 1, 0, 1)), dict(K=1, strides=(1, 1, 64, 1, 64, 1)),
    dict(ab=ts.TS_E4M3, ct=ts.TS_BF16, strides=(64, 1, 1, 64, 64, 1), epi=dict(scale_a=FAKE, scale_b=FAKE)),
    dict(epi=dict(activation=3, bias=FAKE, bias_dtype=3, residual=FAKE, stride_rm=64, preact=FAKE + 65536, stride_pm=64)),
    dict(K=65, strides=(65, 1, 64, 1, 64, 1), ws=FAKE, wb=1 << 20),
    dict(M=512, N=512, K=512, strides=(512, 1, 512, 1, 512, 1), sched=ts.Schedule(mode="streamk", num_programs=7),
         ws=FAKE, wb=1 << 24),
])
def test_valid_epilogues_reach_the_device(kw):
    got = epilogue(**kw)
    assert got == DEV, ts.status_string(got)


def norm(x=FAKE, res=None, w=FAKE, y=FAKE, h=None, s=None, M=4, N=64, ld=(64, 64, 64, 64), t=(1, 1, 1), eps=1e-6):
    return ts._lib.ts_rmsnorm(x, res, w, y, h, s, M, N, *ld, *t, eps, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(N=1 << 31), UNS), (dict(t=(4, 1, 4)), INV), (dict(t=(1, 4, 1)), INV), (dict(t=(1, 1, 0)), INV),
    (dict(t=(1, 1, 3)), UNS), (dict(t=(1, 2, 1)), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(x=0), INV), (dict(y=0), INV), (dict(res=FAKE), INV), (dict(h=FAKE), INV),
    (dict(t=(1, 1, 4)), INV), (dict(ld=(63, 64, 64, 64)), INV), (dict(ld=(64, 64, 0, 64)), INV),
    (dict(res=FAKE, h=FAKE, ld=(64, 60, 64, 64)), INV), (dict(x=FAKE + 1), ALI), (dict(w=FAKE + 1), ALI),
    (dict(t=(1, 1, 4), s=FAKE + 2), ALI)])
def test_norm_refusals(kw, expect):
    assert norm(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(t=(4, 1)), INV), (dict(t=(1, 2)), UNS), (dict(dx=0), INV), (dict(ws=None), INV),
    (dict(wb=64), INV), (dict(ws=FAKE + 16), INV), (dict(ld=(64, 64, 63, 64)), INV), (dict(h=FAKE + 1), ALI),
    (dict(eps=-1.0), INV)])
def test_norm_backward_refusals(kw, expect):
    def call(M=4, N=64, dy=FAKE, h=FAKE, w=FAKE, dh=FAKE, dx=FAKE, dw=FAKE, ld=(64, 64, 64, 64), t=(1, 1), eps=1e-6,
             ws=FAKE, wb=1 << 24):
        return ts._lib.ts_rmsnorm_backward(dy, h, w, dh, dx, dw, M, N, *ld, *t, eps, None, ws, wb)

    assert call(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(t=(4, 1, 3)), INV), (dict(t=(1, 2, 3)), UNS), (dict(t=(1, 1, 0)), INV), (dict(act=5), INV),
    (dict(dc=0), INV), (dict(z=0), INV), (dict(ws=None), INV), (dict(wb=8), INV), (dict(ld=(63, 64, 64)), INV),
    (dict(ld=(64, 64, 63)), INV), (dict(dz=FAKE + 1), ALI), (dict(db=FAKE + 2), ALI)])
def test_act_grad_refusals(kw, expect):
    assert ts._lib.ts_act_grad_workspace(16, 64) == 0 and ts._lib.ts_act_grad_workspace(40, 64) == 3 * 64 * 4
    def call(M=40, N=64, dc=FAKE, z=FAKE, dz=FAKE, db=FAKE, ld=(64, 64, 64), t=(1, 1, 3), act=2, ws=FAKE, wb=1 << 24):
        return ts._lib.ts_act_grad(dc, z, dz, db, M, N, *ld, *t, act, None, ws, wb)

    assert call(**kw) == expect


def test_python_refusals_need_no_gpu():
    a, b = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8, 6, dtype=torch.float16)
    with pytest.raises(ValueError, match="multiply"):
        ts.gemm_epilogue(a, a)
    with pytest.raises(ValueError, match="GPU"):
        ts.gemm_epilogue(a, b)
    with pytest.raises(ValueError, match="activation"):
        ts.gemm_epilogue(a, b, activation="tanh")
    with pytest.raises(ValueError, match="expected torch.float8"):
        ts.gemm_scaled(a, b)
    with pytest.raises(ValueError, match="preact"):
        ts.act_grad(a, None, "gelu")
    with pytest.raises(ValueError, match="gradient of"):
        ts.gemm_epilogue_backward(a, a, b)
    with pytest.raises(ValueError, match="GPU"):
        ts.rmsnorm(a)
    with pytest.raises(ValueError, match="residual"):
        ts.rmsnorm(a, h=a)


def test_header_states_every_activation():
    import os

    text = open(os.path.join(os.path.dirname(ts.__file__), "..", "include", "tsgemm.h")).read()
    codes = {n.lower(): int(v) for n, v in re.findall(r"TS_ACT_([A-Z_]+) = (\d)", text)}
    assert codes == ts.ACTIVATIONS
