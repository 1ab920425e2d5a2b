"""Layer norm, int8 products, rows in 8 bits on the CPU: every refusal comes before any HIP call, and
valid calls reach the device check."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

import tile_scheduling_amd as ts
from tests.test_operators_abi_cpu import ALI, DEV, FAKE, INV, UNS, epilogue, no_gpu

I8, Q8 = ts.TS_I8, ts.TS_Q8
NT = (64, 1, 1, 64, 64, 1)   # A [M][K], B [N][K]


def layernorm(x=FAKE, res=None, w=FAKE, b=FAKE, y=FAKE, h=None, s=None, kept=None, M=4, N=64, ld=(64, 64, 64, 64, 80),
              t=(1, 1, 1), eps=1e-5):
    return ts._lib.ts_layernorm(x, res, w, b, y, h, s, kept, M, N, *ld, *t, eps, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(N=1 << 31), UNS), (dict(t=(4, 1, 4)), INV), (dict(t=(1, 4, 1)), INV), (dict(t=(1, 1, 0)), INV),
    (dict(t=(1, 1, Q8)), INV), (dict(t=(I8, 1, I8)), INV), (dict(t=(1, 1, 3)), UNS), (dict(t=(1, 2, 1)), UNS),
    (dict(w=None, t=(1, 2, 1)), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(x=0), INV), (dict(y=0), INV), (dict(res=FAKE), INV), (dict(h=FAKE), INV),
    (dict(t=(1, 1, 4)), INV), (dict(t=(1, 1, I8)), INV), (dict(ld=(63, 64, 64, 64, 80)), INV),
    (dict(ld=(64, 64, 0, 64, 80)), INV), (dict(res=FAKE, h=FAKE, ld=(64, 60, 64, 64, 80)), INV),
    (dict(x=FAKE + 1), ALI), (dict(w=FAKE + 1), ALI), (dict(b=FAKE + 1), ALI), (dict(t=(1, 1, I8), s=FAKE + 2), ALI),
    (dict(kept=FAKE + 4096 + 8), ALI), (dict(kept=FAKE + 4096, ld=(64, 64, 64, 64, 64)), INV),
    (dict(kept=FAKE + 4096, ld=(64, 64, 64, 64, 72)), INV), (dict(kept=FAKE, x=FAKE), INV),
    (dict(y=FAKE + 512, res=FAKE + 512, h=FAKE + 512), INV),                        # y on h
    (dict(t=(1, 1, I8), s=FAKE, y=FAKE), INV),                                      # codes on x
    (dict(ld=(64, 64, 72, 64, 80)), INV)])                                          # y on x with another row stride
def test_layernorm_refusals(kw, expect):
    assert layernorm(**kw) == expect


def layernorm_backward(M=4, N=64, dy=FAKE, h=FAKE, w=FAKE, dh=FAKE, dx=FAKE, dw=FAKE, db=FAKE + 1024, ld=(64, 64, 64, 64),
                       t=(1, 1, 1), eps=1e-5, ws=FAKE, wb=1 << 24):
    return ts._lib.ts_layernorm_backward(dy, h, w, dh, dx, dw, db, M, N, *ld, *t, eps, None, ws, wb)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(N=1 << 25, ld=(1 << 26,) * 4), UNS), (dict(t=(4, 4, 1)), INV), (dict(t=(1, 2, 1)), INV), (dict(t=(1, 1, 2)), UNS), (dict(dx=0), INV),
    (dict(ws=None), INV), (dict(wb=64), INV), (dict(ws=FAKE + 16), INV), (dict(ld=(64, 64, 63, 64)), INV),
    (dict(h=FAKE + 1), ALI), (dict(db=FAKE + 1), ALI), (dict(eps=-1.0), INV), (dict(db=FAKE), INV), (dict(wb=-1), INV),
    (dict(t=(1, Q8, 1), h=FAKE + 4096), INV),                                       # rows of 64 bytes for 64 columns
    (dict(t=(1, Q8, 1), h=FAKE + 4096, ld=(64, 72, 64, 64)), INV), (dict(t=(1, Q8, 1), h=FAKE + 8, ld=(64, 80, 64, 64)), ALI),
    (dict(t=(1, Q8, 1), ld=(64, 80, 64, 64)), INV)])                                # dx on the kept rows
def test_layernorm_backward_refusals(kw, expect):
    assert layernorm_backward(**kw) == expect


def test_layernorm_backward_workspace():
    need = ts._lib.ts_layernorm_backward_workspace
    assert need(0, 64) == 0 and need(4, 0) == 0 and need(-1, 4) == INV
    assert need(1, 100) == 1024                                  # one workgroup: two rows of 100 fp32
    assert need(3, 16384) == 3 * 2 * 16384 * 4 and need(8192, 4096) == 512 * 2 * 4096 * 4
    assert need(70, 16385) == 2 * 2 * 16385 * 4 // 256 * 256 + 256 + 70 * 16   # long rows: groups of 64, four numbers a row


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(N=1 << 31), UNS), (dict(t=(4, I8)), INV), (dict(t=(1, 1)), INV), (dict(t=(1, Q8)), INV),
    (dict(x=0), INV), (dict(y=0), INV), (dict(s=0), INV), (dict(x=FAKE), INV), (dict(ld=(63, 64)), INV),
    (dict(ld=(64, 63)), INV), (dict(x=FAKE + 513), ALI), (dict(s=FAKE + 2), ALI)])
def test_quantize_rows_refusals(kw, expect):
    def call(x=FAKE + 512, y=FAKE, s=FAKE + 1024, M=4, N=64, ld=(64, 64), t=(1, I8)):
        return ts._lib.ts_quantize_rows(x, y, s, M, N, *ld, *t, None)

    assert call(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INV), (dict(N=1 << 31), UNS), (dict(t=4), INV), (dict(x=0), INV), (dict(kept=0), INV),
    (dict(kept=FAKE + 8), ALI), (dict(x=FAKE + 4097), ALI), (dict(ld=(63, 80)), INV), (dict(ld=(64, 65)), INV),
    (dict(ld=(64, 74)), INV), (dict(x=FAKE), INV)])
def test_checkpoint_refusals(kw, expect):
    def call(x=FAKE + 4096, kept=FAKE, M=4, N=64, ld=(64, 80), t=1):
        pack = ts._lib.ts_checkpoint_pack(x, kept, M, N, *ld, t, None)
        unpack = ts._lib.ts_checkpoint_unpack(kept, x, M, N, ld[1], ld[0], t, 2, None)
        assert pack == unpack
        return pack

    assert call(**kw) == expect


def test_checkpoint_rows():
    size = ts._lib.ts_checkpoint_row_bytes
    assert [size(n) for n in (0, 1, 32, 33, 64, 4096)] == [0, 48, 48, 80, 80, 4096 + 128]
    assert size(-1) == INV and size(1 << 26) == UNS
    assert ts._lib.ts_checkpoint_unpack(FAKE, FAKE + 4096, 4, 64, 80, 64, 1, 5, None) == INV   # no such activation
    for m, n in ((1, 1), (3, 32), (5, 33), (2, 4096)):
        c = ts.Checkpoint.empty(m, n, "cpu")
        assert c.shape == (m, n) and c.data.shape[1] % 64 == 0 and c.data.shape[1] >= size(n) - 15


def test_checkpoint_checks_its_data():
    good = torch.zeros(4, 128, dtype=torch.uint8)
    assert ts.Checkpoint(good, 64).shape == (4, 64)
    assert ts.Checkpoint(good[1:3], 64).shape == (2, 64)         # rows of a checkpoint are one
    for bad, n in ((good.int(), 64), (good[0], 64), (good, 128), (good[:, ::2], 32), (good[:, 8:], 32), (good[:, :66].contiguous(), 64),
                   (good, -1)):
        with pytest.raises(ValueError):
            ts.Checkpoint(bad, n)


KEPT = dict(preact=FAKE + (1 << 20), stride_pm=80, preact_dtype=Q8)


@pytest.mark.parametrize("kw,expect", [
    (dict(ab=I8, ct=ts.TS_BF16), UNS),                                              # B stored [K][N]
    (dict(ab=I8, ct=ts.TS_BF16, strides=(1, 64, 1, 64, 64, 1)), UNS),               # A stored [K][M]
    (dict(ab=I8, ct=I8, strides=NT), UNS), (dict(ab=Q8, ct=ts.TS_F32), INV), (dict(ct=Q8), INV),
    (dict(ab=I8, ct=ts.TS_F32, K=1 << 17, strides=(1 << 17, 1, 1, 1 << 17, 64, 1)), UNS),
    (dict(ab=I8, ct=ts.TS_F32, strides=NT, epi=dict(scale_b=FAKE + 2)), ALI),
    (dict(epi=dict(KEPT, preact_dtype=ts.TS_F32)), INV), (dict(epi=dict(KEPT, preact_dtype=7)), INV),
    (dict(epi=dict(KEPT, stride_pm=64)), INV), (dict(epi=dict(KEPT, stride_pm=88)), INV),
    (dict(epi=dict(KEPT, preact=FAKE + 8)), ALI), (dict(c=FAKE + (1 << 20), epi=KEPT), INV),
    (dict(c=FAKE + (1 << 20), epi=dict(KEPT, grad=1)), INV),
    (dict(ab=I8, ct=ts.TS_BF16, strides=NT, epi=KEPT), UNS), (dict(ab=ts.TS_E4M3, ct=ts.TS_BF16, strides=NT, epi=KEPT), UNS),
    (dict(M=512, N=512, K=512, strides=(512, 1, 512, 1, 512, 1), sched=ts.Schedule(mode="streamk", num_programs=7), ws=FAKE,
          wb=1 << 24, epi=dict(KEPT, stride_pm=528)), UNS)])
def test_epilogue_refusals(kw, expect):
    got = epilogue(**kw)
    assert got == expect, (ts.status_string(got), kw)


@pytest.mark.parametrize("kw,expect", [
    (dict(t=(1, 2, 1, 3)), INV), (dict(t=(1, Q8, 2, 3)), UNS), (dict(z=0), INV), (dict(act=0, z=0), INV), (dict(act=5), INV),
    (dict(v=FAKE, dz=FAKE), INV), (dict(v=FAKE + 1), ALI), (dict(ld=(64, 80, 64, 63)), INV), (dict(ld=(64, 64, 64, 64)), INV),
    (dict(ld=(64, 88, 64, 64)), INV), (dict(z=FAKE + 8), ALI), (dict(v=FAKE + (1 << 16)), INV), (dict(ws=None), INV)])
def test_act_grad_value_refusals(kw, expect):
    def call(M=40, N=64, dc=FAKE, z=FAKE + (1 << 16), dz=FAKE, v=FAKE + 4096 * 8, db=FAKE, ld=(64, 80, 64, 64),
             t=(1, Q8, 1, 3), act=2, ws=FAKE, wb=1 << 24):
        return ts._lib.ts_act_grad_value(dc, z, dz, v, db, M, N, *ld, *t, act, None, ws, wb)

    assert call(**kw) == expect


def test_empty_matrices_are_no_ops():
    assert layernorm(M=0) == ts.TS_OK and layernorm(N=0) == ts.TS_OK
    assert layernorm_backward(M=0, dw=None, db=None) == ts.TS_OK and layernorm_backward(N=0) == ts.TS_OK
    assert ts._lib.ts_quantize_rows(None, None, None, 0, 8, 8, 8, 1, I8, None) == ts.TS_OK
    assert ts._lib.ts_quantize_rows(None, None, None, 4, 0, 0, 0, 1, I8, None) == INV   # a place for the scales
    assert ts._lib.ts_checkpoint_pack(None, None, 0, 8, 8, 48, 1, None) == ts.TS_OK
    assert ts._lib.ts_checkpoint_unpack(None, None, 8, 0, 48, 8, 1, 0, None) == ts.TS_OK


@no_gpu
def test_valid_calls_reach_the_device():
    for t in ((1, 1, 1), (2, 3, 4), (3, 3, I8)):
        assert layernorm(t=t, s=FAKE, y=FAKE + 8192, kept=FAKE + 16384) == DEV
        assert layernorm(t=t, s=FAKE, y=FAKE + 8192, res=FAKE + 4096, h=FAKE, w=None) == DEV
    assert layernorm_backward() == DEV and layernorm_backward(w=None, dw=None, dh=None) == DEV
    assert layernorm_backward(t=(2, Q8, 3), h=FAKE + 4096, ld=(64, 80, 64, 64)) == DEV
    assert layernorm_backward(M=0) == DEV   # the sums of no rows
    assert ts._lib.ts_quantize_rows(FAKE, FAKE + 4096, FAKE, 4, 64, 64, 64, 2, I8, None) == DEV
    assert ts._lib.ts_checkpoint_pack(FAKE, FAKE + 4096, 4, 64, 64, 80, 2, None) == DEV
    for s, epi in ((NT, dict(scale_a=FAKE, scale_b=FAKE)), (NT, None)):
        assert epilogue(ab=I8, ct=ts.TS_BF16, strides=s, epi=epi) == DEV
    assert epilogue(ab=I8, ct=ts.TS_F32, K=(1 << 17) - 16, strides=((1 << 17) - 16, 1, 1, (1 << 17) - 16, 64, 1), ws=FAKE,
                    wb=1 << 30) == DEV
    for s in (NT, (64, 1, 64, 1, 64, 1), (1, 64, 64, 1, 64, 1), (1, 64, 1, 64, 64, 1)):
        for M in (4, 64):
            assert epilogue(M=M, strides=s, epi=dict(KEPT, activation=2)) == DEV
            assert epilogue(M=M, strides=s, epi=dict(KEPT, activation=2, grad=1)) == DEV


def test_workspace_of_int8():
    def need(M, N, K, ld=None, ab=I8, a=FAKE, b=FAKE):
        ld = ld or K
        return ts._lib.ts_gemm_epilogue_workspace(a, b, M, N, K, ld, 1, 1, ld, ab, ts.TS_BF16, None)

    up = lambda v: -(-v // 256) * 256
    for M, N, K in ((4, 64, 64), (200, 64, 64), (200, 64, 2048), (300, 516, 2051)):   # whole chunks, or rows of odd bytes
        assert need(M, N, K) == need(M, N, K, ab=ts.TS_E4M3) >= 0
    # rows of 4-byte words: one operand, that of fewer rows, is copied with zeros behind K
    assert need(200, 160, 100) == up(160 * 112) and need(160, 200, 100) == up(160 * 112)
    assert need(200, 160, 100, ld=112) == up(160 * 112)                 # whatever lies behind K
    assert need(200, 160, 96, ld=100) == 0                              # no chunk reaches behind K
    assert need(200, 160, 102, ld=104) == up(200 * 112) + up(160 * 112)
    assert need(200, 160, 100, a=FAKE + 2) == up(200 * 112) and need(200, 160, 100, b=FAKE + 1) == up(160 * 112)
    # up to 128 rows in one pass over B, as far as that pays
    assert need(128, 64, 2047) == 0 and need(64, 8192, 4095) == 0 and need(32, 9000, 9001) == 0
    assert need(129, 64, 2047) > 0 and need(128, 64, 2051) > 0 and need(65, 64, 4095) > 0 and need(64, 8193, 4095) > 0


def test_python_refusals_need_no_gpu():
    a = torch.zeros(4, 8, dtype=torch.float16)
    q = torch.zeros(4, 8, dtype=torch.int8)
    c = ts.Checkpoint.empty(4, 8, "cpu")
    with pytest.raises(ValueError, match="GPU"):
        ts.layernorm(a)
    with pytest.raises(ValueError, match="residual"):
        ts.layernorm(a, h=a)
    with pytest.raises(ValueError, match="GPU"):
        ts.layernorm_backward(a, c)
    with pytest.raises(ValueError, match="GPU"):
        ts.quantize_rows(a)
    with pytest.raises(ValueError, match="GPU"):
        ts.checkpoint_pack(a)
    with pytest.raises(ValueError, match="GPU"):
        ts.checkpoint_unpack(c)
    with pytest.raises(ValueError, match="GPU"):
        ts.gemm_scaled(q, q.t())
    with pytest.raises(ValueError, match="expected torch.float8"):
        ts.gemm_scaled(torch.zeros(4, 8, dtype=torch.uint8), q.t())
    with pytest.raises(ValueError, match="A is"):
        ts.gemm_scaled(q, a.t())
    with pytest.raises(ValueError, match="preact"):
        ts.act_grad(a, None, "none", act_out=a)
    with pytest.raises(ValueError, match="shape"):
        ts.act_grad(a, ts.Checkpoint.empty(4, 9, "cpu"), "gelu")
    for bad in (torch.zeros(8), torch.zeros(2, 2, 2)):
        for f in (ts.layernorm, ts.quantize_rows, ts.checkpoint_pack):
            with pytest.raises(ValueError, match="matrix"):
                f(bad)


def test_arguments_of_other_types():
    a = torch.zeros(4, 8, dtype=torch.float16)
    for f in (ts.layernorm, ts.rmsnorm, ts.quantize_rows, ts.checkpoint_pack):
        with pytest.raises(TypeError, match="tensor"):
            f("rows")
    with pytest.raises(TypeError, match="dtype"):
        ts.layernorm(a, out_dtype="int8")
    with pytest.raises(TypeError, match="tensor"):
        ts.gemm_epilogue(a, [1, 2])
    with pytest.raises(TypeError, match="eps"):
        ts.layernorm(a, eps="small")
    with pytest.raises(TypeError, match="tensor"):
        ts.act_grad(a, 3, "gelu")


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(ts._Epilogue) == 4 * 4 + 7 * 8   # four int32, seven pointers and strides


def test_arguments_without_a_truth():
    # the caller's own error comes back, before anything else happens
    class Unsure:
        def __bool__(self):
            raise KeyError("no truth")

    a = torch.zeros(4, 8, dtype=torch.float16)
    for call in (lambda: ts.act_grad(a, dbias=Unsure()), lambda: ts.act_grad(a, dbias=torch.ones(2)),
                 lambda: ts.rmsnorm_backward(a, a, a[0], dweight=Unsure()), lambda: ts.layernorm_backward(a, a, a[0], dweight=Unsure()),
                 lambda: ts.layernorm_backward(a, a, dbias=Unsure())):
        with pytest.raises((KeyError, RuntimeError), match="no truth|ambiguous"):
            call()


def test_a_checkpoint_changed_after_its_checks():
    # data and n can be set anew: every call looks at them again
    a, w = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(64, 64, dtype=torch.float16)

    def changed(**kw):
        k = ts.Checkpoint.empty(4, 64, "cpu")
        for name, v in kw.items():
            setattr(k, name, v)
        return k

    def calls(k):
        return (lambda: ts.checkpoint_unpack(k), lambda: ts.checkpoint_pack(a, k), lambda: ts.act_grad(a, k, "gelu"),
                lambda: ts.layernorm(a, keep=k), lambda: ts.layernorm_backward(a, k), lambda: ts.rmsnorm_backward(a, k),
                lambda: ts.gemm_epilogue(a, w, preact=k), lambda: ts.gemm_dact(a, w, k, "gelu"),
                lambda: ts.gemm_epilogue_backward(a, k, w))

    good = ts.Checkpoint.empty(4, 64, "cpu").data
    for k in (changed(data=good[:, :48]), changed(data=good.int()), changed(data=good[0]), changed(data=good.t()),
              changed(data=torch.zeros(256, 4, dtype=torch.uint8).t()), changed(data=good.unsqueeze(0))):
        for call in calls(k):
            with pytest.raises(ValueError, match="checkpoint's"):
                call()
    big = torch.zeros(4, 4096, dtype=torch.float16)
    for call in (lambda k: ts.checkpoint_unpack(k), lambda k: ts.checkpoint_pack(big, k), lambda k: ts.act_grad(big, k, "gelu"),
                 lambda k: ts.layernorm_backward(big, k)):
        with pytest.raises(ValueError, match="checkpoint's"):
            call(changed(n=4096))
    for call in (lambda: ts.checkpoint_unpack(changed(n=-1)), lambda: ts.checkpoint_unpack(changed(n=1 << 62))):
        with pytest.raises(ValueError, match="checkpoint's"):
            call()


@pytest.mark.parametrize("module,reason", [(None, "_binding"), ("built_for = 'torch 1.0, Python 2.7'\n", "torch 1.0"),
                                           ("raise ImportError('undefined symbol')\n", "undefined symbol")])
def test_package_without_a_fitting_binding(tmp_path, module, reason):
    # the product and its schedules need the library alone; the operators' calls say what is missing
    package = tmp_path / "tile_scheduling_amd"
    package.mkdir()
    here = os.path.dirname(ts.__file__)
    shutil.copy(os.path.join(here, "__init__.py"), package)
    os.symlink(os.path.join(here, "libtsgemm.so"), package / "libtsgemm.so")
    if module:
        (package / "_binding.py").write_text(module)
    code = f"""
import torch, tile_scheduling_amd as ts
assert ts.schedule_trace_host(256, 256, 256, ts.Schedule(), 4, 1).shape[1] == 5
a = torch.zeros(4, 8)
for call in (lambda: ts.layernorm(a), lambda: ts.gemm_epilogue(a, a.t()), lambda: ts.checkpoint_pack(a)):
    try:
        call()
    except ImportError as e:
        assert {reason!r} in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no error")
print("ended")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ended" in r.stdout, r.stderr
