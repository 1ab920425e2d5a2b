"""The operators around the product at the edges of what their contract allows, without a GPU."""
import ctypes

import pytest
import torch

import tile_scheduling_amd as ts

FAKE = 0x10000   # 256-byte aligned, never dereferenced: every call below ends before a launch
INV, DEV = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_NO_DEVICE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


@pytest.mark.parametrize("M", [0, 1, 4, 40, 1 << 20])
def test_act_grad_of_no_columns(M):
    assert ts._lib.ts_act_grad_workspace(M, 0) == 0
    for t, act in ((ts.TS_F16, 0), (ts.TS_BF16, 2), (ts.TS_F32, 4)):
        assert ts._lib.ts_act_grad(FAKE, FAKE, FAKE, FAKE, M, 0, 0, 0, 0, t, t, t, act, None, None, 0) == ts.TS_OK
        assert ts._lib.ts_act_grad(None, None, None, None, M, 0, 0, 0, 0, t, t, t, act, None, None, 0) == ts.TS_OK


def norm_of_no_columns(M, y_dtype, scale):
    return ts._lib.ts_rmsnorm(None, None, None, None, None, scale, M, 0, 0, 0, 0, 0, ts.TS_BF16, ts.TS_BF16, y_dtype, 1e-6, None)


def test_norm_of_no_columns_needs_a_place_for_its_scales():
    assert norm_of_no_columns(4, ts.TS_E4M3, None) == INV
    assert norm_of_no_columns(0, ts.TS_E4M3, None) == ts.TS_OK
    assert norm_of_no_columns(4, ts.TS_BF16, None) == ts.TS_OK


@no_gpu
def test_norm_of_no_columns_writes_its_scales():
    assert norm_of_no_columns(4, ts.TS_E4M3, FAKE) == DEV   # not TS_OK without a launch


# An output in an input's place: element on element, or refused.  (On another type or row stride an
# element would be overwritten before its own thread has read it.)

def product_in_place(preact=None, residual=None, ld_in=64, ldc=64, grad=0, M=40):
    e = ts._Epilogue(activation=2, grad=grad, residual=residual, stride_rm=ld_in, preact=preact, stride_pm=ld_in)
    return ts._lib.ts_gemm_epilogue(FAKE, FAKE, FAKE + 4096, M, 64, 64, 64, 1, 64, 1, ldc, 1, ts.TS_F16, ts.TS_F32,
                                    ctypes.byref(e), None, None, None, 0)


def test_product_in_place_needs_one_row_stride():
    assert product_in_place(residual=FAKE + 4096, ld_in=128) == INV
    assert product_in_place(preact=FAKE + 4096, ld_in=128, grad=1) == INV
    assert product_in_place(preact=FAKE + 4096, ldc=128, grad=1, M=200) == INV


@no_gpu
def test_product_in_place():
    assert product_in_place(residual=FAKE + 4096) == DEV
    assert product_in_place(preact=FAKE + 4096, grad=1) == DEV
    assert product_in_place(residual=FAKE + 4096, ld_in=128, M=1) == DEV
    assert product_in_place(residual=FAKE + 65536, ld_in=128) == DEV


def act_grad_in_place(dz=FAKE, z=FAKE + 65536, ld=(64, 64, 64), t=(3, 3), M=40):
    return ts._lib.ts_act_grad(FAKE, z, dz, None, M, 64, *ld, *t, 3, 2, None, None, 0)


def test_act_grad_in_place_needs_one_type_and_row_stride():
    for dz in (FAKE, FAKE + 65536):   # in dC's place, in preact's
        assert act_grad_in_place(dz, t=(ts.TS_F32, ts.TS_BF16)) == INV
        assert act_grad_in_place(dz, t=(ts.TS_F32, ts.TS_F16)) == INV
        assert act_grad_in_place(dz, ld=(64, 64, 128)) == INV


@no_gpu
def test_act_grad_in_place():
    for dz in (FAKE, FAKE + 65536):
        assert act_grad_in_place(dz) == DEV
        assert act_grad_in_place(dz, ld=(64, 64, 128), M=1) == DEV
    assert act_grad_in_place(FAKE + 131072, t=(ts.TS_F32, ts.TS_BF16), ld=(64, 128, 192)) == DEV


def norm_in_place(res=None, y=FAKE + 65536, h=None, s=None, ld=(64, 64, 64, 64), t=(2, 2, 2), M=4):
    return ts._lib.ts_rmsnorm(FAKE, res, None, y, h, s, M, 64, *ld, *t, 1e-6, None)


def test_norm_in_place_needs_one_type_and_row_stride():
    r = FAKE + 4096
    assert norm_in_place(r, FAKE + 65536, FAKE + 65536) == INV                 # y and h on each other
    assert norm_in_place(r, FAKE, FAKE) == INV
    assert norm_in_place(y=FAKE, t=(2, 2, 4), s=FAKE + 8192) == INV            # e4m3 over 16 bits
    assert norm_in_place(r, r, FAKE, t=(2, 2, 4), s=FAKE + 8192) == INV
    assert norm_in_place(y=FAKE, ld=(64, 64, 128, 64)) == INV
    assert norm_in_place(r, h=r, ld=(64, 64, 64, 128)) == INV
    assert norm_in_place(r, h=FAKE, ld=(128, 64, 64, 64)) == INV


@no_gpu
def test_norm_in_place():
    r = FAKE + 4096
    assert norm_in_place(y=FAKE) == DEV and norm_in_place(r, r, FAKE) == DEV and norm_in_place(r, FAKE, r) == DEV
    assert norm_in_place(r, FAKE, r, ld=(128, 64, 128, 64)) == DEV
    assert norm_in_place(r, FAKE + 65536, r, t=(2, 2, 4), s=FAKE + 8192) == DEV


def norm_grad_in_place(dx, ld=(64, 64, 64, 64), M=4):
    return ts._lib.ts_rmsnorm_backward(FAKE, FAKE + 4096, None, FAKE + 8192, dx, None, M, 64, *ld, 2, 2, 1e-6, None, None, 0)


def test_norm_gradient_in_place_needs_one_row_stride():
    for dx in (FAKE, FAKE + 4096, FAKE + 8192):
        assert norm_grad_in_place(dx, ld=(64, 64, 64, 128)) == INV


@no_gpu
def test_norm_gradient_in_place():
    for dx in (FAKE, FAKE + 8192, FAKE + 65536):
        assert norm_grad_in_place(dx) == DEV
