"""The operators around the product at the edges of what their contract allows, without a GPU."""
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
