"""The operators around the product on the GPU at the edges of what their contract allows: empty
matrices, values at the ends of the types' ranges, infinities, calls that overlap in time.  Against
definitions in 64 bits (bounds derived in operator_reference)."""
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
