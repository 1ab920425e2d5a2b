"""Python binding of libtsgemm (tiled GEMM with tile-order schedules, MI355X).

Argument marshalling only (ctypes here, the operators' in ``_binding``): every step of
the computation runs in the HIP kernels of ``libtsgemm.so``.  PyTorch supplies device
memory and streams.  Both libraries are built in-tree by ``python
tile_scheduling_amd/build.py``.  Without ``libtsgemm.so`` importing this package raises ImportError,
without a ``_binding`` built for this torch and Python an operator's call does (the product and its
schedules do without); there is no fallback path.

    import torch, tile_scheduling_amd as ts
    c = ts.gemm(a, b, out_dtype=torch.float16,
                schedule=ts.Schedule(order="grouped", group_m=8, mode="persistent"))
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import sys

import torch  # loaded first: libtsgemm binds to the HIP runtime torch already loaded

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtsgemm.so")
_BUILD = f"python {os.path.join(_HERE, 'build.py')}"

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `{_BUILD}`")

_lib = ctypes.CDLL(LIB_PATH)


class _Missing:
    """In _binding's place: every call of an operator says why."""

    def __init__(self, reason):
        self._reason = reason

    def __getattr__(self, name):
        raise ImportError(f"{self._reason}: build the package with `{_BUILD}`")


try:
    from . import _binding   # the operators' calls, checked and made in C++ (csrc/binding.cpp)

    _running = f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"
    _built = getattr(_binding, "built_for", "an earlier version of it")
    if _built != _running:
        _binding = _Missing(f"_binding was built for {_built}, this is {_running}")
except ImportError as e:
    _binding = _Missing(str(e))

_i32, _i64, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p

# status codes, element types and schedule enums (include/tsgemm.h)
TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_ALIGNMENT, TS_ERR_HIP, TS_ERR_NO_DEVICE = 0, -1, -2, -3, -4, -5
TS_F16, TS_BF16, TS_F32, TS_E4M3, TS_I8, TS_Q8 = 1, 2, 3, 4, 5, 6
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ORDERS = {"row_major": 0, "grouped": 1, "auto": 2}
MODES = {"tiled": 0, "persistent": 1, "crosstile": 2, "streamk": 3, "auto": 4}
INDEX_MATH = {"divide": 0, "mulshift": 1}
TILES = {"auto": 0, "64x64x32": 1, "128x128x64": 2, "256x256x64": 3, "256x256x64w8": 4, "256x256x64pp": 5}


class _Schedule(ctypes.Structure):
    _fields_ = [("order", _i32), ("group_m", _i32), ("mode", _i32),
                ("num_programs", _i32), ("xcd_remap", _i32), ("tile_config", _i32), ("index_math", _i32)]


class LaunchInfo(ctypes.Structure):
    _fields_ = [("block_m", _i32), ("block_n", _i32), ("block_k", _i32), ("threads", _i32),
                ("num_m_tiles", _i64), ("num_n_tiles", _i64), ("k_steps", _i64), ("num_tiles", _i64),
                ("grid", _i64), ("programs_per_cu", _i32), ("cu_count", _i32), ("xcds", _i32),
                ("lds_bytes", _i32), ("masked", _i32), ("workspace_bytes", _i64), ("trace_items", _i64),
                ("vgprs", _i32), ("scratch_bytes", _i32),
                ("arch_vgprs", _i32), ("agprs", _i32), ("sgprs", _i32), ("spilled_vgprs", _i32),
                ("spilled_sgprs", _i32), ("compiler_occupancy", _i32),
                ("order", _i32), ("group_m", _i32), ("mode", _i32), ("xcd_remap", _i32), ("index_math", _i32),
                ("model_l2_reuse_pm", _i32)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_lib.ts_gemm.argtypes = [_p, _p, _p] + [_i64] * 9 + [_i32, _i32, ctypes.POINTER(_Schedule), _p]
_lib.ts_gemm.restype = _i32
_lib.ts_gemm_workspace.argtypes = _lib.ts_gemm.argtypes + [_p, _i64]
_lib.ts_gemm_workspace.restype = _i32
_lib.ts_gemm_noalloc.argtypes = list(_lib.ts_gemm.argtypes)
_lib.ts_gemm_noalloc.restype = _i32
_lib.ts_noalloc_scratch_bytes.argtypes = []
_lib.ts_noalloc_scratch_bytes.restype = _i64
_lib.ts_gemm_clocked.argtypes = _lib.ts_gemm.argtypes + [_p, _i64, _p, _i64]
_lib.ts_gemm_clocked.restype = _i32
_lib.ts_mfma_loop_probe.argtypes = [_i32, _p, _i64, ctypes.POINTER(ctypes.c_double), _p]
_lib.ts_mfma_loop_probe.restype = _i32
_lib.ts_mfma_phase_probe.argtypes = [_i32, _i32, _p, _i64, ctypes.POINTER(ctypes.c_double), _p]
_lib.ts_mfma_phase_probe.restype = _i32
_lib.ts_schedule_trace.argtypes = [_i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_Schedule), _p, _i64, _p]
_lib.ts_schedule_trace.restype = _i32
_lib.ts_schedule_trace_host.argtypes = [_i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_Schedule),
                                        _i32, _i32, _p, _i64]
_lib.ts_schedule_trace_host.restype = _i32
_lib.ts_query.argtypes = [_i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_Schedule), ctypes.POINTER(LaunchInfo)]
_lib.ts_query.restype = _i32


class _Epilogue(ctypes.Structure):
    _fields_ = [("activation", _i32), ("grad", _i32), ("bias", _p), ("bias_dtype", _i32), ("preact_dtype", _i32),
                ("residual", _p), ("stride_rm", _i64), ("preact", _p), ("stride_pm", _i64),
                ("scale_a", _p), ("scale_b", _p)]


_lib.ts_gemm_epilogue.argtypes = [_p, _p, _p] + [_i64] * 9 + [_i32, _i32, ctypes.POINTER(_Epilogue),
                                                               ctypes.POINTER(_Schedule), _p, _p, _i64]
_lib.ts_gemm_epilogue.restype = _i32
_lib.ts_gemm_epilogue_workspace.argtypes = [_p, _p] + [_i64] * 7 + [_i32, _i32, ctypes.POINTER(_Schedule)]
_lib.ts_gemm_epilogue_workspace.restype = _i64
_lib.ts_rmsnorm.argtypes = [_p] * 6 + [_i64] * 6 + [_i32] * 3 + [ctypes.c_float, _p]
_lib.ts_rmsnorm.restype = _i32
_lib.ts_rmsnorm_backward.argtypes = [_p] * 6 + [_i64] * 6 + [_i32] * 2 + [ctypes.c_float, _p, _p, _i64]
_lib.ts_rmsnorm_backward.restype = _i32
_lib.ts_rmsnorm_backward_workspace.argtypes = [_i64, _i64]
_lib.ts_rmsnorm_backward_workspace.restype = _i64
_lib.ts_act_grad.argtypes = [_p] * 4 + [_i64] * 5 + [_i32] * 4 + [_p, _p, _i64]
_lib.ts_act_grad.restype = _i32
_lib.ts_act_grad_workspace.argtypes = [_i64, _i64]
_lib.ts_act_grad_workspace.restype = _i64
_lib.ts_act_grad_value.argtypes = [_p] * 5 + [_i64] * 6 + [_i32] * 5 + [_p, _p, _i64]
_lib.ts_act_grad_value.restype = _i32
_lib.ts_layernorm.argtypes = [_p] * 8 + [_i64] * 7 + [_i32] * 3 + [ctypes.c_float, _p]
_lib.ts_layernorm.restype = _i32
_lib.ts_layernorm_backward.argtypes = [_p] * 7 + [_i64] * 6 + [_i32] * 3 + [ctypes.c_float, _p, _p, _i64]
_lib.ts_layernorm_backward.restype = _i32
_lib.ts_layernorm_backward_workspace.argtypes = [_i64, _i64]
_lib.ts_layernorm_backward_workspace.restype = _i64
_lib.ts_quantize_rows.argtypes = [_p] * 3 + [_i64] * 4 + [_i32] * 2 + [_p]
_lib.ts_quantize_rows.restype = _i32
_lib.ts_checkpoint_row_bytes.argtypes = [_i64]
_lib.ts_checkpoint_row_bytes.restype = _i64
_lib.ts_checkpoint_pack.argtypes = [_p] * 2 + [_i64] * 4 + [_i32, _p]
_lib.ts_checkpoint_pack.restype = _i32
_lib.ts_checkpoint_unpack.argtypes = [_p] * 2 + [_i64] * 4 + [_i32] * 2 + [_p]
_lib.ts_checkpoint_unpack.restype = _i32
_lib.ts_status_string.argtypes = [_i32]
_lib.ts_status_string.restype = ctypes.c_char_p

EXPORTS = ("ts_gemm", "ts_gemm_workspace", "ts_gemm_noalloc", "ts_noalloc_scratch_bytes", "ts_gemm_clocked", "ts_schedule_trace", "ts_schedule_trace_host", "ts_query",
           "ts_status_string", "ts_mfma_loop_probe", "ts_mfma_phase_probe", "ts_gemm_epilogue",
           "ts_gemm_epilogue_workspace", "ts_rmsnorm", "ts_rmsnorm_backward", "ts_rmsnorm_backward_workspace",
           "ts_act_grad", "ts_act_grad_workspace", "ts_act_grad_value", "ts_layernorm", "ts_layernorm_backward",
           "ts_layernorm_backward_workspace", "ts_quantize_rows", "ts_checkpoint_row_bytes", "ts_checkpoint_pack",
           "ts_checkpoint_unpack")


class TsError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(status_string(status))


def status_string(status: int) -> str:
    return _lib.ts_status_string(int(status)).decode()


@dataclasses.dataclass(frozen=True)
class Schedule:
    """Tile order and mode of one launch (see ts_schedule in include/tsgemm.h)."""

    order: str = "row_major"      # "row_major" | "grouped" | "auto"
    group_m: int = 8              # GROUP_SIZE_M for the grouped order
    mode: str = "tiled"           # "tiled" | "persistent" | "crosstile" | "streamk" | "auto"
    num_programs: int = 0         # persistent grid; 0 = CUs x workgroups per CU
    xcd_remap: bool = False       # contiguous tile-id runs per XCD
    tile: str = "auto"            # "auto" | "64x64x32" | "128x128x64" | "256x256x64" | "256x256x64w8" | "256x256x64pp"
    index_math: str = "divide"    # "divide" | "mulshift"

    def _c(self) -> _Schedule:
        return _Schedule(ORDERS[self.order], int(self.group_m), MODES[self.mode],
                         int(self.num_programs), 1 if self.xcd_remap else 0, TILES[self.tile],
                         INDEX_MATH[self.index_math])

    def label(self) -> str:
        o = {"row_major": "rowmajor", "auto": "autoorder"}.get(self.order, f"grouped{self.group_m}")
        r = "+remap" if self.xcd_remap and self.order != "auto" else ""
        p = f"/P{self.num_programs}" if self.mode != "tiled" and self.num_programs else ""
        x = "/mulshift" if self.index_math == "mulshift" else ""
        return f"{o}{r}/{self.mode}{p}/{self.tile}{x}"


_TORCH_DTYPE = {torch.float16: TS_F16, torch.bfloat16: TS_BF16, torch.float32: TS_F32}


def _check(status: int):
    if status != TS_OK:
        raise TsError(status)


def _stream_handle(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_WORKSPACES: dict = {}


def workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """A zeroed device workspace of at least ``nbytes`` for ts_gemm_workspace, one per
    device and stream, reused by later calls (every call leaves its flags zero)."""
    key = (device, torch.cuda.current_stream(device).cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


def gemm(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
         out_dtype: torch.dtype | None = None, schedule: Schedule | None = None,
         ws: torch.Tensor | None = None) -> torch.Tensor:
    """C = A @ B with A [M,K], B [K,N] fp16/bf16 CUDA tensors; C fp16/bf16/fp32.

    Enqueued on the current stream of A's device; returns C (``out`` if given).
    A stream-K schedule that splits tiles runs with ``ws`` (a uint8 CUDA tensor
    of at least ``query(...)["workspace_bytes"]`` bytes whose header is zero), or
    with a cached zeroed workspace of the device and stream.
    """
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"shapes {tuple(a.shape)} @ {tuple(b.shape)} do not multiply")
    if not (a.is_cuda and b.is_cuda) or a.device != b.device:
        raise ValueError("A and B must be on the same GPU")
    M, K = a.shape
    N = b.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or a.dtype, device=a.device)
    elif out.shape != (M, N) or out.device != a.device:
        raise ValueError("out has the wrong shape or device")
    sched = schedule or Schedule()
    s = sched._c()
    ab_t, c_t = _TORCH_DTYPE.get(a.dtype, 0), _TORCH_DTYPE.get(out.dtype, 0)
    if sched.mode == "streamk":
        need = query(M, N, K, sched, ab_t, c_t)["workspace_bytes"]
        if ws is None and need > 0:
            ws = workspace(need, a.device)
        wptr, wbytes = (ws.data_ptr(), ws.numel() * ws.element_size()) if ws is not None else (None, 0)
        st = _lib.ts_gemm_workspace(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K,
                                    a.stride(0), a.stride(1), b.stride(0), b.stride(1), out.stride(0),
                                    out.stride(1), ab_t, c_t, ctypes.byref(s), _stream_handle(a.device),
                                    wptr, wbytes)
    else:
        st = _lib.ts_gemm(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K,
                          a.stride(0), a.stride(1), b.stride(0), b.stride(1), out.stride(0), out.stride(1),
                          ab_t, c_t, ctypes.byref(s), _stream_handle(a.device))
    _check(st)
    return out


def gemm_clocked(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor, schedule: Schedule | None = None):
    """ts_gemm_clocked: C = A @ B into ``out`` plus the per-workgroup clock record.

    Returns an int64 [grid, 4] CUDA tensor (shader-clock counter at start and end,
    100 MHz counter at start and end of every workgroup); use ``clock_ghz`` on it.
    """
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0] or out.shape != (a.shape[0], b.shape[1]):
        raise ValueError("shapes do not multiply")
    M, K = a.shape
    N = b.shape[1]
    sched = schedule or Schedule()
    grid = query(M, N, K, sched, _TORCH_DTYPE.get(a.dtype, 0), _TORCH_DTYPE.get(out.dtype, 0))["grid"]
    rec = torch.zeros((max(grid, 1), 4), dtype=torch.int64, device=a.device)
    s = sched._c()
    ab_t, c_t = _TORCH_DTYPE.get(a.dtype, 0), _TORCH_DTYPE.get(out.dtype, 0)
    need = query(M, N, K, sched, ab_t, c_t)["workspace_bytes"]
    ws = workspace(need, a.device) if need > 0 else None
    _check(_lib.ts_gemm_clocked(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K,
                                a.stride(0), a.stride(1), b.stride(0), b.stride(1), out.stride(0), out.stride(1),
                                ab_t, c_t, ctypes.byref(s), _stream_handle(a.device), rec.data_ptr(), rec.shape[0],
                                ws.data_ptr() if ws is not None else None, need))
    return rec


def clock_ghz(rec) -> dict:
    """Shader clock per workgroup from a ts_gemm_clocked record (s_memtime ticks over
    100 MHz s_memrealtime ticks): mean / min / max over workgroups, in GHz."""
    r = rec.cpu().to(torch.float64)
    ticks = r[:, 1] - r[:, 0]
    secs = (r[:, 3] - r[:, 2]) / 100e6
    ok = secs > 0
    ghz = ticks[ok] / secs[ok] / 1e9
    return {"mean": float(ghz.mean()), "min": float(ghz.min()), "max": float(ghz.max()),
            "programs": int(ok.sum())}


def _probe_tflops(launch, iters: int, reps: int, device) -> float:
    q = query(256, 256, 256)
    sink = torch.empty(q["cu_count"] * 512, dtype=torch.float32, device=device)
    flops = ctypes.c_double(0.0)
    stream = _stream_handle(sink.device)
    _check(launch(iters, sink, flops, stream))
    best = 0.0
    for _ in range(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        _check(launch(iters, sink, flops, stream))
        e1.record()
        torch.cuda.synchronize()
        best = max(best, flops.value / (e0.elapsed_time(e1) * 1e-3) / 1e12)
    return best


def mfma_loop_tflops(iters: int = 20000, reps: int = 3, device: int | str = "cuda") -> float:
    """Sustained MFMA rate (TFLOP/s) of the no-memory probe, best of ``reps`` timed launches."""
    return _probe_tflops(lambda n, sink, flops, stream: _lib.ts_mfma_loop_probe(
        n, sink.data_ptr(), sink.numel(), ctypes.byref(flops), stream), iters, reps, device)


def mfma_phase_tflops(pattern: int, iters: int = 10000, reps: int = 3, device: int | str = "cuda") -> float:
    """MFMA rate (TFLOP/s) of the barrier-phase probe (ts_mfma_phase_probe), best of ``reps``."""
    return _probe_tflops(lambda n, sink, flops, stream: _lib.ts_mfma_phase_probe(
        n, pattern, sink.data_ptr(), sink.numel(), ctypes.byref(flops), stream), iters, reps, device)


def gemm_raw(a_ptr: int, b_ptr: int, c_ptr: int, M: int, N: int, K: int,
             strides=(None, 1, None, 1, None, 1), ab_dtype: int = TS_F16, c_dtype: int = TS_F16,
             schedule: Schedule | None = None, stream: int = 0) -> int:
    """Direct call of ts_gemm with integer pointers; returns the status code."""
    sam, sak, sbk, sbn, scm, scn = strides
    sam = K if sam is None else sam
    sbk = N if sbk is None else sbk
    scm = N if scm is None else scm
    s = (schedule or Schedule())._c()
    return _lib.ts_gemm(a_ptr, b_ptr, c_ptr, M, N, K, sam, sak, sbk, sbn, scm, scn,
                        ab_dtype, c_dtype, ctypes.byref(s), stream)


def query(M: int, N: int, K: int, schedule: Schedule | None = None,
          ab_dtype: int = TS_F16, c_dtype: int = TS_F16) -> dict:
    info = LaunchInfo()
    s = (schedule or Schedule())._c()
    _check(_lib.ts_query(M, N, K, ab_dtype, c_dtype, ctypes.byref(s), ctypes.byref(info)))
    return info.as_dict()


def schedule_trace(M: int, N: int, K: int, schedule: Schedule | None = None,
                   ab_dtype: int = TS_F16, c_dtype: int = TS_F16, device: int | str = "cuda"):
    """GPU-computed work sequence of every workgroup, as an int32 [rows, 5] CPU tensor."""
    info = query(M, N, K, schedule, ab_dtype, c_dtype)
    grid = info["grid"]
    rows = grid * info["trace_items"]
    out = torch.empty((max(rows, 1), 5), dtype=torch.int32, device=device)
    s = (schedule or Schedule())._c()
    _check(_lib.ts_schedule_trace(M, N, K, ab_dtype, c_dtype, ctypes.byref(s), out.data_ptr(), rows,
                                  _stream_handle(out.device)))
    torch.cuda.synchronize(out.device)
    return out[:rows].cpu()


def schedule_trace_host(M: int, N: int, K: int, schedule: Schedule, cu_count: int = 0,
                        programs_per_cu: int = 0, ab_dtype: int = TS_F16, c_dtype: int = TS_F16):
    """The same work sequence computed by the library on the CPU (no GPU needed).

    In persistent modes with num_programs == 0, cu_count * programs_per_cu stands
    in for the device's grid.
    """
    import numpy as np

    sized = schedule
    if schedule.mode != "tiled" and schedule.num_programs == 0:
        sized = dataclasses.replace(schedule, num_programs=cu_count * programs_per_cu)
    info = query(M, N, K, sized, ab_dtype, c_dtype)
    rows = info["grid"] * info["trace_items"]
    out = np.full((max(rows, 1), 5), -7, dtype=np.int32)
    s = schedule._c()
    _check(_lib.ts_schedule_trace_host(M, N, K, ab_dtype, c_dtype, ctypes.byref(s), cu_count,
                                       programs_per_cu, out.ctypes.data, rows))
    return out[:rows]


# ---- operators around the product ------------------------------------------------------

if not isinstance(_binding, _Missing):
    _binding.set_error(TsError)


class Checkpoint:
    """Rows kept in 8 bits for a backward pass: an [M, N] matrix in ``data``, a uint8 [M, pitch] CUDA
    tensor of unit column stride (16-byte aligned, row stride a multiple of 16).

    32 neighbours of a row share one step 2^e, the least for which the largest of them is at most
    127 steps; a value is a whole number of steps (int8), off by at most half a step.  A row of ``data``:
    32 ceil(N / 32) values, then a byte e + 127 for each 32; 255: they held an infinity or a NaN, and
    all of them stand for NaN.  A finite value is read as a finite one of its own type (2^128 as the largest
    bf16 number, in fp16 2^16 as 65504).  ``checkpoint_pack``, ``layernorm`` and the product (``preact``) write
    it; ``checkpoint_unpack``, ``act_grad``, ``gemm_dact``, the products' and the norms' gradients read it.
    Its rows are ``data``'s: a slice of those is a checkpoint of the same rows.
    """

    __slots__ = ("data", "n")

    def __init__(self, data: torch.Tensor, n: int):
        self.data, self.n = data, int(n)
        if data.dim() != 2 or data.dtype != torch.uint8:
            raise ValueError("a checkpoint's data is a uint8 matrix")
        if n < 0 or data.shape[1] < 33 * -(-self.n // 32):
            raise ValueError(f"rows of {data.shape[1]} bytes do not hold {n} columns")
        row, col = data.stride()
        if (col != 1 and data.shape[1] > 1) or (row % 16 and data.shape[0] > 1) or data.data_ptr() % 16:
            raise ValueError("a checkpoint's rows are contiguous and 16-byte aligned")

    @classmethod
    def empty(cls, m: int, n: int, device=None) -> "Checkpoint":
        """Room for an [m, n] matrix (rows of whole 64-byte lines)."""
        return _kept(torch.empty((m, -(-33 * -(-n // 32) // 64) * 64), dtype=torch.uint8, device=device or "cuda"), n)

    @property
    def shape(self):
        return torch.Size((self.data.shape[0], self.n))

    @property
    def device(self):
        return self.data.device


def _data(t):
    """A tensor's or a Checkpoint's storage, and the columns that it holds (-1: as many as the tensor has)."""
    return (t.data, t.n) if type(t) is Checkpoint else (t, -1)


def _kept(data: torch.Tensor, n: int) -> Checkpoint:
    """A Checkpoint of data that this library made."""
    k = Checkpoint.__new__(Checkpoint)
    k.data, k.n = data, n
    return k


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def _product(a, b, out, out_dtype, act: str, grad: int, schedule, residual=None, preact=None, bias=None, scale_a=None,
             scale_b=None):
    s = schedule._c() if schedule is not None else None
    preact, n = _data(preact)
    return _binding.product(a, b, out, out_dtype, _activation(act), grad, ctypes.addressof(s) if s is not None else 0,
                            residual, preact, n, bias, scale_a, scale_b)


def gemm_epilogue(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "none",
                  residual: torch.Tensor | None = None, preact: torch.Tensor | Checkpoint | None = None,
                  out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  schedule: Schedule | None = None) -> torch.Tensor:
    """C = act(A @ B + bias) + residual, A [M,K] and B [K,N] fp16/bf16; C fp16/bf16/fp32.

    ``activation``: "none", "relu", "gelu" (exact), "gelu_tanh" or "silu".  ``bias``: [N],
    fp16/bf16/fp32.  ``residual``: [M,N] of C's type (may be ``out``).  ``preact``: an [M,N]
    tensor of C's type that receives A @ B + bias, for the backward pass, or a ``Checkpoint``
    that receives it in 8 bits (no stream-K).  A and B may be
    transposed views and have any row stride; ``schedule=None`` chooses order, mode and tile.
    Enqueued on the current stream of A's device.  A 2-D product: batched or 1-D operands
    are reshaped by the caller.  The gradients: ``gemm_epilogue_backward`` (autograd does not see
    the call, as it does not see ``gemm``).
    """
    return _product(a, b, out, out_dtype or (out.dtype if out is not None else None), activation, 0, schedule, residual,
                    preact, bias)


def gemm_dact(a: torch.Tensor, b: torch.Tensor, preact: torch.Tensor | Checkpoint, activation: str,
              out: torch.Tensor | None = None, schedule: Schedule | None = None) -> torch.Tensor:
    """C = (A @ B) * act'(preact): the gradient that reaches the input of an activation whose
    output feeds a product, in that product's own backward launch (A the gradient of its
    output, B its weights transposed).  C has ``preact``'s type and may be ``preact``; with a
    ``Checkpoint`` it has A's type (or ``out``'s)."""
    kept = type(preact) is Checkpoint
    dtype = preact.dtype if not kept else out.dtype if out is not None else a.dtype
    return _product(a, b, out, dtype, activation, 1, schedule, preact=preact)


def gemm_scaled(a: torch.Tensor, b: torch.Tensor, scale_a: torch.Tensor | None = None,
                scale_b: torch.Tensor | None = None, bias: torch.Tensor | None = None, activation: str = "none",
                residual: torch.Tensor | None = None, preact: torch.Tensor | None = None,
                out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                schedule: Schedule | None = None) -> torch.Tensor:
    """C = act(((A @ B) * scale_a[:, None]) * scale_b[None, :] + bias) + residual with e4m3 or int8 A
    [M,K] (rows contiguous) and B [K,N] stored [N][K] (a transposed view of [N,K] weights).

    ``scale_a`` [M] (tokens) and ``scale_b`` [N] (channels) are fp32 (None: 1); an element's value is
    code * scale, as the norms and ``quantize_rows`` return them.  int8: the sums are exact (K up to
    131071) and rounded once, to fp32.  C is fp16, bf16 (default) or fp32.  Otherwise as
    ``gemm_epilogue`` (``preact``: a tensor).
    """
    if a.dtype != torch.float8_e4m3fn and a.dtype != torch.int8:
        raise ValueError(f"A is {a.dtype}, expected torch.float8_e4m3fn or torch.int8")
    return _product(a, b, out, out_dtype or (out.dtype if out is not None else torch.bfloat16), activation, 0, schedule,
                    residual, preact, bias, scale_a, scale_b)


def act_grad(dc: torch.Tensor, preact: torch.Tensor | Checkpoint | None = None, activation: str = "none",
             out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, dbias: bool = True,
             dbias_dtype: torch.dtype = torch.float32, act_out: torch.Tensor | None = None):
    """dZ = dC * act'(preact) and the bias gradient, its column sums; returns (dZ, dbias).

    dC and ``preact`` are [M,N] of one type (fp16, bf16, fp32), or ``preact`` is a ``Checkpoint``.  dZ:
    ``out`` or a new tensor of ``out_dtype`` (dC's type; fp16 or bf16 from fp32).  dbias sums the
    unrounded fp32 products in a fixed order (the same bits on every run); None if ``dbias`` is False.
    ``act_out``: an [M,N] tensor of dZ's type that receives act(preact), the operand of the next weight's
    gradient, which the forward pass then need not keep.
    With activation "none", ``preact`` is read for ``act_out`` only, and dZ is dC itself (not a copy)
    unless ``out`` or ``out_dtype`` asks for one.
    """
    preact, n = _data(preact)
    return _binding.act_grad(dc, preact, n, _activation(activation), out, out_dtype, dbias, dbias_dtype, act_out)


def gemm_epilogue_backward(dc: torch.Tensor, a: torch.Tensor | Checkpoint, b: torch.Tensor,
                           preact: torch.Tensor | Checkpoint | None = None,
                           activation: str = "none", dbias: bool = True,
                           dbias_dtype: torch.dtype = torch.float32, schedule: Schedule | None = None):
    """Gradients of C = act(A @ B + bias) + residual given dC: returns (dA, dB, dbias).

    dZ = dC * act'(preact) is formed once, rounded to A's type (an operand of the two
    products that follow); dA = dZ @ B^T and dB = A^T @ dZ have A's and B's type, dbias
    (None if not asked for) sums the unrounded dZ.  The residual's gradient is dC itself.
    ``preact`` is what the forward call stored, of dC's type or in 8 bits; not needed for "none".  A
    kept in 8 bits is read back in B's type first (one pass).
    """
    if type(a) is Checkpoint:
        a = checkpoint_unpack(a, out_dtype=b.dtype)
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0] or tuple(dc.shape) != (a.shape[0], b.shape[1]):
        raise ValueError(f"dC {tuple(dc.shape)} is not the gradient of {tuple(a.shape)} @ {tuple(b.shape)}")
    if a.dtype not in (torch.float16, torch.bfloat16) or b.dtype != a.dtype:
        raise ValueError("A and B must be fp16 or bf16, of one type")
    dz, db = act_grad(dc, preact, activation, out_dtype=a.dtype, dbias=dbias, dbias_dtype=dbias_dtype)
    da = gemm_epilogue(dz, b.t(), schedule=schedule)
    dw = gemm_epilogue(a.t(), dz, schedule=schedule)
    return da, dw, db


def rmsnorm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
            eps: float = 1e-6, out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
            h: torch.Tensor | None = None):
    """h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight, row by row; returns
    (y, scale, h).

    x [M,N] fp16, bf16 or fp32; ``residual`` [M,N] of x's type; ``weight`` [N], x's type or
    fp32 (None: 1).  The norm reads the unrounded fp32 sum; h (x itself without a residual)
    is its rounding to x's type, what the next block adds to and ``rmsnorm_backward`` takes.
    The tensor given as ``h`` receives it and may be ``residual`` or x (in place).
    y has ``out_dtype``: x's type (default), torch.float8_e4m3fn or torch.int8, which add one fp32
    ``scale`` per row, max|y| / 448 or / 127 (at least 2^-100), with y = code * scale: the operand and
    scale_a of ``gemm_scaled``.  Else scale is None.  The gradients: ``rmsnorm_backward``
    (autograd does not see the call).
    """
    return _binding.rmsnorm(x, weight, residual, eps, out_dtype, out, h)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor | Checkpoint, weight: torch.Tensor | None = None, eps: float = 1e-6,
                     dh: torch.Tensor | None = None, dweight: bool = True, out: torch.Tensor | None = None):
    """Gradients of y = h / sqrt(mean(h^2) + eps) * weight given dy; returns (dx, dweight).

    dx = dL/dh + ``dh``, where ``dh`` is the gradient that reaches h along the residual
    stream (None: 0): the gradient of x and of the residual alike.  dy, h and dh are [M,N]
    of one type, dx has it too (``out`` may be dy or dh).  dweight has weight's type, summed
    in fp32 in a fixed order; None without a weight or if ``dweight`` is False.  The 8-bit
    output of the forward pass is differentiated as y itself (straight through).  h kept in 8 bits
    is read back in dy's type first (one pass).
    """
    if type(h) is Checkpoint:
        h = checkpoint_unpack(h, out_dtype=dy.dtype)
    return _binding.rmsnorm_backward(dy, h, weight, eps, dh, dweight, out)


def layernorm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
              residual: torch.Tensor | None = None, eps: float = 1e-5, out_dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None, h: torch.Tensor | None = None, keep: Checkpoint | None = None):
    """h = x + residual;  y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias, row by row; returns
    (y, scale, h).

    As ``rmsnorm``: x [M,N] fp16, bf16 or fp32, ``residual`` of its type, h its rounding; ``weight`` (None:
    1) and ``bias`` (None: 0) [N], of one type, x's or fp32; y in x's type, or torch.float8_e4m3fn or
    torch.int8 with one fp32 ``scale`` per row.  The variance is the mean square of the differences from
    the mean.  ``keep``: receives h in 8 bits, what ``layernorm_backward`` takes in place of h.
    The gradients: ``layernorm_backward`` (autograd does not see the call).
    """
    keep, n = _data(keep)
    return _binding.layernorm(x, weight, bias, residual, eps, out_dtype, out, h, keep, n)


def layernorm_backward(dy: torch.Tensor, h: torch.Tensor | Checkpoint, weight: torch.Tensor | None = None,
                       eps: float = 1e-5, dh: torch.Tensor | None = None, dweight: bool = True, dbias: bool = True,
                       dbias_dtype: torch.dtype | None = None, out: torch.Tensor | None = None):
    """Gradients of ``layernorm`` given dy; returns (dx, dweight, dbias).

    dx = dL/dh + ``dh`` (the gradient that reaches h along the residual stream, None: 0).  dy and dh are
    [M,N] of one type, h of the same or a ``Checkpoint``; dx has dy's type (``out`` may be dy or dh).
    dweight and dbias, the column sums of dy (h - mean) / deviation and of dy, have weight's type, without a
    weight ``dbias_dtype`` (fp32) and dweight is None; summed in fp32 in a fixed order.  The 8-bit output
    of the forward pass is differentiated as y itself (straight through).
    """
    h, n = _data(h)
    return _binding.layernorm_backward(dy, h, n, weight, eps, dh, dweight, dbias, dbias_dtype, out)


def quantize_rows(x: torch.Tensor, out_dtype: torch.dtype = torch.int8, out: torch.Tensor | None = None):
    """x [M,N] (fp16, bf16, fp32) in 8 bits with one fp32 scale per row; returns (codes, scale).

    scale = max|x| / 127 (torch.int8) or / 448 (torch.float8_e4m3fn), at least 2^-100; codes = x / scale
    rounded to nearest even: the operand and scale_a of ``gemm_scaled`` where no norm stands before the
    product.  A row with an infinity or a NaN has such a scale, and a product of it is NaN.
    """
    return _binding.quantize_rows(x, out_dtype, out)


def checkpoint_pack(x: torch.Tensor, out: Checkpoint | None = None) -> Checkpoint:
    """x [M,N] (fp16, bf16, fp32) in 8 bits (``out`` or a new ``Checkpoint``): 33/32 bytes a value."""
    if out is None:
        return _kept(_binding.checkpoint_pack(x, None, -1), x.shape[1])
    _binding.checkpoint_pack(x, out.data, out.n)
    return out


def checkpoint_unpack(kept: Checkpoint, activation: str = "none", out: torch.Tensor | None = None,
                      out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """act(value) of what a ``Checkpoint`` keeps, in ``out`` or a new tensor of ``out_dtype`` (fp32).

    The values themselves are exact in bf16 and fp32 (8 significant bits); in fp16 those beyond 2^16 are
    infinite."""
    return _binding.checkpoint_unpack(kept.data, kept.n, _activation(activation), out, out_dtype)
