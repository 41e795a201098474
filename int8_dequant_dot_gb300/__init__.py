"""Python binding of libloom (the C ABI in include/loom.h, loom_tuning.h and loom_token.h).

The functions keep the C names and only marshal arguments: tensors become
device pointers, the stream defaults to torch's current stream, and a status
other than LOOM_OK raises LoomError.  Every step of the computation runs in
libloom's CUDA kernels; there is no fallback, and importing this module
fails loudly when libloom.so has not been built (see build.py).

Each function accepts either torch tensors or raw integer addresses; the token
operators take their sizes from tensors and check them (type, length, order, device);
addresses they take for packed bytes, scales, statistics, sums and tokens that they
write, for error words and for the product's bias.  Output
tensors may be passed in; when omitted they are allocated with torch (on
the inputs' device) and returned.  No call records a gradient: torch's autograd
sees its outputs as new tensors, and loom_layer_norm_backward is called by hand.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
#: the library this instance of the binding loads (the fault tests load a second
#: instance of this module bound to libloom_test.so, by setting LIB_PATH first)
LIB_PATH = globals().get("LIB_PATH") or os.path.join(HERE, "libloom.so")

LOOM_OK = 0
LOOM_ERR_NULL = -1
LOOM_ERR_ALIGN = -2
LOOM_ERR_SHAPE = -3
LOOM_ERR_RANGE = -4
LOOM_ERR_CUDA = -5
LOOM_ERR_TIMEOUT = -6
LOOM_ERR_ARG = -7

LOOM_DEVERR_COUNT_RANGE = 0x1
LOOM_DEVERR_TIMEOUT = 0x2
LOOM_DEVERR_NONFINITE = 0x4
LOOM_DEVERR_NO_TOKEN = 0x8

LOOM_OP_I8_UNPACK = 0
LOOM_OP_FULL_TILE_SUM = 1
LOOM_OP_ROW_SUM_BATCHED = 2
LOOM_OP_I8_DEQUANT_DOT = 3
LOOM_OP_PACKED_DOT = 4
LOOM_OP_LANE_SUMS = 5
LOOM_OP_ROUTED_COMBINE = 6
LOOM_OP_STAGE_ROWS = 7
LOOM_OP_QUANTIZE_TOKENS = 8
LOOM_OP_I8_MATMUL = 9
LOOM_OP_LAYER_NORM = 10
LOOM_OP_LAYER_NORM_BACKWARD = 11
LOOM_OP_SAMPLE_TOKENS = 12
LOOM_OP_I4_MATVEC = 13
LOOM_OP_ROUTE_TOKENS = 14
LOOM_OP_ROUTE_TOKENS_BACKWARD = 15
LOOM_OP_ADJUST_LOGITS = 16

LOOM_KERNEL_UNPACK = 1
LOOM_KERNEL_ROWSUM_STAGED = 2
LOOM_KERNEL_ROWSUM_DIRECT = 3
LOOM_KERNEL_DOT_STAGED_K = 4
LOOM_KERNEL_DOT_STAGED_B = 5
LOOM_KERNEL_DOT_DIRECT = 6
LOOM_KERNEL_DOT_TENSOR = 7
LOOM_KERNEL_DOT_TENSOR_SPLIT = 8
LOOM_KERNEL_PACKED_STAGED = 9
LOOM_KERNEL_PACKED_DIRECT = 10
LOOM_KERNEL_LANESUM_STAGED = 11
LOOM_KERNEL_LANESUM_DIRECT = 12
LOOM_KERNEL_ROUTED_STAGED = 13
LOOM_KERNEL_ROUTED_DIRECT = 14
LOOM_KERNEL_STAGE_ROWS = 15
LOOM_KERNEL_DOT_TENSOR_ROWS = 16
LOOM_KERNEL_ROWSUM_SEGMENTS = 17
LOOM_KERNEL_I8_MATMUL_DP4A = 18
LOOM_KERNEL_I8_MATMUL_TENSOR = 19
LOOM_KERNEL_NORM_ROWS = 20
LOOM_KERNEL_NORM_LONG = 21
LOOM_KERNEL_NORM_BACKWARD = 22
LOOM_KERNEL_SAMPLE = 24
LOOM_KERNEL_I4_MATVEC = 25
LOOM_KERNEL_ROUTE = 26
LOOM_KERNEL_ROUTE_BACKWARD = 27
LOOM_KERNEL_ADJUST = 28

LOOM_F32 = 0
LOOM_F16 = 1
LOOM_BF16 = 2

LOOM_SCORE_SOFTMAX = 0
LOOM_SCORE_SIGMOID = 1

LOOM_MAX_DEPTH = 8
LOOM_PATH_AUTO = 0
LOOM_PATH_STAGED = 1
LOOM_PATH_DIRECT = 2
LOOM_PATH_TENSOR = 3

LOOM_FLOOR_GRID_STRIDE = 0
LOOM_FLOOR_WARP_RANGE = 1
LOOM_FLOOR_BULK_RING = 2

#: every extern "C" symbol the headers declare
EXPORTS = (
    "loom_launch_config", "loom_full_tile_sum", "loom_row_sum_batched", "loom_i8_dequant_dot",
    "loom_i8_unpack", "loom_status_string", "loom_abi_version", "loom_row_sum_batched_ex",
    "loom_i8_dequant_dot_ex", "loom_i8_dequant_dot_workspace_bytes", "loom_i8_dequant_dot_noalloc",
    "loom_packed_dot", "loom_packed_dot_ex", "loom_sum_rows", "loom_sum_rows_ex", "loom_sum_guarded_rows",
    "loom_sum_guarded_rows_ex", "loom_routed_combine", "loom_routed_combine_ex", "loom_stage_rows",
    "loom_stream_floor", "loom_token_launch_config", "loom_quantize_tokens", "loom_i8_matmul", "loom_i8_matmul_ex",
    "loom_layer_norm", "loom_layer_norm_i8", "loom_layer_norm_backward", "loom_layer_norm_backward_workspace_bytes",
    "loom_sample_tokens", "loom_adjust_logits", "loom_i4_matvec", "loom_i4_matvec_routed", "loom_route_tokens",
    "loom_route_tokens_backward",
)


class LoomError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {loom_status_string(status)} (status {status})")


class loom_launch(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_uint32 * 3), ("block", ctypes.c_uint32 * 3),
                ("cluster", ctypes.c_uint32 * 3), ("subgroup_size", ctypes.c_uint32),
                ("smem_bytes", ctypes.c_uint32), ("units_per_cta", ctypes.c_uint32),
                ("kernel", ctypes.c_uint32)]

    def as_dict(self) -> dict:
        return {"grid": tuple(self.grid), "block": tuple(self.block), "cluster": tuple(self.cluster),
                "subgroup_size": self.subgroup_size, "smem_bytes": self.smem_bytes,
                "units_per_cta": self.units_per_cta, "kernel": self.kernel}


class loom_tuning(ctypes.Structure):
    _fields_ = [("depth", ctypes.c_int32), ("path", ctypes.c_int32),
                ("units_per_warp", ctypes.c_int32), ("warps_per_cta", ctypes.c_int32),
                ("chunk_bytes", ctypes.c_int32), ("wait_ns", ctypes.c_int64),
                ("tc_units_per_stage", ctypes.c_int32),
                ("tc_a_buffers", ctypes.c_int32), ("tc_pipelines", ctypes.c_int32),
                ("tc_schedule", ctypes.c_int32)]


def _bind() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libloom.so is not built ({LIB_PATH}); run "
                          "`python int8_dequant_dot_gb300/build.py` or __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sig = {
        "loom_launch_config": [i32, P, i32, ctypes.POINTER(loom_launch)],
        "loom_full_tile_sum": [P, i32, i32, i32, f32, i32, P, P, P, P, P],
        "loom_row_sum_batched": [P, i64, i64, i32, i32, P, P, i32, P, P, P, P, P, P],
        "loom_row_sum_batched_ex": [P, i64, i64, i32, i32, P, P, i32, P, P, P, P, P,
                                    ctypes.POINTER(loom_tuning), P],
        "loom_i8_dequant_dot": [P, P, i32, i32, P, P, i32, P, P, P, i64, P],
        "loom_i8_dequant_dot_ex": [P, P, i32, i32, P, P, i32, P, P, P, i64, P,
                                   ctypes.POINTER(loom_tuning), P],
        "loom_i8_dequant_dot_workspace_bytes": [i32, i32, i32, ctypes.POINTER(i64)],
        "loom_i8_dequant_dot_noalloc": [P, P, i32, i32, P, P, i32, P, P, P],
        "loom_packed_dot": [P, P, P, i32, i32, i32, i32, P, i32, P, P, P],
        "loom_packed_dot_ex": [P, P, P, i32, i32, i32, i32, P, i32, P, P, P, ctypes.POINTER(loom_tuning), P],
        "loom_sum_rows": [P, i64, i64, i32, i32, i32, P, i32, P, P],
        "loom_sum_rows_ex": [P, i64, i64, i32, i32, i32, P, i32, P, P, ctypes.POINTER(loom_tuning), P],
        "loom_sum_guarded_rows": [P, i64, i64, i32, i32, P, i32, i32, i32, P, P],
        "loom_sum_guarded_rows_ex": [P, i64, i64, i32, i32, P, i32, i32, i32, P, P, ctypes.POINTER(loom_tuning), P],
        "loom_routed_combine": [P, P, P, i64, i32, i32, i32, P, P],
        "loom_routed_combine_ex": [P, P, P, i64, i32, i32, i32, P, P, ctypes.POINTER(loom_tuning), P],
        "loom_stage_rows": [P, P, i64, i64, i32, i32, P, i32, P],
        "loom_i8_unpack": [P, i64, P, P],
        "loom_stream_floor": [P, i64, i32, i32, i32, P, P, P],
        "loom_token_launch_config": [i32, P, i32, ctypes.POINTER(loom_launch)],
        "loom_quantize_tokens": [P, i32, i64, i32, i64, P, P, P, P],
        "loom_i8_matmul": [P, P, i32, i32, P, P, i32, P, P, i32, i64, P, P],
        "loom_i8_matmul_ex": [P, P, i32, i32, P, P, i32, P, P, i32, i64, P, P, ctypes.POINTER(loom_tuning), P],
        "loom_layer_norm": [P, i32, i64, i32, i64, P, P, f32, P, i64, P, P, P],
        "loom_layer_norm_i8": [P, i32, i64, i32, i64, P, P, f32, P, P, P, P],
        "loom_layer_norm_backward": [P, i64, P, i64, i32, i64, i32, P, P, P, P, i64, P, P, P, i64, P],
        "loom_layer_norm_backward_workspace_bytes": [i64, i32, ctypes.POINTER(i64)],
        "loom_sample_tokens": [P, i32, i64, i32, i64, P, f32, P, i32, P, f32, P, f32, P, P, P, P, P],
        "loom_adjust_logits": [P, i32, i64, i32, i64, P, i32, i64, P, P, P, f32, P, f32, P, f32, P, P, i32, P, i32, P, P, i64, P, P],
        "loom_i4_matvec": [P, P, i32, i32, i32, i32, P, P, i32, P, P, i32, i64, P],
        "loom_i4_matvec_routed": [P, P, i32, i32, i32, i32, i32, P, P, i64, P, i32, i32, P, P, i32, i64, P, P],
        "loom_route_tokens": [P, i32, i64, i32, i64, P, i32, i32, i32, i32, i32, i32, f32, P, P, P, P],
        "loom_route_tokens_backward": [P, P, i32, i64, i32, i64, P, i32, i32, i32, f32, P, i64, P, P],
        "loom_status_string": [i32],
        "loom_abi_version": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32
    lib.loom_status_string.restype = ctypes.c_char_p
    return lib


_lib = _bind()


def library() -> ctypes.CDLL:
    return _lib


def loom_abi_version() -> int:
    return int(_lib.loom_abi_version())


def loom_status_string(status: int) -> str:
    return _lib.loom_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != LOOM_OK:
        raise LoomError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, like=None):
    if stream is None:
        import torch
        dev = like.device if like is not None and hasattr(like, "device") else None
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def loom_launch_config(op: int, workload) -> dict:
    arr = (ctypes.c_int64 * max(1, len(workload)))(*[int(v) for v in workload])
    out = loom_launch()
    _check(_lib.loom_launch_config(int(op), arr, len(workload), ctypes.byref(out)),
           "loom_launch_config")
    return out.as_dict()


def _empty(like, shape, dtype):
    import torch
    return torch.empty(shape, dtype=dtype, device=like.device)


def loom_full_tile_sum(values, count: int, initial: float, tile_size: int = 8, *,
                       rows: int | None = None, lanes: int | None = None, out=None, stream=None):
    """One segment ``values[rows][lanes]``; returns ``(final_row, tail_count, full_sum,
    tail_sum)`` as four one-element device tensors (or fills ``out``)."""
    import torch
    if rows is None or lanes is None:
        rows, lanes = values.shape
    if out is None:
        out = (_empty(values, (1,), torch.int32), _empty(values, (1,), torch.int32),
               _empty(values, (1,), torch.float32), _empty(values, (1,), torch.float32))
    fr, tc, fs, ts = out
    _check(_lib.loom_full_tile_sum(_ptr(values), int(rows), int(lanes), int(count), float(initial),
                                   int(tile_size), _ptr(fr), _ptr(tc), _ptr(fs), _ptr(ts),
                                   _stream(stream, values)), "loom_full_tile_sum")
    return out


def _row_sum_outputs(values, n):
    import torch
    return (_empty(values, (n,), torch.int32), _empty(values, (n,), torch.int32),
            _empty(values, (n,), torch.float32), _empty(values, (n,), torch.float32))


def loom_row_sum_batched(values, num_segments: int, seg_stride: int, rows: int, lanes: int,
                         counts, initial=None, tile_size: int = 8, *, out=None, error=None,
                         stream=None):
    """Batched segments; returns ``(final_row, tail_count, full_sum, tail_sum)``."""
    if out is None:
        out = _row_sum_outputs(values, num_segments)
    fr, tc, fs, ts = out
    _check(_lib.loom_row_sum_batched(_ptr(values), int(num_segments), int(seg_stride), int(rows),
                                     int(lanes), _ptr(counts), _ptr(initial), int(tile_size),
                                     _ptr(fr), _ptr(tc), _ptr(fs), _ptr(ts), _ptr(error),
                                     _stream(stream, values)), "loom_row_sum_batched")
    return out


def make_tuning(depth: int = 0, path: int = LOOM_PATH_AUTO, units_per_warp: int = 0,
                warps_per_cta: int = 0, chunk_bytes: int = 0, wait_ns: int = 0,
                tc_units_per_stage: int = 0, tc_a_buffers: int = 0, tc_pipelines: int = 0,
                tc_schedule: int = 0) -> loom_tuning:
    return loom_tuning(int(depth), int(path), int(units_per_warp), int(warps_per_cta),
                       int(chunk_bytes), int(wait_ns), int(tc_units_per_stage), int(tc_a_buffers),
                       int(tc_pipelines), int(tc_schedule))


def loom_row_sum_batched_ex(values, num_segments: int, seg_stride: int, rows: int, lanes: int,
                            counts, initial=None, tile_size: int = 8, *, tuning=None, out=None,
                            error=None, stream=None):
    if out is None:
        out = _row_sum_outputs(values, num_segments)
    fr, tc, fs, ts = out
    tp = ctypes.byref(tuning) if tuning is not None else None
    _check(_lib.loom_row_sum_batched_ex(_ptr(values), int(num_segments), int(seg_stride), int(rows),
                                        int(lanes), _ptr(counts), _ptr(initial), int(tile_size),
                                        _ptr(fr), _ptr(tc), _ptr(fs), _ptr(ts), _ptr(error), tp,
                                        _stream(stream, values)), "loom_row_sum_batched_ex")
    return out


def _dot_outputs(w, n_rows, batch, want_acc):
    import torch
    y = _empty(w, (n_rows, batch), torch.float32)
    acc = _empty(w, (n_rows, batch), torch.int32) if want_acc else None
    return y, acc


def loom_i8_dequant_dot_workspace_bytes(n_rows: int, k: int, batch: int) -> int:
    """Bytes of the split-band workspace on the current device (0: none is used)."""
    out = ctypes.c_int64(0)
    _check(_lib.loom_i8_dequant_dot_workspace_bytes(int(n_rows), int(k), int(batch),
                                                    ctypes.byref(out)),
           "loom_i8_dequant_dot_workspace_bytes")
    return int(out.value)


def dot_workspace(n_rows: int, k: int, batch: int, device=None):
    """A workspace for ``loom_i8_dequant_dot`` on ``device`` (None when the call would not
    use one).  The caller owns it; calls that may overlap need one each."""
    import torch
    nbytes = loom_i8_dequant_dot_workspace_bytes(n_rows, k, batch)
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device if device is not None else "cuda")


#: workspace="auto": one workspace per (device, stream), kept for reuse
AUTO = "auto"
_workspaces: dict = {}
_workspaces_lock = threading.Lock()
#: the largest problem the workspace query accepts: its workspace is the most any
#: call on the device uses (the size grows with the CTAs, at most one per SM)
_MAX_PROBLEM = (0x7FFFFFFF, 16, 16)


def _workspace(workspace, like, n_rows, k, batch, stream_handle):
    """(address, bytes) of the workspace argument.  "auto" keeps one workspace per
    (device, stream), allocated once at its first use with the most any call on that
    device needs, so it never grows and no call waits for the device."""
    if workspace is None:
        return None, 0
    if not (isinstance(workspace, str) and workspace == AUTO):
        if isinstance(workspace, tuple):
            return workspace
        return _ptr(workspace), workspace.numel() * workspace.element_size()
    import torch
    if loom_i8_dequant_dot_workspace_bytes(n_rows, k, batch) == 0:
        return None, 0
    dev = like.device if hasattr(like, "device") else torch.device("cuda", torch.cuda.current_device())
    key = (dev.index, stream_handle)
    with _workspaces_lock:
        ws = _workspaces.get(key)
        if ws is None:
            nbytes = loom_i8_dequant_dot_workspace_bytes(*_MAX_PROBLEM)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _workspaces[key] = ws
    return ws.data_ptr(), ws.numel()


def _on_device(t):
    """The device of tensor `t` made current for the call (the library sizes the
    tensor-core grid and finds its scratch on the current device)."""
    import contextlib
    if hasattr(t, "device") and getattr(t.device, "type", None) == "cuda":
        import torch
        return torch.cuda.device(t.device)
    return contextlib.nullcontext()


def loom_i8_dequant_dot(w_packed, scale_w, n_rows: int, k: int, x_packed, scale_x, batch: int, *,
                        y=None, acc=None, want_acc: bool = False, workspace=AUTO, stream=None):
    """``y[n_rows][batch]`` (and ``acc`` when requested); returns ``(y, acc)``.
    ``workspace``: a tensor (see ``dot_workspace``), an ``(address, bytes)`` pair, None
    (no split), or "auto" (kept per device and stream)."""
    if y is None:
        y, acc2 = _dot_outputs(w_packed, n_rows, batch, want_acc and acc is None)
        acc = acc if acc is not None else acc2
    with _on_device(w_packed):
        st = _stream(stream, w_packed)
        wp, wb = _workspace(workspace, w_packed, n_rows, k, batch, st)
        _check(_lib.loom_i8_dequant_dot(_ptr(w_packed), _ptr(scale_w), int(n_rows), int(k),
                                        _ptr(x_packed), _ptr(scale_x), int(batch), _ptr(y), _ptr(acc),
                                        wp, int(wb), st), "loom_i8_dequant_dot")
    return y, acc


def loom_i8_dequant_dot_ex(w_packed, scale_w, n_rows: int, k: int, x_packed, scale_x, batch: int,
                           *, y=None, acc=None, want_acc: bool = False, workspace=AUTO, error=None,
                           tuning=None, stream=None):
    if y is None:
        y, acc2 = _dot_outputs(w_packed, n_rows, batch, want_acc and acc is None)
        acc = acc if acc is not None else acc2
    tp = ctypes.byref(tuning) if tuning is not None else None
    with _on_device(w_packed):
        st = _stream(stream, w_packed)
        wp, wb = _workspace(workspace, w_packed, n_rows, k, batch, st)
        _check(_lib.loom_i8_dequant_dot_ex(_ptr(w_packed), _ptr(scale_w), int(n_rows), int(k),
                                           _ptr(x_packed), _ptr(scale_x), int(batch), _ptr(y), _ptr(acc),
                                           wp, int(wb), _ptr(error), tp, st),
               "loom_i8_dequant_dot_ex")
    return y, acc


def loom_i8_dequant_dot_noalloc(w_packed, scale_w, n_rows: int, k: int, x_packed, scale_x,
                                batch: int, *, y=None, acc=None, want_acc: bool = False, stream=None):
    """``loom_i8_dequant_dot`` with the library's fixed device scratch (no workspace, no
    allocation in the library); calls that may overlap must be serialised."""
    if y is None:
        y, acc2 = _dot_outputs(w_packed, n_rows, batch, want_acc and acc is None)
        acc = acc if acc is not None else acc2
    with _on_device(w_packed):
        _check(_lib.loom_i8_dequant_dot_noalloc(_ptr(w_packed), _ptr(scale_w), int(n_rows), int(k),
                                                _ptr(x_packed), _ptr(scale_x), int(batch), _ptr(y),
                                                _ptr(acc), _stream(stream, w_packed)),
               "loom_i8_dequant_dot_noalloc")
    return y, acc


def loom_packed_dot(fields, scales, rhs, counts=None, count: int = 0, initial=None, *,
                    problems: int | None = None, records: int | None = None, lanes: int | None = None,
                    streams: int | None = None, out=None, stream=None):
    """The pages' packed signed-byte dot for ``problems`` instances; returns ``out``
    float32 ``[problems][lanes]``.  ``fields`` int32 ``[P][R][L]``, ``scales`` f16 (or
    their int16 bit patterns) ``[P][R][L]``, ``rhs`` float32 ``[P][R][S][4]``; ``counts``
    int32 ``[P]`` on the device, or None with ``count`` for every instance."""
    return loom_packed_dot_ex(fields, scales, rhs, counts, count, initial, problems=problems,
                              records=records, lanes=lanes, streams=streams, out=out, stream=stream,
                              _name="loom_packed_dot")


def loom_packed_dot_ex(fields, scales, rhs, counts=None, count: int = 0, initial=None, *,
                       problems: int | None = None, records: int | None = None, lanes: int | None = None,
                       streams: int | None = None, out=None, error=None, tuning=None, stream=None,
                       _name: str = "loom_packed_dot_ex"):
    import torch
    if problems is None or records is None or lanes is None:
        problems, records, lanes = fields.shape
    if streams is None:
        streams = rhs.shape[2]
    if out is None:
        out = _empty(fields, (int(problems), int(lanes)), torch.float32)
    st = _stream(stream, fields)
    args = (_ptr(fields), _ptr(scales), _ptr(rhs), int(problems), int(records), int(lanes), int(streams),
            _ptr(counts), int(count), _ptr(initial), _ptr(out))
    if _name == "loom_packed_dot":
        _check(_lib.loom_packed_dot(*args, st), _name)
    else:
        tp = ctypes.byref(tuning) if tuning is not None else None
        _check(_lib.loom_packed_dot_ex(*args, _ptr(error), tp, st), _name)
    return out


def loom_sum_rows(values, num_segments: int, seg_stride: int, rows: int, lanes: int, width: int = 1,
                  counts=None, count: int = 0, *, out=None, error=None, tuning=None, stream=None):
    """Per-lane f32 sums (the pages' sum_rows, width 1, and sum_vector_rows, width 4):
    returns ``out`` float32 ``[num_segments][lanes]``."""
    import torch
    if out is None:
        out = _empty(values, (int(num_segments), int(lanes)), torch.float32)
    st = _stream(stream, values)
    args = (_ptr(values), int(num_segments), int(seg_stride), int(rows), int(lanes), int(width), _ptr(counts),
            int(count), _ptr(out))
    if tuning is None and error is None:
        _check(_lib.loom_sum_rows(*args, st), "loom_sum_rows")
    else:
        tp = ctypes.byref(tuning) if tuning is not None else None
        _check(_lib.loom_sum_rows_ex(*args, _ptr(error), tp, st), "loom_sum_rows_ex")
    return out


def loom_sum_guarded_rows(values, num_segments: int, seg_stride: int, rows: int, lanes: int, counts=None,
                          count: int = 0, columns: int = 4, active_lanes: int = 32, *, out=None, error=None,
                          tuning=None, stream=None):
    """The pages' guarded ragged rows over segments ``[rows][lanes][4]``: returns ``out``
    float32 ``[num_segments][lanes]``."""
    import torch
    if out is None:
        out = _empty(values, (int(num_segments), int(lanes)), torch.float32)
    st = _stream(stream, values)
    args = (_ptr(values), int(num_segments), int(seg_stride), int(rows), int(lanes), _ptr(counts), int(count),
            int(columns), int(active_lanes), _ptr(out))
    if tuning is None and error is None:
        _check(_lib.loom_sum_guarded_rows(*args, st), "loom_sum_guarded_rows")
    else:
        tp = ctypes.byref(tuning) if tuning is not None else None
        _check(_lib.loom_sum_guarded_rows_ex(*args, _ptr(error), tp, st), "loom_sum_guarded_rows_ex")
    return out


def loom_routed_combine(ids, weights, payload, *, tokens: int | None = None, routes: int | None = None,
                        rows: int | None = None, width: int | None = None, out=None, error=None, tuning=None,
                        stream=None):
    """Routed row combine: ``out`` float32 ``[tokens][width]`` from ``ids`` int32 and
    ``weights`` float32 ``[tokens][routes]`` (negative id = missing route) and
    ``payload`` float32 ``[rows][width]``."""
    import torch
    if tokens is None or routes is None:
        tokens, routes = ids.shape
    if rows is None or width is None:
        rows, width = payload.shape
    if out is None:
        out = _empty(payload, (int(tokens), int(width)), torch.float32)
    st = _stream(stream, payload)
    args = (_ptr(ids), _ptr(weights), _ptr(payload), int(tokens), int(routes), int(rows), int(width), _ptr(out))
    if tuning is None and error is None:
        _check(_lib.loom_routed_combine(*args, st), "loom_routed_combine")
    else:
        tp = ctypes.byref(tuning) if tuning is not None else None
        _check(_lib.loom_routed_combine_ex(*args, _ptr(error), tp, st), "loom_routed_combine_ex")
    return out


def loom_stage_rows(h_values, d_values, num_segments: int, seg_stride: int, rows: int, lanes: int,
                    counts=None, count: int = 0, *, stream=None):
    """Copy only each segment's first ``counts[s]`` rows from ``h_values`` (pinned host
    memory, or any memory the device can read) to the same offsets of ``d_values``."""
    _check(_lib.loom_stage_rows(_ptr(h_values), _ptr(d_values), int(num_segments), int(seg_stride), int(rows),
                                int(lanes), _ptr(counts), int(count), _stream(stream, d_values)),
           "loom_stage_rows")
    return d_values


def loom_i8_unpack(packed, n_words: int, out=None, *, stream=None):
    """``out[4j+i]`` = signed byte i of word j, as f32."""
    import torch
    if out is None:
        out = _empty(packed, (4 * int(n_words),), torch.float32)
    _check(_lib.loom_i8_unpack(_ptr(packed), int(n_words), _ptr(out), _stream(stream, packed)),
           "loom_i8_unpack")
    return out


def loom_stream_floor(src, nbytes: int, schedule: int, depth: int, ctas_per_sm: int, sink, *, error=None,
                      stream=None):
    """The read-only streaming probe: one launch reading ``nbytes`` at ``src`` (a device
    tensor or address); ``sink`` is a device int64 word."""
    _check(_lib.loom_stream_floor(_ptr(src), int(nbytes), int(schedule), int(depth), int(ctas_per_sm),
                                  _ptr(sink), _ptr(error), _stream(stream, sink)), "loom_stream_floor")


# ---- token operators (loom_token.h) ----------------------------------------------------
# One new token takes a few microseconds on the device, so these calls keep their own work
# short: no context manager unless the device differs, one lookup for the stream.
_torch = None
_dtypes: dict = {}
_current_stream = None      # device index -> handle of torch's current stream
_current_device = None      # -> index of the current device


def _lazy():
    """torch, and what the calls below look up in it, on first use."""
    global _torch, _current_stream, _current_device
    if _torch is None:
        import torch
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _dtypes.update({torch.float32: LOOM_F32, torch.float16: LOOM_F16, torch.bfloat16: LOOM_BF16})
        _torch = torch
    return _torch


def _dtype(dtype) -> int:
    """LOOM_F32 / LOOM_F16 / LOOM_BF16 of a torch dtype."""
    code = _dtypes.get(dtype)
    if code is None:
        raise LoomError(LOOM_ERR_ARG, f"element type {dtype}")
    return code


def _matrix(t, where: str):
    """(rows, width, stride) of a 2-D tensor whose rows are contiguous."""
    shape = t.shape
    if len(shape) == 2:
        rows, width = shape
        stride, inner = t.stride()
        if inner == 1 or width <= 1:
            return rows, width, stride
    raise LoomError(LOOM_ERR_SHAPE, f"{where}: a matrix with contiguous rows is wanted")


def _foreign(where: str, t):
    """A tensor that is not on the call's device: refused, but for pinned host memory, which it reaches."""
    if t.get_device() >= 0 or not t.is_pinned():
        raise LoomError(LOOM_ERR_ARG, f"{where}: a tensor on {t.device}, not on the call's device")


def _floats(where: str, n: int, device: int, *tensors):
    """The optional tensors are contiguous f32 of n elements each, on the call's device."""
    f32 = _torch.float32
    for t in tensors:
        if t is not None:
            if t.dtype is not f32 or t.numel() != n or not t.is_contiguous():
                raise LoomError(LOOM_ERR_SHAPE, f"{where}: {n} contiguous float32 values are wanted")
            if t.get_device() != device:
                _foreign(where, t)


def _like(where: str, name: str, t, x, device: int) -> int:
    """Stride of a matrix `t` of the type and shape of x, on the call's device."""
    if t.dtype != x.dtype or t.shape != x.shape:
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: {name} has another type or shape than x")
    if t.get_device() != device:
        _foreign(where, t)
    return _matrix(t, where)[2]


def _dense(where: str, t, n: int, dtype, device: int):
    """Address of an operand of n contiguous elements (or more) of type `dtype`; None and raw addresses
    stay as they are."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: {n} contiguous {dtype} values are wanted")
    if t.get_device() != device:
        _foreign(where, t)
    return t.data_ptr()


def _packed(where: str, t, nbytes: int, device: int) -> int:
    """Address of `nbytes` contiguous signed bytes (or more), as such or in int32 words; raw addresses stay
    as they are."""
    if isinstance(t, int):
        return t
    dtype = t.dtype
    size = 1 if dtype is _torch.int8 else 4 if dtype is _torch.int32 else 0
    if not size or t.numel() * size < nbytes or not t.is_contiguous():
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: {nbytes} contiguous signed bytes (int8 or int32) are wanted")
    if t.get_device() != device:
        _foreign(where, t)
    return t.data_ptr()


def _new(stream, like, dtype, *shape):
    """An uninitialised tensor on the device of `like` for a call on `stream`.  Of another stream than the
    current one it is taken from that stream's memory, as within torch.cuda.stream(stream): a block of the
    current stream's may still be in use by what is queued there.  It may then be used on the current stream
    too (after a wait, as ever) and given up at any time."""
    empty = _torch.empty
    if stream is None:
        return empty(*shape, dtype=dtype, device=like.device)
    device = like.get_device()
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if device < 0 or handle == _current_stream(device):
        return empty(*shape, dtype=dtype, device=like.device)
    cuda = _torch.cuda
    with cuda.stream(cuda.ExternalStream(handle, device=like.device)):
        t = empty(*shape, dtype=dtype, device=like.device)
    t.record_stream(cuda.current_stream(device))
    return t


def _launch(where: str, like, stream, *args):
    """The library call `where` on the device of `like` and on `stream` (its current one)."""
    fn = getattr(_lib, where)
    device = like.get_device()
    if device < 0:
        raise LoomError(LOOM_ERR_ARG, f"{where}: tensors on a GPU are wanted")
    if stream is None:
        stream = _current_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == device:
        status = fn(*args, stream)
    else:
        with _torch.cuda.device(device):
            status = fn(*args, stream)
    if status != LOOM_OK:
        raise LoomError(status, where)


def loom_token_launch_config(op: int, workload) -> dict:
    arr = (ctypes.c_int64 * max(1, len(workload)))(*[int(v) for v in workload])
    out = loom_launch()
    _check(_lib.loom_token_launch_config(int(op), arr, len(workload), ctypes.byref(out)), "loom_token_launch_config")
    return out.as_dict()


def loom_quantize_tokens(x, *, q=None, scale=None, error=None, stream=None):
    """Tokens ``x[tokens][k]`` (float32, float16 or bfloat16) to signed bytes with one scale
    each; returns ``(q_packed int32 [tokens][k/4], scale float32 [tokens])``."""
    torch = _torch or _lazy()
    where = "loom_quantize_tokens"
    tokens, k, stride = _matrix(x, where)
    dtype = _dtype(x.dtype)
    q, q_at, scale, scale_at, error = _byte_outputs(where, stream, x, tokens, k, q, scale, error)
    _launch(where, x, stream, x.data_ptr(), dtype, tokens, k, stride, q_at, scale_at, error)
    return q, scale


def _byte_outputs(where, stream, x, tokens, k, q, scale, error):
    """(q, its address, scale, its address, the error word's address) of a call to bytes."""
    torch = _torch
    device = x.get_device()
    if q is None:
        q = _new(stream, x, torch.int32, tokens, k // 4)
        q_at = q.data_ptr()
    else:
        q_at = _packed(where, q, tokens * k, device)
    if scale is None:
        scale = _new(stream, x, torch.float32, tokens)
        scale_at = scale.data_ptr()
    else:
        scale_at = _dense(where, scale, tokens, torch.float32, device)
    return q, q_at, scale, scale_at, _dense(where, error, 1, torch.int32, device)


def loom_i8_matmul(w_packed, scale_w, n_rows: int, k: int, x_packed, scale_x, tokens: int, *, bias=None, y=None,
                   y_dtype=None, acc=None, want_acc: bool = False, stream=None):
    """``y[tokens][n_rows]`` of type ``y_dtype`` (float32 by default; the type of ``y`` where it
    is given) and, when requested, ``acc`` int32; returns ``(y, acc)``.  ``w_packed`` and
    ``x_packed`` hold the signed bytes row after row (int8 tensors, or their int32 words)."""
    return _i8_matmul("loom_i8_matmul", w_packed, scale_w, n_rows, k, x_packed, scale_x, tokens, bias, y, y_dtype, acc,
                      want_acc, stream)


def loom_i8_matmul_ex(w_packed, scale_w, n_rows: int, k: int, x_packed, scale_x, tokens: int, *, bias=None, y=None,
                      y_dtype=None, acc=None, want_acc: bool = False, error=None, tuning=None, stream=None):
    tp = ctypes.byref(tuning) if tuning is not None else None
    if error is not None:
        _lazy()
        error = _dense("loom_i8_matmul_ex", error, 1, _torch.int32, w_packed.get_device())
    return _i8_matmul("loom_i8_matmul_ex", w_packed, scale_w, n_rows, k, x_packed, scale_x, tokens, bias, y, y_dtype, acc,
                      want_acc, stream, error, tp)


def _i8_matmul(where, w_packed, scale_w, n_rows, k, x_packed, scale_x, tokens, bias, y, y_dtype, acc, want_acc, stream, *more):
    torch = _torch or _lazy()
    device = w_packed.get_device()
    if y is None:
        if tokens < 0 or n_rows < 0:
            raise LoomError(LOOM_ERR_SHAPE, where)
        y = _new(stream, w_packed, torch.float32 if y_dtype is None else y_dtype, tokens, n_rows)
        stride = n_rows
    else:
        rows, width, stride = _matrix(y, where)
        if rows < tokens or width < n_rows:
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: y is smaller than {tokens} x {n_rows}")
        if y.get_device() != device:
            _foreign(where, y)
    if acc is not None:
        acc_at = _dense(where, acc, tokens * n_rows, torch.int32, device)
    elif want_acc:
        acc = _new(stream, w_packed, torch.int32, tokens, n_rows)
        acc_at = acc.data_ptr()
    else:
        acc_at = None
    f32, work = torch.float32, tokens > 0 and n_rows > 0       # (without work the operands may be empty)
    _launch(where, w_packed, stream, _packed(where, w_packed, n_rows * k if work else 0, device),
            _dense(where, scale_w, n_rows if work else 0, f32, device), n_rows, k,
            _packed(where, x_packed, tokens * k if work else 0, device), _dense(where, scale_x, tokens if work else 0, f32, device), tokens,
            _dense(where, bias, n_rows if work else 0, f32, device), y.data_ptr(), _dtype(y.dtype), stride, acc_at, *more)
    return y, acc


def loom_layer_norm(x, gain=None, bias=None, eps: float = 1e-5, *, y=None, mean=None, rstd=None,
                    want_stats: bool = True, stream=None):
    """Layer norm of the rows of ``x`` (float32, float16 or bfloat16); ``gain`` and ``bias``
    float32 or None.  Returns ``(y, mean, rstd)``, the last two float32 per row as the
    backward pass takes them (None without ``want_stats``)."""
    torch = _torch or _lazy()
    where = "loom_layer_norm"
    rows, width, stride = _matrix(x, where)
    dtype, device = _dtype(x.dtype), x.get_device()
    _floats(where, width, device, gain, bias)
    if y is None:
        y = _new(stream, x, x.dtype, rows, width)
        y_stride = width
    else:
        y_stride = _like(where, "y", y, x, device)
    mean_at, rstd_at = _dense(where, mean, rows, torch.float32, device), _dense(where, rstd, rows, torch.float32, device)
    if want_stats:
        if mean is None:
            mean = _new(stream, x, torch.float32, rows)
            mean_at = mean.data_ptr()
        if rstd is None:
            rstd = _new(stream, x, torch.float32, rows)
            rstd_at = rstd.data_ptr()
    _launch(where, x, stream, x.data_ptr(), dtype, rows, width, stride, _ptr(gain), _ptr(bias), eps, y.data_ptr(),
            y_stride, mean_at, rstd_at)
    return y, mean, rstd


def loom_layer_norm_i8(x, gain=None, bias=None, eps: float = 1e-5, *, q=None, scale=None, error=None, stream=None):
    """``loom_quantize_tokens`` of layer norm's rows, which are never written; returns
    ``(q_packed, scale)``."""
    torch = _torch or _lazy()
    where = "loom_layer_norm_i8"
    rows, width, stride = _matrix(x, where)
    dtype = _dtype(x.dtype)
    _floats(where, width, x.get_device(), gain, bias)
    q, q_at, scale, scale_at, error = _byte_outputs(where, stream, x, rows, width, q, scale, error)
    _launch(where, x, stream, x.data_ptr(), dtype, rows, width, stride, _ptr(gain), _ptr(bias), eps, q_at, scale_at, error)
    return q, scale


def loom_layer_norm_backward_workspace_bytes(rows: int, width: int) -> int:
    """Bytes of the workspace of ``loom_layer_norm_backward`` on the current device."""
    out = ctypes.c_int64(0)
    _check(_lib.loom_layer_norm_backward_workspace_bytes(rows, width, ctypes.byref(out)),
           "loom_layer_norm_backward_workspace_bytes")
    return out.value


def loom_layer_norm_backward(dy, x, mean, rstd, gain=None, *, dx=None, dgain=None, dbias=None, want_dx: bool = True,
                             want_params: bool = True, workspace=AUTO, stream=None):
    """Gradients of layer norm: ``(dx, dgain, dbias)`` from ``dy`` and ``x`` (same type), the
    forward pass's ``mean`` and ``rstd``, and ``gain``.  ``want_dx`` / ``want_params`` leave
    out what is not needed (None).  ``workspace``: a tensor, an ``(address, bytes)`` pair, None,
    or "auto" (taken for the call from torch's allocator)."""
    torch = _torch or _lazy()
    where = "loom_layer_norm_backward"
    rows, width, x_stride = _matrix(x, where)
    dtype = _dtype(x.dtype)
    device, index = x.device, x.get_device()
    dy_stride = _like(where, "dy", dy, x, index)
    _floats(where, width, index, gain, dgain, dbias)
    _floats(where, rows, index, mean, rstd)
    dx_stride = width
    if dx is not None:
        dx_stride = _like(where, "dx", dx, x, index)
    elif want_dx:
        dx = _new(stream, x, x.dtype, rows, width)
    if want_params:
        if dgain is None:
            dgain = _new(stream, x, torch.float32, width)
        if dbias is None:
            dbias = _new(stream, x, torch.float32, width)
    if workspace is None or (dgain is None and dbias is None):      # dx alone needs none
        wp, wb = None, 0
    elif isinstance(workspace, tuple):
        wp, wb = workspace
    else:
        if workspace is AUTO or (isinstance(workspace, str) and workspace == AUTO):
            if index < 0:
                raise LoomError(LOOM_ERR_ARG, f"{where}: tensors on a GPU are wanted")
            if index == _current_device():
                nbytes = loom_layer_norm_backward_workspace_bytes(rows, width)
            else:
                with torch.cuda.device(device):
                    nbytes = loom_layer_norm_backward_workspace_bytes(rows, width)
            workspace = _new(stream, x, torch.uint8, nbytes)
        else:
            _dense(where, workspace, 0, workspace.dtype, index)
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(where, x, stream, dy.data_ptr(), dy_stride, x.data_ptr(), x_stride, dtype, rows, width, _ptr(gain), mean.data_ptr(),
            rstd.data_ptr(), _ptr(dx), dx_stride, _ptr(dgain), _ptr(dbias), wp, wb)
    return dx, dgain, dbias


def _setting(name: str, v, dtype, rows: int, device: int, where: str = "loom_sample_tokens"):
    """(device address or None, host value) of a setting that rows may have one by one."""
    if isinstance(v, _torch.Tensor):
        if v.dtype != dtype or v.numel() != rows or not v.is_contiguous():
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: {name}: {rows} contiguous {dtype} values are wanted")
        if v.get_device() != device:
            _foreign(f"{where}: {name}", v)
        return v.data_ptr(), 0
    return None, v


def loom_sample_tokens(logits, uniform, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, logprob=None,
                       want_logprob: bool = True, error=None, stream=None):
    """The next token of each row of ``logits[rows][vocab]`` from ``uniform`` float32 ``[rows]``
    in [0, 1); each setting is a number for every row or a device tensor with one per row
    (``top_k`` int32, the others float32).  Returns ``(token int32, logprob float32)``."""
    torch = _torch or _lazy()
    where = "loom_sample_tokens"
    rows, vocab, stride = _matrix(logits, where)
    dtype, device = _dtype(logits.dtype), logits.get_device()
    _floats(where, rows, device, uniform)
    dt, t = _setting("temperature", temperature, torch.float32, rows, device)
    dk, k = _setting("top_k", top_k, torch.int32, rows, device)
    dp, p = _setting("top_p", top_p, torch.float32, rows, device)
    dm, m = _setting("min_p", min_p, torch.float32, rows, device)
    if token is None:
        token = _new(stream, logits, torch.int32, rows)
        token_at = token.data_ptr()
    else:
        token_at = _dense(where, token, rows, torch.int32, device)
    if logprob is None and want_logprob:
        logprob = _new(stream, logits, torch.float32, rows)
        logprob_at = logprob.data_ptr()
    else:
        logprob_at = _dense(where, logprob, rows, torch.float32, device)
    _launch(where, logits, stream, logits.data_ptr(), dtype, rows, vocab, stride, dt, t, dk, k, dp, p, dm, m,
            uniform.data_ptr(), token_at, logprob_at, _dense(where, error, 1, torch.int32, device))
    return token, logprob


def loom_adjust_logits(logits, *, history=None, lengths=None, prompts=None, repetition=1.0, frequency=0.0, presence=0.0,
                       bias_ids=None, bias_values=None, mask=None, mask_rows=None, y=None, error=None, stream=None):
    """``logits[rows][vocab]`` with penalties for the tokens of ``history`` (int32 ``[rows][n]``, the first
    ``lengths[row]`` of them, of which the first ``prompts[row]`` count for ``repetition`` alone), biases
    (``bias_ids`` int32 and ``bias_values`` float32 ``[rows][m]``) and a grammar's ``mask`` (int32
    ``[masks][ceil(vocab / 32)]`` bits; ``mask_rows`` int32 ``[rows]``, negative for none).  A penalty is a number
    for every row or a device tensor with one per row.  Returns ``y``, which may be ``logits``."""
    torch = _torch or _lazy()
    where = "loom_adjust_logits"
    rows, vocab, stride = _matrix(logits, where)
    dtype, device = _dtype(logits.dtype), logits.get_device()
    i32, f32 = torch.int32, torch.float32
    n = history_stride = 0
    if history is not None:
        if history.dtype is not i32:
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: history: int32 tokens are wanted")
        if history.get_device() != device:
            _foreign(where, history)
        of, n, history_stride = _matrix(history, where)
        if of != rows:
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: history: {rows} rows are wanted")
    m = 0
    if bias_ids is not None or bias_values is not None:
        if bias_ids is None or bias_values is None:
            raise LoomError(LOOM_ERR_NULL, f"{where}: bias_ids and bias_values come together")
        m = bias_ids.shape[-1] if bias_ids.dim() == 2 else -1
        if tuple(bias_ids.shape) != (rows, m) or bias_values.shape != bias_ids.shape:
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: bias_ids and bias_values: {rows} rows of one length are wanted")
    masks = 0
    if mask is not None:
        masks, words = mask.shape if mask.dim() == 2 else (0, -1)
        if words != (vocab + 31) // 32:
            raise LoomError(LOOM_ERR_SHAPE, f"{where}: mask: rows of {(vocab + 31) // 32} words are wanted")
    dr, r = _setting("repetition", repetition, f32, rows, device, where)
    df, f = _setting("frequency", frequency, f32, rows, device, where)
    dp, p = _setting("presence", presence, f32, rows, device, where)
    if y is None:
        y = _new(stream, logits, logits.dtype, rows, vocab)
        y_stride = vocab
    else:
        y_stride = _like(where, "y", y, logits, device)
    _launch(where, logits, stream, logits.data_ptr(), dtype, rows, vocab, stride, _ptr(history), n, history_stride,
            _dense(where, lengths, rows, i32, device), _dense(where, prompts, rows, i32, device), dr, r, df, f, dp, p,
            _dense(where, bias_ids, rows * m, i32, device), _dense(where, bias_values, rows * m, f32, device), m,
            _dense(where, mask, 0, i32, device), masks, _dense(where, mask_rows, rows, i32, device), y.data_ptr(), y_stride,
            _dense(where, error, 1, i32, device))
    return y


def _i4_operands(where, w_packed, scale_w, matrices, n_rows, k, group, x_packed, scale_x, x_rows, bias, work, device):
    """Addresses of a 4-bit product's operands: (weights, scales, their type, tokens, their scales, bias)."""
    groups = -(-k // group) if group > 0 else 0
    rows = matrices * n_rows if work else 0          # (without work the operands may be empty)
    f32, i32 = _torch.float32, _torch.int32
    return (_dense(where, w_packed, rows * (k // 8), i32, device), _dense(where, scale_w, rows * groups, scale_w.dtype, device),
            _dtype(scale_w.dtype), _packed(where, x_packed, x_rows * k if work else 0, device),
            _dense(where, scale_x, x_rows if work else 0, f32, device), _dense(where, bias, rows, f32, device))


def _product_output(where, stream, y, y_dtype, like, rows, n_rows, device):
    """(y, its stride) of a product's rows."""
    if y is None:
        if rows < 0 or n_rows < 0:
            raise LoomError(LOOM_ERR_SHAPE, where)
        return _new(stream, like, _torch.float32 if y_dtype is None else y_dtype, rows, n_rows), n_rows
    have, width, stride = _matrix(y, where)
    if have < rows or width < n_rows:
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: y is smaller than {rows} x {n_rows}")
    if y.get_device() != device:
        _foreign(where, y)
    return y, stride


def loom_i4_matvec(w_packed, scale_w, n_rows: int, k: int, group: int, x_packed, scale_x, tokens: int, *, bias=None, y=None,
                   y_dtype=None, stream=None):
    """``y[tokens][n_rows]`` of type ``y_dtype`` (float32 by default) from 4-bit weights ``w_packed`` (int32, eight
    signed nibbles a word, row after row) with a scale of ``scale_w`` (float32, float16 or bfloat16
    ``[n_rows][ceil(k / group)]``) for each ``group`` of a row, and 8-bit tokens as of ``loom_quantize_tokens``."""
    _torch or _lazy()
    where = "loom_i4_matvec"
    device = w_packed.get_device()
    y, y_stride = _product_output(where, stream, y, y_dtype, w_packed, tokens, n_rows, device)
    w, s, s_dtype, x, sx, b = _i4_operands(where, w_packed, scale_w, 1, n_rows, k, group, x_packed, scale_x, tokens, bias,
                                           tokens > 0 and n_rows > 0, device)
    _launch(where, w_packed, stream, w, s, s_dtype, n_rows, k, group, x, sx, tokens, b, y.data_ptr(), _dtype(y.dtype), y_stride)
    return y


def loom_i4_matvec_routed(w_packed, scale_w, experts: int, n_rows: int, k: int, group: int, x_packed, scale_x, ids, *,
                          x_rows: int | None = None, bias=None, y=None, y_dtype=None, error=None, stream=None):
    """The products of ``loom_i4_matvec`` with the matrix ``ids[t][j]`` of ``experts`` for each pair: ``y[tokens *
    routes][n_rows]`` (zeros for a negative id), the payload of ``loom_routed_combine``.  ``ids`` int32
    ``[tokens][routes]``; ``x_rows``: ``tokens`` (the default) where a token's routes share its row of
    ``x_packed``, or ``tokens * routes``."""
    torch = _torch or _lazy()
    where = "loom_i4_matvec_routed"
    if ids.dim() != 2:
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: ids: [tokens][routes] are wanted")
    tokens, routes = ids.shape
    device = w_packed.get_device()
    if x_rows is None:
        x_rows = tokens
    y, y_stride = _product_output(where, stream, y, y_dtype, w_packed, tokens * routes, n_rows, device)
    w, s, s_dtype, x, sx, b = _i4_operands(where, w_packed, scale_w, experts, n_rows, k, group, x_packed, scale_x, x_rows, bias,
                                           tokens > 0 and routes > 0 and n_rows > 0, device)
    _launch(where, w_packed, stream, w, s, s_dtype, experts, n_rows, k, group, x, sx, x_rows,
            _dense(where, ids, tokens * routes, torch.int32, device), tokens, routes, b, y.data_ptr(), _dtype(y.dtype), y_stride,
            _dense(where, error, 1, torch.int32, device))
    return y


_SCORES = {"softmax": LOOM_SCORE_SOFTMAX, "sigmoid": LOOM_SCORE_SIGMOID, LOOM_SCORE_SOFTMAX: LOOM_SCORE_SOFTMAX,
           LOOM_SCORE_SIGMOID: LOOM_SCORE_SIGMOID}


def _score(where: str, score) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise LoomError(LOOM_ERR_ARG, f"{where}: score {score!r}")
    return code


def loom_route_tokens(logits, top_k: int, *, score="softmax", bias=None, groups: int = 1, top_groups: int | None = None,
                      group_best: int = 1, renormalise: bool = True, factor: float = 1.0, ids=None, weights=None, counts=None,
                      stream=None):
    """The ``top_k`` experts of each row of ``logits[tokens][experts]`` and their weights; returns ``(ids int32,
    weights float32)``, ``[tokens][top_k]``, as ``loom_routed_combine`` takes them.  ``score`` "softmax" or
    "sigmoid" (or LOOM_SCORE_*); ``bias`` float32 ``[experts]`` counts for the choice alone; of ``groups`` equal runs of experts the best
    ``top_groups`` (by their ``group_best`` best experts) stay; ``counts`` int32 ``[experts]`` is added to."""
    torch = _torch or _lazy()
    where = "loom_route_tokens"
    tokens, experts, stride = _matrix(logits, where)
    dtype, device = _dtype(logits.dtype), logits.get_device()
    if bias is not None:
        _floats(where, experts, device, bias)
    if ids is None:
        ids = _new(stream, logits, torch.int32, tokens, max(top_k, 0))
    if weights is None:
        weights = _new(stream, logits, torch.float32, tokens, max(top_k, 0))
    _launch(where, logits, stream, logits.data_ptr(), dtype, tokens, experts, stride, _ptr(bias), _score(where, score), groups,
            groups if top_groups is None else top_groups, group_best, top_k, renormalise, factor,
            _dense(where, ids, tokens * top_k, torch.int32, device), _dense(where, weights, tokens * top_k, torch.float32, device),
            _dense(where, counts, experts, torch.int32, device))
    return ids, weights


def loom_route_tokens_backward(dweights, logits, ids, *, score="softmax", renormalise: bool = True, factor: float = 1.0,
                               dlogits=None, error=None, stream=None):
    """The gradient of ``loom_route_tokens``'s weights to its logits, the choice ``ids`` held fixed, from ``dweights``
    float32 ``[tokens][top_k]``; returns ``dlogits`` of the logits' type."""
    torch = _torch or _lazy()
    where = "loom_route_tokens_backward"
    tokens, experts, stride = _matrix(logits, where)
    dtype, device = _dtype(logits.dtype), logits.get_device()
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise LoomError(LOOM_ERR_SHAPE, f"{where}: ids: {tokens} rows are wanted")
    top_k = ids.shape[1]
    if dlogits is None:
        dlogits = _new(stream, logits, logits.dtype, tokens, experts)
        dstride = experts
    else:
        dstride = _like(where, "dlogits", dlogits, logits, device)
    _launch(where, logits, stream, _dense(where, dweights, tokens * top_k, torch.float32, device), logits.data_ptr(), dtype, tokens,
            experts, stride, _dense(where, ids, tokens * top_k, torch.int32, device), _score(where, score), top_k, renormalise,
            factor, dlogits.data_ptr(), dstride, _dense(where, error, 1, torch.int32, device))
    return dlogits
