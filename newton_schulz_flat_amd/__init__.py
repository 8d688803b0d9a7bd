"""MI355X (gfx950) Muon optimizer step over flat buffers.

A thin ctypes binding of ``libmuon_step.so`` (C ABI in ``include/muon_step.h``).
It only marshals arguments: every step of the computation runs in the
library's HIP kernels.  PyTorch provides device memory and the current
stream.  If the library is missing, every entry point raises: there is no
fallback.

Entry points (same names as the C ABI):

``muon_step``           momentum, Nesterov input, Newton-Schulz, decay + apply
``muon_step_noalloc``   ``muon_step`` without workspace or device allocation
``muon_step_grouped``   the same with per-matrix optimizer groups read from a
                        device table (graph-capturable) and an optional
                        bfloat16 copy of float32 weights
``muon_momentum``       momentum update and orthogonalization input only
``muon_orthogonalize``  Newton-Schulz orthogonalization (with shape scale) only
``muon_apply``          decoupled decay and update, scattered into slices
``muon_step_clipped``   ``muon_step_grouped`` on the clipped gradient
``muon_grad_norm``      global 2-norm of many tensors and the clipping coefficient
``muon_clip_grads``     every tensor times the coefficient, in place or into others
``muon_clip_finish``    norm and coefficient from a record's (all-reduced) sum of squares
``muon_adamw``          AdamW on ranges of flat buffers, for the parameters Muon skips
``muon_fp8_cast``       a matrix and its transpose into 8 bits, a scale for each block of 128
``muon_fp8_matmul``     product of two such matrices, also added into float32 gradients
``muon_orthogonalize_stack``  Newton-Schulz of stacked matrices with strides, in float32
                        accuracy, with coefficients for each step
``muon_workspace_bytes``      workspace for one wave
``muon_workspace_min_bytes``  smallest workspace (the matrices then run in waves)

Descriptors are objects with ``offset, rows, cols`` and optionally
``param_offset`` (default ``offset``), ``shard_stride`` (0), ``n_shards`` (1)
and ``group`` (0), or tuples in that field order.  Ranges (``muon_adamw``) are
objects with ``offset, numel`` and optionally ``param_offset`` (default
``offset``) and ``group`` (0), or tuples in that field order.

A training step clips by the global norm without a word to the host::

    clip = clip_state(device)                       # kept
    tensors = tensor_list([*matrix_grads, *other_grads])    # kept while they stay where they are
    muon_grad_norm(tensors, 1.0, clip)
    muon_step_clipped(params, grads, momentum, descs, groups, clip)
    muon_adamw(other_params, other_grads, m, v, ranges, adamw_groups, clip=clip)
    adamw_steps(adamw_groups).add_(1)

Where ranks hold parts of the gradient, ``dist.all_reduce(clip_sumsq(clip))`` and
``muon_clip_finish(clip, 1.0)`` come after the norm.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Iterable, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuon_step.so")

MUON_OK = 0
MUON_DTYPE_F32 = 0
MUON_DTYPE_BF16 = 1
MUON_GEMM_BF16_MFMA = 0
MUON_GEMM_F32 = 1
_MODES = {"bf16": MUON_GEMM_BF16_MFMA, "f32": MUON_GEMM_F32}

#: C names of every exported entry point (mirrors include/muon_step.h).
EXPORTS = ("muon_workspace_bytes", "muon_workspace_min_bytes", "muon_step", "muon_step_grouped",
           "muon_step_noalloc", "muon_step_clipped", "muon_momentum", "muon_orthogonalize",
           "muon_apply", "muon_clip_workspace_bytes", "muon_grad_norm", "muon_clip_finish",
           "muon_clip_grads", "muon_adamw", "muon_fp8_cast", "muon_fp8_workspace_bytes",
           "muon_fp8_matmul", "muon_stack_workspace_bytes", "muon_orthogonalize_stack",
           "muon_profile_begin", "muon_profile_end", "muon_status_string", "muon_last_error")


class MatrixDescC(ctypes.Structure):
    """``muon_matrix_desc_t``."""

    _fields_ = [("offset", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("param_offset", ctypes.c_int64), ("shard_stride", ctypes.c_int64),
                ("n_shards", ctypes.c_int32), ("group", ctypes.c_int32)]


class TensorC(ctypes.Structure):
    """``muon_tensor_t``."""

    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RangeC(ctypes.Structure):
    """``muon_range_t``."""

    _fields_ = [("offset", ctypes.c_int64), ("numel", ctypes.c_int64),
                ("param_offset", ctypes.c_int64), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Fp8C(ctypes.Structure):
    """``muon_fp8_t``."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("scale_row", ctypes.c_int64), ("scale_col", ctypes.c_int64),
                ("format", ctypes.c_int32), ("block_rows", ctypes.c_int32)]


class StackC(ctypes.Structure):
    """``muon_stack_t``."""

    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("in_stride", ctypes.c_int64),
                ("in_row", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("out_row", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class KernelTimeC(ctypes.Structure):
    """``muon_kernel_time_t``."""

    _fields_ = [("name", ctypes.c_char * 48), ("total_ms", ctypes.c_double),
                ("launches", ctypes.c_int64)]


class MuonError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, status: int, name: str, message: str):
        super().__init__(f"{name}: {message}")
        self.status = status
        self.name = name


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m newton_schulz_flat_amd.build` (no fallback exists)")
    lib = ctypes.CDLL(path)
    p, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                            ctypes.c_size_t)
    dp = ctypes.POINTER(MatrixDescC)
    lib.muon_workspace_bytes.argtypes = [dp, i64, i32, ctypes.POINTER(sz)]
    lib.muon_workspace_min_bytes.argtypes = [dp, i64, i32, ctypes.POINTER(sz)]
    lib.muon_step.argtypes = [p, i32, i64, p, p, i64, dp, i64, f32, f32, f32, i32, i32, i32, p,
                              sz, p]
    lib.muon_step_grouped.argtypes = [p, i32, i64, p, p, p, i64, dp, i64, p, ctypes.c_int32, i32,
                                      i32, p, sz, p]
    lib.muon_step_noalloc.argtypes = [p, i32, i64, p, p, i64, dp, i64, f32, f32, f32, i32, i32,
                                      i32, p]
    lib.muon_momentum.argtypes = [p, p, p, i64, dp, i64, f32, i32, p]
    lib.muon_orthogonalize.argtypes = [p, p, i64, dp, i64, i32, i32, p, sz, p]
    lib.muon_apply.argtypes = [p, i32, i64, p, i64, dp, i64, f32, f32, p]
    tp = ctypes.POINTER(TensorC)
    lib.muon_step_clipped.argtypes = [p, i32, i64, p, p, p, i64, dp, i64, p, ctypes.c_int32, p,
                                      i32, i32, p, sz, p]
    lib.muon_clip_workspace_bytes.argtypes = [tp, i64, ctypes.POINTER(sz)]
    lib.muon_grad_norm.argtypes = [tp, i64, f32, p, p, p, sz, p]
    lib.muon_clip_finish.argtypes = [p, f32, p]
    lib.muon_clip_grads.argtypes = [tp, tp, i64, p, p]
    lib.muon_adamw.argtypes = [p, i32, i64, p, p, i32, p, p, i64, ctypes.POINTER(RangeC), i64, p,
                               ctypes.c_int32, p, p]
    fp, sp = ctypes.POINTER(Fp8C), ctypes.POINTER(StackC)
    lib.muon_fp8_cast.argtypes = [p, i32, i64, i64, i64, fp, fp, p]
    lib.muon_fp8_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    lib.muon_fp8_matmul.argtypes = [fp, fp, p, i32, i64, i32, p, sz, p]
    lib.muon_stack_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.muon_orthogonalize_stack.argtypes = [sp, ctypes.POINTER(f32), i32, f32, p, sz, p]
    lib.muon_profile_begin.argtypes = []
    lib.muon_profile_end.argtypes = [ctypes.POINTER(KernelTimeC), i32, ctypes.POINTER(i32)]
    lib.muon_status_string.argtypes = [i32]
    lib.muon_status_string.restype = ctypes.c_char_p
    lib.muon_last_error.argtypes = []
    lib.muon_last_error.restype = ctypes.c_char_p
    for name in ("muon_workspace_bytes", "muon_workspace_min_bytes", "muon_step",
                 "muon_step_grouped", "muon_step_noalloc", "muon_momentum", "muon_orthogonalize",
                 "muon_apply", "muon_step_clipped", "muon_clip_workspace_bytes",
                 "muon_grad_norm", "muon_clip_finish", "muon_clip_grads", "muon_adamw",
                 "muon_fp8_cast", "muon_fp8_workspace_bytes", "muon_fp8_matmul",
                 "muon_stack_workspace_bytes", "muon_orthogonalize_stack",
                 "muon_profile_begin", "muon_profile_end"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def check(status: int) -> None:
    """Raise MuonError for a non-zero status."""
    if status != MUON_OK:
        lib = load_library()
        raise MuonError(status, lib.muon_status_string(status).decode(),
                        lib.muon_last_error().decode())


def descs_array(descs: Iterable) -> ctypes.Array:
    """Descriptors as a ``muon_matrix_desc_t`` array."""
    items = list(descs)
    arr = (MatrixDescC * max(1, len(items)))()
    for k, d in enumerate(items):
        if isinstance(d, (tuple, list)):
            vals = list(d) + [None] * (7 - len(d))
            off, rows, cols, poff, stride, shards, group = vals[:7]
        else:
            off, rows, cols = d.offset, d.rows, d.cols
            poff = getattr(d, "param_offset", None)
            stride = getattr(d, "shard_stride", None)
            shards = getattr(d, "n_shards", None)
            group = getattr(d, "group", None)
        arr[k] = MatrixDescC(int(off), int(rows), int(cols), int(off if poff is None else poff),
                             int(stride or 0), int(1 if shards is None else shards),
                             int(group or 0))
    return arr


def _listed(descs) -> Sequence:
    """Descriptors as something that can be read more than once, with a length."""
    return descs if isinstance(descs, Sequence) else list(descs)


def _mode(mode: str) -> int:
    try:
        return _MODES[mode]
    except KeyError:
        raise ValueError(f"mode must be one of {sorted(_MODES)}, got {mode!r}") from None


def _launch(index: int, call, *args) -> None:
    """``call(*args, stream)`` on the current stream of GPU ``index``.  Launches go to the
    current device, which another one than ``index`` gives way for the call."""
    import torch
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            check(call(*args, _current_stream(index)))
    else:
        check(call(*args, _current_stream(index)))


def _current_stream(index: int) -> int:
    """Handle of the current stream, without the stream object that
    ``torch.cuda.current_stream`` makes around it (1 us a call)."""
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(index)
    except AttributeError:
        return torch.cuda.current_stream(index).cuda_stream


def _require(t, name, dtypes):
    import torch
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _together(first, first_name: str, **others) -> None:
    """Refuses tensors on another device than ``first``."""
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, {first_name} on {first.device}")


def _shorter(a, b, *more) -> int:
    """Elements that all state buffers have: the bound against which the library checks
    the matrices."""
    return min(t.numel() for t in (a, b, *more))


def muon_workspace_bytes(descs, mode: str = "bf16") -> int:
    """Workspace bytes with which the descriptors run in one wave."""
    lib = load_library()
    descs = _listed(descs)
    arr = descs_array(descs)
    out = ctypes.c_size_t(0)
    check(lib.muon_workspace_bytes(arr, len(descs), _mode(mode), ctypes.byref(out)))
    return out.value


def muon_workspace_min_bytes(descs, mode: str = "bf16") -> int:
    """Smallest workspace that runs the descriptors (in waves, one matrix or more each)."""
    lib = load_library()
    descs = _listed(descs)
    arr = descs_array(descs)
    out = ctypes.c_size_t(0)
    check(lib.muon_workspace_min_bytes(arr, len(descs), _mode(mode), ctypes.byref(out)))
    return out.value


#: Default workspaces, one per (device, stream): calls sharing a workspace must
#: be ordered on one stream.  Each is allocated on the stream it serves, so the
#: caching allocator hands a replaced (smaller) one out again only in that
#: stream's order.
_workspaces: dict = {}


def _capturing(dev) -> bool:
    """Whether the current stream of ``dev``, or that of the current device, is being captured."""
    import torch
    if torch.cuda.is_current_stream_capturing():
        return True
    if dev.index is None or dev.index == torch.cuda.current_device():
        return False
    with torch.cuda.device(dev):
        return torch.cuda.is_current_stream_capturing()


def workspace_for(descs, mode: str, device):
    """A cached uint8 workspace of at least the one-wave size, for the current
    stream of ``device``.  Not usable under graph capture (the graph would keep
    a pointer that a later, larger set frees): pass an explicit workspace there."""
    import torch
    dev = torch.device(device)
    if _capturing(dev):
        raise RuntimeError("pass an explicit workspace to calls made under graph capture")
    stream = torch.cuda.current_stream(dev)
    need = muon_workspace_bytes(descs, mode)
    key = (dev, stream.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        _workspaces.pop(key, None)
        with torch.cuda.stream(stream):
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


#: Locks of the default workspaces, one per (device, stream).  A call is several
#: launches that hand results on through its workspace, and threads on one
#: stream share the default one: each enqueues its whole call under the lock, so that
#: stream order keeps calls apart as well as launches.
_stream_locks: dict = {}


def _stream_lock(device):
    import torch
    key = (device, torch.cuda.current_stream(device).cuda_stream)
    return _stream_locks.setdefault(key, threading.RLock())


@contextlib.contextmanager
def _workspace(given, descs, mode, device):
    """The workspace of a call that is enqueued inside this context: ``given``, or the default
    one under its lock."""
    if given is not None:
        if given.device != device:
            raise ValueError(f"workspace is on {given.device}, the tensors on {device}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        yield given
    else:
        with _stream_lock(device):
            yield workspace_for(descs, mode, device)


def muon_step(params, grads, momentum, descs, lr: float, weight_decay: float, beta: float,
              nesterov: bool = True, ns_steps: int = 5, mode: str = "bf16", workspace=None):
    """One Muon step in place on ``params`` (f32 or bf16) and ``momentum`` (f32).

    ``workspace``: a uint8 GPU tensor (default: a cached one per device and
    stream, of the one-wave size).  A workspace smaller than
    ``muon_workspace_bytes`` but at least ``muon_workspace_min_bytes`` runs the
    matrices in waves that fit it, with identical results."""
    import torch
    _require(params, "params", (torch.float32, torch.bfloat16))
    _require(grads, "grads", (torch.float32,))
    _require(momentum, "momentum", (torch.float32,))
    _together(grads, "grads", params=params, momentum=momentum)
    descs, lib = _listed(descs), load_library()
    dt = MUON_DTYPE_BF16 if params.dtype == torch.bfloat16 else MUON_DTYPE_F32
    with _workspace(workspace, descs, mode, grads.device) as ws:
        _launch(grads.get_device(), lib.muon_step, params.data_ptr(), dt, params.numel(),
                grads.data_ptr(), momentum.data_ptr(), _shorter(grads, momentum),
                descs_array(descs), len(descs), lr, weight_decay, beta, int(bool(nesterov)),
                int(ns_steps), _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size())


def muon_step_noalloc(params, grads, momentum, descs, lr: float, weight_decay: float,
                      beta: float, nesterov: bool = True, ns_steps: int = 5, mode: str = "bf16"):
    """``muon_step`` without a workspace and without any device allocation:
    the library's fixed per-GPU scratch array holds every intermediate.  Calls
    that overlap on one GPU race (they share the array)."""
    import torch
    _require(params, "params", (torch.float32, torch.bfloat16))
    _require(grads, "grads", (torch.float32,))
    _require(momentum, "momentum", (torch.float32,))
    _together(grads, "grads", params=params, momentum=momentum)
    descs, lib = _listed(descs), load_library()
    dt = MUON_DTYPE_BF16 if params.dtype == torch.bfloat16 else MUON_DTYPE_F32
    _launch(grads.get_device(), lib.muon_step_noalloc, params.data_ptr(), dt, params.numel(),
            grads.data_ptr(), momentum.data_ptr(), _shorter(grads, momentum), descs_array(descs),
            len(descs), lr, weight_decay, beta, int(bool(nesterov)), int(ns_steps),
            _mode(mode))


def group_table(groups, device):
    """A device table of optimizer groups for ``muon_step_grouped``: rows of
    ``(lr, weight_decay, beta, nesterov)``, stored as ``muon_group_t`` (three
    float32 and one int32) in an int32 tensor of shape (len(groups), 4)."""
    import numpy as np
    import torch
    rows = np.zeros((len(groups), 4), dtype=np.int32)
    for k, (lr, wd, beta, nesterov) in enumerate(groups):
        rows[k, :3] = np.array([lr, wd, beta], dtype=np.float32).view(np.int32)
        rows[k, 3] = int(bool(nesterov))
    return torch.from_numpy(rows).to(device)


def muon_step_grouped(params, grads, momentum, descs, groups, ns_steps: int = 5,
                      mode: str = "bf16", model_copy=None, workspace=None):
    """One Muon step with per-matrix optimizer groups: descriptor ``group`` k
    uses row k of ``groups`` (a ``group_table`` on the GPU, read when the
    kernels run).  ``model_copy`` (bf16, shaped like float32 ``params``)
    receives the updated weights rounded to bfloat16."""
    _step_grouped(params, grads, momentum, descs, groups, None, ns_steps, mode, model_copy,
                  workspace)


def muon_step_clipped(params, grads, momentum, descs, groups, clip, ns_steps: int = 5,
                      mode: str = "bf16", model_copy=None, workspace=None):
    """``muon_step_grouped`` on ``grads`` times the coefficient of ``clip`` (a
    ``clip_state`` that ``muon_grad_norm`` filled); ``grads`` is only read.  The
    first call with a descriptor set is made outside graph capture: it builds the plan."""
    _require_clip(clip, grads.device)
    _step_grouped(params, grads, momentum, descs, groups, clip, ns_steps, mode, model_copy,
                  workspace)


def _step_grouped(params, grads, momentum, descs, groups, clip, ns_steps, mode, model_copy,
                  workspace):
    import torch
    _require(params, "params", (torch.float32, torch.bfloat16))
    _require(grads, "grads", (torch.float32,))
    _require(momentum, "momentum", (torch.float32,))
    _require(groups, "groups", (torch.int32,))
    if groups.dim() != 2 or groups.shape[1] != 4:
        raise ValueError("groups must be a group_table of shape (n_groups, 4)")
    copy_ptr = None
    if model_copy is not None:
        _require(model_copy, "model_copy", (torch.bfloat16,))
        if model_copy.numel() != params.numel():
            raise ValueError("model_copy must have as many elements as params")
        copy_ptr = model_copy.data_ptr()
    _together(grads, "grads", params=params, momentum=momentum, groups=groups,
              model_copy=model_copy)
    descs, lib = _listed(descs), load_library()
    dt = MUON_DTYPE_BF16 if params.dtype == torch.bfloat16 else MUON_DTYPE_F32
    head = (params.data_ptr(), dt, params.numel(), copy_ptr, grads.data_ptr(),
            momentum.data_ptr(), _shorter(grads, momentum), descs_array(descs), len(descs),
            groups.data_ptr(), groups.shape[0])
    with _workspace(workspace, descs, mode, grads.device) as ws:
        tail = (int(ns_steps), _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size())
        if clip is None:
            _launch(grads.get_device(), lib.muon_step_grouped, *head, *tail)
        else:
            _launch(grads.get_device(), lib.muon_step_clipped, *head, clip.record.data_ptr(), *tail)


def muon_momentum(grads, momentum, u_out, descs, beta: float, nesterov: bool = True):
    """Momentum update (in place) and orthogonalization input written to ``u_out``."""
    import torch
    for t, nm in ((grads, "grads"), (momentum, "momentum"), (u_out, "u_out")):
        _require(t, nm, (torch.float32,))
    _together(grads, "grads", momentum=momentum, u_out=u_out)
    descs, lib = _listed(descs), load_library()
    _launch(grads.get_device(), lib.muon_momentum, grads.data_ptr(), momentum.data_ptr(),
            u_out.data_ptr(), _shorter(grads, momentum, u_out), descs_array(descs), len(descs),
            beta, int(bool(nesterov)))


def muon_orthogonalize(u, o_out, descs, ns_steps: int = 5, mode: str = "bf16", workspace=None):
    """``o_out = sqrt(max(1, rows/cols)) * NS(u)`` for every descriptor."""
    import torch
    _require(u, "u", (torch.float32,))
    _require(o_out, "o_out", (torch.float32,))
    _together(u, "u", o_out=o_out)
    descs, lib = _listed(descs), load_library()
    with _workspace(workspace, descs, mode, u.device) as ws:
        _launch(u.get_device(), lib.muon_orthogonalize, u.data_ptr(), o_out.data_ptr(),
                _shorter(u, o_out), descs_array(descs), len(descs), int(ns_steps),
                _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size())


def muon_apply(params, updates, descs, lr: float, weight_decay: float):
    """``W <- W (1 - lr wd) - lr O`` scattered into ``params`` slices."""
    import torch
    _require(params, "params", (torch.float32, torch.bfloat16))
    _require(updates, "updates", (torch.float32,))
    _together(updates, "updates", params=params)
    descs, lib = _listed(descs), load_library()
    dt = MUON_DTYPE_BF16 if params.dtype == torch.bfloat16 else MUON_DTYPE_F32
    _launch(updates.get_device(), lib.muon_apply, params.data_ptr(), dt, params.numel(),
            updates.data_ptr(), updates.numel(), descs_array(descs), len(descs), lr,
            weight_decay)


class ClipState:
    """A clipping record (``muon_clip_t``) in device memory: ``record``, two float64,
    and views of its fields: ``sumsq`` (float64, shape (1,), to be all-reduced),
    ``norm`` and ``coef`` (float32, without dimensions)."""

    def __init__(self, device):
        import torch
        self.record = torch.zeros(2, dtype=torch.float64, device=device)
        self.sumsq = self.record[:1]
        self.norm = self.record.view(torch.float32)[2]
        self.coef = self.record.view(torch.float32)[3]
        self.device = self.record.device


def clip_state(device) -> ClipState:
    """A clipping record on ``device``: zero until ``muon_grad_norm`` fills it."""
    return ClipState(device)


def clip_sumsq(clip: ClipState):
    """The record's sum of squares: a float64 view of shape (1,), to be all-reduced."""
    return clip.sumsq


def clip_norm(clip: ClipState):
    """The record's norm: a float32 view without dimensions."""
    return clip.norm


def clip_coef(clip: ClipState):
    """The record's clipping coefficient: a float32 view without dimensions."""
    return clip.coef


def _require_clip(clip, device):
    if not isinstance(clip, ClipState):
        raise TypeError("clip must be a clip_state")
    if not clip.record.is_cuda:
        raise ValueError("clip must be on a GPU (no CPU path exists)")
    if clip.device != device:
        raise ValueError(f"clip is on {clip.device}, the tensors are on {device}")


class TensorList:
    """Tensors as a ``muon_tensor_t`` array.  Keeps the tensors and the memory that they had;
    their addresses are taken once, so a tensor whose storage is replaced, moved or
    freed needs a new list: calls refuse one that holds it."""

    def __init__(self, tensors: Iterable):
        import torch
        self.tensors = list(tensors)
        self.array = (TensorC * max(1, len(self.tensors)))()
        self.device = None
        self.workspace_bytes = None
        for k, t in enumerate(self.tensors):
            _require(t, f"tensors[{k}]", (torch.float32, torch.bfloat16))
            if self.device is None:
                self.device = t.device
            elif t.device != self.device:
                raise ValueError(f"tensors[{k}] is on {t.device}, the first one on {self.device}")
            bf16 = t.dtype == torch.bfloat16
            self.array[k] = TensorC(t.data_ptr(), t.numel(),
                                    MUON_DTYPE_BF16 if bf16 else MUON_DTYPE_F32, 0)
        # With the storages held, no other tensor's memory can come to lie at an address of
        # the list, so an unchanged address is the same memory.
        self._data_ptr = torch.Tensor.data_ptr
        self._addresses = list(map(self._data_ptr, self.tensors))
        self._storages = [t.untyped_storage() for t in self.tensors]

    def check(self) -> None:
        """Refuses the list if one of its tensors has moved.  Less than 0.1 us a tensor."""
        now = list(map(self._data_ptr, self.tensors))
        if now != self._addresses:
            k = next(i for i, (a, b) in enumerate(zip(now, self._addresses)) if a != b)
            raise ValueError(f"tensors[{k}] has moved since the list was made: make a new one")

    def __len__(self) -> int:
        return len(self.tensors)


def tensor_list(tensors) -> TensorList:
    """``tensors`` as a list that the norm and clipping calls take as it is: a
    program that keeps its gradient buffers makes it once (about 1 us a tensor).
    Where gradients get new memory every step (``zero_grad(set_to_none=True)``), make a
    new one, or pass the tensors themselves, every step."""
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def _tensors_now(tensors) -> TensorList:
    """``tensors`` as a list whose addresses hold at this moment."""
    if isinstance(tensors, TensorList):
        tensors.check()
        return tensors
    return TensorList(tensors)


def muon_clip_workspace_bytes(tensors) -> int:
    """Workspace bytes of ``muon_grad_norm`` for these tensors."""
    tl = tensor_list(tensors)
    if tl.workspace_bytes is None:
        out = ctypes.c_size_t(0)
        check(load_library().muon_clip_workspace_bytes(tl.array, len(tl), ctypes.byref(out)))
        tl.workspace_bytes = out.value
    return tl.workspace_bytes


#: Default workspaces of muon_grad_norm, one per (device, stream).
_clip_workspaces: dict = {}


def _clip_workspace_for(tl: TensorList, device):
    import torch
    with torch.cuda.device(device):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("pass an explicit workspace to calls made under graph capture")
        stream = torch.cuda.current_stream()
        key = (device, stream.cuda_stream)
        need = muon_clip_workspace_bytes(tl)
        ws = _clip_workspaces.get(key)
        if ws is None or ws.numel() < need:
            _clip_workspaces.pop(key, None)
            ws = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
            _clip_workspaces[key] = ws
    return ws


def muon_grad_norm(tensors, max_norm: float, clip, tensor_norms=None, workspace=None):
    """Global 2-norm of ``tensors`` (f32 or bf16, any mix) and the coefficient
    ``min(1, max_norm / (norm + 1e-6))``, written to ``clip`` (a ``clip_state``)
    on its device's current stream; nothing returns to the host.

    ``tensor_norms``: float32, one element per tensor, receives their norms.
    ``workspace``: a uint8 GPU tensor of ``muon_clip_workspace_bytes`` (default: a
    cached one per device and stream; give one under graph capture)."""
    import torch
    tl = _tensors_now(tensors)
    _require_clip(clip, tl.device if tl.device is not None else clip.device)
    norms_ptr = None
    if tensor_norms is not None:
        _require(tensor_norms, "tensor_norms", (torch.float32,))
        if tensor_norms.numel() != len(tl) or tensor_norms.device != clip.device:
            raise ValueError("tensor_norms must have one element per tensor, on their device")
        norms_ptr = tensor_norms.data_ptr()
    head = (clip.device.index, load_library().muon_grad_norm, tl.array, len(tl), max_norm,
            clip.record.data_ptr(), norms_ptr)
    if workspace is None:
        with _stream_lock(clip.device):
            workspace = _clip_workspace_for(tl, clip.device)
            _launch(*head, workspace.data_ptr(), workspace.numel())
    else:
        _require(workspace, "workspace", (torch.uint8,))
        if workspace.device != clip.device:
            raise ValueError("workspace is on another device than the tensors")
        _launch(*head, workspace.data_ptr(), workspace.numel())


def muon_clip_finish(clip, max_norm: float):
    """Norm and coefficient of ``clip`` from its ``clip_sumsq``, as it stands after
    the sums of several ranks (or calls) were added up."""
    _require_clip(clip, clip.device)
    _launch(clip.device.index, load_library().muon_clip_finish, clip.record.data_ptr(), max_norm)


def muon_clip_grads(tensors, clip, out=None):
    """Every tensor times the coefficient of ``clip``, in place, or into the
    tensors of ``out`` (same lengths; f32 or bf16, rounded once)."""
    src = _tensors_now(tensors)
    dst = src if out is None else _tensors_now(out)
    if len(src) != len(dst):
        raise ValueError(f"{len(src)} tensors, but {len(dst)} in out")
    if len(src) == 0:
        return
    _require_clip(clip, src.device)
    if dst.device != src.device:
        raise ValueError("out is on another device than the tensors")
    _launch(clip.device.index, load_library().muon_clip_grads, src.array, dst.array, len(src),
            clip.record.data_ptr())


def ranges_array(ranges) -> ctypes.Array:
    """Ranges as a ``muon_range_t`` array (which ``muon_adamw`` takes as it is)."""
    if isinstance(ranges, ctypes.Array) and ranges._type_ is RangeC:
        return ranges
    items = list(ranges)
    arr = (RangeC * len(items))()
    for k, r in enumerate(items):
        if isinstance(r, (tuple, list)):
            vals = list(r) + [None] * (4 - len(r))
            off, numel, poff, group = vals[:4]
        else:
            off, numel = r.offset, r.numel
            poff = getattr(r, "param_offset", None)
            group = getattr(r, "group", None)
        arr[k] = RangeC(int(off), int(numel), int(off if poff is None else poff), int(group or 0),
                        0)
    return arr


def adamw_group_table(groups, device):
    """A device table of optimizer groups for ``muon_adamw``: rows of ``(lr,
    weight_decay, beta1, beta2, eps)`` or ``(..., step)``, stored as
    ``muon_adamw_group_t`` in an int64 tensor of shape (len(groups), 4).  ``step``
    is the number of the next step (default 1); see ``adamw_steps``."""
    import numpy as np
    import torch
    rows = np.zeros((len(groups), 8), dtype=np.int32)
    steps = rows.view(np.int64)
    for k, row in enumerate(groups):
        if len(row) not in (5, 6):
            raise ValueError("a group is (lr, weight_decay, beta1, beta2, eps[, step])")
        rows[k, :5] = np.array(row[:5], dtype=np.float32).view(np.int32)
        steps[k, 3] = int(row[5]) if len(row) == 6 else 1
    return torch.from_numpy(rows.view(np.int64)).to(device)


def adamw_steps(groups):
    """The step numbers of an ``adamw_group_table``: an int64 view; ``.add_(1)``
    between steps (it may be captured into the graph with them)."""
    return groups[:, 3]


def muon_adamw(params, grads, exp_avg, exp_avg_sq, ranges, groups, clip=None, model_copy=None):
    """One AdamW step in place on ``params`` (f32 or bf16), ``exp_avg`` and
    ``exp_avg_sq`` (f32) over ``ranges`` of the flat buffers; ``grads`` (f32 or bf16)
    is multiplied by the coefficient of ``clip`` (a ``clip_state``) as it is read.
    ``groups``: an ``adamw_group_table``, read when the kernels run.
    ``model_copy`` (bf16, shaped like float32 ``params``) receives the updated
    weights rounded to bfloat16."""
    import torch
    both = (torch.float32, torch.bfloat16)
    _require(params, "params", both)
    _require(grads, "grads", both)
    _require(exp_avg, "exp_avg", (torch.float32,))
    _require(exp_avg_sq, "exp_avg_sq", (torch.float32,))
    _require(groups, "groups", (torch.int64,))
    if groups.dim() != 2 or groups.shape[1] != 4:
        raise ValueError("groups must be an adamw_group_table of shape (n_groups, 4)")
    if not grads.numel() == exp_avg.numel() == exp_avg_sq.numel():
        raise ValueError("grads, exp_avg and exp_avg_sq must have as many elements as each other")
    copy_ptr = clip_ptr = None
    if model_copy is not None:
        _require(model_copy, "model_copy", (torch.bfloat16,))
        if model_copy.numel() != params.numel():
            raise ValueError("model_copy must have as many elements as params")
        copy_ptr = model_copy.data_ptr()
    if clip is not None:
        _require_clip(clip, grads.device)
        clip_ptr = clip.record.data_ptr()
    at = grads.get_device()
    for t, name in ((params, "params"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"),
                    (groups, "groups"), (model_copy, "model_copy")):
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} is on {t.device}, grads on {grads.device}")
    arr = ranges_array(ranges)
    pdt = MUON_DTYPE_BF16 if params.dtype == torch.bfloat16 else MUON_DTYPE_F32
    gdt = MUON_DTYPE_BF16 if grads.dtype == torch.bfloat16 else MUON_DTYPE_F32
    _launch(at, load_library().muon_adamw, params.data_ptr(), pdt, params.numel(), copy_ptr,
            grads.data_ptr(), gdt, exp_avg.data_ptr(), exp_avg_sq.data_ptr(), grads.numel(), arr,
            len(arr), groups.data_ptr(), groups.shape[0], clip_ptr)


#: Formats of the 8-bit types; filled at the first call that needs it (torch is loaded then).
_FP8: dict = {}


def _fp8_formats() -> dict:
    if not _FP8:
        import torch
        _FP8.update({torch.float8_e4m3fn: 0, torch.float8_e5m2: 1})
    return _FP8


def fp8_scales(rows: int, cols: int, block: str, device):
    """Scales of a rows x cols matrix in 8 bits, uninitialised: float32 of shape
    (rows, ceil(cols / 128)) for 1 x 128 blocks (``block`` "row") or (ceil(rows / 128),
    ceil(cols / 128)) for 128 x 128 blocks ("square").  The scales of one block column
    lie together, as products read them fastest."""
    import torch
    if block not in ("row", "square"):
        raise ValueError(f"block must be 'row' or 'square', got {block!r}")
    high = rows if block == "row" else -(-rows // 128)
    return torch.empty(-(-cols // 128), high, dtype=torch.float32, device=device).t()


def _matrix(t, name, dtypes):
    """Shape and row stride of a GPU matrix with neighbouring elements in a row; refuses others."""
    try:
        (rows, cols), (row, col) = t.shape, t.stride()
        if t.is_cuda and t.dtype in dtypes and (col == 1 or cols <= 1):
            return rows, cols, row
    except (AttributeError, ValueError):
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, it has {t.dim()}")
    raise ValueError(f"the elements of a row of {name} must be neighbours")


def _fp8(codes, scales, name, scales_name) -> Fp8C:
    """Codes and scales as ``muon_fp8_t``.  Rows of blocks are told by the scales' shape; a
    matrix of one row is the same either way."""
    import torch
    formats = _fp8_formats()
    rows, cols, row = _matrix(codes, name, formats)
    if not (isinstance(scales, torch.Tensor) and scales.dtype is torch.float32 and scales.is_cuda
            and scales.dim() == 2):
        raise TypeError(f"{scales_name} must be a float32 GPU matrix")
    if scales.get_device() != codes.get_device():
        raise ValueError(f"{scales_name} is on {scales.device}, {name} on {codes.device}")
    high, across = scales.shape
    if across == -(-cols // 128) and high == rows:
        block_rows = 1
    elif across == -(-cols // 128) and high == -(-rows // 128):
        block_rows = 128
    else:
        raise ValueError(f"{scales_name} has shape {tuple(scales.shape)}, {name} {tuple(codes.shape)}: "
                         "expected one scale for each 1 x 128 or 128 x 128 block")
    down, right = scales.stride()
    return Fp8C(codes.data_ptr(), scales.data_ptr(), rows, cols, row, down, right,
                formats[codes.dtype], block_rows)


def _same_device(first, first_name, **others) -> None:
    """``_together`` for tensors that are known to be on GPUs."""
    at = first.get_device()
    for t in others.values():
        if t is not None and t.get_device() != at:
            _together(first, first_name, **others)


def muon_fp8_cast(x, codes=None, scales=None, codes_t=None, scales_t=None):
    """``x`` (a matrix, f32 or bf16, with any row stride) into 8 bits: into ``codes``
    (float8_e4m3fn or float8_e5m2, shaped like x) with ``scales``, its transpose into
    ``codes_t`` with ``scales_t``, or both.  The scales' shape says the blocks: see
    ``fp8_scales``."""
    import torch
    bf16 = torch.bfloat16
    rows, cols, row = _matrix(x, "x", (torch.float32, bf16))
    if codes is None and codes_t is None:
        raise ValueError("codes or codes_t must be given")
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None):
        raise ValueError("codes and scales belong together, and so do codes_t and scales_t")
    out = None if codes is None else _fp8(codes, scales, "codes", "scales")
    out_t = None if codes_t is None else _fp8(codes_t, scales_t, "codes_t", "scales_t")
    _same_device(x, "x", codes=codes, codes_t=codes_t)
    if out is not None and out_t is not None and out.block_rows != out_t.block_rows:
        # one row or one column: its 1 x 128 and 128 x 128 blocks are the same
        if rows <= 1:
            out.block_rows = out_t.block_rows
        elif cols <= 1:
            out_t.block_rows = out.block_rows
    _launch(x.get_device(), load_library().muon_fp8_cast, x.data_ptr(),
            MUON_DTYPE_BF16 if x.dtype is bf16 else MUON_DTYPE_F32, rows, cols, row, None if out is None else ctypes.byref(out),
            None if out_t is None else ctypes.byref(out_t))


def muon_fp8_workspace_bytes(m: int, n: int, k: int) -> int:
    """Workspace bytes of ``muon_fp8_matmul`` for m x n products over k (0 for most)."""
    out = ctypes.c_size_t(0)
    check(load_library().muon_fp8_workspace_bytes(m, n, k, ctypes.byref(out)))
    return out.value


#: Default workspaces of the calls that keep no plan, one per (device, stream).
_call_workspaces: dict = {}


def _call_workspace(need: int, device):
    """A cached workspace of at least ``need`` bytes for the current stream of ``device``;
    called under that stream's lock."""
    import torch
    if _capturing(device):
        raise RuntimeError("pass an explicit workspace to calls made under graph capture")
    stream = torch.cuda.current_stream(device)
    key = (device, stream.cuda_stream)
    ws = _call_workspaces.get(key)
    if ws is None or ws.numel() < need:
        _call_workspaces.pop(key, None)
        with torch.cuda.stream(stream):
            ws = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
        _call_workspaces[key] = ws
    return ws


def _launch_with_workspace(workspace, need: int, beside, call, *args) -> None:
    """``call(*args, workspace, bytes, stream)`` on the device of ``beside`` with the given
    workspace, or, where one is needed, the stream's default one under its lock."""
    import torch
    index = beside.get_device()
    if workspace is not None:
        _require(workspace, "workspace", (torch.uint8,))
        if workspace.get_device() != index:
            raise ValueError(f"workspace is on {workspace.device}, the tensors on {beside.device}")
        _launch(index, call, *args, workspace.data_ptr(), workspace.numel())
    elif need == 0:
        _launch(index, call, *args, None, 0)
    else:
        device = beside.device
        with _stream_lock(device):
            ws = _call_workspace(need, device)
            _launch(index, call, *args, ws.data_ptr(), ws.numel())


def muon_fp8_matmul(a, a_scales, b, b_scales, out, accumulate: bool = False, workspace=None):
    """``out = a b^T``, or ``out += a b^T``: a (m, k) and b (n, k) in 8 bits with their
    scales, out (m, n) f32 or bf16 (f32 with ``accumulate``), all with any row stride.

    ``workspace``: a uint8 GPU tensor of ``muon_fp8_workspace_bytes`` (default: a cached
    one per device and stream, where one is needed; give one under graph capture)."""
    import torch
    bf16 = torch.bfloat16
    left, right = _fp8(a, a_scales, "a", "a_scales"), _fp8(b, b_scales, "b", "b_scales")
    m, n, row = _matrix(out, "out", (torch.float32, bf16))
    _same_device(a, "a", b=b, out=out)
    if m != left.rows or n != right.rows:
        raise ValueError(f"out has shape {(m, n)}, expected {(left.rows, right.rows)}")
    need = 0 if workspace is not None else muon_fp8_workspace_bytes(m, n, left.cols)
    _launch_with_workspace(workspace, need, a, load_library().muon_fp8_matmul, ctypes.byref(left),
                           ctypes.byref(right), out.data_ptr(),
                           MUON_DTYPE_BF16 if out.dtype is bf16 else MUON_DTYPE_F32, row,
                           1 if accumulate else 0)


#: Coefficients of ``muon_orthogonalize_stack`` where none are given: those of ``muon_step``.
QUINTIC = ((3.4445, -4.7750, 2.0315),) * 5


def _stack(x, out) -> StackC:
    import torch
    both = (torch.float32, torch.bfloat16)
    for t, name in ((x, "x"), (out, "out")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
        if t.dtype not in both:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {both}")
        if t.dim() not in (2, 3):
            raise ValueError(f"{name} must be a matrix or a stack of them, it has {t.dim()} dimensions")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"the elements of a row of {name} must be neighbours")

    def dt(t):
        return MUON_DTYPE_BF16 if t.dtype == torch.bfloat16 else MUON_DTYPE_F32

    if out is None:
        out = x
    count = x.shape[0] if x.dim() == 3 else 1
    return StackC(x.data_ptr(), out.data_ptr(), count, x.shape[-2], x.shape[-1],
                  x.stride(0) if x.dim() == 3 else 0, x.stride(-2),
                  out.stride(0) if out.dim() == 3 else 0, out.stride(-2), dt(x), dt(out))


def muon_stack_workspace_bytes(x) -> int:
    """Workspace bytes with which ``muon_orthogonalize_stack`` takes all of ``x`` at once;
    of a stack, a ``len(x)``-th part of them is the least."""
    stack = _stack(x, None)
    need = ctypes.c_size_t(0)
    check(load_library().muon_stack_workspace_bytes(ctypes.byref(stack), ctypes.byref(need)))
    return need.value


def muon_orthogonalize_stack(x, out, coefficients=None, scale=None, workspace=None):
    """``out = scale * NS(x)`` for a matrix or every matrix of a stack (count, rows, cols), f32
    or bf16, with any strides between rows and matrices, in float32 accuracy.

    ``coefficients``: (a, b, c) of every step (default ``QUINTIC``).  ``scale``: default
    sqrt(max(1, rows / cols)).  ``workspace``: a uint8 GPU tensor of
    ``muon_stack_workspace_bytes``, or less (default: a cached one per device and
    stream; give one under graph capture)."""
    stack = _stack(x, out)
    _together(x, "x", out=out)
    if x.shape != out.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, x {tuple(x.shape)}")
    steps = [tuple(c) for c in (QUINTIC if coefficients is None else coefficients)]
    if any(len(c) != 3 for c in steps):
        raise ValueError("coefficients are (a, b, c) for every step")
    flat = (ctypes.c_float * max(1, 3 * len(steps)))(*[float(v) for c in steps for v in c])
    if scale is None:
        scale = max(1.0, stack.rows / max(1, stack.cols)) ** 0.5
    need = 0 if workspace is not None else muon_stack_workspace_bytes(x)
    _launch_with_workspace(workspace, need, x, load_library().muon_orthogonalize_stack,
                           ctypes.byref(stack), flat, len(steps), scale)


def muon_profile_begin() -> None:
    """Start timing every kernel launch with HIP events on its stream."""
    check(load_library().muon_profile_begin())


def muon_profile_end() -> dict:
    """Stop timing; returns {kernel name: (total_ms, launches)}."""
    lib = load_library()
    rows = (KernelTimeC * 64)()
    count = ctypes.c_int(0)
    check(lib.muon_profile_end(rows, 64, ctypes.byref(count)))
    return {rows[k].name.decode(): (rows[k].total_ms, rows[k].launches)
            for k in range(min(count.value, 64))}
