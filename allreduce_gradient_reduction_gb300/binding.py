"""Python binding of libar_gb300.so (include/ar.h): argument marshalling only.

Every function takes the same arguments as its C counterpart.  Where the C
function takes an array of device pointers, this binding accepts a sequence of
torch CUDA tensors (their data pointers are passed) or plain integers.  Enum
arguments accept the C value or its lower-case name ("f32", "sum", "ring",
...).  A stream is a torch.cuda.Stream, an integer cudaStream_t, or None (the
current torch stream).  Each call returns the C status; ``check()`` raises
ArError on a non-zero one.

Loading fails loudly: without the compiled library there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libar_gb300.so")

DTYPE = {"f32": 0, "bf16": 1, "i32": 2, "f16": 3}
OP = {"sum": 0, "max": 1, "avg": 2}
ALGO = {"ring": 0, "ring_stepwise": 1, "tree": 2, "tree_stepwise": 3, "naive": 4, "dbtree": 5,
        "binomial_stepwise": 6}
STATUS = {0: "AR_OK", -1: "AR_ERR_INVALID_ARG", -2: "AR_ERR_UNSUPPORTED", -3: "AR_ERR_CUDA",
          -4: "AR_ERR_TIMEOUT", -5: "AR_ERR_NO_DEVICE", -6: "AR_ERR_TOO_LARGE", -7: "AR_ERR_HOST"}
AR_OK, AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED, AR_ERR_CUDA, AR_ERR_TIMEOUT = 0, -1, -2, -3, -4
MAX_RANKS = 64
MAX_COUNT = 1 << 56  # AR_MAX_COUNT
DEFAULT_BUCKET_CAP_BYTES = 25 << 20

EXPORTS = ("ar_allreduce", "ar_reduce_scatter", "ar_all_gather", "ar_reduce", "ar_broadcast", "ar_allreduce_int8_ef",
           "ar_allreduce_host",
           "ar_bucket_plan",
           "ar_bucketed_allreduce",
           "ar_bucketed_allreduce_noalloc", "ar_chunk_range", "ar_device_status", "ar_set_barrier_timeout_ns", "ar_debug_skip_barrier",
           "ar_last_cuda_error", "ar_strerror", "ar_version", "ar_kernel_launches", "ar_reducer_create",
           "ar_reducer_mark_ready", "ar_reducer_finish", "ar_reducer_destroy", "ar_reducer_buckets",
           "ar_reducer_set_max_blocks", "ar_plan_create", "ar_plan_run", "ar_plan_destroy",
           "ar_layer_norm", "ar_layer_norm_backward", "ar_layer_norm_workspace_bytes", "ar_distill_loss",
           "ar_distill_loss_backward", "ar_attention", "ar_attention_backward", "ar_attention_workspace_bytes")


class AttentionTensor(ctypes.Structure):
    """ar_attention_tensor: an operand of the attention calls."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class ArError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({code})")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(the CUDA library is required; there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, vp, cint = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int
    pp = ctypes.POINTER(vp)
    L.ar_allreduce.argtypes = [pp, cint, i64, cint, cint, cint, vp]
    L.ar_reduce_scatter.argtypes = [pp, cint, i64, cint, cint, cint, vp]
    L.ar_all_gather.argtypes = [pp, cint, i64, cint, cint, vp]
    L.ar_reduce.argtypes = [pp, cint, i64, cint, cint, cint, cint, vp]
    L.ar_broadcast.argtypes = [pp, cint, i64, cint, cint, vp]
    L.ar_allreduce_int8_ef.argtypes = [pp, pp, cint, i64, cint, vp]
    L.ar_allreduce_host.argtypes = [pp, pp, cint, i64, cint, cint, cint, i64, vp]
    L.ar_bucket_plan.argtypes = [ctypes.POINTER(i64), cint, cint, i64, ctypes.POINTER(i32), ctypes.POINTER(i64),
                                 ctypes.POINTER(i64), ctypes.POINTER(i32)]
    L.ar_bucketed_allreduce.argtypes = [pp, ctypes.POINTER(i64), cint, cint, cint, cint, cint, i64, pp, i64, vp]
    L.ar_bucketed_allreduce_noalloc.argtypes = [pp, ctypes.POINTER(i64), cint, cint, cint, cint, cint, i64, vp]
    L.ar_chunk_range.argtypes = [i64, cint, cint, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.ar_device_status.argtypes = [vp, ctypes.POINTER(cint)]
    L.ar_set_barrier_timeout_ns.argtypes = [i64]
    L.ar_debug_skip_barrier.argtypes = [cint]
    L.ar_last_cuda_error.argtypes = []
    L.ar_strerror.argtypes = [cint]
    L.ar_strerror.restype = ctypes.c_char_p
    L.ar_version.argtypes = []
    L.ar_kernel_launches.argtypes = []
    L.ar_reducer_create.argtypes = [pp, ctypes.POINTER(i64), cint, cint, cint, cint, cint, i64, vp,
                                    ctypes.POINTER(vp)]
    L.ar_reducer_mark_ready.argtypes = [vp, cint, vp]
    L.ar_reducer_finish.argtypes = [vp, vp]
    L.ar_reducer_destroy.argtypes = [vp]
    L.ar_reducer_buckets.argtypes = [vp]
    L.ar_reducer_set_max_blocks.argtypes = [vp, cint]
    L.ar_plan_create.argtypes = [cint, pp, cint, i64, cint, cint, cint, cint, ctypes.POINTER(vp)]
    L.ar_plan_run.argtypes = [vp, vp]
    L.ar_plan_destroy.argtypes = [vp]
    flt, at = ctypes.c_float, vp  # vp: the address of an AttentionTensor
    L.ar_layer_norm.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, i64, i64, flt, cint, cint, vp]
    L.ar_layer_norm_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i64, i64, cint, cint, vp, i64,
                                         vp]
    L.ar_layer_norm_workspace_bytes.argtypes = [i64, i64]
    L.ar_distill_loss.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, flt, cint, cint, vp]
    L.ar_distill_loss_backward.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64, flt, cint, cint, vp]
    L.ar_attention.argtypes = [at, at, at, vp, at, vp, i64, i64, i64, i64, i64, flt, cint, vp]
    L.ar_attention_backward.argtypes = [at, at, at, at, at, vp, vp, at, at, at, i64, i64, i64, i64, i64, flt, cint, vp,
                                        i64, vp]
    L.ar_attention_workspace_bytes.argtypes = [i64, i64, i64, i64]
    for name in EXPORTS:
        if name != "ar_strerror":
            getattr(L, name).restype = cint
    for name in ("ar_kernel_launches", "ar_layer_norm_workspace_bytes", "ar_attention_workspace_bytes"):
        getattr(L, name).restype = i64
    return L


lib = _load()


def _enum(table, v):
    return table[v] if isinstance(v, str) else int(v)


def _ptr(x) -> int:
    if isinstance(x, int):
        return x
    if x is None:
        return 0
    return int(x.data_ptr())


_ARRAY_TYPES = {}


def _ptr_array(xs):
    """A C array of the addresses of xs (tensors, addresses or None), built
    over an array of 64-bit words: at 64 ranks about half the cost of ctypes'
    element-by-element constructor."""
    n = max(len(xs), 1)
    t = _ARRAY_TYPES.get(n)
    if t is None:
        t = _ARRAY_TYPES[n] = ctypes.c_void_p * n
    try:
        addrs = [x.data_ptr() for x in xs]
    except AttributeError:
        addrs = [_ptr(x) for x in xs]
    return t.from_buffer(array.array("Q", addrs or [0]))


def _stream(s) -> int:
    if s is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _count(bufs, count):
    if count is not None:
        return int(count)
    return int(bufs[0].numel()) if len(bufs) and not isinstance(bufs[0], int) else 0


def check(rc: int, what: str = "ar") -> int:
    if rc != AR_OK:
        raise ArError(rc, what)
    return rc


def ar_allreduce(bufs, nranks=None, count=None, dtype="f32", op="sum", algo="ring", stream=None) -> int:
    n = len(bufs) if nranks is None else int(nranks)
    return lib.ar_allreduce(_ptr_array(bufs), n, _count(bufs, count), _enum(DTYPE, dtype), _enum(OP, op),
                            _enum(ALGO, algo), _stream(stream))


def ar_reduce_scatter(bufs, nranks=None, count=None, dtype="f32", op="sum", algo="ring", stream=None) -> int:
    n = len(bufs) if nranks is None else int(nranks)
    return lib.ar_reduce_scatter(_ptr_array(bufs), n, _count(bufs, count), _enum(DTYPE, dtype), _enum(OP, op),
                                 _enum(ALGO, algo), _stream(stream))


def ar_all_gather(bufs, nranks=None, count=None, dtype="f32", algo="ring", stream=None) -> int:
    n = len(bufs) if nranks is None else int(nranks)
    return lib.ar_all_gather(_ptr_array(bufs), n, _count(bufs, count), _enum(DTYPE, dtype), _enum(ALGO, algo),
                             _stream(stream))


def ar_reduce(bufs, nranks=None, count=None, dtype="f32", op="sum", algo="ring", root=0, stream=None) -> int:
    n = len(bufs) if nranks is None else int(nranks)
    return lib.ar_reduce(_ptr_array(bufs), n, _count(bufs, count), _enum(DTYPE, dtype), _enum(OP, op),
                         _enum(ALGO, algo), int(root), _stream(stream))


def ar_broadcast(bufs, nranks=None, count=None, dtype="f32", root=0, stream=None) -> int:
    n = len(bufs) if nranks is None else int(nranks)
    return lib.ar_broadcast(_ptr_array(bufs), n, _count(bufs, count), _enum(DTYPE, dtype), int(root),
                            _stream(stream))


def ar_allreduce_host(host_bufs, dev_bufs=None, nranks=None, count=None, dtype="f32", op="sum", algo="ring",
                      piece_elems=0, stream=None) -> int:
    """host_bufs: CPU tensors or host addresses.  dev_bufs None: zero-copy on
    page-locked host buffers; else device working buffers (staged pieces)."""
    n = len(host_bufs) if nranks is None else int(nranks)
    return lib.ar_allreduce_host(_ptr_array(host_bufs), None if dev_bufs is None else _ptr_array(dev_bufs), n,
                                 _count(host_bufs, count),
                                 _enum(DTYPE, dtype), _enum(OP, op), _enum(ALGO, algo), int(piece_elems),
                                 _stream(stream))


def ar_allreduce_int8_ef(grads, residuals, nranks=None, count=None, op="sum", stream=None) -> int:
    n = len(grads) if nranks is None else int(nranks)
    return lib.ar_allreduce_int8_ef(_ptr_array(grads), _ptr_array(residuals), n, _count(grads, count),
                                    _enum(OP, op), _stream(stream))


def ar_bucket_plan(counts, dtype="f32", cap_bytes=DEFAULT_BUCKET_CAP_BYTES):
    """Returns (status, bucket_of_tensor, offset_in_bucket, bucket_count) as lists."""
    t = len(counts)
    c = (ctypes.c_int64 * max(t, 1))(*[int(x) for x in counts])
    bo = (ctypes.c_int32 * max(t, 1))()
    off = (ctypes.c_int64 * max(t, 1))()
    bc = (ctypes.c_int64 * max(t, 1))()
    nb = ctypes.c_int32()
    rc = lib.ar_bucket_plan(c, t, _enum(DTYPE, dtype), int(cap_bytes), bo, off, bc, ctypes.byref(nb))
    return rc, list(bo[:t]), list(off[:t]), list(bc[:nb.value])


def ar_bucketed_allreduce(grads, counts=None, ntensors=None, nranks=None, dtype="f32", op="avg", algo="ring",
                          bucket_cap_bytes=DEFAULT_BUCKET_CAP_BYTES, workspace=None, workspace_bytes=0,
                          stream=None) -> int:
    """``grads`` is a list over ranks of lists over tensors (or a flat
    row-major list with ``ntensors``/``nranks`` given)."""
    if len(grads) and isinstance(grads[0], (list, tuple)):
        nr, nt = len(grads), len(grads[0])
        flat = [g for row in grads for g in row]
        if counts is None:
            counts = [int(g.numel()) for g in grads[0]]
    else:
        nr, nt, flat = int(nranks), int(ntensors), list(grads)
    c = (ctypes.c_int64 * max(nt, 1))(*[int(x) for x in counts])
    ws = _ptr_array(workspace) if workspace is not None else None
    if workspace is not None and workspace_bytes == 0 and not isinstance(workspace[0], int):
        workspace_bytes = int(workspace[0].numel() * workspace[0].element_size())
    return lib.ar_bucketed_allreduce(_ptr_array(flat), c, nt, nr, _enum(DTYPE, dtype), _enum(OP, op),
                                     _enum(ALGO, algo), int(bucket_cap_bytes), ws, int(workspace_bytes),
                                     _stream(stream))


def ar_bucketed_allreduce_noalloc(grads, counts=None, ntensors=None, nranks=None, dtype="f32", op="avg",
                                  algo="ring", bucket_cap_bytes=DEFAULT_BUCKET_CAP_BYTES, stream=None) -> int:
    """Same arguments as ar_bucketed_allreduce without the workspace: the
    library's fixed scratch array stands in for it (see include/ar.h)."""
    if len(grads) and isinstance(grads[0], (list, tuple)):
        nr, nt = len(grads), len(grads[0])
        flat = [g for row in grads for g in row]
        if counts is None:
            counts = [int(g.numel()) for g in grads[0]]
    else:
        nr, nt, flat = int(nranks), int(ntensors), list(grads)
    c = (ctypes.c_int64 * max(nt, 1))(*[int(x) for x in counts])
    return lib.ar_bucketed_allreduce_noalloc(_ptr_array(flat), c, nt, nr, _enum(DTYPE, dtype), _enum(OP, op),
                                             _enum(ALGO, algo), int(bucket_cap_bytes), _stream(stream))


NOALLOC_SCRATCH_BYTES = 32 << 20
NOALLOC_MAX_TENSORS = 1024


class Reducer:
    """Overlapped bucket reduction (ar_reducer_*): create once over the
    gradient tensors, then per iteration ``mark_ready(t, stream)`` for every
    tensor as its gradients are produced and ``finish(stream)``."""

    def __init__(self, grads, counts=None, dtype="f32", op="avg", algo="ring",
                 bucket_cap_bytes=DEFAULT_BUCKET_CAP_BYTES, comm_stream=None):
        nr, nt = len(grads), len(grads[0])
        flat = [g for row in grads for g in row]
        if counts is None:
            counts = [int(g.numel()) for g in grads[0]]
        c = (ctypes.c_int64 * max(nt, 1))(*[int(x) for x in counts])
        h = ctypes.c_void_p()
        check(lib.ar_reducer_create(_ptr_array(flat), c, nt, nr, _enum(DTYPE, dtype), _enum(OP, op),
                                    _enum(ALGO, algo), int(bucket_cap_bytes), _stream(comm_stream), ctypes.byref(h)),
              "ar_reducer_create")
        self.handle = h
        self.ntensors = nt

    @property
    def buckets(self) -> int:
        return lib.ar_reducer_buckets(self.handle)

    def set_max_blocks(self, max_blocks: int) -> int:
        return lib.ar_reducer_set_max_blocks(self.handle, int(max_blocks))

    def mark_ready(self, tensor: int, stream=None) -> int:
        return lib.ar_reducer_mark_ready(self.handle, int(tensor), _stream(stream))

    def finish(self, stream=None) -> int:
        return lib.ar_reducer_finish(self.handle, _stream(stream))

    def close(self):
        if self.handle:
            lib.ar_reducer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


PLAN_KIND = {"allreduce": 0, "reduce_scatter": 1, "all_gather": 2, "reduce": 3}


class Plan:
    """A prepared collective (ar_plan_*): arguments checked and launch tables
    built once; ``run(stream)`` only enqueues the kernels."""

    def __init__(self, kind, bufs, count=None, dtype="f32", op="sum", algo="ring", root=0):
        h = ctypes.c_void_p()
        check(lib.ar_plan_create(PLAN_KIND[kind] if isinstance(kind, str) else int(kind), _ptr_array(bufs),
                                 len(bufs), _count(bufs, count), _enum(DTYPE, dtype), _enum(OP, op), _enum(ALGO, algo),
                                 int(root), ctypes.byref(h)), "ar_plan_create")
        self.handle = h

    def run(self, stream=None) -> int:
        return lib.ar_plan_run(self.handle, _stream(stream))

    def close(self):
        if self.handle:
            lib.ar_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- training-step operators ----------------------------------------------------------
#
# These take torch CUDA tensors and read sizes, strides and element types from
# them.  Operands whose shapes, types or inner strides do not belong together
# are refused (AR_ERR_INVALID_ARG, or AR_ERR_UNSUPPORTED for an element type
# the library does not have) before the library is called.  A small call costs
# as much here as on the device, so the checks read each property once.

_TORCH_DTYPE = {}  # torch dtype: the library's; filled on first use, as torch may not be there before
_F32 = []          # torch.float32


def _dtypes():
    if not _TORCH_DTYPE:
        import torch
        _F32.append(torch.float32)
        _TORCH_DTYPE.update({torch.float32: 0, torch.bfloat16: 1, torch.int32: 2, torch.float16: 3})
    return _TORCH_DTYPE


def _stream_of(stream, tensor) -> int:
    """As _stream; None is the current stream of the tensor's device."""
    if stream is not None:
        return _stream(stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None or not tensor.is_cuda:
        return _stream(None)
    return raw(tensor.get_device())


def _vector(t, n, dtype):
    """t is a contiguous vector of n elements of a torch dtype."""
    return t.dtype is dtype and t.dim() == 1 and t.numel() == n and t.is_contiguous()


def _row_stride(t, shape, dtype):
    """The row stride of a matrix of this shape and torch dtype with contiguous rows; else None."""
    if t.dtype is not dtype or t.shape != shape:
        return None
    row, inner = t.stride()
    return row if inner == 1 or shape[1] <= 1 else None


def ar_layer_norm(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None) -> int:
    """y = layer norm of the rows of the matrix x.  bias, mean and rstd may be
    None; weight and bias have x's type or f32; y may be x."""
    types = _TORCH_DTYPE or _dtypes()
    shape, dtype, pdtype = x.shape, x.dtype, weight.dtype
    if len(shape) != 2:
        return AR_ERR_INVALID_ARG
    dt, pt = types.get(dtype), types.get(pdtype)
    if dt is None or pt is None:
        return AR_ERR_UNSUPPORTED
    rows, cols = shape
    xs, ys = _row_stride(x, shape, dtype), _row_stride(y, shape, dtype)
    if xs is None or ys is None or not _vector(weight, cols, pdtype) or (
            bias is not None and not _vector(bias, cols, pdtype)):
        return AR_ERR_INVALID_ARG
    f32 = _F32[0]
    if (mean is not None and not _vector(mean, rows, f32)) or (rstd is not None and not _vector(rstd, rows, f32)):
        return AR_ERR_INVALID_ARG
    return lib.ar_layer_norm(x.data_ptr(), xs, weight.data_ptr(), None if bias is None else bias.data_ptr(),
                             y.data_ptr(), ys, None if mean is None else mean.data_ptr(),
                             None if rstd is None else rstd.data_ptr(), rows, cols, eps, dt, pt,
                             _stream_of(stream, x))


def ar_layer_norm_workspace_bytes(rows, cols) -> int:
    return lib.ar_layer_norm_workspace_bytes(int(rows), int(cols))


def ar_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, stream=None) -> int:
    """dx (may be dy or x), dweight and dbias (may be None) for an upstream
    dy, from the forward call's mean and rstd.  workspace: a tensor of at least
    ar_layer_norm_workspace_bytes(rows, cols) bytes."""
    types = _TORCH_DTYPE or _dtypes()
    shape, dtype, pdtype = x.shape, x.dtype, weight.dtype
    if len(shape) != 2:
        return AR_ERR_INVALID_ARG
    dt, pt = types.get(dtype), types.get(pdtype)
    if dt is None or pt is None:
        return AR_ERR_UNSUPPORTED
    rows, cols = shape
    xs, dys, dxs = _row_stride(x, shape, dtype), _row_stride(dy, shape, dtype), _row_stride(dx, shape, dtype)
    f32 = _F32[0]
    if (xs is None or dys is None or dxs is None or not _vector(weight, cols, pdtype)
            or not _vector(dweight, cols, pdtype) or (dbias is not None and not _vector(dbias, cols, pdtype))
            or not _vector(mean, rows, f32) or not _vector(rstd, rows, f32) or not workspace.is_contiguous()):
        return AR_ERR_INVALID_ARG
    return lib.ar_layer_norm_backward(dy.data_ptr(), dys, x.data_ptr(), xs, weight.data_ptr(), mean.data_ptr(),
                                      rstd.data_ptr(), dx.data_ptr(), dxs, dweight.data_ptr(),
                                      None if dbias is None else dbias.data_ptr(), rows, cols, dt, pt,
                                      workspace.data_ptr(), workspace.nbytes, _stream_of(stream, x))


def _distill_operands(logits, teacher_index, teacher_logits, rows_f32, dlogits):
    """(status, element types of the logits and of the teacher's, row strides of logits and dlogits)."""
    types = _TORCH_DTYPE or _dtypes()
    shape, lists, dtype, vdtype = logits.shape, teacher_index.shape, logits.dtype, teacher_logits.dtype
    if len(shape) != 2:
        return AR_ERR_INVALID_ARG, 0, 0, 0, 0
    dt, vt = types.get(dtype), types.get(vdtype)
    if dt is None or vt is None:
        return AR_ERR_UNSUPPORTED, 0, 0, 0, 0
    zs = _row_stride(logits, shape, dtype)
    ds = 0 if dlogits is None else _row_stride(dlogits, shape, dtype)
    if (zs is None or ds is None or len(lists) != 2 or lists[0] != shape[0] or teacher_logits.shape != lists
            or types.get(teacher_index.dtype) != 2 or not teacher_index.is_contiguous()
            or not teacher_logits.is_contiguous()):
        return AR_ERR_INVALID_ARG, 0, 0, 0, 0
    f32, rows = _F32[0], shape[0]
    for r in rows_f32:
        if r is not None and not _vector(r, rows, f32):
            return AR_ERR_INVALID_ARG, 0, 0, 0, 0
    return AR_OK, dt, vt, zs, ds


def ar_distill_loss(logits, teacher_index, teacher_logits, loss, lse, scale=None, dlogits=None, temperature=1.0,
                    stream=None) -> int:
    """loss and lse of each row of logits against the teacher's lists and, with
    dlogits (which may be logits), the gradient of sum(scale * loss)."""
    rc, dt, vt, zs, ds = _distill_operands(logits, teacher_index, teacher_logits, (loss, lse, scale), dlogits)
    if rc:
        return rc
    rows, vocab = logits.shape
    return lib.ar_distill_loss(logits.data_ptr(), zs, teacher_index.data_ptr(), teacher_logits.data_ptr(),
                               None if scale is None else scale.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                               None if dlogits is None else dlogits.data_ptr(), ds, rows, vocab,
                               teacher_index.shape[1], temperature, dt, vt, _stream_of(stream, logits))


def ar_distill_loss_backward(logits, teacher_index, teacher_logits, lse, dloss, dlogits, temperature=1.0,
                             stream=None) -> int:
    """dlogits (which may be logits) for an upstream dloss, from the forward
    call's lse."""
    rc, dt, vt, zs, ds = _distill_operands(logits, teacher_index, teacher_logits, (lse, dloss), dlogits)
    if rc:
        return rc
    rows, vocab = logits.shape
    return lib.ar_distill_loss_backward(logits.data_ptr(), zs, teacher_index.data_ptr(), teacher_logits.data_ptr(),
                                        lse.data_ptr(), dloss.data_ptr(), dlogits.data_ptr(), ds, rows, vocab,
                                        teacher_index.shape[1], temperature, dt, vt, _stream_of(stream, logits))


_TENSOR_BYTES = ctypes.sizeof(AttentionTensor)


def _attention_operands(q, k, queries, keys, cu_seqlens, lse):
    """(status, element type, the operands as an array of ar_attention_tensor):
    q and `queries` are [tokens, heads, dim], k and `keys` [tokens, kv_heads,
    dim], all of one type."""
    types = _TORCH_DTYPE or _dtypes()
    qshape, kshape, dtype = q.shape, k.shape, q.dtype
    if len(qshape) != 3 or len(kshape) != 3 or qshape[0] != kshape[0] or qshape[2] != kshape[2] or qshape[2] < 1:
        return AR_ERR_INVALID_ARG, 0, None
    dt = types.get(dtype)
    if dt is None:
        return AR_ERR_UNSUPPORTED, 0, None
    flat = []
    for t, shape in ((q, qshape), (k, kshape), *((t, kshape) for t in keys), *((t, qshape) for t in queries)):
        if t.dtype is not dtype or t.shape != shape:
            return AR_ERR_INVALID_ARG, 0, None
        token, head, inner = t.stride()
        if inner != 1 and shape[2] > 1:
            return AR_ERR_INVALID_ARG, 0, None
        flat += (t.data_ptr(), token, head)
    if (types.get(cu_seqlens.dtype) != 2 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
            or not cu_seqlens.is_contiguous()):
        return AR_ERR_INVALID_ARG, 0, None
    if lse is not None and (lse.dtype is not _F32[0] or lse.shape != (qshape[1], qshape[0]) or not lse.is_contiguous()):
        return AR_ERR_INVALID_ARG, 0, None
    return AR_OK, dt, array.array("q", flat)


def ar_attention(q, k, v, cu_seqlens, out, lse=None, scale=None, stream=None) -> int:
    """Causal attention of q [tokens, heads, dim] over k and v [tokens,
    kv_heads, dim], tokens packed by cu_seqlens [seqs + 1] (i32, on the
    device).  scale None: dim ** -0.5.  lse [heads, tokens] is what the
    backward call needs."""
    rc, dt, operands = _attention_operands(q, k, (out,), (v,), cu_seqlens, lse)
    if rc:
        return rc
    tokens, heads, dim = q.shape
    at, n = operands.buffer_info()[0], _TENSOR_BYTES
    return lib.ar_attention(at, at + n, at + 2 * n, cu_seqlens.data_ptr(), at + 3 * n,
                            None if lse is None else lse.data_ptr(), tokens, cu_seqlens.numel() - 1, heads,
                            k.shape[1], dim, dim ** -0.5 if scale is None else scale, dt, _stream_of(stream, q))


def ar_attention_workspace_bytes(tokens, heads, kv_heads, dim) -> int:
    return lib.ar_attention_workspace_bytes(int(tokens), int(heads), int(kv_heads), int(dim))


def ar_attention_backward(dout, q, k, v, out, lse, cu_seqlens, dq, dk, dv, workspace, scale=None, stream=None) -> int:
    """dq, dk and dv for an upstream dout, from the forward call's out and
    lse.  workspace: a tensor of at least ar_attention_workspace_bytes(tokens,
    heads, kv_heads, dim) bytes."""
    rc, dt, operands = _attention_operands(q, k, (out, dout, dq), (v, dk, dv), cu_seqlens, lse)
    if rc:
        return rc
    if lse is None or not workspace.is_contiguous():
        return AR_ERR_INVALID_ARG
    tokens, heads, dim = q.shape
    at, n = operands.buffer_info()[0], _TENSOR_BYTES  # q, k, v, dk, dv, out, dout, dq
    return lib.ar_attention_backward(at + 6 * n, at, at + n, at + 2 * n, at + 5 * n, lse.data_ptr(),
                                     cu_seqlens.data_ptr(), at + 7 * n, at + 3 * n, at + 4 * n, tokens,
                                     cu_seqlens.numel() - 1, heads, k.shape[1], dim,
                                     dim ** -0.5 if scale is None else scale, dt, workspace.data_ptr(),
                                     workspace.nbytes, _stream_of(stream, q))


def ar_chunk_range(count, nranks, c):
    lo, hi = ctypes.c_int64(), ctypes.c_int64()
    rc = lib.ar_chunk_range(int(count), int(nranks), int(c), ctypes.byref(lo), ctypes.byref(hi))
    return rc, lo.value, hi.value


def ar_device_status(stream=None):
    """Returns (status of the call, asynchronous device status)."""
    st = ctypes.c_int()
    rc = lib.ar_device_status(_stream(stream), ctypes.byref(st))
    return rc, st.value


def ar_set_barrier_timeout_ns(ns: int) -> int:
    return lib.ar_set_barrier_timeout_ns(int(ns))


def ar_debug_skip_barrier(barrier: int) -> int:
    return lib.ar_debug_skip_barrier(int(barrier))


def ar_last_cuda_error() -> int:
    return lib.ar_last_cuda_error()


def ar_strerror(code: int) -> str:
    return lib.ar_strerror(int(code)).decode()


def ar_version() -> int:
    return lib.ar_version()


def ar_kernel_launches() -> int:
    return lib.ar_kernel_launches()
