"""Thin Python binding of libcoco (include/coco.h): argument marshalling only.

Each ``coco_*`` function here has the name and argument order of the C entry
point. Distributed tensors are described with ``local``, ``sliced`` and
``replicated`` ([CoCoNet] "Breaking the Computation and Communication
Abstraction Barrier in Distributed Machine Learning Workloads", tensor
layouts) from per-rank ``torch.Tensor`` lists (group-major for several
groups); PyTorch provides device memory and streams, every computation runs in
the library's kernels. A failing call raises ``CocoError``.

Importing this module loads ``libcoco.so`` from this package directory and
raises ``ImportError`` if it has not been built (``__graft_entry__.build()``):
there is no fallback.
"""

import ctypes
import functools
import operator
import os
import struct

import torch

# COCO_LIBRARY selects another build of the same library (e.g. build.build_sanitized's).
_LIB_PATH = os.environ.get("COCO_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcoco.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
_lib = ctypes.CDLL(_LIB_PATH)

MAX_PTRS = 64
MAX_DIMS = 3

F32, F16, BF16, F8E4M3 = 0, 1, 2, 3
LOCAL, SLICED, REPLICATED = 0, 1, 2
SCHED_RING, SCHED_UNROLL2, SCHED_BIDIRECTIONAL = 0, 1, 2

STATUS = {
    0: "COCO_OK", 1: "COCO_ERR_NULL", 2: "COCO_ERR_SHAPE", 3: "COCO_ERR_DTYPE", 4: "COCO_ERR_LAYOUT",
    5: "COCO_ERR_ALIGN", 6: "COCO_ERR_ALIAS", 7: "COCO_ERR_UNSUPPORTED", 8: "COCO_ERR_CUDA",
    9: "COCO_ERR_TIMEOUT", 10: "COCO_ERR_VALUE",
}

_DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: F8E4M3}


class CocoTensor(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("ndim", ctypes.c_int32),
        ("slice_dim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * MAX_DIMS),
        ("nranks", ctypes.c_int32),
        ("ngroups", ctypes.c_int32),
        ("ptr", ctypes.c_void_p * MAX_PTRS),
    ]


class CocoScatteredPlan(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("nbuckets", ctypes.c_int64), ("nranks", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class CocoError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        self.name = STATUS.get(status, str(status))
        msg = _lib.coco_status_string(status).decode()
        if status == 8:
            msg += f" (cudaError {_lib.coco_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


_P = ctypes.POINTER(CocoTensor)
_S = ctypes.c_void_p
_B = ctypes.c_void_p  # a coco_tensor or a pointer array, packed into a bytes object (see Dist.packed)
for _name, _args in {
    "coco_fused_allreduce": [_P, ctypes.c_void_p, _P, ctypes.c_float, ctypes.c_uint64, _P, _S],
    "coco_fused_allreduce_at": [_P, ctypes.c_void_p, _P, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, _P, _S],
    "coco_allreduce": [_P, _P, _S],
    "coco_reduce_scatter": [_P, _P, _S],
    "coco_allgather": [_P, _P, _S],
    "coco_allreduce_rs_ag": [_P, _P, _P, _S],
    "coco_allreduce_rs_ag_noalloc": [_P, _P, _S],
    "coco_einsum": [ctypes.c_char_p, _P, _P, _P, _S],
    "coco_einsum_accumulate": [ctypes.c_char_p, _P, _P, _P, _S],
    "coco_matmul_fused_allreduce": [ctypes.c_char_p, _P, _P, ctypes.c_void_p, _P, ctypes.c_float, ctypes.c_uint64,
                                    _P, _S],
    "coco_looped_ag_einsum": [ctypes.c_char_p, _P, _P, _P, _S],
    "coco_looped_einsum_rs": [ctypes.c_char_p, _P, _P, _P, _S],
    "coco_looped_ag_einsum_sched": [ctypes.c_char_p, _P, _P, _P, ctypes.c_int, _S],
    "coco_looped_einsum_rs_sched": [ctypes.c_char_p, _P, _P, _P, ctypes.c_int, _S],
    "coco_dropout_keep_mask": [ctypes.c_uint64, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_void_p, _S],
    "coco_allreduce_rmsnorm": [_B, _B, ctypes.c_void_p, ctypes.c_float, _B, _B, _B, ctypes.c_void_p, _S],
    "coco_allreduce_rmsnorm_backward": [_B, _B, _B, ctypes.c_void_p, ctypes.c_void_p, _B, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, _S],
    "coco_quantize_fp8": [_B, ctypes.c_int32, _B, _B, _S],
    "coco_einsum_fp8": [ctypes.c_char_p, _B, _B, _B, _B, _B, _S],
    "coco_grouped_einsum": [ctypes.c_char_p, _B, _B, _B, _B, ctypes.c_void_p, _B, _S],
    "coco_expert_sort": [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                         ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, _S],
    "coco_expert_dispatch": [_B, _B, ctypes.c_void_p, _B, _B, _S],
    "coco_expert_combine": [_B, ctypes.c_void_p, ctypes.c_void_p, _B, _B, _S],
    "coco_expert_combine_backward": [_B, _B, ctypes.c_void_p, ctypes.c_void_p, _B, ctypes.c_void_p, _S],
    "coco_allreduce_layernorm": [_B, _B, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, _B, _B, _B,
                                 ctypes.c_void_p, ctypes.c_void_p, _S],
    "coco_allreduce_layernorm_backward": [_B, _B, _B, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, _B,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, _S],
    "coco_scattered_clip": [ctypes.POINTER(CocoScatteredPlan), ctypes.c_int32, ctypes.c_float,
                            ctypes.POINTER(CocoScatteredPlan), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, _S],
    "coco_scattered_allreduce_clip": [ctypes.POINTER(CocoScatteredPlan), ctypes.c_float, ctypes.c_float,
                                      ctypes.POINTER(CocoScatteredPlan), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_size_t, _S],
    "coco_device_status": [_S],
    "coco_wait_selftest": [ctypes.c_uint64, _S],
}.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
_lib.coco_scattered_table_bytes.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), ctypes.c_int32]
_lib.coco_scattered_table_bytes.restype = ctypes.c_size_t
_lib.coco_scattered_table_build.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), ctypes.c_int32,
                                            ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.POINTER(CocoScatteredPlan), _S]
_lib.coco_scattered_table_build.restype = ctypes.c_int
_lib.coco_scattered_allreduce.argtypes = [ctypes.POINTER(CocoScatteredPlan), ctypes.c_float, _S]
_lib.coco_scattered_allreduce.restype = ctypes.c_int
_lib.coco_allreduce_rmsnorm_backward_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
_lib.coco_allreduce_rmsnorm_backward_bytes.restype = ctypes.c_size_t
_lib.coco_allreduce_layernorm_backward_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
_lib.coco_allreduce_layernorm_backward_bytes.restype = ctypes.c_size_t
_lib.coco_scattered_clip_bytes.argtypes = []
_lib.coco_scattered_clip_bytes.restype = ctypes.c_size_t
_lib.coco_status_string.argtypes = [ctypes.c_int]
_lib.coco_status_string.restype = ctypes.c_char_p
_lib.coco_last_cuda_error.restype = ctypes.c_int
_lib.coco_version.restype = ctypes.c_int
_lib.coco_kernel_launches.restype = ctypes.c_uint64
_lib.coco_shard_order.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.POINTER(ctypes.c_int32)]
_lib.coco_shard_order.restype = ctypes.c_int
_lib.coco_loop_profitable.argtypes = [ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                      ctypes.POINTER(ctypes.c_int32)]
_lib.coco_loop_profitable.restype = ctypes.c_int
_lib.coco_plan_cache_stats.argtypes = [ctypes.POINTER(ctypes.c_uint64)] * 3
_lib.coco_plan_cache_stats.restype = None
_lib.coco_plan_cache_clear.argtypes = []
_lib.coco_plan_cache_clear.restype = None

EXPORTED = [
    "coco_fused_allreduce", "coco_fused_allreduce_at", "coco_allreduce", "coco_reduce_scatter", "coco_allgather", "coco_allreduce_rs_ag",
    "coco_allreduce_rs_ag_noalloc",
    "coco_einsum", "coco_einsum_accumulate", "coco_matmul_fused_allreduce", "coco_looped_ag_einsum", "coco_looped_einsum_rs",
    "coco_looped_ag_einsum_sched", "coco_looped_einsum_rs_sched", "coco_dropout_keep_mask",
    "coco_scattered_table_bytes", "coco_scattered_table_build", "coco_scattered_allreduce",
    "coco_device_status", "coco_wait_selftest", "coco_kernel_launches", "coco_last_cuda_error", "coco_status_string", "coco_version",
    "coco_shard_order", "coco_loop_profitable", "coco_plan_cache_stats", "coco_plan_cache_clear",
    "coco_allreduce_rmsnorm", "coco_allreduce_rmsnorm_backward", "coco_allreduce_rmsnorm_backward_bytes",
    "coco_quantize_fp8", "coco_einsum_fp8", "coco_grouped_einsum",
    "coco_expert_sort", "coco_expert_dispatch", "coco_expert_combine", "coco_expert_combine_backward",
    "coco_allreduce_layernorm", "coco_allreduce_layernorm_backward", "coco_allreduce_layernorm_backward_bytes",
    "coco_scattered_clip", "coco_scattered_allreduce_clip", "coco_scattered_clip_bytes",
]


def library_path():
    return _LIB_PATH


def version():
    return _lib.coco_version()


def coco_kernel_launches():
    return int(_lib.coco_kernel_launches())


# ------------------------------------------------------------ tensor specs


class Dist:
    """A distributed tensor: per-rank tensors plus layout (marshalled to coco_tensor)."""

    def __init__(self, layout, tensors, shape, slice_dim=-1, ngroups=1, dtype=None):
        self.layout = layout
        self.tensors = list(tensors)
        self.shape = tuple(shape) if type(shape) is torch.Size else tuple(map(int, shape))
        self.slice_dim = slice_dim
        self.ngroups = ngroups
        self.nranks = len(self.tensors) // ngroups
        self.dtype = dtype if dtype is not None else _DTYPES[self.tensors[0].dtype]

    def c(self):
        t = CocoTensor()
        t.dtype = self.dtype
        t.layout = self.layout
        t.ndim = len(self.shape)
        t.slice_dim = self.slice_dim
        for i, s in enumerate(self.shape):
            t.shape[i] = s
        t.nranks = self.nranks
        t.ngroups = self.ngroups
        for i, x in enumerate(self.tensors):
            t.ptr[i] = x.data_ptr() if x is not None else None
        return t

    def packed(self, what):
        """The coco_tensor as bytes: one struct.pack instead of a field at a time, which is most of what a call
        on small tensors costs. The library sees addresses only: that every tensor is dense, and as large as the
        others, is checked here (which costs as much again as taking an address, so once for one that is repeated)."""
        ts, shape = self.tensors, self.shape
        first = ts[0]
        if self.layout == REPLICATED and first is not None:
            for t in ts:
                if t is not first:
                    break
            else:  # (its address, packed once)
                if not first.is_contiguous():
                    raise CocoError(2, what)
                n = len(ts)
                return _tensor_head.pack(self.dtype, REPLICATED, len(shape), self.slice_dim, *(shape + (0, 0, 0))[:3],
                                         self.nranks, self.ngroups) + _one_pointer(first.data_ptr()) * n + _no_pointers(n)
        try:
            addresses = list(map(torch.Tensor.data_ptr, ts))
        except TypeError:  # a None stands for a null pointer
            addresses = [0 if x is None else x.data_ptr() for x in ts]
            ts = [x for x in ts if x is not None]
        if not all(map(torch.Tensor.is_contiguous, ts)) or (len(ts) > 1 and len(set(map(_nbytes, ts))) > 1):
            raise CocoError(2, what)
        return _tensor_struct(len(self.tensors)).pack(
            self.dtype, self.layout, len(shape), self.slice_dim, *(shape + (0, 0, 0))[:3], self.nranks, self.ngroups,
            *addresses)


_nbytes = operator.attrgetter("nbytes")
_tensor_head = struct.Struct("=4i3q2i")
_one_pointer = struct.Struct("=Q").pack


@functools.lru_cache(maxsize=None)
def _no_pointers(n):
    return bytes(8 * max(0, MAX_PTRS - n))


@functools.lru_cache(maxsize=None)
def _tensor_struct(n):
    return struct.Struct(f"=4i3q2i{n}Q{8 * max(0, MAX_PTRS - n)}x")


@functools.lru_cache(maxsize=None)
def _pointer_struct(n):
    return struct.Struct(f"={n}Q")


def local(tensors, ngroups=1):
    """Same shape, different values on every rank."""
    return Dist(LOCAL, tensors, tensors[0].shape, ngroups=ngroups)


def replicated(tensors, ngroups=1):
    """Same values on every rank (a single tensor may be repeated)."""
    return Dist(REPLICATED, tensors, tensors[0].shape, ngroups=ngroups)


def sliced(tensors, dim, ngroups=1):
    """Rank r holds slice r of a tensor split equally along ``dim``."""
    nranks = len(tensors) // ngroups
    shape = list(tensors[0].shape)
    shape[dim] *= nranks
    return Dist(SLICED, tensors, shape, slice_dim=dim, ngroups=ngroups)


def _stream(stream):
    if stream is None:  # the current stream's handle, without building a Stream object around it (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ref(d):
    return None if d is None else ctypes.byref(d.c())


def _check(status, where):
    if status != 0:
        raise CocoError(status, where)


# ------------------------------------------------------------- entry points


def coco_fused_allreduce(partials, bias, residual, dropout_p, seed, out, stream=None):
    bias_ptr = None if bias is None else ctypes.c_void_p(bias.data_ptr())
    _check(_lib.coco_fused_allreduce(_ref(partials), bias_ptr, _ref(residual), float(dropout_p), int(seed),
                                     _ref(out), _stream(stream)), "coco_fused_allreduce")


def coco_fused_allreduce_at(partials, bias, residual, dropout_p, seed, index_base, out, stream=None):
    """coco_fused_allreduce over a contiguous part of larger tensors; index_base is the whole-tensor
    row-major index of the part's first element (dropout indices and bias phase continue from it)."""
    bias_ptr = None if bias is None else ctypes.c_void_p(bias.data_ptr())
    _check(_lib.coco_fused_allreduce_at(_ref(partials), bias_ptr, _ref(residual), float(dropout_p), int(seed),
                                        int(index_base), _ref(out), _stream(stream)), "coco_fused_allreduce_at")


def coco_allreduce(inp, out, stream=None):
    _check(_lib.coco_allreduce(_ref(inp), _ref(out), _stream(stream)), "coco_allreduce")


def coco_reduce_scatter(inp, out, stream=None):
    _check(_lib.coco_reduce_scatter(_ref(inp), _ref(out), _stream(stream)), "coco_reduce_scatter")


def coco_allgather(inp, out, stream=None):
    _check(_lib.coco_allgather(_ref(inp), _ref(out), _stream(stream)), "coco_allgather")


def coco_allreduce_rs_ag(inp, scratch, out, stream=None):
    _check(_lib.coco_allreduce_rs_ag(_ref(inp), _ref(scratch), _ref(out), _stream(stream)), "coco_allreduce_rs_ag")


def coco_allreduce_rs_ag_noalloc(inp, out, stream=None):
    """RS-AG with the library's fixed scratch array (for callers that cannot allocate)."""
    _check(_lib.coco_allreduce_rs_ag_noalloc(_ref(inp), _ref(out), _stream(stream)), "coco_allreduce_rs_ag_noalloc")


def coco_einsum(spec, lhs, rhs, out, stream=None):
    _check(_lib.coco_einsum(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), _stream(stream)), "coco_einsum")


def coco_einsum_accumulate(spec, lhs, rhs, out, stream=None):
    _check(_lib.coco_einsum_accumulate(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), _stream(stream)),
           "coco_einsum_accumulate")


def coco_matmul_fused_allreduce(spec, lhs, rhs, bias, residual, dropout_p, seed, out, stream=None):
    bias_ptr = None if bias is None else ctypes.c_void_p(bias.data_ptr())
    _check(_lib.coco_matmul_fused_allreduce(spec.encode(), _ref(lhs), _ref(rhs), bias_ptr, _ref(residual),
                                            float(dropout_p), int(seed), _ref(out), _stream(stream)),
           "coco_matmul_fused_allreduce")


def coco_looped_ag_einsum(spec, lhs, rhs, out, stream=None):
    _check(_lib.coco_looped_ag_einsum(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), _stream(stream)),
           "coco_looped_ag_einsum")


def coco_looped_einsum_rs(spec, lhs, rhs, out, stream=None):
    _check(_lib.coco_looped_einsum_rs(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), _stream(stream)),
           "coco_looped_einsum_rs")


def coco_looped_ag_einsum_sched(spec, lhs, rhs, out, schedule, stream=None):
    _check(_lib.coco_looped_ag_einsum_sched(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), int(schedule),
                                            _stream(stream)), "coco_looped_ag_einsum_sched")


def coco_looped_einsum_rs_sched(spec, lhs, rhs, out, schedule, stream=None):
    _check(_lib.coco_looped_einsum_rs_sched(spec.encode(), _ref(lhs), _ref(rhs), _ref(out), int(schedule),
                                            _stream(stream)), "coco_looped_einsum_rs_sched")


# -------------------------------------------- 8-bit and expert-grouped operators


def _packed(d, what):
    return None if d is None else d.packed(what)


def _blocks(n):
    return (n + 127) // 128


def _rows_cols(d):
    """Rows and columns of a rank's tensor (all leading dimensions are rows)."""
    x = d.tensors[0]
    cols = x.shape[-1]
    return (x.numel() // cols if cols else 0), cols


def _vector(t, dtype, numel, what):
    """A plain tensor argument's address; the library sees nothing else of it, so its type, size and layout are
    checked here."""
    if t.dtype is not dtype:
        raise CocoError(3, what)
    if t.numel() != numel or not t.is_contiguous():
        raise CocoError(2, what)
    return t.data_ptr()


def _scales(tensors, d, blocks, what):
    """The scale tensors of ``d`` (one per pointer, ``blocks`` values each) as an array of device pointers."""
    if tensors is None:
        return None
    if len(tensors) != len(d.tensors):
        raise CocoError(2, what)
    ptrs, last, p = [], None, 0
    for t in tensors:
        if t is not last:
            last, p = t, _vector(t, torch.float32, blocks, what)
        ptrs.append(p)
    return _pointer_struct(len(ptrs)).pack(*ptrs)


def _check_device(what, *tensors):
    """Refuses host memory. Of a list of ranks' tensors or scales the first stands for all (a look at each costs as
    much as taking its address)."""
    for t in tensors:
        t = t.tensors[0] if type(t) is Dist else t[0] if type(t) is list and t else t
        if isinstance(t, torch.Tensor) and not t.is_cuda:
            raise CocoError(7, f"{what}: a tensor that is not in device memory")


def coco_allreduce_rmsnorm(partials, residual, weight, eps, hidden, normed, scales, rstd, stream=None):
    """h = sum of the ranks' partials + residual; normed = h / sqrt(mean(h^2) + eps) * weight over the last
    dimension. ``hidden`` (the stored h), ``residual`` and ``rstd`` ([groups, rows] fp32) may be None;
    ``normed`` holds the partials' type (``scales`` None) or float8_e4m3fn, with one fp32 scale tensor
    [rows, ceil(cols / 128)] per normed pointer in ``scales``."""
    what = "coco_allreduce_rmsnorm"
    rows, cols = _rows_cols(partials)
    w = _vector(weight, partials.tensors[0].dtype, cols, what)
    r = None if rstd is None else _vector(rstd, torch.float32, rows * partials.ngroups, what)
    sc = _scales(scales, normed, rows * _blocks(cols), what)
    p, res, hid, nrm = partials.packed(what), _packed(residual, what), _packed(hidden, what), normed.packed(what)
    _check_device(what, partials, residual, hidden, normed, weight, rstd, scales)
    _check(_lib.coco_allreduce_rmsnorm(p, res, w, eps, hid, nrm, sc, r, _stream(stream)), what)


def coco_allreduce_rmsnorm_backward_bytes(rows, cols):
    """Workspace bytes of coco_allreduce_rmsnorm_backward for ``rows`` rows (all groups together)."""
    return int(_lib.coco_allreduce_rmsnorm_backward_bytes(int(rows), int(cols)))


def coco_allreduce_rmsnorm_backward(dnormed, dhidden, hidden, weight, rstd, dx, dweight, workspace, stream=None):
    """The gradient of coco_allreduce_rmsnorm: ``dnormed`` LOCAL (summed over the ranks here), ``dhidden`` the
    residual stream's gradient or None; writes ``dx`` (of each partial and of the residual) and ``dweight``
    (fp32). ``workspace``: a device tensor of coco_allreduce_rmsnorm_backward_bytes() bytes."""
    what = "coco_allreduce_rmsnorm_backward"
    rows, cols = _rows_cols(dnormed)
    w = _vector(weight, dnormed.tensors[0].dtype, cols, what)
    r = _vector(rstd, torch.float32, rows * dnormed.ngroups, what)
    dw = _vector(dweight, torch.float32, cols, what)
    if not workspace.is_contiguous():
        raise CocoError(2, what)
    dn, dh, hid, o = dnormed.packed(what), _packed(dhidden, what), hidden.packed(what), dx.packed(what)
    _check_device(what, dnormed, dhidden, hidden, dx, weight, rstd, dweight, workspace)
    _check(_lib.coco_allreduce_rmsnorm_backward(dn, dh, hid, w, r, o, dw, workspace.data_ptr(), workspace.nbytes,
                                                _stream(stream)), what)


def coco_quantize_fp8(x, block_rows, q, scales, stream=None):
    """Every rank's x as float8_e4m3fn values ``q`` and fp32 ``scales`` (one tensor per rank): one scale per row
    and 128 columns (``block_rows`` 1) or per 128 x 128 tile of each matrix (128)."""
    what = "coco_quantize_fp8"
    rows, cols = _rows_cols(x)
    if block_rows == 128:
        mats = x.shape[0] if len(x.shape) == 3 else 1
        blocks = mats * _blocks(rows // mats if mats else 0) * _blocks(cols)
    else:
        blocks = rows * _blocks(cols)
    sc = _scales(scales, q, blocks, what)
    xp, qp = x.packed(what), q.packed(what)
    _check_device(what, x, q, scales)
    _check(_lib.coco_quantize_fp8(xp, block_rows, qp, sc, _stream(stream)), what)


def _operand_scales(lhs, lhs_scales, rhs, rhs_scales, what):
    """The scale arrays of a product's operands: per row and 128 columns, and per 128 x 128 tile of each matrix."""
    if lhs_scales is None and rhs_scales is None:
        return None, None
    rows, cols = _rows_cols(lhs)
    shape = rhs.tensors[0].shape
    tiles = (shape[0] if len(shape) == 3 else 1) * _blocks(shape[-2] if len(shape) > 1 else 1) * _blocks(shape[-1])
    return _scales(lhs_scales, lhs, rows * _blocks(cols), what), _scales(rhs_scales, rhs, tiles, what)


def coco_einsum_fp8(spec, lhs, lhs_scales, rhs, rhs_scales, out, stream=None):
    """out_r = lhs_r @ rhs_r on float8_e4m3fn operands with fp32 scales per 1 x 128 (lhs) and 128 x 128 (rhs)
    block; ``spec`` "mk,kn->mn" or "mk,nk->mn". Scale tensors: one per pointer of the operand."""
    what = "coco_einsum_fp8"
    sa, sb = _operand_scales(lhs, lhs_scales, rhs, rhs_scales, what)
    a, b, o = lhs.packed(what), rhs.packed(what), out.packed(what)
    _check_device(what, lhs, rhs, out, lhs_scales, rhs_scales)
    _check(_lib.coco_einsum_fp8(spec.encode(), a, sa, b, sb, o, _stream(stream)), what)


def coco_grouped_einsum(spec, lhs, lhs_scales, rhs, rhs_scales, offsets, out, stream=None):
    """Products grouped by expert: rows [offsets[e], offsets[e + 1]) of lhs belong to expert e. ``spec``
    "tk,ekn->tn", "tk,enk->tn" or the weight gradient "tk,tn->ekn"; ``offsets`` an int32 device tensor
    [ranks, experts + 1]; scale lists for float8_e4m3fn operands, else None."""
    what = "coco_grouped_einsum"
    sa, sb = _operand_scales(lhs, lhs_scales, rhs, rhs_scales, what)
    experts = (rhs if len(rhs.shape) == 3 else out).shape[0]
    off = None if offsets is None else _vector(offsets, torch.int32, len(lhs.tensors) * (experts + 1), what)
    a, b, o = lhs.packed(what), rhs.packed(what), out.packed(what)
    _check_device(what, lhs, rhs, out, offsets, lhs_scales, rhs_scales)
    _check(_lib.coco_grouped_einsum(spec.encode(), a, sa, b, sb, off, o, _stream(stream)), what)


# --------------------------------- experts' rows, layer norm, gradient clipping


def _check_here(what, *tensors):
    """Refuses host memory and any device but the current one, on which the call runs; of lists the first tensor stands
    for all, as in _check_device (this is one look at each)."""
    here = None
    for t in tensors:
        kind = type(t)
        if kind is Dist:
            t = t.tensors[0]
        elif kind is list or kind is tuple:
            t = t[0] if t else None
        if t is not None:
            at = t.get_device()
            if at < 0:
                raise CocoError(7, f"{what}: a tensor that is not in device memory")
            if at != here:
                if here is not None or at != torch._C._cuda_getDevice():
                    raise CocoError(7, f"{what}: a tensor of another device than the current one")
                here = at


def _pointer(t, dtype, numel, what):
    """A plain tensor argument's address, or None."""
    return None if t is None else _vector(t, dtype, numel, what)


def _per_choice(t, dtype, tokens, rows, groups, what):
    """The address of a tensor with a value for every token's choices, or None: [groups, tokens, choices] in this order, of
    which neighbours may be one dimension. The number of its elements does not tell it from another order."""
    if t is None:
        return None
    p = _vector(t, dtype, rows * groups, what)
    shape = t.shape
    if len(shape) != 2 or shape[1] * tokens != rows:
        n, runs = 1, (1, rows // tokens if tokens else 0, rows, rows * groups)
        for d in reversed(shape):
            n *= d
            if n not in runs and t.numel():
                raise CocoError(2, what)
    return p


def coco_expert_sort(expert_of, experts, row_of_choice, choice_of_row, offsets, stream=None):
    """The rows of a mixture of experts, sorted by expert. ``expert_of`` [tokens, choices] or [groups, tokens, choices]
    (int32 or int64; a number outside [0, experts) has no row) gives ``row_of_choice`` (int32, the same shape, -1 for
    no row), ``choice_of_row`` (int32 [groups, tokens * choices] or None; -1 behind the last expert's rows) and
    ``offsets`` (int32 [groups * ranks, experts + 1], a line per rank as coco_grouped_einsum reads them)."""
    what = "coco_expert_sort"
    shape = expert_of.shape
    if not 2 <= len(shape) <= 3 or not expert_of.is_contiguous() or offsets.dim() != 2:
        raise CocoError(2, what)
    if expert_of.dtype not in (torch.int64, torch.int32):
        raise CocoError(3, what)
    groups = shape[0] if len(shape) == 3 else 1
    lines = offsets.shape[0]
    if groups < 1 or lines % groups:
        raise CocoError(2, what)
    n = expert_of.numel()
    row = _per_choice(row_of_choice, torch.int32, shape[-2], n // groups, groups, what)
    choice = _pointer(choice_of_row, torch.int32, n, what)
    off = _vector(offsets, torch.int32, lines * (experts + 1), what)
    _check_here(what, expert_of, row_of_choice, choice_of_row, offsets)
    _check(_lib.coco_expert_sort(expert_of.data_ptr(), expert_of.element_size(), shape[-2], shape[-1], experts, groups,
                                 lines // groups, row, choice, off, _stream(stream)), what)


def _row_scales(tensors, d, what):
    if tensors is None:
        return None
    rows, cols = _rows_cols(d)
    return _scales(tensors, d, rows * _blocks(cols), what)


def coco_expert_dispatch(x, x_scales, row_of_choice, rows, row_scales, stream=None):
    """rows[row_of_choice[t, k]] = x[t]: ``x`` REPLICATED [tokens, cols] to ``rows`` REPLICATED [tokens * choices,
    cols], with a scale tensor per pointer where they are float8_e4m3fn (else None). Rows that no choice names are left
    as they were."""
    what = "coco_expert_dispatch"
    sx, sr = _row_scales(x_scales, x, what), _row_scales(row_scales, rows, what)
    row = _per_choice(row_of_choice, torch.int32, x.shape[0], rows.shape[0], rows.ngroups, what)
    xp, rp = x.packed(what), rows.packed(what)
    _check_here(what, x, rows, row_of_choice, x_scales, row_scales)
    _check(_lib.coco_expert_dispatch(xp, sx, row, rp, sr, _stream(stream)), what)


def coco_expert_combine(rows, row_of_choice, gates, residual, out, stream=None):
    """out[t] = sum over k of gates[t, k] * rows[row_of_choice[t, k]]: every rank's own sum (``out`` LOCAL, ``residual``
    None), or their AllReduce with the residual (``out`` REPLICATED). ``gates``: fp32, the shape of ``row_of_choice``, or
    None for ones, which is the dispatch's gradient."""
    what = "coco_expert_combine"
    tokens, n, groups = out.shape[0], rows.shape[0], rows.ngroups
    row = _per_choice(row_of_choice, torch.int32, tokens, n, groups, what)
    w = _per_choice(gates, torch.float32, tokens, n, groups, what)
    rp, res, o = rows.packed(what), _packed(residual, what), out.packed(what)
    _check_here(what, rows, residual, out, row_of_choice, gates)
    _check(_lib.coco_expert_combine(rp, row, w, res, o, _stream(stream)), what)


def coco_expert_combine_backward(dout, rows, row_of_choice, gates, drows, dgates, stream=None):
    """The gradient of coco_expert_combine: ``drows`` (REPLICATED: every rank's is the same) and ``dgates`` (fp32, the
    shape of ``row_of_choice``; None with ``rows`` None) for ``dout``, the gradient of the summed output."""
    what = "coco_expert_combine_backward"
    tokens, n, groups = dout.shape[0], drows.shape[0], drows.ngroups
    row = _per_choice(row_of_choice, torch.int32, tokens, n, groups, what)
    w = _per_choice(gates, torch.float32, tokens, n, groups, what)
    dw = _per_choice(dgates, torch.float32, tokens, n, groups, what)
    d, rp, o = dout.packed(what), _packed(rows, what), drows.packed(what)
    _check_here(what, dout, rows, drows, row_of_choice, gates, dgates)
    _check(_lib.coco_expert_combine_backward(d, rp, row, w, o, dw, _stream(stream)), what)


def coco_allreduce_layernorm(partials, residual, weight, bias, eps, hidden, normed, scales, mean, rstd, stream=None):
    """h = sum of the ranks' partials + residual; normed = (h - mean) / sqrt(variance + eps) * weight + bias over the
    last dimension. ``bias``, ``residual``, ``hidden`` (the stored h), ``mean`` and ``rstd`` ([groups, rows] fp32) may be
    None; ``normed`` and ``scales`` as coco_allreduce_rmsnorm's."""
    what = "coco_allreduce_layernorm"
    rows, cols = _rows_cols(partials)
    dtype, n = partials.tensors[0].dtype, rows * partials.ngroups
    w, b = _vector(weight, dtype, cols, what), _pointer(bias, dtype, cols, what)
    m, r = _pointer(mean, torch.float32, n, what), _pointer(rstd, torch.float32, n, what)
    sc = _scales(scales, normed, rows * _blocks(cols), what)
    p, res, hid, nrm = partials.packed(what), _packed(residual, what), _packed(hidden, what), normed.packed(what)
    _check_here(what, partials, residual, hidden, normed, weight, bias, mean, rstd, scales)
    _check(_lib.coco_allreduce_layernorm(p, res, w, b, eps, hid, nrm, sc, m, r, _stream(stream)), what)


def coco_allreduce_layernorm_backward_bytes(rows, cols):
    """Workspace bytes of coco_allreduce_layernorm_backward for ``rows`` rows (all groups together)."""
    return int(_lib.coco_allreduce_layernorm_backward_bytes(int(rows), int(cols)))


def coco_allreduce_layernorm_backward(dnormed, dhidden, hidden, weight, mean, rstd, dx, dweight, dbias, workspace,
                                      stream=None):
    """The gradient of coco_allreduce_layernorm: ``dnormed`` LOCAL (summed over the ranks here), ``dhidden`` the
    residual stream's gradient or None; writes ``dx`` (of each partial and of the residual), ``dweight`` and ``dbias``
    (fp32; the latter may be None). ``workspace``: coco_allreduce_layernorm_backward_bytes() bytes."""
    what = "coco_allreduce_layernorm_backward"
    rows, cols = _rows_cols(dnormed)
    w = _vector(weight, dnormed.tensors[0].dtype, cols, what)
    m = _vector(mean, torch.float32, rows * dnormed.ngroups, what)
    r = _vector(rstd, torch.float32, rows * dnormed.ngroups, what)
    dw, db = _vector(dweight, torch.float32, cols, what), _pointer(dbias, torch.float32, cols, what)
    if not workspace.is_contiguous():
        raise CocoError(2, what)
    dn, dh, hid, o = dnormed.packed(what), _packed(dhidden, what), hidden.packed(what), dx.packed(what)
    _check_here(what, dnormed, dhidden, hidden, dx, weight, mean, rstd, dweight, dbias, workspace)
    _check(_lib.coco_allreduce_layernorm_backward(dn, dh, hid, w, m, r, o, dw, db, workspace.data_ptr(),
                                                  workspace.nbytes, _stream(stream)), what)


def coco_scattered_clip_bytes():
    """Workspace bytes of coco_scattered_clip and coco_scattered_allreduce_clip."""
    return int(_lib.coco_scattered_clip_bytes())


def _clip(name, plan, second, max_norm, out, norm, workspace, stream):
    n = _vector(norm, torch.float32, 1, name)
    if not workspace.is_contiguous():
        raise CocoError(2, name)
    _check_here(name, norm, workspace)
    _check(getattr(_lib, name)(ctypes.byref(plan), second, float(max_norm), None if out is None else ctypes.byref(out), n,
                               workspace.data_ptr(), workspace.nbytes, _stream(stream)), name)


def coco_scattered_clip(plan, layout, max_norm, out, norm, workspace, stream=None):
    """Scales the plan's tensors so that their norm is at most ``max_norm`` (inf: only the norm), into the tensors of
    the plan ``out`` (None: in place); ``norm`` (one fp32) receives the norm before. ``layout`` LOCAL: the ranks'
    tensors are parts of one gradient; REPLICATED: copies of it. ``workspace``: coco_scattered_clip_bytes() bytes."""
    _clip("coco_scattered_clip", plan, layout, max_norm, out, norm, workspace, stream)


def coco_scattered_allreduce_clip(plan, alpha, max_norm, out, norm, workspace, stream=None):
    """coco_scattered_allreduce (alpha times the sum over the ranks) with the sum's norm and clipping fused in."""
    _clip("coco_scattered_allreduce_clip", plan, alpha, max_norm, out, norm, workspace, stream)


def coco_dropout_keep_mask(seed, dropout_p, first_index, count, mask, stream=None):
    ptr = None if mask is None else ctypes.c_void_p(mask.data_ptr())
    _check(_lib.coco_dropout_keep_mask(int(seed), float(dropout_p), int(first_index), int(count), ptr,
                                       _stream(stream)), "coco_dropout_keep_mask")


def coco_device_status(stream=None):
    _check(_lib.coco_device_status(_stream(stream)), "coco_device_status")


def coco_wait_selftest(timeout_ns, stream=None):
    """Launches the failure-path self-test: a bounded wait on a barrier nothing completes
    (``timeout_ns`` limit); the next coco_device_status raises COCO_ERR_TIMEOUT."""
    _check(_lib.coco_wait_selftest(int(timeout_ns), _stream(stream)), "coco_wait_selftest")


def raw_call(name, *args):
    """Calls a C entry point with already-marshalled ctypes arguments and
    returns its status code (used by the interface tests)."""
    return getattr(_lib, name)(*args)


def coco_scattered_table_bytes(numels, nranks):
    arr = (ctypes.c_int64 * len(numels))(*[int(n) for n in numels])
    return int(_lib.coco_scattered_table_bytes(len(numels), arr, int(nranks)))


def coco_scattered_table_build(per_rank, table, stream=None):
    """``per_rank[r][t]``: rank r's tensor t (same sizes and dtype on every rank);
    ``table``: a device uint8 tensor of at least coco_scattered_table_bytes() bytes.
    Returns the plan for coco_scattered_allreduce."""
    nranks, ntensors = len(per_rank), len(per_rank[0])
    numels = (ctypes.c_int64 * ntensors)(*[x.numel() for x in per_rank[0]])
    ptrs = (ctypes.c_void_p * (nranks * ntensors))(*[x.data_ptr() if x.numel() else None
                                                     for row in per_rank for x in row])
    plan = CocoScatteredPlan()
    dtype = _DTYPES[per_rank[0][0].dtype] if ntensors else F32
    _check(_lib.coco_scattered_table_build(ntensors, numels, dtype, nranks, ptrs, ctypes.c_void_p(table.data_ptr()),
                                           table.numel() * table.element_size(), ctypes.byref(plan), _stream(stream)),
           "coco_scattered_table_build")
    return plan


def coco_scattered_allreduce(plan, alpha=1.0, stream=None):
    _check(_lib.coco_scattered_allreduce(ctypes.byref(plan), float(alpha), _stream(stream)), "coco_scattered_allreduce")


AG_ORDER, RS_ORDER = 0, 1


def coco_shard_order(kind, schedule, rank, nranks):
    """The planner's shard schedule for one rank (see coco.h): kind AG_ORDER gives the shard visited at
    each AllGather-Einsum step, RS_ORDER the rank whose partial output shard ``rank`` collects at each
    Einsum-ReduceScatter step."""
    arr = (ctypes.c_int32 * max(1, int(nranks)))()
    _check(_lib.coco_shard_order(int(kind), int(schedule), int(rank), int(nranks), arr), "coco_shard_order")
    return [int(arr[i]) for i in range(int(nranks))]


def coco_loop_profitable(orig_comp, orig_comm, ring_comm, epilogue_cost):
    """[Decomp] §5.5 cost model: True when the Looped CollectiveEinsum is expected to beat the original
    collective followed by the einsum (times in one unit)."""
    out = ctypes.c_int32(-1)
    _check(_lib.coco_loop_profitable(float(orig_comp), float(orig_comm), float(ring_comm), float(epilogue_cost),
                                     ctypes.byref(out)), "coco_loop_profitable")
    return bool(out.value)


def coco_plan_cache_stats():
    """(hits, misses, entries) of the library's plan cache."""
    h, m, e = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    _lib.coco_plan_cache_stats(ctypes.byref(h), ctypes.byref(m), ctypes.byref(e))
    return int(h.value), int(m.value), int(e.value)


def coco_plan_cache_clear():
    _lib.coco_plan_cache_clear()
