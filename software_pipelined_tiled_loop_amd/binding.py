"""ctypes binding of the C ABI in include/pgemm.h (argument marshalling only).

Every entry point keeps its C name and argument order.  Pointer arguments
accept either an integer device address or a torch tensor (its data_ptr());
``stream`` accepts an integer hipStream_t, a torch stream, or None for torch's
current stream on the current device.  The functions return the C status code;
``gemm`` is a convenience wrapper that raises PgemmError on a nonzero status.

Importing this module loads libpgemm.so and raises ImportError when the HIP
library has not been built: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpgemm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libpgemm.so is not built (run __graft_entry__.build() or "
                      "python -m software_pipelined_tiled_loop_amd.build); there is no fallback")

# torch ships its own HIP and HSA runtimes under the same sonames as the ROCm
# install the library is linked against.  Whichever is loaded first is the one
# the other binds to; loading libpgemm.so first would leave two HIP runtimes in
# the process, and the library's would find no device.  So torch, when
# present, is loaded first and the library shares its runtime, its device
# memory and its streams.
try:
    import torch  # noqa: F401
except ImportError:  # a caller without torch uses the ROCm runtime directly
    pass

_lib = ctypes.CDLL(LIB_PATH)

PGEMM_F32, PGEMM_F16, PGEMM_BF16, PGEMM_I8 = 0, 1, 2, 3
DTYPE_CODE = {"f32": PGEMM_F32, "f16": PGEMM_F16, "bf16": PGEMM_BF16, "i8": PGEMM_I8}
PRODUCER = {"auto": 0, "direct": 1, "register": 2, "generic": 3, "staged_a": 4, "staged_b": 5}
# pgemm_aligned: which operands meet the chunk rule (rows of whole 16-byte chunks)
ALIGNED_NONE, ALIGNED_BOTH, ALIGNED_A, ALIGNED_B = 0, 1, 2, 3
PRODUCER_NAME = {v: k for k, v in PRODUCER.items()}
STATUS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED_DTYPE", -3: "BAD_STAGES", -4: "INFEASIBLE_PLAN",
          -5: "NONINTEGRAL_SCALAR", -6: "HIP", -7: "TOO_LARGE"}


class pgemm_opts(ctypes.Structure):
    _fields_ = [("producer", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_k", ctypes.c_int), ("skew", ctypes.c_int), ("workgroups", ctypes.c_int),
                ("waves", ctypes.c_int), ("reserved", ctypes.c_int * 1)]


class pgemm_plan_info(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int), ("tile_k", ctypes.c_int),
                ("stages", ctypes.c_int), ("stages_eff", ctypes.c_int), ("num_k_tiles", ctypes.c_int),
                ("producer", ctypes.c_int), ("threads", ctypes.c_int), ("waves_m", ctypes.c_int),
                ("waves_n", ctypes.c_int), ("lds_bytes", ctypes.c_int), ("wg_per_cu", ctypes.c_int),
                ("grid", ctypes.c_int), ("variant", ctypes.c_int), ("est_uncovered_cycles", ctypes.c_double)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["producer"] = PRODUCER_NAME.get(d["producer"], d["producer"])
        return d


_i64, _dbl, _vp, _int = ctypes.c_int64, ctypes.c_double, ctypes.c_void_p, ctypes.c_int
_lib.pgemm_gemm.argtypes = [_i64, _i64, _i64, _dbl, _vp, _i64, _vp, _i64, _dbl, _vp, _i64, _int, _int, _vp]
_lib.pgemm_gemm.restype = _int
_lib.pgemm_gemm_ex.argtypes = [_i64, _i64, _i64, _dbl, _vp, _i64, _vp, _i64, _dbl, _vp, _i64, _int, _int,
                               ctypes.POINTER(pgemm_opts), _vp]
_lib.pgemm_gemm_ex.restype = _int
_lib.pgemm_plan.argtypes = [_i64, _i64, _i64, _int, _int, _int, ctypes.POINTER(pgemm_opts),
                            ctypes.POINTER(pgemm_plan_info)]
_lib.pgemm_plan.restype = _int
_lib.pgemm_strerror.argtypes = [_int]
_lib.pgemm_strerror.restype = ctypes.c_char_p
_lib.pgemm_num_variants.argtypes = []
_lib.pgemm_num_variants.restype = _int
_lib.pgemm_variant_info.argtypes = [_int, ctypes.POINTER(pgemm_plan_info), ctypes.POINTER(_int)]
_lib.pgemm_variant_info.restype = _int
_lib.pgemm_version.restype = _int
_lib.pgemm_model_uncovered_cycles.argtypes = [_dbl, _dbl, _int]
_lib.pgemm_model_uncovered_cycles.restype = _dbl
_lib.pgemm_model_lds_bytes.argtypes = [_int, _int, _int, _int, _int, _int]
_lib.pgemm_model_lds_bytes.restype = _i64
_lib.pgemm_model_global_loads_per_output.argtypes = [_int, _int, _i64]
_lib.pgemm_model_global_loads_per_output.restype = _dbl
_lib.pgemm_model_compute_load_ratio.argtypes = [_int, _int, _int, _int]
_lib.pgemm_model_compute_load_ratio.restype = _dbl
_lib.pgemm_hazard_copy_reduce.argtypes = [_vp, _i64, _i64, _i64, _vp, _int, _int, _int, _vp, _i64, _int, _vp]
_lib.pgemm_hazard_copy_reduce.restype = _int
_lib.pgemm_diag_mfma_ceiling.argtypes = [_int, _int, _int, _int, _int, _int, ctypes.c_uint32, _vp, ctypes.POINTER(_i64),
                                         _vp, _vp]
_lib.pgemm_diag_mfma_ceiling.restype = _int
_lib.pgemm_diag_lds_stream.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _int, _int, _int, _int, _int,
                                       ctypes.POINTER(_i64), _vp]
_lib.pgemm_diag_lds_stream.restype = _int
_lib.pgemm_diag_wait_profile.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _int, _int, _int,
                                         _int, _vp, _i64, _vp]
_lib.pgemm_diag_wait_profile.restype = _int
_lib.pgemm_diag_parts.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _int, _int, _int, _int,
                                  _int, _vp, _i64, _vp]
_lib.pgemm_diag_parts.restype = _int
for _f, _n in (("pgemm_linear_workspace", 3), ("pgemm_gated_workspace", 3), ("pgemm_linear_backward_workspace", 3),
               ("pgemm_gated_backward_workspace", 3)):
    getattr(_lib, _f).argtypes = [_i64] * _n + [_int] * (2 if _f == "pgemm_linear_backward_workspace" else 1)
    getattr(_lib, _f).restype = _i64
_lib.pgemm_linear.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _vp, _i64, _int, _vp, _i64, _vp, _i64,
                              _int, _int, _vp, _i64, _vp]
_lib.pgemm_linear.restype = _int
_lib.pgemm_gated.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _int, _vp, _vp, _int, _vp, _i64, _vp, _i64,
                             _vp, _i64, _int, _int, _vp, _i64, _vp]
_lib.pgemm_gated.restype = _int
_lib.pgemm_linear_backward.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _int, _vp,
                                       _i64, _vp, _i64, _int, _vp, _int, _int, _vp, _i64, _vp]
_lib.pgemm_linear_backward.restype = _int
_lib.pgemm_gated_backward.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _int, _vp, _i64, _vp,
                                      _i64, _int, _vp, _i64, _vp, _vp, _i64, _int, _vp, _vp, _int, _int, _vp, _i64,
                                      _vp]
_lib.pgemm_gated_backward.restype = _int

ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
ORDER_KN, ORDER_NK = 0, 1

# Steady-state parts of a parts-ladder build (enum pgemm_part).
PART_DMA, PART_BARRIER, PART_AREADS, PART_BREADS, PART_ALL = 1, 2, 4, 8, 15

EXPORTED = ("pgemm_gemm", "pgemm_gemm_ex", "pgemm_plan", "pgemm_strerror", "pgemm_num_variants",
            "pgemm_variant_info", "pgemm_version", "pgemm_model_uncovered_cycles", "pgemm_model_lds_bytes",
            "pgemm_model_global_loads_per_output", "pgemm_model_compute_load_ratio", "pgemm_hazard_copy_reduce",
            "pgemm_diag_mfma_ceiling", "pgemm_diag_lds_stream", "pgemm_diag_wait_profile", "pgemm_diag_parts",
            "pgemm_linear", "pgemm_gated", "pgemm_linear_backward", "pgemm_gated_backward", "pgemm_linear_workspace",
            "pgemm_gated_workspace", "pgemm_linear_backward_workspace", "pgemm_gated_backward_workspace")


class PgemmError(RuntimeError):
    def __init__(self, status):
        super().__init__("pgemm status %d (%s): %s" % (status, STATUS.get(status, "?"), pgemm_strerror(status)))
        self.status = status


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _opts(producer=None, tile=None, skew=0, workgroups=0, waves=0):
    if producer is None and tile is None and not skew and not workgroups and not waves:
        return None
    o = pgemm_opts()
    o.producer = PRODUCER[producer] if isinstance(producer, str) else int(producer or 0)
    if tile is not None:
        o.tile_m, o.tile_n, o.tile_k = (int(v) for v in tile)
    o.skew = int(skew)
    o.workgroups = int(workgroups)
    o.waves = int(waves)
    return o


def _opts_from(d):
    return _opts(d.get("producer"), d.get("tile"), d.get("skew", 0), d.get("workgroups", 0), d.get("waves", 0))


def pgemm_gemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype, stages, stream=None):
    return _lib.pgemm_gemm(M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb, float(beta), _ptr(C), ldc,
                           DTYPE_CODE.get(dtype, dtype), stages, _stream(stream))


def pgemm_gemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype, stages, opts=None, stream=None):
    if isinstance(opts, dict):
        opts = _opts_from(opts)
    p = ctypes.byref(opts) if opts is not None else None
    return _lib.pgemm_gemm_ex(M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb, float(beta), _ptr(C), ldc,
                              DTYPE_CODE.get(dtype, dtype), stages, p, _stream(stream))


def pgemm_plan(M, N, K, dtype, stages=0, aligned=1, opts=None):
    """Returns (status, plan dict or None)."""
    if isinstance(opts, dict):
        opts = _opts_from(opts)
    info = pgemm_plan_info()
    r = _lib.pgemm_plan(M, N, K, DTYPE_CODE.get(dtype, dtype), stages, int(aligned),
                        ctypes.byref(opts) if opts is not None else None, ctypes.byref(info))
    return r, (info.as_dict() if r == 0 else None)


def pgemm_strerror(status):
    return _lib.pgemm_strerror(int(status)).decode()


def pgemm_num_variants():
    return _lib.pgemm_num_variants()


def pgemm_variant_info(index):
    info = pgemm_plan_info()
    dt = _int(0)
    r = _lib.pgemm_variant_info(index, ctypes.byref(info), ctypes.byref(dt))
    if r != 0:
        raise PgemmError(r)
    d = info.as_dict()
    d["dtype"] = {v: k for k, v in DTYPE_CODE.items()}[dt.value]
    return d


def pgemm_version():
    return _lib.pgemm_version()


def pgemm_model_uncovered_cycles(latency, compute, stages):
    return _lib.pgemm_model_uncovered_cycles(float(latency), float(compute), int(stages))


def pgemm_model_lds_bytes(bm, bn, bk, stages, elem_bytes, a_pad=0):
    return _lib.pgemm_model_lds_bytes(bm, bn, bk, stages, elem_bytes, a_pad)


def pgemm_model_global_loads_per_output(bm, bn, K):
    return _lib.pgemm_model_global_loads_per_output(bm, bn, K)


def pgemm_model_compute_load_ratio(bm, bn, bk, elem_bytes):
    return _lib.pgemm_model_compute_load_ratio(bm, bn, bk, elem_bytes)


def _regions_overlap(X, xr, xc, Y, yr, yc):
    """Whether the first xr rows x xc columns of 2-D tensor X share a byte
    with the first yr x yc of Y (rows at each tensor's row stride).  Exact
    when both row strides in bytes are equal (slices of one matrix); with
    different strides, any overlap of the two byte ranges counts."""
    if not (xr and xc and yr and yc):
        return False
    sx, sy = X.stride(0) * X.element_size(), Y.stride(0) * Y.element_size()
    wx, wy = xc * X.element_size(), yc * Y.element_size()
    x0, y0 = X.data_ptr(), Y.data_ptr()
    if x0 >= y0 + (yr - 1) * sy + wy or y0 >= x0 + (xr - 1) * sx + wx:
        return False
    if sx != sy or sx == 0:
        return True
    # row i of X and row j of Y meet iff -wy < d + (j - i) * s < wx, d = y0 - x0
    d = y0 - x0
    t0 = -d // sx
    for t in range(t0 - 1, t0 + 3):
        if -(xr - 1) <= t <= yr - 1 and -wy < d + t * sx < wx:
            return True
    return False


def gemm(A, B, C, alpha=1.0, beta=0.0, stages=0, producer=None, tile=None, M=None, N=None, K=None,
         stream=None):
    """C = alpha*A@B + beta*C on torch tensors (2-D, row-major, unit column stride).

    dtype is taken from A: float32 -> f32, float16 -> f16, bfloat16 -> bf16, int8 -> i8.
    B must have A's dtype; C is float32 (int32 for int8).  Sizes default to the
    logical shapes and must fit inside the tensors; leading dimensions are the
    row strides.  All three tensors must live on one GPU, and C must not
    overlap A or B; the call runs on that GPU (torch's current stream there
    unless `stream` is given).  Every check runs
    before anything reaches the library, so a bad call raises ValueError and
    launches nothing.
    """
    import torch
    in_dt = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16", torch.int8: "i8"}
    if A.dtype not in in_dt:
        raise ValueError("A has unsupported dtype %s" % A.dtype)
    dt = in_dt[A.dtype]
    out_dt = torch.int32 if dt == "i8" else torch.float32
    if B.dtype != A.dtype:
        raise ValueError("B must have A's dtype %s, got %s" % (A.dtype, B.dtype))
    if C.dtype != out_dt:
        raise ValueError("C must be %s for %s inputs, got %s" % (out_dt, A.dtype, C.dtype))
    for name, t in (("A", A), ("B", B), ("C", C)):
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError("%s must be a 2-D row-major tensor with unit column stride" % name)
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[1] if N is None else N
    for name, t, rows, cols in (("A", A, M, K), ("B", B, K, N), ("C", C, M, N)):
        if rows < 0 or cols < 0 or (rows and cols and (t.shape[0] < rows or t.shape[1] < cols)):
            raise ValueError("%s is %s, the call needs %d x %d" % (name, tuple(t.shape), rows, cols))
    for name, t, rows, cols in (("A", A, M, K), ("B", B, K, N)):
        if t.device == C.device and _regions_overlap(t, rows, cols, C, M, N):
            raise ValueError("C overlaps %s: the output must not share memory with an input" % name)
    devs = {t.device for t in (A, B, C)}
    if len(devs) != 1 or next(iter(devs)).type != "cuda":
        raise ValueError("A, B and C must be GPU tensors on one device, got %s" % sorted(str(d) for d in devs))
    # the library launches on the current device: make it the tensors' one
    with torch.cuda.device(C.device):
        r = pgemm_gemm_ex(M, N, K, alpha, A, max(A.stride(0), 1), B, max(B.stride(0), 1), beta, C,
                          max(C.stride(0), 1), dt, stages, _opts(producer, tile), stream)
    if r != 0:
        raise PgemmError(r)
    return C


# ---- feed-forward operators ------------------------------------------------------------

# The C entry points, with their names and argument order; every pointer is a
# device address (or None) and the stream a hipStream_t.
pgemm_linear = _lib.pgemm_linear
pgemm_gated = _lib.pgemm_gated
pgemm_linear_backward = _lib.pgemm_linear_backward
pgemm_gated_backward = _lib.pgemm_gated_backward
pgemm_linear_workspace = _lib.pgemm_linear_workspace
pgemm_gated_workspace = _lib.pgemm_gated_workspace
pgemm_linear_backward_workspace = _lib.pgemm_linear_backward_workspace
pgemm_gated_backward_workspace = _lib.pgemm_gated_backward_workspace


class _Call:
    """The checks that the four operators share, and their launch.

    An operator's checks of types, shapes, strides and devices depend on
    nothing else, so they run once for each combination of them: the operator
    describes its call on an instance, which `_cached` then keeps.  What
    depends on addresses (overlaps, the workspace) is checked at every call.
    """

    __slots__ = ("dtype", "device", "index", "tensors", "pairs", "args", "need", "function")

    def __init__(self, X):
        code = _FLOAT_CODE.get(X.dtype)
        if code is None:
            raise ValueError("X has unsupported dtype %s: float32, float16 or bfloat16 is needed" % X.dtype)
        self.dtype = code
        self.device = X.device
        self.index = X.device.index
        self.tensors = []  # (name, tensor's place among the operator's, bytes from first to last, written)

    def _place(self, name, slot, t, dtypes, out):
        if t.dtype not in dtypes:
            raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
        if t.device != self.device:
            raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, self.device))
        if t.numel():
            last = sum((d - 1) * s for d, s in zip(t.shape, t.stride()))
            self.tensors.append((name, slot, (last + 1) * t.element_size(), out))

    def rows(self, name, slot, t, shape, dtypes, out=False):
        """Leading dimension of a row-major matrix with unit column stride."""
        if t is None:
            return 0
        if t.dim() != 2 or tuple(t.shape) != shape:
            raise ValueError("%s is %s, the call needs %s" % (name, tuple(t.shape), shape))
        self._place(name, slot, t, dtypes, out)
        r, c = shape
        s0, s1 = t.stride()
        if (s1 != 1 and c > 1) or (s0 < c and r > 1):
            raise ValueError("%s must be row-major with unit column stride, got strides %s" % (name, (s0, s1)))
        return (s0 if r > 1 else c) or 1

    def weight(self, name, slot, t, shape, dtypes, out=False):
        """(leading dimension, order) of a K x N weight stored either way."""
        if t is None:
            return 0, ORDER_KN
        if t.dim() != 2 or tuple(t.shape) != shape:
            raise ValueError("%s is %s, the call needs %s" % (name, tuple(t.shape), shape))
        self._place(name, slot, t, dtypes, out)
        k, n = shape
        s0, s1 = t.stride()
        if (s1 == 1 or n <= 1) and (s0 >= n or k <= 1):
            return (s0 if k > 1 else n) or 1, ORDER_KN
        if (s0 == 1 or k <= 1) and (s1 >= k or n <= 1):
            return (s1 if n > 1 else k) or 1, ORDER_NK
        raise ValueError("%s must have unit stride along one axis and whole rows along the other, got strides %s"
                         % (name, (s0, s1)))

    def weights(self, names, slots, ts, shape, dtypes, out=False):
        """The same of two weights, which must agree."""
        if (ts[0] is None) != (ts[1] is None):
            raise ValueError("%s and %s must be given together" % names)
        a, b = (self.weight(n, i, t, shape, dtypes, out) for n, i, t in zip(names, slots, ts))
        if a != b:
            raise ValueError("%s and %s must have the same strides, got %s and %s"
                             % (names + tuple(tuple(t.stride()) for t in ts)))
        return a

    def vector(self, name, slot, t, n, dtypes, out=False):
        if t is None:
            return
        if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
            raise ValueError("%s must be a contiguous vector of %d, got %s" % (name, n, tuple(t.shape)))
        self._place(name, slot, t, dtypes, out)

    def done(self, function, need, args):
        """`args(pointers)` gives the C function's arguments before the workspace."""
        self.function, self.need, self.args = function, need, args
        self.pairs = [(i, bi, j, bj) for x, (_, i, bi, oi) in enumerate(self.tensors)
                      for _, j, bj, oj in self.tensors[x + 1:] if oi or oj]
        return self

    def _overlap(self, ts, i, j, same):
        """Raises unless the matrices at places i and j share no byte (their ranges do)."""
        x, y = ts[i], ts[j]
        if same == (i, j) and x.data_ptr() == y.data_ptr() and x.stride() == y.stride():
            return
        if x.dim() == 2 and y.dim() == 2:
            x, y = _stored_rows(x), _stored_rows(y)
            if not _regions_overlap(x, x.shape[0], x.shape[1], y, y.shape[0], y.shape[1]):
                return
        names = {slot: name for name, slot, _, _ in self.tensors}
        raise ValueError("%s and %s overlap: outputs must not share memory with inputs or each other"
                         % (names[i], names[j]))

    def run(self, ts, workspace, stream, same=None):
        """Launches on the tensors' GPU; `same`: places of an input and an output that may be one matrix."""
        p = [None if t is None else t.data_ptr() for t in ts]
        for i, bi, j, bj in self.pairs:
            if p[i] < p[j] + bj and p[j] < p[i] + bi:
                self._overlap(ts, i, j, same)
        if stream is not None and getattr(stream, "device", self.device) != self.device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, self.device))
        index = self.index
        if self.device.type != "cuda":
            raise ValueError("the tensors must be on a GPU, got %s" % self.device)
        need = self.need
        if need < 0:
            raise PgemmError(need)
        if index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return self.run(ts, workspace, stream, same)
        if workspace is not None:
            w, n = self._given(p, workspace)
        elif need == 0:
            w, n = None, 0
        elif stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            w, n = workspace.data_ptr(), need
        else:
            # from the pool of the stream that the kernels run on: freed with
            # this call, it can only be handed out again behind them
            with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else
                                   torch.cuda.ExternalStream(stream, device=self.device)):
                workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            w, n = workspace.data_ptr(), need
        r = self.function(*self.args(p), w, n, _raw_stream(index) if stream is None else _stream(stream))
        if r != 0:
            raise PgemmError(r)

    def _given(self, p, workspace):
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % self.device)
        w, n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        if n < self.need or w % 16:
            raise ValueError("workspace must be 16-byte aligned and hold %d bytes, got %d" % (self.need, n))
        for name, i, bytes_, _ in self.tensors:
            if n and p[i] < w + n and w < p[i] + bytes_:
                raise ValueError("workspace overlaps %s" % name)
        return w, n


_CALLS = {}


def _cached(describe, ts, act):
    """The checked call of these types, shapes, strides and devices."""
    try:
        key = (describe, act) + tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in ts])
        c = _CALLS.get(key)
    except TypeError:  # an activation that is no name
        raise ValueError("unknown activation %r: one of %s" % (act, ", ".join(ACT))) from None
    if c is None:
        c = describe(*ts, act)
        if len(_CALLS) >= 4096:
            _CALLS.clear()
        _CALLS[key] = c
    return c


def _stored_rows(t):
    return t if t.stride(0) >= t.stride(1) else t.t()


try:
    _FLOAT_CODE = {torch.float32: PGEMM_F32, torch.float16: PGEMM_F16, torch.bfloat16: PGEMM_BF16}
    _BY_CODE = {c: t for t, c in _FLOAT_CODE.items()}
    _OUT_TYPES = {c: (t,) if c == PGEMM_F32 else (t, torch.float32) for c, t in _BY_CODE.items()}
    _OWN_TYPE = {c: (t,) for c, t in _BY_CODE.items()}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
except NameError:  # without torch only the C entry points above are used
    pass


def _act_code(act):
    try:
        return ACT[act]
    except (KeyError, TypeError):
        raise ValueError("unknown activation %r: one of %s" % (act, ", ".join(ACT))) from None


def _required(**ts):
    for name, t in ts.items():
        if t is None:
            raise ValueError("%s is needed" % name)


def _sizes(X, W, name="W"):
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[0]:
        raise ValueError("X is %s and %s is %s: M x K and K x N are needed" % (tuple(X.shape), name, tuple(W.shape)))
    return X.shape[0], W.shape[1], X.shape[1]


def linear(X, W, Y, bias=None, residual=None, act="none", Z=None, workspace=None, stream=None):
    """Y = act(X @ W + bias) + residual on torch tensors.

    X is M x K, row-major with unit column stride; W is K x N in either storage
    order (a contiguous K x N tensor, or the transposed view of an N x K
    parameter), bias N.  float32, float16 or bfloat16, all of one type; Y (and
    residual) may be float32 instead.  Y and residual are M x N; residual may
    be Y itself.  Z, when given, receives the pre-activation X @ W + bias in
    X's type, which linear_backward reads.  act: "none", "relu", "silu",
    "gelu", "gelu_tanh".  Accumulation, bias, activation and residual are in
    fp32; Y and Z are each rounded once.

    The call runs on the tensors' GPU, on torch's current stream there unless
    `stream` is given, and does not synchronise.  A workspace of
    pgemm_linear_workspace bytes is taken from torch's allocator for the call
    unless one is passed.  Bad arguments raise ValueError before anything is
    launched; a status the library returns raises PgemmError.  Returns Y.
    """
    ts = (X, W, Y, bias, residual, Z)
    _cached(_describe_linear, ts, act).run(ts, workspace, stream, (2, 4))
    return Y


def _describe_linear(X, W, Y, bias, residual, Z, act):
    _required(X=X, W=W, Y=Y)
    M, N, K = _sizes(X, W)
    c = _Call(X)
    t, own = c.dtype, _OWN_TYPE[c.dtype]
    a = _act_code(act)
    ldx = c.rows("X", 0, X, (M, K), own)
    ldw, order = c.weight("W", 1, W, (K, N), own)
    ldy = c.rows("Y", 2, Y, (M, N), _OUT_TYPES[t], True)
    c.vector("bias", 3, bias, N, own)
    ldr = c.rows("residual", 4, residual, (M, N), (Y.dtype,))
    ldz = c.rows("Z", 5, Z, (M, N), own, True)
    out = _FLOAT_CODE[Y.dtype]
    return c.done(pgemm_linear, pgemm_linear_workspace(M, N, K, t), lambda p: (
        M, N, K, p[0], ldx, p[1], ldw, order, p[3], p[4], ldr, a, p[5], ldz, p[2], ldy, out, t))


def gated(X, Wg, Wu, H, bias_g=None, bias_u=None, act="silu", G=None, U=None, workspace=None, stream=None):
    """H = act(X @ Wg + bias_g) * (X @ Wu + bias_u) on torch tensors, in one product kernel.

    As linear, with two weights of the same strides.  G and U, when given,
    receive the two projections (with bias, before the activation) in X's type,
    which gated_backward reads.  Returns H.
    """
    ts = (X, Wg, Wu, H, bias_g, bias_u, G, U)
    _cached(_describe_gated, ts, act).run(ts, workspace, stream)
    return H


def _describe_gated(X, Wg, Wu, H, bias_g, bias_u, G, U, act):
    _required(X=X, Wg=Wg, Wu=Wu, H=H)
    M, N, K = _sizes(X, Wg, "Wg")
    c = _Call(X)
    t, own = c.dtype, _OWN_TYPE[c.dtype]
    a = _act_code(act)
    ldx = c.rows("X", 0, X, (M, K), own)
    ldw, order = c.weights(("Wg", "Wu"), (1, 2), (Wg, Wu), (K, N), own)
    ldh = c.rows("H", 3, H, (M, N), _OUT_TYPES[t], True)
    c.vector("bias_g", 4, bias_g, N, own)
    c.vector("bias_u", 5, bias_u, N, own)
    ldg = c.rows("G", 6, G, (M, N), own, True)
    ldu = c.rows("U", 7, U, (M, N), own, True)
    out = _FLOAT_CODE[H.dtype]
    return c.done(pgemm_gated, pgemm_gated_workspace(M, N, K, t), lambda p: (
        M, N, K, p[0], ldx, p[1], p[2], ldw, order, p[4], p[5], a, p[6], ldg, p[7], ldu, p[3], ldh, out, t))


def _grad_type(c, outs):
    """The one type of the weight and bias gradients: X's, or float32."""
    types = {t.dtype for t in outs if t is not None}
    if len(types) > 1:
        raise ValueError("weight and bias gradients must share one type, got %s" % sorted(str(t) for t in types))
    t = types.pop() if types else _BY_CODE[c.dtype]
    if t not in _OUT_TYPES[c.dtype]:
        raise ValueError("weight and bias gradients must be %s, got %s"
                         % (" or ".join(str(d) for d in _OUT_TYPES[c.dtype]), t))
    return t


def linear_backward(dY, X, W, Z=None, act="none", dX=None, dW=None, dbias=None, workspace=None, stream=None):
    """Gradients of linear for dY, the gradient at Y, into the tensors given.

    With dZ = dY * act'(Z): dX = dZ @ W.T (M x K, X's type), dW = X.T @ dZ
    (K x N in either storage order) and dbias = dZ summed over rows; dW and
    dbias have X's type or float32.  What is None is not computed.  Z is the
    pre-activation that linear wrote (not needed for act "none"); the
    residual's gradient is dY itself.  dZ is rounded to X's type before the two
    products (float16: scaled by rows and columns, so that it neither overflows nor
    vanishes there); dbias sums it unrounded.  Streams, workspace
    (pgemm_linear_backward_workspace) and errors as for linear.
    Returns (dX, dW, dbias).
    """
    ts = (dY, X, W, Z, dX, dW, dbias)
    _cached(_describe_linear_backward, ts, act).run(ts, workspace, stream)
    return dX, dW, dbias


def _describe_linear_backward(dY, X, W, Z, dX, dW, dbias, act):
    _required(dY=dY, X=X, W=W)
    M, N, K = _sizes(X, W)
    c = _Call(X)
    t, own = c.dtype, _OWN_TYPE[c.dtype]
    a = _act_code(act)
    if a != 0 and Z is None:
        raise ValueError("Z, the pre-activation, is needed for act %r" % act)
    gt = _grad_type(c, (dW, dbias))
    lddy = c.rows("dY", 0, dY, (M, N), own)
    ldx = c.rows("X", 1, X, (M, K), own)
    ldw, order = c.weight("W", 2, W, (K, N), own)
    ldz = c.rows("Z", 3, Z, (M, N), own)
    lddx = c.rows("dX", 4, dX, (M, K), own, True)
    lddw, dorder = c.weight("dW", 5, dW, (K, N), (gt,), True)
    c.vector("dbias", 6, dbias, N, (gt,), True)
    g = _FLOAT_CODE[gt]
    return c.done(pgemm_linear_backward, pgemm_linear_backward_workspace(M, N, K, a, t), lambda p: (
        M, N, K, p[0], lddy, p[1], ldx, p[2], ldw, order, p[3], ldz, a, p[4], lddx, p[5], lddw, dorder, p[6], g, t))


def gated_backward(dH, X, Wg, Wu, G, U, act="silu", dX=None, dWg=None, dWu=None, dbias_g=None, dbias_u=None,
                   workspace=None, stream=None):
    """Gradients of gated for dH, the gradient at H, into the tensors given.

    G and U are the projections that gated wrote.  With dG = dH * U * act'(G)
    and dU = dH * act(G): dX = dG @ Wg.T + dU @ Wu.T, dWg = X.T @ dG,
    dWu = X.T @ dU (both or neither, of the same strides), dbias_g and dbias_u
    the sums of dG and dU over rows.  Types, streams, workspace
    (pgemm_gated_backward_workspace) and errors as for linear_backward.
    Returns (dX, dWg, dWu, dbias_g, dbias_u).
    """
    ts = (dH, X, Wg, Wu, G, U, dX, dWg, dWu, dbias_g, dbias_u)
    _cached(_describe_gated_backward, ts, act).run(ts, workspace, stream)
    return dX, dWg, dWu, dbias_g, dbias_u


def _describe_gated_backward(dH, X, Wg, Wu, G, U, dX, dWg, dWu, dbias_g, dbias_u, act):
    _required(dH=dH, X=X, Wg=Wg, Wu=Wu, G=G, U=U)
    M, N, K = _sizes(X, Wg, "Wg")
    c = _Call(X)
    t, own = c.dtype, _OWN_TYPE[c.dtype]
    a = _act_code(act)
    gt = _grad_type(c, (dWg, dWu, dbias_g, dbias_u))
    lddh = c.rows("dH", 0, dH, (M, N), own)
    ldx = c.rows("X", 1, X, (M, K), own)
    ldw, order = c.weights(("Wg", "Wu"), (2, 3), (Wg, Wu), (K, N), own)
    ldg = c.rows("G", 4, G, (M, N), own)
    ldu = c.rows("U", 5, U, (M, N), own)
    lddx = c.rows("dX", 6, dX, (M, K), own, True)
    lddw, dorder = c.weights(("dWg", "dWu"), (7, 8), (dWg, dWu), (K, N), (gt,), True)
    c.vector("dbias_g", 9, dbias_g, N, (gt,), True)
    c.vector("dbias_u", 10, dbias_u, N, (gt,), True)
    g = _FLOAT_CODE[gt]
    return c.done(pgemm_gated_backward, pgemm_gated_backward_workspace(M, N, K, t), lambda p: (
        M, N, K, p[0], lddh, p[1], ldx, p[2], p[3], ldw, order, p[4], ldg, p[5], ldu, a, p[6], lddx, p[7], p[8],
        lddw, dorder, p[9], p[10], g, t))


def pgemm_hazard_copy_reduce(X, rows, cols, ldx, row_sums, reuse_wait, delay_wave=-1, delay_cycles=0, trace=None,
                             trace_len=0, trace_wg=0, stream=None):
    return _lib.pgemm_hazard_copy_reduce(_ptr(X), rows, cols, ldx, _ptr(row_sums), int(reuse_wait), int(delay_wave),
                                         int(delay_cycles), _ptr(trace), int(trace_len), int(trace_wg),
                                         _stream(stream))


def pgemm_diag_mfma_ceiling(dtype, zero_operands, iters, grid, seed, out, clock=None, stream=None, waves_per_simd=2,
                            block=16):
    """Returns (status, flops of the launch)."""
    fl = _i64(0)
    r = _lib.pgemm_diag_mfma_ceiling(DTYPE_CODE.get(dtype, dtype), int(zero_operands), int(waves_per_simd), int(block),
                                     int(iters), int(grid), int(seed) & 0xFFFFFFFF, _ptr(out), ctypes.byref(fl),
                                     _ptr(clock), _stream(stream))
    return r, fl.value


def pgemm_diag_lds_stream(M, N, K, A, lda, B, ldb, dtype, tile, stages, stream=None):
    """Returns (status, LDS bytes the launch fills)."""
    nb = _i64(0)
    r = _lib.pgemm_diag_lds_stream(M, N, K, _ptr(A), lda, _ptr(B), ldb, DTYPE_CODE.get(dtype, dtype),
                                   int(tile[0]), int(tile[1]), int(tile[2]), int(stages), ctypes.byref(nb),
                                   _stream(stream))
    return r, nb.value


def pgemm_diag_wait_profile(M, N, K, A, lda, B, ldb, C, ldc, dtype, tile, stages, out, out_len, stream=None):
    return _lib.pgemm_diag_wait_profile(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, DTYPE_CODE.get(dtype, dtype),
                                        int(tile[0]), int(tile[1]), int(tile[2]), int(stages), _ptr(out),
                                        int(out_len), _stream(stream))


def pgemm_diag_parts(M, N, K, A, lda, B, ldb, C, ldc, dtype, tile, stages, parts, clock, clock_len, stream=None):
    return _lib.pgemm_diag_parts(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, DTYPE_CODE.get(dtype, dtype),
                                 int(tile[0]), int(tile[1]), int(tile[2]), int(stages), int(parts), _ptr(clock),
                                 int(clock_len), _stream(stream))
