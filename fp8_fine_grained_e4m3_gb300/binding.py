"""ctypes binding over libfp8gemm.so (include/fp8gemm.h).

Argument marshalling only: every function here checks tensor metadata,
allocates outputs with torch when the caller gives none, and passes raw
device pointers plus the current CUDA stream to the C ABI.  All arithmetic
runs in the library's kernels.  There is no fallback: if the library is
missing or a call fails, an exception is raised.

FP8 operands are uint8 tensors holding e4m3 bytes (a torch.float8_e4m3fn
tensor is accepted and viewed as uint8); scales are float32; outputs are
bfloat16.
"""

import ctypes
import os
import threading

from . import build as _build

OK = 0
ERR_NULL = -1
ERR_ALIGN = -2
ERR_SHAPE = -3
ERR_ARCH = -4
ERR_LAUNCH = -5
ERR_DEVICE_STATUS = -6
ERR_TIMEOUT = -7
ERR_SCRATCH_LIMIT = -8
ERR_FORMAT = -9
ERR_FLAGS = -10
FMT = {"e4m3": 0, "e5m2": 1}  # FP8GEMM_FMT_*
FLAG_B_READ_ONLY = 1  # FP8GEMM_FLAG_B_READ_ONLY

_lib = None
_lock = threading.Lock()

# (name, restype, argtypes) for every entry point of include/fp8gemm.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
SIGNATURES = [
    ("fp8_quant_1x128", _I, [_P, _P, _P, _I, _I, _P]),
    ("fp8_quant_128x128", _I, [_P, _P, _P, _I, _I, _I, _P]),
    ("fp8gemm_dense", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("fp8_quant_1x128_fmt", _I, [_P, _P, _P, _I, _I, _I, _P]),
    ("fp8_quant_128x128_fmt", _I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    ("fp8_quant_1x128_ex", _I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    ("fp8_quant_128x128_ex", _I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    ("fp8gemm_dense_fmt", _I, [_P, _P, _I, _P, _P, _I, _P, _I, _I, _I, _P]),
    ("fp8gemm_dense_ex", _I, [_P, _P, _I, _P, _P, _I, _P, _I, _I, _I, ctypes.c_uint, _P]),
    ("fp8gemm_grouped_table", _I, [_P, _I, _I, _P]),
    ("fp8gemm_dense_batch", _I, [_P, _I, _P]),
    ("fp8gemm_grouped_contiguous_fmt", _I,
     [_P, _P, _I, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P]),
    ("fp8gemm_grouped_masked_fmt", _I, [_P, _P, _I, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P]),
    ("fp8gemm_dense_quant_a", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("fp8gemm_dense_quant_a_ex", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    ("fp8gemm_grouped_contiguous", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("fp8gemm_grouped_masked", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("fp8gemm_dense_small_m_noalloc", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("fp8_rmsnorm_quant", _I,
     [_P, _P, _I, _P, ctypes.c_float, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("fp8_rmsnorm_backward", _I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _P]),
    ("fp8_kv_append", _I,
     [_P, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, *[_I] * 9, _P]),
    ("fp8_kv_attention", _I,
     [_P, _L, _P, _P, _P, _P, _P, _P, _P, ctypes.c_float, _P, *[_I] * 10, _P]),
    ("fp8_moe_few", _I, [*[_P] * 10, *[_I] * 6, _P]),
    ("fp8gemm_get_device_status", _I, [_P, ctypes.POINTER(ctypes.c_int)]),
    ("fp8gemm_strerror", ctypes.c_char_p, [_I]),
    ("fp8gemm_num_kernel_launches", ctypes.c_uint64, []),
    ("fp8gemm_release_workspaces", _I, [_P]),
    ("fp8gemm_workspace_bytes", ctypes.c_uint64, []),
    ("fp8gemm_set_wait_limit_ns", _I, [ctypes.c_uint64]),
]


class FP8GemmError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


def library_path():
    return _build.LIB_PATH


def lib():
    """Load libfp8gemm.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                path = library_path()
                if not os.path.exists(path):
                    raise RuntimeError(
                        f"{path} is missing: build it first "
                        "(python -c 'import __graft_entry__ as g; g.build()')")
                L = ctypes.CDLL(path)
                for name, res, args in SIGNATURES:
                    f = getattr(L, name)
                    f.restype = res
                    f.argtypes = args
                _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().fp8gemm_strerror(int(code)).decode()


def num_kernel_launches() -> int:
    return int(lib().fp8gemm_num_kernel_launches())


def _check(code, where):
    if code != OK:
        raise FP8GemmError(code, where)


# ----------------------------------------------------------------- helpers
def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _u8(t, name):
    torch = _torch()
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must hold e4m3 bytes (uint8 or float8_e4m3fn), got {t.dtype}")
    return t


def _f32(t, name):
    if t.dtype != _torch().float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return t


def _i32(t, name):
    if t.dtype != _torch().int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    return t


def _bf16(t, name):
    if t.dtype != _torch().bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    return t


def _cdiv(a, b):
    return -(-a // b)


def _need(t, name, elems, last=None):
    """The library reads or writes exactly `elems` contiguous elements of t
    (a row length of `last` when given): refuse a tensor of another size
    before any pointer reaches a kernel, where it would be read or written
    out of bounds."""
    if t.numel() != elems or (last is not None and elems > 0 and t.shape[-1] != last):
        want = f"{elems} elements" + (f" in rows of {last}" if last is not None else "")
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs {want}")
    return t


def _shape_dense(A, sA, B, sB, D, M, N, K):
    """Operand sizes of the dense forms: A [M, K], sA [M, ceil(K/128)],
    B [N, K], sB [ceil(N/128), ceil(K/128)], D bf16 [M, N]."""
    Kb = _cdiv(K, 128)
    if B.dim() != 2 or B.shape[1] != K:
        raise ValueError(f"B has shape {tuple(B.shape)}; the call needs [N, {K}]")
    _need(sA, "sA", M * Kb, Kb)
    _need(sB, "sB", _cdiv(N, 128) * Kb, Kb)
    _need(_bf16(D, "D"), "D", M * N, N)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t, name="tensor"):
    return ctypes.c_void_p(_dev(t, name).data_ptr())


# ------------------------------------------------------------ entry points
def fp8_quant_1x128(X, Q=None, sX=None, stream=None):
    """X f32 [..., K] -> (Q u8 [..., K], sX f32 [..., ceil(K/128)]).  Leading dims
    are flattened into M."""
    torch = _torch()
    X = _f32(X, "X")
    K = X.shape[-1]
    M = X.numel() // K if K else 0
    if Q is None:
        Q = torch.empty(X.shape, dtype=torch.uint8, device=X.device)
    if sX is None:
        sX = torch.empty((*X.shape[:-1], _cdiv(K, 128)), dtype=torch.float32, device=X.device)
    _need(_u8(Q, "Q"), "Q", M * K, K)
    _need(_f32(sX, "sX"), "sX", M * _cdiv(K, 128), _cdiv(K, 128))
    _check(lib().fp8_quant_1x128(_ptr(X, "X"), _ptr(_u8(Q, "Q"), "Q"), _ptr(sX, "sX"), M, K,
                                 _stream(stream)), "fp8_quant_1x128")
    return Q, sX


def _weights3(W):
    W = _f32(W, "W")
    if W.dim() not in (2, 3):
        raise ValueError(f"W has shape {tuple(W.shape)}; the call needs [N, K] or [E, N, K]")
    return W, W.dim() == 2, (W.unsqueeze(0) if W.dim() == 2 else W)


def fp8_quant_128x128(W, Q=None, sW=None, stream=None):
    """W f32 [N, K] or [E, N, K] -> (Q u8 same shape, sW f32 [(E,) ceil(N/128), K/128])."""
    torch = _torch()
    W, squeeze, W3 = _weights3(W)
    E, N, K = W3.shape
    shp = (_cdiv(N, 128), _cdiv(K, 128))
    if Q is None:
        Q = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    if sW is None:
        sW = torch.empty(shp if squeeze else (E, *shp), dtype=torch.float32, device=W.device)
    _need(_u8(Q, "Q"), "Q", E * N * K, K)
    _need(_f32(sW, "sW"), "sW", E * shp[0] * shp[1], shp[1])
    _check(lib().fp8_quant_128x128(_ptr(W3, "W"), _ptr(_u8(Q, "Q"), "Q"), _ptr(sW, "sW"), E, N,
                                   K, _stream(stream)), "fp8_quant_128x128")
    return Q, sW


def _dense_mnk(A, B, name_a="A"):
    if A.dim() != 2:
        raise ValueError(f"{name_a} has shape {tuple(A.shape)}; the call needs [M, K]")
    M, K = A.shape
    if B.dim() != 2:
        raise ValueError(f"B has shape {tuple(B.shape)}; the call needs [N, {K}]")
    return M, B.shape[0], K


def fp8gemm_dense(A, sA, B, sB, D=None, stream=None):
    """A u8 [M, K], sA [M, K/128], B u8 [N, K], sB [ceil(N/128), K/128] -> D bf16 [M, N]."""
    torch = _torch()
    A, B = _u8(A, "A"), _u8(B, "B")
    M, N, K = _dense_mnk(A, B)
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
    _check(lib().fp8gemm_dense(_ptr(A, "A"), _ptr(sA, "sA"), _ptr(B, "B"), _ptr(sB, "sB"),
                               _ptr(D, "D"), M, N, K, _stream(stream)), "fp8gemm_dense")
    return D


def _fmt(name):
    if name not in FMT:
        raise ValueError(f"format must be one of {sorted(FMT)}, got {name!r}")
    return FMT[name]


def _u8_fmt(t, fmt, name):
    """FP8 bytes in format `fmt`: a uint8 tensor, or a torch float8 tensor
    whose own format agrees with `fmt` (viewed as uint8)."""
    torch = _torch()
    _fmt(fmt)
    own = {torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}.get(t.dtype)
    if own is not None:
        if own != fmt:
            raise TypeError(f"{name} is {t.dtype} but its format is given as {fmt!r}")
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must hold FP8 bytes (uint8 or a float8 dtype), got {t.dtype}")
    return t


def _counter(t):
    """Device address of a saturation counter: an int64 CUDA tensor (its
    first element is added to), or None."""
    torch = _torch()
    if t is None:
        return None
    if t.dtype != torch.int64 or t.numel() < 1:
        raise TypeError(f"sat_count must be an int64 tensor of at least one element, got {t.dtype}")
    return _ptr(t, "sat_count")


def fp8_quant_1x128_fmt(X, fmt, Q=None, sX=None, stream=None, sat_count=None):
    """fp8_quant_1x128 with the output format ("e4m3" or "e5m2").  sat_count
    (an int64 CUDA tensor) receives, added to its first element, the number of
    values the saturating encoding clamped (fp8_quant_1x128_ex)."""
    torch = _torch()
    X = _f32(X, "X")
    K = X.shape[-1]
    M = X.numel() // K if K else 0
    if Q is None:
        Q = torch.empty(X.shape, dtype=torch.uint8, device=X.device)
    if sX is None:
        sX = torch.empty((*X.shape[:-1], _cdiv(K, 128)), dtype=torch.float32, device=X.device)
    Q = _need(_u8_fmt(Q, fmt, "Q"), "Q", M * K, K)
    _need(_f32(sX, "sX"), "sX", M * _cdiv(K, 128), _cdiv(K, 128))
    if sat_count is not None:
        _check(lib().fp8_quant_1x128_ex(_ptr(X, "X"), _ptr(Q, "Q"), _ptr(sX, "sX"), M, K,
                                        _fmt(fmt), _counter(sat_count), _stream(stream)),
               "fp8_quant_1x128_ex")
        return Q, sX
    _check(lib().fp8_quant_1x128_fmt(_ptr(X, "X"), _ptr(Q, "Q"), _ptr(sX, "sX"), M, K, _fmt(fmt),
                                     _stream(stream)), "fp8_quant_1x128_fmt")
    return Q, sX


def fp8_quant_128x128_fmt(W, fmt, Q=None, sW=None, stream=None, sat_count=None):
    """fp8_quant_128x128 with the output format ("e4m3" or "e5m2"); sat_count
    as for fp8_quant_1x128_fmt (fp8_quant_128x128_ex)."""
    torch = _torch()
    W, squeeze, W3 = _weights3(W)
    E, N, K = W3.shape
    shp = (_cdiv(N, 128), _cdiv(K, 128))
    if Q is None:
        Q = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    if sW is None:
        sW = torch.empty(shp if squeeze else (E, *shp), dtype=torch.float32, device=W.device)
    Qb = _need(_u8_fmt(Q, fmt, "Q"), "Q", E * N * K, K)
    _need(_f32(sW, "sW"), "sW", E * shp[0] * shp[1], shp[1])
    if sat_count is not None:
        _check(lib().fp8_quant_128x128_ex(_ptr(W3, "W"), _ptr(Qb, "Q"), _ptr(sW, "sW"), E, N, K,
                                          _fmt(fmt), _counter(sat_count), _stream(stream)),
               "fp8_quant_128x128_ex")
        return Q, sW
    _check(lib().fp8_quant_128x128_fmt(_ptr(W3, "W"), _ptr(Qb, "Q"), _ptr(sW, "sW"), E, N, K,
                                       _fmt(fmt), _stream(stream)), "fp8_quant_128x128_fmt")
    return Q, sW


def fp8gemm_dense_fmt(A, sA, a_fmt, B, sB, b_fmt, D=None, stream=None):
    """fp8gemm_dense with operand formats ("e4m3" / "e5m2") for A and B."""
    torch = _torch()
    A, B = _u8_fmt(A, a_fmt, "A"), _u8_fmt(B, b_fmt, "B")
    M, N, K = _dense_mnk(A, B)
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
    _check(lib().fp8gemm_dense_fmt(_ptr(A, "A"), _ptr(sA, "sA"), _fmt(a_fmt), _ptr(B, "B"),
                                   _ptr(sB, "sB"), _fmt(b_fmt), _ptr(D, "D"), M, N, K,
                                   _stream(stream)), "fp8gemm_dense_fmt")
    return D


def fp8gemm_dense_ex(A, sA, a_fmt, B, sB, b_fmt, D=None, flags=0, stream=None):
    """fp8gemm_dense_fmt with flags, e.g. FLAG_B_READ_ONLY: B and sB are not
    written by any kernel still running when this one starts (constant
    weights), so the decode path may stage them before its dependency wait."""
    torch = _torch()
    A, B = _u8_fmt(A, a_fmt, "A"), _u8_fmt(B, b_fmt, "B")
    M, N, K = _dense_mnk(A, B)
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
    _check(lib().fp8gemm_dense_ex(_ptr(A, "A"), _ptr(sA, "sA"), _fmt(a_fmt), _ptr(B, "B"),
                                  _ptr(sB, "sB"), _fmt(b_fmt), _ptr(D, "D"), M, N, K,
                                  int(flags), _stream(stream)), "fp8gemm_dense_ex")
    return D


def fp8gemm_dense_quant_a(X, B, sB, D=None, Q=None, sA=None, stream=None, flags=0):
    """X f32 [M, K], B u8 [N, K], sB [ceil(N/128), K/128] -> D bf16 [M, N], with A
    quantised 1x128 on load.  Q u8 [M, K] and sA f32 [M, K/128] (both or neither)
    receive the quantised activations.  flags (e.g. FLAG_B_READ_ONLY) go to
    fp8gemm_dense_quant_a_ex."""
    torch = _torch()
    X, B = _f32(X, "X"), _u8(B, "B")
    M, N, K = _dense_mnk(X, B, "X")
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if (Q is None) != (sA is None):
        raise ValueError("Q and sA go together: give both or neither")
    Kb = _cdiv(K, 128)
    if B.shape[1] != K:
        raise ValueError(f"B has shape {tuple(B.shape)}; the call needs [N, {K}]")
    _need(_f32(sB, "sB"), "sB", _cdiv(N, 128) * Kb, Kb)
    _need(_bf16(D, "D"), "D", M * N, N)
    if Q is not None:
        _need(_u8(Q, "Q"), "Q", M * K, K)
        _need(_f32(sA, "sA"), "sA", M * Kb, Kb)
    qp = _ptr(_u8(Q, "Q"), "Q") if Q is not None else None
    sp = _ptr(sA, "sA") if sA is not None else None
    if flags:
        rc = lib().fp8gemm_dense_quant_a_ex(_ptr(X, "X"), qp, sp, _ptr(B, "B"), _ptr(sB, "sB"),
                                            _ptr(D, "D"), M, N, K, int(flags), _stream(stream))
    else:
        rc = lib().fp8gemm_dense_quant_a(_ptr(X, "X"), qp, sp, _ptr(B, "B"), _ptr(sB, "sB"),
                                         _ptr(D, "D"), M, N, K, _stream(stream))
    _check(rc, "fp8gemm_dense_quant_a_ex" if flags else "fp8gemm_dense_quant_a")
    return D


class Problem(ctypes.Structure):
    """One entry of the fp8gemm_grouped_table problem table (C layout)."""
    _fields_ = [("A", _P), ("sA", _P), ("B", _P), ("sB", _P), ("D", _P),
                ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("formats", ctypes.c_int)]


def problem_table(problems, out=None):
    """Device table for fp8gemm_grouped_table from (A, sA, B, sB, D) tensor
    tuples, optionally extended by the operand formats, (A, sA, B, sB, D,
    a_fmt, b_fmt) with "e4m3" / "e5m2": a uint8 CUDA tensor of
    len(problems) * sizeof(Problem) bytes (written into `out` when given, e.g.
    to update a table a graph captured).  Every entry's tensors are checked
    against its (M, N, K) here, since the kernel only sees the pointers."""
    torch = _torch()
    arr = (Problem * len(problems))()
    for e, prob in zip(arr, problems):
        A, sA, B, sB, D = prob[:5]
        a_fmt, b_fmt = (prob[5], prob[6]) if len(prob) > 5 else ("e4m3", "e4m3")
        A, B = _u8_fmt(A, a_fmt, "A"), _u8_fmt(B, b_fmt, "B")
        M, N, K = _dense_mnk(A, B)
        _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
        e.A, e.sA, e.B = _dev(A, "A").data_ptr(), _dev(sA, "sA").data_ptr(), _dev(B, "B").data_ptr()
        e.sB, e.D = _dev(sB, "sB").data_ptr(), _dev(D, "D").data_ptr()
        e.M, e.N, e.K = M, N, K
        e.formats = _fmt(a_fmt) | (_fmt(b_fmt) << 8)
    host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
    if out is None:
        return host.to("cuda")
    out.copy_(host)
    return out


MAX_DENSE_BATCH = 32  # FP8GEMM_MAX_DENSE_BATCH


def fp8gemm_dense_batch(problems, stream=None):
    """Independent dense problems in one launch: `problems` is a list of at
    most MAX_DENSE_BATCH tuples (A, sA, B, sB) or (A, sA, B, sB, D), optionally
    followed by (a_fmt, b_fmt); returns the list of D (bf16 [M, N], allocated
    where not given).  The entries are read on the host during the call."""
    torch = _torch()
    if len(problems) > MAX_DENSE_BATCH:
        raise ValueError(f"{len(problems)} problems; one call takes at most {MAX_DENSE_BATCH}")
    arr = (Problem * max(len(problems), 1))()
    outs = []
    for e, prob in zip(arr, problems):
        A, sA, B, sB = prob[:4]
        D = prob[4] if len(prob) in (5, 7) else None
        fmts = prob[-2:] if len(prob) in (6, 7) else ("e4m3", "e4m3")
        A, B = _u8_fmt(A, fmts[0], "A"), _u8_fmt(B, fmts[1], "B")
        M, N, K = _dense_mnk(A, B)
        if D is None:
            D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
        _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
        e.A, e.sA, e.B = _ptr(A, "A").value, _ptr(sA, "sA").value, _ptr(B, "B").value
        e.sB, e.D = _ptr(sB, "sB").value, _ptr(D, "D").value
        e.M, e.N, e.K = M, N, K
        e.formats = _fmt(fmts[0]) | (_fmt(fmts[1]) << 8)
        outs.append(D)
    _check(lib().fp8gemm_dense_batch(ctypes.cast(arr, _P), len(problems), _stream(stream)),
           "fp8gemm_dense_batch")
    return outs


def fp8gemm_grouped_table(table, num_problems, max_M, stream=None):
    """Run every problem of a device table (see problem_table); max_M bounds
    every entry's M and picks the kernel's padded width (16, 32 or 64 rows;
    larger entries are taken 64 rows at a time)."""
    if table.numel() < int(num_problems) * ctypes.sizeof(Problem):
        raise ValueError(f"table holds {table.numel()} bytes; {num_problems} entries need "
                         f"{int(num_problems) * ctypes.sizeof(Problem)}")
    _check(lib().fp8gemm_grouped_table(_ptr(table, "table"), int(num_problems), int(max_M),
                                       _stream(stream)), "fp8gemm_grouped_table")


def _shape_grouped(A, sA, B, sB, info, D, rows, N, K, E, info_len, a_name="A"):
    """Operand sizes of the grouped forms: A holds `rows` rows of K bytes,
    sA [rows, ceil(K/128)], B [E, N, K], sB [E, ceil(N/128), ceil(K/128)],
    the index array `info_len` int32 entries, D bf16 [rows, N]."""
    Kb = _cdiv(K, 128)
    _need(A, a_name, rows * K, K)
    _need(sA, "sA", rows * Kb, Kb)
    if B.dim() != 3 or B.shape[0] != E or B.shape[2] != K:
        raise ValueError(f"B has shape {tuple(B.shape)}; the call needs [{E}, N, {K}]")
    _need(sB, "sB", E * _cdiv(N, 128) * Kb, Kb)
    _need(info, "the index array", info_len)
    _need(_bf16(D, "D"), "D", rows * N, N)


def _contiguous(A, sA, B, sB, m_indices, D, a_fmt, b_fmt, stream, fmt_call):
    torch = _torch()
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError(f"A {tuple(A.shape)} / B {tuple(B.shape)}: the call needs A [M_pad, K]"
                         " and B [E, N, K]")
    M_pad, K = A.shape
    E, N = B.shape[0], B.shape[1]
    if D is None:
        D = torch.empty((M_pad, N), dtype=torch.bfloat16, device=A.device)
    _shape_grouped(A, _f32(sA, "sA"), B, _f32(sB, "sB"), _i32(m_indices, "m_indices"), D,
                   M_pad, N, K, E, M_pad)
    if fmt_call:
        rc = lib().fp8gemm_grouped_contiguous_fmt(
            _ptr(A, "A"), _ptr(sA, "sA"), _fmt(a_fmt), _ptr(B, "B"), _ptr(sB, "sB"),
            _fmt(b_fmt), _ptr(m_indices, "m_indices"), _ptr(D, "D"), M_pad, N, K, E,
            _stream(stream))
    else:
        rc = lib().fp8gemm_grouped_contiguous(
            _ptr(A, "A"), _ptr(sA, "sA"), _ptr(B, "B"), _ptr(sB, "sB"),
            _ptr(m_indices, "m_indices"), _ptr(D, "D"), M_pad, N, K, E, _stream(stream))
    _check(rc, "fp8gemm_grouped_contiguous" + ("_fmt" if fmt_call else ""))
    return D


def _masked(A, sA, B, sB, masked_m, D, a_fmt, b_fmt, stream, fmt_call):
    torch = _torch()
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError(f"A {tuple(A.shape)} / B {tuple(B.shape)}: the call needs A "
                         "[E, M_max, K] and B [E, N, K]")
    E, M_max, K = A.shape
    N = B.shape[1]
    if D is None:
        D = torch.empty((E, M_max, N), dtype=torch.bfloat16, device=A.device)
    _shape_grouped(A, _f32(sA, "sA"), B, _f32(sB, "sB"), _i32(masked_m, "masked_m"), D,
                   E * M_max, N, K, E, E)
    if fmt_call:
        rc = lib().fp8gemm_grouped_masked_fmt(
            _ptr(A, "A"), _ptr(sA, "sA"), _fmt(a_fmt), _ptr(B, "B"), _ptr(sB, "sB"),
            _fmt(b_fmt), _ptr(masked_m, "masked_m"), _ptr(D, "D"), E, M_max, N, K,
            _stream(stream))
    else:
        rc = lib().fp8gemm_grouped_masked(
            _ptr(A, "A"), _ptr(sA, "sA"), _ptr(B, "B"), _ptr(sB, "sB"),
            _ptr(masked_m, "masked_m"), _ptr(D, "D"), E, M_max, N, K, _stream(stream))
    _check(rc, "fp8gemm_grouped_masked" + ("_fmt" if fmt_call else ""))
    return D


def fp8gemm_grouped_contiguous(A, sA, B, sB, m_indices, D=None, stream=None):
    """A u8 [M_pad, K], B u8 [E, N, K], m_indices i32 [M_pad] -> D bf16 [M_pad, N]."""
    return _contiguous(_u8(A, "A"), sA, _u8(B, "B"), sB, m_indices, D, "e4m3", "e4m3", stream,
                       False)


def fp8gemm_grouped_masked(A, sA, B, sB, masked_m, D=None, stream=None):
    """A u8 [E, M_max, K], B u8 [E, N, K], masked_m i32 [E] -> D bf16 [E, M_max, N]
    (rows >= masked_m[e] are not written)."""
    return _masked(_u8(A, "A"), sA, _u8(B, "B"), sB, masked_m, D, "e4m3", "e4m3", stream, False)


def fp8gemm_grouped_contiguous_fmt(A, sA, a_fmt, B, sB, b_fmt, m_indices, D=None, stream=None):
    """fp8gemm_grouped_contiguous with operand formats ("e4m3" / "e5m2")."""
    return _contiguous(_u8_fmt(A, a_fmt, "A"), sA, _u8_fmt(B, b_fmt, "B"), sB, m_indices, D,
                       a_fmt, b_fmt, stream, True)


def fp8gemm_grouped_masked_fmt(A, sA, a_fmt, B, sB, b_fmt, masked_m, D=None, stream=None):
    """fp8gemm_grouped_masked with operand formats ("e4m3" / "e5m2")."""
    return _masked(_u8_fmt(A, a_fmt, "A"), sA, _u8_fmt(B, b_fmt, "B"), sB, masked_m, D,
                   a_fmt, b_fmt, stream, True)


def fp8gemm_dense_small_m_noalloc(A, sA, B, sB, D, stream=None):
    """fp8gemm_dense for M <= 64 without any device allocation by the library:
    the caller provides D, and the split-K scratch is a fixed array inside the
    library (shared by every call on the device; calls must not overlap on the
    GPU)."""
    A, B = _u8(A, "A"), _u8(B, "B")
    M, N, K = _dense_mnk(A, B)
    _shape_dense(A, _f32(sA, "sA"), B, _f32(sB, "sB"), D, M, N, K)
    _check(lib().fp8gemm_dense_small_m_noalloc(
        _ptr(A, "A"), _ptr(sA, "sA"), _ptr(B, "B"), _ptr(sB, "sB"), _ptr(D, "D"),
        M, N, K, _stream(stream)), "fp8gemm_dense_small_m_noalloc")
    return D


# The decoder-layer calls below are short enough on the GPU for the host to be
# what a caller waits for, so their checks take few attribute reads per tensor.
_fast = None


class _Fast:
    """What those calls look up once: torch's types and the handle of the
    current stream as a number."""

    def __init__(self):
        torch = _torch()
        self.empty, self.empty_like = torch.empty, torch.empty_like
        self.u8, self.f32, self.i32, self.bf16 = (torch.uint8, torch.float32, torch.int32,
                                                  torch.bfloat16)
        self.f8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
        self.kind = {torch.bfloat16: 0, torch.float32: 1}  # FP8GEMM_TYPE_*
        self.current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if self.current is None:
            self.current = lambda device: torch.cuda.current_stream(device).cuda_stream
        self.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        L = lib()
        self.rmsnorm_quant, self.rmsnorm_backward = L.fp8_rmsnorm_quant, L.fp8_rmsnorm_backward
        self.kv_append, self.kv_attention = L.fp8_kv_append, L.fp8_kv_attention
        self.moe_few = L.fp8_moe_few


def _lookup():
    global _fast
    if _fast is None:
        _fast = _Fast()
    return _fast


def _size(t, name, want, elems, last=None):
    """Refuses a tensor of another type or size: the slow end of the checks
    below (`last`: the length of a row)."""
    if t.dtype != want:
        raise TypeError(f"{name} must be {want}, got {t.dtype}")
    _need(t, name, elems, last)


def _codes(f, t, name, fmt):
    """FP8 bytes in format `fmt`: uint8, or the float8 type of that format."""
    if t.dtype is not f.u8 and t.dtype is not f.f8[fmt]:
        _u8_fmt(t, fmt, name)


def _on(f, t, name):
    """The device of a call: its first tensor's, which has to be the current one,
    where the library launches."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device != f.device():
        raise ValueError(f"{name} is on cuda:{device}; the current device is cuda:{f.device()}")
    return device


def _at(t, name, device):
    """Address of a tensor on that device."""
    if t.get_device() != device:
        raise ValueError(f"{name} is not on cuda:{device}, the device of the call")
    return t.data_ptr()


def _here(t, name, device):
    """Address of a contiguous tensor on that device."""
    if t.get_device() != device or not t.is_contiguous():
        _dev(t, name)
        raise ValueError(f"{name} is on cuda:{t.get_device()}; the call is on cuda:{device}")
    return t.data_ptr()


def fp8_rmsnorm_quant(X, gain, eps=1e-6, residual=None, fmt="e4m3", H=None, Q=None, sQ=None,
                      rstd=None, stream=None):
    """Residual addition, RMS norm and 1x128 FP8 output in one pass: X bf16 or
    f32 [..., K], gain f32 [K] -> (Q u8 [..., K], sQ f32 [..., ceil(K/128)], H,
    rstd f32 [...]).  H is X + residual in X's type (X itself without one);
    H=residual updates the stream in place."""
    f = _fast or _lookup()
    dtype, shape = X.dtype, X.shape
    kind = f.kind.get(dtype)
    if kind is None:
        raise TypeError(f"X must be bfloat16 or float32, got {dtype}")
    code = _fmt(fmt)
    K, n = shape[-1], X.numel()
    M = n // K if K else 0
    Kb = -(-K // 128)
    if gain.dtype is not f.f32 or gain.numel() != K:
        _size(gain, "gain", f.f32, K)
    r = h = None
    if residual is not None:
        if residual.dtype is not dtype or residual.shape != shape:
            _size(residual, "residual", dtype, n, K)
        if H is None:
            H = f.empty_like(X)
        elif H is not residual and (H.dtype is not dtype or H.shape != shape):
            _size(H, "H", dtype, n, K)
    elif H is not None:
        raise ValueError("H is the sum with the residual: give residual too")
    if Q is None:
        Q = f.empty(shape, dtype=f.u8, device=X.device)
    else:
        _codes(f, Q, "Q", fmt)
        if Q.shape != shape:
            _need(Q, "Q", n, K)
    if sQ is None:
        sQ = f.empty((*shape[:-1], Kb), dtype=f.f32, device=X.device)
    elif sQ.dtype is not f.f32 or sQ.numel() != M * Kb or (M and sQ.size(-1) != Kb):
        _size(sQ, "sQ", f.f32, M * Kb, Kb)
    if rstd is None:
        rstd = f.empty(shape[:-1], dtype=f.f32, device=X.device)
    elif rstd.dtype is not f.f32 or rstd.numel() != M:
        _size(rstd, "rstd", f.f32, M)
    device = _on(f, X, "X")
    if residual is not None:
        r, h = _here(residual, "residual", device), _here(H, "H", device)
    rc = f.rmsnorm_quant(_here(X, "X", device), r, kind, _here(gain, "gain", device), eps, h,
                         _here(Q, "Q", device), _here(sQ, "sQ", device),
                         _here(rstd, "rstd", device), M, K, code,
                         f.current(device) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "fp8_rmsnorm_quant")
    return Q, sQ, (X if residual is None else H), rstd


def fp8_rmsnorm_backward(dY, H, rstd, gain, dH=None, dX=None, dgain=None, stream=None):
    """Gradients of fp8_rmsnorm_quant's norm (straight through the quantiser):
    dY and H bf16 or f32 [..., K], rstd f32 [...], gain f32 [K], dH (the
    gradient that reaches H past the norm) as dY or None -> (dX, dgain f32 [K])."""
    f = _fast or _lookup()
    dtype, shape = H.dtype, H.shape
    kind = f.kind.get(dtype)
    if kind is None:
        raise TypeError(f"H must be bfloat16 or float32, got {dtype}")
    K, n = shape[-1], H.numel()
    M = n // K if K else 0
    if dY.dtype is not dtype or dY.shape != shape:
        _size(dY, "dY", dtype, n, K)
    if dH is not None and (dH.dtype is not dtype or dH.shape != shape):
        _size(dH, "dH", dtype, n, K)
    if dX is None:
        dX = f.empty_like(H)
    elif dX.dtype is not dtype or dX.shape != shape:
        _size(dX, "dX", dtype, n, K)
    if dgain is None:
        dgain = f.empty(K, dtype=f.f32, device=H.device)
    elif dgain.dtype is not f.f32 or dgain.numel() != K:
        _size(dgain, "dgain", f.f32, K)
    if rstd.dtype is not f.f32 or rstd.numel() != M:
        _size(rstd, "rstd", f.f32, M)
    if gain.dtype is not f.f32 or gain.numel() != K:
        _size(gain, "gain", f.f32, K)
    device = _on(f, H, "H")
    rc = f.rmsnorm_backward(_here(dY, "dY", device), _here(H, "H", device), kind,
                            _here(rstd, "rstd", device), _here(gain, "gain", device),
                            None if dH is None else _here(dH, "dH", device),
                            _here(dX, "dX", device), _here(dgain, "dgain", device), M, K,
                            f.current(device) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "fp8_rmsnorm_backward")
    return dX, dgain


def _tokens(f, t, name, T, heads, dim):
    """bf16 [T, heads, dim] whose tokens may lie apart (parts of the rows of a
    fused projection's output): returns the token stride in elements."""
    if t.dtype is not f.bf16:
        _bf16(t, name)
    if t.shape != (T, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs [{T}, {heads}, {dim}]")
    ld, sh, sd = t.stride()
    if sd != 1 or (sh != dim and heads > 1):
        raise ValueError(f"{name} must hold each token's heads contiguously")
    return ld if T > 1 else heads * dim


def _cache(f, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu, T, fmt):
    """Checks a paged cache and its index arrays: blocks, heads, block, dim, B,
    table width."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache {tuple(shape)} / v_cache {tuple(v_cache.shape)}: the"
                         " call needs [num_blocks, heads, block, dim] twice")
    n, heads, block, dim = shape
    if block_table.dtype is not f.i32:
        _i32(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}; the call needs"
                         " [B, table_width]")
    B, width = block_table.shape
    _codes(f, k_cache, "k_cache", fmt)
    _codes(f, v_cache, "v_cache", fmt)
    nh = n * heads
    if k_scale.dtype is not f.f32 or k_scale.numel() != nh:
        _size(k_scale, "k_scale", f.f32, nh)
    if v_scale.dtype is not f.f32 or v_scale.numel() != nh:
        _size(v_scale, "v_scale", f.f32, nh)
    if seq_lens.dtype is not f.i32 or seq_lens.numel() != B:
        _size(seq_lens, "seq_lens", f.i32, B)
    if cu is None:
        if B > 0 and T % B != 0:
            raise ValueError(f"{T} tokens for {B} sequences: give the offsets")
    elif cu.dtype is not f.i32 or cu.numel() != B + 1:
        _size(cu, "the offsets", f.i32, B + 1)
    return n, heads, block, dim, B, width


def fp8_kv_append(K, V, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu_new=None,
                  max_new=None, fmt="e4m3", stream=None):
    """Write new keys and values (bf16 [T, heads, dim], tokens may lie apart)
    into the paged FP8 cache (codes u8 [num_blocks, heads, block, dim], scales
    f32 [num_blocks, heads]), at the end of each sequence: seq_lens i32 [B]
    counts them already.  cu_new i32 [B + 1] are the offsets of each sequence's
    tokens (None: T / B each); max_new bounds a sequence's (None: T)."""
    f = _fast or _lookup()
    code = _fmt(fmt)
    T = K.size(0)
    n, heads, block, dim, B, width = _cache(f, k_cache, k_scale, v_cache, v_scale, block_table,
                                            seq_lens, cu_new, T, fmt)
    ld_k, ld_v = _tokens(f, K, "K", T, heads, dim), _tokens(f, V, "V", T, heads, dim)
    if max_new is None:
        max_new = T if cu_new is not None else -(-T // max(B, 1))
    device = _on(f, K, "K")
    rc = f.kv_append(K.data_ptr(), _at(V, "V", device), ld_k, ld_v,
                     _here(k_cache, "k_cache", device), _here(k_scale, "k_scale", device),
                     _here(v_cache, "v_cache", device), _here(v_scale, "v_scale", device),
                     _here(block_table, "block_table", device),
                     _here(seq_lens, "seq_lens", device),
                     None if cu_new is None else _here(cu_new, "cu_new", device), T, B, heads,
                     dim, block,
                     width, n, max_new, code,
                     f.current(device) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "fp8_kv_append")


def fp8_kv_attention(Q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu_q=None,
                     max_q=None, scale=None, fmt="e4m3", O=None, stream=None):
    """Attention of the newest tokens (Q bf16 [T, heads * group, dim], tokens
    may lie apart) over the paged FP8 cache that holds their keys and values
    already -> O bf16 [T, heads * group, dim].  cu_q and max_q as
    fp8_kv_append's; scale defaults to dim ** -0.5."""
    f = _fast or _lookup()
    code = _fmt(fmt)
    T = Q.size(0)
    n, heads, block, dim, B, width = _cache(f, k_cache, k_scale, v_cache, v_scale, block_table,
                                            seq_lens, cu_q, T, fmt)
    if Q.dim() != 3 or heads == 0 or Q.size(1) % heads != 0:
        raise ValueError(f"Q has shape {tuple(Q.shape)}; the call needs [T, heads * group, dim]"
                         f" with {heads} cached heads")
    hq = Q.size(1)
    ld_q = _tokens(f, Q, "Q", T, hq, dim)
    if O is None:
        O = f.empty(Q.shape, dtype=f.bf16, device=Q.device)
    elif O.dtype is not f.bf16 or O.shape != Q.shape:
        _size(O, "O", f.bf16, T * hq * dim, dim)
    if max_q is None:
        max_q = T if cu_q is not None else -(-T // max(B, 1))
    if scale is None:
        scale = dim ** -0.5
    device = _on(f, Q, "Q")
    rc = f.kv_attention(Q.data_ptr(), ld_q, _here(k_cache, "k_cache", device),
                        _here(k_scale, "k_scale", device), _here(v_cache, "v_cache", device),
                        _here(v_scale, "v_scale", device),
                        _here(block_table, "block_table", device),
                        _here(seq_lens, "seq_lens", device),
                        None if cu_q is None else _here(cu_q, "cu_q", device), scale,
                        _here(O, "O", device), T, B,
                        heads, hq // heads, dim, block, width, n, max_q, code,
                        f.current(device) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "fp8_kv_attention")
    return O


def fp8_moe_few(A, sA, logits, W1, s1, W2, s2, top_k, renormalise=True, D=None, ids=None,
                weights=None, stream=None):
    """A mixture-of-experts layer for at most 64 tokens: A u8 [T, H], sA f32
    [T, ceil(H/128)], logits f32 [T, E], W1 u8 [E, 2 I, H] (gate rows, then up
    rows), W2 u8 [E, H, I] with their 128x128 scales -> (D bf16 [T, H], ids i32
    [T, top_k], weights f32 [T, top_k])."""
    f = _fast or _lookup()
    f32 = f.f32
    a, w1, w2 = A.shape, W1.shape, W2.shape
    if len(a) != 2 or len(w1) != 3:
        raise ValueError(f"A {tuple(a)} / W1 {tuple(w1)}: the call needs [T, H] and [E, 2 I, H]")
    T, H = a
    E, I2, Hw = w1
    I = I2 // 2
    if I2 != 2 * I or Hw != H or w2 != (E, H, I):
        raise ValueError(f"W1 {tuple(w1)} / W2 {tuple(w2)}: the call needs [E, 2 I, {H}] and"
                         f" [E, {H}, I]")
    _codes(f, A, "A", "e4m3")
    _codes(f, W1, "W1", "e4m3")
    _codes(f, W2, "W2", "e4m3")
    Hb, Ib, k = -(-H // 128), -(-I // 128), int(top_k)
    if sA.dtype is not f32 or sA.shape != (T, Hb):
        _size(sA, "sA", f32, T * Hb, Hb)
    if logits.dtype is not f32 or logits.shape != (T, E):
        _size(logits, "logits", f32, T * E, E)
    if s1.dtype is not f32 or s1.shape != (E, -(-I2 // 128), Hb):
        _size(s1, "s1", f32, E * -(-I2 // 128) * Hb, Hb)
    if s2.dtype is not f32 or s2.shape != (E, Hb, Ib):
        _size(s2, "s2", f32, E * Hb * Ib, Ib)
    if D is None:
        D = f.empty((T, H), dtype=f.bf16, device=A.device)
    elif D.dtype is not f.bf16 or D.shape != a:
        _size(D, "D", f.bf16, T * H, H)
    if ids is None:
        ids = f.empty((T, k), dtype=f.i32, device=A.device)
    elif ids.dtype is not f.i32 or ids.shape != (T, k):
        _size(ids, "ids", f.i32, T * k, k)
    if weights is None:
        weights = f.empty((T, k), dtype=f32, device=A.device)
    elif weights.dtype is not f32 or weights.shape != (T, k):
        _size(weights, "weights", f32, T * k, k)
    device = _on(f, A, "A")
    rc = f.moe_few(_here(A, "A", device), _here(sA, "sA", device),
                   _here(logits, "logits", device), _here(W1, "W1", device),
                   _here(s1, "s1", device), _here(W2, "W2", device), _here(s2, "s2", device),
                   _here(D, "D", device), _here(ids, "ids", device),
                   _here(weights, "weights", device), T, H, I, E, k, 1 if renormalise else 0,
                   f.current(device) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "fp8_moe_few")
    return D, ids, weights


def fp8gemm_get_device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word."""
    out = ctypes.c_int(0)
    _check(lib().fp8gemm_get_device_status(_stream(stream), ctypes.byref(out)),
           "fp8gemm_get_device_status")
    return out.value


def fp8gemm_release_workspaces(stream=None):
    """Free the library's workspaces of `stream` (current stream by default)
    on the current device, after synchronising it."""
    _check(lib().fp8gemm_release_workspaces(_stream(stream)), "fp8gemm_release_workspaces")


def workspace_bytes() -> int:
    """Bytes of library-owned workspaces currently held (all devices, streams)."""
    return int(lib().fp8gemm_workspace_bytes())


def set_wait_limit_ns(ns: int):
    """Time limit of every pipeline wait in kernels launched from now on
    (process-wide); 0 restores the default (2 s)."""
    _check(lib().fp8gemm_set_wait_limit_ns(int(ns)), "fp8gemm_set_wait_limit_ns")
