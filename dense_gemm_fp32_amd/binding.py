"""ctypes binding of libgemm.so: the C entry points of include/gemm.h under
the same names, plus a torch-tensor convenience wrapper.

Only argument marshalling happens here; every step of the GEMM runs in the
HIP kernels of libgemm.so.  There is no fallback: if the library is missing
the import fails with an error that says how to build it.
"""
import ctypes
import functools
import os

import torch  # noqa: F401  (loads torch's HIP runtime first, so libgemm.so binds to the same one)

HERE = os.path.dirname(os.path.abspath(__file__))
# DENSE_GEMM_FP32_AMD_LIB selects another build of the same library (the
# LDS-poison debug build of build.py); by default the release build next to
# this file.
LIB_PATH = os.environ.get("DENSE_GEMM_FP32_AMD_LIB") or os.path.join(HERE, "libgemm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libgemm.so is not built (%s); run `python -m dense_gemm_fp32_amd.build`"
                      % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

_I = ctypes.c_int
_F = ctypes.c_float
_P = ctypes.c_void_p

_lib.gemm_f32.argtypes = [_I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, _P]
_lib.gemm_f32.restype = _I
_lib.gemm_f16.argtypes = [_I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, _P]
_lib.gemm_f16.restype = _I
_lib.gemm_f16f32.argtypes = [_I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, _P]
_lib.gemm_f16f32.restype = _I
LAYOUT_NAMES = tuple("gemm_%s_%s" % (t, l) for t in ("f32", "f16", "f16f32") for l in ("nt", "tn", "tt"))
for _n in ("gemm_f32_colmajor", "gemm_f16_colmajor", "gemm_f16f32_colmajor",
           "gemm_f32_valu", "gemm_f32_noalloc") + LAYOUT_NAMES:
    getattr(_lib, _n).argtypes = [_I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, _P]
    getattr(_lib, _n).restype = _I
_lib.gemm_status_string.argtypes = [_I]
_lib.gemm_status_string.restype = ctypes.c_char_p
_lib.gemm_describe.argtypes = [_I, _I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, ctypes.c_char_p, _I]
_lib.gemm_describe.restype = _I
_lib.gemm_set_load_mode.argtypes = [_I]
_lib.gemm_set_load_mode.restype = _I
_lib.gemm_set_tile_config.argtypes = [_I]
_lib.gemm_set_tile_config.restype = _I
_lib.gemm_set_split.argtypes = [_I]
_lib.gemm_set_split.restype = _I
_lib.gemm_set_tail_split.argtypes = [_I]
_lib.gemm_set_tail_split.restype = _I
_lib.gemm_set_pack.argtypes = [_I]
_lib.gemm_set_pack.restype = _I
_lib.gemm_set_stream_k.argtypes = [_I]
_lib.gemm_set_stream_k.restype = _I
_lib.gemm_set_workspace_limit.argtypes = [ctypes.c_longlong]
_lib.gemm_set_workspace_limit.restype = ctypes.c_longlong
_lib.gemm_probe_mfma.argtypes = [_I, _I, _P, ctypes.c_size_t, _P, ctypes.c_size_t,
                                 ctypes.POINTER(ctypes.c_double), _P]
_lib.gemm_probe_mfma.restype = _I

_L = ctypes.c_longlong
_Z = ctypes.c_size_t
_LORA = [_I, _I, _I, _F, _P, _I, _P, _I, _F, _P, _I, _I, _I, _P, _I, _L, _P, _I, _L, _P, _P, _P,
         _P, _Z, _P]
_LORA_GRAD = [_I, _I, _I, _F, _P, _I, _P, _I, _P, _I, _I, _I, _P, _I, _L, _P, _I, _L, _P, _P, _P,
              _F, _P, _I, _F, _P, _I, _L, _P, _I, _L, _P, _Z, _P]
_MOE = [_I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _I, _P, _I, _L, _P, _I, _L, _F, _P, _I, _P, _P,
        _P, _Z, _P]
ROW_NAMES = ("gemm_lora_f16", "gemm_lora_f32", "gemm_lora_grad_f16", "gemm_lora_grad_f32",
             "gemm_moe_f16", "gemm_moe_f32", "gemm_lora_workspace", "gemm_lora_grad_workspace",
             "gemm_moe_workspace")
for _n, _args in (("gemm_lora", _LORA), ("gemm_lora_grad", _LORA_GRAD), ("gemm_moe", _MOE)):
    for _t in ("f16", "f32"):
        getattr(_lib, "%s_%s" % (_n, _t)).argtypes = _args
        getattr(_lib, "%s_%s" % (_n, _t)).restype = _I
    getattr(_lib, _n + "_workspace").argtypes = [_I] * 6
    getattr(_lib, _n + "_workspace").restype = _Z

_QUANT = [_I, _I, _P, _I, _P, _I, _P, _P]
_I8 = [_I, _I, _I, _F, _P, _I, _P, _P, _I, _P, _F, _P, _I, _P, _Z, _P]
_GLU = [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _Z, _P]
_GLU_I8 = [_I, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _I, _P, _Z, _P]
_GLU_GRAD = [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _F, _P, _I, _F, _P, _I, _P, _Z, _P]
BLOCK_NAMES = ("gemm_quant_i8_f16", "gemm_quant_i8_f32", "gemm_i8_f16", "gemm_i8_f32",
               "gemm_i8_workspace", "gemm_glu_f16", "gemm_glu_f32", "gemm_glu_i8_f16",
               "gemm_glu_i8_f32", "gemm_glu_workspace", "gemm_glu_grad_f16",
               "gemm_glu_grad_f16f32", "gemm_glu_grad_f32", "gemm_glu_grad_workspace")
for _n, _args in (("gemm_quant_i8", _QUANT), ("gemm_i8", _I8), ("gemm_glu", _GLU),
                  ("gemm_glu_i8", _GLU_I8), ("gemm_glu_grad", _GLU_GRAD)):
    for _t in ("f16", "f32"):
        getattr(_lib, "%s_%s" % (_n, _t)).argtypes = _args
        getattr(_lib, "%s_%s" % (_n, _t)).restype = _I
_lib.gemm_glu_grad_f16f32.argtypes = _GLU_GRAD
_lib.gemm_glu_grad_f16f32.restype = _I
for _n, _args in (("gemm_i8_workspace", 4), ("gemm_glu_workspace", 5),
                  ("gemm_glu_grad_workspace", 5)):
    getattr(_lib, _n).argtypes = [_I] * _args
    getattr(_lib, _n).restype = _Z

EXPORTS = ("gemm_f32", "gemm_f16", "gemm_f16f32", "gemm_f32_valu", "gemm_f32_noalloc",
           "gemm_f32_colmajor", "gemm_f16_colmajor", "gemm_f16f32_colmajor", "gemm_status_string",
           "gemm_describe", "gemm_set_load_mode", "gemm_set_tile_config", "gemm_set_split",
           "gemm_set_tail_split", "gemm_set_pack", "gemm_set_stream_k", "gemm_set_workspace_limit",
           "gemm_probe_mfma") + LAYOUT_NAMES + ROW_NAMES + BLOCK_NAMES
GEMM_ERR_SCRATCH_LIMIT = -200
GEMM_ERR_NO_WORKSPACE = -201


class GemmError(RuntimeError):
    def __init__(self, status):
        super().__init__("gemm status %d: %s" % (status, gemm_status_string(status)))
        self.status = status


def _addr(x):
    """Device address of a torch tensor, or an integer address as given."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _stream(s):
    if s is None:
        return None
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream
    return int(s)


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """C := alpha*A*B + beta*C in fp32 (see include/gemm.h).  A, B, C are
    device addresses or torch tensors; stream is a hipStream_t handle, a
    torch.cuda.Stream or None (the null stream).  Returns the status code."""
    return _lib.gemm_f32(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                         _stream(stream))


def gemm_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """fp16-in / fp16-out GEMM with fp32 accumulation (see include/gemm.h)."""
    return _lib.gemm_f16(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                         _stream(stream))


def gemm_f16f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """fp16 A and B, fp32 C and result, fp32 accumulation (see include/gemm.h)."""
    return _lib.gemm_f16f32(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                            _stream(stream))


def gemm_f32_valu(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """fp32 GEMM on the vector ALUs (ablation of the matrix-core path; see
    include/gemm.h)."""
    return _lib.gemm_f32_valu(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                              _stream(stream))


def gemm_f32_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """gemm_f32 with its split-K workspace in the library's fixed scratch
    region: no allocation (see include/gemm.h); GEMM_ERR_SCRATCH_LIMIT when
    the call would need more workspace than the region holds."""
    return _lib.gemm_f32_noalloc(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C),
                                 ldc, _stream(stream))


def gemm_f32_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """Column-major (BLAS layout) fp32 GEMM (see include/gemm.h)."""
    return _lib.gemm_f32_colmajor(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C),
                                  ldc, _stream(stream))


def gemm_f16_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """Column-major fp16 GEMM with fp32 accumulation (see include/gemm.h)."""
    return _lib.gemm_f16_colmajor(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C),
                                  ldc, _stream(stream))


def gemm_f16f32_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """Column-major fp16 A and B with an fp32 C (see include/gemm.h)."""
    return _lib.gemm_f16f32_colmajor(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta,
                                     _addr(C), ldc, _stream(stream))


def gemm_status_string(status):
    return _lib.gemm_status_string(int(status)).decode()


def gemm_describe(dtype, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc):
    """(status, text) describing the variant chosen for these arguments."""
    buf = ctypes.create_string_buffer(256)
    dt = {"f32": 0, "f16": 1, "f16f32": 2}.get(dtype, dtype)
    rc = _lib.gemm_describe(dt, M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                            buf, len(buf))
    return rc, buf.value.decode()


def gemm_set_load_mode(mode):
    """0 = vector/scalar loads by alignment (default), 1 = force scalar."""
    return _lib.gemm_set_load_mode(int(mode))


def gemm_set_tile_config(config):
    """0 = tile configuration by problem size (default); 1/2/3/4 = force the
    large/medium/small/tiny configuration (fp16 maps 4 to small); 5 = fp32
    medium with loads issued together; 6 = fp32 256x256 (fp16 large on
    32x32x16 blocks); 7 = fp32 64x64 with four waves (fp16 small); 8 = fp32
    128x64 with four waves (fp16 medium); 9 = fp32 64x64 with four waves in
    64-k steps (fp16 small); 10 = fp32 32x32, one wave, 64-k steps (fp16
    small)."""
    return _lib.gemm_set_tile_config(int(config))


def _layout_entry(name):
    fn = getattr(_lib, name)

    def call(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
        return fn(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                  _stream(stream))
    call.__name__ = name
    call.__doc__ = ("%s: C := alpha*op(A)*op(B) + beta*C with the operand layouts its suffix "
                    "names (see include/gemm.h).  Returns the status code." % name)
    return call


for _n in LAYOUT_NAMES:
    globals()[_n] = _layout_entry(_n)


def gemm_probe_mfma(dtype, iters, operands, out, stream=None):
    """Matrix-core ceiling probe (see include/gemm.h): `operands` and `out`
    are device torch tensors (at least 64 KiB and 1 MiB).  Returns (status,
    flops of the launch)."""
    flops = ctypes.c_double(0.0)
    rc = _lib.gemm_probe_mfma(int(dtype), int(iters), _addr(operands),
                              operands.numel() * operands.element_size(), _addr(out),
                              out.numel() * out.element_size(), ctypes.byref(flops),
                              _stream(stream))
    return rc, flops.value


def gemm_set_tail_split(mode):
    """fp32: 0 = split the last partly filled round of tiles by size
    (default), 1 = never, 2..64 = force that many K chunks for it."""
    return _lib.gemm_set_tail_split(int(mode))


def gemm_set_pack(mode):
    """0 = copy operands whose rows do not allow 16-byte loads to 16-byte rows
    in fp32 calls of at least 5e9 flops, or 1.5e9 with N % 4 == 0 (default);
    1 = never; 2 = whenever their rows do not allow 16-byte loads (fp16
    too).  Returns the previous mode, or -1."""
    return _lib.gemm_set_pack(int(mode))


def gemm_set_stream_k(mode):
    """fp32: 0 = Stream-K by size (default), 1 = never; with the 64x64
    four-wave tile or a forced tile configuration (1, 5, 6, 7): 2..4 = every
    tile's K steps over 1..3 workgroups per CU, 5..6 = whole rounds first,
    the rest over 1..2 more workgroups per CU.  Returns the previous mode,
    or -1."""
    return _lib.gemm_set_stream_k(int(mode))


def gemm_set_workspace_limit(nbytes):
    """Cap on one call's split-K workspace from the pool: -1 = none
    (default), 0 = never split, n = splits needing more than n bytes run
    unsplit.  Returns the previous setting."""
    return _lib.gemm_set_workspace_limit(int(nbytes))


def gemm_set_split(mode):
    """0 = split K by problem size (default), 1 = never, 2..64 = force that
    many K chunks."""
    return _lib.gemm_set_split(int(mode))


def _operand(name, t):
    """(transposed, ld) of a 2-D operand: rows contiguous (stride(1) == 1) as
    stored, or columns contiguous (stride(0) == 1: the transpose of a
    row-major tensor, e.g. X.t())."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = t.shape
    if t.stride(1) == 1 and (t.stride(0) >= cols or rows <= 1):
        return False, max(t.stride(0), cols, 1)
    if t.stride(0) == 1 and (t.stride(1) >= rows or cols <= 1):
        return True, max(t.stride(1), rows, 1)
    raise ValueError("%s must have contiguous rows (stride(1) == 1) or contiguous columns "
                     "(stride(0) == 1)" % name)


def gemm(A, B, C, alpha=1.0, beta=0.0, stream=None):
    """C := alpha*A@B + beta*C for 2-D torch tensors on the GPU (in place).

    A and B may be row-major (stride(1) == 1, rows possibly padded) or
    transposed views of row-major tensors (stride(0) == 1, e.g. X.t()); the
    latter run the _nt / _tn / _tt entry points, which read the operand in
    its stored orientation.  C must have stride(1) == 1.  float32 tensors go
    to the fp32 entry points, float16 to the fp16 ones, float16 A and B with a
    float32 C to the fp16-in / fp32-out ones.  Uses the current torch stream
    unless one is given."""
    ta, lda = _operand("A", A)
    tb, ldb = _operand("B", B)
    if C.dim() != 2 or C.stride(1) != 1 or (C.shape[0] > 1 and C.stride(0) < C.shape[1]):
        raise ValueError("C must be 2-D with stride(1) == 1 and stride(0) >= its column count")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape),
                                                             tuple(C.shape)))
    if A.dtype != B.dtype:
        raise ValueError("A and B must share a dtype")
    if A.dtype not in (torch.float32, torch.float16):
        raise ValueError("unsupported dtype %s" % A.dtype)
    mixed = A.dtype == torch.float16 and C.dtype == torch.float32
    if C.dtype != A.dtype and not mixed:
        raise ValueError("C must have A's dtype, or float32 with float16 A and B")
    if not (A.is_cuda and B.is_cuda and C.is_cuda):
        raise ValueError("A, B and C must be GPU tensors")
    if stream is None:
        stream = torch.cuda.current_stream(C.device)
    ldc = max(C.stride(0), N, 1)
    kind = "f32" if A.dtype == torch.float32 else ("f16f32" if mixed else "f16")
    name = "gemm_" + kind + ("" if not (ta or tb) else "_" + ("t" if ta else "n") + ("t" if tb else "n"))
    rc = globals()[name](M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)
    if rc != 0:
        raise GemmError(rc)
    return C


def _row_entry(name):
    fn = getattr(_lib, name)
    # pointers and the stream may be torch objects; numbers pass as they are
    at = [i for i, t in enumerate(fn.argtypes) if t is _P]

    def call(*args):
        args = list(args)
        if len(args) == len(fn.argtypes) - 1:
            args.append(None)
        for i in at[:-1]:
            args[i] = _addr(args[i])
        args[-1] = _stream(args[-1])
        return fn(*args)
    call.__name__ = name
    call.__doc__ = "%s (see include/gemm.h).  Returns the status code." % name
    return call


for _n in ROW_NAMES + BLOCK_NAMES:
    globals()[_n] = getattr(_lib, _n) if _n.endswith("_workspace") else _row_entry(_n)

_LORA_FN = {t: getattr(_lib, "gemm_lora_" + t) for t in ("f16", "f32")}
_LORA_GRAD_FN = {t: getattr(_lib, "gemm_lora_grad_" + t) for t in ("f16", "f32")}
_MOE_FN = {t: getattr(_lib, "gemm_moe_" + t) for t in ("f16", "f32")}
# the workspace depends on these sizes alone
_lora_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_lora_workspace)
_lora_grad_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_lora_grad_workspace)
_moe_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_moe_workspace)

_QUANT_FN = {t: getattr(_lib, "gemm_quant_i8_" + t) for t in ("f16", "f32")}
_I8_FN = {t: getattr(_lib, "gemm_i8_" + t) for t in ("f16", "f32")}
_GLU_FN = {t: getattr(_lib, "gemm_glu_" + t) for t in ("f16", "f32", "i8_f16", "i8_f32")}
_GLU_GRAD_FN = {t: getattr(_lib, "gemm_glu_grad_" + t) for t in ("f16", "f16f32", "f32")}
_i8_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_i8_workspace)
_glu_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_glu_workspace)
_glu_grad_bytes = functools.lru_cache(maxsize=4096)(_lib.gemm_glu_grad_workspace)

# activations of gated blocks: include/gemm.h's GEMM_ACT_*
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}

# of a call's type: suffix of the entry point, its workspace function's code
_KINDS = {torch.float16: ("f16", 1), torch.float32: ("f32", 0)}


# The checks below stand in front of calls that take some microseconds on the
# GPU: each looks at a tensor's shape and strides once.

_INT_MAX = 2 ** 31 - 1     # the entry points' sizes and leading dimensions; ctypes drops what is above

def _rows(name, t, rows, cols, dtype, dev):
    """Leading dimension of a rows x cols matrix with contiguous rows."""
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on GPU %d, like the first tensor" % (name, dev))
    if t.shape != (rows, cols):
        raise ValueError("%s must be %d x %d, not %s" % (name, rows, cols, tuple(t.shape)))
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError("%s must have contiguous rows (stride(1) == 1)" % name)
    if ld > _INT_MAX or rows > _INT_MAX:
        raise ValueError("%s is beyond 32 bits: size %s, rows %d elements apart"
                         % (name, tuple(t.shape), ld))
    return ld if ld > 1 else 1


def _stack(name, t, n, rows, cols, dtype, dev):
    """(leading dimension, stride) of n stacked rows x cols matrices."""
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on GPU %d, like the first tensor" % (name, dev))
    if t.shape != (n, rows, cols):
        raise ValueError("%s must be %d x %d x %d, not %s" % (name, n, rows, cols,
                                                              tuple(t.shape)))
    stride, ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError("%s must have contiguous rows (stride(2) == 1)" % name)
    if ld > _INT_MAX or rows > _INT_MAX or n > _INT_MAX:
        raise ValueError("%s is beyond 32 bits: size %s, rows %d elements apart"
                         % (name, tuple(t.shape), ld))
    return (ld if ld > 1 else 1), (stride if n > 1 else 0)


def _vector(name, t, n, dtype, dev):
    """Address of n contiguous values, None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be %d contiguous values of %s" % (name, n, dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on GPU %d, like the first tensor" % (name, dev))
    return t.data_ptr()


def _kind(X):
    """(suffix, code, device index) of a call on X."""
    kind = _KINDS.get(X.dtype)
    if kind is None:
        raise ValueError("unsupported dtype %s" % X.dtype)
    if not X.is_cuda:
        raise ValueError("the tensors must be GPU tensors")
    return kind[0], kind[1], X.get_device()


def _call_rows(fn, dev, stream, workspace, need, args):
    """Run entry point `fn` on the current stream of GPU `dev` or the one given.
    Without a workspace, one comes from torch's allocator on the current
    stream, or from the library's pool on a stream that was given (unless it is
    the current one and is being captured: then from torch's allocator too)."""
    if dev != _current_device():      # a default stream means the current GPU's
        with torch.cuda.device(dev):
            return _call_rows(fn, dev, stream, workspace, need, args)
    if stream is None and workspace is None and need == 0:
        rc = fn(*args, None, 0, _current_stream(dev))
        if rc != 0:
            raise GemmError(rc)
        return
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError("the stream must be one of GPU %d, like the first tensor" % dev)
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on GPU %d" % dev)
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need == 0:
        ws, size = None, 0
    elif stream is None or (torch.cuda.is_initialized()
                            and torch.cuda.is_current_stream_capturing()
                            and _stream(stream) == _current_stream(dev)):
        workspace = torch.empty(need, dtype=torch.uint8, device=_device(dev))
        ws, size = workspace.data_ptr(), need
    else:
        ws, size = None, 0
    stream = _current_stream(dev) if stream is None else _stream(stream)
    rc = fn(*args, ws, size, stream)
    if rc != 0:
        raise GemmError(rc)


def _call(fn, dev, stream, args):
    """Run entry point `fn`, which takes no workspace, on the current stream of
    GPU `dev` or the one given."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, args)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError("the stream must be one of GPU %d, like the first tensor" % dev)
    rc = fn(*args, _current_stream(dev) if stream is None else _stream(stream))
    if rc != 0:
        raise GemmError(rc)


@functools.lru_cache(maxsize=None)
def _device(index):
    return torch.device("cuda", index)


def _public_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# handle of a GPU's current stream, without a Stream object where torch offers that
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)


def lora(X, W, A, B, rows, Y, scale=None, ranks=None, alpha=1.0, beta=0.0, workspace=None,
         stream=None):
    """Y := alpha*(X @ W.t() + the low-rank term of each row's adapter) + beta*Y
    (in place): row i adds scale[a] * (X[i] @ A[a].t()) @ B[a].t() for a =
    rows[i], nothing where rows[i] is outside 0 .. L-1.

    X is M x K, W N x K, Y M x N, A L x R x K, B L x N x R (float16, or all
    float32; rows contiguous, possibly padded).  rows: M int32; scale: L
    float32 or None (1); ranks: L int32 or None (R), the ranks in use.
    workspace: a uint8 tensor of gemm_lora_workspace bytes to use instead of
    a new one.  Uses the current torch stream unless one is given; see
    gemm_lora_f16 in include/gemm.h."""
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3:
        raise ValueError("X and W must be 2-D and A 3-D")
    M, K = X.shape
    N = W.shape[0]
    L, R = A.shape[0], A.shape[1]
    dt = X.dtype
    kind, code, dev = _kind(X)
    ldx, ldw = _rows("X", X, M, K, dt, dev), _rows("W", W, N, K, dt, dev)
    ldy = _rows("Y", Y, M, N, dt, dev)
    lda, sa = _stack("A", A, L, R, K, dt, dev)
    ldb, sb = _stack("B", B, L, N, R, dt, dev)
    _call_rows(_LORA_FN[kind], dev, stream, workspace, _lora_bytes(code, M, N, K, L, R),
               (M, N, K, alpha, X.data_ptr(), ldx, W.data_ptr(), ldw, beta, Y.data_ptr(), ldy, L,
                R, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb,
                _vector("scale", scale, L, torch.float32, dev),
                _vector("ranks", ranks, L, torch.int32, dev),
                _vector("rows", rows, M, torch.int32, dev)))
    return Y


def lora_grad(dY, X, W, A, B, rows, dX=None, dA=None, dB=None, scale=None, ranks=None, alpha=1.0,
              beta_x=0.0, beta_ab=0.0, workspace=None, stream=None):
    """Gradients of lora() for dY (M x N), into those of dX (M x K, X's type),
    dA and dB (A's and B's shapes, float32) that are given:

        dX := alpha*(dY @ W + G @ A[a]) + beta_x*dX,  G[i] = scale[a] * dY[i] @ B[a]
        dA[a] := alpha * sum of G[i]^T X[i] over a's rows + beta_ab*dA[a]
        dB[a] := alpha*scale[a] * sum of dY[i]^T (X[i] @ A[a].t()) + beta_ab*dB[a]

    The other arguments are lora()'s; see gemm_lora_grad_f16 in
    include/gemm.h.  Returns (dX, dA, dB)."""
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3:
        raise ValueError("X and W must be 2-D and A 3-D")
    M, K = X.shape
    N = W.shape[0]
    L, R = A.shape[0], A.shape[1]
    dt = X.dtype
    kind, code, dev = _kind(X)
    lddy = _rows("dY", dY, M, N, dt, dev)
    ldx, ldw = _rows("X", X, M, K, dt, dev), _rows("W", W, N, K, dt, dev)
    lda, sa = _stack("A", A, L, R, K, dt, dev)
    ldb, sb = _stack("B", B, L, N, R, dt, dev)
    lddx = ldda = sda = lddb = sdb = 0
    if dX is not None:
        lddx = _rows("dX", dX, M, K, dt, dev)
    if dA is not None:
        ldda, sda = _stack("dA", dA, L, R, K, torch.float32, dev)
    if dB is not None:
        lddb, sdb = _stack("dB", dB, L, N, R, torch.float32, dev)
    _call_rows(_LORA_GRAD_FN[kind], dev, stream, workspace,
               _lora_grad_bytes(code, M, N, K, L, R),
               (M, N, K, alpha, dY.data_ptr(), lddy, X.data_ptr(), ldx, W.data_ptr(), ldw, L, R,
                A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb,
                _vector("scale", scale, L, torch.float32, dev),
                _vector("ranks", ranks, L, torch.int32, dev),
                _vector("rows", rows, M, torch.int32, dev),
                beta_x, _addr(dX), lddx, beta_ab, _addr(dA), ldda, sda, _addr(dB), lddb, sdb))
    return dX, dA, dB


def moe(X, router, W1, W2, top_k, Y, renorm=True, alpha=1.0, beta=0.0, ids=None, weights=None,
        workspace=None, stream=None):
    """A mixture-of-experts layer for a few tokens: Y := alpha * (the weighted
    sum of each token's top_k gated experts) + beta*Y (in place).

    X is M x D (1 <= M <= 256), router E x D, W1 E x 2F x D (gate rows, then up
    rows), W2 E x D x F, Y M x D (float16, or all float32).  ids (M x top_k
    int32) and weights (M x top_k float32), if given, receive the experts
    chosen, largest logit first, and their weights: softmax over the chosen
    (renorm) or over all experts.  workspace: a uint8 tensor of
    gemm_moe_workspace bytes to use instead of a new one.  Uses the current
    torch stream unless one is given; see gemm_moe_f16 in include/gemm.h."""
    if X.dim() != 2 or W2.dim() != 3:
        raise ValueError("X must be 2-D and W2 3-D")
    M, D = X.shape
    E, F = W2.shape[0], W2.shape[2]
    dt = X.dtype
    kind, code, dev = _kind(X)
    ldx, ldr = _rows("X", X, M, D, dt, dev), _rows("router", router, E, D, dt, dev)
    ldy = _rows("Y", Y, M, D, dt, dev)
    ld1, s1 = _stack("W1", W1, E, 2 * F, D, dt, dev)
    ld2, s2 = _stack("W2", W2, E, D, F, dt, dev)
    _call_rows(_MOE_FN[kind], dev, stream, workspace, _moe_bytes(code, M, D, F, E, top_k),
               (M, D, F, E, top_k, 1 if renorm else 0, alpha, X.data_ptr(), ldx,
                router.data_ptr(), ldr, W1.data_ptr(), ld1, s1, W2.data_ptr(), ld2, s2, beta,
                Y.data_ptr(), ldy, _vector("ids", ids, M * top_k, torch.int32, dev),
                _vector("weights", weights, M * top_k, torch.float32, dev)))
    return Y


def _act(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, not %r" % (", ".join(ACTIVATIONS), act))
    return code


def _in_place(X, ldx, W, ldw, eb):
    """Whether every row of X and of W starts at a multiple of 16 bytes (floats:
    anywhere), less than 2^23 from the one before."""
    ldx, ldw = ldx * eb, ldw * eb
    return (eb == 4 or ((X.data_ptr() | W.data_ptr() | ldx | ldw) & 15) == 0) and \
        (ldx | ldw) < 1 << 23


def quantize(X, Q=None, scale=None, stream=None):
    """Rows of X (M x K float16 or float32, contiguous, possibly padded) to 8-bit
    integers Q (M x K int8) with a scale each (M float32): scale = max |x| / 127,
    Q = the whole number nearest to x / scale, ties to even.  Q and scale are made
    where they are not given.  Returns (Q, scale); see gemm_quant_i8_f16 in
    include/gemm.h."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    kind, _, dev = _kind(X)
    ldx = _rows("X", X, M, K, X.dtype, dev)
    if Q is None:
        Q = torch.empty(M, K, dtype=torch.int8, device=X.device)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=X.device)
    _call(_QUANT_FN[kind], dev, stream,
          (M, K, X.data_ptr(), ldx, Q.data_ptr(), _rows("Q", Q, M, K, torch.int8, dev),
           _vector("scale", scale, M, torch.float32, dev)))
    return Q, scale


def gemm_i8(X, W, Y, x_scale=None, w_scale=None, alpha=1.0, beta=0.0, workspace=None,
            stream=None):
    """Y := alpha * (w_scale * (x_scale[:, None] * (X @ W.t()))) + beta*Y (in place)
    for 8-bit integers: X M x K and W N x K int8, Y M x N float16 or float32 (rows
    contiguous, possibly padded), x_scale M and w_scale N float32 or None (1).  The
    sum is exact.  workspace: a uint8 tensor of gemm_i8_workspace bytes to use
    instead of a new one.  Uses the current torch stream unless one is given; see
    gemm_i8_f16 in include/gemm.h."""
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be 2-D")
    M, K = X.shape
    N = W.shape[0]
    kind, _, dev = _kind(Y)
    ldx, ldw = _rows("X", X, M, K, torch.int8, dev), _rows("W", W, N, K, torch.int8, dev)
    ldy = _rows("Y", Y, M, N, Y.dtype, dev)
    _call_rows(_I8_FN[kind], dev, stream, workspace,
               _i8_bytes(M, N, K, _in_place(X, ldx, W, ldw, 1)),
               (M, N, K, alpha, X.data_ptr(), ldx, _vector("x_scale", x_scale, M, torch.float32, dev),
                W.data_ptr(), ldw, _vector("w_scale", w_scale, N, torch.float32, dev), beta,
                Y.data_ptr(), ldy))
    return Y


def glu(X, W, H, act="silu", Z=None, x_scale=None, w_scale=None, workspace=None, stream=None):
    """A gated block: H := act(G) * U, [G U] = X @ W.t() (in place), one kernel.

    X is M x K, W 2F x K (gate rows, then up rows), H M x F (float16, or all
    float32; rows contiguous, possibly padded).  act: "silu", "gelu", "gelu_tanh"
    or "relu".  Z (M x 2F), if given, receives [G U] for glu_grad().  X and W may be
    int8 with x_scale (M float32) and w_scale (2F float32), None for 1; Z then is
    not offered.  workspace: a uint8 tensor of gemm_glu_workspace bytes to use
    instead of a new one.  Uses the current torch stream unless one is given; see
    gemm_glu_f16 in include/gemm.h."""
    if X.dim() != 2 or H.dim() != 2:
        raise ValueError("X and H must be 2-D")
    M, K = X.shape
    F = H.shape[1]
    kind, code, dev = _kind(H)
    code_act = _act(act)
    i8 = X.dtype is torch.int8
    dt = torch.int8 if i8 else H.dtype
    ldx, ldw = _rows("X", X, M, K, dt, dev), _rows("W", W, 2 * F, K, dt, dev)
    ldh = _rows("H", H, M, F, H.dtype, dev)
    if i8:
        if Z is not None:
            raise ValueError("Z goes with float16 or float32 X and W only")
        _call_rows(_GLU_FN["i8_" + kind], dev, stream, workspace,
                   _glu_bytes(2, M, F, K, _in_place(X, ldx, W, ldw, 1)),
                   (M, F, K, code_act, X.data_ptr(), ldx,
                    _vector("x_scale", x_scale, M, torch.float32, dev), W.data_ptr(), ldw,
                    _vector("w_scale", w_scale, 2 * F, torch.float32, dev), H.data_ptr(), ldh))
        return H
    if x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale go with int8 X and W only")
    z, ldz = None, 0
    if Z is not None:
        z, ldz = Z.data_ptr(), _rows("Z", Z, M, 2 * F, dt, dev)
    _call_rows(_GLU_FN[kind], dev, stream, workspace,
               _glu_bytes(code, M, F, K, _in_place(X, ldx, W, ldw, 2 if code else 4)),
               (M, F, K, code_act, X.data_ptr(), ldx, W.data_ptr(), ldw, H.data_ptr(), ldh, z, ldz))
    return H


def glu_grad(dH, X, W, dX=None, dW=None, act="silu", Z=None, beta_x=0.0, beta_w=0.0,
             workspace=None, stream=None):
    """Gradients of glu() for dH (M x F), into those of dX (M x K) and dW (2F x K)
    that are given:

        dG, dU = dH * U * act'(G), dH * act(G)
        dX := dG @ W[:F] + dU @ W[F:] + beta_x*dX
        dW := cat(dG.t() @ X, dU.t() @ X) + beta_w*dW

    Z: what glu() left, or None: G and U are computed again.  All float16, or all
    float32; dW may be float32 beside float16.  In float16 dG and dU are rounded to it
    once (scale the loss: below 2^-14 they lose digits, from 65520 on they are
    infinite).  workspace: a uint8 tensor of
    gemm_glu_grad_workspace bytes to use instead of a new one.  Uses the current
    torch stream unless one is given; see gemm_glu_grad_f16 in include/gemm.h.
    Returns (dX, dW)."""
    if X.dim() != 2 or dH.dim() != 2:
        raise ValueError("X and dH must be 2-D")
    M, K = X.shape
    F = dH.shape[1]
    dt = X.dtype
    kind, code, dev = _kind(X)
    code_act = _act(act)
    ldx, ldw = _rows("X", X, M, K, dt, dev), _rows("W", W, 2 * F, K, dt, dev)
    lddh = _rows("dH", dH, M, F, dt, dev)
    z, ldz, lddx, lddw = None, 0, 0, 0
    if Z is not None:
        z, ldz = Z.data_ptr(), _rows("Z", Z, M, 2 * F, dt, dev)
    if dX is not None:
        lddx = _rows("dX", dX, M, K, dt, dev)
    if dW is not None:
        if code and dW.dtype is torch.float32:
            kind = "f16f32"
        lddw = _rows("dW", dW, 2 * F, K, torch.float32 if kind == "f16f32" else dt, dev)
    _call_rows(_GLU_GRAD_FN[kind], dev, stream, workspace,
               _glu_grad_bytes(code, M, F, K, _in_place(X, ldx, W, ldw, 2 if code else 4)),
               (M, F, K, code_act, dH.data_ptr(), lddh, X.data_ptr(), ldx, W.data_ptr(), ldw, z,
                ldz, beta_x, _addr(dX), lddx, beta_w, _addr(dW), lddw))
    return dX, dW
