"""ctypes binding of libfp8lm.so (include/lm_fp8.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  If the
library is missing the import fails loudly -- there is no fallback.
"""
import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfp8lm.so")

E4M3, E5M2 = 0, 1
EPI_NONE, EPI_RELU2_FWD, EPI_RELU2_BWD, EPI_ACCUM_F32 = 0, 1, 2, 3
GEMM_A_MN_MAJOR, GEMM_B_MN_MAJOR = 1, 2
MLP_REUSE_WEIGHT_CASTS, MLP_ACCUMULATE_WGRAD = 1, 2
LINEAR_REUSE_WEIGHT_CAST, LINEAR_ACCUMULATE_WGRAD = 1, 2
DTYPE_BF16, DTYPE_F32 = 0, 1
NORM_ACCUMULATE_WGRAD = 1
ROPE_INTERLEAVED, ROPE_INVERSE = 1, 2
ROPE_UNSCALED, ROPE_LINEAR, ROPE_NTK, ROPE_BY_PARTS = 0, 1, 2, 3

STATUS = {0: "LM_OK", 1: "LM_ERR_INVALID_ARG", 2: "LM_ERR_ALIGNMENT",
          3: "LM_ERR_UNSUPPORTED_SHAPE", 4: "LM_ERR_UNSUPPORTED_FORMAT", 5: "LM_ERR_CUDA",
          6: "LM_ERR_TIMEOUT", 7: "LM_ERR_NONFINITE"}

EXPORTED = ["lm_fp8_amax_scale_cast", "lm_fp8_gemm", "lm_relu2_mlp_saved_bytes",
            "lm_relu2_mlp_saved_carve", "lm_relu2_mlp_workspace_size", "lm_relu2_mlp_fwd",
            "lm_relu2_mlp_bwd", "lm_get_error", "lm_status_string", "lm_version",
            "lm_timing_attach", "lm_timing_detach", "lm_timing_kinds",
            "lm_relu2_mlp_bwd_noalloc", "lm_relu2_mlp_bwd_noalloc_max_bytes",
            "lm_selftest_bounded_wait", "lm_relu2_mlp_fwd_ex", "lm_relu2_mlp_bwd_ex",
            "lm_rmsnorm_fp8_cast", "lm_swiglu_mlp_saved_bytes", "lm_swiglu_mlp_saved_carve",
            "lm_swiglu_mlp_workspace_size", "lm_swiglu_mlp_fwd", "lm_swiglu_mlp_bwd",
            "lm_fp8_lmhead_ce_workspace_size", "lm_fp8_lmhead_ce", "lm_fp8_gemm_ex",
            "lm_fp8_gemm_workspace_size", "lm_fp8_linear_saved_bytes",
            "lm_fp8_linear_saved_carve", "lm_fp8_linear_workspace_size", "lm_fp8_linear_fwd",
            "lm_fp8_linear_bwd", "lm_fp8_gemm_split_plan", "lm_layernorm_fwd",
            "lm_layernorm_workspace_size", "lm_layernorm_bwd", "lm_dropout_add_fwd",
            "lm_dropout_add_bwd", "lm_dropout_add_layernorm_fwd",
            "lm_dropout_add_layernorm_bwd", "lm_rope", "lm_rope_inv_freq"]


class LmError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class MlpSaved(ctypes.Structure):
    """Mirror of lm_mlp_saved."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("Xq", "Wuq", "Wdq", "H", "hq", "scales")]


class LinearSaved(ctypes.Structure):
    """Mirror of lm_linear_saved."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("Xq", "Wq", "scales")]


class SwigluSaved(ctypes.Structure):
    """Mirror of lm_swiglu_saved."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("Xq", "Wguq", "Wdq", "GU", "h", "hq", "scales")]


class RopeTensor(ctypes.Structure):
    """Mirror of lm_rope_tensor."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "y")]
                + [(n, ctypes.c_int64) for n in
                   ("heads", "x_batch_stride", "x_seq_stride", "x_head_stride",
                    "y_batch_stride", "y_seq_stride", "y_head_stride")])


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m fp8_gemms_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int
    L.lm_fp8_amax_scale_cast.argtypes = [P, i64, i64, i64, i32, i32, P, P, P, P, P, P, P]
    L.lm_fp8_amax_scale_cast.restype = st
    L.lm_fp8_gemm.argtypes = [P, i32, P, i32, i64, i64, i64, P, P, i32, P, P, P, P]
    L.lm_fp8_gemm.restype = st
    L.lm_fp8_gemm_ex.argtypes = [P, i32, P, i32, i64, i64, i64, ctypes.c_uint32, P, P, i32, P, P,
                                 P, P, ctypes.c_size_t, P]
    L.lm_fp8_gemm_ex.restype = st
    L.lm_fp8_gemm_workspace_size.argtypes = []
    L.lm_fp8_gemm_workspace_size.restype = ctypes.c_size_t
    L.lm_relu2_mlp_saved_bytes.argtypes = [i64, i64, i64]
    L.lm_relu2_mlp_saved_bytes.restype = ctypes.c_size_t
    L.lm_relu2_mlp_saved_carve.argtypes = [P, ctypes.c_size_t, i64, i64, i64,
                                           ctypes.POINTER(MlpSaved)]
    L.lm_relu2_mlp_saved_carve.restype = st
    L.lm_relu2_mlp_workspace_size.argtypes = [i64, i64, i64]
    L.lm_relu2_mlp_workspace_size.restype = ctypes.c_size_t
    L.lm_relu2_mlp_fwd.argtypes = [P, P, P, i64, i64, i64, P, ctypes.POINTER(MlpSaved), P,
                                   ctypes.c_size_t, P]
    L.lm_relu2_mlp_fwd.restype = st
    L.lm_relu2_mlp_bwd.argtypes = [P, ctypes.POINTER(MlpSaved), i64, i64, i64, P, P, P, P,
                                   ctypes.c_size_t, P]
    L.lm_relu2_mlp_bwd.restype = st
    L.lm_get_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    L.lm_get_error.restype = st
    L.lm_status_string.argtypes = [st]
    L.lm_status_string.restype = ctypes.c_char_p
    L.lm_version.restype = ctypes.c_int
    L.lm_timing_attach.argtypes = [ctypes.POINTER(ctypes.c_void_p), i32]
    L.lm_timing_attach.restype = None
    L.lm_timing_detach.argtypes = []
    L.lm_timing_detach.restype = i32
    L.lm_timing_kinds.argtypes = [ctypes.c_char_p, i32]
    L.lm_timing_kinds.restype = i32
    L.lm_relu2_mlp_bwd_noalloc.argtypes = [P, ctypes.POINTER(MlpSaved), i64, i64, i64, P, P, P, P]
    L.lm_relu2_mlp_bwd_noalloc.restype = st
    L.lm_relu2_mlp_bwd_noalloc_max_bytes.argtypes = []
    L.lm_relu2_mlp_bwd_noalloc_max_bytes.restype = ctypes.c_size_t
    L.lm_relu2_mlp_fwd_ex.argtypes = [P, P, P, i64, i64, i64, P, ctypes.POINTER(MlpSaved),
                                      P, ctypes.c_size_t, ctypes.c_uint32, P]
    L.lm_relu2_mlp_fwd_ex.restype = st
    L.lm_relu2_mlp_bwd_ex.argtypes = [P, ctypes.POINTER(MlpSaved), i64, i64, i64, P, P, P, P,
                                      ctypes.c_size_t, ctypes.c_uint32, P]
    L.lm_relu2_mlp_bwd_ex.restype = st
    L.lm_rmsnorm_fp8_cast.argtypes = [P, P, i64, i64, ctypes.c_float, i32, P, P, P, P, P, P, P]
    L.lm_rmsnorm_fp8_cast.restype = st
    L.lm_swiglu_mlp_saved_bytes.argtypes = [i64, i64, i64]
    L.lm_swiglu_mlp_saved_bytes.restype = ctypes.c_size_t
    L.lm_swiglu_mlp_saved_carve.argtypes = [P, ctypes.c_size_t, i64, i64, i64,
                                            ctypes.POINTER(SwigluSaved)]
    L.lm_swiglu_mlp_saved_carve.restype = st
    L.lm_swiglu_mlp_workspace_size.argtypes = [i64, i64, i64]
    L.lm_swiglu_mlp_workspace_size.restype = ctypes.c_size_t
    L.lm_swiglu_mlp_fwd.argtypes = [P, P, P, i64, i64, i64, P, ctypes.POINTER(SwigluSaved), P,
                                    ctypes.c_size_t, P]
    L.lm_swiglu_mlp_fwd.restype = st
    L.lm_swiglu_mlp_bwd.argtypes = [P, ctypes.POINTER(SwigluSaved), i64, i64, i64, P, P, P, P,
                                    ctypes.c_size_t, P]
    L.lm_swiglu_mlp_bwd.restype = st
    L.lm_fp8_lmhead_ce_workspace_size.argtypes = [i64, i64, i64, i64]
    L.lm_fp8_lmhead_ce_workspace_size.restype = ctypes.c_size_t
    L.lm_fp8_lmhead_ce.argtypes = [P, P, P, i64, i64, i64, i64, ctypes.c_float, P, P, P, P,
                                   ctypes.c_size_t, P]
    L.lm_fp8_lmhead_ce.restype = st
    L.lm_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P]
    L.lm_selftest_bounded_wait.restype = st
    L.lm_fp8_gemm_split_plan.argtypes = [i64, i64, i64, i32, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_int)]
    L.lm_fp8_gemm_split_plan.restype = st
    for fn in ("lm_fp8_linear_saved_bytes", "lm_fp8_linear_workspace_size"):
        getattr(L, fn).argtypes = [i64, i64, i64]
        getattr(L, fn).restype = ctypes.c_size_t
    L.lm_fp8_linear_saved_carve.argtypes = [P, ctypes.c_size_t, i64, i64, i64,
                                            ctypes.POINTER(LinearSaved)]
    L.lm_fp8_linear_saved_carve.restype = st
    L.lm_fp8_linear_fwd.argtypes = [P, P, i64, i64, i64, P, ctypes.POINTER(LinearSaved), P,
                                    ctypes.c_size_t, ctypes.c_uint32, P]
    L.lm_fp8_linear_fwd.restype = st
    L.lm_fp8_linear_bwd.argtypes = [P, ctypes.POINTER(LinearSaved), i64, i64, i64, P, P, P,
                                    ctypes.c_size_t, ctypes.c_uint32, P]
    L.lm_fp8_linear_bwd.restype = st
    f32, f64, u32, u64 = ctypes.c_float, ctypes.c_double, ctypes.c_uint32, ctypes.c_uint64
    size = ctypes.c_size_t
    L.lm_layernorm_fwd.argtypes = [P, i64, P, P, i64, i64, f32, i32, P, i64, P, P, P, P]
    L.lm_layernorm_workspace_size.argtypes = [i64, i64]
    L.lm_layernorm_workspace_size.restype = size
    L.lm_layernorm_bwd.argtypes = [P, i64, P, i64, P, P, P, i64, i64, i32, P, i64, P, P, P, size,
                                   u32, P]
    L.lm_dropout_add_fwd.argtypes = [P, i64, P, i64, i64, i64, i32, f64, P, u64, P, i64, P]
    L.lm_dropout_add_bwd.argtypes = [P, i64, i64, i64, i32, f64, P, u64, P, i64, P]
    L.lm_dropout_add_layernorm_fwd.argtypes = [P, i64, P, i64, P, P, i64, i64, f32, i32, f64, P,
                                               u64, P, i64, P, i64, P, P, P, P]
    L.lm_dropout_add_layernorm_bwd.argtypes = [P, i64, P, i64, P, i64, P, P, P, i64, i64, i32, f64,
                                               P, u64, P, i64, P, i64, P, P, P, size, u32, P]
    L.lm_rope.argtypes = [ctypes.POINTER(RopeTensor), i32, i64, i64, i64, i64, i32, P, P, i64, f32,
                          u32, P]
    L.lm_rope_inv_freq.argtypes = [f64, i64, i32, f64, f64, f64, f64, ctypes.POINTER(f64),
                                   ctypes.POINTER(f32)]
    for fn in ("lm_layernorm_fwd", "lm_layernorm_bwd", "lm_dropout_add_fwd", "lm_dropout_add_bwd",
               "lm_dropout_add_layernorm_fwd", "lm_dropout_add_layernorm_bwd", "lm_rope",
               "lm_rope_inv_freq"):
        getattr(L, fn).restype = st
    return L


lib = _load()


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: building a torch.cuda.Stream for it takes 3 us
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status, what):
    if status != 0:
        raise LmError(status, what)


# ------------------------------------------------------- C-ABI mirrors
def lm_fp8_amax_scale_cast(x, fmt, amax_out, scale_out, inv_scale_out, q=None, qT=None,
                           relu2_input=False, amax_in=None, stream=None):
    """x: 2-D bf16 CUDA tensor (row stride = ld).  Scales are 1-element (or
    sliced) fp32 CUDA tensors.  Raises LmError on a non-zero status."""
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    assert x.dtype == torch.bfloat16 and x.stride(-1) == 1
    _check(lib.lm_fp8_amax_scale_cast(_p(x), rows, cols, ld, fmt, int(relu2_input), _p(amax_in),
                                      _p(amax_out), _p(scale_out), _p(inv_scale_out), _p(q),
                                      _p(qT), _stream(stream)), "lm_fp8_amax_scale_cast")


def lm_fp8_gemm(A, fa, B, fb, inv_scale_a, inv_scale_b, D, epi=EPI_NONE, aux=None,
                amax_out=None, stream=None):
    """D[M x N] (bf16) = epi(A[M x K] B[N x K]^T * inv_a * inv_b); A, B uint8 codes."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and tuple(D.shape) == (M, N)
    _check(lib.lm_fp8_gemm(_p(A), fa, _p(B), fb, M, N, K, _p(inv_scale_a), _p(inv_scale_b), epi,
                           _p(aux), _p(D), _p(amax_out), _stream(stream)), "lm_fp8_gemm")


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def lm_fp8_gemm_workspace_size():
    return lib.lm_fp8_gemm_workspace_size()


def lm_fp8_gemm_split_plan(M, N, K, sm_count):
    """(parts, tail_tiles): the split-K tail lm_fp8_gemm_ex uses for this shape
    on a GPU of sm_count multiprocessors (host arithmetic only)."""
    parts, tail = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib.lm_fp8_gemm_split_plan(M, N, K, sm_count, ctypes.byref(parts), ctypes.byref(tail)),
           "lm_fp8_gemm_split_plan")
    return parts.value, tail.value


def lm_fp8_gemm_ex(A, fa, B, fb, inv_scale_a, inv_scale_b, D, flags=0, epi=EPI_NONE, aux=None,
                   amax_out=None, workspace=None, stream=None):
    """lm_fp8_gemm with per-operand storage: with GEMM_A_MN_MAJOR, A is given as
    its [K x M] transpose (row-major); with GEMM_B_MN_MAJOR, B as [K x N].
    workspace (a device buffer, or None) enables the split-K tail."""
    M, K = (A.shape[1], A.shape[0]) if flags & GEMM_A_MN_MAJOR else tuple(A.shape)
    N, K2 = (B.shape[1], B.shape[0]) if flags & GEMM_B_MN_MAJOR else tuple(B.shape)
    assert K == K2 and tuple(D.shape) == (M, N)
    _check(lib.lm_fp8_gemm_ex(_p(A), fa, _p(B), fb, M, N, K, flags, _p(inv_scale_a),
                              _p(inv_scale_b), epi, _p(aux), _p(D), _p(amax_out), _p(workspace),
                              _nbytes(workspace), _stream(stream)),
           "lm_fp8_gemm_ex")


def lm_rmsnorm_fp8_cast(R, weight, X, fmt, amax_out, scale_out, inv_scale_out, q=None, qT=None,
                        eps=1e-6, stream=None):
    rows, cols = R.shape
    assert R.is_contiguous() and X.is_contiguous()
    _check(lib.lm_rmsnorm_fp8_cast(_p(R), _p(weight), rows, cols, eps, fmt, _p(X), _p(amax_out),
                                   _p(scale_out), _p(inv_scale_out), _p(q), _p(qT),
                                   _stream(stream)), "lm_rmsnorm_fp8_cast")


def lm_relu2_mlp_saved_bytes(M, d, f):
    return lib.lm_relu2_mlp_saved_bytes(M, d, f)


def lm_relu2_mlp_workspace_size(M, d, f):
    return lib.lm_relu2_mlp_workspace_size(M, d, f)


def lm_relu2_mlp_saved_carve(buf, M, d, f):
    s = MlpSaved()
    _check(lib.lm_relu2_mlp_saved_carve(_p(buf), buf.numel() * buf.element_size(), M, d, f,
                                        ctypes.byref(s)), "lm_relu2_mlp_saved_carve")
    return s


def lm_relu2_mlp_fwd(X, W_up, W_down, Y, saved, workspace=None, stream=None):
    M, d = X.shape
    f = W_up.shape[0]
    _check(lib.lm_relu2_mlp_fwd(_p(X), _p(W_up), _p(W_down), M, d, f, _p(Y),
                                ctypes.byref(saved), _p(workspace), _nbytes(workspace),
                                _stream(stream)),
           "lm_relu2_mlp_fwd")


def lm_relu2_mlp_bwd(dY, saved, dX, dW_up, dW_down, workspace, stream=None):
    M, d = dY.shape
    f = dW_up.shape[0]
    _check(lib.lm_relu2_mlp_bwd(_p(dY), ctypes.byref(saved), M, d, f, _p(dX), _p(dW_up),
                                _p(dW_down), _p(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "lm_relu2_mlp_bwd")


def lm_relu2_mlp_fwd_ex(X, W_up, W_down, Y, saved, f, flags=0, workspace=None, stream=None):
    """f: hidden size (W_up may be None when its cast is reused)."""
    M, d = X.shape
    _check(lib.lm_relu2_mlp_fwd_ex(_p(X), _p(W_up), _p(W_down), M, d, f, _p(Y),
                                   ctypes.byref(saved), _p(workspace), _nbytes(workspace), flags,
                                   _stream(stream)),
           "lm_relu2_mlp_fwd_ex")


def lm_relu2_mlp_bwd_ex(dY, saved, dX, dW_up, dW_down, workspace, flags=0, stream=None):
    M, d = dY.shape
    f = dW_up.shape[0]
    _check(lib.lm_relu2_mlp_bwd_ex(_p(dY), ctypes.byref(saved), M, d, f, _p(dX), _p(dW_up),
                                   _p(dW_down), _p(workspace),
                                   workspace.numel() * workspace.element_size(), flags,
                                   _stream(stream)), "lm_relu2_mlp_bwd_ex")


def lm_relu2_mlp_bwd_noalloc(dY, saved, dX, dW_up, dW_down, stream=None):
    """The relu^2 MLP backward with the library's own fixed scratch (no workspace
    argument); see include/lm_fp8.h for its size limit and sharing rules."""
    M, d = dY.shape
    f = dW_up.shape[0]
    _check(lib.lm_relu2_mlp_bwd_noalloc(_p(dY), ctypes.byref(saved), M, d, f, _p(dX), _p(dW_up),
                                        _p(dW_down), _stream(stream)),
           "lm_relu2_mlp_bwd_noalloc")


def lm_fp8_linear_saved_bytes(M, K, N):
    return lib.lm_fp8_linear_saved_bytes(M, K, N)


def lm_fp8_linear_workspace_size(M, K, N):
    return lib.lm_fp8_linear_workspace_size(M, K, N)


def lm_fp8_linear_saved_carve(buf, M, K, N):
    s = LinearSaved()
    _check(lib.lm_fp8_linear_saved_carve(_p(buf), _nbytes(buf), M, K, N, ctypes.byref(s)),
           "lm_fp8_linear_saved_carve")
    return s


def lm_fp8_linear_fwd(X, W, Y, saved, N, flags=0, workspace=None, stream=None):
    """X [M x K] -> Y [M x N]; N is given because W may be None when its cast
    is reused (LINEAR_REUSE_WEIGHT_CAST)."""
    M, K = X.shape
    _check(lib.lm_fp8_linear_fwd(_p(X), _p(W), M, K, N, _p(Y), ctypes.byref(saved),
                                 _p(workspace), _nbytes(workspace), flags, _stream(stream)),
           "lm_fp8_linear_fwd")


def lm_fp8_linear_bwd(dY, saved, K, dX, dW, workspace, flags=0, stream=None):
    """dY [M x N]; dX [M x K] (or None: no dgrad); dW [N x K] bf16, or fp32
    with LINEAR_ACCUMULATE_WGRAD."""
    M, N = dY.shape
    _check(lib.lm_fp8_linear_bwd(_p(dY), ctypes.byref(saved), M, K, N, _p(dX), _p(dW),
                                 _p(workspace), _nbytes(workspace), flags, _stream(stream)),
           "lm_fp8_linear_bwd")


def lm_swiglu_mlp_saved_carve(buf, M, d, f):
    s = SwigluSaved()
    _check(lib.lm_swiglu_mlp_saved_carve(_p(buf), buf.numel() * buf.element_size(), M, d, f,
                                         ctypes.byref(s)), "lm_swiglu_mlp_saved_carve")
    return s


def lm_swiglu_mlp_fwd(X, W_gu, W_down, Y, saved, workspace=None, stream=None):
    M, d = X.shape
    f = W_gu.shape[0] // 2
    _check(lib.lm_swiglu_mlp_fwd(_p(X), _p(W_gu), _p(W_down), M, d, f, _p(Y),
                                 ctypes.byref(saved), _p(workspace), _nbytes(workspace),
                                 _stream(stream)), "lm_swiglu_mlp_fwd")


def lm_swiglu_mlp_bwd(dY, saved, dX, dW_gu, dW_down, workspace, stream=None):
    M, d = dY.shape
    f = dW_gu.shape[0] // 2
    _check(lib.lm_swiglu_mlp_bwd(_p(dY), ctypes.byref(saved), M, d, f, _p(dX), _p(dW_gu),
                                 _p(dW_down), _p(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "lm_swiglu_mlp_bwd")


def lm_fp8_lmhead_ce(X, W, labels, loss_out, dX, dW, workspace, chunk, softcap=15.0,
                     stream=None):
    M, d = X.shape
    V = W.shape[0]
    assert labels.dtype == torch.int32 and dW.dtype == torch.float32
    _check(lib.lm_fp8_lmhead_ce(_p(X), _p(W), _p(labels), M, d, V, chunk, softcap, _p(loss_out),
                                _p(dX), _p(dW), _p(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "lm_fp8_lmhead_ce")


# ------------------------------------------- operators between the GEMMs
# The checks return what the call needs (sizes, strides), so that nothing is asked of a
# tensor twice: a small call's time is mostly this.
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _refuse(what, why, status=1):
    raise LmError(status, f"{what}: {why}")


def _check_device(what, device):
    # the launch, its stream and the multiprocessor count are those of the current device
    if device != torch.cuda.current_device():
        _refuse(what, "the tensors' device is not the current one")


def _check_rows(what, x, *others):
    """x and `others` (each may be None): [rows x cols] CUDA tensors of one type
    on the current device whose columns are adjacent.  Returns (rows, cols, lm_dtype, device index)
    and the row strides (0 for None)."""
    shape, dtype, device = x.shape, x.dtype, x.get_device()
    if len(shape) != 2 or device < 0:
        _refuse(what, "a 2-D CUDA tensor is wanted")
    _check_device(what, device)
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse(what, f"{dtype} is not supported", 4)
    rows, cols = shape
    ld, step = x.stride()
    if step != 1 and cols > 1:
        _refuse(what, "adjacent columns are wanted")
    lds = [ld]
    for t in others:
        if t is None:
            lds.append(0)
            continue
        if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
            _refuse(what, "tensors of one shape, type and device are wanted")
        ld, step = t.stride()
        if step != 1 and cols > 1:
            _refuse(what, "adjacent columns are wanted")
        lds.append(ld)
    return (rows, cols, code, device), lds


def _check_vectors(what, n, dtype, device, *vectors):
    for t in vectors:
        if t is not None and (t.shape != (n,) or t.dtype is not dtype
                              or t.get_device() != device or not t.is_contiguous()):
            _refuse(what, f"a contiguous {dtype} [{n}] vector of the same device is wanted")


def _check_rng(what, rng, offset, device):
    if (rng is None or rng.dtype not in (torch.int64, torch.uint64) or rng.numel() != 2
            or rng.get_device() != device or not rng.is_contiguous()):
        _refuse(what, "rng is a contiguous 64-bit integer {seed, offset} of the same device")
    if not 0 <= offset < 1 << 64:
        _refuse(what, "offset is an unsigned 64-bit integer")


def _check_wgrads(what, cols, x, flags, workspace, *wgrads):
    _check_vectors(what, cols, torch.float32 if flags & NORM_ACCUMULATE_WGRAD else x.dtype,
                   x.get_device(), *wgrads)
    if workspace is not None and (workspace.get_device() != x.get_device() or not workspace.is_contiguous()):
        _refuse(what, "the workspace is a contiguous buffer of the same device")


def lm_layernorm_fwd(X, weight, bias, Y, mean=None, rstd=None, eps=1e-5, amax_out=None,
                     stream=None):
    what = "lm_layernorm_fwd"
    (rows, cols, dt, device), (ldx, ldy) = _check_rows(what, X, Y)
    _check_vectors(what, cols, X.dtype, device, weight, bias)
    _check_vectors(what, rows, torch.float32, device, mean, rstd)
    _check_vectors(what, 1, torch.float32, device, amax_out)
    _check(lib.lm_layernorm_fwd(X.data_ptr(), ldx, _p(weight), _p(bias), rows, cols, eps, dt,
                                _p(Y), ldy, _p(mean), _p(rstd), _p(amax_out), _stream(stream)),
           what)


def lm_layernorm_workspace_size(rows, cols):
    return lib.lm_layernorm_workspace_size(rows, cols)


def lm_layernorm_bwd(dY, X, weight, mean, rstd, dX, dweight, dbias, workspace, flags=0,
                     stream=None):
    """dweight, dbias: [cols] of X's type, or fp32 with NORM_ACCUMULATE_WGRAD;
    either may be None."""
    what = "lm_layernorm_bwd"
    (rows, cols, dt, device), (ldx, lddy, lddx) = _check_rows(what, X, dY, dX)
    _check_vectors(what, cols, X.dtype, device, weight)
    _check_vectors(what, rows, torch.float32, device, mean, rstd)
    _check_wgrads(what, cols, X, flags, workspace, dweight, dbias)
    _check(lib.lm_layernorm_bwd(_p(dY), lddy, X.data_ptr(), ldx, _p(weight), _p(mean), _p(rstd),
                                rows, cols, dt, _p(dX), lddx, _p(dweight), _p(dbias),
                                _p(workspace), _nbytes(workspace), flags, _stream(stream)), what)


def lm_dropout_add_fwd(X, residual, Y, p, rng, offset=0, stream=None):
    what = "lm_dropout_add_fwd"
    (rows, cols, dt, device), (ldx, ldr, ldy) = _check_rows(what, X, residual, Y)
    _check_rng(what, rng, offset, device)
    _check(lib.lm_dropout_add_fwd(X.data_ptr(), ldx, _p(residual), ldr, rows, cols, dt, p,
                                  rng.data_ptr(), offset, _p(Y), ldy, _stream(stream)), what)


def lm_dropout_add_bwd(dY, dX, p, rng, offset=0, stream=None):
    what = "lm_dropout_add_bwd"
    (rows, cols, dt, device), (lddy, lddx) = _check_rows(what, dY, dX)
    _check_rng(what, rng, offset, device)
    _check(lib.lm_dropout_add_bwd(dY.data_ptr(), lddy, rows, cols, dt, p, rng.data_ptr(), offset,
                                  _p(dX), lddx, _stream(stream)), what)


def lm_dropout_add_layernorm_fwd(X, residual, weight, bias, S, Y, p, rng, offset=0, mean=None,
                                 rstd=None, eps=1e-5, amax_out=None, stream=None):
    what = "lm_dropout_add_layernorm_fwd"
    (rows, cols, dt, device), (ldx, ldr, lds, ldy) = _check_rows(what, X, residual, S, Y)
    _check_vectors(what, cols, X.dtype, device, weight, bias)
    _check_vectors(what, rows, torch.float32, device, mean, rstd)
    _check_vectors(what, 1, torch.float32, device, amax_out)
    _check_rng(what, rng, offset, device)
    _check(lib.lm_dropout_add_layernorm_fwd(
        X.data_ptr(), ldx, _p(residual), ldr, _p(weight), _p(bias), rows, cols, eps, dt, p,
        rng.data_ptr(), offset, _p(S), lds, _p(Y), ldy, _p(mean), _p(rstd), _p(amax_out),
        _stream(stream)), what)


def lm_dropout_add_layernorm_bwd(dY, dS, S, weight, mean, rstd, p, rng, dX, dR, dweight, dbias,
                                 workspace, offset=0, flags=0, stream=None):
    what = "lm_dropout_add_layernorm_bwd"
    (rows, cols, dt, device), (lds, lddy, ldds, lddx, lddr) = _check_rows(what, S, dY, dS, dX, dR)
    _check_vectors(what, cols, S.dtype, device, weight)
    _check_vectors(what, rows, torch.float32, device, mean, rstd)
    _check_rng(what, rng, offset, device)
    _check_wgrads(what, cols, S, flags, workspace, dweight, dbias)
    _check(lib.lm_dropout_add_layernorm_bwd(
        _p(dY), lddy, _p(dS), ldds, S.data_ptr(), lds, _p(weight), _p(mean), _p(rstd), rows, cols,
        dt, p, rng.data_ptr(), offset, _p(dX), lddx, _p(dR), lddr, _p(dweight), _p(dbias),
        _p(workspace), _nbytes(workspace), flags, _stream(stream)), what)


def lm_rope(xs, ys, inv_freq, positions=None, start=0, magnitude=1.0, flags=0, stream=None):
    """xs, ys: one or two [batch, seq, heads, head_dim] tensors each, which share
    all but the number of heads; inv_freq: fp64 [rot_dim / 2]; positions: int64
    [batch, seq], or None (start + s)."""
    if not 1 <= len(xs) <= 2 or len(ys) != len(xs) or xs[0].dim() != 4 or not xs[0].is_cuda:
        _refuse("lm_rope", "one or two 4-D CUDA tensors and as many outputs are wanted")
    batch, seq, _, head_dim = xs[0].shape
    dtype, device = xs[0].dtype, xs[0].get_device()
    _check_device("lm_rope", device)
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse("lm_rope", f"{dtype} is not supported", 4)
    if (inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.get_device() != device
            or not inv_freq.is_contiguous()):
        _refuse("lm_rope", "inv_freq is a contiguous fp64 vector of the same device")
    if positions is not None and (positions.dtype != torch.int64 or positions.get_device() != device
                                  or positions.numel() != batch * seq
                                  or not positions.is_contiguous()):
        _refuse("lm_rope", "positions is a contiguous int64 [batch, seq] of the same device")
    if not -1 << 63 <= start < 1 << 63:
        _refuse("lm_rope", "start is a signed 64-bit integer")
    parts = []
    for x, y in zip(xs, ys):
        shape, sx, sy = x.shape, x.stride(), y.stride()
        if (len(shape) != 4 or y.shape != shape or shape[0] != batch or shape[1] != seq
                or shape[3] != head_dim or x.dtype is not dtype or y.dtype is not dtype
                or x.get_device() != device or y.get_device() != device
                or (head_dim > 1 and (sx[3] != 1 or sy[3] != 1))):
            _refuse("lm_rope", "tensors of one type, device, batch, seq and head_dim with adjacent "
                               "elements are wanted")
        parts.append(RopeTensor(x.data_ptr(), y.data_ptr(), shape[2], *sx[:3], *sy[:3]))
    arr = (RopeTensor * len(parts))(*parts)
    _check(lib.lm_rope(arr, len(parts), batch, seq, head_dim, 2 * inv_freq.shape[0], code,
                       inv_freq.data_ptr(), _p(positions), start, magnitude, flags, _stream(stream)),
           "lm_rope")


def lm_rope_inv_freq(rot_dim, theta=10000.0, scaling=ROPE_UNSCALED, factor=1.0, context=0.0,
                     slow=1.0, fast=32.0):
    """(frequencies, magnitude): a list of rot_dim / 2 floats, and a float
    (host arithmetic only)."""
    out, mag = (ctypes.c_double * max(1, rot_dim // 2))(), ctypes.c_float(0.0)
    _check(lib.lm_rope_inv_freq(theta, rot_dim, scaling, factor, context, slow, fast, out,
                                ctypes.byref(mag)), "lm_rope_inv_freq")
    return list(out[:rot_dim // 2]), mag.value


def lm_get_error(stream=None):
    where = ctypes.c_uint32(0)
    st = lib.lm_get_error(_stream(stream), ctypes.byref(where))
    return st, where.value


def lm_selftest_bounded_wait(limit_ms, stream=None):
    _check(lib.lm_selftest_bounded_wait(limit_ms, _stream(stream)), "lm_selftest_bounded_wait")


def lm_status_string(status):
    return lib.lm_status_string(status).decode()


def lm_version():
    return lib.lm_version()


class KernelTimer:
    """Context manager over lm_timing_attach/detach: records a CUDA event before
    every library kernel launched on this host thread (at most `capacity`).
    After exit, `.kinds` labels each launch and `.durations_ms(end_event)`
    gives per-launch times, the last one ending at `end_event`."""

    def __init__(self, capacity=64):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.events:       # torch creates the CUDA event on first record
            e.record()
        self._arr = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.events])
        self.n = 0
        self.kinds = ""

    def __enter__(self):
        lib.lm_timing_attach(self._arr, len(self.events))
        return self

    def __exit__(self, *exc):
        self.n = lib.lm_timing_detach()
        buf = ctypes.create_string_buffer(self.n + 1)
        k = lib.lm_timing_kinds(buf, self.n)
        self.kinds = buf.raw[:k].decode()

    def durations_ms(self, end_event):
        marks = self.events[:self.n] + [end_event]
        return [a.elapsed_time(b) for a, b in zip(marks[:-1], marks[1:])]
