"""ctypes binding of libgg_moe (include/gg_moe.h) -- argument marshalling only.

Each function takes torch tensors (device memory allocated by PyTorch) or, for
the grouped GEMMs, raw integers for pointers, converts them to the C
arguments, calls the C entry point of the same name and raises GGError on a
non-GG_OK status.
Every step of the computation runs in the library's HIP kernels; if the
library has not been built, loading it raises.
"""
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgg_moe.so")

# enums of gg_moe.h
GG_BF16, GG_F16, GG_F32, GG_F8E4M3, GG_F8E5M2, GG_MXFP4 = 0, 1, 2, 3, 4, 5
GG_MAJOR_K, GG_MAJOR_M, GG_MAJOR_N = 0, 1, 2
GG_DSWIGLU, GG_DGEGLU, GG_DSITUGLU = 0, 1, 2
GG_FLAG_GATE_FIRST, GG_FLAG_GEGLU_MASK_FILTER, GG_FLAG_VALIDATE_OFFSETS = 1, 2, 4
GG_FLAG_TENSOR_RAGGED, GG_FLAG_STATIC_SCHED, GG_FLAG_AB_E5M2 = 8, 16, 32
GG_DEVERR_DECREASING, GG_DEVERR_GRANULE, GG_DEVERR_LAST, GG_DEVERR_SKIPPED = 1, 2, 4, 8
GG_DEVERR_IDS = 16
GG_FLAG_NORMALIZE = 64
GG_SOFTMAX, GG_SIGMOID = 0, 1
STATUS_NAMES = ["GG_OK", "GG_ERR_NULL", "GG_ERR_SHAPE", "GG_ERR_DTYPE", "GG_ERR_LAYOUT",
                "GG_ERR_ALIGN", "GG_ERR_MODE", "GG_ERR_WORKSPACE", "GG_ERR_UNSUPPORTED",
                "GG_ERR_DEVICE", "GG_ERR_HIP", "GG_ERR_OFFSETS", "GG_ERR_VALUE"]
EXPORTS = ["gg_abi_version", "gg_last_error", "gg_device_error", "gg_wgrad_workspace_size",
           "gg_wgrad", "gg_wgrad_noalloc", "gg_wgrad_mx", "gg_dglu_workspace_size", "gg_dglu", "gg_dglu_mx",
           "gg_dsrelu_workspace_size", "gg_dsrelu", "gg_route_workspace_size", "gg_route",
           "gg_route_bwd", "gg_plan_workspace_size", "gg_plan_max_rows", "gg_plan", "gg_permute",
           "gg_combine", "gg_combine_bwd", "gg_grad_workspace_size", "gg_grad_norm", "gg_grad_clip",
           "gg_mx4_quant", "gg_mx4_dequant", "gg_glu", "gg_gemm_mx4_workspace_size", "gg_gemm_mx4",
           "gg_moe_few_workspace_size", "gg_moe_few"]

_TORCH_DTYPE = {torch.bfloat16: GG_BF16, torch.float16: GG_F16, torch.float32: GG_F32,
                torch.float8_e4m3fn: GG_F8E4M3, torch.float8_e5m2: GG_F8E5M2}


class GGError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{name}: {message}")


_lib = None


def load_library(path=LIB_PATH):
    """Load libgg_moe.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run __graft_entry__.build() or "
                           "python moe_grouped_gemm_offset_amd/build.py")
    L = ctypes.CDLL(path)
    P, I32, I64, U32, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                               ctypes.c_uint32, ctypes.c_size_t, ctypes.c_float)
    L.gg_abi_version.restype = ctypes.c_int
    L.gg_abi_version.argtypes = []
    L.gg_last_error.restype = ctypes.c_char_p
    L.gg_last_error.argtypes = []
    L.gg_device_error.restype = ctypes.c_int
    L.gg_device_error.argtypes = [P, P, ctypes.POINTER(I32)]
    L.gg_wgrad_workspace_size.restype = SZ
    L.gg_wgrad_workspace_size.argtypes = [I32]
    L.gg_dglu_workspace_size.restype = SZ
    L.gg_dglu_workspace_size.argtypes = [I32, I32, I32]
    L.gg_dsrelu_workspace_size.restype = SZ
    L.gg_dsrelu_workspace_size.argtypes = [I32]
    L.gg_wgrad.restype = ctypes.c_int
    L.gg_wgrad.argtypes = [P, I32, P, I32, P, I32, I64, I32, I32, P, P, I32, I32, U32, P, SZ, P]
    L.gg_wgrad_noalloc.restype = ctypes.c_int
    L.gg_wgrad_noalloc.argtypes = [P, I32, P, I32, P, I32, I64, I32, I32, P, P, I32, I32, U32, P]
    L.gg_wgrad_mx.restype = ctypes.c_int
    L.gg_wgrad_mx.argtypes = [P, P, P, P, P, I32, I64, I32, I32, P, P, I32, I32, U32, P, SZ, P]
    L.gg_dglu.restype = ctypes.c_int
    L.gg_dglu.argtypes = [P, I64, I32, P, P, I32, I32, P, I32, P, I32, P, P, P, P, I32, P, P,
                          I32, F, F, F, F, U32, P, SZ, P]
    L.gg_dglu_mx.restype = ctypes.c_int
    L.gg_dglu_mx.argtypes = [P, P, I64, I32, P, P, P, P, I32, I32, P, I32, P, I32, P, P, P, P, I32, P,
                             P, P, P, I32, F, F, F, F, F, F, U32, P, SZ, P]
    L.gg_dsrelu.restype = ctypes.c_int
    L.gg_dsrelu.argtypes = [P, P, I64, I32, P, P, P, P, I32, I32, P, I32, P, I32, P, P, P, I32, P, P,
                            P, U32, P, SZ, P]
    L.gg_route_workspace_size.restype = SZ
    L.gg_route_workspace_size.argtypes = [I64, I32]
    L.gg_route.restype = ctypes.c_int
    L.gg_route.argtypes = [P, I32, I64, I64, I32, P, I32, I32, F, U32, P, P, P, P, P, P, SZ, P]
    L.gg_route_bwd.restype = ctypes.c_int
    L.gg_route_bwd.argtypes = [P, I32, I64, I64, I32, I32, I32, F, U32, P, P, P, P, P, I64, P, P, P]
    L.gg_plan_workspace_size.restype = SZ
    L.gg_plan_workspace_size.argtypes = [I64, I32]
    L.gg_plan_max_rows.restype = I64
    L.gg_plan_max_rows.argtypes = [I64, I32, I32, I32]
    L.gg_plan.restype = ctypes.c_int
    L.gg_plan.argtypes = [P, I64, I32, I32, I32, I64, P, P, P, P, P, P, SZ, P]
    L.gg_permute.restype = ctypes.c_int
    L.gg_permute.argtypes = [P, I32, I64, I64, I32, P, I32, P, P, I32, I64, P, P]
    L.gg_combine.restype = ctypes.c_int
    L.gg_combine.argtypes = [P, I32, I64, I32, P, I64, I32, P, P, I64, P]
    L.gg_combine_bwd.restype = ctypes.c_int
    L.gg_combine_bwd.argtypes = [P, I32, I64, I64, I32, P, I64, P, P, I32, P, P, I32, P, P, P]
    L.gg_grad_workspace_size.restype = SZ
    L.gg_grad_workspace_size.argtypes = []
    L.gg_grad_norm.restype = ctypes.c_int
    L.gg_grad_norm.argtypes = [P, P, P, I32, I64, P, I32, P, SZ, P]
    L.gg_grad_clip.restype = ctypes.c_int
    L.gg_grad_clip.argtypes = [P, P, P, I32, I64, P, F, F, P, P, P]
    L.gg_mx4_quant.restype = ctypes.c_int
    L.gg_mx4_quant.argtypes = [P, I32, I64, I64, I32, P, P, P, P]
    L.gg_mx4_dequant.restype = ctypes.c_int
    L.gg_mx4_dequant.argtypes = [P, P, I64, I32, P, I32, I64, P, P]
    L.gg_glu.restype = ctypes.c_int
    L.gg_glu.argtypes = [P, I32, I64, P, I64, I32, P, I32, I64, I32, F, F, F, F, F, F, U32, P, P]
    L.gg_gemm_mx4_workspace_size.restype = SZ
    L.gg_gemm_mx4_workspace_size.argtypes = []
    L.gg_gemm_mx4.restype = ctypes.c_int
    L.gg_gemm_mx4.argtypes = [P, P, I64, I32, P, P, P, P, I32, P, I32, P, P, P, I32, U32, P, SZ, P]
    L.gg_moe_few_workspace_size.restype = SZ
    L.gg_moe_few_workspace_size.argtypes = [I32, I32, I32, I32]
    L.gg_moe_few.restype = ctypes.c_int
    L.gg_moe_few.argtypes = [P, I64, I32, I32, P, P, I32, I32, P, P, P, P, P, P, I32, I32, P, I32, I64,
                             I32, F, F, F, F, F, F, U32, P, SZ, P]
    _lib = L
    return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Fp8Out(ctypes.Structure):
    """gg_fp8_out of gg_moe.h (device pointers)."""
    _fields_ = [("d_col", ctypes.c_void_p), ("sfd_row", ctypes.c_void_p),
                ("sfd_col", ctypes.c_void_p), ("norm_const", ctypes.c_void_p)]


def _fp8_out(f):
    """A dict of tensors (sfd_row, norm_const and optionally d_col, sfd_col)
    as a gg_fp8_out, or None."""
    if f is None:
        return None
    return Fp8Out(_ptr(f.get("d_col")), _ptr(f.get("sfd_row")), _ptr(f.get("sfd_col")),
                  _ptr(f.get("norm_const")))


def _ref(s):
    return None if s is None else ctypes.addressof(s)


def _check(status):
    if status != 0:
        raise GGError(status, gg_last_error())


def gg_abi_version():
    return load_library().gg_abi_version()


def gg_last_error():
    return load_library().gg_last_error().decode()


def gg_wgrad_workspace_size(num_experts):
    return load_library().gg_wgrad_workspace_size(num_experts)


def gg_dglu_workspace_size(L, n, generate_dbias):
    return load_library().gg_dglu_workspace_size(L, n, int(bool(generate_dbias)))


def gg_dsrelu_workspace_size(L):
    return load_library().gg_dsrelu_workspace_size(L)


def _torch_stream(stream):
    """The torch stream object of a call's stream argument (None: the current
    stream; an int: the raw hipStream_t)."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream)
    return stream


def _workspace(ws, nbytes, like, stream):
    """The caller's workspace, or a new one allocated on the stream the call
    runs on: torch's caching allocator ties a freed block to the stream it
    was allocated on, so a workspace the caller drops is not handed to work
    on another stream while this call's kernels may still use it."""
    if ws is not None:
        return ws, ws.numel() * ws.element_size()
    with torch.cuda.stream(_torch_stream(stream)):
        t = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=like.device)
    return t, t.numel()


def _ab(a, flags):
    """Operand codes given as a float8_e5m2 tensor add GG_FLAG_AB_E5M2 (uint8
    or float8_e4m3fn codes leave flags as they are)."""
    return flags | GG_FLAG_AB_E5M2 if a is not None and a.dtype == torch.float8_e5m2 else flags


def _sched(flags):
    """GG_SCHED=static in the environment adds GG_FLAG_STATIC_SCHED (a
    benchmarking override; GG_SCHED=dynamic or unset leaves flags alone)."""
    return flags | GG_FLAG_STATIC_SCHED if os.environ.get("GG_SCHED") == "static" else flags


def gg_device_error(workspace, stream=None):
    code = ctypes.c_int32(0)
    _check(load_library().gg_device_error(_ptr(workspace), _stream(stream), ctypes.byref(code)))
    return code.value


def gg_wgrad(a, a_major, b, b_major, offsets, tokens_sum, hidden, intermediate,
             wgrad_dense=None, wgrad_ptrs=None, wgrad_dtype=None, accumulate=False, flags=0,
             workspace=None, stream=None):
    """Grouped wgrad (gg_wgrad of gg_moe.h).  a_major: GG_MAJOR_K/GG_MAJOR_M,
    b_major: GG_MAJOR_K/GG_MAJOR_N.  Returns the workspace used."""
    L = load_library()
    E = offsets.numel()
    if wgrad_dtype is None:
        wgrad_dtype = _TORCH_DTYPE[wgrad_dense.dtype]
    ws, nbytes = _workspace(workspace, L.gg_wgrad_workspace_size(E), offsets, stream)
    _check(L.gg_wgrad(_ptr(a), a_major, _ptr(b), b_major, _ptr(offsets), E, tokens_sum, hidden,
                      intermediate, _ptr(wgrad_dense), _ptr(wgrad_ptrs), wgrad_dtype,
                      int(bool(accumulate)), _sched(flags), _ptr(ws), nbytes, _stream(stream)))
    return ws


def gg_wgrad_noalloc(a, a_major, b, b_major, offsets, tokens_sum, hidden, intermediate,
                     wgrad_dense=None, wgrad_ptrs=None, wgrad_dtype=None, accumulate=False, flags=0,
                     stream=None):
    """Grouped wgrad on the library's static scratch (gg_wgrad_noalloc of
    gg_moe.h): no workspace is allocated or passed."""
    L = load_library()
    E = offsets.numel()
    if wgrad_dtype is None:
        wgrad_dtype = _TORCH_DTYPE[wgrad_dense.dtype]
    _check(L.gg_wgrad_noalloc(_ptr(a), a_major, _ptr(b), b_major, _ptr(offsets), E, tokens_sum, hidden,
                              intermediate, _ptr(wgrad_dense), _ptr(wgrad_ptrs), wgrad_dtype,
                              int(bool(accumulate)), _sched(flags), _stream(stream)))


def gg_wgrad_mx(a, sfa, b, sfb, offsets, tokens_sum, hidden, intermediate, wgrad_dense=None,
                wgrad_ptrs=None, wgrad_dtype=None, accumulate=False, flags=0, workspace=None,
                stream=None):
    """Grouped MXFP8 wgrad (gg_wgrad_mx of gg_moe.h): FP8 codes (uint8 /
    float8_e4m3fn tensors: E4M3; float8_e5m2 tensors or GG_FLAG_AB_E5M2:
    E5M2) and E8M0 scales, both operands K-major.  Returns the workspace
    used."""
    L = load_library()
    E = offsets.numel()
    if wgrad_dtype is None:
        wgrad_dtype = _TORCH_DTYPE[wgrad_dense.dtype]
    ws, nbytes = _workspace(workspace, L.gg_wgrad_workspace_size(E), offsets, stream)
    _check(L.gg_wgrad_mx(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(offsets), E, tokens_sum,
                         hidden, intermediate, _ptr(wgrad_dense), _ptr(wgrad_ptrs), wgrad_dtype,
                         int(bool(accumulate)), _sched(_ab(a, flags)), _ptr(ws), nbytes,
                         _stream(stream)))
    return ws


def gg_dglu(a, b_dense, b_ptrs, b_major, n, c, padded_offsets, alpha, beta, prob, d_row, dprob,
            dbias=None, act=GG_DSWIGLU, geglu_alpha=1.702, clamp_min=-7.0, clamp_max=7.0,
            linear_offset=1.0, flags=0, workspace=None, stream=None):
    """Grouped dgrad + dSwiGLU/dGeGLU (gg_dglu of gg_moe.h).  Returns the
    workspace used."""
    L = load_library()
    nl = padded_offsets.numel()
    ws, nbytes = _workspace(workspace, L.gg_dglu_workspace_size(nl, n, dbias is not None), a, stream)
    _check(L.gg_dglu(_ptr(a), a.shape[0], a.shape[1], _ptr(b_dense), _ptr(b_ptrs), b_major, n,
                     _ptr(c), _TORCH_DTYPE[c.dtype], _ptr(padded_offsets), nl, _ptr(alpha),
                     _ptr(beta), _ptr(prob), _ptr(d_row), _TORCH_DTYPE[d_row.dtype], _ptr(dprob),
                     _ptr(dbias), act, geglu_alpha, clamp_min, clamp_max, linear_offset, flags,
                     _ptr(ws), nbytes, _stream(stream)))
    return ws


def gg_dglu_mx(a, sfa, b, sfb, b_ptrs, sfb_ptrs, n, c, padded_offsets, alpha, beta, prob, d_row,
               dprob, dbias=None, amax=None, fp8_out=None, act=GG_DSWIGLU, geglu_alpha=1.702, clamp_min=-7.0,
               clamp_max=7.0, linear_offset=1.0, situ_beta1=4.0, situ_beta2=25.0, flags=0,
               workspace=None, stream=None, b_major=GG_MAJOR_K):
    """Grouped MXFP8 dgrad + dSwiGLU/dGeGLU/dSiTU-GLU (gg_dglu_mx of
    gg_moe.h): a is an (m_rows, k) tensor of FP8 codes (uint8 or
    float8_e4m3fn: E4M3; float8_e5m2: E5M2, as for gg_wgrad_mx).  b / b_ptrs
    hold (n, k) codes per expert with b_major GG_MAJOR_K, (k, n) ones with
    GG_MAJOR_N.  c may be float8_e4m3fn / float8_e5m2.  With a float8_e4m3fn / float8_e5m2 d_row
    fp8_out is a dict of the other FP8 outputs (sfd_row, norm_const and
    optionally d_col, sfd_col).  Returns the workspace used."""
    q = _fp8_out(fp8_out)
    L = load_library()
    nl = padded_offsets.numel()
    ws, nbytes = _workspace(workspace, L.gg_dglu_workspace_size(nl, n, dbias is not None), a, stream)
    _check(L.gg_dglu_mx(_ptr(a), _ptr(sfa), a.shape[0], a.shape[1], _ptr(b), _ptr(sfb),
                        _ptr(b_ptrs), _ptr(sfb_ptrs), b_major, n, _ptr(c), _TORCH_DTYPE[c.dtype],
                        _ptr(padded_offsets), nl, _ptr(alpha), _ptr(beta), _ptr(prob),
                        _ptr(d_row), _TORCH_DTYPE[d_row.dtype], _ptr(dprob), _ptr(dbias),
                        _ptr(amax), _ref(q), act, geglu_alpha, clamp_min, clamp_max, linear_offset,
                        situ_beta1, situ_beta2, _ab(a, flags), _ptr(ws), nbytes, _stream(stream)))
    return ws


def gg_dsrelu(a, sfa, b, sfb, b_ptrs, sfb_ptrs, n, c, padded_offsets, alpha, prob, d_row, dprob,
              amax=None, fp8_out=None, flags=0, workspace=None, stream=None, b_major=GG_MAJOR_K):
    """Grouped MXFP8 dgrad + dsReLU (gg_dsrelu of gg_moe.h); operand, C and
    D dtypes and fp8_out as for gg_dglu_mx.  Returns the workspace used."""
    q = _fp8_out(fp8_out)
    L = load_library()
    nl = padded_offsets.numel()
    ws, nbytes = _workspace(workspace, L.gg_dsrelu_workspace_size(nl), a, stream)
    _check(L.gg_dsrelu(_ptr(a), _ptr(sfa), a.shape[0], a.shape[1], _ptr(b), _ptr(sfb),
                       _ptr(b_ptrs), _ptr(sfb_ptrs), b_major, n, _ptr(c), _TORCH_DTYPE[c.dtype],
                       _ptr(padded_offsets), nl, _ptr(alpha), _ptr(prob), _ptr(d_row),
                       _TORCH_DTYPE[d_row.dtype], _ptr(dprob), _ptr(amax), _ref(q), _ab(a, flags), _ptr(ws),
                       nbytes, _stream(stream)))
    return ws


# --------------------------------------------------------------------------
# around the grouped GEMMs: router, dispatch and combine, gradient clipping
# --------------------------------------------------------------------------

def _refuse(t, what, shape, dtype, dev, rows):
    """Raises what _need or _need_rows found wrong with a tensor argument."""
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise GGError(3, f"{what} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise GGError(2, f"{what} has shape {tuple(t.shape)}, not {shape}")
    if t.get_device() != dev:
        raise GGError(9, f"{what} is on {t.device}, not on the device of the other arguments")
    raise GGError(4, f"{what} needs contiguous rows that do not overlap" if rows
                  else f"{what} must be contiguous")


def _need(t, what, shape, dtype, dev):
    """The address of a tensor argument of this shape, type and device index,
    contiguous; raises otherwise.  (Written for few steps: a call's host time
    is what a small call costs.)"""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _refuse(t, what, shape, dtype, dev, False)


def _need_rows(t, what, dtypes):
    """(address, rows, columns, row pitch, device index) of a matrix of one of
    the types whose rows are contiguous, at any pitch."""
    if t.dtype not in dtypes:
        _refuse(t, what, t.shape, dtypes, t.get_device(), True)
    if t.dim() != 2:
        raise GGError(2, f"{what} has shape {tuple(t.shape)}, not two dimensions")
    n, width = t.shape
    if t.is_contiguous():
        return t.data_ptr(), n, width, width, t.get_device()
    pitch, step = t.stride()
    if n * width and ((width > 1 and step != 1) or (n > 1 and pitch < width)):
        _refuse(t, what, t.shape, t.dtype, t.get_device(), True)
    return t.data_ptr(), n, width, pitch if n > 1 else width, t.get_device()


def _scratch(ws, size, stream, dev, *of):
    """(address, bytes, tensor) of a call's workspace: the caller's, or a new
    one of size(*of) bytes."""
    if ws is None:
        if dev < 0:
            raise GGError(9, "the arguments are not on a GPU")
        with torch.cuda.stream(_torch_stream(stream)):
            ws = torch.empty(size(*of), dtype=torch.uint8, device=dev)
    elif ws.get_device() != dev or not ws.is_contiguous():
        _refuse(ws, "workspace", ws.shape, ws.dtype, dev, False)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _first(t):
    return t.shape[0] if t.dim() else 0


def _last(t):
    return t.shape[-1] if t.dim() else 0


def _extent(t, what):
    """The length of a one-dimensional tensor argument."""
    if t.dim() != 1:
        raise GGError(2, f"{what} has shape {tuple(t.shape)}, not one dimension")
    return t.shape[0]


def _raw_stream(stream, dev):
    """The hipStream_t of a call's stream argument (None: the current stream).
    The arguments' device has to be the current one, where the library
    launches."""
    if dev < 0:
        raise GGError(9, "the arguments are not on a GPU")
    if torch._C._cuda_getDevice() != dev:
        raise GGError(9, f"the arguments are on device {dev}, which is not the current one")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


_FLOATS = (torch.bfloat16, torch.float16, torch.float32)
_BYTES = (torch.float8_e4m3fn, torch.float8_e5m2, torch.uint8)
_I32, _F32 = torch.int32, torch.float32


def gg_route_workspace_size(tokens, num_experts):
    return load_library().gg_route_workspace_size(tokens, num_experts)


def gg_plan_workspace_size(tokens, num_experts):
    return load_library().gg_plan_workspace_size(tokens, num_experts)


def gg_plan_max_rows(tokens, top_k, num_experts, granule=256):
    return load_library().gg_plan_max_rows(tokens, top_k, num_experts, granule)


def gg_grad_workspace_size():
    return load_library().gg_grad_workspace_size()


def gg_route(logits, ids, prob, counts, routed, balance=None, bias=None, score=GG_SOFTMAX, scale=1.0,
             flags=0, workspace=None, stream=None):
    """The router (gg_route of gg_moe.h): logits (T, E) at any row pitch; ids
    int32 and prob float32 (T, top_k), counts int32 (E,), routed int32 (1,)
    and balance float32 (1,) are written.  Returns the workspace used."""
    L = load_library()
    px, T, E, ld, dev = _need_rows(logits, "logits", _FLOATS)
    k = _last(ids)
    p_ids = _need(ids, "ids", (T, k), _I32, dev)
    p_prob = _need(prob, "prob", (T, k), _F32, dev)
    p_counts = _need(counts, "counts", (E,), _I32, dev)
    p_routed = _need(routed, "routed", (1,), _I32, dev)
    p_bal = None if balance is None else _need(balance, "balance", (1,), _F32, dev)
    p_bias = None if bias is None else _need(bias, "bias", (E,), _F32, dev)
    p_ws, nbytes, ws = _scratch(workspace, L.gg_route_workspace_size, stream, dev, T, E)
    _check(L.gg_route(px, _TORCH_DTYPE[logits.dtype], ld, T, E, p_bias, k, score, scale, flags, p_ids,
                      p_prob, p_counts, p_routed, p_bal, p_ws, nbytes, _raw_stream(stream, dev)))
    return ws


def gg_route_bwd(logits, ids, counts, routed, dprob, dlogits, row_of=None, dbalance=None,
                 score=GG_SOFTMAX, scale=1.0, flags=0, stream=None):
    """The gradient of gg_route's logits (gg_route_bwd of gg_moe.h).  dprob is
    float32: (T, top_k), or with row_of (T, top_k) one value per expert row,
    (m_rows,), as gg_dglu and gg_dsrelu write it."""
    L = load_library()
    px, T, E, ld, dev = _need_rows(logits, "logits", _FLOATS)
    k = _last(ids)
    p_ids = _need(ids, "ids", (T, k), _I32, dev)
    p_counts = _need(counts, "counts", (E,), _I32, dev)
    p_routed = _need(routed, "routed", (1,), _I32, dev)
    if row_of is None:
        m, p_row, p_dprob = 0, None, _need(dprob, "dprob", (T, k), _F32, dev)
    else:
        m = _extent(dprob, "dprob")
        p_row, p_dprob = _need(row_of, "row_of", (T, k), _I32, dev), _need(dprob, "dprob", (m,), _F32, dev)
    p_db = None if dbalance is None else _need(dbalance, "dbalance", (1,), _F32, dev)
    p_d = _need(dlogits, "dlogits", (T, E), logits.dtype, dev)
    _check(L.gg_route_bwd(px, _TORCH_DTYPE[logits.dtype], ld, T, E, k, score, scale, flags, p_ids,
                          p_counts, p_routed, p_dprob, p_row, m, p_db, p_d, _raw_stream(stream, dev)))


def gg_plan(ids, counts, padded_offsets, row_of, m_rows, granule=256, prob=None, prob_rows=None,
            workspace=None, stream=None):
    """Rows of every token's choices in the expert-sorted layout (gg_plan of
    gg_moe.h): ids int32 (T, top_k); counts and padded_offsets int32 (E,),
    row_of int32 (T, top_k) and prob_rows float32 (m_rows,) are written.
    Returns the workspace used (gg_device_error reads its error word)."""
    L = load_library()
    if ids.dim() != 2:
        raise GGError(2, f"ids has shape {tuple(ids.shape)}, not two dimensions")
    shape, dev, E = ids.shape, ids.get_device(), _extent(counts, "counts")
    T, k = shape
    p_ids = _need(ids, "ids", shape, _I32, dev)
    p_counts = _need(counts, "counts", (E,), _I32, dev)
    p_ends = _need(padded_offsets, "padded_offsets", (E,), _I32, dev)
    p_row = _need(row_of, "row_of", shape, _I32, dev)
    p_prob = None if prob is None else _need(prob, "prob", shape, _F32, dev)
    p_rows = None if prob_rows is None else _need(prob_rows, "prob_rows", (m_rows,), _F32, dev)
    p_ws, nbytes, ws = _scratch(workspace, L.gg_plan_workspace_size, stream, dev, T, E)
    _check(L.gg_plan(p_ids, T, k, E, granule, m_rows, p_prob, p_counts, p_ends, p_row, p_rows,
                     p_ws, nbytes, _raw_stream(stream, dev)))
    return ws


def gg_permute(x, row_of, counts, padded_offsets, x_rows, stream=None):
    """x_rows[row_of[t, j]] = x[t], zeros in the padding (gg_permute of
    gg_moe.h): x (T, width) at any row pitch, x_rows (m_rows, width); one- to
    four-byte types."""
    L = load_library()
    px, T, width, ld, dev = _need_rows(x, "x", _FLOATS + _BYTES)
    k, E, m = _last(row_of), _extent(counts, "counts"), _first(x_rows)
    p_row = _need(row_of, "row_of", (T, k), _I32, dev)
    p_counts = _need(counts, "counts", (E,), _I32, dev)
    p_ends = _need(padded_offsets, "padded_offsets", (E,), _I32, dev)
    p_out = _need(x_rows, "x_rows", (m, width), x.dtype, dev)
    _check(L.gg_permute(px, _TORCH_DTYPE.get(x.dtype, GG_F8E4M3), ld, T, width, p_row, k, p_counts,
                        p_ends, E, m, p_out, _raw_stream(stream, dev)))


def gg_combine(y_rows, row_of, out, weights=None, stream=None):
    """out[t] = sum_j weights[t, j] y_rows[row_of[t, j]] (gg_combine of
    gg_moe.h); weights None: 1.  out (T, width) at any row pitch."""
    L = load_library()
    p_out, T, width, ld, dev = _need_rows(out, "out", _FLOATS)
    k, m = _last(row_of), _first(y_rows)
    p_y = _need(y_rows, "y_rows", (m, width), out.dtype, dev)
    p_row = _need(row_of, "row_of", (T, k), _I32, dev)
    p_w = None if weights is None else _need(weights, "weights", (T, k), _F32, dev)
    _check(L.gg_combine(p_y, _TORCH_DTYPE[out.dtype], m, width, p_row, T, k, p_w, p_out, ld,
                        _raw_stream(stream, dev)))


def gg_combine_bwd(dout, y_rows, row_of, weights, counts, padded_offsets, dy_rows, dweights,
                   stream=None):
    """The gradients of gg_combine (gg_combine_bwd of gg_moe.h): dy_rows
    (m_rows, width), zeros in the padding, and dweights float32 (T, top_k)."""
    L = load_library()
    p_d, T, width, ld, dev = _need_rows(dout, "dout", _FLOATS)
    k, E, m = _last(row_of), _extent(counts, "counts"), _first(y_rows)
    p_y = _need(y_rows, "y_rows", (m, width), dout.dtype, dev)
    p_row = _need(row_of, "row_of", (T, k), _I32, dev)
    p_w = _need(weights, "weights", (T, k), _F32, dev)
    p_counts = _need(counts, "counts", (E,), _I32, dev)
    p_ends = _need(padded_offsets, "padded_offsets", (E,), _I32, dev)
    p_dy = _need(dy_rows, "dy_rows", (m, width), dout.dtype, dev)
    p_dw = _need(dweights, "dweights", (T, k), _F32, dev)
    _check(L.gg_combine_bwd(p_d, _TORCH_DTYPE[dout.dtype], ld, T, width, p_y, m, p_w, p_row, k, p_counts,
                            p_ends, E, p_dy, p_dw, _raw_stream(stream, dev)))


def grad_table(tensors):
    """What gg_grad_norm and gg_grad_clip take of a list of tensors on one
    GPU, built once and kept while the tensors keep their memory:
    (ptrs, ends, dtypes, total)."""
    for i, t in enumerate(tensors):
        if t.dtype not in _FLOATS:
            raise GGError(3, f"tensor {i} has dtype {t.dtype}")
        if not t.is_contiguous():
            raise GGError(4, f"tensor {i} must be contiguous")
        if t.device != tensors[0].device:
            raise GGError(9, f"tensor {i} is on {t.device}, not {tensors[0].device}")
    dev = tensors[0].device if tensors else torch.device("cuda")
    ends, total = [], 0
    for t in tensors:
        total += t.numel()
        ends.append(total)
    return (torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=dev),
            torch.tensor(ends, dtype=torch.int64, device=dev),
            torch.tensor([_TORCH_DTYPE[t.dtype] for t in tensors], dtype=torch.int32, device=dev), total)


def _need_table(ptrs, ends, dtypes, sumsq):
    n, dev = _extent(ptrs, "ptrs"), ptrs.get_device()
    return (_need(ptrs, "ptrs", (n,), torch.int64, dev), _need(ends, "ends", (n,), torch.int64, dev),
            _need(dtypes, "dtypes", (n,), _I32, dev), n, _need(sumsq, "sumsq", (1,), torch.float64, dev), dev)


def gg_grad_norm(ptrs, ends, dtypes, total, sumsq, accumulate=False, workspace=None, stream=None):
    """sumsq (float64, (1,)) = the sum of squares over many tensors
    (gg_grad_norm of gg_moe.h; grad_table makes the first four arguments).
    Returns the workspace used."""
    L = load_library()
    p_ptrs, p_ends, p_dt, n, p_sum, dev = _need_table(ptrs, ends, dtypes, sumsq)
    p_ws, nbytes, ws = _scratch(workspace, L.gg_grad_workspace_size, stream, dev)
    _check(L.gg_grad_norm(p_ptrs, p_ends, p_dt, n, total, p_sum, int(bool(accumulate)), p_ws, nbytes,
                          _raw_stream(stream, dev)))
    return ws


def gg_grad_clip(ptrs, ends, dtypes, total, sumsq, max_norm, norm, eps=1e-6, out_ptrs=None,
                 stream=None):
    """Scales every tensor by min(1, max_norm / (sqrt(sumsq) + eps)), in place
    or into out_ptrs' tensors; norm (float32, (2,)) = the norm and the factor
    (gg_grad_clip of gg_moe.h)."""
    L = load_library()
    p_ptrs, p_ends, p_dt, n, p_sum, dev = _need_table(ptrs, ends, dtypes, sumsq)
    p_norm = _need(norm, "norm", (2,), _F32, dev)
    p_out = None if out_ptrs is None else _need(out_ptrs, "out_ptrs", (n,), torch.int64, dev)
    _check(L.gg_grad_clip(p_ptrs, p_ends, p_dt, n, total, p_sum, max_norm, eps, p_norm, p_out,
                          _raw_stream(stream, dev)))


# --------------------------------------------------------------------------
# the experts' forward pass: MXFP4, the gated activation, a few tokens' layer
# --------------------------------------------------------------------------

# (those that this torch has)
_CODES = tuple(getattr(torch, t) for t in ("uint8", "float4_e2m1fn_x2") if hasattr(torch, t))
_SCALES = tuple(getattr(torch, t) for t in ("uint8", "float8_e8m0fnu") if hasattr(torch, t))


def _need_one(t, what, shape, dtypes, dev):
    """As _need, for any of the types."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _refuse(t, what, shape, dtypes, dev, False)


def _need_end(end, dev):
    return None if end is None else _need(end, "end", (1,), _I32, dev)


def gg_mx4_quant(x, codes, scales, end=None, stream=None):
    """Rows to MXFP4 (gg_mx4_quant of gg_moe.h): x (rows, width) at any row
    pitch; codes (rows, width / 2) and scales (rows, width / 32) are written,
    uint8 (or float4_e2m1fn_x2 and float8_e8m0fnu).  end: int32 (1,), the rows
    in use."""
    L = load_library()
    px, n, width, ld, dev = _need_rows(x, "x", _FLOATS)
    p_codes = _need_one(codes, "codes", (n, width // 2), _CODES, dev)
    p_scales = _need_one(scales, "scales", (n, width // 32), _SCALES, dev)
    _check(L.gg_mx4_quant(px, _TORCH_DTYPE[x.dtype], ld, n, width, p_codes, p_scales, _need_end(end, dev),
                          _raw_stream(stream, dev)))


def gg_mx4_dequant(codes, scales, out, end=None, stream=None):
    """The values of MXFP4 rows (gg_mx4_dequant of gg_moe.h): out (rows,
    width) at any row pitch, arguments as for gg_mx4_quant."""
    L = load_library()
    po, n, width, ld, dev = _need_rows(out, "out", _FLOATS)
    p_codes = _need_one(codes, "codes", (n, width // 2), _CODES, dev)
    p_scales = _need_one(scales, "scales", (n, width // 32), _SCALES, dev)
    _check(L.gg_mx4_dequant(p_codes, p_scales, n, width, po, _TORCH_DTYPE[out.dtype], ld, _need_end(end, dev),
                            _raw_stream(stream, dev)))


def gg_glu(c, y, prob=None, act=GG_DSWIGLU, geglu_alpha=1.702, clamp_min=-7.0, clamp_max=7.0,
           linear_offset=1.0, situ_beta1=4.0, situ_beta2=25.0, flags=0, end=None, stream=None):
    """The gated activation (gg_glu of gg_moe.h): c (rows, 2n) in 32-wide
    blocks of inputs and gates to y (rows, n), both at any row pitch, times
    prob (rows,) if given."""
    L = load_library()
    pc, rows, two_n, ldc, dev = _need_rows(c, "c", _FLOATS)
    py, n, width, ldy, ydev = _need_rows(y, "y", _FLOATS)
    if n != rows or 2 * width != two_n:
        raise GGError(2, f"y has shape {tuple(y.shape)}, not {(rows, two_n // 2)}")
    if ydev != dev:
        _refuse(y, "y", y.shape, y.dtype, dev, True)
    p_prob = None if prob is None else _need(prob, "prob", (rows,), _F32, dev)
    _check(L.gg_glu(pc, _TORCH_DTYPE[c.dtype], ldc, p_prob, rows, width, py, _TORCH_DTYPE[y.dtype], ldy, act,
                    geglu_alpha, clamp_min, clamp_max, linear_offset, situ_beta1, situ_beta2, flags,
                    _need_end(end, dev), _raw_stream(stream, dev)))


def gg_gemm_mx4_workspace_size():
    return load_library().gg_gemm_mx4_workspace_size()


def gg_gemm_mx4(a, sfa, b, sfb, offsets, d, alpha=None, bias=None, b_ptrs=None, sfb_ptrs=None, flags=0,
                workspace=None, stream=None):
    """The grouped product of MXFP4 rows and weights (gg_gemm_mx4 of
    gg_moe.h): a (m_rows, k / 2) codes, sfa (m_rows, k / 32) scales; b (L, n,
    k / 2), sfb (L, n, k / 32), or b = sfb = None and int64 (L,) addresses of
    each expert's in b_ptrs, sfb_ptrs; offsets int32 (L,) group ends; d
    (m_rows, n).  alpha float32 (L,), bias float32 (L, n).  Returns the
    workspace used (gg_device_error reads its error word)."""
    L = load_library()
    pd, m, n, ld, dev = _need_rows(d, "d", _FLOATS)
    if ld != n:
        _refuse(d, "d", d.shape, d.dtype, dev, False)
    k, E = 2 * _last(a), _extent(offsets, "offsets")
    p_a = _need_one(a, "a", (m, k // 2), _CODES, dev)
    p_sfa = _need_one(sfa, "sfa", (m, k // 32), _SCALES, dev)
    p_b = None if b is None else _need_one(b, "b", (E, n, k // 2), _CODES, dev)
    p_sfb = None if sfb is None else _need_one(sfb, "sfb", (E, n, k // 32), _SCALES, dev)
    p_bp = None if b_ptrs is None else _need(b_ptrs, "b_ptrs", (E,), torch.int64, dev)
    p_sp = None if sfb_ptrs is None else _need(sfb_ptrs, "sfb_ptrs", (E,), torch.int64, dev)
    p_off = _need(offsets, "offsets", (E,), _I32, dev)
    p_alpha = None if alpha is None else _need(alpha, "alpha", (E,), _F32, dev)
    p_bias = None if bias is None else _need(bias, "bias", (E, n), _F32, dev)
    p_ws, nbytes, ws = _scratch(workspace, L.gg_gemm_mx4_workspace_size, stream, dev)
    _check(L.gg_gemm_mx4(p_a, p_sfa, m, k, p_b, p_sfb, p_bp, p_sp, n, p_off, E, p_alpha, p_bias, pd,
                         _TORCH_DTYPE[d.dtype], flags, p_ws, nbytes, _raw_stream(stream, dev)))
    return ws


def gg_moe_few_workspace_size(tokens, top_k, hidden, inner):
    return load_library().gg_moe_few_workspace_size(tokens, top_k, hidden, inner)


def gg_moe_few(x, ids, prob, w1, w2, y, sf1=None, sf2=None, bias1=None, bias2=None, act=GG_DSWIGLU,
               geglu_alpha=1.702, clamp_min=-7.0, clamp_max=7.0, linear_offset=1.0, situ_beta1=4.0,
               situ_beta2=25.0, flags=0, workspace=None, stream=None):
    """A whole layer for up to 64 tokens (gg_moe_few of gg_moe.h): x (T, H)
    bf16 at any row pitch that is a multiple of 8; ids int32 and prob float32
    (T, top_k); w1 (E, 2I, H) and w2 (E, H, I) bf16, or their MXFP4 codes
    (E, 2I, H / 2), (E, H, I / 2) with scales sf1 (E, 2I, H / 32), sf2 (E, H,
    I / 32); bias1 float32 (E, 2I), bias2 (E, H); y (T, H) at any row pitch.
    Returns the workspace used."""
    L = load_library()
    px, T, H, ldx, dev = _need_rows(x, "x", (torch.bfloat16,))
    py, Ty, Hy, ldy, ydev = _need_rows(y, "y", _FLOATS)
    if (Ty, Hy) != (T, H):
        raise GGError(2, f"y has shape {tuple(y.shape)}, not {(T, H)}")
    if ydev != dev:
        _refuse(y, "y", y.shape, y.dtype, dev, True)
    if w1.dim() != 3:
        raise GGError(2, f"w1 has shape {tuple(w1.shape)}, not three dimensions")
    k, E, I = _last(ids), w1.shape[0], w1.shape[1] // 2
    mx4 = w1.dtype is not torch.bfloat16
    per, types = (2, _CODES) if mx4 else (1, (torch.bfloat16,))
    p_ids = _need(ids, "ids", (T, k), _I32, dev)
    p_prob = _need(prob, "prob", (T, k), _F32, dev)
    p_w1 = _need_one(w1, "w1", (E, 2 * I, H // per), types, dev)
    p_w2 = _need_one(w2, "w2", (E, H, I // per), types, dev)
    p_sf1 = None if sf1 is None else _need_one(sf1, "sf1", (E, 2 * I, H // 32), _SCALES, dev)
    p_sf2 = None if sf2 is None else _need_one(sf2, "sf2", (E, H, I // 32), _SCALES, dev)
    p_b1 = None if bias1 is None else _need(bias1, "bias1", (E, 2 * I), _F32, dev)
    p_b2 = None if bias2 is None else _need(bias2, "bias2", (E, H), _F32, dev)
    p_ws, nbytes, ws = _scratch(workspace, _few_bytes, stream, dev, T, k, H, I)
    _check(L.gg_moe_few(px, ldx, T, H, p_ids, p_prob, k, E, p_w1, p_sf1, p_b1, p_w2, p_sf2, p_b2,
                        GG_MXFP4 if mx4 else GG_BF16, I, py, _TORCH_DTYPE[y.dtype], ldy, act, geglu_alpha,
                        clamp_min, clamp_max, linear_offset, situ_beta1, situ_beta2, flags, p_ws, nbytes,
                        _raw_stream(stream, dev)))
    return ws


def _few_bytes(*of):
    # (at least the header, so that the call itself refuses what is out of range)
    return max(256, gg_moe_few_workspace_size(*of))
