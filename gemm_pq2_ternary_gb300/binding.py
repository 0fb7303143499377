"""Thin Python binding of the C ABI in include/pq2.h (argument marshalling only).

Every function has the name of its C entry point, takes torch CUDA tensors,
passes their data pointers and the current CUDA stream, and raises
``PQ2Error`` when the C call returns a non-zero status.  All computation runs
in the CUDA kernels of libpq2.so; there is no other implementation here, and
importing this module fails if the library has not been built.
"""
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpq2.so")

PQ2_OK = 0
PQ2_ERR_INVALID_ARG = 1
PQ2_ERR_UNSUPPORTED_SHAPE = 2
PQ2_ERR_MISALIGNED = 3
PQ2_ERR_CUDA = 4
PQ2_ERR_TIMEOUT = 5
PQ2_ERR_WORKSPACE = 6
PQ2_ERR_BOUNDS = 7

PQ2_OP_GEMV = 0
PQ2_OP_SMALL = 1
PQ2_OP_PREFILL = 2
PQ2_OP_MATMUL = 3
PQ2_OP_SWIGLU_DOWN = 4

PQ2_WEIGHTS_STATIC = 1

# element types
PQ2_F32 = 0
PQ2_F16 = 1
PQ2_BF16 = 2
_I32, _F32 = torch.int32, torch.float32
_TYPE = {torch.float32: PQ2_F32, torch.float16: PQ2_F16, torch.bfloat16: PQ2_BF16}

# flags of the norms
PQ2_NORM_UNIT_OFFSET = 2
PQ2_NORM_NO_POST = 4
PQ2_GATE_SIGMOID = 8
PQ2_GATE_SILU = 16

# frequencies of rotary positions, flags of pq2_rope and pq2_cache4_append
PQ2_ROPE_PLAIN = 0
PQ2_ROPE_LINEAR = 1
PQ2_ROPE_BASE = 2
PQ2_ROPE_RAMP = 3
PQ2_ROPE_BANDS = 4
PQ2_ROPE_NEIGHBOURS = 1
PQ2_ROPE_INVERSE = 2
PQ2_ROPE_MAX_DIM = 512
PQ2_CACHE4_MAX_HEADS = 1024

PQ2_NORM_MAX_H = 49152
PQ2_LORA_MAX_R = 256
PQ2_LORA_MAX_L = 16384
PQ2_LORA_MAX_M = 1048576

# kernel variants for pq2_debug_force_kernel
PQ2_VARIANT_DEFAULT = 0
PQ2_VARIANT_GEMV_DIRECT = 1
PQ2_VARIANT_GEMV_RING = 2
PQ2_VARIANT_GEMV_STAGED = 3
PQ2_VARIANT_SMALL_DP4A = 1
PQ2_VARIANT_SMALL_TC = 2
PQ2_VARIANT_SMALL_TILE = 3
PQ2_VARIANT_SMALL_WTILE = 4
PQ2_VARIANT_PREFILL_128 = 1
PQ2_VARIANT_PREFILL_WIDE = 2
PQ2_VARIANT_PREFILL_TILE = 3
PQ2_VARIANT_PREFILL_WTILE = 4

SIZE_MAX = ctypes.c_size_t(-1).value

# Exported names and argument types (every one declared in include/pq2.h).
_P, _I64, _SZ, _I, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
_U32 = ctypes.c_uint32
_F = ctypes.c_float


class NormResidualArgs(ctypes.Structure):
    """pq2_norm_residual_args of include/pq2.h."""
    _fields_ = ([(n, _P) for n in ("y", "r", "r_out", "w_post", "gate", "w_next", "x")] +
                [(n, _I64) for n in ("ld_y", "ld_r", "ld_r_out", "ld_gate", "ld_x")] +
                [(n, ctypes.c_int32) for n in ("y_type", "r_type", "w_type", "gate_type", "x_type")] +
                [("eps", _F), ("alpha", _F), ("flags", _U32)])


# The same as bytes (packing them takes a third of the time of the Structure's
# fields); ctypes passes their address.
_norm_residual_args = struct.Struct("=7Q5q5i2fI")
assert _norm_residual_args.size == ctypes.sizeof(NormResidualArgs)

# pq2_lora_add_args and pq2_verify_drafts_args, likewise
_lora_add_args = struct.Struct("=9Q8qQ2i")
_verify_drafts_args = struct.Struct("=10Q6qQ")

# pq2_rope_scaling; pq2_cache4 and the arguments of the calls on it and on its
# pages, likewise
_rope_scaling = struct.Struct("=if4d")
_rope_args = struct.Struct("=6Q10q6iIi")
_CACHE4 = "4Q5q4i"
_cache4_append_args = struct.Struct("=" + _CACHE4 + "6Q10q4iIi")
_cache4_read_args = struct.Struct("=" + _CACHE4 + "2Q5q2i")
_cache4_attend_args = struct.Struct("=" + _CACHE4 + "3Q7qQf3i")
_pages_update_args = struct.Struct("=11Q6qQ")
_pages_compact_args = struct.Struct("=8Q6qQ")


SIGNATURES = {
    "pq2_status_string": ([_I], ctypes.c_char_p),
    "pq2_version": ([], ctypes.c_char_p),
    "pq2_quantize_act": ([_P, _I64, _I64, _P, _P, _P, _P], _I),
    "pq2_pack_weights": ([_P, _P, _I64, _I64, _P, _P, _P], _I),
    "pq2_gemv": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _P], _I),
    "pq2_gemm_small": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _I),
    "pq2_gemm_small_ex": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _U32, _P, _SZ, _P], _I),
    "pq2_gemm_prefill": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _I),
    "pq2_matmul": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _I),
    "pq2_matmul_ex": ([_P, _P, _P, _P, _I64, _I64, _I64, _U32, _P, _SZ, _P], _I),
    "pq2_quantize_swiglu": ([_P, _I64, _I64, _P, _P, _P, _P], _I),
    "pq2_gemm_bf16_splitk": ([_P, _P, _P, _I64, _I64, _I64, _U32, _P], _I),
    "pq2_mlp_down_swiglu": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _I),
    "pq2_rmsnorm": ([_P, _I, _I64, _P, _I, _P, _I, _I64, _I64, _I64, _F, _U32, _P], _I),
    "pq2_norm_residual": ([ctypes.c_void_p, _I64, _I64, _P], _I),
    "pq2_lora_workspace_bytes": ([_I64] * 5, _SZ),
    "pq2_lora_add": ([_P, _I64, _P, _P, _I, _P, _P, _P, _P, _I64, _P, _I64, _I] + [_I64] * 5 +
                     [_P, _SZ, _P], _I),
    "pq2_lora_add_packed": ([_P, _P], _I),
    "pq2_verify_workspace_bytes": ([_I64] * 3, _SZ),
    "pq2_verify_drafts": ([_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _P, _P, _P] + [_I64] * 3 +
                          [_P, _SZ, _P], _I),
    "pq2_verify_drafts_packed": ([_P, _P], _I),
    "pq2_rope_table": ([_P, _I64, _I64, _I64, ctypes.c_double, _P, _P], _I),
    "pq2_rope": ([_P, _P], _I),
    "pq2_cache4_page_bytes": ([_I64] * 3, _SZ),
    "pq2_cache4_append": ([_P, _P], _I),
    "pq2_cache4_read": ([_P, _P], _I),
    "pq2_cache4_attend_workspace_bytes": ([_I64] * 4, _SZ),
    "pq2_cache4_attend": ([_P, _P], _I),
    "pq2_pages_workspace_bytes": ([_I64] * 2, _SZ),
    "pq2_pages_update": ([_P, _P], _I),
    "pq2_pages_compact": ([_P, _P], _I),
    "pq2_pages_copy": ([_P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P], _I),
    "pq2_workspace_bytes": ([_I, _I64, _I64, _I64], _SZ),
    "pq2_group_dots": ([_I, _P, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P], _I),
    "pq2_last_device_error": ([_P], _I),
    "pq2_debug_set_wait_limit_ns": ([_U64], _I),
    "pq2_debug_skip_stage": ([_I], _I),
    "pq2_bounds_checked": ([], _I),
    "pq2_debug_shrink_bounds": ([_I], _I),
    "pq2_debug_force_kernel": ([_I, _I], _I),
    "pq2_debug_gemv_floor": ([_I64, _I64, _U32, _P], _I),
    "pq2_debug_mma_rate": ([_I, _I, _P, _P], _I),
    "pq2_gemm_small_noalloc": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _I),
    "pq2_gemm_small_noalloc_max_scratch": ([], _SZ),
}


def load_library(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = load_library()


class PQ2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.pq2_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(status: int, where: str):
    if status != PQ2_OK:
        raise PQ2Error(status, where)


def _stream(stream):
    """The cudaStream_t as an int (ctypes passes it as the void* argument).
    The current stream is asked for as a raw handle: 0.2 us against 2.9 us for
    torch.cuda.current_stream(), which builds an object around it."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptr(t):
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("expected a contiguous CUDA tensor")
    return t.data_ptr()


def _dtype(t, dt, name):
    if t.dtype != dt:
        raise ValueError(f"{name}: expected {dt}, got {t.dtype}")


def pq2_version() -> str:
    return _lib.pq2_version().decode()


def pq2_status_string(status: int) -> str:
    return _lib.pq2_status_string(status).decode()


def pq2_workspace_bytes(op: int, M: int, N: int, K: int) -> int:
    return int(_lib.pq2_workspace_bytes(op, M, N, K))


def pq2_quantize_act(x, qp, S, T, stream=None):
    """x fp16 [M,K] -> qp int8 [M,K] (plane order), S fp32 [M,G], T int32 [M,G]."""
    _dtype(x, torch.float16, "x")
    _dtype(qp, torch.int8, "qp")
    _dtype(S, torch.float32, "S")
    _dtype(T, torch.int32, "T")
    M, K = x.shape
    _check(_lib.pq2_quantize_act(_ptr(x), M, K, _ptr(qp), _ptr(S), _ptr(T), _stream(stream)),
           "pq2_quantize_act")


def pq2_pack_weights(tern, ws, codes, ws_out, stream=None):
    """tern int8 [N,K] in {-1,0,1} -> codes uint8 [N,K/4]; ws copied to ws_out."""
    _dtype(tern, torch.int8, "tern")
    _dtype(codes, torch.uint8, "codes")
    N, K = tern.shape
    _check(_lib.pq2_pack_weights(_ptr(tern), _ptr(ws), N, K, _ptr(codes), _ptr(ws_out),
                                 _stream(stream)), "pq2_pack_weights")


def _mm_shapes(qp, codes):
    M, K = qp.shape
    N = codes.shape[0]
    if codes.shape[1] * 4 != K:
        raise ValueError("codes must be [N, K/4]")
    return M, N, K


def pq2_gemv(qp, S, T, codes, ws, y, stream=None):
    M, N, K = _mm_shapes(qp, codes)
    _dtype(y, torch.float32, "y")
    _check(_lib.pq2_gemv(_ptr(qp), _ptr(S), _ptr(T), _ptr(codes), _ptr(ws), _ptr(y), N, K,
                         _stream(stream)), "pq2_gemv")


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def pq2_gemm_small(qp, S, T, codes, ws, y, workspace=None, stream=None):
    M, N, K = _mm_shapes(qp, codes)
    wp, wb = _ws(workspace)
    _check(_lib.pq2_gemm_small(_ptr(qp), _ptr(S), _ptr(T), _ptr(codes), _ptr(ws), _ptr(y),
                               M, N, K, wp, wb, _stream(stream)), "pq2_gemm_small")


def pq2_gemm_small_ex(qp, S, T, codes, ws, y, flags, workspace=None, stream=None):
    M, N, K = _mm_shapes(qp, codes)
    wp, wb = _ws(workspace)
    _check(_lib.pq2_gemm_small_ex(_ptr(qp), _ptr(S), _ptr(T), _ptr(codes), _ptr(ws), _ptr(y),
                                  M, N, K, flags, wp, wb, _stream(stream)), "pq2_gemm_small_ex")


def pq2_gemm_prefill(qp, S, T, codes, ws, y, workspace=None, stream=None):
    M, N, K = _mm_shapes(qp, codes)
    wp, wb = _ws(workspace)
    _check(_lib.pq2_gemm_prefill(_ptr(qp), _ptr(S), _ptr(T), _ptr(codes), _ptr(ws), _ptr(y),
                                 M, N, K, wp, wb, _stream(stream)), "pq2_gemm_prefill")


def pq2_gemm_small_noalloc(qp, S, T, codes, ws, y, stream=None):
    """pq2_gemm_small without a workspace: its scratch is a fixed device array
    inside the library (for callers that cannot allocate device memory)."""
    M, N, K = _mm_shapes(qp, codes)
    _check(_lib.pq2_gemm_small_noalloc(_ptr(qp), _ptr(S), _ptr(T), _ptr(codes), _ptr(ws), _ptr(y),
                                       M, N, K, _stream(stream)), "pq2_gemm_small_noalloc")


def pq2_gemm_small_noalloc_max_scratch() -> int:
    return int(_lib.pq2_gemm_small_noalloc_max_scratch())


def pq2_matmul(x, codes, ws, y, workspace, stream=None):
    M, K = x.shape
    N = codes.shape[0]
    wp, wb = _ws(workspace)
    _check(_lib.pq2_matmul(_ptr(x), _ptr(codes), _ptr(ws), _ptr(y), M, N, K, wp, wb,
                           _stream(stream)), "pq2_matmul")


def pq2_matmul_ex(x, codes, ws, y, flags, workspace, stream=None):
    M, K = x.shape
    N = codes.shape[0]
    wp, wb = _ws(workspace)
    _check(_lib.pq2_matmul_ex(_ptr(x), _ptr(codes), _ptr(ws), _ptr(y), M, N, K, flags, wp, wb,
                              _stream(stream)), "pq2_matmul_ex")


def pq2_gemm_bf16_splitk(x, w, y, flags=0, stream=None):
    """x [M, K], w [N, K], y [M, N]: torch.bfloat16 (or int16 bit patterns)
    on the device."""
    for t, name in ((x, "x"), (w, "w"), (y, "y")):
        if t.dtype not in (torch.bfloat16, torch.int16):
            raise ValueError(f"{name}: expected torch.bfloat16 (or int16 bit patterns), got {t.dtype}")
    M, K = x.shape
    N, Kw = w.shape
    if Kw != K or tuple(y.shape) != (M, N):
        raise ValueError(f"shapes: x {tuple(x.shape)}, w {tuple(w.shape)}, y {tuple(y.shape)}")
    _check(_lib.pq2_gemm_bf16_splitk(_ptr(x), _ptr(w), _ptr(y), M, N, K, flags,
                                     _stream(stream)), "pq2_gemm_bf16_splitk")


def pq2_quantize_swiglu(gu, qp, S, T, stream=None):
    """gu [M, 2I] fp32 (gate | up) -> qp, S, T of h = fp16(silu(gate) * up)."""
    M, I2 = gu.shape
    _check(_lib.pq2_quantize_swiglu(_ptr(gu), M, I2 // 2, _ptr(qp), _ptr(S), _ptr(T),
                                    _stream(stream)), "pq2_quantize_swiglu")


def pq2_mlp_down_swiglu(gu, codes, ws, y, workspace, stream=None):
    M, I2 = gu.shape
    N = codes.shape[0]
    wp, wb = _ws(workspace)
    _check(_lib.pq2_mlp_down_swiglu(_ptr(gu), _ptr(codes), _ptr(ws), _ptr(y), M, N, I2 // 2,
                                    wp, wb, _stream(stream)), "pq2_mlp_down_swiglu")


def _row(t, shape, name):
    """(pointer, element type, row stride) of a 2-D CUDA tensor whose rows are
    contiguous."""
    ty = _TYPE.get(t.dtype)
    if ty is None or not t.is_cuda or t.shape != shape:
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        if ty is None:
            raise ValueError(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # a single row's stride says nothing
    if shape[0] <= 1:
        ld = shape[1]
    return t.data_ptr(), ty, ld


def _vec(t, shape, dt, name):
    """Pointer of a contiguous CUDA vector of that shape (n,)."""
    if t.dtype is dt and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dt or t.shape != shape:
        raise ValueError(f"{name}: expected {dt} of shape {shape}, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name}: expected a contiguous CUDA tensor")


def _weight(w, H, name):
    """(pointer, element type) of a contiguous CUDA vector [H]."""
    ty = _TYPE.get(w.dtype)
    if ty is None or w.shape != (H,):
        raise ValueError(f"{name}: expected a float tensor of shape ({H},)")
    return _ptr(w), ty


def pq2_rmsnorm(r, w, x, eps=1e-6, flags=0, stream=None):
    """x = r / sqrt(mean(r^2) + eps) * w per row; r and x [M, H] (rows
    contiguous, any row stride), w [H] or None."""
    shape = r.shape
    rp, rt, rl = _row(r, shape, "r")
    xp, xt, xl = _row(x, shape, "x")
    wp, wt = (None, 0) if w is None else _weight(w, shape[1], "w")
    _check(_lib.pq2_rmsnorm(rp, rt, rl, wp, wt, xp, xt, xl, shape[0], shape[1], eps, flags,
                            _stream(stream)), "pq2_rmsnorm")


def pq2_norm_residual(y, r, r_out, w_post=None, gate=None, w_next=None, x=None, eps=1e-6, alpha=1.0,
                      flags=0, stream=None):
    """r_out = r + alpha * act(gate) * norm(y) * w_post and, if x is given,
    x = norm(r_out) * w_next, in one pass.  y, r, r_out, x [M, H]; gate [M, H]
    or [H]; rows contiguous, any row stride.  r_out may be r."""
    shape = r.shape
    yp, yt, yl = _row(y, shape, "y")
    rp, rt, rl = _row(r, shape, "r")
    op, ol = rp, rl
    if r_out is not r:
        op, ot, ol = _row(r_out, shape, "r_out")
        if ot != rt:
            raise ValueError("r_out: expected r's type")
    H = shape[1]
    pp = np_ = gp = xp = 0
    wt = gt = gl = xt = xl = 0
    if w_post is not None:
        pp, wt = _weight(w_post, H, "w_post")
    if w_next is not None:
        np_, nt = _weight(w_next, H, "w_next")
        if pp and nt != wt:
            raise ValueError("w_post and w_next: expected one type")
        wt = nt
    if gate is not None:
        if gate.dim() == 1:
            gp, gt = _weight(gate, H, "gate")
        else:
            gp, gt, gl = _row(gate, shape, "gate")
    if x is not None:
        xp, xt, xl = _row(x, shape, "x")
    args = _norm_residual_args.pack(yp, rp, op, pp, gp, np_, xp, yl, rl, ol, gl, xl, yt, rt, wt, gt, xt,
                                    eps, alpha, flags)
    _check(_lib.pq2_norm_residual(args, shape[0], H, _stream(stream)), "pq2_norm_residual")


def pq2_lora_workspace_bytes(M, N, K, L, R) -> int:
    return int(_lib.pq2_lora_workspace_bytes(M, N, K, L, R))


def alloc_lora_workspace(M, N, K, L, R, device="cuda"):
    n = pq2_lora_workspace_bytes(M, N, K, L, R)
    if n == SIZE_MAX:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_lora_workspace_bytes")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def pq2_lora_add(x, A, B, ids, y_in, y_out, workspace, ranks=None, scales=None, stream=None):
    """y_out[m] = y_in[m] + scales[l] * B[l] (A[l] x[m]) with l = ids[m]
    (l < 0: y_in[m]).  x [M, K], A [L, R, K], B [L, N, R] fp16 or bf16; ids
    int32 [M]; ranks int32 [L], scales fp32 [L] or None; y fp32 or bf16 [M, N]."""
    M, K = x.shape
    L, N, R = B.shape
    if A.shape != (L, R, K):
        raise ValueError(f"shapes: x {tuple(x.shape)}, A {tuple(A.shape)}, B {tuple(B.shape)}")
    xp, xt, xl = _row(x, (M, K), "x")
    dt = x.dtype
    if A.dtype is not dt or B.dtype is not dt:
        raise ValueError("A and B: expected x's type")
    if not (A.is_contiguous() and B.is_contiguous() and A.is_cuda and B.is_cuda):
        raise ValueError("expected a contiguous CUDA tensor")
    ip, it, il = _row(y_in, (M, N), "y_in")
    op, ol = ip, il
    if y_out is not y_in:
        op, ot, ol = _row(y_out, (M, N), "y_out")
        if it != ot:
            raise ValueError("y_out: expected y_in's type")
    wp, wb = (0, 0) if workspace is None else (_ptr(workspace), workspace.nbytes)
    args = _lora_add_args.pack(
        xp, A.data_ptr(), B.data_ptr(), _vec(ids, (M,), _I32, "ids"),
        0 if ranks is None else _vec(ranks, (L,), _I32, "ranks"),
        0 if scales is None else _vec(scales, (L,), _F32, "scales"),
        ip, op, wp, xl, il, ol, M, N, K, L, R, wb, xt, it)
    status = _lib.pq2_lora_add_packed(args, _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_lora_add")


def pq2_verify_workspace_bytes(B, rows, V) -> int:
    return int(_lib.pq2_verify_workspace_bytes(B, rows, V))


def alloc_verify_workspace(B, rows, V, device="cuda"):
    n = pq2_verify_workspace_bytes(B, rows, V)
    if n == SIZE_MAX:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_verify_workspace_bytes")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def pq2_verify_drafts(logits, row_start, drafts, q, u, e, temperature, accepted, tokens, workspace,
                      stream=None):
    """Kept drafts of each sequence and the token after them: logits, q (or
    None) fp32 [rows, V]; row_start int32 [B + 1]; drafts, tokens int32
    [rows]; u fp32 [rows]; e fp32 [B, V]; temperature fp32, accepted int32 [B]."""
    shape = logits.shape
    rows, V = shape
    nb = temperature.shape[0]
    lp, lt, ll = _row(logits, shape, "logits")
    ep, et, el = _row(e, (nb, V), "e")
    qp, qt, ql = (0, PQ2_F32, 0) if q is None else _row(q, shape, "q")
    if lt or et or qt:
        raise ValueError("logits, q and e: expected torch.float32")
    wp, wb = (0, 0) if workspace is None else (_ptr(workspace), workspace.nbytes)
    n, m = (rows,), (nb,)
    args = _verify_drafts_args.pack(
        lp, _vec(row_start, (nb + 1,), _I32, "row_start"), _vec(drafts, n, _I32, "drafts"), qp,
        _vec(u, n, _F32, "u"), ep, _vec(temperature, m, _F32, "temperature"),
        _vec(accepted, m, _I32, "accepted"), _vec(tokens, n, _I32, "tokens"), wp,
        ll, ql, el, nb, rows, V, wb)
    status = _lib.pq2_verify_drafts_packed(args, _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_verify_drafts")


def _heads(t, shape, name):
    """(pointer, element type, token stride, head stride) of a CUDA tensor
    [tokens, heads, values] whose heads are contiguous."""
    ty = _TYPE.get(t.dtype)
    if ty is None or not t.is_cuda or t.shape != shape:
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        if ty is None:
            raise ValueError(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, hs, unit = t.stride()
    M, H, D = shape
    if unit != 1 and D > 1:
        raise ValueError(f"{name}: a head's values must be contiguous")
    # a single head's, or token's, stride says nothing
    if H <= 1:
        hs = D
    if M <= 1:
        ld = H * hs
    return t.data_ptr(), ty, ld, hs


def pq2_rope_table(table, base, first=0, kind=PQ2_ROPE_PLAIN, factor=1.0, old_len=0.0, low=0.0, high=0.0,
                   magnitude=0.0, stream=None):
    """table fp32 [count, rot / 2, 2]: cosines and sines of positions first ..
    first + count - 1; kind and the rest: how the frequencies are scaled."""
    _dtype(table, _F32, "table")
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError(f"table: expected shape [count, rot / 2, 2], got {tuple(table.shape)}")
    _check(_lib.pq2_rope_table(_ptr(table), first, table.shape[0], 2 * table.shape[1], base,
                               _rope_scaling.pack(kind, magnitude, factor, old_len, low, high), _stream(stream)),
           "pq2_rope_table")


def _rot(table):
    """(pointer, rows, rot) of a table fp32 [rows, rot / 2, 2]."""
    if table is None:
        return 0, 0, 0
    rows, half, two = table.shape
    if table.dtype is not _F32 or two != 2:
        raise ValueError(f"table: expected {_F32} [rows, rot / 2, 2], got {table.dtype} {tuple(table.shape)}")
    return _ptr(table), rows, 2 * half


def pq2_rope(x, table, positions, out, x2=None, out2=None, flags=0, stream=None):
    """out = x with the first rot values of every head turned by their token's
    angles; x, out [M, heads, dim], x2, out2 [M, heads2, dim] likewise or None;
    table fp32 [rows, rot / 2, 2]; positions int32 [M], its rows.  out may be x."""
    shape = x.shape
    M, H, D = shape
    xp, xt, xl, xh = _heads(x, shape, "x")
    op, ot, ol, oh = (xp, xt, xl, xh) if out is x else _heads(out, shape, "out")
    x2p = o2p = H2 = x2l = x2h = o2l = o2h = 0
    if x2 is not None:
        shape2 = x2.shape
        H2 = shape2[1]
        if shape2 != (M, H2, D) or out2 is None:
            raise ValueError("x2: expected x's tokens and head size, and out2 with it")
        x2p, t2, x2l, x2h = _heads(x2, shape2, "x2")
        o2p, t3, o2l, o2h = (x2p, t2, x2l, x2h) if out2 is x2 else _heads(out2, shape2, "out2")
        if t2 != xt or t3 != ot:
            raise ValueError("x2 and out2: expected the types of x and out")
    tp, rows, rot = _rot(table)
    status = _lib.pq2_rope(_rope_args.pack(
        xp, x2p, op, o2p, tp, _vec(positions, (M,), _I32, "positions"), xl, xh, x2l, x2h, ol, oh, o2l, o2h, M, rows,
        H, H2, D, rot, xt, ot, flags, 0), _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_rope")


def pq2_cache4_page_bytes(heads, dim, page_tokens) -> int:
    return int(_lib.pq2_cache4_page_bytes(heads, dim, page_tokens))


def alloc_cache4(pages, heads, dim, page_tokens, device="cuda"):
    """A pool of pages: uint8 [pages, heads, page_tokens * (dim + 8)], zeros."""
    if pq2_cache4_page_bytes(heads, dim, page_tokens) == 0:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_cache4_page_bytes")
    return torch.zeros((pages, heads, page_tokens * (dim + 8)), dtype=torch.uint8, device=device)


def _cache4(pool, pages, row_start, lens, dim):
    """The fields of pq2_cache4: pool uint8 [pages, heads, T * (dim + 8)] (any
    page stride), pages int32 [B, W] (any row stride)."""
    P, heads, nbytes = pool.shape
    B, W = pages.shape
    T, rest = divmod(nbytes, dim + 8)
    if rest or pool.dtype is not torch.uint8 or not pool.is_cuda:
        raise ValueError(f"pool: expected a uint8 CUDA tensor [pages, heads, T * {dim + 8}], got {pool.dtype} "
                         f"{tuple(pool.shape)}")
    ps, hs, unit = pool.stride()
    if unit != 1 or (heads > 1 and hs != nbytes):
        raise ValueError("pool: a page must be contiguous")
    if P <= 1:
        ps = heads * nbytes
    if pages.dtype is not _I32 or not pages.is_cuda or (W > 1 and pages.stride(1) != 1):
        raise ValueError("pages: expected an int32 CUDA tensor with contiguous rows")
    return (pool.data_ptr(), pages.data_ptr(), _vec(row_start, (B + 1,), _I32, "row_start"),
            _vec(lens, (B,), _I32, "lens"), ps, P, pages.stride(0) if B > 1 else W, B, W, heads, dim, T, 0)


def pq2_cache4_append(k, v, pool, pages, row_start, lens, q=None, q_out=None, table=None, positions=None,
                      flags=0, stream=None):
    """New tokens into the cache: k (turned) and v [M, heads, dim], quantised;
    with q [M, q_heads, dim], q_out = q turned.  pool uint8 [pages, heads,
    T * (dim + 8)], pages int32 [B, W], row_start int32 [B + 1], lens int32 [B]
    (with the new tokens); table fp32 [rows, rot / 2, 2] or None; positions
    int32 [M] or None (the tokens' places)."""
    shape = k.shape
    M, H, D = shape
    kp, kt, kl, kh = _heads(k, shape, "k")
    vp, vt, vl, vh = _heads(v, shape, "v")
    if pool.shape[1] != H:
        raise ValueError(f"pool: expected {H} heads, got {pool.shape[1]}")
    qp = op = Hq = ql = qh = ol = oh = ot = 0
    qt = kt
    if q is not None:
        qshape = q.shape
        Hq = qshape[1]
        if qshape != (M, Hq, D) or q_out is None:
            raise ValueError("q: expected k's tokens and head size, and q_out with it")
        qp, qt, ql, qh = _heads(q, qshape, "q")
        op, ot, ol, oh = (qp, qt, ql, qh) if q_out is q else _heads(q_out, qshape, "q_out")
    if vt != kt or qt != kt:
        raise ValueError("k, v and q: expected one type")
    tp, rows, rot = _rot(table)
    status = _lib.pq2_cache4_append(_cache4_append_args.pack(
        *_cache4(pool, pages, row_start, lens, D), kp, vp, qp, op, tp,
        0 if positions is None else _vec(positions, (M,), _I32, "positions"), kl, kh, vl, vh, ql, qh, ol, oh, M, rows,
        Hq, rot, kt, ot, flags, 0), _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_cache4_append")


def pq2_cache4_read(pool, pages, row_start, lens, k_out, v_out, stream=None):
    """The cache's keys and values of the call's token rows: k_out, v_out
    [M, heads, dim], either may be None."""
    a = k_out if k_out is not None else v_out
    shape = a.shape
    if pool.shape[1] != shape[1]:
        raise ValueError(f"pool: expected {shape[1]} heads, got {pool.shape[1]}")
    kp, kt, kl, kh = (0, 0, 0, 0) if k_out is None else _heads(k_out, shape, "k_out")
    vp, vt, vl, vh = (0, kt, 0, 0) if v_out is None else _heads(v_out, shape, "v_out")
    if k_out is not None and vt != kt:
        raise ValueError("v_out: expected k_out's type")
    status = _lib.pq2_cache4_read(_cache4_read_args.pack(
        *_cache4(pool, pages, row_start, lens, shape[2]), kp, vp, kl, kh, vl, vh, shape[0], vt, 0), _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_cache4_read")


def pq2_cache4_attend_workspace_bytes(M, q_heads, heads, dim) -> int:
    return int(_lib.pq2_cache4_attend_workspace_bytes(M, q_heads, heads, dim))


def alloc_attend_workspace(M, q_heads, heads, dim, device="cuda"):
    n = pq2_cache4_attend_workspace_bytes(M, q_heads, heads, dim)
    if n == SIZE_MAX:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_cache4_attend_workspace_bytes")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def pq2_cache4_attend(q, pool, pages, row_start, lens, out, workspace, scale=None, window=0, max_rows=0, stream=None):
    """out = attention of the token rows q [M, q_heads, dim] (fp16 or bf16)
    over the cache, each over its sequence's positions up to its own (the last
    `window` of them); out of q's type.  scale: 1 / sqrt(dim) by default.
    max_rows: an upper bound of the sequences' rows (1 in a decode step)."""
    shape = q.shape
    M, Hq, D = shape
    qp, qt, ql, qh = _heads(q, shape, "q")
    op, ot, ol, oh = _heads(out, shape, "out")
    if ot != qt or qt == PQ2_F32:
        raise ValueError("q and out: expected float16 or bfloat16, both the same")
    wp, wb = (0, 0) if workspace is None else (_ptr(workspace), workspace.nbytes)
    status = _lib.pq2_cache4_attend(_cache4_attend_args.pack(
        *_cache4(pool, pages, row_start, lens, D), qp, op, wp, ql, qh, ol, oh, M, max_rows, window, wb,
        D ** -0.5 if scale is None else scale, Hq, qt, 0), _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_cache4_attend")


def pq2_pages_workspace_bytes(B, P) -> int:
    return int(_lib.pq2_pages_workspace_bytes(B, P))


def alloc_pages_workspace(B, P, device="cuda"):
    n = pq2_pages_workspace_bytes(B, P)
    if n == SIZE_MAX:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_pages_workspace_bytes")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _pages(t, shape, name):
    """(pointer, row stride) of an int32 CUDA tensor [B, W] with contiguous rows."""
    if t.dtype is not _I32 or t.shape != shape or not t.is_cuda or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected an int32 CUDA tensor of shape {tuple(shape)} with contiguous rows")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def pq2_pages_update(pages, refs, lens, source, keep, new_lens, page_tokens, pages_out, refs_out, copies, info,
                     workspace, stream=None):
    """Slot b goes on from slot source[b] (itself, another, or < 0: none) with
    its first keep[b] tokens, and gets pages for new_lens[b]: pages, pages_out
    int32 [B, W]; refs, refs_out int32 [P] (may be one); lens, source, keep,
    new_lens int32 [B]; copies int32 [B, 2] (for pq2_pages_copy); info int32 [2]."""
    shape = pages.shape
    B, W = shape
    P = refs.shape[0]
    pp, pl = _pages(pages, shape, "pages")
    op, ol = _pages(pages_out, shape, "pages_out")
    n = (B,)
    wp, wb = (0, 0) if workspace is None else (_ptr(workspace), workspace.nbytes)
    status = _lib.pq2_pages_update(_pages_update_args.pack(
        pp, _vec(lens, n, _I32, "lens"), _vec(refs, (P,), _I32, "refs"), _vec(source, n, _I32, "source"),
        _vec(keep, n, _I32, "keep"), _vec(new_lens, n, _I32, "new_lens"), op, _vec(refs_out, (P,), _I32, "refs_out"),
        _vec(copies, (B, 2), _I32, "copies"), _vec(info, (2,), _I32, "info"), wp, pl, ol, B, W, P, page_tokens, wb),
        _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_pages_update")


def pq2_pages_compact(pages, refs, lens, page_tokens, pages_out, refs_out, copies, info, workspace, stream=None):
    """The moves after which the pages in use (refs > 0) are the first ones:
    copies int32 [P // 2, 2] (for pq2_pages_copy), and pages and refs after them."""
    shape = pages.shape
    B, W = shape
    P = refs.shape[0]
    pp, pl = _pages(pages, shape, "pages")
    op, ol = _pages(pages_out, shape, "pages_out")
    wp, wb = (0, 0) if workspace is None else (_ptr(workspace), workspace.nbytes)
    status = _lib.pq2_pages_compact(_pages_compact_args.pack(
        pp, _vec(lens, (B,), _I32, "lens"), _vec(refs, (P,), _I32, "refs"), op, _vec(refs_out, (P,), _I32, "refs_out"),
        _vec(copies, (P // 2, 2), _I32, "copies"), _vec(info, (2,), _I32, "info"), wp, pl, ol, B, W, P, page_tokens,
        wb), _stream(stream))
    if status:
        raise PQ2Error(status, "pq2_pages_compact")


def pq2_pages_copy(pool, copies, layers=False, stream=None):
    """Copies pages within a pool: copies int32 [n, 2], pairs (old, new), those
    with a negative page skipped.  pool [pages, ...] of any type, a page
    contiguous; with layers, [layers, pages, ...], the same pairs in each."""
    if not pool.is_cuda:
        raise ValueError("pool: expected a CUDA tensor")
    at = 1 if layers else 0
    if pool.dim() <= at or (pool.numel() and not pool[(0,) * (at + 1)].is_contiguous()):
        raise ValueError("pool: a page must be contiguous")
    size = pool.element_size()
    P = pool.shape[at]
    nbytes = size
    for n in pool.shape[at + 1:]:
        nbytes *= n
    page_stride = pool.stride(at) * size if P > 1 else nbytes
    n = copies.shape[0]
    _check(_lib.pq2_pages_copy(pool.data_ptr(), nbytes, page_stride, P, pool.shape[0] if layers else 1,
                               pool.stride(0) * size if layers else 0, _vec(copies, (n, 2), _I32, "copies"), n,
                               _stream(stream)), "pq2_pages_copy")


def pq2_group_dots(op, qp, T, codes, dots, workspace=None, stream=None):
    M, N, K = _mm_shapes(qp, codes)
    wp, wb = _ws(workspace)
    _check(_lib.pq2_group_dots(op, _ptr(qp), _ptr(T), _ptr(codes), M, N, K, _ptr(dots), wp, wb,
                               _stream(stream)), "pq2_group_dots")


def pq2_last_device_error(stream=None) -> int:
    return int(_lib.pq2_last_device_error(_stream(stream)))


def pq2_debug_set_wait_limit_ns(ns: int):
    _check(_lib.pq2_debug_set_wait_limit_ns(ns), "pq2_debug_set_wait_limit_ns")


def pq2_debug_skip_stage(stage: int):
    _check(_lib.pq2_debug_skip_stage(stage), "pq2_debug_skip_stage")


def pq2_bounds_checked() -> bool:
    return bool(_lib.pq2_bounds_checked())


def pq2_debug_shrink_bounds(elements: int):
    _check(_lib.pq2_debug_shrink_bounds(elements), "pq2_debug_shrink_bounds")


def pq2_debug_force_kernel(op: int, variant: int):
    _check(_lib.pq2_debug_force_kernel(op, variant), "pq2_debug_force_kernel")


def pq2_debug_gemv_floor(N: int, K: int, flags: int = 0, stream=None):
    """One empty launch shaped like a fused M = 1 call (the latency floor)."""
    _check(_lib.pq2_debug_gemv_floor(N, K, flags, _stream(stream)), "pq2_debug_gemv_floor")


def pq2_debug_mma_rate(n: int, iters: int, cycles, stream=None):
    """cycles: int64 CUDA tensor with (at least) one entry per SM."""
    _dtype(cycles, torch.int64, "cycles")
    sms = torch.cuda.get_device_properties(cycles.device).multi_processor_count
    if cycles.numel() < sms:
        raise ValueError(f"cycles: needs {sms} entries, got {cycles.numel()}")
    _check(_lib.pq2_debug_mma_rate(n, iters, _ptr(cycles), _stream(stream)), "pq2_debug_mma_rate")


class forced_kernel:
    """Context manager: calls of `op` run kernel `variant` inside the block
    (pq2_debug_force_kernel), the library's own routing again after it."""

    def __init__(self, op: int, variant: int):
        self.op, self.variant = op, variant

    def __enter__(self):
        pq2_debug_force_kernel(self.op, self.variant)
        return self

    def __exit__(self, *exc):
        pq2_debug_force_kernel(self.op, PQ2_VARIANT_DEFAULT)
        return False


# ---------------------------------------------------------------------------
# Allocation helpers (torch owns the memory; the library never allocates).
# ---------------------------------------------------------------------------
def alloc_act(M: int, K: int, device="cuda"):
    qp = torch.empty((M, K), dtype=torch.int8, device=device)
    S = torch.empty((M, K // 128), dtype=torch.float32, device=device)
    T = torch.empty((M, K // 128), dtype=torch.int32, device=device)
    return qp, S, T


def alloc_workspace(op: int, M: int, N: int, K: int, device="cuda"):
    n = pq2_workspace_bytes(op, M, N, K)
    if n == SIZE_MAX:
        raise PQ2Error(PQ2_ERR_UNSUPPORTED_SHAPE, "pq2_workspace_bytes")
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)


def pack(tern, ws, stream=None):
    """Convenience: returns (codes, ws_copy) for device tensors tern, ws."""
    N, K = tern.shape
    codes = torch.empty((N, K // 4), dtype=torch.uint8, device=tern.device)
    ws_out = torch.empty_like(ws)
    pq2_pack_weights(tern, ws, codes, ws_out, stream)
    return codes, ws_out


def quantize(x, stream=None):
    M, K = x.shape
    qp, S, T = alloc_act(M, K, x.device)
    pq2_quantize_act(x, qp, S, T, stream)
    return qp, S, T


def matmul_q(qp, S, T, codes, ws, stream=None):
    """Route quantised activations to pq2_gemv / pq2_gemm_small / pq2_gemm_prefill."""
    M, N, K = _mm_shapes(qp, codes)
    y = torch.empty((M, N), dtype=torch.float32, device=qp.device)
    if M == 1:
        pq2_gemv(qp, S, T, codes, ws, y, stream)
    elif M <= 16:
        pq2_gemm_small(qp, S, T, codes, ws, y, alloc_workspace(PQ2_OP_SMALL, M, N, K, qp.device),
                       stream)
    else:
        pq2_gemm_prefill(qp, S, T, codes, ws, y,
                         alloc_workspace(PQ2_OP_PREFILL, M, N, K, qp.device), stream)
    return y
