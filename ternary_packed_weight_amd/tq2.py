"""Thin ctypes binding of libtq2 (include/tq2.h), same names as the C ABI.

Argument marshalling only: every step runs in the library's HIP kernels.
Tensors are torch device tensors; binary16 data (x, scales) may be passed as
torch.float16 (the bit patterns are what crosses the ABI).  Calls enqueue on
torch's current stream unless `stream` is given (the caller then orders that
stream against the ones that write the inputs and read the outputs; what a call
allocates belongs to `stream`), and raise Tq2Error on a non-zero status.  There is no fallback: if libtq2.so is missing the import
fails.  _tq2call.so is a shorter way into the calls around the projections; without it
their checks and marshalling are Python's.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq2.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtq2.so not built at {LIB_PATH}; run __graft_entry__.build()")

# torch is imported first so that libtq2 binds to the HIP runtime torch loaded.
_lib = ctypes.CDLL(LIB_PATH)

try:
    from . import _tq2call  # noqa: E402  (the short way of the attention calls; built beside libtq2)
except ModuleNotFoundError:
    class _tq2call:
        """Answers None to every call: not the plain case, so the binding's own checks decide."""
        bind = bind_step = qk_norm_rope = kv4_store = kv4_load = kv4_attn = staticmethod(lambda *a: None)
        add_rms_norm = add_rms_norm_i8 = gate_up_silu = token_logprobs = staticmethod(lambda *a: None)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_F = ctypes.c_float

_lib.tq2_abi_version.argtypes = []
_lib.tq2_abi_version.restype = _I32
_lib.tq2_status_string.argtypes = [_I32]
_lib.tq2_status_string.restype = ctypes.c_char_p
_lib.tq2_codes_bytes.argtypes = [_I64, _I64]
_lib.tq2_codes_bytes.restype = _SZ
_lib.tq2_scales_bytes.argtypes = [_I64, _I64]
_lib.tq2_scales_bytes.restype = _SZ
_lib.tq2_workspace_bytes.argtypes = [_I32, _I64, _I64]
_lib.tq2_workspace_bytes.restype = _SZ
_lib.tq2_pack.argtypes = [_P, _I64, _I64, _P, _P, _P, _P]
_lib.tq2_pack.restype = _I32
_lib.tq2_dequant.argtypes = [_P, _P, _I64, _I64, _P, _P]
_lib.tq2_dequant.restype = _I32
_lib.tq2_gemv.argtypes = [_P, _P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv.restype = _I32
_lib.tq2_gemv_gate_up.argtypes = [_P, _P, _P, _P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv_gate_up.restype = _I32
_lib.tq2_quantize_i8.argtypes = [_P, _I64, _F, _P, _P]
_lib.tq2_quantize_i8.restype = _I32
_lib.tq2_gemv_i8q.argtypes = [_P, _P, _I64, _I64, _P, _F, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv_i8q.restype = _I32
_lib.tq2_gemv_i8.argtypes = [_P, _P, _I64, _I64, _P, _F, _P, _P, _SZ, _P]
_lib.tq2_gemv_i8.restype = _I32
_lib.tq2_gemv_fused.argtypes = [_I32, _P, _P, _P, _I64, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv_fused.restype = _I32
_lib.tq2_gemv_i8_fused.argtypes = [_I32, _P, _P, _P, _I64, _P, _F, _P, _P, _SZ, _P]
_lib.tq2_gemv_i8_fused.restype = _I32
_lib.tq2_gemv_gate_up_silu.argtypes = [_P, _P, _P, _P, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv_gate_up_silu.restype = _I32
_lib.tq2_gemv_i8_requant.argtypes = [_P, _P, _I64, _I64, _P, _F, _F, _P, _P, _P, _SZ, _P]
_lib.tq2_gemv_i8_requant.restype = _I32
_lib.tq2_gemm_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.tq2_gemm_workspace_bytes.restype = _SZ
_lib.tq2_gemm.argtypes = [_P, _P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P]
_lib.tq2_gemm.restype = _I32
_lib.tq2_gemm_noalloc.argtypes = [_P, _P, _I64, _I64, _P, _I64, _P, _P]
_lib.tq2_gemm_noalloc.restype = _I32
_lib.tq2_gemm_i8q_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.tq2_gemm_i8q_workspace_bytes.restype = _SZ
_lib.tq2_gemm_i8q.argtypes = [_P, _P, _I64, _I64, _P, _I64, _F, _P, _P, _SZ, _P]
_lib.tq2_gemm_i8q.restype = _I32
_lib.tq2_qk_norm_rope.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _I64, _I32, _I32, _I64, _I32, _P, _P, _F, _P, _P,
                                  _I32, _I32, _P, _P, _I32, _P]
_lib.tq2_qk_norm_rope.restype = _I32
_lib.tq2_kv4_page_bytes.argtypes = [_I32, _I32, _I32]
_lib.tq2_kv4_page_bytes.restype = _SZ
_lib.tq2_kv4_store.argtypes = [_P, _I64, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _I32, _P, _I64, _P]
_lib.tq2_kv4_store.restype = _I32
_lib.tq2_kv4_load.argtypes = [_P, _I64, _I32, _I32, _I32, _P, _I64, _P, _P, _I32, _P]
_lib.tq2_kv4_load.restype = _I32
_lib.tq2_kv4_attn_workspace_bytes.argtypes = [_I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32]
_lib.tq2_kv4_attn_workspace_bytes.restype = _SZ
_lib.tq2_kv4_attn.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, _P, _I64, _I32, _I32, _I32, _P, _I64, _I32, _P, _P,
                              _I32, _I32, _F, _I32, _P, _P, _P, _SZ, _P]
_lib.tq2_kv4_attn.restype = _I32
_lib.tq2_add_rms_norm.argtypes = [_P, _I64, _I32, _P, _I64, _I32, _P, _I64, _I32, _P, _F, _P, _I32, _P]
_lib.tq2_add_rms_norm.restype = _I32
_lib.tq2_add_rms_norm_i8.argtypes = [_P, _I64, _I32, _P, _I64, _I32, _P, _I64, _I32, _P, _F, _F, _P, _P, _P]
_lib.tq2_add_rms_norm_i8.restype = _I32
_lib.tq2_gemm_gate_up_silu_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.tq2_gemm_gate_up_silu_workspace_bytes.restype = _SZ
_lib.tq2_gemm_gate_up_silu.argtypes = [_P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _I32, _P, _SZ, _P]
_lib.tq2_gemm_gate_up_silu.restype = _I32
_lib.tq2_gemm_i8q_gate_up_silu_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.tq2_gemm_i8q_gate_up_silu_workspace_bytes.restype = _SZ
_lib.tq2_gemm_i8q_gate_up_silu.argtypes = [_P, _P, _P, _P, _I64, _I64, _P, _I64, _F, _P, _P, _I32, _P, _SZ, _P]
_lib.tq2_gemm_i8q_gate_up_silu.restype = _I32
_lib.tq2_token_logprobs_workspace_bytes.argtypes = [_I64, _I64, _I32]
_lib.tq2_token_logprobs_workspace_bytes.restype = _SZ
_lib.tq2_token_logprobs.argtypes = [_P, _I64, _I32, _I64, _I64, _F, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]
_lib.tq2_token_logprobs.restype = _I32

TQ2_OK = 0
TQ2_OP_GEMV, TQ2_OP_GATE_UP, TQ2_OP_GEMV_I8, TQ2_OP_GEMV_I8Q = 0, 1, 2, 3
EXPORTED = ("tq2_abi_version", "tq2_status_string", "tq2_codes_bytes", "tq2_scales_bytes",
            "tq2_workspace_bytes", "tq2_pack", "tq2_dequant", "tq2_gemv", "tq2_gemv_gate_up",
            "tq2_quantize_i8", "tq2_gemv_i8q", "tq2_gemv_i8", "tq2_gemv_fused", "tq2_gemv_i8_fused",
            "tq2_gemv_gate_up_silu", "tq2_gemv_i8_requant", "tq2_gemm_workspace_bytes", "tq2_gemm",
            "tq2_gemm_i8q_workspace_bytes", "tq2_gemm_i8q", "tq2_gemm_noalloc", "tq2_qk_norm_rope",
            "tq2_kv4_page_bytes", "tq2_kv4_store", "tq2_kv4_load", "tq2_kv4_attn_workspace_bytes", "tq2_kv4_attn",
            "tq2_add_rms_norm", "tq2_add_rms_norm_i8", "tq2_gemm_gate_up_silu_workspace_bytes",
            "tq2_gemm_gate_up_silu", "tq2_gemm_i8q_gate_up_silu_workspace_bytes", "tq2_gemm_i8q_gate_up_silu",
            "tq2_token_logprobs_workspace_bytes", "tq2_token_logprobs")
TQ2_ERR_SCRATCH = 7
TQ2_GEMM_SCRATCH_BYTES = 4194304
TQ2_F16, TQ2_BF16, TQ2_F32 = 0, 1, 2
TQ2_MAX_TOP = 64


_tq2call.bind(*(ctypes.cast(getattr(_lib, f), _P).value for f in (
    "tq2_qk_norm_rope", "tq2_kv4_store", "tq2_kv4_load", "tq2_kv4_attn", "tq2_kv4_attn_workspace_bytes")))
_tq2call.bind_step(*(ctypes.cast(getattr(_lib, f), _P).value for f in (
    "tq2_add_rms_norm", "tq2_add_rms_norm_i8", "tq2_gemm_gate_up_silu", "tq2_gemm_i8q_gate_up_silu",
    "tq2_gemm_gate_up_silu_workspace_bytes", "tq2_gemm_i8q_gate_up_silu_workspace_bytes", "tq2_token_logprobs",
    "tq2_token_logprobs_workspace_bytes")))


class Tq2Error(RuntimeError):
    def __init__(self, fn, status):
        msg = _lib.tq2_status_string(status).decode()
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def lib():
    return _lib


def _check(fn, status):
    if status != TQ2_OK:
        raise Tq2Error(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream, read=True):
    """A new tensor that a call on `stream` (None: the current one) writes.  It
    is allocated under that stream, so its memory was free there before and
    goes back to that stream's work only: a workspace is dropped when the call
    returns, long before its kernels have run.  An output is read by work of
    the current stream later, which the allocator is told of."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if read and t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


_F16_BITS = (torch.float16, torch.int16) + ((torch.uint16,) if hasattr(torch, "uint16") else ())
_DTYPE_NAMES = {torch.uint8: "uint8", torch.int8: "int8", torch.int32: "int32", torch.float32: "float32"}


def _dev(t, name, dtypes=None, numel=None, at_least=False):
    """Check a tensor argument's layout before anything reaches the library:
    dtype (binary16 data may be float16 or 16-bit integer bit patterns),
    element count (exact, or a minimum for workspaces) and contiguity.  The
    C ABI sees pointers only, so a short or mistyped buffer would otherwise
    be read or written past its end.  Where the tensors live is checked last,
    for all of a call's tensors at once (_placed)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if dtypes is not None and t.dtype not in dtypes:
        want = "/".join(_DTYPE_NAMES.get(d, str(d).replace("torch.", "")) for d in dtypes)
        raise ValueError(f"{name} must have dtype {want}, got {t.dtype}")
    if numel is not None:
        n = t.numel()
        if (n < numel) if at_least else (n != numel):
            rel = "at least " if at_least else ""
            raise ValueError(f"{name} must hold {rel}{numel} elements, got {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _placed(**named):
    """Every tensor of the call is on the GPU, and all on one device."""
    devs = set()
    for name, t in named.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        devs.add(t.device)
    if len(devs) > 1:
        raise ValueError(f"all tensors of a call must be on one device, got {sorted(map(str, devs))}")


def tq2_abi_version():
    return int(_lib.tq2_abi_version())


def tq2_status_string(status):
    return _lib.tq2_status_string(int(status)).decode()


def tq2_codes_bytes(N, K):
    return int(_lib.tq2_codes_bytes(N, K))


def tq2_scales_bytes(N, K):
    return int(_lib.tq2_scales_bytes(N, K))


def tq2_workspace_bytes(op, N, K):
    return int(_lib.tq2_workspace_bytes(op, N, K))


def _shape(codes, scales):
    """(N, K) of a packed weight: codes uint8 [N][K/4], scales binary16 with
    N*K/256 elements."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a 2-D [N][K/4] uint8 tensor")
    N, K = codes.shape[0], codes.shape[1] * 4
    _dev(codes, "codes", (torch.uint8,))
    if K % 256:
        raise ValueError(f"codes must be [N][K/4] with K a multiple of 256, got K = {K}")
    _dev(scales, "scales", _F16_BITS, N * (K // 256))
    return N, K


def _ws(ws):
    if ws is not None:
        _dev(ws, "ws")
    return ws


def _mat_tensors(mats):
    out = {}
    for i, (c, s) in enumerate(mats):
        out[f"codes[{i}]"], out[f"scales[{i}]"] = c, s
    return out


def _wsb(ws):
    if ws is None:
        return 0
    return ws.numel() * ws.element_size()


def tq2_pack(W, codes=None, scales=None, bad_blocks=None, stream=None):
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D [N][K] float32 tensor")
    N, K = W.shape
    _dev(W, "W", (torch.float32,))
    if K % 256:
        raise ValueError(f"K must be a multiple of 256, got {K}")
    if codes is None:
        codes = _empty((N, K // 4), torch.uint8, W.device, stream)
    if scales is None:
        scales = _empty((N, K // 256), torch.float16, W.device, stream)
    if bad_blocks is None:
        bad_blocks = _empty(1, torch.int32, W.device, stream)
    _dev(codes, "codes", (torch.uint8,), N * (K // 4))
    _dev(scales, "scales", _F16_BITS, N * (K // 256))
    _dev(bad_blocks, "bad_blocks", (torch.int32,), 1, at_least=True)
    _placed(W=W, codes=codes, scales=scales, bad_blocks=bad_blocks)
    _check("tq2_pack", _lib.tq2_pack(_ptr(W), N, K, _ptr(codes), _ptr(scales), _ptr(bad_blocks),
                                     _stream(stream)))
    return codes, scales, bad_blocks


def tq2_dequant(codes, scales, W=None, stream=None):
    N, K = _shape(codes, scales)
    if W is None:
        W = _empty((N, K), torch.float32, codes.device, stream)
    _dev(W, "W", (torch.float32,), N * K)
    _placed(codes=codes, scales=scales, W=W)
    _check("tq2_dequant", _lib.tq2_dequant(_ptr(codes), _ptr(scales), N, K, _ptr(W), _stream(stream)))
    return W


def _out(t, name, numel, dtype, device, stream):
    """An output buffer: allocated when not given, else checked."""
    if t is None:
        return _empty(numel, dtype, device, stream)
    return _dev(t, name, (dtype,), numel)


def tq2_gemv(codes, scales, x, y=None, ws=None, stream=None):
    N, K = _shape(codes, scales)
    _dev(x, "x", _F16_BITS, K)
    y = _out(y, "y", N, torch.float32, codes.device, stream)
    _placed(codes=codes, scales=scales, x=x, y=y, ws=_ws(ws))
    _check("tq2_gemv", _lib.tq2_gemv(_ptr(codes), _ptr(scales), N, K, _ptr(x), _ptr(y), _ptr(ws),
                                     _wsb(ws), _stream(stream)))
    return y


def tq2_gemv_gate_up(codes_g, scales_g, codes_u, scales_u, x, y=None, ws=None, stream=None):
    N, K = _shape(codes_g, scales_g)
    if _shape(codes_u, scales_u) != (N, K):
        raise ValueError("gate and up must have the same shape")
    _dev(x, "x", _F16_BITS, K)
    y = _out(y, "y", 2 * N, torch.float32, codes_g.device, stream)
    _placed(codes_g=codes_g, scales_g=scales_g, codes_u=codes_u, scales_u=scales_u, x=x, y=y, ws=_ws(ws))
    _check("tq2_gemv_gate_up", _lib.tq2_gemv_gate_up(
        _ptr(codes_g), _ptr(scales_g), _ptr(codes_u), _ptr(scales_u), N, K, _ptr(x), _ptr(y),
        _ptr(ws), _wsb(ws), _stream(stream)))
    return y.view(2, N)


def tq2_quantize_i8(x, s, x_q=None, stream=None):
    _dev(x, "x", _F16_BITS)
    K = x.numel()
    x_q = _out(x_q, "x_q", K, torch.int8, x.device, stream)
    _placed(x=x, x_q=x_q)
    _check("tq2_quantize_i8", _lib.tq2_quantize_i8(_ptr(x), K, float(s), _ptr(x_q), _stream(stream)))
    return x_q.view(x.shape)


def _workspace(op, N, K, ws, device, stream):
    need = tq2_workspace_bytes(op, N, K)
    if ws is None and need not in (0, 2 ** 64 - 1):
        ws = _empty(need, torch.uint8, device, stream, read=False)
    return ws, _wsb(ws)


def tq2_gemv_i8q(codes, scales, x_q, s, y=None, partials=None, ws=None, stream=None):
    N, K = _shape(codes, scales)
    _dev(x_q, "x_q", (torch.int8,), K)
    y = _out(y, "y", N, torch.float32, codes.device, stream)
    if partials is not None:
        _dev(partials, "partials", (torch.int32,), N * (K // 256))
    ws, wsb = _workspace(TQ2_OP_GEMV_I8Q, N, K, ws, codes.device, stream)
    _placed(codes=codes, scales=scales, x_q=x_q, y=y, partials=partials, ws=_ws(ws))
    _check("tq2_gemv_i8q", _lib.tq2_gemv_i8q(_ptr(codes), _ptr(scales), N, K, _ptr(x_q), float(s),
                                             _ptr(y), _ptr(partials), _ptr(ws), wsb, _stream(stream)))
    return y


def tq2_gemv_i8(codes, scales, x, s, y=None, ws=None, stream=None):
    N, K = _shape(codes, scales)
    _dev(x, "x", _F16_BITS, K)
    y = _out(y, "y", N, torch.float32, codes.device, stream)
    ws, wsb = _workspace(TQ2_OP_GEMV_I8, N, K, ws, codes.device, stream)
    _placed(codes=codes, scales=scales, x=x, y=y, ws=_ws(ws))
    _check("tq2_gemv_i8", _lib.tq2_gemv_i8(_ptr(codes), _ptr(scales), N, K, _ptr(x), float(s),
                                           _ptr(y), _ptr(ws), wsb, _stream(stream)))
    return y


def _host_arrays(mats):
    """Host pointer/size arrays for the fused entry points: mats is a list
    of (codes, scales) device tensors sharing K."""
    if not 1 <= len(mats) <= 3:
        raise ValueError("1 to 3 matrices")
    shapes = [_shape(c, s) for c, s in mats]
    K = shapes[0][1]
    if any(k != K for _, k in shapes):
        raise ValueError("fused matrices must share K")
    n = len(mats)
    cp = (ctypes.c_void_p * n)(*[c.data_ptr() for c, _ in mats])
    sp = (ctypes.c_void_p * n)(*[s.data_ptr() for _, s in mats])
    Np = (ctypes.c_int64 * n)(*[N for N, _ in shapes])
    return n, cp, sp, Np, [N for N, _ in shapes], K


def tq2_gemv_fused(mats, x, y=None, ws=None, stream=None):
    """y = concatenation of W_i x over mats = [(codes_i, scales_i), ...]."""
    n, cp, sp, Np, Ns, K = _host_arrays(mats)
    _dev(x, "x", _F16_BITS, K)
    y = _out(y, "y", sum(Ns), torch.float32, x.device, stream)
    _placed(x=x, y=y, ws=_ws(ws), **_mat_tensors(mats))
    _check("tq2_gemv_fused", _lib.tq2_gemv_fused(n, cp, sp, Np, K, _ptr(x), _ptr(y), _ptr(ws), _wsb(ws),
                                                 _stream(stream)))
    return y


def tq2_gemv_i8_fused(mats, x, s, y=None, ws=None, stream=None):
    n, cp, sp, Np, Ns, K = _host_arrays(mats)
    _dev(x, "x", _F16_BITS, K)
    y = _out(y, "y", sum(Ns), torch.float32, x.device, stream)
    _placed(x=x, y=y, ws=_ws(ws), **_mat_tensors(mats))
    _check("tq2_gemv_i8_fused", _lib.tq2_gemv_i8_fused(n, cp, sp, Np, K, _ptr(x), float(s), _ptr(y),
                                                       _ptr(ws), _wsb(ws), _stream(stream)))
    return y


def tq2_gemv_gate_up_silu(codes_g, scales_g, codes_u, scales_u, x, h=None, ws=None, stream=None):
    N, K = _shape(codes_g, scales_g)
    if _shape(codes_u, scales_u) != (N, K):
        raise ValueError("gate and up must have the same shape")
    _dev(x, "x", _F16_BITS, K)
    h = _out(h, "h", N, torch.float32, codes_g.device, stream)
    _placed(codes_g=codes_g, scales_g=scales_g, codes_u=codes_u, scales_u=scales_u, x=x, h=h, ws=_ws(ws))
    _check("tq2_gemv_gate_up_silu", _lib.tq2_gemv_gate_up_silu(
        _ptr(codes_g), _ptr(scales_g), _ptr(codes_u), _ptr(scales_u), N, K, _ptr(x), _ptr(h),
        _ptr(ws), _wsb(ws), _stream(stream)))
    return h


def tq2_gemv_i8_requant(codes, scales, x, s_in, s_out, y_q=None, y_deq=None, want_deq=True,
                        ws=None, stream=None):
    N, K = _shape(codes, scales)
    _dev(x, "x", _F16_BITS, K)
    y_q = _out(y_q, "y_q", N, torch.int8, codes.device, stream)
    if y_deq is not None or want_deq:
        y_deq = _out(y_deq, "y_deq", N, torch.float32, codes.device, stream)
    _placed(codes=codes, scales=scales, x=x, y_q=y_q, y_deq=y_deq, ws=_ws(ws))
    _check("tq2_gemv_i8_requant", _lib.tq2_gemv_i8_requant(
        _ptr(codes), _ptr(scales), N, K, _ptr(x), float(s_in), float(s_out), _ptr(y_q), _ptr(y_deq),
        _ptr(ws), _wsb(ws), _stream(stream)))
    return y_q, y_deq


def tq2_gemm_workspace_bytes(N, K, M):
    return int(_lib.tq2_gemm_workspace_bytes(N, K, M))


def tq2_gemm(codes, scales, x, y=None, ws=None, stream=None):
    """Y[M][N] = X[M][K] W^T for x of shape [M, K] (fp16); allocates the
    workspace when none is given."""
    N, K = _shape(codes, scales)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be a [M, {K}] tensor")
    M = x.shape[0]
    _dev(x, "x", _F16_BITS, M * K)
    y = _out(y, "y", M * N, torch.float32, codes.device, stream)
    need = tq2_gemm_workspace_bytes(N, K, M)
    if ws is None and need and need != 2 ** 64 - 1:
        ws = _empty(need, torch.uint8, codes.device, stream, read=False)
    if ws is not None and need and need != 2 ** 64 - 1:
        _dev(ws, "ws", None, need // ws.element_size(), at_least=True)
    _placed(codes=codes, scales=scales, x=x, y=y, ws=ws)
    _check("tq2_gemm", _lib.tq2_gemm(_ptr(codes), _ptr(scales), N, K, _ptr(x), M, _ptr(y), _ptr(ws), _wsb(ws),
                                      _stream(stream)))
    return y.view(M, N)


def tq2_gemm_i8q_workspace_bytes(N, K, M):
    return int(_lib.tq2_gemm_i8q_workspace_bytes(N, K, M))


def tq2_gemm_i8q(codes, scales, x_q, s, y=None, ws=None, stream=None):
    """Y[M][N]: the int8 matvec of every row of x_q (shape [M, K], int8,
    quantized with s); allocates the workspace when none is given."""
    N, K = _shape(codes, scales)
    if not isinstance(x_q, torch.Tensor) or x_q.dim() != 2 or x_q.shape[1] != K:
        raise ValueError(f"x_q must be a [M, {K}] tensor")
    M = x_q.shape[0]
    _dev(x_q, "x_q", (torch.int8,), M * K)
    y = _out(y, "y", M * N, torch.float32, codes.device, stream)
    need = tq2_gemm_i8q_workspace_bytes(N, K, M)
    if ws is None and need and need != 2 ** 64 - 1:
        ws = _empty(need, torch.uint8, codes.device, stream, read=False)
    if ws is not None and need and need != 2 ** 64 - 1:
        _dev(ws, "ws", None, need // ws.element_size(), at_least=True)
    _placed(codes=codes, scales=scales, x_q=x_q, y=y, ws=ws)
    _check("tq2_gemm_i8q", _lib.tq2_gemm_i8q(_ptr(codes), _ptr(scales), N, K, _ptr(x_q), M, float(s), _ptr(y),
                                              _ptr(ws), _wsb(ws), _stream(stream)))
    return y.view(M, N)


def tq2_gemm_noalloc(codes, scales, x, y=None, stream=None):
    """tq2_gemm with the split partials in the library's static scratch (no
    workspace argument, nothing allocated by the library; y is allocated
    here only when not given)."""
    N, K = _shape(codes, scales)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be a [M, {K}] tensor")
    M = x.shape[0]
    _dev(x, "x", _F16_BITS, M * K)
    y = _out(y, "y", M * N, torch.float32, codes.device, stream)
    _placed(codes=codes, scales=scales, x=x, y=y)
    _check("tq2_gemm_noalloc", _lib.tq2_gemm_noalloc(_ptr(codes), _ptr(scales), N, K, _ptr(x), M, _ptr(y),
                                                      _stream(stream)))
    return y.view(M, N)


# ---- the attention half of a decode step ----
#
# A call whose arguments are the plain case (every output given) goes through
# _tq2call, which checks and marshals them in native code; it answers None
# where they are not, and the checks below decide.

_TQ2_DTYPE = {torch.float16: TQ2_F16, torch.bfloat16: TQ2_BF16, torch.float32: TQ2_F32}
_HEAD_TYPES = tuple(_TQ2_DTYPE)


def _heads(t, name, dtypes=_HEAD_TYPES):
    """[T, H, D] heads: their shape and the strides of tokens and heads.  The
    D elements of a head are contiguous; tokens and heads may be strided (a
    slice of a q/k/v output)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [T, heads, D] tensor")
    if t.dtype not in dtypes:
        want = "/".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must have dtype {want}, got {t.dtype}")
    T, H, D = t.shape
    ts, hs, ds = t.stride()
    if ds != 1 and D > 1:
        raise ValueError(f"the channels of a head of {name} must be contiguous")
    return T, H, D, ts, hs


def _cache(cache, D):
    """(pages, P, Hk) of a cache [pages, Hk, P*(D+8)]."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3:
        raise ValueError("cache must be a [pages, heads, P*(D+8)] uint8 tensor")
    _dev(cache, "cache", (torch.uint8,))
    pages, Hk, block = cache.shape
    if D < 1 or block % (D + 8):
        raise ValueError(f"cache blocks of {block} bytes hold no whole number of tokens of {D} channels")
    return pages, block // (D + 8), Hk


def _short(fn, status):
    """Whether the short way has made the call; raises on its status."""
    if status is None:
        return False
    _check(fn, status)
    return True


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def tq2_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                     out_dtype=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [T, Hq, D] and k [T, Hk, D] (where a weight
    [D] is given) and their rotation by positions [T] (int32) * inv_freq
    [rot/2] (float32).  Returns (q_out, k_out), contiguous, of out_dtype
    (default: the type of the given output, else that of q)."""
    if out_dtype is None and _short("tq2_qk_norm_rope", _tq2call.qk_norm_rope(
            q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, _handle(stream))):
        return q_out, k_out
    T, Hq, D, qts, qhs = _heads(q, "q")
    Tk, Hk, Dk, kts, khs = _heads(k, "k")
    if (Tk, Dk) != (T, D) or k.dtype != q.dtype:
        raise ValueError("q and k must have the same tokens, head size and dtype")
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else k_out.dtype if k_out is not None else q.dtype
    if out_dtype not in _TQ2_DTYPE:
        raise ValueError(f"out_dtype must be float16/bfloat16/float32, got {out_dtype}")
    _dev(positions, "positions", (torch.int32,), T)
    _dev(inv_freq, "inv_freq", (torch.float32,))
    if q_weight is not None:
        _dev(q_weight, "q_weight", (torch.float32,), D)
    if k_weight is not None:
        _dev(k_weight, "k_weight", (torch.float32,), D)
    q_out = _out(q_out, "q_out", T * Hq * D, out_dtype, q.device, stream)
    k_out = _out(k_out, "k_out", T * Hk * D, out_dtype, q.device, stream)
    _placed(q=q, k=k, positions=positions, inv_freq=inv_freq, q_weight=q_weight, k_weight=k_weight, q_out=q_out,
            k_out=k_out)
    _check("tq2_qk_norm_rope", _lib.tq2_qk_norm_rope(
        _ptr(q), qts, qhs, Hq, _ptr(k), kts, khs, Hk, _TQ2_DTYPE[q.dtype], T, D, _ptr(q_weight), _ptr(k_weight),
        float(eps), _ptr(positions), _ptr(inv_freq), 2 * inv_freq.numel(), int(bool(interleaved)), _ptr(q_out),
        _ptr(k_out), _TQ2_DTYPE[out_dtype], _stream(stream)))
    return q_out.view(T, Hq, D), k_out.view(T, Hk, D)


def tq2_kv4_page_bytes(P, Hk, D):
    return int(_lib.tq2_kv4_page_bytes(P, Hk, D))


def tq2_kv4_store(cache, k, v, slots, stream=None):
    """Quantizes k and v [T, Hk, D] into the slots (int64 [T]; page*P + place)
    of cache [pages, Hk, P*(D+8)] (uint8)."""
    if _short("tq2_kv4_store", _tq2call.kv4_store(cache, k, v, slots, _handle(stream))):
        return cache
    T, Hk, D, kts, khs = _heads(k, "k")
    Tv, Hv, Dv, vts, vhs = _heads(v, "v")
    if (Tv, Hv, Dv) != (T, Hk, D) or v.dtype != k.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    pages, P, heads = _cache(cache, D)
    if heads != Hk:
        raise ValueError(f"cache has {heads} heads, k and v have {Hk}")
    _dev(slots, "slots", (torch.int64,), T)
    _placed(cache=cache, k=k, v=v, slots=slots)
    _check("tq2_kv4_store", _lib.tq2_kv4_store(_ptr(cache), pages, P, Hk, D, _ptr(k), kts, khs, _ptr(v), vts, vhs,
                                               _TQ2_DTYPE[k.dtype], _ptr(slots), T, _stream(stream)))
    return cache


def tq2_kv4_load(cache, slots, D, dtype=None, k_out=None, v_out=None, stream=None):
    """The keys and values [T, Hk, D] that the slots (int64 [T]) hold, of
    dtype (default: that of the given outputs, else float16)."""
    if dtype is None and _short("tq2_kv4_load", _tq2call.kv4_load(cache, slots, D, k_out, v_out, _handle(stream))):
        return k_out, v_out
    pages, P, Hk = _cache(cache, D)
    _dev(slots, "slots", (torch.int64,))
    T = slots.numel()
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else torch.float16
    if dtype not in _TQ2_DTYPE:
        raise ValueError(f"dtype must be float16/bfloat16/float32, got {dtype}")
    k_out = _out(k_out, "k_out", T * Hk * D, dtype, cache.device, stream)
    v_out = _out(v_out, "v_out", T * Hk * D, dtype, cache.device, stream)
    _placed(cache=cache, slots=slots, k_out=k_out, v_out=v_out)
    _check("tq2_kv4_load", _lib.tq2_kv4_load(_ptr(cache), pages, P, Hk, D, _ptr(slots), T, _ptr(k_out), _ptr(v_out),
                                             _TQ2_DTYPE[dtype], _stream(stream)))
    return k_out.view(T, Hk, D), v_out.view(T, Hk, D)


def tq2_kv4_attn_workspace_bytes(T, Hq, Hk, D, P, table_width, B, max_q):
    return int(_lib.tq2_kv4_attn_workspace_bytes(T, Hq, Hk, D, P, table_width, B, max_q))


def tq2_kv4_attn(q, cache, table, ctx_len, q_start=None, max_q=None, scale=None, window=0, out=None, lse=None,
                 ws=None, stream=None):
    """Causal attention of the new tokens q [T, Hq, D] over the cache.  table
    int32 [B, width], ctx_len int32 [B] (cached tokens, the new ones among
    them), q_start int32 [B+1] with max_q the most new tokens of a sequence
    (neither: T/B tokens each; T is at most B*max_q), scale default 1/sqrt(D), window 0 for none;
    lse float32 [T, Hq] is written when given.  Returns out [T, Hq, D] of q's
    dtype; allocates the workspace when none is given."""
    if _short("tq2_kv4_attn", _tq2call.kv4_attn(q, cache, table, ctx_len, q_start, max_q, scale, window, out, lse, ws,
                                                _handle(stream))):
        return out
    T, Hq, D, qts, qhs = _heads(q, "q", _HEAD_TYPES[:2])
    pages, P, Hk = _cache(cache, D)
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.dtype != torch.int32:
        raise ValueError("table must be a [B, width] int32 tensor")
    B, width = table.shape
    if width > 1 and table.stride(1) != 1:
        raise ValueError("the rows of table must be contiguous")
    _dev(ctx_len, "ctx_len", (torch.int32,), B)
    if q_start is not None:
        _dev(q_start, "q_start", (torch.int32,), B + 1)
        if max_q is None:
            raise ValueError("q_start needs max_q, the most new tokens of a sequence")
    elif max_q is None or max_q * B != T:
        if max_q is not None or B < 1 or T % B:
            raise ValueError(f"{T} rows of q are not max_q tokens of each of {B} sequences")
        max_q = max(1, T // B)
    out = _out(out, "out", T * Hq * D, q.dtype, q.device, stream)
    if lse is not None:
        _dev(lse, "lse", (torch.float32,), T * Hq)
    need = int(_lib.tq2_kv4_attn_workspace_bytes(T, Hq, Hk, D, P, width, B, max_q))
    if need and need != 2 ** 64 - 1:
        if ws is None:
            ws = _empty(need, torch.uint8, q.device, stream, read=False)
        else:
            _dev(ws, "ws", None, -(-need // ws.element_size()), at_least=True)
    _placed(q=q, cache=cache, table=table, ctx_len=ctx_len, q_start=q_start, out=out, lse=lse, ws=ws)
    _check("tq2_kv4_attn", _lib.tq2_kv4_attn(
        _ptr(q), qts, qhs, T, Hq, _TQ2_DTYPE[q.dtype], _ptr(cache), pages, P, Hk, D, _ptr(table), table.stride(0),
        width, _ptr(ctx_len), _ptr(q_start), B, max_q, float(D ** -0.5 if scale is None else scale), int(window),
        _ptr(out), _ptr(lse), _ptr(ws), _wsb(ws), _stream(stream)))
    return out.view(T, Hq, D)


# ---- the feed-forward half of a decode step, and the answer ----
#
# As above, the plain case goes through _tq2call.


def _here(stream, **named):
    """The tensors' place, which has to be the current device (calls run on its streams), and the stream."""
    _placed(**named)
    dev = next(t.device for t in named.values() if t is not None)
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    return _stream(stream)


def _rows(t, name, D=None):
    """[T, D] rows of a floating type: their shape and row stride.  The
    elements of a row are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or (D is not None and t.shape[1] != D):
        raise ValueError(f"{name} must be a [T, {D or 'D'}] tensor")
    if t.dtype not in _TQ2_DTYPE:
        raise ValueError(f"{name} must have dtype float16/bfloat16/float32, got {t.dtype}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return t.shape[0], t.shape[1], t.stride(0)


def _norm_inputs(x, residual, weight, h_out, stream):
    """The checks that both norms share; h_out, allocated when a residual is given without one."""
    T, D, _ = _rows(x, "x")
    if weight is not None:
        _dev(weight, "weight", (torch.float32,), D)
    if residual is None:
        if h_out is not None:
            raise ValueError("h_out needs a residual")
        return T, D, None
    if _rows(residual, "residual", D)[0] != T:
        raise ValueError(f"residual must hold {T} rows")
    if h_out is None:
        h_out = _empty((T, D), residual.dtype, residual.device, stream)
        if T > 1 and residual.stride(0) != D:  # of the residual's row stride
            raise ValueError("a residual with strided rows needs an h_out with the same ones")
    elif _rows(h_out, "h_out", D)[0] != T or h_out.dtype != residual.dtype:
        raise ValueError("h_out must have the shape and dtype of the residual")
    elif T > 1 and h_out.stride(0) != residual.stride(0):
        raise ValueError("h_out must have the row stride of the residual")
    return T, D, h_out


def _norm_args(x, residual, h_out, T, D, weight, eps):
    r = (None, 0, 0) if residual is None else (_ptr(residual), residual.stride(0), _TQ2_DTYPE[residual.dtype])
    return (_ptr(x), x.stride(0), _TQ2_DTYPE[x.dtype], *r, _ptr(h_out), T, D, _ptr(weight), float(eps))


def tq2_add_rms_norm(x, residual=None, weight=None, eps=1e-6, out_dtype=None, h_out=None, out=None, stream=None):
    """h = residual + x (rounded to the residual's type; x alone without one),
    out = h / sqrt(mean(h^2) + eps) * weight over rows [T, D].  weight float32
    [D]; out contiguous, of out_dtype (default: the type of the given out, else
    float16); h_out may be the residual itself.  Returns (out, h_out), the
    latter None without a residual."""
    if out_dtype is None and _short("tq2_add_rms_norm", _tq2call.add_rms_norm(
            x, residual, weight, eps, h_out, out, _handle(stream))):
        return out, h_out
    T, D, h_out = _norm_inputs(x, residual, weight, h_out, stream)
    if out_dtype is None:
        out_dtype = torch.float16 if out is None else out.dtype
    if out_dtype not in _TQ2_DTYPE:
        raise ValueError(f"out_dtype must be float16/bfloat16/float32, got {out_dtype}")
    out = _out(out, "out", T * D, out_dtype, x.device, stream)
    st = _here(stream, x=x, residual=residual, weight=weight, h_out=h_out, out=out)
    _check("tq2_add_rms_norm", _lib.tq2_add_rms_norm(*_norm_args(x, residual, h_out, T, D, weight, eps), _ptr(out),
                                                     _TQ2_DTYPE[out_dtype], st))
    return out.view(T, D), h_out


def tq2_add_rms_norm_i8(x, residual=None, weight=None, eps=1e-6, s=None, h_out=None, x_q=None, x_scales=None,
                        stream=None):
    """tq2_add_rms_norm into int8 codes: with the scale s, or (s None) with a
    scale for each row, written to x_scales (float32 [T]).  Returns (x_q [T, D],
    x_scales, h_out), x_scales None where s is given."""
    if _short("tq2_add_rms_norm_i8", _tq2call.add_rms_norm_i8(
            x, residual, weight, eps, h_out, s, x_q, x_scales, _handle(stream))):
        return x_q, x_scales, h_out
    T, D, h_out = _norm_inputs(x, residual, weight, h_out, stream)
    x_q = _out(x_q, "x_q", T * D, torch.int8, x.device, stream)
    if s is None:
        x_scales = _out(x_scales, "x_scales", T, torch.float32, x.device, stream)
    elif x_scales is not None:
        raise ValueError("x_scales is written where no scale s is given")
    elif not float(s) > 0.0:
        raise Tq2Error("tq2_add_rms_norm_i8", 5)
    st = _here(stream, x=x, residual=residual, weight=weight, h_out=h_out, x_q=x_q, x_scales=x_scales)
    _check("tq2_add_rms_norm_i8", _lib.tq2_add_rms_norm_i8(
        *_norm_args(x, residual, h_out, T, D, weight, eps), 0.0 if s is None else float(s), _ptr(x_q), _ptr(x_scales),
        st))
    return x_q.view(T, D), x_scales, h_out


def tq2_gemm_gate_up_silu_workspace_bytes(N, K, M):
    return int(_lib.tq2_gemm_gate_up_silu_workspace_bytes(N, K, M))


def tq2_gemm_i8q_gate_up_silu_workspace_bytes(N, K, M):
    return int(_lib.tq2_gemm_i8q_gate_up_silu_workspace_bytes(N, K, M))


def _gated(fn, codes_g, scales_g, codes_u, scales_u, x, x_types, s, out_dtype, h, ws, stream):
    if out_dtype is None and _short(fn, _tq2call.gate_up_silu(codes_g, scales_g, codes_u, scales_u, x, s, h, ws,
                                                              _handle(stream))):
        return h
    N, K = _shape(codes_g, scales_g)
    if _shape(codes_u, scales_u) != (N, K):
        raise ValueError("gate and up must have the same shape")
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be a [M, {K}] tensor")
    M = x.shape[0]
    _dev(x, "x", x_types, M * K)
    if out_dtype is None:
        out_dtype = torch.float16 if h is None else h.dtype
    if out_dtype not in _TQ2_DTYPE:
        raise ValueError(f"out_dtype must be float16/bfloat16/float32, got {out_dtype}")
    token = isinstance(s, torch.Tensor)
    if token:
        _dev(s, "s", (torch.float32,), M)
    h = _out(h, "h", M * N, out_dtype, codes_g.device, stream)
    need = int(getattr(_lib, fn + "_workspace_bytes")(N, K, M))
    if need and need != 2 ** 64 - 1:
        if ws is None:
            ws = _empty(need, torch.uint8, codes_g.device, stream, read=False)
        else:
            _dev(ws, "ws", None, -(-need // ws.element_size()), at_least=True)
    st = _here(stream, codes_g=codes_g, scales_g=scales_g, codes_u=codes_u, scales_u=scales_u, x=x,
               s=s if token else None, h=h, ws=ws)
    scale = () if s is None else (0.0, _ptr(s)) if token else (float(s), None)
    if scale and not token and not scale[0] > 0.0:
        raise Tq2Error(fn, 5)
    _check(fn, getattr(_lib, fn)(_ptr(codes_g), _ptr(scales_g), _ptr(codes_u), _ptr(scales_u), N, K, _ptr(x), M, *scale,
                                 _ptr(h), _TQ2_DTYPE[out_dtype], _ptr(ws), _wsb(ws), st))
    return h.view(M, N)


def tq2_gemm_gate_up_silu(codes_g, scales_g, codes_u, scales_u, x, out_dtype=None, h=None, ws=None, stream=None):
    """h [M, N] = silu(X Wg^T) * (X Wu^T) for x [M, K] (fp16), of out_dtype
    (default: the type of the given h, else float16); allocates the workspace
    when none is given."""
    return _gated("tq2_gemm_gate_up_silu", codes_g, scales_g, codes_u, scales_u, x, _F16_BITS, None, out_dtype, h, ws,
                  stream)


def tq2_gemm_i8q_gate_up_silu(codes_g, scales_g, codes_u, scales_u, x_q, s, out_dtype=None, h=None, ws=None,
                              stream=None):
    """The same for x_q [M, K] (int8) with the scale s, a number or a float32
    tensor [M] with a scale for each token."""
    if s is None:
        raise ValueError("s must be a number or a float32 tensor [M]")
    return _gated("tq2_gemm_i8q_gate_up_silu", codes_g, scales_g, codes_u, scales_u, x_q, (torch.int8,), s, out_dtype, h,
                  ws, stream)


def tq2_token_logprobs_workspace_bytes(T, V, top):
    return int(_lib.tq2_token_logprobs_workspace_bytes(T, V, top))


def tq2_token_logprobs(logits, tokens=None, top=0, scale=1.0, want_entropy=False, logprobs=None, entropy=None,
                       top_tokens=None, top_logprobs=None, ws=None, stream=None):
    """Of rows logits [T, V]: the log probabilities of tokens (int64 [T]; 0 for
    one outside 0 .. V-1), the entropy (where it is wanted or given a place), and
    the `top` likeliest tokens (int64 [T, top], lowest first of equals) with
    theirs, of softmax(scale * logits).
    Returns (logprobs, entropy, top_tokens, top_logprobs), None for what is not
    asked for; allocates the workspace when none is given."""
    if (entropy is not None or not want_entropy) and _short("tq2_token_logprobs", _tq2call.token_logprobs(
            logits, tokens, top, scale, logprobs, entropy, top_tokens, top_logprobs, ws, _handle(stream))):
        return logprobs, entropy, top_tokens, top_logprobs
    T, V, stride = _rows(logits, "logits")
    dev = logits.device
    if top < 0:
        raise ValueError(f"top must not be negative, got {top}")
    if tokens is not None:
        _dev(tokens, "tokens", (torch.int64,), T)
        logprobs = _out(logprobs, "logprobs", T, torch.float32, dev, stream)
    elif logprobs is not None:
        raise ValueError("logprobs needs tokens")
    if entropy is not None or want_entropy:
        entropy = _out(entropy, "entropy", T, torch.float32, dev, stream)
    if top:
        top_tokens = _out(top_tokens, "top_tokens", T * top, torch.int64, dev, stream)
        top_logprobs = _out(top_logprobs, "top_logprobs", T * top, torch.float32, dev, stream)
    elif top_tokens is not None or top_logprobs is not None:
        raise ValueError("top_tokens and top_logprobs need top > 0")
    need = tq2_token_logprobs_workspace_bytes(T, V, top)
    if need and need != 2 ** 64 - 1:
        if ws is None:
            ws = _empty(need, torch.uint8, dev, stream, read=False)
        else:
            _dev(ws, "ws", None, -(-need // ws.element_size()), at_least=True)
    st = _here(stream, logits=logits, tokens=tokens, logprobs=logprobs, entropy=entropy, top_tokens=top_tokens,
               top_logprobs=top_logprobs, ws=ws)
    _check("tq2_token_logprobs", _lib.tq2_token_logprobs(
        _ptr(logits), stride, _TQ2_DTYPE[logits.dtype], T, V, float(scale), _ptr(tokens), _ptr(logprobs), _ptr(entropy),
        top, _ptr(top_tokens), _ptr(top_logprobs), _ptr(ws), _wsb(ws), st))
    return (logprobs, entropy, top_tokens.view(T, top) if top else None, top_logprobs.view(T, top) if top else None)
