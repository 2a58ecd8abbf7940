"""ctypes binding of libqgemm.so (the C ABI declared in include/qgemm.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels. PyTorch tensors provide device memory and the current stream.
If the shared library is missing this module raises -- there is no fallback.
"""
import ctypes
import functools
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(HERE, "libqgemm.so")
HEADER = os.path.join(HERE, "..", "include", "qgemm.h")

QG_OK, QG_EINVAL, QG_EALIGN, QG_EUNSUPPORTED, QG_ECUDA, QG_ETIMEOUT, QG_ERANGE = range(7)
QG_BF16, QG_F32 = 0, 1
QG_PATH_AUTO, QG_PATH_SMALL, QG_PATH_LARGE = 0, 1, 2
PATHS = {"auto": QG_PATH_AUTO, "small": QG_PATH_SMALL, "large": QG_PATH_LARGE}

_lib = None


class QGError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s (%s)" % (msg, status))
        self.status = status


def load():
    """Load libqgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(SO_PATH):
        raise RuntimeError("libqgemm.so is not built: run `python -m bit_quantized_gemm_gb300.build` "
                           "(or __graft_entry__.build()); there is no CPU fallback")
    L = ctypes.CDLL(SO_PATH)
    P, I64, I, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "qg_status_string": ([I], ctypes.c_char_p),
        "qg_last_error": ([], ctypes.c_char_p),
        "qg_version": ([], I),
        "qg_small_m_max": ([], I64),
        "qg_check_device_error": ([P], I),
        "qg_quantize_act": ([P, I, I64, I64, I64, P, P, P, P, P], I),
        "qg_quantize_act_static": ([P, I, I64, I64, I64, P, I64, P, P, P, P], I),
        "qg_q8_0_packed_bytes": ([I64, I64], SZ),
        "qg_pack_q8_0": ([P, I64, I64, P, P], I),
        "qg_gemm_w8a8_q8_0": ([P, P, P, I64, I64, P, I64, P, I, I64, P], I),
        "qg_gemm_w8a8_q8_0_ex": ([P, P, P, I64, I64, P, I64, P, I, I64, I, P], I),
        "qg_q4k_packed_bytes": ([I64, I64], SZ),
        "qg_pack_q4k": ([P, I64, I64, P, P], I),
        "qg_gemm_w4a8_q4k": ([P, P, P, P, I64, I64, P, I64, P, I, I64, P], I),
        "qg_gemm_w4a8_q4k_ex": ([P, P, P, P, I64, I64, P, I64, P, I, I64, I, P], I),
        "qg_debug_block_sums_q8_0": ([P, P, I64, I64, P, I64, P, I, P], I),
        "qg_debug_block_sums_q4k": ([P, P, I64, I64, P, I64, P, I, P], I),
        "qg_debug_wait_timeout": ([ctypes.c_uint32, P], I),
        "qg_gemm_launch_count": ([I, I64, I64, I64, I], I),
        "qg_linear_workspace_bytes": ([I, I64, I64], SZ),
        "qg_debug_prefill_plan_q8_0": ([I64, I64, I, P, P, P], I),
        "qg_debug_prefill_tile_q4k": ([I64, I64, I, P, P], I),
        "qg_debug_gemm_fp8_tile": ([I64, I64, I, P, P], I),
        "qg_debug_gemm_fp8_grouped_tile": ([I64, I64, I64, I, P, P], I),
        "qg_debug_logprobs_pieces": ([I64, I64, I, P], I),
        "qg_linear_w8a8_q8_0": ([P, I, I64, I64, I64, P, I64, P, I, I64, P, P, SZ, P], I),
        "qg_linear_w4a8_q4k": ([P, I, I64, I64, I64, P, I64, P, I, I64, P, P, SZ, P], I),
        "qg_linear_w8a8_q8_0_noalloc": ([P, I, I64, I64, I64, P, I64, P, I, I64, P, P], I),
        "qg_mxfp4_packed_bytes": ([I64, I64], SZ),
        "qg_pack_mxfp4_q8_0": ([P, I64, I64, P, P], I),
        "qg_gemm_w4a8_mxfp4": ([P, P, P, I64, I64, P, I64, P, I, I64, P], I),
        "qg_linear_w4a8_mxfp4": ([P, I, I64, I64, I64, P, I64, P, I, I64, P, P, SZ, P], I),
        "qg_quantize_act_fp8": ([P, I, I64, I64, I64, P, P, I64, P], I),
        "qg_gemm_fp8": ([P, P, I64, I64, I64, P, I64, P, I64, P, I, I64, P], I),
        "qg_linear_fp8_workspace_bytes": ([I64, I64], SZ),
        "qg_linear_fp8": ([P, I, I64, I64, I64, P, I64, P, I64, P, I, I64, P, SZ, P], I),
        "qg_token_logprobs": ([P, I, I64, I64, I64, P, I64, P, P, I, P, P, P], I),
        "qg_rmsnorm_quantize_act_fp8": ([P, P, I, I64, I64, I64, I64, P, I, F, P, I64, P, P, I64, P], I),
        "qg_rmsnorm_quantize_act": ([P, P, I, I64, I64, I64, I64, P, I, F, P, I64, P, P, P, P, P], I),
        "qg_silu_mul_quantize_act_fp8": ([P, I, I64, I64, I64, P, P, I64, P], I),
        "qg_gemm_fp8_grouped": ([P, P, I64, I64, I64, P, I64, P, I64, I64, P, I64, P, I, I64, P], I),
        "qg_add_lora_workspace_bytes": ([I64, I64, I64], SZ),
        "qg_add_lora": ([P, I, I64, P, I, I64, I64, I64, P, P, I64, I64, I64, P, P, P, I64, P, SZ, P], I),
    }
    for name, (args, res) in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def declared_symbols():
    """Names of the functions include/qgemm.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(qg_[a-z0-9_]+)\s*\(", text)))


def _check(status):
    if status != QG_OK:
        L = load()
        raise QGError(status, L.qg_last_error().decode() or L.qg_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return QG_BF16
    if dt == torch.float32:
        return QG_F32
    raise ValueError("dtype must be torch.bfloat16 or torch.float32")


# ----------------------------------------------------------------------- API
def quantize_act(x, block_sums=False, q16=False, out=None, stream=None, int8=True):
    """x: cuda [M, K] bf16/fp32 (rows may be strided) ->
    (q int8 [M,K] or None, scale fp32 [M], block_sums int32 [M,K/32] or None,
    q16 fp16 [M,K] or None). `out` may supply preallocated (q, scale, block_sums,
    q16); int8=False skips q (the prefill GEMM reads q16 alone)."""
    assert x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        dev = x.device
        q = torch.empty((M, K), dtype=torch.int8, device=dev) if int8 else None
        s = torch.empty((M,), dtype=torch.float32, device=dev)
        bs = torch.empty((M, K // 32), dtype=torch.int32, device=dev) if block_sums else None
        h = torch.empty((M, K), dtype=torch.float16, device=dev) if q16 else None
    else:
        q, s, bs, h = out
    _check(load().qg_quantize_act(_ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), _ptr(q),
                                  _ptr(s), _ptr(bs), _ptr(h), _stream(stream)))
    return q, s, bs, h


def quantize_act_static(x, scale, block_sums=False, q16=False, out=None, stream=None):
    """x: cuda [M, K] bf16/fp32; scale: cuda fp32 [M] (per row) or [1] (all rows)
    -> (q int8, block_sums or None, q16 or None). Values beyond s*127 saturate."""
    assert x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    stride = 0 if scale.numel() == 1 else 1
    if out is None:
        dev = x.device
        q = torch.empty((M, K), dtype=torch.int8, device=dev)
        bs = torch.empty((M, K // 32), dtype=torch.int32, device=dev) if block_sums else None
        h = torch.empty((M, K), dtype=torch.float16, device=dev) if q16 else None
    else:
        q, bs, h = out
    _check(load().qg_quantize_act_static(_ptr(x), _dtype_code(x.dtype), M, K, x.stride(0),
                                         _ptr(scale), stride, _ptr(q), _ptr(bs), _ptr(h),
                                         _stream(stream)))
    return q, bs, h


def q8_0_packed_bytes(N, K):
    return int(load().qg_q8_0_packed_bytes(N, K))


def q4k_packed_bytes(N, K):
    return int(load().qg_q4k_packed_bytes(N, K))


def pack_q8_0(blocks, N, K, stream=None):
    """blocks: cuda uint8 tensor holding N*K/32 Q8_0 blocks of 34 bytes -> packed uint8 tensor."""
    nbytes = q8_0_packed_bytes(N, K)
    if nbytes == 0:
        raise QGError(QG_EINVAL, "bad N/K for Q8_0")
    packed = torch.empty((nbytes,), dtype=torch.uint8, device=blocks.device)
    _check(load().qg_pack_q8_0(_ptr(blocks), N, K, _ptr(packed), _stream(stream)))
    return packed


def pack_q4k(superblocks, N, K, stream=None):
    nbytes = q4k_packed_bytes(N, K)
    if nbytes == 0:
        raise QGError(QG_EINVAL, "bad N/K for Q4_K")
    packed = torch.empty((nbytes,), dtype=torch.uint8, device=superblocks.device)
    _check(load().qg_pack_q4k(_ptr(superblocks), N, K, _ptr(packed), _stream(stream)))
    return packed


def gemm_w8a8_q8_0(q, q16, scale, packed, N, out=None, out_dtype=torch.bfloat16, path="auto",
                   stream=None):
    """q (may be None when the prefill kernel runs), q16, scale from quantize_act."""
    M, K = (q if q is not None else q16).shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=scale.device)
    _check(load().qg_gemm_w8a8_q8_0_ex(_ptr(q), _ptr(q16), _ptr(scale), M, K, _ptr(packed), N,
                                       _ptr(out), _dtype_code(out.dtype), out.stride(0),
                                       PATHS[path], _stream(stream)))
    return out


def gemm_w4a8_q4k(q, q16, scale, block_sums, packed, N, out=None, out_dtype=torch.bfloat16,
                  path="auto", stream=None):
    M, K = (q if q is not None else q16).shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=scale.device)
    _check(load().qg_gemm_w4a8_q4k_ex(_ptr(q), _ptr(q16), _ptr(scale), _ptr(block_sums), M, K,
                                      _ptr(packed), N, _ptr(out), _dtype_code(out.dtype),
                                      out.stride(0), PATHS[path], _stream(stream)))
    return out


def debug_block_sums(kind, q, q16, packed, N, path, stream=None):
    """Exact per-block integer sums isum[M][N][K/32] as the chosen kernel computes them."""
    M, K = q.shape
    isum = torch.empty((M, N, K // 32), dtype=torch.int32, device=q.device)
    fn = load().qg_debug_block_sums_q8_0 if kind == "q8_0" else load().qg_debug_block_sums_q4k
    _check(fn(_ptr(q), _ptr(q16), M, K, _ptr(packed), N, _ptr(isum), PATHS[path], _stream(stream)))
    return isum


def debug_wait_timeout(polls, stream=None):
    """Launch one bounded wait that is made to run out (failure-detection test)."""
    _check(load().qg_debug_wait_timeout(polls, _stream(stream)))


def check_device_error(stream=None):
    _check(load().qg_check_device_error(_stream(stream)))


def gemm_launch_count(kind, M, K, N, path="auto"):
    """Kernel launches one GEMM call of these sizes makes (kind "q8_0" or "q4k")."""
    return int(load().qg_gemm_launch_count(0 if kind == "q8_0" else 1, M, K, N, PATHS[path]))


def small_m_max():
    return int(load().qg_small_m_max())


def linear_workspace_bytes(kind, M, K):
    """Workspace bytes a linear_* call of these sizes needs."""
    return int(load().qg_linear_workspace_bytes(0 if kind == "q8_0" else 1, M, K))


def _linear(kind, x, packed, N, out, out_dtype, scale_out, workspace, stream, fn=None):
    assert x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    need = linear_workspace_bytes(kind, M, K)
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if fn is None:
        fn = load().qg_linear_w8a8_q8_0 if kind == "q8_0" else load().qg_linear_w4a8_q4k
    _check(fn(_ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), _ptr(packed), N, _ptr(out),
              _dtype_code(out.dtype), out.stride(0), _ptr(scale_out), _ptr(workspace), nbytes,
              _stream(stream)))
    return out


def linear_w8a8_q8_0(x, packed, N, out=None, out_dtype=torch.bfloat16, scale_out=None,
                     workspace=None, stream=None):
    """The whole layer: x cuda [M, K] bf16/fp32 (rows may be strided) -> out [M, N].
    Quantize, then GEMM, through `workspace` (allocated here when not given);
    for M <= small_m_max() the GEMM overlaps the quantize kernel (programmatic
    dependent launch). scale_out: optional fp32 [M] receiving the row scales."""
    return _linear("q8_0", x, packed, N, out, out_dtype, scale_out, workspace, stream)


def linear_w4a8_q4k(x, packed, N, out=None, out_dtype=torch.bfloat16, scale_out=None,
                    workspace=None, stream=None):
    """As linear_w8a8_q8_0, with Q4_K weights."""
    return _linear("q4k", x, packed, N, out, out_dtype, scale_out, workspace, stream)


def pack_mxfp4_q8_0(blocks, N, K, stream=None):
    """Q8_0 blocks (cuda uint8, N*K/32 x 34 bytes) converted to MXFP4 and packed
    (lossy: see include/qgemm.h). check_device_error() raises QG_ERANGE when a
    block scale does not fit the decode kernels' fp16 scales."""
    nbytes = int(load().qg_mxfp4_packed_bytes(N, K))
    if nbytes == 0:
        raise QGError(QG_EINVAL, "bad N/K for MXFP4")
    packed = torch.empty((nbytes,), dtype=torch.uint8, device=blocks.device)
    _check(load().qg_pack_mxfp4_q8_0(_ptr(blocks), N, K, _ptr(packed), _stream(stream)))
    return packed


def gemm_w4a8_mxfp4(q, q16, scale, packed, N, out=None, out_dtype=torch.bfloat16, stream=None):
    """As gemm_w8a8_q8_0 (AUTO path), on weights from pack_mxfp4_q8_0."""
    M, K = (q if q is not None else q16).shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=(q if q is not None else q16).device)
    _check(load().qg_gemm_w4a8_mxfp4(_ptr(q), _ptr(q16), _ptr(scale), M, K, _ptr(packed), N,
                                     _ptr(out), _dtype_code(out.dtype), out.stride(0),
                                     _stream(stream)))
    return out


def linear_w4a8_mxfp4(x, packed, N, out=None, out_dtype=torch.bfloat16, scale_out=None,
                      workspace=None, stream=None):
    """As linear_w8a8_q8_0, on weights from pack_mxfp4_q8_0."""
    return _linear("q8_0", x, packed, N, out, out_dtype, scale_out, workspace, stream,
                   fn=load().qg_linear_w4a8_mxfp4)


def _empty(shape, dtype, device, stream, ld=None):
    """Memory for work on `stream`: taken from that stream's pool, so that its reuse follows that work.
    `ld`: distance of a matrix's rows (a view of a wider tensor costs several us of host time)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(shape, dtype, device, None, ld)
    if ld is not None:
        return torch.empty_strided(shape, (ld, 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _raw_stream(stream, device):
    """The cudaStream_t of `stream`, or of the current stream of `device`, as a number."""
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


# torch's own number of the current stream, without the Stream object around it (the calls below
# are short next to the kernels of a decode step: 9-12 us of host time in place of 20-26)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# (the same without its check that CUDA has been initialised: a cuda tensor is at hand)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_CODES = {_BF16: QG_BF16, _F32: QG_F32}


def _device(first, stream):
    """Index of a call's device, that of its first tensor; `stream` has to be one of its streams. (The
    library launches on the current device: where that is another one, a call enters itself again.)"""
    dev = first.get_device()
    if stream is not None and stream.device_index != dev:
        raise ValueError("the stream must belong to the tensors' device")
    return dev


def _rows(t, name, dtypes, dev=None):
    """(rows, columns, row stride) of a cuda matrix of one of `dtypes` whose rows are contiguous, on
    device `dev` if one is given."""
    if (t.is_cuda if dev is None else t.get_device() == dev) and t.dtype in dtypes and t.dim() == 2:
        m, n = t.shape
        ld, step = t.stride()
        if step == 1 or n <= 1:
            # (the distance of a single row to the next says nothing)
            return m, n, ld if m > 1 else n
    raise ValueError("%s must be a 2-D cuda tensor of %s with contiguous rows%s" %
                     (name, " or ".join(str(d) for d in dtypes),
                      "" if dev is None else ", on device %d like the others of its call" % dev))


def _fp8_scale(scale, M, K, dev):
    """Row stride of the scales [ceil(K/128), M] of activations [M, K]."""
    kb, m, ld = _rows(scale, "scale", (_F32,), dev)
    if kb != (K + 127) // 128 or m != M:
        raise ValueError("scale must have the shape [ceil(K/128), M]")
    # a single block of K has one row of scales: any stride does
    return ld if kb > 1 else (M + 3) // 4 * 4


def _fp8_weights(w, w_scale, M, K, out, out_dtype, stream, dev):
    """(N, row stride of w, out, its row stride), checked; `out` is allocated when None."""
    N, k, ldw = _rows(w, "w", (_FP8,), dev)
    if k != K:
        raise ValueError("w has rows of %d values, the activations of %d" % (k, K))
    if (w_scale.get_device() != dev or w_scale.dtype != _F32 or not w_scale.is_contiguous()
            or w_scale.shape != ((N + 127) // 128, (K + 127) // 128)):
        raise ValueError("w_scale must be a contiguous fp32 tensor of shape [ceil(N/128), ceil(K/128)] on w's device")
    if out is None:
        if out_dtype not in _CODES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        return N, ldw, _empty((M, N), out_dtype, w.device, stream), N
    m, n, ldo = _rows(out, "out", _CODES, dev)
    if m != M or n != N:
        raise ValueError("out must have the shape (%d, %d)" % (M, N))
    return N, ldw, out, ldo


def quantize_act_fp8(x, out=None, stream=None):
    """x: cuda [M, K] bf16/fp32 (rows may be strided; K % 16 == 0) -> (q float8_e4m3fn [M, K],
    scale fp32 [ceil(K/128), M], one per token and 128 values of K; its rows start on 16-byte
    boundaries). `out` may supply preallocated (q, scale)."""
    M, K, ldx = _rows(x, "x", _CODES)
    dev = _device(x, stream)
    if out is None:
        lds = (M + 3) // 4 * 4
        q = _empty((M, K), _FP8, x.device, stream)
        scale = _empty(((K + 127) // 128, M), _F32, x.device, stream, lds)
    else:
        q, scale = out
        if _rows(q, "q", (_FP8,), dev) != (M, K, K):
            raise ValueError("q must be contiguous and of the shape of x")
        lds = _fp8_scale(scale, M, K, dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return quantize_act_fp8(x, (q, scale), stream)
    _check((_lib or load()).qg_quantize_act_fp8(x.data_ptr(), _CODES[x.dtype], M, K, ldx, q.data_ptr(),
                                                scale.data_ptr(), lds, _raw_stream(stream, dev)))
    return q, scale


def gemm_fp8(q, scale, w, w_scale, out=None, out_dtype=torch.bfloat16, stream=None):
    """q, scale from quantize_act_fp8; w: cuda float8_e4m3fn [N, K] as stored (rows may be strided);
    w_scale: cuda fp32 [ceil(N/128), ceil(K/128)] -> out [M, N]."""
    M, K, ldq = _rows(q, "q", (_FP8,))
    if ldq != K:
        raise ValueError("q must be contiguous")
    dev = _device(q, stream)
    lds = _fp8_scale(scale, M, K, dev)
    N, ldw, out, ldo = _fp8_weights(w, w_scale, M, K, out, out_dtype, stream, dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gemm_fp8(q, scale, w, w_scale, out, stream=stream)
    _check((_lib or load()).qg_gemm_fp8(q.data_ptr(), scale.data_ptr(), lds, M, K, w.data_ptr(), ldw,
                                        w_scale.data_ptr(), N, out.data_ptr(), _CODES[out.dtype], ldo,
                                        _raw_stream(stream, dev)))
    return out


@functools.lru_cache(maxsize=4096)
def linear_fp8_workspace_bytes(M, K):
    """Workspace bytes a linear_fp8 call of these sizes needs (0: invalid sizes)."""
    return int(load().qg_linear_fp8_workspace_bytes(M, K))


def linear_fp8(x, w, w_scale, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """The whole layer: x cuda [M, K] bf16/fp32 -> out [M, N] with e4m3 weights (see gemm_fp8).
    Quantize, then GEMM, through `workspace` (allocated here when not given)."""
    M, K, ldx = _rows(x, "x", _CODES)
    dev = _device(x, stream)
    N, ldw, out, ldo = _fp8_weights(w, w_scale, M, K, out, out_dtype, stream, dev)
    if workspace is None:
        nbytes = linear_fp8_workspace_bytes(M, K)
        workspace = _empty((nbytes,), torch.uint8, x.device, stream)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on x's device")
        nbytes = workspace.numel() * workspace.element_size()
    if dev != _current_device():
        with torch.cuda.device(dev):
            return linear_fp8(x, w, w_scale, out, workspace=workspace, stream=stream)
    _check((_lib or load()).qg_linear_fp8(x.data_ptr(), _CODES[x.dtype], M, K, ldx, w.data_ptr(), ldw,
                                          w_scale.data_ptr(), N, out.data_ptr(), _CODES[out.dtype], ldo,
                                          workspace.data_ptr(), nbytes, _raw_stream(stream, dev)))
    return out


def token_logprobs(logits, ids, top=0, stream=None):
    """logits: cuda [M, V] bf16/fp32 (rows may be strided); ids: cuda int64 [M, G] or [M] (-1: no
    token) -> (logprobs fp32 of ids' shape, entropy fp32 [M], top_ids int64 [M, top], top_logprobs
    fp32 [M, top]): log probabilities of the given tokens, the rows' entropies in nats and their
    `top` likeliest tokens, ties to the lowest id; -1 where a row has fewer (see include/qgemm.h).
    The last bits of the floats depend on the number of rows and on where a row lies."""
    M, V, ldl = _rows(logits, "logits", _CODES)
    shape = ids.shape
    dev = _device(logits, stream)
    if (ids.get_device() != dev or ids.dtype != torch.int64 or len(shape) not in (1, 2) or shape[0] != M
            or not ids.is_contiguous()):
        raise ValueError("ids must be a contiguous int64 tensor of shape [M] or [M, G] on the logits' device")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return token_logprobs(logits, ids, top, stream)
    G = shape[1] if len(shape) == 2 else 1
    where, k = logits.device, max(top, 0)
    logprobs = _empty(shape, _F32, where, stream)
    entropy = _empty((M,), _F32, where, stream)
    top_ids = _empty((M, k), torch.int64, where, stream)
    top_logprobs = _empty((M, k), _F32, where, stream)
    _check((_lib or load()).qg_token_logprobs(logits.data_ptr(), _CODES[logits.dtype], M, V, ldl,
                                              ids.data_ptr(), G, logprobs.data_ptr(), entropy.data_ptr(),
                                              top, top_ids.data_ptr(), top_logprobs.data_ptr(),
                                              _raw_stream(stream, dev)))
    return logprobs, entropy, top_ids, top_logprobs


def _norm_inputs(x, weight, residual):
    """(M, K, row stride of x, of residual, device), checked."""
    M, K, ldx = _rows(x, "x", _CODES)
    dev = x.get_device()
    if (weight.get_device() != dev or weight.dtype not in _CODES or weight.shape != (K,)
            or not weight.is_contiguous()):
        raise ValueError("weight must be a contiguous bf16 or fp32 tensor of shape [K] on x's device")
    if residual is None:
        return M, K, ldx, 0, dev
    m, k, ldr = _rows(residual, "residual", (x.dtype,), dev)
    if m != M or k != K:
        raise ValueError("residual must have the shape of x")
    return M, K, ldx, ldr, dev


def _norm_sum(total, residual, x, M, K, stream, dev):
    """(sum, its row stride): checked, allocated when None; (None, 0) without a residual."""
    if residual is None:
        if total is not None:
            raise ValueError("sum is written where there is a residual only")
        return None, 0
    if total is None:
        return _empty((M, K), x.dtype, x.device, stream), K
    m, k, ld = _rows(total, "sum", (x.dtype,), dev)
    if m != M or k != K:
        raise ValueError("sum must have the shape of x")
    return total, ld


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def rmsnorm_quantize_act_fp8(x, weight, eps=1e-6, residual=None, out=None, stream=None):
    """Norm of the rows of x (cuda [M, K] bf16/fp32, rows may be strided; K % 16 == 0), or of
    x + residual, times weight (bf16/fp32 [K]), quantized in the layout of quantize_act_fp8, by products
    with 1/s -> (q float8_e4m3fn [M, K], scale fp32 [ceil(K/128), M], x + residual in x's dtype or
    None). `out` may supply preallocated (q, scale, sum); sum may be residual or x itself, and is None
    without a residual."""
    M, K, ldx, ldr, dev = _norm_inputs(x, weight, residual)
    _device(x, stream)
    if out is None:
        lds = (M + 3) // 4 * 4
        q = _empty((M, K), _FP8, x.device, stream)
        scale = _empty(((K + 127) // 128, M), _F32, x.device, stream, lds)
        total = None
    else:
        q, scale, total = out
        if _rows(q, "q", (_FP8,), dev) != (M, K, K):
            raise ValueError("q must be contiguous and of the shape of x")
        lds = _fp8_scale(scale, M, K, dev)
    total, ldsum = _norm_sum(total, residual, x, M, K, stream, dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return rmsnorm_quantize_act_fp8(x, weight, eps, residual, (q, scale, total), stream)
    _check((_lib or load()).qg_rmsnorm_quantize_act_fp8(
        x.data_ptr(), _ptr_or_none(residual), _CODES[x.dtype], M, K, ldx, ldr, weight.data_ptr(),
        _CODES[weight.dtype], eps, _ptr_or_none(total), ldsum, q.data_ptr(), scale.data_ptr(), lds,
        _raw_stream(stream, dev)))
    return q, scale, total


def rmsnorm_quantize_act(x, weight, eps=1e-6, residual=None, block_sums=False, q16=False, out=None,
                         stream=None, int8=True):
    """As rmsnorm_quantize_act_fp8, in the layout of quantize_act (K % 32 == 0) -> (q int8 [M, K] or
    None, scale fp32 [M], block_sums int32 [M, K/32] or None, q16 fp16 [M, K] or None, x + residual
    or None). `out` may supply preallocated (q, scale, block_sums, q16, sum)."""
    M, K, ldx, ldr, dev = _norm_inputs(x, weight, residual)
    _device(x, stream)
    total = None
    if out is None:
        where = x.device
        q = _empty((M, K), torch.int8, where, stream) if int8 else None
        scale = _empty((M,), _F32, where, stream)
        bs = _empty((M, K // 32), torch.int32, where, stream) if block_sums else None
        h = _empty((M, K), torch.float16, where, stream) if q16 else None
    else:
        q, scale, bs, h, total = out
        for t, name, dtype, shape in ((q, "q", torch.int8, (M, K)), (scale, "scale", _F32, (M,)),
                                      (bs, "block_sums", torch.int32, (M, K // 32)),
                                      (h, "q16", torch.float16, (M, K))):
            if t is not None and (t.get_device() != dev or t.dtype != dtype or t.shape != shape
                                  or not t.is_contiguous()):
                raise ValueError("%s must be a contiguous %s tensor of shape %s on x's device" %
                                 (name, dtype, shape))
    total, ldsum = _norm_sum(total, residual, x, M, K, stream, dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return rmsnorm_quantize_act(x, weight, eps, residual, out=(q, scale, bs, h, total), stream=stream)
    _check((_lib or load()).qg_rmsnorm_quantize_act(
        x.data_ptr(), _ptr_or_none(residual), _CODES[x.dtype], M, K, ldx, ldr, weight.data_ptr(),
        _CODES[weight.dtype], eps, _ptr_or_none(total), ldsum, _ptr_or_none(q), _ptr_or_none(scale),
        _ptr_or_none(bs), _ptr_or_none(h), _raw_stream(stream, dev)))
    return q, scale, bs, h, total


def silu_mul_quantize_act_fp8(x, out=None, stream=None):
    """x: cuda [M, 2K] bf16/fp32 (rows may be strided; K % 16 == 0), K gates and K values up a row ->
    silu(gate) * up quantized as by rmsnorm_quantize_act_fp8: (q float8_e4m3fn [M, K], scale fp32
    [ceil(K/128), M]). `out` may supply preallocated (q, scale)."""
    M, K2, ldx = _rows(x, "x", _CODES)
    if K2 % 2:
        raise ValueError("x must have an even number of columns: gates, then values")
    K = K2 // 2
    dev = _device(x, stream)
    if out is None:
        lds = (M + 3) // 4 * 4
        q = _empty((M, K), _FP8, x.device, stream)
        scale = _empty(((K + 127) // 128, M), _F32, x.device, stream, lds)
    else:
        q, scale = out
        if _rows(q, "q", (_FP8,), dev) != (M, K, K):
            raise ValueError("q must be contiguous and of half the columns of x")
        lds = _fp8_scale(scale, M, K, dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return silu_mul_quantize_act_fp8(x, (q, scale), stream)
    _check((_lib or load()).qg_silu_mul_quantize_act_fp8(x.data_ptr(), _CODES[x.dtype], M, K, ldx,
                                                         q.data_ptr(), scale.data_ptr(), lds,
                                                         _raw_stream(stream, dev)))
    return q, scale


def _matrices(t, name, dtype, dev):
    """(matrices, rows, columns, row stride, matrix stride) of a cuda tensor whose rows are contiguous."""
    if t.get_device() == dev and t.dtype == dtype and t.dim() == 3:
        e, n, k = t.shape
        lde, ld, step = t.stride()
        if step == 1 or k <= 1:
            # (the distance of a single row or matrix to the next says nothing)
            return e, n, k, ld if n > 1 else k, lde
    raise ValueError("%s must be a 3-D cuda tensor of %s with contiguous rows, on device %d like the others "
                     "of its call" % (name, dtype, dev))


def gemm_fp8_grouped(q, scale, offsets, w, w_scale, out=None, out_dtype=torch.bfloat16, stream=None):
    """gemm_fp8 with the weights of each row's expert: q, scale from quantize_act_fp8 (or one of its
    siblings), rows sorted by expert; offsets: cuda int64 [E+1], expert e owns rows offsets[e] up to
    offsets[e+1] (read on the device: no synchronisation); w: cuda float8_e4m3fn [E, N, K] (rows and
    experts may be strided); w_scale: cuda fp32 [E, ceil(N/128), ceil(K/128)] -> out [M, N]. Rows of
    no expert are left as they were (undefined in an `out` allocated here)."""
    M, K, ldq = _rows(q, "q", (_FP8,))
    if ldq != K:
        raise ValueError("q must be contiguous")
    dev = _device(q, stream)
    lds = _fp8_scale(scale, M, K, dev)
    E, N, k, ldw, lde = _matrices(w, "w", _FP8, dev)
    if k != K:
        raise ValueError("w has rows of %d values, the activations of %d" % (k, K))
    if (offsets.get_device() != dev or offsets.dtype != torch.int64 or offsets.shape != (E + 1,)
            or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int64 tensor of shape [E + 1] on q's device")
    if (w_scale.get_device() != dev or w_scale.dtype != _F32 or not w_scale.is_contiguous()
            or w_scale.shape != (E, (N + 127) // 128, (K + 127) // 128)):
        raise ValueError("w_scale must be a contiguous fp32 tensor of shape [E, ceil(N/128), ceil(K/128)] "
                         "on w's device")
    if out is None:
        if out_dtype not in _CODES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out, ldo = _empty((M, N), out_dtype, q.device, stream), N
    else:
        m, n, ldo = _rows(out, "out", _CODES, dev)
        if m != M or n != N:
            raise ValueError("out must have the shape (%d, %d)" % (M, N))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gemm_fp8_grouped(q, scale, offsets, w, w_scale, out, stream=stream)
    _check((_lib or load()).qg_gemm_fp8_grouped(q.data_ptr(), scale.data_ptr(), lds, M, K, offsets.data_ptr(),
                                                E, w.data_ptr(), ldw, lde, w_scale.data_ptr(), N,
                                                out.data_ptr(), _CODES[out.dtype], ldo,
                                                _raw_stream(stream, dev)))
    return out


@functools.lru_cache(maxsize=4096)
def add_lora_workspace_bytes(M, K, rank):
    """Workspace bytes an add_lora call of these sizes needs (0: invalid sizes)."""
    return int(load().qg_add_lora_workspace_bytes(M, K, rank))


def add_lora(base, x, a, b, ids, scaling=None, out=None, workspace=None, stream=None):
    """Low-rank adapters beside a projection: out = base + scaling[id] * (x . a[id]^T) . b[id]^T row by
    row, id = ids[m]; rows whose id is no adapter's (-1) keep base's bits. base: cuda [M, N] bf16/fp32,
    the projection's output; x: cuda [M, K] bf16/fp32, its input (K % 16 == 0); rows of both may be
    strided; a, b: contiguous cuda bf16 [adapters, rank, K], [adapters, N, rank] (rank a multiple of 8,
    at most 128); ids: cuda int64 [M]; scaling: cuda fp32 [adapters] or None for 1 -> out [M, N] of
    base's dtype. `out` may be base itself. Through `workspace` (allocated here when not given). A
    row's bits do not depend on the other rows among calls of few rows (up to 128 of ranks up to 32, 32
    of ranks up to 64, 16 of higher ranks), nor among calls of more, which tensor cores compute."""
    M, N, ldb = _rows(base, "base", _CODES)
    dev = _device(base, stream)
    m, K, ldx = _rows(x, "x", _CODES, dev)
    if m != M:
        raise ValueError("x has %d rows, base %d" % (m, M))
    for t, name in ((a, "a"), (b, "b")):
        if t.get_device() != dev or t.dtype != _BF16 or t.dim() != 3 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous 3-D bf16 tensor on base's device" % name)
    count, rank, k = a.shape
    if k != K or b.shape != (count, N, rank):
        raise ValueError("a and b must have the shapes [adapters, rank, %d] and [adapters, %d, rank]" % (K, N))
    if ids.get_device() != dev or ids.dtype != torch.int64 or ids.shape != (M,) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 tensor of shape [M] on base's device")
    if scaling is not None and (scaling.get_device() != dev or scaling.dtype != _F32
                                or scaling.shape != (count,) or not scaling.is_contiguous()):
        raise ValueError("scaling must be a contiguous fp32 tensor of shape [adapters] on base's device")
    if out is None:
        out, ldo = _empty((M, N), base.dtype, base.device, stream), N
    else:
        m, n, ldo = _rows(out, "out", (base.dtype,), dev)
        if m != M or n != N:
            raise ValueError("out must have the shape (%d, %d)" % (M, N))
    if workspace is None:
        nbytes = add_lora_workspace_bytes(M, K, rank)
        workspace = _empty((nbytes,), torch.uint8, base.device, stream)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on base's device")
        nbytes = workspace.numel() * workspace.element_size()
    if dev != _current_device():
        with torch.cuda.device(dev):
            return add_lora(base, x, a, b, ids, scaling, out, workspace, stream)
    _check((_lib or load()).qg_add_lora(base.data_ptr(), _CODES[base.dtype], ldb, x.data_ptr(),
                                        _CODES[x.dtype], M, K, ldx, a.data_ptr(), b.data_ptr(), count, rank, N,
                                        ids.data_ptr(), _ptr_or_none(scaling), out.data_ptr(), ldo,
                                        workspace.data_ptr(), nbytes, _raw_stream(stream, dev)))
    return out


def linear_noalloc_scratch_bytes():
    """QG_LINEAR_NOALLOC_SCRATCH_BYTES, read from include/qgemm.h."""
    m = re.search(r"#define\s+QG_LINEAR_NOALLOC_SCRATCH_BYTES\s+\(\(size_t\)(\d+)\s*<<\s*(\d+)\)",
                  open(HEADER).read())
    return int(m.group(1)) << int(m.group(2))


def linear_w8a8_q8_0_noalloc(x, packed, N, out=None, out_dtype=torch.bfloat16, scale_out=None,
                             stream=None):
    """As linear_w8a8_q8_0, with the library's static scratch in place of a
    workspace: the library call allocates nothing (`out` is allocated here
    when not given). Sizes are limited to linear_noalloc_scratch_bytes() of
    scratch; calls that overlap on the GPU share the scratch and race."""
    assert x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check(load().qg_linear_w8a8_q8_0_noalloc(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), _ptr(packed), N, _ptr(out),
        _dtype_code(out.dtype), out.stride(0), _ptr(scale_out), _stream(stream)))
    return out


def gemm_fp8_tile(M, N, sms):
    """Test support (host-only): (tokens, weight rows) of gemm_fp8's tile for M x N on `sms` SMs."""
    tokens, rows = ctypes.c_int(), ctypes.c_int()
    _check(load().qg_debug_gemm_fp8_tile(M, N, sms, ctypes.byref(tokens), ctypes.byref(rows)))
    return tokens.value, rows.value


def gemm_fp8_grouped_tile(M, N, experts, sms):
    """Test support (host-only): (rows, weight rows) of gemm_fp8_grouped's tile for M rows of `experts` on `sms` SMs."""
    tokens, rows = ctypes.c_int(), ctypes.c_int()
    _check(load().qg_debug_gemm_fp8_grouped_tile(M, N, experts, sms, ctypes.byref(tokens), ctypes.byref(rows)))
    return tokens.value, rows.value


def logprobs_pieces(M, V, sms):
    """Test support (host-only): the pieces token_logprobs cuts a row of V into, for M rows on `sms` SMs."""
    pieces = ctypes.c_int()
    _check(load().qg_debug_logprobs_pieces(M, V, sms, ctypes.byref(pieces)))
    return pieces.value


def prefill_tile_q4k(M, N, sms):
    """The W4A8 GEMM's tiles for M x N on `sms` SMs: ("tensor" / "16-row", token width)."""
    kind = ctypes.c_int()
    tokens = ctypes.c_int()
    _check(load().qg_debug_prefill_tile_q4k(M, N, sms, ctypes.byref(kind), ctypes.byref(tokens)))
    return {1: "tensor", 2: "16-row"}[kind.value], tokens.value


def prefill_plan(M, N, sms):
    """The W8A8 prefill wave plan on `sms` SMs: (rows of the 256-token launch,
    narrow-part kind: None / "tensor" / "16-row", its token-tile width)."""
    rows = ctypes.c_int64()
    kind = ctypes.c_int()
    tokens = ctypes.c_int()
    _check(load().qg_debug_prefill_plan_q8_0(M, N, sms, ctypes.byref(rows), ctypes.byref(kind),
                                             ctypes.byref(tokens)))
    return rows.value, {0: None, 1: "tensor", 2: "16-row"}[kind.value], tokens.value
