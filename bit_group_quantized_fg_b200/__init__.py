"""Python binding of the 4-bit group-wise compressed decode path (B200, sm_100a).

Argument marshalling only: every step runs in the CUDA kernels of ``libfg.so`` behind the
C ABI of ``include/fg.h``; PyTorch supplies device memory and streams.  There is no CPU
path: importing works without a GPU (for builds and symbol checks), but every call needs
the compiled library and a CUDA device and raises otherwise.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int, c_int64, c_size_t, c_void_p

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfg.so")

FG_OK = 0
STATUS = {0: "FG_OK", -1: "FG_ERR_INVALID_ARG", -2: "FG_ERR_SHAPE", -3: "FG_ERR_ALIGN",
          -4: "FG_ERR_CAPACITY", -5: "FG_ERR_CUDA", -6: "FG_ERR_UNSUPPORTED", -7: "FG_ERR_WORKSPACE"}
(PROF_GEMM, PROF_DECODE_ATTN, PROF_PREFILL_ATTN, PROF_QUANT, PROF_OTHER, PROF_GEMM_DECODE,
 PROF_LM_HEAD) = range(7)
PROF_NAMES = ["gemm_prefill", "decode_attention", "prefill_attention", "quantize_append", "other",
              "gemm_decode", "lm_head"]


class FGError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class QLinear(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("params", c_void_p), ("bias", c_void_p),
                ("K", c_int), ("N", c_int), ("group", c_int), ("w16", c_void_p), ("group_along_k", c_int)]


class Layer(ctypes.Structure):
    _fields_ = [("ln1_g", c_void_p), ("ln1_b", c_void_p), ("ln2_g", c_void_p), ("ln2_b", c_void_p),
                ("qkv", QLinear), ("out", QLinear), ("fc1", QLinear), ("fc2", QLinear)]


class KVCache(ctypes.Structure):
    _fields_ = [("k_codes", c_void_p), ("v_codes", c_void_p), ("k_params", c_void_p),
                ("v_params", c_void_p), ("B", c_int), ("n_heads", c_int), ("head_dim", c_int),
                ("group", c_int), ("capacity", c_int), ("len", c_int)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k_codes", c_void_p), ("v_codes", c_void_p), ("k_params", c_void_p),
                ("v_params", c_void_p), ("page_table", c_void_p), ("B", c_int), ("n_kv_heads", c_int),
                ("head_dim", c_int), ("group", c_int), ("page_size", c_int), ("n_pages", c_int),
                ("max_pages", c_int)]


class Model(ctypes.Structure):
    _fields_ = [("n_layers", c_int), ("hidden", c_int), ("n_heads", c_int), ("head_dim", c_int),
                ("ffn", c_int), ("vocab", c_int), ("max_pos", c_int), ("group", c_int),
                ("embed", c_void_p), ("pos_embed", c_void_p), ("lnf_g", c_void_p), ("lnf_b", c_void_p),
                ("layers", POINTER(Layer))]


class Timing(ctypes.Structure):
    _fields_ = [("prefill_ms", c_float), ("decode_ms", c_float), ("tokens", c_int64),
                ("tok_per_s", c_double)]


_SIGS = {
    "fg_status_string": (ctypes.c_char_p, [c_int]),
    "fg_last_error": (ctypes.c_char_p, []),
    "fg_version": (c_int, []),
    "fg_quantize_pack": (c_int, [c_void_p, c_int64, c_int64, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "fg_dequantize": (c_int, [c_void_p, c_void_p, c_int64, c_int64, c_int, c_int, c_void_p, c_void_p]),
    "fg_kv_append": (c_int, [POINTER(KVCache), c_void_p, c_void_p, c_int64, c_int, c_void_p]),
    "fg_qgemm_workspace_bytes": (c_size_t, [c_int64, c_int, c_int]),
    "fg_qgemm": (c_int, [c_void_p, c_int64, POINTER(QLinear), c_void_p, c_int, c_void_p, c_void_p, c_size_t,
                         c_void_p]),
    "fg_gemm_f16_workspace_bytes": (c_size_t, [c_int64, c_int, c_int]),
    "fg_gemm_f16": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_int, c_void_p, c_void_p, c_int, c_void_p,
                            c_void_p, c_size_t, c_void_p]),
    "fg_decode_attention_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int]),
    "fg_decode_attention": (c_int, [c_void_p, c_int64, POINTER(KVCache), c_void_p, c_void_p, c_size_t,
                                    c_void_p]),
    "fg_decode_attention_noalloc": (c_int, [c_void_p, c_int64, POINTER(KVCache), c_void_p, c_void_p]),
    "fg_prefill_attention": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p]),
    "fg_layernorm": (c_int, [c_void_p, c_int64, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "fg_embed": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_int, c_void_p, c_void_p]),
    "fg_lm_head_workspace_bytes": (c_size_t, [c_int, c_int]),
    "fg_lm_head_argmax": (c_int, [c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p, c_void_p,
                                  c_size_t, c_void_p]),
    "fg_paged_append": (c_int, [POINTER(PagedCache), c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                c_void_p]),
    "fg_paged_read": (c_int, [POINTER(PagedCache), c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_int64,
                              c_void_p]),
    "fg_paged_attention_workspace_bytes": (c_size_t, [c_int, c_int, c_int]),
    "fg_paged_attention": (c_int, [c_void_p, c_int64, POINTER(PagedCache), c_void_p, c_int, c_int, c_int, c_void_p,
                                   c_void_p, c_size_t, c_void_p]),
    "fg_varlen_attention": (c_int, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_int64, c_void_p,
                                    c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p]),
    "fg_sample": (c_int, [c_void_p, c_int64, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                          c_void_p, c_void_p]),
    "fg_lm_head_sample": (c_int, [c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "fg_decode_layer_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "fg_decode_layer": (c_int, [POINTER(Layer), POINTER(KVCache), c_void_p, c_void_p, c_int, c_void_p,
                                c_size_t, c_void_p]),
    "fg_prefill_layer_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int]),
    "fg_prefill_layer": (c_int, [POINTER(Layer), POINTER(KVCache), c_void_p, c_int, c_int, c_void_p,
                                 c_size_t, c_void_p]),
    "fg_workspace_bytes": (c_size_t, [POINTER(Model), c_int, c_int, c_int]),
    "fg_generate": (c_int, [POINTER(Model), c_void_p, c_int, c_int, c_int, c_void_p, POINTER(KVCache),
                            c_void_p, c_size_t, POINTER(Timing), c_void_p]),
    "fg_offload_workspace_bytes": (c_size_t, [POINTER(Model), c_int, c_int, c_int]),
    "fg_generate_offload": (c_int, [POINTER(Model), c_void_p, c_int, c_int, c_int, c_void_p, POINTER(KVCache),
                                    c_void_p, c_size_t, POINTER(Timing), POINTER(c_double), c_void_p]),
    "fg_profile_enable": (c_int, [c_int]),
    "fg_profile_select": (c_int, [ctypes.c_uint]),
    "fg_profile_read": (c_int, [c_int, POINTER(c_double), POINTER(c_int64), POINTER(c_double),
                                POINTER(c_double)]),
    "fg_profile_reset": (c_int, []),
    "fg_launch_count": (c_int64, []),
}

_lib = None


def lib():
    """Load libfg.so (raises if it has not been built: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with bit_group_quantized_fg_b200/build.py")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != FG_OK:
        raise FGError(status, lib().fg_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _empty(shape, dtype, device):
    import torch
    return torch.empty(shape, dtype=dtype, device=device)


# ------------------------------------------------------------------------- compression
def fg_quantize_pack(x, group: int = 64, axis: int = 1, codes=None, params=None, stream=None):
    """x fp16 [rows, cols] (CUDA) -> (codes uint8 [rows, cols/2], params fp16 [..., 2])."""
    import torch
    rows, cols = x.shape
    if codes is None:
        codes = _empty((rows, cols // 2), torch.uint8, x.device)
    if params is None:
        pshape = (rows, cols // group, 2) if axis == 1 else (rows // group, cols, 2)
        params = _empty(pshape, torch.float16, x.device)
    _check(lib().fg_quantize_pack(_ptr(x), rows, cols, group, axis, _ptr(codes), _ptr(params), _stream(stream)))
    return codes, params


def fg_dequantize(codes, params, rows: int, cols: int, group: int = 64, axis: int = 1, out=None, stream=None):
    import torch
    if out is None:
        out = _empty((rows, cols), torch.float16, codes.device)
    _check(lib().fg_dequantize(_ptr(codes), _ptr(params), rows, cols, group, axis, _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------------------------- state holders
class DeviceQLinear:
    """A 4-bit linear layer resident in HBM (keeps the tensors alive for the C struct)."""

    def __init__(self, codes, params, bias, K: int, N: int, group: int = 64, w16=None, along_k: bool = False):
        self.codes, self.params, self.bias, self.w16 = codes, params, bias, w16
        self.K, self.N, self.group, self.along_k = K, N, group, along_k
        self.c = QLinear(_ptr(codes), _ptr(params), _ptr(bias), K, N, group, _ptr(w16), int(along_k))

    @staticmethod
    def from_fp16(w, bias, group: int = 64, stream=None, along_k: bool = False) -> "DeviceQLinear":
        """Quantize an fp16 weight [K][N] on the GPU: groups along N (output channel) by
        default, along K (input dimension) with along_k."""
        K, N = w.shape
        codes, params = fg_quantize_pack(w, group, 0 if along_k else 1, stream=stream)
        return DeviceQLinear(codes, params, bias, K, N, group, along_k=along_k)

    @staticmethod
    def uncompressed(w, bias) -> "DeviceQLinear":
        """The same layer over the fp16 weight itself (no compression)."""
        K, N = w.shape
        return DeviceQLinear(None, None, bias, K, N, 64, w16=w)


class DeviceLayer:
    def __init__(self, ln1_g, ln1_b, ln2_g, ln2_b, qkv: DeviceQLinear, out: DeviceQLinear,
                 fc1: DeviceQLinear, fc2: DeviceQLinear):
        self.t = (ln1_g, ln1_b, ln2_g, ln2_b)
        self.qkv, self.out, self.fc1, self.fc2 = qkv, out, fc1, fc2
        self.c = Layer(_ptr(ln1_g), _ptr(ln1_b), _ptr(ln2_g), _ptr(ln2_b), qkv.c, out.c, fc1.c, fc2.c)


class DeviceKVCache:
    """4-bit KV cache of one layer in HBM: codes [B][nh][cap][hd/2], params [B][nh][cap][hd/g][2]."""

    def __init__(self, B: int, n_heads: int, head_dim: int, capacity: int, group: int = 64, device="cuda"):
        import torch
        self.k_codes = torch.zeros((B, n_heads, capacity, head_dim // 2), dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_params = torch.zeros((B, n_heads, capacity, head_dim // group, 2), dtype=torch.float16,
                                    device=device)
        self.v_params = torch.zeros_like(self.k_params)
        self.c = KVCache(_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_params), _ptr(self.v_params),
                         B, n_heads, head_dim, group, capacity, 0)

    @property
    def length(self) -> int:
        return self.c.len

    @length.setter
    def length(self, v: int):
        self.c.len = v


class DevicePagedKVCache:
    """Paged 4-bit KV cache of one layer in HBM: codes [n_pages][n_kv][page][hd/2], params
    [n_pages][n_kv][page][hd/g][2]; page_table int32 [B][max_pages] on the device (entries that
    are not a page are -1).  `tensors`: (k_codes, v_codes, k_params, v_params) to use instead of new ones."""

    def __init__(self, page_table, n_kv_heads: int, head_dim: int, n_pages: int, page_size: int = 64, group: int = 64,
                 tensors=None):
        import torch
        dev = page_table.device
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise ValueError("page_table: a contiguous int32 tensor [B, max_pages]")
        if head_dim <= 0 or group <= 0 or n_kv_heads <= 0 or n_pages <= 0 or page_size <= 0 or head_dim % group:
            raise ValueError("sizes must be positive and group divide head_dim")
        cs = (n_pages, n_kv_heads, page_size, head_dim // 2)
        ps = (n_pages, n_kv_heads, page_size, head_dim // group, 2)
        if tensors is None:
            tensors = (torch.zeros(cs, dtype=torch.uint8, device=dev), torch.zeros(cs, dtype=torch.uint8, device=dev),
                       torch.zeros(ps, dtype=torch.float16, device=dev), torch.zeros(ps, dtype=torch.float16, device=dev))
        for t, shape, dt in zip(tensors, (cs, cs, ps, ps), (torch.uint8,) * 2 + (torch.float16,) * 2):
            if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"expected a contiguous {dt} tensor {shape} on {dev}")
        self.page_table = page_table
        self.k_codes, self.v_codes, self.k_params, self.v_params = tensors
        self.c = PagedCache(*[_ptr(t) for t in tensors], _ptr(page_table), page_table.shape[0], n_kv_heads, head_dim,
                            group, page_size, n_pages, page_table.shape[1])
        self.ref, self.h, self.device_index = ctypes.pointer(self.c), n_kv_heads * head_dim, page_table.get_device()

    def check(self, dev: int):
        if self.device_index != dev:
            raise ValueError("the cache is not on the current CUDA device")


class DeviceModel:
    def __init__(self, n_layers, hidden, n_heads, head_dim, ffn, vocab, max_pos, group, embed, pos_embed,
                 lnf_g, lnf_b, layers):
        self.tensors = (embed, pos_embed, lnf_g, lnf_b)
        self.layers = list(layers)
        self._arr = (Layer * max(1, len(self.layers)))(*[l.c for l in self.layers])
        self.c = Model(n_layers, hidden, n_heads, head_dim, ffn, vocab, max_pos, group, _ptr(embed),
                       _ptr(pos_embed), _ptr(lnf_g), _ptr(lnf_b), ctypes.cast(self._arr, POINTER(Layer)))


# ------------------------------------------------------------------------- steps
def fg_kv_append(cache: DeviceKVCache, k, v, row_stride: int, n_tokens: int, stream=None):
    _check(lib().fg_kv_append(ctypes.byref(cache.c), _ptr(k), _ptr(v), row_stride, n_tokens, _stream(stream)))


def fg_qgemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().fg_qgemm_workspace_bytes(M, N, K)


def fg_qgemm(X, W: DeviceQLinear, R=None, relu: bool = False, Y=None, workspace=None, stream=None):
    import torch
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, W.N), torch.float16, X.device)
    wsb = fg_qgemm_workspace_bytes(M, W.N, W.K)
    if workspace is None and wsb:
        workspace = _empty((wsb,), torch.uint8, X.device)
    _check(lib().fg_qgemm(_ptr(X), M, ctypes.byref(W.c), _ptr(R), int(relu), _ptr(Y), _ptr(workspace),
                          0 if workspace is None else workspace.numel(), _stream(stream)))
    return Y


def fg_gemm_f16(X, W, bias=None, R=None, relu: bool = False, Y=None, workspace=None, stream=None):
    """Y = [relu](X @ W + b) [+ R] with an uncompressed fp16 weight W [K, N] on the tensor cores."""
    import torch
    M = X.shape[0]
    K, N = W.shape
    if Y is None:
        Y = _empty((M, N), torch.float16, X.device)
    wsb = lib().fg_gemm_f16_workspace_bytes(M, N, K)
    if workspace is None and wsb:
        workspace = _empty((wsb,), torch.uint8, X.device)
    _check(lib().fg_gemm_f16(_ptr(X), M, _ptr(W), K, N, _ptr(bias), _ptr(R), int(relu), _ptr(Y), _ptr(workspace),
                             0 if workspace is None else workspace.numel(), _stream(stream)))
    return Y


def fg_decode_attention(q, q_stride: int, cache: DeviceKVCache, out=None, workspace=None, stream=None):
    import torch
    B, nh, hd = cache.c.B, cache.c.n_heads, cache.c.head_dim
    if out is None:
        out = _empty((B, nh * hd), torch.float16, q.device)
    wsb = lib().fg_decode_attention_workspace_bytes(B, nh, hd, cache.c.len)
    if workspace is None and wsb:
        workspace = _empty((wsb,), torch.uint8, q.device)
    _check(lib().fg_decode_attention(_ptr(q), q_stride, ctypes.byref(cache.c), _ptr(out), _ptr(workspace),
                                     0 if workspace is None else workspace.numel(), _stream(stream)))
    return out


def fg_decode_attention_noalloc(q, q_stride: int, cache: DeviceKVCache, out=None, stream=None):
    """fg_decode_attention with its scratch in the library's fixed device array (no workspace).
    Only `out` may be allocated here, and only when the caller passes none."""
    import torch
    B, nh, hd = cache.c.B, cache.c.n_heads, cache.c.head_dim
    if out is None:
        out = _empty((B, nh * hd), torch.float16, q.device)
    _check(lib().fg_decode_attention_noalloc(_ptr(q), q_stride, ctypes.byref(cache.c), _ptr(out), _stream(stream)))
    return out


def fg_prefill_attention(qkv, B: int, L: int, n_heads: int, head_dim: int, out=None, stream=None):
    import torch
    if out is None:
        out = _empty((B * L, n_heads * head_dim), torch.float16, qkv.device)
    _check(lib().fg_prefill_attention(_ptr(qkv), B, L, n_heads, head_dim, _ptr(out), _stream(stream)))
    return out


def fg_layernorm(x, g, b, y=None, stream=None):
    rows, cols = x.shape
    if y is None:
        y = _empty((rows, cols), x.dtype, x.device)
    _check(lib().fg_layernorm(_ptr(x), rows, cols, _ptr(g), _ptr(b), _ptr(y), _stream(stream)))
    return y


def fg_embed(ids, pos0: int, E, P, out=None, stream=None):
    import torch
    B, T = ids.shape
    h = E.shape[1]
    if out is None:
        out = _empty((B * T, h), torch.float16, E.device)
    _check(lib().fg_embed(_ptr(ids), B, T, pos0, _ptr(E), _ptr(P), h, _ptr(out), _stream(stream)))
    return out


def fg_lm_head_argmax(x, E, logits=None, tokens=None, workspace=None, stream=None):
    import torch
    B, h = x.shape
    V = E.shape[0]
    if tokens is None:
        tokens = _empty((B,), torch.int32, x.device)
    if logits is None and workspace is None:
        workspace = _empty((lib().fg_lm_head_workspace_bytes(B, V),), torch.uint8, x.device)
    _check(lib().fg_lm_head_argmax(_ptr(x), B, h, _ptr(E), V, _ptr(logits), _ptr(tokens), _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(stream)))
    return tokens


_torch = None


def _ragged(stream):
    """torch, the current device and the raw stream of a ragged-batch call (launched on that device)."""
    global _torch
    if _torch is None:
        import torch
        torch.cuda.init()
        _torch = torch
    dev = _torch._C._cuda_getDevice()
    if stream is None:
        return _torch, dev, _torch._C._cuda_getCurrentRawStream(dev)
    return _torch, dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _made(shape, dtype, dev, st, zero=False):
    """A new tensor that belongs to the stream `st` of the call: its memory is filled and given back in that stream's
    order, whatever the current stream does with the allocator meanwhile."""
    new = _torch.zeros if zero else _torch.empty
    if st == _torch._C._cuda_getCurrentRawStream(dev):
        return new(shape, dtype=dtype, device=dev)
    with _torch.cuda.stream(_torch.cuda.ExternalStream(st, device=dev)):
        return new(shape, dtype=dtype, device=dev)


def _index(t, n, dtype, dev, what):
    """An index or per-row array of a ragged batch: on the current device, contiguous, at least n values."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor of at least {n} values on the current CUDA device")
    return t.data_ptr()


def _rows(t, n_rows, cols, stride, dev, what, stated=False):
    """fp16 rows `stride` elements apart on the current device: those of the tensor's first dimension, each contiguous, or
    of a contiguous tensor cut into rows.  Where the caller states the stride, a flat buffer or a tensor of one row names
    the start of the rows, and the last of them must lie inside its storage."""
    if t.dtype is not _torch.float16 or t.get_device() != dev:
        raise ValueError(f"{what}: an fp16 tensor on the current CUDA device")
    if n_rows <= 0 or (t.dim() == 2 and t.stride(0) == stride and t.size(0) >= n_rows and t.size(1) >= cols
                       and t.stride(1) == 1):
        return t.data_ptr()
    inner = 1                       # values of a row, 0 when they do not lie together
    for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        inner = inner * size if step == inner or size == 1 else 0
    if t.dim() >= 2 and t.size(0) >= n_rows and inner >= cols and (n_rows == 1 or t.stride(0) == stride):
        return t.data_ptr()
    need = (n_rows - 1) * stride + cols
    if not stated:
        fits = t.is_contiguous() and need <= t.numel() and (t.dim() == 1 or inner and stride % inner == 0)
    else:
        fits = (t.is_contiguous() or inner and (t.size(0) == 1 or t.dim() >= 2 and t.stride(0) == stride)) \
            and need <= t.untyped_storage().nbytes() // 2 - t.storage_offset()
    if not fits or stride < cols:
        raise ValueError(f"{what}: {n_rows} rows of {cols} values, {stride} apart, are not those of the tensor")
    return t.data_ptr()


def _bytes(t, dev, what):
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor on the current CUDA device")
    return t.data_ptr(), t.numel() * t.element_size()


def fg_paged_append(cache: DevicePagedKVCache, k, v, row_stride: int, n_rows: int, pos0, row_start=None, stream=None):
    """Quantize n_rows K/V rows into the pages; row_start int32 [B + 1] (None: one row per sequence)."""
    torch, dev, st = _ragged(stream)
    c, i32 = cache.c, torch.int32
    cache.check(dev)
    _check(lib().fg_paged_append(cache.ref, _rows(k, n_rows, cache.h, row_stride, dev, "k", True),
                                 _rows(v, n_rows, cache.h, row_stride, dev, "v", True), row_stride, n_rows,
                                 _index(row_start, c.B + 1, i32, dev, "row_start"), _index(pos0, c.B, i32, dev, "pos0"), st))


def fg_paged_read(cache: DevicePagedKVCache, n_rows: int, row_start, pos0=None, k=None, v=None, stream=None):
    """Dequantized fp16 rows (k, v) [n_rows, n_kv*hd] of the cached positions; `k` and `v` may be
    given (the same row stride), otherwise they are made with zeros in rows of no sequence."""
    torch, dev, st = _ragged(stream)
    c, i32 = cache.c, torch.int32
    cache.check(dev)
    if k is None:
        k = _made((n_rows, cache.h), torch.float16, dev, st, zero=True)
    if v is None:
        v = _made((n_rows, cache.h), torch.float16, dev, st, zero=True)
    stride = k.stride(0)
    if n_rows > 1 and v.stride(0) != stride:
        raise ValueError("k and v must have the same row stride")
    _check(lib().fg_paged_read(cache.ref, n_rows, _index(row_start, c.B + 1, i32, dev, "row_start"),
                               _index(pos0, c.B, i32, dev, "pos0"), _rows(k, n_rows, cache.h, stride, dev, "k"),
                               _rows(v, n_rows, cache.h, stride, dev, "v"), stride, st))
    return k, v


def fg_paged_attention_workspace_bytes(n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return lib().fg_paged_attention_workspace_bytes(n_heads, n_kv_heads, head_dim)


def fg_paged_attention(q, q_stride: int, cache: DevicePagedKVCache, lens, n_heads: int, window: int = 0, n_sink: int = 0,
                       out=None, workspace=None, stream=None):
    """One query token per sequence over the paged cache; lens int32 [B] on the device."""
    torch, dev, st = _ragged(stream)
    B, h = cache.c.B, n_heads * cache.c.head_dim
    cache.check(dev)
    if out is None:
        out = _made((B, h), torch.float16, dev, st)
    if workspace is None:
        workspace = _made((fg_paged_attention_workspace_bytes(n_heads, cache.c.n_kv_heads, cache.c.head_dim),),
                          torch.uint8, dev, st)
    _check(lib().fg_paged_attention(_rows(q, B, h, q_stride, dev, "q", True), q_stride, cache.ref,
                                    _index(lens, B, torch.int32, dev, "lens"), n_heads, window, n_sink,
                                    _rows(out, B, h, h, dev, "out"), *_bytes(workspace, dev, "workspace"), st))
    return out


def fg_varlen_attention(q, k, v, q_start, k_start, max_q: int, n_heads: int, n_kv_heads: int, head_dim: int,
                        window: int = 0, n_sink: int = 0, out=None, stream=None):
    """Causal attention over packed rows: q [n_q, n_heads*hd], k, v [n_k, n_kv*hd] (views of wider
    rows allowed), q_start and k_start int32 [B + 1] on the device; a sequence's queries are the
    last of its positions.  `out` is made with zeros in rows of no sequence when not given."""
    torch, dev, st = _ragged(stream)
    B, h, hk = q_start.numel() - 1, n_heads * head_dim, n_kv_heads * head_dim
    n_q, n_k = q.shape[0], k.shape[0]
    # the stride of a single row says nothing: take one that the calls accept
    qs, ks = q.stride(0) if n_q > 1 else h, k.stride(0) if n_k > 1 else hk
    if v.shape[0] != n_k or (n_k > 1 and v.stride(0) != ks):
        raise ValueError("k and v must have the same rows and row stride")
    if out is None:
        out = _made((n_q, h), torch.float16, dev, st, zero=True)
    _check(lib().fg_varlen_attention(_rows(q, n_q, h, qs, dev, "q"), qs, n_q, _rows(k, n_k, hk, ks, dev, "k"),
                                     _rows(v, n_k, hk, ks, dev, "v"), ks, n_k,
                                     _index(q_start, B + 1, torch.int32, dev, "q_start"),
                                     _index(k_start, B + 1, torch.int32, dev, "k_start"), B, max_q, n_heads, n_kv_heads,
                                     head_dim, window, n_sink, _rows(out, n_q, h, h, dev, "out"), st))
    return out


def _sample_args(torch, dev, B, temperature, top_k, top_p, min_p, u):
    f = torch.float32
    if u is None:
        raise ValueError("u: a uniform number per row")
    return (_index(temperature, B, f, dev, "temperature"), _index(top_k, B, torch.int32, dev, "top_k"),
            _index(top_p, B, f, dev, "top_p"), _index(min_p, B, f, dev, "min_p"), _index(u, B, f, dev, "u"))


def fg_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprob=None, stream=None):
    """One token per row of fp32 logits [B, V], drawn with the uniform numbers u [B]; temperature,
    top_k (int32), top_p and min_p are per-row CUDA tensors or None.  Returns int32 tokens [B];
    `logprob` fp32 [B] receives the drawn token's log probability."""
    torch, dev, st = _ragged(stream)
    B, V = logits.shape
    if logits.dtype is not torch.float32 or logits.get_device() != dev or (V > 1 and logits.stride(1) != 1):
        raise ValueError("logits: an fp32 tensor [B, V] on the current CUDA device, contiguous along V")
    if tokens is None:
        tokens = _made((B,), torch.int32, dev, st)
    _check(lib().fg_sample(logits.data_ptr(), logits.stride(0) if B > 1 else V, B, V,
                           *_sample_args(torch, dev, B, temperature, top_k, top_p, min_p, u),
                           _index(tokens, B, torch.int32, dev, "tokens"),
                           _index(logprob, B, torch.float32, dev, "logprob"), st))
    return tokens


def fg_lm_head_sample(x, E, u, temperature=None, top_k=None, top_p=None, min_p=None, logits=None, tokens=None,
                      logprob=None, workspace=None, stream=None):
    """fg_lm_head_argmax with fg_sample in the place of the arg max."""
    torch, dev, st = _ragged(stream)
    B, h = x.shape
    V = E.shape[0]
    if tokens is None:
        tokens = _made((B,), torch.int32, dev, st)
    if logits is None and workspace is None:
        workspace = _made((lib().fg_lm_head_workspace_bytes(B, V),), torch.uint8, dev, st)
    _check(lib().fg_lm_head_sample(_rows(x, B, h, h, dev, "x"), B, h, _rows(E, V, h, h, dev, "E"), V,
                                   _index(logits, B * V, torch.float32, dev, "logits"),
                                   *_sample_args(torch, dev, B, temperature, top_k, top_p, min_p, u),
                                   _index(tokens, B, torch.int32, dev, "tokens"),
                                   _index(logprob, B, torch.float32, dev, "logprob"),
                                   *_bytes(workspace, dev, "workspace"), st))
    return tokens


def fg_decode_layer(layer: DeviceLayer, cache: DeviceKVCache, x_in, x_out=None, workspace=None, stream=None):
    import torch
    B, h = x_in.shape
    F = layer.fc1.N
    if x_out is None:
        x_out = _empty((B, h), torch.float16, x_in.device)
    if workspace is None:
        wsb = lib().fg_decode_layer_workspace_bytes(h, F, cache.c.n_heads, B, cache.c.capacity)
        workspace = _empty((wsb,), torch.uint8, x_in.device)
    _check(lib().fg_decode_layer(ctypes.byref(layer.c), ctypes.byref(cache.c), _ptr(x_in), _ptr(x_out), B,
                                 _ptr(workspace), workspace.numel(), _stream(stream)))
    return x_out


def fg_prefill_layer(layer: DeviceLayer, cache: DeviceKVCache, x, B: int, L: int, workspace=None, stream=None):
    import torch
    h = x.shape[-1]
    F = layer.fc1.N
    if workspace is None:
        wsb = lib().fg_prefill_layer_workspace_bytes(h, F, B, L)
        workspace = _empty((wsb,), torch.uint8, x.device)
    _check(lib().fg_prefill_layer(ctypes.byref(layer.c), ctypes.byref(cache.c), _ptr(x), B, L, _ptr(workspace),
                                  workspace.numel(), _stream(stream)))
    return x


def fg_workspace_bytes(model: DeviceModel, B: int, L: int, gen_len: int) -> int:
    return lib().fg_workspace_bytes(ctypes.byref(model.c), B, L, gen_len)


def fg_generate(model: DeviceModel, prompt_ids, gen_len: int, caches, out_ids=None, workspace=None,
                stream=None):
    """Greedy generation; returns (out_ids int32 [B, gen_len] on the device, Timing)."""
    import torch
    B, L = prompt_ids.shape
    if out_ids is None:
        out_ids = _empty((B, gen_len), torch.int32, prompt_ids.device)
    if workspace is None:
        workspace = _empty((fg_workspace_bytes(model, B, L, gen_len),), torch.uint8, prompt_ids.device)
    arr = (KVCache * len(caches))(*[c.c for c in caches])
    timing = Timing()
    st = lib().fg_generate(ctypes.byref(model.c), _ptr(prompt_ids), B, L, gen_len, _ptr(out_ids), arr,
                           _ptr(workspace), workspace.numel(), ctypes.byref(timing), _stream(stream))
    for i, c in enumerate(caches):
        c.c.len = arr[i].len
    _check(st)
    return out_ids, timing


def pinned_layer(layer: DeviceLayer) -> DeviceLayer:
    """A copy of a layer whose tensors live in pinned host memory (for fg_generate_offload)."""
    def pin(t):
        return None if t is None else t.detach().cpu().pin_memory()

    def lin(q: DeviceQLinear) -> DeviceQLinear:
        return DeviceQLinear(pin(q.codes), pin(q.params), pin(q.bias), q.K, q.N, q.group, pin(q.w16), q.along_k)
    return DeviceLayer(*[pin(t) for t in layer.t], lin(layer.qkv), lin(layer.out), lin(layer.fc1), lin(layer.fc2))


def fg_offload_workspace_bytes(model: DeviceModel, B: int, L: int, gen_len: int) -> int:
    return lib().fg_offload_workspace_bytes(ctypes.byref(model.c), B, L, gen_len)


def fg_generate_offload(model: DeviceModel, prompt_ids, gen_len: int, caches, out_ids=None, workspace=None,
                        stream=None):
    """Greedy generation with the layers' weights in pinned host memory, streamed to the GPU
    layer by layer; returns (out_ids int32 [B, gen_len] on the device, Timing, h2d bytes)."""
    import torch
    B, L = prompt_ids.shape
    if out_ids is None:
        out_ids = _empty((B, gen_len), torch.int32, prompt_ids.device)
    if workspace is None:
        workspace = _empty((fg_offload_workspace_bytes(model, B, L, gen_len),), torch.uint8, prompt_ids.device)
    arr = (KVCache * len(caches))(*[c.c for c in caches])
    timing = Timing()
    h2d = c_double()
    st = lib().fg_generate_offload(ctypes.byref(model.c), _ptr(prompt_ids), B, L, gen_len, _ptr(out_ids), arr,
                                   _ptr(workspace), workspace.numel(), ctypes.byref(timing), ctypes.byref(h2d),
                                   _stream(stream))
    for i, c in enumerate(caches):
        c.c.len = arr[i].len
    _check(st)
    return out_ids, timing, h2d.value


def fg_profile_enable(on: bool = True):
    _check(lib().fg_profile_enable(int(on)))


def fg_profile_select(kinds=None):
    """Time only these kinds (indices into PROF_NAMES) while profiling is on; None = all."""
    mask = (1 << len(PROF_NAMES)) - 1 if kinds is None else sum(1 << int(k) for k in kinds)
    _check(lib().fg_profile_select(mask))


def fg_profile_reset():
    _check(lib().fg_profile_reset())


def fg_launch_count() -> int:
    return lib().fg_launch_count()


def fg_profile_read(kind: int):
    ms, n, fl, by = c_double(), c_int64(), c_double(), c_double()
    _check(lib().fg_profile_read(kind, ctypes.byref(ms), ctypes.byref(n), ctypes.byref(fl), ctypes.byref(by)))
    return {"ms": ms.value, "launches": n.value, "flops": fl.value, "bytes": by.value}
