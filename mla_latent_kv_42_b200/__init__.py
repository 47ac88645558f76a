"""Python binding of libmla, the MLA absorbed-decode library for B200 (sm_100a).

Argument marshalling only: every step of the path runs in libmla's CUDA kernels, reached
through the C ABI of ``include/mla.h``. Torch supplies device memory and streams. If the
shared library is missing, every call raises; there is no fallback of any kind.

A call given a ``stream`` is queued there and takes the outputs and workspaces that the caller did
not pass from that stream's memory, so that they may be used at once; that the inputs are ready
there, and the outputs are not read before, is the caller's to order (``wait_stream``, events).

Method: "DeepSeek-V2 from Scratch", §6 (the complete MLA algorithm) in the absorbed form of
§5.3: append the new token's latent row, absorb W^UK into the query, attend in latent space,
fold W^UV into the output projection.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

__all__ = [
    "MLAError", "load_library", "library_path", "c_dims", "workspace_size", "cache_elems_per_token",
    "append_kv", "absorb_query", "decode_attention", "decode_attention_noalloc", "prefill_attention", "out_proj",
    "read_device_status", "last_launch_count", "LayerState", "layer_step", "layer_step_small",
    "layer_step_small_supported", "fp8_page_bytes", "fp8_supported", "append_kv_fp8", "decode_attention_fp8",
    "CALL_APPEND_KV", "CALL_ABSORB_QUERY", "CALL_DECODE_ATTENTION", "CALL_OUT_PROJ", "CALL_PREFILL_ATTENTION",
    "CALL_LAYER_STEP_SMALL", "CALL_APPEND_KV_FP8", "CALL_DECODE_ATTENTION_FP8",
    "norm_append_kv", "norm_append_kv_fp8", "read_kv", "read_kv_fp8", "shared_prefix_attention",
    "CALL_NORM_APPEND_KV", "CALL_NORM_APPEND_KV_FP8", "CALL_READ_KV", "CALL_READ_KV_FP8",
    "CALL_SHARED_PREFIX_ATTENTION",
]

CALL_APPEND_KV, CALL_ABSORB_QUERY, CALL_DECODE_ATTENTION, CALL_OUT_PROJ, CALL_PREFILL_ATTENTION = 0, 1, 2, 3, 4
CALL_LAYER_STEP_SMALL = 5
CALL_APPEND_KV_FP8, CALL_DECODE_ATTENTION_FP8 = 6, 7
CALL_NORM_APPEND_KV, CALL_NORM_APPEND_KV_FP8, CALL_READ_KV, CALL_READ_KV_FP8 = 9, 10, 11, 12
CALL_SHARED_PREFIX_ATTENTION = 13
_PKG = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_PKG, "libmla.so")


class MLAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_lib().mla_error_string(code).decode()} ({code})")


class _Dims(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("d_head", ctypes.c_int32),
                ("d_c", ctypes.c_int32), ("d_cq", ctypes.c_int32), ("d_rope", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rope_base", ctypes.c_double),
                ("rope_inv_freq", ctypes.c_void_p)]


_LIB = None
_P, _I32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_I64, _F64 = ctypes.c_int64, ctypes.c_double
_SIGS = {
    "mla_check_dims": (ctypes.c_int, [_P]),
    "mla_cache_elems_per_token": (_I32, [_P]),
    "mla_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "mla_append_kv": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _P, _SZ, _P]),
    "mla_absorb_query": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _I32, _P, _SZ, _P]),
    "mla_decode_attention": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "mla_prefill_attention": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _SZ,
                                             _P]),
    "mla_out_proj": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _SZ, _P]),
    "mla_read_device_status": (ctypes.c_int, [_P, ctypes.POINTER(_I32)]),
    "mla_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mla_last_launch_count": (_I32, [_I32]),
    "mla_decode_attention_noalloc": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _P]),
    "mla_set_decode_timing_events": (ctypes.c_int, [_P, _P]),
    "mla_debug_inject_missing_load": (ctypes.c_int, [_I32]),
    "mla_layer_step_small_supported": (ctypes.c_int, [_P]),
    "mla_fp8_page_bytes": (ctypes.c_int64, [_P]),
    "mla_fp8_supported": (ctypes.c_int, [_P]),
    "mla_append_kv_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _P, _SZ, _P]),
    "mla_decode_attention_fp8": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "mla_norm_append_kv": (ctypes.c_int, [_P, _P, _I64, _P, _P, _F64, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _P]),
    "mla_norm_append_kv_fp8": (ctypes.c_int, [_P, _P, _I64, _P, _P, _F64, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _P]),
    "mla_read_kv": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _I32, _I32, _P, _I64, _I32, _P]),
    "mla_read_kv_fp8": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _I32, _I32, _P, _I64, _I32, _P]),
    "mla_shared_prefix_attention": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _P, _I32, _P, _P, _P,
                                                   _SZ, _P]),
    "mla_layer_step_small": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _P, _P,
                                            _P, _P, _P, _SZ, _P]),
}


def load_library(path: str | None = None):
    """Load libmla.so (built by ``python -m mla_latent_kv_42_b200.build``); raise if absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"libmla.so is not built ({p}); run `python -m mla_latent_kv_42_b200.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        _LIB = lib
    return lib


_lib = load_library


_ROPE_TABLES = {}


def _rope_table_ptr(d):
    """Device copy (float64, current device) of a dims' RoPE frequency table, or None. The copies are
    kept for the life of the process so that queued kernels can still read them."""
    table = getattr(d, "rope_inv_freq", None)
    if table is None:
        return None
    import torch
    key = (tuple(float(x) for x in table), torch.cuda.current_device())
    t = _ROPE_TABLES.get(key)
    if t is None:
        if len(key[0]) != d.d_rope // 2:
            raise ValueError(f"rope_inv_freq has {len(key[0])} entries, d_rope/2 = {d.d_rope // 2}")
        t = torch.tensor(key[0], dtype=torch.float64, device="cuda")
        _ROPE_TABLES[key] = t
    return t.data_ptr()


def c_dims(d) -> _Dims:
    """mla_dims from a ``synth.Dims`` (or anything with the same attributes). A dims with a RoPE
    frequency table (``rope_inv_freq``, d_rope/2 floats) gets a device copy of it."""
    return _Dims(d.d_model, d.n_heads, d.d_head, d.d_c, d.d_cq, d.d_rope, d.page_size,
                 {"bf16": 0, "fp16": 1}[d.dtype], float(d.rope_base), _rope_table_ptr(d))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, what: str):
    if code != 0:
        raise MLAError(code, what)


def _need(t, dtype, name, dims=None):
    import torch
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _elem(d):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[d.dtype]


def workspace_size(dims, call: int, B: int, max_seq_len: int = 0) -> int:
    cd = c_dims(dims)
    return int(_lib().mla_workspace_size(ctypes.byref(cd), call, B, max_seq_len))


def cache_elems_per_token(dims) -> int:
    cd = c_dims(dims)
    return int(_lib().mla_cache_elems_per_token(ctypes.byref(cd)))


def _own(stream, like, shape, dtype):
    """A tensor of a call's own on the device of ``like``, from the memory of the stream that the call
    runs on: what another stream's tensors have freed may still be in use there."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _out(stream, like, shape, dtype):
    """The same for an output, which the caller's current stream may read: once freed it is also kept
    from reuse until that stream is through with what it has queued by then."""
    t = _own(stream, like, shape, dtype)
    if stream is not None:
        import torch
        t.record_stream(torch.cuda.current_stream())
    return t


def _ws(dims, call, B, max_seq_len, ws, stream, like):
    import torch
    n = workspace_size(dims, call, B, max_seq_len)
    if ws is None:
        ws = _own(stream, like, max(n, 16), torch.uint8)
    return ws, ws.numel() * ws.element_size()


def append_kv(dims, h, w_dkv_kr, seq_idx, pos, block_table, pool, ws=None, stream=None):
    """mla_append_kv: write [c ‖ RoPE(k^)] of each new token into its paged slot of ``pool``."""
    import torch
    e = _elem(dims)
    for t, n, dt in ((h, "h", e), (w_dkv_kr, "w_dkv_kr", e), (seq_idx, "seq_idx", torch.int32),
                     (pos, "pos", torch.int32), (block_table, "block_table", torch.int32), (pool, "pool", e)):
        _need(t, dt, n)
    T = h.shape[0]
    ws, nbytes = _ws(dims, CALL_APPEND_KV, T, 0, ws, stream, h)
    cd = c_dims(dims)
    _check(_lib().mla_append_kv(ctypes.byref(cd), _ptr(h), _ptr(w_dkv_kr), _ptr(seq_idx), _ptr(pos),
                                _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(pool),
                                pool.shape[0], T, _ptr(ws), nbytes, _stream(stream)), "mla_append_kv")
    return pool


def absorb_query(dims, h, w_dq, w_uq_qr, w_uk, pos, q_out=None, ws=None, stream=None):
    """mla_absorb_query: q_out[b][i] = [(W^UK_i)^T q^C_i ‖ RoPE(q^_i, pos[b])]."""
    import torch
    e = _elem(dims)
    for t, n, dt in ((h, "h", e), (w_dq, "w_dq", e), (w_uq_qr, "w_uq_qr", e), (w_uk, "w_uk", e),
                     (pos, "pos", torch.int32)):
        _need(t, dt, n)
    B = h.shape[0]
    if q_out is None:
        q_out = _out(stream, h, (B, dims.n_heads, dims.d_c + dims.d_rope), e)
    _need(q_out, e, "q_out")
    ws, nbytes = _ws(dims, CALL_ABSORB_QUERY, B, 0, ws, stream, h)
    cd = c_dims(dims)
    _check(_lib().mla_absorb_query(ctypes.byref(cd), _ptr(h), _ptr(w_dq), _ptr(w_uq_qr), _ptr(w_uk), _ptr(pos),
                                   _ptr(q_out), B, _ptr(ws), nbytes, _stream(stream)), "mla_absorb_query")
    return q_out


def decode_attention(dims, q, pool, block_table, seq_lens, max_seq_len, o_lat=None, lse=None, want_lse=True,
                     ws=None, stream=None):
    """mla_decode_attention: latent-space softmax attention of every head over its sequence's cache."""
    import torch
    e = _elem(dims)
    for t, n, dt in ((q, "q", e), (pool, "pool", e), (block_table, "block_table", torch.int32),
                     (seq_lens, "seq_lens", torch.int32)):
        _need(t, dt, n)
    B = q.shape[0]
    if o_lat is None:
        o_lat = _out(stream, q, (B, dims.n_heads, dims.d_c), e)
    if lse is None and want_lse:
        lse = _out(stream, q, (B, dims.n_heads), torch.float32)
    _need(o_lat, e, "o_lat")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    ws, nbytes = _ws(dims, CALL_DECODE_ATTENTION, B, max_seq_len, ws, stream, q)
    cd = c_dims(dims)
    _check(_lib().mla_decode_attention(ctypes.byref(cd), _ptr(q), _ptr(pool), pool.shape[0], _ptr(block_table),
                                       block_table.shape[1], _ptr(seq_lens), B, int(max_seq_len), _ptr(o_lat),
                                       _ptr(lse), _ptr(ws), nbytes, _stream(stream)), "mla_decode_attention")
    return o_lat, lse


def fp8_page_bytes(dims) -> int:
    """Bytes of one FP8 cache page: page_size rows of d_c + d_rope e4m3 bytes, then page_size
    float32 pairs (s_c, s_r)."""
    cd = c_dims(dims)
    return int(_lib().mla_fp8_page_bytes(ctypes.byref(cd)))


def fp8_supported(dims) -> bool:
    cd = c_dims(dims)
    return _lib().mla_fp8_supported(ctypes.byref(cd)) == 0


def append_kv_fp8(dims, h, w_dkv_kr, seq_idx, pos, block_table, pool, ws=None, stream=None):
    """mla_append_kv_fp8: the rows of mla_append_kv, quantised to e4m3 with two scales per token,
    into ``pool`` (uint8 [num_pages, fp8_page_bytes(dims)])."""
    import torch
    e = _elem(dims)
    for t, n, dt in ((h, "h", e), (w_dkv_kr, "w_dkv_kr", e), (seq_idx, "seq_idx", torch.int32),
                     (pos, "pos", torch.int32), (block_table, "block_table", torch.int32), (pool, "pool", torch.uint8)):
        _need(t, dt, n)
    if pool.dim() != 2 or pool.shape[1] != fp8_page_bytes(dims):
        raise ValueError("pool must be uint8 [num_pages, fp8_page_bytes(dims)]")
    T = h.shape[0]
    ws, nbytes = _ws(dims, CALL_APPEND_KV_FP8, T, 0, ws, stream, h)
    cd = c_dims(dims)
    _check(_lib().mla_append_kv_fp8(ctypes.byref(cd), _ptr(h), _ptr(w_dkv_kr), _ptr(seq_idx), _ptr(pos),
                                    _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(pool),
                                    pool.shape[0], T, _ptr(ws), nbytes, _stream(stream)), "mla_append_kv_fp8")
    return pool


def decode_attention_fp8(dims, q, pool, block_table, seq_lens, max_seq_len, o_lat=None, lse=None, want_lse=True,
                         ws=None, stream=None):
    """mla_decode_attention_fp8: mla_decode_attention over an FP8 cache (uint8 [num_pages,
    fp8_page_bytes(dims)])."""
    import torch
    e = _elem(dims)
    for t, n, dt in ((q, "q", e), (pool, "pool", torch.uint8), (block_table, "block_table", torch.int32),
                     (seq_lens, "seq_lens", torch.int32)):
        _need(t, dt, n)
    if pool.dim() != 2 or pool.shape[1] != fp8_page_bytes(dims):
        raise ValueError("pool must be uint8 [num_pages, fp8_page_bytes(dims)]")
    B = q.shape[0]
    if o_lat is None:
        o_lat = _out(stream, q, (B, dims.n_heads, dims.d_c), e)
    if lse is None and want_lse:
        lse = _out(stream, q, (B, dims.n_heads), torch.float32)
    _need(o_lat, e, "o_lat")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    ws, nbytes = _ws(dims, CALL_DECODE_ATTENTION_FP8, B, max_seq_len, ws, stream, q)
    cd = c_dims(dims)
    _check(_lib().mla_decode_attention_fp8(ctypes.byref(cd), _ptr(q), _ptr(pool), pool.shape[0], _ptr(block_table),
                                           block_table.shape[1], _ptr(seq_lens), B, int(max_seq_len), _ptr(o_lat),
                                           _ptr(lse), _ptr(ws), nbytes, _stream(stream)), "mla_decode_attention_fp8")
    return o_lat, lse


def prefill_attention(dims, q, pool, block_table, seq_idx, pos, max_seq_len, o_lat=None, lse=None, want_lse=True,
                      ws=None, stream=None):
    """mla_prefill_attention: causal latent attention of several new tokens per sequence.

    Token t (sequence ``seq_idx[t]``, position ``pos[t]``) attends to its sequence's cached
    positions 0..pos[t]; the new tokens' rows must already be appended.
    """
    import torch
    e = _elem(dims)
    for t, n, dt in ((q, "q", e), (pool, "pool", e), (block_table, "block_table", torch.int32),
                     (seq_idx, "seq_idx", torch.int32), (pos, "pos", torch.int32)):
        _need(t, dt, n)
    T = q.shape[0]
    if o_lat is None:
        o_lat = _out(stream, q, (T, dims.n_heads, dims.d_c), e)
    if lse is None and want_lse:
        lse = _out(stream, q, (T, dims.n_heads), torch.float32)
    _need(o_lat, e, "o_lat")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    ws, nbytes = _ws(dims, CALL_PREFILL_ATTENTION, T, max_seq_len, ws, stream, q)
    cd = c_dims(dims)
    _check(_lib().mla_prefill_attention(ctypes.byref(cd), _ptr(q), _ptr(pool), pool.shape[0], _ptr(block_table),
                                        block_table.shape[0], block_table.shape[1], _ptr(seq_idx), _ptr(pos), T,
                                        int(max_seq_len), _ptr(o_lat), _ptr(lse), _ptr(ws), nbytes,
                                        _stream(stream)), "mla_prefill_attention")
    return o_lat, lse


def decode_attention_noalloc(dims, q, pool, block_table, seq_lens, max_seq_len, o_lat=None, lse=None,
                             want_lse=True, stream=None):
    """mla_decode_attention_noalloc: the same attention with the library's static scratch.

    For callers that cannot allocate device memory when they decode (memory reserved up front
    by their own allocator, no tolerance for cudaMalloc's synchronisation, no workspace
    allocator). Problems needing more than 64 MiB of split-KV scratch raise MLAError (-3).
    The scratch is shared by every call on the device: calls overlapping on the GPU race.
    """
    import torch
    e = _elem(dims)
    for t, n, dt in ((q, "q", e), (pool, "pool", e), (block_table, "block_table", torch.int32),
                     (seq_lens, "seq_lens", torch.int32)):
        _need(t, dt, n)
    B = q.shape[0]
    if o_lat is None:
        o_lat = _out(stream, q, (B, dims.n_heads, dims.d_c), e)
    if lse is None and want_lse:
        lse = _out(stream, q, (B, dims.n_heads), torch.float32)
    _need(o_lat, e, "o_lat")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    cd = c_dims(dims)
    _check(_lib().mla_decode_attention_noalloc(ctypes.byref(cd), _ptr(q), _ptr(pool), pool.shape[0],
                                               _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B,
                                               int(max_seq_len), _ptr(o_lat), _ptr(lse), _stream(stream)),
           "mla_decode_attention_noalloc")
    return o_lat, lse


def out_proj(dims, o_lat, w_uv, w_o, u=None, ws=None, stream=None):
    """mla_out_proj: u = W^O [W^UV_1 o_lat_1; ...; W^UV_n_h o_lat_n_h]."""
    e = _elem(dims)
    for t, n in ((o_lat, "o_lat"), (w_uv, "w_uv"), (w_o, "w_o")):
        _need(t, e, n)
    B = o_lat.shape[0]
    if u is None:
        u = _out(stream, o_lat, (B, dims.d_model), e)
    _need(u, e, "u")
    ws, nbytes = _ws(dims, CALL_OUT_PROJ, B, 0, ws, stream, o_lat)
    cd = c_dims(dims)
    _check(_lib().mla_out_proj(ctypes.byref(cd), _ptr(o_lat), _ptr(w_uv), _ptr(w_o), _ptr(u), B, _ptr(ws), nbytes,
                               _stream(stream)), "mla_out_proj")
    return u


# The row and shared-prefix calls are short on the device (2 us for a decode step's rows), so their
# host side is kept short too: one expression decides whether every tensor is as the call needs it,
# and only a failed one looks closer.
def _ok(t, dtype, shape, here):
    return t.dtype is dtype and t.get_device() == here and t.shape == shape and t.is_contiguous()


def _refuse(here, *named, strided=None):
    """Raise for the first (tensor, name, dtype, shape) that is not on the current device, contiguous (but
    for the rows of the one called ``strided``), with that type and shape; always raises."""
    for t, name, dtype, shape in named:
        if t.get_device() < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != here:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            if name != strided:
                raise ValueError(f"{name} must be contiguous")
            if t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < shape[1]:
                raise ValueError(f"{name} must be contiguous but for its rows, a multiple of 8 elements apart")
    raise ValueError("arguments refused: " + ", ".join(f"{name} {tuple(t.shape)} {t.dtype}" for t, name, *_ in named))


def _rows_ok(t, dtype, shape, here):
    """_ok for a tensor whose rows may be strided (a slice of a wider product)."""
    return _ok(t, dtype, shape, here) or (t.dtype is dtype and t.get_device() == here and t.shape == shape
                                          and t.stride(1) == 1 and t.stride(0) % 8 == 0 and t.stride(0) >= shape[1])


def _sizes(t, n, name):
    """Shape of ``t``, which must have n dimensions."""
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _pool_shape(dims, pool, fp8):
    D = dims.d_c + dims.d_rope
    n = pool.shape[0] if pool.dim() else 0
    return (n, dims.page_size * (D + 8)) if fp8 else (n, dims.page_size, D)


def _raw_stream(torch, here, stream):
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _norm_append(fn, name, fp8, dims, x, seq_idx, pos, block_table, pool, gain_c, gain_r, eps, stream):
    import torch
    e, i32 = _elem(dims), torch.int32
    here = torch.cuda.current_device()
    T, D = _sizes(x, 2, "x")[0], dims.d_c + dims.d_rope
    S, width = _sizes(block_table, 2, "block_table")
    shape = _pool_shape(dims, pool, fp8)
    pool_type = torch.uint8 if fp8 else e
    if not (_rows_ok(x, e, (T, D), here) and _ok(seq_idx, i32, (T,), here) and _ok(pos, i32, (T,), here)
            and _ok(block_table, i32, (S, width), here) and _ok(pool, pool_type, shape, here)
            and (gain_c is None or _ok(gain_c, e, (dims.d_c,), here))
            and (gain_r is None or _ok(gain_r, e, (dims.d_rope,), here))):
        _refuse(here, (x, "x", e, (T, D)), (seq_idx, "seq_idx", i32, (T,)), (pos, "pos", i32, (T,)),
                (block_table, "block_table", i32, (S, width)), (pool, "pool", pool_type, shape),
                *([] if gain_c is None else [(gain_c, "gain_c", e, (dims.d_c,))]),
                *([] if gain_r is None else [(gain_r, "gain_r", e, (dims.d_rope,))]), strided="x")
    code = fn(ctypes.byref(c_dims(dims)), x.data_ptr(), x.stride(0) if T > 1 else D,
              None if gain_c is None else gain_c.data_ptr(), None if gain_r is None else gain_r.data_ptr(), eps,
              seq_idx.data_ptr(), pos.data_ptr(), block_table.data_ptr(), S, width, pool.data_ptr(), shape[0], T,
              _raw_stream(torch, here, stream))
    if code:
        raise MLAError(code, name)
    return pool


def norm_append_kv(dims, x, seq_idx, pos, block_table, pool, gain_c=None, gain_r=None, eps=1e-6, stream=None):
    """mla_norm_append_kv: write rows [c ‖ k^] that the caller has (``x`` [T, d_c + d_rope], rows may be
    strided), each part RMS-normalised where its gain is given, k^ rotated, into their slots."""
    return _norm_append(_lib().mla_norm_append_kv, "mla_norm_append_kv", False, dims, x, seq_idx, pos, block_table,
                        pool, gain_c, gain_r, eps, stream)


def norm_append_kv_fp8(dims, x, seq_idx, pos, block_table, pool, gain_c=None, gain_r=None, eps=1e-6, stream=None):
    """mla_norm_append_kv_fp8: the same into ``pool`` (uint8 [num_pages, fp8_page_bytes(dims)])."""
    return _norm_append(_lib().mla_norm_append_kv_fp8, "mla_norm_append_kv_fp8", True, dims, x, seq_idx, pos,
                        block_table, pool, gain_c, gain_r, eps, stream)


def _read(fn, name, fp8, dims, pool, seq_idx, pos, block_table, out, stream):
    import torch
    e, i32 = _elem(dims), torch.int32
    here = torch.cuda.current_device()
    T, D = _sizes(seq_idx, 1, "seq_idx")[0], dims.d_c + dims.d_rope
    S, width = _sizes(block_table, 2, "block_table")
    shape = _pool_shape(dims, pool, fp8)
    pool_type = torch.uint8 if fp8 else e
    if not (_ok(pool, pool_type, shape, here) and _ok(seq_idx, i32, (T,), here) and _ok(pos, i32, (T,), here)
            and _ok(block_table, i32, (S, width), here) and (out is None or _rows_ok(out, e, (T, D), here))):
        _refuse(here, (pool, "pool", pool_type, shape), (seq_idx, "seq_idx", i32, (T,)), (pos, "pos", i32, (T,)),
                (block_table, "block_table", i32, (S, width)),
                *([] if out is None else [(out, "out", e, (T, D))]), strided="out")
    if out is None:
        out = _out(stream, pool, (T, D), e)
    code = fn(ctypes.byref(c_dims(dims)), pool.data_ptr(), shape[0], seq_idx.data_ptr(), pos.data_ptr(),
              block_table.data_ptr(), S, width, out.data_ptr(), out.stride(0) if T > 1 else D, T,
              _raw_stream(torch, here, stream))
    if code:
        raise MLAError(code, name)
    return out


def read_kv(dims, pool, seq_idx, pos, block_table, out=None, stream=None):
    """mla_read_kv: the cached rows of the given (sequence, position) pairs, [T, d_c + d_rope]."""
    return _read(_lib().mla_read_kv, "mla_read_kv", False, dims, pool, seq_idx, pos, block_table, out, stream)


def read_kv_fp8(dims, pool, seq_idx, pos, block_table, out=None, stream=None):
    """mla_read_kv_fp8: the same from an FP8 cache, as element-type rows."""
    return _read(_lib().mla_read_kv_fp8, "mla_read_kv_fp8", True, dims, pool, seq_idx, pos, block_table, out, stream)


def shared_prefix_attention(dims, q, pool, block_table, seq_lens, max_seq_len, shared_pages, o_lat=None, lse=None,
                            want_lse=True, ws=None, stream=None):
    """mla_shared_prefix_attention: decode_attention for a batch whose sequences begin with the pages
    ``shared_pages`` (int32 [num_shared_pages], all full), which are attended once for the batch."""
    import torch
    e, i32, H = _elem(dims), torch.int32, dims.n_heads
    here = torch.cuda.current_device()
    B = _sizes(q, 3, "q")[0]
    width = _sizes(block_table, 2, "block_table")[1]
    n_shared = _sizes(shared_pages, 1, "shared_pages")[0]
    max_seq_len = int(max_seq_len)
    shape, q_shape = _pool_shape(dims, pool, False), (B, H, dims.d_c + dims.d_rope)
    if not (_ok(q, e, q_shape, here) and _ok(pool, e, shape, here) and _ok(block_table, i32, (B, width), here)
            and _ok(seq_lens, i32, (B,), here) and _ok(shared_pages, i32, (n_shared,), here)
            and (o_lat is None or _ok(o_lat, e, (B, H, dims.d_c), here))
            and (lse is None or _ok(lse, torch.float32, (B, H), here))
            and (ws is None or ws.is_contiguous() and ws.get_device() == here)):
        _refuse(here, (q, "q", e, q_shape), (pool, "pool", e, shape), (block_table, "block_table", i32, (B, width)),
                (seq_lens, "seq_lens", i32, (B,)), (shared_pages, "shared_pages", i32, (n_shared,)),
                *([] if o_lat is None else [(o_lat, "o_lat", e, (B, H, dims.d_c))]),
                *([] if lse is None else [(lse, "lse", torch.float32, (B, H))]),
                *([] if ws is None else [(ws, "ws", ws.dtype, ws.shape)]))
    if o_lat is None:
        o_lat = _out(stream, q, (B, H, dims.d_c), e)
    if lse is None and want_lse:
        lse = _out(stream, q, (B, H), torch.float32)
    lib, cd = _lib(), ctypes.byref(c_dims(dims))
    if ws is None:
        n = lib.mla_workspace_size(cd, CALL_SHARED_PREFIX_ATTENTION, B, max_seq_len)
        ws = _own(stream, q, max(n, 16), torch.uint8)
    code = lib.mla_shared_prefix_attention(
        cd, q.data_ptr(), pool.data_ptr(), shape[0], block_table.data_ptr(), width, seq_lens.data_ptr(), B,
        max_seq_len, shared_pages.data_ptr(), n_shared, o_lat.data_ptr(), None if lse is None else lse.data_ptr(),
        ws.data_ptr(), ws.nbytes, _raw_stream(torch, here, stream))
    if code:
        raise MLAError(code, "mla_shared_prefix_attention")
    return o_lat, lse


def read_device_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device status word (0 = no device-side error)."""
    v = ctypes.c_int32(0)
    _check(_lib().mla_read_device_status(_stream(stream), ctypes.byref(v)), "mla_read_device_status")
    return int(v.value)


def last_launch_count(call: int) -> int:
    return int(_lib().mla_last_launch_count(call))


def set_decode_timing_events(before=None, after=None):
    """mla_set_decode_timing_events: record two torch.cuda.Event objects around the attention
    kernel of this thread's later decode calls (None, None: stop). The events must have been
    recorded once (so that they exist) before they are handed over."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    r = _lib().mla_set_decode_timing_events(h(before), h(after))
    if r != 0:
        raise MLAError(r, "mla_set_decode_timing_events")



@dataclass
class LayerState:
    """Device-resident state of one layer: weights and its paged latent cache."""
    dims: object
    w: dict            # w_dkv_kr, w_dq, w_uq_qr, w_uk, w_uv, w_o (CUDA tensors)
    pool: object       # [num_pages, page_size, d_c + d_rope]
    block_table: object  # int32 [B, max_pages]


def layer_step(st: LayerState, h, pos, seq_idx, seq_lens, max_seq_len, ws=None, out=None, stream=None,
               shared_pages=None):
    """One decode step of one layer through the four C-ABI calls; returns (u, q, o_lat, lse).

    ``pos`` = cached length of each sequence (the new token's position), ``seq_lens`` = pos + 1.
    ``ws`` is one byte buffer at least as large as the largest of the four workspaces (the calls
    run in order on one stream, so they can share it). ``shared_pages``: the pages that the sequences
    begin with in common; the attention is then shared_prefix_attention's.
    """
    d, w = st.dims, st.w
    out = out or {}
    append_kv(d, h, w["w_dkv_kr"], seq_idx, pos, st.block_table, st.pool, ws=ws, stream=stream)
    q = absorb_query(d, h, w["w_dq"], w["w_uq_qr"], w["w_uk"], pos, q_out=out.get("q"), ws=ws, stream=stream)
    outs = dict(o_lat=out.get("o_lat"), lse=out.get("lse"), want_lse=out.get("want_lse", True), ws=ws, stream=stream)
    if shared_pages is None:
        o_lat, lse = decode_attention(d, q, st.pool, st.block_table, seq_lens, max_seq_len, **outs)
    else:
        o_lat, lse = shared_prefix_attention(d, q, st.pool, st.block_table, seq_lens, max_seq_len, shared_pages, **outs)
    u = out_proj(d, o_lat, w["w_uv"], w["w_o"], u=out.get("u"), ws=ws, stream=stream)
    return u, q, o_lat, lse


def layer_step_small_supported(dims) -> bool:
    cd = c_dims(dims)
    return _lib().mla_layer_step_small_supported(ctypes.byref(cd)) == 0


def layer_step_small(st: LayerState, h, seq_lens, max_seq_len, ws=None, out=None, stream=None):
    """mla_layer_step_small: the same decode step as ``layer_step`` (one new token per sequence,
    sequence b = batch row b, new token at position seq_lens[b] - 1) in one launch, for small head
    counts; returns (u, q, o_lat, lse)."""
    import torch
    d, w = st.dims, st.w
    out = out or {}
    e = _elem(d)
    B = h.shape[0]
    q = out.get("q")
    if q is None:
        q = _out(stream, h, (B, d.n_heads, d.d_c + d.d_rope), e)
    o_lat = out.get("o_lat")
    if o_lat is None:
        o_lat = _out(stream, h, (B, d.n_heads, d.d_c), e)
    lse = out.get("lse")
    if lse is None and out.get("want_lse", True):
        lse = _out(stream, h, (B, d.n_heads), torch.float32)
    u = out.get("u")
    if u is None:
        u = _out(stream, h, (B, d.d_model), e)
    ws, nbytes = _ws(d, CALL_LAYER_STEP_SMALL, B, max_seq_len, ws, stream, h)
    cd = c_dims(d)
    pool, bt = st.pool, st.block_table
    _check(_lib().mla_layer_step_small(ctypes.byref(cd), _ptr(h), _ptr(w["w_dkv_kr"]), _ptr(w["w_dq"]),
                                       _ptr(w["w_uq_qr"]), _ptr(w["w_uk"]), _ptr(w["w_uv"]), _ptr(w["w_o"]),
                                       _ptr(pool), pool.shape[0], _ptr(bt), bt.shape[1], _ptr(seq_lens), B,
                                       max_seq_len, _ptr(q), _ptr(o_lat), _ptr(lse), _ptr(u), _ptr(ws), nbytes,
                                       _stream(stream)), "mla_layer_step_small")
    return u, q, o_lat, lse


def step_workspace_bytes(dims, B: int, max_seq_len: int, shared: bool = False) -> int:
    """Bytes that every call of a ``layer_step`` fits in (``shared``: one with shared pages)."""
    calls = [CALL_APPEND_KV, CALL_ABSORB_QUERY, CALL_DECODE_ATTENTION, CALL_OUT_PROJ]
    return max(workspace_size(dims, c, B, max_seq_len) for c in calls + [CALL_SHARED_PREFIX_ATTENTION] * shared)
