"""Fused decode-step attention for GB300: KV append + GQA over a paged cache or a
sliding-window ring + per-head attention sinks.

A thin ctypes binding over the C ABI in ``include/decode_attn.h`` (library
``libdecode_attn.so`` next to this file, built by ``build.py``). Every step of
the computation runs in the library's CUDA kernels; this module only turns
torch tensors into device pointers, sizes and the current CUDA stream, and
turns error codes into exceptions. There is no CPU fallback: if the library
is missing, every call raises.

Tensor layouts (all contiguous, bf16 unless noted):
  q, out            [B, Hq, D]
  k_new, v_new      [B, Hkv, D]
  paged caches      [num_pages, Hkv, page_size, D]
  ring caches       [B, Hkv, window, D]
  block_table       [B, max_pages_per_seq] int32
  seq_lens          [B] int32, length after this step's append (0 = inactive)
  sinks             [Hq] float32, or None
  weights           [num_pages, Hkv, page_size] float32, accumulated attention weights
"""
import ctypes
import os

import torch

__all__ = [
    "da_shape",
    "DecodeAttnError", "decode_attn_paged", "decode_attn_ring", "kv_append",
    "decode_attn_workspace_bytes", "decode_attn_reserve", "decode_attn_device_status",
    "decode_attn_error_string", "library_path", "load_library",
    "DA_STATUS_BAD_SEQ_LEN", "DA_STATUS_BAD_PAGE", "DA_STATUS_TIMEOUT", "DA_STATUS_BAD_POSITION",
    "DA_FP8_SCALE_RECIPROCAL", "DA_FP8_SCALE_DIVIDE",
    "decode_attn_paged_rope", "decode_attn_ring_rope", "decode_attn_paged_fp8", "decode_attn_ring_fp8",
    "decode_attn_paged_multi", "decode_attn_ring_multi", "decode_attn_multi_workspace_bytes",
    "decode_attn_multi_reserve", "decode_attn_multi_launches", "decode_attn_test_expire_wait",
    "decode_attn_paged_fp8_rope", "decode_attn_ring_fp8_rope", "decode_attn_set_early_inputs",
    "decode_attn_stream_reserve", "decode_attn_stream_release",
    "decode_attn_paged_multi_rope", "decode_attn_ring_multi_rope",
    "decode_attn_paged_weights", "decode_attn_paged_fp8_weights", "decode_attn_paged_multi_weights",
    "kv_evict", "kv_evict_fp8", "decode_attn_weights_workspace_bytes", "kv_evict_workspace_bytes",
    "decode_attn_weights_reserve",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdecode_attn.so"

DA_OK = 0
DA_ERR_INVALID_ARG = -1
DA_ERR_UNSUPPORTED = -2
DA_ERR_WORKSPACE = -3
DA_ERR_CUDA = -4
DA_STATUS_BAD_SEQ_LEN = 1
DA_STATUS_BAD_PAGE = 2
DA_STATUS_TIMEOUT = 4
DA_STATUS_BAD_POSITION = 8
DA_FP8_SCALE_RECIPROCAL = 0  # scale of a row appended to fp8 blocks: amax * (1 / 448), or
DA_FP8_SCALE_DIVIDE = 1      # amax / 448 (fp32)


class da_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class DecodeAttnError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"decode_attn error {code}: {message}")
        self.code = code


_lib = None


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library():
    """Load the CUDA library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    c_int, c_float = ctypes.c_int, ctypes.c_float
    lib.decode_attn_paged.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, f32p, c_int, c_float, vp,
                                      da_shape, c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_ring.argtypes = [vp, vp, vp, vp, vp, i32p, f32p, c_int, c_float, vp,
                                     da_shape, vp]
    lib.kv_append.argtypes = [vp, vp, vp, vp, i32p, i32p, c_int, da_shape, c_int, c_int, c_int, vp]
    lib.decode_attn_paged_rope.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, f32p, f32p, f32p, c_int,
                                           c_int, c_float, vp, da_shape, c_int, c_int, c_int, c_int,
                                           vp]
    lib.decode_attn_ring_rope.argtypes = [vp, vp, vp, vp, vp, i32p, f32p, f32p, f32p, c_int, c_int,
                                          c_float, vp, da_shape, vp]
    lib.decode_attn_paged_fp8.argtypes = [vp, vp, vp, vp, i32p, i32p, f32p, c_int, c_float, vp,
                                          da_shape, c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_ring_fp8.argtypes = [vp, vp, vp, vp, i32p, f32p, c_int, c_float, vp, da_shape,
                                         vp]
    lib.decode_attn_paged_fp8_rope.argtypes = [vp, vp, vp, vp, i32p, i32p, f32p, f32p, f32p,
                                               c_int, c_int, c_float, vp, da_shape, c_int, c_int,
                                               c_int, c_int, vp]
    lib.decode_attn_ring_fp8_rope.argtypes = [vp, vp, vp, vp, i32p, f32p, f32p, f32p, c_int, c_int,
                                              c_float, vp, da_shape, vp]
    lib.decode_attn_paged_multi.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, i32p, f32p, c_int,
                                            c_float, vp, da_shape, c_int, c_int, c_int, c_int,
                                            c_int, vp]
    lib.decode_attn_ring_multi.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, f32p, c_int, c_float,
                                           vp, da_shape, c_int, vp]
    lib.decode_attn_paged_multi_rope.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, i32p, f32p, f32p,
                                                 f32p, c_int, c_int, c_float, vp, da_shape, c_int,
                                                 c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_ring_multi_rope.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, f32p, f32p, f32p,
                                                c_int, c_int, c_float, vp, da_shape, c_int, vp]
    lib.decode_attn_multi_workspace_bytes.argtypes = [da_shape, c_int, c_int, c_int]
    lib.decode_attn_multi_workspace_bytes.restype = ctypes.c_size_t
    lib.decode_attn_multi_launches.argtypes = [da_shape, c_int, c_int, c_int]
    lib.decode_attn_multi_launches.restype = c_int
    lib.decode_attn_multi_reserve.argtypes = [ctypes.c_size_t]
    lib.decode_attn_workspace_bytes.argtypes = [da_shape, c_int]
    lib.decode_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.decode_attn_reserve.argtypes = [ctypes.c_size_t]
    lib.decode_attn_stream_reserve.argtypes = [vp, ctypes.c_size_t, ctypes.c_size_t]
    lib.decode_attn_stream_release.argtypes = [vp]
    lib.decode_attn_device_status.argtypes = [vp]
    lib.decode_attn_test_expire_wait.argtypes = [c_int]
    lib.decode_attn_set_early_inputs.argtypes = [c_int]
    lib.decode_attn_error_string.argtypes = [c_int]
    lib.decode_attn_error_string.restype = ctypes.c_char_p
    lib.decode_attn_paged_weights.argtypes = [vp, vp, vp, vp, vp, f32p, i32p, i32p, f32p, c_int, c_float, vp,
                                              da_shape, c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_paged_fp8_weights.argtypes = [vp, vp, vp, vp, f32p, i32p, i32p, f32p, c_int, c_float, vp,
                                                  da_shape, c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_paged_fp8_weights_rule.argtypes = [vp, vp, vp, vp, f32p, i32p, i32p, f32p, c_int, c_float, c_int,
                                                       vp, da_shape, c_int, c_int, c_int, c_int, vp]
    lib.decode_attn_paged_multi_weights.argtypes = [vp, vp, vp, vp, vp, f32p, i32p, i32p, i32p, f32p, c_int,
                                                    c_float, vp, da_shape, c_int, c_int, c_int, c_int, c_int, vp]
    lib.kv_evict.argtypes = [vp, vp, f32p, i32p, i32p, i32p, i32p, c_int, c_int, c_int, da_shape, c_int, c_int,
                             c_int, c_int, vp]
    lib.kv_evict_fp8.argtypes = [vp, f32p, i32p, i32p, i32p, i32p, c_int, c_int, c_int, da_shape, c_int, c_int,
                                 c_int, c_int, vp]
    lib.decode_attn_weights_workspace_bytes.argtypes = [da_shape, c_int, c_int]
    lib.decode_attn_weights_workspace_bytes.restype = ctypes.c_size_t
    lib.kv_evict_workspace_bytes.argtypes = [da_shape, c_int]
    lib.kv_evict_workspace_bytes.restype = ctypes.c_size_t
    lib.decode_attn_weights_reserve.argtypes = [vp, ctypes.c_size_t]
    for fn in (lib.decode_attn_paged_weights, lib.decode_attn_paged_fp8_weights,
               lib.decode_attn_paged_fp8_weights_rule, lib.decode_attn_paged_multi_weights, lib.kv_evict, lib.kv_evict_fp8,
               lib.decode_attn_weights_reserve, lib.decode_attn_paged, lib.decode_attn_ring, lib.kv_append, lib.decode_attn_reserve,
               lib.decode_attn_device_status, lib.decode_attn_paged_rope, lib.decode_attn_ring_rope,
               lib.decode_attn_paged_fp8, lib.decode_attn_ring_fp8, lib.decode_attn_paged_multi,
               lib.decode_attn_ring_multi, lib.decode_attn_multi_reserve,
               lib.decode_attn_test_expire_wait, lib.decode_attn_paged_fp8_rope,
               lib.decode_attn_ring_fp8_rope, lib.decode_attn_set_early_inputs,
               lib.decode_attn_stream_reserve, lib.decode_attn_stream_release,
               lib.decode_attn_paged_multi_rope, lib.decode_attn_ring_multi_rope):
        fn.restype = c_int
    _lib = lib
    return lib


def decode_attn_error_string(code: int) -> str:
    return load_library().decode_attn_error_string(int(code)).decode()


def _check(code):
    if code != 0:
        raise DecodeAttnError(code, decode_attn_error_string(code))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shape(q, k_cache_heads):
    B, Hq, D = q.shape
    return da_shape(B, Hq, k_cache_heads, D)


def decode_attn_paged(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, sinks, window,
                      scale, out, max_seq_len=None, stream=None):
    """One decode step over a paged cache, with the KV append fused in.

    k_new/v_new None = no append. window 0 = full attention. max_seq_len
    defaults to the block table's capacity (max_pages_per_seq * page_size).
    """
    num_pages, Hkv, P, _ = k_cache.shape
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * P
    lib = load_library()
    _check(lib.decode_attn_paged(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(sinks), int(window), float(scale), _ptr(out), _shape(q, Hkv), P,
        max_pages, num_pages, int(max_seq_len), _stream(stream)))
    return out


def decode_attn_ring(q, k_new, v_new, k_cache, v_cache, seq_lens, sinks, scale, out,
                     stream=None):
    """One decode step over a sliding-window ring [B, Hkv, W, D] (W = its capacity)."""
    B, Hkv, W, _ = k_cache.shape
    lib = load_library()
    _check(lib.decode_attn_ring(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(sinks), int(W), float(scale), _ptr(out), _shape(q, Hkv), _stream(stream)))
    return out


def decode_attn_paged_rope(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, sinks,
                           rope_cos, rope_sin, window, scale, out, max_seq_len=None, stream=None):
    """decode_attn_paged with the rotary embedding of position L - 1 applied to q and k_new
    first; rope_cos/rope_sin are fp32 [max_position, D/2] device tables."""
    num_pages, Hkv, P, _ = k_cache.shape
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * P
    lib = load_library()
    _check(lib.decode_attn_paged_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(sinks), _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]),
        int(window), float(scale), _ptr(out), _shape(q, Hkv), P, max_pages, num_pages,
        int(max_seq_len), _stream(stream)))
    return out


def decode_attn_ring_rope(q, k_new, v_new, k_cache, v_cache, seq_lens, sinks, rope_cos, rope_sin,
                          scale, out, stream=None):
    """decode_attn_ring with the rotary embedding of position L - 1 applied first."""
    B, Hkv, W, _ = k_cache.shape
    lib = load_library()
    _check(lib.decode_attn_ring_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(sinks), _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), int(W), float(scale),
        _ptr(out), _shape(q, Hkv), _stream(stream)))
    return out


FP8_BLOCK_BYTES = 2176  # 16 tokens of one KV head: K codes, V^T codes, K and V scales


def decode_attn_paged_fp8(q, k_new, v_new, kv_cache, block_table, seq_lens, sinks, window, scale,
                          out, max_seq_len=None, stream=None):
    """decode_attn_paged over an fp8 cache: kv_cache uint8 [num_pages, Hkv, 2176], one block
    per page and KV head (K codes [16][64], V codes [64][16], K scales [16], V scales [16])."""
    num_pages, Hkv, nb = kv_cache.shape
    if nb != FP8_BLOCK_BYTES:
        raise ValueError(f"kv_cache blocks must be {FP8_BLOCK_BYTES} bytes, got {nb}")
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * 16
    lib = load_library()
    _check(lib.decode_attn_paged_fp8(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
        _ptr(sinks), int(window), float(scale), _ptr(out), _shape(q, Hkv), 16, max_pages,
        num_pages, int(max_seq_len), _stream(stream)))
    return out


def decode_attn_ring_fp8(q, k_new, v_new, kv_cache, seq_lens, sinks, scale, out, stream=None):
    """decode_attn_ring over an fp8 ring: kv_cache uint8 [B, Hkv, W / 16, 2176]."""
    B, Hkv, nblk, nb = kv_cache.shape
    if nb != FP8_BLOCK_BYTES:
        raise ValueError(f"kv_cache blocks must be {FP8_BLOCK_BYTES} bytes, got {nb}")
    lib = load_library()
    _check(lib.decode_attn_ring_fp8(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kv_cache), _ptr(seq_lens), _ptr(sinks),
        int(nblk * 16), float(scale), _ptr(out), _shape(q, Hkv), _stream(stream)))
    return out


def decode_attn_paged_fp8_rope(q, k_new, v_new, kv_cache, block_table, seq_lens, sinks, rope_cos,
                               rope_sin, window, scale, out, max_seq_len=None, stream=None):
    """decode_attn_paged_fp8 with the rotary embedding of position L - 1 applied to q and
    k_new first (the key before it is quantised); rope_cos/rope_sin fp32 [max_position, 32]."""
    num_pages, Hkv, nb = kv_cache.shape
    if nb != FP8_BLOCK_BYTES:
        raise ValueError(f"kv_cache blocks must be {FP8_BLOCK_BYTES} bytes, got {nb}")
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * 16
    lib = load_library()
    _check(lib.decode_attn_paged_fp8_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
        _ptr(sinks), _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), int(window),
        float(scale), _ptr(out), _shape(q, Hkv), 16, max_pages, num_pages, int(max_seq_len),
        _stream(stream)))
    return out


def decode_attn_ring_fp8_rope(q, k_new, v_new, kv_cache, seq_lens, sinks, rope_cos, rope_sin, scale,
                              out, stream=None):
    """decode_attn_ring_fp8 with the rotary embedding of position L - 1 applied first."""
    B, Hkv, nblk, nb = kv_cache.shape
    if nb != FP8_BLOCK_BYTES:
        raise ValueError(f"kv_cache blocks must be {FP8_BLOCK_BYTES} bytes, got {nb}")
    lib = load_library()
    _check(lib.decode_attn_ring_fp8_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kv_cache), _ptr(seq_lens), _ptr(sinks),
        _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), int(nblk * 16), float(scale),
        _ptr(out), _shape(q, Hkv), _stream(stream)))
    return out


def kv_append(k_new, v_new, k_cache, v_cache, seq_lens, block_table=None, stream=None):
    """Append alone: paged when block_table is given, else ring [B, Hkv, W, D]."""
    B, Hkv, D = k_new.shape
    lib = load_library()
    if block_table is not None:
        num_pages, _, P, _ = k_cache.shape
        args = (0, da_shape(B, Hkv, Hkv, D), P, block_table.shape[1], num_pages)
    else:
        W = k_cache.shape[2]
        args = (W, da_shape(B, Hkv, Hkv, D), 0, 0, 0)
    _check(lib.kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                         _ptr(block_table), _ptr(seq_lens), *args, _stream(stream)))


def decode_attn_paged_multi(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, sinks, window,
                            scale, out, q_lens=None, max_seq_len=None, stream=None):
    """Several query tokens per sequence: q / out [B, T, Hq, 64], k_new / v_new [B, T, Hkv, 64]
    bf16; seq_lens counts the cached tokens plus the q_lens[b] (or T) new ones. Attention is
    causal over the cache and the new tokens, which are then appended to the pages."""
    B, T, Hq, D = q.shape
    num_pages, Hkv = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * 16
    lib = load_library()
    _check(lib.decode_attn_paged_multi(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(q_lens), _ptr(sinks), int(window), float(scale), _ptr(out),
        da_shape(B, Hq, Hkv, D), T, 16, max_pages, num_pages, int(max_seq_len), _stream(stream)))
    return out


def decode_attn_ring_multi(q, k_new, v_new, k_cache, v_cache, seq_lens, sinks, scale, out,
                           q_lens=None, stream=None):
    """decode_attn_paged_multi over a ring of capacity W = k_cache.shape[2]; the ring holds
    the window of the history before the step."""
    B, T, Hq, D = q.shape
    Hkv, W = k_cache.shape[1], k_cache.shape[2]
    lib = load_library()
    _check(lib.decode_attn_ring_multi(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(q_lens), _ptr(sinks), int(W), float(scale), _ptr(out), da_shape(B, Hq, Hkv, D), T,
        _stream(stream)))
    return out


def decode_attn_paged_multi_rope(q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, sinks,
                                 rope_cos, rope_sin, window, scale, out, q_lens=None, max_seq_len=None,
                                 stream=None):
    """decode_attn_paged_multi with the rotary embedding: each new token's query rows and key
    rotated to its own position (rope_cos / rope_sin fp32 [max_position, 32] device tables)."""
    B, T, Hq, D = q.shape
    num_pages, Hkv = k_cache.shape[0], k_cache.shape[1]
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * 16
    lib = load_library()
    _check(lib.decode_attn_paged_multi_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(q_lens), _ptr(sinks), _ptr(rope_cos), _ptr(rope_sin),
        int(rope_cos.shape[0]), int(window), float(scale), _ptr(out), da_shape(B, Hq, Hkv, D), T,
        16, max_pages, num_pages, int(max_seq_len), _stream(stream)))
    return out


def decode_attn_ring_multi_rope(q, k_new, v_new, k_cache, v_cache, seq_lens, sinks, rope_cos,
                                rope_sin, scale, out, q_lens=None, stream=None):
    """decode_attn_ring_multi with the rotary embedding (see decode_attn_paged_multi_rope)."""
    B, T, Hq, D = q.shape
    Hkv, W = k_cache.shape[1], k_cache.shape[2]
    lib = load_library()
    _check(lib.decode_attn_ring_multi_rope(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(q_lens), _ptr(sinks), _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), int(W),
        float(scale), _ptr(out), da_shape(B, Hq, Hkv, D), T, _stream(stream)))
    return out


def decode_attn_multi_workspace_bytes(batch, num_q_heads, num_kv_heads, q_tokens, ring_window=0,
                                      max_seq_len=0, head_dim=64):
    return int(load_library().decode_attn_multi_workspace_bytes(
        da_shape(batch, num_q_heads, num_kv_heads, head_dim), int(q_tokens), int(ring_window),
        int(max_seq_len)))


def decode_attn_multi_launches(batch, num_q_heads, num_kv_heads, q_tokens, ring_window=0,
                               max_seq_len=0, head_dim=64):
    """Kernel launches of one multi-token call of this shape (0: invalid, or no device)."""
    return int(load_library().decode_attn_multi_launches(
        da_shape(batch, num_q_heads, num_kv_heads, head_dim), int(q_tokens), int(ring_window),
        int(max_seq_len)))


def decode_attn_multi_reserve(nbytes: int):
    _check(load_library().decode_attn_multi_reserve(int(nbytes)))


def decode_attn_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim=64, max_seq_len=0):
    return int(load_library().decode_attn_workspace_bytes(
        da_shape(batch, num_q_heads, num_kv_heads, head_dim), int(max_seq_len)))


def decode_attn_reserve(nbytes: int):
    _check(load_library().decode_attn_reserve(int(nbytes)))


def decode_attn_stream_reserve(stream, nbytes: int = 0, multi_nbytes: int = 0):
    """Workspaces of its own for the attention calls issued on `stream` (a torch.cuda.Stream
    or a raw handle), so that they may overlap calls on other streams; held until
    decode_attn_stream_release(stream)."""
    _check(load_library().decode_attn_stream_reserve(_stream(stream), int(nbytes), int(multi_nbytes)))


def decode_attn_stream_release(stream):
    """Synchronise `stream` and free its own workspaces (no-op if it has none)."""
    _check(load_library().decode_attn_stream_release(_stream(stream)))


def decode_attn_device_status(stream=None) -> int:
    """Wait for the stream, return and clear the device status bits."""
    rc = load_library().decode_attn_device_status(_stream(stream))
    if rc < 0:
        _check(rc)
    return rc


def decode_attn_set_early_inputs(level: int) -> int:
    """Process-wide: what the attention kernels read before waiting for the kernel launched
    just before each call; returns the previous level. 0 (default): nothing. 1: seq_lens,
    q_lens, block_table and sinks (they must have been written before that kernel started).
    2: as 1, and the first cache tiles of each long worker share are prefetched into L2 (a
    hint to the GPU-wide cache: the same conditions as level 1)."""
    rc = load_library().decode_attn_set_early_inputs(int(level))
    if rc < 0:
        _check(rc)
    return rc


def decode_attn_test_expire_wait(tile: int):
    """Testing aid: the next one-token attention call gives up at its first worker's tile
    wait number `tile` (after the tile landed) as if the wait had expired; < 0 disarms."""
    _check(load_library().decode_attn_test_expire_wait(int(tile)))


def _refuse(name, t, dtype, shape):
    if t.is_cuda and t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {shape}, got {t.dtype} "
                     f"{tuple(t.shape)} strides {t.stride()} on {t.device}")


def _tensor(name, t, dtype, shape, dev):
    """t's address, if it is as the library reads it: this type and shape, contiguous, on device dev."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda and t.get_device() == dev:
        return t.data_ptr()
    _refuse(name, t, dtype, shape)


def _paged_tensors(k, v, weights, block_table, seq_lens, dev):
    """Checked addresses of a paged cache (v None: fp8 blocks) and its tables, and its sizes."""
    if k.dim() != (3 if v is None else 4) or block_table.dim() != 2:
        raise ValueError(f"the cache is {tuple(k.shape)}, the block table {tuple(block_table.shape)}")
    num_pages, Hkv = k.shape[0], k.shape[1]
    B, max_pages = block_table.shape
    if v is None:
        kp, vp = _tensor("kv_cache", k, torch.uint8, (num_pages, Hkv, FP8_BLOCK_BYTES), dev), None
    else:
        pool = (num_pages, Hkv, 16, 64)
        kp = _tensor("k_cache", k, torch.bfloat16, pool, dev)
        vp = _tensor("v_cache", v, torch.bfloat16, pool, dev)
    return (kp, vp, _tensor("weights", weights, torch.float32, (num_pages, Hkv, 16), dev),
            _tensor("block_table", block_table, torch.int32, (B, max_pages), dev),
            _tensor("seq_lens", seq_lens, torch.int32, (B,), dev), B, Hkv, max_pages, num_pages)


def _new_tensors(q, k_new, v_new, sinks, out, lead, Hkv, dev):
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new are given together")
    Hq = q.shape[-2] if q.dim() > 1 else 0
    rows, new = lead + (Hq, 64), lead + (Hkv, 64)
    return (_tensor("q", q, torch.bfloat16, rows, dev),
            None if k_new is None else _tensor("k_new", k_new, torch.bfloat16, new, dev),
            None if v_new is None else _tensor("v_new", v_new, torch.bfloat16, new, dev),
            None if sinks is None else _tensor("sinks", sinks, torch.float32, (Hq,), dev),
            _tensor("out", out, torch.bfloat16, rows, dev), Hq)


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def decode_attn_paged_weights(q, k_new, v_new, k_cache, v_cache, weights, block_table, seq_lens, sinks,
                              window, scale, out, max_seq_len=None, stream=None):
    """decode_attn_paged that also adds every attended token's attention weight (its probabilities
    summed over the query heads of its KV head) to its cell of weights, fp32
    [num_pages, Hkv, 16]; the appended token's cell is set to its weight. The weights workspace
    holds 4 bytes per query head and position up to max_seq_len (default: what the block table
    can hold), so give the longest sequence's length where the table is much wider."""
    dev = torch.cuda.current_device()
    kp, vp, wp, bp, lp, B, Hkv, max_pages, num_pages = _paged_tensors(k_cache, v_cache, weights, block_table, seq_lens,
                                                                       dev)
    qp, knp, vnp, sp, op, Hq = _new_tensors(q, k_new, v_new, sinks, out, (B,), Hkv, dev)
    _check(load_library().decode_attn_paged_weights(
        qp, knp, vnp, kp, vp, wp, bp, lp, sp, int(window), float(scale), op, da_shape(B, Hq, Hkv, 64), 16, max_pages, num_pages,
        max_pages * 16 if max_seq_len is None else int(max_seq_len), _raw_stream(stream, dev)))
    return out


def decode_attn_paged_fp8_weights(q, k_new, v_new, kv_cache, weights, block_table, seq_lens, sinks, window,
                                  scale, out, max_seq_len=None, stream=None, scale_rule=DA_FP8_SCALE_RECIPROCAL):
    """decode_attn_paged_weights over an fp8 cache (kv_cache as in decode_attn_paged_fp8). scale_rule: how the
    appended token is scaled, DA_FP8_SCALE_RECIPROCAL as torch code on a GPU does it, DA_FP8_SCALE_DIVIDE as
    decode_attn_paged_fp8 does it (for a cache that both calls append to)."""
    dev = torch.cuda.current_device()
    kp, _, wp, bp, lp, B, Hkv, max_pages, num_pages = _paged_tensors(kv_cache, None, weights, block_table, seq_lens, dev)
    qp, knp, vnp, sp, op, Hq = _new_tensors(q, k_new, v_new, sinks, out, (B,), Hkv, dev)
    _check(load_library().decode_attn_paged_fp8_weights_rule(
        qp, knp, vnp, kp, wp, bp, lp, sp, int(window), float(scale), int(scale_rule), op, da_shape(B, Hq, Hkv, 64), 16,
        max_pages, num_pages, max_pages * 16 if max_seq_len is None else int(max_seq_len), _raw_stream(stream, dev)))
    return out


def decode_attn_paged_multi_weights(q, k_new, v_new, k_cache, v_cache, weights, block_table, seq_lens, sinks,
                                    window, scale, out, q_lens=None, max_seq_len=None, stream=None):
    """decode_attn_paged_multi that also adds every attended token's attention weight, summed over
    the new tokens and the query heads of its KV head, to its cell of weights; the new tokens'
    cells are set to theirs."""
    dev = torch.cuda.current_device()
    kp, vp, wp, bp, lp, B, Hkv, max_pages, num_pages = _paged_tensors(k_cache, v_cache, weights, block_table, seq_lens,
                                                                       dev)
    if q.dim() != 4 or k_new is None:
        raise ValueError("q is [B, T, Hq, 64] and k_new, v_new are required")
    T = q.shape[1]
    qp, knp, vnp, sp, op, Hq = _new_tensors(q, k_new, v_new, sinks, out, (B, T), Hkv, dev)
    _check(load_library().decode_attn_paged_multi_weights(
        qp, knp, vnp, kp, vp, wp, bp, lp, None if q_lens is None else _tensor("q_lens", q_lens, torch.int32, (B,), dev), sp,
        int(window), float(scale), op, da_shape(B, Hq, Hkv, 64), T, 16, max_pages, num_pages,
        max_pages * 16 if max_seq_len is None else int(max_seq_len), _raw_stream(stream, dev)))
    return out


def kv_evict(k_cache, v_cache, weights, block_table, seq_lens, new_lens, kept, keep_first=0, keep_last=0,
             max_seq_len=None, stream=None):
    """Shrink every sequence longer than keep = kept.shape[2] cells to keep cells per KV head, in
    place: the first keep_first and the last keep_last cells stay, and of those between them the
    ones of the largest accumulated weight. new_lens [B] int32 receives the lengths, kept
    [B, Hkv, keep] int32 the old cell of each kept cell (-1 beyond a shorter sequence's end). The
    work is cut for sequences of max_seq_len (default: what the block table can hold): give the
    longest length where the table is much wider."""
    dev = torch.cuda.current_device()
    kp, vp, wp, bp, lp, B, Hkv, max_pages, num_pages = _paged_tensors(k_cache, v_cache, weights, block_table, seq_lens,
                                                                       dev)
    keep = kept.shape[-1] if kept.dim() else 0
    _check(load_library().kv_evict(
        kp, vp, wp, bp, lp, _tensor("new_lens", new_lens, torch.int32, (B,), dev),
        _tensor("kept", kept, torch.int32, (B, Hkv, keep), dev), keep, int(keep_first), int(keep_last), da_shape(B, Hkv, Hkv, 64), 16,
        max_pages, num_pages, max_pages * 16 if max_seq_len is None else int(max_seq_len), _raw_stream(stream, dev)))
    return new_lens


def kv_evict_fp8(kv_cache, weights, block_table, seq_lens, new_lens, kept, keep_first=0, keep_last=0,
                 max_seq_len=None, stream=None):
    """kv_evict over an fp8 cache: codes and scales move as they are."""
    dev = torch.cuda.current_device()
    kp, _, wp, bp, lp, B, Hkv, max_pages, num_pages = _paged_tensors(kv_cache, None, weights, block_table, seq_lens, dev)
    keep = kept.shape[-1] if kept.dim() else 0
    _check(load_library().kv_evict_fp8(
        kp, wp, bp, lp, _tensor("new_lens", new_lens, torch.int32, (B,), dev),
        _tensor("kept", kept, torch.int32, (B, Hkv, keep), dev), keep, int(keep_first), int(keep_last), da_shape(B, Hkv, Hkv, 64), 16,
        max_pages, num_pages, max_pages * 16 if max_seq_len is None else int(max_seq_len), _raw_stream(stream, dev)))
    return new_lens


def decode_attn_weights_workspace_bytes(batch, num_q_heads, num_kv_heads, q_tokens=1, max_seq_len=0, head_dim=64):
    """Bytes of the weights workspace for a call of q_tokens new tokens (1: the one-token calls)."""
    return int(load_library().decode_attn_weights_workspace_bytes(
        da_shape(batch, num_q_heads, num_kv_heads, head_dim), int(q_tokens), int(max_seq_len)))


def kv_evict_workspace_bytes(batch, num_kv_heads, keep):
    return int(load_library().kv_evict_workspace_bytes(da_shape(batch, num_kv_heads, num_kv_heads, 64), int(keep)))


def decode_attn_weights_reserve(nbytes: int, stream=None):
    """Grow the weights workspace that calls on `stream` use (the stream's own after
    decode_attn_stream_reserve, else the device's) to at least nbytes; call before a capture."""
    _check(load_library().decode_attn_weights_reserve(_raw_stream(stream, torch.cuda.current_device()), int(nbytes)))
