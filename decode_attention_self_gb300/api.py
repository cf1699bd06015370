"""Thin ctypes binding of libdecoderattn.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks that the torch tensors it is given are CUDA,
contiguous and of the right dtype, and passes their device pointers, sizes and
the current CUDA stream through the C ABI declared in include/dr_api.h.
PyTorch only provides device memory and streams.

Importing this module loads the library and fails loudly if it is missing:
there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdecoderattn.so")

DR_OK, DR_ERR_INVALID_ARG, DR_ERR_UNSUPPORTED, DR_ERR_CUDA = 0, 1, 2, 3
DR_KV_CONTIGUOUS, DR_KV_PAGED = 0, 1
DR_BF16, DR_F32 = 0, 1
DR_KV_BF16, DR_KV_FP8_E4M3 = 0, 1
DR_ERRF_SEQ_LEN, DR_ERRF_BLOCK_ID, DR_ERRF_POS, DR_ERRF_TOKEN, DR_ERRF_TIMEOUT, DR_ERRF_ROW_START = 1, 2, 4, 8, 16, 32
DR_SAMPLE_ADVANCE = 1
DR_ACT_NONE, DR_ACT_RELU, DR_ACT_GELU, DR_ACT_GELU_TANH, DR_ACT_SILU = 0, 1, 2, 3, 4
DR_NORM_NONE, DR_NORM_LAYER, DR_NORM_RMS = 0, 1, 2
DR_LINEAR_MAX_OUTS = 4

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
_lib = ctypes.CDLL(LIB_PATH)


class dr_kv_cache(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("max_len", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class dr_score_opts(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("first_key", ctypes.c_void_p)]


class dr_linear_opts(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("gated", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64)]


class dr_linear_out(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride", ctypes.c_int64), ("cols", ctypes.c_int32)]


class dr_norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_i64, _sz = ctypes.c_int64, ctypes.c_size_t
_cs = ctypes.c_char_p   # a C structure packed as bytes
_lib.dr_kv_append.argtypes = [ctypes.POINTER(dr_kv_cache), _vp, _vp, _vp, _i, _i, _i, _vp, _vp]
_lib.dr_decode_self_attn.argtypes = [_vp, ctypes.POINTER(dr_kv_cache), _vp, _i, _i, _i, _i, _f, _vp, _i, _vp, _vp]
_lib.dr_decode_cross_attn.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _i, _vp, _vp]
_lib.dr_decode_layer.argtypes = [_vp, ctypes.POINTER(dr_kv_cache), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                 _i, _f, _vp, _vp, _i, _vp, _vp]
_lib.dr_sample_topk_delayed.argtypes = [_vp, _i, _i, _i, _i, _f, _i, _vp, _vp, ctypes.c_int32, _vp, _vp, _i, _vp]
_lib.dr_embed_tokens.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _vp]
_lib.dr_lm_head.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp]
_lib.dr_lm_head_stall_test.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp]
_lib.dr_decode_self_attn_stall_test.argtypes = [_vp, ctypes.POINTER(dr_kv_cache), _vp, _i, _i, _i, _i, _f, _vp, _i, _vp,
                                                _i, _vp]
_lib.dr_rope_table.argtypes = [_vp, _i, _i, ctypes.c_double, _vp]
_lib.dr_rope_append.argtypes = [_cs, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp]
_lib.dr_prompt_attn.argtypes = [_vp, _i64, _cs, _vp, _vp, _cs, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _sz, _vp, _vp]
_lib.dr_prompt_attn_stall_test.argtypes = _lib.dr_prompt_attn.argtypes[:-1] + [_i, _vp]
_lib.dr_prompt_attn_workspace.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.dr_prompt_attn_workspace.restype = _sz
_lib.dr_shared_prefix_attn.argtypes = [_vp, _i64, _cs, _vp, _cs, _vp, _cs, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _sz,
                                       _vp, _vp]
_lib.dr_shared_prefix_attn_stall_test.argtypes = _lib.dr_shared_prefix_attn.argtypes[:-1] + [_i, _vp]
_lib.dr_shared_prefix_attn_workspace.argtypes = [_i, _i, _i, _i, _i]
_lib.dr_shared_prefix_attn_workspace.restype = _sz
_lib.dr_linear.argtypes = [_vp, _i64, _vp, _cs, _i, _i, _i, _cs, _i, _i, _vp, _vp]
_lib.dr_linear_stall_test.argtypes = _lib.dr_linear.argtypes[:-1] + [_i, _vp]
_lib.dr_residual_norm.argtypes = [_vp, _i64, _i, _cs, _vp, _i64, _f, _vp, _i64, _vp, _i64, _i, _cs, _vp, _i64, _i, _i, _i, _vp]
_lib.dr_plan_splits.argtypes = [_i, _i, _i, _i, _i]
_lib.dr_plan_splits.restype = _i
_lib.dr_status_string.argtypes = [_i]
_lib.dr_status_string.restype = ctypes.c_char_p
for _fn in ("dr_kv_append", "dr_decode_self_attn", "dr_decode_cross_attn", "dr_decode_layer",
            "dr_sample_topk_delayed", "dr_embed_tokens", "dr_lm_head", "dr_lm_head_stall_test",
            "dr_decode_self_attn_stall_test", "dr_rope_table", "dr_rope_append", "dr_prompt_attn",
            "dr_shared_prefix_attn", "dr_prompt_attn_stall_test", "dr_shared_prefix_attn_stall_test",
            "dr_linear", "dr_linear_stall_test", "dr_residual_norm"):
    getattr(_lib, _fn).restype = _i


class DrError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {dr_status_string(status)} (status {status})")
        self.status = status


def dr_status_string(status: int) -> str:
    return _lib.dr_status_string(int(status)).decode()


def dr_plan_splits(B: int, H: int, max_len: int, kv_dtype: int, num_sms: int) -> int:
    return int(_lib.dr_plan_splits(B, H, max_len, kv_dtype, num_sms))


def _check(fn: str, status: int):
    if status != DR_OK:
        raise DrError(fn, status)


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


@dataclasses.dataclass
class KVCache:
    """One layer's self-attention cache (device tensors owned by the caller).

    contiguous: k, v [B, H, max_len, D] bf16, or uint8 e4m3 codes with k_scale/v_scale.
    paged:      k, v [num_blocks, H, 16, D] (same element formats) and block_table [B, max_blocks] int32.
    """

    k: torch.Tensor
    v: torch.Tensor
    block_table: torch.Tensor | None = None
    k_scale: float = 1.0
    v_scale: float = 1.0

    @property
    def fp8(self) -> bool:
        return self.k.dtype == torch.uint8

    @property
    def paged(self) -> bool:
        return self.block_table is not None

    @property
    def capacity(self) -> int:
        return self.block_table.shape[1] * self.k.shape[2] if self.paged else self.k.shape[2]

    def as_c(self) -> dr_kv_cache:
        c = dr_kv_cache()
        dt = torch.uint8 if self.fp8 else torch.bfloat16
        c.k = _ptr(self.k, dt, "cache.k")
        c.v = _ptr(self.v, dt, "cache.v")
        c.kv_dtype = DR_KV_FP8_E4M3 if self.fp8 else DR_KV_BF16
        c.k_scale = float(self.k_scale)
        c.v_scale = float(self.v_scale)
        if self.paged:
            c.layout = DR_KV_PAGED
            c.block_size = self.k.shape[2]
            c.num_blocks = self.k.shape[0]
            c.max_blocks_per_seq = self.block_table.shape[1]
            c.block_table = _ptr(self.block_table, torch.int32, "cache.block_table")
        else:
            c.layout = DR_KV_CONTIGUOUS
            c.max_len = self.k.shape[2]
        return c


def dr_kv_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor,
                 err_flag: torch.Tensor | None = None, stream=None) -> None:
    """Write k_new, v_new [B, H, D] bf16 at position pos[b] (int32 [B]) of every row."""
    B, H, D = k_new.shape
    c = cache.as_c()
    _check("dr_kv_append", _lib.dr_kv_append(ctypes.byref(c), _ptr(k_new, torch.bfloat16, "k_new"),
                                             _ptr(v_new, torch.bfloat16, "v_new"), _ptr(pos, torch.int32, "pos"),
                                             B, H, D, _ptr(err_flag, torch.int32, "err_flag"), _stream(stream)))


def dr_decode_self_attn(q: torch.Tensor, cache: KVCache, seq_len: torch.Tensor, out: torch.Tensor,
                        max_seq_len_hint: int = 0, scale: float = 0.0, err_flag: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """out[b,h] = softmax(scale q[b,h].K[b,h,:seq_len[b]]) V[b,h,:seq_len[b]] (out bf16 or float32)."""
    B, H, D = q.shape
    c = cache.as_c()
    od = DR_F32 if out.dtype == torch.float32 else DR_BF16
    _check("dr_decode_self_attn",
           _lib.dr_decode_self_attn(_ptr(q, torch.bfloat16, "q"), ctypes.byref(c), _ptr(seq_len, torch.int32, "seq_len"),
                                    B, H, D, int(max_seq_len_hint), float(scale), _ptr(out, None, "out"), od,
                                    _ptr(err_flag, torch.int32, "err_flag"), _stream(stream)))
    return out


def dr_decode_self_attn_stall_test(q: torch.Tensor, cache: KVCache, seq_len: torch.Tensor, out: torch.Tensor,
                                   stall_row: int, max_seq_len_hint: int = 0, scale: float = 0.0,
                                   err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Test hook: dr_decode_self_attn with row stall_row's cluster merge left waiting until its bound runs out."""
    B, H, D = q.shape
    c = cache.as_c()
    od = DR_F32 if out.dtype == torch.float32 else DR_BF16
    _check("dr_decode_self_attn_stall_test",
           _lib.dr_decode_self_attn_stall_test(_ptr(q, torch.bfloat16, "q"), ctypes.byref(c),
                                               _ptr(seq_len, torch.int32, "seq_len"), B, H, D, int(max_seq_len_hint),
                                               float(scale), _ptr(out, None, "out"), od,
                                               _ptr(err_flag, torch.int32, "err_flag"), int(stall_row),
                                               _stream(stream)))
    return out


def dr_decode_cross_attn(q: torch.Tensor, k_enc: torch.Tensor, v_enc: torch.Tensor, enc_len: torch.Tensor,
                         out: torch.Tensor, scale: float = 0.0, err_flag: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Attention of q [B,H,D] over k_enc, v_enc [B,H,Lc_max,D] limited to enc_len[b] keys."""
    B, H, D = q.shape
    Lc_max = k_enc.shape[2]
    od = DR_F32 if out.dtype == torch.float32 else DR_BF16
    _check("dr_decode_cross_attn",
           _lib.dr_decode_cross_attn(_ptr(q, torch.bfloat16, "q"), _ptr(k_enc, torch.bfloat16, "k_enc"),
                                     _ptr(v_enc, torch.bfloat16, "v_enc"), _ptr(enc_len, torch.int32, "enc_len"),
                                     B, H, D, Lc_max, float(scale), _ptr(out, None, "out"), od,
                                     _ptr(err_flag, torch.int32, "err_flag"), _stream(stream)))
    return out


def dr_decode_layer(q: torch.Tensor, cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, seq_len: torch.Tensor,
                    q_cross: torch.Tensor, k_enc: torch.Tensor, v_enc: torch.Tensor, enc_len: torch.Tensor,
                    out: torch.Tensor, out_cross: torch.Tensor, max_seq_len_hint: int = 0, scale: float = 0.0,
                    err_flag: torch.Tensor | None = None, stream=None) -> None:
    """One launch: append k_new, v_new at seq_len-1, self-attention over seq_len keys, cross-attention."""
    B, H, D = q.shape
    if out_cross.dtype != out.dtype:
        raise ValueError("out and out_cross must have the same dtype")
    c = cache.as_c()
    od = DR_F32 if out.dtype == torch.float32 else DR_BF16
    _check("dr_decode_layer",
           _lib.dr_decode_layer(_ptr(q, torch.bfloat16, "q"), ctypes.byref(c), _ptr(k_new, torch.bfloat16, "k_new"),
                                _ptr(v_new, torch.bfloat16, "v_new"), _ptr(seq_len, torch.int32, "seq_len"),
                                _ptr(q_cross, torch.bfloat16, "q_cross"), _ptr(k_enc, torch.bfloat16, "k_enc"),
                                _ptr(v_enc, torch.bfloat16, "v_enc"), _ptr(enc_len, torch.int32, "enc_len"),
                                k_enc.shape[2], B, H, D, int(max_seq_len_hint), float(scale), _ptr(out, None, "out"),
                                _ptr(out_cross, None, "out_cross"), od, _ptr(err_flag, torch.int32, "err_flag"),
                                _stream(stream)))


def dr_sample_topk_delayed(logits: torch.Tensor, temperature: float, top_k: int, seeds: torch.Tensor,
                           step: torch.Tensor, pad_id: int, tokens: torch.Tensor, probs: torch.Tensor | None = None,
                           V: int | None = None, advance: bool = False, stream=None) -> torch.Tensor:
    """tokens [B,C] int32 from logits [B,C,ldv] float32; seeds [B] int64 (uint64 bits); step [B] int32."""
    B, C, ldv = logits.shape
    V = ldv if V is None else V
    if seeds.dtype not in (torch.int64, torch.uint64):
        raise ValueError("seeds must be a 64-bit integer tensor")
    _check("dr_sample_topk_delayed",
           _lib.dr_sample_topk_delayed(_ptr(logits, torch.float32, "logits"), B, C, V, ldv, float(temperature),
                                       int(top_k), _ptr(seeds, None, "seeds"), _ptr(step, torch.int32, "step"),
                                       int(pad_id), _ptr(tokens, torch.int32, "tokens"),
                                       _ptr(probs, torch.float32, "probs"), DR_SAMPLE_ADVANCE if advance else 0,
                                       _stream(stream)))
    return tokens


def dr_embed_tokens(tokens: torch.Tensor, table: torch.Tensor, V: int, out: torch.Tensor,
                    err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[b] = sum_c table[c*V + tokens[b,c]]; tokens [B,C] int32, table [C*V, Dm] bf16, out [B,Dm]."""
    B, C = tokens.shape
    Dm = table.shape[1]
    od = DR_F32 if out.dtype == torch.float32 else DR_BF16
    _check("dr_embed_tokens",
           _lib.dr_embed_tokens(_ptr(tokens, torch.int32, "tokens"), _ptr(table, torch.bfloat16, "table"), B, C, V, Dm,
                                _ptr(out, None, "out"), od, _ptr(err_flag, torch.int32, "err_flag"), _stream(stream)))
    return out


def dr_lm_head(hidden: torch.Tensor, W: torch.Tensor, C: int, logits: torch.Tensor,
               err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """logits [B,C,ldv] float32 from hidden [B,K] bf16 and merged heads W [C*V, K] bf16 (V = W rows / C)."""
    B, K = hidden.shape
    V = W.shape[0] // C
    ldv = logits.shape[2]
    _check("dr_lm_head",
           _lib.dr_lm_head(_ptr(hidden, torch.bfloat16, "hidden"), _ptr(W, torch.bfloat16, "W"), B, K, C, V, ldv,
                           _ptr(logits, torch.float32, "logits"), _ptr(err_flag, torch.int32, "err_flag"),
                           _stream(stream)))
    return logits


def dr_lm_head_stall_test(hidden: torch.Tensor, W: torch.Tensor, C: int, logits: torch.Tensor, stall_slab: int,
                          err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Test hook: dr_lm_head with the CTAs of weight slab `stall_slab` made to time out (see dr_api.h)."""
    B, K = hidden.shape
    V = W.shape[0] // C
    ldv = logits.shape[2]
    _check("dr_lm_head_stall_test",
           _lib.dr_lm_head_stall_test(_ptr(hidden, torch.bfloat16, "hidden"), _ptr(W, torch.bfloat16, "W"), B, K, C, V,
                                      ldv, _ptr(logits, torch.float32, "logits"),
                                      _ptr(err_flag, torch.int32, "err_flag"), int(stall_slab), _stream(stream)))
    return logits


# The prompt-side calls below check up to fourteen tensors each, and a small call's device work takes a few
# microseconds, so their checks are written out flat: a tensor that passes costs a few attribute reads, and only one
# that fails is looked at again to say why.  The C structures are packed as bytes (a ctypes.Structure takes twice the time).
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_pack_cache = struct.Struct("@iiiiiiPPPff").pack   # dr_kv_cache
_pack_opts = struct.Struct("@ifPPP").pack          # dr_score_opts
assert struct.calcsize("@iiiiiiPPPff") == ctypes.sizeof(dr_kv_cache)
assert struct.calcsize("@ifPPP") == ctypes.sizeof(dr_score_opts)


def _refuse(t, dev: int, dtype, shape, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != dev:
        raise ValueError(f"{name} must be on the current CUDA device {dev}, is on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _vec(t, dev: int, dtype, n: int, name: str):
    """Address of n contiguous elements on device dev; None for None."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _refuse(t, dev, dtype, (n,), name)
    return t.data_ptr()


def _rows(t, dev: int, shape, name: str):
    """(address, elements between tokens) of a bf16 [T, heads, D] tensor whose tokens are dense but may lie apart."""
    if t.get_device() != dev or t.dtype is not _BF16 or t.shape != shape:
        _refuse(t, dev, _BF16, shape, name)
    T, heads, D = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * D
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and heads > 1):
        raise ValueError(f"{name} must be [T, heads, D] with contiguous heads")
    return t.data_ptr(), (s0 if T > 1 else heads * D)


def _cache(cache: KVCache, dev: int, B: int, Hkv: int, D: int, name: str) -> bytes:
    """The C description of a cache of at least B rows of Hkv heads, all of it on device dev."""
    k, v, table = cache.k, cache.v, cache.block_table
    shape, dt = k.shape, k.dtype
    if len(shape) != 4 or shape[1] != Hkv or shape[3] != D:
        raise ValueError(f"{name}.k and {name}.v must be [.., {Hkv}, .., {D}], k is {tuple(shape)}")
    if dt is not _BF16 and dt is not _U8:
        raise ValueError(f"{name}.k must be {_BF16}, or {_U8} for e4m3 codes, got {dt}")
    if k.get_device() != dev or not k.is_contiguous():
        _refuse(k, dev, dt, shape, name + ".k")
    if v.get_device() != dev or v.dtype is not dt or v.shape != shape or not v.is_contiguous():
        _refuse(v, dev, dt, shape, name + ".v")
    fp8 = DR_KV_FP8_E4M3 if dt is _U8 else DR_KV_BF16
    rows, _, keys, _ = shape
    if table is None:
        packed = _pack_cache(DR_KV_CONTIGUOUS, keys, 0, 0, 0, fp8, k.data_ptr(), v.data_ptr(), 0, cache.k_scale,
                             cache.v_scale)
    else:
        if table.dim() != 2 or table.get_device() != dev or table.dtype is not _I32 or not table.is_contiguous():
            _refuse(table, dev, _I32, None if table.dim() == 2 else (B, "max_blocks"), name + ".block_table")
        blocks = rows
        rows, width = table.shape
        packed = _pack_cache(DR_KV_PAGED, 0, keys, blocks, width, fp8, k.data_ptr(), v.data_ptr(), table.data_ptr(),
                             cache.k_scale, cache.v_scale)
    if rows < B:
        raise ValueError(f"{name} holds {rows} rows, the call has {B}")
    return packed


def _stream_arg(stream, dev: int):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _shape3(t, name: str):
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [T, heads, D]")
    return shape


def _out(out, dev: int, shape):
    """(address, C type) of an output of the queries' shape."""
    dt = out.dtype
    if dt is not _BF16 and dt is not _F32:
        raise ValueError(f"out must be {_BF16} or {_F32}, got {dt}")
    if out.get_device() != dev or out.shape != shape or not out.is_contiguous():
        _refuse(out, dev, dt, shape, "out")
    return out.data_ptr(), DR_F32 if dt is _F32 else DR_BF16


def dr_rope_table(table: torch.Tensor, base: float = 10000.0, stream=None) -> torch.Tensor:
    """Fill table [max_pos, rot_dim] float32 with cos (first half) and sin of p * base^(-2i / rot_dim)."""
    dev = _device()
    if table.dim() != 2:
        raise ValueError("table must be [max_pos, rot_dim]")
    n, rot = table.shape
    _check("dr_rope_table", _lib.dr_rope_table(_vec(table, dev, _F32, n * rot, "table"), n, rot, base,
                                               _stream_arg(stream, dev)))
    return table


def dr_rope_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor, start_pos: torch.Tensor,
                   q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   table: torch.Tensor | None = None, interleaved: bool = False,
                   pos_offset: torch.Tensor | None = None, err_flag: torch.Tensor | None = None, stream=None) -> None:
    """Rotate q [T,Hq,D] (into q_out) and k [T,Hkv,D] by position and append k, v of ragged tokens to the cache.

    Row b's tokens row_start[b] .. row_start[b+1]-1 go to slots start_pos[b], start_pos[b]+1, ...; q, k, v and q_out
    may be slices of a fused projection (dense heads, any token stride that is a multiple of 8).
    """
    dev = _device()
    kshape = _shape3(k, "k")
    T, Hkv, D = kshape
    B = start_pos.numel()
    if q is None:
        Hq, qshape = Hkv, kshape
    else:
        qshape = _shape3(q, "q")
        Hq = qshape[1]
        if qshape[0] != T or qshape[2] != D:
            raise ValueError(f"q must have shape ({T}, heads, {D}), has {tuple(qshape)}")
    c = _cache(cache, dev, B, Hkv, D, "cache")
    kp, ks = _rows(k, dev, kshape, "k")
    vp, vs = _rows(v, dev, kshape, "v")
    qp, qs = (None, 0) if q is None else _rows(q, dev, qshape, "q")
    op, os_ = (None, 0) if q_out is None else _rows(q_out, dev, qshape, "q_out")
    if table is None:
        tp = rope_len = rot = 0
    else:
        if table.dim() != 2:
            raise ValueError("table must be [positions, rot_dim]")
        rope_len, rot = table.shape
        tp = _vec(table, dev, _F32, rope_len * rot, "table")
    st = _lib.dr_rope_append(c, qp, qs, kp, ks, vp, vs, op, os_, _vec(row_start, dev, _I32, B + 1, "row_start"),
                             _vec(start_pos, dev, _I32, B, "start_pos"),
                             _vec(pos_offset, dev, _I32, B, "pos_offset"), tp, rope_len, rot, 1 if interleaved else 0,
                             T, B, Hq, Hkv, D, _vec(err_flag, dev, _I32, 1, "err_flag"), _stream_arg(stream, dev))
    if st:
        raise DrError("dr_rope_append", st)


def _score_opts(dev: int, causal: bool, softcap: float, slopes, prefix_len, first_key, T: int, B: int, Hq: int) -> bytes:
    return _pack_opts(1 if causal else 0, softcap, _vec(slopes, dev, _F32, Hq, "slopes") or 0,
                      _vec(prefix_len, dev, _I32, B, "prefix_len") or 0, _vec(first_key, dev, _I32, T, "first_key") or 0)


def _sms() -> int:
    return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count


def dr_prompt_attn_workspace(T: int, B: int, Hq: int, Hkv: int, max_len: int, num_sms: int | None = None) -> int:
    """Bytes of workspace dr_prompt_attn wants (0: none), for the current device unless num_sms is given."""
    return int(_lib.dr_prompt_attn_workspace(T, B, Hq, Hkv, max_len, _sms() if num_sms is None else num_sms))


def _workspace_arg(ws, dev: int):
    if ws is None:
        return None, 0
    n = ws.numel()
    return _vec(ws, dev, _U8, n, "workspace"), n


def dr_prompt_attn(q: torch.Tensor, cache: KVCache, row_start: torch.Tensor, kv_len: torch.Tensor, out: torch.Tensor,
                   causal: bool = True, softcap: float = 0.0, slopes: torch.Tensor | None = None,
                   prefix_len: torch.Tensor | None = None, first_key: torch.Tensor | None = None,
                   max_len_hint: int = 0, scale: float = 0.0, workspace: torch.Tensor | None = None,
                   err_flag: torch.Tensor | None = None, stream=None, _stall_head=None) -> torch.Tensor:
    """Attention of ragged tokens q [T,Hq,D]: row b's tokens are the last of its kv_len[b] keys in the cache."""
    dev = _device()
    qshape = _shape3(q, "q")
    T, Hq, D = qshape
    B, Hkv = kv_len.numel(), cache.k.shape[1]
    c = _cache(cache, dev, B, Hkv, D, "cache")
    qp, qs = _rows(q, dev, qshape, "q")
    op, od = _out(out, dev, qshape)
    o = _score_opts(dev, causal, softcap, slopes, prefix_len, first_key, T, B, Hq)
    wp, wn = _workspace_arg(workspace, dev)
    args = (qp, qs, c, _vec(row_start, dev, _I32, B + 1, "row_start"), _vec(kv_len, dev, _I32, B, "kv_len"), o, T, B, Hq,
            Hkv, D, max_len_hint, scale, op, od, wp, wn, _vec(err_flag, dev, _I32, 1, "err_flag"))
    if _stall_head is None:
        st = _lib.dr_prompt_attn(*args, _stream_arg(stream, dev))
    else:
        st = _lib.dr_prompt_attn_stall_test(*args, _stall_head, _stream_arg(stream, dev))
    if st:
        raise DrError("dr_prompt_attn", st)
    return out


def dr_prompt_attn_stall_test(stall_head: int, *args, **kwargs) -> torch.Tensor:
    """Test hook: dr_prompt_attn with one CTA of key/value head stall_head made to time out (see dr_api.h)."""
    return dr_prompt_attn(*args, _stall_head=int(stall_head), **kwargs)


def dr_shared_prefix_attn_workspace(B: int, Hq: int, Hkv: int, max_prefix: int, num_sms: int | None = None) -> int:
    """Bytes of workspace dr_shared_prefix_attn needs for prefixes of up to max_prefix keys."""
    return int(_lib.dr_shared_prefix_attn_workspace(B, Hq, Hkv, max_prefix, _sms() if num_sms is None else num_sms))


def dr_shared_prefix_attn(q: torch.Tensor, prefix: KVCache, prefix_len: torch.Tensor, out: torch.Tensor,
                          workspace: torch.Tensor, cache: KVCache | None = None, seq_len: torch.Tensor | None = None,
                          softcap: float = 0.0, slopes: torch.Tensor | None = None, max_prefix_hint: int = 0,
                          max_seq_len_hint: int = 0, scale: float = 0.0, err_flag: torch.Tensor | None = None,
                          stream=None, _stall_head=None) -> torch.Tensor:
    """One query per row, q [B,Hq,D], over the one-row cache `prefix` that all rows share and the row's own keys."""
    dev = _device()
    qshape = _shape3(q, "q")
    B, Hq, D = qshape
    Hkv = prefix.k.shape[1]
    if (cache is None) != (seq_len is None):
        raise ValueError("cache and seq_len go together")
    pc = _cache(prefix, dev, 1, Hkv, D, "prefix")
    cp = None if cache is None else _cache(cache, dev, B, Hkv, D, "cache")
    qp, qs = _rows(q, dev, qshape, "q")
    op, od = _out(out, dev, qshape)
    o = _score_opts(dev, False, softcap, slopes, None, None, B, B, Hq)
    wp, wn = _workspace_arg(workspace, dev)
    args = (qp, qs, pc, _vec(prefix_len, dev, _I32, 1, "prefix_len"), cp, _vec(seq_len, dev, _I32, B, "seq_len"), o, B,
            Hq, Hkv, D, max_prefix_hint, max_seq_len_hint, scale, op, od, wp, wn,
            _vec(err_flag, dev, _I32, 1, "err_flag"))
    if _stall_head is None:
        st = _lib.dr_shared_prefix_attn(*args, _stream_arg(stream, dev))
    else:
        st = _lib.dr_shared_prefix_attn_stall_test(*args, _stall_head, _stream_arg(stream, dev))
    if st:
        raise DrError("dr_shared_prefix_attn", st)
    return out


def dr_shared_prefix_attn_stall_test(stall_head: int, *args, **kwargs) -> torch.Tensor:
    """Test hook: dr_shared_prefix_attn with one CTA of key/value head stall_head made to time out (see dr_api.h)."""
    return dr_shared_prefix_attn(*args, _stall_head=int(stall_head), **kwargs)


# The layer calls: as above, checks written out flat.
_ACTS = {None: DR_ACT_NONE, "none": DR_ACT_NONE, "relu": DR_ACT_RELU, "gelu": DR_ACT_GELU, "gelu_tanh": DR_ACT_GELU_TANH,
         "silu": DR_ACT_SILU}
_NORMS = {"none": DR_NORM_NONE, "layer": DR_NORM_LAYER, "rms": DR_NORM_RMS}
_pack_linear_opts = struct.Struct("@iiPPq").pack   # dr_linear_opts
_pack_linear_out = struct.Struct("@Pqi4x").pack    # dr_linear_out
_pack_norm = struct.Struct("@ifPP").pack           # dr_norm
assert struct.calcsize("@iiPPq") == ctypes.sizeof(dr_linear_opts)
assert struct.calcsize("@Pqi4x") == ctypes.sizeof(dr_linear_out)
assert struct.calcsize("@ifPP") == ctypes.sizeof(dr_norm)


def _tokens(t, dev: int, dtype, shape, name: str):
    """(address, elements between tokens) of a tensor of shape (T, n) whose rows are dense but may lie apart."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, dev, dtype, shape, name)
    if shape[0] == 1:
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have contiguous rows")
        return t.data_ptr(), (shape[1] + 7) & -8   # no second row: any stride will do
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), s0


def _float_type(t, name: str):
    dt = t.dtype
    if dt is _BF16:
        return DR_BF16
    if dt is _F32:
        return DR_F32
    raise ValueError(f"{name} must be {_BF16} or {_F32}, got {dt}")


def dr_linear(x: torch.Tensor, W: torch.Tensor, out, bias: torch.Tensor | None = None, act: str | None = None,
              gated: bool = False, residual: torch.Tensor | None = None, err_flag: torch.Tensor | None = None, stream=None,
              _stall_tile=None):
    """out = residual + act(x W^T + bias): x [T, K] bf16, W [N, K] bf16 ([2N, K] when gated), out [T, N] bf16 or float32.

    act: None, "relu", "gelu", "gelu_tanh" or "silu"; gated: the activated first N columns times the last N.  out may be
    a list of up to four [T, n] tensors of one type that share the columns (all but the last a multiple of 64 wide).
    x, out and residual may be slices with dense rows; residual may be out itself.
    """
    dev = _device()
    shape, wshape = x.shape, W.shape
    if len(shape) != 2 or len(wshape) != 2:
        raise ValueError("x must be [T, K] and W [N, K]")
    T, K = shape
    rows = wshape[0]
    xp, xs = _tokens(x, dev, _BF16, shape, "x")
    if wshape[1] != K or W.get_device() != dev or W.dtype is not _BF16 or not W.is_contiguous():
        _refuse(W, dev, _BF16, (rows, K), "W")
    if isinstance(out, torch.Tensor):
        od, dt = _float_type(out, "out"), out.dtype
        if out.dim() != 2:
            raise ValueError("out must be [T, N]")
        N, n_outs = out.shape[1], 1
        packed = _pack_linear_out(*_tokens(out, dev, dt, (T, N), "out"), N)
    else:
        n_outs = len(out)
        if n_outs < 1 or n_outs > DR_LINEAR_MAX_OUTS:
            raise ValueError(f"out must hold 1 to {DR_LINEAR_MAX_OUTS} tensors")
        od, dt = _float_type(out[0], "out"), out[0].dtype
        N, packed = 0, b""
        for o in out:
            if o.dim() != 2:
                raise ValueError("out must be [T, N]")
            n = o.shape[1]
            packed += _pack_linear_out(*_tokens(o, dev, dt, (T, n), "out"), n)
            N += n
    if rows != (2 * N if gated else N):
        raise ValueError(f"W must have {2 * N if gated else N} rows for {N} columns, has {rows}")
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(k for k in _ACTS if k)}, got {act!r}")
    rp, rs = (0, 0) if residual is None else _tokens(residual, dev, dt, (T, N), "residual")
    bp = 0 if bias is None else _vec(bias, dev, _BF16, rows, "bias")
    opts = _pack_linear_opts(code, 1 if gated else 0, bp, rp, rs)
    args = (xp, xs, W.data_ptr(), opts, T, K, N, packed, n_outs, od,
            None if err_flag is None else _vec(err_flag, dev, _I32, 1, "err_flag"))
    if _stall_tile is None:
        st = _lib.dr_linear(*args, _stream_arg(stream, dev))
    else:
        st = _lib.dr_linear_stall_test(*args, _stall_tile, _stream_arg(stream, dev))
    if st:
        raise DrError("dr_linear", st)
    return out


def dr_linear_stall_test(stall_tile: int, *args, **kwargs):
    """Test hook: dr_linear with the CTAs of output tile `stall_tile` made to time out (see dr_api.h)."""
    return dr_linear(*args, _stall_tile=int(stall_tile), **kwargs)


@dataclasses.dataclass
class Norm:
    """A norm over a token's elements: kind "layer" or "rms" ("none": nothing), weight and bias [Dm] bf16 or None."""

    kind: str
    eps: float = 1e-5
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None


def _norm_arg(n: Norm, dev: int, Dm: int, name: str):
    kind = _NORMS.get(n.kind)
    if kind is None:
        raise ValueError(f"{name}.kind must be one of {sorted(_NORMS)}, got {n.kind!r}")
    w, b = n.weight, n.bias
    return _pack_norm(kind, n.eps, 0 if w is None else _vec(w, dev, _BF16, Dm, name + ".weight"),
                      0 if b is None else _vec(b, dev, _BF16, Dm, name + ".bias"))


def dr_residual_norm(x: torch.Tensor, y: torch.Tensor | None = None, pre: Norm | None = None,
                     residual: torch.Tensor | None = None, h: torch.Tensor | None = None, post: Norm | None = None,
                     gate: torch.Tensor | None = None, scale: float = 1.0, stream=None) -> None:
    """h = residual + scale * gate * post(x) and y = pre(h), rows of [T, Dm]; what is None is left out.

    x, y: bf16 or float32; residual and h: of one type, bf16 or float32 (h may be residual itself); gate: bf16 [Dm] for all
    tokens or [T, Dm].
    """
    dev = _device()
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [T, Dm]")
    T, Dm = shape
    xd = _float_type(x, "x")
    xp, xs = _tokens(x, dev, x.dtype, shape, "x")
    hd, rp, rs, hp, hs, yp, ys, yd, gp, gs = DR_BF16, None, 0, None, 0, None, 0, DR_BF16, None, 0
    if residual is not None:
        hd = _float_type(residual, "residual")
        rp, rs = _tokens(residual, dev, residual.dtype, shape, "residual")
    if h is not None:
        hd = _float_type(h, "h")
        hp, hs = _tokens(h, dev, h.dtype if residual is None else residual.dtype, shape, "h")
    if y is not None:
        yd = _float_type(y, "y")
        yp, ys = _tokens(y, dev, y.dtype, shape, "y")
    if gate is not None:
        if gate.dim() == 1:
            gp = _vec(gate, dev, _BF16, Dm, "gate")
        else:
            gp, gs = _tokens(gate, dev, _BF16, shape, "gate")
    st = _lib.dr_residual_norm(xp, xs, xd, None if post is None else _norm_arg(post, dev, Dm, "post"), gp, gs, scale, rp, rs, hp,
                               hs, hd, None if pre is None else _norm_arg(pre, dev, Dm, "pre"), yp, ys, yd, T, Dm,
                               _stream_arg(stream, dev))
    if st:
        raise DrError("dr_residual_norm", st)


def loaded_library_path() -> str:
    return LIB_PATH
