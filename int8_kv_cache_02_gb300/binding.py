"""Thin ctypes binding over ``libint8kv.so`` (the C ABI of include/int8kv.h).

Only argument marshalling happens here: torch tensors are checked for device,
dtype and contiguity and turned into raw pointers; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: when
the library is missing or a call fails, an exception is raised.

Function names follow the C ABI.  ``KVPool`` is a convenience owner of the
device regions (allocated with torch, which only provides memory).
"""

import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libint8kv.so")

K8V8, K8V16, K16V8, K8V4, Q4_0 = 0, 1, 2, 3, 4
K8V8_BLOCK, F8_BLOCK = 8, 9     # one fp32 scale per (group_size positions, kv head)
VARIANTS = {"k8v8": K8V8, "k8v16": K8V16, "k16v8": K16V8, "k8v4": K8V4, "q4_0": Q4_0,
            "k8v8_block": K8V8_BLOCK, "f8_block": F8_BLOCK}
REGION_K_STORE, REGION_V_STORE, REGION_K_SCALES, REGION_V_SCALES = 0, 1, 2, 3
DEVERR_PAGE_ID, DEVERR_LENGTH, DEVERR_TIMEOUT = 1, 2, 4
DEVERR_NO_PAGE, DEVERR_FORK = 8, 16
ERR_FORMAT = -9
DECODE_AUTO, DECODE_WARP_MMA, DECODE_SIMT = 0, 1, 3
ROPE_STYLES = {"halves": 0, "pairs": 1}

_c_int, _c_size, _vp, _c_float = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_c_ll = ctypes.c_longlong
_SIGS = {
    "int8kv_status_string": (ctypes.c_char_p, [_c_int]),
    "int8kv_pool_region_bytes": (_c_int, [_c_int] * 8 + [ctypes.POINTER(_c_size)]),
    "kv_pool_create": (_c_int, [ctypes.POINTER(_vp)] + [_c_int] * 7 + [_vp] * 5),
    "kv_pool_destroy": (None, [_vp]),
    "kv_quant_append": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _c_int, _vp, _vp, _c_int, _vp]),
    "kv_rope_append": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _c_ll, _c_ll, _c_ll, _c_int, _c_int,
                                _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _vp,
                                _vp, _vp, _c_int, _vp]),
    "kv_rope_append_packed": (_c_int, [ctypes.c_char_p]),
    "attn_decode_scored_int8_packed": (_c_int, [ctypes.c_char_p]),
    "attn_prefill_chunk_scored_int8_packed": (_c_int, [ctypes.c_char_p]),
    "kv_verify_drafts_packed": (_c_int, [ctypes.c_char_p]),
    "kv_verify_drafts": (_c_int, [_c_int, _c_int, _c_int, _vp, _c_ll, _vp, _c_ll, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp, _vp]),
    "attn_decode_scored_int8": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _vp, _c_int,
                                         _c_int, _c_float, _c_float, _vp, _vp, _c_int, _vp, _vp,
                                         _c_size, _vp]),
    "attn_prefill_chunk_scored_int8": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_int,
                                                _c_int, _c_float, _c_float, _vp, _c_int, _c_int, _vp,
                                                _vp, _c_size, _vp]),
    "attn_decode_n_splits": (_c_int, [_vp, _c_int, _c_int]),
    "attn_decode_workspace_bytes": (_c_int, [_c_int] * 5 + [ctypes.POINTER(_c_size)]),
    "attn_decode_int8": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _vp, _vp, _c_int, _c_int,
                                  _c_float, _c_int, _vp, _vp, _c_size, _vp]),
    "kv_pool_read_device_error": (_c_int, [_vp, ctypes.POINTER(ctypes.c_int32), _vp]),
    "attn_decode_append_int8": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp,
                                         _c_int, _c_int, _c_float, _c_int, _vp, _vp, _c_size,
                                         _vp]),
    "attn_decode_multi_int8": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _vp,
                                        _c_int, _c_float, _c_int, _vp, _vp, _c_size, _vp]),
    "attn_prefill_n_splits": (_c_int, [_vp, _c_int, _c_int, _c_int]),
    "attn_prefill_workspace_bytes": (_c_int, [_c_int] * 5 + [ctypes.POINTER(_c_size)]),
    "attn_prefill_chunk_int8": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_int,
                                         _c_float, _c_int, _vp, _vp, _c_size, _vp]),
    "attn_decode_int8_noalloc": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _vp, _vp, _c_int,
                                          _c_int, _c_float, _c_int, _vp, _vp]),
    "kv_pool_set_decode_kernel": (_c_int, [_vp, _c_int]),
    "kv_pool_image_bytes": (_c_int, [_vp, _c_int, _vp, ctypes.POINTER(_c_size)]),
    "kv_pool_test_expire_waits": (_c_int, [_vp, ctypes.c_uint32]),
    "kv_pool_test_expire_prefill_waits": (_c_int, [_vp, ctypes.c_uint32]),
    "kv_pool_save": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _vp, _c_size, _vp, _c_size, _vp]),
    "kv_pages_workspace_bytes": (_c_int, [_vp, _c_int, ctypes.POINTER(_c_size)]),
    "kv_pages_copy": (_c_int, [_vp, _c_int, _vp, _vp, _vp]),
    "kv_pages_resize": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _c_size, _vp]),
    "kv_pages_fork": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp,
                               _c_size, _vp]),
    "kv_pages_compact": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size,
                                  _vp]),
    "kv_pool_load": (_c_int, [_vp, _vp, _c_size, _c_int, _vp, _c_int, _vp, _c_size, _vp, _vp]),
}

_lib = None

# Arguments of the packed calls as 64-bit words (ctypes takes 70 ns and more for each of its own).
_pack_rope = struct.Struct("24q").pack
_pack_decode = struct.Struct("10q2d7q").pack
_pack_chunk = struct.Struct("9q2d7q").pack
_pack_verify = struct.Struct("16q").pack


class Int8KVError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_name(status)} ({status})")


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "int8_kv_cache_02_gb300.build.build() (nvcc, sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_name(status):
    return lib().int8kv_status_string(status).decode()


def int8kv_status_string(status):
    return status_name(status)


def _check(status, where):
    if status != 0:
        raise Int8KVError(status, where)


# The current stream's handle of a device, without building a torch.cuda.Stream for every call,
# and the current device, without the lazy initialisation (a call's tensors are on a device).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t, dtype, name):
    """The address of a contiguous CUDA tensor of this dtype (argtypes take the integer)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def int8kv_pool_region_bytes(n_layers, n_kv_heads, head_dim, group_size, page_size, n_pages,
                             variant, region):
    out = _c_size(0)
    _check(lib().int8kv_pool_region_bytes(n_layers, n_kv_heads, head_dim, group_size, page_size,
                                          n_pages, variant, region, ctypes.byref(out)),
           "int8kv_pool_region_bytes")
    return out.value


def kv_pool_create(n_layers, n_kv_heads, head_dim, group_size, page_size, n_pages, variant,
                   k_store, v_store, k_scales, v_scales, dev_error):
    """Raw descriptor over caller tensors (any dtype; only the pointers are used)."""
    h = ctypes.c_void_p()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    _check(lib().kv_pool_create(ctypes.byref(h), n_layers, n_kv_heads, head_dim, group_size,
                                page_size, n_pages, variant, ptr(k_store), ptr(v_store),
                                ptr(k_scales), ptr(v_scales), ptr(dev_error)), "kv_pool_create")
    return h


def kv_pool_destroy(handle):
    lib().kv_pool_destroy(handle)


def kv_quant_append(pool, layer, k_new, v_new, seq_pos, page_table, stream=None):
    """k_new, v_new: fp16 [n_seqs][n_new][Hkv][D]; seq_pos int32 [n_seqs];
    page_table int32 [n_seqs][max_pages]."""
    n_seqs, n_new = k_new.shape[0], k_new.shape[1]
    _block_rows(pool, k_new, (n_seqs, n_new), "k_new")
    _block_rows(pool, v_new, (n_seqs, n_new), "v_new")
    if getattr(pool, "block", False):
        _shape(seq_pos, (n_seqs,), "seq_pos")
        _shape(page_table, (n_seqs, page_table.shape[-1]), "page_table")
        _here(pool, seq_pos, page_table)
    _check(lib().kv_quant_append(pool.handle, layer, _dev(k_new, torch.float16, "k_new"),
                                 _dev(v_new, torch.float16, "v_new"), n_seqs, n_new,
                                 _dev(seq_pos, torch.int32, "seq_pos"),
                                 _dev(page_table, torch.int32, "page_table"),
                                 page_table.shape[1], _stream(stream)), "kv_quant_append")


def _handle(pool):
    h = pool.handle
    return (h.value or 0) if h is not None else 0


def _ptr(t, dtype, shape, device, name):
    """The address of a contiguous tensor of this dtype and shape on a device: one test where all is
    well (a step's calls are short next to their checks), and what is wrong where it is not."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name)
    _shape(t, shape, name)
    raise ValueError(f"{name} is on device {t.get_device()}, not on {device}")


def _token_rows(t, shape, device, name):
    """Address and token stride of fp16 rows [n_seqs][n_new][n_heads][head_dim], evenly spaced (a part
    of a wider projection's rows will do)."""
    try:
        there = t.dtype is torch.float16 and t.shape == shape and t.get_device() == device
    except AttributeError:
        there = False
    if not there:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        if t.dtype != torch.float16:
            raise TypeError(f"{name} must be {torch.float16}, got {t.dtype}")
        _shape(t, shape, name)
        raise ValueError(f"{name} is on device {t.get_device()}, not on {device}")
    seqs, n_new, n_heads, head_dim = shape
    if t.is_contiguous():
        return t.data_ptr(), n_heads * head_dim
    s0, s1, s2, s3 = t.stride()
    if n_new <= 1:
        s1 = s0 if seqs > 1 else n_heads * head_dim
    if s3 != 1 or (n_heads > 1 and s2 != head_dim) or (seqs > 1 and s0 != n_new * s1):
        raise ValueError(f"{name}'s tokens must lie evenly apart, each token's heads together")
    return t.data_ptr(), s1


def kv_rope_append(pool, layer, k_new, v_new, seq_pos, page_table, rope_table, q=None, q_out=None,
                   positions=None, pair_axis=None, rope_dim=None, style="halves", new_lens=None,
                   stream=None):
    """Rotate q (fp16 [n_seqs][n_new][H][D], may be None) into q_out (the same shape, contiguous) and
    k_new (fp16 [n_seqs][n_new][Hkv][D]) by their positions, and append k_new and v_new behind
    seq_pos (int32 [n_seqs]).

    rope_table: fp32 [n_table][rope_dim], cosines then sines.  positions: int32
    [n_axes][n_seqs][n_new] or [n_seqs][n_new]; None: seq_pos[b] + i.  pair_axis: uint8
    [rope_dim / 2] on the HOST, the axis of each pair.  new_lens: int32 [n_seqs], tokens that each
    sequence brings.  q, k_new and v_new may be parts of one projection's rows."""
    dev, i32 = pool.device_index, torch.int32
    if k_new.dim() != 4 or page_table.dim() != 2 or rope_table.dim() != 2:
        raise ValueError("k_new must have shape [n_seqs][n_new][n_kv_heads][head_dim], page_table "
                         "[n_seqs][max_pages], rope_table [n_table][rope_dim]")
    n_seqs, n_new = k_new.shape[:2]
    shape = (n_seqs, n_new, pool.n_kv_heads, pool.head_dim)
    k, ks = _token_rows(k_new, shape, dev, "k_new")
    v, vs = _token_rows(v_new, shape, dev, "v_new")
    qp = qo = axis = at = lens = n_heads = qs = 0
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must have shape [n_seqs][n_new][n_heads][head_dim]")
        n_heads = q.shape[2]
        shape = (n_seqs, n_new, n_heads, pool.head_dim)
        qp, qs = _token_rows(q, shape, dev, "q")
        qo = _ptr(q_out, torch.float16, shape, dev, "q_out")
    n_table, dim = rope_table.shape
    if rope_dim is not None and rope_dim != dim:
        raise ValueError(f"rope_table must have shape [n_table][{rope_dim}]")
    n_axes = 1
    if positions is not None:
        if positions.dim() == 3:
            n_axes = positions.shape[0]
            at = _ptr(positions, i32, (n_axes, n_seqs, n_new), dev, "positions")
        else:
            at = _ptr(positions, i32, (n_seqs, n_new), dev, "positions")
    if pair_axis is not None:
        if pair_axis.is_cuda or pair_axis.dtype != torch.uint8 or not pair_axis.is_contiguous():
            raise TypeError("pair_axis must be a contiguous uint8 tensor on the host")
        _shape(pair_axis, (dim // 2,), "pair_axis")
        axis = pair_axis.data_ptr()
    if new_lens is not None:
        lens = _ptr(new_lens, i32, (n_seqs,), dev, "new_lens")
    max_pages = page_table.shape[1]
    _check((_lib or lib()).kv_rope_append_packed(_pack_rope(
        _handle(pool), layer, qp, k, v, qs, ks, vs, n_seqs, n_new, n_heads,
        _ptr(seq_pos, i32, (n_seqs,), dev, "seq_pos"), lens,
        _ptr(rope_table, torch.float32, (n_table, dim), dev, "rope_table"), n_table, dim,
        ROPE_STYLES[style], at, n_axes, axis, qo,
        _ptr(page_table, i32, (n_seqs, max_pages), dev, "page_table"), max_pages,
        _stream(stream))), "kv_rope_append")


def _prob_rows(t, shape, device, name):
    """Address and row stride of fp32 probabilities [batch][rows][vocab], rows evenly spaced."""
    try:
        there = t.dtype is torch.float32 and t.shape == shape and t.get_device() == device
    except AttributeError:
        there = False
    if not there:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be {torch.float32}, got {t.dtype}")
        _shape(t, shape, name)
        raise ValueError(f"{name} is on device {t.get_device()}, not on {device}")
    batch, rows, vocab = shape
    if t.is_contiguous():
        return t.data_ptr(), vocab
    s0, s1, s2 = t.stride()
    if rows <= 1:
        s1 = s0 if batch > 1 else vocab
    if (vocab > 1 and s2 != 1) or (batch > 1 and s0 != rows * s1):
        raise ValueError(f"{name}'s rows must lie evenly apart")
    return t.data_ptr(), s1


def kv_verify_drafts(target_probs, draft_tokens, accept_u, sample_u, tokens, n_accepted,
                     draft_probs=None, n_drafts=None, seq_lens=None, seq_lens_out=None,
                     stream=None):
    """Accept drafted tokens (int32 [batch][n_draft]) by the target's probabilities (fp32
    [batch][n_draft + 1][vocab]) and draw the token behind them.

    draft_probs: fp32 [batch][n_draft][vocab], None for drafts without probabilities; accept_u fp32
    [batch][n_draft], sample_u fp32 [batch]; n_drafts int32 [batch], drafts of each sequence.
    Writes tokens (int32 [batch][n_draft + 1]) and n_accepted (int32 [batch]), and seq_lens less the
    refused drafts to seq_lens_out (int32 [batch] each).  Vocabularies may be padded: a slice of
    wider rows will do.  The tensors are on the current device."""
    if draft_tokens.dim() != 2 or target_probs.dim() != 3:
        raise ValueError("draft_tokens must have shape [batch][n_draft], target_probs "
                         "[batch][n_draft + 1][vocab]")
    dev, i32, f32 = target_probs.get_device(), torch.int32, torch.float32
    if dev < 0:
        raise ValueError("target_probs must be on a CUDA device")
    if dev != _device():
        raise ValueError(f"target_probs is on device {dev}, the current one is {_device()}")
    batch, n = draft_tokens.shape
    vocab = target_probs.shape[2]
    one = (batch,)
    p, ps = _prob_rows(target_probs, (batch, n + 1, vocab), dev, "target_probs")
    q, qs = (_prob_rows(draft_probs, (batch, n, vocab), dev, "draft_probs")
             if draft_probs is not None else (0, 0))
    _check((_lib or lib()).kv_verify_drafts_packed(_pack_verify(
        batch, n, vocab, p, ps, q, qs, _ptr(draft_tokens, i32, (batch, n), dev, "draft_tokens"),
        _ptr(n_drafts, i32, one, dev, "n_drafts") if n_drafts is not None else 0,
        _ptr(accept_u, f32, (batch, n), dev, "accept_u"),
        _ptr(sample_u, f32, one, dev, "sample_u"),
        _ptr(tokens, i32, (batch, n + 1), dev, "tokens"),
        _ptr(n_accepted, i32, one, dev, "n_accepted"),
        _ptr(seq_lens, i32, one, dev, "seq_lens") if seq_lens is not None else 0,
        _ptr(seq_lens_out, i32, one, dev, "seq_lens_out") if seq_lens_out is not None else 0,
        _stream(stream))), "kv_verify_drafts")


def attn_decode_n_splits(pool, batch, max_ctx):
    n = lib().attn_decode_n_splits(pool.handle, batch, max_ctx)
    if n < 0:
        raise Int8KVError(n, "attn_decode_n_splits")
    return n


def attn_decode_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, n_splits):
    out = _c_size(0)
    _check(lib().attn_decode_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, n_splits,
                                             ctypes.byref(out)), "attn_decode_workspace_bytes")
    return out.value


def attn_decode_int8(pool, layer, q, seq_lens, page_table, out, workspace=None, window=0,
                     softmax_scale=0.0, n_splits=0, stream=None):
    """q fp16 [B][H][D]; seq_lens int32 [B]; page_table int32 [B][max_pages];
    out fp32 [B][H][D]; workspace uint8 tensor (any contents) or None."""
    B, H = q.shape[0], q.shape[1]
    _block_call(pool, q, seq_lens, page_table, out, workspace)
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(lib().attn_decode_int8(pool.handle, layer, _dev(q, torch.float16, "q"), B, H,
                                  _dev(seq_lens, torch.int32, "seq_lens"),
                                  _dev(page_table, torch.int32, "page_table"),
                                  page_table.shape[1], window, float(softmax_scale), n_splits,
                                  _dev(out, torch.float32, "out"), ws, nbytes, _stream(stream)),
           "attn_decode_int8")


def attn_decode_int8_noalloc(pool, layer, q, seq_lens, page_table, out, window=0,
                             softmax_scale=0.0, n_splits=0, stream=None):
    """attn_decode_int8 without a workspace: the partials use the library's own
    fixed scratch (for callers that cannot allocate device memory)."""
    B, H = q.shape[0], q.shape[1]
    _block_call(pool, q, seq_lens, page_table, out)
    _check(lib().attn_decode_int8_noalloc(pool.handle, layer, _dev(q, torch.float16, "q"), B, H,
                                          _dev(seq_lens, torch.int32, "seq_lens"),
                                          _dev(page_table, torch.int32, "page_table"),
                                          page_table.shape[1], window, float(softmax_scale),
                                          n_splits, _dev(out, torch.float32, "out"),
                                          _stream(stream)), "attn_decode_int8_noalloc")


def attn_decode_append_int8(pool, layer, q, k_new, v_new, seq_lens, page_table, out,
                            workspace=None, window=0, softmax_scale=0.0, n_splits=0, stream=None):
    """Append k_new, v_new (fp16 [B][Hkv][D]) at position seq_lens[b] - 1, then decode."""
    B, H = q.shape[0], q.shape[1]
    _block_rows(pool, k_new, (B,), "k_new")
    _block_rows(pool, v_new, (B,), "v_new")
    _block_call(pool, q, seq_lens, page_table, out, workspace)
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(lib().attn_decode_append_int8(pool.handle, layer, _dev(q, torch.float16, "q"),
                                         _dev(k_new, torch.float16, "k_new"),
                                         _dev(v_new, torch.float16, "v_new"), B, H,
                                         _dev(seq_lens, torch.int32, "seq_lens"),
                                         _dev(page_table, torch.int32, "page_table"),
                                         page_table.shape[1], window, float(softmax_scale),
                                         n_splits, _dev(out, torch.float32, "out"), ws, nbytes,
                                         _stream(stream)), "attn_decode_append_int8")


def attn_decode_multi_int8(pool, layer, q, seq_lens, page_table, out, workspace=None,
                           softmax_scale=0.0, n_splits=0, stream=None):
    """Decode of a window of queries per sequence, causal within the window.

    q: fp16 [B][q_len][H][D]; query i of sequence b sits at position
    seq_lens[b] - q_len + i.  out: fp32 [B][q_len][H][D].  The workspace is sized
    by attn_decode_workspace_bytes(B * q_len, H, ...)."""
    B, Q, H = q.shape[0], q.shape[1], q.shape[2]
    _block_call(pool, q, seq_lens, page_table, out, workspace)
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(lib().attn_decode_multi_int8(pool.handle, layer, _dev(q, torch.float16, "q"), B, Q, H,
                                        _dev(seq_lens, torch.int32, "seq_lens"),
                                        _dev(page_table, torch.int32, "page_table"),
                                        page_table.shape[1], float(softmax_scale), n_splits,
                                        _dev(out, torch.float32, "out"), ws, nbytes,
                                        _stream(stream)), "attn_decode_multi_int8")


def _scored_args(pool, q, out, slopes, workspace):
    """Addresses of a scored call's queries, output, slopes and workspace, and the workspace's size."""
    if not pool.block:
        raise ValueError("shaped scores want a block-scaled pool")
    dev = pool.device_index
    shape = q.shape
    if shape[-1] != pool.head_dim:
        raise ValueError(f"q must have shape [..., {pool.head_dim}], got {list(shape)}")
    ws = nbytes = 0
    if workspace is not None:
        nbytes = workspace.numel()
        ws = _ptr(workspace, torch.uint8, (nbytes,), dev, "workspace")
    return (_ptr(q, torch.float16, shape, dev, "q"), _ptr(out, torch.float32, shape, dev, "out"),
            _ptr(slopes, torch.float32, (shape[-2],), dev, "slopes") if slopes is not None else 0,
            ws, nbytes)


def attn_decode_scored_int8(pool, layer, q, seq_lens, page_table, out, workspace=None, window=0,
                            softcap=0.0, slopes=None, prefix_lens=None, softmax_scale=0.0,
                            n_splits=0, stream=None):
    """Decode with scores capped at softcap by a tanh, biased by slopes[h] * (key - query) (fp32 [H]),
    and a prefix that every query sees (prefix_lens int32 [B]) beside its window.

    q: fp16 [B][H][D], or a window of queries [B][q_len][H][D], the last of them at seq_lens[b] - 1;
    out: fp32, the same shape; block-scaled pools."""
    n = q.dim()
    if n not in (3, 4) or page_table.dim() != 2:
        raise ValueError("q must have shape [B][H][D] or [B][q_len][H][D], page_table [B][max_pages]")
    qp, op, sp, ws, nbytes = _scored_args(pool, q, out, slopes, workspace)
    dev, i32, B, max_pages = pool.device_index, torch.int32, q.shape[0], page_table.shape[1]
    _check((_lib or lib()).attn_decode_scored_int8_packed(_pack_decode(
        _handle(pool), layer, qp, B, q.shape[1] if n == 4 else 1, q.shape[-2],
        _ptr(seq_lens, i32, (B,), dev, "seq_lens"),
        _ptr(page_table, i32, (B, max_pages), dev, "page_table"), max_pages, window, softmax_scale,
        softcap, sp,
        _ptr(prefix_lens, i32, (B,), dev, "prefix_lens") if prefix_lens is not None else 0,
        n_splits, op, ws, nbytes, _stream(stream))), "attn_decode_scored_int8")


def attn_prefill_n_splits(pool, n_new, n_heads, start_pos):
    n = lib().attn_prefill_n_splits(pool.handle, n_new, n_heads, start_pos)
    if n < 0:
        raise Int8KVError(n, "attn_prefill_n_splits")
    return n


def attn_prefill_workspace_bytes(n_new, n_heads, n_kv_heads, head_dim, n_splits):
    out = _c_size(0)
    _check(lib().attn_prefill_workspace_bytes(n_new, n_heads, n_kv_heads, head_dim, n_splits,
                                              ctypes.byref(out)), "attn_prefill_workspace_bytes")
    return out.value


def attn_prefill_chunk_int8(pool, layer, q, start_pos, page_table, out, workspace=None,
                            softmax_scale=0.0, n_splits=0, stream=None):
    """q fp16 [n_new][H][D]; page_table int32 [max_pages] (one sequence); out fp32 [n_new][H][D]."""
    n_new, H = q.shape[0], q.shape[1]
    if getattr(pool, "block", False):
        _shape(q, (n_new, H, pool.head_dim), "q")
        _shape(out, q.shape, "out")
        if page_table.numel() != page_table.shape[-1]:
            raise ValueError("page_table must be one sequence's row")
        _here(pool, q, page_table, out, workspace)
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(lib().attn_prefill_chunk_int8(pool.handle, layer, _dev(q, torch.float16, "q"), n_new,
                                         H, start_pos, _dev(page_table, torch.int32, "page_table"),
                                         page_table.shape[-1], float(softmax_scale), n_splits,
                                         _dev(out, torch.float32, "out"), ws, nbytes,
                                         _stream(stream)), "attn_prefill_chunk_int8")


def attn_prefill_chunk_scored_int8(pool, layer, q, start_pos, page_table, out, workspace=None,
                                   window=0, softcap=0.0, slopes=None, prefix_len=0,
                                   softmax_scale=0.0, n_splits=0, stream=None):
    """attn_prefill_chunk_int8 with scores shaped as by attn_decode_scored_int8: q fp16 [n_new][H][D],
    query i at start_pos + i; positions below prefix_len are seen by all; block-scaled pools."""
    if q.dim() != 3:
        raise ValueError("q must have shape [n_new][H][D]")
    qp, op, sp, ws, nbytes = _scored_args(pool, q, out, slopes, workspace)
    row = page_table.shape
    if page_table.numel() != row[-1]:
        raise ValueError("page_table must be one sequence's row")
    _check((_lib or lib()).attn_prefill_chunk_scored_int8_packed(_pack_chunk(
        _handle(pool), layer, qp, q.shape[0], q.shape[1], start_pos,
        _ptr(page_table, torch.int32, row, pool.device_index, "page_table"), row[-1], window,
        softmax_scale, softcap, sp, prefix_len, n_splits, op, ws, nbytes, _stream(stream))),
        "attn_prefill_chunk_scored_int8")


def kv_pool_set_decode_kernel(pool, kind):
    """kind: DECODE_AUTO, DECODE_WARP_MMA or DECODE_SIMT."""
    _check(lib().kv_pool_set_decode_kernel(pool.handle, int(kind)), "kv_pool_set_decode_kernel")


def _here(pool, *tensors):
    """Block-scaled pools and the page calls: tensors of the pool's device, which is current."""
    at = pool.device_index
    for t in tensors:
        if t is not None and t.get_device() != at and t.is_cuda:
            raise ValueError(f"a tensor is on device {t.get_device()}, the pool on {at}")


def _block_rows(pool, t, lead, name):
    """A block-scaled pool's K/V rows have the shape lead + [n_kv_heads][head_dim]."""
    if getattr(pool, "block", False):
        _shape(t, (*lead, pool.n_kv_heads, pool.head_dim), name)
        _here(pool, t)


def _block_call(pool, q, seq_lens, page_table, out, workspace=None):
    """Shapes and devices of a decode call on a block-scaled pool."""
    if getattr(pool, "block", False):
        shape = q.shape
        if shape[-1] != pool.head_dim:
            raise ValueError(f"q must have shape [..., {pool.head_dim}], got {list(shape)}")
        _shape(out, shape, "out")
        _shape(seq_lens, shape[:1], "seq_lens")
        if page_table.shape[:-1] != shape[:1]:
            raise ValueError(f"page_table must have shape [{shape[0]}, max_pages]")
        _here(pool, q, seq_lens, page_table, out, workspace)


def _host_lens(seq_lens):
    lens = torch.as_tensor(seq_lens, dtype=torch.int32).cpu().contiguous()
    return lens, ctypes.c_void_p(lens.data_ptr())


def kv_pool_image_bytes(pool, seq_lens):
    """Bytes of the saved image of sequences of these lengths (a host sequence)."""
    lens, lp = _host_lens(seq_lens)
    out = _c_size(0)
    _check(lib().kv_pool_image_bytes(pool.handle, lens.numel(), lp, ctypes.byref(out)),
           "kv_pool_image_bytes")
    return out.value


def kv_pool_save(pool, seq_lens, page_table, staging=None, stream=None):
    """The saved image (bytes) of positions 0..L_b-1 of every layer of each sequence.
    seq_lens: host lengths; page_table: int32 [n_seqs][max_pages] on the device;
    staging: a device uint8 tensor of at least the image's bytes (allocated here
    when None)."""
    lens, lp = _host_lens(seq_lens)
    n = kv_pool_image_bytes(pool, lens)
    if staging is None:
        staging = torch.empty(max(n, 16), dtype=torch.uint8, device=page_table.device)
    host = torch.empty(max(n, 1), dtype=torch.uint8)
    _check(lib().kv_pool_save(pool.handle, lens.numel(), lp,
                              _dev(page_table, torch.int32, "page_table"), page_table.shape[1],
                              _dev(staging, torch.uint8, "staging"), staging.numel(),
                              ctypes.c_void_p(host.data_ptr()), host.numel(), _stream(stream)),
           "kv_pool_save")
    return bytes(host[:n].numpy())


def kv_pool_load(pool, image, page_table, staging=None, stream=None):
    """Load a saved image into the pool through page_table (int32 [n_seqs][max_pages]
    on the device); returns the sequences' lengths."""
    n_seqs = page_table.shape[0]
    buf = torch.frombuffer(bytearray(image), dtype=torch.uint8) if len(image) else \
        torch.zeros(1, dtype=torch.uint8)
    if staging is None:
        staging = torch.empty(max(len(image), 16), dtype=torch.uint8, device=page_table.device)
    lens = torch.zeros(max(n_seqs, 1), dtype=torch.int32)
    _check(lib().kv_pool_load(pool.handle, ctypes.c_void_p(buf.data_ptr()), len(image), n_seqs,
                              _dev(page_table, torch.int32, "page_table"), page_table.shape[1],
                              _dev(staging, torch.uint8, "staging"), staging.numel(),
                              ctypes.c_void_p(lens.data_ptr()), _stream(stream)), "kv_pool_load")
    return lens[:n_seqs].tolist()


def kv_pages_workspace_bytes(pool, n_seqs):
    out = _c_size(0)
    _check(lib().kv_pages_workspace_bytes(pool.handle, n_seqs, ctypes.byref(out)),
           "kv_pages_workspace_bytes")
    return out.value


def kv_pages_copy(pool, src, dst, stream=None):
    """Copy page src[i] of every layer, codes and scales, to page dst[i] (int32 [n])."""
    s, d = _dev(src, torch.int32, "src"), _dev(dst, torch.int32, "dst")
    _shape(dst, (src.numel(),), "dst")
    _here(pool, src, dst)
    _check(lib().kv_pages_copy(pool.handle, src.numel(), s, d, _stream(stream)), "kv_pages_copy")


def kv_pages_resize(pool, page_refs, page_table, seq_lens, workspace, stream=None):
    """Give every row of page_table (int32 [n_seqs][max_pages]) the pages that seq_lens (int32
    [n_seqs]) needs and take back the others; page_refs: int32 [n_pages]."""
    r, t = _dev(page_refs, torch.int32, "page_refs"), _dev(page_table, torch.int32, "page_table")
    n = _dev(seq_lens, torch.int32, "seq_lens")
    w = _dev(workspace, torch.uint8, "workspace")
    _shape(page_refs, (pool.n_pages,), "page_refs")
    _shape(seq_lens, (page_table.shape[0],), "seq_lens")
    _here(pool, page_refs, page_table, seq_lens, workspace)
    _check(lib().kv_pages_resize(pool.handle, r, t, page_table.shape[0], page_table.shape[1], n,
                                 w, workspace.numel(), _stream(stream)), "kv_pages_resize")


def kv_pages_fork(pool, page_refs, page_table, seq_lens, parents, children, workspace,
                  stream=None):
    """Row children[i] of page_table becomes a fork of row parents[i] (int32 [n_forks] each):
    full pages are shared, the page that the length ends inside is copied."""
    r, t = _dev(page_refs, torch.int32, "page_refs"), _dev(page_table, torch.int32, "page_table")
    n = _dev(seq_lens, torch.int32, "seq_lens")
    p, c = _dev(parents, torch.int32, "parents"), _dev(children, torch.int32, "children")
    w = _dev(workspace, torch.uint8, "workspace")
    _shape(page_refs, (pool.n_pages,), "page_refs")
    _shape(seq_lens, (page_table.shape[0],), "seq_lens")
    _shape(children, (parents.numel(),), "children")
    _here(pool, page_refs, page_table, seq_lens, parents, children, workspace)
    _check(lib().kv_pages_fork(pool.handle, r, t, page_table.shape[0], page_table.shape[1], n,
                               parents.numel(), p, c, w, workspace.numel(), _stream(stream)),
           "kv_pages_fork")


def kv_pages_compact(pool, page_refs, page_table, page_refs_out, page_table_out, n_used,
                     workspace, stream=None):
    """Move the used pages to ids 0 .. n_used - 1 (int32 [1] on the device); the counts and the
    table afterwards go to page_refs_out and page_table_out (which may be the inputs)."""
    r, t = _dev(page_refs, torch.int32, "page_refs"), _dev(page_table, torch.int32, "page_table")
    ro = _dev(page_refs_out, torch.int32, "page_refs_out")
    to = _dev(page_table_out, torch.int32, "page_table_out")
    u = _dev(n_used, torch.int32, "n_used")
    w = _dev(workspace, torch.uint8, "workspace")
    _shape(page_refs, (pool.n_pages,), "page_refs")
    _shape(page_refs_out, (pool.n_pages,), "page_refs_out")
    _shape(page_table_out, page_table.shape, "page_table_out")
    _shape(n_used, (1,), "n_used")
    _here(pool, page_refs, page_table, page_refs_out, page_table_out, n_used, workspace)
    _check(lib().kv_pages_compact(pool.handle, r, t, page_table.shape[0], page_table.shape[1], ro,
                                  to, u, w, workspace.numel(), _stream(stream)),
           "kv_pages_compact")


def kv_pool_test_expire_waits(pool, max_polls):
    """Diagnostic: later decode calls arm their copy waits so that they expire after
    max_polls polls and report INT8KV_DEVERR_TIMEOUT (0 switches it off)."""
    _check(lib().kv_pool_test_expire_waits(pool.handle, int(max_polls)),
           "kv_pool_test_expire_waits")


def kv_pool_read_device_error(pool, stream=None):
    v = ctypes.c_int32(0)
    _check(lib().kv_pool_read_device_error(pool.handle, ctypes.byref(v), _stream(stream)),
           "kv_pool_read_device_error")
    return v.value


def kv_pool_test_expire_prefill_waits(pool, max_us):
    """Diagnostic: later prefill chunks of a block-scaled pool (on the tensor-memory kernel) let a
    wait of every thread block run out after max_us microseconds and report
    INT8KV_DEVERR_TIMEOUT (0 switches it off)."""
    _check(lib().kv_pool_test_expire_prefill_waits(pool.handle, int(max_us)),
           "kv_pool_test_expire_prefill_waits")


class KVPool:
    """Owns the device regions of a pool (torch allocations) and its descriptor."""

    def __init__(self, n_layers, n_kv_heads, head_dim, group_size, page_size, n_pages,
                 variant=K8V8, device=None):
        if isinstance(variant, str):
            variant = VARIANTS[variant]
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.device_index = dev.index
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        self.block = variant in (K8V8_BLOCK, F8_BLOCK)
        if self.block:
            codes = torch.int8 if variant == K8V8_BLOCK else torch.float8_e4m3fn
            self.k_store = torch.zeros(shape, dtype=torch.int8, device=dev).view(codes)
            self.v_store = torch.zeros(shape, dtype=torch.int8, device=dev).view(codes)
            self.k_scales = torch.zeros(shape[:-2] + (page_size // max(group_size, 1),),
                                        dtype=torch.float32, device=dev)
            self.v_scales = torch.zeros_like(self.k_scales)
        else:
            self._rows_with_scales(shape, group_size, variant, dev)
        self.dev_error = torch.zeros(4, dtype=torch.int32, device=dev)
        for region, t in ((REGION_K_STORE, self.k_store), (REGION_V_STORE, self.v_store),
                          (REGION_K_SCALES, self.k_scales), (REGION_V_SCALES, self.v_scales)):
            want = int8kv_pool_region_bytes(n_layers, n_kv_heads, head_dim, group_size,
                                            page_size, n_pages, variant, region)
            have = 0 if t is None else t.numel() * t.element_size()
            assert want == have, (region, want, have)
        self.n_layers, self.n_kv_heads, self.head_dim = n_layers, n_kv_heads, head_dim
        self.group_size, self.page_size, self.n_pages, self.variant = (group_size, page_size,
                                                                       n_pages, variant)
        with torch.cuda.device(dev):     # the descriptor belongs to the device that is current
            self.handle = kv_pool_create(n_layers, n_kv_heads, head_dim, group_size, page_size,
                                         n_pages, variant, self.k_store, self.v_store,
                                         self.k_scales, self.v_scales, self.dev_error)

    def _rows_with_scales(self, shape, group_size, variant, dev):
        head_dim = shape[-1]
        sshape = shape[:-1] + (head_dim // group_size,)
        k8 = variant in (K8V8, K8V16, K8V4)
        v8 = variant in (K8V8, K16V8)
        k4 = variant == Q4_0
        v4 = variant in (K8V4, Q4_0)
        self.k_store = torch.zeros(shape, dtype=torch.int8 if k8 else torch.float16, device=dev)
        self.v_store = torch.zeros(shape, dtype=torch.int8 if v8 else torch.float16, device=dev)
        self.k_scales = torch.zeros(sshape, dtype=torch.float16, device=dev) if k8 else None
        self.v_scales = torch.zeros(sshape, dtype=torch.float16, device=dev) if v8 else None
        if k4:   # 4-bit stores: two codes per byte, one fp16 scale per 32 values
            self.k_store = torch.zeros(shape[:-1] + (head_dim // 2,), dtype=torch.uint8, device=dev)
            self.k_scales = torch.zeros(shape[:-1] + (head_dim // 32,), dtype=torch.float16,
                                        device=dev)
        if v4:
            self.v_store = torch.zeros(shape[:-1] + (head_dim // 2,), dtype=torch.uint8, device=dev)
            self.v_scales = torch.zeros(shape[:-1] + (head_dim // 32,), dtype=torch.float16,
                                        device=dev)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kv_pool_destroy(h)
            self.handle = None

    def set_decode_kernel(self, kind):
        kv_pool_set_decode_kernel(self, kind)

    def decode_workspace(self, batch, n_heads, n_splits):
        n = attn_decode_workspace_bytes(batch, n_heads, self.n_kv_heads, self.head_dim, n_splits)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k_store.device)

    def pages_workspace(self, n_seqs):
        """Workspace of kv_pages_resize, kv_pages_fork and kv_pages_compact for n_seqs rows."""
        return torch.zeros(kv_pages_workspace_bytes(self, n_seqs), dtype=torch.uint8,
                           device=self.k_store.device)
