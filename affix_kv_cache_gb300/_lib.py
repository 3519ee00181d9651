"""ctypes binding of libacache.so (include/acache.h).

Argument marshalling only: every function takes torch tensors (device memory) or plain
integers, passes their device pointers, sizes and the current CUDA stream to the C entry
point of the same name, and raises AcacheError on a non-zero status.  No step of the
path runs here, and there is no fallback: if the library is missing, importing this
module's functions fails loudly.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libacache.so")

ACACHE_OK = 0
ACACHE_ERR_INVALID_ARG = -1
ACACHE_ERR_UNSUPPORTED = -2
ACACHE_ERR_CUDA = -3
ACACHE_ERR_WORKSPACE = -4
ACACHE_ERR_TIMEOUT = -5
ACACHE_F32 = 0
ACACHE_BF16 = 1
ACACHE_PATH_RECOMPUTE = 0
ACACHE_PATH_BLOCK_DECODE = 1
ACACHE_PATH_CUDA_CORES = 2
ACACHE_PATH_RECOMPUTE_PERSISTENT = 3
SLOT_NONE = -1
DEV_BAD_SLOT, DEV_SHARED_WRITE, DEV_BAD_ROW, DEV_BAD_ANCHOR, DEV_NAN, DEV_TIMEOUT = 1, 2, 4, 8, 16, 32
DEV_BAD_LENGTH = 64
DEV_BAD_VALUE = 128
DEV_BAD_TOKEN = 256
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = 0, 1, 2, 3, 4
MAX_ALTERNATIVES = 32

EXPORTS = ("acache_status_string", "acache_version", "acache_wait_budget", "acache_probe_workspace_bytes",
           "acache_probe_scores", "acache_probe_scores_layers", "acache_probe_scores_noalloc", "acache_topk_anchors", "acache_build_slot_maps",
           "acache_write_slots", "acache_slot_attention", "acache_gather_slots",
           "acache_kv_deviation_scores", "acache_slot_attention_dropna", "acache_slot_attention_varlen",
           "acache_slot_attention_path",
           "acache_store_attend", "acache_store_attend_layers", "acache_rerotate_keys", "acache_pool_create",
           "acache_pool_destroy",
           "acache_pool_register_affix", "acache_pool_release_affix", "acache_pool_alloc_private",
           "acache_pool_free_private", "acache_pool_stats",
           "acache_write_slots_q8", "acache_gather_slots_q8", "acache_slot_attention_q8",
           "acache_slot_attention_varlen_q8", "acache_store_attend_q8",
           "acache_rope_init", "acache_rope_init_frequencies", "acache_rotate_qk", "acache_rotate_store",
           "acache_rotate_store_q8", "acache_slot_attention_masked", "acache_slot_attention_masked_varlen",
           "acache_token_scores")


class AcacheError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} returned {status} ({status_string(status)})")
        self.status = status


class AttnDesc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("phase", ctypes.c_uint64 * 64)]


class Mask(ctypes.Structure):
    _fields_ = [("row_range", ctypes.c_void_p), ("q_pos", ctypes.c_void_p), ("slopes", ctypes.c_void_p),
                ("softcap", ctypes.c_float), ("drop_none", ctypes.c_int32)]


def attn_desc(hq: int, hkv: int, d: int, scale: float, dtype) -> AttnDesc:
    if isinstance(dtype, torch.dtype):
        dtype = {torch.float32: ACACHE_F32, torch.bfloat16: ACACHE_BF16}[dtype]
    elif isinstance(dtype, str):
        dtype = {"f32": ACACHE_F32, "bf16": ACACHE_BF16}[dtype]
    return AttnDesc(hq, hkv, d, scale, dtype)


_lib = None


def lib() -> ctypes.CDLL:
    """Load libacache.so (built by __graft_entry__.build() or build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libacache.so is not built ({LIB_PATH} missing); "
                               "run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        D, R, M = ctypes.POINTER(AttnDesc), ctypes.POINTER(Rope), ctypes.POINTER(Mask)
        F = ctypes.c_float
        sig = {
            "acache_status_string": (ctypes.c_char_p, [I]),
            "acache_version": (I, []),
            "acache_wait_budget": (I64, [I64]),
            "acache_probe_workspace_bytes": (S, [D, I, I, I, I]),
            "acache_probe_scores": (I, [D, I, I, I, I, P, I, P, P, P, P, P, P, P, P, S, P, P]),
            "acache_probe_scores_layers": (I, [D, I, I, I, I, I, P, I, P, P, P, P, P, P, P, P, S, P, P]),
            "acache_probe_scores_noalloc": (I, [D, I, I, I, I, P, I, P, P, P, P, P, P, P, P, P]),
            "acache_topk_anchors": (I, [P, I, I, I, P, P, P]),
            "acache_build_slot_maps": (I, [I, I, I, I, I, P, P, P, P, P, P, P]),
            "acache_write_slots": (I, [D, I, I, P, P, P, P, P, I64, I64, P, P]),
            "acache_slot_attention": (I, [D, I, I, P, I, P, P, P, I64, P, P, P]),
            "acache_slot_attention_path": (I, [D, I, I, I]),
            "acache_gather_slots": (I, [D, I, I, P, P, P, I64, P, P, P, P]),
            "acache_kv_deviation_scores": (I, [D, I, I, P, P, P, P, P, P]),
            "acache_slot_attention_dropna": (I, [D, I, I, P, I, P, P, P, I64, P, P, P]),
            "acache_slot_attention_varlen": (I, [D, I, P, I, I, P, P, I, P, P, P, I64, P, I, P, P]),
            "acache_store_attend": (I, [D, I, I, P, P, P, P, P, I64, I64, I, P, I, P, P, P, P]),
            "acache_store_attend_layers": (I, [D, I, I, I, P, P, P, P, P, I64, I64, I, P, I, P, P, P, P]),
            "acache_rerotate_keys": (I, [D, I64, P, P, ctypes.c_int32, ctypes.c_double, I, P]),
            "acache_write_slots_q8": (I, [D, I, I, P, P, P, P, P, P, I64, I64, P, P]),
            "acache_gather_slots_q8": (I, [D, I, I, P, P, P, P, I64, P, P, P, P]),
            "acache_slot_attention_q8": (I, [D, I, I, P, I, P, P, P, P, I64, P, I, P, P]),
            "acache_slot_attention_varlen_q8": (I, [D, I, P, I, I, P, P, I, P, P, P, P, I64, P, I, P, P]),
            "acache_store_attend_q8": (I, [D, I, I, P, P, P, P, P, P, I64, I64, I, P, I, P, P, I, P, P]),
            "acache_rope_init": (I, [ctypes.POINTER(Rope), I, I, ctypes.c_double, I, ctypes.c_double, I64,
                                     ctypes.c_double, ctypes.c_double]),
            "acache_rope_init_frequencies": (I, [ctypes.POINTER(Rope), I, I, ctypes.POINTER(ctypes.c_double),
                                                 ctypes.c_float]),
            "acache_rotate_qk": (I, [D, R, I64, P, P, I64, P, I64, P, P, F, P, I64, P, I64, P]),
            "acache_rotate_store": (I, [D, R, I, I, P, P, P, I64, P, I64, P, I64, P, P, F, P, P, P, I64, I64, P, P]),
            "acache_rotate_store_q8": (I, [D, R, I, I, P, P, P, I64, P, I64, P, I64, P, P, F, P, P, P, P, I64, I64,
                                           P, P]),
            "acache_slot_attention_masked": (I, [D, M, I, I, P, I, P, P, P, I64, P, P, P]),
            "acache_slot_attention_masked_varlen": (I, [D, M, I, P, I, I, P, P, I, P, P, P, I64, P, P, P]),
            "acache_token_scores": (I, [I, I64, I, P, I64, F, P, P, P, I, P, P, P, P]),
            "acache_pool_create": (I, [I64, I64, ctypes.c_int32, ctypes.POINTER(P)]),
            "acache_pool_destroy": (None, [P]),
            "acache_pool_register_affix": (I, [P, ctypes.c_uint64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                               ctypes.POINTER(ctypes.c_int32)]),
            "acache_pool_release_affix": (I, [P, ctypes.c_uint64]),
            "acache_pool_alloc_private": (I, [P, ctypes.c_int32, P, ctypes.POINTER(I64)]),
            "acache_pool_free_private": (I, [P, I64]),
            "acache_pool_stats": (I, [P, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32)]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().acache_status_string(int(status)).decode()


def version() -> int:
    return int(lib().acache_version())


def _p(t):
    if t is None:
        return None
    try:
        return t.data_ptr() or None
    except AttributeError:       # a plain address
        return t or None


def _stream(stream, device=None):
    """The handle of a call's stream; `device`: the current one, where the caller has looked it up."""
    if stream is None:
        if device is not None:
            return torch._C._cuda_getCurrentRawStream(device)
        # the current stream's handle, as torch.cuda.current_stream().cuda_stream gives it in 15 times the
        # time; before torch has touched CUDA that is the default stream
        if not torch.cuda.is_initialized():
            return None
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def _current_device():
    """The device that every tensor of a call lives on; before torch has touched CUDA there is none."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None


def _on(device, t):
    """_p, for a call on `device`."""
    if t is None:
        return None
    try:
        at = t.data_ptr()
        if at and t.get_device() != device:
            raise ValueError(f"tensor on {t.device}, not on the current device")
        return at or None
    except AttributeError:       # a plain address
        return t or None


def _dense(device, t):
    """_on, of a tensor that a call reads or writes as one dense block: with gaps or repeats it were another one, or none."""
    if t is None:
        return None
    try:
        if not t.is_contiguous():
            raise ValueError("a tensor that has to be contiguous is not")
        at = t.data_ptr()
        if at and t.get_device() != device:
            raise ValueError(f"tensor on {t.device}, not on the current device")
        return at or None
    except AttributeError:       # a plain address
        return t or None


def _check(fn, status):
    if status != ACACHE_OK:
        raise AcacheError(fn, status)
    return status


def acache_wait_budget(cycles: int = 0) -> int:
    """Set (cycles > 0) or read (cycles <= 0) the SM-cycle budget of the kernels' bounded
    waits; returns the budget in force before the call (see include/acache.h)."""
    return int(lib().acache_wait_budget(int(cycles)))


def acache_probe_workspace_bytes(desc, batch, seq_len, affix_len, num_masked) -> int:
    return int(lib().acache_probe_workspace_bytes(ctypes.byref(desc), batch, seq_len, affix_len,
                                                  num_masked))


def acache_probe_scores(desc, batch, seq_len, affix_begin, affix_len, masked_rows, num_masked,
                        q, k_req, v_req, k_affix, v_affix, out, scores, workspace,
                        workspace_bytes=None, dev_status=None, stream=None, check=True):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().acache_probe_scores(ctypes.byref(desc), batch, seq_len, affix_begin, affix_len,
                                   _p(masked_rows), num_masked, _p(q), _p(k_req), _p(v_req),
                                   _p(k_affix), _p(v_affix), _p(out), _p(scores), _p(workspace),
                                   workspace_bytes, _p(dev_status), _stream(stream))
    return _check("acache_probe_scores", st) if check else st


def acache_probe_scores_layers(desc, batch, seq_len, affix_begin, affix_len, masked_rows, num_masked,
                               q, k_req, v_req, k_affix, v_affix, out, scores, workspace,
                               workspace_bytes=None, dev_status=None, stream=None, check=True):
    """The probe of every layer in one call (see include/acache.h): q, k_req, v_req, k_affix,
    v_affix and out are lists of tensors, one per layer (out, k_affix and v_affix may be None)."""
    layers = len(q)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    keep = [_ptr_array(x, layers) for x in (q, k_req, v_req, k_affix, v_affix, out)]
    ptrs = [k[0] if k is not None else None for k in keep]
    st = lib().acache_probe_scores_layers(ctypes.byref(desc), layers, batch, seq_len, affix_begin, affix_len,
                                          _p(masked_rows), num_masked, ptrs[0], ptrs[1], ptrs[2], ptrs[3],
                                          ptrs[4], ptrs[5], _p(scores), _p(workspace), workspace_bytes,
                                          _p(dev_status), _stream(stream))
    del keep
    return _check("acache_probe_scores_layers", st) if check else st


def acache_probe_scores_noalloc(desc, batch, seq_len, affix_begin, affix_len, masked_rows,
                                num_masked, q, k_req, v_req, k_affix, v_affix, out, scores,
                                dev_status=None, stream=None, check=True):
    """acache_probe_scores without a workspace, for callers that cannot allocate device
    memory: the scratch is a fixed 16 MiB array inside the library (see include/acache.h)."""
    st = lib().acache_probe_scores_noalloc(ctypes.byref(desc), batch, seq_len, affix_begin,
                                           affix_len, _p(masked_rows), num_masked, _p(q),
                                           _p(k_req), _p(v_req), _p(k_affix), _p(v_affix),
                                           _p(out), _p(scores), _p(dev_status), _stream(stream))
    return _check("acache_probe_scores_noalloc", st) if check else st


def acache_topk_anchors(scores, batch, affix_len, k, anchors, dev_status=None, stream=None,
                        check=True):
    st = lib().acache_topk_anchors(_p(scores), batch, affix_len, k, _p(anchors), _p(dev_status),
                                   _stream(stream))
    return _check("acache_topk_anchors", st) if check else st


def acache_build_slot_maps(batch, seq_len, affix_begin, affix_len, k, anchors, shared_slot,
                           private_slots, write_pos, read_slot, dev_status=None, stream=None,
                           check=True):
    st = lib().acache_build_slot_maps(batch, seq_len, affix_begin, affix_len, k, _p(anchors),
                                      _p(shared_slot), _p(private_slots), _p(write_pos),
                                      _p(read_slot), _p(dev_status), _stream(stream))
    return _check("acache_build_slot_maps", st) if check else st


def acache_write_slots(desc, batch, rows, write_slot, k_new, v_new, k_cache, v_cache, num_slots,
                       private_begin, dev_status=None, stream=None, check=True):
    st = lib().acache_write_slots(ctypes.byref(desc), batch, rows, _p(write_slot), _p(k_new),
                                  _p(v_new), _p(k_cache), _p(v_cache), num_slots, private_begin,
                                  _p(dev_status), _stream(stream))
    return _check("acache_write_slots", st) if check else st


def acache_slot_attention(desc, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, num_slots,
                          out, dev_status=None, stream=None, check=True):
    st = lib().acache_slot_attention(ctypes.byref(desc), batch, n_q, _p(q), seq_len, _p(read_slot),
                                     _p(k_cache), _p(v_cache), num_slots, _p(out), _p(dev_status),
                                     _stream(stream))
    return _check("acache_slot_attention", st) if check else st


def acache_gather_slots(desc, batch, seq_len, read_slot, k_cache, v_cache, num_slots, k_out,
                        v_out, dev_status=None, stream=None, check=True):
    st = lib().acache_gather_slots(ctypes.byref(desc), batch, seq_len, _p(read_slot), _p(k_cache),
                                   _p(v_cache), num_slots, _p(k_out), _p(v_out), _p(dev_status),
                                   _stream(stream))
    return _check("acache_gather_slots", st) if check else st


def acache_kv_deviation_scores(desc, batch, affix_len, k_shared, v_shared, k_full, v_full, scores,
                               stream=None, check=True):
    """High-KV-deviation (CacheBlend-style) scores of one layer, accumulated into `scores`."""
    st = lib().acache_kv_deviation_scores(ctypes.byref(desc), batch, affix_len, _p(k_shared),
                                          _p(v_shared), _p(k_full), _p(v_full), _p(scores),
                                          _stream(stream))
    return _check("acache_kv_deviation_scores", st) if check else st


def acache_slot_attention_dropna(desc, batch, n_q, q, seq_len, read_slot, k_cache, v_cache,
                                 num_slots, out, dev_status=None, stream=None, check=True):
    """Read-slot attention where read_slot entries equal to SLOT_NONE are discarded keys."""
    st = lib().acache_slot_attention_dropna(ctypes.byref(desc), batch, n_q, _p(q), seq_len,
                                            _p(read_slot), _p(k_cache), _p(v_cache), num_slots,
                                            _p(out), _p(dev_status), _stream(stream))
    return _check("acache_slot_attention_dropna", st) if check else st


def acache_slot_attention_path(desc, batch, n_q, seq_len) -> int:
    """The kernel acache_slot_attention runs for this geometry: ACACHE_PATH_RECOMPUTE,
    ACACHE_PATH_RECOMPUTE_PERSISTENT, ACACHE_PATH_BLOCK_DECODE or ACACHE_PATH_CUDA_CORES (see
    include/acache.h)."""
    st = int(lib().acache_slot_attention_path(ctypes.byref(desc), batch, n_q, seq_len))
    return _check("acache_slot_attention_path", st) if st < 0 else st


def acache_slot_attention_varlen(desc, batch, q_start, max_q_rows, total_q_rows, q, kv_start,
                                 max_seq_len, read_slot, k_cache, v_cache, num_slots, out,
                                 drop_none=False, dev_status=None, stream=None, check=True):
    """Read-slot attention over a ragged batch: q_start / kv_start are [B+1] int32 device
    offsets into the flattened query rows and read-slot entries."""
    st = lib().acache_slot_attention_varlen(ctypes.byref(desc), batch, _p(q_start), max_q_rows,
                                            total_q_rows, _p(q), _p(kv_start), max_seq_len,
                                            _p(read_slot), _p(k_cache), _p(v_cache), num_slots, _p(out),
                                            int(bool(drop_none)), _p(dev_status), _stream(stream))
    return _check("acache_slot_attention_varlen", st) if check else st


def _ptr_array(ts, n):
    """Host array of n device pointers (None when ts is None; a None entry is a null pointer)."""
    if ts is None:
        return None
    if len(ts) != n:
        raise ValueError(f"expected {n} per-layer tensors, got {len(ts)}")
    arr = (ctypes.c_void_p * n)(*[None if t is None else t.data_ptr() for t in ts])
    return ctypes.cast(arr, ctypes.c_void_p), arr


def acache_store_attend_layers(desc, batch, rows, write_slot, k_new, v_new, k_cache, v_cache, num_slots,
                               private_begin, n_q, q, seq_len, read_slot, out, dev_status=None, stream=None,
                               check=True):
    """Store-then-attend for every layer of a recompute point in one call (see include/acache.h);
    the per-layer arguments are lists of tensors, one per layer."""
    layers = len(k_cache)
    keep = [_ptr_array(x, layers) for x in (k_new, v_new, k_cache, v_cache, q, out)]
    ptrs = [k[0] if k is not None else None for k in keep]
    st = lib().acache_store_attend_layers(ctypes.byref(desc), layers, batch, rows, _p(write_slot), ptrs[0],
                                          ptrs[1], ptrs[2], ptrs[3], num_slots, private_begin, n_q, ptrs[4],
                                          seq_len, _p(read_slot), ptrs[5], _p(dev_status), _stream(stream))
    del keep
    return _check("acache_store_attend_layers", st) if check else st


def acache_store_attend(desc, batch, rows, write_slot, k_new, v_new, k_cache, v_cache, num_slots,
                        private_begin, n_q, q, seq_len, read_slot, out, dev_status=None, stream=None,
                        check=True):
    """Store step then read-slot attention of one layer in one call (see include/acache.h)."""
    st = lib().acache_store_attend(ctypes.byref(desc), batch, rows, _p(write_slot), _p(k_new), _p(v_new),
                                   _p(k_cache), _p(v_cache), num_slots, private_begin, n_q, _p(q),
                                   seq_len, _p(read_slot), _p(out), _p(dev_status), _stream(stream))
    return _check("acache_store_attend", st) if check else st


def acache_rerotate_keys(desc, rows, k_in, k_out, delta_pos, rope_theta, interleaved=False, stream=None,
                         check=True):
    """Move rotary-embedded keys [rows][Hkv][d] by delta_pos positions (see include/acache.h)."""
    st = lib().acache_rerotate_keys(ctypes.byref(desc), rows, _p(k_in), _p(k_out), int(delta_pos),
                                    float(rope_theta), int(bool(interleaved)), _stream(stream))
    return _check("acache_rerotate_keys", st) if check else st


# ---- the 8-bit KV pool (see include/acache.h): k_cache / v_cache [num_slots][Hkv][d] e4m3 codes
# (torch.float8_e4m3fn or uint8), kv_scale [num_slots][Hkv][2] uint8 exponents
def acache_write_slots_q8(desc, batch, rows, write_slot, k_new, v_new, k_cache, v_cache, kv_scale, num_slots,
                          private_begin, dev_status=None, stream=None, check=True):
    """The store step into an 8-bit pool: quantises as it writes."""
    dev = _current_device()
    st = lib().acache_write_slots_q8(ctypes.byref(desc), batch, rows, _on(dev, write_slot), _on(dev, k_new),
                                     _on(dev, v_new), _on(dev, k_cache), _on(dev, v_cache), _on(dev, kv_scale),
                                     num_slots, private_begin, _on(dev, dev_status), _stream(stream))
    return _check("acache_write_slots_q8", st) if check else st


def acache_gather_slots_q8(desc, batch, seq_len, read_slot, k_cache, v_cache, kv_scale, num_slots, k_out, v_out,
                           dev_status=None, stream=None, check=True):
    """The logical K/V view of an 8-bit pool, in the descriptor's dtype."""
    dev = _current_device()
    st = lib().acache_gather_slots_q8(ctypes.byref(desc), batch, seq_len, _on(dev, read_slot), _on(dev, k_cache),
                                      _on(dev, v_cache), _on(dev, kv_scale), num_slots, _on(dev, k_out),
                                      _on(dev, v_out), _on(dev, dev_status), _stream(stream))
    return _check("acache_gather_slots_q8", st) if check else st


def acache_slot_attention_q8(desc, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, kv_scale, num_slots, out,
                             drop_none=False, dev_status=None, stream=None, check=True):
    """Read-slot attention over an 8-bit pool; with drop_none, SLOT_NONE entries are discarded keys."""
    dev = _current_device()
    st = lib().acache_slot_attention_q8(ctypes.byref(desc), batch, n_q, _on(dev, q), seq_len, _on(dev, read_slot),
                                        _on(dev, k_cache), _on(dev, v_cache), _on(dev, kv_scale), num_slots,
                                        _on(dev, out), int(bool(drop_none)), _on(dev, dev_status), _stream(stream))
    return _check("acache_slot_attention_q8", st) if check else st


def acache_slot_attention_varlen_q8(desc, batch, q_start, max_q_rows, total_q_rows, q, kv_start, max_seq_len,
                                    read_slot, k_cache, v_cache, kv_scale, num_slots, out, drop_none=False,
                                    dev_status=None, stream=None, check=True):
    """Read-slot attention over a ragged batch and an 8-bit pool (offsets as in
    acache_slot_attention_varlen)."""
    dev = _current_device()
    st = lib().acache_slot_attention_varlen_q8(ctypes.byref(desc), batch, _on(dev, q_start), max_q_rows,
                                               total_q_rows, _on(dev, q), _on(dev, kv_start), max_seq_len,
                                               _on(dev, read_slot), _on(dev, k_cache), _on(dev, v_cache),
                                               _on(dev, kv_scale), num_slots, _on(dev, out), int(bool(drop_none)),
                                               _on(dev, dev_status), _stream(stream))
    return _check("acache_slot_attention_varlen_q8", st) if check else st


def acache_store_attend_q8(desc, batch, rows, write_slot, k_new, v_new, k_cache, v_cache, kv_scale, num_slots,
                           private_begin, n_q, q, seq_len, read_slot, out, drop_none=False, dev_status=None,
                           stream=None, check=True):
    """Store step into an 8-bit pool, then read-slot attention over it, in one call."""
    dev = _current_device()
    st = lib().acache_store_attend_q8(ctypes.byref(desc), batch, rows, _on(dev, write_slot), _on(dev, k_new),
                                      _on(dev, v_new), _on(dev, k_cache), _on(dev, v_cache), _on(dev, kv_scale),
                                      num_slots, private_begin, n_q, _on(dev, q), seq_len, _on(dev, read_slot),
                                      _on(dev, out), int(bool(drop_none)), _on(dev, dev_status), _stream(stream))
    return _check("acache_store_attend_q8", st) if check else st


# ---- the steps around the attention, and attention under a mask (see include/acache.h)
_SCALINGS = {"none": ROPE_NONE, "linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN, "bands": ROPE_BANDS}


def rope_desc(rotary_dim, theta=10000.0, interleaved=False, scaling="none", factor=1.0, trained_len=0, turns_low=0.0,
              turns_high=0.0, amplitude=None) -> Rope:
    """The rotation of a head's first rotary_dim elements, to be kept and passed to the calls below."""
    r = Rope()
    _check("acache_rope_init", lib().acache_rope_init(
        ctypes.byref(r), rotary_dim, int(bool(interleaved)), float(theta), _SCALINGS.get(scaling, scaling), float(factor),
        int(trained_len), float(turns_low), float(turns_high)))
    if amplitude is not None:
        r.amplitude = amplitude
    return r


def rope_desc_frequencies(frequencies, interleaved=False, amplitude=1.0) -> Rope:
    """The same from a sequence of angles per position, one per pair."""
    f = [float(x) for x in frequencies]
    r = Rope()
    _check("acache_rope_init_frequencies", lib().acache_rope_init_frequencies(
        ctypes.byref(r), 2 * len(f), int(bool(interleaved)), (ctypes.c_double * max(len(f), 1))(*f), float(amplitude)))
    return r


def _step_of(shape, stride):
    """Elements from one row to the next, where `shape` and `stride` are of the dimensions that number the rows (None: one)."""
    step, rows = None, 1
    for size, at in zip(reversed(shape), reversed(stride)):
        if size != 1:
            if step is None:
                step = at
            elif at != step * rows:
                raise ValueError("the rows have to be evenly spaced")
            rows *= size
    return step


def _row_stride(t, heads, d, rows=None):
    """Elements from one row [heads][d] of a tensor [..., heads or more, d] to the next; rows must be evenly spaced.
    A dense tensor of another shape holds its rows one after the other."""
    if t is None:
        return heads * d
    try:
        if t.is_contiguous() and (rows is None or t.numel() == rows * heads * d):
            return heads * d
        shape, stride = t.shape, t.stride()
    except AttributeError:       # a plain address
        return heads * d
    n = len(shape)
    if n == 4:                               # slices of a batch of fused rows
        a, b, h, w = shape
        sa, sb, sh, sw = stride
        if w == d and h >= heads and sw == 1 and sh == d and b > 1 and sa == sb * b and (rows is None or a * b >= rows):
            return sb
    if n > 1 and shape[-1] == d and shape[-2] >= heads:
        if stride[-1] != 1 or (stride[-2] != d and heads > 1):
            raise ValueError("the heads of a row have to follow one another")
        step = _step_of(shape[:-2], stride[:-2])
        if rows is None or math.prod(shape[:-2]) >= rows:
            return heads * d if step is None else step
    if rows is None or not t.is_contiguous() or t.numel() < rows * heads * d or (n > 1 and shape[-1] not in (d, heads * d)):
        raise ValueError(f"rows have to be [..., {heads}, {d}]" + ("" if rows is None else f", {rows} of them"))
    return heads * d


def acache_rotate_qk(desc, rope, rows, positions, q, k, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6,
                     stream=None, check=True):
    """Norm (with a weight) and rotary position of query and key rows [..., heads, d], which may be slices
    of a wider row (of rows with more heads the first are taken); rope=None rotates nothing, q or k None is left out."""
    dev = _current_device()
    hq, hkv, d = desc.num_q_heads, desc.num_kv_heads, desc.head_dim
    st = lib().acache_rotate_qk(
        desc, rope, rows, _dense(dev, positions), _on(dev, q),
        _row_stride(q, hq, d, rows), _on(dev, k), _row_stride(k, hkv, d, rows), _dense(dev, q_weight), _dense(dev, k_weight), eps,
        _on(dev, q_out), _row_stride(q_out, hq, d, rows), _on(dev, k_out), _row_stride(k_out, hkv, d, rows), _stream(stream, dev))
    return _check("acache_rotate_qk", st) if check else st


def _new_rows(dev, desc, rope, batch, rows, positions, write_slot, q, k, v, q_weight, k_weight, eps, q_out, k_cache,
              v_cache):
    hq, hkv, d, n = desc.num_q_heads, desc.num_kv_heads, desc.head_dim, batch * rows
    if q is not None and n > 1 and _row_stride(q_out, hq, d, n) != hq * d:
        raise ValueError("the rows of q_out have to follow one another")
    return (desc, rope, batch, rows, _dense(dev, positions),
            _dense(dev, write_slot), _on(dev, q), _row_stride(q, hq, d, n), _on(dev, k), _row_stride(k, hkv, d, n), _on(dev, v),
            _row_stride(v, hkv, d, n), _dense(dev, q_weight), _dense(dev, k_weight), eps, _on(dev, q_out), _dense(dev, k_cache),
            _dense(dev, v_cache))


def acache_rotate_store(desc, rope, batch, rows, positions, write_slot, q, k, v, q_out, k_cache, v_cache, num_slots,
                        private_begin, q_weight=None, k_weight=None, eps=1e-6, dev_status=None, stream=None,
                        check=True):
    """acache_rotate_qk with the rotated keys and the values stored to their slots."""
    dev = _current_device()
    st = lib().acache_rotate_store(*_new_rows(dev, desc, rope, batch, rows, positions, write_slot, q, k, v, q_weight,
                                              k_weight, eps, q_out, k_cache, v_cache),
                                   num_slots, private_begin, _on(dev, dev_status), _stream(stream, dev))
    return _check("acache_rotate_store", st) if check else st


def acache_rotate_store_q8(desc, rope, batch, rows, positions, write_slot, q, k, v, q_out, k_cache, v_cache, kv_scale,
                           num_slots, private_begin, q_weight=None, k_weight=None, eps=1e-6, dev_status=None,
                           stream=None, check=True):
    """The same into an 8-bit pool."""
    dev = _current_device()
    st = lib().acache_rotate_store_q8(*_new_rows(dev, desc, rope, batch, rows, positions, write_slot, q, k, v, q_weight,
                                                 k_weight, eps, q_out, k_cache, v_cache),
                                      _dense(dev, kv_scale), num_slots, private_begin, _on(dev, dev_status),
                                      _stream(stream, dev))
    return _check("acache_rotate_store_q8", st) if check else st


def acache_slot_attention_masked(desc, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, num_slots, out,
                                 row_range=None, q_pos=None, slopes=None, softcap=0.0, drop_none=False,
                                 dev_status=None, stream=None, check=True):
    """Read-slot attention whose rows see a range of keys (row_range [B, n_q, 2]), with capped scores and a
    bias of -slopes[h] * |q_pos - t|."""
    dev = _current_device()
    mask = Mask(_dense(dev, row_range), _dense(dev, q_pos), _dense(dev, slopes), softcap, int(bool(drop_none)))
    st = lib().acache_slot_attention_masked(desc, mask, batch, n_q, _dense(dev, q), seq_len,
                                            _dense(dev, read_slot), _dense(dev, k_cache), _dense(dev, v_cache), num_slots,
                                            _dense(dev, out), _on(dev, dev_status), _stream(stream, dev))
    return _check("acache_slot_attention_masked", st) if check else st


def acache_slot_attention_masked_varlen(desc, batch, q_start, max_q_rows, total_q_rows, q, kv_start, max_seq_len,
                                        read_slot, k_cache, v_cache, num_slots, out, row_range=None, q_pos=None,
                                        slopes=None, softcap=0.0, drop_none=False, dev_status=None, stream=None,
                                        check=True):
    """The same over a ragged batch (offsets as in acache_slot_attention_varlen)."""
    dev = _current_device()
    mask = Mask(_dense(dev, row_range), _dense(dev, q_pos), _dense(dev, slopes), softcap, int(bool(drop_none)))
    st = lib().acache_slot_attention_masked_varlen(
        desc, mask, batch, _dense(dev, q_start), max_q_rows, total_q_rows, _dense(dev, q),
        _dense(dev, kv_start), max_seq_len, _dense(dev, read_slot), _dense(dev, k_cache), _dense(dev, v_cache), num_slots,
        _dense(dev, out), _on(dev, dev_status), _stream(stream, dev))
    return _check("acache_slot_attention_masked_varlen", st) if check else st


def _logit_stride(logits, rows, vocab):
    """Elements from one row to the next of logits of any shape [..., at least vocab]."""
    if logits.is_contiguous() and (logits.numel() == rows * vocab or (logits.dim() == 1 and logits.numel() > rows * vocab)):
        return vocab                         # rows that follow one another, however they are shaped
    if logits.shape[-1] < vocab or logits.numel() < rows * logits.shape[-1]:
        raise ValueError("logits of fewer rows or tokens than are to be scored")
    step = _step_of(logits.shape[:-1], logits.stride()[:-1])
    return vocab if step is None else step


def acache_token_scores(rows, vocab, logits, tokens=None, token_logprob=None, entropy=None, top_tokens=None,
                        top_logprob=None, temperature=1.0, k=None, dev_status=None, stream=None, check=True):
    """Log probabilities of given tokens, entropy and the likeliest tokens (k = the last dimension of top_tokens)
    of logits [rows, vocab] in bf16 or float32, whose rows may lie apart."""
    dtype = {torch.float32: ACACHE_F32, torch.bfloat16: ACACHE_BF16}.get(logits.dtype, -1)
    shape, step = logits.shape, logits.stride()
    if not shape or (vocab > 1 and step[-1] != 1):
        raise ValueError("the logits of a row have to follow one another")
    dev = _current_device()
    if len(shape) == 2 and shape[0] >= rows and shape[1] >= vocab:
        stride = step[0] if shape[0] > 1 else vocab
    else:
        stride = _logit_stride(logits, rows, vocab)
    if k is None:
        k = 0 if top_tokens is None else top_tokens.shape[-1]
    for t in (top_tokens, top_logprob):
        if t is not None and k > 0 and rows > 1 and hasattr(t, "shape") and t.shape[-1] != k and t.dim() > 1:
            raise ValueError(f"alternatives are [rows, {k}]")
    st = lib().acache_token_scores(dtype, rows, vocab, _on(dev, logits), stride, temperature, _dense(dev, tokens),
                                   _dense(dev, token_logprob), _dense(dev, entropy), k, _dense(dev, top_tokens),
                                   _dense(dev, top_logprob), _on(dev, dev_status), _stream(stream, dev))
    return _check("acache_token_scores", st) if check else st


class Pool:
    """Host-side admission runtime of one KV slot layout (include/acache.h, acache_pool_*):
    the shared-affix registry and the private-page allocator.  Marshalling only."""

    def __init__(self, num_slots, private_begin, page_slots):
        h = ctypes.c_void_p()
        _check("acache_pool_create", lib().acache_pool_create(num_slots, private_begin, page_slots,
                                                              ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            lib().acache_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def register_affix(self, key, affix_len):
        """Returns (shared_base, created)."""
        base, created = ctypes.c_int32(), ctypes.c_int32()
        _check("acache_pool_register_affix", lib().acache_pool_register_affix(
            self._h, ctypes.c_uint64(key & (2 ** 64 - 1)), affix_len, ctypes.byref(base), ctypes.byref(created)))
        return base.value, bool(created.value)

    def release_affix(self, key):
        _check("acache_pool_release_affix", lib().acache_pool_release_affix(self._h, ctypes.c_uint64(key & (2 ** 64 - 1))))

    def alloc_private(self, rows):
        """Returns (slots as a CPU int32 tensor [rows], request_id)."""
        slots = torch.empty(rows, dtype=torch.int32)
        rid = ctypes.c_int64()
        _check("acache_pool_alloc_private", lib().acache_pool_alloc_private(
            self._h, rows, ctypes.c_void_p(slots.data_ptr()) if rows else None, ctypes.byref(rid)))
        return slots, rid.value

    def free_private(self, request_id):
        _check("acache_pool_free_private", lib().acache_pool_free_private(self._h, request_id))

    def stats(self):
        fs, fp, na, nr = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check("acache_pool_stats", lib().acache_pool_stats(self._h, ctypes.byref(fs), ctypes.byref(fp),
                                                            ctypes.byref(na), ctypes.byref(nr)))
        return {"free_shared": fs.value, "free_private": fp.value, "affixes": na.value, "requests": nr.value}
