"""Thin Python binding of libpagedkv, the GB300 paged KV-cache decode library.

Argument marshalling only: every step of the decode path (slot mapping,
append, attention, split merge) runs in the native library declared in
``include/paged_kv.h``.  Importing this package without the built library
raises ``ImportError``; there is no fallback.

Typical decode step for one layer::

    alloc = BlockAllocator(num_blocks, kv_heads, head_dim)
    slots, tables, lens, cow = alloc.step(seq_ids, max_blocks)      # host
    kv_copy_blocks(k_cache, v_cache, cow_src, cow_dst)              # if any copy-on-write
    kv_append(k_new, v_new, k_cache, v_cache, slots_dev)            # GPU
    paged_decode_attention(out, q, k_cache, v_cache, tables_dev, lens_dev, scale, ws)  # GPU
"""
import ctypes
import os

import numpy as np

from .build import LIB as _LIB_PATH

KV_OK = 0
KV_ERR_INVALID_ARG = -1
KV_ERR_OUT_OF_BLOCKS = -2
KV_ERR_UNSUPPORTED = -3
KV_ERR_CUDA = -4
KV_ERR_NOT_FOUND = -5
KV_ERR_EXISTS = -6
KV_ERR_TOO_LARGE = -7
KV_ERR_OUT_OF_MEMORY = -8
NOALLOC_WORKSPACE_BYTES = 16 << 20

BF16 = 0
FP8_E4M3 = 1
F32 = 2
BLOCK_SIZE = 16

DEVERR_SLOT_OUT_OF_RANGE = 1
DEVERR_BLOCK_OUT_OF_RANGE = 2
DEVERR_CONTEXT_TOO_LONG = 4
DEVERR_PIPELINE_TIMEOUT = 8
DEVERR_BAD_PREFIX = 16
DEVERR_BAD_TREE = 32

TREE_MAX_NODES = 128        # KV_TREE_MAX_NODES
TREE_PAD = -2               # KV_TREE_PAD, the parent of a padding node

# columns of a kv_alloc_trace row (KV_TRACE_*)
TRACE_KEYS = ("seq_id", "slot", "len", "position", "blocks", "shared_blocks", "cache_bytes",
              "reorder_src")
TRACE_FIELDS = len(TRACE_KEYS)

_ERRNAMES = {KV_ERR_INVALID_ARG: "KV_ERR_INVALID_ARG", KV_ERR_OUT_OF_BLOCKS: "KV_ERR_OUT_OF_BLOCKS",
             KV_ERR_UNSUPPORTED: "KV_ERR_UNSUPPORTED", KV_ERR_CUDA: "KV_ERR_CUDA",
             KV_ERR_NOT_FOUND: "KV_ERR_NOT_FOUND", KV_ERR_EXISTS: "KV_ERR_EXISTS",
             KV_ERR_TOO_LARGE: "KV_ERR_TOO_LARGE", KV_ERR_OUT_OF_MEMORY: "KV_ERR_OUT_OF_MEMORY"}


class KVError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s failed: %s (%d)" % (what, _ERRNAMES.get(code, "?"), code))
        self.code = code


if not os.path.exists(_LIB_PATH):
    raise ImportError("libpagedkv.so is not built (expected at %s); run "
                      "`python -c 'import __graft_entry__ as g; g.build()'`" % _LIB_PATH)

_lib = ctypes.CDLL(_LIB_PATH)
_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_f = ctypes.c_float

# exported entry points with their C signatures (include/paged_kv.h)
_SIGS = {
    "kv_bytes": (_i64, [_i, _i, _i, _i64, _i, _i]),
    "kv_cache_alloc": (_i, [ctypes.POINTER(_p), _i, _i, _i, _i, _i]),
    "kv_alloc_destroy": (None, [_p]),
    "kv_seq_add": (_i, [_p, _i64, _i64]),
    "kv_seq_fork": (_i, [_p, _i64, _i64, _i64]),
    "kv_seq_free": (_i, [_p, _i64]),
    "kv_step": (_i, [_p, _p, _i, _p, _p, _i, _p, _p, _p, _i, ctypes.POINTER(_i)]),
    "kv_seq_reorder": (_i, [_p, _p, _p, _i]),
    "kv_seq_info": (_i, [_p, _i64, ctypes.POINTER(_i64), _p, _i, ctypes.POINTER(_i)]),
    "kv_alloc_stats": (_i, [_p, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i), _i,
                            ctypes.POINTER(_i)]),
    "kv_alloc_shape": (_i, [_p, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i),
                            ctypes.POINTER(_i)]),
    "kv_alloc_trace": (_i, [_p, _p, _i, _p, ctypes.POINTER(_i)]),
    "kv_slot_mapping": (_i, [_p, _i, _p, _i, _p]),
    "kv_append": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _f, _f, _p]),
    "kv_copy_blocks": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _p]),
    "paged_decode_workspace_bytes": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]),
    "paged_decode_attention": (_i, [_p, _i, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i, _i, _i,
                                    _i, _f, _p, ctypes.c_size_t, _p]),
    "paged_decode_attention_timed": (_i, [_p, _i, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i,
                                          _i, _i, _i, _f, _p, ctypes.c_size_t, _p, _p, _p, _p]),
    "paged_decode_step": (_i, [_p, _i, _p, _p, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i, _i,
                               _i, _i, _f, _p, ctypes.c_size_t, _p]),
    "paged_decode_attention_noalloc": (_i, [_p, _i, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i,
                                            _i, _i, _i, _f, _p]),
    "kv_prefix_chunks": (_i, [_p, _i, _p, _i, _i, _i, _p, _p, ctypes.POINTER(_i)]),
    "kv_prefix_plan": (_i, [_p, _i, _p, _i, _i, _i, _i, _i, _i, _p, _p, ctypes.POINTER(_i)]),
    "paged_decode_prefix_workspace_bytes": (_i, [_i, _i, _i, _i, _i, _i,
                                                 ctypes.POINTER(ctypes.c_size_t)]),
    "paged_decode": (_i, [_p, _i, _p, _p, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i, _i, _i,
                          _i, _f, _p, _p, _i, ctypes.c_uint, _p, ctypes.c_size_t, _p]),
    "paged_decode_timed": (_i, [_p, _i, _p, _p, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _i, _i,
                                _i, _i, _f, _p, _p, _i, ctypes.c_uint, _p, ctypes.c_size_t, _p,
                                _p, _p, _p]),
    "kv_tree_step": (_i, [_p, _p, _p, _i, _p, _p, _i, _p, _p, _p, _p, _i, ctypes.POINTER(_i)]),
    "kv_seq_truncate": (_i, [_p, _p, _p, _i]),
    "paged_tree_workspace_bytes": (_i, [_i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]),
    "paged_tree_attention": (_i, [_p, _i, _p, _p, _p, _i, _f, _f, _i, _p, _i, _p, _p, _p, _i, _i,
                                  _i, _i, _i, _i, _f, _p, ctypes.c_size_t, _p]),
    "kv_tree_verify": (_i, [_p, _p, _p, _p, _i64, _p, _i64, _i, _p, _p, _p, _p, _p, _i, _i, _i,
                            _i, ctypes.c_uint, _p]),
    "kv_tree_compact": (_i, [_p, _p, _i, _p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p]),
    "kv_latent_bytes": (_i64, [_i, _i, _i64, _i, _i]),
    "kv_rotary_frequencies": (_i, [_p, _p, _i, ctypes.c_double, _i, ctypes.c_double,
                                   ctypes.c_double, ctypes.c_double, ctypes.c_double]),
    "kv_append_rotary": (_i, [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _i,
                              ctypes.c_uint, _f, _i, _i, _i, _i, _i, _i, _f, _f, _p]),
    "kv_latent_append": (_i, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _p, _i64, _p, _f, _p, _p,
                              _p, _p, ctypes.c_uint, _f, _i, _i, _i, _i, _i, _p]),
    "paged_latent_workspace_bytes": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]),
    "paged_latent_attention": (_i, [_p, _p, _p, _i, _p, _i, _p, _p, _p, _i, _i, _i, _i, _i, _i,
                                    _f, _p, ctypes.c_size_t, _p]),
    "kv_read_ceiling": (_i, [_p, ctypes.c_size_t, _p, _p]),
    "kv_test_pipeline_stall": (_i, [ctypes.c_longlong]),
    "kv_get_device_error": (_i, [ctypes.POINTER(_i), ctypes.POINTER(_i64)]),
    "kv_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

# The per-step calls go through the CPython-API module _pkvfast when it was
# built (plain integers and floats, no ctypes marshalling); it links the same
# libpagedkv.so, which the dynamic loader shares with the ctypes handle above.
try:
    from . import _pkvfast as _fast
except ImportError:
    _fast = None


def _hot(name):
    return getattr(_fast, name) if _fast is not None else getattr(_lib, name)


_HOT_PAGED_DECODE = _hot("paged_decode")
_HOT_PAGED_DECODE_STEP = _hot("paged_decode_step")
_HOT_PAGED_DECODE_ATTENTION = _hot("paged_decode_attention")
_HOT_KV_APPEND = _hot("kv_append")
_HOT_TREE_ATTENTION = _hot("paged_tree_attention")
_HOT_TREE_VERIFY = _hot("kv_tree_verify")
_HOT_TREE_COMPACT = _hot("kv_tree_compact")
_HOT_APPEND_ROTARY = _hot("kv_append_rotary")
_HOT_LATENT_APPEND = _hot("kv_latent_append")
_HOT_LATENT_ATTENTION = _hot("paged_latent_attention")


def fast_path():
    """True when the per-step calls bypass ctypes (module _pkvfast)."""
    return _fast is not None


def native_library_path():
    return _LIB_PATH


def version():
    return _lib.kv_version().decode()


def _check(rc, what):
    if rc != KV_OK:
        raise KVError(rc, what)


def _np_ptr(a):
    return ctypes.c_void_p(a.ctypes.data)


def _dptr(t):
    """Device (or host) address of a torch tensor."""
    return ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _stream_int(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _cache_dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        return FP8_E4M3
    raise ValueError("cache tensors must be bfloat16 or uint8 (E4M3 codes)")


def _cache_shape(cache, latent):
    """(blocks, KV heads, head dim) of a cache; a latent one ([NB, 16, W]) has one head."""
    if latent:
        NB, block, W = cache.shape
        if block != BLOCK_SIZE:
            raise ValueError("a latent cache must be [NB, 16, W]")
        return NB, 1, W
    NB, Hkv, _, D = cache.shape
    return NB, Hkv, D


# ------------------------------------------------------------------ sizing

def kv_bytes(layers, batch, kv_heads, seq, head_dim, dtype_bytes):
    """2 x layers x batch x kv_heads x seq x head_dim x dtype_bytes (int)."""
    r = _lib.kv_bytes(layers, batch, kv_heads, seq, head_dim, dtype_bytes)
    if r < 0:
        raise ValueError("kv_bytes: negative argument or overflow")
    return r


def latent_bytes(layers, batch, seq, width, dtype_bytes=2):
    """layers x batch x seq x width x dtype_bytes: latent caches of rows of `width`
    (latent_dim + rope_dim) elements (int)."""
    r = _lib.kv_latent_bytes(layers, batch, seq, width, dtype_bytes)
    if r < 0:
        raise ValueError("kv_latent_bytes: negative argument or overflow")
    return r


def slot_mapping(block_tables, positions):
    """Host slot of positions[i] in block-table row i (numpy int32 [n, max_blocks])."""
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    pos = np.ascontiguousarray(positions, dtype=np.int64)
    n = pos.shape[0]
    assert bt.shape[0] == n
    out = np.empty(n, dtype=np.int64)
    _check(_lib.kv_slot_mapping(_np_ptr(bt), bt.shape[1], _np_ptr(pos), n, _np_ptr(out)),
           "kv_slot_mapping")
    return out


# ---------------------------------------------------------------- allocator

class BlockAllocator:
    """Host block pool with free list, reference counts and copy-on-write."""

    def __init__(self, num_blocks, num_kv_heads, head_dim, kv_dtype=BF16):
        h = ctypes.c_void_p()
        _check(_lib.kv_cache_alloc(ctypes.byref(h), num_blocks, num_kv_heads, head_dim,
                                   BLOCK_SIZE, kv_dtype), "kv_cache_alloc")
        self._h = h
        self.num_blocks = num_blocks

    def close(self):
        if self._h:
            _lib.kv_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add(self, seq_id, length):
        _check(_lib.kv_seq_add(self._h, seq_id, length), "kv_seq_add")

    def fork(self, parent, child, shared_len):
        _check(_lib.kv_seq_fork(self._h, parent, child, shared_len), "kv_seq_fork")

    def free(self, seq_id):
        _check(_lib.kv_seq_free(self._h, seq_id), "kv_seq_free")

    def step(self, seq_ids, max_blocks, cow_cap=None):
        """Plan one decode step; returns (slot_mapping int64[n], block_tables
        int32[n, max_blocks], context_lens int32[n], (cow_src, cow_dst))."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        n = ids.shape[0]
        cap = n if cow_cap is None else cow_cap
        slots = np.empty(n, dtype=np.int64)
        bt = np.empty((n, max_blocks), dtype=np.int32)
        lens = np.empty(n, dtype=np.int32)
        src = np.empty(max(cap, 1), dtype=np.int32)
        dst = np.empty(max(cap, 1), dtype=np.int32)
        ncow = _i(0)
        _check(_lib.kv_step(self._h, _np_ptr(ids), n, _np_ptr(slots), _np_ptr(bt), max_blocks,
                            _np_ptr(lens), _np_ptr(src), _np_ptr(dst), cap, ctypes.byref(ncow)),
               "kv_step")
        return slots, bt, lens, (src[:ncow.value].copy(), dst[:ncow.value].copy())

    def tree_step(self, seq_ids, num_nodes, max_blocks, cow_cap=None):
        """Plan one step that appends num_nodes[i] drafted tokens to sequence
        seq_ids[i] (kv_tree_step); returns (slot_mapping int64[sum],
        block_tables int32[n, max_blocks], context_lens int32[n], node_starts
        int32[n + 1], (cow_src, cow_dst))."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        counts = np.ascontiguousarray(num_nodes, dtype=np.int32)
        n = ids.shape[0]
        assert counts.shape == ids.shape
        cap = n if cow_cap is None else cow_cap
        slots = np.empty(max(int(np.maximum(counts, 0).sum(dtype=np.int64)), 1), dtype=np.int64)
        bt = np.empty((n, max_blocks), dtype=np.int32)
        lens = np.empty(n, dtype=np.int32)
        starts = np.empty(n + 1, dtype=np.int32)
        src = np.empty(max(cap, 1), dtype=np.int32)
        dst = np.empty(max(cap, 1), dtype=np.int32)
        ncow = _i(0)
        _check(_lib.kv_tree_step(self._h, _np_ptr(ids), _np_ptr(counts), n, _np_ptr(slots),
                                 _np_ptr(bt), max_blocks, _np_ptr(lens), _np_ptr(starts),
                                 _np_ptr(src), _np_ptr(dst), cap, ctypes.byref(ncow)),
               "kv_tree_step")
        return (slots[:starts[n]], bt, lens, starts,
                (src[:ncow.value].copy(), dst[:ncow.value].copy()))

    def truncate(self, seq_ids, new_lens):
        """Cut sequence seq_ids[i] to new_lens[i] tokens; blocks behind them
        return to the pool (kv_seq_truncate)."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        lens = np.ascontiguousarray(new_lens, dtype=np.int64)
        assert ids.shape == lens.shape
        _check(_lib.kv_seq_truncate(self._h, _np_ptr(ids), _np_ptr(lens), ids.shape[0]),
               "kv_seq_truncate")

    def reorder(self, seq_ids, src_index):
        """Row i of seq_ids takes the KV state row src_index[i] had (beam
        reorder / duplication; block tables only, reference counted)."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        src = np.ascontiguousarray(src_index, dtype=np.int32)
        assert ids.shape == src.shape
        _check(_lib.kv_seq_reorder(self._h, _np_ptr(ids), _np_ptr(src), ids.shape[0]),
               "kv_seq_reorder")

    def info(self, seq_id, max_blocks=None):
        """(length, block ids) of a sequence."""
        ln = _i64(0)
        nb = _i(0)
        _check(_lib.kv_seq_info(self._h, seq_id, ctypes.byref(ln), None, 0, ctypes.byref(nb)),
               "kv_seq_info")
        row = np.empty(max(nb.value, 1), dtype=np.int32)
        _check(_lib.kv_seq_info(self._h, seq_id, None, _np_ptr(row), row.shape[0], None),
               "kv_seq_info")
        return ln.value, row[:nb.value].copy()

    def stats(self, block=-1):
        """(free blocks, used blocks, live sequences, refcount of `block` or None)."""
        fb, ub, ns, rc = _i(0), _i(0), _i(0), _i(0)
        _check(_lib.kv_alloc_stats(self._h, ctypes.byref(fb), ctypes.byref(ub), ctypes.byref(ns),
                                   block, ctypes.byref(rc)), "kv_alloc_stats")
        return fb.value, ub.value, ns.value, (rc.value if block >= 0 else None)

    def shape(self):
        """Per-layer cache shape [num_blocks, num_kv_heads, 16, head_dim] and dtype."""
        nb, h, d, dt = _i(0), _i(0), _i(0), _i(0)
        _check(_lib.kv_alloc_shape(self._h, ctypes.byref(nb), ctypes.byref(h), ctypes.byref(d),
                                   ctypes.byref(dt)), "kv_alloc_shape")
        return (nb.value, h.value, BLOCK_SIZE, d.value), dt.value

    def trace(self, seq_ids=None):
        """Debug trace of the cache state, one dict per sequence (the given
        ids in order, else every live sequence by ascending id): request id,
        batch slot, length, position offset, blocks, shared blocks, cache
        bytes per layer, the last reorder's source row, and the decode mask
        shape [1, length]."""
        if seq_ids is None:
            n = self.stats()[2]
            ids_ptr = None
        else:
            ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
            n = ids.shape[0]
            ids_ptr = _np_ptr(ids)
        rows = np.empty((max(n, 1), TRACE_FIELDS), dtype=np.int64)
        cnt = _i(0)
        _check(_lib.kv_alloc_trace(self._h, ids_ptr, n, _np_ptr(rows), ctypes.byref(cnt)),
               "kv_alloc_trace")
        out = []
        for r in rows[:cnt.value]:
            rec = dict(zip(TRACE_KEYS, (int(x) for x in r)))
            rec["mask_shape"] = [1, rec["len"]]
            out.append(rec)
        return out

    def dump(self, seq_ids=None):
        """The trace as text: a header line with the pool and cache shape,
        then one JSON line per sequence."""
        import json
        shape, dt = self.shape()
        fb, ub, ns, _ = self.stats()
        head = {"kv_shape": list(shape), "kv_dtype": "fp8_e4m3" if dt == FP8_E4M3 else "bf16",
                "free_blocks": fb, "used_blocks": ub, "num_seqs": ns}
        return "\n".join([json.dumps(head)] + [json.dumps(r) for r in self.trace(seq_ids)])


# -------------------------------------------------------------------- GPU ops

def kv_append(k, v, k_cache, v_cache, slot_mapping, k_scale=1.0, v_scale=1.0, stream=None):
    """Append K/V ([T, Hkv, D] bfloat16, device) at slot_mapping (int64 [T],
    device) into the caches ([NB, Hkv, 16, D], bfloat16 or uint8 E4M3)."""
    T, Hkv, D = k.shape
    NB = k_cache.shape[0]
    _check(_HOT_KV_APPEND(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                          slot_mapping.data_ptr(), T, Hkv, D, NB, _cache_dtype(k_cache),
                          float(k_scale), float(v_scale), _stream_int(stream)), "kv_append")


def kv_copy_blocks(k_cache, v_cache, src, dst, stream=None):
    """Copy whole blocks src[i] -> dst[i] (device int32 tensors).  v_cache None:
    k_cache is a latent cache ([NB, 16, W])."""
    NB, Hkv, D = _cache_shape(k_cache, v_cache is None)
    _check(_lib.kv_copy_blocks(_dptr(k_cache), _dptr(v_cache) if v_cache is not None else None,
                               _dptr(src), _dptr(dst),
                               src.shape[0], Hkv, D, NB, _cache_dtype(k_cache),
                               _stream_ptr(stream)), "kv_copy_blocks")


def workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype=BF16):
    n = ctypes.c_size_t(0)
    _check(_lib.paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                             kv_dtype, ctypes.byref(n)),
           "paged_decode_workspace_bytes")
    return n.value


def alloc_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype=BF16, device=None):
    import torch
    nbytes = workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device or "cuda")


def paged_decode_attention(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                           k_scale=1.0, v_scale=1.0, stream=None):
    """out[B, Hq, D] (bfloat16 or float32) = decode attention of q [B, Hq, D]
    (bfloat16) over the paged caches; block_tables int32 [B, max_blocks] and
    context_lens int32 [B] on the device; workspace a uint8 device tensor of
    at least workspace_bytes(...) bytes."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, D2 = k_cache.shape
    assert D == D2
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    _check(_HOT_PAGED_DECODE_ATTENTION(
        out.data_ptr(), out_dtype, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _cache_dtype(k_cache), float(k_scale), float(v_scale), NB, block_tables.data_ptr(),
        block_tables.shape[1], context_lens.data_ptr(), B, Hq, Hkv, D, float(scale),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_int(stream)),
        "paged_decode_attention")


def paged_decode_attention_timed(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                                 workspace, events, k_scale=1.0, v_scale=1.0, stream=None):
    """paged_decode_attention that also records three torch.cuda.Event objects
    (already recorded once, so that their handles exist, or None) before the
    split kernel, after it and after the merge kernel: events = (begin,
    split_end, end)."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, _ = k_cache.shape
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    ev = [ctypes.c_void_p(e._as_parameter_.value) if e is not None else None for e in events]
    _check(_lib.paged_decode_attention_timed(
        _dptr(out), out_dtype, _dptr(q), _dptr(k_cache), _dptr(v_cache), _cache_dtype(k_cache),
        float(k_scale), float(v_scale), NB, _dptr(block_tables), block_tables.shape[1],
        _dptr(context_lens), B, Hq, Hkv, D, float(scale), _dptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream), ev[0], ev[1], ev[2]),
        "paged_decode_attention_timed")


def paged_decode_step(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
                      workspace, k_scale=1.0, v_scale=1.0, stream=None):
    """One decode step in one launch: append k_new/v_new ([B, Hkv, D] bfloat16)
    at position context_lens-1 of each sequence, then attend (see
    paged_decode_attention for the other arguments)."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, _ = k_cache.shape
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    _check(_HOT_PAGED_DECODE_STEP(
        out.data_ptr(), out_dtype, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _cache_dtype(k_cache), float(k_scale),
        float(v_scale), NB, block_tables.data_ptr(), block_tables.shape[1],
        context_lens.data_ptr(), B, Hq, Hkv, D, float(scale), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_int(stream)), "paged_decode_step")


PREFIX_CHUNK_INTS = 18      # KV_PREFIX_CHUNK_INTS
PREFIX_MAX_ROWS = 16        # KV_PREFIX_MAX_ROWS


def prefix_chunks(block_tables, context_lens, group_size, min_blocks=1):
    """Prefix chunks of sequences whose block tables start with the same
    blocks (host numpy int32 arrays in, kv_prefix_chunks): returns
    (chunks int32 [nc, 18], seq_chunk int32 [B])."""
    import numpy as np
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    cl = np.ascontiguousarray(context_lens, dtype=np.int32)
    B, mb = bt.shape
    chunks = np.full((max(B // 2, 1), PREFIX_CHUNK_INTS), -1, dtype=np.int32)
    seq_chunk = np.full(max(B, 1), -1, dtype=np.int32)
    nc = ctypes.c_int(0)
    _check(_lib.kv_prefix_chunks(_np_ptr(bt), mb, _np_ptr(cl), B, int(group_size),
                                 int(min_blocks), _np_ptr(chunks), _np_ptr(seq_chunk),
                                 ctypes.byref(nc)), "kv_prefix_chunks")
    return chunks[:nc.value].copy(), seq_chunk[:B].copy()


def prefix_plan(block_tables, context_lens, num_q_heads, num_kv_heads, head_dim,
                kv_dtype=BF16, resident_warps=0):
    """prefix_chunks with the library's decision whether shared-prefix
    decoding pays for these tables (kv_prefix_plan; resident_warps 0: those
    of the current device): (chunks int32 [nc, 18], seq_chunk int32 [B]),
    nc == 0 for plain decoding."""
    import numpy as np
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    cl = np.ascontiguousarray(context_lens, dtype=np.int32)
    B, mb = bt.shape
    chunks = np.full((max(B // 2, 1), PREFIX_CHUNK_INTS), -1, dtype=np.int32)
    seq_chunk = np.full(max(B, 1), -1, dtype=np.int32)
    nc = ctypes.c_int(0)
    _check(_lib.kv_prefix_plan(_np_ptr(bt), mb, _np_ptr(cl), B, int(num_q_heads),
                               int(num_kv_heads), int(head_dim), int(kv_dtype),
                               int(resident_warps), _np_ptr(chunks),
                               _np_ptr(seq_chunk), ctypes.byref(nc)), "kv_prefix_plan")
    return chunks[:nc.value].copy(), seq_chunk[:B].copy()


def prefix_workspace_bytes(num_seqs, num_chunks, num_q_heads, num_kv_heads, head_dim,
                           kv_dtype=BF16):
    n = ctypes.c_size_t(0)
    _check(_lib.paged_decode_prefix_workspace_bytes(num_seqs, num_chunks, num_q_heads,
                                                    num_kv_heads, head_dim, kv_dtype,
                                                    ctypes.byref(n)),
           "paged_decode_prefix_workspace_bytes")
    return n.value


def alloc_prefix_workspace(num_seqs, num_chunks, num_q_heads, num_kv_heads, head_dim,
                           kv_dtype=BF16, device=None):
    import torch
    nbytes = prefix_workspace_bytes(num_seqs, num_chunks, num_q_heads, num_kv_heads, head_dim,
                                    kv_dtype)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device or "cuda")


DECODE_EARLY_INPUTS = 1     # KV_DECODE_EARLY_INPUTS


def paged_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                 k_scale=1.0, v_scale=1.0, k_new=None, v_new=None, chunks=None, seq_chunk=None,
                 early_inputs=False, stream=None):
    """One decode step, general form (paged_decode): with k_new/v_new
    ([B, Hkv, D] bfloat16) the step's token is appended first (as
    paged_decode_step); with chunks (int32 [nc, 18]) and seq_chunk (int32 [B])
    on the device (from prefix_chunks) shared prefix blocks are read once per
    chunk (workspace from alloc_prefix_workspace); early_inputs lets the
    kernel read the block tables, lengths and caches while the previous
    kernel on the stream drains (see KV_DECODE_EARLY_INPUTS in the header for
    the caller's guarantee).  Other arguments as paged_decode_attention."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, _ = k_cache.shape
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    nc = int(chunks.shape[0]) if chunks is not None else 0
    _check(_HOT_PAGED_DECODE(
        out.data_ptr(), out_dtype, q.data_ptr(), k_new.data_ptr() if k_new is not None else 0,
        v_new.data_ptr() if v_new is not None else 0, k_cache.data_ptr(), v_cache.data_ptr(),
        _cache_dtype(k_cache), float(k_scale), float(v_scale), NB, block_tables.data_ptr(),
        block_tables.shape[1], context_lens.data_ptr(), B, Hq, Hkv, D, float(scale),
        chunks.data_ptr() if nc else 0, seq_chunk.data_ptr() if nc else 0, nc,
        DECODE_EARLY_INPUTS if early_inputs else 0, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_int(stream)), "paged_decode")


def paged_decode_timed(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                       events, k_scale=1.0, v_scale=1.0, k_new=None, v_new=None, chunks=None,
                       seq_chunk=None, early_inputs=False, stream=None):
    """paged_decode that also records three torch.cuda.Event objects (already
    recorded once so that their handles exist, or None) before the split
    kernel, after it and after the merge kernel: events = (begin, split_end,
    end).  A measurement hook."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, _ = k_cache.shape
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    nc = int(chunks.shape[0]) if chunks is not None else 0
    ev = [ctypes.c_void_p(e._as_parameter_.value) if e is not None else None for e in events]
    _check(_lib.paged_decode_timed(
        _dptr(out), out_dtype, _dptr(q), _dptr(k_new) if k_new is not None else None,
        _dptr(v_new) if v_new is not None else None, _dptr(k_cache), _dptr(v_cache),
        _cache_dtype(k_cache), float(k_scale), float(v_scale), NB, _dptr(block_tables),
        block_tables.shape[1], _dptr(context_lens), B, Hq, Hkv, D, float(scale),
        _dptr(chunks) if nc else None, _dptr(seq_chunk) if nc else None, nc,
        DECODE_EARLY_INPUTS if early_inputs else 0, _dptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream), ev[0], ev[1], ev[2]),
        "paged_decode_timed")


# ------------------------------------------------------- trees of drafted tokens

_torch = None               # torch, once one of the functions below has been called


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _place(t):
    """The device index the tensors of a call have to be on: that of `t`, which
    has to be the current device (a call launches there).  Host memory the device
    can address (pinned) will do for all but the caches and the workspace."""
    i = t.get_device()
    if i < 0:
        if not t.is_pinned():
            raise ValueError("tensors must be on the device or in pinned host memory")
        return _torch.cuda.current_device()
    if i != _torch.cuda.current_device():
        raise ValueError("tensor on cuda:%d, current device is cuda:%d"
                         % (i, _torch.cuda.current_device()))
    return i


def _device_only(*tensors):
    """Refuses caches and workspaces in host memory."""
    for t in tensors:
        if t.get_device() < 0:
            raise ValueError("caches and workspace must be device memory (only a step's own "
                             "tensors may be pinned host memory)")


def _ptr(name, t, dtype, n, dev):
    """The address of a contiguous tensor of n elements of `dtype` on device `dev`."""
    if (t.dtype is dtype and t.numel() == n and t.is_contiguous()
            and (t.get_device() == dev or (t.get_device() < 0 and t.is_pinned()))):
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s tensor of %d elements on cuda:%d or in pinned "
                     "host memory" % (name, dtype, n, dev))


def _raw_stream(stream, dev):
    return stream.cuda_stream if stream is not None else _torch._C._cuda_getCurrentRawStream(dev)


def tree_workspace_bytes(num_seqs, max_nodes, num_q_heads, num_kv_heads, head_dim, kv_dtype=BF16):
    n = ctypes.c_size_t(0)
    _check(_lib.paged_tree_workspace_bytes(num_seqs, max_nodes, num_q_heads, num_kv_heads,
                                           head_dim, kv_dtype, ctypes.byref(n)),
           "paged_tree_workspace_bytes")
    return n.value


def alloc_tree_workspace(num_seqs, max_nodes, num_q_heads, num_kv_heads, head_dim, kv_dtype=BF16,
                         device=None):
    import torch
    nbytes = tree_workspace_bytes(num_seqs, max_nodes, num_q_heads, num_kv_heads, head_dim,
                                  kv_dtype)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device or "cuda")


def paged_tree_attention(out, q, k_cache, v_cache, block_tables, context_lens, node_starts,
                         parents, max_nodes, scale, workspace, k_scale=1.0, v_scale=1.0,
                         stream=None):
    """out [T, Hq, D] (bfloat16 or float32) = attention of the T nodes' queries
    q [T, Hq, D] (bfloat16) over the paged caches, each node seeing its
    sequence's committed tokens, its ancestors in the drafted tree and itself
    (paged_tree_attention): node_starts int32 [B + 1], parents int32 [T]
    (None: chains), context_lens int32 [B] including the nodes, at most
    max_nodes nodes a sequence; workspace from alloc_tree_workspace."""
    torch = _torch or _load_torch()
    T, Hq, D = q.shape
    cache = k_cache.shape
    NB, Hkv, block, D2 = cache
    B, max_blocks = block_tables.shape
    f32 = out.dtype is torch.float32
    if (q.dtype is not torch.bfloat16 or not (f32 or out.dtype is torch.bfloat16)
            or out.shape != q.shape or D != D2 or block != BLOCK_SIZE or v_cache.shape != cache
            or k_cache.dtype is not v_cache.dtype):
        raise ValueError("q must be bfloat16 [T, Hq, D], out bfloat16 or float32 of its shape, "
                         "k_cache and v_cache [NB, Hkv, 16, D], alike")
    _device_only(k_cache, v_cache, workspace)
    dev = _place(k_cache)
    i32, n = torch.int32, q.numel()
    _check(_HOT_TREE_ATTENTION(
        _ptr("out", out, out.dtype, n, dev), F32 if f32 else BF16,
        _ptr("q", q, torch.bfloat16, n, dev),
        _ptr("k_cache", k_cache, k_cache.dtype, k_cache.numel(), dev),
        _ptr("v_cache", v_cache, k_cache.dtype, v_cache.numel(), dev),
        BF16 if k_cache.dtype is torch.bfloat16 else _cache_dtype(k_cache),
        float(k_scale), float(v_scale), NB,
        _ptr("block_tables", block_tables, i32, B * max_blocks, dev), max_blocks,
        _ptr("context_lens", context_lens, i32, B, dev),
        _ptr("node_starts", node_starts, i32, B + 1, dev),
        _ptr("parents", parents, i32, T, dev) if parents is not None else 0, B, T,
        int(max_nodes), Hq, Hkv, D, float(scale),
        _ptr("workspace", workspace, workspace.dtype, workspace.numel(), dev),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)),
        "paged_tree_attention")


VERIFY_GREEDY = 1           # KV_VERIFY_GREEDY


def kv_tree_verify(accept_lens, accept_nodes, out_tokens, target_probs, tokens, parents,
                   node_starts, accept_u=None, sample_u=None, draft_probs=None, greedy=False,
                   stream=None):
    """Verify drafted trees against the target's probabilities from given
    uniform numbers (kv_tree_verify).  target_probs [T, V] (and draft_probs,
    or None: the children were chosen, not drawn) float32 or bfloat16 with any
    row stride; tokens, parents (None: chains) int32 [T], node_starts int32
    [B + 1], accept_u float32 [T], sample_u float32 [B].  Writes accept_lens
    int32 [B], accept_nodes and out_tokens int32 [B, max_nodes].  greedy:
    target_probs may be logits; accept_u, sample_u and draft_probs are not
    used."""
    torch = _torch or _load_torch()
    T, V = target_probs.shape
    B, max_nodes = accept_nodes.shape
    dtype, i32, f32 = target_probs.dtype, torch.int32, torch.float32
    if dtype is not f32 and dtype is not torch.bfloat16:
        raise ValueError("target_probs must be float32 or bfloat16")
    draft = None if greedy else draft_probs
    if draft is not None and (draft.dtype is not dtype or draft.shape != target_probs.shape):
        raise ValueError("draft_probs must have target_probs' type and shape")
    if not greedy and (accept_u is None or sample_u is None):
        raise ValueError("accept_u and sample_u are needed")
    # the rows may be apart, their entries not
    t_stride, t_step = target_probs.stride()
    d_stride, d_step = draft.stride() if draft is not None else (0, 1)
    if V > 1 and (t_step != 1 or d_step != 1):
        raise ValueError("the rows of probabilities must be contiguous")
    if T <= 1:
        t_stride, d_stride = max(t_stride, V), max(d_stride, V)
    dev = _place(target_probs)
    if draft is not None and (draft.get_device() != target_probs.get_device()
                              or (draft.get_device() < 0 and not draft.is_pinned())):
        raise ValueError("draft_probs must be where target_probs is")
    _check(_HOT_TREE_VERIFY(
        _ptr("accept_lens", accept_lens, i32, B, dev),
        _ptr("accept_nodes", accept_nodes, i32, B * max_nodes, dev),
        _ptr("out_tokens", out_tokens, i32, B * max_nodes, dev), target_probs.data_ptr(), t_stride,
        draft.data_ptr() if draft is not None else 0, d_stride, F32 if dtype is f32 else BF16,
        _ptr("tokens", tokens, i32, T, dev),
        _ptr("parents", parents, i32, T, dev) if parents is not None else 0,
        _ptr("node_starts", node_starts, i32, B + 1, dev),
        0 if greedy else _ptr("accept_u", accept_u, f32, T, dev),
        0 if greedy else _ptr("sample_u", sample_u, f32, B, dev), B, T, max_nodes, V,
        VERIFY_GREEDY if greedy else 0, _raw_stream(stream, dev)), "kv_tree_verify")


class CacheLayers:
    """The K and V caches of a model's layers, all of one shape, dtype and
    device: what a program keeps to pass to kv_tree_compact.  v_caches None:
    latent caches ([NB, 16, W])."""

    def __init__(self, k_caches, v_caches=None):
        latent = v_caches is None
        if not k_caches or (not latent and len(k_caches) != len(v_caches)):
            raise ValueError("one K and one V cache per layer")
        first, vs = k_caches[0], [] if latent else list(v_caches)
        for t in list(k_caches) + vs:
            if (t.shape != first.shape or t.dtype != first.dtype or t.device != first.device
                    or not t.is_contiguous() or t.dim() != (3 if latent else 4)
                    or t.shape[-2] != BLOCK_SIZE):
                raise ValueError("caches must be contiguous [NB, Hkv, 16, D] (latent caches: "
                                 "[NB, 16, W]), all alike")
        self.tensors = (list(k_caches), vs)                 # keeps the memory alive
        self.num_layers = len(k_caches)
        self.num_blocks, self.num_kv_heads, self.head_dim = _cache_shape(first, latent)
        self.kv_dtype = _cache_dtype(first)
        self.first = first
        self._k = (_p * self.num_layers)(*[t.data_ptr() for t in k_caches])
        self._v = None if latent else (_p * self.num_layers)(*[t.data_ptr() for t in vs])
        self.k_ptrs = ctypes.addressof(self._k)
        self.v_ptrs = 0 if latent else ctypes.addressof(self._v)


def kv_tree_compact(layers, block_tables, context_lens, node_starts, accept_nodes, accept_lens,
                    stream=None):
    """Move the accepted nodes' K and V together in the caches of all layers (a
    CacheLayers), in place (kv_tree_compact): node accept_nodes[s, i] goes to
    position base + i, base = context_lens[s] less the tree's nodes."""
    torch = _torch or _load_torch()
    B, max_nodes = accept_nodes.shape
    max_blocks = block_tables.shape[1]
    _device_only(layers.first)                                  # (the others are like it)
    dev, i32 = _place(layers.first), torch.int32
    _check(_HOT_TREE_COMPACT(
        layers.k_ptrs, layers.v_ptrs, layers.num_layers,
        _ptr("block_tables", block_tables, i32, B * max_blocks, dev), max_blocks,
        _ptr("context_lens", context_lens, i32, B, dev),
        _ptr("node_starts", node_starts, i32, B + 1, dev),
        _ptr("accept_nodes", accept_nodes, i32, B * max_nodes, dev),
        _ptr("accept_lens", accept_lens, i32, B, dev), B, max_nodes, layers.num_kv_heads,
        layers.head_dim, layers.num_blocks, layers.kv_dtype, _raw_stream(stream, dev)),
        "kv_tree_compact")


# ------------------------------------------------ rotary positions, latent caches

ROTARY_INTERLEAVED = 1      # KV_ROTARY_INTERLEAVED
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3, "bands": 4}      # KV_ROTARY_*


def rotary_frequencies(rotary_dim, theta=10000.0, scaling="plain", factor=1.0, low=1.0, high=32.0,
                       original_len=0.0):
    """(inv_freq float32 numpy [rotary_dim / 2], magnitude) of rotary positions,
    scaled for long contexts by `scaling` (kv_rotary_frequencies)."""
    out = np.empty(max(int(rotary_dim), 0) // 2, dtype=np.float32)
    mag = _f(1.0)
    if scaling not in ROTARY_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROTARY_SCALINGS))
    _check(_lib.kv_rotary_frequencies(_np_ptr(out), ctypes.byref(mag), int(rotary_dim),
                                      float(theta), ROTARY_SCALINGS[scaling], float(factor),
                                      float(low), float(high), float(original_len)),
           "kv_rotary_frequencies")
    return out, mag.value


def _rows(name, t, dtype, shape, dev, inner=1):
    """Address of a tensor of `shape` whose last `inner` dimensions are contiguous."""
    if t.dtype is not dtype or tuple(t.shape) != shape or not (
            t.get_device() == dev or (t.get_device() < 0 and t.is_pinned())):
        raise ValueError("%s must be a %s tensor of shape %s on cuda:%d or in pinned host memory"
                         % (name, dtype, shape, dev))
    want = 1
    for n, step in zip(reversed(shape[-inner:]), reversed(t.stride()[-inner:])):
        if n > 1 and step != want:
            raise ValueError("the last %d dimensions of %s must be contiguous" % (inner, name))
        want *= n
    return t.data_ptr()


def _current(t):
    """The device index of a cache, which has to be the current device's memory."""
    i = t.get_device()
    if i < 0 or i != _torch._C._cuda_getDevice():
        _device_only(t)
        _place(t)
    return i


def _heads(name, t, dtype, shape, dev):
    """(address, elements from one token to the next) of a [T, heads, D] tensor, of the shape
    that has been read from it or compared with it, whose tokens may be apart."""
    T, n, D = shape
    token, head, step = t.stride()
    if not (t.dtype is dtype and t.get_device() == dev and step == 1 and (head == D or n == 1)):
        _rows(name, t, dtype, tuple(shape), dev, 2)
    # (of one token, what a tensor of several would have at least)
    return t.data_ptr(), token if T > 1 else n * D


def _vectors(name, t, dtype, shape, dev):
    """(address, elements from one vector to the next) of a [T, n] tensor of vectors, of the
    shape that has been read from it or compared with it, that may be apart."""
    row, step = t.stride()
    if not (t.dtype is dtype and t.get_device() == dev and step == 1):
        _rows(name, t, dtype, tuple(shape), dev)
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _head_vectors(name, t, dtype, shape, dev):
    """(address, strides of tokens and heads) of a [T, H, R] tensor of vectors, of the shape
    that has been read from it or compared with it, that may be apart."""
    T, H, R = shape
    token, head, step = t.stride()
    if not (t.dtype is dtype and t.get_device() == dev and step == 1):
        _rows(name, t, dtype, tuple(shape), dev)
    # (of a single one, what a tensor of several would have at least)
    if H == 1:
        head = R
    return t.data_ptr(), token if T > 1 else (H - 1) * head + R, head


def _tables(slot_mapping, positions, inv_freq, T, n, dev):
    """Addresses of an append's slots, positions and frequencies."""
    i64, f32 = _torch.int64, _torch.float32
    if (slot_mapping.dtype is i64 and positions.dtype is i64 and inv_freq.dtype is f32
            and slot_mapping.numel() == T and positions.numel() == T and inv_freq.numel() == n
            and slot_mapping.get_device() == dev and positions.get_device() == dev
            and inv_freq.get_device() == dev and slot_mapping.is_contiguous()
            and positions.is_contiguous() and inv_freq.is_contiguous()):
        return slot_mapping.data_ptr(), positions.data_ptr(), inv_freq.data_ptr()
    return (_ptr("slot_mapping", slot_mapping, i64, T, dev),
            _ptr("positions", positions, i64, T, dev), _ptr("inv_freq", inv_freq, f32, n, dev))


def kv_append_rotary(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, inv_freq,
                     interleaved=False, magnitude=1.0, k_scale=1.0, v_scale=1.0, stream=None):
    """kv_append with rotary positions on the way (kv_append_rotary): k [T, Hkv, D]
    is turned and appended, v [T, Hkv, D] appended, q [T, Hq, D] turned into q_out
    (which may be q; both None: no queries), all bfloat16, with any distance between
    tokens (slices of one projection's output); slot_mapping and positions int64
    [T]; inv_freq float32 [rotary_dim / 2], the first rotary_dim elements of a head
    being turned."""
    torch = _torch or _load_torch()
    kshape = k.shape
    T, Hkv, D = kshape
    cshape, cdtype, bf16 = k_cache.shape, k_cache.dtype, torch.bfloat16
    NB, H2, block, D2 = cshape
    if (H2 != Hkv or D2 != D or block != BLOCK_SIZE or v.shape != kshape
            or v_cache.shape != cshape or v_cache.dtype is not cdtype
            or (q is None) != (q_out is None)):
        raise ValueError("k and v must be [T, Hkv, D], k_cache and v_cache [NB, Hkv, 16, D], alike")
    dev = _current(k_cache)
    if v_cache.get_device() != dev:
        _device_only(v_cache)
    Hq = po = so = pq = sq = 0
    if q is not None:
        qshape = q.shape
        Hq = qshape[1]
        if len(qshape) != 3 or qshape[0] != T or qshape[2] != D or q_out.shape != qshape:
            raise ValueError("q and q_out must be [T, Hq, D]")
        if Hq:
            pq, sq = _heads("q", q, bf16, qshape, dev)
            po, so = _heads("q_out", q_out, bf16, qshape, dev)
    pk, sk = _heads("k", k, bf16, kshape, dev)
    pv, sv = _heads("v", v, bf16, kshape, dev)
    n = inv_freq.numel()
    _check(_HOT_APPEND_ROTARY(
        po, so, pq, sq, pk, sk, pv, sv, _ptr("k_cache", k_cache, cdtype, k_cache.numel(), dev),
        _ptr("v_cache", v_cache, cdtype, v_cache.numel(), dev),
        *_tables(slot_mapping, positions, inv_freq, T, n, dev), 2 * n,
        ROTARY_INTERLEAVED if interleaved else 0, float(magnitude), T, Hq, Hkv, D, NB,
        BF16 if cdtype is bf16 else _cache_dtype(k_cache), float(k_scale), float(v_scale),
        _raw_stream(stream, dev)), "kv_append_rotary")


def kv_latent_append(q_out, q_rope, latent, k_rope, cache, slot_mapping, positions, inv_freq,
                     norm_weight=None, eps=1e-6, interleaved=False, magnitude=1.0, stream=None):
    """Append rows to a latent cache [NB, 16, L + R] (kv_latent_append): latent
    [T, L], normalised with norm_weight [L] if given, and k_rope [T, R], turned by
    positions; the queries' rotary parts q_rope [T, H, R] are turned into q_out
    [T, H, R] (a slice of the attention's queries, say; both None: no queries).
    All bfloat16 with any distance between vectors; slot_mapping and positions
    int64 [T], inv_freq float32 [R / 2]."""
    torch = _torch or _load_torch()
    bf16 = torch.bfloat16
    T, L = lshape = latent.shape
    T2, R = rshape = k_rope.shape
    NB, _, W = _cache_shape(cache, True)
    if T2 != T or W != L + R or cache.dtype is not bf16 or (q_rope is None) != (q_out is None):
        raise ValueError("latent must be [T, L], k_rope [T, R], cache bfloat16 [NB, 16, L + R]")
    dev = _current(cache)
    H, qs = 0, (0, 0, 0, 0, 0, 0)
    if q_rope is not None:
        qshape = q_rope.shape
        H = qshape[1]
        if len(qshape) != 3 or qshape[0] != T or qshape[2] != R or q_out.shape != qshape:
            raise ValueError("q_rope and q_out must be [T, H, R]")
        if H:
            qs = (_head_vectors("q_out", q_out, bf16, qshape, dev)
                  + _head_vectors("q_rope", q_rope, bf16, qshape, dev))
    _check(_HOT_LATENT_APPEND(
        *qs, *_vectors("latent", latent, bf16, lshape, dev),
        *_vectors("k_rope", k_rope, bf16, rshape, dev),
        _ptr("norm_weight", norm_weight, bf16, L, dev) if norm_weight is not None else 0,
        float(eps), _ptr("cache", cache, bf16, cache.numel(), dev),
        *_tables(slot_mapping, positions, inv_freq, T, R // 2, dev),
        ROTARY_INTERLEAVED if interleaved else 0, float(magnitude), T, H, L, R, NB,
        _raw_stream(stream, dev)), "kv_latent_append")


def latent_workspace_bytes(num_seqs, max_nodes, num_q_heads, latent_dim, rope_dim):
    n = ctypes.c_size_t(0)
    _check(_lib.paged_latent_workspace_bytes(num_seqs, max_nodes, num_q_heads, latent_dim,
                                             rope_dim, ctypes.byref(n)),
           "paged_latent_workspace_bytes")
    return n.value


def alloc_latent_workspace(num_seqs, max_nodes, num_q_heads, latent_dim, rope_dim, device=None):
    import torch
    nbytes = latent_workspace_bytes(num_seqs, max_nodes, num_q_heads, latent_dim, rope_dim)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device or "cuda")


def paged_latent_attention(out, q, cache, block_tables, context_lens, scale, workspace,
                           node_starts=None, parents=None, max_nodes=1, stream=None):
    """out [T, H, L] = attention of q [T, H, L + R] over a latent cache
    [NB, 16, L + R], all bfloat16 (paged_latent_attention): keys are the cache's
    rows, values their first L elements.  One token a sequence, or, with
    node_starts int32 [B + 1], trees of up to max_nodes drafted tokens (parents
    int32 [T], None: chains), as paged_tree_attention's; block_tables int32
    [B, max_blocks], context_lens int32 [B] including the nodes; workspace from
    alloc_latent_workspace."""
    torch = _torch or _load_torch()
    T, H, W = q.shape
    L = out.shape[-1]
    NB, _, W2 = _cache_shape(cache, True)
    B, max_blocks = block_tables.shape
    bf16, i32 = torch.bfloat16, torch.int32
    if tuple(out.shape) != (T, H, L) or W2 != W or L >= W:
        raise ValueError("q must be [T, H, L + R], out [T, H, L], cache [NB, 16, L + R]")
    _device_only(out, q, workspace)
    dev = _current(cache)
    _check(_HOT_LATENT_ATTENTION(
        _ptr("out", out, bf16, out.numel(), dev), _ptr("q", q, bf16, q.numel(), dev),
        _ptr("cache", cache, bf16, cache.numel(), dev), NB,
        _ptr("block_tables", block_tables, i32, B * max_blocks, dev), max_blocks,
        _ptr("context_lens", context_lens, i32, B, dev),
        _ptr("node_starts", node_starts, i32, B + 1, dev) if node_starts is not None else 0,
        _ptr("parents", parents, i32, T, dev) if parents is not None else 0, B, T, int(max_nodes),
        H, L, W - L, float(scale), _ptr("workspace", workspace, workspace.dtype,
                                        workspace.numel(), dev),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)),
        "paged_latent_attention")


def read_ceiling(buf, sink, stream=None):
    """Stream the device tensor ``buf`` through shared memory with the decode
    kernel's bulk-copy pattern and no arithmetic (kv_read_ceiling), on
    ``stream``; ``sink`` is a zeroed int32 device tensor of 2 elements.  A
    measurement hook: bytes / elapsed time is a read-only bandwidth ceiling."""
    _check(_lib.kv_read_ceiling(_dptr(buf), buf.numel() * buf.element_size(), _dptr(sink),
                                _stream_ptr(stream)), "kv_read_ceiling")


def set_pipeline_stall(cycles):
    """Test hook (kv_test_pipeline_stall): with cycles > 0 every split-kernel
    warp takes the bounded-wait time-out path on its first wait; 0 turns it
    off."""
    _check(_lib.kv_test_pipeline_stall(int(cycles)), "kv_test_pipeline_stall")


def paged_decode_attention_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                                   k_scale=1.0, v_scale=1.0, stream=None):
    """paged_decode_attention without a caller workspace, for callers that
    cannot allocate device memory: the library's own fixed 16 MiB scratch is
    used (shared by every call on the device, so calls must not overlap on
    the GPU).  Shapes needing more raise KVError(KV_ERR_TOO_LARGE)."""
    import torch
    B, Hq, D = q.shape
    NB, Hkv, _, _ = k_cache.shape
    out_dtype = F32 if out.dtype == torch.float32 else BF16
    _check(_lib.paged_decode_attention_noalloc(
        _dptr(out), out_dtype, _dptr(q), _dptr(k_cache), _dptr(v_cache), _cache_dtype(k_cache),
        float(k_scale), float(v_scale), NB, _dptr(block_tables), block_tables.shape[1],
        _dptr(context_lens), B, Hq, Hkv, D, float(scale), _stream_ptr(stream)),
        "paged_decode_attention_noalloc")


def get_device_error():
    """(flags, detail) of the kernels' sticky bounds-check flags; clears them."""
    f = _i(0)
    d = _i64(0)
    _check(_lib.kv_get_device_error(ctypes.byref(f), ctypes.byref(d)), "kv_get_device_error")
    return f.value, d.value


class DecodeStepStaging:
    """Host-to-device plumbing for a stream of decode steps.

    Each of ``slots`` staging slots is one pinned host buffer holding every
    per-step input -- q [B, Hq, D] bf16, k_new / v_new [B, Hkv, D] bf16,
    block_tables [B, max_blocks] int32, context_lens [B] int32 -- at 256-byte
    aligned offsets, mirrored by one device buffer, plus an output buffer on
    each side.  A step costs one host-to-device copy, the fused step kernels
    (paged_decode with the append and KV_DECODE_EARLY_INPUTS) and one
    device-to-host copy of the output.  Uploads
    and downloads run on two copy streams of their own and the slots
    alternate, so step i+1's upload and step i's download overlap the kernels
    of the steps around them.

    The compute stream waits for each upload through an event, which also
    ends the programmatic overlap of consecutive steps.  With
    ``host_ordered=True`` the host instead blocks until the step's upload has
    finished before launching its kernels (the upload was queued a step
    earlier, so the host stays about one step ahead): the compute stream then
    holds only kernel launches and consecutive steps keep their overlap.

    With ``zero_copy=True`` there are no copies and no device slots: the
    kernels read the step's inputs from the pinned host slot and write the
    output into it directly (over NVLink-C2C on a Grace-Blackwell node), and
    the stream of steps stays one chain of kernel launches.

    Use: fill ``host(i)`` views of slot i % slots (``q``, ``k_new``,
    ``v_new``, ``block_tables``, ``context_lens``) once ``ready_for_input(i)``
    holds, call ``step(i, ...)``, and read ``host(i).out`` after
    ``wait_output(i)``."""

    _ALIGN = 256

    class _Slot:
        pass

    def __init__(self, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks,
                 kv_dtype=BF16, device=None, out_dtype=None, slots=2, zero_copy=False,
                 host_ordered=False):
        import torch
        self.device = torch.device(device or "cuda")
        self.zero_copy = bool(zero_copy)
        self.host_ordered = bool(host_ordered)
        B, Hq, Hkv, D = num_seqs, num_q_heads, num_kv_heads, head_dim
        parts = [("q", (B, Hq, D), torch.bfloat16), ("k_new", (B, Hkv, D), torch.bfloat16),
                 ("v_new", (B, Hkv, D), torch.bfloat16),
                 ("block_tables", (B, max_blocks), torch.int32),
                 ("context_lens", (B,), torch.int32)]
        offs, off = {}, 0
        for name, shape, dt in parts:
            nbytes = int(np.prod(shape)) * torch.empty((), dtype=dt).element_size()
            offs[name] = (off, shape, dt, nbytes)
            off = -(-(off + nbytes) // self._ALIGN) * self._ALIGN
        self.nbytes = off
        od = out_dtype or torch.bfloat16
        self._slots = []
        for _ in range(slots):
            h, d = self._Slot(), self._Slot()
            h.raw = torch.empty(off, dtype=torch.uint8).pin_memory()
            h.out = torch.empty((B, Hq, D), dtype=od).pin_memory()
            if self.zero_copy:
                d = h                   # the kernels address the pinned slot itself
            else:
                d.raw = torch.empty(off, dtype=torch.uint8, device=self.device)
                d.out = torch.empty((B, Hq, D), dtype=od, device=self.device)
            for name, (o, shape, dt, nb) in offs.items():
                setattr(h, name, h.raw[o:o + nb].view(dt).view(shape))
                if d is not h:
                    setattr(d, name, d.raw[o:o + nb].view(dt).view(shape))
            ev = {k: torch.cuda.Event() for k in ("uploaded", "computed", "downloaded")}
            self._slots.append((h, d, ev))
        self.upload_stream = torch.cuda.Stream(self.device)
        self.download_stream = torch.cuda.Stream(self.device)
        self.workspace = alloc_workspace(B, Hq, Hkv, D, kv_dtype, device=self.device)

    def host(self, i):
        return self._slots[i % len(self._slots)][0]

    @property
    def h2d_bytes(self):
        """Bytes of inputs a step moves host to device (copied, or read in
        place with zero_copy)."""
        return self.nbytes

    @property
    def d2h_bytes(self):
        h = self._slots[0][0]
        return h.out.numel() * h.out.element_size()

    def ready_for_input(self, i):
        """Block the host until slot i % slots may be refilled (its previous
        upload has finished; with zero_copy, its previous step)."""
        ev = self._slots[i % len(self._slots)][2]
        (ev["computed"] if self.zero_copy else ev["uploaded"]).synchronize()

    def wait_output(self, i):
        ev = self._slots[i % len(self._slots)][2]
        (ev["computed"] if self.zero_copy else ev["downloaded"]).synchronize()

    def step(self, i, k_cache, v_cache, scale, k_scale=1.0, v_scale=1.0, stream=None):
        """Upload slot i's inputs, run the fused decode step on `stream`,
        download its output (all asynchronous)."""
        import torch
        h, d, ev = self._slots[i % len(self._slots)]
        s = stream or torch.cuda.current_stream(self.device)
        if self.zero_copy:
            # the slot is refilled by the host only after ready_for_input(i),
            # and the kernel before is the previous step's: early reads are safe
            paged_decode(h.out, h.q, k_cache, v_cache, h.block_tables, h.context_lens, scale,
                         self.workspace, k_scale, v_scale, k_new=h.k_new, v_new=h.v_new,
                         early_inputs=True, stream=s)
            ev["computed"].record(s)
            return
        up, down = self.upload_stream, self.download_stream
        # the device slot is free once its previous step has been computed and
        # its output downloaded (the download follows the computation)
        up.wait_event(ev["downloaded"])
        with torch.cuda.stream(up):
            d.raw.copy_(h.raw, non_blocking=True)
            ev["uploaded"].record(up)
        if self.host_ordered:
            ev["uploaded"].synchronize()
        else:
            s.wait_event(ev["uploaded"])
        # the inputs arrive by a copy joined through an event, and the kernel
        # before is the previous step's: the early reads are safe
        paged_decode(d.out, d.q, k_cache, v_cache, d.block_tables, d.context_lens, scale,
                     self.workspace, k_scale, v_scale, k_new=d.k_new, v_new=d.v_new,
                     early_inputs=True, stream=s)
        ev["computed"].record(s)
        down.wait_event(ev["computed"])
        with torch.cuda.stream(down):
            h.out.copy_(d.out, non_blocking=True)
            ev["downloaded"].record(down)

    def join(self, stream=None):
        """Make `stream` wait for every upload and download issued so far."""
        import torch
        s = stream or torch.cuda.current_stream(self.device)
        s.wait_stream(self.upload_stream)
        s.wait_stream(self.download_stream)
