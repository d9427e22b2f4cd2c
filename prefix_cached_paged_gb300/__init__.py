"""prefix_cached_paged_gb300 -- RadixAttention's data path on one GB300 (sm_103a).

A thin binding of librc (include/rc.h): a token-granular KV pool, a radix tree that finds each
request's longest cached prefix and evicts unreferenced leaves in LRU order (host C++), and the
extend / decode attention kernels that run on a paged KV pool through a slot table (CUDA).
The binding only marshals arguments: every step runs in librc, and there is no fallback path --
without the compiled library every call raises.

Names follow the C ABI without the `rc_` prefix. Device functions take torch CUDA tensors (used
for device memory and streams only) and launch on the current torch stream.
"""
from __future__ import annotations

import ctypes

import numpy as np

from ._lib import (RC_DTYPE_BF16, RC_DTYPE_F32, RC_ERR_CUDA, RC_ERR_DEVICE, RC_ERR_INSUFFICIENT,
                   RC_ERR_INVALID, RC_ERR_OOM, RC_OK, RC_SCHED_FCFS, RC_SCHED_LSPF, RcDecodeArgs,
                   RcError, RcExtendArgs, RcKvAppendArgs, RcKvBlockBoundsArgs, RcKvCopyArgs,
                   RcQkNormRopeArgs, RcSlotWriteArgs, RcSparseDecodeArgs, RcStackPlan,
                   RcStackPlanArgs, RcStats, check, lib)

__all__ = [
    "Pool", "RadixTree", "RcError", "slot_table_write", "extend_attention", "decode_attention",
    "rope_table", "qk_norm_rope", "kv_append", "kv_block_bounds", "sparse_decode_attention",
    "sparse_decode_workspace_bytes",
    "decode_workspace_bytes", "decode_attention_noalloc", "device_status", "launch_count", "RC_OK", "RC_ERR_INVALID",
    "RC_ERR_OOM", "RC_ERR_INSUFFICIENT", "RC_ERR_CUDA", "RC_ERR_DEVICE", "RC_SCHED_LSPF",
    "RC_SCHED_FCFS",
]


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def _p(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def launch_count() -> int:
    return int(lib().rc_launch_count())


def set_wait_limit_ns(ns: int) -> None:
    """Test hook (rc_debug_set_wait_limit_ns): bound of the extend kernel's waits for later
    launches; 0 restores the default."""
    check(lib().rc_debug_set_wait_limit_ns(int(ns)), "rc_debug_set_wait_limit_ns")


class Pool:
    """The token pool (free list of KV slots). rc_pool_* / rc_kv_pool_*."""

    def __init__(self, num_slots: int, initial_order=None):
        self._order = None if initial_order is None else _i32(initial_order)
        h = ctypes.c_void_p()
        check(lib().rc_pool_create(int(num_slots), None if self._order is None else
                                   _p(self._order), ctypes.byref(h)), "rc_pool_create")
        self.h = h
        self.num_slots = int(num_slots)

    def __del__(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().rc_pool_destroy(self.h)
            self.h = None

    def alloc(self, n: int, out: np.ndarray | None = None) -> np.ndarray:
        out = np.empty(int(n), dtype=np.int32) if out is None else out
        check(lib().rc_kv_pool_alloc(self.h, int(n), _p(out)), "rc_kv_pool_alloc")
        return out

    def free(self, slots) -> None:
        s = _i32(slots)
        check(lib().rc_kv_pool_free(self.h, _p(s), len(s)), "rc_kv_pool_free")

    def available(self) -> int:
        v = ctypes.c_int64()
        check(lib().rc_kv_pool_available(self.h, ctypes.byref(v)), "rc_kv_pool_available")
        return int(v.value)

    def inject_alloc_failure(self, after_calls: int) -> None:
        """Test hook: the alloc() after `after_calls` more successful ones fails with
        RC_ERR_OOM and changes nothing (one shot; -1 disarms)."""
        check(lib().rc_pool_inject_alloc_failure(self.h, int(after_calls)),
              "rc_pool_inject_alloc_failure")


class RadixTree:
    """The radix tree over token sequences. rc_radix_*."""

    def __init__(self, pool: Pool):
        self.pool = pool
        h = ctypes.c_void_p()
        check(lib().rc_radix_create(pool.h, ctypes.byref(h)), "rc_radix_create")
        self.h = h

    def __del__(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().rc_radix_destroy(self.h)
            self.h = None

    def match_prefix(self, tokens):
        t = _i32(tokens)
        out = np.empty(len(t), dtype=np.int32)
        n = ctypes.c_int64()
        node = ctypes.c_uint64()
        check(lib().rc_radix_match_prefix(self.h, _p(t), len(t), _p(out), ctypes.byref(n),
                                          ctypes.byref(node)), "rc_radix_match_prefix")
        return int(n.value), out[: n.value].copy(), int(node.value)

    def insert(self, tokens, slots):
        t, s = _i32(tokens), _i32(slots)
        ex = ctypes.c_int64()
        node = ctypes.c_uint64()
        check(lib().rc_radix_insert(self.h, _p(t), _p(s), len(t), ctypes.byref(ex),
                                    ctypes.byref(node)), "rc_radix_insert")
        return int(ex.value), int(node.value)

    def lock(self, node: int) -> None:
        check(lib().rc_radix_lock(self.h, int(node)), "rc_radix_lock")

    def unlock(self, node: int) -> None:
        check(lib().rc_radix_unlock(self.h, int(node)), "rc_radix_unlock")

    def evict_lru(self, n_tokens: int):
        """Returns (status, freed): status RC_OK or RC_ERR_INSUFFICIENT."""
        f = ctypes.c_int64()
        rc = lib().rc_radix_evict_lru(self.h, int(n_tokens), ctypes.byref(f))
        if rc not in (RC_OK, RC_ERR_INSUFFICIENT):
            check(rc, "rc_radix_evict_lru")
        return rc, int(f.value)

    def stats(self) -> dict:
        s = RcStats()
        check(lib().rc_radix_stats(self.h, ctypes.byref(s)), "rc_radix_stats")
        return {k: int(getattr(s, k)) for k, _ in RcStats._fields_}

    def dump(self) -> np.ndarray:
        n = lib().rc_radix_dump(self.h, None, 0)
        need = -n if n < 0 else n
        buf = np.empty(max(need, 1), dtype=np.int64)
        w = lib().rc_radix_dump(self.h, _p(buf), need)
        assert w >= 0
        return buf[:w].copy()

    def match_batch(self, tokens: np.ndarray, indptr: np.ndarray, match_len, rows: np.ndarray):
        """Match + lock B sequences in order. rows: [B, row_stride] int32 (written in place).
        Returns (prefix_len int32[B], nodes uint64[B])."""
        B = len(indptr) - 1
        pl = np.empty(B, dtype=np.int32)
        nodes = np.empty(B, dtype=np.uint64)
        ml = None if match_len is None else _i32(match_len)
        check(lib().rc_radix_match_batch(self.h, _p(tokens), _p(indptr), B,
                                         None if ml is None else _p(ml), _p(rows),
                                         rows.shape[1], _p(pl), _p(nodes)),
              "rc_radix_match_batch")
        return pl, nodes

    def attach_host_tier(self, host_pool: "Pool") -> None:
        """Evicted device leaves move to host_pool's slots instead of being freed."""
        check(lib().rc_radix_attach_host_tier(self.h, host_pool.h), "rc_radix_attach_host_tier")
        self.host_pool = host_pool

    def match_batch_tiered(self, tokens, indptr, match_len, rows):
        """Match + lock B sequences through both tiers. Returns (prefix_len int32[B] = the
        device-resident part, nodes uint64[B], host_len int32[B])."""
        B = len(indptr) - 1
        pl = np.empty(B, dtype=np.int32)
        nodes = np.empty(B, dtype=np.uint64)
        hl = np.empty(B, dtype=np.int32)
        ml = None if match_len is None else _i32(match_len)
        check(lib().rc_radix_match_batch_tiered(self.h, _p(tokens), _p(indptr), B,
                                                None if ml is None else _p(ml), _p(rows),
                                                rows.shape[1], _p(pl), _p(nodes), _p(hl)),
              "rc_radix_match_batch_tiered")
        return pl, nodes, hl

    def load_batch(self, tokens, indptr, rows, prefix_len, host_len) -> None:
        """Move the matched host-resident tokens back to the device; prefix_len (int32, in
        place) grows by host_len and rows receive the new device slots."""
        assert prefix_len.dtype == np.int32 and prefix_len.flags.c_contiguous
        hl = _i32(host_len)
        check(lib().rc_radix_load_batch(self.h, _p(tokens), _p(indptr), len(indptr) - 1,
                                        _p(rows), rows.shape[1], _p(prefix_len), _p(hl)),
              "rc_radix_load_batch")

    def drain_copies(self):
        """The copies owed since the last drain: (spill_dev, spill_host, load_host, load_dev),
        spills to run before loads."""
        ns, nl = ctypes.c_int64(), ctypes.c_int64()
        check(lib().rc_radix_pending_copies(self.h, ctypes.byref(ns), ctypes.byref(nl)),
              "rc_radix_pending_copies")
        sd = np.empty(ns.value, np.int32)
        sh = np.empty(ns.value, np.int32)
        lh = np.empty(nl.value, np.int32)
        ld = np.empty(nl.value, np.int32)
        check(lib().rc_radix_drain_copies(self.h, _p(sd), _p(sh), _p(lh), _p(ld)),
              "rc_radix_drain_copies")
        return sd, sh, lh, ld

    def tiers(self) -> np.ndarray:
        """(node id, 1 if host-resident) per node, in the dump's order."""
        n = lib().rc_radix_tiers(self.h, None, 0)
        need = -n if n < 0 else n
        buf = np.empty(max(need, 1), dtype=np.int64)
        w = lib().rc_radix_tiers(self.h, _p(buf), need)
        assert w >= 0
        return buf[:w]

    def schedule_batch(self, tokens: np.ndarray, indptr: np.ndarray, match_len=None,
                       policy: int = 0, max_batch: int = 1 << 30, max_new_tokens: int = -1,
                       reserve_slots: int = 0):
        """Batch formation over W waiting sequences (the tree is not changed); policy
        RC_SCHED_LSPF (longest shared prefix first) or RC_SCHED_FCFS (queue order). Returns
        (order int32[W], match int32[W], admitted): the batch is order[:admitted]."""
        W = len(indptr) - 1
        order = np.empty(W, dtype=np.int32)
        match = np.empty(W, dtype=np.int32)
        adm = ctypes.c_int32()
        ml = None if match_len is None else _i32(match_len)
        tok = _i32(tokens)
        ip = np.ascontiguousarray(indptr, np.int64)
        check(lib().rc_schedule_batch(self.h, _p(tok), _p(ip), W,
                                      None if ml is None else _p(ml), int(policy),
                                      int(max_batch), int(max_new_tokens), int(reserve_slots),
                                      _p(order), _p(match), ctypes.byref(adm)),
              "rc_schedule_batch")
        return order, match, int(adm.value)

    def schedule_batch_ranges(self, tokens: np.ndarray, starts: np.ndarray, lengths: np.ndarray,
                              match_len=None, policy: int = 0, max_batch: int = 1 << 30,
                              max_new_tokens: int = -1, reserve_slots: int = 0):
        """schedule_batch over W sequences given as ranges of one buffer: sequence w is
        tokens[starts[w] : starts[w] + lengths[w]]. Same outputs as schedule_batch."""
        W = len(starts)
        order = np.empty(W, dtype=np.int32)
        match = np.empty(W, dtype=np.int32)
        adm = ctypes.c_int32()
        ml = None if match_len is None else _i32(match_len)
        tok = _i32(tokens)
        st = np.ascontiguousarray(starts, np.int64)
        ln = np.ascontiguousarray(lengths, np.int64)
        check(lib().rc_schedule_batch_ranges(self.h, _p(tok), _p(st), _p(ln), W,
                                             None if ml is None else _p(ml), int(policy),
                                             int(max_batch), int(max_new_tokens),
                                             int(reserve_slots), _p(order), _p(match),
                                             ctypes.byref(adm)),
              "rc_schedule_batch_ranges")
        return order, match, int(adm.value)

    def insert_batch(self, tokens, indptr, rows, prefix_len, unlock_nodes, keep_locked=False):
        """Insert B sequences with their slot rows, free duplicates, optionally lock the ends,
        unlock the matched nodes. Returns (end_nodes uint64[B], duplicates freed)."""
        B = len(indptr) - 1
        ends = np.empty(B, dtype=np.uint64)
        freed = ctypes.c_int64()
        un = None if unlock_nodes is None else np.ascontiguousarray(unlock_nodes, np.uint64)
        check(lib().rc_radix_insert_batch(self.h, _p(tokens), _p(indptr), B, _p(rows),
                                          rows.shape[1], _p(_i32(prefix_len)),
                                          None if un is None else _p(un), int(keep_locked),
                                          _p(ends), ctypes.byref(freed)),
              "rc_radix_insert_batch")
        return ends, int(freed.value)


# ------------------------------------------------------------------ device entry points
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return RC_DTYPE_BF16
    if t.dtype == torch.float32:
        return RC_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def slot_table_write(req_to_token, seg_row, seg_col, seg_indptr, values, stream=None):
    """req_to_token[seg_row[i], seg_col[i] + j] = values[seg_indptr[i] + j] (device int32)."""
    a = RcSlotWriteArgs(num_segments=seg_row.numel(), max_reqs=req_to_token.shape[0],
                        max_ctx=req_to_token.shape[1], total_values=values.numel(),
                        seg_row=seg_row.data_ptr(), seg_col=seg_col.data_ptr(),
                        seg_indptr=seg_indptr.data_ptr(), values=values.data_ptr(),
                        req_to_token=req_to_token.data_ptr())
    check(lib().rc_slot_table_write(ctypes.byref(a), _stream(stream)), "rc_slot_table_write")


def kv_copy(src_k, src_v, src_slots, dst_k, dst_v, dst_slots, stream=None):
    """For every i and layer: K and V rows of src_slots[i] -> dst_slots[i]. Planes are
    [layers, num_slots, Hkv, d] tensors on the device or in pinned host memory (the host tier);
    slot arrays are device int32."""
    for t in (src_k, src_v, dst_k, dst_v):
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("kv_copy: planes must be device tensors or pinned host tensors")
        if not t.is_contiguous():
            raise ValueError("kv_copy: planes must be contiguous")
    if src_k.shape[0] != dst_k.shape[0] or src_k.shape[2:] != dst_k.shape[2:] or \
            src_k.dtype != dst_k.dtype or src_k.shape != src_v.shape or dst_k.shape != dst_v.shape:
        raise ValueError("kv_copy: plane shapes or dtypes differ")
    if src_slots.numel() != dst_slots.numel():
        raise ValueError("kv_copy: slot arrays differ in length")
    row = src_k.shape[2] * src_k.shape[3] * src_k.element_size()
    a = RcKvCopyArgs(n=src_slots.numel(), layers=src_k.shape[0], row_bytes=row,
                     src_slots=src_slots.data_ptr(), dst_slots=dst_slots.data_ptr(),
                     src_k=src_k.data_ptr(), src_v=src_v.data_ptr(),
                     src_num_slots=src_k.shape[1], dst_k=dst_k.data_ptr(),
                     dst_v=dst_v.data_ptr(), dst_num_slots=dst_k.shape[1])
    check(lib().rc_kv_copy(ctypes.byref(a), _stream(stream)), "rc_kv_copy")


def _extend_args(q, k_new, v_new, out_loc, qo_indptr, prefix_len, req_idx, req_to_token,
                 k_pool, v_pool, o, lse, sm_scale, max_q_len, max_prefix_len, stack=None,
                 workspace=None):
    T, Hq, d = q.shape
    Hkv = k_new.shape[1]
    g = {}
    if stack is not None:
        # (ranges, shared, max_rows) or, for a cascade over tree levels, (ranges, shared,
        # max_rows, start, level_indptr) -- level_indptr a host int32 numpy array
        ranges, shared, max_rows = stack[:3]
        g = dict(num_groups=int(shared.numel()), max_group_rows=int(max_rows),
                 group_range=ranges.data_ptr(), group_shared=shared.data_ptr(),
                 workspace=0 if workspace is None else workspace.data_ptr(),
                 workspace_bytes=0 if workspace is None else
                 workspace.numel() * workspace.element_size())
        if len(stack) >= 5:
            start, level_indptr = stack[3], stack[4]
            assert level_indptr.dtype == np.int32 and level_indptr.flags.c_contiguous
            g.update(num_levels=len(level_indptr) - 1, level_indptr=level_indptr.ctypes.data,
                     group_start=start.data_ptr())
        if len(stack) >= 7 and stack[5] is not None:
            # (..., group_fold device int32 [G], every request folded)
            g.update(group_fold=stack[5].data_ptr(), skip_request_pass=int(bool(stack[6])))
    return RcExtendArgs(**g,
        dtype=_dtype_code(q), num_reqs=prefix_len.numel(), num_q_heads=Hq, num_kv_heads=Hkv,
        head_dim=d, max_reqs=req_to_token.shape[0], max_ctx=req_to_token.shape[1], max_q_len=int(max_q_len),
        max_prefix_len=int(max_prefix_len), num_tokens=T, num_slots=k_pool.shape[0],
        sm_scale=float(sm_scale), q=q.data_ptr(), k_new=k_new.data_ptr(),
        v_new=v_new.data_ptr(), out_loc=out_loc.data_ptr(), qo_indptr=qo_indptr.data_ptr(),
        prefix_len=prefix_len.data_ptr(), req_idx=req_idx.data_ptr(),
        req_to_token=req_to_token.data_ptr(), k_pool=k_pool.data_ptr(),
        v_pool=v_pool.data_ptr(), o=o.data_ptr(), lse=0 if lse is None else lse.data_ptr())


def extend_workspace_bytes(num_tokens: int, num_q_heads: int) -> int:
    """Workspace of the stacked prefix pass (rc_extend_workspace_bytes)."""
    a = RcExtendArgs(num_tokens=int(num_tokens), num_q_heads=int(num_q_heads))
    n = ctypes.c_size_t()
    check(lib().rc_extend_workspace_bytes(ctypes.byref(a), ctypes.byref(n)),
          "rc_extend_workspace_bytes")
    return int(n.value)


def extend_attention(q, k_new, v_new, out_loc, qo_indptr, prefix_len, req_idx, req_to_token,
                     k_pool, v_pool, o, *, sm_scale, max_q_len, max_prefix_len, lse=None,
                     stack=None, workspace=None, stream=None):
    """Extend attention of one layer (see rc_extend_attention). k_pool / v_pool are this layer's
    planes [num_slots, Hkv, d]. stack: optional prefix-stacking groups (ranges, shared,
    max_group_rows) -- int32 CUDA tensors and an int, as built by prefix_stacking_groups() --
    with a uint8 CUDA workspace of extend_workspace_bytes(T, Hq) bytes."""
    a = _extend_args(q, k_new, v_new, out_loc, qo_indptr, prefix_len, req_idx, req_to_token,
                     k_pool, v_pool, o, lse, sm_scale, max_q_len, max_prefix_len, stack,
                     workspace)
    check(lib().rc_extend_attention(ctypes.byref(a), _stream(stream)), "rc_extend_attention")


def _decode_args(q, k_new, v_new, out_loc, seq_len, req_idx, req_to_token, k_pool, v_pool, o,
                 lse, sm_scale, max_total_tokens, kv_chunk, groups=None):
    B, Hq, d = q.shape
    g = dict(num_groups=0, group_indptr=0, group_members=0, group_shared=0)
    if groups is not None:
        indptr, members, shared = groups
        g = dict(num_groups=int(shared.numel()), group_indptr=indptr.data_ptr(),
                 group_members=members.data_ptr(), group_shared=shared.data_ptr())
    return RcDecodeArgs(**g,
        dtype=_dtype_code(q), num_reqs=B, num_q_heads=Hq, num_kv_heads=k_new.shape[1],
        head_dim=d, max_reqs=req_to_token.shape[0], max_ctx=req_to_token.shape[1], kv_chunk=int(kv_chunk),
        max_total_tokens=int(max_total_tokens), num_slots=k_pool.shape[0],
        sm_scale=float(sm_scale), q=q.data_ptr(), k_new=k_new.data_ptr(),
        v_new=v_new.data_ptr(), out_loc=out_loc.data_ptr(), seq_len=seq_len.data_ptr(),
        req_idx=req_idx.data_ptr(), req_to_token=req_to_token.data_ptr(),
        k_pool=k_pool.data_ptr(), v_pool=v_pool.data_ptr(), o=o.data_ptr(),
        lse=0 if lse is None else lse.data_ptr())


def decode_workspace_bytes(q, k_new, req_to_token, k_pool, *, max_total_tokens, kv_chunk=0) -> int:
    B, Hq, d = q.shape
    a = RcDecodeArgs(dtype=_dtype_code(q), num_reqs=B, num_q_heads=Hq,
                     num_kv_heads=k_new.shape[1], head_dim=d, max_reqs=req_to_token.shape[0],
                     max_ctx=req_to_token.shape[1],
                     kv_chunk=int(kv_chunk), max_total_tokens=int(max_total_tokens),
                     num_slots=k_pool.shape[0])
    n = ctypes.c_size_t()
    check(lib().rc_decode_workspace_bytes(ctypes.byref(a), ctypes.byref(n)),
          "rc_decode_workspace_bytes")
    return int(n.value)


def decode_attention(q, k_new, v_new, out_loc, seq_len, req_idx, req_to_token, k_pool, v_pool,
                     o, workspace, *, sm_scale, max_total_tokens, kv_chunk=0, lse=None,
                     groups=None, stream=None, reuse_plan=False):
    """Split-K decode attention of one layer (see rc_decode_attention). workspace: a uint8 CUDA
    tensor of at least decode_workspace_bytes(...) bytes. groups: optional shared-context groups
    (indptr, members, shared), int32 CUDA tensors, as built by shared_context_groups().
    reuse_plan: the previous call on this workspace had the same requests and sizes (the other
    layers of a decode step) -- its job list is reused."""
    a = _decode_args(q, k_new, v_new, out_loc, seq_len, req_idx, req_to_token, k_pool, v_pool,
                     o, lse, sm_scale, max_total_tokens, kv_chunk, groups)
    a.reuse_plan = 1 if reuse_plan else 0
    check(lib().rc_decode_attention(ctypes.byref(a), ctypes.c_void_p(workspace.data_ptr()),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "rc_decode_attention")


DEFAULT_KV_CHUNK = 512   # tokens per split-K chunk when kv_chunk = 0 (rc.h)


MAX_STACK_LEVELS = 4   # RC_MAX_STACK_LEVELS
_FOLD_MODES = {False: 0, True: 1, "always": 2}   # RC_FOLD_NONE / RC_FOLD_COST / RC_FOLD_ALL


def plan_extend_stacking(rows, prefix_len, new_len, min_shared: int, group: int,
                         max_levels: int = MAX_STACK_LEVELS, policy="cost", fold=True):
    """rc_plan_extend_stacking: the extend batch's stacking groups over the levels of the tree.
    rows: int32 [B, stride] host slot rows; policy "cost" (groups estimated to pay) or "all";
    fold True (where estimated to pay), "always" or False. Returns (ranges [2 G], shared [G],
    start [G], level_indptr [L + 1], max_group_rows, fold [G], all_folded) as int32 numpy arrays
    (and an int and a bool); G = 0 when there is none."""
    rows = np.ascontiguousarray(rows, dtype=np.int32)
    B = rows.shape[0]
    P, S = _i32(prefix_len), _i32(new_len)
    a = RcStackPlanArgs(num_reqs=B, rows=_p(rows), row_stride=rows.shape[1] if rows.ndim == 2 else 0,
                        prefix_len=_p(P), new_len=_p(S), min_shared=int(min_shared),
                        group_size=int(group), max_levels=int(max_levels),
                        policy={"cost": 0, "all": 1}[policy], fold=_FOLD_MODES[fold])
    cap = max(B * int(max_levels), 1)
    rng, sh, st, fo = (np.zeros(2 * cap, np.int32), np.zeros(cap, np.int32),
                       np.zeros(cap, np.int32), np.zeros(cap, np.int32))
    out = RcStackPlan(capacity=cap, group_range=_p(rng), group_shared=_p(sh), group_start=_p(st),
                      group_fold=_p(fo))
    check(lib().rc_plan_extend_stacking(ctypes.byref(a), ctypes.byref(out)),
          "rc_plan_extend_stacking")
    G, L = out.num_groups, out.num_levels
    return (rng[:2 * G].copy(), sh[:G].copy(), st[:G].copy(),
            np.asarray(out.level_indptr[:L + 1], np.int32), int(out.max_group_rows),
            fo[:G].copy(), bool(out.all_folded))


def shared_context_groups(rows, lengths, group_size: int, min_shared: int):
    """rc_plan_decode_groups: decode requests whose slot rows start with the same slots share
    that prefix's KV. rows: int32 [B, >= max(lengths)] host slot rows, lengths: context tokens
    per request. Returns (indptr, members, shared) int32 numpy arrays (no groups: [0] and two
    empty arrays)."""
    rows = np.ascontiguousarray(rows, dtype=np.int32)
    L = np.ascontiguousarray(lengths, dtype=np.int64)
    B = len(L)
    indptr = np.zeros(B + 1, np.int32)
    members = np.zeros(max(B, 1), np.int32)
    shared = np.zeros(max(B, 1), np.int32)
    ng = ctypes.c_int32()
    check(lib().rc_plan_decode_groups(_p(rows), rows.shape[1] if rows.ndim == 2 else 0, _p(L),
                                      B, int(group_size), int(min_shared), _p(indptr),
                                      _p(members), _p(shared), ctypes.byref(ng)),
          "rc_plan_decode_groups")
    G = ng.value
    return indptr[:G + 1].copy(), members[:indptr[G]].copy(), shared[:G].copy()


STATIC_SCRATCH_BYTES = 32 << 20


def decode_attention_noalloc(q, k_new, v_new, out_loc, seq_len, req_idx, req_to_token, k_pool,
                             v_pool, o, *, sm_scale, max_total_tokens, kv_chunk=0, lse=None,
                             stream=None):
    """decode_attention without a workspace, for callers that cannot allocate device memory
    (see rc_decode_attention_noalloc): its scratch is a fixed STATIC_SCRATCH_BYTES area inside
    librc shared by every call on the device, so calls that overlap on the GPU race."""
    a = _decode_args(q, k_new, v_new, out_loc, seq_len, req_idx, req_to_token, k_pool, v_pool,
                     o, lse, sm_scale, max_total_tokens, kv_chunk)
    check(lib().rc_decode_attention_noalloc(ctypes.byref(a), _stream(stream)),
          "rc_decode_attention_noalloc")


# ------------------------------------------------------------------ norms, rotation, append, sparse
def _raw_stream(dev, stream):
    """The stream to launch on, as an integer: the given one, or device dev's current one."""
    return (_torch()._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _require(fn, dev, tensors):
    """Each (name, tensor, dtype, shape) is a contiguous CUDA tensor on the current device (the call
    launches on a stream of it), of that dtype and shape."""
    for name, t, dtype, shape in tensors:
        if t.get_device() != dev:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor on the current device "
                             f"(cuda:{dev})")
        if t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")


def _dims(fn, name, t, n):
    """The shape of an n-dimensional tensor."""
    if t.dim() != n:
        raise ValueError(f"{fn}: {name} must have {n} dimensions, not {t.dim()}")
    return t.shape


def _heads(fn, dev, name, t, dtype, shape, out=False):
    """(token stride, head stride) in elements of a [T, H, d] tensor whose heads are contiguous."""
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor on the current device (cuda:{dev})")
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    T, H, d = shape
    if t.is_contiguous():
        return H * d, d
    st, sh, se = t.stride()
    if se != 1 and d > 1:
        raise ValueError(f"{fn}: the heads of {name} must be contiguous")
    # the stride of a dimension of size 1 says nothing
    st, sh = st if T > 1 else 0, sh if H > 1 else 0
    if out and ((st == 0 and T > 1) or (sh == 0 and H > 1)):
        raise ValueError(f"{fn}: {name} is expanded: its rows share memory")
    return st, sh


def rope_table(inv_freq, num_positions: int, *, first_position: int = 0,
               scale: float = 1.0) -> np.ndarray:
    """rc_rope_table: float32 numpy array [num_positions, 2 * len(inv_freq)] of the rotation's
    cosines and sines, computed in double precision on the host. inv_freq: one frequency per
    rotated pair (for the usual base: base ** (-2 i / rotary_dim)), a multiple of 8 of them."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.ndim != 1:
        raise ValueError("rope_table: inv_freq must be one-dimensional")
    out = np.empty((max(int(num_positions), 0), 2 * len(f)), dtype=np.float32)
    check(lib().rc_rope_table(_p(f), len(f), int(first_position), int(num_positions),
                              float(scale), _p(out)), "rc_rope_table")
    return out


def qk_norm_rope(q, k, positions=None, rope=None, *, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head with the position rotation in the same pass (see
    rc_qk_norm_rope). q [T, Hq, d] and k [T, Hkv, d]: CUDA tensors whose heads are contiguous, any
    token and head strides (slices of a fused projection); either may be None. positions: int32
    [T]; rope: fp32 [max_position, rotary_dim] (rope_table) or None for norms only; q_weight /
    k_weight: [d] or None for no norm. q_out / k_out: where the results go, in place when None; any
    other overlap with an input or with one another is refused."""
    fn = "qk_norm_rope"
    torch = _torch()
    dev = torch.cuda.current_device()
    x = q if q is not None else k
    if x is None:
        raise ValueError(f"{fn}: neither q nor k is given")
    if (q is None and (q_out is not None or q_weight is not None)) or \
            (k is None and (k_out is not None or k_weight is not None)):
        raise ValueError(f"{fn}: a weight or an output without its input")
    if rope is None and q_weight is None and k_weight is None:
        raise ValueError(f"{fn}: neither a rotation nor a norm is given")
    T, _, d = _dims(fn, "q" if q is not None else "k", x, 3)
    dt = x.dtype
    rot = max_pos = p_rope = p_pos = Hq = Hkv = p_q = p_k = p_wq = p_wk = p_qo = p_ko = 0
    qt = qh = kt = kh = qot = qoh = kot = koh = 0
    if rope is not None:
        if positions is None:
            raise ValueError(f"{fn}: the rotation needs positions")
        max_pos, rot = _dims(fn, "rope", rope, 2)
        _require(fn, dev, (("rope", rope, torch.float32, (max_pos, rot)),
                           ("positions", positions, torch.int32, (T,))))
        p_rope, p_pos = rope.data_ptr(), positions.data_ptr()
    if q is not None:
        Hq = q.shape[1]
        shape = (T, Hq, d)
        qt, qh = _heads(fn, dev, "q", q, dt, shape, q_out is None)
        p_q = p_qo = q.data_ptr()
        qot, qoh = qt, qh
        if q_out is not None:
            p_qo = q_out.data_ptr()
            qot, qoh = _heads(fn, dev, "q_out", q_out, dt, shape, True)
        if q_weight is not None:
            _require(fn, dev, (("q_weight", q_weight, dt, (d,)),))
            p_wq = q_weight.data_ptr()
    if k is not None:
        Hkv = _dims(fn, "k", k, 3)[1]
        shape = (T, Hkv, d)
        kt, kh = _heads(fn, dev, "k", k, dt, shape, k_out is None)
        p_k = p_ko = k.data_ptr()
        kot, koh = kt, kh
        if k_out is not None:
            p_ko = k_out.data_ptr()
            kot, koh = _heads(fn, dev, "k_out", k_out, dt, shape, True)
        if k_weight is not None:
            _require(fn, dev, (("k_weight", k_weight, dt, (d,)),))
            p_wk = k_weight.data_ptr()
    a = RcQkNormRopeArgs(_dtype_code(x), Hq, Hkv, d, rot, 1 if interleaved else 0, eps, T, max_pos,
                         p_q, qt, qh, p_k, kt, kh, p_wq, p_wk, p_pos, p_rope, p_qo, qot, qoh, p_ko,
                         kot, koh)
    check(lib().rc_qk_norm_rope(ctypes.byref(a), _raw_stream(dev, stream)), "rc_qk_norm_rope")


def kv_append(k, v, out_loc, qo_indptr, prefix_len, k_pool, v_pool, *, rope=None, k_weight=None,
              eps=1e-6, interleaved=False, bounds=None, req_idx=None, block=64, stream=None):
    """Append the new tokens' keys (normalised with k_weight and rotated by rope, each optional)
    and values to one layer's planes [num_slots, Hkv, d] (see rc_kv_append). k, v [T, Hkv, d] with
    any token and head strides; out_loc [T], qo_indptr [B + 1], prefix_len [B], req_idx [B] int32.
    bounds: one layer's block bounds [max_reqs, max_blocks, Hkv, 2, d], updated for the blocks the
    tokens fall into (with req_idx)."""
    fn = "kv_append"
    torch = _torch()
    dev = torch.cuda.current_device()
    dt, i32 = k_pool.dtype, torch.int32
    S, Hkv, d = _dims(fn, "k_pool", k_pool, 3)
    T, B = _dims(fn, "k", k, 3)[0], prefix_len.numel()
    kt, kh = _heads(fn, dev, "k", k, dt, (T, Hkv, d))
    vt, vh = _heads(fn, dev, "v", v, dt, (T, Hkv, d))
    _require(fn, dev, (("k_pool", k_pool, dt, (S, Hkv, d)), ("v_pool", v_pool, dt, (S, Hkv, d)),
                       ("out_loc", out_loc, i32, (T,)), ("qo_indptr", qo_indptr, i32, (B + 1,)),
                       ("prefix_len", prefix_len, i32, (B,))))
    rot = max_pos = p_rope = p_w = p_b = p_req = R = nb = 0
    if rope is not None:
        max_pos, rot = _dims(fn, "rope", rope, 2)
        _require(fn, dev, (("rope", rope, torch.float32, (max_pos, rot)),))
        p_rope = rope.data_ptr()
    if k_weight is not None:
        _require(fn, dev, (("k_weight", k_weight, dt, (d,)),))
        p_w = k_weight.data_ptr()
    if bounds is not None:
        if req_idx is None:
            raise ValueError(f"{fn}: bounds need req_idx")
        R, nb = _dims(fn, "bounds", bounds, 5)[:2]
        _require(fn, dev, (("bounds", bounds, dt, (R, nb, Hkv, 2, d)),
                           ("req_idx", req_idx, i32, (B,))))
        p_b, p_req = bounds.data_ptr(), req_idx.data_ptr()
    a = RcKvAppendArgs(_dtype_code(k_pool), B, Hkv, d, rot, 1 if interleaved else 0, eps, block, T, S,
                       max_pos, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, out_loc.data_ptr(),
                       qo_indptr.data_ptr(), prefix_len.data_ptr(), p_w, p_rope, k_pool.data_ptr(),
                       v_pool.data_ptr(), p_b, p_req, R, nb)
    check(lib().rc_kv_append(ctypes.byref(a), _raw_stream(dev, stream)), "rc_kv_append")


def kv_block_bounds(k_pool, req_to_token, req_idx, seq_len, bounds, *, block=64, stream=None):
    """Build the block bounds of cached contexts (see rc_kv_block_bounds): row req_idx[n]'s first
    seq_len[n] tokens. k_pool [num_slots, Hkv, d] with bounds [max_reqs, max_blocks, Hkv, 2, d], or
    both with a leading layers dimension."""
    fn = "kv_block_bounds"
    torch = _torch()
    dev = torch.cuda.current_device()
    if k_pool.dim() not in (3, 4) or bounds.dim() != k_pool.dim() + 2:
        raise ValueError(f"{fn}: k_pool and bounds must both have a layers dimension or neither")
    dt, i32 = k_pool.dtype, torch.int32
    *lead, S, Hkv, d = k_pool.shape
    R, C = _dims(fn, "req_to_token", req_to_token, 2)
    N, nb = seq_len.numel(), bounds.shape[-4]
    _require(fn, dev, (("k_pool", k_pool, dt, k_pool.shape),
                       ("bounds", bounds, dt, (*lead, R, nb, Hkv, 2, d)),
                       ("req_to_token", req_to_token, i32, (R, C)), ("seq_len", seq_len, i32, (N,)),
                       ("req_idx", req_idx, i32, (N,))))
    a = RcKvBlockBoundsArgs(_dtype_code(k_pool), lead[0] if lead else 1, N, Hkv, d, R, C, block, nb,
                            S, seq_len.data_ptr(), req_idx.data_ptr(), req_to_token.data_ptr(),
                            k_pool.data_ptr(), bounds.data_ptr())
    check(lib().rc_kv_block_bounds(ctypes.byref(a), _raw_stream(dev, stream)),
          "rc_kv_block_bounds")


def sparse_decode_workspace_bytes(q, k_pool, *, max_seq_len, block, top_blocks) -> int:
    """Workspace of sparse_decode_attention for these sizes (rc_sparse_decode_workspace_bytes)."""
    N, Hq, d = q.shape
    a = RcSparseDecodeArgs(dtype=_dtype_code(q), num_rows=N, num_q_heads=Hq,
                           num_kv_heads=k_pool.shape[1], head_dim=d, block=block,
                           max_seq_len=max_seq_len, top_blocks=top_blocks, recent_blocks=1)
    n = ctypes.c_size_t()
    check(lib().rc_sparse_decode_workspace_bytes(ctypes.byref(a), ctypes.byref(n)),
          "rc_sparse_decode_workspace_bytes")
    return int(n.value)


def sparse_decode_attention(q, seq_len, req_idx, req_to_token, k_pool, v_pool, bounds, o,
                            workspace, *, sm_scale, max_seq_len, block, top_blocks,
                            sink_blocks=1, recent_blocks=1, lse=None, selected=None, stream=None):
    """Decode attention of one layer over the blocks that their bounds select for each query row
    and KV head (see rc_sparse_decode_attention). q, o [N, Hq, d]; seq_len, req_idx [N] int32, a
    row's own token already in the pool (kv_append); bounds: this layer's block bounds
    [max_reqs, max_blocks, Hkv, 2, d]; workspace: a uint8 CUDA tensor of at least
    sparse_decode_workspace_bytes(...) bytes; lse fp32 [N, Hq] and selected int32
    [N, Hkv, top_blocks] optional."""
    fn = "sparse_decode_attention"
    torch = _torch()
    dev = torch.cuda.current_device()
    dt, i32 = q.dtype, torch.int32
    N, Hq, d = _dims(fn, "q", q, 3)
    S, Hkv, _ = _dims(fn, "k_pool", k_pool, 3)
    R, C = _dims(fn, "req_to_token", req_to_token, 2)
    nb = _dims(fn, "bounds", bounds, 5)[1]
    _require(fn, dev, (("q", q, dt, (N, Hq, d)), ("o", o, dt, (N, Hq, d)),
                       ("k_pool", k_pool, dt, (S, Hkv, d)), ("v_pool", v_pool, dt, (S, Hkv, d)),
                       ("bounds", bounds, dt, (R, nb, Hkv, 2, d)),
                       ("req_to_token", req_to_token, i32, (R, C)),
                       ("seq_len", seq_len, i32, (N,)), ("req_idx", req_idx, i32, (N,)),
                       ("workspace", workspace, torch.uint8, workspace.shape)))
    a = RcSparseDecodeArgs(_dtype_code(q), N, Hq, Hkv, d, R, C, block, nb, max_seq_len, top_blocks,
                           sink_blocks, recent_blocks, S, sm_scale, q.data_ptr(),
                           seq_len.data_ptr(), req_idx.data_ptr(), req_to_token.data_ptr(),
                           k_pool.data_ptr(), v_pool.data_ptr(), bounds.data_ptr(), o.data_ptr())
    if lse is not None:
        _require(fn, dev, (("lse", lse, torch.float32, (N, Hq)),))
        a.lse = lse.data_ptr()
    if selected is not None:
        _require(fn, dev, (("selected", selected, i32, (N, Hkv, top_blocks)),))
        a.selected = selected.data_ptr()
    check(lib().rc_sparse_decode_attention(ctypes.byref(a), workspace.data_ptr(), workspace.numel(),
                                           _raw_stream(dev, stream)), "rc_sparse_decode_attention")


def device_status(stream=None) -> int:
    """Read and clear the device status word (0 = no kernel reported bad data)."""
    v = ctypes.c_int32()
    check(lib().rc_device_status(ctypes.byref(v), _stream(stream)), "rc_device_status")
    return int(v.value)
