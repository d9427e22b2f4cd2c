"""One model's prefix-cached paged attention state and its per-step calls.

`Engine` ties the host pool and radix tree (HostCache) to the device KV planes and slot table
(DeviceKV) and exposes the steps a scheduler runs, each a composition of librc calls:

  extend_begin   plan a batch (match + lock, evict if short, allocate), write each request's slot
                 row into the device slot table and upload the kernel metadata;
  extend_layer   extend attention of one layer (scatters the new K/V into the pool);
  extend_end     insert the sequences, free duplicate slots, unlock, release slot-table rows;
  decode_begin   requests enter decoding: match their cached context, lock it, take a row;
  decode_step    allocate one slot per request for its new token and write it to the row;
  decode_layer   split-K decode attention of one layer;
  decode_end     insert the finished sequences (context + generated tokens) or free the generated
                 tokens' slots, unlock, release rows.

Between a model's projections and attention, at a batch's positions (an extend or a decode batch):

  norm_rope      norms of queries and keys for each head and the position rotation (the engine's
                 `rope` table), in place or into given tensors;
  append_layer   append one layer's new K/V to the cache (norm and rotation on the way, if wanted)
                 and, with `sparse_block`, extend the block bounds of the batch's rows;
  sparse_layer   attention of one layer over the blocks that the bounds select for each query and
                 KV head, after append_layer: decode steps, and short chunks of new tokens.

With kv_bits=4 the cache is held in 4 bits (kv4_append): the same steps, append_layer and norm_rope
among them, on a pool of 5 / 16 of the bf16 bytes. New tokens of an extend attend to each other as
given and to the cached prefix as it is held, read back once per layer into rows of the batch; later
steps see them as they are held too.

The model's projections (q, k_new, v_new per layer) are the caller's: this module never
computes them.
"""
from __future__ import annotations

from contextlib import contextmanager
from dataclasses import dataclass, field

import numpy as np

from . import (DEFAULT_KV_CHUNK, decode_attention, decode_workspace_bytes, extend_attention,
               extend_workspace_bytes, kv4_append, kv4_decode_attention, kv4_decode_workspace_bytes,
               kv4_read, kv4_row_bytes, kv_append, kv_block_bounds, kv_copy, plan_extend_stacking,
               qk_norm_rope, shared_context_groups, sparse_decode_attention,
               sparse_decode_workspace_bytes, MAX_STACK_LEVELS)
from .runtime import DeviceKV, HostCache, Plan


@dataclass
class ExtendBatch:
    plan: Plan
    row_ids: np.ndarray
    qo_indptr: object      # device int32 [B+1]
    prefix_len: object     # device int32 [B]
    req_idx: object        # device int32 [B]
    out_loc: object        # device int32 [T]
    max_q_len: int
    max_prefix_len: int
    stack: object = None       # (device ranges, device shared, max_group_rows) or None
    workspace: object = None   # device scratch of the stacked pass
    token_pos: object = None   # device int32 [T]: position of each new token (see Engine.rope)
    token_len: object = None   # device int32 [T]: position + 1, what its query may see
    token_row: object = None   # device int32 [T]: its request's slot-table row
    max_len: int = 0           # longest request
    bounded: set = field(default_factory=set)   # layers whose bounds hold the new tokens
    prefix: object = None      # the cached tokens of a 4-bit cache, as numbers (Engine._stage)

    @property
    def num_tokens(self) -> int:
        return self.plan.num_tokens


@dataclass
class Prefix:
    """The cached tokens that an extend batch over a 4-bit cache attends to, each once, in rows 0 ..;
    behind them a row per new token."""
    slots: object      # device int32 [U]: the cached tokens' slots
    table: object      # device int32 [B, columns]: the rows' counterpart of the slot table
    req_idx: object    # device int32 [B]: 0, 1, ..
    out_loc: object    # device int32 [T]: U, U + 1, ..
    k: object          # [U + T, Hkv, d], the layer in hand
    v: object


@dataclass
class DecodeBatch:
    row_ids: np.ndarray
    nodes: np.ndarray      # locked context nodes
    seq_len: np.ndarray    # host int32 [B], including the current new token
    new_slots: np.ndarray  # host int32 [B], slots of the current new tokens
    dev_seq_len: object = None
    dev_req_idx: object = None
    dev_out_loc: object = None
    groups: object = None   # device (indptr, members, shared) of shared-context groups, or None
    num_groups: int = 0
    step_id: object = None  # identity of the current step's lengths (a fresh object per step)
    context_rows: object = None  # host int32 [B, max_ctx]: each context's slots (decode_begin)
    context_len: object = None   # host int64 [B]
    gen_slots: list = None       # host int32 [B] per decode_step: the generated tokens' slots
    steps: int = 0               # decode_steps taken
    token_pos: object = None     # device int32 [B]: position of the step's new tokens
    one_each: object = None      # device int32 [B + 1]: 0, 1, .. B
    bounded: dict = field(default_factory=dict)   # layer -> steps whose tokens its bounds hold (with
                                                  # kv_bits=4: the last step appended)


# shortest shared prefix worth a stacked pass: two key tiles
STACK_MIN_SHARED = 256


class Engine:
    rope = None        # fp32 table [positions, rotary_dim] on the device, or None
    sparse_block = 0   # positions per block of the bounds, 0: none are kept
    bounds = None      # [layers, max_reqs, blocks, Hkv, 2, d]
    kv_bits = 16       # 4: the cache is held in 4 bits; 16: in the engine's dtype
    _no_workspace = None

    def __init__(self, layers, n_q_heads, n_kv_heads, head_dim, dtype, num_slots, max_reqs,
                 max_ctx, initial_order=None, device="cuda", kv_chunk=0, share_decode=True,
                 stack_extend=True, host_tier_slots=0, host_planes=None,
                 stack_levels=MAX_STACK_LEVELS, fold_extend=True, rope=None, sparse_block=0, kv_bits=16):
        if kv_bits not in (4, 16):
            raise ValueError("kv_bits must be 16 (the cache in dtype) or 4")
        if kv_bits == 4 and head_dim not in (64, 128):
            raise ValueError("kv_bits=4 attends to heads of 64 or 128")
        if kv_bits == 4 and (n_q_heads % n_kv_heads or n_q_heads > 16 * n_kv_heads):
            raise ValueError("kv_bits=4 attends with up to 16 query heads for each KV head")
        if kv_bits == 4 and sparse_block:
            raise ValueError("kv_bits=4 keeps no block bounds: sparse_block must be 0")
        if kv_bits == 4 and host_tier_slots and n_kv_heads * kv4_row_bytes(head_dim) % 16:
            raise ValueError("kv_bits=4 with a host tier needs slots of a multiple of 16 bytes: an "
                             "even number of KV heads of 64")
        self.kv_bits, self.dtype = int(kv_bits), dtype
        self.layers = layers
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.sm_scale = 1.0 / float(np.sqrt(head_dim))
        self.host = HostCache(num_slots, max_ctx, initial_order, host_slots=host_tier_slots)
        if self.kv_bits == 4:
            import torch
            row, dtype = kv4_row_bytes(head_dim), torch.uint8
        else:
            row = head_dim
        self.dev = DeviceKV(layers, num_slots, n_kv_heads, row, dtype, max_reqs, max_ctx, device)
        self.host_k = self.host_v = None
        if host_tier_slots:
            # the host tier's KV planes: pinned host memory the kernels address directly
            # (host_planes: a caller's (k, v) pair of that shape, reused across engines)
            torch = self.dev.torch
            shape = (layers, host_tier_slots, n_kv_heads, row)
            if host_planes is not None:
                self.host_k, self.host_v = host_planes
                if tuple(self.host_k.shape) != shape or not self.host_k.is_pinned():
                    raise ValueError(f"host_planes must be pinned tensors of shape {shape}")
            else:
                self.host_k = torch.empty(shape, dtype=dtype, pin_memory=True)
                self.host_v = torch.empty(shape, dtype=dtype, pin_memory=True)
        # rope: the rotation's fp32 table [positions, rotary_dim] (rope_table), at least max_ctx
        # positions, for norm_rope and append_layer
        if rope is not None:
            self.rope = self.dev.torch.as_tensor(rope, device=self.dev.device).contiguous()
            if self.rope.dtype != self.dev.torch.float32 or self.rope.dim() != 2 or \
                    self.rope.shape[0] < max_ctx:
                raise ValueError(f"rope must be an fp32 table of at least {max_ctx} positions")
        # sparse_block: positions per block of the bounds that sparse_layer selects blocks by
        # (16, 32, 64 or 128; 0: no bounds are kept). They take two elements per block, KV head and
        # dimension of every slot-table row, used or not: 2 / sparse_block of the keys that full rows
        # would hold (32 layers, 256 rows of 131072 positions, 8 KV heads of 128 in bf16, blocks of
        # 64: 64 GiB). A prefix that rows share has its bounds in each of them, built per batch.
        self.sparse_block = int(sparse_block)
        if self.sparse_block:
            if self.sparse_block not in (16, 32, 64, 128):
                raise ValueError("sparse_block must be 0, 16, 32, 64 or 128")
            nb = -(-max_ctx // self.sparse_block)
            self.bounds = self.dev.torch.empty((layers, max_reqs, nb, n_kv_heads, 2, head_dim),
                                               dtype=dtype, device=self.dev.device)
        self.max_ctx = max_ctx
        self.kv_chunk = kv_chunk
        # decode reads a context prefix that several requests share once for all of them; with
        # kv_bits=4 once for each of them, whatever this says
        self.share_decode = share_decode
        # extend stacks the new tokens of consecutive requests over a prefix they share, where
        # that is estimated to pay (True), for every group found ("always"), or never (False)
        self.stack_extend = stack_extend
        self.stack_levels = stack_levels   # tree levels stacked (1: the shallowest group only)
        # an innermost stacked group takes its members' remainders in its own pass where that is
        # estimated to pay (True), always ("always"), or never (False)
        self.fold_extend = fold_extend
        self._ext_ws = None
        self._free_rows = list(range(max_reqs - 1, -1, -1))
        self._ws = None
        self._ws_plan = None   # (step id, workspace address, token bound) of the plan in _ws

    def _tier_copies(self, copies):
        """Perform the host tier's owed copies on the stream: spills (device -> host) before
        loads (host -> device), both before any later kernel that writes a recycled slot."""
        if copies is None:
            return
        sd, sh, lh, ld = copies
        if len(sd) == 0 and len(lh) == 0:
            return
        d_sd, d_sh, d_lh, d_ld = self.dev.upload_i32([sd, sh, lh, ld])
        if len(sd):
            kv_copy(self.dev.k, self.dev.v, d_sd, self.host_k, self.host_v, d_sh)
        if len(lh):
            kv_copy(self.host_k, self.host_v, d_lh, self.dev.k, self.dev.v, d_ld)

    # ---------------------------------------------------------------- rows
    def _check_rows(self, n):
        if n > len(self._free_rows):
            raise RuntimeError(f"slot table has {len(self._free_rows)} free rows, {n} needed")

    def _take_rows(self, n):
        self._check_rows(n)
        return np.array([self._free_rows.pop() for _ in range(n)], dtype=np.int32)

    def _release_rows(self, rows):
        self._free_rows.extend(int(r) for r in rows[::-1])

    # ---------------------------------------------------------------- extend
    def _owed_copies(self):
        """Host-tier copies a failed call left owed: on the stream first. Those that fail now are
        still owed."""
        owed = self.host.take_owed()
        try:
            while owed:
                self._tier_copies(owed[0])
                owed.pop(0)
        finally:
            self.host.owe(owed)

    @contextmanager
    def _begin(self, plan: Plan):
        """What a batch does on the device to begin, its plan's host-tier copies first. If any of it
        fails, the plan's slots and locks and the rows taken go back, and copies not made are owed."""
        rows, owed = list(self._free_rows), plan.copies
        try:
            self._tier_copies(owed)
            owed = None
            yield
        except BaseException:
            self._free_rows[:] = rows
            self.host.cancel(plan, owed)
            raise

    def extend_begin(self, seqs, extra: int = 0, match_all: bool = False) -> ExtendBatch:
        self._check_rows(len(seqs))
        self._owed_copies()
        plan = self.host.plan(seqs, extra=extra, match_all=match_all)
        with self._begin(plan):
            return self._extend_batch(plan)

    def _extend_batch(self, plan: Plan) -> ExtendBatch:
        B = len(plan.lengths)
        row_ids = self._take_rows(B)
        self.dev.write_rows(row_ids, plan.rows, plan.lengths)
        qo, pl, ri, ol = self.dev.upload_i32([plan.qo_indptr, plan.prefix_len, row_ids,
                                              plan.out_loc])
        S = plan.lengths - plan.prefix_len
        batch = ExtendBatch(plan, row_ids, qo, pl, ri, ol, int(S.max()) if B else 0,
                            int(plan.prefix_len.max()) if B else 0,
                            max_len=int(plan.lengths.max()) if B else 0)
        if self.rope is not None or self.sparse_block:
            T = plan.num_tokens
            pos = np.arange(T) - np.repeat(plan.qo_indptr[:-1] - plan.prefix_len, S)
            batch.token_pos, batch.token_len, batch.token_row = self.dev.upload_i32(
                [pos, pos + 1, np.repeat(row_ids, S)])
        if self.kv_bits == 4:
            batch.prefix = self._stage(batch)
        if self.stack_extend and B > 1:
            # stacking groups over the levels of the tree, each kept where it is estimated to pay
            G = self.n_q_heads // self.n_kv_heads
            ranges, shared, start, level_indptr, max_rows, fold, all_folded = plan_extend_stacking(
                plan.rows, plan.prefix_len, S, STACK_MIN_SHARED, G, self.stack_levels,
                policy="all" if self.stack_extend == "always" else "cost",
                fold=self.fold_extend)
            if len(shared):
                r, sh, st, fo = self.dev.upload_i32([ranges, shared, start, fold])
                batch.stack = (r, sh, max_rows, st, level_indptr, fo, all_folded)
                need = extend_workspace_bytes(plan.num_tokens, self.n_q_heads)
                if self._ext_ws is None or self._ext_ws.numel() < need:
                    self._ext_ws = self.dev.torch.empty(need, dtype=self.dev.torch.uint8,
                                                        device=self.dev.device)
                batch.workspace = self._ext_ws
        return batch

    def _stage(self, batch: ExtendBatch) -> Prefix:
        """Rows for a batch's cached tokens as numbers and its new tokens, and the slot table's
        counterpart over them. Slots that requests share are one row, so stacking groups hold."""
        plan = batch.plan
        P, B, T = plan.prefix_len, len(plan.lengths), plan.num_tokens
        slots = np.unique(np.concatenate([plan.rows[b, :P[b]] for b in range(B)] +
                                         [np.zeros(0, np.int32)]))
        U = len(slots)
        cols = -(-max(batch.max_len, 1) // 4) * 4
        table = np.zeros((max(B, 1), cols), np.int32)
        for b in range(B):
            table[b, :P[b]] = np.searchsorted(slots, plan.rows[b, :P[b]])
            table[b, P[b]:plan.lengths[b]] = U + np.arange(plan.qo_indptr[b], plan.qo_indptr[b + 1])
        d_slots, d_table, d_req, d_loc = self.dev.upload_i32(
            [slots, table, np.arange(B), U + np.arange(T)])
        shape = (max(U + T, 1), self.n_kv_heads, self.head_dim)
        k, v = (self.dev.torch.empty(shape, dtype=self.dtype, device=self.dev.device)
                for _ in range(2))
        return Prefix(d_slots, d_table.reshape(table.shape), d_req, d_loc, k, v)

    def extend_layer(self, batch: ExtendBatch, layer: int, q, k_new, v_new, o, lse=None):
        if self.kv_bits == 4:
            x = batch.prefix
            kv4_read(self.dev.k[layer], self.dev.v[layer], x.slots, x.k, x.v)
            extend_attention(q, k_new, v_new, x.out_loc, batch.qo_indptr, batch.prefix_len,
                             x.req_idx, x.table, x.k, x.v, o, sm_scale=self.sm_scale,
                             max_q_len=batch.max_q_len, max_prefix_len=batch.max_prefix_len, lse=lse,
                             stack=batch.stack, workspace=batch.workspace)
            kv4_append(k_new, v_new, batch.out_loc, batch.qo_indptr, self.dev.k[layer],
                       self.dev.v[layer])
            return
        extend_attention(q, k_new, v_new, batch.out_loc, batch.qo_indptr, batch.prefix_len,
                         batch.req_idx, self.dev.req_to_token, self.dev.k[layer],
                         self.dev.v[layer], o, sm_scale=self.sm_scale,
                         max_q_len=batch.max_q_len, max_prefix_len=batch.max_prefix_len, lse=lse,
                         stack=batch.stack, workspace=batch.workspace)

    def extend_end(self, batch: ExtendBatch, keep_locked: bool = False):
        ends, dups = self.host.finish(batch.plan, keep_locked=keep_locked)
        self._release_rows(batch.row_ids)
        return ends, dups

    # ---------------------------------------------------------------- decode
    def decode_begin(self, contexts) -> DecodeBatch:
        """Requests enter decoding: each context must be cached; it is matched and locked, its
        slots written to a fresh slot-table row. The first decode_step allocates the new tokens."""
        self._check_rows(len(contexts))
        self._owed_copies()
        plan = self.host.plan(contexts, match_all=True)
        with self._begin(plan):
            if plan.num_tokens:
                raise ValueError("decode_begin: every context must already be cached")
            return self._decode_batch(plan)

    def _decode_batch(self, plan: Plan) -> DecodeBatch:
        row_ids = self._take_rows(len(plan.lengths))
        self.dev.write_rows(row_ids, plan.rows, plan.lengths)
        self._decode_plan = plan
        batch = DecodeBatch(row_ids, plan.nodes, plan.lengths.astype(np.int32),
                            np.zeros(len(plan.lengths), np.int32), context_rows=plan.rows,
                            context_len=plan.lengths.astype(np.int64), gen_slots=[])
        if self.share_decode and self.kv_bits != 4:
            # the contexts' slots never change while they decode (new tokens get new slots), so
            # the groups hold for the whole batch
            G = self.n_q_heads // self.n_kv_heads
            indptr, members, shared = shared_context_groups(
                plan.rows, plan.lengths, 8 // G, self.kv_chunk or DEFAULT_KV_CHUNK)
            if len(shared):
                batch.groups = tuple(self.dev.upload_i32([indptr, members, shared]))
                batch.num_groups = len(shared)
        return batch

    def decode_step(self, batch: DecodeBatch, new_slots=None) -> DecodeBatch:
        """Append one token per request: allocate its slot (evicting if needed) unless given,
        write it to the request's row at position seq_len, and upload the step's metadata."""
        B = len(batch.row_ids)
        self._owed_copies()
        if new_slots is None:
            new_slots = self.host.alloc(B)
            self._tier_copies(self.host.last_alloc_copies)
        cols = batch.seq_len.astype(np.int64)
        rows = np.zeros((B, self.max_ctx), dtype=np.int32)
        rows[np.arange(B), cols] = new_slots
        self.dev.write_rows(batch.row_ids, rows, cols + 1, cols=cols)
        batch.seq_len = batch.seq_len + 1
        batch.new_slots = np.asarray(new_slots, dtype=np.int32)
        if batch.gen_slots is not None:
            batch.gen_slots.append(batch.new_slots.copy())
        batch.step_id = object()   # the lengths changed: the next layer plans again
        meta = [batch.seq_len, batch.row_ids, batch.new_slots]
        if self.rope is not None or self.sparse_block or self.kv_bits == 4:
            meta += [cols, np.arange(B + 1)]
        batch.dev_seq_len, batch.dev_req_idx, batch.dev_out_loc, *more = self.dev.upload_i32(meta)
        if more:
            batch.token_pos, batch.one_each = more
        batch.steps += 1
        return batch

    def workspace(self, q, k_new, max_total_tokens):
        need = decode_workspace_bytes(q, k_new, self.dev.req_to_token, self.dev.k[0],
                                      max_total_tokens=max_total_tokens, kv_chunk=self.kv_chunk)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self.dev.torch.empty(need, dtype=self.dev.torch.uint8,
                                            device=self.dev.device)
        return self._ws

    def decode_layer(self, batch: DecodeBatch, layer: int, q, k_new, v_new, o, lse=None,
                     max_total_tokens=None):
        """Decode attention of one layer over each request's whole context, its new token's k_new
        and v_new appended. With kv_bits=4 they may be None where append_layer of this layer and
        step has written them; max_total_tokens says nothing there."""
        if self.kv_bits == 4:
            if batch.one_each is None:
                raise ValueError("decode_layer: no decode_step has been taken")
            if k_new is not None:
                kv4_append(k_new, v_new, batch.dev_out_loc, batch.one_each, self.dev.k[layer],
                           self.dev.v[layer])
                batch.bounded[layer] = batch.steps
            elif batch.bounded.get(layer, -1) != batch.steps:
                raise ValueError(f"decode_layer: without keys and values, append_layer of layer "
                                 f"{layer} comes first")
            longest = int(batch.seq_len.max()) if len(batch.seq_len) else 0
            need = kv4_decode_workspace_bytes(q, self.dev.k[layer], max_seq_len=longest)
            # of this call alone, as sparse_layer's
            ws = self.dev.torch.empty(need, dtype=self.dev.torch.uint8, device=self.dev.device)
            kv4_decode_attention(q, batch.dev_seq_len, batch.dev_req_idx, self.dev.req_to_token,
                                 self.dev.k[layer], self.dev.v[layer], o, ws, sm_scale=self.sm_scale,
                                 max_seq_len=longest, lse=lse)
            return
        mt = int(batch.seq_len.sum()) if max_total_tokens is None else max_total_tokens
        ws = self.workspace(q, k_new, mt)
        # every layer of a step has the same requests and lengths: the first plans, the others
        # reuse its job list (same workspace, same bound)
        key = (batch.step_id, ws.data_ptr(), mt)
        reuse = batch.step_id is not None and self._ws_plan is not None and \
            self._ws_plan[0] is key[0] and self._ws_plan[1:] == key[1:]
        decode_attention(q, k_new, v_new, batch.dev_out_loc, batch.dev_seq_len,
                         batch.dev_req_idx, self.dev.req_to_token, self.dev.k[layer],
                         self.dev.v[layer], o, ws, sm_scale=self.sm_scale, max_total_tokens=mt,
                         kv_chunk=self.kv_chunk, lse=lse, groups=batch.groups,
                         reuse_plan=reuse)
        self._ws_plan = key     # the workspace now holds this step's plan

    # ---------------------------------------------------------------- norms, rotation, sparse
    def _metadata(self, batch, what):
        if batch.token_pos is None:
            raise ValueError(f"{what}: the engine was made without rope and sparse_block, or no "
                             "decode_step has been taken")

    def norm_rope(self, batch, q=None, k=None, *, q_weight=None, k_weight=None, eps=1e-6,
                  interleaved=False, q_out=None, k_out=None):
        """Norms of q [T, Hq, d] and k [T, Hkv, d] for each head (with the given weights) and, if
        the engine has a rope table, their rotation to the positions of the batch's new tokens; in
        place unless q_out / k_out are given (qk_norm_rope)."""
        self._metadata(batch, "norm_rope")
        qk_norm_rope(q, k, batch.token_pos if self.rope is not None else None, self.rope,
                     q_weight=q_weight, k_weight=k_weight, eps=eps, interleaved=interleaved,
                     q_out=q_out, k_out=k_out)

    def append_layer(self, batch, layer: int, k, v, *, rotate=True, k_weight=None, eps=1e-6,
                     interleaved=False):
        """Append the new tokens' k and v [T, Hkv, d] of one layer to the cache (kv_append). rotate:
        the keys are rotated by the engine's table on the way (False for keys that norm_rope has
        rotated already). With sparse_block the layer's block bounds follow; a batch's first append
        of a layer, and one after steps that only decode_layer has written, builds the bounds of
        what is cached from the cache first. With kv_bits=4 the keys are normalised and rotated in a
        pass of their own, rounded to their type and quantised with the values."""
        if self.kv_bits == 4:
            self._append4(batch, layer, k, v, rotate and self.rope is not None, k_weight, eps,
                          interleaved)
            return
        self._metadata(batch, "append_layer")
        if isinstance(batch, DecodeBatch):
            loc, ip, pre, req = batch.dev_out_loc, batch.one_each, batch.token_pos, \
                batch.dev_req_idx
            current = batch.bounded.get(layer, -1) >= batch.steps - 1
        else:
            loc, ip, pre, req = batch.out_loc, batch.qo_indptr, batch.prefix_len, batch.req_idx
            current = layer in batch.bounded
        bounds = None
        if self.sparse_block:
            bounds = self.bounds[layer]
            if not current:
                kv_block_bounds(self.dev.k[layer], self.dev.req_to_token, req, pre, bounds,
                                block=self.sparse_block)
        kv_append(k, v, loc, ip, pre, self.dev.k[layer], self.dev.v[layer],
                  rope=self.rope if rotate else None, k_weight=k_weight, eps=eps,
                  interleaved=interleaved, bounds=bounds,
                  req_idx=req if self.sparse_block else None, block=self.sparse_block or 64)
        if isinstance(batch, DecodeBatch):
            batch.bounded[layer] = batch.steps
        else:
            batch.bounded.add(layer)

    def _append4(self, batch, layer, k, v, rotate, k_weight, eps, interleaved):
        decode = isinstance(batch, DecodeBatch)
        if decode and batch.one_each is None:
            raise ValueError("append_layer: no decode_step has been taken")
        if rotate or k_weight is not None:
            given, k = k, self.dev.torch.empty(tuple(k.shape), dtype=k.dtype, device=k.device)
            qk_norm_rope(None, given, batch.token_pos if rotate else None,
                         self.rope if rotate else None, k_weight=k_weight, eps=eps,
                         interleaved=interleaved, k_out=k)
        loc, ip = (batch.dev_out_loc, batch.one_each) if decode else (batch.out_loc, batch.qo_indptr)
        kv4_append(k, v, loc, ip, self.dev.k[layer], self.dev.v[layer])
        if decode:
            batch.bounded[layer] = batch.steps

    def sparse_layer(self, batch, layer: int, q, o, *, top_blocks, sink_blocks=1, recent_blocks=1,
                     lse=None, selected=None):
        """Attention of one layer over the blocks selected for each query row and KV head
        (sparse_decode_attention): a decode batch's new tokens, or every new token of an extend
        batch, each seeing what its position may. append_layer of this layer and step comes
        first."""
        if not self.sparse_block:
            raise ValueError("sparse_layer: the engine was made without sparse_block")
        self._metadata(batch, "sparse_layer")
        if isinstance(batch, DecodeBatch):
            length, row, longest = batch.dev_seq_len, batch.dev_req_idx, int(batch.seq_len.max()) \
                if len(batch.seq_len) else 0
            current = batch.bounded.get(layer, -1) == batch.steps
        else:
            length, row, longest = batch.token_len, batch.token_row, batch.max_len
            current = layer in batch.bounded
        if not current:
            raise ValueError(f"sparse_layer: append_layer of layer {layer} comes first")
        need = sparse_decode_workspace_bytes(q, self.dev.k[layer], max_seq_len=longest,
                                             block=self.sparse_block, top_blocks=top_blocks)
        # of this call alone: a captured call keeps the memory it was captured with, and calls on
        # other streams may overlap
        ws = self._no_workspace
        if need or ws is None:
            ws = self.dev.torch.empty(need, dtype=self.dev.torch.uint8, device=self.dev.device)
        if need == 0:
            self._no_workspace = ws   # of 0 bytes: most calls need none
        sparse_decode_attention(q, length, row, self.dev.req_to_token, self.dev.k[layer],
                                self.dev.v[layer], self.bounds[layer], o, ws,
                                sm_scale=self.sm_scale, max_seq_len=longest,
                                block=self.sparse_block, top_blocks=top_blocks,
                                sink_blocks=sink_blocks, recent_blocks=recent_blocks, lse=lse,
                                selected=selected)

    def decode_end(self, batch: DecodeBatch, seqs=None):
        """The requests leave decoding. With `seqs` (each request's context followed by the
        tokens its decode steps fed in, one per step), the sequences are inserted into the tree
        like a finished extend (the generated tokens' KV stays cached; slots of tokens the tree
        already holds are freed); without, the generated tokens' slots return to the pool. Then
        the contexts are unlocked and the slot-table rows released."""
        B = len(batch.row_ids)
        gen = (np.stack(batch.gen_slots, axis=1) if batch.gen_slots
               else np.zeros((B, 0), dtype=np.int32))
        if seqs is not None:
            seqs = [np.asarray(s, dtype=np.int32) for s in seqs]
            want = batch.context_len + gen.shape[1]
            if len(seqs) != B or any(len(s) != int(n) for s, n in zip(seqs, want)):
                raise ValueError("decode_end: each sequence must be its context plus one token "
                                 f"per decode step ({gen.shape[1]})")
            lengths = want.astype(np.int64)
            indptr = np.zeros(B + 1, dtype=np.int64)
            np.cumsum(lengths, out=indptr[1:])
            rows = np.array(batch.context_rows, dtype=np.int32, copy=True)
            for b in range(B):
                rows[b, batch.context_len[b]:lengths[b]] = gen[b]
            empty = np.zeros(0, dtype=np.int32)
            self.host.finish(Plan(np.concatenate(seqs) if B else empty, indptr, lengths,
                                  batch.context_len.astype(np.int32), batch.nodes, rows,
                                  empty, empty, empty))
        else:
            if gen.size:
                self.host.pool.free(gen.reshape(-1))
            for n in batch.nodes:
                self.host.tree.unlock(int(n))
        self._release_rows(batch.row_ids)
