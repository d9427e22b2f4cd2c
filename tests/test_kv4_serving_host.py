"""Host side of an engine whose cache is held in 4 bits (CPU): the rows that an extend's cached tokens
are read back into, what a decode step appends, and what is refused before anything reaches a device."""
import numpy as np
import pytest
import torch

from prefix_cached_paged_gb300 import runtime, serving
import synth
from tests.test_sparse_serving_host import _Recorder


def _engine():
    eng = serving.Engine.__new__(serving.Engine)
    eng.host = runtime.HostCache(500, 64)
    eng.dev = _Recorder()
    eng.dev.torch, eng.dev.device = torch, torch.device("cpu")
    eng._free_rows = list(range(7, -1, -1))
    eng.max_ctx, eng.kv_chunk, eng.kv_bits, eng.dtype = 64, 0, 4, torch.float32
    eng.n_q_heads, eng.n_kv_heads, eng.head_dim, eng.sm_scale = 2, 2, 64, 0.125
    eng.share_decode = eng.stack_extend = False
    eng._tier_copies = lambda copies: None
    return eng


def test_every_cached_slot_has_one_row_and_every_new_token_one_behind_them():
    eng = _engine()
    pre = synth.tokens(3, 1, 20)
    eng.extend_end(eng.extend_begin([pre]))
    seqs = [np.concatenate([pre, synth.tokens(3, 5, 7)]).astype(np.int32), synth.tokens(3, 6, 1),
            np.concatenate([pre[:11], synth.tokens(3, 7, 2)]).astype(np.int32)]
    b = eng.extend_begin(seqs)
    x, plan = b.prefix, b.plan
    assert plan.prefix_len.tolist() == [20, 0, 11]
    U, T = len(x.slots), plan.num_tokens
    assert U == 20 and x.table.shape == (3, 28) and x.k.shape == x.v.shape == (U + T, 2, 64)
    at = 0
    for i, (P, n) in enumerate(zip(plan.prefix_len, plan.lengths)):
        assert x.slots[x.table[i, :P]].tolist() == plan.rows[i, :P].tolist()
        assert x.table[i, P:n].tolist() == [U + at + j for j in range(n - P)]
        at += n - P
    assert x.out_loc.tolist() == list(range(U, U + T)) and x.req_idx.tolist() == [0, 1, 2]
    # shared slots are one row, so runs of requests that share a prefix stay such runs
    assert x.table[0, :11].tolist() == x.table[2, :11].tolist()
    eng.extend_end(b)
    b = eng.extend_begin([])
    assert b.prefix.slots.tolist() == []
    eng.extend_end(b)


def test_a_step_appends_before_it_attends(monkeypatch):
    calls = []
    monkeypatch.setattr(serving, "kv4_append", lambda k, v, loc, ip, kp, vp:
                        calls.append(("append", k, loc.tolist(), ip.tolist())))
    monkeypatch.setattr(serving, "kv4_decode_workspace_bytes", lambda *a, **kw: 64)
    monkeypatch.setattr(serving, "kv4_decode_attention", lambda q, n, req, *a, **kw:
                        calls.append(("attend", n.tolist(), kw["max_seq_len"], a[4])))
    eng = _engine()
    seqs = [synth.tokens(3, 1, 20), synth.tokens(3, 2, 5)]
    eng.extend_end(eng.extend_begin(seqs))
    db = eng.decode_begin(seqs)
    for call in (lambda: eng.decode_layer(db, 0, None, None, None, None),
                 lambda: eng.append_layer(db, 0, None, None)):
        with pytest.raises(ValueError):
            call()                                        # no step yet
    eng.decode_step(db)
    eng.decode_layer(db, 0, None, "k", "v", None)
    assert [c[0] for c in calls] == ["append", "attend"]
    assert calls[0][1:] == ("k", db.new_slots.tolist(), [0, 1, 2])
    assert calls[1][1:3] == ([21, 6], 21)
    with pytest.raises(ValueError):                       # another layer has not been appended to
        eng.decode_layer(db, 1, None, None, None, None)
    eng.append_layer(db, 1, "k1", "v1")
    eng.decode_layer(db, 1, None, None, None, None)
    assert [c[0] for c in calls[2:]] == ["append", "attend"]
    eng.decode_step(db)
    with pytest.raises(ValueError):                       # nor this one at this step
        eng.decode_layer(db, 1, None, None, None, None)
    eng.decode_layer(db, 1, None, "k", "v", None)
    workspaces = [c[3] for c in calls if c[0] == "attend"]
    assert len({w.data_ptr() for w in workspaces}) == 3
    with pytest.raises(ValueError):
        eng.sparse_layer(db, 0, None, None, top_blocks=4)
    eng.decode_end(db)


def test_refused_engines():
    args = dict(layers=1, n_q_heads=4, n_kv_heads=1, head_dim=64, dtype=torch.float32, num_slots=512,
                max_reqs=4, max_ctx=128, device="cpu")
    for bad in (dict(kv_bits=8), dict(kv_bits=4, head_dim=96), dict(kv_bits=4, head_dim=256),
                dict(kv_bits=4, sparse_block=16), dict(kv_bits=4, host_tier_slots=64)):
        with pytest.raises(ValueError):
            serving.Engine(**{**args, **bad})
    eng = serving.Engine(**args, kv_bits=4)
    assert eng.dev.k.dtype == torch.uint8 and eng.dev.k.shape == (1, 512, 1, 40)
    assert serving.Engine(**args).dev.k.dtype == torch.float32
