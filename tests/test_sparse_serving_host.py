"""Host side of the engine's rotated and block-sparse steps (CPU): the metadata of a batch's new
tokens, which append builds bounds anew, and what is refused before anything reaches a device."""
import numpy as np
import pytest

from prefix_cached_paged_gb300 import runtime, serving
import synth


class _Recorder:
    """Stands in for the device side: uploads come back as the host arrays they were."""
    k = v = req_to_token = [None] * 4

    def write_rows(self, row_ids, rows, ends, cols=None):
        pass

    def upload_i32(self, arrays):
        return [np.ascontiguousarray(a, dtype=np.int32).ravel() for a in arrays]


def _engine(rope=True, block=16):
    eng = serving.Engine.__new__(serving.Engine)
    eng.host = runtime.HostCache(500, 64)
    eng.dev = _Recorder()
    eng._free_rows = list(range(7, -1, -1))
    eng.max_ctx, eng.kv_chunk = 64, 0
    eng.n_q_heads = eng.n_kv_heads = 2
    eng.share_decode = eng.stack_extend = False
    eng.rope = object() if rope else None
    eng.sparse_block = block
    eng.bounds = ["bounds of layer %d" % i for i in range(4)]
    eng._tier_copies = lambda copies: None
    return eng


@pytest.mark.parametrize("rope,block", [(True, 0), (False, 16), (True, 16)])
def test_positions_lengths_and_rows_of_new_tokens(rope, block):
    eng = _engine(rope, block)
    pre = synth.tokens(3, 1, 20)
    eng.extend_end(eng.extend_begin([pre]))
    seqs = [np.concatenate([pre, synth.tokens(3, 5, 7)]).astype(np.int32), synth.tokens(3, 6, 1),
            np.concatenate([pre[:11], synth.tokens(3, 7, 2)]).astype(np.int32)]
    b = eng.extend_begin(seqs)
    want = [(r, p) for r, P, n in zip(b.row_ids, b.plan.prefix_len, b.plan.lengths)
            for p in range(P, n)]
    assert [int(x) for x in b.plan.prefix_len] == [20, 0, 11] and b.max_len == 27
    assert b.token_pos.tolist() == [p for _, p in want]
    assert b.token_len.tolist() == [p + 1 for _, p in want]
    assert b.token_row.tolist() == [r for r, _ in want]
    eng.extend_end(b)
    db = eng.decode_begin([seqs[0], seqs[1]])
    assert db.token_pos is None and db.steps == 0
    for step in range(2):
        eng.decode_step(db)
        assert db.token_pos.tolist() == [27 + step, 1 + step] and db.steps == step + 1
        assert db.dev_seq_len.tolist() == [28 + step, 2 + step]
        assert db.one_each.tolist() == [0, 1, 2]
    eng.decode_end(db)
    eng = _engine(False, 0)
    b = eng.extend_begin([pre])
    assert b.token_pos is None and b.token_len is None
    with pytest.raises(ValueError):
        eng.norm_rope(b, None)


def test_bounds_are_built_once_and_again_where_a_step_was_missed(monkeypatch):
    calls = []
    monkeypatch.setattr(serving, "kv_block_bounds", lambda k, t, req, n, bounds, block:
                        calls.append(("build", bounds, n.tolist())))
    monkeypatch.setattr(serving, "kv_append", lambda *a, **kw:
                        calls.append(("append", kw["bounds"], kw["rope"] is not None)))
    eng = _engine()
    seq = synth.tokens(3, 1, 20)
    b = eng.extend_begin([seq])
    for _ in range(2):                      # a repeated append builds nothing again
        eng.append_layer(b, 1, None, None)
    assert calls == [("build", "bounds of layer 1", [0]), ("append", "bounds of layer 1", True),
                     ("append", "bounds of layer 1", True)]
    with pytest.raises(ValueError):         # another layer has not been appended to
        eng.sparse_layer(b, 2, None, None, top_blocks=4)
    eng.extend_end(b)
    db = eng.decode_begin([seq])
    with pytest.raises(ValueError):
        eng.append_layer(db, 0, None, None)     # no step yet
    log = []
    for step in range(5):
        eng.decode_step(db)
        calls.clear()
        if step != 2:                       # step 2 goes by dense attention alone
            eng.append_layer(db, 0, None, None, rotate=False)
            eng.append_layer(db, 0, None, None, rotate=False)
        else:
            with pytest.raises(ValueError):
                eng.sparse_layer(db, 0, None, None, top_blocks=4)
        log.append([c[0] for c in calls])
        assert all(not c[2] for c in calls if c[0] == "append")
        assert all(c[2] == [20 + step] for c in calls if c[0] == "build")
    assert log == [["build", "append", "append"], ["append"] * 2, [],
                   ["build", "append", "append"], ["append"] * 2]
    eng.decode_end(db)
    eng.sparse_block = 0
    with pytest.raises(ValueError):
        eng.sparse_layer(db, 0, None, None, top_blocks=4)


def test_empty_batches_have_metadata():
    eng = _engine()
    b = eng.extend_begin([])
    assert b.num_tokens == 0 and b.token_pos.tolist() == [] and b.max_len == 0
    eng.extend_end(b)


def test_every_sparse_call_has_a_workspace_of_its_own(monkeypatch):
    """A captured call goes on using the workspace it was captured with, so no later call may have
    the same one, or have it replaced by a larger one and freed."""
    import torch
    need, used = [64], []
    monkeypatch.setattr(serving, "kv_block_bounds", lambda *a, **kw: None)
    monkeypatch.setattr(serving, "kv_append", lambda *a, **kw: None)
    monkeypatch.setattr(serving, "sparse_decode_workspace_bytes", lambda *a, **kw: need[0])
    monkeypatch.setattr(serving, "sparse_decode_attention", lambda *a, **kw: used.append(a[8]))
    eng = _engine()
    eng.dev.torch, eng.dev.device = torch, torch.device("cpu")
    eng.sm_scale = 1.0
    b = eng.extend_begin([synth.tokens(3, 1, 20)])
    eng.append_layer(b, 0, None, None)
    for n in (64, 64, 32, 128, 0):
        need[0] = n
        eng.sparse_layer(b, 0, None, None, top_blocks=4)
        assert used[-1].dtype == torch.uint8 and used[-1].numel() >= n
    assert len({w.data_ptr() for w in used[:4]}) == 4
