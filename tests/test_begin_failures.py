"""A batch whose device side cannot begin (an allocation or a transfer fails after its plan) leaves slots, locks
and slot-table rows as they were, and owed host-tier copies to the next call. CPU only: the device side is a
recorder that fails at a chosen call."""
import numpy as np
import pytest
import torch

from prefix_cached_paged_gb300 import runtime, serving
import synth
from tests.test_kv4_serving_host import _engine as _engine4
from tests.test_sparse_serving_host import _Recorder, _engine as _engine16


class _Failing(_Recorder):
    """Counts device calls; the one numbered `at` runs out of memory."""

    def __init__(self):
        self.at, self.calls, self.device = -1, 0, torch.device("cpu")
        self.torch = self

    def step(self):
        self.calls += 1
        if self.calls - 1 == self.at:
            raise torch.OutOfMemoryError("out of memory")

    def write_rows(self, *a, **kw):
        self.step()

    def upload_i32(self, arrays):
        self.step()
        return super().upload_i32(arrays)

    uint8 = torch.uint8

    def empty(self, *a, **kw):
        self.step()
        return torch.empty(*a, **kw)


def _state(eng):
    s = eng.host.tree.stats()
    return (list(eng._free_rows), eng.host.pool.available(), s["protected_tokens"],
            s["evictable_tokens"], s["nodes"])


def _engines():
    four, sixteen = _engine4(), _engine16(True, 16)
    four.rope = object()
    sixteen.kv_bits = 16
    stacked = _engine16(False, 0)
    stacked.stack_extend, stacked.stack_levels, stacked.fold_extend = "always", 4, True
    stacked.share_decode, stacked._ext_ws = True, None
    return {"4 bits": four, "bounds": sixteen, "stacked": stacked}


@pytest.mark.parametrize("kind", ["4 bits", "bounds", "stacked"])
def test_nothing_is_kept_by_a_batch_that_did_not_begin(kind, monkeypatch):
    monkeypatch.setattr(serving, "STACK_MIN_SHARED", 8)
    eng = _engines()[kind]
    eng.dev = _Failing()
    pre = synth.tokens(3, 1, 20)
    eng.extend_end(eng.extend_begin([pre]))
    seqs = [np.concatenate([pre, synth.tokens(3, 5 + i, 5 + 3 * i)]).astype(np.int32)
            for i in range(3)]
    before = _state(eng)
    eng.dev.at, eng.dev.calls, fails = 0, 0, 0
    while True:
        try:
            batch = eng.extend_begin(seqs)
            break
        except torch.OutOfMemoryError:
            assert _state(eng)[:4] == before[:4], eng.dev.at
            eng.dev.at, eng.dev.calls, fails = eng.dev.at + 1, 0, fails + 1
    assert fails >= (5 if kind == "4 bits" else 3)    # every device call of a beginning failed once
    assert batch.plan.prefix_len.tolist() == [20, 20, 20]
    eng.extend_end(batch)
    before = _state(eng)
    eng.dev.at, eng.dev.calls, fails = 0, 0, 0
    while True:
        try:
            batch = eng.decode_begin(seqs)
            break
        except torch.OutOfMemoryError:
            assert _state(eng) == before, eng.dev.at
            eng.dev.at, eng.dev.calls, fails = eng.dev.at + 1, 0, fails + 1
    assert fails >= 1 and batch.seq_len.tolist() == [len(s) for s in seqs]
    eng.dev.at = -1
    eng.decode_end(batch)
    assert _state(eng) == before
    with pytest.raises(ValueError):
        eng.decode_begin([synth.tokens(3, 90, 9)])
    assert _state(eng)[:4] == before[:4]


def test_owed_tier_copies_of_a_failed_beginning_are_made_by_the_next():
    eng = _engine4()
    eng.host = runtime.HostCache(60, 64, host_slots=200)
    made, fail = [], [False]

    def tier_copies(copies):
        if copies is None:
            return
        if fail[0]:
            raise torch.OutOfMemoryError("out of memory")
        made.append([c.tolist() for c in copies])

    eng._tier_copies = tier_copies
    a, b = synth.tokens(3, 1, 40), synth.tokens(3, 2, 40)
    eng.extend_end(eng.extend_begin([a]))
    before, done = _state(eng), len(made)
    fail[0] = True
    for _ in range(2):                     # spills a's tokens, which the failed calls still owe
        with pytest.raises(torch.OutOfMemoryError):
            eng.extend_begin([b])
        assert _state(eng)[0] == before[0] and _state(eng)[2] == 0
    fail[0] = False
    batch = eng.extend_begin([b])
    spilled = [m for m in made[done:] if len(m[0])]
    assert len(spilled) == 1 and len(spilled[0][0]) >= 20
    eng.extend_end(batch)
    assert eng.host.take_owed() == []


def test_contexts_of_a_4_bit_cache_are_not_grouped():
    """Groups of requests that share a prefix are dense decode's: none are planned or uploaded."""
    pre = synth.tokens(3, 1, 40)
    seqs = [np.concatenate([pre, synth.tokens(3, 5 + i, 5)]).astype(np.int32) for i in range(3)]
    for bits in (16, 4):
        eng = _engine4()
        eng.dev = _Failing()
        eng.kv_bits, eng.share_decode, eng.kv_chunk = bits, True, 16
        eng.extend_end(eng.extend_begin(seqs))
        eng.dev.calls = 0
        batch = eng.decode_begin(seqs)
        assert batch.num_groups == (1 if bits == 16 else 0) and eng.dev.calls == (2 if bits == 16 else 1)
        eng.decode_end(batch)


@pytest.mark.parametrize("hq,hkv", [(17, 1), (34, 2), (3, 2)])
def test_head_counts_that_4_bit_decode_refuses_are_refused_before_any_prompt(hq, hkv):
    args = dict(layers=1, head_dim=64, dtype=torch.float32, num_slots=64, max_reqs=2, max_ctx=32, device="cpu",
                kv_bits=4)
    with pytest.raises(ValueError):
        serving.Engine(n_q_heads=hq, n_kv_heads=hkv, **args)
    assert serving.Engine(n_q_heads=16 * hkv, n_kv_heads=hkv, **args).kv_bits == 4
