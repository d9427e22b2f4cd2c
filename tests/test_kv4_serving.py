"""An engine whose cache is held in 4 bits, as a model's layers would drive it: extend over a cached
prefix that is read back, decode steps over the cache as it is held, the host tier."""
import numpy as np
import pytest
import torch

import prefix_cached_paged_gb300 as rc
import synth
from tests import cache_ops_ref as C
from tests import harness as H
from tests import kv4_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def qkv(tag, layer, n, hq, hkv, d, dt):
    g = torch.Generator().manual_seed(tag * 100 + layer)
    x = torch.randn((n, hq + 2 * hkv, d), generator=g).to(dt)
    return [t.contiguous() for t in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])]


def causal(q, k, v, first, scale):
    """q [S, Hq, d] at positions first .., k, v [first + S, Hkv, d] -> [S, Hq, d], float64."""
    S, hq, d = q.shape
    g = hq // k.shape[1]
    k, v = (t.double().repeat_interleave(g, 1) for t in (k, v))
    s = torch.einsum("shd,thd->hst", q.double(), k) * scale
    seen = torch.arange(k.shape[0])[None] <= first + torch.arange(S)[:, None]
    return torch.einsum("hst,thd->shd", s.masked_fill(~seen, -np.inf).softmax(-1), v)


@pytest.mark.parametrize("dtype,hq,hkv,d,stack", [
    ("bf16", 16, 4, 128, "always"), ("bf16", 4, 4, 128, True), ("f32", 6, 2, 64, True),
    ("f32", 3, 3, 64, True)])
def test_a_model_step_over_a_4_bit_cache(dtype, hq, hkv, d, stack):
    from prefix_cached_paged_gb300.serving import Engine
    dt, layers = DT[dtype], 2
    table = rc.rope_table(10000.0 ** (-np.arange(16) / 16), 800)
    eng = Engine(layers, hq, hkv, d, dt, 4096, 16, 800, synth.permutation(5, 4096), kv_bits=4,
                 stack_extend=stack, rope=table)
    pre = synth.tokens(9, 1, 300)
    seqs = [np.concatenate([pre, synth.tokens(9, 10 + i, 25 + 40 * i)]).astype(np.int32)
            for i in range(3)]
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(2))).to(dt)

    def slots(layer, plane, rows, n):
        return plane[layer].cpu()[torch.from_numpy(np.asarray(rows[:n], np.int64))]

    for tag, batch in enumerate(([pre], seqs)):
        b = eng.extend_begin(batch)
        for layer in range(layers):
            q, k, v = qkv(tag, layer, b.num_tokens, hq, hkv, d, dt)
            o = torch.empty(q.shape, dtype=dt, device="cuda")
            eng.extend_layer(b, layer, q.cuda(), k.cuda(), v.cuda(), o)
            o = o.cpu()
            for i, (P, n) in enumerate(zip(b.plan.prefix_len, b.plan.lengths)):
                a, e = b.plan.qo_indptr[i], b.plan.qo_indptr[i + 1]
                held = [slots(layer, t, b.plan.rows[i], n) for t in (eng.dev.k, eng.dev.v)]
                # new tokens are held as their formula says; attention saw them as given and the
                # prefix as it is held, rounded to the type
                for got, x in zip(held, (k, v)):
                    assert torch.equal(got[P:], R.quantise(x[a:e]))
                kv = [torch.cat([R.values(t[:P], d).float().to(dt), x[a:e]])
                      for t, x in zip(held, (k, v))]
                ok, ma, rl = H.compare(o[a:e].double().numpy(),
                                       causal(q[a:e], *kv, int(P), eng.sm_scale).numpy(), dtype)
                assert ok, (tag, layer, i, ma, rl)
        eng.extend_end(b)
    db = eng.decode_begin(seqs)
    for step in range(3):
        eng.decode_step(db)
        for layer in range(layers):
            q, k, v = (t.cuda() for t in qkv(50 + step, layer, 3, hq, hkv, d, dt))
            o, lse = torch.empty_like(q), torch.empty((3, hq), device="cuda")
            if step == 1:      # normalised and rotated on the way, attention in a call of its own
                kn = torch.empty_like(k)
                eng.norm_rope(db, q, k, q_weight=w.cuda(), k_weight=w.cuda(), k_out=kn)
                eng.append_layer(db, layer, k, v, k_weight=w.cuda())
                eng.decode_layer(db, layer, q, None, None, o, lse=lse)
                ref, tol = C.norm_rope(k.cpu(), w, torch.from_numpy(table), db.token_pos.cpu(), False,
                                       1e-6)
                assert ((kn.cpu().double() - ref).abs() <= tol + C.half_step(dt) *
                        (ref.abs() + tol)).all()
                k = kn
            else:
                eng.decode_layer(db, layer, q, k, v, o, lse=lse)
            kp, vp = eng.dev.k[layer].cpu(), eng.dev.v[layer].cpu()
            new = torch.from_numpy(db.new_slots).long()
            assert torch.equal(kp[new], R.quantise(k)) and torch.equal(vp[new], R.quantise(v))
            rows = eng.dev.req_to_token.cpu()
            for i, (r, n) in enumerate(zip(db.row_ids, db.seq_len)):
                ro, rl, to, tl = R.attend(q[i].cpu(), int(n), rows[int(r)], kp, vp, eng.sm_scale)
                err = (o[i].cpu().double() - ro).abs()
                assert (err <= to + R.half_step(dt) * (ro.abs() + to)).all(), (step, layer, i)
                assert ((lse[i].cpu().double() - rl).abs() <= tl).all()
    done = [np.concatenate([s, synth.tokens(9, 70 + i, 3)]).astype(np.int32)
            for i, s in enumerate(seqs)]
    eng.decode_end(db, done)
    # generated tokens stay cached and are read back by the next extend
    b = eng.extend_begin([np.concatenate([done[1], synth.tokens(9, 80, 9)]).astype(np.int32)])
    assert int(b.plan.prefix_len[0]) == len(done[1])
    q, k, v = qkv(90, 0, 9, hq, hkv, d, dt)
    o = torch.empty(q.shape, dtype=dt, device="cuda")
    eng.extend_layer(b, 0, q.cuda(), k.cuda(), v.cuda(), o)
    P = len(done[1])
    kv = [torch.cat([R.values(slots(0, t, b.plan.rows[0], P), d).float().to(dt), x])
          for t, x in ((eng.dev.k, k), (eng.dev.v, v))]
    ok, ma, rl = H.compare(o.cpu().double().numpy(), causal(q, *kv, P, eng.sm_scale).numpy(), dtype)
    assert ok, (ma, rl)
    eng.extend_end(b)
    assert rc.device_status() == 0


def test_spilled_tokens_come_back_as_they_were_held():
    from prefix_cached_paged_gb300.serving import Engine
    hq, hkv, d, dt = 4, 2, 64, torch.float32
    eng = Engine(1, hq, hkv, d, dt, 200, 4, 160, kv_bits=4, host_tier_slots=400)
    held = {}
    for i in range(3):                     # 120 tokens each: a pool of 200 spills the older ones
        seq = synth.tokens(4, 30 + i, 120)
        b = eng.extend_begin([seq])
        q, k, v = (t.cuda() for t in qkv(i, 0, 120, hq, hkv, d, dt))
        eng.extend_layer(b, 0, q, k, v, torch.empty_like(q))
        eng.extend_end(b)
        held[i] = (seq, R.quantise(k), R.quantise(v))
    assert eng.host.tree.stats()["spilled_tokens"] > 0
    seq, k, v = held[0]
    db = eng.decode_begin([seq])
    at = torch.from_numpy(db.context_rows[0, :120].astype(np.int64))
    assert torch.equal(eng.dev.k[0].cpu()[at], k) and torch.equal(eng.dev.v[0].cpu()[at], v)
    eng.decode_step(db)
    q, k1, v1 = (t.cuda() for t in qkv(9, 0, 1, hq, hkv, d, dt))
    o, lse = torch.empty_like(q), torch.empty((1, hq), device="cuda")
    eng.decode_layer(db, 0, q, k1, v1, o, lse=lse)
    n = torch.arange(121)
    ro, rl, to, tl = R.attend(q[0].cpu(), 121, n, torch.cat([k, R.quantise(k1)]),
                              torch.cat([v, R.quantise(v1)]), eng.sm_scale)
    assert ((o[0].cpu().double() - ro).abs() <= to + R.half_step(dt) * (ro.abs() + to)).all()
    assert ((lse[0].cpu().double() - rl).abs() <= tl).all()
    eng.decode_end(db)
    assert rc.device_status() == 0


def test_a_captured_layer_keeps_its_workspace():
    """decode_layer captured, replayed after calls that took other workspaces."""
    from prefix_cached_paged_gb300.serving import Engine
    hq, hkv, d, dt = 8, 2, 128, torch.bfloat16
    eng = Engine(1, hq, hkv, d, dt, 3000, 8, 1600, kv_bits=4)
    seqs = [synth.tokens(4, 40 + i, n) for i, n in enumerate((700, 1500))]
    for i, s in enumerate(seqs):
        b = eng.extend_begin([s])
        q, k, v = (t.cuda() for t in qkv(20 + i, 0, len(s), hq, hkv, d, dt))
        eng.extend_layer(b, 0, q, k, v, torch.empty_like(q))
        eng.extend_end(b)
    one, two = eng.decode_begin([seqs[0]]), eng.decode_begin([seqs[1]])
    runs = {}
    for name, batch in (("one", one), ("two", two)):
        eng.decode_step(batch)
        q, k, v = (t.cuda() for t in qkv(30 + len(runs), 0, 1, hq, hkv, d, dt))
        runs[name] = (batch, q, k, v, torch.empty_like(q), torch.empty((1, hq), device="cuda"))

    def run(name):
        batch, q, k, v, o, lse = runs[name]
        eng.decode_layer(batch, 0, q, k, v, o, lse=lse)

    for name in runs:
        run(name)
    want = {n: [t.clone() for t in r[4:]] for n, r in runs.items()}
    graphs = {}
    torch.cuda.synchronize()
    for name in runs:
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            run(name)
    for n, r in runs.items():
        for t in r[4:]:
            t.zero_()
    taken = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(30)]
    for _ in range(3):
        for g in graphs.values():
            g.replay()
    torch.cuda.synchronize()
    for n, r in runs.items():
        assert all(torch.equal(t, w) for t, w in zip(r[4:], want[n]))
    assert all((t == 7).all() for t in taken) and rc.device_status() == 0
