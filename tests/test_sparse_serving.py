"""The operators around the cache run together through serving.Engine, as a model's layers would
call them: norms and rotation, extend and append, block bounds, block-sparse and dense decode."""
import math

import numpy as np
import pytest
import torch

import prefix_cached_paged_gb300 as rc
import synth
from tests import cache_ops_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Model:
    """Seeded projections per (layer, request, position) and the 64-bit forms of what is cached."""

    def __init__(self, dtype, layers, hq, hkv, d, rot, inter, block, max_ctx=600):
        self.dt, self.layers, self.hq, self.hkv, self.d = DT[dtype], layers, hq, hkv, d
        self.inter, self.block = inter, block
        self.table = torch.from_numpy(rc.rope_table(
            10000.0 ** (-np.arange(rot // 2) * 2.0 / rot), max_ctx))
        g = torch.Generator().manual_seed(3)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(self.dt) for _ in range(2))

    def qkv(self, tag, layer, n):
        g = torch.Generator().manual_seed(tag * 100 + layer)
        return torch.randn((n, self.hq + 2 * self.hkv, self.d), generator=g).to(self.dt)

    def split(self, x):
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _engine(m, **kw):
    from prefix_cached_paged_gb300.serving import Engine
    return Engine(m.layers, m.hq, m.hkv, m.d, m.dt, 4096, 16, 600, synth.permutation(5, 4096),
                  rope=m.table, sparse_block=m.block, **kw)


def _check_rows(m, eng, layer, q, o, lse, sel, rows, top):
    """rows: (slot-table row, visible tokens) per query row. Against what is in the cache."""
    kp, vp = eng.dev.k[layer].cpu(), eng.dev.v[layer].cpu()
    table = eng.dev.req_to_token.cpu()
    q, o, lse, sel = q.cpu(), o.cpu(), lse.cpu(), sel.cpu()
    for i, (row, n) in enumerate(rows):
        keys = kp[table[row, :n].long()]
        want = R.select(q[i], R.bounds_of(keys, m.block), n, m.block, top, 1, 1)
        assert torch.equal(sel[i], want), (i, row, n)
        ro, rl, to, tl = R.attend(q[i], want, n, table[row], kp, vp, m.block, eng.sm_scale)
        tol = to + R.half_step(m.dt) * (ro.abs() + to)
        assert ((o[i].double() - ro).abs() <= tol).all() and \
            ((lse[i].double() - rl).abs() <= tl).all(), (i, row, n)


@pytest.mark.parametrize("dtype,hq,hkv,d,rot,inter,block", [
    ("bf16", 16, 4, 128, 128, False, 32), ("f32", 4, 2, 64, 32, True, 16)])
def test_a_model_step_through_the_engine(dtype, hq, hkv, d, rot, inter, block):
    m = Model(dtype, 2, hq, hkv, d, rot, inter, block)
    eng = _engine(m)
    pre = synth.tokens(9, 1, 170)
    seqs = [np.concatenate([pre, synth.tokens(9, 10 + i, 25 + 40 * i)]).astype(np.int32)
            for i in range(3)]
    kw = dict(eps=1e-6, interleaved=inter)
    cu = lambda t: t.cuda()  # noqa: E731
    wq, wk = cu(m.wq), cu(m.wk)
    tag, top = 0, 4
    # the shared prefix, then its continuations (a cached prefix of 170 in every row): the keys
    # that extend attends to and scatters are those of the formula
    for batch_seqs in ([pre], seqs):
        tag += 1
        b = eng.extend_begin(batch_seqs)
        T = b.num_tokens
        pos = torch.tensor([p for s, P in zip(batch_seqs, b.plan.prefix_len)
                            for p in range(int(P), len(s))], dtype=torch.int32)
        for layer in range(m.layers):
            x = m.qkv(tag, layer, T)
            q, k, v = m.split(cu(x))
            qo = torch.empty((T, hq, d), dtype=m.dt, device="cuda")
            ko = torch.empty((T, hkv, d), dtype=m.dt, device="cuda")
            v = v.contiguous()
            eng.norm_rope(b, q, k, q_weight=wq, k_weight=wk, q_out=qo, k_out=ko, **kw)
            o = torch.empty_like(qo)
            if dtype == "bf16" and d == 128 or dtype == "f32":
                eng.extend_layer(b, layer, qo, ko, v, o)
            ref, tol = R.norm_rope(m.split(x)[1], m.wk, m.table, pos, inter, 1e-6)
            got = eng.dev.k[layer][torch.from_numpy(b.plan.out_loc).long().cuda()].cpu()
            err = (got.double() - ref).abs()
            assert (err <= tol + R.half_step(m.dt) * (ref.abs() + tol)).all()
            # append puts the same keys and values where they are, and sparse attention of every
            # new token (a chunk) follows the definition
            k_before, v_before = eng.dev.k[layer].clone(), eng.dev.v[layer].clone()
            with pytest.raises(ValueError):
                eng.sparse_layer(b, layer, qo, o, top_blocks=top)
            eng.append_layer(b, layer, k, v, k_weight=wk, **kw)
            assert torch.equal(_bits(eng.dev.k[layer]), _bits(k_before))
            assert torch.equal(_bits(eng.dev.v[layer]), _bits(v_before))
            lse = torch.empty((T, hq), device="cuda")
            sel = torch.empty((T, hkv, top), dtype=torch.int32, device="cuda")
            eng.sparse_layer(b, layer, qo, o, top_blocks=top, lse=lse, selected=sel)
            rows = [(int(r), int(p) + 1) for r, S, P in zip(b.row_ids, b.plan.lengths -
                                                            b.plan.prefix_len, b.plan.prefix_len)
                    for p in range(int(P), int(P + S))]
            some = sorted(set(range(0, T, 29)) | {T - 1})
            pick = torch.tensor(some)
            _check_rows(m, eng, layer, qo.cpu()[pick], o.cpu()[pick], lse.cpu()[pick],
                        sel.cpu()[pick], [rows[i] for i in some], top)
        eng.extend_end(b)
    # decode: three steps, the second with dense attention alone on layer 1, so that its bounds
    # miss a token until the third builds them anew
    db = eng.decode_begin(seqs)
    with pytest.raises(ValueError):
        eng.append_layer(db, 0, None, None)
    B = len(seqs)
    for step in range(3):
        tag += 1
        eng.decode_step(db)
        for layer in range(m.layers):
            q, k, v = m.split(cu(m.qkv(tag, layer, B)))
            v = v.contiguous()
            qo, ko = (torch.empty((B, h, d), dtype=m.dt, device="cuda") for h in (hq, hkv))
            eng.norm_rope(db, q, k, q_weight=wq, k_weight=wk, q_out=qo, k_out=ko, **kw)
            dense, dl = torch.empty_like(qo), torch.empty((B, hq), device="cuda")
            eng.decode_layer(db, layer, qo, ko, v, dense, lse=dl)
            if step == 1 and layer == 1:
                with pytest.raises(ValueError):
                    eng.sparse_layer(db, layer, qo, dense, top_blocks=top)
                continue
            # once with the keys rotated already, once on the way
            if step == 0:
                eng.append_layer(db, layer, ko, v, rotate=False)
            else:
                eng.append_layer(db, layer, k, v, k_weight=wk, **kw)
            o, lse = torch.empty_like(qo), torch.empty_like(dl)
            rows = [(int(r), int(n)) for r, n in zip(db.row_ids, db.seq_len)]
            for t in (top, 40):
                sel = torch.empty((B, hkv, t), dtype=torch.int32, device="cuda")
                eng.sparse_layer(db, layer, qo, o, top_blocks=t, lse=lse, selected=sel)
                _check_rows(m, eng, layer, qo, o, lse, sel, rows, t)
            # all blocks: what dense decode gives, within both kernels' tolerances of fp64
            for i, (row, n) in enumerate(rows):
                _, rl, to, tl = R.attend(qo.cpu()[i], sel.cpu()[i], n,
                                         eng.dev.req_to_token.cpu()[row], eng.dev.k[layer].cpu(),
                                         eng.dev.v[layer].cpu(), m.block, eng.sm_scale)
                d64 = (o[i].cpu().double() - dense[i].cpu().double()).abs()
                step_err = 2 * R.half_step(m.dt) * (dense[i].cpu().double().abs() + to)
                assert (d64 <= 2 * to + step_err).all()
                assert ((lse[i] - dl[i]).cpu().double().abs() <= 2 * tl).all()
    eng.decode_end(db)
    # rows and slots go to other requests: nothing of the old bounds is left in the way
    b = eng.decode_begin([seqs[2][:100], seqs[0]])
    eng.decode_step(b)
    q, k, v = m.split(cu(m.qkv(99, 0, 2)))
    qo = torch.empty((2, hq, d), dtype=m.dt, device="cuda")
    eng.norm_rope(b, q, None, q_weight=wq, q_out=qo, **kw)
    eng.append_layer(b, 0, k, v, k_weight=wk, **kw)
    o, lse = torch.empty_like(qo), torch.empty((2, hq), device="cuda")
    sel = torch.empty((2, hkv, top), dtype=torch.int32, device="cuda")
    eng.sparse_layer(b, 0, qo, o, top_blocks=top, lse=lse, selected=sel)
    _check_rows(m, eng, 0, qo, o, lse, sel, [(int(r), int(n)) for r, n in zip(b.row_ids, b.seq_len)],
                top)
    assert rc.device_status() == 0


def test_engine_without_rope_or_bounds():
    from prefix_cached_paged_gb300.serving import Engine
    args = (1, 4, 2, 64, torch.float32, 512, 4, 128)
    for bad in (dict(rope=np.zeros((64, 32), np.float32)), dict(rope=np.zeros((128, 32))),
                dict(sparse_block=24)):
        with pytest.raises(ValueError):
            Engine(*args, **bad)
    eng = Engine(*args)
    b = eng.extend_begin([synth.tokens(1, 1, 20)])
    x = torch.zeros((20, 2, 64), device="cuda")
    for call in (lambda: eng.norm_rope(b, x), lambda: eng.append_layer(b, 0, x, x),
                 lambda: eng.sparse_layer(b, 0, x, x, top_blocks=4)):
        with pytest.raises(ValueError):
            call()
    # bounds alone: norms without a rotation
    eng = Engine(*args, sparse_block=16)
    b = eng.extend_begin([synth.tokens(1, 1, 20)])
    q = torch.randn((20, 4, 64), generator=torch.Generator().manual_seed(1)).cuda()
    k = q[:, :2].contiguous()
    w = torch.ones(64, device="cuda")
    ref, tol = R.norm_rope(q.cpu(), w.cpu(), None, None, False, 1e-6)
    eng.norm_rope(b, q, q_weight=w)
    assert ((q.cpu().double() - ref).abs() <= tol + R.U32 * ref.abs()).all()
    eng.append_layer(b, 0, k, k)
    o = torch.empty_like(q)
    eng.sparse_layer(b, 0, q, o, top_blocks=2)
    assert torch.equal(eng.dev.k[0][torch.from_numpy(b.plan.out_loc).long().cuda()], k)
    assert math.isfinite(float(o.sum())) and rc.device_status() == 0


def test_a_captured_long_step_keeps_its_workspace():
    """Contexts beyond the blocks whose scores shared memory holds: a captured call replayed after
    a call that needs more workspace, with memory taken in between, gives what it gave and touches
    nothing else."""
    lens = (121_000, 130_000)
    m = Model("bf16", 1, 4, 1, 64, 32, False, 16, max_ctx=131_072)
    from prefix_cached_paged_gb300.serving import Engine
    n = sum(lens) + 64
    eng = Engine(1, 4, 1, 64, m.dt, n, 4, 131_072, synth.permutation(5, n), rope=m.table,
                 sparse_block=16)
    seqs = [synth.tokens(9, 20 + i, x) for i, x in enumerate(lens)]
    for i, s in enumerate(seqs):
        b = eng.extend_begin([s])
        _, k, v = m.split(m.qkv(30 + i, 0, len(s)).cuda())
        eng.append_layer(b, 0, k, v)
        eng.extend_end(b)
    db = eng.decode_begin([seqs[0]])
    both = eng.decode_begin(seqs)
    top = 9
    out = {}
    for name, batch in (("one", db), ("both", both)):
        eng.decode_step(batch)
        B = len(batch.row_ids)
        q, k, v = (t.contiguous() for t in m.split(m.qkv(40 + B, 0, B).cuda()))
        eng.append_layer(batch, 0, k, v)
        out[name] = (q, torch.empty_like(q), torch.empty((B, 4), device="cuda"),
                     torch.empty((B, 1, top), dtype=torch.int32, device="cuda"))

    def run(name, batch):
        q, o, lse, sel = out[name]
        eng.sparse_layer(batch, 0, q, o, top_blocks=top, lse=lse, selected=sel)

    run("one", db)
    want = [t.clone() for t in out["one"][1:]]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run("one", db)
    need = rc.sparse_decode_workspace_bytes(out["one"][0], eng.dev.k[0], max_seq_len=lens[0] + 1,
                                            block=16, top_blocks=top)
    assert need > 0
    run("both", both)
    taken = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    want2 = [t.clone() for t in out["both"][1:]]
    for t in out["one"][1:]:
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in zip(out["one"][1:], want))
    assert all((t == 7).all() for t in taken)
    run("both", both)
    assert all(torch.equal(x, w) for x, w in zip(out["both"][1:], want2))
    for name, batch in (("one", db), ("both", both)):
        q, o, lse, sel = out[name]
        _check_rows(m, eng, 0, q, o, lse, sel,
                    [(int(r), int(s)) for r, s in zip(batch.row_ids, batch.seq_len)], top)
    assert rc.device_status() == 0
