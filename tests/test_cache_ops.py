"""Norms with rotation, paged append and block bounds on the GPU against 64-bit plain forms, and
the refusals of their entry points (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import prefix_cached_paged_gb300 as rc
from tests import cache_ops_ref as R

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _close(got, ref, tol, dtype):
    got = got.double().cpu()
    bound = tol + R.half_step(dtype) * (ref.abs() + tol)
    bad = (got - ref).abs() > bound
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


# ---------------------------------------------------------------------------------- host
def test_rope_table_is_computed_in_double_precision():
    f = 10000.0 ** (-np.arange(32) / 32)
    t = rc.rope_table(f, 5, first_position=1_000_003, scale=0.5)
    ang = np.arange(1_000_003, 1_000_008)[:, None] * f
    assert t.dtype == np.float32 and t.shape == (5, 64)
    assert np.array_equal(t, np.concatenate([0.5 * np.cos(ang), 0.5 * np.sin(ang)], 1)
                          .astype(np.float32))
    assert rc.rope_table(f, 0).shape == (0, 64)
    for bad in (dict(inv_freq=f[:12], num_positions=2), dict(inv_freq=f, num_positions=-1),
                dict(inv_freq=f, num_positions=2, first_position=-1),
                dict(inv_freq=np.full(8, np.inf), num_positions=2),
                dict(inv_freq=f, num_positions=2, scale=float("nan"))):
        with pytest.raises(rc.RcError) as e:
            rc.rope_table(**bad)
        assert e.value.code == rc.RC_ERR_INVALID


def _fake(i):
    # a 16-byte aligned address that is never dereferenced: every call is rejected, or returns,
    # before anything reaches a device
    return 0x10000 + 256 * i


def test_norm_rope_rejects_bad_arguments_before_any_device_work():
    from prefix_cached_paged_gb300._lib import RcQkNormRopeArgs, lib
    ptrs = ["q", "k", "q_weight", "k_weight", "positions", "rope", "q_out", "k_out"]

    def call(**kw):
        a = dict(dtype=rc.RC_DTYPE_BF16, num_q_heads=8, num_kv_heads=2, head_dim=128,
                 rotary_dim=128, eps=1e-6, num_tokens=3, max_position=64)
        a.update({n: _fake(i) for i, n in enumerate(ptrs)})
        a.update(kw)
        return lib().rc_qk_norm_rope(ctypes.byref(RcQkNormRopeArgs(**a)), None)

    for kw in (dict(dtype=5), dict(num_q_heads=-1), dict(num_tokens=-1), dict(head_dim=0),
               dict(head_dim=100), dict(head_dim=264), dict(rotary_dim=24), dict(rotary_dim=144),
               dict(rope=0), dict(rope=_fake(5) + 4), dict(max_position=0), dict(positions=0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(q=0), dict(k_out=0),
               dict(q=_fake(0) + 8), dict(q_token_stride=4), dict(k_head_stride=129)):
        assert call(**kw) == rc.RC_ERR_INVALID, kw
    assert call(num_tokens=0) == rc.RC_OK and call(num_q_heads=0, num_kv_heads=0) == rc.RC_OK
    assert lib().rc_qk_norm_rope(None, None) == rc.RC_ERR_INVALID


def test_norm_rope_refuses_outputs_that_overlap():
    """Outputs that share a byte with an input other than their own rows, with the other output or
    with themselves, against all bytes counted out; views of one fused tensor that share none are
    taken. (The weight is misaligned: no call of this test gets past the checks.)"""
    from prefix_cached_paged_gb300._lib import RcQkNormRopeArgs, lib
    base, d, es = 1 << 20, 16, 2

    def refused(T, hq, hk, q, k, qo, ko):
        """Views as (offset, token stride, head stride) in elements."""
        a = RcQkNormRopeArgs(dtype=rc.RC_DTYPE_BF16, num_q_heads=hq, num_kv_heads=hk, head_dim=d,
                             eps=1e-6, num_tokens=T, q_weight=_fake(1) + 8)
        for name, v in (("q", q), ("k", k), ("q_out", qo), ("k_out", ko)):
            setattr(a, name, base + es * v[0])
            setattr(a, name + "_token_stride", v[1])
            setattr(a, name + "_head_stride", v[2])
        assert lib().rc_qk_norm_rope(ctypes.byref(a), None) == rc.RC_ERR_INVALID
        msg = lib().rc_last_error().decode()
        assert "overlaps" in msg or "multiples of 16" in msg, msg
        return "overlaps" in msg

    def rows(T, h, v):
        return [v[0] + t * v[1] + i * v[2] for t in range(T) for i in range(h)]

    def share(x, y):
        return bool({e + j for e in x for j in range(d)} & {e + j for e in y for j in range(d)})

    def wrong(T, hq, hk, q, k, qo, ko):
        r = [rows(T, h, v) for h, v in ((hq, q), (hk, k), (hq, qo), (hk, ko))]
        own = [len({e + j for e in x for j in range(d)}) < len(x) * d for x in r]
        return own[2] or own[3] or (r[2] != r[0] and share(r[2], r[0])) or \
            (r[3] != r[1] and share(r[3], r[1])) or share(r[2], r[1]) or share(r[3], r[0]) or \
            share(r[2], r[3])

    T, hq, hk = 5, 6, 2
    w = (hq + 2 * hk) * d
    far = 1 << 16
    fused_q, fused_k, fused_v = (0, w, d), (hq * d, w, d), ((hq + hk) * d, w, d)
    out_q, out_k = (far, hq * d, d), (2 * far, hk * d, d)
    for q, k, qo, ko in (
            (fused_q, fused_k, fused_q, fused_k), (fused_q, fused_k, out_q, out_k),
            (fused_q, fused_k, fused_q, out_k), (fused_q, fused_k, out_q, fused_v),
            # heads first: one buffer [hq + hk, T, d]
            ((0, d, T * d), (hq * T * d, d, T * d), (0, d, T * d), (hq * T * d, d, T * d)),
            # every KV head's queries beside its key and value: [T, hk, 5, d] with 3 queries a head
            # has no view of all queries; one query a head has
            ((0, hq * 3 * d, 3 * d), (d, hq * 3 * d, 3 * d), (0, hq * 3 * d, 3 * d),
             (2 * d, hq * 3 * d, 3 * d))):
        assert not wrong(T, hq, hk, q, k, qo, ko)
        assert not refused(T, hq, hk, q, k, qo, ko), (q, k, qo, ko)
    for q, k, qo, ko in (
            (fused_q, fused_k, (d, w, d), out_k), (fused_q, fused_k, (8, w, d), out_k),
            (fused_q, fused_k, (w, w, d), out_k), (fused_q, fused_k, out_q, (hq * d - 8, w, d)),
            (fused_q, fused_k, out_q, (far + 3 * d, hk * d, d)),
            (fused_q, fused_k, (far, 0, d), out_k), (fused_q, fused_k, (far, w, 0), out_k),
            (fused_q, fused_k, (far, d, d), out_k), (fused_q, fused_k, (far, w, 8), out_k)):
        assert wrong(T, hq, hk, q, k, qo, ko)
        assert refused(T, hq, hk, q, k, qo, ko), (q, k, qo, ko)
    # tokens and heads of one have no strides to speak of
    assert not refused(1, hq, 1, (0, 0, d), (hq * d, 7, 3), (0, 5 * w, d), (hq * d, 0, 0))
    g = np.random.default_rng(1)
    seen = [0, 0, 0]
    for _ in range(4000):
        T, hq, hk = (int(g.integers(1, 5)) for _ in range(3))
        ts = 8 * int(g.integers(-6, 40))

        def view():
            return (8 * int(g.integers(0, 60)), ts if g.random() < 0.8 else 8 * int(g.integers(0, 40)),
                    8 * int(g.integers(-4, 14)))

        q, k, qo, ko = (view() for _ in range(4))
        qo, ko = (q if g.random() < 0.5 else qo), (k if g.random() < 0.5 else ko)
        bad, got = wrong(T, hq, hk, q, k, qo, ko), refused(T, hq, hk, q, k, qo, ko)
        assert got or not bad, (T, hq, hk, q, k, qo, ko)
        alike = T == 1 or len({v[1] for v in (q, k, qo, ko)}) == 1
        assert bad or not got or not alike, (T, hq, hk, q, k, qo, ko)
        seen[bad + (got and not bad)] += got == bad
    assert min(seen[:2]) > 200, seen


def test_append_and_bounds_reject_bad_arguments_before_any_device_work():
    from prefix_cached_paged_gb300._lib import RcKvAppendArgs, RcKvBlockBoundsArgs, lib
    ptrs = ["k", "v", "out_loc", "qo_indptr", "prefix_len", "k_weight", "rope", "k_pool",
            "v_pool", "bounds", "req_idx"]

    def append(**kw):
        a = dict(dtype=rc.RC_DTYPE_F32, num_reqs=2, num_kv_heads=2, head_dim=64, rotary_dim=64,
                 eps=1e-6, block=64, num_tokens=9, num_slots=40, max_position=64, max_reqs=4,
                 max_blocks=2)
        a.update({n: _fake(i) for i, n in enumerate(ptrs)})
        a.update(kw)
        return lib().rc_kv_append(ctypes.byref(RcKvAppendArgs(**a)), None)

    for kw in (dict(dtype=2), dict(num_reqs=-1), dict(num_kv_heads=0), dict(num_slots=0),
               dict(head_dim=63), dict(rotary_dim=80), dict(block=48), dict(block=0),
               dict(max_blocks=0), dict(max_reqs=0), dict(req_idx=0), dict(k=0), dict(v_pool=0),
               dict(out_loc=0), dict(k_pool=_fake(7) + 8), dict(v_token_stride=2),
               dict(bounds=_fake(9) + 4), dict(eps=float("inf"))):
        assert append(**kw) == rc.RC_ERR_INVALID, kw
    assert append(num_reqs=0) == rc.RC_OK and append(num_tokens=0) == rc.RC_OK
    ptrs2 = ["seq_len", "req_idx", "req_to_token", "k_pool", "bounds"]

    def bounds(**kw):
        a = dict(dtype=rc.RC_DTYPE_BF16, num_layers=1, num_rows=2, num_kv_heads=2, head_dim=128,
                 max_reqs=4, max_ctx=100, block=32, max_blocks=4, num_slots=40)
        a.update({n: _fake(i) for i, n in enumerate(ptrs2)})
        a.update(kw)
        return lib().rc_kv_block_bounds(ctypes.byref(RcKvBlockBoundsArgs(**a)), None)

    for kw in (dict(dtype=9), dict(num_layers=0), dict(num_rows=-1), dict(head_dim=260),
               dict(block=8), dict(max_blocks=0), dict(max_ctx=0), dict(max_ctx=(1 << 24) + 1),
               dict(k_pool=0), dict(seq_len=0), dict(bounds=_fake(4) + 8)):
        assert bounds(**kw) == rc.RC_ERR_INVALID, kw
    assert bounds(num_rows=0) == rc.RC_OK


def test_calls_of_more_than_2_24_tokens_are_refused():
    """Items of an append are counted in 32 bits, 1024 requests together."""
    from prefix_cached_paged_gb300._lib import RcKvAppendArgs, RcQkNormRopeArgs, lib
    a = RcKvAppendArgs(dtype=rc.RC_DTYPE_BF16, num_reqs=2000, num_kv_heads=1, head_dim=64, block=16,
                       num_tokens=(1 << 24) + 1, num_slots=1 << 26,
                       **{n: _fake(i) for i, n in enumerate(["k", "v", "out_loc", "qo_indptr",
                                                             "prefix_len", "k_pool", "v_pool"])})
    assert lib().rc_kv_append(ctypes.byref(a), None) == rc.RC_ERR_INVALID
    a = RcQkNormRopeArgs(dtype=rc.RC_DTYPE_BF16, num_q_heads=1, head_dim=64, eps=1e-6,
                         num_tokens=(1 << 24) + 1, q=_fake(0), q_out=_fake(0), q_weight=_fake(1))
    assert lib().rc_qk_norm_rope(ctypes.byref(a), None) == rc.RC_ERR_INVALID


# ---------------------------------------------------------------------------------- norms, rotation
CASES = [  # dtype, T, hq, hkv, d, rot, interleaved, norm
    ("bf16", 1, 1, 1, 128, 128, False, True),
    ("bf16", 7, 32, 8, 128, 128, False, True),
    ("bf16", 33, 8, 8, 64, 64, True, True),
    ("bf16", 5, 5, 1, 256, 64, False, True),
    ("bf16", 3, 3, 3, 80, 80, False, False),
    ("bf16", 9, 4, 2, 96, 48, True, True),
    ("bf16", 4, 2, 2, 8, 0, False, True),
    ("bf16", 6, 40, 1, 192, 16, True, True),
    ("f32", 1, 2, 2, 64, 64, False, True),
    ("f32", 131, 6, 2, 64, 32, True, True),
    ("f32", 17, 3, 1, 128, 128, False, False),
    ("f32", 2, 4, 4, 256, 256, False, True),
    ("f32", 11, 1, 5, 72, 64, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,hq,hkv,d,rot,inter,norm", CASES)
@pytest.mark.parametrize("where", ["fused", "inplace"])
def test_norm_rope_matches_the_formula(dtype, T, hq, hkv, d, rot, inter, norm, where):
    g = _gen(T * 1000 + d)
    dt = DT[dtype]
    qkv = torch.randn((T, hq + 2 * hkv, d), generator=g).to(dt)
    table = R.rope_table(rot, 4099) if rot else None
    pos = torch.randint(0, 4099, (T,), generator=g, dtype=torch.int32)
    wq = (1 + 0.2 * torch.randn(d, generator=g)).to(dt) if norm else None
    wk = (1 + 0.2 * torch.randn(d, generator=g)).to(dt) if norm else None
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hkv]
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo, ko = (None, None) if where == "inplace" else (torch.full((T, hq, d), 7., dtype=dt,
                                                                 device="cuda"),
                                                      torch.full((T, hkv, d), 7., dtype=dt,
                                                                 device="cuda"))
    rc.qk_norm_rope(q, k, cu(pos) if rot else None, cu(table), q_weight=cu(wq), k_weight=cu(wk),
                    eps=1e-5, interleaved=inter, q_out=qo, k_out=ko)
    assert rc.device_status() == 0
    for got, x, w in ((q if qo is None else qo, qkv[:, :hq], wq),
                      (k if ko is None else ko, qkv[:, hq:hq + hkv], wk)):
        ref, tol = R.norm_rope(x, w, table, pos, inter, 1e-5)
        _close(got, ref, tol, dt)
    assert torch.equal(dev[:, hq + hkv:].cpu(), qkv[:, hq + hkv:])   # v untouched
    if where == "fused":
        assert torch.equal(dev.cpu(), qkv)


@pytest.mark.gpu
def test_norm_rope_parts_bad_positions_streams_and_graphs():
    g = _gen(3)
    T, d = 6, 128
    x = torch.randn((T, 4, d), generator=g).bfloat16().cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    table = R.rope_table(d, 50).cuda()
    pos = torch.tensor([0, 49, 50, -1, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 5.0)
    rc.qk_norm_rope(x, None, pos, table, q_weight=w, q_out=out)      # queries alone
    assert rc.device_status() == 2                                    # positions outside the table
    bad = torch.tensor([2, 3, 5])
    assert (out[bad.cuda()] == 5.0).all()                             # their rows are not written
    good = torch.tensor([0, 1, 4])
    ref, tol = R.norm_rope(x.cpu()[good], w.cpu(), table.cpu(), pos.cpu()[good], False, 1e-6)
    _close(out[good.cuda()], ref, tol, torch.bfloat16)
    # one weight only, keys and queries in one call: the other rows keep their norm
    k = torch.randn((T, 2, d), generator=g).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(x), torch.empty_like(k)
    rc.qk_norm_rope(x, k, pos, table, k_weight=w, q_out=qo, k_out=ko)
    for got, src, ww in ((qo, x, None), (ko, k, w.cpu())):
        ref, tol = R.norm_rope(src.cpu(), ww, table.cpu(), pos.cpu(), False, 1e-6)
        _close(got, ref, tol, torch.bfloat16)
    # captured on a side stream and replayed on new data
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2 = torch.empty_like(qo)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        rc.qk_norm_rope(x, None, pos, table, q_weight=w, q_out=o2)
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        rc.qk_norm_rope(x, None, pos, table, q_weight=w, q_out=o2)
    x.copy_(torch.randn(x.shape, generator=g).bfloat16())
    gr.replay()
    o3 = torch.empty_like(qo)
    rc.qk_norm_rope(x, None, pos, table, q_weight=w, q_out=o3, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o2, o3)
    # a row of zeros stays zero, one with an infinity or a NaN does not spread to other heads
    z = torch.zeros((1, 3, d), device="cuda")
    z[0, 1, 5], z[0, 2, 7] = float("inf"), float("nan")
    zo = torch.empty_like(z)
    rc.qk_norm_rope(z, None, pos[:1], table, q_weight=w.float(), q_out=zo)
    assert (zo[0, 0] == 0).all() and zo[0, 1].isnan().any() and zo[0, 2].isnan().all()
    # nothing to do
    rc.qk_norm_rope(x[:0], k[:0], pos[:0], table, q_weight=w)
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_norm_rope_refusals():
    x = torch.zeros((2, 2, 64), device="cuda")
    w, p = torch.ones(64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    t = R.rope_table(64, 4).cuda()
    for args, kw in (((None, None), {}), ((x, None), {}), ((x, None, None, t), {}),
                     ((x.cpu(), None, p, t), {}), ((x, None, p.cpu(), t), {}),
                     ((x.transpose(0, 2), None, p, t), {}),
                     ((x, None, p[:1], t), {}), ((x, None, p, t), dict(q_weight=w[:32])),
                     ((x, None, p, t), dict(k_weight=w)),
                     ((x, None, p, t), dict(q_out=x[:1])),
                     ((x, None, p, t), dict(q_out=x[:, :1].expand(2, 2, 64))),
                     ((x, x[:1], p, t), {})):
        with pytest.raises(ValueError):
            rc.qk_norm_rope(*args, **kw)
    for args, kw in (((x.half(), None, p, t), {}), ((x, None, p.long(), t), {}),
                     ((x, None, p, t.double()), {}), ((x, x.bfloat16(), p, t), {}),
                     ((x, None, p, t), dict(q_weight=w.bfloat16()))):
        with pytest.raises(TypeError):
            rc.qk_norm_rope(*args, **kw)
    with pytest.raises(rc.RcError):
        rc.qk_norm_rope(x[..., :60], None, p, t[:, :32].contiguous())


# ---------------------------------------------------------------------------------- append
def _append_case(dtype, new, pre, hkv, d, rot, inter, norm, block, with_bounds, seed=0, pad=3,
                 slots_extra=9):
    """Runs one append; checks pools, bounds and everything that must stay as it was."""
    g = _gen(seed + 17 * d + len(new))
    dt = DT[dtype]
    B, total = len(new), sum(new)
    T = total + pad
    slots = T + slots_extra
    kv = torch.randn((T, 2 * hkv, d), generator=g).to(dt)
    kp, vp = (torch.randn((slots, hkv, d), generator=g).to(dt) for _ in range(2))
    loc = torch.randperm(slots, generator=g)[:T].to(torch.int32)
    ip = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32)
    pl = torch.tensor(pre, dtype=torch.int32)
    ctx = max(p + n for p, n in zip(pre, new)) + 1
    nb = -(-ctx // block)
    table = R.rope_table(rot, ctx) if rot else None
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dt) if norm else None
    rows = B + 2
    req = torch.randperm(rows, generator=g)[:B].to(torch.int32)
    bd = torch.randn((rows, nb, hkv, 2, d), generator=g)
    bd[:, :, :, 0], bd[:, :, :, 1] = -bd[:, :, :, 0].abs(), bd[:, :, :, 1].abs()
    bd = bd.to(dt)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dkv, dkp, dvp, dbd = kv.cuda(), kp.cuda(), vp.cuda(), bd.cuda()
    kw = dict(rope=cu(table), k_weight=cu(w), eps=1e-6, interleaved=inter, block=block)
    if with_bounds:
        kw.update(bounds=dbd, req_idx=req.cuda())
    args = (dkv[:, :hkv], dkv[:, hkv:], loc.cuda(), ip.cuda(), pl.cuda(), dkp, dvp)
    rc.kv_append(*args, **kw)
    assert rc.device_status() == 0
    pos = torch.tensor([p + i for n, p in zip(new, pre) for i in range(n)], dtype=torch.int32)
    ref, tol = R.norm_rope(kv[:total, :hkv], w, table, pos, inter, 1e-6)
    at = loc[:total].long()
    gk, gv = dkp.cpu(), dvp.cpu()
    _close(gk[at], ref, tol, dt)
    assert torch.equal(gv[at], kv[:total, hkv:])
    rest = torch.ones(slots, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(gk[rest], kp[rest]) and torch.equal(gv[rest], vp[rest])
    want = bd.clone()
    if with_bounds:
        t = 0
        for n, p, r in zip(new, pre, req.tolist()):
            for i in range(n):
                key, b = gk[at[t]], (p + i) // block
                if (p + i) % block == 0 or (i == 0 and b * block >= p):
                    want[r, b, :, 0], want[r, b, :, 1] = key, key
                else:
                    want[r, b, :, 0] = torch.minimum(want[r, b, :, 0], key)
                    want[r, b, :, 1] = torch.maximum(want[r, b, :, 1], key)
                t += 1
    assert torch.equal(dbd.cpu(), want)
    # once more: nothing changes
    rc.kv_append(*args, **kw)
    assert torch.equal(dkp.cpu(), gk) and torch.equal(dvp.cpu(), gv)
    assert torch.equal(dbd.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,pre,hkv,d,rot,inter,norm,block,bounds", [
    ("bf16", [1], [0], 1, 128, 128, False, True, 64, True),
    ("bf16", [1, 1, 1, 1], [0, 63, 64, 65], 8, 128, 128, False, True, 64, True),
    ("bf16", [64, 65, 1, 0, 130], [0, 63, 127, 5, 1], 32, 128, 128, False, True, 64, True),
    ("bf16", [200, 3], [1500, 77], 3, 64, 32, True, False, 32, True),
    ("bf16", [33], [31], 40, 128, 64, True, True, 16, True),
    ("bf16", [300, 0, 17], [0, 0, 255], 2, 256, 128, False, True, 128, True),
    ("bf16", [40], [9], 5, 72, 0, False, True, 32, True),
    ("bf16", [7, 9], [0, 4], 4, 128, 128, False, True, 64, False),
    ("f32", [1, 70], [15, 16], 2, 64, 64, True, True, 16, True),
    ("f32", [129], [0], 1, 128, 128, False, False, 128, True),
    ("f32", [50, 1], [3, 0], 2, 256, 256, False, True, 64, True),
    ("f32", [5, 0, 12], [0, 3, 7], 7, 64, 0, False, False, 64, False),
])
def test_append_matches_the_formula(dtype, new, pre, hkv, d, rot, inter, norm, block, bounds):
    _append_case(dtype, new, pre, hkv, d, rot, inter, norm, block, bounds)


@pytest.mark.gpu
def test_append_of_more_requests_than_one_window():
    g = np.random.default_rng(5)
    new = g.integers(0, 4, 2500).tolist()
    pre = g.integers(0, 200, 2500).tolist()
    _append_case("bf16", new, pre, 2, 64, 64, False, True, 32, True, pad=0)


@pytest.mark.gpu
def test_append_skips_bad_requests_and_slots():
    """A request past the table, past its row's blocks, with a bad row or bad offsets is skipped
    whole; a token with a slot outside the pool alone. Each sets the status word; neighbours are
    written as if alone."""
    d, hkv, block = 64, 2, 16
    x = torch.randn((12, hkv, d), generator=_gen(1)).cuda()
    table = R.rope_table(d, 40).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(loc, ip, pl, req, nb=2):
        kp = torch.zeros((20, hkv, d), device="cuda")
        vp, bd = torch.zeros_like(kp), torch.full((3, nb, hkv, 2, d), 9.0, device="cuda")
        rc.kv_append(x, x, i32(loc), i32(ip), i32(pl), kp, vp, rope=table, bounds=bd,
                     req_idx=i32(req), block=block)
        return kp.cpu(), vp.cpu(), bd.cpu(), rc.device_status()

    loc = list(range(12))
    good = run(loc, [0, 4, 8, 12], [0, 3, 0], [0, 1, 2])
    assert good[3] == 0
    for kind, args in (("table", (loc, [0, 4, 8, 12], [0, 37, 0], [0, 1, 2], 3)),
                       ("blocks", (loc, [0, 4, 8, 12], [0, 30, 0], [0, 1, 2])),
                       ("row", (loc, [0, 4, 8, 12], [0, 3, 0], [0, 3, 2])),
                       ("negative row", (loc, [0, 4, 8, 12], [0, 3, 0], [0, -1, 2])),
                       ("prefix", (loc, [0, 4, 8, 12], [0, -1, 0], [0, 1, 2]))):
        kp, vp, bd, st = run(*args)
        assert st == 2, kind
        assert (vp[4:8] == 0).all() and (kp[4:8] == 0).all() and (bd[1] == 9.0).all(), kind
        for s in (slice(0, 4), slice(8, 12)):
            assert torch.equal(kp[s], good[0][s]) and torch.equal(vp[s], good[1][s]), kind
    # a request without new tokens is passed over, whatever the rest of it says
    kp, vp, bd, st = run(loc, [0, 4, 4, 12], [0, -7, 0], [0, 99, 2])
    assert st == 0 and torch.equal(vp[4:12], x[4:12].cpu())
    # offsets that run backwards or past the tokens
    kp, vp, bd, st = run(loc, [0, 4, 2, 12], [0, 0, 0], [0, 1, 2])
    assert st == 2 and (bd[1] == 9.0).all()
    kp, vp, bd, st = run(loc, [0, 4, 8, 13], [0, 3, 0], [0, 1, 2])
    assert st == 2 and torch.equal(kp[:8], good[0][:8]) and (kp[8:] == 0).all()
    # slots
    kp, vp, bd, st = run([0, 20, -1, 3] + loc[4:], [0, 4, 8, 12], [0, 3, 0], [0, 1, 2])
    assert st == 1
    keep = [0, 3] + loc[4:]
    assert torch.equal(kp[keep], good[0][keep]) and torch.equal(vp[keep], good[1][keep])
    assert (kp[[1, 2]] == 0).all()
    assert torch.equal(bd[0, 0], R.bounds_of(kp[[0, 3]], block)[0])


@pytest.mark.gpu
def test_append_strides_graph_and_refusals():
    g = _gen(9)
    d, hkv = 128, 4
    kp = torch.zeros((64, hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # heads-major storage: token stride d, head stride T * d; v expanded over heads
    k = torch.randn((hkv, 10, d), generator=g).bfloat16().cuda().transpose(0, 1)
    v = torch.randn((10, 1, d), generator=g).bfloat16().cuda().expand(10, hkv, d)
    loc, ip, pl = i32(list(range(30, 40))), i32([0, 10]), i32([5])
    rc.kv_append(k, v, loc, ip, pl, kp, vp)
    assert torch.equal(kp[30:40], k) and torch.equal(vp[30:40], v)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        rc.kv_append(k, v, loc, ip, pl, kp, vp)
    loc.copy_(i32(list(range(10))))
    k.copy_(torch.randn(k.shape, generator=g).bfloat16())
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(kp[:10], k) and (kp[10:30] == 0).all() and rc.device_status() == 0
    ok = dict(k=k, v=v, out_loc=loc, qo_indptr=ip, prefix_len=pl, k_pool=kp, v_pool=vp)
    bd = torch.zeros((2, 1, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=k.cpu()), dict(k=k[:, :2]), dict(v=v[:5]), dict(out_loc=loc[:5]),
                dict(qo_indptr=ip[:1]), dict(v_pool=vp[:3]), dict(k_pool=kp.transpose(0, 1)),
                dict(bounds=bd), dict(bounds=bd[:, :, :2], req_idx=pl),
                dict(bounds=bd, req_idx=i32([0, 1])), dict(rope=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            rc.kv_append(**{**ok, **bad})
    for bad in (dict(k=k.float()), dict(out_loc=loc.long()), dict(bounds=bd.float(), req_idx=pl)):
        with pytest.raises(TypeError):
            rc.kv_append(**{**ok, **bad})


@pytest.mark.gpu
def test_first_calls_of_a_process_may_be_captured():
    """A fresh process whose first call of each operator is inside a graph capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, prefix_cached_paged_gb300 as rc
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
T, hkv, d = 40, 2, 128
q = torch.randn((T, 4, d), device="cuda").bfloat16(); k = torch.randn((T, hkv, d), device="cuda").bfloat16()
w = torch.ones(d, device="cuda").bfloat16()
t = torch.from_numpy(rc.rope_table([0.5] * 64, 64)).cuda()
kp = torch.zeros((64, hkv, d), device="cuda").bfloat16(); vp = torch.zeros_like(kp)
bd = torch.zeros((1, 4, hkv, 2, d), device="cuda").bfloat16(); b2 = torch.zeros_like(bd)
table = torch.arange(64, dtype=torch.int32, device="cuda")[None].contiguous()
pos, ip, pl, zero, n = i32(list(range(T))), i32([0, T]), i32([0]), i32([0]), i32([T])
qo, ko, o = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q[:1])
ws = torch.empty(16, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rc.qk_norm_rope(q, k, pos, t, q_weight=w, q_out=qo, k_out=ko)
    rc.kv_append(ko, k, pos, ip, pl, kp, vp, bounds=bd, req_idx=zero, block=16)
    rc.kv_block_bounds(kp, table, zero, n, b2, block=16)
    rc.sparse_decode_attention(qo[-1:], n, zero, table, kp, vp, bd, o, ws, sm_scale=0.1,
                               max_seq_len=T, block=16, top_blocks=2)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
assert torch.equal(kp[:T], ko) and torch.equal(vp[:T], k) and torch.equal(bd[:, :3], b2[:, :3])
assert o.float().abs().sum() > 0 and rc.device_status() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# ---------------------------------------------------------------------------------- bounds
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,lens,hkv,d,block,layers", [
    ("bf16", [1], 1, 128, 64, 0), ("bf16", [0, 64, 65, 1000, 17], 8, 128, 64, 0),
    ("bf16", [300, 31], 32, 128, 128, 2), ("bf16", [129, 5], 3, 72, 16, 0),
    ("bf16", [77], 40, 64, 32, 3), ("bf16", [200], 1, 8, 32, 0),
    ("f32", [65, 0, 200], 2, 64, 32, 0), ("f32", [130], 5, 256, 64, 2),
])
def test_block_bounds_are_the_extremes_of_the_cached_keys(dtype, lens, hkv, d, block, layers):
    g = _gen(sum(lens) + d)
    dt = DT[dtype]
    slots, ctx, rows = sum(lens) + 5, max(lens) + 3, len(lens) + 2
    kp = torch.randn((max(layers, 1), slots, hkv, d), generator=g).to(dt)
    table = torch.full((rows, ctx), -7, dtype=torch.int32)     # unused entries are never read
    req = torch.randperm(rows, generator=g)[:len(lens)].to(torch.int32)
    perm, at = torch.randperm(slots, generator=g).to(torch.int32), 0
    for r, n in zip(req.tolist(), lens):
        table[r, :n] = perm[at:at + n]
        at += n
    nb = -(-ctx // block) + 1
    bd = torch.full((max(layers, 1), rows, nb, hkv, 2, d), 3.0, dtype=dt)
    want = bd.clone()
    for r, n in zip(req.tolist(), lens):
        for la in range(max(layers, 1)):
            b = R.bounds_of(kp[la][table[r, :n].long()], block)
            want[la, r, :b.shape[0]] = b
    dk, db = kp.cuda(), bd.cuda()
    if not layers:
        dk, db = dk[0], db[0]
    rc.kv_block_bounds(dk, table.cuda(), req.cuda(),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"), db, block=block)
    assert rc.device_status() == 0
    assert torch.equal(db.cpu().reshape(want.shape), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hkv,d", [  # keys of 1, 2, 3, 4, 5, 7 and 8 chunks of 16 bytes
    ("bf16", 1, 8), ("bf16", 2, 8), ("bf16", 1, 16), ("bf16", 3, 8), ("bf16", 1, 24),
    ("bf16", 1, 32), ("bf16", 2, 16), ("bf16", 4, 8), ("bf16", 5, 8), ("bf16", 7, 8),
    ("bf16", 1, 64), ("f32", 1, 8), ("f32", 1, 16), ("f32", 2, 8), ("f32", 1, 24), ("f32", 1, 32)])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_block_bounds_of_narrow_tokens(dtype, hkv, d, block):
    """Tokens whose keys are narrower than a warp's copies: several tokens stand beside one another,
    and every one of them has to be read. Lengths end inside a block and on its border; slots
    outside the pool late in a block are left out and reported."""
    lens = [1, 31, 33, 63, 64, 65, 97, 127, 128, 129, 200, 256, 0, 300]
    g = _gen(hkv * 1000 + d + block)
    dt, ctx = DT[dtype], 310
    n = sum(lens) + 3
    kp = torch.randn((n, hkv, d), generator=g).to(dt)
    perm, at = torch.randperm(n, generator=g).to(torch.int32), 0
    table = torch.full((len(lens), ctx), -7, dtype=torch.int32)
    for r, m in enumerate(lens):
        table[r, :m] = perm[at:at + m]
        at += m
    nb = -(-ctx // block)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def check():
        bd = torch.full((len(lens), nb, hkv, 2, d), 3.0, dtype=dt)
        want = bd.clone()
        for r, m in enumerate(lens):
            for b in range(-(-m // block)):
                s = table[r, b * block:min(m, (b + 1) * block)].long()
                s = s[(s >= 0) & (s < n)]
                want[r, b, :, 0], want[r, b, :, 1] = kp[s].amin(0), kp[s].amax(0)
        bd = bd.cuda()
        rc.kv_block_bounds(kp.cuda(), table.cuda(), i32(list(range(len(lens)))), i32(lens), bd,
                           block=block)
        assert torch.equal(bd.cpu(), want)

    check()
    assert rc.device_status() == 0
    table[13, 45], table[13, 110], table[13, 255] = -1, n, 2 ** 31 - 1
    check()
    assert rc.device_status() == 1


@pytest.mark.gpu
def test_block_bounds_of_more_rows_than_one_window():
    n = 2300
    lens = np.random.default_rng(3).integers(0, 40, n)
    lens[7] = 0
    g = _gen(12)
    kp = torch.randn((500, 1, 64), generator=g)
    table = torch.randint(0, 500, (n, 40), generator=g, dtype=torch.int32)
    bd = torch.full((n, 3, 1, 2, 64), 3.0)
    want = bd.clone()
    for r in range(n):
        b = R.bounds_of(kp[table[r, :int(lens[r])].long()], 16)
        want[r, :b.shape[0]] = b
    db = bd.cuda()
    rc.kv_block_bounds(kp.cuda(), table.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(lens.astype(np.int32)).cuda(), db, block=16)
    assert rc.device_status() == 0 and torch.equal(db.cpu(), want)


@pytest.mark.gpu
def test_block_bounds_nan_bad_rows_and_slots():
    g = _gen(2)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.randn((40, 1, 64), generator=g).bfloat16().cuda()
    kp[3, 0, 7], kp[4, 0, 8], kp[5, 0, 9] = float("nan"), float("inf"), -float("inf")
    table = torch.arange(40, dtype=torch.int32, device="cuda").repeat(4, 1)
    bd = torch.full((4, 3, 1, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    rc.kv_block_bounds(kp, table, i32([0]), i32([20]), bd, block=16)
    assert rc.device_status() == 0
    ref = R.bounds_of(kp[:20].cpu(), 16)
    assert torch.equal(bd[0, :2].cpu().nan_to_num(99.0), ref.nan_to_num(99.0))
    assert bd[0, 0, 0, 0, 7].isnan() and bd[0, 0, 0, 1, 7].isnan()
    for req, n in ((4, 20), (-1, 20), (1, 41), (1, -1), (1, 49)):
        rc.kv_block_bounds(kp, table, i32([req, 2]), i32([n, 33]), bd, block=16)
        assert rc.device_status() == 2, (req, n)
        assert (bd[1] == 3.0).all()
        assert torch.equal(bd[2].cpu().nan_to_num(99.0), R.bounds_of(kp[:33].cpu(), 16)
                           .nan_to_num(99.0))
    rc.kv_block_bounds(kp, table, i32([-1, 99]), i32([0, 0]), bd, block=16)   # padded rows
    assert rc.device_status() == 0
    table[3, 1], table[3, 2] = 40, -1
    rc.kv_block_bounds(kp, table, i32([3]), i32([8]), bd, block=16)
    assert rc.device_status() == 1
    keep = torch.tensor([0, 3, 4, 5, 6, 7])
    assert torch.equal(bd[3, 0].cpu().nan_to_num(99.0),
                       R.bounds_of(kp.cpu()[keep], 16)[0].nan_to_num(99.0))
    ok = dict(k_pool=kp, req_to_token=table, req_idx=i32([0]), seq_len=i32([3]), bounds=bd)
    for bad in (dict(bounds=bd[0]), dict(bounds=bd[:2]), dict(req_idx=i32([0, 1])),
                dict(k_pool=kp[None]), dict(seq_len=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rc.kv_block_bounds(**{**ok, **bad})
    with pytest.raises(TypeError):
        rc.kv_block_bounds(**{**ok, "bounds": bd.float()})
    with pytest.raises(rc.RcError):
        rc.kv_block_bounds(**ok, block=24)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_block_without_a_valid_token_ranks_last(dtype):
    """Slots outside the pool for every token of a block, in a short append, one whose blocks the
    warps of a CTA share, and a build: the block's bounds are the largest and the lowest finite
    number, which no query takes for a good block, and which later tokens replace."""
    dt, d, hkv, block = DT[dtype], 64, 2, 16
    big = torch.finfo(dt).max
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for n in (3, 100):
        x = torch.randn((n, hkv, d), generator=_gen(n)).to(dt).cuda()
        kp = torch.zeros((300, hkv, d), dtype=dt, device="cuda")
        vp, bd = torch.zeros_like(kp), torch.full((1, 8, hkv, 2, d), 9.0, dtype=dt, device="cuda")
        loc = torch.arange(n, dtype=torch.int32, device="cuda")
        loc[-(n % block or block):] = -1
        last = (n - 1) // block
        rc.kv_append(x, x, loc, i32([0, n]), i32([0]), kp, vp, bounds=bd, req_idx=i32([0]),
                     block=block)
        assert rc.device_status() == 1
        assert (bd[0, last, :, 0] == big).all() and (bd[0, last, :, 1] == -big).all()
        assert (bd[0, last + 1:] == 9.0).all()
        if last:
            assert torch.equal(bd[0, :last], R.bounds_of(x[:last * block], block))
        # a build of the same row says the same
        table = torch.full((1, 128), 300, dtype=torch.int32, device="cuda")
        table[0, :n] = loc
        b2 = torch.full_like(bd, 9.0)
        rc.kv_block_bounds(kp, table, i32([0]), i32([n]), b2, block=block)
        assert rc.device_status() == 1 and torch.equal(b2, bd)
        # the block's next token is its only one
        rc.kv_append(x[:1], x[:1], i32([250]), i32([0, 1]), i32([n]), kp, vp, bounds=bd,
                     req_idx=i32([0]), block=block)
        assert rc.device_status() == 0
        assert torch.equal(bd[0, last, :, 0], x[0]) and torch.equal(bd[0, last, :, 1], x[0])
    # selection: zeros in the query, the empty block among real ones of negative scores
    nb = 8
    q = torch.zeros((1, hkv, d), dtype=dt, device="cuda")
    q[:, :, 5] = 1.0
    kp = -torch.rand((200, hkv, d), generator=_gen(1)).add(0.1).to(dt).cuda()
    vp = torch.randn((200, hkv, d), generator=_gen(2)).to(dt).cuda()
    table = torch.arange(nb * block, dtype=torch.int32, device="cuda")[None].contiguous()
    table[0, 3 * block:4 * block] = 999
    bd = torch.zeros((1, nb, hkv, 2, d), dtype=dt, device="cuda")
    rc.kv_block_bounds(kp, table, i32([0]), i32([nb * block]), bd, block=block)
    assert rc.device_status() == 1
    o = torch.empty_like(q)
    sel = torch.empty((1, hkv, nb - 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    rc.sparse_decode_attention(q, i32([nb * block]), i32([0]), table, kp, vp, bd, o, ws,
                               sm_scale=0.1, max_seq_len=nb * block, block=block,
                               top_blocks=nb - 1, sink_blocks=0, selected=sel)
    assert rc.device_status() == 0
    assert sel[0].tolist() == [[0, 1, 2, 4, 5, 6, 7]] * hkv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hkv,d,rot", [(5, 64, 64), (2, 128, 96), (3, 80, 32), (1, 256, 256)])
def test_a_key_has_the_same_bits_whichever_call_rotates_it(dtype, inter, norm, hkv, d, rot):
    """qk_norm_rope and kv_append have kernels, and arithmetic, of their own; requests of one token,
    whose warps take heads beside one another, and of many, whose warps take tokens."""
    g, dt = _gen(d + hkv), DT[dtype]
    new = [1] * 9 if d == 80 else [70, 1, 45]
    pre = [7 * i for i in range(len(new))]
    T = sum(new)
    k = (3 * torch.randn((T, hkv, d), generator=g)).to(dt).cuda()
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).cuda() if norm else None
    table = R.rope_table(rot, 200).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pos = i32([p + i for n, p in zip(new, pre) for i in range(n)])
    ko = torch.empty_like(k)
    rc.qk_norm_rope(None, k, pos, table, k_weight=w, interleaved=inter, k_out=ko)
    kp, vp = torch.zeros((T, hkv, d), dtype=dt, device="cuda"), torch.zeros_like(k)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    for bounds in (False, True):
        kp.zero_()
        kw = dict(bounds=torch.zeros((len(new), 16, hkv, 2, d), dtype=dt, device="cuda"),
                  req_idx=i32(list(range(len(new)))), block=16) if bounds else {}
        rc.kv_append(k, k, i32(list(range(T))), i32([sum(new[:i]) for i in range(len(new) + 1)]),
                     i32(pre), kp, vp, rope=table, k_weight=w, interleaved=inter, **kw)
        assert torch.equal(kp.view(bits), ko.view(bits)) and rc.device_status() == 0
