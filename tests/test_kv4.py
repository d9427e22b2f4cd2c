"""The cache held in 4 bits: written, read back and attended to on the GPU, against plain 64-bit
forms (kv4_ref). Bytes and numbers read back exactly; attention within tolerances counted from the
roundings."""
import ctypes
import math

import pytest
import torch

import prefix_cached_paged_gb300 as rc
from tests import kv4_ref as R

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
fake = lambda i: 0x10000000 * (1 + i)  # noqa: E731  (never dereferenced)


def same(a, b):
    """The first places where two tensors differ: none."""
    assert a.shape == b.shape and a.dtype == b.dtype
    return (a.cpu() != b.cpu()).nonzero()[:4].tolist()


# ---------------------------------------------------------------- on the CPU
def test_append_and_read_reject_bad_arguments_before_any_device_work():
    from prefix_cached_paged_gb300._lib import RcKv4AppendArgs, RcKv4ReadArgs, lib
    sizes = dict(dtype=rc.RC_DTYPE_BF16, num_kv_heads=4, head_dim=128, num_tokens=10, num_slots=50,
                 k_token_stride=512, k_head_stride=128, v_token_stride=512, v_head_stride=128)

    def append(**kw):
        a = dict(sizes, num_reqs=2)
        a.update({n: fake(i) for i, n in enumerate(("k", "v", "out_loc", "qo_indptr", "k_pool",
                                                    "v_pool"))})
        a.update(kw)
        return lib().rc_kv4_append(ctypes.byref(RcKv4AppendArgs(**a)), None)

    def read(**kw):
        a = dict(sizes, out_rows=10)
        a.update({n: fake(i) for i, n in enumerate(("k_pool", "v_pool", "slots", "k_out", "v_out"))})
        a.update(kw)
        return lib().rc_kv4_read(ctypes.byref(RcKv4ReadArgs(**a)), None)

    both = [dict(dtype=2), dict(num_kv_heads=0), dict(num_kv_heads=65537), dict(head_dim=0),
            dict(head_dim=32), dict(head_dim=96), dict(head_dim=320), dict(num_tokens=-1),
            dict(num_tokens=(1 << 24) + 1), dict(num_slots=0), dict(k_token_stride=513),
            dict(v_head_stride=4), dict(k_pool=0), dict(v_pool=0), dict(k_pool=fake(0) + 8),
            dict(k_pool=fake(9), v_pool=fake(9) + 1600)]
    for kw in both + [dict(num_reqs=-1), dict(k=0), dict(v=0), dict(out_loc=0), dict(qo_indptr=0),
                      dict(k=fake(0) + 4), dict(k=fake(4) + 160), dict(v=fake(5) + 15984)]:
        assert append(**kw) == rc.RC_ERR_INVALID, kw
    # planes may share memory when they are only read
    for kw in both[:-1] + [dict(k_out=0), dict(v_out=0), dict(slots=0), dict(out_rows=9),
                           dict(out_rows=-1), dict(out_rows=1 << 31), dict(v_out=fake(4) + 2),
                           dict(k_out=fake(0) + 160), dict(v_out=fake(3) + 256),
                           dict(k_head_stride=64), dict(v_token_stride=256),
                           dict(out_rows=9, out_loc=0)]:
        assert read(**kw) == rc.RC_ERR_INVALID, kw
    assert append(num_tokens=0) == append(num_reqs=0) == read(num_tokens=0) == rc.RC_OK
    assert lib().rc_kv4_append(None, None) == lib().rc_kv4_read(None, None) == rc.RC_ERR_INVALID


def test_decode_rejects_bad_arguments_before_any_device_work():
    from prefix_cached_paged_gb300._lib import RcKv4DecodeArgs, lib
    ptrs = ("q", "seq_len", "req_idx", "req_to_token", "k_pool", "v_pool", "o")

    def args(**kw):
        a = dict(dtype=rc.RC_DTYPE_BF16, num_rows=3, num_q_heads=8, num_kv_heads=2, head_dim=128,
                 max_reqs=4, max_ctx=1000, max_seq_len=1000, num_slots=50, sm_scale=0.1)
        a.update({n: fake(i) for i, n in enumerate(ptrs)})
        a.update(kw)
        return RcKv4DecodeArgs(**a)

    need = ctypes.c_size_t()
    assert lib().rc_kv4_decode_workspace_bytes(ctypes.byref(args()), ctypes.byref(need)) == 0

    def call(ws=fake(20), ws_bytes=1 << 30, **kw):
        return lib().rc_kv4_decode_attention(ctypes.byref(args(**kw)), ws, ws_bytes, None)

    for kw in (dict(dtype=3), dict(num_rows=-1), dict(num_rows=(1 << 20) + 1), dict(num_q_heads=7),
               dict(num_kv_heads=0), dict(num_q_heads=34), dict(num_q_heads=65537, num_kv_heads=65537),
               dict(head_dim=96), dict(head_dim=256), dict(max_seq_len=-1), dict(max_seq_len=(1 << 24) + 1),
               dict(num_rows=1 << 20, num_q_heads=256, num_kv_heads=32)):
        assert call(**kw) == rc.RC_ERR_INVALID, kw
        n = ctypes.c_size_t()
        assert lib().rc_kv4_decode_workspace_bytes(ctypes.byref(args(**kw)), ctypes.byref(n)) == \
            rc.RC_ERR_INVALID, kw
    for kw in (dict(max_seq_len=1001), dict(max_reqs=0), dict(num_slots=0), dict(sm_scale=0.0),
               dict(sm_scale=-1.0), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")),
               dict(q=0), dict(seq_len=0), dict(v_pool=0), dict(o=0), dict(o=fake(6) + 8),
               dict(k_pool=fake(4) + 2), dict(ws=fake(20) + 4), dict(o=fake(0)),
               dict(o=fake(0) + 3 * 8 * 256 - 16), dict(o=fake(4)), dict(o=fake(5) + 16),
               dict(o=fake(20) + 64)):
        assert call(**kw) == rc.RC_ERR_INVALID, kw
    if need.value:
        assert call(ws=0) == call(ws_bytes=need.value - 1) == rc.RC_ERR_INVALID
    assert call(num_rows=0) == rc.RC_OK
    assert lib().rc_kv4_decode_attention(None, fake(20), 1 << 20, None) == rc.RC_ERR_INVALID
    assert lib().rc_kv4_decode_workspace_bytes(ctypes.byref(args()), None) == rc.RC_ERR_INVALID


def test_row_bytes():
    assert [rc.kv4_row_bytes(d) for d in (64, 128, 192, 256)] == [40, 80, 120, 160]
    for d in (0, 32, 96, 320):
        with pytest.raises(ValueError):
            rc.kv4_row_bytes(d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_plain_form_keeps_numbers_within_half_a_scale(dtype):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((400, 64), generator=g) * torch.exp2(torch.randint(-40, 25, (400, 1), generator=g))
    x = (x + torch.randn((400, 1), generator=g)).to(DT[dtype])
    held = R.quantise(x)
    a, b = R.parts(held, 64)
    scale = held[:, 32:].contiguous().view(torch.bfloat16).double()[:, ::2].repeat_interleave(32, 1)
    # the difference, the reciprocal and the product are fp32: a code of 15 moves by 15 * 3 * 2^-24
    assert ((a + b - x.double()).abs() <= scale * (0.5 + 2.0 ** -18)).all()
    # the scale is at most an eighth more than covers the group from its minimum rounded down
    lo, hi = (f(x.double().view(400, 2, 32), -1) for f in (torch.amin, torch.amax))
    width = (hi - lo + lo.abs() * 2.0 ** -7).repeat_interleave(32, 1)
    assert (scale <= width / 15 * 1.1251).all()


# ---------------------------------------------------------------- writing and reading back
def special_rows(dtype, d):
    """Heads whose groups are at the borders of what the format holds."""
    g = torch.Generator().manual_seed(2)
    base = torch.randn(d, generator=g)
    rows = [torch.zeros(d), torch.full((d,), -0.0), torch.full((d,), 3.7), torch.full((d,), -3.7),
            base * 1e-30, base * 1e-39, base * 2.0 ** 27, base.abs(), -base.abs(), 100 + base,
            -100 + base, base * 1e-3 + 1e4, torch.arange(d) % 16 * 1.0, (torch.arange(d) % 31) * 0.5,
            torch.arange(d) % 16 * 1.0 - 7.5, torch.where(torch.arange(d) % 3 == 0, 1e-38, 1.0)]
    for bad in (math.nan, math.inf, -math.inf, 2.0 ** 30, -2.0 ** 30, 3e38):
        r = base.clone()
        r[d // 2 + 5] = bad
        rows.append(r)
    near = base.clone()
    near[3], near[40] = 2.0 ** 30 * (1 - 2.0 ** -8), -2.0 ** 30 * (1 - 2.0 ** -8)
    rows.append(near)
    alone = torch.zeros(d)
    alone[7] = 1.0
    return torch.stack(rows + [alone, -alone]).to(DT[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_append_at_the_borders_of_the_format(dtype, d):
    x = special_rows(dtype, d)
    n = x.shape[0]
    k, v = x[:, None].cuda(), x.flip(0)[:, None].contiguous().cuda()
    kp, vp = (torch.zeros((n, 1, d * 5 // 8), dtype=torch.uint8, device="cuda") for _ in "kv")
    loc = torch.arange(n, dtype=torch.int32, device="cuda")
    ip = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rc.kv4_append(k, v, loc, ip, kp, vp)
    for got, src in ((kp, k), (vp, v)):
        assert same(got, R.quantise(src)) == []
    for out_t in DT.values():
        ko, vo = (torch.empty((n, 1, d), dtype=out_t, device="cuda") for _ in "kv")
        rc.kv4_read(kp, vp, loc, ko, vo)
        for got, held in ((ko, kp), (vo, vp)):
            want = R.values(held, d).float().to(out_t)
            assert torch.equal(got.cpu().isnan(), want.isnan())
            assert same(got.nan_to_num(7), want.nan_to_num(7)) == []
    assert rc.device_status() == 0


WRITES = [  # dtype, tokens of each request, padding, heads, d, fused (k and v slices of one tensor)
    ("bf16", [1], 0, 1, 64, False), ("bf16", [1], 0, 8, 128, True), ("bf16", [], 3, 2, 128, False),
    ("bf16", [0, 0], 4, 2, 128, True), ("bf16", [5, 0, 17], 6, 3, 128, True),
    ("bf16", [33], 0, 32, 128, False), ("bf16", [300, 211], 1, 5, 64, True),
    ("bf16", [7, 7], 0, 6, 192, True), ("bf16", [40], 2, 2, 256, False),
    ("bf16", [2000, 3], 2, 1, 64, True), ("bf16", [700], 0, 8, 64, False),
    ("bf16", [301], 3, 4, 128, True), ("bf16", [1001], 1, 2, 192, True), ("f32", [900], 0, 2, 256, False),
    ("bf16", [2500], 2, 9, 64, True), ("bf16", [700, 3], 1, 15, 128, False),
    ("bf16", [420], 0, 16, 192, True), ("f32", [900], 0, 7, 256, True), ("f32", [2001], 3, 10, 64, False),
    ("bf16", [1, 2], 1, 32, 256, True),
    ("f32", [1], 0, 1, 64, False), ("f32", [13, 2], 5, 3, 64, True), ("f32", [64], 0, 8, 128, True),
    ("f32", [9], 1, 7, 192, False), ("f32", [21], 0, 1, 256, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,pad,h,d,fused", WRITES)
def test_append_writes_the_bytes_and_read_gives_the_numbers(dtype, new, pad, h, d, fused):
    g = torch.Generator().manual_seed(sum(new) + h + d)
    n, dt = sum(new), DT[dtype]
    t, slots = n + pad, n + pad + 9
    kv = torch.randn((t, 2 * h + 1, d), generator=g).to(dt)
    cu = kv.cuda()
    k, v = cu[:, :h], cu[:, h:2 * h]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    planes = torch.randint(0, 256, (2, slots, h, d * 5 // 8), generator=g, dtype=torch.uint8)
    loc = torch.randperm(slots, generator=g)[:t].to(torch.int32)
    used = loc.clone()
    used[n:] = -5          # not read
    ip = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    kp, vp = planes.cuda()
    rc.kv4_append(k, v, used.cuda(), ip.cuda(), kp, vp)
    want = planes.clone()
    want[0, loc[:n].long()] = R.quantise(kv[:n, :h])
    want[1, loc[:n].long()] = R.quantise(kv[:n, h:2 * h])
    assert same(torch.stack([kp, vp]), want) == []
    # read back: every written slot, twice, dense; then into rows of strided outputs
    if n == 0:
        assert rc.device_status() == 0
        return
    at = torch.cat([loc[:n], loc[:n].flip(0)]).cuda()
    num = [R.values(want[i, at.cpu().long()], d).float() for i in range(2)]
    for out_t in DT.values():
        ko, vo = (torch.full((2 * n + 1, h, d), 7.0, dtype=out_t, device="cuda") for _ in "kv")
        rc.kv4_read(kp, vp, at, ko, vo)
        for got, w in ((ko, num[0]), (vo, num[1])):
            assert same(got[:2 * n], w.to(out_t)) == [] and (got[2 * n:] == 7).all()
        both = torch.full((3 * n + 2, 2 * h + 1, d), 7.0, dtype=out_t, device="cuda")
        rows = torch.randperm(3 * n + 2, generator=g)[:2 * n].to(torch.int32)
        rc.kv4_read(kp, vp, at, both[:, h + 1:], both[:, :h], out_loc=rows.cuda())
        expect = torch.full(both.shape, 7.0, dtype=out_t)
        expect[rows.long(), h + 1:] = num[0].to(out_t)
        expect[rows.long(), :h] = num[1].to(out_t)
        assert same(both, expect) == []
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_every_scale_and_its_ties():
    """All significands of a scale at all exponents, elements on and beside the borders between codes;
    widths just above and below what a scale covers."""
    e = torch.arange(-82, 28).double()
    scale = ((8 + torch.arange(8)).double() / 8 * torch.exp2(e)[:, None]).reshape(-1)   # [110 * 8]
    k = torch.arange(14).double() + 0.5
    eps = torch.tensor([0, 2.0 ** -22, -2.0 ** -22]).double()
    rows = []
    for shift in (0.0, -7.0):
        x = torch.zeros((len(scale), 64), dtype=torch.float64)
        x[:, 0], x[:, 1] = shift, 15 + shift
        x[:, 2:16], x[:, 16:30] = k + shift, k * (1 + 2.0 ** -21) + shift
        x[:, 30:32] = shift + 3
        for i, d in enumerate(eps):   # the second group: widths at a scale's border
            y = x.clone()
            y[:, 32:48], y[:, 48:] = shift, 15 * (1 + d) + shift
            rows.append(y * scale[:, None])
    x = torch.cat(rows).float()[:, None]
    n = x.shape[0]
    loc = torch.arange(n, dtype=torch.int32, device="cuda")
    ip = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for dt in DT.values():
        y = x.to(dt)
        kp, vp = (torch.zeros((n, 1, 40), dtype=torch.uint8, device="cuda") for _ in "kv")
        rc.kv4_append(y.cuda(), (-y).cuda(), loc, ip, kp, vp)
        assert same(kp, R.quantise(y)) == [] and same(vp, R.quantise(-y)) == []
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_bad_slots_are_reported_and_skipped():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((6, 2, 64), generator=g).cuda()
    kp, vp = torch.randint(0, 256, (2, 10, 2, 40), generator=g, dtype=torch.uint8).cuda()
    k0, v0 = kp.clone(), vp.clone()
    loc = torch.tensor([3, -1, 10, 5, 2 ** 31 - 1, 0], dtype=torch.int32)
    rc.kv4_append(x, x, loc.cuda(), torch.tensor([0, 6], dtype=torch.int32, device="cuda"), kp, vp)
    assert rc.device_status() == 1
    ok = [0, 3, 5]
    for got, old in ((kp, k0), (vp, v0)):
        old[loc[ok].long().cuda()] = R.quantise(x[ok]).cuda()
        assert same(got, old) == []
    ko, vo = torch.full((2, 6, 2, 64), 7.0, device="cuda")
    rc.kv4_read(kp, vp, loc.cuda(), ko, vo)
    assert rc.device_status() == 1
    want = R.values(kp[loc[ok].long().cuda()], 64).float()
    assert torch.equal(ko[ok].cpu().nan_to_num(9), want.nan_to_num(9))
    assert (ko[[1, 2, 4]] == 7).all() and (vo[[1, 2, 4]] == 7).all()
    # rows outside the outputs
    ko.fill_(7)
    rows = torch.tensor([6, 1, -2, 0, 2, 3], dtype=torch.int32)
    rc.kv4_read(kp, vp, torch.full((6,), 5, dtype=torch.int32, device="cuda"), ko, vo,
                out_loc=rows.cuda())
    assert rc.device_status() == 1
    want = R.values(kp[5], 64).float().nan_to_num(9)
    assert all(torch.equal(ko[i].cpu().nan_to_num(9), want) for i in (0, 1, 2, 3))
    assert (ko[4:] == 7).all()
    # tokens past the arrays' end in the offsets: what is there is written
    ip = torch.tensor([0, 99], dtype=torch.int32, device="cuda")
    loc = torch.tensor([1, 2, 4, 6, 7, 8], dtype=torch.int32, device="cuda")
    rc.kv4_append(x, x, loc, ip, kp, vp)
    assert torch.equal(kp[loc.long()].cpu(), R.quantise(x)) and rc.device_status() == 0
    rc.kv4_append(x, x, loc, torch.tensor([0, -4], dtype=torch.int32, device="cuda"), kp, vp)
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_python_refusals():
    x = torch.zeros((4, 2, 64), device="cuda")
    kp, vp = (torch.zeros((9, 2, 40), dtype=torch.uint8, device="cuda") for _ in "kv")
    loc = torch.arange(4, dtype=torch.int32, device="cuda")
    ip = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    app = lambda **kw: rc.kv4_append(*{**dict(k=x, v=x.clone(), l=loc, ip=ip, kp=kp, vp=vp),  # noqa: E731
                                       **kw}.values())
    for kw in (dict(kp=kp[:, :, :39]), dict(kp=kp.float()), dict(vp=vp[:8]), dict(l=loc.long()),
               dict(l=loc[:3]), dict(v=x[:3]), dict(v=x.bfloat16()), dict(k=x.cpu()),
               dict(k=x.half(), v=x.half()), dict(kp=kp[::2], vp=vp[::2]), dict(vp=kp),
               dict(k=x.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError, rc.RcError)):
            app(**kw)
    for kw in (dict(slots=loc.long()), dict(ko=x[:3]), dict(ko=x.half()), dict(vo=x),
               dict(ko=x[:, :1]), dict(ko=x[:1].expand(4, 2, 64)), dict(kp=kp.cpu()),
               dict(out=loc[:2])):
        a = {**dict(kp=kp, vp=vp, slots=loc, ko=x, vo=x.clone(), out=None), **kw}
        with pytest.raises((ValueError, TypeError, rc.RcError)):
            rc.kv4_read(a["kp"], a["vp"], a["slots"], a["ko"], a["vo"], out_loc=a["out"])
    q = torch.zeros((2, 4, 64), device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    t = torch.zeros((3, 16), dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, rc.kv4_decode_workspace_bytes(q, kp, max_seq_len=16)),
                     dtype=torch.uint8, device="cuda")
    for kw in (dict(n=n.long()), dict(o=q[:1]), dict(o=q.bfloat16()), dict(t=t.long()),
               dict(kp=kp[:, :1], vp=vp[:, :1]), dict(q=q.cpu()), dict(lse=torch.zeros(2, 4)),
               dict(most=17), dict(kp=kp[:, :1].expand(9, 2, 40)), dict(ws=ws.cpu())):
        a = {**dict(q=q, n=n, r=n, t=t, kp=kp, vp=vp, o=q.clone(), ws=ws, lse=None, most=16), **kw}
        with pytest.raises((ValueError, TypeError, rc.RcError)):
            rc.kv4_decode_attention(a["q"], a["n"], a["r"], a["t"], a["kp"], a["vp"], a["o"], a["ws"],
                                    sm_scale=0.1, max_seq_len=a["most"], lse=a["lse"])


# ---------------------------------------------------------------- attention
class Case:
    """Contexts in a scattered pool and query rows (request, visible tokens)."""

    def __init__(self, dtype, ctx, rows, hq, hkv, d, seed=0, k_scale=1.0, v_scale=1.0, extra=5):
        g = torch.Generator().manual_seed(seed + sum(ctx) * 31 + hq * 7 + d)
        self.g, self.dt, self.hq, self.hkv, self.d, self.rows = g, DT[dtype], hq, hkv, d, rows
        n = sum(ctx) + extra
        self.k = R.quantise(k_scale * torch.randn((n, hkv, d), generator=g))
        self.v = R.quantise(v_scale * torch.randn((n, hkv, d), generator=g) + 0.3)
        self.max_ctx = max(ctx) + 2
        r = len(ctx) + 1
        self.table = torch.full((r, self.max_ctx), -9, dtype=torch.int32)   # never read
        self.req = torch.randperm(r, generator=g)[:len(ctx)]
        perm, at = torch.randperm(n, generator=g).to(torch.int32), 0
        for i, m in zip(self.req.tolist(), ctx):
            self.table[i, :m] = perm[at:at + m]
            at += m
        self.q = torch.randn((len(rows), hq, d), generator=g).to(self.dt)

    def device(self):
        seq = torch.tensor([m for _, m in self.rows], dtype=torch.int32)
        req = self.req[torch.tensor([b for b, _ in self.rows])].to(torch.int32)
        self.max_seq = max(1, int(seq.max()))
        return [t.cuda() for t in (self.q, seq, req, self.table, self.k, self.v)]

    def call(self, scale=None, max_seq=None, stream=None):
        args = self.device()
        self.scale = scale or 1 / math.sqrt(self.d)
        self.max_seq = max_seq or self.max_seq
        n = len(self.rows)
        self.o = torch.full((n, self.hq, self.d), 7.0, dtype=self.dt, device="cuda")
        self.lse = torch.full((n, self.hq), 7.0, device="cuda")
        need = rc.kv4_decode_workspace_bytes(args[0], args[4], max_seq_len=self.max_seq)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        rc.kv4_decode_attention(*args, self.o, ws[:need], sm_scale=self.scale,
                                max_seq_len=self.max_seq, lse=self.lse, stream=stream)
        torch.cuda.synchronize()
        assert (ws[need:] == 255).all()
        return self

    def check(self, only=None):
        o, lse = self.o.cpu(), self.lse.cpu()
        for i, (b, m) in enumerate(self.rows):
            if only is not None and i not in only:
                continue
            ro, rl, to, tl = R.attend(self.q[i], m, self.table[int(self.req[b])], self.k, self.v,
                                      self.scale)
            err = (o[i].double() - ro).abs()
            tol = to + R.half_step(self.dt) * (ro.abs() + to)
            assert (err <= tol).all(), (i, m, float(err.max()), float((err - tol).max()))
            fin = rl.isfinite()
            assert torch.equal(lse[i].isfinite(), fin)
            assert ((lse[i].double() - rl).abs()[fin] <= tl[fin]).all(), (i, m)
            assert (lse[i][~fin] == -math.inf).all() and (o[i][~fin] == 0).all()
        return self


SHAPES = [  # dtype, contexts, hq, hkv, d
    ("bf16", [1], 1, 1, 128), ("bf16", [0, 15, 16, 17], 8, 2, 128), ("bf16", [0, 0], 4, 4, 64),
    ("bf16", [31, 32, 33, 63, 64, 65], 4, 4, 128), ("bf16", [1000, 129, 700], 32, 8, 128),
    ("bf16", [2049, 40], 8, 8, 128), ("bf16", [777], 64, 8, 128), ("bf16", [901, 333], 6, 2, 128),
    ("bf16", [1500], 10, 2, 64), ("bf16", [1200, 17], 16, 1, 128), ("bf16", [1024], 32, 2, 64),
    ("bf16", [3500], 12, 1, 128), ("bf16", [500, 1], 24, 2, 64), ("bf16", [400, 90], 9, 3, 128),
    ("bf16", [300, 600], 5, 5, 64), ("bf16", [257, 100], 14, 7, 128), ("bf16", [200], 12, 12, 128),
    ("bf16", [150, 151], 32, 32, 128), ("bf16", [90, 1], 6, 6, 64),
    ("f32", [1, 33], 2, 2, 64), ("f32", [700, 0, 97], 6, 2, 64), ("f32", [1111], 8, 1, 128),
    ("f32", [515], 13, 1, 128), ("f32", [260, 260], 4, 4, 128), ("f32", [2000], 16, 1, 64),
    ("f32", [64, 1, 500], 16, 8, 128), ("f32", [333], 15, 5, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ctx,hq,hkv,d", SHAPES)
def test_decode_matches_the_definition(dtype, ctx, hq, hkv, d):
    Case(dtype, ctx, [(b, m) for b, m in enumerate(ctx)], hq, hkv, d).call().check()
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_of_new_tokens(dtype):
    """Rows of one request with growing lengths, an empty one among them."""
    rows = [(0, 190 + i) for i in range(11)] + [(1, i) for i in range(9)] + [(2, 70)]
    Case(dtype, [200, 8, 70], rows, 8, 2, 128).call().check()
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_very_long_rows(dtype):
    """A context far longer than the pool (slots repeat) beside short ones."""
    c = Case(dtype, [300, 5, 77], [(0, 40_000), (1, 5), (2, 77)], 4, 2, 64)
    c.max_ctx = 40_001
    table = torch.randint(0, 380, (c.table.shape[0], c.max_ctx), generator=c.g, dtype=torch.int32)
    table[:, :c.table.shape[1]] = torch.where(c.table >= 0, c.table, table[:, :c.table.shape[1]])
    c.table = table
    c.call().check()
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,k_scale,v_scale", [
    ("bf16", 30.0, 1e6), ("bf16", 1e-9, 1e-9), ("bf16", 1e-25, 1e8), ("f32", 30.0, 1e-12),
    ("f32", 1e-9, 1e6), ("bf16", 200.0, 1e-3)])
def test_large_and_small_caches(dtype, k_scale, v_scale):
    Case(dtype, [300, 70], [(0, 300), (1, 70)], 8, 2, 128, k_scale=k_scale,
         v_scale=v_scale).call().check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_queries(dtype):
    c = Case(dtype, [200, 90, 40], [(0, 200), (1, 90), (2, 40)], 4, 2, 128)
    c.q[0] *= 1e-20
    c.q[1] *= 1e6
    c.k = R.quantise(R.values(c.k, 128) * 1e-6)
    c.q[2, 1] = 0
    c.q[2, 2, 5:] = 0
    c.q[2, 3, 7] = 3e4
    c.call().check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_rows_and_slots(dtype):
    ctx = [100, 64, 50, 40]
    c = Case(dtype, ctx, [(b, m) for b, m in enumerate(ctx)], 8, 2, 64)
    r = c.req.tolist()
    c.table[r[0], 7], c.table[r[0], 99] = -1, c.k.shape[0]   # weigh nothing
    c.table[r[1], :64] = 2 ** 31 - 1                         # a row of such tokens alone
    c.call()
    assert rc.device_status() == 1
    c.check()
    # a length beyond max_seq_len and a request beyond the table; row 3 is as it was
    c = Case(dtype, ctx, [(b, m) for b, m in enumerate(ctx)], 8, 2, 64)
    args = c.device()
    args[1] = torch.tensor([100, 65, -1, 40], dtype=torch.int32, device="cuda")
    args[2][0] = 5
    c.scale = 0.125
    for max_seq in (64,):
        c.o = torch.full((4, 8, 64), 7.0, dtype=c.dt, device="cuda")
        c.lse = torch.full((4, 8), 7.0, device="cuda")
        ws = torch.empty(rc.kv4_decode_workspace_bytes(args[0], args[4], max_seq_len=max_seq),
                         dtype=torch.uint8, device="cuda")
        rc.kv4_decode_attention(*args, c.o, ws, sm_scale=c.scale, max_seq_len=max_seq, lse=c.lse)
        assert rc.device_status() == 2
        c.check(only=[3])
        assert (c.o[:3] == 0).all() and (c.lse[:3] == -math.inf).all()
    # an empty row may name any request
    args[1] = torch.tensor([0, 0, 0, 40], dtype=torch.int32, device="cuda")
    args[2][:3] = torch.tensor([-7, 2 ** 31 - 1, 99], dtype=torch.int32)
    rc.kv4_decode_attention(*args, c.o, ws, sm_scale=c.scale, max_seq_len=64, lse=c.lse)
    assert rc.device_status() == 0
    c.check(only=[3])
    assert (c.o[:3] == 0).all() and (c.lse[:3] == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_is_never_hidden_and_stays_where_it_is(dtype):
    """A lost group makes its head's outputs NaN, and no other's; one behind the row's end or in
    another request's slots changes nothing."""
    c = Case(dtype, [100, 90], [(0, 90), (1, 90)], 4, 2, 128)
    nan = R.quantise(torch.full((1, 1, 128), math.nan))[0, 0]
    r = c.req.tolist()
    held = c.table[c.table >= 0].tolist()
    c.table[r[0], 90:100] = next(s for s in range(c.k.shape[0]) if s not in held)
    c.k[c.table[r[0], 95].long()] = nan
    c.v[c.table[r[0], 95].long()] = nan
    c.call().check()
    c.k[c.table[r[1], 30].long(), 1] = nan
    c.v[c.table[r[0], 3].long(), 0, :] = torch.where(torch.arange(80) < 64, c.v[0, 0], nan)
    c.call()
    assert c.o[1, 2:].isnan().all() and c.lse[1, 2:].isnan().all()
    assert c.o[0, :2].isnan().all() and c.lse[0, :2].isfinite().all()
    assert c.o[0, 2:].isfinite().all() and c.o[1, :2].isfinite().all()
    c.q[0, 3, 8] = math.nan
    c.call()
    assert c.o[0, 3].isnan().all() and c.o[0, 2].isfinite().all()


@pytest.mark.gpu
def test_equal_scores_give_means():
    c = Case("f32", [500], [(0, 500)], 2, 2, 64)
    c.q.zero_()
    c.call().check()
    mean = R.values(c.v[c.table[int(c.req[0]), :500].long()], 64).mean(0)
    assert (c.o[0].cpu().double() - mean).abs().max() < 1e-5
    assert (c.lse.cpu() - math.log(500)).abs().max() < 1e-5


@pytest.mark.gpu
def test_many_rows_and_calls_on_two_streams():
    """5000 rows of one request; calls that may overlap, each with its workspace; repeated calls
    give the same bits."""
    n = 5000
    c = Case("bf16", [90], [(0, i % 91) for i in range(n)], 4, 2, 64)
    c.call().check(only=list(range(0, n, 499)) + [n - 1])
    cases = [Case("bf16", [2000, 333], [(0, 2000), (1, 333)], 16, 4, 128),
             Case("f32", [1500], [(0, 1500), (0, 1490)], 4, 2, 64)]
    jobs = []
    for x in cases:
        x.call().check()
        args = x.device()
        ws = torch.empty(rc.kv4_decode_workspace_bytes(args[0], args[4], max_seq_len=x.max_seq),
                         dtype=torch.uint8, device="cuda")
        jobs.append((x, args, ws, [torch.empty_like(x.o) for _ in range(20)]))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(20):
        for s, (x, args, ws, o) in zip(streams, jobs):
            rc.kv4_decode_attention(*args, o[i], ws, sm_scale=x.scale, max_seq_len=x.max_seq,
                                    stream=s)
    torch.cuda.synchronize()
    for x, _, _, o in jobs:
        assert all(torch.equal(y, x.o) for y in o)
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_a_captured_step_follows_the_cache():
    """Append and attention captured once, replayed with other new tokens, lengths and slots."""
    c = Case("bf16", [130, 60], [(0, 130), (1, 60)], 8, 2, 128)
    q, seq, req, table, kp, vp = c.device()
    new = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    k, v = new[:, :2], new[:, 2:]
    loc = torch.zeros(2, dtype=torch.int32, device="cuda")
    ip = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    ws = torch.empty(rc.kv4_decode_workspace_bytes(q, kp, max_seq_len=132), dtype=torch.uint8,
                     device="cuda")

    def step():
        rc.kv4_append(k, v, loc, ip, kp, vp)
        rc.kv4_decode_attention(q, seq, req, table, kp, vp, o, ws, sm_scale=0.1, max_seq_len=132,
                                lse=lse)

    loc.copy_(table[req.long(), seq.long() - 1])
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        new.copy_(torch.randn(new.shape, generator=c.g))
        c.q = torch.randn(c.q.shape, generator=c.g).to(c.dt)
        q.copy_(c.q)
        c.rows = [(0, 130 - 40 * turn), (1, 60 - turn)]
        seq.copy_(torch.tensor([m for _, m in c.rows]))
        loc.copy_(table[req.long(), seq.long() - 1])
        graph.replay()
        torch.cuda.synchronize()
        c.k, c.v, c.o, c.lse, c.scale = kp.cpu(), vp.cpu(), o, lse, 0.1
        assert torch.equal(c.k[loc.cpu().long()], R.quantise(k))
        assert torch.equal(c.v[loc.cpu().long()], R.quantise(v))
        c.check()
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Planes of more than 2^32 bytes: slots at both ends."""
    h, d = 8, 128
    slots = (1 << 32) // (h * 80) + 1000
    kp, vp = (torch.empty((slots, h, 80), dtype=torch.uint8, device="cuda") for _ in "kv")
    g = torch.Generator().manual_seed(4)
    n = 70
    x = torch.randn((n, 2 * h, d), generator=g).bfloat16()
    loc = torch.cat([torch.arange(35), slots - 1 - torch.arange(35)]).to(torch.int32)
    cu = x.cuda()
    rc.kv4_append(cu[:, :h], cu[:, h:], loc.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                  kp, vp)
    ko, vo = torch.empty((2, n, h, d), dtype=torch.bfloat16, device="cuda")
    rc.kv4_read(kp, vp, loc.cuda(), ko, vo)
    held = R.quantise(x)
    assert torch.equal(ko.cpu(), R.values(held[:, :h], d).float().bfloat16())
    assert torch.equal(vo.cpu(), R.values(held[:, h:], d).float().bfloat16())
    q = torch.randn((1, 2 * h, d), generator=g).bfloat16()
    o, lse = torch.empty_like(q).cuda(), torch.empty((1, 2 * h), device="cuda")
    ws = torch.empty(rc.kv4_decode_workspace_bytes(q, kp, max_seq_len=n), dtype=torch.uint8,
                     device="cuda")
    one = torch.tensor([n], dtype=torch.int32, device="cuda")
    rc.kv4_decode_attention(q.cuda(), one, torch.zeros_like(one), loc[None].contiguous().cuda(), kp,
                            vp, o, ws, sm_scale=0.1, max_seq_len=n, lse=lse)
    ro, rl, to, tl = R.attend(q[0], n, torch.arange(n), held[:, :h], held[:, h:], 0.1)
    assert ((o[0].cpu().double() - ro).abs() <= to + R.half_step(o.dtype) * (ro.abs() + to)).all()
    assert ((lse[0].cpu().double() - rl).abs() <= tl).all()
    assert rc.device_status() == 0
