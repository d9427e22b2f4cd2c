"""Block-sparse decode attention on the GPU against a plain 64-bit form: the selected blocks
exactly, outputs and log-sum-exp within tolerances counted from the roundings (cache_ops_ref)."""
import ctypes
import math

import pytest
import torch

import prefix_cached_paged_gb300 as rc
from tests import cache_ops_ref as R

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def test_sparse_decode_rejects_bad_arguments_before_any_device_work():
    from prefix_cached_paged_gb300._lib import RcSparseDecodeArgs, lib
    ptrs = ["q", "seq_len", "req_idx", "req_to_token", "k_pool", "v_pool", "bounds", "o"]
    fake = lambda i: 0x10000 + 256 * i  # noqa: E731  (never dereferenced)

    def args(**kw):
        a = dict(dtype=rc.RC_DTYPE_BF16, num_rows=3, num_q_heads=8, num_kv_heads=2, head_dim=128,
                 max_reqs=4, max_ctx=1000, block=64, max_blocks=16, max_seq_len=1000,
                 top_blocks=8, sink_blocks=1, recent_blocks=1, num_slots=50, sm_scale=0.1)
        a.update({n: fake(i) for i, n in enumerate(ptrs)})
        a.update(kw)
        return RcSparseDecodeArgs(**a)

    need = ctypes.c_size_t()
    long = dict(max_ctx=1 << 20, max_seq_len=1 << 20, max_blocks=1 << 14)
    assert lib().rc_sparse_decode_workspace_bytes(ctypes.byref(args(**long)),
                                                  ctypes.byref(need)) == 0 and need.value > 0

    def call(ws=fake(20), ws_bytes=need.value, **kw):
        return lib().rc_sparse_decode_attention(ctypes.byref(args(**kw)), ws, ws_bytes, None)

    sizes = [dict(dtype=3), dict(num_rows=-1), dict(num_q_heads=7), dict(num_kv_heads=0),
             dict(num_q_heads=34), dict(head_dim=96), dict(head_dim=256), dict(block=63),
             dict(block=256), dict(max_seq_len=-1), dict(max_seq_len=(1 << 24) + 1),
             dict(top_blocks=0), dict(top_blocks=1), dict(sink_blocks=-1), dict(recent_blocks=0),
             dict(sink_blocks=5, recent_blocks=4), dict(num_rows=1 << 28),
             dict(top_blocks=8193)]
    for kw in sizes:
        assert call(**kw) == rc.RC_ERR_INVALID, kw
        a = args(**kw)
        n = ctypes.c_size_t()
        assert lib().rc_sparse_decode_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == \
            rc.RC_ERR_INVALID, kw
    for kw in (dict(max_seq_len=1001), dict(max_blocks=15), dict(max_reqs=0), dict(num_slots=0),
               dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(sm_scale=float("nan")),
               dict(sm_scale=float("inf")), dict(q=0), dict(bounds=0), dict(o=fake(7) + 8),
               dict(k_pool=fake(4) + 2), dict(ws=0, **long), dict(ws=fake(20) + 4),
               dict(ws_bytes=need.value - 1, **long),
               # 2^27 - 1 units of 16 CTAs each
               dict(num_rows=(1 << 27) - 1, num_q_heads=1, num_kv_heads=1, top_blocks=1024, **long)):
        assert call(**kw) == rc.RC_ERR_INVALID, kw
    assert call(num_rows=0) == rc.RC_OK
    assert lib().rc_sparse_decode_attention(None, fake(20), 1 << 20, None) == rc.RC_ERR_INVALID
    assert lib().rc_sparse_decode_workspace_bytes(ctypes.byref(args()), None) == rc.RC_ERR_INVALID


class Case:
    """Contexts in a scattered pool, their bounds, and query rows (request, visible tokens)."""

    def __init__(self, dtype, ctx, rows, hq, hkv, d, block, seed=0, spread=1.0, extra=5):
        g = torch.Generator().manual_seed(seed + sum(ctx) * 31 + hq * 7 + d)
        self.g, self.dt, self.block = g, DT[dtype], block
        self.hq, self.hkv, self.d, self.rows = hq, hkv, d, rows
        n = sum(ctx) + extra
        self.k = (spread * torch.randn((n, hkv, d), generator=g)).to(self.dt)
        self.v = torch.randn((n, hkv, d), generator=g).to(self.dt)
        self.max_ctx = max(ctx) + 2
        R_, nb = len(ctx) + 1, -(-self.max_ctx // block)
        self.table = torch.full((R_, self.max_ctx), -9, dtype=torch.int32)   # never read
        self.req = torch.randperm(R_, generator=g)[:len(ctx)]
        perm, at = torch.randperm(n, generator=g).to(torch.int32), 0
        # entries past a context hold what must not be read as a bound
        self.bounds = torch.full((R_, nb, hkv, 2, d), float("nan"), dtype=self.dt)
        for r, m in zip(self.req.tolist(), ctx):
            self.table[r, :m] = perm[at:at + m]
            at += m
            b = R.bounds_of(self.k[self.table[r, :m].long()], block)
            self.bounds[r, :b.shape[0]] = b
        self.q = torch.randn((len(rows), hq, d), generator=g).to(self.dt)

    def call(self, top, sink=1, recent=1, scale=None, ws=None, max_seq=None, stream=None):
        cu = lambda t: t.cuda()  # noqa: E731
        seq = torch.tensor([m for _, m in self.rows], dtype=torch.int32)
        req = self.req[torch.tensor([b for b, _ in self.rows])].to(torch.int32)
        self.top, self.sink, self.recent = top, sink, recent
        self.scale = scale or 1 / math.sqrt(self.d)
        self.max_seq = max_seq or max(1, int(seq.max()))
        q, k = cu(self.q), cu(self.k)
        n = len(self.rows)
        self.o = torch.full((n, self.hq, self.d), 7.0, dtype=self.dt, device="cuda")
        self.lse = torch.full((n, self.hq), 7.0, device="cuda")
        self.sel = torch.full((n, self.hkv, top), 77, dtype=torch.int32, device="cuda")
        need = rc.sparse_decode_workspace_bytes(q, k, max_seq_len=self.max_seq, block=self.block,
                                                top_blocks=top)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        rc.sparse_decode_attention(q, cu(seq), cu(req), cu(self.table), k, cu(self.v),
                                   cu(self.bounds), self.o, ws, sm_scale=self.scale,
                                   max_seq_len=self.max_seq, block=self.block, top_blocks=top,
                                   sink_blocks=sink, recent_blocks=recent, lse=self.lse,
                                   selected=self.sel, stream=stream)
        torch.cuda.synchronize()
        return self

    def check(self, only=None):
        o, lse, sel = self.o.cpu(), self.lse.cpu(), self.sel.cpu()
        for i, (b, m) in enumerate(self.rows):
            if only is not None and i not in only:
                continue
            row = int(self.req[b])
            want = R.select(self.q[i], self.bounds[row], m, self.block, self.top, self.sink,
                            self.recent)
            assert torch.equal(sel[i], want), (i, b, m, sel[i], want)
            ro, rl, to, tl = R.attend(self.q[i], want, m, self.table[row], self.k, self.v,
                                      self.block, self.scale)
            err = (o[i].double() - ro).abs()
            tol = to + R.half_step(self.dt) * (ro.abs() + to)
            assert (err <= tol).all(), (i, m, float(err.max()), float((err - tol).max()))
            fin = rl.isfinite()
            assert torch.equal(lse[i].isfinite(), fin)
            assert ((lse[i].double() - rl).abs()[fin] <= tl[fin]).all(), (i, m)
            assert (lse[i][~fin] == -math.inf).all() and (o[i][~fin] == 0).all()
        return self


SHAPES = [  # dtype, contexts, hq, hkv, d, block, top, sink, recent
    ("bf16", [1], 1, 1, 128, 64, 2, 1, 1),
    ("bf16", [0, 63, 64, 65], 8, 2, 128, 64, 2, 1, 1),
    ("bf16", [0, 0], 4, 4, 64, 32, 3, 0, 1),
    ("bf16", [1000, 129, 700], 32, 8, 128, 64, 5, 1, 2),
    ("bf16", [2049, 40], 8, 8, 128, 64, 7, 0, 1),
    ("bf16", [777], 64, 8, 128, 16, 20, 1, 1),
    ("bf16", [901, 333], 6, 2, 128, 32, 9, 2, 2),
    ("bf16", [1500], 10, 2, 64, 128, 4, 1, 1),
    ("bf16", [1200, 17], 16, 1, 128, 16, 33, 1, 1),
    ("bf16", [1024], 32, 2, 64, 64, 16, 1, 1),
    ("bf16", [3500], 12, 1, 128, 32, 64, 1, 3),
    ("bf16", [5000, 1], 24, 2, 64, 16, 3, 1, 1),
    ("bf16", [9000], 2, 2, 128, 16, 300, 1, 2),
    ("bf16", [130], 4, 1, 128, 16, 2, 1, 1),
    ("f32", [1, 33], 2, 2, 64, 16, 1, 0, 1),
    ("f32", [700, 0, 97], 6, 2, 64, 32, 5, 1, 1),
    ("f32", [1111], 8, 1, 128, 64, 6, 1, 2),
    ("f32", [515], 13, 1, 128, 16, 7, 0, 1),
    ("f32", [260, 260], 4, 4, 128, 128, 2, 1, 1),
    ("f32", [4000], 16, 1, 64, 64, 40, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ctx,hq,hkv,d,block,top,sink,recent", SHAPES)
def test_sparse_decode_matches_the_definition(dtype, ctx, hq, hkv, d, block, top, sink, recent):
    c = Case(dtype, ctx, [(b, m) for b, m in enumerate(ctx)], hq, hkv, d, block)
    c.call(top, sink, recent).check()
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_blocks_than_shared_memory_holds(dtype):
    """Contexts of 130 000 and 70 000 tokens in blocks of 16: the scores live in the workspace. The
    pool is small (slots repeat), the selection is checked over all blocks."""
    g = torch.Generator().manual_seed(7)
    hq, hkv, d, block, n = 2, 1, 64, 16, (130_000, 70_001)
    c = Case(dtype, [600, 300], [(0, n[0]), (1, n[1])], hq, hkv, d, block)
    c.max_ctx = n[0]
    c.table = torch.randint(0, 900, (c.table.shape[0], n[0]), generator=g, dtype=torch.int32)
    nb = -(-n[0] // block)
    c.bounds = torch.randn((c.table.shape[0], nb, hkv, 2, d), generator=g).to(c.dt)
    c.bounds = torch.cat([c.bounds.amin(3, True), c.bounds.amax(3, True)], 3).contiguous()
    q, k = c.q.cuda(), c.k.cuda()
    assert rc.sparse_decode_workspace_bytes(q, k, max_seq_len=n[0], block=block, top_blocks=90) > 0
    c.call(90).check()
    # with a score that is infinite every block is ranked in 64 bits
    c.bounds[:, 77, 0, 1] = float("inf")
    c.call(90).check()
    assert 77 in c.sel[0, 0].tolist() and rc.device_status() == 0
    # the most blocks that shared memory holds: no workspace
    c.rows = [(0, 120_000), (1, 70_001)]
    assert rc.sparse_decode_workspace_bytes(q, k, max_seq_len=120_000, block=block,
                                            top_blocks=90) == 0
    c.call(90).check()
    c.bounds[:, 77, 0, 1] = 1.0
    c.call(90).check()


@pytest.mark.gpu
def test_largest_selection():
    """8192 blocks selected of 12 500: the longest list, and the most tokens of a CTA."""
    g = torch.Generator().manual_seed(8)
    n, block = 200_000, 16
    c = Case("bf16", [600], [(0, n)], 2, 1, 64, block)
    c.max_ctx = n
    c.table = torch.randint(0, 600, (c.table.shape[0], n), generator=g, dtype=torch.int32)
    x = torch.randn((c.table.shape[0], n // block, 1, 2, 64), generator=g).to(c.dt)
    c.bounds = torch.cat([x.amin(3, True), x.amax(3, True)], 3).contiguous()
    c.call(8192).check()
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_many_short_rows_and_calls_on_two_streams_at_once():
    """5000 rows of one short request, and two different calls that may overlap (sizes that need no
    workspace share nothing)."""
    n = 5000
    c = Case("bf16", [90], [(0, 1 + i % 90) for i in range(n)], 4, 2, 64, 16)
    c.call(3).check(only=list(range(0, n, 499)) + [n - 1])
    a = Case("bf16", [2000, 333], [(0, 2000), (1, 333)], 16, 4, 128, 64)
    b = Case("f32", [1500], [(0, 1500), (0, 1490)], 4, 2, 64, 32)
    want = [(x.call(6).o.clone(), x.sel.clone()) for x in (a, b)]
    args = []
    for x in (a, b):
        seq = torch.tensor([m for _, m in x.rows], dtype=torch.int32).cuda()
        req = x.req[torch.tensor([i for i, _ in x.rows])].to(torch.int32).cuda()
        q = x.q.cuda()
        o = [torch.empty_like(q) for _ in range(20)]
        sel = torch.empty((len(x.rows), x.hkv, 6), dtype=torch.int32, device="cuda")
        args.append((x, q, seq, req, x.table.cuda(), x.k.cuda(), x.v.cuda(), x.bounds.cuda(), o, sel))
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for s, (x, q, seq, req, t, k, v, bd, o, sel) in zip(streams, args):
            rc.sparse_decode_attention(q, seq, req, t, k, v, bd, o[i], ws, sm_scale=x.scale,
                                       max_seq_len=x.max_seq, block=x.block, top_blocks=6,
                                       selected=sel, stream=s)
    torch.cuda.synchronize()
    for (w, ws_), (*_, o, sel) in zip(want, args):
        assert all(torch.equal(x, w) for x in o) and torch.equal(sel, ws_)
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("units,top", [(1, 4), (1, 40), (3, 40), (40, 12), (150, 12), (460, 3)])
def test_every_number_of_parts_per_row(units, top):
    """From 16 CTAs per row to one, rows of unlike lengths among them."""
    ctx = [64 * 60 + 13 + 5 * i if i < 3 else 70 + i for i in range(units)]
    c = Case("bf16", ctx, [(b, m) for b, m in enumerate(ctx)], 2, 1, 64, 64)
    c.call(top).check(only=[0, 1, 2, 7, units - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f32", 3, 1, 64)])
def test_chunk_of_new_tokens_is_rows_of_growing_length(dtype, hq, hkv, d):
    """Several rows of one request, and rows of other requests between them; a block's bounds
    already hold the later tokens of the chunk, which may not change what an earlier row takes of
    the blocks before its own."""
    rows = [(0, m) for m in range(190, 201)] + [(1, 64), (1, 65), (0, 3), (1, 0)]
    Case(dtype, [200, 65], rows, hq, hkv, d, 32).call(4).check()
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_all_blocks_selected_is_dense_attention():
    c = Case("bf16", [500], [(0, 500)], 8, 2, 128, 64).call(8).check()
    q = c.q[0].double().view(2, 4, 128)
    slots = c.table[int(c.req[0]), :500].long()
    k, v = c.k[slots].double().transpose(0, 1), c.v[slots].double().transpose(0, 1)
    p = (q @ k.transpose(1, 2) / math.sqrt(128)).softmax(-1)
    ref = (p @ v).view(8, 128)
    # half a step of the output, the weights' 2^-16 and their scores' errors (see cache_ops_ref)
    assert ((c.o[0].cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_scores_take_the_lowest_blocks(dtype):
    """Every key alike: all scores tie exactly, for any order of summation."""
    c = Case(dtype, [640], [(0, 640), (0, 333)], 4, 2, 128, 32)
    c.k[:] = c.k[:1]
    r = int(c.req[0])
    c.bounds[r, :20] = R.bounds_of(c.k[c.table[r, :640].long()], 32)
    c.call(6, sink=0).check()
    assert c.sel[0, 0].tolist() == [0, 1, 2, 3, 4, 19]
    # zero bounds, and zeros of both signs
    c.bounds[r, :20] = 0.0
    c.bounds[r, 5, :, 0] = -0.0
    c.call(6, sink=0).check()
    assert c.sel[0, 1].tolist() == [0, 1, 2, 3, 4, 19]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("step,nb", [(2.0 ** -20, 24), (2.0 ** -40, 24), (2.0 ** -40, 250)])
def test_scores_a_hair_apart_are_told_apart(dtype, step, nb):
    """Blocks whose scores differ by less than an fp32 sum can resolve (one large term and its
    negative cancel, a tiny one decides; in fp32 the order of the sum would choose), or a sum of
    twice that precision, few of them and many."""
    d, block = 128, 16
    c = Case(dtype, [nb * block], [(0, nb * block)], 2, 1, d, block)
    r = int(c.req[0])
    c.q[:] = 0.0
    c.q[0, :, 0] = 1.0
    c.q[0, :, 60] = 1.0
    c.q[0, :, 127] = 1.0
    box = torch.zeros((nb, 1, 2, d))
    box[:, 0, :, 0], box[:, 0, :, 60] = 1024.0, -1024.0
    tiny = torch.randperm(nb, generator=torch.Generator().manual_seed(4)).float()
    box[:, 0, :, 127] = (1 + tiny)[:, None] * step      # 1024 holds 2^-13 at most in fp32
    c.bounds[r, :nb] = box.to(c.dt)
    c.call(9, sink=0).check()
    top = sorted(sorted(range(nb - 1), key=lambda b: -float(tiny[b]))[:8]) + [nb - 1]
    assert c.sel[0, 0].tolist() == top


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q2", [1.0, 2.0 ** -2, 2.0 ** -4, 2.0 ** -7])
def test_scores_closer_than_fp32_sums_are_ranked_exactly(dtype, q2):
    """Hundreds of blocks whose scores agree to 2^-11 .. 2^-20 of the sum of their terms'
    magnitudes, some to the last bit: around and within what fp32 sums of such terms may be off, so
    whatever they say near the border has to be looked at again."""
    d, block, nb, rows = 128, 16, 600, 8
    c = Case(dtype, [nb * block], [(0, nb * block)] * rows, 2, 2, d, block)
    g = torch.Generator().manual_seed(11)
    r = int(c.req[0])
    q = torch.randn(d, generator=g).bfloat16().double()
    q[d - 1], q[d - 2] = 1.0, q2
    x = torch.randn((nb, d), generator=g).bfloat16().double()
    x[:, d - 2:] = 0
    for i in (d - 1, d - 2):     # the last dimensions bring every score near 40, ever nearer
        x[:, i] = ((40.0 - x @ q) / q[i]).bfloat16().double()
    c.q[:] = q.to(c.dt)
    c.q[1::2] *= 0.5             # rows of two scales
    c.bounds[r, :nb] = x[:, None, None].expand(nb, 2, 2, d).to(c.dt)
    c.call(40, sink=0).check()


@pytest.mark.gpu
def test_scores_that_overflow_or_are_no_numbers():
    """Infinite and NaN bounds and finite ones whose fp32 products overflow: NaN and +inf count as
    the largest finite number (lowest block first), -inf as the smallest."""
    d, block, nb = 64, 16, 12
    for dtype in ("bf16", "f32"):
        c = Case(dtype, [nb * block], [(0, nb * block)], 2, 2, d, block)
        r = int(c.req[0])
        c.q[0, :, 3] = 2.0
        c.bounds[r, 7, 0, 1, 3] = float("inf")
        c.bounds[r, 4, 0, 1, 3] = float("nan")
        c.bounds[r, 9, 0, 1, 3] = 3.0e38          # finite in 64 bits, not in 32
        c.bounds[r, 2, 0, 1, 3] = 2.9e38
        c.bounds[r, 1, 1, 1, 3] = -float("inf")
        c.bounds[r, 0, 1, 1, 3] = -3.0e38
        c.call(3, sink=0).check()
        assert c.sel[0, 0].tolist() == [4, 7, 11]
        c.call(4, sink=0).check()
        assert c.sel[0, 0].tolist() == [4, 7, 9, 11]
        c.call(5, sink=0).check()
        c.call(11, sink=0).check()
        assert c.sel[0, 1].tolist() == [0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]


@pytest.mark.gpu
def test_keys_with_infinities_and_nan_behave_as_in_a_dense_softmax():
    for dtype in ("bf16", "f32"):
        c = Case(dtype, [64], [(0, 64)], 2, 2, 64, 16)
        r = int(c.req[0])
        slots = c.table[r, :64].long()
        c.q[0, :, 0] = 1.0
        c.k[slots[5], 0, 0] = -float("inf")       # weight 0: the rest as without it
        c.k[slots[40], 1, 0] = float("nan")       # NaN reaches that head's output alone
        c.call(4)
        o, lse = c.o.cpu(), c.lse.cpu()
        assert o[0, 0].isfinite().all() and o[0, 1].isnan().all() and lse[0, 1].isnan()
        keep = torch.tensor([p for p in range(64) if p != 5])
        s = (c.k[slots[keep], 0].double() @ c.q[0, 0].double()) / 8
        ref = s.softmax(0) @ c.v[slots[keep], 0].double()
        assert ((o[0, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-3).all()
        # every key of a row at -inf: nothing has weight
        c.k[slots, 0, 0] = -float("inf")
        c.call(4)
        assert (c.o.cpu()[0, 0] == 0).all() and c.lse.cpu()[0, 0] == -math.inf
        # every key of a row NaN: nothing is hidden
        c.k[slots, 0] = float("nan")
        c.call(4)
        assert c.o.cpu()[0, 0].isnan().all()
        assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hq,d", [("bf16", 1, 64), ("bf16", 8, 128), ("bf16", 12, 64),
                                        ("bf16", 16, 128), ("f32", 1, 128), ("f32", 3, 64),
                                        ("f32", 16, 128)])
def test_softmax_weights_keep_all_bits_of_fp32(dtype, hq, d):
    """Element i of an output is the difference of the weights of tokens 2 i and 2 i + 1, whose
    scores are near one another or not: what is lost of a weight shows undivided.

    The products q k and their two-term sums are exact in any order (18 bits), so a weight is off
    by: the scale to base 2 (constant, product and, where q is scaled first, the sum: three half
    steps of at most 2.2), the difference from the maximum (half a step of a number below 4: 2^-23),
    0.7 * 8.6 * 2^-24 together by the logarithm's base; exp2f, 2 ulp: 4 * 2^-24. That is 10 * 2^-24
    of it, and half a step more in the sum with its neighbour. Normalisation and the output's
    rounding are relative."""
    n, block = 2 * d + 1, 16
    c = Case(dtype, [n], [(0, n)], hq, 1, d, block, extra=0)
    g = torch.Generator().manual_seed(hq + d)
    slots = c.table[int(c.req[0]), :n].long()
    k, v = torch.zeros((n, d)), torch.zeros((n, d))
    k[:n - 1, 0] = -torch.randint(1, 96, (n - 1,), generator=g) / 64
    k[1:n - 1:2, 0] = k[0:n - 1:2, 0]
    k[:n - 1, 1] = -torch.randint(0, 128, (n - 1,), generator=g) / 64
    i = torch.arange(d)
    v[2 * i, i], v[2 * i + 1, i] = 1.0, -1.0
    c.k[slots, 0], c.v[slots, 0] = k.to(c.dt), v.to(c.dt)
    c.q[:] = 0.0
    c.q[0, :, 0] = 1.0
    c.q[0, :, 1] = 2.0 ** -8 * 2.0 ** -torch.arange(hq).remainder(3).float()
    c.call(n, scale=1.0)
    assert rc.device_status() == 0
    for h in range(hq):
        s = k[:, 0].double() + k[:, 1].double() * c.q[0, h, 1].double()
        p = s.softmax(0)
        ref = p[2 * i] - p[2 * i + 1]
        tol = 11 * R.U32 * (p[2 * i] + p[2 * i + 1]) + (n + 64) * R.U32 * ref.abs()
        tol = tol + R.half_step(c.dt) * (ref.abs() + tol)
        err = (c.o[0, h].double().cpu() - ref).abs()
        assert (err <= tol).all(), (h, float((err / tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hq,d", [("bf16", 2, 64), ("bf16", 12, 128), ("f32", 2, 64),
                                        ("f32", 16, 128)])
def test_values_with_infinities_and_nan(dtype, hq, d):
    """An infinite value gives an infinite output, values of both signs or a NaN give a NaN, in
    their element alone; values past a row's length stay unseen."""
    n = 70
    c = Case(dtype, [n], [(0, n), (0, 33)], hq, 1, d, 16)
    r = int(c.req[0])
    slots = c.table[r, :n].long()
    inf = float("inf")
    c.v[slots[5], 0, 7] = inf
    c.v[slots[31], 0, 8] = -inf
    c.v[slots[6], 0, 9], c.v[slots[7], 0, 9] = inf, -inf
    c.v[slots[8], 0, 10] = float("nan")
    c.v[slots[33:], 0, 11] = inf          # the second row ends before them
    c.call(8)
    for i, m in enumerate((n, 33)):
        ro, rl, to, tl = R.attend(c.q[i], R.select(c.q[i], c.bounds[r], m, 16, 8, 1, 1), m,
                                  c.table[r], c.k, c.v, 16, c.scale)
        o = c.o[i].double().cpu()
        assert (o[:, 7] == inf).all() and (o[:, 8] == -inf).all()
        assert o[:, 9:11].isnan().all()
        assert (o[:, 11] == inf).all() if m > 33 else o[:, 11].isfinite().all()
        fin = ro.isfinite()
        assert torch.equal(fin, o.isfinite())
        tol = to + R.half_step(c.dt) * (ro.abs() + to)
        assert ((o - ro).abs()[fin] <= tol[fin]).all()
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hq,hkv,d,n", [("bf16", 2, 1, 64, 700), ("bf16", 16, 1, 128, 300),
                                              ("f32", 4, 2, 64, 700), ("f32", 16, 1, 128, 300)])
def test_values_near_the_largest_number(dtype, hq, hkv, d, n):
    """Values up to the type's largest, of one sign per dimension and of both: their weighted mean
    is finite, whatever the sum of unnormalised weights would be. Scores grow along the context, so
    that a running maximum lags behind."""
    c = Case(dtype, [n], [(0, n)], hq, hkv, d, 16)
    r = int(c.req[0])
    slots = c.table[r, :n].long()
    c.k[slots, :, 0] = (torch.arange(n) / n * 40)[:, None].to(c.dt)
    c.q[:, :, 0] = 1.0
    for b in range(-(-n // 16)):
        c.bounds[r, b] = R.bounds_of(c.k[slots[16 * b:16 * b + 16]], 16)[0]
    big = torch.rand((n, hkv, d), generator=c.g) * 3e38
    big[:, :, 1::2] *= torch.randn((n, hkv, d // 2), generator=c.g).sign()
    big[3, 0, 0] = torch.finfo(c.dt).max
    c.v[slots] = big.to(c.dt)
    c.call(-(-n // 16)).check()
    assert c.o.isfinite().all() and rc.device_status() == 0


@pytest.mark.gpu
def test_bad_rows_and_slots_are_reported_and_skipped():
    c = Case("bf16", [300, 100], [(0, 300), (1, 100)], 8, 2, 128, 32)
    r = int(c.req[0])
    c.table[r, 299], c.table[r, 3] = c.k.shape[0], -1
    c.call(4, sink=1)
    assert rc.device_status() == 1
    c.check()
    # a row longer than max_seq_len: empty, the other as it was
    c = Case("bf16", [300, 100], [(0, 300), (1, 100)], 8, 2, 128, 32)
    c.call(4, max_seq=120)
    assert rc.device_status() == 2
    assert (c.o[0] == 0).all() and (c.lse[0] == -math.inf).all() and (c.sel[0] == -1).all()
    c.check(only=[1])
    for bad in (-1, 99):
        c = Case("bf16", [300, 100], [(0, 300), (1, 100)], 8, 2, 128, 32)
        keep = c.req.clone()
        c.req[0] = bad
        c.call(4)
        assert rc.device_status() == 2
        assert (c.o[0] == 0).all() and (c.sel[0] == -1).all()
        c.req = keep
        c.check(only=[1])
    # an empty row of a padded batch may name any request
    c = Case("bf16", [300, 100], [(0, 0), (1, 100)], 8, 2, 128, 32)
    keep = c.req.clone()
    c.req[0] = -1
    c.call(4)
    assert rc.device_status() == 0 and (c.o[0] == 0).all() and (c.sel[0] == -1).all()
    c.req = keep
    c.check(only=[1])
    c = Case("bf16", [300, 100], [(0, -4), (1, 100)], 8, 2, 128, 32).call(4)
    assert rc.device_status() == 2 and (c.o[0] == 0).all()
    c.check(only=[1])


@pytest.mark.gpu
def test_workspace_reused_by_other_shapes_graphs_and_streams():
    """One workspace for calls of different shapes in turn, captured and replayed on changed
    inputs, and on a side stream: outputs as of fresh calls, bit for bit."""
    a = Case("bf16", [900, 50], [(0, 900), (1, 50)], 8, 2, 128, 64)
    b = Case("f32", [333], [(0, 333), (0, 332), (0, 331)], 6, 2, 64, 16)
    ws = torch.full((1 << 24,), 170, dtype=torch.uint8, device="cuda")
    want = [x.call(5).check() and (x.o.clone(), x.lse.clone(), x.sel.clone()) for x in (a, b)]
    for _ in range(2):
        for x, w in zip((a, b), want):
            x.call(5, ws=ws)
            assert all(torch.equal(u, v) for u, v in zip((x.o, x.lse, x.sel), w))
    s = torch.cuda.Stream()
    a.call(5, ws=ws, stream=s)
    assert torch.equal(a.o, want[0][0])
    # two graphs on one workspace, replayed one after the other, lengths changed in between
    outs = []
    for x in (a, b):
        q, k, v = x.q.cuda(), x.k.cuda(), x.v.cuda()
        seq = torch.tensor([m for _, m in x.rows], dtype=torch.int32, device="cuda")
        req = x.req[torch.tensor([i for i, _ in x.rows])].to(torch.int32).cuda()
        t, bd = x.table.cuda(), x.bounds.cuda()
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        sel = torch.empty((q.shape[0], x.hkv, 5), dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            rc.sparse_decode_attention(q, seq, req, t, k, v, bd, o, ws, sm_scale=x.scale,
                                       max_seq_len=x.max_seq, block=x.block, top_blocks=5,
                                       lse=lse, selected=sel)
        outs.append((g, seq, q, o, lse, sel, k, v, t, bd, req))
    for turn in range(2):
        for g, *_ in outs:
            g.replay()
        torch.cuda.synchronize()
        for x, (_, seq, q, o, lse, sel, *_) in zip((a, b), outs):
            x.o, x.lse, x.sel = o, lse, sel
            x.check()
            x.rows = [(i, max(0, m - 35)) for i, m in x.rows]
            seq.copy_(torch.tensor([m for _, m in x.rows], dtype=torch.int32))
            x.q = torch.randn(x.q.shape, generator=x.g).to(x.dt)
            q.copy_(x.q)
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_workspace_of_long_rows_reused_by_other_shapes_and_graphs():
    """Two calls whose scores outgrow shared memory, of unlike rows, heads and types, on one
    workspace filled with NaN patterns: in turn, and as two graphs replayed one after the other
    with lengths and queries changed in between. Outputs as of a fresh workspace, bit for bit."""
    def long(dtype, rows, hq, hkv, seed):
        g = torch.Generator().manual_seed(seed)
        n, block, d = max(m for _, m in rows), 16, 64
        c = Case(dtype, [600], rows, hq, hkv, d, block)
        c.max_ctx = n
        c.table = torch.randint(0, 600, (c.table.shape[0], n), generator=g, dtype=torch.int32)
        x = torch.randn((c.table.shape[0], -(-n // block), hkv, 2, d), generator=g).to(c.dt)
        x[:, 100:140, 0] = x[:, 100:101, 0]          # some scores tie
        c.bounds = torch.cat([x.amin(3, True), x.amax(3, True)], 3).contiguous()
        return c

    a = long("bf16", [(0, 125_000), (0, 700), (0, 120_017)], 4, 2, 1)
    b = long("f32", [(0, 140_001), (0, 0)], 3, 1, 2)
    top, cases = 12, (a, b)
    need = [rc.sparse_decode_workspace_bytes(x.q, x.k, max_seq_len=max(m for _, m in x.rows),
                                             block=16, top_blocks=top) for x in cases]
    assert min(need) > 0 and need[0] != need[1]
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")
    want = [x.call(top).check() and (x.o.clone(), x.lse.clone(), x.sel.clone()) for x in cases]
    for _ in range(2):
        for x, w in zip(cases, want):
            x.call(top, ws=ws)
            assert all(torch.equal(u, v) for u, v in zip((x.o, x.lse, x.sel), w))
    graphs = []
    for x in cases:
        keep = [t.cuda() for t in (x.q, x.table, x.k, x.v, x.bounds)]
        q, t, k, v, bd = keep
        seq = torch.tensor([m for _, m in x.rows], dtype=torch.int32, device="cuda")
        req = x.req[torch.zeros(len(x.rows), dtype=torch.long)].to(torch.int32).cuda()
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        sel = torch.empty((q.shape[0], x.hkv, top), dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            rc.sparse_decode_attention(q, seq, req, t, k, v, bd, o, ws, sm_scale=x.scale,
                                       max_seq_len=x.max_seq, block=16, top_blocks=top, lse=lse,
                                       selected=sel)
        graphs.append((g, keep, seq, req, o, lse, sel))
    for _ in range(2):
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, (_, keep, seq, _, o, lse, sel) in zip(cases, graphs):
            x.o, x.lse, x.sel = o, lse, sel
            x.check()
            x.rows = [(i, max(0, m - 3333)) for i, m in x.rows]
            seq.copy_(torch.tensor([m for _, m in x.rows], dtype=torch.int32))
            x.q = torch.randn(x.q.shape, generator=x.g).to(x.dt)
            keep[0].copy_(x.q)
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool plane of more than 2^31 elements and a bounds table of more than 2^31 elements; the
    request uses their far ends."""
    hkv, d, block, n = 8, 128, 64, 500
    slots = (1 << 31) // (hkv * d) + 1000
    rows, nb = 70, 16384
    k = torch.zeros((slots, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    bd = torch.zeros((rows, nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 1 << 31 and bd.numel() > 1 << 31
    c = Case("bf16", [n], [(0, n)], 16, hkv, d, block, extra=0)
    far = torch.arange(slots - n, slots, device="cuda")
    k[far], v[far] = c.k.cuda(), c.v.cuda()
    table = torch.zeros((rows, 1 << 20), dtype=torch.int32, device="cuda")
    table[rows - 1, :n] = (c.table[int(c.req[0]), :n] + (slots - n)).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rc.kv_block_bounds(k, table, i32([rows - 1]), i32([n]), bd, block=block)
    c.o = torch.empty_like(c.q, device="cuda")
    c.lse = torch.empty((1, 16), device="cuda")
    c.sel = torch.empty((1, hkv, 4), dtype=torch.int32, device="cuda")
    need = rc.sparse_decode_workspace_bytes(c.o, k, max_seq_len=n, block=block, top_blocks=4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc.sparse_decode_attention(c.q.cuda(), i32([n]), i32([rows - 1]), table, k, v, bd, c.o, ws,
                               sm_scale=1 / math.sqrt(d), max_seq_len=n, block=block,
                               top_blocks=4, lse=c.lse, selected=c.sel)
    c.top, c.sink, c.recent, c.scale = 4, 1, 1, 1 / math.sqrt(d)
    c.check()
    assert rc.device_status() == 0


@pytest.mark.gpu
def test_sparse_decode_refusals():
    c = Case("bf16", [100], [(0, 100)], 8, 2, 128, 64).call(2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k = c.k.cuda()
    need = rc.sparse_decode_workspace_bytes(c.o, k, max_seq_len=100, block=64, top_blocks=2)
    ok = dict(q=c.q.cuda(), seq_len=i32([100]), req_idx=i32([int(c.req[0])]),
              req_to_token=c.table.cuda(), k_pool=k, v_pool=c.v.cuda(), bounds=c.bounds.cuda(),
              o=c.o, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), sm_scale=0.1,
              max_seq_len=100, block=64, top_blocks=2)
    rc.sparse_decode_attention(**ok)
    for bad in (dict(q=c.q), dict(q=ok["q"][:, :, :64]), dict(o=c.o[:, :4]),
                dict(v_pool=ok["v_pool"][1:]), dict(bounds=ok["bounds"][:, :, :1]),
                dict(bounds=ok["bounds"][:1]), dict(seq_len=i32([1, 2])), dict(req_idx=i32([])),
                dict(lse=torch.zeros((1, 2), device="cuda")), dict(selected=c.sel[:, :, :1]),
                dict(req_to_token=ok["req_to_token"][:, ::2]),
                dict(workspace=ok["workspace"].cpu())):
        with pytest.raises(ValueError):
            rc.sparse_decode_attention(**{**ok, **bad})
    for bad in (dict(q=ok["q"].float()), dict(seq_len=ok["seq_len"].long()),
                dict(lse=torch.zeros((1, 8), device="cuda", dtype=torch.float64)),
                dict(bounds=ok["bounds"].float())):
        with pytest.raises(TypeError):
            rc.sparse_decode_attention(**{**ok, **bad})
    for bad in (dict(max_seq_len=200), dict(top_blocks=1), dict(block=65), dict(sm_scale=0.0)):
        with pytest.raises(rc.RcError) as e:
            rc.sparse_decode_attention(**{**ok, **bad})
        assert e.value.code == rc.RC_ERR_INVALID
