"""Cases of the operators around the paged cache: norms and rotation of queries and keys, appending
to the cache, block bounds of cached keys, and decode attention over the blocks that they select.

A case is a dict of plain values; `op` names the operator. `run` computes it with the package when
`own` is true and with elementary torch operations otherwise."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a handful of users, 32 query and 8 KV heads: latency only
        dict(name="norm_rope_step", op="norm_rope", dtype="bf16", tokens=8, hq=32, hkv=8, d=128,
             rot=128, inter=False, norm=True, ctx=16384),
        # the computed tokens of a fork step, 16 programs x 5 forks x 200 tokens, 32 heads
        dict(name="norm_rope_fork", op="norm_rope", dtype="bf16", tokens=16000, hq=32, hkv=32,
             d=128, rot=128, inter=False, norm=True, ctx=8192),
        # fp32, an odd head group, half of each head rotated, interleaved pairs
        dict(name="norm_rope_f32", op="norm_rope", dtype="f32", tokens=2311, hq=6, hkv=2, d=64,
             rot=32, inter=True, norm=True, ctx=4099),
        # 256 requests of a multi-turn batch append one token each; their block bounds follow
        dict(name="append_step", op="append", dtype="bf16", reqs=256, new_lo=1, new_hi=1, pre_lo=128,
             pre_hi=16300, pad=0, hkv=8, d=128, rot=128, inter=False, norm=True, bounds=True,
             block=64, ctx=16384, slots=65536),
        # the same fork step's keys and values, 80 forks behind a prefix of 1500 tokens
        dict(name="append_fork", op="append", dtype="bf16", reqs=80, new_lo=200, new_hi=200,
             pre_lo=1500, pre_hi=1500, pad=0, hkv=32, d=128, rot=128, inter=False, norm=True,
             bounds=True, block=64, ctx=2048, slots=32768),
        # fp32 prompts of odd lengths into empty and started rows, padded batch, no bounds
        dict(name="append_f32", op="append", dtype="f32", reqs=7, new_lo=0, new_hi=613, pre_lo=0,
             pre_hi=97, pad=13, hkv=2, d=64, rot=64, inter=True, norm=False, bounds=False, block=64,
             ctx=1001, slots=4096),
        # the bounds of a whole multi-turn batch's contexts, as decoding begins
        dict(name="bounds_multi_turn", op="bounds", dtype="bf16", reqs=256, len_lo=128,
             len_hi=16384, hkv=8, d=128, block=64, ctx=16384),
        # a few short fp32 contexts, one of them empty
        dict(name="bounds_f32", op="bounds", dtype="f32", reqs=5, len_lo=0, len_hi=301, hkv=2, d=64,
             block=32, ctx=320),
        # one user with a very long context, 64 query and 8 KV heads: latency of a single row
        dict(name="sparse_one_long", op="sparse", dtype="bf16", reqs=1, chunk=1, len_lo=131071,
             len_hi=131071, hq=64, hkv=8, d=128, block=64, top=64, sink=1, recent=2, ctx=131072),
        # decode of the fork step: 128 requests, contexts 512..8192, 32 heads, 16 blocks each
        dict(name="sparse_fork", op="sparse", dtype="bf16", reqs=128, chunk=1, len_lo=512,
             len_hi=8192, hq=32, hkv=32, d=128, block=64, top=16, sink=1, recent=1, ctx=8192),
        # long documents: 64 requests, 4096..32768 tokens, 32 query and 8 KV heads, 64 blocks each
        dict(name="sparse_long_batch", op="sparse", dtype="bf16", reqs=64, chunk=1, len_lo=4096,
             len_hi=32768, hq=32, hkv=8, d=128, block=64, top=64, sink=1, recent=2, ctx=32768),
        # fp32, chunks of 11 new tokens, an odd head group, an empty row, small blocks
        dict(name="sparse_chunk_f32", op="sparse", dtype="f32", reqs=5, chunk=11, len_lo=0,
             len_hi=1503, hq=6, hkv=2, d=64, block=32, top=9, sink=1, recent=1, ctx=1600),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "bounds", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    inter = rng.random() < 0.4
    if op == "norm_rope":
        g = rng.choice([1, 2, 3, 4, 6, 8])
        hkv = min(hkv, 8) if g > 1 else hkv
        d = rng.choice([64, 80, 96, 128, 192, 256])
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 6000), hq=g * hkv, hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2 // 16 * 16]), inter=inter, norm=rng.random() < 0.8,
                    ctx=_log(rng, 64, 32768))
    block = rng.choice([16, 32, 64, 128])
    if op == "append":
        reqs = _log(rng, 1, 300)
        new = _log(rng, 1, max(2, 12000 // reqs))
        lo = rng.choice([new, new // 2, 0])
        pre = _log(rng, 1, 8192)
        bounds = rng.random() < 0.7
        return dict(op=op, dtype=dtype, reqs=reqs, new_lo=lo, new_hi=max(new, 1), pre_lo=pre // 3,
                    pre_hi=pre, pad=rng.choice([0, 0, 5]), hkv=hkv, d=d, rot=rng.choice([d, 32]),
                    inter=inter, norm=rng.random() < 0.5, bounds=bounds, block=block,
                    ctx=pre + new + rng.randrange(64), slots=reqs * max(new, 1) + rng.randrange(8, 999))
    es = ES[dtype]
    if op == "bounds":
        n = _log(rng, 1, 200)
        top = max(2, min(20000, int(1.2e9 / (n * hkv * d * es))))
        hi = _log(rng, 1, top)
        return dict(op=op, dtype=dtype, reqs=n, len_lo=rng.choice([0, hi // 3, hi]), len_hi=hi,
                    hkv=hkv, d=d, block=block, ctx=hi + rng.randrange(100))
    g = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    hkv = min(hkv, 32 // g)
    n = _log(rng, 1, 96)
    chunk = rng.choice([1, 1, 1, _log(rng, 2, 16)]) if n <= 4 else 1
    top = max(64, min(60000, int(0.8e9 / (n * hkv * d * es))))
    hi = _log(rng, 64, top)
    return dict(op=op, dtype=dtype, reqs=n, chunk=chunk, len_lo=rng.choice([0, hi // 4, hi]),
                len_hi=hi, hq=g * hkv, hkv=hkv, d=d, block=block, top=rng.randrange(3, 4097 // block),
                sink=rng.choice([0, 1, 1]), recent=rng.choice([1, 1, 2]),
                ctx=hi + chunk + rng.randrange(50))


# ---------------------------------------------------------------------------------- their sizes
def _lens(case, lo, hi, n, salt):
    """n lengths between lo and hi, of the case alone (both ends among them); over a wide range
    short ones are as common as long ones."""
    r = random.Random("%s %d %d %d %d" % (case["op"], salt, lo, hi, n))
    got = [_log(r, lo, hi) if hi > 64 * lo > 0 else r.randint(lo, hi) for _ in range(n)]
    got[0] = hi
    if n > 1:
        got[1] = lo
    return got


def _new(case):
    return _lens(case, case["new_lo"], case["new_hi"], case["reqs"], 1)


def _pre(case):
    return _lens(case, case["pre_lo"], case["pre_hi"], case["reqs"], 2)


def _ctx(case):
    return _lens(case, case["len_lo"], case["len_hi"], case["reqs"], 3)


def _rows(case):
    """(request, visible tokens) of each query row: a request's chunk ends at its length."""
    out = []
    for b, n in enumerate(_ctx(case)):
        out += [(b, max(0, n - case["chunk"] + 1 + i)) for i in range(case["chunk"])]
    return out


def work(case):
    es, d = ES[case["dtype"]], case["d"]
    if case["op"] == "norm_rope":
        x = case["tokens"] * (case["hq"] + case["hkv"]) * d
        table = min(case["tokens"], case["ctx"]) * case["rot"] * 4
        return {"bytes": 2 * x * es + 4 * case["tokens"] + table + 2 * d * es, "flops": 7 * x}
    if case["op"] == "append":
        new, pre = _new(case), _pre(case)
        t, row = sum(new), case["hkv"] * d
        n = 4 * t * row * es + 4 * t + min(t, case["ctx"]) * case["rot"] * 4
        if case["bounds"]:
            blk = case["block"]
            for s, p in zip(new, pre):
                if s:
                    touched = (p + s - 1) // blk - p // blk + 1
                    n += (touched + (1 if p % blk else 0)) * 2 * row * es
        return {"bytes": n, "flops": 8 * t * row}
    if case["op"] == "bounds":
        lens, row = _ctx(case), case["hkv"] * d
        blocks = sum(-(-n // case["block"]) for n in lens)
        return {"bytes": sum(lens) * (row * es + 4) + blocks * 2 * row * es,
                "flops": 2 * sum(lens) * row}
    blk, n, f = case["block"], 0, 0
    by_req = {}
    for b, m in _rows(case):
        nb = -(-m // blk)
        sel = m if nb <= case["top"] else (case["top"] - 1) * blk + (m - (nb - 1) * blk)
        f += case["hq"] * d * (4 * nb + 4 * sel)
        n += 2 * case["hq"] * d * es + 4 * case["hq"] + 4 * case["hkv"] * case["top"] + 8
        got = by_req.setdefault(b, [0, 0, 0])
        got[0], got[1], got[2] = max(got[0], nb), max(got[1], m), got[2] + sel
    for nb, m, sel in by_req.values():   # rows of one request may read the same tokens
        n += nb * case["hkv"] * 2 * d * es + min(m, sel) * case["hkv"] * (2 * d * es) + 4 * min(m, sel)
    return {"bytes": n, "flops": f}


# ---------------------------------------------------------------------------------- inputs
def _rope(case, positions):
    """cos and sin of every position, [positions, rot] (cos of the pairs, then sin), from 64 bits."""
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = DT[case["dtype"]], case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def weight():   # a learned weight of a norm
        return (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)

    s = {"case": case}
    if case["op"] == "norm_rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        qkv = randn(t, hq + 2 * hkv, d)   # the fused projection's output; q and k are views of it
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["positions"] = torch.randint(0, case["ctx"], (t,), generator=g, device="cuda",
                                       dtype=torch.int32)
        s["rope"] = _rope(case, case["ctx"])
        s["wq"], s["wk"] = (weight(), weight()) if case["norm"] else (None, None)
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((t, hkv, d), dtype=dt, device="cuda")
        return s
    hkv, blk = case["hkv"], case["block"]
    nb = -(-case["ctx"] // blk)
    if case["op"] == "append":
        new, pre = _new(case), _pre(case)
        s["total"] = sum(new)
        t = s["total"] + case["pad"]
        kv = randn(t, 2 * hkv, d)
        s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
        perm = torch.randperm(case["slots"], generator=g, device="cuda")[:t]
        s["out_loc"] = perm.to(torch.int32)
        s["qo_indptr"] = _i32([sum(new[:i]) for i in range(len(new) + 1)])
        s["prefix_len"] = _i32(pre)
        s["k_pool"], s["v_pool"] = randn(case["slots"], hkv, d), randn(case["slots"], hkv, d)
        s["rope"] = _rope(case, case["ctx"])
        s["w"] = weight() if case["norm"] else None
        if case["bounds"]:
            s["req_idx"] = torch.randperm(case["reqs"], generator=g, device="cuda").to(torch.int32)
            x = randn(case["reqs"], nb, hkv, 2, d)
            x[:, :, :, 0].abs_().neg_()
            x[:, :, :, 1].abs_()
            s["bounds"] = x
        return s
    # contexts in token slots scattered over the pool
    lens = _ctx(case)
    total = sum(lens)
    slots = total + 64
    k = randn(slots, hkv, d)
    perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    req = torch.randperm(case["reqs"], generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["reqs"], case["ctx"]), dtype=torch.int32, device="cuda")
    bounds = torch.zeros((case["reqs"], nb, hkv, 2, d), dtype=dt, device="cuda")
    rows, at = req.tolist(), 0
    for b, n in enumerate(lens):
        mine = perm[at:at + n]
        at += n
        table[rows[b], :n] = mine
        if case["op"] == "sparse" and n:
            # neighbouring tokens have keys alike, so that some blocks matter to a query
            m = -(-n // blk)
            near = 0.6 * randn(m, 1, hkv, d).expand(m, blk, hkv, d).reshape(m * blk, hkv, d)[:n]
            x = 0.8 * k[mine.long()] + near
            k[mine.long()] = x
            pad = m * blk - n
            x = torch.cat([x, x[-1:].expand(pad, hkv, d)]) if pad else x
            x = x.view(m, blk, hkv, d)
            bounds[rows[b], :m, :, 0] = x.amin(1)
            bounds[rows[b], :m, :, 1] = x.amax(1)
    s.update(k_pool=k, table=table, bounds=bounds)
    if case["op"] == "bounds":
        s.update(req_idx=req, seq_len=_i32(lens), total=total)
        return s
    which = _rows(case)
    s["q"] = randn(len(which), case["hq"], d)
    s["v_pool"] = randn(slots, hkv, d)
    s["req_idx"] = req[torch.tensor([b for b, _ in which], device="cuda")]
    s["seq_len"] = _i32([m for _, m in which])
    s["max_seq"] = max(m for _, m in which)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((len(which), case["hq"]), dtype=torch.float32, device="cuda")
    s["selected"] = torch.empty((len(which), hkv, case["top"]), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------- plain forms
def _norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, rope, positions, inter):
    half = rope.shape[1] // 2
    c = rope[positions, :half][:, None]
    n = rope[positions, half:][:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else \
        (x[..., :half], x[..., half:2 * half])
    p, q = a * c - b * n, b * c + a * n
    y = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_norm_rope(s):
    case = s["case"]
    at = s["positions"].long()
    return [_rotate(_norm(x.float(), w), s["rope"], at, case["inter"]).to(x.dtype)
            for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"]))]


def _tokens_of(s):
    """Request and position of each token that the batch's offsets cover."""
    t = torch.arange(s["total"], device="cuda")
    ip = s["qo_indptr"].long()
    b = torch.searchsorted(ip[1:].contiguous(), t, right=True)
    return b, s["prefix_len"].long()[b] + t - ip[b]


def _plain_append(s):
    case, n = s["case"], s["total"]
    b, pos = _tokens_of(s)
    k = _rotate(_norm(s["k"][:n].float(), s["w"]), s["rope"], pos, case["inter"])
    k = k.to(s["k"].dtype)
    at = s["out_loc"][:n].long()
    s["k_pool"][at] = k
    s["v_pool"][at] = s["v"][:n]
    if not case["bounds"]:
        return [s["k_pool"], s["v_pool"]]
    x = s["bounds"]
    r, nb, h, _, d = x.shape
    cell = s["req_idx"].long()[b] * nb + pos // case["block"]
    fresh = cell[pos // case["block"] * case["block"] >= s["prefix_len"].long()[b]]
    kf = k.float().view(n, h * d)
    for i, (how, empty) in enumerate((("amin", math.inf), ("amax", -math.inf))):
        part = x[:, :, :, i].reshape(r * nb, h * d).float()
        part[fresh] = empty
        part.index_reduce_(0, cell, kf, how)
        x[:, :, :, i] = part.view(r, nb, h, d).to(x.dtype)
    return [s["k_pool"], s["v_pool"], x]


def _plain_bounds(s):
    case, x = s["case"], s["bounds"]
    r, nb, h, _, d = x.shape
    t = torch.arange(s["total"], device="cuda")
    end = s["seq_len"].long().cumsum(0)
    b = torch.searchsorted(end, t, right=True)
    pos = t - (end - s["seq_len"].long())[b]
    row = s["req_idx"].long()[b]
    k = s["k_pool"][s["table"][row, pos].long()].float().view(-1, h * d)
    cell = row * nb + pos // case["block"]
    for i, (how, empty) in enumerate((("amin", math.inf), ("amax", -math.inf))):
        part = x[:, :, :, i].reshape(r * nb, h * d).float()
        part[cell] = empty
        part.index_reduce_(0, cell, k, how)
        x[:, :, :, i] = part.view(r, nb, h, d).to(x.dtype)
    return [x]


def _select(case, q, box, seq_len):
    """Blocks of each query row and KV head: 64-bit scores, since near a border 32 bits choose
    another block. q [n, h, g, d], box [n, nb, h, 2, d]."""
    blk, nb = case["block"], box.shape[1]
    q = q.double()
    lo, hi = box[:, :, :, 0].double().permute(0, 2, 3, 1), box[:, :, :, 1].double().permute(0, 2, 3, 1)
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)            # [n, h, nb]
    top = torch.finfo(torch.float64).max
    score = torch.nan_to_num(score, nan=top, posinf=top, neginf=-top)
    i = torch.arange(nb, device="cuda")
    have = ((seq_len + blk - 1) // blk)[:, None]
    forced = (i < case["sink"]) | (i >= have - case["recent"])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((i < have)[:, None], score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :case["top"]]
    order = torch.where(order < have[:, None], order, nb)
    order = order.sort(-1).values
    order = torch.where(order < nb, order, -1)
    short = case["top"] - order.shape[-1]
    return torch.nn.functional.pad(order, (0, short), value=-1) if short > 0 else order


def _plain_sparse(s):
    case = s["case"]
    n, hq, d = s["q"].shape
    h, blk = case["hkv"], case["block"]
    row, seq = s["req_idx"].long(), s["seq_len"].long()
    q = s["q"].view(n, h, hq // h, d)
    sel = _select(case, q, s["bounds"][row], seq)
    pos = (sel[..., None] * blk + torch.arange(blk, device="cuda")).flatten(2)
    real = (sel >= 0).repeat_interleave(blk, 2) & (pos < seq[:, None, None])
    slot = s["table"][row[:, None, None], torch.where(real, pos, 0)].long()
    head = torch.arange(h, device="cuda")[None, :, None]
    k, v = s["k_pool"][slot, head].float(), s["v_pool"][slot, head].float()
    logit = (q.float() / math.sqrt(d)) @ k.transpose(2, 3)
    logit = torch.where(real[:, :, None], logit, -math.inf)
    m = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(m == -math.inf, 0, m))
    den = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(den == 0, 1, den)
    return [o.view(n, hq, d).to(s["q"].dtype), (m + den.log()).view(n, hq), sel.to(torch.int32)]


# ---------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "append": _plain_append, "bounds": _plain_bounds,
                "sparse": _plain_sparse}[case["op"]](s)
    import prefix_cached_paged_gb300 as rc
    if case["op"] == "norm_rope":
        rc.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], q_weight=s["wq"],
                        k_weight=s["wk"], eps=EPS, interleaved=case["inter"], q_out=s["q_out"],
                        k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if case["op"] == "append":
        if not case["bounds"]:
            rc.kv_append(s["k"], s["v"], s["out_loc"], s["qo_indptr"], s["prefix_len"],
                         s["k_pool"], s["v_pool"], rope=s["rope"], k_weight=s["w"], eps=EPS,
                         interleaved=case["inter"])
            return [s["k_pool"], s["v_pool"]]
        rc.kv_append(s["k"], s["v"], s["out_loc"], s["qo_indptr"], s["prefix_len"], s["k_pool"],
                     s["v_pool"], rope=s["rope"], k_weight=s["w"], eps=EPS,
                     interleaved=case["inter"], bounds=s["bounds"], req_idx=s["req_idx"],
                     block=case["block"])
        return [s["k_pool"], s["v_pool"], s["bounds"]]
    if case["op"] == "bounds":
        rc.kv_block_bounds(s["k_pool"], s["table"], s["req_idx"], s["seq_len"], s["bounds"],
                           block=case["block"])
        return [s["bounds"]]
    if "workspace" not in s:
        need = rc.sparse_decode_workspace_bytes(s["q"], s["k_pool"], max_seq_len=s["max_seq"],
                                                block=case["block"], top_blocks=case["top"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc.sparse_decode_attention(s["q"], s["seq_len"], s["req_idx"], s["table"], s["k_pool"],
                               s["v_pool"], s["bounds"], s["o"], s["workspace"],
                               sm_scale=1.0 / math.sqrt(case["d"]), max_seq_len=s["max_seq"],
                               block=case["block"], top_blocks=case["top"],
                               sink_blocks=case["sink"], recent_blocks=case["recent"],
                               lse=s["lse"], selected=s["selected"])
    return [s["o"], s["lse"], s["selected"]]


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_rows(x, w, rope, positions, inter):
    """Norm and rotation as a product of complex numbers."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    half = rope.shape[1] // 2
    turn = torch.complex(rope[:, :half].double(), rope[:, half:].double())[positions][:, None]
    t, h, d = x.shape
    y = x.clone()
    if inter:
        z = torch.view_as_complex(x[..., :2 * half].reshape(t, h, half, 2)) * turn
        y[..., :2 * half] = torch.view_as_real(z).flatten(2)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        at = s["positions"].long()
        return [_exact_rows(x, w, s["rope"], at, case["inter"])
                for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"]))]
    if case["op"] == "append":
        new, pre, n = _new(case), _pre(case), s["total"]
        at = torch.tensor([p + i for c, p in zip(new, pre) for i in range(c)], device="cuda",
                          dtype=torch.long)
        k = _exact_rows(s["k"][:n], s["w"], s["rope"], at, case["inter"])
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        loc = s["out_loc"][:n].long()
        kp[loc], vp[loc] = k, s["v"][:n].double()
        if not case["bounds"]:
            return [kp, vp]
        x, blk, t = s["bounds"].double(), case["block"], 0
        for row, c, p in zip(s["req_idx"].tolist(), new, pre):
            i = 0
            while i < c:   # the part of the new tokens that lies in one block
                b = (p + i) // blk
                j = min(c, (b + 1) * blk - p)
                part = k[t + i:t + j]
                lo, hi = part.amin(0), part.amax(0)
                if b * blk < p:
                    lo, hi = torch.minimum(lo, x[row, b, :, 0]), torch.maximum(hi, x[row, b, :, 1])
                x[row, b, :, 0], x[row, b, :, 1] = lo, hi
                i = j
            t += c
        return [kp, vp, x]
    if case["op"] == "bounds":
        x, blk = s["bounds"].double(), case["block"]
        for row, n in zip(s["req_idx"].tolist(), _ctx(case)):
            if n:
                k = s["k_pool"][s["table"][row, :n].long()]
                m = -(-n // blk)
                k = torch.cat([k, k[-1:].expand(m * blk - n, -1, -1)]) if m * blk > n else k
                k = k.view(m, blk, *k.shape[1:])
                x[row, :m, :, 0], x[row, :m, :, 1] = k.amin(1).double(), k.amax(1).double()
        return [x]
    rows = _rows(case)
    hq, h, d, blk, top = case["hq"], case["hkv"], case["d"], case["block"], case["top"]
    o = torch.zeros((len(rows), hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((len(rows), hq), -math.inf, dtype=torch.float64, device="cuda")
    sel = torch.full((len(rows), h, top), -1, dtype=torch.int32, device="cuda")
    for i, ((_, n), row) in enumerate(zip(rows, s["req_idx"].tolist())):
        if n == 0:
            continue
        m = -(-n // blk)
        q = s["q"][i].double().view(h, hq // h, d)
        box = s["bounds"][row, :m].double()                                  # [m, h, 2, d]
        best = torch.maximum(q[:, :, None] * box[:, :, 0].transpose(0, 1)[:, None],
                             q[:, :, None] * box[:, :, 1].transpose(0, 1)[:, None])
        score = best.sum(-1).amax(1)                                         # [h, m]
        score[:, :case["sink"]] = math.inf
        score[:, max(0, m - case["recent"]):] = math.inf
        pick = score.argsort(dim=1, descending=True, stable=True)[:, :top].sort(1).values
        sel[i, :, :pick.shape[1]] = pick.to(torch.int32)
        pos = (pick[..., None] * blk + torch.arange(blk, device="cuda")).flatten(1)
        real = pos < n
        slot = s["table"][row, torch.where(real, pos, 0)].long()
        head = torch.arange(h, device="cuda")[:, None]
        k, v = s["k_pool"][slot, head].double(), s["v_pool"][slot, head].double()
        logit = (q @ k.transpose(1, 2)) / math.sqrt(d)
        logit = logit.masked_fill(~real[:, None], -math.inf)
        o[i] = (logit.softmax(-1) @ v).view(hq, d)
        lse[i] = logit.logsumexp(-1).view(hq)
    return [o, lse, sel]
