"""Cases of the paged cache held in 4 bits: keys and values quantised as they are written into their
slots, read back as numbers, and decode attention over the cached tokens as they are held.

Of every head's elements, 32 neighbours make a group with a scale and a minimum, both bf16; an element
is held as a code of 0 to 15 and stands for code * scale + minimum. A head takes d * 5 / 8 bytes of a
slot: d / 2 of codes (element 32 j + 8 t + n is nibble n of the little-endian 32-bit word t * d / 32 + j),
then scale and minimum of each group.

A case is a dict of plain values; `op` names the operator. `run` computes it with the package when
`own` is true and with elementary torch operations otherwise."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a handful of users, 8 KV heads, written and read back: latency only
        dict(name="write_step", op="write", dtype="bf16", reqs=8, new_lo=1, new_hi=1, pad=0, hkv=8,
             d=128, slots=4096),
        # the computed tokens of a fork step, 80 forks x 200 tokens, 32 heads, as they are cached and
        # as later steps will see them
        dict(name="write_fork", op="write", dtype="bf16", reqs=80, new_lo=200, new_hi=200, pad=0,
             hkv=32, d=128, slots=32768),
        # fp32 prompts of odd lengths, a padded batch, slices of a fused projection
        dict(name="write_f32", op="write", dtype="f32", reqs=7, new_lo=0, new_hi=613, pad=13, hkv=2,
             d=64, slots=4096),
        # the cached prefixes of the fork step's 16 programs, read for the extend attention
        dict(name="read_prefix", op="read", dtype="bf16", tokens=24000, scatter=False, hkv=32, d=128,
             slots=30000),
        # fp32, three heads, into slots of other planes, whose other rows stay
        dict(name="read_f32", op="read", dtype="f32", tokens=1001, scatter=True, hkv=3, d=64,
             slots=2048),
        # four users with short contexts: latency only
        dict(name="decode_step", op="decode", dtype="bf16", reqs=4, chunk=1, len_lo=97, len_hi=700,
             hq=32, hkv=8, d=128, ctx=1024),
        # one user with a very long context, 64 query and 8 KV heads
        dict(name="decode_one_long", op="decode", dtype="bf16", reqs=1, chunk=1, len_lo=131071,
             len_hi=131071, hq=64, hkv=8, d=128, ctx=131072),
        # decode of the fork step: 128 requests, contexts 512..8192, 32 heads
        dict(name="decode_fork", op="decode", dtype="bf16", reqs=128, chunk=1, len_lo=512,
             len_hi=8192, hq=32, hkv=32, d=128, ctx=8192),
        # a multi-turn batch: 256 requests of 128..16384 tokens, 32 query and 8 KV heads
        dict(name="decode_multi_turn", op="decode", dtype="bf16", reqs=256, chunk=1, len_lo=128,
             len_hi=16384, hq=32, hkv=8, d=128, ctx=16384),
        # long documents, 16 query heads for each KV head
        dict(name="decode_long_batch", op="decode", dtype="bf16", reqs=64, chunk=1, len_lo=4096,
             len_hi=32768, hq=64, hkv=4, d=128, ctx=32768),
        # fp32, chunks of 11 new tokens, an odd head group, an empty row
        dict(name="decode_chunk_f32", op="decode", dtype="f32", reqs=5, chunk=11, len_lo=0,
             len_hi=1503, hq=6, hkv=2, d=64, ctx=1600),
        # a layer of a decode step: the new token's key and value written, then attention; 96 requests,
        # heads of 64
        dict(name="step_layer", op="step", dtype="bf16", reqs=96, chunk=1, len_lo=33, len_hi=2048,
             hq=16, hkv=4, d=64, ctx=2304),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "decode", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 12, 16, 32])
    if op in ("write", "read"):
        d = rng.choice([64, 128, 128, 192, 256])
        most = int(4e7 / (hkv * d))
        if op == "read":
            n = _log(rng, 1, most)
            return dict(op=op, dtype=dtype, tokens=n, scatter=rng.random() < 0.4, hkv=hkv, d=d,
                        slots=n + rng.randrange(1, 999))
        reqs = _log(rng, 1, 300)
        new = _log(rng, 1, max(2, most // reqs))
        return dict(op=op, dtype=dtype, reqs=reqs, new_lo=rng.choice([new, new // 2, 0]), new_hi=new,
                    pad=rng.choice([0, 0, 5]), hkv=hkv, d=d,
                    slots=reqs * new + rng.randrange(8, 999))
    d = rng.choice([64, 128])
    g = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
    hkv = max(h for h in (1, 2, 3, 4, 5, 6, 8, 12, 16, 32) if h <= hkv and h * g <= 64)
    n = _log(rng, 1, 256)
    chunk = _log(rng, 2, 16) if op == "decode" and n <= 6 and rng.random() < 0.4 else 1
    top = max(64, min(131072, int(1.2e9 / (n * chunk * hkv * d))))
    hi = _log(rng, 16, top)
    return dict(op=op, dtype=dtype, reqs=n, chunk=chunk,
                len_lo=rng.choice([op == "step" and 1 or 0, max(1, hi // 8), hi]), len_hi=hi, hq=g * hkv,
                hkv=hkv, d=d, ctx=hi + chunk + rng.randrange(50))


# ---------------------------------------------------------------------------------- their sizes
def _lens(case, lo, hi, n, salt):
    """n lengths between lo and hi, of the case alone (both ends among them); over a wide range
    short ones are as common as long ones."""
    r = random.Random("%s %d %d %d %d" % (case["op"], salt, lo, hi, n))
    got = [_log(r, lo, hi) if hi > 8 * lo > 0 else r.randint(lo, hi) for _ in range(n)]
    got[0] = hi
    if n > 1:
        got[1] = lo
    return got


def _new(case):
    return _lens(case, case["new_lo"], case["new_hi"], case["reqs"], 1)


def _ctx(case):
    return _lens(case, case["len_lo"], case["len_hi"], case["reqs"], 3)


def _rows(case):
    """(request, visible tokens) of each query row: a request's chunk ends at its length."""
    out = []
    for b, n in enumerate(_ctx(case)):
        out += [(b, max(0, n - case["chunk"] + 1 + i)) for i in range(case["chunk"])]
    return out


def work(case):
    es, d, h = ES[case["dtype"]], case["d"], case["hkv"]
    held = 2 * h * (d * 5 // 8)          # bytes of a token's key and value
    plain = 2 * h * d * es
    if case["op"] == "write":
        t = sum(_new(case))
        return {"bytes": t * (2 * plain + held + 4) + case["pad"] * (held + plain),
                "flops": t * 20 * h * d}
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (held + plain + 4), "flops": case["tokens"] * 4 * h * d}
    n, f = 0, 0
    for b, m in enumerate(_ctx(case)):
        n += m * (held + 4)              # rows of one request may read the same tokens
    for b, m in _rows(case):
        f += 4 * case["hq"] * d * m
        n += 2 * case["hq"] * d * es + 4 * case["hq"] + 8
    if case["op"] == "step":
        n += case["reqs"] * (plain + held)
    return {"bytes": n, "flops": f}


# ---------------------------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(g, slots, hkv, d):
    """A plane of cached heads: codes of all kinds, groups of unlike spread, not all around zero."""
    groups = d // 32
    plane = torch.randint(0, 256, (slots, hkv, d * 5 // 8), generator=g, device="cuda",
                          dtype=torch.uint8)
    scale = torch.randint(8, 16, (slots, hkv, groups), generator=g, device="cuda",
                          dtype=torch.int32).float() / 32
    low = -scale * (6 + 3 * torch.rand((slots, hkv, groups), generator=g, device="cuda"))
    plane[..., d // 2:] = torch.stack([scale, low], -1).to(torch.bfloat16).flatten(-2).view(torch.uint8)
    return plane


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hkv = DT[case["dtype"]], case["d"], case["hkv"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def keys(n):
        """The fused projection's keys and values; a few channels of a key are larger, as in use."""
        kv = randn(n, 2 * hkv, d)
        kv[:, :hkv, ::29] *= 6
        return kv[:, :hkv], kv[:, hkv:]

    s = {"case": case}
    if case["op"] in ("write", "read"):
        s["k_pool"], s["v_pool"] = (_cache(g, case["slots"], hkv, d) for _ in "kv")
        if case["op"] == "write":
            new = _new(case)
            s["total"] = sum(new)
            t = s["total"] + case["pad"]
            s["k"], s["v"] = keys(t)
            s["qo_indptr"] = _i32([sum(new[:i]) for i in range(len(new) + 1)])
            rows = t
        else:
            t = case["tokens"]
            rows = case["slots"] if case["scatter"] else t
            s["out_loc"] = torch.randperm(rows, generator=g, device="cuda")[:t].to(torch.int32) \
                if case["scatter"] else None
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:t].to(torch.int32)
        s["k_out"], s["v_out"] = randn(rows, hkv, d), randn(rows, hkv, d)
        return s
    lens = _ctx(case)
    total = sum(lens)
    slots = total + 64
    s["k_pool"], s["v_pool"] = (_cache(g, slots, hkv, d) for _ in "kv")
    perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    req = torch.randperm(case["reqs"], generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["reqs"], case["ctx"]), dtype=torch.int32, device="cuda")
    n = _i32(lens)
    pos = torch.arange(case["ctx"], device="cuda")
    inside = pos < n[:, None]
    at = (n.cumsum(0) - n)[:, None] + pos
    table[req.long()] = torch.where(inside, perm[torch.where(inside, at, 0)], 0)
    which = _rows(case)
    s["q"] = randn(len(which), case["hq"], d)
    s["table"] = table
    s["req_idx"] = req[torch.tensor([b for b, _ in which], device="cuda")]
    s["seq_len"] = _i32([m for _, m in which])
    s["max_seq"] = max(m for _, m in which)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((len(which), case["hq"]), dtype=torch.float32, device="cuda")
    if case["op"] == "step":
        s["k"], s["v"] = keys(case["reqs"])
        s["qo_indptr"] = _i32(list(range(case["reqs"] + 1)))
        s["slots"] = table[s["req_idx"].long(), s["seq_len"].long() - 1].contiguous()
    return s


# ---------------------------------------------------------------------------------- plain forms
def _quantise(x):
    """The bytes of [.., d] numbers: groups' minimum rounded down to bf16, scale rounded up to four
    significant bits; a group that holds a NaN or a magnitude of 2^30 and more is NaN."""
    d = x.shape[-1]
    x = x.float().unflatten(-1, (d // 32, 32))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    bits = lo.view(torch.int32)
    low = (torch.where(lo < 0, bits + 0xFFFF, bits) & ~0xFFFF).view(torch.float32) + 0.0
    step = (hi - low) / torch.full_like(hi, 15)
    scale = ((step.view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(torch.float32).clamp(min=2.0 ** -80)
    code = ((x - low) * scale.reciprocal()).round()
    lost = ~((lo > -2.0 ** 30) & (hi < 2.0 ** 30))
    code = torch.where(lost, 0, code).to(torch.uint8)
    pair = torch.cat([scale, low], -1).masked_fill(lost, math.nan).to(torch.bfloat16)
    code = code.unflatten(-1, (4, 8)).transpose(-3, -2).flatten(-3)   # words in their order
    return torch.cat([code[..., ::2] | code[..., 1::2] << 4, pair.flatten(-2).view(torch.uint8)], -1)


def _numbers(plane, d):
    """What the bytes [.., d * 5 / 8] of heads stand for, fp32."""
    groups = d // 32
    pair = plane[..., d // 2:].contiguous().view(torch.bfloat16).float().unflatten(-1, (groups, 2))
    byte = plane[..., :d // 2]
    code = torch.stack([byte & 15, byte >> 4], -1).unflatten(-2, (4, groups, 4)).flatten(-2)
    code = code.transpose(-3, -2).flatten(-2).float()                 # [.., group, 32]
    return (code * pair[..., :1] + pair[..., 1:]).flatten(-2)


def _plain_write(s):
    n, d = s["total"], s["case"]["d"]
    at, every = s["slots"][:n].long(), s["slots"].long()
    for x, pool in ((s["k"], s["k_pool"]), (s["v"], s["v_pool"])):
        pool[at] = _quantise(x[:n])
    return [_numbers(pool[every], d).to(s["k"].dtype) for pool in (s["k_pool"], s["v_pool"])]


def _plain_read(s):
    at, d = s["slots"].long(), s["case"]["d"]
    for pool, out in ((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"])):
        got = _numbers(pool[at], d).to(out.dtype)
        out[slice(None) if s["out_loc"] is None else s["out_loc"].long()] = got
    return [s["k_out"], s["v_out"]]


def _plain_decode(s):
    case = s["case"]
    n, hq, d = s["q"].shape
    h = case["hkv"]
    if case["op"] == "step":
        at = s["slots"].long()
        s["k_pool"][at], s["v_pool"][at] = _quantise(s["k"]), _quantise(s["v"])
    real = torch.arange(s["max_seq"], device="cuda") < s["seq_len"][:, None]
    slot = torch.where(real, s["table"][s["req_idx"].long(), :s["max_seq"]], 0).long()
    k = _numbers(s["k_pool"][slot], d)
    q = s["q"].view(n, h, hq // h, d).float() / math.sqrt(d)
    logit = q @ k.permute(0, 2, 3, 1)
    del k
    logit = torch.where(real[:, None, None], logit, -math.inf)
    m = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(m == -math.inf, 0, m))
    den = p.sum(-1, keepdim=True)
    o = (p @ _numbers(s["v_pool"][slot], d).transpose(1, 2)) / torch.where(den == 0, 1, den)
    return [o.view(n, hq, d).to(s["q"].dtype), (m + den.log()).view(n, hq)]


# ---------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode,
                "step": _plain_decode}[case["op"]](s)
    import prefix_cached_paged_gb300 as rc
    if case["op"] in ("write", "step"):
        rc.kv4_append(s["k"], s["v"], s["slots"], s["qo_indptr"], s["k_pool"], s["v_pool"])
    if case["op"] == "write":
        rc.kv4_read(s["k_pool"], s["v_pool"], s["slots"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if case["op"] == "read":
        rc.kv4_read(s["k_pool"], s["v_pool"], s["slots"], s["k_out"], s["v_out"],
                    out_loc=s["out_loc"])
        return [s["k_out"], s["v_out"]]
    if "workspace" not in s:
        need = rc.kv4_decode_workspace_bytes(s["q"], s["k_pool"], max_seq_len=s["max_seq"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc.kv4_decode_attention(s["q"], s["seq_len"], s["req_idx"], s["table"], s["k_pool"], s["v_pool"],
                            s["o"], s["workspace"], sm_scale=1.0 / math.sqrt(case["d"]),
                            max_seq_len=s["max_seq"], lse=s["lse"])
    return [s["o"], s["lse"]]


# ---------------------------------------------------------------------------------- in 64 bits
def _single(x):
    """64-bit numbers rounded to 32 bits, as the definition's differences, steps and products are."""
    return x.float().double()


def _exact_held(x):
    """What numbers stand for once they are held: the definition, group by group."""
    x = x.double()
    out = torch.empty_like(x)
    for j in range(0, x.shape[-1], 32):
        y = x[..., j:j + 32]
        least, most = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        part, e = torch.frexp(least)
        low = torch.ldexp((part * 256).floor() / 256, e)                 # bf16: eight bits
        part, e = torch.frexp(_single(_single(most - low) / 15))
        scale = torch.ldexp((part * 16).ceil() / 16, e).clamp(min=2.0 ** -80)
        code = _single(_single(y - low) * _single(1 / scale)).round()
        out[..., j:j + 32] = code * scale + low
    return out


def _exact_numbers(plane, d):
    """The same numbers as _numbers, element by element of a head."""
    words = plane[..., :d // 2].contiguous().view(torch.int32)
    pair = plane[..., d // 2:].contiguous().view(torch.bfloat16).double()
    e = torch.arange(d, device="cuda")
    word = words[..., e % 32 // 8 * (d // 32) + e // 32]
    return (word >> e % 8 * 4 & 15) * pair[..., e // 32 * 2] + pair[..., e // 32 * 2 + 1]


def exact(case, seed):
    s = prepare(case, seed)
    d, h = case["d"], case["hkv"]
    if case["op"] == "write":
        n, at = s["total"], s["slots"].long()
        return [torch.cat([_exact_held(x[:n]), _exact_numbers(pool[at[n:]], d)])
                for x, pool in ((s["k"], s["k_pool"]), (s["v"], s["v_pool"]))]
    if case["op"] == "read":
        out = []
        for pool, old in ((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"])):
            x = _exact_numbers(pool[s["slots"].long()], d)
            if s["out_loc"] is not None:
                y = old.double()
                y[s["out_loc"].long()] = x
                x = y
            out.append(x)
        return out
    n, hq, _ = s["q"].shape
    o = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, ((_, m), row) in enumerate(zip(_rows(case), s["req_idx"].tolist())):
        if m == 0:
            continue
        slot = s["table"][row, :m].long()
        k, v = _exact_numbers(s["k_pool"][slot], d), _exact_numbers(s["v_pool"][slot], d)
        if case["op"] == "step":
            k[-1], v[-1] = _exact_held(s["k"][i]), _exact_held(s["v"][i])
        q = s["q"][i].double().view(h, hq // h, d)
        logit = (q @ k.permute(1, 2, 0)) / math.sqrt(d)
        o[i] = (logit.softmax(-1) @ v.transpose(0, 1)).view(hq, d)
        lse[i] = logit.logsumexp(-1).view(hq)
    return [o, lse]
