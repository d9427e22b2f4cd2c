"""Plain 64-bit forms of the operators around the paged cache (norms with rotation, append, block
bounds, block-sparse decode), for the tests only, and the tolerances derived from them.

A rounding to a type is off by at most half a step, torch.finfo(t).eps / 2 relative to the value.
Everything before the single rounding is fp32: a sum of n terms is off by at most n * 2^-24 of the
sum of their magnitudes.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rope_table(rot, positions, base=10000.0):
    f = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rope(x, w, table, positions, interleaved, eps):
    """x [T, H, d] -> (float64 result, tolerance of the fp32 arithmetic per element)."""
    x = x.double().cpu()
    d = x.shape[-1]
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    # the norm's sum of d squares halves in the root; its quotient, root, weight and the rotation's
    # two products and sum, and rsqrtf (2 ulp = 4 half steps) add a few roundings
    rel = ((d / 2 + 10) if w is not None else 4) * U32
    y, mag = x.clone(), x.abs()
    if table is not None:
        half = table.shape[1] // 2
        c, s = table[positions.long().cpu()].double().split(half, 1)
        c, s = c[:, None], s[:, None]
        ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, rel * mag


def bounds_of(keys, block):
    """keys [n, Hkv, d] (stored) -> [blocks, Hkv, 2, d]; min and max keep a NaN."""
    n = keys.shape[0]
    out = []
    for p in range(0, n, block):
        part = keys[p:p + block]
        out.append(torch.stack([part.amin(0), part.amax(0)], 1))
    return torch.stack(out) if out else keys.new_zeros((0, keys.shape[1], 2, keys.shape[2]))


def select(q, box, seq_len, block, top, sink, recent):
    """q [Hq, d], box [blocks, Hkv, 2, d] -> chosen blocks per KV head, ascending, padded by -1."""
    hkv = box.shape[1]
    g = q.shape[0] // hkv
    have = -(-seq_len // block)
    q, box = q.double(), box.double()
    out = torch.full((hkv, top), -1, dtype=torch.int32)
    big = torch.finfo(torch.float64).max
    for h in range(hkv):
        ranks = []
        for b in range(have):
            if b < sink or b >= have - recent:
                ranks.append((-math.inf, b))
                continue
            best = -big
            for i in range(g):
                x = q[h * g + i]
                s = float(torch.where(x >= 0, x * box[b, h, 1], x * box[b, h, 0]).sum())
                s = big if math.isnan(s) or s == math.inf else max(s, -big)
                best = max(best, s)
            ranks.append((-best, b))
        pick = sorted(b for _, b in sorted(ranks)[:top])
        out[h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return out


def attend(q, sel, seq_len, row_slots, k_pool, v_pool, block, scale):
    """One row: q [Hq, d], sel [Hkv, top] -> (o, lse, tolerance of o before rounding, of lse)."""
    hq, d = q.shape
    hkv = sel.shape[0]
    g = hq // hkv
    o = torch.zeros((hq, d), dtype=torch.float64)
    lse = torch.full((hq,), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros((hq, d), dtype=torch.float64), torch.zeros(hq, dtype=torch.float64)
    for h in range(hkv):
        pos = [b * block + i for b in sel[h].tolist() if b >= 0 for i in range(block)
               if b * block + i < seq_len]
        pos = [p for p in pos if 0 <= int(row_slots[p]) < k_pool.shape[0]]
        if not pos:
            continue
        slots = row_slots[torch.tensor(pos)].long()
        k, v = k_pool[slots, h].double(), v_pool[slots, h].double()
        for i in range(g):
            x = q[h * g + i].double()
            s = (k @ x) * scale
            o[h * g + i] = s.softmax(0) @ v
            lse[h * g + i] = s.logsumexp(0)
            # a score: d products and sums, twice half a step each (a matrix unit may truncate),
            # then the scale to base 2; a weight: its score's error, exp2f (2 ulp) and, where it is
            # held as two bf16 parts, 2^-16; sums over n weights, normalisation, joining parts
            delta = (2 * d + 8) * U32 * float((k.abs() @ x.abs()).max() * scale) + \
                4 * U32 * float(s.abs().max())
            n = len(pos)
            wgt = 2 * delta + 2.0 ** -16 + (n + 64) * U32
            to[h * g + i] = wgt * (s.softmax(0) @ v.abs())
            tl[h * g + i] = delta + (n + 64) * U32 + 4 * U32 * abs(float(lse[h * g + i]))
    return o, lse, to, tl
