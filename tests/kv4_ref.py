"""The 4-bit cache in plain 64-bit form, for the tests only: the bytes of a head, what they stand
for, attention over it, and the tolerances derived from the kernels' roundings.

A rounding to a type is off by at most half a step, torch.finfo(t).eps / 2 relative to the value; a
matrix unit may cut a sum off instead of rounding it, which counts as two half steps.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _f32(x):
    """float64 rounded to fp32: exact arithmetic of two fp32 numbers followed by this is fp32's."""
    return x.float().double()


def quantise(x):
    """x [..., d] -> the bytes [..., d * 5 / 8] that hold it (CPU)."""
    d = x.shape[-1]
    ng = d // 32
    x = x.double().cpu().reshape(*x.shape[:-1], ng, 32)
    lo, hi = x.amin(-1), x.amax(-1)
    lost = ~((lo > -2.0 ** 30) & (hi < 2.0 ** 30))
    lo, hi = (torch.where(lost, 0.0, t) for t in (lo, hi))
    mant, ex = torch.frexp(lo)
    low = torch.ldexp(torch.floor(mant * 256) / 256, ex)
    # below bf16's smallest normal number its steps are 2^-133
    low = torch.where(low.abs() < 2.0 ** -126, torch.floor(lo * 2.0 ** 133) / 2.0 ** 133, low)
    low = low + 0.0   # no -0
    mant, ex = torch.frexp(_f32(_f32(hi - low) / 15))
    scale = torch.ldexp(torch.ceil(mant * 16) / 16, ex).clamp(min=2.0 ** -80)
    inv = _f32(1 / scale)
    code = torch.round(_f32(_f32(x - low[..., None]) * inv[..., None]))
    code = torch.where(lost[..., None], 0.0, code).to(torch.int32)
    assert ((code >= 0) & (code <= 15)).all()
    out = torch.zeros((*x.shape[:-2], d * 5 // 8), dtype=torch.uint8)
    for e in range(d):
        j, t, n = e // 32, e % 32 // 8, e % 8
        byte = 4 * (t * ng + j) + n // 2
        out[..., byte] |= (code[..., j, e % 32] << 4 * (n % 2)).to(torch.uint8)
    pair = torch.stack([scale, low], -1).masked_fill(lost[..., None], math.nan)
    out[..., d // 2:] = pair.to(torch.bfloat16).flatten(-2).view(torch.uint8)
    return out


def parts(plane, d):
    """bytes [..., d * 5 / 8] -> (code * scale, minimum), each float64 [..., d]."""
    plane = plane.cpu()
    ng = d // 32
    pair = plane[..., d // 2:].contiguous().view(torch.bfloat16).double()
    a = torch.zeros((*plane.shape[:-1], d), dtype=torch.float64)
    b = torch.zeros_like(a)
    for e in range(d):
        j, t, n = e // 32, e % 32 // 8, e % 8
        code = plane[..., 4 * (t * ng + j) + n // 2] >> 4 * (n % 2) & 15
        a[..., e] = code.double() * pair[..., 2 * j]
        b[..., e] = pair[..., 2 * j + 1]
    return a, b


def values(plane, d):
    a, b = parts(plane, d)
    return a + b


def attend(q, seq_len, row_slots, k_pool, v_pool, scale):
    """One row: q [Hq, d] -> (o, lse, tolerance of o before its rounding, of lse)."""
    hq, d = q.shape
    hkv = k_pool.shape[1]
    g = hq // hkv
    o = torch.zeros((hq, d), dtype=torch.float64)
    lse = torch.full((hq,), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros((hq, d), dtype=torch.float64), torch.zeros(hq, dtype=torch.float64)
    slots = row_slots[:seq_len].long()
    slots = slots[(slots >= 0) & (slots < k_pool.shape[0])]
    n = len(slots)
    if n == 0:
        return o, lse, to, tl
    ka, kb = parts(k_pool[slots], d)
    va, vb = parts(v_pool[slots], d)
    for i in range(hq):
        h = i // g
        x = q[i].double()
        s = ((ka[:, h] + kb[:, h]) @ x) * scale
        o[i] = s.softmax(0) @ (va[:, h] + vb[:, h])
        lse[i] = s.logsumexp(0)
        # a score: d products and sums of codes' part and minimum's part, cut off or rounded, then
        # the groups joined and the scale to base 2
        size = (ka[:, h].abs() + kb[:, h].abs()) @ x.abs()
        delta = (2 * d + 24) * U32 * float(size.max() * scale) + 4 * U32 * float(s.abs().max())
        # a weight: its score's error, exp2 (2 ulp) and its parts in bf16 (two for bf16 outputs,
        # three for fp32); sums over n weights, rescaling, normalising, joining parts
        part = 2.0 ** -16 if q.dtype == torch.bfloat16 else 2.0 ** -22
        wgt = 2 * delta + part + 2 * (n + 64) * U32
        to[i] = wgt * (s.softmax(0) @ (va[:, h].abs() + vb[:, h].abs()))
        tl[i] = delta + (n + 64) * U32 + 4 * U32 * abs(float(lse[i]))
    return o, lse, to, tl
