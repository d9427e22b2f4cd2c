"""Limits on decode attention over the 4-bit cache that are counted closely, for the tests only.

Roundings of different tokens are independent of one another, so their errors add up as a root of a sum of
squares: FIVE times the root of the sum of the squares of the largest errors. With a rounding's errors even
over their interval that is 8.6 standard deviations, and for up to 25 terms no less than their plain sum. What
is the same for all tokens adds up as it is. u is half a step of fp32, 2^-24; a matrix instruction may cut
its sum off, 2 u."""
import math

import torch

from tests import kv4_ref as R

U = R.U32
FIVE = 5.0


def half_spacing(x, dtype):
    """Half the distance between the numbers of dtype around x: what a rounding may be off by."""
    _, e = torch.frexp(x.abs())
    return torch.ldexp(torch.full_like(x, torch.finfo(dtype).eps / 4), e)


def groups_of(plane, d):
    """bytes [n, d * 5 / 8] -> codes, scales, minima, each float64 [n, d], on the plane's device."""
    ng = d // 32
    pair = plane[:, d // 2:].contiguous().view(torch.bfloat16).double()
    words = plane[:, :d // 2].contiguous().view(torch.int32)
    e = torch.arange(d, device=plane.device)
    code = words[:, e % 32 // 8 * ng + e // 32] >> e % 8 * 4 & 15
    return code.double(), pair[:, e // 32 * 2], pair[:, e // 32 * 2 + 1]


def attend(q, k, v, scale):
    """Query rows q [r, d] over the tokens k, v [n, d * 5 / 8] of their KV head, in 64 bits.
    -> (o, lse, limit of o before its rounding, limit of lse)"""
    n, d = k.shape[0], q.shape[1]
    q = q.double()
    code, step, low = groups_of(k, d)
    s = q @ (code * step + low).T * scale
    top = s.amax(-1, keepdim=True)
    p = s.softmax(-1)
    # a score: sums of query elements (10 u), two matrix instructions for the minima and two for each
    # group's codes (8 u), a sum over groups (4 u), the parts of a query (2 u); fp32 counts codes and
    # minima from the groups' middles, which is never more than this
    size = q.abs() @ (code * step + low.abs() + 8 * step).T * scale
    # a weight: its score, the difference to the reference and exp2 (2^-22)
    e = p * (24 * U * size + 2 * U * (s - top).abs() + 4 * U)
    code, step, low = groups_of(v, d)
    x = code * step + low
    o = p @ x
    spread = (e * e) @ (x * x) - 2 * o * ((e * e) @ x) + o * o * (e * e).sum(-1, keepdim=True)
    # the scores' factor is the same for all tokens (3 u): a weight moves with its score
    mean = (p * s).sum(-1, keepdim=True)
    lean = p * (s - mean).abs()
    same = 3 * U * (lean @ x.abs() + o.abs() * lean.sum(-1, keepdim=True))
    # sums: three matrix instructions for 16 tokens (6 u), those added in fp32, joins and the quotient
    size = p @ ((code - 8) * step).abs() + p @ (low + 8 * step).abs() + o.abs()
    to = FIVE * spread.clamp(min=0).sqrt() + same + (26 + FIVE * math.sqrt(max(1, n / 16))) * U * size
    lse = s.logsumexp(-1)
    tl = FIVE * (e * e).sum(-1).sqrt() + 3 * U * mean[:, 0].abs() + 4 * U * top[:, 0].abs() + \
        6 * U * lse.abs() + (10 + FIVE * math.sqrt(max(1, n / 8))) * U
    return o, lse, to, tl


def held(code, step, low):
    """codes [.., d] and, for each group, scales and minima [.., d / 32] -> bytes [.., d * 5 / 8]."""
    d = code.shape[-1]
    words = code.to(torch.uint8).unflatten(-1, (d // 32, 4, 8)).transpose(-3, -2).flatten(-3)
    pair = torch.stack([step, low], -1)
    assert torch.equal(pair.to(torch.bfloat16).double(), pair.double())
    return torch.cat([words[..., ::2] | words[..., 1::2] << 4,
                      pair.to(torch.bfloat16).flatten(-2).view(torch.uint8)], -1)


def run(q, rows, table, k, v, scale, max_seq=None):
    """rc.kv4_decode_attention on the GPU; rows: (request, visible tokens)."""
    import prefix_cached_paged_gb300 as rc
    seq = torch.tensor([m for _, m in rows], dtype=torch.int32, device="cuda")
    req = torch.tensor([b for b, _ in rows], dtype=torch.int32, device="cuda")
    q, table, k, v = (t.cuda() for t in (q, table, k, v))
    max_seq = max_seq or max(1, max(m for _, m in rows))
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.empty(rc.kv4_decode_workspace_bytes(q, k, max_seq_len=max_seq), dtype=torch.uint8,
                     device="cuda")
    rc.kv4_decode_attention(q, seq, req, table, k, v, o, ws, sm_scale=scale, max_seq_len=max_seq, lse=lse)
    return o, lse
