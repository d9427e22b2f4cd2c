"""Decode attention over the 4-bit cache: how many bits its weights, scores and sums keep, and that no token of
a long row is lost or counted twice (limits: kv4_tight)."""
import pytest
import torch

import prefix_cached_paged_gb300 as rc
from tests import kv4_ref as R
from tests import kv4_tight as T

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,g,hkv,d", [("bf16", 1, 8, 128), ("bf16", 8, 8, 128),
                                           ("bf16", 16, 4, 128), ("bf16", 2, 8, 64), ("f32", 2, 4, 128)])
def test_sums_over_long_rows_are_fp32(dtype, g, hkv, d):
    """Zero queries, so every weight is 1, and more rows of about 32 000 tokens than CTAs, so a warp sums a
    row's outputs from end to end. Values are positive, of 12 binades, around groups' middles of zero. Rounded
    sums of 16 tokens are off by a root of a sum of squares, u of what is summed by then; matrix instructions
    that kept the sums would cut them off 2000 times, towards zero each time."""
    n, rows, hq = 32000, 700, g * hkv
    gen = torch.Generator().manual_seed(11 * g + d)
    code = torch.randint(9, 16, (n, hkv, d), generator=gen)
    step = torch.randint(8, 16, (n, hkv, d // 32), generator=gen).double() * \
        torch.exp2(-torch.randint(0, 12, (n, hkv, d // 32), generator=gen).double())
    v = T.held(code, step, -8 * step).cuda()
    lens = n - torch.arange(rows)
    q = torch.zeros((rows, hq, d), dtype=DT[dtype], device="cuda")
    table = torch.arange(n, dtype=torch.int32)[None]
    o, lse = T.run(q, [(0, m) for m in lens.tolist()], table, v, v, d ** -0.5)
    code, step, low = T.groups_of(v.reshape(-1, v.shape[-1]), d)
    ro = (code * step + low).reshape(n, hkv, d).cumsum(0)[lens.cuda() - 1] / lens.cuda()[:, None, None]
    ro = ro.repeat_interleave(g, 1)
    # sums, cut off once for 16 tokens (2 u), joins of a row's ranges and the quotient
    limit = (T.FIVE * (n / 16 / 3) ** 0.5 + 16) * T.U
    beyond = (o.double() - ro).abs() - T.half_spacing(ro * (1 + limit), q.dtype)
    assert (beyond <= ro * limit).all(), (int((beyond > ro * limit).sum()), float((beyond / ro).max()) / T.U)
    rl = lens.double().log()[:, None].cuda()
    assert ((lse.double() - rl).abs() <= 4 * T.U * rl).all()     # whole numbers, log2, its product
    assert rc.device_status() == 0
