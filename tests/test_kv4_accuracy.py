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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("g", [8, 16])
def test_weights_keep_24_bits(dtype, d, g):
    """Outputs that are differences of two weights 2^-15 of them apart, so that 8 bits of an output show the
    weights' last ones. A query has one element, a power of two, and keys code * scale + minimum of 17 bits at
    most: scores are exact. Tokens 2 i and 2 i + 1 have the same code and scale there, and minima that are
    neighbours; their values are + and - 1 in element i, + and - 7 in element i + d / 2, zero elsewhere."""
    hkv, n = 4, d
    gen = torch.Generator().manual_seed(3 * d + g)
    scale = 0.3

    def pairs(t):
        return t.repeat_interleave(2, 0)

    k_code = pairs(torch.randint(0, 16, (n // 2, hkv, d), generator=gen))
    k_step = pairs(torch.randint(8, 16, (n // 2, hkv, d // 32), generator=gen).double() / 128)
    k_low = pairs(torch.randint(128, 255, (n // 2, hkv, d // 32), generator=gen).double())
    k_low[1::2] += 1
    k = T.held(k_code, k_step, k_low / 32768)
    v_code = torch.full((n, hkv, d), 8)
    i = torch.arange(n // 2)
    v_code[2 * i, :, i], v_code[2 * i + 1, :, i] = 9, 7
    v_code[2 * i, :, i + d // 2], v_code[2 * i + 1, :, i + d // 2] = 15, 1
    one = torch.ones((n, hkv, d // 32), dtype=torch.float64)
    v = T.held(v_code, one, -8 * one)
    q = torch.zeros((1, hkv, g, d))
    at = torch.randint(0, d, (hkv, g), generator=gen)
    q.scatter_(-1, at[None, ..., None], torch.tensor([2.0, -2, 1, -1, 0.5, -0.5, 2, -1] * 2)[:g, None]
               .expand(1, hkv, g, 1))
    q = q.flatten(1, 2).to(DT[dtype])
    o, lse = T.run(q, [(0, n)], torch.arange(n, dtype=torch.int32)[None], k, v, scale)
    o = o[0].double().cpu()
    # a weight of at most 2.1: the difference to the reference (half a step of 2 to 4, times ln 2) and exp2
    # (2^-22), 5.4 u; a sum of 16 products of which two count (2 u); the quotient goes with the output
    for h in range(hkv * g):
        c, s, m = T.groups_of(k[:, h // g], d)
        p = ((c * s + m) @ q[0, h].double() * scale).softmax(0)
        c, s, m = T.groups_of(v[:, h // g], d)
        ro = p @ (c * s + m)
        limit = 8 * T.U * (p @ (c * s + m).abs())
        beyond = (o[h] - ro).abs() - T.half_spacing(ro.abs() + limit, q.dtype)
        assert (beyond <= limit + 40 * T.U * ro.abs()).all(), (h, float((beyond / limit).max()))
    assert rc.device_status() == 0


def check_one_hot(q, k, v, scale, o, lse, h, kv):
    """Query head h: its lse, and its output where one token has all the weight."""
    d = q.shape[-1]
    code, step, low = T.groups_of(k[:, kv], d)
    x = q[0, h].double()
    s = (code * step + low) @ x * scale
    size = float(((code * step + low.abs() + 8 * step) @ x.abs()).max() * scale)
    first, second = s.topk(2).values.tolist()
    assert abs(float(lse[0, h]) - float(s.logsumexp(0))) <= 32 * T.U * size + 4 * T.U
    one = first - second > 100 + 64 * T.U * size
    if one:
        assert torch.equal(o[0, h].cpu(), R.values(v[s.argmax(), kv], d).float().to(q.dtype))
    return one


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 50, 2100])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(dtype, n, sign):
    """Scores of 1e3 to 1e30, all of them negative too (keys of one sign): the greatest has the weight."""
    hkv, d, scale = 2, 128, 0.088
    gen = torch.Generator().manual_seed(8 + n)
    k = R.quantise(1e-6 * (torch.randn((n, hkv, d), generator=gen) * 0.3 + 4))
    v = R.quantise(torch.randn((n, hkv, d), generator=gen))
    q = torch.rand((1, 16, d), generator=gen) + 0.5
    q = (q * sign * 10.0 ** torch.linspace(8, 35, 16)[:, None]).to(DT[dtype])
    o, lse = T.run(q, [(0, n)], torch.arange(n, dtype=torch.int32)[None], k, v, scale)
    assert sum(check_one_hot(q, k, v, scale, o, lse, h, h // 8) for h in range(16)) >= 8
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,scale", [("bf16", 0.088), ("bf16", 1.0), ("bf16", 3e37), ("f32", 0.088),
                                         ("f32", 1.0), ("f32", 1e37)])
def test_the_largest_queries_are_right_or_nan(dtype, scale):
    """Queries up to the largest numbers, or factors up to them, and keys small enough for finite scores."""
    n, hkv, d = 50, 2, 128
    gen = torch.Generator().manual_seed(8)
    k = R.quantise(1e-6 * torch.randn((n, hkv, d), generator=gen))
    v = R.quantise(torch.randn((n, hkv, d), generator=gen))
    at = 10.0 ** torch.tensor([38.4, 37.5, 37.0, 36.6, 36.0, 35.0, 30.0, 20.0])
    q = torch.randn((1, 8, d), generator=gen)
    q = (q / q.abs().amax(-1, keepdim=True) * at[:, None] * min(1, 1 / scale)).to(DT[dtype])
    o, lse = T.run(q, [(0, n)], torch.arange(n, dtype=torch.int32)[None], k, v, scale)
    right = 0
    for h in range(8):
        if lse[0, h].isnan():
            assert o[0, h].isnan().all() and float(q[0, h].double().abs().max()) * scale >= 2.0 ** 120
        else:
            right += check_one_hot(q, k, v, scale, o, lse, h, h // 4)
    assert right >= 4 and rc.device_status() == 0   # 1e36 and less is below 2^120 (1.33e36), 4e36 is not


def beyond(o, ro, to, dtype):
    """By how much outputs are further off than a rounding and the limit allow."""
    return (o.double() - ro).abs() - T.half_spacing(ro.abs() + to, dtype) - to


def case(dtype, n, g, d, seed):
    gen = torch.Generator().manual_seed(seed + n * 7 + g)
    k, v = R.quantise(torch.randn((n, d), generator=gen)), R.quantise(torch.randn((n, d), generator=gen) + 0.3)
    return torch.randn((g, d), generator=gen).to(DT[dtype]), k, v


@pytest.mark.parametrize("dtype,n,g,d", [
    ("bf16", 64, 4, 128), ("bf16", 700, 8, 64), ("bf16", 2049, 8, 128), ("bf16", 3500, 12, 128),
    ("f32", 33, 4, 64), ("f32", 260, 2, 128), ("f32", 500, 4, 64), ("f32", 1111, 8, 128), ("f32", 2000, 16, 64)])
def test_the_limits_see_what_they_are_for(dtype, n, g, d):
    """Mistakes planted in the 64-bit form are beyond the limits: weights of one bf16 part, bf16 queries, one
    token left out, one counted twice. The form itself, rounded, is within."""
    q, k, v = case(dtype, n, g, d, 5)
    scale = d ** -0.5
    o, lse, to, tl = T.attend(q, k, v, scale)
    kn, vn = R.values(k, d), R.values(v, d)

    def outside(q=q, part=False, count=None):
        s = q.double() @ kn.T * scale
        w = (s - s.amax(-1, keepdim=True)).exp()
        if count is not None:
            w = w * count
        x = (w.bfloat16().double() if part else w) @ vn / w.sum(-1, keepdim=True)
        y = w.sum(-1).log() + s.amax(-1)
        return bool((beyond(x.to(q.dtype), o, to, q.dtype) > 0).any()), \
            bool(((y.float().double() - lse).abs() > tl).any())

    assert outside() == (False, False)
    assert outside(part=True)[0]
    if dtype == "f32":
        assert outside(q=q.bfloat16().float()) == (True, True)
    for t in (0, n // 2, n - 1):
        for times in (0.0, 2.0):
            count = torch.ones(n, dtype=torch.float64)
            count[t] = times
            assert outside(count=count) == (True, True), (t, times)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ctx,hq,hkv,d", [
    ("bf16", [1], 1, 1, 128), ("bf16", [15, 16, 17], 8, 2, 128), ("bf16", [31, 32, 33, 63, 64, 65], 4, 4, 128),
    ("bf16", [1000, 129, 700], 32, 8, 128), ("bf16", [2049, 40], 8, 8, 128), ("bf16", [901, 333], 6, 2, 128),
    ("bf16", [1500], 10, 2, 64), ("bf16", [1200, 17], 16, 1, 128), ("bf16", [3500], 12, 1, 128),
    ("bf16", [400, 90], 9, 3, 128), ("bf16", [257, 100], 14, 7, 128), ("bf16", [90, 1], 6, 6, 64),
    ("bf16", [40_000, 7000], 8, 2, 64), ("bf16", [30_000, 5], 32, 2, 128),
    ("f32", [1, 33], 2, 2, 64), ("f32", [700, 97], 6, 2, 64), ("f32", [1111], 8, 1, 128),
    ("f32", [515], 13, 1, 128), ("f32", [260, 260], 4, 4, 128), ("f32", [2000], 16, 1, 64),
    ("f32", [64, 1, 500], 16, 8, 128), ("f32", [40_000, 3000], 4, 2, 64)])
def test_decode_within_close_limits(dtype, ctx, hq, hkv, d):
    """Rows of all shapes, and repeated ones: a call's second row of each length is cut elsewhere."""
    n, g = max(ctx), hq // hkv
    gen = torch.Generator().manual_seed(sum(ctx) + hq + d)
    k = R.quantise(torch.randn((min(n, 5000), hkv, d), generator=gen))
    v = R.quantise(torch.randn((min(n, 5000), hkv, d), generator=gen) + 0.3)
    table = torch.randint(0, k.shape[0], (len(ctx), n), generator=gen, dtype=torch.int32)
    rows = [(b, m) for b, m in enumerate(ctx)] * 2
    q = torch.randn((len(rows), hq, d), generator=gen).to(DT[dtype])
    o, lse = T.run(q, rows, table, k, v, d ** -0.5)
    for i, (b, m) in enumerate(rows):
        at = table[b, :m].long()
        for h in range(hkv):
            own = slice(h * g, h * g + g)
            ro, rl, to, tl = T.attend(q[i, own].cuda(), k[at, h].cuda(), v[at, h].cuda(), d ** -0.5)
            assert (beyond(o[i, own], ro, to, q.dtype) <= 0).all(), (i, h)
            assert ((lse[i, own].double() - rl).abs() <= tl).all(), (i, h)
    assert rc.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hq,hkv,d", [
    ("bf16", 8, 8, 128), ("bf16", 4, 1, 128), ("bf16", 6, 3, 64), ("bf16", 32, 2, 128), ("bf16", 10, 5, 64),
    ("bf16", 64, 4, 64), ("f32", 4, 4, 128), ("f32", 16, 1, 64), ("f32", 12, 6, 64)])
def test_every_token_counts_once(dtype, hq, hkv, d):
    """Zero queries: lse is the logarithm of the number of tokens, and an element that is 1 in one token only
    shows whether that token counted. Marked are the first tokens, those on both sides of steps, and others
    anywhere; rows of all lengths in one call, and long ones alone, which all CTAs share."""
    most = 131_071
    gen = torch.Generator().manual_seed(hq + 3 * d)
    edge = torch.cat([16 * 2 ** torch.arange(0, 13) + i for i in (-1, 0, 1)])
    marks = torch.cat([torch.arange(min(300, hkv * d // 2)), edge, most - 1 - torch.arange(5),
                       torch.randint(0, most, (hkv * d,), generator=gen)])[:hkv * d].reshape(hkv, d)
    tokens, at = marks.flatten().unique(return_inverse=True)
    code = torch.full((len(tokens), hkv, d), 8)
    code[at.reshape(hkv, d), torch.arange(hkv)[:, None], torch.arange(d)] = 9
    one = torch.ones((len(tokens), hkv, d // 32), dtype=torch.float64)
    v = T.held(torch.full((1, 1, d), 8), one[:1, :1], -8 * one[:1, :1]).expand(most, hkv, -1).contiguous()
    v[tokens] = T.held(code, one, -8 * one)
    v, marks = v.cuda(), marks.cuda()
    table = torch.arange(most, dtype=torch.int32)[None].cuda()
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 2047,
            2048, 2049, 4097, 9999, 33_333, most]
    for some in (lens, [most], [40_000], [700, 2500], [100 + 3 * i for i in range(400)]):
        q = torch.zeros((len(some), hq, d), dtype=DT[dtype], device="cuda")
        o, lse = T.run(q, [(0, m) for m in some], table, v, v, 0.1)
        n = torch.tensor(some, dtype=torch.float64, device="cuda")[:, None]
        assert ((lse.double() - n.log()).abs() <= 4 * T.U * n.log()).all()
        # whole numbers and one quotient, then the outputs' type
        want = ((marks < n[..., None]) / n[..., None]).repeat_interleave(hq // hkv, 1)
        assert (beyond(o, want, 2 * T.U * want, q.dtype) <= 0).all()
    assert rc.device_status() == 0


def test_elements_are_within_half_a_scale_and_what_fp32_adds():
    """The code's difference, reciprocal and product are off by 3 half steps of fp32, 45 * 2^-24 of a scale at a code
    of 15. More than 2^-20 of half a scale happens: the first row."""
    g = torch.Generator().manual_seed(3)
    x = torch.rand((20_000, 32), generator=g) * torch.rand((20_000, 1), generator=g) - 0.9
    x[0] = torch.linspace(-0.9199936, -0.09474992, 32)
    x[0, 5] = -0.24804693
    x = torch.cat([x, x], 1)
    code, step, low = T.groups_of(R.quantise(x), 64)
    off = (code * step + low - x.double()).abs() / step - 0.5
    assert off.max() <= 45 * 2.0 ** -24
    assert off[0, 5] > 2.0 ** -20 / 2 and step[0, 5] == 0.05859375


@pytest.mark.gpu
def test_the_quotient_by_15_of_every_significand():
    """Groups of 0 and w for all 2^23 significands of w: the scale is w / 15, rounded to fp32 and then up to four
    significant bits. (A 64-bit quotient rounded to 24 bits is the quotient rounded once: 53 >= 2 * 24 + 2.)"""
    n = 1 << 20
    loc = torch.arange(n, dtype=torch.int32, device="cuda")
    ip = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((n, 1, 40), dtype=torch.uint8, device="cuda") for _ in "kv")
    x = torch.zeros((n, 1, 64), device="cuda")
    for part in range(0, 1 << 23, 2 * n):
        w = torch.arange(part, part + 2 * n, device="cuda").double() * 2.0 ** -23 + 1
        x[:, 0, 9], x[:, 0, 40] = w[:n].float(), w[n:].float()
        rc.kv4_append(x, x, loc, ip, kp, vp)
        mant, e = torch.frexp((w / 15).float().double())
        want = torch.ldexp((mant * 16).ceil() / 16, e)
        got = kp[:, 0, 32:].contiguous().view(torch.bfloat16).double()
        assert torch.equal(torch.cat([got[:, 0], got[:, 2]]), want) and not got[:, 1::2].any()
    assert torch.equal(kp, vp) and rc.device_status() == 0
