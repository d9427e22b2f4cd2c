"""Waits of decode attention over the 4-bit cache that run out (a test-only limit, rc_debug_set_wait_limit_ns).

A warp whose copies or whose neighbours' do not come within the limit reports it in the device status word and
goes on without waiting; what it could not compute is NaN, in the outputs and in the states that the second
kernel joins, so nothing that a workspace held before passes for an output. Here the limit is one
nanosecond: every output has the bits of a call with the default limit or is NaN, some are NaN, the
calls return, and the next one with the default limit is clean. Nothing faults or hangs: the only
failure made is a wait that stops early."""
import pytest
import torch

import prefix_cached_paged_gb300 as rc
from tests import kv4_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype,hq,hkv,d,lens", [
    ("bf16", 8, 8, 128, [3000, 1, 700, 0, 5000]),       # a warp per KV head
    ("bf16", 32, 16, 128, [900 + 7 * i for i in range(90)]),
    ("bf16", 8, 1, 128, [60_000, 70, 9000]),            # eight warps share a head
    ("bf16", 6, 3, 64, [60_000, 33, 2000, 2001]),       # two warps of three heads
    ("bf16", 48, 4, 64, [40_000, 5, 3333]),             # two tiles of query heads
    ("f32", 4, 4, 64, [60_000, 64, 1000]), ("f32", 48, 4, 64, [40_000, 300])])
def test_waits_that_run_out_leave_right_outputs_or_nan(dtype, hq, hkv, d, lens):
    slots, ctx = max(4000, max(lens)), max(lens)
    g = torch.Generator().manual_seed(hq + d)
    k, v = (R.quantise(torch.randn((slots, hkv, d), generator=g)).cuda() for _ in "kv")
    table = torch.randint(0, slots, (len(lens), ctx), generator=g, dtype=torch.int32).cuda()
    q = torch.randn((len(lens), hq, d), generator=g).to(DT[dtype]).cuda()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    req = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    need = rc.kv4_decode_workspace_bytes(q, k, max_seq_len=ctx)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def call():
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")   # states of zeros would pass for outputs
        o, lse = torch.full_like(q, 7.0), torch.full((len(lens), hq), 7.0, device="cuda")
        cold.zero_()                                               # copies come from memory,
        q.mul_(1)                                                  # queries do not
        rc.kv4_decode_attention(q, seq, req, table, k, v, o, ws, sm_scale=0.1, max_seq_len=ctx, lse=lse)
        torch.cuda.synchronize()
        return o, lse

    want = call()
    assert rc.device_status() == 0 and not want[0].isnan().any()
    gave_up = 0
    rc.set_wait_limit_ns(1)
    try:
        for _ in range(10):   # whether a wait lasts for a tick of the clock is the hardware's; here all did
            short = call()
            lost = short[1].isnan()
            for x, y in zip(short, want):
                assert ((x == y) | x.isnan()).all()
            assert torch.equal(lost[..., None].expand_as(q), short[0].isnan())
            assert rc.device_status() == (3 if lost.any() else 0)
            gave_up += bool(lost.any())
    finally:
        rc.set_wait_limit_ns(0)
    print("calls that gave up:", gave_up)
    assert gave_up
    for x, y in zip(call(), want):
        assert torch.equal(x, y)
    assert rc.device_status() == 0
