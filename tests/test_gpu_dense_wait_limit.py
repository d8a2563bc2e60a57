"""The give-up path of the dense decode: with hils_set_wait_limit(0) every ordinary wait of
the kernel gives up at its first poll.  The call reports a timeout, writes nothing that it has
not waited for, and leaves the workspace ready: the next call gives the first one's bits."""
import pytest
import torch

import chunk_wise_hierarchical_b200 as hils

pytestmark = pytest.mark.gpu

HILS_ERR_DEVICE_TIMEOUT = 6


@pytest.mark.parametrize("dtype,lens,h,g,d", [
    (torch.bfloat16, [9000, 5, 0, 700], 8, 2, 128),   # cut between warps and SMs, and whole
    (torch.bfloat16, [90001], 4, 1, 64),              # joined in two steps
    (torch.float32, [3000, 64], 2, 2, 64),
])
def test_a_call_that_gives_up_leaves_the_next_one_whole(dtype, lens, h, g, d):
    gen = torch.Generator(device="cuda").manual_seed(0)
    chunks = [-(-n // 64) for n in lens]
    b, m, pool = len(lens), max(chunks), sum(chunks) + 1
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    q, kp, vp = rnd(b, h, d), rnd(pool, g, 64, d), rnd(pool, g, 64, d)
    table = torch.full((b, m), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(chunks):
        table[i, :c] = torch.arange(at, at + c, dtype=torch.int32)
        at += c
    args = (q, kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    call = hils.DenseDecode(b, h, g, d, m, dtype)
    want = call(*args).clone()
    assert call.device_status() == 0
    prev = hils.set_wait_limit(0)
    try:
        out = torch.full_like(want, 7.0)
        call(*args, out=out)
        assert call.device_status() == HILS_ERR_DEVICE_TIMEOUT
    finally:
        hils.set_wait_limit(prev)
    live = torch.tensor([n > 0 for n in lens], device="cuda")
    assert (out[live] == 7.0).all() and (out[~live] == 0).all()
    for _ in range(2):
        assert torch.equal(call(*args), want) and call.device_status() == 0
