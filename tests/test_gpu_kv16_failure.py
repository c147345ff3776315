"""Waits of the 16-bit cache's attention that run out, made by copies that are never issued (nothing faults or spins without
a bound): the call returns, its status word says so, rows behind the last sequence stay, and the next call is right."""
import pytest

from gpu_common import require_gpu, torch
from test_gpu_kv16_attention import Setup, _bits, trees

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def b():
    require_gpu()
    from speculative_decoding_rvq_gb300 import binding
    yield binding
    binding.kv16_test_hooks()


# few rows: split, unsplit, short (one tile), 256 channels; tiles: one block split, unsplit, one tile, pairs of blocks
CASES = [([(3000, 1)], 4, 2, 128, BF, False), ([(700, 2)] * 40, 4, 2, 64, FP, False), ([(20, 3)], 2, 1, 128, BF, False),
         ([(900, 40)], 4, 2, 256, BF, False), ([(5000, 60)], 4, 2, 128, BF, False), ([(600, 100)] * 20, 8, 8, 64, FP, False),
         ([(100, 100)], 1, 1, 128, BF, False), ([(700, 600)] * 2, 32, 8, 128, BF, False), ([(400, 20)] * 3, 8, 2, 128, FP, True)]


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("lens,nq,nkv,dim,dtype,tree", CASES)
def test_a_wait_that_runs_out_is_reported(b, lens, nq, nkv, dim, dtype, tree, stall):
    s = Setup(b, lens, nq, nkv, dim, 16, dtype, spare=3)
    masks = trees(lens) if tree else None
    want, want_lse = s.call(masks)
    n = s.starts[-1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(s.q, 3.0)
    b.kv16_test_hooks(wait_limit_ns=2_000_000, stall=stall)
    try:
        s.call(masks, status=status, out=out)
        s.call(masks)  # (without a status word)
        torch.cuda.synchronize()
    finally:
        b.kv16_test_hooks()
    assert status.item() == b.E_DEVICE_TIMEOUT
    assert (out[n:] == 3).all()
    status.zero_()
    for _ in range(3):
        got, lse = s.call(masks, status=status)
        assert torch.equal(_bits(got[:n]), _bits(want[:n])) and torch.equal(_bits(lse[:n]), _bits(want_lse[:n]))
    assert status.item() == 0


def test_a_status_that_is_set_stays(b):
    s = Setup(b, [(300, 2)], 2, 1, 128, 16, BF)
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    b.kv16_test_hooks(wait_limit_ns=1_000_000, stall=1)
    try:
        s.call(status=status)
        torch.cuda.synchronize()
    finally:
        b.kv16_test_hooks()
    assert status.item() == 7
