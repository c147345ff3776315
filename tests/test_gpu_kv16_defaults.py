"""Defaults and tables that a caller of the 16-bit cache's operators may leave out or set."""
import math

import pytest

import kv16_reference as R
from gpu_common import require_gpu, torch
from test_gpu_kv16_attention import Setup, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    require_gpu()
    from speculative_decoding_rvq_gb300 import binding
    return binding


def test_trees_without_max_rows(b):
    """Several trees with more than 64 rows together, and a padded batch: each tree is within 64."""
    lens = [(100, 30), (300, 24), (64, 64), (90, 1)]
    for spare in (0, 50):
        s = Setup(b, lens, 4, 2, 128, 16, torch.bfloat16, spare=spare)
        masks = trees(lens)
        s.check(*s.call(masks, max_rows=None), masks=masks)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_frequencies_that_begin_anew_at_each_axis(b, dtype):
    """The rotation of image patches: height and width with theta^(-2 j / (rot / 2)), j from 0 at either; and a scaled table."""
    rot, theta, m = 64, 10000.0, 333
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(m, 3, rot, generator=g, device="cuda").to(dtype)
    pos = torch.stack([torch.arange(m) // 18, torch.arange(m) % 18]).int().cuda()
    for scale in (1.0, 0.25):
        rope = b.Rope(rot, theta, [16, 16])
        freq = [scale * theta ** (-2.0 * (i % 16) / (rot // 2)) for i in range(32)]
        for i, f in enumerate(freq):
            rope.struct.turns[i] = int(f / (2 * math.pi) * 2.0 ** 64)
        out, _ = rope.rotate(q, None, pos)
        angle = (pos.double().repeat_interleave(16, 0).t() * torch.tensor(freq, dtype=torch.float64, device="cuda")).unsqueeze(1)
        x, y = q.double()[..., :32], q.double()[..., 32:]
        ref = torch.cat([x * torch.cos(angle) - y * torch.sin(angle), y * torch.cos(angle) + x * torch.sin(angle)], -1)
        # (a result is off by 4 * 2^-23 of both channels' sizes, and rounded once)
        both = (x.abs() + y.abs()).repeat(1, 1, 2)
        assert ((out.double() - ref).abs() <= R.HALF_STEP[dtype] * ref.abs() + 4 * 2.0 ** -23 * both).all()
