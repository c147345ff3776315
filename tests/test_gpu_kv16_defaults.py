"""Defaults and tables that a caller of the 16-bit cache's operators may leave out or set."""
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
