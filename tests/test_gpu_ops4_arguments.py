"""What the calls of the 4-bit operators count and take, beside their results."""
import pytest

from gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_rvq_gb300 import binding
    return binding


def _randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_the_launch_count_is_that_of_the_kernels(b):
    """One kernel a call; two where a sequence is split and its shares are joined; none without rows."""
    lib = b.load()

    def count(f):
        before = lib.cp_spec_launch_count(None)
        f()
        return lib.cp_spec_launch_count(None) - before
    cache, k, q = b.Kv4Cache(512, 16, 2, 64), _randn(1, 1, 2, 2, 64), _randn(2, 1, 2, 4, 64)
    w = b.w4_pack(_randn(3, 32, 128))
    pos, lens, page = _int([0]), _int([2]), _int([[0]])
    assert count(lambda: b.w4_pack(_randn(3, 32, 128))) == 1
    assert count(lambda: b.w4_unpack(w)) == 1
    assert count(lambda: b.w4_gemv(_randn(4, 2, 128), w)) == 1
    assert count(lambda: b.w4_gemv(_randn(4, 0, 128), w)) == 0
    assert count(lambda: cache.append(k, k, pos)) == 1
    assert count(lambda: cache.read(2)) == 1
    assert count(lambda: cache.attention(q, lens, pages=page)) == 1
    per = lib.cp_spec_kv4_attention_bytes(cache._shape, 512, 1, 2, 4, 0)
    assert per > 0  # a table of 8192 positions is split
    assert count(lambda: cache.attention(q, lens)) == 2
