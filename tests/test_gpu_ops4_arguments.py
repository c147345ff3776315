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


def test_tables_lengths_and_masks_may_be_slices(b):
    """Parts of larger tensors that do not start on 16 bytes, all at once, give what their copies give; in a captured
    call the values at the time of the replay count."""
    seqs, m, nkv, nq, d, per = 3, 3, 2, 4, 64, 5
    k, v, q = (_randn(i, seqs, m, h, d) for i, h in ((1, nkv), (2, nkv), (3, nq)))
    pages = torch.randperm(4 * per).to(torch.int32).view(4, per).cuda()
    pos, count, lens = _int([99, 5, 70, 33]), _int([99, 3, 2, 1]), _int([99, 8, 72, 34])
    mask = torch.tensor([[0] * m, [1, 2, 5], [1, 3, 7], [1, 1, 4]], dtype=torch.int64, device="cuda")
    parts = [t[1:] for t in (pos, count, lens, pages, mask)]
    assert all(t.is_contiguous() and t.data_ptr() % 16 for t in parts)

    def call(cache, pos, count, lens, pages, mask):
        out = torch.zeros_like(q)
        cache.append(k, v, pos, pages=pages, n_rows=count)
        cache.attention(q, lens, pages=pages, n_rows=count, mask=mask, out=out)
        return [out, *cache.read(80, pages=pages, lens=lens)]

    def new():
        return b.Kv4Cache(4 * per, 16, nkv, d)
    got, want = call(new(), *parts), call(new(), *[t.clone() for t in parts])
    for x, y in zip(got, want):
        assert y.any() and torch.equal(x, y)
    cache, graph = new(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = call(cache, *parts)
    pos[2] -= 20
    lens[2] -= 20
    graph.replay()
    torch.cuda.synchronize()
    later = call(new(), *[t.clone() for t in parts])
    assert not torch.equal(later[0], want[0])
    for x, y in zip(got, later):
        assert torch.equal(x, y)
