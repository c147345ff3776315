"""What attention over the 4-bit cache does with positions that a row does not see, and with values that are not finite
in positions that it does see but weighs with zero."""
import pytest

from fp4_reference import DTYPES
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


def _largest(dtype, size):
    return min(size, float(torch.finfo(DTYPES[dtype]).max))


@pytest.mark.parametrize("size", [1e6, 1e10, 1e30, float("inf")])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,nq,nkv,d,lens", [
    (4, 16, 8, 128, [4, 16, 21]),      # frames: one tile holds prefix and window
    (6, 4, 2, 64, [6, 500, 37]),       # two column tiles
    (24, 4, 1, 128, [40, 24, 1300]),   # four column tiles (16-bit types), several row tiles
    (8, 2, 1, 256, [8, 90, 700])])
def test_what_a_row_does_not_see_changes_no_bit(b, m, nq, nkv, d, lens, dtype, tree, size):
    """One row of the window becomes large (or NaN): the outputs and the sums of every row that does not see it keep
    every bit, by causal order and by a mask."""
    seqs, spoilt = len(lens), m // 2
    per = -(-max(lens) // 16)
    cache = b.Kv4Cache(seqs * per, 16, nkv, d)
    pages = torch.randperm(seqs * per, generator=torch.Generator().manual_seed(m)).to(torch.int32).view(seqs, per).cuda()
    k, v = (_randn(i, seqs, max(lens), nkv, d, dtype=DTYPES[dtype]) for i in (1, 2))
    cache.append(k, v, _int([0] * seqs), pages=pages, n_rows=_int(lens))
    q = _randn(3, seqs, m, nq, d, dtype=DTYPES[dtype], scale=2.0)
    # row i of the mask sees itself and the rows of its own parity before it: half of the rows do not see `spoilt`
    rows = [sum(1 << j for j in range(i + 1) if (i - j) % 2 == 0) for i in range(m)]
    mask = torch.tensor([rows] * seqs, dtype=torch.int64, device="cuda") if tree else None
    kv_len = _int(lens)
    clean, lse = cache.attention(q, kv_len, pages=pages, mask=mask, want_lse=True)
    assert torch.isfinite(clean).all() and torch.isfinite(lse).all()
    bad = _largest(dtype, size) * _randn(4, seqs, 1, nkv, d).sign()
    if size == float("inf"):
        bad = torch.full_like(bad, float("nan"))
    bad = bad.to(DTYPES[dtype])
    cache.append(bad, bad, kv_len - m + spoilt, pages=pages)
    got, got_lse = cache.attention(q, kv_len, pages=pages, mask=mask, want_lse=True)
    changed = 0
    for i in range(m):
        if rows[i] >> spoilt & 1 if tree else i >= spoilt:
            changed += int((got[:, i] != clean[:, i]).any())
        else:
            assert torch.equal(got[:, i], clean[:, i]), (i, float((got[:, i].float() - clean[:, i].float()).abs().max()))
            assert torch.equal(got_lse[:, i], lse[:, i]), i
    assert changed


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("at", [3, 20, 34, 37])
def test_a_value_weighed_with_zero_still_counts(b, at, dtype):
    """softmax(s) v with a NaN in v is NaN wherever the row sees it, however small its weight: the same in the prefix (3,
    20), in a tile that the window shares (34) and in the window (37), where rows before it do not see it."""
    n, m, nkv, d = 40, 4, 2, 64
    cache = b.Kv4Cache(3, 16, nkv, d)
    k, v = torch.zeros(1, n, nkv, d, device="cuda"), _randn(2, 1, n, nkv, d)
    k[0, 1], k[0, at], v[0, at, :, 40] = 1.0, -10.0, float("nan")
    q = torch.full((1, m, 4, d), 10.0, device="cuda")  # scores of 80, 0 and -800: weights of 1, 2e-35 and 0
    cache.append(k.to(DTYPES[dtype]), v.to(DTYPES[dtype]), _int([0]))
    o = cache.attention(q.to(DTYPES[dtype]), _int([n]))
    for i in range(m):
        assert torch.isfinite(o[0, i, :, :32]).all()
        if at <= n - m + i:
            assert torch.isnan(o[0, i, :, 32:]).all(), i
        else:
            assert torch.isfinite(o[0, i]).all(), i


@pytest.mark.parametrize("value", [0.0, 2.0 ** -110])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sums_of_many_tiny_values(b, dtype, value):
    """2^19 positions of 160 sequences (one run of pages: nothing is split), whose values are zero or far below the
    smallest scale that the weights are brought to, and whose scores lie just below the step at which the reference
    moves: the sum of the weights stays finite."""
    n, seqs = 1 << 19, 160
    cache = b.Kv4Cache(n // 64, 64, 1, 64)
    pages = torch.arange(n // 64, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    k = torch.full((1, n, 1, 64), 6.0, dtype=DTYPES[dtype], device="cuda")
    k[:, :256] = 0.0  # the first pairs of tiles of the eight warps
    cache.append(k, torch.full_like(k, value), _int([0]), pages=pages[:1])
    q = torch.full((seqs, 1, 1, 64), 5.4 / (6 * 64), dtype=DTYPES[dtype], device="cuda")
    o, lse = cache.attention(q, _int([n] * seqs), pages=pages, scale=1.0, want_lse=True)
    s = 6.0 * float(q.double().sum()) / seqs  # 5.4 = 7.8 in powers of two
    want = s + torch.log(torch.tensor(n - 256 + 256 * 2.718281828459045 ** -s, dtype=torch.float64)).item()
    # a lane adds 2^13 weights in float32 (2^-24 of the sum each, in the worst case all to one side)
    assert torch.isfinite(lse).all() and float((lse.double() - want).abs().max()) <= 2.0 ** -11 + 2.0 ** -18
    # scales count as 2^-80 at least, so a product of 2^86 times the scale may be off by half of fp16's smallest step, 2^-25,
    # times a code of at most 6, over a weight of 2^7.79: 2^-116.2; the output's rounding 2^-118
    assert float((o.double() - value).abs().max()) <= (2.0 ** -115 if value else 0.0)
