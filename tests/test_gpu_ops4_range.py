"""The largest magnitudes that the product and the attention are made for, and inputs of very different size side by side."""
import pytest

from fp4_reference import DTYPES, HALF_STEP, attention64, gemv_bound, hold, visible
from gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu
BIG = 2.0 ** 100


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


def _upto(t, size):
    """Scaled so that the largest magnitude is `size`."""
    return (t.double() * (size / t.double().abs().max())).to(t.dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
def test_large_weights(b, dtype, group):
    w = _upto(_randn(1, 100, 1000).abs(), BIG)  # of one sign: the sums are as large as they get
    x = _randn(2, 5, 1000, dtype=DTYPES[dtype]).abs()
    y = b.w4_gemv(x, b.w4_pack(w, group), out_dtype=torch.float32)
    ref, bound = gemv_bound(x, w, group, torch.float32)
    assert ((y.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("keys,values", [(BIG, 1.0), (1.0, BIG), (BIG, BIG), (1.0 / BIG, 2.0 ** -50)])
def test_large_and_small_keys_and_values(b, d, keys, values, dtype):
    n, m, nq, nkv = 700, 3, 4, 2
    cache = b.Kv4Cache(44, 16, nkv, d)
    k, v = (_upto(_randn(i, 1, n, nkv, d, dtype=DTYPES[dtype]), s) for i, s in ((1, keys), (2, values)))
    cache.append(k, v, _int([0]))
    q = _randn(3, 1, m, nq, d, dtype=DTYPES[dtype])
    scale = float(torch.tensor(4 * d ** -0.5 / keys, dtype=torch.float32))
    o, lse = cache.attention(q, _int([n]), scale=scale, want_lse=True)
    see = visible(n, m, m, None).cuda()
    ref, ls, bound, lbound = attention64(q[0], hold(k[0], 32), hold(v[0], 32), see, scale)
    assert ((o[0].double() - ref).abs() <= bound + HALF_STEP[q.dtype] * ref.abs()).all()
    assert ((lse[0].double() - ls).abs() <= lbound).all()


@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -20, 2.0 ** -30])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_small_inputs_beside_a_large_one(b, dtype, ratio):
    """The bound that the header states for the rows of x: 22 bits (or all of a 16-bit type's), never finer than 2^-39 of
    the largest of an input's 128 neighbours; weights of zero keep the large one out of half of the outputs."""
    w, x = _randn(1, 64, 256), _randn(2, 3, 256, scale=ratio).to(DTYPES[dtype])
    w[:, 7] = 0.0
    x[:, 7] = 4.0
    y = b.w4_gemv(x, b.w4_pack(w, 32), out_dtype=torch.float32)
    ref, bound = gemv_bound(x, w, 32, torch.float32)
    floor = 2.0 ** -39 * 4.0 * hold(w, 32).abs()[:, :128].sum(-1)
    assert ((y.double() - ref).abs() <= bound + floor).all()


@pytest.mark.parametrize("ratio", [2.0 ** -8, 2.0 ** -16, 2.0 ** -24])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_small_channels_beside_large_ones(b, dtype, ratio):
    """The bound that the header states for values: 11 or 22 bits, never finer than 2^-31 of the largest scale that the row
    sees, at a weight of 1 for the largest.  Small channels beside a large group, and a small position beside a large one
    of little weight; each channel is held to its own size, and each row to what it sees."""
    n, m, nq, nkv, d = 300, 4, 2, 1, 128
    cache = b.Kv4Cache(19, 16, nkv, d)
    k, v = (_randn(i, 1, n, nkv, d, dtype=DTYPES[dtype]) for i in (1, 2))
    v[..., 32:] *= ratio
    v[:, n - 2] *= 64.0  # a window row: rows before it do not see it
    cache.append(k, v, _int([0]))
    q = _randn(3, 1, m, nq, d, dtype=DTYPES[dtype])
    o = cache.attention(q, _int([n]))
    hk, hv, see = hold(k[0], 32), hold(v[0], 32), visible(n, m, m, None).cuda()
    for i in range(m):  # row by row over what it sees, so that the bound's floor counts nothing else
        n_i = n - m + 1 + i
        ref, _, bound, _ = attention64(q[0, i:i + 1], hk[:n_i], hv[:n_i], see[i:i + 1, :n_i], d ** -0.5)
        err = (o[0, i:i + 1].double() - ref).abs()
        assert (err <= bound + HALF_STEP[q.dtype] * ref.abs()).all(), (i, float((err / bound).max()))
