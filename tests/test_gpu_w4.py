"""Products with 4-bit weights against float64 on the values that the format holds."""
import pytest

from fp4_reference import DTYPES, E2M1, gemv_bound, hold
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


def _check(b, x, w, group, out_dtype=None, **kw):
    y = b.w4_gemv(x, b.w4_pack(w, group), out_dtype=out_dtype, **kw)
    ref, bound = gemv_bound(x, w, group, y.dtype)
    err = (y.double() - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 128), (17, 129), (40, 95), (1000, 1003), (100, 4100)])
def test_pack_holds_the_nearest_values(b, n, k, dtype, group):
    w = _randn(n + k, n, k, dtype=DTYPES[dtype])
    p = b.w4_pack(w, group)
    assert torch.equal(b.w4_unpack(p).double(), hold(w, group))
    for out in (torch.bfloat16, torch.float16):
        assert torch.equal(b.w4_unpack(p, out), hold(w, group).to(torch.float32).to(out))


def test_pack_ties_zeros_and_values_without_a_scale(b):
    """Every tie point goes to the even code, both signs; a group with an infinity or a NaN reads back as NaN, a group
    whose scale rounds to zero as zeros; scales near both ends of float32."""
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    ties = torch.cat([mid, -mid, E2M1, -E2M1]).float()  # 30 values, the largest 6
    w = torch.zeros(12, 64)
    for i, s in enumerate((1.0, 0.375, 2.0 ** -130, 2.0 ** 120)):
        w[i, :30] = ties * s
    w[4, 5], w[5, 40], w[6, 0] = float("inf"), float("nan"), -float("inf")
    w[7] = 1e-41
    w[8, 3] = 3e38
    w[9] = torch.linspace(-1, 1, 64)
    w[10, 32:] = -0.0
    w = w.cuda()
    got, want = b.w4_unpack(b.w4_pack(w, 32)).double(), hold(w, 32)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.isnan(got[4, :32]).all() and not torch.isnan(got[4, 32:]).any()


def test_pack_of_a_slice(b):
    """A row stride, and rows that are not 16-byte aligned."""
    w = _randn(3, 50, 301, dtype=torch.bfloat16)
    for part in (w[:, :200], w[::2, :77]):
        assert torch.equal(b.w4_unpack(b.w4_pack(part, 32)).double(), hold(part, 32))


@pytest.mark.parametrize("dtype,out", [("fp32", None), ("bf16", None), ("fp16", None), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("rows,n,k,group", [
    (1, 1, 1, 32), (1, 16, 128, 32), (1, 4096, 1024, 32), (2, 33, 257, 64), (3, 17, 129, 128), (4, 2048, 1024, 32),
    (5, 1999, 1001, 32), (7, 300, 640, 128), (8, 2048, 6144, 64), (9, 5000, 384, 64), (16, 640, 2049, 32),
    (17, 48, 2000, 128), (31, 100, 96, 32), (33, 129, 1024, 64), (64, 1024, 2048, 128), (70, 36, 300, 32),
    (1, 20000, 512, 128), (2, 8192, 8192, 32)])
def test_product(b, rows, n, k, group, dtype, out):
    w = _randn(7 * n + k, n, k, dtype=torch.bfloat16, scale=0.02)
    x = _randn(rows, rows, k, dtype=DTYPES[dtype])
    _check(b, x, w, group, DTYPES[out] if out else None)


@pytest.mark.parametrize("rows,dtype", [(1, "fp32"), (3, "fp32"), (6, "bf16"), (20, "fp16")])
def test_longest_rows(b, rows, dtype):
    """k at its limit: fewer rows fit beside the rings, so they go in several blocks."""
    k = b.MAX_W4_K
    w = _randn(1, 24, k, dtype=torch.bfloat16)
    _check(b, _randn(2, rows, k, dtype=DTYPES[dtype]), w, 32)


def test_sums_of_one_sign(b):
    """All products positive: a truncating accumulation over a long row would show as a bias."""
    w = _randn(5, 64, 8192).abs()
    x = _randn(6, 2, 8192).abs()
    y = _check(b, x, w, 128)
    ref, _ = gemv_bound(x, w, 128, torch.float32)
    # one group of 128 is the longest sum in the tensor core: 8 steps, measured below 2^-21 relative in all
    assert float(((y.double() - ref) / ref).abs().max()) < 2.0 ** -21


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-9, 1e9, 1e30])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_range_of_the_rows(b, scale, dtype):
    w = _randn(8, 50, 300)
    x = _randn(9, 3, 300, dtype=DTYPES[dtype], scale=scale)
    _check(b, x, w, 32)


def test_one_large_element(b):
    """Elements 2^-24 of the block's largest still count with 11 bits and more."""
    w = _randn(8, 64, 128)
    w[:, 7] = 0.0
    w[::2, 7] = 1e-3  # even rows see the large element, odd rows only the small ones
    x = _randn(9, 2, 128, dtype=torch.bfloat16)
    x[:, 7] = 2.0 ** 24
    y = b.w4_gemv(x, b.w4_pack(w, 32), out_dtype=torch.float32)
    h = hold(w, 32)
    odd = h[:, 7] == 0
    ref, mag = x.double() @ h.t(), x.double().abs() @ h.abs().t()
    assert odd.any()
    assert ((y.double() - ref).abs()[:, odd] <= 2.0 ** -11 * mag[:, odd]).all()


def test_values_that_are_not_finite(b):
    w = _randn(1, 40, 256)
    x = _randn(2, 4, 256)
    x[1, 5], x[2, 200], x[2, 3] = float("inf"), float("nan"), 1.0
    y = b.w4_gemv(x, b.w4_pack(w, 32))
    want = x.double() @ hold(w, 32).t()
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
    assert torch.equal(y[1][torch.isinf(y[1])].double(), want[1][torch.isinf(want[1])])
    w[3, 7] = float("nan")
    y = b.w4_gemv(x, b.w4_pack(w, 32))
    assert torch.isnan(y[0, 3]) and torch.isfinite(y[0, :3]).all() and torch.isfinite(y[0, 4:]).all()


def test_strided_rows_and_outputs(b):
    """Rows of x and y inside wider tensors, aligned and not; what lies between the rows of y stays."""
    w = _randn(1, 70, 200, dtype=torch.bfloat16)
    p = b.w4_pack(w, 64)
    for width, at in ((256, 0), (256, 16), (203, 0)):
        x = _randn(width, 5, width, dtype=torch.bfloat16)[:, at:at + 200]
        if x.data_ptr() % 16:
            continue
        for ywidth in (70, 96):
            y = torch.full((5, ywidth), 7.0, dtype=torch.bfloat16, device="cuda")
            b.w4_gemv(x, p, out=y[:, :70])
            ref, bound = gemv_bound(x, w, 64, torch.bfloat16)
            assert ((y[:, :70].double() - ref).abs() <= bound).all()
            assert (y[:, 70:] == 7.0).all()


def test_no_rows(b):
    p = b.w4_pack(_randn(1, 16, 128))
    assert b.w4_gemv(torch.empty(0, 128, device="cuda"), p).shape == (0, 16)


@pytest.mark.parametrize("rows", [4, 16, 40])
def test_a_row_does_not_depend_on_its_neighbours(b, rows):
    p = b.w4_pack(_randn(1, 500, 700), 32)
    x = _randn(2, rows, 700)
    y = b.w4_gemv(x, p)
    other = _randn(3, rows, 700, scale=100.0)
    other[rows // 2] = x[rows // 2]
    assert torch.equal(b.w4_gemv(other, p)[rows // 2], y[rows // 2])
    assert torch.equal(b.w4_gemv(x, p), y)


def test_captured_and_on_two_streams(b):
    w = [_randn(i, 900, 1024, dtype=torch.bfloat16) for i in range(2)]
    p = [b.w4_pack(a, 32) for a in w]
    x = _randn(5, 4, 1024)
    want = [b.w4_gemv(x, q) for q in p]
    out = [torch.empty_like(a) for a in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for q, o in zip(p, out):
            b.w4_gemv(x, q, out=o)
    for scale in (1.0, 2.0):  # powers of two: the same bits, scaled
        x2 = _randn(5, 4, 1024) * scale
        x.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        for o, a in zip(out, want):
            assert torch.equal(o, a * scale)
    x.copy_(_randn(5, 4, 1024))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, q, o in zip(streams, p, out):
        with torch.cuda.stream(s):
            for _ in range(20):
                b.w4_gemv(x, q, out=o)
    torch.cuda.synchronize()
    for o, a in zip(out, want):
        assert torch.equal(o, a)


def test_offsets_beyond_32_bits(b):
    """A packed matrix of more than 2^31 bytes: the rows at its end."""
    n, k = 140000, 32768  # 2.36 GB packed
    lib = b.load()
    nbytes = lib.cp_spec_w4_bytes(n, k, 128)
    assert nbytes > 1 << 31
    w = _randn(1, n, k, dtype=torch.bfloat16)
    p = b.w4_pack(w, 128)
    x = _randn(2, 1, k, dtype=torch.bfloat16)
    y = b.w4_gemv(x, p, out_dtype=torch.float32)
    for rows in (slice(0, 64), slice(n - 64, n)):
        ref, bound = gemv_bound(x, w[rows], 128, torch.float32)
        assert ((y[:, rows].double() - ref).abs() <= bound).all()
