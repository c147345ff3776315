"""The 4-bit KV cache and attention over it against float64 on the values that the format holds."""
import math
import random

import pytest

from fp4_reference import DTYPES, HALF_STEP, attention64, hold, visible
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


def _table(seed, seqs, per, spare=0):
    """A shuffled page table [seqs, per] over seqs * per + spare pages."""
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(seqs * per + spare, generator=g)[:seqs * per].to(torch.int32).view(seqs, per).cuda()


def _poison(cache):
    """Codes and scales as an unused page may hold them: every scale a NaN."""
    cache.data.fill_(0xFF)


# ----------------------------------------------------------- write and read
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("nkv,d,page", [(1, 64, 16), (8, 128, 16), (3, 128, 48), (2, 256, 64)])
@pytest.mark.parametrize("rows,first", [(1, 0), (1, 5), (2, 15), (7, 30), (33, 1), (64, 16)])
def test_rows_read_back_as_the_held_values(b, nkv, d, page, dtype, rows, first):
    seqs, per = 3, -(-(first + rows + 9) // page)
    cache = b.Kv4Cache(seqs * per + 2, page, nkv, d)
    pages = _table(rows + first, seqs, per, spare=2)
    k, v = (_randn(i + rows, seqs, rows, nkv, d, dtype=DTYPES[dtype]) for i in (1, 2))
    pos = _int([first, first + 1, max(first - 1, 0)])
    cache.append(k, v, pos, pages=pages)
    length = first + rows + 3
    for out in (torch.float32, DTYPES[dtype]):
        gk, gv = cache.read(length, pages=pages, dtype=out)
        for i in range(seqs):
            p = int(pos[i])
            for got, want in ((gk, k), (gv, v)):
                assert torch.equal(got[i, p:p + rows], hold(want[i], 32).float().to(out))
                assert (got[i, :p] == 0).all() and (got[i, p + rows:] == 0).all()


def test_scales_between_two_bfloat16_numbers(b):
    """Largest magnitudes whose sixth lies within a float32 step of the middle of two bfloat16 numbers: the scale is the
    rounded product with float32(1/6) in the cache and in a packed matrix."""
    top = [float.fromhex(h) for h in ("0x1.907ffep+1", "0x1.c07ffep+1", "0x1.c67ffep+1", "0x1.cc7ffep+1")]
    x = torch.zeros(1, 16, 1, 64, device="cuda")
    for i, t in enumerate(top):
        for j in range(4):
            x[0, 4 * i + j, 0, 5], x[0, 4 * i + j, 0, 40] = t * 2.0 ** (j - 2), -t * 2.0 ** j
            x[0, 4 * i + j, 0, 20] = 1.5 * 2.0 ** (j - 2)
    cache = b.Kv4Cache(1, 16, 1, 64)
    cache.append(x, -x, _int([0]))
    k, v = cache.read(16)
    assert torch.equal(k.double(), hold(x, 32)) and torch.equal(v.double(), hold(-x, 32))
    assert torch.equal(b.w4_unpack(b.w4_pack(x[0, :, 0], 32)).double(), hold(x[0, :, 0], 32))


def test_values_that_are_not_finite_read_back_as_nan(b):
    cache = b.Kv4Cache(1, 16, 1, 64)
    k, v = _randn(1, 1, 4, 1, 64), _randn(2, 1, 4, 1, 64)
    k[0, 1, 0, 3], v[0, 2, 0, 40], v[0, 3, 0, 0] = float("inf"), float("nan"), 1e-44
    cache.append(k, v, _int([0]))
    gk, gv = cache.read(4)
    for got, want in ((gk, hold(k, 32)), (gv, hold(v, 32))):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got).double(), torch.nan_to_num(want))
    assert torch.isnan(gk[0, 1, 0, :32]).all() and not torch.isnan(gk[0, 1, 0, 32:]).any()


def test_token_by_token_is_the_same_as_at_once(b):
    """Single-row writes share the bytes of a token pair with the row before; every slot keeps what it held."""
    seqs, n, nkv, d = 2, 37, 2, 128
    k, v = _randn(1, seqs, n, nkv, d), _randn(2, seqs, n, nkv, d)
    whole, steps = b.Kv4Cache(8, 16, nkv, d), b.Kv4Cache(8, 16, nkv, d)
    whole.append(k, v, _int([0, 0]))
    _poison(steps)
    order = list(range(n))
    random.Random(3).shuffle(order)
    for p in order:
        steps.append(k[:, p:p + 1].contiguous(), v[:, p:p + 1].contiguous(), _int([p, p]))
    for a, c in zip(whole.read(n, n_seqs=2), steps.read(n, n_seqs=2)):
        assert torch.equal(a, c)


def test_rows_counts_slices_and_untouched_slots(b):
    """n_rows per sequence (clamped), rows inside a fused projection, positions outside the pages; the rest stays."""
    seqs, m, nkv, d = 4, 6, 2, 64
    cache = b.Kv4Cache(8, 16, nkv, d)
    k0, v0 = _randn(1, seqs, 32, nkv, d), _randn(2, seqs, 32, nkv, d)
    cache.append(k0, v0, _int([0] * seqs))
    fused = _randn(3, seqs, m, 3 * nkv * d, dtype=torch.bfloat16)
    k = fused[..., nkv * d:2 * nkv * d].unflatten(-1, (nkv, d))
    v = fused[..., 2 * nkv * d:].unflatten(-1, (nkv, d))
    pos, count = [3, 29, -2, 10], [6, 99, 5, -4]
    cache.append(k, v, _int(pos), n_rows=_int(count))
    want_k, want_v = hold(k0, 32), hold(v0, 32)
    for i in range(seqs):
        for r in range(min(max(count[i], 0), m)):
            if 0 <= pos[i] + r < 32:
                want_k[i, pos[i] + r], want_v[i, pos[i] + r] = hold(k[i, r], 32), hold(v[i, r], 32)
    gk, gv = cache.read(32, n_seqs=seqs)
    assert torch.equal(gk.double(), want_k) and torch.equal(gv.double(), want_v)


def test_two_sequences_write_one_page(b):
    """Neighbouring slots of one page, written by two sequences of one call: they share the bytes of the value codes."""
    cache = b.Kv4Cache(1, 16, 4, 128)
    pages = torch.zeros(16, 1, dtype=torch.int32, device="cuda")
    k, v = _randn(1, 16, 1, 4, 128), _randn(2, 16, 1, 4, 128)
    for _ in range(10):
        _poison(cache)
        cache.append(k, v, torch.arange(16, dtype=torch.int32, device="cuda"), pages=pages)
        gk, gv = cache.read(16, pages=pages[:1])
        assert torch.equal(gk[0].double(), hold(k[:, 0], 32)) and torch.equal(gv[0].double(), hold(v[:, 0], 32))


def test_pages_outside_the_cache(b):
    """They are neither written nor read; the cache beside them stays as it was."""
    cache = b.Kv4Cache(3, 16, 1, 64)
    before = cache.data.clone()
    bad = _int([[-1, 3], [1 << 30, -(1 << 31)]])
    k, v = _randn(1, 2, 32, 1, 64), _randn(2, 2, 32, 1, 64)
    cache.append(k, v, _int([0, 0]), pages=bad)
    assert torch.equal(cache.data, before)
    _poison(cache)
    gk, gv = cache.read(40, pages=bad)  # 40: past the table too
    assert (gk == 0).all() and (gv == 0).all()
    mixed = _int([[7, 2], [1, 9]])
    cache.append(k, v, _int([0, 0]), pages=mixed)
    gk, gv = cache.read(32, pages=mixed, lens=_int([32, 20]))
    assert (gk[0, :16] == 0).all() and torch.equal(gk[0, 16:].double(), hold(k[0, 16:], 32))
    assert torch.equal(gv[1, :16].double(), hold(v[1, :16], 32)) and (gv[1, 16:] == 0).all()


# ---------------------------------------------------------------- attention
def _filled(b, seqs, length, nkv, d, page, dtype, seed, poison=True):
    per = max(1, -(-length // page))
    cache = b.Kv4Cache(seqs * per + 1, page, nkv, d)
    if poison:
        _poison(cache)
    pages = _table(seed, seqs, per, spare=1)
    k = _randn(seed, seqs, max(length, 1), nkv, d, dtype=DTYPES[dtype])
    v = _randn(seed + 1, seqs, max(length, 1), nkv, d, dtype=DTYPES[dtype]) + 0.5
    return cache, pages, k, v.to(DTYPES[dtype])


def _against_64(b, cache, pages, k, v, q, lens, n_rows=None, mask=None, scale=None, hide=None):
    """Attention through the library, compared sequence by sequence; hide(i, see) may take positions away (bad pages)."""
    seqs, m, nq, d = q.shape
    out = torch.full_like(q, 3.0)
    got, lse = cache.attention(q, _int(lens), pages=pages, n_rows=None if n_rows is None else _int(n_rows), mask=mask,
                               scale=scale, out=out, want_lse=True)
    assert got is out
    sc = d ** -0.5 if scale is None else scale
    for i in range(seqs):
        n = m if n_rows is None else min(max(n_rows[i], 0), m)
        length = min(max(lens[i], 0), pages.shape[1] * cache.page_size)
        see = visible(length, n, m, None if mask is None else mask[i].tolist())
        if hide is not None:
            hide(i, see)
        see = see[:n].to(q.device)
        o, ls, bound, lbound = attention64(q[i, :n], hold(k[i, :length], 32), hold(v[i, :length], 32), see, sc)
        err = (got[i, :n].double() - o).abs()
        full = bound + HALF_STEP[q.dtype] * o.abs()
        assert (err <= full).all(), (i, float((err / full).max()))
        none = torch.isinf(ls)
        assert torch.equal(torch.isinf(lse[i, :n]), none) and (got[i, :n][none] == 0).all()
        lerr = (lse[i, :n].double() - ls).abs()[~none]
        assert (lerr <= lbound[~none]).all(), (i, float((lerr / lbound[~none]).max()))
        assert (got[i, n:] == 3.0).all()  # rows past the sequence's own are left as they were
    return got, lse


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("nq,nkv,d", [(4, 4, 64), (16, 8, 128), (8, 1, 128), (4, 2, 256), (6, 2, 64)])
@pytest.mark.parametrize("m,lens", [(1, [1, 2, 15, 16, 17, 100]), (4, [4, 5, 33, 64, 250, 3]), (8, [8, 40, 0, 1, 129, 500]),
                                    (13, [13, 20, 300, 47, 16, 90])])
def test_windows(b, nq, nkv, d, m, lens, dtype):
    """Causal windows; lengths below the window leave its first rows with nothing to see."""
    cache, pages, k, v = _filled(b, len(lens), max(lens), nkv, d, 16, dtype, seed=m)
    cache.append(k, v, _int([0] * len(lens)), pages=pages, n_rows=_int(lens))
    q = _randn(9, len(lens), m, nq, d, dtype=DTYPES[dtype], scale=2.0)
    _against_64(b, cache, pages, k, v, q, lens)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("seqs,m,nq,nkv,d,length,page", [
    (1, 1, 32, 8, 128, 20000, 64), (1, 1, 8, 8, 64, 5000, 16), (2, 4, 16, 8, 128, 3001, 48), (1, 2, 4, 1, 256, 9999, 128),
    (40, 1, 8, 4, 64, 777, 32)])
def test_long_sequences(b, seqs, m, nq, nkv, d, length, page, dtype):
    """Sequences that several CTAs split, unequal lengths."""
    lens = [max(m, length - 131 * i) for i in range(seqs)]
    cache, pages, k, v = _filled(b, seqs, length, nkv, d, page, dtype, seed=length)
    cache.append(k, v, _int([0] * seqs), pages=pages, n_rows=_int(lens))
    q = _randn(9, seqs, m, nq, d, dtype=DTYPES[dtype])
    if seqs > 4:  # a few of many, compared on the host side
        got, lse = cache.attention(q, _int(lens), pages=pages, want_lse=True)
        pick = [0, 1, seqs // 2, seqs - 1]
        one, l1 = _against_64(b, cache, pages[pick], k[pick], v[pick], q[pick], [lens[i] for i in pick])
        assert ((got[pick] - one).abs().double() <= 4 * HALF_STEP[q.dtype] * (one.abs().double() + 1)).all()
    else:
        _against_64(b, cache, pages, k, v, q, lens)


def _trees(seed, seqs, m):
    rng = random.Random(seed)
    rows = []
    for _ in range(seqs):
        of = []
        for i in range(m):
            parent = rng.randint(-1, i - 1)
            of.append((1 << i) | (of[parent] if parent >= 0 else 0))
        rows.append(of)
    return rows


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,nq,nkv,d", [(7, 8, 4, 64), (24, 32, 8, 64), (63, 4, 2, 128), (64, 2, 2, 128), (20, 6, 2, 256)])
def test_tree_masks(b, m, nq, nkv, d, dtype):
    lens = [m, m + 1, 200, m + 77]
    cache, pages, k, v = _filled(b, 4, max(lens), nkv, d, 32, dtype, seed=m)
    cache.append(k, v, _int([0] * 4), pages=pages, n_rows=_int(lens))
    rows = _trees(m, 4, m)
    rows[1][m // 2] = 0                      # sees the prefix alone
    rows[0][0] = 0                           # sees nothing at all
    rows[2] = [(1 << 64) - 1] * m            # every bit, those past the window among them
    mask = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows], dtype=torch.int64, device="cuda")
    q = _randn(5, 4, m, nq, d, dtype=DTYPES[dtype])
    _against_64(b, cache, pages, k, v, q, lens, mask=mask)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_fewer_rows_than_the_window(b, dtype):
    """n_rows: rows past it are left as they were, lengths beyond the pages are clamped, none at all is fine."""
    lens, n_rows = [40, 9, 0, 1000, 5, 30], [3, 0, 2, 5, -1, 99]
    cache, pages, k, v = _filled(b, 6, 64, 2, 128, 32, dtype, seed=4)
    cache.append(k, v, _int([0] * 6), pages=pages)
    q = _randn(9, 6, 5, 4, 128, dtype=DTYPES[dtype])
    _against_64(b, cache, pages, k, v, q, lens, n_rows=n_rows)


def test_what_a_row_does_not_see_cannot_reach_it(b):
    """NaN and infinities in masked positions, past the length and in unused pages (the cache starts as NaN scales)."""
    m, lens = 4, [20, 35]
    cache, pages, k, v = _filled(b, 2, 48, 2, 128, 16, "bf16", seed=4)
    cache.append(k, v, _int([0, 0]), pages=pages, n_rows=_int(lens))
    rows = [[1, 2, 4, 8], [1, 3, 7, 8]]
    mask = torch.tensor(rows, dtype=torch.int64, device="cuda")
    q = _randn(9, 2, m, 4, 128, dtype=torch.bfloat16)
    clean = cache.attention(q, _int(lens), pages=pages, mask=mask)
    # the window's row 1 of both sequences is spoilt: only rows that see it may change
    bad = torch.full((2, 1, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    bad[1] = float("inf")
    cache.append(bad, bad, _int([n - m + 1 for n in lens]), pages=pages)
    spoilt = cache.attention(q, _int(lens), pages=pages, mask=mask)
    for i in range(2):
        for r in range(m):
            if rows[i][r] & 2:
                assert torch.isnan(spoilt[i, r]).all()
            else:
                assert torch.equal(spoilt[i, r], clean[i, r])


def test_nan_values_reach_their_own_channels(b):
    cache, pages, k, v = _filled(b, 1, 32, 1, 64, 16, "fp32", seed=4)
    v[0, 5, 0, 40] = float("nan")
    cache.append(k, v, _int([0]), pages=pages)
    o = cache.attention(_randn(1, 1, 2, 1, 64), _int([32]), pages=pages)
    assert torch.isnan(o[..., 32:]).all() and torch.isfinite(o[..., :32]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_pages_outside_the_cache_are_left_out(b, dtype):
    lens = [64, 50, 16]
    cache, pages, k, v = _filled(b, 3, 64, 2, 64, 16, dtype, seed=4)
    cache.append(k, v, _int([0] * 3), pages=pages)
    pages[0, 1], pages[1, 0], pages[1, 3], pages[2, 0] = -1, cache.n_pages, 1 << 30, -7
    q = _randn(9, 3, 2, 4, 64, dtype=DTYPES[dtype])

    def hide(i, see):
        for at in ([1], [0, 3], [0])[i]:
            see[:, 16 * at:16 * at + 16] = False
    _against_64(b, cache, pages, k, v, q, lens, hide=hide)


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 1e3, 1e6])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_values_of_unequal_size(b, spread, dtype):
    """The scales of the values grow or shrink along the sequence by many powers of two."""
    cache, pages, k, v = _filled(b, 1, 600, 1, 128, 16, dtype, seed=4)
    v = (v.float() * torch.logspace(0, math.log10(spread), 600, device="cuda").view(1, -1, 1, 1)).to(v.dtype)
    cache.append(k, v, _int([0]), pages=pages)
    _against_64(b, cache, pages, k, v, _randn(9, 1, 3, 2, 128, dtype=DTYPES[dtype]), [600])


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0, 1e-30])
def test_scales_and_peaked_scores(b, scale):
    cache, pages, k, v = _filled(b, 2, 300, 2, 64, 16, "fp32", seed=4)
    cache.append(k, v, _int([0] * 2), pages=pages)
    _against_64(b, cache, pages, k, v, _randn(9, 2, 4, 4, 64, scale=5.0), [300, 77], scale=scale)


def test_scores_that_keep_growing(b):
    """Each position scores higher than the last: the running maximum moves all along, over several CTAs."""
    n, d = 4000, 64
    cache, pages, k, v = _filled(b, 1, n, 1, d, 16, "fp32", seed=4)
    q = torch.ones(1, 2, 1, d, device="cuda")
    k = torch.linspace(-20, 60, n, device="cuda").view(1, n, 1, 1).expand(1, n, 1, d).contiguous()
    for keys in (k, k.flip(1).contiguous()):
        cache.append(keys, v, _int([0]), pages=pages)
        _against_64(b, cache, pages, keys, v, q, [n])


def test_strided_queries_and_outputs(b):
    cache, pages, k, v = _filled(b, 3, 50, 2, 64, 16, "bf16", seed=4)
    cache.append(k, v, _int([0] * 3), pages=pages)
    lens = _int([50, 20, 33])
    fused = _randn(1, 3, 5, 8 * 64 + 24, dtype=torch.bfloat16)
    q = fused[..., 8:8 + 256].unflatten(-1, (4, 64))
    assert q.data_ptr() % 16 == 0
    want = cache.attention(q.contiguous(), lens, pages=pages)
    wide = torch.full((3, 5, 6, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    got = cache.attention(q, lens, pages=pages, out=wide[:, :, 1:5])
    assert torch.equal(got, want) and (wide[:, :, 0] == 9.0).all() and (wide[:, :, 5] == 9.0).all()


def test_offsets_beyond_32_bits(b):
    """A cache of more than 4 GB: pages at its end."""
    n_pages = 1 << 16
    cache = b.Kv4Cache(n_pages, 64, 8, 128)  # 4.8 GB
    assert cache.data.numel() > 1 << 32
    pages = torch.arange(n_pages - 1, n_pages - 9, -1, dtype=torch.int32, device="cuda").view(2, 4)
    k, v = _randn(1, 2, 200, 8, 128, dtype=torch.bfloat16), _randn(2, 2, 200, 8, 128, dtype=torch.bfloat16)
    cache.append(k, v, _int([0, 0]), pages=pages)
    gk, gv = cache.read(200, pages=pages)
    assert torch.equal(gk.double(), hold(k, 32)) and torch.equal(gv.double(), hold(v, 32))
    _against_64(b, cache, pages, k, v, _randn(9, 2, 2, 8, 128, dtype=torch.bfloat16), [200, 150])


def test_offsets_within_a_page_beyond_32_bits(b):
    """Pages of 2.4 GB: the last head's slots lie past 2^31 bytes of their page."""
    for nkv, d, page, first in ((1024, 64, 1 << 15, 0), (8, 256, 1 << 20, 131072 - 7)):
        cache = b.Kv4Cache(1, page, nkv, d)
        assert cache.data.numel() > 1 << 31
        k, v = _randn(1, 1, 20, nkv, d, dtype=torch.bfloat16), _randn(2, 1, 20, nkv, d, dtype=torch.bfloat16)
        cache.append(k, v, _int([first]))
        # the same memory as pages of one tile of one head: the last head's first tiles with these rows
        tiles = page // 16
        small = b.Kv4Cache(1, 16, 1, d)
        small.shape.n_pages = small.n_pages = nkv * tiles
        small.data = cache.data
        t0 = first // 16
        table = _int([[(nkv - 1) * tiles + t0 + j for j in range(3)]])
        skip = first - 16 * t0
        gk, gv = small.read(skip + 20, pages=table)
        for got, want in ((gk, hold(k, 32)), (gv, hold(v, 32))):
            assert torch.equal(got[0, skip:, 0].double(), want[0, :, -1]) and (got[0, :skip] == 0).all()
        gk, gv = cache.read(first + 20, dtype=torch.bfloat16)
        for got, want in ((gk, hold(k, 32)), (gv, hold(v, 32))):
            assert torch.equal(got[:, first:], want.float().to(torch.bfloat16)) and not got[:, :first].any()
        del gk, gv
        if first == 0:
            _against_64(b, cache, _int([[0]]), k, v, _randn(9, 1, 2, nkv, d, dtype=torch.bfloat16), [20])


def test_same_results_again_captured_and_on_another_stream(b):
    """Long enough to be split over CTAs; lengths and queries change between the replays of one graph."""
    cache, pages, k, v = _filled(b, 2, 4000, 2, 128, 64, "bf16", seed=4)
    cache.append(k, v, _int([0, 0]), pages=pages)
    q, lens = _randn(9, 2, 4, 8, 128, dtype=torch.bfloat16), _int([4000, 1234])
    want = cache.attention(q, lens, pages=pages)
    for _ in range(5):
        assert torch.equal(cache.attention(q, lens, pages=pages), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = cache.attention(q, lens, pages=pages)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    kn, vn, pos = k[:, :4].clone(), v[:, :4].clone(), _int([3996, 1230])
    with torch.cuda.graph(graph):
        cache.append(kn, vn, pos, pages=pages)
        cache.attention(q, lens, pages=pages, out=out)
    for step in range(2):
        q.copy_(_randn(20 + step, 2, 4, 8, 128))
        kn.copy_(_randn(30 + step, 2, 4, 2, 128))
        lens.copy_(_int([3000 + step, 70]))
        pos.copy_(_int([2996 + step, 66]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cache.attention(q, lens, pages=pages))


def test_one_decoder_layer_in_4_bits(b):
    """The operators in a run, as a decoding step uses them: fused projection, rows written, attention, output
    projection; a prompt, then single tokens, then a verify window, each step held against 64 bits on its own inputs."""
    from fp4_reference import gemv_bound
    seqs, nq, nkv, d, hidden = 3, 4, 2, 64, 192
    wqkv = _randn(1, (nq + 2 * nkv) * d, hidden, dtype=torch.bfloat16, scale=0.1)
    wo = _randn(2, hidden, nq * d, dtype=torch.bfloat16, scale=0.1)
    pq, po = b.w4_pack(wqkv, 32), b.w4_pack(wo, 64)
    cache = b.Kv4Cache(12, 16, nkv, d)
    pages = _table(1, seqs, 4)
    held = [[torch.zeros(seqs, 0, nkv, d, device="cuda")] for _ in range(2)]
    done = 0
    for step, m in enumerate((20, 1, 1, 4)):
        x = _randn(10 + step, seqs, m, hidden)
        qkv = b.w4_gemv(x.view(seqs * m, hidden), pq).view(seqs, m, -1)
        ref, bound = gemv_bound(x.view(seqs * m, hidden), wqkv, 32, torch.float32)
        assert ((qkv.view(seqs * m, -1).double() - ref).abs() <= bound).all()
        q = qkv[..., :nq * d].unflatten(-1, (nq, d))
        k = qkv[..., nq * d:(nq + nkv) * d].unflatten(-1, (nkv, d))
        v = qkv[..., (nq + nkv) * d:].unflatten(-1, (nkv, d))
        cache.append(k, v, _int([done] * seqs), pages=pages)
        held[0].append(k)
        held[1].append(v)
        done += m
        o, _ = _against_64(b, cache, pages, torch.cat(held[0], 1), torch.cat(held[1], 1), q, [done] * seqs)
        y = b.w4_gemv(o.view(seqs * m, nq * d), po)
        ref, bound = gemv_bound(o.view(seqs * m, nq * d), wo, 64, torch.float32)
        assert ((y.double() - ref).abs() <= bound).all()
    gk, gv = cache.read(done, pages=pages)
    assert torch.equal(gk.double(), hold(torch.cat(held[0], 1), 32)) and torch.equal(gv.double(), hold(torch.cat(held[1], 1), 32))
