"""The softmax weights of the attention over the 16-bit cache as numbers: tails far below the largest weight, values near
the type's end, the second term of a weight, and rows that share a warp.

Scores are made of few products that float32 holds exactly, so that the distances below count only what the kernels round:
a score times scale * log2(e) and its distance from the reference (2^-19 of a weight for scores within 2^5), the power of
two (2^-21), the weight's 16-bit form, sums and the output."""
import math

import pytest

import kv16_reference as R
from gpu_common import require_gpu, torch
from test_gpu_kv16_attention import Setup, _bits

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def b():
    require_gpu()
    from speculative_decoding_rvq_gb300 import binding
    return binding


def plain(s, scores, values, rows, window=0, sinks=0):
    """Outputs [rows, dim] and the weights [rows, n], in 64 bits, of causal rows at the end whose scores are the same in every row."""
    n = scores.numel()
    see = R.visible(n, rows, window, sinks).cuda()
    e = torch.where(see, torch.exp(scores - scores.max()), 0.0)
    p = e / e.sum(-1, keepdim=True)
    return p @ values, p


def write(s, scores, values):
    """One KV head's keys (channel 0 the score: the queries are 1 there, 0 elsewhere) and values, in every head."""
    n = scores.numel()
    s.q.zero_()
    s.q[..., 0] = 1
    k = torch.zeros(n, s.cache.n_kv_heads, s.dim, device="cuda")
    k[..., 0] = scores.view(-1, 1)
    v = values.unsqueeze(1).expand(n, s.cache.n_kv_heads, s.dim)
    p = torch.arange(n, device="cuda")
    s.cache.append(k.to(s.dtype), v.to(s.dtype).contiguous(), s.table[0, p // s.page].long() * s.page + p % s.page)
    return k[:, 0, 0].to(s.dtype).double(), v[:, 0].to(s.dtype).double()


@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("gap", [12, 14, 16, 18, 20])
@pytest.mark.parametrize("rows,nq,nkv,dim,n", [(1, 8, 2, 128, 32768), (5, 4, 2, 64, 9000), (2, 8, 1, 256, 20000), (60, 2, 1, 256, 9000),
                                                (40, 8, 2, 64, 20000), (200, 4, 2, 128, 32768), (700, 32, 8, 128, 9000)])
def test_tails_below_a_sink(b, rows, nq, nkv, dim, n, gap, spread):
    """A first position of value zero outweighs all others by e^gap: the others are the whole output.

    fp16 weights that lie this far apart are held as 2^13 times themselves at least, with steps of 2^-24: off by 2^-38
    of the largest, and by 2^-11 relative (half a step of one number).  A sum takes at most 1024 additions of 16 positions one
    after the other, each cutting 2^-23: 2^-13, in the values' sum and in the weights'."""
    s = Setup(b, [(n, rows)], nq, nkv, dim, 64, FP)
    g = torch.Generator(device="cuda").manual_seed(gap)
    scores = spread * torch.randn(n, generator=g, device="cuda")
    scores[0] = gap
    values = 1 + 0.25 * torch.rand(n, dim, generator=g, device="cuda")
    values[0] = 0
    scores, values = write(s, scores, values)
    out, lse = s.call(scale=1.0)
    o, p = plain(s, scores, values, rows)
    lost = torch.minimum(p, 2.0 ** -38 * p.amax(-1, keepdim=True)) @ values
    tol = o * (2.0 ** -11 + 2.0 ** -11 + 2 * 2.0 ** -13 + 2 * 2.0 ** -18) + lost + 2.0 ** -25
    off = (out.double() - o.unsqueeze(1)).abs() / tol.unsqueeze(1)
    assert float(off.max()) <= 1, float(((out.double() - o.unsqueeze(1)).abs() / o.unsqueeze(1)).max())


@pytest.mark.parametrize("window", [48, 700])
@pytest.mark.parametrize("gap", [12, 16, 20])
@pytest.mark.parametrize("rows,nq,nkv,dim", [(3, 4, 2, 128), (40, 8, 2, 64), (200, 4, 2, 128), (700, 32, 8, 128), (90, 2, 1, 256)])
def test_tails_of_a_window_below_its_sink(b, rows, nq, nkv, dim, gap, window):
    """The same with a window so short that no row sees a whole tile of it, and a longer one; distances as above."""
    n = 3000
    s = Setup(b, [(n, rows)], nq, nkv, dim, 16, FP)
    g = torch.Generator(device="cuda").manual_seed(gap)
    scores = 0.2 * torch.randn(n, generator=g, device="cuda")
    scores[0] = gap
    values = 1 + 0.25 * torch.rand(n, dim, generator=g, device="cuda")
    values[0] = 0
    scores, values = write(s, scores, values)
    out, lse = s.call(scale=1.0, window=window, sinks=1)
    o, p = plain(s, scores, values, rows, window, 1)
    lost = torch.minimum(p, 2.0 ** -38 * p.amax(-1, keepdim=True)) @ values
    tol = o * (2.0 ** -11 + 2.0 ** -11 + 2 * 2.0 ** -13 + 2 * 2.0 ** -18) + lost + 2.0 ** -25
    off = (out.double() - o.unsqueeze(1)).abs() / tol.unsqueeze(1)
    assert float(off.max()) <= 1, float(((out.double() - o.unsqueeze(1)).abs() / o.unsqueeze(1)).max())


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("nq,nkv,dim", [(1, 1, 64), (4, 2, 128), (2, 1, 256)])
def test_the_second_term_of_a_weight_counts(b, nq, nkv, dim, dtype):
    """Values that cancel: the output is far below the sum of weight * |value|, and its own rounding says nothing.

    A weight as two numbers is off by 2^-16 of itself in bfloat16 (2^-9 twice, and float32's own) and by less than 2^-20
    in fp16; as one number by up to 2^-9 and 2^-12, here about a third of that for the 40 positions together."""
    n = 40
    s = Setup(b, [(n, 1)], nq, nkv, dim, 16, dtype)
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        scores, values = write(s, torch.randn(n, generator=g, device="cuda"), torch.randn(n, dim, generator=g, device="cuda"))
        scores[-1] = 2.0  # (a power of two: no rounding)
        _, p = plain(s, scores, values, 1)
        values[-1] = -(p[:, :-1] @ values[:-1]) / p[0, -1]
        scores, values = write(s, scores, values)
        out, _ = s.call(scale=1.0)
        o, p = plain(s, scores, values, 1)
        A = p @ values.abs()
        rel = 2.0 ** -16 if dtype is BF else 2.0 ** -20
        tol = R.HALF_STEP[dtype] * o.abs() + A * (rel + 2 * (2.0 ** -19 + 2.0 ** -21) + n * 2.0 ** -23) + (2.0 ** -25 if dtype is FP else 0)
        assert ((out.double() - o.unsqueeze(1)).abs() <= tol.unsqueeze(1)).all(), float(((out.double() - o.unsqueeze(1)).abs() / A).max())


@pytest.mark.parametrize("size", ["largest", "tiny"])
@pytest.mark.parametrize("rising", [0.0, 5.4])
@pytest.mark.parametrize("rows,nq,nkv,dim", [(1, 2, 1, 128), (3, 4, 2, 64), (50, 2, 2, 256), (40, 4, 1, 64), (300, 4, 2, 128), (600, 32, 8, 128)])
def test_values_average_to_themselves(b, rows, nq, nkv, dim, rising, size):
    """bfloat16's largest value everywhere: so is the mean, though the sum of n of them is not a float32.  And a tiny one.

    rising: the scores grow by 5.4 (7.8 binary orders) from one tile of 128 positions to the next, so that a running
    maximum that follows late leaves weights above 1.  The sums are off by (n / 16) 2^-23 and the output by half a step,
    so the value itself comes back, or its neighbour."""
    n = 1500
    s = Setup(b, [(n, rows)], nq, nkv, dim, 64, BF)
    top = torch.finfo(BF).max if size == "largest" else 2.0 ** -100
    scores, values = write(s, rising * (torch.arange(n, device="cuda") // 128).float(), torch.full((n, dim), top, device="cuda"))
    values[:, 1::2] *= -1
    write(s, scores.float(), values.float())
    out, lse = s.call(scale=1.0)
    assert torch.isfinite(out).all()
    assert ((out.double().abs() / top - 1).abs() <= 2.0 ** -8).all()
    assert (torch.sign(out[..., 0::2].float()) == 1).all() and (torch.sign(out[..., 1::2].float()) == -1).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("rows,nq,nkv,dim", [(1, 2, 1, 128), (2, 8, 2, 64), (60, 2, 1, 128), (1, 1, 1, 256)])
def test_an_infinity_reaches_from_a_share_that_weighs_nothing(b, rows, nq, nkv, dim, bad):
    """The first half of a split sequence has weights that are zero in float32: an infinite value there still reaches."""
    n = 6000
    s = Setup(b, [(n, rows)], nq, nkv, dim, 64, BF)
    assert n // 64 > 32
    scores = torch.zeros(n, device="cuda")
    scores[: n // 2] = -200.0
    values = torch.ones(n, dim, device="cuda")
    values[7, 5] = bad
    write(s, scores, values)
    out, _ = s.call(scale=1.0)
    if bad == bad:
        assert (out[..., 5] == bad).all()
    else:
        assert torch.isnan(out[..., 5]).all()
    keep = [c for c in range(dim) if c != 5]
    assert torch.equal(out[..., keep], torch.ones_like(out[..., keep]))


@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 2)])
def test_a_rows_bits_are_its_own_at_large_scores(b, dim, heads):
    """Scores around 2^20, where float32 has steps of 1/16 and 1/8: a later row's own largest score moves no bit of an
    earlier row of the same warp."""
    n, rows = 320, 64  # three tiles: one share, the first and the third through one product
    s = Setup(b, [(n, rows)], heads, 1, dim, 16, FP)
    s.q.zero_()
    s.q[..., 0], s.q[..., 1], s.q[..., 2] = 1024, 2, 2.0 ** -6
    k = torch.zeros(n, 1, dim, device="cuda")
    # score * log2(e): 2^20 - 4 or so in the first tile, about 7 more at the first row's own position, far less elsewhere
    x = (2.0 ** 20 - 4) / 1.4426950408889634
    k[:128, 0, 0] = math.floor(x / 1024)
    k[:128, 0, 1] = (x - 1024 * math.floor(x / 1024)) // 2
    slot = torch.arange(n, device="cuda")
    at = s.table[0, slot // 16].long() * 16 + slot % 16
    outs = []
    for far in (0.0, 800.0):
        res = []
        for step in range(16):  # the first row's own score, in steps of 1/16 of a unit
            k[256, 0, 0], k[256, 0, 1], k[256, 0, 2] = k[0, 0, 0], k[0, 0, 1] + 2, 4.0 * step
            k[276, 0, 0] = far
            s.cache.append(k.to(FP), s.v[0], at)
            out, lse = s.call(scale=1.0)
            res.append((out[:20].clone(), lse[:20].clone()))
        outs.append(res)
    for (o0, l0), (o1, l1) in zip(*outs):
        assert torch.equal(_bits(o0), _bits(o1)) and torch.equal(_bits(l0), _bits(l1))


@pytest.mark.parametrize("rows", [2, 150])
def test_a_scale_of_zero_is_zero_however_large_the_products(b, rows):
    s = Setup(b, [(400, rows)], 2, 1, 64, 16, BF)
    s.q.fill_(1e17)
    s.cache.keys.mul_(1e17)
    out, _ = s.call(scale=0.0)
    v = s.v[0].double()
    for r in range(rows):
        n = 400 - rows + r + 1
        mean = v[:n].mean(0)
        tol = 2.0 ** -8 * mean.abs() + (n * 2.0 ** -24 + 2.0 ** -20) * v[:n].abs().mean(0)
        assert ((out[r].double() - mean).abs() <= tol).all(), r


@pytest.mark.parametrize("where", ["one", "all", "behind"])
@pytest.mark.parametrize("rows,nq,nkv,dim,n", [(1, 8, 2, 128, 65536), (2048, 8, 2, 128, 16384), (40, 2, 1, 256, 16384)])
def test_values_that_are_not_finite_cost_a_few_passes(b, rows, nq, nkv, dim, n, where):
    """A NaN among the values (one, every value infinite, or garbage behind the last position only) slows a call by a
    bounded factor: 11 at most was measured."""
    s = Setup(b, [(n - 3, rows)], nq, nkv, dim, 64, BF)

    def time():
        s.call()
        torch.cuda.synchronize()
        best = math.inf
        for _ in range(3):
            t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            t0.record()
            s.call()
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1))
        return best

    clean = time()
    if where == "one":
        s.cache.values[int(s.table[0, 1]), :, 5] = float("nan")
    elif where == "all":
        s.cache.values.fill_(float("inf"))
    else:
        s.cache.data[:, int(s.table[0, (n - 1) // 64]), :, 61:] = float("nan")
    slow = time()
    out, _ = s.call()
    assert torch.isnan(out).all() if where == "one" else (out == float("inf")).all() if where == "all" else torch.isfinite(out).all()
    print(f"rows {rows} dim {dim} n {n} {where}: {clean * 1e3:.0f} -> {slow * 1e3:.0f} us")
    assert slow <= 20 * clean + 0.1, (clean, slow)
