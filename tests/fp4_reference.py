"""The 4-bit format and its operators in 64 bits, for the tests (test infrastructure; shares no code with the library)."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# a rounding to the type is off by at most half a step of the value
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# ... and below the smallest normal number by half the type's constant step there (bf16 2^-134, fp16 2^-25, fp32 2^-150)
HALF_TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2 for t in HALF_STEP}
# One m16n8k16 step adds 16 products to an accumulator, each addend aligned to the largest and truncated
# (measured: addends below 2^-24 of the largest are lost): at most 17 such losses per step.
MMA_STEP = 17 * 2.0 ** -24

# the float32 number nearest to 1/6: a group's scale is bf16(float32(largest magnitude * SIXTH)); a product of two float32
# numbers is exact in float64, so .float() is its one rounding
SIXTH = float.fromhex("0x1.555556p-3")


def hold(x, group):
    """float64 values that the format holds for x [..., width], groups along the last axis."""
    table = E2M1.to(x.device)
    width = x.shape[-1]
    x = torch.nn.functional.pad(x.double(), (0, -width % group))
    x = x.view(*x.shape[:-1], x.shape[-1] // group, group)
    finite = torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(finite, x, torch.zeros_like(x))
    s = (x.abs().amax(-1, keepdim=True) * SIXTH).float().bfloat16().double()
    r = (x / torch.where(s > 0, s, torch.ones_like(s))).abs()
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = torch.bucketize(r, mid), torch.bucketize(r, mid, right=True)
    code = torch.where(lo % 2 == 0, lo, hi)  # a tie goes to the even code
    v = torch.sign(x) * table[code] * s
    v = torch.where(finite, v, torch.full_like(v, math.nan))
    return v.flatten(-2)[..., :width]


def gemv64(x, w, group):
    """x @ hold(w)^T and sum |x| |w|, in float64."""
    h = hold(w, group)
    return x.double() @ h.t(), x.double().abs() @ h.abs().t()


def gemv_bound(x, w, group, out_dtype):
    """Largest error of the product: the 22 bits of a float32 input, the accumulation of one group in the tensor core,
    the float32 sums of groups, blocks and shares of K, the rounding of the result."""
    ref, mag = gemv64(x, w, group)
    k = x.shape[1]
    blocks = -(-k // 128)
    c = (2.0 ** -22 if x.dtype == torch.float32 else 0.0) + (group // 16) * MMA_STEP + (6 * blocks + 16) * 2.0 ** -24
    # every float32 step and the result's rounding may also lose half a step of the subnormal range
    return ref, c * mag + HALF_STEP[out_dtype] * ref.abs() + (6 * blocks + 16) * 2.0 ** -150 + HALF_TINY[out_dtype]


def visible(length, n_rows, rows, mask):
    """[rows, length] of one sequence: what the rows see (rows past n_rows see nothing)."""
    see = torch.zeros(rows, max(length, 0), dtype=torch.bool)
    base = length - n_rows
    for i in range(n_rows):
        for p in range(max(length, 0)):
            j = p - base
            see[i, p] = j < 0 or (j <= i if mask is None else bool(int(mask[i]) >> j & 1))
    return see


def attention64(q, k, v, see, scale):
    """One sequence: q [rows, nq, d], held k, v [length, nkv, d] float64, see [rows, length].  Output, log-sum-exp and a
    bound of the error that does not count the output's own rounding."""
    rows, nq, d = q.shape
    nkv = k.shape[1]
    o = torch.zeros(rows, nq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((rows, nq), -math.inf, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    lse_bound = torch.zeros_like(lse)
    if k.shape[0] == 0:
        return o, lse, bound, lse_bound
    # scores: float32 q in 22 bits, groups of 32 in the tensor core (two steps, twice for two terms), their float32 sums
    cs = (2.0 ** -22 if q.dtype == torch.float32 else 0.0) + 4 * MMA_STEP + (d // 32 + 3) * 2.0 ** -24
    # weights: fp16 (one rounding, or two terms) and the exponential; sums: one step per 16 tokens, joins in float32
    cp = (2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -21) + 2.0 ** -21
    steps = -(-k.shape[0] // 16)
    cp += (steps * MMA_STEP if q.dtype != torch.float32 else 8 * MMA_STEP + steps * 2.0 ** -24) + 2.0 ** -19
    for e in range(nq):
        h = e // (nq // nkv)
        qe = q[:, e].double()
        s = (qe @ k[:, h].t() * scale).masked_fill(~see, -math.inf)
        off = (cs * abs(scale) * (qe.abs() @ k[:, h].abs().t())).masked_fill(~see, 0.0).amax(-1, keepdim=True)
        off = off + 2.0 ** -22 * s.masked_fill(~see, 0.0).abs().amax(-1, keepdim=True)  # float32 exponents
        some = see.any(-1)
        p = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], s, torch.zeros_like(s)), -1), torch.zeros_like(s))
        p = torch.where(see, p, torch.zeros_like(p))
        held_v = torch.where(see.any(0)[:, None], v[:, h], torch.zeros_like(v[:, h]))
        o[:, e] = p @ held_v
        # A weight times its scale s is held in fp16 with the largest scale S brought to [2^6, 2^7) at weight 1, so below
        # the normal range it is off by at most 2^-25 / 2^6 of S; times a code of at most 6, and 6 S <= 1.01 max |v|.  The
        # sum of the weights that divides it is at least 1.
        floor = 2.0 ** -31 * 1.01 * held_v.abs().amax() * see.sum(-1, keepdim=True)
        bound[:, e] = (2 * off + cp) * (p @ held_v.abs()) + floor + HALF_TINY[q.dtype]  # (its rounding in the subnormal range)
        lse[:, e] = torch.where(some, torch.logsumexp(torch.where(some[:, None], s, torch.zeros_like(s)), -1), lse[:, e])
        lse_bound[:, e] = off[:, 0] + 2.0 ** -20 + 2.0 ** -22 * torch.where(some, lse[:, e].abs(), torch.zeros_like(lse[:, e]))
    return o, lse, bound, lse_bound
