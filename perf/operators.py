"""The 4-bit operators of the library, as they are measured: products with
4-bit weights, a KV cache quantised as it is written (and read back), and
attention over that cache.

The 4-bit format is the same everywhere.  A value is s * c: c one of the
sixteen E2M1 numbers 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, s the
bfloat16 scale of a group of consecutive elements (32, 64 or 128 along the
rows of a weight matrix; 32 channels of one token and head in the cache).
s = bf16(max |x| / 6); c is the E2M1 number nearest to x / s, ties to the even
code, saturating at 6.

The plain form keeps c as twice its value in int8 and the scales beside it.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZES = {"fp32": 4, "bf16": 2, "fp16": 2}
KV_GROUP = 32


def listed():
    return [
        # the fused query, key and value rows of the 0.6B-class decoder, one pass row: an autoregressive step of one stream
        dict(name="w4_qkv_row", op="gemv", rows=1, n=4096, k=1024, group=32, dtype="fp32", out="fp32"),
        # four lm_heads of that decoder on the four rows of a verify window
        dict(name="w4_heads_window", op="gemv", rows=4, n=8192, k=1024, group=32, dtype="fp32", out="fp32"),
        # the down projection of the large decoder for eight single-row streams
        dict(name="w4_down_streams", op="gemv", rows=8, n=2048, k=6144, group=64, dtype="bf16", out="bf16"),
        # gate and up of the large decoder for sixteen streams with a window of four
        dict(name="w4_gate_up_batch", op="gemv", rows=64, n=12288, k=2048, group=128, dtype="bf16", out="bf16"),
        # a ragged matrix: no size a multiple of a tile
        dict(name="w4_ragged", op="gemv", rows=5, n=1999, k=1001, group=32, dtype="fp16", out="fp16"),
        # a large-vocabulary head of an outer model, one row, logits in 32 bits
        dict(name="w4_vocabulary_row", op="gemv", rows=1, n=65536, k=4096, group=128, dtype="bf16", out="fp32"),
        # the verify windows of 64 streams written into their frame caches, the frames read back
        dict(name="kv4_frames", op="cache", seqs=64, rows=4, length=16, kv_heads=8, dim=128, page=16, dtype="fp32"),
        # prompts of an outer model written in pieces of 512, each sequence read back whole
        dict(name="kv4_prompts", op="cache", seqs=4, rows=512, length=8192, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # one frame's verify windows of 64 streams against their frame caches
        dict(name="attn_frames", op="attention", seqs=64, rows=4, length=16, heads=16, kv_heads=8, dim=128, page=16,
             dtype="fp32", ragged=True, tree=False),
        # one token of one stream against a long context
        dict(name="attn_long_row", op="attention", seqs=1, rows=1, length=32768, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", ragged=False, tree=False),
        # verify windows of 32 streams of unequal lengths
        dict(name="attn_windows", op="attention", seqs=32, rows=4, length=8192, heads=16, kv_heads=8, dim=128, page=32,
             dtype="bf16", ragged=True, tree=False),
        # sparse-tree rounds: 24 nodes a stream, each seeing the prefix and its ancestors
        dict(name="attn_trees", op="attention", seqs=8, rows=24, length=2047, heads=32, kv_heads=8, dim=64, page=16,
             dtype="fp16", ragged=True, tree=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "cache", "attention", "attention"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    if op == "gemv":
        n, k = _log(rng, 200, 65536), _log(rng, 200, 8192)
        n = min(n, (65536 * 4096) // k)
        rows = min(_log(rng, 1, 64), max(1, (64 * 12288 * 2048) // (n * k)))
        return dict(op=op, rows=rows, n=n, k=k, group=rng.choice([32, 64, 128]), dtype=dtype,
                    out=rng.choice([dtype, "fp32"]))
    kv_heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    if op == "cache":
        seqs, length = _log(rng, 1, 64), _log(rng, 1, 8192)
        length = min(length, max(1, (4 * 8192 * 8 * 128) // (seqs * kv_heads * dim)))
        return dict(op=op, seqs=seqs, rows=min(length, _log(rng, 1, 512)), length=length, kv_heads=kv_heads, dim=dim,
                    page=page, dtype=dtype)
    seqs, length = _log(rng, 1, 64), _log(rng, 16, 32768)
    length = min(length, max(16, (32 * 8192 * 8 * 128) // (seqs * kv_heads * dim)))
    tree = rng.random() < 0.25
    rows = rng.randint(1, min(length, 63 if tree else 8))
    group = rng.choice([1, 2, 4, 8])
    # the scores of the plain form stay below those of the largest listed case
    while seqs * rows * kv_heads * group * length > 32 * 4 * 16 * 8192 and rows > 1:
        rows = (rows + 1) // 2
    return dict(op=op, seqs=seqs, rows=rows, length=length, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                dtype=dtype, ragged=rng.random() < 0.7, tree=tree)


def _lengths(case):
    """Tokens of each sequence, the window's rows among them."""
    length, rows = case["length"], case["rows"]
    if not case.get("ragged"):
        return [length] * case["seqs"]
    return [max(rows, length - (97 * b) % (length // 2 + 1)) for b in range(case["seqs"])]


def work(case):
    if case["op"] == "gemv":
        r, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": n * k // 2 + 2 * n * -(-k // case["group"]) + r * k * SIZES[case["dtype"]] + r * n * SIZES[case["out"]],
                "flops": 2 * r * n * k}
    width = case["kv_heads"] * case["dim"]
    held = 2 * (width // 2 + 2 * width // KV_GROUP)  # bytes of one token's keys and values in the cache
    es = SIZES[case["dtype"]]
    if case["op"] == "cache":
        new, all_ = case["seqs"] * case["rows"], case["seqs"] * case["length"]
        return {"bytes": 2 * new * width * es + new * held + all_ * held + 2 * all_ * width * es,
                "flops": 4 * new * width + 2 * all_ * width}
    lens = _lengths(case)
    out = case["seqs"] * case["rows"] * case["heads"]
    return {"bytes": sum(lens) * held + 2 * out * case["dim"] * es + 4 * out,
            "flops": 4 * sum(lens) * case["rows"] * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _gemv_inputs(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    w = (0.02 * torch.randn(case["n"], case["k"], generator=g, device="cuda")).to(torch.bfloat16)
    # activations as a norm leaves them: unit variance, a few large channels
    x = torch.randn(case["rows"], case["k"], generator=g, device="cuda")
    x[:, :: 61] *= 8.0
    return w, x.to(dt)


def _cache_rows(g, count, case):
    """Keys whose channels differ in size (as after a rotary embedding) and values of unit variance."""
    shape = (count, case["kv_heads"], case["dim"])
    size = torch.exp(0.5 * torch.randn(case["kv_heads"], case["dim"], generator=g, device="cuda"))
    k = (torch.randn(shape, generator=g, device="cuda") * size).to(DTYPES[case["dtype"]])
    v = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return k, v


def _page_table(case, g):
    """A shuffled page table: the pages of a sequence are anywhere."""
    per = -(-case["length"] // case["page"])
    return torch.randperm(case["seqs"] * per, generator=g, device="cuda").to(torch.int32).view(case["seqs"], per)


def _kv_inputs(case, seed):
    """Every sequence's keys and values [seqs, length, kv_heads, dim], the page table, and for attention the queries and masks."""
    g = _gen(seed)
    b, t = case["seqs"], case["length"]
    pages = _page_table(case, g)
    k, v = _cache_rows(g, b * t, case)
    k, v = k.view(b, t, case["kv_heads"], case["dim"]), v.view(b, t, case["kv_heads"], case["dim"])
    if case["op"] == "cache":
        return pages, k, v, None, None
    q = torch.randn(b, case["rows"], case["heads"], case["dim"], generator=g, device="cuda").to(DTYPES[case["dtype"]])
    mask = None
    if case["tree"]:
        rng = random.Random(seed)
        seen = []
        for _ in range(b):
            of = []
            for i in range(case["rows"]):
                parent = rng.randint(-1, i - 1)
                of.append((1 << i) | (of[parent] if parent >= 0 else 0))
            seen.append(of)
        mask = torch.tensor(seen, dtype=torch.int64, device="cuda")
    return pages, k, v, q, mask


# ------------------------------------------------------------- plain form
def _quantise(x, group):
    """Twice the E2M1 values in int8, and the bfloat16 scales, of groups along the last axis (padded with zeros)."""
    pad = -x.shape[-1] % group
    x = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, group))
    s = (x.abs().amax(-1, keepdim=True) / 6.0).to(torch.bfloat16)
    r = torch.where(s == 0, torch.zeros_like(x), x / s.float())
    a = r.abs()
    twice = ((a > 0.25).to(torch.int8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + 2 * (a > 2.5) + 2 * (a >= 3.5)
             + 4 * (a > 5.0))
    return torch.where(r < 0, -twice, twice).flatten(-2).to(torch.int8), s.squeeze(-1)


def _values(twice, s, group):
    return ((twice.float() * 0.5).unflatten(-1, (-1, group)) * s.float().unsqueeze(-1)).flatten(-2)


def _empty_pages(case):
    per = case["seqs"] * -(-case["length"] // case["page"])
    shape = (per, case["page"], case["kv_heads"])
    codes = [torch.zeros(*shape, case["dim"], dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(*shape, case["dim"] // KV_GROUP, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return codes, scales


def _write(state, k, v, first):
    """Rows k, v [seqs, rows, kv_heads, dim] into the pages, from position first on."""
    case, pages = state["case"], state["pages"]
    pos = torch.arange(first, first + k.shape[1], device="cuda")
    page, slot = pages.long()[:, pos // case["page"]], (pos % case["page"]).expand(k.shape[0], -1)
    for x, codes, scales in zip((k, v), state["codes"], state["scales"]):
        c, s = _quantise(x, KV_GROUP)
        codes[page, slot] = c
        scales[page, slot] = s


def _gather(state, which, length):
    """Keys (0) or values (1) of positions 0 .. length - 1 in 32 bits: [seqs, length, kv_heads, dim]."""
    pages = state["pages"].long()
    c = state["codes"][which][pages].flatten(1, 2)[:, :length]
    s = state["scales"][which][pages].flatten(1, 2)[:, :length]
    return _values(c, s, KV_GROUP)


def _visible(case, lens, mask):
    """[seqs, rows, length]: whether a window row sees a position (the prefix; then the window by causal order or by the mask's bits)."""
    pos = torch.arange(case["length"], device="cuda").view(1, 1, -1)
    row = torch.arange(case["rows"], device="cuda").view(1, -1, 1)
    base = (lens - case["rows"]).view(-1, 1, 1)
    if mask is None:
        return pos <= base + row
    bit = (pos - base).clamp(0, 63)
    return (pos < base) | ((pos < base + case["rows"]) & (((mask.unsqueeze(-1) >> bit) & 1) == 1))


# ---------------------------------------------------------- prepare and run
def prepare(case, seed):
    if case["op"] == "gemv":
        w, x = _gemv_inputs(case, seed)
        state = dict(case=case, x=x, out=DTYPES[case["out"]])
        if own:
            from speculative_decoding_rvq_gb300 import binding
            state["w"] = binding.w4_pack(w, group=case["group"])
        else:
            state["twice"], state["scales"] = _quantise(w, case["group"])
        return state
    pages, k, v, q, mask = _kv_inputs(case, seed)
    b, t, rows = case["seqs"], case["length"], case["rows"]
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    state = dict(case=case, pages=pages, lens=lens, q=q, mask=mask)
    if own:
        from speculative_decoding_rvq_gb300 import binding
        state["cache"] = binding.Kv4Cache(pages.numel(), case["page"], case["kv_heads"], case["dim"])
        state["cache"].append(k, v, torch.zeros(b, dtype=torch.int32, device="cuda"), pages=pages)
    else:
        state["codes"], state["scales"] = _empty_pages(case)
        _write(state, k, v, 0)
    if case["op"] == "cache":  # the last rows of every sequence are written again, with new values
        g = _gen(seed + 1)
        k, v = _cache_rows(g, b * rows, case)
        state["k"], state["v"] = k.view(b, rows, *k.shape[1:]), v.view(b, rows, *v.shape[1:])
        state["first"] = torch.full((b,), t - rows, dtype=torch.int32, device="cuda")
    return state


def _run_own(state):
    case = state["case"]
    if case["op"] == "gemv":
        from speculative_decoding_rvq_gb300 import binding
        return binding.w4_gemv(state["x"], state["w"], out_dtype=state["out"])
    if case["op"] == "cache":
        state["cache"].append(state["k"], state["v"], state["first"], pages=state["pages"])
        return state["cache"].read(case["length"], pages=state["pages"], dtype=DTYPES[case["dtype"]])
    return state["cache"].attention(state["q"], state["lens"], pages=state["pages"], mask=state["mask"], want_lse=True)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "gemv":
        w = _values(state["twice"], state["scales"], case["group"])[:, : case["k"]]
        return (state["x"].float() @ w.t()).to(state["out"])
    dt = DTYPES[case["dtype"]]
    if case["op"] == "cache":
        _write(state, state["k"], state["v"], case["length"] - case["rows"])
        return _gather(state, 0, case["length"]).to(dt), _gather(state, 1, case["length"]).to(dt)
    k, v = _gather(state, 0, case["length"]), _gather(state, 1, case["length"])
    b, m, nq, d = state["q"].shape
    nkv = case["kv_heads"]
    q = state["q"].float().view(b, m, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4).reshape(b, nkv, -1, d)
    s = (q @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    s = s.view(b, nkv, nq // nkv, m, -1)
    s = torch.where(_visible(case, state["lens"], state["mask"]).view(b, 1, 1, m, -1), s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    # the sum over positions in pieces of 256, so that a long one keeps its 32 bits
    pad = -s.shape[-1] % 256
    p = torch.nn.functional.pad((e / total).view(b, nkv, -1, s.shape[-1]), (0, pad)).unflatten(-1, (-1, 256))
    v = torch.nn.functional.pad(v, (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, 256))
    o = (p.transpose(2, 3) @ v.permute(0, 3, 1, 2, 4)).sum(2)
    o = o.view(b, nkv, nq // nkv, m, d).permute(0, 3, 1, 2, 4).reshape(b, m, nq, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(b, m, nq)
    return o.to(dt), lse


# ------------------------------------------------------------------- exact
def _held(x, group):
    """What the 4-bit format holds for x, in 64 bits: the table's nearest number to each quotient, the even code on a tie."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    width = x.shape[-1]
    x = x.double()
    x = torch.cat([x, x.new_zeros(*x.shape[:-1], -width % group)], -1)
    x = x.view(*x.shape[:-1], x.shape[-1] // group, group)
    s = (x.abs().max(-1, keepdim=True).values / 6.0).float().bfloat16().double()
    r = x / torch.where(s > 0, s, 1.0)
    mid = (table[1:] + table[:-1]) / 2
    below, upto = torch.bucketize(r.abs(), mid), torch.bucketize(r.abs(), mid, right=True)
    code = torch.where(below % 2 == 0, below, upto)
    return (torch.sign(r) * table[code] * s).reshape(*x.shape[:-2], -1)[..., :width]


def exact(case, seed):
    if case["op"] == "gemv":
        w, x = _gemv_inputs(case, seed)
        out = [x.double() @ _held(part, case["group"]).t() for part in w.split(4096)]
        return torch.cat(out, 1)
    pages, k, v, q, mask = _kv_inputs(case, seed)
    if case["op"] == "cache":
        nk, nv = _cache_rows(_gen(seed + 1), case["seqs"] * case["rows"], case)
        first = case["length"] - case["rows"]
        k[:, first:] = nk.view_as(k[:, first:])
        v[:, first:] = nv.view_as(v[:, first:])
        return _held(k, KV_GROUP), _held(v, KV_GROUP)
    b, m, nq, d = q.shape
    per = nq // case["kv_heads"]
    out = torch.empty(b, m, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(b, m, nq, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        base = n - m
        see = torch.ones(m, n, dtype=torch.bool, device="cuda")
        for r in range(m):
            if mask is None:
                see[r, base + r + 1:] = False
            else:
                bits = int(mask[i, r])
                see[r, base:] = torch.tensor([bool(bits >> j & 1) for j in range(m)], device="cuda")
        for h in range(case["kv_heads"]):
            kh, vh = _held(k[i, :n, h], KV_GROUP), _held(v[i, :n, h], KV_GROUP)
            for e in range(h * per, (h + 1) * per):
                s = q[i, :, e].double() @ kh.t() / math.sqrt(d)
                s = s.masked_fill(~see, -math.inf)
                lse[i, :, e] = torch.logsumexp(s, -1)
                out[i, :, e] = torch.softmax(s, -1) @ vh
    return out, lse
