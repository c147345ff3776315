"""The operators of a 16-bit paged KV cache, as they are measured: page tables
and slot maps made from request lengths, rotary embedding over several position
axes (alone, and as the rows of a step are written into the cache), and
attention over the cache: with a sliding window whose first tokens (sinks) stay
visible, and of trees of drafted tokens.

Rows of all sequences are packed one sequence after the other; sequence b has
the rows row_start[b] .. row_start[b + 1] - 1, its last positions.  The cache
holds pages [n_pages, kv_heads, page, dim] of keys and of values.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZES = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # 64 streams take the pages of a verify window of four, and give them back when it is rejected
        dict(name="plan_windows", op="plan", seqs=64, length=2000, new=4, page=16, spare=1.0),
        # a full server: prompts of unequal lengths admitted until the pool's pages run out, then released
        dict(name="plan_prompts", op="plan", seqs=512, length=900, new=1023, page=64, spare=0.8),
        # the verify windows of 64 streams rotated and written, one position axis
        dict(name="append_windows", op="append", rows=256, heads=16, kv_heads=8, dim=128, rot=128, axes=1, interleaved=False,
             page=16, dtype="bf16"),
        # a prompt with images and video, written in one piece: time, height and width
        dict(name="append_prompt", op="append", rows=16384, heads=16, kv_heads=8, dim=128, rot=128, axes=3, interleaved=True,
             page=64, dtype="bf16"),
        # the patches of a vision encoder: queries and keys, height and width, an odd count
        dict(name="rope_patches", op="rope", rows=9001, heads=16, kv_heads=16, dim=64, rot=64, axes=2, interleaved=False,
             dtype="fp32"),
        # one token of one stream behind a long context
        dict(name="window_row", op="window", seqs=1, rows=1, length=32768, window=4096, sinks=4, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bf16", ragged=False),
        # verify windows of 32 streams of unequal lengths
        dict(name="window_streams", op="window", seqs=32, rows=4, length=8191, window=2048, sinks=4, heads=16, kv_heads=8,
             dim=128, page=32, dtype="bf16", ragged=True),
        # short prompts of unequal lengths in one batch, ragged rows
        dict(name="window_prompts", op="window", seqs=13, rows=777, length=1555, window=500, sinks=16, heads=8, kv_heads=8,
             dim=64, page=16, dtype="fp16", ragged=True),
        # the second half of a long prompt
        dict(name="window_long_prompt", op="window", seqs=1, rows=8192, length=16384, window=4096, sinks=4, heads=32,
             kv_heads=8, dim=128, page=64, dtype="bf16", ragged=False),
        # one stream's tree of 62 nodes behind a long context
        dict(name="tree_long", op="tree", seqs=1, rows=62, length=32768, window=0, sinks=0, heads=16, kv_heads=8, dim=128,
             page=64, dtype="bf16", ragged=False),
        # trees of 24 nodes of eight streams
        dict(name="tree_streams", op="tree", seqs=8, rows=24, length=2047, window=0, sinks=0, heads=32, kv_heads=8, dim=64,
             page=16, dtype="fp16", ragged=True),
        # small trees of a full batch
        dict(name="tree_batch", op="tree", seqs=64, rows=7, length=4000, window=0, sinks=0, heads=16, kv_heads=8, dim=128,
             page=32, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "rope", "window", "window", "tree", "tree"])
    if op == "plan":
        seqs, new = _log(rng, 1, 512), _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, length=_log(rng, 1, 8192), new=min(new, (512 * 1023) // seqs),
                    page=rng.choice([16, 32, 64, 128]), spare=rng.choice([0.5, 0.8, 1.0, 1.0]))
    if op in ("append", "rope"):
        kv_heads, dim, group = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 4])
        case = dict(op=op, rows=min(_log(rng, 1, 16384), (16384 * 32 * 128) // (kv_heads * (group + 2) * dim)),
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5)
        if op == "append":
            return dict(case, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]))
        return dict(case, dtype=rng.choice(["fp32", "bf16", "fp16"]))
    kv_heads, dim, group = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
    seqs, length = _log(rng, 1, 64), _log(rng, 16, 32768)
    length = min(length, max(16, (64 * 4000 * 8 * 128) // (seqs * kv_heads * dim)))
    many = op == "window" and rng.random() < 0.5
    rows = _log(rng, 1, min(length, 8192)) if many else rng.randint(1, min(length, 62 if op == "tree" else 8))
    # the scores of the plain form stay well below those of the largest listed case
    while seqs * rows * kv_heads * group * length * dim > 16384 * 16384 * 16 * 128 and rows > 1:
        rows = (rows + 1) // 2
    window = rng.choice([0, _log(rng, 1, 8192), _log(rng, 64, 4096)]) if op == "window" or rng.random() < 0.3 else 0
    return dict(op=op, seqs=seqs, rows=rows, length=length, window=window, sinks=rng.choice([0, 1, 4, 64]) if window else 0,
                heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.7)


# ------------------------------------------------------------------- sizes
def _lengths(case):
    """Tokens of each sequence and, of these, the rows of the call."""
    length, rows = case["length"], case["rows"]
    if not case["ragged"]:
        return [(length, rows)] * case["seqs"]
    out = []
    for b in range(case["seqs"]):
        m = max(1, rows - (31 * b) % (rows // 2 + 1))
        out.append((max(m, length - (97 * b) % (length // 2 + 1)), m))
    return out


def _plan_lengths(case, seed):
    """Kept and new tokens: the same requests whatever the seed, in another order."""
    rng = random.Random(case["seqs"])
    both = [(rng.randint(0, case["length"]), rng.randint(1, case["new"])) for _ in range(case["seqs"])]
    random.Random(seed).shuffle(both)
    return [a for a, _ in both], [n for _, n in both]


def _sections(case):
    """Pairs of each axis: time the rest, height and width each 20 of 64 (two axes: half each)."""
    pairs, axes = case["rot"] // 2, case["axes"]
    each = {1: 0, 2: pairs // 2, 3: pairs * 20 // 64}[axes]
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


def _span(base, m, window, sinks):
    """Positions that rows at base .. base + m - 1 see, summed over the rows, and their union."""
    if window == 0:
        return m * base + m * (m + 1) // 2, base + m
    total = 0
    for p in range(base, base + m):
        total += p + 1 if p + 1 <= window else window + min(sinks, p + 1 - window)
    first = max(0, base - window + 1)
    return total, base + m - first + min(sinks, first)


def work(case):
    op = case["op"]
    if op == "plan":
        kept, new = _plan_lengths(case, 0)
        page, pages = case["page"], 0
        for a, n in zip(kept, new):
            pages += -(-(a + n) // page) - -(-a // page)
        # taken and given back: the table's and the stack's entries each way; lengths in and out, twice; a row's slot and position
        return {"bytes": 4 * pages * 4 + 2 * len(kept) * 4 * 5 + sum(new) * 12, "flops": 0}
    if op in ("append", "rope"):
        turned = (case["heads"] + case["kv_heads"]) * case["dim"]
        width = turned + (case["kv_heads"] * case["dim"] if op == "append" else 0)
        return {"bytes": case["rows"] * (2 * width * SIZES[case["dtype"]] + 4 * case["axes"] + (8 if op == "append" else 0)),
                "flops": case["rows"] * 3 * (case["heads"] + case["kv_heads"]) * case["rot"]}
    seen = held = rows = 0
    for n, m in _lengths(case):
        pairs, union = _span(n - m, m, case["window"], case["sinks"])
        seen, held, rows = seen + (pairs if op == "window" else m * union), held + union, rows + m
    es = SIZES[case["dtype"]]
    return {"bytes": held * 2 * case["kv_heads"] * case["dim"] * es + rows * case["heads"] * (2 * case["dim"] * es + 4),
            "flops": 4 * seen * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _plan_inputs(case, seed):
    """Kept and new tokens, the page table as the kept tokens left it, its pages anywhere in the pool, and the free ones."""
    kept, new = _plan_lengths(case, seed)
    page = case["page"]
    held = [-(-a // page) for a in kept]
    most = -(-(case["length"] + case["new"]) // page)
    lack = sum(-(-(a + n) // page) for a, n in zip(kept, new)) - sum(held)
    n_pages = sum(held) + max(1, int(case["spare"] * lack))
    order = torch.randperm(n_pages, generator=_gen(seed), device="cuda").to(torch.int32)
    held_t = _ints(held)
    j = torch.arange(most, device="cuda")
    first = torch.cumsum(held_t, 0) - held_t
    at = (first.unsqueeze(1) + j).clamp(max=n_pages - 1)
    table = torch.where(j < held_t.unsqueeze(1), order[at], -1).to(torch.int32)
    free = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    free[: n_pages - sum(held)] = order[sum(held):]
    return _ints(kept), _ints(new), table, held_t, free, _ints([n_pages - sum(held)])


def _positions(case, seed):
    """[axes, rows]: text, then pictures of 24 x 36 patches one after the other (time, height, width), behind a long context."""
    rows, axes = case["rows"], case["axes"]
    r = torch.arange(rows, device="cuda")
    start = random.Random(seed).randint(0, 100000)
    text = rows // 3
    patch = (r - text).clamp(min=0)
    frame, inside = patch // 864, patch % 864
    time, height, width = start + text + frame, start + text + inside // 36, start + text + inside % 36
    plain = start + r
    if axes == 1:
        pos = [plain]
    elif axes == 2:
        pos = [inside // 36 + 0 * r, inside % 36 + 0 * r]
    else:
        pos = [torch.where(r < text, plain, x) for x in (time, height, width)]
    return torch.stack(pos).to(torch.int32)


def _rows_inputs(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    q = torch.randn(case["rows"], case["heads"], case["dim"], generator=g, device="cuda").to(dt)
    k = (1.5 * torch.randn(case["rows"], case["kv_heads"], case["dim"], generator=g, device="cuda")).to(dt)
    v = torch.randn(case["rows"], case["kv_heads"], case["dim"], generator=g, device="cuda").to(dt)
    slot = None
    if case["op"] == "append":  # pages anywhere in a pool a quarter larger
        page = case["page"]
        per = -(-case["rows"] // page)
        order = torch.randperm(per + per // 4 + 1, generator=g, device="cuda")
        r = torch.arange(case["rows"], device="cuda")
        slot = order[r // page] * page + r % page
    return q, k, v, slot, _positions(case, seed)


def _tree_masks(case, seed):
    """For each row of each sequence the bits of the rows that it sees: its ancestors and itself."""
    rng = random.Random(seed)
    seen = []
    for _, m in _lengths(case):
        of = []
        for i in range(m):
            parent = rng.randint(-1, i - 1)
            of.append((1 << i) | (of[parent] if parent >= 0 else 0))
        seen += of
    return torch.tensor(seen, dtype=torch.int64, device="cuda")


def _attention_inputs(case, seed):
    """Keys and values of all sequences one after the other, their slots, the table, the queries, lengths, row starts and masks."""
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    lens = _lengths(case)
    page = case["page"]
    per = -(-max(n for n, _ in lens) // page)
    table = torch.randperm(case["seqs"] * per, generator=g, device="cuda").to(torch.int32).view(case["seqs"], per)
    shape = (sum(n for n, _ in lens), case["kv_heads"], case["dim"])
    # keys whose channels differ in size, as after a rotary embedding, and values of unit variance
    size = torch.exp(0.5 * torch.randn(case["kv_heads"], case["dim"], generator=g, device="cuda"))
    k = (torch.randn(shape, generator=g, device="cuda") * size).to(dt)
    v = torch.randn(shape, generator=g, device="cuda").to(dt)
    kv_len = _ints([n for n, _ in lens])
    ends = torch.cumsum(kv_len, 0)
    r = torch.arange(shape[0], device="cuda")
    b = torch.searchsorted(ends, r, right=True)
    pos = r - (ends - kv_len)[b]
    slot = table[b, pos // page].long() * page + pos % page
    starts = [0]
    for _, m in lens:
        starts.append(starts[-1] + m)
    q = torch.randn(starts[-1], case["heads"], case["dim"], generator=g, device="cuda").to(dt)
    mask = _tree_masks(case, seed) if case["op"] == "tree" else None
    return k, v, slot, table, q, kv_len, _ints(starts), mask


# ------------------------------------------------------------- plain form
def _plan_step(state, length, new, n_rows):
    """One step of the pool: pages past the need given back, lacking ones taken, and the rows' positions and slots."""
    pages, free, page = state["pages"], state["free"], state["case"]["page"]
    n_seqs, most = pages.shape
    length, new, held, n_free = length.long(), new.long(), state["held"].long(), state["n_free"].long()
    need = (length + new + page - 1) // page
    fits = need <= most
    j = torch.arange(most, device="cuda")
    goes = fits.unsqueeze(1) & (j >= need.unsqueeze(1)) & (j < held.unsqueeze(1))
    behind = torch.cumsum(goes.flatten(), 0)
    given = behind[-1]
    at = torch.where(goes.flatten(), n_free + given - behind, free.shape[0])
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, at, pages.flatten())[:-1]
    there = n_free + given
    lack = torch.where(fits, (need - held).clamp(min=0), 0)
    paged = (lack == 0) | (torch.cumsum(lack, 0) <= there)
    roomy = (new == 0) | (torch.cumsum(new, 0) <= n_rows)
    served = fits & paged & roomy
    comes = served.unsqueeze(1) & (j >= held.unsqueeze(1)) & (j < need.unsqueeze(1))
    taken = torch.cumsum(comes.flatten(), 0).view_as(comes)
    table = torch.where(comes, free[(there - taken).clamp(0, free.shape[0] - 1)], torch.where(goes, -1, pages))
    held = torch.where(served | (need < held) & fits, need, held)
    rows = torch.where(served, new, 0)
    kv_len = torch.where(served, length + new, torch.minimum(length, held * page))
    row_start = torch.nn.functional.pad(torch.cumsum(rows, 0), (1, 0))
    r = torch.arange(n_rows, device="cuda")
    b = torch.searchsorted(row_start[1:], r, right=True).clamp(max=n_seqs - 1)
    live = r < row_start[-1]
    pos = torch.where(live, length[b] + r - row_start[b], 0)
    slot = torch.where(live, table[b, (pos // page).clamp(max=most - 1)].long() * page + pos % page, -1)
    refused = torch.where(~fits, 2, torch.where(~paged, 1, torch.where(~roomy, 3, 0)))
    state["pages"].copy_(table)
    state["free"].copy_(free)
    state["held"].copy_(held)
    state["n_free"].copy_(there - taken[-1, -1])
    return kv_len.int(), row_start.int(), pos.int(), slot, refused.int()


def _angles(case, pos):
    """[rows, 1, pairs] in 64 bits: the position of a pair's axis times its frequency."""
    pairs, axes, sections = case["rot"] // 2, case["axes"], _sections(case)
    i = torch.arange(pairs, device="cuda")
    if case["interleaved"]:
        axis = i % axes
        count = torch.tensor(sections, device="cuda")[axis]
        axis = torch.where(i < axes * count, axis, 0)
    else:
        axis = torch.searchsorted(torch.tensor(sections, device="cuda").cumsum(0), i, right=True)
    freq = torch.exp(i.double() * (-2.0 / case["rot"] * math.log(1000000.0)))
    return (pos[axis].t().double() * freq).unsqueeze(1)


def _turn(x, angle):
    """The pairs (i, i + rot / 2) of x turned, the channels past rot kept."""
    half = angle.shape[-1]
    c, s = torch.cos(angle).to(torch.float32), torch.sin(angle).to(torch.float32)
    a, b, rest = x[..., :half].float(), x[..., half: 2 * half].float(), x[..., 2 * half:].float()
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1).to(x.dtype)


def _visible(case, base, m, bits, n):
    """[seqs, rows, n]: whether a row sees a position.  base and m: [seqs, 1, 1]; bits [seqs, rows] or None."""
    j = torch.arange(n, device="cuda").view(1, 1, -1)
    i = torch.arange(case["rows"], device="cuda").view(1, -1, 1)
    if bits is None:
        at = base + i
        near = j <= at
    else:
        shift = torch.arange(64, device="cuda")
        at = base + (bits.unsqueeze(-1) >> shift & 1).sum(-1, keepdim=True) - 1
        near = (j < base) | (j < base + m) & (bits.unsqueeze(-1) >> (j - base).clamp(0, 63) & 1 == 1)
    if case["window"]:
        kept = (j > at - case["window"]) | (j < case["sinks"])
        near = near & (kept if bits is None else kept | (j >= base))
    return near


def _attention(state):
    case, pages, q = state["case"], state["pages"].long(), state["q"]
    nkv, d, rows = case["kv_heads"], case["dim"], case["rows"]
    group = case["heads"] // nkv
    k = state["keys"][pages].transpose(1, 2).flatten(2, 3).float()
    v = state["values"][pages].transpose(1, 2).flatten(2, 3).float()
    seqs, n = pages.shape[0], k.shape[2]
    start = state["row_start"].long()
    m = start[1:] - start[:-1]
    at = (start[:-1].unsqueeze(1) + torch.arange(rows, device="cuda")).clamp(max=q.shape[0] - 1)
    qs = q.float()[at].view(seqs, rows, nkv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, nkv, -1, d)
    bits = None if state["mask"] is None else state["mask"][at]
    see = _visible(case, (state["kv_len"].long() - m).view(-1, 1, 1), m.view(-1, 1, 1), bits, n)
    s = (qs @ k.transpose(2, 3)).view(seqs, nkv, group, rows, n) * (1.0 / math.sqrt(d))
    s = torch.where(see.view(seqs, 1, 1, rows, n), s, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp(min=torch.finfo(torch.float32).tiny)
    o = (p.view(seqs, nkv, -1, n) @ v).view(seqs, nkv, group, rows, d).permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).flatten(2)
    r = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(start[1:], r, right=True)
    i = r - start[b]
    return o[b, i].to(q.dtype), lse[b, i]


# ---------------------------------------------------------- prepare and run
def prepare(case, seed):
    if case["op"] == "plan":
        length, new, pages, held, free, n_free = _plan_inputs(case, seed)
        state = dict(case=case, length=length, new=new, zero=torch.zeros_like(new), n_rows=case["seqs"] * case["new"])
        if own:
            from speculative_decoding_rvq_gb300 import binding
            pool = binding.PagePool(free.numel(), case["page"], case["seqs"], pages.shape[1])
            for mine, given in ((pool.pages, pages), (pool.held, held), (pool.free, free), (pool.n_free, n_free)):
                mine.copy_(given)
            return dict(state, pool=pool)
        return dict(state, pages=pages, held=held, free=free, n_free=n_free)
    if case["op"] in ("append", "rope"):
        q, k, v, slot, pos = _rows_inputs(case, seed)
        state = dict(case=case, q=q, k=k, v=v, slot=slot, pos=pos)
        if own:
            from speculative_decoding_rvq_gb300 import binding
            state["rope"] = binding.Rope(case["rot"], 1000000.0, sections=_sections(case), interleaved=case["interleaved"])
        if case["op"] == "rope":
            return state
        per = -(-case["rows"] // case["page"])
        n_pages = per + per // 4 + 1
        if own:
            state["cache"] = binding.Kv16Cache(n_pages, case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]])
        else:
            state["keys"], state["values"] = _empty_pages(case, n_pages)
        return state
    k, v, slot, pages, q, kv_len, row_start, mask = _attention_inputs(case, seed)
    state = dict(case=case, pages=pages, q=q, kv_len=kv_len, row_start=row_start, mask=mask)
    if own:
        from speculative_decoding_rvq_gb300 import binding
        state["cache"] = binding.Kv16Cache(pages.numel(), case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]])
        state["cache"].append(k, v, slot)
    else:
        state["keys"], state["values"] = _empty_pages(case, pages.numel())
        _write(state, k, v, slot)
    return state


def _empty_pages(case, n_pages):
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    return [torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda") for _ in range(2)]


def _write(state, k, v, slot):
    page = state["case"]["page"]
    state["keys"][slot // page, :, slot % page] = k
    state["values"][slot // page, :, slot % page] = v


def _run_own(state):
    case = state["case"]
    if case["op"] == "plan":
        pool = state["pool"]
        rows = pool.plan(state["length"], state["new"], state["n_rows"])
        back = pool.plan(state["length"])
        return (rows.kv_len, rows.row_start, rows.pos, rows.slot, rows.refused, back.kv_len, pool.pages, pool.held, pool.free,
                pool.n_free)
    if case["op"] == "rope":
        return state["rope"].rotate(state["q"], state["k"], state["pos"])
    if case["op"] == "append":
        q = state["cache"].append(state["k"], state["v"], state["slot"], rope=state["rope"], pos=state["pos"], q=state["q"])
        return q, state["cache"].keys, state["cache"].values
    return state["cache"].attention(state["q"], state["kv_len"], state["row_start"], pages=state["pages"], max_rows=case["rows"],
                                    window=case["window"], sinks=case["sinks"], mask=state["mask"], want_lse=True)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "plan":
        rows = _plan_step(state, state["length"], state["new"], state["n_rows"])
        back = _plan_step(state, state["length"], state["zero"], 0)
        return (*rows, back[0], state["pages"], state["held"], state["free"], state["n_free"])
    if case["op"] in ("append", "rope"):
        angle = _angles(case, state["pos"])
        q, k = _turn(state["q"], angle), _turn(state["k"], angle)
        if case["op"] == "rope":
            return q, k
        _write(state, k, state["v"], state["slot"])
        return q, state["keys"], state["values"]
    return _attention(state)


# ------------------------------------------------------------------- exact
def _exact_plan(case, seed):
    """The pool step by step, one page at a time, on the host."""
    length, new, pages, held, free, n_free = [x.tolist() for x in _plan_inputs(case, seed)]
    page, n_rows, most = case["page"], case["seqs"] * case["new"], len(pages[0])
    table, stack = [row[:] for row in pages], free[: n_free[0]]
    lacks = [max(0, -(-(a + n) // page) - h) for a, n, h in zip(length, new, held)]
    kv_len, row_start, pos, slot, refused, back = [], [0], [], [], [], []
    there, asked = len(stack), 0
    for b, (a, n) in enumerate(zip(length, new)):
        asked += lacks[b]
        if lacks[b] and asked > there:
            kv_len.append(min(a, held[b] * page))
            refused.append(1)
        else:
            for j in range(held[b], held[b] + lacks[b]):
                table[b][j] = stack.pop()
            pos += range(a, a + n)
            slot += [table[b][p // page] * page + p % page for p in range(a, a + n)]
            kv_len.append(a + n)
            refused.append(0)
        row_start.append(len(pos))
        back.append(a)
    assert most and len(pos) <= n_rows
    pos += [0] * (n_rows - len(pos))
    slot += [-1] * (n_rows - len(slot))
    whole = [_ints(kv_len), _ints(row_start), _ints(pos), torch.tensor(slot, device="cuda"), _ints(refused), _ints(back)]
    return (*whole, _ints(pages), _ints(held), _ints(free), _ints(n_free))  # all that was taken is given back


def _exact_turn(case, x, pos):
    x, rot, axes = x.double(), case["rot"], case["axes"]
    out = x.clone()
    left = _sections(case)
    owner = []
    for a, count in enumerate(left):
        owner += [a] * count
    if case["interleaved"]:
        owner = [0] * (rot // 2)
        for a in range(1, axes):
            for t in range(left[a]):
                owner[a + axes * t] = a
    for i in range(rot // 2):
        w = pos[owner[i]].double() * 1000000.0 ** (-2.0 * i / rot)
        z = torch.complex(x[..., i], x[..., i + rot // 2]) * torch.polar(torch.ones_like(w), w).unsqueeze(-1)
        out[..., i], out[..., i + rot // 2] = z.real, z.imag
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return _exact_plan(case, seed)
    if case["op"] in ("append", "rope"):
        q, k, v, slot, pos = _rows_inputs(case, seed)
        q, k = _exact_turn(case, q, pos), _exact_turn(case, k, pos)
        if case["op"] == "rope":
            return q, k
        page = case["page"]
        per = -(-case["rows"] // page)
        held = []
        for x in (k, v.double()):
            flat = torch.zeros((per + per // 4 + 1) * page, *x.shape[1:], dtype=torch.float64, device="cuda")
            flat[slot] = x
            held.append(flat.view(-1, page, *x.shape[1:]).transpose(1, 2).contiguous())
        return q, held[0], held[1]
    k, v, _, _, q, _, _, mask = _attention_inputs(case, seed)
    per = case["heads"] // case["kv_heads"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    window, sinks = case["window"], case["sinks"]
    at = first = 0
    for n, m in _lengths(case):
        base = n - m
        see = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if mask is None:
            p = torch.arange(base, n, device="cuda").unsqueeze(1)
            j = torch.arange(n, device="cuda").unsqueeze(0)
            see = j <= p
            if window:
                see &= ~((j <= p - window) & (j >= sinks))
        else:
            for i, bits in enumerate(mask[at: at + m].tolist()):
                deep = bin(bits).count("1")
                see[i, :base] = True
                if window:
                    see[i, min(sinks, base): max(0, min(base, base + deep - window))] = False
                    see[i, : min(sinks, base)] = True
                see[i, base:] = torch.tensor([bool(bits >> t & 1) for t in range(m)], device="cuda")
        for e in range(case["heads"]):
            kh, vh = k[first: first + n, e // per].double(), v[first: first + n, e // per].double()
            s = q[at: at + m, e].double() @ kh.t() / math.sqrt(case["dim"])
            s = s.masked_fill(~see, -math.inf)
            lse[at: at + m, e] = torch.logsumexp(s, -1)
            out[at: at + m, e] = torch.softmax(s, -1) @ vh
        at, first = at + m, first + n
    return out, lse
