"""Contexts over packed 4-bit weights (cp_spec_init_w4) against the CPU oracle on the values the packed matrices stand
for, and with a 4-bit KV cache against a float64 forward pass that holds keys and values in the format.

Tolerances as for the float contexts: logits within 1e-4 of the float64 oracle (rows are float32, counted with 22 bits),
codes identical except where an oracle decision has a margin below 1e-4."""
import dataclasses
import math

import numpy as np
import pytest

from fp4_reference import SIXTH, hold
from gpu_common import compare_codes_with_margins, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _bf16_spec():
    from speculative_decoding_rvq_gb300 import synth as S
    return S.ModelSpec(512, 2, 8, 4, 64, 1040, 528, 9, S.DTYPE_BF16)


_cache = {}


def _model(orc, spec, group, offsets=0):
    """Oracle over the held values, packed device weights, held values."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    key = (spec, group, offsets)
    if key not in _cache:
        w = S.gen_weights(spec, 0)
        if offsets:
            w["draft_offset"] = S.gen_draft_offsets(spec, offsets, seed=1, std=1.0)
        packed = binding.pack_weights(spec, binding.weights_to_device(spec, w), group)
        plain = lambda m: binding.w4_unpack(m).cpu().numpy()
        held = dict(w, lm_head=plain(packed["lm_head"]).reshape(w["lm_head"].shape))
        held["layers"] = [{k: v if k.endswith("norm") else plain(p[k]) for k, v in lw.items()}
                          for lw, p in zip(w["layers"], packed["layers"])]
        _cache[key] = (orc.Model(spec, held), packed, held)
    return _cache[key]


def _decode(cp, x, c0):
    codes = cp.decode_frames(torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda())
    torch.cuda.synchronize()
    cp.status()
    return codes.cpu().numpy()


def _specs():
    from speculative_decoding_rvq_gb300 import synth as S
    return {"tiny": S.TINY_FP32, "bf16": _bf16_spec()}


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", ["tiny", "bf16"])
@pytest.mark.parametrize("N,B", [(0, 1), (4, 1), (8, 3)])
def test_teacher_logits(orc, name, group, N, B):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _specs()[name]
    m, dw, _ = _model(orc, spec, group)
    cp = binding.CpSpec(spec, dw, N, 50, 0.9, 1, max_streams=B)
    G = spec.num_code_groups
    x, _ = S.gen_frames(spec, B, 1, seed=5)
    codes = np.random.default_rng(0).integers(0, spec.vocab, (B, G - 1)).astype(np.int32)
    lg, dl = cp.teacher_logits(torch.from_numpy(x[0]).cuda(), torch.from_numpy(codes).cuda(), G, draft=N >= 2)
    torch.cuda.synchronize()
    cp.status()
    for b in range(B):
        o_lg, o_dl = m.teacher_logits(x[0, b], codes[b], G, n_draft=max(N - 1, 0))
        np.testing.assert_allclose(lg[b].cpu().numpy(), o_lg, atol=1e-4, rtol=0)
        if N >= 2:
            np.testing.assert_allclose(dl[b].cpu().numpy(), o_dl, atol=1e-4, rtol=0)


@pytest.mark.parametrize("name", ["tiny", "bf16"])
@pytest.mark.parametrize("N,T,B", [(0, 0.9, 2), (2, 0.9, 1), (4, 0.0, 2), (8, 0.9, 5)])
def test_decode_matches_oracle(orc, name, N, T, B):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _specs()[name]
    m, dw, _ = _model(orc, spec, 32)
    cp = binding.CpSpec(spec, dw, N, 50, T, 1, max_streams=B)
    x, c0 = S.gen_frames(spec, B, 5, seed=7)
    got = _decode(cp, x, c0)
    ref, _, log = m.decode_frames(N, 50, T, 1, x, c0)
    compare_codes_with_margins(got, ref, log, 1e-4)
    st = cp.stats()
    assert st["committed"] == 5 * B * (spec.num_code_groups - 1)
    assert st["kernel_launches"] == st["passes"] * (5 * spec.n_layers + 3) or B > 1
    # the whole call and the step-wise rounds give the same codes
    cps = binding.CpSpec(spec, dw, N, 50, T, 1, max_streams=B)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    G = spec.num_code_groups
    codes, done = torch.zeros((B, G), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    cps.begin_frame(xd[0].clone(), cd[0].clone(), 0)
    for _ in range(G):
        cps.round(codes, done)
    assert np.array_equal(codes.cpu().numpy(), got[0])


@pytest.mark.parametrize("name", ["tiny", "bf16"])
def test_greedy_speculation_is_greedy_decoding(orc, name):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _specs()[name]
    _, dw, _ = _model(orc, spec, 64)
    x, c0 = S.gen_frames(spec, 2, 12, seed=3)
    ar = _decode(binding.CpSpec(spec, dw, 0, 50, 0.0, 1, max_streams=2), x, c0)
    for N in range(2, 9):
        assert np.array_equal(_decode(binding.CpSpec(spec, dw, N, 50, 0.0, 1, max_streams=2), x, c0), ar), N
    # the row tiles: 9 streams x 4 rows are several blocks of 8 rows
    xx, cc = np.repeat(x[:, :1], 9, axis=1), np.repeat(c0[:, :1], 9, axis=1)
    many = _decode(binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=9), np.ascontiguousarray(xx), np.ascontiguousarray(cc))
    assert (many == ar[:, :1]).all()


def test_offsets_and_trees(orc):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = S.TINY_FP32
    m, dw, _ = _model(orc, spec, 32, offsets=2)
    x, c0 = S.gen_frames(spec, 2, 5, seed=9)
    got = _decode(binding.CpSpec(spec, dw, 4, 50, 0.9, 1, max_streams=2), x, c0)
    ref, _, log = m.decode_frames(4, 50, 0.9, 1, x, c0)
    compare_codes_with_margins(got, ref, log, 1e-4)
    m, dw, _ = _model(orc, spec, 32)
    par, rk = [-1, -1, 0, 0, 1, 2, 3], [0, 1, 0, 1, 0, 0, 0]
    got = _decode(binding.CpSpec(spec, dw, 4, 50, 0.9, 1, max_streams=2, tree=(par, rk)), x, c0)
    ref, _, log = m.decode_frames_tree(par, rk, 50, 0.9, 1, x, c0)
    compare_codes_with_margins(got, ref, log, 1e-4)


def test_benchmark_shapes(orc):
    """Two layers of the 0.6B-class decoder and of the large one (K up to 6144: fewer rows per CTA)."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    for spec, G in ((S.TTS06B_BF16, 5), (S.LARGE_BF16, 4)):
        spec = dataclasses.replace(spec, n_layers=2, num_code_groups=G)
        m, dw, _ = _model(orc, spec, 32)
        cp = binding.CpSpec(spec, dw, 4, 50, 0.9, 1, max_streams=2)
        x, c0 = S.gen_frames(spec, 2, 2, seed=6)
        codes = np.random.default_rng(1).integers(0, spec.vocab, (2, G - 1)).astype(np.int32)
        lg, _ = cp.teacher_logits(torch.from_numpy(x[0]).cuda(), torch.from_numpy(codes).cuda(), G)
        for b in range(2):
            o_lg, _ = m.teacher_logits(x[0, b], codes[b], G, n_draft=0)
            np.testing.assert_allclose(lg[b].cpu().numpy(), o_lg, atol=1e-4, rtol=0)
        got = _decode(cp, x, c0)
        ref, _, log = m.decode_frames(4, 50, 0.9, 1, x, c0)
        compare_codes_with_margins(got, ref, log, 1e-4, max_frac=0.5)


# ------------------------------------------------------------- 4-bit KV cache
def _border(x):
    """Smallest distance of a group's quotients x / s from a point between two held numbers, relative."""
    x = x.double().unflatten(-1, (-1, 32))
    s = (x.abs().amax(-1, keepdim=True) * SIXTH).float().bfloat16().double()
    r = (x / s).abs().unsqueeze(-1)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    return float(((r - mid).abs() / mid).min())


def _forward64(spec, held, x, codes):
    """Teacher-forced logits [G-1, V] in float64 with keys and values held in 4 bits, and the smallest border distance."""
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().double()
    emb = held["embed"]
    if emb.dtype == np.uint16:
        from speculative_decoding_rvq_gb300.synth import bf16_bits_to_f32
        emb = bf16_bits_to_f32(emb)
    G, d, nq, nkv = spec.num_code_groups, spec.head_dim, spec.n_q_heads, spec.n_kv_heads
    h = torch.stack([f(x)] + [f(emb[j - 1, codes[j - 1]]) for j in range(1, G)])
    norm = lambda a, g: a / torch.sqrt((a * a).mean(-1, keepdim=True) + spec.rms_eps) * f(g)
    ang = torch.arange(G, device="cuda").double().view(-1, 1) * spec.rope_theta ** (
        -torch.arange(0, d, 2, device="cuda").double() / d)
    cos, sin = torch.cos(ang).view(G, 1, -1), torch.sin(ang).view(G, 1, -1)

    def rope(a):
        lo, hi = a[..., :d // 2], a[..., d // 2:]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    near = math.inf
    for lw in held["layers"]:
        b = norm(h, lw["attn_norm"])
        q = rope((b @ f(lw["wq"]).t()).view(G, nq, d))
        k = rope((b @ f(lw["wk"]).t()).view(G, nkv, d))
        v = (b @ f(lw["wv"]).t()).view(G, nkv, d)
        near = min(near, _border(k), _border(v))
        k, v = (hold(a, 32).repeat_interleave(nq // nkv, 1) for a in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
        s = s.masked_fill(torch.ones(G, G, device="cuda").triu(1).bool(), -math.inf)
        h = h + torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).reshape(G, -1) @ f(lw["wo"]).t()
        b = norm(h, lw["ffn_norm"])
        g = b @ f(lw["w_gate"]).t()
        h = h + (g * torch.sigmoid(g) * (b @ f(lw["w_up"]).t())) @ f(lw["w_down"]).t()
    o = norm(h, held["final_norm"])
    return torch.stack([f(held["lm_head"][j - 1]) @ o[j] for j in range(1, G)]), near


@pytest.mark.parametrize("name", ["tiny", "bf16"])
@pytest.mark.parametrize("N,B", [(0, 1), (3, 2), (8, 4)])
def test_logits_with_a_4_bit_cache(orc, name, N, B):
    """A key or value within 1e-5 of a border between two held numbers may fall to either side in float32 (its own error
    is near 1e-6); the 1e-4 of the float contexts holds where none is, and such a step (at most 2 of 6 in one channel)
    stays well inside 0.05 of logits of unit size."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _specs()[name]
    _, dw, held = _model(orc, spec, 32)
    cp = binding.CpSpec(spec, dw, N, 50, 0.9, 1, max_streams=B, kv_bits=4)
    G = spec.num_code_groups
    x, _ = S.gen_frames(spec, B, 1, seed=5)
    codes = np.random.default_rng(0).integers(0, spec.vocab, (B, G - 1)).astype(np.int32)
    lg, _ = cp.teacher_logits(torch.from_numpy(x[0]).cuda(), torch.from_numpy(codes).cuda(), G)
    cp.status()
    for b in range(B):
        ref, near = _forward64(spec, held, x[0, b], codes[b])
        err = float((lg[b].double() - ref).abs().max())
        assert err <= (1e-4 if near > 1e-5 else 0.05), (err, near)


@pytest.mark.parametrize("name", ["tiny", "bf16"])
def test_decoding_with_a_4_bit_cache(orc, name):
    """Greedy codes are the argmax of the teacher-forced logits over them, for chain rounds, several streams and step-wise
    calls; the counters see a smaller cache and two kernels where there was one."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _specs()[name]
    _, dw, _ = _model(orc, spec, 32)
    G, F, B = spec.num_code_groups, 4, 3
    x, c0 = S.gen_frames(spec, B, F, seed=11)
    cp = binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=B, kv_bits=4)
    got = _decode(cp, x, c0)
    st = cp.stats()
    assert st["committed"] == F * B * (G - 1) and st["kernel_launches"] % (6 * spec.n_layers + 3) == 0
    full = binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=B)
    _decode(full, x, c0)
    fs = full.stats()
    assert cp.workspace.numel() < full.workspace.numel()
    assert abs(st["kv_bytes"] / st["passes"] / (fs["kv_bytes"] / fs["passes"]) / (1.125 / 8) - 1) < 0.2
    ahead = binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=B, kv_bits=4)
    for i in range(F):
        lg, _ = ahead.teacher_logits(torch.from_numpy(x[i]).cuda(), torch.from_numpy(np.ascontiguousarray(got[i][:, :G - 1])).cuda(), G)
        top = lg.double().topk(2, -1)
        want = top.indices[..., 0].cpu().numpy()
        sure = ((top.values[..., 0] - top.values[..., 1]) > 1e-3).cpu().numpy()
        assert (got[i][:, 1:][sure] == want[sure]).all() and sure.mean() > 0.9
    again = _decode(binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=B, kv_bits=4), x, c0)
    assert np.array_equal(again, got)


def test_context_refusals(orc):
    from speculative_decoding_rvq_gb300 import binding as b, synth as S
    spec = S.TINY_FP32
    _, dw, _ = _model(orc, spec, 32)
    w, m = S.gen_weights(spec, 0), None
    with pytest.raises(b.CpSpecError):
        b.CpSpec(spec, b.weights_to_device(spec, w), 4, 50, 0.9, 1, kv_bits=4)
    with pytest.raises(b.CpSpecError):
        b.CpSpec(spec, dw, 4, 50, 0.9, 1, kv_bits=8)
    with pytest.raises(b.CpSpecError) as e:
        b.CpSpec(spec, dw, 4, 50, 0.9, 1, kv_bits=4, tree=([-1, 0], [0, 0]))
    assert e.value.code in (b.E_UNSUPPORTED, b.E_INVALID)
    cp = b.CpSpec(spec, dw, 4, 50, 0.9, 1, kv_bits=4)
    for kw in (dict(stall_first_wait=True), dict(poison_kv=True)):
        with pytest.raises(b.CpSpecError) as e:
            cp.test_hooks(**kw)
        assert e.value.code == b.E_UNSUPPORTED
