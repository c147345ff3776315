"""Packed contexts at shapes and options beside the small models': frames of several tiles, many query heads to a KV head,
every head size of the 4-bit cache, the adaptive window, sampling per stream, draft offsets over the 4-bit cache."""
import numpy as np
import pytest

from gpu_common import compare_codes_with_margins, require_gpu, torch
from test_gpu_w4_context import _forward64, _model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _spec(nq, nkv, d, G, dtype=0):
    from speculative_decoding_rvq_gb300 import synth as S
    return S.ModelSpec(256, 2, nq, nkv, d, 320, 256, G, dtype)


@pytest.mark.parametrize("nq,nkv,d,G", [(4, 2, 64, 40), (16, 1, 64, 17), (8, 4, 128, 64), (4, 1, 256, 33), (2, 2, 64, 3)])
@pytest.mark.parametrize("N,B", [(0, 3), (8, 2)])
def test_logits_with_a_4_bit_cache(orc, nq, nkv, d, G, N, B):
    """As in the small models: 1e-4 where no key or value lies within 1e-5 of a border between two held numbers."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _spec(nq, nkv, d, G)
    _, dw, held = _model(orc, spec, 32)
    cp = binding.CpSpec(spec, dw, N, 50, 0.9, 1, max_streams=B, kv_bits=4)
    x, _ = S.gen_frames(spec, B, 1, seed=5)
    codes = np.random.default_rng(0).integers(0, spec.vocab, (B, G - 1)).astype(np.int32)
    lg, _ = cp.teacher_logits(torch.from_numpy(x[0]).cuda(), torch.from_numpy(codes).cuda(), G)
    cp.status()
    for b in range(B):
        ref, near = _forward64(spec, held, x[0, b], codes[b])
        err = float((lg[b].double() - ref).abs().max())
        assert err <= (1e-4 if near > 1e-5 else 0.05), (err, near)


@pytest.mark.parametrize("kv_bits", [32, 4])
def test_adaptive_window_and_sampling_per_stream(orc, kv_bits):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec, B, F = _spec(8, 4, 64, 12), 3, 12
    m, dw, _ = _model(orc, spec, 64)
    x, c0 = S.gen_frames(spec, B, F, seed=3)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    cp = binding.CpSpec(spec, dw, 6, 50, 0.9, 1, max_streams=B, adapt_pct=40, adapt_min=8, kv_bits=kv_bits)
    top_k, temp = [50, 7, 20], [0.9, 0.0, 1.3]
    cp.set_stream_sampling(top_k, temp)
    got = cp.decode_frames(xd, cd).cpu().numpy()
    cp.status()
    if kv_bits == 32:
        ref, _, log = m.decode_frames(6, top_k, temp, 1, x, c0, adapt_pct=40, adapt_min=8, log_cap=F * B * 12)
        compare_codes_with_margins(got, ref, log, 1e-4)
    else:  # the greedy stream: the argmax of its own logits; the others: codes of the vocabulary
        assert (got >= 0).all() and (got < spec.vocab).all()
        sure = right = 0
        for f in range(F):
            lg, _ = cp.teacher_logits(xd[f].contiguous(), torch.from_numpy(np.ascontiguousarray(got[f][:, :11])).cuda(), 12)
            top = lg[1].double().topk(2, -1)
            ok = ((top.values[:, 0] - top.values[:, 1]) > 1e-3).cpu().numpy()
            sure += ok.sum()
            right += (got[f, 1, 1:] == top.indices[:, 0].cpu().numpy())[ok].sum()
        assert sure == right and sure > 0.9 * F * 11


@pytest.mark.parametrize("kv_bits", [32, 4])
def test_draft_offsets(orc, kv_bits):
    """Offsets move the drafts, not the law: greedy codes are those without offsets and of the AR loop."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec, B, F = _spec(4, 2, 64, 9), 2, 8
    _, plain, _ = _model(orc, spec, 32)
    _, moved, _ = _model(orc, spec, 32, offsets=3)
    x, c0 = S.gen_frames(spec, B, F, seed=3)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    run = lambda dw, N: binding.CpSpec(spec, dw, N, 50, 0.0, 1, max_streams=B, kv_bits=kv_bits).decode_frames(xd, cd).cpu().numpy()
    ar = run(plain, 0)
    for N in (2, 5):
        a, c = run(plain, N), run(moved, N)
        if kv_bits == 32:
            assert np.array_equal(a, ar) and np.array_equal(c, ar)
        else:  # (a value on a rounding border may fall to the other side in another window)
            assert (a == ar).all(-1).mean() >= 0.75 and (c == ar).all(-1).mean() >= 0.75


@pytest.mark.parametrize("kv_bits", [32, 4])
def test_many_streams(orc, kv_bits):
    """300 streams of the same few frames: each decodes as it does beside 2."""
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = _spec(4, 2, 64, 9)
    _, dw, _ = _model(orc, spec, 32)
    x, c0 = S.gen_frames(spec, 3, 2, seed=3)
    few = binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=3, kv_bits=kv_bits)
    want = few.decode_frames(torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()).cpu().numpy()
    cp = binding.CpSpec(spec, dw, 4, 50, 0.0, 1, max_streams=300, kv_bits=kv_bits)
    xx, cc = (torch.from_numpy(np.ascontiguousarray(np.tile(a, (1, 100) + (1,) * (a.ndim - 2)))).cuda() for a in (x, c0))
    got = cp.decode_frames(xx, cc).cpu().numpy()
    cp.status()
    assert np.array_equal(got, np.tile(want, (1, 100, 1)))
