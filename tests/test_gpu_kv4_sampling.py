"""Sampled decoding over a 4-bit KV cache: the codes are the ones that the oracle's sampling and acceptance draw from the
teacher-forced logits of the same context over those codes.

The target row of a draft is read only while every draft before it was accepted, so its inputs are the committed codes
and its logits are the teacher-forced ones.  What is left between the two sides is the float32 softmax of the kernels
against the oracle's float64 one: decisions with a margin below 1e-4, as in the float contexts."""
import numpy as np
import pytest

from gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu
SEED, TOP_K, T = 5, 50, 0.9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _spec(name):
    from speculative_decoding_rvq_gb300 import synth as S
    return S.TINY_FP32 if name == "tiny" else S.ModelSpec(512, 2, 8, 4, 64, 1040, 528, 9, S.DTYPE_BF16)


def _frame(orc, N, G, stream, frame, lg, dl, got):
    """Replays one frame; True where every code is got's, False where the first difference was a near-tie."""
    u = lambda depth, purpose: orc.uniform(SEED, stream, frame, depth, purpose)
    law = lambda logits: orc.process(logits, TOP_K, T)

    def agree(at, codes, margin):
        want = got[at:at + len(codes)].tolist()
        assert codes == want or margin < 1e-4, (stream, frame, at, codes, want, margin)
        return codes == want
    p, m0 = law(lg[0])
    c, m1 = orc.sample(p, u(1, orc.ORC_TARGET))
    if not agree(1, [c], min(m0, m1)):
        return False
    s = 1
    while s < G - 1:
        left = G - 1 - s
        n_d = min(N - 1, left) if N else 0
        margins, q, drafts = [], [], []
        for t in range(1, n_d + 1):
            row, m0 = law(dl[s - 1, t - 1])  # lookahead t at position s
            y, m1 = orc.sample(row, u(s + t, orc.ORC_DRAFT))
            q.append(row)
            drafts.append(y)
            margins += [m0, m1]
        rows = min(n_d + 1, left)
        p = []
        for i in range(rows):
            row, m0 = law(lg[s + i])  # position s + 1 + i
            p.append(row)
            margins.append(m0)
        if n_d:
            _, codes, m1 = orc.accept_chain(np.stack(q), drafts, np.stack(p), [u(s + t, orc.ORC_ACCEPT) for t in range(1, n_d + 1)],
                                            [u(s + t, orc.ORC_TARGET) for t in range(1, n_d + 2)])
        else:
            c, m1 = orc.sample(p[0], u(s + 1, orc.ORC_TARGET))
            codes = [c]
        if not agree(s + 1, codes, min(margins + [m1])):
            return False
        s += len(codes)
    return True


@pytest.mark.parametrize("name", ["tiny", "bf16"])
@pytest.mark.parametrize("N", [0, 2, 4, 8])
def test_sampled_codes_follow_the_logits(orc, name, N):
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec, F, B = _spec(name), 6, 3
    dw = binding.pack_weights(spec, binding.weights_to_device(spec, S.gen_weights(spec, 0)), 32)
    x, c0 = S.gen_frames(spec, B, F, seed=13)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    new = lambda: binding.CpSpec(spec, dw, N, TOP_K, T, SEED, max_streams=B, kv_bits=4)
    cp = new()
    got = cp.decode_frames(xd, cd).cpu().numpy()
    cp.status()
    G, ties, steps = spec.num_code_groups, 0, new()
    ahead = new()
    for f in range(F):
        codes = torch.from_numpy(np.ascontiguousarray(got[f][:, :G - 1])).cuda()
        lg, dl = ahead.teacher_logits(xd[f].contiguous(), codes, G, draft=N >= 2)
        lg, dl = lg.cpu().numpy(), None if dl is None else dl.cpu().numpy()
        for i in range(B):
            ties += not _frame(orc, N, G, i, f, lg[i], None if dl is None else dl[i], got[f, i])
    assert ties <= 1
    # pass by pass: the same codes
    codes, done = torch.zeros((B, G), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    for f in range(F):
        steps.begin_frame(xd[f].clone(), cd[f].clone(), f)
        for _ in range(G):
            steps.round(codes, done)
        assert (done == G).all() and np.array_equal(codes.cpu().numpy(), got[f])
