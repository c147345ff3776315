"""Packed weights reach the calls that take them and no other, with the shapes and groups that the call names (no GPU
needed: the library is replaced by a recorder that nothing may reach)."""
import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_rvq_gb300 import binding as b, synth as S

SPEC = S.TINY_FP32


@pytest.fixture
def no_library(monkeypatch):
    class Untouched:
        def __getattr__(self, name):
            raise AssertionError(f"the binding reached {name}")
    monkeypatch.setattr(b, "load", lambda: Untouched())


def _matrix(n, k, group, rows=None):
    return b.W4Matrix(n, k, group, torch.zeros(16, dtype=torch.uint8))


def _packed(group=32):
    """Weights as pack_weights returns them, with empty codes."""
    s, qd, kvd = SPEC, SPEC.n_q_heads * SPEC.head_dim, SPEC.n_kv_heads * SPEC.head_dim
    shapes = dict(wq=(qd, s.hidden), wk=(kvd, s.hidden), wv=(kvd, s.hidden), wo=(s.hidden, qd), w_gate=(s.ffn, s.hidden),
                  w_up=(s.ffn, s.hidden), w_down=(s.hidden, s.ffn))
    norm = torch.ones(s.hidden)
    layers = [dict({k: _matrix(*v, group) for k, v in shapes.items()}, attn_norm=norm, ffn_norm=norm)
              for _ in range(s.n_layers)]
    return dict(w4_group=group, embed=torch.zeros(s.num_code_groups - 1, s.vocab, s.hidden), final_norm=norm,
                lm_head=_matrix((s.num_code_groups - 1) * s.vocab, s.hidden, group), layers=layers)


def _refused(f):
    with pytest.raises(b.CpSpecError) as e:
        f()
    assert e.value.code == b.E_INVALID, e.value
    return str(e.value)


def test_decode_without_a_context_refuses_packed_weights(no_library):
    x, c0 = torch.zeros(1, 1, SPEC.hidden), torch.zeros(1, 1, dtype=torch.int32)
    assert "packed" in _refused(lambda: b.decode_frames_static(SPEC, _packed(), 4, 50, 0.9, 1, x, c0))
    w = _packed()
    del w["w4_group"]  # (the matrices alone say it too)
    _refused(lambda: b.decode_frames_static(SPEC, w, 4, 50, 0.9, 1, x, c0))


def test_contexts_refuse_mixed_weights(no_library):
    """A plain matrix among packed ones, and packed ones without their group."""
    spec = (4, 50, 0.9, 1)
    for name in ("wq", "w_down"):
        w = _packed()
        w["layers"][-1][name] = torch.zeros(w["layers"][-1][name].n, SPEC.hidden)
        _refused(lambda: b.CpSpec(SPEC, w, *spec))
    w = _packed()
    w["lm_head"] = torch.zeros(SPEC.num_code_groups - 1, SPEC.vocab, SPEC.hidden)
    _refused(lambda: b.CpSpec(SPEC, w, *spec))
    w = _packed()
    del w["w4_group"]
    _refused(lambda: b.CpSpec(SPEC, w, *spec))


@pytest.mark.parametrize("name", ["wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "lm_head"])
def test_contexts_refuse_other_shapes_and_groups(no_library, name):
    """Each matrix has the model's rows and columns and the one group that the context is made for."""
    for change in (dict(n=16), dict(n=-16), dict(k=128), dict(k=-128), dict(group=64)):
        w = _packed()
        at = w if name == "lm_head" else w["layers"][-1]
        m = at[name]
        at[name] = _matrix(m.n + change.get("n", 0), m.k + change.get("k", 0), change.get("group", m.group))
        assert name in _refused(lambda: b.CpSpec(SPEC, w, 4, 50, 0.9, 1)), change
    w = _packed(32)
    w["w4_group"] = 128  # matrices packed with groups of 32
    _refused(lambda: b.CpSpec(SPEC, w, 4, 50, 0.9, 1))


def test_contexts_refuse_short_matrices(monkeypatch):
    """Fewer bytes than a packed matrix of that shape has."""
    class Sizes:
        def cp_spec_w4_bytes(self, n, k, group):
            return (n + 15) // 16 * ((k + 127) // 128) * (1024 + 32 * (128 // group))
    monkeypatch.setattr(b, "load", lambda: Sizes())
    assert "bytes" in _refused(lambda: b.CpSpec(SPEC, _packed(), 4, 50, 0.9, 1))


def test_sizes_beyond_32_bits_are_refused(no_library):
    """The library takes 32-bit sizes: a larger one must not reach it as its low half."""
    many = (1 << 32) + 16
    assert "rows" in _refused(lambda: b.w4_pack(torch.zeros(1, 1).expand(many, 1)))
    assert "rows" in _refused(lambda: b.w4_gemv(torch.zeros(1, 1).expand(many, 1), _matrix(16, 1, 32)))
    for at in range(3):
        sizes = [8, 16, 2, 64]
        sizes[at] += 1 << 32
        _refused(lambda: b.Kv4Cache(*sizes, device="cpu"))


def test_a_missing_library_says_so_every_time(monkeypatch):
    """The second call too (PyTorch is imported by then)."""
    monkeypatch.setattr(b, "_lib", None)
    monkeypatch.setattr(b, "LIB_PATH", "/nowhere/libcpspec.so")
    for _ in range(2):
        with pytest.raises(RuntimeError, match="not built"):
            b.w4_gemv(torch.zeros(2, 128), _matrix(16, 128, 32))
