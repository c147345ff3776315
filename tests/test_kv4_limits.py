"""Sizes at the edge of what the 4-bit cache takes (on the host, no GPU needed)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_rvq_gb300 import binding, build
    build.build()
    return binding.load()


def test_a_cache_whose_size_passes_64_bits_is_refused(lib):
    """n_pages is the one size without a limit of its own: the bytes of all pages have to stay below 2^48, where no
    offset wraps."""
    from speculative_decoding_rvq_gb300 import binding as b
    page = 1024 * (1 << 16) * 18 * 256  # the largest page: 1024 heads x 256 channels x 2^20 slots
    most = (1 << 48) // page
    size = lambda *shape: lib.cp_spec_kv4_bytes(C.byref(b.Kv4(*shape)))
    assert size(most, 1 << 20, 1024, 256) == most * page < 1 << 48
    for n in (most + 1, 1 << 26, (1 << 26) + 1, 0x7FFFFFFF):
        assert size(n, 1 << 20, 1024, 256) == 0, n
    assert size(0x7FFFFFFF, 16, 1, 64) == 0x7FFFFFFF * 18 * 64  # the most pages of the smallest kind fit
    huge = b.Kv4(0x7FFFFFFF, 1 << 20, 1024, 256)
    A = 4096  # an aligned address that is never followed
    assert lib.cp_spec_kv4_append(C.byref(huge), A, A, 1, 0, 1, A, None, 0, A, 1 << 18, A, 1 << 18, None) == b.E_UNSUPPORTED
    assert lib.cp_spec_kv4_read(C.byref(huge), A, A, 1, 0, 1, None, 0, A, A, None) == b.E_UNSUPPORTED
    assert lib.cp_spec_kv4_attention(C.byref(huge), A, A, 1, 0, 1, 1024, A, None, None, 1.0, 0, A, 1 << 18, A, 1 << 18, None,
                                     None, 0, None) == b.E_UNSUPPORTED
    assert lib.cp_spec_kv4_attention_bytes(C.byref(huge), 1, 1, 1, 1024, 0) == 0


def test_sizes_above_two_gigabytes_come_back_whole(lib):
    """A context over packed weights with many streams: its workspace passes 2^31 and 2^32 bytes, as the plain one's does."""
    from speculative_decoding_rvq_gb300 import binding as b, synth as S
    m = b.model_struct(S.TTS06B_BF16)
    for streams in (256, 512, 1024, 2048, 4096):
        cfg = b.Config(8, 50, 0.9, 1, streams)
        plain = lib.cp_spec_workspace_bytes(C.byref(m), C.byref(cfg))
        assert lib.cp_spec_workspace_bytes_w4(C.byref(m), C.byref(cfg), None, C.byref(b.Quant(32, 32))) == plain
        assert 0 < lib.cp_spec_workspace_bytes_w4(C.byref(m), C.byref(cfg), None, C.byref(b.Quant(32, 4))) < plain
    assert plain > 1 << 32
