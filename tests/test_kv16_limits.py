"""Limits of the 16-bit cache's operators that the library refuses on the host (no GPU needed)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_rvq_gb300 import binding, build
    build.build()
    return binding.load()


A = 4096  # an aligned address that is never followed


def test_scales_past_the_range_of_powers_of_two(lib):
    """Scores are formed with scale * log2(e): a scale for which that is no float32 is refused, not turned into NaN."""
    from speculative_decoding_rvq_gb300 import binding as b
    shape = b.Kv16(8, 16, 2, 64, 1)

    def attend(scale, rows=6):
        return lib.cp_spec_kv16_attention(C.byref(shape), A, A, 4, 2, rows, 3, 4, A, A, None, 0, 0, scale, A, 256, A, 256, None, None, 0,
                                          None, None)

    for scale in (3e38, -3e38, 2.4e38):
        assert attend(scale) == b.E_INVALID, scale
    for scale in (0.0, -0.0, 1e-45, 2.0 ** 127, -(2.0 ** 127)):  # (no rows: nothing is launched)
        assert attend(scale, rows=0) == b.OK, scale


def test_hooks_without_a_context(lib):
    from speculative_decoding_rvq_gb300 import binding as b
    for ns, flags in ((100, 0), (10 ** 11, 0), (2_000_000_000, 3), (2_000_000_000, -1)):
        assert lib.cp_spec_test_hooks(None, ns, flags) == b.E_INVALID
    assert lib.cp_spec_test_hooks(None, 2_000_000_000, 0) == b.OK
