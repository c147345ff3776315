"""The message of a call without a context belongs to the thread that made the call (no GPU needed)."""
import threading

import pytest


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_rvq_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def test_each_thread_keeps_its_own_message(b):
    lib, seen = b.load(), []
    assert lib.cp_spec_w4_bytes(0, 128, 32) == 0
    mine = lib.cp_spec_last_error(None)
    assert mine

    def other():
        before = lib.cp_spec_last_error(None)
        assert lib.cp_spec_w4_bytes(16, 128, 33) == 0
        seen.extend([before, lib.cp_spec_last_error(None)])
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert seen[0] == b"" and seen[1] and seen[1] != mine
    assert lib.cp_spec_last_error(None) == mine


def test_refusals_from_many_threads(b):
    """Each thread's refusals carry its own message, of different lengths, while the others are refused too."""
    lib, bad = b.load(), []
    calls = [lambda: lib.cp_spec_w4_bytes(0, 128, 32), lambda: lib.cp_spec_w4_bytes(16, 1 << 20, 32),
             lambda: lib.cp_spec_w4_bytes(16, 128, 33), lambda: lib.cp_spec_kv4_bytes(None)]
    want = []
    for f in calls:
        f()
        want.append(lib.cp_spec_last_error(None))
    assert len(set(want)) == 4

    def work(i):
        for _ in range(3000):
            calls[i]()
            got = lib.cp_spec_last_error(None)
            if got != want[i]:
                bad.append((i, got))
                return
    threads = [threading.Thread(target=work, args=(i % 4,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]
