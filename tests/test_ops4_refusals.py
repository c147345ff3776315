"""The 4-bit operators refuse bad arguments on the host, before any device work (no GPU needed)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_rvq_gb300 import binding, build
    build.build()
    return binding.load()


A = 4096  # an aligned address that is never followed
OFF = 4100


def _cache(b, **kw):
    d = dict(n_pages=8, page_size=16, n_kv_heads=2, head_dim=64)
    d.update(kw)
    return b.Kv4(*(d[n] for n in ("n_pages", "page_size", "n_kv_heads", "head_dim")))


def test_w4_sizes(lib):
    assert lib.cp_spec_w4_bytes(16, 128, 32) == 1024 + 128
    assert lib.cp_spec_w4_bytes(16, 128, 128) == 1024 + 32
    assert lib.cp_spec_w4_bytes(17, 129, 64) == 4 * (1024 + 64)
    # beyond 32 bits
    assert lib.cp_spec_w4_bytes(1 << 22, 32768, 128) == (1 << 18) * 256 * (1024 + 32)
    for bad in ((0, 128, 32), (16, 0, 32), (16, 128, 16), (16, 128, 0), (16, 32769, 32), (-1, 128, 32)):
        assert lib.cp_spec_w4_bytes(*bad) == 0, bad


def test_w4_refusals(lib):
    from speculative_decoding_rvq_gb300 import binding as b
    pack = lambda n=16, k=128, g=32, dt=0, w=A, st=128, p=A: lib.cp_spec_w4_pack(n, k, g, dt, w, st, p, None)
    for kw in (dict(n=0), dict(k=0), dict(g=33), dict(dt=3), dict(dt=-1), dict(w=None), dict(w=OFF), dict(p=None),
               dict(p=OFF), dict(st=127)):
        assert pack(**kw) == b.E_INVALID, kw
    assert pack(k=40000, st=40000) == b.E_UNSUPPORTED
    unpack = lambda dt=0, p=A, w=A: lib.cp_spec_w4_unpack(16, 128, 32, dt, p, w, None)
    for kw in (dict(dt=3), dict(p=None), dict(w=OFF)):
        assert unpack(**kw) == b.E_INVALID, kw
    gemv = lambda r=1, n=16, k=128, g=32, dt=1, o=1, x=A, xs=128, p=A, y=A, ys=16: lib.cp_spec_w4_gemv(
        r, n, k, g, dt, o, x, xs, p, y, ys, None)
    for kw in (dict(r=-1), dict(r=65536), dict(n=0), dict(g=48), dict(dt=3), dict(o=2), dict(dt=2, o=1), dict(x=None),
               dict(x=OFF), dict(xs=127), dict(p=None), dict(y=OFF), dict(ys=15)):
        assert gemv(**kw) == b.E_INVALID, kw
    assert gemv(r=0, x=None, y=None) == b.OK
    assert b"stride" not in lib.cp_spec_last_error(None) or gemv(ys=1) == b.E_INVALID


def test_kv4_refusals(lib):
    from speculative_decoding_rvq_gb300 import binding as b
    ok = _cache(b)
    assert lib.cp_spec_kv4_bytes(C.byref(ok)) == 8 * 2 * 18 * 64
    assert lib.cp_spec_kv4_bytes(C.byref(_cache(b, n_pages=1 << 20, page_size=128, n_kv_heads=8, head_dim=256))) == (
        (1 << 20) * 8 * 8 * 18 * 256)
    for bad in (dict(n_pages=0), dict(page_size=8), dict(page_size=24), dict(page_size=0), dict(n_kv_heads=0),
                dict(n_kv_heads=2000), dict(head_dim=96), dict(head_dim=0), dict(head_dim=512)):
        assert lib.cp_spec_kv4_bytes(C.byref(_cache(b, **bad))) == 0, bad
    assert lib.cp_spec_kv4_bytes(None) == 0

    def append(shape=ok, cache=A, pages=A, per=2, seqs=4, rows=3, pos=A, nr=None, dt=0, k=A, ks=128, v=A, vs=128):
        return lib.cp_spec_kv4_append(C.byref(shape), cache, pages, per, seqs, rows, pos, nr, dt, k, ks, v, vs, None)

    def read(shape=ok, cache=A, pages=A, per=2, seqs=4, n=20, ln=None, dt=0, k=A, v=A):
        return lib.cp_spec_kv4_read(C.byref(shape), cache, pages, per, seqs, n, ln, dt, k, v, None)

    def attn(shape=ok, cache=A, pages=A, per=2, seqs=4, rows=3, nq=4, kl=A, nr=None, mask=None, scale=0.125, dt=0, q=A, qs=256,
             o=A, os_=256, lse=None, work=None, nbytes=0):
        return lib.cp_spec_kv4_attention(C.byref(shape), cache, pages, per, seqs, rows, nq, kl, nr, mask, scale, dt, q, qs, o,
                                         os_, lse, work, nbytes, None)

    shared = (dict(cache=None), dict(cache=OFF), dict(pages=OFF), dict(per=0), dict(per=1 << 28), dict(seqs=-1),
              dict(pages=None, per=3), dict(dt=3), dict(shape=_cache(b, page_size=8)))
    for f in (append, read, attn):
        for kw in shared:
            assert f(**kw) == b.E_INVALID, (f.__name__, kw)
        assert f(shape=_cache(b, head_dim=80)) == b.E_UNSUPPORTED
        assert f(seqs=0) == b.OK
    assert append(rows=1 << 26) == read(n=1 << 26) == b.E_UNSUPPORTED  # 2^25 pairs of rows of 128 elements: above 2^32
    for kw in (dict(rows=-1), dict(pos=None), dict(pos=OFF), dict(nr=OFF), dict(k=None), dict(v=OFF), dict(ks=127), dict(vs=0)):
        assert append(**kw) == b.E_INVALID, kw
    assert append(rows=0) == b.OK
    for kw in (dict(n=-1), dict(ln=OFF), dict(k=None), dict(v=OFF)):
        assert read(**kw) == b.E_INVALID, kw
    assert read(n=0) == b.OK
    for kw in (dict(nq=3), dict(nq=0), dict(nq=8192), dict(kl=None), dict(kl=OFF), dict(nr=OFF), dict(mask=OFF),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=OFF), dict(qs=255), dict(o=None),
               dict(os_=255), dict(lse=OFF), dict(work=OFF)):
        assert attn(**kw) == b.E_INVALID, kw
    assert attn(rows=65) == attn(seqs=1 << 27) == b.E_UNSUPPORTED
    assert attn(rows=0) == b.OK
    for bad in (dict(rows=65), dict(nq=3), dict(dt=3), dict(per=0), dict(seqs=0)):
        d = dict(per=2, seqs=4, rows=3, nq=4, dt=0)
        d.update(bad)
        assert lib.cp_spec_kv4_attention_bytes(C.byref(ok), d["per"], d["seqs"], d["rows"], d["nq"], d["dt"]) == 0


def test_binding_refuses_wrong_tensors(lib):
    """What the binding checks before it hands pointers on (CPU tensors never reach the library)."""
    torch = pytest.importorskip("torch")
    from speculative_decoding_rvq_gb300 import binding as b

    def refused(f):
        with pytest.raises(b.CpSpecError) as e:
            f()
        assert e.value.code == b.E_INVALID
    w = b.W4Matrix(16, 128, 32, torch.zeros(2304, dtype=torch.uint8))
    x = torch.zeros(2, 128)
    refused(lambda: b.w4_gemv(torch.zeros(2, 127), w))
    refused(lambda: b.w4_gemv(torch.zeros(128, 2).t(), w))
    refused(lambda: b.w4_gemv(x.double(), w))
    refused(lambda: b.w4_gemv(x, w, out=torch.zeros(2, 15)))
    refused(lambda: b.w4_gemv(x, w, out=torch.zeros(2, 16), out_dtype=torch.bfloat16))
    refused(lambda: b.w4_gemv(x, w))  # not on a CUDA device
    refused(lambda: b.w4_pack(torch.zeros(4, 4, 4)))
    refused(lambda: b.w4_pack(torch.zeros(4, 8).t()))
    refused(lambda: b.w4_unpack(w))
    c = b.Kv4Cache(8, 16, 2, 64, device="cpu")
    k = torch.zeros(2, 3, 2, 64)
    pos = torch.zeros(2, dtype=torch.int32)
    refused(lambda: c.append(k, k[:, :2], pos))
    refused(lambda: c.append(k, k.double(), pos))
    refused(lambda: c.append(torch.zeros(2, 3, 2, 32), torch.zeros(2, 3, 2, 32), pos))
    refused(lambda: c.append(k, k, pos.long()))
    refused(lambda: c.append(k, k, pos[:1]))
    refused(lambda: c.append(k, k, pos, pages=torch.zeros(3, 4, dtype=torch.int32)))
    refused(lambda: c.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, pos))
    refused(lambda: c.append(k, k, pos))  # not on a CUDA device
    refused(lambda: c.attention(torch.zeros(2, 3, 4, 32), pos))
    refused(lambda: c.attention(torch.zeros(2, 3, 4, 64), pos, mask=torch.zeros(2, 2, dtype=torch.int64)))
    refused(lambda: c.attention(torch.zeros(2, 3, 4, 64), pos, mask=torch.zeros(2, 3, dtype=torch.int32)))
    refused(lambda: c.attention(torch.zeros(2, 3, 4, 64), pos, out=torch.zeros(2, 3, 4, 64, dtype=torch.float16)))
    refused(lambda: c.read(4, n_seqs=2))
    for bad in ((0, 16, 2, 64), (8, 20, 2, 64), (8, 16, 2, 72)):
        with pytest.raises(b.CpSpecError):
            b.Kv4Cache(*bad, device="cpu")


def test_w4_context_sizes_and_refusals(lib):
    from speculative_decoding_rvq_gb300 import binding as b, synth as S
    m = b.model_struct(S.TINY_FP32)
    cfg = b.Config(4, 50, 0.9, 1, 2)
    size = lambda model=m, group=32, bits=32: lib.cp_spec_workspace_bytes_w4(C.byref(model), C.byref(cfg), None,
                                                                             C.byref(b.Quant(group, bits)))
    assert size() == lib.cp_spec_workspace_bytes(C.byref(m), C.byref(cfg))
    assert 0 < size(bits=4) < size()
    for bad in (dict(group=16), dict(group=0), dict(bits=8), dict(bits=0)):
        assert size(**bad) == 0, bad
    for d, v in ((48, 256), (64, 250)):
        other = b.model_struct(S.ModelSpec(256, 2, 4, 4, d, 768, v, 8, 0))
        assert size(model=other) == 0
    narrow = b.model_struct(S.ModelSpec(256, 2, 4, 4, 32, 768, 256, 8, 0))
    assert size(model=narrow) > 0 and size(model=narrow, bits=4) == 0
    ctx = C.c_void_p()
    w = b.Weights()
    q = b.Quant(32, 32)
    assert lib.cp_spec_init_w4(C.byref(m), C.byref(w), C.byref(cfg), None, None, A, 1 << 30, C.byref(ctx)) == b.E_INVALID
    assert lib.cp_spec_init_w4(C.byref(m), C.byref(w), C.byref(cfg), None, C.byref(q), A, 1 << 30, C.byref(ctx)) == b.E_INVALID
    assert lib.cp_spec_init_w4(C.byref(m), None, C.byref(cfg), None, C.byref(q), A, 1 << 30, C.byref(ctx)) == b.E_INVALID
