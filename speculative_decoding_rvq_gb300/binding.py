"""Thin ctypes binding of the C ABI in include/cp_spec.h.

Argument marshalling only: every step of the decode runs in the CUDA
library.  PyTorch provides device memory and the current CUDA stream.  If the
library is missing or cannot be loaded this module raises; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

from . import synth

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcpspec.so")
MAX_LAYERS = 64

OK, W_AR_FALLBACK = 0, 1
E_INVALID, E_UNSUPPORTED, E_CUDA, E_WORKSPACE, E_DEVICE_TIMEOUT, E_STATE, E_DEVICE = -1, -2, -3, -4, -5, -6, -7

# Every symbol include/cp_spec.h declares.
EXPORTS = ("cp_spec_workspace_bytes", "cp_spec_init", "cp_spec_set_stream_sampling", "cp_spec_decode_frames",
           "cp_spec_begin_frame", "cp_spec_round", "cp_spec_teacher_logits", "cp_spec_accept_batch",
           "cp_spec_status_word", "cp_spec_read_stats", "cp_spec_reset_stats", "cp_spec_launch_count",
           "cp_spec_last_error", "cp_spec_destroy", "cp_spec_decode_frames_static", "cp_spec_test_hooks",
           "cp_spec_workspace_bytes_tree", "cp_spec_init_tree", "cp_spec_w4_bytes", "cp_spec_w4_pack",
           "cp_spec_w4_unpack", "cp_spec_w4_gemv", "cp_spec_kv4_bytes", "cp_spec_kv4_append", "cp_spec_kv4_read",
           "cp_spec_kv4_attention", "cp_spec_kv4_attention_bytes", "cp_spec_workspace_bytes_w4", "cp_spec_init_w4",
           "cp_spec_kv_plan", "cp_spec_rope_init", "cp_spec_rope_rows", "cp_spec_kv16_bytes", "cp_spec_kv16_append",
           "cp_spec_kv16_attention", "cp_spec_kv16_attention_bytes")
MAX_W4_N, MAX_W4_K, MAX_KV4_ROWS = 1 << 30, 32768, 64
MAX_PLAN_SEQS, MAX_TREE_ROWS, MAX_KV16_ROWS = 4096, 64, 1 << 24


class CpSpecError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"cp_spec status {code}: {msg}")
        self.code = code


class Model(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("hidden", "n_layers", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab",
                                         "num_code_groups", "dtype")] + [("rope_theta", C.c_float),
                                                                          ("rms_eps", C.c_float)]


class Weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("lm_head", C.c_void_p), ("final_norm", C.c_void_p)] + [
        (n, C.c_void_p * MAX_LAYERS) for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up",
                                               "w_down")] + [("draft_offset", C.c_void_p)]


class Config(C.Structure):
    _fields_ = [("verify_window", C.c_int32), ("top_k", C.c_int32), ("temperature", C.c_float),
                ("seed", C.c_uint64), ("max_streams", C.c_int32), ("draft_offsets", C.c_int32),
                ("adapt_accept_pct", C.c_int32), ("adapt_min_reached", C.c_int32)]


class Tree(C.Structure):
    _fields_ = [("n", C.c_int32), ("parent", C.c_void_p), ("rank", C.c_void_p)]


class Quant(C.Structure):
    _fields_ = [("group", C.c_int32), ("kv_bits", C.c_int32)]


class Kv4(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim")]


class RopeStruct(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("n_axes", C.c_int32), ("axis", C.c_uint8 * 128), ("turns", C.c_uint64 * 128)]


class Kv16(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim", "dtype")]


class Stats(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("frames", "passes", "rounds", "committed", "bonus", "rejections")] + [
        ("drafted_by_offset", C.c_int64 * 9), ("accepted_by_offset", C.c_int64 * 9)] + [
        (n, C.c_int64) for n in ("weight_bytes", "kv_bytes", "heads_applied", "kernel_launches")] + [("reserved", C.c_int64 * 7)]

    def as_dict(self) -> dict:
        d = {n: int(getattr(self, n)) for n, _ in self._fields_ if not n.endswith("_offset") and n != "reserved"}
        d["drafted_by_offset"] = [int(v) for v in self.drafted_by_offset]
        d["accepted_by_offset"] = [int(v) for v in self.accepted_by_offset]
        return d


_lib = None


def load():
    """Load libcpspec.so (raises if it is missing: the path has no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} (run __graft_entry__.build())")
    L = C.CDLL(LIB_PATH)
    vp, i32, f32, u64, sz = C.c_void_p, C.c_int32, C.c_float, C.c_uint64, C.c_size_t
    L.cp_spec_workspace_bytes.argtypes = [vp, vp]
    L.cp_spec_workspace_bytes.restype = sz
    L.cp_spec_init.argtypes = [vp, vp, vp, vp, sz, C.POINTER(vp)]
    L.cp_spec_workspace_bytes_tree.argtypes = [vp, vp, vp]
    L.cp_spec_workspace_bytes_tree.restype = sz
    L.cp_spec_init_tree.argtypes = [vp, vp, vp, vp, vp, sz, C.POINTER(vp)]
    L.cp_spec_set_stream_sampling.argtypes = [vp, i32, vp, vp]
    L.cp_spec_decode_frames.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    L.cp_spec_begin_frame.argtypes = [vp, i32, vp, vp, i32, vp]
    L.cp_spec_round.argtypes = [vp, vp, vp, vp]
    L.cp_spec_teacher_logits.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp]
    L.cp_spec_accept_batch.argtypes = [i32, i32, i32, i32, f32, u64, i32, vp, vp, vp, vp, vp, vp]
    L.cp_spec_decode_frames_static.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    i64 = C.c_int64
    L.cp_spec_w4_bytes.argtypes = [i32, i32, i32]
    L.cp_spec_w4_bytes.restype = sz
    L.cp_spec_w4_pack.argtypes = [i32, i32, i32, i32, vp, i64, vp, vp]
    L.cp_spec_w4_unpack.argtypes = [i32, i32, i32, i32, vp, vp, vp]
    L.cp_spec_w4_gemv.argtypes = [i32, i32, i32, i32, i32, i32, vp, i64, vp, vp, i64, vp]
    L.cp_spec_kv4_bytes.argtypes = [vp]
    L.cp_spec_kv4_bytes.restype = sz
    L.cp_spec_kv4_append.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, i64, vp, i64, vp]
    L.cp_spec_kv4_read.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp]
    L.cp_spec_kv4_attention.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, f32, i32, vp, i64, vp, i64, vp, vp, sz, vp]
    L.cp_spec_kv4_attention_bytes.argtypes = [vp, i32, i32, i32, i32, i32]
    L.cp_spec_kv4_attention_bytes.restype = sz
    L.cp_spec_workspace_bytes_w4.argtypes = [vp, vp, vp, vp]
    L.cp_spec_workspace_bytes_w4.restype = sz
    L.cp_spec_init_w4.argtypes = [vp, vp, vp, vp, vp, vp, sz, C.POINTER(vp)]
    L.cp_spec_kv_plan.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]
    L.cp_spec_rope_init.argtypes = [vp, i32, C.c_double, i32, vp, i32]
    L.cp_spec_rope_rows.argtypes = [vp, i32, i32, i32, vp, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp, i64, vp]
    L.cp_spec_kv16_bytes.argtypes = [vp]
    L.cp_spec_kv16_bytes.restype = sz
    L.cp_spec_kv16_append.argtypes = [vp, vp, i32, vp, vp, i64, vp, i64, vp, vp, i64, i32, vp, i64, vp, i64, vp]
    L.cp_spec_kv16_attention.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, f32, vp, i64, vp, i64, vp, vp,
                                         sz, vp, vp]
    L.cp_spec_kv16_attention_bytes.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, i32]
    L.cp_spec_kv16_attention_bytes.restype = sz
    L.cp_spec_status_word.argtypes = [vp, vp]
    L.cp_spec_test_hooks.argtypes = [vp, u64, i32]
    L.cp_spec_read_stats.argtypes = [vp, vp, vp]
    L.cp_spec_reset_stats.argtypes = [vp, vp]
    L.cp_spec_launch_count.argtypes = [vp]
    L.cp_spec_launch_count.restype = C.c_int64
    L.cp_spec_last_error.argtypes = [vp]
    L.cp_spec_last_error.restype = C.c_char_p
    L.cp_spec_destroy.argtypes = [vp]
    L.cp_spec_destroy.restype = None
    for name in ("cp_spec_init", "cp_spec_init_tree", "cp_spec_set_stream_sampling", "cp_spec_decode_frames", "cp_spec_begin_frame",
                 "cp_spec_round", "cp_spec_teacher_logits", "cp_spec_accept_batch", "cp_spec_status_word",
                 "cp_spec_read_stats", "cp_spec_reset_stats", "cp_spec_decode_frames_static", "cp_spec_test_hooks", "cp_spec_w4_pack",
                 "cp_spec_w4_unpack", "cp_spec_w4_gemv", "cp_spec_kv4_append", "cp_spec_kv4_read",
                 "cp_spec_kv4_attention", "cp_spec_init_w4", "cp_spec_kv_plan", "cp_spec_rope_init", "cp_spec_rope_rows",
                 "cp_spec_kv16_append", "cp_spec_kv16_attention"):
        getattr(L, name).restype = C.c_int
    _lib = L
    return L


def _check(rc: int, ctx=None, allow=(OK,)):
    if rc in allow:
        return rc
    msg = load().cp_spec_last_error(ctx).decode(errors="replace")
    raise CpSpecError(rc, msg)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream():
    import torch
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def model_struct(spec: synth.ModelSpec) -> Model:
    return Model(spec.hidden, spec.n_layers, spec.n_q_heads, spec.n_kv_heads, spec.head_dim, spec.ffn, spec.vocab,
                 spec.num_code_groups, spec.dtype, spec.rope_theta, spec.rms_eps)


def weights_to_device(spec: synth.ModelSpec, w: dict, device="cuda") -> dict:
    """Copy numpy weights (float32, or uint16 bf16 bits) to device tensors of the storage dtype."""
    import torch

    def dev(a):
        a = np.ascontiguousarray(a)
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
        return torch.from_numpy(a).to(device)

    out = {k: dev(w[k]) for k in ("embed", "lm_head", "final_norm")}
    out["layers"] = [{k: dev(v) for k, v in lw.items()} for lw in w["layers"]]
    if w.get("draft_offset") is not None and len(w["draft_offset"]) > 0:
        out["draft_offset"] = dev(np.asarray(w["draft_offset"], np.float32).reshape(-1, spec.hidden))
    return out


def pack_weights(spec: synth.ModelSpec, dw: dict, group: int = 32) -> dict:
    """Device weights with every matrix packed to 4 bits (W4Matrix), for CpSpec (cp_spec_init_w4)."""
    out = dict(dw, w4_group=group)
    out["lm_head"] = w4_pack(dw["lm_head"].view(-1, spec.hidden), group)
    out["layers"] = [{k: v if k.endswith("norm") else w4_pack(v, group) for k, v in lw.items()} for lw in dw["layers"]]
    return out


def n_draft_offsets(dw: dict) -> int:
    """K of the position-aware draft offsets held in device weights (0 if none)."""
    off = dw.get("draft_offset")
    return 0 if off is None else int(off.shape[0])


def weights_struct(dw: dict, packed: bool = False) -> Weights:
    """The pointers of device weights; packed: every matrix but embed is a W4Matrix (cp_spec_init_w4), else none is."""
    def matrix(m):
        if isinstance(m, W4Matrix) != packed:
            raise CpSpecError(E_INVALID, "plain matrices among packed weights" if packed else
                              "packed 4-bit matrices where plain ones are wanted")
        return _ptr(m.data if packed else m)

    ws = Weights()
    ws.embed, ws.lm_head, ws.final_norm = _ptr(dw["embed"]), matrix(dw["lm_head"]), _ptr(dw["final_norm"])
    for l, lw in enumerate(dw["layers"]):
        for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down"):
            getattr(ws, n)[l] = _ptr(lw[n]) if n.endswith("norm") else matrix(lw[n])
    ws.draft_offset = _ptr(dw.get("draft_offset"))
    return ws


def _check_packed(spec: synth.ModelSpec, dw: dict, group: int):
    """Refuses packed matrices that do not have the model's shapes, the context's group and all their bytes."""
    H, F, qd, kvd = spec.hidden, spec.ffn, spec.n_q_heads * spec.head_dim, spec.n_kv_heads * spec.head_dim
    shapes = {"wq": (qd, H), "wk": (kvd, H), "wv": (kvd, H), "wo": (H, qd), "w_gate": (F, H), "w_up": (F, H), "w_down": (H, F)}
    named = [("lm_head", dw["lm_head"], ((spec.num_code_groups - 1) * spec.vocab, H))]
    named += [(f"layer {l} {n}", lw[n], shape) for l, lw in enumerate(dw["layers"]) for n, shape in shapes.items()]
    for name, m, (n, k) in named:
        if (m.n, m.k, m.group) != (n, k, group):
            raise CpSpecError(E_INVALID, f"{name}: [{m.n}, {m.k}] in groups of {m.group}, [{n}, {k}] in groups of {group} wanted")
    for name, m, _ in named:
        if m.data.numel() < load().cp_spec_w4_bytes(m.n, m.k, m.group):
            raise CpSpecError(E_INVALID, f"{name}: fewer bytes than a packed matrix of its shape has")


class CpSpec:
    """One context of the CUDA library over device-resident weights."""

    def __init__(self, spec: synth.ModelSpec, device_weights: dict, verify_window: int, top_k: int,
                 temperature: float, seed: int, max_streams: int = 1, adapt_pct: int = 0, adapt_min: int = 16,
                 tree=None, kv_bits: int = 32):
        """tree: None (chain rounds of verify_window), or (parent, rank) sequences of a sparse
        draft tree (cp_spec_init_tree; verify_window and the adaptive window are then ignored).
        device_weights from pack_weights make a context over 4-bit weights (cp_spec_init_w4), with
        kv_bits = 4 its KV cache in 4 bits too."""
        import numpy as np
        import torch
        self.lib = load()
        self.spec = spec
        self.dw = device_weights
        self.model = model_struct(spec)
        self.weights = weights_struct(device_weights, packed=bool(device_weights.get("w4_group")))
        self.config = Config(verify_window, top_k, temperature, seed, max_streams, n_draft_offsets(device_weights),
                             adapt_pct, adapt_min)
        self.tree = None
        group = device_weights.get("w4_group")
        self.quant = Quant(group, kv_bits) if group else None
        if group:
            _check_packed(spec, device_weights, group)
        if group is None and kv_bits != 32:
            raise CpSpecError(E_INVALID, "a 4-bit KV cache needs packed weights (pack_weights)")
        if tree is not None:
            par = np.ascontiguousarray(tree[0], dtype=np.int32)
            rk = np.ascontiguousarray(tree[1], dtype=np.int32)
            self._tree_arrays = (par, rk)  # kept alive for the call
            self.tree = Tree(len(par), par.ctypes.data, rk.ctypes.data)
        tree_ref = None if self.tree is None else C.byref(self.tree)
        if self.quant is not None:
            nbytes = self.lib.cp_spec_workspace_bytes_w4(C.byref(self.model), C.byref(self.config), tree_ref,
                                                         C.byref(self.quant))
        elif self.tree is not None:
            nbytes = self.lib.cp_spec_workspace_bytes_tree(C.byref(self.model), C.byref(self.config),
                                                           C.byref(self.tree))
        else:
            nbytes = self.lib.cp_spec_workspace_bytes(C.byref(self.model), C.byref(self.config))
        if nbytes == 0:
            _check(E_INVALID)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        ctx = C.c_void_p()
        if self.quant is not None:
            rc = self.lib.cp_spec_init_w4(C.byref(self.model), C.byref(self.weights), C.byref(self.config), tree_ref,
                                          C.byref(self.quant), C.c_void_p(_ptr(self.workspace)), nbytes, C.byref(ctx))
        elif self.tree is not None:
            rc = self.lib.cp_spec_init_tree(C.byref(self.model), C.byref(self.weights), C.byref(self.config),
                                            C.byref(self.tree), C.c_void_p(_ptr(self.workspace)), nbytes,
                                            C.byref(ctx))
        else:
            rc = self.lib.cp_spec_init(C.byref(self.model), C.byref(self.weights), C.byref(self.config),
                                       C.c_void_p(_ptr(self.workspace)), nbytes, C.byref(ctx))
        _check(rc, None, allow=(OK, W_AR_FALLBACK))
        self.ar_fallback = rc == W_AR_FALLBACK
        self.ctx = ctx

    def close(self):
        if getattr(self, "ctx", None):
            self.lib.cp_spec_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_stream_sampling(self, top_k, temperature):
        tk = np.ascontiguousarray(top_k, dtype=np.int32)
        tp = np.ascontiguousarray(temperature, dtype=np.float32)
        _check(self.lib.cp_spec_set_stream_sampling(self.ctx, tk.size, tk.ctypes.data_as(C.c_void_p),
                                                    tp.ctypes.data_as(C.c_void_p)), self.ctx)

    def decode_frames(self, x, c0, codes=None, first_frame: int = 0):
        """x [F, B, H] float32 cuda, c0 [F, B] int32 cuda -> codes [F, B, G] int32 (asynchronous)."""
        import torch
        F, B, _ = x.shape
        if codes is None:
            codes = torch.empty((F, B, self.spec.num_code_groups), dtype=torch.int32, device=x.device)
        _check(self.lib.cp_spec_decode_frames(self.ctx, B, F, first_frame, _ptr(x), _ptr(c0), _ptr(codes), _stream()),
               self.ctx)
        return codes

    def begin_frame(self, x, c0, frame_idx: int):
        _check(self.lib.cp_spec_begin_frame(self.ctx, x.shape[0], _ptr(x), _ptr(c0), frame_idx, _stream()), self.ctx)

    def round(self, codes, committed=None):
        _check(self.lib.cp_spec_round(self.ctx, _ptr(codes), _ptr(committed), _stream()), self.ctx)

    def teacher_logits(self, x, codes, P: int, draft: bool = False):
        import torch
        B = x.shape[0]
        V = self.spec.vocab
        lg = torch.empty((B, P - 1, V), dtype=torch.float32, device=x.device)
        nd = self.config.verify_window - 1
        dl = torch.empty((B, P - 1, nd, V), dtype=torch.float32, device=x.device) if draft else None
        _check(self.lib.cp_spec_teacher_logits(self.ctx, B, P, _ptr(x), _ptr(codes), _ptr(lg), _ptr(dl), _stream()),
               self.ctx)
        return lg, dl

    def status(self):
        _check(self.lib.cp_spec_status_word(self.ctx, _stream()), self.ctx)

    def status_code(self) -> int:
        """cp_spec_status_word as a code (clears the word)."""
        return int(self.lib.cp_spec_status_word(self.ctx, _stream()))

    def test_hooks(self, wait_limit_ns: int = 2_000_000_000, stall_first_wait: bool = False, poison_kv: bool = False):
        flags = (1 if stall_first_wait else 0) | (2 if poison_kv else 0)
        _check(self.lib.cp_spec_test_hooks(self.ctx, int(wait_limit_ns), flags), self.ctx)

    def stats(self) -> dict:
        st = Stats()
        _check(self.lib.cp_spec_read_stats(self.ctx, C.byref(st), _stream()), self.ctx)
        return st.as_dict()

    def reset_stats(self):
        _check(self.lib.cp_spec_reset_stats(self.ctx, _stream()), self.ctx)

    def launch_count(self) -> int:
        return int(self.lib.cp_spec_launch_count(self.ctx))


def accept_batch(target, draft, top_k: int, temperature: float, seed: int, mode: int = 0, want_drafts=True):
    """Acceptance kernels alone.  target [R, N, V], draft [R, N-1, V] float32 cuda tensors."""
    import torch
    lib = load()
    R, N, V = target.shape
    tok = torch.empty((R, N), dtype=torch.int32, device=target.device)
    na = torch.empty((R,), dtype=torch.int32, device=target.device)
    dr = torch.empty((R, N - 1), dtype=torch.int32, device=target.device) if want_drafts else None
    _check(lib.cp_spec_accept_batch(R, N, V, top_k, temperature, seed, mode, _ptr(target), _ptr(draft), _ptr(tok),
                                    _ptr(na), _ptr(dr), _stream()))
    return tok, na, dr


def decode_frames_static(spec: synth.ModelSpec, device_weights: dict, verify_window: int, top_k: int,
                         temperature: float, seed: int, x, c0, codes=None, first_frame: int = 0, max_streams=None,
                         status=None):
    """cp_spec_decode_frames_static: one decode in the library's static scratch, no context (no packed weights).

    x [F, B, H] float32 cuda, c0 [F, B] int32 cuda -> codes [F, B, G] int32 (asynchronous).
    status (optional) is a 1-element int32 cuda tensor that receives the device status word.
    Returns (codes, rc) with rc OK or W_AR_FALLBACK."""
    import torch
    weights = weights_struct(device_weights)
    lib = load()
    F, B, _ = x.shape
    if codes is None:
        codes = torch.empty((F, B, spec.num_code_groups), dtype=torch.int32, device=x.device)
    model = model_struct(spec)
    config = Config(verify_window, top_k, temperature, seed, B if max_streams is None else max_streams,
                    n_draft_offsets(device_weights))
    rc = lib.cp_spec_decode_frames_static(C.byref(model), C.byref(weights), C.byref(config), B, F, first_frame,
                                          _ptr(x), _ptr(c0), _ptr(codes), _ptr(status), _stream())
    _check(rc, None, allow=(OK, W_AR_FALLBACK))
    return codes, rc


# ------------------------------------------------------- 4-bit operators
# These calls take a few microseconds on the device, so what they do here is kept short: no message is built
# unless it is raised, and the stream comes as the raw handle of PyTorch's current stream.
_torch = None
_DTYPES = None  # torch dtype -> element type of the C ABI


def _fast():
    """The library and PyTorch, imported on first use."""
    global _torch, _DTYPES
    if _torch is None:
        import torch
        _DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        _torch = torch
    return _lib or load()


def _refuse(what: str):
    raise CpSpecError(E_INVALID, what)


def _elem_type(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse(f"element type {dtype}: float32, bfloat16 or float16 wanted")
    return code


def _stream_on(dev: int) -> int:
    """Handle of the current stream, after a check that `dev` (Tensor.get_device()) is the current CUDA device."""
    if dev < 0 or dev != _torch._C._cuda_getDevice():
        _refuse(f"tensor on device {dev}: the library runs on the current CUDA device")
    return _torch._C._cuda_getCurrentRawStream(dev)


def _aligned(t, keep: list) -> int:
    """Pointer of a dense tensor; a slice that does not start on 16 bytes is copied, the copy kept for the call."""
    at = t.data_ptr()
    if at & 15:
        t = t.clone()
        keep.append(t)
        at = t.data_ptr()
    return at


def _index(t, n: int, what: str, dev: int, keep: list) -> int:
    """Pointer of a dense int32 tensor of n elements on device dev, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is not _torch.int32 or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        _refuse(f"{what}: {n} dense int32 values beside the cache wanted")
    return _aligned(t, keep)


def _row_stride(t, what: str) -> int:
    """Elements between the rows of t [n_seqs, rows, heads, head_dim]: its last two axes dense, its first two one axis."""
    b, m, h, d = t.shape
    if t.is_contiguous():
        return h * d
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (h > 1 and s2 != d) or (b > 1 and m > 1 and s0 != m * s1):
        _refuse(f"{what}: rows [heads, head_dim] must be dense and evenly spaced")
    return s1 if m > 1 else (s0 if b > 1 else h * d)


class W4Matrix:
    """A weight matrix [n, k] packed by w4_pack (data: the library's own layout)."""

    def __init__(self, n: int, k: int, group: int, data):
        self.n, self.k, self.group, self.data = n, k, group, data


def w4_pack(w, group: int = 32) -> W4Matrix:
    """Quantise w [n, k] (float32, bfloat16 or float16, rows dense) to 4 bits with a scale per `group` columns."""
    lib = _fast()
    if w.dim() == 2 and w.shape[0] > MAX_W4_N:
        _refuse(f"w: {w.shape[0]} rows, at most {MAX_W4_N} wanted")
    if w.dim() != 2 or (w.shape[1] > 1 and w.stride(1) != 1):
        _refuse("w: a matrix with dense rows wanted")
    n, k = w.shape
    code, stream = _elem_type(w.dtype), _stream_on(w.get_device())
    nbytes = lib.cp_spec_w4_bytes(n, k, group)
    if nbytes == 0:
        _check(E_INVALID)
    out = W4Matrix(n, k, group, _torch.empty(nbytes, dtype=_torch.uint8, device=w.device))
    _check(lib.cp_spec_w4_pack(n, k, group, code, w.data_ptr(), w.stride(0) if n > 1 else k, out.data.data_ptr(), stream))
    return out


def w4_unpack(w: W4Matrix, dtype=None):
    """The values [n, k] that a packed matrix stands for (float32 unless dtype says otherwise)."""
    lib = _fast()
    stream = _stream_on(w.data.get_device())
    out = _torch.empty((w.n, w.k), dtype=dtype or _torch.float32, device=w.data.device)
    _check(lib.cp_spec_w4_unpack(w.n, w.k, w.group, _elem_type(out.dtype), w.data.data_ptr(), out.data_ptr(), stream))
    return out


def w4_gemv(x, w: W4Matrix, out=None, out_dtype=None):
    """x [rows, k] times the packed matrix: [rows, n] of x's type (or float32; asynchronous)."""
    lib = _lib if _torch is not None and _lib is not None else _fast()
    n, k, dt, dev, shape, st = w.n, w.k, x.dtype, x.get_device(), x.shape, x.stride()
    if len(shape) != 2 or shape[1] != k or (st[1] != 1 and k > 1):
        _refuse(f"x: [rows, {k}] with dense rows wanted")
    rows = shape[0]
    if rows > 65535:
        _refuse(f"x: {rows} rows, at most 65535 wanted")
    code, stream = _elem_type(dt), _stream_on(dev)
    if w.data.get_device() != dev:
        _refuse("x and the packed matrix on one device wanted")
    if out is None:
        out_dtype = out_dtype or dt
        out = _torch.empty((rows, n), dtype=out_dtype, device=x.device)
        ys = n
    else:
        if (tuple(out.shape) != (rows, n) or (n > 1 and out.stride(1) != 1) or out.get_device() != dev
                or (out_dtype is not None and out.dtype is not out_dtype)):
            _refuse(f"out: [{rows}, {n}] with dense rows beside x wanted")
        out_dtype = out.dtype
        ys = out.stride(0) if rows > 1 else n
    rc = lib.cp_spec_w4_gemv(rows, n, k, w.group, code, code if out_dtype is dt else _elem_type(out_dtype), x.data_ptr(),
                             st[0] if rows > 1 else k, w.data.data_ptr(), out.data_ptr(), ys, stream)
    if rc:
        _check(rc)
    return out


class Kv4Cache:
    """Keys and values held in 4 bits, in n_pages pages of page_size token slots.

    pages (int32 [n_seqs, max_pages]) maps the positions of each sequence to pages; without it
    sequence b owns n_pages // n_seqs neighbouring pages.  The memory starts as zeros.  Slices of tables,
    positions, lengths and masks may start anywhere; rows of keys, values and queries start on 16 bytes."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda"):
        lib = _fast()
        if max(n_pages, page_size, n_kv_heads, head_dim) > 0x7FFFFFFF:
            _refuse("sizes of 31 bits wanted")
        self.shape = Kv4(n_pages, page_size, n_kv_heads, head_dim)
        self._shape = C.addressof(self.shape)
        nbytes = lib.cp_spec_kv4_bytes(self._shape)
        if nbytes == 0:
            _check(E_INVALID)
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = n_pages, page_size, n_kv_heads, head_dim
        self.data = _torch.zeros(nbytes, dtype=_torch.uint8, device=device)

    def _pages(self, pages, n_seqs: int, dev: int, keep: list):
        """Pointer of the page table and pages per sequence."""
        if pages is None:
            return 0, self.n_pages // max(n_seqs, 1)
        if pages.dim() != 2 or pages.shape[0] != n_seqs:
            _refuse(f"pages: [{n_seqs}, max_pages] wanted")
        return _index(pages, pages.numel(), "pages", dev, keep), pages.shape[1]

    def append(self, k, v, pos, pages=None, n_rows=None):
        """Write rows k, v [n_seqs, rows, n_kv_heads, head_dim]: row i of sequence b at position pos[b] + i (i < n_rows[b])."""
        lib, data = _fast(), self.data
        shape, dev, dt = k.shape, data.get_device(), k.dtype
        if (len(shape) != 4 or shape != v.shape or dt is not v.dtype or shape[2] != self.n_kv_heads
                or shape[3] != self.head_dim or k.get_device() != dev or v.get_device() != dev):
            _refuse(f"k, v: [n_seqs, rows, {self.n_kv_heads}, {self.head_dim}] of one type beside the cache wanted")
        b = shape[0]
        code, stream = _elem_type(dt), _stream_on(dev)
        keep = []
        table, per = self._pages(pages, b, dev, keep)
        rc = lib.cp_spec_kv4_append(self._shape, data.data_ptr(), table, per, b, shape[1], _index(pos, b, "pos", dev, keep),
                                    _index(n_rows, b, "n_rows", dev, keep), code, k.data_ptr(), _row_stride(k, "k"), v.data_ptr(),
                                    _row_stride(v, "v"), stream)
        if rc:
            _check(rc)

    def read(self, length: int, pages=None, lens=None, n_seqs=None, dtype=None):
        """Keys and values of positions 0 .. length - 1: two tensors [n_seqs, length, n_kv_heads, head_dim].

        Positions at or past lens[b] read as zeros."""
        lib, data = _fast(), self.data
        dev = data.get_device()
        stream = _stream_on(dev)
        b = n_seqs if n_seqs is not None else (pages.shape[0] if pages is not None else 1)
        keep = []
        table, per = self._pages(pages, b, dev, keep)
        dtype = dtype or _torch.float32
        size, code = (b, length, self.n_kv_heads, self.head_dim), _elem_type(dtype)
        k, v = _torch.empty(size, dtype=dtype, device=data.device), _torch.empty(size, dtype=dtype, device=data.device)
        rc = lib.cp_spec_kv4_read(self._shape, data.data_ptr(), table, per, b, length, _index(lens, b, "lens", dev, keep), code,
                                  k.data_ptr(), v.data_ptr(), stream)
        if rc:
            _check(rc)
        return k, v

    def attention(self, q, kv_len, pages=None, n_rows=None, mask=None, scale=None, out=None, want_lse=False):
        """Attention of q [n_seqs, rows, n_q_heads, head_dim] over the cache (see cp_spec_kv4_attention).

        kv_len int32 [n_seqs] counts the window's own rows, mask int64 [n_seqs, rows] holds the bits of the window
        rows that a row sees (None: causal), scale is head_dim ** -0.5 unless given.  Returns the output, and with
        want_lse also the log of the sums of exponentials [n_seqs, rows, n_q_heads] (rows past n_rows[b] are not written)."""
        lib, data = _fast(), self.data
        shape, dev, dt = q.shape, data.get_device(), q.dtype
        if len(shape) != 4 or shape[3] != self.head_dim or q.get_device() != dev:
            _refuse(f"q: [n_seqs, rows, n_q_heads, {self.head_dim}] beside the cache wanted")
        b, m, nq, d = shape
        code, stream = _elem_type(dt), _stream_on(dev)
        if out is None:
            out = _torch.empty(shape, dtype=dt, device=data.device)
            os = nq * d
        else:
            if out.shape != shape or out.dtype is not dt or out.get_device() != dev:
                _refuse("out: q's shape, type and device wanted")
            os = _row_stride(out, "out")
        bits, keep = 0, []
        if mask is not None:
            if (mask.dtype is not _torch.int64 or tuple(mask.shape) != (b, m) or not mask.is_contiguous()
                    or mask.get_device() != dev):
                _refuse(f"mask: dense int64 [{b}, {m}] wanted")
            bits = _aligned(mask, keep)
        lse = _torch.empty((b, m, nq), dtype=_torch.float32, device=data.device) if want_lse else None
        table, per = self._pages(pages, b, dev, keep)
        need = lib.cp_spec_kv4_attention_bytes(self._shape, per, b, m, nq, code)
        work = _torch.empty(need, dtype=_torch.uint8, device=data.device) if need else None  # (freed in stream order)
        rc = lib.cp_spec_kv4_attention(self._shape, data.data_ptr(), table, per, b, m, nq, _index(kv_len, b, "kv_len", dev, keep),
                                       _index(n_rows, b, "n_rows", dev, keep), bits, d ** -0.5 if scale is None else scale, code,
                                       q.data_ptr(), _row_stride(q, "q"), out.data_ptr(), os,
                                       lse.data_ptr() if want_lse else 0, work.data_ptr() if need else 0, need, stream)
        if rc:
            _check(rc)
        return (out, lse) if want_lse else out


# ------------------------------------------- 16-bit paged KV cache
def kv16_test_hooks(wait_limit_ns: int = 2_000_000_000, stall: int = 0):
    """Diagnostics of Kv16Cache.attention, for the whole process (cp_spec_test_hooks without a context).

    stall 1: the last copy of every CTA is not made, 2: none is; the waits for it run out after wait_limit_ns."""
    _check(_fast().cp_spec_test_hooks(None, int(wait_limit_ns), stall))


class PlanRows:
    """What a step of a PagePool gives: kv_len, refused [n_seqs], row_start [n_seqs + 1], pos, slot [n_rows].

    All lie in one tensor (int32; slot as int64 in front); the views are made where they are asked for."""

    __slots__ = ("_all", "_n", "_rows", "_at")

    def __init__(self, whole, n_seqs, n_rows, at):
        self._all, self._n, self._rows, self._at = whole, n_seqs, n_rows, at

    slot = property(lambda r: r._all[: 2 * r._rows].view(_torch.int64))
    kv_len = property(lambda r: r._all[r._at[0]: r._at[0] + r._n])
    refused = property(lambda r: r._all[r._at[1]: r._at[1] + r._n])
    row_start = property(lambda r: r._all[r._at[2]: r._at[2] + r._n + 1])
    pos = property(lambda r: r._all[r._at[3]: r._at[3] + r._rows])


class PagePool:
    """The pages of a cache and the page tables of n_seqs sequences, kept on the device (see cp_spec_kv_plan).

    pages int32 [n_seqs, max_pages] (-1: none), held int32 [n_seqs], free int32 [n_pages] with n_free int32 [1] are the
    state; a new pool has all pages free, page 0 on top."""

    def __init__(self, n_pages: int, page_size: int, n_seqs: int, max_pages: int, device="cuda"):
        _fast()
        if not 1 <= n_seqs <= MAX_PLAN_SEQS:
            _refuse(f"n_seqs: 1 to {MAX_PLAN_SEQS} wanted")
        if page_size < 16 or page_size % 16 or page_size > 1 << 20:
            _refuse("page_size: a multiple of 16 in [16, 2^20] wanted")
        if not 1 <= n_pages <= 0x7FFFFFFF or max_pages < 1 or max(max_pages * page_size, n_seqs * max_pages) > 0x7FFFFFFF:
            _refuse("n_pages, max_pages >= 1, with max_pages * page_size and n_seqs * max_pages below 2^31 wanted")
        self.n_pages, self.page_size, self.n_seqs, self.max_pages = n_pages, page_size, n_seqs, max_pages
        new = dict(dtype=_torch.int32, device=device)
        self.pages = _torch.full((n_seqs, max_pages), -1, **new)
        self.held = _torch.zeros(n_seqs, **new)
        self.free = _torch.arange(n_pages - 1, -1, -1, **new)
        self.n_free = _torch.full((1,), n_pages, **new)

    def plan(self, length, new=None, n_rows: int = 0) -> PlanRows:
        """One step: every sequence keeps length[b] tokens and adds new[b] rows (int32 [n_seqs]; new None: no rows).

        n_rows is the room for the rows of all sequences; rows past them get position 0 and slot -1."""
        lib, n, table = _fast(), self.n_seqs, self.pages
        dev = table.get_device()
        stream = _stream_on(dev)
        if not 0 <= n_rows <= 0x7FFFFFFF:
            _refuse("n_rows: 31 bits wanted")
        keep = []
        if length is None:
            _refuse("length: the tokens that each sequence keeps wanted")
        len_at, new_at = _index(length, n, "length", dev, keep), _index(new, n, "new", dev, keep)
        # one allocation for all results, each on 16 bytes: slots, lengths, reasons, starts, positions
        a = (2 * n_rows + 3) & -4
        b = a + ((n + 3) & -4)
        c = b + ((n + 3) & -4)
        d = c + ((n + 4) & -4)
        out = _torch.empty(d + n_rows, dtype=_torch.int32, device=table.device)
        at = out.data_ptr()
        rc = lib.cp_spec_kv_plan(n, self.max_pages, self.page_size, self.n_pages, len_at, new_at, table.data_ptr(), self.held.data_ptr(),
                                 self.free.data_ptr(), self.n_free.data_ptr(), n_rows, at + 4 * a, at + 4 * c, at + 4 * d, at, at + 4 * b,
                                 stream)
        if rc:
            _check(rc)
        return PlanRows(out, n, n_rows, (a, b, c, d))


def _row_heads(t, dim, what: str, dev: int) -> int:
    """Row stride of t [n_rows, heads, dim]: rows dense, evenly spaced, on device dev."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or t.get_device() != dev:
        _refuse(f"{what}: [n_rows, heads, {dim}] beside the other tensors wanted")
    if t.is_contiguous():
        return shape[1] * dim
    m, h, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != d) or (m > 1 and s0 < h * d):
        _refuse(f"{what}: dense, evenly spaced rows wanted")
    return s0 if m > 1 else h * d


class Rope:
    """A rotary embedding over one or several position axes (see cp_spec_rope_init).

    sections: pairs of each axis (None: one axis); interleaved: the axes take turns pair by pair.  Pair i has the frequency
    theta^(-2 i / rot_dim) whatever its axis; other ones are set in struct.turns (turns a position, times 2^64)."""

    def __init__(self, rot_dim: int, theta: float, sections=None, interleaved: bool = False):
        lib = _fast()
        sections = [rot_dim // 2] if sections is None else [int(x) for x in sections]
        if not 1 <= len(sections) <= 4 or max(map(abs, sections)) > 0x7FFFFFFF or abs(rot_dim) > 0x7FFFFFFF:
            _refuse("sections: one to four numbers of pairs wanted")
        self.struct = RopeStruct()
        self._struct = C.addressof(self.struct)
        self.rot_dim, self.n_axes = rot_dim, len(sections)
        _check(lib.cp_spec_rope_init(self._struct, rot_dim, theta, len(sections), (C.c_int32 * len(sections))(*sections),
                                     int(interleaved)))

    def _pos(self, pos, n_rows: int, dev: int, keep: list):
        """Pointer and axis stride of pos: int32 [n_rows] (for all axes) or [n_axes, n_rows]."""
        shape = pos.shape
        each = len(shape) == 2
        if not (shape[0] == self.n_axes and shape[1] == n_rows if each else len(shape) == 1 and shape[0] == n_rows):
            _refuse(f"pos: [{n_rows}] or [{self.n_axes}, {n_rows}] wanted")
        return _index(pos, self.n_axes * n_rows if each else n_rows, "pos", dev, keep), n_rows if each else 0

    def rotate(self, q, k, pos, out=None):
        """q [n_rows, heads, dim] and k [n_rows, k heads, dim] (or None) rotated: new tensors, or those of out (a pair)."""
        lib = _lib or _fast()
        shape, dt = q.shape, q.dtype
        if len(shape) != 3:
            _refuse("q: [n_rows, heads, dim] wanted")
        dev = q.get_device()
        m, nq, d = shape
        if m > MAX_KV16_ROWS:
            _refuse(f"q: {m} rows, at most {MAX_KV16_ROWS} wanted")
        code, stream, keep = _elem_type(dt), _stream_on(dev), []
        if k is not None and (k.dtype is not dt or k.dim() != 3 or k.shape[0] != m):
            _refuse("q, k and out: rows of one number and type wanted")
        nk = k_at = ks = ko_at = kos = 0
        if out is None:
            qo, qos = _torch.empty((m, nq, d), dtype=dt, device=q.device), nq * d
            ko = None
        else:
            qo, ko = out
            if qo.shape != shape or qo.dtype is not dt or (k is None) != (ko is None):
                _refuse("out: the shapes and type of q and k wanted")
            qos = _row_heads(qo, d, "out", dev)
        if k is not None:
            ks, nk = _row_heads(k, d, "k", dev), k.shape[1]
            if ko is None:
                ko, kos = _torch.empty((m, nk, d), dtype=dt, device=q.device), nk * d
            elif ko.shape != k.shape or ko.dtype is not dt:
                _refuse("out: the shapes and type of q and k wanted")
            else:
                kos = _row_heads(ko, d, "out", dev)
            k_at, ko_at = k.data_ptr(), ko.data_ptr()
        at, stride = self._pos(pos, m, dev, keep)
        rc = lib.cp_spec_rope_rows(self._struct, m, d, code, at, stride, nq, q.data_ptr(), _row_heads(q, d, "q", dev), qo.data_ptr(), qos,
                                   nk, k_at, ks, ko_at, kos, stream)
        if rc:
            _check(rc)
        return qo, ko


class Kv16Cache:
    """Keys and values in bfloat16 or float16, in n_pages pages of page_size token slots (see cp_spec_kv16).

    keys and values are views [n_pages, n_kv_heads, page_size, head_dim] of the memory, which starts as zeros."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=None, device="cuda"):
        lib = _fast()
        dtype = dtype or _torch.bfloat16
        if max(map(abs, (n_pages, page_size, n_kv_heads, head_dim))) > 0x7FFFFFFF:
            _refuse("sizes of 31 bits wanted")
        self.shape = Kv16(n_pages, page_size, n_kv_heads, head_dim, _elem_type(dtype))
        self._shape = C.addressof(self.shape)
        if lib.cp_spec_kv16_bytes(self._shape) == 0:
            _check(E_INVALID)
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, self.dtype = n_pages, page_size, n_kv_heads, head_dim, dtype
        self.data = _torch.zeros((2, n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=device)
        self.keys, self.values = self.data[0], self.data[1]

    def append(self, k, v, slot, rope: Rope = None, pos=None, q=None, q_out=None):
        """Write rows k, v [n_rows, n_kv_heads, head_dim] to slots slot [n_rows] (int64; outside the cache: left out).

        With rope the keys are rotated by pos (see Rope.rotate) as they are written, and queries q [n_rows, heads,
        head_dim] into q_out (a new tensor unless given; rows whose slot is outside the cache are not written), which is
        returned."""
        lib, data, d, dt, shape = _lib or _fast(), self.data, self.head_dim, self.dtype, k.shape
        dev = data.get_device()
        if len(shape) != 3 or shape != v.shape or shape[1] != self.n_kv_heads or k.dtype is not dt or v.dtype is not dt:
            _refuse(f"k, v: [n_rows, {self.n_kv_heads}, {d}] of the cache's type wanted")
        m = shape[0]
        if m > MAX_KV16_ROWS:
            _refuse(f"k: {m} rows, at most {MAX_KV16_ROWS} wanted")
        stream, keep = _stream_on(dev), []
        if slot.dtype is not _torch.int64 or slot.numel() != m or not slot.is_contiguous() or slot.get_device() != dev:
            _refuse(f"slot: {m} dense int64 values beside the cache wanted")
        turns = at = stride = nq = qs = qos = q_at = out_at = 0
        if rope is not None and pos is not None:
            turns = rope._struct
            at, stride = rope._pos(pos, m, dev, keep)
        elif rope is not None or pos is not None or q is not None:
            _refuse("rope and pos together, and q only with them wanted")
        if q is not None:
            if q.dtype is not dt or q.dim() != 3 or q.shape[0] != m:
                _refuse(f"q: [{m}, heads, {d}] of the cache's type wanted")
            qs, nq = _row_heads(q, d, "q", dev), q.shape[1]
            if q_out is None:
                q_out, qos = _torch.empty((m, nq, d), dtype=dt, device=data.device), nq * d
            elif q_out.shape != q.shape or q_out.dtype is not dt:
                _refuse("q_out: q's shape and type wanted")
            else:
                qos = _row_heads(q_out, d, "q_out", dev)
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            _refuse("q_out only with q wanted")
        rc = lib.cp_spec_kv16_append(self._shape, data.data_ptr(), m, _aligned(slot, keep), k.data_ptr(), _row_heads(k, d, "k", dev),
                                     v.data_ptr(), _row_heads(v, d, "v", dev), turns, at, stride, nq, q_at, qs, out_at, qos, stream)
        if rc:
            _check(rc)
        return q_out

    def attention(self, q, kv_len, row_start, pages=None, max_rows=None, window: int = 0, sinks: int = 0, mask=None, scale=None,
                  out=None, want_lse: bool = False, status=None):
        """Attention of packed rows q [n_rows, heads, head_dim] over the cache (see cp_spec_kv16_attention).

        kv_len int32 [n_seqs] counts a sequence's own rows, which are row_start[b] .. row_start[b + 1] - 1 (int32
        [n_seqs + 1]), at most max_rows of them: give it for batches, where the most rows of a sequence are far fewer than
        n_rows, which is taken otherwise.  window and sinks: each row sees the last `window` positions and the first `sinks`
        (window 0: all).  mask int64 [n_rows]: trees of up to 64 rows (max_rows 64 unless given), the bits of the sequence's
        rows that a row sees.  status (int32, one element): set to E_DEVICE_TIMEOUT if a kernel gave up.
        Returns the output and with want_lse also the log of the sums of exponentials [n_rows, heads]; rows past the last
        sequence are not written."""
        lib, data, d, dt, shape = _lib or _fast(), self.data, self.head_dim, self.dtype, q.shape
        dev = data.get_device()
        if q.dtype is not dt:
            _refuse(f"q: [n_rows, heads, {d}] of the cache's type beside it wanted")
        qs = _row_heads(q, d, "q", dev)
        m, nq = shape[0], shape[1]
        if m > MAX_KV16_ROWS:
            _refuse(f"q: {m} rows, at most {MAX_KV16_ROWS} wanted")
        stream, keep, n, where = _stream_on(dev), [], kv_len.numel(), data.device
        if out is None:
            out, os = _torch.empty((m, nq, d), dtype=dt, device=where), nq * d
        elif out.shape != shape or out.dtype is not dt:
            _refuse("out: q's shape and type wanted")
        else:
            os = _row_heads(out, d, "out", dev)
        bits = 0
        if mask is not None:
            if mask.dtype is not _torch.int64 or mask.numel() != m or not mask.is_contiguous() or mask.get_device() != dev:
                _refuse(f"mask: {m} dense int64 values beside the cache wanted")
            bits = _aligned(mask, keep)
        if status is not None and (status.dtype is not _torch.int32 or status.numel() != 1 or status.get_device() != dev):
            _refuse("status: one int32 beside the cache wanted")
        if pages is None:
            table, per = 0, self.n_pages // max(n, 1)
        else:
            shape = pages.shape
            if len(shape) != 2 or shape[0] != n:
                _refuse(f"pages: [{n}, max_pages] wanted")
            per = shape[1]
            table = _index(pages, n * per, "pages", dev, keep)
        most = (m if mask is None else min(m, MAX_TREE_ROWS)) if max_rows is None else max_rows
        if not (0 <= most <= 0x7FFFFFFF and 0 <= window <= 0x7FFFFFFF and 0 <= sinks <= 0x7FFFFFFF):
            _refuse("max_rows, window and sinks of 31 bits wanted")
        need = lib.cp_spec_kv16_attention_bytes(self._shape, per, n, m, most, nq, window, sinks, 0 if mask is None else 1)
        lse = lse_at = work_at = work = None
        if want_lse:
            lse = _torch.empty((m, nq), dtype=_torch.float32, device=where)
            lse_at = lse.data_ptr()
        if need:
            work = _torch.empty(need, dtype=_torch.uint8, device=where)  # (freed in stream order)
            work_at = work.data_ptr()
        rc = lib.cp_spec_kv16_attention(self._shape, data.data_ptr(), table, per, n, m, most, nq, _index(kv_len, n, "kv_len", dev, keep),
                                        _index(row_start, n + 1, "row_start", dev, keep), bits, window, sinks,
                                        d ** -0.5 if scale is None else scale, q.data_ptr(), qs, out.data_ptr(), os, lse_at, work_at,
                                        need, _ptr(status), stream)
        if rc:
            _check(rc)
        return (out, lse) if want_lse else out
