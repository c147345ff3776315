#!/usr/bin/env python3
"""Benchmark: committed RVQ codes/s of the CodePredictor speculative round.

Workload (one step): decode 1000 frames of 1 stream with the bf16
0.6B-class synthetic CodePredictor (hidden 1024, 5 layers, 16 q / 8 kv heads
of 128, SwiGLU 3072, vocab 2048, 16 code groups), verify window N = 4,
top-k 50, temperature 0.9, weights N(0, 0.02) from seed 0, per-frame talker
hidden N(0, 1) and first code uniform.  Inputs are resident in HBM when the
timed region starts; weights (220 MB with the lm_heads) exceed the 129 MB
L2, so no flush is needed between steps.

One JSON line on rank 0.  --impl reference times the CPU oracle (the
reference arm of this build) on a bounded sample of the same workload.
Multi-GPU (torchrun): every rank decodes its own replica of the workload
(streams are independent; no collective on the data path); the timed region
is bracketed by barriers and the maximum over ranks is reported.
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import statistics
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "committed RVQ codes/s (B=1 and batched); verify-pass HBM GB/s vs GB300 peak"
UNIT = "codes/s"
FRAMES = 1000
WINDOW = 4
TOP_K, TEMP, SEED = 50, 0.9, 1
HBM_NOMINAL_GBS = 7900.0  # GB300 HBM3e nominal bandwidth, reported beside the measured peak


def workload_config(spec, frames, n_streams, window):
    return {
        "workload": (f"bf16 0.6B-class CodePredictor (H{spec.hidden}, {spec.n_layers}L, {spec.n_q_heads}q/"
                     f"{spec.n_kv_heads}kv x{spec.head_dim}, FFN{spec.ffn}, V{spec.vocab}, G{spec.num_code_groups}),"
                     f" {n_streams} stream x {frames} frames, N={window}, top-k {TOP_K}, T {TEMP}"),
        "streams": n_streams, "frames": frames, "verify_window": window, "top_k": TOP_K, "temperature": TEMP,
        "weights": "synthetic N(0,0.02) bf16, seed 0", "inputs": "x ~ N(0,1), c0 ~ U[0,V), seed 1",
        "l2": "no flush: weights + lm_heads 220 MB > 129 MB L2",
        "compute": "bf16 weights, fp32 accumulation and activations, fp32 KV cache",
    }


# ------------------------------------------------------------------ clocks
class ClockSampler:
    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,clocks_event_reasons.hw_slowdown,"
              "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
              "clocks_event_reasons.sw_power_cap")

    def __init__(self, index: int):
        self.index = index
        self.rows = []
        self.proc = None

    def __enter__(self):
        try:
            self.proc = subprocess.Popen(["nvidia-smi", "-i", str(self.index), f"--query-gpu={self.FIELDS}",
                                          "--format=csv,noheader,nounits", "-lms", "200"],
                                         stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            self.thread = threading.Thread(target=self._read, daemon=True)
            self.thread.start()
        except (OSError, FileNotFoundError):
            self.proc = None
        return self

    def _read(self):
        for line in self.proc.stdout:
            parts = [p.strip() for p in line.split(",")]
            if len(parts) >= 8:
                self.rows.append(parts)

    def __exit__(self, *a):
        if self.proc:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except subprocess.TimeoutExpired:
                self.proc.kill()

    def summary(self):
        if not self.rows:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["unavailable"]}
        sm = [float(r[0]) for r in self.rows if r[0].replace(".", "").isdigit()]
        mx = [float(r[1]) for r in self.rows if r[1].replace(".", "").isdigit()]
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        reasons = sorted({names[i] for r in self.rows for i in range(4) if r[4 + i].lower() == "active"})
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(mx) if mx else None,
                "reasons": reasons, "samples": len(self.rows)}


# ------------------------------------------------------------------- peaks
def measured_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        d = json.load(open(p))
        return float(d["hbm_gbs"]), "measured"
    return 6800.0, "fallback"


PASS_KERNEL_SOURCES = ("cp_common.cuh", "cp_sampling.cuh", "cp_frame.cuh", "cp_gemv.cuh", "cp_t5.cuh", "cp_pass_kernels.cu")


def kernel_source_hash():
    """Hash of the sources the pass kernels are compiled from."""
    h = hashlib.sha256()
    csrc = os.path.join(ROOT, "speculative_decoding_rvq_gb300", "csrc")
    for fn in PASS_KERNEL_SOURCES:
        h.update(open(os.path.join(csrc, fn), "rb").read())
    return h.hexdigest()[:16]


def recorded_traffic():
    """DRAM bytes per decoder pass (the pass's kernels summed) from the committed ncu
    summary, if it was taken on the current kernel sources (else None).  Every pass
    streams the same weights, so a step's traffic scales with its number of passes."""
    p = os.path.join(ROOT, "profiles", "pass_kernels_traffic.json")
    if not os.path.exists(p):
        return None
    d = json.load(open(p))
    if d.get("kernel_source_hash") != kernel_source_hash():
        return None
    return d.get("dram_bytes_per_pass")


# ------------------------------------------------------------- multi-rank
def job_throughput(units_local: float, ms_local: float, world: int):
    """Whole-job throughput: the units every rank processed over the slowest rank's time.

    Returns (units per second, max ms over ranks).  At world size 1 no process group is used."""
    if world <= 1:
        return units_local / (ms_local / 1e3), ms_local
    import torch
    import torch.distributed as dist
    dev = "cuda" if dist.get_backend() == "nccl" else "cpu"
    u = torch.tensor([units_local], dtype=torch.float64, device=dev)
    t = torch.tensor([ms_local], dtype=torch.float64, device=dev)
    dist.all_reduce(u, op=dist.ReduceOp.SUM)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(u.item()) / (float(t.item()) / 1e3), float(t.item())


# ------------------------------------------------------------------ GPU arm
def run_gpu(args, rank, world):
    import numpy as np
    import torch

    from speculative_decoding_rvq_gb300 import binding, synth as S

    torch.cuda.set_device(rank % max(torch.cuda.device_count(), 1))
    spec = S.TTS06B_BF16
    w = S.gen_weights(spec, 0)
    dw = binding.weights_to_device(spec, w)
    frames = args.frames
    x, c0 = S.gen_frames(spec, 1, frames, seed=SEED)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    cp = binding.CpSpec(spec, dw, args.window, TOP_K, TEMP, SEED, max_streams=1)
    codes = torch.empty((frames, 1, spec.num_code_groups), dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream()

    def step():
        cp.decode_frames(xd, cd, codes)

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    cp.status()
    cp.reset_stats()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(args.steps)]
    if world > 1:
        torch.distributed.barrier()
    torch.cuda.synchronize()
    with ClockSampler(torch.cuda.current_device()) as clk:
        t0 = torch.cuda.Event(enable_timing=True)
        t1 = torch.cuda.Event(enable_timing=True)
        t0.record(stream)
        for i in range(args.steps):
            ev[i][0].record(stream)
            step()
            ev[i][1].record(stream)
        t1.record(stream)
        torch.cuda.synchronize()
    if world > 1:
        torch.distributed.barrier()
    total_ms = t0.elapsed_time(t1)
    launch_ms = [a.elapsed_time(b) for a, b in ev]
    st = cp.stats()
    cp.status()
    codes_total = args.steps * frames * (spec.num_code_groups - 1)
    value, total_ms = job_throughput(codes_total, total_ms, world)

    peak, peak_kind = measured_peaks()
    per_launch_bytes = (st["weight_bytes"] + st["kv_bytes"]) / args.steps
    mean_launch_s = statistics.mean(launch_ms) / 1e3
    achieved = per_launch_bytes / mean_launch_s / 1e9
    traffic_pp = recorded_traffic()
    passes = st["passes"] / args.steps
    roofline = {"bound": "hbm", "achieved": round(achieved, 1), "peak": peak, "unit": "GB/s",
                "frac": round(achieved / peak, 4), "peak_source": peak_kind,
                "peak_nominal": HBM_NOMINAL_GBS, "frac_nominal": round(achieved / HBM_NOMINAL_GBS, 4),
                "traffic": (round(traffic_pp * passes) if traffic_pp else None),
                "kernel": "verify pass: the call graph's pass kernels (5 per layer + lm_heads, top-k, accept), "
                          "timed per step; GEMV kernels are 21 of the 28 per pass",
                "algorithmic_bytes_per_launch": int(per_launch_bytes),
                "mean_launch_ms": round(statistics.mean(launch_ms), 3)}
    rounds = st["rounds"] / args.steps
    result = {
        "metric": METRIC, "value": round(value, 1), "unit": UNIT, "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": round(total_ms / args.steps, 3), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": dict(workload_config(spec, frames, 1, args.window), parallelism=f"replicas x{world}"),
        "roofline": roofline, "gpu_launches": int(st["kernel_launches"] + args.steps),
        "decode": {"passes_per_frame": round(passes / frames, 3),
                   "codes_per_round": round((frames * (spec.num_code_groups - 2)) / max(rounds, 1), 3),
                   "accepted_by_offset": st["accepted_by_offset"][1:args.window],
                   "drafted_by_offset": st["drafted_by_offset"][1:args.window],
                   "us_per_pass": round(mean_launch_s * 1e6 / passes, 2),
                   "heads_per_pass": round(st["heads_applied"] / st["passes"], 2)},
        "clocks": clk.summary(),
    }

    # end to end through the C ABI with host buffers: pinned H2D of the step's
    # inputs, decode, D2H of the codes, every step
    xh = torch.from_numpy(x).pin_memory()
    ch = torch.from_numpy(c0).pin_memory()
    out_h = torch.empty((frames, 1, spec.num_code_groups), dtype=torch.int32).pin_memory()
    for _ in range(2):
        xd.copy_(xh, non_blocking=True); cd.copy_(ch, non_blocking=True); step()
        out_h.copy_(codes, non_blocking=True)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e_steps = max(2, args.steps // 2)
    e0.record(stream)
    for _ in range(e_steps):
        xd.copy_(xh, non_blocking=True)
        cd.copy_(ch, non_blocking=True)
        step()
        out_h.copy_(codes, non_blocking=True)
    e1.record(stream)
    torch.cuda.synchronize()
    e_ms = e0.elapsed_time(e1)
    result["e2e"] = {"value": round(e_steps * frames * (spec.num_code_groups - 1) / (e_ms / 1e3), 1), "unit": UNIT,
                     "h2d_bytes_per_step": int(xh.numel() * 4 + ch.numel() * 4),
                     "d2h_bytes_per_step": int(out_h.numel() * 4)}

    if rank == 0 and not args.no_sweep:
        result["sweep"] = sweep(cp_factory=lambda n: binding.CpSpec(spec, dw, n, TOP_K, TEMP, SEED, 1),
                                xd=xd, cd=cd, G=spec.num_code_groups, peak=peak)
        result["accept_microbench"] = accept_microbench(peak)
        result["batched"] = batched(spec, dw, peak)
        result["draft_offsets"] = offsets_line(spec, dw, xd[:200], cd[:200], peak)
        result["sparse_tree"] = tree_line(spec, dw, xd[:200], cd[:200], peak)
        result["packed_weights"] = packed_line(spec, dw, xd[:200], cd[:200], peak)
        if not args.no_large:
            result["large"] = large_line(peak)
    return result


def large_line(peak, frames=256):
    """The large model (H 2048, 8 layers, 32 q / 8 kv heads x 64, FFN 6144, V 4096, G 32: 31
    lm_heads of 16.8 MB), T 0.8, top-k 50, `frames` frames per stream: at one stream the AR
    loop, N = 4, and N = 4 with the adaptive window; then N = 4 at 8, 64 and 256 streams
    (tcgen05 GEMV tiles).  One warm-up decode of 4 frames, then the timed decode.  codes/s,
    time per pass and the algorithmic HBM fraction."""
    import torch
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = S.LARGE_BF16
    dw = binding.weights_to_device(spec, S.gen_weights(spec, 0))
    G = spec.num_code_groups
    out = {"model": "H2048, 8L, 32q/8kv x64, FFN6144, V4096, G32, bf16", "frames": frames, "temperature": 0.8}
    # N4_adaptive: the per-stream adaptive window (keep an offset at >= 30 % acceptance,
    # decided after 16 reached drafts)
    for name, n, pct, B in (("N0", 0, 0, 1), ("N4", 4, 0, 1), ("N4_adaptive", 4, 30, 1), ("N4_B8", 4, 0, 8),
                            ("N4_B64", 4, 0, 64), ("N4_B256", 4, 0, 256)):
        F = frames
        x, c0 = S.gen_frames(spec, B, F, seed=SEED)
        xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
        cp = binding.CpSpec(spec, dw, n, TOP_K, 0.8, SEED, B, adapt_pct=pct, adapt_min=16)
        codes = torch.empty((F, B, G), dtype=torch.int32, device="cuda")
        cp.decode_frames(xd[:4], cd[:4], codes[:4])
        torch.cuda.synchronize()
        cp.status()
        cp.reset_stats()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        cp.decode_frames(xd, cd, codes)
        b.record()
        torch.cuda.synchronize()
        cp.status()
        ms = a.elapsed_time(b)
        st = cp.stats()
        out[name] = {"streams": B, "frames": F, "codes_per_s": round(B * F * (G - 1) / (ms / 1e3), 1),
                     "passes_per_frame": round(st["passes"] / F, 3),
                     "us_per_pass": round(ms * 1e3 / st["passes"], 2),
                     "hbm_frac": round((st["weight_bytes"] + st["kv_bytes"]) / (ms / 1e3) / 1e9 / peak, 4)}
        cp.close()
    del dw
    torch.cuda.empty_cache()
    return out


def offsets_line(spec, dw, xd, cd, peak, K=3):
    """N = 4 with K = 3 position-aware draft offsets (synthetic N(0, 0.25^2): the pages'
    trained offsets need speech data) on the sweep's 200 frames: the cost per pass and the
    acceptance by offset, next to the same run without offsets."""
    import torch
    from speculative_decoding_rvq_gb300 import binding, synth as S
    dwo = dict(dw)
    dwo["draft_offset"] = torch.from_numpy(S.gen_draft_offsets(spec, K, seed=1)).cuda()
    out = {"K": K, "offsets": "synthetic N(0, 0.25^2), seed 1"}
    for name, w in (("with_offsets", dwo), ("without", dw)):
        made = []

        def factory(n, w=w):
            made.append(binding.CpSpec(spec, w, n, TOP_K, TEMP, SEED, 1))
            return made[-1]

        r = sweep(factory, xd, cd, spec.num_code_groups, peak, windows=(4,))["N4"]
        r["accepted_by_offset"] = made[-1].last_stats["accepted_by_offset"][1:4]
        out[name] = r
    return out


TREE_SHAPES = {
    # parent, rank per node (parents first): rank r of depth t = the r-th largest draft logit of head_{s+t}
    "chain3": ([-1, 0, 1], [0, 0, 0]),
    "sparse7": ([-1, -1, 0, 0, 1, 2, 3], [0, 1, 0, 1, 0, 0, 0]),
    "wide15": ([-1, -1, -1, 0, 0, 1, 2, 3, 3, 4, 5, 6, 7, 8, 9], [0, 1, 2, 0, 1, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0]),
}


def tree_line(spec, dw, xd, cd, peak):
    """Sparse-tree rounds on the frames of xd (1 stream), top-k 50, T 0.9: per tree shape
    codes/s, passes per frame, time per pass, mean committed codes per round and the
    acceptance by depth."""
    import torch
    from speculative_decoding_rvq_gb300 import binding
    out = {"frames": int(xd.shape[0]), "shapes": {k: {"parent": v[0], "rank": v[1]} for k, v in TREE_SHAPES.items()}}
    G = spec.num_code_groups
    F = xd.shape[0]
    for name, (par, rk) in TREE_SHAPES.items():
        cp = binding.CpSpec(spec, dw, 4, TOP_K, TEMP, SEED, 1, tree=(par, rk))
        codes = torch.empty((F, 1, G), dtype=torch.int32, device="cuda")
        cp.decode_frames(xd[:4], cd[:4], codes[:4])
        torch.cuda.synchronize()
        cp.reset_stats()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        cp.decode_frames(xd, cd, codes)
        b.record()
        torch.cuda.synchronize()
        cp.status()
        ms = a.elapsed_time(b)
        st = cp.stats()
        out[name] = {"nodes": len(par), "codes_per_s": round(F * (G - 1) / (ms / 1e3), 1),
                     "passes_per_frame": round(st["passes"] / F, 3), "us_per_pass": round(ms * 1e3 / st["passes"], 2),
                     "codes_per_round": round((F * (G - 2)) / max(st["rounds"], 1), 3),
                     "accepted_by_depth": st["accepted_by_offset"][1:4],
                     "hbm_frac": round((st["weight_bytes"] + st["kv_bytes"]) / (ms / 1e3) / 1e9 / peak, 4)}
        cp.close()
    return out


def packed_line(spec, dw, xd, cd, peak):
    """The frames of xd (1 stream), top-k 50, T 0.9, over 4-bit weights (scales per 32), the AR loop and N = 4, with
    the float32 KV cache and with the 4-bit one."""
    import torch
    from speculative_decoding_rvq_gb300 import binding
    packed = binding.pack_weights(spec, dw, 32)
    G, F = spec.num_code_groups, xd.shape[0]
    out = {"frames": int(F), "group": 32}
    for name, N, bits in (("AR", 0, 32), ("N4", 4, 32), ("N4_kv4", 4, 4)):
        cp = binding.CpSpec(spec, packed, N, TOP_K, TEMP, SEED, 1, kv_bits=bits)
        codes = torch.empty((F, 1, G), dtype=torch.int32, device="cuda")
        cp.decode_frames(xd[:4], cd[:4], codes[:4])
        torch.cuda.synchronize()
        cp.reset_stats()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        cp.decode_frames(xd, cd, codes)
        b.record()
        torch.cuda.synchronize()
        cp.status()
        ms = a.elapsed_time(b)
        st = cp.stats()
        out[name] = {"codes_per_s": round(F * (G - 1) / (ms / 1e3), 1), "passes_per_frame": round(st["passes"] / F, 3),
                     "us_per_pass": round(ms * 1e3 / st["passes"], 2),
                     "weight_mb_per_pass": round(st["weight_bytes"] / st["passes"] / 1e6, 1),
                     "hbm_frac": round((st["weight_bytes"] + st["kv_bytes"]) / (ms / 1e3) / 1e9 / peak, 4)}
        cp.close()
    return out


def sweep(cp_factory, xd, cd, G, peak, windows=(0, 2, 3, 4, 5, 6, 7, 8)):
    """codes/s and per-pass time for the AR loop (N=0) and windows 2..8 on the frames of
    xd (one warm-up decode, then two timed)."""
    import torch
    out = {}
    F = xd.shape[0]
    for n in windows:
        cp = cp_factory(n)
        codes = torch.empty((F, 1, G), dtype=torch.int32, device="cuda")
        cp.decode_frames(xd, cd, codes)
        torch.cuda.synchronize()
        cp.reset_stats()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        reps = 2
        a.record()
        for _ in range(reps):
            cp.decode_frames(xd, cd, codes)
        b.record()
        torch.cuda.synchronize()
        ms = a.elapsed_time(b) / reps
        st = cp.stats()
        cp.last_stats = st
        passes = st["passes"] / reps
        out[f"N{n}"] = {"codes_per_s": round(F * (G - 1) / (ms / 1e3), 1), "passes_per_frame": round(passes / F, 3),
                        "us_per_pass": round(ms * 1e3 / passes, 2),
                        "hbm_frac": round((st["weight_bytes"] + st["kv_bytes"]) / reps / (ms / 1e3) / 1e9 / peak, 4)}
        cp.close()
    return out


def batched(spec, dw, peak, streams=64, frames=500):
    """The batched configuration: `streams` concurrent streams (ragged accept counts and KV
    lengths arise on their own), N=4, half the streams greedy and half top-k 50 / T 0.9,
    `frames` frames each.  max_streams = streams, so the GEMV kernels take the tensor-core
    path (bf16, many rows per pass)."""
    import numpy as np
    import torch
    from speculative_decoding_rvq_gb300 import binding, synth as S
    G = spec.num_code_groups
    x, c0 = S.gen_frames(spec, streams, frames, seed=3)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    cp = binding.CpSpec(spec, dw, 4, TOP_K, TEMP, SEED, streams)
    tk = np.full(streams, TOP_K, np.int32)
    tt = np.full(streams, TEMP, np.float32)
    tt[: streams // 2] = 0.0
    cp.set_stream_sampling(tk, tt)
    codes = torch.empty((frames, streams, G), dtype=torch.int32, device="cuda")
    cp.decode_frames(xd[:4], cd[:4], codes[:4])
    torch.cuda.synchronize()
    cp.reset_stats()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    cp.decode_frames(xd, cd, codes)
    b.record()
    torch.cuda.synchronize()
    cp.status()
    ms = a.elapsed_time(b)
    st = cp.stats()
    out = {"streams": streams, "frames": frames, "verify_window": 4, "greedy_streams": streams // 2,
           "codes_per_s": round(streams * frames * (G - 1) / (ms / 1e3), 1),
           "passes": st["passes"], "us_per_pass": round(ms * 1e3 / st["passes"], 2),
           "hbm_frac": round((st["weight_bytes"] + st["kv_bytes"]) / (ms / 1e3) / 1e9 / peak, 4),
           "gemv_path": "tcgen05 tiles (TMA-staged bf16 weights x inputs split hi/lo, TMEM accumulators)"}
    cp.close()
    return out


def expected_accepted(tgt, drf, k: int, T: float) -> float:
    """Closed-form mean of accepted drafts per round for given logits: with
    beta_t = sum_v min(p_t(v), q_t(v)) (p, q the processed target and draft laws of
    position t), a round accepts at least j drafts with probability prod_{t<=j} beta_t,
    so E[accepted] = sum_j prod_{t<=j} beta_t ("Speculative Decoding, Beyond Text",
    section 02: sum-min = 1 - TV).  Analysis of the benchmark's inputs, outside the
    timed region; tgt [R, N, V], drf [R, N-1, V] torch tensors."""
    import torch

    def proc(x):
        z = x / T
        v, i = z.topk(min(k, z.shape[-1]), dim=-1)
        return torch.zeros_like(z).scatter_(-1, i, torch.softmax(v, dim=-1))

    n = drf.shape[1]
    beta = torch.minimum(proc(tgt[:, :n]), proc(drf)).sum(-1)  # [R, N-1]
    return float(torch.cumprod(beta, dim=1).sum(1).mean().item())


def expected_accepted_greedy(tgt, drf) -> float:
    """Greedy mode: a draft is accepted while the argmax of its draft row equals the argmax
    of the target row at the same position, so the mean accepted count is the mean length
    of the agreeing prefix (ties between equal maxima have probability zero for these
    continuous inputs)."""
    import torch
    n = drf.shape[1]
    eq = (drf.argmax(-1) == tgt[:, :n].argmax(-1)).to(torch.float64)
    return float(torch.cumprod(eq, dim=1).sum(1).mean().item())


def accepted_tail(tgt, drf, k: int, T: float) -> list:
    """P(a round accepts at least j drafts) for j = 1..N-1, averaged over the rounds of
    the given logits: prod_{t<=j} beta_t with beta_t = sum_v min(p_t(v), q_t(v)) when
    sampling ("Speculative Decoding, Beyond Text", section 02), the indicator that the
    first j draft argmaxes equal the target argmaxes when greedy (T = 0)."""
    import torch
    n = drf.shape[1]
    if T > 0:
        def proc(x):
            z = x / T
            v, i = z.topk(min(k, z.shape[-1]), dim=-1)
            return torch.zeros_like(z).scatter_(-1, i, torch.softmax(v, dim=-1))
        per = torch.minimum(proc(tgt[:, :n]), proc(drf)).sum(-1).to(torch.float64)
    else:
        per = (drf.argmax(-1) == tgt[:, :n].argmax(-1)).to(torch.float64)
    return [float(v) for v in torch.cumprod(per, dim=1).mean(0).tolist()]


def accept_extras(n_accepted, N: int, V: int, ms: float, tail: list, peak: float) -> dict:
    """Per-line analysis of the acceptance microbench, from the kernel's accepted counts
    [R]: the histogram of accepted drafts (fractions of rounds with 0..N-1) beside the
    closed-form one from `tail` (P(n = j) = P(n >= j) - P(n >= j + 1)), and the bytes of
    the rows a left-to-right chain must read, per second: the N - 1 draft rows and the
    target rows up to the first rejection or the bonus (n + 1 of them), so (N + n) V 4
    bytes for a round that accepts n."""
    import torch
    na = n_accepted.reshape(-1).long()
    R = na.numel()
    hist = torch.bincount(na, minlength=N)[:N].to(torch.float64) / R
    t = [1.0] + list(tail) + [0.0]
    rows = float((N + na).sum().item())
    gbs = rows * V * 4 / (ms / 1e3) / 1e9
    return {"accept_hist": [round(float(h), 4) for h in hist.tolist()],
            "closed_form_hist": [round(t[j] - t[j + 1], 4) for j in range(N)],
            "rows_touched_GB_s": round(gbs, 1), "rows_touched_hbm_frac": round(gbs / peak, 4)}


def accept_microbench(peak):
    """Acceptance kernels alone (the acceptance-kernel microbench configuration): 65536
    independent rounds, V 2048, target logits N(0, 3^2), draft logits
    rho * target + sqrt(1 - rho^2) * N(0, 3^2) for rho in {0.3, 0.7, 0.95}, N in {2, 4, 8},
    top-k 50; sampling mode (T 0.9, Philox draws) and greedy mode (T 0, argmax equality).
    Each line: rounds/s, the logit bytes read per second against the measured HBM peak, the
    mean accepted drafts per round and their histogram, each beside its closed form for the
    same inputs, and the bytes of the rows the chain must read (rows touched) per second."""
    import torch
    from speculative_decoding_rvq_gb300 import binding
    R, V = 65536, 2048
    res = {}
    g = torch.Generator(device="cuda").manual_seed(1)
    for N in (2, 4, 8):
        tgt = torch.randn((R, N, V), device="cuda", generator=g) * 3.0
        for rho in (0.3, 0.7, 0.95):
            drf = rho * tgt[:, : N - 1] + (1 - rho * rho) ** 0.5 * torch.randn((R, N - 1, V), device="cuda",
                                                                               generator=g) * 3.0
            drf = drf.contiguous()
            for mode, T in (("sampling", TEMP), ("greedy", 0.0)):
                for _ in range(3):
                    binding.accept_batch(tgt, drf, TOP_K, T, SEED, 0)
                torch.cuda.synchronize()
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                a.record()
                reps = 5
                for _ in range(reps):
                    tok, na, _ = binding.accept_batch(tgt, drf, TOP_K, T, SEED, 0)
                b.record()
                torch.cuda.synchronize()
                ms = a.elapsed_time(b) / reps
                gbs = (2 * N - 1) * V * 4 * R / (ms / 1e3) / 1e9
                line = {"rounds_per_s": round(R / (ms / 1e3), 1), "ms": round(ms, 3), "GB_s": round(gbs, 1),
                        "hbm_frac": round(gbs / peak, 4),
                        "mean_accepted": round(float(na.float().mean().item()), 4)}
                try:
                    line["closed_form_accepted"] = round(
                        expected_accepted(tgt, drf, TOP_K, TEMP) if T > 0 else expected_accepted_greedy(tgt, drf), 4)
                except Exception as exc:  # analysis only: never lose the measured line over it
                    line["closed_form_accepted"] = f"unavailable: {type(exc).__name__}"
                try:
                    line.update(accept_extras(na, N, V, ms, accepted_tail(tgt, drf, TOP_K, T), peak))
                except Exception as exc:  # analysis only, as above
                    line["accept_hist"] = f"unavailable: {type(exc).__name__}"
                res[f"N{N}_rho{rho}_{mode}"] = line
            del drf
        del tgt
        torch.cuda.empty_cache()
    return res


# ------------------------------------------------------------ CPU baselines
def oracle_model():
    """The CPU oracle (single-threaded C, float64 forward) loaded with the workload's weights."""
    from oracle import oracle as O
    from speculative_decoding_rvq_gb300 import synth as S
    spec = S.TTS06B_BF16
    return O.Model(spec, S.gen_weights(spec, 0))


def oracle_codes_per_s(frames: int, window: int, model=None, first_frame: int = 0):
    """Codes/s of the CPU oracle on `frames` frames of the workload (frames first_frame..)."""
    from speculative_decoding_rvq_gb300 import synth as S
    spec = S.TTS06B_BF16
    m = model if model is not None else oracle_model()
    x, c0 = S.gen_frames(spec, 1, first_frame + frames, seed=SEED)
    x, c0 = x[first_frame:], c0[first_frame:]
    t = time.perf_counter()
    m.decode_frames(window, TOP_K, TEMP, SEED, x, c0, first_frame=first_frame)
    dt = time.perf_counter() - t
    return frames * (spec.num_code_groups - 1) / dt, dt


def cpu_baseline_entry(frames=3):
    v, dt = oracle_codes_per_s(frames, WINDOW)
    return {"value": round(v, 3), "unit": UNIT, "cores": 1, "host_cores": os.cpu_count(), "kind": "oracle",
            "sample": f"{frames} frames of the 1-stream workload (N={WINDOW}), {dt:.1f} s single-threaded"}


def run_reference(args, rank, world):
    spec_frames = max(1, args.ref_frames)
    model = oracle_model()
    times = []
    for _ in range(min(max(args.warmup, 0), 1)):  # one untimed frame warms caches; more adds nothing
        oracle_codes_per_s(1, WINDOW, model)
    vals = []
    for i in range(args.steps):
        v, dt = oracle_codes_per_s(spec_frames, WINDOW, model, first_frame=i * spec_frames)
        vals.append(v)
        times.append(dt)
    from speculative_decoding_rvq_gb300 import synth as S
    value = statistics.mean(vals)
    return {
        "impl": "reference", "metric": METRIC, "value": round(value, 3), "unit": UNIT, "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(1e3 * statistics.mean(times), 1),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": dict(workload_config(S.TTS06B_BF16, FRAMES, 1, WINDOW), parallelism="cpu oracle, 1 thread"),
        "cpu_baseline": {"value": round(value, 3), "unit": UNIT, "cores": 1, "host_cores": os.cpu_count(), "kind": "oracle",
                         "sample": f"{spec_frames} frames per step of the 1-stream workload"},
        "e2e": {"value": round(value, 3), "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }


def profile_rounds(args):
    """Profiling case for ncu: the default workload's model, `args.profile_streams` streams,
    `args.profile_rounds`
    decoder passes through the step-wise API (cp_spec_round launches the pass kernels
    directly, so a profiler sees each kernel launch; inside the call graph the pass
    kernels run under a device-side loop).  Prints one status line."""
    import torch
    from speculative_decoding_rvq_gb300 import binding, synth as S
    spec = S.TTS06B_BF16
    B = args.profile_streams
    dw = binding.weights_to_device(spec, S.gen_weights(spec, 0))
    x, c0 = S.gen_frames(spec, B, 8, seed=1)
    xd, cd = torch.from_numpy(x).cuda(), torch.from_numpy(c0).cuda()
    cp = binding.CpSpec(spec, dw, args.window, TOP_K, TEMP, SEED, B)
    codes = torch.zeros((B, spec.num_code_groups), dtype=torch.int32, device="cuda")
    done, f = 0, 0
    while done < args.profile_rounds:
        cp.begin_frame(xd[f].clone(), cd[f].clone(), f)
        for _ in range(spec.num_code_groups - 1):
            cp.round(codes)
            done += 1
            if done >= args.profile_rounds:
                break
        f = (f + 1) % 8
    torch.cuda.synchronize()
    cp.status()
    st = cp.stats()
    print(json.dumps({"profile_rounds": done, "passes": st["passes"], "kernel_launches": st["kernel_launches"]}))


def profile_accept(args):
    """Profiling case for ncu: one acceptance call of the microbench kind (8192 rounds, N = 4,
    V 2048, rho 0.7, top-k 50, T 0.9), after one untimed call.  Inputs 470 MB > L2."""
    import torch
    from speculative_decoding_rvq_gb300 import binding
    R, N, V = 8192, 4, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    tgt = torch.randn((R, N, V), device="cuda", generator=g) * 3.0
    drf = (0.7 * tgt[:, : N - 1] + 0.51 ** 0.5 * torch.randn((R, N - 1, V), device="cuda", generator=g) * 3.0).contiguous()
    for _ in range(2):
        tok, na, _ = binding.accept_batch(tgt, drf, TOP_K, TEMP, SEED, 0)
    torch.cuda.synchronize()
    print(json.dumps({"profile_accept": R, "mean_accepted": round(float(na.float().mean().item()), 4)}))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--impl", default="gb300", choices=["gb300", "reference"])
    ap.add_argument("--frames", type=int, default=FRAMES)
    ap.add_argument("--window", type=int, default=WINDOW)
    ap.add_argument("--ref-frames", type=int, default=2)
    ap.add_argument("--no-sweep", action="store_true")
    ap.add_argument("--no-large", action="store_true", help="skip the large-model line")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--profile-rounds", type=int, default=0,
                    help="run this many step-wise passes (direct kernel launches, for a profiler) and exit")
    ap.add_argument("--profile-streams", type=int, default=1, help="streams of the --profile-rounds case")
    ap.add_argument("--profile-accept", action="store_true", help="run one acceptance-kernel call and exit")
    args = ap.parse_args()
    if args.profile_rounds > 0:
        profile_rounds(args)
        return
    if args.profile_accept:
        profile_accept(args)
        return
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    if args.impl == "reference":
        if rank != 0:
            return
        print(json.dumps(run_reference(args, rank, world)), flush=True)
        return
    if world > 1:
        import torch
        torch.distributed.init_process_group("nccl")
    res = run_gpu(args, rank, world)
    if rank == 0:
        if not args.no_cpu_baseline and world == 1:
            res["cpu_baseline"] = cpu_baseline_entry()
        print(json.dumps(res), flush=True)
    if world > 1:
        import torch
        torch.distributed.destroy_process_group()


if __name__ == "__main__":
    main()
