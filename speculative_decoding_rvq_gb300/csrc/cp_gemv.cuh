// cp_gemv.cuh -- what the GEMV kernels of a decoder pass share: weight element
// types, programmatic launches, the shapes of the GEMV kinds, where a pass row
// comes from and where its outputs go.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cp_common.cuh"
#include "cp_frame.cuh"

namespace cpk {

// ------------------------------------------------------------ weight types
// One 16-byte chunk of a weight row in shared memory: loaded raw, then
// converted to float2 pairs.
template <typename WT> struct WTraits;
template <> struct WTraits<float> {
  static constexpr int EB = 4;   // bytes per element
  static constexpr int EPC = 4;  // elements per 16-byte chunk
  typedef float4 Raw;
  __device__ __forceinline__ static Raw ld_raw(const unsigned char* p) { return *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ static void cvt(const Raw& v, float2 (&w)[2]) {
    w[0] = make_float2(v.x, v.y);
    w[1] = make_float2(v.z, v.w);
  }
  __device__ __forceinline__ static float load1(const void* base, size_t i) {
    return __ldg(static_cast<const float*>(base) + i);
  }
};
template <> struct WTraits<__nv_bfloat16> {
  static constexpr int EB = 2;
  static constexpr int EPC = 8;
  typedef uint4 Raw;
  __device__ __forceinline__ static Raw ld_raw(const unsigned char* p) { return *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ static void cvt(const Raw& v, float2 (&w)[4]) {
    w[0] = bf16x2_to_f2(v.x);
    w[1] = bf16x2_to_f2(v.y);
    w[2] = bf16x2_to_f2(v.z);
    w[3] = bf16x2_to_f2(v.w);
  }
  __device__ __forceinline__ static float load1(const void* base, size_t i) {
    const unsigned short u = __ldg(static_cast<const unsigned short*>(base) + i);
    return __uint_as_float((uint32_t)u << 16);
  }
};

// -------------------------------------------------- programmatic launches
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------ GEMV shapes
// Output units of a GEMV kind: QKV = RoPE pair (e, e + d/2) of a head;
// O, down = output row; gate/up = feature (gate row + up row);
// lm_heads = (head of the pass, vocabulary row).
__host__ __device__ __forceinline__ int rows_per_unit(int kind) { return (kind == kQKV || kind == kGU) ? 2 : 1; }

__device__ __forceinline__ int gemv_K(const FrameParams& P, int kind) {
  return kind == kO ? P.nq * P.d : (kind == kDown ? P.F : P.H);
}

__device__ __forceinline__ int gemv_units(const FrameParams& P, int kind, int nheads) {
  switch (kind) {
    case kQKV: return (P.nq + 2 * P.nkv) * (P.d / 2);
    case kO: case kDown: return P.H;
    case kGU: return P.F;
    default: return nheads * P.V;
  }
}

// Where a GEMV input row comes from: an fp32 row, or (first layer, positions
// >= 1) a row of the code embedding in the weight type.
struct ActRow {
  const float* f;
  const void* w;
};

// Raw input element values k0 .. k0 + EPC - 1 of row `src` (as float2 pairs).
template <typename WT>
__device__ __forceinline__ void load_act(const ActRow& src, int k0, float2 (&out)[WTraits<WT>::EPC / 2]) {
  constexpr int EPC = WTraits<WT>::EPC, PPC = EPC / 2;
  if (src.f != nullptr) {
#pragma unroll
    for (int i = 0; i < EPC; i += 4) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(src.f + k0 + i));
      out[i / 2] = make_float2(x.x, x.y);
      out[i / 2 + 1] = make_float2(x.z, x.w);
    }
  } else {
    WTraits<WT>::cvt(__ldg(reinterpret_cast<const typename WTraits<WT>::Raw*>(
                         static_cast<const unsigned char*>(src.w) + (size_t)k0 * WTraits<WT>::EB)),
                     out);
  }
  (void)PPC;
}

// The pass rows as a GEMV CTA sees them: the plan's arrays, copied to
// shared memory before the dependency wait (the plan is written before the
// pass's first kernel starts).
struct PassRows {
  const int* prow;
  const int* ppos;
  const int* pcode;
};

// Input row i of the pass (compacted index) for a GEMV kind.
template <typename WT>
__device__ __forceinline__ ActRow act_row(const FrameParams& P, const CallArgs& ca, const PassRows& pr, int kind, int l,
                                          int i) {
  const int r = pr.prow[i];
  ActRow a{nullptr, nullptr};
  switch (kind) {
    case kQKV:
      if (l == 0) {
        const int pos = pr.ppos[i], code = pr.pcode[i], b = r / P.NS;
        if (pos == 0)
          a.f = ca.mode == kModeTeacher ? ca.x + (size_t)b * P.H : ca.x + ((size_t)code * ca.B + b) * P.H;
        else
          a.w = static_cast<const WT*>(P.embed) + ((size_t)(pos - 1) * P.V + code) * P.H;
      } else {
        a.f = P.h + (size_t)r * P.H;
      }
      break;
    case kO: a.f = P.abuf + (size_t)r * P.nq * P.d; break;
    case kGU: a.f = P.h + (size_t)r * P.H; break;
    case kDown: a.f = P.fbuf + (size_t)r * P.F; break;
    default: a.f = P.h + (size_t)r * P.H;
  }
  return a;
}

// Outputs of one unit for pass row gi: RoPE + q / KV append (QKV), residual
// update (O, down), SwiGLU (gate/up), logits (lm_heads).
template <int KIND>
__device__ __forceinline__ void gemv_out(const FrameParams& P, int l, const int* heads, const PassRows& pr,
                                         const float2* rope, int u, int gi, float y0, float y1, float hold) {
  const int r = pr.prow[gi], pos = pr.ppos[gi];
  if (KIND == kQKV) {
    const int half = P.d / 2, hh = u / half, e = u - hh * half;
    const int b = r / P.NS;
    if (hh < P.nq + P.nkv) {
      const float2 cs2 = rope[(size_t)pos * half + e];
      const float r0 = y0 * cs2.x - y1 * cs2.y;
      const float r1 = y1 * cs2.x + y0 * cs2.y;
      if (hh < P.nq) {
        float* qd = P.qbuf + (size_t)r * P.nq * P.d + (size_t)hh * P.d;
        qd[e] = r0;
        qd[e + half] = r1;
      } else {
        const int slot = P.tree_n ? __ldcg(P.pslot + gi) : pos;  // KV slot (a tree node's own slot)
        float* kd = P.kv + (((((size_t)b * P.L + l) * 2 + 0) * P.GS + slot) * P.nkv + (hh - P.nq)) * P.d;
        kd[e] = r0;
        kd[e + half] = r1;
      }
    } else {
      const int slot = P.tree_n ? __ldcg(P.pslot + gi) : pos;
      float* vd = P.kv + (((((size_t)b * P.L + l) * 2 + 1) * P.GS + slot) * P.nkv + (hh - P.nq - P.nkv)) * P.d;
      vd[e] = y0;
      vd[e + half] = y1;
    }
  } else if (KIND == kO || KIND == kDown) {
    P.h[(size_t)r * P.H + u] = hold + y0;
  } else if (KIND == kGU) {
    P.fbuf[(size_t)r * P.F + u] = y0 / (1.0f + expf(-y0)) * y1;
  } else {
    const int hi = u / P.V, v = u - hi * P.V;
    const int slot = heads[hi] - pos;
    // a lookahead-t draft with a position-aware offset reads head_j on
    // h + b_t = head_j . h + head_j . b_t (the second term from the table)
    if (slot >= 1 && slot <= P.KO) y0 += __ldg(&P.otab[((size_t)(heads[hi] - 1) * P.KO + slot - 1) * P.V + v]);
    if (pos >= 1 && slot >= 0 && slot <= P.ND) P.logits[((size_t)r * (1 + P.ND) + slot) * P.V + v] = y0;
  }
}

}  // namespace cpk
