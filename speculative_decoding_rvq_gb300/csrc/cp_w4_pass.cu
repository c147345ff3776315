// cp_w4_pass.cu -- the GEMVs of a decoder pass over packed 4-bit weights (the
// product itself is in cp_w4.cuh), and the attention of a pass over a 4-bit
// KV cache.
//
// One CTA of 8 warps takes up to rb rows of the pass and walks over groups of
// 16-row weight tiles, like the public operator: wk warps split K, the others
// take neighbouring tiles, the shares are added in warp order through shared
// memory, and gemv_out writes the outputs.  What differs is around the
// product.  The rows come from the pass plan: embeddings or x in layer 0, else
// the residual stream (times the norm's gain), attention outputs or SwiGLU
// activations.  A norm's scale is a row's factor on the outputs, from sums of
// squares taken block by block as the rows are converted.  For QKV and gate/up
// the tiles of a unit's two rows (RoPE halves; gate and up) are neighbours in
// the walk, so one CTA has both.  Weights do not change within a pass: their
// first copies are issued before the wait for the previous kernel.
//
// A pass row counts as two fp16 columns (22 bits), so results are those of
// float32 rows; every order of summation depends on the model and the context
// only, as in the other GEMV kernels.
//
// With a 4-bit KV cache the QKV kernel leaves the rows' keys (after RoPE) and
// values in a row buffer and says which positions each stream's rows have; the
// public cache write and attention kernels do the rest, a stream's frame being
// one page per layer.
#include <algorithm>

#include "cp_gemv.cuh"
#include "cp_ops4.h"
#include "cp_w4.cuh"

namespace cpk {

// Shared memory of the kernel for one kind.
struct W4PassSmem {
  int XS, ring, red, fac, ssq, inv;
  size_t total;
};
__host__ __device__ inline W4PassSmem w4_pass_smem(int rb, int KB, int tile_bytes) {
  W4PassSmem L;
  L.XS = KB * 256 + 64;
  size_t at = (size_t)rb * 2 * L.XS;
  L.ring = (int)at;
  at += (size_t)kW4Warps * w4_stages(1) * tile_bytes;
  L.red = (int)at;
  at += (size_t)2 * kW4Warps * 16 * rb * 4;
  L.fac = (int)at;
  at += (size_t)KB * rb * 4;
  L.ssq = (int)at;
  at += (size_t)KB * rb * 4;
  L.inv = (int)at;
  at += (size_t)rb * 4;
  L.total = (at + 127) / 128 * 128;
  return L;
}

// Tiles of a kind in walk order: pairs of tiles for QKV (the halves of 16
// RoPE pairs) and gate/up.
__host__ __device__ inline long long w4_pass_tiles(const FrameParams& P, int kind, int nheads) {
  switch (kind) {
    case kQKV: return (long long)(P.nq + 2 * P.nkv) * (P.d / 16);
    case kO: case kDown: return P.H / 16;
    case kGU: return (long long)(P.F / 16) * 2;
    default: return (long long)nheads * (P.V / 16);
  }
}

// Packed tiles (all blocks of K) of tile `i` of the walk.
__device__ __forceinline__ const unsigned char* w4_pass_tile(const FrameParams& P, int kind, int l, const int* heads, int i,
                                                             size_t row_tile_bytes) {
  const unsigned char* base;
  int at = i;
  switch (kind) {
    case kQKV: {
      const int per = P.d / 32, p = i >> 1, hh = p / per, t16 = p - hh * per + (i & 1) * per;
      if (hh < P.nq) {
        base = static_cast<const unsigned char*>(P.wq[l]);
        at = hh * (P.d / 16) + t16;
      } else if (hh < P.nq + P.nkv) {
        base = static_cast<const unsigned char*>(P.wk[l]);
        at = (hh - P.nq) * (P.d / 16) + t16;
      } else {
        base = static_cast<const unsigned char*>(P.wv[l]);
        at = (hh - P.nq - P.nkv) * (P.d / 16) + t16;
      }
      break;
    }
    case kO: base = static_cast<const unsigned char*>(P.wo[l]); break;
    case kGU:
      base = static_cast<const unsigned char*>((i & 1) ? P.w_up[l] : P.w_gate[l]);
      at = i >> 1;
      break;
    case kDown: base = static_cast<const unsigned char*>(P.w_down[l]); break;
    default: {
      const int per = P.V / 16, hi = i / per;
      base = static_cast<const unsigned char*>(P.head);
      at = (heads[hi] - 1) * per + (i - hi * per);
    }
  }
  return base + (size_t)at * row_tile_bytes;
}

// Eight input values of a row: float32, or an embedding row in the model's type.
template <typename WT>
__device__ __forceinline__ void w4_load_act(const ActRow& a, int k0, float (&v)[8]) {
  constexpr int EPC = WTraits<WT>::EPC;
#pragma unroll
  for (int c = 0; c < 8; c += EPC) {
    float2 w[EPC / 2];
    load_act<WT>(a, k0 + c, w);
#pragma unroll
    for (int i = 0; i < EPC / 2; ++i) {
      v[c + 2 * i] = w[i].x;
      v[c + 2 * i + 1] = w[i].y;
    }
  }
}

// Keys (heads 0 .. nkv - 1, with RoPE) and values (the next nkv) of pass row gi
// to the row buffer of a 4-bit cache.
__device__ __forceinline__ void w4_kv_row(const FrameParams& P, const PassRows& pr, int h, int e, int gi, float y0, float y1) {
  const int r = pr.prow[gi], half = P.d / 2;
  const bool value = h >= P.nkv;
  if (!value) {
    const float2 cs = P.rope[(size_t)pr.ppos[gi] * half + e];
    const float a = y0 * cs.x - y1 * cs.y, c = y1 * cs.x + y0 * cs.y;
    y0 = a;
    y1 = c;
  }
  const size_t rows = (size_t)P.Bmax * P.NS;
  float* dst = P.kvrow + ((value ? rows : 0) + r) * P.nkv * P.d + (size_t)(value ? h - P.nkv : h) * P.d + e;
  dst[0] = y0;
  dst[half] = y1;
}

template <typename WT, int NT, int NS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_pass_kernel(const __grid_constant__ FrameParams P, int lk) {
  constexpr int TB = 1024 + 32 * NS, ST = w4_stages(1);
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ int s_heads[kMaxHeadsPerPass];
  pdl_launch_dependents();
  const int l = lk >> 3, kind = lk & 7;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int K = gemv_K(P, kind), KB = (K + kW4TileK - 1) / kW4TileK, rb = P.w4_rb;
  const int WK = P.w4_wk[kind], WM = kW4Warps / WK, wk = warp % WK, wm = warp / WK;
  const W4PassSmem L = w4_pass_smem(rb, KB, TB);
  unsigned char* ring = sm + L.ring + (size_t)warp * ST * TB;
  float* red = reinterpret_cast<float*>(sm + L.red);  // [2][8 warps][rb][16]
  float* fac = reinterpret_cast<float*>(sm + L.fac);  // [KB][rb]
  float* ssq = reinterpret_cast<float*>(sm + L.ssq);  // [KB][rb]
  float* inv = reinterpret_cast<float*>(sm + L.inv);  // [rb]
  // the plan is written before the pass starts
  const int nrows = min(__ldcg(&P.plan->nrows), P.Bmax * P.NS), r0 = blockIdx.y * rb;
  const int rows = min(rb, nrows - r0);
  if (rows <= 0) return;
  const int nheads = kind == kHeads ? min(__ldcg(&P.plan->nheads), kMaxHeadsPerPass) : 0;
  if (kind == kHeads) {
    if (tid < nheads) s_heads[tid] = __ldcg(&P.plan->heads[tid]);
    __syncthreads();
  }
  const int tiles = (int)w4_pass_tiles(P, kind, nheads), groups = (tiles + WM - 1) / WM;
  const int gx = gridDim.x, mine = (groups - (int)blockIdx.x + gx - 1) / gx;
  if (mine <= 0) return;
  const int kb0 = KB * wk / WK, nb = KB * (wk + 1) / WK - kb0;
  const size_t row_tile = (size_t)KB * TB;

  int left = 0, ctile = (int)blockIdx.x * WM + wm, cslot = 0;
  const unsigned char* src = nullptr;
  auto issue = [&]() {
    if (ctile < tiles && nb > 0) {
      if (left == 0) {
        left = nb;
        src = w4_pass_tile(P, kind, l, s_heads, ctile, row_tile) + (size_t)kb0 * TB + lane * 16;
      }
      unsigned char* dst = ring + cslot * TB + lane * 16;
      cp_async16(dst, src);
      cp_async16(dst + 512, src + 512);
      if (lane < 2 * NS) cp_async16(dst + 1024, src + 1024);
      src += TB;
      if (--left == 0) ctile += gx * WM;
    }
    cslot = cslot + 1 == ST ? 0 : cslot + 1;
    cp_async_commit();
  };
#pragma unroll 1
  for (int q = 0; q < ST - 1; ++q) issue();
  pdl_wait();

  const PassRows pr{P.prow, P.ppos, P.pcode};
  const bool opens = kind == kQKV && l == 0;
  if (opens && P.kv4 && blockIdx.x == 0 && blockIdx.y == 0) {  // the streams' rows (consecutive slots and positions)
    for (int b = tid; b < P.Bmax; b += kW4Threads) P.kv4_pos[b] = P.kv4_rows[b] = P.kv4_len[b] = 0;
    __syncthreads();
    for (int i = tid; i < nrows; i += kW4Threads) {
      const int r = pr.prow[i], b = r / P.NS;
      if (i == 0 || pr.prow[i - 1] / P.NS != b) P.kv4_pos[b] = pr.ppos[i];
      if (i == nrows - 1 || pr.prow[i + 1] / P.NS != b) {
        P.kv4_rows[b] = r - b * P.NS + 1;
        P.kv4_len[b] = pr.ppos[i] + 1;
      }
    }
  }
  const float* gain = kind == kQKV ? P.attn_norm[l] : (kind == kGU ? P.ffn_norm[l] : (kind == kHeads ? P.final_norm : nullptr));
  {
    constexpr int U = 2;
    const unsigned pairs = (KB + 1) / 2;
    const int units = rows * (int)pairs;
    const int kl0 = lane >> 4, at = (lane & 15) * 8;
    for (int u0 = warp; u0 < units; u0 += U * kW4Warps) {
      float f[U][8];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + i * kW4Warps, r = u / (int)pairs, k0 = (2 * (u - r * (int)pairs) + kl0) * kW4TileK + at;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = 0.0f;
        if (u < units && k0 < K) {  // (K is a multiple of 16: eight elements are all inside or all outside)
          const ActRow a = act_row<WT>(P, *P.call, pr, kind, l, r0 + r);
          w4_load_act<WT>(a, k0, f[i]);
          if (opens && blockIdx.x == 0) {  // the residual stream starts as the input rows
            float4* h = reinterpret_cast<float4*>(P.h + (size_t)pr.prow[r0 + r] * P.H + k0);
            h[0] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
            h[1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + i * kW4Warps;
        if (u >= units) break;
        const int r = u / (int)pairs, kl = 2 * (u - r * (int)pairs) + kl0, k0 = kl * kW4TileK + at;
        if (gain != nullptr) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(f[i][e], f[i][e], s);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (kl < KB && at == 0) ssq[kl * rb + r] = s;
          if (k0 < K) {
            const float4 a = *reinterpret_cast<const float4*>(gain + k0), c = *reinterpret_cast<const float4*>(gain + k0 + 4);
            f[i][0] *= a.x; f[i][1] *= a.y; f[i][2] *= a.z; f[i][3] *= a.w;
            f[i][4] *= c.x; f[i][5] *= c.y; f[i][6] *= c.z; f[i][7] *= c.w;
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[i][e]) & 0x7FFFFFFFu);
        const bool odd = __any_sync(0xffffffffu, top >= 0x7F800000u);
        if (odd) {
          top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max(top, finite_abs_bits(f[i][e]));
        }
        uint4 hi, lo;
        const float down = to_fp16_block<2>(f[i], top, odd, &hi, &lo);
        if (kl < KB) {
          unsigned char* dst = sm + (size_t)(2 * r) * L.XS + kl * 256 + at * 2;
          *reinterpret_cast<uint4*>(dst) = hi;
          *reinterpret_cast<uint4*>(dst + L.XS) = lo;
          if (at == 0) fac[kl * rb + r] = down;
        }
      }
    }
  }
  __syncthreads();
  if (tid < rows) {  // (read after the first group's barrier)
    float s = 1.0f;
    if (gain != nullptr) {
      s = 0.0f;
      for (int k = 0; k < KB; ++k) s += ssq[k * rb + tid];
      s = 1.0f / sqrtf(s / (float)P.H + P.eps);
    }
    inv[tid] = s;
  }

  const int cols = 2 * rows;
  const unsigned char* xcol[NT];
  const float* fcol[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xcol[n] = sm + (size_t)min(n * 8 + g, cols - 1) * L.XS + kb0 * 256 + t * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) fcol[n][c] = fac + kb0 * rb + min(n * 8 + 2 * t + c, cols - 1) / 2;
  }
  const bool pair = kind == kQKV || kind == kGU;
  int slot = 0;
#pragma unroll 1
  for (int j = 0; j < mine; ++j) {
    const int first = ((int)blockIdx.x + j * gx) * WM, tile = first + wm;
    float tot[1][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) tot[0][n][c] = 0.0f;
    if (tile < tiles)
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        W4Codes<1, NS> A;
        A.load(ring + slot * TB, lane);
        slot = slot + 1 == ST ? 0 : slot + 1;
        __syncwarp();  // every lane has read the stage that the next copy may reuse
        issue();
        w4_block<1, NT, NS>(A, xcol, b * 256, fcol, b * rb, tot);
      }
    float* part = red + ((j & 1) * kW4Warps + warp) * 16 * rb;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = n * 4 + t;
        if (r < rows) part[r * 16 + g + 8 * h] = tot[0][n][2 * h] + tot[0][n][2 * h + 1];
      }
    __syncthreads();
    const float* from = red + (j & 1) * kW4Warps * 16 * rb;
    const int outs = rows * 16 * (pair ? WM / 2 : WM);
    for (int i = tid; i < outs; i += kW4Threads) {
      const int m = i / (rows * 16), rest = i - m * rows * 16, r = rest >> 4, row = rest & 15;
      float y0 = 0.0f, y1 = 0.0f;
      if (pair) {
        if (first + 2 * m >= tiles) continue;
        for (int k = 0; k < WK; ++k) {
          y0 += from[(2 * m * WK + k) * 16 * rb + rest];
          y1 += from[((2 * m + 1) * WK + k) * 16 * rb + rest];
        }
        const int p = (first >> 1) + m;  // pair of tiles
        int u = p * 16 + row;            // gate/up: the feature
        if (kind == kQKV) {
          const int per = P.d / 32, hh = p / per, e = (p - hh * per) * 16 + row;
          u = hh * (P.d / 2) + e;
          if (P.kv4 && hh >= P.nq) {
            w4_kv_row(P, pr, hh - P.nq, e, r0 + r, y0 * inv[r], y1 * inv[r]);
          } else {
            gemv_out<kQKV>(P, l, s_heads, pr, P.rope, u, r0 + r, y0 * inv[r], y1 * inv[r], 0.0f);
          }
        } else {
          gemv_out<kGU>(P, l, s_heads, pr, P.rope, u, r0 + r, y0 * inv[r], y1 * inv[r], 0.0f);
        }
      } else {
        if (first + m >= tiles) continue;
        for (int k = 0; k < WK; ++k) y0 += from[(m * WK + k) * 16 * rb + rest];
        const int u = (first + m) * 16 + row;
        if (kind == kHeads) gemv_out<kHeads>(P, l, s_heads, pr, P.rope, u, r0 + r, y0 * inv[r], 0.0f, 0.0f);
        else gemv_out<kO>(P, l, s_heads, pr, P.rope, u, r0 + r, y0, 0.0f, __ldcg(P.h + (size_t)pr.prow[r0 + r] * P.H + u));
      }
    }
  }
  cp_async_wait_group<0>();
}

}  // namespace cpk

// -------------------------------------------------------------- host side
namespace cpk_host {

using cpk::FrameParams;

static int w4_pass_K(const FrameParams& P, int kind) {
  return kind == cpk::kO ? P.nq * P.d : (kind == cpk::kDown ? P.F : P.H);
}

size_t w4_pass_smem_bytes(const FrameParams& P, int kind) {
  const int KB = (w4_pass_K(P, kind) + cpk::kW4TileK - 1) / cpk::kW4TileK;
  return cpk::w4_pass_smem(P.w4_rb, KB, cpk::w4_tile_bytes(P.w4)).total;
}

// Rows per CTA: up to eight (two MMA columns each) that fit; per kind the most
// warps along K that leave no more groups of tiles than CTAs fit the SMs (a
// pass's GEMVs are short: what counts is how soon the last weight arrives).
bool plan_w4(FrameParams& P, int sms) {
  constexpr size_t kBudget = 200 * 1024;
  for (P.w4_rb = std::min(P.Bmax * P.NS, 8);; P.w4_rb = (P.w4_rb + 1) / 2) {
    bool fits = true;
    for (int kind = cpk::kQKV; kind <= cpk::kHeads; ++kind) fits = fits && w4_pass_smem_bytes(P, kind) <= kBudget;
    if (fits) break;
    if (P.w4_rb == 1) return false;
  }
  for (int kind = cpk::kQKV; kind <= cpk::kHeads; ++kind) {
    const bool pair = kind == cpk::kQKV || kind == cpk::kGU;
    const int KB = (w4_pass_K(P, kind) + cpk::kW4TileK - 1) / cpk::kW4TileK;
    const long long slots = (long long)sms * std::min<size_t>(2, kBudget / w4_pass_smem_bytes(P, kind));
    const long long tiles = cpk::w4_pass_tiles(P, kind, std::min(P.G - 1, P.ND + 2));
    int wk = pair ? 4 : 8;
    auto groups = [&](int k) { return (tiles + cpk::kW4Warps / k - 1) / (cpk::kW4Warps / k); };
    while (wk > 1 && (wk > KB || groups(wk) > slots)) wk /= 2;
    P.w4_wk[kind] = wk;
    P.w4_gx[kind] = (int)std::min(slots, groups(wk));
  }
  return true;
}

dim3 w4_pass_grid(const FrameParams& P, int kind) {
  return dim3(P.w4_gx[kind], (P.Bmax * P.NS + P.w4_rb - 1) / P.w4_rb);
}

template <typename WT, int NT>
static const void* w4_pass_fn_ns(int group) {
  if (group == 32) return (const void*)cpk::w4_pass_kernel<WT, NT, 4>;
  if (group == 64) return (const void*)cpk::w4_pass_kernel<WT, NT, 2>;
  return (const void*)cpk::w4_pass_kernel<WT, NT, 1>;
}

const void* w4_pass_fn(const FrameParams& P) {
  const bool one = P.w4_rb <= 4;
  if (P.dtype == 1) return one ? w4_pass_fn_ns<__nv_bfloat16, 1>(P.w4) : w4_pass_fn_ns<__nv_bfloat16, 2>(P.w4);
  return one ? w4_pass_fn_ns<float, 1>(P.w4) : w4_pass_fn_ns<float, 2>(P.w4);
}

// The rows of layer l into its cache, then their attention.
cudaError_t enqueue_kv4_attention(const FrameParams& P, int l, int sms, cudaStream_t s) {
  const Kv4Shape S{P.Bmax, P.kv4, P.nkv, P.d};
  void* cache = P.kv4_cache + (size_t)l * P.kv4_layer;
  const long long width = (long long)P.nkv * P.d;
  const float* v = P.kvrow + (size_t)P.Bmax * P.NS * width;
  cudaError_t e = launch_kv4_append(S, cache, nullptr, 1, P.Bmax, P.NS, P.kv4_pos, P.kv4_rows, 0, P.kvrow, width, v, width, s);
  if (e != cudaSuccess) return e;
  Kv4Attention A{};
  A.cache = cache; A.kv_len = P.kv4_len; A.n_rows = P.kv4_rows;
  A.q = P.qbuf; A.o = P.abuf;
  A.qs = A.os = (long long)P.nq * P.d;
  A.max_pages = 1; A.B = P.Bmax; A.M = P.NS; A.nq = P.nq; A.dtype = 0;
  A.scale = 1.0f / sqrtf((float)P.d);
  return launch_kv4_attention(S, A, sms, s);  // (a page is too short to be split: no workspace)
}

// Shared-memory limits of the cache kernels, before their first capture.
cudaError_t configure_kv4_attention(const FrameParams& P) {
  return kv4_attention_configure(Kv4Shape{P.Bmax, P.kv4, P.nkv, P.d}, 1, P.Bmax, P.NS, P.nq, 0);
}

// The table head_j . b_t of the draft offsets: [G - 1][KO][V], one product per head.
cudaError_t launch_offset_table_w4(const FrameParams& P, int sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const size_t head = w4_bytes(P.V, P.H, P.w4);
  for (int j = 0; j < P.G - 1 && e == cudaSuccess; ++j)
    e = launch_w4_gemv(P.KO, P.V, P.H, P.w4, 0, 0, P.draft_offset, P.H, static_cast<const unsigned char*>(P.head) + j * head,
                       P.otab + (size_t)j * P.KO * P.V, P.V, sms, s);
  return e;
}

}  // namespace cpk_host
