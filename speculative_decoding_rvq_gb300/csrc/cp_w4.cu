// cp_w4.cu -- products with 4-bit weights: y[r][n] = sum_k x[r][k] w[n][k],
// w[n][k] = s[n][k / group] * c[n][k] in the format of cp_fp4.cuh.
//
// Packed matrix.  A tile is 16 rows x 128 columns: 1024 bytes of codes and
// the tile's scales, contiguous; the tiles of 16 rows follow one another along
// K, so a warp that owns a K range of 16 rows streams one run of memory.
// Codes are in the order of the m16n8k16 A operand: lane 4 g + t of a warp
// holds 16 bytes of row g and 16 bytes of row g + 8, one 32-bit word per 32
// columns, the word's byte j holding columns 8 t + 2 j and 8 t + 2 j + 1.
// Rows and columns past the matrix are zero codes with zero scales.
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include "cp_fp4.cuh"
#include "cp_ops4.h"

namespace cpk {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4TileK = 128;
constexpr int kW4Stages = 6;  // tiles in flight per warp

__host__ __device__ inline int w4_groups(int group) { return kW4TileK / group; }  // scales per tile row
__host__ __device__ inline int w4_tile_bytes(int group) { return 1024 + 32 * w4_groups(group); }
// Byte offset of the scale of row i (0..15), group q of a tile.
__device__ __forceinline__ int w4_scale_at(int i, int q, int ns) { return 1024 + (i * ns + q) * 2; }

// ---------------------------------------------------------- pack, unpack
// One warp per tile: each lane takes four consecutive columns of each of the
// 16 rows, and the lanes of a group share its largest magnitude.  Runs once
// per matrix.
__global__ void __launch_bounds__(256) w4_pack_kernel(const void* w, int dtype, long long stride, bool vec, int N, int K,
                                                      int KB, int group, unsigned char* out) {
  const long long tile = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long tiles = (long long)((N + 15) / 16) * KB;
  if (tile >= tiles) return;
  const int n0 = (int)(tile / KB) * 16, kb = (int)(tile % KB);
  const int ns = w4_groups(group), lanes = group / 4;
  unsigned char* dst = out + tile * w4_tile_bytes(group);
  const int k0 = kb * kW4TileK + lane * 4;
  for (int i = 0; i < 16; ++i) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n0 + i < N)
      v = load4(static_cast<const unsigned char*>(w) + (long long)(n0 + i) * stride * elem_bytes(dtype), dtype, k0, K, vec);
    const float a = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
    uint32_t bits = __float_as_uint(a);
    if (!(fabsf(v.x) <= 3.4028234e38f && fabsf(v.y) <= 3.4028234e38f && fabsf(v.z) <= 3.4028234e38f &&
          fabsf(v.w) <= 3.4028234e38f))
      bits = 0x7F800000u;
    for (int o = lanes / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    const uint32_t sb = fp4_scale_bits(__uint_as_float(bits), bits >= 0x7F800000u);
    const float s = bf16_bits_f32(sb);
    const uint32_t c = float2_to_e2m1(fp4_quotient(v.x, s), fp4_quotient(v.y, s)) |
                       float2_to_e2m1(fp4_quotient(v.z, s), fp4_quotient(v.w, s)) << 8;
    // columns lane * 4 ..: word lane / 8, t = (lane % 8) / 2, upper or lower half of the word
    const int g = i & 7, t = (lane & 7) >> 1;
    *reinterpret_cast<uint16_t*>(dst + (i >> 3) * 512 + (g * 4 + t) * 16 + (lane >> 3) * 4 + (lane & 1) * 2) = (uint16_t)c;
    if (lane % lanes == 0) *reinterpret_cast<uint16_t*>(dst + w4_scale_at(i, lane / lanes, ns)) = (uint16_t)sb;
  }
}

__global__ void __launch_bounds__(256) w4_unpack_kernel(const unsigned char* packed, int N, int K, int KB, int group,
                                                        void* out, int dtype) {
  const long long tile = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long tiles = (long long)((N + 15) / 16) * KB;
  if (tile >= tiles) return;
  const int n0 = (int)(tile / KB) * 16, kb = (int)(tile % KB), ns = w4_groups(group);
  const unsigned char* src = packed + tile * w4_tile_bytes(group);
  const int k0 = kb * kW4TileK + lane * 4;
  for (int i = 0; i < 16 && n0 + i < N; ++i) {
    const int g = i & 7, t = (lane & 7) >> 1;
    const uint32_t c =
        *reinterpret_cast<const uint16_t*>(src + (i >> 3) * 512 + (g * 4 + t) * 16 + (lane >> 3) * 4 + (lane & 1) * 2);
    const float s = bf16_bits_f32(*reinterpret_cast<const uint16_t*>(src + w4_scale_at(i, lane * 4 / group, ns)));
    uint32_t h[4];
    e2m1_to_half2x4(c, h);
    const float2 lo = unpack_half2(h[0]), hi = unpack_half2(h[1]);
    const float v[4] = {lo.x * s, lo.y * s, hi.x * s, hi.y * s};
    for (int j = 0; j < 4; ++j)
      if (k0 + j < K) store_elem(out, (long long)(n0 + i) * K + k0 + j, dtype, v[j]);
  }
}

// ---------------------------------------------------------------- product
// Tensor-core product of few rows.  A CTA of 8 warps takes `rb` rows of x and
// walks over groups of 16-row tiles of w: WK of its warps split K, the other
// factor takes neighbouring tiles.  A warp streams its tiles through a ring
// of kW4Stages asynchronous copies in shared memory, turns codes into fp16
// (exact), and multiplies them with the rows of x, which are the N operand
// (8 columns per MMA).
//
// The rows of x are held as fp16, each block of 128 columns scaled by a power
// of two that the result is scaled back by: bfloat16 and fp16 inputs exactly
// (down to 2^-29 of the block's largest magnitude), float32 inputs as two
// columns hi + lo, 22 bits.  The MMAs accumulate one group in float32; the
// group's scale and the block's power of two are applied in float32, so the
// tensor core's truncating accumulation never runs over more than a group.
//
// Bound: the bytes of w.  Deep rings rather than wide tiles keep them
// streaming; the A operand is built in registers straight from the codes, so
// nothing but x and the copies goes through shared memory.
struct W4Gemv {
  const void* x;
  const unsigned char* w;
  void* y;
  long long xs, ys;  // row strides, in elements
  int R, N, K, KB, group;
  int xdt, ydt;
  int rb;       // rows of x per CTA
  int XS;       // bytes of one column of x in shared memory
  int wk;       // warps that split K
  int ring_at, red_at, fac_at;  // shared-memory offsets
  bool xvec;
};

template <int NT, int TERMS>
__global__ void __launch_bounds__(kW4Threads, NT == 1 ? 3 : (NT == 2 ? 2 : 1)) w4_gemv_kernel(const __grid_constant__ W4Gemv P) {
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int WK = P.wk, WM = kW4Warps / WK, wk = warp % WK, wm = warp / WK;
  const int r0 = blockIdx.y * P.rb, rows = min(P.rb, P.R - r0), cols = rows * TERMS;
  const int tiles = (P.N + 15) / 16, groups = (tiles + WM - 1) / WM;  // tile groups of WM neighbouring tiles
  const int kb0 = (int)((long long)P.KB * wk / WK), nb = (int)((long long)P.KB * (wk + 1) / WK) - kb0;
  const int ns = w4_groups(P.group), tb = w4_tile_bytes(P.group);
  const int mine = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // groups of this CTA
  unsigned char* ring = sm + P.ring_at + (size_t)warp * kW4Stages * tb;
  float* fac = reinterpret_cast<float*>(sm + P.fac_at);  // [KB][rb] powers of two
  float* red = reinterpret_cast<float*>(sm + P.red_at);  // [2][8 warps][16][rb]

  // items: this warp's tile of each group, block by block; an item past the matrix copies nothing
  const int items = mine * nb;
  int ij = 0, ib = 0;  // group and block of the next copy
  auto issue = [&](int q) {
    if (q < items) {
      const int tile = ((int)blockIdx.x + ij * (int)gridDim.x) * WM + wm;
      if (tile < tiles) {
        const unsigned char* src = P.w + ((long long)tile * P.KB + kb0 + ib) * tb;
        unsigned char* dst = ring + (q % kW4Stages) * tb;
        cp_async16(dst + lane * 16, src + lane * 16);
        cp_async16(dst + 512 + lane * 16, src + 512 + lane * 16);
        if (lane < 2 * ns) cp_async16(dst + 1024 + lane * 16, src + 1024 + lane * 16);
      }
      if (++ib == nb) { ib = 0; ++ij; }
    }
    cp_async_commit();
  };
  for (int q = 0; q < kW4Stages - 1; ++q) issue(q);

  // x: one warp per (row, block of 128 columns), four elements a lane
  {
    const int units = rows * P.KB, es = elem_bytes(P.xdt);
    for (int u0 = warp; u0 < units; u0 += 4 * kW4Warps) {
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = u0 + i * kW4Warps;
        if (u >= units) continue;
        const int r = u / P.KB, kb = u - r * P.KB;
        v[i] = load4(static_cast<const unsigned char*>(P.x) + (long long)(r0 + r) * P.xs * es, P.xdt,
                     kb * kW4TileK + lane * 4, P.K, P.xvec);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = u0 + i * kW4Warps;
        if (u >= units) continue;
        const int r = u / P.KB, kb = u - r * P.KB;
        const uint32_t m = max(max(finite_abs_bits(v[i].x), finite_abs_bits(v[i].y)),
                               max(finite_abs_bits(v[i].z), finite_abs_bits(v[i].w)));
        float up, down;
        pow2_normaliser(__reduce_max_sync(0xffffffffu, m), &up, &down);
        if (lane == 0) fac[kb * P.rb + r] = down;
        const float a = v[i].x * up, b = v[i].y * up, c = v[i].z * up, d = v[i].w * up;
        unsigned char* dst = sm + (size_t)(r * TERMS) * P.XS + kb * 256 + lane * 8;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_half2(a, b), pack_half2(c, d));
        if (TERMS == 2)
          *reinterpret_cast<uint2*>(dst + P.XS) =
              make_uint2(pack_half2(fp16_rest(a), fp16_rest(b)), pack_half2(fp16_rest(c), fp16_rest(d)));
      }
    }
  }
  __syncthreads();

  // columns of x: this lane's column as B operand, and the rows of its two
  // accumulator columns (a column past the rows repeats the last one and is
  // never stored)
  const unsigned char* xcol[NT];
  int arow[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xcol[n] = sm + (size_t)min(n * 8 + g, cols - 1) * P.XS + t * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) arow[n][c] = min(n * 8 + 2 * t + c, cols - 1) / TERMS;
  }

  int q = 0;
  for (int j = 0; j < mine; ++j) {
    const int tile = ((int)blockIdx.x + j * (int)gridDim.x) * WM + wm;
    float tot[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) tot[n][c] = 0.0f;
    for (int b = 0; b < nb; ++b, ++q) {
      cp_async_wait_group<kW4Stages - 2>();
      __syncwarp();
      const unsigned char* st = ring + (q % kW4Stages) * tb;
      const uint4 lo4 = *reinterpret_cast<const uint4*>(st + lane * 16);
      const uint4 hi4 = *reinterpret_cast<const uint4*>(st + 512 + lane * 16);
      uint32_t slo[2], shi[2];  // scales of rows g and g + 8, two to a word
      if (ns == 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(st + w4_scale_at(g, 0, 4));
        const uint2 c = *reinterpret_cast<const uint2*>(st + w4_scale_at(g + 8, 0, 4));
        slo[0] = a.x; slo[1] = a.y; shi[0] = c.x; shi[1] = c.y;
      } else if (ns == 2) {
        slo[0] = *reinterpret_cast<const uint32_t*>(st + w4_scale_at(g, 0, 2));
        shi[0] = *reinterpret_cast<const uint32_t*>(st + w4_scale_at(g + 8, 0, 2));
        slo[1] = shi[1] = 0;
      } else {
        slo[0] = *reinterpret_cast<const uint16_t*>(st + w4_scale_at(g, 0, 1));
        shi[0] = *reinterpret_cast<const uint16_t*>(st + w4_scale_at(g + 8, 0, 1));
        slo[1] = shi[1] = 0;
      }
      __syncwarp();  // every lane has read the stage that the next copy may reuse
      issue(q + kW4Stages - 1);
      if (tile >= tiles) continue;
      const int kb = kb0 + b;
      const uint32_t lw[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hw[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
      float blk[NT][4], acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) blk[n][c] = acc[n][c] = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t al[4], ah[4];
        e2m1_to_half2x4(lw[w], al);
        e2m1_to_half2x4(hw[w], ah);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(xcol[n] + kb * 256 + w * 64);
          mma_f16_16816(acc[n], al[0], ah[0], al[1], ah[1], x4.x, x4.y);
          mma_f16_16816(acc[n], al[2], ah[2], al[3], ah[3], x4.z, x4.w);
        }
        if (((w + 1) & (4 / ns - 1)) == 0) {  // the end of a group
          const int s = (w + 1) * ns / 4 - 1;
          const float a = bf16_bits_f32((slo[s >> 1] >> (16 * (s & 1))) & 0xFFFFu);
          const float c = bf16_bits_f32((shi[s >> 1] >> (16 * (s & 1))) & 0xFFFFu);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            blk[n][0] = fmaf(a, acc[n][0], blk[n][0]);
            blk[n][1] = fmaf(a, acc[n][1], blk[n][1]);
            blk[n][2] = fmaf(c, acc[n][2], blk[n][2]);
            blk[n][3] = fmaf(c, acc[n][3], blk[n][3]);
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f0 = fac[kb * P.rb + arow[n][0]], f1 = fac[kb * P.rb + arow[n][1]];
        tot[n][0] = fmaf(f0, blk[n][0], tot[n][0]);
        tot[n][1] = fmaf(f1, blk[n][1], tot[n][1]);
        tot[n][2] = fmaf(f0, blk[n][2], tot[n][2]);
        tot[n][3] = fmaf(f1, blk[n][3], tot[n][3]);
      }
    }
    // the tile's outputs: hi and lo columns of a row sit in one thread
    float* mine_red = red + ((j & 1) * kW4Warps + warp) * 16 * P.rb;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
#pragma unroll
        for (int c = 0; c < 2 / TERMS; ++c) {
          const int r = (n * 8 + 2 * t) / TERMS + c;
          const float v = TERMS == 2 ? tot[n][2 * h] + tot[n][2 * h + 1] : tot[n][2 * h + c];
          if (r < rows) {
            if (WK == 1) {
              const int o = tile * 16 + row;
              if (o < P.N) store_elem(P.y, (long long)(r0 + r) * P.ys + o, P.ydt, v);
            } else {
              mine_red[r * 16 + row] = v;
            }
          }
        }
      }
    }
    if (WK > 1) {  // add the K shares in warp order; the buffer of this parity is free again two groups on
      __syncthreads();
      const int outs = rows * 16 * WM;
      for (int i = tid; i < outs; i += kW4Threads) {
        const int m = i / (rows * 16), rest = i - m * rows * 16;  // rest = r * 16 + row
        const float* src = red + ((j & 1) * kW4Warps + m * WK) * 16 * P.rb + rest;
        float v = 0.0f;
        for (int k = 0; k < WK; ++k) v += src[k * 16 * P.rb];
        const long long o = (((long long)blockIdx.x + (long long)j * gridDim.x) * WM + m) * 16 + (rest & 15);
        if (o < P.N) store_elem(P.y, (long long)(r0 + (rest >> 4)) * P.ys + o, P.ydt, v);
      }
    }
  }
  cp_async_wait_group<0>();
}

}  // namespace cpk

// -------------------------------------------------------------- host side
namespace cpk_host {

using namespace cpk;

cudaError_t ops4_smem_limit(const void* fn, size_t bytes) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, size_t> high;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  size_t& h = high[std::make_pair(dev, fn)];
  if (bytes <= h) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) h = bytes;
  return e;
}

size_t w4_bytes(int N, int K, int group) {
  const size_t tiles = (size_t)((N + 15) / 16) * ((K + kW4TileK - 1) / kW4TileK);
  return tiles * w4_tile_bytes(group);
}

static unsigned tile_blocks(int N, int K) {
  const long long tiles = (long long)((N + 15) / 16) * ((K + kW4TileK - 1) / kW4TileK);
  return (unsigned)((tiles + 7) / 8);
}

cudaError_t launch_w4_pack(int N, int K, int group, int dtype, const void* w, long long stride, void* packed, cudaStream_t s) {
  const bool vec = stride * elem_bytes(dtype) % 16 == 0;
  w4_pack_kernel<<<tile_blocks(N, K), 256, 0, s>>>(w, dtype, stride, vec, N, K, (K + kW4TileK - 1) / kW4TileK, group,
                                                   static_cast<unsigned char*>(packed));
  return cudaGetLastError();
}

cudaError_t launch_w4_unpack(int N, int K, int group, int dtype, const void* packed, void* w, cudaStream_t s) {
  w4_unpack_kernel<<<tile_blocks(N, K), 256, 0, s>>>(static_cast<const unsigned char*>(packed), N, K,
                                                     (K + kW4TileK - 1) / kW4TileK, group, w, dtype);
  return cudaGetLastError();
}

// Shared memory of one CTA: the columns of x, the rings, the K shares of two
// groups of outputs, the powers of two.
static size_t w4_smem(W4Gemv& P, int terms) {
  size_t at = (size_t)P.rb * terms * P.XS;
  P.ring_at = (int)at;
  at += (size_t)kW4Warps * kW4Stages * w4_tile_bytes(P.group);
  P.red_at = (int)at;
  if (P.wk > 1) at += (size_t)2 * kW4Warps * 16 * P.rb * 4;
  P.fac_at = (int)at;
  at += (size_t)P.KB * P.rb * 4;
  return (at + 127) / 128 * 128;
}

constexpr size_t kW4SmemMax = 227 * 1024;

cudaError_t launch_w4_gemv(int R, int N, int K, int group, int xdt, int ydt, const void* x, long long xs, const void* packed,
                           void* y, long long ys, int sms, cudaStream_t s) {
  W4Gemv P{};
  P.x = x; P.w = static_cast<const unsigned char*>(packed); P.y = y;
  P.xs = xs; P.ys = ys;
  P.R = R; P.N = N; P.K = K; P.group = group; P.xdt = xdt; P.ydt = ydt;
  P.KB = (K + kW4TileK - 1) / kW4TileK;
  P.XS = P.KB * 256 + 64;  // neighbouring columns half a bank row apart: a quarter warp's 16-byte reads meet no conflict
  P.xvec = xs * elem_bytes(xdt) % 16 == 0;
  const int terms = xdt == kF32 ? 2 : 1;
  // rows of x per CTA: as many as there are, up to 32 columns, that fit beside the rings
  int rb = std::min(R, 32 / terms);
  for (;; rb = (rb + 1) / 2) {
    P.rb = rb;
    P.wk = kW4Warps;
    if (w4_smem(P, terms) <= kW4SmemMax) break;
    if (rb == 1) return cudaErrorInvalidValue;
  }
  const int rblocks = (R + rb - 1) / rb;
  P.rb = rb = (R + rblocks - 1) / rblocks;
  const int cols = rb * terms, NT = cols <= 8 ? 1 : (cols <= 16 ? 2 : 4);
  const int tiles = (N + 15) / 16;
  // Warps that split K: the fewest that still give every resident CTA a group
  // of tiles (no shares to add, no barrier), all eight when tiles are scarce.
  const int regs_ctas = NT == 1 ? 3 : (NT == 2 ? 2 : 1);
  int wk = 1, ctas = 1;
  size_t smem = 0;
  for (;; wk *= 2) {
    P.wk = wk;
    smem = w4_smem(P, terms);
    ctas = (int)std::max<size_t>(1, std::min<size_t>(regs_ctas, kW4SmemMax / (smem + 1024)));
    const int wm = kW4Warps / wk;
    if (wk == kW4Warps || 2 * wk > P.KB || (long long)((tiles + wm - 1) / wm) * rblocks >= (long long)sms * ctas) break;
  }
  const int wm = kW4Warps / wk, groups = (tiles + wm - 1) / wm;
  const int slots = std::max(1, sms * ctas / rblocks);
  const int per = (groups + slots - 1) / slots;
  const dim3 grid((groups + per - 1) / per, rblocks);
  const void* fn = nullptr;
  if (terms == 2) fn = NT == 1 ? (const void*)w4_gemv_kernel<1, 2> : (NT == 2 ? (const void*)w4_gemv_kernel<2, 2> : (const void*)w4_gemv_kernel<4, 2>);
  else fn = NT == 1 ? (const void*)w4_gemv_kernel<1, 1> : (NT == 2 ? (const void*)w4_gemv_kernel<2, 1> : (const void*)w4_gemv_kernel<4, 1>);
  cudaError_t e = ops4_smem_limit(fn, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {&P};
  return cudaLaunchKernel(fn, grid, dim3(kW4Threads), args, smem, s);
}

}  // namespace cpk_host
