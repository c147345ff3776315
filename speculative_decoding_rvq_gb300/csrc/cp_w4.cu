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
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include "cp_ops4.h"
#include "cp_w4.cuh"

namespace cpk {

// ---------------------------------------------------------- pack, unpack
// One warp per tile: each lane takes four consecutive columns of each of the
// 16 rows, and the lanes of a group share its largest magnitude.  Runs once
// per matrix, and is bound by the chain of a row's load, shuffles and quotients
// (65536 x 4096 bfloat16 in groups of 32: 378 us, floor 101; the way back, with
// two-byte stores, 151 us).
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
// walks over groups of 16-row tiles of w: WK of its warps split its share of
// K, the other factor takes neighbouring tiles; the CTAs of a cluster split K
// further.  A warp streams its tiles through a ring of kW4Stages asynchronous
// copies in shared memory, turns codes into fp16 (exact), and multiplies them
// with the rows of x, which are the N operand (8 columns per MMA).  Shares of
// K are added in a fixed order through (distributed) shared memory.
//
// The rows of x are held as fp16, each block of 128 columns scaled by a power
// of two that the result is scaled back by: bfloat16 and fp16 inputs exactly
// (down to 2^-29 of the block's largest magnitude), float32 inputs as two
// columns hi + lo, 22 bits.  The MMAs accumulate one group in float32; the
// group's scale and the block's power of two are applied in float32, so the
// tensor core's truncating accumulation never runs over more than a group.
//
// Bound: for a large matrix and a row the latency of conversions and MMAs, and
// how the tiles divide over the SMs: 1 x 65536 x 4096 in groups of 128 takes 28.7
// us, 4.8 TB/s, 71 % of the measured bandwidth (137 instructions per tile, 56 of
// them to convert its codes; issue slots 61 %, ALU 47 % busy).  Its 512 groups of
// tiles go to 256 CTAs, so the busiest SM works 1.12 times the mean; 77824 rows,
// four groups on each SM, run at 5.5 TB/s, 116736 at 5.8.  Deep rings rather than
// wide tiles keep the bytes streaming; the A operand is built in registers straight
// from the codes, so nothing but x and the copies goes through shared memory.  Small
// products are a chain of latencies (1 x 4096 x 1024: 3.7 us), those with many
// columns are bound by the conversion of x, which every CTA does for its share
// of K (8 x 2048 x 6144: 6.7 us, 15 us without the cluster's split), and by
// instruction latency and shares (64 x 12288 x 2048: 24.9 us, the weights
// converted again for every 16 rows; 9728 rows 18.8 us).
struct W4Gemv {
  const void* x;
  const unsigned char* w;
  void* y;
  long long xs, ys;  // row strides, in elements
  int R, N, K, KB;
  int xdt, ydt;
  int rb;       // rows of x per CTA
  int XS;       // bytes of one column of x in shared memory
  int wk, ck;   // warps of a CTA and CTAs of a cluster that split K
  int ring_at, red_at, fac_at;  // shared-memory offsets
  bool xvec;
};

template <int NT, int TERMS, int NS>
__global__ void __launch_bounds__(kW4Threads, NT == 1 ? 3 : (NT == 2 ? 2 : 1)) w4_gemv_kernel(const __grid_constant__ W4Gemv P) {
  constexpr int TB = 1024 + 32 * NS, MT = w4_mt(NT), ST = w4_stages(NT);
  extern __shared__ __align__(128) unsigned char sm[];
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int WK = P.wk, CK = P.ck, WM = kW4Warps / WK, wk = warp % WK, wm = warp / WK;
  const int cr = CK > 1 ? (int)blockIdx.x % CK : 0, cx = (int)blockIdx.x / CK, gx = (int)gridDim.x / CK;
  const int r0 = blockIdx.y * P.rb, rows = min(P.rb, P.R - r0), cols = rows * TERMS;
  const int tiles = (P.N + 15) / 16, groups = (tiles + WM * MT - 1) / (WM * MT);  // groups of WM * MT neighbouring tiles
  const int shares = CK * WK, share = cr * WK + wk;
  const int kb0 = (int)((long long)P.KB * share / shares), nb = (int)((long long)P.KB * (share + 1) / shares) - kb0;
  const int cb0 = (int)((long long)P.KB * cr / CK), cnb = (int)((long long)P.KB * (cr + 1) / CK) - cb0;  // the CTA's blocks
  const int mine = (groups - cx + gx - 1) / gx;  // groups of this CTA
  unsigned char* ring = sm + P.ring_at + (size_t)warp * ST * MT * TB;
  float* fac = reinterpret_cast<float*>(sm + P.fac_at);  // [blocks of the CTA][rb] powers of two
  float* red = reinterpret_cast<float*>(sm + P.red_at);  // [2][8 warps][MT][rb][16]

  // copies: this warp's tiles of each group, block by block; a tile past the matrix copies nothing
  int left = nb;  // blocks left in the tiles being copied
  int ctile = (cx * WM + wm) * MT, cslot = 0;
  const long long tile_stride = (long long)P.KB * TB;
  const unsigned char* src = P.w + ctile * tile_stride + (long long)kb0 * TB + lane * 16;
  const long long jump = gx * WM * MT * tile_stride - (long long)nb * TB;
  auto issue = [&]() {
    if (ctile < tiles) {
      unsigned char* dst = ring + cslot * (MT * TB) + lane * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (m == 0 || ctile + m < tiles) {
          const unsigned char* from = src + m * tile_stride;
          cp_async16(dst + m * TB, from);
          cp_async16(dst + m * TB + 512, from + 512);
          if (lane < 2 * NS) cp_async16(dst + m * TB + 1024, from + 1024);
        }
      src += TB;
      if (--left == 0) {
        left = nb;
        src += jump;
        ctile += gx * WM * MT;
      }
    }
    cslot = cslot + 1 == ST ? 0 : cslot + 1;
    cp_async_commit();
  };
#pragma unroll 1
  for (int q = 0; q < ST - 1; ++q) issue();

  // x: one warp per (row, two blocks of 128 columns), eight elements a lane
  {
    constexpr int U = NT == 4 ? 8 : 4;
    const unsigned pairs = (cnb + 1) / 2, inverse = 0xFFFFFFFFu / pairs + 1u;  // u / pairs by a product (u * pairs < 2^32)
    const int units = rows * (int)pairs;
    const long long row_bytes = P.xs * (TERMS == 2 ? 4 : 2);
    const unsigned char* x0 = static_cast<const unsigned char*>(P.x) + r0 * row_bytes;
    const int kl0 = lane >> 4, at = (lane & 15) * 8;
    for (int u0 = warp; u0 < units; u0 += U * kW4Warps) {
      uint32_t v[U][TERMS == 2 ? 8 : 4];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const unsigned u = u0 + i * kW4Warps, r = pairs == 1 ? u : __umulhi(u, inverse);
        if ((int)u < units) load8<TERMS>(x0 + r * row_bytes, (cb0 + 2 * (int)(u - r * pairs) + kl0) * kW4TileK + at, P.K, P.xvec, v[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const unsigned u = u0 + i * kW4Warps, r = pairs == 1 ? u : __umulhi(u, inverse);
        if ((int)u >= units) break;
        const int kl = 2 * (int)(u - r * pairs) + kl0;
        uint4 hi, lo;
        const float down = convert8<TERMS>(v[i], P.xdt == kBF16, &hi, &lo);
        if (kl < cnb) {
          unsigned char* dst = sm + (int)r * TERMS * P.XS + kl * 256 + at * 2;
          *reinterpret_cast<uint4*>(dst) = hi;
          if (TERMS == 2) *reinterpret_cast<uint4*>(dst + P.XS) = lo;
          if (at == 0) fac[kl * P.rb + r] = down;
        }
      }
    }
  }
  __syncthreads();

  // columns of x: this lane's column as B operand, and the rows of its two
  // accumulator columns (a column past the rows repeats the last one and is
  // never stored)
  const unsigned char* xcol[NT];
  const float* fcol[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xcol[n] = sm + (size_t)min(n * 8 + g, cols - 1) * P.XS + (kb0 - cb0) * 256 + t * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) fcol[n][c] = fac + (kb0 - cb0) * P.rb + min(n * 8 + 2 * t + c, cols - 1) / TERMS;
  }

  int slot = 0;
#pragma unroll 1
  for (int j = 0; j < mine; ++j) {
    const int tile = ((cx + j * gx) * WM + wm) * MT;
    float tot[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) tot[m][n][c] = 0.0f;
    if (tile < tiles)
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const unsigned char* st = ring + slot * (MT * TB);
        slot = slot + 1 == ST ? 0 : slot + 1;
        W4Codes<MT, NS> A;
        A.load(st, lane);
        __syncwarp();  // every lane has read the stage that the next copy may reuse
        issue();
        w4_block<MT, NT, NS>(A, xcol, b * 256, fcol, b * P.rb, tot);
      }
    // the tiles' outputs: hi and lo columns of a row sit in one thread
    float* part = red + ((j & 1) * kW4Warps + warp) * (MT * 16) * P.rb;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2 / TERMS; ++c) {
            const int row = g + 8 * h, r = (n * 8 + 2 * t) / TERMS + c;
            const float v = TERMS == 2 ? tot[m][n][2 * h] + tot[m][n][2 * h + 1] : tot[m][n][2 * h + c];
            if (r < rows) {
              if (shares == 1) {
                const int o = (tile + m) * 16 + row;
                if (o < P.N) store_elem(P.y, (long long)(r0 + r) * P.ys + o, P.ydt, v);
              } else {
                part[(m * P.rb + r) * 16 + row] = v;
              }
            }
          }
    if (shares > 1) {  // add the shares of K in order; the buffer of this parity is free again two groups on
      const int outs = rows * 16 * WM * MT;
      const float* from = red + (j & 1) * kW4Warps * (MT * 16) * P.rb;
      if (CK == 1) __syncthreads();
      else cg::this_cluster().sync();
      for (int i = cr * kW4Threads + tid; i < outs; i += CK * kW4Threads) {
        const int m = i / (rows * 16), rest = i - m * rows * 16;  // m: tile of the group; rest = r * 16 + row
        const float* at = from + ((m / MT) * WK * MT + m % MT) * 16 * P.rb + rest;
        float v = 0.0f;
        if (CK == 1) {
          for (int k = 0; k < WK; ++k) v += at[k * (MT * 16) * P.rb];
        } else {
          float f[8];
          for (int k = 0; k < WK; ++k) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < CK) f[q] = *cg::this_cluster().map_shared_rank(at + k * (MT * 16) * P.rb, q);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < CK) v += f[q];
          }
        }
        const long long o = (((long long)cx + (long long)j * gx) * (WM * MT) + m) * 16 + (rest & 15);
        if (o < P.N) store_elem(P.y, (long long)(r0 + (rest >> 4)) * P.ys + o, P.ydt, v);
      }
    }
  }
  cp_async_wait_group<0>();
  if (CK > 1) cg::this_cluster().sync();  // no CTA leaves while another reads its shared memory
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
  try {  // (nothing is thrown across the C entry)
    std::lock_guard<std::mutex> lock(mu);
    size_t& h = high[std::make_pair(dev, fn)];
    if (bytes <= h) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) h = bytes;
    return e;
  } catch (...) {
    return cudaErrorMemoryAllocation;
  }
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
static int w4_columns(const W4Gemv& P, int terms) {
  const int cols = P.rb * terms;
  return cols <= 8 ? 1 : (cols <= 16 ? 2 : 4);
}
static size_t w4_smem(W4Gemv& P, int terms, int tile_bytes) {
  const int blocks = (P.KB + P.ck - 1) / P.ck, NT = w4_columns(P, terms), MT = w4_mt(NT);
  // neighbouring columns half a bank row apart: a quarter warp's 16-byte reads meet no conflict
  P.XS = blocks * 256 + 64;
  size_t at = (size_t)P.rb * terms * P.XS;
  P.ring_at = (int)at;
  at += (size_t)kW4Warps * w4_stages(NT) * MT * tile_bytes;
  P.red_at = (int)at;
  if (P.wk * P.ck > 1) at += (size_t)2 * kW4Warps * MT * 16 * P.rb * 4;
  P.fac_at = (int)at;
  at += (size_t)blocks * P.rb * 4;
  return (at + 127) / 128 * 128;
}

// Estimated time of a plan in clocks, fitted to times of 16 shapes (1 to 64
// rows, matrices of 2 to 270 million weights) under every split of K: the
// conversion of x, which every CTA does, in batches of loads; `per` groups of
// tiles of `blocks` blocks each, bound by a block's latency or by what the
// SM's warps issue; the joins of the shares of K.  `share`: CTAs on an SM.
static long long w4_cost(const W4Gemv& P, int NT, int per, int blocks, int share) {
  const int units = P.rb * (((P.KB + P.ck - 1) / P.ck + 1) / 2), batch = (NT == 4 ? 8 : 4) * kW4Warps;
  const int load = NT == 4 ? 2450 : 1300, lat = NT == 1 ? 470 : (NT == 2 ? 700 : 1770), thr = NT == 1 ? 340 : (NT == 2 ? 420 : 2010);
  const long long prep = (long long)(units + batch - 1) / batch * load * (3 + share) / 4 + units * 18 * share;
  const long long outs = (long long)P.rb * 16 * (kW4Warps / P.wk) * w4_mt(NT);
  const long long join = P.ck > 1 ? 1860 + outs * P.wk * 228 / 256 : (P.wk > 1 ? 760 + outs * P.wk * 240 / 256 : 0);
  return prep + per * ((long long)blocks * std::max(lat, thr * share) + join);
}

constexpr size_t kW4SmemMax = 227 * 1024;

// How a product is laid out: rows of x per CTA (up to 32 columns; halved where
// that pays or has to be for x to fit), CTAs of a cluster and warps of a CTA
// that split K, CTAs along the tiles.
struct W4Plan {
  int rb, ck, wk, grid;
};

static W4Plan w4_plan(int R, int N, int K, int group, int terms, int sms) {
  W4Gemv P{};
  P.KB = (K + kW4TileK - 1) / kW4TileK;
  const int tb = w4_tile_bytes(group), rb_max = std::min(R, 32 / terms);
  W4Plan best{};
  long long best_cost = -1;
  for (int rb = rb_max; rb >= 1; rb = rb == 1 ? 0 : (rb + 1) / 2) {
    if (best_cost >= 0 && rb * 4 <= rb_max) break;
    const int rblocks = (R + rb - 1) / rb;
    P.rb = (R + rblocks - 1) / rblocks;
    const int NT = w4_columns(P, terms), MT = w4_mt(NT), most = NT == 1 ? 3 : (NT == 2 ? 2 : 1);
    for (P.ck = 1; P.ck <= 8 && P.ck <= P.KB; P.ck *= 2)
      for (P.wk = 1; P.wk <= kW4Warps && P.wk * P.ck <= P.KB; P.wk *= 2) {
        const size_t smem = w4_smem(P, terms, tb);
        if (smem > kW4SmemMax) continue;
        const int ctas = (int)std::max<size_t>(1, std::min<size_t>(most, kW4SmemMax / (smem + 1024)));
        const int rows = kW4Warps / P.wk * MT * 16, groups = (N + rows - 1) / rows;
        const int slots = std::max(1, sms * ctas / (rblocks * P.ck)), per = (groups + slots - 1) / slots;
        const int grid = (groups + per - 1) / per * P.ck;
        const int share = (int)std::min<long long>(ctas, ((long long)grid * rblocks + sms - 1) / sms);
        const long long cost = w4_cost(P, NT, per, (P.KB + P.ck * P.wk - 1) / (P.ck * P.wk), share);
        if (best_cost < 0 || cost < best_cost) {
          best_cost = cost;
          best = W4Plan{P.rb, P.ck, P.wk, grid};
        }
      }
  }
  return best;  // (one row of the longest K always fits: rb is never 0)
}

// The same few shapes come again with every pass: a thread keeps their plans.
static W4Plan w4_plan_cached(int R, int N, int K, int group, int terms, int sms) {
  struct Entry {
    int R, N, K, group, terms, sms;
    W4Plan plan;
  };
  static thread_local Entry kept[32];
  const unsigned hash = ((unsigned)R * 2654435761u ^ (unsigned)N * 2246822519u ^ (unsigned)K * 3266489917u ^ (unsigned)(group + terms)) >> 27;
  Entry& e = kept[hash];
  if (e.R != R || e.N != N || e.K != K || e.group != group || e.terms != terms || e.sms != sms)
    e = Entry{R, N, K, group, terms, sms, w4_plan(R, N, K, group, terms, sms)};
  return e.plan;
}

template <int NT, int TERMS>
static const void* w4_fn_ns(int group) {
  if (group == 32) return (const void*)w4_gemv_kernel<NT, TERMS, 4>;
  if (group == 64) return (const void*)w4_gemv_kernel<NT, TERMS, 2>;
  return (const void*)w4_gemv_kernel<NT, TERMS, 1>;
}
template <int TERMS>
static const void* w4_fn(int NT, int group) {
  return NT == 1 ? w4_fn_ns<1, TERMS>(group) : (NT == 2 ? w4_fn_ns<2, TERMS>(group) : w4_fn_ns<4, TERMS>(group));
}

cudaError_t launch_w4_gemv(int R, int N, int K, int group, int xdt, int ydt, const void* x, long long xs, const void* packed,
                           void* y, long long ys, int sms, cudaStream_t s) {
  W4Gemv P{};
  P.x = x; P.w = static_cast<const unsigned char*>(packed); P.y = y;
  P.xs = xs; P.ys = ys;
  P.R = R; P.N = N; P.K = K; P.xdt = xdt; P.ydt = ydt;
  P.KB = (K + kW4TileK - 1) / kW4TileK;
  P.xvec = xs * elem_bytes(xdt) % 16 == 0;
  const int terms = xdt == kF32 ? 2 : 1, tb = w4_tile_bytes(group);
  const W4Plan plan = w4_plan_cached(R, N, K, group, terms, sms);
  P.rb = plan.rb;
  P.ck = plan.ck;
  P.wk = plan.wk;
  const size_t smem = w4_smem(P, terms, tb);
  const int NT = w4_columns(P, terms);
  const void* fn = terms == 2 ? w4_fn<2>(NT, group) : w4_fn<1>(NT, group);
  cudaError_t e = ops4_smem_limit(fn, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.grid, (R + P.rb - 1) / P.rb);
  cfg.blockDim = dim3(kW4Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = P.ck;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = P.ck > 1 ? 1 : 0;
  void* args[] = {&P};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace cpk_host
