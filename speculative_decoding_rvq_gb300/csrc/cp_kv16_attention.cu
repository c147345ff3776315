// cp_kv16_attention.cu -- attention over the 16-bit paged KV cache for few
// rows a sequence (single tokens, verify windows, small draft trees), and for any
// number of rows with 256 channels, where the tiles of cp_kv16_prompt.cu do not
// fit their memory.
//
//   o = softmax(scale q k^T) v over the positions that a row sees.
//
// A CTA takes 16 WM packed rows (rows x query heads of one KV head) of one
// sequence and a share of its tiles of 64 positions.  One warp brings tiles in
// by TMA (boxes of 64 channels x up to 64 tokens of one page, 128-byte swizzle)
// through a ring of stages; four warps compute: WM along the rows times WN = 4 /
// WM along the positions of a tile, each with its own running maximum and sum,
// joined at the end in shared memory.  With few rows the keys' and values' bytes bound it, so
// the ring's depth is what counts: three stages of 32 KB (128 channels) and two
// CTAs an SM keep about 190 KB in flight there.  A sequence is split over several CTAs
// where there are too few for the SMs; a second kernel, started while the first
// one runs, joins their shares.  Measured: 64 sequences of up to 4000 positions, 7
// rows, 16 / 8 heads x 128: 134 us, 5.9 TB/s (88 % of a copy's rate; 512 CTAs in
// not quite two waves); one row over a window of 4096, 32 / 8 heads: 9.7 us, a
// chain of latencies (lengths, pages, tiles, two products, join).
//
// Weights enter the product with the values as a sum of two 16-bit numbers (16
// bits of bfloat16 pairs; 22 of fp16, whose weights reach 2^15 so that they have
// steps of 2^-39 of the largest): the second MMA hides behind the copies.
// Blocks of 64 rows (256 channels only) are bound by the MMAs: one number there,
// as in the tiles of cp_kv16_prompt.cu (two are half as many MMAs again).  2048
// rows over 4096 positions, 16 / 4 heads x 256: 770 us, 134 TFLOP/s, about what
// mma.sync gives on this card; 1246 us with each load right before its product.
//
// A position that a row does not see never reaches it: its score is replaced
// by -infinity, so its weight is zero, and values that are infinite or NaN
// are replaced by zeros in every tile that some row of the block does not see
// whole.  Rows that do see such a value get it at the end, from the cache (in a
// whole tile, too: an infinity times the second term of a weight may be a NaN).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "cp_kv16.cuh"
#include "cp_kv16_prompt.h"
#include "cp_ops4.h"

namespace cpk {

constexpr int kFewTile = 64;
// Packed rows up to which this kernel is taken; above, the tiles of
// cp_kv16_prompt.cu (us of both, 8 sequences of 4000 positions, 8 KV heads: 128
// channels 16 rows 30.3 and 34.7, 24 rows 45.5 and 35.0; 64 channels 32 rows 29.6
// and 30.7, 48 rows 54.6 and 31.0).
constexpr int few_most(int d) { return d == 64 ? 32 : (d == 128 ? 16 : 1 << 30); }
constexpr int kFewThreads = 160;  // four warps of rows, one of copies

__host__ __device__ constexpr int few_stage_bytes(int d) { return 2 * kFewTile * d * 2; }
__host__ __device__ constexpr int few_stages(int d) { return d == 64 ? 6 : 3; }
__host__ __device__ constexpr size_t few_smem(int d, int wm) {
  return 1024 + (size_t)few_stages(d) * few_stage_bytes(d) + (size_t)wm * 16 * d * 2;
}

struct FewShared {
  uint64_t full[6], empty[6];
  float m[4][16], l[4][16];
  uint32_t held[6];  // bit g: the page of positions 16 g .. 16 g + 15 of the stage's tile exists
  uint32_t odd[32];  // values that are not finite, by eight channels (kv16_odd), of the tiles that all rows see
  int abort, bad, shown;
};

template <bool BF>
__device__ __forceinline__ void few_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void few_ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void few_ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// 16-byte piece `chunk` of row `row` in a tile of `rows` rows: halves of 64 channels, 128-byte swizzle.
__device__ __forceinline__ uint32_t few_at(uint32_t tile, int rows, int row, int chunk) {
  return tile + (uint32_t)((chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

template <int D, int WM, bool BF>
__global__ void __launch_bounds__(kFewThreads, D == 256 ? 1 : 2) kv16_few_kernel(const __grid_constant__ Kv16Call P) {
  constexpr int WN = 4 / WM, TW = kFewTile / WN, STAGES = few_stages(D), SB = few_stage_bytes(D), HALVES = D / 64, ROWS = 16 * WM;
  constexpr bool TWO = WM < 4;  // terms of a weight
  extern __shared__ __align__(1024) unsigned char few_raw[];
  __shared__ FewShared sh;
  unsigned char* smem = few_raw + ((1024u - (smem_u32(few_raw) & 1023u)) & 1023u);
  unsigned char* qsm = smem + STAGES * SB;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x % P.splits, mt = blockIdx.x / P.splits, h = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Kv16Seq s = kv16_seq(P, b);
  const int r0 = mt * ROWS, packed = s.m * P.group;
  if (r0 >= packed) return;
  const int i0 = r0 / P.group, i1 = (min(r0 + ROWS, packed) - 1) / P.group;
  const Kv16Tiles T = kv16_tiles<kFewTile>(P, s, i0, i1);
  const int k0 = (int)((long long)T.n * split / P.splits), k1 = (int)((long long)T.n * (split + 1) / P.splits);

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 4);
    }
    sh.abort = sh.bad = sh.shown = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == 4) {
    // ================= copies
    const int end = P.mask ? s.len : min(s.len, s.base + i1 + 1);
    Kv16Pages<kFewTile> pages;
    pages.start(P, b, T, k0, k1 - k0, end, lane);
    bool ok = true;
    int issued = k0;
    const int copied = P.stall == 0 ? k1 : (P.stall == 1 ? max(k0, k1 - 1) : k0);
#pragma unroll 1
    for (int k = k0; k < copied; ++k) {
      const int st = (k - k0) % STAGES, turn = (k - k0) / STAGES;
      const int id = pages.of(P, b, T, k0, k1 - k0, end, k - k0, lane), lane0 = ((k - k0) & (pages.each - 1)) * pages.per;
      const uint32_t held = pages.held(id, k - k0);
      if (turn > 0) ok = __all_sync(0xffffffffu, kv16_wait(&sh.empty[st], (uint32_t)(turn - 1) & 1u, &sh.abort, P.wait_ns));
      if (!ok) break;
      if (lane == 0) {
        sh.held[st] = held;
        mbar_arrive_expect_tx(&sh.full[st], SB);
      }
      __syncwarp();
      // a lane a box: keys or values, 64 channels of `half`, tokens `piece` (one lane for all boxes takes twice as long)
      const int piece = lane & (pages.per - 1), e = lane / pages.per, half = e & (HALVES - 1), page = __shfl_sync(0xffffffffu, id, lane0 + piece);
      if (e < 2 * HALVES) {
        const bool is_v = e >= HALVES;
        const int t0 = T.tile(k) * kFewTile + piece * pages.box;
        // (a page that does not exist: the box past the last page, which reads as zeros)
        kv16_box(smem_u32(smem + st * SB + (is_v ? SB / 2 : 0) + half * (kFewTile * 128) + piece * pages.box * 128), is_v ? &P.vmap : &P.kmap, half * 64,
                 page >= 0 ? (h << P.page_shift) + (t0 & ((1 << P.page_shift) - 1)) : 0, page >= 0 ? page : P.n_pages, smem_u32(&sh.full[st]));
      }
      __syncwarp();
      issued = k + 1;
    }
    __syncthreads();
    if (sh.abort)  // nothing in flight at exit: whoever gave up, copies may not have landed
      for (int k = max(k0, issued - STAGES); k < issued; ++k) kv16_drain(&sh.full[(k - k0) % STAGES], (uint32_t)((k - k0) / STAGES) & 1u);
    return;
  }

  // ================= rows
  const int wm = warp / WN, wn = warp % WN, g = lane >> 2, t = lane & 3;
  // queries to shared memory, swizzled like the keys
  for (int e = tid; e < ROWS * (D / 8); e += 128) {
    const int row = e / (D / 8), c = e % (D / 8), r = r0 + row;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < packed) {
      const int i = r / P.group;
      const unsigned short* src = P.q + (long long)(s.start + i) * P.qs + (long long)(h * P.group + (r - i * P.group)) * D + 8 * c;
      if (P.qvec) v = __ldg(reinterpret_cast<const uint4*>(src));
      else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = src[2 * j] | (uint32_t)src[2 * j + 1] << 16;
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *reinterpret_cast<uint4*>(qsm + few_at(0, ROWS, row, c)) = v;
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  const uint32_t qb = smem_u32(qsm), kb = smem_u32(smem);
  const int mid = lane >> 3, mr = lane & 7;
  constexpr bool QREG = D <= 128 && WM < 4;  // (else reloaded for every tile: the registers go to the sums)
  uint32_t qf[QREG ? D / 16 : 1][4];
  if (QREG) {
#pragma unroll
    for (int kk = 0; kk < (QREG ? D / 16 : 1); ++kk) few_ldsm(qf[kk], few_at(qb, ROWS, wm * 16 + (mid & 1) * 8 + mr, kk * 2 + (mid >> 1)));
  }
  Kv16Row rows[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + wm * 16 + g + 8 * e;
    rows[e] = kv16_row(P, s, r < packed ? r / P.group : -1);
  }
  float O[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) O[n][j] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  bool ok = true, bad = false;
  for (int k = k0; k < k1; ++k) {
    const int st = (k - k0) % STAGES;
    ok = kv16_wait(&sh.full[st], (uint32_t)((k - k0) / STAGES) & 1u, &sh.abort, P.wait_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t ks = kb + st * SB, vs = ks + SB / 2;
    const int t0 = T.tile(k) * kFewTile;
    const uint32_t held = *(volatile uint32_t*)&sh.held[st];
    const bool whole = held == 0xFu && kv16_whole<kFewTile>(P, s, i0, i1, t0);
    float S[TW / 8][4];
#pragma unroll
    for (int n = 0; n < TW / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[n][j] = 0.0f;
    // (four loads ahead of the products that wait for them)
    constexpr int NP = TW / 16, KU = 4 / NP;
#pragma unroll
    for (int k4 = 0; k4 < D / 16; k4 += KU) {
      uint32_t a[KU][4], f[KU][NP][4];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int kk = k4 + u;
        if (QREG) {
#pragma unroll
          for (int j = 0; j < 4; ++j) a[u][j] = qf[QREG ? kk : 0][j];
        } else {
          few_ldsm(a[u], few_at(qb, ROWS, wm * 16 + (mid & 1) * 8 + mr, kk * 2 + (mid >> 1)));
        }
#pragma unroll
        for (int np = 0; np < NP; ++np) few_ldsm(f[u][np], few_at(ks, kFewTile, wn * TW + np * 16 + (mid >> 1) * 8 + mr, kk * 2 + (mid & 1)));
      }
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int np = 0; np < NP; ++np) {
          few_mma<BF>(S[2 * np], a[u], f[u][np][0], f[u][np][1]);
          few_mma<BF>(S[2 * np + 1], a[u], f[u][np][2], f[u][np][3]);
        }
    }
    // scores, masked; running maximum
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < TW / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = S[n][j] * P.scale_log2;
        if (!whole) {
          const int at = wn * TW + n * 8 + 2 * t + (j & 1);
          if (!((held >> (at >> 4)) & 1u) || !kv16_sees(P, s, rows[j >> 1], t0 + at)) x = -INFINITY;
        }
        S[n][j] = x;
        top[j >> 1] = fmaxf(top[j >> 1], x);
      }
    float base[2], fade[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      const float next = fmaxf(m[e], kv16_base<BF>(top[e], P.lift));
      base[e] = next == -INFINITY ? 0.0f : next;
      fade[e] = kv16_exp2(m[e] - base[e]);
      m[e] = next;
      l[e] *= fade[e];
    }
    if (__any_sync(0xffffffffu, fade[0] != 1.0f || fade[1] != 1.0f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        O[n][0] *= fade[0]; O[n][1] *= fade[0];
        O[n][2] *= fade[1]; O[n][3] *= fade[1];
      }
    }
#pragma unroll
    for (int n = 0; n < TW / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[n][j] = kv16_exp2(S[n][j] - base[j >> 1]);
        l[j >> 1] += S[n][j];
      }
#pragma unroll
    for (int c = 0; c < TW / 16; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = S[2 * c + (j >> 1)][2 * (j & 1)], y = S[2 * c + (j >> 1)][2 * (j & 1) + 1];
        hi[j] = kv16_pack<BF>(x, y);
        const float2 f = kv16_unpack<BF>(hi[j]);
        lo[j] = TWO ? kv16_pack<BF>(x - f.x, y - f.y) : 0u;
      }
#pragma unroll
      for (int d4 = 0; d4 < D / 16; d4 += 4) {
        uint32_t f[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          few_ldsm_t(f[u], few_at(vs, kFewTile, wn * TW + c * 16 + (mid & 1) * 8 + mr, (d4 + u) * 2 + (mid >> 1)));
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j >> 2][j & 3] = kv16_finite<BF>(f[j >> 2][j & 3], bad);
        }
        if (TWO) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            few_mma<BF>(O[2 * (d4 + u)], lo, f[u][0], f[u][1]);
            few_mma<BF>(O[2 * (d4 + u) + 1], lo, f[u][2], f[u][3]);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          few_mma<BF>(O[2 * (d4 + u)], hi, f[u][0], f[u][1]);
          few_mma<BF>(O[2 * (d4 + u) + 1], hi, f[u][2], f[u][3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[st]);
  }
  if (bad) sh.bad = 1;
  float odd = 0.0f;
#pragma unroll
  for (int n = 0; n < D / 8; ++n) odd += fmaf(O[n][0], 0.0f, O[n][1] * 0.0f) + fmaf(O[n][2], 0.0f, O[n][3] * 0.0f);
  if (odd != 0.0f) sh.shown = 1;
  if (tid < D / 8) sh.odd[tid] = 0;
  if (!ok && P.status) atomicCAS(P.status, 0, kStatusTimeout);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    if (t == 0) {
      sh.m[warp][g + 8 * e] = m[e];
      sh.l[warp][g + 8 * e] = l[e];
    }
  }
  __syncthreads();  // the copies have all landed: the ring is free for the sums of the warps
  if (sh.abort) return;
  float* sums = reinterpret_cast<float*>(smem) + warp * 16 * (D + 4);  // (rows padded against bank conflicts)
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    *reinterpret_cast<float2*>(sums + g * (D + 4) + n * 8 + 2 * t) = make_float2(O[n][0], O[n][1]);
    *reinterpret_cast<float2*>(sums + (g + 8) * (D + 4) + n * 8 + 2 * t) = make_float2(O[n][2], O[n][3]);
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  // Values that are not finite: those left out of tiles that some row does not see whole, and all of them where a sum shows one.
  const bool left = sh.bad != 0, shown = sh.shown != 0;
  if (left || shown) {
    const int c = tid % (D / 8);
    const uint32_t bits = kv16_odd_shared<BF, D, kFewTile>(P, s, T, b, h, i0, i1, k0, k1 - k0, 8 * c, tid / (D / 8), 128 / (D / 8), shown);
    if (bits) atomicOr(&sh.odd[c], bits);
    asm volatile("bar.sync 1, 128;" ::: "memory");
  }
  for (int e = tid; e < ROWS * (D / 8); e += 128) {
    const int row = e / (D / 8), c = e % (D / 8), r = r0 + row;
    if (r >= packed) continue;
    const int w0 = (row >> 4) * WN, rr = row & 15, i = r / P.group, hq = h * P.group + (r - i * P.group);
    float M = sh.m[w0][rr];
#pragma unroll
    for (int w = 1; w < WN; ++w) M = fmaxf(M, sh.m[w0 + w][rr]);
    const float base = M == -INFINITY ? 0.0f : M;
    float x[8] = {}, L = 0.0f;
#pragma unroll
    for (int w = 0; w < WN; ++w) {
      const float f = kv16_exp2(sh.m[w0 + w][rr] - base);
      const float* from = reinterpret_cast<float*>(smem) + ((w0 + w) * 16 + rr) * (D + 4) + 8 * c;
      L += f * sh.l[w0 + w][rr];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += f * from[j];
    }
    if (fabsf(L) < INFINITY && (left || shown)) {  // (with a NaN among the scores the row is NaN anyway)
      uint32_t bits[1] = {sh.odd[c]};
      kv16_odd_own<BF, D, kFewTile, 1>(P, s, kv16_row(P, s, i), T, b, h, i0, i1, k0, k1 - k0, 8 * c, bits);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = kv16_odd_sum(bits[0], j, x[j]);
    }
    const long long at = (long long)(s.start + i) * P.nq + hq;
    if (P.splits > 1) {
      float* w = P.work + ((long long)split * P.n_rows * P.nq + at) * D + 8 * c;
      reinterpret_cast<float4*>(w)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(w)[1] = make_float4(x[4], x[5], x[6], x[7]);
      if (c == 0)
        reinterpret_cast<float2*>(P.work + (long long)P.splits * P.n_rows * P.nq * D)[(long long)split * P.n_rows * P.nq + at] = make_float2(M, L);
    } else {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = kv16_pack<BF>(x[2 * j] * inv, x[2 * j + 1] * inv);
      unsigned short* dst = P.o + (long long)(s.start + i) * P.os + (long long)hq * D + 8 * c;
      if (P.ovec) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      else {
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = (unsigned short)(w[j >> 1] >> (16 * (j & 1)));
      }
      if (c == 0 && P.lse) P.lse[at] = kv16_lse(P, M, L);
    }
  }
}

// The shares of split sequences joined: W warps for each row and query head (four
// where there are more than eight shares), each with up to eight in flight at once.
template <int D, bool BF, int W>
__global__ void __launch_bounds__(128) kv16_join_kernel(const __grid_constant__ Kv16Call P) {
  constexpr int V = D / 32;
  __shared__ float sums[W > 1 ? W : 1][W > 1 ? D : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W, b = blockIdx.y;
  const int id = blockIdx.x * (4 / W) + warp / W, i = id / P.nq, hq = id - i * P.nq;
  const Kv16Seq s = kv16_seq(P, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= s.m) return;  // (W > 1: the whole CTA)
  const long long all = (long long)P.n_rows * P.nq, at = (long long)(s.start + i) * P.nq + hq;
  const float2* ml = reinterpret_cast<const float2*>(P.work + (long long)P.splits * all * D);
  float2 mine = make_float2(-INFINITY, 0.0f);
  if (lane < P.splits) mine = load_l2(ml + lane * all + at);
  float2 v[8][V / 2];
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      v[k][j] = sub + W * k < P.splits ? load_l2(reinterpret_cast<const float2*>(P.work + ((sub + W * k) * all + at) * D + V * lane) + j)
                                       : make_float2(0.0f, 0.0f);
  const float M = warp_max(mine.x);
  const float f = kv16_exp2(mine.x - (M == -INFINITY ? 0.0f : M));
  const float L = warp_sum(lane < P.splits ? f * mine.y : 0.0f), inv = L == 0.0f ? 0.0f : 1.0f / L;
  float x[V] = {};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float w = __shfl_sync(0xffffffffu, f, (sub + W * k) & 31);
    if (sub + W * k < P.splits) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        // (a share whose weight is zero in float32 still hands on an infinity)
        x[2 * j] += w == 0.0f && fabsf(v[k][j].x) == INFINITY ? v[k][j].x : w * v[k][j].x;
        x[2 * j + 1] += w == 0.0f && fabsf(v[k][j].y) == INFINITY ? v[k][j].y : w * v[k][j].y;
      }
    }
  }
  unsigned short* dst = P.o + (long long)(s.start + i) * P.os + (long long)hq * D;
  auto put = [&](int c, float y0, float y1) {
    const uint32_t w = kv16_pack<BF>(y0 * inv, y1 * inv);
    if (P.ovec) *reinterpret_cast<uint32_t*>(dst + c) = w;
    else {
      dst[c] = (unsigned short)w;
      dst[c + 1] = (unsigned short)(w >> 16);
    }
  };
  if (W == 1) {
#pragma unroll
    for (int j = 0; j < V; j += 2) put(V * lane + j, x[j], x[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) sums[sub][W > 1 ? V * lane + j : 0] = x[j];
    __syncthreads();
    for (int c = 2 * threadIdx.x; c < D; c += 256) {
      float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        y0 += sums[k][W > 1 ? c : 0];
        y1 += sums[k][W > 1 ? c + 1 : 0];
      }
      put(c, y0, y1);
    }
  }
  if (sub == 0 && lane == 0 && P.lse) P.lse[at] = kv16_lse(P, M, L);
}

}  // namespace cpk

namespace cpk_host {

using namespace cpk;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

cudaError_t kv16_prepare(const Kv16Shape& S, const Kv16Attention& A, Kv16Call* P) {
  const size_t elems = (size_t)S.n_pages * S.nkv * S.page_size * S.d;
  P->keys = static_cast<const unsigned short*>(A.cache);
  P->values = P->keys + elems;
  P->pages = A.pages; P->kv_len = A.kv_len; P->row_start = A.row_start; P->mask = A.mask;
  P->q = static_cast<const unsigned short*>(A.q);
  P->o = static_cast<unsigned short*>(A.o);
  P->lse = A.lse; P->work = static_cast<float*>(A.work); P->status = A.status;
  P->qs = A.qs; P->os = A.os;
  P->n_pages = S.n_pages; P->page_shift = __builtin_ctz(S.page_size); P->box_shift = std::min(P->page_shift, 6);
  P->nkv = S.nkv; P->max_pages = A.max_pages; P->n_seqs = A.n_seqs; P->n_rows = A.n_rows; P->max_rows = A.max_rows;
  P->nq = A.nq; P->group = A.nq / S.nkv;
  // a window that covers the longest sequence is none
  P->window = (long long)A.window >= (long long)A.max_pages * S.page_size ? 0 : A.window;
  P->sinks = A.sinks;
  P->stall = A.stall;
  P->wait_ns = A.wait_ns;
  P->scale_log2 = (float)((double)A.scale * 1.44269504088896340736);
  // (masked scores are infinities that the factor multiplies; with float32's least number all weights are 1, whatever the products)
  if (P->scale_log2 == 0.0f) P->scale_log2 = 1.401298464e-45f;
  P->qvec = ((uintptr_t)A.q & 15u) == 0 && A.qs % 8 == 0;
  P->ovec = ((uintptr_t)A.o & 15u) == 0 && A.os % 8 == 0;
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)S.d, (cuuint64_t)S.nkv * S.page_size, (cuuint64_t)S.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)S.d * 2, (cuuint64_t)S.nkv * S.page_size * S.d * 2};
  const cuuint32_t box[3] = {64u, 1u << P->box_shift, 1u}, es[3] = {1u, 1u, 1u};
  for (int i = 0; i < 2; ++i)
    if (enc(i ? &P->vmap : &P->kmap, S.dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<unsigned short*>(i ? P->values : P->keys), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  return cudaSuccess;
}

// How a call is dealt: warps along the rows (0: the tensor-core tiles of
// cp_kv16_prompt.cu, in pairs of row blocks or not), blocks of rows, splits of a
// sequence.
struct Kv16Plan {
  int wm, mtiles, splits;
  bool pair;
};
static Kv16Plan kv16_plan(const Kv16Shape& S, const Kv16Attention& A, int sms) {
  Kv16Plan p{};
  const long long packed = (long long)A.max_rows * (A.nq / S.nkv), heads = (long long)A.n_seqs * S.nkv;
  const long long most = (long long)A.max_pages * S.page_size;
  int rows, tile, places;
  if (packed > few_most(S.d)) {
    p.wm = 0;
    tile = 128;
    // two blocks of rows share a CTA's tiles where that fills the SMs
    p.pair = packed > 128 && heads * ((packed + 255) / 256) >= sms;
    rows = p.pair ? 256 : 128;
    places = sms;
  } else {
    p.wm = packed <= 16 ? 1 : (packed <= 32 ? 2 : 4);
    tile = kFewTile;
    rows = 16 * p.wm;
    places = sms * (S.d == 256 ? 1 : 2);
  }
  p.mtiles = (int)((packed + rows - 1) / rows);
  long long seen = most;
  if (A.window > 0) seen = std::min<long long>(most, (long long)A.window + A.sinks + rows + 2 * tile);
  const long long tiles = (seen + tile - 1) / tile, ctas = std::max<long long>(1, heads * p.mtiles);
  // as many shares as fill the SMs once, of two tiles or more
  p.splits = (int)std::max<long long>(1, std::min<long long>({32, places / ctas, tiles / 2}));
  return p;
}

size_t kv16_attention_work(const Kv16Shape& S, const Kv16Attention& A, int sms) {
  const Kv16Plan p = kv16_plan(S, A, sms);
  return p.splits > 1 ? (size_t)p.splits * A.n_rows * A.nq * (S.d + 2) * 4 : 0;
}

template <int D, bool BF>
static cudaError_t attention_launch(const Kv16Call& P, const Kv16Plan& p, int* kernels, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  Kv16Call call = P;
  void* args[] = {&call};
  cudaError_t e;
  *kernels = 1;
  if (D <= 128 && p.wm == 0) {
    e = launch_kv16_prompt(P, D, BF, p.pair, s);
  } else {
    constexpr int W2 = few_most(D) > 16 ? 2 : 1, W4 = few_most(D) > 32 ? 4 : W2;  // (what the rule never reaches is not built)
    const void* fn = p.wm == 1 ? (const void*)kv16_few_kernel<D, 1, BF>
                               : (p.wm == 2 ? (const void*)kv16_few_kernel<D, W2, BF> : (const void*)kv16_few_kernel<D, W4, BF>);
    cfg.gridDim = dim3((unsigned)(p.splits * p.mtiles), (unsigned)P.nkv, (unsigned)P.n_seqs);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = few_smem(D, p.wm);
    cfg.stream = s;
    e = ops4_smem_limit(fn, cfg.dynamicSmemBytes);
    if (e == cudaSuccess) e = cudaLaunchKernelExC(&cfg, fn, args);
  }
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg = cudaLaunchConfig_t{};
  const int each = p.splits > 8 ? 1 : 4;  // rows and heads of a CTA
  cfg.gridDim = dim3((unsigned)(((long long)P.max_rows * P.nq + each - 1) / each), (unsigned)P.n_seqs);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  *kernels = 2;
  return cudaLaunchKernelExC(&cfg, each == 1 ? (const void*)kv16_join_kernel<D, BF, 4> : (const void*)kv16_join_kernel<D, BF, 1>, args);
}

cudaError_t launch_kv16_attention(const Kv16Shape& S, const Kv16Attention& A, int sms, int* kernels, cudaStream_t s) {
  Kv16Call P{};
  cudaError_t e = kv16_prepare(S, A, &P);
  if (e != cudaSuccess) return e;
  const Kv16Plan p = kv16_plan(S, A, sms);
  P.splits = p.splits;
  P.mtiles = p.mtiles;
  const bool bf = S.dtype == 1;
  const float late = p.wm == 0 ? kPromptLate : 0.0f;
  // bfloat16 weights are put so low that no sum of weight * value over the positions a row sees passes the largest value
  // (they, and float32, have the range); fp16's values are far from float32's end, its weights are put high (kv16_base).
  long long seen = (long long)A.max_pages * S.page_size;
  if (P.window > 0) seen = std::min<long long>(seen, (long long)P.window + P.sinks + CP_SPEC_MAX_TREE_ROWS);
  P.lift = bf ? -(late + (float)(64 - __builtin_clzll((unsigned long long)seen))) : 15.0f - late;
  P.unlift = exp2f(-P.lift);
  P.grow = P.lift + late;
  switch (S.d) {
    case 64: return bf ? attention_launch<64, true>(P, p, kernels, s) : attention_launch<64, false>(P, p, kernels, s);
    case 128: return bf ? attention_launch<128, true>(P, p, kernels, s) : attention_launch<128, false>(P, p, kernels, s);
    default: return bf ? attention_launch<256, true>(P, p, kernels, s) : attention_launch<256, false>(P, p, kernels, s);
  }
}

}  // namespace cpk_host
