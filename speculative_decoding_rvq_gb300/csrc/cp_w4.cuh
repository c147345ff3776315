// cp_w4.cuh -- parts that the products with 4-bit weights share: the public
// operator (cp_w4.cu) and the decoder pass of a context over packed weights
// (cp_w4_pass.cu).  The packed layout is described in cp_w4.cu.
#pragma once
#include "cp_fp4.cuh"

namespace cpk {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4TileK = 128;

// Tiles of 16 rows that a warp multiplies at once, by the MMA column tiles NT
// of x: two where there are many columns, so that a fragment of x read from
// shared memory serves two MMAs; and the tiles in flight per warp.
__host__ __device__ constexpr int w4_mt(int NT) { return NT == 4 ? 2 : 1; }
__host__ __device__ constexpr int w4_stages(int NT) { return NT == 4 ? 3 : 6; }
__host__ __device__ inline int w4_groups(int group) { return kW4TileK / group; }  // scales per tile row
__host__ __device__ inline int w4_tile_bytes(int group) { return 1024 + 32 * w4_groups(group); }
// Byte offset of the scale of row i (0..15), group q of a tile.
__device__ __forceinline__ int w4_scale_at(int i, int q, int ns) { return 1024 + (i * ns + q) * 2; }

// Eight consecutive elements of a row as they are stored (16-bit types in the
// first four words), zeros at and past n.
template <int TERMS>
__device__ __forceinline__ void load8(const void* row, int k0, int n, bool vec, uint32_t (&v)[TERMS == 2 ? 8 : 4]) {
  if constexpr (TERMS == 2) {
    const uint32_t* p = static_cast<const uint32_t*>(row) + k0;
    if (vec && k0 + 7 < n) {
      const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + i < n ? p[i] : 0u;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + k0;
    if (vec && k0 + 7 < n) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (k0 + 2 * i < n ? p[2 * i] : 0u) | (k0 + 2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
  }
}

// The second half of a block's conversion: eight elements a lane with the
// largest magnitude (bits) of each lane, half a warp a block, to fp16 scaled by
// a power of two; returns its inverse.  `odd`: some element of the warp is not
// finite (the finite ones set the power).
template <int TERMS>
__device__ __forceinline__ float to_fp16_block(float (&f)[8], uint32_t top, bool odd, uint4* hi, uint4* lo) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  float up, down;
  pow2_normaliser(top, &up, &down);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= up;
  *hi = make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
  if constexpr (TERMS == 2) {
    const uint32_t h[4] = {hi->x, hi->y, hi->z, hi->w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_half2(h[i]);
      float a = f[2 * i] - x.x, c = f[2 * i + 1] - x.y;
      if (odd) {
        a = fp16_rest(f[2 * i]);
        c = fp16_rest(f[2 * i + 1]);
      }
      r[i] = pack_half2(a, c);
    }
    *lo = make_uint4(r[0], r[1], r[2], r[3]);
  }
  return down;
}

// One warp's pair of blocks of a row of x, eight elements a lane, to fp16
// scaled by a power of two per block (half a warp): returns its inverse.
// Where a block holds an infinity or a NaN the finite elements set the power.
template <int TERMS>
__device__ __forceinline__ float convert8(const uint32_t (&v)[TERMS == 2 ? 8 : 4], bool bf16, uint4* hi, uint4* lo) {
  float f[8];
  uint32_t top = 0, limit = 0x7F800000u;  // the largest magnitude's bits, and where the numbers that are not finite begin
  if constexpr (TERMS == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = __uint_as_float(v[i]);
      top = max(top, v[i] & 0x7FFFFFFFu);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top = __vmaxu2(top, v[i] & 0x7FFF7FFFu);
      const float2 x = bf16 ? bf16x2_to_f2(v[i]) : unpack_half2(v[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
    top = max(top & 0xFFFFu, top >> 16);
    limit = bf16 ? 0x7F80u : 0x7C00u;
  }
  const bool odd = __any_sync(0xffffffffu, top >= limit);
  if (odd) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, finite_abs_bits(f[i]));
  } else if (TERMS == 1) {
    top = bf16 ? top << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
  }
  return to_fp16_block<TERMS>(f, top, odd, hi, lo);
}

// The A operands of a block: codes and scales of MT tiles from a ring stage.
template <int MT, int NS>
struct W4Codes {
  uint32_t lw[MT][4], hw[MT][4];                          // codes of rows g and g + 8
  uint32_t slo[MT][(NS + 1) / 2], shi[MT][(NS + 1) / 2];  // their scales, two to a word
  __device__ __forceinline__ void load(const unsigned char* st, int lane) {
    constexpr int TB = 1024 + 32 * NS;
    const int g = lane >> 2;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const unsigned char* T = st + m * TB;
      const uint4 lo4 = *reinterpret_cast<const uint4*>(T + lane * 16);
      const uint4 hi4 = *reinterpret_cast<const uint4*>(T + 512 + lane * 16);
      lw[m][0] = lo4.x; lw[m][1] = lo4.y; lw[m][2] = lo4.z; lw[m][3] = lo4.w;
      hw[m][0] = hi4.x; hw[m][1] = hi4.y; hw[m][2] = hi4.z; hw[m][3] = hi4.w;
      if constexpr (NS == 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(T + w4_scale_at(g, 0, 4));
        const uint2 c = *reinterpret_cast<const uint2*>(T + w4_scale_at(g + 8, 0, 4));
        slo[m][0] = a.x; slo[m][1] = a.y; shi[m][0] = c.x; shi[m][1] = c.y;
      } else if constexpr (NS == 2) {
        slo[m][0] = *reinterpret_cast<const uint32_t*>(T + w4_scale_at(g, 0, 2));
        shi[m][0] = *reinterpret_cast<const uint32_t*>(T + w4_scale_at(g + 8, 0, 2));
      } else {
        slo[m][0] = *reinterpret_cast<const uint16_t*>(T + w4_scale_at(g, 0, 1));
        shi[m][0] = *reinterpret_cast<const uint16_t*>(T + w4_scale_at(g + 8, 0, 1));
      }
    }
  }
};

// One block of 128 columns: tot += (tile values) x (rows of x), with the rows'
// powers of two in fcol.
template <int MT, int NT, int NS>
__device__ __forceinline__ void w4_block(const W4Codes<MT, NS>& A, const unsigned char* const (&xcol)[NT], int x_at,
                                         const float* const (&fcol)[NT][2], int f_at, float (&tot)[MT][NT][4]) {
  float blk[MT][NT][4], acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) blk[m][n][c] = acc[m][n][c] = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t al[MT][4], ah[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      e2m1_to_half2x4(A.lw[m][w], al[m]);
      e2m1_to_half2x4(A.hw[m][w], ah[m]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 x4 = *reinterpret_cast<const uint4*>(xcol[n] + x_at + w * 64);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma_f16_16816(acc[m][n], al[m][0], ah[m][0], al[m][1], ah[m][1], x4.x, x4.y);
        mma_f16_16816(acc[m][n], al[m][2], ah[m][2], al[m][3], ah[m][3], x4.z, x4.w);
      }
    }
    if (((w + 1) & (4 / NS - 1)) == 0) {  // the end of a group
      constexpr int per = 4 / NS;
      const int q = (w + 1) / per - 1;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float a = __uint_as_float((q & 1) ? A.slo[m][q >> 1] & 0xFFFF0000u : A.slo[m][q >> 1] << 16);
        const float c = __uint_as_float((q & 1) ? A.shi[m][q >> 1] & 0xFFFF0000u : A.shi[m][q >> 1] << 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          blk[m][n][0] = fmaf(a, acc[m][n][0], blk[m][n][0]);
          blk[m][n][1] = fmaf(a, acc[m][n][1], blk[m][n][1]);
          blk[m][n][2] = fmaf(c, acc[m][n][2], blk[m][n][2]);
          blk[m][n][3] = fmaf(c, acc[m][n][3], blk[m][n][3]);
          acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float f0 = fcol[n][0][f_at], f1 = fcol[n][1][f_at];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      tot[m][n][0] = fmaf(f0, blk[m][n][0], tot[m][n][0]);
      tot[m][n][1] = fmaf(f1, blk[m][n][1], tot[m][n][1]);
      tot[m][n][2] = fmaf(f0, blk[m][n][2], tot[m][n][2]);
      tot[m][n][3] = fmaf(f1, blk[m][n][3], tot[m][n][3]);
    }
  }
}

}  // namespace cpk
