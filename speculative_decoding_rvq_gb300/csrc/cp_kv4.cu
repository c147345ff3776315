// cp_kv4.cu -- a KV cache held in 4 bits (format of cp_fp4.cuh, one bfloat16
// scale per 32 channels of a token and head): rows written into it, read
// back, and attention over it.
//
// The cache is n_pages pages of page_size token slots; a page table maps the
// positions of a sequence to pages.  Within a page, each head's slots are
// grouped in tiles of 16 tokens, 18 * head_dim bytes each and contiguous, in
// the order in which the m16n8k16 A operand of the attention kernel wants them:
//   keys    [16 tokens][4 lanes t][head_dim / 32 groups] words of 8 codes, the
//           word's byte j holding channels 8 t + 2 j and 8 t + 2 j + 1 of the group;
//   values  [8 token pairs][8 lanes g][head_dim / 32 groups] words of 4 bytes,
//           byte j holding channel 4 g + j of the group, the pair's even token
//           in the low nibble (the values' product sums over tokens, so a pair
//           of tokens makes one fp16x2 operand);
//   scales  [16 tokens][head_dim / 32] of the keys, then of the values.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "cp_fp4.cuh"
#include "cp_ops4.h"

namespace cpk {

constexpr int kKvGroup = 32;

__host__ __device__ inline int kv4_tile_bytes(int d) { return 18 * d; }

// Where positions are: a position's page by the table, its tile within the page.
struct Kv4Map {
  unsigned char* cache;
  const int* pages;  // [B][max_pages], or null: sequence b owns pages b * max_pages ..
  int max_pages, page_size, n_pages, nkv, d;
  int tpp, tpp_shift;     // tiles per page, and its logarithm where it is a power of two (else -1)
  long long page_stride;  // bytes
};

// Page index of a tile of the sequence (a division only where the page size is no power of two).
__device__ __forceinline__ int kv4_page_of_tile(const Kv4Map& M, int tile) {
  return M.tpp_shift >= 0 ? tile >> M.tpp_shift : tile / M.tpp;
}

__device__ __forceinline__ int kv4_page(const Kv4Map& M, int b, int at) {
  if (at >= M.max_pages) return -1;
  const int id = M.pages ? __ldg(M.pages + (long long)b * M.max_pages + at) : b * M.max_pages + at;
  return id >= 0 && id < M.n_pages ? id : -1;
}

__device__ __forceinline__ unsigned char* kv4_tile(const Kv4Map& M, int page, int h, int tile_in_page) {
  return M.cache + page * M.page_stride + (long long)(h * M.tpp + tile_in_page) * kv4_tile_bytes(M.d);  // (a page may pass 2^31 bytes)
}

// ------------------------------------------------------------ write, read
// One thread per (sequence, pair of token slots, 8 channels of a head): the 4
// threads of a scale group are neighbours in a warp, so are the groups of a
// row, and a row's loads and stores coalesce.  A pair shares the bytes of its
// value codes; where only one of its tokens is written the other's nibbles
// are left by an atomic exclusive-or of the nibbles that change (another
// sequence, or another call, may be writing them).  Bound by the bytes of the
// rows at a few of them, by the quotients at many (16-byte loads and quotients
// of three instructions; 4 x 8192 tokens of 8 x 128 channels: bfloat16 58.6 us,
// 2.9 TB/s, float32 with twice the bytes 60.7 us, 5.0 TB/s; 113 us for bfloat16
// with 4 channels a thread, 8-byte loads and packed nibbles spread for the values).
struct Kv4Rows {
  Kv4Map map;
  const void* k;
  const void* v;
  void* ko;
  void* vo;
  long long ks, vs;  // row strides in elements
  const int* pos;    // first position of each sequence (append), null in read
  const int* len;    // rows of each sequence that count, or null
  int B, M, npairs, chunks, dtype;  // chunks: of 8 channels, per row
  bool kvec, vvec;
};

// a / b for a scale b of ordinary size, correctly rounded, from the
// correctly rounded reciprocal y of b: q = a y, then q + (a - q b) y with fused
// multiply-adds (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990).
__device__ __forceinline__ float quotient_by(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

// Eight channels of one row (float32 bits, or 16-bit types two to a word) to
// float quotients by their group's scale, whose bits are returned; the 4 lanes
// of a group take part together, and every lane of the warp must.
__device__ __forceinline__ uint32_t kv4_scaled(const uint32_t (&raw)[8], int dtype, float (&q)[8]) {
  uint32_t top = 0, limit = 0x7F800000u;  // the largest magnitude's bits, and where the numbers that are not finite begin
  if (dtype == kF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = __uint_as_float(raw[i]);
      top = max(top, raw[i] & 0x7FFFFFFFu);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = dtype == kBF16 ? bf16x2_to_f2(raw[i]) : unpack_half2(raw[i]);
      q[2 * i] = f.x;
      q[2 * i + 1] = f.y;
      top = __vmaxu2(top, raw[i] & 0x7FFF7FFFu);
    }
    top = max(top & 0xFFFFu, top >> 16);
    limit = dtype == kBF16 ? 0x7F80u : 0x7C00u;
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool bad = top >= limit;
  const float amax = dtype == kF32 ? __uint_as_float(top)
                                   : (dtype == kBF16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top)));
  uint32_t bits;
  if (amax > 0x1p-90f && amax < 0x1p100f) {  // (false for what is not finite)
    bits = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(amax, kSixth)));
    const float s = bf16_bits_f32(bits), y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient_by(q[i], s, y);
  } else {
    bits = fp4_scale_bits(amax, bad);
    const float s = bf16_bits_f32(bits);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp4_quotient(q[i], s);
  }
  return bits;
}

// Eight elements of a row as they are stored.
__device__ __forceinline__ void kv4_load(const void* row, int dtype, int at, bool vec, uint32_t (&v)[8]) {
  if (dtype == kF32) {
    const uint32_t* p = static_cast<const uint32_t*>(row) + at;
    if (vec) {
      const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + at;
    if (vec) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    }
  }
}

__global__ void __launch_bounds__(256) kv4_append_kernel(const __grid_constant__ Kv4Rows P) {
  const Kv4Map& M = P.map;
  const int ng = M.d / kKvGroup, es = elem_bytes(P.dtype);
  const unsigned id = blockIdx.x * 256u + threadIdx.x, pair = id / (unsigned)P.chunks, chunk = id - pair * P.chunks;
  const int h = chunk / (M.d / 8), c8 = chunk - h * (M.d / 8), w = c8 >> 2, t = c8 & 3;
  for (int b = blockIdx.y; b < P.B; b += gridDim.y) {  // (the loop is uniform: the shuffles below see whole warps)
    const int n = pair < (unsigned)P.npairs ? (P.len ? min(max(__ldg(P.len + b), 0), P.M) : P.M) : 0;
    const int p0 = __ldg(P.pos + b);
    const long long even = ((long long)(p0 >> 1) + pair) * 2;  // position of the pair's even token
    uint32_t kr[2][8] = {}, vr[2][8] = {};
    bool on[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long m = even + e - p0;  // row of the window
      on[e] = m >= 0 && m < n;
      const long long row = (long long)b * P.M + m;
      if (on[e]) {
        kv4_load(static_cast<const unsigned char*>(P.k) + row * P.ks * es, P.dtype, 8 * chunk, P.kvec, kr[e]);
        kv4_load(static_cast<const unsigned char*>(P.v) + row * P.vs * es, P.dtype, 8 * chunk, P.vvec, vr[e]);
      }
    }
    uint32_t kc[2], ks[2], vs[2];
    float vq[2][8];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float q[8];
      ks[e] = kv4_scaled(kr[e], P.dtype, q);
      kc[e] = float2_to_e2m1(q[0], q[1]) | float2_to_e2m1(q[2], q[3]) << 8 | float2_to_e2m1(q[4], q[5]) << 16 |
              float2_to_e2m1(q[6], q[7]) << 24;
      vs[e] = kv4_scaled(vr[e], P.dtype, vq[e]);
    }
    if (even < 0 || even > 0x7FFFFFFEll || (!on[0] && !on[1])) continue;
    const int tile = (int)even >> 4, at = kv4_page_of_tile(M, tile), page = kv4_page(M, b, at);
    if (page < 0) continue;
    unsigned char* T = kv4_tile(M, page, h, tile - at * M.tpp);
    const int slot = (int)even & 15;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!on[e]) continue;
      *reinterpret_cast<uint32_t*>(T + (slot + e) * (M.d / 2) + t * (ng * 4) + w * 4) = kc[e];
      if (t == 0) {
        uint16_t* sc = reinterpret_cast<uint16_t*>(T + 16 * M.d) + (slot + e) * ng + w;
        sc[0] = (uint16_t)ks[e];
        sc[16 * ng] = (uint16_t)vs[e];
      }
    }
    // channels 8 t .. 8 t + 3 and 8 t + 4 .. 8 t + 7 of the pair
    unsigned char* vw = T + 8 * M.d + (slot >> 1) * M.d + 2 * t * (ng * 4) + w * 4;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) bits |= float2_to_e2m1(vq[0][4 * g + j], vq[1][4 * g + j]) << (8 * j);
      uint32_t* at32 = reinterpret_cast<uint32_t*>(vw + g * (ng * 4));
      if (on[0] && on[1]) {
        *at32 = bits;
      } else {
        const uint32_t mask = on[0] ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
        const uint32_t flip = (*reinterpret_cast<volatile uint32_t*>(at32) ^ bits) & mask;
        if (flip) atomicXor(at32, flip);
      }
    }
  }
}

__device__ __forceinline__ void store4(void* base, long long at, int dtype, float4 v) {
  if (dtype == kF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = v;
  } else if (dtype == kBF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<uint2*>(static_cast<__half*>(base) + at) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
  }
}

// Eight channels: their codes times s, rounded once to the type (streamed past
// L2: 27.9 against 31.7 us for 4 x 8192 tokens of 8 x 128 channels, bfloat16).
__device__ __forceinline__ void store8_held(void* base, long long at, int dtype, uint32_t codes, float s) {
  uint32_t h[4];
  e2m1_to_half2x4(codes, h);
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = unpack_half2(h[i]);
    f[i] = make_float2(f[i].x * s, f[i].y * s);
  }
  if (dtype == kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    __stcs(p, make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
    __stcs(p + 1, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == kBF16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&a);
    } else {
      w[i] = pack_half2(f[i].x, f[i].y);
    }
  }
  __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at), make_uint4(w[0], w[1], w[2], w[3]));
}

// One thread per (sequence, pair of token slots, 8 channels of a head): one
// word of key codes per token, two words of value codes for both.
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4Rows P) {
  const Kv4Map& M = P.map;
  const int ng = M.d / kKvGroup;
  const unsigned id = blockIdx.x * 256u + threadIdx.x, pair = id / (unsigned)P.chunks, chunk = id - pair * P.chunks;
  if (pair >= (unsigned)P.npairs) return;
  const int h = chunk / (M.d / 8), c8 = chunk - h * (M.d / 8), w = c8 >> 2, t = c8 & 3;
  const int even = 2 * (int)pair, tile = even >> 4, at = kv4_page_of_tile(M, tile), slot = even & 15;
  const long long width = (long long)M.nkv * M.d;
  for (int b = blockIdx.y; b < P.B; b += gridDim.y) {
    const int n = P.len ? min(max(__ldg(P.len + b), 0), P.M) : P.M;
    const int page = even < n ? kv4_page(M, b, at) : -1;
    uint32_t kc[2] = {0u, 0u}, vc[2] = {0u, 0u}, ks[2] = {0u, 0u}, vs[2] = {0u, 0u};
    if (page >= 0) {
      const unsigned char* T = kv4_tile(M, page, h, tile - at * M.tpp);
      const unsigned char* vp = T + 8 * M.d + (slot >> 1) * M.d + 2 * t * (ng * 4) + w * 4;
      const uint32_t v0 = *reinterpret_cast<const uint32_t*>(vp), v1 = *reinterpret_cast<const uint32_t*>(vp + ng * 4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (even + e >= n) continue;
        kc[e] = *reinterpret_cast<const uint32_t*>(T + (slot + e) * (M.d / 2) + t * (ng * 4) + w * 4);
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(T + 16 * M.d) + (slot + e) * ng + w;
        ks[e] = sc[0];
        vs[e] = sc[16 * ng];
        // this token's nibbles of the eight bytes, packed to 32 bits
        uint32_t a = (v0 >> (4 * e)) & 0x0F0F0F0Fu, c = (v1 >> (4 * e)) & 0x0F0F0F0Fu;
        a = (a | a >> 4) & 0x00FF00FFu;
        c = (c | c >> 4) & 0x00FF00FFu;
        vc[e] = __byte_perm(a, c, 0x6420);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (even + e >= P.M) continue;
      const long long o = ((long long)b * P.M + even + e) * width + 8 * chunk;
      store8_held(P.ko, o, P.dtype, kc[e], bf16_bits_f32(ks[e]));
      store8_held(P.vo, o, P.dtype, vc[e], bf16_bits_f32(vs[e]));
    }
  }
}

// -------------------------------------------------------------- attention
// o = softmax(scale q k^T) v of a window of rows against the held keys and
// values, one pass with a running maximum and sum.  A CTA takes one KV head
// of one sequence and up to 8 NT of its query rows (rows of the window x the
// query heads that share the KV head); its warps take pairs of 16-token tiles
// in turn.  Where that leaves SMs idle several CTAs split a sequence, write
// their shares to the caller's workspace, and a second kernel joins them in
// order (no atomics: results do not depend on the order of arrival; nothing in
// the workspace outlives the call).  Joining through the shared memory of a
// cluster was slower: a cluster of 16 packs two CTAs on an SM and left half of
// the SMs idle (one row over 8 heads x 32768 tokens: 23.7 us).
//
// Per pair of tiles a warp forms S^T = K q^T with the 16 tokens of a tile as
// the M operand, straight from the codes, and 8 query rows as N.  The group's
// scale multiplies the 32-channel partial sums in float32.  The weights
// p = 2^(s - m), times the scales of the values, go to fp16 and are transposed
// in registers (movmatrix) to be the N operand of O^T += V^T P^T, again with
// the codes as M operand.  Tokens as M leave no row of the tensor core unused
// for the few query rows of decoding (rows as M would waste 8 to 15 of 16).
//
// Precision.  q: fp16 with a power of two per row (bfloat16 and fp16 exactly,
// float32 as hi + lo, QT = 2).  p * scale: fp16 under a power of two per column
// that brings the largest scale S which the column has seen, in any group of the
// head, to [2^6, 2^7) at weight 1 (p <= 256 then stays in range): eleven bits
// down to 2^-20 of S, below that an error of at most 2^-31 of S; fp16 and float32
// outputs take the rest as a second term (PT = 2: 22 bits down to 2^-9 of S, the
// same 2^-31 below), since one term would add about as much error
// as fp16's own rounding.  S counts as 2^-80 at least.  For bfloat16 outputs one
// term is an eighth of their own rounding (0.0016 off the 64-bit result with one
// or two terms), and a second one costs: 32 windows of 4 rows 73.4 against 63.5 us
// a call, one row over 32768 tokens 22.7 against 21.4.  The sum of p is float32.
// Float32 outputs are added up outside the tensor core, whose accumulation
// truncates (QT = 2); the 16-bit types inside it, up to 3e-8 for every 128 tokens
// of an unsplit sequence (8192 steps, 2^20 tokens: 2.5e-4, half of fp16's rounding).
//
// The reference m is only moved when a score exceeds it by 8 (p <= 256), so
// most tiles need no reduction across lanes.
//
// Bound: instructions where an SM holds two CTAs, and uneven shares of the work.
// Per 32 tokens of a head of 128 channels a warp converts 256 pairs of codes (96
// byte extractions, 128 conversions: about 100 of the 192 clocks that HBM takes
// for the 4608 bytes), applies 64 scales and packs and transposes the weights.
// 304 CTAs of one length, two on each of the 152 SMs, read 5.0 TB/s (74 % of the
// measured bandwidth); 152, one on each, 3.8, whether from HBM or from L2.
// Measured: 32 windows of 4 rows, 16 / 8 heads x 128, 5185 to 8192 tokens,
// bfloat16: 61.9 us, 4.0 TB/s: 256 CTAs leave 48 SMs with one, and the busiest SM
// works 1.17 times the mean; one row over 32768 tokens, 32 / 8 heads: 19.1 us; 64
// windows over 16 tokens: 7.6 us, a chain of latencies.
struct Kv4Attn {
  Kv4Map map;
  const void* q;
  void* o;
  float* lse;
  const int* kv_len;
  const int* n_rows;
  const unsigned long long* mask;
  long long qs, os;
  float scale_log2e;      // its magnitude; the sign goes to q
  int M, nq, grp, row_tiles, splits, dtype;
  int ring_at, ring_stride, stages;
  float* part;  // shares of the splits: [unit][split] of m[C], l[C], O[C][D]
  bool qvec, ovec, negative;
};

constexpr int kKvMaxSplits = 64;
constexpr int kKvMaxWarps = 8;
// CTAs of 8 warps that share an SM, by the registers of the accumulators.
__host__ __device__ constexpr int kv4_ctas(int NG, int NT) { return NT * NG <= 4 ? 2 : 1; }

template <int N>
__device__ __forceinline__ void lds_words(const unsigned char* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x; w[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
  }
}

// Scale w of a packed row of scales, as float.
template <int N>
__device__ __forceinline__ float scale_of(const uint32_t (&s)[N], int w) {
  return __uint_as_float((w & 1) ? s[w >> 1] & 0xFFFF0000u : s[w >> 1] << 16);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2_of_biased(int e) { return __uint_as_float((uint32_t)e << 23); }

// Factor of a share whose reference is m in a sum whose reference is top.
__device__ __forceinline__ float share_factor(float m, float top) {
  return m == -INFINITY && top == -INFINITY ? 0.0f : (m == top ? 1.0f : ex2(m - top));
}

// Four channels of query row rr (of those that share KV head h): v over the
// sum s whose reference is m (log2 units), and the log-sum-exp.
template <int D>
__device__ __forceinline__ void kv4_write(const Kv4Attn& P, int b, int h, int rr, int ch, float m, float s, float4 v) {
  const int row = rr / P.grp, e = rr - row * P.grp;
  if (s == 0.0f) {
    v = make_float4(0.f, 0.f, 0.f, 0.f);  // a row that sees nothing
  } else {
    const float inv = __frcp_rn(s);
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  }
  const long long at = ((long long)b * P.M + row) * P.os + (long long)(h * P.grp + e) * D + ch;
  if (P.ovec) {
    store4(P.o, at, P.dtype, v);
  } else {
    store_elem(P.o, at, P.dtype, v.x);
    store_elem(P.o, at + 1, P.dtype, v.y);
    store_elem(P.o, at + 2, P.dtype, v.z);
    store_elem(P.o, at + 3, P.dtype, v.w);
  }
  if (ch == 0 && P.lse)
    P.lse[((long long)b * P.M + row) * P.nq + h * P.grp + e] =
        s == 0.0f ? -INFINITY : (m + log2f(s)) * 0.69314718055994530942f;
}

template <int NG, int NT, int QT, int PT>
__global__ void __launch_bounds__(32 * kKvMaxWarps, kv4_ctas(NG, NT)) kv4_attention_kernel(const __grid_constant__ Kv4Attn P) {
  constexpr int D = 32 * NG, TB = 18 * D, CH = TB / 16, C = 8 * NT, QS = 2 * D + 64, RS = D + 8;
  // Biased exponent that the scales of the values start from: smaller ones count
  // as 2^-80.  Sums of weights carry 2^(133 - E0) = 2^86 then, and stay finite for
  // 2^31 positions of 2^8 each.
  constexpr int E0 = 47;
  constexpr bool QREG = NG * NT * QT <= 4;  // q operands kept in registers
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_fac[C];
  __shared__ int s_row[C];
  __shared__ unsigned long long s_mask[C];
  __shared__ float s_m[C], s_l[C];                              // this CTA's references and sums
  __shared__ float s_pm[kKvMaxWarps][C], s_pl[kKvMaxWarps][C];  // the warps'; s_pm becomes their factors
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the kernel that joins the splits, where there is one)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, W = blockDim.x >> 5;
  const Kv4Map& M = P.map;
  const int unit = blockIdx.x / P.splits, sp = blockIdx.x - unit * P.splits;
  const int rt = unit % P.row_tiles, bh = unit / P.row_tiles, h = bh % M.nkv, b = bh / M.nkv;
  const int nr = P.n_rows ? min(max(__ldg(P.n_rows + b), 0), P.M) : P.M;
  const int ncol = min(C, nr * P.grp - rt * C);
  if (ncol <= 0) return;
  const int len = min(max(__ldg(P.kv_len + b), 0), M.max_pages * M.page_size);
  const int base = len - nr;  // position of the window's row 0
  // Pairs of tiles go round the warps of all splits in turn: which a warp takes
  // does not depend on the length, so its first pages are known before it is.
  const int tiles = (len + 15) >> 4, all_warps = W * P.splits, me = sp * W + warp;
  const int pairs = (tiles + 1) >> 1, nit = pairs > me ? (pairs - me + all_warps - 1) / all_warps : 0;
  unsigned char* ring = sm + P.ring_at + (size_t)warp * P.ring_stride;
  const unsigned char* head = M.cache + (long long)h * M.tpp * TB + lane * 16;

  uint32_t okbits = 0;  // tiles of the ring that hold tokens: bit 2 * stage + sub
  int page[2], in[2];   // pages of the pair that is copied next, and the tiles' places in them
  auto look = [&](int i) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = 2 * (me + all_warps * i) + u, at = kv4_page_of_tile(M, j);
      in[u] = j - at * M.tpp;
      page[u] = kv4_page(M, b, at);
    }
  };
  auto issue = [&](int i, int stage) {
    if (i < nit) {
      unsigned char* dst = ring + stage * (2 * TB) + lane * 16;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t bit = 1u << (2 * stage + u);
        if (page[u] >= 0 && 2 * (me + all_warps * i) + u < tiles) {
          okbits |= bit;
          const unsigned char* src = head + page[u] * M.page_stride + in[u] * TB;
#pragma unroll
          for (int r = 0; r < (CH + 31) / 32; ++r)
            if (32 * r + 32 <= CH || lane < CH - 32 * r) cp_async16(dst + u * TB + r * 512, src + r * 512);
        } else {
          okbits &= ~bit;
        }
      }
      look(i + 1);
    }
    cp_async_commit();
  };
  look(0);
  const int ST = P.stages;
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) issue(i, i);

  // query rows: one warp per row, several loads in flight; a column past the rows holds zeros
  constexpr int QU = 4, QC = (D + 127) / 128;
  for (int c0 = warp; c0 < C; c0 += QU * W) {
    float4 v[QU][QC];
#pragma unroll
    for (int k = 0; k < QU; ++k) {
      const int c = c0 + k * W, rr = rt * C + c, m = rr / P.grp, e = rr - m * P.grp;
      const long long at = ((long long)b * P.M + m) * P.qs + (long long)(h * P.grp + e) * D;
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int x = i * 128 + lane * 4;
        if (c < ncol && x < D)
          v[k][i] = load4(static_cast<const unsigned char*>(P.q) + at * elem_bytes(P.dtype), P.dtype, x, D, P.qvec);
      }
    }
#pragma unroll
    for (int k = 0; k < QU; ++k) {
      const int c = c0 + k * W;
      if (c >= C) break;
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < QC; ++i)
        mx = max(mx, max(max(finite_abs_bits(v[k][i].x), finite_abs_bits(v[k][i].y)),
                         max(finite_abs_bits(v[k][i].z), finite_abs_bits(v[k][i].w))));
      float up, down;
      pow2_normaliser(__reduce_max_sync(0xffffffffu, mx), &up, &down);
      if (P.negative) up = -up;
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        const int x = i * 128 + lane * 4;
        if (x >= D) continue;
        const float x0 = v[k][i].x * up, x1 = v[k][i].y * up, x2 = v[k][i].z * up, x3 = v[k][i].w * up;
        *reinterpret_cast<uint2*>(sm + c * QS + x * 2) = make_uint2(pack_half2(x0, x1), pack_half2(x2, x3));
        if (QT == 2)
          *reinterpret_cast<uint2*>(sm + (C + c) * QS + x * 2) =
              make_uint2(pack_half2(fp16_rest(x0), fp16_rest(x1)), pack_half2(fp16_rest(x2), fp16_rest(x3)));
      }
      if (lane == 0) {
        const int m = (rt * C + c) / P.grp;
        s_fac[c] = fmaxf(down * P.scale_log2e, 1e-37f);  // never zero: -infinity times it stays -infinity
        s_row[c] = m;
        s_mask[c] = c < ncol && P.mask ? P.mask[(long long)b * P.M + m] : ~0ull;
      }
    }
  }
  __syncthreads();

  float fac[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) fac[n][c] = s_fac[n * 8 + 2 * t + c];
  const unsigned char* qcol = sm + g * QS + t * 16;  // column g of n-tile 0
  uint4 qr[QREG ? NG * NT * QT : 1];
  if (QREG) {
#pragma unroll
    for (int w = 0; w < NG; ++w)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < QT; ++x)
          qr[(w * NT + n) * QT + x] = *reinterpret_cast<const uint4*>(qcol + (x * C + n * 8) * QS + w * 64);
  }

  // Per column: the reference m (log2 units), the score above which it moves
  // (in raw score units), and what is taken from a score: m less the power of
  // two that brings the values' scales to [2^6, 2^7), so that it costs nothing
  // to apply.  l and O carry that power; it is taken out at the end.  All of
  // them follow from the positions that the column sees and from nothing else:
  // a position that it does not see changes no bit of it.
  float O[NG][2][NT][4], mref[NT][2], thr[NT][2], sub[NT][2], l[NT][2];
  uint32_t ecol[NT];  // biased exponents of the largest value scales that the two columns have seen, 16 bits each
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) { mref[n][c] = thr[n][c] = -INFINITY; l[n][c] = sub[n][c] = 0.0f; }
    ecol[n] = E0 * 0x10001u;
#pragma unroll
    for (int w = 0; w < NG; ++w)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) O[w][u][n][c] = 0.0f;
  }
  uint32_t emin = E0;  // the smallest of this lane's columns' exponents

  int stage = 0;
#pragma unroll 1
  for (int i = 0; i < nit; ++i) {
    __syncwarp();  // every lane is done with the stage that is filled next
    issue(i + ST - 1, stage == 0 ? ST - 1 : stage - 1);
    if (ST == 2) cp_async_wait_group<1>();
    else cp_async_wait_group<3>();
    __syncwarp();
    const int p0 = 32 * (me + all_warps * i);
    const unsigned char* st = ring + stage * (2 * TB);
    const uint32_t ok = (okbits >> (2 * stage)) & 3u;
    stage = stage + 1 == ST ? 0 : stage + 1;
    const bool edge = ok != 3u || p0 + 31 >= base;  // some token is not seen by every row

    float sc[2][NT][4];
    uint32_t vs[2][2][NG / 2];
    uint32_t hidden = 0;  // bit ((2 s + hh) NT + n) 2 + c: column c of n-tile n does not see token g + 8 hh of tile s
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const unsigned char* T = st + s * TB;
      uint32_t ka[NG], kb[NG], sa[NG / 2], sb[NG / 2];
      lds_words<NG>(T + g * (D / 2) + t * (NG * 4), ka);
      lds_words<NG>(T + (g + 8) * (D / 2) + t * (NG * 4), kb);
      lds_words<NG / 2>(T + 16 * D + g * (NG * 2), sa);
      lds_words<NG / 2>(T + 16 * D + (g + 8) * (NG * 2), sb);
      lds_words<NG / 2>(T + 17 * D + g * (NG * 2), vs[s][0]);
      lds_words<NG / 2>(T + 17 * D + (g + 8) * (NG * 2), vs[s][1]);
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        uint32_t a[4], c4[4];
        e2m1_to_half2x4(ka[w], a);
        e2m1_to_half2x4(kb[w], c4);
        const float f0 = scale_of(sa, w), f1 = scale_of(sb, w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int x = QT - 1; x >= 0; --x) {
            const uint4 q4 = QREG ? qr[QREG ? (w * NT + n) * QT + x : 0]
                                  : *reinterpret_cast<const uint4*>(qcol + (x * C + n * 8) * QS + w * 64);
            mma_f16_16816(acc, a[0], c4[0], a[1], c4[1], q4.x, q4.y);
            mma_f16_16816(acc, a[2], c4[2], a[3], c4[3], q4.z, q4.w);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[s][n][c] = w == 0 ? (c < 2 ? f0 : f1) * acc[c] : fmaf(c < 2 ? f0 : f1, acc[c], sc[s][n][c]);
        }
      }
      if (edge) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int pos = p0 + 16 * s + g + 8 * hh, j = pos - base;
          const bool there = ((ok >> s) & 1u) && pos < len;
          if (!there)
#pragma unroll
            for (int w = 0; w < NG / 2; ++w) vs[s][hh][w] = 0u;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = n * 8 + 2 * t + c;
              const bool see = there && (j < 0 || (P.mask ? (s_mask[col] >> j) & 1ull : (unsigned long long)(j <= s_row[col])));
              if (!see) {
                sc[s][n][2 * hh + c] = -INFINITY;
                hidden |= 1u << (((2 * s + hh) * NT + n) * 2 + c);
              }
            }
        }
      }
    }

    // does a reference, or a power of two, have to move?
    bool move = false;
    uint32_t top2 = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) top2 = __vmaxu2(top2, __vmaxu2(vs[s][0][w], vs[s][1][w]));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        move |= fmaxf(fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), sc[1][n][c]), sc[1][n][2 + c]) > thr[n][c];
    if (__any_sync(0xffffffffu, move || (max(top2 & 0xFFFFu, top2 >> 16) >> 7) > emin)) {
      uint32_t e[2][2];  // the largest exponent of a token's finite scales
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          e[s][hh] = 0;
#pragma unroll
          for (int w = 0; w < NG; ++w) {
            const uint32_t x = (vs[s][hh][w >> 1] >> (16 * (w & 1)) & 0xFFFFu) >> 7;
            if (x < 255u) e[s][hh] = max(e[s][hh], x);
          }
        }
      emin = 255u;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t seen = 0;  // the largest of the tokens that a column sees, for both columns
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            seen = __vmaxu2(seen, (sc[s][n][2 * hh] == -INFINITY ? 0u : e[s][hh]) |
                                      (sc[s][n][2 * hh + 1] == -INFINITY ? 0u : e[s][hh] << 16));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) seen = __vmaxu2(seen, __shfl_xor_sync(0xffffffffu, seen, o));
        const uint32_t enew = __vmaxu2(seen, ecol[n]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          // (a column moves for its own scores only, not because another one does)
          mx = mx > thr[n][c] ? fmaxf(mx * fac[n][c], mref[n][c]) : mref[n][c];
          const int e0 = ecol[n] >> (16 * c) & 0xFFFFu, e1 = enew >> (16 * c) & 0xFFFFu;
          const float al = (mx == mref[n][c] ? 1.0f : ex2(mref[n][c] - mx)) * pow2_of_biased(max(127 + e0 - e1, 0));
          mref[n][c] = mx;
          thr[n][c] = __fdiv_rn(mx + 8.0f, fac[n][c]);
          sub[n][c] = mx == -INFINITY ? 0.0f : mx - (float)(6 + 127 - e1);
          emin = min(emin, (uint32_t)e1);
          l[n][c] *= al;
#pragma unroll
          for (int w = 0; w < NG; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              O[w][u][n][c] *= al;
              O[w][u][n][2 + c] *= al;
            }
        }
        ecol[n] = enew;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sc[s][n][c] = ex2(fmaf(sc[s][n][c], fac[n][c & 1], -sub[n][c & 1]));
          l[n][c & 1] += sc[s][n][c];
        }

    // O^T += V^T P^T.  KEEP: some tokens are hidden, and a hidden token adds
    // nothing whatever its scale is.  (A token that is seen and whose weight
    // underflows to zero still brings a NaN of its values, as in any other tile.)
    auto values = [&](auto keep_tag) {
      constexpr bool KEEP = decltype(keep_tag)::value;
      uint32_t keep[2][2][NT];
      if constexpr (KEEP) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t two = hidden >> (((2 * s + hh) * NT + n) * 2);
              keep[s][hh][n] = (two & 1u ? 0u : 0x0000FFFFu) | (two & 2u ? 0u : 0xFFFF0000u);
            }
      }
      uint32_t va[2][NG], vb[2][NG];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        lds_words<NG>(st + s * TB + 8 * D + t * D + g * (NG * 4), va[s]);
        lds_words<NG>(st + s * TB + 8 * D + (t + 4) * D + g * (NG * 4), vb[s]);
      }
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        uint32_t B[2][NT][PT][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float f = scale_of(vs[s][hh], w);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float x = sc[s][n][2 * hh] * f, y = sc[s][n][2 * hh + 1] * f;
              uint32_t hi = pack_half2(x, y);
              if constexpr (KEEP) hi &= keep[s][hh][n];
              B[s][n][0][hh] = movmatrix_trans(hi);
              if constexpr (PT == 2) {
                const float2 r = unpack_half2(hi);
                uint32_t lo = pack_half2(x - r.x, y - r.y);
                if constexpr (KEEP) lo &= keep[s][hh][n];
                B[s][n][PT - 1][hh] = movmatrix_trans(lo);
              }
            }
          }
        uint32_t a[2][4], c4[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          e2m1_to_half2x4(va[s][w], a[s]);
          e2m1_to_half2x4(vb[s][w], c4[s]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float acc[NT][4];
          if constexpr (QT == 2)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int x = PT - 1; x >= 0; --x)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16_16816(QT == 2 ? acc[n] : O[w][u][n], a[s][2 * u], a[s][2 * u + 1], c4[s][2 * u], c4[s][2 * u + 1],
                              B[s][n][x][0], B[s][n][x][1]);
          if constexpr (QT == 2)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) O[w][u][n][c] += acc[n][c];
        }
      }
    };
    if (edge) values(std::true_type{});
    else values(std::false_type{});
  }
  cp_async_wait_group<0>();
  __syncwarp();

  // the warps' shares through shared memory (each over its own ring)
  {
    float* mo = reinterpret_cast<float*>(ring);  // [C][RS]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float back = pow2_of_biased((int)(ecol[n] >> (16 * c) & 0xFFFFu) - 6);  // 2^(exponent - 127 - 6)
        float s = l[n][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int col = n * 8 + 2 * t + c;
        if (g == 0) {
          s_pm[warp][col] = mref[n][c];
          s_pl[warp][col] = s * back;
        }
#pragma unroll
        for (int w = 0; w < NG; ++w)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float2*>(mo + col * RS + w * 32 + g * 4 + 2 * u) =
                make_float2(O[w][u][n][c] * back, O[w][u][n][2 + c] * back);
      }
  }
  __syncthreads();
  // one reference and sum per column; the warps' factors replace their references
  if (tid < C) {
    float m = -INFINITY, sum = 0.0f;
    for (int k = 0; k < W; ++k) m = fmaxf(m, s_pm[k][tid]);
    for (int k = 0; k < W; ++k) {
      const float f = share_factor(s_pm[k][tid], m);
      sum = fmaf(f, s_pl[k][tid], sum);
      s_pm[k][tid] = f;
    }
    s_m[tid] = m;
    s_l[tid] = sum;
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(sm + P.ring_at);
  float* part = P.splits > 1 ? P.part + (long long)blockIdx.x * (C * (D + 2)) : nullptr;
  for (int i = tid; i < ncol * (D / 4); i += blockDim.x) {
    const int col = i / (D / 4), ch = 4 * (i - col * (D / 4));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kKvMaxWarps; ++k) {
      if (k >= W) break;
      const float4 x = *reinterpret_cast<const float4*>(all + k * (P.ring_stride / 4) + col * RS + ch);
      const float f = s_pm[k][col];
      v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
    }
    if (P.splits == 1) {
      kv4_write<D>(P, b, h, rt * C + col, ch, s_m[col], s_l[col], v);
    } else {
      *reinterpret_cast<float4*>(part + 2 * C + col * D + ch) = v;
      if (ch == 0) {
        part[col] = s_m[col];
        part[C + col] = s_l[col];
      }
    }
  }
}

// Joins the splits of a sequence: one warp per column, four channels a lane
// (D / 128 times); the references of all splits first, a lane each.
template <int NG, int NT>
__global__ void __launch_bounds__(128) kv4_join_kernel(const __grid_constant__ Kv4Attn P) {
  constexpr int D = 32 * NG, C = 8 * NT, SIZE = C * (D + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int id = blockIdx.x * 4 + warp, unit = id / C, col = id - unit * C;  // (the grid is units * C / 4 exactly)
  const int rt = unit % P.row_tiles, bh = unit / P.row_tiles, h = bh % P.map.nkv, b = bh / P.map.nkv;
  const int nr = P.n_rows ? min(max(__ldg(P.n_rows + b), 0), P.M) : P.M;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rt * C + col >= nr * P.grp) return;
  const float* part = P.part + (long long)unit * P.splits * SIZE;
  float m[kKvMaxSplits / 32], l[kKvMaxSplits / 32], top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kKvMaxSplits / 32; ++i) {
    const int k = i * 32 + lane;
    m[i] = k < P.splits ? __ldcg(part + (long long)k * SIZE + col) : -INFINITY;
    l[i] = k < P.splits ? __ldcg(part + (long long)k * SIZE + C + col) : 0.0f;
    top = fmaxf(top, m[i]);
  }
  top = warp_max(top);
#pragma unroll
  for (int i = 0; i < kKvMaxSplits / 32; ++i) {
    m[i] = share_factor(m[i], top);
    sum = fmaf(m[i], l[i], sum);
  }
  sum = warp_sum(sum);
#pragma unroll 1
  for (int ch = lane * 4; ch < (D < 128 ? 128 : D); ch += 128) {  // (every lane takes part in the shuffles)
    const float* at = part + 2 * C + col * D + min(ch, D - 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < P.splits; k0 += 8) {
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < P.splits) x[k] = __ldcg(reinterpret_cast<const float4*>(at + (long long)(k0 + k) * SIZE));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = __shfl_sync(0xffffffffu, k0 >= 32 ? m[1] : m[0], (k0 + k) & 31);
        if (k0 + k < P.splits)
          v = make_float4(fmaf(f, x[k].x, v.x), fmaf(f, x[k].y, v.y), fmaf(f, x[k].z, v.z), fmaf(f, x[k].w, v.w));
      }
    }
    if (ch < D) kv4_write<D>(P, b, h, rt * C + col, ch, top, sum, v);
  }
}

}  // namespace cpk

// -------------------------------------------------------------- host side
namespace cpk_host {

using namespace cpk;

size_t kv4_bytes(int n_pages, int page_size, int nkv, int d) {
  return (size_t)n_pages * nkv * (page_size / 16) * kv4_tile_bytes(d);
}

static Kv4Map kv4_map(const Kv4Shape& S, void* cache, const int* pages, int max_pages) {
  Kv4Map M;
  M.cache = static_cast<unsigned char*>(cache);
  M.pages = pages;
  M.max_pages = max_pages;
  M.page_size = S.page_size;
  M.n_pages = S.n_pages;
  M.nkv = S.nkv;
  M.d = S.d;
  M.tpp = S.page_size / 16;
  M.tpp_shift = -1;
  for (int i = 0; i < 20; ++i)
    if (M.tpp == 1 << i) M.tpp_shift = i;
  M.page_stride = (long long)S.nkv * M.tpp * kv4_tile_bytes(S.d);
  return M;
}

// One thread per pair of slots and chunk of a sequence; sequences past the grid's second axis by a loop.
static dim3 rows_grid(const Kv4Rows& P) {
  return dim3((unsigned)(((long long)P.npairs * P.chunks + 255) / 256), std::min(P.B, 65535));
}

cudaError_t launch_kv4_append(const Kv4Shape& S, void* cache, const int* pages, int max_pages, int B, int M, const int* pos,
                              const int* len, int dtype, const void* k, long long ks, const void* v, long long vs,
                              cudaStream_t s) {
  Kv4Rows P{};
  P.map = kv4_map(S, cache, pages, max_pages);
  P.k = k; P.v = v; P.ks = ks; P.vs = vs;
  P.pos = pos; P.len = len;
  P.B = B; P.M = M; P.dtype = dtype;
  P.npairs = M / 2 + 1;
  P.chunks = S.nkv * S.d / 8;
  P.kvec = ks * elem_bytes(dtype) % 16 == 0;
  P.vvec = vs * elem_bytes(dtype) % 16 == 0;
  kv4_append_kernel<<<rows_grid(P), 256, 0, s>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Shape& S, const void* cache, const int* pages, int max_pages, int B, int T, const int* len,
                            int dtype, void* k, void* v, cudaStream_t s) {
  Kv4Rows P{};
  P.map = kv4_map(S, const_cast<void*>(cache), pages, max_pages);
  P.ko = k; P.vo = v;
  P.len = len;
  P.B = B; P.M = T; P.dtype = dtype;
  P.npairs = (T + 1) / 2;
  P.chunks = S.nkv * S.d / 8;
  kv4_read_kernel<<<rows_grid(P), 256, 0, s>>>(P);
  return cudaGetLastError();
}

// How a call is laid out: query rows per CTA (8 NT), warps of a CTA, and CTAs
// that split a sequence.
struct Kv4Plan {
  int NT, W, row_tiles, splits;
  long long units;
  size_t work;  // bytes of the shares
};

static Kv4Plan kv4_plan(const Kv4Shape& S, int max_pages, int B, int M, int nq, int dtype, int sms) {
  Kv4Plan L;
  const int NG = S.d / 32, rows = M * (nq / S.nkv), tiles = max_pages * (S.page_size / 16);
  // the MMA's 8 columns, or 16; 32 only at 128 channels and 16-bit types (64
  // rows x 4 over 4096 tokens: 205 against 218 us), not at 64 channels, where
  // two CTAs of 16 columns share an SM (111 against 128 us), nor where the
  // accumulators spill
  const int most = NG == 4 && dtype != kF32 ? 4 : 2;
  L.NT = std::min(rows <= 8 ? 1 : (rows <= 16 ? 2 : 4), most);
  L.row_tiles = (rows + 8 * L.NT - 1) / (8 * L.NT);
  L.units = (long long)B * S.nkv * L.row_tiles;
  // warps: two tiles each at least, but four for the rows of q and the outputs
  L.W = 4;
  while (L.W < kKvMaxWarps && 4 * L.W <= tiles) L.W *= 2;
  // CTAs of a sequence: as many as the SMs hold at once, while every warp
  // keeps four tiles
  const long long slots = (long long)sms * kv4_ctas(NG, L.NT);
  L.splits = (int)std::max<long long>(1, std::min<long long>(std::min<long long>(slots / std::max(L.units, 1ll), kKvMaxSplits),
                                                             tiles / (4 * L.W)));
  L.work = L.splits > 1 ? (size_t)L.units * L.splits * (8 * L.NT) * (S.d + 2) * 4 : 0;
  return L;
}

size_t kv4_attention_work(const Kv4Shape& S, int max_pages, int B, int M, int nq, int dtype, int sms) {
  return kv4_plan(S, max_pages, B, M, nq, dtype, sms).work;
}

template <int NG, int NT, int QT, int PT>
static cudaError_t launch_attention(Kv4Attn& P, const Kv4Plan& L, int sms, cudaStream_t s) {
  constexpr int D = 32 * NG, C = 8 * NT;
  // Pairs of tiles in the ring of a warp: two, four where one CTA has the SM
  // to itself or the pairs are small, so that enough bytes are on their way.
  P.stages = NG == 2 || (NG == 4 && L.units * P.splits <= sms) ? 4 : 2;
  const size_t merge = (size_t)C * (D + 8) * 4, ring = (size_t)P.stages * 2 * kv4_tile_bytes(D);
  P.ring_at = (C * QT * (2 * D + 64) + 127) / 128 * 128;
  P.ring_stride = (int)(std::max(merge, ring) + 127) / 128 * 128;
  const size_t smem = P.ring_at + (size_t)L.W * P.ring_stride;
  const void* fn = (const void*)kv4_attention_kernel<NG, NT, QT, PT>;
  cudaError_t e = ops4_smem_limit(fn, smem);
  if (e != cudaSuccess || P.q == nullptr) return e;  // (no queries: only readied)
  void* args[] = {&P};
  e = cudaLaunchKernel(fn, dim3((unsigned)(L.units * P.splits)), dim3(32 * L.W), args, smem, s);
  if (e != cudaSuccess || P.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(L.units * C / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, (const void*)kv4_join_kernel<NG, NT>, args);
}

template <int NG, int QT, int PT>
static cudaError_t launch_attention_nt(Kv4Attn& P, const Kv4Plan& L, int sms, cudaStream_t s) {
  if (L.NT == 1) return launch_attention<NG, 1, QT, PT>(P, L, sms, s);
  if constexpr (NG == 4 && QT == 1)
    if (L.NT == 4) return launch_attention<NG, 4, QT, PT>(P, L, sms, s);
  return launch_attention<NG, 2, QT, PT>(P, L, sms, s);
}

template <int NG>
static cudaError_t launch_attention_types(Kv4Attn& P, const Kv4Plan& L, int sms, cudaStream_t s) {
  if (P.dtype == kF32) return launch_attention_nt<NG, 2, 2>(P, L, sms, s);
  if (P.dtype == kF16) return launch_attention_nt<NG, 1, 2>(P, L, sms, s);
  return launch_attention_nt<NG, 1, 1>(P, L, sms, s);
}

cudaError_t kv4_attention_configure(const Kv4Shape& S, int max_pages, int B, int M, int nq, int dtype) {
  Kv4Attention A{};
  A.max_pages = max_pages; A.B = B; A.M = M; A.nq = nq; A.dtype = dtype;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, (const void*)kv4_append_kernel);  // (loads it)
  for (int sms : {1, 1 << 16})  // (both ring depths)
    if (e == cudaSuccess) e = launch_kv4_attention(S, A, sms, 0);
  return e;
}

cudaError_t launch_kv4_attention(const Kv4Shape& S, const Kv4Attention& A, int sms, cudaStream_t s) {
  Kv4Attn P{};
  P.map = kv4_map(S, const_cast<void*>(A.cache), A.pages, A.max_pages);
  P.q = A.q; P.o = A.o; P.lse = A.lse;
  P.kv_len = A.kv_len; P.n_rows = A.n_rows; P.mask = A.mask;
  P.qs = A.qs; P.os = A.os;
  P.scale_log2e = fabsf(A.scale) * 1.4426950408889634f;
  P.negative = A.scale < 0.0f;
  P.M = A.M; P.nq = A.nq; P.grp = A.nq / S.nkv; P.dtype = A.dtype;
  P.qvec = A.qs % 4 == 0;
  P.ovec = A.os % 4 == 0;
  const Kv4Plan L = kv4_plan(S, A.max_pages, A.B, A.M, A.nq, A.dtype, sms);
  P.row_tiles = L.row_tiles;
  P.splits = L.splits;
  P.part = static_cast<float*>(A.work);
  switch (S.d) {
    case 64: return launch_attention_types<2>(P, L, sms, s);
    case 128: return launch_attention_types<4>(P, L, sms, s);
    default: return launch_attention_types<8>(P, L, sms, s);
  }
}

}  // namespace cpk_host
