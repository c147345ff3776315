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
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cp_fp4.cuh"
#include "cp_ops4.h"

namespace cpk {

constexpr int kKvGroup = 32;

__host__ __device__ inline int kv4_tile_bytes(int d) { return 18 * d; }

// Address of the tile that holds position `pos` of sequence b for head h, or
// null where the position has no page.  *slot: the position's slot in the tile.
struct Kv4Map {
  unsigned char* cache;
  const int* pages;  // [B][max_pages], or null: sequence b owns pages b * max_pages ..
  int max_pages, page_size, n_pages, nkv, d;
};

__device__ __forceinline__ int kv4_page(const Kv4Map& M, int b, int at) {
  if (at >= M.max_pages) return -1;
  const int id = M.pages ? __ldg(M.pages + (long long)b * M.max_pages + at) : b * M.max_pages + at;
  return id >= 0 && id < M.n_pages ? id : -1;
}

__device__ __forceinline__ unsigned char* kv4_tile(const Kv4Map& M, int page, int h, int tile_in_page) {
  return M.cache + (((long long)page * M.nkv + h) * (M.page_size >> 4) + tile_in_page) * kv4_tile_bytes(M.d);
}

// ------------------------------------------------------------ write, read
// One thread per (sequence, pair of token slots, 4 channels of a head): the 8
// threads of a scale group are neighbours in a warp, so are the groups of a
// row, and a row's loads and stores coalesce.  A pair shares the bytes of its
// value codes; where only one of its tokens is written the other's nibbles
// are left by an atomic exclusive-or of the nibbles that change (another
// sequence, or another call, may be writing them).  Bound by the bytes of the
// rows.
struct Kv4Rows {
  Kv4Map map;
  const void* k;
  const void* v;
  void* ko;
  void* vo;
  long long ks, vs;  // row strides in elements
  const int* pos;    // first position of each sequence (append), null in read
  const int* len;    // rows of each sequence that count, or null
  int B, M, npairs, dtype;
  bool kvec, vvec;
};

// Quantises four channels; every lane of the warp takes part.  Returns the
// codes, *scale the group's scale bits.
__device__ __forceinline__ uint32_t kv4_quantise(float4 x, uint32_t* scale) {
  uint32_t m = max(max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu),
                   max(__float_as_uint(x.z) & 0x7FFFFFFFu, __float_as_uint(x.w) & 0x7FFFFFFFu));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  *scale = fp4_scale_bits(__uint_as_float(m), m >= 0x7F800000u);
  const float s = bf16_bits_f32(*scale);
  return float2_to_e2m1(fp4_quotient(x.x, s), fp4_quotient(x.y, s)) |
         float2_to_e2m1(fp4_quotient(x.z, s), fp4_quotient(x.w, s)) << 8;
}

// The four 4-bit codes of c spread to the low nibbles of four bytes.
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t c) {
  c = (c | c << 8) & 0x00FF00FFu;
  return (c | c << 4) & 0x0F0F0F0Fu;
}

__global__ void __launch_bounds__(256) kv4_append_kernel(const __grid_constant__ Kv4Rows P) {
  const Kv4Map& M = P.map;
  const int chunks = M.nkv * M.d / 4, ng = M.d / kKvGroup;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const int chunk = (int)(id % chunks);
  const long long rest = id / chunks;
  const int pair = (int)(rest % P.npairs);
  const long long bl = rest / P.npairs;
  const int b = (int)min(bl, (long long)P.B - 1);
  const int n = bl < P.B ? (P.len ? min(max(__ldg(P.len + b), 0), P.M) : P.M) : 0;
  const int p0 = __ldg(P.pos + b);
  const long long even = ((long long)(p0 >> 1) + pair) * 2;  // position of the pair's even token
  float4 kx[2], vx[2];
  bool on[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const long long m = even + e - p0;  // row of the window
    on[e] = m >= 0 && m < n;
    const long long row = (long long)b * P.M + m;
    kx[e] = vx[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on[e]) {
      const int es = elem_bytes(P.dtype);
      kx[e] = load4(static_cast<const unsigned char*>(P.k) + row * P.ks * es, P.dtype, 4 * chunk, 4 * chunk + 4, P.kvec);
      vx[e] = load4(static_cast<const unsigned char*>(P.v) + row * P.vs * es, P.dtype, 4 * chunk, 4 * chunk + 4, P.vvec);
    }
  }
  uint32_t kc[2], vc[2], ksc[2], vsc[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    kc[e] = kv4_quantise(kx[e], &ksc[e]);
    vc[e] = kv4_quantise(vx[e], &vsc[e]);
  }
  if (even < 0 || (!on[0] && !on[1])) return;  // (positions are below 2^31: the launcher bounds max_pages * page_size)
  const long long at = even / M.page_size;
  if (at >= M.max_pages) return;
  const int page = kv4_page(M, b, (int)at);
  if (page < 0) return;
  const int in_page = (int)(even - at * M.page_size);
  const int h = chunk / (M.d / 4), c4 = chunk - h * (M.d / 4), w = c4 >> 3, lane8 = c4 & 7;
  unsigned char* tile = kv4_tile(M, page, h, in_page >> 4);
  const int slot = in_page & 15;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!on[e]) continue;
    *reinterpret_cast<uint16_t*>(tile + (slot + e) * (M.d / 2) + (lane8 >> 1) * (ng * 4) + w * 4 + (lane8 & 1) * 2) =
        (uint16_t)kc[e];
    if (lane8 == 0) {
      uint16_t* sc = reinterpret_cast<uint16_t*>(tile + 16 * M.d) + (slot + e) * ng + w;
      sc[0] = (uint16_t)ksc[e];
      sc[16 * ng] = (uint16_t)vsc[e];
    }
  }
  uint32_t* vw = reinterpret_cast<uint32_t*>(tile + 8 * M.d + (slot >> 1) * M.d + lane8 * (ng * 4) + w * 4);
  const uint32_t bits = spread_nibbles(vc[0]) | spread_nibbles(vc[1]) << 4;
  if (on[0] && on[1]) {
    *vw = bits;
  } else {
    const uint32_t mask = on[0] ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
    const uint32_t flip = (*reinterpret_cast<volatile uint32_t*>(vw) ^ bits) & mask;
    if (flip) atomicXor(vw, flip);
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

__device__ __forceinline__ float4 codes_to_float4(uint32_t c, float s) {
  uint32_t h[4];
  e2m1_to_half2x4(c, h);
  const float2 lo = unpack_half2(h[0]), hi = unpack_half2(h[1]);
  return make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s);
}

__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4Rows P) {
  const Kv4Map& M = P.map;
  const int chunks = M.nkv * M.d / 4, ng = M.d / kKvGroup;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const int chunk = (int)(id % chunks);
  const long long rest = id / chunks;
  const int pair = (int)(rest % P.npairs);
  const long long bl = rest / P.npairs;
  if (bl >= P.B) return;
  const int b = (int)bl, even = 2 * pair;
  const int n = P.len ? min(max(__ldg(P.len + b), 0), P.M) : P.M;
  const int page = even < n ? kv4_page(M, b, even / M.page_size) : -1;
  float4 k[2], v[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) k[e] = v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (page >= 0) {
    const int in_page = even % M.page_size, slot = in_page & 15;
    const int h = chunk / (M.d / 4), c4 = chunk - h * (M.d / 4), w = c4 >> 3, lane8 = c4 & 7;
    const unsigned char* tile = kv4_tile(M, page, h, in_page >> 4);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(tile + 8 * M.d + (slot >> 1) * M.d + lane8 * (ng * 4) + w * 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (even + e >= n) continue;
      const uint32_t kc = *reinterpret_cast<const uint16_t*>(tile + (slot + e) * (M.d / 2) + (lane8 >> 1) * (ng * 4) + w * 4 +
                                                              (lane8 & 1) * 2);
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(tile + 16 * M.d) + (slot + e) * ng + w;
      k[e] = codes_to_float4(kc, bf16_bits_f32(sc[0]));
      // this token's nibbles of the pair's four bytes, packed to 16 bits
      uint32_t c = (vw >> (4 * e)) & 0x0F0F0F0Fu;
      c = (c | c >> 4) & 0x00FF00FFu;
      c = (c | c >> 8) & 0xFFFFu;
      v[e] = codes_to_float4(c, bf16_bits_f32(sc[16 * ng]));
    }
  }
  const long long width = (long long)M.nkv * M.d;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (even + e >= P.M) continue;
    const long long at = ((long long)b * P.M + even + e) * width + 4 * chunk;
    store4(P.ko, at, P.dtype, k[e]);
    store4(P.vo, at, P.dtype, v[e]);
  }
}

// -------------------------------------------------------------- attention
// o = softmax(scale q k^T) v of a window of rows against the held keys and
// values, one pass with a running maximum and sum.  A CTA takes one KV head
// of one sequence and up to 8 NT of its query rows (rows of the window x the
// query heads that share the KV head); its warps take pairs of 16-token tiles
// in turn, and the CTAs of a cluster split the sequence and join through
// distributed shared memory (no workspace, no atomics: results do not depend
// on the order of arrival).
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
// float32 as hi + lo, QT = 2).  p * scale: fp16 brought to at most 2^15 by
// a power of two that follows the largest scale seen, so it keeps eleven bits
// down to 2^-29 of the largest product; fp16 and float32 outputs take the
// rest as a second term (PT = 2), since one term would add about as much error
// as fp16's own rounding.  The sum of p is float32.  Float32 outputs are added
// up outside the tensor core, whose accumulation truncates (QT = 2).
//
// The reference m is only moved when a score exceeds it by 8 (p <= 256), so
// most tiles need no reduction across lanes.
//
// Bound: the bytes of the cache for few rows, then the legacy tensor pipe
// (2 clocks per m16n8k16 and SM).
struct Kv4Attn {
  Kv4Map map;
  const void* q;
  void* o;
  float* lse;
  const int* kv_len;
  const int* n_rows;
  const unsigned long long* mask;
  long long qs, os;
  float scale_log2e;
  int M, nq, grp, row_tiles, splits, dtype;
  int ring_at, ring_stride, res_at;
  bool qvec;
};

__host__ __device__ constexpr int kv4_stages(int NG) { return NG == 2 ? 4 : 2; }

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

template <int NG, int NT, int QT, int PT>
__global__ void __launch_bounds__(256, (NT * NG <= 8 && NG <= 4) ? 2 : 1) kv4_attention_kernel(const __grid_constant__ Kv4Attn P) {
  constexpr int D = 32 * NG, TB = 18 * D, CH = TB / 16, ST = kv4_stages(NG), C = 8 * NT, QS = 2 * D + 64, RS = D + 8;
  constexpr bool QREG = NG * NT * QT <= 4;  // q operands kept in registers
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_fac[C];
  __shared__ int s_row[C];
  __shared__ unsigned long long s_mask[C];
  __shared__ float s_ml[2 * C];
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, W = blockDim.x >> 5;
  const Kv4Map& M = P.map;
  const int unit = blockIdx.x / P.splits, sp = blockIdx.x - unit * P.splits;
  const int rt = unit % P.row_tiles, bh = unit / P.row_tiles, h = bh % M.nkv, b = bh / M.nkv;
  const int nr = P.n_rows ? min(max(__ldg(P.n_rows + b), 0), P.M) : P.M;
  const int ncol = min(C, nr * P.grp - rt * C);
  if (ncol <= 0) return;  // the same for every CTA of the cluster
  const int len = min(max(__ldg(P.kv_len + b), 0), M.max_pages * M.page_size);
  const int base = len - nr;  // position of the window's row 0
  const int tiles = (len + 15) >> 4;
  const int ta = (int)((long long)tiles * sp / P.splits), te = (int)((long long)tiles * (sp + 1) / P.splits);
  const int own = te - ta - 2 * warp;
  const int nit = own > 0 ? (own + 2 * W - 1) / (2 * W) : 0;
  unsigned char* ring = sm + P.ring_at + (size_t)warp * P.ring_stride;

  uint32_t okbits = 0;  // tiles of the ring that hold tokens: bit 2 * stage + sub
  auto issue = [&](int i) {
    if (i < nit) {
      const int j0 = ta + 2 * (warp + W * i), stage = i % ST;
      const unsigned char* src[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        src[u] = nullptr;
        if (j0 + u < te) {
          const int p0 = (j0 + u) * 16, at = p0 / M.page_size, page = kv4_page(M, b, at);
          if (page >= 0) src[u] = kv4_tile(M, page, h, (p0 - at * M.page_size) >> 4);
        }
        const uint32_t bit = 1u << (2 * stage + u);
        okbits = src[u] ? okbits | bit : okbits & ~bit;
      }
      unsigned char* dst = ring + stage * (2 * TB);
#pragma unroll
      for (int c0 = 0; c0 < 2 * CH; c0 += 32) {
        const int c = c0 + lane;
        if (c < 2 * CH) {
          const unsigned char* s = c < CH ? src[0] : src[1];
          if (s) cp_async16(dst + c * 16, s + (c < CH ? c : c - CH) * 16);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue(i);

  // query rows: one warp per row; a column past the rows holds zeros
  for (int c = warp; c < C; c += W) {
    const int rr = rt * C + c, m = rr / P.grp, e = rr - m * P.grp;
    const bool in = c < ncol;
    const long long at = ((long long)b * P.M + m) * P.qs + (long long)(h * P.grp + e) * D;
    float4 v[(D + 127) / 128];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < (D + 127) / 128; ++i) {
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int k = i * 128 + lane * 4;
      if (in && k < D) v[i] = load4(static_cast<const unsigned char*>(P.q) + at * elem_bytes(P.dtype), P.dtype, k, D, P.qvec);
      mx = max(mx, max(max(finite_abs_bits(v[i].x), finite_abs_bits(v[i].y)),
                       max(finite_abs_bits(v[i].z), finite_abs_bits(v[i].w))));
    }
    float up, down;
    pow2_normaliser(__reduce_max_sync(0xffffffffu, mx), &up, &down);
#pragma unroll
    for (int i = 0; i < (D + 127) / 128; ++i) {
      const int k = i * 128 + lane * 4;
      if (k >= D) continue;
      const float x0 = v[i].x * up, x1 = v[i].y * up, x2 = v[i].z * up, x3 = v[i].w * up;
      *reinterpret_cast<uint2*>(sm + c * QS + k * 2) = make_uint2(pack_half2(x0, x1), pack_half2(x2, x3));
      if (QT == 2)
        *reinterpret_cast<uint2*>(sm + (C + c) * QS + k * 2) =
            make_uint2(pack_half2(fp16_rest(x0), fp16_rest(x1)), pack_half2(fp16_rest(x2), fp16_rest(x3)));
    }
    if (lane == 0) {
      s_fac[c] = down * P.scale_log2e;
      s_row[c] = m;
      s_mask[c] = in && P.mask ? P.mask[(long long)b * P.M + m] : ~0ull;
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

  float O[NG][2][NT][4], mref[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) { mref[n][c] = -INFINITY; l[n][c] = 0.0f; }
#pragma unroll
    for (int w = 0; w < NG; ++w)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) O[w][u][n][c] = 0.0f;
  }
  int ecur = 7;  // biased exponent of the largest value scale seen
  float en = __uint_as_float((uint32_t)(127 + 6 + 127 - 7) << 23);  // 2^(6 - (ecur - 127))

  for (int i = 0; i < nit; ++i) {
    __syncwarp();  // every lane is done with the stage that is filled next
    issue(i + ST - 1);
    cp_async_wait_group<ST - 1>();
    __syncwarp();
    const int stage = i % ST, p0 = (ta + 2 * (warp + W * i)) * 16;
    const unsigned char* st = ring + stage * (2 * TB);
    const uint32_t ok = (okbits >> (2 * stage)) & 3u;
    const bool edge = ok != 3u || p0 + 31 >= base;  // some token is not seen by every row

    float sc[2][NT][4];
    uint32_t vs[2][2][NG / 2], keep[2][2][NT];
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
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[s][n][c] = 0.0f;
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
          sc[s][n][0] = fmaf(f0, acc[0], sc[s][n][0]);
          sc[s][n][1] = fmaf(f0, acc[1], sc[s][n][1]);
          sc[s][n][2] = fmaf(f1, acc[2], sc[s][n][2]);
          sc[s][n][3] = fmaf(f1, acc[3], sc[s][n][3]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[s][n][c] *= fac[n][c & 1];
        keep[s][0][n] = keep[s][1][n] = 0xFFFFFFFFu;
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
                keep[s][hh][n] &= c ? 0x0000FFFFu : 0xFFFF0000u;  // a masked token adds nothing, whatever its scale is
              }
            }
        }
      }
    }

    // does the reference have to move?
    bool move = false;
    uint32_t top2 = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) move |= sc[s][n][c] > mref[n][c & 1] + 8.0f;
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) top2 = __vmaxu2(top2, __vmaxu2(vs[s][0][w], vs[s][1][w]));
    }
    const int etop = (int)(max(top2 & 0xFFFFu, top2 >> 16) >> 7);
    if (__any_sync(0xffffffffu, move || etop > ecur)) {
      uint32_t e = 0;  // the largest exponent of a finite scale
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int w = 0; w < NG; ++w) {
            const uint32_t x = (vs[s][hh][w >> 1] >> (16 * (w & 1)) & 0xFFFFu) >> 7;
            if (x < 255u) e = max(e, x);
          }
      const int enew = max(ecur, (int)__reduce_max_sync(0xffffffffu, e));
      const float er = __uint_as_float((uint32_t)max(127 + ecur - enew, 0) << 23);
      ecur = enew;
      en = __uint_as_float((uint32_t)(127 + 6 + 127 - ecur) << 23);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(mx, mref[n][c]);
          const float al = mx == mref[n][c] ? 1.0f : ex2(mref[n][c] - mx);
          mref[n][c] = mx;
          l[n][c] *= al;
#pragma unroll
          for (int w = 0; w < NG; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              O[w][u][n][c] *= al * er;
              O[w][u][n][2 + c] *= al * er;
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float ref = mref[n][c] == -INFINITY ? 0.0f : mref[n][c];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float pa = ex2(sc[s][n][c] - ref), pb = ex2(sc[s][n][2 + c] - ref);
          l[n][c] += pa + pb;
          sc[s][n][c] = pa;
          sc[s][n][2 + c] = pb;
        }
      }

    // O^T += V^T P^T
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
          const float f = scale_of(vs[s][hh], w) * en;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float x = sc[s][n][2 * hh] * f, y = sc[s][n][2 * hh + 1] * f;
            const uint32_t hi = pack_half2(x, y) & keep[s][hh][n];
            B[s][n][0][hh] = movmatrix_trans(hi);
            if (PT == 2) {
              const float2 r = unpack_half2(hi);
              B[s][n][PT - 1][hh] = movmatrix_trans(pack_half2(x - r.x, y - r.y) & keep[s][hh][n]);
            }
          }
        }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float acc[NT][4];
        if (QT == 2)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a[4], c4[4];
          e2m1_to_half2x4(va[s][w], a);
          e2m1_to_half2x4(vb[s][w], c4);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = PT - 1; x >= 0; --x)
              mma_f16_16816(QT == 2 ? acc[n] : O[w][u][n], a[2 * u], a[2 * u + 1], c4[2 * u], c4[2 * u + 1], B[s][n][x][0],
                            B[s][n][x][1]);
        }
        if (QT == 2)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) O[w][u][n][c] += acc[n][c];
      }
    }
  }
  cp_async_wait_group<0>();
  __syncwarp();

  // the warps' shares through shared memory (each over its own ring)
  {
    float* mo = reinterpret_cast<float*>(ring);  // [C][RS], then m[C], l[C]
    const float back = __uint_as_float((uint32_t)(127 + ecur - 127 - 6) << 23);  // 2^(ecur - 127 - 6)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float s = l[n][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int col = n * 8 + 2 * t + c;
        if (g == 0) {
          mo[C * RS + col] = mref[n][c];
          mo[C * RS + C + col] = s;
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
  const int stride = P.ring_stride / 4;
  const float* all = reinterpret_cast<const float*>(sm + P.ring_at);
  float* res = reinterpret_cast<float*>(sm + P.res_at);
  const float ln2 = 0.69314718055994530942f;
  auto write = [&](int col, int ch, float m, float s, float v) {
    const int rr = rt * C + col, row = rr / P.grp, e = rr - row * P.grp;
    store_elem(P.o, ((long long)b * P.M + row) * P.os + (long long)(h * P.grp + e) * D + ch, P.dtype, s > 0.0f || s != s ? v / s : 0.0f);
    if (ch == 0 && P.lse)
      P.lse[((long long)b * P.M + row) * P.nq + h * P.grp + e] = s == 0.0f ? -INFINITY : (m + log2f(s)) * ln2;
  };
  for (int i = tid; i < ncol * D; i += blockDim.x) {
    const int col = i / D, ch = i - col * D;
    float m = -INFINITY;
    for (int k = 0; k < W; ++k) m = fmaxf(m, all[k * stride + C * RS + col]);
    float s = 0.0f, v = 0.0f;
    const float ref = m == -INFINITY ? 0.0f : m;
    for (int k = 0; k < W; ++k) {
      const float* x = all + k * stride;
      const float mk = x[C * RS + col], f = mk == m && m != -INFINITY ? 1.0f : ex2(mk - ref);
      s = fmaf(f, x[C * RS + C + col], s);
      v = fmaf(f, x[col * RS + ch], v);
    }
    if (P.splits == 1) {
      write(col, ch, m, s, v);
    } else {
      res[i] = v;
      if (ch == 0) { s_ml[col] = m; s_ml[C + col] = s; }
    }
  }
  if (P.splits == 1) return;
  // the CTAs of the cluster: each joins a share of the outputs
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int i = sp * blockDim.x + tid; i < ncol * D; i += P.splits * blockDim.x) {
    const int col = i / D, ch = i - col * D;
    float m = -INFINITY;
    for (int k = 0; k < P.splits; ++k) m = fmaxf(m, *cl.map_shared_rank(s_ml + col, k));
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, v = 0.0f;
    for (int k = 0; k < P.splits; ++k) {
      const float mk = *cl.map_shared_rank(s_ml + col, k), f = mk == m && m != -INFINITY ? 1.0f : ex2(mk - ref);
      s = fmaf(f, *cl.map_shared_rank(s_ml + C + col, k), s);
      v = fmaf(f, *cl.map_shared_rank(res + i, k), v);
    }
    write(col, ch, m, s, v);
  }
  cl.sync();  // no CTA leaves while another reads its shared memory
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
  return M;
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
  const int es = elem_bytes(dtype);
  P.kvec = ks * es % (4 * es) == 0;
  P.vvec = vs * es % (4 * es) == 0;
  const long long threads = (long long)B * P.npairs * (S.nkv * S.d / 4);
  kv4_append_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(P);
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
  const long long threads = (long long)B * P.npairs * (S.nkv * S.d / 4);
  kv4_read_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(P);
  return cudaGetLastError();
}

template <int NG, int NT, int QT, int PT>
static cudaError_t launch_attention(Kv4Attn& P, int W, long long units, cudaStream_t s) {
  constexpr int D = 32 * NG, C = 8 * NT;
  const size_t merge = (size_t)(C * (D + 8) + 2 * C) * 4, ring = (size_t)kv4_stages(NG) * 2 * kv4_tile_bytes(D);
  P.ring_at = (C * QT * (2 * D + 64) + 127) / 128 * 128;
  P.ring_stride = (int)(std::max(merge, ring) + 127) / 128 * 128;
  P.res_at = P.ring_at + W * P.ring_stride;
  const size_t smem = P.res_at + (P.splits > 1 ? (size_t)C * D * 4 : 0);
  const void* fn = (const void*)kv4_attention_kernel<NG, NT, QT, PT>;
  cudaError_t e = ops4_smem_limit(fn, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * P.splits));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = P.splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = P.splits > 1 ? 1 : 0;
  void* args[] = {&P};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int NG, int QT, int PT>
static cudaError_t launch_attention_nt(int NT, Kv4Attn& P, int W, long long units, cudaStream_t s) {
  if (NT == 1) return launch_attention<NG, 1, QT, PT>(P, W, units, s);
  if (NT == 2 || NG == 8) return launch_attention<NG, 2, QT, PT>(P, W, units, s);
  return launch_attention<NG, NG == 8 ? 2 : 4, QT, PT>(P, W, units, s);
}

template <int NG>
static cudaError_t launch_attention_types(int NT, Kv4Attn& P, int W, long long units, cudaStream_t s) {
  if (P.dtype == kF32) return launch_attention_nt<NG, 2, 2>(NT, P, W, units, s);
  if (P.dtype == kF16) return launch_attention_nt<NG, 1, 2>(NT, P, W, units, s);
  return launch_attention_nt<NG, 1, 1>(NT, P, W, units, s);
}

cudaError_t launch_kv4_attention(const Kv4Shape& S, const Kv4Attention& A, int sms, cudaStream_t s) {
  Kv4Attn P{};
  P.map = kv4_map(S, const_cast<void*>(A.cache), A.pages, A.max_pages);
  P.q = A.q; P.o = A.o; P.lse = A.lse;
  P.kv_len = A.kv_len; P.n_rows = A.n_rows; P.mask = A.mask;
  P.qs = A.qs; P.os = A.os;
  P.scale_log2e = A.scale * 1.4426950408889634f;
  P.M = A.M; P.nq = A.nq; P.grp = A.nq / S.nkv; P.dtype = A.dtype;
  P.qvec = A.qs % 4 == 0;
  // query rows per CTA: the MMA's 8 columns, or 16, or 32 (16 where the accumulators of 256 channels fill the registers)
  const int rows = A.M * P.grp;
  const int NT = rows <= 8 ? 1 : (rows <= 16 || S.d == 256 ? 2 : 4);
  P.row_tiles = (rows + 8 * NT - 1) / (8 * NT);
  const long long units = (long long)A.B * S.nkv * P.row_tiles;
  // Warps: two tiles each at least.  CTAs per sequence: enough to fill the
  // SMs, while every warp keeps four tiles.
  const int tiles = A.max_pages * (S.page_size / 16);
  int W = 1;
  while (W < 8 && 4 * W <= tiles) W *= 2;
  P.splits = 1;
  while (P.splits < 8 && units * P.splits * 2 <= 2ll * sms && tiles / (P.splits * 2) >= 4 * W) P.splits *= 2;
  switch (S.d) {
    case 64: return launch_attention_types<2>(NT, P, W, units, s);
    case 128: return launch_attention_types<4>(NT, P, W, units, s);
    default: return launch_attention_types<8>(NT, P, W, units, s);
  }
}

}  // namespace cpk_host
