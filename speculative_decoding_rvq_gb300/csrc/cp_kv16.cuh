// cp_kv16.cuh -- what the attention kernels over the 16-bit paged KV cache
// share: which positions a row sees, which tiles of positions a block of rows
// has to read, and the copies that bring them in.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "cp_common.cuh"
#include "cp_kv16.h"

namespace cpk {

// One attention call.  Rows of a sequence and KV head are packed: packed row
// r = i * group + g is row i of the sequence with query head h * group + g.
struct Kv16Call {
  CUtensorMap kmap, vmap;  // [pages][heads * page][dim], boxes of 64 channels x min(page, 64) tokens
  const unsigned short* keys;
  const unsigned short* values;
  const int* pages;
  const int* kv_len;
  const int* row_start;
  const unsigned long long* mask;
  const unsigned short* q;
  unsigned short* o;
  float* lse;
  float* work;  // [splits][n_rows * nq][dim] sums, then [splits][n_rows * nq] (maximum, sum of weights)
  int* status;
  long long qs, os;
  int n_pages, page_shift, box_shift, nkv, max_pages, n_seqs, n_rows, max_rows, nq, group, window, sinks, splits, mtiles;
  float scale_log2;  // scale * log2(e): weights are powers of two
  // A row's weights are 2^(score - base), its base `lift` below a score that was its largest (kv16_base); unlift: 2^-lift.
  // The tiles of cp_kv16_prompt.cu keep a base until a score passes it by `grow`.
  float lift, unlift, grow;
  int qvec, ovec;    // rows on 16 bytes
  int stall;         // test hook: 1 the last copy of a CTA is not made, 2 none is
  uint64_t wait_ns;  // bound of every wait
};

// The part of a call that belongs to one sequence.
struct Kv16Seq {
  int start, m, len, base;  // first row, rows, positions, position of the first row (may be negative)
};

__device__ __forceinline__ Kv16Seq kv16_seq(const Kv16Call& P, int b) {
  Kv16Seq s;
  const int r0 = __ldg(P.row_start + b), r1 = __ldg(P.row_start + b + 1);
  const long long most = (long long)P.max_pages << P.page_shift;
  s.start = r0;
  s.m = r0 >= 0 && r1 <= P.n_rows && r1 > r0 ? min(r1 - r0, P.max_rows) : 0;  // (starts outside the call's rows: none)
  s.len = (int)min((long long)max(__ldg(P.kv_len + b), 0), most);
  s.base = s.len - s.m;
  return s;
}

// What a row sees: positions up to `last` that lie past `first` or below the
// sinks; of the window's own positions (from base on) with a mask those of its bits.
struct Kv16Row {
  int last, first;
  unsigned long long bits;
};

__device__ __forceinline__ Kv16Row kv16_row(const Kv16Call& P, const Kv16Seq& s, int i) {
  Kv16Row r;
  r.bits = 0;
  if (i < 0 || i >= s.m) {  // a row of padding sees nothing
    r.last = -1;
    r.first = 0;
    return r;
  }
  int at = s.base + i;
  r.last = at;
  if (P.mask) {
    r.bits = __ldg(P.mask + s.start + i) & (s.m >= 64 ? ~0ull : (1ull << s.m) - 1ull);
    at = s.base + __popcll(r.bits) - 1;
    r.last = s.len - 1;
  }
  r.first = P.window > 0 ? max(at, -1) - P.window + 1 : 0;
  return r;
}

__device__ __forceinline__ bool kv16_sees(const Kv16Call& P, const Kv16Seq& s, const Kv16Row& r, int j) {
  if (P.mask && j >= s.base) return j <= r.last && ((r.bits >> (j - s.base)) & 1ull);
  return j <= r.last && (j >= r.first || j < P.sinks);
}

// Tiles of TILE positions that rows i0 .. i1 of a sequence have to read: the
// first `ns` (sinks), then `n - ns` from tile `first` on.
struct Kv16Tiles {
  int ns, first, n;
  __device__ __forceinline__ int tile(int k) const { return k < ns ? k : first + (k - ns); }
};

template <int TILE>
__device__ __forceinline__ Kv16Tiles kv16_tiles(const Kv16Call& P, const Kv16Seq& s, int i0, int i1) {
  Kv16Tiles t{0, 0, 0};
  const int end = P.mask ? s.len : min(s.len, s.base + i1 + 1);  // positions that any row sees end here
  if (end <= 0 || i0 > i1) return t;
  const int tiles = (end - 1) / TILE + 1;
  if (P.window > 0) {
    const int low = max(0, max(s.base + (P.mask ? -1 : i0), -1) - P.window + 1);
    t.first = min(low, end) / TILE;
    t.ns = min(t.first, min(P.sinks, end) > 0 ? (min(P.sinks, end) - 1) / TILE + 1 : 0);
  }
  t.n = t.ns + max(0, tiles - t.first);
  return t;
}

// Whether every row i0 .. i1 sees all TILE positions of a tile from t0 on
// (pages apart): no mask is needed then.
template <int TILE>
__device__ __forceinline__ bool kv16_whole(const Kv16Call& P, const Kv16Seq& s, int i0, int i1, int t0) {
  const int t1 = t0 + TILE - 1;
  if (t1 > (P.mask ? s.base - 1 : s.base + i0)) return false;
  if (P.window == 0 || t1 < P.sinks) return true;
  return t0 >= max(s.base + (P.mask ? s.m - 1 : i1), -1) - P.window + 1;
}

// Page of a position, or -1: past the table, or an entry that is no page.
__device__ __forceinline__ int kv16_page(const Kv16Call& P, int b, int pos) {
  const int at = pos >> P.page_shift;
  if (at >= P.max_pages) return -1;
  const int id = P.pages ? __ldg(P.pages + (long long)b * P.max_pages + at) : b * P.max_pages + at;
  return id >= 0 && id < P.n_pages ? id : -1;
}

// The same with the pages: whether the tile went through the product as it is.
template <int TILE>
__device__ __forceinline__ bool kv16_every(const Kv16Call& P, const Kv16Seq& s, int b, int i0, int i1, int t0) {
  bool every = kv16_whole<TILE>(P, s, i0, i1, t0);
  for (int p = t0; every && p < t0 + TILE; p += 16) every = kv16_page(P, b, p) >= 0;
  return every;
}

// A box of a tensor map to shared memory; its bytes complete on `bar`.
__device__ __forceinline__ void kv16_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool kv16_elect() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}

// Pages of the tiles that a warp copies, looked up for as many tiles as its 32
// lanes hold boxes of (4 or more), the next ones while these are used: one
// lookup takes longer than a tile.  Lane l holds box l % per of tile l / per.
template <int TILE>
struct Kv16Pages {
  int box, per, each, shift;  // tokens of a box; boxes of a tile; tiles of a lookup, and its logarithm
  int prev, cur, next, at;    // lookups at - 1, at, at + 1

  __device__ __forceinline__ int look(const Kv16Call& P, int b, const Kv16Tiles& T, int k0, int n, int end, int g, int lane) const {
    const int k = g * each + lane / per;
    int id = -1;
    if (k < n) {
      const int p = T.tile(k0 + k) * TILE + (lane & (per - 1)) * box, e = p >> P.page_shift;
      if (p < end && e < P.max_pages) id = P.pages ? __ldg(P.pages + (long long)b * P.max_pages + e) : b * P.max_pages + e;
    }
    return id;  // (not looked at here: the load stays in flight)
  }
  __device__ __forceinline__ void start(const Kv16Call& P, int b, const Kv16Tiles& T, int k0, int n, int end, int lane) {
    box = 1 << P.box_shift;
    per = TILE >> P.box_shift;
    each = 32 / per;
    shift = 31 - __clz(each);
    at = 0;
    prev = -1;
    cur = look(P, b, T, k0, n, end, 0, lane);
    next = look(P, b, T, k0, n, end, 1, lane);
  }
  // The lookup that holds tile k: the newest one's, the one's before, or the next, which then becomes the newest.
  __device__ __forceinline__ int of(const Kv16Call& P, int b, const Kv16Tiles& T, int k0, int n, int end, int k, int lane) {
    const int g = k >> shift;
    if (g > at) {
      prev = cur;
      cur = next;
      at = g;
      next = look(P, b, T, k0, n, end, g + 1, lane);
    }
    const int id = g == at ? cur : prev;
    return id >= 0 && id < P.n_pages ? id : -1;
  }
  // Bits of the 16-token pieces of tile k that have a page.
  __device__ __forceinline__ uint32_t held(int id, int k) const {
    const uint32_t have = __ballot_sync(0xffffffffu, id >= 0) >> ((k & (each - 1)) * per);
    uint32_t bits = 0;
    for (int j = 0; j < per; ++j) bits |= ((have >> j) & 1u) * (((1u << (box / 16)) - 1u) << (j * (box / 16)));
    return bits;
  }
};

// Wait for a phase of `bar`, bounded, that also ends when another thread of the
// CTA gave up.  The clock is read only every 256 tries: reading it takes longer
// than a wait of these kernels.
__device__ __forceinline__ bool kv16_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
}

// Wait for copies and MMAs in flight after a wait that ran out: they were issued, so they do arrive.
__device__ __forceinline__ void kv16_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 2000000000ull) {
  }
}

// 2^x; zero for -infinity.
__device__ __forceinline__ float kv16_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The base of a row whose largest score is `top`.  bfloat16: its sums then end where its values do.  fp16 numbers end at 2^16 and have steps of 2^-24 below 2^-14: weights
// that reach 2^15 instead of 1 keep 15 binary orders more of a long tail.  Rounded up there, so that no weight passes 2^lift
// where float32's steps are coarse.
template <bool BF>
__device__ __forceinline__ float kv16_base(float top, float lift) { return BF ? top - lift : __fsub_ru(top, lift); }

// The log of a row's sum of exponentials, from its base and its sum of weights.
__device__ __forceinline__ float kv16_lse(const Kv16Call& P, float base, float sum) {
  return sum == 0.0f ? -INFINITY : ((base + P.lift) + log2f(sum * P.unlift)) * 0.693147180559945309f;
}

// Infinities and NaN of a pair of 16-bit numbers replaced by zero; `bad` is set if there were any.
template <bool BF>
__device__ __forceinline__ uint32_t kv16_finite(uint32_t w, bool& bad) {
  const uint32_t e = BF ? 0x7F80u : 0x7C00u;
  const bool lo = (w & e) == e, hi = (w & (e << 16)) == (e << 16);
  bad |= lo | hi;
  return (lo ? 0u : w & 0xFFFFu) | (hi ? 0u : w & 0xFFFF0000u);
}

template <bool BF>
__device__ __forceinline__ uint32_t kv16_pack(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool BF>
__device__ __forceinline__ float2 kv16_unpack(uint32_t w) {
  return BF ? bf16x2_to_f2(w) : __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Values that are not finite, of eight neighbouring channels: bit c (channel c) plus infinity, 8 + c minus infinity, 16 + c
// NaN.  Or'ed over positions they tell what the sum is, whatever the weights.
template <bool BF>
__device__ __forceinline__ uint32_t kv16_odd(const uint4& u) {
  constexpr uint32_t E = BF ? 0x7F80u : 0x7C00u, ONE = BF ? 0x00800080u : 0x04000400u, EE = E | E << 16;
  // (an exponent of ones carries into the sign's place when one is added to it)
  if (((((u.x & EE) + ONE) | ((u.y & EE) + ONE) | ((u.z & EE) + ONE) | ((u.w & EE) + ONE)) & 0x80008000u) == 0) return 0;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t bits = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t x = w[c >> 1] >> (16 * (c & 1)) & 0xFFFFu;
    if ((x & E) == E) bits |= 1u << (c + ((x & ~E & 0x7FFFu) ? 16 : (x & 0x8000u ? 8 : 0)));
  }
  return bits;
}
// What they add up to in channel c, or x if there are none.
__device__ __forceinline__ float kv16_odd_sum(uint32_t bits, int c, float x) {
  const uint32_t b = bits >> c;
  if (b & 0x10000u || (b & 0x101u) == 0x101u) return __int_as_float(0x7FC00000);
  return b & 1u ? INFINITY : (b & 0x100u ? -INFINITY : x);
}

template <int D>
__device__ __forceinline__ uint4 kv16_value(const Kv16Call& P, int page, int h, int j, int c0) {
  const int in = j & ((1 << P.page_shift) - 1);
  return __ldg(reinterpret_cast<const uint4*>(P.values + ((((long long)page * P.nkv + h) << P.page_shift) + in) * D + c0));
}

// Values that are not finite (kv16_odd) in eight channels from c0 on, at the positions first, first + step, .. of each of the
// tiles k0 .. k0 + n - 1 that all rows i0 .. i1 see whole (pages apart).  Shared by the rows: with these tiles looked
// over by a warp or more, a NaN costs a few passes over the values (2048 rows over 16384 positions, 8 / 2 heads x 128: 0.23 ms
// without one, 2.0 with one; 79 where each row looked for itself; one row over 65536: 0.06 and 0.15).  shown: all tiles; else those with pages that are not.
template <bool BF, int D, int TILE>
__device__ __noinline__ uint32_t kv16_odd_shared(const Kv16Call& P, const Kv16Seq& s, const Kv16Tiles& T, int b, int h, int i0, int i1,
                                                 int k0, int n, int c0, int first, int step, bool shown) {
  uint32_t bits = 0;
  for (int k = k0; k < k0 + n; ++k) {
    const int t0 = T.tile(k) * TILE;
    if (!kv16_whole<TILE>(P, s, i0, i1, t0)) continue;
    if (!shown && kv16_every<TILE>(P, s, b, i0, i1, t0)) continue;
#pragma unroll 8
    for (int j = t0 + first; j < t0 + TILE; j += step) {
      const int page = kv16_page(P, b, j);
      if (page >= 0) bits |= kv16_odd<BF>(kv16_value<D>(P, page, h, j, c0));
    }
    if (bits >> 16 == 0xFFu) break;  // (all NaN)
  }
  return bits;
}
// The same for one row in the other tiles, of which a block of rows has few (the ends of what its rows see), for G times
// eight channels.
template <bool BF, int D, int TILE, int G>
__device__ __noinline__ void kv16_odd_own(const Kv16Call& P, const Kv16Seq& s, const Kv16Row& r, const Kv16Tiles& T, int b, int h, int i0,
                                          int i1, int k0, int n, int c0, uint32_t (&bits)[G]) {
  for (int k = k0; k < k0 + n; ++k) {
    const int t0 = T.tile(k) * TILE;
    if (kv16_whole<TILE>(P, s, i0, i1, t0)) continue;
    for (int j0 = t0; j0 < t0 + TILE && j0 < s.len; j0 += 16) {
      const int page = kv16_page(P, b, j0);
      if (page < 0) continue;
#pragma unroll 4
      for (int j = j0; j < j0 + 16; ++j) {
        if (j >= s.len || !kv16_sees(P, s, r, j)) continue;
#pragma unroll
        for (int g = 0; g < G; ++g) bits[g] |= kv16_odd<BF>(kv16_value<D>(P, page, h, j, c0 + 8 * g));
      }
    }
  }
}

}  // namespace cpk

namespace cpk_host {
// The parameters and tensor maps of a call, the same for all its kernels.
cudaError_t kv16_prepare(const Kv16Shape& S, const Kv16Attention& A, cpk::Kv16Call* P);
}  // namespace cpk_host
