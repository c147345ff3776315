// cp_kv16_prompt.cu -- attention over the 16-bit paged KV cache on the
// fifth-generation tensor cores, for many packed rows (prompts, pieces of
// prompts, wide draft trees) with 64 or 128 channels a head.
//
// A block of rows is 128 packed rows, the M of one MMA; tiles of 128 positions.
//   S = Q K^T   operands in shared memory, both K-major, accumulator in TMEM
//   O += P V    P (16-bit weights) in TMEM, V in shared memory as it lies in
//               the cache (token by token: the MN-major operand)
// A CTA keeps two products in flight, w = 0 and 1, each with its own S, P
// (in the columns of its S), O, and a warpgroup that turns S into P, one thread
// a row: while one warpgroup works, the tensor cores serve the other.  PAIR:
// w are two blocks of rows that read the same tiles (256 packed rows a CTA);
// else w are the even and the odd tiles of one block, joined at the end.  One warp
// brings tiles in by TMA (boxes of 64 channels x up to 64 tokens of a page)
// through a ring of stages, a lane for each product issues its MMAs.
//
// The base of a row's weights stays until a score exceeds the row's largest by
// 2^8: O is then rescaled in TMEM (each row by its own decision, so that no row's bits
// depend on another's), else the weights simply grow; sums are float32, weights
// enter the product as one 16-bit number (half a step of the type, as much as the
// output's own rounding; the sum uses the unrounded ones).
//
// fp16 weights have steps of 2^-24 and end at 2^16.  The largest is put at 2^7,
// which leaves the 2^8 above: a weight 2^-21 of it has all its bits.  A row that has
// one far above the others (a sink) would lose its tail: where all that it
// sees of 64 positions weighs less than 2^-8, or the least of those among which its base was found less
// than 2^-20 of the largest, its base goes 2^6 lower, once (`tall`): all bits down to 2^-27 of the largest, steps of 2^-37.  With
// that base from the start, and so 2^2 of room above, random scores move it again
// and again: 671 us instead of 485 for the long prompt below in fp16.
//
// What a row does not see cannot reach it: masked scores weigh zero, and in
// tiles that are not seen whole by every row values that are not finite are
// replaced by zeros in shared memory before the product (by a warp that looks over
// a tile as it lands, ahead of its use); the rows that do see them get them
// at the end, from the cache.
//
// Every wait is bounded; one that runs out ends all roles, and the CTA with them
// once its copies and MMAs in flight are through.
//
// Measured: 8192 rows over 16384 positions, window 4096, 32 / 8 heads x 128: 467
// us, 1178 TFLOP/s (62 % of the burst rate).  A turn of both blocks of rows takes
// 2550 to 2700 clocks, of which the MMAs are 2048; what is left is the way from a
// block's last weights to its next scores (commit, barrier, wake-up: about 500).
// The steps there: one warp issuing for both products 647 us, a warp each with the
// weights in halves and the maximum found beside them 469.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "cp_kv16.cuh"
#include "cp_kv16_prompt.h"
#include "cp_ops4.h"

namespace cpk {

constexpr int kPTile = 128;
constexpr int kPThreads = 384;  // two warpgroups of rows; a third: copies (warp 8), MMAs (9, 10), values looked over (11)
constexpr int kPHeld = 8;       // tiles whose page bits are kept
constexpr float kPTall = 6.0f;  // binary orders by which a row of fp16 weights far apart lowers its base
constexpr int kPFirst = 3;      // ring items whose copies start before the CTA's first barrier

__host__ __device__ constexpr int prompt_stages(int d) { return d == 64 ? 4 : 2; }  // of keys, and as many of values (an even number)
__host__ __device__ constexpr size_t prompt_smem(int d) {
  return 1024 + (size_t)(2 + 2 * prompt_stages(d)) * kPTile * d * 2;
}

struct PromptShared {
  uint64_t kfull[4], vfull[4], kempty[4], vempty[4], clean[4];  // rings: landed; read; values looked over
  uint64_t sfull[2], pready[2][2], ohalf[2], oend[2], last[2];
  float m[2][128], l[2][128];
  uint32_t held[kPHeld];
  uint32_t tmem;
  int abort, bad, keys, values;  // tiles copied
};

// Shared-memory descriptors: 128-byte swizzle; K-major rows of 128 bytes in
// groups of 8 (1024 bytes apart); MN-major the same memory read the other way:
// 64 channels x 8 tokens an atom, atoms 1024 bytes apart along the tokens and
// `lead` bytes along the channels.
__device__ __forceinline__ uint64_t prompt_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

// kind::f16, float32 accumulator, M = 128, N columns; B K-major or MN-major.
template <bool BF>
__device__ __forceinline__ uint32_t prompt_idesc(int n, bool mn) {
  return (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void prompt_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void prompt_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void prompt_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}

#define CP_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define CP_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// 32 columns of the warp's 32 lanes, from column address `at`.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CP_R8(v, 0), CP_R8(v, 8), CP_R8(v, 16), CP_R8(v, 24)
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::CP_I8(v, 0),
      CP_I8(v, 8), CP_I8(v, 16), CP_I8(v, 24), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What is copied at place `it` of 2 n.  PAIR: K0 V0 K1 V1 ..; else K0 K1 V0 K2 V1 .. (both products start before the
// first ends).  Keys and values have a ring each: tile k lies in stage k mod STAGES, in use for the k / STAGES-th time.
// A waiter of a stage then always has waited for its use before (STAGES is even, so with two products that take turns
// it is the same product's), which a wait by parity needs: with one ring for both, a product's first wait could take
// for its values' arrival that of keys that had not come yet.
struct PromptItem {
  bool v;
  int k;
};
template <bool PAIR>
__device__ __forceinline__ PromptItem prompt_item(int it, int n) {
  if (PAIR) return {(it & 1) != 0, it >> 1};
  if (it == 2 * n - 1) return {true, n - 1};
  if (it == 0 || (it & 1)) return {false, (it + 1) >> 1};
  return {true, (it >> 1) - 1};
}

// Place of 16-byte piece c of an output row in shared memory, against bank conflicts both ways.
template <int D>
__device__ __forceinline__ int prompt_out(int row, int c) { return row * D * 2 + ((c ^ (row & (D / 8 - 1))) << 4); }

// Bits 0 .. n - 1.
__device__ __forceinline__ unsigned long long prompt_below(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

// What a row sees (kv16_sees) of the 64 positions from t0 on, as bits; held: the four pages' bits.
__device__ __forceinline__ unsigned long long prompt_sees(const Kv16Call& P, const Kv16Seq& s, const Kv16Row& r, int t0, uint32_t held) {
  unsigned long long see = ~prompt_below(r.first - t0) | prompt_below(P.sinks - t0);
  if (P.mask) {
    const int own = s.base - t0;
    const unsigned long long before = prompt_below(own);
    const unsigned long long bits = own >= 64 || own <= -64 ? 0ull : (own >= 0 ? r.bits << own : r.bits >> -own);
    see = (see & before) | (bits & ~before);
  }
  see &= prompt_below(r.last + 1 - t0);
#pragma unroll
  for (int g = 0; g < 4; ++g)
    if (!((held >> g) & 1u)) see &= ~(0xFFFFull << (16 * g));
  return see;
}

// Weights 2^(f x - base) of 64 scores of a row to 32 columns of TMEM as 16-bit
// numbers; their sum, and the largest exponent.
template <bool BF>
__device__ __forceinline__ void prompt_weights(const uint32_t (&x)[64], float f, float base, uint32_t at, float& high, float& sum) {
  float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  float h2[2] = {-INFINITY, -INFINITY};
  uint32_t p[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float2 z = ffma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), make_float2(f, f), make_float2(-base, -base));
    h2[j & 1] = fmaxf(h2[j & 1], fmaxf(z.x, z.y));
    const float2 e = make_float2(kv16_exp2(z.x), kv16_exp2(z.y));
    s2[j & 1] = ffma2(e, make_float2(1.0f, 1.0f), s2[j & 1]);
    p[j] = kv16_pack<BF>(e.x, e.y);
  }
  tmem_st32(at, p);
  high = fmaxf(h2[0], h2[1]);
  sum = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
}

template <int D, bool BF, bool PAIR>
__global__ void __launch_bounds__(kPThreads, 1) kv16_prompt_kernel(const __grid_constant__ Kv16Call P) {
  constexpr int STAGES = prompt_stages(D), SB = kPTile * D * 2, HALVES = D / 64, ROWS = PAIR ? 256 : 128;
  extern __shared__ __align__(1024) unsigned char prompt_raw[];
  __shared__ PromptShared sh;
  unsigned char* smem = prompt_raw + ((1024u - (smem_u32(prompt_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + 2 * SB;  // after the queries of both blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x % P.splits, mt = P.mtiles - 1 - blockIdx.x / P.splits, h = blockIdx.y, b = blockIdx.z;
  // Only the kernel that joins the shares may start early: one that takes tensor memory before it waits for this
  // kernel could sit beside a CTA that then never gets its own.
  if (P.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Kv16Seq s = kv16_seq(P, b);
  const int r0 = mt * ROWS, packed = s.m * P.group;
  if (r0 >= packed) return;
  const int i0 = r0 / P.group, i1 = (min(r0 + ROWS, packed) - 1) / P.group;
  const Kv16Tiles T = kv16_tiles<kPTile>(P, s, i0, i1);
  const int k0 = (int)((long long)T.n * split / P.splits), n = (int)((long long)T.n * (split + 1) / P.splits) - k0;

  // copies of ring items
  const int items = P.stall == 0 ? 2 * n : (P.stall == 1 ? max(0, 2 * n - 1) : 0);
  const int end = P.mask ? s.len : min(s.len, s.base + i1 + 1);
  Kv16Pages<kPTile> pages;
  auto issue = [&](int it) {
    const PromptItem a = prompt_item<PAIR>(it, n);
    const int st = a.k % STAGES, id = pages.of(P, b, T, k0, n, end, a.k, lane), lane0 = (a.k & (pages.each - 1)) * pages.per;
    const uint32_t held = pages.held(id, a.k);
    uint64_t* full = a.v ? &sh.vfull[st] : &sh.kfull[st];
    if (lane == 0) {
      if (!a.v) sh.held[a.k % kPHeld] = held;
      mbar_arrive_expect_tx(full, SB);
    }
    __syncwarp();
    // a lane a box: 64 channels of `half`, tokens `piece` (one lane for all boxes takes twice as long)
    const int piece = lane & (pages.per - 1), half = lane / pages.per, page = __shfl_sync(0xffffffffu, id, lane0 + piece);
    if (half < HALVES) {
      const int t0 = T.tile(k0 + a.k) * kPTile + piece * pages.box;
      // (a page that does not exist: the box past the last page, which reads as zeros)
      kv16_box(smem_u32(ring + ((a.v ? STAGES : 0) + st) * SB + half * (kPTile * 128) + piece * pages.box * 128), a.v ? &P.vmap : &P.kmap, half * 64,
               page >= 0 ? (h << P.page_shift) + (t0 & ((1 << P.page_shift) - 1)) : 0, page >= 0 ? page : P.n_pages, smem_u32(full));
    }
    __syncwarp();
  };
  if (warp == 8) {  // the barriers, and the first copies at once: they wait for nobody
    pages.start(P, b, T, k0, n, end, lane);
    if (lane == 0) {
      for (int i = 0; i < STAGES; ++i) {
        mbar_init(&sh.kfull[i], 1);
        mbar_init(&sh.vfull[i], 1);
        mbar_init(&sh.clean[i], 32);
        mbar_init(&sh.kempty[i], PAIR ? 2 : 1);  // (both products read a tile of a pair)
        mbar_init(&sh.vempty[i], PAIR ? 2 : 1);
      }
      for (int w = 0; w < 2; ++w) {
        mbar_init(&sh.sfull[w], 1);
        mbar_init(&sh.pready[w][0], 128);
        mbar_init(&sh.pready[w][1], 128);
        mbar_init(&sh.ohalf[w], 1);
        mbar_init(&sh.oend[w], 1);
        mbar_init(&sh.last[w], 1);
      }
      sh.abort = sh.bad = sh.keys = sh.values = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
#pragma unroll 1
    for (int it = 0; it < min(kPFirst, items); ++it) issue(it);
  } else if (warp == 9) {  // all of TMEM: S0, S1, O0, O1
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp < 8) {
    // queries to shared memory, swizzled like the keys
    {
      constexpr int STEP = 256 / (D / 8), N = ROWS / STEP, B = N < 16 ? N : 16;  // rows a step of all threads; steps; loads in flight
      const int c = tid % (D / 8), rr0 = tid / (D / 8), dq = STEP / P.group, dr = STEP - dq * P.group;
      int r = r0 + rr0, i = r / P.group, g = r - i * P.group;
#pragma unroll 1
      for (int e = 0; e < N; e += B) {
        uint4 v[B];
#pragma unroll
        for (int a = 0; a < B; ++a) {
          v[a] = make_uint4(0, 0, 0, 0);
          if (r < packed) {
            const unsigned short* src = P.q + (long long)(s.start + i) * P.qs + (long long)(h * P.group + g) * D + 8 * c;
            if (P.qvec) v[a] = __ldg(reinterpret_cast<const uint4*>(src));
            else {
              uint32_t x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = src[2 * j] | (uint32_t)src[2 * j + 1] << 16;
              v[a] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
          r += STEP;
          i += dq;
          g += dr;
          if (g >= P.group) {
            g -= P.group;
            ++i;
          }
        }
#pragma unroll
        for (int a = 0; a < B; ++a) {
          const int rr = rr0 + (e + a) * STEP;
          *reinterpret_cast<uint4*>(smem + (rr >> 7) * SB + (c >> 3) * (kPTile * 128) + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v[a];
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sh.tmem;

  if (warp >= 8) {
    // (the launch has 168 registers a thread: 2 x 128 x 208 + 128 x 88 = 384 x 168)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 && n > 0) {
      // ================= copies
      bool ok = true;
      int keys = 0, values = 0;  // copied
#pragma unroll 1
      for (int it = 0; it < items; ++it) {
        const PromptItem a = prompt_item<PAIR>(it, n);
        if (it >= kPFirst) {
          if (a.k >= STAGES)
            ok = __all_sync(0xffffffffu, kv16_wait(a.v ? &sh.vempty[a.k % STAGES] : &sh.kempty[a.k % STAGES], (uint32_t)(a.k / STAGES - 1) & 1u, &sh.abort, P.wait_ns));
          if (!ok) break;
          issue(it);
        }
        if (a.v) ++values; else ++keys;
      }
      if (lane == 0) {
        sh.keys = keys;
        sh.values = values;
      }
    } else if (warp <= 10 && n > 0) {
      // ================= MMAs: a warp for each of the two products, one lane of it waits and issues.  (One warp for
      // both spends some 200 clocks on each of four waits a turn, ready or not, while the tensor cores run dry.)
      const int w = warp - 9;
      if (kv16_elect()) {
        const uint64_t qdesc = prompt_desc(smem_u32(smem), 16) + (PAIR ? w * (SB / 16) : 0), kdesc = prompt_desc(smem_u32(ring), 16),
                       vdesc = prompt_desc(smem_u32(ring + STAGES * SB), kPTile * 128);  // (an address's 16-byte units add in the low bits)
        const uint32_t sdesc = prompt_idesc<BF>(kPTile, false), odesc = prompt_idesc<BF>(D, true);
        const uint32_t ts = tmem + w * 128, to = tmem + 256 + w * D;
        auto scores = [&](int k) {  // S = Q K^T of tile k
          const uint64_t kk = kdesc + (k % STAGES) * (SB / 16);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = ((c >> 2) * (kPTile * 128) + (c & 3) * 32) / 16;
            prompt_mma_ss(ts, qdesc + off, kk + off, sdesc, c != 0);
          }
          prompt_commit(&sh.sfull[w]);
          prompt_commit(&sh.kempty[k % STAGES]);
        };
        const int k1 = PAIR ? 0 : w;
        bool ok = true;
        if (k1 < n) ok = kv16_wait(&sh.kfull[k1 % STAGES], 0, &sh.abort, P.wait_ns);
        if (ok && k1 < n) scores(k1);
#pragma unroll 1
        for (int t = 0; ok; ++t) {
          const int k = PAIR ? t : 2 * t + w, next = PAIR ? t + 1 : k + 2;
          if (k >= n) break;
          ok = kv16_wait(&sh.clean[k % STAGES], (uint32_t)(k / STAGES) & 1u, &sh.abort, P.wait_ns);
          const uint64_t vv = vdesc + (k % STAGES) * (SB / 16);
#pragma unroll 1
          for (int half = 0; half < 2 && ok; ++half) {  // O += P V, half the tokens
            ok = kv16_wait(&sh.pready[w][half], (uint32_t)t & 1u, &sh.abort, P.wait_ns);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
            for (int c = 0; c < kPTile / 32; ++c)
              prompt_mma_ts(to, ts + half * 32 + c * 8, vv + half * (64 * 128 / 16) + c * (2048 / 16), odesc, t + half + c > 0);
            if (half == 0) {
              prompt_commit(&sh.ohalf[w]);
              if (next < n) ok = kv16_wait(&sh.kfull[next % STAGES], (uint32_t)(next / STAGES) & 1u, &sh.abort, P.wait_ns);
            }
          }
          if (!ok) break;
          prompt_commit(&sh.vempty[k % STAGES]);
          if (next < n) scores(next); else prompt_commit(&sh.oend[w]);
        }
        // every MMA issued completes before the CTA ends
        prompt_commit(&sh.last[w]);
        kv16_drain(&sh.last[w], 0);
      }
      __syncwarp();
    } else if (n > 0) {
      // ================= values looked over, tile by tile as they land
      bool ok = true;
      for (int k = 0; k < n && ok; ++k) {
        ok = kv16_wait(&sh.vfull[k % STAGES], (uint32_t)(k / STAGES) & 1u, &sh.abort, P.wait_ns);
        if (!ok) break;
        {
          const int t0 = T.tile(k0 + k) * kPTile;
          const uint32_t held = *(volatile uint32_t*)&sh.held[k % kPHeld];
          if (held != 0xFFu || !kv16_whole<kPTile>(P, s, i0, i1, t0)) {
            uint4* vt = reinterpret_cast<uint4*>(ring + (STAGES + k % STAGES) * SB);
            // an exponent of ones carries into the sign's place when one is added to it
            constexpr uint32_t E = BF ? 0x7F807F80u : 0x7C007C00u, ONE = BF ? 0x00800080u : 0x04000400u;
            uint32_t found = 0;
#pragma unroll 8
            for (int e = lane; e < SB / 16; e += 32) {
              const uint4 u = vt[e];
              found |= ((u.x & E) + ONE) | ((u.y & E) + ONE) | ((u.z & E) + ONE) | ((u.w & E) + ONE);
            }
            if (found & 0x80008000u) {
              sh.bad = 1;
              bool bad = false;
              for (int e = lane; e < SB / 16; e += 32) {
                uint4 u = vt[e];
                u.x = kv16_finite<BF>(u.x, bad);
                u.y = kv16_finite<BF>(u.y, bad);
                u.z = kv16_finite<BF>(u.z, bad);
                u.w = kv16_finite<BF>(u.w, bad);
                vt[e] = u;
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
          }
        }
        mbar_arrive(&sh.clean[k % STAGES]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ================= rows
    const int w = warp >> 2, row = tid & 127;

    const int pr = r0 + (PAIR ? w * 128 : 0) + row, i = pr < packed ? pr / P.group : -1;
    const Kv16Row vis = kv16_row(P, s, i);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, sa = tmem + lanes + w * 128, oa = tmem + lanes + 256 + w * D;
    const float sl = P.scale_log2;
    float m = -INFINITY, l = 0.0f;
    float high_most = -INFINITY, high_least = -INFINITY;  // exponents between which a half's largest leaves the base where it is
    bool ok = true, tall = false;
    int t = 0;
    for (; (PAIR ? t : 2 * t + w) < n; ++t) {
      const int k = PAIR ? t : 2 * t + w, t0 = T.tile(k0 + k) * kPTile;
      ok = __all_sync(0xffffffffu, kv16_wait(&sh.sfull[w], (uint32_t)t & 1u, &sh.abort, P.wait_ns));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      uint32_t xs[2][64];
      tmem_ld32(sa, xs[0]);
      tmem_ld32(sa + 32, xs[0] + 32);
      const uint32_t held = *(volatile uint32_t*)&sh.held[k % kPHeld];
      const bool whole = held == 0xFFu && kv16_whole<kPTile>(P, s, i0, i1, t0);
      tmem_wait_ld();
      tmem_ld32(sa + 64, xs[1]);
      tmem_ld32(sa + 96, xs[1] + 32);
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // 64 positions at a time: the first half's product runs beside the second's weights
        uint32_t(&x)[64] = xs[half];
        if (half == 1) tmem_wait_ld();
        float f = sl;
        if (!whole) {
          // a warp's rows that see all of the half need no mask, those that see none of it weigh nothing
          const unsigned long long see = prompt_sees(P, s, vis, t0 + 64 * half, held >> (4 * half));
          if (__all_sync(0xffffffffu, see == 0)) {
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) p[c] = 0;
            tmem_st32(sa + 32 * half, p);
            tmem_wait_st();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            mbar_arrive(&sh.pready[w][half]);
            continue;
          }
          if (!__all_sync(0xffffffffu, see == ~0ull)) {
            const uint32_t never = f > 0.0f ? 0xFF800000u : 0x7F800000u;  // -infinity once scaled
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = (c < 32 ? (uint32_t)see : (uint32_t)(see >> 32)) & (1u << (c & 31)) ? x[c] : never;
          }
        }
        // weights by the maximum so far, while the scores' excess over it is found
        float high, sum;
#pragma unroll 1
        for (bool again = false;; again = true) {
          prompt_weights<BF>(x, f, m == -INFINITY ? 0.0f : m, sa + 32 * half, high, sum);
          const bool raise = !BF && high < high_least && high > -INFINITY, own = high > high_most || raise;
          if (again || !__any_sync(0xffffffffu, own)) break;
          // some row's base moves: again, each row by its own decision (one that would have kept its weights gets the same ones)
          const float sign = f < 0.0f ? -1.0f : 1.0f;
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; ++c) top = fmaxf(top, sign * __uint_as_float(x[c]));
          top *= sign * f;
          float low = INFINITY;  // the lowest score that the row sees
          if (!BF) {
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const float y = sign * __uint_as_float(x[c]);
              low = fminf(low, y == -INFINITY ? INFINITY : y);
            }
            low *= sign * f;
          }
          if (own && !(fabsf(top) < 1048576.0f) && top != -INFINITY && f != 1.0f) {
            // such scores are rounded like the maximum before the difference
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f);
            f = 1.0f;
          }
          const bool grow = own && top - m > P.grow;  // (a difference: m + grow may round past it)
          if (!BF) tall |= raise || (grow && top - low > 20.0f);
          const float next = grow ? kv16_base<BF>(top, tall ? P.lift + kPTall : P.lift) : (raise ? __fsub_ru(m, kPTall) : m);
          const float fade = grow || raise ? kv16_exp2(m - next) : 1.0f;
          l *= fade;
          m = next;
          // (a base of 2^20 and more: the exact products lie off its rounding by whole powers of two, so every half is gone over again)
          high_most = fabsf(m) < 1048576.0f ? P.grow : -INFINITY;
          if (!BF) high_least = tall || m == -INFINITY ? -INFINITY : -8.0f;
          if (t + half > 0) {
            // (the scores of this tile came after the products of the tile before)
            if (half == 1) ok = __all_sync(0xffffffffu, kv16_wait(&sh.ohalf[w], (uint32_t)t & 1u, &sh.abort, P.wait_ns));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(oa + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fade);
              tmem_st32(oa + c, o);
            }
          }
          tmem_wait_st();  // (the weights are written again)
        }
        if (!ok) break;
        l += sum;
        tmem_wait_st();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive(&sh.pready[w][half]);
      }
      if (!ok) break;
    }
    if (!ok) {  // loads and stores of TMEM that were under way
      tmem_wait_ld();
      tmem_wait_st();
    }
    if (ok && t > 0) ok = __all_sync(0xffffffffu, kv16_wait(&sh.oend[w], 0, &sh.abort, P.wait_ns));
    if (!ok && P.status) atomicCAS(P.status, 0, kStatusTimeout);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const bool have = t > 0;  // O holds something
    // Columns that this warpgroup writes: all of its own rows' (PAIR), or its half of the one block's, the other
    // product's sums of which come through the ring once both products have read it.
    constexpr int COLS = PAIR ? D : D / 2;
    const int first = PAIR ? 0 : w * COLS;
    float* mine_s = reinterpret_cast<float*>(ring) + w * (128 * COLS);   // [COLS][128]
    const float* other_s = reinterpret_cast<float*>(ring) + (1 - w) * (128 * COLS);
    float f0 = 1.0f, f1 = 0.0f;
    asm volatile("bar.sync 1, 256;" ::: "memory");  // (also: all values have been looked over)
    const bool go = *(volatile int*)&sh.abort == 0;  // the same in all warps: a warp that gave up set it before
    if (!PAIR) {
      sh.m[w][row] = m;
      sh.l[w][row] = l;
      if (go) {
#pragma unroll 1
        for (int c = 0; c < COLS; c += 32) {
          uint32_t o[32];
          if (have) {
            tmem_ld32(oa + (1 - w) * COLS + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) mine_s[(c + j) * 128 + row] = have ? __uint_as_float(o[j]) : 0.0f;
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float m1 = sh.m[1 - w][row], next = fmaxf(m, m1), base = next == -INFINITY ? 0.0f : next;
      f0 = kv16_exp2(m - base);
      f1 = kv16_exp2(m1 - base);
      l = l * f0 + sh.l[1 - w][row] * f1;
      m = next;
    }
    if (go) {
      const bool write = i >= 0, bad = *(volatile int*)&sh.bad != 0;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      unsigned char* part = ring + (PAIR ? w : 1) * (128 * D * 4);  // a share's sums [128][D] (behind what went between the products)
      unsigned char* whole = smem + (PAIR ? w * SB : 0);            // outputs [128][D]: the queries' place, which nothing reads any more
#pragma unroll 1
      for (int c = first; c < first + COLS; c += 32) {
        __syncwarp();
        uint32_t o[32];
        if (have) {
          tmem_ld32(oa + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        float fine = 0.0f, y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          y[j] = __uint_as_float(o[j]);
          if (!PAIR) y[j] = y[j] * f0 + other_s[(c - first + j) * 128 + row] * f1;
          fine = fmaf(y[j], 0.0f, fine);
        }
        // Values that are not finite: those left out of tiles that some row does not see whole, and all of them
        // where a sum shows one.  (With a NaN among the scores the row is NaN anyway.)
        const bool shown = write && fabsf(l) < INFINITY && fine != 0.0f, any = __any_sync(0xffffffffu, shown);
        if (any || bad) {
          // the warp together for the tiles that all rows see, a lane every eighth position of eight channels
          uint32_t bits = kv16_odd_shared<BF, D, kPTile>(P, s, T, b, h, i0, i1, k0, n, c + 8 * (lane & 3), lane >> 2, 8, any), own[4];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
#pragma unroll
          for (int g = 0; g < 4; ++g) own[g] = __shfl_sync(0xffffffffu, bits, g);
          if (write && fabsf(l) < INFINITY) {
            kv16_odd_own<BF, D, kPTile, 4>(P, s, vis, T, b, h, i0, i1, k0, n, c, own);
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = kv16_odd_sum(own[j / 8], j % 8, y[j]);
          }
        }
        if (!write) continue;
        if (P.splits > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(part + prompt_out<2 * D>(row, c / 4 + j)) = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        } else {
          uint32_t z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = kv16_pack<BF>(y[2 * j] * inv, y[2 * j + 1] * inv);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(whole + prompt_out<D>(row, c / 8 + j)) = make_uint4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
        }
      }
      if (write && (PAIR || w == 0)) {
        const long long at = (long long)(s.start + i) * P.nq + h * P.group + (pr - i * P.group);
        if (P.splits > 1)
          reinterpret_cast<float2*>(P.work + (long long)P.splits * P.n_rows * P.nq * D)[(long long)split * P.n_rows * P.nq + at] = make_float2(m, l);
        else if (P.lse)
          P.lse[at] = kv16_lse(P, m, l);
      }
      // whole rows' pieces of 16 bytes from shared memory: neighbouring threads, neighbouring pieces
      asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
      const bool shares = P.splits > 1;
      const int pieces = shares ? COLS / 4 : COLS / 8, step = 128 / pieces, c = row % pieces + first / (shares ? 4 : 8);
      const int dq = step / P.group, dr = step - dq * P.group;
      int rr = row / pieces, r = r0 + (PAIR ? w * 128 : 0) + rr, ii = r / P.group, g = r - ii * P.group;
#pragma unroll 4
      for (; rr < 128 && r < packed; rr += step, r += step) {
        if (shares) {
          float* dst = P.work + ((long long)split * P.n_rows * P.nq + (long long)(s.start + ii) * P.nq + h * P.group + g) * D + 4 * c;
          *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(part + prompt_out<2 * D>(rr, c));
        } else {
          const uint4 z = *reinterpret_cast<const uint4*>(whole + prompt_out<D>(rr, c));
          unsigned short* dst = P.o + (long long)(s.start + ii) * P.os + (long long)(h * P.group + g) * D + 8 * c;
          if (P.ovec) *reinterpret_cast<uint4*>(dst) = z;
          else {
            const uint32_t zz[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[j] = (unsigned short)(zz[j >> 1] >> (16 * (j & 1)));
          }
        }
        ii += dq;
        g += dr;
        if (g >= P.group) {
          g -= P.group;
          ++ii;
        }
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  if (warp == 8 && sh.abort) {  // nothing in flight at exit: whoever gave up, copies may not have landed
    for (int k = max(0, sh.keys - STAGES); k < sh.keys; ++k) kv16_drain(&sh.kfull[k % STAGES], (uint32_t)(k / STAGES) & 1u);
    for (int k = max(0, sh.values - STAGES); k < sh.values; ++k) kv16_drain(&sh.vfull[k % STAGES], (uint32_t)(k / STAGES) & 1u);
  }
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace cpk

namespace cpk_host {

using namespace cpk;

template <int D, bool BF>
static cudaError_t launch(const Kv16Call& P, bool pair, cudaStream_t s) {
  const void* fn = pair ? (const void*)kv16_prompt_kernel<D, BF, true> : (const void*)kv16_prompt_kernel<D, BF, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.splits * P.mtiles), (unsigned)P.nkv, (unsigned)P.n_seqs);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = prompt_smem(D);
  cfg.stream = s;
  cudaError_t e = ops4_smem_limit(fn, cfg.dynamicSmemBytes);
  Kv16Call call = P;
  void* args[] = {&call};
  return e == cudaSuccess ? cudaLaunchKernelExC(&cfg, fn, args) : e;
}

cudaError_t launch_kv16_prompt(const Kv16Call& P, int d, bool bf, bool pair, cudaStream_t s) {
  if (d == 64) return bf ? launch<64, true>(P, pair, s) : launch<64, false>(P, pair, s);
  return bf ? launch<128, true>(P, pair, s) : launch<128, false>(P, pair, s);
}

}  // namespace cpk_host
