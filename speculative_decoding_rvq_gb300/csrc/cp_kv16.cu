// cp_kv16.cu -- the steps of an outer model's pass around its attention: page
// tables and slot maps from request lengths, rotary embedding over several
// position axes, and rows written into the 16-bit paged KV cache.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cp_fp4.cuh"
#include "cp_kv16.h"
#include "cp_ops4.h"

namespace cpk {

using cpk_host::KvPlan;
using cpk_host::kPlanMaxSeqs;
using cpk_host::RopeRows;

// ------------------------------------------------- page tables, slot maps
// A step of the pool: sequence b keeps len tokens, adds new rows and needs
// need = ceil((len + new) / page) pages.  Pages past the need go back to the
// stack of free ones, lacking ones come from its top; all positions follow from
// prefix sums over the sequences:
//   given before b   G[b] = sum of (held - need)+
//   taken before b   T[b] = sum of (need - held)+ of the served sequences
//   rows before b    R[b] = sum of new of the served sequences.
// The returned pages are pushed last sequence and last page first, the lacking
// ones popped first sequence and first page first, so a step that gives back
// what the step before took restores the stack.
//
// One cluster of C CTAs.  Every CTA forms all prefix sums for itself (12 bytes a
// sequence from L2: cheaper than handing them over), the entries of the table
// and the stack, and the rows, are then dealt to all threads, each finding its
// sequence by bisection in shared memory.  Two cluster barriers: the lengths and
// counts are read before they are replaced, and the pushes come before the pops.
// Bound by that chain of loads and sums: 64 sequences and 256 rows 3.5 us (one
// CTA; an empty kernel takes 1.1), 512 sequences taking 8000 pages 10 us with the
// slots of 523,776 rows (a cluster, and a second kernel over all SMs for the rows).
struct PlanShared {
  long long sum[32][3];
  long long total[3];
  int need[kPlanMaxSeqs], had[kPlanMaxSeqs], len[kPlanMaxSeqs];
  int G[kPlanMaxSeqs + 1], T[kPlanMaxSeqs + 1], R[kPlanMaxSeqs + 1];
};

// Exclusive prefix sums of three numbers over the threads of the CTA; the totals in sh.total.
__device__ __forceinline__ void plan_scan(PlanShared& sh, long long (&v)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long own[3];
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    own[c] = v[c];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v[c], o);
      if (lane >= o) v[c] += u;
    }
    if (lane == 31) sh.sum[warp][c] = v[c];
  }
  __syncthreads();
  if (warp < 3) {
    long long u = lane < warps ? sh.sum[lane][warp] : 0;
    const long long mine = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long w = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += w;
    }
    if (lane < warps) sh.sum[lane][warp] = u - mine;
    if (lane == 31) sh.total[warp] = u;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 3; ++c) v[c] += sh.sum[warp][c] - own[c];
}

// The last b < n with at[b] <= i, for i < at[n].
__device__ __forceinline__ int plan_find(const int* at, int n, int i) {
  int lo = 0, hi = n;  // at[lo] <= i < at[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void plan_row(const KvPlan& P, const int* R, const int* len, int r, int shift, int* pos, long long* slot) {
  *pos = 0;
  *slot = -1;
  if (r >= R[P.n_seqs]) return;
  const int b = plan_find(R, P.n_seqs, r);
  *pos = len[b] + (r - R[b]);
  const int at = shift >= 0 ? *pos >> shift : *pos / P.page_size;
  const int id = load_l2(P.pages + (long long)b * P.max_pages + at);
  if (id >= 0 && id < P.n_pages) *slot = (long long)id * P.page_size + (*pos - at * P.page_size);
}

template <int C>
__global__ void __launch_bounds__(1024, 1) kv_plan_kernel(const __grid_constant__ KvPlan P, int shift, int fill) {
  extern __shared__ __align__(16) unsigned char plan_smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(plan_smem);
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, rank = C > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int each = (P.n_seqs + blockDim.x - 1) / blockDim.x, b0 = min(tid * each, P.n_seqs), b1 = min(b0 + each, P.n_seqs);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n_free = min(max(load_l2(P.n_free), 0), P.n_pages);
  // first sums: what each sequence gives back, lacks, and adds
  long long v[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int len = max(__ldg(P.len + b), 0), held = min(max(load_l2(P.held + b), 0), P.max_pages);
    const long long fresh = P.fresh ? max(__ldg(P.fresh + b), 0) : 0, want = len + fresh;
    const long long need = shift >= 0 ? (want + P.page_size - 1) >> shift : (want + P.page_size - 1) / P.page_size;
    sh.len[b] = len;
    sh.had[b] = held;
    sh.need[b] = need <= P.max_pages ? (int)need : -1;  // -1: more than the table holds
    sh.G[b] = (int)fresh;                               // (kept there until the second sums)
    v[0] += need <= P.max_pages ? max(held - (int)need, 0) : 0;
    v[1] += need <= P.max_pages ? max((int)need - held, 0) : 0;
    v[2] += fresh;
  }
  plan_scan(sh, v);
  const long long given = sh.total[0], there = n_free + given;
  const int full = (int)min(there, (long long)P.n_pages);  // (more than n_pages only if the caller's lists hold a page twice)
  // second sums: only what the served sequences take and add
  long long lacks = v[1], asks = v[2], w[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int need = sh.need[b], lack = need < 0 ? 0 : max(need - sh.had[b], 0), fresh = sh.G[b];
    lacks += lack;
    asks += fresh;
    const int why = need < 0 ? 2 : (lack > 0 && lacks > full ? 1 : (fresh > 0 && asks > P.n_rows ? 3 : 0));
    sh.T[b] = why == 0 ? lack : 0;
    sh.R[b] = why == 0 ? fresh : -1 - why;
    w[1] += why == 0 ? lack : 0;
    w[2] += why == 0 ? fresh : 0;
  }
  __syncthreads();  // (sh.total is read before it is written again)
  plan_scan(sh, w);
  const int taken = (int)sh.total[1];
  long long g = v[0], t = w[1], r = w[2];
  if (C > 1) cg::this_cluster().sync();  // every CTA has read the counts that are replaced now
  for (int b = b0; b < b1; ++b) {
    const int why = sh.R[b] < 0 ? -1 - sh.R[b] : 0, rows = why ? 0 : sh.R[b], take = sh.T[b];
    const int give = sh.need[b] < 0 ? 0 : max(sh.had[b] - sh.need[b], 0), held = sh.had[b] - give + take;
    sh.G[b] = (int)g;
    sh.T[b] = (int)t;
    sh.R[b] = (int)r;
    if (b % C == rank) {
      P.held[b] = held;
      P.kv_len[b] = (int)(why ? min((long long)sh.len[b], (long long)held * P.page_size) : (long long)sh.len[b] + rows);
      P.row_start[b] = (int)r;
      if (P.refused) P.refused[b] = why;
    }
    g += give;
    t += take;
    r += rows;
  }
  if (b0 < P.n_seqs && b1 == P.n_seqs) {
    sh.G[b1] = (int)g;
    sh.T[b1] = (int)t;
    sh.R[b1] = (int)r;
    if (rank == 0) {
      P.row_start[b1] = (int)r;
      *P.n_free = full - taken;
    }
  }
  __syncthreads();
  const int step = C * blockDim.x, first = rank * blockDim.x + tid;
  // pages given back: entry e of the list in order of (sequence, page), pushed from its end (up to 2^31 - 1 of them: e passes 31 bits)
  for (long long e = first; e < given; e += step) {
    const int b = plan_find(sh.G, P.n_seqs, (int)e);
    int* at = P.pages + (long long)b * P.max_pages + sh.need[b] + (e - sh.G[b]);
    const long long to = n_free + given - 1 - e;
    if (to < P.n_pages) P.free[to] = load_l2(at);
    *at = -1;
  }
  if (given > 0 && taken > 0) {  // the same in every CTA
    if (C > 1) cg::this_cluster().sync(); else __syncthreads();
  }
  for (long long e = first; e < taken; e += step) {
    const int b = plan_find(sh.T, P.n_seqs, (int)e);
    P.pages[(long long)b * P.max_pages + sh.had[b] + (e - sh.T[b])] = load_l2(P.free + (full - 1 - e));
  }
  if (!fill) return;
  if (taken > 0) {
    if (C > 1) cg::this_cluster().sync(); else __syncthreads();
  }
  for (int i = first; i < P.n_rows; i += step) {
    int pos;
    long long slot;
    plan_row(P, sh.R, sh.len, i, shift, &pos, &slot);
    P.pos[i] = pos;
    P.slot[i] = slot;
  }
}

// Positions and slots of many rows: a kernel of its own over all SMs, started
// while the plan runs.
__global__ void __launch_bounds__(256) kv_slots_kernel(const __grid_constant__ KvPlan P, int shift) {
  extern __shared__ __align__(16) unsigned char plan_smem[];
  int* R = reinterpret_cast<int*>(plan_smem);
  int* len = R + P.n_seqs + 1;
  for (int b = threadIdx.x; b < P.n_seqs; b += 256) len[b] = max(__ldg(P.len + b), 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int b = threadIdx.x; b <= P.n_seqs; b += 256) R[b] = load_l2(P.row_start + b);
  __syncthreads();
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < P.n_rows; i += gridDim.x * 256ll) {
    int pos;
    long long slot;
    plan_row(P, R, len, (int)i, shift, &pos, &slot);
    P.pos[i] = pos;
    P.slot[i] = slot;
  }
}

// ------------------------------------------- rotary embedding, cache write
// Pair i of a head (channels i and i + rot / 2) turns by the position of its
// axis times its frequency.  The angle is formed exactly in fixed point: the
// frequency in turns as a 64-bit fraction times the integer position, modulo
// one turn, then the nearest quarter turn split off; what is left is rounded to
// float32, so far positions lose nothing.
__device__ __forceinline__ void rope_angle(long long pos, unsigned long long turns, float& c, float& s) {
  const unsigned long long t = (unsigned long long)pos * turns;
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62) & 3u;
  const int rest = (int)((long long)(t - ((unsigned long long)quarter << 62)) >> 30);  // 1/8 turn is 2^31
  float sn, cs;
  sincospif((float)rest * 0x1p-33f, &sn, &cs);  // half turns: 2^-34 turns times 2
  const float a = quarter & 1u ? sn : cs, b = quarter & 1u ? cs : sn;
  c = quarter == 1u || quarter == 2u ? -a : a;
  s = quarter & 2u ? -b : b;
}

// Eight neighbouring elements as they are stored.
template <int DT, bool VEC>
struct RopeVec {
  static constexpr int kWords = DT == kF32 ? 8 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, long long at) {
    const unsigned char* a = static_cast<const unsigned char*>(p) + at * (DT == kF32 ? 4 : 2);
    if (VEC) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(a) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    } else if (DT == kF32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(a)[i];
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(a);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
  }
  __device__ __forceinline__ void store(void* p, long long at, bool vec) const {
    unsigned char* a = static_cast<unsigned char*>(p) + at * (DT == kF32 ? 4 : 2);
    if (VEC || vec) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(a)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if (DT == kF32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(a)[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) reinterpret_cast<uint16_t*>(a)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if (DT == kF32) f[i] = __uint_as_float(w[i]);
      else {
        const float2 x = DT == kBF16 ? bf16x2_to_f2(w[i]) : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i % 8] = x.x;
        f[(2 * i + 1) % 8] = x.y;
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if (DT == kF32) w[i] = __float_as_uint(f[i]);
      else if (DT == kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i % 8], f[(2 * i + 1) % 8]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i % 8], f[(2 * i + 1) % 8]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};

// A CTA takes R rows with all their heads.  Its threads first form each row's
// sines and cosines once, in shared memory, with the first heads' loads already
// in flight; then a thread keeps one row and one pair of 8-channel pieces (d / 16
// of them a head: the rotating pairs first, then the channels past rot two pieces
// at a time) and walks through every G-th of the query, key and value heads, the
// next two heads' loads in flight while it turns two.  Bound by the rows' bytes:
// 16384 rows of 32 heads x 128 channels (bfloat16) 50.8 us, 5.3 TB/s, 78 % of a
// copy's rate (61 us where every five threads of a row formed its sines again).
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) rope_rows_kernel(const __grid_constant__ RopeRows P, int units, int R, int G) {
  extern __shared__ float2 rope_turns[];  // [R][pairs] (cosine, sine)
  const int tid = threadIdx.x, pairs = P.pos ? P.rope.rot_dim / 2 : 0, rots = pairs / 8, heads = P.nq + P.nk + P.nv;
  const int rg = tid / units, u = tid - rg * units, g = rg / R, rr = rg - g * R;
  const long long first = (long long)blockIdx.x * R, row = first + rr;
  bool on = g < G && row < P.n_rows;
  long long cell = 0;  // element of (page, slot in it) for head 0
  if (on && P.slot) {
    const long long slot = __ldg(P.slot + row);
    on = slot >= 0 && slot < P.n_slots;
    const long long page = slot >> P.page_shift;
    cell = (((page * P.nk) << P.page_shift) + (slot - (page << P.page_shift))) * P.d;
  }
  const bool turns = u < rots;
  const int lo = turns ? 8 * u : 16 * u, hi = turns ? lo + pairs : lo + 8;
  RopeVec<DT, VEC> x[2], y[2];
  auto load = [&](int h, RopeVec<DT, VEC>& a, RopeVec<DT, VEC>& b) {
    if (!on || h >= heads) return;
    const bool is_q = h < P.nq, is_k = !is_q && h < P.nq + P.nk;
    const void* src = is_q ? P.q : (is_k ? P.k : P.v);
    const long long from = row * (is_q ? P.qs : (is_k ? P.ks : P.vs)) + (long long)(is_q ? h : (is_k ? h - P.nq : h - P.nq - P.nk)) * P.d;
    a.load(src, from + (is_q || is_k ? lo : 16 * u));  // (the values' pieces are plain 16 channels)
    b.load(src, from + (is_q || is_k ? hi : 16 * u + 8));
  };
  load(g, x[0], y[0]);
  load(g + G, x[1], y[1]);
  for (int e = tid; e < R * pairs; e += 256) {
    const int r = e / pairs, i = e - r * pairs;
    if (first + r < P.n_rows) {
      float c, s;
      rope_angle(__ldg(P.pos + P.rope.axis[i] * P.pos_stride + first + r), P.rope.turns[i], c, s);
      rope_turns[e] = make_float2(c, s);
    }
  }
  __syncthreads();
  if (!on) return;
  float c[8], s[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(rope_turns + rr * pairs + lo + 2 * i);
      c[2 * i] = t.x; s[2 * i] = t.y; c[2 * i + 1] = t.z; s[2 * i + 1] = t.w;
    }
  }
  for (int h0 = g; h0 < heads; h0 += 2 * G) {
    RopeVec<DT, VEC> nx[2], ny[2];
    load(h0 + 2 * G, nx[0], ny[0]);
    load(h0 + 3 * G, nx[1], ny[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = h0 + e * G;
      if (h >= heads) break;
      const bool is_q = h < P.nq, is_k = !is_q && h < P.nq + P.nk, held = !is_q && P.slot != nullptr;
      const int hh = is_q ? h : (is_k ? h - P.nq : h - P.nq - P.nk);
      void* dst = is_q ? P.qo : (held ? (void*)(is_k ? P.keys : P.values) : P.ko);
      const long long to = held ? cell + ((long long)hh << P.page_shift) * P.d : row * (is_q ? P.qos : P.kos) + (long long)hh * P.d;
      if (turns && (is_q || is_k)) {
        float a[8], b[8], p[8], q[8];
        x[e].get(a);
        y[e].get(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = a[i] * c[i] - b[i] * s[i];
          q[i] = b[i] * c[i] + a[i] * s[i];
        }
        x[e].put(p);
        y[e].put(q);
      }
      x[e].store(dst, to + (is_q || is_k ? lo : 16 * u), held);
      y[e].store(dst, to + (is_q || is_k ? hi : 16 * u + 8), held);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[e] = nx[e];
      y[e] = ny[e];
    }
  }
}

}  // namespace cpk

namespace cpk_host {

using namespace cpk;

cudaError_t launch_kv_plan(const KvPlan& P, int* kernels, cudaStream_t s) {
  const int shift = (P.page_size & (P.page_size - 1)) == 0 ? __builtin_ctz(P.page_size) : -1;
  // Few rows and table entries: one CTA, without cluster barriers.  Many rows: their slots by a second kernel.
  const long long entries = (long long)P.n_seqs * P.max_pages;
  const bool one = P.n_rows <= 2048 && entries <= 16384 && P.n_seqs <= 1024, fill = P.n_rows <= 16384;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(one ? 1 : 8);
  cfg.blockDim = dim3(one && P.n_seqs <= 256 && P.n_rows <= 256 ? 256 : 1024);
  cfg.dynamicSmemBytes = sizeof(PlanShared);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 8;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = one ? 0 : 1;
  const void* fn = one ? (const void*)kv_plan_kernel<1> : (const void*)kv_plan_kernel<8>;
  int sh = shift, fl = fill;
  KvPlan p = P;
  void* args[] = {&p, &sh, &fl};
  cudaError_t e = ops4_smem_limit(fn, cfg.dynamicSmemBytes);
  if (e == cudaSuccess) e = cudaLaunchKernelExC(&cfg, fn, args);
  *kernels = 1;
  if (e != cudaSuccess || fill) return e;
  cudaLaunchConfig_t c2 = {};
  c2.gridDim = dim3((unsigned)std::min<long long>((P.n_rows + 255ll) / 256, 608));
  c2.blockDim = dim3(256);
  c2.dynamicSmemBytes = (2 * (size_t)P.n_seqs + 1) * 4;
  c2.stream = s;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c2.attrs = at;
  c2.numAttrs = 1;
  void* args2[] = {&p, &sh};
  *kernels = 2;
  return cudaLaunchKernelExC(&c2, (const void*)kv_slots_kernel, args2);
}

template <int DT>
static cudaError_t rope_launch(const RopeRows& P, bool vec, unsigned grid, size_t smem, int units, int R, int G, cudaStream_t s) {
  if (vec) rope_rows_kernel<DT, true><<<grid, 256, smem, s>>>(P, units, R, G);
  else rope_rows_kernel<DT, false><<<grid, 256, smem, s>>>(P, units, R, G);
  return cudaGetLastError();
}

cudaError_t launch_rope_rows(const RopeRows& P, int sms, cudaStream_t s) {
  const int units = P.d / 16;
  // rows of a CTA: as many as leave four CTAs an SM, so that few rows fill the SMs (at most 16 pairs of pieces a head
  // times 8 rows: 128 threads a group of heads)
  int R = 8;
  while (R > 1 && (long long)P.n_rows < (long long)R * 4 * sms) R /= 2;
  const int G = 256 / (R * units);
  const size_t smem = P.pos ? (size_t)R * P.rope.rot_dim / 2 * 8 : 0;
  const int es = P.dtype == kF32 ? 4 : 2;
  auto even = [&](const void* p, long long stride) { return !p || (((uintptr_t)p & 15u) == 0 && stride * es % 16 == 0); };
  const bool vec = even(P.q, P.qs) && even(P.qo, P.qos) && even(P.k, P.ks) && even(P.ko, P.kos) && even(P.v, P.vs);
  const unsigned grid = (unsigned)((P.n_rows + R - 1) / R);
  switch (P.dtype) {
    case kF32: return rope_launch<kF32>(P, vec, grid, smem, units, R, G, s);
    case kBF16: return rope_launch<kBF16>(P, vec, grid, smem, units, R, G, s);
    default: return rope_launch<kF16>(P, vec, grid, smem, units, R, G, s);
  }
}

}  // namespace cpk_host
