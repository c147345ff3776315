// cp_kv16.h -- launchers of the operators of the 16-bit paged KV cache
// (cp_kv16.cu, cp_kv16_attention.cu), called by the C ABI in cp_spec.cu after
// its checks of arguments.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/cp_spec.h"

namespace cpk_host {

// What cp_spec_kv_plan takes.
struct KvPlan {
  int n_seqs, max_pages, page_size, n_pages, n_rows;
  const int* len;
  const int* fresh;  // rows that each sequence adds, or null: none
  int* pages;
  int* held;
  int* free;
  int* n_free;
  int* kv_len;
  int* row_start;
  int* pos;
  long long* slot;
  int* refused;  // or null
};
constexpr int kPlanMaxSeqs = CP_SPEC_MAX_PLAN_SEQS;
cudaError_t launch_kv_plan(const KvPlan& P, int* kernels, cudaStream_t s);

// What the rotary embedding and the cache write take; strides in elements.
struct RopeRows {
  cp_spec_rope rope;
  const int* pos;  // [axes][pos_stride], null without rotation
  long long pos_stride;
  const long long* slot;  // [n_rows], null: no cache
  unsigned char* keys;    // [n_pages][kv heads][page][dim]
  unsigned char* values;
  const void* q;
  void* qo;
  const void* k;
  void* ko;  // without a cache
  const void* v;
  long long qs, qos, ks, kos, vs;
  long long n_slots;
  int n_rows, nq, nk, nv, d, dtype, page_shift;
};
cudaError_t launch_rope_rows(const RopeRows& P, int sms, cudaStream_t s);

struct Kv16Shape {
  int n_pages, page_size, nkv, d, dtype;
};
// Everything kv16_attention takes; row strides in elements.
struct Kv16Attention {
  const void* cache;
  const int* pages;               // [n_seqs][max_pages], or null: sequence b owns pages b * max_pages ..
  const int* kv_len;              // [n_seqs] positions of each sequence, its rows among them
  const int* row_start;           // [n_seqs + 1]
  const unsigned long long* mask; // [n_rows] window rows that a row sees, or null: causal
  const void* q;
  void* o;
  float* lse;  // [n_rows][nq] or null
  long long qs, os;
  int max_pages, n_seqs, n_rows, max_rows, nq, window, sinks;
  float scale;
  void* work;
  int* status;  // or null
  int stall;          // test hook: 1 the last copy of a CTA is not made, 2 none is
  uint64_t wait_ns;   // bound of every device-side wait
};
size_t kv16_attention_work(const Kv16Shape& S, const Kv16Attention& A, int sms);
cudaError_t launch_kv16_attention(const Kv16Shape& S, const Kv16Attention& A, int sms, int* kernels, cudaStream_t s);

}  // namespace cpk_host
