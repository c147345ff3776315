// cp_ops4.h -- launchers of the 4-bit operators (cp_w4.cu, cp_kv4.cu), called
// by the C ABI in cp_spec.cu after its checks of arguments.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace cpk_host {

// Raise (never lower) a kernel's dynamic shared-memory limit on the current device.
cudaError_t ops4_smem_limit(const void* fn, size_t bytes);

size_t w4_bytes(int N, int K, int group);
cudaError_t launch_w4_pack(int N, int K, int group, int dtype, const void* w, long long stride, void* packed, cudaStream_t s);
cudaError_t launch_w4_unpack(int N, int K, int group, int dtype, const void* packed, void* w, cudaStream_t s);
cudaError_t launch_w4_gemv(int R, int N, int K, int group, int xdt, int ydt, const void* x, long long xs, const void* packed,
                           void* y, long long ys, int sms, cudaStream_t s);

struct Kv4Shape {
  int n_pages, page_size, nkv, d;
};
size_t kv4_bytes(int n_pages, int page_size, int nkv, int d);
cudaError_t launch_kv4_append(const Kv4Shape& S, void* cache, const int* pages, int max_pages, int B, int M, const int* pos,
                              const int* len, int dtype, const void* k, long long ks, const void* v, long long vs,
                              cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4Shape& S, const void* cache, const int* pages, int max_pages, int B, int T, const int* len,
                            int dtype, void* k, void* v, cudaStream_t s);

// Everything kv4_attention takes; row strides in elements.
struct Kv4Attention {
  const void* cache;
  const int* pages;
  const int* kv_len;  // [B] positions of each sequence, the window's rows among them
  const int* n_rows;  // [B] rows of the window that count, or null
  const unsigned long long* mask;  // [B][M] window rows that a row sees, or null: causal
  const void* q;
  void* o;
  float* lse;  // [B][M][nq] or null
  long long qs, os;
  int max_pages, B, M, nq, dtype;
  float scale;
  void* work;  // kv4_attention_work bytes
};
size_t kv4_attention_work(const Kv4Shape& S, int max_pages, int B, int M, int nq, int dtype, int sms);
// Readies the kernels of such a call on the current device, for a caller that captures its first one.
cudaError_t kv4_attention_configure(const Kv4Shape& S, int max_pages, int B, int M, int nq, int dtype);
cudaError_t launch_kv4_attention(const Kv4Shape& S, const Kv4Attention& A, int sms, cudaStream_t s);

}  // namespace cpk_host
