// cp_kv16_prompt.h -- the launcher of the tensor-core tiles of
// cp_kv16_prompt.cu, called by cp_kv16_attention.cu.
#pragma once
#include <cuda_runtime.h>

namespace cpk {
struct Kv16Call;
}

namespace cpk_host {
// Binary orders by which a score may pass a row's largest before its base follows (each move costs a pass over the row's sums).
constexpr float kPromptLate = 8.0f;
// pair: blocks of 256 packed rows; else 128 (P.mtiles counts them).
cudaError_t launch_kv16_prompt(const cpk::Kv16Call& P, int d, bool bf, bool pair, cudaStream_t s);
}  // namespace cpk_host
