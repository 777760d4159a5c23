// Parameter block and launcher of the partial kernel over an E2M1 cache.
#pragma once
#include <cuda_runtime.h>
#include <cuda_fp8.h>
#include <cstdint>

namespace mla {

struct Fp4Params {
  const void* q_abs;
  const void* q_pe;
  const uint8_t* kv_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const void* kv_cur;
  void* o_part;
  float* lse_part;
  int* err;
  int B, q_len, H, num_blocks, bs, max_blocks, S, P, head_slices;
  float scale_log2;      // softmax scale * log2(e)
  float kv_scale;
  int part_dtype;        // 0 bf16, 1 fp16, 2 fp32
};
int launch_partial_fp4(const Fp4Params& fp, bool bf16, cudaStream_t stream);

}  // namespace mla
