// Parameter block and launcher of the partial kernel over an E2M1 cache.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace mla {

constexpr int kFp4MaxCtas = 256;     // the partition keeps per-CTA state in arrays of this size
constexpr int kFp4MaxRows = 64;      // query rows of a unit, at most

// Shards of this many tiles or fewer are not cut where each has a CTA of its own: a
// cut gains their length at most, and costs the partition, a merge and the pieces'
// own ends (16 heads, 1 to 128 such shards of 8 tiles: whole 16 us, cut 16 to 21; of
// 12 and 16 tiles 21 and 26 against 17 to 26 and 17 to 31).
constexpr int kWholeTiles4 = 8;

// Query rows (query token, head) that a unit carries: the smallest of 16, 32
// and 64 that holds a sequence's rows, 64 where none does.
inline int fp4_unit_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct Fp4Params {
  const uint8_t* kv_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const void* kv_cur;
  void* o_part;
  float* lse_part;
  int* err;
  int B, q_len, H, num_blocks, bs, max_blocks, S, P, head_slices;
  int hs;                // heads of a slice
  uint32_t inv_H, inv_hs;   // 2^32 / H and / hs rounded up, 0 for 1
  int T;                 // B * q_len
  int R;                 // query rows of a sequence: q_len * H
  int G;                 // row groups of a sequence: R / rows, rounded up
  int num_units;         // G * B * P
  int box;               // tokens per copy: min(64, block size)
  int bs_shift;
  float scale_log2;      // softmax scale * log2(e)
  float kv_scale;
  int part_dtype;        // 0 bf16, 1 fp16, 2 fp32
  uint32_t spin_limit;
  // workspace (split: CTAs that share the tiles exactly, 0: whole units)
  int split;
  float* ws_o;           // pieces of O / l, [2 * ctas][rows][512]
  float* ws_lse;         // [2 * ctas][rows], log2
  int4* ws_units;        // [ctas]: {unit, its first tile, first CTA, last CTA} of the unit that ends here
  int* ws_bounds;        // [ctas + 1]: first tile of each CTA's share, then the tile total
};

inline size_t fp4_workspace_recs(int ctas) {
  return (static_cast<size_t>(ctas + 1) * (16 + 4) + 255) / 256 * 256;
}
inline size_t fp4_workspace_bytes(int ctas) {
  return fp4_workspace_recs(ctas) + 2 * static_cast<size_t>(ctas) * kFp4MaxRows * (4 + 512 * 4);
}
// CTAs of the kernel on the current device (one per SM); < 1 if it cannot run.
int fp4_max_ctas();
int launch_partial_fp4(const CUtensorMap& qlat, const CUtensorMap& qpe, const Fp4Params& fp, int rows,
                       bool bf16, cudaStream_t stream);

}  // namespace mla
