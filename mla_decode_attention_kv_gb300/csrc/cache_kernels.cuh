// Parameter blocks and launchers of the cache operators: the append, the page
// operations and the formats of a cached row that they share.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>
#include <utility>

namespace mla {

// Device error codes of the cache operators, after those of ptx.cuh.
enum CacheError : int {
  kDevBadSlot = 4,        // slots entry outside [-1, num_blocks * block_size)
  kDevBadPosition = 5,    // positions entry outside [0, max_pos)
  kDevBadRow = 6,         // a row id out of range, or a fork into a row that is taken
  kDevNoFreePage = 7,     // fewer free pages than a fork needs
  kDevBadRefCount = 8,    // a page given back that no row holds
};

// A programmatic launch: the grid's start overlaps the end of the one before it in
// the stream, for which every block waits (griddep_wait) before it reads or writes.
// Only behind that wait does a block let the next grid go (griddep_launch_dependents):
// a grid that does some reading before its own wait, the V-up's of W_UV, then still
// finds everything but its direct predecessor done.  What the grid before may have
// written (tables, ids, lengths) is read by plain loads: __ldg asks for data that
// nothing writes as long as the kernel lives, its time before the wait included.
// Calls back to back, without it and so: 8 pages copied 4.1 and 2.8 us, 8192 tokens
// appended 14.3 and 11.8, 64 rows forked 16.4 and 14.7.
template <class... A, class... B>
inline cudaError_t launch_overlapped(void (*kernel)(A...), dim3 grid, unsigned threads, cudaStream_t stream, B&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<B>(args)...);
}

// Formats of a cached row (mla_kv_format of the header).
enum KvKind : int { kKvModel = 0, kKvE4M3 = 1, kKvE2M1 = 2 };

// E2M1 pages: bs x 288 bytes of codes (two a byte, the even element in the low
// half), then bs x 36 E4M3 block scales (one for every 16 values).
constexpr int kE2m1Codes = 288;
constexpr int kE2m1Scales = 36;
constexpr int kE2m1Row = kE2m1Codes + kE2m1Scales;

constexpr int kAppendThreads = 64;      // (32 sequences' tokens, 128 heads: 4.0 us, 4.4 with 256)
constexpr int kQueryHeads = 16;         // heads of one token that a warp rotates
constexpr int kMaxForkRows = 65536;   // rows of a block table that mla_kv_fork takes

struct AppendParams {
  const void* c_kv;        // [T, 512], rows c_stride elements apart
  const void* k_pe;        // [T, 64], rows k_stride elements apart
  const void* q_pe;        // [T, H, 64] or nullptr
  const void* weight;      // [512] or nullptr (no norm)
  const float* cos_sin;    // [max_pos, 64]: 32 cosines, 32 sines
  const int32_t* positions;   // [axes, T]
  const int32_t* slots;    // [T], -1: stored nowhere
  void* cache;
  void* q_out;
  void* kv_out;            // [T, 576] or nullptr
  int* err;
  int64_t c_stride, k_stride, q_stride, q_head_stride, qo_stride, qo_head_stride;
  int T, H, max_pos, bs, num_slots;
  int sec1, sec2;          // first pair of the second and of the third axis (32: none)
  int interleaved;
  float eps, kv_scale, kv6;   // kv6 = 6 kv_scale
  float inv_kv, inv_kv6;      // their reciprocals, rounded
  int row_blocks, q_groups;   // blocks that make rows; warps per token that rotate queries
};
// Blocks of a launch: those that make rows, a warp a token, then those that rotate queries.
inline int64_t append_blocks(int64_t T, int64_t H) {
  constexpr int64_t kWarps = kAppendThreads / 32;
  return (T + kWarps - 1) / kWarps + (T * ((H + kQueryHeads - 1) / kQueryHeads) + kWarps - 1) / kWarps;
}
int launch_append(AppendParams ap, int kind, bool bf16, cudaStream_t stream);

// Pages of `page_bytes` in `layers` pools, `*_layer` bytes apart.
struct CopyParams {
  const char* src;
  char* dst;
  uint64_t src_layer, dst_layer, page_bytes;
  const int32_t* src_ids;
  const int32_t* dst_ids;
  int n, layers, src_blocks, dst_blocks;
  int chunks;              // blocks per page and layer
  int* err;
};
int launch_copy_pages(CopyParams cp, cudaStream_t stream);

struct ForkParams {
  char* cache;
  uint64_t layer, page_bytes;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  const int32_t* parents;
  const int32_t* children;
  int n, layers, rows, num_blocks, bs, max_blocks;
  int chunks;              // copy blocks per page and layer
  int32_t* ws;             // {state, -, -, -}, fresh page of each pair, list of free pages
  int* err;
};
int launch_fork(ForkParams fp, cudaStream_t stream);

struct FreeParams {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  const int32_t* rows;
  int n, num_rows, num_blocks, bs, max_blocks;
  int* err;
};
int launch_free(const FreeParams& fp, cudaStream_t stream);

}  // namespace mla
