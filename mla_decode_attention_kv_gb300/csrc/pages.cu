// Page operations of the paged latent cache: mla_kv_copy_pages, mla_kv_fork
// and mla_kv_free.  A pool's pages are shared by reference counts (the number
// of block-table rows that hold a page; 0: free).
//
// What bounds them: the copies move each byte once in and once out of HBM (1024
// E2M1 pages of 64 tokens in 8 layers: 50.9 us, 6.7 TB/s, 0.98 of the measured copy
// bandwidth); the bookkeeping is a few dependent reads, so for few pages the launch
// and that chain count (8 pages copied 1.6 us; 4 rows given back and forked into again
// 9.5 us, 64 rows with 4 layers' pages of 73 KB 14.5 us, in three launches).
#include "cache_kernels.cuh"
#include "common.cuh"

namespace mla {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;                                      // 16-byte loads in flight a thread
constexpr uint64_t kCopyChunk = kCopyThreads * kCopyUnroll * 16;    // bytes a block copies

// Bytes [chunk * kCopyChunk, ...) of one page, all threads of the block.
__device__ __forceinline__ void copy_chunk(const char* src, char* dst, uint64_t page_bytes, int chunk) {
  const uint64_t at = static_cast<uint64_t>(chunk) * kCopyChunk;
  const uint32_t units = static_cast<uint32_t>(min(page_bytes - at, kCopyChunk) / 16);
  const uint4* s = reinterpret_cast<const uint4*>(src + at);
  uint4* d = reinterpret_cast<uint4*>(dst + at);
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k) {
    const uint32_t u = threadIdx.x + k * kCopyThreads;
    if (u < units) v[k] = s[u];
  }
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k) {
    const uint32_t u = threadIdx.x + k * kCopyThreads;
    if (u < units) d[u] = v[k];
  }
}

}  // namespace

// ---------------------------------------------------------------- copy
__global__ void __launch_bounds__(kCopyThreads) mla_copy_pages_kernel(const CopyParams cp) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x / cp.chunks, chunk = blockIdx.x - i * cp.chunks;
  const int a = cp.src_ids[i], b = cp.dst_ids[i];
  if (a < 0 || a >= cp.src_blocks || b < 0 || b >= cp.dst_blocks) {
    if (threadIdx.x == 0) set_error(cp.err, kDevBadBlockId);
    return;
  }
  copy_chunk(cp.src + blockIdx.y * cp.src_layer + a * cp.page_bytes,
             cp.dst + blockIdx.y * cp.dst_layer + b * cp.page_bytes, cp.page_bytes, chunk);
}

int launch_copy_pages(CopyParams cp, cudaStream_t stream) {
  cp.chunks = static_cast<int>((cp.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const dim3 grid(static_cast<unsigned>(cp.n) * cp.chunks, cp.layers);
  return launch_overlapped(mla_copy_pages_kernel, grid, kCopyThreads, stream, cp) == cudaSuccess ? 0 : -1;
}

// ---------------------------------------------------------------- free
// One block per row.  The row's length is taken (swapped for 0) by its first
// thread, so a row named twice is given back once.
__global__ void __launch_bounds__(256) mla_kv_free_kernel(const FreeParams fp) {
  __shared__ int s_pages;
  griddep_wait();
  griddep_launch_dependents();
  const int r = fp.rows[blockIdx.x];
  if (r < 0 || r >= fp.num_rows) {
    if (threadIdx.x == 0) set_error(fp.err, kDevBadRow);
    return;
  }
  if (threadIdx.x == 0) {
    int L = *static_cast<volatile const int32_t*>(fp.lens + r);
    const int64_t cap = static_cast<int64_t>(fp.max_blocks) * fp.bs;
    if (L < 0 || L > cap) {   // left as it is: an emptied row would lose its pages
      set_error(fp.err, kDevBadSeqLen);
      L = 0;
    } else if (atomicCAS(fp.lens + r, L, 0) != L) {
      L = 0;
    }
    s_pages = static_cast<int>((static_cast<int64_t>(L) + fp.bs - 1) / fp.bs);
  }
  __syncthreads();
  int32_t* row = fp.table + static_cast<int64_t>(r) * fp.max_blocks;
  for (int j = threadIdx.x; j < s_pages; j += 256) {
    const int id = row[j];
    row[j] = -1;
    if (id < 0 || id >= fp.num_blocks) {
      set_error(fp.err, kDevBadBlockId);
    } else if (atomicSub(fp.refs + id, 1) <= 0) {
      atomicAdd(fp.refs + id, 1);
      set_error(fp.err, kDevBadRefCount);
    }
  }
}

int launch_free(const FreeParams& fp, cudaStream_t stream) {
  return launch_overlapped(mla_kv_free_kernel, dim3(fp.n), 256, stream, fp) == cudaSuccess ? 0 : -1;
}

// ---------------------------------------------------------------- fork
// Two launches.  The plan, one block: checks the pairs, finds as many of the
// lowest free pages as there are parents whose last page is not full, and
// hands them out in the order of the pairs; nothing is changed unless every
// pair can be served.  The application, a grid: one block per pair writes the
// child's row and counts the shared pages, the others copy the last pages.
constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 8;   // pages a thread looks at per round

// exclusive scan of v over the block, and the total
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // s_warp of the last call has been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const int t = s_warp[w];
    base += w < warp ? t : 0;
    all += t;
  }
  total = all;
  return base + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) mla_kv_fork_plan_kernel(const ForkParams fp) {
  __shared__ uint32_t s_child[kMaxForkRows / 32], s_parent[kMaxForkRows / 32];
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_bad;
  int32_t* fresh = fp.ws + 4;
  int32_t* list = fresh + fp.n;
  for (int i = threadIdx.x; i < (fp.rows + 31) / 32; i += kPlanThreads) s_child[i] = s_parent[i] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  griddep_wait();   // the grid before, a mla_kv_free for one, is done
  griddep_launch_dependents();
  __syncthreads();
  const int per = (fp.n + kPlanThreads - 1) / kPlanThreads;
  const int a = min(fp.n, static_cast<int>(threadIdx.x) * per), e = min(fp.n, a + per);
  const int64_t cap = static_cast<int64_t>(fp.max_blocks) * fp.bs;
  int need = 0;
  for (int k = a; k < e; ++k) {
    const int p = fp.parents[k], c = fp.children[k];
    if (p < 0 || p >= fp.rows || c < 0 || c >= fp.rows) {
      atomicCAS(&s_bad, 0, kDevBadRow);
      continue;
    }
    // a row is forked into once, and only when it holds nothing
    const uint32_t bit = 1u << (c & 31);
    if ((atomicOr(&s_child[c >> 5], bit) & bit) || fp.lens[c] != 0) atomicCAS(&s_bad, 0, kDevBadRow);
    atomicOr(&s_parent[p >> 5], 1u << (p & 31));
    const int L = fp.lens[p];
    if (L < 0 || L > cap) atomicCAS(&s_bad, 0, kDevBadSeqLen);
    need += L % fp.bs != 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (fp.rows + 31) / 32; i += kPlanThreads)
    if (s_child[i] & s_parent[i]) atomicCAS(&s_bad, 0, kDevBadRow);
  int total;
  const int first = block_scan(need, s_warp, total);   // (its barriers order s_bad too)
  if (s_bad) {
    if (threadIdx.x == 0) {
      set_error(fp.err, s_bad);
      fp.ws[0] = 0;
    }
    return;
  }
  int found = 0;
  for (int64_t base = 0; base < fp.num_blocks && found < total; base += kPlanThreads * kPlanPer) {
    const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * kPlanPer;
    int ref[kPlanPer], cnt = 0;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) ref[k] = 1;
    if (p0 + kPlanPer <= fp.num_blocks) {
      const int4* r4 = reinterpret_cast<const int4*>(fp.refs + p0);
      const int4 x = r4[0], y = r4[1];
      ref[0] = x.x; ref[1] = x.y; ref[2] = x.z; ref[3] = x.w;
      ref[4] = y.x; ref[5] = y.y; ref[6] = y.z; ref[7] = y.w;
    } else {
#pragma unroll
      for (int k = 0; k < kPlanPer; ++k)
        if (p0 + k < fp.num_blocks) ref[k] = fp.refs[p0 + k];
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) cnt += ref[k] <= 0;
    int all;
    int rank = found + block_scan(cnt, s_warp, all);
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k)
      if (ref[k] <= 0 && rank < total) list[rank++] = static_cast<int>(p0 + k);
    found += all;
  }
  if (found < total) {
    if (threadIdx.x == 0) {
      set_error(fp.err, kDevNoFreePage);
      fp.ws[0] = 0;
    }
    return;
  }
  __syncthreads();   // the list is complete
  int at = first;
  for (int k = a; k < e; ++k) {
    const int L = fp.lens[fp.parents[k]];
    int id = -1;
    if (L % fp.bs != 0) {
      id = list[at++];
      fp.refs[id] = 1;
    }
    fresh[k] = id;
    fp.lens[fp.children[k]] = L;   // (no child is a parent)
  }
  if (threadIdx.x == 0) fp.ws[0] = 1;
}

__global__ void __launch_bounds__(kCopyThreads) mla_kv_fork_apply_kernel(const ForkParams fp) {
  griddep_wait();   // the plan is complete
  griddep_launch_dependents();
  if (fp.ws[0] == 0) return;
  const int per = fp.layers * fp.chunks + 1;
  const int k = blockIdx.x / per, j = blockIdx.x - k * per;
  const int p = fp.parents[k], f = fp.ws[4 + k];
  const int full = fp.lens[p] / fp.bs;
  const int32_t* from = fp.table + static_cast<int64_t>(p) * fp.max_blocks;
  if (j == 0) {
    int32_t* to = fp.table + static_cast<int64_t>(fp.children[k]) * fp.max_blocks;
    for (int b = threadIdx.x; b < fp.max_blocks; b += kCopyThreads) {
      int id = -1;
      if (b < full) {
        id = from[b];
        if (id < 0 || id >= fp.num_blocks) {
          set_error(fp.err, kDevBadBlockId);
          id = -1;
        } else {
          atomicAdd(fp.refs + id, 1);
        }
      } else if (b == full) {
        id = f;
      }
      to[b] = id;
    }
    return;
  }
  if (f < 0) return;
  const int src = from[full];   // (a page that is not full lies inside the row)
  if (src < 0 || src >= fp.num_blocks) {
    if (threadIdx.x == 0) set_error(fp.err, kDevBadBlockId);
    return;
  }
  const int layer = (j - 1) / fp.chunks, chunk = (j - 1) - layer * fp.chunks;
  char* pool = fp.cache + layer * fp.layer;
  copy_chunk(pool + src * fp.page_bytes, pool + f * fp.page_bytes, fp.page_bytes, chunk);
}

int launch_fork(ForkParams fp, cudaStream_t stream) {
  fp.chunks = static_cast<int>((fp.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const unsigned blocks = static_cast<unsigned>(fp.n) * (fp.layers * fp.chunks + 1);
  if (launch_overlapped(mla_kv_fork_plan_kernel, dim3(1), kPlanThreads, stream, fp) != cudaSuccess) return -1;
  return launch_overlapped(mla_kv_fork_apply_kernel, dim3(blocks), kCopyThreads, stream, fp) == cudaSuccess ? 0 : -1;
}

}  // namespace mla
