// Partial attention per context shard over a 4-bit (E2M1) latent cache:
// mla_dcp_decode_partial_fp4.
//
// A cached value is code * s * kv_scale: a 4-bit code, an E4M3 scale s for
// every 16 values.  code * s has at most six significant bits, so it is a
// value of either 16-bit type, and the tensor cores multiply the cache as it
// is stored by the query as it is given.  The attention is that of the 16-bit
// kernel (units, shards, CURRENT part, lazily rescaled online softmax).
//
// What bounds it.  A token is 324 bytes against 1152, and its codes have to
// become 16-bit operands in shared memory before an MMA can read them, so an
// SM's shared memory (and the unpacking) is what a token costs, not HBM: 64
// tokens cost 576 cycles of it as written, 1090 as the two products read them
// (128 bytes a cycle), and with queries, weights and raw pages 2300 for 16 rows.
// So each token is unpacked once per SM and used for both products, and the
// MMAs' cost is made to follow the number of query rows:
//   S^T = K Q^T     A = K tile [64 tokens x 576] (K-major), B = Q [rows x 576]
//   O^T += V^T P^T  A = the same tile read MN-major [latent x 64 tokens],
//                   B = P^T [64 tokens x rows] (MN-major)
// The tokens and the latents fill the MMAs' M, the rows (query tokens x heads
// of one sequence, 16, 32 or 64 a unit) are N, so that few heads cost less,
// where M = heads would cost the same for any number.  O^T [512 x rows] is 4
// x rows columns of tensor memory, at most half of it, so one CTA holds all of
// a unit, and several query tokens' rows share one pass over the history.
// Measured (16 sequences of 131072 tokens): 16 heads 299 us, 2.27 TB/s of pages
// and 0.34 of the measured copy bandwidth (2700 cycles a tile of 64 tokens), 32
// heads 316, 64 heads 408, 128 heads 771 us (two units of 64 rows; the products
// alone would take 305 us at the measured bf16 rate).  The 16-bit kernel takes 780
// us for 128 heads.
//
// One persistent CTA per SM, 896 threads:
//   w0      producer: raw pages (codes, scales) by bulk copies, queries by TMA
//   w1      QK issuer            w2  PV issuer           w3  empty parts
//   w4-11   softmax: two groups of four warps with half of the rows each, 8 or
//           16 at a time; a token (16 TMEM lanes a warp in an M = 64 accumulator)
//           has two threads of a group, one for each half of the rows at hand.
//           O rescale and epilogue (thread = latent)
//   w12-27  unpacking: codes and scales to 128-byte-swizzled 16-bit chunks
// A tile's 512 latents are unpacked in parts through a ring of slots, its RoPE
// columns with the first half: the QK MMAs of a part start while the next is
// unpacked, and a slot is free when its PV MMAs are done.  Up to 32 rows: halves, a
// ring of two tiles.  64 rows, whose queries take 72 KB: quarters, a ring of one
// tile and three quarters, and one raw tile instead of two; there the way from the
// weights of a tile over the slots that they free to the scores of the next sets the
// pace, and a quarter is the shortest step on it (128 heads: halves in a ring of one
// and a half tiles 836 us, quarters 801, with the ring above 785 at that step).  With 16 rows,
// where shared memory sets it, quarters are 9 % slower.
//
// Only a tile with a weight past 2^8 of the reference (and the first of a piece) reduces the rows'
// maxima over the tokens (the lanes) and rescales O.  Row sums stay in registers,
// one partial sum per token lane and row, and are reduced once per piece.
//
// Roundings: the weights go to the query's 16-bit type for the PV product, whose two
// operands share a type and whose V is exact in it (a second term would double that
// product): o is off by half a step of sqrt(sum p^2 c^2), 0.3 to 0.9 of what rounding
// the output itself takes.  Scores, maxima, row sums (of the unrounded weights), O and
// the pieces of a cut unit are fp32; an output is rounded once.  (Pieces in fp32 and
// not in the output's type: 16 x 131072 x 16 heads 297 -> 299 us, ragged 142 -> 145, 8 x
// 32768 of two tokens 211 -> 217, with errors against 64 bits of 1.14, 1.22 and 1.08
// times those of an output rounded alone, 1.31, 1.24 and 1.14 before.)
//
// Every wait is bounded, as in the 16-bit kernel.
#include <mutex>
#include <type_traits>
#include "cache_kernels.cuh"
#include "partial_fp4.cuh"
#include "partial_sched.cuh"

namespace mla {

namespace {

constexpr int kTile4 = 64;                       // tokens
constexpr int kSoftWarp = 4;                     // first warp of the softmax
constexpr int kGroups4 = 2;                      // softmax groups of four warps
constexpr int kUnpackWarps = 16;                 // eight for each half of a tile
constexpr int kRawCodes = kTile4 * kE2m1Codes;   // 18432
constexpr int kRawStage = kTile4 * kE2m1Row;     // 20736
constexpr int kChunk = kTile4 * 128;             // 8 KB: 64 columns of a tile
constexpr int kUnits4 = 8;                       // units whose geometry is kept in shared memory
// A poll limit (mla_debug_set_spin_limit) below this one is a test of the giving up: no
// wait here lasts as long as one poll may suspend its thread, so the producer then
// copies nothing, and every wait runs out.
constexpr uint32_t kShortPolls = 64;

struct Unit4 {
  int b, g, p, lo, hi;
};

template <int N>
struct Smem4 {
  static constexpr int kParts = N == 64 ? 4 : 2;             // parts that a tile's latents are unpacked in
  static constexpr int kPart = 8 * kChunk / kParts;          // bytes of one
  static constexpr int kSlots = N == 64 ? 7 : 4;             // of them in the ring
  static constexpr int kNRaw = N == 64 ? 1 : 2;              // raw tiles
  static constexpr int kNR = N == 64 ? 1 : 2;    // RoPE slots
  static constexpr int kRows = N == 16 ? 8 : 16;               // rows (columns of S^T) that a group takes at a time
  static constexpr int kPasses = N / (kGroups4 * kRows);
  static constexpr int kUnpackWarp = kSoftWarp + 4 * kGroups4;
  static constexpr int kThreads = (kUnpackWarp + kUnpackWarps) * 32;
  static constexpr int kQ = N * 128 * 9;
  static constexpr int kLatOff = 0;
  static constexpr int kRopeOff = kLatOff + kSlots * kPart;
  static constexpr int kQOff = kRopeOff + kNR * kChunk;
  static constexpr int kPOff = kQOff + kQ;
  static constexpr int kP = kTile4 * N * 2;
  static constexpr int kStageOff = kPOff + kP;               // 16 rows: the epilogue's staging
  static constexpr int kRawOff = kStageOff + (N == 16 ? 8192 : 0);
  static constexpr int kMOff = kRawOff + kNRaw * kRawStage;  // reference maxima [N]
  static constexpr int kRedOff = kMOff + N * 4;              // reductions over the warps, [4][rows] for each pass:
                                                             // maxima, then sums
  static constexpr int kFlagOff = kRedOff + 2 * N * 16;      // [3 tiles][2 groups]: weights past the limit
  static constexpr int kUnitOff = kFlagOff + 32;
  static constexpr int kBarOff = kUnitOff + ((kUnits4 * 20 + 8 + 15) / 16) * 16;
  // barrier slots
  enum : int {
    B_RAW_FULL = 0,
    B_RAW_EMPTY = kNRaw,
    B_FULL = 2 * kNRaw,
    B_EMPTY = B_FULL + kSlots,
    B_Q_FULL = B_EMPTY + kSlots,
    B_Q_EMPTY,
    B_S_FULL,
    B_S_EMPTY = B_S_FULL + 2,
    B_P_FULL = B_S_EMPTY + 2,
    B_P_EMPTY,
    B_P_FIXED,
    B_ROPE_EMPTY,
    B_DONE_QK,
    B_DONE_PV,
    B_COUNT
  };
  static constexpr int kTotal = kBarOff + (B_COUNT + 2) * 8;   // (from a 1024-aligned base)
  static constexpr int kTmemO = 0;
  static constexpr int kTmemS = 4 * N;
  static constexpr int kTmemCols = N == 64 ? 512 : N == 32 ? 256 : 128;   // 6 N, a power of two
};
static_assert(Smem4<64>::kTotal <= 232448 && Smem4<32>::kTotal <= 232448, "shared memory budget");

// ---------------------------------------------------------------- units
// u = (g * B + b) * P + p: the row groups outermost, so that the CTAs of
// several groups stream the same histories at the same time (as the query
// tokens of the 16-bit kernel).
template <int N>
__device__ __noinline__ Unit4 unit4(const Fp4Params& fp, int u) {
  Unit4 ui;
  ui.p = u % fp.P;
  const int gb = u / fp.P;
  ui.b = gb % fp.B;
  ui.g = gb / fp.B;
  if (ui.p == fp.S) {
    // CURRENT: the tokens that the group's last row sees (one tile)
    ui.lo = 0;
    ui.hi = (min(fp.R, (ui.g + 1) * N) - 1) / fp.H + 1;
  } else {
    int L = fp.seq_lens[ui.b];
    const int cap = fp.max_blocks * fp.bs;
    if (L < 0 || L > cap) {
      set_error(fp.err, kDevBadSeqLen);
      L = max(0, min(L, cap));
    }
    const int chunk = fp.S * fp.bs;
    const int len = L > 0 ? fp.bs * ((L + chunk - 1) / chunk) : 0;
    ui.lo = min(L, ui.p * len);
    ui.hi = min(L, (ui.p + 1) * len);
  }
  return ui;
}

__device__ __forceinline__ int tiles4(const Unit4& ui) { return (ui.hi - ui.lo + kTile4 - 1) / kTile4; }

struct UnitTable {
  int first, n;
  Unit4 u[kUnits4];
};

template <int N>
__device__ __noinline__ Unit4 unit4_get(const Fp4Params& fp, const UnitTable* tab, int u) {
  const unsigned k = static_cast<unsigned>(u - tab->first);
  if (k < static_cast<unsigned>(tab->n)) return tab->u[k];
  return unit4<N>(fp, u);
}

struct Range4 {
  int u_begin, j_begin, u_last, j_stop;
};

// The tiles of a CTA's range as one stream; a piece is the part of one unit in it.
template <int N>
struct Iter4 {
  int u, j, jfirst, jend, u_last, j_stop, key, nq;
  bool valid, newq;
  Unit4 ui;
  const UnitTable* tab;
  __device__ __forceinline__ void start(const Fp4Params& fp, const UnitTable* t, const Range4& r) {
    tab = t;
    u_last = r.u_last;
    j_stop = r.j_stop;
    key = nq = -1;
    valid = r.u_begin <= r.u_last;
    if (!valid) return;
    u = r.u_begin;
    ui = unit4_get<N>(fp, tab, u);
    enter(fp, r.j_begin);
  }
  __device__ __forceinline__ void enter(const Fp4Params& fp, int j0) {
    j = jfirst = j0;
    jend = u == u_last ? j_stop : tiles4(ui);
    const int k = ui.g * fp.B + ui.b;
    newq = k != key;
    if (newq) {
      ++nq;
      key = k;
    }
  }
  __device__ __forceinline__ void advance(const Fp4Params& fp) {
    if (++j < jend) return;
    while (u < u_last) {
      ++u;
      ui = unit4_get<N>(fp, tab, u);
      if (ui.hi > ui.lo) {
        enter(fp, 0);
        return;
      }
    }
    valid = false;
  }
  __device__ __forceinline__ void next_piece(const Fp4Params& fp) {
    j = jend - 1;
    advance(fp);
  }
  __device__ __forceinline__ bool first() const { return j == jfirst; }
  __device__ __forceinline__ bool last() const { return j == jend - 1; }
  __device__ __forceinline__ bool whole() const { return jfirst == 0 && jend == tiles4(ui); }
  __device__ __forceinline__ int tok0() const { return ui.lo + j * kTile4; }
};

// ---------------------------------------------------------------- partition
// Equal shares of cost, as partition_tiles of the 16-bit kernel: a tile costs
// kCostTile, a unit kCostUnit besides (its first tile's latency, the epilogue).
// With a workspace the shares are exact (units are cut where whole ones would
// leave the busiest CTA more than kCut4 tiles above the even share), without one a
// CTA takes the whole units whose first tile lies in its share.
// Measured over a ragged batch (64 sequences of 512 to 65536 tokens in 16
// shards) with a unit at 1, 2, 3 and 4 tiles: 16 heads 162, 146, 152 and 158 us,
// 128 heads (units of 64 rows) at 2, 3 and 4: 413, 394 and 410 us.
constexpr int kCostTile = 1;
template <int N>
constexpr int kCostUnit = N == 64 ? 3 : 2;
// What a cut costs in tiles, its pieces' ends and the merge among it.  Measured both
// ways for 96 to 101 calls a size (160 to 760 units of 6 to 32 equal tiles), by how far
// whole units leave the busiest CTA above the even share, whole minus cut: 16 rows -0.4
// us at 6, +0.5 at 7, +1.8 at 8; 32 rows -0.8, +0.2, +1.7; 64 rows and 128 heads -3.8 at
// 7, -1.3 at 8, -0.5 at 9, +0.8 at 10, spread over 2 us either way.  With these limits the
// mean loss against the better of the two is 0.01, 0.01 and 0.1 %, the worst 3 %.
template <int N>
constexpr int kCut4 = N == 64 ? 8 : 6;

struct PartScratch {
  int2 scan[32];
  int4 pre[1024];                  // of each thread's units: tiles and cost before, tiles of the first
  int bound[kFp4MaxCtas + 1];      // first tile of each CTA's share
  int whole[kFp4MaxCtas + 1];      // cost before the first unit that starts at or behind it
  int4 at[kFp4MaxCtas + 1];        // where that is: a unit, its tiles, the tiles before it, those of it before the boundary
  Range4 rng;
};

template <int N, int NT>
__device__ __forceinline__ Range4 partition4(const Fp4Params& fp, PartScratch* ps, UnitTable* tab, int cid, int ncta) {
  constexpr int kWarps = NT / 32;
  static_assert(NT <= 1024 && NT > kFp4MaxCtas, "block size");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int U = fp.num_units;
  const int per = (U + NT - 1) / NT;
  auto cost_of = [](int nt) { return nt > 0 ? kCostTile * nt + kCostUnit<N> : 0; };
  Unit4 mine = {0, 0, 0, 0, 0};      // the thread's first unit
  int cnt = 0, cost = 0, ntiles = 0;
  {
    const int a = min(U, tid * per), e = min(U, a + per);
    for (int u = a; u < e; ++u) {
      const Unit4 ui = unit4<N>(fp, u);
      const int nt = tiles4(ui);
      if (u == a) {
        mine = ui;
        ntiles = nt;
      }
      cnt += nt;
      cost += cost_of(nt);
    }
  }
  int incl_t = cnt, incl_c = cost;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl_t, o), z = __shfl_up_sync(0xffffffffu, incl_c, o);
    if (lane >= o) {
      incl_t += y;
      incl_c += z;
    }
  }
  if (lane == 31) ps->scan[warp] = make_int2(incl_t, incl_c);
  if (tid == 0) ps->rng = {0, 0, -1, 0};
  __syncthreads();
  // (the warps' sums by reductions: as a loop in every warp 1 us of a call)
  const int2 sums = lane < kWarps ? ps->scan[lane] : make_int2(0, 0);
  const int total = __reduce_add_sync(0xffffffffu, sums.x), all_cost = __reduce_add_sync(0xffffffffu, sums.y);
  ps->pre[tid] = make_int4(__reduce_add_sync(0xffffffffu, lane < warp ? sums.x : 0) + incl_t - cnt,
                           __reduce_add_sync(0xffffffffu, lane < warp ? sums.y : 0) + incl_c - cost, ntiles, 0);
  if (total == 0) {
    if (fp.split && tid == 0) {
      fp.ws_units[cid] = make_int4(-1, 0, 0, 0);
      fp.ws_bounds[cid] = 0;
      if (cid == 0) fp.ws_bounds[ncta] = 0;
    }
    if (tid == 0) tab->first = tab->n = 0;
    return {0, 0, -1, 0};
  }
  __syncthreads();
  // boundary c: the tiles that start below the cost c * all_cost / ncta
  if (tid <= ncta) {
    const int share = all_cost / ncta, rest = all_cost - share * ncta;
    const int tc = tid == ncta ? all_cost - 1 : tid * share + tid * rest / ncta;
    // the unit that holds it: the thread with its tiles by bisection, then a walk along the thread's units
    int lo = 0, hi = min(U, NT) - 1;   // the last thread with a cost before it of at most tc
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (ps->pre[mid].y <= tc) lo = mid;
      else hi = mid - 1;
    }
    const int4 p = ps->pre[lo];
    int u = lo * per, nt = p.z, t0 = p.x, c0 = p.y;
    while (tc >= c0 + cost_of(nt)) {
      t0 += nt;
      c0 += cost_of(nt);
      nt = tiles4(unit4<N>(fp, ++u));
    }
    const int into = tc - c0 - kCostUnit<N>;
    int j = tid == 0 || into <= 0 ? 0 : min(nt, (into + kCostTile - 1) / kCostTile);
    if (tid == ncta) j = nt;
    ps->bound[tid] = t0 + j;
    ps->whole[tid] = j == 0 ? c0 : c0 + cost_of(nt);
    ps->at[tid] = make_int4(u, nt, t0, j);
  }
  __syncthreads();
  bool split = false;
  if (fp.split) {
    const int even = (all_cost + ncta - 1) / ncta;
    const bool over = tid < ncta && ps->whole[tid + 1] - ps->whole[tid] > even + kCut4<N> * kCostTile;
    split = __syncthreads_or(over) != 0;
  }
  const int lo = ps->bound[cid], hi = ps->bound[cid + 1];
  if (tid == 0) {
    // the share's first unit and tile: the boundary's, or the next unit with tiles
    if (lo < hi) {
      const int4 f = ps->at[cid];
      int u = f.x, j = f.w;
      if (split ? j >= f.y : j > 0) {
        j = 0;
        do ++u;
        while (u < U && tiles4(unit4<N>(fp, u)) == 0);
      }
      ps->rng.u_begin = u;
      ps->rng.j_begin = j;
    }
  } else if (tid == 32) {
    // the last unit, and how many of its tiles: those before the next boundary
    if (lo < hi) {
      const int4 f = ps->at[cid + 1];
      int u = f.x, nt = f.y, j = f.w;
      if (j == 0) {
        do nt = tiles4(unit4<N>(fp, --u));
        while (nt == 0);
        j = nt;
      }
      ps->rng.u_last = u;
      ps->rng.j_stop = split ? j : nt;
    }
  } else if (tid == 64 && fp.split) {
    // the record of a unit cut before this share that ends inside it
    const int4 f = ps->at[cid];
    int4 rec = make_int4(-1, 0, 0, 0);
    if (split && lo < hi && f.w > 0 && f.w < f.y && f.z + f.y <= hi) {
      // the CTA with its first tile: the last whose boundary lies at most a unit's
      // fixed cost behind the cost before it
      const int64_t x = ps->whole[cid] - cost_of(f.y) + kCostUnit<N>;
      rec = make_int4(f.x, f.z, static_cast<int>(((x + 1) * ncta + all_cost - 1) / all_cost) - 1, cid);
    }
    fp.ws_units[cid] = rec;
    fp.ws_bounds[cid] = lo;
    if (cid == 0) fp.ws_bounds[ncta] = total;
  }
  __syncthreads();
  const Range4 r = ps->rng;
  // the geometry of the first units (mostly threads' own)
  const int n = r.u_begin <= r.u_last ? min(r.u_last - r.u_begin + 1, kUnits4) : 0;
  if (per == 1) {
    if (static_cast<unsigned>(tid - r.u_begin) < static_cast<unsigned>(n)) tab->u[tid - r.u_begin] = mine;
  } else if (tid < n) {
    tab->u[tid] = unit4<N>(fp, r.u_begin + tid);
  }
  if (tid == 0) {
    tab->first = r.u_begin;
    tab->n = n;
  }
  return r;
}

// A CTA for every unit (no unit cut, no more units than CTAs): nothing to share out.
// (256 tokens, 16 heads: 10.7 us with the partition, 8.3 so.  As a branch of the one
// kernel it cost the 64-row kernel registers, 2 % of the time of long calls.)
template <int N>
__device__ __forceinline__ Range4 single4(const Fp4Params& fp, UnitTable* tab, int cid) {
  const Unit4 ui = unit4<N>(fp, cid);
  const int nt = tiles4(ui);
  if (threadIdx.x == 0) {
    tab->first = cid;
    tab->n = 1;
    tab->u[0] = ui;
  }
  return nt > 0 ? Range4{cid, 0, cid, nt} : Range4{0, 0, -1, 0};
}

// r / d for 0 <= r < 2^13, d <= 128, with inv = 2^32 / d rounded up (0 for d = 1):
// the product is off by less than 2^-19, and r / d at least 2^-7 below the next integer
__device__ __forceinline__ int quotient(int r, uint32_t inv) { return inv ? static_cast<int>(__umulhi(r, inv)) : r; }

// Row of o_part / lse_part of query row r (of R) of sequence b in part p.
__device__ __forceinline__ int64_t out_row4(const Fp4Params& fp, int b, int r, int p) {
  const int hs = fp.hs, i = quotient(r, fp.inv_H), h = r - i * fp.H, s = quotient(h, fp.inv_hs);
  return ((static_cast<int64_t>(s) * fp.T + static_cast<int64_t>(b) * fp.q_len + i) * fp.P + p) * hs + (h - s * hs);
}

// ---------------------------------------------------------------- pieces of PTX
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Columns [c, c + NC) of an M = 64 accumulator for lanes 0-15 of the warp and
// [c + NC, c + 2 NC) for lanes 16-31, both of the rows in TMEM lanes 0-15.
__device__ __forceinline__ void tmem_half_issue(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0,%1,%2,%3}, [%4], 4;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void tmem_half_issue(uint32_t a, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(a));
}

template <int K>
__device__ __forceinline__ void tmem_half(uint32_t a, uint32_t (&r)[K]) {
  tmem_half_issue(a, r);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) asm volatile("" : "+r"(r[k])::"memory");
}

// Eight columns of this warp's 32 lanes, loaded and waited for
__device__ __forceinline__ void tmem_get(uint32_t a, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_put(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 8 X columns of 16 lanes (issued; tmem_wait_frag waits): thread t has, of each
// 8 columns, columns 2 (t % 4) and + 1 of lanes t / 4 (r[0], r[1]) and t / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
template <int K>
__device__ __forceinline__ void tmem_wait_frag(uint32_t (&r)[K], uint32_t (&q)[K]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) asm volatile("" : "+r"(r[k]), "+r"(q[k])::"memory");   // (no use before the wait)
}

// Four 8 x 8 matrices of 16-bit values stored transposed: lane 8 i + k gives the
// address of row k of matrix i.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// P^T, the MN-major B operand: each 16 columns are a block of their own, [64
// tokens][16] 16-bit values with the 32-byte swizzle, LBO from block to block.
constexpr int kPRow = 16 * 2;
constexpr int kPBlock = kTile4 * kPRow;
constexpr int kPStep = 16 * kPRow;       // bytes from one k-step (16 tokens) to the next
__device__ __forceinline__ uint64_t p_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(kPBlock >> 4) << 16) |
         (static_cast<uint64_t>(8 * kPRow >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{6} << 61);
}
// byte offset of 16-byte unit k (0, 1) of token t in a block
__device__ __forceinline__ uint32_t p_offset(int t, int k) { return t * kPRow + ((k ^ ((t >> 2) & 1)) << 4); }

// Reduction over the 16 lanes of a half warp of NC columns held one row per
// lane: every step halves the columns a lane keeps, so 16 columns take 15
// shuffles.  Lane l ends with column (l & 15) / (16 / NC).
template <int NC, bool MAX>
__device__ __forceinline__ float col_reduce(float (&v)[NC], int lane) {
  auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
  int n = NC;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int k = 0; k < NC / 2; ++k) {
        if (k < n) {
          const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
          v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

// ---------------------------------------------------------------- unpacking
// Eight codes (a word of the page) times their block's scale -> four 16-bit
// pairs.  One conversion makes an fp16 pair of a byte's two codes; the product
// with the scale, an fp16 number too, is exact in fp16 (2^-10 to 2688, six
// significant bits) and, through fp32, in bf16.
template <bool BF16>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t mul, uint32_t (&out)[4]) {
  uint32_t h[4];
  // (as one block: the conversions then read the word's bytes in place; through
  // cuda_fp4.h's byte arguments the same work takes three times the time)
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16) {
      float lo, hi;
      asm("{\n .reg .b16 a, b, c, d;\n mov.b32 {a, b}, %2;\n mov.b32 {c, d}, %3;\n"
          " fma.rn.f32.f16 %0, a, c, 0f00000000;\n fma.rn.f32.f16 %1, b, d, 0f00000000;\n}\n"
          : "=f"(lo), "=f"(hi)
          : "r"(h[j]), "r"(mul));
      out[j] = pack2<true>(lo, hi);
    } else {
      const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h[j]), *reinterpret_cast<const __half2*>(&mul));
      out[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// fp16 pairs (s, s) of two block scales (E4M3 bytes); 0 for a token past the
// end, whatever its bytes.
__device__ __forceinline__ void multipliers(uint32_t s2, bool valid, uint32_t& m0, uint32_t& m1) {
  uint32_t x;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(x) : "r"(s2));
  x = valid ? x : 0u;
  m0 = __byte_perm(x, 0, 0x1010);
  m1 = __byte_perm(x, 0, 0x3232);
}

// Not 0 where one of eight 16-bit values is a NaN or an infinity (exponent bits
// all ones: adding the lowest of them carries into the sign's place).
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(const uint4& v) {
  constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
  return (((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne)) & 0x80008000u;
}

// Whether latents of a CURRENT token are not finite: this thread's 64 of half h
// and, with h = 0, the same of the other half; `row` is at the thread's place in
// the first half.  h < 0: no token.  (Out of line: inlined, its registers cost
// the history's tiles 4 to 7 % more time.)
template <bool BF16>
__device__ __noinline__ bool current_bad(const uint4* row, int h) {
  uint32_t bad = 0;
  if (h >= 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= not_finite<BF16>(row[32 + j]);
    if (h == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) bad |= not_finite<BF16>(row[j]);
    }
  }
  return bad != 0;
}

}  // namespace

// ---------------------------------------------------------------- the kernel
template <bool BF16, int N, bool SHARES>
__global__ void __launch_bounds__(Smem4<N>::kThreads, 1)
    mla_partial_fp4_kernel(const __grid_constant__ CUtensorMap tm_qlat, const __grid_constant__ CUtensorMap tm_qpe,
                           const Fp4Params fp) {
  using L = Smem4<N>;
  // Weights are taken relative to a row's reference maximum and, for fp16, whose least
  // normal value is 2^-14, times 2^7: a weight down to 2^-21 of the maximum's keeps its
  // eleven bits and one down to 2^-32 some, where a long history has many of those.
  constexpr float kLift = BF16 ? 0.f : 7.f;
  constexpr float kThresh = 8.f + kLift;       // lazy rescale: weights stay below 2^8 (2^15 as lifted)

  // (the kernel has no static shared memory, so the block starts where the
  // alignment puts it; the 128-byte swizzle needs 1024)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + L::B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + L::B_COUNT + 1);
  UnitTable* tab = reinterpret_cast<UnitTable*>(smem + L::kUnitOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cid = blockIdx.x, ncta = gridDim.x;
  int* err = fp.err;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kNRaw; ++s) {
      mbar_init(&bar[L::B_RAW_FULL + s], 1);
      mbar_init(&bar[L::B_RAW_EMPTY + s], kUnpackWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[L::B_S_FULL + s], 1);
      mbar_init(&bar[L::B_S_EMPTY + s], 4 * kGroups4);
    }
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&bar[L::B_FULL + s], kUnpackWarps / L::kParts);
      mbar_init(&bar[L::B_EMPTY + s], 1);
    }
    mbar_init(&bar[L::B_Q_FULL], 1);
    mbar_init(&bar[L::B_Q_EMPTY], 1);
    mbar_init(&bar[L::B_P_FULL], 4 * kGroups4);
    mbar_init(&bar[L::B_P_EMPTY], 1);
    mbar_init(&bar[L::B_P_FIXED], 4 * kGroups4);
    mbar_init(&bar[L::B_ROPE_EMPTY], 1);
    for (int k = 0; k < 6; ++k) reinterpret_cast<int*>(smem + L::kFlagOff)[k] = 0;
    mbar_init(&bar[L::B_DONE_QK], 1);
    mbar_init(&bar[L::B_DONE_PV], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_qlat);
    prefetch_tmap(&tm_qpe);
  }
  // (programmatic launches: this grid's start overlaps the one before, the
  // next grid's start this one; each waits for the other to be done, and lets the
  // next go only then: the V-up reads W_UV before its own wait)
  griddep_wait();
  griddep_launch_dependents();
  Range4 rng;
  if constexpr (SHARES) rng = partition4<N, L::kThreads>(fp, reinterpret_cast<PartScratch*>(smem), tab, cid, ncta);
  else rng = single4<N>(fp, tab, cid);
  tc_fence_before();
  __syncthreads();   // barriers, TMEM address, table; the scratch is free
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Waits waits{fp.spin_limit, abort_flag, err};

  if (warp == 0) {
    // ------------------------------------------------ producer
    Iter4<N> it;
    it.start(fp, tab, rng);
    if (fp.spin_limit < kShortPolls) it.valid = false;
    const int nbox = kTile4 / fp.box;
    int rs = 0, qloads = 0;
    // (the id of a lane's page is loaded one tile ahead)
    auto fetch = [&](const Iter4<N>& t) {
      if (!t.valid || t.ui.p == fp.S || lane >= nbox) return 0;
      const int tk = min(t.tok0() + lane * fp.box, t.ui.hi - 1);
      return fp.block_table[static_cast<int64_t>(t.ui.b) * fp.max_blocks + (tk >> fp.bs_shift)];
    };
    int id_cur = fetch(it);
    while (it.valid) {
      Iter4<N> nx = it;
      nx.advance(fp);
      const int id_next = fetch(nx);
      if (it.ui.p != fp.S) {
        const int st = rs % L::kNRaw;
        if (rs >= L::kNRaw && !__all_sync(0xffffffffu, waits.wait(&bar[L::B_RAW_EMPTY + st], (rs / L::kNRaw - 1) & 1)))
          break;
        uint8_t* raw = smem + L::kRawOff + st * kRawStage;
        if (lane == 0) mbar_arrive_expect_tx(&bar[L::B_RAW_FULL + st], kRawStage);
        __syncwarp();
        if (lane < nbox) {
          int tk = it.tok0() + lane * fp.box;
          const bool past = tk >= it.ui.hi;   // a box past the end reads the last one again (masked)
          if (past) tk = it.ui.hi - 1;
          int id = id_cur;
          if (id < 0 || id >= fp.num_blocks) {
            set_error(err, kDevBadBlockId);
            id = 0;
          }
          int off = tk & (fp.bs - 1);
          if (past) off &= ~(fp.box - 1);
          const uint8_t* page = fp.kv_cache + (static_cast<int64_t>(id) << fp.bs_shift) * kE2m1Row;
          bulk_load(raw + lane * fp.box * kE2m1Codes, page + off * kE2m1Codes, fp.box * kE2m1Codes,
                    &bar[L::B_RAW_FULL + st]);
          bulk_load(raw + kRawCodes + lane * fp.box * kE2m1Scales,
                    page + fp.bs * kE2m1Codes + off * kE2m1Scales, fp.box * kE2m1Scales, &bar[L::B_RAW_FULL + st]);
        }
        ++rs;
      }
      if (it.first() && it.newq) {
        if (it.nq >= 1 && !__all_sync(0xffffffffu, waits.wait(&bar[L::B_Q_EMPTY], (it.nq - 1) & 1))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar[L::B_Q_FULL], L::kQ);
        __syncwarp();
        const int qrow = it.ui.b * fp.R + it.ui.g * N;
        if (lane < 9)
          tma_load_2d(smem + L::kQOff + lane * (N * 128), lane < 8 ? &tm_qlat : &tm_qpe, &bar[L::B_Q_FULL],
                      lane < 8 ? lane * 64 : 0, qrow);
        ++qloads;
      }
      id_cur = id_next;
      it = nx;
    }
    if (lane == 0) {   // what was issued has landed before the CTA ends
      for (int s = 0; s < L::kNRaw && s < rs; ++s) {
        const int last = rs - 1 - (rs - 1 - s) % L::kNRaw;
        mbar_wait(&bar[L::B_RAW_FULL + s], (last / L::kNRaw) & 1, err);
      }
      if (qloads > 0) mbar_wait(&bar[L::B_Q_FULL], (qloads - 1) & 1, err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ QK issuer: S^T = K Q^T
    // The warp runs converged and one elected lane issues: the descriptors
    // then live in uniform registers.  (Issued from a branch of one lane, an
    // MMA of 16 rows cost 45 cycles of issue, against 25 of execution.)  What
    // changes at a unit's end is worked out once per piece, not per tile.
    const bool leader = elect_one();
    constexpr uint32_t idesc = make_idesc_f16(64, N, BF16, false, false);
    const uint64_t a0 = make_desc_sw128(smem_u32(smem + L::kLatOff), 16, 1024);
    const uint64_t r0 = make_desc_sw128(smem_u32(smem + L::kRopeOff), 16, 1024);
    const uint64_t q0 = make_desc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
    auto wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, waits.wait(b, parity)) != 0; };
    Iter4<N> it;
    it.start(fp, tab, rng);
    int g = 0;
    bool ok = true;
    while (ok && it.valid) {
      const int n = it.jend - it.j;
      if (it.newq && !wait(&bar[L::B_Q_FULL], it.nq & 1)) break;
      it.next_piece(fp);
      const bool lastq = !it.valid || it.newq;
      for (int k = 0; k < n; ++k, ++g) {
        const int sb = g & 1;
        if (g >= 2 && !wait(&bar[L::B_S_EMPTY + sb], ((g >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + L::kTmemS + sb * N;
#pragma unroll
        for (int h = 0; h < L::kParts; ++h) {
          const int hc = L::kParts * g + h, sl = hc % L::kSlots;
          if (!wait(&bar[L::B_FULL + sl], (hc / L::kSlots) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          constexpr int kOps = 32 / L::kParts;
          const uint64_t a = a0 + sl * (L::kPart >> 4);
#pragma unroll
          for (int kk = 0; kk < kOps; ++kk)
            if (leader)
              umma_ss(d, a + (kk >> 2) * (kChunk >> 4) + (kk & 3) * 2,
                      q0 + ((kOps / 4) * h + (kk >> 2)) * (N * 8) + (kk & 3) * 2, idesc, h || kk ? 1u : 0u);
          if (h == L::kParts / 2 - 1) {   // the RoPE columns come with the first half
            const uint64_t r = r0 + (g % L::kNR) * (kChunk >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (leader) umma_ss(d, r + kk * 2, q0 + 8 * (N * 8) + kk * 2, idesc, 1u);
            if (L::kNR == 1 && leader) umma_commit(&bar[L::B_ROPE_EMPTY]);
          }
        }
        if (!ok) break;
        if (leader) {
          umma_commit(&bar[L::B_S_FULL + sb]);
          if (lastq && k == n - 1) umma_commit(&bar[L::B_Q_EMPTY]);
        }
      }
    }
    if (leader) umma_commit(&bar[L::B_DONE_QK]);
    __syncwarp();
    mbar_wait(&bar[L::B_DONE_QK], 0, err);
  } else if (warp == 2) {
    // ------------------------------------------------ PV issuer: O^T += V^T P^T
    const bool leader = elect_one();
    constexpr uint32_t idesc = make_idesc_f16(128, N, BF16, true, true);
    const uint64_t v0 = make_desc_sw128(smem_u32(smem + L::kLatOff), kChunk, 1024);
    const uint64_t p0 = p_desc(smem_u32(smem + L::kPOff));
    auto wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, waits.wait(b, parity)) != 0; };
    Iter4<N> it;
    it.start(fp, tab, rng);
    int g = 0, nfix = 0;
    bool ok = true;
    while (ok && it.valid) {
      const int n = it.jend - it.j;
      for (int k = 0; k < n; ++k, ++g) {
        if (!wait(&bar[L::B_P_FULL], g & 1)) {
          ok = false;
          break;
        }
        // weights past the limit are made again first (the softmax, below)
        const volatile int* fl = reinterpret_cast<const volatile int*>(smem + L::kFlagOff) + (g % 3) * 2;
        if (fl[0] | fl[1]) {
          if (!wait(&bar[L::B_P_FIXED], nfix & 1)) {
            ok = false;
            break;
          }
          ++nfix;
        }
        tc_fence_after();
        const uint32_t more = k > 0 ? 1u : 0u;
#pragma unroll
        for (int h = 0; h < L::kParts; ++h) {
          const int sl = (L::kParts * g + h) % L::kSlots;
          const uint64_t v = v0 + sl * (L::kPart >> 4);
          constexpr int kBlocks = 4 / L::kParts;
#pragma unroll
          for (int p = 0; p < kBlocks; ++p) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (leader)
                umma_ss(tmem + L::kTmemO + (kBlocks * h + p) * N, v + p * (2 * kChunk >> 4) + kk * 128,
                        p0 + kk * (kPStep >> 4), idesc, kk ? 1u : more);
          }
          if (leader) umma_commit(&bar[L::B_EMPTY + sl]);
        }
        if (leader) umma_commit(&bar[L::B_P_EMPTY]);
      }
      it.next_piece(fp);
    }
    if (leader) umma_commit(&bar[L::B_DONE_PV]);
    __syncwarp();
    mbar_wait(&bar[L::B_DONE_PV], 0, err);
  } else if (warp == 3) {
    // ------------------------------------------------ parts without tokens: o = 0, lse = -inf
    for (int u = cid; u < fp.num_units; u += ncta) {
      const Unit4 ui = unit4<N>(fp, u);
      if (ui.hi > ui.lo) continue;
      const int r1 = min(fp.R, (ui.g + 1) * N);
      for (int r = ui.g * N; r < r1; ++r) {
        const int64_t row = out_row4(fp, ui.b, r, ui.p);
        if (lane == 0) fp.lse_part[row] = -INFINITY;
        uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(fp.o_part) + row * (fp.part_dtype == kFP32 ? 2048 : 1024));
        for (int c = lane; c < (fp.part_dtype == kFP32 ? 128 : 64); c += 32) o[c] = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (warp < L::kUnpackWarp) {
    // ------------------------------------------------ softmax, O rescale, epilogue
    // Two groups of four warps with half of the rows (columns of S^T) each and
    // nothing shared between them; a group takes its rows 8 or 16 at a time, and
    // a token has two threads of a group, one for each half of those.
    constexpr int NG = L::kRows, NC = NG / 2, PASSES = L::kPasses;
    constexpr int NO = 8;                      // columns of O at a time
    const int grp = (warp - kSoftWarp) >> 2, wq = warp & 3;
    const int barid = 1 + grp;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const int tok = wq * 16 + (lane & 15);     // token of the tile
    const int cg = (lane >> 4) * NC;           // first column of this thread in a pass
    const int cr = cg + (lane & 15) / (16 / NC);   // column that col_reduce leaves here
    auto col0 = [&](int q) { return (grp * PASSES + q) * NG; };   // first column of pass q
    auto red_of = [&](int q) { return reinterpret_cast<float*>(smem + L::kRedOff) + (grp * PASSES + q) * (4 * NG); };   // [4][NG]
    volatile int* flags = reinterpret_cast<volatile int*>(smem + L::kFlagOff);
    float l[PASSES][NC];
    // Reference maxima of pass q (less the lift), in shared memory; the 64-row kernel, which would
    // spill them, reads them there, the others keep a copy in registers (64 rows, 32 x
    // 4096 tokens x 128 heads: 93 us with registers, 86 without; 16 rows, 16 x 131072
    // tokens: 306 and 312).
    constexpr bool kKeepM = PASSES == 1;
    alignas(16) float m[NC];
    auto m_of = [&](int q) { return reinterpret_cast<float*>(smem + L::kMOff) + col0(q) + cg; };
    Iter4<N> it;
    it.start(fp, tab, rng);
    int g = 0;
    bool ok = true;
    // where this token's weights go in P^T, and a warp's staging of the epilogue: its quarter of the pass's block of P, which no MMA
    // reads then (16 rows: both groups are in one block, so a region of its own)
    auto put = [&](int q, const uint32_t (&w)[NC / 2]) {
      uint8_t* block = smem + L::kPOff + (N == 16 ? 0 : (grp * PASSES + q) * kPBlock);
      if constexpr (NC == 4)
        *reinterpret_cast<uint2*>(block + p_offset(tok, grp) + (lane >> 4) * 8) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint4*>(block + p_offset(tok, lane >> 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto stage_of = [&](int i) {
      return N == 16 ? smem + L::kStageOff + (warp - kSoftWarp) * 1024 + i * 512
                     : smem + L::kPOff + (grp * PASSES + i) * kPBlock + wq * (kPBlock / 4);
    };
    // the tile's scores of pass q in the log2 domain, relative to mq, columns
    // below nmin masked (`all`: there are none)
    auto rel = [&](int q, float sl, bool all, int nmin, const uint32_t (&v)[NC], float (&x)[NC]) {
      if constexpr (!kKeepM) {
#pragma unroll
        for (int k = 0; k < NC; k += 4) *reinterpret_cast<float4*>(m + k) = *reinterpret_cast<const float4*>(m_of(q) + k);
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) x[k] = fmaf(__uint_as_float(v[k]), sl, -m[k]);
      if (!all) {
#pragma unroll
        for (int k = 0; k < NC; ++k) x[k] = col0(q) + cg + k >= nmin ? x[k] : -INFINITY;
      }
    };
    auto scores = [&](int q, float sl, bool all, int nmin, bool first, float (&x)[NC]) {
      uint32_t v[NC];
      tmem_half(tmem + lanes + L::kTmemS + (g & 1) * N + col0(q), v);
      if (first) {
#pragma unroll
        for (int k = 0; k < NC; ++k) x[k] = __uint_as_float(v[k]) * sl;
      } else {
        if constexpr (!kKeepM) {
#pragma unroll
          for (int k = 0; k < NC; k += 4) *reinterpret_cast<float4*>(m + k) = *reinterpret_cast<const float4*>(m_of(q) + k);
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) x[k] = fmaf(__uint_as_float(v[k]), sl, -m[k]);
      }
      if (!all) {
#pragma unroll
        for (int k = 0; k < NC; ++k) x[k] = col0(q) + cg + k >= nmin ? x[k] : -INFINITY;
      }
    };
    // New reference maxima of a pass's rows from the tile's scores x, with O and l
    // brought to them (the maxima of a piece's first tile are taken below).
    auto new_maxima = [&](int q, const float (&x)[NC], float (&lq)[NC]) {
      float* red = red_of(q);
      float y[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) y[k] = x[k];
      const float mx = col_reduce<NC, true>(y, lane);
      red[wq * NG + cr] = mx;
      named_bar_sync(barid, 128);
      float a[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const float* r = red + cg + k;
        const float t = fmaxf(fmaxf(r[0], r[NG]), fmaxf(r[2 * NG], r[3 * NG]));
        a[k] = 1.f;
        if (t > kThresh) {   // (t is relative to m, which `scores` left here)
          const float mn = m[k] + (t - kLift);
          a[k] = fast_exp2(m[k] - mn);
          m[k] = mn;
          lq[k] *= a[k];
        }
      }
      named_bar_sync(barid, 128);   // red and the maxima have been read
      if (wq == 0 && (lane & 15) == 0) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          m_of(q)[k] = m[k];
          red[cg + k] = a[k];
        }
      }
      named_bar_sync(barid, 128);
      // O *= alpha (the PV product of the tile before is done)
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4 * NG; c += NO) {
        uint32_t o[NO];
        const uint32_t oa = tmem + lanes + L::kTmemO + (c / NG) * N + col0(q) + c % NG;
        tmem_get(oa, o);
#pragma unroll
        for (int k = 0; k < NO; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * red[c % NG + k]);
        tmem_put(oa, o);
      }
      tmem_wait_st();
      tc_fence_before();
      named_bar_sync(barid, 128);   // alpha has been read
    };
    // weights of the scores, in place (masked: exp2(-inf) = 0), and in 16 bits
    auto weights = [&](float (&x)[NC], uint32_t (&pk)[NC / 2]) {
#pragma unroll
      for (int k = 0; k < NC; k += 2) {
        x[k] = fast_exp2(x[k]);
        x[k + 1] = fast_exp2(x[k + 1]);
        pk[k / 2] = pack2<BF16>(x[k], x[k + 1]);
      }
    };
    // One tile: the first and the last of its piece, with `left` tokens of the unit from
    // its first on.  False: given up (the barriers of a group agree on it).
    auto tile = [&](const Unit4& ui, bool first, bool last, int left) {
      const int sb = g & 1;
      const bool cur = ui.p == fp.S;
      const float sl = cur ? fp.scale_log2 : fp.scale_log2 * fp.kv_scale;
      // rows below nmin are masked for this thread's token: all of a token past
      // the end; in the CURRENT part the rows of earlier query tokens
      int nmin = N;
      if (tok < left) nmin = cur ? min(N, max(0, tok * fp.H - ui.g * N)) : 0;
      const bool all = !cur && left >= kTile4;
      // P's place is as a rule free before the scores are there: waited for first, it is
      // off the path from the scores to the weights (16 rows 307 -> 304 us, 64 rows 862
      // -> 838 us; with 32 rows it is the other way round, 324 -> 343 us)
      if (N != 32 && g >= 1) ok = ok && waits.lazy(&bar[L::B_P_EMPTY], (g - 1) & 1);
      ok = __all_sync(0xffffffffu, ok && waits.lazy(&bar[L::B_S_FULL + sb], (g >> 1) & 1)) != 0;
      tc_fence_after();
      if (first) {
        // reference maxima of the piece
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
          float x[NC];
#pragma unroll
          for (int k = 0; k < NC; ++k) l[q][k] = 0.f;
          scores(q, sl, all, nmin, true, x);
          const float mx = col_reduce<NC, true>(x, lane);
          red_of(q)[wq * NG + cr] = mx;
        }
        if (!named_bar_and(barid, 128, ok)) return false;
        if (wq == 0 && lane < NG * PASSES) {
          const float* r = red_of(0) + (lane / NG) * (4 * NG) + lane % NG;
          const float t = fmaxf(fmaxf(r[0], r[NG]), fmaxf(r[2 * NG], r[3 * NG]));
          reinterpret_cast<float*>(smem + L::kMOff)[col0(0) + lane] = t == -INFINITY ? 0.f : t - kLift;
        }
        named_bar_sync(barid, 128);
        if constexpr (kKeepM) {
#pragma unroll
          for (int k = 0; k < NC; ++k) m[k] = m_of(0)[k];
        }
      }
      // The weights are made and handed over against the reference maxima as
      // they stand; a warp that finds one past the limit raises its group's flag of
      // this tile, and the group makes them again before the PV product, which
      // looks at the flags, reads them.  (A barrier to agree first cost 500
      // cycles of every tile.)
      uint32_t pk[PASSES][NC / 2];
      uint32_t sv[PASSES][NC];
#pragma unroll
      for (int q = 0; q < PASSES; ++q) tmem_half_issue(tmem + lanes + L::kTmemS + (g & 1) * N + col0(q), sv[q]);
      tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < PASSES; ++q)
#pragma unroll
        for (int k = 0; k < NC; ++k) asm volatile("" : "+r"(sv[q][k])::"memory");
      uint32_t over = 0;   // passes of this warp with such a weight: not in l yet
#pragma unroll
      for (int q = 0; q < PASSES; ++q) {
        float x[NC];
        rel(q, sl, all, nmin, sv[q], x);
        float top = fmaxf(x[0], x[1]);
#pragma unroll
        for (int k = 2; k < NC; ++k) top = fmaxf(top, x[k]);
        weights(x, pk[q]);
        if (__any_sync(0xffffffffu, top > kThresh)) {
          over |= 1u << q;
        } else {
#pragma unroll
          for (int k = 0; k < NC; ++k) l[q][k] += x[k];
        }
      }
      if (N == 32 && g >= 1) ok = __all_sync(0xffffffffu, ok && waits.lazy(&bar[L::B_P_EMPTY], (g - 1) & 1)) != 0;
      if (ok) {
#pragma unroll
        for (int q = 0; q < PASSES; ++q) put(q, pk[q]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          // (three tiles' flags in turn: every reader of the one cleared here
          // is behind P_FULL of the tile before, every writer behind this one)
          if (wq == 0) flags[((g + 1) % 3) * 2 + grp] = 0;
          if (over) flags[(g % 3) * 2 + grp] = 1;
          mbar_arrive(&bar[L::B_P_FULL]);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, waits.lazy(&bar[L::B_P_FULL], g & 1)) != 0;
      }
      if (ok) {
        const int mine = flags[(g % 3) * 2 + grp], other = flags[(g % 3) * 2 + (grp ^ 1)];
        if (mine | other) {
          if (mine) {
            if (!named_bar_and(barid, 128, ok)) return false;
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
              float x[NC];
              scores(q, sl, all, nmin, false, x);
              new_maxima(q, x, l[q]);   // (scales what l has of this tile, too)
              scores(q, sl, all, nmin, false, x);
              weights(x, pk[q]);
              put(q, pk[q]);
              if (over >> q & 1) {
#pragma unroll
                for (int k = 0; k < NC; ++k) l[q][k] += x[k];
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[L::B_P_FIXED]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::B_S_EMPTY + sb]);
      if (last) {
        // ---- epilogue of the piece: row sums over the tokens, O / l, LSE.  The sums,
        // factors and places are worked out while the last PV product runs.
        const bool whole = it.whole();
        // (a piece goes to the workspace in fp32, so that a row is rounded once, cut or not)
        const bool narrow = whole && fp.part_dtype != kFP32;
        char* out = static_cast<char*>(whole ? fp.o_part : fp.ws_o);
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
          const float part = col_reduce<NC, false>(l[q], lane);
          red_of(q)[N * 4 + wq * NG + cr] = part;
        }
        if (!named_bar_and(barid, 128, ok)) return false;
        // row `lane` of the group's, in every warp: its sum, its factor and where it goes (-1: nowhere)
        constexpr int NR = NG * PASSES;
        float inv = 0.f;
        int dst = -1;
        if (lane < NR) {
          const int n = col0(0) + lane, r = ui.g * N + n;
          const float* rl = red_of(0) + N * 4 + (lane / NG) * (4 * NG) + lane % NG;
          const float sum = (rl[0] + rl[NG]) + (rl[2 * NG] + rl[3 * NG]);
          inv = (cur ? 1.f : fp.kv_scale) / sum;
          if (r < fp.R) {
            const int slot = 2 * cid + (it.u == rng.u_begin ? 0 : 1);
            dst = whole ? static_cast<int>(out_row4(fp, ui.b, r, ui.p)) : slot * N + n;
            if (wq == 0) {
              const float lse2 = reinterpret_cast<const float*>(smem + L::kMOff)[n] + log2f(sum);
              if (whole) fp.lse_part[dst] = lse2 * kLn2;
              else fp.ws_lse[dst] = lse2;
            }
          }
        }
        // (a wait that gives up shows at the group's next barrier)
        ok = __all_sync(0xffffffffu, waits.lazy(&bar[L::B_P_EMPTY], g & 1)) != 0;
        tc_fence_after();
        if (!ok) {
        } else if (narrow) {
          // 32 latents of 8 rows at a time: read as matrix fragments, scaled,
          // stored transposed into the warp's staging (16-byte unit j of row k at
          // unit j ^ (k / 2 & 3): no bank conflicts) and from there to the rows,
          // 16 bytes a lane
          constexpr int NF = NG / 2;             // registers of a fragment: 4 for 8 rows
          constexpr int CU = N == 16 ? 2 : 1;    // blocks of 128 latents at a time
          constexpr int KA = N == 64 ? 2 : 1;    // eights of rows at a time
          float f[PASSES][NG / 4];
          int to[PASSES][NG / 8];                // rows of the output
          const int row = lane >> 2, unit = (lane & 3) ^ ((lane >> 3) & 3);
          const int mrow = lane & 7, munit = (lane >> 3) ^ ((mrow >> 1) & 3);
#pragma unroll
          for (int q = 0; q < PASSES; ++q) {
#pragma unroll
            for (int k = 0; k < NG / 8; ++k) {
              f[q][2 * k] = __shfl_sync(0xffffffffu, inv, q * NG + 8 * k + 2 * (lane & 3));
              f[q][2 * k + 1] = __shfl_sync(0xffffffffu, inv, q * NG + 8 * k + 2 * (lane & 3) + 1);
              to[q][k] = __shfl_sync(0xffffffffu, dst, q * NG + 8 * k + row);
            }
          }
          out += wq * 64 + (lane & 3) * 16;
          auto rows = [&](auto bf16) {   // (a branch for each pair of values otherwise)
            constexpr bool kToBf16 = decltype(bf16)::value;
#pragma unroll 1
          for (int c = 0; c < 4; c += CU) {
            uint32_t lo_[PASSES][CU][NF], hi_[PASSES][CU][NF];
#pragma unroll
            for (int q = 0; q < PASSES; ++q)
#pragma unroll
              for (int e = 0; e < CU; ++e) {
                const uint32_t oa = tmem + lanes + L::kTmemO + (c + e) * N + col0(q);
                tmem_ld_frag(oa, lo_[q][e]);
                tmem_ld_frag(oa + (16u << 16), hi_[q][e]);
              }
#pragma unroll
            for (int q = 0; q < PASSES; ++q)
#pragma unroll
              for (int e = 0; e < CU; ++e) tmem_wait_frag(lo_[q][e], hi_[q][e]);
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
              auto& lo = lo_[q];
              auto& hi = hi_[q];
#pragma unroll
              for (int k0 = 0; k0 < NG / 8; k0 += KA) {
                __syncwarp();   // the staging has been read
#pragma unroll
                for (int i = 0; i < CU * KA; ++i) {
                  const int e = i / KA, k = k0 + i % KA;
                  uint32_t w[4];
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    w[j] = pack2<kToBf16>(__uint_as_float(lo[e][4 * k + 2 * j]) * f[q][2 * k],
                                          __uint_as_float(lo[e][4 * k + 2 * j + 1]) * f[q][2 * k + 1]);
                    w[2 + j] = pack2<kToBf16>(__uint_as_float(hi[e][4 * k + 2 * j]) * f[q][2 * k],
                                              __uint_as_float(hi[e][4 * k + 2 * j + 1]) * f[q][2 * k + 1]);
                  }
                  stmatrix_x4_trans(smem_u32(stage_of(i)) + mrow * 64 + munit * 16, w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < CU * KA; ++i) {
                  const int e = i / KA, k = k0 + i % KA;
                  const uint4 x = ld_shared_v4(smem_u32(stage_of(i)) + row * 64 + unit * 16);
                  if (to[q][k] >= 0) *reinterpret_cast<uint4*>(out + to[q][k] * int64_t{1024} + (c + e) * 256) = x;
                }
              }
            }
          }
          };
          if (fp.part_dtype == kBF16) rows(std::true_type{});
          else rows(std::false_type{});
          tc_fence_before();
        } else {
          // fp32 rows: 8 rows of 32 latents at a time, written a latent per lane
#pragma unroll 1
          for (int c = 0; c < 4 * NG; c += NO) {
            const int n0 = c % NG;
            const int lat0 = (c / NG) * 128 + wq * 32;
#pragma unroll 1
            for (int q = 0; q < PASSES; ++q) {
              uint32_t o[NO];
              tmem_get(tmem + lanes + L::kTmemO + (c / NG) * N + col0(q) + n0, o);
              uint8_t* stage = stage_of(q);
#pragma unroll
              for (int h = 0; h < NO; h += NO / 2) {
#pragma unroll
                for (int k = 0; k < NO / 2; ++k)
                  reinterpret_cast<float*>(stage)[k * 32 + lane] = __uint_as_float(o[h + k]) * __shfl_sync(0xffffffffu, inv, q * NG + n0 + h + k);
                __syncwarp();
                const uint4 x = *reinterpret_cast<const uint4*>(stage + lane * 16);
                const int64_t d = __shfl_sync(0xffffffffu, dst, q * NG + n0 + h + (lane >> 3));
                if (d >= 0) *reinterpret_cast<uint4*>(out + d * 2048 + lat0 * 4 + (lane & 7) * 16) = x;
                __syncwarp();
              }
            }
          }
          tc_fence_before();
        }
      }
      return true;
    };
    // 64 rows: a piece at a time, so that little lives along its tiles (128 heads 778 ->
    // 766 us); fewer rows, where all of it fits the registers: tile by tile (16 heads 313
    // -> 300 us)
    if constexpr (N == 64) {
      bool go = true;
      while (go && it.valid) {
        const Unit4 ui = it.ui;
        int n = it.jend - it.j, left = ui.hi - it.tok0();
#pragma unroll 1
        for (bool first = true; go && n > 0; --n, ++g, left -= kTile4, first = false) go = tile(ui, first, n == 1, left);
        it.next_piece(fp);
      }
    } else {
      while (it.valid && tile(it.ui, it.first(), it.last(), it.ui.hi - it.tok0())) {
        it.advance(fp);
        ++g;
      }
    }
  } else {
    // ------------------------------------------------ unpacking
    // Eight warps for each half of the latents; a lane is a token, and its two
    // 32-column units of the half (the RoPE columns too, in the first) are decoded into
    // registers ahead of the slot, so that a slot that gets free waits for the
    // stores alone.  One fence and one arrival a tile and warp.
    const int w = warp - L::kUnpackWarp;
    const int h = w >> 3, t = (w & 1) * 32 + lane, grp = (w >> 1) & 3;
    const int part = L::kParts == 2 ? h : 2 * h + (grp >> 1);
    uint8_t* lat0 = smem + L::kLatOff + (L::kParts == 2 ? grp : grp & 1) * kChunk;   // (a chunk is the thread's two units)
    Iter4<N> it;
    it.start(fp, tab, rng);
    int g = 0, rs = 0;
    while (it.valid) {
      const bool cur = it.ui.p == fp.S;
      const bool valid = it.tok0() + t < it.ui.hi;
      uint4 x[2][4], xr[2];
      if (!cur) {
        const int st = rs % L::kNRaw;
        if (!__all_sync(0xffffffffu, waits.wait(&bar[L::B_RAW_FULL + st], (rs / L::kNRaw) & 1))) break;
        const uint8_t* codes = smem + L::kRawOff + st * kRawStage + t * kE2m1Codes;
        const uint8_t* scales = smem + L::kRawOff + st * kRawStage + kRawCodes + t * kE2m1Scales;
        uint4 c[2];
        uint32_t sc[2], rsc = 0;
        uint2 rc = make_uint2(0, 0);
        // Rows are 72 words apart, so eight lanes' 16 bytes of one unit fall on half
        // of the banks; four of them read the thread's two (adjacent) units in
        // the other order, and all banks are used.
        const int u0 = h * 8 + grp * 2;                       // 32-column unit of the 16
        const bool swap = (lane & 4) != 0;
        {
          const uint4 a = *reinterpret_cast<const uint4*>(codes + (u0 + (swap ? 1 : 0)) * 16);
          const uint4 b = *reinterpret_cast<const uint4*>(codes + (u0 + (swap ? 0 : 1)) * 16);
          c[0] = swap ? b : a;
          c[1] = swap ? a : b;
        }
        sc[0] = *reinterpret_cast<const uint16_t*>(scales + u0 * 2);
        sc[1] = *reinterpret_cast<const uint16_t*>(scales + u0 * 2 + 2);
        if (h == 0) {
          rc = *reinterpret_cast<const uint2*>(codes + 256 + grp * 8);
          rsc = scales[32 + grp];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[L::B_RAW_EMPTY + st]);
        ++rs;
        uint32_t m0, m1, a[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          multipliers(sc[k], valid, m0, m1);
          unpack8<BF16>(c[k].x, m0, a);
          x[k][0] = make_uint4(a[0], a[1], a[2], a[3]);
          unpack8<BF16>(c[k].y, m0, a);
          x[k][1] = make_uint4(a[0], a[1], a[2], a[3]);
          unpack8<BF16>(c[k].z, m1, a);
          x[k][2] = make_uint4(a[0], a[1], a[2], a[3]);
          unpack8<BF16>(c[k].w, m1, a);
          x[k][3] = make_uint4(a[0], a[1], a[2], a[3]);
        }
        if (h == 0) {
          multipliers(rsc, valid, m0, m1);
          unpack8<BF16>(rc.x, m0, a);
          xr[0] = make_uint4(a[0], a[1], a[2], a[3]);
          unpack8<BF16>(rc.y, m0, a);
          xr[1] = make_uint4(a[0], a[1], a[2], a[3]);
        }
      } else {
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(fp.kv_cur) +
                                                          (static_cast<int64_t>(it.ui.b) * fp.q_len + t) * 576);
        const uint4 none = make_uint4(0, 0, 0, 0);
        const bool clean = !current_bad<BF16>(row + grp * 8, valid ? h : -1);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[k][j] = valid && clean ? row[h * 32 + (grp * 2 + k) * 4 + j] : none;
#pragma unroll
        for (int j = 0; j < 2; ++j) xr[j] = valid && h == 0 ? row[64 + grp * 2 + j] : none;
        if (!clean) xr[0].x = 0x7FFF7FFFu;
      }
      const int hc = L::kParts * g + part, sl = hc % L::kSlots;
      if (hc >= L::kSlots && !__all_sync(0xffffffffu, waits.wait(&bar[L::B_EMPTY + sl], ((hc / L::kSlots) - 1) & 1))) break;
      // (with two RoPE slots the last reader of this one was done before the part's slot)
      if (L::kNR == 1 && h == 0 && g >= 1 &&
          !__all_sync(0xffffffffu, waits.wait(&bar[L::B_ROPE_EMPTY], (g - 1) & 1)))
        break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint8_t* d = lat0 + sl * L::kPart;
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(d + sw128_offset(t, k * 4 + j)) = x[k][j];
      }
      if (h == 0) {
        uint8_t* d = smem + L::kRopeOff + (g % L::kNR) * kChunk;
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4*>(d + sw128_offset(t, grp * 2 + j)) = xr[j];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::B_FULL + sl]);
      it.advance(fp);
      ++g;
    }
  }

  __syncwarp();
  tmem_wait_st();
  tmem_wait_ld();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------- merge of cut units
// A warp per row of the cut unit whose last tile the CTA blockIdx.x held: merges
// the unit's pieces by their LSEs.  A lane looks up a piece (up to 32 at a
// time), so their places and weights are there after three dependent reads;
// then the pieces' rows are summed in their order, 16 columns a lane.
__global__ void __launch_bounds__(256) mla_partial_fp4_merge_kernel(const Fp4Params fp, int rows) {
  griddep_wait();
  const int4 rec = fp.ws_units[blockIdx.x];
  const int u = rec.x, lane = threadIdx.x & 31;
  const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (u < 0) return;
  const int p = u % fp.P, gb = u / fp.P, b = gb % fp.B, r = (gb / fp.B) * rows + n;
  if (r >= fp.R) return;
  float acc[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) acc[t] = 0.f;
  float m = -INFINITY, wsum = 0.f;
  for (int c0 = rec.z; c0 <= rec.w; c0 += 32) {
    const int c = c0 + lane;
    int64_t row = 0;
    float l = -INFINITY;
    if (c <= rec.w) {
      const int s0 = fp.ws_bounds[c], s1 = fp.ws_bounds[c + 1];
      if (s1 > s0) {   // (else a CTA without tiles)
        row = static_cast<int64_t>(2 * c + (s0 >= rec.y ? 0 : 1)) * rows + n;   // its first or last piece
        l = fp.ws_lse[row];
      }
    }
    float mx = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx > m) {   // a new reference maximum (at first the scale is 0)
      const float sc = exp2f(m - mx);
#pragma unroll
      for (int t = 0; t < 16; ++t) acc[t] *= sc;
      wsum *= sc;
      m = mx;
    }
    // (a NaN is no maximum; it goes through its weight)
    const float w = row == 0 && l == -INFINITY ? 0.f : l == m ? 1.f : exp2f(l - m);
    const int np = min(32, rec.w - c0 + 1);
#pragma unroll 4
    for (int k = 0; k < np; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const int64_t e0 = __shfl_sync(0xffffffffu, row, k) * 512 + lane * 16;
      if (wk == 0.f) continue;
      wsum += wk;
      const float4* src = reinterpret_cast<const float4*>(fp.ws_o + e0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = src[j];
        acc[4 * j] = fmaf(wk, f.x, acc[4 * j]);
        acc[4 * j + 1] = fmaf(wk, f.y, acc[4 * j + 1]);
        acc[4 * j + 2] = fmaf(wk, f.z, acc[4 * j + 2]);
        acc[4 * j + 3] = fmaf(wk, f.w, acc[4 * j + 3]);
      }
    }
  }
  const float inv = 1.f / wsum;
  const int64_t row = out_row4(fp, b, r, p);
  if (fp.part_dtype == kFP32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(fp.o_part) + row * 512 + lane * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      d[j] = make_float4(acc[4 * j] * inv, acc[4 * j + 1] * inv, acc[4 * j + 2] * inv, acc[4 * j + 3] * inv);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack2_dt(acc[2 * j] * inv, acc[2 * j + 1] * inv, fp.part_dtype);
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(fp.o_part) + row * 512 + lane * 16);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  if (lane == 0) fp.lse_part[row] = (m + log2f(wsum)) * kLn2;
}

// ---------------------------------------------------------------- launcher
template <bool BF16, int N, bool SHARES>
static bool prepare4(int dev) {
  static bool done[64] = {false};
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (cudaFuncSetAttribute(mla_partial_fp4_kernel<BF16, N, SHARES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem4<N>::kTotal) != cudaSuccess)
      return false;
    done[dev] = true;
  }
  return true;
}

int fp4_max_ctas() {
  static int cache[64] = {0};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return -1;
    cache[dev] = std::min(n, kFp4MaxCtas);
  }
  return cache[dev];
}

template <bool BF16, int N, bool SHARES>
static int launch4(const CUtensorMap& qlat, const CUtensorMap& qpe, const Fp4Params& fp, int ctas, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !prepare4<BF16, N, SHARES>(dev)) return -1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(Smem4<N>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Smem4<N>::kTotal;
  if (cudaLaunchKernelEx(&cfg, mla_partial_fp4_kernel<BF16, N, SHARES>, qlat, qpe, fp) != cudaSuccess) return -1;
  if (!fp.split) return 0;
  cfg.gridDim = dim3(ctas, N / 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mla_partial_fp4_merge_kernel, fp, N) != cudaSuccess ? -1 : 0;
}

template <bool BF16, int N>
static int launch4(const CUtensorMap& qlat, const CUtensorMap& qpe, const Fp4Params& fp, cudaStream_t stream) {
  const int most = fp4_max_ctas();
  if (most < 1) return -1;
  if (fp.split) return launch4<BF16, N, true>(qlat, qpe, fp, fp.split, stream);
  return fp.num_units <= most ? launch4<BF16, N, false>(qlat, qpe, fp, fp.num_units, stream)
                              : launch4<BF16, N, true>(qlat, qpe, fp, most, stream);
}

int launch_partial_fp4(const CUtensorMap& qlat, const CUtensorMap& qpe, const Fp4Params& fp, int rows,
                       bool bf16, cudaStream_t stream) {
  if (rows == 16) return bf16 ? launch4<true, 16>(qlat, qpe, fp, stream) : launch4<false, 16>(qlat, qpe, fp, stream);
  if (rows == 32) return bf16 ? launch4<true, 32>(qlat, qpe, fp, stream) : launch4<false, 32>(qlat, qpe, fp, stream);
  return bf16 ? launch4<true, 64>(qlat, qpe, fp, stream) : launch4<false, 64>(qlat, qpe, fp, stream);
}

}  // namespace mla
