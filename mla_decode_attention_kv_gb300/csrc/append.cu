// mla_kv_append: what a step's projections leave of a token, made into a
// cached row and written to its slot, in one launch:
//   latent   y = c * rsqrt(mean c^2 + eps) * w           (512 values)
//   key      the 64 RoPE values, rotated pair by pair by their positions
//   queries  every head's 64 RoPE values, rotated the same way
// The row goes to the paged cache as 16-bit values, as E4M3 bytes, or as E2M1
// codes with an E4M3 scale for every 16 values.
//
// Mathematics.  A pair (a, b) at position m turns into (a cos - b sin, a sin +
// b cos) with cos and sin read from a table row of that position; with several
// axes (time, height, width) a pair reads the row of its section's position.
//
// What is stored in 8 or 4 bits is the nearest code of the value itself.  A
// value computed in plain fp32 is off by up to 2^-20 (in halves of a last bit: the
// sum of squares 15, halved by the root, rsqrtf 4, its products with the value and
// the scale 4) and lands, once in a few million values, on the wrong side of a border between
// two 4-bit codes that lie a third of their size apart; the cache would then
// depend on the order of a sum.  So a row is made twice over: in fp32, where
// each code is taken at a little less and a little more (2^-19) than the value,
// and, where some code of the row differs (a row in some 400 for E2M1, in 30
// for E4M3), again exactly: values as unevaluated sums hi + lo of two fp32
// numbers (sums and products with their exact errors, Dekker and Knuth), about
// 2^-46 off, rounded with lo folded into the last bit of hi (round to odd),
// which rounds on to fewer bits the same way as hi + lo itself.  16-bit rows
// are always made the exact way.
//
// What bounds it: the launch for few tokens (one token 2.2 us, 32 tokens of 128
// heads into E2M1 3.7, 1.3 of them where a row needs the exact form); for many the
// row arithmetic (8192 tokens of 16 heads into E2M1: 12.9 us, of which the rows
// alone 9.8; 57 MB at 4.4 TB/s, 0.65 of the measured copy bandwidth; with other inputs
// each time 14.0, into E4M3 12.7, into 16 bits 15.7).  With half the
// blocks on an SM the time is the same, with smaller register budgets 17 and 22 us.
// One warp makes a token's row:
// lane l owns latents 16 l .. 16 l + 15, which are one block of the E2M1 form,
// so a block's maximum and its 8 bytes of codes stay in a lane; the key's pair
// l belongs to lane l.  The queries go to blocks of their own, eight lanes a
// head, 16 bytes a lane, four heads of a token per lane.
#include <cuda_fp8.h>
#include "cache_kernels.cuh"
#include "common.cuh"

namespace mla {

namespace {

// hi + lo, |lo| <= ulp(hi) / 2
struct F2 {
  float hi, lo;
};

__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = a + b;
  const float bb = s - a;
  return {s, (a - (s - bb)) + (b - bb)};
}

__device__ __forceinline__ F2 renorm(float hi, float lo) {
  const float s = hi + lo;
  return {s, lo - (s - hi)};
}

// hi + lo rounded to odd: the fp32 neighbour of the value whose last bit is 1
// (hi itself where lo is 0).  Rounding that to fewer bits gives the nearest
// code of hi + lo.  NaN and infinities pass.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  const uint32_t u = __float_as_uint(hi);
  const bool neg = (u >> 31) != 0;
  uint32_t v = u;
  if ((lo > 0.f && !neg) || (lo < 0.f && neg)) v = u | 1u;
  if ((lo > 0.f && neg) || (lo < 0.f && !neg)) v = (u - 1u) | 1u;
  return __uint_as_float(v);
}

// a / d rounded to odd, a >= 0 and d > 0: the correctly rounded quotient and
// the sign of its exact remainder say on which side the quotient lies.
__device__ __forceinline__ float div_odd(float a, float d) {
  const float q = __fdiv_rn(a, d);
  const float r = fmaf(-q, d, a);
  uint32_t u = __float_as_uint(q);
  if (r > 0.f) u |= 1u;
  if (r < 0.f) u = (u - 1u) | 1u;
  return __uint_as_float(u);
}

// (a, b) turned by (cos, sin): the exact products' sums, as hi + lo
__device__ __forceinline__ F2 mul_diff(float a, float c, float b, float s) {   // a c - b s
  const float p1 = a * c, e1 = fmaf(a, c, -p1);
  const float p2 = b * s, e2 = fmaf(b, s, -p2);
  const F2 d = two_sum(p1, -p2);
  const float lo = d.lo + (e1 - e2);
  // (a zero keeps the sum's sign; an infinity, whose errors are NaN, stays one)
  return lo == 0.f || lo != lo ? F2{d.hi, 0.f} : renorm(d.hi, lo);
}

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  return unpack2(w, BF16 ? kBF16 : kFP16);
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  const uint16_t u = static_cast<const uint16_t*>(p)[i];
  return unpack<BF16>(u).x;
}

template <bool BF16>
__device__ __forceinline__ uint16_t pack1(float a) {
  return static_cast<uint16_t>(pack2<BF16>(a, 0.f) & 0xFFFFu);
}

__device__ __forceinline__ uint32_t to_e4m3(float x) {
  return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float from_e4m3(uint32_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// Four E4M3 bytes of four values, and eight E2M1 codes of eight (the first in
// the low bits; rounded to nearest even, saturating, zeros with their signs).
// One block of PTX each: through the headers' byte types the packing takes
// several times the conversions' instructions.
__device__ __forceinline__ uint32_t to_e4m3x4(const float* v, float m) {
  uint32_t o;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
      " mov.b32 %0, {a, b};\n}\n"
      : "=r"(o)
      : "f"(v[0] * m), "f"(v[1] * m), "f"(v[2] * m), "f"(v[3] * m));
  return o;
}

__device__ __forceinline__ uint32_t to_e2m1x8(const float* v, float m) {
  uint32_t o;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(o)
      : "f"(v[0] * m), "f"(v[1] * m), "f"(v[2] * m), "f"(v[3] * m), "f"(v[4] * m), "f"(v[5] * m), "f"(v[6] * m),
        "f"(v[7] * m));
  return o;
}

__device__ __forceinline__ uint32_t to_e2m1x2(float x, float y) {   // x in the low half
  uint32_t o;
  asm("{\n .reg .b8 a, z;\n mov.b16 {a, z}, 0;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n mov.b32 %0, {a, z, z, z};\n}\n"
      : "=r"(o)
      : "f"(x), "f"(y));
  return o;
}

// A little less and a little more than a value: the bounds of its fp32 error.
constexpr float kLess = 1.f - 0x1p-19f, kMore = 1.f + 0x1p-19f;

// The mean square plus eps counts as at least this, so that a row of zeros with
// eps 0 stays zeros, and the estimate's square stays in range (a NaN passes).
constexpr float kLeastMean = 0x1p-120f;

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}

// E4M3 byte of a block's scale, max / (6 kv_scale); NaN where a value is NaN.
// EXACT: amax is rounded to odd.  Otherwise `same` turns false where amax's
// error could change the byte.
template <bool EXACT>
__device__ __forceinline__ uint32_t block_scale(float amax, const AppendParams& ap, bool& same) {
  uint32_t b;
  if constexpr (EXACT) {
    b = to_e4m3(div_odd(amax, ap.kv6));
  } else {
    const float q = amax * ap.inv_kv6;
    b = to_e4m3(q * kLess);
    same &= b == to_e4m3(q * kMore);
  }
  return amax != amax ? 0x7Fu : b;
}

// The signed quotient v / d rounded to odd, 0 (with v's sign) for d = 0.
__device__ __forceinline__ float div_signed(float v, float d) {
  return copysignf(d > 0.f ? div_odd(fabsf(v), d) : 0.f, v);
}

// The values of four bytes of codes, times d, as 16-bit pairs.
template <bool BF16>
__device__ __forceinline__ void e2m1_values(uint32_t c, float d, uint32_t* w) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
    w[k] = pack2<BF16>(f.x * d, f.y * d);
  }
}

// Position of RoPE pair i of token t: that of the axis its section belongs to.
// Out-of-range positions are recorded and read as 0.
__device__ __forceinline__ int pair_position(const AppendParams& ap, int t, int i) {
  const int axis = (i >= ap.sec1) + (i >= ap.sec2);
  int pos = ap.positions[static_cast<int64_t>(axis) * ap.T + t];
  if (pos < 0 || pos >= ap.max_pos) {
    set_error(ap.err, kDevBadPosition);
    pos = 0;
  }
  return pos;
}

// One token's row, by one warp.  EXACT false: false, with nothing stored, if
// some code of the row needs the exact form.
template <bool BF16, int KIND, bool EXACT>
__device__ __forceinline__ bool append_row(const AppendParams& ap, int t, int lane) {
  // ---- latent: 16 values a lane
  uint32_t cw[8];
  {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(ap.c_kv) +
                                                      t * ap.c_stride + 16 * lane);
    const uint4 a = src[0], b = src[1];
    cw[0] = a.x; cw[1] = a.y; cw[2] = a.z; cw[3] = a.w;
    cw[4] = b.x; cw[5] = b.y; cw[6] = b.z; cw[7] = b.w;
  }
  // ---- key: pair `lane`
  float ka, kb;
  if (ap.interleaved) {
    const float2 f = unpack<BF16>(*reinterpret_cast<const uint32_t*>(
        static_cast<const uint16_t*>(ap.k_pe) + t * ap.k_stride + 2 * lane));
    ka = f.x;
    kb = f.y;
  } else {
    ka = load1<BF16>(ap.k_pe, t * ap.k_stride + lane);
    kb = load1<BF16>(ap.k_pe, t * ap.k_stride + 32 + lane);
  }
  const float* cs = ap.cos_sin + static_cast<int64_t>(pair_position(ap, t, lane)) * 64;
  const float co = cs[lane], si = cs[32 + lane];
  const int slot = ap.slots[t];

  float y[16];       // the row's values: EXACT, rounded to odd; otherwise y * by
  float by = 1.f;
  bool same = true;
  if (ap.weight) {
    uint32_t ww[8];
    const uint4* wsrc = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(ap.weight) + 16 * lane);
    const uint4 a = wsrc[0], b = wsrc[1];
    ww[0] = a.x; ww[1] = a.y; ww[2] = a.z; ww[3] = a.w;
    ww[4] = b.x; ww[5] = b.y; ww[6] = b.z; ww[7] = b.w;
    if constexpr (EXACT) {
      // sum of squares: the squares of 16-bit values are exact in fp32, each
      // addition's error is kept.  Where it passes fp32 (bf16 rows from some 1e18 on)
      // it is taken again of the values times 2^-70, the same for the lanes' products.
      float s, e, sc = 1.f;
      while (true) {
        s = e = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = unpack<BF16>(cw[k]);
          const float fx = f.x * sc, fy = f.y * sc;
          F2 u = two_sum(s, fx * fx);
          e += u.lo;
          u = two_sum(u.hi, fy * fy);
          s = u.hi;
          e += u.lo;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
          const F2 u = two_sum(s, s2);
          s = u.hi;
          e = (e + e2) + u.lo;
        }
        if (!BF16 || s < INFINITY || sc != 1.f) break;   // (all lanes have the same s)
        sc = 0x1p-70f;
      }
      F2 m = two_sum(s * (1.f / 512), ap.eps * (sc * sc));
      m = renorm(m.hi, m.lo + e * (1.f / 512));
      if (m.hi < kLeastMean) m = {kLeastMean, 0.f};
      // 1 / sqrt(m): the fp32 estimate and one Newton step on its exact residual
      float r0 = rsqrtf(m.hi);
      const float r2 = r0 * r0, r2e = fmaf(r0, r0, -r2);
      const float res = fmaf(-m.hi, r2, 1.f) - (m.hi * r2e + m.lo * r2);
      float rl = 0.5f * r0 * res;
      if (s == INFINITY) r0 = rl = 0.f;   // a row with an infinity
      const bool plain = s < INFINITY;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = unpack<BF16>(cw[k]), w = unpack<BF16>(ww[k]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float xw = h ? f.y * sc * w.y : f.x * sc * w.x;   // exact
          const float p = xw * r0;
          const F2 v = renorm(p, fmaf(xw, r0, -p) + xw * rl);
          y[2 * k + h] = xw == 0.f || !plain ? p : to_odd(v.hi, v.lo);
        }
      }
    } else {
      float s = 0.f, e = 0.f;   // (two chains: half the latency and half the error)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = unpack<BF16>(cw[k]);
        s = fmaf(f.x, f.x, s);
        e = fmaf(f.y, f.y, e);
      }
      s += e;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      same = s < INFINITY;
      const float mean = fmaf(s, 1.f / 512, ap.eps);
      by = rsqrtf(mean < kLeastMean ? kLeastMean : mean);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = unpack<BF16>(cw[k]), w = unpack<BF16>(ww[k]);
        y[2 * k] = f.x * w.x;
        y[2 * k + 1] = f.y * w.y;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = unpack<BF16>(cw[k]);
      y[2 * k] = f.x;
      y[2 * k + 1] = f.y;
    }
  }
  const F2 v0 = mul_diff(ka, co, kb, si), v1 = mul_diff(ka, si, kb, -co);
  const float r0 = to_odd(v0.hi, v0.lo), r1 = to_odd(v1.hi, v1.lo);

  bool store = slot >= 0;
  if (slot < -1 || slot >= ap.num_slots) {
    if (lane == 0) set_error(ap.err, kDevBadSlot);
    store = false;
  }
  // element of the key's two values within the row
  const int e0 = 512 + (ap.interleaved ? 2 * lane : lane);
  const int e1 = ap.interleaved ? e0 + 1 : e0 + 32;

  if constexpr (KIND == kKvModel || KIND == kKvE2M1) {
    uint32_t w[8];
    float q0 = r0, q1 = r1;
    if constexpr (KIND == kKvE2M1) {
      // latent: the lane's 16 values are one block
      float am = fabsf(y[0]);
#pragma unroll
      for (int k = 1; k < 16; ++k) am = max_nan(am, fabsf(y[k]));
      am *= by;
      const bool nan = am != am;
      const uint32_t sb = block_scale<EXACT>(am, ap, same);
      const float d = from_e4m3(sb) * ap.kv_scale;
      uint32_t code[2];
      if constexpr (EXACT) {
        float q[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) q[k] = div_signed(y[k], d);
        code[0] = to_e2m1x8(q, 1.f);
        code[1] = to_e2m1x8(q + 8, 1.f);
      } else {
        const float rd = d > 0.f ? __frcp_rn(d) * by : 0.f;
        same &= rd < INFINITY || nan;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          code[k] = to_e2m1x8(y + 8 * k, rd * kLess);
          same &= code[k] == to_e2m1x8(y + 8 * k, rd * kMore) || nan;
        }
      }
      if (ap.kv_out) {
        e2m1_values<BF16>(code[0], d, w);
        e2m1_values<BF16>(code[1], d, w + 4);
      }
      // key: a block is 8 lanes' pairs (interleaved) or 16 lanes' first or
      // second values (halves)
      float a0 = fabsf(r0), a1 = fabsf(r1);
      // (the key's values are exact in either form, so its codes are taken once)
      bool unused = true;
      uint32_t sb0, sb1;
      if (ap.interleaved) {
        a0 = max_nan(a0, a1);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) a0 = max_nan(a0, __shfl_xor_sync(0xffffffffu, a0, o));
        sb0 = sb1 = block_scale<true>(a0, ap, unused);
      } else {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          a0 = max_nan(a0, __shfl_xor_sync(0xffffffffu, a0, o));
          a1 = max_nan(a1, __shfl_xor_sync(0xffffffffu, a1, o));
        }
        sb0 = block_scale<true>(a0, ap, unused);
        sb1 = block_scale<true>(a1, ap, unused);
      }
      const float d0 = from_e4m3(sb0) * ap.kv_scale, d1 = from_e4m3(sb1) * ap.kv_scale;
      const uint32_t kc = to_e2m1x2(div_signed(r0, d0), div_signed(r1, d1));
      {
        uint32_t v[4];
        e2m1_values<BF16>(kc, 1.f, v);
        const float2 f = unpack<BF16>(v[0]);
        q0 = f.x * d0;
        q1 = f.y * d1;
      }
      if constexpr (!EXACT)
        if (!__all_sync(0xffffffffu, same)) return false;
      // scales of four lanes in a word: lane 4 j writes blocks 4 j .. 4 j + 3
      uint32_t sw = sb;
      sw |= __shfl_down_sync(0xffffffffu, sw, 1) << 8;
      sw |= __shfl_down_sync(0xffffffffu, sw, 2) << 16;
      // the key's four block scales: one per eighth lane (interleaved), or the
      // two halves' of lanes 0 and 16
      const uint32_t ks = ap.interleaved
                              ? (__shfl_sync(0xffffffffu, sb0, 0) | (__shfl_sync(0xffffffffu, sb0, 8) << 8) |
                                 (__shfl_sync(0xffffffffu, sb0, 16) << 16) | (__shfl_sync(0xffffffffu, sb0, 24) << 24))
                              : (__shfl_sync(0xffffffffu, sb0, 0) | (__shfl_sync(0xffffffffu, sb0, 16) << 8) |
                                 (__shfl_sync(0xffffffffu, sb1, 0) << 16) | (__shfl_sync(0xffffffffu, sb1, 16) << 24));
      // byte `lane` of the key's 32 (halves: even lanes hold the pair of first
      // values of lanes l, l + 1, odd ones that of the second values)
      const uint32_t other = __shfl_xor_sync(0xffffffffu, kc, 1);
      uint32_t kbyte = kc;
      int kat = lane;
      if (!ap.interleaved) {
        kbyte = (lane & 1) ? ((other >> 4) | (kc & 0xF0u)) : ((kc & 15u) | ((other & 15u) << 4));
        kat = (lane & 1) * 16 + (lane >> 1);
      }
      if (store) {
        const int page = slot / ap.bs, off = slot - page * ap.bs;
        uint8_t* base = static_cast<uint8_t*>(ap.cache) + static_cast<int64_t>(page) * ap.bs * kE2m1Row;
        uint8_t* codes = base + off * kE2m1Codes;
        uint8_t* scales = base + ap.bs * kE2m1Codes + off * kE2m1Scales;
        *reinterpret_cast<uint2*>(codes + 8 * lane) = make_uint2(code[0], code[1]);
        codes[256 + kat] = static_cast<uint8_t>(kbyte);
        if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(scales + lane) = sw;
        if (lane == 0) *reinterpret_cast<uint32_t*>(scales + 32) = ks;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = pack2<BF16>(y[2 * k], y[2 * k + 1]);
    }
    auto put = [&](uint16_t* row) {
      uint4* d4 = reinterpret_cast<uint4*>(row + 16 * lane);
      d4[0] = make_uint4(w[0], w[1], w[2], w[3]);
      d4[1] = make_uint4(w[4], w[5], w[6], w[7]);
      if (ap.interleaved) {
        *reinterpret_cast<uint32_t*>(row + e0) = pack2<BF16>(q0, q1);
      } else {
        row[e0] = pack1<BF16>(q0);
        row[e1] = pack1<BF16>(q1);
      }
    };
    if (ap.kv_out) put(static_cast<uint16_t*>(ap.kv_out) + static_cast<int64_t>(t) * 576);
    if (KIND == kKvModel && store) put(static_cast<uint16_t*>(ap.cache) + static_cast<int64_t>(slot) * 576);
  } else {
    uint32_t w[4];
    if constexpr (EXACT) {
      float q[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k] = div_signed(y[k], ap.kv_scale);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = to_e4m3x4(q + 4 * k, 1.f);
    } else {
      const float rd = ap.inv_kv * by;
      // (a product below fp32's normal range keeps too few bits; a NaN goes that way too)
      same &= rd < INFINITY && rd >= 0x1p-100f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = to_e4m3x4(y + 4 * k, rd * kLess);
        same &= w[k] == to_e4m3x4(y + 4 * k, rd * kMore);
      }
      if (!__all_sync(0xffffffffu, same)) return false;
    }
    const uint32_t b0 = to_e4m3(div_signed(r0, ap.kv_scale)), b1 = to_e4m3(div_signed(r1, ap.kv_scale));
    auto put = [&](uint8_t* row) {
      *reinterpret_cast<uint4*>(row + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
      if (ap.interleaved) {
        *reinterpret_cast<uint16_t*>(row + e0) = static_cast<uint16_t>(b0 | (b1 << 8));
      } else {
        row[e0] = static_cast<uint8_t>(b0);
        row[e1] = static_cast<uint8_t>(b1);
      }
    };
    if (ap.kv_out) put(static_cast<uint8_t*>(ap.kv_out) + static_cast<int64_t>(t) * 576);
    if (store) put(static_cast<uint8_t*>(ap.cache) + static_cast<int64_t>(slot) * 576);
  }
  return true;
}

template <bool BF16, int KIND>
__device__ __noinline__ void append_row_exact(const AppendParams& ap, int t, int lane) {
  append_row<BF16, KIND, true>(ap, t, lane);
}

// Up to kQueryHeads heads of one token's queries, by one warp: lane j of a
// head's eight has pairs 4 j .. 4 j + 3, and the same pairs of every fourth
// head, so the cosines are read once and all heads' loads are in flight with
// them.
template <bool BF16>
__device__ void rotate_queries(const AppendParams& ap, int64_t item, int lane) {
  const int t = static_cast<int>(item / ap.q_groups);
  const int h0 = static_cast<int>(item - static_cast<int64_t>(t) * ap.q_groups) * kQueryHeads + (lane >> 3);
  const int j = lane & 7;
  const uint16_t* src = static_cast<const uint16_t*>(ap.q_pe) + t * ap.q_stride;
  uint16_t* dst = static_cast<uint16_t*>(ap.q_out) + t * ap.qo_stride;
  constexpr int kN = kQueryHeads / 4;
  uint2 x[kN] = {}, z[kN] = {};
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int h = h0 + 4 * n;
    if (h >= ap.H) continue;
    if (ap.interleaved) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + h * ap.q_head_stride + 8 * j);
      x[n] = make_uint2(v.x, v.y);
      z[n] = make_uint2(v.z, v.w);
    } else {
      x[n] = *reinterpret_cast<const uint2*>(src + h * ap.q_head_stride + 4 * j);
      z[n] = *reinterpret_cast<const uint2*>(src + h * ap.q_head_stride + 32 + 4 * j);
    }
  }
  float4 co, si;
  const int i0 = 4 * j;
  // the four pairs read one row unless a section ends among them
  const bool cut = (ap.sec1 > i0 && ap.sec1 < i0 + 4) || (ap.sec2 > i0 && ap.sec2 < i0 + 4);
  if (!cut) {
    const float* cs = ap.cos_sin + static_cast<int64_t>(pair_position(ap, t, i0)) * 64 + i0;
    co = *reinterpret_cast<const float4*>(cs);
    si = *reinterpret_cast<const float4*>(cs + 32);
  } else {
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* cs = ap.cos_sin + static_cast<int64_t>(pair_position(ap, t, i0 + k)) * 64 + i0 + k;
      c[k] = cs[0];
      s[k] = cs[32];
    }
    co = make_float4(c[0], c[1], c[2], c[3]);
    si = make_float4(s[0], s[1], s[2], s[3]);
  }
  const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int h = h0 + 4 * n;
    if (h >= ap.H) continue;
    const float2 f0 = unpack<BF16>(x[n].x), f1 = unpack<BF16>(x[n].y), f2 = unpack<BF16>(z[n].x), f3 = unpack<BF16>(z[n].y);
    const float e[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
    float u[4], v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = ap.interleaved ? e[2 * k] : e[k], b = ap.interleaved ? e[2 * k + 1] : e[4 + k];
      u[k] = fmaf(a, c[k], -(b * s[k]));
      v[k] = fmaf(a, s[k], b * c[k]);
    }
    uint16_t* row = dst + h * ap.qo_head_stride;
    if (ap.interleaved) {
      *reinterpret_cast<uint4*>(row + 8 * j) =
          make_uint4(pack2<BF16>(u[0], v[0]), pack2<BF16>(u[1], v[1]), pack2<BF16>(u[2], v[2]), pack2<BF16>(u[3], v[3]));
    } else {
      *reinterpret_cast<uint2*>(row + 4 * j) = make_uint2(pack2<BF16>(u[0], u[1]), pack2<BF16>(u[2], u[3]));
      *reinterpret_cast<uint2*>(row + 32 + 4 * j) = make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
    }
  }
}

}  // namespace

template <bool BF16, int KIND>
__global__ void __launch_bounds__(kAppendThreads, 16) mla_kv_append_kernel(const __grid_constant__ AppendParams ap) {
  griddep_wait();
  griddep_launch_dependents();
  const int blk = static_cast<int>(blockIdx.x);
  if (blk < ap.row_blocks) {
    const int t = blk * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= ap.T) return;
    if constexpr (KIND == kKvModel)
      append_row<BF16, KIND, true>(ap, t, threadIdx.x & 31);
    else if (!append_row<BF16, KIND, false>(ap, t, threadIdx.x & 31))
      append_row_exact<BF16, KIND>(ap, t, threadIdx.x & 31);
  } else {
    const int64_t item = static_cast<int64_t>(blk - ap.row_blocks) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (item < static_cast<int64_t>(ap.T) * ap.q_groups) rotate_queries<BF16>(ap, item, threadIdx.x & 31);
  }
}

template <bool BF16>
static int launch_append_t(const AppendParams& ap, int kind, unsigned blocks, cudaStream_t stream) {
  auto* kernel = kind == kKvModel  ? mla_kv_append_kernel<BF16, kKvModel>
                 : kind == kKvE4M3 ? mla_kv_append_kernel<BF16, kKvE4M3>
                                   : mla_kv_append_kernel<BF16, kKvE2M1>;
  return launch_overlapped(kernel, dim3(blocks), kAppendThreads, stream, ap) == cudaSuccess ? 0 : -1;
}

int launch_append(AppendParams ap, int kind, bool bf16, cudaStream_t stream) {
  ap.row_blocks = ceil_div(ap.T, kAppendThreads / 32);
  ap.q_groups = ap.q_pe ? ceil_div(ap.H, kQueryHeads) : 0;
  const int64_t blocks = append_blocks(ap.T, ap.q_pe ? ap.H : 0);
  return bf16 ? launch_append_t<true>(ap, kind, static_cast<unsigned>(blocks), stream)
              : launch_append_t<false>(ap, kind, static_cast<unsigned>(blocks), stream);
}

}  // namespace mla
