// Partial attention per context shard over a 4-bit (E2M1) latent cache:
// mla_dcp_decode_partial_fp4.  The attention is the one of the 16-bit kernel
// on the decoded values e * s * kv_scale.
#include "cache_kernels.cuh"
#include "partial_fp4.cuh"
#include "partial_sched.cuh"

namespace mla {

namespace {
constexpr int kTok = 16;   // tokens per tile

__device__ __forceinline__ float e2m1_f32(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float mag = e == 0 ? 0.5f * m : __uint_as_float((126u + e) << 23) * (1.f + 0.5f * m);
  return (c & 8u) ? -mag : mag;
}
}  // namespace

// One block per (sequence, query token, part, 8 heads), a warp per head.
template <bool BF16>
__global__ void __launch_bounds__(256) mla_partial_fp4_kernel(const Fp4Params fp) {
  __shared__ float tile[kTok][576];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = blockIdx.x;
  const int p = u % fp.P, i = (u / fp.P) % fp.q_len, b = u / (fp.P * fp.q_len);
  const int h = blockIdx.y * 8 + warp;
  const bool cur = p == fp.S;
  int lo = 0, hi = i + 1;
  if (!cur) {
    int L = fp.seq_lens[b];
    const int cap = fp.max_blocks * fp.bs;
    if (L < 0 || L > cap) {
      set_error(fp.err, kDevBadSeqLen);
      L = max(0, min(L, cap));
    }
    const int chunk = fp.S * fp.bs;
    const int len = fp.bs * ((L + chunk - 1) / chunk);
    lo = min(L, p * len);
    hi = min(L, (p + 1) * len);
  }
  const int64_t row = (static_cast<int64_t>(b) * fp.q_len + i) * fp.H + min(h, fp.H - 1);
  float q[18], o[16];
  const uint16_t* qa = static_cast<const uint16_t*>(fp.q_abs) + row * 512;
  const uint16_t* qp = static_cast<const uint16_t*>(fp.q_pe) + row * 64;
  for (int k = 0; k < 18; ++k) {
    const int c = lane + 32 * k;
    q[k] = unpack2(c < 512 ? qa[c] : qp[c - 512], BF16 ? kBF16 : kFP16).x;
  }
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int t0 = lo; t0 < hi; t0 += kTok) {
    const int n = min(kTok, hi - t0);
    __syncthreads();
    for (int x = threadIdx.x; x < n * 36; x += 256) {
      const int t = x / 36, g = x - t * 36, tok = t0 + t;
      if (cur) {
        const uint16_t* src = static_cast<const uint16_t*>(fp.kv_cur) +
                              (static_cast<int64_t>(b) * fp.q_len + tok) * 576 + g * 16;
        for (int e = 0; e < 16; ++e) tile[t][g * 16 + e] = unpack2(src[e], BF16 ? kBF16 : kFP16).x;
      } else {
        int id = fp.block_table[static_cast<int64_t>(b) * fp.max_blocks + tok / fp.bs];
        if (id < 0 || id >= fp.num_blocks) {
          set_error(fp.err, kDevBadBlockId);
          id = 0;
        }
        const uint8_t* page = fp.kv_cache + static_cast<int64_t>(id) * fp.bs * kE2m1Row;
        const int off = tok & (fp.bs - 1);
        const uint8_t* codes = page + off * kE2m1Codes + g * 8;
        const __half_raw hr = __nv_cvt_fp8_to_halfraw(page[fp.bs * kE2m1Codes + off * kE2m1Scales + g], __NV_E4M3);
        const float s = __half2float(*reinterpret_cast<const __half*>(&hr)) * fp.kv_scale;
        for (int e = 0; e < 8; ++e) {
          tile[t][g * 16 + 2 * e] = e2m1_f32(codes[e] & 15u) * s;
          tile[t][g * 16 + 2 * e + 1] = e2m1_f32(codes[e] >> 4) * s;
        }
      }
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      float s = 0.f;
      for (int k = 0; k < 18; ++k) s = fmaf(q[k], tile[t][lane + 32 * k], s);
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= fp.scale_log2;
      const float mn = fmaxf(m, s);
      const float a = exp2f(m - mn), w = exp2f(s - mn);
      m = mn;
      l = l * a + w;
      for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], a, w * tile[t][lane + 32 * k]);
    }
  }
  if (h >= fp.H) return;
  const int hs = fp.H / fp.head_slices, sl = h / hs;
  const int64_t out = ((static_cast<int64_t>(sl) * fp.B * fp.q_len + static_cast<int64_t>(b) * fp.q_len + i) * fp.P + p) * hs + (h - sl * hs);
  const float inv = hi > lo ? 1.f / l : 0.f;
  for (int k = 0; k < 16; ++k) {
    const float v = o[k] * inv;
    const int64_t e = out * 512 + lane + 32 * k;
    if (fp.part_dtype == kFP32) static_cast<float*>(fp.o_part)[e] = v;
    else static_cast<uint16_t*>(fp.o_part)[e] = static_cast<uint16_t>(pack2_dt(v, 0.f, fp.part_dtype) & 0xFFFFu);
  }
  if (lane == 0) fp.lse_part[out] = hi > lo ? (m + log2f(l)) * kLn2 : -INFINITY;
}

int launch_partial_fp4(const Fp4Params& fp, bool bf16, cudaStream_t stream) {
  const dim3 grid(fp.B * fp.q_len * fp.P, (fp.H + 7) / 8);
  if (bf16) mla_partial_fp4_kernel<true><<<grid, 256, 0, stream>>>(fp);
  else mla_partial_fp4_kernel<false><<<grid, 256, 0, stream>>>(fp);
  return 0;
}

}  // namespace mla
