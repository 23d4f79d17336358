// Latent cache append: the RMSNorm of a token's 512 latent values and the write of its 576
// cached values (latent and shared key part) into the page that holds its position.
//
//     y = x[0:512] / sqrt(mean(x[0:512]^2) + eps) * w,   row = [y, x[512:576]]
//
// Bound: 1,152 bytes read and 1,152 written per token (1,024 more with the latent output),
// no reuse, so HBM for long batches and launch latency for a few tokens. One warp per token:
// each lane takes two 16-byte pieces of the latent, the sum of squares is one warp reduction,
// and the row is written as it was read, so every access is a full 512-byte line run. 63,657
// tokens with the latent output (212 MB): 41.2 to 41.8 us, 5.1 TB/s, 0.79 of the measured copy rate
// (more warps, or the next row's loads ahead of the present row's work, were 8 to 20 % slower).
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace mla {

constexpr int LATENT = 512;              // latent values per token (keys and values of all heads)
constexpr int SHARED_K = 64;             // key values every head shares as they are
constexpr int WIDTH = LATENT + SHARED_K; // values cached per token

constexpr int APPEND_THREADS = 256;

// The sequence that owns `token`: the number of ends cu[1..n_seqs] at or below it, found by the
// whole warp in steps of 32 (one round up to 32 sequences, two up to 1,024). For a bad
// cu_seqlens the result is some index in range; the caller checks the bounds it gives.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int n_seqs,
                                             int64_t token, int lane) {
  int lo = 0, span = n_seqs;   // the answer lies in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32;
    const int end = lo + (lane + 1) * step;   // lane's block is [lo + lane step, end)
    const bool past = end >= lo + span || (int64_t)cu[end] > token;
    const unsigned b = __ballot_sync(0xffffffffu, past);
    const int first = __ffs(b) - 1;           // (lane 31's block always reaches the end)
    lo += first * step;
    const int left = span - first * step;
    span = left < step ? left : step;
  }
  return lo;
}

// sum of the squares of eight bf16 values, each first multiplied by `by`
__device__ __forceinline__ float sumsq8(uint4 v, float by) {
  float s = 0.f;
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(u[i] << 16) * by, b = __uint_as_float(u[i] & 0xFFFF0000u) * by;
    s = fmaf(a, a, fmaf(b, b, s));
  }
  return s;
}
// eight bf16 values times `by` (a power of two), r and their weights
__device__ __forceinline__ uint4 scale8(uint4 v, float by, float r, const float (&w)[8]) {
  uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(u[i] << 16) * by * r * w[2 * i];
    const float b = __uint_as_float(u[i] & 0xFFFF0000u) * by * r * w[2 * i + 1];
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}
// Rows whose squares leave fp32: at 2^80 or 2^-70 of their size, where they do not. Below 2^-100 a
// sum of squares loses bits to subnormals (up to 2^-150 of it per product), which counts unless
// eps is above 2^-120; past 2^128 it is infinite (bf16 holds values from 2^-133 to 2^128).
constexpr float SUM_LEAST = 7.888609052210118e-31f;    // 2^-100
constexpr float EPS_LEAST = 7.52316384526264e-37f;     // 2^-120
constexpr float BY_SMALL = 1.2089258196146292e24f;     // 2^80
constexpr float BY_LARGE = 8.470329472543003e-22f;     // 2^-70

__global__ void __launch_bounds__(APPEND_THREADS)
kda_mla_append_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride,
                      const float* __restrict__ norm_w, float eps, __nv_bfloat16* __restrict__ cache,
                      int64_t n_pages, int page_size, const int32_t* __restrict__ page_table,
                      int max_pages, const int32_t* __restrict__ cache_lens,
                      const int32_t* __restrict__ cu, int n_seqs, int64_t t_total,
                      __nv_bfloat16* __restrict__ latent) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (APPEND_THREADS / 32);
  float w0[8], w1[8];   // this lane's weights: latent channels 8 lane .. + 7 and 256 further
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w0[i] = norm_w ? norm_w[8 * lane + i] : 1.f;
    w1[i] = norm_w ? norm_w[256 + 8 * lane + i] : 1.f;
  }
  const int64_t per = cu ? 0 : t_total / n_seqs;   // equal runs without cu_seqlens
  for (int64_t t = (int64_t)blockIdx.x * (APPEND_THREADS / 32) + (threadIdx.x >> 5); t < t_total; t += warps) {
    const uint4* src = reinterpret_cast<const uint4*>(x + t * x_stride);
    uint4 a = src[lane], b = src[32 + lane], c = make_uint4(0, 0, 0, 0);
    if (lane < 8) c = src[64 + lane];
    // where the row goes: position len - (tokens of the sequence from t on)
    int n;
    int64_t bos, eos;
    bool ok = true;
    if (cu) {
      n = find_sequence(cu, n_seqs, t, lane);
      seq_bounds(cu, n, n_seqs, t_total, bos, eos);
      ok = t >= bos && t < eos;
      if (!ok && lane == 0) flag_error(DEVERR_SEQLENS);
    } else {
      n = (int)(t / per);
      eos = (n + 1) * per;
    }
    const int64_t pos = (int64_t)cache_lens[n] - (eos - t);
    int page = -1;
    if (ok) {
      const int64_t pi = pos / page_size;
      if (pos >= 0 && pi < max_pages) page = page_table[(int64_t)n * max_pages + pi];
      if ((page < 0 || page >= n_pages)) {
        page = -1;
        if (lane == 0) flag_error(DEVERR_PAGE);
      }
    }
    if (norm_w) {
      float s = warp_sum(sumsq8(a, 1.f) + sumsq8(b, 1.f));
      if (s < INFINITY && (s >= SUM_LEAST || eps >= EPS_LEAST)) {
        const float r = 1.f / sqrtf(s * (1.f / LATENT) + eps);
        a = scale8(a, 1.f, r, w0);
        b = scale8(b, 1.f, r, w1);
      } else {
        const float by = s < INFINITY ? BY_SMALL : BY_LARGE;   // (2^160 eps stays below 2^40)
        s = warp_sum(sumsq8(a, by) + sumsq8(b, by));
        const float r = 1.f / sqrtf(fmaf(eps * by, by, s * (1.f / LATENT)));
        a = scale8(a, by, r, w0);
        b = scale8(b, by, r, w1);
      }
    }
    if (page >= 0) {
      uint4* dst = reinterpret_cast<uint4*>(cache + ((int64_t)page * page_size + pos % page_size) * WIDTH);
      dst[lane] = a;
      dst[32 + lane] = b;
      if (lane < 8) dst[64 + lane] = c;
    }
    if (latent && ok) {   // (rows of no sequence are left as they are)
      uint4* dst = reinterpret_cast<uint4*>(latent + t * LATENT);
      dst[lane] = a;
      dst[32 + lane] = b;
    }
  }
}

}  // namespace mla
}  // namespace kda
