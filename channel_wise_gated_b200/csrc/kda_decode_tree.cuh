// KDA outputs for a tree of drafted tokens per (sequence, head): every token's output under the
// recurrence along its own path from the state, which is read once and left as it is.
//
// Tokens of one path see each other as the tokens of a chunk do, so the chunk form holds with
// "earlier token" replaced by "ancestor". With G_r the sum of log alpha along r's path:
//
//     A_ri = beta_r sum_c k_rc k_ic e^{G_rc - G_ic}     (i a proper ancestor of r)
//     P_ri = sum_c q_rc k_ic e^{G_rc - G_ic}            (i an ancestor of r, or r)
//     delta_r = beta_r (v_r - (k_r * e^{G_r})^T S) - sum_i A_ri delta_i
//     o_r = (q_r * e^{G_r})^T S + sum_i P_ri delta_i
//
// Every exponent is at most 0 (log alpha <= 0 along the path from i to r), so no factor
// overflows however strong the decay.
//
// Bound: 64 KiB of state per (sequence, head) read once and nothing written back, half the
// bytes of the in-place step: HBM up to about 8 tokens, then the 2 t products of 128 x 128 on
// the fp32 units. One CTA of 256 threads per state, as the single step: thread (warp w, lane l)
// holds rows 16w .. 16w+15 of columns 4l .. 4l+3 in registers. The state loads go out first
// and the inputs' staging, the decay sums and the pair products run while they are in flight.
#pragma once

#include "kda_common.cuh"
#include "kda_decode.cuh"

namespace kda {

constexpr int TREE_MAX_TOKENS = 16;
constexpr int TREE_BATCH = 8;   // products with the state reduced over the warps at a time (32 KiB)

// Shared memory in floats: k, q, v and G rows of every token (k and q scaled by e^G in rows of
// their own), A and P, the partial products, and the reduced products.
__host__ __device__ constexpr size_t tree_smem_bytes(int n_tokens) {
  return ((size_t)6 * n_tokens * D + 2 * TREE_MAX_TOKENS * TREE_MAX_TOKENS + TREE_MAX_TOKENS +
          (size_t)TREE_BATCH * (DEC_THREADS / 32) * D + (size_t)2 * n_tokens * D) * sizeof(float) +
         2 * TREE_MAX_TOKENS * sizeof(int);
}

template <typename TQ, typename TG>
__global__ void __launch_bounds__(DEC_THREADS, 2)
kda_decode_tree_kernel(const TQ* __restrict__ q, const TQ* __restrict__ k, const TQ* __restrict__ v,
                       const TG* __restrict__ log_alpha, const TG* __restrict__ beta,
                       const float* __restrict__ state, const int32_t* __restrict__ tree,
                       TQ* __restrict__ o, int n_heads, int n_tokens) {
  extern __shared__ __align__(16) unsigned char tree_smem[];
  float* s_k = reinterpret_cast<float*>(tree_smem);    // [t][D]
  float* s_q = s_k + n_tokens * D;
  float* s_v = s_q + n_tokens * D;
  float* s_g = s_v + n_tokens * D;
  float* s_x = s_g + n_tokens * D;                     // [2t][D]: k e^G rows, then q e^G rows
  float* s_A = s_x + 2 * n_tokens * D;                 // [16][16]
  float* s_P = s_A + TREE_MAX_TOKENS * TREE_MAX_TOKENS;
  float* s_beta = s_P + TREE_MAX_TOKENS * TREE_MAX_TOKENS;
  float* s_part = s_beta + TREE_MAX_TOKENS;            // [batch][warp][D]
  float* s_u = s_part + TREE_BATCH * (DEC_THREADS / 32) * D;   // [2t][D]
  int* s_anc = reinterpret_cast<int*>(s_u + 2 * n_tokens * D); // ancestors and itself, as bits
  int* s_par = s_anc + TREE_MAX_TOKENS;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chain = blockIdx.x;
  const int seq = chain / n_heads, h = chain - seq * n_heads;
  const float4* S = reinterpret_cast<const float4*>(state + (size_t)chain * D * D);
  const int row0 = warp * DEC_ROWS_PER_WARP;
  float4 s[DEC_ROWS_PER_WARP];
#pragma unroll
  for (int i = 0; i < DEC_ROWS_PER_WARP; ++i) s[i] = __ldcs(&S[(row0 + i) * (D / 4) + lane]);

  const size_t first = (size_t)seq * n_tokens * n_heads + h;   // row of token 0; a token further: + n_heads
  for (int i = tid; i < n_tokens * D; i += DEC_THREADS) {
    const int t = i / D, c = i - t * D;
    const size_t at = (first + (size_t)t * n_heads) * D + c;
    s_k[i] = to_f32(k[at]);
    s_q[i] = to_f32(q[at]);
    s_v[i] = to_f32(v[at]);
    s_g[i] = to_f32(log_alpha[at]);
  }
  if (tid < n_tokens) s_beta[tid] = to_f32(beta[first + (size_t)tid * n_heads]);
  if (tid == 0) {
    // A token's parent is the highest bit below its own; its ancestors are its parent's and its
    // parent. A row that says anything else (its own bit missing, a bit above it, a set that is
    // no path) is taken by its parent alone and flagged.
    bool bad = false;
    for (int r = 0; r < n_tokens; ++r) {
      const uint32_t given = tree ? (uint32_t)tree[(size_t)seq * n_tokens + r] : (2u << r) - 1u;
      const uint32_t below = given & ((1u << r) - 1u);
      const int p = below ? 31 - __clz(below) : -1;
      const uint32_t anc = (p >= 0 ? (uint32_t)s_anc[p] : 0u) | (1u << r);
      bad = bad || anc != given;
      s_anc[r] = (int)anc;
      s_par[r] = p;
    }
    if (bad) flag_error(DEVERR_TREE);
  }
  __syncthreads();
  // decay sums along the paths (parents come before their children)
  if (tid < D) {
    for (int r = 0; r < n_tokens; ++r) {
      const int p = s_par[r];
      if (p >= 0) s_g[r * D + tid] += s_g[p * D + tid];
    }
  }
  __syncthreads();
  for (int i = tid; i < n_tokens * D; i += DEC_THREADS) {
    const float e = expf(s_g[i]);
    s_x[i] = s_k[i] * e;
    s_x[n_tokens * D + i] = s_q[i] * e;
  }
  // pair products, one warp per (r, i)
  for (int pr = warp; pr < n_tokens * n_tokens; pr += DEC_THREADS / 32) {
    const int r = pr / n_tokens, i = pr - r * n_tokens;
    if (!((s_anc[r] >> i) & 1)) continue;
    const float4 gr = reinterpret_cast<const float4*>(s_g + r * D)[lane];
    const float4 gi = reinterpret_cast<const float4*>(s_g + i * D)[lane];
    const float4 ki = reinterpret_cast<const float4*>(s_k + i * D)[lane];
    const float4 kr = reinterpret_cast<const float4*>(s_k + r * D)[lane];
    const float4 qr = reinterpret_cast<const float4*>(s_q + r * D)[lane];
    const float e0 = ki.x * expf(gr.x - gi.x), e1 = ki.y * expf(gr.y - gi.y);
    const float e2 = ki.z * expf(gr.z - gi.z), e3 = ki.w * expf(gr.w - gi.w);
    float a = fmaf(kr.x, e0, fmaf(kr.y, e1, fmaf(kr.z, e2, kr.w * e3)));
    float p = fmaf(qr.x, e0, fmaf(qr.y, e1, fmaf(qr.z, e2, qr.w * e3)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, off);
      p += __shfl_xor_sync(0xffffffffu, p, off);
    }
    if (lane == 0) {
      s_A[r * TREE_MAX_TOKENS + i] = s_beta[r] * a;
      s_P[r * TREE_MAX_TOKENS + i] = p;
    }
  }
  __syncthreads();
  // products of the 2t scaled rows with the state, TREE_BATCH at a time
  for (int x0 = 0; x0 < 2 * n_tokens; x0 += TREE_BATCH) {
    const int nx = min(TREE_BATCH, 2 * n_tokens - x0);
    for (int x = 0; x < nx; ++x) {
      const float* xs = s_x + (x0 + x) * D + row0;
      float2 u0 = make_float2(0.f, 0.f), u1 = u0;
#pragma unroll
      for (int i4 = 0; i4 < DEC_ROWS_PER_WARP; i4 += 4) {
        const float4 x4 = *reinterpret_cast<const float4*>(xs + i4);
        const float xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x2 = make_float2(xv[e], xv[e]);
          u0 = __ffma2_rn(x2, make_float2(s[i4 + e].x, s[i4 + e].y), u0);
          u1 = __ffma2_rn(x2, make_float2(s[i4 + e].z, s[i4 + e].w), u1);
        }
      }
      reinterpret_cast<float4*>(s_part + (x * (DEC_THREADS / 32) + warp) * D)[lane] =
          make_float4(u0.x, u0.y, u1.x, u1.y);
    }
    __syncthreads();
    for (int i = tid; i < nx * D; i += DEC_THREADS) {
      const float* p = s_part + (i / D) * (DEC_THREADS / 32) * D + (i & (D - 1));
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < DEC_THREADS / 32; ++w) sum += p[w * D];
      s_u[x0 * D + i] = sum;
    }
    __syncthreads();
  }
  // forward substitution and the readout, one column per thread
  if (tid < D) {
    float dl[TREE_MAX_TOKENS];
#pragma unroll
    for (int r = 0; r < TREE_MAX_TOKENS; ++r) {
      if (r < n_tokens) {
        const int anc = s_anc[r];
        float d = s_beta[r] * (s_v[r * D + tid] - s_u[r * D + tid]);
        float y = s_u[(n_tokens + r) * D + tid];
#pragma unroll
        for (int i = 0; i < r; ++i)
          if ((anc >> i) & 1) {
            d = fmaf(-s_A[r * TREE_MAX_TOKENS + i], dl[i], d);
            y = fmaf(s_P[r * TREE_MAX_TOKENS + i], dl[i], y);
          }
        dl[r] = d;
        o[(first + (size_t)r * n_heads) * D + tid] = from_f32<TQ>(fmaf(s_P[r * TREE_MAX_TOKENS + r], d, y));
      }
    }
  }
}

template <typename TQ, typename TG>
cudaError_t launch_decode_tree(const TQ* q, const TQ* k, const TQ* v, const TG* log_alpha, const TG* beta,
                               const float* state, const int32_t* tree, TQ* o, int n_seqs, int n_tokens,
                               int n_heads, cudaStream_t stream) {
  const size_t smem = tree_smem_bytes(n_tokens);
  cudaError_t e = cudaFuncSetAttribute(kda_decode_tree_kernel<TQ, TG>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)tree_smem_bytes(TREE_MAX_TOKENS));
  if (e != cudaSuccess) return e;
  kda_decode_tree_kernel<TQ, TG><<<(unsigned)(n_seqs * n_heads), DEC_THREADS, smem, stream>>>(
      q, k, v, log_alpha, beta, state, tree, o, n_heads, n_tokens);
  return cudaGetLastError();
}

}  // namespace kda
