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
// bytes of the in-place step: HBM.
//
// The 2 t rows k_r e^G, q_r e^G times the state are one product of 16 (32 past 8 tokens) x 128 x
// 128. On the fp32 units, rows in registers as the multi-token step has them, it took 2,150
// instructions a warp and 267 us for 256 x 32 states and 8 tokens (FMA pipe 34 % busy, the rest
// of the issue spent on pairing operands and summing over warps). So it runs on the warp-level
// tensor cores with every fp32 operand split in two, a = a1 + a2, and a b = a1 b1 + a1 b2 + a2 b1.
// For fp32 inputs the parts are tf32: the products left out and the parts' own roundings are at most
// 3 2^-22 of |a b|, the accuracy of fp32 sums. For bf16 inputs they are bf16, at most 3 2^-16 of |a b|
// (of the state too, although that is fp32), against an output rounded by 2^-8 of its value: fewer
// bits than decode_tokens keeps, which show where a sum cancels to 2^-8 of its terms. That halves
// the products. A warp takes 8 columns and the whole depth, so no sums cross warps.
//
// Two persistent CTAs of 512 threads per SM walk the states (a chain of short dependent steps
// per state: with 256 threads it took 223 us). A state comes into shared memory by four TMA boxes
// of 32 columns with 128-byte swizzle: the k index of a product's step runs over eight rows as 0
// 2 4 6 | 1 3 5 7, which makes the fragments' reads free of bank conflicts. The next state's
// inputs come through registers meanwhile. 256 x 32 states, 8 tokens: 157 to 162 us, 3.8 to 4.0
// TB/s, 0.59 to 0.61 of the measured copy rate; issue is 54 % busy, shared memory's pipe 61 %, the rest is barriers.
#pragma once

#include "kda_common.cuh"
#include "kda_decode.cuh"
#include "kda_sm100.cuh"

#include <type_traits>

namespace kda {

constexpr int TREE_MAX_TOKENS = 16;
constexpr int TREE_THREADS = 512;
constexpr int TREE_XS = D + 8;    // row stride of the x rows (fp32, or bf16 parts): fragment reads of 8 rows hit 32 banks
constexpr int TREE_US = D + 16;   // and of the products' rows

// Rows of the product: the k rows of all tokens, then the q rows, 8 or 16 each.
__host__ __device__ constexpr int tree_rows(int t) { return t <= 8 ? 16 : 32; }
// Shared memory: the state's buffer and its barrier; region 0: k, q and log2 alpha rows in fp32,
// then the products; x rows; v rows as stored; A, P, beta, bits.
__host__ __device__ constexpr size_t tree_region0(int t) {
  const size_t in = (size_t)3 * t * D * sizeof(float), out = (size_t)tree_rows(t) * TREE_US * sizeof(float);
  return in > out ? in : out;
}
constexpr size_t TREE_BAR = 128;
__host__ __device__ constexpr size_t tree_smem_bytes(int t, size_t q_bytes) {
  return 1024 + DEC_STATE_BYTES + TREE_BAR + tree_region0(t) + (size_t)tree_rows(t) * TREE_XS * sizeof(float) +
         (size_t)t * D * q_bytes + (2 * TREE_MAX_TOKENS * TREE_MAX_TOKENS + TREE_MAX_TOKENS) * sizeof(float) +
         2 * TREE_MAX_TOKENS * sizeof(int);
}

template <typename T>
__device__ __forceinline__ void piece_to_f32(uint4 raw, float* dst, float by = 1.f) {   // 16 bytes of T as fp32
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(__uint_as_float(raw.x) * by, __uint_as_float(raw.y) * by,
                                                  __uint_as_float(raw.z) * by, __uint_as_float(raw.w) * by);
  } else {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16) * by;
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u) * by;
    }
    reinterpret_cast<float4*>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// a = a1 + a2 + (at most 2^-22 |a|), both parts in tf32
__device__ __forceinline__ void split_tf32(float a, uint32_t& a1, uint32_t& a2) {
  a1 = sm100::f2tf32(a);
  a2 = sm100::f2tf32(a - __uint_as_float(a1));
}

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Four 8x8 b16 matrices from the rows that threads 8m .. 8m+7 address: matrix m to register m, row
// t / 4, columns 2(t % 4) and one further.
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Warp-level bf16 MMA m16n8k16 (fp32 accumulate). Fragments (g = lane / 4, t = lane % 4), pairs of k:
//   A 16x16: a0 = A[g][2t..], a1 = A[g+8][2t..], a2 = A[g][2t+8..], a3 = A[g+8][2t+8..]
//   B 16x8:  b0 = B[2t..][g], b1 = B[2t+8..][g];  C as the tf32 product's
__device__ __forceinline__ void mma_bf16_16x8x16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// MAXT, 8 or 16: a bound on n_tokens
template <typename TQ, typename TG, int MAXT>
__global__ void __launch_bounds__(TREE_THREADS, 2)
kda_decode_tree_kernel(const __grid_constant__ CUtensorMap map_s, const TQ* __restrict__ q, const TQ* __restrict__ k, const TQ* __restrict__ v,
                       const TG* __restrict__ log_alpha, const TG* __restrict__ beta,
                       const int32_t* __restrict__ tree, TQ* __restrict__ o, int n_heads,
                       int n_tokens, int n_chains) {
  using namespace sm100;
  constexpr int MT = MAXT / 8;   // tiles of 16 product rows
  constexpr bool BF = sizeof(TQ) == 2;   // operands split into bf16 parts, else tf32
  extern __shared__ unsigned char tree_smem_raw[];
  unsigned char* sm = tree_smem_raw + ((1024u - (smem_u32(tree_smem_raw) & 1023u)) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + DEC_STATE_BYTES);
  float* s_k = reinterpret_cast<float*>(sm + DEC_STATE_BYTES + TREE_BAR);
  float* s_q = s_k + n_tokens * D;
  float* s_g = s_q + n_tokens * D;
  float* s_u = s_k;                                             // [row][TREE_US]
  float* s_x = s_k + tree_region0(n_tokens) / sizeof(float);    // [row][TREE_XS], or as bf16 parts:
  __nv_bfloat16* s_x1 = reinterpret_cast<__nv_bfloat16*>(s_x);
  __nv_bfloat16* s_x2 = s_x1 + 16 * MT * TREE_XS;
  TQ* s_v = reinterpret_cast<TQ*>(s_x + tree_rows(n_tokens) * TREE_XS);
  float* s_A = reinterpret_cast<float*>(s_v + n_tokens * D);    // [16][16]
  float* s_P = s_A + TREE_MAX_TOKENS * TREE_MAX_TOKENS;
  float* s_beta = s_P + TREE_MAX_TOKENS * TREE_MAX_TOKENS;
  int* s_anc = reinterpret_cast<int*>(s_beta + TREE_MAX_TOKENS); // ancestors and itself, as bits
  int* s_par = s_anc + TREE_MAX_TOKENS;
  constexpr float LOG2E = 1.4426950408889634f;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;   // the fragments' group and thread in it

  // Inputs of a chain in 16-byte pieces: k, q, v rows of QP pieces, then log alpha rows of GP, each
  // tensor with room for MAXT rows (so that a piece's place takes no division).
  constexpr int QP = D * sizeof(TQ) / 16, GP = D * sizeof(TG) / 16, NQ = MAXT * QP;
  constexpr int PRE = (3 * NQ + MAXT * GP + TREE_THREADS - 1) / TREE_THREADS;
  uint4 pre[PRE];
  TG beta_next = from_f32<TG>(0.f);   // (as stored: a conversion would wait for the load)
  uint32_t bits_next = 0;
  auto prefetch = [&](int ch) {
    const int seq = ch / n_heads, h = ch - seq * n_heads;
    const size_t first = (size_t)seq * n_tokens * n_heads + h;   // token 0's row; a token further: + n_heads
#pragma unroll
    for (int j = 0; j < PRE; ++j) {
      const int i = tid + j * TREE_THREADS;
      if (i < 3 * NQ) {
        const int which = i / NQ, t = (i % NQ) / QP, piece = i % QP;
        const TQ* src = (which == 0 ? k : which == 1 ? q : v) + (first + (size_t)t * n_heads) * D;
        if (t < n_tokens) pre[j] = __ldg(reinterpret_cast<const uint4*>(src) + piece);
      } else {
        const int t = (i - 3 * NQ) / GP, piece = (i - 3 * NQ) % GP;
        if (t < n_tokens)
          pre[j] = __ldg(reinterpret_cast<const uint4*>(log_alpha + (first + (size_t)t * n_heads) * D) + piece);
      }
    }
    if (tid < n_tokens) {
      beta_next = beta[first + (size_t)tid * n_heads];
      bits_next = tree ? (uint32_t)tree[(size_t)seq * n_tokens + tid] : (2u << tid) - 1u;
    }
  };

  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  for (int i = tid; i < 16 * MT * TREE_XS; i += TREE_THREADS) s_x[i] = 0.f;   // (rows of no token stay zero)
  __syncthreads();
  auto load_state = [&](int ch) {
    mbar_arrive_expect_tx(bar, DEC_STATE_BYTES);
    for (int b = 0; b < 4; ++b) tma_load_2d(sm + b * (DEC_STATE_BYTES / 4), &map_s, 32 * b, ch * D, bar);
  };
  int chain = blockIdx.x;
  if (tid == 0 && chain < n_chains) load_state(chain);
  if (chain < n_chains) prefetch(chain);
  uint32_t phase = 0;
#pragma unroll 1
  for (; chain < n_chains; chain += gridDim.x) {
    const int seq = chain / n_heads, h = chain - seq * n_heads;
    TQ* od = o + ((size_t)seq * n_tokens * n_heads + h) * D;
    const size_t o_step = (size_t)n_heads * D;
    // inputs to shared memory (the chain before is done with it: its last barrier), then the
    // next chain's loads go out
#pragma unroll
    for (int j = 0; j < PRE; ++j) {
      const int i = tid + j * TREE_THREADS;
      if (i < 3 * NQ) {
        const int which = i / NQ, t = (i % NQ) / QP, piece = i % QP;
        if (t < n_tokens) {
          if (which < 2)
            piece_to_f32<TQ>(pre[j], (which == 0 ? s_k : s_q) + t * D + piece * (D / QP));
          else
            reinterpret_cast<uint4*>(s_v)[t * QP + piece] = pre[j];
        }
      } else {
        const int t = (i - 3 * NQ) / GP, piece = (i - 3 * NQ) % GP;
        if (t < n_tokens) piece_to_f32<TG>(pre[j], s_g + t * D + piece * (D / GP), LOG2E);
      }
    }
    if (warp == 0) {
      // A token's parent is the highest bit below its own; its ancestors are its parent's and its
      // parent. A row that says anything else (its own bit missing, a bit above it, a set that is
      // no path) is taken by its parent alone and flagged.
      const bool here = lane < n_tokens;
      const uint32_t own = 1u << (lane & 31), below = bits_next & (own - 1u);
      const int p = here && below ? 31 - __clz(below) : -1;
      uint32_t anc = bits_next;
      const uint32_t up = __shfl_sync(0xffffffffu, bits_next, p < 0 ? 0 : p);
      if (__any_sync(0xffffffffu, here && bits_next != ((p < 0 ? 0u : up) | own))) {
        anc = own;
        for (int r = 1; r < n_tokens; ++r) {
          const uint32_t a = __shfl_sync(0xffffffffu, anc, p < 0 ? 0 : p);
          if (lane == r && p >= 0) anc = a | own;
        }
        if (lane == 0) flag_error(DEVERR_TREE);
      }
      if (here) {
        s_anc[lane] = (int)anc;
        s_par[lane] = p;
        s_beta[lane] = to_f32(beta_next);
      }
    }
    __syncthreads();
    if (chain + (int)gridDim.x < n_chains) prefetch(chain + gridDim.x);
    // the rows for the product: e^G of the decay summed along the token's path
    for (int r = tid >> 7; r < n_tokens; r += TREE_THREADS / D) {
      const int c = tid & (D - 1);
      float g = 0.f;
      for (int i = r; i >= 0; i = s_par[i]) g += s_g[i * D + c];
      const float e = exp2f(g);
      const float xk = s_k[r * D + c] * e, xq = s_q[r * D + c] * e;
      const int ak = r * TREE_XS + c, aq = (8 * MT + r) * TREE_XS + c;
      if constexpr (BF) {
        s_x1[ak] = __float2bfloat16_rn(xk);
        s_x1[aq] = __float2bfloat16_rn(xq);
        s_x2[ak] = __float2bfloat16_rn(xk - __bfloat162float(s_x1[ak]));
        s_x2[aq] = __float2bfloat16_rn(xq - __bfloat162float(s_x1[aq]));
      } else {
        s_x[ak] = xk;
        s_x[aq] = xq;
      }
    }
    // Pair products: a warp takes a token and walks from it to its root, so that the decay between
    // the two is a sum of its own and not the difference of two long ones.
    static_assert(TREE_THREADS / 32 >= TREE_MAX_TOKENS, "a warp per token");
    if (warp < n_tokens) {
      const int r = warp;
      if (lane < TREE_MAX_TOKENS)   // (0 for what is no ancestor)
        s_A[r * TREE_MAX_TOKENS + lane] = s_P[r * TREE_MAX_TOKENS + lane] = 0.f;
      __syncwarp();
      const float4 kr = reinterpret_cast<const float4*>(s_k + r * D)[lane];
      const float4 qr = reinterpret_cast<const float4*>(s_q + r * D)[lane];
      const float br = s_beta[r];
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int i = r; i >= 0;) {
        const float4 ki = reinterpret_cast<const float4*>(s_k + i * D)[lane];
        const float4 li = reinterpret_cast<const float4*>(s_g + i * D)[lane];
        const float e0 = ki.x * exp2f(g.x), e1 = ki.y * exp2f(g.y), e2 = ki.z * exp2f(g.z), e3 = ki.w * exp2f(g.w);
        float a = fmaf(kr.x, e0, fmaf(kr.y, e1, fmaf(kr.z, e2, kr.w * e3)));
        float p = fmaf(qr.x, e0, fmaf(qr.y, e1, fmaf(qr.z, e2, qr.w * e3)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, off);
          p += __shfl_xor_sync(0xffffffffu, p, off);
        }
        if (lane == 0) {
          s_A[r * TREE_MAX_TOKENS + i] = br * a;
          s_P[r * TREE_MAX_TOKENS + i] = p;
        }
        g = make_float4(g.x + li.x, g.y + li.y, g.z + li.z, g.w + li.w);
        i = s_par[i];
      }
    }
    const bool landed = mbar_wait(bar, phase);
    phase ^= 1u;
    if (!__syncthreads_and(landed)) {   // (and: the x rows are written, the k, q and decay rows read)
      if (tid == 0) {
        flag_error(DEVERR_TIMEOUT);
        mbar_wait(bar, phase ^ 1u, 100000000ull);   // (never leave with the copy in flight)
      }
      break;
    }
    // columns 8w .. 8w+7 of the product (the small products have sums of their own: chains of
    // dependent products a third as long)
    float acc[MT][4], sml[MT][4], sm2[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = sml[m][i] = sm2[m][i] = 0.f;
    {
      const unsigned char* sb = sm + (warp >> 2) * (DEC_STATE_BYTES / 4);
      // The swizzle of a row goes by its number modulo 8, which is 2t or 2t + 1 in every step: two
      // pointers, and the step in the instruction's offset.
      const uint32_t cb = (uint32_t)((8 * (warp & 3) + g8) * sizeof(float));   // byte of the column in its box
      const unsigned char* s_even = sb + swz128((uint32_t)(2 * t4) * 128u + cb);
      const unsigned char* s_odd = sb + swz128((uint32_t)(2 * t4 + 1) * 128u + cb);
      auto s_at = [&](int eight, int odd) {
        return *reinterpret_cast<const float*>((odd ? s_odd : s_even) + eight * 1024);
      };
      if constexpr (BF) {
        // (thread l gives the address of row l % 16 of a fragment's 16 x 16 block, its left or
        // right half)
        const uint32_t x1 = smem_u32(s_x1 + (lane & 15) * TREE_XS + 8 * (lane >> 4));
        const uint32_t x2 = smem_u32(s_x2 + (lane & 15) * TREE_XS + 8 * (lane >> 4));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b1[2], b2[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float lo = s_at(2 * ks + hf, 0), hi = s_at(2 * ks + hf, 1);
            b1[hf] = pack_pair(lo, hi);
            b2[hf] = pack_pair(lo - __uint_as_float(b1[hf] << 16), hi - __uint_as_float(b1[hf] & 0xFFFF0000u));
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t a1[4], a2[4];
            ldmatrix_x4(x1 + (uint32_t)((16 * m * TREE_XS + 16 * ks) * sizeof(__nv_bfloat16)), a1);
            ldmatrix_x4(x2 + (uint32_t)((16 * m * TREE_XS + 16 * ks) * sizeof(__nv_bfloat16)), a2);
            mma_bf16_16x8x16(sml[m], a2, b1);
            mma_bf16_16x8x16(sm2[m], a1, b2);
            mma_bf16_16x8x16(acc[m], a1, b1);
          }
        }
      } else {
#pragma unroll 4
        for (int ks = 0; ks < D / 8; ++ks) {
          uint32_t b1[2], b2[2];
          split_tf32(s_at(ks, 0), b1[0], b2[0]);
          split_tf32(s_at(ks, 1), b1[1], b2[1]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float2 lo = *reinterpret_cast<const float2*>(s_x + (16 * m + g8) * TREE_XS + 8 * ks + 2 * t4);
            const float2 hi = *reinterpret_cast<const float2*>(s_x + (16 * m + 8 + g8) * TREE_XS + 8 * ks + 2 * t4);
            uint32_t a1[4], a2[4];
            split_tf32(lo.x, a1[0], a2[0]);
            split_tf32(hi.x, a1[1], a2[1]);
            split_tf32(lo.y, a1[2], a2[2]);
            split_tf32(hi.y, a1[3], a2[3]);
            mma_tf32_16x8x8(sml[m], a2, b1);
            mma_tf32_16x8x8(sm2[m], a1, b2);
            mma_tf32_16x8x8(acc[m], a1, b1);
          }
        }
      }
    }
    fence_proxy_async_smem();   // (the state's reads come before the next copy into its buffer)
    // the products over the k, q and decay rows, each warp its own columns
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        *reinterpret_cast<float2*>(s_u + (16 * m + 8 * hf + g8) * TREE_US + 8 * warp + 2 * t4) =
            make_float2(acc[m][2 * hf] + (sml[m][2 * hf] + sm2[m][2 * hf]),
                        acc[m][2 * hf + 1] + (sml[m][2 * hf + 1] + sm2[m][2 * hf + 1]));
    __syncthreads();
    if (tid == TREE_THREADS - 32 && chain + (int)gridDim.x < n_chains) load_state(chain + gridDim.x);   // (a warp without columns below)
    // Forward substitution and readout, 16 columns a warp by half of the warps: both groups of lanes
    // form every delta, each reads out every other token. (More lanes to a column only add issue.)
    if (warp < D / 16) {
      const int col = 16 * warp + (lane & 15), par = lane >> 4;
      // A coefficient of 0 takes out what is no ancestor, unless that is NaN or infinite: then the
      // columns go once more, by the bits (another branch's token counts for nothing).
      auto solve = [&](auto by_bits) {
        constexpr bool BITS = decltype(by_bits)::value;
        float dl[MAXT], worst = 0.f;
#pragma unroll
        for (int r = 0; r < MAXT; ++r) {
          dl[r] = 0.f;
          if (r < n_tokens) {
            const uint32_t anc = BITS ? (uint32_t)s_anc[r] : 0u;
            float row[MAXT];
#pragma unroll
            for (int i = 0; i < r; i += 4)
              *reinterpret_cast<float4*>(&row[i]) = *reinterpret_cast<const float4*>(s_A + r * TREE_MAX_TOKENS + i);
            float d = s_beta[r] * (to_f32(s_v[r * D + col]) - s_u[r * TREE_US + col]);
#pragma unroll
            for (int i = 0; i < r; ++i)
              if (!BITS || ((anc >> i) & 1u)) d = fmaf(-row[i], dl[i], d);
            dl[r] = d;
            worst = fmaf(d, 0.f, worst);   // (0, or NaN)
          }
        }
#pragma unroll
        for (int r0 = 0; r0 < MAXT; r0 += 2) {
          const int r = r0 + par;
          if (r < n_tokens) {
            const uint32_t anc = BITS ? (uint32_t)s_anc[r] : 0u;
            float row[MAXT];
#pragma unroll
            for (int i = 0; i < r0 + 2; i += 4)
              *reinterpret_cast<float4*>(&row[i]) = *reinterpret_cast<const float4*>(s_P + r * TREE_MAX_TOKENS + i);
            float y = s_u[(8 * MT + r) * TREE_US + col];
#pragma unroll
            for (int i = 0; i < r0 + 2; ++i)
              if (!BITS || ((anc >> i) & 1u)) y = fmaf(row[i], dl[i], y);
            od[r * o_step + col] = from_f32<TQ>(y);
          }
        }
        return worst;
      };
      if (!(solve(std::false_type()) == 0.f)) solve(std::true_type());
    }
    __syncthreads();   // (the next chain's inputs go where this one's were)
  }
}

template <typename TQ, typename TG, int MAXT>
cudaError_t launch_decode_tree_as(const CUtensorMap& map_s, const TQ* q, const TQ* k, const TQ* v,
                                  const TG* log_alpha, const TG* beta, const int32_t* tree, TQ* o, int n_tokens,
                                  int n_heads, int chains, int sms, int smem_sm, int reserved,
                                  cudaStream_t stream) {
  // (The attribute belongs to the kernel, not to the call: every call sets the same value, the most
  // that any of them needs, so that calls from several host threads do not undo one another's.)
  const cudaError_t e = cudaFuncSetAttribute(kda_decode_tree_kernel<TQ, TG, MAXT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)tree_smem_bytes(MAXT, sizeof(TQ)));
  if (e != cudaSuccess) return e;
  const size_t smem = tree_smem_bytes(n_tokens, sizeof(TQ));
  // (one CTA per SM where two do not fit: fp32 inputs past 14 tokens)
  const int per_sm = 2 * (smem + (size_t)reserved) <= (size_t)smem_sm ? 2 : 1;
  const int grid = chains < per_sm * sms ? chains : per_sm * sms;
  kda_decode_tree_kernel<TQ, TG, MAXT><<<(unsigned)grid, TREE_THREADS, smem, stream>>>(
      map_s, q, k, v, log_alpha, beta, tree, o, n_heads, n_tokens, chains);
  return cudaGetLastError();
}

// map_s: the states as one fp32 matrix of 128 columns in swizzled boxes of 32 columns, 128 rows.
template <typename TQ, typename TG>
cudaError_t launch_decode_tree(const CUtensorMap& map_s, const TQ* q, const TQ* k, const TQ* v,
                               const TG* log_alpha, const TG* beta, const int32_t* tree, TQ* o, int n_seqs,
                               int n_tokens, int n_heads, cudaStream_t stream) {
  int dev = 0, sms = 0, smem_sm = 0, reserved = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  const int chains = n_seqs * n_heads;
  return n_tokens <= 8 ? launch_decode_tree_as<TQ, TG, 8>(map_s, q, k, v, log_alpha, beta, tree, o, n_tokens,
                                                          n_heads, chains, sms, smem_sm, reserved, stream)
                       : launch_decode_tree_as<TQ, TG, 16>(map_s, q, k, v, log_alpha, beta, tree, o, n_tokens,
                                                           n_heads, chains, sms, smem_sm, reserved, stream);
}

}  // namespace kda
