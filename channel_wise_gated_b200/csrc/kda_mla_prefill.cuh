// Latent attention, expanded form: causal softmax attention of packed sequences with 192 key
// values per head (128 expanded from the latent, 64 shared by the heads) and 128 value channels.
//
//     s_ij = scale (q_i[0:128] . k_j + q_i[128:192] . ks_j),   o_i = sum_j softmax_j(s_i) v_j
//
// Bound: 2 (192 + 128) flops per (query, key, head) pair on the tensor cores; keys and values are
// re-read from L2 once per 256 queries.
//
// One CTA takes 256 queries of one head as two tiles A and B of 128, so that one tile's softmax
// runs while the other's products do. Warps 0-3 and 4-7 hold the softmax of A and B (thread =
// query row, so row maxima and sums need no exchange), warp 8 issues the copies, warp 9 the
// products. Tensor memory holds S_A, S_B (128 x 128 fp32 each) and O_A, O_B; the weights P (bf16)
// overwrite the first half of their S and are the A operand of P V from there. Keys are double-
// buffered in shared memory, values single: 96 + 96 + 32 KiB.
//
// The running reference m of a row's exponents moves only when its maximum has grown by more
// than 8 (in powers of two): until then weights up to 2^8 are exact in the same bf16 relative
// precision and the accumulators need no pass of their own. Maxima, sums and O are fp32; P is
// rounded to bf16 once (half a step, 2^-8 relative per weight) as the matrix units take it.
#pragma once

#include "kda_common.cuh"
#include "kda_mla_append.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace mla {

// Bounded wait of a whole warp (the same answer in every lane): false once the wait runs out
// (2 s) or another role has given up. `one` is the same for a single thread.
struct Waiter {
  volatile int* abort_flag;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, one(bar, parity));
  }
  __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
    return sm100::mbar_try_wait(bar, parity) || slow(bar, parity);
  }
  __device__ __forceinline__ bool slow(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = sm100::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      if (sm100::mbar_try_wait(bar, parity)) return true;
      if ((it & 63u) == 0) {
        if (*abort_flag) return false;
        if (sm100::globaltimer_ns() - t0 > 2000000000ull) {
          *abort_flag = 1;
          flag_error(DEVERR_TIMEOUT);
          return false;
        }
      }
    }
  }
};
// On the way out after a timeout: a bounded wait that ignores the abort flag, so that no copy
// or product is left in flight.
__device__ __forceinline__ void settle_bar(uint64_t* bar, uint32_t parity) {
  sm100::mbar_wait(bar, parity, 100000000ull);
}

__device__ __forceinline__ void tma_load_3d(void* dst_smem, const CUtensorMap* map, int32_t x, int32_t y,
                                            int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sm100::smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(sm100::smem_u32(bar))
      : "memory");
}
// True in one lane of a converged warp. Under this predicate, and not under a comparison of the
// lane's number, the compiler issues a product from uniform registers as it stands; the
// comparison cost about 80 cycles of issue per product here.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
constexpr float LOG2E_F = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.f;

namespace pf {

constexpr int BM = 128;             // queries per tile
constexpr int PAIR = 2 * BM;        // queries per CTA
constexpr int BN = 128;             // keys per tile
constexpr int THREADS = 384;        // (warps 10 and 11 idle: registers are split by groups of four)
constexpr uint32_t BLK = 128 * 128; // a 128-row block of 64 bf16 columns, 16 KiB
constexpr uint32_t Q_BYTES = 3 * BLK, K_BYTES = 3 * BLK, V_BYTES = 2 * BLK;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + 2 * K_BYTES;
constexpr uint32_t OFF_BAR = OFF_V + V_BYTES;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;   // (1 KiB to align the base)
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

enum { B_QFULL = 0, B_KFULL = 2, B_KFREE = 4, B_VFULL = 6, B_VFREE, B_SFULL = 8, B_PFULL = 10, B_OFULL = 12, B_DRAIN = 14, N_BARS };
constexpr uint32_t TM_S = 0, TM_O = 256;   // S_A, S_B, O_A, O_B: 128 columns each

constexpr uint32_t IDESC_S = sm100::idesc_bf16(128, 128, 0, 0);
constexpr uint32_t IDESC_PV = sm100::idesc_bf16(128, 128, 0, 1);   // V is read MN-major

struct Args {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int n_seqs, n_heads, tiles;       // tiles: upper bound of the pairs of query tiles, all sequences
  int64_t tq, tk;
  __nv_bfloat16* o;
  float* lse;
  float scale;
  int causal;
};

// Which sequence and which pair of query tiles a CTA's index means: index among the sequences'
// pair counts, found by one warp, 32 sequences a round; a sequence's last (longest) pair first.
__device__ __forceinline__ void locate(const Args& a, int idx, int lane, int& n, int& pair) {
  if (a.cu_q == nullptr) {
    const int cnt = (int)((a.tq + PAIR - 1) / PAIR);
    n = idx < cnt ? 0 : -1;
    pair = cnt - 1 - idx;
    return;
  }
  int base = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
    int cnt = 0;
    if (s0 + lane < a.n_seqs) {
      int64_t b, e;
      seq_bounds(a.cu_q, s0 + lane, a.n_seqs, a.tq, b, e);
      cnt = (int)((e - b + PAIR - 1) / PAIR);
    }
    int upto = cnt;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, idx < base + upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int c = __shfl_sync(0xffffffffu, cnt, l), u = __shfl_sync(0xffffffffu, upto, l);
      n = s0 + l;
      pair = c - 1 - (idx - (base + u - c));
      return;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
  n = -1;
  pair = 0;
}

__global__ void __launch_bounds__(THREADS, 1)
kda_mla_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_ks, const __grid_constant__ CUtensorMap map_v,
                       const Args a) {
  using namespace sm100;
  extern __shared__ unsigned char pf_smem_raw[];
  unsigned char* sm = pf_smem_raw + ((1024u - (smem_u32(pf_smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_seq, s_pair;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.x / a.tiles;
  if (warp == 9) {
    int n, pair;
    locate(a, blockIdx.x % a.tiles, lane, n, pair);
    if (lane == 0) {
      s_seq = n;
      s_pair = pair;
      s_abort = 0;
      for (int i = 0; i < N_BARS; ++i) mbar_init(&bars[i], i == B_PFULL || i == B_PFULL + 1 ? BM : 1);
      fence_mbar_init();
    }
  }
  __syncthreads();
  const int seq = s_seq;
  if (seq < 0) return;   // (the bound on the pairs counts up to one more per sequence)
  int64_t bq, eq, bk, ek;
  seq_bounds(a.cu_q, seq, a.n_seqs, a.tq, bq, eq);
  seq_bounds(a.cu_k, seq, a.n_seqs, a.tk, bk, ek);
  const int len_q = (int)(eq - bq), len_k = (int)(ek - bk), off = len_k - len_q;
  // keys that a tile's rows see, and the key tiles that makes
  int kend[2], nt[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r0 = s_pair * PAIR + x * BM, rows = min(BM, len_q - r0);
    const int e = a.causal ? min(len_k, r0 + rows + off) : len_k;
    kend[x] = rows > 0 && e > 0 ? e : 0;
    nt[x] = (kend[x] + BN - 1) / BN;
  }
  const int n_tiles = max(nt[0], nt[1]);
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
    if (lane == 0 && n_tiles > 0) {
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_ks);
      prefetch_tensormap(&map_v);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Waiter wait{&s_abort};

  // A softmax thread holds a row of S (128 registers): the launch's 3 x 168 registers per
  // thread of the three warpgroups are split 208 + 208 + 88.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
    // ---- copies ----
    if (lane == 0 && n_tiles > 0) {
      int k_issued = 0, v_issued = 0;
      bool alive = true;
      auto issue_k = [&](int j) {
        uint64_t* full = &bars[B_KFULL + (j & 1)];
        unsigned char* dst = sm + OFF_K + (j & 1) * K_BYTES;
        const int y = (int)(bk + (int64_t)j * BN);
        mbar_arrive_expect_tx(full, K_BYTES);
        tma_load_3d(dst, &map_k, 0, head, y, full);
        tma_load_3d(dst + BLK, &map_k, 64, head, y, full);
        tma_load_2d(dst + 2 * BLK, &map_ks, 0, y, full);
        ++k_issued;
      };
      for (int x = 0; x < 2; ++x) {
        if (nt[x] > 0) {
          const int y = (int)(bq + s_pair * PAIR + x * BM);
          mbar_arrive_expect_tx(&bars[B_QFULL + x], Q_BYTES);
          for (int b = 0; b < 3; ++b)
            tma_load_3d(sm + OFF_Q + x * Q_BYTES + b * BLK, &map_q, 64 * b, head, y, &bars[B_QFULL + x]);
        }
        if (x == 0) issue_k(0);
      }
      if (n_tiles > 1) issue_k(1);
      for (int j = 0; j < n_tiles && alive; ++j) {
        if (j >= 1) alive = wait.one(&bars[B_VFREE], (j - 1) & 1);
        if (!alive) break;
        mbar_arrive_expect_tx(&bars[B_VFULL], V_BYTES);
        const int y = (int)(bk + (int64_t)j * BN);
        tma_load_3d(sm + OFF_V, &map_v, 0, head, y, &bars[B_VFULL]);
        tma_load_3d(sm + OFF_V + BLK, &map_v, 64, head, y, &bars[B_VFULL]);
        ++v_issued;
        if (j + 2 < n_tiles) {
          alive = wait.one(&bars[B_KFREE + (j & 1)], (j >> 1) & 1);
          if (alive) issue_k(j + 2);
        }
      }
      if (!alive) {
        for (int x = 0; x < 2; ++x)
          if (nt[x] > 0) settle_bar(&bars[B_QFULL + x], 0);
        for (int j = max(0, k_issued - 2); j < k_issued; ++j) settle_bar(&bars[B_KFULL + (j & 1)], (j >> 1) & 1);
        if (v_issued > 0) settle_bar(&bars[B_VFULL], (v_issued - 1) & 1);
      }
    }
    } else if (warp == 9) {
    // ---- products ----
    const uint32_t sb = smem_u32(sm);
    const uint64_t v0 = make_sdesc(sb + OFF_V, BLK, 1024, SWZ_128B);
    bool alive = n_tiles > 0;
    auto issue_s = [&](int x, int j) {   // S_x = Q_x K_j^T
      tc_fence_after();
      if (elect_one()) {
        const uint64_t q0 = make_sdesc(sb + OFF_Q + x * Q_BYTES, 16, 1024, SWZ_128B);
        const uint64_t k0 = make_sdesc(sb + OFF_K + (j & 1) * K_BYTES, 16, 1024, SWZ_128B);
#pragma unroll
        for (int kk = 0; kk < 12; ++kk) {
          const uint32_t at = ((kk >> 2) * BLK + (kk & 3) * 32) >> 4;
          umma_bf16(tmem + TM_S + x * 128, q0 + at, k0 + at, IDESC_S, kk > 0 ? 1u : 0u);
        }
        umma_commit(&bars[B_SFULL + x]);
      }
    };
    alive = alive && wait(&bars[B_KFULL], 0);
    for (int x = 0; x < 2; ++x)
      if (nt[x] > 0) {
        alive = alive && wait(&bars[B_QFULL + x], 0);
        if (alive) issue_s(x, 0);
      }
    if (alive && elect_one()) umma_commit(&bars[B_KFREE]);
    for (int j = 0; j < n_tiles && alive; ++j) {
      if (!(alive = wait(&bars[B_VFULL], j & 1))) break;
      const int valid = len_k - j * BN;
      if (valid < BN && (valid & 15)) {
        // rows behind the sequence's last key inside its 16-row step: whatever the copy
        // brought (the next sequence's values), their weights of zero must meet zeros
        const int r1 = (valid + 15) & ~15;
        for (int i = lane; i < (r1 - valid) * 16; i += 32) {
          const int r = valid + (i >> 4), b = (i >> 3) & 1, c = i & 7;
          *reinterpret_cast<uint4*>(sm + OFF_V + b * BLK + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      bool have_k = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j >= nt[x]) continue;
        if (!(alive = alive && wait(&bars[B_PFULL + x], j & 1))) break;
        tc_fence_after();
        const int steps = min(8, (kend[x] - j * BN + 15) >> 4);
        if (elect_one()) {
          for (int kk = 0; kk < steps; ++kk)
            umma_bf16_tmem_a(tmem + TM_O + x * 128, tmem + TM_S + x * 128 + kk * 8, v0 + ((kk * 2048) >> 4),
                             IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
          if (j + 1 == nt[x]) umma_commit(&bars[B_OFULL + x]);
        }
        if (j + 1 < nt[x]) {
          if (!have_k) alive = wait(&bars[B_KFULL + ((j + 1) & 1)], ((j + 1) >> 1) & 1);
          have_k = true;
          if (!alive) break;
          // S_x(j+1) overwrites P_x(j): products of one thread run in the order of issue
          issue_s(x, j + 1);
        }
      }
      if (alive && elect_one()) {
        umma_commit(&bars[B_VFREE]);
        if (j + 1 < n_tiles) umma_commit(&bars[B_KFREE + ((j + 1) & 1)]);
      }
    }
    if (n_tiles > 0 && !alive && elect_one()) {
      umma_commit(&bars[B_DRAIN]);
      settle_bar(&bars[B_DRAIN], 0);
    }
    __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax: thread = query row ----
    const int x = warp >> 2;
    const int row = s_pair * PAIR + x * BM + (tid & 127);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + TM_S + x * 128 + lane_base, t_o = tmem + TM_O + x * 128 + lane_base;
    const float sc = a.scale * LOG2E_F;
    const int see = a.causal ? min(len_k, row + off + 1) : len_k;   // keys this row sees
    const int n_x = nt[x];
    float m = -INFINITY, l = 0.f;
    bool alive = true;
    for (int j = 0; j < n_x; ++j) {
      if (!(alive = wait(&bars[B_SFULL + x], j & 1))) break;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
      tmem_ld_wait();
      const int lim = see - j * BN;
      if (__any_sync(0xffffffffu, lim < BN)) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= lim) s[c] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = mt;
      } else {
        const bool move = mt > m && (mt - m) * sc > RESCALE_LOG2;   // (from -inf: always)
        if (__any_sync(0xffffffffu, move)) {
          // (P V of the tile before has completed: it was issued before the S waited for)
          const float f = move ? exp2_fast((m - mt) * sc) : 1.f;
          if (move) m = mt;
          l *= f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(t_o + 32 * c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= f;
            tmem_st32(t_o + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&v));
          }
          tmem_st_wait();
        }
      }
      const float ms = m == -INFINITY ? 0.f : m * sc;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 128; c += 64) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const float e0 = exp2_fast(fmaf(s[c + i], sc, -ms)), e1 = exp2_fast(fmaf(s[c + i + 1], sc, -ms));
          sum[i & 3] += e0;
          sum[(i & 3) + 1] += e1;
          p[i >> 1] = pack2(e0, e1);
        }
        tmem_st32(t_s + (c >> 1), p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars[B_PFULL + x]);
    }
    if (n_x > 0 && alive) {
      alive = wait(&bars[B_OFULL + x], 0);
      tc_fence_after();
    }
    if (alive) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      __nv_bfloat16* od = a.o + ((bq + row) * a.n_heads + head) * D;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v[32];
        if (n_x > 0) {
          tmem_ld32(t_o + 32 * c, v);
          tmem_ld_wait();
        }
        if (row < len_q) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (l != 0.f)
              w = make_uint4(pack2(v[i] * inv, v[i + 1] * inv), pack2(v[i + 2] * inv, v[i + 3] * inv),
                             pack2(v[i + 4] * inv, v[i + 5] * inv), pack2(v[i + 6] * inv, v[i + 7] * inv));
            *reinterpret_cast<uint4*>(od + 32 * c + i) = w;
          }
        }
      }
      if (a.lse != nullptr && row < len_q)
        a.lse[(bq + row) * a.n_heads + head] =
            l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * a.scale) + logf(l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace pf
}  // namespace mla
}  // namespace kda
