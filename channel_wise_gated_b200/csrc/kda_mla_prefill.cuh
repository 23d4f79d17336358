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
// query row, so row maxima and sums need no exchange), warps 8 and 11 issue the copies, warps 9 and
// 10 the products of A and B. Tensor memory holds S_A, S_B (128 x 128 fp32 each) and O_A, O_B; the
// weights P (bf16) overwrite the first half of their S and are the A operand of P V from there.
// Queries take 96 KiB of shared memory; keys and values share a ring of eight 16 KiB slots, freed
// one by one.
//
// The running reference m of a row's exponents moves only when its maximum has grown by more
// than 8 (in powers of two): until then weights up to 2^8 have the same relative precision in
// bf16 and the accumulators need no pass of their own. Maxima, sums and O are fp32; P is rounded
// to bf16 once (half a step, 2^-8 relative per weight) as the matrix units take it.
//
// Measured, by clock: 4,096 tokens, 32 heads in 164 to 193 us (1.05 to 0.89 PFLOP/s), 32,768 tokens,
// 4 heads in 1.15 to 1.25 ms (1.19 to 1.10): 0.64 to 0.54 and 0.73 to 0.67 of the measured bf16 rate
// (0.85 to 0.78 of its sustained one for the latter). A pair of key tiles takes about 4,100 cycles
// where its products need 2,680: both tiles' chains (S, softmax of 2,000 cycles, P V) run nearly in
// step, so that the tensor cores and the softmax's units are busy half of the time each and
// mostly not together.
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
constexpr int LATE_START = 40;      // key tiles from which on tile B starts behind A
constexpr int BN = 128;             // keys per tile
// Key tiles after which a row's accumulators are taken out and begin anew, in calls that can have
// more (PARTS): the matrix units cut each sum to fp32 instead of rounding it, and 65,536 of them
// in a row (1,048,576 keys) lost 0.6 % of values of one sign, more than the output's rounding. 4,096
// lose 0.05 % at most, and the parts are added with rounding. In every call it would cost 1 to 2 %
// (190 against 188 us for 4,096 tokens and 32 heads, 1,253 against 1,226 for 32,768 and 4: the
// loop's registers). Where a call has more keys: 64 prompts of 1,100 (none of them long), 8 heads 424
// against 416 us; 1,024 tokens behind 130,048, 4 heads 2,252 against 2,405.
constexpr int FOLD = 512;
constexpr int THREADS = 384;
constexpr uint32_t BLK = 128 * 128; // 16 KiB: a 128-row block of 64 bf16 columns
constexpr uint32_t Q_BYTES = 3 * BLK;
constexpr int SLOTS = 8;            // keys and values pass through a ring of 16 KiB slots: a tile's
constexpr int PER_TILE = 5;         // keys in three (64 columns each), its values in two (64 rows each)
constexpr uint32_t OFF_Q = 0, OFF_RING = 2 * Q_BYTES;
constexpr uint32_t OFF_BAR = OFF_RING + SLOTS * BLK;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;   // (1 KiB to align the base)
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

// (P's barriers: two halves of 64 keys per query tile)
enum { B_QFULL = 0, B_KFULL = 2, B_VFULL = 4, B_FREE = 6, B_SFULL = B_FREE + SLOTS, B_PFULL = B_SFULL + 2,
       B_OFULL = B_PFULL + 4, B_DRAIN = B_OFULL + 2, B_START = B_DRAIN + 2, N_BARS };
static_assert(N_BARS * 8 <= 256, "barriers");
constexpr uint32_t TM_S = 0, TM_O = 256;   // S_A, S_B, O_A, O_B: 128 columns each

constexpr uint32_t IDESC_S = sm100::idesc_bf16(128, 128, 0, 0);
constexpr uint32_t IDESC_PV = sm100::idesc_bf16(128, 128, 0, 1);   // V is read MN-major

struct Args {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int n_seqs, n_heads;
  int64_t tq, tk;
  __nv_bfloat16* o;
  float* lse;
  float scale;
  int causal;
};

// Which sequence and which pair of query tiles a CTA's index means (n = -1: none).
__device__ __forceinline__ int pair_count(const Args& a, int n) {
  int64_t b, e;
  seq_bounds(a.cu_q, n, a.n_seqs, a.tq, b, e);
  return (int)((e - b + PAIR - 1) / PAIR);
}
// Up to 32 sequences, by one warp: the pairs of all sequences go by their number within the
// sequence, the last first. With causal masking the longest work is then started first and the
// SMs finish together (sequence by sequence, 40 % of their time was idle at 4,096 tokens and 16
// heads). Level p holds the sequences with more than p pairs; F(p), the number of pairs at level p
// or above, falls with p.
__device__ __forceinline__ void locate_by_level(const Args& a, int idx, int lane, int& n, int& pair) {
  n = -1;
  pair = 0;
  const int mine = a.cu_q == nullptr ? (lane == 0 ? (int)((a.tq + PAIR - 1) / PAIR) : 0)
                                     : (lane < a.n_seqs ? pair_count(a, lane) : 0);
  auto above = [&](int p) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)max(mine - p, 0)); };
  int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)mine), f1 = 0;   // F(lo) > idx >= F(hi) = f1
  if (above(0) <= idx) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, f = above(mid);
    if (f > idx) {
      lo = mid;
    } else {
      hi = mid;
      f1 = f;
    }
  }
  // of the sequences with more than lo pairs, the one at place idx - F(lo + 1)
  n = (int)__fns(__ballot_sync(0xffffffffu, mine > lo), 0, idx - f1 + 1);
  pair = lo;
}
// More sequences, by the whole block: sequence by sequence, a sequence's last pair first (with that
// many, the items even out by themselves, and the search stays one pass over the lengths).
__device__ __forceinline__ void locate_in_order(const Args& a, int idx, int (&sums)[THREADS / 32], int& n_out, int& pair_out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + THREADS - 1) / THREADS;
  const int n0 = min(a.n_seqs, tid * per), n1 = min(a.n_seqs, n0 + per);
  int mine = 0;
  for (int n = n0; n < n1; ++n) mine += pair_count(a, n);
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int before = upto - mine;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w)
    if (w < warp) before += sums[w];
  if (idx >= before && idx < before + mine)
    for (int n = n0; n < n1; ++n) {
      const int c = pair_count(a, n);
      if (idx < before + c) {
        n_out = n;
        pair_out = c - 1 - (idx - before);
        break;
      }
      before += c;
    }
}

__device__ __forceinline__ float row_max(const float* s) {
  float mx[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(s[k], s[k + 4]), s[k + 8]);
#pragma unroll
  for (int c = 12; c < 124; c += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[c + k]), s[c + k + 4]);
#pragma unroll
  for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[124 + k]);
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// Weights 2^(s sc - ms) of 64 scores, as bf16 pairs into tensor memory 16 registers at a time (32
// made the loop spill, 2 to 3 % of its time), their sum added to `sum`. (Leaving every
// fourth pair to a polynomial on the FMA units made an early form of this kernel slower, 238 against
// 221 us for 4,096 tokens; with the present order of work it has not been tried.)
__device__ __forceinline__ void weights(const float* s, float sc, float ms, uint32_t t_p, float2& sum) {
  const float2 sc2 = make_float2(sc, sc), ms2 = make_float2(-ms, -ms);
  float2 part = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = __ffma2_rn(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), sc2, ms2);
      const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
      if (i & 1)
        part = __fadd2_rn(part, e);
      else
        sum = __fadd2_rn(sum, e);
      p[i] = pack2(e.x, e.y);
    }
    sm100::tmem_st16(t_p + (c >> 1), p);
  }
  sum = __fadd2_rn(sum, part);
}

// PARTS: some sequence may have more than FOLD key tiles
template <bool PARTS>
__global__ void __launch_bounds__(THREADS, 1)
kda_mla_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_ks, const __grid_constant__ CUtensorMap map_v,
                       const Args a) {
  using namespace sm100;
  extern __shared__ unsigned char pf_smem_raw[];
  unsigned char* sm = pf_smem_raw + ((1024u - (smem_u32(pf_smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_seq, s_pair, s_sums[THREADS / 32];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.x % a.n_heads;
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
    if (lane == 0 && a.tk > 0) {
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_ks);
      prefetch_tensormap(&map_v);
    }
  }
  if (warp == 9) {
    int n = -1, pair = 0;
    if (a.n_seqs <= 32) locate_by_level(a, blockIdx.x / a.n_heads, lane, n, pair);
    if (lane == 0) {
      s_seq = n;
      s_pair = pair;
      s_abort = 0;
      for (int i = 0; i < N_BARS; ++i)
        mbar_init(&bars[i], (i >= B_PFULL && i < B_PFULL + 4) || i == B_START ? BM : i >= B_FREE && i < B_FREE + SLOTS ? 2 : 1);
      fence_mbar_init();
    }
  }
  // (s_seq is set above before the search's own barrier, so a hit below comes after it)
  if (a.n_seqs > 32) locate_in_order(a, blockIdx.x / a.n_heads, s_sums, s_seq, s_pair);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int seq = s_seq;
  if (seq < 0) {   // (the bound on the pairs counts up to one more per sequence)
    if (warp == 8) tmem_dealloc(tmem, 512);
    return;
  }
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
  const Waiter wait{&s_abort};

  // A softmax thread holds a row of S (128 registers): the launch's 3 x 168 registers per
  // thread of the three warpgroups are split 208 + 208 + 88.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 || warp == 11) {
      // ---- copies: warp 8 queries and keys, warp 11 values (each waits for its own slots) ----
      if (lane == 0 && n_tiles > 0) {
        const bool keys = warp == 8;
        bool alive = true;
        int j = 0;
        auto load_q = [&](int x) {
          if (nt[x] == 0) return;
          const int y = (int)(bq + s_pair * PAIR + x * BM);
          mbar_arrive_expect_tx(&bars[B_QFULL + x], Q_BYTES);
          for (int b = 0; b < 3; ++b)
            tma_load_3d(sm + OFF_Q + x * Q_BYTES + b * BLK, &map_q, 64 * b, head, y, &bars[B_QFULL + x]);
        };
        if (keys) load_q(0);
        for (; j < n_tiles && alive; ++j) {
          const int y = (int)(bk + (int64_t)j * BN);
          // (a tile's keys complete one phase, its values one: every wait of the products' warps costs)
          uint64_t* full = &bars[(keys ? B_KFULL : B_VFULL) + (j & 1)];
          for (int part = keys ? 0 : 3; part < (keys ? 3 : PER_TILE); ++part) {
            const int i = j * PER_TILE + part, slot = i % SLOTS, use = i / SLOTS;
            if (use > 0 && !(alive = wait.one(&bars[B_FREE + slot], (use - 1) & 1))) break;
            unsigned char* dst = sm + OFF_RING + slot * BLK;
            if (part == 0) mbar_arrive_expect_tx(full, 3 * BLK);
            if (part == 3) mbar_arrive_expect_tx(full, 2 * BLK);
            if (part < 2) {
              tma_load_3d(dst, &map_k, 64 * part, head, y, full);
            } else if (part == 2) {
              tma_load_2d(dst, &map_ks, 0, y, full);
              if (j == 0) load_q(1);
            } else {
              tma_load_3d(dst, &map_v, 0, head, y + 64 * (part - 3), full);
              tma_load_3d(dst + BLK / 2, &map_v, 64, head, y + 64 * (part - 3), full);
            }
          }
        }
        if (!alive) {
          for (int x = 0; x < 2; ++x)
            if (keys && nt[x] > 0) settle_bar(&bars[B_QFULL + x], 0);
          for (int i = max(0, j - 2); i <= j; ++i)   // (a part of a tile leaves its phase open: the wait ends by its limit)
            settle_bar(&bars[(keys ? B_KFULL : B_VFULL) + (i & 1)], (i >> 1) & 1);
        }
      }
    } else if (warp < 11) {
      // ---- products of one query tile ----
      // A warp each for A and B: a wait leaves its issuer's products idle for 160 to 220 cycles
      // even when it is over at once (measured between groups of four), which the other's fill.
      const int x = warp - 9, n_x = nt[x];
      const uint32_t sb = smem_u32(sm);
      const uint64_t q0 = make_sdesc(sb + OFF_Q + x * Q_BYTES, 16, 1024, SWZ_128B);
      bool alive = n_x == 0 || wait(&bars[B_QFULL + x], 0);
      // Over many tiles B starts when A's first weights are there, so that one tile's softmax falls
      // into the other's products from then on; short rows lose the start. In every CTA against in
      // none, 32 heads (16), us: prompts of 32 tiles 167 / 164 (106 / 104), 40: 248 / 246, 48:
      // 344 / 346 (226 / 208), 64: 593 / 599 (324 / 332), 96 at 4 heads 251 / 283; 1,024 queries
      // behind a prefix, where all CTAs are long, 32 tiles in all 92 / 99, 40: 107 / 115, 64:
      // 155 / 170. (The rule goes by a CTA's own tiles, so a prompt's first pairs start together.)
      if (x == 1 && nt[0] >= LATE_START) alive = alive && wait(&bars[B_START], 0);
      for (int j = -1; j < n_tiles && alive; ++j) {
        if (j >= 0) {
          // O_x += P_x V_j, by halves of 64 keys
          if (!(alive = wait(&bars[B_VFULL + (j & 1)], (j >> 1) & 1))) break;
          const int valid = len_k - j * BN;
          const int steps = j < n_x ? min(8, (kend[x] - j * BN + 15) >> 4) : 0;
#pragma unroll 1
          for (int h = 0; h < 2 && alive; ++h) {
            const int slot = (j * PER_TILE + 3 + h) % SLOTS;
            const int r0 = max(valid - 64 * h, 0), r1 = min((r0 + 15) & ~15, 64);
            if (r0 < r1) {
              // rows behind the sequence's last key inside its 16-row step: whatever the copy
              // brought (the next sequence's values), their weights of zero must meet zeros
              // (written by both warps: each before its own products)
              unsigned char* v = sm + OFF_RING + slot * BLK;
              for (int k = lane; k < (r1 - r0) * 16; k += 32)
                *reinterpret_cast<uint4*>(v + ((k >> 3) & 1) * (BLK / 2) + (r0 + (k >> 4)) * 128 + (k & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (j < n_x && !(alive = wait(&bars[B_PFULL + 2 * x + h], j & 1))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t v0 = make_sdesc(sb + OFF_RING + slot * BLK, BLK / 2, 1024, SWZ_128B);
              const int n = min(4, steps - 4 * h);
              for (int kk = 0; kk < n; ++kk)
                umma_bf16_tmem_a(tmem + TM_O + x * 128, tmem + TM_S + x * 128 + (4 * h + kk) * 8,
                                 v0 + ((kk * 2048) >> 4), IDESC_PV, (j > 0 || h > 0 || kk > 0) ? 1u : 0u);
              umma_commit(&bars[B_FREE + slot]);
              if (h == 1 && j + 1 == n_x) umma_commit(&bars[B_OFULL + x]);
            }
          }
        }
        // S_x(j+1) = Q_x K_j+1^T overwrites P_x(j): products of one thread run in the order of issue.
        // (A tile of keys that x does not see any more is freed all the same.)
        if (alive && j + 1 < n_tiles) {
          if (!(alive = wait(&bars[B_KFULL + ((j + 1) & 1)], ((j + 1) >> 1) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int b = 0; b < 3; ++b) {
              const int slot = ((j + 1) * PER_TILE + b) % SLOTS;
              const uint64_t k0 = make_sdesc(sb + OFF_RING + slot * BLK, 16, 1024, SWZ_128B);
              if (j + 1 < n_x) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16(tmem + TM_S + x * 128, q0 + ((b * BLK + kk * 32) >> 4), k0 + ((kk * 32) >> 4), IDESC_S,
                            b > 0 || kk > 0 ? 1u : 0u);
              }
              umma_commit(&bars[B_FREE + slot]);
            }
            if (j + 1 < n_x) umma_commit(&bars[B_SFULL + x]);
          }
        }
      }
      if (!alive && elect_one()) {
        umma_commit(&bars[B_DRAIN + x]);
        settle_bar(&bars[B_DRAIN + x], 0);
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
    float kept[D + 1];   // (PARTS) accumulators taken out, and the reference they belong to: local memory
    kept[D] = 0.f;
    auto kept_by = [&]() { return kept[D] == m ? 1.f : exp2_fast((kept[D] - m) * sc); };
    bool alive = true;
    for (int j = 0; j < n_x; ++j) {
      if (!(alive = wait(&bars[B_SFULL + x], j & 1))) break;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
      tmem_ld_wait();
      const int lim = see - j * BN;
      const bool masked = __any_sync(0xffffffffu, lim < BN);
      if (masked) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= lim) s[c] = -INFINITY;
      }
      // The weights of the first half are formed with the old reference while the tile's maximum
      // is found, and again in the rare tile that moves it. (The first tile, and a masked one,
      // find their maximum first.)
      float2 sum = make_float2(0.f, 0.f);
      auto move_to = [&](float mt) {   // true for the warp if a row's reference moves, or the part ends
        const bool move = mt > m && (mt - m) * sc > RESCALE_LOG2;   // (from -inf: always)
        const bool out = PARTS && j % FOLD == 0;
        if (!__any_sync(0xffffffffu, move || out)) return false;
        // (P V of the tile before has completed: it was issued before the S waited for)
        const float f = move ? exp2_fast((m - mt) * sc) : 1.f;
        if (move) m = mt;
        l *= f;
        float kf = 0.f;
        if constexpr (PARTS) {
          if (out) {
            kf = kept_by();
            kept[D] = m;
          }
        }
#pragma unroll (PARTS ? 1 : 8)
        for (int c = 0; c < 8; ++c) {
          float v[16];
          tmem_ld16(t_o + 16 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= f;
          if constexpr (PARTS) {
            if (out)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                kept[16 * c + i] = j == FOLD ? v[i] : fmaf(kept[16 * c + i], kf, v[i]);
                v[i] = 0.f;
              }
          }
          tmem_st16(t_o + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&v));
        }
        return true;
      };
      auto reference = [&]() { return m == -INFINITY ? 0.f : m * sc; };
      if (j == 0 || masked) {
        const float mt = row_max(s);
        if (j == 0)
          m = mt;
        else
          move_to(mt);
        weights(s, sc, reference(), t_s, sum);
      } else {
        weights(s, sc, reference(), t_s, sum);
        if (move_to(row_max(s))) {
          sum = make_float2(0.f, 0.f);
          tmem_st_wait();   // (stores have no order among themselves: the first weights land before these)
          weights(s, sc, reference(), t_s, sum);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars[B_PFULL + 2 * x]);   // its product starts while the second half is formed
      if (x == 0 && j == 0) mbar_arrive(&bars[B_START]);
      weights(s + 64, sc, reference(), t_s + 32, sum);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars[B_PFULL + 2 * x + 1]);
      l += sum.x + sum.y;
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
        if constexpr (PARTS) {
          if (n_x > FOLD) {
            const float f = kept_by();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(kept[32 * c + i], f, v[i]);
          }
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
