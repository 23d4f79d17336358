// Latent attention, absorbed form: queries already multiplied into the latent space attend to
// the paged cache itself, whose 576 values per token are the key and whose first 512 the value
// of every head.
//
//     s_rj = scale q_r . c_j,   o_r = sum_j softmax_j(s_r) c_j[0:512],   r = (token, head)
//
// A token sees the rows before the sequence's n_tokens newest and, of those, the ones its
// ancestor bits name (a chain: those not after it).
//
// Bound: 1,152 bytes per cached token, read once for up to 64 (token, head) rows, against
// 2 (576 + 512) flops per row: HBM up to about 100 rows.
//
// A tile of 32 keys is copied once into shared memory and serves both products from there: as
// the K-major B operand of S = Q K^T (64 x 32), and, read the other way round, as the MN-major A
// operand of O^T = V^T P^T, whose 512 latents fill four accumulators of 128 lanes with the rows
// as columns. That way few rows cost few columns (a 64-row O would always cost 128 lanes), and
// P needs no transpose: a softmax warp writes its rows as the K-major B operand.
// Warps 0-3: softmax of rows 16w .. 16w+15 of S, rescaling and output of latents 32w .. + 31 of
// every accumulator; warp 4: copies; warps 5 and 6: the two products.
//
// The work of all sequences is one line of tiles, cut into equal runs, one per CTA, so ragged
// lengths and few long sequences fill the GPU alike. A run covers parts of one or more
// (sequence, row group) items; an item cut by a run's border is left as partial sums (fp32) in
// the workspace and joined by a second kernel in a fixed order. The matrix units cut each sum to
// fp32, twice a tile: a run of 131,072 rows of one sequence loses up to 0.1 % of values of one sign,
// which takes 22 GB of cache in one call.
//
// Measured: 128 sequences of 1k to 8k rows, 32 heads, one token: 134 to 154 us by clock (720 MB; a
// read of them alone takes 121). Per tile of 32 keys S takes 36 products of 27 cycles (64 x 32 x
// 16: the operands' reads, not the multiplications), P V 8 of 43 (32 rows) to 50 (64); copies of
// the stages not held by products keep about 110 KiB in flight per SM. 48 trees of 8 tokens (256
// rows a sequence, four items that share the cache in L2): 203 to 237 us, bound by S.
#pragma once

#include "kda_common.cuh"
#include "kda_mla_append.cuh"
#include "kda_mla_prefill.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace mla {
namespace dec {

constexpr int BN = 32;                                  // keys per tile
constexpr int ROWS = 64;                                // (token, head) rows of one item at most
constexpr int THREADS = 224;
constexpr uint32_t GROUP = 8 * WIDTH * 2;               // 8 cached rows: nine 1 KiB swizzle atoms
constexpr uint32_t STAGE = BN / 8 * GROUP;              // 36,864 bytes
constexpr int MAX_STAGES = 5;
constexpr int LOOK = 4;                                 // tiles from reading a page's number to its copy
// A CTA's run is at least this long. One sequence of 640 / 5,003 / 9,001 rows, us with 2 (more parts to
// join, and no idle SM for the join to start on), 3 and 4 tiles: 4 heads 9.9 / 13.4 / 16.5, 10.6 /
// 13.3 / 15.2, 11.6 / 14.0 / 14.9; 32 heads 11.0 / 15.0 / 18.0, 11.6 / 14.6 / 17.4, 12.6 / 15.0 / 16.8;
// 64 heads 12.5 / 17.6 / 20.9, 13.1 / 16.4 / 19.5, 14.2 / 16.9 / 18.9; 128 heads 13.1 / 18.4 / 19.9,
// 13.9 / 20.7 / 19.9, 14.8 / 19.7 / 22.7. From 20,000 rows on they are the same.
constexpr int MIN_TILES = 3;
constexpr int MAX_GRID = 160;                           // CTAs of the main kernel at most (the join holds a part per lane and round)
enum { B_KVFULL = 0, B_KVFREE = MAX_STAGES, B_SFULL = 2 * MAX_STAGES, B_PFULL = B_SFULL + 8, B_PVDONE = B_PFULL + 2,
       B_QFULL = B_PVDONE + 2, B_QFREE, B_OFREE, B_DRAIN, N_BARS = B_DRAIN + 2 };
constexpr uint32_t TM_O = 0, TM_S = 256;                // four accumulators 64 columns apart; eight S

// Shared memory: Q, the stages (as many as fit, 5 up to 32 rows, else 4), P twice, barriers, the
// rows' factors.
constexpr uint32_t SMEM_MOST = 232448 - 1024;           // (less the static part)
__host__ __device__ constexpr uint32_t p_bytes(int rb) { return (uint32_t)rb * BN * 2; }
__host__ __device__ constexpr uint32_t off_kv(int rb) { return (uint32_t)rb * WIDTH * 2; }
constexpr uint32_t TAIL = 256 + 2 * ROWS * 4 + 1024;    // barriers, factors, alignment
__host__ __device__ constexpr int stages_of(int rb) {
  return off_kv(rb) + MAX_STAGES * STAGE + 2 * p_bytes(rb) + TAIL <= SMEM_MOST ? MAX_STAGES : MAX_STAGES - 1;
}
__host__ __device__ constexpr uint32_t off_p(int rb) { return off_kv(rb) + stages_of(rb) * STAGE; }
__host__ __device__ constexpr uint32_t off_bar(int rb) { return off_p(rb) + 2 * p_bytes(rb); }
__host__ __device__ constexpr uint32_t smem_bytes(int rb) { return off_bar(rb) + TAIL; }
static_assert(smem_bytes(16) <= SMEM_MOST && smem_bytes(32) <= SMEM_MOST && smem_bytes(48) <= SMEM_MOST &&
                  smem_bytes(64) <= SMEM_MOST && N_BARS * 8 <= 256,
              "shared memory of one CTA");

struct Args {
  const int32_t* page_table;
  const int32_t* cache_lens;
  const int32_t* tree;
  __nv_bfloat16* o;
  float* lse;
  float* part;          // [2 workers][rb][512] partial sums, then [2 workers][rb][2] (m, l)
  int n_seqs, n_tokens, n_heads;
  int rows;             // n_tokens * n_heads
  int groups;           // items per sequence
  int rb;               // rows of an item, padded: 16, 32, 48 or 64
  int n_pages, page_size, max_pages;
  int page_rows;        // rows per copy: the largest power of two up to a tile's that divides page_size
  int grid;             // CTAs of the main kernel
  float scale;
};

__device__ __forceinline__ int seq_len(const Args& a, int n, bool flag) {
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  const int64_t len = a.cache_lens[n];
  if (flag && (len < 0 || len > cap)) flag_error(DEVERR_PAGE);
  return (int)(len < 0 ? 0 : len > cap ? cap : len);
}
__device__ __forceinline__ int seq_tiles(const Args& a, int n) { return (seq_len(a, n, false) + BN - 1) / BN; }

// CTAs that work on a line of `total` tiles.
__device__ __forceinline__ int worker_count(const Args& a, int64_t total) {
  const int64_t want = (total + MIN_TILES - 1) / MIN_TILES;
  return (int)(want < a.grid ? want : a.grid);
}

// The run [begin, end) of worker `who` on the line of tiles (empty past the last worker), the
// sequence that holds its first tile and that sequence's own first tile. Returns the tiles in
// all. By the whole block of T threads: each sums a run of sequences, so the loads are
// independent.
template <int T>
__device__ __forceinline__ int64_t locate(const Args& a, int64_t (&sums)[T / 32], int64_t (&found)[2], int who,
                                          int& workers, int64_t& begin, int64_t& end, int& n_at,
                                          int64_t& first_at) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + T - 1) / T;
  const int n0 = min(a.n_seqs, tid * per), n1 = min(a.n_seqs, n0 + per);
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += seq_tiles(a, n);
  mine *= a.groups;
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  workers = worker_count(a, total);
  begin = end = total;
  if (who < workers) {
    begin = total * who / workers;
    end = total * (who + 1) / workers;
  }
  int64_t f = before + upto - mine;
  if (mine > 0 && begin >= f && begin < f + mine)
    for (int n = n0; n < n1; ++n) {
      const int64_t c = (int64_t)seq_tiles(a, n) * a.groups;
      if (begin < f + c) {
        found[0] = n;
        found[1] = f;
        break;
      }
      f += c;
    }
  __syncthreads();
  n_at = (int)found[0];
  first_at = found[1];
  return total;
}

// A CTA's run, item by item.
struct Walk {
  int n, g, t0, t1, tiles, len;   // the item, and the tiles of it that belong to the run
  int64_t left;
  __device__ __forceinline__ bool start(const Args& a, int n_at, int64_t first_at, int64_t begin, int64_t end) {
    left = end - begin;
    if (left <= 0) return false;
    n = n_at;
    len = seq_len(a, n, false);
    tiles = (len + BN - 1) / BN;
    const int64_t in = begin - first_at;
    g = (int)(in / tiles);
    t0 = (int)(in - (int64_t)g * tiles);
    t1 = (int)(left < tiles - t0 ? t0 + left : tiles);
    return true;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++g == a.groups) {
      g = 0;
      do {
        if (++n >= a.n_seqs) return false;
        len = seq_len(a, n, false);
      } while (len == 0);
      tiles = (len + BN - 1) / BN;
    }
    t0 = 0;
    t1 = (int)(left < tiles ? left : tiles);
    return true;
  }
};

__device__ __forceinline__ void tma_load_4d(void* dst_smem, const CUtensorMap* map, int32_t w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(sm100::smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(0), "r"(w), "r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t q0, uint32_t q1, uint32_t q2, uint32_t q3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(q0), "r"(q1),
               "r"(q2), "r"(q3)
               : "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
kda_mla_decode_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
                      const Args a) {
  using namespace sm100;
  extern __shared__ unsigned char dec_smem_raw[];
  unsigned char* sm = dec_smem_raw + ((1024u - (smem_u32(dec_smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + off_bar(a.rb));
  float* s_fac = reinterpret_cast<float*>(sm + off_bar(a.rb) + 256);   // a factor per row
  const int stages = stages_of(a.rb);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int64_t s_sums[THREADS / 32], s_found[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (what needs no lengths goes out before they are loaded: a short call is all latency)
  if (warp == 4) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
    if (lane == 0) {
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_c);
    }
  }
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < N_BARS; ++i) mbar_init(&bars[i], i == B_PFULL || i == B_PFULL + 1 || i == B_OFREE ? 128 : 1);
    fence_mbar_init();
  }
  tc_fence_before();
  int workers, n_at;
  int64_t begin, end, first_at;
  locate<THREADS>(a, s_sums, s_found, blockIdx.x, workers, begin, end, n_at, first_at);   // (with its barriers)
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the join waits for this kernel's end)
  const uint32_t tmem = s_tmem;
  const Waiter wait{&s_abort};
  Walk w;
  bool more = w.start(a, n_at, first_at, begin, end);   // (false for a CTA without a run: every role passes)

  if (warp == 4) {
    // ---- copies: lane c brings the c-th piece of page_rows rows of a tile ----
    // The page's number is read LOOK tiles ahead of the copy, off its path. (Bringing the piece
    // into L2 along with it gained nothing: 152 against 148 us for 128 sequences.)
    const int pieces = BN / a.page_rows;
    Walk wa = w;
    int ia = w.t0;
    bool a_left = more;
    // the cursor's piece of this lane: its first row over 8, or -1; then a tile further
    auto look = [&]() {
      int row8 = -1;
      if (a_left) {
        const int pos = ia * BN + lane * a.page_rows;
        if (lane < pieces && pos < wa.len) {
          const int pi = pos / a.page_size;
          int page = a.page_table[(int64_t)wa.n * a.max_pages + pi];
          if (page < 0 || page >= a.n_pages) {
            flag_error(DEVERR_PAGE);
            page = 0;
          }
          row8 = (int)(((int64_t)page * a.page_size + (pos - pi * a.page_size)) >> 3);
        }
        if (++ia == wa.t1) {
          a_left = wa.next(a);
          ia = wa.t0;
        }
      }
      return row8;
    };
    int queue[LOOK];
#pragma unroll
    for (int k = 0; k < LOOK; ++k) queue[k] = look();
    int it = 0, sg = 0, st = 0, round = 0;   // tile, item, stage and its use
    bool alive = true;
    for (; more && alive; more = w.next(a), ++sg) {
      for (int i = w.t0; i < w.t1 && alive; ++i, ++it, st = st + 1 == stages ? 0 : st + 1, round += st == 0) {
        const int row8 = queue[0];
#pragma unroll
        for (int k = 1; k < LOOK; ++k) queue[k - 1] = queue[k];
        queue[LOOK - 1] = look();
        const int count = __popc(__ballot_sync(0xffffffffu, row8 >= 0));
        uint64_t* full = &bars[B_KVFULL + st];
        if (round > 0) alive = wait(&bars[B_KVFREE + st], (round - 1) & 1);
        if (!alive) break;
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)count * a.page_rows * (WIDTH * 2));
        __syncwarp();
        if (row8 >= 0)
          tma_load_4d(sm + off_kv(a.rb) + st * STAGE + lane * (a.page_rows / 8) * GROUP, &map_c, row8, full);
        if (i == w.t0) {   // (after the item's first keys, which need not wait for the item before)
          if (sg > 0) alive = wait(&bars[B_QFREE], (sg - 1) & 1);
          if (alive && lane == 0) {
            mbar_arrive_expect_tx(&bars[B_QFULL], (uint32_t)a.rb * WIDTH * 2);
            tma_load_3d(sm, &map_q, 0, (int)((int64_t)w.n * a.rows + w.g * a.rb), 0, &bars[B_QFULL]);
          }
        }
      }
      if (!alive) break;
    }
    if (!alive && lane == 0) {   // (sg: Q loads issued so far lie at or below it)
      for (int j = max(0, it + 1 - stages); j <= it; ++j)
        settle_bar(&bars[B_KVFULL + j % stages], (j / stages) & 1);
      settle_bar(&bars[B_QFULL], sg & 1);
    }
  } else if (warp == 5) {
    // ---- S = Q K^T ----
    // The two products have a warp each: from one, in any order, every wait between them left
    // the tensor cores idle for 400 to 500 cycles (the barriers share the port of shared memory
    // that the operands keep busy), 1,000 of a tile's 2,400. S goes on into eight buffers: the
    // one a tile takes was read when the tile's stage came free.
    const uint32_t sb = smem_u32(sm);
    const uint32_t idesc = idesc_bf16(64, BN, 0, 0);
    const uint64_t q0 = make_sdesc(sb, 16, 1024, SWZ_128B);
    const uint32_t q_blk = ((uint32_t)a.rb * 128) >> 4;
    int it = 0, sg = 0, st = 0, round = 0;
    bool alive = true;
    for (; more && alive; more = w.next(a), ++sg) {
      alive = wait(&bars[B_QFULL], sg & 1);
      for (int i = w.t0; i < w.t1 && alive; ++i, ++it, st = st + 1 == stages ? 0 : st + 1, round += st == 0) {
        if (!(alive = wait(&bars[B_KVFULL + st], round & 1))) break;
        const int valid = w.len - i * BN;
        if (valid < BN && (valid & 15)) {
          // rows behind the last key in its 16-row step (an earlier tile's, or nothing yet):
          // their weights of zero must meet zeros
          const int r1 = (valid + 15) & ~15;
          unsigned char* kv = sm + off_kv(a.rb) + st * STAGE;
          for (int k = lane; k < (r1 - valid) * (WIDTH / 8); k += 32) {
            const int r = valid + k / (WIDTH / 8), c = k % (WIDTH / 8);
            *reinterpret_cast<uint4*>(kv + (r >> 3) * GROUP + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t k0 = make_sdesc(sb + off_kv(a.rb) + st * STAGE, 16, GROUP, SWZ_128B);
          const uint32_t d = tmem + TM_S + (it & 7) * BN;
#pragma unroll 1
          for (int blk = 0; blk < 9; ++blk)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(d, q0 + blk * q_blk + ((kk * 32) >> 4), k0 + ((blk * 1024 + kk * 32) >> 4), idesc,
                        (blk > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars[B_SFULL + (it & 7)]);
          if (i + 1 == w.t1) umma_commit(&bars[B_QFREE]);
        }
      }
      if (!alive) break;
    }
    if (!alive && elect_one()) {
      umma_commit(&bars[B_DRAIN]);
      settle_bar(&bars[B_DRAIN], 0);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ---- O^T += V^T P^T ----
    const uint32_t sb = smem_u32(sm);
    const uint32_t idesc = idesc_bf16(128, (uint32_t)a.rb, 1, 0);
    const uint64_t p0 = make_sdesc(sb + off_p(a.rb), 16, 512, SWZ_64B);
    int it = 0, sg = 0, st = 0;
    bool alive = true;
    for (; more && alive; more = w.next(a), ++sg) {
      if (sg > 0) alive = wait(&bars[B_OFREE], (sg - 1) & 1);
      for (int i = w.t0; i < w.t1 && alive; ++i, ++it, st = st + 1 == stages ? 0 : st + 1) {
        if (!(alive = wait(&bars[B_PFULL + (it & 1)], (it >> 1) & 1))) break;
        tc_fence_after();
        const int steps = min(BN / 16, (w.len - i * BN + 15) >> 4);
        if (elect_one()) {
          const uint64_t v0 = make_sdesc(sb + off_kv(a.rb) + st * STAGE, 1024, GROUP, SWZ_128B);
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk)
#pragma unroll
            for (int mb = 0; mb < 4; ++mb)
              umma_bf16(tmem + TM_O + mb * 64, v0 + ((kk * 2 * GROUP + mb * 2048) >> 4),
                        p0 + (((it & 1) * p_bytes(a.rb) + kk * 32) >> 4), idesc, (i > w.t0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars[B_KVFREE + st]);
          umma_commit(&bars[B_PVDONE + (it & 1)]);
        }
      }
      if (!alive) break;
    }
    if (!alive && elect_one()) {
      umma_commit(&bars[B_DRAIN + 1]);
      settle_bar(&bars[B_DRAIN + 1], 0);
    }
    __syncwarp();
  } else {
    // ---- softmax, rescaling, output ----
    // rows of S that this thread holds a quarter of: 16w + lane/4 and 8 further; keys 2(lane%4),
    // + 1 of every eight
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const int ra = 16 * warp + (lane >> 2);
    const bool busy = 16 * warp < a.rb;     // (warps beyond the item's rows only rescale and store)
    const float sc = a.scale * LOG2E_F;
    const uint32_t p_base = smem_u32(sm) + off_p(a.rb);
    int it = 0;
    bool alive = true;
    for (; more && alive; more = w.next(a)) {
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      uint32_t bits[2] = {0u, 0u};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = w.g * a.rb + ra + 8 * h;
        if (r < a.rows) {
          const int j = r / a.n_heads;
          bits[h] = a.tree ? (uint32_t)a.tree[(int64_t)w.n * a.n_tokens + j] : (2u << j) - 1u;
        }
      }
      const int prefix = w.len - a.n_tokens;   // rows every token sees (may be negative)
      // No warp leaves the loop on its own: after a timeout every wait fails at once and the
      // tiles run out, so that the four warps always meet at the same barriers.
      for (int i = w.t0; i < w.t1; ++i, ++it) {
        const uint32_t half = (it >> 1) & 1;
        alive = wait(&bars[B_SFULL + (it & 7)], (it >> 3) & 1) && alive;
        tc_fence_after();
        float s[16];
        bool move = false;
        float f[2] = {1.f, 1.f};
        if (busy) {
          tmem_ld16x256b_x4(tmem + TM_S + (it & 7) * BN + lane_base, *reinterpret_cast<uint32_t(*)[16]>(&s));
          tmem_ld_wait();
          if ((i + 1) * BN > prefix) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int d = i * BN + 8 * (e >> 2) + 2 * (lane & 3) + (e & 1) - prefix;   // the row among the newest
              const bool seen = d < 0 || (d < a.n_tokens && ((bits[(e >> 1) & 1] >> d) & 1u));
              if (!seen) s[e] = -INFINITY;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mt = fmaxf(fmaxf(fmaxf(s[2 * h], s[2 * h + 1]), fmaxf(s[2 * h + 4], s[2 * h + 5])),
                             fmaxf(fmaxf(s[2 * h + 8], s[2 * h + 9]), fmaxf(s[2 * h + 12], s[2 * h + 13])));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
            if (i == w.t0) {
              m[h] = mt;
            } else if (mt > m[h] && (mt - m[h]) * sc > RESCALE_LOG2) {
              f[h] = exp2_fast((m[h] - mt) * sc);
              l[h] *= f[h];
              m[h] = mt;
              move = true;
            }
          }
        }
        const bool rescale = i > w.t0 && named_bar_or(1, 128, move);
        uint32_t p[8];
        if (busy) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float ms = m[h] == -INFINITY ? 0.f : m[h] * sc;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float e0 = exp2_fast(fmaf(s[e + 2 * h], sc, -ms)), e1 = exp2_fast(fmaf(s[e + 2 * h + 1], sc, -ms));
              l[h] += e0 + e1;
              p[(e >> 1) + h] = pack2(e0, e1);
            }
          }
        }
        // the P buffer is free once the products of two tiles before are done
        if (it >= 2) alive = wait(&bars[B_PVDONE + (it & 1)], half ^ 1u) && alive;
        if (rescale) {   // and the accumulators with those of the tile before
          if (busy && (lane & 3) == 0) {
            s_fac[ra] = f[0];
            s_fac[ra + 8] = f[1];
          }
          alive = wait(&bars[B_PVDONE + ((it - 1) & 1)], ((it - 1) >> 1) & 1) && alive;
          tc_fence_after();
          named_bar_sync(1, 128);
          for (int mb = 0; mb < 4; ++mb)
            for (int c = 0; c < a.rb; c += 16) {
              float v[16];
              const uint32_t at = tmem + TM_O + mb * 64 + c + lane_base;
              tmem_ld16(at, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] *= s_fac[c + k];
              tmem_st16(at, *reinterpret_cast<uint32_t(*)[16]>(&v));
            }
          tmem_st_wait();
        }
        if (busy) {
          const int mi = lane >> 3;
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const uint32_t row = (uint32_t)(16 * warp + (mi & 1) * 8 + (lane & 7)), col = 8u * (k + (mi >> 1));
            stmatrix_x4(p_base + (it & 1) * p_bytes(a.rb) + swz64(row * 64u + col * 2u), p[2 * k], p[2 * k + 1],
                        p[2 * k + 2], p[2 * k + 3]);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&bars[B_PFULL + (it & 1)]);
      }
      // output: every row's maximum and sum, then the accumulators
      const bool whole = w.t0 == 0 && w.t1 == w.tiles;
      const int slot = 2 * (int)blockIdx.x + (w.t0 == 0 ? 1 : 0);
      float* part = a.part + (int64_t)slot * a.rb * LATENT;
      float* ml = a.part + (int64_t)2 * a.grid * a.rb * LATENT + (int64_t)slot * a.rb * 2;
      if (busy) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
          l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
          const int r = ra + 8 * h;
          if ((lane & 3) == 0) {
            s_fac[ROWS + r] = l[h] == 0.f ? 0.f : 1.f / l[h];
            const int64_t row = (int64_t)w.g * a.rb + r;
            if (!whole) {
              ml[2 * r] = m[h] == -INFINITY ? -INFINITY : m[h] * sc;
              ml[2 * r + 1] = l[h];
            } else if (a.lse && row < a.rows) {
              a.lse[(int64_t)w.n * a.rows + row] =
                  l[h] == 0.f ? -INFINITY : (m[h] == -INFINITY ? 0.f : m[h] * a.scale) + logf(l[h]);
            }
          }
        }
      }
      alive = wait(&bars[B_PVDONE + ((it - 1) & 1)], ((it - 1) >> 1) & 1) && alive;
      tc_fence_after();
      alive = !named_bar_or(2, 128, !alive);
      if (!alive) break;
      {
        const int rows = min(a.rb, a.rows - w.g * a.rb);
        __nv_bfloat16* od = a.o + ((int64_t)w.n * a.rows + w.g * a.rb) * LATENT + 32 * warp + lane;
        for (int mb = 0; mb < 4; ++mb)
          for (int c = 0; c < a.rb; c += 16) {
            float v[16];
            tmem_ld16(tmem + TM_O + mb * 64 + c + lane_base, v);
            tmem_ld_wait();
            if (whole) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (c + k < rows) {
                  const float inv = s_fac[ROWS + c + k];
                  od[(int64_t)(c + k) * LATENT + mb * 128] = __float2bfloat16_rn(inv == 0.f ? 0.f : v[k] * inv);
                }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) part[(c + k) * LATENT + mb * 128 + 32 * warp + lane] = v[k];
            }
          }
      }
      tc_fence_before();
      named_bar_sync(1, 128);   // (the factors are read before the next item writes its own)
      mbar_arrive(&bars[B_OFREE]);
    }
  }
  // sequences without keys: zeros and -inf, spread over the CTAs
  for (int n = blockIdx.x; n < a.n_seqs; n += gridDim.x)
    if (seq_len(a, n, tid == 0) == 0) {
      const int64_t r0 = (int64_t)n * a.rows;
      uint4* od = reinterpret_cast<uint4*>(a.o + r0 * LATENT);
      for (int64_t i = tid; i < (int64_t)a.rows * (LATENT / 8); i += THREADS) od[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = tid; i < a.rows; i += THREADS) a.lse[r0 + i] = -INFINITY;
    }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the items that a run's border cuts. With no more items than borders a block takes an
// item, else a border (and the item that it cuts, if it is the first to cut it). A row is one
// warp's (ALONE: most items have two or three parts) or four blocks' (few items of many parts: a
// block takes 128 of the latents, its warps every eighth part each). Its shared memory is small
// enough for a block to wait beside a CTA of the main kernel of up to 48 rows: with room for
// that, 5,000 rows of one sequence take 15 us, without it 20. Which part holds what follows from the lengths alone,
// so it is worked out while the main kernel's last CTAs still run; 19 to 38 MB of sums, mostly
// from L2.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_THREADS = 32 * JOIN_WARPS;

template <bool ALONE>
__global__ void __launch_bounds__(JOIN_THREADS)
kda_mla_decode_join_kernel(const Args a, int by_item) {
  __shared__ int64_t s_sums[JOIN_WARPS], s_found[2], s_mine[JOIN_WARPS];
  constexpr int SPAN = ALONE ? 4 : 1;   // 16-byte pieces of a row per lane
  __shared__ float4 s_acc[ALONE ? 1 : JOIN_WARPS / 2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int workers, n, g, tiles;
  int64_t begin, end, first_at, total, f;
  if (by_item) {
    // the position of the item's first tile: the tiles of the sequences before it
    n = blockIdx.x / a.groups;
    g = blockIdx.x - n * a.groups;
    int64_t mine = 0, all = 0;
    for (int k = tid; k < a.n_seqs; k += JOIN_THREADS) {
      const int t = seq_tiles(a, k);
      all += t;
      if (k < n) mine += t;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      mine += __shfl_xor_sync(0xffffffffu, mine, off);
      all += __shfl_xor_sync(0xffffffffu, all, off);
    }
    if (lane == 0) {
      s_sums[warp] = all;
      s_mine[warp] = mine;
    }
    __syncthreads();
    total = f = 0;
    for (int k = 0; k < JOIN_WARPS; ++k) {
      total += s_sums[k];
      f += s_mine[k];
    }
    total *= a.groups;
    tiles = seq_tiles(a, n);
    f = f * a.groups + (int64_t)g * tiles;
    workers = worker_count(a, total);
  } else {
    total = locate<JOIN_THREADS>(a, s_sums, s_found, blockIdx.x + 1, workers, begin, end, n, first_at);
  }
  // Every block waits, also one with nothing to do: what follows in the stream counts on the
  // main kernel's end too.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (by_item) {
    if (tiles == 0) return;
  } else {
    if (begin >= end) return;
    tiles = seq_tiles(a, n);
    g = (int)((begin - first_at) / tiles);
    f = first_at + (int64_t)g * tiles;
    if (f == begin) return;
  }
  const int b0 = (int)(((f + 1) * workers - 1) / total), b1 = (int)(((f + tiles) * workers - 1) / total);
  if (b0 == b1 || (!by_item && b0 != (int)blockIdx.x)) return;
  const int r = ALONE ? (int)blockIdx.y * JOIN_WARPS + warp : (int)blockIdx.y >> 2;
  const int c0 = ALONE ? 0 : 32 * ((int)blockIdx.y & 3);   // first piece
  if (r >= min(a.rb, a.rows - g * a.rb)) return;   // (not ALONE: the same for the whole block)

  // Row of the k-th part, which worker b0 + k left: in its second slot if the item begins in it,
  // else its first. All parts' maxima and sums come in one round of loads, lane by lane, and with
  // them the first part's sums.
  const int parts = b1 - b0 + 1;
  const float2* ml = reinterpret_cast<const float2*>(a.part + (int64_t)2 * a.grid * a.rb * LATENT);
  auto row_of = [&](int k) { return (int64_t)(2 * (b0 + k) + (k == 0)) * a.rb + r; };
  constexpr int MOST = (MAX_GRID + 31) / 32, STEP = ALONE ? 1 : JOIN_WARPS;
  const int k0 = ALONE ? 0 : warp;
  float2 v[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int k = 32 * i + lane;
    v[i] = k < parts ? ml[row_of(k)] : make_float2(-INFINITY, 0.f);
  }
  float4 ahead[SPAN];
#pragma unroll
  for (int c = 0; c < SPAN; ++c)
    ahead[c] = k0 < parts ? reinterpret_cast<const float4*>(a.part + row_of(k0) * LATENT)[c0 + 32 * c + lane]
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < MOST; ++i) m = fmaxf(m, v[i].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    v[i].x = exp2_fast(v[i].x - ms);   // the part's weight
    l = fmaf(v[i].x, v[i].y, l);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  float4 acc[SPAN];
  {
    const float w = __shfl_sync(0xffffffffu, v[0].x, k0);
#pragma unroll
    for (int c = 0; c < SPAN; ++c) acc[c] = make_float4(w * ahead[c].x, w * ahead[c].y, w * ahead[c].z, w * ahead[c].w);
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int last = min(parts, 32 * i + 32);
#pragma unroll 4
    for (int k = 32 * i + k0 + (i == 0 ? STEP : 0); k < last; k += STEP) {
      const float w = __shfl_sync(0xffffffffu, v[i].x, k & 31);
      const float4* src = reinterpret_cast<const float4*>(a.part + row_of(k) * LATENT);
#pragma unroll
      for (int c = 0; c < SPAN; ++c) {
        const float4 x = src[c0 + 32 * c + lane];
        acc[c].x = fmaf(w, x.x, acc[c].x);
        acc[c].y = fmaf(w, x.y, acc[c].y);
        acc[c].z = fmaf(w, x.z, acc[c].z);
        acc[c].w = fmaf(w, x.w, acc[c].w);
      }
    }
  }
  const int64_t row = (int64_t)n * a.rows + g * a.rb + r;
  uint2* od = reinterpret_cast<uint2*>(a.o + row * LATENT);
  if constexpr (!ALONE) {
#pragma unroll
    for (int half = JOIN_WARPS / 2; half > 0; half >>= 1) {   // the upper half's sums onto the lower's
      if (warp >= half && warp < 2 * half) s_acc[warp - half][lane] = acc[0];
      __syncthreads();
      if (warp < half) {
        const float4 v = s_acc[warp][lane];
        acc[0].x += v.x;
        acc[0].y += v.y;
        acc[0].z += v.z;
        acc[0].w += v.w;
      }
      __syncthreads();
    }
    if (warp != 0) return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < SPAN; ++k)
    od[c0 + 32 * k + lane] =
        l == 0.f ? make_uint2(0, 0)
                 : make_uint2(pack2(acc[k].x * inv, acc[k].y * inv), pack2(acc[k].z * inv, acc[k].w * inv));
  if (a.lse && c0 == 0 && lane == 0)
    a.lse[row] = l == 0.f ? -INFINITY : ms * 0.6931471805599453f + logf(l);
}

}  // namespace dec
}  // namespace mla
}  // namespace kda
