// dsa_mla_weights, dsa_mla_weights_selected: the attention weight that each cached position gets,
// summed over the heads, and added up over the queries.
//
// w[b][t][s] = sum_h exp(scale * q[b][t][h] . kv[b][s] - lse[b][t][h]) with the lse that the
// attention returned, for the visible rows (dense) or for the selected ones (w[b][t][u] for slot u).
//
// The scores are computed transposed, S^T = K Q^T, so that a TMEM lane holds one key and the 128
// columns its heads: the sum over the heads stays inside a thread pair. A CTA pair (cta_group::2, M = 256
// keys, 128 per CTA) takes an equal share of all (query, 256-key tile) pairs; each CTA keeps 64 heads of
// the query in shared memory (72 KB) while 48 KB slots of its keys (128 keys x 192 features) pass through a
// ring of three. Per tile: 36 MMAs of 256 x 128 x 16 (65 cycles each, 2340) and 128 x 128 exponentials per
// CTA (1024 cycles of MUFU). For one query per sequence HBM is the bound: a CTA's 147 KB a tile take an SM's
// share of it 6300 cycles, and the ring's 144 KB cover its latency (48 to 50 us for 64 queries over 2048 to
// 4096 rows each, 4.9 TB/s; with 128 KB in slots of 128 features, a tenth of them empty, 51 us).
//
// A tile's contraction is cut into parts that are added in registers, an accumulator of 128 columns each. The
// exponential turns an absolute error of the score into a relative one of the weight, and the tensor core cuts off
// its running fp32 sum, 36 times over 576 features, so the error grows with the length of a part: one part left 6.7e-6
// in the weights, three (192 features, a slot each) leave 2.1e-6 over 2048 to 4096 keys, where fp32 matrix products
// leave 2.0e-6. Over fewer keys the heaviest scores are smaller and so are the roundings that both forms share: over
// 64 to 200 keys three parts left 1.1e-6 to 1.4e-6 against 0.5e-6 to 0.9e-6. Queries of at most kFineKeys keys
// therefore get six parts (96 features, two per slot), which leave 0.7e-6 there and 1.0e-6 against 1.5e-6 over 1024
// keys; beyond, three are at most 1.3 times as far off as fp32 products. Six everywhere cost the long prompt
// chunks a third of their speed (250 queries over 4050 rows: 165 instead of 126 us), and the short
// queries a twentieth (64 over about 1000 rows: 36.9 instead of 34.8 us). The parts take the four accumulators
// of TMEM in turn, so that the next ones are computed while one is read.
//
// Selected rows are gathered by four warps with 16-byte cp.async into the swizzled operand layout,
// 384 bytes of each row per slot (64 queries of 2048 rows: 45 us, 48 with 256 bytes at a time, 58 with 128, since
// shorter pieces open more of the pages of HBM for the same bytes); a fifth hands the slots that have landed to the
// leader. (Hinting whole rows into L2 a tile ahead was slower; so was hinting the next dense tile.)
//
// Prompt chunks are bounded otherwise: a key tile serves one query, so at the matrix rate each SM would take in 147 KB
// every 2340 cycles, 63 bytes a cycle. They run at about 3500 cycles a tile, 42 bytes a cycle, and leaving the
// exponentials out changes nothing (250 causal queries over 4050 rows, caches cold: 130 us with the addition over the
// queries, 20 us of it).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "pair.cuh"

namespace dsa {

namespace {

constexpr int kHeads = 128, kDqk = 576;
constexpr int kRows = 128;                         // keys of a tile on each CTA of a pair
constexpr int kTile = 2 * kRows;
constexpr int kQBlock = 64 * 128;                  // 8 KB: 64 features of this CTA's 64 heads
constexpr int kBlock = kRows * 128;                // 16 KB: 64 features of 128 keys
constexpr int kParts = 3;                          // ring slots of a tile, 192 features each
constexpr int kFineKeys = 1024;                    // queries of at most as many keys get two parts per slot, others one
constexpr int kSlot = 3 * kBlock;                  // 48 KB
constexpr int kSlots = 3;
constexpr int kAccs = 4;                           // accumulators of 128 columns, taken by the parts in turn
constexpr int kOffRing = 9 * kQBlock;
constexpr int kOffBar = kOffRing + kSlots * kSlot;
constexpr int kOffLse = kOffBar + 256;             // [4][128] fp32
constexpr int kOffSum = kOffLse + 4 * 128 * 4;     // [2][128] fp32
constexpr int kOffScan = kOffSum + 2 * 128 * 4;    // set-up words
constexpr int kSmem = 1024 + kOffScan + 256;
static_assert(kOffRing % 1024 == 0 && kSmem <= 232448, "shared memory per CTA");
constexpr int kGatherWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

}  // namespace

struct WeightsParams {
  const uint16_t* q;
  const uint16_t* kv;
  const int32_t* idx;      // [B][T][k] (selected rows), or NULL (dense)
  const float* lse;        // [B][T][128]
  const int32_t* q_pos;    // dense only
  const int32_t* kv_len;
  int64_t BT;
  int T, S_max, k;
  int64_t ld;
  float scale_log2;
  float* w;
  const float* acc;
  float* acc_out;
  int* status;
};

namespace {

// keys (or slots) of query `tok`
__device__ __forceinline__ int keys_of(const WeightsParams& p, int64_t tok) {
  if (p.idx) return p.k;
  const int64_t v = (int64_t)__ldg(p.q_pos + tok) + 1;
  const int64_t n = __ldg(p.kv_len + tok / p.T);
  return (int)max((int64_t)0, min(min(v, n), (int64_t)p.S_max));
}
__device__ __forceinline__ int tiles_of(const WeightsParams& p, int64_t tok) {
  return (keys_of(p, tok) + kTile - 1) / kTile;
}

// The runs of tiles [t0, t1) of one query each that make up this CTA's range.
struct Runs {
  int64_t left, tok;
  int t0, t1, keys;
  __device__ __forceinline__ void settle(const WeightsParams& p) {
    while (left > 0) {
      keys = keys_of(p, tok);
      const int tiles = (keys + kTile - 1) / kTile;
      if (tiles > t0) {
        t1 = (int)min((int64_t)tiles, t0 + left);
        return;
      }
      ++tok;
      t0 = 0;
    }
  }
  __device__ __forceinline__ void start(const WeightsParams& p, int64_t t, int64_t off, int64_t count) {
    tok = t;
    t0 = (int)off;
    left = count;
    settle(p);
  }
  __device__ __forceinline__ void next(const WeightsParams& p) {
    left -= t1 - t0;
    ++tok;
    t0 = 0;
    settle(p);
  }
};

}  // namespace

template <bool SELECTED>
__global__ void __launch_bounds__(SELECTED ? 512 : 384, 1)
    mla_weights_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const WeightsParams p) {
  constexpr int kThreads = SELECTED ? 512 : 384;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* full = bars;                 // leader [kSlots]: both CTAs' keys landed
  uint64_t* empty = full + kSlots;       // [kSlots] their MMAs are done
  uint64_t* gathered = empty + kSlots;   // [kSlots] this CTA's keys landed (selected rows)
  uint64_t* acc_full = gathered + kSlots;  // [kAccs] a part of the scores ready
  uint64_t* acc_empty = acc_full + kAccs;  // leader [kAccs]: both CTAs have read it
  uint64_t* q_full = acc_empty + kAccs;    // leader: both halves of the query landed
  uint64_t* q_empty = q_full + 1;        // the run's MMAs are done
  uint64_t* sum_full = q_empty + 1;      // [2][4] the second half of the heads is summed, per quadrant
  float* lse_sh = reinterpret_cast<float*>(smem + kOffLse);
  float* sum_sh = reinterpret_cast<float*>(smem + kOffSum);
  long long* scan_sh = reinterpret_cast<long long*>(smem + kOffScan);       // [kThreads / 32]
  long long* start_sh = scan_sh + 16;                                       // first query, tile of it
  uint32_t& tmem_base_sh = *reinterpret_cast<uint32_t*>(start_sh + 2);
  int& abort_flag = *reinterpret_cast<int*>(start_sh + 3);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
      mbar_init(&gathered[s], kGatherWarps * 32);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&sum_full[i], 1);
    mbar_init(q_full, 2);
    mbar_init(q_empty, 1);
    fence_barrier_init();
    start_sh[0] = start_sh[1] = 0;
  }
  if (warp == 2) pair_tmem_alloc(&tmem_base_sh, 512);
  __syncwarp();
  cluster_arrive();                      // this thread's part of the set-up; waited for below
  grid_dep_wait();
  grid_dep_launch();

  // This pair's share of the tiles. Selections all have the same number; otherwise thread i sums the tiles of the
  // queries [i * per, (i + 1) * per).
  long long count, first_tok, first_tile;
  if (SELECTED) {
    const uint32_t each = (uint32_t)(p.k + kTile - 1) / kTile;
    const long long total = p.BT * each, lo = total * pair / pairs;
    count = total * (pair + 1) / pairs - lo;
    first_tok = lo / each;
    first_tile = lo - first_tok * each;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    const int64_t per = (p.BT + kThreads - 1) / kThreads;
    const int64_t ua = min(p.BT, tid * per), ub = min(p.BT, ua + per);
    long long sum = 0;
    for (int64_t u = ua; u < ub; ++u) sum += tiles_of(p, u);
    long long pre = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, pre, d);
      if (lane >= d) pre += o;
    }
    if (lane == 31) scan_sh[warp] = pre;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long total = 0, base = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) base = total;
      total += scan_sh[w];
    }
    const long long excl = base + pre - sum;
    const long long lo = total * pair / pairs;
    count = total * (pair + 1) / pairs - lo;
    if (sum > 0 && lo >= excl && lo < excl + sum) {
      long long off = lo - excl;
      int64_t u = ua;
      for (; u < ub; ++u) {
        const int n = tiles_of(p, u);
        if (off < n) break;
        off -= n;
      }
      start_sh[0] = u;
      start_sh[1] = off;
    }
    __syncthreads();
    first_tok = start_sh[0];
    first_tile = start_sh[1];
  }
  cluster_wait();                        // both CTAs' barriers are initialised, both hold their TMEM
  const uint32_t tmem = tmem_base_sh;
  const uint32_t ring = smem_u32(smem + kOffRing);
  Runs r;
  r.start(p, first_tok, first_tile, count);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA: queries (64 heads a CTA), and dense keys
    if (elect_one()) {
      int slot = 0, run = 0;
      uint32_t ph = 1;                   // a fresh slot counts as freed
      bool ok = true;
      auto acquire = [&]() {
        if (!mbar_wait(&empty[slot], ph, &abort_flag, p.status, DSA_SITE_WEIGHTS_EMPTY)) ok = false;
        return ok;
      };
      auto advance = [&]() {
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1;
        }
      };
      for (; ok && r.left > 0; r.next(p), ++run) {
        if (run > 0 && !mbar_wait(q_empty, (run + 1) & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_EMPTY)) {
          ok = false;
          break;
        }
        const uint32_t q_bar = cluster_addr(q_full, 0);
        arrive_expect_tx_cluster(q_bar, 9 * kQBlock);
        for (int f = 0; f < 9; ++f)
          pair_load_2d(smem_u32(smem) + f * kQBlock, &q_map, q_bar, 64 * f, (int32_t)(r.tok * kHeads + 64 * rank));
        if (r.left > r.t1 - r.t0 && r.tok + 1 < p.BT)            // the next run's, into L2
          for (int i = 0; i < 9; ++i)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.q + ((r.tok + 1) * kHeads + 64 * rank) * kDqk + i * (kQBlock / 2)),
                         "r"(kQBlock)
                         : "memory");
        if (SELECTED) continue;
        const int b = (int)(r.tok / p.T);
        for (int t = r.t0; ok && t < r.t1; ++t)
          for (int part = 0; part < kParts && acquire(); ++part, advance()) {
            const uint32_t bar = cluster_addr(&full[slot], 0);
            const int row = t * kTile + rank * kRows;
            if (row < r.keys) {
              arrive_expect_tx_cluster(bar, kSlot);
              pair_load_4d(ring + slot * kSlot, &k_map, bar, 0, row, 3 * part, b);
            } else {
              arrive_cluster(bar);       // no key of the tile on this CTA: its scores are not used
            }
          }
      }
      // the last MMAs' arrivals have to reach this CTA before it leaves
      if (!SELECTED)
        for (int i = 0; i < kSlots && acquire(); ++i) advance();
      if (ok && run > 0) mbar_wait(q_empty, (run + 1) & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_EMPTY);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue, one thread of the leader
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_f32acc(1, 1, 256, kHeads, 0, 0);
      const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(smem)), k_desc = sdesc_kmajor_sw128(ring);
      int slot = 0, run = 0;
      uint32_t ph = 0, i = 0;               // parts issued
      bool ok = true;
      // the tiles of a run, a slot's 12 MMAs into one accumulator (PER = 1) or six each into two
      auto tiles = [&](auto per) {
        constexpr int PER = decltype(per)::value, kSteps = 12 / PER;
        for (int t = r.t0; ok && t < r.t1; ++t) {
#pragma unroll
          for (int part = 0; part < kParts * PER; ++part) {
            if (!ok || !mbar_wait(&acc_empty[i & 3], ((i >> 2) + 1) & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_ACC) ||
                (part % PER == 0 && !mbar_wait(&full[slot], ph, &abort_flag, p.status, DSA_SITE_WEIGHTS_FULL))) {
              ok = false;
              break;
            }
            if (SELECTED && part % PER == 0) cluster_fence();  // both CTAs' threads wrote this slot
            tc_fence_after();
            const uint64_t a = k_desc + (uint64_t)(slot * (kSlot >> 4)), b = q_desc + (uint64_t)(3 * (part / PER) * (kQBlock >> 4));
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              const int k = part % PER * kSteps + j;
              pair_mma_ss((i & 3) * kHeads, a + 2 * (k & 3) + (k >> 2) * (kBlock >> 4),
                          b + 2 * (k & 3) + (k >> 2) * (kQBlock >> 4), idesc, j > 0);
            }
            if (part % PER == PER - 1) pair_commit(&empty[slot], 3);
            pair_commit(&acc_full[i & 3], 3);
            ++i;
            if (part % PER == PER - 1 && ++slot == kSlots) {
              slot = 0;
              ph ^= 1;
            }
          }
        }
      };
      for (; ok && r.left > 0; r.next(p), ++run) {
        if (!mbar_wait(q_full, run & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_Q)) break;
        tc_fence_after();
        if (r.keys <= kFineKeys) tiles(std::integral_constant<int, 2>());
        else tiles(std::integral_constant<int, 1>());
        if (ok) pair_commit(q_empty, 3);
      }
    }
  } else if (SELECTED && warp == 2) {
    // ------------------------------------------------------------------ hands gathered slots to the leader
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; ok && r.left > 0; r.next(p))
      for (int i = 0; ok && i < kParts * (r.t1 - r.t0); ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&gathered[slot], ph, &abort_flag, p.status, DSA_SITE_WEIGHTS_FULL));
        if (!ok) break;
        fence_proxy_async_smem();        // cp.async writes -> MMA reads
        cluster_fence();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(&full[slot], 0));
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1;
        }
      }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ gather (selected rows)
    // warp v copies rows 32 v .. 32 v + 31 of this CTA's half of the tile: lane i holds the row number of row 32 v + i
    const int v = warp - 12;
    int slot = 0;
    uint32_t ph = 1;
    bool ok = true;
    auto acquire = [&]() {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&empty[slot], ph, &abort_flag, p.status, DSA_SITE_WEIGHTS_EMPTY));
      return ok;
    };
    auto advance = [&]() {
      if (++slot == kSlots) {
        slot = 0;
        ph ^= 1;
      }
    };
    for (; ok && r.left > 0; r.next(p)) {
      const uint16_t* kv = p.kv + r.tok / p.T * p.S_max * kDqk;
      const int32_t* idx = p.idx + r.tok * p.k;
      auto row_of = [&](int t) {
        const int u = t * kTile + rank * kRows + 32 * v + lane;
        const int row = t < r.t1 && u < p.k ? __ldg(idx + u) : -1;
        if (row >= p.S_max) set_status(p.status, DSA_ERR_DEVICE_BOUNDS);
        return row < p.S_max ? row : -1;
      };
      int row = row_of(r.t0);
      for (int t = r.t0; ok && t < r.t1; ++t) {
        const int next = row_of(t + 1);
        for (int part = 0; part < kParts && acquire(); ++part, advance()) {
          const uint32_t dst = ring + slot * kSlot;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // four rows per step, eight 16-byte chunks of each of three blocks; rows that take no part are zeros
            const int rr = 4 * i + (lane >> 3), c = lane & 7;
            const int src = __shfl_sync(0xffffffffu, row, rr);
            const int at = 32 * v + rr;
            const uint32_t to = dst + at * 128 + ((c ^ (at & 7)) << 4);
            const uint16_t* from = kv + (int64_t)max(src, 0) * kDqk + 192 * part + 8 * c;
#pragma unroll
            for (int j = 0; j < 3; ++j) cp_async_16_zfill(to + j * kBlock, from + 64 * j, src >= 0);
          }
          cp_async_mbar_arrive(&gathered[slot]);
        }
        row = next;
      }
    }
    cp_async_wait_all();
    // the last MMAs' arrivals have to reach this CTA before it leaves
    for (int i = 0; i < kSlots && acquire(); ++i) advance();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ exponentials, two threads per key, 64 heads each
    const int key = (tid - 128) & 127, half = (tid - 128) >> 7, quad = warp & 3;
    const uint32_t t_row = tmem + ((uint32_t)(quad * 32) << 16) + 64 * half;
    uint32_t g = 0, i = 0;               // tiles, parts
    int run = 0;
    bool ok = true;
    for (; ok && r.left > 0; r.next(p), ++run) {
      // the run's lse in units of log 2 (the four warps of a half write the same values). A part needs every
      // warp's release of the one four before it, so no warp gets more than two tiles ahead of another: four buffers.
      float* ls = lse_sh + (run & 3) * kHeads + 64 * half;
      const float2 l2 = __ldg(reinterpret_cast<const float2*>(p.lse + r.tok * kHeads + 64 * half) + lane);
      __syncwarp();
      *reinterpret_cast<float2*>(ls + 2 * lane) = make_float2(l2.x * kLog2e, l2.y * kLog2e);
      __syncwarp();
      const bool fine = r.keys <= kFineKeys;
      for (int t = r.t0; ok && t < r.t1; ++t, ++g) {
        const int u = t * kTile + rank * kRows + key;
        bool take = u < r.keys;
        int row = u;
        if (SELECTED && take) {
          row = __ldg(p.idx + r.tok * p.k + u);
          take = row >= 0 && row < p.S_max;
        }
        // dense, one query per sequence: the row's total is read ahead of the scores (the gathering kernel has no registers
        // left for it)
        const bool add = half == 0 && take && p.T == 1 && p.acc_out != nullptr;
        const float before = !SELECTED && add ? p.acc[r.tok * p.S_max + row] : 0.f;
        float z[64];
        auto read = [&](bool first) {                          // the next part's 64 scores
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&acc_full[i & 3], (i >> 2) & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_ACC));
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld32(t_row + (i & 3) * kHeads + 32 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              z[32 * c + j] = first ? __uint_as_float(x[j]) : z[32 * c + j] + __uint_as_float(x[j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(cluster_addr(&acc_empty[i & 3], 0));
          ++i;
        };
        read(true);
#pragma unroll
        for (int part = 1; part < kParts; ++part) read(false);
        if (fine)
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) read(false);
        if (!ok) break;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(ls + j);
          s4[0] += exp2_approx(fmaf(z[j], p.scale_log2, -l4.x));
          s4[1] += exp2_approx(fmaf(z[j + 1], p.scale_log2, -l4.y));
          s4[2] += exp2_approx(fmaf(z[j + 2], p.scale_log2, -l4.z));
          s4[3] += exp2_approx(fmaf(z[j + 3], p.scale_log2, -l4.w));
        }
        float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        float* other = sum_sh + (g & 1) * kRows + key;
        if (half == 1) {
          *other = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sum_full[4 * (g & 1) + quad]);
          continue;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sum_full[4 * (g & 1) + quad], (g >> 1) & 1, &abort_flag, p.status, DSA_SITE_WEIGHTS_ACC))) {
          ok = false;
          break;
        }
        sum = take ? sum + *other : 0.f;
        if (u < r.keys) p.w[r.tok * p.ld + u] = sum;
        // one query per sequence: no other weight meets this row's
        if (add) p.acc_out[r.tok * p.S_max + row] = (SELECTED ? p.acc[r.tok * p.S_max + row] : before) + sum;
      }
    }
  }
  if (!SELECTED && p.T == 1 && (warp == 2 || warp == 3)) {
    // One query per sequence: its hidden rows get their zeros here, and acc is done above. These two warps have nothing
    // else to do, but they are only 64 threads: where the lengths are far below S_max they bound the call (64 sequences
    // of about 1000 rows: 96 us in caches of 16384 rows, 37 us in caches of 1024).
    const int64_t n = p.BT * p.S_max;
    for (int64_t i = (int64_t)blockIdx.x * 64 + (warp - 2) * 32 + lane; i < n; i += (int64_t)gridDim.x * 64) {
      const int64_t tok = i / p.S_max;
      const int s = (int)(i - tok * p.S_max);
      if (s >= keys_of(p, tok)) {
        p.w[tok * p.ld + s] = 0.f;
        if (p.acc_out) p.acc_out[i] = p.acc[i];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                      // nothing of the pair is in flight towards a CTA that has left
  cluster_wait();
  if (warp == 2) pair_tmem_dealloc(tmem, 512);
}

// Dense, several queries per sequence: zeros behind each query's keys, and acc_out = acc + the weights
// of the queries. Each of 8 warps adds every eighth query for 32 rows, then the eight sums join in order.
__global__ void __launch_bounds__(256) mla_weights_sum_kernel(const WeightsParams p) {
  __shared__ float part[8][32];
  const int64_t b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.x * 32 + lane;
  grid_dep_wait();
  grid_dep_launch();
  const int len = min(__ldg(p.kv_len + b), p.S_max);
  float a = 0.f;
  if (s < p.S_max) {
    const int32_t* last = p.q_pos + b * p.T;
    float* w = p.w + b * p.T * p.ld + s;
#pragma unroll 4
    for (int t = warp; t < p.T; t += 8) {
      if (s < len && s <= __ldg(last + t)) {
        if (p.acc_out) a += w[t * p.ld];
      } else {
        w[t * p.ld] = 0.f;
      }
    }
  }
  part[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && s < p.S_max && p.acc_out) {
    a = p.acc[b * p.S_max + s];
    for (int i = 0; i < 8; ++i) a += part[i][lane];
    p.acc_out[b * p.S_max + s] = a;
  }
}

// Selected, one query per sequence: what nobody selected, ahead of the kernel that adds the rest.
__global__ void __launch_bounds__(256) mla_weights_copy_kernel(const float4* acc, float4* acc_out, int64_t n) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n / 4; i += stride) acc_out[i] = acc[i];
  if (blockIdx.x == 0 && threadIdx.x < n % 4)
    reinterpret_cast<float*>(acc_out)[n - 1 - threadIdx.x] = reinterpret_cast<const float*>(acc)[n - 1 - threadIdx.x];
}

// Selected, several queries per sequence: acc_out = acc + their weights, in their order; a block holds kRange positions of
// one sequence in shared memory. Positions of one query are distinct, so no two threads meet. The queries follow one
// another, with a barrier each, on a block per 4096 positions: for one sequence this takes longer than the weights
// themselves (256 queries of 2048 out of 16384 rows: 113 us without it, 329 with it; 2048 queries: 725 and 3390).
constexpr int kRange = 4096;
__global__ void __launch_bounds__(1024) mla_weights_scatter_kernel(const WeightsParams p) {
  __shared__ float a[kRange];
  const int64_t b = blockIdx.y;
  const int s0 = blockIdx.x * kRange, n = min(kRange, p.S_max - s0);
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < n; i += 1024) a[i] = p.acc[b * p.S_max + s0 + i];
  __syncthreads();
  for (int t = 0; t < p.T; ++t) {
    const int64_t q = b * p.T + t;
    for (int u = threadIdx.x; u < p.k; u += 1024) {
      const int i = __ldg(p.idx + q * p.k + u) - s0;
      if (i >= 0 && i < n) a[i] += p.w[q * p.ld + u];
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += 1024) p.acc_out[b * p.S_max + s0 + i] = a[i];
}

namespace {

template <bool SELECTED>
int launch_weights(const uint16_t* q, const WeightsParams& p, int64_t B, cudaStream_t stream) {
  const auto dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap q_map, k_map;
  const uint64_t row = kDqk * 2;
  if (!dsa_host::encode_tensor_map_2d(&q_map, dt, const_cast<uint16_t*>(q), kDqk, (uint64_t)p.BT * kHeads, row, 64, 64, sw))
    return DSA_ERR_CUDA;
  k_map = q_map;
  if (!SELECTED) {
    // feature, row, block of 64 features, sequence: one box is three blocks of 128 rows, block by block
    const uint64_t dims[4] = {64, (uint64_t)p.S_max, 9, (uint64_t)B}, strides[3] = {row, 128, row * (uint64_t)p.S_max};
    const uint32_t box[4] = {64, kRows, 3, 1};
    if (!dsa_host::encode_tensor_map(&k_map, dt, 4, const_cast<uint16_t*>(p.kv), dims, strides, box, sw)) return DSA_ERR_CUDA;
  }
  static uint64_t seen[dsa_host::kMaxSetupDevices];
  if (dsa_host::needs_setup(seen, nullptr)) {
    if (cudaFuncSetAttribute(mla_weights_kernel<SELECTED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return DSA_ERR_CUDA;
    dsa_host::mark_setup(seen);
  }
  if (SELECTED && p.T == 1 && p.acc_out && p.acc_out != p.acc) {
    const int64_t n = B * p.S_max;
    const int rc = dsa_host::launch(mla_weights_copy_kernel, dim3((unsigned)std::min<int64_t>((n / 4 + 255) / 256 + 1, 1024)),
                                    dim3(256), 0, stream, reinterpret_cast<const float4*>(p.acc),
                                    reinterpret_cast<float4*>(p.acc_out), n);
    if (rc != DSA_OK) return rc;
  }
  const int64_t tiles = p.BT * (((SELECTED ? p.k : p.S_max) + kTile - 1) / kTile);
  const unsigned pairs = (unsigned)std::min<int64_t>(dsa_host::device_sm_count() / 2, tiles);
  const int rc = dsa_host::launch_clusters(mla_weights_kernel<SELECTED>, 2, pairs, SELECTED ? 512 : 384, kSmem, stream, q_map,
                                           k_map, p);
  if (rc != DSA_OK) return rc;
  if (p.T == 1) return DSA_OK;
  if (!SELECTED)
    return dsa_host::launch(mla_weights_sum_kernel, dim3((unsigned)((p.S_max + 31) / 32), (unsigned)B), dim3(256), 0, stream, p);
  if (!p.acc_out) return DSA_OK;
  return dsa_host::launch(mla_weights_scatter_kernel, dim3((unsigned)((p.S_max + kRange - 1) / kRange), (unsigned)B),
                          dim3(1024), 0, stream, p);
}

}  // namespace

int launch_mla_weights(const uint16_t* q, const uint16_t* kv, const int32_t* idx, const float* lse, const int32_t* q_pos,
                       const int32_t* kv_len, int B, int T, int S_max, int k, float softmax_scale, float* w, int64_t ld,
                       const float* acc, float* acc_out, cudaStream_t stream, int* status) {
  WeightsParams p = {};
  p.q = q;
  p.kv = kv;
  p.idx = idx;
  p.lse = lse;
  p.q_pos = q_pos;
  p.kv_len = kv_len;
  p.BT = (int64_t)B * T;
  p.T = T;
  p.S_max = S_max;
  p.k = k;
  p.ld = ld;
  p.scale_log2 = softmax_scale * kLog2e;
  p.w = w;
  p.acc = acc;
  p.acc_out = acc_out;
  p.status = status;
  return idx ? launch_weights<true>(q, p, B, stream) : launch_weights<false>(q, p, B, stream);
}

}  // namespace dsa
