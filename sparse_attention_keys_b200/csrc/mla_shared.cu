// dsa_mla_shared: dense latent attention of a batch whose sequences share a prefix of the cache.
//
// For query (b, t) and head h the visible keys are the P rows of the prefix and the first vis rows
// of sequence b's own cache (vis = min(q_pos + 1, kv_len)): z = scale * q . key over 576 features,
// out = softmax(z) . key[0:512], lse = ln sum e^z. The prefix is stored once and its tiles are
// multiplied with the queries of every sequence, so its part is a matrix product with B*T*128 rows.
//
// Work. Two tokens (256 rows of q) form a unit; a CTA pair (cta_group::2, M = 256, one token per
// CTA) accumulates one half (256 features) of the unit's output, since 128 x 512 fp32 would fill
// the whole TMEM and leave none for the scores. So the scores are computed by both halves: 832
// instead of 544 multiply-adds per (row, key, CTA pair), the price of keeping O in TMEM. A unit's
// keys are the prefix, then the own rows of its token(s), in tiles of 128, all accumulated into one
// O with a running maximum and sum. The tiles of all (unit, half) items in a row are cut into equal
// ranges, one per CTA pair; an item that a cut divides leaves fp32 partials in the workspace, which
// a second kernel joins. Every pair holds at most two such pieces, so the workspace is bounded
// whatever the lengths are, and the device alone reads the lengths.
//
// Per CTA: Q (128 x 576, 144 KB) stays in shared memory; K and V stream through one ring of 16 KB
// slots of 64 keys x 128 features in the order the MMAs consume them (K: this CTA's half of the
// tile's keys, five slots; V: its half of the 256 output features, two slots). TMEM: O [0, 256),
// two score buffers of 128 columns; the probabilities (bf16) replace the scores they came from and
// are the A operand of P V. Q K^T of tile j + 1 runs while the softmax of tile j does.
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "pair.cuh"

namespace dsa {

namespace {

constexpr int kHeads = 128;
constexpr int kDqk = 576, kDv = 512;
constexpr int kTile = 128;                         // keys per tile
constexpr int kQBlock = kHeads * 128;              // 16 KB: 64 features of 128 rows
constexpr int kQBytes = 9 * kQBlock;
constexpr int kSlot = 16384;                       // 64 keys x two blocks of 64 features
constexpr int kSlots = 5;
constexpr int kOffRing = kQBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlot;
constexpr int kSmem = 1024 + kOffBar + 512;
static_assert(kSmem <= 232448, "shared memory per CTA");
constexpr int kThreads = 256;
constexpr uint32_t kTmemS = 256;                   // O in [0, 256), scores in 2 x 128 columns
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum moves, and O is rescaled, only when a tile exceeds it by 2^32: P stays below
// 2^32, where bf16 has its full relative precision, and the sums stay far inside fp32.
constexpr float kRescale = 32.0f;

}  // namespace

struct SharedParams {
  const uint16_t* kv;
  const int32_t* q_pos;
  const int32_t* kv_len;
  int BT, T, P, S_max;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* info;       // [pairs][2]: the item continued from the previous pair, the item cut at the end (-1: none)
  float* part_ml;      // [pairs][2][256][2]: maximum (log2 units), sum
  float* part_o;       // [pairs][2][64][256][4]: feature group, row, feature
  int* status;
};

namespace {

// Two tokens and their keys, in tiles: the prefix, then the own rows of token A's sequence (of both
// tokens when they share it), then those of token B's.
struct Unit {
  int bA, bB, visA, visB;
  int ptiles, tilesA, tiles;
  bool same, hasB;
};

__device__ __forceinline__ int visible(const SharedParams& p, int tok, int b) {
  if (p.S_max == 0) return 0;
  const int last = __ldg(p.q_pos + tok), n = __ldg(p.kv_len + b);
  return max(0, min(min(last, p.S_max - 1) + 1, n));
}

__device__ __forceinline__ Unit load_unit(const SharedParams& p, int u) {
  Unit x;
  const int ta = 2 * u, tb = ta + 1;
  x.hasB = tb < p.BT;
  x.bA = ta / p.T;
  x.bB = x.hasB && tb == (x.bA + 1) * p.T ? x.bA + 1 : x.bA;
  x.same = x.bA == x.bB;
  x.visA = visible(p, ta, x.bA);
  x.visB = x.hasB ? visible(p, tb, x.bB) : 0;
  x.ptiles = (p.P + kTile - 1) / kTile;
  const int va = x.same ? max(x.visA, x.visB) : x.visA;
  x.tilesA = (va + kTile - 1) / kTile;
  const int tb_tiles = x.same ? 0 : (x.visB + kTile - 1) / kTile;
  x.tiles = max(1, x.ptiles + x.tilesA + tb_tiles);   // a unit without keys still has its zeros to write
  return x;
}

struct Tile {
  int src;             // -1: the prefix, else the sequence
  int k0;              // first key
  int nA, nB;          // keys of the tile that token A / B sees
  __device__ __forceinline__ int most() const { return max(nA, nB); }
};

__device__ __forceinline__ int clamp_tile(int v) { return max(0, min(kTile, v)); }

__device__ __forceinline__ Tile get_tile(const SharedParams& p, const Unit& x, int t) {
  Tile r;
  if (t < x.ptiles) {
    r.src = -1;
    r.k0 = t * kTile;
    r.nA = clamp_tile(p.P - r.k0);
    r.nB = x.hasB ? r.nA : 0;
  } else if (t - x.ptiles < x.tilesA) {
    r.src = x.bA;
    r.k0 = (t - x.ptiles) * kTile;
    r.nA = clamp_tile(x.visA - r.k0);
    r.nB = x.same ? clamp_tile(x.visB - r.k0) : 0;
  } else {
    r.src = x.bB;
    r.k0 = (t - x.ptiles - x.tilesA) * kTile;
    r.nA = 0;
    r.nB = clamp_tile(x.visB - r.k0);
  }
  return r;
}

// The pieces of a pair's range of tiles, one item after the other; every role walks it for itself.
struct Walk {
  int64_t left;        // tiles left in the range
  int u;
  int half, t0, t1;    // the piece: tiles [t0, t1) of (u, half)
  Unit x;
  __device__ __forceinline__ void start(const SharedParams& p, int unit, int64_t off, int64_t count) {
    left = count;
    u = unit;
    if (left <= 0) return;
    x = load_unit(p, u);
    half = off >= x.tiles;
    t0 = (int)(off - (half ? x.tiles : 0));
    t1 = (int)min((int64_t)x.tiles, t0 + left);
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next(const SharedParams& p) {
    left -= t1 - t0;
    if (left <= 0) return;
    if (half) {
      ++u;
      x = load_unit(p, u);
    }
    half ^= 1;
    t0 = 0;
    t1 = (int)min((int64_t)x.tiles, left);
  }
};

// Rows [row, row + 64) of a tile's source, feature blocks [block, block + 2) of 64: [block][row][64]
__device__ __forceinline__ void load_slot(const CUtensorMap* pmap, const CUtensorMap* smap, int src, int row, int block,
                                          uint32_t dst, uint32_t bar) {
  if (src < 0) pair_load_3d(dst, pmap, bar, 0, row, block);
  else pair_load_4d(dst, smap, bar, 0, row, block, src);
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    mla_shared_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap p_map,
                      const __grid_constant__ CUtensorMap s_map, const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // both CTAs of a pair see the same offsets: the MMA reads them with one descriptor
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* full = bars;                 // leader: both CTAs' parts of the slot have landed
  uint64_t* empty = full + kSlots;       // both: the MMAs that read the slot are done
  uint64_t* s_full = empty + kSlots;     // both [2]: scores ready
  uint64_t* p_full = s_full + 2;         // leader [2]: probabilities of both CTAs written
  uint64_t* pv_done = p_full + 2;        // both [2]: P V of the tile done
  uint64_t* q_full = pv_done + 2;        // leader [5]: two blocks of 64 features of both CTAs' Q landed
  uint64_t* q_empty = q_full + 5;        // both: the piece's Q K^T done
  uint64_t* o_free = q_empty + 1;        // leader: both CTAs have read O
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ long long scan_sh[kThreads / 32];
  __shared__ long long start_sh[2];      // first unit of this pair's range, offset in its 2 x tiles

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = pair_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 5; ++i) mbar_init(&q_full[i], 2);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 8);
    fence_barrier_init();
  }
  if (warp == 2) pair_tmem_alloc(&tmem_base_sh, 512);
  __syncwarp();
  pair_arrive();                         // this thread's part of the set-up; waited for below
  grid_dep_wait();                       // lengths, queries and caches may come from the preceding kernel
  grid_dep_launch();

  // The pair's range of tiles: thread i sums the units [i * per, (i + 1) * per).
  const int units = (p.BT + 1) / 2;
  const int per = (units + kThreads - 1) / kThreads;
  const int ua = min(units, tid * per), ub = min(units, ua + per);
  long long sum = 0;
  for (int u = ua; u < ub; ++u) sum += 2 * load_unit(p, u).tiles;
  long long pre = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, pre, d);
    if (lane >= d) pre += o;
  }
  if (lane == 31) scan_sh[warp] = pre;
  if (tid == 0) start_sh[0] = start_sh[1] = 0;
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
  // no more pairs than tiles: the join walks over consecutive pairs, none of them without a tile
  const int active = (int)min((long long)pairs, total);
  const long long share = total < (1ll << 31) ? (long long)((uint32_t)total / (uint32_t)active) : total / active;
  const int rest = (int)(total - share * active);
  const long long lo = pair < active ? share * pair + min(pair, rest) : total;
  const long long count = pair < active ? share + (pair < rest) : 0;
  if (sum > 0 && lo >= excl && lo < excl + sum) {
    long long off = lo - excl;
    int u = ua;
    if (per > 1)
      for (; u < ub; ++u) {
        const long long n = 2 * load_unit(p, u).tiles;
        if (off < n) break;
        off -= n;
      }
    start_sh[0] = u;
    start_sh[1] = off;
  }
  __syncthreads();
  pair_wait();                           // barriers of both CTAs are initialised, both hold their TMEM
  const uint32_t tmem = tmem_base_sh;
  Walk w;
  w.start(p, (int)start_sh[0], start_sh[1], count);

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------------ loads
    // Waiting for a slot and issuing its load take one warp about 400 cycles, more than the MMAs of a
    // block (260): three warps take the blocks in turn (shared_chunk 3059 -> 0 us).
    const int mine = warp == 0 ? 0 : warp - 1;
    int turn = 0;
    const bool el = elect_one();
    const uint32_t ring = smem_u32(smem + kOffRing);
    int slot = 0, round = 0;
    bool ok = true;
    auto acquire = [&]() {
      if (round > 0 && !mbar_wait(&empty[slot], (round + 1) & 1, &abort_flag, p.status, DSA_SITE_SHARED_EMPTY))
        ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    auto advance = [&]() {
      if (++slot == kSlots) {
        slot = 0;
        ++round;
      }
      if (++turn == 3) turn = 0;
    };
    auto k_tile = [&](const Tile& t, bool first) {
      for (int f = 0; ok && f < 9; f += 2, advance()) {
        if (turn != mine) continue;
        acquire();
        if (!ok) break;
        if (el) {
          if (first) {                                   // with the first keys, the same features of Q
            const uint32_t qbar = leader_addr(&q_full[f / 2]);
            arrive_expect_tx_cluster(qbar, f < 8 ? 2 * kQBlock : kQBlock);
            for (int i = f; i < min(f + 2, 9); ++i)
              pair_load_2d(smem_u32(smem) + i * kQBlock, &q_map, qbar, 64 * i, (2 * w.u + (int)rank) * kHeads);
          }
          const uint32_t bar = leader_addr(&full[slot]);
          arrive_expect_tx_cluster(bar, kSlot);          // there is no block 9: zeros
          load_slot(&p_map, &s_map, t.src, t.k0 + 64 * (int)rank, f, ring + slot * kSlot, bar);
        }
      }
    };
    auto v_tile = [&](const Tile& t, int half) {
      const int n = t.most();
      for (int kb = 0; ok && kb < n; kb += 64, advance()) {
        if (turn != mine) continue;
        acquire();
        if (!ok) break;
        const uint32_t dst = ring + slot * kSlot, bar = leader_addr(&full[slot]);
        const int block = 4 * half + 2 * (int)rank;
        if (t.src < 0 || n - kb >= 64) {
          if (el) {
            arrive_expect_tx_cluster(bar, kSlot);
            load_slot(&p_map, &s_map, t.src, t.k0 + kb, block, dst, bar);
          }
        } else {
          // the rows behind the last visible key may hold anything, and 0 * NaN is NaN: the warp
          // copies the visible rows itself and puts zeros behind them
          const uint16_t* src = p.kv + ((int64_t)t.src * p.S_max + t.k0 + kb) * kDqk + 64 * block;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint4 v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = 32 * h + 2 * i + (lane >> 4), c = lane & 15;    // row, 16-byte chunk of its 256 bytes
              v[i] = r < n - kb ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * kDqk) + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = 32 * h + 2 * i + (lane >> 4), c = lane & 15;
              const uint32_t a = dst + 8192 * (c >> 3) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[i].x), "r"(v[i].y), "r"(v[i].z),
                           "r"(v[i].w)
                           : "memory");
            }
          }
          fence_proxy_async_smem();
          cluster_fence();
          __syncwarp();
          if (el) arrive_cluster(bar);
        }
      }
    };
    int piece = 0;
    for (; ok && w.valid(); w.next(p)) {
      if (get_tile(p, w.x, w.t0).most() == 0) continue;          // a unit without keys
      if (piece > 0) {
        if (!mbar_wait(q_empty, (piece + 1) & 1, &abort_flag, p.status, DSA_SITE_SHARED_EMPTY)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      ++piece;
      Tile prev = get_tile(p, w.x, w.t0);
      k_tile(prev, true);
      for (int t = w.t0 + 1; ok && t < w.t1; ++t) {
        const Tile cur = get_tile(p, w.x, t);
        k_tile(cur, false);
        v_tile(prev, w.half);
        prev = cur;
      }
      if (ok) v_tile(prev, w.half);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue: one thread of the leader
    if (rank == 0 && elect_one()) {
      const uint32_t idesc_s = idesc_f32acc(1, 1, 256, kTile, 0, 0);
      const uint32_t idesc_o = idesc_f32acc(1, 1, 256, 256, 0, 1);
      const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(smem));
      const uint64_t k_desc = sdesc_kmajor_sw128(smem_u32(smem + kOffRing));
      const uint64_t v_desc = sdesc_mnmajor_sw128(smem_u32(smem + kOffRing), 8192, 1024);
      int slot = 0, piece = 0;
      uint32_t ph = 0, g = 0;             // ring phase, tiles so far
      bool ok = true;
      auto wait_full = [&]() {
        if (!mbar_wait(&full[slot], ph, &abort_flag, p.status, DSA_SITE_SHARED_FULL)) ok = false;
        tc_fence_after();
      };
      auto advance = [&]() {
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1;
        }
      };
      auto qk = [&](uint32_t buf, bool first) {
        const uint32_t d = tmem + kTmemS + buf * kTile;
#pragma unroll
        for (int f = 0; f < 9; f += 2) {
          if (ok && first && !mbar_wait(&q_full[f / 2], piece & 1, &abort_flag, p.status, DSA_SITE_SHARED_Q)) ok = false;
          if (ok) wait_full();
          if (!ok) break;
          const uint64_t a = q_desc + (uint64_t)((f * kQBlock) >> 4), b = k_desc + (uint64_t)((slot * kSlot) >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (f + (k >> 2) < 9)
              pair_mma_ss(d, a + 2 * (k & 3) + (k >> 2) * (kQBlock >> 4), b + 2 * (k & 3) + (k >> 2) * (8192 >> 4), idesc_s,
                          (f | k) != 0);
          pair_commit(&empty[slot]);
          advance();
        }
        if (ok) pair_commit(&s_full[buf]);
      };
      for (; ok && w.valid(); w.next(p)) {
        Tile cur = get_tile(p, w.x, w.t0);
        if (cur.most() == 0) continue;
        bool startedA = false, startedB = false;
        qk(g & 1, true);
        for (int t = w.t0; ok && t < w.t1; ++t, ++g) {
          if (t + 1 < w.t1) qk((g + 1) & 1, false);
          else pair_commit(q_empty);
          if (!ok) break;
          cur = get_tile(p, w.x, t);
          // the token that sees nothing of the tile keeps its O
          const uint32_t off0 = cur.nA > 0 ? 0u : 0xffffffffu, off1 = cur.nB > 0 ? 0u : 0xffffffffu;
          bool acc = (cur.nA > 0 && startedA) || (cur.nB > 0 && startedB);
          startedA |= cur.nA > 0;
          startedB |= cur.nB > 0;
          const int n = cur.most();
          const uint32_t a = tmem + kTmemS + (g & 1) * kTile;
          if (t == w.t0 && piece > 0 && !mbar_wait(o_free, (piece + 1) & 1, &abort_flag, p.status, DSA_SITE_SHARED_O))
            ok = false;
          if (!ok || !mbar_wait(&p_full[g & 1], (g >> 1) & 1, &abort_flag, p.status, DSA_SITE_SHARED_P)) ok = false;
          tc_fence_after();
          for (int kb = 0; ok && kb < n; kb += 64) {
            wait_full();
            if (!ok) break;
            const bool part = n - kb < 64;
            if (cur.src >= 0 && part) cluster_fence();               // both CTAs' warps wrote this slot
            const uint64_t b = v_desc + (uint64_t)((slot * kSlot) >> 4);
            if ((off0 | off1) == 0 && !part) {
#pragma unroll
              for (int k = 0; k < 4; ++k) pair_mma_ts(tmem, a + kb / 2 + 8 * k, b + 128 * k, idesc_o, acc || k > 0);
            } else {
              for (int k = 0; k < 4 && kb + 16 * k < n; ++k)
                pair_mma_ts_masked(tmem, a + kb / 2 + 8 * k, b + 128 * k, idesc_o, off0, off1, acc || k > 0);
            }
            pair_commit(&empty[slot]);
            acc = true;
            advance();
          }
          if (ok) pair_commit(&pv_done[g & 1]);
        }
        ++piece;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax, one thread per row
    const int row = tid - 128;            // head; TMEM lane
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t g = 0;
    bool ok = true;
    int32_t info_cont = -1, info_head = -1;
    for (; ok && w.valid(); w.next(p)) {
      const int tok = 2 * w.u + (int)rank;
      float m = -INFINITY, l = 0.f;
      bool any = false;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        const Tile tile = get_tile(p, w.x, t);
        if (tile.most() == 0) continue;
        const int n = rank == 0 ? tile.nA : tile.nB;
        const uint32_t buf = g & 1, ph = (g >> 1) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[buf], ph, &abort_flag, p.status, DSA_SITE_SHARED_S))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (n > 0) {
          uint32_t r[4][32];
          const uint32_t s = t_row + kTmemS + buf * kTile;
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s + 32 * c, r[c]);
          tmem_ld_wait();
          if (n < kTile) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= n) r[c][i] = 0xff800000u;
          }
          float mx4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx4[c] = __uint_as_float(r[c][0]);
#pragma unroll
            for (int i = 1; i < 32; ++i) mx4[c] = fmaxf(mx4[c], __uint_as_float(r[c][i]));
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m + kRescale) {
            alpha = exp2_approx(m - mx);  // 0 for the first
            rescale = m != -INFINITY;
            m = mx;
          }
          const float mm = m == -INFINITY ? 0.f : m;   // every score -inf: e^-inf = 0, not NaN
          float sum4[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[2][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float e0 = exp2_approx(fmaf(__uint_as_float(r[c][i]), p.scale_log2, -mm));
              const float e1 = exp2_approx(fmaf(__uint_as_float(r[c][i + 1]), p.scale_log2, -mm));
              sum4[(i >> 1) & 3] += e0 + e1;
              pk[c >> 1][(c & 1) * 16 + i / 2] = pack_bf16(e0, e1);
            }
          }
          l = l * alpha + ((sum4[0] + sum4[1]) + (sum4[2] + sum4[3]));
          if (__any_sync(0xffffffffu, rescale)) {
            // P V of every earlier tile has to be in O first
            if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &abort_flag,
                                                           p.status, DSA_SITE_SHARED_O))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[32];
              tmem_ld32(t_row + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (rescale ? alpha : 1.f));
              tmem_st32(t_row + 32 * c, o);
            }
          }
          any = true;
          tmem_st32(s, pk[0]);
          tmem_st32(s + 32, pk[1]);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(leader_addr(&p_full[buf]));
        ++g;
      }
      if (!ok) break;
      // ---- the piece is done: output, or a partial for the join
      const bool whole = w.t0 == 0 && w.t1 == w.x.tiles;
      const int where = w.t0 == 0 ? 1 : 0;
      if (!whole) (where ? info_head : info_cont) = 2 * w.u + w.half;
      const bool had = get_tile(p, w.x, w.t0).most() > 0;
      if (had) {
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &abort_flag, p.status,
                                                       DSA_SITE_SHARED_O))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const int64_t slot = (int64_t)pair * 2 + where;
      const int prow = (int)rank * kHeads + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (whole) {
        if (tok < p.BT && w.half == 0 && p.lse)
          p.lse[(int64_t)tok * kHeads + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float2*>(p.part_ml + (slot * 256 + prow) * 2) = make_float2(m, l);
      }
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[32];
        if (any) {
          tmem_ld32(t_row + 32 * c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (whole) {
          if (tok < p.BT) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)tok * kHeads + row) * kDv + 256 * w.half + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 v;
              v.x = pack_bf16(__uint_as_float(o[8 * i]) * inv, __uint_as_float(o[8 * i + 1]) * inv);
              v.y = pack_bf16(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv);
              v.z = pack_bf16(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv);
              v.w = pack_bf16(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv);
              dst[i] = v;
            }
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o) + (slot * 64 + 8 * c) * 256 + prow;
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i * 256] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (had) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(leader_addr(o_free));
      }
    }
    if (rank == 0 && tid == 128) {
      p.info[2 * pair] = info_cont;
      p.info[2 * pair + 1] = info_head;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pair_barrier();                        // nothing of the pair is still in flight towards either CTA
  if (warp == 2) pair_tmem_dealloc(tmem, 512);
}

// Joins the pieces of items that were cut: block (p, y) takes 32 rows x 64 features of the item whose
// first piece is the last one of pair p; the pieces that follow are the first ones of the next pairs.
__global__ void __launch_bounds__(256) mla_shared_join_kernel(const SharedParams p, int pairs) {
  extern __shared__ float2 ml_sh[];      // [pieces][32 rows]: maximum, sum
  const int pair = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int item = __ldcg(p.info + 2 * pair + 1);
  if (item < 0) return;
  const int row = (blockIdx.y >> 2) * 32 + lane, col = (blockIdx.y & 3) * 64 + 8 * warp;
  const int tok = 2 * (item >> 1) + (row >> 7);
  const int head = row & 127, half = item & 1;
  if (tok >= p.BT) return;               // the same for the whole block
  int n = 1;                             // pieces
  for (int q = pair + 1; q < pairs; q += 32) {
    const uint32_t other = __ballot_sync(0xffffffffu, q + lane >= pairs || __ldcg(p.info + 2 * (q + lane)) != item);
    n += other ? __ffs(other) - 1 : 32;
    if (other) break;
  }
  auto slot_of = [&](int i) { return i == 0 ? (int64_t)pair * 2 + 1 : (int64_t)(pair + i) * 2; };
  for (int i = warp; i < n; i += 8)
    ml_sh[i * 32 + lane] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(i) * 256 + row);
  __syncthreads();
  float m = -INFINITY, l = 0.f;
  for (int i = 0; i < n; ++i) m = fmaxf(m, ml_sh[i * 32 + lane].x);
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  const float4* src = reinterpret_cast<const float4*>(p.part_o) + (int64_t)(col / 4) * 256 + row;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = ml_sh[i * 32 + lane];
    // a piece without a visible key has sum 0 and no maximum
    const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - m);
    l += ml.y * f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 v = __ldcg(src + slot_of(i) * (64 * 256) + j * 256);
      acc[j].x = fmaf(v.x, f, acc[j].x);
      acc[j].y = fmaf(v.y, f, acc[j].y);
      acc[j].z = fmaf(v.z, f, acc[j].z);
      acc[j].w = fmaf(v.w, f, acc[j].w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t out_row = (int64_t)tok * kHeads + head;
  *reinterpret_cast<uint4*>(p.out + out_row * kDv + 256 * half + col) =
      make_uint4(pack_bf16(acc[0].x * inv, acc[0].y * inv), pack_bf16(acc[0].z * inv, acc[0].w * inv),
                 pack_bf16(acc[1].x * inv, acc[1].y * inv), pack_bf16(acc[1].z * inv, acc[1].w * inv));
  if (col == 0 && half == 0 && p.lse) p.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

namespace {

// Pairs of the launch: one per two SMs, at most one per tile.
int shared_pairs(int64_t BT, int T, int P, int S_max) {
  const int64_t units = (BT + 1) / 2;
  const int64_t own = (S_max + kTile - 1) / kTile;
  const int64_t tiles = std::max<int64_t>(1, (P + kTile - 1) / kTile + 2 * own);
  return (int)std::max<int64_t>(1, std::min<int64_t>(dsa_host::device_sm_count() / 2, 2 * units * tiles));
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t mla_shared_workspace_size(int B, int T, int P, int S_max) {
  const size_t pairs = (size_t)shared_pairs((int64_t)B * T, T, P, S_max);
  return align256(pairs * 8) + pairs * 2 * 256 * 8 + pairs * 2 * 64 * 256 * 16;
}

int launch_mla_shared(const uint16_t* q, const uint16_t* prefix, int P, const uint16_t* kv, const int32_t* q_pos,
                      const int32_t* kv_len, int B, int T, int S_max, float softmax_scale, uint16_t* out, float* lse,
                      void* workspace, size_t ws_bytes, cudaStream_t stream, int* status) {
  if (!workspace || ws_bytes < mla_shared_workspace_size(B, T, P, S_max)) return DSA_ERR_WORKSPACE;
  SharedParams p;
  p.kv = kv;
  p.q_pos = q_pos;
  p.kv_len = kv_len;
  p.BT = B * T;
  p.T = T;
  p.P = P;
  p.S_max = S_max;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.status = status;
  const int pairs = shared_pairs(p.BT, T, P, S_max);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.info = reinterpret_cast<int32_t*>(ws);
  ws += align256((size_t)pairs * 8);
  p.part_ml = reinterpret_cast<float*>(ws);
  ws += (size_t)pairs * 2 * 256 * 8;
  p.part_o = reinterpret_cast<float*>(ws);

  const auto dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t row = kDqk * 2;
  CUtensorMap q_map, pm, sm;
  if (!dsa_host::encode_tensor_map_2d(&q_map, dt, const_cast<uint16_t*>(q), kDqk, (uint64_t)p.BT * kHeads, row, 64, kHeads,
                                      sw))
    return DSA_ERR_CUDA;
  pm = sm = q_map;                                   // an empty source is never loaded from
  // feature, row, block of 64 features (, sequence): one box is two blocks of 64 rows, block by block
  const uint32_t box[4] = {64, 64, 2, 1};
  if (P > 0) {
    const uint64_t dims[3] = {64, (uint64_t)P, 9}, strides[2] = {row, 128};
    if (!dsa_host::encode_tensor_map(&pm, dt, 3, const_cast<uint16_t*>(prefix), dims, strides, box, sw)) return DSA_ERR_CUDA;
  }
  if (S_max > 0) {
    const uint64_t dims[4] = {64, (uint64_t)S_max, 9, (uint64_t)B}, strides[3] = {row, 128, row * (uint64_t)S_max};
    if (!dsa_host::encode_tensor_map(&sm, dt, 4, const_cast<uint16_t*>(kv), dims, strides, box, sw)) return DSA_ERR_CUDA;
  }
  static uint64_t seen[dsa_host::kMaxSetupDevices];
  if (dsa_host::needs_setup(seen, nullptr)) {
    if (cudaFuncSetAttribute(mla_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return DSA_ERR_CUDA;
    dsa_host::mark_setup(seen);
  }
  int rc = dsa_host::launch_pairs(mla_shared_kernel, (unsigned)pairs, kThreads, kSmem, stream, q_map, pm, sm, p);
  if (rc != DSA_OK) return rc;
  return dsa_host::launch(mla_shared_join_kernel, dim3((unsigned)pairs, 32), dim3(256), (size_t)pairs * 32 * 8, stream, p, pairs);
}

}  // namespace dsa
