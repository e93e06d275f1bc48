// dsa_mla_shared: dense latent attention of a batch whose sequences share a prefix of the cache.
//
// For query (b, t) and head h the visible keys are the P rows of the prefix and the first vis rows
// of sequence b's own cache (vis = min(q_pos + 1, kv_len)): z = scale * q . key over 576 features,
// out = softmax(z) . key[0:512], lse = ln sum e^z. The prefix is stored once and its tiles are
// multiplied with the queries of every sequence, so its part is a matrix product with B*T*128 rows.
//
// Work. Two tokens (256 rows of q) form a unit. Its keys are the prefix, then the own rows of its
// token(s), in tiles of 128, all accumulated into one output with a running maximum and sum. A
// 128 x 512 fp32 output fills a whole TMEM and leaves none for scores, so a unit runs on a cluster of
// four CTAs, two tcgen05 pairs (M = 256, one token per CTA of a pair): the score pair (ranks 0, 1)
// computes Q K^T and the softmax, the value pair (ranks 2, 3) holds the output and computes P V. Per
// tile that is 36 MMAs of 256 x 128 x 16 (2306 cycles) against 16 of 256 x 256 x 16 (2052), side by
// side: nothing is computed twice. (Before, two pairs held half of the output each and both computed
// the scores: 3330 cycles per tile, and 1.53 times the arithmetic of this power-bound kernel.)
// The probabilities go from the score CTA's shared memory into its value CTA's with bulk copies that
// count on the receiver's barrier, with the factor by which the running maximum moved.
//
// The tiles of all units in a row are cut into equal ranges, one per cluster; a unit that a cut
// divides leaves fp32 partials in the workspace, which a second kernel joins. Every cluster holds at
// most two such pieces, so the workspace is bounded whatever the lengths are, and the device alone
// reads the lengths.
//
// Measured: 2620 cycles a tile, 88% of it the score pair's MMAs. 512 queries over 16384 shared rows take 1.92 ms,
// 1.23 PFLOP/s (75% of the measured matrix rate; the clock falls under the power limit), 64 queries over 8192
// shared and up to 512 own rows 144 us. 33 clusters of four fit, which leaves 16 SMs idle, and with 32 units 20. A tile
// of one sequence's own rows is multiplied with both tokens' rows although the other token's are thrown away, so own
// rows of different sequences run at half the matrix rate.
//
// The probabilities are rounded to bf16, the type of the values, for P V: an MMA takes both operands in one type.
// Their row sum is taken in fp32 before that. It is what the outputs' error consists of beside their own rounding to
// bf16: 2.0e-3 to 2.3e-3 of them against 1.7e-3 from the rounding alone.
//
// A softmax thread holds its row's 128 scores in registers: at the 168 that 384 threads may have, ptxas spills 300
// bytes (540 of loads).
//
// Score CTA: Q features 0..511 in TMEM [0, 256) (A operand, bf16 pairs), 512..575 in shared memory;
// two score buffers in TMEM [256, 512); three staging buffers for P; K through a ring of 16 KB slots
// (64 keys x 128 features, this CTA's half of the tile's keys, five slots a tile).
// Value CTA: O in all 512 TMEM columns; three P buffers; V through a ring of the same slots (64 keys x
// 128 features: this CTA's half of the 256 features of an MMA, four slots a tile).
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "pair.cuh"

namespace dsa {

namespace {

constexpr int kHeads = 128;
constexpr int kDqk = 576, kDv = 512;
constexpr int kTile = 128;                         // keys per tile
constexpr int kBlock = 16384;                      // 64 features (or keys) of 128 rows; a ring slot
constexpr int kSlots = 6;
constexpr int kPBufs = 3;
// the same offsets in every CTA of the cluster, so that one descriptor serves both CTAs of a pair and
// a buffer's address in another CTA is its own address there
constexpr int kOffP = kBlock;                      // [3][2 blocks of 64 keys]: staging, or P
constexpr int kOffRing = kOffP + kPBufs * 2 * kBlock;   // [0, kBlock): Q features 512..575
constexpr int kOffAlpha = kOffRing + kSlots * kBlock;   // [3][128] fp32
constexpr int kOffL = kOffAlpha + kPBufs * 128 * 4;     // [4][128] fp32
constexpr int kOffMax = kOffL + 4 * 128 * 4;            // [2][128] fp32
constexpr int kOffSum = kOffMax + 2 * 128 * 4;          // [4][128][2] fp32
constexpr int kOffScratch = kOffSum + 4 * 128 * 8;      // [4][32 rows][64 bytes]
constexpr int kOffBar = kOffScratch + 4 * 2048;
constexpr int kSmem = 1024 + kOffBar + 512;
static_assert(kSmem + 1024 <= 232448, "shared memory per CTA");
constexpr int kThreads = 384;
constexpr uint32_t kTmemS = 256;                   // score CTA: Q in [0, 256), scores in 2 x 128 columns
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum moves, and O is rescaled, only when a tile exceeds it by 2^32: P stays below
// 2^32, where bf16 has its full relative precision, and the sums stay far inside fp32.
constexpr float kRescale = 32.0f;

}  // namespace

struct SharedParams {
  const uint16_t* q;
  const uint16_t* kv;
  const int32_t* q_pos;
  const int32_t* kv_len;
  int BT, T, P, S_max;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* info;       // [clusters][2]: the unit continued from the previous cluster, the one cut at the end (-1: none)
  float* part_ml;      // [clusters][2][256][2]: maximum (log2 units), sum
  float* part_o;       // [clusters][2][128][256][4]: feature group, row, feature
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

// What the value pair does with keys [kb, kb + 64) of a tile: one pass for both tokens where they see the
// same number of them, else one for each that sees any. A pass multiplies only rows that its tokens see:
// a hidden row may hold anything, and 0 * NaN is NaN.
struct Pass {
  int n;                 // rows
  uint32_t off0, off1;   // lanes of token A / B: ~0 where their O stays as it is
};
__device__ __forceinline__ bool get_pass(const Tile& t, int kb, int j, Pass& r) {
  const int a = max(0, min(64, t.nA - kb)), b = max(0, min(64, t.nB - kb));
  const bool both = a == b, single = a == 0 || b == 0;
  if (max(a, b) == 0 || j > (both || single ? 0 : 1)) return false;
  const bool first = both || (single ? a > 0 : j == 0), second = both || (single ? b > 0 : j == 1);
  r.n = first ? a : b;
  r.off0 = first ? 0u : 0xffffffffu;
  r.off1 = second ? 0u : 0xffffffffu;
  return true;
}

// The pieces of a cluster's range of tiles, one unit after the other; every role walks it for itself.
struct Walk {
  int64_t left;        // tiles left in the range
  int u, t0, t1;       // the piece: tiles [t0, t1) of unit u
  Unit x;
  __device__ __forceinline__ void start(const SharedParams& p, int unit, int64_t off, int64_t count) {
    left = count;
    u = unit;
    t0 = (int)off;
    if (left <= 0) return;
    x = load_unit(p, u);
    t1 = (int)min((int64_t)x.tiles, t0 + left);
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next(const SharedParams& p) {
    left -= t1 - t0;
    if (left <= 0) return;
    x = load_unit(p, ++u);
    t0 = 0;
    t1 = (int)min((int64_t)x.tiles, left);
  }
  // a unit that sees no key has one empty tile: only its zeros are written
  __device__ __forceinline__ bool empty(const SharedParams& p) const { return get_tile(p, x, t0).most() == 0; }
};

// Rows [row, row + 64) of a tile's source, feature blocks [block, block + 2) of 64: [block][row][64]
__device__ __forceinline__ void load_slot(const CUtensorMap* pmap, const CUtensorMap* smap, int src, int row, int block,
                                          uint32_t dst, uint32_t bar) {
  if (src < 0) pair_load_3d(dst, pmap, bar, 0, row, block);
  else pair_load_4d(dst, smap, bar, 0, row, block, src);
}

// The barriers, as offsets in one array.
enum Bar : int {
  kFull = 0,                 // leader of each pair [kSlots]: both CTAs' parts of the slot have landed
  kEmpty = kFull + kSlots,   // both of a pair [kSlots]: the MMAs that read the slot are done
  kSFull = kEmpty + kSlots,  // score CTAs [2]: scores ready
  kSFree = kSFull + 2,       // rank 0 [2]: both score CTAs have read the scores
  kPFull = kSFree + 2,       // value CTAs [3]: this CTA's probabilities and factors have landed
  kPReady = kPFull + kPBufs, // rank 2 [3]: both value CTAs have them, O is rescaled
  kPvDone = kPReady + kPBufs,  // all [3]: P V of the tile done
  kLFull = kPvDone + kPBufs, // value CTAs [4]: the piece's sums have landed
  kQFull = kLFull + 4,       // rank 0: Q of both score CTAs in place
  kQEmpty = kQFull + 1,      // score CTAs: the piece's Q K^T done
  kOFree = kQEmpty + 1,      // rank 2: both value CTAs have read O
  kQStage = kOFree + 1,      // score CTAs: most of the first Q in shared memory
  kQHelp = kQStage + 1,      // rank 0: it is in both score CTAs' TMEM
  kMFull = kQHelp + 1,       // score CTAs [2][4]: to a softmax group, per quadrant: the running maximum
  kSumFull = kMFull + 8,     // score CTAs [4][4]: to the first group: the second one's sums of a piece
  kBars = kSumFull + 16
};
static_assert(kBars * 8 <= 512, "room for the barriers");

// The Q K^T of a piece, issued by one warp of rank 0 (`done` tiles came before). The loops and waits are the
// whole warp's and every value in them the same in all lanes, only the MMAs are one thread's: then their
// operands stay in uniform registers and an MMA takes its 65 cycles to issue. (With the loops inside the one
// thread's branch it took about 120: 4000 instead of 2620 cycles a tile.) For the same reason TMEM addresses
// are constants: a CTA that allocates all 512 columns gets them from column 0 on.
__device__ __forceinline__ bool issue_scores(uint8_t* smem, uint64_t* bars, uint32_t done, uint32_t tiles, uint32_t parity,
                                             int* abort_flag, int* status) {
  const uint32_t idesc = idesc_f32acc(1, 1, 256, kTile, 0, 0);
  const uint64_t q_desc = sdesc_kmajor_sw128(smem_u32(smem)), k_desc = sdesc_kmajor_sw128(smem_u32(smem + kOffRing));
  done = __shfl_sync(0xffffffffu, done, 0);
  tiles = __shfl_sync(0xffffffffu, tiles, 0);
  auto wait = [&](uint64_t* bar, uint32_t phase, int site) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase, abort_flag, status, site)) != 0;
  };
  if (!wait(bars + kQFull, parity, DSA_SITE_SHARED_Q)) return false;
  if (done == 0 && !wait(bars + kQHelp, 0, DSA_SITE_SHARED_Q)) return false;
  tc_fence_after();
  uint32_t slot = 5 * done % kSlots, ph = (5 * done / kSlots) & 1;
  for (uint32_t g = done; g < done + tiles; ++g) {
    const uint32_t buf = g & 1, d = kTmemS + buf * kTile;
    if (!wait(bars + kSFree + buf, ((g >> 1) + 1) & 1, DSA_SITE_SHARED_S)) return false;
#pragma unroll
    for (int f = 0; f < 9; f += 2) {
      if (!wait(bars + kFull + slot, ph, DSA_SITE_SHARED_FULL)) return false;
      tc_fence_after();
      const uint64_t b = k_desc + (uint64_t)((slot * kBlock) >> 4);
      if (elect_one()) {
        if (f < 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            pair_mma_ts(d, 32 * f + 8 * k, b + 2 * (k & 3) + (k >> 2) * (8192 >> 4), idesc, (f | k) != 0);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) pair_mma_ss(d, q_desc + 2 * k, b + 2 * k, idesc, 1);
        }
        pair_commit(bars + kEmpty + slot, 3);
        if (f == 8) pair_commit(bars + kSFull + buf, 3);
      }
      __syncwarp();
      if (++slot == kSlots) {
        slot = 0;
        ph ^= 1;
      }
    }
  }
  if (elect_one()) pair_commit(bars + kQEmpty, 3);
  __syncwarp();
  return true;
}

// Features [128 from, 512) of 32 rows of Q (q: the first one) into TMEM at t_row, a row per lane. The reads
// are coalesced, eight rows of 64 bytes each, and turn over in 2 KB of shared memory. (Every lane
// reading its own row took 13000 cycles for the 512 features.)
__device__ __forceinline__ void q_features(const uint16_t* q, bool there, uint32_t scratch, uint32_t t_row, int from) {
  const int lane = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(q + (lane >> 2) * kDqk) + (lane & 3);
  const uint32_t put = scratch + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
#pragma unroll 1
  for (int h = from; h < 4; ++h) {
    uint4 v[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[j][i] = there ? __ldg(src + (4 * h + j) * 4 + i * 8 * (kDqk / 8)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) st_shared_16(put + i * 512, v[j][i]);
      __syncwarp();
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 y = ld_shared_16(scratch + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
        x[4 * i] = y.x;
        x[4 * i + 1] = y.y;
        x[4 * i + 2] = y.z;
        x[4 * i + 3] = y.w;
      }
      tmem_st16(t_row + (4 * h + j) * 16, x);
      __syncwarp();
    }
  }
  tmem_st_wait();
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    mla_shared_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap p_map,
                      const __grid_constant__ CUtensorMap s_map, const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* alpha_sm = reinterpret_cast<float*>(smem + kOffAlpha);
  float* l_sm = reinterpret_cast<float*>(smem + kOffL);
  float* max_sm = reinterpret_cast<float*>(smem + kOffMax);
  float2* sum_sm = reinterpret_cast<float2*>(smem + kOffSum);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t *full = bars + kFull, *empty = bars + kEmpty, *s_full = bars + kSFull, *s_free = bars + kSFree;
  uint64_t *p_full = bars + kPFull, *p_ready = bars + kPReady, *pv_done = bars + kPvDone, *l_full = bars + kLFull;
  uint64_t *q_full = bars + kQFull, *q_empty = bars + kQEmpty, *o_free = bars + kOFree, *m_full = bars + kMFull;
  uint64_t *sum_full = bars + kSumFull, *q_stage = bars + kQStage, *q_help = bars + kQHelp;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ long long scan_sh[kThreads / 32];
  __shared__ int longest_sh[kThreads / 32];
  __shared__ long long start_sh[2];      // first unit of this cluster's range, first tile of it

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), side = rank & 1;     // side: the token of the unit, the half of a B operand
  const bool values = rank >= 2;
  const int cluster = blockIdx.x >> 2, clusters = gridDim.x >> 2;

  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8);
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(&p_full[i], 4);
      mbar_init(&p_ready[i], 16);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&l_full[i], 4);
    for (int i = 0; i < 8; ++i) mbar_init(&m_full[i], 1);
    for (int i = 0; i < 16; ++i) mbar_init(&sum_full[i], 1);
    mbar_init(q_full, 8 + 2);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 16);
    mbar_init(q_stage, 1);
    mbar_init(q_help, 16);
    fence_barrier_init();
  }
  if (warp == 2) pair_tmem_alloc(&tmem_base_sh, 512);
  __syncwarp();
  cluster_arrive();                      // this thread's part of the set-up; waited for below
  grid_dep_wait();                       // lengths, queries and caches may come from the preceding kernel
  grid_dep_launch();

  // The cluster's range of tiles: thread i sums the units [i * per, (i + 1) * per).
  const int units = (p.BT + 1) / 2;
  const int per = (units + kThreads - 1) / kThreads;
  const int ua = min(units, tid * per), ub = min(units, ua + per);
  long long sum = 0;
  for (int u = ua; u < ub; ++u) sum += load_unit(p, u).tiles;
  long long pre = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, pre, d);
    if (lane >= d) pre += o;
  }
  int longest = per == 1 ? (int)sum : 0;   // the longest unit (asked for only where per is 1)
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    scan_sh[warp] = pre;
    longest_sh[warp] = longest;
  }
  if (tid == 0) start_sh[0] = start_sh[1] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) base = total;
    total += scan_sh[w];
    longest = max(longest, longest_sh[w]);
  }
  const long long excl = base + pre - sum;
  // Equal shares of whole tiles; the join walks over consecutive clusters, none of them without a tile.
  const long long share = total < (1ll << 31) ? (long long)(((uint32_t)total + clusters - 1) / (uint32_t)clusters)
                                              : (total + clusters - 1) / clusters;
  long long lo = min(total, share * cluster), count = min(total - lo, share);
  // A cut inside a share costs its cluster another Q, another pipeline fill and 256 KB of fp32 per value CTA, about 8
  // tiles: where there are no more units than clusters, every unit gets the same number of clusters and an equal
  // share in each, if the longest share is not that much longer (64 queries over 8192 shared rows: 72 against 67
  // tiles and no cuts at all, 167 -> 145 us; 8 queries over 1031: eight clusters a unit).
  const int group = units <= clusters ? (int)((uint32_t)clusters / (uint32_t)units) : 1;
  const int part = (int)((uint32_t)(longest + group - 1) / (uint32_t)group);
  if (units <= clusters && part <= share + 8) {
    lo = -1;                             // found here, not by the search below
    const int u = (int)((uint32_t)cluster / (uint32_t)group), first = (cluster - u * group) * part;
    count = u < units ? max(0, min(part, load_unit(p, u).tiles - first)) : 0;
    if (tid == 0) {
      start_sh[0] = u;
      start_sh[1] = first;
    }
  }
  if (sum > 0 && lo >= excl && lo < excl + sum) {
    long long off = lo - excl;
    int u = ua;
    if (per > 1)
      for (; u < ub; ++u) {
        const int n = load_unit(p, u).tiles;
        if (off < n) break;
        off -= n;
      }
    start_sh[0] = u;
    start_sh[1] = off;
  }
  __syncthreads();
  cluster_wait();                        // the barriers of every CTA are initialised, every pair holds its TMEM
  const uint32_t tmem = tmem_base_sh;
  const uint32_t ring = smem_u32(smem + kOffRing);
  Walk w;
  w.start(p, (int)start_sh[0], start_sh[1], count);

  // Score CTA: Q of a piece, once the MMAs of the piece before are done. Features 512..575 stay in shared memory, the
  // others go into TMEM, by warps 0..3 (one per TMEM quadrant). The first piece has no pipeline to overlap with:
  // there TMA brings features 0..383 into the still unused P buffers, and the softmax warps take them from there.
  auto q_tma = [&](int piece) {
    const int row = (2 * w.u + (int)side) * kHeads;
    const uint32_t bar = cluster_addr(q_full, 0);
    arrive_expect_tx_cluster(bar, kBlock);
    pair_load_2d(smem_u32(smem), &q_map, bar, 512, row);
    if (piece > 0) return;
    mbar_arrive_expect_tx(q_stage, 6 * kBlock);
    for (int i = 0; i < 6; ++i) tma_load_2d(smem + kOffP + i * kBlock, &q_map, q_stage, 64 * i, row);
  };
  auto q_rows = [&](int piece) {
    if (piece > 0 && !__all_sync(0xffffffffu, mbar_wait(q_empty, (piece + 1) & 1, &abort_flag, p.status,
                                                        DSA_SITE_SHARED_EMPTY)))
      return false;
    if (piece > 0 && warp == 0 && elect_one()) q_tma(piece);
    __syncwarp();
    tc_fence_after();
    const int tok = 2 * w.u + (int)side;
    const bool there = tok < p.BT;         // a unit's second token may not exist: its rows are zeros
    q_features(p.q + ((int64_t)(there ? tok : 0) * kHeads + 32 * warp) * kDqk, there,
               smem_u32(smem + kOffScratch) + warp * 2048, tmem + ((uint32_t)(32 * warp) << 16), piece > 0 ? 0 : 3);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_cluster(cluster_addr(q_full, 0));
    return true;
  };

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------------ loads
    // Waiting for a slot and issuing its load take a warp about as long as the MMAs that free it, so
    // three warps take the slots in turn.
    const int mine = warp == 0 ? 0 : warp - 1;
    int turn = 0, slot = 0, piece = 0;
    uint32_t ph = 1;                     // a fresh slot counts as freed
    const bool el = elect_one();
    bool ok = true;
    auto acquire = [&]() {
      if (!mbar_wait(&empty[slot], ph, &abort_flag, p.status, DSA_SITE_SHARED_EMPTY)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    auto advance = [&]() {
      if (++slot == kSlots) {
        slot = 0;
        ph ^= 1;
      }
      if (++turn == 3) turn = 0;
    };
    auto k_tile = [&](const Tile& t) {
      for (int f = 0; ok && f < 9; f += 2, advance()) {
        if (turn != mine) continue;
        acquire();
        if (!ok) break;
        if (el) {
          const uint32_t bar = cluster_addr(&full[slot], 0);
          arrive_expect_tx_cluster(bar, kBlock);         // there is no block 9: zeros
          load_slot(&p_map, &s_map, t.src, t.k0 + 64 * (int)side, f, ring + slot * kBlock, bar);
        }
      }
    };
    auto v_slot = [&](const Tile& t, int kb, int n, int half) {
      const uint32_t dst = ring + slot * kBlock, bar = cluster_addr(&full[slot], 2);
      const int block = 4 * half + 2 * (int)side;
      if (t.src < 0 || n >= 64) {
        if (el) {
          arrive_expect_tx_cluster(bar, kBlock);
          load_slot(&p_map, &s_map, t.src, t.k0 + kb, block, dst, bar);
        }
        return;
      }
      // the warp copies the visible rows itself and puts zeros behind them
      const uint16_t* src = p.kv + ((int64_t)t.src * p.S_max + t.k0 + kb) * kDqk + 64 * block;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = 32 * h + 2 * i + (lane >> 4), c = lane & 15;    // row, 16-byte chunk of its 256 bytes
          v[i] = r < n ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * kDqk) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = 32 * h + 2 * i + (lane >> 4), c = lane & 15;
          st_shared_16(dst + 8192 * (c >> 3) + r * 128 + (((c & 7) ^ (r & 7)) << 4), v[i]);
        }
      }
      fence_proxy_async_smem();
      cluster_fence();
      __syncwarp();
      if (el) arrive_cluster(bar);
    };
    for (; ok && w.valid(); w.next(p)) {
      if (w.empty(p)) continue;
      if (!values) {
        k_tile(get_tile(p, w.x, w.t0));
        ok = ok && q_rows(piece);
      }
      ++piece;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        const Tile tile = get_tile(p, w.x, t);
        if (!values) {
          if (t > w.t0) k_tile(tile);
          continue;
        }
        Pass pass;
        for (int kb = 0; kb < kTile; kb += 64)
          for (int j = 0; ok && get_pass(tile, kb, j, pass); ++j)
            for (int half = 0; ok && half < 2; ++half, advance()) {
              if (turn != mine) continue;
              acquire();
              if (ok) v_slot(tile, kb, pass.n, half);
            }
      }
    }
    // the last MMAs' arrivals have to reach this CTA before it leaves
    if (mine == 0) {
      for (int i = 0; ok && i < kSlots; ++i, advance()) acquire();
      if (ok && !values && piece > 0)
        mbar_wait(q_empty, (piece + 1) & 1, &abort_flag, p.status, DSA_SITE_SHARED_EMPTY);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue: one thread of each leader
    if (!values) {
      uint32_t done = 0;                  // tiles of earlier pieces
      int piece = 0;
      for (; w.valid(); w.next(p)) {
        if (w.empty(p)) continue;
        if (!q_rows(piece)) break;        // the whole warp
        const bool fine = side != 0 || issue_scores(smem, bars, done, (uint32_t)(w.t1 - w.t0), piece & 1, &abort_flag, p.status);
        if (!__all_sync(0xffffffffu, fine)) break;
        done += w.t1 - w.t0;
        ++piece;
      }
    } else if (side == 0) {
      const uint32_t idesc = idesc_f32acc(1, 1, 256, 256, 0, 1);
      const uint64_t p_desc = sdesc_kmajor_sw128(smem_u32(smem + kOffP)), v_desc = sdesc_mnmajor_sw128(ring, 8192, 1024);
      auto wait = [&](uint64_t* bar, uint32_t phase, int site) {
        return __all_sync(0xffffffffu, mbar_wait(bar, phase, &abort_flag, p.status, site)) != 0;
      };
      uint32_t slot = 0, ph = 0, buf = 0, pb = 0;          // ring slot and phase, P buffer and phase
      int piece = 0;
      bool ok = true;
      for (; ok && w.valid(); w.next(p)) {
        if (w.empty(p)) continue;
        if (piece > 0 && !wait(o_free, (piece + 1) & 1, DSA_SITE_SHARED_O)) break;
        bool startedA = false, startedB = false;
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const Tile tile = get_tile(p, w.x, t);
          if (!wait(&p_ready[buf], pb, DSA_SITE_SHARED_P)) {
            ok = false;
            break;
          }
          tc_fence_after();
          Pass pass;
#pragma unroll
          for (int kb = 0; kb < kTile; kb += 64) {
            for (int j = 0; ok && get_pass(tile, kb, j, pass); ++j) {
              const bool acc = (pass.off0 == 0 && startedA) || (pass.off1 == 0 && startedB);
              const bool plain = acc && (pass.off0 | pass.off1) == 0 && pass.n == 64;
              startedA |= pass.off0 == 0;
              startedB |= pass.off1 == 0;
#pragma unroll
              for (int half = 0; half < 2; ++half) {         // 256 features each
                if (!wait(&full[slot], ph, DSA_SITE_SHARED_FULL)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                if (tile.src >= 0 && pass.n < 64) cluster_fence();     // both CTAs' warps wrote this slot
                const uint64_t a = p_desc + (uint64_t)((2 * buf + (kb >> 6)) * (kBlock >> 4));
                const uint64_t b = v_desc + (uint64_t)(slot * (kBlock >> 4));
                if (elect_one()) {
                  if (plain) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) pair_mma_ss(256 * half, a + 2 * k, b + 128 * k, idesc, 1);
                  } else {
                    for (int k = 0; k < 4 && 16 * k < pass.n; ++k)
                      pair_mma_ss_masked(256 * half, a + 2 * k, b + 128 * k, idesc, pass.off0, pass.off1, acc || k > 0);
                  }
                  pair_commit(&empty[slot], 12);
                }
                __syncwarp();
                if (++slot == kSlots) {
                  slot = 0;
                  ph ^= 1;
                }
              }
            }
          }
          if (ok && elect_one()) pair_commit(&pv_done[buf], 15);
          __syncwarp();
          if (++buf == kPBufs) {
            buf = 0;
            pb ^= 1;
          }
        }
        ++piece;
      }
    }
  } else if (!values) {
    // ------------------------------------------------------------------ softmax: one thread per row, two warpgroups that
    // take the tiles in turn. A tile takes a warpgroup about 3500 cycles, 4300 beside the other (1024 of MUFU each),
    // so one alone would be slower than the MMAs (2306). The running maximum passes from one to the other as soon
    // as it is known.
    const int row = (tid - 128) & 127, group = (tid - 128) >> 7, quad = warp & 3;    // row: head, TMEM lane
    const uint32_t t_row = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t peer = rank + 2;
    uint32_t g = 0, pb = 0, pph = 1;                       // tiles; P buffer and the phase of its release
    int piece = 0;
    bool ok = true;
    int32_t info_cont = -1, info_head = -1;
    for (; ok && w.valid(); w.next(p)) {
      const int tok = 2 * w.u + (int)side;
      const bool some = !w.empty(p);
      if (some && piece == 0) {                            // three blocks of 64 features of the first Q
        if (warp == 4 && elect_one()) q_tma(0);
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(q_stage, 0, &abort_flag, p.status, DSA_SITE_SHARED_Q))) break;
#pragma unroll 1
        for (int f = 3 * group; f < 3 * group + 3; ++f) {
          uint32_t x[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 y = ld_shared_16(smem_u32(smem + kOffP) + f * kBlock + row * 128 + ((c ^ (row & 7)) << 4));
            x[4 * c] = y.x;
            x[4 * c + 1] = y.y;
            x[4 * c + 2] = y.z;
            x[4 * c + 3] = y.w;
          }
          tmem_st32(t_row + 32 * f, x);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(q_help, 0));
      }
      float m = -INFINITY, l = 0.f;                        // l: of this group's tiles, relative to m
      for (int t = w.t0; some && ok && t < w.t1; ++t) {
        const uint32_t buf = g & 1, ph = (g >> 1) & 1, pbuf = pb, pphase = pph;
        const bool mine = buf == (uint32_t)group;
        ++g;
        if (++pb == kPBufs) {
          pb = 0;
          pph ^= 1;
        }
        if (!mine) continue;
        const Tile tile = get_tile(p, w.x, t);
        const int n = side == 0 ? tile.nA : tile.nB;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[buf], ph, &abort_flag, p.status, DSA_SITE_SHARED_S))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[4][32];
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_row + kTmemS + buf * kTile + 32 * c, r[c]);
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(&s_free[buf], 0));
        float mx = -INFINITY;
        if (n > 0) {
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
          mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
        }
        // the maximum after the tile before (g - 2; g counts this one), from the other group
        if (g > 1 && !__all_sync(0xffffffffu, mbar_wait(&m_full[4 * group + quad], ((g - 2) >> 1) & 1, &abort_flag, p.status,
                                                        DSA_SITE_SHARED_S))) {
          ok = false;
          break;
        }
        const float before = t > w.t0 ? max_sm[(buf ^ 1) * 128 + row] : -INFINITY;
        const float now = mx > before + kRescale ? mx : before;
        max_sm[buf * 128 + row] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m_full[4 * (group ^ 1) + quad]);
        // the staging buffer, and the value CTA's, held an earlier tile
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[pbuf], pphase, &abort_flag, p.status, DSA_SITE_SHARED_P))) {
          ok = false;
          break;
        }
        const uint32_t bar = cluster_addr(&p_full[pbuf], peer);
        if (n == 0) {
          if (lane == 0) arrive_cluster(bar);
          continue;
        }
        const float mm = now == -INFINITY ? 0.f : now;     // every score -inf: e^-inf = 0, not NaN
        if (now != m) {
          l *= m == -INFINITY ? 0.f : exp2_approx(m - now);
          m = now;
        }
        const uint32_t stage = smem_u32(smem + kOffP) + pbuf * 2 * kBlock + row * 128;
        float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 16; ++c) {                      // eight keys, 16 bytes
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e0 = exp2_approx(fmaf(__uint_as_float(r[c >> 2][(c & 3) * 8 + 2 * i]), p.scale_log2, -mm));
            const float e1 = exp2_approx(fmaf(__uint_as_float(r[c >> 2][(c & 3) * 8 + 2 * i + 1]), p.scale_log2, -mm));
            sum4[i] += e0 + e1;
            pk[i] = pack_bf16(e0, e1);
          }
          st_shared_16(stage + (c >> 3) * kBlock + (((c & 7) ^ (row & 7)) << 4), make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
        l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
        alpha_sm[pbuf * 128 + row] = now == before || before == -INFINITY ? 1.f : exp2_approx(before - now);
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          arrive_expect_tx_cluster(bar, 2 * 4096 + 128);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* src = smem + kOffP + (2 * pbuf + i) * kBlock + quad * 4096;
            copy_to_cluster(cluster_addr(src, peer), smem_u32(src), 4096, bar);
          }
          const float* src = alpha_sm + pbuf * 128 + 32 * quad;
          copy_to_cluster(cluster_addr(src, peer), smem_u32(src), 128, bar);
        }
      }
      if (!ok) break;
      const bool whole = w.t0 == 0 && w.t1 == w.x.tiles;
      const int where = w.t0 == 0 ? 1 : 0;
      if (!whole) (where ? info_head : info_cont) = w.u;
      // the row's sum over both groups, for the value CTA too (four buffers: a reader may be two pieces behind)
      const int i = piece & 3;
      if (some && group == 1) {
        sum_sm[i * 128 + row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sum_full[4 * i + quad]);
      }
      if (group == 0) {
        if (some) {
          if (!__all_sync(0xffffffffu, mbar_wait(&sum_full[4 * i + quad], (piece >> 2) & 1, &abort_flag, p.status,
                                                 DSA_SITE_SHARED_S))) {
            ok = false;
            break;
          }
          const float2 other = sum_sm[i * 128 + row];
          const float both = fmaxf(m, other.x);
          l = (l == 0.f ? 0.f : l * exp2_approx(m - both)) + (other.y == 0.f ? 0.f : other.y * exp2_approx(other.x - both));
          m = both;
          l_sm[i * 128 + row] = l;
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            const uint32_t bar = cluster_addr(&l_full[i], peer);
            arrive_expect_tx_cluster(bar, 128);
            const float* src = l_sm + i * 128 + 32 * quad;
            copy_to_cluster(cluster_addr(src, peer), smem_u32(src), 128, bar);
          }
        }
        if (whole) {
          if (tok < p.BT && p.lse) p.lse[(int64_t)tok * kHeads + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          const int64_t slot = (int64_t)cluster * 2 + where;
          *reinterpret_cast<float2*>(p.part_ml + (slot * 256 + (int)side * kHeads + row) * 2) = make_float2(m, l);
        }
      }
      piece += some;
    }
    // as in the loads: the last arrivals
    for (uint32_t i = g > kPBufs ? g - kPBufs : 0; ok && i < g; ++i)
      if (!mbar_wait(&pv_done[i % kPBufs], (i / kPBufs) & 1, &abort_flag, p.status, DSA_SITE_SHARED_P)) ok = false;
    if (rank == 0 && tid == 128) {
      p.info[2 * cluster] = info_cont;
      p.info[2 * cluster + 1] = info_head;
    }
  } else {
    // ------------------------------------------------------------------ O: rescaling and output; one thread per row and
    // half of the features
    const int row = (tid - 128) & 127, half = (tid - 128) >> 7;
    const uint32_t t_o = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 * half;
    uint32_t g = 0;
    int piece = 0;
    bool ok = true;
    for (; ok && w.valid(); w.next(p)) {
      const int tok = 2 * w.u + (int)side;
      const bool some = !w.empty(p);
      bool any = false;                                    // O of this token holds something
      for (int t = w.t0; some && ok && t < w.t1; ++t, ++g) {
        const Tile tile = get_tile(p, w.x, t);
        const uint32_t buf = g % kPBufs, ph = (g / kPBufs) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&p_full[buf], ph, &abort_flag, p.status, DSA_SITE_SHARED_P))) {
          ok = false;
          break;
        }
        if ((side == 0 ? tile.nA : tile.nB) > 0) {
          const float alpha = any ? alpha_sm[buf * 128 + row] : 1.f;
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // P V of every earlier tile has to be in O first
            if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) % kPBufs], ((g - 1) / kPBufs) & 1, &abort_flag, p.status,
                                                   DSA_SITE_SHARED_O))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[32];
              tmem_ld32(t_o + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(t_o + 32 * c, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          any = true;
        }
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(&p_ready[buf], 2));
      }
      if (!ok) break;
      const bool whole = w.t0 == 0 && w.t1 == w.x.tiles;
      float l = 0.f;
      if (some) {
        const bool there = mbar_wait(&l_full[piece & 3], (piece >> 2) & 1, &abort_flag, p.status, DSA_SITE_SHARED_P) &&
                           mbar_wait(&pv_done[(g - 1) % kPBufs], ((g - 1) / kPBufs) & 1, &abort_flag, p.status, DSA_SITE_SHARED_O);
        if (!__all_sync(0xffffffffu, there)) {
          ok = false;
          break;
        }
        tc_fence_after();
        l = l_sm[(piece & 3) * 128 + row];
        ++piece;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t slot = (int64_t)cluster * 2 + (w.t0 == 0 ? 1 : 0);
      const int prow = (int)side * kHeads + row;
#pragma unroll 1
      for (int c = 0; c < 8; c += 2) {
        uint32_t o[2][32];
        if (any) {
          tmem_ld32(t_o + 32 * c, o[0]);
          tmem_ld32(t_o + 32 * c + 32, o[1]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[0][i] = o[1][i] = 0u;
        }
        if (whole) {
          if (tok < p.BT) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)tok * kHeads + row) * kDv + 256 * half + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t* y = &o[i >> 2][8 * (i & 3)];
              uint4 v;
              v.x = pack_bf16(__uint_as_float(y[0]) * inv, __uint_as_float(y[1]) * inv);
              v.y = pack_bf16(__uint_as_float(y[2]) * inv, __uint_as_float(y[3]) * inv);
              v.z = pack_bf16(__uint_as_float(y[4]) * inv, __uint_as_float(y[5]) * inv);
              v.w = pack_bf16(__uint_as_float(y[6]) * inv, __uint_as_float(y[7]) * inv);
              dst[i] = v;
            }
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o) + (slot * 128 + 64 * half + 8 * c) * 256 + prow;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t* y = &o[i >> 3][4 * (i & 7)];
            dst[i * 256] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (some) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(o_free, 2));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                      // nothing of the cluster is in flight towards a CTA that has left
  cluster_wait();
  if (warp == 2) pair_tmem_dealloc(tmem, 512);
}

// Joins the pieces of units that were cut. A unit's first piece is the last one of some cluster c, the others
// are the first ones of the clusters behind it. The blocks take (cut unit, 32 rows x 64 features) in turn: most
// clusters head no unit, and blocks for all of them took longer than the joining (10 of 40 us for 8 queries).
__global__ void __launch_bounds__(256) mla_shared_join_kernel(const SharedParams p, int clusters) {
  extern __shared__ float2 ml_sh[];      // [pieces][32 rows]: maximum, sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  for (int work = blockIdx.x;; work += gridDim.x) {
    int c = -1, heads = 0;
    for (int q = 0; q < clusters && c < 0; q += 32) {
      const uint32_t mask = __ballot_sync(0xffffffffu, q + lane < clusters && __ldcg(p.info + 2 * (q + lane) + 1) >= 0);
      const int k = (work >> 6) - heads;
      if (k < __popc(mask)) c = q + (int)__fns(mask, 0, k + 1);
      heads += __popc(mask);
    }
    if (c < 0) return;
    const int unit = __ldcg(p.info + 2 * c + 1), part = work & 63;
    const int row = (part >> 3) * 32 + lane, col = (part & 7) * 64 + 8 * warp;
    const int tok = 2 * unit + (row >> 7), head = row & 127;
    if (tok >= p.BT) continue;             // the same for the whole block
    int n = 1;                             // pieces
    for (int q = c + 1; q < clusters; q += 32) {
      const uint32_t other = __ballot_sync(0xffffffffu, q + lane >= clusters || __ldcg(p.info + 2 * (q + lane)) != unit);
      n += other ? __ffs(other) - 1 : 32;
      if (other) break;
    }
    auto slot_of = [&](int i) { return i == 0 ? (int64_t)c * 2 + 1 : (int64_t)(c + i) * 2; };
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + (int64_t)(col / 4) * 256 + row;
    // the first four pieces' values travel together with the maxima and sums
    float4 v[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) v[i][j] = __ldcg(src + slot_of(min(i, n - 1)) * (128 * 256) + j * 256);
    for (int i = warp; i < n; i += 8)
      ml_sh[i * 32 + lane] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(i) * 256 + row);
    __syncthreads();
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, ml_sh[i * 32 + lane].x);
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int i0 = 0; i0 < n; i0 += 4) {
      float4 next[4][2];
      if (i0 + 4 < n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) next[i][j] = __ldcg(src + slot_of(min(i0 + 4 + i, n - 1)) * (128 * 256) + j * 256);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= n) break;
        const float2 ml = ml_sh[(i0 + i) * 32 + lane];
        // a piece without a visible key has sum 0 and no maximum
        const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - m);
        l += ml.y * f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[j].x = fmaf(v[i][j].x, f, acc[j].x);
          acc[j].y = fmaf(v[i][j].y, f, acc[j].y);
          acc[j].z = fmaf(v[i][j].z, f, acc[j].z);
          acc[j].w = fmaf(v[i][j].w, f, acc[j].w);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) v[i][j] = next[i][j];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t out_row = (int64_t)tok * kHeads + head;
    *reinterpret_cast<uint4*>(p.out + out_row * kDv + col) =
        make_uint4(pack_bf16(acc[0].x * inv, acc[0].y * inv), pack_bf16(acc[0].z * inv, acc[0].w * inv),
                   pack_bf16(acc[1].x * inv, acc[1].y * inv), pack_bf16(acc[1].z * inv, acc[1].w * inv));
    if (col == 0 && p.lse) p.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    __syncthreads();                     // ml_sh is written again
  }
}

namespace {

// Clusters of four that the device holds at once, one CTA per SM (33 on a B200: its SM groups do not
// all divide by four). More would wait for a second wave.
int resident_clusters() {
  static uint64_t seen[dsa_host::kMaxSetupDevices];
  static int count[dsa_host::kMaxSetupDevices];
  int dev = 0;
  if (!dsa_host::needs_setup(seen, &dev)) return count[dev];
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(dsa_host::device_sm_count() / 4 * 4));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(mla_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, mla_shared_kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return dsa_host::device_sm_count() / 4;              // no device here: the most there can be
  }
  if (dev >= 0 && dev < dsa_host::kMaxSetupDevices) {
    count[dev] = n;
    dsa_host::mark_setup(seen);
  }
  return n;
}

// Clusters of the launch, at most one per tile.
int shared_clusters(int64_t BT, int P, int S_max) {
  const int64_t units = (BT + 1) / 2;
  const int64_t own = (S_max + kTile - 1) / kTile;
  const int64_t tiles = std::max<int64_t>(1, (P + kTile - 1) / kTile + 2 * own);
  return (int)std::max<int64_t>(1, std::min<int64_t>(resident_clusters(), units * tiles));
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t mla_shared_workspace_size(int B, int T, int P, int S_max) {
  const size_t n = (size_t)shared_clusters((int64_t)B * T, P, S_max);
  return align256(n * 8) + n * 2 * 256 * 8 + n * 2 * 128 * 256 * 16;
}

int launch_mla_shared(const uint16_t* q, const uint16_t* prefix, int P, const uint16_t* kv, const int32_t* q_pos,
                      const int32_t* kv_len, int B, int T, int S_max, float softmax_scale, uint16_t* out, float* lse,
                      void* workspace, size_t ws_bytes, cudaStream_t stream, int* status) {
  if (!workspace || ws_bytes < mla_shared_workspace_size(B, T, P, S_max)) return DSA_ERR_WORKSPACE;
  SharedParams p;
  p.q = q;
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
  const int clusters = shared_clusters(p.BT, P, S_max);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.info = reinterpret_cast<int32_t*>(ws);
  ws += align256((size_t)clusters * 8);
  p.part_ml = reinterpret_cast<float*>(ws);
  ws += (size_t)clusters * 2 * 256 * 8;
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
  int rc = dsa_host::launch_clusters(mla_shared_kernel, 4, (unsigned)clusters, kThreads, kSmem, stream, q_map, pm, sm, p);
  if (rc != DSA_OK) return rc;
  return dsa_host::launch(mla_shared_join_kernel, dim3((unsigned)(2 * dsa_host::device_sm_count())), dim3(256),
                          (size_t)clusters * 32 * 8, stream, p, clusters);
}

}  // namespace dsa
