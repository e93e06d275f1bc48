// dsa_cache_evict: cuts each sequence's cache back to a budget of rows, by the attention weight its
// rows collected.
//
// Of a sequence's n rows the kept ones are the first `keep` in the order (protected, larger weight,
// lower row), protected meaning among the newest positions or the first ones. Rows need not stay in
// order (every row carries its position), so a kept row below `keep` stays where it is and the i-th
// kept row behind `keep` moves into the i-th row given up before it: sources and destinations never
// overlap, the moves need no order, and the bytes moved are the fewest that leave a dense cache.
//
// select: a cluster of CTAs per sequence holds the rows in registers where they fit, 16 to a thread, each as
// an order-preserving 32-bit image of its weight and bits of masks that say what it is, and finds the
// border key by three histogram passes (11 + 11 + 10 bits), the CTAs reading one another's histograms
// through distributed shared memory; a last pass breaks ties by row and lists movers and holes in order.
// move: a warp per two moved rows. Bound: the n (weight, position) pairs once, and HBM for the moves. 64
// sequences of 12000 to 16384 rows cut to 8192 (about 550 MB): select 20 us, move 95 us, 4.8 TB/s in all; one
// sequence of 131072 cut to 8191: 25 us, most of it the select's barriers and passes.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kFine = 8;                 // bins of a histogram that make a coarse one
constexpr int kCoarse = kBins / kFine;
constexpr int kCachedGroups = 16;        // groups of 32 rows that a warp holds, a row of each per lane
constexpr int kCachedRows = kCachedGroups * kThreads;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Order-preserving image of a weight; -0 equals +0 and NaN comes below everything.
__device__ __forceinline__ uint32_t weight_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace

struct EvictParams {
  const float* acc;
  const int32_t* pos;
  const int32_t* kv_len;
  int S_max, keep, recent, sinks;
  int C;                   // CTAs per sequence
  float* acc_out;
  int32_t* pos_out;
  int32_t* len_out;
  int32_t* src;            // [B][keep]
  int32_t* moves;          // [B][1 + 2 L]: count, movers, holes
  int L;
  uint8_t* kv;             // caches moved row by row (or NULL)
  uint8_t* k8;
  float* k_scale;
};

// CACHED: the rows of a CTA fit into its registers; otherwise every pass reads them again, a chunk at a time.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p) {
  constexpr int kGroups = CACHED ? kCachedGroups : 4;        // that a warp holds at a time
  __shared__ __align__(16) uint32_t hist[2][kBins];                        // ordinary and protected rows
  __shared__ __align__(16) uint32_t coarse[2][kCoarse], all_sm[kCoarse];   // of this CTA's histograms, of all CTAs'
  __shared__ uint32_t cnt_sm[8];                             // this CTA's words that the others read (kNewest ...)
  __shared__ uint32_t warp_sm[kWarps], scan_sm[3][kWarps], found_sm[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / p.C;
  // a barrier of the sequence's CTAs (a single one needs no cluster barrier)
  auto sync_all = [&]() {
    if (p.C == 1) __syncthreads();
    else cluster_sync();
  };
  grid_dep_wait();
  grid_dep_launch();
  const int n = max(0, min(__ldg(p.kv_len + b), p.S_max));
  const float* acc = p.acc + (int64_t)b * p.S_max;
  const int32_t* pos = p.pos + (int64_t)b * p.S_max;
  float* acc_out = p.acc_out + (int64_t)b * p.S_max;
  int32_t* pos_out = p.pos_out + (int64_t)b * p.S_max;
  int32_t* src = p.src ? p.src + (int64_t)b * p.keep : nullptr;
  int32_t* moves = p.moves + (int64_t)b * (1 + 2 * p.L);
  const bool copy_acc = acc_out != acc, copy_pos = pos_out != pos;
  // this CTA's rows: a contiguous run, each warp a run of whole groups of 32
  const int per_warp = ((n + p.C * kWarps - 1) / (p.C * kWarps) + 31) / 32 * 32;
  const int per = per_warp * kWarps;
  const int r0 = (int)min((int64_t)n, (int64_t)rank * per), r1 = (int)min((int64_t)n, (int64_t)r0 + per);

  if (n <= p.keep) {                                          // nothing to give up (uniform in the cluster)
    for (int r = r0 + tid; r < r1; r += kThreads) {
      if (copy_acc) acc_out[r] = acc[r];
      if (copy_pos) pos_out[r] = pos[r];
      if (src) src[r] = r;
    }
    if (src)
      // in 64 bits: the budget may be any int, the largest included
      for (int64_t r = (int64_t)n + rank * kThreads + tid; r < p.keep; r += p.C * kThreads) src[r] = -1;
    if (rank == 0 && tid == 0) {
      p.len_out[b] = n;
      moves[0] = 0;
    }
    return;
  }

  enum { kNewest, kSafe, kTies, kHoles, kMovers };            // words of cnt_sm
  // word `slot` of every CTA before this one, of every one behind it, and of all, summed
  auto gather = [&](int slot, uint32_t& before, uint32_t& behind) {
    const uint32_t v = lane < p.C ? ld_cluster(&cnt_sm[slot], (uint32_t)lane) : 0u;
    before = __reduce_add_sync(0xffffffffu, lane < (int)rank ? v : 0u);
    behind = __reduce_add_sync(0xffffffffu, lane > (int)rank ? v : 0u);
    return __reduce_add_sync(0xffffffffu, v);
  };
  for (int i = tid; i < 2 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  // A warp's run of rows [w0, w1) comes in chunks of kGroups groups; lane i holds row `at + 32 * it + i` of
  // the chunk's group `it`, and bit `it` of a lane's masks is that row's.
  const int w0 = min(r1, r0 + warp * per_warp), w1 = min(r1, w0 + per_warp);
  uint32_t key[kGroups];
  int ps[kGroups];
  uint32_t valid = 0, safe_rows = 0;                          // rows there are, protected ones
  // the bits of the lane's rows below `end`
  auto below = [&](int at, int end) {
    return (1u << max(0, min(kGroups, (int)(((int64_t)end - at - lane + 31) >> 5)))) - 1u;
  };
  int groups = 0;                                             // of the chunk
  auto load = [&](int at) {
    valid = below(at, w1);
    groups = (w1 - at + 31) >> 5;
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it) {
      if (!((valid >> it) & 1u)) continue;
      key[it] = __float_as_uint(acc[at + 32 * it + lane]);
      ps[it] = pos[at + 32 * it + lane];
    }
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it)
      if ((valid >> it) & 1u) key[it] = weight_key(__uint_as_float(key[it]));
  };
  int newest = INT32_MIN;
  for (int at = w0; at < w1; at += 32 * kGroups) {
    load(at);
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it)
      if ((valid >> it) & 1u) newest = max(newest, ps[it]);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, d));
  if (lane == 0) warp_sm[warp] = (uint32_t)newest;
  __syncthreads();
  if (warp == 0) {
    newest = (int)warp_sm[lane];
#pragma unroll
    for (int d = 16; d; d >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, d));
    if (lane == 0) {
      cnt_sm[kNewest] = (uint32_t)newest;
      cnt_sm[kSafe] = 0;
    }
  }
  sync_all();
  newest = __reduce_max_sync(0xffffffffu, lane < p.C ? (int)ld_cluster(&cnt_sm[kNewest], (uint32_t)lane) : INT32_MIN);
  // positions above `recent_from` are protected (all of them, if that lies below the range)
  const int64_t from = (int64_t)newest - p.recent;
  const int recent_from = (int)max(from, (int64_t)INT32_MIN);
  auto protects = [&](int ps) { return ps > recent_from || ps < p.sinks || from < INT32_MIN; };
  auto classify = [&]() {
    safe_rows = 0;
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it)
      if (((valid >> it) & 1u) && protects(ps[it])) safe_rows |= 1u << it;
  };
  // f(at) for every chunk of the warp's run, its rows in registers
  auto each_chunk = [&](auto f) {
    if (CACHED) {
      f(w0);
    } else {
      for (int at = w0; at < w1; at += 32 * kGroups) {
        load(at);
        classify();
        f(at);
      }
    }
  };
  if (CACHED) classify();
  // The state of every row below the budget, as if all of them stayed: a given-up one's is written again when its
  // successor moves there. (Copying only those that stay, after the selection, took 7000 cycles more.)
  const int step = p.C * kThreads;
  for (int r = (int)rank * kThreads + tid; r < p.keep; r += 4 * step) {
    float a[4];
    int q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (copy_acc && r + i * step < p.keep) a[i] = acc[r + i * step];
      if (copy_pos && r + i * step < p.keep) q[i] = pos[r + i * step];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r + i * step >= p.keep) break;
      if (copy_acc) acc_out[r + i * step] = a[i];
      if (copy_pos) pos_out[r + i * step] = q[i];
      if (src) src[r + i * step] = r + i * step;
    }
  }

  // The coarse bins of this CTA's histogram `which`, once it is complete.
  auto sum_bins = [&](int which, int i) {
    const uint4* h = reinterpret_cast<const uint4*>(&hist[which][kFine * i]);
    const uint4 x = h[0], y = h[1];
    coarse[which][i] = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
  };

  // first digit, for both classes
  uint32_t safe = 0;
  each_chunk([&](int) {
    safe += __popc(safe_rows);
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it)
      if ((valid >> it) & 1u) atomicAdd(&hist[(safe_rows >> it) & 1u][key[it] >> 21], 1u);
  });
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0 && safe) atomicAdd(&cnt_sm[kSafe], safe);
  __syncthreads();
  if (tid < 2 * kCoarse) sum_bins(tid / kCoarse, tid % kCoarse);
  sync_all();
  // the warps' words of scan_sm[slot] summed over the warps before this one, and over all of the block
  auto scan_warps = [&](int slot, uint32_t& total) {
    uint32_t s = scan_sm[slot][lane];
    const uint32_t v = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - v, warp);
  };
  // The bin of histogram `which` in which the want-th largest key lies; `want` becomes its rank among the
  // bin's keys. The CTAs' coarse bins are added up first, then one warp finds the bin among the eight of the one
  // it is in. (Adding up all 2048 bins of eight CTAs took 4500 cycles a digit, most of it remote reads; every
  // warp finding the bin for itself, 1000 more than the barrier.)
  auto find_bin = [&](int which, uint32_t& want) {
    if (tid < kCoarse) {
      uint32_t h = 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < p.C) h += ld_cluster(&coarse[which][tid], (uint32_t)c);
      all_sm[tid] = h;
    }
    __syncthreads();
    if (warp == 0) {
      // lane i: coarse bins [8 i, 8 i + 8), and how many keys lie in those above
      const uint4* h = reinterpret_cast<const uint4*>(&all_sm[8 * lane]);
      const uint4 x = h[0], y = h[1];
      const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      uint32_t up = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) up += v[i];
      const uint32_t own = up;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_down_sync(0xffffffffu, up, d);
        if (lane + d < 32) up += o;
      }
      up -= own;
      uint32_t bin = 0, above = 0;
      const bool here = want > up && want <= up + own;
      if (here) {
        above = up;
        bin = 7;
#pragma unroll
        for (int i = 7; i > 0; --i)
          if ((int)bin == i && want > above + v[i]) {
            above += v[i];
            bin = i - 1;
          }
        bin += 8 * lane;
      }
      const int where = __ffs(__ballot_sync(0xffffffffu, here)) - 1;       // the histogram holds at least `want` keys
      bin = __shfl_sync(0xffffffffu, bin, where);
      const uint32_t in = want - __shfl_sync(0xffffffffu, above, where);
      // the eight bins of it: lane i adds up bin i % 8 of the CTAs i / 8 and i / 8 + 4
      uint32_t f = 0;
      const uint32_t* fine = &hist[which][kFine * bin + (lane & 7)];
      if (lane >> 3 < p.C) f = ld_cluster(fine, (uint32_t)lane >> 3);
      if ((lane >> 3) + 4 < p.C) f += ld_cluster(fine, ((uint32_t)lane >> 3) + 4);
      f += __shfl_xor_sync(0xffffffffu, f, 8);
      f += __shfl_xor_sync(0xffffffffu, f, 16);
      uint32_t over = f;                                        // keys in this bin and those of the eight above it
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const uint32_t o = __shfl_down_sync(0xffffffffu, over, d, 8);
        if ((lane & 7) + d < 8) over += o;
      }
      const int at = __ffs(__ballot_sync(0xffffffffu, in > over - f && in <= over)) - 1;
      const uint32_t rank_in = in - __shfl_sync(0xffffffffu, over - f, at);
      if (lane == 0) {
        found_sm[0] = kFine * bin + (uint32_t)(at & 7);
        found_sm[1] = rank_in;
      }
    }
    __syncthreads();
    want = found_sm[1];
    return found_sm[0];
  };
  uint32_t unused0, unused1;
  const uint32_t safe_total = gather(kSafe, unused0, unused1);
  // the class that the border runs through, and how many of it are kept
  const uint32_t cls = safe_total >= (uint32_t)p.keep ? 1 : 0;
  uint32_t want = cls ? (uint32_t)p.keep : (uint32_t)p.keep - safe_total;
  uint32_t prefix = find_bin((int)cls, want) << 21;
  // Second and third digit, over the rows of the class that share the prefix. The histogram of the other class was
  // for this CTA alone, and when the third digit takes the first one's again, every CTA has passed a barrier since.
  for (int digit = 1; digit <= 2; ++digit) {
    const int shift = digit == 1 ? 10 : 0, which = (int)(digit == 1 ? cls ^ 1u : cls);
    const uint32_t mask = digit == 1 ? 0xffe00000u : 0xfffffc00u;
    hist[which][2 * tid] = hist[which][2 * tid + 1] = 0;
    __syncthreads();
    each_chunk([&](int) {
      const uint32_t rows = valid & (cls ? safe_rows : ~safe_rows);
#pragma unroll
      for (int it = 0; it < kGroups && it < groups; ++it)
        if (((rows >> it) & 1u) && (key[it] & mask) == prefix)
          atomicAdd(&hist[which][(key[it] >> shift) & (digit == 1 ? 2047u : 1023u)], 1u);
    });
    __syncthreads();
    if (tid < kCoarse) sum_bins(which, tid);
    sync_all();
    prefix |= find_bin(which, want) << shift;
  }
  // The border key is `prefix`; `want` rows of the class on it are kept, the lowest ones. Rows kept whatever
  // the ties, and those on the border:
  auto judge = [&](uint32_t& kept, uint32_t& border) {
    const uint32_t rows = valid & (cls ? safe_rows : ~safe_rows);
    kept = cls ? 0u : safe_rows;
    border = 0;
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it) {
      if (!((rows >> it) & 1u)) continue;
      if (key[it] > prefix) kept |= 1u << it;
      if (key[it] == prefix) border |= 1u << it;
    }
  };
  uint32_t kept = 0, border = 0, ties = 0, total, before, behind;
  each_chunk([&](int) {
    judge(kept, border);
    ties += __popc(border);
  });
  // rows on the border in this warp's run, then before it in the sequence
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) scan_sm[0][warp] = ties;
  __syncthreads();
  const uint32_t tie_base = scan_warps(0, total);
  if (tid == 0) cnt_sm[kTies] = total;
  sync_all();
  const uint32_t all_ties = gather(kTies, before, behind);
  const uint32_t ties_before = before + tie_base;
  const uint32_t lower = (1u << lane) - 1u;
  // the chunk's kept rows; t: rows on the border before it
  auto settle = [&](uint32_t& t) {
    if (!CACHED) judge(kept, border);
    if (all_ties == want) {
      kept |= border;
      return;
    }
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it) {
      const uint32_t eq = __ballot_sync(0xffffffffu, (border >> it) & 1u);
      if (((border >> it) & 1u) && t + __popc(eq & lower) < want) kept |= 1u << it;
      t += __popc(eq);
    }
  };
  // Holes (given up, below the budget) and movers (kept, behind it): counted, then listed in row order.
  uint32_t holes = 0, movers = 0, t = ties_before;
  each_chunk([&](int at) {
    settle(t);
    const uint32_t low = below(at, p.keep);
    holes += __popc(valid & ~kept & low);
    movers += __popc(kept & ~low);
  });
  holes = __reduce_add_sync(0xffffffffu, holes);
  movers = __reduce_add_sync(0xffffffffu, movers);
  // both in one barrier: a CTA's counts are at most its rows
  if (lane == 0) {
    scan_sm[1][warp] = holes;
    scan_sm[2][warp] = movers;
  }
  __syncthreads();
  const uint32_t hole_base = scan_warps(1, total);
  if (tid == 0) cnt_sm[kHoles] = total;
  const uint32_t mover_base = scan_warps(2, total);
  if (tid == 0) cnt_sm[kMovers] = total;
  sync_all();
  const uint32_t all_holes = gather(kHoles, holes, behind);
  gather(kMovers, movers, behind);
  holes += hole_base;
  movers += mover_base;
  t = ties_before;
  each_chunk([&](int at) {
    if (!CACHED) settle(t);
    const uint32_t low = below(at, p.keep), hole = valid & ~kept & low, mover = kept & ~low;
#pragma unroll
    for (int it = 0; it < kGroups && it < groups; ++it) {
      const int first = at + 32 * it;
      if (first < p.keep) {
        const uint32_t hb = __ballot_sync(0xffffffffu, (hole >> it) & 1u);
        if ((hole >> it) & 1u) moves[1 + p.L + holes + __popc(hb & lower)] = first + lane;
        holes += __popc(hb);
      }
      if (first + 31 >= p.keep) {
        const uint32_t mb = __ballot_sync(0xffffffffu, (mover >> it) & 1u);
        if ((mover >> it) & 1u) moves[1 + movers + __popc(mb & lower)] = first + lane;
        movers += __popc(mb);
      }
    }
  });
  if (rank == 0 && tid == 0) {
    p.len_out[b] = p.keep;
    moves[0] = (int)all_holes;                                 // as many holes as movers
  }
  sync_all();                                                  // no CTA leaves while another reads it
}

// A warp moves two rows at a time: 2.3 KB in flight per warp.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p) {
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int32_t* moves = p.moves + (int64_t)b * (1 + 2 * p.L);
  const int count = moves[0];
  const int64_t base = (int64_t)b * p.S_max;
  for (int i = 2 * (blockIdx.x * 8 + warp); i < count; i += 2 * (int)gridDim.x * 8) {
    int64_t from[2], to[2];
    const bool two = i + 1 < count;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      from[k] = base + moves[1 + min(i + k, count - 1)];
      to[k] = base + moves[1 + p.L + min(i + k, count - 1)];
    }
    uint4 v[2][3];
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (p.kv) {
        const uint4* s = reinterpret_cast<const uint4*>(p.kv + from[k] * 1152);
        v[k][0] = s[lane];
        v[k][1] = s[lane + 32];
        if (lane < 8) v[k][2] = s[lane + 64];
      }
      if (p.k8) c[k] = reinterpret_cast<const uint32_t*>(p.k8 + from[k] * 128)[lane];
    }
    if (lane < (two ? 2 : 1)) {
      const int64_t f = lane ? from[1] : from[0], t = lane ? to[1] : to[0];
      p.acc_out[t] = p.acc[f];
      p.pos_out[t] = p.pos[f];
      if (p.k_scale) p.k_scale[t] = p.k_scale[f];
      if (p.src) p.src[(int64_t)b * p.keep + (t - base)] = (int32_t)(f - base);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !two) break;
      if (p.kv) {
        uint4* d = reinterpret_cast<uint4*>(p.kv + to[k] * 1152);
        d[lane] = v[k][0];
        d[lane + 32] = v[k][1];
        if (lane < 8) d[lane + 64] = v[k][2];
      }
      if (p.k8) reinterpret_cast<uint32_t*>(p.k8 + to[k] * 128)[lane] = c[k];
    }
  }
}

size_t cache_evict_workspace_size(int B, int S_max, int keep) {
  const int64_t L = std::max(0, std::min(keep, S_max - keep));
  return (size_t)(((int64_t)B * (1 + 2 * L) * 4 + 15) & ~(int64_t)15);
}

int launch_cache_evict(const float* acc, const int32_t* pos, const int32_t* kv_len, int B, int S_max, int keep, int recent,
                       int sinks, uint16_t* kv, uint8_t* k8, float* k_scale, float* acc_out, int32_t* pos_out,
                       int32_t* kv_len_out, int32_t* src, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!workspace || ws_bytes < cache_evict_workspace_size(B, S_max, keep)) return DSA_ERR_WORKSPACE;
  EvictParams p = {};
  p.acc = acc;
  p.pos = pos;
  p.kv_len = kv_len;
  p.S_max = S_max;
  p.keep = keep;
  p.recent = recent;
  p.sinks = sinks;
  p.acc_out = acc_out;
  p.pos_out = pos_out;
  p.len_out = kv_len_out;
  p.src = src;
  p.moves = static_cast<int32_t*>(workspace);
  p.L = std::max(0, std::min(keep, S_max - keep));
  p.kv = reinterpret_cast<uint8_t*>(kv);
  p.k8 = k8;
  p.k_scale = k_scale;
  // CTAs per sequence: enough that each takes at most 4096 rows, as far as one wave of SMs goes
  int C = 1;
  // (clusters of 16, which are not portable, were slower for one sequence of 131072: their barriers cost more)
  while (C < kMaxCluster && (int64_t)C * 4096 < S_max && (int64_t)2 * C * B <= dsa_host::device_sm_count()) C *= 2;
  while (C < kMaxCluster && (int64_t)C * kCachedRows < S_max) C *= 2;
  p.C = C;
  const int64_t per_warp = (((int64_t)S_max + C * kWarps - 1) / (C * kWarps) + 31) / 32 * 32;
  const bool cached = per_warp * kWarps <= kCachedRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, cached ? evict_select_kernel<true> : evict_select_kernel<false>, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (p.L == 0) return DSA_OK;                               // the budget holds every row: no moves
  const int blocks = std::max(1, std::min((p.L + 7) / 8, std::max(1, 8 * dsa_host::device_sm_count() / B)));
  return dsa_host::launch(evict_move_kernel, dim3((unsigned)blocks, (unsigned)B), dim3(256), 0, stream, p);
}

}  // namespace dsa
