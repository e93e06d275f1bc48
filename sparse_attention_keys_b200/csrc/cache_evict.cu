// dsa_cache_evict: cuts each sequence's cache back to a budget of rows, by the attention weight its
// rows collected.
//
// Of a sequence's n rows the kept ones are the first `keep` in the order (protected, larger weight,
// lower row), protected meaning among the newest positions or the first ones. Rows need not stay in
// order (every row carries its position), so a kept row below `keep` stays where it is and the i-th
// kept row behind `keep` moves into the i-th row given up before it: sources and destinations never
// overlap, the moves need no order, and the bytes moved are the fewest that leave a dense cache.
//
// select: a cluster of CTAs per sequence holds the rows' (weight, position) in shared memory where
// they fit, and finds the border key by three histogram passes over an order-preserving 32-bit
// image of the weight (11 + 11 + 10 bits), the CTAs reading one another's histograms through
// distributed shared memory; a last pass breaks ties by row and lists movers and holes in order.
// move: a warp per two moved rows. Bound: the n (weight, position) pairs once, and HBM for the moves. 64
// sequences of 12000 to 16384 rows cut to 8192 (about 550 MB): select 23 us, move 95 us, 4.6 TB/s in all; one
// sequence of 131072 cut to 8191: 34 us, most of it the select's barriers and passes.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCachedRows = 16384;       // rows per CTA kept in shared memory (8 bytes each)
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
__device__ __forceinline__ uint2 ld_cluster_2(const void* p, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
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

// CACHED: the rows of a CTA fit into shared memory.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t rows_sm[];        // [per][2]: weight bits, position
  __shared__ __align__(16) uint32_t hist[2][kBins];                        // ordinary and protected rows
  __shared__ uint32_t cnt_sm[8];                             // this CTA's words that the others read (kNewest ...)
  __shared__ uint32_t warp_sm[kWarps];
  __shared__ uint32_t found_sm[2];
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
      for (int r = n + (int)rank * kThreads + tid; r < p.keep; r += p.C * kThreads) src[r] = -1;
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
  int newest = INT32_MIN;
  for (int r = r0 + tid; r < r1; r += kThreads) {
    const int ps = pos[r];
    if (CACHED) *reinterpret_cast<uint2*>(rows_sm + 2 * (r - r0)) = make_uint2(__float_as_uint(acc[r]), (uint32_t)ps);
    newest = max(newest, ps);
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
  // A row's key and class; shared memory holds (weight, position) until the next loop, then these.
  auto row_of = [&](int r) {
    return CACHED ? *reinterpret_cast<const uint2*>(rows_sm + 2 * (r - r0))
                  : make_uint2(weight_key(acc[r]), protects(pos[r]) ? 1u : 0u);
  };

  // first digit, for both classes
  uint32_t safe = 0;
  for (int r = r0 + tid; r < r1; r += kThreads) {
    const uint2 row = CACHED ? *reinterpret_cast<const uint2*>(rows_sm + 2 * (r - r0))
                               : make_uint2(__float_as_uint(acc[r]), (uint32_t)pos[r]);
    const uint32_t key = weight_key(__uint_as_float(row.x));
    const bool yes = protects((int)row.y);
    if (CACHED) *reinterpret_cast<uint2*>(rows_sm + 2 * (r - r0)) = make_uint2(key, yes ? 1u : 0u);
    safe += yes;
    atomicAdd(&hist[yes ? 1 : 0][key >> 21], 1u);
  }
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0 && safe) atomicAdd(&cnt_sm[kSafe], safe);
  sync_all();
  // exclusive sum over the block's threads of v, and the total
  auto block_scan = [&](uint32_t v, uint32_t& total) {
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) warp_sm[warp] = s;
    __syncthreads();
    uint32_t ws = warp_sm[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, ws, d);
      if (lane >= d) ws += o;
    }
    total = __shfl_sync(0xffffffffu, ws, 31);
    const uint32_t base = __shfl_sync(0xffffffffu, ws, warp ? warp - 1 : 0);
    return (warp ? base : 0u) + s - v;
  };
  // The bin of histogram `which` in which the want-th largest key lies; `want` becomes its rank among the
  // bin's keys. Every CTA adds up all histograms for itself, two bins a thread: that costs one cluster
  // barrier a digit (sharing the bins out moves less, but took two more barriers and twice the time).
  auto find_bin = [&](int which, uint32_t& want) {
    uint32_t h0 = 0, h1 = 0, total;
    if (p.C == 1) {
      h0 = hist[which][2 * tid];
      h1 = hist[which][2 * tid + 1];
    } else {
      uint2 h[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) h[c] = c < p.C ? ld_cluster_2(&hist[which][2 * tid], (uint32_t)c) : make_uint2(0, 0);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        h0 += h[c].x;
        h1 += h[c].y;
      }
    }
    const uint32_t before = block_scan(h0 + h1, total);       // keys in lower bins
    const uint32_t up1 = total - before - h0 - h1, up0 = up1 + h1;     // keys in bins above
    if (want > up1 && want <= up1 + h1) {
      found_sm[0] = 2 * tid + 1;
      found_sm[1] = up1;
    } else if (want > up0 && want <= up0 + h0) {
      found_sm[0] = 2 * tid;
      found_sm[1] = up0;
    }
    __syncthreads();
    want -= found_sm[1];
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
    for (int r = r0 + tid; r < r1; r += kThreads) {
      const uint2 row = row_of(r);
      if ((row.x & mask) == prefix && row.y == cls)
        atomicAdd(&hist[which][(row.x >> shift) & (digit == 1 ? 2047u : 1023u)], 1u);
    }
    sync_all();
    prefix |= find_bin(which, want) << shift;
  }
  // The border key is `prefix`; `want` rows of the class on it are kept, the lowest ones.
  // 0: given up, 1: kept, 2: kept if among the first `want` on the border
  auto judge = [&](int r) {
    const uint2 row = row_of(r);
    return row.y != cls ? (int)row.y : (row.x > prefix ? 1 : (row.x == prefix ? 2 : 0));
  };
  // rows on the border in this warp's run, then before it in the sequence
  const int w0 = min(r1, r0 + warp * per_warp), w1 = min(r1, w0 + per_warp);
  auto exclusive = [&](uint32_t mine, int slot) {             // over the cluster's warps, row order
    uint32_t total, before, behind;
    const uint32_t base = block_scan(lane == 0 ? mine : 0u, total);
    if (tid == 0) cnt_sm[slot] = total;
    sync_all();
    gather(slot, before, behind);
    return before + __shfl_sync(0xffffffffu, base, 0);
  };
  // two bits a row keep the judgement of the first 16 groups of a warp's run
  uint32_t codes = 0, ties = 0;
  auto code = [&](int it, int r) { return it < 16 ? (int)((codes >> (2 * it)) & 3u) : (r < w1 ? judge(r) : 0); };
  for (int r = w0 + lane, it = 0; r - lane < w1; r += 32, ++it) {
    const int j = r < w1 ? judge(r) : 0;
    if (it < 16) codes |= (uint32_t)j << (2 * it);
    ties += __popc(__ballot_sync(0xffffffffu, j == 2));
  }
  const uint32_t ties_before = exclusive(ties, kTies);
  // holes (given up, below the budget) and movers (kept, behind it): counted, then listed in row order
  const uint32_t lower = (1u << lane) - 1u;
  uint32_t holes = 0, movers = 0;
  {
    uint32_t t = ties_before;
    for (int r = w0 + lane, it = 0; r - lane < w1; r += 32, ++it) {
      const int j = code(it, r);
      const uint32_t eq = __ballot_sync(0xffffffffu, j == 2);
      const bool kept = j == 1 || (j == 2 && t + __popc(eq & lower) < want);
      t += __popc(eq);
      holes += __popc(__ballot_sync(0xffffffffu, r < w1 && !kept && r < p.keep));
      movers += __popc(__ballot_sync(0xffffffffu, kept && r >= p.keep));
    }
  }
  // both in one barrier: a CTA's counts are at most its rows
  uint32_t total, behind;
  const uint32_t hole_base = block_scan(lane == 0 ? holes : 0u, total);
  if (tid == 0) cnt_sm[kHoles] = total;
  const uint32_t mover_base = block_scan(lane == 0 ? movers : 0u, total);
  if (tid == 0) cnt_sm[kMovers] = total;
  sync_all();
  const uint32_t all_holes = gather(kHoles, holes, behind);
  gather(kMovers, movers, behind);
  holes += __shfl_sync(0xffffffffu, hole_base, 0);
  movers += __shfl_sync(0xffffffffu, mover_base, 0);
  // the state of rows that stay is read four groups ahead of the walk that needs it
  float a4[4];
  int p4[4];
  auto fetch = [&](int r) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = r + 32 * k;
      if (at < w1 && at < p.keep) {
        if (copy_acc) a4[k] = acc[at];
        if (copy_pos) p4[k] = pos[at];
      }
    }
  };
  uint32_t t = ties_before;
  for (int r4 = w0 + lane, it4 = 0; r4 - lane < w1; r4 += 128, it4 += 4) {
    fetch(r4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r4 + 32 * k;
      if (r - lane >= w1) break;
      const int j = code(it4 + k, r);
      const uint32_t eq = __ballot_sync(0xffffffffu, j == 2);
      const bool kept = j == 1 || (j == 2 && t + __popc(eq & lower) < want);
      t += __popc(eq);
      const bool hole = r < w1 && !kept && r < p.keep, mover = kept && r >= p.keep;
      const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
      if (hole) moves[1 + p.L + holes + __popc(hb & lower)] = r;
      if (mover) moves[1 + movers + __popc(mb & lower)] = r;
      if (kept && r < p.keep) {
        if (copy_acc) acc_out[r] = a4[k];
        if (copy_pos) pos_out[r] = p4[k];
        if (src) src[r] = r;
      }
      holes += __popc(hb);
      movers += __popc(mb);
    }
  }
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
  const size_t smem = cached ? (size_t)per_warp * kWarps * 8 : 0;
  static uint64_t seen[dsa_host::kMaxSetupDevices];
  if (dsa_host::needs_setup(seen, nullptr)) {
    if (cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCachedRows * 8) != cudaSuccess)
      return DSA_ERR_CUDA;
    dsa_host::mark_setup(seen);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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
