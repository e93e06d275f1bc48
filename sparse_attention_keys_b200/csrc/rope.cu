// dsa_rope: rotary positions on part of each head, for any layout the framework's models use.
//
// y = scale * R(pos * f_i) x on each pair i of the rotary features; the others are copied. The
// angle is never formed in floating point: f_i comes as a fraction of a turn in units of 2^-64, so
// pos * f_i modulo 2^64 is the fraction of a turn at any position, exact to the frequency's last
// bit, and is rounded once (to fp32, at most half a turn) for sincospi. No table is read.
//
// Bound by HBM: each element once in, once out. A block takes a run of consecutive (row, head)
// units, about 1024 items of 16 bytes, computes the sines of the rows it spans once into shared
// memory while its first loads are in flight, and every head of a row shares them. Rows or
// offsets that 16-byte accesses do not fit run the same code one pair at a time. 4096 rows of 64
// heads of 128 in fp32 (268 MB) take 47 us, 5.7 TB/s or 89% of the measured copy.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                // items in flight per thread
constexpr int kMaxCs = 4096;             // (row, pair) entries per block

// i / d for i < 2^16, d <= 2^16: m = ceil(2^32 / d) is off by less than d / 2^32 per unit of i
struct SmallDiv {
  uint32_t d, m;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return d == 1 ? i : __umulhi(i, m); }
};
SmallDiv small_div(uint32_t d) { return {d, (uint32_t)(((1ull << 32) + d - 1) / d)}; }

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

struct RopeParams {
  const void* x;
  void* out;
  int64_t x_row, x_head, out_row, out_head;      // strides, elements
  int64_t units;                                 // rows * heads
  const int32_t* pos;
  const uint64_t* freqs;
  float scale;
  int heads, offset, pairs, dim;
  int inverse;
  int unit_items, rot_items, pass_items;         // per unit
  int per_block;                                 // units per block
  SmallDiv div_items, div_heads, div_pairs;
};

// V elements per access; a rotary item is V elements of interleaved pairs (two for V = 1), or V
// first and V second elements of the half layout.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int E = INTERLEAVED ? (V > 1 ? V : 2) : V;       // elements of the first access
  extern __shared__ float2 cs[];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t u0 = (int64_t)blockIdx.x * p.per_block;
  const int nu = (int)min((int64_t)p.per_block, p.units - u0);
  const int64_t row0 = u0 / p.heads;
  const uint32_t head0 = (uint32_t)(u0 - row0 * p.heads);
  const int items = nu * p.unit_items;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);

  alignas(16) T a[kBatch][E];
  alignas(16) T b[kBatch][INTERLEAVED ? 1 : V];
  auto locate = [&](int i, uint32_t& row, int64_t& xo, int64_t& oo, int& item) {
    const uint32_t unit = p.div_items((uint32_t)i);
    item = i - (int)unit * p.unit_items;
    const uint32_t hr = head0 + unit;                        // < heads + per_block
    row = p.div_heads(hr);
    const int64_t head = hr - row * p.heads, r = row0 + row;
    xo = r * p.x_row + head * p.x_head;
    oo = r * p.out_row + head * p.out_head;
  };
  // first element of a copied item: those before the rotary features, then those behind them
  auto pass_at = [&](int item) {
    const int e = (item - p.rot_items) * V;
    return e < p.offset ? e : e + 2 * p.pairs;
  };
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kThreads + (int)threadIdx.x;
      if (i >= items) continue;
      uint32_t row;
      int64_t xo, oo;
      int item;
      locate(i, row, xo, oo, item);
      if (item < p.rot_items) {
        if (INTERLEAVED) {
          if (V > 1) *reinterpret_cast<Vec<T, V>*>(a[k]) = *reinterpret_cast<const Vec<T, V>*>(x + xo + p.offset + item * E);
          else {
            a[k][0] = x[xo + p.offset + item * 2];
            a[k][E - 1] = x[xo + p.offset + item * 2 + 1];
          }
        } else {
          *reinterpret_cast<Vec<T, V>*>(a[k]) = *reinterpret_cast<const Vec<T, V>*>(x + xo + p.offset + item * V);
          *reinterpret_cast<Vec<T, V>*>(b[k]) =
              *reinterpret_cast<const Vec<T, V>*>(x + xo + p.offset + p.pairs + item * V);
        }
      } else {
        *reinterpret_cast<Vec<T, V>*>(a[k]) = *reinterpret_cast<const Vec<T, V>*>(x + xo + pass_at(item));
      }
    }
  };
  load(0);
  // cos and sin of every (row, pair) of the block
  const int nrows = (int)p.div_heads(head0 + (uint32_t)nu - 1) + 1;
  for (int i = threadIdx.x; i < nrows * p.pairs; i += kThreads) {
    const uint32_t r = p.div_pairs((uint32_t)i);
    const uint64_t turn = (uint64_t)(int64_t)__ldg(p.pos + row0 + r) * __ldg(p.freqs + (i - r * p.pairs));
    // a signed fraction of a turn, in units of half a turn
    float s, c;
    sincospif(__ll2float_rn((long long)turn) * 0x1p-63f, &s, &c);
    cs[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
  }
  __syncthreads();
  for (int base = 0; base < items; base += kBatch * kThreads) {
    if (base > 0) load(base);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kThreads + (int)threadIdx.x;
      if (i >= items) continue;
      uint32_t row;
      int64_t xo, oo;
      int item;
      locate(i, row, xo, oo, item);
      if (item < p.rot_items) {
        if (INTERLEAVED) {
          const float2* t = cs + row * p.pairs + item * (E / 2);
          alignas(16) T y[E];
#pragma unroll
          for (int j = 0; j < E / 2; ++j) {
            const float c = t[j].x, s = t[j].y, u = Elem<T>::get(a[k][2 * j]), v = Elem<T>::get(a[k][2 * j + 1]);
            y[2 * j] = Elem<T>::put(fmaf(u, c, -(v * s)));
            y[2 * j + 1] = Elem<T>::put(fmaf(u, s, v * c));
          }
          if (V > 1) *reinterpret_cast<Vec<T, V>*>(out + oo + p.offset + item * E) = *reinterpret_cast<Vec<T, V>*>(y);
          else {
            out[oo + p.offset + item * 2] = y[0];
            out[oo + p.offset + item * 2 + 1] = y[E - 1];
          }
        } else {
          const float2* t = cs + row * p.pairs + item * V;
          Vec<T, V> y, z;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float c = t[j].x, s = t[j].y, u = Elem<T>::get(a[k][j]), v = Elem<T>::get(b[k][j]);
            y.v[j] = Elem<T>::put(fmaf(u, c, -(v * s)));
            z.v[j] = Elem<T>::put(fmaf(u, s, v * c));
          }
          *reinterpret_cast<Vec<T, V>*>(out + oo + p.offset + item * V) = y;
          *reinterpret_cast<Vec<T, V>*>(out + oo + p.offset + p.pairs + item * V) = z;
        }
      } else {
        *reinterpret_cast<Vec<T, V>*>(out + oo + pass_at(item)) = *reinterpret_cast<Vec<T, V>*>(a[k]);
      }
    }
  }
}

template <typename T, int V>
int launch_typed(RopeParams p, bool interleaved, bool in_place, cudaStream_t stream) {
  const int e = interleaved ? (V > 1 ? V : 2) : V;
  p.rot_items = interleaved ? 2 * p.pairs / e : p.pairs / V;
  p.pass_items = in_place ? 0 : (p.dim - 2 * p.pairs) / V;
  p.unit_items = p.rot_items + p.pass_items;
  // 1024 items a block, down to one a thread where that leaves SMs without work, and no more sines
  // than its shared memory holds (16384 keys of 64 features: 10.4 us with 1024 items, 6.0 with 256)
  int64_t items = kBatch * kThreads;
  while (items > kThreads && p.units * p.unit_items < items * 8 * dsa_host::device_sm_count()) items /= 2;
  const int most = std::max(1, std::min((int)items / p.unit_items, kMaxCs / p.pairs));
  p.per_block = (int)std::min<int64_t>(most, p.units);
  p.div_items = small_div((uint32_t)p.unit_items);
  p.div_heads = small_div((uint32_t)p.heads);
  p.div_pairs = small_div((uint32_t)p.pairs);
  const int rows = p.heads == 1 ? p.per_block : (p.per_block + 2 * p.heads - 2) / p.heads;
  const size_t smem = (size_t)rows * p.pairs * sizeof(float2);
  const int64_t blocks = (p.units + p.per_block - 1) / p.per_block;
  if (blocks > 0x7fffffffLL) return DSA_ERR_INVALID_ARG;
  return interleaved ? dsa_host::launch(rope_kernel<T, V, true>, dim3((unsigned)blocks), dim3(kThreads), smem, stream, p)
                     : dsa_host::launch(rope_kernel<T, V, false>, dim3((unsigned)blocks), dim3(kThreads), smem, stream, p);
}

template <typename T>
int launch_elem(const RopeParams& p, bool interleaved, bool in_place, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte accesses: every address and every boundary inside a head lies on 16 bytes
  const int64_t s = p.x_row | p.x_head | p.out_row | p.out_head | p.offset | p.dim | (interleaved ? 2 * p.pairs : p.pairs);
  const bool wide = s % V == 0 && dsa_host::aligned16(p.x) && dsa_host::aligned16(p.out);
  return wide ? launch_typed<T, V>(p, interleaved, in_place, stream) : launch_typed<T, 1>(p, interleaved, in_place, stream);
}

}  // namespace

int launch_rope(const void* x, int dtype, int64_t rows, int heads, int64_t x_row, int64_t x_head, int dim, int offset,
                int pairs, const int32_t* pos, const uint64_t* freqs, float scale, bool interleaved, bool inverse, void* out,
                int64_t out_row, int64_t out_head, cudaStream_t stream) {
  RopeParams p = {};
  p.x = x;
  p.out = out;
  p.x_row = x_row;
  p.x_head = x_head;
  p.out_row = out_row;
  p.out_head = out_head;
  p.units = rows * heads;
  p.pos = pos;
  p.freqs = freqs;
  p.scale = scale;
  p.heads = heads;
  p.offset = offset;
  p.pairs = pairs;
  p.dim = dim;
  p.inverse = inverse;
  const bool in_place = out == x;
  if (dtype == DSA_F32) return launch_elem<float>(p, interleaved, in_place, stream);
  if (dtype == DSA_BF16) return launch_elem<__nv_bfloat16>(p, interleaved, in_place, stream);
  return launch_elem<__half>(p, interleaved, in_place, stream);
}

}  // namespace dsa
