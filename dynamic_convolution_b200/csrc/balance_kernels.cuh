// Kernels of the router's load-balance loss (include/dynconv_train.h).
//
// A row of n attentions is held by L neighbouring lanes of a warp, V values in
// each lane's registers (n <= L * V), so a warp holds 32 / L rows: lane l of a
// row owns the elements (c * L + l) * 4 + q, c = 0.., q = 0..3, which 16-byte
// loads fetch contiguously. The top k are found by k rounds of "largest value,
// then lowest index among its holders" over the row's lanes.
#pragma once

#include <climits>
#include <cstdint>

namespace dct {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxN = 1024;
constexpr int kBalMaxTopK = 32;
constexpr int kBalFinishThreads = 1024;

// Ascending integer order of floats: numbers as themselves, -0 as +0, NaN
// below everything (above kTaken, the mark of a value already chosen).
constexpr int kTaken = INT_MIN;
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return v != v ? INT_MIN + 1 : (b ^ ((b >> 31) & 0x7fffffff));
}

template <int L>
__device__ __forceinline__ int row_max(int v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ int row_min(int v) {
  if constexpr (L == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's V elements of a row (0 where the row ends or `live` is false).
template <int L, int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int n, int lane, bool vec,
                                         bool live, float (&a)[V]) {
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = (c * L + lane) * 4;
    if (vec) {  // n is a multiple of 4 here
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live && e < n) f = *reinterpret_cast<const float4*>(row + e);
      a[4 * c] = f.x; a[4 * c + 1] = f.y; a[4 * c + 2] = f.z; a[4 * c + 3] = f.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) a[4 * c + q] = live && e + q < n ? row[e + q] : 0.f;
    }
  }
}

template <int L, int V>
__device__ __forceinline__ int element_of(int slot, int lane) {
  return ((slot >> 2) * L + lane) * 4 + (slot & 3);
}

struct BalParams {
  int rows, groups, n, top_k, sigmoid, vec;
  long long stride;            // floats between rows of alpha
  const float* alpha;
  const unsigned char* mask;   // or null
  double* part_sum;            // [parts][groups][n]
  int* part_count;             // [parts][groups][n]
  int* part_kept;              // [parts]
};

// One CTA: every (gridDim.x)-th batch of kBalWarps * 32 / L rows of one group
// (blockIdx.y), its column sums in fp64 registers and its counts in shared
// memory, written as this part's partial results.
template <int L, int V>
__global__ void __launch_bounds__(kBalThreads)
balance_forward_kernel(BalParams p) {
  constexpr int R = 32 / L;  // rows per warp
  __shared__ int s_count[kBalMaxN];
  __shared__ double s_sum[kBalMaxN];
  __shared__ int s_kept;
  const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31, lane = wl % L, sub = wl / L;
  const int j = blockIdx.y, n = p.n;
  const bool select = p.top_k < n;
  for (int i = tid; i < n; i += kBalThreads) {
    s_count[i] = 0;
    s_sum[i] = 0.0;
  }
  if (tid == 0) s_kept = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double acc[V];
#pragma unroll
  for (int s = 0; s < V; ++s) acc[s] = 0.0;
  int kept = 0;
  const long long step = static_cast<long long>(gridDim.x) * (kBalWarps * R);
  for (long long base = (static_cast<long long>(blockIdx.x) * kBalWarps + warp) * R; base < p.rows;
       base += step) {
    const long long r = base + sub;
    const bool live = r < p.rows && (!p.mask || p.mask[r]);
    float a[V];
    load_row<L, V>(p.alpha + r * p.stride + static_cast<long long>(j) * n, n, lane, p.vec, live, a);
    if (live && lane == 0) ++kept;
    if (select) {
      int key[V];
#pragma unroll
      for (int s = 0; s < V; ++s)
        key[s] = element_of<L, V>(s, lane) < n ? order_key(a[s]) : kTaken;
      for (int t = 0; t < p.top_k; ++t) {
        int best = key[0], slot = 0;
#pragma unroll
        for (int s = 1; s < V; ++s)
          if (key[s] > best) {
            best = key[s];
            slot = s;
          }
        const int top = row_max<L>(best);
        const int mine = element_of<L, V>(slot, lane);
        const int at = row_min<L>(best == top ? mine : INT_MAX);
        if (live && at == mine) {  // the holder
          atomicAdd(&s_count[at], 1);
#pragma unroll
          for (int s = 0; s < V; ++s)
            if (s == slot) key[s] = kTaken;
        }
      }
    }
    if (p.sigmoid) {
      float total = 0.f;
#pragma unroll
      for (int s = 0; s < V; ++s) total += a[s];
      total = row_sum<L>(total);
#pragma unroll
      for (int s = 0; s < V; ++s) a[s] = total != 0.f ? __fdiv_rn(a[s], total) : 0.f;
    }
#pragma unroll
    for (int s = 0; s < V; ++s) acc[s] += static_cast<double>(a[s]);
  }
  // rows of the warp, then the warps in order
#pragma unroll
  for (int s = 0; s < V; ++s)
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) acc[s] += __shfl_xor_sync(0xffffffffu, acc[s], o);
  if (kept) atomicAdd(&s_kept, kept);
  for (int w = 0; w < kBalWarps; ++w) {
    if (warp == w && sub == 0) {
#pragma unroll
      for (int s = 0; s < V; ++s) {
        const int e = element_of<L, V>(s, lane);
        if (e < n) s_sum[e] += acc[s];
      }
    }
    __syncthreads();
  }
  const long long out = (static_cast<long long>(blockIdx.x) * p.groups + j) * n;
  for (int i = tid; i < n; i += kBalThreads) {
    p.part_sum[out + i] = s_sum[i];
    p.part_count[out + i] = select ? s_count[i] : s_kept;
  }
  if (j == 0 && tid == 0) p.part_kept[blockIdx.x] = s_kept;
}

struct BalFinish {
  int parts, width, n, top_k, groups;  // width = groups * n
  float coef;
  const double* part_sum;
  const int* part_count;
  const int* part_kept;
  int* counts;
  float* mean;
  int* rows_kept;
  float* loss;
};

// The parts added in order, the means and the loss: one CTA.
__global__ void __launch_bounds__(kBalFinishThreads) balance_finish_kernel(BalFinish p) {
  __shared__ double s_loss[kBalFinishThreads / 32];
  __shared__ int s_kept;
  const int tid = threadIdx.x;
  if (tid == 0) s_kept = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int k = 0;
  for (int q = tid; q < p.parts; q += kBalFinishThreads) k += p.part_kept[q];
  if (k) atomicAdd(&s_kept, k);
  __syncthreads();
  const int kept = s_kept;
  const double over = kept > 0 ? 1.0 / kept : 0.0;
  double dot = 0.0;
  for (int i = tid; i < p.width; i += kBalFinishThreads) {
    double sum = 0.0;
    int count = 0;
    for (int q = 0; q < p.parts; ++q) {
      sum += p.part_sum[static_cast<long long>(q) * p.width + i];
      count += p.part_count[static_cast<long long>(q) * p.width + i];
    }
    const double mean = sum * over;
    p.counts[i] = count;
    p.mean[i] = static_cast<float>(mean);
    dot += static_cast<double>(count) * over * mean;
  }
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if ((tid & 31) == 0) s_loss[tid >> 5] = dot;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    for (int w = 0; w < kBalFinishThreads / 32; ++w) total += s_loss[w];
    *p.loss = static_cast<float>(static_cast<double>(p.coef) * p.n /
                                 (static_cast<double>(p.top_k) * p.groups) * total);
    *p.rows_kept = kept;
  }
}

struct BalBack {
  int rows, groups, n, width, top_k, vec, accumulate;
  long long stride, dstride;
  float coef;
  const float* alpha;          // sigmoid only
  const unsigned char* mask;   // or null
  const int* counts;
  const int* rows_kept;
  const float* dloss;          // or null
  float* dalpha;
};

// coef n / (top_k groups) dloss / M^2: the gradient per count.
__device__ __forceinline__ double slope_of(const BalBack& p) {
  const int kept = *p.rows_kept;
  if (kept <= 0) return 0.0;
  const double d = p.dloss ? static_cast<double>(*p.dloss) : 1.0;
  return d * p.coef * p.n / (static_cast<double>(p.top_k) * p.groups) / kept / kept;
}

// SOFTMAX: the same row of coefficients on every kept row. A thread owns four
// columns and walks down the rows.
__global__ void __launch_bounds__(kBalThreads) balance_backward_softmax_kernel(BalBack p, int tx) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ty = kBalThreads / tx;
  const int col = (blockIdx.y * tx + threadIdx.x % tx) * 4;
  if (col >= p.width) return;
  const double slope = slope_of(p);
  float c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c[q] = col + q < p.width ? static_cast<float>(slope * p.counts[col + q]) : 0.f;
  const long long step = static_cast<long long>(gridDim.x) * ty;
#pragma unroll 4
  for (long long r = static_cast<long long>(blockIdx.x) * ty + threadIdx.x / tx; r < p.rows;
       r += step) {
    const bool live = !p.mask || p.mask[r];
    if (!live && p.accumulate) continue;
    float* d = p.dalpha + r * p.dstride + col;
    if (p.vec) {
      float4 o = live ? make_float4(c[0], c[1], c[2], c[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.accumulate) {
        const float4 b = *reinterpret_cast<const float4*>(d);
        o.x += b.x; o.y += b.y; o.z += b.z; o.w += b.w;
      }
      *reinterpret_cast<float4*>(d) = o;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (col + q < p.width) d[q] = p.accumulate ? d[q] + c[q] : (live ? c[q] : 0.f);
    }
  }
}

// SIGMOID: (c - sum_l c_l p_l) / S of every kept row; rows held as in the forward.
template <int L, int V>
__global__ void __launch_bounds__(kBalThreads) balance_backward_sigmoid_kernel(BalBack p) {
  constexpr int R = 32 / L;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31, lane = wl % L, sub = wl / L;
  const int j = blockIdx.y, n = p.n;
  const double slope = slope_of(p);
  float c[V];
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int e = element_of<L, V>(s, lane);
    c[s] = e < n ? static_cast<float>(slope * p.counts[j * n + e]) : 0.f;
  }
  const long long step = static_cast<long long>(gridDim.x) * (kBalWarps * R);
  for (long long base = (static_cast<long long>(blockIdx.x) * kBalWarps + warp) * R; base < p.rows;
       base += step) {
    const long long r = base + sub;
    const bool live = r < p.rows && (!p.mask || p.mask[r]);
    float a[V];
    load_row<L, V>(p.alpha + r * p.stride + static_cast<long long>(j) * n, n, lane, p.vec, live, a);
    float total = 0.f;
#pragma unroll
    for (int s = 0; s < V; ++s) total += a[s];
    total = row_sum<L>(total);
    float dot = 0.f;
#pragma unroll
    for (int s = 0; s < V; ++s) {
      a[s] = total != 0.f ? __fdiv_rn(a[s], total) : 0.f;
      dot += c[s] * a[s];
    }
    dot = row_sum<L>(dot);
    if (r >= p.rows || (!live && p.accumulate)) continue;  // (a row's lanes agree)
    float* d = p.dalpha + r * p.dstride + static_cast<long long>(j) * n;
#pragma unroll
    for (int ch = 0; ch < V / 4; ++ch) {
      const int e = (ch * L + lane) * 4;
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = live && total != 0.f ? __fdiv_rn(c[4 * ch + q] - dot, total) : 0.f;
      if (p.vec) {
        if (e < n) {
          float4* at = reinterpret_cast<float4*>(d + e);
          float4 b = p.accumulate ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
          *at = make_float4(b.x + o[0], b.y + o[1], b.z + o[2], b.w + o[3]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < n) d[e + q] = p.accumulate ? d[e + q] + o[q] : o[q];
      }
    }
  }
}

}  // namespace dct
