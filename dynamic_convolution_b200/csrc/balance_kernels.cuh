// Kernels of the router's load-balance loss (include/dynconv_train.h).
//
// A row of n attentions is held by L neighbouring lanes of a warp, V values in
// each lane's registers (n <= L * V), so a warp holds 32 / L rows: lane l of a
// row owns the elements (c * L + l) * 4 + q, c = 0.., q = 0..3 (four to a chunk c),
// which 16-byte loads fetch contiguously. More values per lane mean fewer steps
// across lanes, which the top k need in every round.
#pragma once

#include <climits>
#include <cstdint>

#include <cooperative_groups.h>

namespace dct {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxN = 1024;
constexpr int kBalMaxTopK = 32;
constexpr int kBalCluster = 8;          // CTAs of a cluster at most
constexpr int kBalFinishThreads = 512;

// Largest (NaN ignored unless all are) and smallest over a row's lanes.
template <int L>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (L == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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
  float coef;
  long long stride;            // floats between rows of alpha
  const float* alpha;
  const unsigned char* mask;   // or null
  double* part_sum;            // [parts][groups][n]
  int* part_count;             // [parts][groups][n]
  int* part_kept;              // [parts]
  int* counts;                 // results (the one-launch form)
  float* mean;
  int* rows_kept;
  float* loss;
};

// Running sums as an fp32 pair: `hi` the rounded sum, `lo` the rounding errors,
// which six more additions recover exactly (two values to an instruction). That
// keeps what an fp64 sum would at the rate of fp32: the conversions to fp64 took
// as long as the rest of the kernel.
struct Sum2 {
  unsigned long long hi, lo;
};
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long sub2(unsigned long long a, unsigned long long b) {
  unsigned long long r;  // a - b, rounded once
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(pack2(-1.f, -1.f)), "l"(a));
  return r;
}
__device__ __forceinline__ void accumulate(Sum2& t, unsigned long long x) {
  const unsigned long long s = add2(t.hi, x), b = sub2(s, t.hi);
  t.lo = add2(t.lo, add2(sub2(t.hi, sub2(s, b)), sub2(x, b)));
  t.hi = s;
}
__device__ __forceinline__ double total_of(float hi, float lo) {
  // (an infinite sum's error terms are NaN)
  return isfinite(hi) ? static_cast<double>(hi) + static_cast<double>(lo) : static_cast<double>(hi);
}

// The k largest of each row, k rounds: the largest value left, the lowest of the
// chunks that hold it, the lowest of that chunk's elements. Chosen elements (and
// those past the row's end) become NaN, which no maximum takes; only the chosen
// chunk's maximum is taken again. Returns the chosen slots of this lane as bits.
// `a` is used up.
template <int L, int V>
__device__ __forceinline__ uint32_t choose(float (&a)[V], int n, int lane, bool live, int k) {
  constexpr int C = V / 4;
  const float kNone = __int_as_float(0x7fffffff);
  float g[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if ((c * L + lane) * 4 + 3 >= n) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((c * L + lane) * 4 + q >= n) a[4 * c + q] = kNone;
    }
    g[c] = fmaxf(fmaxf(a[4 * c], a[4 * c + 1]), fmaxf(a[4 * c + 2], a[4 * c + 3]));
  }
  uint32_t taken = 0;
  float top = 0.f;
  for (int t = 0; t < k; ++t) {
    float best = g[0];
#pragma unroll
    for (int c = 1; c < C; ++c) best = fmaxf(best, g[c]);
    top = row_max<L>(best);
    int at = INT_MAX;
#pragma unroll
    for (int c = C - 1; c >= 0; --c)
      if (g[c] == top) at = c * L + lane;
    const int first = row_min<L>(at);
    const bool mine = live && at == first && first != INT_MAX;
    const int chunk = L == 32 ? first / 32 : at / L;  // one for the whole warp where L is 32
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (chunk == c && mine) {
        const bool q0 = a[4 * c] == top, q1 = a[4 * c + 1] == top, q2 = a[4 * c + 2] == top;
        const int q = q0 ? 0 : q1 ? 1 : q2 ? 2 : 3;
        taken |= 1u << (4 * c + q);
        a[4 * c] = q == 0 ? kNone : a[4 * c];
        a[4 * c + 1] = q == 1 ? kNone : a[4 * c + 1];
        a[4 * c + 2] = q == 2 ? kNone : a[4 * c + 2];
        a[4 * c + 3] = q == 3 ? kNone : a[4 * c + 3];
        g[c] = fmaxf(fmaxf(a[4 * c], a[4 * c + 1]), fmaxf(a[4 * c + 2], a[4 * c + 3]));
      }
    }
  }
  // A row with fewer than k numbers: its NaN in the order of their places.
  if (__any_sync(0xffffffffu, live && top != top)) {
    int chosen = __popc(taken);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) chosen += __shfl_xor_sync(0xffffffffu, chosen, o);
    for (int t = 0; t < k; ++t) {
      int at = INT_MAX, slot = 0;
#pragma unroll
      for (int s = V - 1; s >= 0; --s) {
        const int e = element_of<L, V>(s, lane);
        if (e < n && !((taken >> s) & 1u)) {
          at = e;
          slot = s;
        }
      }
      const int first = row_min<L>(at);
      if (live && chosen + t < k && at == first && at != INT_MAX) taken |= 1u << slot;
    }
  }
  return taken;
}

// p = a / S with S = sum a, and 0 where S = 0: a reciprocal and products, except
// where the reciprocal of so small a sum would overflow.
template <int L, int V>
__device__ __forceinline__ float normalise(float (&a)[V]) {
  float total = 0.f;
#pragma unroll
  for (int s = 0; s < V; ++s) total += a[s];
  total = row_sum<L>(total);
  if (fabsf(total) < 1e-30f) {
#pragma unroll
    for (int s = 0; s < V; ++s) a[s] = total != 0.f ? __fdiv_rn(a[s], total) : 0.f;
  } else {
    const float inv = __frcp_rn(total);
#pragma unroll
    for (int s = 0; s < V; ++s) a[s] *= inv;
  }
  return total;
}

struct BalShared {
  double sum[kBalMaxN];
  int count[kBalMaxN];
  int kept;
};

// The column sums and counts of one group over every gridwise-strided batch of
// rows, into `sh` (which no thread may still be reading).
template <int L, int V>
__device__ __forceinline__ void group_sums(const BalParams& p, int j, long long part,
                                           long long parts, BalShared& sh) {
  constexpr int R = 32 / L;          // rows per warp
  constexpr bool kRegCounts = V <= 8;  // counts in registers; else in shared memory
  const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31, lane = wl % L, sub = wl / L;
  const int n = p.n;
  const bool select = p.top_k < n;
  for (int i = tid; i < n; i += kBalThreads) {
    sh.count[i] = 0;
    sh.sum[i] = 0.0;
  }
  if (tid == 0) sh.kept = 0;
  __syncthreads();
  Sum2 acc[V / 2];
  int cnt[kRegCounts ? V : 1];
#pragma unroll
  for (int s = 0; s < V / 2; ++s) acc[s].hi = acc[s].lo = 0ull;
#pragma unroll
  for (int s = 0; s < (kRegCounts ? V : 1); ++s) cnt[s] = 0;
  int kept = 0;
  const long long step = parts * (kBalWarps * R);
  for (long long base = (part * kBalWarps + warp) * R; base < p.rows; base += step) {
    const long long r = base + sub;
    const bool live = r < p.rows && (!p.mask || p.mask[r]);
    float a[V];
    load_row<L, V>(p.alpha + r * p.stride + static_cast<long long>(j) * n, n, lane, p.vec, live, a);
    if (live && lane == 0) ++kept;
    float w[V];
#pragma unroll
    for (int s = 0; s < V; ++s) w[s] = a[s];
    if (p.sigmoid) normalise<L, V>(w);
#pragma unroll
    for (int s = 0; s < V; s += 2) accumulate(acc[s / 2], pack2(w[s], w[s + 1]));
    if (select) {
      uint32_t taken = choose<L, V>(a, n, lane, live, p.top_k);
      if (kRegCounts) {
#pragma unroll
        for (int s = 0; s < V; ++s) cnt[kRegCounts ? s : 0] += (taken >> s) & 1u;
      } else {
        for (; taken; taken &= taken - 1)
          atomicAdd(&sh.count[element_of<L, V>(__ffs(taken) - 1, lane)], 1);
      }
    }
  }
  // the rows of a warp, then the warps in order
  double sum[V];
#pragma unroll
  for (int s = 0; s < V; s += 2) {
    float h0, h1, l0, l1;
    unpack2(acc[s / 2].hi, h0, h1);
    unpack2(acc[s / 2].lo, l0, l1);
    sum[s] = total_of(h0, l0);
    sum[s + 1] = total_of(h1, l1);
  }
#pragma unroll
  for (int s = 0; s < V; ++s) {
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) {
      sum[s] += __shfl_xor_sync(0xffffffffu, sum[s], o);
      if (kRegCounts) cnt[kRegCounts ? s : 0] += __shfl_xor_sync(0xffffffffu, cnt[kRegCounts ? s : 0], o);
    }
  }
  if (kept) atomicAdd(&sh.kept, kept);
  for (int w = 0; w < kBalWarps; ++w) {
    if (warp == w && sub == 0) {
#pragma unroll
      for (int s = 0; s < V; ++s) {
        const int e = element_of<L, V>(s, lane);
        if (e < n) {
          sh.sum[e] += sum[s];
          if (kRegCounts) sh.count[e] += cnt[kRegCounts ? s : 0];
        }
      }
    }
    __syncthreads();
  }
  if (!select)
    for (int i = tid; i < n; i += kBalThreads) sh.count[i] = sh.kept;
}

// One part of the sums of one group (blockIdx.y).
template <int L, int V>
__global__ void __launch_bounds__(kBalThreads, V <= 8 ? 4 : 2)
balance_forward_kernel(BalParams p) {
  __shared__ BalShared sh;
  const int j = blockIdx.y, n = p.n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  group_sums<L, V>(p, j, blockIdx.x, gridDim.x, sh);
  const long long out = (static_cast<long long>(blockIdx.x) * p.groups + j) * n;
  for (int i = threadIdx.x; i < n; i += kBalThreads) {
    p.part_sum[out + i] = sh.sum[i];
    p.part_count[out + i] = sh.count[i];
  }
  if (j == 0 && threadIdx.x == 0) p.part_kept[blockIdx.x] = sh.kept;
}

// Adds `dot` of every thread of the cluster's CTAs, in a fixed order; the sum
// comes back to thread 0 of rank 0.
template <int THREADS>
__device__ __forceinline__ double cluster_sum(double dot) {
  namespace cg = cooperative_groups;
  __shared__ double s_warp[THREADS / 32], s_cta;
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double cta = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) cta += s_warp[w];
    s_cta = cta;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  double all = 0.0;
  if (cluster.block_rank() == 0 && threadIdx.x == 0)
    for (unsigned r = 0; r < cluster.num_blocks(); ++r) all += *cluster.map_shared_rank(&s_cta, r);
  cluster.sync();  // no CTA leaves while rank 0 reads
  return all;
}

// loss / sum of counts/M * mean
__device__ __forceinline__ double loss_factor(float coef, int n, int top_k, int groups) {
  return static_cast<double>(coef) * n / (static_cast<double>(top_k) * groups);
}

// Few rows: the whole forward in one launch of one cluster, which takes the
// groups in turn and meets only for the loss (a launch less: 4 of 13 us of a
// forward and backward over 64 rows).
template <int L, int V>
__global__ void __launch_bounds__(kBalThreads) balance_small_kernel(BalParams p) {
  __shared__ BalShared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double dot = 0.0;
  for (int j = blockIdx.x; j < p.groups; j += gridDim.x) {
    group_sums<L, V>(p, j, 0, 1, sh);
    const double over = sh.kept > 0 ? 1.0 / sh.kept : 0.0;
    for (int i = threadIdx.x; i < p.n; i += kBalThreads) {
      // (without top_k < n the count was written by this thread just now)
      const double mean = sh.sum[i] * over;
      p.counts[j * p.n + i] = sh.count[i];
      p.mean[j * p.n + i] = static_cast<float>(mean);
      dot += sh.count[i] * over * mean;
    }
    if (j == 0 && threadIdx.x == 0) *p.rows_kept = sh.kept;
    __syncthreads();
  }
  const double total = cluster_sum<kBalThreads>(dot);
  if (blockIdx.x == 0 && threadIdx.x == 0)
    *p.loss = static_cast<float>(loss_factor(p.coef, p.n, p.top_k, p.groups) * total);
}

struct BalFinish {
  int parts, width, n, top_k, groups;  // width = groups * n
  int tile;                            // columns side by side, a power of two
  float coef;
  const double* part_sum;
  const int* part_count;
  const int* part_kept;
  int* counts;
  float* mean;
  int* rows_kept;
  float* loss;
};

// The parts added in a fixed order, the means and the loss: one cluster, its CTAs
// taking tiles of columns in turn, a tile's threads splitting the parts.
__global__ void __launch_bounds__(kBalFinishThreads) balance_finish_kernel(BalFinish p) {
  __shared__ double s_sum[kBalFinishThreads];
  __shared__ int s_count[kBalFinishThreads];
  __shared__ int s_kept;
  const int tid = threadIdx.x, col = tid % p.tile, slice = tid / p.tile;
  const int slices = kBalFinishThreads / p.tile;
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
  for (int i0 = blockIdx.x * p.tile; i0 < p.width; i0 += gridDim.x * p.tile) {
    const int i = i0 + col;
    double sum = 0.0;
    int count = 0;
    if (i < p.width) {
#pragma unroll 8
      for (int q = slice; q < p.parts; q += slices) {
        sum += p.part_sum[static_cast<long long>(q) * p.width + i];
        count += p.part_count[static_cast<long long>(q) * p.width + i];
      }
    }
    s_sum[tid] = sum;
    s_count[tid] = count;
    __syncthreads();
    if (slice == 0 && i < p.width) {
      for (int q = 1; q < slices; ++q) {
        sum += s_sum[q * p.tile + col];
        count += s_count[q * p.tile + col];
      }
      const double mean = sum * over;
      p.counts[i] = count;
      p.mean[i] = static_cast<float>(mean);
      dot += count * over * mean;
    }
    __syncthreads();
  }
  const double total = cluster_sum<kBalFinishThreads>(dot);
  if (blockIdx.x == 0 && tid == 0) {
    *p.loss = static_cast<float>(loss_factor(p.coef, p.n, p.top_k, p.groups) * total);
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
    const float total = normalise<L, V>(a);
    float dot = 0.f;
#pragma unroll
    for (int s = 0; s < V; ++s) dot += c[s] * a[s];
    dot = row_sum<L>(dot);
    const bool small = fabsf(total) < 1e-30f;
    const float inv = small ? 0.f : __frcp_rn(total);
    if (r >= p.rows || (!live && p.accumulate)) continue;  // (a row's lanes agree)
    float* d = p.dalpha + r * p.dstride + static_cast<long long>(j) * n;
#pragma unroll
    for (int ch = 0; ch < V / 4; ++ch) {
      const int e = (ch * L + lane) * 4;
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = (c[4 * ch + q] - dot) * inv;
      if (!live || small) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = live && total != 0.f ? __fdiv_rn(c[4 * ch + q] - dot, total) : 0.f;
      }
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
