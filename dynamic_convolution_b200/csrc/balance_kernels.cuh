// Kernels of the router's load-balance loss (include/dynconv_train.h).
//
// A row of n attentions is held by L neighbouring lanes of a warp, V values in
// each lane's registers (n <= L * V), so a warp holds 32 / L rows. More values per
// lane mean fewer steps across lanes, which the top k need in every round. Up to
// V = 8 lane l of a row owns the elements l V .. l V + V - 1, so that the lowest
// index among equals is the lowest lane's; above, 16-byte loads at that distance
// would waste the L1, and it owns (c * L + l) * 4 + q, c = 0.., q = 0..3 (chunks c
// of four).
#pragma once

#include <climits>
#include <cstdint>

#include <cooperative_groups.h>

namespace dct {

constexpr int kBalThreads = 256;
// Threads of a forward CTA that has an SM to itself, so that few parts are left to
// be added; where those do not fill the GPU the CTAs have kBalThreads.
// (32 values a lane with their sums want more than the 128 registers of 512.)
constexpr int forward_threads(int values) { return values <= 8 ? 1024 : values <= 16 ? 512 : 384; }
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

template <int L, int V>
__device__ __forceinline__ int element_of(int slot, int lane) {
  return V <= 8 ? lane * V + slot : ((slot >> 2) * L + lane) * 4 + (slot & 3);
}

// The lane's V elements of a row (0 where the row ends or `live` is false).
template <int L, int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int n, int lane, bool vec,
                                         bool live, float (&a)[V]) {
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = element_of<L, V>(4 * c, lane);
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

struct BalParams {
  int rows, groups, n, top_k, sigmoid, vec;
  float coef;
  long long stride;            // floats between rows of alpha
  const float* alpha;
  const unsigned char* mask;   // or null
  double* part_sum;            // [parts][groups][n]
  int* part_count;             // [parts][groups][n]
  int* part_kept;              // [parts]
  unsigned* ticket;            // zeroed for the finishing kernel
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

constexpr uint32_t kFull = 0xffffffffu;

// The choice of every row whose attentions hold NaN, which come last: k rounds
// over integer keys in the order of the values. Returns the lane's chosen slots.
// Rare, and out of the way of the loop's registers.
template <int L, int V>
__device__ __noinline__ uint32_t choose_with_nan(const float (&a)[V], int n, int lane, int k) {
  uint32_t taken = 0;
  for (int t = 0; t < k; ++t) {
    int best = INT_MIN, at = INT_MAX, slot = 0;
    for (int s = 0; s < V; ++s) {
      const int e = element_of<L, V>(s, lane);
      if (e >= n || ((taken >> s) & 1u)) continue;
      const float v = a[s] + 0.f;  // -0 as +0
      const int b = __float_as_int(v);
      const int key = v != v ? INT_MIN + 1 : (b ^ ((b >> 31) & 0x7fffffff));
      if (key > best || (key == best && e < at)) {
        best = key;
        at = e;
        slot = s;
      }
    }
    int top = best;
    for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    const int first = row_min<L>(best == top ? at : INT_MAX);
    if (at == first && first != INT_MAX) taken |= 1u << slot;
  }
  return taken;
}

// The k largest of each row, k rounds: the largest value left, the lowest index
// of those that hold it; `cnt` counts the lane's chosen slots. Chosen elements
// become NaN, which no maximum takes; the caller has seen to it that the row has
// none. Elements past the row's end become NaN too. `a` is used up.
template <int L, int V>
__device__ __forceinline__ void choose_few(float (&a)[V], int n, int lane, bool live, int k,
                                           int (&cnt)[V]) {
  static_assert(V <= 8, "lane order");
  const float kNone = __int_as_float(0x7fffffff);
  const uint32_t below = L == 1 ? 0u : ((1u << (threadIdx.x & 31)) - 1u) &
                                           ~((1u << ((threadIdx.x & 31) - lane)) - 1u);
  if (n < L * V) {
#pragma unroll
    for (int s = 0; s < V; ++s)
      if (lane * V + s >= n) a[s] = kNone;
  }
  for (int t = 1;; ++t) {
    float best = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
    if (V == 8) best = fmaxf(best, fmaxf(fmaxf(a[4 % V], a[5 % V]), fmaxf(a[6 % V], a[7 % V])));
    const float top = row_max<L>(best);
    bool mine = live && best == top;
    if (L > 1) mine = (__ballot_sync(kFull, best == top) & below) == 0 && mine;  // the lowest lane
    const float gone = mine ? top : kNone;  // (nothing equals NaN)
    bool found = false;
    if (t == k) {
#pragma unroll
      for (int s = 0; s < V; ++s) {
        const bool hit = a[s] == gone && !found;
        if (hit) ++cnt[s];
        found = found || hit;
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < V; ++s) {
      const bool hit = a[s] == gone && !found;
      if (hit) {
        ++cnt[s];
        a[s] = kNone;
      }
      found = found || hit;
    }
  }
}

// The same where a lane holds many values: every lane keeps the maximum of each
// of its chunks, and the best of those with its chunk; a round takes the winner
// from those and renews them for the one chunk it took from. Counts go to shared
// memory. Returns whether the row ran out of numbers (NaN in it are still to be
// chosen).
template <int V>
__device__ __forceinline__ bool choose_many(float (&a)[V], int n, int lane, bool live, int k,
                                            int* count) {
  constexpr int C = V / 4;
  const float kNone = __int_as_float(0x7fffffff);
  float g[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if ((c + 1) * 128 > n) {  // the chunks that reach past the row's end
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((c * 32 + lane) * 4 + q >= n) a[4 * c + q] = kNone;
    }
    g[c] = fmaxf(fmaxf(a[4 * c], a[4 * c + 1]), fmaxf(a[4 * c + 2], a[4 * c + 3]));
  }
  float best = kNone, top = 0.f;
  int chunk = 0;
  const auto renew = [&] {
    best = g[0];
#pragma unroll
    for (int c = 1; c < C; ++c) best = fmaxf(best, g[c]);
#pragma unroll
    for (int c = C - 1; c >= 0; --c)
      if (g[c] == best) chunk = c;
  };
  renew();
  for (int t = 0; t < k; ++t) {
    top = row_max<32>(best);
    const int first = row_min<32>(best == top ? chunk * 32 + lane : INT_MAX);
    const bool mine = live && (first & 31) == lane && first != INT_MAX;
    int q = 0;
    switch (first >> 5) {  // the same chunk for the whole warp
#define DCT_TAKE(c)                                                                           \
  case c:                                                                                     \
    if (c < C && mine) {                                                                      \
      constexpr int b = 4 * (c < C ? c : 0);                                                  \
      q = a[b] == top ? 0 : a[b + 1] == top ? 1 : a[b + 2] == top ? 2 : 3;                    \
      a[b] = q == 0 ? kNone : a[b];                                                           \
      a[b + 1] = q == 1 ? kNone : a[b + 1];                                                   \
      a[b + 2] = q == 2 ? kNone : a[b + 2];                                                   \
      a[b + 3] = q == 3 ? kNone : a[b + 3];                                                   \
      g[c < C ? c : 0] = fmaxf(fmaxf(a[b], a[b + 1]), fmaxf(a[b + 2], a[b + 3]));             \
    }                                                                                         \
    break;
      DCT_TAKE(0) DCT_TAKE(1) DCT_TAKE(2) DCT_TAKE(3)
      DCT_TAKE(4) DCT_TAKE(5) DCT_TAKE(6) DCT_TAKE(7)
#undef DCT_TAKE
      default: break;
    }
    if (mine) {
      atomicAdd(&count[first * 4 + q], 1);
      renew();
    }
  }
  return live && top != top;
}

// The same for most rows at a fraction of the rounds' cost. The k-th largest of the
// 32 lanes' maxima is a lower bound of the k-th largest value, so only values not
// below it can be chosen: k of them or a few more. Those are gathered into `list`
// (their places; the values are read again from the row), and each lane counts how
// many come before its own. Returns false, with nothing counted, for a row with
// more than 32 such values (ties) or with fewer than k lanes that hold a number.
template <int V>
__device__ __forceinline__ bool choose_filtered(const float (&a)[V], const float* row, int n,
                                                int lane, int k, int* count, int* list) {
  const float kNone = __int_as_float(0x7fffffff);
  float best = kNone;
#pragma unroll
  for (int s = 0; s < V; s += 4) {
    const int e = element_of<32, V>(s, lane);
    float m = fmaxf(fmaxf(a[s], a[s + 1]), fmaxf(a[s + 2], a[s + 3]));
    if ((s / 4 + 1) * 128 > n) {  // a chunk that reaches past the row's end
      m = kNone;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (e + q < n) m = fmaxf(m, a[s + q]);
    }
    best = fmaxf(best, m);
  }
  float bound = 0.f;
  for (int t = 0; t < k; ++t) {
    bound = row_max<32>(best);
    if (lane == __ffs(__ballot_sync(kFull, best == bound)) - 1) best = kNone;
  }
  uint32_t bits = 0;
#pragma unroll
  for (int s = 0; s < V; ++s)
    if (a[s] >= bound) bits |= 1u << s;
  if (n < 32 * V) {
#pragma unroll
    for (int s = 0; s < V; s += 4)
      if ((s / 4 + 1) * 128 > n) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (element_of<32, V>(s + q, lane) >= n) bits &= ~(1u << (s + q));
      }
  }
  const int held = __popc(bits), all = __reduce_add_sync(kFull, held);
  if (bound != bound || all > 32) return false;
  if (all == k) {
    for (; bits; bits &= bits - 1)
      atomicAdd(&count[element_of<32, V>(__ffs(bits) - 1, lane)], 1);
    return true;
  }
  int at = held;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int other = __shfl_up_sync(kFull, at, o);
    if (lane >= o) at += other;
  }
  at -= held;
  for (; bits; bits &= bits - 1) list[at++] = element_of<32, V>(__ffs(bits) - 1, lane);
  __syncwarp();
  const int e = lane < all ? list[lane] : INT_MAX;
  const float v = lane < all ? row[e] : kNone;
  int before = 0;
  for (int j = 0; j < all; ++j) {
    const float w = __shfl_sync(kFull, v, j);
    const int f = __shfl_sync(kFull, e, j);
    before += w > v || (w == v && f < e) ? 1 : 0;
  }
  if (lane < all && before < k) atomicAdd(&count[e], 1);
  __syncwarp();  // the list is read
  return true;
}

// The sum of a lane's values.
template <int V>
__device__ __forceinline__ float lane_sum(const float (&a)[V]) {
  unsigned long long t = pack2(a[0], a[1]);
#pragma unroll
  for (int s = 2; s < V; s += 2) t = add2(t, pack2(a[s], a[s + 1]));
  float x, y;
  unpack2(t, x, y);
  return x + y;
}

// p = a / total, and 0 where the total is 0: a product with the reciprocal, corrected
// by its residual (a row of one expert has p = 1 and no gradient left), except where
// the reciprocal would leave fp32's normal numbers.
template <int V>
__device__ __forceinline__ void normalise(float (&a)[V], float total) {
  if (fabsf(total) >= 1e-30f && fabsf(total) <= 1e30f) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(total));
#pragma unroll
    for (int s = 0; s < V; ++s) {
      const float q = a[s] * inv;
      a[s] = fmaf(fmaf(-q, total, a[s]), inv, q);
    }
  } else {
#pragma unroll
    for (int s = 0; s < V; ++s) a[s] = total != 0.f ? __fdiv_rn(a[s], total) : 0.f;
  }
}

struct BalShared {
  double sum[kBalMaxN];
  int count[kBalMaxN];
  double part[8 * 256];   // eight warps' sums of up to 256 columns
  int list[16][32];       // each warp's candidates (rows of more than 256)
  int kept;
};

// Dynamic shared memory of the forward where a lane holds many values: two rows, or
// in the end the fp64 sums, of each warp.
constexpr int forward_smem(int values, int threads) {
  return values <= 8 ? 0 : threads / 32 * 2 * values * 128;
}

// The column sums and counts of one group over batches part, part + parts, ... of
// rows, into `sh` (which no thread may still be reading).
template <int L, int V, int THREADS>
__device__ __forceinline__ void group_sums(const BalParams& p, int j, long long part,
                                           long long parts, BalShared& sh, float4* stage) {
  constexpr int R = 32 / L, W = THREADS / 32;   // rows per warp, warps
  constexpr bool kFew = V <= 8;                 // counts in registers; else in shared memory
  const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31, lane = wl % L, sub = wl / L;
  const int n = p.n;
  const bool select = p.top_k < n;
  for (int i = tid; i < n; i += THREADS) {
    sh.count[i] = 0;
    sh.sum[i] = 0.0;
  }
  if (tid == 0) sh.kept = 0;
  __syncthreads();
  Sum2 acc[V / 2];
  int cnt[V];  // (used where kFew)
#pragma unroll
  for (int s = 0; s < V / 2; ++s) acc[s].hi = acc[s].lo = 0ull;
#pragma unroll
  for (int s = 0; s < V; ++s) cnt[s] = 0;
  int kept = 0;
  // The next row is on its way while this one is worked on: in registers where a
  // lane holds few values, through shared memory where it holds many (each lane
  // copies and reads its own 16-byte pieces; without alignment for those, not ahead).
  const long long step = parts * (W * R);
  const bool staged = !kFew && p.vec;
  const auto alive = [&](long long r) { return r < p.rows && (!p.mask || p.mask[r]); };
  const auto row_at = [&](long long r) { return p.alpha + r * p.stride + static_cast<long long>(j) * n; };
  const auto stage_of = [&](int k) { return stage + ((k * W + warp) * (V / 4)) * 32 + wl; };
  const auto copy = [&](long long r, bool live, int k) {
    if (live) {
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(stage_of(k)));
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        const int e = element_of<L, V>(4 * c, lane);
        if (e < n)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + c * 512),
                       "l"(row_at(r) + e) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float a[V], ahead[kFew ? V : 1];
  long long base = (part * W + warp) * R;
  bool live = base < p.rows && alive(base + sub), next_live = false;
  if constexpr (kFew) {
    if (base < p.rows) load_row<L, V>(row_at(base + sub), n, lane, p.vec, live, a);
  } else if (staged && base < p.rows) {
    copy(base, live, 0);
  }
  for (int turn = 0; base < p.rows; base += step, ++turn) {
    const long long r = base + sub, next = r + step;
    if (turn > 0) {
      live = next_live;
      if constexpr (kFew) {
#pragma unroll
        for (int s = 0; s < V; ++s) a[s] = ahead[s];
      }
    }
    next_live = alive(next);
    if constexpr (kFew) {
      load_row<L, V>(row_at(next), n, lane, p.vec, next_live, ahead);
    } else if (staged) {
      copy(next, next_live, (turn + 1) & 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (!live) continue;  // (a warp holds one row)
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        const bool in = element_of<L, V>(4 * c, lane) < n;
        const float4 f = in ? stage_of(turn & 1)[c * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
        a[4 * c] = f.x; a[4 * c + 1] = f.y; a[4 * c + 2] = f.z; a[4 * c + 3] = f.w;
      }
    } else {
      if (!live) continue;
      load_row<L, V>(row_at(r), n, lane, false, true, a);
    }
    if (live && lane == 0) ++kept;
    const float mine = p.sigmoid || (kFew && select) ? lane_sum<V>(a) : 0.f;
    {
      float w[V];
#pragma unroll
      for (int s = 0; s < V; ++s) w[s] = a[s];
      if (p.sigmoid) normalise<V>(w, row_sum<L>(mine));
#pragma unroll
      for (int s = 0; s < V; s += 2) accumulate(acc[s / 2], pack2(w[s], w[s + 1]));
    }
    if (!select) continue;
    if constexpr (kFew) {
      // NaN (or opposite infinities) in the lane's values show in their sum
      if (__any_sync(kFull, mine != mine)) {
        float copy[V];  // (only this branch puts the row into local memory)
#pragma unroll
        for (int s = 0; s < V; ++s) copy[s] = a[s];
        const uint32_t taken = choose_with_nan<L, V>(copy, n, lane, p.top_k);
#pragma unroll
        for (int s = 0; s < V; ++s) cnt[s] += live ? (taken >> s) & 1u : 0;
      } else {
        choose_few<L, V>(a, n, lane, live, p.top_k, cnt);
      }
    } else {
      const float* row = row_at(r);
      if (choose_filtered<V>(a, row, n, lane, p.top_k, sh.count, sh.list[warp])) continue;
      if (__any_sync(kFull, choose_many<V>(a, n, lane, live, p.top_k, sh.count))) {
        // the numbers are counted; the NaN that follow them, from the row as it was
        float copy[V];
        load_row<L, V>(row, n, lane, p.vec, live, copy);
        const uint32_t taken = choose_with_nan<L, V>(copy, n, lane, p.top_k);
#pragma unroll
        for (int s = 0; s < V; ++s)
          if (copy[s] != copy[s] && ((taken >> s) & 1u))
            atomicAdd(&sh.count[element_of<L, V>(s, lane)], 1);
      }
    }
  }
  if (!kFew) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (kept) atomicAdd(&sh.kept, kept);
  // a warp's rows by shuffles, then the warps in order
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
      sum[s] += __shfl_xor_sync(kFull, sum[s], o);
      if (kFew) cnt[s] += __shfl_xor_sync(kFull, cnt[s], o);
    }
  }
  if constexpr (kFew) {
    if (select && sub == 0) {
#pragma unroll
      for (int s = 0; s < V; ++s)
        if (lane * V + s < n && cnt[s]) atomicAdd(&sh.count[lane * V + s], cnt[s]);
    }
    for (int w0 = 0; w0 < W; w0 += 8) {
      if ((warp & ~7) == w0 && sub == 0) {
#pragma unroll
        for (int s = 0; s < V; ++s)
          if (lane * V + s < n) sh.part[(warp & 7) * n + lane * V + s] = sum[s];
      }
      __syncthreads();
      for (int i = tid; i < n; i += THREADS) {
        double t = sh.sum[i];
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sh.part[w * n + i];
        sh.sum[i] = t;
      }
      if (w0 + 8 < W) __syncthreads();
    }
  } else {
    double* own = reinterpret_cast<double*>(stage);  // [W][32 V], where the rows were
    __syncthreads();
#pragma unroll
    for (int s = 0; s < V; ++s) own[warp * 32 * V + element_of<L, V>(s, lane)] = sum[s];
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
      double t = 0.0;
#pragma unroll
      for (int w = 0; w < W; ++w) t += own[w * 32 * V + i];
      sh.sum[i] = t;
    }
  }
  if (!select)
    for (int i = tid; i < n; i += THREADS) sh.count[i] = sh.kept;
  __syncthreads();
}

// One part of the sums of one group (blockIdx.y). Reads the attentions once; bound by
// instruction issue, most of it the choice of the top k: 1 M rows of 16 sigmoid
// attentions, top 2, a fifth masked: 33 us (64 MB; 19 us without the choice); 30 K rows
// of 1000, top 8: 50 us (96 MB; 29 without it; 67 before the lanes' maxima filtered the
// candidates and while 512 threads spilled registers).
template <int L, int V, int T>
__global__ void __launch_bounds__(T)
balance_forward_kernel(BalParams p) {
  extern __shared__ float4 stage[];
  __shared__ BalShared sh;
  const int j = blockIdx.y, n = p.n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  group_sums<L, V, T>(p, j, blockIdx.x, gridDim.x, sh, stage);
  const long long out = (static_cast<long long>(blockIdx.x) * p.groups + j) * n;
  for (int i = threadIdx.x; i < n; i += T) {
    p.part_sum[out + i] = sh.sum[i];
    p.part_count[out + i] = sh.count[i];
  }
  if (j == 0 && threadIdx.x == 0) {
    p.part_kept[blockIdx.x] = sh.kept;
    if (blockIdx.x == 0) *p.ticket = 0;
  }
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
// groups in turn and meets only for the loss (64 rows of 4 experts, forward and
// backward: 10.1 us for 12.8 with a finishing launch; bound by the calls).
template <int L, int V, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_small_kernel(BalParams p) {
  __shared__ BalShared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double dot = 0.0;
  for (int j = blockIdx.x; j < p.groups; j += gridDim.x) {
    group_sums<L, V, THREADS>(p, j, 0, 1, sh, nullptr);
    const double over = sh.kept > 0 ? 1.0 / sh.kept : 0.0;
    for (int i = threadIdx.x; i < p.n; i += THREADS) {
      const double mean = sh.sum[i] * over;
      p.counts[j * p.n + i] = sh.count[i];
      p.mean[j * p.n + i] = static_cast<float>(mean);
      dot += sh.count[i] * over * mean;
    }
    if (j == 0 && threadIdx.x == 0) *p.rows_kept = sh.kept;
    __syncthreads();
  }
  const double total = cluster_sum<THREADS>(dot);
  if (blockIdx.x == 0 && threadIdx.x == 0)
    *p.loss = static_cast<float>(loss_factor(p.coef, p.n, p.top_k, p.groups) * total);
}

struct BalFinish {
  int parts, width, n, top_k, groups;  // width = groups * n
  float coef;
  const double* part_sum;
  const int* part_count;
  const int* part_kept;
  double* part_dot;                    // [CTAs]
  unsigned* ticket;                    // zeroed by the forward kernel
  int* counts;
  float* mean;
  int* rows_kept;
  float* loss;
};

constexpr int kBalTile = 16;           // columns of a finishing CTA

// The parts added in a fixed order and the means; the CTA that is done last adds
// what each found of the loss, in the order of the CTAs.
__global__ void __launch_bounds__(kBalFinishThreads) balance_finish_kernel(BalFinish p) {
  constexpr int S = kBalFinishThreads / kBalTile;
  __shared__ double s_sum[kBalFinishThreads];
  __shared__ int s_count[kBalFinishThreads];
  __shared__ int s_kept;
  __shared__ bool s_last;
  const int tid = threadIdx.x, col = tid % kBalTile, slice = tid / kBalTile;
  const int i = blockIdx.x * kBalTile + col;
  if (tid == 0) s_kept = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int k = 0;
  for (int q = tid; q < p.parts; q += kBalFinishThreads) k += p.part_kept[q];
  if (k) atomicAdd(&s_kept, k);
  double sum = 0.0;
  int count = 0;
  if (i < p.width) {
    constexpr int B = 8;  // loads in flight
    for (int q0 = slice; q0 < p.parts; q0 += B * S) {
      double x[B];
      int y[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int q = q0 + b * S;
        const bool in = q < p.parts;
        x[b] = in ? p.part_sum[static_cast<long long>(q) * p.width + i] : 0.0;
        y[b] = in ? p.part_count[static_cast<long long>(q) * p.width + i] : 0;
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        sum += x[b];
        count += y[b];
      }
    }
  }
  sum += __shfl_xor_sync(kFull, sum, kBalTile);  // the warp's two rows of the tile
  count += __shfl_xor_sync(kFull, count, kBalTile);
  if ((tid & kBalTile) == 0) {
    s_sum[slice / 2 * kBalTile + col] = sum;
    s_count[slice / 2 * kBalTile + col] = count;
  }
  __syncthreads();
  if (tid < 32) {
    double dot = 0.0;
    if (tid < kBalTile && i < p.width) {
#pragma unroll
      for (int q = 1; q < S / 2; ++q) {
        sum += s_sum[q * kBalTile + col];
        count += s_count[q * kBalTile + col];
      }
      const double over = s_kept > 0 ? 1.0 / s_kept : 0.0;
      const double mean = sum * over;
      p.counts[i] = count;
      p.mean[i] = static_cast<float>(mean);
      dot = count * over * mean;
    }
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if (tid == 0) {
      p.part_dot[blockIdx.x] = dot;
      __threadfence();
      s_last = atomicAdd(p.ticket, 1u) + 1 == gridDim.x;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double total = 0.0;
  for (int q = tid; q < static_cast<int>(gridDim.x); q += kBalFinishThreads)
    total += __ldcg(p.part_dot + q);
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  __syncthreads();
  if ((tid & 31) == 0) s_sum[tid >> 5] = total;
  __syncthreads();
  if (tid == 0) {
    total = 0.0;
    for (int w = 0; w < kBalFinishThreads / 32; ++w) total += s_sum[w];
    *p.loss = static_cast<float>(loss_factor(p.coef, p.n, p.top_k, p.groups) * total);
    *p.rows_kept = s_kept;
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
// columns and walks down the rows. Bound by memory: 30 K rows of 1000, a fifth masked,
// added to dalpha, 30 us (6.4 TB/s). Rows off the 16-byte grid take four single words in
// place of each 16 bytes: all 30 K rows 123 us at 999 experts, 47 at 1000.
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
// 1 M rows of 16, added to dalpha: 33 us (154 MB of kept rows, 4.7 TB/s; 36 with
// dalpha read where it is added to). Bound by the latency of its loads: with 56
// registers half of the warps are resident, each with one group of rows under way
// (waiting for loads takes 10 of the 17 cycles between a warp's instructions). Rows off
// the 16-byte grid: 53 us at 15 experts, 72 at 17, by accesses of single words.
// The quotient by the row's sum is a product with the one-instruction reciprocal
// (2^-23 relative, two half steps more than a division's; the forward corrects its own
// because a single expert's probability has to be exactly 1).
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
  const long long step = static_cast<long long>(gridDim.x) * ((kBalThreads / 32) * R);
  for (long long base = (static_cast<long long>(blockIdx.x) * (kBalThreads / 32) + warp) * R;
       base < p.rows; base += step) {
    const long long r = base + sub;
    const bool live = r < p.rows && (!p.mask || p.mask[r]);
    float* d = p.dalpha + r * p.dstride + static_cast<long long>(j) * n;
    float a[V], old[V];  // both on their way before either is used
    load_row<L, V>(p.alpha + r * p.stride + static_cast<long long>(j) * n, n, lane, p.vec, live, a);
    load_row<L, V>(d, n, lane, p.vec, live && p.accumulate, old);
    const float total = row_sum<L>(lane_sum<V>(a));
    normalise<V>(a, total);
    float dot = 0.f;
#pragma unroll
    for (int s = 0; s < V; ++s) dot += c[s] * a[s];
    dot = row_sum<L>(dot);
    const bool usual = fabsf(total) >= 1e-30f && fabsf(total) <= 1e30f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(total));
    if (r >= p.rows || (!live && p.accumulate)) continue;  // (a row's lanes agree)
#pragma unroll
    for (int ch = 0; ch < V / 4; ++ch) {
      const int e = element_of<L, V>(4 * ch, lane);
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = (c[4 * ch + q] - dot) * inv;
      if (!live || !usual) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = live && total != 0.f ? __fdiv_rn(c[4 * ch + q] - dot, total) : 0.f;
      }
      if (p.vec) {
        if (e < n) {
          const float* b = old + 4 * ch;
          *reinterpret_cast<float4*>(d + e) =
              make_float4(b[0] + o[0], b[1] + o[1], b[2] + o[2], b[3] + o[3]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < n) d[e + q] = old[4 * ch + q] + o[q];
      }
    }
  }
}

}  // namespace dct
