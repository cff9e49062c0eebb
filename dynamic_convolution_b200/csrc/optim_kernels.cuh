// Kernels over lists of tensors (include/dynconv_train.h): the norm of all
// gradients and the AdamW step. The list travels as the kernel's parameter, so
// a call copies nothing to the device and a captured launch keeps its own list.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>

namespace dct {

constexpr int kOptThreads = 256;
constexpr int kBlock = 256;                       // elements per scale of an 8-bit state
constexpr int kChunk = kOptThreads / 32 * kBlock;  // 2048: a block for every warp

template <typename E>
__device__ __forceinline__ int find_tensor(const E* e, int count, long long unit) {
  int lo = 0, hi = count - 1;  // the last entry whose first unit is not after `unit`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].first <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------ the norm

constexpr int kNormPiece = 4096;  // elements that a CTA's threads take at a time, 16 each
struct NormEntry {
  const void* grad;
  long long numel;
  long long first;  // units of the list before this tensor
  int bf16, vec;    // vec: 16-byte loads
};
constexpr int kNormCap = 768;
template <int CAP>
struct NormTable {
  NormEntry e[CAP];
  long long units;   // of `pieces` pieces
  int count, pieces;
  double* part;
};
static_assert(sizeof(NormTable<kNormCap>) <= 32764, "kernel parameters");

constexpr int kNormParts = 1184;  // CTAs of a launch at most: eight per SM of 148

// Squares in fp64. The conversion instruction to fp64 issues at a fraction of the
// FMA rate (it bound the kernel: 85 us for 113 M bf16 gradients), so the bits of a
// value x are moved into place instead: exponent and mantissa three places to the
// right, and the exponent's bias set by an OR, which gives |x| 2^-128 exactly for
// normal numbers. The sum is kept in units of 2^-256. Zeros and subnormals come
// out as up to 2^-126 in place of themselves, below 2^-52 of the sum while the
// largest of the values added together is at least 2^-100; otherwise, and with an
// infinity or NaN among them, they are converted by the instruction.
constexpr uint32_t kWideBias = 0x30000000u;
__device__ __forceinline__ bool in_range(uint32_t top) {  // 2^-100 <= top < infinity
  return top - 0x0d800000u < 0x7f800000u - 0x0d800000u;
}
__device__ __forceinline__ void add_square(uint32_t hi, uint32_t lo, double& s) {
  const double d = __hiloint2double(static_cast<int>(hi), static_cast<int>(lo));
  s = fma(d, d, s);
}
__device__ __forceinline__ void add_square(float x, double& s) {
  const double d = static_cast<double>(x) * 0x1p-128;
  s = fma(d, d, s);
}
// Four fp32 values by their bits.
__device__ __forceinline__ void add_squares(const uint4& a, double& s0, double& s1) {
  constexpr uint32_t kMag = 0x7fffffffu;
  if (in_range(max(max(a.x & kMag, a.y & kMag), max(a.z & kMag, a.w & kMag)))) {
    add_square(((a.x >> 3) & 0x0fffffffu) | kWideBias, a.x << 29, s0);
    add_square(((a.y >> 3) & 0x0fffffffu) | kWideBias, a.y << 29, s1);
    add_square(((a.z >> 3) & 0x0fffffffu) | kWideBias, a.z << 29, s0);
    add_square(((a.w >> 3) & 0x0fffffffu) | kWideBias, a.w << 29, s1);
  } else {
    add_square(__uint_as_float(a.x), s0);
    add_square(__uint_as_float(a.y), s0);
    add_square(__uint_as_float(a.z), s0);
    add_square(__uint_as_float(a.w), s0);
  }
}
// Eight bf16 values, two to a word (their low fp64 words are zero).
__device__ __forceinline__ void add_squares_bf16(const uint4& a, double& s0, double& s1) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  const uint32_t two = __vmaxu2(__vmaxu2(a.x & kMag, a.y & kMag), __vmaxu2(a.z & kMag, a.w & kMag));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  if (in_range(max(two << 16, two & 0xffff0000u))) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      add_square(((w[q] << 13) & 0x0fffe000u) | kWideBias, 0u, s0);
      add_square(((w[q] >> 3) & 0x0fffe000u) | kWideBias, 0u, s1);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      add_square(__uint_as_float(w[q] << 16), s0);
      add_square(__uint_as_float(w[q] & 0xffff0000u), s0);
    }
  }
}

// One pass over the gradients: bound by memory with fp32 (151 M of them: 92 us, 6.57
// TB/s), by instruction issue with bf16, which brings twice the values per byte (113 M
// in 48 tensors: 50 us, 4.6 TB/s, 70% of the issue slots). The CTAs go through the
// list side by side (a contiguous run for each of them was slower: 95 us and 78); a
// tensor's place is looked up when a unit leaves the last one.
template <int CAP>
__global__ void __launch_bounds__(kOptThreads, 8)
grad_norm_kernel(const __grid_constant__ NormTable<CAP> t) {
  __shared__ double s_sum[kOptThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s0 = 0.0, s1 = 0.0;
  const void* grad = nullptr;
  long long first = 0, stop = 0, numel = 0;
  int bf16 = 0, vec = 0, k = 0;
  for (long long u = blockIdx.x; u < t.units; u += gridDim.x) {
    if (u >= stop) {  // most often in the next tensor, or the one after it
      const int near = k + 1 < t.count ? k + 1 : k;
      if (stop > 0 && (near + 1 >= t.count || u < t.e[near + 1].first)) k = near;
      else if (stop > 0 && (near + 2 >= t.count || u < t.e[near + 2].first)) k = near + 1;
      else k = find_tensor(t.e, t.count, u);
      grad = t.e[k].grad;
      numel = t.e[k].numel;
      first = t.e[k].first;
      bf16 = t.e[k].bf16;
      vec = t.e[k].vec;
      stop = k + 1 < t.count ? t.e[k + 1].first : t.units;
    }
    long long i = (u - first) * t.pieces * kNormPiece;
    const long long end = min(i + static_cast<long long>(t.pieces) * kNormPiece, numel);
    if (vec) {
      if (bf16) {
        for (; i + kNormPiece <= end; i += kNormPiece) {
          const uint4* g = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(grad) + i) + threadIdx.x;
          const uint4 a = g[0], b = g[kOptThreads];
          add_squares_bf16(a, s0, s1);
          add_squares_bf16(b, s0, s1);
        }
      } else {
        for (; i + kNormPiece <= end; i += kNormPiece) {
          const uint4* g = reinterpret_cast<const uint4*>(static_cast<const float*>(grad) + i) +
                           threadIdx.x;
          const uint4 a = g[0], b = g[kOptThreads], x = g[2 * kOptThreads], y = g[3 * kOptThreads];
          add_squares(a, s0, s1);
          add_squares(b, s0, s1);
          add_squares(x, s0, s1);
          add_squares(y, s0, s1);
        }
      }
    }
    // the tensor's end, or a start off the 16-byte grid
    for (i += threadIdx.x; i < end; i += kOptThreads)
      add_square(bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(grad)[i])
                      : static_cast<const float*>(grad)[i], s0);
  }
  double sum = s0 + s1;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < kOptThreads / 32; ++w) total += s_sum[w];
    t.part[blockIdx.x] = total;
  }
}

// One CTA: the parts (in units of 2^-256) in a fixed order, the factor, the step's
// number.
__global__ void __launch_bounds__(kOptThreads)
grad_norm_finish_kernel(const double* part, int parts, double max_norm, float* stats,
                        long long* step) {
  __shared__ double s_sum[kOptThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kOptThreads) sum += part[i];
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < kOptThreads / 32; ++w) total += s_sum[w];
    const double norm = sqrt(total) * 0x1p128;
    const float shown = static_cast<float>(norm);
    const bool fine = isfinite(shown);
    stats[0] = shown;
    stats[1] = fine ? static_cast<float>(fmin(1.0, max_norm / (norm + 1e-6)))
                    : __int_as_float(0x7fc00000);
    if (step && fine) *step += 1;
  }
}

// ------------------------------------------------------------------- AdamW

enum : int { kParamF32 = 0, kParamBf16 = 1, kParamMaster = 2 };

struct AdamEntry {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long numel;
  long long first;   // chunks of the list before this tensor
  float size, keep;  // lr lr_scale / (1 - beta1^t) and 1 - lr lr_scale weight_decay, or, with a
                     // rate or step on the device, lr_scale and weight_decay
  int kind;          // param kind | grad bf16 << 2 | 8-bit state << 3 | vec << 4
  int place;         // in the caller's list
};

struct AdamShared {
  double lr, beta1_d, beta2_d;
  long long step, chunks;
  float beta1, omb1, beta2, omb2, eps, root2;  // root2 = 1 / sqrt(1 - beta2^t)
  unsigned int seed;
  int count;
  int dynamic;                 // lr_dev or step_dev is given
  const float* grad_scale;
  const float* lr_dev;
  const long long* step_dev;
};

template <int CAP>
struct AdamTable {
  AdamShared h;
  AdamEntry e[CAP];
};

// Multiply-xorshift mixing of a 32-bit word; the multipliers are the fractional
// bits of the golden ratio and of the square root of two, made odd.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ (x >> 16);
}

// One-instruction reciprocal and square root (relative error at most 2^-23 each;
// they enter the update's bound of 12 half steps). The denominator is at least
// eps, a normal number, so flushing subnormals cannot divide by zero.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations in one instruction, each rounded like the single one: the
// 8-bit kernel is bound by its instruction issue.
struct Pair {
  unsigned long long bits;
};
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.bits) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(Pair a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.bits));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
  return r;
}
// Sums of products that were rounded before: two single additions, because the
// assembler contracts a packed product and a packed sum into one packed
// multiply-add in spite of their .rn (seen on 26% of random operands).
__device__ __forceinline__ Pair add_apart(Pair a, Pair b) {
  float a0, a1, b0, b1;
  unpair(a, a0, a1);
  unpair(b, b0, b1);
  return pair_of(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}
// Two square roots by Newton's method. With y = (1 + e) / sqrt(x), |e| <= 2^-22.9 (the
// instruction's documented bound), r = x y is the root times 1 + d, |d| <= 2^-22.3 with
// the product's rounding; x - r^2, one multiply-add, is -x (2 d + d^2) but for its own
// rounding of 2^-24; so r + (x - r^2) y / 2 is off the root by at most
// |d| (|d| / 2 + |e| + 2^-24) < 2^-44 of it before it is rounded, 2^-20 of a unit in the
// last place. That rounds to the correctly rounded root unless the root lies as close as
// that to the border between two numbers, which about forty of the 2^24 mantissas (of
// both exponent parities) have it do; the tests find the right root at those too, over
// all exponents. For x from 2^-100 (from there on down the residual's last bits go below
// fp32's least number) to the largest finite number.
__device__ __forceinline__ Pair sqrt2(float lo, float hi) {
  const Pair x = pair_of(lo, hi), y = pair_of(rsqrt_approx(lo), rsqrt_approx(hi));
  const Pair r = x * y;
  const Pair rest = fma2(r * pair_of(-1.f, -1.f), r, x);
  return fma2(rest, y * pair_of(0.5f, 0.5f), r);
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// |y| <= 448 (1 + 2^-22) to the e4m3 grid, as fp32: the 20 mantissa bits that
// e4m3 does not hold get the dither (16 bits, moved up by four) added and are cut
// off; a sign-magnitude word grows in magnitude whatever its sign, and the four
// low bits keep 448 (1 + 2^-22) from reaching 480. Below 2^-6, where e4m3 has the
// fixed spacing 2^-9, the magnitude is first moved to [2^-6, 2^-5), whose spacing
// is the same, and then back. LOW = false: no value of the block is below 2^-6,
// the common case, which saves a tenth of the kernel's instructions.
template <bool LOW>
__device__ __forceinline__ float dither_e4m3(float y, uint32_t u) {
  const bool low = LOW && fabsf(y) < 0.015625f;
  const float base = __uint_as_float((__float_as_uint(y) & 0x80000000u) | 0x3c800000u);
  if (low) y = __fadd_rn(y, base);
  y = __uint_as_float((__float_as_uint(y) + (u << 4)) & 0xfff00000u);
  if (low) y = __fadd_rn(y, -base);
  return y;
}

// Four consecutive elements from element i of a tensor of numel, as words; FAST:
// they are inside and the address is a multiple of four elements.
template <bool FAST>
__device__ __forceinline__ void load4(const float* p, long long i, long long numel,
                                      uint32_t (&x)[4]) {
  if (FAST) {
    const uint4 f = *reinterpret_cast<const uint4*>(p + i);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i + q < numel ? __float_as_uint(p[i + q]) : 0u;
  }
}
template <bool FAST>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, long long i, long long numel,
                                      uint32_t (&x)[2]) {
  if (FAST) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + i);
    x[0] = u.x; x[1] = u.y;
  } else {
    const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
    x[0] = x[1] = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) x[q >> 1] |= static_cast<uint32_t>(s[i + q]) << (16 * (q & 1));
  }
}
__device__ __forceinline__ float value(const uint32_t (&x)[4], int q) {
  return __uint_as_float(x[q]);
}
__device__ __forceinline__ float value(const uint32_t (&x)[2], int q) {
  return __uint_as_float(q & 1 ? x[q >> 1] & 0xffff0000u : x[q >> 1] << 16);
}
template <bool FAST>
__device__ __forceinline__ void store4(float* p, long long i, long long numel,
                                       const float (&x)[4]) {
  if (FAST) {
    *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) p[i + q] = x[q];
  }
}
// Four bf16 values, two to a word.
template <bool FAST>
__device__ __forceinline__ void store4_bf16(__nv_bfloat16* p, long long i, long long numel,
                                            const uint2& u) {
  if (FAST) {
    *reinterpret_cast<uint2*>(p + i) = u;
  } else {
    unsigned short* s = reinterpret_cast<unsigned short*>(p);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) s[i + q] = static_cast<unsigned short>(w[q >> 1] >> (16 * (q & 1)));
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <bool FAST>
__device__ __forceinline__ void load4(const uint8_t* p, long long i, long long numel,
                                      uint32_t (&x)[1]) {
  if (FAST) {
    x[0] = *reinterpret_cast<const uint32_t*>(p + i);
  } else {
    x[0] = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) x[0] |= static_cast<uint32_t>(p[i + q]) << (8 * q);
  }
}
__device__ __forceinline__ void widen4(uint32_t w, float (&x)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * h)) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(two));
    x[2 * h] = f.x;
    x[2 * h + 1] = f.y;
  }
}
template <bool FAST>
__device__ __forceinline__ void store4_codes(uint8_t* p, long long i, long long numel,
                                             const float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t w = lo | (hi << 16);
  if (FAST) {
    *reinterpret_cast<uint32_t*>(p + i) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) p[i + q] = static_cast<uint8_t>(w >> (8 * q));
  }
}

// The block's factor and its inverse from its largest magnitude (a non-finite
// one passes through both: the block is spoilt, not hidden).
__device__ __forceinline__ void block_scale(float top, float& scale, float& inv) {
  const bool none = top < 7.888609052210118e-31f;  // 2^-100
  scale = none ? 0.f : __fmul_rn(top, 1.f / 448.f);
  inv = none ? 0.f : __fmul_rn(__frcp_rn(top), 448.f);
}

struct Hyper {
  float beta1, omb1, beta2, omb2, eps, size, root2, keep, scale;
  uint32_t key;
};

template <int PARAM, bool GRAD16, bool STATE8>
struct AdamTypes {
  using Grad = typename std::conditional<GRAD16, __nv_bfloat16, float>::type;
  using Param = typename std::conditional<PARAM == kParamBf16, __nv_bfloat16, float>::type;
  using State = typename std::conditional<STATE8, uint8_t, float>::type;
  // What one lane holds of a block before it is computed: 2 x 4 elements.
  struct Raw {
    uint32_t g[2][GRAD16 ? 2 : 4], p[2][PARAM == kParamBf16 ? 2 : 4];
    uint32_t m[2][STATE8 ? 1 : 4], v[2][STATE8 ? 1 : 4];
    float ms, vs;
  };
};

// One block of 256 elements of one tensor by one warp: lane l owns the elements
// 4 l + {0..3} of both halves.
template <int PARAM, bool GRAD16, bool STATE8, bool FAST>
__device__ __forceinline__ void adam_load(
    const AdamEntry& e, long long block, typename AdamTypes<PARAM, GRAD16, STATE8>::Raw& r) {
  using T = AdamTypes<PARAM, GRAD16, STATE8>;
  const typename T::Param* param = static_cast<const typename T::Param*>(
      PARAM == kParamMaster ? static_cast<const void*>(e.master) : e.param);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = block * kBlock + 128 * j + (threadIdx.x & 31) * 4;
    load4<FAST>(static_cast<const typename T::Grad*>(e.grad), i, e.numel, r.g[j]);
    load4<FAST>(param, i, e.numel, r.p[j]);
    load4<FAST>(static_cast<const typename T::State*>(e.m), i, e.numel, r.m[j]);
    load4<FAST>(static_cast<const typename T::State*>(e.v), i, e.numel, r.v[j]);
  }
  if (STATE8) {
    r.ms = e.m_scale[block];
    r.vs = e.v_scale[block];
  }
}

// With 8-bit states m and v are advanced with separately rounded products and sums
// and rooted correctly, so that the codes follow from the formula's fp32 arithmetic
// and not from how it is contracted: next to a border between codes a difference in
// the last bit is a difference of a whole code, and that feeds the next step.
template <int PARAM, bool GRAD16, bool STATE8, bool FAST>
__device__ __forceinline__ void adam_block(
    const AdamEntry& e, const Hyper& h, long long block,
    const typename AdamTypes<PARAM, GRAD16, STATE8>::Raw& r) {
  const int lane = threadIdx.x & 31;
  const long long numel = e.numel, first = block * kBlock + lane * 4;
  constexpr int J = 2;
  float p[J][4], m[J][4], v[J][4];
  const Pair beta1 = pair_of(h.beta1, h.beta1), omb1 = pair_of(h.omb1, h.omb1);
  const Pair beta2 = pair_of(h.beta2, h.beta2), omb2 = pair_of(h.omb2, h.omb2);
  const Pair scale = pair_of(h.scale, h.scale);
  float mtop = 0.f, vtop = 0.f;            // the block's largest |m| and v,
  float mlow = INFINITY, vlow = INFINITY;  // and its smallest
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if constexpr (STATE8) {
      widen4(r.m[j][0], m[j]);
      widen4(r.v[j][0], v[j]);
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const Pair g = pair_of(value(r.g[j], q), value(r.g[j], q + 1)) * scale;
      Pair m0, v0;
      if constexpr (STATE8) {
        m0 = pair_of(m[j][q], m[j][q + 1]) * pair_of(r.ms, r.ms);
        v0 = pair_of(v[j][q], v[j][q + 1]) * pair_of(r.vs, r.vs);
        v0 = v0 * v0;
      } else {
        m0 = pair_of(value(r.m[j], q), value(r.m[j], q + 1));
        v0 = pair_of(value(r.v[j], q), value(r.v[j], q + 1));
      }
      if (STATE8) {
        m0 = add_apart(m0 * beta1, g * omb1);
        v0 = add_apart(v0 * beta2, (g * g) * omb2);
      } else {
        m0 = fma2(m0, beta1, g * omb1);
        v0 = fma2(v0, beta2, (g * g) * omb2);
      }
      unpair(m0, m[j][q], m[j][q + 1]);
      unpair(v0, v[j][q], v[j][q + 1]);
      if (STATE8) {
        mtop = max3_nan(mtop, fabsf(m[j][q]), fabsf(m[j][q + 1]));
        vtop = max3_nan(vtop, v[j][q], v[j][q + 1]);
        mlow = min3(mlow, fabsf(m[j][q]), fabsf(m[j][q + 1]));
        vlow = min3(vlow, v[j][q], v[j][q + 1]);
      }
    }
  }
  // 8-bit codes are taken from roots rounded correctly; 32-bit states need the root
  // for the update alone.
  float root[J][4];
  if constexpr (STATE8) {
    mtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
    vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
    const bool usual = vlow >= 7.888609052210118e-31f && vtop < INFINITY;  // 2^-100
    if (__all_sync(0xffffffffu, usual)) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 4; q += 2)
          unpair(sqrt2(v[j][q], v[j][q + 1]), root[j][q], root[j][q + 1]);
      unpair(sqrt2(vtop, vlow), vtop, vlow);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) root[j][q] = __fsqrt_rn(v[j][q]);
      vtop = __fsqrt_rn(vtop);
      vlow = __fsqrt_rn(vlow);
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) root[j][q] = sqrt_approx(v[j][q]);
  }
  const Pair root2 = pair_of(h.root2, h.root2), eps = pair_of(h.eps, h.eps);
  const Pair down = pair_of(-h.size, -h.size), keep = pair_of(h.keep, h.keep);
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      float lo, hi;
      unpair(fma2(pair_of(root[j][q], root[j][q + 1]), root2, eps), lo, hi);
      const Pair ratio = pair_of(m[j][q], m[j][q + 1]) * pair_of(rcp_approx(lo), rcp_approx(hi));
      const Pair old = pair_of(value(r.p[j], q), value(r.p[j], q + 1));
      unpair(fma2(ratio, down, old * keep), p[j][q], p[j][q + 1]);
    }
  }
  uint32_t u[J][2];   // two elements' 16 bits in a word
  if (STATE8 || PARAM == kParamBf16) {
    const uint32_t far = static_cast<uint32_t>(block >> 25);  // element >> 33
    const uint32_t key = far ? h.key ^ mix32(far) : h.key;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t pair = static_cast<uint32_t>((first + 128 * j) >> 1);
      u[j][0] = mix32(key ^ pair);
      u[j][1] = mix32(key ^ (pair + 1));
    }
  }
  const auto dither = [&](int j, int q) {
    return q & 1 ? u[j][q >> 1] >> 16 : u[j][q >> 1] & 0xffffu;
  };
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const long long i = first + 128 * j;
    if (PARAM == kParamF32) {
      store4<FAST>(static_cast<float*>(e.param), i, numel, p[j]);
    } else if (PARAM == kParamMaster) {
      store4_bf16<FAST>(static_cast<__nv_bfloat16*>(e.param), i, numel,
                        make_uint2(bf16_pair(p[j][0], p[j][1]), bf16_pair(p[j][2], p[j][3])));
      store4<FAST>(e.master, i, numel, p[j]);
    } else {
      // up or down by the 16 bits that bf16 does not hold (an infinity has none
      // of them set and stays; a NaN would overflow)
      uint32_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = __float_as_uint(p[j][q]);
        b[q] = p[j][q] == p[j][q] ? w + dither(j, q) : 0x7fc00000u;
      }
      store4_bf16<FAST>(static_cast<__nv_bfloat16*>(e.param), i, numel,
                        make_uint2(__byte_perm(b[0], b[1], 0x7632), __byte_perm(b[2], b[3], 0x7632)));
    }
    if (!STATE8) {
      store4<FAST>(static_cast<float*>(e.m), i, numel, m[j]);
      store4<FAST>(static_cast<float*>(e.v), i, numel, v[j]);
    }
  }
  if (STATE8) {
    float msc, minv, vsc, vinv;
    block_scale(mtop, msc, minv);
    block_scale(vtop, vsc, vinv);
    if (lane == 0) {
      e.m_scale[block] = msc;
      e.v_scale[block] = vsc;
    }
    const bool low = !(mlow * minv >= 0.015625f && vlow * vinv >= 0.015625f);
    const auto store = [&](auto is_low) {
      constexpr bool LOW = decltype(is_low)::value;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const long long i = first + 128 * j;
        float qm[4], qv[4];
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          unpair(pair_of(m[j][q], m[j][q + 1]) * pair_of(minv, minv), qm[q], qm[q + 1]);
          unpair(pair_of(root[j][q], root[j][q + 1]) * pair_of(vinv, vinv), qv[q], qv[q + 1]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          qm[q] = dither_e4m3<LOW>(qm[q], dither(j, q));
          qv[q] = dither_e4m3<LOW>(qv[q], dither(j, q));
          if (LOW && root[j][q] > 0.f) qv[q] = fmaxf(qv[q], 0.001953125f);  // 2^-9: not zero
        }
        store4_codes<FAST>(static_cast<uint8_t*>(e.m), i, numel, qm);
        store4_codes<FAST>(static_cast<uint8_t*>(e.v), i, numel, qv);
      }
    };
    if (__any_sync(0xffffffffu, low)) store(std::true_type{});
    else store(std::false_type{});
  }
}

// A block at the tensor's end, or of a tensor whose buffers are not aligned for
// the wide loads; kept out of line so that it costs the loop no registers.
template <int PARAM, bool GRAD16, bool STATE8>
__device__ __noinline__ void adam_block_slow(const AdamEntry& e, Hyper h, long long block) {
  typename AdamTypes<PARAM, GRAD16, STATE8>::Raw r;
  adam_load<PARAM, GRAD16, STATE8, false>(e, block, r);
  adam_block<PARAM, GRAD16, STATE8, false>(e, h, block, r);
}

__device__ __forceinline__ void stage_words(const unsigned char* p, uint32_t (&x)[4]) {
  const uint4 f = *reinterpret_cast<const uint4*>(p);
  x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
}
__device__ __forceinline__ void stage_words(const unsigned char* p, uint32_t (&x)[2]) {
  const uint2 f = *reinterpret_cast<const uint2*>(p);
  x[0] = f.x; x[1] = f.y;
}
__device__ __forceinline__ void stage_words(const unsigned char* p, uint32_t (&x)[1]) {
  x[0] = *reinterpret_cast<const uint32_t*>(p);
}

// Shared-memory staging of an 8-bit block's inputs: every thread copies its own
// 2 x 4 elements of each array asynchronously, kStages - 1 chunks ahead, and reads
// them back itself, so nothing but its own wait orders them within a tensor. The
// arrays' places depend on the tensor's types, so each warp has a part of its own,
// and its lanes meet before they go on to another tensor.
constexpr int kStages = 2;
constexpr int kWarpStage = 32 * 80;              // 2 x 4 of two fp32 and two byte arrays per lane
constexpr int kStageBytes = kOptThreads / 32 * kWarpStage;
constexpr int kAdamSmem = kStages * kStageBytes;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

template <int PARAM, bool GRAD16>
__device__ __forceinline__ void adam_run_staged(const AdamEntry& e, const Hyper& h, long long c,
                                                long long stride, unsigned char* smem) {
  using T = AdamTypes<PARAM, GRAD16, true>;
  constexpr int G = 4 * sizeof(typename T::Grad), P = 4 * sizeof(typename T::Param);
  constexpr int S = 4;   // bytes of four elements
  constexpr int per = kChunk / kBlock;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncwarp();
  const int count = static_cast<int>(c / stride) + 1;
  const long long hop = stride * per;            // blocks from one chunk of this warp's to the next
  const void* param = PARAM == kParamMaster ? static_cast<const void*>(e.master) : e.param;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const auto issue = [&](int k, long long block) {
    const uint32_t st = base + (k % kStages) * kStageBytes;
    const long long at = block * kBlock + lane * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const long long i = at + 128 * j;
      const uint32_t slot = (j * 32 + lane) * 4;   // bytes of one-byte elements
      copy_async<G>(st + slot * (G / 4), static_cast<const typename T::Grad*>(e.grad) + i);
      copy_async<P>(st + 64 * G + slot * (P / 4), static_cast<const typename T::Param*>(param) + i);
      copy_async<S>(st + 64 * (G + P) + slot, static_cast<const uint8_t*>(e.m) + i);
      copy_async<S>(st + 64 * (G + P + S) + slot, static_cast<const uint8_t*>(e.v) + i);
    }
  };
  const auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  long long block = c * per + warp;
  typename T::Raw r;
  adam_load<PARAM, GRAD16, true, true>(e, block, r);   // the first one straight away
#pragma unroll
  for (int k = 1; k < kStages - 1; ++k) {
    if (k < count) issue(k, block - k * hop);
    commit();
  }
  for (int k = 0; k < count; ++k, block -= hop) {
    if (k + kStages - 1 < count) issue(k + kStages - 1, block - (kStages - 1) * hop);
    commit();
    float next_ms = 0.f, next_vs = 0.f;
    if (k + 1 < count) {
      next_ms = e.m_scale[block - hop];
      next_vs = e.v_scale[block - hop];
    }
    if (k > 0) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const unsigned char* st = smem + (k % kStages) * kStageBytes;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t slot = j * 32 + lane;
        stage_words(st + slot * G, r.g[j]);
        stage_words(st + 64 * G + slot * P, r.p[j]);
        stage_words(st + 64 * (G + P) + slot * S, r.m[j]);
        stage_words(st + 64 * (G + P + S) + slot * S, r.v[j]);
      }
    }
    adam_block<PARAM, GRAD16, true, true>(e, h, block, r);
    r.ms = next_ms;
    r.vs = next_vs;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The warp's blocks of chunks c, c - stride, c - 2 stride, ... >= 0 of one tensor.
template <int PARAM, bool GRAD16, bool STATE8>
__device__ __forceinline__ void adam_run(const AdamEntry& e, const Hyper& h, long long c,
                                         long long stride, unsigned char* smem) {
  using T = AdamTypes<PARAM, GRAD16, STATE8>;
  constexpr int per = kChunk / kBlock;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!((e.kind >> 4) & 1)) {
    for (; c >= 0; c -= stride)
      if ((c * per + warp) * kBlock < e.numel)
        adam_block_slow<PARAM, GRAD16, STATE8>(e, h, c * per + warp);
    return;
  }
  const long long last = c * per + warp;  // the first block to do: the only one that can be ragged
  if ((last + 1) * kBlock > e.numel) {
    if (last * kBlock < e.numel) adam_block_slow<PARAM, GRAD16, STATE8>(e, h, last);
    c -= stride;
  }
  if constexpr (!STATE8) {
    for (; c >= 0; c -= stride) {
      typename T::Raw r;
      adam_load<PARAM, GRAD16, STATE8, true>(e, c * per + warp, r);
      adam_block<PARAM, GRAD16, STATE8, true>(e, h, c * per + warp, r);
    }
  } else if (c >= 0) {
    adam_run_staged<PARAM, GRAD16>(e, h, c, stride, smem + warp * kWarpStage);
  }
}

// One pass over parameters, gradients and states. The CTAs go through the list side
// by side, the last chunk first: the norm's kernel goes upwards, so what it read
// last is still in the L2. Measured: 75 M parameters with fp32 master copies, fp32
// gradients and states 367 us, 6.2 TB/s of the 30 bytes per element (bound by
// memory); 151 M with 8-bit states 502 us, 5.4 TB/s of their 18 bytes, at 62
// instructions per element (issue slots 63% taken; fetching, rounding and memory
// overlap only in part); 37.7 M bf16 parameters and gradients with 8-bit states,
// 10 bytes per element, are bound by instruction issue.
// HAS8 = false: no tensor of the list has 8-bit states. That kernel is bound by
// memory and is fastest with few CTAs side by side (75 M parameters with master
// copies: 363 us with two per SM, 379 with three or four, 400 with inputs staged
// ahead: more reads in flight only get in the way of the writes). With 8-bit
// states the arithmetic takes about as long as the traffic, and more warps and
// loads ahead of it overlap the two.
template <bool HAS8>
struct AdamShape {
  static constexpr int ctas = HAS8 ? 3 : 2;   // per SM
  static constexpr int smem = HAS8 ? kAdamSmem : 0;
};

template <int CAP, bool HAS8>
__global__ void __launch_bounds__(kOptThreads, AdamShape<HAS8>::ctas)
adamw_kernel(const __grid_constant__ AdamTable<CAP> t) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ double s_inv_bc1, s_root2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Hyper h;
  h.beta1 = t.h.beta1; h.omb1 = t.h.omb1; h.beta2 = t.h.beta2; h.omb2 = t.h.omb2;
  h.eps = t.h.eps;
  h.root2 = t.h.root2;
  h.scale = t.h.grad_scale ? *t.h.grad_scale : 1.f;
  if (!isfinite(h.scale)) return;  // a bad step: nothing changes
  long long step = t.h.step;
  double lr = 0.0, inv_bc1 = 0.0;
  if (t.h.dynamic) {
    if (t.h.step_dev) step = *t.h.step_dev;
    lr = t.h.lr_dev ? static_cast<double>(*t.h.lr_dev) : t.h.lr;
    if (threadIdx.x == 0) {
      const double n = static_cast<double>(step > 1 ? step : 1);
      s_inv_bc1 = 1.0 / (1.0 - pow(t.h.beta1_d, n));
      s_root2 = rsqrt(1.0 - pow(t.h.beta2_d, n));
    }
    __syncthreads();
    inv_bc1 = s_inv_bc1;
    h.root2 = static_cast<float>(s_root2);
  }
  const uint32_t call_key = mix32(mix32(t.h.seed) ^ static_cast<uint32_t>(step));
  for (long long u = t.h.chunks - 1 - blockIdx.x; u >= 0;) {
    const AdamEntry& e = t.e[find_tensor(t.e, t.h.count, u)];
    const long long c = u - e.first;
    h.size = e.size;
    h.keep = e.keep;
    if (t.h.dynamic) {
      const double rate = lr * static_cast<double>(e.size);
      h.size = static_cast<float>(rate * inv_bc1);
      h.keep = static_cast<float>(1.0 - rate * static_cast<double>(e.keep));
    }
    h.key = mix32(call_key ^ static_cast<uint32_t>(e.place));
    switch (e.kind & 15) {
#define DCT_ADAM(K, P, G, S) case K: adam_run<P, G, S>(e, h, c, gridDim.x, smem); break;
      DCT_ADAM(0, kParamF32, false, false)
      DCT_ADAM(1, kParamBf16, false, false)
      DCT_ADAM(2, kParamMaster, false, false)
      DCT_ADAM(4, kParamF32, true, false)
      DCT_ADAM(5, kParamBf16, true, false)
      DCT_ADAM(6, kParamMaster, true, false)
    }
    if constexpr (HAS8) {
      switch (e.kind & 15) {
        DCT_ADAM(8, kParamF32, false, true)
        DCT_ADAM(9, kParamBf16, false, true)
        DCT_ADAM(10, kParamMaster, false, true)
        DCT_ADAM(12, kParamF32, true, true)
        DCT_ADAM(13, kParamBf16, true, true)
        DCT_ADAM(14, kParamMaster, true, true)
      }
    }
#undef DCT_ADAM
    u -= (c / gridDim.x + 1) * gridDim.x;
  }
}

}  // namespace dct
