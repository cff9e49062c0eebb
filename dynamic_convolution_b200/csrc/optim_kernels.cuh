// Kernels over lists of tensors (include/dynconv_train.h): the norm of all
// gradients and the AdamW step. The list travels as the kernel's parameter, so
// a call copies nothing to the device and a captured launch keeps its own list.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace dct {

constexpr int kOptThreads = 256;
constexpr int kOptVec = 8;                            // elements per thread and chunk
constexpr int kChunk = kOptThreads * kOptVec;         // 2048: eight blocks of 256, one per warp
constexpr int kBlock = 256;                           // elements per scale of an 8-bit state

// ------------------------------------------------------------------ the norm

struct NormEntry {
  const void* grad;
  long long numel;
  long long first_chunk;  // chunks of the list before this tensor
  int bf16, vec;          // vec: 16-byte loads
};
constexpr int kNormCap = 768;
struct NormTable {
  NormEntry e[kNormCap];
  long long chunks;
  int count;
  double* part;
};
static_assert(sizeof(NormTable) <= 32764, "kernel parameters");

constexpr int kNormParts = 1184;  // CTAs of a launch at most: eight per SM of 148

template <typename E>
__device__ __forceinline__ int find_tensor(const E* e, int count, long long chunk) {
  int lo = 0, hi = count - 1;  // the last entry whose first chunk is not after `chunk`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].first_chunk <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Four consecutive elements as fp32, from element `i` of a tensor of numel.
__device__ __forceinline__ void load4(const float* p, long long i, long long numel, bool vec,
                                      float (&x)[4]) {
  if (vec && i + 4 <= numel) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i + q < numel ? p[i + q] : 0.f;
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, long long i, long long numel,
                                      bool vec, float (&x)[4]) {
  if (vec && i + 4 <= numel) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + i);
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i + q < numel ? __bfloat162float(p[i + q]) : 0.f;
  }
}

// Element of a thread's group j (two groups of four): the warp's 256-element
// block is read as two contiguous halves.
__device__ __forceinline__ long long element_at(long long chunk_in_tensor, int j) {
  return chunk_in_tensor * kChunk + (threadIdx.x >> 5) * kBlock + j * 128 + (threadIdx.x & 31) * 4;
}

__global__ void __launch_bounds__(kOptThreads)
grad_norm_kernel(const __grid_constant__ NormTable t) {
  __shared__ double s_sum[kOptThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double sum = 0.0;
  for (long long c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const NormEntry& e = t.e[find_tensor(t.e, t.count, c)];
#pragma unroll
    for (int j = 0; j < kOptVec / 4; ++j) {
      const long long i = element_at(c - e.first_chunk, j);
      float x[4];
      if (e.bf16) load4(static_cast<const __nv_bfloat16*>(e.grad), i, e.numel, e.vec, x);
      else load4(static_cast<const float*>(e.grad), i, e.numel, e.vec, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum = fma(static_cast<double>(x[q]), static_cast<double>(x[q]), sum);
    }
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < kOptThreads / 32; ++w) total += s_sum[w];
    t.part[blockIdx.x] = total;
  }
}

// One CTA: the parts in a fixed order, the factor, the step's number.
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
    const double norm = sqrt(total);
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
  long long first_chunk;
  float lr_scale, decay;
  int kind;     // param kind | grad bf16 << 2 | 8-bit state << 3 | vec << 4
  int place;    // in the caller's list
};

struct AdamShared {
  double lr, inv_bc1, root2;   // root2 = 1 / sqrt(1 - beta2^t)
  float beta1, omb1, beta2, omb2, eps;
  double beta1_d, beta2_d;
  long long step;
  unsigned int seed;
  const float* grad_scale;
  const float* lr_dev;
  const long long* step_dev;
  long long chunks;
  int count;
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

// |y| <= 448 (1 + 2^-22) to the e4m3 grid, as fp32: the 20 mantissa bits that
// e4m3 does not hold get the dither added and are cut off. Below 2^-6, where
// e4m3 has the fixed spacing 2^-9, the value is first moved to [2^-6, 2^-5),
// whose spacing is the same.
__device__ __forceinline__ float dither_e4m3(float y, uint32_t u) {
  const float base = y < 0.015625f ? 0.015625f : 0.f;
  const uint32_t bits = __float_as_uint(__fadd_rn(y, base)) + (u << 4);
  return fminf(__fadd_rn(__uint_as_float(bits & 0xfff00000u), -base), 448.f);
}

__device__ __forceinline__ void store4(float* p, long long i, long long numel, bool vec,
                                       const float (&x)[4]) {
  if (vec && i + 4 <= numel) {
    *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) p[i + q] = x[q];
  }
}
// The upper halves of four fp32 words (values already on the bf16 grid).
__device__ __forceinline__ void store4_bf16(__nv_bfloat16* p, long long i, long long numel,
                                            bool vec, const uint32_t (&b)[4]) {
  if (vec && i + 4 <= numel) {
    uint2 u;
    u.x = __byte_perm(b[0], b[1], 0x7632);
    u.y = __byte_perm(b[2], b[3], 0x7632);
    *reinterpret_cast<uint2*>(p + i) = u;
  } else {
    unsigned short* s = reinterpret_cast<unsigned short*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) s[i + q] = static_cast<unsigned short>(b[q] >> 16);
  }
}

__device__ __forceinline__ void load4_codes(const uint8_t* p, long long i, long long numel,
                                            bool vec, float (&x)[4]) {
  uint32_t w = 0;
  if (vec && i + 4 <= numel) {
    w = *reinterpret_cast<const uint32_t*>(p + i);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) w |= static_cast<uint32_t>(p[i + q]) << (8 * q);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * h)) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(two));
    x[2 * h] = f.x;
    x[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ void store4_codes(uint8_t* p, long long i, long long numel, bool vec,
                                             const float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t w = lo | (hi << 16);
  if (vec && i + 4 <= numel) {
    *reinterpret_cast<uint32_t*>(p + i) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < numel) p[i + q] = static_cast<uint8_t>(w >> (8 * q));
  }
}

// The block's factor and its inverse from its largest magnitude (a non-finite
// one passes through both: the block is spoilt, not hidden).
__device__ __forceinline__ void block_scale(uint32_t top_bits, float& scale, float& inv) {
  const float top = __uint_as_float(top_bits);
  const bool none = top < 7.888609052210118e-31f;  // 2^-100
  scale = none ? 0.f : __fmul_rn(top, 1.f / 448.f);
  inv = none ? 0.f : __fmul_rn(__frcp_rn(top), 448.f);
}

struct Hyper {
  float beta1, omb1, beta2, omb2, eps, size, root2, decay, scale;
  uint32_t key;
};

// One chunk of one tensor. m and v are advanced with separately rounded
// products and sums, so that an 8-bit code follows from the inputs alone and
// not from how a compiler contracts them.
template <int PARAM, bool GRAD16, bool STATE8>
__device__ __forceinline__ void adam_chunk(const AdamEntry& e, const Hyper& h, long long chunk) {
  const bool vec = (e.kind >> 4) & 1;
  const long long numel = e.numel;
  constexpr int J = kOptVec / 4;
  float g[J][4], p[J][4], m[J][4], v[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const long long i = element_at(chunk, j);
    if (GRAD16) load4(static_cast<const __nv_bfloat16*>(e.grad), i, numel, vec, g[j]);
    else load4(static_cast<const float*>(e.grad), i, numel, vec, g[j]);
    if (PARAM == kParamF32) load4(static_cast<const float*>(e.param), i, numel, vec, p[j]);
    if (PARAM == kParamBf16) load4(static_cast<const __nv_bfloat16*>(e.param), i, numel, vec, p[j]);
    if (PARAM == kParamMaster) load4(e.master, i, numel, vec, p[j]);
    if (STATE8) {
      load4_codes(static_cast<const uint8_t*>(e.m), i, numel, vec, m[j]);
      load4_codes(static_cast<const uint8_t*>(e.v), i, numel, vec, v[j]);
    } else {
      load4(static_cast<const float*>(e.m), i, numel, vec, m[j]);
      load4(static_cast<const float*>(e.v), i, numel, vec, v[j]);
    }
  }
  const long long block = chunk * (kChunk / kBlock) + (threadIdx.x >> 5);
  const bool any = block * kBlock < numel;  // this warp's block lies in the tensor
  float ms = 1.f, vs = 1.f;
  if (STATE8 && any) {
    ms = e.m_scale[block];
    vs = e.v_scale[block];
  }
  uint32_t u[J][4];
  if (STATE8 || PARAM == kParamBf16) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t pair = static_cast<uint32_t>(element_at(chunk, j) >> 1);
      const uint32_t h0 = mix32(h.key ^ pair), h1 = mix32(h.key ^ (pair + 1));
      u[j][0] = h0 & 0xffffu; u[j][1] = h0 >> 16;
      u[j][2] = h1 & 0xffffu; u[j][3] = h1 >> 16;
    }
  }
  float root[J][4];
  uint32_t mtop = 0, vtop = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float gr = __fmul_rn(g[j][q], h.scale);
      float m0 = m[j][q], v0 = v[j][q];
      if (STATE8) {
        m0 = __fmul_rn(m0, ms);
        v0 = __fmul_rn(v0, vs);
        v0 = __fmul_rn(v0, v0);
      }
      m0 = __fadd_rn(__fmul_rn(m0, h.beta1), __fmul_rn(gr, h.omb1));
      v0 = __fadd_rn(__fmul_rn(v0, h.beta2), __fmul_rn(__fmul_rn(gr, gr), h.omb2));
      const float r = __fsqrt_rn(v0);
      p[j][q] = p[j][q] * h.decay - h.size * __fdividef(m0, fmaf(r, h.root2, h.eps));
      m[j][q] = m0;
      v[j][q] = v0;
      if (STATE8) {
        root[j][q] = r;
        mtop = max(mtop, __float_as_uint(m0) & 0x7fffffffu);
        vtop = max(vtop, __float_as_uint(r) & 0x7fffffffu);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const long long i = element_at(chunk, j);
    if (PARAM == kParamF32) {
      store4(static_cast<float*>(e.param), i, numel, vec, p[j]);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (PARAM == kParamMaster) {
          b[q] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(p[j][q]))) << 16;
        } else {
          // up or down by the 16 bits that bf16 does not hold; not finite: as it is
          const uint32_t w = __float_as_uint(p[j][q]);
          b[q] = (w & 0x7f800000u) == 0x7f800000u ? (p[j][q] != p[j][q] ? 0x7fc00000u : w)
                                                  : w + u[j][q];
        }
      }
      store4_bf16(static_cast<__nv_bfloat16*>(e.param), i, numel, vec, b);
      if (PARAM == kParamMaster) store4(e.master, i, numel, vec, p[j]);
    }
    if (!STATE8) {
      store4(static_cast<float*>(e.m), i, numel, vec, m[j]);
      store4(static_cast<float*>(e.v), i, numel, vec, v[j]);
    }
  }
  if (STATE8) {
    float msc, minv, vsc, vinv;
    block_scale(__reduce_max_sync(0xffffffffu, mtop), msc, minv);
    block_scale(__reduce_max_sync(0xffffffffu, vtop), vsc, vinv);
    if (any && (threadIdx.x & 31) == 0) {
      e.m_scale[block] = msc;
      e.v_scale[block] = vsc;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const long long i = element_at(chunk, j);
      float qm[4], qv[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        qm[q] = copysignf(dither_e4m3(__fmul_rn(fabsf(m[j][q]), minv), u[j][q]), m[j][q]);
        qv[q] = dither_e4m3(__fmul_rn(root[j][q], vinv), u[j][q]);
        if (root[j][q] > 0.f && vsc > 0.f) qv[q] = fmaxf(qv[q], 0.001953125f);
      }
      store4_codes(static_cast<uint8_t*>(e.m), i, numel, vec, qm);
      store4_codes(static_cast<uint8_t*>(e.v), i, numel, vec, qv);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kOptThreads)
adamw_kernel(const __grid_constant__ AdamTable<CAP> t) {
  __shared__ double s_inv_bc1, s_root2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Hyper h;
  h.beta1 = t.h.beta1; h.omb1 = t.h.omb1; h.beta2 = t.h.beta2; h.omb2 = t.h.omb2;
  h.eps = t.h.eps;
  h.scale = t.h.grad_scale ? *t.h.grad_scale : 1.f;
  if (!isfinite(h.scale)) return;  // a bad step: nothing changes
  const double lr = t.h.lr_dev ? static_cast<double>(*t.h.lr_dev) : t.h.lr;
  long long step = t.h.step;
  double inv_bc1 = t.h.inv_bc1, root2 = t.h.root2;
  if (t.h.step_dev) {
    step = *t.h.step_dev;
    if (threadIdx.x == 0) {
      const double n = static_cast<double>(step > 1 ? step : 1);
      s_inv_bc1 = 1.0 / (1.0 - pow(t.h.beta1_d, n));
      s_root2 = rsqrt(1.0 - pow(t.h.beta2_d, n));
    }
    __syncthreads();
    inv_bc1 = s_inv_bc1;
    root2 = s_root2;
  }
  h.root2 = static_cast<float>(root2);
  const uint32_t call_key = mix32(mix32(t.h.seed) ^ static_cast<uint32_t>(step));
  for (long long c = blockIdx.x; c < t.h.chunks; c += gridDim.x) {
    const AdamEntry& e = t.e[find_tensor(t.e, t.h.count, c)];
    const long long chunk = c - e.first_chunk;
    const double rate = lr * static_cast<double>(e.lr_scale);
    h.size = static_cast<float>(rate * inv_bc1);
    h.decay = static_cast<float>(1.0 - rate * static_cast<double>(e.decay));
    h.key = mix32(call_key ^ static_cast<uint32_t>(e.place));
    const uint32_t far = static_cast<uint32_t>(chunk * kChunk >> 33);
    if (far) h.key ^= mix32(far);
    switch (e.kind & 15) {
      case 0: adam_chunk<kParamF32, false, false>(e, h, chunk); break;
      case 1: adam_chunk<kParamBf16, false, false>(e, h, chunk); break;
      case 2: adam_chunk<kParamMaster, false, false>(e, h, chunk); break;
      case 4: adam_chunk<kParamF32, true, false>(e, h, chunk); break;
      case 5: adam_chunk<kParamBf16, true, false>(e, h, chunk); break;
      case 6: adam_chunk<kParamMaster, true, false>(e, h, chunk); break;
      case 8: adam_chunk<kParamF32, false, true>(e, h, chunk); break;
      case 9: adam_chunk<kParamBf16, false, true>(e, h, chunk); break;
      case 10: adam_chunk<kParamMaster, false, true>(e, h, chunk); break;
      case 12: adam_chunk<kParamF32, true, true>(e, h, chunk); break;
      case 13: adam_chunk<kParamBf16, true, true>(e, h, chunk); break;
      case 14: adam_chunk<kParamMaster, true, true>(e, h, chunk); break;
    }
  }
}

}  // namespace dct
