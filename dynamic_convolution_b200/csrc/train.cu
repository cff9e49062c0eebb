// Host side of the training entry points declared in include/dynconv_train.h:
// argument checks, workspace layout and launches of the balance-loss, gradient
// norm and AdamW kernels. A translation unit of its own (device state and error
// reporting through internal.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <new>
#include <utility>

#include "dynconv.h"
#include "dynconv_train.h"
#include "internal.h"

#include "balance_kernels.cuh"
#include "optim_kernels.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t align16(size_t v) { return (v + 15) & ~size_t(15); }
// Units that hold `total` items (64 bits throughout: rows and elements reach 2^31).
long long units_of(long long total, long long unit) { return (total + unit - 1) / unit; }

// Launch with a programmatic edge: the kernel may be scheduled while the
// previous one on the stream finishes, and waits for it (griddepcontrol.wait)
// before it touches global memory. cluster > 1: that many CTAs to a cluster.
template <typename Kern, typename... Args>
int launch_cluster(const char* what, Kern kern, dim3 grid, int cluster, int threads, size_t smem,
                   cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return dc_lib::cuda_error(e, what);
  }
  return dc_lib::launched(what);
}
template <typename Kern, typename... Args>
int launch(const char* what, Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t stream,
           const Args&... args) {
  return launch_cluster(what, kern, grid, 1, threads, smem, stream, args...);
}

// ------------------------------------------------------------------- balance

int check_balance(const dynconv_balance_desc* d) {
  if (!d || d->rows < 0 || d->groups < 1 || d->n < 1 || d->top_k < 1 || d->top_k > d->n)
    return DYNCONV_ERR_INVALID_ARG;
  if (d->mode != DYNCONV_SIGMOID && d->mode != DYNCONV_SOFTMAX) return DYNCONV_ERR_INVALID_ARG;
  const long long width = 1LL * d->groups * d->n;
  if (d->row_stride < width) return DYNCONV_ERR_INVALID_ARG;
  if (d->n > dct::kBalMaxN || width > 65536 || d->groups > 65535 || d->row_stride >= (1LL << 40) ||
      (d->top_k > dct::kBalMaxTopK && d->top_k != d->n))
    return DYNCONV_ERR_UNSUPPORTED;
  return DYNCONV_OK;
}

constexpr int kBalWarps = dct::kBalThreads / 32;

// Lanes of a warp that hold one row (see balance_kernels.cuh).
int row_lanes(int n) {
  int lanes = 1;
  while (lanes < 32 && lanes * 8 < n) lanes *= 2;
  return lanes;
}

// The whole forward in one launch of one cluster of up to eight CTAs of 256 or
// 1024 threads, each taking every eighth group: while the busiest of them has at
// most 4 K attentions of at most 256 experts. (64 rows of 4 in one group: forward and
// backward 10.1 us, 12.8 with two launches. The groups of a CTA come one after another,
// about 2 us each: 2 rows of 4 in 16 groups 8 us, in 64 groups 18, in 1024 groups 231.)
bool balance_small(const dynconv_balance_desc* d) {
  const long long turns = (d->groups + dct::kBalCluster - 1) / dct::kBalCluster;
  return d->n <= 256 && turns * d->rows * d->n <= 4096;
}

// The forward's split over CTAs (per group): CTAs with an SM of 148 to themselves,
// or, where those would leave SMs idle, four times as many of 256 threads.
struct BalSplit {
  int parts, threads;
};
BalSplit balance_split(const dynconv_balance_desc* d) {
  const int lanes = row_lanes(d->n);
  const auto ctas = [&](int threads) { return units_of(d->rows, threads / lanes); };
  BalSplit s;
  s.threads = dct::forward_threads(d->n <= 256 ? 8 : d->n <= 512 ? 16 : 32);
  int most = 148;
  if (ctas(s.threads) * d->groups < 148) {
    s.threads = dct::kBalThreads;
    most = 592;
  }
  s.parts = static_cast<int>(std::max(1LL, std::min<long long>(ctas(s.threads), most / d->groups)));
  return s;
}

// The forward's workspace: its parts' sums, counts and rows, the finishing CTAs'
// shares of the loss, and their ticket.
struct BalLayout {
  size_t count, kept, dot, ticket, total;
};
BalLayout balance_layout(const dynconv_balance_desc* d) {
  const size_t parts = balance_split(d).parts, width = 1ull * d->groups * d->n;
  BalLayout l;
  l.count = align16(parts * width * 8);
  l.kept = l.count + align16(parts * width * 4);
  l.dot = l.kept + align16(parts * 4);
  l.ticket = l.dot + align16((width + dct::kBalTile - 1) / dct::kBalTile * 8);
  l.total = l.ticket + 16;
  return l;
}

// Calls f with the row layout <L, V> for n attentions.
template <typename F>
int with_layout(int n, F f) {
  if (n <= 4) return f.template operator()<1, 4>();
  if (n <= 8) return f.template operator()<1, 8>();
  if (n <= 16) return f.template operator()<2, 8>();
  if (n <= 32) return f.template operator()<4, 8>();
  if (n <= 64) return f.template operator()<8, 8>();
  if (n <= 128) return f.template operator()<16, 8>();
  if (n <= 256) return f.template operator()<32, 8>();
  if (n <= 512) return f.template operator()<32, 16>();
  return f.template operator()<32, 32>();
}

struct LaunchForward {
  dim3 grid;
  int threads;
  cudaStream_t s;
  const dct::BalParams& p;
  template <int L, int V>
  int operator()() const {
    return threads == dct::kBalThreads ? with_threads<L, V, dct::kBalThreads>()
                                       : with_threads<L, V, dct::forward_threads(V)>();
  }
  template <int L, int V, int T>
  int with_threads() const {
    const auto kern = dct::balance_forward_kernel<L, V, T>;
    constexpr int smem = dct::forward_smem(V, T);
    if (smem > 0) {
      const cudaError_t e = dc_lib::set_smem(reinterpret_cast<const void*>(kern), smem);
      if (e != cudaSuccess) return dc_lib::cuda_error(e, "cudaFuncSetAttribute(balance_forward)");
    }
    return launch("balance_forward_kernel", kern, grid, T, smem, s, p);
  }
};
struct LaunchSmall {
  int ctas;
  cudaStream_t s;
  const dct::BalParams& p;
  template <int L, int V>
  int operator()() const {
    if constexpr (V <= 8) {
      if (p.rows <= 256 / L)  // one turn of the rows
        return launch_cluster("balance_small_kernel", dct::balance_small_kernel<L, V, 256>,
                              dim3(ctas), ctas, 256, 0, s, p);
      return launch_cluster("balance_small_kernel", dct::balance_small_kernel<L, V, 1024>,
                            dim3(ctas), ctas, 1024, 0, s, p);
    }
    return DYNCONV_ERR_UNSUPPORTED;  // not reached: balance_small() is false above n = 256
  }
};
struct LaunchSigmoid {
  dim3 grid;
  cudaStream_t s;
  const dct::BalBack& p;
  template <int L, int V>
  int operator()() const {
    return launch("balance_backward_sigmoid_kernel", dct::balance_backward_sigmoid_kernel<L, V>,
                  grid, dct::kBalThreads, 0, s, p);
  }
};

// ---------------------------------------------------------- lists of tensors

constexpr int kSmallCap = 32;   // tensors in the short form of the list
constexpr int kAdamCap = 360;   // in the long one (32764 bytes of kernel parameters)
static_assert(sizeof(dct::AdamTable<kAdamCap>) <= 32764, "kernel parameters");

constexpr long long kMaxNumel = 1LL << 40;
constexpr double kMinEps = 1.1754943508222875e-38;  // 2^-126

bool valid_dtype(int t) { return t == DYNCONV_F32 || t == DYNCONV_BF16; }
size_t size_of(int dtype) { return dtype == DYNCONV_F32 ? 4 : 2; }

// No param range given twice (or overlapping another).
int params_apart(const dynconv_train_tensor* t, int count) {
  const auto begin = [&](int i) { return reinterpret_cast<uintptr_t>(t[i].param); };
  const auto end = [&](int i) { return begin(i) + t[i].numel * size_of(t[i].dtype); };
  uintptr_t last = 0;
  bool ascending = true;
  for (int i = 0; i < count && ascending; ++i)
    if (t[i].numel) {
      ascending = begin(i) >= last;
      last = end(i);
    }
  if (ascending) return DYNCONV_OK;
  auto* r = new (std::nothrow) std::pair<uintptr_t, uintptr_t>[count];
  if (!r) return dc_lib::fail(DYNCONV_ERR_INVALID_ARG, "out of host memory");
  int k = 0;
  for (int i = 0; i < count; ++i)
    if (t[i].numel) r[k++] = {begin(i), end(i)};
  std::sort(r, r + k);
  bool apart = true;
  for (int i = 1; i < k; ++i) apart = apart && r[i].first >= r[i - 1].second;
  delete[] r;
  return apart ? DYNCONV_OK
               : dc_lib::fail(DYNCONV_ERR_INVALID_ARG, "a param is given twice or overlaps another");
}

int check_grad(const dynconv_train_tensor& t) {
  if (t.numel < 0 || !valid_dtype(t.grad_dtype)) return DYNCONV_ERR_INVALID_ARG;
  if (t.numel >= kMaxNumel) return DYNCONV_ERR_UNSUPPORTED;
  if (t.numel && !t.grad) return DYNCONV_ERR_INVALID_ARG;
  if (t.numel && !aligned(t.grad, size_of(t.grad_dtype))) return DYNCONV_ERR_MISALIGNED;
  return DYNCONV_OK;
}

int check_state(const dynconv_train_tensor& t) {
  if (!valid_dtype(t.dtype)) return DYNCONV_ERR_INVALID_ARG;
  if (t.state_bits != 8 && t.state_bits != 32) return DYNCONV_ERR_UNSUPPORTED;
  if (!std::isfinite(t.lr_scale) || t.lr_scale < 0 || !std::isfinite(t.weight_decay) ||
      t.weight_decay < 0)
    return DYNCONV_ERR_INVALID_ARG;
  if (t.master && t.dtype != DYNCONV_BF16) return DYNCONV_ERR_INVALID_ARG;
  if (t.numel == 0) return DYNCONV_OK;
  if (!t.param || !t.m || !t.v || (t.state_bits == 8 && (!t.m_scale || !t.v_scale)))
    return DYNCONV_ERR_INVALID_ARG;
  const size_t st = t.state_bits == 8 ? 1 : 4;
  if (!aligned(t.param, size_of(t.dtype)) || !aligned(t.master, 4) || !aligned(t.m, st) ||
      !aligned(t.v, st))
    return DYNCONV_ERR_MISALIGNED;
  if (t.state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
    return DYNCONV_ERR_MISALIGNED;
  return DYNCONV_OK;
}

// Four elements of the type are one load of 4 * size bytes.
bool vec_ok(const void* p, size_t elem) { return aligned(p, 4 * elem); }

template <int CAP, bool HAS8>
int launch_adam(const dct::AdamShared& h, const dct::AdamEntry* e, int sms, cudaStream_t s) {
  using Shape = dct::AdamShape<HAS8>;
  const auto kern = dct::adamw_kernel<CAP, HAS8>;
  if (Shape::smem > 0) {
    const cudaError_t err = dc_lib::set_smem(reinterpret_cast<const void*>(kern), Shape::smem);
    if (err != cudaSuccess) return dc_lib::cuda_error(err, "cudaFuncSetAttribute(adamw)");
  }
  dct::AdamTable<CAP> t;
  t.h = h;
  std::copy(e, e + h.count, t.e);
  const int grid = static_cast<int>(std::min<long long>(h.chunks, 1LL * sms * Shape::ctas));
  return launch("adamw_kernel", kern, dim3(grid), dct::kOptThreads, Shape::smem, s, t);
}

}  // namespace

extern "C" {

size_t dynconv_balance_workspace_size(const dynconv_balance_desc* desc) {
  return check_balance(desc) == DYNCONV_OK ? balance_layout(desc).total : 0;
}

int dynconv_balance_forward(const dynconv_balance_desc* desc, const float* alpha,
                            const unsigned char* row_mask, float coef, int* counts, float* mean,
                            int* rows_kept, float* loss, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int rc = check_balance(desc);
  if (rc) return rc;
  if ((!alpha && desc->rows > 0) || !counts || !mean || !rows_kept || !loss ||
      !std::isfinite(coef))
    return DYNCONV_ERR_INVALID_ARG;
  const BalLayout layout = balance_layout(desc);
  if (!workspace || workspace_bytes < layout.total) return DYNCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(alpha, 4) || !aligned(counts, 4) || !aligned(mean, 4) ||
      !aligned(rows_kept, 4) || !aligned(loss, 4))
    return DYNCONV_ERR_MISALIGNED;
  dc_lib::DeviceInfo di;
  rc = dc_lib::device_info(&di);
  if (rc) return rc;
  const BalSplit split = balance_split(desc);
  const int parts = split.parts;
  const size_t width = 1ull * desc->groups * desc->n;
  char* ws = static_cast<char*>(workspace);
  dct::BalParams p{};
  p.rows = desc->rows;
  p.groups = desc->groups;
  p.n = desc->n;
  p.top_k = desc->top_k;
  p.sigmoid = desc->mode == DYNCONV_SIGMOID;
  p.vec = aligned(alpha, 16) && desc->n % 4 == 0 && desc->row_stride % 4 == 0;
  p.stride = desc->row_stride;
  p.alpha = alpha;
  p.mask = row_mask;
  p.part_sum = reinterpret_cast<double*>(ws);
  p.part_count = reinterpret_cast<int*>(ws + layout.count);
  p.part_kept = reinterpret_cast<int*>(ws + layout.kept);
  p.ticket = reinterpret_cast<unsigned*>(ws + layout.ticket);
  p.coef = coef;
  p.counts = counts;
  p.mean = mean;
  p.rows_kept = rows_kept;
  p.loss = loss;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (balance_small(desc))
    return with_layout(desc->n, LaunchSmall{std::min(desc->groups, dct::kBalCluster), s, p});
  rc = with_layout(desc->n, LaunchForward{dim3(parts, desc->groups), split.threads, s, p});
  if (rc) return rc;
  dct::BalFinish f{};
  f.parts = parts;
  f.width = static_cast<int>(width);
  f.n = desc->n;
  f.top_k = desc->top_k;
  f.groups = desc->groups;
  f.coef = coef;
  f.part_sum = p.part_sum;
  f.part_count = p.part_count;
  f.part_kept = p.part_kept;
  f.part_dot = reinterpret_cast<double*>(ws + layout.dot);
  f.ticket = p.ticket;
  f.counts = counts;
  f.mean = mean;
  f.rows_kept = rows_kept;
  f.loss = loss;
  return launch("balance_finish_kernel", dct::balance_finish_kernel,
                dim3(static_cast<unsigned>((width + dct::kBalTile - 1) / dct::kBalTile)),
                dct::kBalFinishThreads, 0, s, f);
}

int dynconv_balance_backward(const dynconv_balance_desc* desc, const float* alpha,
                             const unsigned char* row_mask, float coef, const int* counts,
                             const int* rows_kept, const float* dloss, float* dalpha,
                             long long dalpha_stride, int accumulate, void* stream) {
  int rc = check_balance(desc);
  if (rc) return rc;
  const bool sigmoid = desc->mode == DYNCONV_SIGMOID;
  const long long width = 1LL * desc->groups * desc->n;
  if ((sigmoid && !alpha && desc->rows > 0) || !counts || !rows_kept ||
      (!dalpha && desc->rows > 0) || !std::isfinite(coef) || dalpha_stride < width ||
      (accumulate != 0 && accumulate != 1))
    return DYNCONV_ERR_INVALID_ARG;
  if (dalpha_stride >= (1LL << 40)) return DYNCONV_ERR_UNSUPPORTED;
  if (!aligned(alpha, 4) || !aligned(counts, 4) || !aligned(rows_kept, 4) || !aligned(dloss, 4) ||
      !aligned(dalpha, 4))
    return DYNCONV_ERR_MISALIGNED;
  if (desc->rows == 0) return DYNCONV_OK;
  dc_lib::DeviceInfo di;
  rc = dc_lib::device_info(&di);
  if (rc) return rc;
  dct::BalBack p{};
  p.rows = desc->rows;
  p.groups = desc->groups;
  p.n = desc->n;
  p.width = static_cast<int>(width);
  p.top_k = desc->top_k;
  p.accumulate = accumulate;
  p.stride = desc->row_stride;
  p.dstride = dalpha_stride;
  p.coef = coef;
  p.alpha = alpha;
  p.mask = row_mask;
  p.counts = counts;
  p.rows_kept = rows_kept;
  p.dloss = dloss;
  p.dalpha = dalpha;
  p.vec = aligned(dalpha, 16) && dalpha_stride % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sigmoid) {
    p.vec = p.vec && aligned(alpha, 16) && desc->row_stride % 4 == 0 && desc->n % 4 == 0;
    const long long want = units_of(desc->rows, kBalWarps * (32 / row_lanes(desc->n)));
    const int grid = static_cast<int>(
        std::min<long long>(want, std::max(1LL, 8LL * di.sms / desc->groups)));
    return with_layout(desc->n, LaunchSigmoid{dim3(grid, desc->groups), s, p});
  }
  p.vec = p.vec && width % 4 == 0;
  const int vecs = static_cast<int>((width + 3) / 4);
  int tx = 1;
  while (tx < vecs && tx < dct::kBalThreads) tx *= 2;
  const int gy = (vecs + tx - 1) / tx, ty = dct::kBalThreads / tx;
  const long long want = units_of(desc->rows, ty);
  const int gx = static_cast<int>(std::min<long long>(want, std::max(1LL, 8LL * di.sms / gy)));
  return launch("balance_backward_softmax_kernel", dct::balance_backward_softmax_kernel,
                dim3(gx, gy), dct::kBalThreads, 0, s, p, tx);
}

size_t dynconv_grad_norm_workspace_size(int count) {
  if (count < 0) return 0;
  const size_t launches = std::max(1LL, units_of(count, dct::kNormCap));
  return launches * dct::kNormParts * sizeof(double);
}

int dynconv_grad_norm(const dynconv_train_tensor* tensors, int count, double max_norm,
                      float* stats, long long* step, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !stats || !(max_norm > 0))
    return DYNCONV_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (int rc = check_grad(tensors[i])) return rc;
  if (!workspace || workspace_bytes < dynconv_grad_norm_workspace_size(count))
    return DYNCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(stats, 4) || !aligned(step, 8))
    return DYNCONV_ERR_MISALIGNED;
  dc_lib::DeviceInfo di;
  int rc = dc_lib::device_info(&di);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int parts = 0;
  // A CTA takes units of one or two pieces of a tensor: two on large lists, where the
  // tensor is looked up less often then, one where small lists have to spread over
  // the GPU. (Four leave the last round of CTAs uneven: 97 us for 92 on 151 M fp32.)
  long long all = 0;
  for (int i = 0; i < count; ++i) all += units_of(tensors[i].numel, dct::kNormPiece);
  const int pieces = static_cast<int>(std::max(1LL, std::min(2LL, all / (2 * dct::kNormParts))));
  for (int i = 0; i < count;) {
    dct::NormTable<dct::kNormCap> t;
    t.count = 0;
    t.units = 0;
    t.part = part + parts;
    t.pieces = pieces;
    for (; i < count && t.count < dct::kNormCap; ++i) {
      const dynconv_train_tensor& a = tensors[i];
      if (a.numel == 0) continue;
      dct::NormEntry& e = t.e[t.count++];
      e.grad = a.grad;
      e.numel = a.numel;
      e.first = t.units;
      e.bf16 = a.grad_dtype == DYNCONV_BF16;
      e.vec = aligned(a.grad, 16);
      t.units += units_of(a.numel, 1LL * pieces * dct::kNormPiece);
    }
    if (t.count == 0) break;
    const int grid = static_cast<int>(std::min<long long>(t.units, dct::kNormParts));
    if (t.count <= kSmallCap) {
      dct::NormTable<kSmallCap> few;
      std::copy(t.e, t.e + t.count, few.e);
      few.units = t.units;
      few.count = t.count;
      few.part = t.part;
      few.pieces = pieces;
      rc = launch("grad_norm_kernel", dct::grad_norm_kernel<kSmallCap>, dim3(grid),
                  dct::kOptThreads, 0, s, few);
    } else {
      rc = launch("grad_norm_kernel", dct::grad_norm_kernel<dct::kNormCap>, dim3(grid),
                  dct::kOptThreads, 0, s, t);
    }
    if (rc) return rc;
    parts += grid;
  }
  return launch("grad_norm_finish_kernel", dct::grad_norm_finish_kernel, dim3(1),
                dct::kOptThreads, 0, s, static_cast<const double*>(part), parts, max_norm, stats,
                step);
}

int dynconv_adamw(const dynconv_train_tensor* tensors, int count,
                  const dynconv_adamw_hyper* hyper, const float* grad_scale, const float* lr,
                  const long long* step, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !hyper) return DYNCONV_ERR_INVALID_ARG;
  const auto beta_ok = [](double b) { return b >= 0 && b < 1; };
  if (!(hyper->lr >= 0) || !std::isfinite(hyper->lr) || !beta_ok(hyper->beta1) ||
      !beta_ok(hyper->beta2) || !(hyper->eps >= kMinEps) || !(hyper->eps <= 1e30) ||
      (!step && hyper->step < 1))
    return DYNCONV_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (int rc = check_grad(tensors[i])) return rc;
    if (int rc = check_state(tensors[i])) return rc;
  }
  if (!aligned(grad_scale, 4) || !aligned(lr, 4) || !aligned(step, 8))
    return DYNCONV_ERR_MISALIGNED;
  int rc = params_apart(tensors, count);
  if (rc) return rc;
  dc_lib::DeviceInfo di;
  rc = dc_lib::device_info(&di);
  if (rc) return rc;
  dct::AdamShared h{};
  h.lr = hyper->lr;
  h.beta1_d = hyper->beta1;
  h.beta2_d = hyper->beta2;
  h.beta1 = static_cast<float>(hyper->beta1);
  h.omb1 = static_cast<float>(1.0 - hyper->beta1);
  h.beta2 = static_cast<float>(hyper->beta2);
  h.omb2 = static_cast<float>(1.0 - hyper->beta2);
  h.eps = static_cast<float>(hyper->eps);
  h.seed = hyper->seed;
  h.grad_scale = grad_scale;
  h.lr_dev = lr;
  h.step_dev = step;
  h.step = hyper->step;
  h.dynamic = lr || step;
  double inv_bc1 = 0.0;
  if (!h.dynamic) {
    const double t = static_cast<double>(hyper->step);
    inv_bc1 = 1.0 / (1.0 - std::pow(hyper->beta1, t));
    h.root2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(hyper->beta2, t)));
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  dct::AdamEntry entries[kAdamCap];
  for (int i = 0; i < count;) {
    h.count = 0;
    h.chunks = 0;
    bool has8 = false;
    for (; i < count && h.count < kAdamCap; ++i) {
      const dynconv_train_tensor& a = tensors[i];
      if (a.numel == 0) continue;
      dct::AdamEntry& e = entries[h.count++];
      e.param = a.param;
      e.master = a.master;
      e.grad = a.grad;
      e.m = a.m;
      e.v = a.v;
      e.m_scale = a.m_scale;
      e.v_scale = a.v_scale;
      e.numel = a.numel;
      e.first = h.chunks;
      e.size = a.lr_scale;
      e.keep = a.weight_decay;
      if (!h.dynamic) {
        const double rate = hyper->lr * a.lr_scale;
        e.size = static_cast<float>(rate * inv_bc1);
        e.keep = static_cast<float>(1.0 - rate * a.weight_decay);
      }
      e.place = i;
      has8 = has8 || a.state_bits == 8;
      const int param = a.dtype == DYNCONV_F32 ? dct::kParamF32
                                               : a.master ? dct::kParamMaster : dct::kParamBf16;
      const size_t st = a.state_bits == 8 ? 1 : 4;
      const bool vec = vec_ok(a.param, size_of(a.dtype)) && vec_ok(a.master, 4) &&
                       vec_ok(a.grad, size_of(a.grad_dtype)) && vec_ok(a.m, st) && vec_ok(a.v, st);
      e.kind = param | (a.grad_dtype == DYNCONV_BF16 ? 4 : 0) | (a.state_bits == 8 ? 8 : 0) |
               (vec ? 16 : 0);
      h.chunks += units_of(a.numel, dct::kChunk);
    }
    if (h.count == 0) break;
    if (h.count <= kSmallCap)
      rc = has8 ? launch_adam<kSmallCap, true>(h, entries, di.sms, s)
                : launch_adam<kSmallCap, false>(h, entries, di.sms, s);
    else
      rc = has8 ? launch_adam<kAdamCap, true>(h, entries, di.sms, s)
                : launch_adam<kAdamCap, false>(h, entries, di.sms, s);
    if (rc) return rc;
  }
  return DYNCONV_OK;
}

}  // extern "C"
