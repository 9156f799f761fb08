// Global norm of a list of gradients, and their scaling in place.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "lanes.h"

namespace moe {

// An item is a number of consecutive elements of one tensor, a workgroup's unit.
constexpr int kGradThreads = 256, kGradItem = 8192;
constexpr int kGradCounters = 32, kGradApart = 32;       // groups of workgroups; a counter's 128 bytes
constexpr int kGradMaxWG = 2048;         // workgroups of the norm, and so partial sums: 8 a CU

struct GradTensor {
  void* g;
  int64_t n;
  int f32;
};
struct GradTable {
  GradTensor* t;
  uint32_t* first;     // [tensors + 1] the first item of each
  double* part;        // [kGradMaxWG]
  int32_t* done;       // workgroups that have written theirs: groups' counters after that of whole groups; 0 between calls
};
static GradTable grad_table(const void* ws, int tensors) {
  char* p = (char*)ws;
  GradTable g;
  g.t = (GradTensor*)p;
  g.first = (uint32_t*)(p += align_up(sizeof(GradTensor) * (size_t)tensors));
  g.part = (double*)(p += align_up(sizeof(uint32_t) * ((size_t)tensors + 1)));
  g.done = (int32_t*)(p + align_up(sizeof(double) * kGradMaxWG));
  return g;
}
size_t grads_ws_bytes(int tensors) {
  return align_up(sizeof(GradTensor) * (size_t)tensors) + align_up(sizeof(uint32_t) * ((size_t)tensors + 1)) +
         align_up(sizeof(double) * kGradMaxWG) + align_up(sizeof(int32_t) * (1 + kGradCounters) * kGradApart);
}

// The table travels in the arguments of launches, as the optimizer's does.
constexpr int kGradPart = 96;
struct GradPart {
  GradTensor t[kGradPart];
  uint32_t first[kGradPart + 1];
};
static_assert(sizeof(GradPart) <= 3900, "kernel arguments");
__global__ void k_grad_table(GradPart part, int base, int count, GradTensor* t, uint32_t* first, int32_t* done) {
  const int i = threadIdx.x;
  if (i < count) t[base + i] = part.t[i];
  if (i <= count) first[base + i] = part.first[i];
  if (i <= kGradCounters) done[i * kGradApart] = 0;
}

struct GradArgs {
  GradTable tab;
  int tensors;
  uint32_t items;
  double max_norm, mult;
  const float* mult_dev;
  float* norm;
  float* scale;
  int32_t* status;
};

// The n (at most kGradItem) elements at g: f(element) of every one.
template <typename T, class F> MOE_DEV void each_of_item(const T* g, int n, F f) {
  constexpr int N = 16 / sizeof(T), R = kGradItem / (kGradThreads * N);
  const int tid = threadIdx.x;
  T v[R][N];
  if (n == kGradItem) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_n<T, N>(g + (r * kGradThreads + tid) * N, v[r]);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int at = (r * kGradThreads + tid) * N;
      load_upto<T, N>(g + at, n - at, v[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < N; ++i) f(elem_f(v[r][i]));
}

MOE_DEV double sum_doubles(double s) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// Squares and sums in 64 bits: no gradient is too small or too large for its square, and the order of
// the sum, which the sizes alone fix, does not show in the 24 bits of the result.  The last workgroup to
// finish joins the partial sums.  Bound by HBM: 604M fp32 elements in 385 us (6.3 TB/s, as fast as an
// elementwise kernel copies 1 GiB; the runtime's own copy reaches 5.2), two 64-bit instructions an element
// being 50 us of the VALU; a few small tensors take 6 us, the latency of the search, a read and the join.
__global__ __launch_bounds__(kGradThreads) void k_grad_norm(GradArgs a) {
  __shared__ double red[kGradThreads / 64];
  __shared__ int last;
  const int tid = threadIdx.x;
  double s = 0.0;
  int j = -1;
  uint32_t begin = 0, end = 0;                           // items of tensor j
  GradTensor t{};
  for (uint32_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    if (item >= end) {
      j = __builtin_amdgcn_readfirstlane(list_place(a.tab.first, a.tensors, item));
      begin = a.tab.first[j];
      end = a.tab.first[j + 1];
      t = a.tab.t[j];
    }
    const int64_t at = (int64_t)(item - begin) * kGradItem;
    const int n = (int)min((int64_t)kGradItem, t.n - at);
    auto add = [&](float g) { s = fma((double)g, (double)g, s); };
    if (t.f32) each_of_item((const float*)t.g + at, n, add);
    else each_of_item((const uint16_t*)t.g + at, n, add);
  }
  s = sum_doubles(s);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    s = red[0] + red[1] + red[2] + red[3];
    // The partial sums are device-scope stores and loads, which pass the XCD's own L2, so the wait alone
    // orders them with the counters: a release at device scope writes that L2 back, and one counter takes
    // its workgroups one by one (25M bf16: 60 us with both, 31 with one counter and no release, 11 so).  It
    // relies on gfx950 acknowledging a device-scope store once it is past the XCD's L2.
    __hip_atomic_store(a.tab.part + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    const int groups = min((int)gridDim.x, kGradCounters), g = blockIdx.x % groups;
    const int members = ((int)gridDim.x - g + groups - 1) / groups;
    auto count = [&](int32_t* c) {
      return __hip_atomic_fetch_add(c, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    last = count(a.tab.done + (1 + g) * kGradApart) == members - 1 && count(a.tab.done) == groups - 1;
  }
  __syncthreads();
  if (!last) return;
  s = 0.0;
#pragma unroll 8
  for (int i = tid; i < (int)gridDim.x; i += kGradThreads)
    s += __hip_atomic_load(a.tab.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = sum_doubles(s);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  if (tid <= kGradCounters) a.tab.done[tid * kGradApart] = 0;      // for the next call
  if (tid) return;
  s = red[0] + red[1] + red[2] + red[3];
  if (!(s < HUGE_VAL)) atomicOr(a.status, MOE_DEV_BAD_GRAD);
  const double mult = a.mult_dev ? (double)*a.mult_dev : a.mult;
  const double norm = fabs(mult) * sqrt(s);
  *a.norm = (float)norm;
  *a.scale = (float)(norm <= a.max_norm ? mult : mult * (a.max_norm / norm));
}

// g = g * scale, a workgroup an item; nothing is read or written where the scale is 1.  A bf16 element is the fp32
// product rounded again, as the plain product of a bf16 tensor and an fp32 scale is: half a step and 2^-24.
// 25M bf16 elements, 100 MB, in 16 us out of the caches that the norm has filled.
template <typename T> MOE_DEV void scale_item(T* g, int n, float scale) {
  constexpr int N = 16 / sizeof(T), R = kGradItem / (kGradThreads * N);
  const int tid = threadIdx.x;
  T v[R][N];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int at = (r * kGradThreads + tid) * N;
    if (n == kGradItem) load_n<T, N>(g + at, v[r]);
    else load_upto<T, N>(g + at, n - at, v[r]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int at = (r * kGradThreads + tid) * N;
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = elem_f(v[r][i]) * scale;
    to_elems<N>(f, v[r]);
    store_upto<T, N>(g + at, n - at, v[r]);
  }
}
__global__ __launch_bounds__(kGradThreads) void k_grad_scale(GradArgs a) {
  const float scale = *a.scale;
  if (scale == 1.f) return;
  const uint32_t item = blockIdx.x;
  const int j = __builtin_amdgcn_readfirstlane(list_place(a.tab.first, a.tensors, item));
  const GradTensor t = a.tab.t[j];
  const int64_t at = (int64_t)(item - a.tab.first[j]) * kGradItem;
  const int n = (int)min((int64_t)kGradItem, t.n - at);
  if (t.f32) scale_item((float*)t.g + at, n, scale);
  else scale_item((uint16_t*)t.g + at, n, scale);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int launch_grads_table(const moe_grad_tensor* t, int count, moe_grad_list* out, hipStream_t st) {
  const GradTable tab = grad_table(out->table, count);
  // an item is a workgroup, and a launch holds fewer than 2^32 threads
  long long all = 0;
  for (int i = 0; i < count; ++i) all += (t[i].n + kGradItem - 1) / kGradItem;
  if (all >= (1ll << 32) / kGradThreads) return MOE_ERR_UNSUPPORTED;
  uint32_t total = 0;
  int base = 0;
  do {                                                   // once for an empty list: its counter
    GradPart part{};
    const int n = std::min(kGradPart, count - base);
    for (int i = 0; i < n; ++i) {
      const moe_grad_tensor& s = t[base + i];
      part.t[i] = {s.g, s.n, s.dtype == MOE_F32};
      part.first[i] = total;
      total += (uint32_t)((s.n + kGradItem - 1) / kGradItem);
    }
    part.first[n] = total;
    hipLaunchKernelGGL(k_grad_table, dim3(1), dim3(128), 0, st, part, base, n, tab.t, tab.first, tab.done);
    base += kGradPart;
  } while (base < count);
  out->items = total;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_grad_norm(const moe_grad_list& l, const moe_clip& c, float* norm, float* scale, int32_t* status,
                     hipStream_t st) {
  GradArgs a{};
  a.tab = grad_table(l.table, l.tensors);
  a.tensors = l.tensors; a.items = l.items;
  a.max_norm = c.max_norm; a.mult = c.mult; a.mult_dev = c.mult_dev;
  a.norm = norm; a.scale = scale; a.status = status;
  const unsigned grid = std::max(1u, std::min(l.items, (uint32_t)kGradMaxWG));
  hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(kGradThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_grad_scale(const moe_grad_list& l, const float* scale, hipStream_t st) {
  if (l.items == 0) return MOE_OK;
  GradArgs a{};
  a.tab = grad_table(l.table, l.tensors);
  a.tensors = l.tensors; a.items = l.items;
  a.scale = const_cast<float*>(scale);
  hipLaunchKernelGGL(k_grad_scale, dim3(l.items), dim3(kGradThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
