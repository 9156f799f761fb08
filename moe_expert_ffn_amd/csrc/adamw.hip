// AdamW over a list of tensors: parameters in fp32 or bf16, states in fp32 or
// in e4m3 codes with block scales.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "lanes.h"

namespace moe {

// The table of a prepared list: the tensors, and the first item of each.  An
// item is kAdamItem consecutive elements of one tensor, a workgroup's unit.
constexpr int kAdamItem = 4096, kAdamThreads = 256, kAdamVE = 8;
static_assert(MOE_ADAMW_BLOCK == 16 * kAdamVE, "a block of states is a row of 16 lanes");

struct AdamTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int p32, g32, vec, pad;
};
struct AdamTable { AdamTensor* t; uint32_t* first; };
static AdamTable adamw_table(const void* ws, int tensors) {
  return {(AdamTensor*)ws,
          (uint32_t*)((char*)ws + align_up(sizeof(AdamTensor) * (size_t)tensors))};
}
size_t adamw_ws_bytes(int tensors) {
  return align_up(sizeof(AdamTensor) * (size_t)tensors) +
         align_up(sizeof(uint32_t) * ((size_t)tensors + 1));
}

// The table travels in the arguments of launches, a part at a time: no copy
// from host memory, which a captured graph could not keep.
constexpr int kAdamPart = 32;
struct AdamPart {
  AdamTensor t[kAdamPart];
  uint32_t first[kAdamPart + 1];
};
static_assert(sizeof(AdamPart) <= 3900, "kernel arguments");
__global__ void k_adamw_table(AdamPart part, int base, int count, AdamTensor* t, uint32_t* first) {
  const int i = threadIdx.x;
  if (i < count) t[base + i] = part.t[i];
  if (i <= count) first[base + i] = part.first[i];
}

struct AdamArgs {
  const AdamTensor* t;
  const uint32_t* first;
  int tensors;
  uint32_t items;
  float lr, beta1, beta2, c1, c2, eps, wd;   // c = 1 - beta
  double log_beta1, log_beta2;   // -infinity for 0
  int step;
  uint32_t seed;
  const int32_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
};

constexpr uint32_t kGold = 0x9E3779B9u, kRoot2 = 0x6A09E667u, kRoot3 = 0xBB67AE85u;
MOE_DEV uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= kRoot2;
  return x ^ (x >> 15);
}

// Eight elements at p; with FULL there are eight and p is aligned for them, else n (at most eight,
// zeros past them) are read one by one.
template <typename T, bool FULL> MOE_DEV void load8(const T* p, int n, T* v) {
  if constexpr (FULL && sizeof(T) == 1) {
    const u32x2_t w = *(const MOE_GLB u32x2_t*)p;
    __builtin_memcpy(v, &w, 8);
  } else if constexpr (FULL) {
    load_n<T, 8, true>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? *(const MOE_GLB T*)(p + i) : (T)0;
  }
}
template <typename T, bool FULL> MOE_DEV void store8(T* p, int n, const T* v) {
  if constexpr (FULL && sizeof(T) == 1) {
    u32x2_t w;
    __builtin_memcpy(&w, v, 8);
    *(MOE_GLB u32x2_t*)p = w;
  } else if constexpr (FULL) {
    store_n<T, 8, true>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) *(MOE_GLB T*)(p + i) = v[i];
  }
}
template <bool FULL> MOE_DEV void load8f(const void* p, bool f32, int64_t at, int n, float* v) {
  if (f32) {
    load8<float, FULL>((const float*)p + at, n, v);
  } else {
    uint16_t h[8];
    load8<uint16_t, FULL>((const uint16_t*)p + at, n, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf2f(h[i]);
  }
}

// Eight e4m3 codes, converted by hardware in pairs, times their scale.
MOE_DEV void from_e4m3(const uint8_t* codes, float scale, float* v) {
  uint32_t w[2];
  __builtin_memcpy(w, codes, 8);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    v[4 * h] = lo.x * scale;
    v[4 * h + 1] = lo.y * scale;
    v[4 * h + 2] = hi.x * scale;
    v[4 * h + 3] = hi.y * scale;
  }
}

// Eight states of a lane into codes; the 16 lanes of a block share its scale.
// y = |x| * 448 / top is rounded up with the probability of the part cut off:
// the low 20 bits of its fp32 word are that part, so adding u16 + 1/2 in units
// of 2^4 to the word and dropping them is floor(y / step + u) steps, in whole
// numbers.  Below e4m3's normal range the step stays 2^-9: there 2^-6 is added
// first, which puts y into an octave with that step.  y is at most two ulps
// above 448, which no u16 carries to the next code, so no clamp is needed.
// SIGNED: x may be negative.  random: bits SHIFT..SHIFT + 15 of word.
template <bool SIGNED, int SHIFT>
MOE_DEV void to_e4m3(const float* x, const uint32_t* word, uint8_t* codes, float* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));       // NaN is passed over
  top = group_all<16>(top, OpMaxF());
  // a value that is not finite stays out of the scale (rare: a branch of whole waves)
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) odd |= !(fabsf(x[i]) < INFINITY);
  if (__any(odd)) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
    top = group_all<16>(top, OpMaxF());
  }
  if (top < 0x1p-100f) top = 0.f;
  const float inv = top > 0.f ? 448.f / top : 0.f;
  const float small = top * (0x1p-6f / 448.f);
  *scale = top * (1.f / 448.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool low = fabsf(x[i]) < small || inv == 0.f;
    const float y = fabsf(x[i]) * inv + (low ? 0x1p-6f : 0.f);
    const uint32_t r = (SHIFT ? word[i] >> (SHIFT - 4) : word[i] << 4) & 0xFFFF0u;
    uint32_t c = ((__float_as_uint(y) + r + 8u) >> 20) - (low ? 121u << 3 : 120u << 3);
    if (SIGNED) c |= __float_as_uint(x[i]) >> 24 & 0x80u;
    codes[i] = (uint8_t)c;
  }
  if (__any(odd)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(fabsf(x[i]) < INFINITY)) codes[i] = 0x7F;
  }
}

// 1 - beta^t, from log(beta) in double: no cancellation at beta near 1
MOE_DEV float bias(double log_beta, int t) { return (float)-expm1(log_beta * t); }

// The tensor that holds an item: how many of first[1..tensors] are at or below
// it.  64 lanes look at a sorted table of up to 64 * 64 entries in two steps.
MOE_DEV int tensor_of(const uint32_t* first, int tensors, uint32_t item) {
  const int lane = threadIdx.x & 63;
  const int i1 = (lane + 1) * 64;
  const int blk = __popcll(__ballot(i1 <= tensors && first[min(i1, tensors)] <= item));
  const int i2 = blk * 64 + 1 + lane;
  return blk * 64 + __popcll(__ballot(i2 <= tensors && first[min(i2, tensors)] <= item));
}

struct AdamRates { float rate, root, keep, gs; };

// Eight consecutive elements at `at` of tensor t (n of them there).
template <int BITS, bool FULL>
MOE_DEV void adam8(const AdamArgs& a, const AdamTensor& t, const AdamRates& h, uint32_t key,
                   int64_t at, int n) {
  float p[8], g[8], m[8], v[8];
  load8f<FULL>(t.master ? t.master : t.p, t.master || t.p32, at, n, p);
  load8f<FULL>(t.g, t.g32, at, n, g);
  if constexpr (BITS == 32) {
    load8<float, FULL>((const float*)t.m + at, n, m);
    load8<float, FULL>((const float*)t.v + at, n, v);
  } else {
    uint8_t mc[8], vc[8];
    load8<uint8_t, FULL>((const uint8_t*)t.m + at, n, mc);
    load8<uint8_t, FULL>((const uint8_t*)t.v + at, n, vc);
    const float ms = n > 0 ? t.ms[at / MOE_ADAMW_BLOCK] : 0.f;
    const float vs = n > 0 ? t.vs[at / MOE_ADAMW_BLOCK] : 0.f;
    from_e4m3(mc, ms, m);
    from_e4m3(vc, vs, v);
  }
  uint32_t word[8];
  const uint32_t w0 = (uint32_t)at * kGold + key;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    word[i] = mix(w0 + (uint32_t)i * kGold);
    if constexpr (BITS == 8) v[i] *= v[i];
    g[i] *= h.gs;
    m[i] = a.beta1 * m[i] + a.c1 * g[i];
    v[i] = a.beta2 * v[i] + a.c2 * g[i] * g[i];
    // sqrt and reciprocal of 1 ulp: the update is lr times a number near 1
    const float s = __builtin_amdgcn_sqrtf(v[i]);
    p[i] = p[i] * h.keep - h.rate * m[i] * __builtin_amdgcn_rcpf(s * h.root + a.eps);
    if constexpr (BITS == 8) v[i] = s;
  }
  if constexpr (BITS == 32) {
    store8<float, FULL>((float*)t.m + at, n, m);
    store8<float, FULL>((float*)t.v + at, n, v);
  } else {
    uint8_t mc[8], vc[8];
    float ms, vs;
    if constexpr (!FULL) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= n) m[i] = v[i] = 0.f;                    // nothing there: no part of the scale
    }
    to_e4m3<true, 0>(m, word, mc, &ms);
    to_e4m3<false, 16>(v, word, vc, &vs);
    store8<uint8_t, FULL>((uint8_t*)t.m + at, n, mc);
    store8<uint8_t, FULL>((uint8_t*)t.v + at, n, vc);
    if (n > 0 && (threadIdx.x & 15) == 0) {
      t.ms[at / MOE_ADAMW_BLOCK] = ms;
      t.vs[at / MOE_ADAMW_BLOCK] = vs;
    }
  }
  if (t.p32) {
    store8<float, FULL>((float*)t.p + at, n, p);
    return;
  }
  uint16_t o[8];
  if (t.master) {
    store8<float, FULL>(t.master + at, n, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = f2bf(p[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = (uint16_t)((__float_as_uint(p[i]) + (word[i] * kRoot3 >> 16)) >> 16);
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) odd |= !(fabsf(p[i]) < INFINITY);
    if (__any(odd)) {                                     // adding to NaN's or infinity's word
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(fabsf(p[i]) < INFINITY)) o[i] = f2bf(p[i]);
    }
  }
  store8<uint16_t, FULL>((uint16_t*)t.p + at, n, o);
}

template <int BITS>
__global__ __launch_bounds__(kAdamThreads, 4) void k_adamw(AdamArgs a) {
  __shared__ float hyper[2];
  const int tid = threadIdx.x;
  const int step = a.step_dev ? *a.step_dev : a.step;
  if (tid < 2) hyper[tid] = bias(tid ? a.log_beta2 : a.log_beta1, step);
  __syncthreads();
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const AdamRates h{lr / hyper[0], 1.f / sqrtf(hyper[1]), 1.f - lr * a.wd,
                    a.grad_scale ? *a.grad_scale : 1.f};
  AdamTensor t{};
  uint32_t begin = 0, end = 0, key = 0;                   // the tensor's items
  for (uint32_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    if (item >= end) {
      const int j = __builtin_amdgcn_readfirstlane(tensor_of(a.first, a.tensors, item));
      t = a.t[j];
      begin = a.first[j];
      end = a.first[j + 1];
      key = mix(a.seed + (uint32_t)step * kGold + (uint32_t)j * kRoot3);
    }
    const int64_t base = (int64_t)(item - begin) * kAdamItem;
    if (t.vec && t.n - base >= kAdamItem) {
#pragma unroll 1
      for (int o = tid * 8; o < kAdamItem; o += kAdamThreads * 8)
        adam8<BITS, true>(a, t, h, key, base + o, 8);
    } else {
#pragma unroll 1
      for (int o = tid * 8; o < kAdamItem; o += kAdamThreads * 8) {
        const int64_t left = t.n - base - o;
        adam8<BITS, false>(a, t, h, key, base + o, left >= 8 ? 8 : left > 0 ? (int)left : 0);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int launch_adamw_table(const moe_adamw_tensor* t, int count, int bits, uint32_t* items, void* ws,
                       hipStream_t st) {
  const AdamTable tab = adamw_table(ws, count);
  uint32_t total = 0;
  for (int base = 0; base < count; base += kAdamPart) {
    AdamPart part{};
    const int n = std::min(kAdamPart, count - base);
    for (int i = 0; i < n; ++i) {
      const moe_adamw_tensor& s = t[base + i];
      AdamTensor& d = part.t[i];
      d.p = s.p; d.master = s.master; d.g = s.g; d.m = s.m; d.v = s.v;
      d.ms = s.m_scale; d.vs = s.v_scale; d.n = s.n;
      d.p32 = s.p_dtype == MOE_F32; d.g32 = s.g_dtype == MOE_F32;
      // 16-byte pieces; codes come 8 bytes at a time
      const uintptr_t all = (uintptr_t)s.p | (uintptr_t)s.g | (uintptr_t)s.master |
                            (bits == 8 ? ((uintptr_t)s.m | (uintptr_t)s.v) << 1
                                       : (uintptr_t)s.m | (uintptr_t)s.v);
      d.vec = (all & 15u) == 0;
      part.first[i] = total;
      total += (uint32_t)((s.n + kAdamItem - 1) / kAdamItem);
    }
    part.first[n] = total;
    hipLaunchKernelGGL(k_adamw_table, dim3(1), dim3(64), 0, st, part, base, n, tab.t, tab.first);
  }
  *items = total;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adamw(const moe_adamw_list& l, const moe_adamw_hyper& h, hipStream_t st) {
  if (l.items == 0) return MOE_OK;
  const AdamTable tab = adamw_table(l.table, l.tensors);
  AdamArgs a{};
  a.t = tab.t; a.first = tab.first; a.tensors = l.tensors; a.items = l.items;
  a.lr = (float)h.lr; a.eps = (float)h.eps; a.wd = (float)h.weight_decay;
  a.beta1 = (float)h.beta1; a.c1 = (float)(1.0 - h.beta1); a.log_beta1 = std::log(h.beta1);
  a.beta2 = (float)h.beta2; a.c2 = (float)(1.0 - h.beta2); a.log_beta2 = std::log(h.beta2);
  a.step = h.step; a.seed = h.seed;
  a.step_dev = h.step_dev; a.lr_dev = h.lr_dev; a.grad_scale = h.grad_scale;
  const dim3 grid(std::min<uint32_t>(l.items, 256 * 8));
  if (l.state_bits == 8) hipLaunchKernelGGL(k_adamw<8>, grid, dim3(kAdamThreads), 0, st, a);
  else hipLaunchKernelGGL(k_adamw<32>, grid, dim3(kAdamThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
