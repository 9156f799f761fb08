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

// n (at most 8) elements at p, zeros past them
template <typename T> MOE_DEV void load8(const T* p, int n, bool vec, T* v) {
  if (vec && n == 8) {
    if constexpr (sizeof(T) == 1) {
      const u32x2_t w = *(const MOE_GLB u32x2_t*)p;
      __builtin_memcpy(v, &w, 8);
    } else {
      load_n<T, 8, true>(p, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? *(const MOE_GLB T*)(p + i) : (T)0;
  }
}
template <typename T> MOE_DEV void store8(T* p, int n, bool vec, const T* v) {
  if (vec && n == 8) {
    if constexpr (sizeof(T) == 1) {
      u32x2_t w;
      __builtin_memcpy(&w, v, 8);
      *(MOE_GLB u32x2_t*)p = w;
    } else {
      store_n<T, 8, true>(p, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) *(MOE_GLB T*)(p + i) = v[i];
  }
}

MOE_DEV float e4m3_value(uint32_t c) { return (c & 0x7F) == 0x7F ? NAN : e4m3_to_f32(c); }

// The e4m3 code of |y| (below 464), rounded up with the probability of the part
// cut off: in units of the code step at y's exponent (2^-9 below the normal
// range) y is q = 8..16 (0..8), and the code is (exponent + 6) * 8 + floor(q + u).
MOE_DEV uint32_t e4m3_random(float y, uint32_t u16) {
  const int ex = min(max((int)(__float_as_uint(y) >> 23) - 127, -6), 8);
  const float q = y * __uint_as_float((uint32_t)(130 - ex) << 23);
  const float u = ((float)u16 + 0.5f) * (1.f / 65536.f);
  return min((uint32_t)((ex + 6) * 8 + (int)floorf(q + u)), 126u);
}

// Eight states of a lane into codes; the 16 lanes of a block share its scale.
MOE_DEV void states_to_e4m3(const float* x, const uint32_t* u16, uint8_t* codes, float* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
  top = group_all<16>(top, OpMaxF());
  if (top < 0x1p-100f) top = 0.f;
  const float inv = top > 0.f ? 448.f / top : 0.f;
  *scale = top * (1.f / 448.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t c = e4m3_random(fabsf(x[i]) * inv, u16[i]);
    c = fabsf(x[i]) < INFINITY ? c : 0x7Fu;
    codes[i] = (uint8_t)(c | (x[i] < 0.f ? 0x80u : 0u));
  }
}

// 1 - beta^t, from log(beta) in double: no cancellation at beta near 1
MOE_DEV float bias(double log_beta, int t) { return (float)-expm1(log_beta * t); }

template <int BITS>
__global__ __launch_bounds__(kAdamThreads) void k_adamw(AdamArgs a) {
  __shared__ float hyper[4];
  const int tid = threadIdx.x;
  const int step = a.step_dev ? *a.step_dev : a.step;
  if (tid == 0) {
    hyper[0] = bias(a.log_beta1, step);
    hyper[1] = bias(a.log_beta2, step);
  }
  __syncthreads();
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const float rate = lr / hyper[0], root = 1.f / sqrtf(hyper[1]), keep = 1.f - lr * a.wd;
  int j = 0;
  for (uint32_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    while (a.first[j + 1] <= item) ++j;
    const AdamTensor t = a.t[j];
    const uint32_t key = mix(a.seed + (uint32_t)step * kGold + (uint32_t)j * kRoot3);
    const int64_t base = (int64_t)(item - a.first[j]) * kAdamItem;
#pragma unroll 1
    for (int o = tid * 8; o < kAdamItem; o += kAdamThreads * 8) {
      const int64_t at = base + o;
      const int64_t left = t.n - at;
      const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
      const bool vec = t.vec;
      float p[8], g[8], m[8], v[8];
      if (t.master) {
        load8<float>(t.master + at, n, vec, p);
      } else if (t.p32) {
        load8<float>((const float*)t.p + at, n, vec, p);
      } else {
        uint16_t h[8];
        load8<uint16_t>((const uint16_t*)t.p + at, n, vec, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = bf2f(h[i]);
      }
      if (t.g32) {
        load8<float>((const float*)t.g + at, n, vec, g);
      } else {
        uint16_t h[8];
        load8<uint16_t>((const uint16_t*)t.g + at, n, vec, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = bf2f(h[i]);
      }
      if constexpr (BITS == 32) {
        load8<float>((const float*)t.m + at, n, vec, m);
        load8<float>((const float*)t.v + at, n, vec, v);
      } else {
        uint8_t mc[8], vc[8];
        load8<uint8_t>((const uint8_t*)t.m + at, n, vec, mc);
        load8<uint8_t>((const uint8_t*)t.v + at, n, vec, vc);
        const float ms = n > 0 ? t.ms[at / MOE_ADAMW_BLOCK] : 0.f;
        const float vs = n > 0 ? t.vs[at / MOE_ADAMW_BLOCK] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[i] = e4m3_value(mc[i]) * ms;
          const float s = e4m3_value(vc[i]) * vs;
          v[i] = s * s;
        }
      }
      uint32_t word[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        word[i] = mix((uint32_t)(at + i) * kGold + key);
        g[i] *= gs;
        m[i] = a.beta1 * m[i] + a.c1 * g[i];
        v[i] = a.beta2 * v[i] + a.c2 * (g[i] * g[i]);
        const float s = sqrtf(v[i]);
        p[i] = p[i] * keep - rate * m[i] / (s * root + a.eps);
        if constexpr (BITS == 8) v[i] = s;
      }
      if constexpr (BITS == 32) {
        store8<float>((float*)t.m + at, n, vec, m);
        store8<float>((float*)t.v + at, n, vec, v);
      } else {
        uint8_t mc[8], vc[8];
        uint32_t lo[8], hi[8];
        float ms, vs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = word[i] & 0xFFFF;
          hi[i] = word[i] >> 16;
          if (i >= n) m[i] = v[i] = 0.f;                  // nothing there: no part of the scale
        }
        states_to_e4m3(m, lo, mc, &ms);
        states_to_e4m3(v, hi, vc, &vs);
        store8<uint8_t>((uint8_t*)t.m + at, n, vec, mc);
        store8<uint8_t>((uint8_t*)t.v + at, n, vec, vc);
        if (n > 0 && (tid & 15) == 0) {
          t.ms[at / MOE_ADAMW_BLOCK] = ms;
          t.vs[at / MOE_ADAMW_BLOCK] = vs;
        }
      }
      if (t.p32) {
        store8<float>((float*)t.p + at, n, vec, p);
      } else {
        uint16_t h[8];
        if (t.master) {
          store8<float>(t.master + at, n, vec, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = f2bf(p[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(p[i]);
            h[i] = fabsf(p[i]) < INFINITY ? (uint16_t)((b + ((word[i] * kRoot3) >> 16)) >> 16)
                                          : f2bf(p[i]);
          }
        }
        store8<uint16_t>((uint16_t*)t.p + at, n, vec, h);
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
