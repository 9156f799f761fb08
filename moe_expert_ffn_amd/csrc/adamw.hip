// AdamW over a list of tensors: parameters in fp32 or bf16, states in fp32 or
// in e4m3 codes with block scales.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "lanes.h"

namespace moe {

// The table of a prepared list: the tensors, and the first item of each.  An
// item is a number of consecutive elements of one tensor, a workgroup's unit.
constexpr int kAdamThreads = 256, kAdamVE = 8, kAdamPass = kAdamThreads * kAdamVE;
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
  int p32, g32;
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
  int tensors, item;
  float lr, beta1, beta2, c1, c2, eps, wd;   // c = 1 - beta
  float under_v, under_m;        // 8-bit states: limit of root_under_m, per sqrt(v)'s over m's scale and of m alone
  double log_beta1, log_beta2;   // -infinity for 0; only with step_dev
  float bias1, bias2;            // 1 - beta^step without
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

// Eight elements at p, with FULL all eight, else n (at most eight, zeros past them).
template <typename T, bool FULL> MOE_DEV void load8(const T* p, int n, T* v) {
  if constexpr (FULL) load_n<T, 8>(p, v);
  else load_upto<T, 8>(p, n, v);
}
template <typename T, bool FULL> MOE_DEV void store8(T* p, int n, const T* v) {
  if constexpr (FULL) store_n<T, 8>(p, v);
  else store_upto<T, 8>(p, n, v);
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

// sqrt rounded to nearest: the hardware's is within an ulp, and of s and its two neighbours the
// nearest to the root has s (s - ulp) < x <= s (s + ulp).  (0, infinity and NaN pass: their
// neighbours compare false.)
MOE_DEV float sqrt_nearest(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float dn = __uint_as_float(__float_as_uint(s) - 1u), up = __uint_as_float(__float_as_uint(s) + 1u);
  const float low = __builtin_fmaf(-dn, s, x), high = __builtin_fmaf(-up, s, x);
  return high > 0.f ? up : low <= 0.f ? dn : s;
}

// Roots of eight values, to nearest (or within an ulp).  The hardware's root takes subnormal numbers for
// 0, and the remainders of sqrt_nearest leave fp32's range below 2^-100: such values (gradients below some
// 1e-12) go scaled by 2^64, in a branch of whole waves.
template <bool NEAREST> MOE_DEV void roots(const float* v, float* s) {
  auto root = [](float x) { return NEAREST ? sqrt_nearest(x) : __builtin_amdgcn_sqrtf(x); };
  uint32_t low = __float_as_uint(v[0]);                  // magnitudes order as their words do
#pragma unroll
  for (int i = 1; i < 8; ++i) low = min(low, __float_as_uint(v[i]));
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = root(v[i]);
  if (__any(low < __float_as_uint(0x1p-96f))) {
    asm volatile("");
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v[i] < 0x1p-96f) s[i] = root(v[i] * 0x1p64f) * 0x1p-32f;
  }
}

constexpr uint32_t kInfBits = 0x7F800000u;
MOE_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Eight states of a lane into codes; the 16 lanes of a block share its scale.
// y = |x| * (1 / top * 448) is rounded up with the probability of the part cut off:
// with the code step at y, 2^(exponent - 3) and at least 2^-9, and u the random
// 16 bits plus a half over 2^16, t = y + u * step loses what is below a step.
// In e4m3's normal range those are the low 20 bits of t's word, below it the
// fraction of t * 512; of the two readings b and c the right one is the middle
// one of b, c and 8 (b <= c everywhere, both 8 at 2^-6).  y is at most two ulps
// above 448, which no u carries to the next code, so no clamp is needed.
// Every operation is one fp32 rounding in this order, so that equal states give
// equal codes wherever they are computed so.
// SIGNED: x may be negative.  u: bits SHIFT..SHIFT + 15 of word.
template <bool SIGNED, int SHIFT>
MOE_DEV void to_e4m3(float* x, const uint32_t* word, uint8_t* codes, float* scale) {
#pragma clang fp contract(off)
  uint32_t most = 0;                                     // magnitudes order as their words do
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, SIGNED ? abs_bits(x[i]) : __float_as_uint(x[i]));
  most = group_all<16>(most, OpMax());
  // a value that is not finite stays out of the scale (rare: a branch of whole waves)
  uint32_t nan[2] = {0u, 0u};                            // their codes
  const bool odd = __any(most >= kInfBits);
  if (odd) {
    asm volatile("");                                    // keeps the branch: not worth 40 selects
    most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (abs_bits(x[i]) >= kInfBits) {
        x[i] = 0.f;
        nan[i / 4] |= 0x7Fu << 8 * (i % 4);
      }
      most = max(most, abs_bits(x[i]));
    }
    most = group_all<16>(most, OpMax());
  }
  const float top = __uint_as_float(most) < 0x1p-100f ? 0.f : __uint_as_float(most);
  const float inv = top > 0.f ? 1.f / top * 448.f : 0.f;
  *scale = top * (1.f / 448.f);
  uint32_t code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fabsf(x[i]) * inv;
    const float octave = __uint_as_float(__float_as_uint(fmaxf(y, 0x1p-6f)) & kInfBits);   // 8 steps
    const float u = __builtin_fmaf((float)(uint16_t)(word[i] >> SHIFT), 0x1p-19f, 0x1p-20f);
    const float t = __builtin_fmaf(u, octave, y);
    const int b = (int)(__float_as_uint(t) >> 20) - (120 << 3), c = (int)(t * 512.f);
    code[i] = (uint32_t)max(min(b, c), min(max(b, c), 8));
  }
  uint32_t packed[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t* q = code + 4 * h;
    packed[h] = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
    if constexpr (SIGNED) {                              // the words' top bytes, by pairs
      const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(x[4 * h + 1]), __float_as_uint(x[4 * h]), 0x0c0c0703u);
      const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(x[4 * h + 3]), __float_as_uint(x[4 * h + 2]), 0x07030c0cu);
      packed[h] |= (lo | hi) & 0x80808080u;
    }
    packed[h] |= nan[h];
  }
  __builtin_memcpy(codes, packed, 8);
}

// m and sqrt(v) are rounded by different bits.  Where m comes out as a step and sqrt(v) as 0, the next update
// is m's step over sqrt((1 - beta2) g^2) of a small g: thousands of lr.  So a sqrt(v) of code 0 under an m
// that is not 0 becomes the code 1.  `most` (of the block, in m's code units): what m may be for that.  All
// gradients give |m| <= C sqrt(v) (Cauchy-Schwarz over the two sums' weights), here of less than a step of
// sqrt(v) and taken twice for the rounding of larger codes, and m's own rounding adds up to D of its
// steps, five deviations; an m above is no optimizer's, and its codes stay as they are rounded.
// Four codes in a word, each compared in its byte's upper bit; few waves have a code of 0 at all (looking
// first took 604M elements from 1425 to 1408 us).
MOE_DEV void root_under_m(const AdamArgs& a, const uint8_t* mc, float ms, uint8_t* vc, float vs) {
  constexpr uint32_t kUpper = 0x80808080u, kRest = 0x7F7F7F7Fu;
  uint32_t m[2], v[2];
  __builtin_memcpy(m, mc, 8);
  __builtin_memcpy(v, vc, 8);
  if (!__any(((v[0] + kRest) & (v[1] + kRest) & kUpper) != kUpper)) return;
  const float most = vs > 0.f ? fminf(__builtin_fmaf(a.under_v, vs * __builtin_amdgcn_rcpf(ms), a.under_m), 448.f) : 0.f;
  const int b = (int)(__float_as_uint(most) >> 20) - (120 << 3), c = (int)(most * 512.f);
  const uint32_t least = kUpper | (uint32_t)max(min(b, c), min(max(b, c), 8)) * 0x01010101u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = m[h] & kRest;                     // NaN's code is above every limit
    v[h] |= ((least - w) & (w + kRest) & ~(v[h] + kRest) & kUpper) >> 7;
  }
  __builtin_memcpy(vc, v, 8);
}

// 1 - beta^t, from log(beta) in double: no cancellation at beta near 1
static __host__ __device__ float bias(double log_beta, int t) { return (float)-expm1(log_beta * t); }

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
#pragma clang fp contract(off)
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
  if (a.grad_scale) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= h.gs;
  }
  uint32_t word[8];
  const uint32_t w0 = (uint32_t)at * kGold + key;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    word[i] = mix(w0 + (uint32_t)i * kGold);
    if constexpr (BITS == 8) v[i] *= v[i];
    m[i] = a.beta1 * m[i] + a.c1 * g[i];
    v[i] = a.beta2 * v[i] + a.c2 * (g[i] * g[i]);
  }
  // the update is lr times a number near 1: a reciprocal of 1 ulp, and where its root is not stored
  // a root of 1 ulp
  float s[8];
  roots<BITS == 8>(v, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __builtin_amdgcn_rcpf(__builtin_fmaf(s[i], h.root, a.eps));
    p[i] = __builtin_fmaf(-h.rate * m[i], d, p[i] * h.keep);
    if constexpr (BITS == 8) v[i] = s[i];
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
    root_under_m(a, mc, ms, vc, vs);
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
    to_elems<8>(p, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = (uint16_t)((__float_as_uint(p[i]) + (word[i] * kRoot3 >> 16)) >> 16);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, abs_bits(p[i]));
    if (__any(most >= kInfBits)) {                        // adding to a NaN's word may leave NaN
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (abs_bits(p[i]) >= kInfBits) o[i] = f2bf(p[i]);
    }
  }
  store8<uint16_t, FULL>((uint16_t*)t.p + at, n, o);
}

// One pass over everything a step touches; a workgroup an item.  By the kernel trace, with 32-bit states
// 24 bytes an element, 604M elements in 2.63 ms (5.5 TB/s; a 1 GiB copy reaches 4.96): bound by HBM.  With 8-bit
// states, bf16 parameters and fp32 gradients 12.1 bytes, 1.41 ms (5.2 TB/s), bound by HBM and the VALU
// alike: 78 VALU instructions an element (SQ_INSTS_VALU) are 1.21 ms of the chip at 2.4 GHz, which is why
// codes are converted by hardware, rounded as whole numbers and never divided.  A persistent grid was 8% slower,
// non-temporal accesses 3% faster here but 20% slower where the tensors fit the caches.
template <int BITS>
__global__ __launch_bounds__(kAdamThreads, 4) void k_adamw(AdamArgs a) {
  const int tid = threadIdx.x;
  int step = a.step;
  float b1 = a.bias1, b2 = a.bias2;
  if (a.step_dev) {                                       // a few microseconds of fp64
    __shared__ float hyper[2];
    step = *a.step_dev;
    if (tid < 2) hyper[tid] = bias(tid ? a.log_beta2 : a.log_beta1, step);
    __syncthreads();
    b1 = hyper[0];
    b2 = hyper[1];
  }
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const AdamRates h{lr / b1, 1.f / sqrtf(b2), 1.f - lr * a.wd, a.grad_scale ? *a.grad_scale : 1.f};
  const uint32_t item = blockIdx.x;
  const int j = __builtin_amdgcn_readfirstlane(tensor_of(a.first, a.tensors, item));
  const AdamTensor t = a.t[j];
  const uint32_t key = mix(a.seed + (uint32_t)step * kGold + (uint32_t)j * kRoot3);
  // whole blocks of 128 (a row of 16 lanes) take the wide accesses
#pragma unroll 1
  for (int pass = 0; pass < a.item; pass += kAdamPass) {
    const int64_t at = (int64_t)(item - a.first[j]) * a.item + pass + tid * 8;
    const int64_t left = t.n - at, block = t.n - (at & ~(int64_t)(MOE_ADAMW_BLOCK - 1));
    if (block >= MOE_ADAMW_BLOCK)
      adam8<BITS, true>(a, t, h, key, at, 8);
    else if (block > 0)
      adam8<BITS, false>(a, t, h, key, at, left >= 8 ? 8 : left > 0 ? (int)left : 0);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int launch_adamw_table(const moe_adamw_tensor* t, int count, moe_adamw_list* out, hipStream_t st) {
  const AdamTable tab = adamw_table(out->table, count);
  const int bits = out->state_bits;
  // 32-bit states are bound by HBM at any item; 8-bit ones spend their time in the VALU too, where the
  // search at a workgroup's start shows: 604M elements 1598 us at 2048, 1499 at 8192 (1481 at 16384),
  // 20M 53.3 and 50.1 (52.5); 5M 20.3 at 2048 and 22.3 at 8192, which leaves too few workgroups.
  long long elements = 0;
  for (int i = 0; i < count; ++i) elements += t[i].n;
  out->item = bits == 8 && elements >= 2048ll * 4 * kAdamPass ? 4 * kAdamPass : kAdamPass;
  // an item is a workgroup, and a launch holds fewer than 2^32 threads
  long long all = 0;
  for (int i = 0; i < count; ++i) all += (t[i].n + out->item - 1) / out->item;
  if (all >= (1ll << 32) / kAdamThreads) return MOE_ERR_UNSUPPORTED;
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
      part.first[i] = total;
      total += (uint32_t)((s.n + out->item - 1) / out->item);
    }
    part.first[n] = total;
    hipLaunchKernelGGL(k_adamw_table, dim3(1), dim3(64), 0, st, part, base, n, tab.t, tab.first);
  }
  out->items = total;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adamw(const moe_adamw_list& l, const moe_adamw_hyper& h, hipStream_t st) {
  if (l.items == 0) return MOE_OK;
  const AdamTable tab = adamw_table(l.table, l.tensors);
  AdamArgs a{};
  a.t = tab.t; a.first = tab.first; a.tensors = l.tensors; a.item = l.item;
  a.lr = (float)h.lr; a.eps = (float)h.eps; a.wd = (float)h.weight_decay;
  a.beta1 = (float)h.beta1; a.c1 = (float)(1.0 - h.beta1); a.log_beta1 = std::log(h.beta1);
  a.beta2 = (float)h.beta2; a.c2 = (float)(1.0 - h.beta2); a.log_beta2 = std::log(h.beta2);
  const double b1 = h.beta1, b2 = h.beta2;
  const double C = b1 * b1 < b2 ? (1 - b1) / std::sqrt((1 - b2) * (1 - b1 * b1 / b2)) : HUGE_VAL;
  a.under_v = (float)(2 * C / 512);
  a.under_m = (float)(2.5 / std::sqrt(1 - b1 * b1) / 512);
  a.bias1 = h.step_dev ? 1.f : bias(a.log_beta1, h.step);
  a.bias2 = h.step_dev ? 1.f : bias(a.log_beta2, h.step);
  a.step = h.step; a.seed = h.seed;
  a.step_dev = h.step_dev; a.lr_dev = h.lr_dev; a.grad_scale = h.grad_scale;
  const dim3 grid(l.items);
  if (l.state_bits == 8) hipLaunchKernelGGL(k_adamw<8>, grid, dim3(kAdamThreads), 0, st, a);
  else hipLaunchKernelGGL(k_adamw<32>, grid, dim3(kAdamThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
