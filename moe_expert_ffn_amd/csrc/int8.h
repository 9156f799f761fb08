// Rows as 8-bit integers with a scale each: device code of the quantizer, for its own launches and for the
// scheduling launch of an int8 layer.
#pragma once

#include "internal.h"
#include "lanes.h"

namespace moe {

// ---- rows to codes -------------------------------------------------------------
struct QuantI8 {
  const void* src;
  size_t ld;
  int rows, cols;
  int8_t* codes;
  float* scales;             // [rows]; of slots: the gate before, gate times scale after
  // the layer's tokens: their scale to each of their slots as well
  const int32_t* row_to_slot;
  int k;
  // the layer's slots: those in use, by the rows they hold and the blocks' number
  const int32_t* slot_to_row;
  const int32_t* blocks;
  int beta;
};

// The codes of 8 elements, the nearest whole numbers to 127 v / amax, half to even, of the real numbers.
// rate is 127 / amax, in 16 bits and what they leave.  A bf16 v has 8 bits, so v times the 16 is exact and t is
// the real number rounded once, but for the rest's 2^-38.  A real number that is no half is farther from one
// than t 2^-17 (254 V 2^e and an odd number of A 2^f differ by 2^e at least, V and A from 128 to 255), so t lies
// on a half only if it is one; 1.5 2^23 leaves the whole number in the low byte.
struct Rate {
  float whole, hi, lo, amax;
};
MOE_DEV Rate rate_of(float amax) {
  const float inv = 127.f / amax, hi = __uint_as_float(__float_as_uint(inv) & 0xFFFFFF00u);
  return {inv, hi, __builtin_fmaf(-hi, amax, 127.f) * (inv * (1.f / 127.f)), amax};
}
MOE_DEV uint32_t code_of(uint16_t, float v, const Rate& r) {
  return __float_as_uint(__builtin_fmaf(v, r.lo, v * r.hi) + 0x1.8p23f);
}
// A 32-bit v is looked at again, in 64 bits, where v times the rate, which is off by 127 2^-23, is near to a half.
MOE_DEV uint32_t code_of(float, float v, const Rate& r) {
  const float t = v * r.whole, c = rintf(t);
  int n = (int)c;
  if (fabsf(fabsf(t - c) - 0.5f) < 0x1p-15f) {
    const double rest = fma(-(double)c, (double)r.amax, (double)v * 127.0), half = 0.5 * (double)r.amax;
    if (fabs(rest) > half || (fabs(rest) == half && (n & 1))) n += rest > 0.0 ? 1 : -1;
  }
  return (uint32_t)n;
}
// Magnitudes order as their words do: of bf16 two at a time.
struct MostF32 {
  uint32_t m = 0u;
  MOE_DEV void look(const float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  MOE_DEV uint32_t word() const { return m; }
};
struct MostBf16 {
  typedef uint16_t pair_t __attribute__((ext_vector_type(2)));
  pair_t m = {0, 0};
  MOE_DEV void look(const uint16_t* v) {
    uint32_t w[4];
    __builtin_memcpy(w, v, sizeof w);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(pair_t, w[i] & 0x7FFF7FFFu));
  }
  MOE_DEV uint32_t word() const { return (uint32_t)max(m.x, m.y) << 16; }
};

// NT threads take a row; its first KC pieces of 8 elements a thread stay in registers between the maximum
// and the codes, further ones are read again.
// WG threads a workgroup, which is number `block` of `blocks`.  65536 rows of 768 bf16: 151 MB in 34 us
// (4.5 TB/s, some 13 VALU instructions an element).  With short pieces' masks made before the loop, of whose rows a
// lane has one or two, 42, and with codes by comparison as well 45.  196608 rows of 2048 fp32, a layer's weights:
// 2.01 GB in 367 us (5.5 TB/s).
template <typename T, int NT, int KC, int WG> MOE_DEV void quant_i8_rows(const QuantI8& a, int block, int blocks) {
  constexpr int RPW = WG / NT;
  __shared__ uint32_t red[WG / 64];
  const int lane = threadIdx.x % NT;
  size_t rows = a.rows;
  if (a.blocks) rows = min(rows, (size_t)*a.blocks * a.beta);
  for (size_t r = (size_t)block * RPW + threadIdx.x / NT; r < rows; r += (size_t)blocks * RPW) {
    if (a.slot_to_row && a.slot_to_row[r] < 0) continue;               // the whole row's threads
    const int li = fresh_lane(lane);                     // short pieces' masks are made where there are any
    const T* src = (const T*)a.src + r * a.ld;
    int8_t* out = a.codes + r * a.cols;
    T raw[KC][8];
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * 8;
      if (c < a.cols) load_piece<T, 8>(src, c, a.cols, raw[q]);
    }
    std::conditional_t<sizeof(T) == 2, MostBf16, MostF32> seen;
    auto look = [&](int c, T* v) {
      settle_piece<T, 8>(c, a.cols, v);
      seen.look(v);
    };
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * 8;
      if (c < a.cols) look(c, raw[q]);
    }
    for (int c = (li + KC * NT) * 8; c < a.cols; c += NT * 8) {
      T v[8];
      load_piece<T, 8>(src, c, a.cols, v);
      look(c, v);
    }
    uint32_t most = group_all<(NT < 64 ? NT : 64)>(seen.word(), OpMax());
    if constexpr (NT > 64) {
      static_assert(NT == WG, "barriers of whole workgroups");
      __syncthreads();                                   // the row before has been read
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) most = max(most, red[i]);
    }
    // NaN and infinity: a scale of NaN, codes of 0; magnitudes below 2^-100: zeros
    const bool finite = most < 0x7F800000u;
    float amax = finite && most >= __float_as_uint(0x1p-100f) ? __uint_as_float(most) : 0.f;
    const float scale = finite ? amax / 127.f : __builtin_nanf("");
    const bool large = amax >= 0x1p64f;                  // 127 v would leave the range
    if (large) amax *= 0x1p-64f;
    const Rate rate = rate_of(amax > 0.f ? amax : 1.f);
    auto write = [&](int c, const T* v) {
      uint32_t w[2] = {0u, 0u};
      if (amax > 0.f) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = elem_f(v[i]);
        if (large) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= 0x1p-64f;
        }
        uint32_t n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = code_of(T{}, f[i], rate);
#pragma unroll
        for (int q = 0; q < 2; ++q)                      // the low bytes of four
          w[q] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[4 * q + 3], n[4 * q + 2], 0x0c0c0400u),
                                       __builtin_amdgcn_perm(n[4 * q + 1], n[4 * q], 0x0c0c0400u), 0x05040100u);
      }
      int8_t o[8];
      __builtin_memcpy(o, w, 8);
      store_upto<int8_t, 8>(out + c, a.cols - c, o);
    };
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * 8;
      if (c < a.cols) write(c, raw[q]);
    }
    for (int c = (li + KC * NT) * 8; c < a.cols; c += NT * 8) {
      T v[8];
      load_piece<T, 8>(src, c, a.cols, v);
      settle_piece<T, 8>(c, a.cols, v);
      write(c, v);
    }
    if (a.row_to_slot) {
      for (int j = li; j < a.k; j += NT) {
        const int s = a.row_to_slot[r * a.k + j];
        if (s >= 0) a.scales[s] = scale;
      }
    } else if (li == 0) {
      a.scales[r] = a.slot_to_row ? a.scales[r] * scale : scale;
    }
  }
}

// Rows of up to so many columns are a wave's, four pieces a lane, or of half of that half a wave's (768 columns
// are three pieces of 32 lanes: 65536 rows 77 us with 64, of whose second pieces half is empty).
constexpr int kI8WaveCols = 64 * 8 * 4;

}  // namespace moe
