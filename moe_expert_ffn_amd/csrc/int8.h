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

// The nearest whole number to 127 v / amax, half to even, of the real numbers: it is m or m + 1 with m the whole
// number below, by what is left of 127 v after m amax.  Where that is near to half of amax it is exact: a bf16 v
// has 8 bits, m amax 15.  (Positive floats order as their words do, so an odd m's half is one below.)
MOE_DEV int code_of(uint16_t, float v, float inv, float amax) {
  const float m = rintf(__builtin_fmaf(v, inv, -0.501f)), rest = __builtin_fmaf(-m, amax, v * 127.f);
  const int n = (int)m;
  return n + (int)(__float_as_uint(rest) + (uint32_t)(n & 1) > __float_as_uint(0.5f * amax));
}
// A 32-bit v is only looked at again, in 64 bits, where v inv, which is off by 127 2^-23, is near to a half.
MOE_DEV int code_of(float, float v, float inv, float amax) {
  const float t = v * inv, c = rintf(t);
  int n = (int)c;
  if (fabsf(fabsf(t - c) - 0.5f) < 0x1p-15f) {
    const double rest = fma(-(double)c, (double)amax, (double)v * 127.0), half = 0.5 * (double)amax;
    if (fabs(rest) > half || (fabs(rest) == half && (n & 1))) n += rest > 0.0 ? 1 : -1;
  }
  return n;
}

// NT threads take a row; its first KC pieces of 8 elements a thread stay in registers between the maximum
// and the codes, further ones are read again.
// WG threads a workgroup, which is number `block` of `blocks`.
template <typename T, int NT, int KC, int WG> MOE_DEV void quant_i8_rows(const QuantI8& a, int block, int blocks) {
  constexpr int RPW = WG / NT;
  __shared__ uint32_t red[WG / 64];
  const int li = threadIdx.x % NT;
  size_t rows = a.rows;
  if (a.blocks) rows = min(rows, (size_t)*a.blocks * a.beta);
  for (size_t r = (size_t)block * RPW + threadIdx.x / NT; r < rows; r += (size_t)blocks * RPW) {
    if (a.slot_to_row && a.slot_to_row[r] < 0) continue;               // the whole row's threads
    const T* src = (const T*)a.src + r * a.ld;
    int8_t* out = a.codes + r * a.cols;
    T raw[KC][8];
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * 8;
      if (c < a.cols) load_piece<T, 8>(src, c, a.cols, raw[q]);
    }
    uint32_t most = 0u;                                  // magnitudes order as their words do
    auto look = [&](int c, T* v) {
      settle_piece<T, 8>(c, a.cols, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(elem_f(v[i])) & 0x7FFFFFFFu);
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
    most = group_all<(NT < 64 ? NT : 64)>(most, OpMax());
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
    const float inv = amax > 0.f ? 127.f / amax : 0.f;
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
        for (int i = 0; i < 8; ++i) n[i] = (uint32_t)code_of(T{}, f[i], inv, amax);
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
