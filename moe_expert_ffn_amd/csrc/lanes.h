// Reductions over groups of lanes and typed row access, for the kernels that
// work on rows of features or experts.
#pragma once

#include "common.h"

namespace moe {

struct OpAdd { template <typename V> MOE_DEV V operator()(V a, V b) const { return a + b; } };
struct OpMax { template <typename V> MOE_DEV V operator()(V a, V b) const { return a > b ? a : b; } };
struct OpMaxF { MOE_DEV float operator()(float a, float b) const { return fmaxf(a, b); } };
struct OpMin { template <typename V> MOE_DEV V operator()(V a, V b) const { return a < b ? a : b; } };

// Value of another lane by a DPP control (a register move inside the VALU;
// through LDS a step would cost its latency).  Every lane of the controls used
// here has a source inside its row of 16.
template <int CTRL, typename V> MOE_DEV V dpp_of(V v) {
  static_assert(sizeof(V) == 4, "32-bit values");
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf,
                                                        true));
}

// All lanes of a group of L (8, 16, 32 or 64) aligned lanes receive op over the
// group.  The tree is the same for every lane, so all receive the same bits.
template <int L, typename V, typename Op> MOE_DEV V group_all(V v, Op op) {
  v = op(v, dpp_of<0xB1>(v));                            // lane ^ 1 (quad [1, 0, 3, 2])
  v = op(v, dpp_of<0x4E>(v));                            // lane ^ 2 (quad [2, 3, 0, 1])
  v = op(v, dpp_of<0x141>(v));                           // the other quad (mirror of 8)
  if constexpr (L >= 16) v = op(v, dpp_of<0x140>(v));    // the other 8 (mirror of 16)
  if constexpr (L >= 32) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);   // rows 0, 1 and 2, 3
    v = op(__builtin_bit_cast(V, (uint32_t)s[0]), __builtin_bit_cast(V, (uint32_t)s[1]));
  }
  if constexpr (L >= 64) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);   // the halves
    v = op(__builtin_bit_cast(V, (uint32_t)s[0]), __builtin_bit_cast(V, (uint32_t)s[1]));
  }
  return v;
}

MOE_DEV float elem_f(uint16_t h) { return bf2f(h); }
MOE_DEV float elem_f(float f) { return f; }
MOE_DEV void elem_set(uint16_t& o, float f) { o = f2bf(f); }
MOE_DEV void elem_set(float& o, float f) { o = f; }

// N consecutive elements: 16-byte accesses where VEC (p 16-byte aligned, N * size a multiple of
// 16), else one by one.
template <typename T, int N, bool VEC> MOE_DEV void load_n(const T* p, T* v) {
  if constexpr (VEC) {
    constexpr int PER = 16 / sizeof(T);
    static_assert(N % PER == 0, "whole 16-byte pieces");
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
      const u32x4_t w = *(const MOE_GLB u32x4_t*)(p + i * PER);
      __builtin_memcpy(v + i * PER, &w, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = *(const MOE_GLB T*)(p + i);
  }
}
template <typename T, int N, bool VEC> MOE_DEV void store_n(T* p, const T* v) {
  if constexpr (VEC) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
      u32x4_t w;
      __builtin_memcpy(&w, v + i * PER, 16);
      *(MOE_GLB u32x4_t*)(p + i * PER) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) *(MOE_GLB T*)(p + i) = v[i];
  }
}

}  // namespace moe
