// Reductions over groups of lanes and typed row access, for the kernels that
// work on rows of features or experts.
#pragma once

#include "common.h"

namespace moe {

struct OpAdd { template <typename V> MOE_DEV V operator()(V a, V b) const { return a + b; } };
struct OpMax { template <typename V> MOE_DEV V operator()(V a, V b) const { return a > b ? a : b; } };
struct OpMaxF { MOE_DEV float operator()(float a, float b) const { return fmaxf(a, b); } };
struct OpOr { template <typename V> MOE_DEV V operator()(V a, V b) const { return a | b; } };
struct OpMin { template <typename V> MOE_DEV V operator()(V a, V b) const { return a < b ? a : b; } };

// Value of another lane by a DPP control (a register move inside the VALU;
// through LDS a step would cost its latency).  Every lane of the controls used
// here has a source inside its row of 16.
template <int CTRL, typename V> MOE_DEV V dpp_of(V v) {
  static_assert(sizeof(V) == 4, "32-bit values");
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf,
                                                        true));
}

// All lanes of a group of L (a power of two up to 64) aligned lanes receive op over the
// group.  The tree is the same for every lane, so all receive the same bits.
template <int L, typename V, typename Op> MOE_DEV V group_all(V v, Op op) {
  if constexpr (L >= 2) v = op(v, dpp_of<0xB1>(v));      // lane ^ 1 (quad [1, 0, 3, 2])
  if constexpr (L >= 4) v = op(v, dpp_of<0x4E>(v));      // lane ^ 2 (quad [2, 3, 0, 1])
  if constexpr (L >= 8) v = op(v, dpp_of<0x141>(v));     // the other quad (mirror of 8)
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

// Orders a wave's LDS accesses between its lanes: the hardware keeps them in order, the compiler has
// to be told that another lane may have written.
MOE_DEV void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The place in a list of tensors that holds an item: how many of first[1..tensors] are at or below
// it.  64 lanes look at a sorted table of up to 64 * 64 entries in two steps.
MOE_DEV int list_place(const uint32_t* first, int tensors, uint32_t item) {
  const int lane = threadIdx.x & 63;
  const int i1 = (lane + 1) * 64;
  const int blk = __popcll(__ballot(i1 <= tensors && first[min(i1, tensors)] <= item));
  const int i2 = blk * 64 + 1 + lane;
  return blk * 64 + __popcll(__ballot(i2 <= tensors && first[min(i2, tensors)] <= item));
}

MOE_DEV float elem_f(uint16_t h) { return bf2f(h); }
MOE_DEV float elem_f(float f) { return f; }
// N (even) values to the rows' type; bf16 in pairs, one instruction each
template <int N> MOE_DEV void to_elems(const float* v, uint16_t* o) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const bf16x2_t h = __builtin_convertvector(f32x2_t{v[i], v[i + 1]}, bf16x2_t);
    __builtin_memcpy(o + i, &h, 4);
  }
}
template <int N> MOE_DEV void to_elems(const float* v, float* o) { __builtin_memcpy(o, v, sizeof(float) * N); }

// N consecutive elements in 16-byte (8-byte) pieces.  Global memory takes such accesses at any
// element's address, so rows of any stride and views of any offset go the same way.
typedef u32x4_t u32x4_any_t __attribute__((aligned(1)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(1)));
template <typename T, int N> MOE_DEV void load_n(const T* p, T* v) {
  constexpr int BYTES = N * sizeof(T);
  static_assert(BYTES % 16 == 0 || BYTES == 8, "whole pieces");
  if constexpr (BYTES == 8) {
    const u32x2_t w = *(const MOE_GLB u32x2_any_t*)p;
    __builtin_memcpy(v, &w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4_t w = *(const MOE_GLB u32x4_any_t*)((const char*)p + 16 * i);
      __builtin_memcpy((char*)v + 16 * i, &w, 16);
    }
  }
}
template <typename T, int N> MOE_DEV void store_n(T* p, const T* v) {
  constexpr int BYTES = N * sizeof(T);
  if constexpr (BYTES == 8) {
    u32x2_t w;
    __builtin_memcpy(&w, v, 8);
    *(MOE_GLB u32x2_any_t*)p = w;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      u32x4_t w;
      __builtin_memcpy(&w, (const char*)v + 16 * i, 16);
      *(MOE_GLB u32x4_any_t*)((char*)p + 16 * i) = w;
    }
  }
}
// Piece c (its first element) of a row of d elements: N of them, or where the row ends inside the
// piece, after settle_piece, the rest of the row and zeros.  The load itself has no branch on the
// lane: a short piece reads the row's last N elements, and settle_piece moves them down once they
// are used.  (With the short piece loaded one by one in a branch, every further load waited for it:
// 8192 x 2047 took a third longer than 8192 x 2048.)  settle_piece also waits for the load: the
// elements it read belong to another lane, which may write an output over them; call it before the
// barrier (or in the wave) that the outputs come after.
template <typename T, int N> MOE_DEV void load_piece(const T* row, int c, int d, T* v) {
  if (d >= N) {                                          // the whole launch
    load_n<T, N>(row + min(c, d - N), v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = c + i < d ? *(const MOE_GLB T*)(row + c + i) : (T)0;
  }
}
template <typename T, int N> MOE_DEV void settle_piece(int c, int d, T* v) {
  constexpr int W = N * sizeof(T) / 4;
  if (c + N <= d || d < N) return;
  uint32_t w[W];
  __builtin_memcpy(w, v, sizeof w);
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
  const int bytes = min(c + N - d, N) * (int)sizeof(T);  // N: the piece lies behind the row
#pragma unroll
  for (int s = W; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < W; ++i) {                        // ascending: w[i + s] is still the old one
      const uint32_t far = i + s < W ? w[i + s] : 0u;
      w[i] = bytes & 4 * s ? far : w[i];
    }
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t next = i + 1 < W ? w[i + 1] : 0u;
      w[i] = bytes & 2 ? w[i] >> 16 | next << 16 : w[i];
    }
  }
  __builtin_memcpy(v, w, sizeof w);
}
// The first n elements at p, zeros past those.
template <typename T, int N> MOE_DEV void load_upto(const T* p, int n, T* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = i < n ? *(const MOE_GLB T*)(p + i) : (T)0;
}
template <typename T, int N> MOE_DEV void store_upto(T* p, int n, const T* v) {
  if (n >= N) {
    store_n<T, N>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) *(MOE_GLB T*)(p + i) = v[i];
  }
}

// A wave-uniform number that the compiler forgets: its comparisons are made where they are used.  (Kept over
// k_choice's loop of rows as masks, they took 160 scalar registers to VGPRs and back: 65521 x 256 87 us, now 62.)
MOE_DEV int fresh(int v) {
  asm volatile("" : "+s"(v));
  return v;
}
// The same of a lane's number, and so of the addresses and comparisons made of it.
MOE_DEV int fresh_lane(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

}  // namespace moe
