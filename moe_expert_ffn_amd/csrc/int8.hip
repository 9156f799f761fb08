// 8-bit integer rows, and the expert layer's products on them where experts have few rows.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm.h"
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

// The nearest whole number to 127 v / amax, half to even, of the real numbers: c is within one of it, and
// what is left of 127 v after c amax says which of the three it is.  A bf16 v has 8 bits, c amax 15, and c
// is 0 where v is far below amax, so in fp32 the rest is exact.
MOE_DEV int code_of(uint16_t, float v, float inv, float amax) {
  const float c = rintf(v * inv), rest = __builtin_fmaf(-c, amax, v * 127.f), half = 0.5f * amax;
  const int n = (int)c;
  const bool off = fabsf(rest) > half || (fabsf(rest) == half && (n & 1));
  return n + (off ? (rest > 0.f ? 1 : -1) : 0);
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
template <typename T, int NT, int KC>
__global__ __launch_bounds__(256) void k_quant_i8(QuantI8 a) {
  constexpr int RPW = 256 / NT;
  __shared__ uint32_t red[4];
  const int li = threadIdx.x % NT;
  size_t rows = a.rows;
  if (a.blocks) rows = min(rows, (size_t)*a.blocks * a.beta);
  for (size_t r = (size_t)blockIdx.x * RPW + threadIdx.x / NT; r < rows; r += (size_t)gridDim.x * RPW) {
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
    most = group_all<64>(most, OpMax());
    if constexpr (NT > 64) {
      __syncthreads();                                   // the row before has been read
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
      __syncthreads();
      most = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    // NaN and infinity: a scale of NaN, codes of 0; magnitudes below 2^-100: zeros
    const bool finite = most < 0x7F800000u;
    float amax = finite && most >= __float_as_uint(0x1p-100f) ? __uint_as_float(most) : 0.f;
    const float scale = finite ? amax / 127.f : __builtin_nanf("");
    const float down = amax >= 0x1p64f ? 0x1p-64f : 1.f; // so that 127 v stays in range
    amax *= down;
    const float inv = amax > 0.f ? 127.f / amax : 0.f;
    auto write = [&](int c, const T* v) {
      uint32_t w[2] = {0u, 0u};
      if (amax > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i / 4] |= (uint32_t)(code_of(T{}, elem_f(v[i]) * down, inv, amax) & 0xFF) << 8 * (i % 4);
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

static void launch_quant(const QuantI8& a, int dtype, hipStream_t st) {
  if (a.rows == 0) return;
  auto go = [&](auto kernel, int rpw) {
    const size_t all = ((size_t)a.rows + rpw - 1) / rpw;
    // slots: one resident round, whatever their capacity
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<size_t>(all, a.blocks ? 2048 : 1 << 23)), dim3(256), 0, st, a);
  };
  const bool wave = a.cols <= 64 * 8 * 4;
  if (dtype == MOE_F32) wave ? go(k_quant_i8<float, 64, 4>, 4) : go(k_quant_i8<float, 256, 4>, 1);
  else wave ? go(k_quant_i8<uint16_t, 64, 4>, 4) : go(k_quant_i8<uint16_t, 256, 4>, 1);
}
int launch_quant_int8_rows(const void* src, int ld, int dtype, int rows, int cols, int8_t* codes, float* scales,
                           hipStream_t st) {
  QuantI8 a{};
  a.src = src; a.ld = (size_t)ld; a.rows = rows; a.cols = cols; a.codes = codes; a.scales = scales;
  launch_quant(a, dtype, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
// Read no error: they are launches of moe_forward, whose last check sees them all.
void launch_quant_int8_tokens(const void* x, int T, int d, const int32_t* row_to_slot, int k, int8_t* codes,
                              float* slot_scale, hipStream_t st) {
  QuantI8 a{};
  a.src = x; a.ld = (size_t)d; a.rows = T; a.cols = d; a.codes = codes; a.scales = slot_scale;
  a.row_to_slot = row_to_slot; a.k = k;
  launch_quant(a, MOE_BF16, st);
}
void launch_quant_int8_slots(const void* rows, int slots, int dff, const int32_t* slot_to_row, const int32_t* blocks,
                             int beta, int8_t* codes, float* gates, hipStream_t st) {
  QuantI8 a{};
  a.src = rows; a.ld = (size_t)dff; a.rows = slots; a.cols = dff; a.codes = codes; a.scales = gates;
  a.slot_to_row = slot_to_row; a.blocks = blocks; a.beta = beta;
  launch_quant(a, MOE_BF16, st);
}

// ---- products of few rows ----------------------------------------------------------
// An item is a tile of up to 64 rows of one expert and 32 of its weight rows (FC1: 16 of G and the 16 of U).
// The four waves split K in chunks of 64 and read the weights straight into the fragments of
// v_mfma_i32_16x16x64_i8, 16 rows of 64 bytes a load; the rows' codes, which few items share, come out of
// the caches the same way.  The waves' sums are joined in LDS.  Lane l of a fragment holds row l % 16, codes
// 16 (l / 16) to + 15 of the chunk; with the weights first, lane l of a product holds weight rows 4 (l / 16)
// to + 3 of row l % 16.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
struct FewI8 {
  const int8_t* codes;       // FC1: [T][K] by token, FC2: [slots][K]
  const int8_t* w;           // [E][weight rows][K]
  const float* w_scale;      // [E][weight rows]
  const float* slot_scale;   // FC2: with the gate
  const int32_t* slot_to_row;
  uint16_t* out;             // [slots][N]
  const int4* mt;
  const int32_t* mt_cnt;
  int max_mt, P, k, K, N;
};

template <bool FC1, int MB>
MOE_DEV void few_item(const FewI8& a, int4 m, int slab, i32x4_t (*red)[2][4][64]) {
  constexpr int U = MB == 1 ? 8 : MB == 2 ? 4 : 2;       // chunks on their way
  const int lane = threadIdx.x & 63, wave = wave_id(), r16 = lane & 15, quad = lane >> 4;
  const int e = m.x, slot0 = m.y, nrows = m.z, chunks = a.K / 64;
  const size_t wrows = FC1 ? 2 * (size_t)a.N : (size_t)a.N;
  const int first = FC1 ? slab * 16 : slab * 32, second = FC1 ? a.N + first : first + 16;
  const int8_t* w0 = a.w + ((size_t)e * wrows + first + r16) * a.K + quad * 16;
  const int8_t* w1 = a.w + ((size_t)e * wrows + second + r16) * a.K + quad * 16;
  const int8_t* x[MB];
  i32x4_t acc[2][MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int slot = slot0 + min(b * 16 + r16, nrows - 1);             // rows past the tile's: the last again
    x[b] = a.codes + (size_t)(FC1 ? a.slot_to_row[slot] / a.k : slot) * a.K + quad * 16;
    acc[0][b] = acc[1][b] = i32x4_t{0, 0, 0, 0};
  }
  auto load = [](const int8_t* p, int c) {
    return __builtin_bit_cast(i32x4_t, *(const MOE_GLB u32x4_t*)(p + (size_t)c * 64));
  };
  for (int c0 = wave; c0 < chunks; c0 += 4 * U) {
    i32x4_t f0[U], f1[U], fx[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = min(c0 + 4 * u, chunks - 1);
      f0[u] = load(w0, c);
      f1[u] = load(w1, c);
#pragma unroll
      for (int b = 0; b < MB; ++b) fx[u][b] = load(x[b], c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + 4 * u >= chunks) break;                   // the whole wave
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        acc[0][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f0[u], fx[u][b], acc[0][b], 0, 0, 0);
        acc[1][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f1[u], fx[u][b], acc[1][b], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int t = 0; t < 2; ++t) red[wave][t][b][r16 * 4 + quad] = acc[t][b];
  __syncthreads();
  // four outputs of a row each: MB * 64 pieces of every 16 columns
  for (int q = threadIdx.x; q < MB * 64 * (FC1 ? 1 : 2); q += 256) {
    const int t = FC1 ? 0 : q / (MB * 64), p = q % (MB * 64), row = p / 4, col = (p & 3) * 4;
    if (row >= nrows) continue;
    auto sum = [&](int t) {
      const int b = p / 64, at = p % 64;
      return red[0][t][b][at] + red[1][t][b][at] + red[2][t][b][at] + red[3][t][b][at];
    };
    const float* ws = a.w_scale + (size_t)e * wrows;
    const float rs = a.slot_scale[slot0 + row];
    float v[4];
    if constexpr (FC1) {
      const i32x4_t g4 = sum(0), u4 = sum(1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = (float)g4[i] * ws[first + col + i] * rs, u = (float)u4[i] * ws[second + col + i] * rs;
        v[i] = g * __builtin_amdgcn_rcpf(1.f + __expf(-g)) * u;
      }
    } else {
      const i32x4_t o4 = sum(t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (float)o4[i] * ws[first + t * 16 + col + i] * rs;
    }
    uint16_t o[4];
    to_elems<4>(v, o);
    store_n<uint16_t, 4>(a.out + (size_t)(slot0 + row) * a.N + first + t * 16 + col, o);
  }
  __syncthreads();                                       // before the next item's sums
}

template <bool FC1> __global__ __launch_bounds__(256) void k_i8_few(FewI8 a) {
  __shared__ i32x4_t red[4][2][4][64];
  const WorkerSlot w = worker_slot(a.P);
  const int slabs = a.N / (FC1 ? 16 : 32), count = a.mt_cnt[w.r] * slabs;
  for (int idx = w.j; idx < count; idx += w.n) {
    const int4 m = a.mt[(size_t)w.r * a.max_mt + idx / slabs];
    const int slab = idx % slabs;
    if (m.z <= 16) few_item<FC1, 1>(a, m, slab, red);
    else if (m.z <= 32) few_item<FC1, 2>(a, m, slab, red);
    else if (m.z <= 48) few_item<FC1, 3>(a, m, slab, red);
    else few_item<FC1, 4>(a, m, slab, red);
  }
}

void launch_i8_few(bool fc1, const int8_t* codes, const int8_t* w, const float* w_scale, const float* slot_scale,
                   const int32_t* slot_to_row, void* out, const int4* mt, const int32_t* mt_cnt, int max_mt, int P, int k,
                   int K, int N, size_t rows, hipStream_t st) {
  FewI8 a{codes, w, w_scale, slot_scale, slot_to_row, (uint16_t*)out, mt, mt_cnt, max_mt, P, k, K, N};
  // a tile has a row at least; two resident rounds of workgroups take what there is
  const size_t tiles = std::min(rows, (size_t)P * max_mt), items = tiles * (N / (fc1 ? 16 : 32));
  const unsigned grid = (unsigned)((std::min<size_t>(std::max<size_t>(items * P, 1), 2048) + kXcds - 1) / kXcds * kXcds);
  if (fc1) hipLaunchKernelGGL(k_i8_few<true>, dim3(grid), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_i8_few<false>, dim3(grid), dim3(256), 0, st, a);
}

}  // namespace moe
