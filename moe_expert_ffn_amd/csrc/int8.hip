// 8-bit integer rows, and the expert layer's products on them where experts have few rows.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm.h"
#include "int8.h"
#include "internal.h"
#include "lanes.h"

namespace moe {

template <typename T, int NT, int KC> __global__ __launch_bounds__(256) void k_quant_i8(QuantI8 a) {
  quant_i8_rows<T, NT, KC, 256>(a, blockIdx.x, gridDim.x);
}

static void launch_quant(const QuantI8& a, int dtype, hipStream_t st) {
  if (a.rows == 0) return;
  auto go = [&](auto kernel, int rpw) {
    // a launch holds fewer than 2^32 threads; past that the workgroups take further rows
    const size_t all = ((size_t)a.rows + rpw - 1) / rpw;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<size_t>(all, 1 << 23)), dim3(256), 0, st, a);
  };
  const bool wave = a.cols <= kI8WaveCols;
  const bool half = a.cols <= kI8WaveCols / 2;
  if (half) dtype == MOE_F32 ? go(k_quant_i8<float, 32, 4>, 8) : go(k_quant_i8<uint16_t, 32, 4>, 8);
  else if (dtype == MOE_F32) wave ? go(k_quant_i8<float, 64, 4>, 4) : go(k_quant_i8<float, 256, 4>, 1);
  else wave ? go(k_quant_i8<uint16_t, 64, 4>, 4) : go(k_quant_i8<uint16_t, 256, 4>, 1);
}
int launch_quant_int8_rows(const void* src, int ld, int dtype, int rows, int cols, int8_t* codes, float* scales,
                           hipStream_t st) {
  QuantI8 a{};
  a.src = src; a.ld = (size_t)ld; a.rows = rows; a.cols = cols; a.codes = codes; a.scales = scales;
  launch_quant(a, dtype, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
// Reads no error: it is one of the launches of moe_forward, whose last check sees them all.
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
// to + 3 of row l % 16.  Bound by HBM: 512 rows over 125 experts of 2048 x 768, FC1 393 MB of weights in 69 us
// (5.7 TB/s), FC2 197 MB in 45; one token, 25 MB of FC1 in 7 us, the latency of a launch, a read and the join.
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
