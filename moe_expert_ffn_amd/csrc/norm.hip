// Root-mean-square norms before and after a block, with its gate and residual
// scale, and their gradients.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "lanes.h"

namespace moe {

struct NormArgs {
  const void* x;       // before the block: the stream; after: the stream.  backward: r or y
  const void* u;       // before: what the stream takes up (nullable); after: y
  const void* w;
  const float* gate;
  const uint8_t* mask; // rows that are not padding (nullable: all)
  const void* go;      // backward: the gradient of the output
  const void* gr;      // backward: what reaches r from elsewhere (nullable)
  void* r;             // forward: the updated stream (nullable).  backward: du
  void* n;             // forward: the output.  backward: dx or dy
  float* rstd;
  float* dgate;
  float* part_w;       // [workgroups][d] sums of dw, or dw itself with one workgroup
  float* part_g;
  size_t ldx, ldu, ldgo, ldgr, ldr, ldn;
  int T, d, w32, kind;
  int row0;            // forward: the launch's first row
  float alpha, eps, inv_d;
};

template <typename T, int VE> MOE_DEV void settle_f(int c, int d, T* raw, float* v) {
  settle_piece<T, VE>(c, d, raw);
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = elem_f(raw[i]);
}
template <typename T, int VE> MOE_DEV void load_f(const T* row, int c, int d, float* v) {
  T raw[VE];
  load_piece<T, VE>(row, c, d, raw);
  settle_f<T, VE>(c, d, raw, v);
}
template <typename T, int VE> MOE_DEV void store_f(T* row, int c, int d, const float* v) {
  T raw[VE];
  to_elems<VE>(v, raw);
  store_upto<T, VE>(row + c, d - c, raw);
}
template <typename T, int VE> MOE_DEV void load_w(const NormArgs& a, int c, float* v) {
  if (a.w32) load_f<float, VE>((const float*)a.w, c, a.d, v);
  else load_f<T, VE>((const T*)a.w, c, a.d, v);
}
// the gate of the columns from c on (1 where it is not the features')
template <int VE> MOE_DEV void load_g(const NormArgs& a, int c, float* v) {
  if (a.kind == MOE_GATE_FEATURE) {
    load_f<float, VE>(a.gate, c, a.d, v);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = 1.f;
  }
}

// Forward workgroups: several rows of up to a wave, or one row of NT threads.
template <int NT> struct RowsOf {
  static constexpr int WG = NT <= 64 ? 256 : NT, RPW = WG / NT;
};
// Sum over the NT threads of a row, once.
template <int NT> MOE_DEV float row_sum(float s, float* red) {
  s = group_all<(NT < 64 ? NT : 64)>(s, OpAdd());
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += red[i];
  }
  return s;
}

// NT threads take a row, KC pieces of VE elements each, which stay in
// registers between the sum and the output: every row is read once.  Bound by
// HBM: after the block 8192 x 2048 bf16 100.7 MB in 20 us (5 TB/s, a 1 GiB copy's
// rate), before it with the residual 4096 x 7168 235 MB in 38 us (6.2 TB/s); one token
// of 7168 takes 2.8 us, the launch's latency and one row's.
template <typename T, int VE, int NT, int KC, bool OUT>
__global__ __launch_bounds__(RowsOf<NT>::WG) void k_norm(NormArgs a) {
  constexpr int RPW = RowsOf<NT>::RPW;
  __shared__ float red[16];
  const int li = threadIdx.x % NT;
  const size_t t = a.row0 + (size_t)blockIdx.x * RPW + threadIdx.x / NT;
  if (t >= (size_t)a.T) return;                          // only where a row has no barrier
  const float g_row = a.alpha * (a.kind == MOE_GATE_TOKEN ? a.gate[t] : 1.f);
  const bool live = !a.mask || a.mask[t];                // padding may hold NaN: chosen away, not multiplied
  const T* x = (const T*)a.x + t * a.ldx;
  const T* u = (const T*)a.u + t * a.ldu;
  // before the block: x and u make v; after: v is u, x is added at the end
  T rx[KC][VE], ru[KC][VE];
#pragma unroll
  for (int q = 0; q < KC; ++q) {
    const int c = (li + q * NT) * VE;
    if (c >= a.d) continue;
    load_piece<T, VE>(x, c, a.d, rx[q]);
    if (OUT || a.u) load_piece<T, VE>(u, c, a.d, ru[q]);
  }
  float v[KC][VE], xs[OUT ? KC : 1][VE];
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < KC; ++q) {
    const int c = (li + q * NT) * VE;
    if (c >= a.d) continue;
    if constexpr (OUT) {
      settle_f<T, VE>(c, a.d, ru[q], v[q]);
      settle_f<T, VE>(c, a.d, rx[q], xs[q]);
    } else {
      settle_f<T, VE>(c, a.d, rx[q], v[q]);
      if (a.u) {
        float uu[VE], g[VE];
        settle_f<T, VE>(c, a.d, ru[q], uu);
        load_g<VE>(a, c, g);
#pragma unroll
        for (int i = 0; i < VE; ++i) v[q][i] += live ? g[i] * g_row * uu[i] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) s += v[q][i] * v[q][i];
  }
  float ws[VE], gs[VE];                                  // on their way during the sum
  if (KC == 1 && li * VE < a.d) {
    load_w<T, VE>(a, li * VE, ws);
    if (OUT) load_g<VE>(a, li * VE, gs);
  }
  s = row_sum<NT>(s, red);
  const float rstd = live ? 1.f / sqrtf(s * a.inv_d + a.eps) : 0.f;
  if (li == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int q = 0; q < KC; ++q) {
    const int c = (li + q * NT) * VE;
    if (c >= a.d) continue;
    float w[VE], o[VE];
    if constexpr (KC == 1) __builtin_memcpy(w, ws, sizeof w);
    else load_w<T, VE>(a, c, w);
    if constexpr (OUT) {
      float g[VE];
      if constexpr (KC == 1) __builtin_memcpy(g, gs, sizeof g);
      else load_g<VE>(a, c, g);
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] = xs[q][i] + (live ? g[i] * g_row * (v[q][i] * rstd * w[i]) : 0.f);
    } else {
      if (a.r) store_f<T, VE>((T*)a.r + t * a.ldr, c, a.d, v[q]);
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] = live ? v[q][i] * rstd * w[i] : 0.f;
    }
    store_f<T, VE>((T*)a.n + t * a.ldn, c, a.d, o);
  }
}

// Backward.  A workgroup of 16 waves holds 1024 / NT rows at a time (one where NT is 1024);
// threads keep their columns' sums over the rows in registers (dw, and FEAT: the gate's), joined over
// the rows' groups at the end and over the workgroups by k_norm_cols, so the order of every sum is
// fixed by the grid.  A row's loads are issued before the sum of the row before it is joined.  Bound
// by HBM: before the block 4099 x 7168 bf16 with residual and feature gate 353 MB and 15 MB of partial
// sums in 67 us (5.5 TB/s); after it 1000 x 1023 fp32 5.2 us.  Rows of several pieces a thread (bf16
// above 8192 features, fp32 above 4096) reach 3.7 to 5.4 TB/s at 3000 rows of 8192, 12000 and 16384: x / rms
// and its gradient of every piece stand in registers, of which the variants with FEAT spill some before the
// block (fp32 43, bf16 14; after it fp32 8) and fp32's without it 26.  So does one more, of up to 8 bf16
// features with FEAT before the block (3).
constexpr int kNormWG = 1024;
template <typename T, int VE, int NT, int KC, bool OUT, bool FEAT>
__global__ __launch_bounds__(kNormWG) void k_norm_bwd(NormArgs a) {
  constexpr int RPW = kNormWG / NT, NW = NT / 64;        // NW 0: several rows a wave
  constexpr int J = NT < 64 ? kNormWG / 64 : RPW;        // strands joined through LDS
  constexpr int IN = OUT ? 2 : 4;                        // row operands: x, go and (before) gr, u
  // with several pieces a thread the registers hold one row (four: without gr and u until they are used)
  constexpr bool AHEAD = KC == 1, LATE = KC == 4;
  __shared__ float red[2][NW > 1 ? RPW : 1][16];
  __shared__ float join[J > 1 ? J * VE * NT : 1];
  const int li = threadIdx.x % NT, rg = threadIdx.x / NT;
  // a thread's sums: in registers, with several pieces in LDS (its own places, in 16-byte pieces;
  // in registers they spilled: 3000 x 12000 bf16 191 us)
  extern __shared__ __attribute__((aligned(16))) float sums[];
  float dw[VE], dg[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) dw[i] = dg[i] = 0.f;
  auto sum_at = [&](int h, int q, int i) { return sums + (((h * KC + q) * VE + i) / 4 * kNormWG + (int)threadIdx.x) * 4; };
  auto add_to = [&](int h, int q, const float* more) {
    if constexpr (KC == 1) {
#pragma unroll
      for (int i = 0; i < VE; ++i) (h ? dg : dw)[i] += more[i];
    } else {
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        float4* at = (float4*)sum_at(h, q, i);
        float4 v = *at;
        v.x += more[i]; v.y += more[i + 1]; v.z += more[i + 2]; v.w += more[i + 3];
        *at = v;
      }
    }
  };
  if constexpr (KC > 1)
    for (int q = 0; q < KC * (FEAT ? 2 : 1) * VE; q += 4) *(float4*)sum_at(0, 0, q) = make_float4(0.f, 0.f, 0.f, 0.f);
  float ws[VE], gs[VE];                                  // one piece: w and the gate stay
  if constexpr (KC == 1) {
#pragma unroll
    for (int i = 0; i < VE; ++i) ws[i] = gs[i] = 0.f;
    if (li * VE < a.d) {
      load_w<T, VE>(a, li * VE, ws);
      if constexpr (FEAT) load_g<VE>(a, li * VE, gs);
    }
  }
  auto w_of = [&](int c, float* w) {
    if constexpr (KC == 1) __builtin_memcpy(w, ws, sizeof ws);
    else load_w<T, VE>(a, c, w);
  };
  // alpha times the gate; g_row: alpha (times the token's)
  auto g_of = [&](int c, float g_row, float* g) {
    if constexpr (!FEAT) {
#pragma unroll
      for (int i = 0; i < VE; ++i) g[i] = g_row;
    } else {
      if constexpr (KC == 1) __builtin_memcpy(g, gs, sizeof gs);
      else load_g<VE>(a, c, g);
#pragma unroll
      for (int i = 0; i < VE; ++i) g[i] *= g_row;
    }
  };
  const size_t step = (size_t)gridDim.x * RPW;
  T cur[KC][IN][VE];
  float rstd = 0.f, g_row = a.alpha;
  bool live = true;
  auto fetch_more = [&](size_t t) {
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * VE;
      if (c >= a.d || t >= (size_t)a.T) continue;
      if constexpr (!OUT) {
        if (a.gr) load_piece<T, VE>((const T*)a.gr + t * a.ldgr, c, a.d, cur[q][2]);
        if (a.u) load_piece<T, VE>((const T*)a.u + t * a.ldu, c, a.d, cur[q][3]);
      }
    }
  };
  auto fetch = [&](size_t t) {
    if (t >= (size_t)a.T) return;
    rstd = a.rstd[t];
    if (a.mask) live = a.mask[t];
    if (a.kind == MOE_GATE_TOKEN) g_row = a.alpha * a.gate[t];
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      const int c = (li + q * NT) * VE;
      if (c >= a.d) continue;
      load_piece<T, VE>((const T*)a.x + t * a.ldx, c, a.d, cur[q][0]);
      load_piece<T, VE>((const T*)a.go + t * a.ldgo, c, a.d, cur[q][1]);
    }
    if constexpr (!LATE) fetch_more(t);
  };
  int turn = 0;
  // one barrier: the next sum goes to the other buffer
  auto row_join = [&](float s) {
    s = group_all<(NT < 64 ? NT : 64)>(s, OpAdd());
    if constexpr (NW > 1) {
      float* r = red[turn & 1][rg];
      ++turn;
      if ((threadIdx.x & 63) == 0) r[(threadIdx.x % NT) >> 6] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) s += r[i];
    }
    return s;
  };
  if constexpr (AHEAD) fetch((size_t)blockIdx.x * RPW + rg);
  for (size_t t0 = (size_t)blockIdx.x * RPW; t0 < (size_t)a.T; t0 += step) {
    const size_t t = t0 + rg;
    const bool on = t < (size_t)a.T;
    if constexpr (!AHEAD) fetch(t);
    float xh[KC][VE], p[KC][VE];       // x / rms, and the gradient of that
    float s = 0.f;
    const bool use = on && live;       // padding adds to no sum and its own terms are 0
    if (use) {
#pragma unroll
      for (int q = 0; q < KC; ++q) {
        const int c = (li + q * NT) * VE;
        if (c >= a.d) continue;
        float w[VE], g[VE], xs[VE], os[VE];
        w_of(c, w);
        if constexpr (OUT) g_of(c, g_row, g);
        settle_f<T, VE>(c, a.d, cur[q][0], xs);
        settle_f<T, VE>(c, a.d, cur[q][1], os);
        float mw[VE], mg[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float o = os[i];
          xh[q][i] = xs[i] * rstd;
          float dv = o;
          if constexpr (OUT) {
            dv *= g[i];
            mg[i] = o * (w[i] * xh[q][i]);
          }
          mw[i] = dv * xh[q][i];
          p[q][i] = dv * w[i];
          // after the block, a token's gate: the sum without it, which is also its gradient
          s += (OUT && !FEAT ? o * w[i] : p[q][i]) * xh[q][i];
        }
        add_to(0, q, mw);
        if constexpr (OUT && FEAT) add_to(1, q, mg);
      }
    }
    const float rs = rstd, gr_ = g_row;
    T kept[AHEAD && !OUT ? KC : 1][2][VE];               // gr and u of this row
    if constexpr (AHEAD) {
      if constexpr (!OUT) __builtin_memcpy(kept, &cur[0][2], sizeof kept);
      fetch(t + step);
    }
    auto settle_more = [&](T (*own)[VE], int c) {
      settle_piece<T, VE>(c, a.d, own[0]);
      settle_piece<T, VE>(c, a.d, own[1]);
    };
    if constexpr (AHEAD && !OUT) {
      settle_more(kept[0], li * VE);
    } else if constexpr (!OUT && !LATE) {
#pragma unroll
      for (int q = 0; q < KC; ++q) settle_more(&cur[q][2], (li + q * NT) * VE);
    }
    s = row_join(s);
    if constexpr (LATE && !OUT) {
      fetch_more(t);
#pragma unroll
      for (int q = 0; q < KC; ++q) settle_more(&cur[q][2], (li + q * NT) * VE);
      __syncthreads();
    }
    if constexpr (OUT && !FEAT) {
      if (on && a.kind == MOE_GATE_TOKEN && li == 0) a.dgate[t] = a.alpha * s;
      s *= gr_;
    }
    const float mean = s * a.inv_d;
    float b = 0.f;
    if (on) {
#pragma unroll
      for (int q = 0; q < KC; ++q) {
        const int c = (li + q * NT) * VE;
        if (c >= a.d) continue;
        float dx[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) dx[i] = use ? rs * (p[q][i] - xh[q][i] * mean) : 0.f;
        if constexpr (!OUT) {
          T(*own)[VE] = AHEAD ? kept[AHEAD ? q : 0] : &cur[q][2];
          if (a.gr) {
#pragma unroll
            for (int i = 0; i < VE; ++i) dx[i] += elem_f(own[0][i]);
          }
          if (a.u) {
            float g[VE], du[VE], uu[VE];
            g_of(c, gr_, g);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              du[i] = use ? g[i] * dx[i] : 0.f;
              uu[i] = use ? elem_f(own[1][i]) * dx[i] : 0.f;
              if constexpr (!FEAT) b += uu[i];
            }
            if constexpr (FEAT) add_to(1, q, uu);
            store_f<T, VE>((T*)a.r + t * a.ldr, c, a.d, du);
          }
        }
        store_f<T, VE>((T*)a.n + t * a.ldn, c, a.d, dx);
      }
    }
    if constexpr (!OUT && !FEAT)
      if (a.kind == MOE_GATE_TOKEN) {
        b = row_join(b);
        if (on && li == 0) a.dgate[t] = a.alpha * b;
      }
  }
  const bool alone = gridDim.x == 1;
#pragma unroll
  for (int q = 0; q < KC; ++q) {
    const int c = (li + q * NT) * VE;
#pragma unroll
    for (int h = 0; h < (FEAT ? 2 : 1); ++h) {
      float sum[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) sum[i] = KC > 1 ? sum_at(h, q, i)[i % 4] : h ? dg[i] : dw[i];
      if constexpr (J > 1) {
        if constexpr (NT < 64) {                         // the wave's rows first
#pragma unroll
          for (int i = 0; i < VE; ++i)
#pragma unroll
            for (int o = NT; o < 64; o <<= 1) sum[i] += __shfl_xor(sum[i], o, 64);
        }
        const int strand = NT < 64 ? threadIdx.x >> 6 : rg;
        __syncthreads();
        if (NT >= 64 || (threadIdx.x & 63) < NT) {
#pragma unroll
          for (int i = 0; i < VE; ++i) join[(strand * VE + i) * NT + li] = sum[i];
        }
        __syncthreads();
        if (rg) continue;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          sum[i] = 0.f;
          for (int o = 0; o < J; ++o) sum[i] += join[(o * VE + i) * NT + li];
        }
      }
      if (c >= a.d) continue;
      float* to = (h ? a.part_g : a.part_w) + (size_t)blockIdx.x * a.d + c;
#pragma unroll
      for (int i = 0; i < VE; ++i) sum[i] *= h && alone ? a.alpha : 1.f;
      store_upto<float, VE>(to, a.d - c, sum);
    }
  }
}

// dw (and dgate) from the workgroups' sums: 64 columns a workgroup, 16 strands
// of partial rows joined through LDS; 4.2 us for 256 partials of 2 x 7168.
__global__ __launch_bounds__(1024) void k_norm_cols(const float* __restrict__ part_w,
                                                    const float* __restrict__ part_g, int parts,
                                                    int d, float alpha, float* __restrict__ dw,
                                                    float* __restrict__ dgate) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  const float* part = blockIdx.y ? part_g : part_w;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int b = strand; b < parts; b += 16) s += part[(size_t)b * d + c];
  red[strand][lane] = s;
  __syncthreads();
  if (strand == 0 && c < d) {
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    if (blockIdx.y) dgate[c] = alpha * s;
    else dw[c] = s;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// The backward's workgroups: what every d can use; the partial sums are 2 * d
// floats for each.
constexpr int kNormMaxWG = 256;
static int norm_grid(int T, int rpw) {
  if (T <= 2 * rpw) return 1;          // two rounds of rows cost less than the launch that joins (6.9, 7.4 us)
  return std::max(1, std::min((int)(((long long)T + rpw - 1) / rpw), kNormMaxWG));
}

size_t norm_ws_bytes(int T, int d) {
  return 2 * align_up((size_t)norm_grid(T, 1) * d * sizeof(float));
}

// F::go<T, VE, NT, KC>(args...): NT threads with KC pieces of VE elements each take a row, threads
// before pieces.  Four pieces a thread (a wave, or 256 threads, a row) save the sums' barriers but
// wait for a row alone: before the block in bf16 1 x 7168 5.3 us against 2.9, 1024 x 2048 6.8 against
// 4.2, 8192 x 2048 21.8 against 23.0, 8192 x 7168 92.6 against 88.9; in the backward pass its sums left
// room for one wave a SIMD, 4099 x 7168 160 us against 68.
template <class F, typename T, int VE, typename... A> static void norm_shape(int d, A&&... args) {
  const int pieces = (d + VE - 1) / VE;
  if (pieces <= 1) return F::template go<T, VE, 1, 1>(args...);
  if (pieces <= 2) return F::template go<T, VE, 2, 1>(args...);
  if (pieces <= 4) return F::template go<T, VE, 4, 1>(args...);
  if (pieces <= 8) return F::template go<T, VE, 8, 1>(args...);
  if (pieces <= 16) return F::template go<T, VE, 16, 1>(args...);
  if (pieces <= 32) return F::template go<T, VE, 32, 1>(args...);
  if (pieces <= 64) return F::template go<T, VE, 64, 1>(args...);
  if (pieces <= 128) return F::template go<T, VE, 128, 1>(args...);
  if (pieces <= 256) return F::template go<T, VE, 256, 1>(args...);
  if (pieces <= 512) return F::template go<T, VE, 512, 1>(args...);
  if (pieces <= 1024) return F::template go<T, VE, 1024, 1>(args...);
  if (pieces <= 2048) return F::template go<T, VE, 1024, 2>(args...);
  if constexpr (VE == 4) F::template go<T, VE, 1024, 4>(args...);    // 8 elements: d ends at 2048 pieces
}
template <class F, typename... A> static void norm_kind(int dtype, int d, A&&... args) {
  if (dtype == MOE_F32) norm_shape<F, float, 4>(d, args...);
  else norm_shape<F, uint16_t, 8>(d, args...);
}

struct NormFwd {
  template <typename T, int VE, int NT, int KC>
  static void go(NormArgs a, bool out, hipStream_t st) {
    constexpr int RPW = RowsOf<NT>::RPW, WG = RowsOf<NT>::WG;
    // a launch holds fewer than 2^32 threads: more rows go in several
    constexpr int most = (1 << 30) / WG * RPW;
    for (const int T_ = a.T; ; a.row0 += most) {
      const int rows = std::min(T_ - a.row0, most);
      a.T = a.row0 + rows;
      const dim3 grid((unsigned)((rows + RPW - 1) / RPW));
      if (out) hipLaunchKernelGGL((k_norm<T, VE, NT, KC, true>), grid, dim3(WG), 0, st, a);
      else hipLaunchKernelGGL((k_norm<T, VE, NT, KC, false>), grid, dim3(WG), 0, st, a);
      if (a.T == T_) return;
    }
  }
};

struct NormBwd {
  template <typename T, int VE, int NT, int KC>
  static void go(NormArgs& a, bool out, float* dw, float* dgate, hipStream_t st) {
    constexpr int RPW = kNormWG / NT, WG = kNormWG;
    const int parts = norm_grid(a.T, RPW);
    const bool feat = a.kind == MOE_GATE_FEATURE;
    float* pw = a.part_w;
    float* pg = a.part_g;
    if (parts == 1) {
      a.part_w = dw;
      a.part_g = dgate;
    }
    const size_t lds = KC > 1 ? sizeof(float) * KC * VE * kNormWG * (feat ? 2 : 1) : 0;
    auto launch = [&](auto kernel) {
      if (lds > 48 * 1024)
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)lds);
      hipLaunchKernelGGL(kernel, dim3(parts), dim3(WG), lds, st, a);
    };
    if (out && feat) launch(k_norm_bwd<T, VE, NT, KC, true, true>);
    else if (out) launch(k_norm_bwd<T, VE, NT, KC, true, false>);
    else if (feat) launch(k_norm_bwd<T, VE, NT, KC, false, true>);
    else launch(k_norm_bwd<T, VE, NT, KC, false, false>);
    if (parts > 1)
      hipLaunchKernelGGL(k_norm_cols, dim3((a.d + 63) / 64, feat ? 2 : 1), dim3(1024), 0, st, pw,
                         pg, parts, a.d, a.alpha, dw, dgate);
  }
};

static NormArgs norm_args(const moe_norm& N) {
  NormArgs a{};
  a.w = N.w; a.gate = N.gate; a.mask = N.token_mask; a.T = N.T; a.d = N.d; a.kind = N.gate_kind;
  a.w32 = N.w_dtype == MOE_F32 ? 1 : 0;
  a.alpha = N.alpha; a.eps = N.eps; a.inv_d = 1.f / (float)N.d;
  return a;
}

int launch_norm(const moe_norm& N, bool out, NormRows x, NormRows u, NormRows r, NormRows n,
                float* rstd, hipStream_t st) {
  if (N.T == 0) return MOE_OK;
  NormArgs a = norm_args(N);
  a.x = x.p; a.ldx = (size_t)x.ld; a.u = u.p; a.ldu = (size_t)u.ld;
  a.r = const_cast<void*>(r.p); a.ldr = (size_t)r.ld;
  a.n = const_cast<void*>(n.p); a.ldn = (size_t)n.ld;
  a.rstd = rstd;
  norm_kind<NormFwd>(N.dtype, N.d, a, out, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_norm_bwd(const moe_norm& N, bool out, NormRows dn, NormRows dr, NormRows r, NormRows u,
                    const float* rstd, NormRows dx, NormRows du, float* dw, float* dgate, void* ws,
                    hipStream_t st) {
  NormArgs a = norm_args(N);
  a.go = dn.p; a.ldgo = (size_t)dn.ld; a.gr = dr.p; a.ldgr = (size_t)dr.ld;
  a.x = r.p; a.ldx = (size_t)r.ld; a.u = u.p; a.ldu = (size_t)u.ld;
  a.n = const_cast<void*>(dx.p); a.ldn = (size_t)dx.ld;
  a.r = const_cast<void*>(du.p); a.ldr = (size_t)du.ld;
  a.rstd = const_cast<float*>(rstd);
  a.dgate = dgate;
  a.part_w = (float*)ws;
  a.part_g = (float*)((char*)ws + norm_ws_bytes(N.T, N.d) / 2);
  norm_kind<NormBwd>(N.dtype, N.d, a, out, dw, dgate, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
