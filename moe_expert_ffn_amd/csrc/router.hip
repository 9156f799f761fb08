// Top-k router with its balance loss, its gradient, and the gate gradients of
// the expert layer.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "lanes.h"

namespace moe {

// A row of E logits lies in a group of L lanes, V consecutive experts each
// (L * V >= E, V a multiple of 8 so that a lane's logits are whole 16-byte
// pieces); a workgroup of four waves holds 256 / L rows at a time.
constexpr int kRouterThreads = 256;
constexpr int kRouterMaxWG = 256;       // workgroups, and so partial sums, of the forward

struct RouterArgs {
  const void* logits;
  const uint8_t* mask;
  const int32_t* ids_in;
  const float* dlogp;
  const int32_t* counts_in;
  const int32_t* live_in;
  const float* dlosses;
  int32_t* ids;
  float* gates;
  int32_t* counts;
  float* psum;
  int32_t* live;
  float* losses;
  int32_t* status;
  void* dlogits;
  float* part_p;       // [workgroups][E] sums of P
  int32_t* part_c;     // [workgroups][E] counts
  float* part_z;       // [workgroups] sums of lse^2
  int32_t* part_n;     // [workgroups] rows routed
  size_t ld, ld_out;
  int T, E, k, renorm, vec, parts;
  float scale;
};

// Order of 32-bit floats as unsigned integers, 0 for what is never chosen
// (-infinity); adding 0 makes -0 the same as 0.
MOE_DEV uint32_t sort_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return l > -INFINITY ? key : 0u;
}
MOE_DEV float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// log of the score: l, or log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|))
template <int SCORE> MOE_DEV float log_score(float l) {
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) return l;
  else return fminf(l, 0.f) - log1pf(expf(-fabsf(l)));
}

// The lane's V logits in fp32 (-infinity past E).
template <typename T, int V>
MOE_DEV void load_logits(const T* row, int c0, int E, bool vec, bool on, float* v) {
  T raw[V];
  if (on && vec && c0 + V <= E) {
    load_n<T, V, true>(row + c0, raw);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = elem_f(raw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = on && c0 + i < E ? elem_f(row[c0 + i]) : -INFINITY;
  }
}

// Whether a row with these logits is routed: no NaN, no +infinity, and one
// logit above -infinity.  *bad: NaN or +infinity.
template <int L, int V> MOE_DEV bool row_live(const float* v, bool* bad) {
  int f = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f |= !(v[i] < INFINITY) ? 2 : 0;                     // NaN compares false
    f |= v[i] > -INFINITY ? 1 : 0;
  }
  f = group_all<L>(f, [](int a, int b) { return a | b; });
  *bad = (f & 2) != 0;
  return f == 1;
}

// softmax of v (-infinity: 0) into e; *top its maximum, *sum the sum of exp(v - top)
template <int L, int V> MOE_DEV void row_softmax(const float* v, float* e, float* top, float* sum) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
  m = group_all<L>(m, OpMaxF());
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    e[i] = expf(v[i] - m);
    s += e[i];
  }
  s = group_all<L>(s, OpAdd());
  *top = m;
  *sum = s;
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] *= inv;
}

MOE_DEV double balance_of(double sum, int E, int k, int n) {
  return n > 0 ? (double)E / k * sum / n / n : 0.0;
}

// Forward.  Each group takes rows in turn; its lanes keep the sums of P of
// their own experts in registers, so the sums' order is fixed by the grid,
// which follows from T and E alone.  One workgroup writes the totals itself;
// more leave partial sums for k_router_totals.
template <typename T, int L, int V, int SCORE>
__global__ __launch_bounds__(kRouterThreads) void k_router(RouterArgs a) {
  constexpr int G = kRouterThreads / L;                  // rows at a time
  constexpr int C = L * V;
  __shared__ float sp[4][C];
  __shared__ int sc[C];
  __shared__ float sz[G];
  __shared__ int sn[G];
  __shared__ double sred[4];
  const int tid = threadIdx.x, li = tid % L, g = tid / L, c0 = li * V;
  for (int i = tid; i < C; i += kRouterThreads) sc[i] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.f;
  float z = 0.f;
  int n = 0;
  const size_t step = (size_t)gridDim.x * G;
  for (size_t t = (size_t)blockIdx.x * G + g; t < (size_t)a.T; t += step) {
    float v[V], p[V];
    const bool on = !a.mask || a.mask[t];
    load_logits<T, V>((const T*)a.logits + t * a.ld, c0, a.E, a.vec, on, v);
    bool bad;
    const bool live = row_live<L, V>(v, &bad);
    int32_t* ids = a.ids + t * a.k;
    float* gates = a.gates + t * a.k;
    if (!live) {                                         // the whole group
      for (int j = li; j < a.k; j += L) {
        ids[j] = -1;
        gates[j] = 0.f;
      }
      if (bad && li == 0) atomicOr(a.status, MOE_DEV_BAD_LOGIT);
      continue;
    }
    float top, sum, ltop, lsum;
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
      row_softmax<L, V>(v, p, &top, &sum);
      ltop = top;
      lsum = sum;
    } else {
      row_softmax<L, V>(v, p, &ltop, &lsum);
      float s[V];
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = log_score<SCORE>(v[i]);
      row_softmax<L, V>(s, p, &top, &sum);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] += p[i];
    const float lse = ltop + logf(lsum);
    z += lse * lse;
    ++n;
    // the k largest: in turn the largest key, then the lowest index that has it
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = sort_key(v[i]);
    constexpr int KQ = (kRouterMaxK + L - 1) / L;          // choices a lane keeps
    float chosen = 0.f, mine[KQ];
    int where[KQ];
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      best = group_all<L>(best, OpMax());
      int at = C;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == best ? c0 + i : at;
      at = group_all<L>(at, OpMin());
      const bool some = best != 0;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = c0 + i == at ? 0u : key[i];
      const float w = some ? expf(log_score<SCORE>(key_value(best)) - top) : 0.f;
      chosen += w;
#pragma unroll
      for (int q = 0; q < KQ; ++q)
        if (j == q * L + li) {
          mine[q] = w;
          where[q] = some ? at : -1;
        }
    }
    float mul = a.scale;
    if (a.renorm) mul /= chosen;
    else if constexpr (SCORE == MOE_SCORE_SOFTMAX) mul /= sum;
    else mul *= expf(top);
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * L + li;
      if (j >= a.k) continue;
      ids[j] = where[q];
      gates[j] = where[q] >= 0 ? mine[q] * mul : 0.f;
      if (where[q] >= 0) atomicAdd(&sc[where[q]], 1);
    }
  }
  // the wave's groups, then the four waves, each in a fixed order
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = psum[i];
#pragma unroll
    for (int o = L; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if ((tid & 63) < L) sp[tid >> 6][c0 + i] = s;
  }
  if (li == 0) {
    sz[g] = z;
    sn[g] = n;
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  double dot = 0.0;
  for (int e = tid; e < a.E; e += kRouterThreads) {
    const float s = sp[0][e] + sp[1][e] + sp[2][e] + sp[3][e];
    const int c = sc[e];
    if (alone) {
      a.psum[e] = s;
      a.counts[e] = c;
      dot += (double)c * s;
    } else {
      a.part_p[(size_t)blockIdx.x * a.E + e] = s;
      a.part_c[(size_t)blockIdx.x * a.E + e] = c;
    }
  }
  if (alone) {
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
    if ((tid & 63) == 0) sred[tid >> 6] = dot;
    __syncthreads();
  }
  if (tid == 0) {
    double zs = 0.0;
    int ns = 0;
    for (int i = 0; i < G; ++i) {
      zs += sz[i];
      ns += sn[i];
    }
    if (alone) {
      a.live[0] = ns;
      a.losses[0] = (float)balance_of(sred[0] + sred[1] + sred[2] + sred[3], a.E, a.k, ns);
      a.losses[1] = ns > 0 ? (float)(zs / ns) : 0.f;
    } else {
      a.part_z[blockIdx.x] = (float)zs;
      a.part_n[blockIdx.x] = ns;
    }
  }
}

// Totals of the workgroups' partial sums, one workgroup: thread (q, e) adds
// every Q-th partial of expert e, LDS joins the Q strands.
constexpr int kTotalThreads = 1024;
__global__ __launch_bounds__(kTotalThreads) void k_router_totals(RouterArgs a) {
  __shared__ float sp[kTotalThreads];
  __shared__ int sc[kTotalThreads];
  __shared__ double sd[kTotalThreads / 64];
  __shared__ double sz[kTotalThreads / 64];
  __shared__ int sn[kTotalThreads / 64];
  const int tid = threadIdx.x, wide = min(a.E, kTotalThreads);
  const int Q = kTotalThreads / wide, q = tid / wide, e = tid % wide;
  float s = 0.f;
  int c = 0;
  if (q < Q)
    for (int b = q; b < a.parts; b += Q) {
      s += a.part_p[(size_t)b * a.E + e];
      c += a.part_c[(size_t)b * a.E + e];
    }
  sp[tid] = s;
  sc[tid] = c;
  double zs = 0.0;
  int ns = 0;
  for (int b = tid; b < a.parts; b += kTotalThreads) {
    zs += a.part_z[b];
    ns += a.part_n[b];
  }
  __syncthreads();
  double dot = 0.0;
  if (tid < wide) {
    for (int i = 1; i < Q; ++i) {
      s += sp[i * wide + e];
      c += sc[i * wide + e];
    }
    a.psum[e] = s;
    a.counts[e] = c;
    dot = (double)c * s;
  }
  for (int o = 32; o > 0; o >>= 1) {
    dot += __shfl_xor(dot, o, 64);
    zs += __shfl_xor(zs, o, 64);
    ns += __shfl_xor(ns, o, 64);
  }
  if ((tid & 63) == 0) {
    sd[tid >> 6] = dot;
    sz[tid >> 6] = zs;
    sn[tid >> 6] = ns;
  }
  __syncthreads();
  if (tid == 0) {
    double d = 0.0, z = 0.0;
    int n = 0;
    for (int i = 0; i < kTotalThreads / 64; ++i) {
      d += sd[i];
      z += sz[i];
      n += sn[i];
    }
    a.live[0] = n;
    a.losses[0] = (float)balance_of(d, a.E, a.k, n);
    a.losses[1] = n > 0 ? (float)(z / n) : 0.f;
  }
}

// Backward: the row's softmax again from its logits (they have to be read for
// it in any case), every term in registers, one pass.
template <typename T, int L, int V, int SCORE>
__global__ __launch_bounds__(kRouterThreads) void k_router_bwd(RouterArgs a) {
  constexpr int G = kRouterThreads / L;
  const int tid = threadIdx.x, li = tid % L, g = tid / L, c0 = li * V;
  const int n = a.live_in[0];
  const float many = (float)max(n, 1);
  const float db = a.dlosses ? a.dlosses[0] : 0.f, dz = a.dlosses ? a.dlosses[1] : 0.f;
  const float zmul = dz * 2.f / many;
  float ge[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    ge[i] = c0 + i < a.E ? (float)a.counts_in[c0 + i] * (db * ((float)a.E / a.k) / many / many) : 0.f;
  const size_t step = (size_t)gridDim.x * G;
  for (size_t t = (size_t)blockIdx.x * G + g; t < (size_t)a.T; t += step) {
    float v[V], p[V], d[V];
    const bool on = !a.mask || a.mask[t];
    load_logits<T, V>((const T*)a.logits + t * a.ld, c0, a.E, a.vec, on, v);
    bool bad;
    const bool live = row_live<L, V>(v, &bad);
    T* out = (T*)a.dlogits + t * a.ld_out;
    T o[V];
    if (live) {                                          // the whole group
      float top, sum, ltop, lsum, share[V];
      if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
        row_softmax<L, V>(v, p, &top, &sum);
        ltop = top;
        lsum = sum;
      } else {
        row_softmax<L, V>(v, share, &ltop, &lsum);
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = log_score<SCORE>(v[i]);
        row_softmax<L, V>(s, p, &top, &sum);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.f;
      float H = 0.f, Q = 0.f, pg = 0.f;
      uint32_t chosen[(V + 31) / 32];
#pragma unroll
      for (int i = 0; i < (V + 31) / 32; ++i) chosen[i] = 0;
      for (int j0 = 0; j0 < a.k; j0 += L) {
        int id = -1;
        float h = 0.f;
        if (j0 + li < a.k) {
          id = a.ids_in[t * a.k + j0 + li];
          if ((uint32_t)id >= (uint32_t)a.E) id = -1;
          if (id >= 0 && a.dlogp) h = a.dlogp[t * a.k + j0 + li];
        }
        H += h;
        for (int j = 0; j < min(L, a.k - j0); ++j) {
          const int src = (tid & 63 & ~(L - 1)) + j;
          const int ij = __shfl(id, src, 64);
          const float hj = __shfl(h, src, 64);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (ij == c0 + i) {
              d[i] += hj;
              chosen[i / 32] |= 1u << (i % 32);
            }
        }
      }
      H = group_all<L>(H, OpAdd());
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Q += chosen[i / 32] >> (i % 32) & 1 ? p[i] : 0.f;
        pg += p[i] * ge[i];
      }
      Q = group_all<L>(Q, OpAdd());
      pg = group_all<L>(pg, OpAdd());
      const float hq = a.renorm ? (Q > 0.f ? H / Q : 0.f)
                                : (SCORE == MOE_SCORE_SOFTMAX ? H : 0.f);
      const float zs = zmul * (ltop + logf(lsum));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool take = !a.renorm || (chosen[i / 32] >> (i % 32) & 1);
        float x = d[i] - (take ? p[i] * hq : 0.f) + p[i] * (ge[i] - pg);
        if constexpr (SCORE == MOE_SCORE_SIGMOID)        // d log sigmoid(l) / dl = sigmoid(-l)
          x = x * (expf(-fmaxf(v[i], 0.f)) / (1.f + expf(-fabsf(v[i])))) + zs * share[i];
        else
          x += zs * p[i];
        elem_set(o[i], x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) elem_set(o[i], 0.f);
    }
    if (a.vec && c0 + V <= a.E) {
      store_n<T, V, true>(out + c0, o);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + i < a.E) out[c0 + i] = o[i];
    }
  }
}

// ---- gate gradients -----------------------------------------------------------
// dlogp[i] = <dU, U> of row i's slot, a dot of two rows' second halves; a
// group of 16 lanes takes a row, 16 bytes a lane at a time.
template <typename T>
__global__ __launch_bounds__(256) void k_gate_grad(const T* __restrict__ z, const T* __restrict__ dz,
                                                   const int32_t* __restrict__ row_to_slot,
                                                   int rows, int slots, int dff,
                                                   float* __restrict__ dlogp) {
  constexpr int VE = 16 / sizeof(T), L = 16;
  const int li = threadIdx.x % L;
  const size_t row = (size_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= (size_t)rows) return;                       // the whole group
  const int slot = row_to_slot[row];
  float s = 0.f;
  if ((uint32_t)slot < (uint32_t)slots) {
    const size_t base = (size_t)slot * 2 * dff + dff;
    for (int c = li * VE; c < dff; c += L * VE) {
      T u[VE], du[VE];
      load_n<T, VE, true>(z + base + c, u);
      load_n<T, VE, true>(dz + base + c, du);
#pragma unroll
      for (int i = 0; i < VE; ++i) s += elem_f(u[i]) * elem_f(du[i]);
    }
  }
  s = group_all<L>(s, OpAdd());
  if (li == 0) dlogp[row] = s;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int router_lanes(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 32 : 64; }

static int router_grid(int T, int E) {
  const int G = kRouterThreads / router_lanes(E);
  return std::max(1, std::min((int)(((long long)T + G - 1) / G), kRouterMaxWG));
}

size_t router_ws_bytes(int T, int E) {
  const size_t wg = (size_t)router_grid(T, E);
  return align_up(wg * E * 4) * 2 + align_up(wg * 4) * 2;
}

template <template <typename, int, int, int> class K, typename T, int SCORE>
static void router_shape(const RouterArgs& a, int grid, hipStream_t st) {
  if (a.E <= 64) K<T, 8, 8, SCORE>::go(a, grid, st);
  else if (a.E <= 128) K<T, 16, 8, SCORE>::go(a, grid, st);
  else if (a.E <= 256) K<T, 32, 8, SCORE>::go(a, grid, st);
  else if (a.E <= 512) K<T, 64, 8, SCORE>::go(a, grid, st);
  else K<T, 64, 16, SCORE>::go(a, grid, st);
}
template <template <typename, int, int, int> class K>
static void router_kind(const moe_router& R, const RouterArgs& a, int grid, hipStream_t st) {
  const bool f32 = R.dtype == MOE_F32, soft = R.score == MOE_SCORE_SOFTMAX;
  if (f32 && soft) router_shape<K, float, MOE_SCORE_SOFTMAX>(a, grid, st);
  else if (f32) router_shape<K, float, MOE_SCORE_SIGMOID>(a, grid, st);
  else if (soft) router_shape<K, uint16_t, MOE_SCORE_SOFTMAX>(a, grid, st);
  else router_shape<K, uint16_t, MOE_SCORE_SIGMOID>(a, grid, st);
}
template <typename T, int L, int V, int SCORE> struct FwdK {
  static void go(const RouterArgs& a, int grid, hipStream_t st) {
    hipLaunchKernelGGL((k_router<T, L, V, SCORE>), dim3(grid), dim3(kRouterThreads), 0, st, a);
  }
};
template <typename T, int L, int V, int SCORE> struct BwdK {
  static void go(const RouterArgs& a, int grid, hipStream_t st) {
    hipLaunchKernelGGL((k_router_bwd<T, L, V, SCORE>), dim3(grid), dim3(kRouterThreads), 0, st, a);
  }
};

static bool rows_aligned(const void* p, size_t ld, size_t elem, int E) {
  return ((uintptr_t)p & 15u) == 0 && (ld * elem) % 16 == 0 && E % 8 == 0;
}

int launch_router(const moe_router& R, const void* logits, int ld, const uint8_t* mask, int T,
                  int32_t* ids, float* gates, int32_t* counts, float* psum, int32_t* live,
                  float* losses, int32_t* status, void* ws, hipStream_t st) {
  RouterArgs a{};
  a.logits = logits; a.ld = (size_t)ld; a.mask = mask; a.T = T; a.E = R.E; a.k = R.k;
  a.renorm = R.renorm; a.scale = R.scale;
  a.ids = ids; a.gates = gates; a.counts = counts; a.psum = psum; a.live = live;
  a.losses = losses; a.status = status;
  a.vec = rows_aligned(logits, a.ld, R.dtype == MOE_F32 ? 4 : 2, R.E);
  const int grid = router_grid(T, R.E);
  char* w = (char*)ws;
  a.part_p = (float*)w;
  a.part_c = (int32_t*)(w += align_up((size_t)grid * R.E * 4));
  a.part_z = (float*)(w += align_up((size_t)grid * R.E * 4));
  a.part_n = (int32_t*)(w += align_up((size_t)grid * 4));
  a.parts = grid;
  router_kind<FwdK>(R, a, grid, st);
  if (grid > 1)
    hipLaunchKernelGGL(k_router_totals, dim3(1), dim3(kTotalThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_router_bwd(const moe_router& R, const void* logits, int ld, const uint8_t* mask, int T,
                      const int32_t* ids, const float* dlogp, const int32_t* counts,
                      const int32_t* live, const float* dlosses, void* dlogits, int ld_out,
                      hipStream_t st) {
  if (T == 0) return MOE_OK;
  RouterArgs a{};
  a.logits = logits; a.ld = (size_t)ld; a.mask = mask; a.T = T; a.E = R.E; a.k = R.k;
  a.renorm = R.renorm; a.scale = R.scale;
  a.ids_in = ids; a.dlogp = dlogp; a.counts_in = counts; a.live_in = live; a.dlosses = dlosses;
  a.dlogits = dlogits; a.ld_out = (size_t)ld_out;
  const size_t eb = R.dtype == MOE_F32 ? 4 : 2;
  a.vec = rows_aligned(logits, a.ld, eb, R.E) && rows_aligned(dlogits, a.ld_out, eb, R.E);
  const int G = kRouterThreads / router_lanes(R.E);
  const int grid = (int)std::min<long long>(((long long)T + G - 1) / G, 256 * 8);
  router_kind<BwdK>(R, a, grid, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_gate_grad(const void* z, const void* dz, int dtype, const int32_t* row_to_slot,
                     int rows, int slots, int dff, float* dlogp, hipStream_t st) {
  if (rows == 0) return MOE_OK;
  const dim3 grid((unsigned)(((size_t)rows + 15) / 16));
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(k_gate_grad<float>, grid, dim3(256), 0, st, (const float*)z,
                       (const float*)dz, row_to_slot, rows, slots, dff, dlogp);
  else
    hipLaunchKernelGGL(k_gate_grad<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)z,
                       (const uint16_t*)dz, row_to_slot, rows, slots, dff, dlogp);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
