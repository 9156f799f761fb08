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
constexpr int kRouterMaxWG = 1024;       // workgroups, and so partial sums, of the forward
constexpr int kTotalThreads = 1024, kTotalCols = 16;
static_assert(kRouterMaxWG <= kTotalThreads, "a thread for every partial of the totals' small sums");
static_assert(kMaxExperts <= 64 * kTotalCols, "a lane for every workgroup of the totals");

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
  float* dots;         // [workgroups of the totals] sums of c_e prob_sum_e
  int32_t* done;       // workgroups of the totals that have written theirs
  size_t ld, ld_out;
  int T, E, k, renorm, parts;
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

// A bf16 logit and its expert as one word, ordered by the logit and then by the lower index; 0 for what
// is never chosen, all others of a row different.
MOE_DEV uint32_t pick_word(float l, int e) {
  const uint32_t key = sort_key(l);
  return key ? (key & 0xFFFF0000u) | (uint32_t)(0xFFFF - e) : 0u;
}
MOE_DEV int pick_expert(uint32_t w) { return 0xFFFF - (int)(w & 0xFFFFu); }
MOE_DEV uint32_t pick_key(uint32_t w) { return w & 0x80000000u ? w & 0xFFFF0000u : w | 0xFFFFu; }

// N words in descending order: Batcher's odd-even merge sort.
template <int N> MOE_DEV void sort_down(uint32_t* k) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int d = p; d >= 1; d >>= 1)
#pragma unroll
      for (int j = d % p; j + d < N; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < N && (i + j) / (2 * p) == (i + j + d) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + d];
            k[i + j] = max(a, b);
            k[i + j + d] = min(a, b);
          }
}

// e^x by the hardware's 2^x: the product's rounding costs |x| 2^-24 relative,
// next to nothing for the experts that carry a row's weight (x near 0).
MOE_DEV float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
MOE_DEV float inverse(float x) { return __builtin_amdgcn_rcpf(x); }   // 1 ulp

// A row on its way: the lane's V logits as stored, and the row's mask.
template <typename T, int V> struct NextRow {
  T raw[V];
  uint8_t on;
  MOE_DEV void fetch(const RouterArgs& a, size_t t, int c0) {
    if (t >= (size_t)a.T) return;
    load_piece<T, V>((const T*)a.logits + t * a.ld, c0, a.E, raw);
    on = a.mask ? a.mask[t] : 1;
  }
};
// The lane's V logits in fp32 (-infinity past E and in a row that is off).
template <typename T, int V>
MOE_DEV void logits_of(const NextRow<T, V>& row, int c0, int E, float* v) {
  T raw[V];
  __builtin_memcpy(raw, row.raw, sizeof raw);
  settle_piece<T, V>(c0, E, raw);
  const int n = row.on ? E - c0 : 0;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = i < n ? elem_f(raw[i]) : -INFINITY;
}

// The row's scores.  w: the scores' exponentials up to a factor of the row,
// sum their sum, so P = w / sum; top the largest logit.  Softmax: w = e^(l - top).
// Sigmoid: with a = e^-|l|, sigmoid(l) is 1 / (1 + a) or a / (1 + a); where even the
// largest logit is negative, a carries the factor e^-top, so that a row whose
// sigmoids all underflow still has its shares: t = e^(-|l| - low), low = min(top, 0),
// w = (l < 0 ? t : 1) / (1 + t e^low), and sigmoid(l) = w e^low.
// A row that is not routed shows in sum and top alone (see row_live).
template <int SCORE> struct Score {
  float top, low, elow;
  MOE_DEV void at_top(float m) {
    top = m;
    low = SCORE == MOE_SCORE_SOFTMAX ? m : fminf(m, 0.f);
    elow = SCORE == MOE_SCORE_SOFTMAX ? 1.f : exp_of(low);
  }
  // *away: sigmoid(-l), the slope of log sigmoid
  MOE_DEV float weight(float l, float* away = nullptr) const {
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
      return exp_of(l - low);
    } else {
      const float t = exp_of(-fabsf(l) - low), a = t * elow, r = inverse(1.f + a);
      if (away) *away = (l < 0.f ? 1.f : a) * r;
      return (l < 0.f ? t : 1.f) * r;
    }
  }
};

template <int L, int V> MOE_DEV float row_top(const float* v) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);        // NaN is passed over
  return group_all<L>(m, OpMaxF());
}

// Whether a row is routed: NaN makes its sum NaN, so does +infinity in a softmax and a row of
// -infinities anywhere (inf - inf).
MOE_DEV bool row_live(float top, float sum) { return top < INFINITY && sum < INFINITY; }

// A lane's scores, e^(l - top) among them, and the row's sum of w.  Sigmoid scores of a row whose
// largest logit is near 0 need no exponential of their own: sigmoid(l) = e / (e + e^-top) with e =
// e^(l - top), sigmoid(-l) = e^-top / (e + e^-top).  (Off by a rounding of l - top and of top instead of
// l's; a share below e^-87 becomes 0.)
constexpr float kNearTop = 16.f;
template <int L, int V, int SCORE, bool AWAY>
MOE_DEV float row_scores(const Score<SCORE>& sc, const float* v, float* w, float* e, float* away) {
  float sum = 0.f;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = e[i] = exp_of(v[i] - sc.top);
      sum += w[i];
    }
  } else if (fabsf(sc.top) <= kNearTop) {                // the whole group
    const float et = exp_of(-sc.top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      e[i] = exp_of(v[i] - sc.top);
      const float r = inverse(e[i] + et);
      w[i] = e[i] * r;
      if constexpr (AWAY) away[i] = et * r;
      sum += w[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      e[i] = exp_of(v[i] - sc.top);
      w[i] = sc.weight(v[i], AWAY ? away + i : nullptr);
      sum += w[i];
    }
  }
  return group_all<L>(sum, OpAdd());
}
template <int L, int V> MOE_DEV float lane_sum(const float* e) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += e[i];
  return group_all<L>(s, OpAdd());
}

MOE_DEV float balance_of(float sum, int E, int k, int n) {
  return n > 0 ? (float)E / (float)k * (sum / (float)n) / (float)n : 0.f;
}

// Sum over a workgroup of `waves` waves, for every thread of the first wave.
MOE_DEV float block_sum(float s, float* red, int waves) {
  s = group_all<64>(s, OpAdd());
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < waves; ++i) s += red[i];
  return s;
}

// Forward.  Each group takes rows in turn; its lanes keep the sums of P of
// their own experts in registers, so the sums' order is fixed by the grid,
// which follows from T and E alone.  One workgroup writes the totals itself;
// more leave partial sums for k_router_totals.  By the kernel trace 16 x 128 bf16, k 8: 3.8 us, the
// latency of one row; 8192 x 128 fp32 6.6 us (4.2 MB, 0.85 us at HBM's rate), 65521 x 256 bf16 28 us (sigmoid
// 31; 33.5 MB), 131072 x 512 fp32 136 us (268 MB): bound by the VALU, which works in 95 to 97% of the busy CUs'
// cycles of the two large ones (SQ_ACTIVE_INST_VALU over SQ_BUSY_CU_CYCLES; 50% at 8192 x 128): some 40
// instructions a choice and wave of two or four rows, 35 a logit of a lane.  The next row is fetched while
// this one is worked on.
template <typename T, int L, int V, int SCORE>
__global__ __launch_bounds__(kRouterThreads) void k_router(RouterArgs a) {
  constexpr int G = kRouterThreads / L;                  // rows at a time
  constexpr int C = L * V;
  constexpr int KQ = (kRouterMaxK + L - 1) / L;          // choices a lane keeps
  __shared__ float sp[4][C];
  __shared__ int sc[C];
  __shared__ float red[2][4];
  __shared__ int redn[4];
  const int tid = threadIdx.x, li = tid % L, g = tid / L, c0 = li * V;
  for (int i = tid; i < C; i += kRouterThreads) sc[i] = 0;
  if (blockIdx.x == 0 && tid == 0 && gridDim.x > 1) *a.done = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.f;
  float z = 0.f;
  int n = 0;
  const size_t step = (size_t)gridDim.x * G;
  NextRow<T, V> next;
  next.fetch(a, (size_t)blockIdx.x * G + g, c0);
  for (size_t t = (size_t)blockIdx.x * G + g; t < (size_t)a.T; t += step) {
    float v[V], w[V];
    logits_of<T, V>(next, c0, a.E, v);
    next.fetch(a, t + step, c0);
    int32_t* ids = a.ids + t * a.k;
    float* gates = a.gates + t * a.k;
    Score<SCORE> sc_;
    sc_.at_top(row_top<L, V>(v));
    float e[V];
    const float sum = row_scores<L, V, SCORE, false>(sc_, v, w, e, nullptr);
    const float lsum = SCORE == MOE_SCORE_SOFTMAX ? sum : lane_sum<L, V>(e);
    if (!row_live(sc_.top, sum)) {                       // the whole group
      for (int j = li; j < a.k; j += L) {
        ids[j] = -1;
        gates[j] = 0.f;
      }
      bool bad = false;
#pragma unroll
      for (int i = 0; i < V; ++i) bad |= !(v[i] < INFINITY);       // NaN or +infinity
      if (bad) atomicOr(a.status, MOE_DEV_BAD_LOGIT);
      continue;
    }
    const float inv = inverse(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] += w[i] * inv;
    const float lse = sc_.top + logf(lsum);
    z += lse * lse;
    ++n;
    // The k largest.  bf16: the lanes' own words in descending order, then in turn the largest of the
    // lanes' first, which leaves its lane's list (30000 x 512, k 10: 40.7 us against 43.1 by the search
    // below).  32 bits, where a word has no room for the index (a double has: 49.8 us against 47.3): in
    // turn the largest key, then the lowest index that has it.
    constexpr bool kWord = sizeof(T) == 2;
    uint32_t key[V], won[KQ];
    int where[KQ];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = kWord ? pick_word(v[i], c0 + i) : sort_key(v[i]);
    if constexpr (kWord) sort_down<V>(key);
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      won[q] = 0;
      where[q] = -1;
    }
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = key[0];
      int at;
      if constexpr (kWord) {
        best = group_all<L>(best, OpMax());
        at = pick_expert(best);
        const bool mine = key[0] == best;
#pragma unroll
        for (int i = 0; i < V; ++i) {                    // values: a choice of elements would index
          const uint32_t here = key[i], next = i + 1 < V ? key[i + 1 < V ? i + 1 : i] : 0u;
          key[i] = mine ? next : here;
        }
      } else {
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        best = group_all<L>(best, OpMax());
        at = C;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) at = key[i] == best ? c0 + i : at;
        at = group_all<L>(at, OpMin());
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = c0 + i == at ? 0u : key[i];
      }
#pragma unroll
      for (int q = 0; q < KQ; ++q)
        if (j == q * L + li) {
          won[q] = best;
          where[q] = best ? at : -1;
        }
    }
    // lane j's choice: its weight again from its logit, which the key holds
    float mine[KQ], chosen = 0.f;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      mine[q] = won[q] ? sc_.weight(key_value(kWord ? pick_key(won[q]) : won[q])) : 0.f;
      chosen += mine[q];
    }
    chosen = group_all<L>(chosen, OpAdd());
    const float mul = a.renorm ? a.scale / chosen
                      : SCORE == MOE_SCORE_SOFTMAX ? a.scale / sum : a.scale * sc_.elow;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * L + li;
      if (j >= a.k) continue;
      ids[j] = where[q];
      gates[j] = mine[q] * mul;
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
  z = li == 0 ? z : 0.f;
  n = li == 0 ? n : 0;
  z = group_all<64>(z, OpAdd());
  n = group_all<64>(n, OpAdd());
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = z;
    redn[tid >> 6] = n;
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  float dot = 0.f;
  for (int e = tid; e < a.E; e += kRouterThreads) {
    const float s = sp[0][e] + sp[1][e] + sp[2][e] + sp[3][e];
    const int c = sc[e];
    if (alone) {
      a.psum[e] = s;
      a.counts[e] = c;
      dot += (float)c * s;
    } else {
      a.part_p[(size_t)blockIdx.x * a.E + e] = s;
      a.part_c[(size_t)blockIdx.x * a.E + e] = c;
    }
  }
  if (alone) dot = block_sum(dot, red[1], 4);
  if (tid == 0) {
    const float zs = red[0][0] + red[0][1] + red[0][2] + red[0][3];
    const int ns = redn[0] + redn[1] + redn[2] + redn[3];
    if (alone) {
      a.live[0] = ns;
      a.losses[0] = balance_of(dot, a.E, a.k, ns);
      a.losses[1] = ns > 0 ? zs / (float)ns : 0.f;
    } else {
      a.part_z[blockIdx.x] = zs;
      a.part_n[blockIdx.x] = ns;
    }
  }
}

// Totals of the workgroups' partial sums.  A workgroup takes 16 experts, 64
// strands of partials joined through LDS; the last one to finish joins their
// products c_e prob_sum_e, in order, into the losses.  3.5-4.5 us at 512 partials
// of 128 experts, latency alone (one workgroup for all: 11 us).
__global__ __launch_bounds__(kTotalThreads) void k_router_totals(RouterArgs a) {
  constexpr int S = kTotalThreads / kTotalCols;
  __shared__ float sp[S][kTotalCols];
  __shared__ int sc[S][kTotalCols];
  __shared__ float red[kTotalThreads / 64];
  __shared__ int redn[kTotalThreads / 64];
  const int tid = threadIdx.x, col = tid % kTotalCols, q = tid / kTotalCols;
  const int e = blockIdx.x * kTotalCols + col;
  float s = 0.f, z = 0.f;
  int c = 0, n = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = q; b < a.parts; b += S) {
      s += a.part_p[(size_t)b * a.E + e];
      c += a.part_c[(size_t)b * a.E + e];
    }
  }
  if (tid < a.parts) {                                   // at most kTotalThreads; only the last uses them
    z = a.part_z[tid];
    n = a.part_n[tid];
  }
  sp[q][col] = s;
  sc[q][col] = c;
  z = group_all<64>(z, OpAdd());
  n = group_all<64>(n, OpAdd());
  if ((tid & 63) == 0) {
    red[tid >> 6] = z;
    redn[tid >> 6] = n;
  }
  __syncthreads();
  if (tid >= 64) return;
  const int cc = tid >> 2, e4 = blockIdx.x * kTotalCols + cc;      // four lanes a column, 16 strands each
  s = 0.f;
  c = 0;
#pragma unroll
  for (int i = 0; i < S; i += 4) {
    s += sp[i + (tid & 3)][cc];
    c += sc[i + (tid & 3)][cc];
  }
  s += dpp_of<0xB1>(s);
  s += dpp_of<0x4E>(s);
  c += dpp_of<0xB1>(c);
  c += dpp_of<0x4E>(c);
  const bool mine = e4 < a.E && (tid & 3) == 0;
  if (mine) {
    a.psum[e4] = s;
    a.counts[e4] = c;
  }
  float dot = group_all<64>(mine ? (float)c * s : 0.f, OpAdd());
  int last = 0;
  if (tid == 0) {
    __hip_atomic_store(a.dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           (int)gridDim.x - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  // at most 1024 / 16 workgroups
  dot = tid < (int)gridDim.x
            ? __hip_atomic_load(a.dots + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
  dot = group_all<64>(dot, OpAdd());
  if (tid == 0) {
    z = 0.f;
    n = 0;
#pragma unroll
    for (int i = 0; i < kTotalThreads / 64; ++i) {
      z += red[i];
      n += redn[i];
    }
    a.live[0] = n;
    a.losses[0] = balance_of(dot, a.E, a.k, n);
    a.losses[1] = n > 0 ? z / (float)n : 0.f;
  }
}

// Backward: the row's scores again from its logits (they have to be read for
// it in any case), every term in registers, one pass.  The k gate gradients
// reach the lanes of their experts through LDS, a row's C places zeroed,
// written and read by the row's own lanes (LDS keeps a wave's order).  By the kernel trace 4096 x 64
// fp32 4.6 us; 65521 x 256 bf16 with both losses 26 us (sigmoid 30; 71 MB, 14 at HBM's rate): the VALU works in
// 77% (83%) of the busy CUs' cycles, the rest is the latency of a row's five sums and its passage through
// LDS; 131072 x 512 fp32 98 us, 5.5 TB/s of 541 MB.  Sigmoid scores with exponentials of their own: 31.4 us
// against 27.8 in replays of a graph; comparing every expert with every choice instead of LDS, and library
// exponentials: 105 us.
template <typename T, int L, int V, int SCORE>
__global__ __launch_bounds__(kRouterThreads) void k_router_bwd(RouterArgs a) {
  constexpr int G = kRouterThreads / L, C = L * V;
  __shared__ __attribute__((aligned(16))) float sh[G][C];
  __shared__ __attribute__((aligned(16))) uint8_t sf[G][C];       // j + 1 of the choice
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
  constexpr int KQ = (kRouterMaxK + L - 1) / L;          // choices a lane holds
  NextRow<T, V> next;
  int id_next[KQ];
  float h_next[KQ];
  auto fetch = [&](size_t t) {
    next.fetch(a, t, c0);
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * L + li;
      id_next[q] = -1;
      h_next[q] = 0.f;
      if (j < a.k && t < (size_t)a.T) {
        id_next[q] = a.ids_in[t * a.k + j];
        if (a.dlogp) h_next[q] = a.dlogp[t * a.k + j];
      }
    }
  };
  fetch((size_t)blockIdx.x * G + g);
  for (size_t t = (size_t)blockIdx.x * G + g; t < (size_t)a.T; t += step) {
    float v[V], w[V], away[V], h[KQ];
    int id[KQ];
    logits_of<T, V>(next, c0, a.E, v);
    __builtin_memcpy(id, id_next, sizeof id);
    __builtin_memcpy(h, h_next, sizeof h);
    fetch(t + step);
    // the choices: lane j's, and through LDS to the experts' lanes
    float d[V], H = 0.f;
    uint8_t flag[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i] = 0.f;
      flag[i] = 0;
    }
    __builtin_memcpy(&sh[g][c0], d, sizeof d);
    __builtin_memcpy(&sf[g][c0], flag, sizeof flag);
    wave_lds_order();
    bool twice = false;
#pragma unroll
    for (int q = 0; q < KQ; ++q)
      if ((uint32_t)id[q] < (uint32_t)a.E) {
        H += h[q];
        sh[g][id[q]] = h[q];
        sf[g][id[q]] = (uint8_t)(q * L + li + 1);
      }
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < KQ; ++q)
      if ((uint32_t)id[q] < (uint32_t)a.E) twice |= sf[g][id[q]] != (uint8_t)(q * L + li + 1);
    if (__any(twice)) {                                  // an expert given twice: its gradients in order
#pragma unroll
      for (int q = 0; q < KQ; ++q)
        if ((uint32_t)id[q] < (uint32_t)a.E) sh[g][id[q]] = 0.f;
      wave_lds_order();
#pragma unroll
      for (int q = 0; q < KQ; ++q)
        for (int j = 0; j < L; ++j) {
          if (li == j && (uint32_t)id[q] < (uint32_t)a.E) sh[g][id[q]] += h[q];
          wave_lds_order();
        }
    }
    __builtin_memcpy(d, &sh[g][c0], sizeof d);
    __builtin_memcpy(flag, &sf[g][c0], sizeof flag);
    wave_lds_order();
    H = group_all<L>(H, OpAdd());

    Score<SCORE> sc;
    sc.at_top(row_top<L, V>(v));
    float e[V];
    const float sum = row_scores<L, V, SCORE, true>(sc, v, w, e, away);
    T* out = (T*)a.dlogits + t * a.ld_out;
    T o[V];
    float x[V];
    if (row_live(sc.top, sum)) {                         // the whole group
      const float inv = inverse(sum);
      float Q = 0.f, pg = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        w[i] *= inv;                                     // P
        Q += flag[i] ? w[i] : 0.f;
        pg += w[i] * ge[i];
      }
      Q = group_all<L>(Q, OpAdd());
      pg = group_all<L>(pg, OpAdd());
      const float hq = a.renorm ? (Q > 0.f ? H / Q : 0.f)
                                : (SCORE == MOE_SCORE_SOFTMAX ? H : 0.f);
      const float rest = a.renorm ? 0.f : hq;            // of the experts not chosen
      float zs = 0.f;
      if (zmul != 0.f) {
        const float lsum = SCORE == MOE_SCORE_SOFTMAX ? sum : lane_sum<L, V>(e);
        zs = zmul * (sc.top + logf(lsum));
        if constexpr (SCORE == MOE_SCORE_SIGMOID) zs *= inverse(lsum);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = d[i] + w[i] * (ge[i] - pg - (flag[i] ? hq : rest));
        if constexpr (SCORE == MOE_SCORE_SIGMOID) {
          x[i] *= away[i];
          if (zmul != 0.f) x[i] += zs * e[i];
        } else {
          x[i] += zs * w[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.f;
    }
    to_elems<V>(x, o);
    store_upto<T, V>(out + c0, a.E - c0, o);
  }
}

// ---- gate gradients -----------------------------------------------------------
// dlogp[i] = <dU, U> of row i's slot, a dot of two rows' second halves; a
// group of 16 lanes takes a row, 16 bytes a lane at a time.  Bound by HBM: the
// Qwen3-shaped batch (65536 rows, d_ff 768, bf16) reads 202 MB in 36.5 us, 5.5 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_gate_grad(const T* __restrict__ z, const T* __restrict__ dz,
                                                   const int32_t* __restrict__ row_to_slot,
                                                   int rows, int slots, int dff,
                                                   float* __restrict__ dlogp) {
  constexpr int VE = 16 / sizeof(T), L = 16;
  const int li = threadIdx.x % L;
  const size_t step = (size_t)gridDim.x * (256 / L);
  for (size_t row = (size_t)blockIdx.x * (256 / L) + threadIdx.x / L; row < (size_t)rows; row += step) {
    const int slot = row_to_slot[row];
    float s = 0.f;
    if ((uint32_t)slot < (uint32_t)slots) {
      const size_t base = (size_t)slot * 2 * dff + dff;
      for (int c = li * VE; c < dff; c += L * VE) {
        T u[VE], du[VE];
        load_n<T, VE>(z + base + c, u);
        load_n<T, VE>(dz + base + c, du);
#pragma unroll
        for (int i = 0; i < VE; ++i) s += elem_f(u[i]) * elem_f(du[i]);
      }
    }
    s = group_all<L>(s, OpAdd());
    if (li == 0) dlogp[row] = s;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int router_lanes(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 32 : 64; }
// Forward with 16 experts a lane instead of 8: twice the rows a wave, so fewer steps across lanes, but
// half the waves and a longer row.  Worth it once there are four waves a SIMD (T * lanes / 64 >= 4096):
// softmax in 32 bits, k 8: 8192 x 256 13.6 us against 16.2, 131072 x 512 133 against 174; below it 4096 x
// 256 12.6 against 10.9, and at 128 experts even 131072 rows gain nothing (44.0, 45.5).
static bool router_halved(int T, int E) {
  return E > 128 && E <= 512 && (long long)T * router_lanes(E) >= 1ll << 18;
}
static int router_lanes_fwd(int T, int E) { return router_lanes(E) / (router_halved(T, E) ? 2 : 1); }

static int router_grid(int T, int lanes) {
  const int G = kRouterThreads / lanes;
  // one workgroup writes the totals itself: two rounds of its rows cost less than the second launch
  if (T <= 2 * G) return 1;
  return std::min((int)(((long long)T + G - 1) / G), kRouterMaxWG);
}

// Of what T rows need and any fewer: with 8 experts a lane, whose workgroups never decrease with T (where
// 16 experts a lane begin they halve), so that a workspace for the largest batch serves the others.
size_t router_ws_bytes(int T, int E) {
  const size_t wg = (size_t)router_grid(T, router_lanes(E));
  return align_up(wg * E * 4) * 2 + align_up(wg * 4) * 2 + 2 * align_up(64 * 4);
}

template <template <typename, int, int, int> class K, typename T, int SCORE>
static void router_shape(const RouterArgs& a, int grid, hipStream_t st) {
  if constexpr (K<T, 64, 16, SCORE>::kForward)           // the backward pass has no such variants
    if (router_halved(a.T, a.E)) {
      if (a.E <= 256) K<T, 16, 16, SCORE>::go(a, grid, st);
      else K<T, 32, 16, SCORE>::go(a, grid, st);
      return;
    }
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
  static constexpr bool kForward = true;
  static void go(const RouterArgs& a, int grid, hipStream_t st) {
    hipLaunchKernelGGL((k_router<T, L, V, SCORE>), dim3(grid), dim3(kRouterThreads), 0, st, a);
  }
};
template <typename T, int L, int V, int SCORE> struct BwdK {
  static constexpr bool kForward = false;
  static void go(const RouterArgs& a, int grid, hipStream_t st) {
    hipLaunchKernelGGL((k_router_bwd<T, L, V, SCORE>), dim3(grid), dim3(kRouterThreads), 0, st, a);
  }
};

int launch_router(const moe_router& R, const void* logits, int ld, const uint8_t* mask, int T,
                  int32_t* ids, float* gates, int32_t* counts, float* psum, int32_t* live,
                  float* losses, int32_t* status, void* ws, hipStream_t st) {
  RouterArgs a{};
  a.logits = logits; a.ld = (size_t)ld; a.mask = mask; a.T = T; a.E = R.E; a.k = R.k;
  a.renorm = R.renorm; a.scale = R.scale;
  a.ids = ids; a.gates = gates; a.counts = counts; a.psum = psum; a.live = live;
  a.losses = losses; a.status = status;
  const int grid = router_grid(T, router_lanes_fwd(T, R.E));
  char* w = (char*)ws;
  a.part_p = (float*)w;
  a.part_c = (int32_t*)(w += align_up((size_t)grid * R.E * 4));
  a.part_z = (float*)(w += align_up((size_t)grid * R.E * 4));
  a.part_n = (int32_t*)(w += align_up((size_t)grid * 4));
  a.dots = (float*)(w += align_up((size_t)grid * 4));
  a.done = (int32_t*)(w += align_up(64 * 4));
  a.parts = grid;
  router_kind<FwdK>(R, a, grid, st);
  if (grid > 1)
    hipLaunchKernelGGL(k_router_totals, dim3((R.E + kTotalCols - 1) / kTotalCols), dim3(kTotalThreads), 0, st, a);
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
  const int G = kRouterThreads / router_lanes(R.E);
  // four waves a SIMD, what most variants' registers allow at once: 65521 x 256 bf16 25.8 us (sigmoid 27.7)
  // in replays of a graph, with twice as many, the last of them alone, 25.8 (28.5), with one round of rows each 40.8 (43.5)
  const int grid = (int)std::min<long long>(((long long)T + G - 1) / G, 256 * 4);
  router_kind<BwdK>(R, a, grid, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// Reads no error: it is one of the launches of moe_backward_gates, whose last check sees them all.
void launch_gate_grad(const void* z, const void* dz, int dtype, const int32_t* row_to_slot,
                      int rows, int slots, int dff, float* dlogp, hipStream_t st) {
  if (rows == 0) return;
  // a launch holds fewer than 2^32 threads; past that the groups take further rows
  const dim3 grid((unsigned)std::min<size_t>(((size_t)rows + 15) / 16, (size_t)1 << 23));
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(k_gate_grad<float>, grid, dim3(256), 0, st, (const float*)z,
                       (const float*)dz, row_to_slot, rows, slots, dff, dlogp);
  else
    hipLaunchKernelGGL(k_gate_grad<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)z,
                       (const uint16_t*)dz, row_to_slot, rows, slots, dff, dlogp);
}

}  // namespace moe
