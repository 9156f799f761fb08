// C ABI of the MoE expert layer: argument checks on the host, workspace
// carving and kernel launches.  No allocation, no host synchronisation.
#include <hip/hip_runtime.h>

#include <float.h>
#include <stddef.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "moe_ffn.h"

using namespace moe;

namespace {

bool valid_P(int P) { return P == 1 || P == 2 || P == 4 || P == 8; }

bool ws_ok(const void* ws, size_t have, size_t need) {
  if (need == 0) return true;
  if (!ws) return false;
  if (((uintptr_t)ws) & 255u) return false;
  return have >= need;
}

struct Extent {
  const void* at;
  size_t bytes;
  bool meets(const Extent& o) const {
    return (uintptr_t)at < (uintptr_t)o.at + o.bytes && (uintptr_t)o.at < (uintptr_t)at + bytes;
  }
};

bool dtype_ok(int d) { return d == MOE_F32 || d == MOE_BF16; }

// 127 * 127 * K stays below 2^31
constexpr int kI8MaxK = 131072;

// Shared validation of the layer description; returns MOE_OK or an error.
int check_layer(const moe_layer* L, bool backward) {
  if (!L) return MOE_ERR_ARG;
  if (L->E < 1 || L->d < 1 || L->d_ff < 1) return MOE_ERR_ARG;
  if (!L->w1 || !L->w2) return MOE_ERR_ARG;
  if (L->E > kMaxPlanExperts) return MOE_ERR_UNSUPPORTED;
  if (L->d % 128 != 0 || L->d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
  const bool f32 = L->act_dtype == MOE_F32 && L->w_dtype == MOE_F32;
  const bool bf = L->act_dtype == MOE_BF16 && L->w_dtype == MOE_BF16;
  const bool f8 = L->act_dtype == MOE_BF16 && L->w_dtype == MOE_FP8_E4M3;
  const bool i8 = L->act_dtype == MOE_BF16 && L->w_dtype == MOE_INT8;
  if (!f32 && !bf && !f8 && !i8)
    return L->act_dtype > MOE_BF16 || L->w_dtype > MOE_INT8 ? MOE_ERR_ARG : MOE_ERR_UNSUPPORTED;
  if (i8) {
    // read in pieces of 16 bytes, straight into LDS: a byte's address need not be one
    if (!L->w1_scale || !L->w2_scale || (((uintptr_t)L->w1 | (uintptr_t)L->w2) & 15) ||
        (((uintptr_t)L->w1_scale | (uintptr_t)L->w2_scale) & 3))
      return MOE_ERR_ARG;
    if (backward || L->d > kI8MaxK || L->d_ff > kI8MaxK) return MOE_ERR_UNSUPPORTED;
  }
  if (f8) {
    if (L->d_ff % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (!L->w1_scale || !L->w2_scale) return MOE_ERR_ARG;
  }
  return MOE_OK;
}

Sizes make_sizes(const moe_layer* L, int T, int k, int beta, int P, int s) {
  Sizes z{};
  z.T = T; z.k = k; z.E = L->E; z.d = L->d; z.dff = L->d_ff; z.beta = beta; z.P = P; z.s = s;
  z.act_bytes = L->act_dtype == MOE_F32 ? 4 : 2;
  z.fp8 = L->w_dtype == MOE_FP8_E4M3 ? 1 : 0;
  z.i8 = L->w_dtype == MOE_INT8 ? 1 : 0;
  z.max_slots = moe_max_slots(T, k, L->E, beta);
  z.max_blocks = moe_max_blocks(T, k, L->E, beta);
  z.max_mt = max_tiles(z);
  return z;
}

bool sizes_ok(int T, int k, int E, int beta) {
  if (T < 0 || k < 1 || E < 1 || beta < 1) return false;
  const long long slots = (long long)T * k + (long long)E * (beta - 1);
  return slots < (1ll << 31);
}

// The GEMM kernels address every operand through buffer descriptors with
// 32-bit byte offsets, and send masked rows to offset 2^31, which reads as
// zeros only while the descriptor's size is below it.  Each such operand must
// therefore span less than 2 GiB: token rows (x, dy, y, dx), the
// slot-indexed buffers (A or dZ, O, P, z_save, the requantized D), all in the
// activation dtype, and one expert's weights.
bool extents_ok(const Sizes& z) {
  const unsigned long long lim = 1ull << 31, S = (unsigned long long)z.max_slots;
  const unsigned long long d = (unsigned long long)z.d, f = (unsigned long long)z.dff;
  const unsigned long long ab = (unsigned long long)z.act_bytes, wb = z.fp8 || z.i8 ? 1ull : ab;
  return (unsigned long long)z.T * d * ab < lim && S * 2 * f * ab < lim && S * d * ab < lim &&
         2 * f * d * wb < lim;
}

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_status_str(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported configuration";
    case MOE_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case MOE_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

size_t moe_max_slots(int T, int k, int E, int beta) {
  if (!sizes_ok(T, k, E, beta)) return 0;
  return (size_t)T * k + (size_t)E * (beta - 1);
}

size_t moe_max_blocks(int T, int k, int E, int beta) {
  if (!sizes_ok(T, k, E, beta)) return 0;
  return ((size_t)T * k + (size_t)E * (beta - 1)) / beta;
}

size_t moe_workspace_size(const moe_layer* L, int T, int k, int beta, int P, int s,
                          int with_backward) {
  if (!L || !sizes_ok(T, k, L->E, beta) || !valid_P(P) || s < 0) return 0;
  if (L->E > kMaxExperts) return 0;
  size_t need = route_ws_bytes(T, k, L->E);
  if (L->E <= kMaxPlanExperts && L->d > 0 && L->d_ff > 0) {
    const Sizes z = make_sizes(L, T, k, beta, P, s);
    if (!extents_ok(z)) return 0;
    const size_t f = exec_layout(z, false).total;
    if (f > need) need = f;
    if (with_backward && z.i8) return 0;
    if (with_backward) {
      const size_t b = exec_layout(z, true).total;
      if (b > need) need = b;
    }
  }
  return need;
}

int moe_route_stats(const int32_t* topk_ids, int T, int k, int E, int beta, int32_t* counts,
                    int32_t* offsets, int32_t* block_counts, int32_t* block_offsets,
                    int32_t* row_to_slot, int32_t* slot_to_row, double* kappa,
                    int32_t* status_dev, void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(T, k, E, beta)) return MOE_ERR_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!topk_ids || !row_to_slot)) || !counts || !offsets || !block_counts ||
      !block_offsets || !slot_to_row || !kappa || !status_dev)
    return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, route_ws_bytes(T, k, E))) return MOE_ERR_WORKSPACE;
  return launch_route_stats(topk_ids, T, k, E, beta, counts, offsets, block_counts,
                            block_offsets, row_to_slot, slot_to_row, kappa, status_dev, ws,
                            (hipStream_t)stream);
}

int moe_route_stats_noalloc(const int32_t* topk_ids, int T, int k, int E, int beta,
                            int32_t* counts, int32_t* offsets, int32_t* block_counts,
                            int32_t* block_offsets, int32_t* row_to_slot, int32_t* slot_to_row,
                            double* kappa, int32_t* status_dev, void* stream) {
  if (!sizes_ok(T, k, E, beta)) return MOE_ERR_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!topk_ids || !row_to_slot)) || !counts || !offsets || !block_counts ||
      !block_offsets || !slot_to_row || !kappa || !status_dev)
    return MOE_ERR_ARG;
  if (route_ws_bytes(T, k, E) > kRouteScratchBytes) return MOE_ERR_UNSUPPORTED;
  void* scr = nullptr;
  const int rc = route_scratch(&scr);
  if (rc != MOE_OK) return rc;
  return launch_route_stats(topk_ids, T, k, E, beta, counts, offsets, block_counts,
                            block_offsets, row_to_slot, slot_to_row, kappa, status_dev, scr,
                            (hipStream_t)stream);
}

int moe_plan(const int32_t* block_counts, const int32_t* block_offsets, const int32_t* owner,
             int E, int P, int s, int mode, int lambda, int32_t* q, int32_t* load,
             int32_t* block_worker, int block_worker_cap, int32_t* plan_info,
             int32_t* status_dev, void* ws, size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  if (E < 1 || s < 0 || lambda < 0 || block_worker_cap < 0 ||
      (mode != MOE_PLAN_FWD && mode != MOE_PLAN_BWD && mode != MOE_PLAN_QUOTA) ||
      (mode == MOE_PLAN_QUOTA && lambda < 1))
    return MOE_ERR_ARG;
  if (!valid_P(P) || E > kMaxPlanExperts) return MOE_ERR_UNSUPPORTED;
  if (!block_counts || !block_offsets || !owner || !q || !load || !block_worker ||
      !plan_info || !status_dev)
    return MOE_ERR_ARG;
  return launch_plan(block_counts, block_offsets, owner, E, P, s, mode, lambda, q, load,
                     block_worker, block_worker_cap, plan_info, status_dev, (hipStream_t)stream);
}

int moe_plan_gate(const int32_t* block_counts, const int32_t* block_offsets, const int32_t* owner,
                  int E, int P, int rho_milli, int32_t* q, int32_t* load, int32_t* block_worker,
                  int block_worker_cap, int32_t* plan_info, int32_t* status_dev, void* stream) {
  if (E < 1 || rho_milli < 0 || block_worker_cap < 0) return MOE_ERR_ARG;
  if (!valid_P(P) || E > kMaxPlanExperts) return MOE_ERR_UNSUPPORTED;
  if (!block_counts || !block_offsets || !owner || !q || !load || !block_worker || !plan_info ||
      !status_dev)
    return MOE_ERR_ARG;
  return launch_plan_gate(block_counts, block_offsets, owner, E, P, rho_milli, q, load,
                          block_worker, block_worker_cap, plan_info, status_dev,
                          (hipStream_t)stream);
}

int moe_quantize_token_blocks(const void* src, int ld, int src_rows, const int32_t* row_map,
                              int gather, int row_div, const float* row_scale, int rows, int cols,
                              int block_rows, uint8_t* codes, float* scales, void* stream) {
  if (rows < 0 || cols < 8 || cols % 8 || cols > kQtMaxCols || ld < cols || ld % 8 ||
      block_rows < 1 || row_div < 1 || src_rows < 0)
    return MOE_ERR_ARG;
  // rows read in place (no map, or a map without gather) need src_rows >= rows
  if ((!row_map || !gather) && src_rows < rows) return MOE_ERR_ARG;
  if (!src || !codes || !scales) return MOE_ERR_ARG;
  const long long lim = (long long)src_rows * row_div;
  launch_quant_tok((const uint16_t*)src, ld, row_map, gather ? 1 : 0, row_div, row_scale,
                   lim < INT32_MAX ? (int)lim : INT32_MAX, rows, cols, block_rows, codes, scales,
                   (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_quantize_act_rows(const void* src, int rows, int cols, uint8_t* codes, int32_t* exps,
                          void* stream) {
  if (rows < 0 || cols < 128 || cols % 128) return MOE_ERR_ARG;
  if (rows > 0 && (!src || !codes || !exps)) return MOE_ERR_ARG;
  if (rows == 0) return MOE_OK;
  launch_quant_act((const uint16_t*)src, rows, cols, codes, exps, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_quantize_int8_rows(const void* src, int ld, int dtype, int rows, int cols, int8_t* codes, float* scales,
                           void* stream) {
  if (rows < 0 || cols < 1 || ld < cols || !dtype_ok(dtype) || (rows > 0 && (!src || !codes || !scales)))
    return MOE_ERR_ARG;
  if (cols > (1 << 30)) return MOE_ERR_UNSUPPORTED;        // a lane's next piece is counted in 32 bits
  if (rows == 0) return MOE_OK;
  const size_t eb = dtype == MOE_F32 ? 4 : 2;
  const Extent all[3] = {{src, ((size_t)(rows - 1) * ld + cols) * eb}, {codes, (size_t)rows * cols},
                         {scales, (size_t)rows * sizeof(float)}};
  if (all[0].meets(all[1]) || all[0].meets(all[2]) || all[1].meets(all[2])) return MOE_ERR_ARG;
  return launch_quant_int8_rows(src, ld, dtype, rows, cols, codes, scales, (hipStream_t)stream);
}

int moe_predict_cost(const int32_t* counts, const int32_t* block_offsets,
                     const int32_t* block_worker_fwd, const int32_t* block_worker_bwd,
                     const int32_t* owner, int E, int beta, int P, int d, int d_ff,
                     int num_workgroups, int64_t* cost_dev, int32_t* status_dev, void* stream) {
  if (E < 1 || beta < 1 || d < 1 || d_ff < 1) return MOE_ERR_ARG;
  if (!counts || !block_offsets || !block_worker_fwd || !block_worker_bwd || !owner || !cost_dev ||
      !status_dev)
    return MOE_ERR_ARG;
  if (!valid_P(P) || E > kMaxPlanExperts || d % 256 || d_ff % 256) return MOE_ERR_UNSUPPORTED;
  int G = num_workgroups;
  if (G <= 0) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&G, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return MOE_ERR_HIP;
  }
  if (G % P || G / P > 256) return MOE_ERR_UNSUPPORTED;
  return launch_predict_cost(counts, block_offsets, block_worker_fwd, block_worker_bwd, owner, E,
                             beta, P, d, d_ff, G, (long long*)cost_dev, status_dev,
                             (hipStream_t)stream);
}

int moe_predict_split(const int32_t* counts, const int32_t* block_offsets,
                      const int32_t* block_worker, int E, int beta, int P, int d, int d_ff,
                      int num_workgroups, int backward, int64_t* costs_dev, int32_t* choice_dev,
                      int32_t* status_dev, void* stream) {
  if (E < 1 || beta < 1 || d < 1 || d_ff < 1) return MOE_ERR_ARG;
  if (!counts || !block_offsets || !block_worker || !costs_dev || !choice_dev || !status_dev)
    return MOE_ERR_ARG;
  if (!valid_P(P) || E > kMaxPlanExperts || d % 256 || d_ff % 256) return MOE_ERR_UNSUPPORTED;
  int G = num_workgroups;
  if (G <= 0) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&G, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return MOE_ERR_HIP;
  }
  if (G % P || G / P > 256) return MOE_ERR_UNSUPPORTED;
  return launch_predict_split(counts, block_offsets, block_worker, E, beta, P, d, d_ff, G,
                              backward ? 1 : 0, (long long*)costs_dev, choice_dev, status_dev,
                              (hipStream_t)stream);
}

// known bits only; a producer/consumer split only with the two-phase launch
// (its upper bound, the workgroups of one worker, is checked at launch)
static bool exec_flags_ok(int f) {
  const int split = (f >> MOE_EXEC_SPLIT_SHIFT) & 0xff;
  const int known = MOE_EXEC_TWO_PHASE | MOE_EXEC_SPLIT(0xff) | MOE_EXEC_FP8_ACT;
  if (f & ~known) return false;
  return split == 0 || (f & MOE_EXEC_TWO_PHASE);
}

int moe_forward(const moe_layer* L, const void* x, const float* gates, const int32_t* topk_ids,
                int T, int k, int beta, int P, const int32_t* counts,
                const int32_t* block_offsets, const int32_t* row_to_slot,
                const int32_t* slot_to_row, const int32_t* block_worker, void* y, void* z_save,
                int32_t* status_dev, void* ws, size_t ws_bytes, int exec_flags,
                void* const* stage_events, uint64_t* timeline, void* stream) {
  (void)topk_ids;
  const int lc = check_layer(L, false);
  if (!exec_flags_ok(exec_flags)) return MOE_ERR_ARG;
  if (lc != MOE_OK) return lc;
  if (!sizes_ok(T, k, L->E, beta)) return MOE_ERR_ARG;
  if (!valid_P(P)) return MOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!x || !gates || !row_to_slot || !y)) || !counts || !block_offsets ||
      !slot_to_row || !block_worker || !status_dev)
    return MOE_ERR_ARG;
  const Sizes z = make_sizes(L, T, k, beta, P, 0);
  if (!extents_ok(z)) return MOE_ERR_UNSUPPORTED;
  // the fp8 MFMA forward: bf16 x, e4m3 weights on the stream kernels, two launches
  if ((exec_flags & MOE_EXEC_FP8_ACT) &&
      (L->act_dtype != MOE_BF16 || L->w_dtype != MOE_FP8_E4M3 || !use_stream(z) ||
       (exec_flags & MOE_EXEC_TWO_PHASE)))
    return MOE_ERR_ARG;
  if (z.i8 && (z_save || exec_flags)) return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, exec_layout(z, false).total)) return MOE_ERR_WORKSPACE;
  LayerPtrs Lp{L->w1, L->w2, L->w1_scale, L->w2_scale, L->act_dtype, L->w_dtype};
  return launch_forward(z, Lp, x, gates, counts, block_offsets, row_to_slot, slot_to_row,
                        block_worker, y, z_save, status_dev, (char*)ws, exec_flags, stage_events,
                        timeline, (hipStream_t)stream);
}

static int backward(const moe_layer* L, const void* x, const float* gates, const void* dy,
                 const void* z_save, int T, int k, int beta, int P,
                 int s, const int32_t* counts, const int32_t* block_offsets,
                 const int32_t* row_to_slot, const int32_t* slot_to_row, const int32_t* owner,
                 const int32_t* block_worker, void* dx, float* dw1, float* dw2,
                 float* dlogp, int32_t* status_dev, void* ws, size_t ws_bytes, int exec_flags,
                 void* const* stage_events, uint64_t* timeline, void* stream) {
  const int lc = check_layer(L, true);
  if (!exec_flags_ok(exec_flags)) return MOE_ERR_ARG;
  if (lc != MOE_OK) return lc;
  if (!sizes_ok(T, k, L->E, beta) || s < 0) return MOE_ERR_ARG;
  if (!valid_P(P)) return MOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!x || !gates || !dy || !z_save || !row_to_slot || !dx)) || !counts ||
      !block_offsets || !slot_to_row || !owner || !block_worker || !dw1 || !dw2 || !status_dev)
    return MOE_ERR_ARG;
  const Sizes z = make_sizes(L, T, k, beta, P, s);
  if (!extents_ok(z)) return MOE_ERR_UNSUPPORTED;
  // dA and dX on the fp8 MFMA: bf16 dy, e4m3 weights on the stream kernels, two launches
  if ((exec_flags & MOE_EXEC_FP8_ACT) &&
      (L->act_dtype != MOE_BF16 || L->w_dtype != MOE_FP8_E4M3 || !use_stream(z) ||
       (exec_flags & MOE_EXEC_TWO_PHASE)))
    return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, exec_layout(z, true).total)) return MOE_ERR_WORKSPACE;
  LayerPtrs Lp{L->w1, L->w2, L->w1_scale, L->w2_scale, L->act_dtype, L->w_dtype};
  return launch_backward(z, Lp, x, gates, dy, z_save, counts, block_offsets, row_to_slot,
                         slot_to_row, owner, block_worker, dx, dw1, dw2, dlogp, status_dev, (char*)ws,
                         exec_flags, stage_events, timeline, (hipStream_t)stream);
}

int moe_backward(const moe_layer* L, const void* x, const float* gates, const void* dy,
                 const void* z_save, const int32_t* topk_ids, int T, int k, int beta, int P,
                 int s, const int32_t* counts, const int32_t* block_offsets,
                 const int32_t* row_to_slot, const int32_t* slot_to_row, const int32_t* owner,
                 const int32_t* block_worker, void* dx, float* dw1, float* dw2,
                 int32_t* status_dev, void* ws, size_t ws_bytes, int exec_flags,
                 void* const* stage_events, uint64_t* timeline, void* stream) {
  (void)topk_ids;
  return backward(L, x, gates, dy, z_save, T, k, beta, P, s, counts, block_offsets, row_to_slot,
                  slot_to_row, owner, block_worker, dx, dw1, dw2, nullptr, status_dev, ws, ws_bytes,
                  exec_flags, stage_events, timeline, stream);
}

int moe_backward_gates(const moe_layer* L, const void* x, const float* gates, const void* dy,
                       const void* z_save, const int32_t* topk_ids, int T, int k, int beta,
                       int P, int s, const int32_t* counts, const int32_t* block_offsets,
                       const int32_t* row_to_slot, const int32_t* slot_to_row,
                       const int32_t* owner, const int32_t* block_worker, void* dx, float* dw1,
                       float* dw2, float* dlogp, int32_t* status_dev, void* ws, size_t ws_bytes,
                       int exec_flags, void* const* stage_events, uint64_t* timeline,
                       void* stream) {
  (void)topk_ids;
  if (T > 0 && !dlogp) return MOE_ERR_ARG;
  return backward(L, x, gates, dy, z_save, T, k, beta, P, s, counts, block_offsets, row_to_slot,
                  slot_to_row, owner, block_worker, dx, dw1, dw2, dlogp, status_dev, ws, ws_bytes,
                  exec_flags, stage_events, timeline, stream);
}

static int check_router(const moe_router* R, int ld, int T) {
  if (!R || R->E < 1 || R->k < 1 || R->k > R->E || T < 0 || ld < R->E || !dtype_ok(R->dtype) ||
      (R->score != MOE_SCORE_SOFTMAX && R->score != MOE_SCORE_SIGMOID) || !std::isfinite(R->scale))
    return MOE_ERR_ARG;
  if (R->E > kMaxExperts || R->k > kRouterMaxK || (long long)T * R->k >= (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t moe_router_workspace_size(const moe_router* R, int T) {
  if (!R || check_router(R, R->E, T) != MOE_OK) return 0;
  return router_ws_bytes(T, R->E);
}

static int router_forward(const moe_router* R, const moe_choice* C, const void* logits, int ld,
                          const uint8_t* token_mask, int T, int32_t* topk_ids, float* gates,
                          int32_t* counts, float* prob_sum, int32_t* live, float* losses,
                          int32_t* status_dev, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_router(R, ld, T);
  if (rc != MOE_OK) return rc;
  if (C) {
    if (C->groups < 1 || R->E % C->groups || C->top_groups < 1 || C->top_groups > C->groups ||
        R->k > C->top_groups * (R->E / C->groups) ||
        (C->group_score != MOE_GROUP_MAX && C->group_score != MOE_GROUP_TOP2))
      return MOE_ERR_ARG;
    if (C->groups > kRouterMaxGroups) return MOE_ERR_UNSUPPORTED;
  }
  if ((T > 0 && (!logits || !topk_ids || !gates)) || !counts || !prob_sum || !live || !losses ||
      !status_dev)
    return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, router_ws_bytes(T, R->E))) return MOE_ERR_WORKSPACE;
  return launch_router(*R, C, logits, ld, token_mask, T, topk_ids, gates, counts, prob_sum, live,
                       losses, status_dev, ws, (hipStream_t)stream);
}

int moe_router_forward(const moe_router* R, const void* logits, int ld,
                       const uint8_t* token_mask, int T, int32_t* topk_ids, float* gates,
                       int32_t* counts, float* prob_sum, int32_t* live, float* losses,
                       int32_t* status_dev, void* ws, size_t ws_bytes, void* stream) {
  return router_forward(R, nullptr, logits, ld, token_mask, T, topk_ids, gates, counts, prob_sum, live, losses,
                        status_dev, ws, ws_bytes, stream);
}

int moe_router_forward_choice(const moe_router* R, const moe_choice* choice, const void* logits, int ld,
                              const uint8_t* token_mask, int T, int32_t* topk_ids, float* gates,
                              int32_t* counts, float* prob_sum, int32_t* live, float* losses,
                              int32_t* status_dev, void* ws, size_t ws_bytes, void* stream) {
  if (!choice) return MOE_ERR_ARG;
  return router_forward(R, choice, logits, ld, token_mask, T, topk_ids, gates, counts, prob_sum, live, losses,
                        status_dev, ws, ws_bytes, stream);
}

int moe_router_bias_update(const int32_t* counts, int E, float rate, float* bias, void* stream) {
  if (E < 1 || !std::isfinite(rate) || !counts || !bias) return MOE_ERR_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  return launch_bias_update(counts, E, rate, bias, (hipStream_t)stream);
}

int moe_router_backward(const moe_router* R, const void* logits, int ld,
                        const uint8_t* token_mask, int T, const int32_t* topk_ids,
                        const float* dlogp, const int32_t* counts, const int32_t* live,
                        const float* dlosses, void* dlogits, int ld_out, void* stream) {
  const int rc = check_router(R, ld, T);
  if (rc != MOE_OK) return rc;
  if (ld_out < R->E || (T > 0 && (!logits || !topk_ids || !dlogits)) || !counts || !live)
    return MOE_ERR_ARG;
  return launch_router_bwd(*R, logits, ld, token_mask, T, topk_ids, dlogp, counts, live, dlosses,
                           dlogits, ld_out, (hipStream_t)stream);
}

int moe_gate_grad(const void* z, const void* dz, int dtype, const int32_t* row_to_slot, int rows,
                  int slots, int d_ff, float* dlogp, void* stream) {
  if (rows < 0 || slots < 0 || d_ff < 1 || !dtype_ok(dtype)) return MOE_ERR_ARG;
  if (d_ff % 64) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!row_to_slot || !dlogp)) return MOE_ERR_ARG;
  if (slots > 0 && (!z || !dz)) return MOE_ERR_ARG;
  launch_gate_grad(z, dz, dtype, row_to_slot, rows, slots, d_ff, dlogp, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

static int check_norm(const moe_norm* N) {
  if (!N || N->d < 1 || N->T < 0 || !dtype_ok(N->dtype) || !(N->eps > 0.f) ||
      !std::isfinite(N->eps) || !std::isfinite(N->alpha) || N->gate_kind < MOE_GATE_NONE ||
      N->gate_kind > MOE_GATE_FEATURE || !N->w)
    return MOE_ERR_ARG;
  if (N->gate_kind == MOE_GATE_NONE
          ? N->gate != nullptr
          : !N->gate && (N->T > 0 || N->gate_kind == MOE_GATE_FEATURE))
    return MOE_ERR_ARG;
  if (N->d > kNormMaxD || (N->w_dtype != MOE_F32 && N->w_dtype != N->dtype))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t moe_norm_workspace_size(int T, int d) {
  return T < 0 || d < 1 || d > kNormMaxD ? 0 : norm_ws_bytes(T, d);
}

int moe_norm_in(const moe_norm* N, const void* x, int ldx, const void* u, int ldu, void* r,
                int ldr, void* n, int ldn, float* rstd, void* stream) {
  const int rc = check_norm(N);
  if (rc != MOE_OK) return rc;
  if ((N->T > 0 && (!x || !n || !rstd)) || ldx < N->d || ldn < N->d || (u && ldu < N->d) ||
      (r && ldr < N->d) || (N->T > 0 && !u && N->gate_kind != MOE_GATE_NONE))
    return MOE_ERR_ARG;
  return launch_norm(*N, false, {x, ldx}, {u, ldu}, {r, ldr}, {n, ldn}, rstd, (hipStream_t)stream);
}

int moe_norm_out(const moe_norm* N, const void* y, int ldy, const void* x, int ldx, void* out,
                 int ldout, float* rstd, void* stream) {
  const int rc = check_norm(N);
  if (rc != MOE_OK) return rc;
  if ((N->T > 0 && (!y || !x || !out || !rstd)) || ldx < N->d || ldy < N->d || ldout < N->d)
    return MOE_ERR_ARG;
  return launch_norm(*N, true, {x, ldx}, {y, ldy}, {nullptr, 0}, {out, ldout}, rstd,
                     (hipStream_t)stream);
}

int moe_norm_in_backward(const moe_norm* N, const void* dn, int lddn, const void* dr, int lddr,
                         const void* r, int ldr, const void* u, int ldu, const float* rstd,
                         void* dx, int lddx, void* du, int lddu, float* dw, float* dgate,
                         void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_norm(N);
  if (rc != MOE_OK) return rc;
  if ((N->T > 0 && (!dn || !r || !rstd || !dx)) || !dw || lddn < N->d || ldr < N->d ||
      lddx < N->d || (dr && lddr < N->d) || (u && ldu < N->d) || (du && lddu < N->d) ||
      (N->T > 0 && !u != !du) || (N->T > 0 && !u && N->gate_kind != MOE_GATE_NONE) ||
      (N->gate_kind == MOE_GATE_NONE ? dgate != nullptr
                                     : !dgate && (N->T > 0 || N->gate_kind == MOE_GATE_FEATURE)))
    return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, norm_ws_bytes(N->T, N->d))) return MOE_ERR_WORKSPACE;
  return launch_norm_bwd(*N, false, {dn, lddn}, {dr, lddr}, {r, ldr}, {u, ldu}, rstd, {dx, lddx},
                         {du, lddu}, dw, dgate, ws, (hipStream_t)stream);
}

int moe_norm_out_backward(const moe_norm* N, const void* dout, int lddo, const void* y, int ldy,
                          const float* rstd, void* dy, int lddy, float* dw, float* dgate, void* ws,
                          size_t ws_bytes, void* stream) {
  const int rc = check_norm(N);
  if (rc != MOE_OK) return rc;
  if ((N->T > 0 && (!dout || !y || !rstd || !dy)) || !dw || lddo < N->d || ldy < N->d ||
      lddy < N->d ||
      (N->gate_kind == MOE_GATE_NONE ? dgate != nullptr
                                     : !dgate && (N->T > 0 || N->gate_kind == MOE_GATE_FEATURE)))
    return MOE_ERR_ARG;
  if (!ws_ok(ws, ws_bytes, norm_ws_bytes(N->T, N->d))) return MOE_ERR_WORKSPACE;
  return launch_norm_bwd(*N, true, {dout, lddo}, {nullptr, 0}, {y, ldy}, {nullptr, 0}, rstd,
                         {dy, lddy}, {nullptr, 0}, dw, dgate, ws, (hipStream_t)stream);
}

size_t moe_adamw_workspace_size(int tensors) {
  return tensors < 0 || tensors > MOE_ADAMW_MAX_TENSORS ? 0 : adamw_ws_bytes(tensors);
}

namespace {
// A tensor's buffers are its first seven members: p, master, g, m, v and the states' scales.  A buffer's
// number is its tensor's times 8 plus its place there, 16 bits.
constexpr int kAdamBuffers = 7;
static_assert(offsetof(moe_adamw_tensor, g) == 2 * sizeof(void*) &&
              offsetof(moe_adamw_tensor, v_scale) == 6 * sizeof(void*), "seven pointers");
static_assert(8 * MOE_ADAMW_MAX_TENSORS <= 65536, "16 bits");

uintptr_t buffer_at(const moe_adamw_tensor* t, unsigned i) {
  uintptr_t at;
  memcpy(&at, (const char*)(t + i / 8) + sizeof(void*) * (i % 8), sizeof at);
  return at;
}
size_t buffer_bytes(const moe_adamw_tensor* t, int bits, unsigned i) {
  const moe_adamw_tensor& a = t[i / 8];
  const size_t n = (size_t)a.n;
  switch (i % 8) {
    case 0: return n * (a.p_dtype == MOE_F32 ? 4 : 2);
    case 1: return n * 4;
    case 2: return n * (a.g_dtype == MOE_F32 ? 4 : 2);
    case 3:
    case 4: return bits == 8 ? n : n * 4;
    default: return bits == 8 ? (n + MOE_ADAMW_BLOCK - 1) / MOE_ADAMW_BLOCK * 4 : 0;
  }
}

// Whether no written buffer of the list shares memory with another.  Only the buffers' numbers are
// sorted (56 KB of the stack), so nothing is allocated; 4096 tensors take 2 ms.
bool extents_apart(const moe_adamw_tensor* t, int count, int bits) {
  uint16_t order[kAdamBuffers * MOE_ADAMW_MAX_TENSORS];
  size_t m = 0;
  for (int i = 0; i < count; ++i)
    for (int j = 0; j < kAdamBuffers; ++j) {
      const unsigned k = 8u * i + j;
      if (buffer_at(t, k) && buffer_bytes(t, bits, k)) order[m++] = (uint16_t)k;
    }
  std::sort(order, order + m, [&](uint16_t a, uint16_t b) { return buffer_at(t, a) < buffer_at(t, b); });
  uintptr_t end = 0, end_w = 0;      // furthest end of any, and of a written, earlier buffer
  for (size_t i = 0; i < m; ++i) {
    const bool written = order[i] % 8 != 2;
    const uintptr_t at = buffer_at(t, order[i]), past = at + buffer_bytes(t, bits, order[i]);
    if (at < (written ? end : end_w)) return false;
    end = std::max(end, past);
    if (written) end_w = std::max(end_w, past);
  }
  return true;
}
}  // namespace

int moe_adamw_prepare(const moe_adamw_tensor* tensors, int count, int state_bits,
                      moe_adamw_list* out, void* ws, size_t ws_bytes, void* stream) {
  if (count < 0 || count > MOE_ADAMW_MAX_TENSORS || !out || (count > 0 && !tensors))
    return MOE_ERR_ARG;
  if (state_bits != 8 && state_bits != 32) return MOE_ERR_UNSUPPORTED;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype)) return MOE_ERR_ARG;
    if (t.n == 0) continue;
    if (t.n > (1ll << 43) || (total += t.n) > (1ll << 43)) return MOE_ERR_UNSUPPORTED;
    const uintptr_t pb = t.p_dtype == MOE_F32 ? 3 : 1, gb = t.g_dtype == MOE_F32 ? 3 : 1;
    if (!t.p || !t.g || !t.m || !t.v || ((uintptr_t)t.p & pb) || ((uintptr_t)t.g & gb))
      return MOE_ERR_ARG;
    if (t.master && (t.p_dtype != MOE_BF16 || ((uintptr_t)t.master & 3))) return MOE_ERR_ARG;
    if (state_bits == 8) {
      if (!t.m_scale || !t.v_scale || (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) & 3))
        return MOE_ERR_ARG;
    } else if (((uintptr_t)t.m | (uintptr_t)t.v) & 3) {
      return MOE_ERR_ARG;
    }
  }
  if (!ws_ok(ws, ws_bytes, adamw_ws_bytes(count))) return MOE_ERR_WORKSPACE;
  if (!extents_apart(tensors, count, state_bits)) return MOE_ERR_ARG;
  moe_adamw_list list{};
  list.table = ws;
  list.tensors = count;
  list.state_bits = state_bits;
  const int rc = launch_adamw_table(tensors, count, &list, (hipStream_t)stream);
  if (rc == MOE_OK) *out = list;
  return rc;
}

int moe_adamw(const moe_adamw_list* list, const moe_adamw_hyper* h, void* stream) {
  if (!list || !h || list->tensors < 0 || (list->items > 0 && !list->table) ||
      (list->state_bits != 8 && list->state_bits != 32))
    return MOE_ERR_ARG;
  if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1) || (!h->step_dev && h->step < 1))
    return MOE_ERR_ARG;
  // as the kernel holds them: an eps below fp32's normal numbers has no reciprocal, and 0 / eps would be NaN
  if (!((float)h->eps >= FLT_MIN) || !std::isfinite((float)h->eps) ||
      !std::isfinite((float)h->weight_decay) || (!h->lr_dev && !std::isfinite((float)h->lr)))
    return MOE_ERR_ARG;
  return launch_adamw(*list, *h, (hipStream_t)stream);
}

size_t moe_grad_workspace_size(int tensors) {
  return tensors < 0 || tensors > MOE_GRAD_MAX_TENSORS ? 0 : grads_ws_bytes(tensors);
}

// Whether no two tensors of the list share memory; as extents_apart, only their numbers are sorted.
static bool grads_apart(const moe_grad_tensor* t, int count) {
  uint16_t order[MOE_GRAD_MAX_TENSORS];
  int m = 0;
  for (int i = 0; i < count; ++i)
    if (t[i].n > 0) order[m++] = (uint16_t)i;
  std::sort(order, order + m, [&](uint16_t a, uint16_t b) { return (uintptr_t)t[a].g < (uintptr_t)t[b].g; });
  uintptr_t end = 0;
  for (int i = 0; i < m; ++i) {
    const moe_grad_tensor& a = t[order[i]];
    if ((uintptr_t)a.g < end) return false;
    end = std::max(end, (uintptr_t)a.g + (uintptr_t)a.n * (a.dtype == MOE_F32 ? 4 : 2));
  }
  return true;
}

int moe_grad_prepare(const moe_grad_tensor* tensors, int count, moe_grad_list* out, void* ws,
                     size_t ws_bytes, void* stream) {
  if (count < 0 || count > MOE_GRAD_MAX_TENSORS || !out || (count > 0 && !tensors)) return MOE_ERR_ARG;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    const moe_grad_tensor& t = tensors[i];
    if (t.n < 0 || !dtype_ok(t.dtype)) return MOE_ERR_ARG;
    if (t.n == 0) continue;
    if (t.n > (1ll << 43) || (total += t.n) > (1ll << 43)) return MOE_ERR_UNSUPPORTED;
    if (!t.g || ((uintptr_t)t.g & (t.dtype == MOE_F32 ? 3 : 1))) return MOE_ERR_ARG;
  }
  if (!ws_ok(ws, ws_bytes, grads_ws_bytes(count))) return MOE_ERR_WORKSPACE;
  moe_grad_list list{};
  list.table = ws;
  list.tensors = count;
  list.apart = grads_apart(tensors, count);
  const int rc = launch_grads_table(tensors, count, &list, (hipStream_t)stream);
  if (rc == MOE_OK) *out = list;
  return rc;
}

static bool grad_list_ok(const moe_grad_list* l) {
  return l && l->table && l->tensors >= 0 && l->tensors <= MOE_GRAD_MAX_TENSORS && l->items < (1u << 24);
}

int moe_grad_norm(const moe_grad_list* list, const moe_clip* clip, float* norm, float* scale,
                  int32_t* status_dev, void* stream) {
  if (!grad_list_ok(list) || !clip || !norm || !scale || !status_dev || !(clip->max_norm > 0) ||
      (!clip->mult_dev && !std::isfinite(clip->mult)))
    return MOE_ERR_ARG;
  return launch_grad_norm(*list, *clip, norm, scale, status_dev, (hipStream_t)stream);
}

int moe_grad_scale(const moe_grad_list* list, const float* scale, void* stream) {
  if (!grad_list_ok(list) || !scale || !list->apart) return MOE_ERR_ARG;
  return launch_grad_scale(*list, scale, (hipStream_t)stream);
}

int moe_event_create(void** ev) {
  if (!ev) return MOE_ERR_ARG;
  return hipEventCreate((hipEvent_t*)ev) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
int moe_event_destroy(void* ev) {
  return hipEventDestroy((hipEvent_t)ev) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
int moe_event_record(void* ev, void* stream) {
  return hipEventRecord((hipEvent_t)ev, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
int moe_event_elapsed_ms(void* a, void* b, float* ms) {
  if (!ms) return MOE_ERR_ARG;
  if (hipEventSynchronize((hipEvent_t)b) != hipSuccess) return MOE_ERR_HIP;
  return hipEventElapsedTime(ms, (hipEvent_t)a, (hipEvent_t)b) == hipSuccess ? MOE_OK
                                                                              : MOE_ERR_HIP;
}

int moe_device_info(int* num_cus, int* num_xcds, int* wg_per_cu_gemm) {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MOE_ERR_HIP;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return MOE_ERR_HIP;
  if (num_cus) *num_cus = n;
  if (num_xcds) *num_xcds = 8;
  if (wg_per_cu_gemm) *wg_per_cu_gemm = gemm_wg_per_cu();
  return MOE_OK;
}

}  // extern "C"
