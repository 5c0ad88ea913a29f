// Launchers of the mixture-of-experts and weight-only FP4 operators (experts.hip, wlinear.hip).
#pragma once
#include <algorithm>
#include <type_traits>

#include "fp4_device.hpp"
#include "launch.hpp"

namespace fp4k {

// two float32 -> two bf16, nearest-even (v_cvt_pk_bf16_f32), a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Keeps a wave's LDS accesses in program order (the LDS itself serves a wave's accesses in order).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct SortArgs {
  const void* ids;
  bool id64;
  int64_t tokens, ld_ids;
  int topk, n_experts;
  int32_t *order, *pos, *offsets;
  void* ws;
  hipStream_t stream;
};
size_t expert_sort_ws(int64_t n, int n_experts);   // bytes of SortArgs::ws
hipError_t run_expert_sort(const SortArgs& a);

// Token rows [tokens x hidden] and expert-ordered rows [tokens * topk x hidden] of one type.
struct RowsArgs {
  void* tok;          // read by gather, written by join
  void* rows;         // written by gather, read by join
  bool f32;
  int64_t tokens, hidden, ld_tok, ld_rows;
  const int32_t* pos;
  int topk;
  const float* w;     // join: the weights, or null for a plain sum
  int64_t ldw;
  hipStream_t stream;
};
hipError_t run_expert_gather(const RowsArgs& a);
hipError_t run_expert_join(const RowsArgs& a);

struct CombineGradArgs {
  const void *dy, *ys;
  bool f32;
  int64_t tokens, hidden, lddy, ldys;
  const float* w;
  int64_t ldw;
  const int32_t* pos;
  int topk;
  void* dys;          // or null
  int64_t lddys;
  float* dw;          // or null
  int64_t lddw;
  hipStream_t stream;
};
hipError_t run_expert_combine_grad(const CombineGradArgs& a);

// y = x . W^T; with offsets: rows in expert order against n_experts stacked weights.
struct WLinearArgs {
  const void* x;
  bool x_f32, y_f32;
  int64_t rows, ldx, ldy;
  const uint8_t *q, *s;
  const float* g;     // or null
  int fmt, block, layout, g_shift;
  int64_t N, K;
  int n_experts;      // 1 without offsets
  bool offsets_given; // rows in expert order (known before the offsets are)
  const int32_t* offsets;
  void* y;
  void* ws;
  hipStream_t stream;
};
bool wlinear_fits(const WLinearArgs& a);   // its tiles are no more than one launch holds (from the sizes, as below)
size_t wlinear_ws(const WLinearArgs& a);   // bytes of WLinearArgs::ws (x, y and offsets are not looked at)
hipError_t run_wlinear(const WLinearArgs& a);

}  // namespace fp4k
