// Launchers and device helpers of the 8-bit block-scaled operators (fp8_quant.hip, fp8_gemm.hip).
#pragma once
#include "experts.hpp"
#include "fp4_device.hpp"
#include "launch.hpp"

namespace fp4k {

constexpr int F8_BLOCK = 128;

enum : int { F8_VIEW_ROW = 0, F8_VIEW_COL = 1, F8_VIEW_TILE2D = 2, F8_VIEW_ROWCOL = 3 };
enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

struct F8QuantArgs {
  const void* x;
  bool f32;
  int64_t rows, cols, ld;
  int view;
  bool e8;
  uint8_t* q;
  void* s;
  uint8_t* qt;
  void* st;
  hipStream_t stream;
};
bool f8_quantize_fits(int64_t rows, int64_t cols);   // its tiles are no more than one launch holds
hipError_t run_f8_quantize(const F8QuantArgs& a);

struct F8Operand {
  const uint8_t* q;
  const void* s;
  bool e8;
  int layout;        // 0: 1D, 1: 2D, 2: transposed 2D
  int64_t rows, k;
};

hipError_t run_f8_dequantize(const F8Operand& a, void* y, bool f32, int64_t ldy, hipStream_t stream);

// The gradient of the gated projections: plain into dgu, or quantized into q / s and qt / st.
struct GatedGradArgs {
  const void *dh, *gu;
  bool f32;
  int64_t rows, f, lddh, ldgu;
  int act;
  void* dgu;         // plain, or null
  int64_t lddgu;
  bool e8;
  uint8_t* q;        // either pair may be null
  void* s;
  uint8_t* qt;
  void* st;
  hipStream_t stream;
};
bool f8_gated_grad_fits(int64_t rows, int64_t f, bool f32);   // the quantized form's tiles are no more than one launch holds
hipError_t run_gated_grad(const GatedGradArgs& a);

// y = x . W^T over one weight or over rows in expert order; gated: h = act(x . Wg^T) * (x . Wu^T).
struct F8GemmArgs {
  F8Operand x, w;    // w: expert 0's
  int n_experts;     // 1 without offsets
  bool offsets_given;
  const int32_t* offsets;
  bool gated;
  bool f32;          // an output is float32 (the sums are those of the bf16 matrix core)
  bool codes;        // gated: h as E4M3 codes
  int act;
  void* y;           // y, or h of a gated product
  int y_kind;        // 0 bf16, 1 float32, 2 E4M3 with scales ys
  int64_t ldy;
  void* ys;
  void* gu;          // gated: the projections, or null
  bool gu_f32;
  int64_t ldgu;
  void* ws;
  hipStream_t stream;
};
bool f8_gemm_fits(const F8GemmArgs& a);      // its tiles are no more than one launch holds (sizes alone)
size_t f8_gemm_ws(const F8GemmArgs& a);      // bytes of F8GemmArgs::ws (sizes alone)
void f8_gemm_form(const F8GemmArgs& a, int32_t form[4]);   // fp8_gemm_form of fp4bs_fp8.h (sizes alone)
hipError_t run_f8_gemm(const F8GemmArgs& a);

// ---- E4M3 blocks ----

// What a block's elements are multiplied by, and its scale as it is stored.
struct F8Scale {
  float enc;
  uint32_t code;     // E8M0 code, or the bits of the float32 scale
};

// From the bits of the block's largest magnitude (as integers they order like the magnitudes, with
// infinity and NaN on top). A block that is not finite gets a NaN multiplier, so that all its codes
// are NaN, and the scale one.
template <bool E8>
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), E8 ? 127u : 0x3F800000u};
  if constexpr (E8) {
    // 448 = 1.75 2^8: ceil(log2(a / 448)) = exponent(a) - 8, one more where the mantissa is above 1.75
    int c = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    c = amax == 0 ? 127 : max(c, 0);
    return {__uint_as_float((uint32_t)(254 - c) << 23), (uint32_t)c};
  } else {
    const float a = fmaxf(__uint_as_float(amax), 0x1p-100f);
    return amax == 0 ? F8Scale{1.0f, 0x3F800000u} : F8Scale{448.0f / a, __float_as_uint(a / 448.0f)};
  }
}

// four products -> four E4M3 codes, nearest-even (v_cvt_pk_fp8_f32; the products stay below 464)
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ---- activations ----

// sigmoid(x) = 1 / (1 + e^-x) by the hardware's exponential and reciprocal (each within an ulp or two)
__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// The normal distribution's P(g) and density d: with x = |g| / sqrt 2, erfc(x) = (a1 t + .. + a5 t^5) e^-x^2,
// t = 1 / (1 + a0 x), within 1.5e-7 (Abramowitz and Stegun 7.1.26; Hastings, "Approximations for Digital
// Computers"). The exponential serves the density too.
__device__ __forceinline__ void normal_f32(float g, float& p, float& d) {
  const float x = fabsf(g) * 0.70710678118654752f, e = __expf(-x * x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
  float s = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  s = __builtin_fmaf(s, t, 1.421413741f);
  s = __builtin_fmaf(s, t, -0.284496736f);
  s = __builtin_fmaf(s, t, 0.254829592f);
  const float tail = 0.5f * s * t * e;   // P(-|g|)
  p = g < 0.0f ? tail : 1.0f - tail;
  d = e * 0.3989422804014327f;
}

// p with act(g) = g p: the sigmoid, the normal distribution's P, or the sigmoid that its tanh form is,
// (1 + tanh z) / 2 = sigmoid(2 z); and act'(g) = p + g dp/dg
template <int ACT>
__device__ __forceinline__ void act_both(float g, float& p, float& slope) {
  if constexpr (ACT == ACT_SILU) {
    p = sigmoid_f32(g);
    slope = p * (1.0f + g * (1.0f - p));
  } else if constexpr (ACT == ACT_GELU) {
    float d;
    normal_f32(g, p, d);
    slope = p + g * d;
  } else {
    p = sigmoid_f32(1.5957691216057308f * (g + 0.044715f * g * g * g));
    const float c = fminf(fmaxf(g, -64.0f), 64.0f);   // (p (1 - p) is 0 from there on, and g^2 may be infinite)
    slope = p + c * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * c * c);
  }
}
template <int ACT>
__device__ __forceinline__ float act_gate(float g) {
  float p, slope;
  act_both<ACT>(g, p, slope);
  return p;
}

}  // namespace fp4k
