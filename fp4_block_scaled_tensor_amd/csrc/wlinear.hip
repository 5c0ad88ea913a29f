// y = x . W^T with bf16 or float32 activations and block-scaled FP4 weights on gfx950, for one
// weight or for rows in expert order against a stack of weights.
//
// E2M1 times a block scale has at most 6 significant bits and lies in bfloat16's range, so the
// weight decodes to bf16 without rounding and the products run on the bf16 matrix cores with
// float32 accumulation. A float32 activation is split exactly into three bf16 parts (8 + 8 + 8
// significant bits by truncation), each multiplied into the same sums.
#include "experts.hpp"

namespace fp4k {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// the value of a scale code
template <int FMT>
__device__ __forceinline__ float wscale(uint32_t c) {
  if constexpr (FMT == FMT_E8M0) return c ? __uint_as_float(c << 23) : __uint_as_float(1u << 22);
  else return dec_scale3<FMT>(c);
}

template <int FMT, int SEL>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, float sv) {
  if constexpr (FMT == FMT_E8M0) {
    // the conversion applies the scale's power of two
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sv, SEL);
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
    return pack_bf16(v[0] * sv, v[1] * sv);   // exact
  }
}

// 8 codes (one dword, element 0 in the low nibble) times their scale -> 8 bf16, exact
template <int FMT>
__device__ __forceinline__ v8bf decode8_bf16(uint32_t w, float sv) {
  const v4u r = {decode_pair<FMT, 0>(w, sv), decode_pair<FMT, 1>(w, sv), decode_pair<FMT, 2>(w, sv),
                 decode_pair<FMT, 3>(w, sv)};
  return __builtin_bit_cast(v8bf, r);
}

// 8 float32 -> three bf16 vectors whose exact sum they are. Each part keeps the upper 16 bits
// of what is left (truncation, so no part overflows); an infinity has no remainder and a NaN's
// remainder is NaN.
__device__ __forceinline__ void split3(const float* v, v8bf* part) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    v4u o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(r[2 * i]), b = __float_as_uint(r[2 * i + 1]);
      o[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      const float fa = __uint_as_float(a & 0xFFFF0000u), fb = __uint_as_float(b & 0xFFFF0000u);
      r[2 * i] = r[2 * i] == fa ? 0.0f : r[2 * i] - fa;
      r[2 * i + 1] = r[2 * i + 1] == fb ? 0.0f : r[2 * i + 1] - fb;
    }
    part[p] = __builtin_bit_cast(v8bf, o);
  }
}

struct WParams {
  const char* x;
  int64_t rows, ldx;
  const uint8_t *q, *s;
  const float* g;
  int g_shift;
  int64_t N, K;
  int n_experts;
  const int32_t* offsets;
  char* y;
  int64_t ldy;
  int64_t s_stride;   // scale codes of one expert
  int64_t g_stride;   // floats of g of one expert
};

// The rows [lo, hi) of group e (all rows without offsets); the offsets come from device memory
// and are clamped to the tensor.
__device__ __forceinline__ void group_rows(const WParams& p, int e, int64_t& lo, int64_t& hi) {
  if (!p.offsets) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = min(max((int64_t)p.offsets[e], (int64_t)0), p.rows);
  hi = e == p.n_experts ? p.rows : min(max((int64_t)p.offsets[e + 1], lo), p.rows);
}

template <bool F32>
__device__ __forceinline__ void store1(char* y, int64_t i, float v) {
  if constexpr (F32) reinterpret_cast<float*>(y)[i] = v;
  else reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)pack_bf16(v, 0.0f);
}

// Rows form: a workgroup owns 16 weight rows (one expert's, blockIdx.y) and all of the group's
// activation rows, 16 TM at a time; its waves split K and join their sums through LDS. Lane l of a
// 16x16x32 product holds weight row l % 16 and eight consecutive k of K group l / 16; the lane's
// codes come as 32 consecutive bytes (64 k), so one wave reads 128 consecutive bytes of 16 rows.
template <int FMT, int B, int LAYOUT, bool XF32, bool YF32, int TM, int NW>
__global__ __launch_bounds__(NW * 64) void k_wlinear_rows(WParams p) {
  __shared__ float red[NW][TM * 4][64];
  const int e = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, kg = lane >> 4;
  int64_t lo, hi;
  group_rows(p, e, lo, hi);
  if (lo >= hi) return;
  const int64_t n0 = (int64_t)blockIdx.x * 16, n = n0 + r;
  if (p.offsets && e == p.n_experts) {   // the rows of dropped slots
    for (int64_t i = threadIdx.x; i < (hi - lo) * 16; i += NW * 64)
      if (n0 + (i & 15) < p.N) store1<YF32>(p.y, (lo + (i >> 4)) * p.ldy + n0 + (i & 15), 0.0f);
    return;
  }
  const int64_t nr = n < p.N ? n : p.N - 1;   // rows past the weight read the last row and are not stored
  const uint8_t* q = p.q + (int64_t)e * p.N * (p.K / 2) + nr * (p.K / 2);
  const uint8_t* s = p.s + (int64_t)e * p.s_stride;
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * TM) {
    v4f acc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t kb = (int64_t)wave * 256; kb < p.K; kb += NW * 256) {
      const int64_t k0 = kb + kg * 64;
      v4u w[2] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}};
      float sv[64 / B];
#pragma unroll
      for (int i = 0; i < 64 / B; ++i) sv[i] = 0.0f;
      const bool in = k0 < p.K;
      if (in) {
        w[0] = *reinterpret_cast<const v4u*>(q + k0 / 2);
        w[1] = *reinterpret_cast<const v4u*>(q + k0 / 2 + 16);
        if constexpr (LAYOUT == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sv[i] = wscale<FMT>(s[(k0 / 16 + i) * (p.N / 16) + n0 / 16]);
        } else {
          const uint8_t* sp = LAYOUT == 1 ? s + (n0 / 16) * (p.K / 16) + k0 / 16 : s + nr * (p.K / B) + k0 / B;
          if constexpr (B == 16) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(sp);
#pragma unroll
            for (int i = 0; i < 4; ++i) sv[i] = wscale<FMT>((c >> (8 * i)) & 0xFFu);
          } else {
            const uint32_t c = *reinterpret_cast<const uint16_t*>(sp);
            sv[0] = wscale<FMT>(c & 0xFFu);
            sv[1] = wscale<FMT>(c >> 8);
          }
        }
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const v8bf b = decode8_bf16<FMT>(w[d >> 2][d & 3], sv[d * 8 / B]);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const int64_t m = m0 + t * 16 + r;
          const bool have = in && m < hi;
          if constexpr (XF32) {
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (have) {
              const v4f* xp = reinterpret_cast<const v4f*>(p.x + (m * p.ldx + k0 + d * 8) * 4);
              const v4f a0 = xp[0], a1 = xp[1];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[i] = a0[i];
                v[4 + i] = a1[i];
              }
            }
            v8bf part[3];
            split3(v, part);
#pragma unroll
            for (int i = 0; i < 3; ++i) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part[i], b, acc[t], 0, 0, 0);
          } else {
            v4u a = {0, 0, 0, 0};
            if (have) a = *reinterpret_cast<const v4u*>(p.x + (m * p.ldx + k0 + d * 8) * 2);
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), b, acc[t], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][t * 4 + i][lane] = acc[t][i];
    __syncthreads();
    // output (m, n): lane 16 (m / 4 % 4) + n of register m % 4 of tile m / 16
    for (int o = threadIdx.x; o < TM * 256; o += NW * 64) {
      const int m = o >> 4, c = o & 15;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += red[w][(m >> 4) * 4 + (m & 3)][((m >> 2) & 3) * 16 + c];
      const int64_t row = m0 + m, col = n0 + c;
      if (row < hi && col < p.N) {
        const float g = p.g ? p.g[(int64_t)e * p.g_stride + (p.g_shift ? col >> p.g_shift : 0)] : 1.0f;
        store1<YF32>(p.y, row * p.ldy + col, v * g);
      }
    }
    __syncthreads();
  }
}

template <bool F32>
__global__ __launch_bounds__(256) void k_zero_rows(char* y, int64_t rows, int64_t n, int64_t ldy) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * n; i += (int64_t)gridDim.x * 256)
    store1<F32>(y, i / n * ldy + i % n, 0.0f);
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int FMT, int B, int LAYOUT, bool XF32, bool YF32>
void launch(const WLinearArgs& a, const WParams& p) {
  const dim3 grid((uint32_t)div_up(a.N, 16), (uint32_t)(a.offsets ? a.n_experts + 1 : 1));
  const int64_t avg = a.rows / a.n_experts;
  if (avg <= 16) k_wlinear_rows<FMT, B, LAYOUT, XF32, YF32, 1, 8><<<grid, 512, 0, a.stream>>>(p);
  else k_wlinear_rows<FMT, B, LAYOUT, XF32, YF32, 4, 4><<<grid, 256, 0, a.stream>>>(p);
}

template <int FMT, int B, int LAYOUT>
void by_types(const WLinearArgs& a, const WParams& p) {
  if (a.x_f32) a.y_f32 ? launch<FMT, B, LAYOUT, true, true>(a, p) : launch<FMT, B, LAYOUT, true, false>(a, p);
  else a.y_f32 ? launch<FMT, B, LAYOUT, false, true>(a, p) : launch<FMT, B, LAYOUT, false, false>(a, p);
}

template <int FMT>
void by_layout(const WLinearArgs& a, const WParams& p) {
  if (a.block == 32) by_types<FMT, 32, 0>(a, p);
  else if constexpr (FMT != FMT_E8M0) {
    if (a.layout == 0) by_types<FMT, 16, 0>(a, p);
    else if (a.layout == 1) by_types<FMT, 16, 1>(a, p);
    else by_types<FMT, 16, 2>(a, p);
  }
}

}  // namespace

size_t wlinear_ws(const WLinearArgs&) { return 0; }

hipError_t run_wlinear(const WLinearArgs& a) {
  if (a.rows == 0 || a.N == 0) return hipSuccess;
  if (a.K == 0) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(a.rows * a.N, 256), 4096);
    if (a.y_f32) k_zero_rows<true><<<grid, 256, 0, a.stream>>>((char*)a.y, a.rows, a.N, a.ldy);
    else k_zero_rows<false><<<grid, 256, 0, a.stream>>>((char*)a.y, a.rows, a.N, a.ldy);
    return hipGetLastError();
  }
  WParams p{};
  p.x = (const char*)a.x;
  p.rows = a.rows;
  p.ldx = a.ldx;
  p.q = a.q;
  p.s = a.s;
  p.g = a.g;
  p.g_shift = a.g_shift;
  p.N = a.N;
  p.K = a.K;
  p.n_experts = a.n_experts;
  p.offsets = a.offsets;
  p.y = (char*)a.y;
  p.ldy = a.ldy;
  p.s_stride = a.layout == 0 ? a.N * (a.K / a.block) : (a.N / 16) * (a.K / 16);
  p.g_stride = a.g_shift ? div_up(a.N, int64_t(1) << a.g_shift) : 1;
  if (a.fmt == FMT_E8M0) by_layout<FMT_E8M0>(a, p);
  else if (a.fmt == FMT_E4M3) by_layout<FMT_E4M3>(a, p);
  else by_layout<FMT_UE5M3>(a, p);
  return hipGetLastError();
}

}  // namespace fp4k
