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
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// One 16-byte copy per lane from base + off (base wave-uniform) to LDS at dst + 16 * lane, without
// registers in between. Inline assembly, so that the compiler does not wait for it before LDS reads
// of the other buffer; wait_copies() and a barrier come before the copied bytes are read.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, char* dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 1\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"((uint32_t)reinterpret_cast<uintptr_t>(dst))
      : "memory", "m0");
}
// a wave-uniform address, kept in scalar registers
__device__ __forceinline__ const char* uniform_ptr(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Orders a wave's LDS writes before its other lanes' reads (the LDS serves a wave in order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

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

// ---------------------------------------------------------------- tile form
// A workgroup owns a BM x BN tile of one expert's outputs; WM x WN waves hold TM x TN products of
// 32x32x16 each. K advances in steps of 64. The activation rows of a step go straight from global
// memory into LDS; the weight's codes go through registers, are decoded there once per workgroup
// and written to LDS as bf16. Both are double buffered: while a step is multiplied, the next step's
// rows are in flight, its codes are decoded, and the codes of the step after it are loaded.
//
// An LDS row is 128 bytes (64 k); 16-byte chunk j of row r sits at position j ^ ((r >> 1) & 7), so
// sixteen consecutive rows reading one logical chunk cover all banks.
constexpr int BK = 64, ROWB = BK * 2;

template <int WM_, int WN_, int TM_, int TN_>
struct WTile {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NW = WM * WN, NTH = NW * 64;
  static constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  static constexpr int PIECES = BM / (8 * NW);      // 8-row pieces of x a wave copies per step
  static constexpr int TASKS = BN * 2 / NTH;        // 32-code half rows a thread decodes per step
  static constexpr int STAGE = (BM + BN) * ROWB;    // bytes of one buffer
  static_assert(PIECES * 8 * NW == BM && TASKS * NTH == BN * 2, "tile");
};

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return row * ROWB + ((chunk ^ ((row >> 1) & 7)) << 4); }

// The m-tile `mt` of the grouped rows: its expert and first row; false past the last one. The
// experts' tiles follow each other; the rows of dropped slots are the last group.
template <int BM>
__device__ __forceinline__ bool find_tile(const WParams& p, int64_t mt, int& e, int64_t& m0, int64_t& m1) {
  if (!p.offsets) {
    e = 0;
    m0 = mt * BM;
    m1 = p.rows;
    return m0 < m1;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 <= p.n_experts; e0 += 64) {
    int64_t lo = 0, hi = 0;
    if (e0 + lane <= p.n_experts) group_rows(p, e0 + lane, lo, hi);
    const int t = (int)((max(hi - lo, (int64_t)0) + BM - 1) / BM);
    int s = t;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(s, o, 64);
      if (lane >= o) s += u;
    }
    const uint64_t past = __ballot(before + s > mt);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      // wave-uniform (rows fit 31 bits)
      e = __builtin_amdgcn_readfirstlane(e0 + l);
      const int first = before + __shfl(s - t, l, 64);
      m1 = __builtin_amdgcn_readfirstlane(__shfl((int)hi, l, 64));
      m0 = __builtin_amdgcn_readfirstlane(__shfl((int)lo, l, 64) + ((int)mt - first) * BM);
      return true;
    }
    before += __shfl(s, 63, 64);
  }
  return false;
}

template <int FMT, int B, int LAYOUT, bool YF32, class T>
__global__ __launch_bounds__(T::NTH) void k_wlinear_tile(WParams p, int planes, int64_t plane_bytes, uint32_t mtiles,
                                                         uint32_t ntiles) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * T::STAGE];
  constexpr int BM = T::BM, BN = T::BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup ids go round-robin over the 8 dies: give each die a contiguous run of tiles, in
  // groups of 4 m-tiles that share the weight tile in its L2
  const uint32_t total = mtiles * ntiles, per = (total + 7) / 8;
  const uint32_t id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (id >= total) return;
  constexpr uint32_t GM = 4;
  const uint32_t grp = id / (GM * ntiles), gm = min(GM, mtiles - grp * GM), rest = id - grp * GM * ntiles;
  const int64_t mt = grp * GM + rest % gm, n0 = (int64_t)(rest / gm) * BN;
  int e;
  int64_t m0, m1;
  if (!find_tile<BM>(p, mt, e, m0, m1)) return;
  if (p.offsets && e == p.n_experts) {   // the rows of dropped slots
    const int rows = (int)min((int64_t)BM, m1 - m0), cols = (int)min((int64_t)BN, p.N - n0);
    for (int i = threadIdx.x; i < rows * BN; i += T::NTH)
      if (i % BN < cols) store1<YF32>(p.y, (m0 + i / BN) * p.ldy + n0 + i % BN, 0.0f);
    return;
  }
  const int64_t kb = p.K / 2;
  // x: lane offsets of the wave's pieces (rows past the group read its last row; not stored)
  uint32_t xoff[T::PIECES];
#pragma unroll
  for (int j = 0; j < T::PIECES; ++j) {
    const int r = (wave * T::PIECES + j) * 8 + (lane >> 3);
    const int rc = (int)min((int64_t)r, m1 - 1 - m0);
    xoff[j] = (uint32_t)(rc * p.ldx * 2) + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const char* xbase = uniform_ptr(p.x + m0 * p.ldx * 2);
  const int ksteps = (int)(p.K / BK), steps = ksteps * planes;
  // weight: this thread's half rows
  const uint8_t* qp[T::TASKS];
  const uint8_t* sp[T::TASKS];
#pragma unroll
  for (int j = 0; j < T::TASKS; ++j) {
    const int task = j * T::NTH + threadIdx.x, r = task >> 1, h = task & 1;
    const int64_t n = min(n0 + r, p.N - 1);
    qp[j] = p.q + ((int64_t)e * p.N + n) * kb + h * 16;
    const uint8_t* s = p.s + (int64_t)e * p.s_stride;
    if constexpr (LAYOUT == 0) sp[j] = s + n * (p.K / B) + h * (32 / B);
    else if constexpr (LAYOUT == 1) sp[j] = s + (n / 16) * (p.K / 16) + h * 2;
    else sp[j] = s + (int64_t)(h * 2) * (p.N / 16) + n / 16;
  }
  v4u codes[T::TASKS];
  uint32_t sc[T::TASKS][2];
  auto load_codes = [&](int step) {
    const int k = step % ksteps;
#pragma unroll
    for (int j = 0; j < T::TASKS; ++j) {
      codes[j] = *reinterpret_cast<const v4u*>(qp[j] + (int64_t)k * (BK / 2));
      if constexpr (LAYOUT == 2) {
        sc[j][0] = sp[j][(int64_t)k * 4 * (p.N / 16)];
        sc[j][1] = sp[j][(int64_t)(k * 4 + 1) * (p.N / 16)];
      } else if constexpr (B == 16) {
        const uint32_t c = *reinterpret_cast<const uint16_t*>(sp[j] + k * 4);
        sc[j][0] = c & 0xFFu;
        sc[j][1] = c >> 8;
      } else {
        sc[j][0] = sc[j][1] = sp[j][k * 2];
      }
    }
  };
  auto write_weight = [&](char* buf) {
#pragma unroll
    for (int j = 0; j < T::TASKS; ++j) {
      const int task = j * T::NTH + threadIdx.x, r = task >> 1, h = task & 1;
      const float s0 = wscale<FMT>(sc[j][0]), s1 = B == 16 ? wscale<FMT>(sc[j][1]) : s0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<v8bf*>(buf + BM * ROWB + swz(r, h * 4 + c)) = decode8_bf16<FMT>(codes[j][c], c < 2 ? s0 : s1);
    }
  };
  auto copy_x = [&](int step, char* buf) {
    const char* src = xbase + (int64_t)(step / ksteps) * plane_bytes + (int64_t)(step % ksteps) * ROWB;
#pragma unroll
    for (int j = 0; j < T::PIECES; ++j) dma16(src, xoff[j], buf + (wave * T::PIECES + j) * 1024);
  };

  v16f acc[T::TN][T::TM];
#pragma unroll
  for (int i = 0; i < T::TN; ++i)
#pragma unroll
    for (int j = 0; j < T::TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int fr = lane & 31, fk = lane >> 5;

  copy_x(0, lds);
  load_codes(0);
  write_weight(lds);
  if (steps > 1) load_codes(1);
  wait_copies();
  __syncthreads();
  for (int st = 0; st < steps; ++st) {
    char* buf = lds + (st & 1) * T::STAGE;
    char* nxt = lds + ((st & 1) ^ 1) * T::STAGE;
    if (st + 1 < steps) {
      copy_x(st + 1, nxt);
      write_weight(nxt);
      if (st + 2 < steps) load_codes(st + 2);
    }
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      v8bf a[T::TN], b[T::TM];
#pragma unroll
      for (int i = 0; i < T::TN; ++i)
        a[i] = *reinterpret_cast<const v8bf*>(buf + BM * ROWB + swz((wn * T::TN + i) * 32 + fr, kk * 2 + fk));
#pragma unroll
      for (int j = 0; j < T::TM; ++j)
        b[j] = *reinterpret_cast<const v8bf*>(buf + swz((wm * T::TM + j) * 32 + fr, kk * 2 + fk));
#pragma unroll
      for (int i = 0; i < T::TN; ++i)
#pragma unroll
        for (int j = 0; j < T::TM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    wait_copies();
    __syncthreads();
  }

  // Out: lane l of a product holds row m = l % 32 and columns n = 8 (r / 4) + 4 (l / 32) + r % 4.
  // Each wave turns 32 rows of its columns at a time through its own LDS rows (padded by 16 bytes).
  constexpr int OW = T::TN * 32, OLD = OW + 4;
  float* out = reinterpret_cast<float*>(lds) + wave * 32 * OLD;
  static_assert(T::NW * 32 * OLD * 4 <= 2 * T::STAGE, "the output rows fit the buffers");
  const int64_t c0 = n0 + wn * OW;
  const float* g = p.g ? p.g + (int64_t)e * p.g_stride : nullptr;
#pragma unroll
  for (int j = 0; j < T::TM; ++j) {
#pragma unroll
    for (int i = 0; i < T::TN; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        v4f v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r4 * 4 + r];
        *reinterpret_cast<v4f*>(out + fr * OLD + i * 32 + r4 * 8 + fk * 4) = v;
      }
    wave_lds_order();
    const int64_t mrow = m0 + (wm * T::TM + j) * 32;
#pragma unroll 4
    for (int o = lane; o < 32 * OW / 4; o += 64) {
      const int r = o / (OW / 4), c = (o % (OW / 4)) * 4;
      const v4f v = *reinterpret_cast<const v4f*>(out + r * OLD + c);
      const int64_t m = mrow + r, n = c0 + c;
      if (m < m1) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < p.N)
            store1<YF32>(p.y, m * p.ldy + n + k, v[k] * (g ? g[p.g_shift ? (n + k) >> p.g_shift : 0] : 1.0f));
      }
    }
    wave_lds_order();
  }
}

// float32 rows -> three planes of bf16 rows whose exact sum they are
__global__ __launch_bounds__(256) void k_split3(const float* __restrict__ x, int64_t ldx, int64_t rows, int64_t K,
                                                char* __restrict__ out) {
  const int64_t per = K / 8, n = rows * per, plane = rows * K * 2;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per, k = (i - r * per) * 8;
    const v4f* src = reinterpret_cast<const v4f*>(x + r * ldx + k);
    const v4f a = src[0], b = src[1];
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    v8bf part[3];
    split3(v, part);
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<v8bf*>(out + q * plane + (r * K + k) * 2) = part[q];
  }
}

template <bool F32>
__global__ __launch_bounds__(256) void k_zero_rows(char* y, int64_t rows, int64_t n, int64_t ldy) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * n; i += (int64_t)gridDim.x * 256)
    store1<F32>(y, i / n * ldy + i % n, 0.0f);
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

using Tile256 = WTile<2, 4, 4, 2>;
using Tile128 = WTile<2, 2, 2, 2>;

// Rows per expert (on average) from which the tile form is used.
bool use_tile(const WLinearArgs& a) { return a.rows / a.n_experts > 64 && a.ldx <= (int64_t(1) << 22); }

template <int FMT, int B, int LAYOUT, bool YF32, class T>
hipError_t launch_tile(const WLinearArgs& a, WParams p) {
  int planes = 1;
  if (a.x_f32) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(a.rows * (a.K / 8), 256), 8192);
    k_split3<<<grid, 256, 0, a.stream>>>((const float*)a.x, a.ldx, a.rows, a.K, (char*)a.ws);
    planes = 3;
    p.x = (const char*)a.ws;
    p.ldx = a.K;
  }
  const int64_t mt = div_up(a.rows, T::BM) + (a.offsets ? a.n_experts : 0), nt = div_up(a.N, T::BN);
  const int64_t grid = div_up(mt * nt, 8) * 8;
  k_wlinear_tile<FMT, B, LAYOUT, YF32, T><<<(uint32_t)grid, T::NTH, 0, a.stream>>>(
      p, planes, a.rows * a.K * 2, (uint32_t)mt, (uint32_t)nt);
  return hipSuccess;
}

template <int FMT, int B, int LAYOUT, bool XF32, bool YF32>
hipError_t launch(const WLinearArgs& a, const WParams& p) {
  if (use_tile(a)) {
    const int64_t big = div_up(a.rows, 256) * div_up(a.N, 256);
    if (big >= 256) return launch_tile<FMT, B, LAYOUT, YF32, Tile256>(a, p);
    return launch_tile<FMT, B, LAYOUT, YF32, Tile128>(a, p);
  }
  const dim3 grid((uint32_t)div_up(a.N, 16), (uint32_t)(a.offsets ? a.n_experts + 1 : 1));
  const int64_t avg = a.rows / a.n_experts;
  if (avg <= 16) k_wlinear_rows<FMT, B, LAYOUT, XF32, YF32, 1, 8><<<grid, 512, 0, a.stream>>>(p);
  else k_wlinear_rows<FMT, B, LAYOUT, XF32, YF32, 4, 4><<<grid, 256, 0, a.stream>>>(p);
  return hipSuccess;
}

template <int FMT, int B, int LAYOUT>
hipError_t by_types(const WLinearArgs& a, const WParams& p) {
  if (a.x_f32) return a.y_f32 ? launch<FMT, B, LAYOUT, true, true>(a, p) : launch<FMT, B, LAYOUT, true, false>(a, p);
  return a.y_f32 ? launch<FMT, B, LAYOUT, false, true>(a, p) : launch<FMT, B, LAYOUT, false, false>(a, p);
}

template <int FMT>
hipError_t by_layout(const WLinearArgs& a, const WParams& p) {
  if constexpr (FMT != FMT_E8M0) {
    if (a.block == 16 && a.layout == 0) return by_types<FMT, 16, 0>(a, p);
    if (a.block == 16 && a.layout == 1) return by_types<FMT, 16, 1>(a, p);
    if (a.block == 16) return by_types<FMT, 16, 2>(a, p);
  }
  return by_types<FMT, 32, 0>(a, p);
}

}  // namespace

// the three bf16 planes of float32 activations in the tile form
size_t wlinear_ws(const WLinearArgs& a) { return a.x_f32 && use_tile(a) ? (size_t)(3 * a.rows * a.K * 2) : 0; }

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
  const hipError_t err = a.fmt == FMT_E8M0   ? by_layout<FMT_E8M0>(a, p)
                         : a.fmt == FMT_E4M3 ? by_layout<FMT_E4M3>(a, p)
                                             : by_layout<FMT_UE5M3>(a, p);
  return err != hipSuccess ? err : hipGetLastError();
}

}  // namespace fp4k
