// y = x . W^T with bf16 or float32 activations and block-scaled FP4 weights on gfx950, for one
// weight or for rows in expert order against a stack of weights.
//
// E2M1 times a block scale has at most 6 significant bits and lies in bfloat16's range, so the
// weight decodes to bf16 without rounding and the products run on the bf16 matrix cores with
// float32 accumulation. (E8M0 codes 253 and 254 reach past that range, which is float32's, with the
// larger E2M1 values, and those weights are infinite.) A float32 activation is split into three bf16
// parts (8 + 8 + 8 significant bits by truncation), each multiplied into the same sums.
#include "experts.hpp"
#include "lds_copy.hpp"

namespace fp4k {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// all but the newest N of the wave's copies have landed
template <int N>
__device__ __forceinline__ void wait_all_but() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// the wave's LDS reads are done
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// a wave-uniform address, kept in scalar registers
__device__ __forceinline__ const char* uniform_ptr(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}
// this wave's copies have landed and its LDS reads are done
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

template <bool E8, int SEL>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, float sv) {
  if constexpr (E8) {
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
template <bool E8>
__device__ __forceinline__ v8bf decode8_bf16(uint32_t w, float sv) {
  const v4u r = {decode_pair<E8, 0>(w, sv), decode_pair<E8, 1>(w, sv), decode_pair<E8, 2>(w, sv),
                 decode_pair<E8, 3>(w, sv)};
  return __builtin_bit_cast(v8bf, r);
}

// 8 float32 -> three bf16 vectors whose sum they are, exactly from magnitude 2^-110 on (the last part
// holds no bits below 2^-133). Each part keeps the upper 16 bits of what is left (truncation, so no
// part overflows); an infinity has no remainder and a NaN's remainder is NaN.
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

// What both forms need beside the operands.
struct FormArgs {
  int64_t plane_bytes;   // bytes between the bf16 parts of float32 activations
  bool y_f32, y_vec;     // y_vec: rows of y take 4-element stores
  float scale_mul;       // 2^(127 - bias) of the 3-mantissa-bit scales
  int64_t s_row, s_k;    // scale codes: bytes between rows (16-row bands for 2D) and between blocks of K
  int s_band;            // log2 of the rows that share a scale row (0 or 4)
};

// The value of a scale code. E8: 2^(c - 127). Else 3 mantissa bits: the code's bits as a float32 times
// 2^(127 - bias), subnormals included.
template <bool E8>
__device__ __forceinline__ float code_value(uint32_t c, float scale_mul) {
  if constexpr (E8) return c ? __uint_as_float(c << 23) : __uint_as_float(1u << 22);
  else return __uint_as_float(c << 20) * scale_mul;
}

// ---------------------------------------------------------------- weight turns
// What limits reading a weight is the number of cache lines that the vector loads touch: lane l of a
// matrix product holds weight row l % 16 (or l % 32), so loads into that layout touch a line per
// lane, 64 of them for a kilobyte of codes or for 64 bytes of scales (measured at 28672 x 4096, one
// activation row: 26 us with such loads, 18 us with the scales' left out). So codes and scales are
// copied straight from global memory into LDS with neighbouring lanes on neighbouring bytes, a turn
// of 128 k at a time and each wave its own rows (no barrier), and read from there in the products'
// layout.
//
// A turn of 16 G rows: 64 bytes of codes of each row, then the scale codes. Words: 8 bytes (block
// 16) or 4 (block 32) of each row, a dword a lane. BYTES: 8 of each 16-row band (transposed 2D
// scales) or 4 of each row (block 32 with rows that are not whole words), a byte a lane and kept in
// a dword. Codes row r keeps its 16-byte piece j at j ^ (r / 4 % 4), so that the 16 rows of a read
// fall on different banks.
constexpr int TURN_K = 128;

template <int B, bool BYTES, int G>
struct WeightTurns {
  static constexpr int PER = B == 16 ? (BYTES ? 8 : 2) : (BYTES ? 4 : 1);   // lanes to a row's (band's) scales
  static constexpr int NSC = B == 16 ? (BYTES ? 1 : (G * 32 + 63) / 64) : (BYTES ? G : (G * 16 + 63) / 64);
  static constexpr int COPIES = G + NSC, SCALES = G * 1024, SIZE = SCALES + NSC * 256;
  uint32_t qoff[G], soff[NSC];
  const char *qbase, *sbase;
  int64_t s_turn;
  bool half;     // the weight's last turn has only its first 64 k
  int last;      // that turn

  // rows n0 (a multiple of 16, below N) .. of expert e; rows past the weight repeat its last one
  __device__ __forceinline__ void init(const WParams& p, const FormArgs& t, int e, int64_t n0) {
    const int lane = threadIdx.x & 63, nlast = (int)min((int64_t)(16 * G - 1), p.N - 1 - n0);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int row = i * 16 + (lane >> 2);
      qoff[i] = (uint32_t)(min(row, nlast) * (int)(p.K / 2)) + (((lane & 3) ^ ((row >> 2) & 3)) << 4);
    }
#pragma unroll
    for (int i = 0; i < NSC; ++i) {
      const int at = (i * 64 + lane) / PER, row = B == 16 && BYTES ? min(at, G - 1) * 16 : min(at, 16 * G - 1);
      const int64_t band = ((n0 + min(row, nlast)) >> t.s_band) - (n0 >> t.s_band);
      soff[i] = (uint32_t)(band * t.s_row + (lane % PER) * (BYTES ? t.s_k : 4));
    }
    qbase = uniform_ptr(reinterpret_cast<const char*>(p.q + ((int64_t)e * p.N + n0) * (p.K / 2)));
    sbase = uniform_ptr(reinterpret_cast<const char*>(p.s + (int64_t)e * p.s_stride + (n0 >> t.s_band) * t.s_row));
    s_turn = TURN_K / B * t.s_k;
    half = p.K % TURN_K != 0;
    last = (int)((p.K + TURN_K - 1) / TURN_K) - 1;
  }
  __device__ __forceinline__ void copy(int turn, char* to) const {
    const int lane = threadIdx.x & 63;
    const bool cut = half && turn == last;   // what lies past K: the 64 k before it instead (not used)
    const char* src = qbase + (int64_t)turn * (TURN_K / 2);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int piece = (lane & 3) ^ (((j * 16 + (lane >> 2)) >> 2) & 3);
      lds_dma16(src, cut && (piece & 2) ? qoff[j] - 32 : qoff[j], lds_offset(to + j * 1024));
    }
    src = sbase + turn * s_turn;
#pragma unroll
    for (int j = 0; j < NSC; ++j) {
      const uint32_t step = BYTES ? (uint32_t)(s_turn / 2) : 4;
      const uint32_t off = cut && PER > 1 && (lane % PER) >= PER / 2 ? soff[j] - step : soff[j];
      if constexpr (BYTES) lds_dma1(src, off, lds_offset(to + SCALES + j * 256));
      else lds_dma4(src, off, lds_offset(to + SCALES + j * 256));
    }
  }
  // the 32 codes of piece j (32 k) of a row, and their scale codes (two at block 16)
  static __device__ __forceinline__ v4u codes(const char* turn, int row, int j) {
    return *reinterpret_cast<const v4u*>(turn + row * 64 + ((j ^ ((row >> 2) & 3)) << 4));
  }
  static __device__ __forceinline__ void scales(const char* turn, int row, int j, uint32_t* sc) {
    const char* s = turn + SCALES;
    if constexpr (B == 16 && BYTES) {
      sc[0] = *reinterpret_cast<const uint32_t*>(s + ((row >> 4) * 8 + j * 2) * 4);
      sc[1] = *reinterpret_cast<const uint32_t*>(s + ((row >> 4) * 8 + j * 2 + 1) * 4);
    } else if constexpr (B == 16) {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(s + row * 8 + j * 2);
      sc[0] = v & 0xFFu;
      sc[1] = v >> 8;
    } else {
      sc[0] = sc[1] = *reinterpret_cast<const uint8_t*>(s + (row * 4 + j) * (BYTES ? 4 : 1));
    }
  }
};

// ---------------------------------------------------------------- rows form
// For few activation rows the weight's bytes are the bound. A workgroup owns 16 TN weight rows (one
// expert's, blockIdx.y) and the group's activation rows, XR (4, 8 or 16) at a time. Its waves split
// K into contiguous parts and join their sums through LDS. A wave takes a turn of its weight rows
// and 256 bytes of each activation row at a time into its own ring of D turns: the copies of D - 1
// turns are in flight while one is multiplied. Activation rows past the group repeat its last one;
// their products, and those of the 16 - XR rows of a product that are not there, are not stored.
// Activation row r (256 bytes) keeps its 16-byte piece j at j ^ r % 16, against bank conflicts.
// Measured, one row, MXFP4: 114688 x 4096 54 us (4.6 TB/s); 28672 x 4096 18.5 us, 5 to 6 us of it launch
// and ramp; 4096 x 4096 5.4 us (4.5 with three weights in turn, which the L2 holds). Three-mantissa-bit
// scales add the decode: 28672 x 4096 UE5M3 21.0 us with 2D scales, 24.4 us with a row of scales to each
// weight row, whose few bytes a turn are a line each. float32 rows, always 16 at a time and in three
// planes: 28672 x 4096 MXFP4 33 us for one, 41 us for 16.
template <bool E8_, int B_, int PLANES_, int TN_, int XR_, bool BYTES_>
struct RowsForm {
  static constexpr bool E8 = E8_, BYTES = BYTES_;
  static constexpr int B = B_, PLANES = PLANES_, TN = TN_, XR = XR_;
  using Weight = WeightTurns<B, BYTES, TN>;
  static constexpr int NW = TN == 1 && PLANES == 1 ? 8 : 4;
  static constexpr int NXC = PLANES * XR / 4;   // copies of activation rows
  static constexpr int BATCH = Weight::COPIES + NXC;
  static constexpr int XROWS = Weight::SIZE, TURN = XROWS + NXC * 1024;
  static constexpr int D = 3 * NW * TURN <= 80 * 1024 ? 3 : 2;
  static_assert(TN * 1024 <= D * TURN, "the wave's sums fit its ring");
};

template <class F>
__global__ __launch_bounds__(F::NW * 64) void k_wlinear_rows(WParams p, FormArgs t) {
  constexpr bool E8 = F::E8;
  constexpr int PLANES = F::PLANES, TN = F::TN, XR = F::XR, NW = F::NW, D = F::D;
  __shared__ __attribute__((aligned(1024))) char lds[NW * D * F::TURN];
  const int e = blockIdx.y, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kg = lane >> 4;
  int64_t lo, hi;
  group_rows(p, e, lo, hi);
  if (lo >= hi) return;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * TN);
  if (p.offsets && e == p.n_experts) {   // the rows of dropped slots
    for (int64_t i = threadIdx.x; i < (hi - lo) * (16 * TN); i += NW * 64) {
      const int64_t m = lo + i / (16 * TN), n = n0 + i % (16 * TN);
      if (n < p.N) t.y_f32 ? store1<true>(p.y, m * p.ldy + n, 0.0f) : store1<false>(p.y, m * p.ldy + n, 0.0f);
    }
    return;
  }
  const int turns = (int)((p.K + TURN_K - 1) / TURN_K), span = (turns + NW - 1) / NW;
  const int first = min(wave * span, turns - 1), mine = max(0, min(span, turns - wave * span));
  typename F::Weight weight;
  weight.init(p, t, e, n0);
  char* ring = lds + wave * (D * F::TURN);
  uint32_t xoff[XR / 4];

  for (int64_t m0 = lo; m0 < hi; m0 += XR) {
    const int mlast = (int)min(hi - 1 - m0, (int64_t)(XR - 1));
#pragma unroll
    for (int i = 0; i < XR / 4; ++i) {
      const int row = i * 4 + (lane >> 4);
      xoff[i] = (uint32_t)(min(row, mlast) * (int)(p.ldx * 2)) + (((lane & 15) ^ row) << 4);
    }
    const char* xbase = uniform_ptr(p.x + m0 * p.ldx * 2);
    auto copy = [&](int i) {   // this wave's turn i
      char* to = ring + (i % D) * F::TURN;
      weight.copy(first + i, to);
      const bool cut = weight.half && first + i == weight.last;
#pragma unroll
      for (int o = 0; o < PLANES; ++o) {
        const char* src = xbase + o * t.plane_bytes + (int64_t)(first + i) * (TURN_K * 2);
#pragma unroll
        for (int j = 0; j < XR / 4; ++j) {
          const int piece = (lane & 15) ^ (j * 4 + (lane >> 4));
          lds_dma16(src, cut && (piece & 8) ? xoff[j] - 128 : xoff[j], lds_offset(to + F::XROWS + (o * (XR / 4) + j) * 1024));
        }
      }
    };

    v4f acc[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (i < mine) copy(i);
    for (int i = 0; i < mine; ++i) {
      if (D == 3 && i + 2 < mine) wait_all_but<2 * F::BATCH>();
      else if (i + 1 < mine) wait_all_but<F::BATCH>();
      else wait_all_but<0>();
      const char* from = ring + (i % D) * F::TURN;
      v4u w[TN], x[PLANES][4];
      uint32_t sc[TN][2];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        w[j] = F::Weight::codes(from, j * 16 + r, kg);
        F::Weight::scales(from, j * 16 + r, kg, sc[j]);
      }
#pragma unroll
      for (int o = 0; o < PLANES; ++o)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int row = r % XR;
          x[o][d] = *reinterpret_cast<const v4u*>(from + F::XROWS + o * (XR * 256) + row * 256 + (((kg * 4 + d) ^ row) << 4));
        }
      wait_lds();
      if (i + D < mine) copy(i + D);
      if (weight.half && first + i == weight.last && kg >= 2) {   // past K
#pragma unroll
        for (int j = 0; j < TN; ++j) w[j] = v4u{0, 0, 0, 0};
#pragma unroll
        for (int o = 0; o < PLANES; ++o)
#pragma unroll
          for (int d = 0; d < 4; ++d) x[o][d] = v4u{0, 0, 0, 0};
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const float sv = code_value<E8>(sc[j][d / 2], t.scale_mul);
          const v8bf b = decode8_bf16<E8>(w[j][d], sv);
#pragma unroll
          for (int o = 0; o < PLANES; ++o)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x[o][d]), b, acc[j], 0, 0, 0);
        }
    }
    // the waves' sums, each in its own ring (its copies have landed and been read)
    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[(i * 4 + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    // output (m, n): lane 16 (m / 4) + n % 16 of register m % 4 of product n / 16
    const int rows = (int)min(hi - m0, (int64_t)XR);
    for (int o = threadIdx.x; o < rows * 16 * TN; o += NW * 64) {
      const int m = o / (16 * TN), c = o % (16 * TN);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w)
        v += reinterpret_cast<const float*>(lds + w * (D * F::TURN))[((c >> 4) * 4 + (m & 3)) * 64 + (m >> 2) * 16 + (c & 15)];
      const int64_t row = m0 + m, col = n0 + c;
      if (col < p.N) {
        if (p.g) v *= p.g[(int64_t)e * p.g_stride + (p.g_shift ? col >> p.g_shift : 0)];
        t.y_f32 ? store1<true>(p.y, row * p.ldy + col, v) : store1<false>(p.y, row * p.ldy + col, v);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- tile form
// A workgroup owns a BM x 256 tile of one expert's outputs: four waves, each all BM = 32 TM rows of
// x and 64 of the weight's rows (TM x 2 products of 32x32x16), or for BM = 256 eight waves with 32 of
// the weight's rows each, two to a SIMD. K advances in steps of 64. Bound by the matrix cores, which
// are busy 65% of the cycles (8192 rows over eight experts, 4096 -> 14336, MXFP4: 0.88 to 0.92 ms; a
// plain 8192 x 4096 -> 14336 product 754 us, 1.28 PFLOP/s, the library's bf16 product 645 us).
//
// A wave needs its weight rows for itself alone, so it copies their codes and scales a turn of 128 k
// at a time and decodes them in registers: lane l holds row l % 32 and the 32 codes of K half l / 32
// of a step, which feed four products (the order of k inside a step is free as long as both operands
// agree). The rows of x, which every wave needs, are copied into LDS a step at a time, NXB steps
// deep (NXB below). Staging the decoded weight in LDS instead, with 128 x 64 outputs to a wave, was slower: 1.24
// ms against 0.96 for 8192 rows of eight experts, 4096 -> 14336.
//
// Fragments are read one product group ahead. The barrier of a step stands before its last group:
// by then the step's own reads are done and the next step's rows have landed, so the next buffer's
// first fragments load under the last group's products and the freed buffer takes the rows of the
// step after. The next step's codes are decoded in place, group by group, behind their last use.
//
// An LDS row is 128 bytes (64 k); 16-byte chunk j of row r sits at position j ^ ((r >> 1) & 7), so
// sixteen consecutive rows reading one logical chunk cover all banks.
constexpr int BK = 64, ROWB = BK * 2;
constexpr int TILE_BN = 256;   // columns (weight rows) of a tile

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return row * ROWB + ((chunk ^ ((row >> 1) & 7)) << 4); }

// The m-tiles of the grouped rows: the experts' tiles follow each other, the rows of dropped slots
// are the last group. Lane l holds group l of the current 64 (all of them for up to 63 experts).
template <int BM>
struct TileMap {
  int lo, hi, tiles, upto;   // rows, tiles, tiles of this and the groups before it (in the 64)
  __device__ __forceinline__ void load(const WParams& p, int g0) {
    const int lane = threadIdx.x & 63;
    int64_t a = 0, b = 0;
    if (g0 + lane <= p.n_experts) group_rows(p, g0 + lane, a, b);
    lo = (int)a;   // rows fit 31 bits
    hi = (int)b;
    tiles = (max(hi - lo, 0) + BM - 1) / BM;
    upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(upto, o, 64);
      if (lane >= o) upto += u;
    }
  }
  // all tiles; leaves the first 64 groups loaded
  __device__ __forceinline__ uint32_t count(const WParams& p) {
    int n = 0;
    for (int g0 = (p.n_experts / 64) * 64; g0 >= 0; g0 -= 64) {
      load(p, g0);
      n += __shfl(upto, 63, 64);
    }
    return __builtin_amdgcn_readfirstlane(n);
  }
  // after count(): tile mt's group, first row and the group's end, wave-uniform; mt is below the count
  __device__ __forceinline__ void find(const WParams& p, int mt, int& e, int64_t& m0, int64_t& m1) {
    int before = 0;
    for (int g0 = 0;;) {
      const uint64_t past = __ballot(before + upto > mt);
      if (past) {
        const int l = __ffsll((unsigned long long)past) - 1;
        e = __builtin_amdgcn_readfirstlane(g0 + l);
        m1 = __builtin_amdgcn_readfirstlane(__shfl(hi, l, 64));
        m0 = __builtin_amdgcn_readfirstlane(__shfl(lo, l, 64) + (mt - before - __shfl(upto - tiles, l, 64)) * BM);
        return;
      }
      before += __shfl(upto, 63, 64);
      g0 += 64;
      load(p, g0);
    }
  }
};

struct TileArgs {
  FormArgs f;
  uint32_t mtiles, ntiles;   // mtiles: an upper bound with offsets
  int slices;                // parts of K, each with its own output rows in `part`
  float* part;               // [slices][rows][N] sums of a split K (without g), or null: write y
};

// E8: power-of-two scales (block 32), else 3-mantissa-bit ones with block B. PLANES: bf16 parts of x.
template <bool E8_, int B_, int PLANES_, int TM_, bool BYTES_>
struct TileForm {
  static constexpr bool E8 = E8_;
  static constexpr int B = B_, PLANES = PLANES_, TM = TM_;
  // eight waves of 256 x 32 outputs for the tallest tile, else four of 32 TM x 64
  static constexpr int NW = TM == 8 ? 8 : 4, TN = TILE_BN / 32 / NW;
  static constexpr int BM = TM * 32, STAGE = BM * ROWB, PIECES = BM / 8 / NW;
  // Three below 8 would take the LDS of a second workgroup, and gave little where there is only one: 77
  // rows 28672 x 4096 MXFP4 46.1 -> 44.0 us, 4096 x 14336 the same, 20 rows 31.1 -> 31.4.
  static constexpr int NXB = TM == 8 ? 3 : 2;
  using Weight = WeightTurns<B, BYTES_, TN * 2>;
  static constexpr int WBYTES = 2 * Weight::SIZE;          // a wave's two turns
  static constexpr int OW = TN * 32, OLD = OW + 4;         // a wave's output columns, padded by 16 bytes
  static constexpr int LDS = NXB * STAGE + NW * WBYTES;
  static_assert(NW * 32 * OLD * 4 <= LDS, "the output rows fit the buffers");
};

template <class F>
__global__ __launch_bounds__(F::NW * 64, 2) void k_wlinear_tile(WParams p, TileArgs t) {
  constexpr bool E8 = F::E8;
  constexpr int PLANES = F::PLANES, TM = F::TM, TN = F::TN, TILE_NW = F::NW, BM = F::BM, STAGE = F::STAGE;
  constexpr int PIECES = F::PIECES, OW = F::OW, OLD = F::OLD, NXB = F::NXB;
  __shared__ __attribute__((aligned(1024))) char lds[F::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  TileMap<BM> map;
  const uint32_t mtiles = p.offsets ? map.count(p) : t.mtiles;
  // workgroup ids go round-robin over the 8 dies: give each die a contiguous run of the tiles that
  // there are (not of those that there might be: the dies would be loaded unevenly), in groups of 4
  // m-tiles that share the weight tile in its L2
  const uint32_t tiles = mtiles * t.ntiles, total = tiles * t.slices, per = (total + 7) / 8;
  const uint32_t in_die = blockIdx.x >> 3, all = (blockIdx.x & 7) * per + in_die;
  if (in_die >= per || all >= total) return;
  const uint32_t slice = all / tiles, id = all - slice * tiles;
  constexpr uint32_t GM = 4;
  const uint32_t grp = id / (GM * t.ntiles), gm = min(GM, mtiles - grp * GM), rest = id - grp * GM * t.ntiles;
  const int mt = grp * GM + rest % gm;
  const int64_t n0 = (int64_t)(rest / gm) * TILE_BN;
  int e = 0;
  int64_t m0 = (int64_t)mt * BM, m1 = p.rows;
  if (p.offsets) map.find(p, mt, e, m0, m1);
  char* y = t.part ? reinterpret_cast<char*>(t.part + (int64_t)slice * p.rows * p.N) : p.y;
  const int64_t ldy = t.part ? p.N : p.ldy;
  const bool y_f32 = t.part || t.f.y_f32;
  if (p.offsets && e == p.n_experts) {   // the rows of dropped slots
    const int rows = (int)min((int64_t)BM, m1 - m0), cols = (int)min((int64_t)TILE_BN, p.N - n0);
    for (int i = threadIdx.x; i < rows * TILE_BN; i += TILE_NW * 64)
      if (i % TILE_BN < cols) {
        const int64_t at = (m0 + i / TILE_BN) * ldy + n0 + i % TILE_BN;
        y_f32 ? store1<true>(y, at, 0.0f) : store1<false>(y, at, 0.0f);
      }
    return;
  }

  // x: lane offsets of the wave's 8-row pieces (rows past the group read its last row; not stored)
  uint32_t xoff[PIECES];
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int r = (wave * PIECES + j) * 8 + (lane >> 3);
    const int rc = (int)min((int64_t)r, m1 - 1 - m0);
    xoff[j] = (uint32_t)(rc * p.ldx * 2) + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  // this slice's steps of K, whole turns (two steps) but for the last
  const int ksteps = (int)(p.K / BK), turns = (ksteps + 1) / 2;
  const int turn0 = (int)((int64_t)turns * slice / t.slices), turn1 = (int)((int64_t)turns * (slice + 1) / t.slices);
  const int k0 = turn0 * 2, k1 = min(turn1 * 2, ksteps);
  const char* xsrc = uniform_ptr(p.x + m0 * p.ldx * 2 + (int64_t)k0 * ROWB);   // the next rows to copy
  const int steps = (k1 - k0) * PLANES;
  int xplane = 0;
  auto copy_x = [&](char* buf) {
#pragma unroll
    for (int j = 0; j < PIECES; ++j) lds_dma16(xsrc, xoff[j], lds_offset(buf + (wave * PIECES + j) * 1024));
    if (PLANES == 1) {
      xsrc += ROWB;
    } else {
      const bool wrap = ++xplane == PLANES;
      xsrc += wrap ? ROWB - (PLANES - 1) * t.f.plane_bytes : t.f.plane_bytes;
      xplane = wrap ? 0 : xplane;
    }
  };

  // weight: this wave's rows (waves past the weight's last row take its last rows; not stored)
  const int fr = lane & 31, fk = lane >> 5;
  typename F::Weight weight;
  weight.init(p, t.f, e, min(n0 + wave * OW, (p.N - 1) & ~(int64_t)15));
  char* wring = lds + NXB * STAGE + wave * F::WBYTES;
  v4u codes[TN];
  uint32_t sc[TN][2];
  auto take_codes = [&](int k) {   // the codes of step k, whose turn has landed
    const char* turn = wring + ((k >> 1) & 1) * F::Weight::SIZE;
    const int piece = (k & 1) * 2 + fk;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      codes[i] = F::Weight::codes(turn, i * 32 + fr, piece);
      F::Weight::scales(turn, i * 32 + fr, piece, sc[i]);
    }
  };
  auto decode = [&](int i, int s) {   // dword s: k = 32 (lane / 32) + 8 s ..
    const float sv = code_value<E8>(sc[i][s / 2], t.f.scale_mul);
    return decode8_bf16<E8>(codes[i][s], sv);
  };

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  weight.copy(turn0, wring + (turn0 & 1) * F::Weight::SIZE);
  if (turn0 + 1 < turn1) weight.copy(turn0 + 1, wring + ((turn0 + 1) & 1) * F::Weight::SIZE);
  char* xbuf[NXB];   // the rows of this step, the next ..
#pragma unroll
  for (int i = 0; i < NXB; ++i) {
    xbuf[i] = lds + i * STAGE;
    if (i < steps) copy_x(xbuf[i]);
  }
  wait_copies();
  __syncthreads();
  v8bf bw[TN][4];   // the decoded weight of a step, dword by dword
  take_codes(k0);
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int i = 0; i < TN; ++i) bw[i][s] = decode(i, s);
  v8bf ax[2][TM];
  auto read_x = [&](const char* from, int s, v8bf* to) {
#pragma unroll
    for (int j = 0; j < TM; ++j) to[j] = *reinterpret_cast<const v8bf*>(from + swz(j * 32 + fr, fk * 4 + s));
  };
  read_x(xbuf[0], 0, ax[0]);
  int plane = 0, k = k0;
  for (int st = 0; st < steps; ++st) {
    const bool first = PLANES == 1 || plane == 0, last = PLANES == 1 || plane == PLANES - 1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 3) {
        // The next step's rows have landed, and this wave's reads of this step's are done. The newest
        // copies are of rows (codes are copied before the rows of a step), so the codes have, too.
        // (Past the last step: an unused read of another buffer, so that no path joins here with this
        // step's fragments still being waited for.)
        if (NXB == 3 && st + 2 < steps) wait_all_but<PIECES>();
        else wait_all_but<0>();
        wait_lds();
        __syncthreads();
        read_x(xbuf[1], 0, ax[0]);
      } else {
        read_x(xbuf[0], s + 1, ax[(s + 1) & 1]);
      }
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bw[i][s], ax[s & 1][j], acc[i][j], 0, 0, 0);
      if (s == 3) {
        // The turn whose last codes this step took, and this step's rows, make room. Behind the
        // group's products: issued before them, the copies left the matrix cores idle (801 us
        // against 740 for 8192 x 4096 -> 14336).
        if (last && (k & 1) == 0 && (k >> 1) + 2 < turn1) weight.copy((k >> 1) + 2, wring + ((k >> 1) & 1) * F::Weight::SIZE);
        if (st + NXB < steps) copy_x(xbuf[0]);
      }
      // group 0 decodes this step's last dword; groups 1 to 3 replace dwords 0 to 2, whose products
      // are under way, by the next step's
      if (s == 0 ? first : last) {
#pragma unroll
        for (int i = 0; i < TN; ++i) bw[i][(s + 3) & 3] = decode(i, (s + 3) & 3);
      }
      if (s == 0 && last) take_codes(k + 1);   // (past the last step: unused bytes of the ring)
      // per TN products one fragment read and a share of the decoding
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, TN, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, ((E8 ? 6 : 19) * TN + TM - 1) / TM, 0);
      }
    }
    if (PLANES > 1) plane = last ? 0 : plane + 1;
    if (last) ++k;
    char* const b = xbuf[0];
#pragma unroll
    for (int i = 0; i + 1 < NXB; ++i) xbuf[i] = xbuf[i + 1];
    xbuf[NXB - 1] = b;
  }

  // Out: lane l of a product holds row m = l % 32 and columns n = 8 (r / 4) + 4 (l / 32) + r % 4.
  // Each wave turns 32 rows of its columns at a time through its own LDS rows.
  float* out = reinterpret_cast<float*>(lds) + wave * 32 * OLD;
  const int64_t c0 = n0 + wave * OW;
  // parts of a split K are joined before g multiplies them
  const float* g = p.g && !t.part ? p.g + (int64_t)e * p.g_stride : nullptr;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        v4f v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r4 * 4 + r];
        *reinterpret_cast<v4f*>(out + fr * OLD + i * 32 + r4 * 8 + fk * 4) = v;
      }
    wave_order();
#pragma unroll 4
    for (int o = lane; o < 32 * OW / 4; o += 64) {
      const int r = o / (OW / 4), c = (o % (OW / 4)) * 4;
      const v4f v = *reinterpret_cast<const v4f*>(out + r * OLD + c);
      const int64_t m = m0 + j * 32 + r, n = c0 + c;
      if (m >= m1 || n >= p.N) continue;
      const float gn = g ? g[p.g_shift ? n >> p.g_shift : 0] : 1.0f;   // stripes are multiples of 16 columns
      const int64_t at = m * ldy + n;
      if (t.f.y_vec && n + 4 <= p.N) {
        if (y_f32) *reinterpret_cast<v4f*>(y + at * 4) = v4f{v[0] * gn, v[1] * gn, v[2] * gn, v[3] * gn};
        else *reinterpret_cast<uint64_t*>(y + at * 2) =
                 (uint64_t)pack_bf16(v[2] * gn, v[3] * gn) << 32 | pack_bf16(v[0] * gn, v[1] * gn);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < p.N) y_f32 ? store1<true>(y, at + q, v[q] * gn) : store1<false>(y, at + q, v[q] * gn);
      }
    }
    wave_order();
  }
}

// The groups of a wave's rows: the last whose rows start at or before each. Up to 63 experts lane l holds
// offset l, and a row's group is the number of offsets up to it less one, so a wave looks one row up after
// another without a load (its columns are of few rows); else by bisection. Every lane takes part. (1590
// rows over 15 experts, 1920 -> 1102: 42 us for the whole product, 45 by bisection.)
struct GroupOf {
  int offset;
  __device__ __forceinline__ void init(const WParams& p) {
    const int lane = threadIdx.x & 63;
    offset = p.offsets && p.n_experts < 64 && lane <= p.n_experts ? p.offsets[lane] : INT32_MAX;
  }
  __device__ __forceinline__ int find(const WParams& p, int64_t row) const {   // rows fit 31 bits
    if (!p.offsets) return 0;
    if (p.n_experts < 64) {
      int e = -1;
      for (uint64_t left = ~0ull; left;) {
        const int r = __builtin_amdgcn_readfirstlane(__shfl((int)row, __ffsll((unsigned long long)left) - 1, 64));
        const int g = __popcll(__ballot(offset <= r)) - 1;
        if ((int)row == r) e = g;
        left &= ~__ballot((int)row == r);
      }
      return max(e, 0);
    }
    int lo = 0, hi = p.n_experts;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.offsets[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// The slices' sums in slice order, times g, rounded once to y's type; V = 4 columns at a time where rows
// of y and N allow it: 48 x 4096 -> 14336 bf16 33.9 -> 31.5 us, 200 x 14336 -> 4096 bf16 49.9 -> 46.5 us,
// 128 x 4096 -> 14336 float32 64.1 -> 62.5 us for the whole product, one column at a time against four.
template <bool YF32, int V>
__global__ __launch_bounds__(256) void k_join_slices(const float* __restrict__ part, int slices, WParams p) {
  const int64_t n = p.rows * p.N, per = p.N / V, all = p.rows * per;
  GroupOf groups;
  if (p.g) groups.init(p);
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < all; i0 += (int64_t)gridDim.x * 256) {
    const int64_t i = min(i0 + threadIdx.x, all - 1);   // (lanes past the end repeat the last)
    const int64_t row = i / per, col = i % per * V, at = row * p.ldy + col;
    float g = 1.0f;   // V columns share it: stripes are multiples of 16 columns
    if (p.g) {
      const int e = groups.find(p, row);
      if (e < p.n_experts) g = p.g[(int64_t)e * p.g_stride + (p.g_shift ? col >> p.g_shift : 0)];   // else zeros
    }
    if constexpr (V == 4) {
      v4f v = *reinterpret_cast<const v4f*>(part + i * 4);
      for (int s = 1; s < slices; ++s) {
        const v4f u = *reinterpret_cast<const v4f*>(part + s * n + i * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += u[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= g;
      if constexpr (YF32) *reinterpret_cast<v4f*>(p.y + at * 4) = v;
      else *reinterpret_cast<uint64_t*>(p.y + at * 2) = (uint64_t)pack_bf16(v[2], v[3]) << 32 | pack_bf16(v[0], v[1]);
    } else {
      float v = part[i];
      for (int s = 1; s < slices; ++s) v += part[s * n + i];
      store1<YF32>(p.y, at, v * g);
    }
  }
}

// float32 rows -> three planes of bf16 rows whose sum they are (split3)
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

// A grid holds less than 2^32 threads; what is more is cut off without an error.
constexpr int64_t MAX_THREADS = (int64_t(1) << 32) - 1;

// The tile form is used from more than 16 rows per expert (on average) on, and for weights of more rows
// than a grid of the rows form holds (8 threads to each row of such a weight). Measured, us in the rows
// form / the tile form. Eight experts 14336 x 4096, 16 rows each: MXFP4 86.7 / 89.1, UE5M3 105 / 97; 24
// rows 104 / 109, 128 / 119. One weight, 20 rows: 28672 x 4096 MXFP4 30.2 / 31.1, UE5M3 40.1 / 34.8; 64
// rows 53.9 / 43.2, 71.0 / 47.5. Where there are few tiles the rows form would be ahead for longer: 4096 x
// 4096, 20 rows 8.5 / 16.1, 64 rows 13.6 / 24.2; 4096 x 14336, 20 rows 20.8 / 27.2, 64 rows 39.6 / 33.8.
// float32 activations, 17 rows (20 in the tile form): 28672 x 4096 64 / 49, 4096 x 4096 16 / 23.
bool use_tile(const WLinearArgs& a) { return a.rows / a.n_experts > 16 || a.N * 8 > MAX_THREADS - 512; }

struct TilePlan {
  int tm;          // 32-row products per tile
  int64_t mt, nt;  // tiles, at most
  int slices;      // parts of K
};

// The tile height with the least rounds of tiles over the compute units times the time of a tile,
// which is about that of its products and one more. Measured, 8192 rows 4096 -> 14336: 113, 61 and
// 42 us a round for tm 8, 4 and 2; 2048 rows 4096 -> 6144: 118 us at 8 (192 tiles), 139 at 4 (384).
// A K long enough is split where the tiles alone leave compute units idle; the
// low tiles, which are bound by latency, into two workgroups to a unit (24 rows 4096 -> 28672: 37 us, 45 with one).
TilePlan plan_tiles(const WLinearArgs& a) {
  const int64_t cus = device_cu_count(), groups = a.offsets_given ? a.n_experts : 0, ksteps = a.K / BK;
  TilePlan best{};
  double least = 0;
  for (int tm : {8, 4, 3, 2, 1}) {
    TilePlan t;
    t.tm = tm;
    t.nt = div_up(a.N, TILE_BN);
    t.mt = div_up(a.rows, tm * 32) + groups;
    const int64_t tiles = (div_up(a.rows, tm * 32) + groups / 2) * t.nt;   // an expert's last tile is half full
    t.slices = (int)std::max<int64_t>(1, std::min<int64_t>((tm <= 2 ? 2 : 1) * cus / tiles, ksteps / 4));
    const double cost = (double)div_up(tiles * t.slices, cus) * (tm + 1) / t.slices;
    if (best.tm == 0 || cost < least) {
      best = t;
      least = cost;
    }
  }
  return best;
}

// workgroups of a plan, whole rounds of the eight dies
int64_t tile_grid(const TilePlan& t) { return div_up(t.mt * t.nt * t.slices, 8) * 8; }

// the bf16 parts of float32 activations, at the start of the workspace
size_t planes_bytes(const WLinearArgs& a) { return a.x_f32 ? (size_t)div_up(3 * a.rows * a.K * 2, 256) * 256 : 0; }

template <bool E8, int B, int PLANES>
void launch(const WLinearArgs& a, const WParams& p, const FormArgs& f) {
  using std::integral_constant;
  // scale codes byte by byte where a turn's are not aligned words
  const bool bytes = f.s_k != 1 || (B == 32 && a.K % TURN_K != 0);
  if (!use_tile(a)) {
    const uint32_t groups = a.offsets ? a.n_experts + 1 : 1;
    // As many products to an activation fragment as leave no compute unit without a workgroup. Measured,
    // us with 1 / 2 / 4, MXFP4, 4 rows: 4096 x 4096 5.4 / 6.7 / 8.4, 28672 x 4096 21.8 / 19.2 / 19.1 (16
    // rows: 34.6 / 24.2 / 21.7).
    const int64_t cus = device_cu_count(), each = a.n_experts;
    const int tn = PLANES == 1 && div_up(a.N, 64) * each >= cus ? 4 : div_up(a.N, 32) * each >= cus ? 2 : 1;
    auto go = [&](auto tn_, auto xr_, auto bytes_) {
      using F = RowsForm<E8, B, PLANES, decltype(tn_)::value, decltype(xr_)::value, decltype(bytes_)::value>;
      const dim3 grid((uint32_t)div_up(a.N, 16 * F::TN), groups);
      k_wlinear_rows<F><<<grid, F::NW * 64, 0, a.stream>>>(p, f);
    };
    auto with_bytes = [&](auto tn_, auto xr_) { bytes ? go(tn_, xr_, std::true_type{}) : go(tn_, xr_, std::false_type{}); };
    // Activation rows at a time. A group with more rows reads its weight again (from the caches); rows that
    // are not there cost copies and LDS. Measured, us with 4 / 8 / 16 at a time, MXFP4: one weight 28672 x
    // 4096, 1 row 18.5 / 18.9 / 19.4, 5 rows 28.6 / 19.4 / 20.0, 9 rows 38.0 / 29.5 / 20.6. Experts with rows
    // by chance have more than the average in some: eight of 14336 x 4096, on average 1 row 45.6 / 47.1 /
    // 48.6, 2 rows 56.1 / 51.9 / 53.8, 4 rows 65.8 / 57.1 / 59.4, 6 rows 92.2 / 64.8 / 62.0; 64 of 1024 x
    // 2048, 1 row 13.8 / 14.1 / 14.5, 2 rows 19.5 / 17.7 / 18.2, 5 rows 27.9 / 22.1 / 19.5.
    const int64_t avg = div_up(a.rows, a.n_experts);
    const int xr = a.offsets ? (avg <= 1 ? 4 : avg <= 4 ? 8 : 16) : (avg <= 4 ? 4 : avg <= 8 ? 8 : 16);
    auto with_rows = [&](auto tn_) {
      if constexpr (PLANES == 1) {
        if (xr == 4) return with_bytes(tn_, integral_constant<int, 4>{});
        if (xr == 8) return with_bytes(tn_, integral_constant<int, 8>{});
      }
      with_bytes(tn_, integral_constant<int, 16>{});
    };
    if constexpr (PLANES == 1) {
      if (tn == 4) return with_rows(integral_constant<int, 4>{});
    }
    if (tn == 2) with_rows(integral_constant<int, 2>{});
    else with_rows(integral_constant<int, 1>{});
    return;
  }
  const TilePlan plan = plan_tiles(a);
  TileArgs t{};
  t.f = f;
  t.mtiles = (uint32_t)plan.mt;
  t.ntiles = (uint32_t)plan.nt;
  t.slices = plan.slices;
  if (plan.slices > 1) {
    t.part = reinterpret_cast<float*>((char*)a.ws + planes_bytes(a));
    t.f.y_vec = a.N % 4 == 0;
  }
  const uint32_t grid = (uint32_t)tile_grid(plan);
  auto go = [&](auto tm_) {
    constexpr int TM = decltype(tm_)::value;
    if (bytes) {
      using F = TileForm<E8, B, PLANES, TM, true>;
      k_wlinear_tile<F><<<grid, F::NW * 64, 0, a.stream>>>(p, t);
    } else {
      using F = TileForm<E8, B, PLANES, TM, false>;
      k_wlinear_tile<F><<<grid, F::NW * 64, 0, a.stream>>>(p, t);
    }
  };
  if (plan.tm == 1) go(integral_constant<int, 1>{});
  else if (plan.tm == 2) go(integral_constant<int, 2>{});
  else if (plan.tm == 3) go(integral_constant<int, 3>{});
  else if (plan.tm == 4) go(integral_constant<int, 4>{});
  else go(integral_constant<int, 8>{});
  if (t.part) {
    auto join = [&](auto f32, auto v) {
      constexpr bool YF32 = decltype(f32)::value;
      constexpr int V = decltype(v)::value;
      const uint32_t join_grid = (uint32_t)std::min<int64_t>(div_up(a.rows * a.N / V, 256), 4096);
      k_join_slices<YF32, V><<<join_grid, 256, 0, a.stream>>>(t.part, t.slices, p);
    };
    const bool vec = f.y_vec && a.N % 4 == 0;
    auto typed = [&](auto f32) {
      if (vec) join(f32, integral_constant<int, 4>{});
      else join(f32, integral_constant<int, 1>{});
    };
    if (a.y_f32) typed(std::true_type{});
    else typed(std::false_type{});
  }
}

}  // namespace

bool wlinear_fits(const WLinearArgs& a) {
  if (a.rows == 0 || a.N == 0 || a.K == 0 || !use_tile(a)) return true;
  const TilePlan t = plan_tiles(a);
  return tile_grid(t) * (t.tm == 8 ? 512 : 256) <= MAX_THREADS;
}

// the bf16 parts of float32 activations and the sums of a split K
size_t wlinear_ws(const WLinearArgs& a) {
  if (a.rows == 0 || a.N == 0 || a.K == 0) return 0;
  const int slices = use_tile(a) ? plan_tiles(a).slices : 1;
  return planes_bytes(a) + (slices > 1 ? (size_t)slices * a.rows * a.N * 4 : 0);
}

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
  FormArgs f{};
  f.plane_bytes = a.rows * a.K * 2;
  f.y_f32 = a.y_f32;
  const int64_t esz = a.y_f32 ? 4 : 2;
  f.y_vec = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % (4 * esz) == 0;
  f.scale_mul = a.fmt == FMT_E4M3 ? 0x1p120f : 0x1p112f;
  f.s_band = a.layout == 0 ? 0 : 4;
  f.s_row = a.layout == 0 ? a.K / a.block : a.layout == 1 ? a.K / 16 : 1;
  f.s_k = a.layout == 2 ? a.N / 16 : 1;
  if (a.x_f32) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(a.rows * (a.K / 8), 256), 8192);
    k_split3<<<grid, 256, 0, a.stream>>>((const float*)a.x, a.ldx, a.rows, a.K, (char*)a.ws);
    p.x = (const char*)a.ws;
    p.ldx = a.K;
  }
  if (a.fmt == FMT_E8M0) a.x_f32 ? launch<true, 32, 3>(a, p, f) : launch<true, 32, 1>(a, p, f);
  else if (a.block == 16) a.x_f32 ? launch<false, 16, 3>(a, p, f) : launch<false, 16, 1>(a, p, f);
  else a.x_f32 ? launch<false, 32, 3>(a, p, f) : launch<false, 32, 1>(a, p, f);
  return hipGetLastError();
}

}  // namespace fp4k
