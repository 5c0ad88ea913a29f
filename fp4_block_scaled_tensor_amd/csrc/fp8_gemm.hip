// y = x . W^T over two E4M3 operands with one scale to each block of 128, for one weight or for rows
// in expert order against a stack of weights, and the gated projections h = act(x . Wg^T) * (x . Wu^T)
// as one product whose tiles hold both rows of each feature.
//
// A block of 128 k is one 16x16x128 matrix product per 16 x 16 outputs. With E8M0 scales the matrix
// core applies both (v_mfma_scale_f32_16x16x128_f8f6f4) and accumulates over all of K; with float32
// scales each block's product starts from zero and is multiplied into the sums on the vector unit.
//
// The matrix core adds E4M3 products in a window narrower than float32: on normally distributed codes a
// block's sum is off by 1.5e-5 of its norm, whatever the instruction (16x16x128, 16x16x32) and however
// few of its products are not zero. That is under a hundredth of a bf16 output's own rounding (1.7e-3) and
// far below an E4M3 one's, so those outputs take it. Float32 outputs do not: for them the codes
// are widened to bf16 (exact) and go through the bf16 matrix core, whose block sums are off by 1e-8, at
// less than half the rate.
#include "fp8.hpp"
#include "lds_copy.hpp"
#include "row_groups.hpp"

namespace fp4k {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// all but the newest N of the wave's copies have landed
template <int N>
__device__ __forceinline__ void wait_all_but() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// this wave's copies have landed and its LDS reads are done
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }
// a wave-uniform address, kept in scalar registers
__device__ __forceinline__ const char* uniform_ptr(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}

// The copies of lds_copy.hpp for all lanes (mask -1) or, without a branch, for none (0). Only
// in code that all 64 lanes of a wave execute. (Five wait states before the load, as there.)
__device__ __forceinline__ void lds_dma16_masked(const void* sbase, uint32_t voff, uint32_t dst, int mask) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_mov_b32 exec_lo, %3\n\t"
      "s_mov_b32 exec_hi, %3\n\t"
      "s_nop 1\n\t"
      "global_load_lds_dwordx4 %0, %1\n\t"
      "s_mov_b64 exec, -1"
      :
      : "v"(voff), "s"(sbase), "s"(dst), "s"(mask)
      : "memory", "m0");
}
template <bool BYTE>
__device__ __forceinline__ void lds_dma_scale_masked(const void* sbase, uint32_t voff, uint32_t dst, int mask) {
  if constexpr (BYTE)
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_mov_b32 exec_lo, %3\n\t"
        "s_mov_b32 exec_hi, %3\n\t"
        "s_nop 1\n\t"
        "global_load_lds_ubyte %0, %1\n\t"
        "s_mov_b64 exec, -1"
        :
        : "v"(voff), "s"(sbase), "s"(dst), "s"(mask)
        : "memory", "m0");
  else
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_mov_b32 exec_lo, %3\n\t"
        "s_mov_b32 exec_hi, %3\n\t"
        "s_nop 1\n\t"
        "global_load_lds_dword %0, %1\n\t"
        "s_mov_b64 exec, -1"
        :
        : "v"(voff), "s"(sbase), "s"(dst), "s"(mask)
        : "memory", "m0");
}

enum : int { OUT_BF16 = 0, OUT_F32 = 1, OUT_F8 = 2 };
// How a block's scales reach the sums: by the matrix core; as one float32 for 64 (gated: 32 and 32) of the
// weight's rows; or as one for each of them. WIDE_*: the same for codes widened to bf16 (the products of
// the two scales are float32).
enum : int { SC_E8 = 0, SC_F32_BAND = 1, SC_F32_ROWS = 2, WIDE_E8 = 3, WIDE_F32 = 4 };

struct F8Params {
  const char *x, *xs, *w, *ws;
  int64_t rows, N, F;        // rows of x and w; F: gated, the features (N = 2 F)
  int64_t kp;                // bytes of an operand's row
  int kc;                    // blocks of K
  int es;                    // bytes of a scale
  int64_t xs_row, xs_k;      // x's scales: elements between rows, and between blocks
  int64_t ws_row, ws_k;      // w's: between (bands of) rows, and between blocks
  int ws_band;               // log2 of the rows that share a row of scales
  int64_t w_stride, ws_stride;   // bytes of one expert's codes and scales
  int n_experts;
  const int32_t* offsets;
  char* y;                   // y, h, or h's codes
  int64_t ldy;
  char* hs;                  // scales of h's codes
  char* gu;                  // the gated projections, or null
  int64_t ldgu;
  int out;                   // OUT_*
  bool gu_f32, y_vec, gu_vec;   // vec: rows take 16-byte stores
  uint32_t mtiles, ntiles;   // mtiles: an upper bound with offsets
  int slices;                // parts of K, each with its own rows in `part`
  float* part;               // [slices][rows][N] sums of a split K, or null
};

// 4 neighbouring values of a row, those below `have`
__device__ __forceinline__ void store4(char* y, bool f32, bool vec, int64_t at, int have, const v4f& v) {
  if (vec && have >= 4) {
    if (f32) *reinterpret_cast<v4f*>(y + at * 4) = v;
    else *reinterpret_cast<uint2*>(y + at * 2) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < have) {
      if (f32) reinterpret_cast<float*>(y)[at + q] = v[q];
      else reinterpret_cast<uint16_t*>(y)[at + q] = (uint16_t)pack_bf16(v[q], 0.0f);
    }
}

__device__ __forceinline__ void store_hs(const F8Params& p, int64_t m, int64_t block, uint32_t code) {
  const int64_t at = m * ((p.F + F8_BLOCK - 1) / F8_BLOCK) + block;
  if (p.es == 1) reinterpret_cast<uint8_t*>(p.hs)[at] = (uint8_t)code;
  else reinterpret_cast<uint32_t*>(p.hs)[at] = code;
}

__device__ __forceinline__ F8Scale hs_scale(const F8Params& p, uint32_t amax) {
  return p.es == 1 ? f8_scale<true>(amax) : f8_scale<false>(amax);
}

// ---------------------------------------------------------------- tile form
// A workgroup owns BM = 16 TM WM rows of x and BN = 256 rows of a weight (gated: 128 of the gate's and the same
// 128 of the up projection's), or half as many where rows are few: WM x 4 waves of 16 TM x BN / 4 outputs. The
// two operands' rows of one block of K, and their scales, are copied straight into LDS, two blocks deep. Row r
// (128 bytes) keeps its 16-byte piece j at j ^ ((r >> 1) & 7), so that 16 rows reading one piece fall on all banks.
//
// Tall tiles are bound by the matrix cores, busy for 61% of the cycles of 8192 x 4096 -> 14336 (44 to 52% where
// float32 scales, experts' last tiles or a gated product's outputs add to them): a block takes 1.43 to 1.6 us against
// 1.02 of its products alone; without its copies it takes 1.26. 8192 x 4096 -> 14336 380 us with E8M0
// scales (2.5 PFLOP/s), 455 with float32 ones, whose multiply-adds are the vector unit's; widened codes 1.1 PFLOP/s.
// Low tiles are bound by the weight's bytes and a block's latency (17 x 4096 -> 28672 31 us, 3.8 TB/s).
constexpr int ROWB = F8_BLOCK;
template <int TM_, int WM_, int BN_, int SC_, bool GATED_>
struct TileForm {
  static constexpr int TM = TM_, WM = WM_, BN = BN_, SC = SC_, WN = 4, NW = WM * WN, BM = 16 * TM * WM;
  static constexpr int TN = BN / 16 / WN, CW = TN * 16;                 // 16-row groups and weight rows of a wave
  // Streamed stores for tall tiles, us without / with: 8192 x 2048 -> 14336 232 / 210, x 4096 400 / 380, 6144 x
  // 8191 -> 4096 227 / 183; float32 (128 rows) 390 / 385.
  static constexpr bool GATED = GATED_, STREAM = BM >= 128;
  static constexpr int XP = BM / 8 / NW, WP = BN / 8 / NW;              // copies of 8 rows, a wave's
  static constexpr int XS = (BM + 63) / 64, SCALES = XS + BN / 64;      // copies of 64 scales, all
  static constexpr int SP = (SCALES + NW - 1) / NW;
  static constexpr int OPS = XP + WP + SP;                              // a wave's copies of one block
  // LDS: x rows of both buffers, weight rows of both, scales of both (x, then weight)
  static constexpr int XBUF = BM * ROWB, WBUF = BN * ROWB, SBUF = SCALES * 256, WROWS = 2 * XBUF, SROWS = WROWS + 2 * WBUF;
  static constexpr int CODES = BM * F8_BLOCK;                           // h's codes, then its row maxima
  static constexpr int LDS = SROWS + 2 * SBUF;
  static_assert(CODES + WN * BM * 4 <= LDS, "the outputs fit the buffers");
  static_assert(TM % 2 == 0 && BM % (8 * NW) == 0, "");
};

// 32 codes of a lane's row: its 16-byte pieces at two offsets
__device__ __forceinline__ v8i read_row(const char* lds, int at0, int at1) {
  const v4i a = *reinterpret_cast<const v4i*>(lds + at0);
  const v4i b = *reinterpret_cast<const v4i*>(lds + at1);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 8 codes -> 8 bf16, exact
__device__ __forceinline__ v8bf widen8(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The value of an E8M0 code: 2^(c - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t c) {
  return __uint_as_float(c == 0 ? 1u << 22 : c == 255 ? 0x7FC00000u : c << 23);
}

// STREAM: past the L2, which keeps the operands' rows for the tiles that share them (outputs of many tiles, that
// are next read from memory anyway).
template <bool STREAM>
__device__ __forceinline__ void store16(char* to, const uint4& v) {
  typedef uint32_t u4v __attribute__((ext_vector_type(4)));
  if constexpr (STREAM) __builtin_nontemporal_store(u4v{v.x, v.y, v.z, v.w}, reinterpret_cast<u4v*>(to));
  else *reinterpret_cast<uint4*>(to) = v;
}

// Columns i < NI of a wave's products (16 to a product) to rows of y, as float32 or rounded to bf16: as many of
// its rows at a time as its share of the LDS holds, turned there so that lanes store 16 bytes of whole rows.
// Columns from `half` of the NI on (gated: the up projection's) go `up` further on; 0: one run of columns.
// Piece j (16 bytes) of row r stays at j ^ (r & 7) of its eight.
template <class F, bool F32, int NI, bool STREAM>
__device__ __forceinline__ void store_wave(char* lds, const v4f (&acc)[F::TN][F::TM], char* y, int64_t ld, bool vec,
                                           int64_t m0, int64_t m1, int64_t c0, int64_t width, int64_t up) {
  constexpr int E = F32 ? 4 : 2, COLS = NI * 16, RB = COLS * E, PIECES = RB / 16, PER = 16 / E, SW = PIECES < 8 ? PIECES - 1 : 7;
  constexpr int SHARE = F::LDS / F::NW / 256 * 256;   // the same for every call: waves may be in different ones
  constexpr int FIT = SHARE / (16 * RB), JP = FIT >= F::TM ? F::TM : FIT >= 4 ? 4 : FIT >= 2 ? 2 : 1;
  static_assert(FIT >= 1 && F::TM % JP == 0, "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), fr = lane & 15, kg = lane >> 4;
  char* mine = lds + wave * SHARE;
  const int half = up ? COLS / 2 : COLS;
#pragma unroll
  for (int j0 = 0; j0 < F::TM; j0 += JP) {
#pragma unroll
    for (int j = 0; j < JP; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = j * 16 + fr, at = (i * 16 + kg * 4) * E;
        const v4f v = acc[i][j0 + j];
        char* to = mine + r * RB + (((at >> 4) ^ (r & SW)) << 4) + (at & 15);
        if constexpr (F32) *reinterpret_cast<v4f*>(to) = v;
        else *reinterpret_cast<uint2*>(to) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      }
    wave_order();
    if (vec) {
#pragma unroll 8
      for (int o = lane; o < JP * 16 * PIECES; o += 64) {
        const int r = o / PIECES, piece = o % PIECES, c = piece * PER, in = c >= half ? c - half : c;
        const uint4 v = *reinterpret_cast<const uint4*>(mine + r * RB + ((piece ^ (r & SW)) << 4));
        const int64_t m = m0 + j0 * 16 + r;
        if (m >= m1 || c0 + in >= width) continue;
        char* to = y + (m * ld + c0 + in + (c >= half ? up : 0)) * E;
        if (c0 + in + PER <= width) {
          store16<STREAM>(to, v);
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          for (int q = 0; q < (int)(width - c0) - in; ++q) {
            if constexpr (F32) reinterpret_cast<uint32_t*>(to)[q] = w[q];
            else reinterpret_cast<uint16_t*>(to)[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
          }
        }
      }
    } else {
#pragma unroll 4
      for (int o = lane; o < JP * 16 * COLS; o += 64) {
        const int r = o / COLS, c = o % COLS, in = c >= half ? c - half : c, at = c * E;
        const char* from = mine + r * RB + (((at >> 4) ^ (r & SW)) << 4) + (at & 15);
        const int64_t m = m0 + j0 * 16 + r;
        if (m >= m1 || c0 + in >= width) continue;
        const int64_t to = m * ld + c0 + in + (c >= half ? up : 0);
        if constexpr (F32) reinterpret_cast<uint32_t*>(y)[to] = *reinterpret_cast<const uint32_t*>(from);
        else reinterpret_cast<uint16_t*>(y)[to] = *reinterpret_cast<const uint16_t*>(from);
      }
    }
    wave_order();
  }
}

// h of dropped rows, or of a tile's rows, as zeros
template <class F>
__device__ __forceinline__ void zero_tile(const F8Params& p, int64_t m0, int64_t m1, int64_t c0, int slice) {
  const int rows = (int)min((int64_t)F::BM, m1 - m0);
  constexpr int W = F::GATED ? F::BN / 2 : F::BN;
  const int64_t width = F::GATED ? p.F : p.N;
  const int cols = (int)min((int64_t)W, width - c0);
  const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < rows * (W / 4); i += F::NW * 64) {
    const int64_t m = m0 + i / (W / 4), c = c0 + i % (W / 4) * 4;
    const int have = cols - i % (W / 4) * 4;
    if (p.part) {
      float* part = p.part + (int64_t)slice * p.rows * p.N;
      store4((char*)part, true, false, m * p.N + c, have, z);
      if (F::GATED) store4((char*)part, true, false, m * p.N + p.F + c, have, z);
      continue;
    }
    if (F::GATED && p.gu) {
      store4(p.gu, p.gu_f32, p.gu_vec, m * p.ldgu + c, have, z);
      store4(p.gu, p.gu_f32, p.gu_vec, m * p.ldgu + p.F + c, have, z);
    }
    if (F::GATED && p.out == OUT_F8) {
      *reinterpret_cast<uint32_t*>(p.y + m * p.ldy + c) = 0;   // (a row's codes are whole blocks)
      if (i % (W / 4) == 0) store_hs(p, m, c0 / F8_BLOCK, hs_scale(p, 0).code);
    } else {
      store4(p.y, p.out == OUT_F32, p.y_vec, m * p.ldy + c, have, z);
    }
  }
}

template <class F, int ACT>
__global__ __launch_bounds__(F::NW * 64, 2) void k_f8_tile(F8Params p) {
  constexpr int TM = F::TM, TN = F::TN, WN = F::WN, BN = F::BN, CW = F::CW, NW = F::NW, BM = F::BM, SC = F::SC;
  constexpr bool GATED = F::GATED;
  __shared__ __attribute__((aligned(1024))) char lds[F::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  TileMap<BM, F8Params> map;
  const uint32_t mtiles = p.offsets ? map.count(p) : p.mtiles;
  // workgroup ids go round-robin over the 8 dies: each die takes a contiguous run of the tiles that there
  // are, in groups of 4 m-tiles that share the weight's rows in its L2
  const uint32_t tiles = mtiles * p.ntiles, total = tiles * p.slices, per = (total + 7) / 8;
  const uint32_t in_die = blockIdx.x >> 3, all = (blockIdx.x & 7) * per + in_die;
  if (in_die >= per || all >= total) return;
  // (what stands before the first copies is short: 32-bit, and no division that a launch can do without)
  const uint32_t slice = p.slices > 1 ? all / tiles : 0, id = all - slice * tiles;
  constexpr uint32_t GM = 4;
  const uint32_t grp = id / (GM * p.ntiles), gm = min(GM, mtiles - grp * GM), rest = id - grp * GM * p.ntiles;
  const uint32_t nt = gm == GM ? rest / GM : rest / gm;
  const int mt = grp * GM + rest - nt * gm;
  const int64_t c0 = (int64_t)nt * (GATED ? BN / 2 : BN);   // first column (feature)
  int e = 0;
  int64_t m0 = (int64_t)mt * BM, m1 = p.rows;
  if (p.offsets) map.find(p, mt, e, m0, m1);
  if (p.offsets && e == p.n_experts) {
    zero_tile<F>(p, m0, m1, c0, slice);
    return;
  }
  int kc0 = 0, kc1 = p.kc;
  if (p.slices > 1) {   // (kc is at most 2^15, and there are at most kc / 4 slices)
    kc0 = __builtin_amdgcn_readfirstlane((uint32_t)p.kc * slice / (uint32_t)p.slices);
    kc1 = __builtin_amdgcn_readfirstlane((uint32_t)p.kc * (slice + 1) / (uint32_t)p.slices);
  }

  // copies: a lane's 16 bytes of an 8-row piece (rows past the tensor read its last row; not stored)
  const int64_t width = GATED ? p.F : p.N;
  const char* xsrc = uniform_ptr(p.x + m0 * p.kp + (int64_t)kc0 * ROWB);
  const char* wsrc = uniform_ptr(p.w + (int64_t)e * p.w_stride + c0 * p.kp + (int64_t)kc0 * ROWB);
  uint32_t xoff[F::XP], woff[F::WP], soff[F::SP];
  const uint32_t kp = (uint32_t)p.kp;
  const int last_row = (int)min(m1 - m0, (int64_t)BM) - 1, last_col = (int)min(width - c0, (int64_t)BN) - 1;
#pragma unroll
  for (int j = 0; j < F::XP; ++j) {
    const int r = (wave * F::XP + j) * 8 + (lane >> 3);
    xoff[j] = min(r, last_row) * kp + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  // row r of the tile's weight rows: column c0 + r, or of each wave's CW the CW / 2 features' gate and up
  auto column = [&](int r) { return min(GATED ? r / CW * (CW / 2) + r % (CW / 2) : r, last_col); };
#pragma unroll
  for (int j = 0; j < F::WP; ++j) {
    const int r = (wave * F::WP + j) * 8 + (lane >> 3);
    woff[j] = column(r) * kp + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const char* ssrc[F::SP];
  int64_t sstep[F::SP];
#pragma unroll
  for (int j = 0; j < F::SP; ++j) {
    const int at = min(wave + j * NW, F::SCALES - 1);
    const bool of_x = at < F::XS;
    const int r = (of_x ? at : at - F::XS) * 64 + lane;
    if (of_x) {
      soff[j] = min(r, last_row) * (uint32_t)(p.xs_row * p.es);
      ssrc[j] = uniform_ptr(p.xs + (m0 * p.xs_row + kc0 * p.xs_k) * p.es);
      sstep[j] = p.xs_k * p.es;
    } else {   // (a weight's scales are below 2^32 bytes)
      const int64_t row = c0 + column(r) + (GATED && (r & (CW / 2)) ? p.F : 0);
      soff[j] = (uint32_t)(row >> p.ws_band) * (uint32_t)(p.ws_row * p.es);
      ssrc[j] = uniform_ptr(p.ws + (int64_t)e * p.ws_stride + (int64_t)kc0 * p.ws_k * p.es);
      sstep[j] = p.ws_k * p.es;
    }
  }
  const int64_t up = GATED ? p.F * p.kp : 0;
  // copy n of a wave's OPS of the next block; the last one moves on to the block after it
  auto copy_op = [&](int b, int n, int mask) {
    if (n < F::XP) {
      lds_dma16_masked(xsrc, xoff[n], lds_offset(lds + b * F::XBUF + (wave * F::XP + n) * 1024), mask);
    } else if (n < F::XP + F::WP) {
      const int piece = wave * F::WP + n - F::XP;
      lds_dma16_masked(GATED && (piece & (CW / 16)) ? wsrc + up : wsrc, woff[n - F::XP], lds_offset(lds + F::WROWS + b * F::WBUF + piece * 1024),
                       mask);
    } else {
      const int j = n - F::XP - F::WP;
      const uint32_t to = lds_offset(lds + F::SROWS + b * F::SBUF + min(wave + j * NW, F::SCALES - 1) * 256);
      lds_dma_scale_masked<SC == SC_E8 || SC == WIDE_E8>(ssrc[j], soff[j], to, mask);
      ssrc[j] += sstep[j];
    }
    if (n == F::OPS - 1) {
      xsrc += ROWB;
      wsrc += ROWB;
    }
  };
  auto copy = [&](int b) {
#pragma unroll
    for (int n = 0; n < F::OPS; ++n) copy_op(b, n, -1);
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int fr = lane & 15, kg = lane >> 4;
  if (kc0 < kc1) {
    copy(0);
    if (kc0 + 1 < kc1) {
      copy(1);
      wait_all_but<F::OPS>();
    } else {
      wait_all_but<0>();
    }
    __syncthreads();
    constexpr bool WIDE = SC == WIDE_E8 || SC == WIDE_F32;
    constexpr int WC = WIDE ? 4 : 1;   // products of a block
    using Frag = std::conditional_t<WIDE, v8bf, v8i>;
    // A lane's pieces kg and kg + 4 of a row, as offsets of the wave's first row (rows 16 apart keep their pieces
    // at the same places). The order of k inside a block is free as long as both operands agree; with pieces
    // 2 kg and 2 kg + 1 the lanes that the LDS serves together met in its banks (43% of its cycles).
    const int p0 = (kg ^ ((fr >> 1) & 7)) << 4, p1 = p0 ^ 64;
    // Rows of a wave and the two buffers are constants apart. (Opaque, or the compiler keeps a register for each.)
    int xat[2], wat[2], xsat = F::SROWS + (wm * TM * 16 + fr) * 4;
    int wsat = F::SROWS + F::XS * 256 + wn * CW * 4 + (SC == SC_E8 ? fr * 4 : SC == SC_F32_BAND ? 0 : kg * 16);
    xat[0] = (wm * TM * 16 + fr) * ROWB + p0, xat[1] = xat[0] - p0 + p1;
    wat[0] = F::WROWS + (wn * CW + fr) * ROWB + p0, wat[1] = wat[0] - p0 + p1;
    asm("" : "+v"(xat[0]), "+v"(xat[1]), "+v"(wat[0]), "+v"(wat[1]), "+v"(xsat), "+v"(wsat));
    // the weight rows' fragments and scales of this block and, from its last products on, of the next
    // (WIDE: the next block's as codes, widened when it begins: two widened sets spill)
    Frag wf[WIDE ? 1 : 2][TN][WC], xf[2][WC];
    v8i codes[WIDE ? TN : 1];
    uint32_t sx[2], swc[2][TN];   // SC_E8: swc
    v4f swf[2][TN];               // else (BAND: of the wave's first row, or of both halves')
    auto take = [&](Frag* to, int at0, int at1) {
      const v8i c = read_row(lds, at0, at1);
      if constexpr (WIDE) {
#pragma unroll
        for (int q = 0; q < WC; ++q) to[q] = widen8(c[2 * q], c[2 * q + 1]);
      } else {
        to[0] = c;
      }
    };
    auto read_w = [&](int b, int i) {   // buffer b's, which are wf[b] and its scales
      const int at = b * F::WBUF + i * 16 * ROWB;
      if constexpr (WIDE) codes[i] = read_row(lds, wat[0] + at, wat[1] + at);
      else take(wf[b][i], wat[0] + at, wat[1] + at);
      const char* s = lds + wsat + b * F::SBUF + i * 64;
      if constexpr (SC == SC_E8) {
        swc[b][i] = *reinterpret_cast<const uint32_t*>(s);
      } else if constexpr (SC == SC_F32_BAND) {
        swf[b][i][0] = *reinterpret_cast<const float*>(s);
      } else {
        swf[b][i] = *reinterpret_cast<const v4f*>(s);
        if constexpr (SC == WIDE_E8) {
#pragma unroll
          for (int r = 0; r < 4; ++r) swf[b][i][r] = e8m0_value(__float_as_uint(swf[b][i][r]));
        }
      }
    };
    auto read_x = [&](int b, int j, int to) {
      take(xf[to], xat[0] + b * F::XBUF + j * 16 * ROWB, xat[1] + b * F::XBUF + j * 16 * ROWB);
      sx[to] = *reinterpret_cast<const uint32_t*>(lds + xsat + b * F::SBUF + j * 64);
      if constexpr (SC == WIDE_E8) sx[to] = __float_as_uint(e8m0_value(sx[to]));
    };
#pragma unroll
    for (int i = 0; i < TN; ++i) read_w(0, i);
    read_x(0, 0, 0);
    // A block's products, x rows (groups j) outermost. Fragments of x are read one group ahead. The barrier stands
    // in the middle of the last group but one: by then this wave has read all of the block and its copies of the
    // next one have landed, so the next block's first fragments load under the six products left, and the
    // copies into the freed buffer are dealt out between them. Float32 scales: a product's sums are taken one
    // product later, so that it is done by then.
    // (A branch around the copies would let the compiler sink the products behind it, away from their reads:
    // hence the mask.)
    constexpr int SLOTS = TN + TN / 2;
    v4f held[2] = {};
    v4f hscale[2] = {};
    auto block = [&](auto parity, int copies) {
      constexpr int W = decltype(parity)::value, WF = WIDE ? 0 : W;   // its buffer
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int q = 0; q < WC; ++q) wf[0][i][q] = widen8(codes[i][2 * q], codes[i][2 * q + 1]);
      }
#pragma unroll
      for (int n = 0; n < TM * TN; ++n) {
        const int j = n / TN, i = n % TN, slot = n - (TM * TN - SLOTS);
        __builtin_amdgcn_sched_barrier(0);
        if (i == 0 && j + 1 < TM) read_x(W, j + 1, (j + 1) & 1);
        if (slot == 0) {
          // (past the last block: unused reads of the other buffer)
          wait_copies();
          __syncthreads();
        }
        if constexpr (SC == SC_E8) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[WF][i][0], xf[j & 1][0], acc[i][j], 0, 0, 0,
                                                                       (int)swc[W][i], 0, (int)sx[j & 1]);
        } else {
          v4f t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < WC; ++q) {
            if constexpr (WIDE) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[WF][i][q], xf[j & 1][q], t, 0, 0, 0);
            else t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[WF][i][q], xf[j & 1][q], t, 0, 0, 0, 0x7F, 0, 0x7F);
          }
          held[n & 1] = t;
          const float sxf = __uint_as_float(sx[j & 1]);
#pragma unroll
          for (int r = 0; r < 4; ++r) hscale[n & 1][r] = sxf * swf[W][i][SC == SC_F32_BAND ? 0 : r];
          const int b = (n + TM * TN - 1) % (TM * TN), bi = b % TN, bj = b / TN;   // the product before
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[bi][bj][r] = __builtin_fmaf(held[b & 1][r], hscale[b & 1][r], acc[bi][bj][r]);
        }
        if (slot >= 0) {
          if (slot < TN) read_w(1 - W, slot);
          else if (slot == TN) read_x(1 - W, 0, 0);
#pragma unroll
          for (int o = F::OPS * slot / SLOTS; o < F::OPS * (slot + 1) / SLOTS; ++o) copy_op(W, o, copies);
        }
      }
    };
    const std::integral_constant<int, 0> even{};
    const std::integral_constant<int, 1> odd{};
    int k = kc0;
    for (; k + 1 < kc1; k += 2) {
      block(even, __builtin_amdgcn_readfirstlane(k + 2 < kc1 ? -1 : 0));
      block(odd, __builtin_amdgcn_readfirstlane(k + 3 < kc1 ? -1 : 0));
    }
    if (k < kc1) block(even, 0);
    if constexpr (SC != SC_E8) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[TN - 1][TM - 1][r] = __builtin_fmaf(held[(TM * TN - 1) & 1][r], hscale[(TM * TN - 1) & 1][r], acc[TN - 1][TM - 1][r]);
    }
  }

  // Out: lane l of a product holds x row l % 16 and weight rows 4 (l / 16) + r. Each wave turns its columns
  // through LDS rows of its own.
  const int64_t wrow0 = m0 + wm * TM * 16, f0 = c0 + wn * (GATED ? CW / 2 : CW);
  __syncthreads();
  if (p.part) store_wave<F, true, TN, false>(lds, acc, reinterpret_cast<char*>(p.part + (int64_t)slice * p.rows * p.N), p.N,
                                      p.N % 4 == 0 && p.F % 4 == 0, wrow0, m1, f0, width, p.F);
  else if constexpr (!GATED) {
    if (p.out == OUT_F32) store_wave<F, true, TN, F::STREAM>(lds, acc, p.y, p.ldy, p.y_vec, wrow0, m1, f0, width, 0);
    else store_wave<F, false, TN, F::STREAM>(lds, acc, p.y, p.ldy, p.y_vec, wrow0, m1, f0, width, 0);
  } else {
    if (p.gu && p.gu_f32) store_wave<F, true, TN, F::STREAM>(lds, acc, p.gu, p.ldgu, p.gu_vec, wrow0, m1, f0, width, p.F);
    else if (p.gu) store_wave<F, false, TN, F::STREAM>(lds, acc, p.gu, p.ldgu, p.gu_vec, wrow0, m1, f0, width, p.F);
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int i = 0; i < TN / 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[i][j][r];
          acc[i][j][r] = g * act_gate<ACT>(g) * acc[i + TN / 2][j][r];
        }
    if (p.out == OUT_F32) store_wave<F, true, TN / 2, F::STREAM>(lds, acc, p.y, p.ldy, p.y_vec, wrow0, m1, f0, width, 0);
    else if (p.out == OUT_BF16) store_wave<F, false, TN / 2, F::STREAM>(lds, acc, p.y, p.ldy, p.y_vec, wrow0, m1, f0, width, 0);
  }
  if constexpr (GATED) {
    if (p.part || p.out != OUT_F8 || BN != 2 * F8_BLOCK) return;
    // h as codes: the waves across hold the 128 features of a row's block
    uint32_t* red = reinterpret_cast<uint32_t*>(lds + F::CODES);   // [WN][BM]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < TN / 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (c0 + wn * (CW / 2) + i * 16 + kg * 4 + r >= width) acc[i][j][r] = 0.0f;
          a = max(a, mag_bits(acc[i][j][r]));
        }
      a = max(a, (uint32_t)__shfl_xor((int)a, 16, 64));
      a = max(a, (uint32_t)__shfl_xor((int)a, 32, 64));
      if (kg == 0) red[wn * BM + (wm * TM + j) * 16 + fr] = a;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int row = (wm * TM + j) * 16 + fr;
      uint32_t a = red[row];
#pragma unroll
      for (int w = 1; w < WN; ++w) a = max(a, red[w * BM + row]);
      const F8Scale s = hs_scale(p, a);
      if (wn == 0 && kg == 0 && m0 + row < m1) store_hs(p, m0 + row, c0 / F8_BLOCK, s.code);
#pragma unroll
      for (int i = 0; i < TN / 2; ++i)
        *reinterpret_cast<uint32_t*>(lds + row * F8_BLOCK + wn * (CW / 2) + i * 16 + kg * 4) =
            f8_pack4(acc[i][j][0] * s.enc, acc[i][j][1] * s.enc, acc[i][j][2] * s.enc, acc[i][j][3] * s.enc);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < BM * 8; i += NW * 64) {
      const int row = i >> 3, piece = i & 7;
      if (m0 + row < m1)
        store16<F::STREAM>(p.y + (m0 + row) * p.ldy + c0 + piece * 16, *reinterpret_cast<const uint4*>(lds + row * F8_BLOCK + piece * 16));
    }
  }
}

// ---------------------------------------------------------------- rows form
// For few rows of x the weight's bytes are the bound, and a product with one launch ends before one whose split K
// is joined by another. A workgroup owns 16 weight rows (gated: 16 features, so 32 rows) of one expert and takes
// its rows of x 16 at a time. Its eight waves take the blocks of K in turn, four of a wave in flight at a time,
// straight into the registers of the products (16 rows x 64 bytes to a load), and join their sums through the
// LDS. Rows of x past the group's repeat its last one; they are not stored.
constexpr int ROWS_NW = 8, ROWS_AHEAD = 4;

template <int SC, bool GATED, int ACT>
__global__ __launch_bounds__(ROWS_NW * 64) void k_f8_rows(F8Params p) {
  constexpr int TN = GATED ? 2 : 1;
  constexpr bool WIDE = SC == WIDE_E8 || SC == WIDE_F32, E8 = SC == SC_E8 || SC == WIDE_E8;
  __shared__ v4f sums[ROWS_NW][TN][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), fr = lane & 15, kg = lane >> 4;
  const int e = blockIdx.y;
  int64_t lo, hi;
  group_rows(p, e, lo, hi);
  if (lo >= hi) return;
  const int64_t c0 = (int64_t)blockIdx.x * 16, width = GATED ? p.F : p.N;
  if (p.offsets && e == p.n_experts) {   // the rows of dropped slots
    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < (hi - lo) * 4; i += ROWS_NW * 64) {
      const int64_t m = lo + i / 4, c = c0 + i % 4 * 4;
      const int have = (int)min(width - c, (int64_t)4);
      if (p.part) {
        store4((char*)p.part, true, false, m * p.N + c, have, z);
        if (GATED) store4((char*)p.part, true, false, m * p.N + p.F + c, have, z);
      } else {
        if (GATED && p.gu) {
          store4(p.gu, p.gu_f32, false, m * p.ldgu + c, have, z);
          store4(p.gu, p.gu_f32, false, m * p.ldgu + p.F + c, have, z);
        }
        store4(p.y, p.out == OUT_F32, false, m * p.ldy + c, have, z);
      }
    }
    return;
  }
  const char *wrow[TN], *wsc[TN];
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    const int64_t n = min(c0 + fr, width - 1) + i * p.F;
    wrow[i] = p.w + (int64_t)e * p.w_stride + n * p.kp + kg * 16;
    wsc[i] = p.ws + (int64_t)e * p.ws_stride + (n >> p.ws_band) * p.ws_row * p.es;
  }
  auto scale_at = [&](const char* s) {
    if constexpr (E8) return (uint32_t)*reinterpret_cast<const uint8_t*>(s);
    else return *reinterpret_cast<const uint32_t*>(s);
  };
  for (int64_t m0 = lo; m0 < hi; m0 += 16) {
    const int64_t m = min(m0 + fr, hi - 1);
    const char* xrow = p.x + m * p.kp + kg * 16;
    const char* xsc = p.xs + m * p.xs_row * p.es;
    v4f acc[TN] = {};
    for (int k0 = wave; k0 < p.kc; k0 += ROWS_NW * ROWS_AHEAD) {
      v4i w[ROWS_AHEAD][TN][2], x[ROWS_AHEAD][2];
      uint32_t sw[ROWS_AHEAD][TN], sx[ROWS_AHEAD];
#pragma unroll
      for (int a = 0; a < ROWS_AHEAD; ++a) {
        const int64_t k = min(k0 + a * ROWS_NW, p.kc - 1);   // (past the last block: times zeros)
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          w[a][i][0] = *reinterpret_cast<const v4i*>(wrow[i] + k * ROWB);
          w[a][i][1] = *reinterpret_cast<const v4i*>(wrow[i] + k * ROWB + 64);
          sw[a][i] = scale_at(wsc[i] + k * p.ws_k * p.es);
        }
        x[a][0] = *reinterpret_cast<const v4i*>(xrow + k * ROWB);
        x[a][1] = *reinterpret_cast<const v4i*>(xrow + k * ROWB + 64);
        sx[a] = scale_at(xsc + k * p.xs_k * p.es);
      }
      __builtin_amdgcn_sched_barrier(0);   // all loads, then the products
#pragma unroll
      for (int a = 0; a < ROWS_AHEAD; ++a) {
        const int there = k0 + a * ROWS_NW < p.kc ? -1 : 0;
        const v8i xf = __builtin_shufflevector(x[a][0], x[a][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          v8i wf = __builtin_shufflevector(w[a][i][0], w[a][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
          if (a > 0) wf &= there;
          if constexpr (SC == SC_E8) {
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc[i], 0, 0, 0, (int)sw[a][i], 0, (int)sx[a]);
          } else {
            v4f t = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (WIDE) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(wf[2 * q], wf[2 * q + 1]), widen8(xf[2 * q], xf[2 * q + 1]), t, 0, 0, 0);
            } else {
              t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, t, 0, 0, 0, 0x7F, 0, 0x7F);
            }
            const float xv = E8 ? e8m0_value(sx[a]) : __uint_as_float(sx[a]), wv = E8 ? e8m0_value(sw[a][i]) : __uint_as_float(sw[a][i]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float scale = xv * __shfl(wv, kg * 4 + r, 64);
              acc[i][r] = __builtin_fmaf(t[r], a == 0 || there ? scale : 0.0f, acc[i][r]);   // (it may be infinite)
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) sums[wave][i][lane] = acc[i];
    __syncthreads();
    // lane l: x row l % 16, weight rows 4 (l / 16) + r
    if (wave == 0) {
      v4f v[TN];
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        v[i] = sums[0][i][lane];
#pragma unroll
        for (int s = 1; s < ROWS_NW; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[i][r] += sums[s][i][lane][r];
      }
      const int64_t row = m0 + fr, c = c0 + kg * 4;
      const int have = (int)min(width - c, (int64_t)4);
      if (row < hi && have > 0) {
        if (p.part) {
#pragma unroll
          for (int i = 0; i < TN; ++i) store4((char*)p.part, true, p.N % 8 == 0, row * p.N + i * p.F + c, have, v[i]);
        } else if constexpr (!GATED) {
          store4(p.y, p.out == OUT_F32, p.y_vec, row * p.ldy + c, have, v[0]);
        } else {
          if (p.gu) {
            store4(p.gu, p.gu_f32, p.gu_vec, row * p.ldgu + c, have, v[0]);
            store4(p.gu, p.gu_f32, p.gu_vec, row * p.ldgu + p.F + c, have, v[TN - 1]);
          }
          v4f h;
#pragma unroll
          for (int r = 0; r < 4; ++r) h[r] = v[0][r] * act_gate<ACT>(v[0][r]) * v[TN - 1][r];
          store4(p.y, p.out == OUT_F32, p.y_vec, row * p.ldy + c, have, h);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- turning scales
// 1D scales [rows x kc] as [kc x rows]: a copy of 64 rows' scales of one block then touches a line or four
// instead of 64. 64 x 64 at a time through the LDS.
template <typename S>
__global__ __launch_bounds__(256) void k_f8_turn_scales(const S* __restrict__ s, int64_t rows, int kc, S* __restrict__ out) {
  __shared__ S tile[64][64 + 4 / sizeof(S)];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  for (int64_t r0 = (int64_t)blockIdx.x * 64; r0 < rows; r0 += (int64_t)gridDim.x * 64) {
    const int nr = (int)min(rows - r0, (int64_t)64);
    for (int k0 = 0; k0 < kc; k0 += 64) {
      const int nk = min(kc - k0, 64);
      for (int r = q; r < nr; r += 4)
        if (c < nk) tile[r][c] = s[(r0 + r) * kc + k0 + c];
      __syncthreads();
      for (int k = q; k < nk; k += 4)
        if (c < nr) out[(k0 + k) * rows + r0 + c] = tile[c][k];
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- joining a split K
// The slices' sums in slice order, rounded once to y's type.
template <int V>
__global__ __launch_bounds__(256) void k_f8_join(F8Params p) {
  const int64_t n = p.rows * p.N, per = p.N / V, all = p.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, col = i % per * V;
    const float* at = p.part + row * p.N + col;
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.slices; ++s) {
      if constexpr (V == 4) v += *reinterpret_cast<const v4f*>(at + s * n);
      else v[0] += at[s * n];
    }
    store4(p.y, p.out == OUT_F32, V == 4, row * p.ldy + col, V, v);
  }
}

// The same for the gated projections: a wave takes 128 features of a row, two to a lane.
template <int ACT>
__global__ __launch_bounds__(256) void k_f8_join_gated(F8Params p) {
  const int lane = threadIdx.x & 63;
  const int64_t n = p.rows * p.N, per = (p.F + F8_BLOCK - 1) / F8_BLOCK, all = p.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * 4) {
    const int64_t row = i / per, block = i - row * per, f = block * F8_BLOCK + lane * 2;
    float h[2] = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (f + q < p.F) {
        const float* at = p.part + row * p.N + f + q;
        float g = 0.0f, u = 0.0f;
        for (int s = 0; s < p.slices; ++s) {
          g += at[s * n];
          u += at[s * n + p.F];
        }
        h[q] = g * act_gate<ACT>(g) * u;
        const v4f gv = {g, 0.0f, 0.0f, 0.0f}, uv = {u, 0.0f, 0.0f, 0.0f}, hv = {h[q], 0.0f, 0.0f, 0.0f};
        if (p.gu) {
          store4(p.gu, p.gu_f32, false, row * p.ldgu + f + q, 1, gv);
          store4(p.gu, p.gu_f32, false, row * p.ldgu + p.F + f + q, 1, uv);
        }
        if (p.out != OUT_F8) store4(p.y, p.out == OUT_F32, false, row * p.ldy + f + q, 1, hv);
      }
    if (p.out == OUT_F8) {
      uint32_t a = max(mag_bits(h[0]), mag_bits(h[1]));
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, 64));
      const F8Scale s = hs_scale(p, a);
      if (lane == 0) store_hs(p, row, block, s.code);
      *reinterpret_cast<uint16_t*>(p.y + row * p.ldy + f) = (uint16_t)f8_pack4(h[0] * s.enc, h[1] * s.enc, 0.0f, 0.0f);
    }
  }
}

// A grid holds less than 2^32 threads; what is more is cut off without an error.
constexpr int64_t MAX_THREADS = (int64_t(1) << 32) - 1;

struct TilePlan {
  int bm, bn;      // rows and columns of a tile; bm 0: the rows form
  int64_t mt, nt;  // tiles, at most
  int slices;      // parts of K, each with sums of its own in the workspace (rows form: 1, in the workspace for codes)
};

// Measured, us in the tile form / the rows form, bf16 out: 4096 -> 6144 E8M0, 1 row 11.5 / 8.0, 8 rows 12.2 / 9.8,
// 16 rows 12.7 / 11.8; 14336 -> 4096, 1 row 21.1 / 13.3, 16 rows 21.6 / 19.0; 4096 -> 28672 float32 scales, 1 row
// 27.5 / 22.5, 4 rows 27.8 / 25.9, 8 rows 28.3 / 30.2, 16 rows 29.4 / 35.7; gated 4096 -> 2 x 14336, 1 row 23.1 /
// 25.7. Eight experts 4096 -> 14336, on average 2 rows 84 / 64, 16 rows 103 / 162; 64 of 1024 -> 2048, 4 rows 21 / 84.
bool use_rows(const F8GemmArgs& a) {
  const int64_t groups = a.n_experts, width = a.gated ? a.w.rows / 2 : a.w.rows;
  const int64_t most = a.offsets_given ? 2 : a.w.rows > 16384 ? (a.gated ? 0 : 4) : 16;
  return a.x.rows <= most * groups && div_up(width, 16) * ROWS_NW * 64 <= MAX_THREADS / (groups + 1);
}

// The tile and number of slices whose time is least by a model of what the sweeps showed, us: a round of tiles
// takes its blocks at BLOCK each and ROUND for its ends, but not less than the weight takes from memory; slices are
// written and read again. (2047 x 14336 -> 4096 E8M0: 256 rows in one slice 177, in two 124, 128 rows
// in one 151, 64 rows 220; 512 rows: 256 rows in eight slices 49, 128 in four 42, 64 in two 54; 64 x 4096 -> 28672
// float32 scales: 64 rows in two 34, 32 in two 38, 128 in two 38. 128 columns instead of 256: 1000 x 1000 -> 1000
// 8.0 -> 5.5, but 17 x 4096 -> 28672 from memory, 256 columns in two slices 30.7, 128 in one 34.5.)
TilePlan plan_tiles(const F8GemmArgs& a) {
  const int64_t cus = device_cu_count(), groups = a.offsets_given ? a.n_experts : 0, kc = div_up(a.x.k, F8_BLOCK);
  if (use_rows(a)) return {0, 0, 0, 0, 1};
  TilePlan best{};
  double least = 0;
  const double weight = (double)a.w.rows * kc * F8_BLOCK * a.n_experts / 4.5e6;
  // us a block and a round, for a weight that the L2s hold, for one that they do not, and for widened codes
  constexpr int BM[5] = {256, 128, 64, 32, 32};
  constexpr double BLOCK[3][5] = {{1.6, 0.9, 0.75, 0.6, 0.5}, {1.6, 1.15, 1.1, 1.1, 1.15}, {0.0, 1.9, 1.3, 1.1, 0.75}};
  constexpr double ROUND[5] = {7, 5, 4, 4, 4};
  const bool far = weight > 7;
  for (int i = 0; i < 5; ++i) {
    const int bm = BM[i];
    if (bm == 256 && a.f32) continue;    // the widened codes' registers
    if (i == 4 && a.codes) continue;     // a tile holds whole blocks of h
    TilePlan t;
    t.bm = bm;
    t.bn = i == 4 ? 128 : 256;
    t.nt = a.gated ? div_up(a.w.rows / 2, t.bn / 2) : div_up(a.w.rows, t.bn);
    t.mt = div_up(a.x.rows, bm) + groups;
    const int64_t tiles = (div_up(a.x.rows, bm) + groups / 2) * t.nt;   // an expert's last tile is half full
    for (int s = 1; s <= std::max<int64_t>(1, std::min<int64_t>(kc / 4, 2 * cus / tiles)); ++s) {
      t.slices = s;
      // two workgroups of the lowest tiles share a compute unit, and take a third longer each
      const bool two = bm == 32 && tiles * s > cus;
      // and one row of tiles on few of them does not draw the memory's rate
      const bool few = (far || a.f32) && t.mt == 1 && 4 * tiles * s < 3 * cus;
      const double rounds = (double)div_up(tiles * s, two ? 2 * cus : cus);
      const double block = BLOCK[a.f32 ? 2 : far][i] * (two ? 1.35 : few ? 1.2 : 1);
      const double join = s > 1 ? 3 + 8e-7 * s * a.x.rows * a.w.rows : 0;
      const double cost = std::max(rounds * div_up(kc, s) * block, weight) + rounds * ROUND[i] + join;
      if (best.bm == 0 || cost < least) {
        best = t;
        least = cost;
      }
    }
  }
  return best;
}

// workgroups of a plan, whole rounds of the eight dies
int64_t tile_grid(const TilePlan& t) { return div_up(t.mt * t.nt * t.slices, 8) * 8; }

template <class F>
void launch_tile(const F8GemmArgs& a, const F8Params& p, const TilePlan& t) {
  const uint32_t grid = (uint32_t)tile_grid(t);
  if constexpr (!F::GATED) k_f8_tile<F, 0><<<grid, F::NW * 64, 0, a.stream>>>(p);
  else if (a.act == ACT_SILU) k_f8_tile<F, ACT_SILU><<<grid, F::NW * 64, 0, a.stream>>>(p);
  else if (a.act == ACT_GELU) k_f8_tile<F, ACT_GELU><<<grid, F::NW * 64, 0, a.stream>>>(p);
  else k_f8_tile<F, ACT_GELU_TANH><<<grid, F::NW * 64, 0, a.stream>>>(p);
}

template <int SC, bool GATED>
void launch_form(const F8GemmArgs& a, const F8Params& p, const TilePlan& t) {
  if constexpr (SC < WIDE_E8) {
    if (t.bm == 256) return launch_tile<TileForm<8, 2, 256, SC, GATED>>(a, p, t);
  }
  if (t.bm == 128) launch_tile<TileForm<4, 2, 256, SC, GATED>>(a, p, t);
  else if (t.bm == 64) launch_tile<TileForm<4, 1, 256, SC, GATED>>(a, p, t);
  else if (t.bn == 256) launch_tile<TileForm<2, 1, 256, SC, GATED>>(a, p, t);
  else launch_tile<TileForm<2, 1, 128, SC, GATED>>(a, p, t);
}

template <int SC, bool GATED>
void launch_rows(const F8GemmArgs& a, const F8Params& p) {
  const dim3 grid((uint32_t)div_up(GATED ? p.F : p.N, 16), a.offsets ? a.n_experts + 1 : 1);
  if constexpr (!GATED) k_f8_rows<SC, false, 0><<<grid, ROWS_NW * 64, 0, a.stream>>>(p);
  else if (a.act == ACT_SILU) k_f8_rows<SC, true, ACT_SILU><<<grid, ROWS_NW * 64, 0, a.stream>>>(p);
  else if (a.act == ACT_GELU) k_f8_rows<SC, true, ACT_GELU><<<grid, ROWS_NW * 64, 0, a.stream>>>(p);
  else k_f8_rows<SC, true, ACT_GELU_TANH><<<grid, ROWS_NW * 64, 0, a.stream>>>(p);
}

template <bool GATED>
void launch(const F8GemmArgs& a, const F8Params& p, const TilePlan& t) {
  if (t.bm == 0) {
    if (a.f32) a.x.e8 ? launch_rows<WIDE_E8, GATED>(a, p) : launch_rows<WIDE_F32, GATED>(a, p);
    else a.x.e8 ? launch_rows<SC_E8, GATED>(a, p) : launch_rows<SC_F32_ROWS, GATED>(a, p);
    return;
  }
  if (a.f32) {
    if (a.x.e8) launch_form<WIDE_E8, GATED>(a, p, t);
    else launch_form<WIDE_F32, GATED>(a, p, t);
  } else if (a.x.e8) launch_form<SC_E8, GATED>(a, p, t);
  // a wave's 64 rows (gated: its 32 and 32) lie in one band each
  else if (a.w.layout != 0 && (!GATED || p.F % 32 == 0)) launch_form<SC_F32_BAND, GATED>(a, p, t);
  else launch_form<SC_F32_ROWS, GATED>(a, p, t);
}

}  // namespace

bool f8_gemm_fits(const F8GemmArgs& a) {
  if (a.x.rows == 0 || a.w.rows == 0) return true;
  const TilePlan t = plan_tiles(a);
  return t.bm == 0 || tile_grid(t) * (t.bm >= 128 ? 512 : 256) <= MAX_THREADS;
}

// The scales that are turned for a plan, at the start of the workspace: x's, and a single weight's 1D ones.
// From 192 blocks to a compute unit on, as turning them is a launch of its own. Measured, us without / with:
// 8192 x 4096 -> 14336 (224 blocks) 404 / 396, 8192 x 8192 -> 8192 (256) 443 / 420; but 4096 x 4096 -> 4096 (32)
// 53 / 59, 1000 x 14336 -> 4096 (112) 73 / 78, 6144 x 8191 -> 4096 (128) 226 / 227.
struct Turned {
  size_t x, w;   // bytes, or 0
};
Turned turned(const F8GemmArgs& a, const TilePlan& t) {
  const int64_t kc = div_up(a.x.k, F8_BLOCK);
  if (t.bm < 256 || div_up(t.mt * t.nt, device_cu_count()) * kc < 192) return {0, 0};
  auto bytes = [&](const F8Operand& o) { return (size_t)div_up(o.rows * div_up(o.k, F8_BLOCK) * (o.e8 ? 1 : 4), 256) * 256; };
  return {bytes(a.x), a.w.layout == 0 && !a.offsets_given ? bytes(a.w) : 0};
}

// Whether the sums go through the workspace: those of slices, and of the rows form, whose workgroups hold no whole
// block of h, when h is wanted as codes.
bool in_parts(const F8GemmArgs& a, const TilePlan& t) { return t.slices > 1 || (t.bm == 0 && a.codes); }

size_t f8_gemm_ws(const F8GemmArgs& a) {
  if (a.x.rows == 0 || a.w.rows == 0) return 0;
  const TilePlan t = plan_tiles(a);
  const Turned turn = turned(a, t);
  return turn.x + turn.w + (in_parts(a, t) ? (size_t)t.slices * a.x.rows * a.w.rows * 4 : 0);
}

void f8_gemm_form(const F8GemmArgs& a, int32_t form[4]) {
  const bool some = a.x.rows > 0 && a.w.rows > 0;
  const TilePlan t = some ? plan_tiles(a) : TilePlan{};
  const Turned turn = some ? turned(a, t) : Turned{};
  form[0] = t.bm;
  form[1] = t.bn;
  form[2] = t.slices;
  form[3] = (turn.x ? 1 : 0) | (turn.w ? 2 : 0);
}

hipError_t run_f8_gemm(const F8GemmArgs& a) {
  if (a.x.rows == 0 || a.w.rows == 0) return hipSuccess;
  F8Params p{};
  const int64_t kc = div_up(a.x.k, F8_BLOCK), bands = div_up(a.w.rows, F8_BLOCK);
  p.x = (const char*)a.x.q;
  p.xs = (const char*)a.x.s;
  p.w = (const char*)a.w.q;
  p.ws = (const char*)a.w.s;
  p.rows = a.x.rows;
  p.N = a.w.rows;
  p.F = a.gated ? a.w.rows / 2 : 0;
  p.kp = kc * F8_BLOCK;
  p.kc = (int)kc;
  p.es = a.x.e8 ? 1 : 4;
  p.xs_row = kc;
  p.xs_k = 1;
  p.ws_row = a.w.layout == 2 ? 1 : kc;
  p.ws_k = a.w.layout == 2 ? bands : 1;
  p.ws_band = a.w.layout == 0 ? 0 : 7;
  p.w_stride = a.w.rows * p.kp;
  p.ws_stride = (a.w.layout == 0 ? a.w.rows : bands) * kc * p.es;
  p.n_experts = a.n_experts;
  p.offsets = a.offsets;
  p.y = (char*)a.y;
  p.out = a.y_kind;
  p.ldy = a.y_kind == OUT_F8 ? div_up(p.F, F8_BLOCK) * F8_BLOCK : a.ldy;
  p.hs = (char*)a.ys;
  p.gu = (char*)a.gu;
  p.ldgu = a.ldgu;
  p.gu_f32 = a.gu_f32;
  auto vec = [](const void* q, int64_t ld, bool f32) {
    return ld % (f32 ? 4 : 8) == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  };
  p.y_vec = a.y_kind != OUT_F8 && vec(a.y, a.ldy, a.y_kind == OUT_F32);
  p.gu_vec = a.gu && vec(a.gu, a.ldgu, a.gu_f32) && p.F % (a.gu_f32 ? 4 : 8) == 0;
  const TilePlan t = plan_tiles(a);
  p.mtiles = (uint32_t)t.mt;
  p.ntiles = (uint32_t)t.nt;
  p.slices = t.slices;
  const Turned turn = turned(a, t);
  auto turn_scales = [&](const F8Operand& o, void* out, const char*& s, int64_t& s_row, int64_t& s_k) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(o.rows, 64), 1 << 20);
    if (o.e8) k_f8_turn_scales<uint8_t><<<grid, 256, 0, a.stream>>>((const uint8_t*)o.s, o.rows, p.kc, (uint8_t*)out);
    else k_f8_turn_scales<uint32_t><<<grid, 256, 0, a.stream>>>((const uint32_t*)o.s, o.rows, p.kc, (uint32_t*)out);
    s = (const char*)out;
    s_row = 1;
    s_k = o.rows;
  };
  if (turn.x) turn_scales(a.x, a.ws, p.xs, p.xs_row, p.xs_k);
  if (turn.w) turn_scales(a.w, (char*)a.ws + turn.x, p.ws, p.ws_row, p.ws_k);
  if (in_parts(a, t)) p.part = (float*)((char*)a.ws + turn.x + turn.w);
  if (a.gated) launch<true>(a, p, t);
  else launch<false>(a, p, t);
  if (p.part) {
    if (!a.gated) {
      const bool four = p.y_vec && p.N % 4 == 0;
      const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(p.rows * p.N / (four ? 4 : 1), 256), 4096);
      if (four) k_f8_join<4><<<grid, 256, 0, a.stream>>>(p);
      else k_f8_join<1><<<grid, 256, 0, a.stream>>>(p);
    } else {
      const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(p.rows * div_up(p.F, F8_BLOCK), 4), 8192);
      if (a.act == ACT_SILU) k_f8_join_gated<ACT_SILU><<<grid, 256, 0, a.stream>>>(p);
      else if (a.act == ACT_GELU) k_f8_join_gated<ACT_GELU><<<grid, 256, 0, a.stream>>>(p);
      else k_f8_join_gated<ACT_GELU_TANH><<<grid, 256, 0, a.stream>>>(p);
    }
  }
  return hipGetLastError();
}

}  // namespace fp4k
