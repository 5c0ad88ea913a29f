// E4M3 quantizers with one scale to each 128 elements of a row, of a column, or to each 128 x 128
// tile, their decode, and the gradient of the gated projections, plain or quantized in the same pass.
//
// A workgroup takes a 128 x 128 tile, which holds whole blocks of every view, so one read of the
// input serves all of them. Thread (tr, tc) = (id / 16, id % 16) holds the P x 8 elements of rows
// P tr .. and columns 8 tc ..: a row's block is 16 neighbouring lanes, a column's one lane in 16 of
// every wave. Row codes go straight to memory, 128 consecutive bytes from 16 lanes; column codes turn
// in LDS, where a thread has P consecutive bytes of each of its columns. Codes are stored past the L2 (8192 x
// 4096 bf16, both views: 31.6 -> 28.6 us). Bound by HBM: 4.7 TB/s there, 5.5 for one view or 28672 x 4096 float32 in
// tiles, against 5.2 of a copy.
#include "fp8.hpp"
#include "quant_common.hpp"

namespace fp4k {

namespace {

constexpr int T = F8_BLOCK, THREADS = 256;

// A tile kernel's shape: rows of a thread, and its threads.
template <int P_, int OCC_>
struct Shape {
  static constexpr int OCC = OCC_;
  static constexpr int P = P_, THREADS = T * T / 8 / P, WAVES = THREADS / 64;
};
// Rows of a thread and waves to a SIMD. Measured, us with 8 rows, two waves / 4 rows, five: 8192 x 4096 bf16, both
// views 30.6 / 31.9, transposed 18.9 / 25.4, rows 19.0 / 18.3; 8192 x 14336 both 107 / 98.
using QuantShape = Shape<8, 2>;
// The gated gradient, us with 8 rows, two waves / 4 rows, four / 4 rows, three: 8192 x 14336 bf16 297 / 309 / 412,
// 2047 x 14336 float32 158 / 173 / 132.
template <bool F32>
using GradShape = std::conditional_t<F32, Shape<4, 3>, Shape<8, 2>>;

struct Tile {
  int64_t r0, c0;    // first row and column
  int rows, cols;    // what there is of the tile's
};

// 8 elements of a row of a tile as loaded: 32-bit words, two bf16 or one float32 in each.
template <bool F32>
struct Raw8 {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ void to_float(float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = F32 ? __uint_as_float(w[j % (F32 ? 8 : 4)]) : j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
  }
};

// How rows are loaded. ALIGNED: 16-byte aligned. ROWS: aligned to their elements only, 8 columns or more. NARROW:
// fewer columns, an element at a time.
enum : int { LOAD_ALIGNED = 0, LOAD_ROWS = 1, LOAD_NARROW = 2 };

// Those of tile row r from column c on that the tile's rows x cols have, and zeros for the rest; no branches.
// base: the tile's first element, ld <= 2^22. Offsets out of a buffer resource's range load zeros.
// ALIGNED: a row's last 16 bytes are loaded whole (they hold an element, so they lie in its page) and masked.
// ROWS: past the row's last 8 elements those are loaded instead and moved down by what they start too early.
template <bool F32, int LOAD>
__device__ __forceinline__ void load_tile8(const char* base, int r, int rows, int64_t ld, int c, int cols, Raw8<F32>& v) {
  constexpr int E = F32 ? 4 : 2, W = F32 ? 8 : 4;
  const int have = r < rows ? cols - c : 0;
  if constexpr (LOAD == LOAD_ALIGNED) {
    const rsrc_t x = make_rsrc(base);
    const uint32_t at = ((uint32_t)r * (uint32_t)ld + c) * E;
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {   // 16 bytes at a time
      const v4u u = __builtin_amdgcn_raw_buffer_load_b128(x, have > 4 * i ? at + 16 * i : OOB, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[4 * i + j] = u[j];
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (F32) v.w[j] = j < have ? v.w[j] : 0;
      else v.w[j] &= 2 * j + 1 < have ? 0xFFFFFFFFu : 2 * j < have ? 0xFFFFu : 0u;
    }
  } else if constexpr (LOAD == LOAD_ROWS) {
    const bool none = have <= 0;
    const int early = none ? 0 : max(0, 8 - have);
    const char* from = base + (none ? (int64_t)min(0, cols - 8) : (int64_t)r * ld + c - early) * E;
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      v4u u;
      __builtin_memcpy(&u, __builtin_assume_aligned(from + 16 * i, E), 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[4 * i + j] = u[j];
    }
    // (words count up, so each is read before it is replaced)
    const bool by4 = early & 4, by2 = early & 2, by1 = early & 1;
#pragma unroll
    for (int j = 0; j < W; ++j) v.w[j] = by4 ? (j + W / 2 < W ? v.w[(j + W / 2) % W] : 0u) : v.w[j];
#pragma unroll
    for (int j = 0; j < W; ++j) v.w[j] = by2 ? (j + W / 4 < W ? v.w[(j + W / 4) % W] : 0u) : v.w[j];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t next = j + 1 < W ? v.w[(j + 1) % W] : 0u;
      v.w[j] = by1 ? (F32 ? next : v.w[j] >> 16 | next << 16) : v.w[j];
    }
#pragma unroll
    for (int j = 0; j < W; ++j) v.w[j] = none ? 0u : v.w[j];
  } else {
    const rsrc_t x = make_rsrc(base);
    const uint32_t at = ((uint32_t)r * (uint32_t)ld + c) * E;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t o = j < have ? at + j * E : OOB;
      if constexpr (F32) v.w[j] = __builtin_amdgcn_raw_buffer_load_b32(x, o, 0, 0);
      else {
        const uint32_t u = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(x, o, 0, 0);
        v.w[j / 2] = j & 1 ? v.w[j / 2] | u << 16 : u;
      }
    }
  }
}

template <bool E8>
__device__ __forceinline__ void store_scale(void* s, int64_t i, uint32_t code) {
  if constexpr (E8) reinterpret_cast<uint8_t*>(s)[i] = (uint8_t)code;
  else reinterpret_cast<uint32_t*>(s)[i] = code;
}

// Where one tile's codes and scales go. Rows and columns of the outputs start at row0 / col0 of the
// views (the second half of a gated gradient starts at f).
struct TileOut {
  uint8_t* q;
  void* s;
  int64_t kp, sld;       // bytes and scales of a row of q
  uint8_t* qt;
  void* st;
  int64_t ktp, stld;     // the same of qt
  int64_t row0, col0, trow0, tcol0;   // the tile's first row and column in q, and in qt
};

template <class S>
struct Lds {
  uint32_t part[S::WAVES][T];   // columns' maxima, a row of them per wave
  __attribute__((aligned(16))) uint8_t codes[T * T];
};

// v[p][j]: element (P tr + p, 8 tc + j), zeros outside the tensor. VIEW: F8_VIEW_*.
template <class S, int VIEW, bool E8>
__device__ __forceinline__ void quantize_tile(const float (&v)[S::P][8], const Tile& t, const TileOut& o, Lds<S>& lds) {
  constexpr int P = S::P;
  constexpr bool ROW = VIEW != F8_VIEW_COL, COL = VIEW != F8_VIEW_ROW, GRID = VIEW == F8_VIEW_TILE2D;
  const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15, wave = tid >> 6;
  float tile_enc = 0.0f;
  if constexpr (GRID) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[p][j]));
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, x, 64));
    if ((tid & 63) == 0) lds.part[wave][0] = m;
    __syncthreads();
    m = lds.part[0][0];
#pragma unroll
    for (int w = 1; w < S::WAVES; ++w) m = max(m, lds.part[w][0]);
    const F8Scale s = f8_scale<E8>(m);
    tile_enc = s.enc;
    if (tid == 0) store_scale<E8>(o.s, (o.row0 / T) * o.sld + o.col0 / T, s.code);
  }
  if constexpr (ROW) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = tr * P + p;
      float enc = tile_enc;
      if constexpr (!GRID) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[p][j]));
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, x, 64));
        const F8Scale s = f8_scale<E8>(m);
        enc = s.enc;
        if (tc == 0 && r < t.rows) store_scale<E8>(o.s, (o.row0 + r) * o.sld + o.col0 / T, s.code);
      }
      if (r < t.rows) {   // (codes past the columns are those of the zeros there)
        const v2u w = {f8_pack4(v[p][0] * enc, v[p][1] * enc, v[p][2] * enc, v[p][3] * enc),
                       f8_pack4(v[p][4] * enc, v[p][5] * enc, v[p][6] * enc, v[p][7] * enc)};
        __builtin_nontemporal_store(w, reinterpret_cast<v2u*>(o.q + (o.row0 + r) * o.kp + o.col0 + tc * 8));
      }
    }
  }
  if constexpr (COL) {
    float enc[8];
    if constexpr (GRID) {
#pragma unroll
      for (int j = 0; j < 8; ++j) enc[j] = tile_enc;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) m = max(m, mag_bits(v[p][j]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if ((tid & 63) < 16) lds.part[wave][tc * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = tc * 8 + j;
        uint32_t m = lds.part[0][c];
#pragma unroll
        for (int w = 1; w < S::WAVES; ++w) m = max(m, lds.part[w][c]);
        const F8Scale s = f8_scale<E8>(m);
        enc[j] = s.enc;
        if (tr == 0 && c < t.cols) store_scale<E8>(o.st, (o.trow0 + c) * o.stld + o.tcol0 / T, s.code);
      }
    }
    // column c keeps its 16-byte piece i at i ^ (c / 8 % 8): 16 lanes of one row group fall on different banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint8_t* to = lds.codes + (tc * 8 + j) * T + (((tr * P >> 4) ^ (tc & 7)) << 4) + (tr * P & 15);
#pragma unroll
      for (int p = 0; p < P; p += 4)
        *reinterpret_cast<uint32_t*>(to + p) = f8_pack4(v[p][j] * enc[j], v[p + 1][j] * enc[j], v[p + 2][j] * enc[j], v[p + 3][j] * enc[j]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T * T / 16 / S::THREADS; ++i) {
      const int at = i * S::THREADS + tid, c = at >> 3, piece = at & 7;
      if (c < t.cols)   // (codes past the rows are those of the zeros there)
        __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(lds.codes + c * T + ((piece ^ ((c >> 3) & 7)) << 4)),
                                    reinterpret_cast<v4u*>(o.qt + (o.trow0 + c) * o.ktp + o.tcol0 + piece * 16));
    }
  }
}

struct QuantParams {
  const char* x;
  int64_t rows, cols, ld, tiles_c;
  TileOut out;
};

template <int VIEW, bool F32, int LOAD, bool E8>
__global__ __launch_bounds__(QuantShape::THREADS, QuantShape::OCC) void k_f8_quantize(QuantParams p) {
  constexpr int P = QuantShape::P;
  __shared__ Lds<QuantShape> lds;
  const int64_t br = blockIdx.x / p.tiles_c, bc = blockIdx.x - br * p.tiles_c;
  const Tile t{br * T, bc * T, (int)min((int64_t)T, p.rows - br * T), (int)min((int64_t)T, p.cols - bc * T)};
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const char* x = p.x + (t.r0 * p.ld + t.c0) * (F32 ? 4 : 2);
  Raw8<F32> raw[P];
  float v[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i)
    load_tile8<F32, LOAD>(x, tr * P + i, t.rows, p.ld, tc * 8, t.cols, raw[i]);
#pragma unroll
  for (int i = 0; i < P; ++i) raw[i].to_float(v[i]);
  TileOut o = p.out;
  o.row0 = o.tcol0 = t.r0;
  o.col0 = o.trow0 = t.c0;
  quantize_tile<QuantShape, VIEW, E8>(v, t, o, lds);
}

// ---------------------------------------------------------------- gated gradient

struct GradParams {
  const char *dh, *gu;
  int64_t rows, f, lddh, ldgu, tiles_c;
  char* dgu;
  int64_t lddgu;
  TileOut out;
};

// (dh, g, u) -> (dh u act'(g), dh act(g))
template <int ACT>
__device__ __forceinline__ void gated_grad1(float dh, float g, float u, float& dg, float& du) {
  float p, slope;
  act_both<ACT>(g, p, slope);
  // (a slope of 0 meets no infinite dh u; half of one, which is below 1, takes no u past the range)
  dg = 2.0f * (dh * (u * (0.5f * slope)));
  du = dh * (g * p);
}

template <int VIEW, int ACT, bool F32, int LOAD, bool E8>
__global__ __launch_bounds__(GradShape<F32>::THREADS, GradShape<F32>::OCC) void k_f8_gated_grad(GradParams p) {
  using S = GradShape<F32>;
  constexpr int P = S::P, ES = F32 ? 4 : 2;
  __shared__ Lds<S> lds;
  const int64_t br = blockIdx.x / p.tiles_c, bc = blockIdx.x - br * p.tiles_c;
  const Tile t{br * T, bc * T, (int)min((int64_t)T, p.rows - br * T), T};   // f is a multiple of T
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const char* gu = p.gu + (t.r0 * p.ldgu + t.c0) * ES;
  const char *xh = p.dh + (t.r0 * p.lddh + t.c0) * ES, *xg = gu, *xu = gu + p.f * ES;
  Raw8<F32> h[P], g[P], u[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int r = tr * P + i;
    load_tile8<F32, LOAD>(xh, r, t.rows, p.lddh, tc * 8, T, h[i]);
    load_tile8<F32, LOAD>(xg, r, t.rows, p.ldgu, tc * 8, T, g[i]);
    load_tile8<F32, LOAD>(xu, r, t.rows, p.ldgu, tc * 8, T, u[i]);
  }
  TileOut o = p.out;
  o.row0 = o.tcol0 = t.r0;
  // The gate's half, then the up projection's from the inputs anew: both at once take the registers of the other
  // workgroups whose loads would go on meanwhile (8192 x 14336 bf16 457 us at best, 296 so: 4.0 TB/s, bound by the
  // activation's and the quantizer's vector work beside the loads). The words are opaque in between, or the
  // compiler keeps what the halves share.
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float d[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float dh[8], gate[8], up[8];
      h[i].to_float(dh);
      g[i].to_float(gate);
      u[i].to_float(up);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float dg, du;
        gated_grad1<ACT>(dh[j], gate[j], up[j], dg, du);
        d[i][j] = half ? du : dg;
      }
    }
    o.col0 = o.trow0 = half * p.f + t.c0;
    quantize_tile<S, VIEW, E8>(d, t, o, lds);
    if (half == 0) {
      if constexpr (VIEW != F8_VIEW_ROW) __syncthreads();   // the first half's codes have been read
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < (F32 ? 8 : 4); ++j) asm volatile("" : "+v"(h[i].w[j]), "+v"(g[i].w[j]));
    }
  }
}

// 8 elements, or those of `have`, at an address that is aligned to 16 bytes (ALIGNED) or to an element.
template <bool F32, bool ALIGNED>
__device__ __forceinline__ void load_row8(const char* from, int have, float* v) {
  constexpr int E = F32 ? 4 : 2;
  Raw8<F32> r;
  if (have >= 8) {
    __builtin_memcpy(r.w, __builtin_assume_aligned(from, ALIGNED ? 16 : E), 8 * E);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (F32) r.w[j] = j < have ? reinterpret_cast<const uint32_t*>(from)[j] : 0;
      else {
        const uint32_t u = j < have ? reinterpret_cast<const uint16_t*>(from)[j] : 0;
        r.w[j / 2] = j & 1 ? r.w[j / 2] | u << 16 : u;
      }
    }
  }
  r.to_float(v);
}

// One thread to 8 elements of a row of dh.
template <int ACT, bool F32, bool ALIGNED>
__global__ __launch_bounds__(THREADS) void k_gated_grad(GradParams p) {
  constexpr int E = F32 ? 4 : 2;
  const int64_t per = (p.f + 7) / 8, n = p.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS) {
    const int64_t r = i / per, c = (i - r * per) * 8;
    const int have = (int)min((int64_t)8, p.f - c);
    const char* gu = p.gu + (r * p.ldgu + c) * E;
    char* out = p.dgu + (r * p.lddgu + c) * E;
    float h[8], a[2][8];
    load_row8<F32, ALIGNED>(p.dh + (r * p.lddh + c) * E, have, h);
    load_row8<F32, ALIGNED>(gu, have, a[0]);
    load_row8<F32, ALIGNED>(gu + p.f * E, have, a[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) gated_grad1<ACT>(h[j], a[0][j], a[1][j], a[0][j], a[1][j]);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      uint32_t w[F32 ? 8 : 4];
#pragma unroll
      for (int j = 0; j < (F32 ? 8 : 4); ++j) w[j] = F32 ? __float_as_uint(a[o][j]) : pack_bf16(a[o][2 * j % 8], a[o][(2 * j + 1) % 8]);
      char* to = out + o * p.f * E;
      if (have >= 8) {
        __builtin_memcpy(__builtin_assume_aligned(to, ALIGNED ? 16 : E), w, 8 * E);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < have) {
            if constexpr (F32) reinterpret_cast<uint32_t*>(to)[j] = w[j];
            else reinterpret_cast<uint16_t*>(to)[j] = (uint16_t)(w[j / 2] >> 16 * (j & 1));
          }
      }
    }
  }
}

// ---------------------------------------------------------------- decode

struct DequantParams {
  const uint8_t* q;
  const void* s;
  int64_t rows, k, kp, s_row, s_k;   // scales: elements between (bands of) rows and between blocks
  int s_band;                        // log2 of the rows that share a row of scales
  char* y;
  int64_t ldy;
};

// One thread to 4 codes.
template <bool E8, bool F32>
__global__ __launch_bounds__(THREADS) void k_f8_dequantize(DequantParams p) {
  const int64_t per = p.kp / 4, n = p.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS) {
    const int64_t r = i / per, c = (i - r * per) * 4, at = (r >> p.s_band) * p.s_row + c / F8_BLOCK * p.s_k;
    const int w = *reinterpret_cast<const int*>(p.q + r * p.kp + c);
    float s;
    if constexpr (E8) {
      const uint32_t code = reinterpret_cast<const uint8_t*>(p.s)[at];
      s = code ? (code == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(code << 23)) : __uint_as_float(1u << 22);
    } else {
      s = reinterpret_cast<const float*>(p.s)[at];
    }
    const float v[4] = {__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
                        __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < p.k) {
        if constexpr (F32) reinterpret_cast<float*>(p.y)[r * p.ldy + c + j] = v[j] * s;
        else reinterpret_cast<uint16_t*>(p.y)[r * p.ldy + c + j] = (uint16_t)pack_bf16(v[j] * s, 0.0f);
      }
  }
}

int64_t blocks(int64_t n) { return div_up(n, F8_BLOCK); }

// whether a launch of one workgroup to a tile holds fewer than 2^32 threads (what is more is cut off without an error)
bool tiles_fit(int64_t rows, int64_t cols, int threads) { return blocks(rows) * blocks(cols) < (int64_t(1) << 32) / threads; }

// calls f with std::true_type or std::false_type
template <class F>
void with_bool(bool b, F f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

template <class F>
void with_act(int act, F f) {
  if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else f(std::integral_constant<int, ACT_GELU_TANH>{});
}

// rows that take 16-byte loads from every eighth element on
bool vec_rows(const void* p, int64_t ld, bool f32) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (f32 ? 4 : 8) == 0;
}

template <class F>
void with_load(const void* p, int64_t ld, bool f32, int64_t cols, F f) {
  if (vec_rows(p, ld, f32)) f(std::integral_constant<int, LOAD_ALIGNED>{});
  else if (cols >= 8) f(std::integral_constant<int, LOAD_ROWS>{});
  else f(std::integral_constant<int, LOAD_NARROW>{});
}

TileOut tile_out(int64_t rows, int64_t cols, bool grid, uint8_t* q, void* s, uint8_t* qt, void* st) {
  TileOut o{};
  o.q = q;
  o.s = s;
  o.kp = blocks(cols) * T;
  o.sld = blocks(cols);
  o.qt = qt;
  o.st = grid ? s : st;
  o.ktp = blocks(rows) * T;
  o.stld = blocks(rows);
  return o;
}

}  // namespace

bool f8_quantize_fits(int64_t rows, int64_t cols) { return tiles_fit(rows, cols, QuantShape::THREADS); }

bool f8_gated_grad_fits(int64_t rows, int64_t f, bool f32) {
  return tiles_fit(rows, f, f32 ? GradShape<true>::THREADS : GradShape<false>::THREADS);
}

hipError_t run_f8_quantize(const F8QuantArgs& a) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  QuantParams p{(const char*)a.x, a.rows, a.cols, a.ld, blocks(a.cols),
                tile_out(a.rows, a.cols, a.view == F8_VIEW_TILE2D, a.q, a.s, a.qt, a.st)};
  const uint32_t grid = (uint32_t)(blocks(a.rows) * p.tiles_c);
  auto view = [&](auto v) {
    with_bool(a.f32, [&](auto f32) {
      with_load(a.x, a.ld, a.f32, a.cols, [&](auto load) {
        with_bool(a.e8, [&](auto e8) {
          k_f8_quantize<decltype(v)::value, decltype(f32)::value, decltype(load)::value, decltype(e8)::value>
              <<<grid, QuantShape::THREADS, 0, a.stream>>>(p);
        });
      });
    });
  };
  if (a.view == F8_VIEW_ROW) view(std::integral_constant<int, F8_VIEW_ROW>{});
  else if (a.view == F8_VIEW_COL) view(std::integral_constant<int, F8_VIEW_COL>{});
  else if (a.view == F8_VIEW_ROWCOL) view(std::integral_constant<int, F8_VIEW_ROWCOL>{});
  else view(std::integral_constant<int, F8_VIEW_TILE2D>{});
  return hipGetLastError();
}

hipError_t run_gated_grad(const GatedGradArgs& a) {
  if (a.rows == 0 || a.f == 0) return hipSuccess;
  GradParams p{};
  p.dh = (const char*)a.dh;
  p.gu = (const char*)a.gu;
  p.rows = a.rows;
  p.f = a.f;
  p.lddh = a.lddh;
  p.ldgu = a.ldgu;
  const bool vec_in = vec_rows(a.dh, a.lddh, a.f32) && vec_rows(a.gu, a.ldgu, a.f32) && a.f % (a.f32 ? 4 : 8) == 0;
  if (a.dgu) {
    p.dgu = (char*)a.dgu;
    p.lddgu = a.lddgu;
    const bool vec = vec_in && vec_rows(a.dgu, a.lddgu, a.f32);
    const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(a.rows * div_up(a.f, 8), THREADS), 8192);
    with_act(a.act, [&](auto act) {
      with_bool(a.f32, [&](auto f32) {
        with_bool(vec, [&](auto v) {
          k_gated_grad<decltype(act)::value, decltype(f32)::value, decltype(v)::value><<<grid, THREADS, 0, a.stream>>>(p);
        });
      });
    });
    return hipGetLastError();
  }
  p.tiles_c = a.f / T;
  p.out = tile_out(a.rows, 2 * a.f, false, a.q, a.s, a.qt, a.st);
  const uint32_t grid = (uint32_t)(blocks(a.rows) * p.tiles_c);
  auto view = [&](auto v) {
    with_act(a.act, [&](auto act) {
      with_bool(a.f32, [&](auto f32) {
        with_bool(vec_in, [&](auto vec) {
          with_bool(a.e8, [&](auto e8) {
            constexpr int A = decltype(act)::value, LOAD = decltype(vec)::value ? LOAD_ALIGNED : LOAD_ROWS;
            constexpr bool F32 = decltype(f32)::value;
            k_f8_gated_grad<decltype(v)::value, A, F32, LOAD, decltype(e8)::value>
                <<<grid, GradShape<F32>::THREADS, 0, a.stream>>>(p);
          });
        });
      });
    });
  };
  if (!a.qt) view(std::integral_constant<int, F8_VIEW_ROW>{});
  else if (!a.q) view(std::integral_constant<int, F8_VIEW_COL>{});
  else view(std::integral_constant<int, F8_VIEW_ROWCOL>{});
  return hipGetLastError();
}

hipError_t run_f8_dequantize(const F8Operand& a, void* y, bool f32, int64_t ldy, hipStream_t stream) {
  if (a.rows == 0 || a.k == 0) return hipSuccess;
  const int64_t kc = blocks(a.k);
  DequantParams p{a.q, a.s, a.rows, a.k, kc * T, a.layout == 2 ? 1 : kc, a.layout == 2 ? blocks(a.rows) : 1,
                  a.layout == 0 ? 0 : 7, (char*)y, ldy};
  const uint32_t grid = (uint32_t)std::min<int64_t>(div_up(a.rows * p.kp / 4, THREADS), 8192);
  with_bool(a.e8, [&](auto e8) {
    with_bool(f32, [&](auto y32) {
      k_f8_dequantize<decltype(e8)::value, decltype(y32)::value><<<grid, THREADS, 0, stream>>>(p);
    });
  });
  return hipGetLastError();
}

}  // namespace fp4k
