// E4M3 quantizers with one scale to each 128 elements of a row, of a column, or to each 128 x 128
// tile, their decode, and the gradient of the gated projections, plain or quantized in the same pass.
//
// A workgroup takes a 128 x 128 tile, which holds whole blocks of every view, so one read of the
// input serves all of them. Thread (tr, tc) = (id / 16, id % 16) holds the 8 x 8 elements of rows
// 8 tr .. and columns 8 tc ..: a row's block is 16 neighbouring lanes, a column's one lane in 16 of
// every wave. Row codes go straight to memory, 128 consecutive bytes from 16 lanes; column codes turn
// in LDS, where a thread has 8 consecutive bytes of each of its columns.
#include "fp8.hpp"

namespace fp4k {

namespace {

constexpr int T = F8_BLOCK, THREADS = 256;

struct Tile {
  int64_t r0, c0;    // first row and column
  int rows, cols;    // what there is of the tile's
};

// 8 elements of a row from column c on (those of `have`; zeros for the rest)
template <bool F32, bool VEC>
__device__ __forceinline__ void load_row8(const char* row, int64_t c, int have, float* v) {
  if (VEC && have >= 8) {
    if constexpr (F32) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c * 4), b = *reinterpret_cast<const uint4*>(row + c * 4 + 16);
      v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c * 2);
      v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
      v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < have) {
      if constexpr (F32) v[j] = reinterpret_cast<const float*>(row)[c + j];
      else v[j] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[c + j] << 16);
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

struct Lds {
  uint32_t part[4][T];          // columns' maxima, a row of them per wave
  __attribute__((aligned(16))) uint8_t codes[T * T];
};

// v[p][j]: element (8 tr + p, 8 tc + j), zeros outside the tensor. VIEW: F8_VIEW_*.
template <int VIEW, bool E8>
__device__ __forceinline__ void quantize_tile(const float (&v)[8][8], const Tile& t, const TileOut& o, Lds& lds) {
  constexpr bool ROW = VIEW != F8_VIEW_COL, COL = VIEW != F8_VIEW_ROW, GRID = VIEW == F8_VIEW_TILE2D;
  const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15, wave = tid >> 6;
  float tile_enc = 0.0f;
  if constexpr (GRID) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[p][j]));
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, x, 64));
    if ((tid & 63) == 0) lds.part[wave][0] = m;
    __syncthreads();
    m = max(max(lds.part[0][0], lds.part[1][0]), max(lds.part[2][0], lds.part[3][0]));
    const F8Scale s = f8_scale<E8>(m);
    tile_enc = s.enc;
    if (tid == 0) store_scale<E8>(o.s, (o.row0 / T) * o.sld + o.col0 / T, s.code);
  }
  if constexpr (ROW) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int r = tr * 8 + p;
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
        uint2 w;
        w.x = f8_pack4(v[p][0] * enc, v[p][1] * enc, v[p][2] * enc, v[p][3] * enc);
        w.y = f8_pack4(v[p][4] * enc, v[p][5] * enc, v[p][6] * enc, v[p][7] * enc);
        *reinterpret_cast<uint2*>(o.q + (o.row0 + r) * o.kp + o.col0 + tc * 8) = w;
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
        for (int p = 0; p < 8; ++p) m = max(m, mag_bits(v[p][j]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if ((tid & 63) < 16) lds.part[wave][tc * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = tc * 8 + j;
        const F8Scale s = f8_scale<E8>(max(max(lds.part[0][c], lds.part[1][c]), max(lds.part[2][c], lds.part[3][c])));
        enc[j] = s.enc;
        if (tr == 0 && c < t.cols) store_scale<E8>(o.st, (o.trow0 + c) * o.stld + o.tcol0 / T, s.code);
      }
    }
    // column c keeps its 16-byte piece i at i ^ (c / 8 % 8): 16 lanes of one row group fall on all banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint2 w;
      w.x = f8_pack4(v[0][j] * enc[j], v[1][j] * enc[j], v[2][j] * enc[j], v[3][j] * enc[j]);
      w.y = f8_pack4(v[4][j] * enc[j], v[5][j] * enc[j], v[6][j] * enc[j], v[7][j] * enc[j]);
      *reinterpret_cast<uint2*>(lds.codes + (tc * 8 + j) * T + ((((tr >> 1) ^ (tc & 7)) << 4) | ((tr & 1) << 3))) = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T * T / 16 / THREADS; ++i) {
      const int at = i * THREADS + tid, c = at >> 3, piece = at & 7;
      if (c < t.cols)   // (codes past the rows are those of the zeros there)
        *reinterpret_cast<uint4*>(o.qt + (o.trow0 + c) * o.ktp + o.tcol0 + piece * 16) =
            *reinterpret_cast<const uint4*>(lds.codes + c * T + ((piece ^ ((c >> 3) & 7)) << 4));
    }
  }
}

struct QuantParams {
  const char* x;
  int64_t rows, cols, ld, tiles_c;
  TileOut out;
};

template <int VIEW, bool F32, bool VEC, bool E8>
__global__ __launch_bounds__(THREADS) void k_f8_quantize(QuantParams p) {
  __shared__ Lds lds;
  const int64_t br = blockIdx.x / p.tiles_c, bc = blockIdx.x - br * p.tiles_c;
  const Tile t{br * T, bc * T, (int)min((int64_t)T, p.rows - br * T), (int)min((int64_t)T, p.cols - bc * T)};
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = tr * 8 + i;
    load_row8<F32, VEC>(p.x + (t.r0 + r) * p.ld * (F32 ? 4 : 2), t.c0 + tc * 8, r < t.rows ? t.cols - tc * 8 : 0, v[i]);
  }
  TileOut o = p.out;
  o.row0 = o.tcol0 = t.r0;
  o.col0 = o.trow0 = t.c0;
  quantize_tile<VIEW, E8>(v, t, o, lds);
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
  const float p = act_gate<ACT>(g);
  dg = dh * u * act_slope<ACT>(g, p);
  du = dh * (g * p);
}

template <int VIEW, int ACT, bool F32, bool VEC, bool E8>
__global__ __launch_bounds__(THREADS) void k_f8_gated_grad(GradParams p) {
  __shared__ Lds lds;
  constexpr int ES = F32 ? 4 : 2;
  const int64_t br = blockIdx.x / p.tiles_c, bc = blockIdx.x - br * p.tiles_c;
  const Tile t{br * T, bc * T, (int)min((int64_t)T, p.rows - br * T), T};   // f is a multiple of T
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  float dg[8][8], du[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = tr * 8 + i, have = r < t.rows ? 8 : 0;
    const int64_t c = t.c0 + tc * 8;
    const char* gu = p.gu + (t.r0 + r) * p.ldgu * ES;
    float h[8];
    load_row8<F32, VEC>(p.dh + (t.r0 + r) * p.lddh * ES, c, have, h);
    load_row8<F32, VEC>(gu, c, have, dg[i]);
    load_row8<F32, VEC>(gu, p.f + c, have, du[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) gated_grad1<ACT>(h[j], dg[i][j], du[i][j], dg[i][j], du[i][j]);
  }
  TileOut o = p.out;
  o.row0 = o.tcol0 = t.r0;
  o.col0 = o.trow0 = t.c0;
  quantize_tile<VIEW, E8>(dg, t, o, lds);
  if constexpr (VIEW != F8_VIEW_ROW) __syncthreads();   // the first half's codes have been read
  o.col0 = o.trow0 = p.f + t.c0;
  quantize_tile<VIEW, E8>(du, t, o, lds);
}

// One thread to 8 elements of a row of dh.
template <int ACT, bool F32, bool VEC>
__global__ __launch_bounds__(THREADS) void k_gated_grad(GradParams p) {
  constexpr int ES = F32 ? 4 : 2;
  const int64_t per = (p.f + 7) / 8, n = p.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS) {
    const int64_t r = i / per, c = (i - r * per) * 8;
    const int have = (int)min((int64_t)8, p.f - c);
    const char* gu = p.gu + r * p.ldgu * ES;
    char* out = p.dgu + r * p.lddgu * ES;
    float h[8], a[2][8];
    load_row8<F32, VEC>(p.dh + r * p.lddh * ES, c, have, h);
    load_row8<F32, VEC>(gu, c, have, a[0]);
    load_row8<F32, VEC>(gu, p.f + c, have, a[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) gated_grad1<ACT>(h[j], a[0][j], a[1][j], a[0][j], a[1][j]);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int64_t at = o * p.f + c;
      if (VEC && have >= 8) {
        if constexpr (F32) {
          *reinterpret_cast<float4*>(out + at * 4) = float4{a[o][0], a[o][1], a[o][2], a[o][3]};
          *reinterpret_cast<float4*>(out + at * 4 + 16) = float4{a[o][4], a[o][5], a[o][6], a[o][7]};
        } else {
          *reinterpret_cast<uint4*>(out + at * 2) = uint4{pack_bf16(a[o][0], a[o][1]), pack_bf16(a[o][2], a[o][3]),
                                                          pack_bf16(a[o][4], a[o][5]), pack_bf16(a[o][6], a[o][7])};
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < have) {
            if constexpr (F32) reinterpret_cast<float*>(out)[at + j] = a[o][j];
            else reinterpret_cast<uint16_t*>(out)[at + j] = (uint16_t)pack_bf16(a[o][j], 0.0f);
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

hipError_t run_f8_quantize(const F8QuantArgs& a) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  QuantParams p{(const char*)a.x, a.rows, a.cols, a.ld, blocks(a.cols),
                tile_out(a.rows, a.cols, a.view == F8_VIEW_TILE2D, a.q, a.s, a.qt, a.st)};
  const uint32_t grid = (uint32_t)(blocks(a.rows) * p.tiles_c);
  auto view = [&](auto v) {
    with_bool(a.f32, [&](auto f32) {
      with_bool(vec_rows(a.x, a.ld, a.f32), [&](auto vec) {
        with_bool(a.e8, [&](auto e8) {
          k_f8_quantize<decltype(v)::value, decltype(f32)::value, decltype(vec)::value, decltype(e8)::value>
              <<<grid, THREADS, 0, a.stream>>>(p);
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
            k_f8_gated_grad<decltype(v)::value, decltype(act)::value, decltype(f32)::value, decltype(vec)::value,
                            decltype(e8)::value><<<grid, THREADS, 0, a.stream>>>(p);
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
