// Rows in expert order on gfx950: the rows of each expert and the tiles that they make. P holds
// offsets (device int32 [n_experts + 1], or null for one group of all rows), n_experts and rows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4k {

// The rows [lo, hi) of group e (all rows without offsets); the offsets come from device memory
// and are clamped to the tensor.
template <class P>
__device__ __forceinline__ void group_rows(const P& p, int e, int64_t& lo, int64_t& hi) {
  if (!p.offsets) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = min(max((int64_t)p.offsets[e], (int64_t)0), p.rows);
  hi = e == p.n_experts ? p.rows : min(max((int64_t)p.offsets[e + 1], lo), p.rows);
}

// The m-tiles of the grouped rows: the experts' tiles follow each other, the rows of dropped slots
// are the last group. Lane l holds group l of the current 64 (all of them for up to 63 experts).
template <int BM, class P>
struct TileMap {
  int lo, hi, tiles, upto;   // rows, tiles, tiles of this and the groups before it (in the 64)
  __device__ __forceinline__ void load(const P& p, int g0) {
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
  __device__ __forceinline__ uint32_t count(const P& p) {
    int n = 0;
    for (int g0 = (p.n_experts / 64) * 64; g0 >= 0; g0 -= 64) {
      load(p, g0);
      n += __shfl(upto, 63, 64);
    }
    return __builtin_amdgcn_readfirstlane(n);
  }
  // after count(): tile mt's group, first row and the group's end, wave-uniform; mt is below the count
  __device__ __forceinline__ void find(const P& p, int mt, int& e, int64_t& m0, int64_t& m1) {
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

}  // namespace fp4k
