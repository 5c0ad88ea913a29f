// Mixture-of-experts data movement on gfx950: stable sort of (token, choice) slots by expert,
// rows copied into expert order and summed back per token, and the gradients of both.
#include "experts.hpp"

namespace fp4k {

namespace {

// ---------------------------------------------------------------- sort
// Stable counting sort. A wave ranks 64 consecutive slots at a time: the lanes that hold the same
// key are found with one ballot per key bit, the rank of a lane among them is the population
// count below it, and the wave keeps its own running position per key in LDS, so ranks follow
// slot order and no atomic decides an order. Keys are the expert ids; a dropped slot has key E.
// Bound by latency: one launch up to 8192 slots (32 slots over 8 experts 3.3 us), else a launch that
// counts and one that places (262144 slots over 128 experts 11.5 us for 3.1 MB).
constexpr int SORT_ONE_WAVES = 16;       // the one-workgroup form
constexpr int SORT_ONE_MAX = 8192;       // slots it takes
constexpr int SORT_ONE_EXPERTS = 512;    // experts it takes (16 LDS rows of E + 1 counters below 64 KiB)
constexpr int SORT_WAVE_SLOTS = 256;     // slots of a wave in the form with one workgroup per chunk
// waves of that form: every workgroup sums its columns of the chunks' counts, so fewer, larger chunks
// are better (262144 slots, 128 experts: 13.6 us with 128 chunks of 8 waves)
constexpr int sort_waves(int E) { return E <= SORT_ONE_EXPERTS ? 16 : 8; }

template <bool ID64>
__device__ __forceinline__ uint32_t slot_key(const void* ids, int64_t ld, int topk, uint32_t slot, int E) {
  int64_t at = slot;
  if (ld != topk) {   // rows with a stride
    const uint32_t t = slot / (uint32_t)topk;
    at = (int64_t)t * ld + (slot - t * (uint32_t)topk);
  }
  if constexpr (ID64) {
    const int64_t id = reinterpret_cast<const int64_t*>(ids)[at];
    return id >= 0 && id < E ? (uint32_t)id : (uint32_t)E;
  } else {
    const int32_t id = reinterpret_cast<const int32_t*>(ids)[at];
    return id >= 0 && id < E ? (uint32_t)id : (uint32_t)E;
  }
}

__device__ __forceinline__ int wave_excl_scan(int v, int lane, int& total) {
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o, 64);
    if (lane >= o) s += u;
  }
  total = __shfl(s, 63, 64);
  return s - v;
}

// Exclusive scan of v over the workgroup's threads (NW waves); total in every thread.
template <int NW>
__device__ __forceinline__ int block_excl_scan(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int wt;
  const int x = wave_excl_scan(v, lane, wt);
  if (lane == 0) part[w] = wt;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int p = part[i];
    before += i < w ? p : 0;
    all += p;
  }
  __syncthreads();
  total = all;
  return before + x;
}

// The keys of the wave's slots [lo, hi), at most 64 NK of them: lane l's i-th is slot lo + 64 i + l.
// They are read once, all loads under way together, for both passes over them.
template <bool ID64, int NK>
__device__ __forceinline__ void wave_keys(const void* ids, int64_t ld, int topk, int E, int lo, int hi, uint32_t* key) {
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int s = lo + i * 64 + (threadIdx.x & 63);
    key[i] = s < hi ? slot_key<ID64>(ids, ld, topk, (uint32_t)s, E) : 0u;
  }
}

// Counts them into the wave's LDS row.
template <int NK>
__device__ __forceinline__ void wave_count(const uint32_t* key, int lo, int hi, int* row) {
#pragma unroll
  for (int i = 0; i < NK; ++i)
    if (lo + i * 64 + (int)(threadIdx.x & 63) < hi) atomicAdd(&row[key[i]], 1);
}

// Places them: row[key] is the wave's next position of each key.
template <int NK>
__device__ __forceinline__ void wave_place(const uint32_t* keys, int E, int bits, int lo, int hi, int* row,
                                           int32_t* order, int32_t* pos) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    if (lo + k * 64 >= hi) break;
    const int s = lo + k * 64 + lane;
    const bool ok = s < hi;
    const uint32_t key = keys[k];
    uint64_t same = __ballot(ok);
    for (int i = 0; i < bits; ++i) {
      const bool bit = (key >> i) & 1u;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    int p = 0;
    if (ok) p = row[key] + rank;
    wave_order();   // every lane has read its key's position before one lane of each key advances it
    if (ok && rank == 0) row[key] = p + __popcll(same);
    wave_order();
    if (ok) {
      order[p] = s;
      pos[s] = key < (uint32_t)E ? p : ~p;
    }
  }
}

template <bool ID64, int NK>
__global__ __launch_bounds__(SORT_ONE_WAVES * 64) void k_sort_one(const void* __restrict__ ids, int64_t ld, int topk,
                                                                  int n, int E, int bits, int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ pos,
                                                                  int32_t* __restrict__ offsets) {
  extern __shared__ int rows[];   // [SORT_ONE_WAVES][E + 1]
  __shared__ int part[SORT_ONE_WAVES];
  const int w = threadIdx.x >> 6, keys = E + 1;
  const int lo = min(n, w * 64 * NK), hi = min(n, lo + 64 * NK);
  uint32_t key[NK];
  wave_keys<ID64, NK>(ids, ld, topk, E, lo, hi, key);
  for (int i = threadIdx.x; i < SORT_ONE_WAVES * keys; i += SORT_ONE_WAVES * 64) rows[i] = 0;
  __syncthreads();
  wave_count<NK>(key, lo, hi, rows + w * keys);
  __syncthreads();
  // thread t < E: expert t's slots over the waves, its base, then each wave's first position
  const int t = threadIdx.x;
  int mine = 0;
  if (t < E)
    for (int i = 0; i < SORT_ONE_WAVES; ++i) mine += rows[i * keys + t];
  int kept;
  int base = block_excl_scan<SORT_ONE_WAVES>(mine, part, kept);
  if (t < E) {
    offsets[t] = base;
    for (int i = 0; i < SORT_ONE_WAVES; ++i) {
      const int c = rows[i * keys + t];
      rows[i * keys + t] = base;
      base += c;
    }
  }
  if (t == 0) {
    offsets[E] = kept;
    int b = kept;
    for (int i = 0; i < SORT_ONE_WAVES; ++i) {
      const int c = rows[i * keys + E];
      rows[i * keys + E] = b;
      b += c;
    }
  }
  __syncthreads();
  wave_place<NK>(key, E, bits, lo, hi, rows + w * keys, order, pos);
}

// no slots: the experts' offsets alone
__global__ __launch_bounds__(256) void k_sort_none(int E, int32_t* __restrict__ offsets) {
  for (int i = threadIdx.x; i <= E; i += 256) offsets[i] = 0;
}

// counts[chunk][E + 1]
template <bool ID64, int SORT_WAVES>
__global__ __launch_bounds__(SORT_WAVES * 64) void k_sort_count(const void* __restrict__ ids, int64_t ld, int topk,
                                                                int n, int E, int32_t* __restrict__ counts) {
  extern __shared__ int rows[];   // [E + 1]
  const int keys = E + 1;
  constexpr int NK = SORT_WAVE_SLOTS / 64;
  const int lo = min(n, (int)((blockIdx.x * SORT_WAVES + (threadIdx.x >> 6)) * SORT_WAVE_SLOTS));
  const int hi = lo + min(n - lo, SORT_WAVE_SLOTS);   // (lo + SORT_WAVE_SLOTS can pass 2^31)
  uint32_t key[NK];
  wave_keys<ID64, NK>(ids, ld, topk, E, lo, hi, key);
  for (int i = threadIdx.x; i < keys; i += SORT_WAVES * 64) rows[i] = 0;
  __syncthreads();
  wave_count<NK>(key, lo, hi, rows);
  __syncthreads();
  for (int i = threadIdx.x; i < keys; i += SORT_WAVES * 64) counts[(int64_t)blockIdx.x * keys + i] = rows[i];
}

// Each workgroup sums the counts of all chunks (its keys' totals) and of the chunks before its
// own, scans the totals into the experts' offsets and places its chunk.
template <bool ID64, int SORT_WAVES>
__global__ __launch_bounds__(SORT_WAVES * 64) void k_sort_place(const void* __restrict__ ids, int64_t ld, int topk,
                                                                int n, int E, int bits,
                                                                const int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ order, int32_t* __restrict__ pos,
                                                                int32_t* __restrict__ offsets) {
  extern __shared__ int lds[];   // total[E + 1], before[E + 1], rows[SORT_WAVES][E + 1]
  __shared__ int part[SORT_WAVES];
  constexpr int NTH = SORT_WAVES * 64;
  const int keys = E + 1, w = threadIdx.x >> 6, chunk = blockIdx.x, chunks = gridDim.x;
  int* total = lds;
  int* before = lds + keys;
  int* rows = lds + 2 * keys;
  constexpr int NK = SORT_WAVE_SLOTS / 64;
  const int lo = min(n, (chunk * SORT_WAVES + w) * SORT_WAVE_SLOTS), hi = lo + min(n - lo, SORT_WAVE_SLOTS);
  uint32_t key[NK];
  wave_keys<ID64, NK>(ids, ld, topk, E, lo, hi, key);
  for (int i = threadIdx.x; i < (2 + SORT_WAVES) * keys; i += NTH) lds[i] = 0;
  __syncthreads();
  wave_count<NK>(key, lo, hi, rows + w * keys);
  // the keys' columns of counts, `parts` threads to a key when there are few keys
  const int parts = keys >= NTH ? 1 : NTH / keys;
  if (threadIdx.x < parts * keys || keys >= NTH) {
    const int p = keys >= NTH ? 0 : threadIdx.x / keys;
    for (int k = keys >= NTH ? threadIdx.x : threadIdx.x - p * keys; k < keys; k += keys >= NTH ? NTH : keys) {
      int all = 0, pre = 0;
#pragma unroll 8
      for (int c = p; c < chunks; c += parts) {
        const int v = counts[(int64_t)c * keys + k];
        all += v;
        pre += c < chunk ? v : 0;
      }
      if (all) atomicAdd(&total[k], all);
      if (pre) atomicAdd(&before[k], pre);
    }
  }
  __syncthreads();
  int kept = 0;
  for (int k0 = 0; k0 < E; k0 += NTH) {
    const int k = k0 + threadIdx.x;
    int sum;
    int base = kept + block_excl_scan<SORT_WAVES>(k < E ? total[k] : 0, part, sum);
    kept += sum;
    if (k < E) {
      if (chunk == 0) offsets[k] = base;
      base += before[k];
      for (int i = 0; i < SORT_WAVES; ++i) {
        const int c = rows[i * keys + k];
        rows[i * keys + k] = base;
        base += c;
      }
    }
  }
  if (threadIdx.x == 0) {
    if (chunk == 0) offsets[E] = kept;
    int b = kept + before[E];
    for (int i = 0; i < SORT_WAVES; ++i) {
      const int c = rows[i * keys + E];
      rows[i * keys + E] = b;
      b += c;
    }
  }
  __syncthreads();
  wave_place<NK>(key, E, bits, lo, hi, rows + w * keys, order, pos);
}

// ---------------------------------------------------------------- rows to and from expert order
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Up to V consecutive elements of a row as float32: 16 bytes (8 bf16 or 4 float32). Rows that are
// not 16-byte aligned take the same 16-byte accesses at the alignment of their elements (the memory
// path allows that) and end in single elements.
template <bool F32, bool ALIGNED>
struct Elems {
  static constexpr int V = F32 ? 4 : 8, ESZ = F32 ? 4 : 2;
  static __device__ __forceinline__ float get(const char* p) {
    if constexpr (F32) return *reinterpret_cast<const float*>(p);
    else return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  }
  static __device__ __forceinline__ void put(char* p, float v) {
    if constexpr (F32) *reinterpret_cast<float*>(p) = v;
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(v, 0.0f);
  }
  // n elements are there; the others are zero
  static __device__ __forceinline__ void load(const char* p, int64_t n, float* v) {
    if (ALIGNED || n >= V) {
      v4u r;
      __builtin_memcpy(&r, ALIGNED ? __builtin_assume_aligned(p, 16) : __builtin_assume_aligned(p, ESZ), 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          v[i] = __uint_as_float(r[i]);
        } else {
          v[2 * i] = bf16_lo(r[i]);
          v[2 * i + 1] = bf16_hi(r[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < n ? get(p + i * ESZ) : 0.0f;
    }
  }
  static __device__ __forceinline__ void store(char* p, int64_t n, const float* v) {
    if (ALIGNED || n >= V) {
      v4u r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) r[i] = __float_as_uint(v[i]);
        else r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      }
      __builtin_memcpy(ALIGNED ? __builtin_assume_aligned(p, 16) : __builtin_assume_aligned(p, ESZ), &r, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) put(p + i * ESZ, v[i]);
    }
  }
  // The same as bits, not through float32: a NaN keeps its payload. (load and store written on top of
  // these took the gradient of a gather of 2047 x 4 rows of 1001 float32 from 8.0 to 8.6 us.)
  static __device__ __forceinline__ v4u load_bits(const char* p, int64_t n) {
    v4u r = {0, 0, 0, 0};
    if (ALIGNED || n >= V) {
      __builtin_memcpy(&r, ALIGNED ? __builtin_assume_aligned(p, 16) : __builtin_assume_aligned(p, ESZ), 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (F32) r[i] = reinterpret_cast<const uint32_t*>(p)[i];
          else r[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (i & 1) * 16;
        }
    }
    return r;
  }
  static __device__ __forceinline__ void store_bits(char* p, int64_t n, v4u r) {
    if (ALIGNED || n >= V) {
      __builtin_memcpy(ALIGNED ? __builtin_assume_aligned(p, 16) : __builtin_assume_aligned(p, ESZ), &r, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (F32) reinterpret_cast<uint32_t*>(p)[i] = r[i];
          else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(r[i / 2] >> (i & 1) * 16);
        }
    }
  }
};

constexpr int MT = 256;   // threads of the row kernels

// The three kernels below move rows and are bound by HBM; a workgroup takes a token (its row, and its
// topk rows in expert order), so each row is read or written once and in order. Measured: gather of
// 8192 x 2 rows of 4096 bf16 40 us (5.0 TB/s; a plain copy of 1 GiB reaches 5.2), gradient of a
// gather of 2047 x 4 rows of 1001 float32 8.0 us (5.1 TB/s), both gradients of the combination of
// 8192 x 2 rows 64 us (5.3 TB/s; 78 us with the weights' gradients in a pass of their own).

// One token's row to its slots' rows (gather): the row is read once and written topk times, bit for bit.
template <bool F32, bool ALIGNED>
__global__ __launch_bounds__(MT) void k_spread(const char* __restrict__ x, int64_t ldx, int64_t hidden,
                                               const int32_t* __restrict__ pos, int topk, int64_t n,
                                               char* __restrict__ xs, int64_t ldxs, int64_t tokens) {
  using E = Elems<F32, ALIGNED>;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
    for (int64_t h = ((int64_t)blockIdx.y * MT + threadIdx.x) * E::V; h < hidden; h += (int64_t)gridDim.y * MT * E::V) {
      const v4u v = E::load_bits(x + (t * ldx + h) * E::ESZ, hidden - h), zero = {0, 0, 0, 0};
      for (int j = 0; j < topk; ++j) {
        const int32_t p = pos[t * topk + j];
        const int64_t row = p < 0 ? ~p : p;
        if (row < n) E::store_bits(xs + (row * ldxs + h) * E::ESZ, hidden - h, p < 0 ? zero : v);
      }
    }
}

// A token's slots' rows summed, with weights or without.
template <bool F32, bool ALIGNED, bool WEIGHT>
__global__ __launch_bounds__(MT) void k_join(const char* __restrict__ ys, int64_t ldys, int64_t hidden,
                                             const int32_t* __restrict__ pos, int topk, int64_t n,
                                             const float* __restrict__ w, int64_t ldw, char* __restrict__ y,
                                             int64_t ldy, int64_t tokens) {
  using E = Elems<F32, ALIGNED>;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
    for (int64_t h = ((int64_t)blockIdx.y * MT + threadIdx.x) * E::V; h < hidden; h += (int64_t)gridDim.y * MT * E::V) {
      float a[E::V] = {};
      for (int j = 0; j < topk; ++j) {
        const int32_t p = pos[t * topk + j];
        if (p < 0 || p >= n) continue;
        float v[E::V];
        E::load(ys + ((int64_t)p * ldys + h) * E::ESZ, hidden - h, v);
        if constexpr (WEIGHT) {
          const float f = w[t * ldw + j];
#pragma unroll
          for (int i = 0; i < E::V; ++i) a[i] = __builtin_fmaf(f, v[i], a[i]);
        } else {
#pragma unroll
          for (int i = 0; i < E::V; ++i) a[i] += v[i];
        }
      }
      E::store(y + (t * ldy + h) * E::ESZ, hidden - h, a);
    }
}

// Gradient of the weighted sum: a workgroup takes a token's dy, scales it into its slots' rows of
// dys and multiplies it with their rows of ys for dw. dy is read once: R chunks of it stay in
// registers (longer rows read the rest again, from the caches).
constexpr int JB = 64;   // slots whose partial sums are kept at a time
template <bool F32, bool ALIGNED, int R>
__global__ __launch_bounds__(MT) void k_combine_grad(const char* __restrict__ dy, int64_t lddy,
                                                     const char* __restrict__ ys, int64_t ldys, int64_t hidden,
                                                     const float* __restrict__ w, int64_t ldw,
                                                     const int32_t* __restrict__ pos, int topk, int64_t n,
                                                     char* __restrict__ dys, int64_t lddys, float* __restrict__ dw,
                                                     int64_t lddw, int64_t tokens) {
  using E = Elems<F32, ALIGNED>;
  constexpr int STEP = MT * E::V;
  __shared__ float part[JB][MT / 64];
  const int64_t h0 = (int64_t)threadIdx.x * E::V;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    float u[R][E::V];
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int64_t h = h0 + c * STEP;
      if (h < hidden) {
        E::load(dy + (t * lddy + h) * E::ESZ, hidden - h, u[c]);
      } else {
#pragma unroll
        for (int i = 0; i < E::V; ++i) u[c][i] = 0.0f;
      }
    }
    for (int j0 = 0; j0 < topk; j0 += JB) {
      const int jn = min(JB, topk - j0);
      for (int j = 0; j < jn; ++j) {
        const int32_t p = pos[t * topk + j0 + j];
        const int64_t row = p < 0 ? ~p : p;
        const bool kept = p >= 0 && row < n;
        float a = 0.0f;
        if (row < n) {
          const float f = kept && dys ? w[t * ldw + j0 + j] : 0.0f;
          auto chunk = [&](int64_t h, const float* g) {
            if (dys) {
              float o[E::V];
#pragma unroll
              for (int i = 0; i < E::V; ++i) o[i] = kept ? f * g[i] : 0.0f;
              E::store(dys + (row * lddys + h) * E::ESZ, hidden - h, o);
            }
            if (kept && dw) {
              float v[E::V];
              E::load(ys + (row * ldys + h) * E::ESZ, hidden - h, v);
#pragma unroll
              for (int i = 0; i < E::V; ++i) a = __builtin_fmaf(g[i], v[i], a);
            }
          };
#pragma unroll
          for (int c = 0; c < R; ++c)
            if (h0 + c * STEP < hidden) chunk(h0 + c * STEP, u[c]);
          for (int64_t h = h0 + R * STEP; h < hidden; h += STEP) {
            float g[E::V];
            E::load(dy + (t * lddy + h) * E::ESZ, hidden - h, g);
            chunk(h, g);
          }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o, 64);
        if ((threadIdx.x & 63) == 0) part[j][threadIdx.x >> 6] = a;
      }
      __syncthreads();
      if (dw && threadIdx.x < jn)
        dw[t * lddw + j0 + threadIdx.x] = (part[threadIdx.x][0] + part[threadIdx.x][1]) + (part[threadIdx.x][2] + part[threadIdx.x][3]);
      __syncthreads();
    }
  }
}

bool vec_ok(const void* p, int64_t ld, int64_t esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * esz) % 16 == 0;
}

// f(F32, ALIGNED) with both as compile-time constants
template <class F>
void by_type(bool f32, bool vec, F&& f) {
  if (f32) vec ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  else vec ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

// workgroups over tokens: a grid holds less than 2^32 threads, so past this many each takes several
uint32_t token_grid(int64_t tokens) { return (uint32_t)std::min<int64_t>(tokens, int64_t(1) << 22); }

dim3 row_grid(const RowsArgs& a) {
  return dim3(token_grid(a.tokens), (uint32_t)std::min<int64_t>(div_up(a.hidden, MT * (a.f32 ? 4 : 8)), 1024));
}

bool sort_in_one(int64_t n, int E) { return n <= SORT_ONE_MAX && E <= SORT_ONE_EXPERTS; }

}  // namespace

size_t expert_sort_ws(int64_t n, int E) {
  return sort_in_one(n, E) ? 0 : (size_t)div_up(n, sort_waves(E) * SORT_WAVE_SLOTS) * (size_t)(E + 1) * sizeof(int32_t);
}

hipError_t run_expert_sort(const SortArgs& a) {
  const int n = (int)(a.tokens * a.topk), E = a.n_experts;
  int bits = 0;
  while ((E >> bits) != 0) ++bits;   // keys 0 .. E
  if (n == 0) {   // no chunk to launch a workgroup for
    k_sort_none<<<1, 256, 0, a.stream>>>(E, a.offsets);
    return hipGetLastError();
  }
  auto go = [&](auto id64) {
    constexpr bool ID64 = decltype(id64)::value;
    if (sort_in_one(n, E)) {
      auto one = [&](auto nk) {
        constexpr int NK = decltype(nk)::value;
        k_sort_one<ID64, NK><<<1, SORT_ONE_WAVES * 64, SORT_ONE_WAVES * (E + 1) * sizeof(int), a.stream>>>(a.ids, a.ld_ids, a.topk, n, E, bits, a.order, a.pos, a.offsets);
      };
      if (n <= SORT_ONE_WAVES * 64) one(std::integral_constant<int, 1>{});
      else if (n <= SORT_ONE_WAVES * 128) one(std::integral_constant<int, 2>{});
      else one(std::integral_constant<int, SORT_ONE_MAX / (SORT_ONE_WAVES * 64)>{});
      return;
    }
    int32_t* counts = reinterpret_cast<int32_t*>(a.ws);
    auto chunked = [&](auto waves) {
      constexpr int W = decltype(waves)::value;
      const uint32_t chunks = (uint32_t)div_up(n, W * SORT_WAVE_SLOTS);
      k_sort_count<ID64, W><<<chunks, W * 64, (E + 1) * sizeof(int), a.stream>>>(a.ids, a.ld_ids, a.topk, n, E, counts);
      k_sort_place<ID64, W><<<chunks, W * 64, (2 + W) * (E + 1) * sizeof(int), a.stream>>>(a.ids, a.ld_ids, a.topk, n, E, bits, counts, a.order, a.pos, a.offsets);
    };
    if (sort_waves(E) == 16) chunked(std::integral_constant<int, 16>{});
    else chunked(std::integral_constant<int, 8>{});
  };
  if (a.id64) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

hipError_t run_expert_gather(const RowsArgs& a) {
  if (a.tokens == 0 || a.hidden == 0) return hipSuccess;
  const int64_t esz = a.f32 ? 4 : 2, v = a.f32 ? 4 : 8;
  const bool al = a.hidden % v == 0 && vec_ok(a.tok, a.ld_tok, esz) && vec_ok(a.rows, a.ld_rows, esz);
  by_type(a.f32, al, [&](auto f32, auto al_) {
    constexpr bool F32 = decltype(f32)::value, AL = decltype(al_)::value;
    k_spread<F32, AL><<<row_grid(a), MT, 0, a.stream>>>((const char*)a.tok, a.ld_tok, a.hidden, a.pos, a.topk,
                                                        a.tokens * a.topk, (char*)a.rows, a.ld_rows, a.tokens);
  });
  return hipGetLastError();
}

hipError_t run_expert_join(const RowsArgs& a) {
  if (a.tokens == 0 || a.hidden == 0) return hipSuccess;
  const int64_t esz = a.f32 ? 4 : 2, v = a.f32 ? 4 : 8, n = a.tokens * a.topk;
  const bool al = a.hidden % v == 0 && vec_ok(a.tok, a.ld_tok, esz) && vec_ok(a.rows, a.ld_rows, esz);
  by_type(a.f32, al, [&](auto f32, auto al_) {
    constexpr bool F32 = decltype(f32)::value, AL = decltype(al_)::value;
    const char* rows = (const char*)a.rows;
    if (a.w) k_join<F32, AL, true><<<row_grid(a), MT, 0, a.stream>>>(rows, a.ld_rows, a.hidden, a.pos, a.topk, n, a.w, a.ldw, (char*)a.tok, a.ld_tok, a.tokens);
    else k_join<F32, AL, false><<<row_grid(a), MT, 0, a.stream>>>(rows, a.ld_rows, a.hidden, a.pos, a.topk, n, nullptr, 0, (char*)a.tok, a.ld_tok, a.tokens);
  });
  return hipGetLastError();
}

hipError_t run_expert_combine_grad(const CombineGradArgs& a) {
  if (a.tokens == 0 || (!a.dys && !a.dw)) return hipSuccess;
  const int64_t esz = a.f32 ? 4 : 2, v = a.f32 ? 4 : 8, n = a.tokens * a.topk;
  const bool al = a.hidden % v == 0 && vec_ok(a.dy, a.lddy, esz) && (!a.dw || vec_ok(a.ys, a.ldys, esz)) &&
                  (!a.dys || vec_ok(a.dys, a.lddys, esz));
  by_type(a.f32, al, [&](auto f32, auto al_) {
    constexpr bool F32 = decltype(f32)::value, AL = decltype(al_)::value;
    auto go = [&](auto r) {
      constexpr int R = decltype(r)::value;
      k_combine_grad<F32, AL, R><<<token_grid(a.tokens), MT, 0, a.stream>>>((const char*)a.dy, a.lddy, (const char*)a.ys, a.ldys, a.hidden, a.w, a.ldw, a.pos, a.topk, n, (char*)a.dys, a.lddys, a.dw, a.lddw, a.tokens);
    };
    if (a.hidden <= MT * v) go(std::integral_constant<int, 1>{});
    else if (a.hidden <= 2 * MT * v) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
  });
  return hipGetLastError();
}

}  // namespace fp4k
