// moe.hip -- tokens sorted by expert, their rows gathered, the experts' rows
// summed back with the routing weights, and the gradients of both (gfx950).
//
// A slot f = t * topk + j is token t's j-th expert.  The sort is a stable counting
// sort of the slots by expert; a slot whose id is outside [0, E) has no expert and
// comes last.  order[row] = f and place[f] = row for a slot with an expert, ~f and
// ~row for one without, so both arrays are whole permutations whose sign says
// whether the row takes part.
#include "nf4_check.h"
#include "nf4_device.h"

namespace nf4 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ sort ----
// Each wave owns up to kSortGroups groups of 64 consecutive slots, whose keys it holds in
// registers from one load.  Up to 64 * kSortGroups slots a wave one workgroup counts,
// scans and ranks by itself; beyond that three kernels do, a workgroup per chunk.  Bound
// by latency up to tens of thousands of slots: 5 x 2 slots 2.4 us, 2048 x 2 6.3, 8191 x 4
// 12 in three launches back to back (kernels of 5.0, 5.1 and 5.7-6.2 when traced apart).
constexpr int kSortGroups = 8;
constexpr int kSortMaxE = NF4_MOE_MAX_E;
// Slots of a chunk (the last one takes what is left, less than two chunks).  More
// than kSortMaxE, so that a chunk's counts fit the part of `place` that is the chunk's.
constexpr int kSortChunk = 2048;
constexpr int kChunkWaves = 8;
static_assert(kSortMaxE < kSortChunk && 2 * kSortChunk <= kChunkWaves * 64 * kSortGroups, "chunks");
static_assert(kSortMaxE < 1024, "a thread for every key in the scan");

// Keys of the wave's slots from `a` up to `b` (kept, ~none above E): lane l of group i
// holds slot a + 64 i + l.  Returns whether an id was neither -1 nor an expert.
__device__ __forceinline__ bool load_keys(const int64_t *experts, int64_t a, int64_t b, int E,
                                          int lane, int key[kSortGroups]) {
  int64_t id[kSortGroups];
#pragma unroll
  for (int i = 0; i < kSortGroups; ++i) {
    const int64_t f = a + i * 64 + lane;
    id[i] = f < b ? experts[f] : -1;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kSortGroups; ++i) {
    const bool in = id[i] >= 0 && id[i] < E;
    bad |= !in && id[i] != -1;
    key[i] = in ? (int)id[i] : E;
  }
  return bad;
}

// Adds the wave's keys to cnt[0 .. E].
__device__ __forceinline__ void count_keys(const int key[kSortGroups], int64_t a, int64_t b,
                                           int *cnt, int lane) {
#pragma unroll
  for (int i = 0; i < kSortGroups; ++i)
    if (a + i * 64 + lane < b) atomicAdd(&cnt[key[i]], 1);
}

// Lanes of the wave that hold the same key, by one ballot per key bit.
__device__ __forceinline__ uint64_t same_key(int key, bool active, int bits) {
  uint64_t m = __ballot(active);
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Exclusive prefix over the threads of the workgroup.
template <int WAVES>
__device__ __forceinline__ int block_exclusive(int v, int *wsum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) base += w < wave ? wsum[w] : 0;
  return base + s - v;
}

// The slots of workgroup b, then of a wave: runs in slot order.
template <int WAVES>
__device__ __forceinline__ void wave_slots(int64_t R, int64_t *f0, int64_t *a, int64_t *b) {
  *f0 = (int64_t)blockIdx.x * kSortChunk;
  const int64_t f1 = blockIdx.x + 1 == gridDim.x ? R : *f0 + kSortChunk;
  const int64_t groups = (f1 - *f0 + 63) / 64;
  const int64_t per = (groups + WAVES - 1) / WAVES * 64;
  const int64_t lo = *f0 + (threadIdx.x >> 6) * per;
  *a = lo < f1 ? lo : f1;
  *b = lo + per < f1 ? lo + per : f1;
}

__global__ void __launch_bounds__(64 * kChunkWaves)
    moe_count_kernel(const int64_t *__restrict__ experts, int64_t R, int E,
                     int32_t *__restrict__ place, int32_t *status) {
  __shared__ int cnt[kSortMaxE + 1];
  int64_t f0, a, b;
  wave_slots<kChunkWaves>(R, &f0, &a, &b);
  const int lane = threadIdx.x & 63;
  int key[kSortGroups];
  const bool bad = load_keys(experts, a, b, E, lane, key);
  for (int e = threadIdx.x; e <= E; e += 64 * kChunkWaves) cnt[e] = 0;
  __syncthreads();
  count_keys(key, a, b, cnt, lane);
  if (bad && status) atomicOr(status, NF4_MOE_BAD_ID);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += 64 * kChunkWaves) place[f0 + e] = cnt[e];
}

// One workgroup: the chunks' counts become each chunk's first row per key; key E (no
// expert) follows every expert's rows.  Thread (g, e) has key e and the g-th share of the
// chunks (2^shift > E keys).  The whole sort, us: 131072 x 8 slots of 64 experts 23.5 (one
// share: 72), of 256 experts 51 (76), 4194304 x 8 of 32 406 (2634).
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads)
    moe_scan_kernel(int nchunks, int E, int shift, int32_t *__restrict__ place,
                    int32_t *__restrict__ offsets) {
  __shared__ int part[kScanThreads], start[kScanThreads], wsum[kScanThreads / 64];
  const int e = threadIdx.x & ((1 << shift) - 1), g = threadIdx.x >> shift;
  const int shares = kScanThreads >> shift, per = (nchunks + shares - 1) / shares;
  const int first = min(g * per, nchunks), last = min(first + per, nchunks);
  int n = 0;
  if (e <= E)
    for (int c0 = first; c0 < last; c0 += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) n += c0 + i < last ? place[(int64_t)(c0 + i) * kSortChunk + e] : 0;
    }
  part[threadIdx.x] = n;
  __syncthreads();
  int total = 0;
  if (g == 0)
    for (int k = 0; k < shares; ++k) total += part[k << shift | e];
  const int base = block_exclusive<kScanThreads / 64>(total, wsum);
  if (g == 0) {
    start[e] = base;
    if (e <= E) offsets[e] = base;
  }
  __syncthreads();
  if (e > E) return;
  int row = start[e];
  for (int k = 0; k < g; ++k) row += part[k << shift | e];
  for (int c0 = first; c0 < last; c0 += 8) {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = c0 + i < last ? place[(int64_t)(c0 + i) * kSortChunk + e] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c0 + i < last) place[(int64_t)(c0 + i) * kSortChunk + e] = row;
      row += v[i];
    }
  }
}

// Ranks and writes a chunk's slots.  SINGLE: the chunk is everything, and this
// kernel counts and scans by itself (E < 64 WAVES).
template <int WAVES, bool SINGLE>
__global__ void __launch_bounds__(64 * WAVES)
    moe_scatter_kernel(const int64_t *__restrict__ experts, int64_t R, int E, int bits,
                       int32_t *__restrict__ offsets, int32_t *__restrict__ order,
                       int32_t *__restrict__ place, int32_t *status) {
  extern __shared__ int cnt[];  // [WAVES][E + 1], then wave sums
  int *wsum = cnt + WAVES * (E + 1);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t f0, a, b;
  wave_slots<WAVES>(R, &f0, &a, &b);
  int key[kSortGroups];
  const bool bad = load_keys(experts, a, b, E, lane, key);
  for (int i = threadIdx.x; i < WAVES * (E + 1); i += 64 * WAVES) cnt[i] = 0;
  __syncthreads();
  int *mine = cnt + wave * (E + 1);
  count_keys(key, a, b, mine, lane);
  if (SINGLE && bad && status) atomicOr(status, NF4_MOE_BAD_ID);
  __syncthreads();
  // first row of each key in this chunk, then of each wave
  const int e = threadIdx.x;
  if constexpr (SINGLE) {
    int n = 0;
    if (e <= E)
#pragma unroll
      for (int w = 0; w < WAVES; ++w) n += cnt[w * (E + 1) + e];
    const int base = block_exclusive<WAVES>(n, wsum);
    if (e <= E) offsets[e] = base;
    if (e <= E) {
      int row = base;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int v = cnt[w * (E + 1) + e];
        cnt[w * (E + 1) + e] = row;
        row += v;
      }
    }
  } else {
    for (int k = e; k <= E; k += 64 * WAVES) {
      int row = place[f0 + k];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int v = cnt[w * (E + 1) + k];
        cnt[w * (E + 1) + k] = row;
        row += v;
      }
    }
  }
  __syncthreads();  // also: this chunk's part of `place` is read before it is written
  const uint64_t below = lane ? ~uint64_t(0) >> (64 - lane) : 0;
#pragma unroll
  for (int i = 0; i < kSortGroups; ++i) {
    const int64_t f = a + i * 64 + lane;
    if (a + i * 64 >= b) break;
    const bool active = f < b;
    const uint64_t peers = same_key(active ? key[i] : 0, active, bits);
    if (active) {
      const int row = mine[key[i]] + __popcll(peers & below);
      const bool kept = key[i] < E;
      place[f] = kept ? row : ~row;
      order[row] = kept ? (int)f : ~(int)f;
    }
    // every lane of the wave has read its count before a leader adds to it, and
    // the next group reads what the leaders left
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (active && (peers & below) == 0) mine[key[i]] += __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int WAVES, bool SINGLE>
static void launch_scatter(unsigned chunks, const int64_t *experts, int64_t R, int E,
                           int32_t *offsets, int32_t *order, int32_t *place, int32_t *status,
                           hipStream_t s) {
  int bits = 1;
  while ((1 << bits) <= E) ++bits;
  const size_t lds = (size_t)(WAVES * (E + 1) + WAVES) * sizeof(int);
  hipLaunchKernelGGL((moe_scatter_kernel<WAVES, SINGLE>), dim3(chunks), dim3(64 * WAVES), lds, s,
                     experts, R, E, bits, offsets, order, place, status);
}

__global__ void moe_clear_status_kernel(int32_t *status) { *status = 0; }

// ------------------------------------------------------- rows by place ----
// A row is cut into chunks of 16 bytes; 2^shift threads share a token, each taking
// every 2^shift-th chunk.  The last chunk of a row that is no whole number of them
// ends with the row and overlaps the one before (rows shorter than a chunk go by the
// element).  ALIGNED: rows and arrays are multiples of 16 bytes; otherwise they have
// the alignment of an element, which the vector loads and stores of the hardware
// take as well (1000 x 3 rows of 1001 bf16: combine 8.8 us by the element).
// STREAM: the rows are more than the L2 caches hold and go past them (8191 x 4 rows
// of 4 KiB: combine 35.4 -> 29.4 us, gather 35.1 -> 26.7; rows that fit are
// slower so: 4000 x 2 of 1.3 KiB, combine 8.3 -> 10.7).
struct RowMap {
  int shift;   // log2 of the threads per token
  int chunks;  // chunks per row
  int bytes;   // of a row
};

template <typename T, int V, bool ALIGNED, bool STREAM>
struct Rows {
  static constexpr int n = V / (int)sizeof(T);  // values of a chunk
  typedef Rows<T, V, ALIGNED, false> Kept;      // (the gather's own rows: 32.1 us past the caches)
  struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    u32x4 v;
  };
  static __device__ __forceinline__ int offset(const RowMap &m, int c) {
    return V == 16 && !ALIGNED ? min(c * 16, m.bytes - 16) : c * V;
  }
  // values at the front of chunk c that the chunk before has, too
  static __device__ __forceinline__ int shared(const RowMap &m, int c) {
    return (c * V - offset(m, c)) / (int)sizeof(T);
  }
  static __device__ __forceinline__ const uint8_t *at(const void *p, const RowMap &m, int64_t row, int c) {
    return reinterpret_cast<const uint8_t *>(p) + row * m.bytes + offset(m, c);
  }
  static __device__ __forceinline__ u32x4 load(const void *p, const RowMap &m, int64_t row, int c) {
    const uint8_t *q = at(p, m, row, c);
    if constexpr (V == 16 && ALIGNED && STREAM)
      return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(q));
    else if constexpr (V == 16 && ALIGNED)
      return *reinterpret_cast<const u32x4 *>(q);
    else if constexpr (V == 16)
      return reinterpret_cast<const Loose *>(q)->v;
    else
      return u32x4{(uint32_t)*reinterpret_cast<const T *>(q), 0u, 0u, 0u};
  }
  static __device__ __forceinline__ void store(void *p, const RowMap &m, int64_t row, int c, u32x4 v) {
    uint8_t *q = const_cast<uint8_t *>(at(p, m, row, c));
    if constexpr (V == 16 && ALIGNED && STREAM)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(q));
    else if constexpr (V == 16 && ALIGNED)
      *reinterpret_cast<u32x4 *>(q) = v;
    else if constexpr (V == 16)
      reinterpret_cast<Loose *>(q)->v = v;
    else
      *reinterpret_cast<T *>(q) = (T)v[0];
  }
  // fp32 values of a chunk and back (bf16: one rounding to nearest even)
  static __device__ __forceinline__ void values(const u32x4 &c, float *v) {
#pragma unroll
    for (int i = 0; i < n; ++i)
      v[i] = sizeof(T) == 4 ? __uint_as_float(c[i]) : i % 2 ? bf16_hi(c[i / 2]) : bf16_lo(c[i / 2]);
  }
  static __device__ __forceinline__ uint32_t bits(float f) {
    return sizeof(T) == 4 ? __float_as_uint(f) : (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ u32x4 chunk(const float *v) {
    u32x4 c = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (sizeof(T) == 4)
        c[i] = bits(v[i]);
      else
        c[i / 2] |= bits(v[i]) << (16 * (i % 2));
    }
    return c;
  }
};

// place[f] as a row, -1 where the slot has no expert or the entry is no row
__device__ __forceinline__ int kept_row(int p, int R) { return p >= 0 && p < R ? p : -1; }

// P[row] = X[t] for every slot of token t, zeros in the rows without an expert; a row
// of X is read once.  Memory: 8191 x 4 rows of 2048 bf16 25.5 us, 6.6 TB/s.
template <typename ROWS>
__global__ void __launch_bounds__(256)
    moe_gather_kernel(const void *__restrict__ X, const int32_t *__restrict__ place, int64_t T,
                      int topk, RowMap map, void *__restrict__ out) {
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = g >> map.shift;
  if (t >= T) return;
  const int R = (int)(T * topk);
  for (int c = (int)(g & ((1 << map.shift) - 1)); c < map.chunks; c += 1 << map.shift) {
    const u32x4 v = ROWS::Kept::load(X, map, t, c);
    for (int j = 0; j < topk; ++j) {
      const int p = place[t * topk + j];
      const int row = p < 0 ? ~p : p;
      if (row < R) ROWS::store(out, map, row, c, p < 0 ? u32x4{0u, 0u, 0u, 0u} : v);
    }
  }
}

// out[t] = sum_j w[t,j] Y[place[t,j]] in fp32, j in order (WEIGHTED false: w = 1); four
// slots' loads in flight.  Memory: 8191 x 4 rows of 2048 bf16 29 us, 5.8 TB/s.
template <typename ROWS, bool WEIGHTED>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const void *__restrict__ Y, const int32_t *__restrict__ place,
                       const float *__restrict__ weights, int64_t T, int topk, RowMap map,
                       void *__restrict__ out) {
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = g >> map.shift;
  if (t >= T) return;
  const int R = (int)(T * topk);
  for (int c = (int)(g & ((1 << map.shift) - 1)); c < map.chunks; c += 1 << map.shift) {
    float acc[ROWS::n] = {};
    for (int j0 = 0; j0 < topk; j0 += 4) {
      u32x4 y[4];
      float w[4];
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = j0 + j < topk ? kept_row(place[t * topk + j0 + j], R) : -1;
        on[j] = row >= 0;
        w[j] = 1.0f;
        if (on[j]) {
          y[j] = ROWS::load(Y, map, row, c);
          if constexpr (WEIGHTED) w[j] = weights[t * topk + j0 + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!on[j]) continue;
        float v[ROWS::n];
        ROWS::values(y[j], v);
#pragma unroll
        for (int i = 0; i < ROWS::n; ++i) acc[i] = WEIGHTED ? fmaf(w[j], v[i], acc[i]) : acc[i] + v[i];
      }
    }
    ROWS::store(out, map, t, c, ROWS::chunk(acc));
  }
}

// dY[place[t,j]] = w[t,j] dOut[t]; dw[t,j] = <dOut[t], Y[place[t,j]]> in fp32.
// L threads per token (64: four tokens a workgroup; 256: one).  Slots are taken
// four at a time; each thread's partial sums are added over the wave, then over
// the waves in order.  Memory: 8191 x 4 rows of 2048 bf16 54.5 us, 5.5 TB/s.
template <typename ROWS, int L>
__global__ void __launch_bounds__(256)
    moe_combine_grad_kernel(const void *__restrict__ dOut, const void *__restrict__ Y,
                            const int32_t *__restrict__ place, const float *__restrict__ weights,
                            int64_t T, int topk, RowMap map, void *__restrict__ dY,
                            float *__restrict__ dw) {
  __shared__ float part[4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = L == 256 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;  // a whole wave (L = 64, no barrier below) or workgroup
  const int first = L == 256 ? (int)threadIdx.x : lane;
  const int R = (int)(T * topk);
  for (int j0 = 0; j0 < topk; j0 += 4) {
    int row[4];
    bool on[4];
    float w[4], dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = j0 + j < topk ? place[t * topk + j0 + j] : R;
      row[j] = p < 0 ? ~p : p;
      on[j] = p >= 0 && p < R;
      w[j] = on[j] ? weights[t * topk + j0 + j] : 0.f;
    }
    for (int c = first; c < map.chunks; c += L) {
      const u32x4 g = ROWS::load(dOut, map, t, c);
      u32x4 y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (on[j]) y[j] = ROWS::load(Y, map, row[j], c);
      float gv[ROWS::n];
      ROWS::values(g, gv);
      const int dup = ROWS::shared(map, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (on[j]) {
          float v[ROWS::n], d[ROWS::n];
          ROWS::values(y[j], v);
#pragma unroll
          for (int i = 0; i < ROWS::n; ++i) {
            dot[j] = i < dup ? dot[j] : fmaf(gv[i], v[i], dot[j]);
            d[i] = w[j] * gv[i];
          }
          ROWS::store(dY, map, row[j], c, ROWS::chunk(d));
        } else if (row[j] < R) {
          ROWS::store(dY, map, row[j], c, u32x4{0u, 0u, 0u, 0u});
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) dot[j] = wave_sum(dot[j]);
    if constexpr (L == 256) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[wave][j] = dot[j];
      __syncthreads();
      if (threadIdx.x < 4 && j0 + (int)threadIdx.x < topk)
        dw[t * topk + j0 + threadIdx.x] = (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                                          (part[2][threadIdx.x] + part[3][threadIdx.x]);
      __syncthreads();
    } else if (lane == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j < topk) dw[t * topk + j0 + j] = dot[j];
    }
  }
}

// Shapes of the row kernels: T tokens, topk slots each, rows of H elements.  Slot
// and row numbers are 32-bit.
static int check_rows(int64_t T, int64_t topk, int64_t H) {
  if (T < 0 || topk < 1 || H < 1) return NF4_EINVAL;
  if (topk > NF4_MOE_MAX_E || H > (int64_t(1) << 20)) return NF4_ERANGE;
  // 256 threads a token fit one dispatch's 2^32 - 1 work-items
  if (T >= (int64_t(1) << 24) || T * topk > (int64_t(1) << 30)) return NF4_ERANGE;
  return NF4_OK;
}

// Threads per token: as many as the row has chunks, up to a workgroup.
static RowMap row_map(int64_t H, int esize, int v) {
  RowMap m{0, (int)((H * esize + v - 1) / v), (int)(H * esize)};
  while (m.shift < 8 && (1 << m.shift) < m.chunks) ++m.shift;
  return m;
}

static dim3 row_grid(int64_t T, RowMap m) { return dim3((unsigned)(((T << m.shift) + 255) >> 8)); }

// Calls f with the Rows type for this call and its map.
template <typename T, typename F>
static void with_rows_of(int64_t H, int64_t rows, bool aligned16, F f) {
  constexpr int es = (int)sizeof(T);
  if (H * es < 16)
    f(Rows<T, es, true, false>(), row_map(H, es, es));
  else if (!aligned16 || H * es % 16 != 0)
    f(Rows<T, 16, false, false>(), row_map(H, es, 16));
  else if (rows * H * es < (int64_t(32) << 20))  // 8 L2 caches of 4 MiB
    f(Rows<T, 16, true, false>(), row_map(H, es, 16));
  else
    f(Rows<T, 16, true, true>(), row_map(H, es, 16));
}
template <typename F>
static void with_rows(int dtype, int64_t H, int64_t rows, bool aligned16, F f) {
  if (dtype == NF4_F32)
    with_rows_of<uint32_t>(H, rows, aligned16, f);
  else
    with_rows_of<uint16_t>(H, rows, aligned16, f);
}

}  // namespace nf4

extern "C" {

int nf4_moe_sort(const int64_t *experts, int64_t T, int64_t topk, int64_t E, int32_t *offsets,
                 int32_t *order, int32_t *place, int32_t *dev_status, void *stream) {
  if (T < 0 || topk < 1 || E < 1 || !offsets || (T > 0 && (!experts || !order || !place)))
    return NF4_EINVAL;
  if (E > NF4_MOE_MAX_E) return NF4_ERANGE;
  if (int r = nf4::check_rows(T, topk, 1)) return r;
  if (!nf4::aligned_to(experts, 8) || !nf4::aligned_to(offsets, 4) ||
      !nf4::aligned_to(order, 4) || !nf4::aligned_to(place, 4) || !nf4::aligned_to(dev_status, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  hipStream_t s = (hipStream_t)stream;
  if (dev_status) {
    hipLaunchKernelGGL(nf4::moe_clear_status_kernel, dim3(1), dim3(1), 0, s, dev_status);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
  }
  const int64_t R = T * topk;
  constexpr int64_t kWave = 64 * nf4::kSortGroups;
  if (R < 4 * kWave && E < 256) {
    nf4::launch_scatter<4, true>(1, experts, R, (int)E, offsets, order, place, dev_status, s);
  } else if (R < 16 * kWave) {
    nf4::launch_scatter<16, true>(1, experts, R, (int)E, offsets, order, place, dev_status, s);
  } else {
    const unsigned chunks = (unsigned)(R / nf4::kSortChunk);
    hipLaunchKernelGGL(nf4::moe_count_kernel, dim3(chunks), dim3(64 * nf4::kChunkWaves), 0, s,
                       experts, R, (int)E, place, dev_status);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
    int shift = 6;
    while ((1 << shift) <= E) ++shift;
    hipLaunchKernelGGL(nf4::moe_scan_kernel, dim3(1), dim3(nf4::kScanThreads), 0, s, (int)chunks,
                       (int)E, shift, place, offsets);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
    nf4::launch_scatter<nf4::kChunkWaves, false>(chunks, experts, R, (int)E, offsets, order, place,
                                                 dev_status, s);
  }
  return nf4::launch_status(hipGetLastError());
}

int nf4_moe_gather(const void *X, int dtype, const int32_t *place, int64_t T, int64_t topk,
                   int64_t H, void *out, void *stream) {
  if (!nf4::known_dtype(dtype) || (T > 0 && (!X || !place || !out))) return NF4_EINVAL;
  if (int r = nf4::check_rows(T, topk, H)) return r;
  const int es = dtype == NF4_F32 ? 4 : 2;
  if (!nf4::aligned_to(X, es) || !nf4::aligned_to(out, es) || !nf4::aligned_to(place, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  if (T == 0) return NF4_OK;
  hipStream_t s = (hipStream_t)stream;
  nf4::with_rows(dtype, H, T * topk, nf4::aligned_to(X, 16) && nf4::aligned_to(out, 16),
                 [&](auto rows, nf4::RowMap m) {
                   hipLaunchKernelGGL(nf4::moe_gather_kernel<decltype(rows)>, nf4::row_grid(T, m),
                                      dim3(256), 0, s, X, place, T, (int)topk, m, out);
                 });
  return nf4::launch_status(hipGetLastError());
}

int nf4_moe_combine(const void *Y, int dtype, const int32_t *place, const float *weights,
                    int64_t T, int64_t topk, int64_t H, void *out, void *stream) {
  if (!nf4::known_dtype(dtype) || (T > 0 && (!Y || !place || !out))) return NF4_EINVAL;
  if (int r = nf4::check_rows(T, topk, H)) return r;
  const int es = dtype == NF4_F32 ? 4 : 2;
  if (!nf4::aligned_to(Y, es) || !nf4::aligned_to(out, es) || !nf4::aligned_to(place, 4) ||
      !nf4::aligned_to(weights, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  if (T == 0) return NF4_OK;
  hipStream_t s = (hipStream_t)stream;
  nf4::with_rows(dtype, H, T * topk, nf4::aligned_to(Y, 16) && nf4::aligned_to(out, 16),
                 [&](auto rows, nf4::RowMap m) {
                   if (weights)
                     hipLaunchKernelGGL((nf4::moe_combine_kernel<decltype(rows), true>),
                                        nf4::row_grid(T, m), dim3(256), 0, s, Y, place, weights, T,
                                        (int)topk, m, out);
                   else
                     hipLaunchKernelGGL((nf4::moe_combine_kernel<decltype(rows), false>),
                                        nf4::row_grid(T, m), dim3(256), 0, s, Y, place, weights, T,
                                        (int)topk, m, out);
                 });
  return nf4::launch_status(hipGetLastError());
}

int nf4_moe_combine_grad(const void *dOut, const void *Y, int dtype, const int32_t *place,
                         const float *weights, int64_t T, int64_t topk, int64_t H, void *dY,
                         float *dweights, void *stream) {
  if (!nf4::known_dtype(dtype) || (T > 0 && (!dOut || !Y || !place || !weights || !dY || !dweights)))
    return NF4_EINVAL;
  if (int r = nf4::check_rows(T, topk, H)) return r;
  const int es = dtype == NF4_F32 ? 4 : 2;
  if (!nf4::aligned_to(dOut, es) || !nf4::aligned_to(Y, es) || !nf4::aligned_to(dY, es) ||
      !nf4::aligned_to(place, 4) || !nf4::aligned_to(weights, 4) || !nf4::aligned_to(dweights, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  if (T == 0) return NF4_OK;
  hipStream_t s = (hipStream_t)stream;
  const bool aligned16 = nf4::aligned_to(dOut, 16) && nf4::aligned_to(Y, 16) && nf4::aligned_to(dY, 16);
  nf4::with_rows(dtype, H, T * topk, aligned16, [&](auto rows, nf4::RowMap m) {
    if (m.chunks >= 256)
      hipLaunchKernelGGL((nf4::moe_combine_grad_kernel<decltype(rows), 256>), dim3((unsigned)T),
                         dim3(256), 0, s, dOut, Y, place, weights, T, (int)topk, m, dY, dweights);
    else
      hipLaunchKernelGGL((nf4::moe_combine_grad_kernel<decltype(rows), 64>),
                         dim3((unsigned)((T + 3) / 4)), dim3(256), 0, s, dOut, Y, place, weights, T,
                         (int)topk, m, dY, dweights);
  });
  return nf4::launch_status(hipGetLastError());
}

}  // extern "C"
