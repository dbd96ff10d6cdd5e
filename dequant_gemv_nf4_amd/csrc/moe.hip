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
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxE = NF4_MOE_MAX_E;
// Slots one workgroup sorts.  At least kSortMaxE + 1, so that a chunk's counts
// fit the part of `place` that belongs to the chunk.
constexpr int kSortChunk = 4096;
static_assert(kSortMaxE < kSortThreads && kSortMaxE < kSortChunk, "one thread per key");

__device__ __forceinline__ int sort_key(const int64_t *experts, int64_t f, int E, int *bad) {
  const int64_t id = experts[f];
  const bool in = id >= 0 && id < E;
  if (!in && id != -1) *bad = 1;
  return in ? (int)id : E;
}

// Counts of this wave's slots [f0, f1) per key, into cnt[0 .. E].
__device__ __forceinline__ int count_keys(const int64_t *experts, int64_t f0, int64_t f1, int E,
                                          int *cnt, int lane) {
  int bad = 0;
  for (int64_t f = f0 + lane; f < f1; f += 64) atomicAdd(&cnt[sort_key(experts, f, E, &bad)], 1);
  return bad;
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

// Exclusive prefix over the threads of the workgroup (kSortThreads).
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
  for (int w = 0; w < kSortWaves; ++w) base += w < wave ? wsum[w] : 0;
  return base + s - v;
}

// The chunk of workgroup b: kSortChunk slots, the last one with what is left.
__device__ __forceinline__ void sort_chunk(int64_t R, int64_t *f0, int64_t *f1) {
  *f0 = (int64_t)blockIdx.x * kSortChunk;
  *f1 = blockIdx.x + 1 == gridDim.x ? R : *f0 + kSortChunk;
}

// Each wave's slots lie together, in order, so ranks follow the slot order.
__device__ __forceinline__ void wave_range(int64_t f0, int64_t f1, int64_t *a, int64_t *b) {
  const int64_t groups = (f1 - f0 + 63) / 64;
  const int64_t per = (groups + kSortWaves - 1) / kSortWaves * 64;
  const int64_t lo = f0 + (threadIdx.x >> 6) * per;
  *a = lo < f1 ? lo : f1;
  *b = lo + per < f1 ? lo + per : f1;
}

__global__ void __launch_bounds__(kSortThreads)
    moe_count_kernel(const int64_t *__restrict__ experts, int64_t R, int E,
                     int32_t *__restrict__ place, int32_t *status) {
  __shared__ int cnt[kSortMaxE + 1];
  int64_t f0, f1, a, b;
  sort_chunk(R, &f0, &f1);
  for (int e = threadIdx.x; e <= E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  wave_range(f0, f1, &a, &b);
  const int bad = count_keys(experts, a, b, E, cnt, threadIdx.x & 63);
  if (bad && status) atomicOr(status, NF4_MOE_BAD_ID);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads) place[f0 + e] = cnt[e];
}

// One workgroup: the chunks' counts become each chunk's first row per key.
__global__ void __launch_bounds__(kSortThreads)
    moe_scan_kernel(int nchunks, int E, int32_t *__restrict__ place, int32_t *__restrict__ offsets) {
  __shared__ int wsum[kSortWaves];
  // thread e has key e; key E (no expert) follows every expert's rows
  const int e = threadIdx.x;
  int n = 0;
  if (e <= E)
    for (int c = 0; c < nchunks; ++c) n += place[(int64_t)c * kSortChunk + e];
  int row = block_exclusive(n, wsum);
  if (e <= E) offsets[e] = row;
  if (e > E) return;
  for (int c0 = 0; c0 < nchunks; c0 += 8) {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = c0 + i < nchunks ? place[(int64_t)(c0 + i) * kSortChunk + e] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c0 + i < nchunks) place[(int64_t)(c0 + i) * kSortChunk + e] = row;
      row += v[i];
    }
  }
}

// Ranks and writes a chunk's slots.  SINGLE: the chunk is everything, and this
// kernel counts and scans by itself (one launch for up to 2 * kSortChunk - 1 slots).
template <bool SINGLE>
__global__ void __launch_bounds__(kSortThreads)
    moe_scatter_kernel(const int64_t *__restrict__ experts, int64_t R, int E, int bits,
                       int32_t *__restrict__ offsets, int32_t *__restrict__ order,
                       int32_t *__restrict__ place, int32_t *status) {
  extern __shared__ int cnt[];  // [kSortWaves][E + 1], then wave sums
  int *wsum = cnt + kSortWaves * (E + 1);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t f0, f1, a, b;
  sort_chunk(R, &f0, &f1);
  for (int i = threadIdx.x; i < kSortWaves * (E + 1); i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  wave_range(f0, f1, &a, &b);
  int *mine = cnt + wave * (E + 1);
  const int bad = count_keys(experts, a, b, E, mine, lane);
  if (SINGLE && bad && status) atomicOr(status, NF4_MOE_BAD_ID);
  __syncthreads();
  // first row of each key in this chunk, then of each wave
  const int e = threadIdx.x;
  int base = 0;
  if constexpr (SINGLE) {
    int n = 0;
    if (e <= E)
      for (int w = 0; w < kSortWaves; ++w) n += cnt[w * (E + 1) + e];
    base = block_exclusive(n, wsum);
    if (e <= E) {
      offsets[e] = base;
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = cnt[w * (E + 1) + e];
        cnt[w * (E + 1) + e] = base;
        base += v;
      }
    }
  } else {
    for (int k = e; k <= E; k += kSortThreads) {
      base = place[f0 + k];
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = cnt[w * (E + 1) + k];
        cnt[w * (E + 1) + k] = base;
        base += v;
      }
    }
  }
  __syncthreads();  // also: this chunk's part of `place` is read before it is written
  const uint64_t below = lane ? ~uint64_t(0) >> (64 - lane) : 0;
  for (int64_t g = a; g < b; g += 64) {
    const int64_t f = g + lane;
    const bool active = f < b;
    int ignored = 0;
    const int key = active ? sort_key(experts, f, E, &ignored) : 0;
    const uint64_t peers = same_key(key, active, bits);
    if (active) {
      const int row = mine[key] + __popcll(peers & below);
      const bool kept = key < E;
      place[f] = kept ? row : ~row;
      order[row] = kept ? (int)f : ~(int)f;
    }
    // every lane of the wave has read its count before a leader adds to it, and
    // the next group reads what the leaders left
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (active && (peers & below) == 0) mine[key] += __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

__global__ void moe_clear_status_kernel(int32_t *status) { *status = 0; }

// ------------------------------------------------------- rows by place ----
// A row is cut into chunks of V bytes; 2^shift threads share a token, each taking
// every 2^shift-th chunk.  V is 16 where rows and pointers allow it, else the
// element.
struct RowMap {
  int shift;   // log2 of the threads per token
  int chunks;  // chunks per row
};

template <int V>
struct Chunk;
template <>
struct Chunk<16> {
  typedef u32x4 type;
};
template <>
struct Chunk<4> {
  typedef uint32_t type;
};
template <>
struct Chunk<2> {
  typedef uint16_t type;
};

// fp32 values of a chunk and back (bf16: one rounding to nearest even)
template <typename T, int V>
struct Conv {
  static constexpr int n = V / (int)sizeof(T);
  typedef typename Chunk<V>::type raw;
  static __device__ __forceinline__ void load(const raw &c, float *v) {
    if constexpr (V == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          v[i] = __uint_as_float(c[i]);
        } else {
          v[2 * i] = bf16_lo(c[i]);
          v[2 * i + 1] = bf16_hi(c[i]);
        }
      }
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(c);
    } else {
      v[0] = __uint_as_float((uint32_t)c << 16);
    }
  }
  static __device__ __forceinline__ uint32_t bits(float f) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ raw store(const float *v) {
    raw c;
    if constexpr (V == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
          c[i] = __float_as_uint(v[i]);
        else
          c[i] = bits(v[2 * i]) | (bits(v[2 * i + 1]) << 16);
      }
    } else if constexpr (sizeof(T) == 4) {
      c = __float_as_uint(v[0]);
    } else {
      c = (uint16_t)bits(v[0]);
    }
    return c;
  }
};

// place[f] as a row, -1 where the slot has no expert or the entry is no row
__device__ __forceinline__ int kept_row(int p, int R) { return p >= 0 && p < R ? p : -1; }

// P[row] = X[t] for every slot of token t, zeros in the rows without an expert.
template <int V>
__global__ void __launch_bounds__(256)
    moe_gather_kernel(const typename Chunk<V>::type *__restrict__ X,
                      const int32_t *__restrict__ place, int64_t T, int topk, RowMap map,
                      typename Chunk<V>::type *__restrict__ out) {
  typedef typename Chunk<V>::type raw;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = g >> map.shift;
  if (t >= T) return;
  const int R = (int)(T * topk);
  for (int c = (int)(g & ((1 << map.shift) - 1)); c < map.chunks; c += 1 << map.shift) {
    const raw v = X[t * map.chunks + c];
    for (int j = 0; j < topk; ++j) {
      const int p = place[t * topk + j];
      const int row = p < 0 ? ~p : p;
      if (row < R) out[(int64_t)row * map.chunks + c] = p < 0 ? raw{} : v;
    }
  }
}

// out[t] = sum_j w[t,j] Y[place[t,j]] in fp32, j in order (WEIGHTED false: w = 1).
template <typename T, int V, bool WEIGHTED>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const typename Chunk<V>::type *__restrict__ Y,
                       const int32_t *__restrict__ place, const float *__restrict__ weights,
                       int64_t T_, int topk, RowMap map, typename Chunk<V>::type *__restrict__ out) {
  typedef Conv<T, V> C;
  typedef typename C::raw raw;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = g >> map.shift;
  if (t >= T_) return;
  const int R = (int)(T_ * topk);
  for (int c = (int)(g & ((1 << map.shift) - 1)); c < map.chunks; c += 1 << map.shift) {
    float acc[C::n] = {};
    for (int j0 = 0; j0 < topk; j0 += 4) {
      raw y[4];
      float w[4];
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = j0 + j < topk ? kept_row(place[t * topk + j0 + j], R) : -1;
        on[j] = row >= 0;
        w[j] = 1.0f;
        if (on[j]) {
          y[j] = Y[(int64_t)row * map.chunks + c];
          if constexpr (WEIGHTED) w[j] = weights[t * topk + j0 + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!on[j]) continue;
        float v[C::n];
        C::load(y[j], v);
#pragma unroll
        for (int i = 0; i < C::n; ++i) acc[i] = WEIGHTED ? fmaf(w[j], v[i], acc[i]) : acc[i] + v[i];
      }
    }
    out[t * map.chunks + c] = C::store(acc);
  }
}

// dY[place[t,j]] = w[t,j] dOut[t]; dw[t,j] = <dOut[t], Y[place[t,j]]> in fp32.
// L threads per token (64: four tokens a workgroup; 256: one).  Slots are taken
// four at a time; each thread's partial sums are added over the wave, then over
// the waves in order.
template <typename T, int V, int L>
__global__ void __launch_bounds__(256)
    moe_combine_grad_kernel(const typename Chunk<V>::type *__restrict__ dOut,
                            const typename Chunk<V>::type *__restrict__ Y,
                            const int32_t *__restrict__ place, const float *__restrict__ weights,
                            int64_t T_, int topk, int chunks,
                            typename Chunk<V>::type *__restrict__ dY, float *__restrict__ dw) {
  typedef Conv<T, V> C;
  typedef typename C::raw raw;
  __shared__ float part[4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = L == 256 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (t >= T_) return;  // a whole wave (L = 64, no barrier below) or workgroup
  const int first = L == 256 ? (int)threadIdx.x : lane;
  const int R = (int)(T_ * topk);
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
    for (int c = first; c < chunks; c += L) {
      const raw g = dOut[t * chunks + c];
      raw y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (on[j]) y[j] = Y[(int64_t)row[j] * chunks + c];
      float gv[C::n];
      C::load(g, gv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (on[j]) {
          float v[C::n], d[C::n];
          C::load(y[j], v);
#pragma unroll
          for (int i = 0; i < C::n; ++i) {
            dot[j] = fmaf(gv[i], v[i], dot[j]);
            d[i] = w[j] * gv[i];
          }
          dY[(int64_t)row[j] * chunks + c] = C::store(d);
        } else if (row[j] < R) {
          dY[(int64_t)row[j] * chunks + c] = raw{};
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

static int chunk_bytes(int64_t H, int esize, const void *a, const void *b, const void *c) {
  if (H * esize % 16 == 0 && aligned_to(a, 16) && aligned_to(b, 16) && aligned_to(c, 16)) return 16;
  return esize;
}

// Threads per token: as many as the row has chunks, up to a workgroup.
static RowMap row_map(int64_t chunks) {
  RowMap m{0, (int)chunks};
  while (m.shift < 8 && (1 << m.shift) < chunks) ++m.shift;
  return m;
}

static dim3 row_grid(int64_t T, RowMap m) { return dim3((unsigned)(((T << m.shift) + 255) >> 8)); }

template <int V>
static void launch_gather(const void *X, const int32_t *place, int64_t T, int64_t topk,
                          int64_t chunks, void *out, hipStream_t s) {
  typedef typename Chunk<V>::type raw;
  const RowMap m = row_map(chunks);
  hipLaunchKernelGGL(moe_gather_kernel<V>, row_grid(T, m), dim3(256), 0, s, (const raw *)X, place,
                     T, (int)topk, m, (raw *)out);
}

template <typename T, int V>
static void launch_combine(const void *Y, const int32_t *place, const float *weights, int64_t T_,
                           int64_t topk, int64_t chunks, void *out, hipStream_t s) {
  typedef typename Chunk<V>::type raw;
  const RowMap m = row_map(chunks);
  if (weights)
    hipLaunchKernelGGL((moe_combine_kernel<T, V, true>), row_grid(T_, m), dim3(256), 0, s,
                       (const raw *)Y, place, weights, T_, (int)topk, m, (raw *)out);
  else
    hipLaunchKernelGGL((moe_combine_kernel<T, V, false>), row_grid(T_, m), dim3(256), 0, s,
                       (const raw *)Y, place, weights, T_, (int)topk, m, (raw *)out);
}

template <typename T, int V>
static void launch_combine_grad(const void *dOut, const void *Y, const int32_t *place,
                                const float *weights, int64_t T_, int64_t topk, int64_t chunks,
                                void *dY, float *dw, hipStream_t s) {
  typedef typename Chunk<V>::type raw;
  if (chunks >= 256)
    hipLaunchKernelGGL((moe_combine_grad_kernel<T, V, 256>), dim3((unsigned)T_), dim3(256), 0, s,
                       (const raw *)dOut, (const raw *)Y, place, weights, T_, (int)topk,
                       (int)chunks, (raw *)dY, dw);
  else
    hipLaunchKernelGGL((moe_combine_grad_kernel<T, V, 64>), dim3((unsigned)((T_ + 3) / 4)),
                       dim3(256), 0, s, (const raw *)dOut, (const raw *)Y, place, weights, T_,
                       (int)topk, (int)chunks, (raw *)dY, dw);
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
  int bits = 1;
  while ((1 << bits) <= E) ++bits;
  const size_t lds = (size_t)(nf4::kSortWaves * (E + 1) + nf4::kSortWaves) * sizeof(int);
  const int64_t chunks = R / nf4::kSortChunk;
  const dim3 wg(nf4::kSortThreads);
  if (chunks <= 1) {
    hipLaunchKernelGGL(nf4::moe_scatter_kernel<true>, dim3(1), wg, lds, s, experts, R, (int)E,
                       bits, offsets, order, place, dev_status);
  } else {
    hipLaunchKernelGGL(nf4::moe_count_kernel, dim3((unsigned)chunks), wg, 0, s, experts, R, (int)E,
                       place, dev_status);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
    hipLaunchKernelGGL(nf4::moe_scan_kernel, dim3(1), wg, 0, s, (int)chunks, (int)E, place,
                       offsets);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
    hipLaunchKernelGGL(nf4::moe_scatter_kernel<false>, dim3((unsigned)chunks), wg, lds, s, experts,
                       R, (int)E, bits, offsets, order, place, dev_status);
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
  const int v = nf4::chunk_bytes(H, es, X, out, out);
  const int64_t chunks = H * es / v;
  if (v == 16)
    nf4::launch_gather<16>(X, place, T, topk, chunks, out, s);
  else if (v == 4)
    nf4::launch_gather<4>(X, place, T, topk, chunks, out, s);
  else
    nf4::launch_gather<2>(X, place, T, topk, chunks, out, s);
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
  const int v = nf4::chunk_bytes(H, es, Y, out, out);
  const int64_t chunks = H * es / v;
  if (v == 16 && es == 4)
    nf4::launch_combine<float, 16>(Y, place, weights, T, topk, chunks, out, s);
  else if (v == 16)
    nf4::launch_combine<uint16_t, 16>(Y, place, weights, T, topk, chunks, out, s);
  else if (es == 4)
    nf4::launch_combine<float, 4>(Y, place, weights, T, topk, chunks, out, s);
  else
    nf4::launch_combine<uint16_t, 2>(Y, place, weights, T, topk, chunks, out, s);
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
  const int v = nf4::chunk_bytes(H, es, dOut, Y, dY);
  const int64_t chunks = H * es / v;
  if (v == 16 && es == 4)
    nf4::launch_combine_grad<float, 16>(dOut, Y, place, weights, T, topk, chunks, dY, dweights, s);
  else if (v == 16)
    nf4::launch_combine_grad<uint16_t, 16>(dOut, Y, place, weights, T, topk, chunks, dY, dweights, s);
  else if (es == 4)
    nf4::launch_combine_grad<float, 4>(dOut, Y, place, weights, T, topk, chunks, dY, dweights, s);
  else
    nf4::launch_combine_grad<uint16_t, 2>(dOut, Y, place, weights, T, topk, chunks, dY, dweights, s);
  return nf4::launch_status(hipGetLastError());
}

}  // extern "C"
