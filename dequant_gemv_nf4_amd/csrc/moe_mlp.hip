// moe_mlp.hip -- a whole layer of experts for a few tokens (gfx950):
//   out[t] = sum_j weights[t][j] W2[e] act(W1[e] X[t]) (+ residual[t]),  e = experts[t][j],
// W1 [E][N1][H] and W2 [E][H][I] packed MXFP4; gated, N1 = 2 I.
//
// The tokens are not sorted beforehand: every workgroup makes for each expert the mask of
// its tokens (at most 64) in LDS.  A pair (token, expert) is one row, whose weight is the
// sum over the token's slots with that expert; rows are numbered by expert, then token.
// The first kernel writes act(W1 x) times the row's weight, in bf16 (one rounding, as
// between two layers); the second one's sums over all its rows are then the output.
#include "mx_act.h"
#include "mx_product.h"

namespace nf4 {
namespace mx {

constexpr int kTokens = NF4_MOE_MLP_MAX_T;
static_assert(kTokens == 64, "a token is a bit of a mask and a lane");

struct Routing {
  const int64_t *experts;  // [T][topk]
  const float *weights;    // [T][topk]
  int T, topk, E;
};

// What every workgroup makes of the routing.
struct Masks {
  uint32_t of[2 * NF4_MOE_MAX_E];  // tokens of each expert
};
__device__ __forceinline__ uint64_t mask_of(const Masks &m, int e) {
  return (uint64_t)m.of[2 * e + 1] << 32 | m.of[2 * e];
}
__device__ __forceinline__ void make_masks(const Routing &r, Masks &m) {
  for (int i = threadIdx.x; i < 2 * r.E; i += blockDim.x) m.of[i] = 0u;
  __syncthreads();
  const int slots = r.T * r.topk;
  for (int f = threadIdx.x; f < slots; f += blockDim.x) {
    const int64_t e = r.experts[f];
    const int t = f / r.topk;
    if (e >= 0 && e < r.E) atomicOr(&m.of[2 * (int)e + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
}

// Inclusive prefix over the wave.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// The slot-th tile of at most bm rows, and in `tokens` the tokens of its rows (T for
// none).  Every wave finds it by itself; tiles and rows (at most 2^15 each) are counted in
// the halves of one word.
__device__ __forceinline__ RowTile find_rows(const Routing &r, const Masks &masks, int slot, int bm, int *tokens) {
  const int lane = threadIdx.x & 63;
  RowTile t{0, 0, 0};
  uint32_t before = 0;
  for (int base = 0; base < r.E; base += 64) {
    const int e = base + lane;
    const int rows = e < r.E ? __popcll(mask_of(masks, e)) : 0;
    const uint32_t own = (uint32_t)((rows + bm - 1) / bm) << 16 | (uint32_t)rows;
    const uint32_t incl = before + wave_prefix(own);
    const uint64_t hit = __ballot((int)(incl >> 16) > slot && rows > 0);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)(incl - own), l);
      const int n = __builtin_amdgcn_readlane(rows, l), part = slot - (int)(first >> 16);
      t.e = base + l;
      t.row0 = (int)(first & 0xffffu) + part * bm;
      t.rows = min(bm, n - part * bm);
      const uint64_t mask = mask_of(masks, t.e);
      const int rank = __popcll(mask & ((uint64_t(1) << lane) - 1)) - part * bm;
      if ((int)threadIdx.x < 64) {
        if (lane >= t.rows && lane < bm) tokens[lane] = r.T;
        if ((mask >> lane & 1) && rank >= 0 && rank < bm) tokens[rank] = lane;
      }
      break;
    }
    before = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  __syncthreads();
  return t;
}

// The weight of a token's row of expert e.
__device__ __forceinline__ float row_weight(const Routing &r, int token, int e) {
  float w = 0.f;
  for (int j = 0; j < r.topk; ++j)
    if (r.experts[token * r.topk + j] == e) w += r.weights[token * r.topk + j];
  return w;
}

struct TileState {
  Masks masks;
  int tokens[kTokens];
  float weight[kTokens];
};
__device__ __forceinline__ TileState &tile_state() {
  __shared__ TileState s;
  return s;
}

// Rows of X by the tokens of a tile.
struct TokenRows {
  Routing r;
  __device__ __forceinline__ RowTile find(const Args &, int slot, int bm) const {
    TileState &s = tile_state();
    make_masks(r, s.masks);
    return find_rows(r, s.masks, slot, bm, s.tokens);
  }
  __device__ __forceinline__ int64_t base(const RowTile &) const { return 0; }
  __device__ __forceinline__ int whole(const Args &, const RowTile &) const { return r.T; }
  __device__ __forceinline__ int place(const RowTile &t, int m) const {
    return m < t.rows ? tile_state().tokens[m] : r.T;  // T: outside the buffer
  }
};

// Rows as the first kernel wrote them.
struct PairRows {
  Routing r;
  __device__ __forceinline__ RowTile find(const Args &, int slot, int bm) const {
    TileState &s = tile_state();
    make_masks(r, s.masks);
    return find_rows(r, s.masks, slot, bm, s.tokens);
  }
  __device__ __forceinline__ int64_t base(const RowTile &t) const { return t.row0; }
  __device__ __forceinline__ int whole(const Args &, const RowTile &t) const { return t.rows; }
  __device__ __forceinline__ int place(const RowTile &, int m) const { return m; }
};

// act(sums) times the row's weight as bf16 rows [pair][I].
template <bool PAIRS>
struct ActRows {
  static constexpr bool kPairs = PAIRS, kPlain = false;
  Routing r;
  int act;

  __device__ __forceinline__ void weights_of(const RowTile &t) const {
    TileState &s = tile_state();
    if ((int)threadIdx.x < t.rows) s.weight[threadIdx.x] = row_weight(r, s.tokens[threadIdx.x], t.e);
    __syncthreads();
  }
  __device__ __forceinline__ void put(const Args &p, const RowTile &t, int m, int n, f32x4_t z, f32x4_t zu) const {
    const int cols = PAIRS ? p.N >> 1 : p.N;
    f32x4_t y = act_values(act, z);
    if constexpr (PAIRS) y *= zu;
    y *= tile_state().weight[m];
    store4<uint16_t>(reinterpret_cast<uint16_t *>(p.Y) + (int64_t)(t.row0 + m) * cols, n, cols, y, true);
  }
  template <int MF, int NF, int WV, int KG, typename OUT, int BYTES, class ROWS>
  __device__ __forceinline__ void tile_out(const Args &p, const ROWS &, const RowTile &t, int n0, int wave,
                                           int kg, const f32x4_t (&acc)[NF][MF], uint8_t *lds) const {
    weights_of(t);
    typedef TileRows<MF, NF, WV, KG, BYTES> T;
    T::each(wave, kg, acc, lds, [&](const float *z, int m0, int rows) __attribute__((always_inline)) {
      constexpr int W = PAIRS ? 8 : 4, quads = T::kCols / W;
      const int n = min(rows, t.rows - m0) * quads;
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += 64 * WV * KG) {
        const int m = i / quads, c = i % quads * W;
        if (n0 + c >= p.N) continue;
        const float *s = z + m * T::kPitch + c;
        const f32x4_t a = *reinterpret_cast<const f32x4_t *>(s);
        if constexpr (PAIRS) {
          const f32x4_t b = *reinterpret_cast<const f32x4_t *>(s + 4);
          put(p, t, m0 + m, (n0 + c) >> 1, f32x4_t{a[0], a[2], b[0], b[2]}, f32x4_t{a[1], a[3], b[1], b[3]});
        } else {
          put(p, t, m0 + m, n0 + c, a, a);
        }
      }
    });
  }
};

// ------------------------------------------------------- up to 16 rows a tile ----
// A wave streams 16 weight rows at a time over its range of kRange k, straight from memory
// into registers: a lane the 16 bytes of block l / 16 of row l % 16, so a load takes 64
// bytes of each row and the four of a range whole lines.  The range of the tile's rows of X
// stays in registers (as the other operand's fragments, up to 16 rows at the cost of one),
// and the range's products of 16 weight rows are 16 matrix instructions.
constexpr int kRange = 512;

template <bool SVEC, bool PAIRS>
struct RangeLoads {
  u32x4_t cw[4];
  u32x4_t sw;
  // 16 weight rows from row r0 of the buffers on; k0: the range's first k
  __device__ __forceinline__ void load(const uint8_t *cbase, const uint8_t *sbase, int wrows, int r0, int N, int K,
                                       int k0) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int kc = K >> 1, kb = K >> 5;
    const __amdgpu_buffer_rsrc_t crs = buffer(cbase, (int64_t)wrows * kc);
    const int row = weight_row<PAIRS>(r0 + l16, N);
    const int b0 = (k0 >> 5) + q;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      cw[s] = __builtin_amdgcn_raw_buffer_load_b128(crs, b0 + 4 * s < kb ? row * kc + (b0 + 4 * s) * 16 : kOutside,
                                                    0, kLoadStream);
    const __amdgpu_buffer_rsrc_t srs = buffer(sbase, (int64_t)wrows * kb);
    if constexpr (SVEC) {
      sw = __builtin_amdgcn_raw_buffer_load_b128(srs, row * kb + (k0 >> 5), 0, 0);
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        sw[s] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(srs, b0 + 4 * s < kb ? row * kb + b0 + 4 * s : kOutside,
                                                              0, 0);
    }
  }
  // scale of step s; past K it is that of another row, perhaps NaN, and not taken
  __device__ __forceinline__ float scale(int s, int K, int k0) const {
    const int q = (threadIdx.x & 63) >> 4;
    const uint32_t byte = SVEC ? (sw[s] >> (8 * q)) & 0xffu : sw[s];
    return scale_of((k0 >> 5) + 4 * s + q < (K >> 5) ? byte : 0u);
  }
};

// The range of up to 16 rows of X: row offsets are the lane's (l16).
__device__ __forceinline__ void load_range(u32x4_t (&x)[4][4], __amdgpu_buffer_rsrc_t xrs, int row_bytes, int K, int k0) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = k0 + 128 * s + 32 * q;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[s][j] = __builtin_amdgcn_raw_buffer_load_b128(xrs, k < K ? row_bytes + k * 2 + j * 16 : kOutside, 0, 0);
  }
}

template <bool SVEC, bool PAIRS>
__device__ __forceinline__ f32x4_t multiply(const RangeLoads<SVEC, PAIRS> &w, const u32x4_t (&x)[4][4], f32x4_t acc,
                                            int K, int k0) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (k0 + 128 * s < K) {  // uniform
      const float sc = w.scale(s, K, k0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = mfma16(decode8(w.cw[s][j], sc), x[s][j], acc);
    }
  }
  return acc;
}

// First product: a workgroup owns 16 G weight rows (columns) of a tile; its waves share out
// the ranges of K.
template <int G, bool SVEC, bool PAIRS>
__global__ void __launch_bounds__(512)
    moe_up_kernel(Args p, int blocks, Routing r, int act) {
  extern __shared__ float part[];  // [wave][row][16 G]
  const int slot = blockIdx.x / blocks, n0 = (blockIdx.x - slot * blocks) * 16 * G;
  const TokenRows rows{r};
  const RowTile t = rows.find(p, slot, 16);
  if (t.rows <= 0) return;
  TileState &st = tile_state();
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int cols = min(16 * G, p.N - n0);
  const int kb = p.K >> 5, kc = p.K >> 1;
  const int64_t first = (int64_t)t.e * p.N + (PAIRS ? n0 >> 1 : n0);
  const int wrows = PAIRS ? (p.N + cols) >> 1 : cols;
  const uint8_t *const cbase = p.codes + first * kc, *const sbase = p.scales + first * kb;
  const __amdgpu_buffer_rsrc_t xrs = buffer(p.X, (int64_t)r.T * p.K * 2);
  const int xrow = (l16 < t.rows ? st.tokens[l16] : r.T) * p.K * 2;
  if ((int)threadIdx.x < t.rows) st.weight[threadIdx.x] = row_weight(r, st.tokens[threadIdx.x], t.e);
  f32x4_t acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * kRange; k0 < p.K; k0 += waves * kRange) {
    RangeLoads<SVEC, PAIRS> w[2];
    u32x4_t x[4][4];
    w[0].load(cbase, sbase, wrows, 0, p.N, p.K, k0);
    load_range(x, xrs, xrow, p.K, k0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g + 1 < G) w[(g + 1) & 1].load(cbase, sbase, wrows, (g + 1) * 16, p.N, p.K, k0);
      acc[g] = multiply(w[g & 1], x, acc[g], p.K, k0);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (l16 < t.rows) *reinterpret_cast<f32x4_t *>(part + (wave * 16 + l16) * (16 * G) + g * 16 + q * 4) = acc[g];
  __syncthreads();
  const ActRows<PAIRS> out{r, act};
  constexpr int W = PAIRS ? 8 : 4, quads = 16 * G / W;
  for (int i = threadIdx.x; i < t.rows * quads; i += blockDim.x) {
    const int m = i / quads, c = i % quads * W;
    if (n0 + c >= p.N) continue;
    f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = a;
    for (int k = 0; k < waves; ++k) {
      const float *s = part + (k * 16 + m) * (16 * G) + c;
      a += *reinterpret_cast<const f32x4_t *>(s);
      if constexpr (PAIRS) b += *reinterpret_cast<const f32x4_t *>(s + 4);
    }
    if constexpr (PAIRS)
      out.put(p, t, m, (n0 + c) >> 1, f32x4_t{a[0], a[2], b[0], b[2]}, f32x4_t{a[1], a[3], b[1], b[3]});
    else
      out.put(p, t, m, n0 + c, a, a);
  }
}

// Second product and the sum over a token's experts: a workgroup owns 16 columns of the
// output for all tokens; its waves share out the ranges of all experts' I and add, each
// for itself and in one order, into sums of its own in LDS.
struct ActiveExperts {
  Masks masks;
  uint16_t expert[NF4_MOE_MAX_E];
  uint16_t row0[NF4_MOE_MAX_E];
  int count;
};
template <bool SVEC, typename OUT>
__global__ void __launch_bounds__(512)
    moe_down_kernel(Args p, Routing r, const void *residual) {
  extern __shared__ float sums[];  // [wave][token][16]
  __shared__ ActiveExperts act;
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, cols = min(16, p.N - n0);
  for (int i = threadIdx.x; i < waves * r.T * 16; i += blockDim.x) sums[i] = 0.f;
  make_masks(r, act.masks);
  if (wave == 0) {
    uint32_t before = 0;
    for (int base = 0; base < r.E; base += 64) {
      const int e = base + lane;
      const int rows = e < r.E ? __popcll(mask_of(act.masks, e)) : 0;
      const uint32_t own = (uint32_t)(rows > 0) << 16 | (uint32_t)rows;
      const uint32_t incl = before + wave_prefix(own);
      if (rows > 0) {
        const uint32_t at = incl - own;
        act.expert[at >> 16] = (uint16_t)e;
        act.row0[at >> 16] = (uint16_t)at;
      }
      before = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    }
    if (lane == 0) act.count = (int)(before >> 16);
  }
  __syncthreads();
  const int kb = p.K >> 5, kc = p.K >> 1;
  const int ranges = (p.K + kRange - 1) / kRange, units = act.count * ranges;
  float *const own = sums + wave * r.T * 16;
  const auto start = [&](RangeLoads<SVEC, false> &w, int u) __attribute__((always_inline)) {
    const int i = u / ranges, k0 = (u - i * ranges) * kRange;
    const int64_t first = (int64_t)act.expert[u < units ? i : 0] * p.N + n0;
    w.load(p.codes + first * kc, p.scales + first * kb, u < units ? cols : 0, 0, p.N, p.K, k0);
  };
  RangeLoads<SVEC, false> w;
  if (units > 0) start(w, wave);
  for (int u = wave; u < units; u += waves) {
    const int i = u / ranges, k0 = (u - i * ranges) * kRange;
    const uint64_t mask = mask_of(act.masks, act.expert[i]);
    const int n = __popcll(mask), rank = __popcll(mask & ((uint64_t(1) << lane) - 1));
    RangeLoads<SVEC, false> now = w;
    start(w, u + waves);
    for (int m0 = 0; m0 < n; m0 += 16) {
      const int rows = min(16, n - m0);
      const __amdgpu_buffer_rsrc_t xrs = buffer(p.X + (int64_t)(act.row0[i] + m0) * p.K, (int64_t)rows * p.K * 2);
      u32x4_t x[4][4];
      load_range(x, xrs, l16 * p.K * 2, p.K, k0);
      // the token of row l16: lanes are tokens, and send theirs to their row
      const bool mine = (mask >> lane & 1) && rank >= m0 && rank < m0 + 16;
      const int token = __builtin_amdgcn_ds_permute(mine ? (rank - m0) * 4 : 63 * 4, lane);
      const int tok = __shfl(token, l16, 64);
      const f32x4_t v = multiply(now, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, p.K, k0);
      if (l16 < rows) {
#pragma unroll
        for (int c = 0; c < 4; ++c) own[tok * 16 + q * 4 + c] += v[c];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < r.T * 4; i += blockDim.x) {
    const int t = i >> 2, c = (i & 3) * 4;
    if (n0 + c >= p.N) continue;
    f32x4_t v = *reinterpret_cast<const f32x4_t *>(sums + t * 16 + c);
    for (int k = 1; k < waves; ++k) v += *reinterpret_cast<const f32x4_t *>(sums + (k * r.T + t) * 16 + c);
    const int64_t at = (int64_t)t * p.N;
    if (residual) {
      const OUT *s = reinterpret_cast<const OUT *>(residual) + at + n0 + c;
      if constexpr (sizeof(OUT) == 4) {
        v += *reinterpret_cast<const f32x4_t *>(s);
      } else {
        const u32x2_t w2 = *reinterpret_cast<const u32x2_t *>(s);
        v += f32x4_t{bf16_lo(w2[0]), bf16_hi(w2[0]), bf16_lo(w2[1]), bf16_hi(w2[1])};
      }
    }
    store4<OUT>(reinterpret_cast<OUT *>(p.Y) + at, n0 + c, p.N, v, true);
  }
}

// The rows' sum per token, in order of expert, where the second product left the rows.
template <typename OUT>
__global__ void __launch_bounds__(256)
    moe_rows_sum_kernel(const float *__restrict__ rows, Routing r, int N, const void *residual, OUT *__restrict__ out) {
  __shared__ Masks masks;
  __shared__ uint16_t row_of[NF4_MOE_MAX_E];
  __shared__ int count;
  const int t = blockIdx.y;
  make_masks(r, masks);
  if (threadIdx.x < 64) {  // the token's rows, by expert
    const int lane = threadIdx.x;
    uint32_t before = 0;
    for (int base = 0; base < r.E; base += 64) {
      const int e = base + lane;
      const uint64_t mask = e < r.E ? mask_of(masks, e) : 0;
      const bool mine = mask >> t & 1;
      const uint32_t own = (uint32_t)mine << 16 | (uint32_t)__popcll(mask);
      const uint32_t incl = before + wave_prefix(own);
      const uint32_t at = incl - own;
      if (mine) row_of[at >> 16] = (uint16_t)((at & 0xffffu) + __popcll(mask & ((uint64_t(1) << t) - 1)));
      before = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    }
    if (lane == 0) count = (int)(before >> 16);
  }
  __syncthreads();
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= N) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < count; ++i) v += *reinterpret_cast<const f32x4_t *>(rows + (int64_t)row_of[i] * N + n);
  const int64_t at = (int64_t)t * N;
  if (residual) {
    const OUT *s = reinterpret_cast<const OUT *>(residual) + at + n;
    if constexpr (sizeof(OUT) == 4) {
      v += *reinterpret_cast<const f32x4_t *>(s);
    } else {
      const u32x2_t w = *reinterpret_cast<const u32x2_t *>(s);
      v += f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    }
  }
  store4<OUT>(out + at, n, N, v, true);
}

struct MlpArgs {
  const uint8_t *codes1, *scales1, *codes2, *scales2;
  int E, H, I, N1;
  const uint16_t *X;
  Routing r;
  int act;
  const void *residual;
  void *out;
  int out_dtype;
  uint16_t *rows;  // [pairs][I]
  float *sums;     // [pairs][H], in the tiled form
  int64_t pairs;
};

// Whether the rows of an expert are few (16 a tile) or the tiles of the longer products are used.
static bool few_rows(int64_t T, int64_t topk, int64_t E) { return T * topk <= 4 * E || T <= 16; }

template <bool PAIRS>
static int launch_up_few(const MlpArgs &a, hipStream_t s) {
  constexpr int G = 4;
  const Args p{a.codes1, a.scales1, a.X, nullptr, a.rows, a.pairs, a.E, a.N1, a.H, {}};
  const int64_t slots = slots_for(a.pairs, a.E, true, 16), blocks = (a.N1 + 16 * G - 1) / (16 * G);
  const int ranges = (a.H + kRange - 1) / kRange, waves = ranges < 8 ? ranges : 8;
  if (slots * blocks * waves * 64 >= (int64_t(1) << 32)) return NF4_ERANGE;
  const dim3 grid((unsigned)(slots * blocks)), threads(64 * waves);
  const size_t lds = (size_t)waves * 16 * 16 * G * 4;
  if (a.H % 128 == 0 && aligned_to(a.scales1, 4))
    hipLaunchKernelGGL((moe_up_kernel<G, true, PAIRS>), grid, threads, lds, s, p, (int)blocks, a.r, a.act);
  else
    hipLaunchKernelGGL((moe_up_kernel<G, false, PAIRS>), grid, threads, lds, s, p, (int)blocks, a.r, a.act);
  return launch_status(hipGetLastError());
}

template <typename OUT>
static int launch_down_few(const MlpArgs &a, hipStream_t s) {
  const Args p{a.codes2, a.scales2, a.rows, nullptr, a.out, a.pairs, a.E, a.H, a.I, {}};
  const int waves = 8;
  const dim3 grid((unsigned)((a.H + 15) / 16)), threads(64 * waves);
  const size_t lds = (size_t)waves * a.r.T * 16 * 4;
  if (a.I % 128 == 0 && aligned_to(a.scales2, 4))
    hipLaunchKernelGGL((moe_down_kernel<true, OUT>), grid, threads, lds, s, p, a.r, a.residual);
  else
    hipLaunchKernelGGL((moe_down_kernel<false, OUT>), grid, threads, lds, s, p, a.r, a.residual);
  return launch_status(hipGetLastError());
}

template <class ROWS, class EPI, bool F32, bool B16>
static int launch_tiles(Product<ROWS, EPI, F32, B16> p) {
  const Args &a = p.a;
  const int64_t rows = (a.R + a.E - 1) / a.E;
  const auto tiles = [&](int bm, int bn) { return slots_for(a.R, a.E, true, bm) * ((a.N + bn - 1) / bn); };
  if (rows > 16 && tiles(32, 128) >= 384) return p.template tile<2, 2, 4, 2, 2, 1>();
  if (rows > 8) return p.template tile<2, 1, 4, 4, 4, 1>();
  return p.template tile<1, 1, 4, 4, 4, 1>();
}

static int launch_mlp(const MlpArgs &a, hipStream_t s) {
  if (few_rows(a.r.T, a.r.topk, a.E)) {
    if (int r = is_gated(a.act) ? launch_up_few<true>(a, s) : launch_up_few<false>(a, s)) return r;
    return a.out_dtype == NF4_F32 ? launch_down_few<float>(a, s) : launch_down_few<uint16_t>(a, s);
  }
  const Args up{a.codes1, a.scales1, a.X, nullptr, a.rows, a.pairs, a.E, a.N1, a.H, {}};
  int r;
  if (is_gated(a.act))
    r = launch_tiles(Product<TokenRows, ActRows<true>, false, true>{up, true, NF4_BF16, {a.r}, {a.r, a.act}, s});
  else
    r = launch_tiles(Product<TokenRows, ActRows<false>, false, true>{up, true, NF4_BF16, {a.r}, {a.r, a.act}, s});
  if (r) return r;
  const Args down{a.codes2, a.scales2, a.rows, nullptr, a.sums, a.pairs, a.E, a.H, a.I, {}};
  if (int q = launch_tiles(Product<PairRows, PlainOut, true, false>{down, true, NF4_F32, {a.r}, {}, s})) return q;
  const dim3 grid((unsigned)((a.H + 1023) / 1024), (unsigned)a.r.T);
  if (a.out_dtype == NF4_F32)
    hipLaunchKernelGGL((moe_rows_sum_kernel<float>), grid, dim3(256), 0, s, a.sums, a.r, a.H, a.residual,
                       static_cast<float *>(a.out));
  else
    hipLaunchKernelGGL((moe_rows_sum_kernel<uint16_t>), grid, dim3(256), 0, s, a.sums, a.r, a.H, a.residual,
                       static_cast<uint16_t *>(a.out));
  return launch_status(hipGetLastError());
}

// pairs (token, expert) at most, and where the second part of the workspace starts
static int64_t pair_count(int64_t T, int64_t topk, int64_t E) { return T * (topk < E ? topk : E); }
static int64_t rows_bytes(int64_t pairs, int64_t I) { return (pairs * I * 2 + 255) / 256 * 256; }

static int check_mlp(int64_t E, int64_t H, int64_t I, int act, int64_t T, int64_t topk) {
  if (E < 1 || T < 0 || topk < 1 || !known_act(act)) return NF4_EINVAL;
  if (int r = check_mx_shape(H, I)) return r;
  if (I > NF4_MAX_K) return NF4_ERANGE;
  if (int r = check_mx_shape(is_gated(act) ? 2 * I : I, H)) return r;
  if (E > NF4_MOE_MAX_E || topk > NF4_MOE_MAX_E || T > kTokens) return NF4_ERANGE;
  return NF4_OK;
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int64_t nf4_moe_mlp_workspace_bytes(int64_t E, int64_t H, int64_t I, int act, int64_t T, int64_t topk) {
  using namespace nf4::mx;
  if (check_mlp(E, H, I, act, T, topk)) return -1;
  const int64_t pairs = pair_count(T, topk, E);
  return rows_bytes(pairs, I) + (few_rows(T, topk, E) ? 0 : pairs * H * 4);
}

int nf4_moe_mlp(const uint8_t *codes1, const uint8_t *scales1, const uint8_t *codes2, const uint8_t *scales2,
                int64_t E, int64_t H, int64_t I, const uint16_t *X, const int64_t *experts, const float *weights,
                int64_t T, int64_t topk, int act, const void *residual, void *out, int out_dtype, void *workspace,
                int64_t workspace_bytes, void *stream) {
  using namespace nf4::mx;
  if (!codes1 || !scales1 || !codes2 || !scales2 || !nf4::known_dtype(out_dtype) ||
      (T > 0 && (!X || !experts || !weights || !out)))
    return NF4_EINVAL;
  if (int r = check_mlp(E, H, I, act, T, topk)) return r;
  if (!nf4::aligned_to(codes1, 16) || !nf4::aligned_to(codes2, 16) || !nf4::aligned_to(X, 16) ||
      !nf4::aligned_to(out, 16) || !nf4::aligned_to(residual, 16) || !nf4::aligned_to(experts, 8) ||
      !nf4::aligned_to(weights, 4) || !nf4::aligned_to(workspace, 256))
    return NF4_EALIGN;
  if (T > 0 && (!workspace || workspace_bytes < nf4_moe_mlp_workspace_bytes(E, H, I, act, T, topk)))
    return NF4_ERANGE;
  if (int r = nf4::device_status()) return r;
  if (T == 0) return NF4_OK;
  const int64_t pairs = pair_count(T, topk, E);
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const MlpArgs a{codes1, scales1, codes2, scales2, (int)E, (int)H, (int)I, (int)(is_gated(act) ? 2 * I : I), X,
                  {experts, weights, (int)T, (int)topk, (int)E}, act, residual, out, out_dtype,
                  reinterpret_cast<uint16_t *>(ws), reinterpret_cast<float *>(ws + rows_bytes(pairs, I)), pairs};
  return launch_mlp(a, (hipStream_t)stream);
}

}  // extern "C"
