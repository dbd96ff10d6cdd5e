// moe_mlp.hip -- a whole layer of experts for a few tokens (gfx950):
//   out[t] = sum_j weights[t][j] W2[e] act(W1[e] X[t]) (+ residual[t]),  e = experts[t][j],
// W1 [E][N1][H] and W2 [E][H][I] packed MXFP4; gated, N1 = 2 I.
//
// The tokens are not sorted beforehand: every workgroup makes for each expert the mask of
// its tokens (at most 64) in LDS.  A pair (token, expert) is one row, whose weight is the
// sum over the token's slots with that expert; rows are numbered by expert, then token.
// The first kernel writes act(W1 x) times the row's weight, in bf16, which is what the second
// one's matrix instructions take (one rounding, as between two layers: out in bf16 is 2.4e-3 of
// its norm off where one rounding at the end leaves 1.7e-3); the second one's sums over all its
// rows are then the output.
#include "moe_units.h"
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

// Inclusive prefix over the wave: within rows of 16 lanes, then the rows' last lanes are
// passed on (row_bcast 15 and 31).
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
#define NF4_ADD_DPP(ctrl, rows) \
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false)
  NF4_ADD_DPP(0x111, 0xf);
  NF4_ADD_DPP(0x112, 0xf);
  NF4_ADD_DPP(0x114, 0xf);
  NF4_ADD_DPP(0x118, 0xf);
  NF4_ADD_DPP(0x142, 0xa);
  NF4_ADD_DPP(0x143, 0xc);
#undef NF4_ADD_DPP
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
#pragma unroll 4
  for (int j = 0; j < r.topk; ++j) {  // both loaded, so that no load waits for another
    const float v = r.weights[token * r.topk + j];
    w += r.experts[token * r.topk + j] == e ? v : 0.f;
  }
  return w;
}

// A tile's rows, for as long as it takes.
struct TileState {
  int tokens[kTokens];
  float weight[kTokens];
};
__device__ __forceinline__ TileState &tile_state() {
  __shared__ TileState s;
  return s;
}
// A tile of the longer products; the masks are done with before the stages come to their place.
__device__ __forceinline__ RowTile tile_rows(const Routing &r, int slot, int bm, void *lds) {
  Masks &masks = *static_cast<Masks *>(lds);
  make_masks(r, masks);
  return find_rows(r, masks, slot, bm, tile_state().tokens);
}

// Rows of X by the tokens of a tile.
struct TokenRows {
  Routing r;
  __device__ __forceinline__ RowTile find(const Args &, int slot, int bm, void *lds) const {
    return tile_rows(r, slot, bm, lds);
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
  __device__ __forceinline__ RowTile find(const Args &, int slot, int bm, void *lds) const {
    return tile_rows(r, slot, bm, lds);
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

// The range of up to 16 rows of X: row offsets are the lane's (l16); lanes without a row (not
// `in`) take zeros.  No branch here or in the products: behind one the compiler could not
// count the loads in flight and would wait for all of them.
__device__ __forceinline__ void load_range(u32x4_t (&x)[4][4], __amdgpu_buffer_rsrc_t xrs, bool in, int row_bytes,
                                           int K, int k0) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = k0 + 128 * s + 32 * q;
    const int at = in && k < K ? row_bytes + k * 2 : kOutside;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[s][j] = __builtin_amdgcn_raw_buffer_load_b128(xrs, at + j * 16, 0, 0);
  }
}

template <bool SVEC, bool PAIRS>
__device__ __forceinline__ f32x4_t multiply(const RangeLoads<SVEC, PAIRS> &w, const u32x4_t (&x)[4][4], f32x4_t acc,
                                            int K, int k0) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float sc = w.scale(s, K, k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mfma16(decode8(w.cw[s][j], sc), x[s][j], acc);
  }
  return acc;
}

// First product.  The work is the items (tile of rows, block of 16 G weight rows), in this
// order, dealt out in runs of equal length: as many workgroups as the CUs hold, each with
// one run, so that nothing depends on how the tokens chose.  In a tile the workgroup's
// waves have a range of K each (several in turn, if K is longer than the waves' ranges),
// whose rows of X stay in registers while the weights pass by; the next two blocks are
// always under way; the waves' sums meet in LDS once a block, in the two halves of `part`
// in turn.
struct UpArgs {
  Args p;
  Routing r;
  int blocks, act;
  uint32_t *counters;  // of the second product, set to zero here
  int ncounters;
};

// Tiles of all experts.
__device__ __forceinline__ int count_tiles(const Routing &r, const Masks &masks) {
  int n = 0;
  for (int base = 0; base < r.E; base += 64) {
    const int e = base + (threadIdx.x & 63);
    const int rows = e < r.E ? __popcll(mask_of(masks, e)) : 0;
    n += __builtin_amdgcn_readlane((int)wave_prefix((uint32_t)(rows + 15) >> 4), 63);
  }
  return n;
}

// Bound by memory, and by the 8 us that it takes to route, to fill and to end: experts of 28672
// x 4096, 17 tokens with 2 of 8 91-100 us (5.0-5.5 TB/s), 16 rows of each of 8 108-112, two
// experts of one token 31 (4.0), 19 x 8 slots of 128 experts of 1536 x 2048 37.  With static shares of the tiles that there could
// be, empty ones among them, the first took 126; weights asked for one block ahead where
// the compiler moved the loads down to their use, 29 of the two experts' became 33.
// LONG: more than one pass.  (Compiled in: with loads of X behind a branch, the products
// would wait for everything in flight.)
template <int G, bool SVEC, bool PAIRS, bool LONG>
__global__ void __launch_bounds__(512)
    moe_up_kernel(UpArgs a) {
  extern __shared__ float part[];  // [2][wave][row][16 G]
  __shared__ Masks masks;
  const Args &p = a.p;
  const Routing &r = a.r;
  TileState &st = tile_state();
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int kb = p.K >> 5, kc = p.K >> 1;
  make_masks(r, masks);
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.ncounters; i += gridDim.x * blockDim.x)
    a.counters[i] = 0u;
  // fp64 (fewer than 2^37 items, so exact but for the rounding of lo and hi, which is one for
  // both sides of a border): a 64-bit division takes a microsecond
  const double items = (double)count_tiles(r, masks) * a.blocks;
  const int64_t lo = (int64_t)(items * blockIdx.x / gridDim.x), hi = (int64_t)(items * (blockIdx.x + 1) / gridDim.x);
  const int passes = LONG ? (p.K + waves * kRange - 1) / (waves * kRange) : 1;
  const ActRows<PAIRS> out{r, a.act};
  float *half = part;
  int first = threadIdx.x;  // of a block's outputs: another wave has them each time
  for (int64_t at = lo; at < hi;) {
    const int tile = (int)((double)at / a.blocks), b0 = (int)(at - (int64_t)tile * a.blocks);
    const int b1 = (int)(hi - at < a.blocks - b0 ? b0 + (hi - at) : a.blocks);
    at += b1 - b0;
    __syncthreads();  // the last tile's state has been read
    const RowTile t = find_rows(r, masks, tile, 16, st.tokens);
    const uint8_t *const ce = p.codes + (int64_t)t.e * p.N * kc, *const se = p.scales + (int64_t)t.e * p.N * kb;
    const __amdgpu_buffer_rsrc_t xrs = buffer(p.X, (int64_t)r.T * p.K * 2);
    const int xrow = (l16 < t.rows ? st.tokens[l16] : 0) * p.K * 2;
    const int kfirst = wave * kRange;
    RangeLoads<SVEC, PAIRS> w[2][G];
    const auto load = [&](RangeLoads<SVEC, PAIRS> &to, int b, int g, int pass) __attribute__((always_inline)) {
      const int n0 = b * 16 * G, cols = b < b1 ? min(16 * G, p.N - n0) : 0;  // past the run the buffers are empty
      const int col = PAIRS ? n0 >> 1 : n0, wrows = PAIRS && cols > 0 ? (p.N + cols) >> 1 : cols;
      to.load(ce + (int64_t)col * kc, se + (int64_t)col * kb, wrows, g * 16, p.N, p.K, kfirst + pass * waves * kRange);
    };
    const auto advance = [&](int &b, int &pass) __attribute__((always_inline)) {
      if (++pass == passes) {
        pass = 0;
        ++b;
      }
    };
    int b = b0, pass = 0, fb = b0, fpass = 0;  // this step, and the one whose weights are asked for
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int g = 0; g < G; ++g) load(w[i][g], fb, g, fpass);
      advance(fb, fpass);
    }
    u32x4_t x[4][4];
    load_range(x, xrs, l16 < t.rows, xrow, p.K, kfirst);
    if ((int)threadIdx.x < t.rows) st.weight[threadIdx.x] = row_weight(r, st.tokens[threadIdx.x], t.e);
    f32x4_t acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const auto step = [&](RangeLoads<SVEC, PAIRS> (&now)[G]) __attribute__((always_inline)) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        acc[g] = multiply(now[g], x, acc[g], p.K, kfirst + pass * waves * kRange);
        load(now[g], fb, g, fpass);
        __builtin_amdgcn_sched_barrier(0);  // else the loads are moved to where they are needed
      }
      advance(fb, fpass);
      const int n0 = b * 16 * G;
      const bool last = pass + 1 == passes;
      advance(b, pass);
      if constexpr (LONG) load_range(x, xrs, l16 < t.rows, xrow, p.K, kfirst + pass * waves * kRange);
      if (!last) return;
      if (l16 < t.rows) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          *reinterpret_cast<f32x4_t *>(half + (wave * 16 + l16) * (16 * G) + g * 16 + q * 4) = acc[g];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      __syncthreads();
      constexpr int W = PAIRS ? 8 : 4, quads = 16 * G / W;
      for (int i = first; i < t.rows * quads; i += blockDim.x) {
        const int m = i / quads, c = i % quads * W;
        if (n0 + c >= p.N) continue;
        f32x4_t u = {0.f, 0.f, 0.f, 0.f}, v = u;
        for (int k = 0; k < waves; ++k) {
          const float *s = half + (k * 16 + m) * (16 * G) + c;
          u += *reinterpret_cast<const f32x4_t *>(s);
          if constexpr (PAIRS) v += *reinterpret_cast<const f32x4_t *>(s + 4);
        }
        if constexpr (PAIRS)
          out.put(p, t, m, (n0 + c) >> 1, f32x4_t{u[0], u[2], v[0], v[2]}, f32x4_t{u[1], u[3], v[1], v[3]});
        else
          out.put(p, t, m, n0 + c, u, u);
      }
      half = half == part ? part + waves * 16 * 16 * G : part;
      first = first < 64 ? first + blockDim.x - 64 : first - 64;
    };
    while (true) {
      step(w[0]);
      if (b >= b1) break;
      step(w[1]);
      if (b >= b1) break;
    }
  }
}

// Second product and the sum over a token's experts: a workgroup owns 16 G columns of the
// output for all tokens (G groups of 16, for which a range of the rows is loaded once).  A
// unit is a range of an expert's I; the units go in turn to the waves of the `splits`
// workgroups that share the columns, and a wave adds its units, in order, into sums of its
// own in LDS.
// Bound by memory (rows' pieces of 256 bytes a wave: 4.2 TB/s) and 7 us of start, fill and end:
// experts of 4096 x 14336, 17 tokens with 2 of 8 60-63 us, 16 rows of each of 8 78-81, two experts
// of one token 22-26; about 90 of 128 of 2048 x 768 28.  (Built and slower: the items of the first product with a last workgroup
// that adds up, 70, 24 and 33, since few workgroups are last for all columns; the sums
// written back by a fence of the whole cache, 76, 23 and 62.)
template <int G, bool SVEC, typename OUT>
__global__ void __launch_bounds__(512)
    moe_down_kernel(Args p, int splits, Routing r, const void *residual, float *parts, uint32_t *counters) {
  constexpr int kCols = 16 * G, kQuads = kCols / 4;
  extern __shared__ float sums[];  // [wave][token][kCols]
  __shared__ ActiveExperts act;
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int block = blockIdx.x / splits, split = blockIdx.x - block * splits;
  const int n0 = block * kCols, cols = min(kCols, p.N - n0);
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
  for (int i = threadIdx.x; i < waves * r.T * (kCols / 4); i += blockDim.x)
    reinterpret_cast<f32x4_t *>(sums)[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const int kb = p.K >> 5, kc = p.K >> 1;
  // read from LDS, but the same for the wave: buffers have to be in scalar registers
  const auto uniform = [](int v) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(v); };
  const int ranges = (p.K + kRange - 1) / kRange, units = uniform(act.count) * ranges, step = waves * splits;
  float *const own = sums + wave * r.T * kCols;
  const auto unit = [&](int u) __attribute__((always_inline)) {
    return unit_of(act, u, units, ranges, kRange, cols, uniform);
  };
  const auto load_x = [&](u32x4_t (&x)[4][4], const Unit &v, int m0) __attribute__((always_inline)) {
    const int rows = max(min(16, v.rows - m0), 0);
    load_range(x, buffer(p.X + (int64_t)(v.row0 + m0) * p.K, (int64_t)rows * p.K * 2), l16 < rows, l16 * p.K * 2, p.K,
               v.k0);
  };
  const auto load_w = [&](RangeLoads<SVEC, false> &w, const Unit &v, int g) __attribute__((always_inline)) {
    const int64_t first = (int64_t)v.e * p.N + n0;
    w.load(p.codes + first * kc, p.scales + first * kb, v.cols, g * 16, p.N, p.K, v.k0);
  };
  // Row l16's token: lanes are tokens, and send theirs to their row.
  const auto token = [&](const Unit &v, int m0) __attribute__((always_inline)) {
    const int rank = (int)__popcll(v.mask & ((uint64_t(1) << lane) - 1)) - m0;
    const bool mine = (v.mask >> lane & 1) && rank >= 0 && rank < 16;
    return __shfl(__builtin_amdgcn_ds_permute(mine ? rank * 4 : 63 * 4, lane), l16, 64);
  };
  const auto add = [&](const Unit &v, int m0, int tok, int g, f32x4_t s) __attribute__((always_inline)) {
    if (m0 + l16 < v.rows) *reinterpret_cast<f32x4_t *>(own + tok * kCols + g * 16 + q * 4) += s;
  };
  // The weights of the next unit are under way while this one's are multiplied, each group's
  // asked for when its registers are free; the rows' values follow at the unit's end.
  RangeLoads<SVEC, false> w[G];
  u32x4_t x[4][4];
  const int u0 = split * waves + wave;
  Unit v = unit(u0);
#pragma unroll
  for (int g = 0; g < G; ++g) load_w(w[g], v, g);
  load_x(x, v, 0);
  for (int u = u0; u < units; u += step) {
    const Unit after = unit(u + step);
    const int tok = token(v, 0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      add(v, 0, tok, g, multiply(w[g], x, f32x4_t{0.f, 0.f, 0.f, 0.f}, p.K, v.k0));
      load_w(w[g], after, g);
      __builtin_amdgcn_sched_barrier(0);  // else the loads are moved to where they are needed
    }
    for (int m0 = 16; m0 < v.rows; m0 += 16) {  // more rows than a tile: the weights once more
      const int more = token(v, m0);
      load_x(x, v, m0);
#pragma unroll 1
      for (int g = 0; g < G; ++g) {
        RangeLoads<SVEC, false> again;
        load_w(again, v, g);
        add(v, m0, more, g, multiply(again, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, p.K, v.k0));
      }
    }
    v = after;
    load_x(x, v, 0);
  }
  __syncthreads();
  const auto put = [&](int t, int c, f32x4_t v) __attribute__((always_inline)) {
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
  };
  float *const all = parts + (int64_t)block * splits * r.T * kCols;
  for (int i = threadIdx.x; i < r.T * kQuads; i += blockDim.x) {
    const int t = i / kQuads, c = i % kQuads * 4;
    f32x4_t v = *reinterpret_cast<const f32x4_t *>(sums + t * kCols + c);
    for (int k = 1; k < waves; ++k) v += *reinterpret_cast<const f32x4_t *>(sums + (k * r.T + t) * kCols + c);
    if (splits == 1) {
      if (n0 + c < p.N) put(t, c, v);
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)  // agent-scope: performed where every XCD sees them
      __hip_atomic_store(all + (split * r.T + t) * kCols + c + k, v[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (splits == 1) return;
  // The last of the columns' workgroups to come here adds all parts, in order.  Each
  // thread waits until its stores are performed (vmcnt), the barrier puts that before the
  // count, and only the workgroup that saw the last count reads, with loads that go where
  // the stores went.
  __shared__ int last;
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(counters + block, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           (uint32_t)(splits - 1);
  __syncthreads();
  if (!last) return;
  for (int i = threadIdx.x; i < r.T * kQuads; i += blockDim.x) {
    const int t = i / kQuads, c = i % kQuads * 4;
    if (n0 + c >= p.N) continue;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] += __hip_atomic_load(all + (s * r.T + t) * kCols + c + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    put(t, c, v);
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
  uint16_t *rows;      // [pairs][I]
  float *sums;         // [pairs][H] in the tiled form, else the second product's parts
  uint32_t *counters;  // of the column blocks that are shared out
  int64_t pairs;
};

constexpr int kFewWaves = 8;  // of a workgroup of the first product of few rows

// Whether the rows of an expert are few (16 a tile) or the tiles of the longer products are
// used; at most 2^13 pairs with few (16 x 512).
// Both, us, rows an expert in brackets: 4096 x 14336 of 8 experts 170 and 182 (4.2), 187 both
// (6), 191 and 189 (8), 242 and 195 (12); 2048 x 768 of 128 91 and 84 (3.8), of 96 77 and 68 (5),
// of 64 60 and 49 (7.5); 2048 x 4096 of 10 62 and 46 (6.4); 4096 x 1536 of 121 259 and 276 (4.2),
// of 32 84 and 86 (6).
// Where H takes the first product more than one pass, that waits for X in each: few and tiles,
// 8 of 64 experts of 7168 x 2048 59 and 47 (one token), of 128 of 6144 x 1024 327 and 253 (32), 4
// of 32 of 5120 x 1536 96 and 77 (8); 1 of 16 of 5120 x 8192 129 and 137 (8); but one of 5120 x
// 2048, one token, 18 and 26.
// The rule does not see I: where that is as small as 768 the tiles would be the faster ones from
// 3.8 rows an expert on, by 8 to 13 %, and 5120 x 8192 is on its slower side by 6 %.
static bool few_rows(int64_t T, int64_t topk, int64_t E, int64_t H) {
  if (H > kFewWaves * kRange && T * (topk < E ? topk : E) >= 8) return false;
  return T * topk <= 5 * E || T <= 16;
}

// the tiles that there can be
static int64_t tiles_of(int64_t pairs, int64_t E) { return slots_for(pairs, E, true, 16); }

template <int G, bool PAIRS>
static int launch_up_as(const UpArgs &u, bool svec, bool longer, dim3 grid, dim3 threads, size_t lds, hipStream_t s) {
  if (svec && !longer)
    hipLaunchKernelGGL((moe_up_kernel<G, true, PAIRS, false>), grid, threads, lds, s, u);
  else if (svec)
    hipLaunchKernelGGL((moe_up_kernel<G, true, PAIRS, true>), grid, threads, lds, s, u);
  else if (!longer)
    hipLaunchKernelGGL((moe_up_kernel<G, false, PAIRS, false>), grid, threads, lds, s, u);
  else
    hipLaunchKernelGGL((moe_up_kernel<G, false, PAIRS, true>), grid, threads, lds, s, u);
  return launch_status(hipGetLastError());
}
template <bool PAIRS>
static int launch_up_few(const MlpArgs &a, int ncounters, hipStream_t s) {
  const int ranges = (a.H + kRange - 1) / kRange, waves = ranges < kFewWaves ? ranges : kFewWaves;
  const int hold = 256 * (8 / waves);
  const int64_t tiles = tiles_of(a.pairs, a.E);
  // blocks of one group where two to a block would leave CUs without one
  const int g = tiles * ((a.N1 + 31) / 32) >= hold ? 2 : 1, blocks = (a.N1 + 16 * g - 1) / (16 * g);
  const dim3 grid((unsigned)(tiles * blocks < hold ? tiles * blocks : hold)), threads(64 * waves);
  const size_t lds = (size_t)waves * 16 * 16 * g * 4 * 2;
  const UpArgs u{{a.codes1, a.scales1, a.X, nullptr, a.rows, a.pairs, a.E, a.N1, a.H, {}}, a.r, blocks, a.act,
                 a.counters, ncounters};
  const bool svec = a.H % 128 == 0 && aligned_to(a.scales1, 4);
  return g == 2 ? launch_up_as<2, PAIRS>(u, svec, ranges > waves, grid, threads, lds, s)
                : launch_up_as<1, PAIRS>(u, svec, ranges > waves, grid, threads, lds, s);
}

// How the second product is dealt out: groups of 16 columns a workgroup, and workgroups that
// share a column block's units, as many as make one a CU.
struct DownPlan {
  int g, blocks, splits;
};
static DownPlan down_plan(int64_t H, int64_t I, int64_t tiles) {
  DownPlan d;
  const int64_t units = tiles * ((I + kRange - 1) / kRange);
  const auto splits = [&](int g) {
    const int64_t b = (H + 16 * g - 1) / (16 * g), most = (units + 7) / 8;
    const int64_t n = b >= 192 ? 1 : 256 / b;
    return n < most ? n : most;
  };
  // G = 4 from where every wave of the chip has a unit and a half, us against G = 1: 2 experts
  // of 4096 x 14336 (56 units) 22.7, 24.1; of 4096 x 8192 (32) 15.1, 15.3; of 4096 x 4096 (16)
  // 13.4, 9.0; 8 of 128 of 2048 x 768 (16) 12.7, 7.9, about 90 of them 28, 34.  And where G = 1
  // makes more than 256 column blocks: 8 experts of 5120 x 2048 (32 units) 20.8, 25.4; 2 of
  // 8192 x 4096 (16) 13.8, 17.0; 1 of 8192 x 512 (1) 5.4, 6.4; 4 of 4608 x 1024 (8) 11.4, 10.3
  const int64_t b4 = (H + 63) / 64;
  d.g = H > 4096 || 2 * units * (b4 < 256 ? b4 : 256) >= 3 * 8 * 256 ? 4 : 1;
  d.blocks = (int)((H + 16 * d.g - 1) / (16 * d.g));
  d.splits = (int)splits(d.g);
  return d;
}

template <int G, typename OUT>
static int launch_down_as(const MlpArgs &a, const DownPlan &d, hipStream_t s) {
  const Args p{a.codes2, a.scales2, a.rows, nullptr, a.out, a.pairs, a.E, a.H, a.I, {}};
  const int waves = 8;
  const dim3 grid((unsigned)(d.blocks * d.splits)), threads(64 * waves);
  const size_t lds = (size_t)waves * a.r.T * 16 * G * 4;
  if (a.I % 128 == 0 && aligned_to(a.scales2, 4))
    hipLaunchKernelGGL((moe_down_kernel<G, true, OUT>), grid, threads, lds, s, p, d.splits, a.r, a.residual, a.sums,
                       a.counters);
  else
    hipLaunchKernelGGL((moe_down_kernel<G, false, OUT>), grid, threads, lds, s, p, d.splits, a.r, a.residual, a.sums,
                       a.counters);
  return launch_status(hipGetLastError());
}
template <typename OUT>
static int launch_down_few(const MlpArgs &a, const DownPlan &d, hipStream_t s) {
  return d.g == 4 ? launch_down_as<4, OUT>(a, d, s) : launch_down_as<1, OUT>(a, d, s);
}

static int launch_few(const MlpArgs &a, hipStream_t s) {
  const DownPlan d = down_plan(a.H, a.I, tiles_of(a.pairs, a.E));
  const int n = d.splits > 1 ? d.blocks : 0;
  if (int r = is_gated(a.act) ? launch_up_few<true>(a, n, s) : launch_up_few<false>(a, n, s)) return r;
  return a.out_dtype == NF4_F32 ? launch_down_few<float>(a, d, s) : launch_down_few<uint16_t>(a, d, s);
}

template <class ROWS, class EPI, bool F32, bool B16>
static int launch_tiles(Product<ROWS, EPI, F32, B16> p) {
  const Args &a = p.a;
  const auto tiles = [&](int bm, int bn) { return slots_for(a.R, a.E, true, bm) * ((a.N + bn - 1) / bn); };
  // 32 x 128, us, first and second product of 64 tokens, 8 experts of 4096 x 14336: 64 k a
  // stage 118 and 66, 128 k (one workgroup a CU) 129 and 55; 32 x 64 137 and 67, 64 x 128 128
  // and 76
  if (tiles(32, 128) >= 768) return p.template tile<2, 2, 4, 2, 2, 1>();
  if (tiles(32, 128) >= 256) return p.template tile<2, 2, 4, 4, 4, 1>();
  return p.template tile<2, 1, 4, 4, 4, 1>();
}

static int launch_mlp(const MlpArgs &a, hipStream_t s) {
  if (few_rows(a.r.T, a.r.topk, a.E, a.H)) return launch_few(a, s);
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
static int64_t whole(int64_t bytes) { return (bytes + 255) / 256 * 256; }
// what of the workspace is whose
struct MlpPlan {
  int64_t pairs, sums, counters, bytes;
};
static MlpPlan mlp_plan(int64_t E, int64_t H, int64_t I, int64_t T, int64_t topk) {
  MlpPlan d;
  d.pairs = pair_count(T, topk, E);
  d.sums = whole(d.pairs * I * 2);
  if (!few_rows(T, topk, E, H)) {
    d.counters = d.bytes = d.sums + whole(d.pairs * H * 4);
    return d;
  }
  const DownPlan s = down_plan(H, I, tiles_of(d.pairs, E));
  d.counters = d.sums + (s.splits > 1 ? whole((int64_t)s.blocks * s.splits * T * 16 * s.g * 4) : 0);
  d.bytes = d.counters + (s.splits > 1 ? whole((int64_t)s.blocks * 4) : 0);
  return d;
}

static int check_mlp(int64_t E, int64_t H, int64_t I, int act, int64_t T, int64_t topk) {
  if (E < 1 || T < 0 || topk < 1 || !known_act(act)) return NF4_EINVAL;
  if (int r = check_mx_shape(H, I)) return r;
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
  return T == 0 ? 0 : mlp_plan(E, H, I, T, topk).bytes;
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
  const MlpPlan d = mlp_plan(E, H, I, T, topk);
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const MlpArgs a{codes1, scales1, codes2, scales2, (int)E, (int)H, (int)I, (int)(is_gated(act) ? 2 * I : I), X,
                  {experts, weights, (int)T, (int)topk, (int)E}, act, residual, out, out_dtype,
                  reinterpret_cast<uint16_t *>(ws), reinterpret_cast<float *>(ws + d.sums),
                  reinterpret_cast<uint32_t *>(ws + d.counters), d.pairs};
  return launch_mlp(a, (hipStream_t)stream);
}

}  // extern "C"
