// mx_device.h -- device-side pieces shared by the MXFP4 products (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_device.h"

namespace nf4 {
namespace mx {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// A voffset that is outside every buffer here (their sizes are below 2^31):
// the load returns zero.
constexpr int kOutside = (int)0x80000000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, kBufferWord3);
}

// 16 bytes a lane from memory straight into LDS at base + 16 * lane.  The compiler
// does not tie these loads to the reads of that memory: lds_loads_done() waits
// for them (and every other load of the wave) and precedes the barrier after
// which the data is read.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rsrc, uint8_t *base, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)base, 16,
                                           voffset, 0, 0, 0);
}
__device__ __forceinline__ void lds_loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 8 codes (one word, low nibble first) times 2^(byte - 127) as bf16: exact, the
// element and the power of two fit bf16.  `scale` holds the byte in the exponent
// field; a byte of 255 gives NaN.
__device__ __forceinline__ u32x4_t decode8(uint32_t w, float scale) {
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return r;
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

// One row tile: rows [row0, row0 + rows) of matrix e (e < 0: rows that belong to
// no expert and are written as zero; rows 0: nothing).
struct RowTile {
  int e, row0, rows;
};

// The slot-th row tile of at most bm rows.  Dense: offsets is null and the tiles
// follow one another.  Grouped: expert e's rows are [offsets[e], offsets[e+1]),
// its tiles come after those of the experts before it, and the tiles of the
// rows from offsets[E] to R come last.  Offsets are held to [0, R] and to
// ascending order, so no tile leaves the arrays whatever they say.  Every wave
// finds its tile by itself, 64 experts at a time.
__device__ __forceinline__ RowTile find_tile(const int32_t *offsets, int E, int64_t R, int slot,
                                             int bm) {
  RowTile t{0, 0, 0};
  const int r = (int)R;
  if (!offsets) {
    t.row0 = slot * bm;
    t.rows = min(bm, r - t.row0);
    return t;
  }
  const int lane = threadIdx.x & 63;
  int before = 0, last = 0;  // tiles so far; end of the last expert's rows
  for (int base = 0; base < E; base += 64) {
    const int e = base + lane;
    int a = 0, b = 0;
    if (e < E) {
      a = min(max(offsets[e], 0), r);
      b = min(max(offsets[e + 1], a), r);
    }
    const int tiles = (b - a + bm - 1) / bm;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    const uint64_t hit = __ballot(before + incl > slot && tiles > 0);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int ea = __builtin_amdgcn_readlane(a, l), eb = __builtin_amdgcn_readlane(b, l);
      const int first = before + __builtin_amdgcn_readlane(incl - tiles, l);
      t.e = base + l;
      t.row0 = ea + (slot - first) * bm;
      t.rows = min(bm, eb - t.row0);
      return t;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
    last = __builtin_amdgcn_readlane(b, min(63, E - 1 - base));
  }
  t.e = -1;
  t.row0 = last + (slot - before) * bm;
  t.rows = t.row0 < r ? min(bm, r - t.row0) : 0;
  return t;
}

// Workgroup -> (row tile slot, column block).  Groups of gm slots times one column
// block are dealt out to the 8 XCDs in turn (workgroup id % 8), so a panel of
// weights is read by one XCD's cache for gm row tiles, and the empty slots at the
// end of a grouped launch are spread evenly.
struct Grid {
  int slots, blocks, gm;
};

inline Grid make_grid(int64_t slots, int64_t blocks, int gm) {
  return Grid{(int)slots, (int)blocks, (int)(slots < gm ? slots : gm)};
}
inline int64_t grid_size(const Grid &g) {
  const int64_t groups = (g.slots + g.gm - 1) / g.gm;
  return (groups * g.blocks + 7) / 8 * 8 * g.gm;
}

__device__ __forceinline__ bool grid_item(const Grid &g, int *slot, int *block) {
  const int id = blockIdx.x;
  const int local = id >> 3;
  const int u = local / g.gm * 8 + (id & 7);
  const int group = u / g.blocks;
  *block = u - group * g.blocks;
  *slot = group * g.gm + local % g.gm;
  return *slot < g.slots;
}

// Row tiles a launch has to allow for: every expert (and the rows of none) can
// leave one partial tile.
inline int64_t slots_for(int64_t R, int64_t E, bool grouped, int bm) {
  if (!grouped) return (R + bm - 1) / bm;
  const int64_t part = R < E + 1 ? R : E + 1;
  return R / bm + part;
}

// Four consecutive outputs of one row, as fp32 or bf16 (one rounding).
template <typename OUT>
__device__ __forceinline__ void store4(OUT *row, int n, int N, f32x4_t v, bool vec) {
  if (vec) {
    if (n < N) {
      if constexpr (sizeof(OUT) == 4)
        *reinterpret_cast<f32x4_t *>(row + n) = v;
      else
        *reinterpret_cast<u32x2_t *>(row + n) = u32x2_t{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16),
                                                        bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) {
        if constexpr (sizeof(OUT) == 4)
          row[n + i] = v[i];
        else
          row[n + i] = (OUT)bf16_bits(v[i]);
      }
  }
}

}  // namespace mx
}  // namespace nf4
