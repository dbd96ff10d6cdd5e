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

// A raw buffer as its four words, for the loads below.
__device__ __forceinline__ u32x4_t buffer_words(const void *p, int bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, (uint32_t)bytes, (uint32_t)kBufferWord3};
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 (4) bytes a lane from memory straight into LDS at lds + 16 (4) * lane; lds is
// uniform over the wave.  Written out because the compiler, which sees a store to
// LDS in its builtin for this load, waits for every such load before the next read
// of LDS, whatever it reads; here only lds_loads_but() waits.  It precedes the barrier
// after which the data is read and the end of the kernel.  (s_nop 4: the wait
// states after a vector instruction that wrote a scalar operand; s_nop 0: after m0.)
// The forms for several loads, STEP bytes of LDS apart, wait once.
__device__ __forceinline__ void load_lds16(u32x4_t rsrc, uint32_t lds, int voffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(voffset), "s"(rsrc)
               : "memory");
}
__device__ __forceinline__ void load_lds4(u32x4_t rsrc, uint32_t lds, int voffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds),
               "v"(voffset), "s"(rsrc)
               : "memory");
}
template <int STEP>
__device__ __forceinline__ void load_lds16x2(u32x4_t r0, u32x4_t r1, uint32_t lds, int v0, int v1) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
               "s_add_u32 m0, m0, %5\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %4, 0 offen lds" ::"s"(lds),
               "v"(v0), "v"(v1), "s"(r0), "s"(r1), "n"(STEP)
               : "memory", "scc");
}
// N loads of one buffer
template <int N, int STEP>
__device__ __forceinline__ void load_lds16xn(u32x4_t rsrc, uint32_t lds, const int *v) {
  int i = 0;
#pragma unroll
  for (; i + 3 < N; i += 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds" ::"s"(
                     lds + i * STEP),
                 "v"(v[i]), "v"(v[i + 1]), "v"(v[i + 2]), "v"(v[i + 3]), "s"(rsrc), "n"(STEP)
                 : "memory", "scc");
#pragma unroll
  for (; i + 1 < N; i += 2) load_lds16x2<STEP>(rsrc, rsrc, lds + i * STEP, v[i], v[i + 1]);
#pragma unroll
  for (; i < N; ++i) load_lds16(rsrc, lds + i * STEP, v[i]);
}
// Waits for the wave's loads, all but the newest N.
template <int N>
__device__ __forceinline__ void lds_loads_but() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Four bytes at any byte offset of `base`, from the two words around them: a load
// that is started with `fetch` and finished, when its words are here, with `word`.
struct LooseWords {
  __amdgpu_buffer_rsrc_t rsrc;
  int shift;  // of the base within its word
  __device__ __forceinline__ LooseWords(const uint8_t *base, int64_t bytes) {
    shift = (int)((uintptr_t)base & 3);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base - shift), 0,
                                             (int)((bytes + shift + 3) & ~int64_t(3)), kBufferWord3);
  }
  __device__ __forceinline__ uint32_t fetch(int offset, int i) const {
    return __builtin_amdgcn_raw_buffer_load_b32(rsrc, ((offset + shift) & ~3) + 4 * i, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int offset, uint32_t lo, uint32_t hi) const {
    return __builtin_amdgcn_alignbyte(hi, lo, (offset + shift) & 3);
  }
};

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
// leave one partial tile, and no tile is empty.
inline int64_t slots_for(int64_t R, int64_t E, bool grouped, int bm) {
  if (!grouped) return (R + bm - 1) / bm;
  const int64_t n = R / bm + E + 1;
  return n < R ? n : R;
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
