// What the tiled products share: copies from memory straight to LDS and the order of
// the tiles (block_gemm.hip, mx_gemm.hip).
#pragma once

#include "qw_internal.h"

namespace qw {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A value that all lanes of a wave have alike, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
         (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
}

// A buffer descriptor of `bytes` from `base`: reads beyond give zeros.  The scalar offset of a
// load counts (measured: voff + soff >= bytes reads nothing, an empty buffer at any soff), on
// which copies behind a row's last scales and behind the last tile rely.
__device__ __forceinline__ i32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), (int)bytes, 0x00020000};
}

// 16 bytes a lane from buffer + voff + soff to LDS at `lds` + 16 * lane.  The
// compiler does not see this write (it would wait for every copy in flight
// before any LDS read): landed() orders it.  Nothing else here uses m0.
__device__ __forceinline__ void copy_to_lds(i32x4 buffer, uint32_t voff, uint32_t soff,
                                            uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}
// The same where `when` (one value for the wave) is not zero.  The compiler sees no branch:
// at one it would move the products before it behind it.
__device__ __forceinline__ void copy_to_lds_when(int when, i32x4 buffer, uint32_t voff,
                                                 uint32_t soff, uint32_t lds) {
  asm volatile("s_cmp_eq_u32 %4, 0\n\ts_cbranch_scc1 .Lskip%=\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
               "buffer_load_dwordx4 %1, %2, %3 offen lds\n.Lskip%=:"
               :: "s"(lds), "v"(voff), "s"(buffer), "s"(soff), "s"(when) : "memory", "scc");
}
// The same, 4 bytes a lane.
__device__ __forceinline__ void copy4_to_lds(i32x4 buffer, uint32_t voff, uint32_t soff,
                                             uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}
// This wave's copies but the LEFT newest, and its LDS accesses, are done, and
// so are the block's.
template <int LEFT>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "i"(LEFT) : "memory");
}

// This wave's LDS accesses are done, and so are the block's; copies stay on
// their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The tile of a block.  Blocks go to the 8 XCDs in turn, each with an L2 of its
// own: an XCD takes a contiguous run of the tiles, ordered in bands of 8 tile
// rows (tokens) and down each band column by column, so that the 32 tiles it
// works on together share 8 tiles of x and 4 of the weight.
__device__ __forceinline__ void tile_place(int64_t block, int64_t tiles, int64_t tiles_m,
                                           int64_t& tm, int64_t& tn) {
  const int64_t xcd = block & 7, each = tiles >> 3, extra = tiles & 7;
  const int64_t t = xcd * each + min(xcd, extra) + (block >> 3);
  const int64_t tiles_n = tiles / tiles_m;
  const int64_t band = t / (8 * tiles_n), in_band = t - band * 8 * tiles_n;
  const int64_t height = min((int64_t)8, tiles_m - band * 8);
  tn = in_band / height;
  tm = band * 8 + in_band - tn * height;
}

}  // namespace qw
