// Device helpers of the many-adapter kernels (sm_100a): masked tcgen05
// products, row-gathering TMA loads, operand descriptors for narrow tiles.
//
// Rows of a batch belong to different adapters.  A product that adds one
// adapter's low-rank term to a tile runs over all of the tile's rows with the
// lanes of the other rows disabled (tcgen05.mma's disable-output-lane mask:
// lane i of the accumulator is row i of the tile), so the rank-r operand needs
// no zero-filled copies and a row never meets another adapter's values.
//
// The rank dimension is cut into units of kUnit = 64, 32 or 16 columns (the
// widest that divides r): a unit is one adapter's slice of that width, and
// 64 / kUnit units share a 64-wide k-step.  A unit's K-major tile
// [rows x kUnit] has rows of 128, 64 or 32 bytes under the swizzle of that
// width, in atoms of 8 rows.
#pragma once

#include "internal.h"
#include "tcgen05.cuh"

namespace qlora {

// Widest of 64, 32, 16 that divides the rank (r % 16 == 0).
__host__ __device__ constexpr int unit_width(int r) { return r % 64 == 0 ? 64 : (r % 32 == 0 ? 32 : 16); }

// Shared-memory operand descriptor for rows of `width` bf16 (64, 32 or 16)
// under the matching 128-, 64- or 32-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_unit(uint32_t addr, uint32_t lbo, uint32_t sbo, int width) {
  const uint64_t layout = width == 64 ? 2ull : (width == 32 ? 4ull : 6ull);
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (layout << 61);
}

// D += A . B on the lanes whose `off` bit is 0 (off[w] covers lanes 32 w ..).
__device__ __forceinline__ void umma_f16_masked(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint4 off) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w)
      : "memory");
}

// The same for a CTA pair: off0 covers the even CTA's lanes (accumulator rows
// 0..127), off1 the odd CTA's (rows 128..255).
__device__ __forceinline__ void umma_f16_pair_masked(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                     uint4 off0, uint4 off1) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off0.x), "r"(off0.y), "r"(off0.z), "r"(off0.w), "r"(off1.x),
      "r"(off1.y), "r"(off1.z), "r"(off1.w)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// As tma_load_2d_pair, three-dimensional.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar_cluster, int x,
                                                 int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}

// Four rows r0..r3 of a 2D tensor (the map's box is one row high), packed one
// after the other at dst.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int4 rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w),
      "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }


// A call's tile lists and rank, as kernel parameters.
struct MultiParams {
  const int32_t *lists;
  int64_t stride;
  int32_t slots, rows;
  int32_t r, width;
};
inline MultiParams multi_params(const AdapterView &ad, const TileLists &l) {
  return MultiParams{l.base, l.stride, l.slots, l.rows, ad.r, unit_width(ad.r)};
}

// One tile's list.  Written by the kernel this one overlaps: read only after
// griddep_wait, and past L1.
struct MultiTile {
  const int32_t *list;
  const uint4 *mask;
  int adapters;
};
__device__ __forceinline__ MultiTile multi_tile(const MultiParams &p, int tile) {
  const int32_t *t = p.lists + tile * p.stride;
  return MultiTile{t + 4, reinterpret_cast<const uint4 *>(t + 4 + p.slots), __ldcg(t)};
}

// A warp's window on the list: lane l holds entry `first` + l, so the latency
// of a list read is paid once per 32 adapters.  Called by whole warps.
struct AdapterWindow {
  int first = -32, id = 0;
  __device__ __forceinline__ int at(const MultiTile &t, int slot) {
    if (slot >= first + 32) {
      first = slot;
      const int i = slot + static_cast<int>(lane_id());
      id = i < t.adapters ? __ldcg(t.list + i) : 0;
    }
    return __shfl_sync(0xffffffffu, id, slot - first);
  }
};
// Likewise the row masks of QUADS * 128 rows; off(q) is the lane mask of rows
// 128 q .. of the tile: set where the row is not the adapter's.
template <int QUADS>
struct MaskWindow {
  int first = -32;
  uint4 on[QUADS];
  uint4 off[QUADS];
  __device__ __forceinline__ void load(const MultiTile &t, int slot) {
    if (slot >= first + 32) {
      first = slot;
      const int i = slot + static_cast<int>(lane_id());
#pragma unroll
      for (int q = 0; q < QUADS; ++q) on[q] = i < t.adapters ? __ldcg(t.mask + i * QUADS + q) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int l = slot - first;
#pragma unroll
    for (int q = 0; q < QUADS; ++q)
      off[q] = make_uint4(~__shfl_sync(0xffffffffu, on[q].x, l), ~__shfl_sync(0xffffffffu, on[q].y, l),
                          ~__shfl_sync(0xffffffffu, on[q].z, l), ~__shfl_sync(0xffffffffu, on[q].w, l));
  }
};
// The adapter steps [lo, hi) of this CTA of a cluster along z.
__device__ __forceinline__ void multi_share(int units, int per_step, int *lo, int *hi) {
  const int steps = (units + per_step - 1) / per_step;
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  *lo = static_cast<int>((static_cast<int64_t>(steps) * z) / nz);
  *hi = static_cast<int>((static_cast<int64_t>(steps) * (z + 1)) / nz);
}

}  // namespace qlora
