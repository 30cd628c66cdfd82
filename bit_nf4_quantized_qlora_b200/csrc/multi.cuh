// Device helpers of the many-adapter kernels (sm_100a): masked tcgen05
// products, row-gathering TMA loads, operand descriptors for narrow tiles.
//
// Rows of a batch belong to different adapters.  A product that adds one
// adapter's low-rank term to a tile runs over all of the tile's rows with the
// lanes of the other rows disabled (tcgen05.mma's disable-output-lane mask:
// lane i of the accumulator is row i of the tile), so the rank-r operand needs
// no zero-filled copies and a row never meets another adapter's values.
//
// The rank dimension is cut into units of 64, 32 or 16 columns (the widest
// that divides r): a unit is one adapter's slice of that width, and units that
// lie in the same 64-column block of the rank share a 64-wide k-step.  The
// rank-r operand (T or U) of a block is one [rows x 64] tile that stays in
// shared memory for all of the block's steps.  A unit of a K-major adapter
// matrix is a tile with rows of 128, 64 or 32 bytes under the swizzle of that
// width, in atoms of 8 rows.
//
// The main kernels overlap the projection that makes T or U (multi_proj.cu):
// they need it only after their main loop.  Back to back, 128 x 8192 -> 28672
// takes 106 us with no adapter in the batch, 108 with one of rank 16, 113 with
// 16 and 126 with 64: 16 steps of four 16-column units, 1.25 us each, where a
// main k-step takes 0.8.  1111 x 11008 -> 4096, r = 64, in any order: 135 with
// none, 140 with one, 152 with 16 and 201 with 64, the projection of that many
// adapters included (a main k-step of a 512-row tile takes 0.75).
#pragma once

#include <type_traits>

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

// 16 accumulator columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// One lane of a converged warp, the same at every call.  Copies and products
// are issued under it: a masked product took 600 cycles to issue under a test
// of the lane's number and 100 under this.
__device__ __forceinline__ bool elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0u;
}

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A call's tile lists and adapters, as kernel parameters.
struct MultiParams {
  const int32_t *lists;
  int64_t stride;
  int32_t slots;
  int32_t r, width;
  const uint16_t *A, *B;    // [count x r x k], [count x n x r]
};
inline MultiParams multi_params(const AdapterView &ad, const TileLists &l) {
  return MultiParams{l.base, l.stride, l.slots, ad.r, unit_width(ad.r), ad.A, ad.B};
}

// One tile's list: its first entries (adapter ids and the masks of QUADS * 128
// rows) in shared memory, as many as the kernels have room for, the rest where
// the projection wrote them.
constexpr int kListEntries = 24;
template <int QUADS>
struct MultiListSmem {
  uint64_t ready;
  int adapters, pad;
  int id[kListEntries];
  uint4 mask[kListEntries * QUADS];
};
struct MultiTile {
  const int32_t *list;
  const uint4 *mask;
  const int *id_smem;
  const uint4 *mask_smem;
  int adapters;
};
__device__ __forceinline__ const int32_t *multi_tile_at(const MultiParams &p, int tile) {
  return p.lists + tile * p.stride;
}

// The warp of a kernel that overlaps the projection, for all of its others:
// waits for the projection (which stops a whole warp, so no warp of the main
// loop may), lets the adapter gradients start, which need the projection but not
// this kernel's product, and takes the list.  Reads past L1: it was written while
// this kernel ran.
template <int QUADS>
__device__ __forceinline__ void multi_scout(const MultiParams &p, int tile, MultiListSmem<QUADS> &s) {
  griddep_wait();
  griddep_launch();
  const int32_t *t = multi_tile_at(p, tile);
  const uint4 *mask = reinterpret_cast<const uint4 *>(t + 4 + p.slots);
  const int lane = static_cast<int>(lane_id()), n = __ldcg(t);
  if (lane < p.slots && lane < kListEntries) {
    s.id[lane] = __ldcg(t + 4 + lane);
#pragma unroll
    for (int q = 0; q < QUADS; ++q) s.mask[lane * QUADS + q] = __ldcg(mask + lane * QUADS + q);
  }
  if (lane == 0) s.adapters = n;
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.ready);
}
// The list in one of the other warps; false if the wait for it ran out.
template <int QUADS>
__device__ __forceinline__ bool multi_open(const MultiParams &p, int tile, MultiListSmem<QUADS> &s, unsigned *err,
                                           MultiTile *out) {
  __syncwarp();
  if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s.ready, 0u, err, kErrTimeoutFullA))) return false;
  const int32_t *t = multi_tile_at(p, tile);
  *out = MultiTile{t + 4, reinterpret_cast<const uint4 *>(t + 4 + p.slots), s.id, s.mask, s.adapters};
  return true;
}

// The adapter k-steps of a tile, block by block of the rank: every full
// 64-column block has one step per adapter, the last partial block packs
// 64 / w units into each.  Units are numbered in that order, so unit g is part
// g % (64 / w) of step g / (64 / w).
struct MultiSteps {
  int adapters, full, rest;            // full 64-column blocks; units of an adapter in the partial one
  int lw, lp;                          // log2 of the unit width; of the units of a step
  int units;
  __device__ __forceinline__ MultiSteps(const MultiParams &p, const MultiTile &t)
      : adapters(t.adapters), full(p.r >> 6), lw(p.width == 64 ? 6 : p.width == 32 ? 5 : 4), lp(6 - lw) {
    rest = (p.r & 63) >> lw;
    units = t.adapters * (p.r >> lw);
  }
  __device__ __forceinline__ int count() const { return (units + (1 << lp) - 1) >> lp; }
  __device__ __forceinline__ int units_of(int step) const {
    const int left = units - (step << lp);
    return left < 1 << lp ? left : 1 << lp;
  }
  // Steps of the walk that starts at `lo` before `step` in its rank block.
  __device__ __forceinline__ int since(int step, int lo) const {
    int first = step < full * adapters ? step - step % adapters : full * adapters;
    return step - (first < lo ? lo : first);
  }
  // This CTA's share [lo, hi) along a cluster's z.
  __device__ __forceinline__ void share(int *lo, int *hi) const {
    const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
    *lo = static_cast<int>((static_cast<int64_t>(count()) * z) / nz);
    *hi = static_cast<int>((static_cast<int64_t>(count()) * (z + 1)) / nz);
  }
};

// A warp's window of 32 units: unit first + i is worked out by lane i.  The
// warps that issue copies and products run one instruction chain each, and a
// walk through the units with its divisions and list reads took them three
// times a main loop's k-step; a window's 32 units cost about as much as one.
struct UnitWindow {
  int first = -32, slot = 0, id = 0, col = 0;      // list entry, adapter, rank column
  // Whole warps; true if the window moved to unit g.
  __device__ __forceinline__ bool move(const MultiTile &t, const MultiSteps &s, int g) {
    if ((g & ~31) == first) return false;
    first = g & ~31;
    const int i = first + static_cast<int>(lane_id()), in_full = (s.full * s.adapters) << s.lp;
    int block, sub;
    if (i < in_full) {
      const int step = i >> s.lp;
      block = step / s.adapters;
      slot = step - block * s.adapters;
      sub = i & ((1 << s.lp) - 1);
    } else {
      const int per = s.rest > 0 ? s.rest : 1;
      block = s.full;
      slot = (i - in_full) / per;
      sub = i - in_full - slot * per;
    }
    if (i >= s.units) slot = 0;
    id = slot < kListEntries ? t.id_smem[slot] : __ldcg(t.list + slot);
    col = block * 64 + (sub << s.lw);
    return true;
  }
  __device__ __forceinline__ int id_of(int g) const { return __shfl_sync(0xffffffffu, id, g & 31); }
  __device__ __forceinline__ int col_of(int g) const { return __shfl_sync(0xffffffffu, col, g & 31); }
};
// With the lane masks of QUADS * 128 rows: off[q] of rows 128 q .. of the
// tile, set where the row is not the unit's adapter's.
template <int QUADS>
struct MaskWindow : UnitWindow {
  uint4 all[QUADS], off[QUADS];
  __device__ __forceinline__ void take(const MultiTile &t, const MultiSteps &s, int g) {
    if (move(t, s, g)) {
#pragma unroll
      for (int q = 0; q < QUADS; ++q) {
        const uint4 on = slot < kListEntries ? t.mask_smem[slot * QUADS + q] : __ldcg(t.mask + slot * QUADS + q);
        all[q] = make_uint4(~on.x, ~on.y, ~on.z, ~on.w);
      }
    }
#pragma unroll
    for (int q = 0; q < QUADS; ++q)
      off[q] = make_uint4(__shfl_sync(0xffffffffu, all[q].x, g & 31), __shfl_sync(0xffffffffu, all[q].y, g & 31),
                          __shfl_sync(0xffffffffu, all[q].z, g & 31), __shfl_sync(0xffffffffu, all[q].w, g & 31));
  }
};

// f(integral_constant<int, unit width>).
template <class F>
__device__ __forceinline__ void by_width(int width, const F &f) {
  if (width == 16)
    f(std::integral_constant<int, 16>{});
  else if (width == 32)
    f(std::integral_constant<int, 32>{});
  else
    f(std::integral_constant<int, 64>{});
}

// A thread's part of a step's K-major adapter tile [ROWS x 64], ROWS threads:
// 8 pieces of 16 bytes, taken from the matrices B_a [n x r] of the step's
// units of W columns and stored as 64 / W tiles of ROWS rows under the
// swizzle of their width.  Plain loads, consecutive lanes on consecutive
// bytes: a unit row of 32 or 64 bytes would cost the copy engine as much as
// one of 128.  Rows past n and units past the step's keep what the registers
// held; they meet no stored column and no product.
template <int ROWS, int W>
struct MultiRows {
  static constexpr int kPieces = W / 8;             // of a unit row
  static constexpr int kRowStep = ROWS / kPieces;   // rows between a thread's pieces (a multiple of 8)
  UnitWindow win;
  const uint16_t *src = nullptr;                    // the lane's unit, from row n0
  uint32_t dst;                                     // of piece 0 in the tile; piece q follows at 16 ROWS q
  int row, left, r;
  uint4 v[8];
  __device__ __forceinline__ MultiRows(const MultiParams &p, int64_t n, int64_t n0, int thread)
      : row(thread / kPieces), left(n - n0 < ROWS ? static_cast<int>(n - n0) : ROWS), r(p.r) {
    const int piece = thread % kPieces, sw = (row >> (W == 64 ? 0 : W == 32 ? 1 : 2)) & (kPieces - 1);
    dst = static_cast<uint32_t>(row * W * 2 + ((piece ^ sw) << 4));
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load(const MultiParams &p, const MultiTile &t, const MultiSteps &s, int step,
                                       int64_t n, int64_t n0, int thread) {
    const int g = step * (64 / W), units = s.units_of(step);
    if (win.move(t, s, g)) src = p.B + (win.id * n + n0) * r + win.col;
    const int mine = row * r + (thread % kPieces) * 8;
#pragma unroll
    for (int u = 0; u < 64 / W; ++u) {
      const uint16_t *from =
          reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), (g + u) & 31)) +
          mine;
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        if (u < units && row + c * kRowStep < left)
          v[u * kPieces + c] = __ldg(reinterpret_cast<const uint4 *>(from + c * kRowStep * r));
    }
  }
  __device__ __forceinline__ void store(uint32_t tile) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t o[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      sts128(tile + dst + static_cast<uint32_t>(q) * (16u * ROWS), o);
    }
  }
};

}  // namespace qlora
