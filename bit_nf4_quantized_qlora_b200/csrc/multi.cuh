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

// 16 bytes of global memory into shared memory, asynchronously (`bytes` = 0:
// zeros), in the groups that cp_async_commit closes; cp_async_wait<N> leaves
// the N youngest groups in flight.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }


// A call's tile lists and adapters, as kernel parameters.
struct MultiParams {
  const int32_t *lists;
  int64_t stride;
  int32_t slots, rows;
  int32_t r, width;
  const uint16_t *A, *B;    // [count x r x k], [count x n x r]
};
inline MultiParams multi_params(const AdapterView &ad, const TileLists &l) {
  return MultiParams{l.base, l.stride, l.slots, l.rows, ad.r, unit_width(ad.r), ad.A, ad.B};
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
// loop may), takes the list and passes its adapters to `prefetch`, whose rows
// are in L2 when the main loop ends.  Reads past L1: the lists were written
// while this kernel ran.
template <int QUADS, class Prefetch>
__device__ __forceinline__ void multi_scout(const MultiParams &p, int tile, MultiListSmem<QUADS> &s,
                                            const Prefetch &prefetch) {
  griddep_wait();
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
  for (int i = lane; i < n; i += 32) prefetch(__ldcg(t + 4 + i));
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

// A warp's window on the list, so that the latency of a list read is paid once
// per 32 adapters: entry first + i is in lane i.  Called by whole warps.
struct AdapterWindow {
  int first = -32, id = 0;
  __device__ __forceinline__ int at(const MultiTile &t, int slot) {
    if (slot < first || slot >= first + 32) {
      first = slot & ~31;
      const int i = first + static_cast<int>(lane_id());
      id = i >= t.adapters ? 0 : i < kListEntries ? t.id_smem[i] : __ldcg(t.list + i);
    }
    return __shfl_sync(0xffffffffu, id, slot - first);
  }
};
// Likewise the row masks; off[q] is the lane mask of rows 128 q .. of the
// tile: set where the row is not the adapter's.
template <int QUADS>
struct MaskWindow {
  int first = -32, current = -1;
  uint4 on[QUADS];
  uint4 off[QUADS];
  __device__ __forceinline__ void load(const MultiTile &t, int slot) {
    if (slot == current) return;
    current = slot;
    if (slot < first || slot >= first + 32) {
      first = slot & ~31;
      const int i = first + static_cast<int>(lane_id());
#pragma unroll
      for (int q = 0; q < QUADS; ++q)
        on[q] = i >= t.adapters ? make_uint4(0u, 0u, 0u, 0u)
                : i < kListEntries ? t.mask_smem[i * QUADS + q]
                                   : __ldcg(t.mask + i * QUADS + q);
    }
    const int l = slot - first;
#pragma unroll
    for (int q = 0; q < QUADS; ++q)
      off[q] = make_uint4(~__shfl_sync(0xffffffffu, on[q].x, l), ~__shfl_sync(0xffffffffu, on[q].y, l),
                          ~__shfl_sync(0xffffffffu, on[q].z, l), ~__shfl_sync(0xffffffffu, on[q].w, l));
  }
};

// `bytes` (a multiple of 16) at `src` into L2.
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// An adapter's part of an output tile: rows [c0, c0 + cols) of B_a (forward),
// or columns [c0, c0 + cols) of A_a's r rows.
__device__ __forceinline__ void prefetch_adapter(const MultiParams &p, bool bwd, int64_t a, int64_t c0, int cols,
                                                 int64_t out_cols) {
  const int64_t left = out_cols - c0;
  if (left <= 0) return;
  const uint32_t c = static_cast<uint32_t>(left < cols ? left : cols);
  if (!bwd) {
    prefetch_l2(p.B + (a * out_cols + c0) * p.r, c * static_cast<uint32_t>(p.r) * 2u);
  } else {
    for (int j = 0; j < p.r; ++j) prefetch_l2(p.A + (a * p.r + j) * out_cols + c0, c * 2u);
  }
}

// The adapter k-steps of a tile, block by block of the rank: every full
// 64-column block has one step per adapter, the last partial block packs
// 64 / width units into each.  A walk over them keeps its place in counters:
// the warps that issue products have one instruction in flight at a time, and a
// division would cost them as much as a step's products.
struct MultiSteps {
  int adapters, full, rest;            // full 64-column blocks; columns of the partial one
  int lw;                              // log2 of the unit width
  int per_step;                        // 64 / width
  __device__ __forceinline__ MultiSteps(const MultiParams &p, const MultiTile &t)
      : adapters(t.adapters), full(p.r >> 6), rest(p.r & 63), lw(p.width == 64 ? 6 : p.width == 32 ? 5 : 4),
        per_step(64 >> lw) {}
  __device__ __forceinline__ int count() const { return full * adapters + ((adapters * rest + 63) >> 6); }
  // This CTA's share [lo, hi) along a cluster's z.
  __device__ __forceinline__ void share(int *lo, int *hi) const {
    const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
    *lo = static_cast<int>((static_cast<int64_t>(count()) * z) / nz);
    *hi = static_cast<int>((static_cast<int64_t>(count()) * (z + 1)) / nz);
  }
};
struct MultiStep {
  int block, units, per_adapter;          // rank block; units of the step, units of an adapter in the block
  int slot, sub;                          // adapter and unit of the step's first
  int left;                               // units of the block from this step on
  int since;                              // steps of the walk in this block
  // The step `st` of a walk that starts there.
  __device__ __forceinline__ MultiStep(const MultiSteps &s, int st) {
    const int in_full = s.full * s.adapters;
    block = 0;
    int at = st;
    while (block < s.full && at >= s.adapters && s.adapters > 0) {
      at -= s.adapters;
      ++block;
    }
    if (st >= in_full) block = s.full;
    open(s);
    sub += at * s.per_step;
    left -= sub;
    slot = sub / per_adapter;
    sub -= slot * per_adapter;
    units = left < s.per_step ? left : s.per_step;
  }
  __device__ __forceinline__ void open(const MultiSteps &s) {
    per_adapter = block < s.full ? s.per_step : (s.rest >> s.lw);
    if (per_adapter == 0) per_adapter = 1;       // past the last block
    left = s.adapters * per_adapter;
    slot = sub = since = 0;
    units = left < s.per_step ? left : s.per_step;
  }
  // To the walk's next step.
  __device__ __forceinline__ void next(const MultiSteps &s) {
    left -= units;
    ++since;
    if (left == 0) {
      ++block;
      open(s);
      return;
    }
    sub += units;
    while (sub >= per_adapter) {
      sub -= per_adapter;
      ++slot;
    }
    units = left < s.per_step ? left : s.per_step;
  }
  // To the step's next unit (of a copy).
  __device__ __forceinline__ void advance() {
    if (++sub == per_adapter) {
      sub = 0;
      ++slot;
    }
  }
};

// A thread's part of a step's K-major adapter tile [ROWS x 64], ROWS threads:
// 8 pieces of 16 bytes, taken from the matrices B_a [n x r] of the step's
// adapters and stored as 64 / w units of ROWS rows under the unit's swizzle.
// Plain loads, consecutive lanes on consecutive bytes: a unit row of 32 or 64
// bytes would cost the copy engine as much as one of 128 (bulk copies of whole
// adapters put in order in shared memory, and boxes for the 128-byte rows, took
// the same time).
template <int ROWS>
struct MultiRows {
  uint4 v[8];
  template <int W, class Window>
  __device__ __forceinline__ void load_w(const MultiParams &p, MultiStep s, Window &win, const MultiTile &t, int64_t n,
                                         int64_t n0, int thread) {
    constexpr int kPieces = W / 8;      // of a unit row
#pragma unroll
    for (int u = 0; u < 64 / W; ++u) {
      const int a = u < s.units ? win.at(t, s.slot) : 0;
      const uint16_t *src = p.B + (a * n + n0) * p.r + s.block * 64 + s.sub * W;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const int j = c * ROWS + thread, row = j / kPieces;
        v[u * kPieces + c] = u < s.units && n0 + row < n
                                 ? __ldg(reinterpret_cast<const uint4 *>(src + row * p.r) + j % kPieces)
                                 : make_uint4(0u, 0u, 0u, 0u);
      }
      s.advance();
    }
  }
  template <class Window>
  __device__ __forceinline__ void load(const MultiParams &p, const MultiStep &s, Window &win, const MultiTile &t,
                                       int64_t n, int64_t n0, int thread) {
    if (p.width == 16)
      load_w<16>(p, s, win, t, n, n0, thread);
    else if (p.width == 32)
      load_w<32>(p, s, win, t, n, n0, thread);
    else
      load_w<64>(p, s, win, t, n, n0, thread);
  }
  template <int W>
  __device__ __forceinline__ void store_w(uint32_t tile, int thread) const {
    constexpr int kPieces = W / 8;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int j = (q % kPieces) * ROWS + thread, row = j / kPieces;
      const int sw = (row >> (W == 64 ? 0 : W == 32 ? 1 : 2)) & (kPieces - 1);
      const uint32_t o[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      sts128(tile + static_cast<uint32_t>(((q / kPieces) * ROWS + row) * W * 2 + (((j % kPieces) ^ sw) << 4)), o);
    }
  }
  __device__ __forceinline__ void store(const MultiParams &p, uint32_t tile, int thread) const {
    if (p.width == 16)
      store_w<16>(tile, thread);
    else if (p.width == 32)
      store_w<32>(tile, thread);
    else
      store_w<64>(tile, thread);
  }
};

}  // namespace qlora
