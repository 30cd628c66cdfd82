// Reduction of a cluster's fp32 partial tiles through distributed shared
// memory (the split-K products).
#pragma once

#include "tcgen05.cuh"

namespace qlora {

// 16 bytes (four fp32) at the same offset in CTA `rank`'s shared memory;
// local_addr must be 16-byte aligned.
__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t local_addr, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_addr), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}

// Adds the cluster's partial tiles (128 rows x BN columns, at shared address
// `base` in every CTA; row-major with rows of part_ld fp32, or 128 fp32 per
// column for a transposed output) and writes bf16(alpha . sum) to
// out[row0 + row][col0 + col] (or transposed).  CTA `rank` finishes a share of
// the tile's rows that exist in the output (in whole groups of four rows for a
// transposed output).  Called by all THREADS threads between two cluster
// barriers.
template <int BN, int THREADS, bool OUT_T>
__device__ __forceinline__ void split_reduce(uint32_t base, uint32_t part_ld, uint16_t *out, int64_t out_ld,
                                             int64_t out_rows, int64_t out_cols, int64_t row0, int64_t col0,
                                             float alpha) {
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t left = out_rows - row0;
  const uint32_t valid = static_cast<uint32_t>(left < 128 ? (left > 0 ? left : 0) : 128);
  const uint32_t units = OUT_T ? (valid + 3u) / 4u : valid;
  const int u_lo = static_cast<int>((units * rank) / size), u_hi = static_cast<int>((units * (rank + 1)) / size);
  const int nu = u_hi - u_lo;
  // Work items are 16-byte pieces along the partial's contiguous dimension:
  // (row, 4 columns) for a row-major output, (column, 4 rows) for a
  // transposed one; consecutive threads take consecutive pieces, so the
  // remote reads and the bf16 stores are contiguous.  A thread takes kBatch
  // pieces at a time and issues all their peer loads (up to 8 peers) before
  // the first add, so the remote-load latency is paid once per batch; each
  // piece's partials are added in peer order.
  constexpr int kBatch = THREADS > 256 ? 1 : 2;   // 32 registers of partials per piece
  constexpr int kPieces = BN / 4;                 // pieces per row (row-major output)
  const int nel = OUT_T ? nu * BN : nu * kPieces;
  const bool vec_ok = (out_ld & 3) == 0 && (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
  for (int i0 = threadIdx.x; i0 < nel; i0 += kBatch * THREADS) {
    float4 part[kBatch][8];
    int row[kBatch], col[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * THREADS;
      const bool live = i < nel;
      const int ii = live ? i : 0;
      uint32_t off;
      if (!OUT_T) {
        row[b] = u_lo + ii / kPieces;
        col[b] = 4 * (ii % kPieces);
        off = base + (static_cast<uint32_t>(row[b]) * part_ld + static_cast<uint32_t>(col[b])) * 4u;
      } else {
        row[b] = 4 * (u_lo + ii % nu);
        col[b] = ii / nu;
        off = base + (static_cast<uint32_t>(col[b]) * 128u + static_cast<uint32_t>(row[b])) * 4u;
      }
      if (!live) col[b] = -1;
#pragma unroll
      for (int pr = 0; pr < 8; ++pr)
        part[b][pr] = (live && static_cast<uint32_t>(pr) < size) ? ld_dsmem_v4(off, static_cast<uint32_t>(pr))
                                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (col[b] < 0) continue;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int pr = 0; pr < 8; ++pr) {
        if (static_cast<uint32_t>(pr) < size) {
          acc.x += part[b][pr].x;
          acc.y += part[b][pr].y;
          acc.z += part[b][pr].z;
          acc.w += part[b][pr].w;
        }
      }
      const int64_t grow = row0 + row[b];
      const int64_t gcol = col0 + col[b];
      const uint32_t h01 = pack_bf16x2(acc.x * alpha, acc.y * alpha);
      const uint32_t h23 = pack_bf16x2(acc.z * alpha, acc.w * alpha);
      const uint16_t h[4] = {static_cast<uint16_t>(h01 & 0xFFFFu), static_cast<uint16_t>(h01 >> 16),
                             static_cast<uint16_t>(h23 & 0xFFFFu), static_cast<uint16_t>(h23 >> 16)};
      if (!OUT_T) {
        // Row grow, columns gcol .. gcol + 3.
        if (grow >= out_rows) continue;
        if (vec_ok && gcol + 4 <= out_cols) {
          *reinterpret_cast<uint2 *>(out + grow * out_ld + gcol) = make_uint2(h01, h23);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (gcol + e < out_cols) out[grow * out_ld + gcol + e] = h[e];
        }
      } else {
        // Column gcol of the tile = row gcol of the transposed output, its
        // entries grow .. grow + 3.
        if (gcol >= out_cols) continue;
        if (vec_ok && grow + 4 <= out_rows) {
          *reinterpret_cast<uint2 *>(out + gcol * out_ld + grow) = make_uint2(h01, h23);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (grow + e < out_rows) out[gcol * out_ld + grow + e] = h[e];
        }
      }
    }
  }
}

}  // namespace qlora
