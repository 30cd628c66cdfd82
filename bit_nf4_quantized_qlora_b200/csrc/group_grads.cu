// Adapter gradients of many adapters, and from 8-bit activation checkpoints:
//
//   out_g = sum over the rows i of group g of  L[i, :]^T . R[i, :]
//
//   dA_a^T = X^T U    (L = X bf16 or its 8-bit checkpoint, R = U [m x r])
//   dB_a   = dY^T T   (L = dY, R = T [m x r])
//
// "QLoRA and Quantized Training", The idea: the adapters hold the gradients;
// "QLoRA", Training setup versus deployment setup: one frozen base serves
// several adapters, so a batch holds the rows of several.
//
// The contraction runs over a group's rows, wherever in the batch they are.
// group_rows_kernel writes each group's row numbers in ascending order, padded
// to whole steps of 64; a step whose rows are consecutive is one TMA box, any
// other is sixteen row-gathering TMA loads of four rows.  So the work is the
// rows themselves (plus the last step's padding), in every order of the batch,
// and a group never reads another group's rows.  The pad rows of the last
// step repeat one of the group's own rows and are zeroed in R's tile before
// the product.
//
// One CTA per (128 columns of L, 64 columns of R, group), the rows split over
// a cluster of up to 8 CTAs when the tiles alone cannot fill the SMs; fp32
// partials are added in rank order, so results do not depend on timing.  An
// M = 128, N = 64 product of K = 64 rows reads 16 KB of L: the kernel is
// bound by reading L once per 64 ranks (HBM, or L2 for r > 64).
//
// Checkpoint form: L's tile arrives as 64 x 128 codes (half the bytes); the
// four epilogue warps expand it to the bf16 tile the product reads, one block
// of 64 elements (one scale) per thread: two integer and half a packed
// floating-point instruction per element.
#include <cuda.h>

#include "act8.cuh"
#include "internal.h"
#include "multi.cuh"
#include "split_reduce.cuh"

namespace qlora {
namespace {

constexpr int kStep = 64;                 // rows of a step
constexpr int kThreads = 192;             // TMA warp, MMA warp, four expand / epilogue warps
constexpr uint32_t kLBytes = 128u * kStep * 2u;   // bf16 tile: two 64-column slabs
constexpr uint32_t kRBytes = 64u * kStep * 2u;
constexpr uint32_t kCBytes = 128u * kStep;        // code tile
constexpr uint32_t kPartLd = 64u + 4u;

template <bool ACT8>
constexpr int stages() { return ACT8 ? 3 : 4; }
template <bool ACT8>
constexpr uint32_t stage_bytes() { return kLBytes + kRBytes + (ACT8 ? kCBytes : 0u); }
template <bool ACT8>
constexpr uint32_t smem_bytes() { return stage_bytes<ACT8>() * stages<ACT8>() + 1024u; }
static_assert(2u * smem_bytes<false>() <= 227u * 1024u && 2u * smem_bytes<true>() <= 227u * 1024u, "two CTAs per SM");
static_assert(stage_bytes<true>() * stages<true>() >= 128u * kPartLd * 4u, "room for the fp32 partial tile");

struct __align__(64) GroupParams {
  CUtensorMap tmL, tmLg;        // L by boxes of 64 rows / by single rows
  CUtensorMap tmR, tmRg;        // R likewise
  const uint16_t *scale;        // checkpoint scales [m x P / 64]
  const int32_t *list;          // row lists (null: one group of all rows, in order)
  const int32_t *start, *count; // first entry (a multiple of 64) and rows of each group
  uint16_t *out;                // [groups x P x r], or [groups x r x P] transposed
  unsigned *err;
  int64_t P;
  int m, r, rtiles;
};

template <bool ACT8, bool OUT_T>
__global__ void __launch_bounds__(kThreads, 2) group_grads_kernel(const __grid_constant__ GroupParams p) {
  constexpr int kStages = stages<ACT8>();
  constexpr uint32_t kStageBytes = stage_bytes<ACT8>();
  constexpr uint32_t kIdesc = make_idesc(64, true, true);
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full[kStages], expanded[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ uint32_t tmem_slot;

  const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p_tile = static_cast<int>(blockIdx.x) / p.rtiles, r_tile = static_cast<int>(blockIdx.x) % p.rtiles;
  const int group = static_cast<int>(blockIdx.y);
  const int rows = p.list ? __ldg(p.count + group) : p.m;
  const int32_t *list = p.list ? p.list + __ldg(p.start + group) : nullptr;
  const int nsteps = (rows + kStep - 1) / kStep;
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  const int s_lo = static_cast<int>((static_cast<int64_t>(nsteps) * z) / nz);
  const int s_hi = static_cast<int>((static_cast<int64_t>(nsteps) * (z + 1)) / nz);
  const int n_iters = s_hi - s_lo;
  const int p0 = p_tile * 128, r0 = r_tile * 64;
  // Second 64-column slab; past P it repeats the first (its output rows are
  // never stored) and every copy stays in range.
  const int p1 = p0 + 64 < p.P ? p0 + 64 : p0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&expanded[s], 4);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(64u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int issued = 0;
    for (int li = 0; li < n_iters; ++li) {
      const int s = li % kStages;
      const uint32_t ph = static_cast<uint32_t>(li / kStages) & 1u;
      const int row0 = (s_lo + li) * kStep;
      // The step's rows, four per lane on lanes 0..15.
      int4 idx = make_int4(row0 + 4 * lane, row0 + 4 * lane + 1, row0 + 4 * lane + 2, row0 + 4 * lane + 3);
      int first = row0;
      bool box = true;
      if (list) {
        if (lane < 16) idx = __ldg(reinterpret_cast<const int4 *>(list + row0) + lane);
        first = __shfl_sync(0xffffffffu, idx.x, 0);
        const int want = first + 4 * lane;
        const bool in_order = idx.x == want && idx.y == want + 1 && idx.z == want + 2 && idx.w == want + 3;
        box = __all_sync(0xffffffffu, lane >= 16 || in_order) != 0;
      }
      int ok = 1;
      const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
      const uint32_t r_s = l_s + kLBytes, c_s = r_s + kRBytes;
      if (lane == 0) {
        ok = mbar_wait_bounded(&empty[s], ph ^ 1u, p.err, kErrTimeoutEmpty);
        if (ok) mbar_arrive_expect_tx(&full[s], (ACT8 ? kCBytes : kLBytes) + kRBytes);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (box) {
        if (lane == 0) {
          if (ACT8) {
            tma_load_2d(c_s, &p.tmL, &full[s], p0, first);
          } else {
            tma_load_2d(l_s, &p.tmL, &full[s], p0, first);
            tma_load_2d(l_s + 8192u, &p.tmL, &full[s], p1, first);
          }
          tma_load_2d(r_s, &p.tmR, &full[s], r0, first);
        }
      } else if (lane < 16) {
        const uint32_t row = static_cast<uint32_t>(lane) * 512u;   // four rows of 128 bytes
        if (ACT8) {
          tma_gather4(c_s + row, &p.tmLg, &full[s], p0, idx);
        } else {
          tma_gather4(l_s + row, &p.tmLg, &full[s], p0, idx);
          tma_gather4(l_s + 8192u + row, &p.tmLg, &full[s], p1, idx);
        }
        tma_gather4(r_s + row, &p.tmRg, &full[s], r0, idx);
      }
      ++issued;
    }
    __syncwarp();
    // Every issued copy has landed before the CTA may exit.
    if (lane == 0)
      for (int li = issued - kStages < 0 ? 0 : issued - kStages; li < issued; ++li)
        mbar_wait_bounded(&full[li % kStages], static_cast<uint32_t>(li / kStages) & 1u, p.err, kErrTimeoutDrain);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int ok = 1;
    for (int li = 0; li < n_iters; ++li) {
      const int s = li % kStages;
      const uint32_t ph = static_cast<uint32_t>(li / kStages) & 1u;
      const int valid = rows - (s_lo + li) * kStep;
      const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
      const uint32_t r_s = l_s + kLBytes;
      if (lane == 0) {
        ok = mbar_wait_bounded(&full[s], ph, p.err, kErrTimeoutFullA);
        if (ok && ACT8) ok = mbar_wait_bounded(&expanded[s], ph, p.err, kErrTimeoutFullB);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (list && valid < kStep) {
        // Pad rows of the last step: zero rows of R (whole 128-byte rows, so
        // the swizzle inside them does not matter).
        const uint32_t zero[4] = {0u, 0u, 0u, 0u};
        for (int c = valid * 8 + lane; c < kStep * 8; c += 32) sts128(r_s + static_cast<uint32_t>(c) * 16u, zero);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        tc_fence_after();
        const int chunks = valid >= kStep ? kStep / 16 : (valid + 15) / 16;
        for (int kk = 0; kk < chunks; ++kk)
          umma_f16(tmem, smem_desc(l_s + kk * 2048u, 8192u, 1024u), smem_desc(r_s + kk * 2048u, 8192u, 1024u), kIdesc,
                   (li > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (lane == 0 && ok) umma_commit(&acc_bar);
  } else {
    const int t = static_cast<int>(threadIdx.x) - 64;
    bool ok = true;
    if (ACT8) {
      // ---------------------------------------------------------- expand
      // Thread t: row t / 2 of the step, 64-column half t % 2.
      const int row = t >> 1, half = t & 1;
      const int64_t kb = p.P / 64, cb = static_cast<int64_t>(p_tile) * 2 + half;
      const uint32_t sw = static_cast<uint32_t>(row & 7);
      const auto row_of = [&](int step) -> int64_t {
        const int i = step * kStep + row;
        return list ? __ldg(list + i) : (i < p.m ? i : -1);
      };
      const auto scale_of = [&](int64_t gr) -> uint32_t {
        return (gr >= 0 && cb < kb) ? static_cast<uint32_t>(__ldg(p.scale + gr * kb + cb)) * 0x10001u : 0u;
      };
      // Row numbers two steps ahead, scales one step ahead.
      int64_t row_nx = n_iters > 1 ? row_of(s_lo + 1) : -1;
      uint32_t s_nx = n_iters > 0 ? scale_of(row_of(s_lo)) : 0u;
      for (int li = 0; li < n_iters; ++li) {
        const int s = li % kStages;
        const uint32_t ph = static_cast<uint32_t>(li / kStages) & 1u;
        const uint32_t s2 = s_nx;
        if (li + 1 < n_iters) s_nx = scale_of(row_nx);
        if (li + 2 < n_iters) row_nx = row_of(s_lo + li + 2);
        if (!mbar_wait_bounded(&full[s], ph, p.err, kErrTimeoutFullA)) { ok = false; break; }
        const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
        const uint32_t code_row = l_s + kLBytes + kRBytes + static_cast<uint32_t>(row) * 128u;
        const uint32_t out_row = l_s + static_cast<uint32_t>(half) * 8192u + static_cast<uint32_t>(row) * 128u;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          // 16 codes -> two 16-byte chunks; the halves walk them in an order
          // that keeps a quarter-warp's stores in distinct bank groups.
          const uint32_t j = static_cast<uint32_t>(jj ^ (2 * half));
          const uint4 c = lds128(code_row + (((4u * half + j) ^ sw) << 4));
          uint32_t o[4];
          act8_decode4(c.x, s2, o[0], o[1]);
          act8_decode4(c.y, s2, o[2], o[3]);
          sts128(out_row + (((2u * j) ^ sw) << 4), o);
          act8_decode4(c.z, s2, o[0], o[1]);
          act8_decode4(c.w, s2, o[2], o[3]);
          sts128(out_row + (((2u * j + 1u) ^ sw) << 4), o);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&expanded[s]);
      }
    }
    // ------------------------------------------------------------ epilogue
    // fp32 partial into the idle ring, along the output's contiguous dimension.
    if (ok) ok = mbar_wait_bounded(&acc_bar, 0u, p.err, kErrTimeoutAcc, 20000000000ull);
    if (ok) {
      tc_fence_after();
      const int quad = warp & 3;
      const uint32_t row = static_cast<uint32_t>(quad * 32 + lane);
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c0), v);
        if (!OUT_T) {
          const uint32_t dst = base + (row * kPartLd + static_cast<uint32_t>(c0)) * 4u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = n_iters > 0 ? v[4 * j + e] : 0u;
            sts128(dst + 16u * static_cast<uint32_t>(j), w);
          }
        } else {
          const uint32_t dst = base + (static_cast<uint32_t>(c0) * 128u + row) * 4u;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float val = n_iters > 0 ? __uint_as_float(v[j]) : 0.f;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(j) * 512u), "f"(val) : "memory");
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  uint16_t *out = p.out + static_cast<int64_t>(group) * p.P * p.r;
  split_reduce<64, kThreads, OUT_T>(base, kPartLd, out, OUT_T ? p.P : p.r, p.P, p.r, p0, r0, 1.0f);
  cluster_sync_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(64u) : "memory");
  }
}

// The rows of each adapter, ascending, one CTA per adapter.  Adapter a's list
// starts at entry 64 (floor(b / 64) + a), b the number of rows with a lower
// id: such a list of c entries padded to a multiple of 64 ends before adapter
// a + 1's starts, so no CTA needs another's count.  Warps take contiguous
// runs of rows and count by ballots; no atomics, so the order is fixed.
constexpr int kListThreads = 512;
__global__ void __launch_bounds__(kListThreads) group_rows_kernel(const int32_t *__restrict__ ids, int m,
                                                                  int32_t *__restrict__ start,
                                                                  int32_t *__restrict__ count,
                                                                  int32_t *__restrict__ list) {
  __shared__ int eq_of[kListThreads / 32], lt_of[kListThreads / 32];
  const int a = static_cast<int>(blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kListThreads / 32;
  const int64_t run = ((static_cast<int64_t>(m) + 32 * kWarps - 1) / (32 * kWarps)) * 32;   // rows per warp
  const int64_t lo = run * warp, hi = lo + run < m ? lo + run : m;
  int eq = 0, lt = 0;
#pragma unroll 4
  for (int64_t i = lo; i < hi; i += 32) {
    const int id = i + lane < hi ? __ldg(ids + i + lane) : -1;
    eq += __popc(__ballot_sync(0xffffffffu, id == a));
    lt += __popc(__ballot_sync(0xffffffffu, id >= 0 && id < a));
  }
  if (lane == 0) {
    eq_of[warp] = eq;
    lt_of[warp] = lt;
  }
  __syncthreads();
  int before = 0, total = 0, lower = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? eq_of[w] : 0;
    total += eq_of[w];
    lower += lt_of[w];
  }
  const int64_t first = 64 * (static_cast<int64_t>(lower / 64) + a);
  if (threadIdx.x == 0) {
    start[a] = static_cast<int32_t>(first);
    count[a] = total;
  }
  int32_t *dst = list + first;
  const int padded = (total + 63) / 64 * 64;
#pragma unroll 4
  for (int64_t i = lo; i < hi; i += 32) {
    const int id = i + lane < hi ? __ldg(ids + i + lane) : -1;
    const unsigned hit = __ballot_sync(0xffffffffu, id == a);
    if (id == a) {
      const int at = before + __popc(hit & ((1u << lane) - 1u));
      dst[at] = static_cast<int32_t>(i + lane);
      // The last row also fills the padding.
      if (at == total - 1)
        for (int j = total; j < padded; ++j) dst[j] = static_cast<int32_t>(i + lane);
    }
    before += __popc(hit);
  }
}

template <bool ACT8, bool OUT_T>
cudaError_t launch(const GroupParams &p, int ptiles, int groups, int split, cudaStream_t stream) {
  static std::atomic<bool> configured[kMaxDevicesPerProcess] = {};
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(group_grads_kernel<ACT8, OUT_T>),
                                static_cast<int>(smem_bytes<ACT8>()), configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ptiles * p.rtiles), static_cast<unsigned>(groups), static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<ACT8>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(split);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, group_grads_kernel<ACT8, OUT_T>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

GroupRows carve_group_rows(void *scratch, int64_t m, int32_t groups) {
  GroupRows g{};
  int32_t *base = static_cast<int32_t *>(scratch);
  g.groups = groups;
  g.start = base;
  g.count = base + groups;
  g.list = base + (2 * static_cast<int64_t>(groups) + 63) / 64 * 64;
  return g;
}

size_t group_rows_bytes(int64_t m, int32_t groups) {
  const size_t head = (2 * static_cast<size_t>(groups) + 63) / 64 * 64;
  return (head + 64 * (static_cast<size_t>(m) / 64 + static_cast<size_t>(groups))) * 4u;
}

cudaError_t launch_group_rows(const int32_t *ids, int64_t m, const GroupRows &g, cudaStream_t stream) {
  group_rows_kernel<<<static_cast<unsigned>(g.groups), kListThreads, 0, stream>>>(ids, static_cast<int>(m), g.start,
                                                                                  g.count, g.list);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_group_grads(const uint16_t *L, const Act8View *L8, int64_t m, int64_t P, const uint16_t *R,
                               int32_t r, const GroupRows *g, uint16_t *out, bool transposed, cudaStream_t stream) {
  GroupParams p{};
  const int64_t cols = P;
  if (L8) {
    const uint8_t *codes = reinterpret_cast<const uint8_t *>(L8->codes);
    if (!encode_codes_map(&p.tmL, codes, m, cols, 128, kStep, true)) return cudaErrorInvalidValue;
    if (!encode_codes_map(&p.tmLg, codes, m, cols, 128, 1, true)) return cudaErrorInvalidValue;
    p.scale = L8->scale;
  } else {
    if (!encode_bf16_map(&p.tmL, L, m, cols, 64, kStep)) return cudaErrorInvalidValue;
    if (!encode_bf16_map(&p.tmLg, L, m, cols, 64, 1)) return cudaErrorInvalidValue;
  }
  if (!encode_bf16_map(&p.tmR, R, m, r, 64, kStep)) return cudaErrorInvalidValue;
  if (!encode_bf16_map(&p.tmRg, R, m, r, 64, 1)) return cudaErrorInvalidValue;
  if (g) {
    p.list = g->list;
    p.start = g->start;
    p.count = g->count;
  }
  p.out = out;
  p.err = device_error_word();
  p.P = P;
  p.m = static_cast<int>(m);
  p.r = r;
  p.rtiles = (r + 63) / 64;
  const int groups = g ? g->groups : 1;
  const int ptiles = static_cast<int>((P + 127) / 128);
  // At most min(groups, m) groups have rows; the split fills about two CTAs
  // per SM with those.
  const int64_t busy = groups < m ? groups : m;
  const int steps = static_cast<int>((m + kStep - 1) / kStep);
  const int split = choose_split(static_cast<int64_t>(ptiles) * p.rtiles * busy, steps);
  if (L8) return launch<true, true>(p, ptiles, groups, split, stream);
  return transposed ? launch<false, true>(p, ptiles, groups, split, stream)
                    : launch<false, false>(p, ptiles, groups, split, stream);
}

}  // namespace qlora
