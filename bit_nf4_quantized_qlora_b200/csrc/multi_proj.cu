// Rank-r projections of a batch whose rows belong to different adapters:
//
//   T[i, :] = bf16(s_a . X[i, :] . A_a^T)      (A [count x r x k], K-major)
//   U[i, :] = bf16(s_a . dY[i, :] . B_a)       (B [count x n x r], r contiguous)
//
// with a = ids[i]; a row whose id is outside [0, count) gets zeros (from
// multi_lists.cu).  "QLoRA", Training setup versus deployment setup: the
// quantized base is served with the adapter, and one base serves several;
// "QLoRA and Quantized Training", In code: r and alpha.
//
// The sums are fp32; T and U are rounded to bf16 once, because the products that
// take them are bf16 tensor-core products (with A_a, B_a, X and dY) and the
// one-adapter layer rounds them there too.  Where the adapter term is of the base
// product's size dX and dA are then off by up to 0.0024 (rms, relative), for 0.0017
// of their own rounding alone; two bf16 parts would double the adapter steps.
//
// tcgen05 path (multi_proj_kernel).  A CTA takes a slot of up to 64 rows of one
// adapter, wherever in the batch they lie: one TMA box per k-step when they are
// consecutive, row-gathering loads of four rows otherwise, and only as many as
// the slot holds.  So a batch in any order costs its rows and one reading of
// each adapter per 64 of them.  (Tiles of 128 consecutive rows against all
// adapters that occur in them, up to 256 rank columns a pass, took 37 us for
// 2000 x 4096 through 32 rank-16 adapters in any order and 181 us for
// 1111 x 11008 through 64 rank-64 ones.)  K is split over a cluster of up to 8
// CTAs whose fp32 partials are added in rank order through distributed shared
// memory; two CTAs share an SM for r <= 64.  A stage holds 128 columns: a warp
// takes about 230 cycles for the waits and the loop around a stage and 50 for
// every copy it issues, so with stages of 64 columns and one issuing warp the
// slots with gathered rows took 1100 cycles each; the idle epilogue warps issue
// the gathers.  Bound by reading X and the adapters present (HBM / L2), at small
// sizes by the latency of a slot's chain.
//
// Decode path (multi_proj_small_kernel, m <= 16): a CTA per (adapter row,
// token), a plain dot product: the tokens' adapters are mostly distinct, so
// each byte of A is used once and the kernel is bound by its latency.
#include <cuda.h>

#include "group_rows.cuh"
#include "internal.h"
#include "multi.cuh"
#include "split_reduce.cuh"

namespace qlora {
namespace {

constexpr int kBK = 64;                           // columns of a copy; a stage holds two
constexpr int kMaxStages = 8;
// TMA warp, MMA warp, four gather / epilogue warps.
constexpr int kThreads = 192;
constexpr uint32_t kABytes = static_cast<uint32_t>(kSlotRows) * kBK * 2u;   // 8 KB, half a stage's
constexpr uint32_t kColBytes = kBK * 2u;          // shared memory of one rank column of a copy
constexpr uint32_t kTmemCols = 256;               // r <= 256
// One CTA to an SM, or two with half the ring each for ranks up to 64, where a
// half still holds three stages (backward of 2000 x 4096, r = 16, 32 adapters:
// 93 us with two and 96 with one; of 4096 x 11008, r = 128, 8 adapters: 403
// with two of two stages and 400 with one of four).
constexpr uint32_t kRing = 200u * 1024u;
constexpr int kSharedRank = 64;
constexpr int stages_of(int r, int per_sm) {
  const int s = static_cast<int>(kRing / static_cast<uint32_t>(per_sm) / (2u * (kABytes + static_cast<uint32_t>(r) * kColBytes)));
  return s < kMaxStages ? s : kMaxStages;
}
static_assert(stages_of(kSharedRank, 2) >= 2 && stages_of(256, 1) >= 2, "two stages");
// A product reads 128 rows of A, 64 of them past the slot's: the last ones lie
// in the adapter tiles behind, and those accumulator rows are not read.
static_assert(static_cast<uint32_t>(stages_of(16, 2)) * 32u * kColBytes >= kABytes, "the second half stays inside the ring");
static_assert(kRing / 2u >= kSlotRows * (kSharedRank + 4u) * 4u && kRing >= kSlotRows * (256u + 4u) * 4u,
              "room for the fp32 partial tile");

struct __align__(64) ProjParams {
  CUtensorMap tmL, tmLg;  // X or dY [m x kc] by boxes of 64 rows / by single rows
  CUtensorMap tmR;        // A {kc, r, count} box {64, w, 1}; B {r, kc, count} box {w, 64, 1}
  RowSlots rows;
  const float *scale;
  uint16_t *out;          // [m x r]
  unsigned *err;
  int r, width, nk, stages;
};

// R_MN: R is [count x kc x r] (MN-major operand); else [count x r x kc].
template <bool R_MN>
__global__ void __launch_bounds__(kThreads) multi_proj_kernel(const __grid_constant__ ProjParams p) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int4 gather[4][kSlotRows / 4];

  // The kernel that consumes the output may start now; it waits for this
  // grid before it reads the output or the lists.
  griddep_launch();
  const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k_lo = static_cast<int>((static_cast<int64_t>(p.nk) * z) / nz);
  const int k_hi = static_cast<int>((static_cast<int64_t>(p.nk) * (z + 1)) / nz);
  const int steps = (k_hi - k_lo + 1) / 2;          // stages; the last may hold one copy's columns

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const int w = p.width, units = p.r / w;
  const uint32_t unit_bytes = static_cast<uint32_t>(w) * kColBytes;
  const uint32_t b_bytes = static_cast<uint32_t>(p.r) * kColBytes;                 // half a stage's
  const uint32_t b_ring = base + static_cast<uint32_t>(p.stages) * 2u * kABytes;
  const uint32_t part_ld = static_cast<uint32_t>(p.r) + 4u;
  int ring = 0;                 // next stage and its parity
  uint32_t parity = 0u;
  int issued = 0;               // stages whose copies were issued (producer)
  bool ok = true;
  uint32_t acc_phase = 0u;
  const auto advance = [&]() {
    if (++ring == p.stages) {
      ring = 0;
      parity ^= 1u;
    }
  };

  // The cluster's share of the slots.
  griddep_wait();
  const int slots = slot_count(p.rows);
  SlotWalk walk(p.rows, static_cast<int>(static_cast<int64_t>(slots) * blockIdx.x / gridDim.x),
                static_cast<int>(static_cast<int64_t>(slots) * (blockIdx.x + 1) / gridDim.x));
  for (int slot = walk.next(); slot >= 0; slot = walk.next()) {
    const int a = walk.part.group, left = walk.part.rows - (slot - walk.part.s) * kSlotRows;
    const int valid = left < kSlotRows ? left : kSlotRows;
    const int32_t *list = p.rows.list + static_cast<int64_t>(slot) * kSlotRows;
    // Consecutive rows come as boxes, others four at a time.
    const int4 idx = __ldcg(reinterpret_cast<const int4 *>(list) + (lane & 15));
    const int first = __shfl_sync(0xffffffffu, idx.x, 0), want = first + 4 * (lane & 15);
    const bool box = __all_sync(0xffffffffu, idx.x == want && idx.y == want + 1 && idx.z == want + 2 && idx.w == want + 3);
    const int fours = (valid + 3) / 4;
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      for (int j = 0; j < steps && ok; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[ring], parity ^ 1u, p.err, kErrTimeoutEmpty));
        if (!ok) break;
        if (elect_lane()) {
          const int kb = k_lo + 2 * j, halves = kb + 1 < k_hi ? 2 : 1;
          uint32_t a_s = base + static_cast<uint32_t>(ring) * 2u * kABytes;
          uint32_t b_s = b_ring + static_cast<uint32_t>(ring) * 2u * b_bytes;
          mbar_arrive_expect_tx(&full[ring], static_cast<uint32_t>(halves) *
                                                 ((box ? kABytes : static_cast<uint32_t>(fours) * 512u) + b_bytes));
          for (int h = 0; h < halves; ++h, a_s += kABytes) {
            const int kx = (kb + h) * kBK;
            if (box) tma_load_2d(a_s, &p.tmL, &full[ring], kx, first);
            for (int u = 0; u < units; ++u, b_s += unit_bytes) {
              if (R_MN)
                tma_load_3d(b_s, &p.tmR, &full[ring], u * w, kx, a);
              else
                tma_load_3d(b_s, &p.tmR, &full[ring], kx, u * w, a);
            }
          }
        }
        ++issued;
        advance();
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (ok) {
        // What a stage does not change is kept in registers: descriptors
        // advance by additions (16-byte units).
        const uint32_t idesc = make_idesc(p.r, false, R_MN);
        const uint64_t ad0 = smem_desc(base, 16u, 1024u);
        // MN-major units: [64 k-rows x w columns], one behind the other.
        const uint64_t bd0 = R_MN ? smem_desc_unit(b_ring, unit_bytes, static_cast<uint32_t>(16 * w), w)
                                  : smem_desc(b_ring, 16u, 1024u);
        const uint32_t b_step = R_MN ? static_cast<uint32_t>(2 * w) : 2u;
        for (int j = 0; j < steps; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[ring], parity, p.err, kErrTimeoutFullA));
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            uint64_t ad = ad0 + static_cast<uint32_t>(ring) * (2u * kABytes >> 4);
            uint64_t bd = bd0 + static_cast<uint32_t>(ring) * (2u * b_bytes >> 4);
            const int halves = k_lo + 2 * j + 1 < k_hi ? 2 : 1;
            for (int h = 0; h < halves; ++h, ad += kABytes >> 4, bd += b_bytes >> 4) {
#pragma unroll
              for (uint32_t kk = 0; kk < kBK / 16; ++kk)
                umma_f16(tmem, ad + 2u * kk, bd + b_step * kk, idesc, j > 0 || h > 0 || kk > 0 ? 1u : 0u);
            }
            umma_commit(&empty[ring]);
          }
          advance();
        }
        if (ok && elect_lane()) umma_commit(&acc_bar);
      }
    } else {
      // ---------------------------------------------------------- gathers
      if (box || warp - 2 >= fours) {
        // Nothing of these stages is this warp's, so they must not be waited
        // for either: they are filled and freed without it, and a parity that
        // has moved on would not come back.
        const int to = ring + steps;
        parity ^= static_cast<uint32_t>(to / p.stages) & 1u;
        ring = to % p.stages;
      } else {
        if (lane < 16) gather[warp - 2][lane] = idx;
        __syncwarp();
        for (int j = 0; j < steps && ok; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[ring], parity ^ 1u, p.err, kErrTimeoutEmpty));
          if (!ok) break;
          if (elect_lane()) {
            const int kb = k_lo + 2 * j;
            const uint32_t a_s = base + static_cast<uint32_t>(ring) * 2u * kABytes;
            // A warp's gathers of both halves; the bytes are the producer's to
            // announce.
            for (int i = warp - 2; i < fours; i += 4) {
              const int4 rows = gather[warp - 2][i];
              tma_gather4(a_s + static_cast<uint32_t>(i) * 512u, &p.tmLg, &full[ring], kb * kBK, rows);
              if (kb + 1 < k_hi)
                tma_gather4(a_s + kABytes + static_cast<uint32_t>(i) * 512u, &p.tmLg, &full[ring], (kb + 1) * kBK, rows);
            }
          }
          advance();
        }
        __syncwarp();
      }
      // ---------------------------------------------------------- epilogue
      if (ok) ok = mbar_wait_bounded(&acc_bar, acc_phase, p.err, kErrTimeoutAcc, 20000000000ull);
      ok = __all_sync(0xffffffffu, ok);
      const int quad = warp & 3, row = quad * 32 + lane;
      if (ok && quad * 32 < valid) {
        tc_fence_after();
        const float s = __ldg(p.scale + a);
        uint16_t *out = row < valid ? p.out + static_cast<int64_t>(__ldcg(list + row)) * p.r : nullptr;
        for (int c = 0; c < p.r; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c), v);
          if (row >= valid) continue;
          if (nz > 1) {
            // The fp32 partial, into the idle ring.
            const uint32_t dst = base + (static_cast<uint32_t>(row) * part_ld + static_cast<uint32_t>(c)) * 4u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t q[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
              sts128(dst + 16u * static_cast<uint32_t>(j), q);
            }
          } else {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = pack_bf16x2(__uint_as_float(v[2 * j]) * s, __uint_as_float(v[2 * j + 1]) * s);
            reinterpret_cast<uint4 *>(out + c)[0] = make_uint4(h[0], h[1], h[2], h[3]);
            reinterpret_cast<uint4 *>(out + c)[1] = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
      }
    }
    acc_phase ^= 1u;
    tc_fence_before();
    if (nz == 1) {
      __syncthreads();
      tc_fence_after();
      continue;
    }
    cluster_sync_all();
    tc_fence_after();
    // This CTA's share of the slot's rows, four columns at a time, the peers'
    // partials added in rank order.
    {
      const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
      const int lo = valid * rank / size, hi = valid * (rank + 1) / size;
      const int pieces = p.r / 4;
      const float s = __ldg(p.scale + a);
      for (int i = threadIdx.x; i < (hi - lo) * pieces; i += kThreads) {
        const int row = lo + i / pieces, col = 4 * (i % pieces);
        const uint32_t off = base + (static_cast<uint32_t>(row) * part_ld + static_cast<uint32_t>(col)) * 4u;
        float4 part[8];
#pragma unroll
        for (int pr = 0; pr < 8; ++pr)
          part[pr] = pr < size ? ld_dsmem_v4(off, static_cast<uint32_t>(pr)) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 acc = part[0];
#pragma unroll
        for (int pr = 1; pr < 8; ++pr) {
          if (pr < size) {
            acc.x += part[pr].x;
            acc.y += part[pr].y;
            acc.z += part[pr].z;
            acc.w += part[pr].w;
          }
        }
        uint16_t *dst = p.out + static_cast<int64_t>(__ldcg(list + row)) * p.r + col;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc.x * s, acc.y * s), pack_bf16x2(acc.z * s, acc.w * s));
      }
    }
    // The partials' generic accesses come before the next slot's TMA writes.
    fence_proxy_async_smem();
    cluster_sync_all();
  }

  // Every issued copy has landed before the CTA may exit: the products waited
  // for them, unless a wait gave up.
  if (warp == 0 && lane == 0 && issued > 0)
    for (int j = issued - p.stages < 0 ? 0 : issued - p.stages; j < issued; ++j)
      mbar_wait_bounded(&full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1u, p.err, kErrTimeoutDrain);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// T[i, j] = bf16(s_a . X[i, :] . A_a[j, :]) for a handful of rows.
constexpr int kSmallThreads = 256;
__global__ void __launch_bounds__(kSmallThreads) multi_proj_small_kernel(
    const uint16_t *__restrict__ X, const int32_t *__restrict__ ids, int64_t k, const uint16_t *__restrict__ A, int r,
    int count, const float *__restrict__ scale, uint16_t *__restrict__ T) {
  __shared__ float red[kSmallThreads / 32];
  griddep_launch();
  const int j = static_cast<int>(blockIdx.x), i = static_cast<int>(blockIdx.y);
  const int a = __ldg(ids + i);
  const bool live = a >= 0 && a < count;
  float s = 0.f;
  if (live) {
    const uint4 *xp = reinterpret_cast<const uint4 *>(X + static_cast<int64_t>(i) * k);
    const uint4 *ap = reinterpret_cast<const uint4 *>(A + (static_cast<int64_t>(a) * r + j) * k);
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < k / 8; c += kSmallThreads) {
      const uint4 xv = __ldg(xp + c), av = __ldg(ap + c);
      const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w}, aa[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(bf16lo_to_f32(xx[e]), bf16lo_to_f32(aa[e]), s);
        s = fmaf(bf16hi_to_f32(xx[e]), bf16hi_to_f32(aa[e]), s);
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallThreads / 32; ++w) v += red[w];
    T[static_cast<int64_t>(i) * r + j] =
        static_cast<uint16_t>(pack_bf16x2(live ? v * __ldg(scale + a) : 0.f, 0.f) & 0xFFFFu);
  }
}

template <bool R_MN>
cudaError_t launch(ProjParams &p, int64_t slots, int64_t free_sms, int64_t main_steps, cudaStream_t stream) {
  static std::atomic<bool> configured[kMaxDevicesPerProcess] = {};
  static ClusterFit fit[2];
  const void *kernel = reinterpret_cast<const void *>(multi_proj_kernel<R_MN>);
  cudaError_t e = set_smem_once(kernel, static_cast<int>(kRing) + 1024, configured);
  if (e != cudaSuccess) return e;
  // The projection keeps to the SMs that the product launched on its heels
  // leaves free, if it is done there before that product needs it: 64 columns
  // of a slot take about 0.33 us, a k-step of the product 0.55 to 0.85 us.
  // Forward of 1111 x 11008 -> 4096, r = 64: 136 us beside the product and 150
  // in front of it with 6 adapters, 205 and 207 with 64 (where the estimate is
  // the product's whole main loop); 128 x 8192 -> 28672, r = 16, 64 adapters: 126
  // and 142.  One CTA to an SM then, since CTAs that could share one are spread
  // over them all.
  // K is split over the largest clusters of which one per slot fits at once.
  const bool beside = free_sms >= 16 && slots * p.nk <= 2 * free_sms * main_steps;
  const int per_sm = beside || p.r > kSharedRank ? 1 : 2;
  const int smem = static_cast<int>(kRing) / per_sm + 1024;
  p.stages = stages_of(p.r, per_sm);
  const int most_split = p.nk / 2 < 1 ? 1 : p.nk / 2 < 8 ? p.nk / 2 : 8;
  int clusters = 1;
  const int split = fit[per_sm - 1].split(kernel, kThreads, smem, slots, per_sm, most_split, &clusters,
                                          beside ? static_cast<int>(free_sms) : 1 << 30);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(slots < clusters ? slots : clusters), 1, static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(split);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, multi_proj_kernel<R_MN>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_multi_proj_small(const uint16_t *X, int64_t m, int64_t k, const AdapterView &s, uint16_t *T,
                                    cudaStream_t stream) {
  multi_proj_small_kernel<<<dim3(static_cast<unsigned>(s.r), static_cast<unsigned>(m)), kSmallThreads, 0, stream>>>(
      X, s.ids, k, s.A, s.r, s.count, s.scale, T);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_multi_proj(const uint16_t *L, int64_t m, int64_t kc, const AdapterView &s, bool through_b,
                              uint16_t *out, const GroupRows &rows, MultiGrid next, cudaStream_t stream) {
  ProjParams p{};
  p.width = unit_width(s.r);
  if (through_b ? !encode_bf16_stack_map(&p.tmR, s.B, s.count, kc, s.r, static_cast<uint32_t>(p.width), 64)
                : !encode_bf16_stack_map(&p.tmR, s.A, s.count, s.r, kc, 64, static_cast<uint32_t>(p.width)))
    return cudaErrorInvalidValue;
  if (!encode_bf16_map(&p.tmL, L, m, kc, 64, kSlotRows) || !encode_bf16_map(&p.tmLg, L, m, kc, 64, 1))
    return cudaErrorInvalidValue;
  p.rows = row_slots(&rows, m);
  p.scale = s.scale;
  p.out = out;
  p.err = device_error_word();
  p.r = s.r;
  p.nk = static_cast<int>((kc + kBK - 1) / kBK);
  // At most m / 64 slots, and one more for every adapter with rows.
  const int64_t slots = m / kSlotRows + (s.count < m ? s.count : m);
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t free_sms = next.ctas > 0 ? sms - next.ctas : 0;
  return through_b ? launch<true>(p, slots, free_sms, next.steps, stream)
                   : launch<false>(p, slots, free_sms, next.steps, stream);
}

}  // namespace qlora
