// Rank-r projections of a batch whose rows belong to different adapters:
//
//   T[i, :] = bf16(s_a . X[i, :] . A_a^T)      (A [count x r x k], K-major)
//   U[i, :] = bf16(s_a . dY[i, :] . B_a)       (B [count x n x r], r contiguous)
//
// with a = ids[i]; a row whose id is outside [0, count) gets zeros.  "QLoRA",
// Training setup versus deployment setup: the quantized base is served with
// the adapter, and one base serves several; "QLoRA and Quantized Training", In
// code: r and alpha.
//
// tcgen05 path (multi_proj_kernel).  A CTA takes 128 rows of the batch, lists
// the adapters that occur in them (in order of first appearance) and packs
// their rank columns into the N dimension of one product: 64 / w units of w
// columns each (w = 64, 32 or 16, the widest that divides r).  The
// accumulator then holds every row against every listed adapter; a row keeps
// only its own adapter's columns.  So rows in any order need no sorting, a
// batch ordered by adapter costs one pass per tile, and the rows of X are read
// once per 64 rank columns present.  Passes are spread over CTAs, K over a
// cluster of up to 8 CTAs whose fp32 partials are added in rank order.
// Bound by reading X and the adapters present (HBM / L2).
//
// Decode path (multi_proj_small_kernel, m <= 16): a CTA per (adapter row,
// token), a plain dot product: the tokens' adapters are mostly distinct, so
// each byte of A is used once and the kernel is bound by its latency.
//
// Tile lists.  The kernels that add T . B^T (or U . A) to a tile need its
// adapters and, for each, which rows use it (the lane masks of the masked
// products).  One extra CTA per 512-row tile (128 rows when m <= 128) writes
// them beside the projection, at no extra launch.
#include <cuda.h>

#include "internal.h"
#include "multi.cuh"
#include "split_reduce.cuh"

namespace qlora {
namespace {

constexpr int kBK = 64;
constexpr int kRows = 128;
constexpr int kStages = 4;
constexpr int kThreads = 192;                     // TMA warp, MMA warp, four epilogue warps
constexpr uint32_t kABytes = 128u * kBK * 2u;     // 16 KB
constexpr uint32_t kBBytes = 64u * kBK * 2u;      // 8 KB
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024u;
constexpr uint32_t kPartLd = 64u + 4u;
static_assert(2u * (kSmemBytes + 4096u) <= 227u * 1024u, "two CTAs per SM");
static_assert(kStages * kStageBytes >= 128u * kPartLd * 4u, "room for the fp32 partial tile");
// The list builder's arrays: ids, first occurrence and slot of 512 rows, then
// 16 mask words for each of up to 512 adapters.
static_assert(kStages * kStageBytes >= 3u * 2048u + 512u * 64u, "room for the tile lists");

struct __align__(64) ProjParams {
  CUtensorMap tmL;        // X or dY [m x kc], box {64, 128}
  CUtensorMap tmR;        // A {kc, r, count} box {64, w, 1}; B {r, kc, count} box {w, 64, 1}
  const int32_t *ids;
  const float *scale;
  uint16_t *out;          // [m x r]
  unsigned *err;
  int32_t *lists;         // tile lists (null: not wanted)
  int64_t list_stride;    // int32 per tile
  int list_slots, list_rows, list_tiles;
  int m, r, count, width, nk, pass_ctas;
};

__device__ __forceinline__ int row_id(const ProjParams &p, int64_t row) {
  const int id = row < p.m ? __ldg(p.ids + row) : -1;
  return id >= 0 && id < p.count ? id : -1;
}

// One tile's adapters and row masks (layout: see TileLists).
__device__ void build_lists(const ProjParams &p, int tile, uint8_t *smem) {
  const int n = p.list_rows, words = n / 32;
  int *ids = reinterpret_cast<int *>(smem), *first = ids + 512, *slot = first + 512;
  uint32_t *mask = reinterpret_cast<uint32_t *>(slot + 512);
  __shared__ int total_s;
  for (int i = threadIdx.x; i < n; i += kThreads) ids[i] = row_id(p, static_cast<int64_t>(tile) * n + i);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int id = ids[i];
    int j = 0;
    while (ids[j] != id) ++j;
    first[i] = j;
  }
  __syncthreads();
  int32_t *out = p.lists + tile * p.list_stride;
  if (threadIdx.x < 32) {
    int base = 0;
    for (int c = 0; c < words; ++c) {
      const int i = 32 * c + static_cast<int>(threadIdx.x);
      const bool lead = ids[i] >= 0 && first[i] == i;
      const unsigned b = __ballot_sync(0xffffffffu, lead);
      const int s = base + __popc(b & ((1u << threadIdx.x) - 1u));
      if (lead) {
        slot[i] = s;
        out[4 + s] = ids[i];
      }
      base += __popc(b);
    }
    if (threadIdx.x == 0) {
      out[0] = base;
      total_s = base;
    }
  }
  __syncthreads();
  const int total = total_s;
  for (int i = threadIdx.x; i < total * words; i += kThreads) mask[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (ids[i] >= 0) atomicOr(&mask[slot[first[i]] * words + (i >> 5)], 1u << (i & 31));
  __syncthreads();
  uint32_t *gmask = reinterpret_cast<uint32_t *>(out + 4 + p.list_slots);
  for (int i = threadIdx.x; i < total * words; i += kThreads) gmask[i] = mask[i];
}

// R_MN: R is [count x kc x r] (MN-major operand); else [count x r x kc].
template <bool R_MN>
__global__ void __launch_bounds__(kThreads, 2) multi_proj_kernel(const __grid_constant__ ProjParams p) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) int ids[kRows];
  __shared__ int list[kRows], slot_of[kRows], lead_count[4];

  // The kernel that consumes the output may start now; it waits for this
  // grid before it reads the output or the lists.
  griddep_launch();
  const uint32_t raw = smem_u32(dsmem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  if (static_cast<int>(blockIdx.x) == p.pass_ctas) {
    if (z == 0 && static_cast<int>(blockIdx.y) < p.list_tiles)
      build_lists(p, static_cast<int>(blockIdx.y), dsmem + (base - raw));
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tile = static_cast<int>(blockIdx.y);
  const int k_lo = static_cast<int>((static_cast<int64_t>(p.nk) * z) / nz);
  const int k_hi = static_cast<int>((static_cast<int64_t>(p.nk) * (z + 1)) / nz);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
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
  // The tile's adapters: a row leads if no earlier row has its id; leaders
  // are numbered in row order.
  const int t = static_cast<int>(threadIdx.x) - 64;
  const int my_id = t >= 0 ? row_id(p, static_cast<int64_t>(m_tile) * kRows + t) : -1;
  if (t >= 0) ids[t] = my_id;
  __syncthreads();
  int first = t;
  unsigned lead_bits = 0u;
  if (t >= 0) {
    for (int j = 0; j < t; j += 4) {
      const int4 v = *reinterpret_cast<const int4 *>(ids + j);
      const int at = v.x == my_id ? j : v.y == my_id ? j + 1 : v.z == my_id ? j + 2 : v.w == my_id ? j + 3 : t;
      if (at < t) {
        first = at;
        break;
      }
    }
    lead_bits = __ballot_sync(0xffffffffu, my_id >= 0 && first == t);
    if (lane == 0) lead_count[t >> 5] = __popc(lead_bits);
  }
  __syncthreads();
  const int listed = lead_count[0] + lead_count[1] + lead_count[2] + lead_count[3];
  if (t >= 0 && my_id >= 0 && first == t) {
    int s = __popc(lead_bits & ((1u << lane) - 1u));
    for (int w = 0; w < (t >> 5); ++w) s += lead_count[w];
    list[s] = my_id;
    slot_of[t] = s;
  }
  __syncthreads();
  // Read by everyone before a non-leader overwrites its own entry.
  const int my_slot = t >= 0 && my_id >= 0 ? slot_of[first] : -1;
  __syncthreads();
  if (t >= 0) slot_of[t] = my_slot;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const int w = p.width, per_adapter = p.r / w, per_pass = 64 / w;
  const int units = listed * per_adapter;
  const int passes = (units + per_pass - 1) / per_pass;
  const uint32_t unit_bytes = static_cast<uint32_t>(w) * 128u;
  int step = 0;         // k-steps of the CTA's earlier passes (ring position)
  int issued = 0;       // k-steps whose copies were issued (producer)
  bool ok = true;
  uint32_t acc_phase = 0u;

  for (int pass = static_cast<int>(blockIdx.x); pass < passes; pass += p.pass_ctas) {
    const int u0 = pass * per_pass;
    const int nu = units - u0 < per_pass ? units - u0 : per_pass;
    const int steps = k_hi - k_lo;
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0 && ok) {
        for (int j = 0; j < steps && ok; ++j) {
          const int s = (step + j) % kStages;
          const uint32_t ph = static_cast<uint32_t>((step + j) / kStages) & 1u;
          ok = mbar_wait_bounded(&empty[s], ph ^ 1u, p.err, kErrTimeoutEmpty);
          if (!ok) break;
          const uint32_t a_s = base + static_cast<uint32_t>(s) * kStageBytes, b_s = a_s + kABytes;
          mbar_arrive_expect_tx(&full[s], kABytes + static_cast<uint32_t>(nu) * unit_bytes);
          const int kx = (k_lo + j) * kBK;
          tma_load_2d(a_s, &p.tmL, &full[s], kx, m_tile * kRows);
          for (int u = 0; u < nu; ++u) {
            const int a = list[(u0 + u) / per_adapter], c = (u0 + u) % per_adapter;
            const uint32_t dst = b_s + static_cast<uint32_t>(u) * unit_bytes;
            if (R_MN)
              tma_load_3d(dst, &p.tmR, &full[s], c * w, kx, a);
            else
              tma_load_3d(dst, &p.tmR, &full[s], kx, c * w, a);
          }
          ++issued;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0 && ok) {
        const uint32_t idesc = make_idesc(nu * w, false, R_MN);
        for (int j = 0; j < steps && ok; ++j) {
          const int s = (step + j) % kStages;
          const uint32_t ph = static_cast<uint32_t>((step + j) / kStages) & 1u;
          ok = mbar_wait_bounded(&full[s], ph, p.err, kErrTimeoutFullA);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_s = base + static_cast<uint32_t>(s) * kStageBytes, b_s = a_s + kABytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            // MN-major units: [64 k-rows x w columns], one behind the other.
            const uint64_t bd = R_MN ? smem_desc_unit(b_s + static_cast<uint32_t>(kk * 32 * w), unit_bytes,
                                                      static_cast<uint32_t>(16 * w), w)
                                     : smem_desc(b_s + kk * 32u, 16u, 1024u);
            umma_f16(tmem, smem_desc(a_s + kk * 32u, 16u, 1024u), bd, idesc, (j > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&acc_bar);
      }
    } else {
      // ---------------------------------------------------------- epilogue
      if (ok) ok = mbar_wait_bounded(&acc_bar, acc_phase, p.err, kErrTimeoutAcc, 20000000000ull);
      if (ok) {
        tc_fence_after();
        const int quad = warp & 3;
        const uint32_t row = static_cast<uint32_t>(quad * 32 + lane);
        for (int c0 = 0; c0 < nu * w; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c0), v);
          const uint32_t dst = base + (row * kPartLd + static_cast<uint32_t>(c0)) * 4u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t q[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
            sts128(dst + 16u * static_cast<uint32_t>(j), q);
          }
        }
      }
    }
    step += steps;
    acc_phase ^= 1u;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();
    // This CTA's share of the tile's rows: each row's own adapter's columns of
    // this pass, four at a time, the peers' partials added in rank order.
    {
      const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
      const int left = p.m - m_tile * kRows;
      const int valid = left < kRows ? left : kRows;
      const int lo = valid * rank / size, hi = valid * (rank + 1) / size;
      const int pieces = nu * w / 4;
      for (int i = threadIdx.x; i < (hi - lo) * pieces; i += kThreads) {
        const int row = lo + i / pieces, col = 4 * (i % pieces);
        const int g = u0 + col / w;
        const int slot = slot_of[row];
        if (slot < 0 || g / per_adapter != slot) continue;
        const uint32_t off = base + (static_cast<uint32_t>(row) * kPartLd + static_cast<uint32_t>(col)) * 4u;
        float4 part[8];
#pragma unroll
        for (int pr = 0; pr < 8; ++pr)
          part[pr] = pr < size ? ld_dsmem_v4(off, static_cast<uint32_t>(pr)) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int pr = 0; pr < 8; ++pr) {
          if (pr < size) {
            acc.x += part[pr].x;
            acc.y += part[pr].y;
            acc.z += part[pr].z;
            acc.w += part[pr].w;
          }
        }
        const float s = __ldg(p.scale + list[slot]);
        uint16_t *dst = p.out + (static_cast<int64_t>(m_tile) * kRows + row) * p.r + (g % per_adapter) * w + col % w;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc.x * s, acc.y * s), pack_bf16x2(acc.z * s, acc.w * s));
      }
    }
    // The partials' generic accesses come before the next pass's TMA writes.
    fence_proxy_async_smem();
    cluster_sync_all();
  }

  // Every issued copy has landed before the CTA may exit.
  if (threadIdx.x == 0)
    for (int j = issued - kStages < 0 ? 0 : issued - kStages; j < issued; ++j)
      mbar_wait_bounded(&full[j % kStages], static_cast<uint32_t>(j / kStages) & 1u, p.err, kErrTimeoutDrain);

  // Rows without an adapter.
  if (blockIdx.x == 0 && z == 0) {
    const int left = p.m - m_tile * kRows;
    const int valid = left < kRows ? left : kRows;
    const int pieces = p.r / 8;
    for (int i = threadIdx.x; i < valid * pieces; i += kThreads) {
      const int row = i / pieces;
      if (slot_of[row] < 0)
        reinterpret_cast<uint4 *>(p.out + (static_cast<int64_t>(m_tile) * kRows + row) * p.r)[i % pieces] =
            make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(64u) : "memory");
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
cudaError_t launch(const ProjParams &p, int m_tiles, int split, cudaStream_t stream) {
  static std::atomic<bool> configured[kMaxDevicesPerProcess] = {};
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(multi_proj_kernel<R_MN>), static_cast<int>(kSmemBytes),
                                configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.pass_ctas + (p.lists ? 1 : 0)), static_cast<unsigned>(m_tiles),
                     static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(split);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, multi_proj_kernel<R_MN>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

int tile_list_rows(int64_t m) { return m <= 128 ? 128 : 512; }

size_t tile_lists_bytes(int64_t m, int32_t count) { return static_cast<size_t>(carve_tile_lists(nullptr, m, count).bytes); }

TileLists carve_tile_lists(void *scratch, int64_t m, int32_t count) {
  TileLists t{};
  t.base = static_cast<int32_t *>(scratch);
  t.rows = tile_list_rows(m);
  t.tiles = (m + t.rows - 1) / t.rows;
  int64_t slots = count < t.rows ? count : t.rows;
  if (m < slots) slots = m;
  t.slots = static_cast<int32_t>((slots + 3) / 4 * 4);
  t.stride = 4 + t.slots + static_cast<int64_t>(t.slots) * (t.rows / 32);
  t.bytes = t.tiles * t.stride * 4;
  return t;
}

cudaError_t launch_multi_proj_small(const uint16_t *X, int64_t m, int64_t k, const AdapterView &s, uint16_t *T,
                                    cudaStream_t stream) {
  multi_proj_small_kernel<<<dim3(static_cast<unsigned>(s.r), static_cast<unsigned>(m)), kSmallThreads, 0, stream>>>(
      X, s.ids, k, s.A, s.r, s.count, s.scale, T);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_multi_proj(const uint16_t *L, int64_t m, int64_t kc, const AdapterView &s, bool through_b,
                              uint16_t *out, const TileLists *lists, cudaStream_t stream) {
  ProjParams p{};
  p.width = unit_width(s.r);
  if (!encode_bf16_map(&p.tmL, L, m, kc, 64, 128)) return cudaErrorInvalidValue;
  if (through_b) {
    if (!encode_bf16_stack_map(&p.tmR, s.B, s.count, kc, s.r, static_cast<uint32_t>(p.width), 64))
      return cudaErrorInvalidValue;
  } else if (!encode_bf16_stack_map(&p.tmR, s.A, s.count, s.r, kc, 64, static_cast<uint32_t>(p.width))) {
    return cudaErrorInvalidValue;
  }
  p.ids = s.ids;
  p.scale = s.scale;
  p.out = out;
  p.err = device_error_word();
  p.m = static_cast<int>(m);
  p.r = s.r;
  p.count = s.count;
  p.nk = static_cast<int>((kc + kBK - 1) / kBK);
  if (lists) {
    p.lists = lists->base;
    p.list_stride = lists->stride;
    p.list_slots = lists->slots;
    p.list_rows = lists->rows;
    p.list_tiles = static_cast<int>(lists->tiles);
  }
  // Passes a tile can need at most (every row or every adapter its own), and
  // the K split that fills about two CTAs per SM with one pass per tile; CTAs
  // for further passes only while that leaves SMs idle.
  const int64_t m_tiles = (m + kRows - 1) / kRows;
  int64_t most = s.count < kRows ? s.count : kRows;
  if (m < most) most = m;
  const int64_t max_passes = (most * s.r + 63) / 64;
  const int split = choose_split(m_tiles, p.nk);
  int64_t ctas = 2 * 148 / (m_tiles * split);
  if (ctas > max_passes) ctas = max_passes;
  p.pass_ctas = static_cast<int>(ctas < 1 ? 1 : ctas);
  return through_b ? launch<true>(p, static_cast<int>(m_tiles), split, stream)
                   : launch<false>(p, static_cast<int>(m_tiles), split, stream);
}

}  // namespace qlora
