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
// their rank columns side by side into the N dimension of one product, up to
// 256 columns a pass, in units of w columns (w = 64, 32 or 16, the widest that
// divides r).  The accumulator then holds every row against every adapter of
// the pass; a row keeps only its own adapter's columns.  So rows in any order
// need no sorting, a batch ordered by adapter takes one pass per tile, and X is
// read once per 256 rank columns present.  K is split over a cluster of up to
// 8 CTAs whose fp32 partials (each row's own r columns) are added in rank
// order; narrower passes on more CTAs when the tiles alone leave SMs idle.
// Bound by reading X and the adapters present (HBM / L2).  The copy engine
// takes as long for a box row of 32 or 64 bytes as for one of 128 bytes, so in
// U's form with w < 64 the epilogue warps fetch the adapter tiles with 16-byte
// asynchronous copies.  (Two warps issuing alternate k-steps into accumulators
// of their own took the same time: the copies set the pace.)
//
// Decode path (multi_proj_small_kernel, m <= 16): a CTA per (adapter row,
// token), a plain dot product: the tokens' adapters are mostly distinct, so
// each byte of A is used once and the kernel is bound by its latency.
//
// Tile lists.  The kernels that add T . B^T (or U . A) to a tile need its
// adapters and, for each, which rows use it (the lane masks of the masked
// products), and the adapter gradients each adapter's rows.  Two more warps
// of the projection write them beside it, at no extra launch.
#include <cuda.h>

#include "internal.h"
#include "multi.cuh"
#include "split_reduce.cuh"

namespace qlora {
namespace {

constexpr int kBK = 64;
constexpr int kRows = 128;
constexpr int kMaxStages = 8;
constexpr int kMaxCols = 256;                     // rank columns of a pass
constexpr int kListThreads = 64;
// TMA warp, MMA warp, four adapter-tile / epilogue warps, two list warps.
constexpr int kThreads = 192 + kListThreads;
constexpr uint32_t kABytes = 128u * kBK * 2u;     // 16 KB
constexpr uint32_t kColBytes = kBK * 2u;          // shared memory of one rank column of a k-step
constexpr uint32_t kRing = 200u * 1024u;
constexpr uint32_t kSmemBytes = kRing + 1024u;
// The ring holds X's 16 KB tiles first, then the adapter tiles: 8 stages at 64
// columns, 4 at 256.
constexpr uint32_t kMinStages = 4;
static_assert(kRing / (kABytes + kMaxCols * kColBytes) >= kMinStages, "four stages at the widest");
static_assert(kRing >= 128u * (kMaxCols + 4u) * 4u, "room for the fp32 partial tile");
constexpr int64_t kRowsInside = 8192;             // batches whose row lists the list warps make
constexpr int kAhead = 3;                         // k-steps of adapter copies in flight per thread
static_assert(kRing / (kABytes + kMaxCols * kColBytes) > kAhead, "a stage is refilled after its copies were reported");

struct __align__(64) ProjParams {
  CUtensorMap tmL;        // X or dY [m x kc], box {64, tile_rows}
  CUtensorMap tmR;        // A {kc, r, count} box {64, w, 1}; B {r, kc, count} box {64, 64, 1} (w = 64)
  const uint16_t *R;      // B [count x kc x r] (w < 64)
  int64_t kc;
  const int32_t *ids;
  const float *scale;
  uint16_t *out;          // [m x r]
  unsigned *err;
  GroupRows rows;         // row lists (null list: not wanted)
  int32_t *lists;         // tile lists (null: not wanted)
  int64_t list_stride;    // int32 per tile
  int list_slots, list_rows;
  int m, r, count, width, nk, pass_ctas;
  int per_pass;           // adapters of a pass
  int tile_rows;          // 128, or 64 where that fills the SMs better
};

__device__ __forceinline__ int row_id(const ProjParams &p, int64_t row) {
  const int id = row < p.m ? __ldg(p.ids + row) : -1;
  return id >= 0 && id < p.count ? id : -1;
}

// Finds or adds `id` in a table of SIZE keys (empty: -1) and notes `row` as a
// row of it: first[place] ends as the lowest row.  Returns the place.
template <int SIZE>
__device__ __forceinline__ int table_add(int *key, int *first, int id, int row) {
  uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 16 & (SIZE - 1);
  for (;;) {     // ends: fewer ids than places
    const int old = atomicCAS(&key[h], -1, id);
    if (old == -1 || old == id) break;
    h = (h + 1) & (SIZE - 1);
  }
  atomicMin(&first[h], row);
  return static_cast<int>(h);
}

// The list warps' arrays: ids, table place and slot of up to 512 rows, and the
// table (key, first row).
struct ListSmem {
  int id[512], place[512], slot[512], key[1024], first[1024];
};

// One tile's adapters and row masks (layout: see TileLists), by thread t of
// the list warps (named barrier 1).
__device__ void build_lists(const ProjParams &p, int tile, ListSmem &s, int t) {
  const int n = p.list_rows, words = n / 32, lane = t & 31;
  for (int i = t; i < 1024; i += kListThreads) {
    s.key[i] = -1;
    s.first[i] = 0x7FFFFFFF;
  }
  for (int i = t; i < n; i += kListThreads) s.id[i] = row_id(p, static_cast<int64_t>(tile) * n + i);
  named_barrier_sync(1, kListThreads);
  for (int i = t; i < n; i += kListThreads)
    if (s.id[i] >= 0) s.place[i] = table_add<1024>(s.key, s.first, s.id[i], i);
  named_barrier_sync(1, kListThreads);
  int32_t *out = p.lists + tile * p.list_stride;
  uint32_t *mask = reinterpret_cast<uint32_t *>(out + 4 + p.list_slots);
  // Both warps number the leaders; each stores half of the entries.
  int total = 0;
  for (int c = 0; c < words; ++c) {
    const int i = 32 * c + lane;
    const bool lead = s.id[i] >= 0 && s.first[s.place[i]] == i;
    const unsigned b = __ballot_sync(0xffffffffu, lead);
    const int at = total + __popc(b & ((1u << lane) - 1u));
    if (lead && (c & 1) == (t >> 5)) {
      s.slot[i] = at;
      out[4 + at] = s.id[i];
    }
    total += __popc(b);
  }
  if (t == 0) out[0] = total;
  for (int i = t; i < total * words; i += kListThreads) mask[i] = 0u;
  named_barrier_sync(1, kListThreads);
  // A mask word per (adapter, 32 rows) that has a row, from the lanes that
  // hold the same id.
  for (int c = t >> 5; c < words; c += 2) {
    const int i = 32 * c + lane, id = s.id[i];
    const unsigned same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0u) mask[s.slot[s.first[s.place[i]]] * words + c] = same;
  }
}

// The rows of adapter a in ascending order (layout: see GroupRows), by thread
// t of `threads`, whose warps take contiguous runs of rows and count by
// ballots: no atomics, so the order is fixed.  Adapter a's list starts at entry
// 64 (floor(b / 64) + a), b the number of rows with a lower id: such a list of
// c entries padded to a multiple of 64 ends before adapter a + 1's starts, so
// nobody needs another adapter's count.
template <int THREADS, class Sync>
__device__ void list_rows(const int32_t *ids, int m, int a, const GroupRows &g, int (*count_of)[2], int t,
                          const Sync &sync) {
  constexpr int kWarps = THREADS / 32;
  const int warp = t >> 5, lane = t & 31;
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
    count_of[warp][0] = eq;
    count_of[warp][1] = lt;
  }
  sync();
  int before = 0, total = 0, lower = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? count_of[w][0] : 0;
    total += count_of[w][0];
    lower += count_of[w][1];
  }
  const int64_t first = 64 * (static_cast<int64_t>(lower / 64) + a);
  if (t == 0) {
    g.start[a] = static_cast<int32_t>(first);
    g.count[a] = total;
  }
  int32_t *dst = g.list + first;
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
  sync();
}

// The lists of a long batch, one CTA per adapter (a short batch's are made by
// the projection's list warps).
constexpr int kRowsThreads = 512;
__global__ void __launch_bounds__(kRowsThreads) group_rows_kernel(const int32_t *__restrict__ ids, int m, GroupRows g) {
  __shared__ int count_of[kRowsThreads / 32][2];
  list_rows<kRowsThreads>(ids, m, static_cast<int>(blockIdx.x), g, count_of, static_cast<int>(threadIdx.x),
                          [] { __syncthreads(); });
}

// R_MN: R is [count x kc x r] (MN-major operand); else [count x r x kc].
template <bool R_MN>
__global__ void __launch_bounds__(kThreads, 1) multi_proj_kernel(const __grid_constant__ ProjParams p) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int2 unit_list[kMaxCols / 16];
  __shared__ const uint16_t *unit_src[kMaxCols / 16];
  __shared__ int key[256], first[256], list[kRows], slot_of[kRows], lead_slot[kRows], lead_count[4];

  __shared__ ListSmem lists_s;
  __shared__ int failed, rows_count[kListThreads / 32][2];

  // The kernel that consumes the output may start now; it waits for this
  // grid before it reads the output or the lists.
  griddep_launch();
  const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tile = static_cast<int>(blockIdx.y);
  const int k_lo = static_cast<int>((static_cast<int64_t>(p.nk) * z) / nz);
  const int k_hi = static_cast<int>((static_cast<int64_t>(p.nk) * (z + 1)) / nz);
  const int steps = k_hi - k_lo;
  const bool loaders = R_MN && p.width < 64;      // adapter tiles by the epilogue warps
  // X's copy for step j of a pass into stage s.  64-row tiles leave the second
  // half of A as it is: its accumulator rows are never read.
  const auto load_x = [&](int s, int j) {
    tma_load_2d(base + static_cast<uint32_t>(s) * kABytes, &p.tmL, &full[s], (k_lo + j) * kBK,
                m_tile * p.tile_rows);
  };
  int issued = 0;               // k-steps whose copies were issued (producer)

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], loaders ? 1 + 4 : 1);     // the copies, and the adapter-tile warps
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_bar, 1);
    failed = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    // The first pass's copies of X start before the adapters are listed (their
    // bytes are announced with the adapters').
    if (blockIdx.x == 0)
      for (; issued < static_cast<int>(kMinStages) && issued < steps; ++issued) load_x(issued, issued);
  }
  // The tile's adapters: a row leads if it is its id's first; leaders are
  // numbered in row order.
  const int t = static_cast<int>(threadIdx.x) - 64;
  const bool row_warp = warp >= 2 && warp < 6;
  const int my_id = row_warp && t < p.tile_rows ? row_id(p, static_cast<int64_t>(m_tile) * p.tile_rows + t) : -1;
  for (int i = threadIdx.x; i < 256; i += kThreads) {
    key[i] = -1;
    first[i] = 0x7FFFFFFF;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(static_cast<uint32_t>(kMaxCols))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  const int place = my_id >= 0 ? table_add<256>(key, first, my_id, t) : -1;
  __syncthreads();
  const bool lead = my_id >= 0 && first[place] == t;
  const unsigned lead_bits = __ballot_sync(0xffffffffu, lead);
  if (row_warp && lane == 0) lead_count[t >> 5] = __popc(lead_bits);
  __syncthreads();
  if (lead) {
    int s = __popc(lead_bits & ((1u << lane) - 1u));
    for (int w = 0; w < (t >> 5); ++w) s += lead_count[w];
    list[s] = my_id;
    lead_slot[t] = s;
  }
  __syncthreads();
  const int listed = lead_count[0] + lead_count[1] + lead_count[2] + lead_count[3];
  const int my_slot = my_id >= 0 ? lead_slot[first[place]] : -1;
  if (row_warp) slot_of[t] = my_slot;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const int w = p.width, per_adapter = p.r / w;
  const int passes = (listed + p.per_pass - 1) / p.per_pass;
  const uint32_t unit_bytes = static_cast<uint32_t>(w) * kColBytes;
  const int widest = listed < p.per_pass ? listed : p.per_pass;
  const uint32_t b_bytes = static_cast<uint32_t>(widest * p.r) * kColBytes;
  const int stages = kRing / (kABytes + b_bytes) < kMaxStages ? static_cast<int>(kRing / (kABytes + b_bytes)) : kMaxStages;
  const uint32_t b_ring = base + static_cast<uint32_t>(stages) * kABytes;
  const uint32_t part_ld = static_cast<uint32_t>(p.r) + 4u;
  int ring = 0;                 // stage and parity of the next k-step (producer, MMA)
  uint32_t parity = 0u;
  bool ok = true;
  uint32_t acc_phase = 0u;

  if (warp >= 6 && p.lists && blockIdx.x == 0 && z == 0 && (m_tile * p.tile_rows) % p.list_rows == 0)
    build_lists(p, m_tile * p.tile_rows / p.list_rows, lists_s, static_cast<int>(threadIdx.x) - 192);
  if (warp >= 6 && p.rows.list) {
    // From the last CTA on: the first ones make the tile lists.
    const int ctas = static_cast<int>(gridDim.x * gridDim.y * gridDim.z);
    const int cta = ctas - 1 - static_cast<int>((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x);
    for (int a = cta; a < p.count; a += ctas)
      list_rows<kListThreads>(p.ids, p.m, a, p.rows, rows_count, static_cast<int>(threadIdx.x) - 192,
                              [] { named_barrier_sync(1, kListThreads); });
  }

  if (warp == 0) issued = __shfl_sync(0xffffffffu, issued, 0);
  for (int pass = static_cast<int>(blockIdx.x); pass < passes; pass += p.pass_ctas) {
    const int a0 = pass * p.per_pass;                                       // the pass's adapters
    const int na = listed - a0 < p.per_pass ? listed - a0 : p.per_pass;
    const int nu = na * per_adapter;
    // The pass's units: adapter and first rank column.
    if (warp < 6) {
      for (int u = threadIdx.x; u < nu; u += 192) {
        const int id = list[a0 + u / per_adapter], c = (u % per_adapter) * w;
        unit_list[u] = make_int2(id, c);
        if (loaders) unit_src[u] = p.R + static_cast<int64_t>(id) * p.kc * p.r + c;
      }
      named_barrier_sync(2, kThreads - kListThreads);
    }
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      for (int j = 0; j < steps && ok; ++j) {
        // The first pass's first copies of X are under way.
        const bool fresh = pass != static_cast<int>(blockIdx.x) || j >= issued;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[ring], parity ^ 1u, p.err, kErrTimeoutEmpty));
        if (!ok) break;
        if (elect_lane()) {
          mbar_arrive_expect_tx(&full[ring], static_cast<uint32_t>(p.tile_rows) * 128u +
                                                 (loaders ? 0u : static_cast<uint32_t>(nu) * unit_bytes));
          if (fresh) load_x(ring, j);
          if (!loaders) {
            const uint32_t b_s = b_ring + static_cast<uint32_t>(ring) * b_bytes;
            for (int u = 0; u < nu; ++u) {
              const int2 unit = unit_list[u];
              if (R_MN)
                tma_load_3d(b_s + static_cast<uint32_t>(u) * unit_bytes, &p.tmR, &full[ring], unit.y, (k_lo + j) * kBK,
                            unit.x);
              else
                tma_load_3d(b_s + static_cast<uint32_t>(u) * unit_bytes, &p.tmR, &full[ring], (k_lo + j) * kBK, unit.y,
                            unit.x);
            }
          }
        }
        if (fresh) ++issued;
        if (++ring == stages) {
          ring = 0;
          parity ^= 1u;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (ok) {
        // What a step does not change is kept in registers: descriptors
        // advance by additions (16-byte units).
        const uint32_t idesc = make_idesc(nu * w, false, R_MN);
        const uint64_t ad0 = smem_desc(base, 16u, 1024u);
        // MN-major units: [64 k-rows x w columns], one behind the other.
        const uint64_t bd0 = R_MN ? smem_desc_unit(b_ring, unit_bytes, static_cast<uint32_t>(16 * w), w)
                                  : smem_desc(b_ring, 16u, 1024u);
        const uint32_t b_step = R_MN ? static_cast<uint32_t>(2 * w) : 2u;
        for (int j = 0; j < steps; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[ring], parity, p.err, kErrTimeoutFullA));
          if (!ok) break;
          tc_fence_after();
          uint64_t ad = ad0 + static_cast<uint32_t>(ring) * (kABytes >> 4);
          uint64_t bd = bd0 + static_cast<uint32_t>(ring) * (b_bytes >> 4);
          if (elect_lane()) {
            umma_f16(tmem, ad, bd, idesc, j > 0 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < kBK / 16; ++kk) {
              ad += 2u;
              bd += b_step;
              umma_f16(tmem, ad, bd, idesc, 1u);
            }
            umma_commit(&empty[ring]);
          }
          if (++ring == stages) {
            ring = 0;
            parity ^= 1u;
          }
        }
        if (ok && elect_lane()) umma_commit(&acc_bar);
      }
    } else if (row_warp) {
      // ---------------------------------------------------------- adapter tiles
      if (loaders) {
        // Units of [64 k-rows x w columns] with rows of 2w bytes, consecutive
        // threads on consecutive 16-byte pieces: one of each unit per thread
        // (w = 16), or two 32 rows apart (w = 32).
        int done_ring = ring;                 // stage whose copies are waited for next
        const int row = t / (w / 8), c = t % (w / 8), sw = (row >> (w == 32 ? 1 : 2)) & (w / 8 - 1);
        const uint32_t dst = b_ring + static_cast<uint32_t>(row * 2 * w + ((c ^ sw) << 4));
        for (int j = 0; j < steps + kAhead && ok; ++j) {
          if (j < steps) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[ring], parity ^ 1u, p.err, kErrTimeoutEmpty));
            if (!ok) break;
            uint32_t at = dst + static_cast<uint32_t>(ring) * b_bytes;
            const int64_t kr = static_cast<int64_t>(k_lo + j) * kBK + row;
            // Rows past the end are zeros.
            const uint32_t in0 = kr < p.kc ? 16u : 0u, in1 = kr + 32 < p.kc ? 16u : 0u;
            const int64_t off0 = (in0 ? kr : 0) * p.r + c * 8, off1 = (in1 ? kr + 32 : 0) * p.r + c * 8;
#pragma unroll 4
            for (int u = 0; u < nu; ++u, at += unit_bytes) {
              const uint16_t *src = unit_src[u];
              cp_async16(at, src + off0, in0);
              if (w == 32) cp_async16(at + 2048u, src + off1, in1);
            }
            if (++ring == stages) {
              ring = 0;
              parity ^= 1u;
            }
          }
          cp_async_commit();
          if (j >= kAhead) {
            cp_async_wait<kAhead>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[done_ring]);
            if (++done_ring == stages) done_ring = 0;
          }
        }
        cp_async_wait<0>();
      }
      // ---------------------------------------------------------- epilogue
      if (ok) ok = mbar_wait_bounded(&acc_bar, acc_phase, p.err, kErrTimeoutAcc, 20000000000ull);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        // Each row's own columns, 16 at a time, into the idle ring; a warp
        // reads only the adapters its rows use.
        const int quad = warp & 3;
        const uint32_t row = static_cast<uint32_t>(quad * 32 + lane);
        const int own = slot_of[row] - a0;
        for (int i = 0; i < na; ++i) {
          if (!__any_sync(0xffffffffu, own == i)) continue;
          for (int c = 0; c < p.r; c += 16) {
            uint32_t v[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(i * p.r + c), v);
            if (own == i) {
              const uint32_t dst = base + (row * part_ld + static_cast<uint32_t>(c)) * 4u;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t q[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
                sts128(dst + 16u * static_cast<uint32_t>(j), q);
              }
            }
          }
        }
      }
    }
    acc_phase ^= 1u;
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    // This CTA's share of the tile's rows, four columns at a time, the peers'
    // partials added in rank order.
    {
      const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
      const int left = p.m - m_tile * p.tile_rows;
      const int valid = left < p.tile_rows ? left : p.tile_rows;
      const int lo = valid * rank / size, hi = valid * (rank + 1) / size;
      const int pieces = p.r / 4;
      for (int i = threadIdx.x; i < (hi - lo) * pieces; i += kThreads) {
        const int row = lo + i / pieces, col = 4 * (i % pieces);
        const int slot = slot_of[row];
        if (slot < a0 || slot >= a0 + na) continue;
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
        const float s = __ldg(p.scale + list[slot]);
        uint16_t *dst = p.out + (static_cast<int64_t>(m_tile) * p.tile_rows + row) * p.r + col;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc.x * s, acc.y * s), pack_bf16x2(acc.z * s, acc.w * s));
      }
    }
    // The partials' generic accesses come before the next pass's TMA writes.
    fence_proxy_async_smem();
    cluster_sync_all();
  }

  // Every issued copy has landed before the CTA may exit: the products waited
  // for them, unless there was none or a wait gave up.
  if (!ok) failed = 1;
  __syncthreads();
  if (threadIdx.x == 0 && (failed || passes == 0))
    for (int j = issued - stages < 0 ? 0 : issued - stages; j < issued; ++j) {
      // Without a pass nobody announced the copies.
      if (passes == 0) {
        mbar_arrive_expect_tx(&full[j], static_cast<uint32_t>(p.tile_rows) * 128u);
        for (int i = 0; loaders && i < 4; ++i) mbar_arrive(&full[j]);
      }
      mbar_wait_bounded(&full[j % stages], static_cast<uint32_t>(j / stages) & 1u, p.err, kErrTimeoutDrain);
    }

  // Rows without an adapter.
  if (blockIdx.x == 0 && z == 0) {
    const int left = p.m - m_tile * p.tile_rows;
    const int valid = left < p.tile_rows ? left : p.tile_rows;
    const int pieces = p.r / 8;
    for (int i = threadIdx.x; i < valid * pieces; i += kThreads) {
      const int row = i / pieces;
      if (slot_of[row] < 0)
        reinterpret_cast<uint4 *>(p.out + (static_cast<int64_t>(m_tile) * p.tile_rows + row) * p.r)[i % pieces] =
            make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kMaxCols))
                 : "memory");
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
  cfg.gridDim = dim3(static_cast<unsigned>(p.pass_ctas), static_cast<unsigned>(m_tiles),
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

size_t tile_lists_bytes(int64_t m, int32_t count) {
  const int64_t a = carve_tile_lists(nullptr, m, count, 128).bytes, b = carve_tile_lists(nullptr, m, count, 512).bytes;
  return static_cast<size_t>(a > b ? a : b);
}

TileLists carve_tile_lists(void *scratch, int64_t m, int32_t count, int32_t rows) {
  TileLists t{};
  t.base = static_cast<int32_t *>(scratch);
  t.rows = rows;
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
                              uint16_t *out, const TileLists *lists, const GroupRows *rows, MultiGrid next,
                              cudaStream_t stream) {
  ProjParams p{};
  if (rows) {
    // Two warps beside a projection of m rows have the time for about one
    // pass over the ids per adapter of theirs; a long batch's lists are made
    // by more threads first.
    if (m <= kRowsInside) {
      p.rows = *rows;
    } else {
      group_rows_kernel<<<static_cast<unsigned>(s.count), kRowsThreads, 0, stream>>>(s.ids, static_cast<int>(m), *rows);
      count_launches(1);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  p.width = unit_width(s.r);
  if (through_b ? p.width == 64 && !encode_bf16_stack_map(&p.tmR, s.B, s.count, kc, s.r, 64, 64)
                : !encode_bf16_stack_map(&p.tmR, s.A, s.count, s.r, kc, 64, static_cast<uint32_t>(p.width)))
    return cudaErrorInvalidValue;
  p.R = s.B;
  p.kc = kc;
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
  }
  // One CTA per SM.  64-row tiles where 128-row ones cannot fill the SMs with
  // clusters of 8; K is split over the largest clusters that all fit at once
  // (a second wave would double the time).  While that leaves SMs idle and a
  // tile may hold more adapters than one pass of 64 columns, passes stay that
  // narrow and go to CTAs of their own; otherwise they take all the columns
  // they can, so that X is read as few times as possible.
  int64_t most = s.count < kRows ? s.count : kRows;                  // adapters of a tile
  if (m < most) most = m;
  const int narrow = s.r < 64 ? 64 / s.r : 1, wide = kMaxCols / s.r;
  const auto tiles_of = [&](int64_t rows) { return (m + rows - 1) / rows; };
  int sms = 148;
  const int64_t free_sms = next.ctas > 0 ? 148 - next.ctas : 0;
  if (free_sms >= 16 && tiles_of(kRows) * ((most + wide - 1) / wide) * p.nk <= free_sms * next.steps)
    sms = static_cast<int>(free_sms);
  static ClusterFit fit[2];
  const void *kernel = through_b ? reinterpret_cast<const void *>(multi_proj_kernel<true>)
                                 : reinterpret_cast<const void *>(multi_proj_kernel<false>);
  p.tile_rows = tiles_of(kRows) * 16 <= sms ? 64 : kRows;
  if (most > p.tile_rows) most = p.tile_rows;
  const int64_t m_tiles = tiles_of(p.tile_rows);
  const int most_split = p.nk / 2 < 1 ? 1 : p.nk / 2 < 8 ? p.nk / 2 : 8;
  int clusters = 1;
  const int split = fit[through_b].split(kernel, kThreads, kSmemBytes, m_tiles, 1, most_split, &clusters, sms);
  const int64_t spare = clusters / m_tiles;              // clusters per tile
  p.per_pass = spare > 1 ? narrow : wide;
  while (p.per_pass < wide && (most + p.per_pass - 1) / p.per_pass > spare) ++p.per_pass;
  if (p.per_pass > most) p.per_pass = static_cast<int>(most);
  const int64_t max_passes = (most + p.per_pass - 1) / p.per_pass;
  p.pass_ctas = static_cast<int>(spare < 1 ? 1 : spare < max_passes ? spare : max_passes);
  if (!encode_bf16_map(&p.tmL, L, m, kc, 64, static_cast<uint32_t>(p.tile_rows))) return cudaErrorInvalidValue;
  return through_b ? launch<true>(p, static_cast<int>(m_tiles), split, stream)
                   : launch<false>(p, static_cast<int>(m_tiles), split, stream);
}

}  // namespace qlora
