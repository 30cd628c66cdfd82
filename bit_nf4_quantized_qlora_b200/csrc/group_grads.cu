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
// multi_lists.cu writes each group's row numbers in ascending order into
// slots of 64 (a group starts on a slot of its own); a slot whose rows are
// consecutive is one TMA box, any other is up to sixteen row-gathering TMA loads
// of four rows for each tile, shared out over three warps (one warp issues a load
// in about 50 cycles).  So the work is the rows themselves (plus the last slot's
// padding), in every order of the batch, and a group never reads another
// group's rows.  The pad rows of a group's last slot repeat one of its own rows
// and are zeroed in both tiles before the product (in one alone, an infinity of
// the repeated row would meet a zero).
//
// A CTA takes 128 columns of L, 64 columns of R and an equal share of the
// slots, whatever groups they belong to: a cluster of up to 8 CTAs covers all
// slots, as many as it takes to fill the SMs.  Inside its share it walks the
// groups with two accumulators in tensor memory, so the next group's products
// run while the last one's result is written.  Only a group that crosses the
// border of two shares is reduced across the cluster (its partials wait in
// tensor memory until the end, then go through distributed shared memory, in
// rank order: results do not depend on timing).  So the time follows the number
// of rows and not how they are spread over the groups.
//
// An M = 128, N = 64 product of K = 64 rows reads 16 KB of L: the kernel is
// bound by reading L once per 64 ranks (HBM, or L2 for r > 64) and, for many
// small groups, by writing their results.
//
// Checkpoint form: L's tile arrives as 64 x 128 codes (half the bytes); the
// eight epilogue warps expand it to the bf16 tile the product reads, half a
// block of 64 elements (one scale) per thread: one and a half integer and one
// packed floating-point instruction per element.  dA of 11008 x 64 from 4096
// rows: 33 us, 1.45 TB/s of codes, scales, U and dA; a CTA takes about 2700
// cycles a slot with two CTAs on the SM, a chain through the expand warps (two
// groups of four warps in turn, with two bf16 tiles, took the same time).
#include <cuda.h>

#include "act8.cuh"
#include "group_rows.cuh"
#include "internal.h"
#include "multi.cuh"
#include "split_reduce.cuh"

namespace qlora {
namespace {

constexpr int kSlot = kSlotRows;          // rows of a step
constexpr int kEpiWarps = 8;              // expand / result warps: four lane quadrants x two column halves
constexpr int kFirstGather = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kFirstGather + 2);   // and a TMA warp, an MMA warp, two gather warps
constexpr uint32_t kLBytes = 128u * kSlot * 2u;   // bf16 tile: two 64-column slabs
constexpr uint32_t kRBytes = 64u * kSlot * 2u;
constexpr uint32_t kCBytes = 128u * kSlot;        // code tile
constexpr uint32_t kPartLd = 64u + 4u;
constexpr uint32_t kPartBytes = 128u * kPartLd * 4u;
// Accumulators: two in turn, and one for the group that began in an earlier
// share, which keeps its partial until the end.
constexpr uint32_t kLeftAcc = 2u;
constexpr uint32_t kTmemCols = 256u;

template <bool ACT8>
constexpr int stages() { return ACT8 ? 3 : 4; }
template <bool ACT8>
constexpr uint32_t stage_bytes() { return kLBytes + kRBytes + (ACT8 ? kCBytes : 0u); }
constexpr uint32_t kRing = stage_bytes<false>() * stages<false>();
constexpr uint32_t kSmem = kRing + 1024u;
static_assert(kRing == stage_bytes<true>() * stages<true>(), "the two forms share a kernel");
static_assert(2u * (kSmem + 4096u) <= 227u * 1024u, "two CTAs per SM");
static_assert(kRing >= 2u * kPartBytes, "room for two fp32 partial tiles");

struct __align__(64) GroupParams {
  CUtensorMap tmL, tmLg;        // L by boxes of 64 rows / by single rows
  CUtensorMap tmR, tmRg;        // R likewise
  const uint16_t *scale;        // checkpoint scales [m x P / 64]
  RowSlots rows;
  uint16_t *out;                // [groups x P x r], or [groups x r x P] transposed
  unsigned *err;
  int64_t P;
  int r, rtiles;
};

// The warp's 32 accumulator columns of this thread's row.
__device__ __forceinline__ void read_acc(uint32_t tmem, uint32_t acc, int quad, int half, uint32_t (&v)[32]) {
  tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 64u + static_cast<uint32_t>(half * 32), v);
}

// Writes 32 ranks from r0 on of the thread's row (column p of L) of a group's
// result.
template <bool OUT_T>
__device__ __forceinline__ void write_result(uint16_t *out, int64_t P, int r, int64_t row, int r0,
                                             const uint32_t (&v)[32]) {
  if (!OUT_T) {
    if (row < P) {
      uint4 *dst = reinterpret_cast<uint4 *>(out + row * r + r0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r0 + 8 * j < r)
          dst[j] = make_uint4(pack_bf16x2(__uint_as_float(v[8 * j]), __uint_as_float(v[8 * j + 1])),
                              pack_bf16x2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3])),
                              pack_bf16x2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5])),
                              pack_bf16x2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7])));
    }
  } else {
    // Transposed: lanes hold consecutive columns of the output.  Neighbours
    // exchange one of two rows, so each stores a pair of columns (P is even).
    const bool odd = lane_id() & 1u;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
      const uint32_t w = odd ? pack_bf16x2(__uint_as_float(got), __uint_as_float(v[j + 1]))
                             : pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(got));
      const int64_t rr = r0 + j + (odd ? 1 : 0);
      if (rr < r && row < P) *reinterpret_cast<uint32_t *>(out + rr * P + (row & ~int64_t(1))) = w;
    }
  }
}

// Puts the thread's 32 columns (from col0 on) of a partial into shared memory,
// along the output's contiguous dimension.
template <bool OUT_T>
__device__ __forceinline__ void store_partial(uint32_t dst, uint32_t row, uint32_t col0, const uint32_t (&v)[32]) {
  if (!OUT_T) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
      sts128(dst + (row * kPartLd + col0 + 4u * static_cast<uint32_t>(j)) * 4u, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + ((col0 + static_cast<uint32_t>(j)) * 128u + row) * 4u), "r"(v[j])
                   : "memory");
  }
}

// One CTA's tile of one product.
template <bool ACT8, bool OUT_T>
__device__ __forceinline__ void group_tile(const GroupParams &p, int tile) {
  constexpr int kStages = stages<ACT8>();
  constexpr uint32_t kStageBytes = stage_bytes<ACT8>();
  constexpr uint32_t kIdesc = make_idesc(64, true, true);
  constexpr int kParts = 3;                   // warps that fill a slot
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full[kStages], expanded[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t acc_full[3], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ Part left_s, right_s;
  __shared__ int4 gather[3][kSlot / 4];
  __shared__ uint2 scale_s[ACT8 ? kStages : 1][kSlot / 2];    // per row, its scales of the tile's two blocks

  const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p_tile = tile / p.rtiles, r_tile = tile % p.rtiles;
  // All slots, and this CTA's share of them.
  const int slots = slot_count(p.rows);
  const int z = static_cast<int>(blockIdx.z), nz = static_cast<int>(gridDim.z);
  // No CTA between two with slots is without: a group that crosses borders is
  // finished by consecutive CTAs, each with a partial.
  const int busy = slots < nz ? (slots > 0 ? slots : 1) : nz;
  const auto share = [&](int i) { return i < busy ? static_cast<int>((static_cast<int64_t>(slots) * i) / busy) : slots; };
  const int lo = share(z), hi = share(z + 1);
  const int p0 = p_tile * 128, r0 = r_tile * 64;
  // Second 64-column slab; past P it repeats the first (its output rows are
  // never stored) and every copy stays in range.
  const int p1 = p0 + 64 < p.P ? p0 + 64 : p0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kParts);
      mbar_init(&expanded[s], kEpiWarps);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&acc_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&acc_empty[i], kEpiWarps);
    fence_mbar_init();
    left_s = right_s = Part{0, 0, 0, 0, 0};
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

  if (ACT8 && warp == kFirstGather + 1) {
    // ------------------------------------------------------------ scales
    // Two rows a lane; requested a slot ahead, their row numbers two.  (In the
    // expand warps these loads were what a slot's proxy fence waited for.)
    SlotWalk walk(p.rows, lo, hi);
    const int64_t kb = p.P / 64, cb = static_cast<int64_t>(p_tile) * 2;
    const auto rows_of = [&](int slot) {
      const int64_t i = static_cast<int64_t>(slot) * kSlot + 2 * lane;
      if (slot < 0) return make_int2(-1, -1);
      if (p.rows.list) return __ldcg(reinterpret_cast<const int2 *>(p.rows.list + i));
      return make_int2(i < p.rows.m ? static_cast<int>(i) : -1, i + 1 < p.rows.m ? static_cast<int>(i + 1) : -1);
    };
    // Packed only when they are stored: arithmetic here would wait for the loads.
    const auto scales_of = [&](const int2 &row) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      const uint16_t *x = p.scale + static_cast<int64_t>(row.x) * kb + cb, *y = p.scale + static_cast<int64_t>(row.y) * kb + cb;
      if (row.x >= 0) v.x = __ldcg(x);
      if (row.x >= 0 && cb + 1 < kb) v.y = __ldcg(x + 1);
      if (row.y >= 0) v.z = __ldcg(y);
      if (row.y >= 0 && cb + 1 < kb) v.w = __ldcg(y + 1);
      return v;
    };
    int slot = walk.next(), slot1 = slot < 0 ? -1 : walk.next(), slot2 = slot1 < 0 ? -1 : walk.next();
    const int2 row = rows_of(slot), row1 = rows_of(slot1);
    int2 row2 = rows_of(slot2);
    uint4 v = scales_of(row), v1 = scales_of(row1);
    for (int li = 0; slot >= 0; ++li) {
      const int s = li % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], (static_cast<uint32_t>(li / kStages) & 1u) ^ 1u, p.err,
                                                     kErrTimeoutEmpty)))
        break;
      scale_s[s][lane] = make_uint2(v.x | v.y << 16, v.z | v.w << 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      v = v1;
      v1 = scales_of(row2);
      slot = slot1;
      slot1 = slot2;
      slot2 = slot2 < 0 ? -1 : walk.next();
      row2 = rows_of(slot2);
    }
  } else if (warp == 0 || warp >= kFirstGather) {
    // ------------------------------------------------------------ producers
    // Warp 0 announces a slot's bytes and copies boxes; gathers are shared
    // out: L's two slabs (or its codes) and R, a warp each.  Every one of them
    // takes part in every slot, so that none can run ahead of the others or
    // fall behind by a whole phase of a stage.
    const int part = warp == 0 ? 0 : warp - kFirstGather + 1;
    SlotWalk walk(p.rows, lo, hi);
    const auto rows_in = [&](int slot) {
      const int left = walk.part.rows - (slot - walk.part.s) * kSlot;
      return left < kSlot ? left : kSlot;
    };
    // A slot's rows, four per lane on lanes 0..15; requested a slot ahead.
    const auto rows_of = [&](int slot) {
      const int r4 = slot * kSlot + 4 * lane;
      if (!p.rows.list || slot < 0 || lane >= 16) return make_int4(r4, r4 + 1, r4 + 2, r4 + 3);
      return __ldcg(reinterpret_cast<const int4 *>(p.rows.list + static_cast<int64_t>(slot) * kSlot) + lane);
    };
    int issued = 0;
    int slot = walk.next(), valid_next = rows_in(slot);
    int4 ahead = rows_of(slot);
    while (slot >= 0) {
      const int4 idx = ahead;
      const int s = issued % kStages, valid = valid_next;
      const uint32_t ph = (static_cast<uint32_t>(issued / kStages) & 1u) ^ 1u;
      slot = walk.next();
      valid_next = rows_in(slot);
      ahead = rows_of(slot);
      ++issued;
      const int first = __shfl_sync(0xffffffffu, idx.x, 0);
      const int want = first + 4 * lane;
      const bool in_order = idx.x == want && idx.y == want + 1 && idx.z == want + 2 && idx.w == want + 3;
      const bool box = __all_sync(0xffffffffu, lane >= 16 || in_order) != 0;
      const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
      const uint32_t r_s = l_s + kLBytes, c_s = r_s + kRBytes;
      // The product takes whole 16s of rows.
      const uint32_t chunks = box ? kSlot / 16u : static_cast<uint32_t>(valid + 15) / 16u;
      if (!box) {
        __syncwarp();
        if (lane < 16) gather[part][lane] = idx;
        __syncwarp();
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ph, p.err, kErrTimeoutEmpty))) {
        --issued;
        break;
      }
      if (elect_lane()) {
        if (part == 0) mbar_arrive_expect_tx(&full[s], chunks * ((ACT8 ? kCBytes : kLBytes) + kRBytes) / (kSlot / 16u));
        if (box && part > 0) {
          // Warp 0's.
        } else if (box) {
          if (ACT8) {
            tma_load_2d(c_s, &p.tmL, &full[s], p0, first);
          } else {
            tma_load_2d(l_s, &p.tmL, &full[s], p0, first);
            tma_load_2d(l_s + 8192u, &p.tmL, &full[s], p1, first);
          }
          tma_load_2d(r_s, &p.tmR, &full[s], r0, first);
        } else {
          const bool right = part == (ACT8 ? 1 : 2);
          const CUtensorMap *map = right ? &p.tmRg : &p.tmLg;
          const uint32_t dst = right ? r_s : ACT8 ? c_s : l_s + static_cast<uint32_t>(part) * 8192u;
          const int x = right ? r0 : part == 1 ? p1 : p0;
          for (uint32_t i = 0; i < 4u * chunks; ++i)     // four rows of 128 bytes
            tma_gather4(dst + i * 512u, map, &full[s], x, gather[part][i]);
        }
        if (part > 0) mbar_arrive(&full[s]);
      }
    }
    __syncwarp();
    // Every issued copy has landed before the CTA may exit.
    if (part == 0 && lane == 0)
      for (int li = issued - kStages < 0 ? 0 : issued - kStages; li < issued; ++li)
        mbar_wait_bounded(&full[li % kStages], static_cast<uint32_t>(li / kStages) & 1u, p.err, kErrTimeoutDrain);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    GroupWalk walk(p.rows, lo, hi);
    Part part;
    int ok = 1, turn = 0, s = 0;
    uint32_t parity = 0u;
    const uint64_t ld0 = smem_desc(base, 8192u, 1024u), rd0 = smem_desc(base + kLBytes, 8192u, 1024u);
    const auto ready = [&]() {
      return __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], parity, p.err, kErrTimeoutFullA) &&
                                         (!ACT8 || mbar_wait_bounded(&expanded[s], parity, p.err, kErrTimeoutFullB)));
    };
    // The products of 16 `chunks` rows of slot s.
    const auto multiply = [&](uint32_t acc, bool first, int chunks) {
      tc_fence_after();
      uint64_t ld = ld0 + static_cast<uint32_t>(s) * (kStageBytes >> 4), rd = rd0 + static_cast<uint32_t>(s) * (kStageBytes >> 4);
      if (elect_lane()) {
        umma_f16(acc, ld, rd, kIdesc, first ? 0u : 1u);
        for (int kk = 1; kk < chunks; ++kk) {
          ld += 2048u / 16u;
          rd += 2048u / 16u;
          umma_f16(acc, ld, rd, kIdesc, 1u);
        }
        umma_commit(&empty[s]);
      }
    };
    const auto advance = [&]() {
      if (++s == kStages) {
        s = 0;
        parity ^= 1u;
      }
    };
    while (ok && walk.next(&part)) {
      const bool left = part.from_left();
      const uint32_t buf = left ? kLeftAcc : static_cast<uint32_t>(turn & 1);
      const uint32_t acc = tmem + buf * 64u;
      // Whole slots, then (if it is in this share) a last one with pad rows.
      const int whole = p.rows.list ? part.s + part.rows / kSlot : part.e;
      const int stop = whole < part.e ? whole : part.e;
      if (!left)
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_empty[buf], (static_cast<uint32_t>(turn >> 1) & 1u) ^ 1u, p.err,
                                                       kErrTimeoutAcc));
      for (int slot = part.b; slot < stop && ok; ++slot) {
        ok = ready();
        if (!ok) break;
        multiply(acc, slot == part.b, kSlot / 16);
        advance();
      }
      if (!left) ++turn;
      if (stop < part.e) {
        ok = ok && ready();
        if (ok) {
          // Zero rows of L's two slabs and of R, as far as the product reads:
          // whole 128-byte rows, so the swizzle inside them does not matter.
          const int valid = part.rows % kSlot, chunks = (valid + 15) / 16;
          const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
          const uint32_t zero[4] = {0u, 0u, 0u, 0u};
          for (int c = valid * 8 + lane; c < chunks * 128; c += 32) {
            const uint32_t at = l_s + static_cast<uint32_t>(c) * 16u;
            sts128(at, zero);
            sts128(at + kLBytes / 2u, zero);
            sts128(at + kLBytes, zero);
          }
          fence_proxy_async_smem();
          __syncwarp();
          multiply(acc, stop == part.b, chunks);
          advance();
        }
      }
      if (ok && elect_lane()) umma_commit(&acc_full[buf]);
    }
  } else {
    const int t = static_cast<int>(threadIdx.x) - 64;
    bool ok = true;
    // The expansion and the results share these warps: after a group's last
    // slot is expanded its result is not waited for until the next group's
    // slots that fit the ring are expanded too.
    const int quad = warp & 3, half = (warp - 2) >> 2;      // TMEM lanes, 32 of the 64 columns
    const uint32_t row = static_cast<uint32_t>(quad * 32 + lane);
    const int rc = r0 + 32 * half;
    GroupWalk results(p.rows, lo, z + 1 == nz ? 0x7FFFFFFF : hi);
    int turn = 0;
    Part part;
    bool more = results.next(&part, true);
    int done = 0;            // slots of the groups before `part`
    // Writes the results of groups whose slots are all among the first
    // `expanded_slots` of the share.
    const auto flush = [&](int expanded_slots) {
      while (ok && more && done + (part.live() ? part.e - part.b : 0) <= expanded_slots) {
        uint16_t *out = p.out + static_cast<int64_t>(part.group) * p.P * p.r;
        if (!part.live()) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
          write_result<OUT_T>(out, p.P, p.r, p0 + row, rc, v);
        } else if (part.from_left()) {
          if (t == 0) left_s = part;
        } else {
          if (part.to_right()) {
            if (t == 0) right_s = part;
          } else {
            ok = mbar_wait_bounded(&acc_full[turn & 1], static_cast<uint32_t>(turn >> 1) & 1u, p.err, kErrTimeoutAcc,
                                   20000000000ull);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            tc_fence_after();
            uint32_t v[32];
            read_acc(tmem, static_cast<uint32_t>(turn & 1), quad, half, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[turn & 1]);
            write_result<OUT_T>(out, p.P, p.r, p0 + row, rc, v);
          }
          ++turn;
        }
        if (part.live()) done += part.e - part.b;
        more = results.next(&part, true);
      }
    };
    if (ACT8) {
      // ---------------------------------------------------------- expand
      // Thread t: row t / 4 of the slot, 32-column quarter t % 4.
      const int erow = t >> 2, quarter = t & 3, slab = quarter >> 1;
      const uint32_t sw = static_cast<uint32_t>(erow & 7);
      SlotWalk walk(p.rows, lo, hi);
      for (int li = 0; walk.next() >= 0; ++li) {
        const int s = li % kStages;
        const uint32_t ph = static_cast<uint32_t>(li / kStages) & 1u;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], ph, p.err, kErrTimeoutFullA));
        if (!ok) break;
        const uint2 sc = scale_s[s][erow >> 1];
        const uint32_t s2 = (((erow & 1 ? sc.y : sc.x) >> (16 * slab)) & 0xFFFFu) * 0x10001u;
        const uint32_t l_s = base + static_cast<uint32_t>(s) * kStageBytes;
        const uint32_t code_row = l_s + kLBytes + kRBytes + static_cast<uint32_t>(erow) * 128u;
        const uint32_t out_row = l_s + static_cast<uint32_t>(slab) * 8192u + static_cast<uint32_t>(erow) * 128u;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          // 16 codes -> two 16-byte chunks; the slabs walk them in an order
          // that keeps a quarter-warp's stores in distinct bank groups.
          const uint32_t j = static_cast<uint32_t>(jj ^ slab), at = 4u * (quarter & 1) + 2u * j;
          const uint4 c = lds128(code_row + (((2u * quarter + j) ^ sw) << 4));
          uint32_t o[4];
          act8_decode4(c.x, s2, o[0], o[1]);
          act8_decode4(c.y, s2, o[2], o[3]);
          sts128(out_row + ((at ^ sw) << 4), o);
          act8_decode4(c.z, s2, o[0], o[1]);
          act8_decode4(c.w, s2, o[2], o[3]);
          sts128(out_row + (((at + 1u) ^ sw) << 4), o);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&expanded[s]);
        // Results two slots late: their products have had time to finish.
        flush(li - 1);
        if (!ok) break;
      }
    }
    // ------------------------------------------------------------ results
    if (ok) flush(0x7FFFFFFF);
    // Partials of the groups that cross the share's borders, into the idle
    // ring: every product of the share is done once the last accumulator is.
    named_barrier_sync(1, 32 * kEpiWarps);
    const bool left = left_s.live(), right = right_s.live();
    if (ok && right)
      ok = mbar_wait_bounded(&acc_full[(turn - 1) & 1], static_cast<uint32_t>((turn - 1) >> 1) & 1u, p.err,
                             kErrTimeoutAcc, 20000000000ull);
    if (ok && left) ok = mbar_wait_bounded(&acc_full[kLeftAcc], 0u, p.err, kErrTimeoutAcc, 20000000000ull);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && (left || right)) {
      tc_fence_after();
      uint32_t v[32];
      if (left) {
        read_acc(tmem, kLeftAcc, quad, half, v);
        store_partial<OUT_T>(base, row, 32u * half, v);
      }
      if (right) {
        read_acc(tmem, static_cast<uint32_t>((turn - 1) & 1), quad, half, v);
        store_partial<OUT_T>(base + kPartBytes, row, 32u * half, v);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (nz > 1) {
    cluster_sync_all();
    // A crossing group is finished by all CTAs that hold a part of it, each
    // an equal share of the tile in 16-byte pieces: the CTA where it starts
    // holds its partial in the second buffer, the others in the first.
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const Part c = side == 0 ? left_s : right_s;
      if (!c.live()) continue;
      int zs = 0, ze = 0;
      for (int i = 0; i < nz; ++i) {
        if (share(i) <= c.s) zs = i;
        if (share(i) <= c.s + c.slots() - 1) ze = i;
      }
      const int n = ze - zs + 1;
      uint16_t *out = p.out + static_cast<int64_t>(c.group) * p.P * p.r;
      const int hi_i = 2048 * (z - zs + 1) / n;
      for (int i = 2048 * (z - zs) / n + static_cast<int>(threadIdx.x); i < hi_i; i += kThreads) {
        // (row, 4 ranks) for a row-major result, (rank, 4 columns) transposed.
        const uint32_t off = OUT_T ? static_cast<uint32_t>(i) * 16u
                                   : (static_cast<uint32_t>(i / 16) * kPartLd + 4u * static_cast<uint32_t>(i % 16)) * 4u;
        float4 part[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          part[q] = q < n ? ld_dsmem_v4(base + off + (q == 0 ? kPartBytes : 0u), static_cast<uint32_t>(zs + q))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 acc = part[0];
#pragma unroll
        for (int q = 1; q < 8; ++q) {
          if (q < n) {
            acc.x += part[q].x;
            acc.y += part[q].y;
            acc.z += part[q].z;
            acc.w += part[q].w;
          }
        }
        const uint2 w = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        const int64_t pr = OUT_T ? p0 + 4 * (i % 32) : p0 + i / 16;
        const int rr = OUT_T ? r0 + i / 32 : r0 + 4 * (i % 16);
        if (pr >= p.P || rr >= p.r) continue;
        *reinterpret_cast<uint2 *>(out + (OUT_T ? static_cast<int64_t>(rr) * p.P + pr : pr * p.r + rr)) = w;
      }
    }
    cluster_sync_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// dA's tiles (transposed, L = X or its checkpoint), then dB's (L = dY): one
// launch, so that neither product's last tiles leave the SMs idle.
struct __align__(64) GradsParams {
  GroupParams da, db;
  int da_tiles;
};
template <bool ACT8>
__global__ void __launch_bounds__(kThreads, 2) group_grads_kernel(const __grid_constant__ GradsParams p) {
  const int tile = static_cast<int>(blockIdx.x);
  if (tile < p.da_tiles)
    group_tile<ACT8, true>(p.da, tile);
  else
    group_tile<false, false>(p.db, tile - p.da_tiles);
  // Started beside the input gradient (see launch): what comes next on the
  // stream may rely on that one too, so this grid does not end before it.
  griddep_wait();
}

template <bool ACT8>
cudaError_t launch(const GradsParams &p, int tiles, int64_t slots, bool beside, cudaStream_t stream) {
  static std::atomic<bool> configured[kMaxDevicesPerProcess] = {};
  static ClusterFit fit;
  const void *kernel = reinterpret_cast<const void *>(group_grads_kernel<ACT8>);
  cudaError_t e = set_smem_once(kernel, static_cast<int>(kSmem), configured);
  if (e != cudaSuccess) return e;
  // Two slots to a CTA at least; the largest clusters that all fit at once.
  const int most_split = static_cast<int>(slots / 2 < 1 ? 1 : slots / 2 < 8 ? slots / 2 : 8);
  int clusters = 1;
  const int split = fit.split(kernel, kThreads, static_cast<int>(kSmem), tiles, 2, most_split, &clusters);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(split);
  // The input gradient before it lets this grid start once all of its CTAs run
  // and what both of them read is complete: it takes the SMs that the last wave
  // leaves idle.
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, group_grads_kernel<ACT8>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// The parameters of one product; null on failure.
bool group_params(GroupParams *p, const uint16_t *L, const Act8View *L8, int64_t m, int64_t P, const uint16_t *R,
                  int32_t r, const GroupRows *g, uint16_t *out) {
  if (L8) {
    const uint8_t *codes = reinterpret_cast<const uint8_t *>(L8->codes);
    if (!encode_codes_map(&p->tmL, codes, m, P, 128, kSlot, true)) return false;
    if (!encode_codes_map(&p->tmLg, codes, m, P, 128, 1, true)) return false;
    p->scale = L8->scale;
  } else {
    if (!encode_bf16_map(&p->tmL, L, m, P, 64, kSlot)) return false;
    if (!encode_bf16_map(&p->tmLg, L, m, P, 64, 1)) return false;
  }
  if (!encode_bf16_map(&p->tmR, R, m, r, 64, kSlot)) return false;
  if (!encode_bf16_map(&p->tmRg, R, m, r, 64, 1)) return false;
  p->rows = row_slots(g, m);
  p->out = out;
  p->err = device_error_word();
  p->P = P;
  p->r = r;
  p->rtiles = (r + 63) / 64;
  return true;
}

}  // namespace

cudaError_t launch_group_grads(const uint16_t *X, const Act8View *X8, const uint16_t *U, int64_t k, uint16_t *dA,
                               const uint16_t *dY, const uint16_t *T, int64_t n, uint16_t *dB, int64_t m, int32_t r,
                               const GroupRows *g, bool beside, cudaStream_t stream) {
  GradsParams p{};
  if (!group_params(&p.da, X, X8, m, k, U, r, g, dA)) return cudaErrorInvalidValue;
  if (dB && !group_params(&p.db, dY, nullptr, m, n, T, r, g, dB)) return cudaErrorInvalidValue;
  p.da_tiles = static_cast<int>((k + 127) / 128) * p.da.rtiles;
  const int tiles = p.da_tiles + (dB ? static_cast<int>((n + 127) / 128) * p.db.rtiles : 0);
  // At most m / 64 slots, and one more for every group with rows.
  const int64_t slots = m / kSlot + (p.da.rows.groups < m ? p.da.rows.groups : m);
  return X8 ? launch<true>(p, tiles, slots, beside, stream) : launch<false>(p, tiles, slots, beside, stream);
}

}  // namespace qlora
