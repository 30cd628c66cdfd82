// The row lists of a batch whose rows belong to different adapters:
//
//   tile lists   the adapters of each tile of the main product, and which of
//                its rows are whose (the lane masks of the masked products)
//   row lists    each adapter's rows in ascending order, in slots of 64, for
//                the products that gather them (the projections, the adapter
//                gradients)
//
// One launch makes both, and writes the zeros of T and U for rows without an
// adapter: a CTA per tile, then a CTA per adapter of the set that scans the ids
// twice, whether it has rows or not.  With few adapters it is bound by its
// latency (4096 rows, 8 adapters: 7 to 8 us captured alone, and the projection's
// prologue runs beside it); the scans cost count . m id reads, and a slot index
// for every adapter that the projection and the gradients step over: forward of
// 4096 rows of 8 adapters through 4096 x 4096, r = 16: 132 us with 8 in the set,
// 147 with 1000, 275 with 10000; of 4096 rows through 64 x 64: 818 with 65535.
#include "internal.h"
#include "multi.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct ListParams {
  const int32_t *ids;
  int m, count, r;
  TileLists tiles;
  GroupRows rows;
  uint16_t *zero[2];      // [m x r] results whose rows without an adapter are zeroed (null: none)
};

__device__ __forceinline__ int row_id(const ListParams &p, int64_t row) {
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

// A tile's arrays: ids, table place and slot of up to 512 rows, and the table
// (key, first row).
struct ListSmem {
  int id[512], place[512], slot[512], key[1024], first[1024];
};

// One tile's adapters and row masks (layout: see TileLists).  A row leads if it
// is its id's first; leaders are numbered in row order.
__device__ void build_lists(const ListParams &p, int tile, ListSmem &s, int t) {
  const int n = p.tiles.rows, words = n / 32, lane = t & 31;
  for (int i = t; i < 1024; i += kThreads) {
    s.key[i] = -1;
    s.first[i] = 0x7FFFFFFF;
  }
  for (int i = t; i < n; i += kThreads) s.id[i] = row_id(p, static_cast<int64_t>(tile) * n + i);
  __syncthreads();
  for (int i = t; i < n; i += kThreads)
    if (s.id[i] >= 0) s.place[i] = table_add<1024>(s.key, s.first, s.id[i], i);
  __syncthreads();
  int32_t *out = p.tiles.base + tile * p.tiles.stride;
  uint32_t *mask = reinterpret_cast<uint32_t *>(out + 4 + p.tiles.slots);
  // Every warp numbers the leaders; each stores its share of the entries.
  int total = 0;
  for (int c = 0; c < words; ++c) {
    const int i = 32 * c + lane;
    const bool lead = s.id[i] >= 0 && s.first[s.place[i]] == i;
    const unsigned b = __ballot_sync(0xffffffffu, lead);
    const int at = total + __popc(b & ((1u << lane) - 1u));
    if (lead && c % kWarps == t >> 5) {
      s.slot[i] = at;
      out[4 + at] = s.id[i];
    }
    total += __popc(b);
  }
  if (t == 0) out[0] = total;
  for (int i = t; i < total * words; i += kThreads) mask[i] = 0u;
  __syncthreads();
  // A mask word per (adapter, 32 rows) that has a row, from the lanes that
  // hold the same id.
  for (int c = t >> 5; c < words; c += kWarps) {
    const int i = 32 * c + lane, id = s.id[i];
    const unsigned same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0u) mask[s.slot[s.first[s.place[i]]] * words + c] = same;
  }
}

// The rows of adapter a in ascending order (layout: see GroupRows), by
// warps that take contiguous runs of rows and count by ballots: no atomics, so
// the order is fixed.  Adapter a's list starts at entry
// 64 (floor(b / 64) + a), b the number of rows with a lower id: such a list of
// c entries padded to a multiple of 64 ends before adapter a + 1's starts, so
// nobody needs another adapter's count.
__device__ void list_rows(const int32_t *__restrict__ ids, int m, int a, const GroupRows &g, int t) {
  __shared__ int count_of[kWarps][2];
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
  __syncthreads();
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
}

__global__ void __launch_bounds__(kThreads) multi_lists_kernel(const ListParams p) {
  __shared__ ListSmem s;
  // The projection may start now; it waits for this grid before it reads a list.
  griddep_launch();
  const int t = static_cast<int>(threadIdx.x), tile = static_cast<int>(blockIdx.x);
  if (tile >= p.tiles.tiles) {
    list_rows(p.ids, p.m, tile - static_cast<int>(p.tiles.tiles), p.rows, t);
    return;
  }
  build_lists(p, tile, s, t);
  const int64_t first = static_cast<int64_t>(tile) * p.tiles.rows;
  const int pieces = p.r / 8;
  for (int i = t; i < p.tiles.rows * pieces; i += kThreads) {
    const int row = i / pieces;
    if (s.id[row] >= 0 || first + row >= p.m) continue;
#pragma unroll
    for (int z = 0; z < 2; ++z)
      if (p.zero[z])
        reinterpret_cast<uint4 *>(p.zero[z] + (first + row) * p.r)[i % pieces] = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace

GroupRows carve_group_rows(void *scratch, int32_t groups) {
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

cudaError_t launch_multi_lists(const AdapterView &s, int64_t m, const TileLists &tiles, const GroupRows &rows,
                               uint16_t *zero0, uint16_t *zero1, cudaStream_t stream) {
  const ListParams p{s.ids, static_cast<int>(m), s.count, s.r, tiles, rows, {zero0, zero1}};
  multi_lists_kernel<<<static_cast<unsigned>(tiles.tiles + s.count), kThreads, 0, stream>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qlora
