// Walks over the row lists of a batch of many adapters (sm_100a): each group's
// rows lie in slots of 64, a group starting on a slot of its own (GroupRows).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qlora {

constexpr int kSlotRows = 64;

// The lists as kernel parameters; one group of all m rows in order without.
struct RowSlots {
  const int32_t *list;          // row numbers (null: one group)
  const int32_t *start, *count; // first entry (a multiple of 64) and rows of each group
  int groups, m;
};
inline RowSlots row_slots(const GroupRows *g, int64_t m) {
  return g ? RowSlots{g->list, g->start, g->count, g->groups, static_cast<int>(m)}
           : RowSlots{nullptr, nullptr, nullptr, 1, static_cast<int>(m)};
}
// Slots up to the last group's end, those of empty groups among them.
__device__ __forceinline__ int slot_count(const RowSlots &p) {
  return p.list ? __ldcg(p.start + p.groups - 1) / kSlotRows + (__ldcg(p.count + p.groups - 1) + kSlotRows - 1) / kSlotRows
                : (p.m + kSlotRows - 1) / kSlotRows;
}

// A CTA's part of a group: slots [b, e) of the group's [s, s + slots()).
struct Part {
  int group, s, rows, b, e;
  __device__ __forceinline__ int slots() const { return (rows + kSlotRows - 1) / kSlotRows; }
  __device__ __forceinline__ bool live() const { return b < e; }
  __device__ __forceinline__ bool from_left() const { return b > s; }
  __device__ __forceinline__ bool to_right() const { return e < s + slots(); }
};

// Walks the groups whose first slot or any slot lies in [lo, hi), by whole
// warps; lane l holds group base + l.  Groups' first slots ascend strictly.
struct GroupWalk {
  const int32_t *start, *count;
  int groups, lo, hi, m;
  int a, base, s, c;
  __device__ __forceinline__ void window(int first) {
    base = first;
    const int g = first + static_cast<int>(lane_id());
    const bool in = g < groups;
    s = !in ? 0x7FFFFFFF : (start ? __ldcg(start + g) / kSlotRows : 0);
    c = !in ? 0 : (start ? __ldcg(count + g) : m);
  }
  __device__ __forceinline__ GroupWalk(const RowSlots &p, int lo_, int hi_)
      : start(p.start), count(p.count), groups(p.groups), lo(lo_), hi(hi_), m(p.m) {
    // The last group that starts at or before lo.
    int first = 0;
    for (int span = groups; span > 32;) {
      const int step = (span + 31) / 32, g = first + static_cast<int>(lane_id()) * step;
      const bool le = g < first + span && __ldcg(start + g) / kSlotRows <= lo;
      const int n = __popc(__ballot_sync(0xffffffffu, le));
      first += (n - 1) * step;
      span = groups - first < step ? groups - first : step;
    }
    window(first);
    a = first + __popc(__ballot_sync(0xffffffffu, s <= lo)) - 1;
  }
  // The next group with slots in the share, or (with `empty`) without rows;
  // false when there is none.
  __device__ __forceinline__ bool next(Part *p, bool empty = false) {
    for (;; ++a) {
      if (a >= groups) return false;
      if (a >= base + 32) window(a);
      const int gs = __shfl_sync(0xffffffffu, s, a - base), gc = __shfl_sync(0xffffffffu, c, a - base);
      if (gs >= hi) return false;
      const int end = gs + (gc + kSlotRows - 1) / kSlotRows;
      *p = Part{a, gs, gc, gs > lo ? gs : lo, end < hi ? end : hi};
      if (p->live() || (empty && gc == 0 && gs >= lo)) {
        ++a;
        return true;
      }
    }
  }
};

// The slots of a share in order.
struct SlotWalk {
  GroupWalk walk;
  Part part{0, 0, 0, 0, 0};
  __device__ __forceinline__ SlotWalk(const RowSlots &p, int lo, int hi) : walk(p, lo, hi) {}
  __device__ __forceinline__ int next() {
    if (part.b >= part.e && !walk.next(&part)) return -1;
    return part.b++;
  }
};

}  // namespace qlora
