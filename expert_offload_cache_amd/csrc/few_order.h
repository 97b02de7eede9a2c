// moe_layer_few: how many work items of each kind a call has and in which order they are handed out (plain C++:
// the order is what launch 2's waits rest on, and is checked on the host).
//
// Items of a kind are numbered c + kLists v: the v-th of list c, 0 <= v < list_items(c).  A list is handed out in
// ascending v by a counter.
// A down item is one run of a row block of y; the workgroup of run 0 adds the other runs' sums and waits for them.  All
// runs of a row block lie in ONE list, the last run first, so that they are handed out before the run
// that waits for them, whatever the number of row blocks: see "Why every wait ends" in few.hip.
#pragma once

#include <cstddef>
#include <cstdint>

#include "moe.h"

namespace moe {

constexpr int kFewUnits = 256;  // compute units: launch 2 has a workgroup for each
constexpr int kFewWaves = 8;    // of a workgroup of launch 2
constexpr int kLists = 8;       // counters of each kind, a cache line each: one word takes 11 ns an increment

// Things 0 .. total - 1 dealt to the lists in turn: those of list c
constexpr int list_share(int total, int c) { return (total - c + kLists - 1) / kLists; }
// items of list c: `runs` for each thing (gate/up items: one)
constexpr int list_items(int total, int runs, int c) { return list_share(total, c) * runs; }

struct DownItem {
    int block, run;
};
// down item `id` (c + kLists v) of a call with `blocks` row blocks of `runs` runs
constexpr DownItem down_item(int id, int blocks, int runs) {
    const int c = id % kLists, v = id / kLists, n = list_share(blocks, c);
    return {c + kLists * (v % n), runs - 1 - v / n};
}

// Columns of y of a down item, in blocks of 16: one where the call's rows of h are few (every unit takes in all of
// them), four elsewhere.
constexpr int few_row_blocks(int T, int f, int k, bool shared, moe_dtype w) {
    const size_t rows = (size_t)T * k + (shared ? T : 0);
    return rows * f * (w == MOE_F32 ? 4 : 2) <= ((size_t)48 << 10) ? 1 : 4;
}
// Runs of a row block: as many as give every one of 256 workgroups an item, while a wave has two steps
// and more.
constexpr int few_splits(int T, int d, int f, int E, int k, bool shared, moe_dtype w) {
    const int items = (T * k < E ? T * k : E) + (shared ? 1 : 0), rb = few_row_blocks(T, f, k, shared, w);
    const int64_t steps = (int64_t)items * (f / (w == MOE_F32 || w == MOE_BF16 ? 32 : 128));
    int s = 1;
    while (s < 16 && 2 * s * (d / (16 * rb)) <= kFewUnits && steps >= (int64_t)2 * s * kFewWaves * 2) s *= 2;
    return s;
}

}  // namespace moe
