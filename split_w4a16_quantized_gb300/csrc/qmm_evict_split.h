// How an eviction's columns (layer, sequence, KV head) are split over blocks; host only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace qmm {

constexpr int kEvictMoveThreads = 256;
// Slots of a column that a block's shared memory holds, 6 bytes each, two blocks an SM, and
// most blocks of a column.
constexpr int kEvictSlots = 16384;
constexpr int kEvictBlocks = 8;

struct EvictSplit {
    int slices, lanes;     // pieces of a row, 16 * lanes bytes each
    int movers;            // blocks of a column's piece
    int cluster, spread;   // blocks of a column; whether it takes them all
    int held;              // slots that a block's shared memory holds
};

// columns of cap slots to `keep`, row_lanes * 16 bytes a row.
inline EvictSplit evict_split(int64_t columns, int cap, int keep, int row_lanes, int num_sms) {
    EvictSplit s;
    // whole rows, or pieces of at least 64 bytes where the columns of K and V would leave SMs
    // idle (152 SMs; 576 columns of 256-byte rows, two pieces: 19.6 us, four 25.8; 16 sequences of 12
    // layers: whole rows 326, four pieces 400), and several blocks a piece where that is not enough
    const int64_t pools = 2 * columns;
    s.slices = 1;
    while (row_lanes / s.slices > 4 && pools * s.slices < 4 * num_sms) s.slices *= 2;
    s.lanes = row_lanes / s.slices;
    s.movers = 1;
    while (s.lanes == 4 && s.movers < kEvictBlocks && pools * s.slices * s.movers < 2 * num_sms &&
           keep / s.movers > kEvictMoveThreads)
        s.movers *= 2;
    // Blocks of a column: as many as its slots need, or more where the columns alone would
    // leave SMs idle.
    s.cluster = 1;
    s.spread = 0;
    while (s.cluster < kEvictBlocks && (cap - 1) / s.cluster + 1 > kEvictSlots) s.cluster *= 2;
    while (s.cluster < kEvictBlocks && columns * s.cluster < num_sms && cap / s.cluster > 2048) {
        s.cluster *= 2;
        s.spread = 1;
    }
    // A long table's columns take their whole cluster, however short, where all blocks run at
    // once (two an SM; 8 columns of 14000 slots in a table of 131,072: 20 us, as many blocks as
    // hold them 32; 32 columns 45 and 63; 2000 slots 15.1 and 14.0).
    if (s.cluster > 1 && columns * s.cluster <= 2 * num_sms) s.spread = 1;
    s.held = std::min(((cap - 1) / s.cluster + 64) / 64 * 64, kEvictSlots);
    return s;
}

}  // namespace qmm
