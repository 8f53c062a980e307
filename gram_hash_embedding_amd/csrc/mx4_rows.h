// Where a tile of the projection on 4-bit weights (wkv_mx4.hip) loads its token rows from: plain index arithmetic, which host
// code can follow too.
#pragma once

#include <stdint.h>

namespace engram {

// BM rows by NW waves, 128 bytes of each a stage (a step of 128 columns in 8 bits, two in 4), 16 bytes a lane and load: load q of a
// wave has rows first + 8 q .. + 7, lane l slot l % 8 of row l / 8 of them, which holds the 16-byte piece (l % 8) ^ (row / 2) % 8.
// A stage's resource begins with the tile's first byte of it and ends with the tile's last row, so that what a lane adds to its
// base is all that is looked up, checked against that end: rows past the last, and behind an odd count of 4-bit steps the last
// row's missing half of a stage, read as zeros.  (As a scalar offset the stage's column would have to be part of the check: it is
// on gfx950, where a lane is fetched if its offset is below the resource's size less the scalar one, or nothing is if that is
// none; the compiler's description of the load says that it is not.)
template <bool kA8, int BM, int NW>
struct Mx4Rows {
    static constexpr int kSub = kA8 ? 1 : 2;                         // steps of a stage
    static constexpr int kLoads = (BM + 8 * NW - 1) / (8 * NW);      // per wave and stage: 8 rows each
    static constexpr int row_bytes(int steps) { return steps * (kA8 ? 128 : 64); }
    // (with fewer rows than the waves load, some load the same)
    static constexpr int first(int wave) { return wave * kLoads * 8 % BM; }
    // a lane's offset in the even loads, or the odd ones (the key of an odd group of 8 rows is that of an even one plus 4), less
    // the load's own rows
    static constexpr uint32_t offset(int first, int lane, bool odd, int row_bytes) {
        const int row = first + (lane >> 3);
        const uint32_t piece = static_cast<uint32_t>(((lane & 7) ^ ((row >> 1) & 7)) << 4);
        return row * row_bytes + (odd ? piece ^ 64u : piece);
    }
    static constexpr uint32_t load_rows(int q, int row_bytes) { return static_cast<uint32_t>(q * 8 * row_bytes); }
    // a stage's resource: its first byte in the tile's rows, and its size, `valid` being the bytes of the rows that there are; past
    // the last step there is none, and zeros are written
    static constexpr int begin(int stage) { return stage * 128; }
    static constexpr int bytes(int stage, int steps, int valid) { return stage * kSub < steps ? valid - begin(stage) : 0; }
};

}  // namespace engram
