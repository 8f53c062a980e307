// Follows every load of token rows of the projection on 4-bit weights, by the index arithmetic that its tiles use.  Prints the
// first mistake and returns 1, or nothing and 0.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "mx4_rows.h"

template <bool kA8, int MI, int NW>
int check(int steps, int rows) {
    constexpr int BM = 16 * MI;
    using R = engram::Mx4Rows<kA8, BM, NW>;
    const int row_bytes = R::row_bytes(steps), valid = std::min(BM, rows) * row_bytes;
    const int stages = (steps + R::kSub - 1) / R::kSub;
    auto bad = [&](const char* what, int stage, int wave, int q, int lane) {
        std::printf("%s: 8 bits %d, %d rows by %d waves, %d steps, %d rows left, stage %d wave %d load %d lane %d\n", what, kA8, BM,
                    NW, steps, rows, stage, wave, q, lane);
        return 1;
    };
    for (int stage = 0; stage < stages + 6; ++stage) {  // (the last ones past the last step)
        const long size = R::bytes(stage, steps, valid);
        if (size < 0) return bad("negative size", stage, 0, 0, 0);
        if (size > 0 && R::begin(stage) + size != valid) return bad("the resource ends elsewhere than the rows", stage, 0, 0, 0);
        std::vector<int> filled(BM * 8, 0);
        for (int wave = 0; wave < NW; ++wave)
            for (int q = 0; q < R::kLoads; ++q)
                for (int lane = 0; lane < 64; ++lane) {
                    const int row = R::first(wave) + 8 * q + lane / 8, slot = lane % 8;
                    if (row >= BM) return bad("a row past the stage", stage, wave, q, lane);
                    filled[row * 8 + slot] = 1;
                    const long off = static_cast<long>(R::offset(R::first(wave), lane, q & 1, row_bytes)) + R::load_rows(q, row_bytes);
                    const bool fetched = off < size;
                    const long at = R::begin(stage) + off;  // in the tile's rows
                    if (fetched && at + 16 > valid) return bad("a read past the rows", stage, wave, q, lane);
                    const long piece = 128l * stage + 16 * (slot ^ ((row / 2) % 8));  // of its row
                    const bool wanted = row < rows && piece < row_bytes;
                    if (wanted && (!fetched || at != static_cast<long>(row) * row_bytes + piece))
                        return bad("another piece than the slot's", stage, wave, q, lane);
                    if (row >= rows && fetched) return bad("a row that there is not", stage, wave, q, lane);
                }
        if (std::count(filled.begin(), filled.end(), 1) != BM * 8) return bad("slots left as they were", stage, 0, 0, 0);
    }
    return 0;
}

template <int MI, int NW>
int both(int steps, int rows) {
    return check<true, MI, NW>(steps, rows) || check<false, MI, NW>(steps, rows);
}

int main() {
    for (int steps : {1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 13, 47, 48, 8192})
        for (int rows : {1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 1000}) {
            if (steps == 8192 && rows != 1 && rows != 127) continue;
            if (both<1, 2>(steps, rows) || both<2, 4>(steps, rows) || both<4, 4>(steps, rows) || both<8, 4>(steps, rows)) return 1;
        }
    return 0;
}
