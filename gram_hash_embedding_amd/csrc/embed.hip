// engram_embed: rows of a trainable table by id, times a scalar.
// engram_embed_grad / engram_embed_grad_rows: the gradient of such a lookup, per table row.
//
//   out[i, :]  = scale * table[id_i - row_start, :]
//   grad[r, :] = scale * sum over the positions i with id_i - row_start = r of up[i, :]
//
// All of it is HBM traffic.  The gradient is a sum over equal ids, so it is made of a stable sort of (row, position)
// and one pass over the sorted positions that adds the upstream rows of equal ids in position order: no atomics on
// floating-point data, the same bits from every call.
//
// Sort: least significant digit first, 8 bytes (row, position) per element, digits of at most kMaxDigitBits bits over
// the bits that rows actually have, so the fewest passes (17 bits of a token vocabulary: two, 29 bits of a 384 M row
// table: three).  A pass counts the digits per tile, then every workgroup ranks a tile of elements (per wave by ballots
// over the digit's bits, so stable), adds the tiles before it from the table of per-tile digit counts, and scatters.
// Up to 8,192 ids one workgroup does all of it, up to kSmall every workgroup does and folds too.
//
// Fold: the sorted positions are cut into chunks of kChunk; a group of lanes adds a segment's positions within a chunk
// in registers and writes the table row if the segment ends there.  A segment that crosses chunks leaves fp32 partial
// sums (one leaving a chunk, one entering) which a last launch adds in a fixed order, so that one hot row costs no more
// than many cold ones.
//
// Measured: the lookup of 65,536 rows of 5,120 bf16 140 us (808 MB, 5.8 TB/s); the dense gradient of 8,192 such rows over
// 129,280 table rows in fp32 465 us (2.73 GB, 5.9 TB/s: 418 the zeros with the sort beneath them, 38 the fold, 8 the
// join); the distinct rows of 1,572,864 hashed ids of 64 220 us (629 MB: 76 the sort, 8 the counts, 120 the fold, 15 the
// join and the tail), of 196,608 ids 65 us, bound by its nine launches at 4 to 9 us each.
#include "rows.h"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
// ids per thread, and so per tile: few for up to this many ids, which else make too few workgroups (24,000 ids of 29 bits
// 61 -> 53 us, 72,000 69 -> 62, 196,608 of 22 bits 70 -> 66, 480,000 of 29 bits 122 -> 117; 1,572,864 220 -> 229)
constexpr int kFewItems = 4, kManyItems = 8;
constexpr int64_t kFewIds = 1 << 19;
constexpr int kMaxDigitBits = 11;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
// up to this many tiles every scattering workgroup adds the digit counts of the tiles before it by itself; past it a
// launch of its own turns the counts into prefixes
constexpr int kDirectTiles = 64;
constexpr int kChunk = 16;   // sorted positions per chunk of the fold
constexpr int kHeadsTile = kThreads * kChunk;  // sorted positions per workgroup that counts distinct rows
constexpr int64_t kMaxIds = 1ll << 30;
constexpr int64_t kMaxGridX = 1ll << 23;  // workgroups along x: x * threads stays below 2^32
// up to this many ids one launch sorts and folds.  Against three launches (one limit for both forms, whose rows have the
// same bits): the rows form of 500 ids 15.6 us and 23, 640 ids 26 and 23; the dense one over 1,000 rows of 256, 256 ids 13.6
// and 16.5, 400 17.2 and 17, 640 28 and 17; over 13,225 rows of 2,048 (zeros beneath the sort there) 400 33 and 26, 640 48
// and 27.
constexpr int kSmall = 512;

// ---------------------------------------------------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------------------------------------------------
struct EmbedArgs {
    const void* ids;
    int id_bytes;
    int64_t n;
    const uint8_t* table;
    int64_t R, row_start;
    int D;
    float scale;
    uint8_t* out;
};

// the table row of an id, or -1 outside [row_start, row_start + R) (whatever 64-bit number it is)
__device__ inline int64_t row_of(const void* ids, int id_bytes, int64_t i, int64_t row_start, int64_t R) {
    const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
    const uint64_t r = static_cast<uint64_t>(id) - static_cast<uint64_t>(row_start);
    return id >= row_start && r < static_cast<uint64_t>(R) ? static_cast<int64_t>(r) : -1;
}

// One piece of kRows rows per thread, the pieces in memory order.  LPR 0: a workgroup (of up to 1,024 threads) takes a row,
// or as much of it as it holds; else LPR lanes take a row.  65,536 Zipf rows of 5,120 bf16: 226 us with one row per
// thread, 176 us with two, 162 us with four (more loads in flight), 136 us with four and non-temporal stores (the output
// does not push the table's rows out of the Infinity Cache).
template <class TT, class OT, int LPR, int kRows, bool kNt>
__global__ __launch_bounds__(LPR == 0 ? 1024 : kThreads) void embed_kernel(EmbedArgs a) {
    constexpr int kGroups = LPR == 0 ? 1 : kThreads / (LPR ? LPR : 1);
    const int64_t block = blockIdx.x + static_cast<int64_t>(blockIdx.z) * gridDim.x;
    const int64_t i0 = block * (kGroups * kRows) + (LPR == 0 ? 0 : threadIdx.x / (LPR ? LPR : 1));
    const int piece = LPR == 0 ? static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x) : threadIdx.x % (LPR ? LPR : 1);
    if (piece >= a.D / 8) return;
    Piece<TT> v[kRows];
    bool ok[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        const int64_t i = i0 + q * kGroups;
        const int64_t r = i < a.n ? row_of(a.ids, a.id_bytes, i, a.row_start, a.R) : -1;
        ok[q] = r >= 0;
        if (ok[q]) v[q].load(a.table + r * a.D * TT::kBytes, piece);
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        const int64_t i = i0 + q * kGroups;
        if (i >= a.n) return;
        float f[8] = {};
        if (ok[q]) {
            v[q].to(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= a.scale;
        }
        Piece<OT> o;
        o.from(f);
        uint8_t* row = a.out + i * a.D * OT::kBytes;
        if constexpr (kNt) o.store_nt(row, piece);
        else o.store(row, piece);
    }
}

template <class TT, class OT, int LPR, int kRows, bool kNt>
int launch_embed_as(const EmbedArgs& a, hipStream_t stream) {
    const int pieces = a.D / 8;
    const int64_t per = (LPR == 0 ? 1 : kThreads / (LPR ? LPR : 1)) * kRows;
    int threads = kThreads, parts = 1;
    if (LPR == 0) {
        parts = (pieces + 1023) / 1024;
        threads = ((pieces + parts - 1) / parts + 63) / 64 * 64;
    }
    const int64_t blocks = (a.n + per - 1) / per;
    const int64_t x = blocks < kMaxGridX / 4 ? blocks : kMaxGridX / 4;
    const int64_t z = (blocks + x - 1) / x;
    if (z > 65535) return fail(ENGRAM_EINVAL, "engram_embed: too many ids");
    hipLaunchKernelGGL((embed_kernel<TT, OT, LPR, kRows, kNt>), dim3(static_cast<unsigned>(x), parts, static_cast<unsigned>(z)),
                       dim3(threads), 0, stream, a);
    return check_launch("engram_embed");
}

// One row per thread where four would leave CUs idle; ordinary stores where the output fits the Infinity Cache (its
// reader then finds it there).
constexpr int64_t kCacheBytes = 256ll << 20;
template <class TT, class OT, int LPR>
int launch_embed_rows(const EmbedArgs& a, hipStream_t stream) {
    if (a.n * a.D < (1ll << 24)) return launch_embed_as<TT, OT, LPR, 1, false>(a, stream);
    if (a.n * a.D * OT::kBytes <= kCacheBytes) return launch_embed_as<TT, OT, LPR, 4, false>(a, stream);
    return launch_embed_as<TT, OT, LPR, 4, true>(a, stream);
}

template <class TT, class OT>
int launch_embed(const EmbedArgs& a, hipStream_t stream) {
    const int pieces = a.D / 8;
    if (pieces <= 8) return launch_embed_rows<TT, OT, 8>(a, stream);
    if (pieces <= 16) return launch_embed_rows<TT, OT, 16>(a, stream);
    if (pieces <= 32) return launch_embed_rows<TT, OT, 32>(a, stream);
    return launch_embed_rows<TT, OT, 0>(a, stream);
}

// ---------------------------------------------------------------------------------------------------------------------
// zeros
// ---------------------------------------------------------------------------------------------------------------------
// A run of 16-byte pieces.  One store per thread, the workgroups in memory order: 2.65 GB in 385 us (6.9 TB/s), against
// 441 us with four stores per thread, 489 us with a grid that walks the memory and 470-480 us with a row per wave (non-
// temporal stores are slower in every form).
struct Zeros {
    u32x4* p;
    int64_t n16;
    __device__ inline void run(int64_t block) const {
        const int64_t i = block * blockDim.x + threadIdx.x;
        if (i < n16) p[i] = u32x4{0, 0, 0, 0};
    }
};

__global__ __launch_bounds__(kThreads) void zero_kernel(Zeros z) {
    z.run(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x);
}

// ---------------------------------------------------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------------------------------------------------
struct Pair {
    uint32_t key;  // table row, or R for an id outside the rows
    uint32_t pos;
};

struct SortArgs {
    const void* ids;   // first pass: element i's id is at (i / C) * stride + i % C
    int id_bytes;
    int C;
    int64_t stride;
    int64_t row_start;
    uint32_t R;
    uint32_t n;
    const Pair* in;    // later passes; null: the first
    Pair* out;
    uint32_t* hist;    // [tiles][digits] this pass's digit counts per tile (or their prefixes over the tiles)
    uint32_t* totals;  // [digits], with prefixes
    int shift, bits;      // this pass's digit
    int tiles;
    int passes;           // one_sort_kernel: all of them
};

__device__ inline uint32_t load_key(const SortArgs& a, uint32_t i) {
    int64_t at = i;
    if (a.stride != a.C) {
        const uint32_t t = i / static_cast<uint32_t>(a.C);
        at = static_cast<int64_t>(t) * a.stride + (i - t * static_cast<uint32_t>(a.C));
    }
    const int64_t r = row_of(a.ids, a.id_bytes, at, a.row_start, a.R);
    return r >= 0 ? static_cast<uint32_t>(r) : a.R;
}

// A pass's digit counts per tile; the first pass's workgroups behind the tiles write the dense form's zeros (skipping the
// rows that will be written costs more than it saves: a byte per row looked up before each store took 520 us for the
// 385 us of stores).
template <bool kFirst, int kItems>
__global__ __launch_bounds__(kSortThreads) void hist_kernel(SortArgs a, Zeros z) {
    __shared__ uint32_t h[kMaxDigits];
    if (kFirst && static_cast<int>(blockIdx.x) >= a.tiles) {
        z.run(blockIdx.x - a.tiles);
        return;
    }
    const int digits = 1 << a.bits;
    for (int d = threadIdx.x; d < digits; d += kSortThreads) h[d] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * (kSortThreads * kItems) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const uint32_t i = base + u * kSortThreads;
        if (i < a.n) atomicAdd(&h[((kFirst ? load_key(a, i) : a.in[i].key) >> a.shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.hist[blockIdx.x * digits + d] = h[d];
}

// hist[tile][digit] into the counts of the tiles before, and the totals: 64 digits per workgroup, 16 runs of tiles, eight
// loads in flight a thread (96 tiles 4.4 us, 384 8.9, of which a launch alone is 4).
__global__ __launch_bounds__(1024) void prefix_kernel(SortArgs a) {
    __shared__ uint32_t part[16][64];
    const int digits = 1 << a.bits;
    const int d = blockIdx.x * 64 + (threadIdx.x & 63);
    const int run = threadIdx.x >> 6;
    const int per = (a.tiles + 15) / 16;
    const int t0 = min(run * per, a.tiles), t1 = min(t0 + per, a.tiles);
    uint32_t sum = 0;
    if (d < digits) {
#pragma unroll 8
        for (int t = t0; t < t1; ++t) sum += a.hist[t * digits + d];
    }
    part[run][threadIdx.x & 63] = sum;
    __syncthreads();
    uint32_t base = 0, total = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const uint32_t v = part[r][threadIdx.x & 63];
        base += r < run ? v : 0;
        total += v;
    }
    if (d >= digits) return;
    for (int t = t0; t < t1; t += 8) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t + j < t1 ? a.hist[(t + j) * digits + d] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (t + j < t1) a.hist[(t + j) * digits + d] = base;
            base += v[j];
        }
    }
    if (run == 0) a.totals[d] = total;
}

// kPer consecutive counts, as one load
template <int kPer>
__device__ inline void load_counts(const uint32_t* p, uint32_t (&v)[kPer]) {
    typedef uint32_t vec __attribute__((ext_vector_type(kPer)));
    if constexpr (kPer == 1) {
        v[0] = *p;
    } else {
        const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = x[j];
    }
}

// Bound by latency, not by its 16 bytes an element: 196,608 elements 9 us, 1,572,864 12 to 16.
// kPer: digits per thread (digits = kPer * kSortThreads, or fewer than kSortThreads with kPer 1)
template <bool kFirst, int kItems, int kPer>
__global__ __launch_bounds__(kSortThreads) void scatter_kernel(SortArgs a) {
    constexpr int kDigits = kPer * kSortThreads, kSortTile = kSortThreads * kItems;
    __shared__ uint16_t cnt[kSortWaves][kDigits];
    __shared__ uint32_t move[kDigits];  // a digit's elements: their place in the output less that in the tile
    __shared__ Pair tile[kSortTile];    // the tile in order of the digit
    __shared__ uint32_t wave_sum[kSortWaves], wave_local[kSortWaves];
    const int digits = 1 << a.bits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t mask_bits = static_cast<uint32_t>(digits - 1);
    for (int d = threadIdx.x; d < kSortWaves * kDigits / 2; d += kSortThreads) reinterpret_cast<uint32_t*>(cnt)[d] = 0;

    // the wave's kItems * 64 consecutive elements
    Pair e[kItems];
    uint32_t rank[kItems];
    const uint32_t first = blockIdx.x * kSortTile + wave * (64 * kItems) + lane;
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const uint32_t i = first + u * 64;
        e[u] = Pair{0, i};
        if (i < a.n) {
            if (kFirst) e[u].key = load_key(a, i);
            else e[u] = a.in[i];
        }
    }
    // each thread owns the digits [own, own + kPer): how many elements have it, and how many of them lie in the tiles
    // before this one
    const int own = threadIdx.x * kPer;
    uint32_t total[kPer] = {}, prior[kPer] = {};
    if (own < digits) {
        if (a.totals) {
            load_counts(a.totals + own, total);
            load_counts(a.hist + blockIdx.x * digits + own, prior);
        } else {
            constexpr int kBatch = 16;
            for (int t = 0; t < a.tiles; t += kBatch) {
                uint32_t v[kBatch][kPer];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) load_counts(a.hist + min(t + i, a.tiles - 1) * digits + own, v[i]);
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        total[j] += t + i < a.tiles ? v[i][j] : 0;
                        prior[j] += t + i < static_cast<int>(blockIdx.x) ? v[i][j] : 0;
                    }
            }
        }
    }
    __syncthreads();
    volatile uint16_t* mine = cnt[wave];  // this wave's counters: its LDS accesses stay in program order
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const bool live = first + u * 64 < a.n;
        const uint32_t d = (e[u].key >> a.shift) & mask_bits;
        uint64_t same = __ballot(live);
        for (int b = 0; b < a.bits; ++b) {
            const bool bit = (d >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const uint32_t before = __popcll(same & below);
        const uint32_t have = live ? mine[d] : 0;
        rank[u] = have + before;
        if (live && before == 0) mine[d] = static_cast<uint16_t>(have + __popcll(same));
    }
    __syncthreads();

    // exclusive sums over the digits, of all elements and of the tile's
    uint32_t sum = 0, local = 0, have[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        uint32_t at = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {  // each wave's elements of the digit begin after those of the waves before
            const uint32_t c = cnt[w][own + j];
            cnt[w][own + j] = static_cast<uint16_t>(at);
            at += c;
        }
        have[j] = at;
        local += at;
        sum += total[j];
    }
    uint32_t scan = sum, scan_local = local;  // inclusive over the wave's threads
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(scan, off, 64), l = __shfl_up(scan_local, off, 64);
        scan += lane >= off ? o : 0;
        scan_local += lane >= off ? l : 0;
    }
    if (lane == 63) {
        wave_sum[wave] = scan;
        wave_local[wave] = scan_local;
    }
    __syncthreads();
    uint32_t base = scan - sum, base_local = scan_local - local;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        base += w < wave ? wave_sum[w] : 0;
        base_local += w < wave ? wave_local[w] : 0;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        move[own + j] = base + prior[j] - base_local;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) cnt[w][own + j] = static_cast<uint16_t>(cnt[w][own + j] + base_local);
        base += total[j];
        base_local += have[j];
    }
    __syncthreads();
    // through LDS in the digit's order, so that the stores of neighbouring lanes fall into the same lines
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        if (first + u * 64 >= a.n) continue;
        tile[cnt[wave][(e[u].key >> a.shift) & mask_bits] + rank[u]] = e[u];
    }
    __syncthreads();
    const uint32_t here = min(a.n - blockIdx.x * kSortTile, static_cast<uint32_t>(kSortTile));
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const uint32_t i = threadIdx.x + u * kSortThreads;
        if (i >= here) continue;
        const Pair x = tile[i];
        a.out[move[(x.key >> a.shift) & mask_bits] + i] = x;
    }
}

template <bool kFirst, int kItems>
void launch_scatter(const SortArgs& a, hipStream_t stream) {
    const dim3 grid(a.tiles), block(kSortThreads);
    const int digits = 1 << a.bits;
    if (digits > 2 * kSortThreads) hipLaunchKernelGGL((scatter_kernel<kFirst, kItems, 4>), grid, block, 0, stream, a);
    else if (digits > kSortThreads) hipLaunchKernelGGL((scatter_kernel<kFirst, kItems, 2>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((scatter_kernel<kFirst, kItems, 1>), grid, block, 0, stream, a);
}

// one pass over the digit: its counts per tile, their prefixes where the tiles are many, and the scatter
template <int kItems>
void launch_pass(SortArgs& a, uint32_t* totals, const Zeros& z, hipStream_t stream) {
    const dim3 block(kSortThreads);
    const dim3 grid(static_cast<unsigned>(a.tiles + (z.n16 + kSortThreads - 1) / kSortThreads));
    if (a.in) hipLaunchKernelGGL((hist_kernel<false, kItems>), grid, block, 0, stream, a, z);
    else hipLaunchKernelGGL((hist_kernel<true, kItems>), grid, block, 0, stream, a, z);
    if (a.tiles > kDirectTiles) {
        a.totals = totals;
        hipLaunchKernelGGL(prefix_kernel, dim3(((1 << a.bits) + 63) / 64), dim3(1024), 0, stream, a);
    }
    if (a.in) launch_scatter<false, kItems>(a, stream);
    else launch_scatter<true, kItems>(a, stream);
}

// ---------------------------------------------------------------------------------------------------------------------
// fold
// ---------------------------------------------------------------------------------------------------------------------
struct FoldArgs {
    const Pair* sorted;
    uint32_t n, R;
    const uint8_t* up;  // [n, D] upstream rows
    int D;
    int cols;           // column blocks of a group's lanes, a piece each
    float scale;
    uint8_t* out;       // dense: [R, D]; rows: [n, D]
    int accumulate;
    // rows form
    int64_t* unique;    // [n], or null: the dense form
    int32_t* count;     // [1]
    int64_t row_start;
    uint32_t* heads;       // [tiles] distinct rows that begin in each kHeadsTile sorted positions
    uint32_t* chunk_base;  // [chunks] of those, the ones before the chunk
    int tiles;
    uint32_t chunks;
    uint32_t* leave_to;  // rows form: [chunks] the distinct row that leaves the chunk
    float* leave;       // [chunks][D] sum of a segment that begins in the chunk and goes on after it
    float* enter;       // [chunks][D] sum of the chunk's share of a segment that began before it
    uint32_t join_blocks;  // workgroups that join; those behind them write the rows form's tail
};

// Distinct rows per chunk (before it in its tile) and per tile: a chunk a thread.  196,608 positions 4.6 us, 1,572,864 8.2.
__global__ __launch_bounds__(kThreads) void heads_kernel(FoldArgs a) {
    __shared__ uint32_t wsum[kThreads / 64];
    const uint32_t chunk = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t s = chunk * kChunk;
    uint32_t c = 0;
    if (s < a.n) {
        uint32_t prev = s ? a.sorted[s - 1].key : 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const uint32_t k = s + j < a.n ? a.sorted[s + j].key : a.R;
            c += k != prev && k < a.R;
            prev = k;
        }
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t scan = c;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(scan, off, 64);
        scan += lane >= off ? o : 0;
    }
    if (lane == 63) wsum[wave] = scan;
    __syncthreads();
    uint32_t base = scan - c, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        base += w < wave ? wsum[w] : 0;
        all += wsum[w];
    }
    if (chunk < a.chunks) a.chunk_base[chunk] = base;
    if (threadIdx.x == 0) a.heads[blockIdx.x] = all;
}

// Up to kOneSort ids: one workgroup sorts them all, through LDS, a digit of at most eight bits per pass, and for the rows
// form counts the distinct rows on the way (what heads_kernel does); the workgroups behind it write the dense form's zeros.
// 1,200 ids of 29 bits take 15 us so, 8,160 of them 35 us, against 42-48 us as launches over tiles; the dense gradient of
// 8,192 tokens over 129,280 rows of 5,120 went from 495 to 467 us.
constexpr int kOneThreads = 1024, kOneItems = 8, kOneSort = kOneThreads * kOneItems, kOneBits = 8;
__global__ __launch_bounds__(kOneThreads, 8) void one_sort_kernel(SortArgs a, FoldArgs f, Zeros z) {
    constexpr int kWaves = kOneThreads / 64, kDigits = 1 << kOneBits;
    __shared__ Pair tile[kOneSort];
    __shared__ uint16_t cnt[kWaves][kDigits];
    __shared__ uint32_t wave_sum[kWaves];
    if (blockIdx.x) {
        z.run(blockIdx.x - 1);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int items = static_cast<int>((a.n + kOneThreads - 1) / kOneThreads);  // per thread
    const uint32_t first = wave * (64 * items) + lane;
    const uint64_t below = (1ull << lane) - 1;
    auto scan = [&](uint32_t v) {  // exclusive over the workgroup's threads
        uint32_t s = v;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(s, off, 64);
            s += lane >= off ? o : 0;
        }
        if (lane == 63) wave_sum[wave] = s;
        __syncthreads();
        uint32_t base = s - v;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) base += w < wave ? wave_sum[w] : 0;
        return base;
    };
    Pair e[kOneItems];
#pragma unroll
    for (int u = 0; u < kOneItems; ++u) {  // what is past the ids sorts behind them
        if (u >= items) break;
        const uint32_t i = first + u * 64;
        e[u] = Pair{i < a.n ? load_key(a, i) : 0xFFFFFFFFu, i};
    }
    const uint32_t mask_bits = (1u << a.bits) - 1;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        for (int d = tid; d < kWaves * kDigits / 2; d += kOneThreads) reinterpret_cast<uint32_t*>(cnt)[d] = 0;
        __syncthreads();
        volatile uint16_t* mine = cnt[wave];  // this wave's counters: its LDS accesses stay in program order
        uint32_t rank[kOneItems];
#pragma unroll
        for (int u = 0; u < kOneItems; ++u) {
            if (u >= items) break;
            const uint32_t d = (e[u].key >> shift) & mask_bits;
            uint64_t same = ~0ull;
#pragma unroll
            for (int b = 0; b < kOneBits; ++b) {
                if (b >= a.bits) break;
                const bool bit = (d >> b) & 1;
                const uint64_t set = __ballot(bit);
                same &= bit ? set : ~set;
            }
            const uint32_t before = __popcll(same & below);
            const uint32_t have = mine[d];
            rank[u] = have + before;
            if (before == 0) mine[d] = static_cast<uint16_t>(have + __popcll(same));
        }
        __syncthreads();
        uint32_t total = 0;
        if (tid < kDigits)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) total += cnt[w][tid];
        uint32_t at = scan(total);
        if (tid < kDigits)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = cnt[w][tid];
                cnt[w][tid] = static_cast<uint16_t>(at);
                at += c;
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOneItems; ++u) {
            if (u >= items) break;
            tile[cnt[wave][(e[u].key >> shift) & mask_bits] + rank[u]] = e[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOneItems; ++u) {
            if (u >= items) break;
            e[u] = tile[first + u * 64];
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kOneItems; ++u)
        if (u < items && first + u * 64 < a.n) a.out[first + u * 64] = e[u];
    if (!f.unique) return;
    // distinct rows that begin before each chunk in its tile, and in each tile
    static_assert(kChunk == 2 * kOneItems, "a chunk per two threads");
    constexpr int kPerTile = kHeadsTile / kOneItems;  // threads
    const uint32_t s = tid * kOneItems;
    uint32_t heads = 0, prev = s && s < a.n ? tile[s - 1].key : 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kOneItems; ++j) {
        const uint32_t k = s + j < a.n ? tile[s + j].key : a.R;
        heads += k != prev && k < a.R;
        prev = k;
    }
    const uint32_t before = scan(heads);
    uint32_t* tile_base = reinterpret_cast<uint32_t*>(cnt);
    if (tid % kPerTile == 0) tile_base[tid / kPerTile] = before;
    if (tid == kOneThreads - 1) tile_base[kOneSort / kHeadsTile] = before + heads;
    __syncthreads();
    const int t = tid / kPerTile;
    if (tid % 2 == 0 && static_cast<uint32_t>(tid / 2) < f.chunks) f.chunk_base[tid / 2] = before - tile_base[t];
    if (tid < f.tiles) f.heads[tid] = tile_base[tid + 1] - tile_base[tid];
}

// The distinct rows before tile `tile` (all of them for tile == tiles): every wave adds them itself.
__device__ inline uint32_t heads_before(const FoldArgs& a, int tile) {
    uint32_t s = 0;
    for (int t = threadIdx.x & 63; t < tile; t += 64) s += a.heads[t];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    return s;
}

template <class OT, bool kPast>
__device__ inline void put_row(const FoldArgs& a, uint32_t key, uint32_t u, int piece, const float (&acc)[8]) {
    float f[8];
    uint8_t* row = a.out + static_cast<int64_t>(a.unique ? u : key) * a.D * OT::kBytes;
    Piece<OT> o;
    if (a.accumulate) {
        o.load(row, piece);
        o.to(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += acc[e] * a.scale;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = acc[e] * a.scale;
    }
    o.from(f);
    if constexpr (kPast) o.store_nt(row, piece);
    else o.store(row, piece);
    if (a.unique && piece == 0) a.unique[u] = static_cast<int64_t>(key) + a.row_start;
}

// One group of LPR lanes per (chunk, column block), with all of the chunk's rows in flight at once (a group per sorted
// position instead, most of them a single row, keeps too few bytes in flight: 241 us against 134 us for 1.57 M rows of
// 64 bf16).
template <class GT, class OT, int LPR, bool kPast>
__global__ __launch_bounds__(kThreads) void fold_kernel(FoldArgs a) {
    constexpr int kGroups = kThreads / LPR, kPerTile = kHeadsTile / kChunk;
    constexpr int kBatch = GT::kBytes == 2 ? kChunk : kChunk / 2;  // rows in flight
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LPR;
    const uint32_t chunk = static_cast<uint32_t>(unit / a.cols);
    const int piece = static_cast<int>(unit % a.cols) * LPR + threadIdx.x % LPR;
    uint32_t u = 0;  // the distinct rows before the chunk
    if (a.unique) {
        const uint32_t c0 = static_cast<uint32_t>(static_cast<int64_t>(blockIdx.x) * kGroups / a.cols);
        const uint32_t t0 = min(c0, a.chunks - 1) / kPerTile;
        u = heads_before(a, static_cast<int>(t0));
        if (chunk < a.chunks) {  // (the workgroup's chunks lie in one tile or two)
            for (uint32_t t = t0; t < chunk / kPerTile; ++t) u += a.heads[t];
            u += a.chunk_base[chunk];
        }
    }
    if (chunk >= a.chunks || piece >= a.D / 8) return;
    const uint32_t s = chunk * kChunk, e = min(s + kChunk, a.n);
    uint32_t cur = s ? a.sorted[s - 1].key : 0xFFFFFFFFu;  // the running segment's row
    const uint32_t after = e < a.n ? a.sorted[e].key : a.R;  // R: nothing goes on
    float acc[8] = {};
    bool entered = true;  // the running segment began before the chunk
    bool open = false;    // it has positions in the chunk
    auto close = [&](bool goes_on) {
        if (!open) return;
        if (entered || goes_on) {
            Piece<F32> p;
            p.from(acc);
            p.store((entered ? a.enter : a.leave) + static_cast<int64_t>(chunk) * a.D, piece);
            if (!entered && a.unique && piece == 0) a.leave_to[chunk] = u - 1;
        } else {
            put_row<OT, kPast>(a, cur, u - 1, piece, acc);
        }
    };
    for (uint32_t b = s; b < e; b += kBatch) {
        Pair pr[kBatch];
        Piece<GT> v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) pr[j] = b + j < e ? a.sorted[b + j] : Pair{a.R, 0};
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (pr[j].key >= a.R) continue;
            const uint8_t* row = a.up + static_cast<int64_t>(pr[j].pos) * a.D * GT::kBytes;
            if constexpr (kPast) v[j].load_nt(row, piece);
            else v[j].load(row, piece);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (pr[j].key >= a.R) continue;
            float f[8];
            v[j].to(f);
            if (pr[j].key != cur) {
                close(false);
                cur = pr[j].key;
                entered = false;
                ++u;
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = f[q];
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] += f[q];
            }
            open = true;
        }
    }
    close(after == cur);
}

// Segments that cross chunks: the chunk where one begins adds its own partial sum and those of the chunks it enters.
// Each group of LPR lanes takes such segments of its wave's chunks in turn; a segment of kLong chunks or more (a hot row)
// is taken by the whole workgroup, kBatch chunks per group at a time.  Every order is fixed.  In the rows form the
// workgroups behind them write the rows past the last distinct one: zeros, and -1 for their ids.
constexpr int kLong = 16;

template <int LPR>
constexpr int join_chunks() {  // chunks per wave: two per group of lanes (four or eight leave too few waves)
    return 64 / LPR * 2;
}

template <class OT, int LPR, bool kPast>
__global__ __launch_bounds__(kThreads) void join_kernel(FoldArgs a) {
    constexpr int kWaves = kThreads / 64, kGroups = 64 / LPR, kBatch = 4, kPerWave = join_chunks<LPR>();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int group = lane / LPR;
    if (blockIdx.x >= a.join_blocks) {
        const uint32_t all = heads_before(a, a.tiles);
        if (blockIdx.x == a.join_blocks && threadIdx.x == 0) *a.count = static_cast<int32_t>(all);
        // 16 bytes a thread of the rows behind the last distinct one, and their ids
        const uint32_t per = static_cast<uint32_t>(a.D * OT::kBytes / 16);
        const int64_t from = static_cast<int64_t>(all) * per, to = static_cast<int64_t>(a.n) * per;
        const int64_t step = static_cast<int64_t>(gridDim.x - a.join_blocks) * kThreads;
        const int64_t me = static_cast<int64_t>(blockIdx.x - a.join_blocks) * kThreads + threadIdx.x;
        for (int64_t i = from + me; i < to; i += step) reinterpret_cast<u32x4*>(a.out)[i] = u32x4{0, 0, 0, 0};
        for (int64_t k = all + me; k < a.n; k += step) a.unique[k] = -1;
        return;
    }
    __shared__ float sums[kWaves][LPR][9];
    __shared__ uint32_t keys[kWaves][kPerWave];
    __shared__ uint64_t far_of[kWaves];
    const int cb = blockIdx.x % a.cols;
    const int piece = cb * LPR + lane % LPR;
    const bool live = piece < a.D / 8;
    const uint32_t base = blockIdx.x / a.cols * (kWaves * kPerWave);
    const uint32_t c0 = base + wave * kPerWave;
    // which of the wave's chunks a segment that began in them leaves, and which of those segments are long
    bool crosses = false, goes_far = false;
    if (lane < kPerWave) {
        uint32_t key = a.R;
        if (c0 + lane < a.chunks) {
            const uint32_t s = (c0 + lane) * kChunk, e = min(s + kChunk, a.n), far = c0 + lane + kLong;
            if (e < a.n) {
                key = a.sorted[e].key;
                const uint32_t last = a.sorted[e - 1].key, prev = s ? a.sorted[s - 1].key : a.R;
                const uint32_t far_key = far < a.chunks ? a.sorted[far * kChunk].key : a.R;
                crosses = key < a.R && last == key && prev != key;
                goes_far = crosses && far_key == key;
            }
        }
        keys[wave][lane] = key;
    }
    const uint64_t near = __ballot(crosses && !goes_far), far = __ballot(goes_far);
    if (lane == 0) far_of[wave] = far;
    __syncthreads();
    auto add = [&](float (&acc)[8], const float* from, uint32_t chunk) {
        float f[8];
        Piece<F32> p;
        p.load(from + static_cast<int64_t>(chunk) * a.D, piece);
        p.to(f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += f[q];
    };
    {
        uint64_t todo = near;
        for (int skip = group; todo && skip; --skip) todo &= todo - 1;
        while (todo && live) {
            const int bit = __builtin_ctzll(todo);
            const uint32_t chunk = c0 + bit, key = keys[wave][bit];
            float acc[8] = {};
            add(acc, a.leave, chunk);
            uint32_t c = chunk + 1;
            do add(acc, a.enter, c++);
            while (c < a.chunks && a.sorted[c * kChunk].key == key);
            put_row<OT, kPast>(a, key, a.unique ? a.leave_to[chunk] : 0, piece, acc);
            for (int skip = kGroups; todo && skip; --skip) todo &= todo - 1;
        }
    }
    for (int w = 0; w < kWaves; ++w)
        for (uint64_t todo = far_of[w]; todo; todo &= todo - 1) {
            const int bit = __builtin_ctzll(todo);
            const uint32_t chunk = base + w * kPerWave + bit, key = keys[w][bit];
            float acc[8] = {};
            if (wave == 0 && group == 0 && live) add(acc, a.leave, chunk);
            constexpr int kStep = kWaves * kGroups * kBatch;
            for (uint32_t c = chunk + 1 + (wave * kGroups + group) * kBatch; c < a.chunks; c += kStep) {
                uint32_t k[kBatch];
                Piece<F32> p[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    k[j] = c + j < a.chunks ? a.sorted[(c + j) * kChunk].key : a.R;
                    // (a chunk that is not entered holds anything: loaded, not used)
                    if (live && c + j < a.chunks) p[j].load(a.enter + static_cast<int64_t>(c + j) * a.D, piece);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (k[j] != key || !live) continue;
                    float f[8];
                    p[j].to(f);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] += f[q];
                }
                if (k[kBatch - 1] != key) break;
            }
#pragma unroll
            for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] += __shfl_xor(acc[q], off, 64);
            if (group == 0)
#pragma unroll
                for (int q = 0; q < 8; ++q) sums[wave][lane][q] = acc[q];
            __syncthreads();
            if (wave == 0 && group == 0 && live) {
#pragma unroll
                for (int v = 1; v < kWaves; ++v)
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] += sums[v][lane][q];
                put_row<OT, kPast>(a, key, a.unique ? a.leave_to[chunk] : 0, piece, acc);
            }
            __syncthreads();
        }
}

// Up to kSmall ids: every workgroup sorts them in LDS (a bitonic network over (row, position)) and folds its share of
// (distinct row, column block) units, one group of LPR lanes each; the units past the last distinct row are the rows
// form's tail.  One launch instead of six or more: at these sizes the launches are the time (64 ids of 256 columns
// over 1,000 rows 13 us, where the launches over tiles took 27).
struct SmallArgs {
    SortArgs ids;
    FoldArgs fold;
};

template <class GT, class OT, int LPR>
__global__ __launch_bounds__(kThreads) void small_kernel(SmallArgs a) {
    constexpr int kBatch = GT::kBytes == 2 ? 8 : 4;
    __shared__ uint64_t s[kSmall];
    __shared__ uint16_t start[kSmall + 1];
    __shared__ uint32_t wsum[kThreads / 64];
    const int n = static_cast<int>(a.fold.n), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = tid; i < size; i += kThreads)
        s[i] = (static_cast<uint64_t>(i < n ? load_key(a.ids, i) : 0xFFFFFFFFu) << 32) | static_cast<uint32_t>(i);
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j >= 1; j >>= 1) {
            __syncthreads();
            for (int i = tid; i < size / 2; i += kThreads) {
                const int lo = (i / j) * 2 * j + i % j, hi = lo + j;  // j is a power of two
                const uint64_t x = s[lo], y = s[hi];
                if ((x > y) == ((lo & k) == 0)) {
                    s[lo] = y;
                    s[hi] = x;
                }
            }
        }
    __syncthreads();
    // where each distinct row begins: kPer positions per thread
    constexpr int kPer = kSmall / kThreads;
    auto key_at = [&](int i) { return i < n ? static_cast<uint32_t>(s[i] >> 32) : 0xFFFFFFFFu; };
    bool head[kPer];
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        const uint32_t key = key_at(i);
        head[j] = key < a.fold.R && (i == 0 || key_at(i - 1) != key);
        mine += head[j];
    }
    uint32_t scan = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(scan, off, 64);
        scan += lane >= off ? o : 0;
    }
    if (lane == 63) wsum[wave] = scan;
    __syncthreads();
    uint32_t u = scan - mine, count = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        u += w < wave ? wsum[w] : 0;
        count += wsum[w];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (head[j]) start[u++] = static_cast<uint16_t>(tid * kPer + j);
    __syncthreads();
    const FoldArgs& f = a.fold;
    if (f.unique && blockIdx.x == 0 && tid == 0) *f.count = static_cast<int32_t>(count);

    const uint32_t unit = blockIdx.x * (kThreads / LPR) + tid / LPR;
    const uint32_t seg = unit / f.cols;
    const int piece = static_cast<int>(unit % f.cols) * LPR + tid % LPR;
    if (seg >= f.n || piece >= f.D / 8) return;
    if (seg >= count) {
        if (f.unique) {
            Piece<OT> z;
            const float zero[8] = {};
            z.from(zero);
            z.store(f.out + static_cast<int64_t>(seg) * f.D * OT::kBytes, piece);
            if (piece == 0) f.unique[seg] = -1;
        }
        return;
    }
    const int b0 = start[seg];
    const uint32_t key = static_cast<uint32_t>(s[b0] >> 32);
    float acc[8] = {};
    for (int b = b0; b < n && static_cast<uint32_t>(s[b] >> 32) == key; b += kBatch) {
        Piece<GT> v[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint64_t e = b + j < n ? s[b + j] : ~0ull;
            in[j] = static_cast<uint32_t>(e >> 32) == key;
            if (in[j]) v[j].load(f.up + static_cast<int64_t>(static_cast<uint32_t>(e)) * f.D * GT::kBytes, piece);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (!in[j]) continue;
            float x[8];
            v[j].to(x);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += x[q];
        }
    }
    put_row<OT, false>(f, key, seg, piece, acc);
}

__global__ void zero_count_kernel(int32_t* count) { *count = 0; }

// ---------------------------------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------------------------------
int bits_of(uint32_t v) { return v ? 32 - __builtin_clz(v) : 1; }

struct Plan {
    int bits, passes;      // digit bits and passes
    int items, tiles, head_tiles;
    uint32_t chunks;
    int64_t pairs, hist, totals, heads, chunk_base, leave_to, leave, enter, bytes;  // offsets
};

int64_t up16(int64_t v) { return (v + 15) & ~15ll; }

Plan plan_of(int64_t n, int32_t D, int64_t R) {
    Plan p;
    const int key_bits = bits_of(static_cast<uint32_t>(R));  // the key R stands for ids outside
    p.passes = (key_bits + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    p.items = n <= kFewIds ? kFewItems : kManyItems;
    p.tiles = static_cast<int>((n + p.items * kSortThreads - 1) / (p.items * kSortThreads));
    p.head_tiles = static_cast<int>((n + kHeadsTile - 1) / kHeadsTile);
    p.chunks = static_cast<uint32_t>((n + kChunk - 1) / kChunk);
    int64_t at = 0;
    p.pairs = at;
    at += up16(2 * n * static_cast<int64_t>(sizeof(Pair)));
    p.hist = at;
    at += up16(static_cast<int64_t>(p.tiles) * (4ll << p.bits));
    p.totals = at;
    at += up16(4ll << p.bits);
    p.heads = at;
    at += up16(4ll * p.head_tiles);
    p.chunk_base = at;
    at += up16(4ll * p.chunks);
    p.leave_to = at;
    at += up16(4ll * p.chunks);
    p.leave = at;
    at += up16(4ll * p.chunks * D);
    p.enter = at;
    at += up16(4ll * p.chunks * D);
    p.bytes = at;
    return p;
}

// sorted (row, position) pairs of the ids, in the workspace; `zeros` bytes at f's output are written on the way
int sort_ids(const Plan& p, const void* ids, int id_bytes, int64_t n, int C, int64_t stride, int64_t R, int64_t row_start,
             uint8_t* ws, FoldArgs& f, int64_t zeros, hipStream_t stream, const char* what) {
    Pair* buf[2] = {reinterpret_cast<Pair*>(ws + p.pairs), reinterpret_cast<Pair*>(ws + p.pairs) + n};
    SortArgs a = {};
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.C = C;
    a.stride = stride;
    a.row_start = row_start;
    a.R = static_cast<uint32_t>(R);
    a.n = static_cast<uint32_t>(n);
    a.bits = p.bits;
    a.tiles = p.tiles;
    a.hist = reinterpret_cast<uint32_t*>(ws + p.hist);
    // (what a grid does not hold, some 32 GiB and more, in a launch of its own)
    const int64_t n16 = zeros / 16, most = (kMaxGridX / 2 - p.tiles) * kSortThreads;
    const Zeros z = {reinterpret_cast<u32x4*>(f.out), n16 < most ? n16 : most};
    if (n16 > most) {
        const int rc = launch_zero(z.p + most, (n16 - most) * 16, stream, what);
        if (rc != ENGRAM_OK) return rc;
    }
    uint32_t* totals = reinterpret_cast<uint32_t*>(ws + p.totals);
    for (int q = 0; q < p.passes; ++q) {
        a.shift = q * p.bits;
        a.in = q ? buf[(q + 1) & 1] : nullptr;
        a.out = buf[q & 1];
        if (p.items == kFewItems) launch_pass<kFewItems>(a, totals, q ? Zeros{} : z, stream);
        else launch_pass<kManyItems>(a, totals, q ? Zeros{} : z, stream);
    }
    f.sorted = buf[(p.passes - 1) & 1];
    return ENGRAM_OK;
}

// the same by one workgroup, the rows form's counts in f's arrays
int one_sort(const Plan& p, const void* ids, int id_bytes, int64_t n, int C, int64_t stride, int64_t R, int64_t row_start,
             uint8_t* ws, FoldArgs& f, int64_t zeros, hipStream_t stream, const char* what) {
    SortArgs a = {};
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.C = C;
    a.stride = stride;
    a.row_start = row_start;
    a.R = static_cast<uint32_t>(R);
    a.n = static_cast<uint32_t>(n);
    const int key_bits = bits_of(a.R);
    a.passes = (key_bits + kOneBits - 1) / kOneBits;
    a.bits = (key_bits + a.passes - 1) / a.passes;
    a.out = reinterpret_cast<Pair*>(ws + p.pairs);
    const int64_t n16 = zeros / 16, most = (kMaxGridX / 4 - 1) * kOneThreads;
    const Zeros z = {reinterpret_cast<u32x4*>(f.out), n16 < most ? n16 : most};
    if (n16 > most) {
        const int rc = launch_zero(z.p + most, (n16 - most) * 16, stream, what);
        if (rc != ENGRAM_OK) return rc;
    }
    hipLaunchKernelGGL(one_sort_kernel, dim3(static_cast<unsigned>(1 + (z.n16 + kOneThreads - 1) / kOneThreads)),
                       dim3(kOneThreads), 0, stream, a, f, z);
    f.sorted = a.out;
    return ENGRAM_OK;
}

// `past`: the call moves more than the Infinity Cache holds.  Then upstream rows and finished ones pass it by, which leaves
// it to the sorted positions and the partial sums (1.57 M rows of 64: 250 -> 220 us; 196,608, which fit: 69 -> 73).
template <class GT, class OT, int LPR>
int launch_fold_as(FoldArgs& a, const SortArgs* small, bool past, hipStream_t stream, const char* what) {
    a.cols = (a.D / 8 + LPR - 1) / LPR;
    if (small) {
        const int64_t blocks = (static_cast<int64_t>(a.n) * a.cols + kThreads / LPR - 1) / (kThreads / LPR);
        hipLaunchKernelGGL((small_kernel<GT, OT, LPR>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream,
                           SmallArgs{*small, a});
        return check_launch(what);
    }
    const int64_t blocks = (static_cast<int64_t>(a.chunks) * a.cols + kThreads / LPR - 1) / (kThreads / LPR);
    constexpr int kPerBlock = kThreads / 64 * join_chunks<LPR>();
    const int64_t joins = static_cast<int64_t>((a.chunks + kPerBlock - 1) / kPerBlock) * a.cols;
    const int64_t tail = a.unique ? (static_cast<int64_t>(a.n) * a.D * OT::kBytes / 16 + 16 * kThreads - 1) / (16 * kThreads) : 0;
    a.join_blocks = static_cast<uint32_t>(joins);
    const dim3 fold(static_cast<unsigned>(blocks)), join(static_cast<unsigned>(joins + (tail < 4096 ? tail : 4096)));
    if (past) {
        hipLaunchKernelGGL((fold_kernel<GT, OT, LPR, true>), fold, dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL((join_kernel<OT, LPR, true>), join, dim3(kThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL((fold_kernel<GT, OT, LPR, false>), fold, dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL((join_kernel<OT, LPR, false>), join, dim3(kThreads), 0, stream, a);
    }
    return check_launch(what);
}

// lanes that share a row in the fold, the join and the one launch of few ids
int lanes_of(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

template <class GT, class OT>
int launch_fold(FoldArgs& a, const SortArgs* small, bool past, hipStream_t stream, const char* what) {
    switch (lanes_of(a.D)) {
        case 4: return launch_fold_as<GT, OT, 4>(a, small, past, stream, what);
        case 8: return launch_fold_as<GT, OT, 8>(a, small, past, stream, what);
        case 16: return launch_fold_as<GT, OT, 16>(a, small, past, stream, what);
        case 32: return launch_fold_as<GT, OT, 32>(a, small, past, stream, what);
        default: return launch_fold_as<GT, OT, 64>(a, small, past, stream, what);
    }
}

int launch_fold_types(FoldArgs& a, const SortArgs* small, bool past, int32_t gd, int32_t od, hipStream_t stream,
                      const char* what) {
    if (gd == ENGRAM_BF16) {
        if (od == ENGRAM_BF16) return launch_fold<Bf16, Bf16>(a, small, past, stream, what);
        return launch_fold<Bf16, F32>(a, small, past, stream, what);
    }
    if (od == ENGRAM_BF16) return launch_fold<F32, Bf16>(a, small, past, stream, what);
    return launch_fold<F32, F32>(a, small, past, stream, what);
}

int check_ids(const char* what, int32_t id_bytes, int64_t T, int64_t stride, int32_t C, int64_t R) {
    if (id_bytes != 4 && id_bytes != 8) return fail(ENGRAM_EINVAL, "%s: id_bytes=%d must be 4 or 8", what, id_bytes);
    if (T < 0) return fail(ENGRAM_EINVAL, "%s: T < 0", what);
    if (C < 1 || C > 1024) return fail(ENGRAM_EINVAL, "%s: C=%d outside [1, 1024]", what, C);
    if (stride < C) return fail(ENGRAM_EINVAL, "%s: id_token_stride < C", what);
    if (T > kMaxIds / C) return fail(ENGRAM_EINVAL, "%s: more than 2^30 ids", what);
    if (R < 1 || R > 0x7FFFFFFF) return fail(ENGRAM_EINVAL, "%s: R=%lld outside [1, 2^31)", what, (long long)R);
    return ENGRAM_OK;
}

// The fold's threads, the most of any launch here: its lanes for every chunk and column block.  2^32 of them, which no grid
// holds, are 2^30 positions times blocks of 512 columns: half a TB of upstream rows at the least.
int check_work(const char* what, int64_t n, int32_t D) {
    const int64_t lanes = lanes_of(D), cols = (D / 8 + lanes - 1) / lanes, chunks = (n + kChunk - 1) / kChunk;
    if (chunks * cols * lanes + kThreads > 1ll << 32) return fail(ENGRAM_EINVAL, "%s: too many ids for the row width", what);
    return ENGRAM_OK;
}

int check_width(const char* what, int32_t D) {
    if (D < 8 || D % 8 != 0 || D > 65536)
        return fail(ENGRAM_EINVAL, "%s: D=%d must be a multiple of 8 in [8, 65536]", what, D);
    return ENGRAM_OK;
}

}  // namespace

int launch_zero(void* p, int64_t bytes, hipStream_t stream, const char* what) {
    const Zeros z = {static_cast<u32x4*>(p), bytes / 16};
    if (z.n16 == 0) return ENGRAM_OK;
    const int64_t blocks = (z.n16 + kThreads - 1) / kThreads;
    const int64_t x = blocks < kMaxGridX ? blocks : kMaxGridX;
    hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x)),
                       dim3(kThreads), 0, stream, z);
    return check_launch(what);
}

}  // namespace engram

using namespace engram;

extern "C" int engram_embed(const void* ids, int32_t id_bytes, int64_t n, const void* table, int32_t table_dtype,
                            int64_t R, int64_t row_start, int32_t D, float scale, void* out, int32_t out_dtype,
                            void* stream) {
    const char* what = "engram_embed";
    int rc = check_width(what, D);
    if (rc != ENGRAM_OK) return rc;
    if (id_bytes != 4 && id_bytes != 8) return fail(ENGRAM_EINVAL, "%s: id_bytes=%d must be 4 or 8", what, id_bytes);
    if (n < 0) return fail(ENGRAM_EINVAL, "%s: n < 0", what);
    if (R < 1) return fail(ENGRAM_EINVAL, "%s: R < 1", what);
    if (!known_dtype(table_dtype) || !known_dtype(out_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    if (n == 0) return ENGRAM_OK;
    if (!ids || !table || !out) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(ids, id_bytes) || !aligned(table, 16) || !aligned(out, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    EmbedArgs a = {};
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.n = n;
    a.table = static_cast<const uint8_t*>(table);
    a.R = R;
    a.row_start = row_start;
    a.D = D;
    a.scale = scale;
    a.out = static_cast<uint8_t*>(out);
    hipStream_t s = as_stream(stream);
    if (table_dtype == ENGRAM_BF16) {
        if (out_dtype == ENGRAM_BF16) return launch_embed<Bf16, Bf16>(a, s);
        return launch_embed<Bf16, F32>(a, s);
    }
    if (out_dtype == ENGRAM_BF16) return launch_embed<F32, Bf16>(a, s);
    return launch_embed<F32, F32>(a, s);
}

extern "C" int64_t engram_embed_grad_workspace_bytes(int64_t n, int32_t D, int64_t R) {
    if (n < 0 || n > kMaxIds || D < 8 || D % 8 != 0 || D > 65536 || R < 1 || R > 0x7FFFFFFF) return -1;
    return n <= kSmall ? 0 : plan_of(n, D, R).bytes;
}

namespace engram {
namespace {

// What both forms of the gradient do once their arguments are checked (n > 0 ids): `f` holds the outputs.
int embed_grad(FoldArgs& f, const void* ids, int32_t id_bytes, int64_t n, int64_t stride, int32_t C, const void* up,
               int32_t up_dtype, int64_t R, int64_t row_start, int32_t D, float scale, int32_t out_dtype, void* workspace,
               int64_t workspace_bytes, hipStream_t s, const char* what) {
    f.n = static_cast<uint32_t>(n);
    f.R = static_cast<uint32_t>(R);
    f.up = static_cast<const uint8_t*>(up);
    f.D = D;
    f.scale = scale;
    f.row_start = row_start;
    const bool fill = !f.unique && !f.accumulate;
    const int64_t in = up_dtype == ENGRAM_BF16 ? 2 : 4, out = out_dtype == ENGRAM_BF16 ? 2 : 4, bytes = R * D * out;
    const bool past = n * D * (in + out) + (fill ? bytes : 0) > kCacheBytes;
    if (n <= kSmall) {
        if (fill) {
            const int rc = launch_zero(f.out, bytes, s, what);
            if (rc != ENGRAM_OK) return rc;
        }
        SortArgs a = {};
        a.ids = ids;
        a.id_bytes = id_bytes;
        a.C = C;
        a.stride = stride;
        a.row_start = row_start;
        a.R = f.R;
        a.n = f.n;
        return launch_fold_types(f, &a, past, up_dtype, out_dtype, s, what);
    }
    const Plan p = plan_of(n, D, R);
    if (!workspace || !aligned(workspace, 16)) return fail(ENGRAM_EINVAL, "%s: workspace is null or misaligned", what);
    if (workspace_bytes < p.bytes)
        return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                    (long long)p.bytes);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    f.tiles = p.head_tiles;
    f.chunks = p.chunks;
    f.heads = reinterpret_cast<uint32_t*>(ws + p.heads);
    f.chunk_base = reinterpret_cast<uint32_t*>(ws + p.chunk_base);
    f.leave_to = reinterpret_cast<uint32_t*>(ws + p.leave_to);
    f.leave = reinterpret_cast<float*>(ws + p.leave);
    f.enter = reinterpret_cast<float*>(ws + p.enter);
    const int rc = (n <= kOneSort ? one_sort : sort_ids)(p, ids, id_bytes, n, C, stride, R, row_start, ws, f,
                                                         fill ? bytes : 0, s, what);
    if (rc != ENGRAM_OK) return rc;
    if (n > kOneSort && f.unique) hipLaunchKernelGGL(heads_kernel, dim3(p.head_tiles), dim3(kThreads), 0, s, f);
    return launch_fold_types(f, nullptr, past, up_dtype, out_dtype, s, what);
}

}  // namespace
}  // namespace engram

extern "C" int engram_embed_grad(const void* ids, int32_t id_bytes, int64_t T, int64_t id_token_stride, int32_t C,
                                 const void* up, int32_t up_dtype, int64_t R, int64_t row_start, int32_t D,
                                 float scale, void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    const char* what = "engram_embed_grad";
    int rc = check_ids(what, id_bytes, T, id_token_stride, C, R);
    if (rc == ENGRAM_OK) rc = check_width(what, D);
    if (rc == ENGRAM_OK) rc = check_work(what, T * C, D);
    if (rc != ENGRAM_OK) return rc;
    if (!known_dtype(up_dtype) || !known_dtype(grad_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    const int64_t n = T * C;
    if (n == 0 && accumulate) return ENGRAM_OK;
    if (!grad) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(grad, 16)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    if (n) {
        if (!ids || !up) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
        if (!aligned(ids, id_bytes) || !aligned(up, 16))
            return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    }
    hipStream_t s = as_stream(stream);
    if (n == 0) return launch_zero(grad, R * D * (grad_dtype == ENGRAM_BF16 ? 2 : 4), s, what);
    FoldArgs f = {};
    f.out = static_cast<uint8_t*>(grad);
    f.accumulate = accumulate != 0;
    return embed_grad(f, ids, id_bytes, n, id_token_stride, C, up, up_dtype, R, row_start, D, scale, grad_dtype, workspace,
                      workspace_bytes, s, what);
}

extern "C" int engram_embed_grad_rows(const void* ids, int32_t id_bytes, int64_t T, int64_t id_token_stride, int32_t C,
                                      const void* up, int32_t up_dtype, int64_t R, int64_t row_start, int32_t D,
                                      float scale, int64_t* unique, void* rows, int32_t rows_dtype, int32_t* count,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
    const char* what = "engram_embed_grad_rows";
    int rc = check_ids(what, id_bytes, T, id_token_stride, C, R);
    if (rc == ENGRAM_OK) rc = check_width(what, D);
    if (rc == ENGRAM_OK) rc = check_work(what, T * C, D);
    if (rc != ENGRAM_OK) return rc;
    if (!known_dtype(up_dtype) || !known_dtype(rows_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    const int64_t n = T * C;
    if (!count || !aligned(count, 4)) return fail(ENGRAM_EINVAL, "%s: count is null or misaligned", what);
    hipStream_t s = as_stream(stream);
    if (n == 0) {
        hipLaunchKernelGGL(zero_count_kernel, dim3(1), dim3(1), 0, s, count);
        return check_launch(what);
    }
    if (!ids || !up || !unique || !rows) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(ids, id_bytes) || !aligned(up, 16) || !aligned(unique, 8) || !aligned(rows, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    FoldArgs f = {};
    f.out = static_cast<uint8_t*>(rows);
    f.unique = unique;
    f.count = count;
    return embed_grad(f, ids, id_bytes, n, id_token_stride, C, up, up_dtype, R, row_start, D, scale, rows_dtype, workspace,
                      workspace_bytes, s, what);
}
