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
// table: three).  A pass is one launch: every workgroup ranks a tile of kSortTile elements (per wave by ballots over
// the digit's bits, so stable), adds the tiles before it from the table of per-tile digit counts, and scatters.  The
// counts of the next pass are gathered by the scatter itself with integer atomics (their order does not matter).
//
// Fold: the sorted positions are cut into chunks of kChunk; a group of lanes walks a chunk with the row sum in
// registers and writes a table row where its segment ends.  A segment that crosses chunks leaves fp32 partial sums
// (one leaving a chunk, one entering) which a last launch adds in chunk order, so that one hot row costs no more than
// many cold ones.
#include "rows.h"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxDigitBits = 10;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
// up to this many tiles every scattering workgroup adds the digit counts of the tiles before it by itself; past it a
// launch of its own turns the counts into prefixes
constexpr int kDirectTiles = 64;
constexpr int kChunk = 16;   // sorted positions per chunk of the fold
constexpr int64_t kMaxIds = 1ll << 30;

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
    int cols;       // column blocks of LPR * U pieces per row
    int64_t units;  // n * cols
};

__device__ inline int64_t load_id(const void* ids, int id_bytes, int64_t i) {
    return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// A unit: one row's column block, LPR lanes with U pieces each.
template <class TT, class OT, int LPR, int U>
__global__ __launch_bounds__(kThreads) void embed_kernel(EmbedArgs a) {
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    if (unit >= a.units) return;
    const int64_t i = a.cols == 1 ? unit : unit / a.cols;
    const int cb = static_cast<int>(unit - i * a.cols);
    const int64_t r = load_id(a.ids, a.id_bytes, i) - a.row_start;
    const bool ok = r >= 0 && r < a.R;
    const int pieces = a.D / 8;
    const uint8_t* row = a.table + (ok ? r : 0) * a.D * TT::kBytes;
    uint8_t* out = a.out + i * a.D * OT::kBytes;
    const int p0 = cb * (LPR * U) + threadIdx.x % LPR;
    Piece<TT> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (ok && p0 + u * LPR < pieces) v[u].load(row, p0 + u * LPR);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (p0 + u * LPR >= pieces) continue;
        float f[8] = {};
        if (ok) {
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= a.scale;
        }
        Piece<OT> o;
        o.from(f);
        o.store(out, p0 + u * LPR);
    }
}

template <class TT, class OT, int LPR, int U>
int launch_embed_as(EmbedArgs& a, hipStream_t stream) {
    const int pieces = a.D / 8;
    a.cols = (pieces + LPR * U - 1) / (LPR * U);
    a.units = a.n * a.cols;
    const int64_t blocks = (a.units + kThreads / LPR - 1) / (kThreads / LPR);
    if (blocks > 0x7FFFFFFF) return fail(ENGRAM_EINVAL, "engram_embed: too many ids");
    hipLaunchKernelGGL((embed_kernel<TT, OT, LPR, U>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
    return check_launch("engram_embed");
}

template <class TT, class OT>
int launch_embed(EmbedArgs& a, hipStream_t stream) {
    const int pieces = a.D / 8;
    if (pieces <= 8) return launch_embed_as<TT, OT, 8, 1>(a, stream);
    if (pieces <= 16) return launch_embed_as<TT, OT, 16, 1>(a, stream);
    if (pieces <= 32) return launch_embed_as<TT, OT, 32, 1>(a, stream);
    return launch_embed_as<TT, OT, 64, 1>(a, stream);
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
    const Pair* in;    // later passes
    Pair* out;
    uint32_t* hist;       // [tiles][digits] this pass's digit counts per tile (or their prefixes over the tiles)
    uint32_t* totals;     // [digits], with prefixes
    uint32_t* hist_next;  // [tiles][digits] of the next pass, zeroed, or null
    int shift, bits;      // this pass's digit
    int tiles;
};

__device__ inline uint32_t load_key(const SortArgs& a, uint32_t i) {
    int64_t at = i;
    if (a.stride != a.C) {
        const uint32_t t = i / static_cast<uint32_t>(a.C);
        at = static_cast<int64_t>(t) * a.stride + (i - t * static_cast<uint32_t>(a.C));
    }
    const int64_t r = load_id(a.ids, a.id_bytes, at) - a.row_start;
    return r >= 0 && r < static_cast<int64_t>(a.R) ? static_cast<uint32_t>(r) : a.R;
}

// The first pass's digit counts per tile, and the later passes' count tables zeroed.
__global__ __launch_bounds__(kSortThreads) void hist_kernel(SortArgs a, uint32_t* zero, uint32_t zero_n) {
    __shared__ uint32_t h[kMaxDigits];
    const int digits = 1 << a.bits;
    for (int d = threadIdx.x; d < digits; d += kSortThreads) h[d] = 0;
    for (uint32_t z = blockIdx.x * kSortThreads + threadIdx.x; z < zero_n; z += gridDim.x * kSortThreads) zero[z] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * kSortTile + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
        const uint32_t i = base + u * kSortThreads;
        if (i < a.n) atomicAdd(&h[load_key(a, i) & (digits - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.hist[blockIdx.x * digits + d] = h[d];
}

// hist[tile][digit] into the counts of the tiles before, and the totals: 64 digits per workgroup, 16 runs of tiles.
__global__ __launch_bounds__(1024) void prefix_kernel(SortArgs a) {
    __shared__ uint32_t part[16][64];
    const int digits = 1 << a.bits;
    const int d = blockIdx.x * 64 + (threadIdx.x & 63);
    const int run = threadIdx.x >> 6;
    const int per = (a.tiles + 15) / 16;
    const int t0 = min(run * per, a.tiles), t1 = min(t0 + per, a.tiles);
    uint32_t sum = 0;
    if (d < digits)
        for (int t = t0; t < t1; ++t) sum += a.hist[t * digits + d];
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
    for (int t = t0; t < t1; ++t) {
        const uint32_t v = a.hist[t * digits + d];
        a.hist[t * digits + d] = base;
        base += v;
    }
    if (run == 0) a.totals[d] = total;
}

template <bool kFirst>
__global__ __launch_bounds__(kSortThreads) void scatter_kernel(SortArgs a) {
    __shared__ uint32_t cnt[kSortWaves][kMaxDigits];
    __shared__ uint32_t wave_sum[kSortWaves];
    const int digits = 1 << a.bits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t mask_bits = static_cast<uint32_t>(digits - 1);
    for (int d = threadIdx.x; d < digits * kSortWaves; d += kSortThreads) cnt[d / digits][d % digits] = 0;

    // the wave's kSortItems * 64 consecutive elements
    Pair e[kSortItems];
    uint32_t rank[kSortItems];
    const uint32_t first = blockIdx.x * kSortTile + wave * (64 * kSortItems) + lane;
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
        const uint32_t i = first + u * 64;
        e[u] = Pair{0, i};
        if (i < a.n) {
            if (kFirst) e[u].key = load_key(a, i);
            else e[u] = a.in[i];
        }
    }
    __syncthreads();
    volatile uint32_t* mine = cnt[wave];  // this wave's counters: its LDS accesses stay in program order
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
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
        if (live && before == 0) mine[d] = have + __popcll(same);
    }
    __syncthreads();

    // each thread owns the digits [own, own + per): the elements with a smaller digit, the tiles before this one and
    // the waves before each wave
    constexpr int kPer = kMaxDigits / kSortThreads;
    const int per = digits >= kSortThreads ? digits / kSortThreads : 1;
    const int own = threadIdx.x * per;
    uint32_t total[kPer] = {}, prior[kPer] = {};
    if (own < digits) {
        if (a.totals) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (j < per) {
                    total[j] = a.totals[own + j];
                    prior[j] = a.hist[blockIdx.x * digits + own + j];
                }
        } else {
            for (int t = 0; t < a.tiles; ++t) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < per) {
                        const uint32_t v = a.hist[t * digits + own + j];
                        total[j] += v;
                        prior[j] += t < static_cast<int>(blockIdx.x) ? v : 0;
                    }
            }
        }
    }
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += total[j];
    uint32_t scan = sum;  // inclusive over the wave's threads
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(scan, off, 64);
        scan += lane >= off ? o : 0;
    }
    if (lane == 63) wave_sum[wave] = scan;
    __syncthreads();
    uint32_t base = scan - sum;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    if (own < digits) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per) {
                uint32_t at = base + prior[j];
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) {
                    const uint32_t c = cnt[w][own + j];
                    cnt[w][own + j] = at;
                    at += c;
                }
                base += total[j];
            }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
        if (first + u * 64 >= a.n) continue;
        const uint32_t to = cnt[wave][(e[u].key >> a.shift) & mask_bits] + rank[u];
        a.out[to] = e[u];
        if (a.hist_next) {
            const uint32_t d2 = (e[u].key >> (a.shift + a.bits)) & mask_bits;
            atomicAdd(&a.hist_next[to / kSortTile * digits + d2], 1u);
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------------
// fold
// ---------------------------------------------------------------------------------------------------------------------
struct FoldArgs {
    const Pair* sorted;
    uint32_t n, R;
    const uint8_t* up;  // [n, D] upstream rows
    int D;
    int cols;           // column blocks of 64 pieces
    float scale;
    uint8_t* out;       // dense: [R, D]; rows: [n, D]
    int accumulate;
    // rows form
    int64_t* unique;    // [n], or null: the dense form
    int32_t* count;     // [1]
    int64_t row_start;
    uint32_t* heads;       // [tiles] distinct rows that begin in each tile of kSortTile sorted positions
    uint32_t* chunk_base;  // [chunks] of those, the ones before the chunk
    int tiles;
    uint32_t chunks;
    float* leave;       // [chunks][D] sum of a segment that begins in the chunk and goes on after it
    float* enter;       // [chunks][D] sum of the chunk's share of a segment that began before it
};

// Distinct rows per chunk (before it in its tile) and per tile.
__global__ __launch_bounds__(kThreads) void heads_kernel(FoldArgs a) {
    constexpr int kPerTile = kSortTile / kChunk;
    static_assert(kPerTile == kThreads, "one chunk per thread");
    __shared__ uint32_t wsum[kThreads / 64];
    const uint32_t chunk = blockIdx.x * kPerTile + threadIdx.x;
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
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        base += w < wave ? wsum[w] : 0;
        all += wsum[w];
    }
    if (chunk < a.chunks) a.chunk_base[chunk] = base + scan - c;
    if (threadIdx.x == 0) a.heads[blockIdx.x] = all;
}

// The distinct rows before tile `tile` (all of them for tile == tiles): every wave adds them itself.
__device__ inline uint32_t heads_before(const FoldArgs& a, int tile) {
    uint32_t s = 0;
    for (int t = threadIdx.x & 63; t < tile; t += 64) s += a.heads[t];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    return s;
}

template <class OT>
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
    o.store(row, piece);
    if (a.unique && piece == 0) a.unique[u] = static_cast<int64_t>(key) + a.row_start;
}

// One group of LPR lanes per (chunk, column block).
template <class GT, class OT, int LPR>
__global__ __launch_bounds__(kThreads) void fold_kernel(FoldArgs a) {
    constexpr int kGroups = kThreads / LPR;
    constexpr int kBatch = GT::kBytes == 2 ? 8 : 4;  // upstream pieces in flight per lane
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LPR;
    const uint32_t chunk = static_cast<uint32_t>(unit / a.cols);
    const int piece = static_cast<int>(unit % a.cols) * LPR + threadIdx.x % LPR;
    uint32_t u = 0;
    if (a.unique) {
        // a workgroup's chunks lie in one or two tiles: the distinct rows before the first, then on by its own count
        const uint32_t c0 = static_cast<uint32_t>(static_cast<int64_t>(blockIdx.x) * kGroups / a.cols);
        constexpr int kPerTile = kSortTile / kChunk;
        const uint32_t t0 = min(c0, a.chunks - 1) / kPerTile;
        u = heads_before(a, static_cast<int>(t0));
        if (chunk < a.chunks) {
            for (uint32_t t = t0; t < chunk / kPerTile; ++t) u += a.heads[t];
            u += a.chunk_base[chunk];
        }
    }
    if (chunk >= a.chunks) return;
    const bool live = piece < a.D / 8;
    const uint32_t s = chunk * kChunk, e = min(s + kChunk, a.n);
    uint32_t prev = s ? a.sorted[s - 1].key : 0xFFFFFFFFu;
    const uint32_t after = e < a.n ? a.sorted[e].key : a.R;  // R: nothing goes on
    float acc[8] = {};
    bool entered = true;   // the running segment began before the chunk
    bool open = false;     // a segment is running
    uint32_t cur = prev;
    auto close = [&](bool goes_on) {
        if (!open || !live) return;
        if (entered) {
            Piece<F32> p;
            p.from(acc);
            p.store(a.enter + static_cast<int64_t>(chunk) * a.D, piece);
        } else if (goes_on) {
            Piece<F32> p;
            p.from(acc);
            p.store(a.leave + static_cast<int64_t>(chunk) * a.D, piece);
        } else {
            put_row<OT>(a, cur, u - 1, piece, acc);
        }
    };
    for (uint32_t b = s; b < e; b += kBatch) {
        Pair pr[kBatch];
        Piece<GT> v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) pr[j] = b + j < e ? a.sorted[b + j] : Pair{a.R, 0};
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (pr[j].key < a.R && live) v[j].load(a.up + static_cast<int64_t>(pr[j].pos) * a.D * GT::kBytes, piece);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (b + j >= e || pr[j].key >= a.R) continue;
            float f[8];
            if (live) v[j].to(f);
            if (pr[j].key != cur) {
                close(false);
                cur = pr[j].key;
                entered = false;
                ++u;
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = live ? f[q] : 0.f;
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] += live ? f[q] : 0.f;
            }
            open = true;
        }
    }
    close(after == cur);
}

// Segments that cross chunks: the chunk where one begins adds its own partial sum and those of the chunks it enters,
// in order.  In the rows form also the rows past the last distinct one: zeros, and -1 for their ids.
template <class OT, int LPR>
__global__ __launch_bounds__(kThreads) void join_kernel(FoldArgs a) {
    constexpr int kGroups = kThreads / LPR;
    constexpr int kPerTile = kSortTile / kChunk;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LPR;
    const uint32_t chunk = static_cast<uint32_t>(unit / a.cols);
    const int piece = static_cast<int>(unit % a.cols) * LPR + threadIdx.x % LPR;
    uint32_t before = 0, all = 0, t0 = 0;
    if (a.unique) {
        const uint32_t c0 = static_cast<uint32_t>(static_cast<int64_t>(blockIdx.x) * kGroups / a.cols);
        t0 = min(c0, a.chunks - 1) / kPerTile;
        before = heads_before(a, static_cast<int>(t0));
        all = heads_before(a, a.tiles);
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = static_cast<int32_t>(all);
    }
    if (chunk >= a.chunks || piece >= a.D / 8) return;
    const uint32_t s = chunk * kChunk, e = min(s + kChunk, a.n);
    if (a.unique) {
        Piece<OT> z;
        const float zero[8] = {};
        z.from(zero);
        for (uint32_t k = max(s, all); k < e; ++k) {
            z.store(a.out + static_cast<int64_t>(k) * a.D * OT::kBytes, piece);
            if (piece == 0) a.unique[k] = -1;
        }
    }
    if (e >= a.n) return;
    const uint32_t key = a.sorted[e].key;
    if (key >= a.R || a.sorted[e - 1].key != key) return;                                  // nothing crosses the end
    if (s && a.sorted[s - 1].key == key) return;                                           // it began before
    float acc[8];
    Piece<F32> p;
    p.load(a.leave + static_cast<int64_t>(chunk) * a.D, piece);
    p.to(acc);
    for (uint32_t c = chunk + 1; c < a.chunks && a.sorted[c * kChunk].key == key; ++c) {
        float f[8];
        p.load(a.enter + static_cast<int64_t>(c) * a.D, piece);
        p.to(f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += f[q];
    }
    uint32_t u = 0;
    if (a.unique) {  // the segment is the last that begins in its chunk
        u = before;
        for (uint32_t t = t0; t < (chunk + 1) / kPerTile; ++t) u += a.heads[t];
        if ((chunk + 1) % kPerTile) u += a.chunk_base[chunk + 1];
        u -= 1;
    }
    put_row<OT>(a, key, u, piece, acc);
}

// zeros over 16-byte pieces
__global__ __launch_bounds__(kThreads) void zero_kernel(u32x4* p, int64_t n16) {
    const u32x4 z = {};
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n16;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
        p[i] = z;
}

__global__ void zero_count_kernel(int32_t* count) { *count = 0; }

// ---------------------------------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------------------------------
int bits_of(uint32_t v) { return v ? 32 - __builtin_clz(v) : 1; }

struct Plan {
    int bits, passes;      // digit bits and passes
    int tiles;
    uint32_t chunks;
    int64_t pairs, hist, totals, heads, chunk_base, leave, enter, bytes;  // offsets
};

int64_t up16(int64_t v) { return (v + 15) & ~15ll; }

Plan plan_of(int64_t n, int32_t D, int64_t R) {
    Plan p;
    const int key_bits = bits_of(static_cast<uint32_t>(R));  // the key R stands for ids outside
    p.passes = (key_bits + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    p.tiles = static_cast<int>((n + kSortTile - 1) / kSortTile);
    p.chunks = static_cast<uint32_t>((n + kChunk - 1) / kChunk);
    int64_t at = 0;
    p.pairs = at;
    at += up16(2 * n * static_cast<int64_t>(sizeof(Pair)));
    p.hist = at;
    at += up16(static_cast<int64_t>(p.passes) * p.tiles * (4ll << p.bits));
    p.totals = at;
    at += up16(4ll << p.bits);
    p.heads = at;
    at += up16(4ll * p.tiles);
    p.chunk_base = at;
    at += up16(4ll * p.chunks);
    p.leave = at;
    at += up16(4ll * p.chunks * D);
    p.enter = at;
    at += up16(4ll * p.chunks * D);
    p.bytes = at;
    return p;
}

// sorted (row, position) pairs of the ids, in the workspace
const Pair* sort_ids(const Plan& p, const void* ids, int id_bytes, int64_t n, int C, int64_t stride, int64_t R,
                     int64_t row_start, uint8_t* ws, hipStream_t stream) {
    Pair* buf[2] = {reinterpret_cast<Pair*>(ws + p.pairs), reinterpret_cast<Pair*>(ws + p.pairs) + n};
    const uint32_t table = static_cast<uint32_t>(p.tiles) << p.bits;
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.hist);
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
    a.hist = hist;
    hipLaunchKernelGGL(hist_kernel, dim3(p.tiles), dim3(kSortThreads), 0, stream, a, hist + table,
                       table * (p.passes - 1));
    for (int q = 0; q < p.passes; ++q) {
        a.shift = q * p.bits;
        a.hist = hist + static_cast<int64_t>(table) * q;
        a.hist_next = q + 1 < p.passes ? a.hist + table : nullptr;
        a.in = buf[(q + 1) & 1];
        a.out = buf[q & 1];
        a.totals = nullptr;
        if (p.tiles > kDirectTiles) {
            a.totals = reinterpret_cast<uint32_t*>(ws + p.totals);
            hipLaunchKernelGGL(prefix_kernel, dim3(((1 << p.bits) + 63) / 64), dim3(1024), 0, stream, a);
        }
        if (q == 0)
            hipLaunchKernelGGL(scatter_kernel<true>, dim3(p.tiles), dim3(kSortThreads), 0, stream, a);
        else
            hipLaunchKernelGGL(scatter_kernel<false>, dim3(p.tiles), dim3(kSortThreads), 0, stream, a);
    }
    return buf[(p.passes - 1) & 1];
}

template <class GT, class OT, int LPR>
int launch_fold_as(FoldArgs& a, hipStream_t stream, const char* what) {
    a.cols = (a.D / 8 + LPR - 1) / LPR;
    const int64_t groups = static_cast<int64_t>(a.chunks) * a.cols;
    const int64_t blocks = (groups + kThreads / LPR - 1) / (kThreads / LPR);
    if (blocks > 0x7FFFFFFF) return fail(ENGRAM_EINVAL, "%s: too many ids for the row width", what);
    hipLaunchKernelGGL((fold_kernel<GT, OT, LPR>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
    hipLaunchKernelGGL((join_kernel<OT, LPR>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
    return check_launch(what);
}

template <class GT, class OT>
int launch_fold(FoldArgs& a, hipStream_t stream, const char* what) {
    const int pieces = a.D / 8;
    if (pieces <= 4) return launch_fold_as<GT, OT, 4>(a, stream, what);
    if (pieces <= 8) return launch_fold_as<GT, OT, 8>(a, stream, what);
    if (pieces <= 16) return launch_fold_as<GT, OT, 16>(a, stream, what);
    if (pieces <= 32) return launch_fold_as<GT, OT, 32>(a, stream, what);
    return launch_fold_as<GT, OT, 64>(a, stream, what);
}

int launch_fold_types(FoldArgs& a, int32_t gd, int32_t od, hipStream_t stream, const char* what) {
    if (gd == ENGRAM_BF16) {
        if (od == ENGRAM_BF16) return launch_fold<Bf16, Bf16>(a, stream, what);
        return launch_fold<Bf16, F32>(a, stream, what);
    }
    if (od == ENGRAM_BF16) return launch_fold<F32, Bf16>(a, stream, what);
    return launch_fold<F32, F32>(a, stream, what);
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

int check_width(const char* what, int32_t D) {
    if (D < 8 || D % 8 != 0 || D > 65536)
        return fail(ENGRAM_EINVAL, "%s: D=%d must be a multiple of 8 in [8, 65536]", what, D);
    return ENGRAM_OK;
}

}  // namespace

int launch_zero(void* p, int64_t bytes, hipStream_t stream, const char* what) {
    const int64_t n16 = bytes / 16;
    if (n16 == 0) return ENGRAM_OK;
    const int64_t blocks = (n16 + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)), dim3(kThreads), 0, stream,
                       static_cast<u32x4*>(p), n16);
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
    return n == 0 ? 0 : plan_of(n, D, R).bytes;
}

extern "C" int engram_embed_grad(const void* ids, int32_t id_bytes, int64_t T, int64_t id_token_stride, int32_t C,
                                 const void* up, int32_t up_dtype, int64_t R, int64_t row_start, int32_t D,
                                 float scale, void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    const char* what = "engram_embed_grad";
    int rc = check_ids(what, id_bytes, T, id_token_stride, C, R);
    if (rc == ENGRAM_OK) rc = check_width(what, D);
    if (rc != ENGRAM_OK) return rc;
    if (!known_dtype(up_dtype) || !known_dtype(grad_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    const int64_t n = T * C;
    if (n == 0 && accumulate) return ENGRAM_OK;
    if (!grad) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(grad, 16)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    if (n) {
        if (!ids || !up || !workspace) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
        if (!aligned(ids, id_bytes) || !aligned(up, 16) || !aligned(workspace, 16))
            return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    }
    hipStream_t s = as_stream(stream);
    Plan p = {};
    if (n) {
        p = plan_of(n, D, R);
        if (workspace_bytes < p.bytes)
            return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                        (long long)p.bytes);
    }
    if (!accumulate) {
        rc = launch_zero(grad, R * D * (grad_dtype == ENGRAM_BF16 ? 2 : 4), s, what);
        if (rc != ENGRAM_OK || n == 0) return rc;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    FoldArgs f = {};
    f.sorted = sort_ids(p, ids, id_bytes, n, C, id_token_stride, R, row_start, ws, s);
    f.n = static_cast<uint32_t>(n);
    f.R = static_cast<uint32_t>(R);
    f.up = static_cast<const uint8_t*>(up);
    f.D = D;
    f.scale = scale;
    f.out = static_cast<uint8_t*>(grad);
    f.accumulate = accumulate != 0;
    f.tiles = p.tiles;
    f.chunks = p.chunks;
    f.leave = reinterpret_cast<float*>(ws + p.leave);
    f.enter = reinterpret_cast<float*>(ws + p.enter);
    return launch_fold_types(f, up_dtype, grad_dtype, s, what);
}

extern "C" int engram_embed_grad_rows(const void* ids, int32_t id_bytes, int64_t T, int64_t id_token_stride, int32_t C,
                                      const void* up, int32_t up_dtype, int64_t R, int64_t row_start, int32_t D,
                                      float scale, int64_t* unique, void* rows, int32_t rows_dtype, int32_t* count,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
    const char* what = "engram_embed_grad_rows";
    int rc = check_ids(what, id_bytes, T, id_token_stride, C, R);
    if (rc == ENGRAM_OK) rc = check_width(what, D);
    if (rc != ENGRAM_OK) return rc;
    if (!known_dtype(up_dtype) || !known_dtype(rows_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    const int64_t n = T * C;
    if (!count || !aligned(count, 4)) return fail(ENGRAM_EINVAL, "%s: count is null or misaligned", what);
    hipStream_t s = as_stream(stream);
    if (n == 0) {
        hipLaunchKernelGGL(zero_count_kernel, dim3(1), dim3(1), 0, s, count);
        return check_launch(what);
    }
    if (!ids || !up || !workspace || !unique || !rows) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(ids, id_bytes) || !aligned(up, 16) || !aligned(workspace, 16) || !aligned(unique, 8) || !aligned(rows, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const Plan p = plan_of(n, D, R);
    if (workspace_bytes < p.bytes)
        return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                    (long long)p.bytes);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    FoldArgs f = {};
    f.sorted = sort_ids(p, ids, id_bytes, n, C, id_token_stride, R, row_start, ws, s);
    f.n = static_cast<uint32_t>(n);
    f.R = static_cast<uint32_t>(R);
    f.up = static_cast<const uint8_t*>(up);
    f.D = D;
    f.scale = scale;
    f.out = static_cast<uint8_t*>(rows);
    f.unique = unique;
    f.count = count;
    f.row_start = row_start;
    f.tiles = p.tiles;
    f.chunks = p.chunks;
    f.heads = reinterpret_cast<uint32_t*>(ws + p.heads);
    f.chunk_base = reinterpret_cast<uint32_t*>(ws + p.chunk_base);
    f.leave = reinterpret_cast<float*>(ws + p.leave);
    f.enter = reinterpret_cast<float*>(ws + p.enter);
    hipLaunchKernelGGL(heads_kernel, dim3(p.tiles), dim3(kThreads), 0, s, f);
    return launch_fold_types(f, up_dtype, rows_dtype, s, what);
}
