// The `wkv` Linear with 4-bit block-scaled weights, in the OCP microscaling (MX) fp4 format: E2M1 elements, one E8M0
// scale per 32 consecutive input columns of a row.
//
//   engram_mx4_quant        -- bf16 rows -> MXFP4 (activations, and the weights' one-off conversion)
//   engram_mx4_pack_weight  -- MXFP4 weights -> the layout that the products read (one-off)
//   engram_wkv_mx4          -- kv = A * W^T, A in MXFP8 or MXFP4, with v_mfma_scale_f32_16x16x128_f8f6f4
//   engram_wkv_mx4_gate     -- the same fused with the gate pre-activation (Engram.forward's rstd and dot)
//
// Weight layout: uint8 [ceil(N/64)][K/128][4352], a record for 64 rows and 128 columns: four W operands of the matrix
// instruction as its lanes hold them, 1 KB each (operand j: rows 16 j .. 16 j + 15; lane l = 16 c + r has the 16 bytes of row
// 16 j + r, columns 32 c .. 32 c + 31, the even column in the low half of a byte), then a 32-bit word per lane with its scale
// in each operand (byte j: row 16 j + r, block c).  So a wave reads a W operand with one load a lane, 1 KB in a row, straight
// into registers, and the scales of four with one load; the instruction picks a scale's byte by its operand selector.
//
// The instruction's lanes, measured on gfx950: of a 4-bit operand lane l holds row l % 16, columns 32 (l / 16) .. +31 (16
// bytes); of an 8-bit one columns 16 (l / 16) .. +15 and 64 + 16 (l / 16) .. +15 (32 bytes); the scale operand of lane l is
// that of row l % 16 and block l / 16 in either format.  Lane l of the result holds rows 4 (l / 16) .. +3 of column l % 16.
// W is the first operand, so a lane has four consecutive outputs of one token.
#include <type_traits>

#include "common.h"
#include "gate.h"
#include "mx.h"
#include "mx4_rows.h"

namespace engram {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kStepCols = 128;    // columns of one matrix instruction
constexpr int kGroupRows = 64;    // weight rows of a record
constexpr int kRecord = 4352;     // bytes of a record: 4 x 1,024 of elements, 256 of scales
constexpr int kFp8 = 0, kFp4 = 4; // the instruction's format selectors

struct Mx4Args {
    const uint8_t* a;    // [M, K] E4M3 or [M, K/2] E2M1 pairs
    const uint8_t* as;   // [K/128][M4][4] E8M0
    const uint8_t* w;    // packed records
    uint16_t* kv;        // [M, ld_out] bf16: the columns from n_key on
    int64_t M, M4, ld_out;
    int N, steps;        // columns, K / 128
    int group, across;   // the tiles' order: groups of so many tile rows (across: tile columns), each walked along the other axis
    // the fused gate: columns below n_key are keys, reduced against the stream and not stored
    const uint16_t* x;   // [M, hc, dim] bf16
    const uint16_t* q;   // [hc, dim] bf16
    const uint16_t* k;
    float* part;         // [hc * dim / 128][3][M]: per 128 columns sum(h w key), sum(key^2), sum(h^2)
    int n_key;
};

__device__ inline bf16x2 as_pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// c + a.lo * b.lo + a.hi * b.hi over packed bf16 pairs, fp32 accumulation
__device__ inline float dot2_bf16(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(as_pair(a), as_pair(b), c, false);
}

// a's two halves of a wave added in the lower one, b's in the upper; of every half the same for a's and b's rows of 16 lanes
__device__ inline float add_halves(float a, float b) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ inline float add_rows(float a, float b) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// a token operand of the matrix instruction
template <bool kA8>
struct AFrag;
template <>
struct AFrag<true> {
    i32x4 lo, hi;
    __device__ inline i32x8 get() const { return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}; }
};
template <>
struct AFrag<false> {
    i32x4 lo;
    __device__ inline i32x8 get() const { return i32x8{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0}; }
};

// acc += (W operand, scales in byte kSel of sw) x (token operand, scale in byte 0 of sa)
template <bool kA8, int kSel>
__device__ inline f32x4 mfma(const i32x4& w, int sw, const AFrag<kA8>& a, int sa, f32x4 acc) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a.get(), acc, kFp4,
                                                            kA8 ? kFp8 : kFp4, kSel, sw, 0, sa);
}

// ---- tiles: a workgroup of NW waves has 16 MI tokens x 64 NW columns, two waves a SIMD, so that one workgroup's stores, sums
// and first loads run under another's matrix instructions.  A wave has all tokens and 64 columns, MI x 4 blocks of 16 x 16.  The
// token rows come through LDS, 128 bytes of each (128 columns in 8 bits, 256 in 4) a stage, by direct-to-LDS loads (rows past M
// are outside their resource and read as zero); the weights go from memory to the registers, kSets steps ahead, each read by one
// wave only.  Large products: matrix instructions, stores and loads add up (of 65,536 x 1,536 x 25,600 without stores 80 % of the
// time, without any load 75 %; tiles of 256 x 128 whose waves share weights, at 64 bytes of a row a load, kept the CU's address
// unit busy for 84 % of the clocks and took 17 % more), so as few bytes and as long runs as the registers allow.  A few tokens are
// bound by the weights' way from HBM, so as many steps in flight as they allow (more than four measured no faster).
//
// 1,536 x 25,600, us with 8-bit / 4-bit rows: 1 token 6.9 / 6.8 with the weights from HBM and 5.9 / 5.8 where the Infinity Cache
// holds them, 256 16.4 / 14.9 and 11.9 / 9.8, 8,192 231 / 166, 65,536 1,834 / 1,291 (2.8 / 4.0 PFLOP/s); 6,144 x 25,600: 8,192
// tokens 819 / 538 (3.1 / 4.8, the instruction alone 4.1 / 6.9).  Fused, 4 x 5,120: 256 20.9 / 19.5 and 19.0 / 17.6, 8,192 266 /
// 199, 65,536 2,064 / 1,540.
//
// LDS rows: the 16-byte piece c of a row at slot c ^ (row / 2) % 8: neighbouring lanes' pieces lie in different banks.
constexpr int kBufferWord3 = 0x00020000;
constexpr int kWaitLgkmcnt0 = 0xC07F;
constexpr int wait_vmcnt(int n) { return (n & 0xF) | ((n >> 4) << 14) | 0x0F70; }
// until at most n of the wave's loads are outstanding (a constant once unrolled; even, up to 14)
__device__ __forceinline__ void wait_loads(int n) {
    switch (n) {
        case 14: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(14));
        case 12: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(12));
        case 10: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(10));
        case 8: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(8));
        case 6: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(6));
        case 4: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(4));
        case 2: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(2));
        default: return __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
    }
}
constexpr int kNonTemporal = 2;  // cache-policy operand of a load or store: streamed past L2
constexpr int kXcds = 8;

__device__ inline i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
    return i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}
__device__ inline int load4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}

template <bool kA8, int MI, int NW, int kSets, bool kGate>
__device__ __forceinline__ void mx4_tile_body(const Mx4Args& p, int tiles_m, int tiles_n) {
    constexpr int BM = 16 * MI, BN = 64 * NW;
    using Rows = Mx4Rows<kA8, BM, NW>;
    constexpr int kSub = Rows::kSub;                        // steps of a stage
    constexpr int kScales = BM * 128;                       // a stage: its rows, then a word per row and step
    constexpr int kScaleRows = BM > 64 ? BM : 64;           // (a load of them writes 64 words)
    constexpr int kStageBytes = kScales + kSub * kScaleRows * 4;
    constexpr int kRowLoads = Rows::kLoads;                 // per wave and stage
    constexpr int kScaleLoads = (kSub * kScaleRows + BN - 1) / BN;  // 64 rows of a step each
    constexpr int kLoads = kRowLoads + kScaleLoads;
    constexpr int kWLoads = 5;
    constexpr int kStages = kSets > 1 ? kSets / kSub + 1 : 2;
    constexpr int kRing = kStages * kStageBytes;
    constexpr int kWaveBytes = BM * 128;                    // a wave's part of the tile as bf16, behind the last step
    // The gate's stream rows are loaded ahead of the steps where they are few (16 tokens 9.9 us, 10.3 behind them), else behind
    // them (256 tokens and their residual 23.3 us, 23.5 ahead).  Up to 64 tokens a tile they stay in the caches for the residual
    // that follows (256 tokens 23.3, past them 24.0); where there are many they go past them (8,192 tokens 320, 330).
    constexpr bool kEarly = kGate && MI <= 2;
    constexpr int kStreamPolicy = MI <= 4 ? 0 : kNonTemporal;
    constexpr int kParts = kEarly ? kRing : 0;
    constexpr int kLds = kParts + NW * kWaveBytes > kRing ? kParts + NW * kWaveBytes : kRing;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;
    const int S = p.steps;
    // the workgroup's tile: an XCD (workgroups % 8) takes a contiguous run of the order
    int64_t m0;
    int n0;
    {
        const uint32_t n = static_cast<uint32_t>(tiles_m) * static_cast<uint32_t>(tiles_n);
        const uint32_t pid = static_cast<uint32_t>(group_index()), xcd = pid % kXcds, per = n / kXcds, rem = n % kXcds;
        if (pid >= n) return;
        const uint32_t at = xcd * per + min(xcd, rem) + pid / kXcds;
        const uint32_t outer = p.across ? tiles_n : tiles_m, inner = p.across ? tiles_m : tiles_n, depth = p.group;
        const uint32_t group = at / (depth * inner), first = group * depth, deep = min(outer - first, depth);
        const uint32_t left = at - first * inner, i = left / deep, o = first + left - i * deep;
        m0 = static_cast<int64_t>(p.across ? i : o) * BM;
        n0 = static_cast<int>(p.across ? o : i) * BN;
    }
    const int row_bytes = Rows::row_bytes(S);
    const int valid_bytes = static_cast<int>(min<int64_t>(BM, p.M - m0)) * row_bytes;
    const int row0 = Rows::first(wave);  // load q of the wave fills 1 KB, rows row0 + 8 q on
    const uint32_t voff[2] = {Rows::offset(row0, lane, false, row_bytes), Rows::offset(row0, lane, true, row_bytes)};
    const int scale_bytes = static_cast<int>(min<int64_t>(BM, p.M4 - m0)) * 4;
    // load q (0 .. kLoads - 1) of a stage into the one at `slot`: the rows', then their scales; past the last step nothing is
    // fetched (zeros are written)
    auto issue = [&](int stage, int slot, int q) {
        uint8_t* st = lds + slot;
        if (q < kRowLoads) {
            const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(p.a + m0 * row_bytes + Rows::begin(stage)), 0, Rows::bytes(stage, S, valid_bytes),
                kBufferWord3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, st + (row0 + 8 * q) * 128, 16,
                                                     voff[q & 1] + Rows::load_rows(q, row_bytes), 0, 0, 0);
        } else {
            const int u = (wave + NW * (q - kRowLoads)) * 64 % (kSub * kScaleRows);  // (some waves load the same here too)
            const int s = stage * kSub + u / kScaleRows;
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(p.as + (static_cast<int64_t>(s) * p.M4 + m0) * 4), 0, s < S ? scale_bytes : 0, kBufferWord3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, st + kScales + u * 4, 4,
                                                     static_cast<uint32_t>((u % kScaleRows + lane) * 4), 0, 0, 0);
        }
    };
    const int group = min(n0 / kGroupRows + wave, (p.N + kGroupRows - 1) / kGroupRows - 1);  // (columns past N are not stored)
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.w + static_cast<int64_t>(group) * S * kRecord), 0, S * kRecord, kBufferWord3);
    uint32_t woff = 16 * lane, wsoff = 4096 + 4 * lane;  // (past the last record: nothing is fetched)
    i32x4 w[kSets][4];
    int sw[kSets];
    AFrag<kA8> fa[MI];
    int sa[MI];
    const uint32_t key = (r >> 1) & 7;
    const uint32_t fo = static_cast<uint32_t>(r * 128) + ((g ^ key) << 4);  // (piece 4 + g: bit 6 the other way)
    const uint32_t sco = static_cast<uint32_t>(kScales + r * 4 + g);
    auto read_a = [&](int slot, int sub, int i) {
        const uint8_t* st = lds + slot;
        fa[i].lo = *reinterpret_cast<const i32x4*>(st + (fo ^ (sub << 6)) + i * 2048);
        if constexpr (kA8) fa[i].hi = *reinterpret_cast<const i32x4*>(st + (fo ^ 64u) + i * 2048);
        sa[i] = st[sco + (sub * kScaleRows + 16 * i) * 4];
    };
    auto fence = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto barrier = [&]() {  // this wave's LDS reads are done; then all waves'
        __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        fence();
    };
    f32x4 acc[MI][4];
    // One step: its operands are in registers, the weights' in set kSet.  A weight operand is replaced by that of kSets steps on
    // behind the MI instructions that use it, a token operand by the next step's behind its last.  In a step that ends its
    // stage (t), the next stage is waited for before the first of the latter (the loads issued after its own are left in
    // flight: kBehind) and published, and the stage read out is refilled.  The last step loads too: zeros, or the columns of
    // another row, which nothing uses.
    //
    // kBehind: behind the loads of stage t + 1, which a wave issued in the step that ended stage t + 1 - kStages, stand that
    // step's last weight load, the kStages - 2 whole stages between, and stage t's weight loads but the last.  The first
    // kStages stages are issued together, before kSets records of weights: behind any of them stand more than kBehind.
    constexpr int kBehind = (kStages - 2) * (kSub * kWLoads + kLoads) + kSub * kWLoads;
    static_assert(kSets > (kStages - 2) * kSub, "the first barriers count on this");
    static_assert(kBehind < 64 && (kSets == 1 || kSets % kSub == 0), "");
    int slot = 0;
    auto step = [&](auto first_tag, auto ends_tag, auto set_tag, int t) {
        constexpr bool kFirst = decltype(first_tag)::value, kEnds = decltype(ends_tag)::value;
        constexpr int kSet = decltype(set_tag)::value % kSets;
        const f32x4 z = {};
        const int next = !kEnds ? slot : slot == (kStages - 1) * kStageBytes ? 0 : slot + kStageBytes;
        int next_sw = 0;
        auto phase = [&](auto j_tag) {
            constexpr int j = decltype(j_tag)::value;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                acc[i][j] = mfma<kA8, j>(w[kSet][j], sw[kSet], fa[i], sa[i], kFirst ? z : acc[i][j]);
                if constexpr (j == 3) {
                    if (kEnds && i == 0) {
                        fence();
                        __builtin_amdgcn_s_waitcnt(wait_vmcnt(kBehind));
                        barrier();
                    }
                    read_a(next, kEnds ? 0 : 1, i);
                    if (kEnds) {
                        if (i < kLoads) issue(t + kStages, slot, i);
                        if (i == MI - 1) {
#pragma unroll
                            for (int q = MI; q < kLoads; ++q) issue(t + kStages, slot, q);
                        }
                    }
                    fence();
                }
            }
            w[kSet][j] = load16(rw, woff + 1024 * j);
            if constexpr (j == 2) next_sw = load4(rw, wsoff);
            fence();
        };
        phase(std::integral_constant<int, 0>{});
        phase(std::integral_constant<int, 1>{});
        phase(std::integral_constant<int, 2>{});
        phase(std::integral_constant<int, 3>{});
        sw[kSet] = next_sw;
        woff += kRecord;
        wsoff += kRecord;
        slot = next;
    };
    uint8_t* const mine = lds + kParts + wave * kWaveBytes;  // the wave's part, behind the last step
    const int nw = n0 + 64 * wave;
    const int line_row = lane >> 3;  // a load or store of 16 bytes a lane has 8 rows: of these the lane's, and its piece
    const bool keys = kGate && n0 < p.n_key;
    u32x2 qw[4], kw[4];  // q and k of the lane's columns
    // the stream's rows of the wave's tokens and columns (rows past M: zeros), and the weights
    auto load_stream = [&]() {  // (the weights first: the rows are waited for one by one)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = nw + 16 * j + 4 * g;
            qw[j] = *reinterpret_cast<const u32x2*>(p.q + n);
            kw[j] = *reinterpret_cast<const u32x2*>(p.k + n);
        }
        fence();
        const int64_t x_bytes = static_cast<int64_t>(p.n_key) * 2;
        const int x_rows = static_cast<int>(min<int64_t>(BM, p.M - m0));
        const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.x + m0 * p.n_key + nw), 0, static_cast<int>(x_rows * x_bytes - 2 * nw), kBufferWord3);
        const uint32_t xo = static_cast<uint32_t>(line_row * x_bytes), xp = ((lane & 7) ^ ((line_row >> 1) & 7)) << 4;
#pragma unroll
        for (int q = 0; q < 2 * MI; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, mine + q * 1024, 16,
                                                     xo + static_cast<uint32_t>(8 * q * x_bytes) + (q & 1 ? xp ^ 64u : xp), 0, 0,
                                                     kStreamPolicy);
    };
#pragma unroll
    for (int t = 0; t < kStages; ++t)
#pragma unroll
        for (int q = 0; q < kLoads; ++q) issue(t, t * kStageBytes, q);
    fence();
#pragma unroll
    for (int e = 0; e < kSets; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[e][j] = load16(rw, woff + 1024 * j);
        sw[e] = load4(rw, wsoff);
        woff += kRecord;
        wsoff += kRecord;
        fence();
    }
    if (kEarly && keys) load_stream();
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(kSets * kWLoads + (kStages - 1) * kLoads));
    barrier();
#pragma unroll
    for (int i = 0; i < MI; ++i) read_a(0, 0, i);
    fence();
    {
        // sets and the steps of a stage in turn: step s has set s % kSets and ends its stage if s % kSub is kSub - 1
        constexpr int kTurn = kSets > kSub ? kSets : kSub;
        auto turn = [&](auto u_tag, int s) {
            constexpr int u = decltype(u_tag)::value;
            step(std::false_type{}, std::integral_constant<bool, u % kSub == kSub - 1>{}, u_tag, s / kSub);
        };
        step(std::true_type{}, std::integral_constant<bool, kSub == 1>{}, std::integral_constant<int, 0>{}, 0);
        int s = 1;
        for (; s + kTurn <= S; s += kTurn) {
            turn(std::integral_constant<int, 1>{}, s);
            if constexpr (kTurn > 1) turn(std::integral_constant<int, 2>{}, s + 1);
            if constexpr (kTurn > 2) turn(std::integral_constant<int, 3>{}, s + 2);
            if constexpr (kTurn > 3) turn(std::integral_constant<int, 4>{}, s + 3);
        }
        if constexpr (kTurn > 1) {
            if (s < S) turn(std::integral_constant<int, 1>{}, s);
        }
        if constexpr (kTurn > 2) {
            if (s + 1 < S) turn(std::integral_constant<int, 2>{}, s + 1);
            if (s + 2 < S) turn(std::integral_constant<int, 3>{}, s + 2);
        }
    }
    // Loads past the last step still write LDS: they land, and every wave has read its last operands, before the stages hold
    // anything else.  From here a wave keeps to its own part of LDS: BM rows of its 64 columns, 16-byte piece c of row t at slot
    // c ^ (t / 2) % 8, so that memory is written and read in whole lines of 128 bytes, two to 16 lanes.
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
    barrier();
    // a lane's four columns 16 j + 4 g .. +3 of token 16 i + r
    const uint32_t quad[2] = {static_cast<uint32_t>(r * 128 + (((g >> 1) ^ key) << 4) + (g & 1) * 8),
                              static_cast<uint32_t>(r * 128 + (((4 + (g >> 1)) ^ key) << 4) + (g & 1) * 8)};
    auto quad_at = [&](int i, int j) { return mine + i * 2048 + (quad[j >> 1] ^ ((j & 1) << 5)); };
    if (!keys) {
        // 16 rows at a time, so that their stores go out under the next ones' rounding (-2 %), by a resource that ends with row M
        // and an offset past it behind column N: no comparison a store (-2 %)
        const int n = nw + 8 * (lane & 7);
        const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
            p.kv + m0 * p.ld_out, 0, static_cast<int>(min<int64_t>(BM, p.M - m0) * p.ld_out * 2), kBufferWord3);
        const uint32_t row_out = static_cast<uint32_t>(p.ld_out) * 2;
        const uint32_t so = n < p.N ? line_row * row_out + static_cast<uint32_t>(n - p.n_key) * 2 : 0x80000000u;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<u32x2*>(quad_at(i, j)) =
                    u32x2{pack2_bf16(acc[i][j][0], acc[i][j][1]), pack2_bf16(acc[i][j][2], acc[i][j][3])};
            fence();
#pragma unroll
            for (int q = 2 * i; q < 2 * i + 2; ++q) {
                const int t = 8 * q + line_row;
                const u32x4 v = *reinterpret_cast<const u32x4*>(mine + t * 128 + (((lane & 7) ^ ((t >> 1) & 7)) << 4));
                __builtin_amdgcn_raw_buffer_store_b128(v, ro, so + static_cast<uint32_t>(8 * q) * row_out, 0, kNonTemporal);
            }
        }
        return;
    }
    if constexpr (kGate) {
        if (!kEarly) load_stream();
        float wq[4][4];  // q * k (exact in fp32)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                wq[j][2 * e] = lo_bf16(qw[j][e]) * lo_bf16(kw[j][e]);
                wq[j][2 * e + 1] = hi_bf16(qw[j][e]) * hi_bf16(kw[j][e]);
            }
        // The sums over the four lanes of a token by swaps of lanes between registers, of four times 16 tokens together: a register
        // then has 64 tokens' (8,192 x 1,536 x 4 x 5,120: 5 % less time with 4-bit rows, 7 % with 8-bit ones, than by shuffles).
        constexpr int kRes = MI >= 4 ? MI / 4 : MI;
        float res[kRes][3], part4[3][4];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if (!kEarly || i == 0) {  // the wave's own rows, the later ones left in flight (8,192 tokens: -3 %)
                fence();
                wait_loads(kEarly ? 0 : 2 * (MI - 1 - i));
                fence();
            }
            float hwk = 0.f, kk = 0.f, hh = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // the product is a bf16 tensor before it is used, as the other forms of the projection round it
                const uint32_t k01 = pack2_bf16(acc[i][j][0], acc[i][j][1]), k23 = pack2_bf16(acc[i][j][2], acc[i][j][3]);
                const u32x2 x = *reinterpret_cast<const u32x2*>(quad_at(i, j));
                const uint32_t x01 = x[0], x23 = x[1];
                hwk += lo_bf16(x01) * wq[j][0] * lo_bf16(k01);
                hwk += hi_bf16(x01) * wq[j][1] * hi_bf16(k01);
                hwk += lo_bf16(x23) * wq[j][2] * lo_bf16(k23);
                hwk += hi_bf16(x23) * wq[j][3] * hi_bf16(k23);
                kk = dot2_bf16(k23, k23, dot2_bf16(k01, k01, kk));
                hh = dot2_bf16(x23, x23, dot2_bf16(x01, x01, hh));
            }
            if constexpr (MI >= 4) {
                part4[0][i % 4] = hwk;
                part4[1][i % 4] = kk;
                part4[2][i % 4] = hh;
                if (i % 4 == 3) {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        res[i / 4][e] = add_rows(add_halves(part4[e][0], part4[e][2]), add_halves(part4[e][1], part4[e][3]));
                }
            } else {
                const float sum[3] = {hwk, kk, hh};
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const float halves = add_halves(sum[e], sum[e]);
                    res[i][e] = add_rows(halves, halves);
                }
            }
        }
        constexpr int kPer = MI >= 4 ? 64 : 16;  // tokens of a register
        const bool has = kPer == 64 || g == 0;
        // two waves' 64 columns make a slice of 128: the right one leaves its sums in its part of LDS
        float* sums = reinterpret_cast<float*>(lds + kParts + (wave | 1) * kWaveBytes);
        fence();
        __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
        fence();
        if ((wave & 1) && has) {
#pragma unroll
            for (int i = 0; i < kRes; ++i)
#pragma unroll
                for (int e = 0; e < 3; ++e) sums[e * BM + kPer * i + lane] = res[i][e];
        }
        __syncthreads();
        if (!(wave & 1) && has) {
            float* out = p.part + static_cast<int64_t>(n0 / 128 + (wave >> 1)) * 3 * p.M;
#pragma unroll
            for (int i = 0; i < kRes; ++i) {
                const int64_t m = m0 + kPer * i + lane;
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (m < p.M) out[e * p.M + m] = res[i][e] + sums[e * BM + kPer * i + lane];
            }
        }
    }
}

template <bool kA8, int MI, int NW, int kSets, bool kGate>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void mx4_tile_kernel(Mx4Args p, int tiles_m,
                                                                                                     int tiles_n) {
    mx4_tile_body<kA8, MI, NW, kSets, kGate>(p, tiles_m, tiles_n);
}

// ---- quantisation of bf16 rows: a thread has 8 consecutive columns, the 4 threads of a block find its largest magnitude (as
// bit patterns, whose order is the magnitudes').  floor(log2 amax) is the pattern's exponent field less the bias; E2M1's
// largest exponent is 2, so the shared scale's code is the field less 2, or 0 where that is below E8M0's range (fields 0, of
// zeros and subnormals, to 2).  v_cvt_scalef32_pk_fp4_bf16 divides by the scale, rounds to nearest even and saturates at 6 --
// checked on every bf16 pattern.  A block with an infinity or a NaN, which E2M1 has not, takes the NaN scale 0xFF and zeros.
// HBM-bound: 65,536 x 1,536 49 us (5.3 TB/s); 256 rows 2.5.
__global__ __launch_bounds__(256) void mx4_quant_kernel(const uint16_t* x, int64_t rows, int K, int64_t rows4, uint8_t* q,
                                                        uint8_t* scale) {
    const int64_t gid = group_index() * 256 + threadIdx.x;
    const int per_row = K / 8;
    const int64_t r = gid / per_row;
    const int c8 = static_cast<int>(gid - r * per_row);
    const bool ok = r < rows;
    u32x4 v = {0, 0, 0, 0};
    if (ok) v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + r * K) + c8);
    // the 4 threads of a block are lanes 4 b .. 4 b + 3 of the wave (K / 8 is a multiple of 4)
    const uint32_t field = block_top(bf16_top8(v)) >> 7;
    const uint32_t code = field == 255 ? 255u : field > 2 ? field - 2 : 0u;
    const float by = __uint_as_float(code == 0 ? 0x00400000u : code << 23);  // 2^(code - 127)
    uint32_t e = 0;
    e = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(e, as_pair(v[0]), by, 0);
    e = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(e, as_pair(v[1]), by, 1);
    e = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(e, as_pair(v[2]), by, 2);
    e = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(e, as_pair(v[3]), by, 3);
    if (!ok) return;
    *reinterpret_cast<uint32_t*>(q + r * (K / 2) + 4 * c8) = field == 255 ? 0u : e;
    if ((c8 & 3) == 0) scale[mx_scale_offset(r, c8 / 4, rows4)] = static_cast<uint8_t>(code);
}

// a workgroup per record
__global__ __launch_bounds__(256) void mx4_pack_kernel(const uint8_t* q, const uint8_t* scale, int N, int steps, int64_t rows4,
                                                       uint8_t* packed) {
    const int64_t at = group_index(), group = at / steps;
    if (group * kGroupRows >= N) return;
    const int s = static_cast<int>(at - group * steps);
    uint8_t* rec = packed + at * kRecord;
    const int t = threadIdx.x;
    {
        const int j = t >> 6, c = (t >> 4) & 3, r = t & 15;
        const int64_t n = group * kGroupRows + 16 * j + r;
        u32x4 v = {0, 0, 0, 0};
        if (n < N) v = *reinterpret_cast<const u32x4*>(q + (n * steps + s) * 64 + 16 * c);
        *reinterpret_cast<u32x4*>(rec + 16 * t) = v;
    }
    {
        const int c = t >> 6, r = (t >> 2) & 15, j = t & 3;
        const int64_t n = group * kGroupRows + 16 * j + r;
        rec[4096 + t] = n < N ? scale[(static_cast<int64_t>(s) * rows4 + n) * 4 + c] : 0;
    }
}

// The order: eight tile rows together along the columns (4 or 16: -1 to +1.5 %), which reads the rows into the L2s once and the
// weights once for every eight; or, of a plain product whose weights an XCD's L2 (4 MB) holds an eighth of, that eighth along
// the rows, which reads the weights once and the rows eight times, where that is less: 65,536 x 1,536 x 25,600 with 4-bit rows
// 1,292 us (1,331 the other way, 1.39 GB of reads instead of 0.47), 8,192 165 (171), with 8-bit rows 233 (232), 8,192 x 512 x 8,192
// 32 (37).  Where it is more, 65,536 x 1,536 x 2,560 139 (135); where an eighth is too large, 8,192 x 6,144 x 25,600 571 (550);
// fused, whose stream's rows it scatters, 8,192 201 (200).
constexpr int kGroupM = 8;
constexpr int64_t kHeld = 3 << 20;

template <bool kA8, int MI, int NW, int kSets, bool kGate>
int launch_tiles(Mx4Args p, hipStream_t stream, const char* what) {
    const int64_t tiles_m = (p.M + 16 * MI - 1) / (16 * MI);
    const int tiles_n = (p.N + 64 * NW - 1) / (64 * NW);
    const int eighth = (tiles_n + kXcds - 1) / kXcds;
    const int64_t row_bytes = p.steps * (kA8 ? 128ll : 64ll), weights = static_cast<int64_t>(tiles_n) * NW * p.steps * kRecord;
    p.across = !kGate && weights <= kXcds * kHeld && (kXcds - 1) * p.M * row_bytes < (tiles_m / kGroupM - 1) * weights;
    p.group = p.across ? eighth : kGroupM;
    hipLaunchKernelGGL((mx4_tile_kernel<kA8, MI, NW, kSets, kGate>), group_grid(tiles_m * tiles_n), dim3(64 * NW), 0,
                       stream, p, static_cast<int>(tiles_m), tiles_n);
    return check_launch(what);
}

// The tile: 128 tokens where that makes one and a half tiles or more for every CU; 64, then 32, where it makes one for half of
// them and is more than half filled; else 16, by two waves.  A small tile has more steps of weights in flight, and few tiles
// take the latency of their chain of steps; many are bound by what they read.  8-bit rows of 1,536 columns, us at 16 / 32 / 64
// / 128 tokens a tile (the weights in the Infinity Cache): 1 x 25,600 5.8 / 6.1 / 7.7 / 11.4; 64 x 25,600 8.3 / 7.0 / 8.3 / 11.8; 128 13.0 / 9.4 / 8.4 / 12.2; and
// at 16 / 64 / 128: 256 20.6 / 12.1 / 12.5; 384 28.6 / 18.3 / 19.4; 512 36 / 22.7 / 19.8; 1,024 x 2,560 10.4 / 8.1 / 12.0.
template <bool kA8, bool kGate>
int launch(const Mx4Args& p, hipStream_t stream, const char* what) {
    constexpr int kCUs = 256;
    const int64_t tiles_n = (p.N + 255) / 256;
    auto tiles = [&](int tokens) { return (p.M + tokens - 1) / tokens * tiles_n; };
    if (p.M > 64 && 2 * tiles(128) >= 3 * kCUs) return launch_tiles<kA8, 8, 4, 1, kGate>(p, stream, what);
    if (p.M > 32 && 2 * tiles(64) >= kCUs) return launch_tiles<kA8, 4, 4, 2, kGate>(p, stream, what);
    if (p.M > 16 && 2 * tiles(32) >= kCUs) return launch_tiles<kA8, 2, 4, 4, kGate>(p, stream, what);
    return launch_tiles<kA8, 1, 2, 4, kGate>(p, stream, what);
}

constexpr int kMaxK = 1 << 20, kMaxN = 1 << 22;

// what is wrong with the operands' sizes, or null
const char* bad_shape(int64_t T, int32_t a_bits, int32_t K, int32_t N) {
    if (T < 0) return "T < 0";
    if (a_bits != 4 && a_bits != 8) return "a_bits must be 4 or 8";
    if (K < kStepCols || K % kStepCols != 0 || K > kMaxK) return "K must be a multiple of 128 in [128, 2^20]";
    if (N < 8 || N % 8 != 0 || N > kMaxN) return "the columns must be a multiple of 8 in [8, 2^22]";
    if (T > 1ll << 34 || T > (1ll << 41) / N) return "too many tokens";
    return nullptr;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_mx4_quant(const uint16_t* x, int64_t rows, int32_t K, uint8_t* q, uint8_t* scale, void* stream) {
    const char* what = "engram_mx4_quant";
    if (rows < 0) return fail(ENGRAM_EINVAL, "%s: rows < 0", what);
    if (K < kStepCols || K % kStepCols != 0 || K > kMaxK)
        return fail(ENGRAM_EINVAL, "%s: K=%d must be a multiple of 128 in [128, 2^20]", what, K);
    if (rows > (1ll << 48) / K) return fail(ENGRAM_EINVAL, "%s: too many rows", what);
    if (rows == 0) return ENGRAM_OK;
    if (!x || !q || !scale) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(x, 16) || !aligned(q, 4)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const int64_t blocks = (rows * (K / 8) + 255) / 256;
    hipLaunchKernelGGL(mx4_quant_kernel, group_grid(blocks), dim3(256), 0, as_stream(stream), x, rows, K,
                       (rows + 3) / 4 * 4, q, scale);
    return check_launch(what);
}

extern "C" int64_t engram_mx4_weight_bytes(int32_t Nout, int32_t K) {
    if (bad_shape(0, 4, K, Nout)) return -1;
    return static_cast<int64_t>((Nout + kGroupRows - 1) / kGroupRows) * (K / kStepCols) * kRecord;
}

extern "C" int engram_mx4_pack_weight(const uint8_t* q, const uint8_t* scale, int32_t Nout, int32_t K, uint8_t* packed,
                                      void* stream) {
    const char* what = "engram_mx4_pack_weight";
    if (const char* bad = bad_shape(0, 4, K, Nout)) return fail(ENGRAM_EINVAL, "%s: %s", what, bad);
    if (!q || !scale || !packed) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(q, 16) || !aligned(packed, 16)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const int64_t records = engram_mx4_weight_bytes(Nout, K) / kRecord;
    hipLaunchKernelGGL(mx4_pack_kernel, group_grid(records), dim3(256), 0, as_stream(stream), q, scale, Nout,
                       K / kStepCols, (static_cast<int64_t>(Nout) + 3) / 4 * 4, packed);
    return check_launch(what);
}

extern "C" int engram_wkv_mx4(const uint8_t* a, const uint8_t* a_scale, int32_t a_bits, const uint8_t* w, uint16_t* kv,
                              int64_t T, int32_t K, int32_t Nout, void* stream) {
    const char* what = "engram_wkv_mx4";
    if (const char* bad = bad_shape(T, a_bits, K, Nout)) return fail(ENGRAM_EINVAL, "%s: %s", what, bad);
    if (T == 0) return ENGRAM_OK;
    if (!a || !a_scale || !w || !kv) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(a, 16) || !aligned(a_scale, 16) || !aligned(w, 16) || !aligned(kv, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    Mx4Args p = {};
    p.a = a;
    p.as = a_scale;
    p.w = w;
    p.kv = kv;
    p.M = T;
    p.M4 = (T + 3) / 4 * 4;
    p.ld_out = Nout;
    p.N = Nout;
    p.steps = K / kStepCols;
    return a_bits == 8 ? launch<true, false>(p, as_stream(stream), what) : launch<false, false>(p, as_stream(stream), what);
}

extern "C" int engram_wkv_mx4_gate(const uint8_t* a, const uint8_t* a_scale, int32_t a_bits, const uint8_t* w,
                                   const uint16_t* x, const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                   uint16_t* value, int64_t ld_value, float* dot, void* workspace, int64_t workspace_bytes,
                                   int64_t T, int32_t K, int32_t hc, int32_t dim, void* stream) {
    const char* what = "engram_wkv_mx4_gate";
    if (hc < 1 || hc > 64) return fail(ENGRAM_EINVAL, "%s: hc=%d outside [1, 64]", what, hc);
    if (dim < 256 || dim % 256 != 0)
        return fail(ENGRAM_EINVAL, "%s: dim=%d must be a positive multiple of 256", what, dim);
    if (static_cast<int64_t>(hc + 1) * dim > kMaxN)
        return fail(ENGRAM_EINVAL, "%s: (hc + 1) * dim = %lld exceeds 2^22", what, static_cast<long long>(hc + 1) * dim);
    const int N = (hc + 1) * dim;
    if (const char* bad = bad_shape(T, a_bits, K, N)) return fail(ENGRAM_EINVAL, "%s: %s", what, bad);
    if (T > (1ll << 31) / hc) return fail(ENGRAM_EINVAL, "%s: too many tokens", what);
    if (ld_value < dim || ld_value % 8 != 0 || ld_value > kMaxN)
        return fail(ENGRAM_EINVAL, "%s: ld_value=%lld must be a multiple of 8 in [dim, 2^22]", what, (long long)ld_value);
    const int64_t need = engram_wkv_gate_workspace_bytes(T, hc, dim);
    if (workspace_bytes < need)
        return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, %lld needed", what, (long long)workspace_bytes,
                    (long long)need);
    if (T == 0) return ENGRAM_OK;
    if (!a || !a_scale || !w || !x || !q_weight || !k_weight || !value || !dot || !workspace)
        return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(a, 16) || !aligned(a_scale, 16) || !aligned(w, 16) || !aligned(x, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(value, 16) || !aligned(dot, 4) || !aligned(workspace, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    Mx4Args p = {};
    p.a = a;
    p.as = a_scale;
    p.w = w;
    p.kv = value;
    p.M = T;
    p.M4 = (T + 3) / 4 * 4;
    p.ld_out = ld_value;
    p.N = N;
    p.steps = K / kStepCols;
    p.x = x;
    p.q = q_weight;
    p.k = k_weight;
    p.part = static_cast<float*>(workspace);
    p.n_key = hc * dim;
    const int rc = a_bits == 8 ? launch<true, true>(p, as_stream(stream), what) : launch<false, true>(p, as_stream(stream), what);
    if (rc != ENGRAM_OK) return rc;
    float* dots[1] = {dot};
    return launch_gate_finalize(static_cast<const float*>(workspace), 0, dots, 1, T, hc, dim, eps, as_stream(stream), what);
}
