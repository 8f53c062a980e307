// engram_wkv_backward: the gradient of the projection kv = a W^T (engram_wkv).
//
//   da [T, K]    = dkv [T, Nout] W [Nout, K]        (over Nout)
//   dW [Nout, K] = dkv^T [Nout, T] a [T, K]         (over T)
//
// Both are products on v_mfma_f32_16x16x32_bf16 with fp32 accumulation.  Neither has both operands contiguous along
// the reduced axis, which is what the instruction's lanes take: W of da and both operands of dW have it as their rows.
// Such an operand's slab (64 rows of the reduced axis) goes into LDS as it lies in memory and is turned on the way to the
// registers by ds_read_b64_tr_b16 (within 16 lanes, lane i supplies the address of four elements, row i / 4, columns
// 4 (i % 4) .. + 3, and receives column i of the four rows: lane layout measured on gfx950), so nothing is transposed in
// memory.  Its rows are swizzled by 32-byte blocks, so that the rows that one read touches lie in different blocks.
//
// A workgroup makes a 256 x 256 tile of the output (eight waves, 128 x 64 each) or, where the work is little, 128 x 128
// (four waves, 64 x 64 each, two workgroups a CU), from slabs of 64 of the reduced axis in two stages of LDS filled by
// direct-to-LDS loads.  Where the tiles are fewer than the CUs the reduced axis is split over workgroups, whose fp32
// partial tiles a second launch adds in order.  da and dW of a call are one launch, the shorter reductions behind the
// longer ones.
//
// Bound by the matrix cores where T is long: 8,192 x 1,536 x 25,600, both products, 1,053 us, 1.22 PFLOP/s (a large square
// library product reaches 1.45-1.55 here; da alone 606 us, dW 584).  Below some 1,000 tokens by memory: W read and dW
// written, 250 MB at 251 tokens in 85 us (64 where two sets of inputs in turn leave some of W in the Infinity Cache; da alone 47, dW 43: da
// waits on its slabs, one of which is in flight per workgroup).
#include <type_traits>

#include "rows.h"

namespace engram {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int BK = 64;  // the reduced axis per slab
constexpr int kXcds = 8;
constexpr int kCUs = 256;
constexpr int kBufferWord3 = 0x00020000;
constexpr int kWaitVm0 = 0x0F70;
constexpr int kWaitLgkm0 = 0xC07F;
constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset past every resource: the load gives zeros

// One product out [M, N] = sum over r < R of P[m, r] Q[r, n].
struct Prod {
    const uint16_t* p;  // da: dkv [M, R]; dW: dkv [R, M]
    const uint16_t* q;  // [R, N]
    int64_t M, N, R;
    void* out;          // [M, N]
    float* part;        // [splits][M, N] when splits > 1
    int out_f32, accumulate;
    int tiles_m, tiles_n, splits, slabs;
    __host__ __device__ int64_t units() const { return static_cast<int64_t>(tiles_m) * tiles_n * splits; }
};
struct GradArgs {
    Prod da, dw;
    int first_dw;           // dW's workgroups come first
    int64_t first_units;    // workgroups of the product that comes first
};

__device__ inline uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// The transposing LDS read.  Its argument is `restrict`, and so is the read marked apart from other memory: without that
// the compiler takes it for a possible reader of every direct-to-LDS load before it and waits for all of them (ordinary LDS
// reads it does not).  What orders the reads after the loads they need is the slab's own wait and barrier.
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
__device__ __forceinline__ s16x4 read_transposed(lds_s16x4 __restrict__ p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// pid of n tiles onto an order in which each XCD (workgroups pid % 8) takes a contiguous run
__device__ inline int64_t xcd_order(int64_t pid, int64_t n) {
    const int64_t xcd = pid % kXcds, per = n / kXcds, rem = n % kXcds;
    return xcd * per + min(xcd, rem) + pid / kXcds;
}

// TS: the tile's rows and columns (256: eight waves of 128 x 64; 128: four of 64 x 64).  kRowsP: P's slab holds rows of
// the reduced axis (dW), else rows of the output (da).
template <int TS, bool kRowsP>
__device__ __forceinline__ void product(const Prod& g, int64_t unit, uint8_t* lds) {
    constexpr int kOpBytes = TS * BK * 2;          // one operand's slab
    constexpr int kStageBytes = 2 * kOpBytes;      // an operand's two stages
    constexpr int PB = TS / 32;                    // blocks of 16 rows per wave (and 4 of 16 columns)
    constexpr int kRow = TS * 2;                   // bytes of a reduced row in LDS
    constexpr int kPieces = TS / 8;                // its 16-byte pieces
    constexpr int kPerLoad = 1024 / kRow;          // reduced rows per load instruction
    constexpr int kParts = 16 / kPerLoad;          // parts of a slab's loads, each one instruction per operand
    constexpr int kBar = 2 * (PB - 1);             // the slab barrier precedes unit kBar of a slab's second k-step
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int tiles = g.tiles_m * g.tiles_n;
    // an XCD takes whole parts of a split reduction, whose tiles read the same rows of P and Q (2,048 x 1,536 x 25,600 313
    // -> 298 us against each part's tiles over all XCDs)
    const int64_t at_unit = xcd_order(unit, g.units());
    const int split = static_cast<int>(at_unit / tiles);
    const int tile = static_cast<int>(at_unit - static_cast<int64_t>(split) * tiles);
    const int tm = tile / g.tiles_n, tn = tile - tm * g.tiles_n;
    const int64_t m0 = static_cast<int64_t>(tm) * TS, n0 = static_cast<int64_t>(tn) * TS;
    const int s0 = static_cast<int>(static_cast<int64_t>(g.slabs) * split / g.splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(g.slabs) * (split + 1) / g.splits);

    auto sync = [&]() {
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // ---- slab loads, by waves 0-3: a quarter of each operand per wave, 1 KB per instruction.  A slab of reduced rows:
    // kPerLoad rows per instruction, each lane the piece that belongs at its place under the swizzle (block b of row k at
    // b XOR (k % 4 + 4 ((k / 8) % (TS / 64))): the rows that half a wave's read touches lie in different blocks); a slab of
    // output rows: eight rows of 128 bytes, lane l at slot l % 8 of row 8 q + l / 8, 16-byte pieces swizzled by row / 2.
    // Rows past the reduced axis or past M lie outside the resource and read as zero (the row term sits in the
    // range-checked offset); columns past M or N read a neighbour's elements, which only reach outputs that are not stored.
    const uint32_t l_row = lane / kPieces;
    const uint32_t t_row = (wave & 3) * 16 + l_row;
    const uint32_t t_piece = (lane % kPieces) ^ (2 * l_row) ^ (TS == 256 ? 16 * (wave & 1) : 0);
    const uint32_t ldp = static_cast<uint32_t>((kRowsP ? g.M : g.R) * 2), ldq = static_cast<uint32_t>(g.N * 2);
    const uint32_t p_row = kRowsP ? t_row * ldp : ((wave & 3) * (TS / 4) + (lane >> 3)) * ldp;
    const uint32_t p_piece = (lane & 7) ^ (lane >> 4);
    const uint32_t q_row = t_row * ldq;
    struct Slab {
        __amdgpu_buffer_rsrc_t p, q;
        int64_t r0;  // first reduced index
        int left;    // how many the slab has
    };
    auto slab_of = [&](int s) {  // s past the unit's last: empty resources
        Slab b;
        b.r0 = static_cast<int64_t>(s) * BK;
        const int64_t rows = s < s1 ? min<int64_t>(BK, g.R - b.r0) : 0;
        const int64_t at = rows > 0 ? b.r0 : 0;
        b.left = static_cast<int>(rows);
        b.q = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.q + at * g.N + n0), 0,
                                                rows > 0 ? static_cast<int>(rows * g.N * 2 - n0 * 2) : 0, kBufferWord3);
        if constexpr (kRowsP) {
            b.p = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.p + at * g.M + m0), 0,
                                                    rows > 0 ? static_cast<int>(rows * g.M * 2 - m0 * 2) : 0, kBufferWord3);
        } else {
            const int64_t outs = min<int64_t>(TS, g.M - m0);
            b.p = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.p + m0 * g.R), 0,
                                                    rows > 0 ? static_cast<int>(outs * g.R * 2) : 0, kBufferWord3);
        }
        return b;
    };
    // part q of a slab into stage st; the offsets are formed here from four held values (opaque, so that they are
    // not hoisted out of the slab loop as 16 registers)
    auto issue_part = [&](const Slab& b, int st, int q) {
        uint32_t tp = t_piece, pr = p_row, qr = q_row;
        asm volatile("" : "+v"(tp), "+v"(pr), "+v"(qr));
        const uint32_t piece = (TS == 256 ? tp ^ (4 * (q & 1)) ^ (8 * (q >> 2)) : tp ^ (8 * (q >> 1))) << 4;
        uint8_t* to = lds + st * kOpBytes + ((wave & 3) * 16 + kPerLoad * q) * kRow;
        if constexpr (kRowsP) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(b.p, to, 16, pr + kPerLoad * q * ldp + piece, 0, 0, 0);
        } else {
            uint32_t pp = p_piece;
            asm volatile("" : "+v"(pp));
            const uint32_t pc = pp ^ (4 * (q & 1));
            const uint32_t voff = static_cast<int>(pc) * 8 < b.left ? pr + 8 * q * ldp + (pc << 4) : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(b.p, lds + st * kOpBytes + ((wave & 3) * (TS / 4) + 8 * q) * 128, 16,
                                                     voff,
                                                     static_cast<int>(b.r0 * 2), 0, 0);
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b.q, to + kStageBytes, 16, qr + kPerLoad * q * ldq + piece, 0, 0, 0);
    };

    // ---- fragments of k-step s (32 of the slab's 64): lane l holds row or column l % 16, reduced 8 (l / 16) .. + 7.
    // LDS: P's two stages, then Q's; k-step and half lie in the instruction's offset, the stage in the address.
    const uint32_t t_lane =
        (8 * (lane >> 4) + ((lane >> 2) & 3)) * kRow + (lane & 3) * 8 + (((lane >> 2) & (TS / 16 - 1)) << 5);
    const uint32_t r_lane = (wm * (TS / 2) + (lane & 15)) * 128 + (((lane >> 4) ^ ((lane >> 1) & 7)) << 4);
    uint32_t p_at[kRowsP ? PB : 2], q_at[4];
    if constexpr (kRowsP) {
#pragma unroll
        for (int i = 0; i < PB; ++i) p_at[i] = t_lane ^ ((wm * PB + i) << 5);
    } else {
        p_at[0] = r_lane;
        p_at[1] = r_lane ^ 64;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) q_at[j] = kStageBytes + (t_lane ^ ((wn * 4 + j) << 5));
    // opaque: one register each, the rest of an address in the instruction's 16-bit offset
#pragma unroll
    for (uint32_t& a : p_at) asm volatile("" : "+v"(a));
#pragma unroll
    for (uint32_t& a : q_at) asm volatile("" : "+v"(a));
    auto read_t = [&](uint32_t at) {
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x4 lo = read_transposed((lds_s16x4)(lds + at));
        const s16x4 hi = read_transposed((lds_s16x4)(lds + at + 4 * kRow));
        const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, v);
    };
    auto read_p = [&](int s, int i) -> bf16x8 {
        if constexpr (kRowsP) return read_t(p_at[i] + s * 32 * kRow);
        else return *reinterpret_cast<const bf16x8*>(lds + p_at[s] + i * 16 * 128);
    };
    auto read_q = [&](int s, int j) { return read_t(q_at[j] + s * 32 * kRow); };
    auto other_stage = [&]() {
#pragma unroll
        for (uint32_t& a : p_at) {
            a ^= kOpBytes;
            asm volatile("" : "+v"(a));
        }
#pragma unroll
        for (uint32_t& a : q_at) {
            a ^= kOpBytes;
            asm volatile("" : "+v"(a));
        }
    };

    f32x4 acc[PB][4] = {};
    bf16x8 fp[PB], fq[4];
    // One k-step: two halves, Q's fragments 0-1 then 2-3, each walking P's; a fragment is read again, for k-step
    // ns, right after its last use, at least 2 PB - 1 MFMAs before its next.  Each MFMA with its reads and
    // `extra(u)` (u = 0 .. 4 PB - 1) is one scheduling unit.
    auto kstep = [&](int ns, auto&& extra) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
            for (int i = 0; i < PB; ++i) {
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    const int j = 2 * jj + jb;
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[j], fp[i], acc[i][j], 0, 0, 0);
                    if (j == 3) fp[i] = read_p(ns, i);
                    if (i == PB - 1) fq[j] = read_q(ns, j);
                    extra(2 * PB * jj + 2 * i + jb);
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    auto run = [&](auto loader_tag) {
        constexpr bool kLoader = decltype(loader_tag)::value;
        if (kLoader) {
            const Slab a = slab_of(s0), b = slab_of(s0 + 1);
#pragma unroll
            for (int q = 0; q < kParts; ++q) issue_part(a, 0, q);
#pragma unroll
            for (int q = 0; q < kParts; ++q) issue_part(b, 1, q);
            __builtin_amdgcn_s_waitcnt(kWaitVm0);
        }
        sync();
#pragma unroll
        for (int i = 0; i < PB; ++i) fp[i] = read_p(0, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) fq[j] = read_q(0, j);
        // A slab: k-step 0, then k-step 1 with the slab barrier before its first LDS read (unit kBar): past it the next
        // slab has landed and nobody reads this stage any more, so the slab after the next goes into it.
        int st = 0;
        for (int kt = s0; kt < s1; ++kt) {
            kstep(1, [](int) {});
            other_stage();
            Slab b;
            if (kLoader) b = slab_of(kt + 2);
            kstep(0, [&](int u) {
                if (u == kBar - 1) {
                    if (kLoader) __builtin_amdgcn_s_waitcnt(kWaitVm0);
                    sync();
                }
                if (kLoader && u >= kBar && (u - kBar) % 2 == 0 && (u - kBar) / 2 < kParts) issue_part(b, st, (u - kBar) / 2);
            });
            st ^= 1;
        }
        if (kLoader) __builtin_amdgcn_s_waitcnt(kWaitVm0);  // empty loads still write LDS
    };
    if (TS == 128 || wave < 4) run(std::true_type{});
    else run(std::false_type{});

    // ---- lane l holds, per block of 16 rows, row l % 16 and the columns 16 j + 4 (l / 16) .. + 3.  Through 4 KB of LDS per
    // wave (16-byte pieces swizzled by the row), so that 16 lanes store a row's 64 columns; stores of finished tiles past
    // the caches.  dW alone, 251 x 1,536 x 25,600: 66 us from the registers, 59 through LDS, 46 past the caches.
    sync();
    uint8_t* mine = lds + wave * 4096;
    const int64_t n = n0 + wn * 64 + 4 * (lane & 15);
#pragma unroll
    for (int i = 0; i < PB; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4*>(mine + (lane & 15) * 256 + (((4 * j + (lane >> 4)) ^ (lane & 15)) << 4)) = acc[i][j];
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
        f32x4 rows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 4 * k + (lane >> 4);
            rows[k] = *reinterpret_cast<const f32x4*>(mine + row * 256 + (((lane & 15) ^ row) << 4));
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t m = m0 + wm * (TS / 2) + 16 * i + 4 * k + (lane >> 4);
            if (m >= g.M || n >= g.N) continue;
            const int64_t at = m * g.N + n;
            f32x4 v = rows[k];
            if (g.splits > 1) {
                *reinterpret_cast<f32x4*>(g.part + split * g.M * g.N + at) = v;
            } else if (g.out_f32) {
                f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
                if (g.accumulate) v += *o;
                __builtin_nontemporal_store(v, o);
            } else {
                u32x2* o = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at);
                if (g.accumulate) {
                    const u32x2 w = *o;
                    v += f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                               __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
                }
                __builtin_nontemporal_store(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, o);
            }
        }
    }
}

template <int TS>
__device__ __forceinline__ void either(const GradArgs& a, uint8_t* lds) {
    const int64_t b = blockIdx.x;
    const bool first = b < a.first_units;
    const int64_t unit = first ? b : b - a.first_units;
    if (first == (a.first_dw != 0)) product<TS, true>(a.dw, unit, lds);
    else product<TS, false>(a.da, unit, lds);
}

__global__ __launch_bounds__(512, 1) void wkv_grad_kernel(GradArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * 256 * BK * 2];
    either<256>(a, lds);
}

// two workgroups a CU: one's stores run under the other's loads
__global__ __launch_bounds__(256, 2) void wkv_grad_small_kernel(GradArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * 128 * BK * 2];
    either<128>(a, lds);
}

// The partial tiles of a split reduction, added in order: eight outputs per thread.
__global__ __launch_bounds__(256) void wkv_grad_join_kernel(const float* part, int splits, int64_t n8, void* out,
                                                            int out_f32, int accumulate) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n8) return;
    float s[8] = {};
    constexpr int kBatch = 8;
    for (int k = 0; k < splits; k += kBatch) {
        Piece<F32> p[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) p[b].load(part, min(k + b, splits - 1) * n8 + i);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (k + b >= splits) break;
            float f[8];
            p[b].to(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
        }
    }
    if (out_f32) {
        Piece<F32> o;
        if (accumulate) {
            float f[8];
            o.load(out, i);
            o.to(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
        }
        o.from(s);
        o.store(out, i);
    } else {
        Piece<Bf16> o;
        if (accumulate) {
            float f[8];
            o.load(out, i);
            o.to(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e];
        }
        o.from(s);
        o.store(out, i);
    }
}

int64_t room_of(int size) { return size == 128 ? 2 * kCUs : kCUs; }  // workgroups that run at once

Prod prod_of(int64_t M, int64_t N, int64_t R, int size) {
    Prod p = {};
    p.M = M;
    p.N = N;
    p.R = R;
    p.tiles_m = static_cast<int>((M + size - 1) / size);
    p.tiles_n = static_cast<int>((N + size - 1) / size);
    p.slabs = static_cast<int>((R + BK - 1) / BK);
    p.splits = 1;
    return p;
}

int64_t tiles_of(const Prod& p) { return static_cast<int64_t>(p.tiles_m) * p.tiles_n; }

int at_most(int64_t splits, const Prod& p) {  // four slabs a part, or one part
    const int64_t most = p.slabs / 4 > 1 ? p.slabs / 4 : 1;
    return static_cast<int>(splits < 1 ? 1 : splits < most ? splits : most);
}

// When n1 units of l1 slabs, then n2 of l2 <= l1, each taken by the workgroup slot that is free first, are done.
int64_t done_at(int64_t n1, int64_t l1, int64_t n2, int64_t l2, int64_t room) {
    const int64_t late = n1 % room, early = room - late;  // slots that the first kind leaves at hi and at lo
    const int64_t lo = n1 / room * l1, hi = lo + l1;
    if (n2 == 0) return late ? hi : lo;
    const int64_t mean = (n1 * l1 + n2 * l2 + room - 1) / room;
    int64_t m = late ? hi : lo + l2;
    if (m < mean) m = mean;
    while (true) {
        const int64_t a = (m - lo) / l2, b = late ? (m - hi) / l2 : 0;
        if (early * a + late * b >= n2) return m;
        const int64_t next_a = lo + (a + 1) * l2, next_b = hi + (b + 1) * l2;
        m = late && next_b < next_a ? next_b : next_a;
    }
}

// us that a launch takes with the products' present parts: a slab at 1.5 PFLOP/s over all slots (1.3 times that time in
// the small tiles: long products of them measured 1.31 times the large ones'), kUnitSlabs more for each unit (its first
// loads and its stores), and the second launch over the partial sums.
constexpr int64_t kUnitSlabs = 2;
double cost_of(const Prod& a, const Prod& b, int size) {
    const int64_t room = room_of(size);
    auto length = [](const Prod& p) { return (p.slabs + p.splits - 1) / p.splits + kUnitSlabs; };
    const int64_t na = a.out ? a.units() : 0, nb = b.out ? b.units() : 0, la = length(a), lb = length(b);
    double us = 2.0 * size * size * BK * static_cast<double>(room) / (size == 128 ? 1.5e9 / 1.3 : 1.5e9) *
                static_cast<double>(la >= lb ? done_at(na, la, nb, lb, room) : done_at(nb, lb, na, la, room));
    for (const Prod* p : {&a, &b})
        if (p->out && p->splits > 1) us += 4.0 + 8.0 * p->splits * p->M * p->N / 5e6;
    return us;
}

// How the reduced axes are split in a call of both products: the cheapest of parts of one length for both, the lengths being the whole of either product's reduction, its half, its third ..., in wider steps from its eighth on.
// Against parts of just a slot's share of the work, which leave a few units to a round of their own: 2,000 x 1,536 x 5,120
// 92 -> 70 us, 4,000 156 -> 118, 2,000 x 344 x 9,624 69 -> 44, 2,377 x 584 x 5,416 80 -> 60; 8,192 x 1,536 x 25,600 as it was.
double split(Prod& a, Prod& b, int size) {
    constexpr int kMost = 64;
    Prod best_a = a, best_b = b;
    double best = -1;
    const int64_t least = (tiles_of(a) * a.slabs + tiles_of(b) * b.slabs) / room_of(size);
    for (const Prod* p : {&a, &b}) {
        for (int k = 1; k <= kMost && 4 * k <= p->slabs + 3; k += k < 8 ? 1 : k / 4) {
            const int64_t length = (p->slabs + k - 1) / k;
            a.splits = at_most((a.slabs + length - 1) / length, a);
            b.splits = at_most((b.slabs + length - 1) / length, b);
            const double us = cost_of(a, b, size);
            if (best < 0 || us < best) {
                best = us;
                best_a.splits = a.splits;
                best_b.splits = b.splits;
            }
            if (2 * length < least) break;  // shorter parts only add to the sums
        }
    }
    a.splits = best_a.splits;
    b.splits = best_b.splits;
    return best;
}

// The products as a call runs them, `da` and `dw` saying which are asked for.
//
// Both: 128 x 128 tiles for little work, two workgroups a CU, and for sizes that the large tiles leave much of idle: what
// costs less.  us with 128 and 256: 64 x 1,536 x 25,600 63 and 69, 251 91 and 86, 512 137 and 109; 251 x 1,536 x 5,120 27 and
// 27, 1,000 48 and 42, 4,000 143 and 120; 8,000 x 456 x 2,000 46 and 52; 5,984 x 344 x 9,624 130 and 159; 5,687 x 584 x 5,416
// 114 and 132; 3,681 x 1,024 x 18,072 373 and 306.
//
// One alone: its sum is split as a call of both splits it, so that its bits do not depend on whether the other is asked
// for.  A split of its own is faster where the two products balance each other (da of 2,048 x 1,536 x 25,600 152 us and 219
// as here, 1,024 89 and 102, 5,984 x 344 x 9,624 82 and 116; dW of the last 76 and 105) and as fast elsewhere.  The tiles are
// its own, for the bits do not depend on them: small ones for little work (dW of 251 x 1,536 x 25,600 45 us with 128, 50 with
// 256; 400 55 and 60), else by the cost, the large ones where it is near (3,681 x 1,024 x 18,072 206 and 188).
struct Choice {
    Prod da, dw;
    int size;
};
Choice choose(int64_t T, int32_t K, int32_t Nout, bool da, bool dw) {
    int asked;  // (no output is written here)
    Choice c[2];
    double us[2];
    for (int i = 0; i < 2; ++i) {
        const int size = i ? 256 : 128;
        c[i] = Choice{prod_of(T, K, Nout, size), prod_of(Nout, K, T, size), size};
        c[i].da.out = c[i].dw.out = &asked;
        us[i] = split(c[i].da, c[i].dw, size);
    }
    int best = us[0] < us[1] ? 0 : 1;
    if (!da || !dw) {
        const int splits_da = c[best].da.splits, splits_dw = c[best].dw.splits;
        for (int i = 0; i < 2; ++i) {
            c[i].da.splits = splits_da;
            c[i].dw.splits = splits_dw;
            if (!da) c[i].da.out = nullptr;
            if (!dw) c[i].dw.out = nullptr;
            us[i] = cost_of(c[i].da, c[i].dw, c[i].size);
        }
        best = 2.0 * T * K * Nout < 3.2e10 || 1.05 * us[0] < us[1] ? 0 : 1;
    }
    Choice got = c[best];
    got.da.out = got.dw.out = nullptr;
    if (!da) got.da = Prod{};
    if (!dw) got.dw = Prod{};
    return got;
}

int64_t part_bytes(const Prod& p) { return p.splits > 1 ? p.splits * p.M * p.N * 4 : 0; }

bool shape_ok(int64_t T, int32_t K, int32_t Nout) {
    return T >= 0 && T <= (1ll << 30) && K >= 8 && K % 8 == 0 && K <= (1 << 20) && Nout >= 8 && Nout % 8 == 0 &&
           Nout <= (1 << 21);
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int64_t engram_wkv_backward_workspace_bytes(int64_t T, int32_t K, int32_t Nout) {
    if (!shape_ok(T, K, Nout)) return -1;
    if (T == 0) return 0;
    const Choice c = choose(T, K, Nout, true, true);
    return part_bytes(c.da) + part_bytes(c.dw);  // (either alone needs its own of the two)
}

extern "C" int engram_wkv_backward(const uint16_t* dkv, const uint16_t* a, const uint16_t* w, uint16_t* da, void* dw,
                                   int32_t dw_dtype, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                   int64_t T, int32_t K, int32_t Nout, void* stream) {
    const char* what = "engram_wkv_backward";
    if (T < 0 || T > (1ll << 30)) return fail(ENGRAM_EINVAL, "%s: T outside [0, 2^30]", what);
    if (K < 8 || K % 8 != 0 || K > (1 << 20))
        return fail(ENGRAM_EINVAL, "%s: K=%d must be a multiple of 8 in [8, 2^20]", what, K);
    if (Nout < 8 || Nout % 8 != 0 || Nout > (1 << 21))
        return fail(ENGRAM_EINVAL, "%s: Nout=%d must be a multiple of 8 in [8, 2^21]", what, Nout);
    if (!known_dtype(dw_dtype)) return fail(ENGRAM_EINVAL, "%s: unknown dtype", what);
    if (!da && !dw) return fail(ENGRAM_EINVAL, "%s: neither da nor dw is asked for", what);
    if (T > 0) {
        if (!dkv || (dw && !a) || (da && !w)) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
        if (!aligned(dkv, 16) || (dw && !aligned(a, 16)) || (da && !aligned(w, 16)) || !aligned(da, 16))
            return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    }
    if (!aligned(dw, 16)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    hipStream_t s = as_stream(stream);
    if (T == 0) {
        if (!dw || accumulate) return ENGRAM_OK;
        return launch_zero(dw, static_cast<int64_t>(Nout) * K * (dw_dtype == ENGRAM_F32 ? 4 : 2), s, what);
    }
    const Choice c = choose(T, K, Nout, da != nullptr, dw != nullptr);
    GradArgs g = {};
    g.da = c.da;
    g.da.p = dkv;
    g.da.q = w;
    g.da.out = da;
    g.dw = c.dw;
    g.dw.p = dkv;
    g.dw.q = a;
    g.dw.out = dw;
    g.dw.out_f32 = dw_dtype == ENGRAM_F32;
    g.dw.accumulate = accumulate != 0;
    const int size = c.size;
    const int64_t need = part_bytes(g.da) + part_bytes(g.dw);
    g.da.part = static_cast<float*>(workspace);
    g.dw.part = g.da.part + part_bytes(g.da) / 4;
    if (need > 0) {
        if (!workspace || !aligned(workspace, 16)) return fail(ENGRAM_EINVAL, "%s: workspace is null or misaligned", what);
        if (workspace_bytes < need)
            return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                        (long long)need);
    }
    const int64_t u_da = da ? g.da.units() : 0, u_dw = dw ? g.dw.units() : 0;
    const int threads = size == 128 ? 256 : 512;
    // (2^23 tiles and more: outputs of 1 TB, or of narrow rows of which the tiles hold little)
    if ((u_da + u_dw) * threads >= 1ll << 32) return fail(ENGRAM_EINVAL, "%s: too many tiles", what);
    // the longer reductions first: the shorter ones fill in behind them
    g.first_dw = !da || (dw && g.dw.slabs / g.dw.splits > g.da.slabs / g.da.splits);
    g.first_units = g.first_dw ? u_dw : u_da;
    const dim3 grid(static_cast<unsigned>(u_da + u_dw));
    if (size == 128) hipLaunchKernelGGL(wkv_grad_small_kernel, grid, dim3(threads), 0, s, g);
    else hipLaunchKernelGGL(wkv_grad_kernel, grid, dim3(threads), 0, s, g);
    for (const Prod* p : {&g.da, &g.dw}) {
        if (!p->out || p->splits <= 1) continue;
        const int64_t n8 = p->M * p->N / 8;
        hipLaunchKernelGGL(wkv_grad_join_kernel, dim3(static_cast<unsigned>((n8 + 255) / 256)), dim3(256), 0, s, p->part,
                           p->splits, n8, p->out, p->out_f32, p->accumulate);
    }
    return check_launch(what);
}
