// engram_gate_output_backward: the gradient of engram_gate_output (the gate pre-activation, the sigmoid gate and the
// residual) with respect to the stream, the keys, the value and the two gate weights.
// engram_gate_output_backward_ckpt: the same from the checkpoints of the stream, the keys and the value in 8 bits
// (checkpoint.hip): the values they stand for, which bf16 holds exactly, in the same arithmetic.
//
// With h = x[t,c], key = kv[t,c], v the token's value row, w = q * k, d = the pre-activation the forward gave,
// rh = rsqrt(mean h^2 + eps), rk = rsqrt(mean key^2 + eps), s = rh rk dim^-1/2 and up the gradient of the output:
//   z = sqrt(max(|d|, 1e-6)) with d's sign,  g = sigmoid(z)  (0 for a masked token)
//   dd   = (sum_j up v) g (1 - g) / (2 |z|)      (0 where |d| < 1e-6: the clamp is flat; 0 for a masked token)
//   dx   = up + dd (s w key - d rh^2 h / dim)
//   dkey = dd (s w h - d rk^2 key / dim)
//   dv   = sum_c g up
//   dq   = k sum_t dd s h key,  dk = q sum_t dd s h key
// The second term of dx and dkey is the derivative of the two norms: sum(h w key) s = d.
//
// HBM-bound: per token (3 hc + 1) rows of dim are read and 2 hc + 1 written, every one once.  A workgroup holds a
// whole token, one 16-byte piece of every row per thread: the rows stay in registers between the sums that need all
// of a row and the outputs that need the sums, and the sum over tokens of dq and dk stays in registers (in LDS for four
// copies of more than 5,120 columns) over all of the workgroup's tokens.  The next token's rows are asked for as this one's
// are used up, so loads are in flight over the barrier (one per token: the sums of the waves, in two LDS buffers taken in
// turn).  A second launch adds the workgroups' sums in their order, so the same call gives the same bits.
//
// 8,192 tokens, both launches: 4 copies of 5,120 335 us (5.5 TB/s of the bytes above), of 2,048 146 (5.0), of 1,024 84
// (4.4), of 256 41 (2.2, bound by the tokens' chains of barrier and sums), of 8,192 633 (4.7); 2 of 5,120 193 (5.2), 1 of
// 5,120 125 (4.7); 3 of 2,048 184 (3.1, the kernel for any count of copies, which takes a barrier a copy).  From checkpoints:
// 4 copies of 5,120 318 us (4.7 TB/s: fewer bytes for the same arithmetic), of 2,048 127, of 1,024 75, of 256 44, of 8,192 484;
// 2 of 5,120 188, 1 of 5,120 128; 3 of 2,048 164.
#include <type_traits>

#include "gate.h"
#include "mx.h"
#include "rows.h"

namespace engram {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxDim = 8192;
constexpr int kCUs = 256;

struct GateGradArgs {
    const uint16_t* x;
    const uint16_t* kv;
    int64_t ld_kv;
    const uint16_t* q;
    const uint16_t* k;
    const int8_t* xq;   // checkpoints instead of x and kv: [T, hc, dim], [T, hc + 1, dim], a scale per 32 columns of a row
    const uint8_t* xs;
    const int8_t* kvq;
    const uint8_t* kvs;
    const float* dot;
    const uint16_t* up;
    const uint8_t* mask;
    uint16_t* dx;
    uint16_t* dkv;
    float* part;  // [gridDim.x][hc * dim] sums over the workgroup's tokens of dd s h key
    int64_t T;
    int hc, dim;
    float eps, inv_dim, rsqrt_dim;
};

// Where the rows of the stream (copy c of token t) and of the keys and the value (row c of token t, the value's being hc)
// come from: eight consecutive elements of one, as they lie in memory until they are widened.
struct FromBf16 {
    Piece<Bf16> r;
    __device__ inline void zero() { r.v = u32x4{0, 0, 0, 0}; }
    template <bool kNt>
    __device__ inline void get(const uint16_t* row, int piece) {
        if constexpr (kNt) r.load_nt(row, piece);
        else r.load(row, piece);
    }
    template <bool kNt>
    __device__ inline void load_x(const GateGradArgs& p, int hc, int64_t t, int c, int piece) {
        get<kNt>(p.x + (t * hc + c) * p.dim, piece);
    }
    template <bool kNt>
    __device__ inline void load_kv(const GateGradArgs& p, int hc, int64_t t, int c, int piece) {
        get<kNt>(p.kv + t * p.ld_kv + static_cast<int64_t>(c) * p.dim, piece);
    }
    __device__ inline void to(float (&f)[8]) const { r.to(f); }
    __device__ inline void keep() { asm volatile("" : "+v"(r.v)); }
};
struct FromInt8 {
    mx_u32x2 q;
    uint32_t code;
    __device__ inline void zero() {
        q = mx_u32x2{0, 0};
        code = 0;
    }
    template <bool kNt>
    __device__ inline void get(const int8_t* rows, const uint8_t* scales, int64_t row, int dim, int piece) {
        const mx_u32x2* at = reinterpret_cast<const mx_u32x2*>(rows + row * dim) + piece;
        if constexpr (kNt) q = __builtin_nontemporal_load(at);
        else q = *at;
        code = scales[row * ((dim + 31) / 32) + (piece >> 2)];
    }
    template <bool kNt>
    __device__ inline void load_x(const GateGradArgs& p, int hc, int64_t t, int c, int piece) {
        get<kNt>(p.xq, p.xs, t * hc + c, p.dim, piece);
    }
    template <bool kNt>
    __device__ inline void load_kv(const GateGradArgs& p, int hc, int64_t t, int c, int piece) {
        get<kNt>(p.kvq, p.kvs, t * (hc + 1) + c, p.dim, piece);
    }
    __device__ inline void to(float (&f)[8]) const { mxint8_decode8(q, mxint8_unit(code), f); }
    __device__ inline void keep() { asm volatile("" : "+v"(q), "+v"(code)); }
};

// the scalars of one (token, copy)
struct Coef {
    float g;   // the gate
    float a;   // dd s
    float bh;  // dd d rh^2 / dim
    float bk;  // dd d rk^2 / dim
};
__device__ inline Coef coef_of(const GateGradArgs& p, float hh, float kk, float dg, float d) {
    const float rh = rsqrtf(hh * p.inv_dim + p.eps), rk = rsqrtf(kk * p.inv_dim + p.eps);
    const float z = sqrtf(fmaxf(fabsf(d), 1e-6f));
    Coef c;
    const float e = expf(-copysignf(z, d));
    c.g = 1.0f / (1.0f + e);
    // 1 - g = e g: where g is near 1 (e small) the difference has lost the digits that the product keeps (3e-4 of the slope
    // at d = 72, all of it from 300), where e is large it has them and the product may overflow
    const float shut = d > 0.f ? e * c.g : 1.0f - c.g;
    const float dd = fabsf(d) < 1e-6f ? 0.f : dg * c.g * shut / (2.0f * z);
    c.a = c.bh = c.bk = 0.f;
    if (dd != 0.f) {  // (a zero gradient stays zero next to the large norms of zero rows; NaN goes on)
        c.a = dd * (rh * rk * p.rsqrt_dim);
        c.bh = dd * (d * rh * rh * p.inv_dim);
        c.bk = dd * (d * rk * rk * p.inv_dim);
    }
    return c;
}

// A masked token: the gate is shut, so the stream's gradient passes and nothing else does.
__device__ inline void masked_token(const GateGradArgs& p, int64_t t, int piece) {
    const Piece<Bf16> zero = {u32x4{0, 0, 0, 0}};
    for (int c = 0; c < p.hc; ++c) {
        Piece<Bf16> u;
        u.load_nt(p.up + (t * p.hc + c) * p.dim, piece);
        u.store_nt(p.dx + (t * p.hc + c) * p.dim, piece);
    }
    for (int c = 0; c <= p.hc; ++c) zero.store_nt(p.dkv + (t * (p.hc + 1) + c) * p.dim, piece);
}

// A wave's sum, in its last lane.
__device__ inline float wave_sum_last(float v) {
    auto add = [&](auto ctrl, auto rows) {
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value,
                                                        0xF, false));
    };
    using std::integral_constant;
    integral_constant<int, 0xF> all;
    add(integral_constant<int, 0x111>{}, all);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has the row's sum
    add(integral_constant<int, 0x112>{}, all);
    add(integral_constant<int, 0x114>{}, all);
    add(integral_constant<int, 0x118>{}, all);
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast 15 into rows 1 and 3
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast 31 into rows 2 and 3
    return v;
}

// The LDS holds q * k (read for every token from L2 it cost 428 us where this takes 342, 8,192 x 4 x 5,120); of a workgroup
// of more than 640 threads and four copies, whose registers do not hold rows and sums together, the sums instead, and q
// and k come from L2 a copy ahead.
template <int HC, int kMaxThreads, class From>
__global__ __launch_bounds__(kMaxThreads) void gate_grad_kernel(GateGradArgs p) {
    constexpr int kSums = 3 * HC, kReads = (kSums + 3) / 4;
    __shared__ float sums[2][4 * kReads][kMaxWaves];  // [sum][wave]; waves the workgroup lacks hold zeros
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int piece = threadIdx.x;
    const bool live = piece < p.dim / 8;
    constexpr bool kSumsInLds = HC == 4 && kMaxThreads > 640;
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ f32x4 held[HC][2][kMaxThreads];  // [copy][half of a piece][thread]: q * k, or the sums
    for (int i = threadIdx.x; i < 2 * 4 * kReads * kMaxWaves; i += blockDim.x) (&sums[0][0][0])[i] = 0.f;
    auto put = [&](int c, const float (&w)[8]) {
        held[c][0][piece] = f32x4{w[0], w[1], w[2], w[3]};
        held[c][1][piece] = f32x4{w[4], w[5], w[6], w[7]};
    };
    auto get = [&](int c, float (&w)[8]) {
        const f32x4 lo = held[c][0][piece], hi = held[c][1][piece];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = lo[e];
            w[4 + e] = hi[e];
        }
    };
    Piece<Bf16> qr, kr_w;
    auto load_weights = [&](int c) {
        int at = c * (p.dim / 8) + piece;
        asm volatile("" : "+v"(at));  // read here, not once for all tokens into registers held over them
        qr.load(p.q, at);
        kr_w.load(p.k, at);
    };
    auto weights = [&](float (&w)[8]) {
        float kf[8];
        qr.to(w);
        kr_w.to(kf);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= kf[e];  // exact: bf16 * bf16 fits fp32
    };
    if (live) {
#pragma unroll
        for (int c = 0; c < HC; ++c) {
            float w[8] = {};
            if constexpr (!kSumsInLds) {
                load_weights(c);
                weights(w);
            }
            put(c, w);
        }
    }
    __syncthreads();
    float acc[kSumsInLds ? 1 : HC][8] = {};
    From hr[HC], kr[HC], vr;
    Piece<Bf16> ur[HC];
    auto load_copy = [&](int64_t t, int c) {
        hr[c].template load_x<true>(p, HC, t, c, piece);
        kr[c].template load_kv<true>(p, HC, t, c, piece);
        ur[c].load_nt(p.up + (t * HC + c) * p.dim, piece);
    };
    auto load_value = [&](int64_t t) { vr.template load_kv<true>(p, HC, t, HC, piece); };
    // the first token from t on that takes part; the masked ones before it are done with on the way
    auto next = [&](int64_t t) {
        for (; t < p.T && p.mask && p.mask[t] == 0; t += gridDim.x)
            if (live) masked_token(p, t, piece);
        return t;
    };
    int turn = 0;
    int64_t t = next(blockIdx.x);
    vr.zero();
#pragma unroll
    for (int c = 0; c < HC; ++c) {
        hr[c].zero();
        kr[c].zero();
        ur[c].v = u32x4{0, 0, 0, 0};
    }
    if (live && t < p.T) {
        load_value(t);
#pragma unroll
        for (int c = 0; c < HC; ++c) load_copy(t, c);
    }
    while (t < p.T) {
        {
            float v[8];
            vr.to(v);
#pragma unroll
            for (int c = 0; c < HC; ++c) {
                float h[8], key[8], u[8], hh = 0.f, kk = 0.f, dg = 0.f;
                hr[c].to(h);
                kr[c].to(key);
                ur[c].to(u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    hh += h[e] * h[e];
                    kk += key[e] * key[e];
                    dg += u[e] * v[e];
                }
                hh = wave_sum_last(hh);
                kk = wave_sum_last(kk);
                dg = wave_sum_last(dg);
                if (lane == 63) {
                    sums[turn][3 * c][wave] = hh;
                    sums[turn][3 * c + 1][wave] = kk;
                    sums[turn][3 * c + 2][wave] = dg;
                }
            }
        }
        if constexpr (kSumsInLds) {
            if (live) load_weights(0);
        }
        __syncthreads();
        // the rows as they were loaded: widened again below rather than held as floats over the barrier
#pragma unroll
        for (int c = 0; c < HC; ++c) {
            hr[c].keep();
            kr[c].keep();
            asm volatile("" : "+v"(ur[c].v));
        }
        // each 16 lanes add one sum over the waves: read j of lane l is sum 4 j + l / 16 of wave l % 16
        float part[kReads];
#pragma unroll
        for (int j = 0; j < kReads; ++j) {
            part[j] = sums[turn][4 * j + (lane >> 4)][lane & 15];
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) part[j] += __shfl_xor(part[j], off, 64);
        }
        auto total = [&](int i) {
            return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(part[i / 4]), (i % 4) * 16));
        };
        auto uniform = [](float f) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(f))); };
        // the next token's rows are asked for as soon as this one's are used up
        const int64_t ahead = next(t + gridDim.x);
        const bool more = live && ahead < p.T;
        if (more) load_value(ahead);
        float dv[8] = {};
#pragma unroll
        for (int c = 0; c < HC; ++c) {
            Coef k = coef_of(p, total(3 * c), total(3 * c + 1), total(3 * c + 2), p.dot[t * HC + c]);
            k = Coef{uniform(k.g), uniform(k.a), uniform(k.bh), uniform(k.bk)};
            if (live) {
                float w[8], sum[8];
                if constexpr (kSumsInLds) {
                    weights(w);
                    if (c + 1 < HC) load_weights(c + 1);
                    get(c, sum);
                } else {
                    get(c, w);
                }
                float h[8], key[8], u[8], ox[8], ok[8];
                hr[c].to(h);
                kr[c].to(key);
                ur[c].to(u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float aw = k.a * w[e];
                    ox[e] = u[e] + (aw * key[e] - k.bh * h[e]);
                    ok[e] = aw * h[e] - k.bk * key[e];
                    dv[e] += k.g * u[e];
                    const float add = k.a * (h[e] * key[e]);
                    if constexpr (kSumsInLds) sum[e] += add;
                    else acc[c][e] += add;
                }
                if constexpr (kSumsInLds) put(c, sum);
                Piece<Bf16> o;
                o.from(ox);
                o.store_nt(p.dx + (t * HC + c) * p.dim, piece);
                o.from(ok);
                o.store_nt(p.dkv + (t * (HC + 1) + c) * p.dim, piece);
                if (more) load_copy(ahead, c);
            }
            __builtin_amdgcn_sched_barrier(0);  // one copy's floats at a time
        }
        if (live) {
            Piece<Bf16> o;
            o.from(dv);
            o.store_nt(p.dkv + (t * (HC + 1) + HC) * p.dim, piece);
        }
        turn ^= 1;
        t = ahead;
    }
    if (!live) return;
#pragma unroll
    for (int c = 0; c < HC; ++c) {
        Piece<F32> o;
        if constexpr (kSumsInLds) {
            float sum[8];
            get(c, sum);
            o.from(sum);
        } else {
            o.from(acc[c]);
        }
        o.store(p.part + (static_cast<int64_t>(blockIdx.x) * HC + c) * p.dim, piece);
    }
}

// Any other number of copies: one copy after the other, the sums over tokens in the workgroup's own row of `part`
// (each thread reads and writes only its piece).
template <class From>
__global__ __launch_bounds__(1024) void gate_grad_any_kernel(GateGradArgs p) {
    __shared__ float sums[2][kMaxWaves][3];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int piece = threadIdx.x;
    const bool live = piece < p.dim / 8;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.hc * p.dim;
    Piece<F32> a;
    const float zero[8] = {};
    a.from(zero);
    if (live)
        for (int c = 0; c < p.hc; ++c) a.store(part + static_cast<int64_t>(c) * p.dim, piece);
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        if (p.mask && p.mask[t] == 0) {
            if (live) masked_token(p, t, piece);
            continue;
        }
        From f;
        f.zero();
        Piece<Bf16> r;
        float v[8], dv[8] = {};
        if (live) f.template load_kv<false>(p, p.hc, t, p.hc, piece);
        f.to(v);
        for (int c = 0; c < p.hc; ++c) {
            float h[8] = {}, key[8] = {}, u[8] = {}, hh = 0.f, kk = 0.f, dg = 0.f;
            if (live) {
                f.template load_x<false>(p, p.hc, t, c, piece);
                f.to(h);
                f.template load_kv<false>(p, p.hc, t, c, piece);
                f.to(key);
                r.load(p.up + (t * p.hc + c) * p.dim, piece);
                r.to(u);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hh += h[e] * h[e];
                kk += key[e] * key[e];
                dg += u[e] * v[e];
            }
            hh = wave_sum(hh);
            kk = wave_sum(kk);
            dg = wave_sum(dg);
            if (lane == 0) {
                sums[turn][wave][0] = hh;
                sums[turn][wave][1] = kk;
                sums[turn][wave][2] = dg;
            }
            __syncthreads();
            hh = kk = dg = 0.f;
            for (int w = 0; w < waves; ++w) {
                hh += sums[turn][w][0];
                kk += sums[turn][w][1];
                dg += sums[turn][w][2];
            }
            turn ^= 1;
            const Coef k = coef_of(p, hh, kk, dg, p.dot[t * p.hc + c]);
            if (!live) continue;
            float qf[8], kf[8], ox[8], ok[8], sum[8];
            r.load(p.q + static_cast<int64_t>(c) * p.dim, piece);
            r.to(qf);
            r.load(p.k + static_cast<int64_t>(c) * p.dim, piece);
            r.to(kf);
            a.load(part + static_cast<int64_t>(c) * p.dim, piece);
            a.to(sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float aw = k.a * (qf[e] * kf[e]);
                ox[e] = u[e] + (aw * key[e] - k.bh * h[e]);
                ok[e] = aw * h[e] - k.bk * key[e];
                dv[e] += k.g * u[e];
                sum[e] += k.a * (h[e] * key[e]);
            }
            a.from(sum);
            a.store(part + static_cast<int64_t>(c) * p.dim, piece);
            r.from(ox);
            r.store(p.dx + (t * p.hc + c) * p.dim, piece);
            r.from(ok);
            r.store(p.dkv + (t * (p.hc + 1) + c) * p.dim, piece);
        }
        if (live) {
            r.from(dv);
            r.store(p.dkv + (t * (p.hc + 1) + p.hc) * p.dim, piece);
        }
    }
}

// dq = k * sum, dk = q * sum over the workgroups' sums: kCols columns per workgroup, 1024 / kCols runs of rows.  Bound by
// the latency of its reads, eight in flight a thread.
template <int kCols>
__global__ __launch_bounds__(1024) void gate_grad_sum_kernel(const float* part, int rows, int cols, const uint16_t* q,
                                                             const uint16_t* k, float* dq, float* dk) {
    constexpr int kRuns = 1024 / kCols;
    __shared__ float run_sum[kRuns][kCols];
    const int col = blockIdx.x * kCols + threadIdx.x % kCols;
    const int run = threadIdx.x / kCols;
    const int per = (rows + kRuns - 1) / kRuns;
    const int r0 = min(run * per, rows), r1 = min(r0 + per, rows);
    float s = 0.f;
    if (col < cols) {
        for (int r = r0; r < r1; r += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = r + j < r1 ? part[static_cast<int64_t>(r + j) * cols + col] : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
    }
    run_sum[run][threadIdx.x % kCols] = s;
    __syncthreads();
    if (run != 0 || col >= cols) return;
    s = 0.f;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) s += run_sum[r][threadIdx.x];
    dq[col] = s * __uint_as_float(static_cast<uint32_t>(k[col]) << 16);
    dk[col] = s * __uint_as_float(static_cast<uint32_t>(q[col]) << 16);
}

template <int HC, class From>
void launch_gate_grad(const GateGradArgs& p, int64_t groups, int threads, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(groups)), block(threads);
    if (threads <= 64) hipLaunchKernelGGL((gate_grad_kernel<HC, 64, From>), grid, block, 0, s, p);
    else if (threads <= 128) hipLaunchKernelGGL((gate_grad_kernel<HC, 128, From>), grid, block, 0, s, p);
    else if (threads <= 256) hipLaunchKernelGGL((gate_grad_kernel<HC, 256, From>), grid, block, 0, s, p);
    else if (threads <= 384) hipLaunchKernelGGL((gate_grad_kernel<HC, 384, From>), grid, block, 0, s, p);
    else if (threads <= 640) hipLaunchKernelGGL((gate_grad_kernel<HC, 640, From>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((gate_grad_kernel<HC, 1024, From>), grid, block, 0, s, p);
}

int threads_of(int dim) { return (dim / 8 + 63) / 64 * 64; }

// Workgroups of a launch: as many as the CUs hold (the kernels' registers leave 12 waves a CU for hc 4, 16 for most, 20
// for hc 1), yet four tokens or more for each once every CU has one: every workgroup leaves a row of sums to be added.
int64_t groups_of(int64_t T, int hc, int dim) {
    const int waves = threads_of(dim) / 64, fit = hc == 4 ? 12 : hc == 1 ? 20 : 16;
    const int64_t per_cu = fit / waves > 1 ? fit / waves : 1;
    const int64_t few = T < kCUs ? T : (T + 3) / 4 > kCUs ? (T + 3) / 4 : kCUs;
    return few < per_cu * kCUs ? few : per_cu * kCUs;
}

bool shape_ok(int64_t T, int32_t hc, int32_t dim) {
    return T >= 0 && hc >= 1 && hc <= 64 && dim >= 8 && dim % 8 == 0 && dim <= kMaxDim;
}

// the two launches of either entry point
template <class From>
int launch_backward(GateGradArgs p, float* dq, float* dk, hipStream_t s, const char* what) {
    p.inv_dim = 1.0f / static_cast<float>(p.dim);
    p.rsqrt_dim = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(p.dim)));
    const int64_t groups = groups_of(p.T, p.hc, p.dim);
    const int threads = threads_of(p.dim);
    if (p.T > 0) {
        if (p.hc == 4) launch_gate_grad<4, From>(p, groups, threads, s);
        else if (p.hc == 2) launch_gate_grad<2, From>(p, groups, threads, s);
        else if (p.hc == 1) launch_gate_grad<1, From>(p, groups, threads, s);
        else hipLaunchKernelGGL(gate_grad_any_kernel<From>, dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s, p);
    }
    const int cols = p.hc * p.dim;
    // few columns: fewer of them per workgroup, so that there are workgroups enough
    const int rows = static_cast<int>(groups);
    if (cols >= 64 * kCUs)
        hipLaunchKernelGGL(gate_grad_sum_kernel<64>, dim3((cols + 63) / 64), dim3(1024), 0, s, p.part, rows, cols, p.q, p.k, dq,
                           dk);
    else
        hipLaunchKernelGGL(gate_grad_sum_kernel<16>, dim3((cols + 15) / 16), dim3(1024), 0, s, p.part, rows, cols, p.q, p.k, dq,
                           dk);
    return check_launch(what);
}

// What either entry point asks of its sizes, and of its pointers (`rows_null`, `rows_misaligned`: of the rows it reads): a
// status, with the reason left for engram_last_error.
int check_sizes(const GateGradArgs& p, const char* what) {
    if (p.T < 0) return fail(ENGRAM_EINVAL, "%s: T < 0", what);
    if (p.hc < 1 || p.hc > 64) return fail(ENGRAM_EINVAL, "%s: hc=%d outside [1, 64]", what, p.hc);
    if (p.dim < 8 || p.dim % 8 != 0 || p.dim > kMaxDim)
        return fail(ENGRAM_EINVAL, "%s: dim=%d must be a multiple of 8 in [8, %d]", what, p.dim, kMaxDim);
    return ENGRAM_OK;
}
int check_pointers(const GateGradArgs& p, const float* dq, const float* dk, bool rows_null, bool rows_misaligned,
                   int64_t workspace_bytes, const char* what) {
    if (!p.q || !p.k || !dq || !dk) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(dq, 4) || !aligned(dk, 4))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    if (p.T == 0) return ENGRAM_OK;
    if (rows_null || !p.dot || !p.up || !p.dx || !p.dkv || !p.part) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (rows_misaligned || !aligned(p.up, 16) || !aligned(p.dx, 16) || !aligned(p.dkv, 16) || !aligned(p.dot, 4) ||
        !aligned(p.part, 16))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const int64_t need = groups_of(p.T, p.hc, p.dim) * p.hc * p.dim * 4;
    if (workspace_bytes < need)
        return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                    (long long)need);
    return ENGRAM_OK;
}

GateGradArgs common_args(const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* dot, const uint16_t* dout,
                         const uint8_t* token_mask, uint16_t* dx, uint16_t* dkv, void* workspace, int64_t T, int32_t hc,
                         int32_t dim) {
    GateGradArgs p = {};
    p.q = q_weight;
    p.k = k_weight;
    p.dot = dot;
    p.up = dout;
    p.mask = token_mask;
    p.dx = dx;
    p.dkv = dkv;
    p.part = static_cast<float*>(workspace);
    p.T = T;
    p.hc = hc;
    p.dim = dim;
    p.eps = eps;
    return p;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int64_t engram_gate_output_backward_workspace_bytes(int64_t T, int32_t hc, int32_t dim) {
    return shape_ok(T, hc, dim) ? groups_of(T, hc, dim) * hc * dim * 4 : -1;
}

extern "C" int engram_gate_output_backward(const uint16_t* x, const uint16_t* kv, int64_t ld_kv, const uint16_t* q_weight,
                                           const uint16_t* k_weight, float eps, const float* dot, const uint16_t* dout,
                                           const uint8_t* token_mask, uint16_t* dx, uint16_t* dkv, float* dq, float* dk,
                                           void* workspace, int64_t workspace_bytes, int64_t T, int32_t hc, int32_t dim,
                                           void* stream) {
    const char* what = "engram_gate_output_backward";
    GateGradArgs p = common_args(q_weight, k_weight, eps, dot, dout, token_mask, dx, dkv, workspace, T, hc, dim);
    int rc = check_sizes(p, what);
    if (rc != ENGRAM_OK) return rc;
    if (ld_kv < static_cast<int64_t>(hc + 1) * dim || ld_kv % 8 != 0)
        return fail(ENGRAM_EINVAL, "%s: ld_kv=%lld must be >= (hc+1)*dim and a multiple of 8", what, (long long)ld_kv);
    rc = check_pointers(p, dq, dk, !x || !kv, !aligned(x, 16) || !aligned(kv, 16), workspace_bytes, what);
    if (rc != ENGRAM_OK) return rc;
    p.x = x;
    p.kv = kv;
    p.ld_kv = ld_kv;
    return launch_backward<FromBf16>(p, dq, dk, as_stream(stream), what);
}

extern "C" int engram_gate_output_backward_ckpt(const int8_t* x_q, const uint8_t* x_scale, const int8_t* kv_q,
                                                const uint8_t* kv_scale, const uint16_t* q_weight, const uint16_t* k_weight,
                                                float eps, const float* dot, const uint16_t* dout, const uint8_t* token_mask,
                                                uint16_t* dx, uint16_t* dkv, float* dq, float* dk, void* workspace,
                                                int64_t workspace_bytes, int64_t T, int32_t hc, int32_t dim, void* stream) {
    const char* what = "engram_gate_output_backward_ckpt";
    GateGradArgs p = common_args(q_weight, k_weight, eps, dot, dout, token_mask, dx, dkv, workspace, T, hc, dim);
    int rc = check_sizes(p, what);
    if (rc == ENGRAM_OK)
        rc = check_pointers(p, dq, dk, !x_q || !x_scale || !kv_q || !kv_scale, !aligned(x_q, 8) || !aligned(kv_q, 8),
                            workspace_bytes, what);
    if (rc != ENGRAM_OK) return rc;
    p.xq = x_q;
    p.xs = x_scale;
    p.kvq = kv_q;
    p.kvs = kv_scale;
    return launch_backward<FromInt8>(p, dq, dk, as_stream(stream), what);
}
