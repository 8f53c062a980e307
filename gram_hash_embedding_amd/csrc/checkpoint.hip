// 8-bit checkpoints of the rows that a backward pass reads again, in OCP MXINT8: 32 consecutive columns of a row share an
// E8M0 scale, elements are integers in [-127, 127], in 64ths of the scale (mx.h).  A row's scales lie together, [rows][ceil(D
// / 32)], the last block of a row may be shorter.
//
//   engram_ckpt_save        -- bf16 rows -> MXINT8
//   engram_ckpt_load        -- MXINT8 -> bf16 rows (exact: an element has 7 bits, bf16 holds 8)
//   engram_gate_output_ckpt -- engram_gate_output that writes the checkpoints of the stream, the keys and the value from the
//                              rows it has in registers, instead of a second pass that reads them (gate_grad.hip reads them)
//
// All three are bound by HBM: 32,768 x 5,120 saved in 92 us (5.6 TB/s), loaded in 86 (5.9); the output of 8,192 x 4 x 5,120 268
// (5.5).  engram_gate_output and then engram_ckpt_save, which reads the same 754 MB again, take 213 and 201.
#include "gate.h"
#include "mx.h"

namespace engram {
namespace {

constexpr int kThreads = 256;

// Four lanes hold a block of 32 (piece j: columns 8 j .. 8 j + 7); lanes without a piece pass zeros and `ok` false.  Every lane
// of the wave takes part.
__device__ inline void save_piece(const u32x4& v, bool ok, int8_t* q, uint8_t* scale, int j) {
    const uint32_t code = block_top(bf16_top8(v)) >> 7;
    const mx_u32x2 e = mxint8_encode8(v, code);
    if (!ok) return;
    __builtin_nontemporal_store(e, reinterpret_cast<mx_u32x2*>(q) + j);
    if ((j & 3) == 0) scale[j >> 2] = static_cast<uint8_t>(code);
}

// A thread per piece; rows of `chunks` pieces padded to whole blocks.
__global__ __launch_bounds__(kThreads) void ckpt_save_kernel(const uint16_t* x, int64_t rows, int chunks, int8_t* q,
                                                             uint8_t* scale) {
    const int blocks = (chunks + 3) / 4;
    const int64_t i = group_index() * kThreads + threadIdx.x;
    const int64_t r = i / (4 * blocks);
    const int j = static_cast<int>(i - r * (4 * blocks));
    const bool ok = r < rows && j < chunks;
    u32x4 v = {0, 0, 0, 0};
    if (ok) v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x) + r * chunks + j);
    save_piece(v, ok, q + r * chunks * 8, scale + r * blocks, j);
}

__global__ __launch_bounds__(kThreads) void ckpt_load_kernel(const int8_t* q, const uint8_t* scale, int64_t rows, int chunks,
                                                             uint16_t* x) {
    const int64_t i = group_index() * kThreads + threadIdx.x;
    const int64_t r = i / chunks;
    const int j = static_cast<int>(i - r * chunks);
    if (r >= rows) return;
    const mx_u32x2 e = __builtin_nontemporal_load(reinterpret_cast<const mx_u32x2*>(q) + i);
    float f[8];
    mxint8_decode8(e, mxint8_unit(scale[r * ((chunks + 3) / 4) + (j >> 2)]), f);
    u32x4 o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = pack2_bf16(f[2 * p], f[2 * p + 1]);
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(x) + i);
}

struct CkptArgs {
    const uint16_t* x;
    const uint16_t* kv;
    int64_t ld_kv;
    const uint16_t* q;
    const uint16_t* k;
    const uint8_t* mask;  // [T] or null
    float eps, inv_dim, rsqrt_dim;
    uint16_t* out;
    float* dot;
    int8_t* xq;           // [T, hc, dim]
    uint8_t* xs;          // [T, hc, blocks]
    int8_t* kvq;          // [T, hc + 1, dim]
    uint8_t* kvs;         // [T, hc + 1, blocks]
    int64_t T;
    int hc, dim;
};

// The sum of v over the lanes of a row: L neighbours in a wave, or a workgroup, whose waves' sums meet in `part` (every thread
// adds them in wave order).
template <int L>
__device__ inline void row_sums(float (&v)[3], float (*part)[3]) {
#pragma unroll
    for (int off = (L < 64 ? L : 64) / 2; off >= 1; off >>= 1)
#pragma unroll
        for (int e = 0; e < 3; ++e) v[e] += __shfl_xor(v[e], off, 64);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0)
            for (int e = 0; e < 3; ++e) part[threadIdx.x >> 6][e] = v[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            v[e] = 0.f;
#pragma unroll
            for (int w = 0; w < L / 64; ++w) v[e] += part[w][e];
        }
    }
}

// L threads per (token, copy), a token's copies in one workgroup or on one XCD, which reads its value row from HBM once (8,192 x
// 4 x 5,120 269 us, 5.5 TB/s; 279 with every copy on another); thread i has the 16-byte pieces i + L u (P of them) of the copy's
// stream and key rows and of the value row.
template <int L, int P>
__global__ __launch_bounds__(L < kThreads ? kThreads : L) void gate_output_ckpt_kernel(CkptArgs a) {
    __shared__ float part[(L + 63) / 64][3];
    constexpr int kRows = L < kThreads ? kThreads / L : 1;  // of a workgroup
    const int64_t n = a.T * a.hc, groups = (n + kRows - 1) / kRows;
    const int64_t group = part_of_group(group_index<kRows * L>(), groups, (a.hc + kRows - 1) / kRows);
    if (group >= groups) return;
    const int lane = kRows == 1 ? threadIdx.x : threadIdx.x % L;
    const int64_t at = kRows == 1 ? group : group * kRows + threadIdx.x / L;  // token * hc + copy
    const bool live = kRows == 1 || at < n;
    const int64_t tc = live ? at : n - 1;
    const int64_t t = tc / a.hc;
    const int c = static_cast<int>(tc - t * a.hc);
    const int chunks = a.dim / 8, blocks = (chunks + 3) / 4;
    const u32x4* q = reinterpret_cast<const u32x4*>(a.q + static_cast<int64_t>(c) * a.dim);
    const u32x4* k = reinterpret_cast<const u32x4*>(a.k + static_cast<int64_t>(c) * a.dim);
    const uint16_t* row = a.kv + t * a.ld_kv;
    const u32x4* h = reinterpret_cast<const u32x4*>(a.x + tc * a.dim);
    const u32x4* key = reinterpret_cast<const u32x4*>(row + static_cast<int64_t>(c) * a.dim);
    const u32x4* val = reinterpret_cast<const u32x4*>(row + static_cast<int64_t>(a.hc) * a.dim);
    u32x4* out = reinterpret_cast<u32x4*>(a.out + tc * a.dim);
    const int64_t krow = t * (a.hc + 1) + c, vrow = t * (a.hc + 1) + a.hc;
    u32x4 hr[P], kr[P], vr[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int j = lane + L * i;
        hr[i] = kr[i] = vr[i] = u32x4{0, 0, 0, 0};
        if (live && j < chunks) {
            hr[i] = __builtin_nontemporal_load(h + j);
            kr[i] = __builtin_nontemporal_load(key + j);
            vr[i] = val[j];
        }
    }
    float sum[3] = {0.f, 0.f, 0.f};  // of h^2, key^2 and h w key
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int j = lane + L * i;
        const bool ok = live && j < chunks;
        if (ok) {
            const u32x4 qv = q[j], kw = k[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w0 = lo_bf16(qv[e]) * lo_bf16(kw[e]);  // exact: bf16 * bf16 fits fp32
                const float w1 = hi_bf16(qv[e]) * hi_bf16(kw[e]);
                const float h0 = lo_bf16(hr[i][e]), h1 = hi_bf16(hr[i][e]);
                const float k0 = lo_bf16(kr[i][e]), k1 = hi_bf16(kr[i][e]);
                sum[0] += h0 * h0 + h1 * h1;
                sum[1] += k0 * k0 + k1 * k1;
                sum[2] += h0 * w0 * k0 + h1 * w1 * k1;
            }
        }
        save_piece(hr[i], ok, a.xq + tc * a.dim, a.xs + tc * blocks, j);
        save_piece(kr[i], ok, a.kvq + krow * a.dim, a.kvs + krow * blocks, j);
        if (kRows > 1 || c == 0) save_piece(vr[i], ok && c == 0, a.kvq + vrow * a.dim, a.kvs + vrow * blocks, j);
    }
    row_sums<L>(sum, part);
    const float rstd = rsqrtf(sum[0] * a.inv_dim + a.eps) * rsqrtf(sum[1] * a.inv_dim + a.eps);
    const float d = sum[2] * rstd * a.rsqrt_dim;
    if (live && lane == 0) a.dot[tc] = d;
    const float gate = (a.mask && a.mask[t] == 0) ? 0.f : gate_of(d);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int j = lane + L * i;
        if (live && j < chunks) __builtin_nontemporal_store(residual(hr[i], vr[i], gate), out + j);
    }
}

template <int L, int P>
int launch_output(const CkptArgs& a, hipStream_t stream, const char* what) {
    constexpr int kRows = L < kThreads ? kThreads / L : 1;
    hipLaunchKernelGGL((gate_output_ckpt_kernel<L, P>), group_grid((a.T * a.hc + kRows - 1) / kRows, kRows * L), dim3(kRows * L),
                       0, stream, a);
    return check_launch(what);
}

// what is wrong with a checkpoint's rows, or null
const char* bad_rows(int64_t rows, int32_t D) {
    if (rows < 0) return "rows < 0";
    if (D < 8 || D % 8 != 0 || D > (1 << 20)) return "D must be a multiple of 8 in [8, 2^20]";
    if (rows > (1ll << 48) / ((D + 31) / 32 * 32)) return "too many rows";
    return nullptr;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int engram_ckpt_save(const uint16_t* x, int64_t rows, int32_t D, int8_t* q, uint8_t* scale, void* stream) {
    const char* what = "engram_ckpt_save";
    if (const char* bad = bad_rows(rows, D)) return fail(ENGRAM_EINVAL, "%s: %s", what, bad);
    if (rows == 0) return ENGRAM_OK;
    if (!x || !q || !scale) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(x, 16) || !aligned(q, 8)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const int64_t blocks = (rows * 4 * ((D + 31) / 32) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(ckpt_save_kernel, group_grid(blocks), dim3(kThreads), 0, as_stream(stream), x, rows,
                       D / 8, q, scale);
    return check_launch(what);
}

extern "C" int engram_ckpt_load(const int8_t* q, const uint8_t* scale, int64_t rows, int32_t D, uint16_t* x, void* stream) {
    const char* what = "engram_ckpt_load";
    if (const char* bad = bad_rows(rows, D)) return fail(ENGRAM_EINVAL, "%s: %s", what, bad);
    if (rows == 0) return ENGRAM_OK;
    if (!x || !q || !scale) return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(x, 16) || !aligned(q, 8)) return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    const int64_t blocks = (rows * (D / 8) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(ckpt_load_kernel, group_grid(blocks), dim3(kThreads), 0, as_stream(stream), q, scale,
                       rows, D / 8, x);
    return check_launch(what);
}

extern "C" int engram_gate_output_ckpt(const uint16_t* x, const uint16_t* kv, int64_t ld_kv, const uint16_t* q_weight,
                                       const uint16_t* k_weight, float eps, const uint8_t* token_mask, uint16_t* out,
                                       float* dot, int8_t* x_q, uint8_t* x_scale, int8_t* kv_q, uint8_t* kv_scale, int64_t T,
                                       int32_t hc, int32_t dim, void* stream) {
    const char* what = "engram_gate_output_ckpt";
    if (T < 0) return fail(ENGRAM_EINVAL, "%s: T < 0", what);
    if (hc < 1 || hc > 64) return fail(ENGRAM_EINVAL, "%s: hc=%d outside [1, 64]", what, hc);
    if (dim < 8 || dim % 8 != 0 || dim > 8192)
        return fail(ENGRAM_EINVAL, "%s: dim=%d must be a multiple of 8 in [8, 8192]", what, dim);
    if (ld_kv < static_cast<int64_t>(hc + 1) * dim || ld_kv % 8 != 0)
        return fail(ENGRAM_EINVAL, "%s: ld_kv=%lld must be >= (hc+1)*dim and a multiple of 8", what, (long long)ld_kv);
    if (T > (1ll << 37) / hc) return fail(ENGRAM_EINVAL, "%s: too many tokens", what);
    if (T == 0) return ENGRAM_OK;
    if (!x || !kv || !q_weight || !k_weight || !out || !dot || !x_q || !x_scale || !kv_q || !kv_scale)
        return fail(ENGRAM_EINVAL, "%s: null pointer", what);
    if (!aligned(x, 16) || !aligned(kv, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(out, 16) ||
        !aligned(dot, 4) || !aligned(x_q, 8) || !aligned(kv_q, 8))
        return fail(ENGRAM_EINVAL, "%s: misaligned pointer", what);
    CkptArgs a = {};
    a.x = x;
    a.kv = kv;
    a.ld_kv = ld_kv;
    a.q = q_weight;
    a.k = k_weight;
    a.mask = token_mask;
    a.eps = eps;
    a.inv_dim = 1.0f / static_cast<float>(dim);
    a.rsqrt_dim = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(dim)));
    a.out = out;
    a.dot = dot;
    a.xq = x_q;
    a.xs = x_scale;
    a.kvq = kv_q;
    a.kvs = kv_scale;
    a.T = T;
    a.hc = hc;
    a.dim = dim;
    // As many threads a row as it has pieces, up to a wave of two each, so that no thread idles and no barrier is met: 8,192 x 4
    // x 256 17 us, of 512 32, of 1,024 56 (a workgroup a row 60, 63 and 75; but 64 x 4 x 1,024 4.7 against 4.0).  Past 1,024 a
    // workgroup of one to three pieces a thread: of 2,048 108 us (a wave a row 124), of 5,120 268 (640 threads 330), of 8,192
    // 430 (1,024 threads 625).
    hipStream_t s = as_stream(stream);
    if (dim <= 128) return launch_output<16, 1>(a, s, what);
    if (dim <= 256) return launch_output<32, 1>(a, s, what);
    if (dim <= 512) return launch_output<64, 1>(a, s, what);
    if (dim <= 1024) return launch_output<64, 2>(a, s, what);
    if (dim <= 2048) return launch_output<256, 1>(a, s, what);
    if (dim <= 4096) return launch_output<256, 2>(a, s, what);
    if (dim <= 6144) return launch_output<256, 3>(a, s, what);
    return launch_output<512, 2>(a, s, what);
}
