// engram_grad_norm: the 2-norm of many tensors taken as one vector.
// engram_clip_grads: every tensor times min(1, max_norm / (norm + 1e-6)).
//
// Both stream each gradient once.  A launch takes up to kTensors tensors, cut into runs, one per workgroup, which finds
// its tensor by binary search in the kernel's arguments.  Squares are added in fp64: fp32 running sums over a run would
// lose digits against the one rounding of the result, and squares past fp32's range (gradients over 1.8e19) would give
// infinity where the norm is finite.  The runs' sums are added in their order by one workgroup, so the norm has the
// same bits from every call.  The clipping takes the runs last to first: what the norm read last is still in the
// Infinity Cache.
//
// HBM-bound: the gradients of two layers and of a token embedding, 1.74 GB in all, take 843 us: the norm some 285 (6.1
// TB/s), its last launch 8, the clipping 560 (3.48 GB, 6.2 TB/s).  Two passes over the gradients are the operator's own:
// no factor is known before the last element is read.
#include "rows.h"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 96;         // per launch: 96 * 28 bytes of kernel arguments
constexpr int kNormPieces = 16;       // 16-byte pieces per thread and run
constexpr int kClipPieces = 1;
constexpr int64_t kMaxBlocks = 1ll << 23;  // workgroups per launch: times the threads stays below 2^32

struct NormList {
    const void* in[kTensors];
    void* out[kTensors];
    int64_t n[kTensors];
    uint32_t first[kTensors];  // first workgroup of the tensor
    uint32_t f32[(kTensors + 31) / 32];
    int tensors;
};

__device__ inline int tensor_of(const NormList& l, uint32_t block) {
    int lo = 0, hi = l.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (l.first[mid] <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ inline double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ inline double block_sum(double v, double* lds) {
    v = wave_sum(v);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < waves; ++w) v += lds[w];
    return v;
}

__device__ inline float element(const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// 16 bytes of a gradient: eight bf16 or four fp32
__device__ inline double squares(u32x4 v, bool f32) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (f32) {
            const double a = __uint_as_float(v[i]);
            s += a * a;
        } else {
            const double a = __uint_as_float(v[i] << 16), b = __uint_as_float(v[i] & 0xFFFF0000u);
            s += a * a;
            s += b * b;
        }
    }
    return s;
}
__device__ inline u32x4 scaled(u32x4 v, bool f32, float c) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (f32) {
            v[i] = __float_as_uint(__uint_as_float(v[i]) * c);
        } else {
            const bf16x2 p = {static_cast<__bf16>(__uint_as_float(v[i] << 16) * c),
                              static_cast<__bf16>(__uint_as_float(v[i] & 0xFFFF0000u) * c)};
            v[i] = __builtin_bit_cast(uint32_t, p);
        }
    }
    return v;
}

// a workgroup's run: its tensor, its elements and how many whole 16-byte pieces it may move at once
struct Run {
    int t;
    bool f32;
    int64_t i0, i1;   // elements
    int64_t p0, p1;   // 16-byte pieces of the tensor, none if it is not aligned to them
    int64_t rest;     // first element after the pieces
};
template <int kPieces>
__device__ inline Run run_of(const NormList& l, uint32_t block, int t, bool pieces) {
    Run r;
    r.t = t;
    r.f32 = (l.f32[r.t >> 5] >> (r.t & 31)) & 1;
    const int per = r.f32 ? 4 : 8;
    r.i0 = static_cast<int64_t>(block - l.first[r.t]) * (per * kPieces * kThreads);
    r.i1 = min(r.i0 + per * kPieces * kThreads, l.n[r.t]);
    r.p0 = r.i0 / per;
    r.p1 = pieces ? r.i1 / per : r.p0;
    r.rest = r.p1 * per;
    return r;
}

// Eight 16-byte loads in flight a thread.
__global__ __launch_bounds__(kThreads) void norm_kernel(NormList l, double* part) {
    __shared__ double lds[kThreads / 64];
    const int t = tensor_of(l, blockIdx.x);
    const Run r = run_of<kNormPieces>(l, blockIdx.x, t, (reinterpret_cast<uintptr_t>(l.in[t]) & 15) == 0);
    constexpr int kBatch = 8;
    double s = 0.0;
#pragma unroll
    for (int b = 0; b < kNormPieces; b += kBatch) {
        u32x4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t p = r.p0 + (b + u) * kThreads + threadIdx.x;
            v[u] = p < r.p1 ? static_cast<const u32x4*>(l.in[t])[p] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) s += squares(v[u], r.f32);
    }
    for (int64_t i = r.rest + threadIdx.x; i < r.i1; i += kThreads) {
        const double x = element(l.in[t], r.f32, i);
        s += x * x;
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// One workgroup: latency, 8 us for 27,000 runs and 3.5 for few.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const double* part, int64_t n, float* norm) {
    __shared__ double lds[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 8 * 1024) {
        double v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = i + u * 1024 < n ? part[i + u * 1024] : 0.0;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

// One 16-byte store a thread in memory order, past the caches: nothing reads the result before the rest is written.
__global__ __launch_bounds__(kThreads) void clip_kernel(NormList l, const float* norm, float max_norm) {
    const float c = max_norm / (*norm + 1e-6f);
    const float coef = c > 1.0f ? 1.0f : c;  // NaN stays NaN
    const uint32_t block = gridDim.x - 1 - blockIdx.x;
    const int t = tensor_of(l, block);
    if (coef == 1.0f && l.in[t] == l.out[t]) return;  // in place and nothing to clip
    const Run r = run_of<kClipPieces>(l, block, t,
                               ((reinterpret_cast<uintptr_t>(l.in[t]) | reinterpret_cast<uintptr_t>(l.out[t])) & 15) == 0);
    u32x4 v[kClipPieces];
#pragma unroll
    for (int u = 0; u < kClipPieces; ++u) {
        const int64_t p = r.p0 + u * kThreads + threadIdx.x;
        if (p < r.p1) v[u] = static_cast<const u32x4*>(l.in[t])[p];
    }
#pragma unroll
    for (int u = 0; u < kClipPieces; ++u) {
        const int64_t p = r.p0 + u * kThreads + threadIdx.x;
        if (p < r.p1) __builtin_nontemporal_store(scaled(v[u], r.f32, coef), static_cast<u32x4*>(l.out[t]) + p);
    }
    for (int64_t i = r.rest + threadIdx.x; i < r.i1; i += kThreads) {
        const float x = element(l.in[t], r.f32, i) * coef;
        if (r.f32) {
            static_cast<float*>(l.out[t])[i] = x;
        } else {
            const __bf16 b = static_cast<__bf16>(x);
            static_cast<uint16_t*>(l.out[t])[i] = __builtin_bit_cast(uint16_t, b);
        }
    }
}

int64_t runs_of(int64_t n, int32_t dtype, int pieces) {
    const int64_t run = static_cast<int64_t>(pieces) * kThreads * (dtype == ENGRAM_F32 ? 4 : 8);
    return (n + run - 1) / run;
}

int check_list(const char* what, int32_t tensors, const void* const* in, const int64_t* n, const int32_t* dtype) {
    if (tensors < 0) return fail(ENGRAM_EINVAL, "%s: tensors < 0", what);
    if (tensors == 0) return ENGRAM_OK;
    if (!in || !n || !dtype) return fail(ENGRAM_EINVAL, "%s: null list", what);
    for (int i = 0; i < tensors; ++i) {
        if (!known_dtype(dtype[i])) return fail(ENGRAM_EINVAL, "%s: tensor %d has an unknown dtype", what, i);
        if (n[i] < 0 || n[i] > (1ll << 40)) return fail(ENGRAM_EINVAL, "%s: tensor %d: size outside [0, 2^40]", what, i);
        if (n[i] == 0) continue;
        if (!in[i]) return fail(ENGRAM_EINVAL, "%s: tensor %d: null pointer", what, i);
        if (!aligned(in[i], dtype[i] == ENGRAM_F32 ? 4 : 2))
            return fail(ENGRAM_EINVAL, "%s: tensor %d: misaligned pointer", what, i);
    }
    return ENGRAM_OK;
}

// The tensors in lists of kTensors and of at most kMaxBlocks workgroups, a tensor that needs more of them cut between two
// runs; `launch(list, blocks, runs before)` until one fails.
template <class F>
int for_lists(int32_t tensors, const void* const* in, void* const* out, const int64_t* n, const int32_t* dtype,
              int pieces, F&& launch) {
    NormList l = {};
    int64_t blocks = 0, before = 0;
    auto flush = [&]() {
        const int rc = l.tensors ? launch(l, static_cast<unsigned>(blocks), before) : ENGRAM_OK;
        before += blocks;
        l = NormList{};
        blocks = 0;
        return rc;
    };
    for (int i = 0; i < tensors; ++i) {
        const int64_t size = dtype[i] == ENGRAM_F32 ? 4 : 2, run = static_cast<int64_t>(pieces) * kThreads * 16 / size;
        for (int64_t done = 0; done < n[i];) {
            if (l.tensors == kTensors || blocks == kMaxBlocks) {
                const int rc = flush();
                if (rc != ENGRAM_OK) return rc;
            }
            const int64_t left = runs_of(n[i] - done, dtype[i], pieces), room = kMaxBlocks - blocks;
            const int64_t r = left < room ? left : room;
            const int at = l.tensors++;
            l.in[at] = static_cast<const uint8_t*>(in[i]) + done * size;
            l.out[at] = out ? static_cast<uint8_t*>(out[i]) + done * size : nullptr;
            l.n[at] = r * run < n[i] - done ? r * run : n[i] - done;
            l.first[at] = static_cast<uint32_t>(blocks);
            if (dtype[i] == ENGRAM_F32) l.f32[at >> 5] |= 1u << (at & 31);
            blocks += r;
            done += l.n[at];
        }
    }
    return flush();
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int64_t engram_grad_norm_workspace_bytes(int32_t tensors, const int64_t* n, const int32_t* dtype) {
    if (tensors < 0 || (tensors > 0 && (!n || !dtype))) return -1;
    int64_t runs = 0;
    for (int i = 0; i < tensors; ++i) {
        if (!known_dtype(dtype[i]) || n[i] < 0 || n[i] > (1ll << 40)) return -1;
        runs += runs_of(n[i], dtype[i], kNormPieces);
    }
    return runs * 8;
}

extern "C" int engram_grad_norm(int32_t tensors, const void* const* grads, const int64_t* n, const int32_t* dtype,
                                float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* what = "engram_grad_norm";
    int rc = check_list(what, tensors, grads, n, dtype);
    if (rc != ENGRAM_OK) return rc;
    if (!norm || !aligned(norm, 4)) return fail(ENGRAM_EINVAL, "%s: norm is null or misaligned", what);
    const int64_t need = engram_grad_norm_workspace_bytes(tensors, n, dtype);
    if (need > 0 && (!workspace || !aligned(workspace, 8)))
        return fail(ENGRAM_EINVAL, "%s: workspace is null or misaligned", what);
    if (workspace_bytes < need)
        return fail(ENGRAM_ERANGE, "%s: workspace of %lld bytes, needs %lld", what, (long long)workspace_bytes,
                    (long long)need);
    hipStream_t s = as_stream(stream);
    double* part = static_cast<double*>(workspace);
    rc = for_lists(tensors, grads, nullptr, n, dtype, kNormPieces, [&](const NormList& l, unsigned blocks, int64_t before) {
        hipLaunchKernelGGL(norm_kernel, dim3(blocks), dim3(kThreads), 0, s, l, part + before);
        return check_launch(what);
    });
    if (rc != ENGRAM_OK) return rc;
    hipLaunchKernelGGL(norm_sum_kernel, dim3(1), dim3(1024), 0, s, part, need / 8, norm);
    return check_launch(what);
}

extern "C" int engram_clip_grads(int32_t tensors, const void* const* grads, void* const* out, const int64_t* n,
                                 const int32_t* dtype, const float* norm, float max_norm, void* stream) {
    const char* what = "engram_clip_grads";
    const int rc = check_list(what, tensors, grads, n, dtype);
    if (rc != ENGRAM_OK) return rc;
    if (!(max_norm >= 0.f)) return fail(ENGRAM_EINVAL, "%s: max_norm must be >= 0", what);
    if (tensors == 0) return ENGRAM_OK;
    if (!norm || !aligned(norm, 4)) return fail(ENGRAM_EINVAL, "%s: norm is null or misaligned", what);
    if (!out) return fail(ENGRAM_EINVAL, "%s: null list", what);
    for (int i = 0; i < tensors; ++i) {
        if (n[i] == 0) continue;
        if (!out[i]) return fail(ENGRAM_EINVAL, "%s: output %d: null pointer", what, i);
        if (!aligned(out[i], dtype[i] == ENGRAM_F32 ? 4 : 2))
            return fail(ENGRAM_EINVAL, "%s: output %d: misaligned pointer", what, i);
    }
    hipStream_t s = as_stream(stream);
    return for_lists(tensors, grads, out, n, dtype, kClipPieces, [&](const NormList& l, unsigned blocks, int64_t) {
        hipLaunchKernelGGL(clip_kernel, dim3(blocks), dim3(kThreads), 0, s, l, norm, max_norm);
        return check_launch(what);
    });
}
