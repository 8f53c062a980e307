// engram_grad_norm: the 2-norm of many tensors taken as one vector.
// engram_clip_grads: every tensor times min(1, max_norm / (norm + 1e-6)).
//
// Both stream each gradient once.  A launch takes up to kTensors tensors, cut into runs of kRunBytes; a workgroup finds
// its tensor by binary search in the kernel's arguments.  The squares of a thread are added in fp32 eight at a time and
// then in fp64: fp32 running sums over a run would lose digits against the one rounding of the result, and squares
// past fp32's range (gradients over 1.8e19) would give infinity where the norm is finite.  The runs' sums are added in
// their order by one workgroup, so the norm has the same bits from every call.
#include "rows.h"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 96;         // per launch: 96 * 28 bytes of kernel arguments
constexpr int64_t kRunBytes = 65536;

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

template <class T>
__device__ inline double run_squares(const void* in, int64_t n, int64_t i0, int64_t i1) {
    double s = 0.0;
    const int64_t p1 = i1 / 8;
#pragma unroll 4
    for (int64_t p = i0 / 8 + threadIdx.x; p < p1; p += kThreads) {
        Piece<T> v;
        v.load(in, p);
        float f[8];
        v.to(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += static_cast<double>(f[e]) * static_cast<double>(f[e]);
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(NormList l, double* part) {
    __shared__ double lds[kThreads / 64];
    const int t = tensor_of(l, blockIdx.x);
    const bool f32 = (l.f32[t >> 5] >> (t & 31)) & 1;
    const int64_t run = kRunBytes / (f32 ? 4 : 2);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - l.first[t]) * run;
    const int64_t i1 = min(i0 + run, l.n[t]);
    double s = 0.0;
    int64_t done = i0;
    if ((reinterpret_cast<uintptr_t>(l.in[t]) & 15) == 0) {
        s = f32 ? run_squares<F32>(l.in[t], l.n[t], i0, i1) : run_squares<Bf16>(l.in[t], l.n[t], i0, i1);
        done = i1 / 8 * 8;
        if (done < i0) done = i0;
    }
    for (int64_t i = done + threadIdx.x; i < i1; i += kThreads) {
        const double v = element(l.in[t], f32, i);
        s += v * v;
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void norm_sum_kernel(const double* part, int64_t n, float* norm) {
    __shared__ double lds[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <class T>
__device__ inline void run_scale(const void* in, void* out, int64_t i0, int64_t i1, float coef) {
    const int64_t p1 = i1 / 8;
#pragma unroll 4
    for (int64_t p = i0 / 8 + threadIdx.x; p < p1; p += kThreads) {
        Piece<T> v;
        v.load(in, p);
        float f[8];
        v.to(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= coef;
        v.from(f);
        v.store(out, p);
    }
}

__global__ __launch_bounds__(kThreads) void clip_kernel(NormList l, const float* norm, float max_norm) {
    const float c = max_norm / (*norm + 1e-6f);
    const float coef = c > 1.0f ? 1.0f : c;  // NaN stays NaN
    const int t = tensor_of(l, blockIdx.x);
    if (coef == 1.0f && l.in[t] == l.out[t]) return;  // in place and nothing to clip
    const bool f32 = (l.f32[t >> 5] >> (t & 31)) & 1;
    const int64_t run = kRunBytes / (f32 ? 4 : 2);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - l.first[t]) * run;
    const int64_t i1 = min(i0 + run, l.n[t]);
    int64_t done = i0;
    if (((reinterpret_cast<uintptr_t>(l.in[t]) | reinterpret_cast<uintptr_t>(l.out[t])) & 15) == 0) {
        if (f32) run_scale<F32>(l.in[t], l.out[t], i0, i1, coef);
        else run_scale<Bf16>(l.in[t], l.out[t], i0, i1, coef);
        done = i1 / 8 * 8;
        if (done < i0) done = i0;
    }
    for (int64_t i = done + threadIdx.x; i < i1; i += kThreads) {
        const float v = element(l.in[t], f32, i) * coef;
        if (f32) {
            static_cast<float*>(l.out[t])[i] = v;
        } else {
            const __bf16 b = static_cast<__bf16>(v);
            static_cast<uint16_t*>(l.out[t])[i] = __builtin_bit_cast(uint16_t, b);
        }
    }
}

int64_t runs_of(int64_t n, int32_t dtype) {
    const int64_t run = kRunBytes / (dtype == ENGRAM_F32 ? 4 : 2);
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

// The tensors in lists of kTensors, each with its workgroups; `launch(list, blocks, runs before)`.
template <class F>
void for_lists(int32_t tensors, const void* const* in, void* const* out, const int64_t* n, const int32_t* dtype,
               F&& launch) {
    NormList l = {};
    int64_t blocks = 0, before = 0;
    auto flush = [&]() {
        if (l.tensors) launch(l, static_cast<unsigned>(blocks), before);
        before += blocks;
        l = NormList{};
        blocks = 0;
    };
    for (int i = 0; i < tensors; ++i) {
        if (n[i] == 0) continue;
        const int64_t r = runs_of(n[i], dtype[i]);
        if (l.tensors == kTensors || blocks + r > 0x7FFFFFFF) flush();
        const int at = l.tensors++;
        l.in[at] = in[i];
        l.out[at] = out ? out[i] : nullptr;
        l.n[at] = n[i];
        l.first[at] = static_cast<uint32_t>(blocks);
        if (dtype[i] == ENGRAM_F32) l.f32[at >> 5] |= 1u << (at & 31);
        blocks += r;
    }
    flush();
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" int64_t engram_grad_norm_workspace_bytes(int32_t tensors, const int64_t* n, const int32_t* dtype) {
    if (tensors < 0 || (tensors > 0 && (!n || !dtype))) return -1;
    int64_t runs = 0;
    for (int i = 0; i < tensors; ++i) {
        if (!known_dtype(dtype[i]) || n[i] < 0 || n[i] > (1ll << 40)) return -1;
        runs += runs_of(n[i], dtype[i]);
    }
    return runs * 8;
}

extern "C" int engram_grad_norm(int32_t tensors, const void* const* grads, const int64_t* n, const int32_t* dtype,
                                float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* what = "engram_grad_norm";
    const int rc = check_list(what, tensors, grads, n, dtype);
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
    for_lists(tensors, grads, nullptr, n, dtype, [&](const NormList& l, unsigned blocks, int64_t before) {
        hipLaunchKernelGGL(norm_kernel, dim3(blocks), dim3(kThreads), 0, s, l, part + before);
    });
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
    for_lists(tensors, grads, out, n, dtype, [&](const NormList& l, unsigned blocks, int64_t) {
        hipLaunchKernelGGL(clip_kernel, dim3(blocks), dim3(kThreads), 0, s, l, norm, max_norm);
    });
    return check_launch(what);
}
