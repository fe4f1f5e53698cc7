// gt_grad_clip.cu -- the norm of all gradients together, and each of them scaled so that it
// does not exceed a limit:  norm = sqrt(sum over all tensors of g^2),
// out = g * (norm <= max_norm ? 1 : max_norm / norm).
//
// The bytes bound it: every gradient is read for the norm, then read again and written (8 layers of width 2048, 403
// million fp32: 745 us, 6.5 TB/s of three passes; 812 with 16-byte accesses).  Two kernels over a table of the tensors in
// the launch's own arguments (nothing is copied to the device, so a captured graph holds it): the warps take units of
// kUnit elements, whichever tensor they fall into, so that hundreds of small tensors and a few large ones fill the SMs
// alike.  The second kernel takes the units in the opposite order: what the first read last is still cached.
//
// Squares of fp32 leave the range of fp32: a unit's sum of squares outside [2^-90, 2^100] is taken again in fp64 (a
// lane's 32 squares below 2^-149 lose less than 2^-53 of a sum above 2^-90).  A lane's units are added in two fp32 words
// (the rounding of each addition is kept), everything above in fp64, in a fixed order.  A factor below 2^-126 multiplies in
// fp64 as well.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "gt_common.cuh"
#include "gt_sm100.cuh"
#include "gt_stats.cuh"
#include "gt_vec8.cuh"

namespace gt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 1024;          // elements a warp takes at a time, all on their way at once
constexpr int kEights = kUnit / 256;  // eights of a lane
constexpr int kTable = 256;          // tensors of a launch

struct Entry {
    const void* g;
    void* out;          // NULL: the tensor only counts
    int64_t numel;
    int32_t unit0;      // units before it
    int8_t g32, o32;    // fp32, else bf16
    int8_t gvec, ovec;  // accesses: 2 by 32 bytes, 1 by 16, 0 by single elements
};

struct Table {
    Entry e[kTable];
    int count;
    int units;
};

// The tensor that unit u falls into: the last whose first unit is not past u.
__device__ __forceinline__ int tensor_of(const int* first, int count, int u) {
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Eight elements of a lane: whole units of 16-byte rows as vectors, lane by lane; others element by element.
template <typename T>
__device__ __forceinline__ void get8(const T* p, int live, int vec, float (&v)[8]) {
    unpack8(load8<Mem::kOutput>(p, live, vec), v);
}

// The element of a unit where lane `lane` starts its eighth k
__device__ __forceinline__ int at_of(int k, int lane) { return k * 256 + lane * 8; }

template <typename T>
__device__ __forceinline__ float unit_squares(const T* p, int64_t left, int vec, int lane, double& wide) {
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    float v[kEights][8];
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
        const int at = at_of(k, lane);
        const int64_t more = left - at;
        get8(p + at, more >= 8 ? 8 : more > 0 ? (int)more : 0, vec, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kEights; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) part[i & 3] = fmaf(v[k][i], v[k][i], part[i & 3]);
    const float s = (part[0] + part[1]) + (part[2] + part[3]);
    if (s >= 0x1p-90f && s <= 0x1p100f) return s;
    // out of fp32's range, zero or not finite
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= __float_as_uint(v[k][i]) << 1;
        if (any) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d += (double)v[k][i] * (double)v[k][i];
        }
    }
    wide += d;
    return 0.f;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += red[w];
    return t;
}

// part[CTA] = its units' sum of squares
__global__ void __launch_bounds__(kThreads) grad_squares(const __grid_constant__ Table T, double* __restrict__ part) {
    __shared__ int first[kTable];
    __shared__ double red[kWarps];
    for (int k = threadIdx.x; k < T.count; k += kThreads) first[k] = T.e[k].unit0;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    float hi = 0.f, lo = 0.f;
    double wide = 0.0;
    for (int u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < T.units; u += gridDim.x * kWarps) {
        const int k = tensor_of(first, T.count, u);
        const Entry& e = T.e[k];
        const int64_t at = (int64_t)(u - first[k]) * kUnit;
        const float s = e.g32 ? unit_squares(static_cast<const float*>(e.g) + at, e.numel - at, e.gvec, lane, wide)
                              : unit_squares(static_cast<const __nv_bfloat16*>(e.g) + at, e.numel - at, e.gvec, lane, wide);
        // hi + s exactly as a sum and its rounding (Knuth's two-sum)
        const float t = __fadd_rn(hi, s), z = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(s, z)));
        hi = t;
    }
    sm100::pdl_trigger();
    const double sum = block_sum((double)hi + (double)lo + wide, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// out = factor g.  Every CTA adds the same partial sums in the same order.
__global__ void __launch_bounds__(kThreads) grad_scale(const __grid_constant__ Table T, const double* __restrict__ part,
                                                       int parts, float max_norm, float* __restrict__ norm_out) {
    __shared__ int first[kTable];
    __shared__ double red[kWarps];
    for (int k = threadIdx.x; k < T.count; k += kThreads) first[k] = T.e[k].unit0;
    sm100::pdl_wait();   // launched to overlap the end of the kernel that writes the partial sums
    double sum = 0.0;
    for (int k = threadIdx.x; k < parts; k += 4 * kThreads) {      // four loads on their way
        double x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = k + u * kThreads < parts ? __ldcg(part + k + u * kThreads) : 0.0;
#pragma unroll
        for (int u = 0; u < 4; ++u) sum += x[u];
    }
    const double norm = sqrt(block_sum(sum, red));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    // (a NaN norm makes every result NaN, unless there is no limit)
    const bool as_is = norm <= (double)max_norm || isinf(max_norm);
    const double quotient = (double)max_norm / norm;
    const float factor = as_is ? 1.f : (float)quotient;
    // fp32 has fewer digits of a quotient below 2^-126, or none, though the products may be ordinary numbers: these are
    // formed in fp64
    const bool small = !as_is && quotient < 0x1p-126 && quotient > 0.0;
    const int lane = threadIdx.x & 31;
    for (int w = blockIdx.x * kWarps + (threadIdx.x >> 5); w < T.units; w += gridDim.x * kWarps) {
        const int u = T.units - 1 - w;
        const int k = tensor_of(first, T.count, u);
        const Entry& e = T.e[k];
        if (!e.out || (as_is && e.out == e.g)) continue;
        const int64_t at = (int64_t)(u - first[k]) * kUnit, left = e.numel - at;
        auto scale = [&](const auto* g, auto* out) {
            float v[kEights][8];
#pragma unroll
            for (int j = 0; j < kEights; ++j) {
                const int a = at_of(j, lane);
                const int64_t more = left - a;
                get8(g + at + a, more >= 8 ? 8 : more > 0 ? (int)more : 0, e.gvec, v[j]);
            }
#pragma unroll
            for (int j = 0; j < kEights; ++j) {
                const int a = at_of(j, lane);
                const int64_t more = left - a;
                if (small)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = (float)((double)v[j][i] * quotient);
                else if (!as_is)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] *= factor;
                store8(out + at + a, v[j], more >= 8 ? 8 : more > 0 ? (int)more : 0, e.ovec);
            }
        };
        if (e.g32) {
            if (e.o32) scale(static_cast<const float*>(e.g), static_cast<float*>(e.out));
            else scale(static_cast<const float*>(e.g), static_cast<__nv_bfloat16*>(e.out));
        } else {
            if (e.o32) scale(static_cast<const __nv_bfloat16*>(e.g), static_cast<float*>(e.out));
            else scale(static_cast<const __nv_bfloat16*>(e.g), static_cast<__nv_bfloat16*>(e.out));
        }
    }
}

// CTAs of a launch at most: those that are resident at once
int most_ctas() { return 4 * num_sms(); }

int64_t units_of(int64_t numel) { return (numel + kUnit - 1) / kUnit; }

// CTAs of the launch over list[at .. at + kTable - 1]
int ctas_of(const gt_grad* list, int count, int at) {
    int64_t units = 0;
    for (int k = at; k < std::min(count, at + kTable); ++k) units += units_of(list[k].numel);
    return (int)std::max<int64_t>(1, std::min<int64_t>((units + kWarps - 1) / kWarps, most_ctas()));
}

bool valid_type(int t) { return t == GT_F32 || t == GT_BF16; }

int check(const gt_grad* list, int count) {
    if (!list || count < 1) return GT_ERR_INVALID_ARG;
    for (int k = 0; k < count; ++k) {
        const gt_grad& g = list[k];
        if (g.numel < 0 || (g.numel > 0 && !g.g) || !valid_type(g.gtype) || (g.out && !valid_type(g.otype)))
            return GT_ERR_INVALID_ARG;
        if (g.out == g.g && g.out && g.otype != g.gtype) return GT_ERR_INVALID_ARG;
        if (g.numel > ((int64_t)1 << 40)) return GT_ERR_UNSUPPORTED;
    }
    for (int at = 0; at < count; at += kTable) {
        int64_t units = 0;
        for (int k = at; k < std::min(count, at + kTable); ++k) units += units_of(list[k].numel);
        if (units > (int64_t)1 << 30) return GT_ERR_UNSUPPORTED;
    }
    return GT_OK;
}

void fill(Table& t, const gt_grad* list, int count, int at) {
    t.count = std::min(count - at, kTable);
    int units = 0;
    for (int k = 0; k < t.count; ++k) {
        const gt_grad& g = list[at + k];
        t.e[k] = Entry{g.g, g.out, g.numel, units, g.gtype == GT_F32, g.otype == GT_F32,
                       (int8_t)row_access(g.g, 0, 4), (int8_t)row_access(g.out, 0, 4)};
        units += (int)units_of(g.numel);
    }
    t.units = units;
}

}  // namespace
}  // namespace gt

extern "C" {

size_t gt_grad_clip_workspace_size(int32_t count) {
    return count < 1 ? 0 : (size_t)((count + gt::kTable - 1) / gt::kTable) * gt::most_ctas() * sizeof(double) + 256;
}

int gt_grad_clip(const gt_grad* list, int32_t count, float max_norm, float* norm, void* workspace, size_t ws_bytes,
                 void* stream) {
    using namespace gt;
    int rc = check(list, count);
    if (rc != GT_OK) return rc;
    if (!norm || !(max_norm >= 0.f)) return GT_ERR_INVALID_ARG;
    int parts = 0;
    for (int at = 0; at < count; at += kTable) parts += ctas_of(list, count, at);
    Carve cv(workspace, ws_bytes);
    double* part = cv.take<double>(parts);
    if (!workspace || !aligned16(workspace) || !cv.fits()) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Table t;
    int done = 0;
    for (int at = 0; at < count; at += kTable) {
        fill(t, list, count, at);
        const int ctas = ctas_of(list, count, at);
        LaunchScope ls("grad_squares", s);
        grad_squares<<<ctas, kThreads, 0, s>>>(t, part + done);
        rc = check_launch();
        if (rc != GT_OK) return rc;
        done += ctas;
    }
    for (int at = 0; at < count; at += kTable) {
        fill(t, list, count, at);
        const int ctas = ctas_of(list, count, at);
        LaunchScope ls("grad_scale", s);
        // (the first overlaps the end of the last grad_squares; the others only follow one another)
        if (launch_overlapped(grad_scale, dim3(ctas), dim3(kThreads), 0, s, t, (const double*)part, parts, max_norm,
                              at == 0 ? norm : (float*)nullptr) != cudaSuccess)
            return GT_ERR_CUDA;
    }
    return GT_OK;
}

}  // extern "C"
