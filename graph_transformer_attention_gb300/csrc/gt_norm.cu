// gt_norm.cu -- LayerNorm over the features of a node at any width, forward and
// backward (the fused encoder layer of gt_layer.cu has its own, at width 64).
//
//   forward   mu = mean_j x_j, r = 1 / sqrt(mean_j (x_j - mu)^2 + eps), xh = (x - mu) r
//             y = gain xh + shift
//   backward  d = gain dy;  dx = r (d - mean d - xh mean(d xh)) [+ dres]
//             dgain = sum over rows of dy xh,  dshift = sum over rows of dy
//
// Bandwidth is the bound: every element is read once and written once.  A row
// stays in registers from its load to its store (mean, then centred squares: two
// passes over registers, one over memory), TPR threads per row and 8 NV
// consecutive-in-eights elements per thread.  Statistics and sums are fp32.
// Rows go to threads by width: 8 threads hold rows of up to 64 features (four
// rows to a warp), a warp rows of up to 1024, a CTA of 256 or 512 threads wider ones.
// In the backward a thread keeps the gradient sums of its columns in registers
// over all its rows; a CTA adds its row groups' sums in shared memory and stores
// one partial row, and a second kernel adds the partial rows in a fixed order
// (no atomics: the same result on every run).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "gt_common.cuh"
#include "gt_stats.cuh"
#include "gt_vec8.cuh"

namespace gt {
namespace {

constexpr int kNormMaxC = 16384;

// Sum of v over the TPR threads of a row, in each of them.  Row groups wider
// than a warp are the whole CTA: `red` holds one value per warp, two buffers in
// turn so that one barrier per sum suffices.
template <int TPR>
struct RowSum {
    float2* red;   // [2][TPR / 32] (TPR > 32)
    int k;
    __device__ __forceinline__ float2 operator()(float2 v) {
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if constexpr (TPR > 32) {
            float2* b = red + (k & 1) * (TPR / 32);
            ++k;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
            __syncthreads();
            v = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) {
                v.x += b[w].x;
                v.y += b[w].y;
            }
        }
        return v;
    }
};

template <int TPR>
constexpr int norm_threads() { return TPR > 256 ? TPR : 256; }

template <typename TX, typename TY, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads<TPR>())
norm_fwd(int64_t n, int c, const TX* __restrict__ x, int64_t ldx, const float* __restrict__ gain,
         const float* __restrict__ shift, float eps, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
         float* __restrict__ rstd, bool vec) {
    constexpr int RG = norm_threads<TPR>() / TPR;
    __shared__ float2 red[TPR > 32 ? 2 * (TPR / 32) : 1];
    RowSum<TPR> rowsum{red, 0};
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const float inv_c = 1.0f / (float)c;
    // every thread of a CTA makes the same number of turns (the sums' barriers and shuffles)
    for (int64_t r0 = (int64_t)blockIdx.x * RG; r0 < n; r0 += (int64_t)gridDim.x * RG) {
        const int64_t row = r0 + g;
        const bool live = row < n;
        Raw8<TX> raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
            raw[i] = load8(x + (live ? row : 0) * ldx + col, live ? c - col : 0, vec);
        }
        float v[NV][8], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack8(raw[i], v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        }
        const float mu = rowsum(make_float2(s, 0.f)).x * inv_c;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mu;
                if (col + j < c) q = fmaf(v[i][j], v[i][j], q);
            }
        }
        const float r = 1.0f / sqrtf(rowsum(make_float2(q, 0.f)).x * inv_c + eps);
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + t) * 8;
                if (col >= c) continue;
                float gv[8], sv[8];
                unpack8(load8(gain + col, c - col, vec), gv);
                unpack8(load8(shift + col, c - col, vec), sv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * r, gv[j], sv[j]);
                store8(y + row * ldy + col, v[i], c - col, vec);
            }
            if (t == 0) {
                mean[row] = mu;
                rstd[row] = r;
            }
        }
    }
}

template <typename TX, typename TY, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads<TPR>())
norm_bwd(int64_t n, int c, const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx,
         const float* __restrict__ gain, const float* __restrict__ mean, const float* __restrict__ rstd,
         const TX* __restrict__ dres, int64_t ldr, TX* __restrict__ dx, int64_t lddx, float* __restrict__ part,
         bool vec) {
    constexpr int TH = norm_threads<TPR>(), RG = TH / TPR;
    __shared__ float2 red[TPR > 32 ? 2 * (TPR / 32) : 1];
    RowSum<TPR> rowsum{red, 0};
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const float inv_c = 1.0f / (float)c;
    float ag[NV][8], as[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ag[i][j] = as[i][j] = 0.f;
    for (int64_t r0 = (int64_t)blockIdx.x * RG; r0 < n; r0 += (int64_t)gridDim.x * RG) {
        const int64_t row = r0 + g, rr = row < n ? row : 0;
        const bool live = row < n;
        Raw8<TX> rx[NV];
        Raw8<TY> rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
            rx[i] = load8(x + rr * ldx + col, live ? c - col : 0, vec);
            rd[i] = load8(dy + rr * lddy + col, live ? c - col : 0, vec);
        }
        const float mu = mean[rr], r = rstd[rr];
        float xh[NV][8], d[NV][8], m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
            float gv[8];
            unpack8(load8(gain + col, c - col, vec), gv);
            unpack8(rx[i], xh[i]);
            unpack8(rd[i], d[i]);
            // a dead column or row has dy = 0, and its xh must not bring a NaN into the sums
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] = live && col + j < c ? (xh[i][j] - mu) * r : 0.f;
                ag[i][j] = fmaf(d[i][j], xh[i][j], ag[i][j]);
                as[i][j] += d[i][j];
                d[i][j] *= gv[j];
                m1 += d[i][j];
                m2 = fmaf(d[i][j], xh[i][j], m2);
            }
        }
        const float2 m = rowsum(make_float2(m1, m2));
        m1 = m.x * inv_c;
        m2 = m.y * inv_c;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + t) * 8;
                if (col >= c) continue;
                float o[8];
                if (dres) unpack8(load8(dres + row * ldr + col, c - col, vec), o);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(r, d[i][j] - m1 - xh[i][j] * m2, o[j]);
                store8(dx + row * lddx + col, o, c - col, vec);
            }
        }
    }
    // this CTA's partial row [2][c]: dgain sums, then dshift sums
    float* pr = part + (int64_t)blockIdx.x * 2 * c;
    if constexpr (RG == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
            if (col >= c) continue;
            store8(pr + col, ag[i], c - col, false);
            store8(pr + c + col, as[i], c - col, false);
        }
    } else {
        constexpr int W = TPR * 8;            // columns of one turn
        __shared__ float sum[RG][W + 4];
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) {
            float(&a)[8] = i < NV ? ag[i % NV] : as[i % NV];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[g][t * 8 + j] = a[j];
            __syncthreads();
            for (int k = threadIdx.x; k < W; k += TH) {
                const int col = (i % NV) * W + k;
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < RG; ++q) v += sum[q][k];
                if (col < c) pr[(i < NV ? 0 : c) + col] = v;
            }
        }
    }
}

// One CTA per 32 columns: warp w adds partial rows w, w + 8, ... (coalesced along
// the columns), then warp 0 adds the 8 warp sums.
__global__ void __launch_bounds__(256) col_sum(const float* __restrict__ part, int rows, int cols,
                                               float* __restrict__ out0, int split, float* __restrict__ out1) {
    __shared__ float red[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + tx;
    float acc = 0.f;
    if (i < cols) {
#pragma unroll 8
        for (int p = ty; p < rows; p += 8) acc += part[(int64_t)p * cols + i];
    }
    red[ty][tx] = acc;
    __syncthreads();
    if (ty == 0 && i < cols) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) sum += red[r][tx];
        if (i < split) out0[i] = sum;
        else out1[i - split] = sum;
    }
}

// Threads per row and eights per thread of rows with c features.
struct NormShape {
    int tpr, nv;
};

NormShape norm_shape(int c) {
    if (c <= 64) return {8, 1};
    if (c <= 256) return {32, 1};
    if (c <= 512) return {32, 2};
    if (c <= 1024) return {32, 4};
    if (c <= 2048) return {256, 1};
    if (c <= 4096) return {512, 1};
    if (c <= 8192) return {512, 2};
    return {512, 4};
}

int norm_rows_per_cta(int c) {
    const int tpr = norm_shape(c).tpr;
    return tpr >= 256 ? 1 : 256 / tpr;
}

// CTAs of the backward: two resident per SM make one partial row each.
int norm_bwd_ctas(int64_t n, int c) {
    const int rg = norm_rows_per_cta(c);
    const int64_t want = (n + rg - 1) / rg, most = 2 * (int64_t)num_sms();
    return (int)(want < most ? want : most);
}

template <typename F>
int norm_dispatch(int c, F&& f) {
    const NormShape s = norm_shape(c);
    if (s.tpr == 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (s.tpr == 32 && s.nv == 1) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (s.tpr == 32 && s.nv == 2) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
    if (s.tpr == 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
    if (s.tpr == 256) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    if (s.nv == 1) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 1>());
    if (s.nv == 2) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
}

bool valid_type(int t) { return t == GT_F32 || t == GT_BF16; }

template <typename TX, typename TY>
int run_fwd(int64_t n, int c, const void* x, int64_t ldx, const float* gain, const float* shift, float eps, void* y,
            int64_t ldy, float* mean, float* rstd, cudaStream_t s) {
    const bool vec = rows16(x, ldx, sizeof(TX)) && rows16(y, ldy, sizeof(TY)) && aligned16(gain) && aligned16(shift);
    return norm_dispatch(c, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, TH = norm_threads<TPR>();
        constexpr int64_t RG = TH / TPR;
        const int64_t want = (n + RG - 1) / RG, most = 16 * (int64_t)num_sms();
        LaunchScope ls("norm_fwd", s);
        norm_fwd<TX, TY, TPR, NV><<<(int)(want < most ? want : most), TH, 0, s>>>(
            n, c, static_cast<const TX*>(x), ldx, gain, shift, eps, static_cast<TY*>(y), ldy, mean, rstd, vec);
        return check_launch();
    });
}

template <typename TX, typename TY>
int run_bwd(int64_t n, int c, const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* gain,
            const float* mean, const float* rstd, const void* dres, int64_t ldr, void* dx, int64_t lddx, float* part,
            cudaStream_t s) {
    const bool vec = rows16(x, ldx, sizeof(TX)) && rows16(dy, lddy, sizeof(TY)) && rows16(dx, lddx, sizeof(TX)) &&
                     (!dres || rows16(dres, ldr, sizeof(TX))) && aligned16(gain);
    return norm_dispatch(c, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, TH = norm_threads<TPR>();
        LaunchScope ls("norm_bwd", s);
        norm_bwd<TX, TY, TPR, NV><<<norm_bwd_ctas(n, c), TH, 0, s>>>(
            n, c, static_cast<const TY*>(dy), lddy, static_cast<const TX*>(x), ldx, gain, mean, rstd,
            static_cast<const TX*>(dres), ldr, static_cast<TX*>(dx), lddx, part, vec);
        return check_launch();
    });
}

int check_norm(int xt, int yt, int64_t n, int c) {
    if (!valid_type(xt) || !valid_type(yt) || n < 1 || c < 1) return GT_ERR_INVALID_ARG;
    if (c > kNormMaxC) return GT_ERR_UNSUPPORTED;
    return GT_OK;
}

}  // namespace

int launch_col_sum(const char* name, const float* part, int rows, int cols, float* out0, int split, float* out1,
                   cudaStream_t s) {
    LaunchScope ls(name, s);
    col_sum<<<(cols + 31) / 32, 256, 0, s>>>(part, rows, cols, out0, split, out1);
    return check_launch();
}

}  // namespace gt

extern "C" {

size_t gt_layer_norm_workspace_size(int32_t n, int32_t c) {
    if (gt::check_norm(GT_F32, GT_F32, n, c) != GT_OK) return 0;
    return (size_t)gt::norm_bwd_ctas(n, c) * 2 * c * sizeof(float) + 256;
}

int gt_layer_norm_fwd(int32_t xtype, int32_t ytype, int32_t n, int32_t c, const void* x, int64_t ldx,
                      const float* gain, const float* shift, float eps, void* y, int64_t ldy, float* mean,
                      float* rstd, void* stream) {
    using namespace gt;
    const int rc = check_norm(xtype, ytype, n, c);
    if (rc != GT_OK) return rc;
    if (!x || !gain || !shift || !y || !mean || !rstd || ldx < c || ldy < c) return GT_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !isfinite(eps)) return GT_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    if (xtype == GT_F32)
        return ytype == GT_F32 ? run_fwd<float, float>(n, c, x, ldx, gain, shift, eps, y, ldy, mean, rstd, s)
                               : run_fwd<float, B>(n, c, x, ldx, gain, shift, eps, y, ldy, mean, rstd, s);
    return ytype == GT_F32 ? run_fwd<B, float>(n, c, x, ldx, gain, shift, eps, y, ldy, mean, rstd, s)
                           : run_fwd<B, B>(n, c, x, ldx, gain, shift, eps, y, ldy, mean, rstd, s);
}

int gt_layer_norm_bwd(int32_t xtype, int32_t ytype, int32_t n, int32_t c, const void* dy, int64_t lddy,
                      const void* x, int64_t ldx, const float* gain, const float* mean, const float* rstd,
                      const void* dres, int64_t ldr, void* dx, int64_t lddx, float* dgain, float* dshift,
                      void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt;
    int rc = check_norm(xtype, ytype, n, c);
    if (rc != GT_OK) return rc;
    if (!dy || !x || !gain || !mean || !rstd || !dx || !dgain || !dshift) return GT_ERR_INVALID_ARG;
    if (lddy < c || ldx < c || lddx < c || (dres && ldr < c)) return GT_ERR_INVALID_ARG;
    const int ctas = norm_bwd_ctas(n, c);
    Carve cv(workspace, ws_bytes);
    float* part = cv.take<float>((size_t)ctas * 2 * c);
    if (!workspace || !aligned16(workspace) || !cv.fits()) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    if (xtype == GT_F32)
        rc = ytype == GT_F32
                 ? run_bwd<float, float>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, s)
                 : run_bwd<float, B>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, s);
    else
        rc = ytype == GT_F32
                 ? run_bwd<B, float>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, s)
                 : run_bwd<B, B>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, s);
    if (rc != GT_OK) return rc;
    return launch_col_sum("norm_grad_sum", part, ctas, 2 * c, dgain, c, dshift, s);
}

}  // extern "C"
