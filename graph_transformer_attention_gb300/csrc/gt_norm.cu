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
// passes over registers, one over memory), eight elements to a thread, and a
// thread has several rows in flight.  Statistics and sums are fp32.
// In the backward a thread keeps the gradient sums of its eight columns in registers
// over all its rows; a CTA adds its row groups' sums in shared memory and stores
// one partial row, and a second kernel adds the partial rows in a fixed order
// (no atomics: the same result on every run).
//
// Measured (one GB300, inputs larger than the L2; share of the copy rate, 6.79 TB/s): forward 32768 x 1024
// fp32 to bf16 34 us (87 %), bf16 26.4 us (75 %), bf16 to fp32 39.5 us (75 %); backward with dres 32768 x 1024 bf16 48 us (82 %),
// x fp32 and dy bf16 73.5 us (94 %), 16384 x 4096 bf16 93 us (85 %), 65536 x 512 fp32 82 us (97 %); small inputs are latency:
// 6800 x 64 fp32 3.0 us and 5.2 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gt_common.cuh"
#include "gt_sm100.cuh"
#include "gt_stats.cuh"
#include "gt_vec8.cuh"

namespace gt {
namespace {

constexpr int kNormMaxC = 16384;

// Sums of v[i] over the TPR threads of a row group, in each of them.  Row groups wider
// than a warp pass their warps' sums through `red`, two buffers in turn, so that one
// barrier of the CTA per sum suffices.
template <int TPR, int R, int TH>
struct RowSum {
    float2* red;   // [2][TH / 32][R] (TPR > 32)
    int k;
    __device__ __forceinline__ void operator()(float2 (&v)[R]) {
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                v[i].x += __shfl_xor_sync(0xffffffffu, v[i].x, o);
                v[i].y += __shfl_xor_sync(0xffffffffu, v[i].y, o);
            }
        }
        if constexpr (TPR > 32) {
            constexpr int W = TPR / 32;
            float2* b = red + (k & 1) * (TH / 32) * R;
            ++k;
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int i = 0; i < R; ++i) b[warp * R + i] = v[i];
            }
            __syncthreads();
            const float2* g = b + (warp / W) * W * R;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                v[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    v[i].x += g[w * R + i].x;
                    v[i].y += g[w * R + i].y;
                }
            }
        }
    }
};

// A layout of rows over threads: TPR threads hold a row, NV eights of elements each (eight t of
// turn i at column 8 (i TPR + t)); a CTA of TH threads takes R rows per group at a time.
// OCC CTAs are resident on an SM.
template <int TPR_, int NV_, int R_, int OCC_>
struct NormCfg {
    static constexpr int TPR = TPR_, NV = NV_, R = R_, OCC = OCC_;
    static constexpr int TH = TPR > 256 ? TPR : 256, RG = TH / TPR, ROWS = RG * R;
    static constexpr int RED = TPR > 32 ? 2 * (TH / 32) * R : 1;
};

template <typename TX, typename TY, typename C, bool WHOLE>
__global__ void __launch_bounds__(C::TH, C::OCC)
norm_fwd(int64_t n, int c, const TX* __restrict__ x, int64_t ldx, const float* __restrict__ gain,
         const float* __restrict__ shift, float eps, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
         float* __restrict__ rstd, int vec) {
    constexpr int TPR = C::TPR, NV = C::NV, R = C::R, RG = C::RG;
    __shared__ float2 red[C::RED];
    RowSum<TPR, R, C::TH> rowsum{red, 0};
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const float inv_c = 1.0f / (float)c;
    auto fetch = [&](int64_t r0, Raw8<TX> (&raw)[R][NV]) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = r0 + k * RG + g;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + t) * 8;
                raw[k][i] = load8_row<WHOLE>(x + (row < n ? row : 0) * ldx + col, row < n ? c - col : 0, vec);
            }
        }
    };
    // Rows of bf16 are fetched a turn ahead, by as many CTAs as are resident; of fp32, whose rows take twice the
    // registers, more CTAs take turns instead (32768 x 1024: bf16 26 against 31 us; fp32 in and bf16 out 34, and 37 with rows fetched ahead).
    constexpr bool kAhead = sizeof(TX) == 2;
    Raw8<TX> raw[R][NV];
    const int64_t step = (int64_t)gridDim.x * C::ROWS;
    if (kAhead) fetch((int64_t)blockIdx.x * C::ROWS, raw);
    // every thread of a CTA makes the same number of turns (the sums' barriers and shuffles)
    for (int64_t r0 = (int64_t)blockIdx.x * C::ROWS; r0 < n; r0 += step) {
        if (!kAhead) fetch(r0, raw);
        float2 v[R][NV][4], s[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float2 a = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack8(raw[k][i], v[k][i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) a = __fadd2_rn(a, v[k][i][j]);
            }
            s[k] = make_float2(a.x + a.y, 0.f);
        }
        if (kAhead && r0 + step < n) fetch(r0 + step, raw);
        rowsum(s);
        float mu[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mu[k] = s[k].x * inv_c;
            const float2 minus = make_float2(-mu[k], -mu[k]);
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int live = c - (i * TPR + t) * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2& u = v[k][i][j];
                    u = __fadd2_rn(u, minus);
                    if (WHOLE ? live <= 0 : live < 8) {   // columns past the end do not count
                        if (2 * j >= live) u.x = 0.f;
                        if (2 * j + 1 >= live) u.y = 0.f;
                    }
                    q = __ffma2_rn(u, u, q);
                }
            }
            s[k] = make_float2(q.x + q.y, 0.f);
        }
        rowsum(s);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            s[k].x = 1.0f / sqrtf(s[k].x * inv_c + eps);
            const int64_t row = r0 + k * RG + g;
            if (t == 0 && row < n) {
                mean[row] = mu[k];
                rstd[row] = s[k].x;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * TPR + t) * 8;
            if (col >= c) continue;
            float2 gv[4], sv[4];
            unpack8(load8_row<WHOLE>(gain + col, c - col, vec), gv);
            unpack8(load8_row<WHOLE>(shift + col, c - col, vec), sv);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = r0 + k * RG + g;
                if (row >= n) continue;
                const float2 r = make_float2(s[k].x, s[k].x);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = __ffma2_rn(__fmul2_rn(v[k][i][j], r), gv[j], sv[j]);
                    o[2 * j] = u.x;
                    o[2 * j + 1] = u.y;
                }
                store8(y + row * ldy + col, o, WHOLE ? 8 : c - col, WHOLE ? max(vec, 1) : vec);
            }
        }
    }
}

template <typename TX, typename TY, typename C, bool WHOLE>
__global__ void __launch_bounds__(C::TH, C::OCC)
norm_bwd(int64_t n, int c, const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx,
         const float* __restrict__ gain, const float* __restrict__ mean, const float* __restrict__ rstd,
         const TX* dres, int64_t ldr, TX* dx, int64_t lddx, float* __restrict__ part, int vec) {   // dres may be dx
    constexpr int TPR = C::TPR, NV = C::NV, R = C::R, RG = C::RG, TH = C::TH;
    __shared__ float2 red[C::RED];
    RowSum<TPR, R, TH> rowsum{red, 0};
    sm100::pdl_trigger();   // the column sums may start; they wait for this kernel
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const float inv_c = 1.0f / (float)c;
    float2 ag[NV][4], as[NV][4], gv[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        unpack8(load8_row<WHOLE>(gain + col, c - col, vec), gv[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) ag[i][j] = as[i][j] = make_float2(0.f, 0.f);
    }
    struct Rows {   // the inputs of R rows
        Raw8<TX> x[R][NV], res[R][NV];
        Raw8<TY> dy[R][NV];
        float mu[R], rs[R];
    };
    auto fetch = [&](int64_t r0, Rows& in) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = r0 + k * RG + g, ra = row < n ? row : 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + t) * 8, live = row < n ? c - col : 0;
                in.x[k][i] = load8_row<WHOLE>(x + ra * ldx + col, live, vec);
                in.dy[k][i] = load8_row<WHOLE>(dy + ra * lddy + col, live, vec);
                if (dres) in.res[k][i] = load8_row<WHOLE, Mem::kOutput>(dres + ra * ldr + col, live, vec);
            }
            // a row past the end is all zeros, and so are its xh and its sums
            in.mu[k] = row < n ? mean[ra] : 0.f;
            in.rs[k] = row < n ? rstd[ra] : 0.f;
        }
    };
    // The next rows are on their way while these are computed, where the registers hold both (with them ahead and without:
    // 8192 x 4096 bf16 46.5 and 64 us, fp32 77 and 107; 4096 x 8192 bf16 61 and 71, fp32, which spills then, 109 and 90;
    // 2048 x 16384 bf16 150 and 113).
    constexpr bool kAhead = TPR * NV * sizeof(TX) <= 2048;
    Rows next;
    const int64_t step = (int64_t)gridDim.x * C::ROWS;
    if (kAhead) fetch((int64_t)blockIdx.x * C::ROWS, next);
    for (int64_t r0 = (int64_t)blockIdx.x * C::ROWS; r0 < n; r0 += step) {
        if (!kAhead) fetch(r0, next);
        const Rows in = next;
        if (kAhead && r0 + step < n) fetch(r0 + step, next);
        // A column past the end has x = dy = 0: it adds nothing to the row's sums (or NaN to a row whose
        // statistics are NaN), and its own sums are not stored.
        auto xhat = [&](int k, float2 x2) {
            return __fmul2_rn(__fadd2_rn(x2, make_float2(-in.mu[k], -in.mu[k])), make_float2(in.rs[k], in.rs[k]));
        };
        float2 m[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float2 m1 = make_float2(0.f, 0.f), m2 = m1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 xv[4], d[4];
                unpack8(in.x[k][i], xv);
                unpack8(in.dy[k][i], d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 xh = xhat(k, xv[j]), dg = __fmul2_rn(d[j], gv[i][j]);
                    ag[i][j] = __ffma2_rn(d[j], xh, ag[i][j]);
                    as[i][j] = __fadd2_rn(as[i][j], d[j]);
                    m1 = __fadd2_rn(m1, dg);
                    m2 = __ffma2_rn(dg, xh, m2);
                }
            }
            m[k] = make_float2(m1.x + m1.y, m2.x + m2.y);
        }
        rowsum(m);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = r0 + k * RG + g;
            const float2 m1 = make_float2(-m[k].x * inv_c, -m[k].x * inv_c), m2 = make_float2(-m[k].y * inv_c, -m[k].y * inv_c);
            const float2 rs = make_float2(in.rs[k], in.rs[k]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * TPR + t) * 8;
                if (row >= n || col >= c) continue;
                float2 xv[4], d[4], o[4] = {};
                unpack8(in.x[k][i], xv);
                unpack8(in.dy[k][i], d);
                if (dres) unpack8(in.res[k][i], o);
                float out[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = __ffma2_rn(xhat(k, xv[j]), m2, __ffma2_rn(d[j], gv[i][j], m1));
                    const float2 w = __ffma2_rn(rs, u, o[j]);
                    out[2 * j] = w.x;
                    out[2 * j + 1] = w.y;
                }
                store8(dx + row * lddx + col, out, WHOLE ? 8 : c - col, WHOLE ? max(vec, 1) : vec);
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
            float u[8], w[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u[2 * j] = ag[i][j].x; u[2 * j + 1] = ag[i][j].y;
                w[2 * j] = as[i][j].x; w[2 * j + 1] = as[i][j].y;
            }
            store8(pr + col, u, c - col, 0);
            store8(pr + c + col, w, c - col, 0);
        }
    } else {
        constexpr int W = TPR * 8;            // columns of one turn
        __shared__ float sum[RG][W + 4];
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) {
            const float2(&a)[4] = i < NV ? ag[i % NV] : as[i % NV];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[g][t * 8 + 2 * j] = a[j].x;
                sum[g][t * 8 + 2 * j + 1] = a[j].y;
            }
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

// One CTA per 32 columns: warp w adds partial rows w, w + 32, ... (coalesced along
// the columns), then warp 0 adds the 32 warp sums.
constexpr int kColSumThreads = 1024;
__global__ void __launch_bounds__(kColSumThreads) col_sum(const float* __restrict__ part, int rows, int cols,
                                                          float* __restrict__ out0, int split, float* __restrict__ out1) {
    __shared__ float red[kColSumThreads / 32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + tx;
    float acc = 0.f;
    sm100::pdl_wait();   // launched to overlap the end of the kernel that writes `part`
    if (i < cols) {
#pragma unroll 8
        for (int p = ty; p < rows; p += kColSumThreads / 32) acc += __ldcg(part + (int64_t)p * cols + i);
    }
    red[ty][tx] = acc;
    __syncthreads();
    if (ty == 0 && i < cols) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kColSumThreads / 32; ++r) sum += red[r][tx];
        if (i < split) out0[i] = sum;
        else out1[i - split] = sum;
    }
}

// The forward's layout by width: two eights to a thread, so that a warp holds rows of up to 512 features.  Measured
// with three and four CTAs on an SM: 32768 x 1024 fp32 to bf16 34.1 and 32.5 us, 65536 x 512 fp32 42.2 and 43.0;
// with one row and two rows of 256 threads: 16384 x 4096 bf16 51.1 and 49.5 us, fp32 to bf16 68.7 and 76.0;
// 8192 x 8192 bf16 59 us with 512 threads to a row, 50 with 256.
template <typename TX, typename TY, typename F>
auto fwd_dispatch(int c, F&& f) {
    constexpr bool HALF = sizeof(TX) == 2;
    constexpr int OCC = sizeof(TX) > sizeof(TY) ? 4 : 3;
    if (c <= 64) return f(NormCfg<8, 1, 2, OCC>());
    if (c <= 128) return f(NormCfg<8, 2, 2, OCC>());
    if (c <= 256) return f(NormCfg<16, 2, 2, OCC>());
    if (c <= 512) return f(NormCfg<32, 2, 2, OCC>());
    if (c <= 1024) return f(NormCfg<64, 2, 2, OCC>());
    if (c <= 2048) return f(NormCfg<128, 2, 2, OCC>());
    if (c <= 4096) return f(NormCfg<256, 2, HALF ? 2 : 1, HALF ? 2 : 4>());
    if (c <= 8192) return f(NormCfg<256, 4, 1, 2>());
    return f(NormCfg<512, 4, 1, HALF ? 1 : 2>());
}

// The backward's: one eight to a thread (more from 1024 features on), whose gradient sums stay in registers beside the next rows.
// Rows of bf16 are half as wide in registers, so more of them are on their way.  Measured (share of the copy rate,
// dres with it): 65536 x 512 bf16 64 % with one row of 64 threads and three CTAs, 86 % with two rows and two CTAs
// (fp32 93 and 83 %, with four rows and one CTA 98 %); 16384 x 2048 bf16 63 % with 256 threads to a row, 82 % with
// 128 (fp32 81 and 96 %); 16384 x 4096 bf16 72 % with one row of 512 threads, 86 % with two of 256 (fp32 90 and 74 %).
template <bool HALF, typename F>
auto bwd_dispatch(int c, F&& f) {
    if (c <= 64) return f(NormCfg<8, 1, 2, 2>());
    if (c <= 128) return f(NormCfg<16, 1, 2, 2>());
    if (c <= 256) return f(NormCfg<32, 1, 2, 2>());
    if (c <= 512) return f(NormCfg<64, 1, HALF ? 2 : 4, HALF ? 2 : 1>());
    if (c <= 1024) return f(NormCfg<128, 1, HALF ? 2 : 4, HALF ? 2 : 1>());
    if (c <= 2048) return f(NormCfg<128, 2, 2, 1>());
    if (c <= 4096) return f(NormCfg<HALF ? 256 : 512, HALF ? 2 : 1, HALF ? 2 : 1, 1>());
    if (c <= 8192) return f(NormCfg<256, 4, 1, 1>());
    return f(NormCfg<512, 4, 1, 1>());
}

// CTAs of the backward, each of which makes one partial row: those that are resident at once.
template <bool HALF>
int norm_bwd_ctas(int64_t n, int c) {
    return bwd_dispatch<HALF>(c, [&](auto cfg) {
        using C = decltype(cfg);
        const int64_t want = (n + C::ROWS - 1) / C::ROWS, most = (int64_t)C::OCC * num_sms();
        return (int)(want < most ? want : most);
    });
}

int least(std::initializer_list<int> v) { return std::min(v); }

bool valid_type(int t) { return t == GT_F32 || t == GT_BF16; }

template <typename TX, typename TY>
int run_fwd(int64_t n, int c, const void* x, int64_t ldx, const float* gain, const float* shift, float eps, void* y,
            int64_t ldy, float* mean, float* rstd, cudaStream_t s) {
    const int vec = least({row_access(x, ldx, sizeof(TX)), row_access(y, ldy, sizeof(TY)), row_access(gain, 0, 4),
                           row_access(shift, 0, 4)});
    return fwd_dispatch<TX, TY>(c, [&](auto cfg) {
        using C = decltype(cfg);
        const int64_t want = (n + C::ROWS - 1) / C::ROWS, most = (sizeof(TX) == 2 ? C::OCC : 16) * (int64_t)num_sms();
        LaunchScope ls("norm_fwd", s);
        // rows of whole eights need no bounds inside an eight (16384 x 4096 bf16 51 us, 53 with them)
        auto kern = vec > 0 && c % 8 == 0 ? norm_fwd<TX, TY, C, true> : norm_fwd<TX, TY, C, false>;
        kern<<<(int)(want < most ? want : most), C::TH, 0, s>>>(n, c, static_cast<const TX*>(x), ldx, gain, shift, eps,
                                                                static_cast<TY*>(y), ldy, mean, rstd, vec);
        return check_launch();
    });
}

template <typename TX, typename TY>
int run_bwd(int64_t n, int c, const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* gain,
            const float* mean, const float* rstd, const void* dres, int64_t ldr, void* dx, int64_t lddx, float* part,
            int ctas, cudaStream_t s) {
    const int vec = least({row_access(x, ldx, sizeof(TX)), row_access(dy, lddy, sizeof(TY)),
                           row_access(dx, lddx, sizeof(TX)), row_access(dres, ldr, sizeof(TX)), row_access(gain, 0, 4)});
    return bwd_dispatch<sizeof(TX) == 2>(c, [&](auto cfg) {
        using C = decltype(cfg);
        LaunchScope ls("norm_bwd", s);
        auto kern = vec > 0 && c % 8 == 0 ? norm_bwd<TX, TY, C, true> : norm_bwd<TX, TY, C, false>;
        kern<<<ctas, C::TH, 0, s>>>(
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

int launch_col_sum(const float* part, int rows, int cols, float* out0, int split, float* out1, cudaStream_t s) {
    LaunchScope ls("norm_grad_sum", s);
    if (launch_overlapped(col_sum, dim3((cols + 31) / 32), dim3(kColSumThreads), 0, s, part, rows, cols, out0, split,
                          out1) != cudaSuccess)
        return GT_ERR_CUDA;
    return check_launch();
}

}  // namespace
}  // namespace gt

extern "C" {

size_t gt_layer_norm_workspace_size(int32_t n, int32_t c) {
    if (gt::check_norm(GT_F32, GT_F32, n, c) != GT_OK) return 0;
    return (size_t)std::max(gt::norm_bwd_ctas<false>(n, c), gt::norm_bwd_ctas<true>(n, c)) * 2 * c * sizeof(float) + 256;
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
    const int ctas = xtype == GT_F32 ? norm_bwd_ctas<false>(n, c) : norm_bwd_ctas<true>(n, c);
    Carve cv(workspace, ws_bytes);
    float* part = cv.take<float>((size_t)ctas * 2 * c);
    if (!workspace || !aligned16(workspace) || !cv.fits()) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    if (xtype == GT_F32)
        rc = ytype == GT_F32
                 ? run_bwd<float, float>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, ctas, s)
                 : run_bwd<float, B>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, ctas, s);
    else
        rc = ytype == GT_F32
                 ? run_bwd<B, float>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, ctas, s)
                 : run_bwd<B, B>(n, c, dy, lddy, x, ldx, gain, mean, rstd, dres, ldr, dx, lddx, part, ctas, s);
    if (rc != GT_OK) return rc;
    return launch_col_sum(part, ctas, 2 * c, dgain, c, dshift, s);
}

}  // extern "C"
