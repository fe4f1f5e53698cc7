// gt_linear.cu -- the linear layer y = act(x W + b) + r at any width, forward and
// backward, on the tensor cores (the fused encoder layer of gt_layer.cu has its
// own products, at width 64).
//
//   forward   a = x W + b (kept when asked for), y = act(a) + r
//   backward  da = dy act'(a);  dx = da W^T [+ add];  dW = x^T da;  db = sum over rows of da
//
// One product kernel, D = A B with the contraction in k-blocks of 64, serves all
// three: x W (A rows along the contraction, B columns along the row), da W^T (both
// along the contraction) and x^T da (both along the row).  tcgen05.mma reads bf16
// operands of either direction from shared memory, so no operand is ever
// transposed: only the TMA boxes and the descriptors differ.
//
// fp32 operands: each value is the exact sum of three bf16 values, v = hi + mid +
// lo (8 significand bits each), and a product of two such sums keeps the six terms
// above 2^-24 of the largest:  lo hi, hi lo, mid mid, mid hi, hi mid, hi hi.  They
// run as one contraction six times as long, the smallest terms first, so that they
// are added while the fp32 accumulator is still small.  Six bf16 products cost a
// sixth of the bf16 rate, which is four times what the fp32 pipes reach.
//
// Rows that TMA cannot read (a base or row stride that is no multiple of 16 bytes)
// are first copied to padded rows in the workspace by the kernel that splits fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gt_common.cuh"
#include "gt_sm100.cuh"
#include "gt_stats.cuh"
#include "gt_tc_common.cuh"
#include "gt_tma.cuh"
#include "gt_vec8.cuh"

namespace gt {
namespace {

using namespace sm100;
using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------------ GELU

// exp(-a^2 / 2) and the normal CDF at -|a|, which is half of
// erfc(|a| / sqrt 2) = t (a1 + a2 t + ... + a5 t^4) exp(-a^2 / 2), t = 1 / (1 + p |a| / sqrt 2),
// Abramowitz and Stegun 7.1.26: at most 1.5e-7 off, the size of an fp32 rounding of the CDF.
__device__ __forceinline__ void gauss(float a, float& e, float& tail) {
    const float z = fabsf(a) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, z, 1.0f));
    e = ex2(a * a * (-0.5f * tc::kLog2e));
    float s = fmaf(t, 1.061405429f, -1.453152027f);
    s = fmaf(t, s, 1.421413741f);
    s = fmaf(t, s, -0.284496736f);
    s = fmaf(t, s, 0.254829592f);
    tail = 0.5f * t * s * e;
}

__device__ __forceinline__ float gelu(float a) {
    float e, tail;
    gauss(a, e, tail);
    return a * (a >= 0.f ? 1.0f - tail : tail);
}

// Phi(a) + a phi(a)
__device__ __forceinline__ float gelu_grad(float a) {
    float e, tail;
    gauss(a, e, tail);
    return fmaf(a * 0.39894228040143268f, e, a >= 0.f ? 1.0f - tail : tail);
}

// -------------------------------------------------- operands in the workspace

// v = hi + mid + lo, each a bf16 (returned as bits).  A value above the largest
// bf16 takes that as its hi; infinities and NaN have no mid and lo.
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v));
    if ((hi & 0x7f80u) == 0x7f80u) {
        if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) {
            mid = lo = 0u;
            return;
        }
        hi = (__float_as_uint(v) >> 31 << 15) | 0x7f7fu;
    }
    const float r1 = v - __uint_as_float(hi << 16);
    mid = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(r1));
    lo = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(r1 - __uint_as_float(mid << 16)));
}

constexpr int kPrepThreads = 256;

// Rows [m][n] of src, times act'(pre) when pre is given, as PARTS bf16 planes
// [m][ldd] (ldd a multiple of 8; columns n .. ldd - 1 zero); dst NULL: none are
// written.  colsum (NULL: none): the sums of the products over this CTA's rows,
// before any rounding, in row blockIdx.y of [gridDim.y][n].
// A CTA takes 8 tx columns and every (gridDim.y ty)-th group of ty rows, tx ty = 256.
template <typename TI, int PARTS>
__global__ void __launch_bounds__(kPrepThreads)
linear_prep(int m, int n, int tx, const TI* __restrict__ src, int64_t lds, bool svec,
            const typename std::conditional<PARTS == 3, float, bf16>::type* __restrict__ pre, int64_t ldp, bool pvec,
            bf16* __restrict__ dst, int64_t ldd, int64_t plane, float* __restrict__ colsum) {
    const int ty = kPrepThreads / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const int col = (blockIdx.x * tx + cx) * 8;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (col < n) {
#pragma unroll 2
        for (int64_t row = (int64_t)blockIdx.y * ty + ry; row < m; row += (int64_t)gridDim.y * ty) {
            float v[8];
            unpack8(load8(src + row * lds + col, n - col, svec), v);
            if (pre) {
                float a[8];
                unpack8(load8(pre + row * ldp + col, n - col, pvec), a);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= gelu_grad(a[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
            if (!dst) continue;
            if constexpr (PARTS == 1) {
                store8(dst + row * ldd + col, v, 8, true);
            } else {
                uint32_t w[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h0, m0, l0, h1, m1, l1;
                    split3(v[2 * i], h0, m0, l0);
                    split3(v[2 * i + 1], h1, m1, l1);
                    w[0][i] = h0 | (h1 << 16);
                    w[1][i] = m0 | (m1 << 16);
                    w[2][i] = l0 | (l1 << 16);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(dst + p * plane + row * ldd + col) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
            }
        }
    }
    if (!colsum) return;
    __shared__ float red[kPrepThreads][9];
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x][i] = acc[i];
    __syncthreads();
    for (int k = threadIdx.x; k < 8 * tx; k += kPrepThreads) {
        const int c = blockIdx.x * tx * 8 + k;
        float s = 0.f;
        for (int y = 0; y < ty; ++y) s += red[y * tx + (k >> 3)][k & 7];
        if (c < n) colsum[(int64_t)blockIdx.y * n + c] = s;
    }
}

// ------------------------------------------------------------------ the epilogue

// What becomes of a finished sum: a = acc + bias; pre = a; y = act(a) + r.
// Any pointer but y may be NULL.
struct Epi {
    const float* bias;
    const void* r;
    void* y;
    void* pre;
    int64_t ldr, ldy, ldpre;
    bool gelu_act, y_f32, pre_f32;   // r has y's type
    bool bvec, rvec, yvec, pvec;     // 16-byte accesses allowed
};

// Columns col .. col + 7 of row `row` (live of them, >= 1); b their biases.
__device__ __forceinline__ void epi8(const Epi& e, int64_t row, int col, int live, float (&v)[8], const float (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    if (e.pre) {
        if (e.pre_f32) store8(static_cast<float*>(e.pre) + row * e.ldpre + col, v, live, e.pvec);
        else store8(static_cast<bf16*>(e.pre) + row * e.ldpre + col, v, live, e.pvec);
    }
    if (e.gelu_act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = gelu(v[i]);
    }
    if (e.r) {
        float r[8];
        if (e.y_f32) unpack8(load8(static_cast<const float*>(e.r) + row * e.ldr + col, live, e.rvec), r);
        else unpack8(load8(static_cast<const bf16*>(e.r) + row * e.ldr + col, live, e.rvec), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    if (e.y_f32) store8(static_cast<float*>(e.y) + row * e.ldy + col, v, live, e.yvec);
    else store8(static_cast<bf16*>(e.y) + row * e.ldy + col, v, live, e.yvec);
}

__device__ __forceinline__ void epi_bias(const Epi& e, int col, int live, float (&b)[8]) {
    if (e.bias) unpack8(load8(e.bias + col, live, e.bvec), b);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.f;
}

// ------------------------------------------------------------- the product kernel

constexpr int kBM = 128;         // rows of a tile = TMEM lanes
constexpr int kBK = 64;          // contraction of a k-block: 128 bytes of bf16, one swizzle row
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (kEpiWarps + 2) * 32;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kStageA = kBM * kBK * 2;

// The terms of a split product, smallest first: planes of A and of B.
__device__ __forceinline__ int term_plane_a(int t) { return (0x001120 >> (4 * t)) & 15; }   // 0 2 1 1 0 0
__device__ __forceinline__ int term_plane_b(int t) { return (0x010102 >> (4 * t)) & 15; }   // 2 0 1 0 1 0

struct GemmShape {
    int M, N;             // of D
    int kblocks;          // of the contraction
    int terms;            // 1, or 6 for split operands
    int tiles_m, tiles_n;
    int splits;           // of the contraction; split s takes k-blocks [s kblocks / splits, (s + 1) kblocks / splits)
    __host__ __device__ int items() const { return tiles_m * tiles_n * splits; }
    __host__ __device__ int kb_lo(int s) const { return (int)((int64_t)s * kblocks / splits); }
};

// A work item: tile (m, n) and split s.  Tiles run in groups of 16 tile rows, down the
// group's column before the next, so that the CTAs of one wave share operands in L2.
struct Item {
    int m, n, s;
};
__device__ __forceinline__ Item item_of(const GemmShape& g, int i) {
    constexpr int kGroup = 16;
    const int tiles = g.tiles_m * g.tiles_n;
    const int s = i / tiles, t = i - s * tiles;
    const int per = kGroup * g.tiles_n;
    const int grp = t / per, w = t - grp * per;
    const int gm = g.tiles_m - grp * kGroup < kGroup ? g.tiles_m - grp * kGroup : kGroup;
    return Item{grp * kGroup + w % gm, w / gm, s};
}

template <int BN>
struct GemmCfg {
    static constexpr int kStageB = BN * kBK * 2;
    static constexpr int kStage = kStageA + kStageB;
    static constexpr int kStages = 192 * 1024 / kStage;
    static constexpr int kStaging = kEpiWarps * 32 * 32 * 4;
    static constexpr int kSmem = kStages * kStage + kStaging + 1024;
    static constexpr uint32_t kTmemCols = 2 * BN;
};

struct GemmBars {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t fin;
    uint32_t tmem_base;
    int abort;
};

// D = A B.  A is [M][contraction] (A_MN false) or [contraction][M] (true), B is
// [N][contraction] (B_MN false) or [contraction][N] (true).  part NULL: the
// finished sums go through `epi`; else split s stores its sums at
// part + (s M + row) ldpart.
//
// One persistent CTA per SM.  Warp kTmaWarp feeds a ring of stages by TMA, warp
// kMmaWarp issues the products into one of two TMEM accumulators, and eight warps
// take the other accumulator out (two per TMEM lane quarter, half of the columns
// each), through a swizzled 4 KB staging tile per warp that turns a lane's row into
// row pieces of whole sectors, so the epilogue of a tile runs under the next tile's products.
template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kGemmThreads, 1)
linear_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const GemmShape g,
            const Epi epi, float* __restrict__ part, int64_t ldpart, int* status) {
    using C = GemmCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ GemmBars bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == kTmaWarp * 32) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bars.acc_full[a], 1);
            mbar_init(&bars.acc_empty[a], kEpiWarps);
        }
        mbar_init(&bars.fin, 1);
        bars.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == kMmaWarp) tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bars.tmem_base;
    volatile int* abort_flag = &bars.abort;
    const int items = g.items();

    if (warp == kTmaWarp) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item w = item_of(g, i);
                const int lo = g.kb_lo(w.s), hi = g.kb_lo(w.s + 1);
                for (int t = 0; ok && t < g.terms; ++t) {
                    const int pa = g.terms == 1 ? 0 : term_plane_a(t), pb = g.terms == 1 ? 0 : term_plane_b(t);
                    for (int kb = lo; kb < hi; ++kb, ++it) {
                        const int st = it % C::kStages;
                        uint64_t* full = &bars.full[st];
                        if (it >= (uint32_t)C::kStages &&
                            !mbar_wait(&bars.empty[st], ((it / C::kStages) - 1) & 1, abort_flag, tc::kWaitNs)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = smem + st * C::kStage;
                        uint8_t* sb = sa + kStageA;
                        mbar_arrive_expect_tx(full, C::kStage);
                        if (A_MN) {
#pragma unroll
                            for (int b = 0; b < kBM / 64; ++b)
                                tma_load_3d(sa + b * 8192, &map_a, w.m * kBM + 64 * b, kb * kBK, pa, full);
                        } else {
                            tma_load_3d(sa, &map_a, kb * kBK, w.m * kBM, pa, full);
                        }
                        if (B_MN) {
#pragma unroll
                            for (int b = 0; b < BN / 64; ++b)
                                tma_load_3d(sb + b * 8192, &map_b, w.n * BN + 64 * b, kb * kBK, pb, full);
                        } else {
                            tma_load_3d(sb, &map_b, kb * kBK, w.n * BN, pb, full);
                        }
                    }
                }
            }
            if (!ok) tc::fail(&bars.abort, status);
            // Nothing may still be on its way into shared memory, or to a barrier in it, when the
            // CTA ends: every stage's last load has landed, and, unless a wait gave up, has been
            // consumed by products that have completed.
            int never = 0;
            for (uint32_t b = it > (uint32_t)C::kStages ? it - C::kStages : 0; b < it; ++b) {
                mbar_wait(&bars.full[b % C::kStages], (b / C::kStages) & 1, &never, tc::kWaitNs);
                if (ok) ok = mbar_wait(&bars.empty[b % C::kStages], (b / C::kStages) & 1, abort_flag, tc::kWaitNs);
            }
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t id = idesc_bf16(kBM, BN, A_MN, B_MN);
        // along the contraction: 8-row groups 1024 bytes apart, 32 bytes per k-step; along the
        // row: 64-element blocks 8192 bytes apart, 8-deep groups 1024 bytes apart, 2048 bytes per k-step
        const SmemDesc da = smem_desc_split(smem_u32(smem), A_MN ? 8192 : 16, 1024, 2);
        const SmemDesc db = smem_desc_split(smem_u32(smem) + kStageA, B_MN ? 8192 : 16, 1024, 2);
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x, ++n) {
            const Item w = item_of(g, i);
            const int steps = g.terms * (g.kb_lo(w.s + 1) - g.kb_lo(w.s));
            const uint32_t a = n & 1, d = tbase + a * BN;
            if (n >= 2 && !mbar_wait_all(&bars.acc_empty[a], ((n >> 1) - 1) & 1, abort_flag, tc::kWaitNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int k = 0; k < steps; ++k, ++it) {
                const int st = it % C::kStages;
                if (!mbar_wait_all(&bars.full[st], (it / C::kStages) & 1, abort_flag, tc::kWaitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t off = st * C::kStage;
#pragma unroll
                    for (int ks = 0; ks < kBK / 16; ++ks)
                        mma_ss(d, desc_at(da, off + (A_MN ? 2048 : 32) * ks), desc_at(db, off + (B_MN ? 2048 : 32) * ks),
                               id, k > 0 || ks > 0);
                    mma_commit(&bars.empty[st]);
                    if (k == steps - 1) mma_commit(&bars.acc_full[a]);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) tc::fail(&bars.abort, status);
            int never = 0;
            if (elect_one()) mma_commit(&bars.fin);
            __syncwarp();
            mbar_wait_all(&bars.fin, 0, &never, tc::kWaitNs);
        }
    } else {
        const uint32_t stg = smem_u32(smem + C::kStages * C::kStage) + warp * 4096;
        const int q = warp & 3, half = warp >> 2;
        const uint32_t tl = tbase + ((uint32_t)(32 * q) << 16);
        uint32_t n = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x, ++n) {
            const Item w = item_of(g, i);
            const uint32_t a = n & 1;
            if (!mbar_wait_all(&bars.acc_full[a], (n >> 1) & 1, abort_flag, tc::kWaitNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int64_t row0 = (int64_t)w.m * kBM + 32 * q;
#pragma unroll 1
            for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
                uint32_t v[32];
                tmem_ld_x32(tl + a * BN + c, v);
                tmem_wait_ld();
                if (c + 32 == (half + 1) * (BN / 2)) {   // the accumulator is out
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.acc_empty[a]);
                }
                __syncwarp();   // the staging tile has been read
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + ((j ^ (lane & 7)) << 4)),
                                 "r"(v[4 * j]), "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3])
                                 : "memory");
                __syncwarp();
                const int col = w.n * BN + c + 8 * (lane & 3), live = g.N - col;
                float b[8];
                if (live > 0 && !part) epi_bias(epi, col, live, b);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int rl = 8 * p + (lane >> 2);
                    const int64_t row = row0 + rl;
                    const uint4 u0 = lds_u4(stg + rl * 128 + (((2 * (lane & 3)) ^ (rl & 7)) << 4));
                    const uint4 u1 = lds_u4(stg + rl * 128 + (((2 * (lane & 3) + 1) ^ (rl & 7)) << 4));
                    if (row >= g.M || live <= 0) continue;
                    float f[8] = {__uint_as_float(u0.x), __uint_as_float(u0.y), __uint_as_float(u0.z), __uint_as_float(u0.w),
                                  __uint_as_float(u1.x), __uint_as_float(u1.y), __uint_as_float(u1.z), __uint_as_float(u1.w)};
                    if (part) store8(part + ((int64_t)w.s * g.M + row) * ldpart + col, f, 8, true);
                    else epi8(epi, row, col, live, f, b);
                }
            }
        }
        if (!ok && lane == 0) tc::fail(&bars.abort, status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, C::kTmemCols);
    }
}

// The splits' sums added in a fixed order, then the epilogue.  One thread per 8 columns.
__global__ void __launch_bounds__(256)
linear_join(int m, int n, int splits, const float* __restrict__ part, int64_t ldpart, const Epi epi) {
    const int per_row = (n + 7) / 8;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (idx >= (int64_t)m * per_row) return;
    const int64_t row = idx / per_row;
    const int col = (int)(idx - row * per_row) * 8, live = n - col;
    float v[8] = {}, b[8];
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        float f[8];
        unpack8(load8(part + ((int64_t)s * m + row) * ldpart + col, 8, true), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
    epi_bias(epi, col, live, b);
    epi8(epi, row, col, live, v, b);
}

// -------------------------------------------------------------------------- host

// A bf16 operand as the product reads it: planes of rows [rows][ld].
struct Operand {
    const bf16* p;
    int64_t ld, plane;
    int planes;
    int rows, cols;   // as stored
};

int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }

// Least contraction of a split: 256 (4 k-blocks) bf16.  Splits fill the SMs when
// the tiles alone do not.
struct GemmPlan {
    GemmShape g;
    int bn;
};

GemmPlan plan_gemm(int M, int N, int K, int terms) {
    GemmPlan best{};
    double best_us = 1e30;
    const int sms = num_sms();
    const int kb = (K + kBK - 1) / kBK;
    for (int bn : {256, 128, 64}) {
        const int tm = (M + kBM - 1) / kBM, tn = (N + bn - 1) / bn;
        const int64_t tiles = (int64_t)tm * tn;
        const double us_kb = bn == 256 ? 0.30 : bn == 128 ? 0.17 : 0.11;
        for (int sp = 1; sp <= 128; sp = sp < 8 ? sp + 1 : sp + sp / 4) {
            if (sp > 1 && (sp * tiles > 2 * sms || kb / sp < (terms == 1 ? 4 : 2))) break;
            const int64_t waves = (tiles * sp + sms - 1) / sms;
            const int64_t steps = (int64_t)((kb + sp - 1) / sp) * terms;
            double us = waves * steps * us_kb + 3.0 + 0.004 * bn * (waves < 4 ? waves : 4);
            if (sp > 1) us += 3.0 + (double)M * N * (sp + 2) * 4 / 4e6;
            if (us < best_us) {
                best_us = us;
                best.g = GemmShape{M, N, kb, terms, tm, tn, sp};
                best.bn = bn;
            }
        }
    }
    return best;
}

size_t part_floats(const GemmPlan& p) {
    return p.g.splits > 1 ? (size_t)p.g.splits * p.g.M * pad8(p.g.N) : 0;
}

template <int BN, bool A_MN, bool B_MN>
int launch_gemm(const GemmPlan& p, const CUtensorMap& ma, const CUtensorMap& mb, const Epi& epi, float* part,
                cudaStream_t s) {
    using C = GemmCfg<BN>;
    auto kern = linear_gemm<BN, A_MN, B_MN>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
        return GT_ERR_CUDA;
    int* status = device_status_ptr();
    if (!status) return GT_ERR_CUDA;
    const int sms = num_sms(), items = p.g.items();
    LaunchScope ls("linear_gemm", s);
    kern<<<items < sms ? items : sms, kGemmThreads, C::kSmem, s>>>(ma, mb, p.g, epi, part, pad8(p.g.N), status);
    return check_launch();
}

// D = A B through the epilogue.  a_mn / b_mn: the operand's rows run along the contraction's
// index and its columns along D's (stored [contraction][M] or [contraction][N]).
template <bool A_MN, bool B_MN>
int run_gemm(const GemmPlan& p, const Operand& a, const Operand& b, const Epi& epi, float* part, cudaStream_t s) {
    CUtensorMap ma, mb;
    const CUtensorMapDataType ty = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map_3d(&ma, a.p, ty, a.planes, a.rows, a.cols, a.plane * 2, a.ld * 2, A_MN ? kBK : kBM, 64,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_3d(&mb, b.p, ty, b.planes, b.rows, b.cols, b.plane * 2, b.ld * 2, B_MN ? kBK : p.bn, 64,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return GT_ERR_CUDA;
    float* out = p.g.splits > 1 ? part : nullptr;
    int rc = p.bn == 256   ? launch_gemm<256, A_MN, B_MN>(p, ma, mb, epi, out, s)
             : p.bn == 128 ? launch_gemm<128, A_MN, B_MN>(p, ma, mb, epi, out, s)
                           : launch_gemm<64, A_MN, B_MN>(p, ma, mb, epi, out, s);
    if (rc != GT_OK || !out) return rc;
    const int64_t threads = (int64_t)p.g.M * ((p.g.N + 7) / 8);
    LaunchScope ls("linear_join", s);
    linear_join<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(p.g.M, p.g.N, p.g.splits, part, pad8(p.g.N), epi);
    return check_launch();
}

// Grid of linear_prep for [m][n]: tx column threads per CTA, and with column sums
// at most kPrepSlabs row slabs (each a partial row of the sums).
constexpr int kPrepSlabs = 512;
struct PrepGrid {
    int tx, gx, gy;
};
PrepGrid prep_grid(int m, int n) {
    int tx = 8;
    while (tx < 32 && tx * 8 < n) tx *= 2;
    const int ty = kPrepThreads / tx, gx = (n + 8 * tx - 1) / (8 * tx);
    int64_t gy = ((int64_t)m + ty - 1) / ty;
    const int64_t most = (8 * (int64_t)num_sms() + gx - 1) / gx;
    if (gy > most) gy = most;
    if (gy > kPrepSlabs) gy = kPrepSlabs;
    return {tx, gx, (int)gy};
}

template <typename TI, int PARTS>
int run_prep(int m, int n, const void* src, int64_t lds, const void* pre, int64_t ldp, bf16* dst, float* colsum,
             cudaStream_t s) {
    using TP = typename std::conditional<PARTS == 3, float, bf16>::type;
    const PrepGrid pg = prep_grid(m, n);
    const int64_t ldd = pad8(n);
    LaunchScope ls("linear_prep", s);
    linear_prep<TI, PARTS><<<dim3(pg.gx, pg.gy), kPrepThreads, 0, s>>>(
        m, n, pg.tx, static_cast<const TI*>(src), lds, rows16(src, lds, sizeof(TI)), static_cast<const TP*>(pre), ldp,
        pre && rows16(pre, ldp, sizeof(TP)), dst, ldd, (int64_t)m * ldd, colsum);
    return check_launch();
}

// src [m][n] of the compute type as an operand: read in place when TMA can, else
// through `buf` (split in three for fp32, copied for bf16).
int make_operand(int dtype, int m, int n, const void* src, int64_t ld, bf16* buf, Operand* o, cudaStream_t s) {
    if (!buf) {
        *o = Operand{static_cast<const bf16*>(src), ld, ld, 1, m, n};
        return GT_OK;
    }
    const int64_t ldd = pad8(n);
    *o = Operand{buf, ldd, m * ldd, dtype == GT_F32 ? 3 : 1, m, n};
    return dtype == GT_F32 ? run_prep<float, 3>(m, n, src, ld, nullptr, 0, buf, nullptr, s)
                           : run_prep<bf16, 1>(m, n, src, ld, nullptr, 0, buf, nullptr, s);
}

size_t operand_elems(int dtype, int m, int n) { return (size_t)m * pad8(n) * (dtype == GT_F32 ? 3 : 1); }

int elem_bytes(int t) { return t == GT_F32 ? 4 : 2; }
int terms_of(int dtype) { return dtype == GT_F32 ? 6 : 1; }

constexpr int kMaxWidth = 65536, kMaxRows = 1 << 24;

int check_linear(int dtype, int ytype, int m, int k, int n, int act) {
    if ((dtype != GT_F32 && dtype != GT_BF16) || (ytype != GT_F32 && ytype != GT_BF16)) return GT_ERR_INVALID_ARG;
    if (m < 1 || k < 1 || n < 1 || (act != GT_ACT_NONE && act != GT_ACT_GELU)) return GT_ERR_INVALID_ARG;
    if (dtype == GT_F32 && ytype != GT_F32) return GT_ERR_UNSUPPORTED;
    if (m > kMaxRows || k > kMaxWidth || n > kMaxWidth) return GT_ERR_UNSUPPORTED;
    return GT_OK;
}

// Workspace of the forward: x and W where they cannot be read in place, and the splits' sums.
struct FwdBufs {
    bf16 *x, *w;
    float* part;
};
size_t fwd_bufs(int dtype, int m, int k, int n, bool pack_x, bool pack_w, void* ws, size_t bytes, FwdBufs* out) {
    Carve c(ws, bytes);
    FwdBufs b;
    b.x = pack_x ? c.take<bf16>(operand_elems(dtype, m, k)) : nullptr;
    b.w = pack_w ? c.take<bf16>(operand_elems(dtype, k, n)) : nullptr;
    b.part = c.take<float>(part_floats(plan_gemm(m, n, k, terms_of(dtype))));
    if (out) *out = b;
    return c.off;
}

// ... and of the backward, with da (where dy itself does not serve), the column sums' partial
// rows, and one buffer for the splits' sums of both products in turn.
struct BwdBufs {
    bf16 *x, *w, *da;
    float *part, *cols;
};
size_t bwd_bufs(int dtype, int m, int k, int n, bool pack_x, bool pack_w, bool own_da, void* ws, size_t bytes,
                BwdBufs* out) {
    Carve c(ws, bytes);
    BwdBufs b;
    b.x = pack_x ? c.take<bf16>(operand_elems(dtype, m, k)) : nullptr;
    b.w = pack_w ? c.take<bf16>(operand_elems(dtype, k, n)) : nullptr;
    b.da = own_da ? c.take<bf16>(operand_elems(dtype, m, n)) : nullptr;
    const size_t px = part_floats(plan_gemm(m, k, n, terms_of(dtype)));
    const size_t pw = part_floats(plan_gemm(k, n, m, terms_of(dtype)));
    b.part = c.take<float>(px > pw ? px : pw);
    b.cols = c.take<float>((size_t)prep_grid(m, n).gy * n);
    if (out) *out = b;
    return c.off;
}

bool ranges_ok(const void* p, int64_t ld, int cols) { return !p || ld >= cols; }

}  // namespace
}  // namespace gt

extern "C" {

size_t gt_linear_fwd_workspace_size(int32_t dtype, int32_t m, int32_t k, int32_t n, int32_t aligned) {
    using namespace gt;
    if (check_linear(dtype, GT_F32, m, k, n, GT_ACT_NONE) != GT_OK) return 0;
    const bool pack = dtype == GT_F32 || !aligned;
    return fwd_bufs(dtype, m, k, n, pack, pack, nullptr, 0, nullptr) + 256;
}

size_t gt_linear_bwd_workspace_size(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, int32_t act,
                                    int32_t aligned) {
    using namespace gt;
    if (check_linear(dtype, ytype, m, k, n, act) != GT_OK) return 0;
    const bool pack = dtype == GT_F32 || !aligned;
    return bwd_bufs(dtype, m, k, n, pack, pack, pack || act != GT_ACT_NONE || ytype != dtype, nullptr, 0, nullptr) + 256;
}

int gt_linear_fwd(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, const void* x, int64_t ldx,
                  const void* w, int64_t ldw, const float* b, int32_t act, const void* r, int64_t ldr, void* y,
                  int64_t ldy, void* pre, int64_t ldpre, void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt;
    int rc = check_linear(dtype, ytype, m, k, n, act);
    if (rc != GT_OK) return rc;
    if (!x || !w || !y || ldx < k || ldw < n || ldy < n || !ranges_ok(r, ldr, n) || !ranges_ok(pre, ldpre, n))
        return GT_ERR_INVALID_ARG;
    const bool pack_x = dtype == GT_F32 || !rows16(x, ldx, 2), pack_w = dtype == GT_F32 || !rows16(w, ldw, 2);
    FwdBufs bufs;
    const size_t need = fwd_bufs(dtype, m, k, n, pack_x, pack_w, workspace, ws_bytes, &bufs);
    if (need > 0 && (!workspace || !aligned16(workspace) || ws_bytes < need)) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Operand ox, ow;
    if ((rc = make_operand(dtype, m, k, x, ldx, bufs.x, &ox, s)) != GT_OK) return rc;
    if ((rc = make_operand(dtype, k, n, w, ldw, bufs.w, &ow, s)) != GT_OK) return rc;
    const int ey = elem_bytes(ytype), ex = elem_bytes(dtype);
    const Epi epi{b, r, y, pre, ldr, ldy, ldpre, act == GT_ACT_GELU, ytype == GT_F32, dtype == GT_F32,
                  aligned16(b), r && rows16(r, ldr, ey), rows16(y, ldy, ey), pre && rows16(pre, ldpre, ex)};
    return run_gemm<false, true>(plan_gemm(m, n, k, terms_of(dtype)), ox, ow, epi, bufs.part, s);
}

int gt_linear_bwd(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, const void* dy, int64_t lddy,
                  const void* x, int64_t ldx, const void* w, int64_t ldw, const void* pre, int64_t ldpre, int32_t act,
                  const void* add, int64_t ldadd, void* dx, int64_t lddx, void* dw, int64_t lddw, float* db,
                  void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt;
    int rc = check_linear(dtype, ytype, m, k, n, act);
    if (rc != GT_OK) return rc;
    if (!dy || lddy < n || (!dx && !dw && !db)) return GT_ERR_INVALID_ARG;
    if ((dw && (!x || ldx < k || lddw < n)) || (dx && (!w || ldw < n || lddx < k))) return GT_ERR_INVALID_ARG;
    if ((act != GT_ACT_NONE) != (pre != nullptr) || !ranges_ok(pre, ldpre, n)) return GT_ERR_INVALID_ARG;
    if (add && (!dx || ldadd < k)) return GT_ERR_INVALID_ARG;
    const bool products = dx || dw;
    const bool pack_x = dw && (dtype == GT_F32 || !rows16(x, ldx, 2));
    const bool pack_w = dx && (dtype == GT_F32 || !rows16(w, ldw, 2));
    const bool own_da = products && (dtype == GT_F32 || ytype != dtype || act != GT_ACT_NONE || !rows16(dy, lddy, 2));
    BwdBufs bufs;
    const size_t need = bwd_bufs(dtype, m, k, n, pack_x, pack_w, own_da, workspace, ws_bytes, &bufs);
    if (!workspace || !aligned16(workspace) || ws_bytes < need) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // da, and the column sums' partial rows
    float* cols = db ? bufs.cols : nullptr;
    if (own_da || db) {
        rc = dtype == GT_F32   ? run_prep<float, 3>(m, n, dy, lddy, pre, ldpre, bufs.da, cols, s)
             : ytype == GT_F32 ? run_prep<float, 1>(m, n, dy, lddy, pre, ldpre, bufs.da, cols, s)
                               : run_prep<bf16, 1>(m, n, dy, lddy, pre, ldpre, bufs.da, cols, s);
        if (rc != GT_OK) return rc;
    }
    const int64_t ldda = own_da ? pad8(n) : lddy;
    const Operand oda{own_da ? bufs.da : static_cast<const bf16*>(dy), ldda, own_da ? m * ldda : ldda,
                      dtype == GT_F32 ? 3 : 1, m, n};
    const int ex = elem_bytes(dtype);
    Operand o;
    if (dx) {
        if ((rc = make_operand(dtype, k, n, w, ldw, bufs.w, &o, s)) != GT_OK) return rc;
        const Epi epi{nullptr, add, dx, nullptr, ldadd, lddx, 0, false, dtype == GT_F32, false,
                      false, add && rows16(add, ldadd, ex), rows16(dx, lddx, ex), false};
        if ((rc = run_gemm<false, false>(plan_gemm(m, k, n, terms_of(dtype)), oda, o, epi, bufs.part, s)) != GT_OK)
            return rc;
    }
    if (dw) {
        if ((rc = make_operand(dtype, m, k, x, ldx, bufs.x, &o, s)) != GT_OK) return rc;
        const Epi epi{nullptr, nullptr, dw, nullptr, 0, lddw, 0, false, dtype == GT_F32, false,
                      false, false, rows16(dw, lddw, ex), false};
        if ((rc = run_gemm<true, true>(plan_gemm(k, n, m, terms_of(dtype)), o, oda, epi, bufs.part, s)) != GT_OK)
            return rc;
    }
    return db ? launch_col_sum("linear_bias_sum", bufs.cols, prep_grid(m, n).gy, n, db, n, nullptr, s) : GT_OK;
}

}  // extern "C"
