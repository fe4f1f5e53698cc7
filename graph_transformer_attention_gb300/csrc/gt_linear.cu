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
// above 2^-24 of the largest:  lo hi, hi lo, mid mid, mid hi, hi mid, hi hi, added up
// in this order, k-block by k-block, so that the small ones meet a small accumulator.
// Six bf16 products run at a sixth of the bf16 rate, which is four times what the
// fp32 pipes reach.
//
// Rows that TMA cannot read (a base or row stride that is no multiple of 16 bytes)
// are first copied to padded rows in the workspace by the kernel that splits fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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

// For two values: e = exp(-a^2 / 2) and the tail of the normal CDF,
//   Phi(-|a|) = e h(|a|),  h(x) = erfcx(x / sqrt 2) / 2 = t (c1 + c2 t + ... + c7 t^6),  t = 1 / (r + k x),
// where h falls smoothly from 1/2, so that the tail keeps its relative accuracy: for Phi(a) = 1/2 - sign(a) (1/2 - tail)
// all digits of a GELU below -5 would cancel.  k = sqrt(log2(e) / 2), so that e = 2^-(k a)^2 shares the product, and r = 4 k.
// The c are this code's own fit: a linear programme for the least largest error on 0 <= x <= 13.5 (beyond, e is 0),
// weighted so that the tail times max(1, x) is 0.5e-8 off at most, or 5e-5 of itself where that is less.
// In fp32 GELU and slope are within 1.1e-7 and 1.9e-7 of the exact ones for |a| <= 2, and GELU within 6e-5 of itself down to
// a = -13.  Abramowitz and Stegun 7.1.26 with that difference (2.3e-7 and 2.6e-7, 2.6e-7 at -4 .. -2, 5 % of itself at -5) has two
// terms less and is the faster by 1 to 2 % (32768x1024x4096 bf16: forward with pre 187 against 190 us, backward 444 against 452).
__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The formula's constants as register pairs.  The compiler would rather build a pair anew at every
// use than keep it, which doubles the instructions of the packed arithmetic; behind an empty asm
// statement it has to keep them.
struct GaussK {
    float2 c7, c6, c5, c4, c3, c2, c1;   // (the c negated)
};
constexpr float kGaussK = 0.849321783f, kGaussR = 3.39728713f;

__device__ __forceinline__ float2 kept(float x) {
    float2 r = f2(x);
    asm volatile("" : "+f"(r.x), "+f"(r.y));
    return r;
}

__device__ __forceinline__ GaussK gauss_constants() {
    return GaussK{kept(483.096161f), kept(-531.246826f), kept(124.012375f), kept(-38.318634f), kept(-0.846040547f),
                  kept(-1.3042357f), kept(-0.33545205f)};
}

// e and minus the tail
__device__ __forceinline__ void gauss2(const GaussK& k, float2 a, float2& e, float2& minus) {
    // (k a by single factors: one constant less in registers, where the 256 x 256 tiles have none left)
    const float2 b = make_float2(a.x * kGaussK, a.y * kGaussK), q = __fmul2_rn(b, b);
    const float2 t = make_float2(rcp(fabsf(b.x) + kGaussR), rcp(fabsf(b.y) + kGaussR));
    e = make_float2(ex2(-q.x), ex2(-q.y));
    float2 s = __ffma2_rn(t, k.c7, k.c6);
    s = __ffma2_rn(t, s, k.c5);
    s = __ffma2_rn(t, s, k.c4);
    s = __ffma2_rn(t, s, k.c3);
    s = __ffma2_rn(t, s, k.c2);
    s = __ffma2_rn(t, s, k.c1);
    minus = __fmul2_rn(__fmul2_rn(t, s), e);
}

// a Phi(a) = max(a, 0) - |a| tail, with the step's factor 0 or 1 for the maximum and a bounded |a|, so that infinities give
// what the product a Phi(a) does: infinity and, for the negative one, NaN.
__device__ __forceinline__ float2 gelu2(const GaussK& k, float2 a) {
    float2 e, minus;
    gauss2(k, a, e, minus);
    const float2 step = make_float2(__saturatef(a.x * 1e38f), __saturatef(a.y * 1e38f));
    return __ffma2_rn(a, step, __fmul2_rn(make_float2(fminf(fabsf(a.x), 1e30f), fminf(fabsf(a.y), 1e30f)), minus));
}

// Phi(a) + a phi(a)
__device__ __forceinline__ float2 gelu_grad2(const GaussK& k, float2 a) {
    float2 e, minus;
    gauss2(k, a, e, minus);
    const float2 cdf = make_float2(a.x >= 0.f ? 1.f + minus.x : -minus.x, a.y >= 0.f ? 1.f + minus.y : -minus.y);
    return __ffma2_rn(__fmul2_rn(a, f2(0.39894228040143268f)), e, cdf);
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

// Rows [m][n] of src (fp32 or bf16), times act'(pre) when pre is given, as bf16 planes
// [m][ldd] (ldd a multiple of 8; columns n .. ldd - 1 zero); dst NULL: none are
// written.  colsum (NULL: none): the sums of the products over a CTA's rows,
// before any rounding, in row y of [gy][n].
// CTA (x, y) of gx gy takes 8 tx columns and every (gy ty)-th group of ty rows, tx ty = 256.
struct PrepJob {
    const void* src;
    const void* pre;   // of the compute type
    bf16* dst;
    float* colsum;
    int64_t lds, ldp, ldd, plane;
    int m, n, tx, gx, gy;
    bool f32;
    int svec, pvec;   // row_access()
};
constexpr int kPrepJobs = 3;
struct PrepJobs {
    PrepJob j[kPrepJobs];
    int count;
};

// With bf16 operands (PARTS 1) da is rounded to bf16, also where dy came in fp32: both products want it in the operands'
// type, and a second plane for what the rounding drops would double their time (154 and 158 us each at 32768x1024x4096).
// dx and dW are 2.3e-3 off in the mean with it, against 1.7e-3 by their own rounding alone; the column sums are
// taken before it.  Callers who want da whole pass fp32 operands (PARTS 3).
//
// Two rows of each input are in flight per thread, four CTAs on an SM (measured on da of 32768 x 4096 bf16 with
// GELU, which issues in 63 % of the cycles: 143 us, 83 % of the copy rate; four rows and two CTAs were 8 % slower).
template <typename TI, int PARTS>
__device__ __forceinline__ void prep_rows(const PrepJob& J, int bx, int by) {
    using TP = typename std::conditional<PARTS == 3, float, bf16>::type;
    constexpr int R = 2;   // rows in flight per thread
    const TI* src = static_cast<const TI*>(J.src);
    const TP* pre = static_cast<const TP*>(J.pre);
    const int m = J.m, n = J.n, tx = J.tx, ty = kPrepThreads / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const int col = (bx * tx + cx) * 8;
    const GaussK gk = gauss_constants();
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (col < n) {
        const int64_t step = (int64_t)J.gy * ty;
        for (int64_t row0 = (int64_t)by * ty + ry; row0 < m; row0 += R * step) {
            Raw8<TI> rs[R];
            Raw8<TP> rp[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = row0 + k * step, r = row < m ? row : row0;
                rs[k] = load8(src + r * J.lds + col, row < m ? n - col : 0, J.svec);
                if (pre) rp[k] = load8(pre + r * J.ldp + col, row < m ? n - col : 0, J.pvec);
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = row0 + k * step;
                float v[8];
                unpack8(rs[k], v);
                if (pre) {
                    float a[8];
                    unpack8(rp[k], a);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 g = gelu_grad2(gk, make_float2(a[i], a[i + 1]));
                        v[i] *= g.x;
                        v[i + 1] *= g.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += v[i];
                if (!J.dst || row >= m) continue;
                if constexpr (PARTS == 1) {
                    store8(J.dst + row * J.ldd + col, v, 8, 1);
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
                        *reinterpret_cast<uint4*>(J.dst + p * J.plane + row * J.ldd + col) =
                            make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
                }
            }
        }
    }
    if (!J.colsum) return;
    __shared__ float red[kPrepThreads][9];
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x][i] = acc[i];
    __syncthreads();
    for (int k = threadIdx.x; k < 8 * tx; k += kPrepThreads) {
        const int c = bx * tx * 8 + k;
        float s = 0.f;
        for (int y = 0; y < ty; ++y) s += red[y * tx + (k >> 3)][k & 7];
        if (c < n) J.colsum[(int64_t)by * n + c] = s;
    }
}

// One launch prepares all of a call's operands, a range of CTAs each.
template <int PARTS>
__global__ void __launch_bounds__(kPrepThreads, PARTS == 3 ? 3 : 4) linear_prep(const PrepJobs jobs) {
    pdl_trigger();
    int b = blockIdx.x, k = 0;
    while (k + 1 < jobs.count && b >= jobs.j[k].gx * jobs.j[k].gy) {
        b -= jobs.j[k].gx * jobs.j[k].gy;
        ++k;
    }
    const PrepJob& J = jobs.j[k];
    const int by = b / J.gx, bx = b - by * J.gx;
    if constexpr (PARTS == 3) {
        prep_rows<float, 3>(J, bx, by);
    } else {
        if (J.f32) prep_rows<float, 1>(J, bx, by);
        else prep_rows<bf16, 1>(J, bx, by);
    }
}

// ------------------------------------------------------------------ the epilogue

// What becomes of a finished sum: a = acc + bias; pre = a; y = act(a) + r.
// Any pointer but y may be NULL.  r has y's type.  The accesses are row_access().
struct Epi {
    const float* bias;
    const void* r;
    void* y;
    void* pre;
    int64_t ldr, ldy, ldpre;
    bool gelu_act, y_f32, pre_f32;
    bool single;   // some rows can only be reached by single elements: through the staging tiles, or left to linear_join
    bool bulk;     // bf16 results go out as TMA boxes (the pair kernel; maps in the kernel's arguments)
    int racc, yacc, pacc;
};

// v[0 .. CW - 1] to p[0 .. live - 1]: whole 32-byte sectors where the rows allow them.
template <int CW>
__device__ __forceinline__ void put_row(void* base, int64_t at, bool f32, const float (&v)[CW], int live, int acc) {
    if (f32) {
        float* p = static_cast<float*>(base) + at;
        if (live >= CW && acc == 2) {
#pragma unroll
            for (int g = 0; g < CW / 8; ++g) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * g + i]);
                stg32(p + 8 * g, w);
            }
            return;
        }
#pragma unroll
        for (int g = 0; g < CW / 8; ++g) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = v[8 * g + i];
            store8(p + 8 * g, t, live - 8 * g, acc);
        }
    } else {
        bf16* p = static_cast<bf16*>(base) + at;
        if (CW % 16 == 0 && live >= CW && acc == 2) {
#pragma unroll
            for (int g = 0; g < CW / 16; ++g) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[16 * g + 2 * i], v[16 * g + 2 * i + 1]);
                stg32(p + 16 * g, w);
            }
            return;
        }
#pragma unroll
        for (int g = 0; g < CW / 8; ++g) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = v[8 * g + i];
            store8(p + 8 * g, t, live - 8 * g, acc);
        }
    }
}

// v[i] += base[at + i], which may be the output itself
template <int CW>
__device__ __forceinline__ void add_row(const void* base, int64_t at, bool f32, float (&v)[CW], int live, int acc) {
    if (f32) {
        const float* p = static_cast<const float*>(base) + at;
        if (live >= CW && acc == 2) {
#pragma unroll
            for (int g = 0; g < CW / 8; ++g) {
                uint32_t w[8];
                ldg32(p + 8 * g, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[8 * g + i] += __uint_as_float(w[i]);
            }
            return;
        }
#pragma unroll
        for (int g = 0; g < CW / 8; ++g) {
            float t[8];
            unpack8(load8<Mem::kOutput>(p + 8 * g, live - 8 * g, acc), t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * g + i] += t[i];
        }
    } else {
        const bf16* p = static_cast<const bf16*>(base) + at;
        if (CW % 16 == 0 && live >= CW && acc == 2) {
#pragma unroll
            for (int g = 0; g < CW / 16; ++g) {
                uint32_t w[8];
                ldg32(p + 16 * g, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[16 * g + 2 * i] += __uint_as_float(w[i] << 16);
                    v[16 * g + 2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
                }
            }
            return;
        }
#pragma unroll
        for (int g = 0; g < CW / 8; ++g) {
            float t[8];
            unpack8(load8<Mem::kOutput>(p + 8 * g, live - 8 * g, acc), t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * g + i] += t[i];
        }
    }
}

// Columns col .. col + CW - 1 (live of them, >= 1) of row `row`; bias: theirs, in shared memory.
template <int CW>
__device__ __forceinline__ void add_bias(float (&v)[CW], uint32_t bias) {
#pragma unroll
    for (int i = 0; i < CW; i += 4) {
        const uint4 w = lds_u4(bias + 4 * i);
        const float2 a = __fadd2_rn(make_float2(v[i], v[i + 1]), make_float2(__uint_as_float(w.x), __uint_as_float(w.y)));
        const float2 b = __fadd2_rn(make_float2(v[i + 2], v[i + 3]), make_float2(__uint_as_float(w.z), __uint_as_float(w.w)));
        v[i] = a.x; v[i + 1] = a.y; v[i + 2] = b.x; v[i + 3] = b.y;
    }
}

template <int CW>
__device__ __forceinline__ void apply_gelu(float (&v)[CW]) {
    const GaussK gk = gauss_constants();
#pragma unroll
    for (int i = 0; i < CW; i += 2) {
        const float2 y = gelu2(gk, make_float2(v[i], v[i + 1]));
        v[i] = y.x;
        v[i + 1] = y.y;
    }
}

template <int CW>
__device__ __forceinline__ void epilogue(const Epi& e, int64_t row, int col, int live, float (&v)[CW], uint32_t bias) {
    add_bias<CW>(v, bias);
    if (e.pre) put_row<CW>(e.pre, row * e.ldpre + col, e.pre_f32, v, live, e.pacc);
    if (e.gelu_act) apply_gelu<CW>(v);
    if (e.r) add_row<CW>(e.r, row * e.ldr + col, e.y_f32, v, live, e.racc);
    put_row<CW>(e.y, row * e.ldy + col, e.y_f32, v, live, e.yacc);
}

// The same for a whole warp and 32 columns of bf16 results, through the warp's 2 KB staging tile: rows of
// 64 bytes, 64-byte swizzle.  They leave by TMA (a lane's row in 32-byte pieces costs the L1 four times
// the cycles of whole lines, and the products need that memory's bandwidth: 32768x1024x4096, GELU and pre, 195 -> 185 us
// alone), or, where rows can only be reached so, by single elements, a row of the tile at a time
// (20000x1001x999 with a residual: 142 us with linear_join's help, 86 us so).
constexpr int kBoxCols = 32, kBoxBytes = 32 * kBoxCols * 2;

__device__ __forceinline__ uint32_t box_unit(uint32_t stg, int row, int unit) {   // 16 bytes, eight columns
    return stg + row * 64 + ((unit ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t box_element(uint32_t stg, int row, int col) {
    return box_unit(stg, row, col >> 3) + (col & 7) * 2;
}

__device__ __forceinline__ void fill_box(const float (&v)[32], uint32_t stg) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts_u4(box_unit(stg, lane, j), pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
               pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
}

__device__ __forceinline__ void put_box(const CUtensorMap* map, int64_t row0, int col, const float (&v)[32], uint32_t stg) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) bulk_wait_read();   // the tile's last box has been read
    __syncwarp();
    fill_box(v, stg);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, stg, col, (int)row0);
        bulk_commit();
    }
}

// p: the array at the box's first row and column, of which `rows` rows and `live` columns exist.
__device__ __forceinline__ void put_elements(bf16* p, int64_t ld, int rows, int live, const float (&v)[32], uint32_t stg) {
    const int lane = threadIdx.x & 31;
    fill_box(v, stg);
    __syncwarp();
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        uint16_t e;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(box_element(stg, i, lane)) : "memory");
        if (i < rows && lane < live) p[i * ld + lane] = __ushort_as_bfloat16(e);
    }
    __syncwarp();
}
__device__ __forceinline__ void add_elements(const bf16* p, int64_t ld, int rows, int live, float (&v)[32], uint32_t stg) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint16_t e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = h + i < rows && lane < live ? __bfloat16_as_ushort(p[(h + i) * ld + lane]) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(box_element(stg, h + i, lane)), "h"(e[i]) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 w = lds_u4(box_unit(stg, lane, j));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * j + 2 * i] += __uint_as_float(u[i] << 16);
            v[8 * j + 2 * i + 1] += __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void epilogue_box(const Epi& e, const CUtensorMap* map_y, const CUtensorMap* map_pre,
                                             int64_t row0, int M, int col, int live, float (&v)[32], uint32_t bias,
                                             uint32_t stg) {
    const int rows = (int)(M - row0);
    add_bias<32>(v, bias);
    if (e.pre) {
        if (e.bulk) put_box(map_pre, row0, col, v, stg);
        else put_elements(static_cast<bf16*>(e.pre) + row0 * e.ldpre + col, e.ldpre, rows, live, v, stg);
    }
    if (e.gelu_act) apply_gelu<32>(v);
    if (e.r) {
        const int64_t row = row0 + (threadIdx.x & 31);
        if (!e.bulk) add_elements(static_cast<const bf16*>(e.r) + row0 * e.ldr + col, e.ldr, rows, live, v, stg);
        else if (row < M) add_row<32>(e.r, row * e.ldr + col, false, v, live, e.racc);
    }
    if (e.bulk) put_box(map_y, row0, col, v, stg);
    else put_elements(static_cast<bf16*>(e.y) + row0 * e.ldy + col, e.ldy, rows, live, v, stg);
}

// ------------------------------------------------------------- the product kernel

constexpr int kBK = 64;          // contraction of a k-block: 128 bytes of bf16, one swizzle row
constexpr int kEpiWarps = 16;
constexpr int kGemmThreads = (kEpiWarps + 4) * 32;   // the fourth warp makes a whole warpgroup
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 2;   // TMA: two warps, one per operand
constexpr int kStageA = 128 * kBK * 2;

// Division by a number known on the host: x / d = the high half of x times (2^64 / d rounded up),
// exact for 32-bit x.
struct Divider {
    uint32_t d;
    uint64_t inv;
    static Divider of(uint32_t d) { return Divider{d, d > 1 ? ~uint64_t(0) / d + 1 : 0}; }
    __device__ __forceinline__ int div(int x) const { return d == 1 ? x : (int)__umul64hi((uint64_t)(uint32_t)x, inv); }
};

struct GemmShape {
    int M, N;             // of D
    int kblocks;          // of the contraction
    int planes;           // of the operands: 1, or 3 (hi, mid, lo)
    int chunk;            // k-blocks that an accumulator may sum (see linear_gemm)
    int tiles_m, tiles_n;
    bool whole_a, whole_b;   // an operand with rows along D, as whole blocks of 64 columns
    int splits;           // of the contraction; split s takes k-blocks [s kblocks / splits, (s + 1) kblocks / splits)
    Divider by_tiles, by_group, by_tail, by_splits;   // tiles, tiles of a whole group, tile rows of the last group, splits
    __host__ __device__ int items() const { return tiles_m * tiles_n * splits; }
};
constexpr int kGroup = 8;

// A work item: tile (m, n) and the k-blocks [lo, hi) of split s.  Tiles run in groups of 8 tile
// rows, down the group's column before the next, so that the CTAs of one wave share operands in L2.
struct Item {
    int m, n, s, lo, hi;
};
__device__ __forceinline__ Item item_of(const GemmShape& g, int i) {
    const int s = g.by_tiles.div(i), t = i - s * (int)g.by_tiles.d;
    const int grp = g.by_group.div(t), w = t - grp * (int)g.by_group.d;
    const bool tail = (grp + 1) * kGroup > g.tiles_m;
    const int n = tail ? g.by_tail.div(w) : w / kGroup;
    const int m = grp * kGroup + w - n * (tail ? (int)g.by_tail.d : kGroup);
    // s kblocks stays below 2^32: a split has at least one of at most 2^18 k-blocks, and at most 128 are made
    return Item{m, n, s, g.by_splits.div(s * g.kblocks), g.by_splits.div((s + 1) * g.kblocks)};
}

// CTAS CTAs (one, or a pair of a cluster) make a tile of 128 CTAS x BN.  SUM: an item may have
// several chunks, whose sums wait in registers (a pair's 64 columns per lane leave room for 16 more).
template <int CTAS, int BN, bool SUM>
struct GemmCfg {
    static constexpr int kBM = 128 * CTAS;
    static constexpr int kStageB = BN / CTAS * kBK * 2;   // a CTA of a pair holds half of B's columns
    static constexpr int kStage = kStageA + kStageB;
    static constexpr bool kBulk = CTAS == 2 && !SUM;      // bf16 results, which go out by staging tiles
    static constexpr int kStages = (kBulk ? 160 : 192) * 1024 / kStage;   // 5 to 8
    static constexpr int kStg = kBulk ? kBoxBytes : 0;    // staging of an epilogue warp
    static constexpr int kSmem = kStages * kStage + kEpiWarps * kStg + 1024;
    static constexpr uint32_t kTmemCols = 2 * BN;
    static constexpr int kCols = BN / 4;                  // accumulator columns of an epilogue warp
    static constexpr int kCW = kCols < 32 || (SUM && kCols > 32) ? 16 : 32;   // columns taken out at once
};

constexpr int kMaxStages = 8;
struct GemmBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t fin;
    uint32_t tmem_base;
    int abort;
};

// A warp's walk round a ring of stage barriers.  A successful wait takes over 100 cycles from issue to
// use, which a step cannot hide, so the barrier of the next stage is asked about a step ahead (measured
// on a step of a wait, an election and an arrival: 281 cycles, 144 with the question ahead).
template <int STAGES>
struct Ring {
    uint64_t* bar;
    uint32_t st, parity;
    bool ahead;
    __device__ __forceinline__ Ring(uint64_t* b, uint32_t p) : bar(b), st(0), parity(p) { ahead = mbar_test(bar, p); }
    // Waits for the current stage, names it in `s` and moves on; false where the wait gave up.
    __device__ __forceinline__ bool next(uint32_t& s, volatile int* abort_flag) {
        s = st;
        bool ok = true;
        if (!__all_sync(0xffffffffu, ahead)) ok = mbar_wait_all(bar + st, parity, abort_flag, tc::kWaitNs);
        if (++st == STAGES) {
            st = 0;
            parity ^= 1u;
        }
        ahead = mbar_test(bar + st, parity);
        return ok;
    }
};

// D = A B.  A is [M][contraction] (A_MN false) or [contraction][M] (true), B is
// [N][contraction] (B_MN false) or [contraction][N] (true).  part NULL: the
// finished sums go through `epi`; else split s stores its sums at
// part + (s M + row) ldpart.
//
// Persistent: one CTA per SM, or pairs of CTAs, walk the items.  Two warps feed a ring of stages by
// TMA, one per operand, warp kMmaWarp (of the pair's first CTA) issues the products into one of two
// TMEM accumulators, and sixteen warps take the other accumulator out (four per TMEM lane
// quarter, a quarter of the columns each), so that a tile's epilogue runs under the next
// tile's products.  A lane holds a row and stores whole 32-byte sectors of it.
//
// The tensor core drops what does not fit when it adds to its fp32 accumulator (measured on
// all-positive sums: 4.4e-8 of the sum lost per 16-deep step in the mean; a whole unit of it, 1.2e-7, at most).  So an
// accumulator takes at most g.chunk k-blocks; the warps that take it out add the chunks up in registers, rounding to nearest.
//
// Measured (single calls on one GB300, the library's product of the same operands beside it): 32768 x 1024 x 4096 bf16 153 to
// 156 us (1.78 PFLOP/s, 95 % of the measured peak; library 140 to 142), with GELU 166 to 171, with GELU and pre 187 to 191
// (its boxes take shared memory's cycles from the products' operands); dx 154 (146), dW 158 to 160 (142 to 146; 64 tiles for
// 76 pairs of SMs); fp32, 4096 x 1024 x 4096: 132 us, preparation included.
// The products of 256 x 256 tiles run at the tensor rate but for the ends of tiles; calls one after another
// run into the power limit, as the library's do.
struct GemmJob {
    CUtensorMap a, b, y, pre;
    GemmShape g;
    Epi epi;
    float* part;
    int64_t ldpart;
    int part_access;   // row_access() of part: a workspace need only be 16-byte aligned
};

// The job's items first, first + stride, ... by one CTA, or a pair.
template <int CTAS, int BN, bool SUM, bool A_MN, bool B_MN>
__device__ __forceinline__ void gemm_job(const GemmJob& job, const int first, const int stride, int* status) {
    using C = GemmCfg<CTAS, BN, SUM>;
    const CUtensorMap &map_a = job.a, &map_b = job.b, &map_y = job.y, &map_pre = job.pre;
    const GemmShape& g = job.g;
    const Epi& epi = job.epi;
    float* __restrict__ part = job.part;
    const int64_t ldpart = job.ldpart;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ GemmBars bars;
    __shared__ alignas(16) float bias_s[kEpiWarps][BN / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0;
    if (threadIdx.x == kTmaWarp * 32) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bars.acc_full[a], 1);
            mbar_init(&bars.acc_empty[a], CTAS * kEpiWarps);
        }
        mbar_init(&bars.fin, 1);
        bars.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == kMmaWarp) {
        if (CTAS == 2) tmem_alloc_pair(&bars.tmem_base, C::kTmemCols);
        else tmem_alloc(&bars.tmem_base, C::kTmemCols);
    }
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync();   // both CTAs' barriers exist
    tc_fence_after();
    const uint32_t tbase = bars.tmem_base;
    volatile int* abort_flag = &bars.abort;
    pdl_trigger();   // the call's next kernel may start; it waits for this one before it reads
    pdl_wait();      // the kernels before this one have finished
    const int items = g.items();

    if (warp == kTmaWarp || warp == kTmaWarp + 1) {
        // The whole warp runs the loop and waits; the elected lane issues (from a diverged warp a
        // TMA instruction costs far more).  MN: the operand's rows run along the contraction; `blocks`
        // of 64 elements along D; r0: this CTA's first row or column of the tile.
        auto feed = [&](auto is_a_, auto mn_, const CUtensorMap& map, bool whole, int across) {
            constexpr bool is_a = decltype(is_a_)::value, mn = decltype(mn_)::value;
            constexpr int blocks = is_a ? 2 : BN / CTAS / 64;
            Ring<C::kStages> ring(bars.empty, 1);   // the first time round finds every stage empty
            uint32_t loads = 0;
            bool ok = true;
            const uint32_t full0 = CTAS == 2 ? map_to_rank(bars.full, 0) : 0;   // a pair's stages count on its first CTA's barriers
            auto load_stage = [&](uint32_t st, int kb, int r0, int plane) {
                if (elect_one()) {
                    uint64_t* full = &bars.full[st];
                    if (is_a && rank == 0) mbar_arrive_expect_tx(full, CTAS * C::kStage);
                    uint8_t* dst = smem + st * C::kStage + (is_a ? 0 : kStageA);
                    auto load = [&](int at, int x, int y, int z) {
                        if (CTAS == 2) tma_load_4d_pair(dst + at, &map, x, y, z, plane, full0 + 8 * st);
                        else tma_load_4d(dst + at, &map, x, y, z, plane, full);
                    };
                    if (!mn) {
                        load(0, kb * kBK, r0, 0);
                    } else if (whole) {
                        load(0, 0, kb * kBK, r0 / 64);
                    } else {
#pragma unroll
                        for (int b = 0; b < blocks; ++b) load(b * 8192, r0 + 64 * b, kb * kBK, 0);
                    }
                }
                __syncwarp();
            };
            for (int i = first; ok && i < items; i += stride) {
                const Item w = item_of(g, i);
                const int r0 = (is_a ? w.m : w.n) * across * CTAS + across * (int)rank;
                uint32_t st;
                if (g.planes == 1) {
                    for (int kb = w.lo; kb < w.hi; ++kb, ++loads) {
                        if (!(ok = ring.next(st, abort_flag))) break;
                        load_stage(st, kb, r0, 0);
                    }
                } else {
                    for (int kb = w.lo; ok && kb < w.hi; ++kb)
                        for (int j = 0; j < 3; ++j, ++loads) {
                            if (!(ok = ring.next(st, abort_flag))) break;
                            load_stage(st, kb, r0, j == 0 ? 2 : j - 1);   // lo, hi, mid: as they are used
                        }
                }
            }
            if (!ok && lane == 0) tc::fail(&bars.abort, status);
            // Nothing may still be on its way into shared memory, or to a barrier in it, when the
            // CTA ends: every stage's last load has landed, and, unless a wait gave up, has been
            // consumed by products that have completed.  (A pair's second CTA has no barrier of its
            // own for its loads; where its wait gave up, they were issued that wait's limit ago.)
            int never = 0;
            for (uint32_t b = loads > (uint32_t)C::kStages ? loads - C::kStages : 0; b < loads; ++b) {
                const uint32_t s = b % C::kStages, p = (b / C::kStages) & 1;
                if (rank == 0) mbar_wait_all(&bars.full[s], p, &never, tc::kWaitNs);
                if (ok) ok = mbar_wait_all(&bars.empty[s], p, abort_flag, tc::kWaitNs);
            }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (warp == kTmaWarp) feed(Yes(), std::integral_constant<bool, A_MN>(), map_a, g.whole_a, 128);
        else feed(No(), std::integral_constant<bool, B_MN>(), map_b, g.whole_b, BN / CTAS);
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            constexpr uint32_t id = idesc_bf16(C::kBM, BN, A_MN, B_MN);
            // along the contraction: 8-row groups 1024 bytes apart, 32 bytes per k-step; along the
            // row: 64-element blocks 8192 bytes apart, 8-deep groups 1024 bytes apart, 2048 bytes per k-step
            const SmemDesc da = smem_desc_split(smem_u32(smem), A_MN ? 8192 : 16, 1024, 2);
            const SmemDesc db = smem_desc_split(smem_u32(smem) + kStageA, B_MN ? 8192 : 16, 1024, 2);
            Ring<C::kStages> ring(bars.full, 0);
            uint32_t n = 0;
            bool ok = true;
            auto landed = [&](uint32_t& s) {
                const bool got = ring.next(s, abort_flag);
                tc_fence_after();
                return got;
            };
            // one lane: D (+)= the k-block of A in stage sa times that of B in stage sb
            auto product = [&](uint32_t d, uint32_t sa, uint32_t sb, bool add) {
                const uint32_t oa = sa * C::kStage, ob = sb * C::kStage;
#pragma unroll
                for (int ks = 0; ks < kBK / 16; ++ks) {
                    const uint64_t ad = desc_at(da, oa + (A_MN ? 2048 : 32) * ks);
                    const uint64_t bd = desc_at(db, ob + (B_MN ? 2048 : 32) * ks);
                    if (CTAS == 2) mma_ss_pair(d, ad, bd, id, add || ks > 0);
                    else mma_ss(d, ad, bd, id, add || ks > 0);
                }
            };
            auto commit = [&](uint64_t* bar) {
                if (CTAS == 2) mma_commit_pair(bar);
                else mma_commit(bar);
            };
            for (int i = first; ok && i < items; i += stride) {
                const Item w = item_of(g, i);
                for (int c0 = w.lo; ok && c0 < w.hi; c0 += g.chunk, ++n) {
                    const int c1 = c0 + g.chunk < w.hi ? c0 + g.chunk : w.hi;
                    const uint32_t a = n & 1, d = tbase + a * BN;
                    if (n >= 2 && !mbar_wait_all(&bars.acc_empty[a], ((n >> 1) - 1) & 1, abort_flag, tc::kWaitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int kb = c0; kb < c1; ++kb) {
                        if (g.planes == 1) {
                            uint32_t s;
                            if (!(ok = landed(s))) break;
                            if (elect_one()) {
                                product(d, s, s, kb > c0);
                                commit(&bars.empty[s]);
                                if (kb == c1 - 1) commit(&bars.acc_full[a]);
                            }
                            __syncwarp();
                        } else {
                            // three stages hold lo, hi, mid; each is given back after its last term
                            uint32_t lo, hi, mid;
                            if (!(ok = landed(lo) && landed(hi))) break;
                            if (elect_one()) {
                                product(d, lo, hi, kb > c0);
                                product(d, hi, lo, true);
                                commit(&bars.empty[lo]);
                            }
                            __syncwarp();
                            if (!(ok = landed(mid))) break;
                            if (elect_one()) {
                                product(d, mid, mid, true);
                                product(d, mid, hi, true);
                                product(d, hi, mid, true);
                                commit(&bars.empty[mid]);
                                product(d, hi, hi, true);
                                commit(&bars.empty[hi]);
                                if (kb == c1 - 1) commit(&bars.acc_full[a]);
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            if (!ok) {
                if (lane == 0) tc::fail(&bars.abort, status);
                int never = 0;
                if (elect_one()) {
                    if (CTAS == 2) mma_commit_pair(&bars.fin);
                    else mma_commit(&bars.fin);
                }
                __syncwarp();
                mbar_wait_all(&bars.fin, 0, &never, tc::kWaitNs);
            }
        }
    } else if (warp < kEpiWarps) {
        constexpr int CW = C::kCW, NC = C::kCols / C::kCW;
        const int q = warp & 3, c0 = (warp >> 2) * C::kCols;
        const uint32_t tl = tbase + ((uint32_t)(32 * q) << 16) + c0, bias = smem_u32(bias_s[warp]);
        uint8_t* stg = smem + C::kStages * C::kStage + warp * C::kStg;
        constexpr int NB = C::kCols > 32 ? C::kCols / 32 : 1;
        float next_b[NB];
        auto fetch_bias = [&](int col) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                next_b[j] = epi.bias && col + 32 * j + lane < g.N ? __ldg(epi.bias + col + 32 * j + lane) : 0.f;
        };
        if (first < items) fetch_bias(item_of(g, first).n * BN + c0);
        uint32_t n = 0;
        bool ok = true;
        for (int i = first; ok && i < items; i += stride) {
            const Item w = item_of(g, i);
            const int64_t row = (int64_t)w.m * C::kBM + 128 * rank + 32 * q + lane;
            const int col0 = w.n * BN + c0;
            // this warp's columns of the bias, fetched an item ahead
            __syncwarp();
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (NB > 1 || lane < C::kCols) bias_s[warp][32 * j + lane] = next_b[j];
            __syncwarp();
            if (i + stride < items) fetch_bias(item_of(g, i + stride).n * BN + c0);
            float sum[SUM ? NC : 1][CW];
#pragma unroll
            for (int c = 0; c < (SUM ? NC : 1); ++c)
#pragma unroll
                for (int j = 0; j < CW; ++j) sum[c][j] = 0.f;
            for (int k0 = w.lo; k0 < w.hi; k0 += g.chunk, ++n) {
                const uint32_t a = n & 1;
                if (!mbar_wait_all(&bars.acc_full[a], (n >> 1) & 1, abort_flag, tc::kWaitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool last = k0 + g.chunk >= w.hi;
#pragma unroll(SUM ? NC : 1)
                for (int c = 0; c < NC; ++c) {
                    const int col = col0 + c * CW, live = g.N - col;
                    uint32_t v[CW];
                    if constexpr (CW == 32) tmem_ld_x32(tl + a * BN + c * CW, v);
                    else tmem_ld_x16(tl + a * BN + c * CW, v);
                    tmem_wait_ld();
                    if (c == NC - 1) {   // the accumulator is out
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (CTAS == 2) mbar_arrive_relaxed_cluster(map_to_rank(&bars.acc_empty[a], 0));
                            else mbar_arrive_relaxed(&bars.acc_empty[a]);
                        }
                    }
                    float(&f)[CW] = sum[SUM ? c : 0];
#pragma unroll
                    for (int j = 0; j < CW; ++j) f[j] = SUM ? f[j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
                    if (!SUM || last) {
                        if (C::kBulk && (epi.bulk || epi.single) && !part) {
                            if constexpr (C::kBulk) {
                                if (live > 0 && row - lane < g.M)
                                    epilogue_box(epi, &map_y, &map_pre, row - lane, g.M, col, live, f, bias + 4 * c * CW,
                                                 smem_u32(stg));
                            }
                        } else if (row < g.M && live > 0) {
                            if (part) put_row<CW>(part, ((int64_t)w.s * g.M + row) * ldpart + col, true, f, (live + 7) & ~7,
                                                  job.part_access);
                            else epilogue<CW>(epi, row, col, live, f, bias + 4 * c * CW);
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (!ok && lane == 0) tc::fail(&bars.abort, status);
        if (C::kBulk && lane == 0) bulk_wait();   // the last boxes are written
    }
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync();   // neither CTA's shared memory or barriers are used by the other any more
    if (warp == kMmaWarp) {
        tc_fence_after();
        if (CTAS == 2) tmem_dealloc_pair(tbase, C::kTmemCols);
        else tmem_dealloc(tbase, C::kTmemCols);
    }
}

template <int CTAS, int BN, bool SUM, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kGemmThreads, 1) linear_gemm(const __grid_constant__ GemmJob job, int* status) {
    gemm_job<CTAS, BN, SUM, A_MN, B_MN>(job, blockIdx.x / CTAS, gridDim.x / CTAS, status);
}

// Both products of a backward in one launch, where each alone would leave pairs of SMs idle and pay a launch: the first
// units_x pairs make da W^T, the others x^T da (device time of the call, before and after: 6800x256x1024 bf16 with GELU
// 34.8 and 29.1 us, 4096x512x512 fp32 45.8 and 39.9, 512x512x2048 bf16 23.0 and 18.1).
constexpr int kBothBN = 128;
template <bool SUM>
__global__ void __launch_bounds__(kGemmThreads, 1)
linear_gemm_both(const __grid_constant__ GemmJob x, const __grid_constant__ GemmJob w, const int units_x, int* status) {
    const int unit = blockIdx.x / 2, units = gridDim.x / 2;
    if (unit < units_x) gemm_job<2, kBothBN, SUM, false, false>(x, unit, units_x, status);
    else gemm_job<2, kBothBN, SUM, true, true>(w, unit - units_x, units - units_x, status);
}

// The end of a call in one launch: the sums that the product kernel left (of the contraction's splits,
// added in a fixed order, and any whose rows can only be reached by single elements) through the
// epilogue (of up to two products: the first j0.ctas CTAs, the next j1.ctas), and the column sums of the
// preparation's partial rows (the CTAs from there on, 32 columns each, as col_sum in gt_norm.cu).  A thread takes 8 consecutive columns of a row, or
// single: every 32nd of 256, so that a warp's accesses are consecutive elements (4099 x 321 x 1001, fp32 y and
// residual: 58 us with those in the product kernel's epilogue, where a lane holds a row, 13 + 9 us so).
constexpr int kJoinThreads = 256;
struct ColSum {
    const float* part;
    float* out;
    int rows, cols;
};

__host__ __device__ __forceinline__ int64_t join_threads(int m, int n, bool single) {
    return (int64_t)m * (single ? (n + 255) / 256 * 32 : (n + 7) / 8);
}

// Elements at, at + 32, ... (eight, of which those below `live` exist).
__device__ __forceinline__ void load_every32(const void* p, int64_t at, bool f32, int live, float (&v)[8]) {
    if (f32) {
        const float* q = static_cast<const float*>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < live) v[i] = q[32 * i];
    } else {
        const bf16* q = static_cast<const bf16*>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < live) v[i] = __bfloat162float(q[32 * i]);
    }
}
__device__ __forceinline__ void store_every32(void* p, int64_t at, bool f32, int live, const float (&v)[8]) {
    if (f32) {
        float* q = static_cast<float*>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < live) q[32 * i] = v[i];
    } else {
        bf16* q = static_cast<bf16*>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < live) q[32 * i] = __float2bfloat16_rn(v[i]);
    }
}

struct JoinJob {
    int ctas, m, n, splits;
    const float* part;
    int64_t ldpart;
    Epi epi;
};

__global__ void __launch_bounds__(kJoinThreads)
linear_join(const __grid_constant__ JoinJob j0, const __grid_constant__ JoinJob j1, const ColSum cs) {
    __shared__ alignas(16) float bias_s[kJoinThreads][8];
    pdl_trigger();
    pdl_wait();
    const int join = j0.ctas + j1.ctas;
    if ((int)blockIdx.x >= join) {
        float(&red)[kJoinThreads][8] = bias_s;
        const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
        const int i = ((int)blockIdx.x - join) * 32 + tx;
        float acc = 0.f;
        if (i < cs.cols) {
#pragma unroll 8
            for (int p = ty; p < cs.rows; p += kJoinThreads / 32) acc += __ldcg(cs.part + (int64_t)p * cs.cols + i);
        }
        red[tx][ty] = acc;
        __syncthreads();
        if (ty == 0 && i < cs.cols) {
            float sum = 0.f;
#pragma unroll
            for (int r = 0; r < kJoinThreads / 32; ++r) sum += red[tx][r];
            cs.out[i] = sum;
        }
        return;
    }
    const bool second = (int)blockIdx.x >= j0.ctas;
    // (values, not references: those of a chosen parameter would be read through the memory pipe)
    const Epi epi = second ? j1.epi : j0.epi;
    const int m = second ? j1.m : j0.m, n = second ? j1.n : j0.n, splits = second ? j1.splits : j0.splits;
    const int64_t ldpart = second ? j1.ldpart : j0.ldpart;
    const float* __restrict__ part = second ? j1.part : j0.part;
    const int64_t idx = (int64_t)(blockIdx.x - (second ? j0.ctas : 0)) * kJoinThreads + threadIdx.x;
    if (idx >= join_threads(m, n, epi.single)) return;
    const int64_t plane = (int64_t)m * ldpart;
    float v[8] = {};
    if (epi.single) {
        const int per_row = (n + 255) / 256 * 32;
        const int64_t row = idx / per_row;
        const int at = (int)(idx - row * per_row), col = at / 32 * 256 + at % 32;   // then col + 32, ...
        // the residual and the bias are on their way while the sums are added
        float r[8] = {}, b[8] = {};
        if (epi.r) load_every32(epi.r, row * epi.ldr + col, epi.y_f32, n - col, r);
        if (epi.bias) load_every32(epi.bias, col, true, n - col, b);
        for (int s = 0; s < splits; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + 32 * i < n) v[i] += __ldcg(part + s * plane + row * ldpart + col + 32 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
        if (epi.pre) store_every32(epi.pre, row * epi.ldpre + col, epi.pre_f32, n - col, v);
        if (epi.gelu_act) apply_gelu<8>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
        store_every32(epi.y, row * epi.ldy + col, epi.y_f32, n - col, v);
        return;
    }
    const int per_row = (n + 7) / 8;
    const int64_t row = idx / per_row;
    const int col = (int)(idx - row * per_row) * 8, live = n - col;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        float f[8];
        unpack8(load8_cg(part + s * plane + row * ldpart + col), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) bias_s[threadIdx.x][i] = epi.bias && i < live ? __ldg(epi.bias + col + i) : 0.f;
    epilogue<8>(epi, row, col, live, v, smem_u32(bias_s[threadIdx.x]));
}

// -------------------------------------------------------------- small products
//
// fp32 products of a few tens of millions of multiplications spend their time on launches: here a
// whole call is one kernel on the fp32 pipes, exact products with no operand split first.  A CTA makes a 64 x 64
// tile, 4 x 4 sums to a thread, its contraction in steps of 32 through shared memory, the next step's
// elements in registers meanwhile.  Forward: tiles of y.  Backward: tiles of dx, then tiles of dw, each by a
// cluster of CTAs that share its rows and add up their sums in a fixed order through each other's shared memory; the
// first row of these tiles makes db too.  da is formed from dy and pre where it is read.
// Elements move singly, consecutive ones to consecutive threads, so any rows will do.
struct Small {
    const float *x, *w, *dy, *pre;
    int64_t ldx, ldw, lddy, ldpre;
    int m, k, n;
    Epi out, dw;          // y or dx; dw
    float* db;
    int tiles;            // of y or dx (backward: their CTAs, whole clusters); then the clusters of dw and db
};

constexpr int kSmT = 64, kSmK = 32, kSmThreads = 256, kSmPitch = kSmT + 4, kSmCluster = 8;

struct SmallSmem {
    union {
        struct {
            float a[kSmK][kSmPitch], b[kSmK][kSmPitch];
        } in;
        struct {
            float tile[kSmT][kSmT], col[kSmT];   // a CTA's share of a dw tile and of db
        } out;
    };
};

// acc += A B over depths d0 .. d1 - 1: A(i, j) is the tile's row i and B(i, j) its column i at depth j, zero outside, as a
// pair (v, a): the element is v gelu'(a) where pre is set for that operand (A_DA, B_DA), else v.
// ALONG: memory runs along the depth.  each(b): every element of B, in the order this thread reads them.
template <bool A_ALONG, bool B_ALONG, bool A_DA, bool B_DA, typename FA, typename FB, typename FE>
__device__ __forceinline__ void small_tile(int d0, int d1, FA A, FB B, FE each, bool product, bool gelu,
                                           float (&acc)[4][4], SmallSmem& S) {
    constexpr int E = kSmT * kSmK / kSmThreads;
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const GaussK gk = gauss_constants();
    // element e of a thread: ALONG, depth t % 32, row t / 32 + 8 e; else depth t / 64 + 4 e, row t % 64
    auto row = [&](bool along, int e) { return along ? t / 32 + 8 * e : t & 63; };
    auto dep = [&](bool along, int e) { return along ? t & 31 : t / 64 + 4 * e; };
    float2 a[E], b[E];
    auto fetch = [&](int at) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            a[e] = product ? A(row(A_ALONG, e), at + dep(A_ALONG, e)) : make_float2(0.f, 0.f);
            b[e] = B(row(B_ALONG, e), at + dep(B_ALONG, e));
        }
    };
    auto value = [&](bool da, float2 v) { return da && gelu ? v.x * gelu_grad2(gk, make_float2(v.y, v.y)).x : v.x; };
    fetch(d0);
    for (int at = d0; at < d1; at += kSmK) {
        __syncthreads();   // the tile before has been read
#pragma unroll
        for (int e = 0; e < E; ++e) {
            S.in.a[dep(A_ALONG, e)][row(A_ALONG, e)] = value(A_DA, a[e]);
            const float v = value(B_DA, b[e]);
            S.in.b[dep(B_ALONG, e)][row(B_ALONG, e)] = v;
            each(v);
        }
        __syncthreads();
        if (at + kSmK < d1) fetch(at + kSmK);
        if (!product) continue;
#pragma unroll 8
        for (int d = 0; d < kSmK; ++d) {
            const float4 u = *reinterpret_cast<const float4*>(&S.in.a[d][4 * ty]);
            const float4 v = *reinterpret_cast<const float4*>(&S.in.b[d][4 * tx]);
            const float p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(p[i], q[j], acc[i][j]);
        }
    }
}

__device__ __forceinline__ void small_store(const Epi& e, int M, int N, int r0, int c0, float (&acc)[4][4]) {
    const int row0 = r0 + 4 * (threadIdx.x >> 4), col0 = c0 + 4 * (threadIdx.x & 15);
    const GaussK gk = gauss_constants();
    const float* r = static_cast<const float*>(e.r);
    float b[4], res[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        b[j] = e.bias && col0 + j < N ? __ldg(e.bias + col0 + j) : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            res[i][j] = r && row0 + i < M && col0 + j < N ? r[(row0 + i) * e.ldr + col0 + j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + i;
        if (row >= M) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = col0 + j;
            if (col >= N) break;
            float a = acc[i][j] + b[j];
            if (e.pre) static_cast<float*>(e.pre)[row * e.ldpre + col] = a;
            if (e.gelu_act) a = gelu2(gk, make_float2(a, a)).x;
            static_cast<float*>(e.y)[row * e.ldy + col] = a + res[i][j];
        }
    }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <bool BACKWARD>
__global__ void __launch_bounds__(kSmThreads) linear_small(const Small p) {
    __shared__ alignas(16) SmallSmem S;
    float acc[4][4] = {};
    auto none = [](float) {};
    if constexpr (!BACKWARD) {
        const int tn = (p.n + kSmT - 1) / kSmT, r0 = blockIdx.x / tn * kSmT, c0 = blockIdx.x % tn * kSmT;
        small_tile<true, false, false, false>(
            0, p.k,
            [&](int i, int d) {
                return make_float2(r0 + i < p.m && d < p.k ? __ldg(p.x + (int64_t)(r0 + i) * p.ldx + d) : 0.f, 0.f);
            },
            [&](int i, int d) {
                return make_float2(c0 + i < p.n && d < p.k ? __ldg(p.w + (int64_t)d * p.ldw + c0 + i) : 0.f, 0.f);
            },
            none, true, false, acc, S);
        small_store(p.out, p.m, p.n, r0, c0, acc);
    } else {
        const bool gelu = p.pre != nullptr;
        auto da = [&](int row, int col) {
            const bool in = row < p.m && col < p.n;
            return make_float2(in ? __ldg(p.dy + (int64_t)row * p.lddy + col) : 0.f,
                               in && gelu ? __ldg(p.pre + (int64_t)row * p.ldpre + col) : 0.f);
        };
        if ((int)blockIdx.x < p.tiles) {
            const int tn = (p.k + kSmT - 1) / kSmT, r0 = blockIdx.x / tn * kSmT, c0 = blockIdx.x % tn * kSmT;
            if (r0 >= p.m) return;   // up to a whole cluster; its CTAs share nothing
            small_tile<true, true, true, false>(
                0, p.n, [&](int i, int d) { return da(r0 + i, d); },
                [&](int i, int d) {
                    return make_float2(c0 + i < p.k && d < p.n ? __ldg(p.w + (int64_t)(c0 + i) * p.ldw + d) : 0.f, 0.f);
                },
                none, true, gelu, acc, S);
            small_store(p.out, p.m, p.k, r0, c0, acc);
        } else {
            const int b = (blockIdx.x - p.tiles) / kSmCluster, tn = (p.n + kSmT - 1) / kSmT;
            const int r0 = b / tn * kSmT, c0 = b % tn * kSmT;
            const int rank = (int)cluster_ctarank();
            const bool product = p.dw.y != nullptr;
            const int t = threadIdx.x;
            float sum = 0.f;   // of column c0 + t % 64, over a quarter of this CTA's rows
            const int lo = (int)((int64_t)p.m * rank / kSmCluster), hi = (int)((int64_t)p.m * (rank + 1) / kSmCluster);
            small_tile<false, false, false, true>(
                lo, hi,
                [&](int i, int d) {
                    return make_float2(r0 + i < p.k && d < hi ? __ldg(p.x + (int64_t)d * p.ldx + r0 + i) : 0.f, 0.f);
                },
                [&](int i, int d) { return d < hi ? da(d, c0 + i) : make_float2(0.f, 0.f); }, [&](float v) { sum += v; },
                product, gelu, acc, S);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) S.out.tile[4 * (t >> 4) + i][4 * (t & 15) + j] = acc[i][j];
            if (t < kSmT) S.out.col[t] = 0.f;
            for (int q = 0; q < kSmThreads / kSmT; ++q) {   // the quarters in order
                __syncthreads();
                if (t / kSmT == q) S.out.col[t & 63] += sum;
            }
            cluster_sync();
            // rows 8 rank .. 8 rank + 7 of the tile, and the first CTA its part of db
            if (product) {
#pragma unroll
                for (int e = 0; e < kSmT * kSmT / kSmCluster / kSmThreads; ++e) {
                    const int i = kSmT / kSmCluster * rank + t / 64 + 4 * e, j = t & 63;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < kSmCluster; ++q) v += ld_cluster_f32(map_to_rank(&S.out.tile[i][j], q));
                    if (r0 + i < p.k && c0 + j < p.n)
                        static_cast<float*>(p.dw.y)[(int64_t)(r0 + i) * p.dw.ldy + c0 + j] = v;
                }
            }
            if (p.db && r0 == 0 && rank == 0 && t < kSmT) {
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < kSmCluster; ++q) v += ld_cluster_f32(map_to_rank(&S.out.col[t], q));
                if (c0 + t < p.n) p.db[c0 + t] = v;
            }
            cluster_sync();   // the CTAs' shared memory has been read
        }
    }
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

struct GemmPlan {
    GemmShape g;
    int ctas, bn;
    bool sum;    // the kernel's SUM: several chunks to an item
    double us;   // modelled
};

// k-blocks an accumulator may sum: 256 deep for an fp32 result (16 steps: 7e-7 of an all-positive sum lost by the mean
// above, 1.9e-6 at most; 3e-7 measured), 4096 deep for a bf16 one (1.1e-5 and 3e-5, against a rounding of 3.9e-3); one
// k-block of split operands, whose large terms are the last four of 24 steps.
int chunk_of(bool f32_out, int planes) { return planes == 3 ? 1 : f32_out ? 4 : 64; }

// The tile and the splits of the contraction with the least modelled time, in microseconds as measured:
// what a product costs but its steps, a 64-deep step, what a further tile of the same CTAs adds (much with fp32
// operands, whose accumulators change with every step: a tile's results are in the way of the next one's sums); for splits
// the partial sums' traffic and the joining kernel.  (256 x 256 tiles step at 94 % of the tensor rate, 256 x 128
// at 64 %, 128 x 64 at 13 %; the smaller tiles are for results that leave SMs idle otherwise: 4096x512x512 bf16
// 8.0, 7.0 and 8.3 us, 512 nodes of 64x64 fp32 8.5, 7.4 and 6.7 us.)
struct TileCost {
    int ctas, bn;
    double once, step, more, step3, more3;   // (3: of fp32 operands)
};
constexpr TileCost kTileCost[3] = {
    {2, 256, 6.2, 0.264, 0.8, 1.57, 6.0}, {2, kBothBN, 5.2, 0.200, 0.6, 0.79, 4.0}, {1, 64, 4.0, 0.252, 0.5, 1.09, 1.5}};
constexpr double kJoinUs = 4.0;
double join_traffic_us(int M, int N, int splits) { return (double)M * N * (splits + 2) * 4 / 2.5e6; }

// The time of a product's steps on `units` CTAs or pairs, and whether so many splits are sensible.
bool cost_of(const TileCost& t, int M, int N, int K, int planes, int units, int splits, double* us) {
    const int bm = 128 * t.ctas, kb = (K + kBK - 1) / kBK;
    const int64_t n = (int64_t)((M + bm - 1) / bm) * ((N + t.bn - 1) / t.bn);
    if (splits > 1 && (splits * n > units || kb / splits < (planes == 1 ? 4 : 2))) return false;
    const int64_t waves = (n * splits + units - 1) / units;
    *us = waves * ((kb + splits - 1) / splits) * (planes == 1 ? t.step : t.step3) + (waves - 1) * (planes == 1 ? t.more : t.more3);
    return true;
}

GemmPlan make_plan(const TileCost& t, int M, int N, int K, int planes, bool f32_out, int splits, double us) {
    const int bm = 128 * t.ctas, tm = (M + bm - 1) / bm, tn = (N + t.bn - 1) / t.bn;
    GemmPlan p{};
    GemmShape& g = p.g;
    g = GemmShape{M, N, (K + kBK - 1) / kBK, planes, chunk_of(f32_out, planes), tm, tn, M % 64 == 0, N % 64 == 0, splits};
    g.by_tiles = Divider::of(tm * tn);
    g.by_group = Divider::of(kGroup * tn);
    g.by_tail = Divider::of(tm % kGroup ? tm % kGroup : kGroup);
    g.by_splits = Divider::of(splits);
    p.ctas = t.ctas;
    p.bn = t.bn;
    p.sum = t.ctas == 1 || (g.kblocks + splits - 1) / splits > g.chunk;
    p.us = us;
    return p;
}

int next_splits(int sp) { return sp < 8 ? sp + 1 : sp + sp / 4; }

GemmPlan plan_gemm(int M, int N, int K, int planes, bool f32_out) {
    const TileCost* best = nullptr;
    int splits = 1;
    double best_us = 1e30, us;
    for (const TileCost& t : kTileCost) {
        const int units = num_sms() > t.ctas ? num_sms() / t.ctas : 1;
        for (int sp = 1; sp <= 128 && cost_of(t, M, N, K, planes, units, sp, &us); sp = next_splits(sp)) {
            us += t.once + (sp > 1 ? kJoinUs + join_traffic_us(M, N, sp) : 0.0);
            if (us < best_us) {
                best_us = us;
                best = &t;
                splits = sp;
            }
        }
    }
    return make_plan(*best, M, N, K, planes, f32_out, splits, best_us);
}

// Whether the product kernel leaves its sums to linear_join: splits, and rows that can only be reached by single
// elements, unless its staging tiles can (bf16: GemmCfg's kBulk).  For fp32 results the joining kernel, with its many
// more warps, is the faster way (4099x321x1001 with a fp32 residual: 25 us, through staging tiles 35).
bool leaves_sums(const GemmPlan& p, bool single, bool f32_out) { return p.g.splits > 1 || (single && (f32_out || p.sum)); }
size_t part_floats(const GemmPlan& p, bool single, bool f32_out) {
    return leaves_sums(p, single, f32_out) ? (size_t)p.g.splits * p.g.M * pad8(p.g.N) : 0;
}

// The plans of a backward's products: each for a launch of its own, or, where that is modelled as faster, for one launch,
// of which units_x pairs make dx.  A call for one of them uses the same plan, so that its result is the same.
struct BwdPlan {
    GemmPlan x, w;
    int units_x = 0;   // 0: launches of their own
};

BwdPlan plan_bwd(int m, int k, int n, int planes, bool f32_out) {
    BwdPlan p;
    p.x = plan_gemm(m, k, n, planes, f32_out);
    p.w = plan_gemm(k, n, m, planes, f32_out);
    const TileCost& t = kTileCost[1];
    const int units = num_sms() / 2;
    double best_us = p.x.us + p.w.us;
    GemmPlan x{}, w{};
    constexpr int kShares = 12;
    for (int i = 1; i < kShares && units >= kShares; ++i) {
        const int ux = units * i / kShares;
        int sx = 1, sw = 1;
        double tx, tw, us;
        const auto steps = [&](int M, int N, int K, int u, int& splits, double& best) {
            cost_of(t, M, N, K, planes, u, 1, &best);
            const int64_t n = (int64_t)((M + 255) / 256) * ((N + t.bn - 1) / t.bn);
            const int most = (int)std::min<int64_t>({u / n, (K + kBK - 1) / kBK / (planes == 1 ? 4 : 2), 128});
            if (most > 1 && cost_of(t, M, N, K, planes, u, most, &us) && (us += join_traffic_us(M, N, most)) < best) {
                best = us;
                splits = most;
            }
        };
        steps(m, k, n, ux, sx, tx);
        steps(k, n, m, units - ux, sw, tw);
        const double total = t.once + (tx > tw ? tx : tw) + (sx > 1 || sw > 1 ? kJoinUs : 0.0);
        if (total >= best_us) continue;
        best_us = total;
        x = make_plan(t, m, k, n, planes, f32_out, sx, total);
        w = make_plan(t, k, n, m, planes, f32_out, sw, total);
        x.sum = w.sum = x.sum || w.sum;   // one kernel serves both
        p.units_x = ux;
    }
    if (p.units_x > 0) {
        p.x = x;
        p.w = w;
    }
    return p;
}

template <int CTAS, int BN, bool SUM>
int make_job(GemmJob* job, const GemmPlan& p, const CUtensorMap& ma, const CUtensorMap& mb, const Epi& e, float* part) {
    *job = GemmJob{ma, mb, {}, {}, p.g, e, part, pad8(p.g.N), row_access(part, pad8(p.g.N), 4)};
    Epi& epi = job->epi;
    CUtensorMap &my = job->y, &mp = job->pre;
    // (whole 16 bytes of columns: a box that ends at an odd column of bf16 writes one column more)
    if (GemmCfg<CTAS, BN, SUM>::kBulk && !part && !epi.single && !epi.y_f32 && !epi.pre_f32 && p.g.N % 8 == 0) {
        const CUtensorMapDataType ty = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (!make_map_2d(&my, epi.y, ty, p.g.M, p.g.N, epi.ldy * 2, 32, kBoxCols, CU_TENSOR_MAP_SWIZZLE_64B) ||
            (epi.pre && !make_map_2d(&mp, epi.pre, ty, p.g.M, p.g.N, epi.ldpre * 2, 32, kBoxCols, CU_TENSOR_MAP_SWIZZLE_64B)))
            return GT_ERR_CUDA;
        epi.bulk = true;
    }
    return GT_OK;
}

// kern on `units` CTAs or pairs; `allowed`: its own set of devices.
template <int CTAS, int BN, bool SUM, typename... P, typename... A>
int launch_products(void (*kern)(P...), std::atomic<uint64_t>& allowed, int units, bool follows, cudaStream_t s,
                    const A&... args) {
    using C = GemmCfg<CTAS, BN, SUM>;
    if (!allow_smem(allowed, reinterpret_cast<const void*>(kern), C::kSmem)) return GT_ERR_CUDA;
    int* status = device_status_ptr();
    if (!status) return GT_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CTAS * units));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = follows;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS;
    LaunchScope ls("linear_gemm", s);
    return cudaLaunchKernelEx(&cfg, kern, args..., status) == cudaSuccess ? check_launch() : GT_ERR_CUDA;
}

template <int CTAS, int BN, bool SUM, bool A_MN, bool B_MN>
int launch_gemm(const GemmPlan& p, const CUtensorMap& ma, const CUtensorMap& mb, const Epi& epi, float* part,
                bool follows, cudaStream_t s) {
    GemmJob job;
    const int rc = make_job<CTAS, BN, SUM>(&job, p, ma, mb, epi, part);
    if (rc != GT_OK) return rc;
    static std::atomic<uint64_t> allowed;
    const int sms = num_sms(), units = sms > CTAS ? sms / CTAS : 1, items = p.g.items();
    return launch_products<CTAS, BN, SUM>(linear_gemm<CTAS, BN, SUM, A_MN, B_MN>, allowed, items < units ? items : units,
                                          follows, s, job);
}

// The map of an operand of which a CTA takes `across` rows (columns, where mn) and 64 of the
// contraction at a time.  Blocks of 64 elements make the 128 bytes of a swizzled row: an operand with
// rows along D that is whole in them (mn, whole) comes as [plane][block][row][64], and all of a CTA's
// blocks with one load; else a load brings one block, ends filled with zeros.
bool operand_map(CUtensorMap* map, const Operand& o, bool mn, bool whole, int across) {
    const uint64_t row = (uint64_t)o.ld * 2, plane = (uint64_t)o.plane * 2;
    const uint64_t rows = o.rows, cols = o.cols, planes = o.planes;
    const CUtensorMapDataType ty = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (mn && whole)
        return make_map_4d(map, o.p, ty, {64, rows, cols / 64, planes}, {row, 128, plane}, {64, (uint32_t)kBK, (uint32_t)across / 64, 1},
                           CU_TENSOR_MAP_SWIZZLE_128B);
    return make_map_4d(map, o.p, ty, {cols, rows, 1, planes}, {row, row, plane}, {64, (uint32_t)(mn ? kBK : across), 1, 1},
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// D = A B through the epilogue, or its splits' sums to `part`.  A_MN / B_MN: the operand's rows run
// along the contraction and its columns along D (stored [contraction][M] or [contraction][N]).
// follows: a kernel of the same call precedes (this one may start while that one ends).
template <bool A_MN, bool B_MN>
int run_gemm(const GemmPlan& p, const Operand& a, const Operand& b, const Epi& epi, float* part, bool follows,
             cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!operand_map(&ma, a, A_MN, p.g.whole_a, 128) || !operand_map(&mb, b, B_MN, p.g.whole_b, p.bn / p.ctas))
        return GT_ERR_CUDA;
    float* out = leaves_sums(p, epi.single, epi.y_f32 || epi.pre_f32) ? part : nullptr;
    if (p.bn == 256)
        return !p.sum ? launch_gemm<2, 256, false, A_MN, B_MN>(p, ma, mb, epi, out, follows, s)
                         : launch_gemm<2, 256, true, A_MN, B_MN>(p, ma, mb, epi, out, follows, s);
    if (p.bn == 128)
        return !p.sum ? launch_gemm<2, 128, false, A_MN, B_MN>(p, ma, mb, epi, out, follows, s)
                         : launch_gemm<2, 128, true, A_MN, B_MN>(p, ma, mb, epi, out, follows, s);
    return launch_gemm<1, 64, true, A_MN, B_MN>(p, ma, mb, epi, out, follows, s);
}

template <bool SUM>
int launch_both(const BwdPlan& p, const CUtensorMap (&mx)[2], const CUtensorMap (&mw)[2], const Epi& epi_x,
                const Epi& epi_w, float* part_x, float* part_w, bool follows, cudaStream_t s) {
    GemmJob x, w;
    int rc = make_job<2, kBothBN, SUM>(&x, p.x, mx[0], mx[1], epi_x, part_x);
    if (rc == GT_OK) rc = make_job<2, kBothBN, SUM>(&w, p.w, mw[0], mw[1], epi_w, part_w);
    if (rc != GT_OK) return rc;
    static std::atomic<uint64_t> allowed;
    return launch_products<2, kBothBN, SUM>(linear_gemm_both<SUM>, allowed, num_sms() / 2, follows, s, x, w, p.units_x);
}

// da W^T and x^T da in one launch.
int run_both(const BwdPlan& p, const Operand& da, const Operand& w, const Operand& x, const Epi& epi_x, const Epi& epi_w,
             float* part_x, float* part_w, bool follows, cudaStream_t s) {
    CUtensorMap mx[2], mw[2];
    const GemmShape &gx = p.x.g, &gw = p.w.g;
    if (!operand_map(&mx[0], da, false, gx.whole_a, 128) || !operand_map(&mx[1], w, false, gx.whole_b, kBothBN / 2) ||
        !operand_map(&mw[0], x, true, gw.whole_a, 128) || !operand_map(&mw[1], da, true, gw.whole_b, kBothBN / 2))
        return GT_ERR_CUDA;
    return p.x.sum ? launch_both<true>(p, mx, mw, epi_x, epi_w, part_x, part_w, follows, s)
                          : launch_both<false>(p, mx, mw, epi_x, epi_w, part_x, part_w, follows, s);
}

JoinJob join_job(const GemmPlan& p, const float* part, const Epi& epi) {
    if (!leaves_sums(p, epi.single, epi.y_f32 || epi.pre_f32)) return JoinJob{};
    const int M = p.g.M, N = p.g.N;
    return JoinJob{(int)((join_threads(M, N, epi.single) + kJoinThreads - 1) / kJoinThreads), M, N, p.g.splits, part, pad8(N), epi};
}

// linear_join of the sums that two products (or one: JoinJob{}) have left, and of the column sums, if any.
int run_joins(const JoinJob& j0, const JoinJob& j1, const ColSum& cs, cudaStream_t s) {
    const int ctas = j0.ctas + j1.ctas + (cs.out ? (cs.cols + 31) / 32 : 0);
    if (ctas == 0) return GT_OK;
    LaunchScope ls("linear_join", s);
    if (launch_overlapped(linear_join, dim3(ctas), dim3(kJoinThreads), 0, s, j0, j1, cs) != cudaSuccess) return GT_ERR_CUDA;
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
    const int64_t most = (4 * (int64_t)num_sms() + gx - 1) / gx;   // four resident CTAs per SM
    if (gy > most) gy = most;
    if (gy > kPrepSlabs) gy = kPrepSlabs;
    return {tx, gx, (int)gy};
}

int elem_bytes(int t) { return t == GT_F32 ? 4 : 2; }

// The preparation of a call: its jobs are collected, then launched at once.
struct Prep {
    int dtype;
    PrepJobs jobs{};
    int ctas = 0;

    // `src` [m][n] of type t, times act'(pre), as operand planes of the compute type in dst; see PrepJob.
    void add(int t, int m, int n, const void* src, int64_t lds, const void* pre, int64_t ldp, bf16* dst, float* colsum) {
        const PrepGrid pg = prep_grid(m, n);
        PrepJob& j = jobs.j[jobs.count++];
        j.src = src; j.pre = pre; j.dst = dst; j.colsum = colsum;
        j.lds = lds; j.ldp = ldp; j.ldd = pad8(n); j.plane = m * j.ldd;
        j.m = m; j.n = n; j.tx = pg.tx; j.gx = pg.gx; j.gy = pg.gy;
        j.f32 = t == GT_F32;
        j.svec = row_access(src, lds, elem_bytes(t));
        j.pvec = row_access(pre, ldp, elem_bytes(dtype));
        ctas += pg.gx * pg.gy;
    }
    // src [m][n] of the compute type as an operand: read in place (buf NULL), or through buf,
    // split in three for fp32 and copied for bf16.
    Operand operand(int m, int n, const void* src, int64_t ld, bf16* buf) {
        if (!buf) return Operand{static_cast<const bf16*>(src), ld, ld, 1, m, n};
        add(dtype, m, n, src, ld, nullptr, 0, buf, nullptr);
        return in_planes(m, n, buf);
    }
    Operand in_planes(int m, int n, const bf16* buf) const {
        return Operand{buf, pad8(n), m * pad8(n), dtype == GT_F32 ? 3 : 1, m, n};
    }
    int launch(cudaStream_t s) const {
        if (jobs.count == 0) return GT_OK;
        LaunchScope ls("linear_prep", s);
        if (dtype == GT_F32) linear_prep<3><<<ctas, kPrepThreads, 0, s>>>(jobs);
        else linear_prep<1><<<ctas, kPrepThreads, 0, s>>>(jobs);
        return check_launch();
    }
};

size_t operand_elems(int dtype, int m, int n) { return (size_t)m * pad8(n) * (dtype == GT_F32 ? 3 : 1); }

int planes_of(int dtype) { return dtype == GT_F32 ? 3 : 1; }

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
size_t fwd_bufs(int dtype, bool y_f32, int m, int k, int n, bool pack_x, bool pack_w, bool single, void* ws,
                size_t bytes, FwdBufs* out) {
    Carve c(ws, bytes);
    FwdBufs b;
    b.x = pack_x ? c.take<bf16>(operand_elems(dtype, m, k)) : nullptr;
    b.w = pack_w ? c.take<bf16>(operand_elems(dtype, k, n)) : nullptr;
    b.part = c.take<float>(part_floats(plan_gemm(m, n, k, planes_of(dtype), y_f32), single, y_f32));
    if (out) *out = b;
    return c.off;
}

// ... and of the backward, with da (where dy itself does not serve), the column sums' partial
// rows, and one buffer for the splits' sums of both products, in turn or at once.
struct BwdBufs {
    bf16 *x, *w, *da;
    float *part, *cols;
};
size_t bwd_bufs(const BwdPlan& p, int dtype, int m, int k, int n, bool pack_x, bool pack_w, bool own_da, bool single_x,
                bool single_w, void* ws, size_t bytes, BwdBufs* out) {
    Carve c(ws, bytes);
    BwdBufs b;
    b.x = pack_x ? c.take<bf16>(operand_elems(dtype, m, k)) : nullptr;
    b.w = pack_w ? c.take<bf16>(operand_elems(dtype, k, n)) : nullptr;
    b.da = own_da ? c.take<bf16>(operand_elems(dtype, m, n)) : nullptr;
    const bool f32 = dtype == GT_F32;
    const size_t px = part_floats(p.x, single_x, f32), pw = part_floats(p.w, single_w, f32);
    b.part = c.take<float>(p.units_x > 0 ? px + pw : std::max(px, pw));
    b.cols = c.take<float>((size_t)prep_grid(m, n).gy * n);
    if (out) *out = b;
    return c.off;
}

Epi make_epi(const float* bias, int act, int ytype, int ptype, const void* r, int64_t ldr, int ey, void* y, int64_t ldy,
             void* pre, int64_t ldpre, int ep) {
    Epi e{bias, r, y, pre, ldr, ldy, ldpre, act == GT_ACT_GELU, ytype == GT_F32, ptype == GT_F32, false, false,
          row_access(r, ldr, ey), row_access(y, ldy, ey), row_access(pre, ldpre, ep)};
    e.single = e.yacc == 0 || (r && e.racc == 0) || (pre && e.pacc == 0);
    return e;
}

int small_tiles(int rows, int cols) { return (rows + kSmT - 1) / kSmT * ((cols + kSmT - 1) / kSmT); }
// Whether a fp32 call goes to the fp32 pipes in one kernel: short contractions and few multiplications.  One launch
// without a workspace for two launches (three in the backward) saves a caller from Python 8 us (12), so the cut-offs let the
// device lose up to 8 % of its time on the way there.  Measured against the split products (us on the device in a captured
// graph, split and this; then as called one after another, split and this):
//   forward   512x64x64 7.2, 5.6; 20, 12     16384x64x64 9.8, 8.3; 21, 12     65536x64x16 24.2, 21.8; 27, 24
//             6800x64x192 10.7, 11.0; 21, 13     512x64x2048 7.7, 8.1; 21, 13     1700x16x2048 17.3, 13.0; 21, 15
//   past it   6800x128x128 9.8, 13.2; 21, 16     512x128x128 8.3, 9.0; 21, 13     1x512x512 9.5, 28.2; 26, 31
//   backward  512x64x64 10.5, 6.9; 31, 17     100x256x64 10.2, 6.1; 30, 17     512x256x128 11.9, 10.2; 30, 17
//             1024x64x128 11.0, 10.9; 31, 17     1000x64x64 10.6, 10.8; 30, 17     300x512x100 12.1, 11.9; 31, 17
//             1024x16x16 10.0, 10.8; 31, 17     64x16x128 8.8, 9.5; 29, 17
//   past it   2048x64x64 11.9, 18.7; 30, 21     512x64x192 11.6, 14.0; 30, 17     1024x256x128 12.5, 15.7; 30, 18
bool small_fwd(int dtype, int m, int k, int n) {
    return dtype == GT_F32 && k <= 64 && (int64_t)m * k * n <= (96 << 20);
}
bool small_bwd(int dtype, int m, int k, int n) {
    return dtype == GT_F32 && m <= 1024 && n <= 128 && (int64_t)m * k * n <= (16 << 20);
}

bool ranges_ok(const void* p, int64_t ld, int cols) { return !p || ld >= cols; }

}  // namespace
}  // namespace gt

extern "C" {

size_t gt_linear_fwd_workspace_size(int32_t dtype, int32_t m, int32_t k, int32_t n, int32_t aligned) {
    using namespace gt;
    if (check_linear(dtype, GT_F32, m, k, n, GT_ACT_NONE) != GT_OK) return 0;
    if (small_fwd(dtype, m, k, n)) return 0;
    const bool pack = dtype == GT_F32 || !aligned;
    const size_t a = fwd_bufs(dtype, false, m, k, n, pack, pack, !aligned, nullptr, 0, nullptr);
    const size_t b = fwd_bufs(dtype, true, m, k, n, pack, pack, !aligned, nullptr, 0, nullptr);
    return a > b ? a : b;   // for either type of y
}

size_t gt_linear_bwd_workspace_size(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, int32_t act,
                                    int32_t aligned) {
    using namespace gt;
    if (check_linear(dtype, ytype, m, k, n, act) != GT_OK || small_bwd(dtype, m, k, n)) return 0;
    const bool pack = dtype == GT_F32 || !aligned;
    return bwd_bufs(plan_bwd(m, k, n, planes_of(dtype), dtype == GT_F32), dtype, m, k, n, pack, pack,
                    pack || act != GT_ACT_NONE || ytype != dtype, !aligned, !aligned, nullptr, 0, nullptr);
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
    const int ey = elem_bytes(ytype), ex = elem_bytes(dtype);
    const Epi epi = make_epi(b, act, ytype, dtype, r, ldr, ey, y, ldy, pre, ldpre, ex);
    if (small_fwd(dtype, m, k, n)) {
        Small p{};
        p.x = static_cast<const float*>(x);
        p.w = static_cast<const float*>(w);
        p.ldx = ldx; p.ldw = ldw;
        p.m = m; p.k = k; p.n = n;
        p.out = epi;
        p.tiles = small_tiles(m, n);
        LaunchScope ls("linear_small", static_cast<cudaStream_t>(stream));
        linear_small<false><<<p.tiles, kSmThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        return check_launch();
    }
    FwdBufs bufs;
    const size_t need = fwd_bufs(dtype, ytype == GT_F32, m, k, n, pack_x, pack_w, epi.single, workspace, ws_bytes, &bufs);
    if (need > 0 && (!workspace || !aligned16(workspace) || ws_bytes < need)) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Prep prep{dtype};
    const Operand ox = prep.operand(m, k, x, ldx, bufs.x), ow = prep.operand(k, n, w, ldw, bufs.w);
    if ((rc = prep.launch(s)) != GT_OK) return rc;
    const GemmPlan plan = plan_gemm(m, n, k, planes_of(dtype), ytype == GT_F32);
    if ((rc = run_gemm<false, true>(plan, ox, ow, epi, bufs.part, prep.jobs.count > 0, s)) != GT_OK) return rc;
    return run_joins(join_job(plan, bufs.part, epi), JoinJob{}, ColSum{}, s);
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
    const int ex = elem_bytes(dtype);
    const Epi epi_x = make_epi(nullptr, GT_ACT_NONE, dtype, dtype, add, ldadd, ex, dx, lddx, nullptr, 0, ex);
    const Epi epi_w = make_epi(nullptr, GT_ACT_NONE, dtype, dtype, nullptr, 0, ex, dw, lddw, nullptr, 0, ex);
    if (small_bwd(dtype, m, k, n)) {
        Small p{};
        p.x = static_cast<const float*>(x);
        p.w = static_cast<const float*>(w);
        p.dy = static_cast<const float*>(dy);
        p.pre = static_cast<const float*>(pre);
        p.ldx = ldx; p.ldw = ldw; p.lddy = lddy; p.ldpre = ldpre;
        p.m = m; p.k = k; p.n = n;
        p.out = epi_x;
        p.dw = epi_w;
        p.db = db;
        p.tiles = dx ? (small_tiles(m, k) + kSmCluster - 1) / kSmCluster * kSmCluster : 0;
        const int more = kSmCluster * (dw ? small_tiles(k, n) : db ? small_tiles(1, n) : 0);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(p.tiles + more));
        cfg.blockDim = dim3(kSmThreads);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kSmCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        LaunchScope ls("linear_small", cfg.stream);
        return cudaLaunchKernelEx(&cfg, linear_small<true>, p) == cudaSuccess ? check_launch() : GT_ERR_CUDA;
    }
    BwdBufs bufs;
    const bool f32 = dtype == GT_F32;
    const BwdPlan plan = plan_bwd(m, k, n, planes_of(dtype), f32);
    const size_t need = bwd_bufs(plan, dtype, m, k, n, pack_x, pack_w, own_da, dx && epi_x.single, dw && epi_w.single, workspace,
                                 ws_bytes, &bufs);
    if (!workspace || !aligned16(workspace) || ws_bytes < need) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Prep prep{dtype};
    Operand oda{static_cast<const bf16*>(dy), lddy, lddy, 1, m, n}, ox{}, ow{};
    if (own_da || db) prep.add(ytype, m, n, dy, lddy, pre, ldpre, bufs.da, db ? bufs.cols : nullptr);
    if (own_da) oda = prep.in_planes(m, n, bufs.da);
    if (dx) ow = prep.operand(k, n, w, ldw, bufs.w);
    if (dw) ox = prep.operand(m, k, x, ldx, bufs.x);
    if ((rc = prep.launch(s)) != GT_OK) return rc;
    bool follows = prep.jobs.count > 0;
    const ColSum cs{db ? bufs.cols : nullptr, db, prep_grid(m, n).gy, n};
    if (dx && dw && plan.units_x > 0) {
        float* part_w = bufs.part + part_floats(plan.x, epi_x.single, f32);
        const JoinJob jx = join_job(plan.x, bufs.part, epi_x), jw = join_job(plan.w, part_w, epi_w);
        if ((rc = run_both(plan, oda, ow, ox, epi_x, epi_w, jx.ctas ? bufs.part : nullptr, jw.ctas ? part_w : nullptr, follows,
                           s)) != GT_OK)
            return rc;
        return run_joins(jx, jw, cs, s);
    }
    if (dx) {
        if ((rc = run_gemm<false, false>(plan.x, oda, ow, epi_x, bufs.part, follows, s)) != GT_OK) return rc;
        follows = true;
        // the column sums go with the last join, or with this one if it is the last
        if ((rc = run_joins(join_job(plan.x, bufs.part, epi_x), JoinJob{}, dw ? ColSum{} : cs, s)) != GT_OK) return rc;
    }
    if (dw) {
        if ((rc = run_gemm<true, true>(plan.w, ox, oda, epi_w, bufs.part, follows, s)) != GT_OK) return rc;
        return run_joins(join_job(plan.w, bufs.part, epi_w), JoinJob{}, cs, s);
    }
    return dx ? GT_OK : run_joins(JoinJob{}, JoinJob{}, cs, s);
}

}  // extern "C"
