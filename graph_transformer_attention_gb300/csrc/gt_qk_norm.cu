// gt_qk_norm.cu -- the norm of every head of the queries and keys, with the rotation
// of their channel pairs by position in the same pass, forward and backward.
//
//   forward   r = 1 / sqrt(sum_c x_c^2 / d + eps),  y = R (gain x r)
//   backward  g = R^T dy,  w = gain g,
//             dx = r (w - x r^2 sum_c w_c x_c / d),  dgain = sum over rows and heads of g x r
//
// R turns the pair (a, b) of channels by the angle pos * freq: (a cos - b sin, a sin + b cos).
//
// The bytes of x, y (dy, dx) bound it.  A head's channels are dealt to a few lanes of a warp, both channels of a pair to
// the same lane, so that the norm is a few shuffles and the turn none; every row is read once and nothing but gradients
// is kept for the backward, which forms r again from the x it reads anyway.  The angles are the same for all heads of a
// row: a warp computes the cosines and sines of its rows once, into shared memory, and fetches the heads of its next rows
// meanwhile.  (CTAs of eight warps with a barrier between angles and rows: forward 56 us, backward 109, now 43 and 74 to
// 75, for 32768 rows of 16 and 8 heads of 64, bf16: 4.7 and 4.0 TB/s.)  Next limits: issue slots (54 and 52 %) at 16
// warps to an SM.
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

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 256;
constexpr int kMaxHeads = 1024;
constexpr int kAngles = 1024;            // cosines and sines of a CTA's rows: 8 KB
constexpr int kWarpAngles = kAngles / kWarps;

// The turns by which one position more turns a pair, as a binary fraction of 64 digits (whole turns dropped):
// freq / (2 pi) mod 1, freq = mant 2^e, with 96 binary digits of 1 / (2 pi) (the reduction of Payne and Hanek, 1983).
// pos times this, in integers mod 2^64, is the fraction of the angle in turns, off by less than 2^-33 turns for any int32
// position while |freq| < 2^24 (a larger one loses digits: the digits of 1 / (2 pi) end 2^(e - 72) turns away).
__device__ __forceinline__ uint64_t rate_of(float freq) {
    const uint32_t bits = __float_as_uint(freq), ex = (bits >> 23) & 255u;
    const uint64_t mant = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int e = (int)(ex ? ex : 1u) - 150;
    const uint64_t c_hi = 0x28BE60DB9391054Aull, c_lo = 0x7F09D5F4ull;   // 1 / (2 pi): the first 64 digits, the next 32
    // mant / (2 pi) = (hi : lo), 64 whole and 64 fraction digits
    const uint64_t tail = (mant * c_lo) >> 32, lo0 = mant * c_hi, lo = lo0 + tail;
    const uint64_t hi = __umul64hi(mant, c_hi) + (lo < lo0 ? 1u : 0u);
    uint64_t f;
    if (e >= 0) f = e < 64 ? lo << e : 0u;
    else if (e > -64) f = (lo >> -e) | (hi << (64 + e));
    else f = e > -128 ? hi >> (-e - 64) : 0u;
    return bits >> 31 ? 0u - f : f;
}

// cos and sin of pos times the rate; per_unit: the angle of 2^-32 turns (NaN spoils both).  The nearest quarter turn is
// taken off in integers, Taylor's polynomials do the rest: 2e-9 and 3e-8 off at pi / 4, the roundings come on top.
__device__ __forceinline__ float2 turn_of(int pos, uint64_t rate, float per_unit) {
    const uint32_t f = (uint32_t)(((uint64_t)(int64_t)pos * rate) >> 32), quarter = (f + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(f - (quarter << 30)) * per_unit, z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;      // turned by quarter: (c, s), (-s, c), (-c, -s), (s, -c)
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// One side of a call: queries or keys.  dy: the backward's; y is then dx.
struct Side {
    const void* x;
    const void* dy;
    void* y;
    const float* gain;
    const int32_t* pos;      // NULL: the row's own index
    float* part;             // [CTAs][d] sums of the gain's gradient
    float* dgain;
    int64_t ldx, hdx, lddy, hddy, ldy, hdy;
    int n, h;
    int rows;                // rows a warp (qk_norm_any: a CTA) takes at a time
    int ctas;
};

struct Job {
    Side side[2];
    const float* freq;
    int d, rot;              // channels of a head, channels that turn
    int lanes;               // lanes to a head (a power of two)
    bool adjacent;           // pairs (2i, 2i + 1), else (i, i + rot / 2)
    float eps, inv_d;
};

// V consecutive elements, as stored and as fp32 pairs
template <int V, typename T> struct Raw;
template <> struct Raw<8, __nv_bfloat16> { uint4 w; };
template <> struct Raw<8, float> { Raw8<float> r; };
template <> struct Raw<4, __nv_bfloat16> { uint2 w; };
template <> struct Raw<4, float> { float4 w; };

template <int V, typename T>
__device__ __forceinline__ Raw<V, T> get(const T* p) {
    Raw<V, T> r;
    if constexpr (V == 8 && sizeof(T) == 4) r.r = load8(p, 8, 1);
    else r.w = __ldg(reinterpret_cast<const decltype(r.w)*>(p));
    return r;
}

__device__ __forceinline__ float2 pair_of(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Raw<8, __nv_bfloat16>& r, float2 (&v)[4]) {
    v[0] = pair_of(r.w.x); v[1] = pair_of(r.w.y); v[2] = pair_of(r.w.z); v[3] = pair_of(r.w.w);
}
__device__ __forceinline__ void unpack(const Raw<8, float>& r, float2 (&v)[4]) { unpack8(r.r, v); }
__device__ __forceinline__ void unpack(const Raw<4, __nv_bfloat16>& r, float2 (&v)[2]) {
    v[0] = pair_of(r.w.x); v[1] = pair_of(r.w.y);
}
__device__ __forceinline__ void unpack(const Raw<4, float>& r, float2 (&v)[2]) {
    v[0] = make_float2(r.w.x, r.w.y); v[1] = make_float2(r.w.z, r.w.w);
}

template <int P, typename T>
__device__ __forceinline__ void put(T* p, const float2 (&v)[P]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < P; i += 2)
            reinterpret_cast<float4*>(p)[i / 2] = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
    } else if constexpr (P == 4) {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(v[0].x, v[0].y), bf16x2_bits(v[1].x, v[1].y),
                                                  bf16x2_bits(v[2].x, v[2].y), bf16x2_bits(v[3].x, v[3].y));
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(v[0].x, v[0].y), bf16x2_bits(v[1].x, v[1].y));
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float t = a * c - b * s;
    b = a * s + b * c;
    a = t;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A mean square (with eps) above 2^126 or below 2^-90 is formed again from the row times a power of two: squares beyond
// fp32's range are infinite, or lose digits.  sum_of(by): that of the row times `by`.  (A norm above 2^126 still has a
// subnormal reciprocal, 2^-22 of it off at most.)
__device__ __forceinline__ bool is_wide(float mean) {
    constexpr uint32_t low = (127 - 90) << 23, high = (127 + 126) << 23;      // 2^-90 and 2^126 as stored
    return __float_as_uint(mean) - low > high - low;
}
template <typename F>
__device__ __forceinline__ float wide_rsqrt(float mean, float rs, float inv_d, float eps, F&& sum_of) {
    const float large = rsqrtf(sum_of(0x1p-80f) * inv_d + eps * 0x1p-80f * 0x1p-80f) * 0x1p-80f;
    const float small = rsqrtf(sum_of(0x1p80f) * inv_d + eps * 0x1p80f * 0x1p80f) * 0x1p80f;
    return !is_wide(mean) ? rs : mean < 1.f ? small : large;
}

// What a CTA has in shared memory.
struct Shared {
    alignas(16) float cos[kAngles];
    alignas(16) float sin[kAngles];
    alignas(16) float minus[kAngles];  // -sin: a packed pair would be negated word by word
    uint64_t rate[kMaxD / 2];
    float per_unit[kMaxD / 2];
    float red[kWarps][kMaxD];   // (backward)
};

__device__ __forceinline__ void make_rates(const Job& J, Shared& sh) {
    for (int p = threadIdx.x; p < J.rot >> 1; p += kThreads) {
        const float f = __ldg(J.freq + p);
        sh.rate[p] = rate_of(f);
        sh.per_unit[p] = isfinite(f) ? 6.28318531f * 0x1p-32f : NAN;
    }
}

// The angles of rows row0 .. row0 + rows - 1, between two barriers.
__device__ __forceinline__ void make_angles(const Job& J, const Side& S, int64_t row0, int rows, Shared& sh) {
    const int half = J.rot >> 1;
    __syncthreads();      // the rates are there, the last rows' angles have been read
    for (int k = threadIdx.x; k < rows * half; k += kThreads) {
        const int r = k / half, p = k - r * half;
        const float2 t = turn_of(S.pos ? __ldg(S.pos + row0 + r) : (int)(row0 + r), sh.rate[p], sh.per_unit[p]);
        sh.cos[k] = t.x;
        sh.sin[k] = t.y;
    }
    __syncthreads();
}

// A CTA's sum of its groups' gradients of channel c, which stand in red[warp][c].
__device__ __forceinline__ void put_gain_sums(const Job& J, const Side& S, int cta, Shared& sh) {
    __syncthreads();
    for (int c = threadIdx.x; c < J.d; c += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += sh.red[w][c];
        S.part[(int64_t)cta * J.d + c] = t;
    }
}

// Heads that a group of lanes has at once; those of the next turn are on their way meanwhile.
constexpr int items_of(bool bwd) { return bwd ? 1 : 2; }

// All channels turn, or none, and move in pieces of V: a lane has channels V s .. V s + V - 1 and d / 2 + V s .., s its
// place in the group.  Every warp is on its own: its turns are `rows` rows each, whose angles it forms (a lane an angle,
// for all their heads) while the next turn's heads are on their way; no barrier of the CTA holds it up.  Arithmetic in
// packed pairs: the issue slots are the next bound behind the bytes.
template <typename TX, typename TY, int V, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm(const __grid_constant__ Job J) {
    constexpr int ITEMS = items_of(BWD), P = V / 2;
    using TO = typename std::conditional<BWD, TX, TY>::type;
    __shared__ Shared sh;
    const int which = blockIdx.x < J.side[0].ctas ? 0 : 1;
    const Side& S = J.side[which];
    const int cta = blockIdx.x - (which ? J.side[0].ctas : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int place = lane & (J.lanes - 1), group = lane / J.lanes, groups = 32 / J.lanes;
    const int half = J.rot >> 1, mid = J.d >> 1;
    const bool mine = V * place < mid;                    // (lanes past the head's channels read the first ones)
    const int c0 = mine ? V * place : 0;
    float* cos_w = sh.cos + warp * kWarpAngles;
    float* sin_w = sh.sin + warp * kWarpAngles;
    float* minus_w = sh.minus + warp * kWarpAngles;
    // (copies: what is read through a reference into the arguments is read again at every use)
    const int n = S.n, h = S.h, rows = S.rows, lanes = J.lanes, ldx = (int)S.ldx, lddy = (int)S.lddy, ldy = (int)S.ldy;
    const int hdx = (int)S.hdx, hddy = (int)S.hddy, hdy = (int)S.hdy;
    const int32_t* const pos = S.pos;
    const float inv_d = J.inv_d, eps = J.eps;
    const bool adjacent = J.adjacent;
    const int turns = (int)(((int64_t)n + rows - 1) / rows), step = S.ctas * kWarps;
    // deal() takes several rows only where their heads make one batch; with one row the batches are its heads
    const int batch = ITEMS * groups, last = rows > 1 ? 0 : (h - 1) / batch;

    // this lane's row in the turn and head in the batch, and where they stand
    int row_k[ITEMS], head_k[ITEMS];
    int64_t x_k[ITEMS], dy_k[ITEMS], y_k[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int it = k * groups + group;
        row_k[k] = rows > 1 ? it / h : 0;
        head_k[k] = it - row_k[k] * h;
        if (row_k[k] >= rows) {      // no such row in a turn: no head is that far, and no call has so many
            row_k[k] = 0;
            head_k[k] = INT32_MAX;
        }
        x_k[k] = (int64_t)row_k[k] * ldx + (int64_t)head_k[k] * hdx;
        dy_k[k] = (int64_t)row_k[k] * lddy + (int64_t)head_k[k] * hddy;
        y_k[k] = (int64_t)row_k[k] * ldy + (int64_t)head_k[k] * hdy;
    }
    int turn = cta * kWarps + warp;
    const TX* x_t = static_cast<const TX*>(S.x) + (int64_t)turn * rows * ldx + c0;
    const TY* dy_t = static_cast<const TY*>(S.dy) + (int64_t)turn * rows * lddy + c0;
    TO* y_t = static_cast<TO*>(S.y) + (int64_t)turn * rows * ldy + c0;
    const int64_t step_x = (int64_t)step * rows * ldx, step_dy = (int64_t)step * rows * lddy, step_y = (int64_t)step * rows * ldy;

    struct Piece {
        Raw<V, TX> xa, xb;
        Raw<V, TY> da, db;
    };
    Piece next[ITEMS];
    auto is_live = [&](int t, int b, int k) { return row_k[k] < n - t * rows && head_k[k] < h - b * batch; };
    auto fetch = [&](int t, int b) {      // (heads that are not there: the turn's first)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const bool live = is_live(t, b, k);
            const TX* x = x_t + (live ? x_k[k] + (int64_t)(b * batch) * hdx : 0);
            next[k].xa = get<V>(x);
            next[k].xb = get<V>(x + mid);
            if constexpr (BWD) {
                const TY* dy = dy_t + (live ? dy_k[k] + (int64_t)(b * batch) * hddy : 0);
                next[k].da = get<V>(dy);
                next[k].db = get<V>(dy + mid);
            }
        }
    };
    if (turn < turns) fetch(turn, 0);
    if (half > 0) make_rates(J, sh);
    float2 ga[P], gb[P], sa[P], sb[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        ga[j] = mine ? make_float2(__ldg(S.gain + c0 + 2 * j), __ldg(S.gain + c0 + 2 * j + 1)) : both(0.f);
        gb[j] = mine ? make_float2(__ldg(S.gain + mid + c0 + 2 * j), __ldg(S.gain + mid + c0 + 2 * j + 1)) : both(0.f);
        sa[j] = sb[j] = both(0.f);
    }
    // this lane's angles: k = lane, lane + 32, ... of the turn's rows x half
    const int r_first = half > 0 ? lane / half : 0, p_first = half > 0 ? lane - r_first * half : 0;
    const int r_step = half > 0 ? 32 / half : 0, p_step = half > 0 ? 32 - r_step * half : 0;
    __syncthreads();      // the rates are there
    int next_b = 0;
    while (turn < turns) {
        float2 x[ITEMS][P], z[ITEMS][P], dx[ITEMS][P], dz[ITEMS][P];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            unpack(next[k].xa, x[k]);
            unpack(next[k].xb, z[k]);
            if constexpr (BWD) {
                unpack(next[k].da, dx[k]);
                unpack(next[k].db, dz[k]);
            }
        }
        const int t = turn, b = next_b;
        TO* const y_now = y_t;
        if (next_b++ == last) {
            next_b = 0;
            turn += step;
            x_t += step_x;
            if constexpr (BWD) dy_t += step_dy;
            y_t += step_y;
        }
        if (turn < turns) fetch(turn, next_b);
        if (half > 0 && b == 0) {
            __syncwarp();      // the last turn's angles have been read
            const int row0 = t * rows, count = min(rows, n - row0) * half;
            for (int k = lane, r = r_first, p = p_first; k < count; k += 32) {
                const float2 cs = turn_of(pos ? __ldg(pos + row0 + r) : row0 + r, sh.rate[p], sh.per_unit[p]);
                cos_w[k] = cs.x;
                sin_w[k] = cs.y;
                minus_w[k] = -cs.y;
                r += r_step;
                p += p_step;
                if (p >= half) {
                    p -= half;
                    ++r;
                }
            }
            __syncwarp();
        }
        // (every lane makes every turn: the shuffles need them all)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const bool live = is_live(t, b, k);
            float2 u[P], w[P];
            float2 ss = __fmul2_rn(x[k][0], x[k][0]);
#pragma unroll
            for (int j = 1; j < P; ++j) ss = __ffma2_rn(x[k][j], x[k][j], ss);
#pragma unroll
            for (int j = 0; j < P; ++j) ss = __ffma2_rn(z[k][j], z[k][j], ss);
            const float mean = lanes_sum(mine ? ss.x + ss.y : 0.f, lanes) * inv_d + eps;
            float rs = rsqrtf(mean);
            auto squares = [&](float by) {
                float2 t = both(0.f);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 a = __fmul2_rn(x[k][j], both(by)), c = __fmul2_rn(z[k][j], both(by));
                    t = __ffma2_rn(a, a, __ffma2_rn(c, c, t));
                }
                return lanes_sum(mine ? t.x + t.y : 0.f, lanes);
            };
            if constexpr (!BWD) {
                if (__any_sync(0xffffffffu, is_wide(mean))) rs = wide_rsqrt(mean, rs, inv_d, eps, squares);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if constexpr (BWD) {
                    u[j] = dx[k][j];
                    w[j] = dz[k][j];
                } else {
                    u[j] = __fmul2_rn(__fmul2_rn(x[k][j], both(rs)), ga[j]);
                    w[j] = __fmul2_rn(__fmul2_rn(z[k][j], both(rs)), gb[j]);
                }
            }
            if (half > 0) {      // (u, w) = R (u, w), backward R^T
                const int at = live && rows > 1 ? row_k[k] * half : 0;
                if (!adjacent) {
#pragma unroll
                    for (int j = 0; j < P; j += 2) {
                        const float4 c4 = *reinterpret_cast<const float4*>(cos_w + at + c0 + 2 * j);
                        const float4 s4 = *reinterpret_cast<const float4*>(sin_w + at + c0 + 2 * j);
                        const float4 m4 = *reinterpret_cast<const float4*>(minus_w + at + c0 + 2 * j);
                        const float2 c[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
                        const float2 s[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
                        const float2 m[2] = {make_float2(m4.x, m4.y), make_float2(m4.z, m4.w)};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 v = __ffma2_rn(w[j + i], BWD ? s[i] : m[i], __fmul2_rn(u[j + i], c[i]));
                            w[j + i] = __ffma2_rn(u[j + i], BWD ? m[i] : s[i], __fmul2_rn(w[j + i], c[i]));
                            u[j + i] = v;
                        }
                    }
                } else {
                    const float* cs = cos_w + at;
                    const float* sn = (BWD ? minus_w : sin_w) + at;
                    const int pa = c0 >> 1, pb = (mid + c0) >> 1;
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        turn_pair(u[j].x, u[j].y, cs[pa + j], sn[pa + j]);
                        turn_pair(w[j].x, w[j].y, cs[pb + j], sn[pb + j]);
                    }
                }
            }
            if constexpr (BWD) {
                // (not before the turn, where it would wait for the sum's shuffles: 67.7 us instead of 64.6)
                if (__any_sync(0xffffffffu, is_wide(mean))) rs = wide_rsqrt(mean, rs, inv_d, eps, squares);
                const float2 rs2 = both(rs);
                float2 wx = both(0.f);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    x[k][j] = __fmul2_rn(x[k][j], rs2);
                    z[k][j] = __fmul2_rn(z[k][j], rs2);
                    const float2 pa = __fmul2_rn(u[j], x[k][j]), pb = __fmul2_rn(w[j], z[k][j]);
                    if (live) {
                        sa[j] = __fadd2_rn(sa[j], pa);
                        sb[j] = __fadd2_rn(sb[j], pb);
                    }
                    wx = __ffma2_rn(pa, ga[j], wx);
                    wx = __ffma2_rn(pb, gb[j], wx);
                }
                // dx = r (w - (x r) sum(w x r) / d)
                const float2 back = both(-lanes_sum(mine ? wx.x + wx.y : 0.f, lanes) * inv_d);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    u[j] = __fmul2_rn(rs2, __ffma2_rn(x[k][j], back, __fmul2_rn(u[j], ga[j])));
                    w[j] = __fmul2_rn(rs2, __ffma2_rn(z[k][j], back, __fmul2_rn(w[j], gb[j])));
                }
            }
            if (live && mine) {
                TO* y = y_now + y_k[k] + (int64_t)(b * batch) * hdy;
                put<P>(y, u);
                put<P>(y + mid, w);
            }
        }
    }
    if constexpr (BWD) {
        sm100::pdl_trigger();
        // the groups' sums: those of a warp here, then the warps' in their order
#pragma unroll
        for (int j = 0; j < P; ++j) {
            for (int o = 16; o >= lanes; o >>= 1) {
                sa[j].x += __shfl_xor_sync(0xffffffffu, sa[j].x, o);
                sa[j].y += __shfl_xor_sync(0xffffffffu, sa[j].y, o);
                sb[j].x += __shfl_xor_sync(0xffffffffu, sb[j].x, o);
                sb[j].y += __shfl_xor_sync(0xffffffffu, sb[j].y, o);
            }
            if (lane < lanes && mine) {
                float* red = sh.red[warp] + c0 + 2 * j;
                red[0] = sa[j].x; red[1] = sa[j].y;
                red[mid] = sb[j].x; red[mid + 1] = sb[j].y;
            }
        }
        put_gain_sums(J, S, cta, sh);
    }
}

// Any width, alignment and number of turning channels: a lane has NS pairs of channels.  Place s is pair s while
// s < rot / 2; past the turning channels two neighbours, the second of which may be missing.
template <typename TX, typename TY, int NS, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm_any(const __grid_constant__ Job J) {
    __shared__ Shared sh;
    const int which = blockIdx.x < J.side[0].ctas ? 0 : 1;
    const Side& S = J.side[which];
    const int cta = blockIdx.x - (which ? J.side[0].ctas : 0);
    const int place = threadIdx.x & (J.lanes - 1), group = threadIdx.x / J.lanes, groups = kThreads / J.lanes;
    const int half = J.rot >> 1, h = S.h;
    if (half > 0) make_rates(J, sh);
    int ca[NS], cb[NS];      // channels, -1: none
    float ga[NS], gb[NS], sa[NS], sb[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int s = place + i * J.lanes;
        if (s < half) {
            ca[i] = J.adjacent ? 2 * s : s;
            cb[i] = J.adjacent ? 2 * s + 1 : s + half;
        } else {
            const int c = J.rot + 2 * (s - half);
            ca[i] = c < J.d ? c : -1;
            cb[i] = c + 1 < J.d ? c + 1 : -1;
        }
        ga[i] = ca[i] >= 0 ? __ldg(S.gain + ca[i]) : 0.f;
        gb[i] = cb[i] >= 0 ? __ldg(S.gain + cb[i]) : 0.f;
        sa[i] = sb[i] = 0.f;
    }
    for (int64_t row0 = (int64_t)cta * S.rows; row0 < S.n; row0 += (int64_t)S.ctas * S.rows) {
        const int rows = (int)(S.n - row0 < S.rows ? S.n - row0 : S.rows), items = rows * h;
        if (half > 0) make_angles(J, S, row0, rows, sh);
        // (every lane of a warp makes every turn: the shuffles need them all)
        for (int it0 = 0; it0 < items; it0 += groups) {
            const bool live = it0 + group < items;
            const int it = live ? it0 + group : 0, r = it / h, head = it - r * h;
            const int64_t row = row0 + r;
            const TX* x = static_cast<const TX*>(S.x) + row * S.ldx + head * S.hdx;
            const TY* dy = static_cast<const TY*>(S.dy) + row * S.lddy + head * S.hddy;
            float a[NS], b[NS], u[NS], w[NS], ss = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                a[i] = ca[i] >= 0 ? to_f32(x[ca[i]]) : 0.f;
                b[i] = cb[i] >= 0 ? to_f32(x[cb[i]]) : 0.f;
                if constexpr (BWD) {
                    u[i] = ca[i] >= 0 ? to_f32(dy[ca[i]]) : 0.f;
                    w[i] = cb[i] >= 0 ? to_f32(dy[cb[i]]) : 0.f;
                }
                ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
            }
            const float mean = lanes_sum(ss, J.lanes) * J.inv_d + J.eps;
            float rs = rsqrtf(mean), wx = 0.f;
            if (__any_sync(0xffffffffu, is_wide(mean)))
                rs = wide_rsqrt(mean, rs, J.inv_d, J.eps, [&](float by) {
                    float t = 0.f;
#pragma unroll
                    for (int i = 0; i < NS; ++i) t = fmaf(a[i] * by, a[i] * by, fmaf(b[i] * by, b[i] * by, t));
                    return lanes_sum(t, J.lanes);
                });
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int s = place + i * J.lanes;
                if constexpr (!BWD) {
                    u[i] = a[i] * rs * ga[i];
                    w[i] = b[i] * rs * gb[i];
                }
                if (s < half) turn_pair(u[i], w[i], sh.cos[r * half + s], BWD ? -sh.sin[r * half + s] : sh.sin[r * half + s]);
                if constexpr (BWD) {
                    a[i] *= rs;
                    b[i] *= rs;
                    const float pa = u[i] * a[i], pb = w[i] * b[i];
                    if (live) {
                        sa[i] += pa;
                        sb[i] += pb;
                    }
                    wx = fmaf(pa, ga[i], fmaf(pb, gb[i], wx));
                }
            }
            using TO = typename std::conditional<BWD, TX, TY>::type;
            TO* y = static_cast<TO*>(S.y) + row * S.ldy + head * S.hdy;
            const float back = BWD ? -lanes_sum(wx, J.lanes) * J.inv_d : 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                if constexpr (BWD) {
                    u[i] = rs * fmaf(a[i], back, u[i] * ga[i]);
                    w[i] = rs * fmaf(b[i], back, w[i] * gb[i]);
                }
                if (live && ca[i] >= 0) y[ca[i]] = from_f32<TO>(u[i]);
                if (live && cb[i] >= 0) y[cb[i]] = from_f32<TO>(w[i]);
            }
        }
    }
    if constexpr (BWD) {
        sm100::pdl_trigger();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            for (int o = 16; o >= J.lanes; o >>= 1) {
                sa[i] += __shfl_xor_sync(0xffffffffu, sa[i], o);
                sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
            }
            if ((threadIdx.x & 31) < J.lanes) {
                if (ca[i] >= 0) sh.red[threadIdx.x >> 5][ca[i]] = sa[i];
                if (cb[i] >= 0) sh.red[threadIdx.x >> 5][cb[i]] = sb[i];
            }
        }
        put_gain_sums(J, S, cta, sh);
    }
}

// dgain: a CTA per 32 channels and side; warp w adds the partial rows w, w + 32, ..., then warp 0 the 32 warp sums.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) qk_gain_sum(const __grid_constant__ Job J) {
    __shared__ float red[kSumThreads / 32][33];
    const Side& S = J.side[blockIdx.y];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    sm100::pdl_wait();   // launched to overlap the end of the kernel that writes the partial rows
    float acc = 0.f;
    constexpr int kStride = kSumThreads / 32, U = 16;      // loads on their way, those past the last row left out
    for (int p = ty; p < S.ctas && c < J.d; p += U * kStride) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = p + u * kStride < S.ctas ? __ldcg(S.part + (int64_t)(p + u * kStride) * J.d + c) : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) acc += x[u];
    }
    red[ty][tx] = acc;
    __syncthreads();
    if (ty == 0 && c < J.d) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kSumThreads / 32; ++r) sum += red[r][tx];
        S.dgain[c] = sum;
    }
}

bool valid_type(int t) { return t == GT_F32 || t == GT_BF16; }

bool pieces16(const void* p, int64_t ld, int64_t hd, int bytes, int piece) {
    return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)(ld * bytes) | (uint64_t)(hd * bytes)) & (uint64_t)(piece - 1)) == 0;
}

// The largest V with which all of a call's pieces are aligned accesses of up to 16 bytes of x (32-bit strides); 1: single
// elements.
template <typename TX, typename TY>
int piece_of(const Job& J, bool bwd) {
    if (J.rot != 0 && J.rot != J.d) return 1;
    for (int v = sizeof(TX) == 2 ? 8 : 4; v >= 4; v /= 2) {
        bool ok = J.d % (2 * v) == 0;
        for (const Side& S : J.side) {
            if (!S.x) continue;
            const int px = std::min<int>(16, v * (int)sizeof(TX)), py = std::min<int>(16, v * (int)sizeof(TY));
            ok = ok && pieces16(S.x, S.ldx, S.hdx, sizeof(TX), px);
            ok = ok && pieces16(S.y, S.ldy, S.hdy, bwd ? sizeof(TX) : sizeof(TY), bwd ? px : py);
            if (bwd) ok = ok && pieces16(S.dy, S.lddy, S.hddy, sizeof(TY), py);
            for (int64_t stride : {S.ldx, S.hdx, S.ldy, S.hdy, S.lddy, S.hddy}) ok = ok && stride <= INT32_MAX;
        }
        if (ok) return v;
    }
    return 1;
}

// CTAs at most: what is resident at once (each of the backward's makes one partial row)
int most_ctas() { return 4 * num_sms(); }

// How the rows are dealt.  A warp takes as many rows at a time as make `items` heads for every group of its lanes (a CTA of
// qk_norm_any: one), as far as the angles' table goes; the CTAs go to the two sides by their heads.
void deal(Job& J, int v, int items) {
    const int slots = v > 1 ? J.d / 2 / v : (J.rot / 2 + (J.d - J.rot + 1) / 2);
    J.lanes = 1;
    while (J.lanes < slots && J.lanes < 32) J.lanes *= 2;
    int64_t want[2] = {0, 0}, all = 0;
    for (int i = 0; i < 2; ++i) {
        Side& S = J.side[i];
        S.rows = 1;
        if (!S.x) continue;
        const int heads = (v > 1 ? items * 32 : kThreads) / J.lanes;
        S.rows = std::max(1, heads / S.h);
        if (J.rot) S.rows = std::min(S.rows, std::max(1, (v > 1 ? kWarpAngles : kAngles) / (J.rot / 2)));
        // enough warps for every SM first
        S.rows = (int)std::max<int64_t>(1, std::min<int64_t>(S.rows, S.n / (4 * num_sms())));
        const int64_t turns = ((int64_t)S.n + S.rows - 1) / S.rows;
        want[i] = v > 1 ? (turns + kWarps - 1) / kWarps : turns;
        all += want[i];
    }
    for (int i = 0; i < 2; ++i) {
        Side& S = J.side[i];
        S.ctas = (int)want[i];
        if (S.x && all > most_ctas()) {
            const int64_t a = (int64_t)J.side[0].n * J.side[0].h, b = J.side[1].x ? (int64_t)J.side[1].n * J.side[1].h : 0;
            const int64_t share = (int64_t)(((double)(i ? b : a) / (double)(a + b)) * (most_ctas() - 2));
            S.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(share, want[i]));
        }
    }
}

template <typename TX, typename TY, bool BWD>
int run(Job& J, cudaStream_t s) {
    const int v = piece_of<TX, TY>(J, BWD);
    deal(J, v, items_of(BWD));
    const int grid = J.side[0].ctas + J.side[1].ctas;
    // the keys' partial rows follow the queries'; deal() keeps both together within most_ctas()
    if (BWD) J.side[1].part = J.side[0].part + (int64_t)J.side[0].ctas * J.d;
    {
        LaunchScope ls(BWD ? "qk_norm_bwd" : "qk_norm_fwd", s);
        if (v == 8) {
            if constexpr (sizeof(TX) == 2) qk_norm<TX, TY, 8, BWD><<<grid, kThreads, 0, s>>>(J);
        } else if (v == 4) {
            qk_norm<TX, TY, 4, BWD><<<grid, kThreads, 0, s>>>(J);
        } else if (J.d <= 63) {   // at most 32 pairs
            qk_norm_any<TX, TY, 1, BWD><<<grid, kThreads, 0, s>>>(J);
        } else {
            qk_norm_any<TX, TY, 4, BWD><<<grid, kThreads, 0, s>>>(J);
        }
        const int rc = check_launch();
        if (rc != GT_OK) return rc;
    }
    if (BWD) {
        LaunchScope ls("qk_gain_sum", s);
        if (launch_overlapped(qk_gain_sum, dim3((J.d + 31) / 32, J.side[1].x ? 2 : 1), dim3(kSumThreads), 0, s, J) !=
            cudaSuccess)
            return GT_ERR_CUDA;
        return check_launch();
    }
    return GT_OK;
}

template <bool BWD>
int dispatch(int xtype, int ytype, Job& J, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (xtype == GT_F32) return ytype == GT_F32 ? run<float, float, BWD>(J, s) : run<float, B, BWD>(J, s);
    return ytype == GT_F32 ? run<B, float, BWD>(J, s) : run<B, B, BWD>(J, s);
}

// The checks that both directions share; fills what they share of the job.
int check(int xtype, int ytype, int d, float eps, const float* freq, int rot, int pairs, Job& J) {
    if (!valid_type(xtype) || !valid_type(ytype) || d < 1 || rot < 0 || rot > d || rot % 2) return GT_ERR_INVALID_ARG;
    if (pairs != GT_ROT_HALVES && pairs != GT_ROT_PAIRS) return GT_ERR_INVALID_ARG;
    if ((rot > 0) != (freq != nullptr) || !(eps > 0.f) || !isfinite(eps)) return GT_ERR_INVALID_ARG;
    for (const Side& S : J.side) {
        if (!S.x) continue;
        if (S.n < 1 || S.h < 1 || !S.gain || !S.y) return GT_ERR_INVALID_ARG;
        if (S.ldx < 0 || S.hdx < 0 || S.ldy < 0 || S.hdy < 0 || S.lddy < 0 || S.hddy < 0) return GT_ERR_INVALID_ARG;
    }
    if (!J.side[0].x) return GT_ERR_INVALID_ARG;
    if (d > kMaxD || J.side[0].h > kMaxHeads || (J.side[1].x && J.side[1].h > kMaxHeads)) return GT_ERR_UNSUPPORTED;
    J.freq = freq;
    J.d = d;
    J.rot = rot;
    J.adjacent = pairs == GT_ROT_PAIRS;
    J.eps = eps;
    J.inv_d = 1.f / (float)d;
    return GT_OK;
}

}  // namespace
}  // namespace gt

extern "C" {

int gt_qk_norm_fwd(int32_t xtype, int32_t ytype, int32_t d, float eps, const float* freq, int32_t rot, int32_t pairs,
                   int32_t nq, int32_t h, const void* q, int64_t ldq, int64_t hdq, const float* gain_q, const int32_t* pos_q,
                   void* yq, int64_t ldyq, int64_t hdyq, int32_t nk, int32_t hk, const void* k, int64_t ldk, int64_t hdk,
                   const float* gain_k, const int32_t* pos_k, void* yk, int64_t ldyk, int64_t hdyk, void* stream) {
    using namespace gt;
    Job J = {};
    J.side[0] = Side{q, nullptr, yq, gain_q, pos_q, nullptr, nullptr, ldq, hdq, 0, 0, ldyq, hdyq, nq, h, 1, 0};
    J.side[1] = Side{k, nullptr, yk, gain_k, pos_k, nullptr, nullptr, ldk, hdk, 0, 0, ldyk, hdyk, nk, hk, 1, 0};
    const int rc = check(xtype, ytype, d, eps, freq, rot, pairs, J);
    return rc != GT_OK ? rc : dispatch<false>(xtype, ytype, J, static_cast<cudaStream_t>(stream));
}

size_t gt_qk_norm_workspace_size(int32_t d) {
    return d < 1 || d > gt::kMaxD ? 0 : (size_t)gt::most_ctas() * d * sizeof(float) + 512;
}

int gt_qk_norm_bwd(int32_t xtype, int32_t ytype, int32_t d, float eps, const float* freq, int32_t rot, int32_t pairs,
                   int32_t nq, int32_t h, const void* dyq, int64_t lddyq, int64_t hddyq, const void* q, int64_t ldq,
                   int64_t hdq, const float* gain_q, const int32_t* pos_q, void* dq, int64_t lddq, int64_t hddq, float* dgain_q,
                   int32_t nk, int32_t hk, const void* dyk, int64_t lddyk, int64_t hddyk, const void* k, int64_t ldk,
                   int64_t hdk, const float* gain_k, const int32_t* pos_k, void* dk, int64_t lddk, int64_t hddk, float* dgain_k,
                   void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt;
    Job J = {};
    J.side[0] = Side{q, dyq, dq, gain_q, pos_q, nullptr, dgain_q, ldq, hdq, lddyq, hddyq, lddq, hddq, nq, h, 1, 0};
    J.side[1] = Side{k, dyk, dk, gain_k, pos_k, nullptr, dgain_k, ldk, hdk, lddyk, hddyk, lddk, hddk, nk, hk, 1, 0};
    const int rc = check(xtype, ytype, d, eps, freq, rot, pairs, J);
    if (rc != GT_OK) return rc;
    for (const Side& S : J.side)
        if (S.x && (!S.dy || !S.dgain)) return GT_ERR_INVALID_ARG;
    Carve cv(workspace, ws_bytes);
    float* part = cv.take<float>((size_t)most_ctas() * d);
    if (!workspace || !aligned16(workspace) || !cv.fits()) return GT_ERR_WORKSPACE;
    J.side[0].part = part;
    return dispatch<true>(xtype, ytype, J, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
