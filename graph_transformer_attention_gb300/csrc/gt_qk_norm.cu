// gt_qk_norm.cu -- the norm of every head of the queries and keys, with the rotation
// of their channel pairs by position in the same pass, forward and backward.
//
//   forward   r = 1 / sqrt(sum_c x_c^2 / d + eps),  y = R (gain x r)
//   backward  g = R^T dy,  w = gain g,
//             dx = r (w - x r^2 sum_c w_c x_c / d),  dgain = sum over rows and heads of g x r
//
// R turns the pair (a, b) of channels by the angle pos * freq: (a cos - b sin, a sin + b cos).
//
// The bytes of x, y (dy, dx) bound it.  A head's channels are dealt to a few lanes of a warp, both channels of a pair
// to the same lane, so that the norm is a few shuffles and the turn none; every row is read once and nothing
// but gradients is kept for the backward, which forms r again from the x it reads anyway.  The angles are the same for
// all heads of a row: a CTA computes the cosines and sines of its rows once, into shared memory.
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
constexpr int kMaxD = 256;
constexpr int kMaxHeads = 1024;
constexpr int kAngles = 2048;   // cosines and sines of a CTA's rows: 16 KB

// cos and sin of pos * freq to fp32 accuracy however far the position.  pos * freq is N 2^e with a whole N < 2^55; the
// angle in turns is that over 2 pi, and only its fraction matters (Payne and Hanek 1983): N times 96 binary digits of
// 1 / (2 pi) in integers, which leaves the fraction off by less than 2^(e - 41) turns, e <= 0 for |freq| < 2^24 (a larger
// freq loses digits).
__device__ __forceinline__ float2 turn_of(int pos, float freq) {
    const uint32_t bits = __float_as_uint(freq), ex = (bits >> 23) & 255u;
    if (ex == 255u) return make_float2(NAN, NAN);
    const uint32_t mant = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int e = (int)(ex ? ex : 1u) - 150;                        // freq = mant 2^e
    const uint64_t n = (uint64_t)(pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos) * mant;
    const uint64_t c_hi = 0x28BE60DB9391054Aull;                    // 1 / (2 pi): the first 64 digits and the next 32
    const uint32_t c_lo = 0x7F09D5F4u;
    const uint64_t tail = (uint64_t)((((unsigned __int128)n * c_lo)) >> 32);
    const unsigned __int128 t = (unsigned __int128)n * c_hi + tail;   // 64 whole and 64 fraction digits
    uint64_t f = e <= -128 ? 0u : e <= 0 ? (uint64_t)(t >> -e) : e < 64 ? (uint64_t)(t << e) : 0u;
    if ((pos < 0) != ((bits >> 31) != 0)) f = 0u - f;
    float s, c;
    sincospif((float)(int64_t)f * 0x1p-63f, &s, &c);                // two half turns to a turn
    return make_float2(c, s);
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
    int rows;                // rows a CTA takes at a time
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

// V consecutive elements
template <int V, typename T>
__device__ __forceinline__ void get(const T* p, float (&v)[V]) {
    if constexpr (V == 8) {
        unpack8(load8(p, 8, 1), v);
    } else if constexpr (V == 4 && sizeof(T) == 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p));
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else if constexpr (V == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
        v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = to_f32(p[i]);
    }
}

template <int V, typename T>
__device__ __forceinline__ void put(T* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        store8(p, v, 8, 1);
    } else if constexpr (V == 4 && sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = from_f32<T>(v[i]);
    }
}

// What a lane holds of a head: NS slots of two pieces of V channels.  With V > 1 slot s is the channels V s .. and
// d / 2 + V s .. (all channels turn, or none); with V = 1 it is the pair s where s < rot / 2, and past the turning channels
// two neighbours, the second of which may be missing.
template <int V, int NS>
struct Held {
    float a[NS][V], b[NS][V];
};

template <int V>
struct Slot {
    int a, b;    // channels; -1: none
};

template <int V>
__device__ __forceinline__ Slot<V> slot_of(const Job& J, int s) {
    if constexpr (V > 1) {
        return Slot<V>{V * s < J.d / 2 ? V * s : -1, V * s < J.d / 2 ? J.d / 2 + V * s : -1};
    } else {
        const int half = J.rot >> 1;
        if (s < half) return J.adjacent ? Slot<V>{2 * s, 2 * s + 1} : Slot<V>{s, s + half};
        const int c = J.rot + 2 * (s - half);
        return Slot<V>{c < J.d ? c : -1, c + 1 < J.d ? c + 1 : -1};
    }
}

template <int V, int NS, typename T>
__device__ __forceinline__ void load_held(const Slot<V> (&sl)[NS], const T* p, Held<V, NS>& v) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (sl[i].a >= 0) get<V>(p + sl[i].a, v.a[i]);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) v.a[i][j] = 0.f;
        if (sl[i].b >= 0) get<V>(p + sl[i].b, v.b[i]);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) v.b[i][j] = 0.f;
    }
}

template <int V, int NS, typename T>
__device__ __forceinline__ void store_held(const Slot<V> (&sl)[NS], T* p, const Held<V, NS>& v) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (sl[i].a >= 0) put<V>(p + sl[i].a, v.a[i]);
        if (sl[i].b >= 0) put<V>(p + sl[i].b, v.b[i]);
    }
}

__device__ __forceinline__ void turn(float& a, float& b, float2 cs, bool back) {
    const float s = back ? -cs.y : cs.y, t = a * cs.x - b * s;
    b = a * s + b * cs.x;
    a = t;
}

// R v, or R^T v; cs: the row's cosines and sines by pair
template <int V, int NS>
__device__ __forceinline__ void turn_held(const Job& J, const Slot<V> (&sl)[NS], int first, const float2* cs, Held<V, NS>& v,
                                          bool back) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if constexpr (V == 1) {
            const int s = first + i * J.lanes;
            if (s < (J.rot >> 1)) turn(v.a[i][0], v.b[i][0], cs[s], back);
        } else if (sl[i].a >= 0) {
            if (J.adjacent) {
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    turn(v.a[i][j], v.a[i][j + 1], cs[(sl[i].a + j) >> 1], back);
                    turn(v.b[i][j], v.b[i][j + 1], cs[(sl[i].b + j) >> 1], back);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) turn(v.a[i][j], v.b[i][j], cs[sl[i].a + j], back);
            }
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A CTA takes `rows` rows at a time; its threads are groups of `lanes`, a head each.
template <typename TX, typename TY, int V, int NS, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm(const __grid_constant__ Job J) {
    __shared__ float2 angles[kAngles];
    __shared__ float red[BWD ? kThreads * 2 : 1];
    const int which = blockIdx.x < J.side[0].ctas ? 0 : 1;
    const Side& S = J.side[which];
    const int cta = blockIdx.x - (which ? J.side[0].ctas : 0);
    const int first = threadIdx.x & (J.lanes - 1), group = threadIdx.x / J.lanes, groups = kThreads / J.lanes;
    const int half = J.rot >> 1, h = S.h;
    Slot<V> sl[NS];
    Held<V, NS> gain, sum;
#pragma unroll
    for (int i = 0; i < NS; ++i) sl[i] = slot_of<V>(J, first + i * J.lanes);
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            gain.a[i][j] = sl[i].a >= 0 ? __ldg(S.gain + sl[i].a + j) : 0.f;
            gain.b[i][j] = sl[i].b >= 0 ? __ldg(S.gain + sl[i].b + j) : 0.f;
            sum.a[i][j] = sum.b[i][j] = 0.f;
        }
    for (int64_t row0 = (int64_t)cta * S.rows; row0 < S.n; row0 += (int64_t)S.ctas * S.rows) {
        const int rows = (int)(S.n - row0 < S.rows ? S.n - row0 : S.rows);
        if (half > 0) {
            if (row0 != (int64_t)cta * S.rows) __syncthreads();   // the last rows' angles have been read
            for (int k = threadIdx.x; k < rows * half; k += kThreads) {
                const int r = k / half, p = k - r * half;
                angles[k] = turn_of(S.pos ? __ldg(S.pos + row0 + r) : (int)(row0 + r), __ldg(J.freq + p));
            }
            __syncthreads();
        }
        const int items = rows * h;
        // (every lane of a warp makes every turn: the shuffles need them all)
        for (int it0 = 0; it0 < items; it0 += groups) {
            const bool live = it0 + group < items;
            const int it = live ? it0 + group : 0, r = it / h, head = it - r * h;
            const int64_t row = row0 + r;
            const TX* x = static_cast<const TX*>(S.x) + row * S.ldx + head * S.hdx;
            Held<V, NS> v;
            load_held<V, NS>(sl, x, v);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) ss += v.a[i][j] * v.a[i][j] + v.b[i][j] * v.b[i][j];
            if constexpr (!BWD) {
                const float rs = 1.f / sqrtf(lanes_sum(ss, J.lanes) * J.inv_d + J.eps);
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        v.a[i][j] *= rs * gain.a[i][j];
                        v.b[i][j] *= rs * gain.b[i][j];
                    }
                if (half > 0) turn_held<V, NS>(J, sl, first, angles + r * half, v, false);
                if (live) store_held<V, NS>(sl, static_cast<TY*>(S.y) + row * S.ldy + head * S.hdy, v);
            } else {
                Held<V, NS> g;
                load_held<V, NS>(sl, static_cast<const TY*>(S.dy) + row * S.lddy + head * S.hddy, g);
                if (half > 0) turn_held<V, NS>(J, sl, first, angles + r * half, g, true);
                float wx = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        wx += gain.a[i][j] * g.a[i][j] * v.a[i][j] + gain.b[i][j] * g.b[i][j] * v.b[i][j];
                const float rs = 1.f / sqrtf(lanes_sum(ss, J.lanes) * J.inv_d + J.eps);
                const float back = rs * rs * lanes_sum(wx, J.lanes) * J.inv_d;
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (live) {
                            sum.a[i][j] += g.a[i][j] * (v.a[i][j] * rs);
                            sum.b[i][j] += g.b[i][j] * (v.b[i][j] * rs);
                        }
                        v.a[i][j] = rs * (gain.a[i][j] * g.a[i][j] - v.a[i][j] * back);
                        v.b[i][j] = rs * (gain.b[i][j] * g.b[i][j] - v.b[i][j] * back);
                    }
                if (live) store_held<V, NS>(sl, static_cast<TX*>(S.y) + row * S.ldy + head * S.hdy, v);
            }
        }
    }
    if constexpr (BWD) {
        sm100::pdl_trigger();
        // the groups' sums, one channel of each piece at a time, in the groups' order
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                __syncthreads();
                red[threadIdx.x] = sum.a[i][j];
                red[kThreads + threadIdx.x] = sum.b[i][j];
                __syncthreads();
                if ((int)threadIdx.x < J.lanes) {
                    float ta = 0.f, tb = 0.f;
                    for (int k = 0; k < groups; ++k) {
                        ta += red[k * J.lanes + threadIdx.x];
                        tb += red[kThreads + k * J.lanes + threadIdx.x];
                    }
                    if (sl[i].a >= 0) S.part[(int64_t)cta * J.d + sl[i].a + j] = ta;
                    if (sl[i].b >= 0) S.part[(int64_t)cta * J.d + sl[i].b + j] = tb;
                }
            }
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
    if (c < J.d)
        for (int p = ty; p < S.ctas; p += kSumThreads / 32) acc += __ldcg(S.part + (int64_t)p * J.d + c);
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

// The largest V with which all of a call's pieces are aligned accesses: 16 bytes of x where they can be.
template <typename TX, typename TY>
int piece_of(const Job& J, bool bwd) {
    if (J.rot != 0 && J.rot != J.d) return 1;
    for (int v = sizeof(TX) == 2 ? 8 : 4; v > 1; v /= 2) {
        bool ok = v >= 4 && (J.d / 2) % v == 0 && J.d % 2 == 0;
        for (const Side& S : J.side) {
            if (!S.x) continue;
            const int px = std::min<int>(16, v * (int)sizeof(TX)), py = std::min<int>(16, v * (int)sizeof(TY));
            ok = ok && pieces16(S.x, S.ldx, S.hdx, sizeof(TX), px);
            ok = ok && pieces16(S.y, S.ldy, S.hdy, bwd ? sizeof(TX) : sizeof(TY), bwd ? px : py);
            if (bwd) ok = ok && pieces16(S.dy, S.lddy, S.hddy, sizeof(TY), py);
        }
        if (ok) return v;
    }
    return 1;
}

// CTAs of the backward at most, each of which makes one partial row
int most_ctas() { return 4 * num_sms(); }

// How the rows are dealt: about four heads to a group of lanes at a time, as far as the angles' table goes.
void deal(Job& J, int v, bool bwd) {
    const int slots = v > 1 ? J.d / 2 / v : (J.rot / 2 + (J.d - J.rot + 1) / 2);
    J.lanes = 1;
    while (J.lanes < slots && J.lanes < 32) J.lanes *= 2;
    int64_t all = 0;
    for (Side& S : J.side) {
        if (!S.x) { S.ctas = 0; S.rows = 1; continue; }
        const int groups = kThreads / J.lanes;
        int64_t rows = std::max(1, 4 * groups / S.h);
        if (J.rot) rows = std::min<int64_t>(rows, kAngles / (J.rot / 2));
        // enough CTAs for every SM first
        rows = std::max<int64_t>(1, std::min<int64_t>(rows, S.n / (2 * num_sms())));
        S.rows = (int)rows;
        S.ctas = (int)((S.n + rows - 1) / rows);
        all += S.ctas;
    }
    if (!bwd || all <= most_ctas()) return;
    for (Side& S : J.side)
        if (S.x) S.ctas = (int)std::max<int64_t>(1, (int64_t)S.ctas * (most_ctas() - 2) / all);
}

template <typename TX, typename TY, bool BWD>
int run(Job& J, cudaStream_t s) {
    const int v = piece_of<TX, TY>(J, BWD);
    deal(J, v, BWD);
    const int grid = J.side[0].ctas + J.side[1].ctas;
    // the keys' partial rows follow the queries'; deal() keeps both together within most_ctas()
    if (BWD) J.side[1].part = J.side[0].part + (int64_t)J.side[0].ctas * J.d;
    {
        LaunchScope ls(BWD ? "qk_norm_bwd" : "qk_norm_fwd", s);
        if (v == 8) {
            if constexpr (sizeof(TX) == 2) qk_norm<TX, TY, 8, 1, BWD><<<grid, kThreads, 0, s>>>(J);
        } else if (v == 4) {
            qk_norm<TX, TY, 4, 1, BWD><<<grid, kThreads, 0, s>>>(J);
        } else if (J.d <= 63) {   // at most 32 slots
            qk_norm<TX, TY, 1, 1, BWD><<<grid, kThreads, 0, s>>>(J);
        } else {
            qk_norm<TX, TY, 1, 4, BWD><<<grid, kThreads, 0, s>>>(J);
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
