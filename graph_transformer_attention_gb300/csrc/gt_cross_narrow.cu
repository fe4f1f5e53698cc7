// gt_cross_narrow.cu -- cross attention of fp32 storage with head dims up to 16, on the CUDA cores.
//
// Four threads to a row of the held side (queries for o and dq, keys for dk and dv), each with the row in registers and
// every fourth row of the streamed tiles, which stand in shared memory and are read by broadcast; the four join at the
// end. A score then costs its d multiply-adds and nothing to lay down weights (the tiles of 64 x 64 of the wider head
// dims pad d to 16 and move every weight through shared memory: 128 queries over 6800 keys, 8 heads of 8, dq 36.7 and dk,
// dv 47.1 us). The next tile's rows are on their way while a tile is worked on.  The issue slots bound it, and at the
// sizes that do not fill the SMs the latency of a tile: 128 queries over 6800 keys, 8 heads of 8, dq 23 us, dk and dv 27;
// 4096 over 6800 forward 510, backward 909, 8 heads of 16 981 and 1722.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gt_cross.cuh"
#include "gt_stats.cuh"

namespace gt {
namespace cross {
namespace {

constexpr int kHeld = 64, kStream = 128, kThreads = 256, kPhases = 4;

// Rows of one side: row r is query r / g (or key r with g = 1) and head r % g from p on.
struct Rows {
    const float* p;
    int64_t row, head;
    int g;
    bool vec;      // 16-byte accesses
};

__device__ __forceinline__ Rows rows_of(const View& v, int64_t first, int head, int g, bool vec) {
    return Rows{static_cast<const float*>(v.p) + first * v.row + (int64_t)head * v.head, v.row, v.head, g, vec};
}

// Four channels of a row, zeros past d and where there is no row.
__device__ __forceinline__ float4 get4(const Rows& R, int r, bool there, int c, int d) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!there || c >= d) return v;
    const float* p = R.p + (int64_t)(r / R.g) * R.row + (r % R.g) * R.head + c;
    if (R.vec && c + 4 <= d) return __ldg(reinterpret_cast<const float4*>(p));
    v.x = p[0];
    if (c + 1 < d) v.y = p[1];
    if (c + 2 < d) v.z = p[2];
    if (c + 3 < d) v.w = p[3];
    return v;
}

// A row in registers, as pairs for the packed arithmetic.
template <int DP>
struct Row {
    float2 v[DP / 2];
};

template <int DP>
__device__ __forceinline__ Row<DP> get_row(const Rows& R, int r, bool there, int d) {
    Row<DP> x;
#pragma unroll
    for (int c = 0; c < DP; c += 4) {
        const float4 v = get4(R, r, there, c, d);
        x.v[c / 2] = make_float2(v.x, v.y);
        x.v[c / 2 + 1] = make_float2(v.z, v.w);
    }
    return x;
}

// The streamed rows: two arrays, two numbers to a row.
template <int DP>
struct Tiles {
    static constexpr int kLd = DP + (DP > 8 ? 4 : 0);      // (rows of four phases in different banks)
    alignas(16) float a[kStream * kLd];
    alignas(16) float b[kStream * kLd];
    float2 s[kStream];
};

template <int DP>
struct Staged {
    static constexpr int N = kStream * DP / 4 / kThreads;
    float4 a[N], b[N];
    float2 s;
};

template <int DP>
__device__ __forceinline__ void put(Tiles<DP>& T, const Staged<DP>& st) {
#pragma unroll
    for (int i = 0; i < Staged<DP>::N; ++i) {
        const int at = threadIdx.x + i * kThreads, r = at / (DP / 4), c = at % (DP / 4) * 4;
        *reinterpret_cast<float4*>(&T.a[r * T.kLd + c]) = st.a[i];
        *reinterpret_cast<float4*>(&T.b[r * T.kLd + c]) = st.b[i];
    }
    if (threadIdx.x < kStream) T.s[threadIdx.x] = st.s;
}

template <int DP>
__device__ __forceinline__ Row<DP> row_at(const float* tile, int r) {
    Row<DP> x;
#pragma unroll
    for (int c = 0; c < DP; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(tile + r * Tiles<DP>::kLd + c);
        x.v[c / 2] = make_float2(v.x, v.y);
        x.v[c / 2 + 1] = make_float2(v.z, v.w);
    }
    return x;
}

template <int DP>
__device__ __forceinline__ float dot(const Row<DP>& x, const Row<DP>& y) {
    float2 a = __fmul2_rn(x.v[0], y.v[0]);
#pragma unroll
    for (int c = 1; c < DP / 2; ++c) a = __ffma2_rn(x.v[c], y.v[c], a);
    return a.x + a.y;
}

template <int DP>
__device__ __forceinline__ void axpy(float w, const Row<DP>& x, Row<DP>& y) {
    const float2 w2 = make_float2(w, w);
#pragma unroll
    for (int c = 0; c < DP / 2; ++c) y.v[c] = __ffma2_rn(w2, x.v[c], y.v[c]);
}

template <int DP>
__device__ __forceinline__ void times(float w, Row<DP>& y) {
    const float2 w2 = make_float2(w, w);
#pragma unroll
    for (int c = 0; c < DP / 2; ++c) y.v[c] = __fmul2_rn(w2, y.v[c]);
}

template <int DP>
__device__ __forceinline__ void put_row(float* p, int d, int phase, const Row<DP>& x, float by) {
#pragma unroll
    for (int c = 0; c < DP; ++c)
        if (c % kPhases == phase && c < d) p[c] = (c & 1 ? x.v[c / 2].y : x.v[c / 2].x) * by;      // (all four threads of the row have it)
}

template <int DP>
__device__ __forceinline__ void phases_sum(Row<DP>& x) {
#pragma unroll
    for (int c = 0; c < DP / 2; ++c)
#pragma unroll
        for (int o = 1; o < kPhases; o <<= 1) {
            x.v[c].x += __shfl_xor_sync(0xffffffffu, x.v[c].x, o);
            x.v[c].y += __shfl_xor_sync(0xffffffffu, x.v[c].y, o);
        }
}

struct Vec {
    bool q, k, v, dO;
};

// Keys of streamed tile n, on their way: k, v and whether anyone sees the key: what is added to a score (0 or
// -infinity), and what bounds it (either infinity).
template <int DP>
__device__ __forceinline__ void fetch_keys(const Shape& S, const Tile& t, const Rows& k, const Rows& v, int n, Staged<DP>& st) {
    const int k0 = n * kStream, keys = min(kStream, t.lk - k0);
    auto seen = [&](int r) { return r < keys && (!S.mask || __ldg(S.mask + t.k0 + k0 + r) != 0); };
#pragma unroll
    for (int i = 0; i < Staged<DP>::N; ++i) {
        const int at = threadIdx.x + i * kThreads, r = at / (DP / 4), c = at % (DP / 4) * 4;
        const bool there = seen(r);
        st.a[i] = get4(k, k0 + r, there, c, S.d);
        st.b[i] = get4(v, k0 + r, there, c, S.d);
    }
    if (threadIdx.x < kStream) st.s = seen(threadIdx.x) ? make_float2(0.f, INFINITY) : make_float2(-INFINITY, -INFINITY);
}

template <int DP>
__global__ void __launch_bounds__(kThreads) cross_fwd_narrow(const Shape S, const View q, const View k, const View v,
                                                             const FwdOut out, const Vec vec) {
    __shared__ Tiles<DP> T;
    const int tq = tile_queries(kHeld, S.g), head = blockIdx.y, z = blockIdx.z;
    sm100::pdl_trigger();
    const Tile t = find_tile(S, true, tq, blockIdx.x);
    if (!t.live) return;
    const int r = threadIdx.x / kPhases, phase = threadIdx.x % kPhases;
    const int first = t.tile * tq, live = min(tq, t.lq - first) * S.g;
    const float c = S.scale * tc::kLog2e;
    const Rows kr = rows_of(k, t.k0, head, 1, vec.k), vr = rows_of(v, t.k0, head, 1, vec.v);
    float m = -INFINITY, l = 0.f;
    Row<DP> o = {};
    const Row<DP> x = get_row<DP>(rows_of(q, t.q0 + first, head * S.g, S.g, vec.q), r, r < live, S.d);
    const int tiles = (t.lk + kStream - 1) / kStream, end = part_begin(tiles, z + 1, out.splits);
    int n = part_begin(tiles, z, out.splits);
    Staged<DP> st;
    if (n < end) fetch_keys<DP>(S, t, kr, vr, n, st);
    for (; n < end; ++n) {
        __syncthreads();
        put<DP>(T, st);
        __syncthreads();
        if (n + 1 < end) fetch_keys<DP>(S, t, kr, vr, n + 1, st);
#pragma unroll 1
        for (int j0 = phase; j0 < kStream; j0 += 4 * kPhases) {
            float s[4], top = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // (the smaller of two is never a NaN: a key that nobody sees gives -infinity whatever the query holds; the NaN
                // of a key that is seen becomes infinity, and its weight NaN again)
                s[u] = fminf(dot<DP>(x, row_at<DP>(T.a, j0 + u * kPhases)) * c, T.s[j0 + u * kPhases].y);
                top = fmaxf(top, s[u]);
            }
            const float base = top == -INFINITY ? 0.f : top, by = sm100::ex2(m - base);
            m = top;
            l *= by;
            times<DP>(by, o);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float p = sm100::ex2(s[u] - base);
                l += p;
                axpy<DP>(p, row_at<DP>(T.b, j0 + u * kPhases), o);
            }
        }
    }
    // the four phases on one base
    float top = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float by = m == -INFINITY ? 0.f : sm100::ex2(m - top);
    l *= by;
    times<DP>(by, o);
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    phases_sum<DP>(o);
    if (r >= live) return;
    const int64_t query = t.q0 + first + r / S.g;
    const int qh = head * S.g + r % S.g;
    const bool some = l != 0.f;      // (a NaN counts)
    const float inv = some ? 1.f / l : 0.f, lse = some ? (top + log2f(l)) * tc::kLn2 : -INFINITY;
    const bool whole = out.splits == 1;
    put_row<DP>(whole ? static_cast<float*>(out.o.p) + query * out.o.row + qh * out.o.head
                      : out.o_part + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d,
                S.d, phase, o, inv);
    if (phase == 0) *(whole ? out.lse + (int64_t)qh * S.nq + query : out.lse_part + (z * (int64_t)S.h + qh) * S.nq + query) = lse;
}

// KEYS: the held side is the keys (dk, dv), else the queries (dq).
template <int DP, bool KEYS>
__global__ void __launch_bounds__(kThreads, DP == 8 ? 3 : 2) cross_bwd_narrow(const Shape S, const BwdIn in, const Out g1, const Out g2,
                                                             float* __restrict__ part1, float* __restrict__ part2, int splits,
                                                             const Vec vec) {
    __shared__ Tiles<DP> T;
    const int tq = tile_queries(KEYS ? kStream : kHeld, S.g), head = blockIdx.y, z = blockIdx.z;
    if (KEYS) sm100::pdl_trigger();
    const Tile t = find_tile(S, !KEYS, KEYS ? kHeld : tq, blockIdx.x);
    if (!KEYS) follow_stats();
    if (!t.live) {
        if (KEYS) sm100::pdl_wait();
        return;
    }
    const int r = threadIdx.x / kPhases, phase = threadIdx.x % kPhases;
    const float c = S.scale * tc::kLog2e;
    // (a sequence may have more than 2^31 rows (query, head): a tile's rows are counted from its first query on)
    auto q_rows = [&](int query) { return rows_of(in.q, t.q0 + (int64_t)query, head * S.g, S.g, vec.q); };
    auto do_rows = [&](int query) { return rows_of(in.dO, t.q0 + (int64_t)query, head * S.g, S.g, vec.dO); };
    auto stats_of = [&](int query) { return in.stats + ((int64_t)head * S.nq + t.q0 + query) * S.g; };
    const Rows kr = rows_of(in.k, t.k0, head, 1, vec.k), vr = rows_of(in.v, t.k0, head, 1, vec.v);
    const int first = t.tile * (KEYS ? kHeld : tq);
    const int live = KEYS ? min(kHeld, t.lk - first) : min(tq, t.lq - first) * S.g;
    const int tiles = KEYS ? (t.lq + tq - 1) / tq : (t.lk + kStream - 1) / kStream;
    Row<DP> x1, x2, a1 = {}, a2 = {};
    float2 own;      // dq: -lse and -D of the row; dk, dv: 0 or -infinity
    if (KEYS) {
        const bool seen = r < live && (!S.mask || __ldg(S.mask + t.k0 + first + r) != 0);
        x1 = get_row<DP>(kr, first + r, seen, S.d);
        x2 = get_row<DP>(vr, first + r, seen, S.d);
        own = make_float2(seen ? 0.f : -INFINITY, 0.f);
    } else {
        x1 = get_row<DP>(q_rows(first), r, r < live, S.d);
        x2 = get_row<DP>(do_rows(first), r, r < live, S.d);
        own = r < live ? __ldg(stats_of(first) + r) : make_float2(-INFINITY, 0.f);
    }
    auto fetch = [&](int n, Staged<DP>& st) {
        if (!KEYS) {
            fetch_keys<DP>(S, t, kr, vr, n, st);
            return;
        }
        const int query = n * tq, rows = min(tq, t.lq - query) * S.g;
        const Rows qr = q_rows(query), dr = do_rows(query);
#pragma unroll
        for (int i = 0; i < Staged<DP>::N; ++i) {
            const int at = threadIdx.x + i * kThreads, row = at / (DP / 4), col = at % (DP / 4) * 4;
            st.a[i] = get4(qr, row, row < rows, col, S.d);
            st.b[i] = get4(dr, row, row < rows, col, S.d);
        }
        if (threadIdx.x < kStream)
            st.s = (int)threadIdx.x < rows ? __ldg(stats_of(query) + threadIdx.x) : make_float2(-INFINITY, 0.f);
    };
    const int end = part_begin(tiles, z + 1, splits);
    int n = part_begin(tiles, z, splits);
    Staged<DP> st;
    if (n < end) fetch(n, st);
    for (; n < end; ++n) {
        __syncthreads();
        put<DP>(T, st);
        __syncthreads();
        if (n + 1 < end) fetch(n + 1, st);
        // (queries that are not there are left out: 0 times an infinity of the key would be NaN)
        const int rows = KEYS ? min(tq, t.lq - n * tq) * S.g : kStream;
#pragma unroll 4
        for (int j = phase; j < rows; j += kPhases) {
            const Row<DP> y1 = row_at<DP>(T.a, j), y2 = row_at<DP>(T.b, j);
            const float2 s = T.s[j];
            // (where nobody sees the key both factors are 0: the rows were cleared, the exponent is -infinity; unless the query
            // is not a number: see below)
            const float p = sm100::ex2(fmaf(dot<DP>(x1, y1), c, own.x + s.x));
            const float ds = p * (dot<DP>(x2, y2) + (KEYS ? s.y : own.y));
            if (KEYS) axpy<DP>(p, y2, a2);
            axpy<DP>(ds, y1, a1);
        }
    }
    phases_sum<DP>(a1);
    if (KEYS) phases_sum<DP>(a2);
    if (KEYS) sm100::pdl_wait();
    if (r >= live) return;
    if (own.x == -INFINITY) a1 = a2 = Row<DP>{};      // a key that nobody sees, a query that sees none
    if (KEYS) {
        const int64_t key = t.k0 + first + r, at = ((z * (int64_t)S.nk + key) * S.hk + head) * S.d;
        put_row<DP>(splits == 1 ? static_cast<float*>(g1.p) + key * g1.row + head * g1.head : part1 + at, S.d, phase, a1, S.scale);
        put_row<DP>(splits == 1 ? static_cast<float*>(g2.p) + key * g2.row + head * g2.head : part2 + at, S.d, phase, a2, 1.f);
    } else {
        const int64_t query = t.q0 + first + r / S.g;
        const int qh = head * S.g + r % S.g;
        put_row<DP>(splits == 1 ? static_cast<float*>(g1.p) + query * g1.row + qh * g1.head
                                : part1 + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d,
                    S.d, phase, a1, S.scale);
    }
}

bool vec16(const View& v) { return aligned16(v.p) && v.row % 4 == 0 && v.head % 4 == 0; }

template <typename F>
int by_width(int d, F&& f) {
    return d <= 8 ? f(std::integral_constant<int, 8>()) : f(std::integral_constant<int, 16>());
}

}  // namespace

int fwd_narrow(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s) {
    return by_width(S.d, [&](auto width) {
        LaunchScope ls("cross_fwd_narrow", s);
        cross_fwd_narrow<decltype(width)::value>
            <<<dim3(slots_of(S, true, tile_queries(kHeld, S.g)), S.hk, out.splits), kThreads, 0, s>>>(
                S, q, k, v, out, Vec{vec16(q), vec16(k), vec16(v), false});
        return check_launch();
    });
}

template <bool KEYS>
static int bwd_narrow(const Shape& S, const BwdIn& in, const Out& g1, const Out& g2, float* p1, float* p2, int splits,
                      cudaStream_t s) {
    return by_width(S.d, [&](auto width) {
        LaunchScope ls(KEYS ? "cross_dkv_narrow" : "cross_dq_narrow", s);
        const Vec vec{vec16(in.q), vec16(in.k), vec16(in.v), vec16(in.dO)};
        if (launch_overlapped(cross_bwd_narrow<decltype(width)::value, KEYS>,
                              dim3(slots_of(S, !KEYS, KEYS ? kHeld : tile_queries(kHeld, S.g)), S.hk, splits), dim3(kThreads), 0, s,
                              S, in, g1, g2, p1, p2, splits, vec) != cudaSuccess)
            return (int)GT_ERR_CUDA;
        return check_launch();
    });
}

int bwd_dq_narrow(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s) {
    return bwd_narrow<false>(S, in, dq, Out{}, part, nullptr, splits, s);
}

int bwd_dkv_narrow(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
                   cudaStream_t s) {
    return bwd_narrow<true>(S, in, dk, dv, dk_part, dv_part, splits, s);
}

}  // namespace cross
}  // namespace gt
