// gt_cross_simt.cu -- cross attention of fp32 storage, head dims above 16: fp32 products on the CUDA cores.
//
// One skeleton for the three passes.  A CTA holds a tile of 64 rows of one side (queries for o and dq, keys
// for dk and dv) and streams tiles of 64 rows of the other: the 64 x 64 scores as 4 x 4 blocks of 256
// threads, turned into weights, laid down in shared memory and multiplied with the streamed rows.  Tiles stand
// row by row with four floats between rows, so that both products read 16 bytes at a time without bank conflicts
// (two such reads to sixteen multiply-adds) and no tile is ever transposed.
//
// The multiply-adds of the fp32 pipes bound it.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "gt_cross.cuh"
#include "gt_stats.cuh"

namespace gt {
namespace cross {
namespace {

constexpr int kRows = 64;
constexpr int kThreads = 256;
constexpr int kLdw = kRows + 4;

template <int DP> constexpr int ldt() { return DP + 4; }

// Row r of a tile to its place: queries q0 + r / g of head first_head + r % g; keys with g = 1.
struct Rows {
    const float* p;
    int64_t row, head;
    int g, live;      // live: rows that exist
    bool vec;         // 16-byte accesses
};

// keep: NULL, or a byte to a row: 0 leaves zeros
template <int DP>
__device__ __forceinline__ void load_tile(float* dst, const Rows& R, int d, const uint8_t* keep) {
    constexpr int Q = DP / 4;
    for (int k = threadIdx.x; k < kRows * Q; k += kThreads) {
        const int r = k / Q, c = (k - r * Q) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < R.live && c < d && (!keep || keep[r])) {
            const float* p = R.p + (int64_t)(r / R.g) * R.row + (r % R.g) * R.head + c;
            if (R.vec && c + 4 <= d) {
                v = __ldg(reinterpret_cast<const float4*>(p));
            } else {
                v.x = p[0];
                if (c + 1 < d) v.y = p[1];
                if (c + 2 < d) v.z = p[2];
                if (c + 3 < d) v.w = p[3];
            }
        }
        *reinterpret_cast<float4*>(dst + r * ldt<DP>() + c) = v;
    }
}

// x[i][j] = <row 4 ty + i of a, row tx + 16 j of b>
template <int DP>
__device__ __forceinline__ void tile_dot(const float* a, const float* b, int ty, int tx, float (&x)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
        float4 u[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * ldt<DP>() + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ldt<DP>() + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = fmaf(u[i].x, w[j].x, x[i][j]);
                x[i][j] = fmaf(u[i].y, w[j].y, x[i][j]);
                x[i][j] = fmaf(u[i].z, w[j].z, x[i][j]);
                x[i][j] = fmaf(u[i].w, w[j].w, x[i][j]);
            }
    }
}

// The columns of a DP-wide row that thread tx sums: 4 of every 64 (2 of 32)
template <int DP> constexpr int cols_per_thread() { return DP / 16; }
template <int DP>
__device__ __forceinline__ int col_of(int tx, int n) {
    constexpr int W = DP >= 64 ? 4 : DP / 16;
    return (n / W) * 64 + tx * W + n % W;
}

// acc[i][n] += sum over the tile's rows j of weight[4 ty + i][j] * b[j][col_of(tx, n)]
template <int DP>
__device__ __forceinline__ void tile_acc(const float* weight, const float* b, int ty, int tx,
                                         float (&acc)[4][cols_per_thread<DP>()]) {
    constexpr int C = cols_per_thread<DP>();
#pragma unroll 2
    for (int j = 0; j < kRows; j += 4) {
        float w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(weight + (4 * ty + i) * kLdw + j);
            w[i][0] = f.x; w[i][1] = f.y; w[i][2] = f.z; w[i][3] = f.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float x[C];
            const float* row = b + (j + u) * ldt<DP>();
            if constexpr (DP >= 64) {
#pragma unroll
                for (int n = 0; n < C; n += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(row + col_of<DP>(tx, n));
                    x[n] = f.x; x[n + 1] = f.y; x[n + 2] = f.z; x[n + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int n = 0; n < C; ++n) x[n] = row[col_of<DP>(tx, n)];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < C; ++n) acc[i][n] = fmaf(w[i][u], x[n], acc[i][n]);
        }
    }
}

template <int DP>
__device__ __forceinline__ void put_weights(float* weight, int ty, int tx, const float (&x)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) weight[(4 * ty + i) * kLdw + tx + 16 * j] = x[i][j];
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ Rows rows_of(const View& v, int64_t first, int head, int g, int live, bool vec) {
    return Rows{static_cast<const float*>(v.p) + first * v.row + (int64_t)head * v.head, v.row, v.head, g, live, vec};
}

template <int DP>
__device__ __forceinline__ void put_row(float* p, int tx, int d, const float (&v)[cols_per_thread<DP>()], float by) {
#pragma unroll
    for (int n = 0; n < cols_per_thread<DP>(); ++n) {
        const int c = col_of<DP>(tx, n);
        if (c < d) p[c] = v[n] * by;
    }
}

struct Vec {
    bool q, k, v, dO;
};

template <int DP>
__global__ void __launch_bounds__(kThreads) cross_fwd_f32(const Shape S, const View q, const View k, const View v,
                                                          const FwdOut out, const Vec vec) {
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;
    float* sk = sq + kRows * ldt<DP>();
    float* sv = sk + kRows * ldt<DP>();
    float* sw = sv + kRows * ldt<DP>();
    __shared__ uint8_t keep[kRows];
    const int tq = tile_queries(kRows, S.g), head = blockIdx.y, z = blockIdx.z;
    sm100::pdl_trigger();
    const Tile t = find_tile(S, true, tq, blockIdx.x);
    if (!t.live) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int first = t.tile * tq, queries = min(tq, t.lq - first), live = queries * S.g;
    const float c = S.scale * tc::kLog2e;
    load_tile<DP>(sq, rows_of(q, t.q0 + first, head * S.g, S.g, live, vec.q), S.d, nullptr);
    float o[4][cols_per_thread<DP>()], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int n = 0; n < cols_per_thread<DP>(); ++n) o[i][n] = 0.f;
    }
    const int tiles = (t.lk + kRows - 1) / kRows;
    const int end = part_begin(tiles, z + 1, out.splits);
    for (int kt = part_begin(tiles, z, out.splits); kt < end; ++kt) {
        const int k0 = kt * kRows, keys = min(kRows, t.lk - k0);
        __syncthreads();      // the last tile has been read
        if (threadIdx.x < kRows)
            keep[threadIdx.x] = (int)threadIdx.x < keys && (!S.mask || S.mask[t.k0 + k0 + threadIdx.x] != 0);
        load_tile<DP>(sk, rows_of(k, t.k0 + k0, head, 1, keys, vec.k), S.d, nullptr);
        __syncthreads();
        load_tile<DP>(sv, rows_of(v, t.k0 + k0, head, 1, keys, vec.v), S.d, keep);
        float x[4][4];
        tile_dot<DP>(sq, sk, ty, tx, x);
        float by[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = keep[tx + 16 * j] ? x[i][j] * c : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
            top = row_max(top);
            const float base = top == -INFINITY ? 0.f : top;
            by[i] = sm100::ex2(m[i] - base);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = sm100::ex2(x[i][j] - base);
                sum += x[i][j];
            }
            l[i] = fmaf(l[i], by[i], row_sum(sum));
#pragma unroll
            for (int n = 0; n < cols_per_thread<DP>(); ++n) o[i][n] *= by[i];
        }
        put_weights<DP>(sw, ty, tx, x);
        __syncthreads();
        tile_acc<DP>(sw, sv, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= live) continue;
        const int64_t query = t.q0 + first + r / S.g;
        const int qh = head * S.g + r % S.g;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const float lse = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * tc::kLn2;
        float* dst;
        float* ldst;
        if (out.splits == 1) {
            dst = static_cast<float*>(out.o.p) + query * out.o.row + qh * out.o.head;
            ldst = out.lse + (int64_t)qh * S.nq + query;
        } else {
            dst = out.o_part + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d;
            ldst = out.lse_part + (z * (int64_t)S.h + qh) * S.nq + query;
        }
        put_row<DP>(dst, tx, S.d, o[i], inv);
        if (tx == 0) *ldst = lse;
    }
}

// KEYS: the CTA holds a tile of keys and streams queries (dk, dv); else the other way round (dq).
template <int DP, bool KEYS>
__global__ void __launch_bounds__(kThreads) cross_bwd_f32(const Shape S, const BwdIn in, const Out g1, const Out g2,
                                                          float* __restrict__ part1, float* __restrict__ part2, int splits,
                                                          const Vec vec) {
    extern __shared__ __align__(16) float sm[];
    constexpr int T = kRows * ldt<DP>();
    float* a1 = sm;             // held: q | k
    float* a2 = a1 + T;         // held: dO | v
    float* b1 = a2 + T;         // streamed: k | q
    float* b2 = b1 + T;         // streamed: v | dO
    float* w1 = b2 + T;         // dS
    float* w2 = w1 + kRows * kLdw;   // p (KEYS)
    __shared__ uint8_t keep[kRows];
    __shared__ float2 stat[kRows];
    const int tq = tile_queries(kRows, S.g), head = blockIdx.y, z = blockIdx.z;
    if (KEYS) sm100::pdl_trigger();
    const Tile t = find_tile(S, !KEYS, KEYS ? kRows : tq, blockIdx.x);
    if (!KEYS) follow_stats();
    if (!t.live) {
        if (KEYS) sm100::pdl_wait();
        return;
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float c = S.scale * tc::kLog2e;
    const int tiles = KEYS ? (t.lq + tq - 1) / tq : (t.lk + kRows - 1) / kRows;
    float acc1[4][cols_per_thread<DP>()], acc2[4][cols_per_thread<DP>()];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < cols_per_thread<DP>(); ++n) acc1[i][n] = acc2[i][n] = 0.f;

    auto keys_of = [&](int tile, float* kd, float* vd) {
        const int k0 = tile * kRows, keys = min(kRows, t.lk - k0);
        if (threadIdx.x < kRows)
            keep[threadIdx.x] = (int)threadIdx.x < keys && (!S.mask || S.mask[t.k0 + k0 + threadIdx.x] != 0);
        __syncthreads();
        load_tile<DP>(kd, rows_of(in.k, t.k0 + k0, head, 1, keys, vec.k), S.d, keep);
        load_tile<DP>(vd, rows_of(in.v, t.k0 + k0, head, 1, keys, vec.v), S.d, keep);
    };
    auto queries_of = [&](int tile, float* qd, float* od) {
        const int first = tile * tq, live = min(tq, t.lq - first) * S.g;
        load_tile<DP>(qd, rows_of(in.q, t.q0 + first, head * S.g, S.g, live, vec.q), S.d, nullptr);
        load_tile<DP>(od, rows_of(in.dO, t.q0 + first, head * S.g, S.g, live, vec.dO), S.d, nullptr);
        if (threadIdx.x < kRows)
            stat[threadIdx.x] = (int)threadIdx.x < live
                                    ? __ldg(in.stats + ((int64_t)head * S.nq + t.q0 + first) * S.g + threadIdx.x)
                                    : make_float2(-INFINITY, 0.f);
    };
    if (KEYS) keys_of(t.tile, a1, a2);
    else queries_of(t.tile, a1, a2);
    const int end = part_begin(tiles, z + 1, splits);
    for (int n = part_begin(tiles, z, splits); n < end; ++n) {
        __syncthreads();      // the last tiles have been read
        if (KEYS) queries_of(n, b1, b2);
        else keys_of(n, b1, b2);
        __syncthreads();
        float x[4][4], y[4][4];
        tile_dot<DP>(a1, b1, ty, tx, x);
        tile_dot<DP>(a2, b2, ty, tx, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int held = 4 * ty + i, other = tx + 16 * j;
                const float2 st = stat[KEYS ? other : held];
                // (a query without a key, or that is not there, weighs nothing, whatever its score: with an infinity in the
                // key that may be NaN)
                const bool seen = keep[KEYS ? held : other] && st.x != -INFINITY;
                const float p = seen ? sm100::ex2(fmaf(x[i][j], c, st.x)) : 0.f;
                x[i][j] = p;
                y[i][j] = seen ? p * (y[i][j] + st.y) : 0.f;
            }
        put_weights<DP>(w1, ty, tx, y);
        if (KEYS) put_weights<DP>(w2, ty, tx, x);
        __syncthreads();
        tile_acc<DP>(w1, b1, ty, tx, acc1);
        if (KEYS) tile_acc<DP>(w2, b2, ty, tx, acc2);
    }
    if (KEYS) sm100::pdl_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (KEYS) {
            if (t.tile * kRows + r >= t.lk) continue;
            const int64_t key = t.k0 + (int64_t)t.tile * kRows + r;
            float *pk, *pv;
            if (splits == 1) {
                pk = static_cast<float*>(g1.p) + key * g1.row + head * g1.head;
                pv = static_cast<float*>(g2.p) + key * g2.row + head * g2.head;
            } else {
                const int64_t at = ((z * (int64_t)S.nk + key) * S.hk + head) * S.d;
                pk = part1 + at;
                pv = part2 + at;
            }
            if (!keep[r])      // (weights of 0 do not cancel queries that are not numbers)
#pragma unroll
                for (int n = 0; n < cols_per_thread<DP>(); ++n) acc1[i][n] = acc2[i][n] = 0.f;
            put_row<DP>(pk, tx, S.d, acc1[i], S.scale);
            put_row<DP>(pv, tx, S.d, acc2[i], 1.f);
        } else {
            const int query = t.tile * tq + r / S.g, qh = head * S.g + r % S.g;
            if (r >= tq * S.g || query >= t.lq) continue;
            const int64_t row = t.q0 + query;
            float* p = splits == 1 ? static_cast<float*>(g1.p) + row * g1.row + qh * g1.head
                                   : part1 + ((z * (int64_t)S.nq + row) * S.h + qh) * S.d;
            put_row<DP>(p, tx, S.d, acc1[i], S.scale);
        }
    }
}

template <typename F>
int by_width(int d, F&& f) {
    if (d <= 32) return f(std::integral_constant<int, 32>());
    if (d <= 64) return f(std::integral_constant<int, 64>());
    return f(std::integral_constant<int, 128>());
}

bool vec16(const View& v) { return aligned16(v.p) && v.row % 4 == 0 && v.head % 4 == 0; }

}  // namespace

int fwd_f32(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s) {
    return by_width(S.d, [&](auto width) {
        constexpr int DP = decltype(width)::value;
        constexpr size_t smem = sizeof(float) * (3 * kRows * ldt<DP>() + kRows * kLdw);
        static std::atomic<uint64_t> allowed;
        auto kern = cross_fwd_f32<DP>;
        if (!allow_smem(allowed, (const void*)kern, smem)) return (int)GT_ERR_CUDA;
        LaunchScope ls("cross_fwd_f32", s);
        kern<<<dim3(slots_of(S, true, tile_queries(kRows, S.g)), S.hk, out.splits), kThreads, smem, s>>>(
            S, q, k, v, out, Vec{vec16(q), vec16(k), vec16(v), false});
        return check_launch();
    });
}

template <bool KEYS>
static int bwd_f32(const Shape& S, const BwdIn& in, const Out& g1, const Out& g2, float* p1, float* p2, int splits,
                   cudaStream_t s) {
    return by_width(S.d, [&](auto width) {
        constexpr int DP = decltype(width)::value;
        constexpr size_t smem = sizeof(float) * (4 * kRows * ldt<DP>() + 2 * kRows * kLdw);
        static std::atomic<uint64_t> allowed;
        auto kern = cross_bwd_f32<DP, KEYS>;
        if (!allow_smem(allowed, (const void*)kern, smem)) return (int)GT_ERR_CUDA;
        LaunchScope ls(KEYS ? "cross_dkv_f32" : "cross_dq_f32", s);
        const Vec vec{vec16(in.q), vec16(in.k), vec16(in.v), vec16(in.dO)};
        if (launch_overlapped(kern, dim3(slots_of(S, !KEYS, KEYS ? kRows : tile_queries(kRows, S.g)), S.hk, splits), dim3(kThreads),
                              smem, s, S, in, g1, g2, p1, p2, splits, vec) != cudaSuccess)
            return (int)GT_ERR_CUDA;
        return check_launch();
    });
}

int bwd_dq_f32(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s) {
    return bwd_f32<false>(S, in, dq, Out{}, part, nullptr, splits, s);
}

int bwd_dkv_f32(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
                cudaStream_t s) {
    return bwd_f32<true>(S, in, dk, dv, dk_part, dv_part, splits, s);
}

}  // namespace cross
}  // namespace gt
