// gt_cross_attn.cu -- entry points of cross attention: checks, workspace, how a call is split over the SMs, and the small
// kernels around the products.
//
//   cross_stats   -lse log2 e and -D, D = <dO, o>, of every query and head, in the order of the tiles' rows
//   cross_join    o and lse from the parts of a split forward, exactly: weights exp(lse_part - lse)
//   cross_sum     the sum of a split backward's parts, in their order
//   cross_pack    rows that TMA cannot read (a base or stride that is no multiple of 16 bytes, or a stride of 0) as padded
//                 rows in the workspace
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "gt_cross.cuh"
#include "gt_stats.cuh"

namespace gt {
namespace cross {
namespace {

constexpr int kThreads = 256;

// Eight lanes to a query and head.
template <typename T>
__global__ void __launch_bounds__(kThreads) cross_stats(const Shape S, const View o, const View dO, const float* __restrict__ lse,
                                                        float2* __restrict__ stats, int vec) {
    sm100::pdl_trigger();
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3);
    const int part = threadIdx.x & 7;
    const bool live = item < (int64_t)S.nq * S.h;
    float sum = 0.f;
    int64_t query = 0;
    int head = 0;
    if (live) {
        query = item / S.h;
        head = (int)(item - query * S.h);
        const T* a = static_cast<const T*>(o.p) + query * o.row + head * o.head;
        const T* b = static_cast<const T*>(dO.p) + query * dO.row + head * dO.head;
        for (int c = part * 8; c < S.d; c += 64) {
            float x[8], y[8];
            unpack8(load8(a + c, S.d - c, vec), x);
            unpack8(load8(b + c, S.d - c, vec), y);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x[i], y[i], sum);
        }
    }
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (live && part == 0) {
        const float l = __ldg(lse + (int64_t)head * S.nq + query);
        // a query without a key: every p and dS is 0, o (and D) of no matter
        const bool none = l == -INFINITY;
        stats[((int64_t)(head / S.g) * S.nq + query) * S.g + head % S.g] =
            make_float2(none ? -INFINITY : -l * tc::kLog2e, none ? 0.f : -sum);
    }
}

// The rows of the sequences: [first, end)
__device__ __forceinline__ bool in_batch(const int32_t* off, int batch, int n, int64_t row) {
    return !off || (row >= clamp_off(off, 0, n) && row < clamp_off(off, batch, n));
}

// LANES lanes to a query and head, one to eight channels: lane p weighs the parts p, p + LANES, ...  The first parts' sums are on
// their way while the weights are formed.
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) cross_join(const Shape S, const FwdOut out) {
    const int64_t item = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int part = threadIdx.x % LANES;
    const bool there = item < (int64_t)S.nq * S.h;
    const int64_t query = there ? item / S.h : 0;
    const int head = there ? (int)(item - query * S.h) : 0;
    const bool live = there && in_batch(S.q_off, S.batch, S.nq, query);
    sm100::pdl_wait();   // launched to overlap the end of the kernel that writes the parts
    constexpr int W = kMaxSplits / LANES;
    const int vec = S.d % 4 == 0 ? 1 : 0;
    const int64_t step = (int64_t)S.nq * S.h * S.d;
    auto load = [&](Raw8<float>(&raw)[4], int c, int z) {      // parts z .. z + 3, from channel c
        const bool mine = live && c < S.d;
        const float* src = out.o_part + (mine ? (query * S.h + head) * S.d + c : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = load8<Mem::kOutput>(src + (z + i < out.splits ? z + i : 0) * step, mine ? S.d - c : 0, vec);
    };
    Raw8<float> raw[4];
    load(raw, part * 8, 0);
    float l[W], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const int z = part + k * LANES;
        l[k] = live && z < out.splits ? __ldcg(out.lse_part + ((int64_t)z * S.h + head) * S.nq + query) : -INFINITY;
        top = fmaxf(top, l[k]);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int k = 0; k < W; ++k) {
        l[k] = l[k] == -INFINITY ? 0.f : expf(l[k] - top);      // (a NaN is not lost)
        sum += l[k];
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool seen = sum != 0.f;
    if (live && part == 0) out.lse[(int64_t)head * S.nq + query] = seen ? top + logf(sum) : -INFINITY;
    const float inv = seen ? 1.f / sum : 0.f;
    T* o = static_cast<T*>(out.o.p) + query * out.o.row + head * out.o.head;
    for (int c0 = 0; c0 < S.d; c0 += 8 * LANES) {
        const int c = c0 + part * 8;
        float acc[8] = {};
#pragma unroll
        for (int k = 0; k < W; ++k)
            for (int u = 0; u < LANES && k * LANES + u < out.splits; u += 4) {      // four loads at a time
                if (c0 + k * LANES + u > 0) load(raw, c, k * LANES + u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float weight = __shfl_sync(0xffffffffu, l[k], u + i, LANES) * inv;
                    float x[8];
                    unpack8(raw[i], x);
                    if (weight != 0.f)      // (nothing was written for a part without a key)
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[j] = fmaf(weight, x[j], acc[j]);
                }
            }
        if (live && c < S.d) store8(o + c, acc, S.d - c, out.o.acc);
    }
}

// One result of a split backward: [parts][rows][heads][d] summed into out; two at once (dk and dv) by blockIdx.y.  LANES
// lanes share the parts of an eight of channels, z = lane, lane + LANES, ..., and join in a fixed order.
struct SumJob {
    const float* part;
    Out out;
};
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) cross_sum(const SumJob j0, const SumJob j1, const int32_t* off, int batch, int rows,
                                                      int heads, int d, int parts) {
    const SumJob& J = blockIdx.y == 0 ? j0 : j1;
    const int pieces = (d + 7) / 8, lane = threadIdx.x % LANES;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES, item = at / pieces;
    const int c = (int)(at - item * pieces) * 8;
    const int64_t row = item / heads;
    const int head = (int)(item - row * heads);
    const bool live = row < rows && in_batch(off, batch, rows, row);
    sm100::pdl_wait();   // launched to overlap the end of the kernel that writes the parts
    float acc[8] = {};
    const float* p = J.part + (live ? item * d + c : 0);
    const int64_t step = (int64_t)rows * heads * d;
    constexpr int U = LANES == 1 ? 8 : 4;      // loads on their way, those past the last part left out
    for (int z = lane; z < parts; z += U * LANES) {
        Raw8<float> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = load8<Mem::kOutput>(p + (z + u * LANES) * step, live && z + u * LANES < parts ? d - c : 0, d % 4 == 0 ? 1 : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[8];
            unpack8(raw[u], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += x[i];
        }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (live && lane == 0)
        store8(static_cast<T*>(J.out.p) + row * J.out.row + head * J.out.head + c, acc, d - c, J.out.acc);
}

// dst: [rows][heads][dp], zeros past d
struct PackJob {
    View src;
    bf16* dst;
    int rows, heads;
};
struct PackJobs {
    PackJob j[4];
    int d, dp;
};
__global__ void __launch_bounds__(kThreads) cross_pack(const PackJobs P) {
    sm100::pdl_trigger();
    const PackJob& J = P.j[blockIdx.y];
    const int pieces = P.dp / 8;
    const int64_t all = (int64_t)J.rows * J.heads * pieces;
    for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < all; at += (int64_t)gridDim.x * kThreads) {
        const int64_t item = at / pieces, row = item / J.heads;
        const int c = (int)(at - item * pieces) * 8, head = (int)(item - row * J.heads);
        const unsigned short* s = static_cast<const unsigned short*>(J.src.p) + row * J.src.row + head * J.src.head + c;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = c + i < P.d ? (uint32_t)__ldg(s + i) : 0u;
        *reinterpret_cast<uint4*>(J.dst + at * 8) =
            make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
    }
}

// ------------------------------------------------------------------------------------------- plans

int width_of(int d) { return (d + 7) / 8 * 8; }

// Whether TMA reads the rows as they are.
bool tma_rows(const View& v) {
    return aligned16(v.p) && v.row % 8 == 0 && v.head % 8 == 0 && v.row > 0 && v.head > 0 &&
           v.row < ((int64_t)1 << 38) && v.head < ((int64_t)1 << 38);
}

int64_t tiles_of(int n, int batch, int rows) { return std::max<int64_t>(batch, ((int64_t)n + rows - 1) / rows); }

// What a pass costs: microseconds of a step of a CTA with the SM's other CTAs beside it (measured for bf16; round estimates
// for fp32), CTAs on an SM, and bytes that each part writes and reads again.
struct Cost {
    double step;
    int per_sm;
    double bytes;
};

// Parts into which the streamed side is cut.  One sequence: `ctas` tiles of `steps` steps each run in whole waves; several: as many
// of unlike length, so the longest (taken as twice the mean) ends last.  Every CTA starts and ends in about two steps' time;
// parts are joined by another launch, and their sums go through L2 at about 5 TB/s.
int parts_for(int64_t ctas, int64_t steps, int batch, const Cost& c) {
    const int64_t slots = (int64_t)c.per_sm * num_sms();
    double best = 0.0;
    int64_t parts = 1;
    for (int64_t p = 1; p <= std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, steps / 2)); ++p) {
        const double each = (double)((steps + p - 1) / p) + 2.0;
        const double turns = batch == 1 ? (double)((ctas * p + slots - 1) / slots)
                                        : std::max(1.0, (double)(ctas * p) / (double)slots) + 1.0;
        const double us = turns * each * c.step + (p > 1 ? 5.0 + (double)p * c.bytes / 5e6 : 0.0);
        if (p == 1 || us < best) {
            best = us;
            parts = p;
        }
    }
    return (int)parts;
}

struct Plan {
    int fwd, dq, dkv;      // parts
};

Plan plan_of(const Shape& S, bool f32) {
    Plan p;
    const double q_bytes = 8.0 * S.nq * S.h * S.d, k_bytes = 16.0 * S.nk * S.hk * S.d;
    const double wide = S.d <= 64 ? 1.0 : 1.6;
    const int few = few_rows(S);
    if (few) {
        // eight CTAs to an SM (more where the sequences are unlike), four turns of a CTA's warps at least to each
        const int64_t tiles = tiles_of(S.nq, S.batch, few / S.g) * S.hk;
        const int64_t want = (int64_t)(S.batch > 1 ? 16 : 8) * num_sms() / std::max<int64_t>(1, tiles);
        int64_t lanes = 1;
        while (lanes * 8 < S.d) lanes *= 2;
        p.fwd = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxSplits), S.nk / S.batch * lanes / 2048));
    }
    if (f32) {
        const int tq = tile_queries(64, S.g);
        const int64_t qt = tiles_of(S.nq, S.batch, tq) * S.hk, kt = tiles_of(S.nk, S.batch, 64) * S.hk;
        const int64_t keys = (S.nk / S.batch + 63) / 64, queries = (S.nq / S.batch + tq - 1) / tq;
        if (S.d <= kNarrow) {
            const int64_t k128 = (S.nk / S.batch + 127) / 128, tq128 = tile_queries(128, S.g);
            const double step = S.d <= 8 ? 1.0 : 2.0;
            if (!few) p.fwd = parts_for(qt, k128, S.batch, Cost{step, 4, q_bytes});
            p.dq = parts_for(qt, k128, S.batch, Cost{1.5 * step, 4, q_bytes});
            p.dkv = parts_for(kt, (S.nq / S.batch + tq128 - 1) / tq128, S.batch, Cost{2.0 * step, 3, k_bytes});
            return p;
        }
        if (!few) p.fwd = parts_for(qt, keys, S.batch, Cost{2.0 * wide, 2, q_bytes});
        p.dq = parts_for(qt, keys, S.batch, Cost{3.0 * wide, 2, q_bytes});
        p.dkv = parts_for(kt, queries, S.batch, Cost{4.0 * wide, 2, k_bytes});
    } else {
        const int keys = S.d <= 64 ? 96 : 64, tq = tile_queries(64, S.g);
        const int64_t qt = tiles_of(S.nq, S.batch, tile_queries(128, S.g)) * S.hk, kt = tiles_of(S.nk, S.batch, 128) * S.hk;
        if (!few) p.fwd = parts_for(qt, (S.nk / S.batch + keys - 1) / keys, S.batch,
                                     few_tile(S) ? Cost{0.7, 2, q_bytes} : Cost{S.d <= 64 ? 0.8 : 1.2, 2, q_bytes});
        p.dq = parts_for(qt, (S.nk / S.batch + 63) / 64, S.batch, Cost{S.d <= 64 ? 0.72 : 1.5, 2, q_bytes});
        p.dkv = parts_for(kt, (S.nq / S.batch + tq - 1) / tq, S.batch, S.d <= 64 ? Cost{1.15, 2, k_bytes} : Cost{1.0, 1, k_bytes});
    }
    return p;
}

struct Room {
    float *o_part, *lse_part, *dq_part, *dk_part, *dv_part;
    float2* stats;
    bf16 *q, *k, *v, *dO;
};

// The workspace of a call; pack[]: which of q, k, v, dO are copied
Room carve(Carve& cv, const Shape& S, const Plan& p, bool bwd, const bool (&pack)[4]) {
    Room r = {};
    const size_t nqh = (size_t)S.nq * S.h, nkh = (size_t)S.nk * S.hk, d = S.d, dp = width_of(S.d);
    if (!bwd && p.fwd > 1) {
        r.o_part = cv.take<float>(p.fwd * nqh * d);
        r.lse_part = cv.take<float>(p.fwd * nqh);
    }
    if (bwd) {
        r.stats = cv.take<float2>(nqh);
        if (p.dq > 1) r.dq_part = cv.take<float>(p.dq * nqh * d);
        if (p.dkv > 1) {
            r.dk_part = cv.take<float>(p.dkv * nkh * d);
            r.dv_part = cv.take<float>(p.dkv * nkh * d);
        }
    }
    if (pack[0]) r.q = cv.take<bf16>(nqh * dp);
    if (pack[1]) r.k = cv.take<bf16>(nkh * dp);
    if (pack[2]) r.v = cv.take<bf16>(nkh * dp);
    if (pack[3]) r.dO = cv.take<bf16>(nqh * dp);
    return r;
}

bool valid_type(int t) { return t == GT_F32 || t == GT_BF16; }

int check_sizes(int dtype, int nq, int nk, int h, int hk, int d, int batch) {
    if (!valid_type(dtype) || nq < 1 || nk < 1 || h < 1 || hk < 1 || d < 1 || batch < 1 || h % hk) return GT_ERR_INVALID_ARG;
    if (d > kMaxD || h > kMaxHeads || h / hk > kMaxShare || batch > (1 << 20) || nq > (1 << 30) || nk > (1 << 30))
        return GT_ERR_UNSUPPORTED;
    return GT_OK;
}

Shape shape_of(int nq, int nk, int h, int hk, int d, int batch, const int32_t* q_off, const int32_t* kv_off,
               const uint8_t* mask, float scale) {
    return Shape{nq, nk, h, hk, h / hk, d, batch, q_off, kv_off, mask, scale};
}

int check_shape(const Shape& S) {
    if ((S.q_off != nullptr) != (S.kv_off != nullptr) || (!S.q_off && S.batch != 1)) return GT_ERR_INVALID_ARG;
    // (the exponents are formed with scale log2 e)
    return S.scale > 0.f && isfinite(S.scale * tc::kLog2e) ? GT_OK : GT_ERR_INVALID_ARG;
}

bool usable(const View& v) { return v.p && v.row >= 0 && v.head >= 0; }

Out out_of(void* p, int64_t row, int64_t head, int bytes) {
    return Out{p, row, head, rows16(p, row, bytes) && rows16(p, head, bytes) ? 1 : 0};
}

// Copies the inputs that need it and points their views at the copies.
int pack_inputs(const Shape& S, View* (&views)[4], bf16* (&room)[4], cudaStream_t s) {
    PackJobs P = {};
    P.d = S.d;
    P.dp = width_of(S.d);
    int count = 0;
    int64_t most = 0;
    for (int i = 0; i < 4; ++i) {
        if (!room[i]) continue;
        const bool query = i == 0 || i == 3;
        const int rows = query ? S.nq : S.nk, heads = query ? S.h : S.hk;
        P.j[count++] = PackJob{*views[i], room[i], rows, heads};
        most = std::max<int64_t>(most, (int64_t)rows * heads * (P.dp / 8));
        *views[i] = View{room[i], (int64_t)heads * P.dp, P.dp};
    }
    if (!count) return GT_OK;
    LaunchScope ls("cross_pack", s);
    const int64_t ctas = std::min<int64_t>((most + kThreads - 1) / kThreads, 16 * (int64_t)num_sms());
    cross_pack<<<dim3((unsigned)ctas, count), kThreads, 0, s>>>(P);
    return check_launch();
}

template <typename T>
int sum_parts(const SumJob& a, const SumJob& b, int jobs, const int32_t* off, int batch, int rows, int heads, int d, int parts,
              cudaStream_t s) {
    LaunchScope ls("cross_sum", s);
    // eight lanes to an eight where there are too few of them to fill the SMs (128 x 8 heads of 8 in 27 parts: 13 us with one
    // lane, 6 with eight; 4096 x 8 heads of 64 in 7 parts: 19 us with one, 25 with two)
    const int64_t eights = (int64_t)rows * heads * ((d + 7) / 8);
    const int lanes = eights < (int64_t)4 * num_sms() * kThreads ? 8 : 1;
    if (launch_overlapped(lanes == 8 ? cross_sum<T, 8> : cross_sum<T, 1>,
                          dim3((unsigned)((eights * lanes + kThreads - 1) / kThreads), jobs),
                          dim3(kThreads), 0, s, a, b, off, batch, rows, heads, d, parts) != cudaSuccess)
        return GT_ERR_CUDA;
    return check_launch();
}

template <typename T>
int run_bwd(Shape S, const Plan& plan, const Room& r, BwdIn in, const View& o, const float* lse, const Out& dq, const Out& dk,
            const Out& dv, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    {
        LaunchScope ls("cross_stats", s);
        const int64_t items = (int64_t)S.nq * S.h;
        const int vec = rows16(o.p, o.row, sizeof(T)) && rows16(o.p, o.head, sizeof(T)) && rows16(in.dO.p, in.dO.row, sizeof(T)) &&
                        rows16(in.dO.p, in.dO.head, sizeof(T));
        cross_stats<T><<<(unsigned)((items + kThreads / 8 - 1) / (kThreads / 8)), kThreads, 0, s>>>(S, o, in.dO, lse, r.stats, vec);
        const int rc = check_launch();
        if (rc != GT_OK) return rc;
    }
    in.stats = r.stats;
    int rc;
    if constexpr (!F32) {
        View* views[4] = {&in.q, &in.k, &in.v, &in.dO};
        bf16* room[4] = {r.q, r.k, r.v, r.dO};
        rc = pack_inputs(S, views, room, s);
        if (rc != GT_OK) return rc;
    }
    const bool narrow = F32 && S.d <= kNarrow;
    rc = narrow ? bwd_dq_narrow(S, in, dq, r.dq_part, plan.dq, s)
         : F32  ? bwd_dq_f32(S, in, dq, r.dq_part, plan.dq, s)
                : bwd_dq_tc(S, in, dq, r.dq_part, plan.dq, s);
    if (rc != GT_OK) return rc;
    rc = narrow ? bwd_dkv_narrow(S, in, dk, dv, r.dk_part, r.dv_part, plan.dkv, s)
         : F32  ? bwd_dkv_f32(S, in, dk, dv, r.dk_part, r.dv_part, plan.dkv, s)
                : bwd_dkv_tc(S, in, dk, dv, r.dk_part, r.dv_part, plan.dkv, s);
    if (rc != GT_OK) return rc;
    if (plan.dq > 1) {
        const SumJob j{r.dq_part, dq};
        rc = sum_parts<T>(j, j, 1, S.q_off, S.batch, S.nq, S.h, S.d, plan.dq, s);
        if (rc != GT_OK) return rc;
    }
    if (plan.dkv > 1)
        rc = sum_parts<T>(SumJob{r.dk_part, dk}, SumJob{r.dv_part, dv}, 2, S.kv_off, S.batch, S.nk, S.hk, S.d, plan.dkv, s);
    return rc;
}

}  // namespace
}  // namespace cross
}  // namespace gt

extern "C" {

size_t gt_cross_attn_workspace_size(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d, int32_t batch,
                                    int32_t backward, int32_t aligned) {
    using namespace gt::cross;
    if (check_sizes(dtype, nq, nk, h, hk, d, batch) != GT_OK) return 0;
    const Shape S = shape_of(nq, nk, h, hk, d, batch, nullptr, nullptr, nullptr, 1.f);
    const bool copies = dtype == GT_BF16 && !aligned && (backward || !few_rows(S));
    gt::Carve cv(nullptr, 0);
    const bool pack[4] = {copies, copies, copies, copies && backward};
    carve(cv, S, plan_of(S, dtype == GT_F32), backward != 0, pack);
    return cv.off == 0 ? 0 : cv.off + 256;
}

int gt_cross_attn_fwd(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d, int32_t batch, const void* q,
                      int64_t ldq, int64_t hdq, const void* k, int64_t ldk, int64_t hdk, const void* v, int64_t ldv,
                      int64_t hdv, const int32_t* q_off, const int32_t* kv_off, const uint8_t* key_mask, float scale, void* o,
                      int64_t ldo, int64_t hdo, float* lse, void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt::cross;
    int rc = check_sizes(dtype, nq, nk, h, hk, d, batch);
    if (rc != GT_OK) return rc;
    const Shape S = shape_of(nq, nk, h, hk, d, batch, q_off, kv_off, key_mask, scale);
    rc = check_shape(S);
    if (rc != GT_OK) return rc;
    View qv{q, ldq, hdq}, kv{k, ldk, hdk}, vv{v, ldv, hdv};
    if (!usable(qv) || !usable(kv) || !usable(vv) || !o || !lse || ldo < 0 || hdo < 0) return GT_ERR_INVALID_ARG;
    const bool f32 = dtype == GT_F32;
    const Plan plan = plan_of(S, f32);
    const bool few = few_rows(S) > 0, tma = !f32 && !few;
    const bool pack[4] = {tma && !tma_rows(qv), tma && !tma_rows(kv), tma && !tma_rows(vv), false};
    gt::Carve cv(workspace, ws_bytes);
    const Room r = carve(cv, S, plan, false, pack);
    if (cv.off > 0 && (!workspace || !gt::aligned16(workspace) || !cv.fits())) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const FwdOut out{out_of(o, ldo, hdo, f32 ? 4 : 2), lse, r.o_part, r.lse_part, plan.fwd};
    if (few) {
        rc = fwd_few(S, f32, qv, kv, vv, out, s);
    } else if (f32) {
        rc = d <= kNarrow ? fwd_narrow(S, qv, kv, vv, out, s) : fwd_f32(S, qv, kv, vv, out, s);
    } else {
        View* views[4] = {&qv, &kv, &vv, nullptr};
        bf16* room[4] = {r.q, r.k, r.v, nullptr};
        rc = pack_inputs(S, views, room, s);
        if (rc == GT_OK) rc = fwd_tc(S, qv, kv, vv, out, s);
    }
    if (rc != GT_OK || plan.fwd == 1) return rc;
    gt::LaunchScope ls("cross_join", s);
    const int64_t items = (int64_t)nq * h;
    const int lanes = d <= 64 ? 8 : 16;
    const unsigned ctas = (unsigned)((items * lanes + kThreads - 1) / kThreads);
    auto join = lanes == 8 ? (f32 ? cross_join<float, 8> : cross_join<bf16, 8>) : (f32 ? cross_join<float, 16> : cross_join<bf16, 16>);
    const cudaError_t e = gt::launch_overlapped(join, dim3(ctas), dim3(kThreads), 0, s, S, out);
    return e == cudaSuccess ? gt::check_launch() : GT_ERR_CUDA;
}

int gt_cross_attn_bwd(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d, int32_t batch, const void* q,
                      int64_t ldq, int64_t hdq, const void* k, int64_t ldk, int64_t hdk, const void* v, int64_t ldv,
                      int64_t hdv, const void* o, int64_t ldo, int64_t hdo, const void* dO, int64_t lddo, int64_t hddo,
                      const float* lse, const int32_t* q_off, const int32_t* kv_off, const uint8_t* key_mask, float scale,
                      void* dq, int64_t lddq, int64_t hddq, void* dk, int64_t lddk, int64_t hddk, void* dv, int64_t lddv,
                      int64_t hddv, void* workspace, size_t ws_bytes, void* stream) {
    using namespace gt::cross;
    int rc = check_sizes(dtype, nq, nk, h, hk, d, batch);
    if (rc != GT_OK) return rc;
    const Shape S = shape_of(nq, nk, h, hk, d, batch, q_off, kv_off, key_mask, scale);
    rc = check_shape(S);
    if (rc != GT_OK) return rc;
    const View ov{o, ldo, hdo};
    BwdIn in{View{q, ldq, hdq}, View{k, ldk, hdk}, View{v, ldv, hdv}, View{dO, lddo, hddo}, nullptr};
    if (!usable(in.q) || !usable(in.k) || !usable(in.v) || !usable(in.dO) || !usable(ov) || !lse || !dq || !dk || !dv ||
        lddq < 0 || hddq < 0 || lddk < 0 || hddk < 0 || lddv < 0 || hddv < 0)
        return GT_ERR_INVALID_ARG;
    const bool f32 = dtype == GT_F32;
    const int e = f32 ? 4 : 2;
    const Plan plan = plan_of(S, f32);
    const bool pack[4] = {!f32 && !tma_rows(in.q), !f32 && !tma_rows(in.k), !f32 && !tma_rows(in.v),
                          !f32 && !tma_rows(in.dO)};
    gt::Carve cv(workspace, ws_bytes);
    const Room r = carve(cv, S, plan, true, pack);
    if (!workspace || !gt::aligned16(workspace) || !cv.fits()) return GT_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Out oq = out_of(dq, lddq, hddq, e), ok = out_of(dk, lddk, hddk, e), okv = out_of(dv, lddv, hddv, e);
    return f32 ? run_bwd<float>(S, plan, r, in, ov, lse, oq, ok, okv, s) : run_bwd<bf16>(S, plan, r, in, ov, lse, oq, ok, okv, s);
}

}  // extern "C"
