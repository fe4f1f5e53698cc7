// gt_cross_few.cu -- cross attention forward for few rows: one query (a few heads that share its keys) to a sequence, as a
// readout or the next token of a decoder has it.
//
// The bytes of the keys and values bound it.  A key's channels are dealt to a few lanes, eight each, so that a warp reads
// whole rows, several at a time; every lane has its channels of all rows' queries and of their outputs in registers.
// Scores are sums over the lanes of a key; each group of lanes, and each warp, keeps a maximum, a sum and outputs of its
// own for its share of the keys, joined at the end.  Nothing waits for anything but its own loads.
//
// At most two rows (kFewRows): every key costs R dot products and R updates on the fp32 pipes, and from four rows on the
// tensor cores are quicker (bf16, 16 queries over 65536 keys, 4 heads sharing keys of 128: 111 us here, 64 there).  That is
// bf16's limit; fp32 has it too, unmeasured, though its kernels for more rows take tiles of 64.  One query over 512 nodes, 8
// heads of 8, fp32: 6 us, against 19 with the tiles for many rows.
#include <cuda_bf16.h>
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

constexpr int kThreads = 128, kWarps = kThreads / 32;

// R rows (query, head) to a CTA, LD lanes to a key
template <typename T, int R, int LD>
__global__ void __launch_bounds__(kThreads) cross_few(const Shape S, const View q, const View k, const View v, const FwdOut out,
                                                      const int rows, const int vec) {
    constexpr int KEYS = 32 / LD, U = 4;      // keys to a warp's load, loads on their way
    const int tq = rows / S.g, head = blockIdx.y, z = blockIdx.z;
    sm100::pdl_trigger();
    const Tile t = find_tile(S, true, tq, blockIdx.x);
    if (!t.live) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / LD, c0 = (lane % LD) * 8;
    const int first = t.tile * tq, live = min(tq, t.lq - first) * S.g;
    const int left = S.d - c0;                 // channels of this lane: 0 or less, 1 .. 8
    const float c = S.scale * tc::kLog2e;
    float2 qr[R][4], o[R][4];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int query = min(t.q0 + first + r / S.g, S.nq - 1), qh = head * S.g + r % S.g;
        const T* p = static_cast<const T*>(q.p) + (int64_t)query * q.row + (int64_t)qh * q.head + c0;
        unpack8(load8(p, r < live ? left : 0, vec), qr[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            qr[r][i].x *= c;
            qr[r][i].y *= c;
            o[r][i] = make_float2(0.f, 0.f);
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const T* kp = static_cast<const T*>(k.p) + (int64_t)t.k0 * k.row + (int64_t)head * k.head + c0;
    const T* vp = static_cast<const T*>(v.p) + (int64_t)t.k0 * v.row + (int64_t)head * v.head + c0;
    const int k1 = part_begin(t.lk, z + 1, out.splits);
    for (int k0 = part_begin(t.lk, z, out.splits) + warp * KEYS * U; k0 < k1; k0 += kWarps * KEYS * U) {
        Raw8<T> kr[U], vr[U];
        bool seen[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * KEYS + group;
            seen[u] = key < k1 && (!S.mask || __ldg(S.mask + t.k0 + key) != 0);
            kr[u] = load8(kp + (int64_t)key * k.row, seen[u] ? left : 0, vec);
            vr[u] = load8(vp + (int64_t)key * v.row, seen[u] ? left : 0, vec);
        }
        float s[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 x[4];
            unpack8(kr[u], x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 a = __fmul2_rn(x[0], qr[r][0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) a = __ffma2_rn(x[i], qr[r][i], a);
                s[u][r] = a.x + a.y;
            }
        }
#pragma unroll
        for (int w = LD / 2; w > 0; w >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) s[u][r] += __shfl_xor_sync(0xffffffffu, s[u][r], w);
        float p[U][R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!seen[u]) s[u][r] = -INFINITY;
                top = fmaxf(top, s[u][r]);
            }
            const float base = top == -INFINITY ? 0.f : top, by = sm100::ex2(m[r] - base);
            m[r] = top;
            l[r] *= by;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p[u][r] = sm100::ex2(s[u][r] - base);
                l[r] += p[u][r];
            }
            const float2 by2 = make_float2(by, by);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][i] = __fmul2_rn(o[r][i], by2);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 x[4];
            unpack8(vr[u], x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 w = make_float2(p[u][r], p[u][r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][i] = __ffma2_rn(w, x[i], o[r][i]);
            }
        }
    }
    // the warp's groups, then the warps, on one base
    auto join = [](float& ma, float& la, float2 (&oa)[4], float mb, float lb, const float2 (&ob)[4]) {
        const float top = fmaxf(ma, mb), base = top == -INFINITY ? 0.f : top;
        const float wa = sm100::ex2(ma - base), wb = sm100::ex2(mb - base);
        la = la * wa + lb * wb;
        ma = top;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            oa[i] = make_float2(oa[i].x * wa + ob[i].x * wb, oa[i].y * wa + ob[i].y * wb);
    };
#pragma unroll
    for (int w = LD; w < 32; w <<= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 ob[4];
            const float mb = __shfl_xor_sync(0xffffffffu, m[r], w), lb = __shfl_xor_sync(0xffffffffu, l[r], w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ob[i] = make_float2(__shfl_xor_sync(0xffffffffu, o[r][i].x, w), __shfl_xor_sync(0xffffffffu, o[r][i].y, w));
            join(m[r], l[r], o[r], mb, lb, ob);
        }
    __shared__ float2 so[kWarps][R][LD][4];
    __shared__ float2 sm[kWarps][R];
    if (group == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < 4; ++i) so[warp][r][lane][i] = o[r][i];
            if (lane == 0) sm[warp][r] = make_float2(m[r], l[r]);
        }
    __syncthreads();
    for (int at = threadIdx.x; at < live * LD; at += kThreads) {
        const int r = at / LD, part = at % LD;
        float ma = sm[0][r].x, la = sm[0][r].y;
        float2 oa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) oa[i] = so[0][r][part][i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) join(ma, la, oa, sm[w][r].x, sm[w][r].y, so[w][r][part]);
        const int64_t query = t.q0 + first + r / S.g;
        const int qh = head * S.g + r % S.g, col = part * 8;
        const bool some = la != 0.f;      // (a NaN counts)
        const float inv = some ? 1.f / la : 0.f, lse = some ? (ma + log2f(la)) * tc::kLn2 : -INFINITY;
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = oa[i].x * inv;
            x[2 * i + 1] = oa[i].y * inv;
        }
        if (out.splits == 1) {
            if (part == 0) out.lse[(int64_t)qh * S.nq + query] = lse;
            if (col < S.d)
                store8(static_cast<T*>(out.o.p) + query * out.o.row + qh * out.o.head + col, x, S.d - col, out.o.acc);
        } else {
            if (part == 0) out.lse_part[(z * (int64_t)S.h + qh) * S.nq + query] = lse;
            if (col < S.d)
                store8(out.o_part + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d + col, x, S.d - col, S.d % 4 == 0 ? 1 : 0);
        }
    }
}

template <typename T, int R, int LD>
int launch(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, int rows, cudaStream_t s) {
    int vec = 1;
    for (const View* p : {&q, &k, &v}) vec = std::min<int>(vec, rows16(p->p, p->row, sizeof(T)) && rows16(p->p, p->head, sizeof(T)));
    LaunchScope ls("cross_few", s);
    cross_few<T, R, LD><<<dim3(slots_of(S, true, rows / S.g), S.hk, out.splits), kThreads, 0, s>>>(S, q, k, v, out, rows, vec);
    return check_launch();
}

template <typename T, int R>
int by_width(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, int rows, cudaStream_t s) {
    if (S.d <= 8) return launch<T, R, 1>(S, q, k, v, out, rows, s);
    if (S.d <= 16) return launch<T, R, 2>(S, q, k, v, out, rows, s);
    if (S.d <= 32) return launch<T, R, 4>(S, q, k, v, out, rows, s);
    if (S.d <= 64) return launch<T, R, 8>(S, q, k, v, out, rows, s);
    return launch<T, R, 16>(S, q, k, v, out, rows, s);
}

template <typename T>
int by_rows(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, int rows, cudaStream_t s) {
    static_assert(kFewRows == 2, "a tile has one row or two");
    return rows <= 1 ? by_width<T, 1>(S, q, k, v, out, rows, s) : by_width<T, 2>(S, q, k, v, out, rows, s);
}

}  // namespace

int few_rows(const Shape& S) {
    // the rows of a sequence of mean length, whole queries
    const int64_t mean = ((int64_t)S.nq + S.batch - 1) / S.batch;
    return mean * S.g <= kFewRows ? (int)mean * S.g : 0;
}

int fwd_few(const Shape& S, bool f32, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s) {
    return f32 ? by_rows<float>(S, q, k, v, out, few_rows(S), s) : by_rows<bf16>(S, q, k, v, out, few_rows(S), s);
}

}  // namespace cross
}  // namespace gt
