// gt_cross.cuh -- what the cross-attention kernels share: the shape of a call, where the tiles of a
// packed batch lie, and a few device helpers.
//
//   s = scale q k^T over the keys of the query's own sequence that are not hidden,
//   o = softmax(s) v,  lse = log sum exp s;  a query that sees no key: o = 0, lse = -infinity
//   backward with p = exp(s - lse), D = <dO, o>:  dS = p (dO v^T - D),
//   dq = scale dS k,  dk = scale dS^T q,  dv = p^T dO  (dk, dv: over all queries and heads that share the key head)
//
// A tile's rows are pairs (query, head) of the g = h / hk heads that share a key head, the heads of a query one after
// another: shared heads read a key tile once, and one query still makes g rows.
//
// Sequences come as device offsets, so the host does not know their lengths.  A tile of T rows of sequence b is slot
// offset[b] / T + b + tile: ceil(length / T) <= offset[b + 1] / T - offset[b] / T + 1, so the slots of a sequence end
// before the next one's begin, n / T + batch slots hold every tile whatever the lengths, and a CTA finds its tile by a
// search over the offsets.  Slots without a tile return at once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gt_common.cuh"
#include "gt_sm100.cuh"
#include "gt_tc_common.cuh"
#include "gt_vec8.cuh"

namespace gt {
namespace cross {

using bf16 = __nv_bfloat16;

constexpr int kMaxD = 128;
constexpr int kMaxShare = 64;     // query heads to a key head
constexpr int kMaxHeads = 1024;
constexpr int kMaxSplits = 64;
constexpr int kNarrow = 16;       // head dims of fp32 storage with kernels of their own
constexpr int kFewRows = 2;       // rows (query, head) of a sequence up to which the forward runs on the CUDA cores

// [rows][heads][d], channels contiguous
struct View {
    const void* p;
    int64_t row, head;
};
struct Out {
    void* p;
    int64_t row, head;
    int acc;      // row_access() of its rows
};

struct Shape {
    int nq, nk, h, hk, g, d, batch;
    const int32_t* q_off;      // both NULL: one sequence
    const int32_t* kv_off;
    const uint8_t* mask;       // NULL, or a byte to a key: 0 hides it
    float scale;
};

// A sequence's rows and the tile of a slot in it.
struct Tile {
    int q0, lq, k0, lk, tile;
    bool live;
};

__device__ __forceinline__ int clamp_off(const int32_t* off, int b, int n) {
    const int v = __ldg(off + b);
    return v < 0 ? 0 : v > n ? n : v;
}

// rows: of a tile, queries where by_q, else keys
__device__ __forceinline__ Tile find_tile(const Shape& S, bool by_q, int rows, int slot) {
    if (!S.q_off) return Tile{0, S.nq, 0, S.nk, slot, (int64_t)slot * rows < (by_q ? S.nq : S.nk)};
    const int32_t* off = by_q ? S.q_off : S.kv_off;
    const int n = by_q ? S.nq : S.nk, lane = threadIdx.x & 31;
    // the last sequence whose slots begin at or in front of this one, a lane a candidate (whole warps)
    int lo = 0, len = S.batch;
    while (len > 1) {
        const int step = (len + 31) / 32, at = lo + lane * step;
        const bool in = lane * step < len && clamp_off(off, at, n) / rows + at <= slot;
        const int last = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0);
        lo += last * step;
        len = min(step, len - last * step);
    }
    Tile t;
    t.q0 = clamp_off(S.q_off, lo, S.nq);
    t.lq = clamp_off(S.q_off, lo + 1, S.nq) - t.q0;
    t.k0 = clamp_off(S.kv_off, lo, S.nk);
    t.lk = clamp_off(S.kv_off, lo + 1, S.nk) - t.k0;
    t.tile = slot - ((by_q ? t.q0 : t.k0) / rows + lo);
    t.live = t.tile >= 0 && (int64_t)t.tile * rows < (by_q ? t.lq : t.lk);
    if (t.lk < 0) t.lk = 0;      // (offsets that fall: nothing to attend to)
    if (t.lq < 0) t.lq = 0;
    return t;
}

inline int slots_of(const Shape& S, bool by_q, int rows) {
    const int n = by_q ? S.nq : S.nk;
    return S.q_off ? n / rows + S.batch : (n + rows - 1) / rows;
}

// Queries of a tile of `rows` rows.
__host__ __device__ inline int tile_queries(int rows, int g) { return rows / g; }

// Part z of `parts` of n steps
__device__ __forceinline__ int part_begin(int n, int z, int parts) { return (int)((int64_t)n * z / parts); }

// Whether all of the tile's keys are the sequence's (below `end`) and not hidden; if not, bit c of word w says so of key
// first + 32 w + c.  Every lane of a warp.
template <int N>
__device__ __forceinline__ bool valid_keys(const Shape& S, int first, int end, uint32_t (&words)[N]) {
    if (!S.mask && end - first >= 32 * N) return true;      // (the words are not set)
    bool all = true;
#pragma unroll
    for (int w = 0; w < N; ++w) {
        const int left = end - first - 32 * w;
        words[w] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
        if (S.mask) {
            const int key = first + 32 * w + (threadIdx.x & 31);
            words[w] &= __ballot_sync(0xffffffffu, key < end && __ldg(S.mask + key) != 0);
        }
        all = all && words[w] == 0xffffffffu;
    }
    return all;
}

// Zeros in the rows of a [rows][128 bytes] operand panel (PANELS of them, panel_bytes apart) whose bit is not set, by
// one warp, visible to the tensor core.  What stands there belongs to another sequence, or to hidden keys: a weight of
// zero would not cancel an infinity or a NaN.
template <int N, int PANELS>
__device__ __forceinline__ void clear_rows(uint32_t base, uint32_t panel_bytes, const uint32_t (&words)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 0; w < N; ++w) {
        uint32_t bad = ~words[w];
        while (bad) {      // four rows at a time, eight lanes to a row
            uint32_t rest = bad;
            int row = -1;
            for (int k = 0; k <= (lane >> 3) && rest; ++k) {
                row = k == (lane >> 3) ? __ffs(rest) - 1 : -1;
                rest &= rest - 1;
            }
            if (row >= 0)
#pragma unroll
                for (int p = 0; p < PANELS; ++p)
                    sm100::sts_u4(base + p * panel_bytes + (32 * w + row) * 128 + (lane & 7) * 16, 0, 0, 0, 0);
            for (int k = 0; k < 4 && bad; ++k) bad &= bad - 1;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Copies of row 0 in rows first .. rows - 1 of a [rows][128 bytes] panel under the 128-byte swizzle (eights of channels
// change places by the row's last three bits).
template <int PANELS>
__device__ __forceinline__ void repeat_row(uint32_t base, uint32_t panel_bytes, int first, int rows) {
    const int lane = threadIdx.x & 31, piece = lane & 7;
#pragma unroll
    for (int p = 0; p < PANELS; ++p) {
        const uint4 x = sm100::lds_u4(base + p * panel_bytes + piece * 16);
        for (int r = first + (lane >> 3); r < rows; r += 4)
            sm100::sts_u4(base + p * panel_bytes + r * 128 + ((piece ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Zeros in rows first .. rows - 1.
template <int PANELS>
__device__ __forceinline__ void clear_tail(uint32_t base, uint32_t panel_bytes, int first, int rows) {
    const int lane = threadIdx.x & 31;
    for (int r = first + (lane >> 3); r < rows; r += 4)
#pragma unroll
        for (int p = 0; p < PANELS; ++p) sm100::sts_u4(base + p * panel_bytes + r * 128 + (lane & 7) * 16, 0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Columns col .. col + 15 of a row, those below d.
template <typename T>
__device__ __forceinline__ void put16(T* row, int col, int d, const float (&v)[16], int acc) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = v[i];
        b[i] = v[8 + i];
    }
    store8(row + col, a, d - col, acc);
    store8(row + col + 8, b, d - col - 8, acc);
}

// How the kernels of a call follow one another.  Each lets the next be scheduled while it ends.  The dq kernel waits for those
// before it (the statistics, copies of the inputs) before it lets dk and dv start, so that these may read them without a wait
// of their own while dq still runs; they wait at their end instead, so that whoever follows sees dq too.
__device__ __forceinline__ void follow_stats() {
    sm100::pdl_wait();
    sm100::pdl_trigger();
}

// ---- entry points of the kernels' files; every one launches on s and returns a gt_status

struct FwdOut {
    Out o;
    float* lse;         // [h][nq]
    float* o_part;      // [splits][nq][h][d] and lse_part [splits][h][nq] where splits > 1
    float* lse_part;
    int splits;
};

struct BwdIn {
    View q, k, v, dO;
    const float2* stats;     // [hk][nq][g]: -lse log2 e (-infinity for a query without a key) and -D
};

// Whether the tensor-core forward takes tiles of kFewTile rows: a sequence of mean length has no more.
constexpr int kFewTile = 32;
bool few_tile(const Shape& S);
// Rows of a tile of the few-rows forward; 0: the call has too many.
int few_rows(const Shape& S);
int fwd_few(const Shape& S, bool f32, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s);
int fwd_narrow(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s);   // d <= kNarrow
int fwd_f32(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s);
int fwd_tc(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s);
// part: fp32 [splits][nq][h][d] where splits > 1
int bwd_dq_narrow(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s);
int bwd_dq_f32(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s);
int bwd_dq_tc(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s);
// part: fp32 [splits][nk][hk][d] where splits > 1, of dk and of dv
int bwd_dkv_narrow(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
                   cudaStream_t s);
int bwd_dkv_f32(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
                cudaStream_t s);
int bwd_dkv_tc(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
               cudaStream_t s);

}  // namespace cross
}  // namespace gt
