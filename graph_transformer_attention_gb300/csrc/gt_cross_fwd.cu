// gt_cross_fwd.cu -- cross attention forward, bf16, on the tensor cores.
//
//   s = scale q k^T,  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - base),  lse = base + log sum_j p_j
//
// A CTA holds 128 rows (query, head) of one key head and streams its sequence's keys: S = Q K^T into TMEM, an online
// softmax by four warps (a row to a thread), P as bf16 over the scores it was made of, O += P V.  One warp loads by TMA, one
// issues the products.  256 TMEM columns (two tiles' scores and O) and at most 105 KB of shared memory: two CTAs share an SM.
//
// What bounds it is the softmax warps' stream of dependent instructions (half of the issue slots; tensor cores half,
// exponentials half), so nothing else may hold them up: the scores of tile i + 2 go out right behind the product with P
// of tile i, whose columns they take, and a warp finds its next scores there when it comes for them, with one barrier
// each way.  (One tile's scores in TMEM and P beside them, the next scores formed while the softmax worked: the way there
// and back, 1100 cycles under load, showed: 304 us instead of 258 for 4096 x 32768, 8 heads of 64, whatever the products
// cost.)  Two tiles of 96 keys beside 64 columns of O fill 256 columns; above 64 channels tiles of 64.  Other splits took
// longer: four CTAs with tiles of 64 keys 286 us, eight warps with half a tile's keys each 285, one warp each for scores
// and for products with P 281.
//
// The maximum is lazy: a row's base is raised only when a score exceeds it by 2^8, so that O is hardly ever rescaled.
// The weights are formed in packed pairs.  P is rounded to bf16 for the product (half a step, 2^-8 of each weight at most,
// independent from key to key); its sum is not.
//
// 4096 x 32768, 8 heads of 64: 257 us and 19 for joining seven parts, 1.01 PFLOP/s.  16 single queries over 65536 keys,
// 32 heads of 128 over 8: 56 us, 4.8 TB/s, and 8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gt_cross_tc.cuh"

namespace gt {
namespace cross {
namespace {

constexpr int kRows = 128;
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr int kThreads = 192;

// FEW: tiles of 32 rows.  The bytes of the keys bound these, and a third tile of keys and of values is on its way in the room
// that the rows leave.  (The tensor core still reads 128 rows from where the queries begin: the rest is whatever stands
// there, and stays in rows that nobody looks at.)
template <int PANELS, bool FEW>
struct Cfg {
    static constexpr int kStages = FEW ? 3 : 2, kTile = FEW ? kFewTile : kRows;
    static constexpr int kKeys = PANELS == 1 ? 96 : 64;         // of a tile
    static constexpr uint32_t kQPanel = kTile * 128, kKvPanel = kKeys * 128;
    static constexpr uint32_t kQ = PANELS * kQPanel, kKv = PANELS * kKvPanel;
    static constexpr size_t kSmem = 1024 + kQ + 2 * kStages * kKv;
    // TMEM columns: the scores of two tiles (each one's P over them), then O
    static constexpr uint32_t kO = 2 * kKeys;
    static constexpr uint32_t kTmem = 256;
};

struct Bars {
    uint64_t q_full, k_full[3], k_empty[3], v_full[3], v_empty[3];
    uint64_t s_full[2], p_full[2], o_done[2], fin;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Weights of 32 scores to a base, packed, and their sums: p = 2^(x c + shift).
__device__ __forceinline__ void weights(const uint32_t (&x)[32], float2 c, float2 shift, uint32_t (&p)[16], float2 (&sum)[2]) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 t = __ffma2_rn(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), c, shift);
        const float2 e = make_float2(ex2(t.x), ex2(t.y));
        sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], e);
        p[j / 2] = pack_bf16x2(e.x, e.y);
    }
}

template <int PANELS, bool FEW>
__global__ void __launch_bounds__(kThreads, 2)
cross_fwd(const Shape S, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
          const __grid_constant__ CUtensorMap map_v, const FwdOut out, int* status) {
    using C = Cfg<PANELS, FEW>;
    constexpr int kKeys = C::kKeys, kChunks = kKeys / 32, kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    const int tq = tile_queries(C::kTile, S.g), head = blockIdx.y, z = blockIdx.z;
    pdl_trigger();      // (the kernel that joins the parts may be scheduled; it waits for this one)
    const Tile t = find_tile(S, true, tq, blockIdx.x);
    if (!t.live) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = t.tile * tq, live = min(tq, t.lq - first) * S.g;
    const int tiles = (t.lk + kKeys - 1) / kKeys;
    const int t0 = part_begin(tiles, z, out.splits), n = part_begin(tiles, z + 1, out.splits) - t0;
    const int steps = (S.d + 15) / 16;
    uint8_t* sq = smem;
    uint8_t* sk = sq + C::kQ;
    uint8_t* sv = sk + kStages * C::kKv;
    if (threadIdx.x == kTmaWarp * 32) {
        mbar_init(&bars.q_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.k_full[s], 1);
            mbar_init(&bars.k_empty[s], 1);
            mbar_init(&bars.v_full[s], 1);
            mbar_init(&bars.v_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.s_full[b], 1);
            mbar_init(&bars.p_full[b], 4);
            mbar_init(&bars.o_done[b], 1);
        }
        mbar_init(&bars.fin, 1);
        bars.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    if (warp == kMmaWarp) tmem_alloc(&bars.tmem_base, C::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = bars.tmem_base;
    Waits w{&bars.abort, true};

    if (warp == kTmaWarp) {
        if (n > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars.q_full, PANELS * tq * S.g * 128);
                load_panels<PANELS>(sq, C::kQPanel, &map_q, head * S.g, t.q0 + first, &bars.q_full);
            }
            __syncwarp();
        }
        // keys a tile ahead of the values: their stage is free long before
        auto load = [&](int i, uint8_t* to, const CUtensorMap* map, uint64_t* full, uint64_t* empty) {
            const int s = i % kStages;
            // (the first time round finds every stage empty)
            if (!w.all(&empty[s], ((i / kStages) & 1) ^ 1)) return false;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], C::kKv);
                load_panels<PANELS>(to + s * C::kKv, C::kKvPanel, map, head, t.k0 + (t0 + i) * kKeys, &full[s]);
            }
            __syncwarp();
            return true;
        };
        int ik = 0, iv = 0;      // tiles under way
        while (iv < n) {
            if (ik < n && ik <= iv + 1) {
                if (!load(ik, sk, &map_k, bars.k_full, bars.k_empty)) break;
                ++ik;
                if (ik <= iv + 1 && ik < n) continue;
            }
            if (!load(iv, sv, &map_v, bars.v_full, bars.v_empty)) break;
            ++iv;
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        // nothing may still be on its way into shared memory when the CTA ends
        int never = 0;
        if (n > 0) mbar_wait_all(&bars.q_full, 0, &never, tc::kWaitNs);
        for (int b = max(0, ik - kStages); b < ik; ++b)
            mbar_wait_all(&bars.k_full[b % kStages], (b / kStages) & 1, &never, tc::kWaitNs);
        for (int b = max(0, iv - kStages); b < iv; ++b)
            mbar_wait_all(&bars.v_full[b % kStages], (b / kStages) & 1, &never, tc::kWaitNs);
    } else if (warp == kMmaWarp) {
        const uint32_t id_s = idesc_bf16(kRows, kKeys, false, false), id_o = idesc_bf16(kRows, 16 * steps, false, true);
        const SmemDesc dq = smem_desc_split(smem_u32(sq), 16, 1024, 2);
        const SmemDesc dk = smem_desc_split(smem_u32(sk), 16, 1024, 2);
        const SmemDesc dv = smem_desc_split(smem_u32(sv), C::kKvPanel, 1024, 2);
        auto at = [](SmemDesc d, int s) { return SmemDesc{d.lo + s * (C::kKv >> 4), d.hi}; };
        // (by one lane)
        auto scores = [&](int i) {
            const int s = i % kStages;
            product_channels<PANELS>(tb + kKeys * (i & 1), dq, C::kQPanel, at(dk, s), C::kKvPanel, steps, id_s);
            mma_commit(&bars.k_empty[s]);
            mma_commit(&bars.s_full[i & 1]);
        };
        if (n > 0) w.all(&bars.q_full, 0);
        for (int i = 0; i < min(n, 2) && w.ok; ++i) {
            if (!w.all(&bars.k_full[i], 0)) break;
            tc_fence_after();
            if (elect_one()) scores(i);
            __syncwarp();
        }
        for (int i = 0; i < n && w.ok; ++i) {      // O += P V of tile i, and behind it the scores of tile i + 2, over P
            const int s = i % kStages;
            if (!w.all(&bars.v_full[s], (i / kStages) & 1)) break;
            uint32_t words[kChunks];
            if (!valid_keys(S, t.k0 + (t0 + i) * kKeys, t.k0 + t.lk, words))
                clear_rows<kChunks, PANELS>(smem_u32(sv + s * C::kKv), C::kKvPanel, words);
            if (i + 2 < n && !w.all(&bars.k_full[(i + 2) % kStages], ((i + 2) / kStages) & 1)) break;
            if (!w.all(&bars.p_full[i & 1], (i >> 1) & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                product_rows<kKeys>(tb + C::kO, tb + kKeys * (i & 1), at(dv, s), id_o, i > 0);
                mma_commit(&bars.v_empty[s]);
                mma_commit(&bars.o_done[i & 1]);
                if (i + 2 < n) scores(i + 2);
            }
            __syncwarp();
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        int never = 0;
        if (elect_one()) mma_commit(&bars.fin);      // all products
        __syncwarp();
        mbar_wait_all(&bars.fin, 0, &never, tc::kWaitNs);
    } else {
        const int r = warp * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const bool some = warp * 32 < live;      // a warp without rows only keeps the barriers going
        const bool mine = r < live;
        const float c = S.scale * tc::kLog2e;
        const float most = 8.f / c;              // scores above the base
        float base = -INFINITY, sum = 0.f;       // (the base in scores before scaling)
        for (int i = 0; i < n; ++i) {
            if (!w.all(&bars.s_full[i & 1], (i >> 1) & 1)) break;
            tc_fence_after();
            if (!some) {
                if (lane == 0) mbar_arrive(&bars.p_full[i & 1]);
                continue;
            }
            const uint32_t at = tb + lanes + kKeys * (i & 1);
            uint32_t x[kChunks][32];
#pragma unroll
            for (int k = 0; k < kChunks; ++k) tmem_ld_x32(at + 32 * k, x[k]);
            tmem_wait_ld();
            uint32_t words[kChunks];      // (not formed any earlier: the scores take nearly all registers)
            if (!valid_keys(S, t.k0 + (t0 + i) * kKeys, t.k0 + t.lk, words)) {
#pragma unroll
                for (int k = 0; k < kChunks; ++k)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((words[k] >> j) & 1u)) x[k][j] = 0xff800000u;     // -infinity
            }
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    top4[(j >> 1) & 3] = max3(top4[(j >> 1) & 3], __uint_as_float(x[k][j]), __uint_as_float(x[k][j + 1]));
            const float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]);
            if (i == 0) {
                base = top;
            } else if (__any_sync(0xffffffffu, mine && (top > base + most || (base == -INFINITY && top > -INFINITY)))) {
                // raise the bases of the warp's rows: O so far, and its sum, in the new ones (rows without a query have no
                // say: what stands in theirs would change the others' roundings)
                const float higher = fmaxf(base, top), by = base == -INFINITY ? 0.f : ex2((base - higher) * c);
                if (!w.all(&bars.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1)) break;      // O is still
                tc_fence_after();
                for (int k = 0; k < steps; ++k) {
                    uint32_t o[16];
                    tmem_ld_x16(tb + lanes + C::kO + 16 * k, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
                    tmem_st_x16(tb + lanes + C::kO + 16 * k, o);
                }
                sum *= by;
                base = higher;
            }
            const float shift = base == -INFINITY ? 0.f : -base * c;
            float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                uint32_t p[16];
                weights(x[k], make_float2(c, c), make_float2(shift, shift), p, sum2);
                tmem_st_x16(at + 16 * k, p);
            }
            const float2 s = __fadd2_rn(sum2[0], sum2[1]);
            sum += s.x + s.y;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[i & 1]);
        }
        // all products, by a barrier of one phase (of o_done's, two may be over by the time a warp asks for the first)
        if (w.ok) w.all(&bars.fin, 0);
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        tc_fence_after();
        if (some && w.ok) {
            const int64_t query = t.q0 + first + r / S.g;
            const int qh = head * S.g + r % S.g;
            const bool seen = n > 0 && sum != 0.f;
            const float inv = seen ? 1.f / sum : 0.f, lse = seen ? base * S.scale + logf(sum) : -INFINITY;
            if (out.splits == 1) {
                bf16* p = static_cast<bf16*>(out.o.p) + query * out.o.row + qh * out.o.head;
                if (mine) out.lse[(int64_t)qh * S.nq + query] = lse;
                for (int k = 0; k < steps; ++k) {
                    uint32_t o[16];
                    if (n > 0) {
                        tmem_ld_x16(tb + lanes + C::kO + 16 * k, o);
                        tmem_wait_ld();
                    }
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = seen ? __uint_as_float(o[j]) * inv : 0.f;
                    if (mine) put16(p, 16 * k, S.d, v, out.o.acc);
                }
            } else {
                // (the join does not read the sums of a part without a key)
                if (mine) out.lse_part[(z * (int64_t)S.h + qh) * S.nq + query] = lse;
                float* p = out.o_part + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d;
                if (n > 0) tmem_row_out(tb + lanes + C::kO, steps, p, S.d, inv, mine && seen, S.d % 4 == 0 ? 1 : 0);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tb, C::kTmem);
}

template <int PANELS, bool FEW>
int launch(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s) {
    using C = Cfg<PANELS, FEW>;
    CUtensorMap mq, mk, mv;
    const int tq = tile_queries(C::kTile, S.g);
    if (!heads_map(&mq, q, S.nq, S.h, S.d, S.g, tq) || !heads_map(&mk, k, S.nk, S.hk, S.d, 1, C::kKeys) ||
        !heads_map(&mv, v, S.nk, S.hk, S.d, 1, C::kKeys))
        return GT_ERR_CUDA;
    int* status = device_status_ptr();
    if (!status) return GT_ERR_CUDA;
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, (const void*)cross_fwd<PANELS, FEW>, C::kSmem)) return GT_ERR_CUDA;
    LaunchScope ls("cross_fwd", s);
    cross_fwd<PANELS, FEW><<<dim3(slots_of(S, true, tq), S.hk, out.splits), kThreads, C::kSmem, s>>>(S, mq, mk, mv, out, status);
    return check_launch();
}

}  // namespace

bool few_tile(const Shape& S) { return ((int64_t)S.nq + S.batch - 1) / S.batch * S.g <= kFewTile; }

int fwd_tc(const Shape& S, const View& q, const View& k, const View& v, const FwdOut& out, cudaStream_t s) {
    if (few_tile(S)) return S.d <= 64 ? launch<1, true>(S, q, k, v, out, s) : launch<2, true>(S, q, k, v, out, s);
    return S.d <= 64 ? launch<1, false>(S, q, k, v, out, s) : launch<2, false>(S, q, k, v, out, s);
}

}  // namespace cross
}  // namespace gt
