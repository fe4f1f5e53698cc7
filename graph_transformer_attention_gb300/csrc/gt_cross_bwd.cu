// gt_cross_bwd.cu -- cross attention backward, bf16, on the tensor cores: dq by CTAs that hold a tile of queries, dk
// and dv by CTAs that hold a tile of keys.  Two kernels, seven products where one with sums in memory takes five: no
// result depends on the order in which CTAs finish.
//
//   p = exp(s - lse),  D = <dO, o>,  dS = p (dO v^T - D),  dq = scale dS k,  dk = scale dS^T q,  dv = p^T dO
//
// In both the scores and dP are formed again tile by tile, p and dS by warps that have a row each, and p and dS go back
// to TMEM as bf16 operands (half a step, 2^-8 of each entry at most, independent from one to the next).  The scores'
// scale comes last.
//
// What bounds both is shared memory, which a product of two operands there reads at 128 bytes a cycle (128 x 64 x 16: 48
// cycles, from TMEM 32), and the way from products to arithmetic and back (with neither products nor arithmetic, only the
// barriers: 248 us each for 4096 x 32768, 8 heads of 64).  There dq takes 329 us, dk and dv 484, 827 TFLOP/s of five
// products over the call; 4099 x 20001, 16 heads of 128 over 4: 106 and 128 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gt_cross_tc.cuh"

namespace gt {
namespace cross {
namespace {

constexpr int kHeld = 128;      // rows a CTA holds
constexpr int kStep = 64;       // rows of a streamed tile
constexpr uint32_t kHeldPanel = kHeld * 128, kStepPanel = kStep * 128;

__device__ __forceinline__ float2 pair_of(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// ---------------------------------------------------------------------------- dq

// Eight warps (four to each half of a tile), 256 TMEM columns, two CTAs to an SM, each one's products beside the other's
// arithmetic.  (What a CTA's issuing warp does for a tile, one instruction after the other between the arithmetic warps',
// bounds it: one CTA with two or three groups of four warps on tiles in turn took longer than two CTAs with one,
// 4096x32768, 8 heads of 64: dq 567 and 422 us, dk and dv 599 and 495.)  Up to 64 channels q and dO are moved to the
// columns that are left: 377 -> 327 us; with two tiles of 48 keys there instead 390.  Head dims above 64 leave room for
// one tile of values, which are done with before the keys.
template <int PANELS>
struct DqCfg {
    static constexpr int kKStages = PANELS == 1 ? 3 : 2, kVStages = PANELS == 1 ? 3 : 1;
    static constexpr uint32_t kHeldBytes = PANELS * kHeldPanel, kStepBytes = PANELS * kStepPanel;
    static constexpr size_t kSmem = 2 * kHeldBytes + (kKStages + kVStages) * kStepBytes;
    // TMEM columns: S (each half's dS over it) at 0, dP at 64, dq at 128; up to 64 channels, q and dO at 192 and 224
    static constexpr uint32_t kAcc = 128, kOwn = 192, kTmem = 256;
    static constexpr bool kInTmem = PANELS == 1;
    static constexpr int kTmaWarp = 8, kMmaWarp = kTmaWarp + 1, kThreads = 32 * (kMmaWarp + 1);
};

struct DqBars {
    uint64_t held_full, k_full[3], k_empty[3], v_full[3], v_empty[3];
    uint64_t own_full, s_full, ds_full, fin;
    uint32_t tmem_base;
    int abort;
};

// D = A B^T along up to 64 channels, A in TMEM (8 columns to 16 channels).
__device__ __forceinline__ void product_own(uint32_t d_tmem, uint32_t a_tmem, SmemDesc b, int steps, uint32_t idesc) {
    if (steps == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_ts(d_tmem, a_tmem + 8 * k, desc_at(b, k * 32), idesc, k > 0);
    } else {
        for (int k = 0; k < steps; ++k) mma_ts(d_tmem, a_tmem + 8 * k, desc_at(b, k * 32), idesc, k > 0);
    }
}

template <int PANELS>
__global__ void __launch_bounds__(DqCfg<PANELS>::kThreads, 2)
cross_dq(const Shape S, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
         const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
         const float2* __restrict__ stats, const Out dq, float* __restrict__ part, const int splits, int* status) {
    using C = DqCfg<PANELS>;
    constexpr int kKStages = C::kKStages, kVStages = C::kVStages;
    extern __shared__ __align__(1024) uint8_t smem[];      // (no room to align it by hand)
    __shared__ DqBars bars;
    const int tq = tile_queries(kHeld, S.g), head = blockIdx.y, z = blockIdx.z;
    const Tile t = find_tile(S, true, tq, blockIdx.x);
    follow_stats();
    if (!t.live) return;
    if (smem_u32(smem) & 1023u) {      // the swizzled tiles would not be where the products look for them
        if (threadIdx.x == 0) atomicOr(status, kStatusTimeout);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = t.tile * tq, live = min(tq, t.lq - first) * S.g;
    const int tiles = (t.lk + kStep - 1) / kStep;
    const int t0 = part_begin(tiles, z, splits), n = part_begin(tiles, z + 1, splits) - t0;
    const int steps = (S.d + 15) / 16;
    uint8_t* sq = smem;
    uint8_t* sdo = sq + C::kHeldBytes;
    uint8_t* sk = sdo + C::kHeldBytes;
    uint8_t* sv = sk + kKStages * C::kStepBytes;
    if (threadIdx.x == C::kTmaWarp * 32) {
        mbar_init(&bars.held_full, 1);
        for (int s = 0; s < 3; ++s) {
            mbar_init(&bars.k_full[s], 1);
            mbar_init(&bars.k_empty[s], 1);
            mbar_init(&bars.v_full[s], 1);
            mbar_init(&bars.v_empty[s], 1);
        }
        mbar_init(&bars.own_full, 8);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.ds_full, 8);
        mbar_init(&bars.fin, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&bars.tmem_base, C::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = bars.tmem_base;
    Waits w{&bars.abort, true};

    if (warp == C::kTmaWarp) {
        if (n > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars.held_full, 2 * PANELS * tq * S.g * 128);
                load_panels<PANELS>(sq, kHeldPanel, &map_q, head * S.g, t.q0 + first, &bars.held_full);
                load_panels<PANELS>(sdo, kHeldPanel, &map_do, head * S.g, t.q0 + first, &bars.held_full);
            }
            __syncwarp();
        }
        auto load = [&](int i, int stages, uint8_t* to, const CUtensorMap* map, uint64_t* full, uint64_t* empty) {
            const int s = i % stages;
            if (!w.all(&empty[s], ((i / stages) & 1) ^ 1)) return false;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], C::kStepBytes);
                load_panels<PANELS>(to + s * C::kStepBytes, kStepPanel, map, head, t.k0 + (t0 + i) * kStep, &full[s]);
            }
            __syncwarp();
            return true;
        };
        int ik = 0, iv = 0;      // tiles under way
        while (iv < n) {
            if (ik <= iv) {
                if (!load(ik, kKStages, sk, &map_k, bars.k_full, bars.k_empty)) break;
                ++ik;
            }
            if (!load(iv, kVStages, sv, &map_v, bars.v_full, bars.v_empty)) break;
            ++iv;
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        int never = 0;      // nothing may still be on its way into shared memory when the CTA ends
        if (n > 0) mbar_wait_all(&bars.held_full, 0, &never, tc::kWaitNs);
        for (int b = max(0, ik - kKStages); b < ik; ++b)
            mbar_wait_all(&bars.k_full[b % kKStages], (b / kKStages) & 1, &never, tc::kWaitNs);
        for (int b = max(0, iv - kVStages); b < iv; ++b)
            mbar_wait_all(&bars.v_full[b % kVStages], (b / kVStages) & 1, &never, tc::kWaitNs);
    } else if (warp == C::kMmaWarp) {
        const uint32_t id_s = idesc_bf16(kHeld, kStep, false, false), id_acc = idesc_bf16(kHeld, 16 * steps, false, true);
        const SmemDesc a_q = smem_desc_split(smem_u32(sq), 16, 1024, 2), a_do = smem_desc_split(smem_u32(sdo), 16, 1024, 2);
        const SmemDesc b_k = smem_desc_split(smem_u32(sk), 16, 1024, 2), b_v = smem_desc_split(smem_u32(sv), 16, 1024, 2);
        const SmemDesc r_k = smem_desc_split(smem_u32(sk), kStepPanel, 1024, 2);      // along its rows
        auto at = [](SmemDesc d, int s) { return SmemDesc{d.lo + s * (C::kStepBytes >> 4), d.hi}; };
        // What can be done ahead of a tile's products: its keys have landed, those that nobody sees are cleared.
        auto ready = [&](int i) {
            const int sk_ = i % kKStages, sv_ = i % kVStages;
            if (!w.all(&bars.k_full[sk_], (i / kKStages) & 1)) return;
            uint32_t words[kStep / 32];
            if (!valid_keys(S, t.k0 + (t0 + i) * kStep, t.k0 + t.lk, words))
                clear_rows<kStep / 32, PANELS>(smem_u32(sk + sk_ * C::kStepBytes), kStepPanel, words);
            w.all(&bars.v_full[sv_], (i / kVStages) & 1);
        };
        auto scores = [&](int i) {      // by one lane
            if constexpr (C::kInTmem) {
                product_own(tb, tb + C::kOwn, at(b_k, i % kKStages), steps, id_s);
                product_own(tb + 64, tb + C::kOwn + 32, at(b_v, i % kVStages), steps, id_s);
            } else {
                product_channels<PANELS>(tb, a_q, kHeldPanel, at(b_k, i % kKStages), kStepPanel, steps, id_s);
                product_channels<PANELS>(tb + 64, a_do, kHeldPanel, at(b_v, i % kVStages), kStepPanel, steps, id_s);
            }
            mma_commit(&bars.v_empty[i % kVStages]);
            mma_commit(&bars.s_full);
        };
        if (n > 0) w.all(C::kInTmem ? &bars.own_full : &bars.held_full, 0);
        if (n > 0 && w.ok) ready(0);
        tc_fence_after();
        if (n > 0 && w.ok && elect_one()) scores(0);
        __syncwarp();
        for (int i = 0; i < n && w.ok; ++i) {
            if (i + 1 < n) ready(i + 1);
            if (!w.ok || !w.all(&bars.ds_full, i & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                // dq += dS k, and behind it the next scores where dS stands (the tensor pipe runs one thread's products
                // in order)
                product_rows<kStep, true>(tb + C::kAcc, tb, at(r_k, i % kKStages), id_acc, i > 0);
                mma_commit(&bars.k_empty[i % kKStages]);
                if (i + 1 < n) scores(i + 1);
            }
            __syncwarp();
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        int never = 0;
        if (elect_one()) mma_commit(&bars.fin);      // all products
        __syncwarp();
        mbar_wait_all(&bars.fin, 0, &never, tc::kWaitNs);
    } else {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;      // 32 of the tile's keys, one row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tb + lanes + 32 * half;
        const bool some = (warp & 3) * 32 < live, mine = r < live;      // a warp without rows only keeps the barriers going
        const float c = S.scale * tc::kLog2e;
        const float2 st = mine ? __ldg(stats + ((int64_t)head * S.nq + t.q0 + first) * S.g + r) : make_float2(-INFINITY, 0.f);
        const float2 c2 = make_float2(c, c), minus_lse = make_float2(st.x, st.x), minus_d = make_float2(st.y, st.y);
        if (C::kInTmem && n > 0 && w.all(&bars.held_full, 0)) {      // the row of q, or of dO, to TMEM
            const uint32_t row = smem_u32(half ? sdo : sq) + r * 128;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                uint32_t x[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 u = lds_u4(row + (((j + k) ^ (r & 7)) << 4));      // (128-byte swizzle)
                    x[4 * k] = u.x, x[4 * k + 1] = u.y, x[4 * k + 2] = u.z, x[4 * k + 3] = u.w;
                }
                tmem_st_x16(tb + lanes + C::kOwn + 32 * half + 4 * j, x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.own_full);
        }
        for (int i = 0; i < n && w.ok; ++i) {
            uint32_t word[1];
            const bool all = valid_keys(S, t.k0 + (t0 + i) * kStep + 32 * half, t.k0 + t.lk, word);
            if (!w.all(&bars.s_full, i & 1)) break;
            tc_fence_after();
            if (some) {
                uint32_t x[32], y[32], ds[16];
                tmem_ld_x32(ts, x);
                tmem_ld_x32(ts + 64, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 a = pair_of(x[j], x[j + 1]), b = pair_of(y[j], y[j + 1]);
                    const float2 e = __ffma2_rn(a, c2, minus_lse);
                    const float2 g = __fmul2_rn(make_float2(ex2(e.x), ex2(e.y)), __fadd2_rn(b, minus_d));
                    ds[j / 2] = pack_bf16x2(g.x, g.y);
                }
                if (!all) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        ds[j] &= (((word[0] >> (2 * j)) & 1u) ? 0xffffu : 0u) | (((word[0] >> (2 * j + 1)) & 1u) ? 0xffff0000u : 0u);
                }
                tmem_st_x16(ts, ds);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ds_full);
        }
        w.all(&bars.fin, 0);
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        tc_fence_after();
        if (some && w.ok) {
            const int64_t query = t.q0 + first + r / S.g;
            const int qh = head * S.g + r % S.g;
            bf16* p = static_cast<bf16*>(dq.p) + query * dq.row + qh * dq.head;
            float* f = part + ((z * (int64_t)S.nq + query) * S.h + qh) * S.d;
            for (int k = half; k < steps; k += 2) {
                uint32_t o[16];
                if (n > 0) {
                    tmem_ld_x16(tb + lanes + C::kAcc + 16 * k, o);
                    tmem_wait_ld();
                }
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = n > 0 ? __uint_as_float(o[j]) * S.scale : 0.f;
                if (mine && splits == 1) put16(p, 16 * k, S.d, v, dq.acc);
                else if (mine) put16(f, 16 * k, S.d, v, S.d % 4 == 0 ? 1 : 0);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc(tb, C::kTmem);
}

// ---------------------------------------------------------------------------- dk, dv

// Head dims up to 64 as for dq (but TMEM has no room for k and v); above, the results take half of TMEM, and one CTA has
// two groups of eight warps on tiles in turn, with scores of their own.
template <int PANELS>
struct DkvCfg {
    static constexpr int kGroups = PANELS, kPerSm = 3 - PANELS;
    static constexpr int kStages = PANELS == 1 ? 3 : 4;
    static constexpr uint32_t kHeldBytes = PANELS * kHeldPanel, kStepBytes = PANELS * kStepPanel;
    static constexpr size_t kSmem = 1024 + 2 * kHeldBytes + 2 * kStages * kStepBytes;
    // TMEM columns: a group's S and dP (p and dS over them), then dv, then dk
    static constexpr uint32_t kDv = 128 * kGroups, kDk = kDv + 64 * PANELS, kTmem = 256 * PANELS;
    static constexpr int kTmaWarp = 8 * kGroups, kMmaWarp = kTmaWarp + 1, kThreads = 32 * (kMmaWarp + 1);
};

struct DkvBars {
    uint64_t held_full, q_full[4], q_empty[4];
    uint64_t s_full[2], p_full[2], fin;
    uint32_t tmem_base;
    int abort;
};

template <int PANELS>
__global__ void __launch_bounds__(DkvCfg<PANELS>::kThreads, DkvCfg<PANELS>::kPerSm)
cross_dkv(const Shape S, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
          const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
          const float2* __restrict__ stats, const Out dk, const Out dv, float* __restrict__ dk_part,
          float* __restrict__ dv_part, const int splits, int* status) {
    using C = DkvCfg<PANELS>;
    constexpr int kStages = C::kStages, kGroups = C::kGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ DkvBars bars;
    __shared__ alignas(16) float st_lse[kStages][kStep], st_d[kStages][kStep];
    const int tq = tile_queries(kStep, S.g), head = blockIdx.y, z = blockIdx.z;
    pdl_trigger();
    const Tile t = find_tile(S, false, kHeld, blockIdx.x);
    if (!t.live) {
        pdl_wait();
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = t.tile * kHeld;
    const int tiles = (t.lq + tq - 1) / tq;
    const int t0 = part_begin(tiles, z, splits), n = part_begin(tiles, z + 1, splits) - t0;
    const int steps = (S.d + 15) / 16;
    uint8_t* sk = smem;
    uint8_t* sv = sk + C::kHeldBytes;
    uint8_t* sq = sv + C::kHeldBytes;
    uint8_t* sdo = sq + kStages * C::kStepBytes;
    if (threadIdx.x == C::kTmaWarp * 32) {
        mbar_init(&bars.held_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.q_full[s], 1);
            mbar_init(&bars.q_empty[s], 1);
        }
        for (int b = 0; b < kGroups; ++b) {
            mbar_init(&bars.s_full[b], 1);
            mbar_init(&bars.p_full[b], 8);
        }
        mbar_init(&bars.fin, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&bars.tmem_base, C::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = bars.tmem_base;
    Waits w{&bars.abort, true};
    // rows of streamed tile i that exist
    auto rows_of = [&](int i) { return min(tq, t.lq - (t0 + i) * tq) * S.g; };

    if (warp == C::kTmaWarp) {
        if (n > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars.held_full, 2 * C::kHeldBytes);
                load_panels<PANELS>(sk, kHeldPanel, &map_k, head, t.k0 + first, &bars.held_full);
                load_panels<PANELS>(sv, kHeldPanel, &map_v, head, t.k0 + first, &bars.held_full);
            }
            __syncwarp();
        }
        int i = 0;
        for (; i < n; ++i) {
            const int s = i % kStages, q0 = t.q0 + (t0 + i) * tq, live = rows_of(i);
            const float2* src = stats + ((int64_t)head * S.nq + q0) * S.g;
            const float2 none = make_float2(-INFINITY, 0.f);
            const float2 a = lane < live ? __ldg(src + lane) : none, b = lane + 32 < live ? __ldg(src + lane + 32) : none;
            if (!w.all(&bars.q_empty[s], ((i / kStages) & 1) ^ 1)) break;
            st_lse[s][lane] = a.x;
            st_lse[s][lane + 32] = b.x;
            st_d[s][lane] = a.y;
            st_d[s][lane + 32] = b.y;
            __syncwarp();
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars.q_full[s], 2 * PANELS * tq * S.g * 128);
                load_panels<PANELS>(sq + s * C::kStepBytes, kStepPanel, &map_q, head * S.g, q0, &bars.q_full[s]);
                load_panels<PANELS>(sdo + s * C::kStepBytes, kStepPanel, &map_do, head * S.g, q0, &bars.q_full[s]);
            }
            __syncwarp();
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        int never = 0;      // nothing may still be on its way into shared memory when the CTA ends
        if (n > 0) mbar_wait_all(&bars.held_full, 0, &never, tc::kWaitNs);
        for (int b = max(0, i - kStages); b < i; ++b)
            mbar_wait_all(&bars.q_full[b % kStages], (b / kStages) & 1, &never, tc::kWaitNs);
    } else if (warp == C::kMmaWarp) {
        const uint32_t id_s = idesc_bf16(kHeld, kStep, false, false), id_acc = idesc_bf16(kHeld, 16 * steps, false, true);
        const SmemDesc a_k = smem_desc_split(smem_u32(sk), 16, 1024, 2), a_v = smem_desc_split(smem_u32(sv), 16, 1024, 2);
        const SmemDesc b_q = smem_desc_split(smem_u32(sq), 16, 1024, 2), b_do = smem_desc_split(smem_u32(sdo), 16, 1024, 2);
        const SmemDesc r_q = smem_desc_split(smem_u32(sq), kStepPanel, 1024, 2);      // along its rows
        const SmemDesc r_do = smem_desc_split(smem_u32(sdo), kStepPanel, 1024, 2);
        auto at = [](SmemDesc d, int s) { return SmemDesc{d.lo + s * (C::kStepBytes >> 4), d.hi}; };
        // What can be done ahead of a tile's products: its rows have landed, and those behind its sequence weigh nothing: dO
        // is 0, the statistic -infinity, and q the tile's first row, whose score with a key that holds an infinity is an
        // infinity and no NaN (0 x infinity), unless that row spoils the key's gradients anyway.  (Masks of p and dS instead:
        // 860 to 909 us a call instead of 830, 4096 x 32768, 8 heads of 64.)
        auto ready = [&](int i) {
            const int s = i % kStages;
            if (!w.all(&bars.q_full[s], (i / kStages) & 1)) return;
            const int live = rows_of(i);
            if (live < kStep) {
                repeat_row<PANELS>(smem_u32(sq + s * C::kStepBytes), kStepPanel, live, kStep);
                clear_tail<PANELS>(smem_u32(sdo + s * C::kStepBytes), kStepPanel, live, kStep);
            }
        };
        auto scores = [&](int i) {      // by one lane
            const int s = i % kStages, b = i % kGroups;
            product_channels<PANELS>(tb + 128 * b, a_k, kHeldPanel, at(b_q, s), kStepPanel, steps, id_s);
            product_channels<PANELS>(tb + 128 * b + 64, a_v, kHeldPanel, at(b_do, s), kStepPanel, steps, id_s);
            mma_commit(&bars.s_full[b]);
        };
        if (n > 0) w.all(&bars.held_full, 0);
        for (int i = 0; i < kGroups && i < n && w.ok; ++i) {
            ready(i);
            tc_fence_after();
            if (w.ok && elect_one()) scores(i);
            __syncwarp();
        }
        for (int i = 0; i < n && w.ok; ++i) {
            const int s = i % kStages, b = i % kGroups;
            if (kGroups == 1 && i + 1 < n) ready(i + 1);
            if (!w.ok || !w.all(&bars.p_full[b], (i / kGroups) & 1)) break;
            tc_fence_after();
            if (elect_one()) {
                // dv += p^T dO, dk += dS^T q, and behind them the next scores where p and dS stand (the tensor pipe runs one
                // thread's products in order)
                product_rows<kStep, true>(tb + C::kDv, tb + 128 * b, at(r_do, s), id_acc, i > 0);
                product_rows<kStep, true>(tb + C::kDk, tb + 128 * b + 64, at(r_q, s), id_acc, i > 0);
                mma_commit(&bars.q_empty[s]);
                if (kGroups == 1 && i + 1 < n) scores(i + 1);
            }
            __syncwarp();
            if (kGroups > 1 && i + kGroups < n) {      // (these rows may still be on their way: not before the products)
                ready(i + kGroups);
                tc_fence_after();
                if (w.ok && elect_one()) scores(i + kGroups);
                __syncwarp();
            }
        }
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        int never = 0;
        if (elect_one()) mma_commit(&bars.fin);      // all products
        __syncwarp();
        mbar_wait_all(&bars.fin, 0, &never, tc::kWaitNs);
    } else {
        const int group = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;      // 32 of the tile's rows, one key
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tb + lanes + 128 * group + 32 * half;
        const float c = S.scale * tc::kLog2e;
        const float2 c2 = make_float2(c, c);
        for (int i = group; i < n; i += kGroups) {
            const int s = i % kStages;
            const uint32_t turn = (i / kGroups) & 1;
            if (!w.all(&bars.q_full[s], (i / kStages) & 1) || !w.all(&bars.s_full[group], turn)) break;
            tc_fence_after();
            const uint32_t s_lse = smem_u32(st_lse[s]) + 128 * half, s_d = smem_u32(st_d[s]) + 128 * half;
            uint32_t x[32], y[32], p[16], ds[16];
            tmem_ld_x32(ts, x);
            tmem_ld_x32(ts + 64, y);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const uint4 l4 = lds_u4(s_lse + 4 * j), d4 = lds_u4(s_d + 4 * j);      // of four rows
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float2 a = pair_of(x[j + u], x[j + u + 1]), b = pair_of(y[j + u], y[j + u + 1]);
                    const float2 t = __ffma2_rn(a, c2, u ? pair_of(l4.z, l4.w) : pair_of(l4.x, l4.y));
                    const float2 e = make_float2(ex2(t.x), ex2(t.y));
                    const float2 g = __fmul2_rn(e, __fadd2_rn(b, u ? pair_of(d4.z, d4.w) : pair_of(d4.x, d4.y)));
                    p[(j + u) / 2] = pack_bf16x2(e.x, e.y);
                    ds[(j + u) / 2] = pack_bf16x2(g.x, g.y);
                }
            }
            tmem_st_x16(ts, p);
            tmem_st_x16(ts + 64, ds);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[group]);
        }
        w.all(&bars.fin, 0);
        if (!w.ok && lane == 0) tc::fail(&bars.abort, status);
        tc_fence_after();
        if (w.ok) {
            const bool mine = first + r < t.lk;
            const int64_t key = t.k0 + first + r;
            const bool seen = n > 0 && mine && (!S.mask || __ldg(S.mask + key) != 0);
            auto result = [&](const Out& g, float* part, uint32_t col, float by) {
                const bool whole = splits == 1;
                bf16* p = static_cast<bf16*>(g.p) + key * g.row + head * g.head;
                float* f = part + ((z * (int64_t)S.nk + key) * S.hk + head) * S.d;
                for (int k = group; k < steps; k += kGroups) {      // (the groups share the columns)
                    uint32_t o[16];
                    if (n > 0) {
                        tmem_ld_x16(tb + lanes + col + 16 * k, o);
                        tmem_wait_ld();
                    }
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = seen ? __uint_as_float(o[j]) * by : 0.f;
                    if (mine && whole) put16(p, 16 * k, S.d, v, g.acc);
                    else if (mine) put16(f, 16 * k, S.d, v, S.d % 4 == 0 ? 1 : 0);
                }
            };
            if (half == 0) result(dv, dv_part, C::kDv, 1.f);
            else result(dk, dk_part, C::kDk, S.scale);
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc(tb, C::kTmem);
    pdl_wait();
}

template <int PANELS>
int launch_dq(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s) {
    using C = DqCfg<PANELS>;
    CUtensorMap mq, mdo, mk, mv;
    const int tq = tile_queries(kHeld, S.g);
    if (!heads_map(&mq, in.q, S.nq, S.h, S.d, S.g, tq) || !heads_map(&mdo, in.dO, S.nq, S.h, S.d, S.g, tq) ||
        !heads_map(&mk, in.k, S.nk, S.hk, S.d, 1, kStep) || !heads_map(&mv, in.v, S.nk, S.hk, S.d, 1, kStep))
        return GT_ERR_CUDA;
    int* status = device_status_ptr();
    if (!status) return GT_ERR_CUDA;
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, (const void*)cross_dq<PANELS>, C::kSmem)) return GT_ERR_CUDA;
    LaunchScope ls("cross_dq", s);
    if (launch_overlapped(cross_dq<PANELS>, dim3(slots_of(S, true, tq), S.hk, splits), dim3(C::kThreads), C::kSmem, s, S, mq, mdo,
                          mk, mv, in.stats, dq, part, splits, status) != cudaSuccess)
        return GT_ERR_CUDA;
    return check_launch();
}

template <int PANELS>
int launch_dkv(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
               cudaStream_t s) {
    using C = DkvCfg<PANELS>;
    CUtensorMap mq, mdo, mk, mv;
    const int tq = tile_queries(kStep, S.g);
    if (!heads_map(&mq, in.q, S.nq, S.h, S.d, S.g, tq) || !heads_map(&mdo, in.dO, S.nq, S.h, S.d, S.g, tq) ||
        !heads_map(&mk, in.k, S.nk, S.hk, S.d, 1, kHeld) || !heads_map(&mv, in.v, S.nk, S.hk, S.d, 1, kHeld))
        return GT_ERR_CUDA;
    int* status = device_status_ptr();
    if (!status) return GT_ERR_CUDA;
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, (const void*)cross_dkv<PANELS>, C::kSmem)) return GT_ERR_CUDA;
    LaunchScope ls("cross_dkv", s);
    if (launch_overlapped(cross_dkv<PANELS>, dim3(slots_of(S, false, kHeld), S.hk, splits), dim3(C::kThreads), C::kSmem, s, S, mk,
                          mv, mq, mdo, in.stats, dk, dv, dk_part, dv_part, splits, status) != cudaSuccess)
        return GT_ERR_CUDA;
    return check_launch();
}

}  // namespace

int bwd_dq_tc(const Shape& S, const BwdIn& in, const Out& dq, float* part, int splits, cudaStream_t s) {
    return S.d <= 64 ? launch_dq<1>(S, in, dq, part, splits, s) : launch_dq<2>(S, in, dq, part, splits, s);
}

int bwd_dkv_tc(const Shape& S, const BwdIn& in, const Out& dk, const Out& dv, float* dk_part, float* dv_part, int splits,
               cudaStream_t s) {
    return S.d <= 64 ? launch_dkv<1>(S, in, dk, dv, dk_part, dv_part, splits, s)
                     : launch_dkv<2>(S, in, dk, dv, dk_part, dv_part, splits, s);
}

}  // namespace cross
}  // namespace gt
