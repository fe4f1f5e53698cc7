// gt_cross_tc.cuh -- what the tensor-core kernels of cross attention share.
//
// Operands stand in shared memory as panels of 64 channels, rows of 128 bytes under the 128-byte swizzle, as TMA lays
// them down; channels past d arrive as zeros.  The same panel serves a product along the channels (K-major) and one
// along the rows (MN-major): only the descriptors differ.  Products along the channels take ceil(d / 16) steps, products
// whose columns are the channels 16 ceil(d / 16) columns.
#pragma once

#include <cuda.h>

#include "gt_cross.cuh"
#include "gt_stats.cuh"
#include "gt_tma.cuh"

namespace gt {
namespace cross {

using namespace sm100;

// Map of [rows][heads][d] with a box of 64 channels, `heads_box` heads and `rows_box` rows.
inline bool heads_map(CUtensorMap* map, const View& v, int rows, int heads, int d, int heads_box, int rows_box) {
    const uint64_t row = (uint64_t)v.row * 2, head = (uint64_t)v.head * 2;
    return make_map_4d(map, v.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, {(uint64_t)d, (uint64_t)heads, (uint64_t)rows, 1},
                       {head, row, row}, {64, (uint32_t)heads_box, (uint32_t)rows_box, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
}

// All panels of a box by the elected lane.
template <int PANELS>
__device__ __forceinline__ void load_panels(uint8_t* dst, uint32_t panel_bytes, const CUtensorMap* map, int head, int row,
                                            uint64_t* bar) {
#pragma unroll
    for (int p = 0; p < PANELS; ++p) tma_load_4d(dst + p * panel_bytes, map, 64 * p, head, row, 0, bar);
}

// D = A B^T along the channels (PANELS of them, `steps` 16-channel steps): rows of A and of B as panels of a_panel and
// b_panel bytes.
template <int PANELS>
__device__ __forceinline__ void product_channels(uint32_t d_tmem, SmemDesc a, uint32_t a_panel, SmemDesc b, uint32_t b_panel,
                                                 int steps, uint32_t idesc) {
    auto step = [&](int k) {
        mma_ss(d_tmem, desc_at(a, (k >> 2) * a_panel + (k & 3) * 32), desc_at(b, (k >> 2) * b_panel + (k & 3) * 32), idesc, k > 0);
    };
    if (steps == 4 * PANELS) {      // (a fixed number goes out without a test between the products)
#pragma unroll
        for (int k = 0; k < 4 * PANELS; ++k) step(k);
    } else {
        for (int k = 0; k < steps; ++k) step(k);
    }
}

// D (+)= W B along B's ROWS rows, W in TMEM (bf16, 8 columns to 16 rows).  HALVES: the columns of rows 32 .. 63 begin 32
// columns on, each half where the fp32 values it was made of stood.
template <int ROWS, bool HALVES = false>
__device__ __forceinline__ void product_rows(uint32_t d_tmem, uint32_t w_tmem, SmemDesc b, uint32_t idesc, bool add) {
#pragma unroll
    for (int k = 0; k < ROWS / 16; ++k)
        mma_ts(d_tmem, w_tmem + (HALVES ? 32 * (k >> 1) + 8 * (k & 1) : 8 * k), desc_at(b, k * 2048), idesc, add || k > 0);
}

// Waits of a role, by whole warps; a wait that gives up says so, and the role ends.
struct Waits {
    volatile int* abort;
    bool ok;
    __device__ __forceinline__ bool all(uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        ok = ok && mbar_wait_all(bar, parity, abort, tc::kWaitNs);
        return ok;
    }
};

// A row of `steps` x 16 fp32 TMEM columns, times `by`, to p[0 .. d - 1].
template <typename T>
__device__ __forceinline__ void tmem_row_out(uint32_t taddr, int steps, T* p, int d, float by, bool live, int acc) {
    for (int k = 0; k < steps; ++k) {
        uint32_t r[16];
        tmem_ld_x16(taddr + 16 * k, r);
        tmem_wait_ld();
        if (live) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]) * by;
            put16(p, 16 * k, d, v, acc);
        }
    }
}

}  // namespace cross
}  // namespace gt
