// gt_vec8.cuh -- eight consecutive row elements at a time, as the LayerNorm and
// linear-layer kernels move them: 16- and 32-byte accesses where rows allow
// them, single elements otherwise.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gt_common.cuh"

namespace gt {

// Whether rows of `ld` elements at p can be moved 16 bytes at a time at column
// offsets that are multiples of 8 elements.
inline bool rows16(const void* p, int64_t ld, int elem_bytes) {
    return aligned16(p) && (ld * elem_bytes) % 16 == 0;
}

// How rows can be moved at column offsets that are multiples of 16 elements: 2 by
// 32 bytes, 1 by 16, 0 by single elements.
inline int row_access(const void* p, int64_t ld, int elem_bytes) {
    if (!rows16(p, ld, elem_bytes)) return 0;
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (ld * elem_bytes) % 32 == 0 ? 2 : 1;
}

// Eight elements as stored: 16 bytes of bf16 or 32 of fp32.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

// 32 bytes at once (32-byte aligned).
__device__ __forceinline__ void ldg32(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

// Whether a kernel only reads an array, so that its loads may go through the read-only path, or may also write it: a
// residual that the caller lets be the output itself.
enum class Mem { kReadOnly, kOutput };

template <Mem MEM, typename T>
__device__ __forceinline__ T load1(const T* p) {
    if constexpr (MEM == Mem::kReadOnly) return __ldg(p);
    else return *p;
}

// Elements p[0 .. 7], those at or past `live` as zeros; acc: the row's row_access().
template <Mem MEM = Mem::kReadOnly, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int live, int acc) {
    Raw8<T> r;
    if (acc > 0 && live >= 8) {
        const uint4* s = reinterpret_cast<const uint4*>(p);
        if constexpr (sizeof(T) == 2) {
            r.a = load1<MEM>(s);
        } else if (acc == 2) {   // one access of 32 bytes: whole sectors
            if constexpr (MEM == Mem::kReadOnly) {
                asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                    : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w)
                    : "l"(p));
            } else {
                uint32_t w[8];
                ldg32(p, w);
                r.a = make_uint4(w[0], w[1], w[2], w[3]);
                r.b = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
            r.a = load1<MEM>(s);
            r.b = load1<MEM>(s + 1);
        }
    } else if constexpr (sizeof(T) == 4) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = i < live ? __float_as_uint(load1<MEM>(reinterpret_cast<const float*>(p) + i)) : 0u;
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        r.b = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < live ? (uint32_t)load1<MEM>(s + i) : 0u;
        r.a = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
    }
    return r;
}

// Eight fp32 that the kernel before this one wrote (16-byte aligned).
__device__ __forceinline__ Raw8<float> load8_cg(const float* p) {
    Raw8<float> r;
    r.a = __ldcg(reinterpret_cast<const uint4*>(p));
    r.b = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
    return r;
}

// load8 where WHOLE says that rows are whole eights in 16-byte accesses: `live` is then 8 or more, or nothing.
template <bool WHOLE, Mem MEM = Mem::kReadOnly, typename T>
__device__ __forceinline__ Raw8<T> load8_row(const T* p, int live, int acc) {
    if constexpr (!WHOLE) {
        return load8<MEM>(p, live, acc);
    } else {
        Raw8<T> r;
        r.a = make_uint4(0, 0, 0, 0);
        if constexpr (sizeof(T) == 4) r.b = r.a;
        if (live > 0) r = load8<MEM>(p, 8, sizeof(T) == 2 ? 1 : acc == 2 ? 2 : 1);
        return r;
    }
}

__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y); v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y); v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The same as pairs, for the packed arithmetic.
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float2 (&v)[4]) {
    float t[8];
    unpack8(r, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(t[2 * i], t[2 * i + 1]);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (32-byte aligned)
__device__ __forceinline__ void stg32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// p[0 .. 7] = v, the elements at or past `live` left alone.
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int live, int acc) {
    if (acc == 2 && live >= 8) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        stg32(p, w);
    } else if (acc > 0 && live >= 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = v[i];
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8], int live, int acc) {
    if (acc > 0 && live >= 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                                  bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = __float2bfloat16_rn(v[i]);
    }
}

}  // namespace gt
