// Element types of the operators that take more than float32 (gbssim_dtype),
// and 16-byte accesses to them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gbssim.h"

namespace gbssim {

using bf16 = __nv_bfloat16;
using f16 = __half;

__host__ __device__ constexpr bool dtype_ok(int t) { return t >= GBSSIM_F32 && t <= GBSSIM_F16; }
__host__ __device__ constexpr int dtype_bytes(int t) { return t == GBSSIM_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(f16 v) { return __half2float(v); }

// One rounding (to nearest even) from the 32-bit result.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float v) { return __float2half_rn(v); }

// The two 16-bit values of a 32-bit word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<bf16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<f16>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<bf16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<f16>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 16 bytes that this kernel reads once (or whose reuse is in L2): no line kept
// in L1.
__device__ __forceinline__ uint4 ld_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight consecutive elements as they lie in memory: one 16-byte word of a
// 16-bit type, two of float32.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) == 4 ? 2 : 1];
};

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(r.w[0].x); v[1] = __uint_as_float(r.w[0].y);
        v[2] = __uint_as_float(r.w[0].z); v[3] = __uint_as_float(r.w[0].w);
        v[4] = __uint_as_float(r.w[1].x); v[5] = __uint_as_float(r.w[1].y);
        v[6] = __uint_as_float(r.w[1].z); v[7] = __uint_as_float(r.w[1].w);
    } else {
        const float2 a = unpack2<T>(r.w[0].x), b = unpack2<T>(r.w[0].y);
        const float2 c = unpack2<T>(r.w[0].z), d = unpack2<T>(r.w[0].w);
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
        v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
    }
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&v)[8])
{
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                            __float_as_uint(v[3]));
        r.w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                            __float_as_uint(v[7]));
    } else {
        r.w[0] = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                            pack2<T>(v[6], v[7]));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void st8(T *p, const Raw8<T> &r)
{
    reinterpret_cast<uint4 *>(p)[0] = r.w[0];
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint4 *>(p)[1] = r.w[1];
}

// p: 32-byte aligned for float32.  One instruction, so that lanes side by side
// write whole lines.
template <typename T>
__device__ __forceinline__ void st8_whole(T *p, const Raw8<T> &r)
{
    if constexpr (sizeof(T) == 4)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0].x),
                     "r"(r.w[0].y), "r"(r.w[0].z), "r"(r.w[0].w), "r"(r.w[1].x), "r"(r.w[1].y),
                     "r"(r.w[1].z), "r"(r.w[1].w)
                     : "memory");
    else
        st8(p, r);
}

// ---------------------------------------------- eight elements at any alignment

// Eight elements that begin `s` elements into consecutive 16-byte words: one
// word more than eight elements fill.
template <typename T>
struct Wide8 {
    static constexpr int kUnits = sizeof(T) == 4 ? 3 : 2;
    uint32_t w[kUnits * 4];
};

// The eight elements from element s on (s < 16 / sizeof(T)).
template <typename T>
__device__ __forceinline__ Raw8<T> shift_down(const Wide8<T> &in, int s)
{
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < Wide8<T>::kUnits * 4; ++i) w[i] = in.w[i];
    Raw8<T> r;
    uint32_t *o = reinterpret_cast<uint32_t *>(&r);
    if constexpr (sizeof(T) == 4) {
        if (s & 2) {
#pragma unroll
            for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s & 1 ? w[i + 1] : w[i];
    } else {
        if (s & 4) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (s & 2) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const unsigned half = (s & 1) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], half);
    }
    return r;
}

// 16 bytes to shared memory (a 32-bit shared address) without passing through
// registers; KEEP: L1 keeps the line, for a neighbour's copy that overlaps.
template <bool KEEP>
__device__ __forceinline__ void copy16_async(unsigned smem, const void *gmem)
{
    if constexpr (KEEP)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

// Zeros, and nothing read, where `wanted` is false (a predicate, no branch).
__device__ __forceinline__ uint4 ld_shared16(unsigned smem, bool wanted)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n"
        " @p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "r"(smem), "r"(unsigned(wanted))
        : "memory");
    return v;
}

// ------------------------------------------------------------ pairs of floats
// Two float32 in one 64-bit register: one instruction does both (fma.rn.f32x2;
// each half rounds as the scalar instruction does).

using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 halves(f32x2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 v)
{
    const float2 h = halves(v);
    return h.x + h.y;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, f32x2 (&v)[4])
{
    float f[8];
    unpack8<T>(r, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const f32x2 (&v)[4])
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 h = halves(v[i]);
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
    }
    return pack8<T>(f);
}

}  // namespace gbssim
