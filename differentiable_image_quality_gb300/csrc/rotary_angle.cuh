// The angle of a rotary position as a fraction of a turn in 64-bit fixed point; on the
// host too, where tests hold it to exact arithmetic.
#pragma once

#include <cmath>
#include <cuda_runtime.h>

namespace gbssim {

using turns64 = unsigned long long;  // of a turn, times 2^64: whole turns wrap by themselves

// How far a unit of position turns: |f| / (2 pi), f finite, as a fraction of a turn and
// whole turns, modulo 2^64, both exact but for the quotient's rounding.  Of a negative f
// the fraction's complement, which is the same for whole units alone.
__host__ __device__ inline double turns_of(double f) { return fabs(f) * 0.15915494309189535; }  // 1 / (2 pi)

__host__ __device__ inline turns64 turn_fraction(double f)
{
    const double t = turns_of(f);
    const turns64 part = turns64((t - floor(t)) * 0x1p64);
    return f < 0.0 ? 0ull - part : part;
}

__host__ __device__ inline turns64 whole_turns(double f)
{
    const double whole = floor(turns_of(f));
    return turns64(whole - floor(whole * 0x1p-64) * 0x1p64);
}

// The high 64 bits of a product.
__host__ __device__ inline turns64 high64(turns64 a, turns64 b)
{
#ifdef __CUDA_ARCH__
    return __umul64hi(a, b);
#else
    return turns64((unsigned __int128)(a)*b >> 64);
#endif
}

__host__ __device__ inline turns64 turn_phase(long long x, turns64 fraction) { return turns64(x) * fraction; }

// |x| below 2^63.  Whole units leave whole turns out; a part of a unit does not: its
// product with them counts too.  The part is exact to 2^-64 of a unit, all that a
// float32 above 2^-40 has.
__host__ __device__ inline turns64 turn_phase(float x, turns64 fraction, turns64 whole, bool negative)
{
    if (negative) fraction = 0ull - fraction;
    const float size = fabsf(x), units = floorf(size);
    const turns64 part = turns64((size - units) * 0x1p64f);
    const turns64 phase = turns64(units) * fraction + high64(part, fraction) + part * whole;
    return negative != (x < 0.0f) ? 0ull - phase : phase;
}

}  // namespace gbssim
