// Rotary positions: the angle of (position, frequency), shared by the rotation of queries
// and the cache write.
#pragma once
#include <stdint.h>

namespace mla {

// A frequency (radians per position) as a 64-bit fixed-point fraction of a turn per position.
// position * turns_fixed(f) modulo 2^64 is then the angle modulo one turn, in integer
// arithmetic and exact but for the frequency's own rounding: an fp32 product position * f
// would be off by 0.06 rad at a million positions, and fp64 units are few on this part.
__device__ __forceinline__ uint64_t turns_fixed(double freq) {
    double t = freq * 0.15915494309189533576888;  // 1 / (2 pi)
    t -= floor(t);
    return (uint64_t)(t * 18446744073709551616.0);
}

// cos and sin of position * frequency, each times mscale.
__device__ __forceinline__ float2 turn(int32_t pos, uint64_t turns, float mscale) {
    const int64_t a = (int64_t)((uint64_t)(int64_t)pos * turns);  // in [-1/2, 1/2) turns, times 2^64
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns in [-1, 1]
    return make_float2(c * mscale, s * mscale);
}

}  // namespace mla
