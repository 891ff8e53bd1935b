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
    // significand x 2^64 / (2 pi), moved to its place: integer arithmetic throughout (fp64
    // instructions here held the cache write's fp64 pipe at 49 %)
    const uint64_t b = (uint64_t)__double_as_longlong(freq);
    const int down = 1075 - (int)((b >> 52) & 0x7FF);  // value = significand x 2^-down
    const uint64_t m = (b & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
    const uint64_t c = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    uint64_t t = 0;  // (frequencies of 2^52 and more, infinities and NaN: 0)
    if (down > 0 && down < 64)
        t = hi << (64 - down) | lo >> down;
    else if (down >= 64 && down < 128)
        t = hi >> (down - 64);
    return b >> 63 ? 0 - t : t;
}

// cos and sin of position * frequency, each times mscale.
__device__ __forceinline__ float2 turn(int32_t pos, uint64_t turns, float mscale) {
    const int64_t a = (int64_t)((uint64_t)(int64_t)pos * turns);  // in [-1/2, 1/2) turns, times 2^64
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns in [-1, 1]
    return make_float2(c * mscale, s * mscale);
}

constexpr int kMaxAxes = 4;  // axes of a position (time, height, width and one more)

// The axes of a head's pairs, from the caller's host array; false where one of them does not exist.
inline bool copy_axes(uint8_t *to, const uint8_t *axes, int pairs, int num_axes) {
    for (int j = 0; j < pairs; ++j) {
        if (axes[j] >= num_axes) return false;
        to[j] = axes[j];
    }
    return true;
}

}  // namespace mla
