// Host side of the rotary operators: turns per position in 64-bit fixed point.
//
// A frequency f (radians per position) is m 2^e with a 53-bit integer m.  With
// C = 1 / (2 pi) in 128 fractional bits, m C 2^e in units of 2^-64 turn is the
// 192-bit product m C moved by 64 - e bits to the right, rounded to nearest and
// taken modulo 2^64: integers only, so every host gives the same words.  C is off
// by at most 2^-129, which is below 2^-10 of a unit for |f| < 2^54.
#include <cmath>
#include <cstdint>

#include "rotary_bi.h"

extern "C" int rotary_turns(const double *frequency, int32_t n, uint64_t *turns) {
    if (n < 0) return RMSNORM_ERR_LAYOUT;
    if (n > 0 && (!frequency || !turns)) return RMSNORM_ERR_NULL;
    const uint64_t c_hi = 0x28be60db9391054aull, c_lo = 0x7f09d5f47d4d3770ull;   // 1 / (2 pi)
    for (int32_t i = 0; i < n; ++i) {
        const double f = frequency[i];
        if (!std::isfinite(f) || std::fabs(f) >= 2147483648.0) return RMSNORM_ERR_VALUE;
        int e = 0;
        const double frac = std::frexp(std::fabs(f), &e);
        const uint64_t m = uint64_t(std::ldexp(frac, 53));
        // product of 192 bits, least significant word first
        const unsigned __int128 a = (unsigned __int128)m * c_lo, b = (unsigned __int128)m * c_hi + uint64_t(a >> 64);
        const uint64_t w[4] = {uint64_t(a), uint64_t(b), uint64_t(b >> 64), 0};
        const int shift = 64 + 53 - e;                   // at least 86: |f| < 2^31
        uint64_t t = 0;
        if (shift < 192) {
            const int word = shift / 64, bit = shift % 64;
            t = bit ? w[word] >> bit | w[word + 1] << (64 - bit) : w[word];
            const int at = shift - 1;                    // the highest bit that falls off
            t += (w[at / 64] >> (at % 64)) & 1;
        } else if (shift == 192) {
            t = w[2] >> 63;
        }
        turns[i] = f < 0 ? 0 - t : t;
    }
    return RMSNORM_OK;
}
