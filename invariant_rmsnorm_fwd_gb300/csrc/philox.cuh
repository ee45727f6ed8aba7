// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011) and the dropout mask made from it.
//
// One evaluation gives 128 bits, a 16-bit uniform for each of the 8 columns of
// a vector: at 32 bits an element the 20 wide products of the ten rounds are
// paid per 4 elements and would take most of the SM's issue slots at the
// memory's pace; at 16 bits p acts in steps of 2^-16, which the factor
// 65536 / (65536 - t) undoes exactly (the expectation stays x).
#pragma once
#include <stdint.h>

namespace rbi {

struct DropParams {
    const uint64_t *state;           // device {seed, offset}; null = no dropout
    uint32_t t;                      // keep when the 16-bit uniform is >= t, 0 .. 65536
    float scale;                     // 65536 / (65536 - t), 0 when t == 65536
};

struct DropKey {                     // the call's seed and offset, loaded once per thread
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const DropParams &d) {
    const uint64_t s = d.state[0], o = d.state[1];
    return {uint32_t(s), uint32_t(s >> 32), uint32_t(o), uint32_t(o >> 32)};
}

__device__ __forceinline__ uint4 philox4x32(uint32_t c0, uint32_t c1, const DropKey &k) {
    uint32_t a = c0, b = c1, c = k.o0, d = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = uint64_t(a) * 0xD2511F53u, p1 = uint64_t(c) * 0xCD9E8D57u;
        a = uint32_t(p1 >> 32) ^ b ^ k0;
        b = uint32_t(p1);
        c = uint32_t(p0 >> 32) ^ d ^ k1;
        d = uint32_t(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
}

// Which of the 8 elements of a vector are kept: word i of its random words holds
// elements 2i (low half) and 2i + 1 (high half).  A half is >= t exactly when the
// half moved to the top of a word (whatever is below it) is >= t << 16.
struct DropRule {
    uint32_t limit;                  // t << 16
    bool any;                        // t < 65536
    float scale;
};
__device__ __forceinline__ DropRule drop_rule(const DropParams &d) { return {d.t << 16, d.t < 65536u, d.scale}; }
__device__ __forceinline__ bool kept_lo(uint32_t w, const DropRule &r) { return r.any && (w << 16) >= r.limit; }
__device__ __forceinline__ bool kept_hi(uint32_t w, const DropRule &r) { return r.any && w >= r.limit; }

}  // namespace rbi
