// Rotary positions of queries and keys, alone and behind an RMS norm of every
// head, and their backward pass (sm_103a): what the kernels share, and the row
// kernels.
//
// A head is held by a team of lanes, 16 columns a lane: always both columns of
// its 8 pairs, so the rotation needs no exchange between lanes.  In the half
// layout a lane has 8 columns of the first half and the 8 that go with them, else 16 in a
// row.  A team stays with one token and walks over a chunk of its heads, so the
// lane's 8 sines and cosines are formed once per chunk.
#pragma once
#include <type_traits>

#include "host.cuh"
#include "layernorm_narrow.cuh"
#include "rotary_bi.h"

namespace rbi {

constexpr int kChunkHeads = 8;                           // most heads of a chunk of the weight gradients' order
constexpr int kQkGroup = 8;                              // logical tokens of a group of that order
constexpr uint64_t kQkMagic = 0x3149422d4b514e52ull;

inline int qk_chunks(int heads) { return (heads + kChunkHeads - 1) / kChunkHeads; }

struct QkWs {
    WsHeader *hdr;                   // n_rows tokens; hidden = the sizes (qk_sizes)
    int32_t *flag;                   // [N] 0 nothing, 1 in its group's partial, 2 its own sums stored
    float *partial;                  // [chunks of q, then k][groups][D]
    float *spill;                    // [chunks][N][D]: a token's sums
    int64_t n, groups, sizes;
    int32_t chunks_q, chunks_k, D;
};

inline int64_t qk_sizes(int64_t D, int32_t hq, int32_t hk) { return D | int64_t(hq) << 16 | int64_t(hk) << 32; }

struct QkWsLayout {
    int64_t off_partial, off_spill, total;
    QkWsLayout(int64_t N, int32_t hq, int32_t hk, int64_t D) {
        const int64_t chunks = qk_chunks(hq) + qk_chunks(hk), groups = (N + kQkGroup - 1) / kQkGroup;
        off_partial = align256(256 + N * 4);
        off_spill = align256(off_partial + chunks * groups * D * 4);
        total = align256(off_spill + chunks * N * D * 4);
    }
};

inline QkWs qk_ws(void *base, int64_t N, int32_t hq, int32_t hk, int64_t D) {
    const QkWsLayout L(N, hq, hk, D);
    uint8_t *b = static_cast<uint8_t *>(base);
    QkWs w;
    w.hdr = reinterpret_cast<WsHeader *>(b);
    w.flag = reinterpret_cast<int32_t *>(b + 256);
    w.partial = reinterpret_cast<float *>(b + L.off_partial);
    w.spill = reinterpret_cast<float *>(b + L.off_spill);
    w.n = N;
    w.groups = (N + kQkGroup - 1) / kQkGroup;
    w.sizes = qk_sizes(D, hq, hk);
    w.chunks_q = qk_chunks(hq);
    w.chunks_k = qk_chunks(hk);
    w.D = int32_t(D);
    return w;
}

__device__ __forceinline__ bool qk_header_ok(const QkWs &ws) {
    const WsHeader *h = ws.hdr;
    const auto magic = h->magic;
    const int64_t n = h->n_rows, sizes = h->hidden;
    return (magic == kQkMagic) & (n == ws.n) & (sizes == ws.sizes);
}
__device__ __forceinline__ void qk_report(const QkWs &ws, int bits) { atomicOr(&ws.hdr->status, bits); }

struct HeadsParams {                 // one tensor's heads; strides in elements
    const void *in, *dy, *w;
    void *out;
    int64_t in_t, in_h, dy_t, dy_h, out_t, out_h;
    int32_t heads, per;              // heads; heads of a chunk
};

struct RotaryParams {
    HeadsParams side[2];             // queries, keys
    const int32_t *tok_id, *position;
    const uint64_t *turns;
    int64_t n_tokens;
    int32_t D, rot, first;
    int32_t chunks_q, chunks;        // chunks of the queries, of both
    int32_t team;                    // lanes of a head
    int32_t most;                    // most heads of a chunk
    int32_t params_f32, in_place;    // in_place: columns outside the rotation are already where they belong
    float scale, sign;               // sign: of the sine (-1 turns back)
    float eps, inv_d;
    uint32_t units;                  // teams' (warps') pieces of work
    Divisor by_chunks{1}, by_team{1};
    QkWs ws;
};

// ----------------------------------------------------------------- a lane's columns

// WIDE: two vectors of 8 columns, at[0] and at[1].  Else (rotary sizes that are not
// made of whole vectors) eight pieces of two columns: at[0..3] go with the first
// vector's pairs of registers, at[4..7] with the second's.  -1: nothing there.
template <bool INTER, bool WIDE>
struct LaneColumns {
    int32_t at[WIDE ? 2 : 8];
    int32_t turned;                  // the lane's first `turned` pairs rotate, 8 lane .. of the head
};

__device__ __forceinline__ int outside(int e, int first, int rot) { return e < first ? e : e + rot; }

template <bool INTER, bool WIDE>
__device__ __forceinline__ LaneColumns<INTER, WIDE> lane_columns(int lane, int D, int rot, int first, bool in_place) {
    LaneColumns<INTER, WIDE> c;
    const int half = rot >> 1, rest = D - rot;
    const int t = half - 8 * lane;
    c.turned = t < 0 ? 0 : t > 8 ? 8 : t;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int e;                                       // column among those outside the rotation
            if constexpr (INTER) {
                const int v = 2 * lane + i;
                c.at[i] = first + 8 * v;
                e = 8 * v - rot;
            } else {
                c.at[i] = first + 8 * lane + i * half;
                e = 16 * lane - rot + 8 * i;
                if (c.turned) e = -1;
            }
            if (e >= 0) c.at[i] = e < rest && !in_place ? outside(e, first, rot) : -1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int e;
            if constexpr (INTER) {
                const int p = 8 * lane + i;
                c.at[i] = first + 2 * p;
                e = 2 * p - rot;
            } else {
                const int p = 8 * lane + 2 * (i & 3);    // first pair of the unit
                c.at[i] = first + p + (i >> 2) * half;
                e = 2 * p - rot + 2 * (i >> 2);
                if (p < half) e = -1;
            }
            if (e >= 0) c.at[i] = e < rest && !in_place ? outside(e, first, rot) : -1;
        }
    }
    return c;
}

// The lane's 16 elements as they are in memory.
template <class E>
struct Raw {
    static constexpr int kW = 4 * int(sizeof(E));        // 32-bit words; pair i of registers is kW / 8 of them
    uint32_t w[kW];
};

__device__ __forceinline__ uint4 ld_stream_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <class E, bool INTER, bool WIDE>
__device__ __forceinline__ void load_lane(Raw<E> &r, const void *base, int64_t off, const LaneColumns<INTER, WIDE> &c, bool on) {
    const E *p = static_cast<const E *>(base) + off;
    constexpr int Q = int(sizeof(E)) / 2;                // 16-byte words of a vector
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (on && c.at[i] >= 0) v = ld_stream_v4(reinterpret_cast<const uint4 *>(p + c.at[i]) + k);
                uint32_t *w = r.w + (i * Q + k) * 4;
                w[0] = v.x;
                w[1] = v.y;
                w[2] = v.z;
                w[3] = v.w;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < Q; ++k)
                r.w[i * Q + k] = on && c.at[i] >= 0 ? reinterpret_cast<const uint32_t *>(p + c.at[i])[k] : 0u;
    }
}

template <class E, bool INTER, bool WIDE>
__device__ __forceinline__ void store_lane(const Raw<E> &r, void *base, int64_t off, const LaneColumns<INTER, WIDE> &c) {
    E *p = static_cast<E *>(base) + off;
    constexpr int Q = int(sizeof(E)) / 2;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (c.at[i] >= 0) {
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const uint32_t *w = r.w + (i * Q + k) * 4;
                    st_global_v4(reinterpret_cast<uint4 *>(p + c.at[i]) + k, make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c.at[i] >= 0) {
#pragma unroll
                for (int k = 0; k < Q; ++k) reinterpret_cast<uint32_t *>(p + c.at[i])[k] = r.w[i * Q + k];
            }
    }
}

template <class E>
__device__ __forceinline__ f2_t up2(const Raw<E> &r, int i) {
    if constexpr (sizeof(E) == 4) {
        return f2_make(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    } else if constexpr (std::is_same_v<E, __half>) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
        return f2_make(p.x, p.y);
    } else {
        return f2_from_bf16x2(r.w[i]);
    }
}
template <class E>
__device__ __forceinline__ void down2(Raw<E> &r, int i, f2_t v) {
    if constexpr (sizeof(E) == 4) {
        r.w[2 * i] = __float_as_uint(f2_lo(v));
        r.w[2 * i + 1] = __float_as_uint(f2_hi(v));
    } else if constexpr (std::is_same_v<E, __half>) {
        const __half2 h = __floats2half2_rn(f2_lo(v), f2_hi(v));
        r.w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        r.w[i] = f2_to_bf16x2(v);
    }
}

// A lane's columns of a parameter vector (NULL: ones).
template <class E, bool INTER, bool WIDE>
__device__ __forceinline__ void lane_weights(const void *w, int f32, const LaneColumns<INTER, WIDE> &c, f2_t (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = WIDE ? c.at[i >> 2] : c.at[i];
        f[i] = f2_make(1.f, 1.f);
        if (w && at >= 0) {
            const int col = WIDE ? at + 2 * (i & 3) : at;
            if (f32 || sizeof(E) == 4) {
                const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(w) + col);
                f[i] = f2_make(v.x, v.y);
            } else {
                Raw<E> r;
                r.w[0] = *reinterpret_cast<const uint32_t *>(static_cast<const E *>(w) + col);
                f[i] = up2<E>(r, 0);
            }
        }
    }
}

// ----------------------------------------------------------------- angles

// Cosine and sine of position * turns / 2^64 turns.  The product modulo 2^64 is
// exact; its top 32 bits, off by less than 2^-32 turn, are split into a quadrant
// and a rest of at most 1/8 turn either way, y = rest in radians.  sin y and cos y
// are their Taylor polynomials of degree 9 and 10: what is left out is below
// (pi/4)^11 / 11! = 1.8e-9 and (pi/4)^12 / 12! = 1.2e-10.  y is formed with what
// the float of the rest loses, and enters as y + d: sin + d cos, cos - d sin.
__device__ __forceinline__ void cos_sin(int32_t position, uint64_t turns, float &c, float &s) {
    const int32_t top = int32_t(uint64_t(int64_t(position)) * turns >> 32);
    const uint32_t quadrant = (uint32_t(top) + 0x20000000u) >> 30;
    const int32_t rest = int32_t(uint32_t(top) - (quadrant << 30));
    const float f = __int2float_rn(rest);
    const float lost = __int2float_rn(rest - __float2int_rn(f));
    // 2 pi / 2^32 in two floats: 0x1.921fb6p-30 and pi's next bits
    const float kHi = 0x1.921fb6p-30f, kLo = -0x1.777a5cp-55f;
    const float y = __fmul_rn(f, kHi);
    const float d = __fmaf_rn(lost, kHi, __fmaf_rn(f, kLo, __fmaf_rn(f, kHi, -y)));
    const float z = __fmul_rn(y, y);
    float p = __fmaf_rn(z, 1.f / 362880.f, -1.f / 5040.f);
    p = __fmaf_rn(z, p, 1.f / 120.f);
    p = __fmaf_rn(z, p, -1.f / 6.f);
    const float sy = __fmaf_rn(__fmul_rn(z, y), p, y);
    float q = __fmaf_rn(z, -1.f / 3628800.f, 1.f / 40320.f);
    q = __fmaf_rn(z, q, -1.f / 720.f);
    q = __fmaf_rn(z, q, 1.f / 24.f);
    q = __fmaf_rn(z, q, -0.5f);
    const float cy = __fmaf_rn(z, q, 1.f);
    const float sn = __fmaf_rn(d, cy, sy), cs = __fmaf_rn(-d, sy, cy);
    c = quadrant & 1 ? sn : cs;
    s = quadrant & 1 ? cs : sn;
    if ((quadrant + 1) & 2) c = -c;
    if (quadrant & 2) s = -s;
}

// The lane's 8 pairs of cosine and sine, times scale, in registers of two.
__device__ __forceinline__ void lane_angles(const RotaryParams &p, int32_t position, int lane, int turned, f2_t (&c)[4],
                                            f2_t (&s)[4]) {
    const ulonglong2 *t = reinterpret_cast<const ulonglong2 *>(p.turns) + lane * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float c0 = 1.f, c1 = 1.f, s0 = 0.f, s1 = 0.f;
        if (2 * i < turned) {                            // the number of pairs is even
            const ulonglong2 v = t[i];
            cos_sin(position, v.x, c0, s0);
            cos_sin(position, v.y, c1, s1);
        }
        c[i] = f2_mul(f2_make(c0, c1), f2_both(p.scale));
        s[i] = f2_mul(f2_make(s0, s1), f2_both(__fmul_rn(p.scale, p.sign)));
    }
}

// Rotates the lane's pairs: f[0..3] first vector, f[4..7] second.
template <bool INTER>
__device__ __forceinline__ void turn_lane(f2_t (&f)[8], const f2_t (&c)[4], const f2_t (&s)[4], int turned) {
    if constexpr (!INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i < turned) {
                const f2_t a = f[i], b = f[4 + i], n = f2_make(-f2_lo(s[i]), -f2_hi(s[i]));
                f[i] = f2_fma(a, c[i], f2_mul(b, n));
                f[4 + i] = f2_fma(b, c[i], f2_mul(a, s[i]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < turned) {
                const float a = f2_lo(f[i]), b = f2_hi(f[i]);
                const float ci = i & 1 ? f2_hi(c[i >> 1]) : f2_lo(c[i >> 1]), si = i & 1 ? f2_hi(s[i >> 1]) : f2_lo(s[i >> 1]);
                f[i] = f2_make(__fmaf_rn(a, ci, -__fmul_rn(b, si)), __fmaf_rn(b, ci, __fmul_rn(a, si)));
            }
        }
    }
}

// Pair i of registers holds rotated columns.
template <bool INTER>
__device__ __forceinline__ bool is_turned(int i, int turned) { return INTER ? i < turned : 2 * (i & 3) < turned; }

// Sum over the lanes of a team of a power of two.
__device__ __forceinline__ float team_add(float v, int team) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        if (o < team) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// Row sums of products f g: pairs 0, 1, .. by FMA, then the two columns of a pair.
__device__ __forceinline__ float lane_dot(const f2_t (&f)[8], const f2_t (&g)[8]) {
    f2_t v = f2_mul(f[0], g[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) v = f2_fma(f[i], g[i], v);
    return __fadd_rn(f2_lo(v), f2_hi(v));
}

__device__ __forceinline__ float qk_rstd(float ss, const RotaryParams &p) { return row_rstd(ss, float(p.D), p.inv_d, p.eps); }

// ----------------------------------------------------------------- forward, and rotation alone

constexpr int kRotaryThreads = 256;

template <class E, bool INTER, bool WIDE, bool NORM>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    const uint32_t mine = p.by_team.quotient(threadIdx.x), teams = p.by_team.quotient(kRotaryThreads);
    const int lane = int(threadIdx.x - mine * uint32_t(p.team));
    const uint32_t unit = blockIdx.x * teams + mine, token = p.by_chunks.quotient(unit);
    int chunk = int(unit - token * uint32_t(p.chunks));
    bool on = mine < teams && unit < p.units;
    if (on) on = p.tok_id[token] >= 0;
    if constexpr (!NORM) {
        if (!on) return;
    }
    const LaneColumns<INTER, WIDE> col = lane_columns<INTER, WIDE>(lane, p.D, p.rot, p.first, p.in_place);
    const HeadsParams &h = p.side[chunk >= p.chunks_q];
    if (chunk >= p.chunks_q) chunk -= p.chunks_q;
    const int head0 = chunk * h.per;
    int n = h.heads - head0;
    if (n > h.per) n = h.per;
    if (!on) n = 0;
    f2_t c[4], s[4], w[8];
    lane_angles(p, on ? p.position[token] : 0, lane, col.turned, c, s);
    if constexpr (NORM) lane_weights<E, INTER, WIDE>(h.w, p.params_f32, col, w);
    int64_t in = int64_t(token) * h.in_t + head0 * h.in_h, out = int64_t(token) * h.out_t + head0 * h.out_h;
    constexpr int U = sizeof(E) == 4 ? 2 : 4;
    for (int i = 0; i < (NORM ? p.most : n); i += U) {
        Raw<E> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load_lane<E, INTER, WIDE>(r[u], h.in, in + u * h.in_h, col, i + u < n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = up2<E>(r[u], j);
            if constexpr (NORM) {
                const float rstd = qk_rstd(team_add(lane_dot(f, f), p.team), p);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = f2_mul(f2_mul(f[j], f2_both(rstd)), w[j]);
            }
            turn_lane<INTER>(f, c, s, col.turned);
            Raw<E> y = r[u];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (NORM || is_turned<INTER>(j, col.turned)) down2<E>(y, j, f[j]);
            if (i + u < n) store_lane<E, INTER, WIDE>(y, h.out, out + u * h.out_h, col);
        }
        in += U * h.in_h;
        out += U * h.out_h;
    }
}

// ----------------------------------------------------------------- backward of the norm and the rotation

constexpr int kQkWarps = 4;

// What a warp of the backward pass does with the 8 slots [8 w, 8 w + 8) of a call and
// one chunk of heads: the run, 8 consecutive slots that hold a whole group in logical
// order and start among them (at most one does), and the active slots that
// belong to no run.  Slots of a run that starts in the window before are that
// window's.
struct Window {
    int64_t run;                     // first slot of the run, -1: none
    uint32_t loose;                  // bit j: slot 8 w + j on its own
};
__device__ __forceinline__ Window window_of(const RotaryParams &p, int64_t w, bool grads) {
    const int lane = threadIdx.x & 31;
    const int64_t first = w * 8 - 7, slot = first + lane;            // lanes 7 .. 14 are the window, 22 the last slot of its run
    const int32_t id = lane < 23 && slot >= 0 && slot < p.n_tokens ? p.tok_id[slot] : -1;
    Window r;
    r.run = -1;
    if (!grads) {
        r.loose = (__ballot_sync(kFull, id >= 0) >> 7) & 0xffu;
        return r;
    }
    const int32_t before = __shfl_up_sync(kFull, id, 1);
    const uint32_t begins = __ballot_sync(kFull, id >= 0 && (id & 7) == 0 && int64_t(id) + 8 <= p.ws.n);
    const uint32_t follows = __ballot_sync(kFull, lane > 0 && id > 0 && (id & 7) != 0 && id == before + 1);
    // run from lane s: begins at s and follows at s + 1 .. s + 7
    const int s = lane - (id & 7);
    const bool whole = id >= 0 && s >= 0 && s + 7 < 23 && ((begins >> s) & 1) && ((follows >> (s + 1)) & 0x7f) == 0x7f;
    const uint32_t starts = __ballot_sync(kFull, whole && (id & 7) == 0) & 0x7f80u;
    r.loose = (__ballot_sync(kFull, id >= 0 && !whole) >> 7) & 0xffu;
    if (starts) r.run = first + (__ffs(starts) - 1);
    return r;
}

template <class E, bool INTER, bool WIDE, bool GRADS>
__global__ void __launch_bounds__(kQkWarps * 32) qk_bwd_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ float4 shared[];
    const int lane32 = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t unit = blockIdx.x * kQkWarps + warp;
    if (unit >= p.units) return;
    const uint32_t win = p.by_chunks.quotient(unit);
    const int chunk_all = int(unit - win * uint32_t(p.chunks));
    const HeadsParams &h = p.side[chunk_all >= p.chunks_q];
    const int chunk = chunk_all >= p.chunks_q ? chunk_all - p.chunks_q : chunk_all;
    const bool grads = GRADS && qk_header_ok(p.ws);
    if (GRADS && !grads && unit == 0 && lane32 == 0) qk_report(p.ws, kStHeader);
    const Window wd = window_of(p, win, grads);

    const int lane = lane32 & (p.team - 1), team = lane32 / p.team, teams = 32 / p.team;
    const LaneColumns<INTER, WIDE> col = lane_columns<INTER, WIDE>(lane, p.D, p.rot, p.first, false);
    const int head0 = chunk * h.per;
    int heads = h.heads - head0;
    if (heads > h.per) heads = h.per;
    f2_t w[8];
    lane_weights<E, INTER, WIDE>(h.w, p.params_f32, col, w);
    float *sums = reinterpret_cast<float *>(shared) + size_t(warp) * kQkGroup * p.D;   // [8][D] of the run's tokens

    const int loose = __popc(wd.loose), in_run = wd.run >= 0 ? 8 : 0;
    // the run's tokens first, then the loose ones
    for (int t0 = 0; t0 < in_run + loose; t0 = t0 < in_run && t0 + teams >= in_run ? in_run : t0 + teams) {
        const int t = t0 + team, end = t0 < in_run ? in_run : in_run + loose;
        const bool on = t < end;
        int64_t slot = 0;
        if (t < in_run) {
            slot = wd.run + t;
        } else if (on) {                                 // the (t - in_run)th loose slot
            uint32_t m = wd.loose;
            for (int i = t - in_run; i > 0; --i) m &= m - 1;
            slot = int64_t(win) * 8 + (__ffs(m) - 1);
        }
        f2_t c[4], s[4], acc[8];
        lane_angles(p, on ? p.position[slot] : 0, lane, col.turned, c, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = f2_make(0.f, 0.f);
        int64_t in = slot * h.in_t + head0 * h.in_h, dyo = slot * h.dy_t + head0 * h.dy_h, out = slot * h.out_t + head0 * h.out_h;
        Raw<E> rx, rg;
        load_lane<E, INTER, WIDE>(rx, h.in, in, col, on);
        load_lane<E, INTER, WIDE>(rg, h.dy, dyo, col, on);
        for (int i = 0; i < heads; ++i) {
            f2_t x[8], g[8], a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = up2<E>(rx, j);
                g[j] = up2<E>(rg, j);
            }
            in += h.in_h;
            dyo += h.dy_h;
            if (i + 1 < heads) {
                load_lane<E, INTER, WIDE>(rx, h.in, in, col, on);
                load_lane<E, INTER, WIDE>(rg, h.dy, dyo, col, on);
            }
            turn_lane<INTER>(g, c, s, col.turned);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = f2_mul(g[j], w[j]);
            const float ss = team_add(lane_dot(x, x), p.team), sa = team_add(lane_dot(a, x), p.team);
            const float rstd = qk_rstd(ss, p), m = row_mean_gxhat(sa, rstd, float(p.D), p.inv_d);
            Raw<E> y;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = f2_mul(x[j], f2_both(rstd));
                if constexpr (GRADS) acc[j] = f2_fma(g[j], x[j], acc[j]);
                down2<E>(y, j, f2_mul(f2_fma(x[j], f2_both(-m), a[j]), f2_both(rstd)));
            }
            if (on) store_lane<E, INTER, WIDE>(y, h.out, out, col);
            out += h.out_h;
        }
        if (GRADS && grads && on) {
            const int32_t id = p.tok_id[slot];
            float *dst = sums + (t & 7) * p.D;
            bool keep = true;
            if (t >= in_run) {
                keep = int64_t(id) < p.ws.n;
                dst = p.ws.spill + (int64_t(chunk_all) * p.ws.n + id) * p.D;
                if (chunk_all == 0 && lane == 0) {
                    const int bad = keep ? (atomicExch(p.ws.flag + id, 2) ? kStDouble : 0) : kStPlan;
                    if (bad) qk_report(p.ws, bad);
                }
            } else if (chunk_all == 0 && lane == 0 && atomicExch(p.ws.flag + id, 1)) {
                qk_report(p.ws, kStDouble);
            }
            if (keep) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = WIDE ? col.at[j >> 2] : col.at[j];
                    if (at >= 0)
                        *reinterpret_cast<float2 *>(dst + (WIDE ? at + 2 * (j & 3) : at)) = make_float2(f2_lo(acc[j]), f2_hi(acc[j]));
                }
            }
        }
    }
    if (GRADS && grads && in_run) {
        __syncwarp();
        const int64_t g = p.tok_id[wd.run] >> 3;
        float *dst = p.ws.partial + (int64_t(chunk_all) * p.ws.groups + g) * p.D;
        for (int k = lane32 * 4; k < p.D; k += 128) {
            float4 v = *reinterpret_cast<const float4 *>(sums + k);
#pragma unroll
            for (int t = 1; t < kQkGroup; ++t) {
                const float4 u = *reinterpret_cast<const float4 *>(sums + t * p.D + k);
                v = make_float4(__fadd_rn(v.x, u.x), __fadd_rn(v.y, u.y), __fadd_rn(v.z, u.z), __fadd_rn(v.w, u.w));
            }
            *reinterpret_cast<float4 *>(dst + k) = v;
        }
    }
}

// Launches the rows of one call for element type E (rotary_*.cu instantiate it).
// mode: 0 rotation alone, 1 norm and rotation, 2 their backward pass, 3 with weight gradients.
template <class E>
int rotary_run(RotaryParams p, int mode, bool interleaved, cudaStream_t stream);

}  // namespace rbi
