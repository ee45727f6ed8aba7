// Rotary positions of queries and keys, alone and behind an RMS norm of every
// head, and their backward pass (sm_103a): what the kernels share, and the row
// kernels.
//
// A head is held by a team of lanes, 16 columns a lane: two vectors of 8, those that turn
// into each other where the halves of the rotation are made of whole vectors (neighbouring
// pairs lie inside a vector anyway), or, halves of other sizes, pieces of four or two
// columns, as many and their partners.  So the rotation needs no exchange between lanes.
// A team stays with one token and walks over a chunk of its heads, queries and keys
// alike, so the lane's cosines and sines are formed once per chunk.
//
// What bounds it (bf16, 32+8 heads of 128, 33,384 tokens; DRAM floor at the copy rate of
// 6.78 TB/s in brackets): memory.  Rotation 100.2 us (100.9), norm and rotation 105 (100.9),
// backward 156 and, with both weight gradients from begin to finalize, 167 (151.4).  FP32,
// 17,620 tokens: 117, 114 (106.5), 191 (159.8).  Fewer rows for a token's angles and a
// warp's start, or idle lanes, make it issue: 1+1 heads of 128, 270,100 tokens, 51 and 64
// (41.1), backward 152 (61.5); heads of 80, backward, 126 (94.6).  Pieces
// pay for their way through shared memory, about 60 instructions a row of a warp more: 16+16
// heads of 72 that turn whole, 17,620 tokens, 32 and 37 (24.0), backward 64 (36.0); 32+8 heads of
// 120, 57 and 59 (49.9), 104 (74.9).  (Vectors that take each partner's value from where its
// lane's copy arrived, with two factors a column: 45, 49, 92; 80, 83, 141.)
#pragma once
#include <type_traits>

#include "host.cuh"
#include "layernorm_narrow.cuh"
#include "rotary_bi.h"

namespace rbi {

constexpr int kChunkHeads = 8;                           // most heads of a warp of the rotation alone; QkGroups reckons with chunks of as many
constexpr int kMostGroup = 10;                           // most logical tokens of a group of the weight gradients' order
constexpr int kBusyWarps = 2432;                         // warps that fill the GPU: 16 on each of 152 SMs
constexpr uint64_t kQkMagic = 0x3149422d4b514e52ull;

// How a warp takes heads of D columns: in teams of as many lanes as hold them, or of the
// power of two above where that makes no fewer teams.
struct QkTeams {
    int size, teams;
    explicit QkTeams(int D) {
        const int lanes = (D + 15) / 16;
        size = 1;
        while (size < lanes) size <<= 1;
        if (32 / lanes > 32 / size) size = lanes;
        teams = 32 / size;
    }
};

// The logical tokens of a group, the unit that a warp of the backward pass adds up, by the sizes
// (tokens, heads, D) alone: as many as a warp has teams, or, fewer than 5 teams, a multiple up to
// 8: each team takes a share of consecutive tokens, from the first to the last, then
// the shares are added likewise.  The multiple is halved while the groups' chunks of heads
// are too few for a round and a half of warps, the chunks taken to be of 8 heads (644 tokens of 60 heads of 192: 41 us
// in groups of 8, 32 of 4, 27 of 2; 17,620 of 17 of 256, permuted: 97, 95, 103).  More than 10 teams (heads up to 32
// columns) have groups of 8.
struct QkGroups {
    int group, share;
    int64_t groups;
    QkGroups(int D, int32_t heads, int64_t tokens) {
        const int teams = QkTeams(D).teams;
        group = teams > kMostGroup ? 8 : teams >= 5 ? teams : 8 / teams * teams;
        while (group / 2 >= teams && group > 2 && (tokens + group - 1) / group * ((heads + kChunkHeads - 1) / kChunkHeads) <= kBusyWarps * 3 / 2)
            group /= 2;
        share = teams >= group ? 1 : group / teams;
        groups = (tokens + group - 1) / group;
    }
};

// The backward pass cuts a token's heads, queries then keys, into chunks of equal size
// (the last one shorter), by the sizes alone: of up to 16 heads, those with which the
// warps' rounds take least if a token's angles and a warp's start take as long as two rows
// each (17,620 tokens of 16+16 heads of 72: 72 us in chunks of 8, 63 of 16; 33,384 of 32+8 of 128: 167 of 10, 168
// of 8, 171 of 14; 46 of 4+2 of 16: 8.6 of 6, 5.1 of 2).  A chunk that holds both
// kinds has a partial sum of each: slots of the queries' chunks come first, then those of the chunks
// that hold keys.
struct QkChunks {
    int32_t chunks, per;             // chunks of a token, heads of a chunk
    int32_t q_slots, k_first, slots; // chunks with queries; first chunk with keys; all partial sums
    QkChunks() = default;
    QkChunks(int32_t hq, int32_t hk, int64_t groups, int share) {
        const int32_t all = hq + hk;
        int64_t best = INT64_MAX;
        int n = 2;
        for (const int most : {16, 12, 8, 6, 4, 3, 2}) {
            const int64_t c = (all + most - 1) / most, rows = (all + c - 1) / c;
            const int64_t time = (groups * c + kBusyWarps - 1) / kBusyWarps * (share * (rows + 2) + 2);
            if (time < best) {
                best = time;
                n = most;
            }
        }
        chunks = (all + n - 1) / n;
        per = (all + chunks - 1) / chunks;
        q_slots = (hq + per - 1) / per;
        k_first = hq / per;
        slots = q_slots + (hk ? chunks - k_first : 0);
    }
};

struct QkWs {
    WsHeader *hdr;                   // n_rows tokens; hidden = the sizes (qk_sizes)
    int32_t *flag;                   // [N] 0 nothing, 1 in its group's partial, 2 its own sums stored
    int32_t *whole;                  // [groups] 1: the group's partial is there
    float *partial;                  // [slots][groups][D]
    float *spill;                    // [slots][N][D]: a token's sums
    int64_t n, groups, sizes;
    QkChunks cut;
    int32_t D, group, share;
};

inline int64_t qk_sizes(int64_t D, int32_t hq, int32_t hk) { return D | int64_t(hq) << 16 | int64_t(hk) << 32; }

struct QkWsLayout {
    int64_t off_whole, off_partial, off_spill, total;
    QkWsLayout(int64_t N, int32_t hq, int32_t hk, int64_t D) {
        const QkGroups t(int(D), hq + hk, N);
        const int64_t groups = t.groups, slots = QkChunks(hq, hk, groups, t.share).slots;
        off_whole = align256(256 + N * 4);
        off_partial = align256(off_whole + groups * 4);
        off_spill = align256(off_partial + slots * groups * D * 4);
        total = align256(off_spill + slots * N * D * 4);
    }
};

inline QkWs qk_ws(void *base, int64_t N, int32_t hq, int32_t hk, int64_t D) {
    const QkWsLayout L(N, hq, hk, D);
    uint8_t *b = static_cast<uint8_t *>(base);
    QkWs w;
    w.hdr = reinterpret_cast<WsHeader *>(b);
    w.flag = reinterpret_cast<int32_t *>(b + 256);
    w.whole = reinterpret_cast<int32_t *>(b + L.off_whole);
    w.partial = reinterpret_cast<float *>(b + L.off_partial);
    w.spill = reinterpret_cast<float *>(b + L.off_spill);
    w.n = N;
    const QkGroups t(int(D), hq + hk, N);
    w.group = t.group;
    w.share = t.share;
    w.groups = t.groups;
    w.sizes = qk_sizes(D, hq, hk);
    w.cut = QkChunks(hq, hk, w.groups, w.share);
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
};

struct RotaryParams {
    HeadsParams side[2];             // queries, keys
    const int32_t *tok_id, *position;
    const uint64_t *turns;
    int64_t n_tokens, active;        // slots; tokens that may be among them
    int32_t D, rot, first;
    int32_t hq, heads;               // query heads, heads of both
    int32_t chunks, per;             // chunks of a token, heads of a chunk
    int32_t lanes, team, teams;      // lanes of a head that hold columns; lanes of a team; a warp's teams
    int32_t group, share;            // backward: tokens of a group, of a team's share of it
    int32_t params_f32, in_place;    // in_place: columns outside the rotation are already where they belong
    // in pieces: vectors that come and go; bytes between teams' places; pieces of a lane (and their partners) that may
    // turn; 1: all columns are taken as pieces (with the norm)
    int32_t vector0, vectors, pitch, turning, all_pieces;
    uint32_t units;                  // warps' pieces of work
    float scale, scale_sin;          // factors of cosine and sine (negative: turns back)
    float eps, inv_d;
    Divisor by_chunks{1}, by_team{1}, by_teams{1}, by_group{1};
    QkWs ws;
};

// ----------------------------------------------------------------- a lane's columns

// Which columns turn into each other.  kHalf: halves made of whole vectors; kNear:
// neighbouring columns; kQuad: halves that begin and end on multiples of 4 columns (whole
// heads of 72, 88, 120); kSplit: others.
enum { kHalf = 0, kNear = 1, kQuad = 2, kSplit = 3 };
__host__ __device__ constexpr bool in_pieces(int pairs) { return pairs >= kQuad; }
// Register pairs (of columns) of a piece.
__host__ __device__ constexpr int piece_pairs(int pairs) { return pairs == kQuad ? 2 : 1; }

struct VectorColumns {
    int32_t at[2];                   // first columns of the lane's vectors, -1: none
    uint32_t turned;                 // bit i: register pair i (0..3 first vector, 4..7 second) turns
};
// In pieces: those of the second half of the list are what the first turn into.  Rows come and
// go as vectors of 8 columns like the others', through a place of the team's in shared memory,
// where lanes next to each other take pieces next to each other.  Pieces that do not
// turn are not taken by the rotation alone.
template <int PAIRS>
struct PieceColumns {
    static constexpr int kPairs = piece_pairs(PAIRS), kPieces = 8 / kPairs, kHalf = kPieces / 2;
    int32_t at[kPieces];             // first columns of the pieces, -1: none
    int32_t vector[2];               // vectors that the lane brings and stores, -1: none
    uint32_t turned;                 // as above
};
template <int PAIRS>
using LaneColumns = std::conditional_t<in_pieces(PAIRS), PieceColumns<PAIRS>, VectorColumns>;

template <int PAIRS>
__device__ __forceinline__ LaneColumns<PAIRS> lane_columns(int lane, int size, const RotaryParams &p) {
    LaneColumns<PAIRS> c;
    const int rest = p.D - p.rot;
    if constexpr (in_pieces(PAIRS)) {
        using C = PieceColumns<PAIRS>;
        constexpr int kPiece = 2 * C::kPairs;            // columns
        const int turning = p.rot / (2 * kPiece), others = p.all_pieces ? rest / (2 * kPiece) : 0;
        c.turned = 0;
#pragma unroll
        for (int j = 0; j < C::kHalf; ++j) {
            const int k = j * size + lane, o = kPiece * (k - turning), o2 = o + (rest >> 1);
            if (k < turning) {
                c.at[j] = p.first + kPiece * k;
                c.at[C::kHalf + j] = c.at[j] + (p.rot >> 1);
                c.turned |= (C::kPairs == 2 ? 0x33u : 0x11u) << (j * C::kPairs);
            } else {
                const bool there = k < turning + others;
                c.at[j] = !there ? -1 : o < p.first ? o : o + p.rot;
                c.at[C::kHalf + j] = !there ? -1 : o2 < p.first ? o2 : o2 + p.rot;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) c.vector[j] = lane + j * size < p.vectors ? p.vector0 + lane + j * size : -1;
    } else if constexpr (PAIRS == kHalf) {
        // first the lanes of the rotation, then those of the other columns
        const int e = 16 * lane - p.rot;
        c.turned = e < 0 ? 0xffu : 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = e + 8 * i;                     // column among those outside
            c.at[i] = e < 0 ? p.first + 8 * lane + i * (p.rot >> 1) : o < rest && !p.in_place ? (o < p.first ? o : o + p.rot) : -1;
        }
    } else {
        c.turned = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c.at[i] = 8 * (lane + i * p.lanes);
            if (lane >= p.lanes || c.at[i] >= p.D) c.at[i] = -1;
            uint32_t t = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = c.at[i] + 2 * j - p.first;
                if (c.at[i] >= 0 && k >= 0 && k < p.rot) t |= 1u << j;
            }
            if (p.in_place && !t) c.at[i] = -1;
            c.turned |= t << (4 * i);
        }
    }
    return c;
}

template <int PAIRS>
__device__ __forceinline__ LaneColumns<PAIRS> no_columns() {
    LaneColumns<PAIRS> c;
    for (int32_t &at : c.at) at = -1;
    if constexpr (in_pieces(PAIRS)) c.vector[0] = c.vector[1] = -1;
    c.turned = 0;
    return c;
}

// The lane's 16 elements as they are in memory.
template <class E>
struct Raw {
    static constexpr int kQ = int(sizeof(E)) / 2;        // 16-byte words of a vector
    uint4 q[2 * kQ];
};

// 8 FP32 elements (32-byte aligned) at once if `on`, else zeros.
__device__ __forceinline__ void load_f32x8(uint4 *q, const float *p, bool on) {
    q[0] = q[1] = make_uint4(0, 0, 0, 0);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
                 "@p ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t}"
                 : "+r"(q[0].x), "+r"(q[0].y), "+r"(q[0].z), "+r"(q[0].w), "+r"(q[1].x), "+r"(q[1].y), "+r"(q[1].z), "+r"(q[1].w)
                 : "l"(p), "r"(uint32_t(on)));
}
template <class E>
__device__ __forceinline__ void store_vector(void *p, const uint4 *q) {
    if constexpr (sizeof(E) == 4) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(q[0].x), "r"(q[0].y), "r"(q[0].z), "r"(q[0].w),
                     "r"(q[1].x), "r"(q[1].y), "r"(q[1].z), "r"(q[1].w)
                     : "memory");
    } else {
        st_global_v4(p, q[0]);
    }
}

template <class E>
__device__ __forceinline__ f2_t up2(const Raw<E> &r, int i) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(r.q);
    if constexpr (sizeof(E) == 4) {
        return f2_make(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (std::is_same_v<E, __half>) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        return f2_make(p.x, p.y);
    } else {
        return f2_from_bf16x2(w[i]);
    }
}
template <class E>
__device__ __forceinline__ void down2(Raw<E> &r, int i, f2_t v) {
    uint32_t *w = reinterpret_cast<uint32_t *>(r.q);
    if constexpr (sizeof(E) == 4) {
        w[2 * i] = __float_as_uint(f2_lo(v));
        w[2 * i + 1] = __float_as_uint(f2_hi(v));
    } else if constexpr (std::is_same_v<E, __half>) {
        const __half2 h = __floats2half2_rn(f2_lo(v), f2_hi(v));
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        w[i] = f2_to_bf16x2(v);
    }
}

// Both weights in shared memory, as FP32 and in the lanes' order: four columns of a team's
// lane at [side][quad][lane], 32 lanes apart, so that a lane's reads need one address.
constexpr int kWeightBytes = 2 * 4 * 32 * 16;
template <class E>
__device__ __forceinline__ f2_t two_params(const void *w, int f32, int at) {
    if (!w) return f2_both(1.f);
    Raw<E> r;
    if constexpr (sizeof(E) == 2)
        if (!f32) {
            r.q[0].x = *reinterpret_cast<const uint32_t *>(static_cast<const E *>(w) + at);
            return up2<E>(r, 0);
        }
    const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(w) + at);
    return f2_make(v.x, v.y);
}
template <class E, int PAIRS>
__device__ __forceinline__ void stage_weights(float4 *sw, const RotaryParams &p, int size) {
    const int i = threadIdx.x, side = i >= 2 * size, lane = (i - side * 2 * size) >> 1, j = i & 1;
    if (i >= 4 * size) return;                           // (a CTA has at least 128 threads)
    const LaneColumns<PAIRS> col = lane_columns<PAIRS>(lane, size, p);
    f2_t f[4] = {0, 0, 0, 0};                            // (columns that are not there: zeros, they enter sums)
    if constexpr (in_pieces(PAIRS)) {
        using C = PieceColumns<PAIRS>;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const int at = j ? col.at[C::kHalf + l / C::kPairs] : col.at[l / C::kPairs];
            if (at >= 0) f[l] = two_params<E>(p.side[side].w, p.params_f32, at + 2 * (l % C::kPairs));
        }
    } else {
        const int at = col.at[j];
        if (at >= 0) oct_param<E>(p.side[side].w, p.params_f32, at >> 3, 1.f, f);
    }
    float4 *to = sw + (side * 4 + 2 * j) * 32 + lane;
    to[0] = make_float4(f2_lo(f[0]), f2_hi(f[0]), f2_lo(f[1]), f2_hi(f[1]));
    to[32] = make_float4(f2_lo(f[2]), f2_hi(f[2]), f2_lo(f[3]), f2_hi(f[3]));
}
// `from`: shared-memory address of the lane's first quad of the side.
__device__ __forceinline__ void lane_weights(uint32_t from, f2_t (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(f[2 * i]), "=l"(f[2 * i + 1]) : "r"(from + i * 512));
}

// ----------------------------------------------------------------- angles

// Cosine and sine of position * turns / 2^64 turns.  The product modulo 2^64 is exact;
// its top 32 bits, off by less than 2^-32 turn, are a quadrant and a rest of at most
// 1/8 turn either way, y = rest in radians.  sin y and cos y are their Taylor polynomials
// of degree 9 and 10: what is left out is below (pi/4)^11 / 11! = 1.8e-9 and
// (pi/4)^12 / 12! = 1.2e-10.  FINE (FP32 heads): y is formed with what the float of the
// rest loses, and enters as y + d: sin + d cos, cos - d sin.  In units of 2^-24, over all
// 2^30 rests, sine and cosine are off by at most 1.16 and 1.38, without FINE 1.52 and 1.71.  (One pair at a time: constants are operands of its
// instructions, in registers of two they are moves.  1+1 heads of 128, 270,100 tokens, with
// the norm: 70 -> 67 us.)
template <bool FINE>
__device__ __forceinline__ void cos_sin(int32_t position, uint64_t turns, float &c, float &s) {
    const uint32_t top = uint32_t(uint64_t(int64_t(position)) * turns >> 32);
    const int32_t rest = int32_t(top << 2);              // 4 times the rest: the quadrant has gone
    const float f = __int2float_rn(rest);
    const float kHi = 0x1.921fb6p-32f, kLo = -0x1.777a5cp-57f;       // 2 pi / 2^34 in two floats
    const float y = __fmul_rn(f, kHi), z = __fmul_rn(y, y);
    float p = __fmaf_rn(z, 1.f / 362880.f, -1.f / 5040.f);
    p = __fmaf_rn(z, p, 1.f / 120.f);
    p = __fmaf_rn(z, p, -1.f / 6.f);
    float sn = __fmaf_rn(__fmul_rn(z, y), p, y);
    float q = __fmaf_rn(z, -1.f / 3628800.f, 1.f / 40320.f);
    q = __fmaf_rn(z, q, -1.f / 720.f);
    q = __fmaf_rn(z, q, 1.f / 24.f);
    q = __fmaf_rn(z, q, -0.5f);
    float cs = __fmaf_rn(z, q, 1.f);
    if constexpr (FINE) {
        // (the float of the rest may be 2^31, beyond an int32)
        const float lost = __ll2float_rn(int64_t(rest) - __float2ll_rn(f));
        const float d = __fmaf_rn(lost, kHi, __fmaf_rn(f, kLo, __fmaf_rn(f, kHi, -y)));
        const float sn1 = __fmaf_rn(d, cs, sn);
        cs = __fmaf_rn(-d, sn, cs);
        sn = sn1;
    }
    // quadrants 1 to 3: (cos, sin) = (-sin, cos), (-cos, -sin), (sin, -cos)
    const uint32_t turned = top + 0x20000000u;           // quadrant in the top two bits
    const bool swap = turned & 0x40000000u;
    c = __uint_as_float(__float_as_uint(swap ? sn : cs) ^ ((turned + 0x40000000u) & 0x80000000u));
    s = __uint_as_float(__float_as_uint(swap ? cs : sn) ^ (turned & 0x80000000u));
}

// The lane's cosines and sines, times scale: kHalf of its 8 pairs in columns' order,
// kNear likewise, 4 pairs a vector; in pieces those of their columns.
struct Angles {
    f2_t c[4], s[4];
};
template <class E, int PAIRS>
__device__ __forceinline__ void lane_angles(const RotaryParams &p, int32_t position, int lane, int size, const LaneColumns<PAIRS> &col,
                                            Angles &a) {
    constexpr int kW = piece_pairs(PAIRS);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float c[2] = {1.f, 1.f}, s[2] = {0.f, 0.f};
        if constexpr (PAIRS == kNear) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 2 * i + j;                 // the register pair
                if ((col.turned >> r) & 1)
                    cos_sin<sizeof(E) == 4>(position, p.turns[(col.at[r >> 2] + 2 * (r & 3) - p.first) >> 1], c[j], s[j]);
            }
        } else if (PAIRS == kHalf ? col.turned != 0 : i / kW < p.turning && ((col.turned >> i) & 1)) {
            const ulonglong2 t = reinterpret_cast<const ulonglong2 *>(p.turns)[PAIRS == kHalf ? 4 * lane + i : (i / kW * size + lane) * kW + i % kW];
            cos_sin<sizeof(E) == 4>(position, t.x, c[0], s[0]);
            cos_sin<sizeof(E) == 4>(position, t.y, c[1], s[1]);
        }
        a.c[i] = f2_make(__fmul_rn(c[0], p.scale), __fmul_rn(c[1], p.scale));
        a.s[i] = f2_make(__fmul_rn(s[0], p.scale_sin), __fmul_rn(s[1], p.scale_sin));
    }
}

// Turns the lane's columns.
template <int PAIRS, bool ALL>
__device__ __forceinline__ void turn_lane(f2_t (&f)[8], const Angles &a, const LaneColumns<PAIRS> &col, const RotaryParams &p) {
    if constexpr (in_pieces(PAIRS)) {
        // (pieces that do not turn have partners that do not either: they keep their values, not times 1 plus times 0, which
        // an infinity would spoil; a lane's pieces that are not there may become anything but are not stored)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i / piece_pairs(PAIRS) >= p.turning) continue;
            const f2_t x = f[i], y = f[4 + i], n = f2_mul(a.s[i], f2_both(-1.f));
            const f2_t u = f2_fma(x, a.c[i], f2_mul(y, n)), v = f2_fma(y, a.c[i], f2_mul(x, a.s[i]));
            const bool turns = !ALL || ((col.turned >> i) & 1);
            f[i] = turns ? u : x;
            f[4 + i] = turns ? v : y;
        }
    } else if constexpr (PAIRS == kHalf) {
        if (col.turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2_t x = f[i], y = f[4 + i], n = f2_mul(a.s[i], f2_both(-1.f));
                f[i] = f2_fma(x, a.c[i], f2_mul(y, n));
                f[4 + i] = f2_fma(y, a.c[i], f2_mul(x, a.s[i]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = f2_lo(f[i]), y = f2_hi(f[i]);
            const float c = i & 1 ? f2_hi(a.c[i >> 1]) : f2_lo(a.c[i >> 1]), s = i & 1 ? f2_hi(a.s[i >> 1]) : f2_lo(a.s[i >> 1]);
            if ((col.turned >> i) & 1) f[i] = f2_make(__fmaf_rn(x, c, -__fmul_rn(y, s)), __fmaf_rn(y, c, __fmul_rn(x, s)));
        }
    }
}

// Register pair i holds rotated columns.
template <int PAIRS>
__device__ __forceinline__ bool is_turned(int i, const LaneColumns<PAIRS> &col) {
    return PAIRS == kHalf ? col.turned != 0 : (col.turned >> i) & 1;
}

// Sum over the lanes of a team, those furthest apart first.  TEAM 0: of `team` lanes,
// known when the kernel runs.  Teams of a power of two exchange both ways; others fold
// into their first lane, which hands the sum out.
template <int TEAM>
__device__ __forceinline__ float team_add(float v, int team, int lane) {
    if constexpr (TEAM > 0 && (TEAM & (TEAM - 1)) == 0) {
#pragma unroll
        for (int o = TEAM / 2; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
        return v;
    } else {
        int n = TEAM ? TEAM : team;
#pragma unroll
        for (int o = TEAM ? 4 : 16; o >= 1; o >>= 1) {
            if (o < n) {                                 // lanes 0 .. n - 1 hold sums; the first o (or n - o) add
                const float u = __shfl_down_sync(kFull, v, o);
                if (lane + o < n) v = __fadd_rn(v, u);
                n = o;
            }
        }
        return __shfl_sync(kFull, v, (threadIdx.x & 31) - lane);
    }
}

// A lane's part of a row's sum of products f g (columns that are not there are zeros):
// register pairs of each vector by FMA, the two vectors, the two columns.
__device__ __forceinline__ float lane_dot(const f2_t (&f)[8], const f2_t (&g)[8]) {
    f2_t a = f2_mul(f[0], g[0]), b = f2_mul(f[4], g[4]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        a = f2_fma(f[i], g[i], a);
        b = f2_fma(f[4 + i], g[4 + i], b);
    }
    a = f2_add(a, b);
    return __fadd_rn(f2_lo(a), f2_hi(a));
}

// 1 / sqrt(ss / D + eps): the function's value and one step of Newton's iteration
// (where that is a number: 0 and infinity keep the function's infinity and 0).
__device__ __forceinline__ float qk_rstd(float ss, const RotaryParams &p) {
    const float v = __fmaf_rn(ss, p.inv_d, p.eps), r = rsqrtf(v);
    const float e = __fmaf_rn(-__fmul_rn(v, r), r, 1.f);
    return e == e ? __fmaf_rn(__fmul_rn(0.5f, r), e, r) : r;
}

// ----------------------------------------------------------------- rows on their way

constexpr int kQkWarps = 4;

// 16-bit heads come through shared memory: a ring of kDepth rows a team, every lane
// copying its own columns of TENSORS tensors to places that only it reads (in pieces: its
// vectors, to the team's place).  FP32 rows
// are twice as long and stay in registers, one row ahead, by loads of 32 bytes a lane
// (17,620 tokens, 32+8 heads of 128: forward 117 us against 175 through a ring, backward 192
// against 269; two rows ahead: equal; in pieces they go to the team's place from there).
// Depths measured (bf16): forward 4, 5, 6, 8 rows, heads
// of 80, 33,384 tokens: 75, 75, 77.5, 80 us, heads of 64: 58, 56.5, 56.7, 58; backward 3, 4, 5
// rows, heads of 128: 173, 168, 168, 16+1 heads of 256: 101, 100, 111.  In pieces the backward
// pass has 3, so that 16 warps fit.
template <class E, int TENSORS, int PAIRS>
struct Ring {
    static constexpr bool kOn = sizeof(E) == 2;
    static constexpr int kRow = in_pieces(PAIRS) ? 768 * int(sizeof(E)) : 1024;   // bytes of a warp's rows of one tensor
    static constexpr int kDepth = !kOn ? 1 : TENSORS == 1 ? 5 : in_pieces(PAIRS) ? 3 : 4;
    static constexpr int kBytes = kOn || in_pieces(PAIRS) ? TENSORS * kRow * kDepth : 0;   // of a warp
};
// In pieces: the bytes from one team's place to the next, so that the lanes of all teams find
// a piece in different banks: the words of a team's pieces, rounded up to whole vectors, modulo the 32
// banks, or, small teams, any odd number of 16 bytes.  At most 768 elements / teams.  Vectors
// and pieces in words.
inline int pieces_pitch(int vectors, int vector, int size, int teams, int piece) {
    const int words = vectors * vector, apart = (size * piece + 3) & ~3;
    const int far = words + ((apart - words) & 31), most = 96 * vector / teams;
    return 4 * (teams == 1 ? words : size * piece > 4 && far <= most ? far : words | 4);
}
template <class E, int PAIRS>
__device__ __forceinline__ void copy_row(uint32_t dst, const E *row, const LaneColumns<PAIRS> &col, bool on) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (in_pieces(PAIRS)) {
            if (col.vector[j] >= 0) cp_async_zfill(dst + col.vector[j] * 16, row + col.vector[j] * 8, on ? 16 : 0);
        } else {
            cp_async_zfill(dst + j * 512, row + (col.at[j] >= 0 ? col.at[j] : 0), on && col.at[j] >= 0 ? 16 : 0);
        }
    }
}
template <class E, int PAIRS>
__device__ __forceinline__ void load_row(Raw<E> &r, const E *row, const LaneColumns<PAIRS> &col, bool on) {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int at = col.at[j];
            if constexpr (in_pieces(PAIRS)) at = col.vector[j] * 8;
            load_f32x8(r.q + 2 * j, reinterpret_cast<const float *>(row) + at, on && at >= 0);
        }
    }
}
template <class E>
__device__ __forceinline__ void take_row(Raw<E> &r, uint32_t src) {
#pragma unroll
    for (int l = 0; l < 2 * Raw<E>::kQ; ++l) ld_shared_vec(src + l * 512, r.q[l]);
}
// In pieces, `place`: shared-memory address of the team's column 0 (which need not be there).
// FP32 vectors from registers to their place.
__device__ __forceinline__ void st_shared_vec(uint32_t to, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <class E, int PAIRS>
__device__ __forceinline__ void bring_row(const Raw<E> &r, uint32_t place, const LaneColumns<PAIRS> &col) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (col.vector[j] >= 0) {
#pragma unroll
            for (int l = 0; l < Raw<E>::kQ; ++l) st_shared_vec(place + col.vector[j] * 8 * int(sizeof(E)) + l * 16, r.q[2 * j + l]);
        }
}
// ALL: also those that do not turn.
template <class E, int PAIRS, bool ALL>
__device__ __forceinline__ void take_pieces(Raw<E> &r, uint32_t place, const LaneColumns<PAIRS> &col, const RotaryParams &p) {
    using C = PieceColumns<PAIRS>;
    constexpr int kWords = C::kPairs * int(sizeof(E)) / 2;           // of a piece
    uint32_t *w = reinterpret_cast<uint32_t *>(r.q);
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
        uint32_t *v = w + i * kWords;
#pragma unroll
        for (int l = 0; l < kWords; ++l) v[l] = 0;
        if (!ALL && i % C::kHalf >= p.turning) continue;
        if (col.at[i] >= 0) {
            const uint32_t from = place + col.at[i] * int(sizeof(E));
            if constexpr (kWords == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(from) : "memory");
            else if constexpr (kWords == 2) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(from) : "memory");
            else asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(from) : "memory");
        }
    }
}
template <class E, int PAIRS, bool ALL>
__device__ __forceinline__ void put_pieces(const Raw<E> &r, uint32_t place, const LaneColumns<PAIRS> &col, const RotaryParams &p) {
    using C = PieceColumns<PAIRS>;
    constexpr int kWords = C::kPairs * int(sizeof(E)) / 2;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(r.q);
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
        const uint32_t *v = w + i * kWords;
        if (!ALL && i % C::kHalf >= p.turning) continue;
        if (col.at[i] >= 0) {
            const uint32_t to = place + col.at[i] * int(sizeof(E));
            if constexpr (kWords == 1) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(v[0]) : "memory");
            else if constexpr (kWords == 2) asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(v[0]), "r"(v[1]) : "memory");
            else st_shared_vec(to, make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
}
// The lane's columns to memory (in pieces: the team's, by way of its place).
template <class E, int PAIRS, bool ALL>
__device__ __forceinline__ void store_row(E *dst, const Raw<E> &r, uint32_t place, const LaneColumns<PAIRS> &col, const RotaryParams &p, bool on) {
    if constexpr (in_pieces(PAIRS)) {
        put_pieces<E, PAIRS, ALL>(r, place, col, p);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (on && col.vector[j] >= 0) {
                uint4 v[Raw<E>::kQ];
#pragma unroll
                for (int l = 0; l < Raw<E>::kQ; ++l) ld_shared_vec(place + col.vector[j] * 8 * int(sizeof(E)) + l * 16, v[l]);
                store_vector<E>(dst + col.vector[j] * 8, v);
            }
    } else if (on) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (col.at[j] >= 0) store_vector<E>(dst + col.at[j], r.q + j * Raw<E>::kQ);
    }
}

// ----------------------------------------------------------------- forward, and rotation alone

// NORM: behind the norm; else the rotation alone.  A warp takes `slots` consecutive slots
// of a call (at most 32) and one chunk of heads; its teams take the active ones in turns,
// so padding costs a warp nothing but its ids.  CTAs an SM: with 6, the norm's 80 registers
// are as fast on large calls and 0.3 us slower on small ones; FP32 at 4 of 128 registers takes
// 125 us where 5 take 117; in pieces FP32 needs them (16 bits, heads of 120: 74 -> 70 us with 5).
template <class E, int PAIRS, bool NORM>
constexpr int kFwdCtas = in_pieces(PAIRS) ? (sizeof(E) == 4 ? 4 : 5) : sizeof(E) == 4 || NORM ? 5 : 6;
template <class E, int PAIRS, bool NORM, int TEAM>
__global__ void __launch_bounds__(kQkWarps * 32, kFwdCtas<E, PAIRS, NORM>)
    rotary_kernel(const __grid_constant__ RotaryParams p, int slots) {
    extern __shared__ float4 shared[];
    using R = Ring<E, 1, PAIRS>;
    const int lane32 = threadIdx.x & 31, warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0);   // (uniform, for the compiler)
    const uint32_t unit = blockIdx.x * kQkWarps + warp;
    const bool in = unit < p.units;
    const uint32_t win = p.by_chunks.quotient(in ? unit : 0);
    const int64_t first = int64_t(win) * slots;
    const bool mine = in && lane32 < slots && first + lane32 < p.n_tokens;
    const int32_t id = mine ? p.tok_id[first + lane32] : -1, position = mine ? p.position[first + lane32] : 0;
    const int head0 = int((in ? unit : 0) - win * uint32_t(p.chunks)) * p.per, end = p.heads - head0 < p.per ? p.heads : head0 + p.per;
    const uint32_t active = __ballot_sync(kFull, id >= 0);
    const int count = __popc(active);
    const bool dense = active == (count == 32 ? kFull : (1u << count) - 1u);
    const int size = TEAM ? TEAM : p.team, teams = TEAM ? 32 / (TEAM ? TEAM : 1) : p.teams;
    if constexpr (NORM) stage_weights<E, PAIRS>(shared, p, size);
    const int team = TEAM ? lane32 / (TEAM ? TEAM : 1) : int(p.by_team.quotient(lane32)), lane = lane32 - team * size;
    const int steps = int(p.by_teams.quotient(count + teams - 1));
    LaneColumns<PAIRS> col = team < teams ? lane_columns<PAIRS>(lane, size, p) : no_columns<PAIRS>();   // (lanes that are left over)
    const uint32_t ring = smem_addr(shared) + (NORM ? kWeightBytes : 0) + warp * R::kBytes +
                          (in_pieces(PAIRS) ? team * p.pitch - p.vector0 * 8 * int(sizeof(E)) : lane32 * 16);

    // Lane (of the slots' ids) of this team's slot in a step, -1: none.
    auto place = [&](int step) {
        const int t = step * teams + team;
        if (t >= count || team >= teams) return -1;
        if (dense) return t;
        uint32_t m = active;
        for (int i = t; i > 0; --i) m &= m - 1;
        return __ffs(m) - 1;
    };
    int f_step = 0, f_head = head0;
    uint32_t f_dst = ring;
    const E *f_x = nullptr;
    bool f_on = false;
    Raw<E> next;
    auto fetch = [&]() {
        if (f_step < steps) {
            const bool keys = f_head >= p.hq;
            const HeadsParams &s = p.side[keys];
            if (f_head == head0 || f_head == p.hq) {
                const int at = place(f_step);
                f_on = at >= 0;
                f_x = static_cast<const E *>(s.in) + ((f_on ? first + at : 0) * s.in_t + (keys ? f_head - p.hq : f_head) * s.in_h);
            }
            if constexpr (R::kOn) {
                copy_row<E, PAIRS>(f_dst, f_x, col, f_on);
                f_dst += R::kRow;
                if (f_dst == ring + R::kBytes) f_dst = ring;
            } else {
                load_row<E, PAIRS>(next, f_x, col, f_on);
            }
            f_x += s.in_h;
            if (++f_head == end) {
                f_head = head0;
                ++f_step;
            }
        }
        if constexpr (R::kOn) cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < (R::kOn ? R::kDepth - 1 : 1); ++i) fetch();
    if constexpr (NORM) __syncthreads();                 // the weights

    Angles a;
    uint32_t from = ring;
    for (int step = 0; step < steps; ++step) {
        const int at = place(step);
        const bool on = at >= 0;
        lane_angles<E, PAIRS>(p, __shfl_sync(kFull, position, on ? at : 0), lane, size, col, a);
        for (int h = head0; h < end;) {                  // the token's heads of one kind after the other
            const bool keys = h >= p.hq;
            const int stop = keys || end < p.hq ? end : p.hq;
            const HeadsParams &s = p.side[keys];
            E *dst = static_cast<E *>(s.out) + ((on ? first + at : 0) * s.out_t + (keys ? h - p.hq : h) * s.out_h);
            const uint32_t weights = smem_addr(shared) + keys * (kWeightBytes / 2) + lane * 16;
            for (; h < stop; ++h) {
                Raw<E> r;
                uint32_t place_of = ring;                // in pieces: where the row is
                if constexpr (R::kOn) {
                    cp_async_wait<R::kDepth - 2>();
                    if constexpr (in_pieces(PAIRS)) __syncwarp();     // everyone's; and the row before has been read
                    fetch();
                    if constexpr (in_pieces(PAIRS)) take_pieces<E, PAIRS, NORM>(r, from, col, p);
                    else take_row<E>(r, from);
                    place_of = from;
                    from += R::kRow;
                    if (from == ring + R::kBytes) from = ring;
                } else if constexpr (in_pieces(PAIRS)) {
                    __syncwarp();                        // the row before has left
                    bring_row<E, PAIRS>(next, ring, col);
                    __syncwarp();
                    fetch();
                    take_pieces<E, PAIRS, NORM>(r, ring, col, p);
                } else {
                    r = next;
                    fetch();
                }
                f2_t f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = up2<E>(r, j);
                f2_t rstd = 0;
                if constexpr (NORM) rstd = f2_both(qk_rstd(team_add<TEAM>(lane_dot(f, f), size, lane), p));
                if constexpr (NORM) {
                    f2_t w[8];
                    lane_weights(weights, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = f2_mul(f2_mul(f[j], rstd), w[j]);
                }
                turn_lane<PAIRS, NORM>(f, a, col, p);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (NORM || in_pieces(PAIRS) || is_turned<PAIRS>(j, col)) down2<E>(r, j, f[j]);
                store_row<E, PAIRS, NORM>(dst, r, place_of, col, p, on);
                dst += s.out_h;
            }
        }
    }
}

// ----------------------------------------------------------------- backward of the norm and the rotation

// What a warp of the backward pass does with the G slots [G w, G w + G) of a call (G the
// tokens of a group) and one chunk of heads: the run, G consecutive slots that hold a whole group in
// logical order and start among them (at most one does), and the active slots that
// belong to no run.  Slots of a run that starts in the window before are that
// window's.  Lanes 0 .. 3 G - 3 hold the ids and positions of slots G w - (G - 1) on.
struct Window {
    int32_t id, position;
    int run;                         // lane of the run's first slot, -1: none
    uint32_t loose;                  // bit j: slot G w + j on its own
};
__device__ __forceinline__ Window window_of(const RotaryParams &p, int64_t w, bool grads) {
    const int lane = threadIdx.x & 31, G = p.group;
    const uint32_t mine = (1u << G) - 1u, behind = mine >> 1;        // the window's slots; the G - 1 that follow a group's first
    const int64_t slot = w * G - (G - 1) + lane;         // lanes G - 1 .. 2 G - 2 are the window
    const bool in = lane < 3 * G - 2 && slot >= 0 && slot < p.n_tokens;
    Window r;
    r.id = in ? p.tok_id[slot] : -1;
    r.position = in ? p.position[slot] : 0;
    r.run = -1;
    if (!grads) {
        r.loose = (__ballot_sync(kFull, r.id >= 0) >> (G - 1)) & mine;
        return r;
    }
    const int32_t before = __shfl_up_sync(kFull, r.id, 1);
    const int nth = r.id < 0 ? 0 : r.id - int(p.by_group.quotient(uint32_t(r.id))) * G;   // of its group
    const uint32_t begins = __ballot_sync(kFull, r.id >= 0 && nth == 0 && int64_t(r.id) + G <= p.ws.n);
    const uint32_t follows = __ballot_sync(kFull, lane > 0 && r.id > 0 && nth != 0 && r.id == before + 1);
    // run from lane s: begins at s and follows at s + 1 .. s + G - 1
    const int s = lane - nth;
    const bool whole = r.id >= 0 && s >= 0 && s + G <= 3 * G - 2 && ((begins >> s) & 1) && ((follows >> (s + 1)) & behind) == behind;
    const uint32_t starts = __ballot_sync(kFull, whole && nth == 0) & (mine << (G - 1));
    r.loose = (__ballot_sync(kFull, r.id >= 0 && !whole) >> (G - 1)) & mine;
    if (starts) r.run = __ffs(starts) - 1;
    return r;
}

inline int qk_bwd_smem(int ring_bytes, bool grads, bool straddles) {
    // both weights, then per warp: ring, the teams' sums (of both kinds where a chunk has both); teams x D floats are at
    // most 2048 bytes
    return kWeightBytes + kQkWarps * (ring_bytes + (grads ? (straddles ? 4096 : 2048) : 0));
}

// The backward pass, for a window and a chunk of heads a warp.  Both row sums of a row (of
// x^2 and of g w x) come from one pass over it; the weight gradients add up in registers
// over a token's heads of one kind, in shared memory over a team's tokens of the run, and
// leave as one partial sum a run.  It holds x, g, g w, a token's angles and the sums: 128
// registers for 16 warps an SM (12 warps at 168 registers: 183 us where 16 take 169; in
// pieces, heads of 72, 82 and 73; FP32, which needs more than 128, has 12).  A few registers spill in two forms:
// neighbours of 16 bits whose team is known only when the kernel runs (16 bytes stored, 28 loaded a thread) and FP32
// pieces of four columns (8 to 12, 12 to 20).  Left on the table: about 330 instructions a warp for 4 rows of 128, of
// which some 20 % are addresses and copies.
// With ws.hdr == NULL there are no gradients: every active slot is one on its own.
template <class E, int PAIRS, int TEAM>
__global__ void __launch_bounds__(kQkWarps * 32, sizeof(E) == 4 ? 3 : 4) qk_bwd_kernel(const __grid_constant__ RotaryParams p, int straddles) {
    extern __shared__ float4 shared[];
    const int lane32 = threadIdx.x & 31, warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0);   // (uniform, for the compiler)
    const uint32_t unit = blockIdx.x * kQkWarps + warp;
    const bool in = unit < p.units;
    const uint32_t win = p.by_chunks.quotient(in ? unit : 0);
    const int chunk = int((in ? unit : 0) - win * uint32_t(p.chunks));
    const bool grads = p.ws.hdr && qk_header_ok(p.ws);
    if (p.ws.hdr && !grads && unit == 0 && lane32 == 0) qk_report(p.ws, kStHeader);
    constexpr int kTeams = TEAM ? 32 / (TEAM ? TEAM : 1) : 1;
    const int size = TEAM ? TEAM : p.team, teams = TEAM ? kTeams : p.teams;
    const int G = p.group, share = p.share;
    Window wd = window_of(p, win, grads);
    if (!in) {
        wd.run = -1;
        wd.loose = 0;
    }

    const int team = TEAM ? lane32 / (TEAM ? TEAM : 1) : int(p.by_team.quotient(lane32)), lane = lane32 - team * size;
    stage_weights<E, PAIRS>(shared, p, size);
    LaneColumns<PAIRS> col = team < teams ? lane_columns<PAIRS>(lane, size, p) : no_columns<PAIRS>();   // (lanes that are left over)
    const int head0 = chunk * p.per, end = p.heads - head0 < p.per ? p.heads : head0 + p.per;
    const int loose = __popc(wd.loose), run_steps = wd.run >= 0 ? share : 0;
    const int steps = run_steps + (TEAM ? (loose + kTeams - 1) / kTeams : int(p.by_teams.quotient(loose + teams - 1)));

    using R = Ring<E, 2, PAIRS>;
    const int sums_bytes = p.ws.hdr ? (straddles ? 4096 : 2048) : 0;
    uint8_t *mine = reinterpret_cast<uint8_t *>(shared) + kWeightBytes + warp * (R::kBytes + sums_bytes);
    const uint32_t ring = smem_addr(mine) + (in_pieces(PAIRS) ? team * p.pitch - p.vector0 * 8 * int(sizeof(E)) : lane32 * 16);
    // [kinds][teams][D]: each team's sums over its share of the run; a lane has its own columns
    float *const sums = reinterpret_cast<float *>(mine + R::kBytes);

    // Lane (of the window's ids) of this team's slot in a step, -1: none.
    auto place = [&](int step) {
        if (team >= teams) return -1;
        if (step < run_steps) return team * share < G ? wd.run + team * share + step : -1;
        const int t = (step - run_steps) * teams + team;
        if (t >= loose) return -1;
        uint32_t m = wd.loose;
        for (int i = t; i > 0; --i) m &= m - 1;
        return G - 2 + __ffs(m);
    };
    // The copies of the next row: one commit a row.  A row's address follows from the
    // one before but for the first of each kind of a token.
    int f_step = 0, f_head = head0;
    uint32_t f_dst = ring;
    const E *f_x = nullptr, *f_g = nullptr;
    bool f_on = false;
    Raw<E> next_x, next_g;
    auto fetch = [&]() {
        if (f_step < steps) {
            const bool keys = f_head >= p.hq;
            const HeadsParams &s = p.side[keys];
            if (f_head == head0 || f_head == p.hq) {
                const int at = place(f_step);
                f_on = at >= 0;
                const int64_t slot = f_on ? int64_t(win) * G - (G - 1) + at : 0;
                const int h = keys ? f_head - p.hq : f_head;
                f_x = static_cast<const E *>(s.in) + (slot * s.in_t + h * s.in_h);
                f_g = static_cast<const E *>(s.dy) + (slot * s.dy_t + h * s.dy_h);
            }
            if constexpr (R::kOn) {
                copy_row<E, PAIRS>(f_dst, f_x, col, f_on);
                copy_row<E, PAIRS>(f_dst + R::kRow, f_g, col, f_on);
                f_dst += 2 * R::kRow;
                if (f_dst == ring + R::kBytes) f_dst = ring;
            } else {
                load_row<E, PAIRS>(next_x, f_x, col, f_on);
                load_row<E, PAIRS>(next_g, f_g, col, f_on);
            }
            f_x += s.in_h;
            f_g += s.dy_h;
            if (++f_head == end) {
                f_head = head0;
                ++f_step;
            }
        }
        if constexpr (R::kOn) cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < (R::kOn ? R::kDepth - 1 : 1); ++i) fetch();
    __syncthreads();                                     // the weights
    if (steps == 0) return;

    Angles a;
    uint32_t from = ring;
    for (int step = 0; step < steps; ++step) {
        const int at = place(step);
        const bool on = at >= 0, run = step < run_steps;
        const int64_t slot = on ? int64_t(win) * G - (G - 1) + at : 0;
        const int32_t id = __shfl_sync(kFull, wd.id, on ? at : 0);
        lane_angles<E, PAIRS>(p, __shfl_sync(kFull, wd.position, on ? at : 0), lane, size, col, a);
        const bool known = int64_t(id) < p.ws.n;
        if (grads && on && chunk == 0 && lane == 0) {
            const int bad = known ? (atomicExch(p.ws.flag + id, run ? 1 : 2) ? kStDouble : 0) : kStPlan;
            if (bad) qk_report(p.ws, bad);
        }
        // the token's heads of one kind after the other
        for (int h = head0; h < end;) {
            const bool keys = h >= p.hq;
            const int stop = keys || end < p.hq ? end : p.hq;
            const HeadsParams &s = p.side[keys];
            E *dst = static_cast<E *>(s.out) + (slot * s.out_t + (keys ? h - p.hq : h) * s.out_h);
            const uint32_t weights = smem_addr(shared) + keys * (kWeightBytes / 2) + lane * 16;
            f2_t acc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = f2_make(0.f, 0.f);
            for (; h < stop; ++h) {
                Raw<E> rx, rg;
                uint32_t place_of = ring;                // in pieces: where the row is
                if constexpr (R::kOn) {
                    cp_async_wait<R::kDepth - 2>();
                    if constexpr (in_pieces(PAIRS)) __syncwarp();
                    fetch();
                    if constexpr (in_pieces(PAIRS)) {
                        take_pieces<E, PAIRS, true>(rx, from, col, p);
                        take_pieces<E, PAIRS, true>(rg, from + R::kRow, col, p);
                    } else {
                        take_row<E>(rx, from);
                        take_row<E>(rg, from + R::kRow);
                    }
                    place_of = from;
                    from += 2 * R::kRow;
                    if (from == ring + R::kBytes) from = ring;
                } else if constexpr (in_pieces(PAIRS)) {
                    __syncwarp();                        // the row before has left
                    bring_row<E, PAIRS>(next_x, ring, col);
                    bring_row<E, PAIRS>(next_g, ring + R::kRow, col);
                    __syncwarp();
                    fetch();
                    take_pieces<E, PAIRS, true>(rx, ring, col, p);
                    take_pieces<E, PAIRS, true>(rg, ring + R::kRow, col, p);
                } else {
                    rx = next_x;
                    rg = next_g;
                    fetch();
                }
                f2_t x[8], g[8], b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = up2<E>(rx, j);
                    g[j] = up2<E>(rg, j);
                }
                turn_lane<PAIRS, true>(g, a, col, p);
                lane_weights(weights, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = f2_mul(g[j], b[j]);
                const float ss = team_add<TEAM>(lane_dot(x, x), size, lane), sb = team_add<TEAM>(lane_dot(b, x), size, lane);
                const float rstd = qk_rstd(ss, p), m = __fmul_rn(__fmul_rn(sb, rstd), p.inv_d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = f2_mul(x[j], f2_both(rstd));
                    acc[j] = f2_fma(g[j], x[j], acc[j]);
                    down2<E>(rx, j, f2_mul(f2_fma(x[j], f2_both(-m), b[j]), f2_both(rstd)));
                }
                store_row<E, PAIRS, true>(dst, rx, place_of, col, p, on);
                dst += s.out_h;
            }
            if (grads && on && (run || known)) {
                const int64_t part = keys ? p.ws.cut.q_slots + chunk - p.ws.cut.k_first : chunk;
                float *to = run ? sums + ((keys && straddles ? teams : 0) + team) * p.D : p.ws.spill + (part * p.ws.n + id) * p.D;
#pragma unroll
                for (int j = 0; j < (in_pieces(PAIRS) ? 8 : 0); ++j)
                    if (col.at[j / piece_pairs(PAIRS)] >= 0) {
                        f2_t *q = reinterpret_cast<f2_t *>(to + col.at[j / piece_pairs(PAIRS)] + 2 * (j % piece_pairs(PAIRS)));
                        *q = run && step > 0 ? f2_add(*q, acc[j]) : acc[j];
                    }
#pragma unroll
                for (int j = 0; j < (in_pieces(PAIRS) ? 0 : 2); ++j)
                    if (col.at[j] >= 0) {
                        ulonglong2 *q = reinterpret_cast<ulonglong2 *>(to + col.at[j]);
                        ulonglong2 u = make_ulonglong2(acc[4 * j], acc[4 * j + 1]), v = make_ulonglong2(acc[4 * j + 2], acc[4 * j + 3]);
                        if (run && step > 0) {
                            u = make_ulonglong2(f2_add(q[0].x, u.x), f2_add(q[0].y, u.y));
                            v = make_ulonglong2(f2_add(q[1].x, v.x), f2_add(q[1].y, v.y));
                        }
                        q[0] = u;
                        q[1] = v;
                    }
            }
        }
    }
    if (grads && run_steps) {
        __syncwarp();
        const uint32_t begins = uint32_t(__shfl_sync(kFull, wd.id, wd.run));
        const int64_t g = p.by_group.quotient(begins);
        if (chunk == 0 && lane32 == 0) p.ws.whole[g] = 1;
        for (int keys = head0 < p.hq ? 0 : 1; keys < 2; ++keys) {
            if (keys && end <= p.hq) break;
            const float *src = sums + (keys && straddles ? teams * p.D : 0);
            const int64_t part = keys ? p.ws.cut.q_slots + chunk - p.ws.cut.k_first : chunk;
            float *dst = p.ws.partial + (part * p.ws.groups + g) * p.D;
            for (int k = lane32 * 4; k < p.D; k += 128) {
                float4 v = *reinterpret_cast<const float4 *>(src + k);
                for (int t = 1; t * share < G; ++t) {
                    const float4 u = *reinterpret_cast<const float4 *>(src + t * p.D + k);
                    v = make_float4(__fadd_rn(v.x, u.x), __fadd_rn(v.y, u.y), __fadd_rn(v.z, u.z), __fadd_rn(v.w, u.w));
                }
                *reinterpret_cast<float4 *>(dst + k) = v;
            }
        }
    }
}

// Launches the rows of one call for element type E (rotary_*.cu instantiate it).
// mode: 0 rotation alone, 1 norm and rotation, 2 their backward pass.
template <class E, int PAIRS>
int rotary_run_pairs(RotaryParams p, int mode, cudaStream_t stream);

}  // namespace rbi
