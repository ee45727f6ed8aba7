// Streaming row kernel of the layer norm for rows of more than 512 columns.
//
// A CTA owns a share of the call (slots dealt out one by one, or with parameter
// gradients consecutive 8-row groups of plan items) and keeps all columns of a
// row: thread i holds the 16-byte vectors i, i + T, ... (NV of them).  Rows arrive in a ring of S shared-memory stages
// by 1-D bulk copies that one thread issues up to S rows ahead, so memory
// stays busy while the CTA computes.
//
// The mean needs one reduction over the row and the variance another one that
// depends on it.  They are taken in one exchange per row all the same: while
// row i's sums of squares (and, backward, of a and a d) are formed, row i + 1
// is already in shared memory and its sum goes into the same exchange, so each
// row costs one CTA barrier and the variance is still the two-pass one.  The
// barrier also releases a stage: every thread has read it, so thread 0 refills
// it without a barrier of its own.
//
// Parameter gradients: the sums of a thread's columns over the 8 rows of a group
// (in logical order), and the fold of a block's groups from its first one on,
// live in tensor memory, which nothing else here needs: a row's terms are added
// on the way through registers.  In registers the sums alone would take 32 of a
// thread's 128 and spill the row, in shared memory they would take the stages'
// place (hidden 8192 with dropout and dres: 322 -> 294 us when they moved here).
//
// What bounds it (bf16, DRAM floor at the copy rate of 6.78 TB/s in brackets):
// forward, hidden 4096, 17,620 rows: 50.5 us (43), 5.7 TB/s; with dropout and
// residual add, hidden 5120, 17,620 active rows among padding: 118 us (107): memory.
// FP32 forward of 1000 columns, 17,163 rows: 28.4 us (20): two warps a CTA, 105 registers
// (16 warps an SM), and a ring that works as one stage less than it has, since nothing
// is issued behind the first exchange, where the first row's stage is free already.
// Backward with both parameter gradients, hidden 4096: 92.5 us (64); hidden 8192
// with dropout and dres, 280 us (213): not memory but the row's chain of
// dependent steps.  A row alone takes about 1,900 cycles (590 of them the
// exchange, 320 the next row's sum, 300 the stores), 380 instructions a warp, and
// 16 warps, all that 128 registers allow, hide half of it (issue slots 50 % busy);
// CTAs of 6 or 12 warps leave 12 an SM.  Next to that the shares are uneven (hidden 4096:
// 80 CTAs have 64 rows, 224 have 56, and the longer ones end alone), and one that starts
// inside a block stores each of its groups there (1,055 partials for 276 blocks).
// Fewer registers (spills), two rows at a time, a copying warp, the outputs put
// off behind the next row and the sums asked for ahead of dx were all measured
// slower or equal.
#pragma once
#include "layernorm_kernels.cuh"
#include "umma.cuh"

namespace rbi {

constexpr int kListRows = 256;                           // rows of one list of a CTA (a multiple of 64)
constexpr int kRedOff = 128, kCountOff = 640, kListOff = 768, kFixedBytes = kListOff + kListRows * 16;
constexpr int kMaxStages = 16;

struct LnEntry {                     // one row of a CTA's list
    int64_t off;                     // element offset of the row
    uint32_t lrow;                   // logical row
    uint32_t tag;                    // forward, dx alone: physical row; parameter gradients: kTag* bits
};
static_assert(sizeof(LnEntry) == 16, "one 16-byte shared-memory load");
// What the last row of a group does with the group's sums: they join the fold
// of the block's first groups (kTagFold) or are stored on their own; kTagStore
// ends the fold (the block's last group, or the last one of this CTA's share).
// kTagSpill: a row of a group that the call holds only partly.
constexpr uint32_t kTagSpill = 1, kTagClose = 2, kTagFold = 4, kTagStore = 8;

template <class E>
struct Lane {                        // a 16-byte vector: kE elements, kP FP32 pairs
    static constexpr int kE = 16 / int(sizeof(E)), kP = kE / 2;
};

__device__ __forceinline__ void f2_unpack(const uint4 &v, f2_t (&f)[4], const __nv_bfloat16 *) { f2_unpack8(v, f); }
__device__ __forceinline__ void f2_unpack(const uint4 &v, f2_t (&f)[4], const __half *) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[i] = f2_make(p.x, p.y);
    }
}
__device__ __forceinline__ void f2_unpack(const uint4 &v, f2_t (&f)[2], const float *) {
    f[0] = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint4 f2_pack(const f2_t (&f)[4], const __nv_bfloat16 *) { return f2_pack8(f); }
__device__ __forceinline__ uint4 f2_pack(const f2_t (&f)[4], const __half *) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f2_lo(f[i]), f2_hi(f[i]));
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 f2_pack(const f2_t (&f)[2], const float *) {
    return make_uint4(__float_as_uint(f2_lo(f[0])), __float_as_uint(f2_hi(f[0])), __float_as_uint(f2_lo(f[1])),
                      __float_as_uint(f2_hi(f[1])));
}
template <class E>
__device__ __forceinline__ void up(const uint4 &v, f2_t (&f)[Lane<E>::kP]) { f2_unpack(v, f, static_cast<const E *>(nullptr)); }
template <class E>
__device__ __forceinline__ uint4 down(const f2_t (&f)[Lane<E>::kP]) { return f2_pack(f, static_cast<const E *>(nullptr)); }

__device__ __forceinline__ f2_t f2_both(float v) { return f2_make(v, v); }

// Parameters of vector v as FP32 pairs.
template <class E>
__device__ __forceinline__ void param_pairs(const void *p, int f32, int v, float none, f2_t (&f)[Lane<E>::kP]) {
    constexpr int P = Lane<E>::kP;
    if (!p) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = f2_both(none);
    } else if (f32) {
        const float2 *q = reinterpret_cast<const float2 *>(static_cast<const float *>(p) + v * Lane<E>::kE);
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = f2_make(q[i].x, q[i].y);
    } else {
        up<E>(static_cast<const uint4 *>(p)[v], f);
    }
}

// Random words of the elements of 16-byte vector v of logical row g, one per pair.
template <class E>
__device__ __forceinline__ void lane_words(int v, uint32_t g, const DropKey &key, uint32_t (&w)[Lane<E>::kP]) {
    if constexpr (Lane<E>::kE == 8) {
        const uint4 r = philox4x32(uint32_t(v), g, key);
        w[0] = r.x;
        w[1] = r.y;
        w[2] = r.z;
        w[3] = r.w;
    } else {
        const uint4 r = philox4x32(uint32_t(v) >> 1, g, key);
        w[0] = v & 1 ? r.z : r.x;
        w[1] = v & 1 ? r.w : r.y;
    }
}

// Pairs times the factor where kept, +0 elsewhere.
template <int P>
__device__ __forceinline__ void drop_pairs(f2_t (&f)[P], const uint32_t (&w)[P], const DropRule &rule) {
    const f2_t s = f2_both(rule.scale);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const f2_t v = f2_mul(f[i], s);
        f[i] = f2_make(kept_lo(w[i], rule) ? f2_lo(v) : 0.f, kept_hi(w[i], rule) ? f2_hi(v) : 0.f);
    }
}
// f = f times the factor + q, with f = +0 where dropped (so that -0 in q becomes +0 there, as in the sum).
template <int P>
__device__ __forceinline__ void drop_add_pairs(f2_t (&f)[P], const f2_t (&q)[P], const uint32_t (&w)[P], const DropRule &rule) {
    const f2_t s = f2_both(rule.scale);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const f2_t kept = f2_make(kept_lo(w[i], rule) ? f2_lo(f[i]) : 0.f, kept_hi(w[i], rule) ? f2_hi(f[i]) : 0.f);
        f[i] = f2_fma(kept, s, q[i]);
    }
}

// Sums K values over the CTA: lanes by a butterfly that hands each value to
// its own lanes on the way (K = 4: 6 shuffles instead of 20), warps through
// shared memory and a second butterfly, or (DIRECT, the most warps of a CTA) by
// reads of all warps' values in every thread: shorter, but more instructions.
// Residual add with dropout in 10 warps (32,768 slots of 5120, 17,624 of them rows):
// butterfly 125 us, reads 119; 8 warps and fewer 92 and 93; 16 warps 92 and 96;
// forward alone and backward as slow or slower by reads.  (CTAs of 9 warps take the
// reads too and were not measured.)  The order of the
// additions is the same in both, warps 8, 4, 2 and 1 apart, and for K = 2 and 4.
// `red` is one of two alternating buffers, zero behind the CTA's warps.
template <int K>
__device__ __forceinline__ void lane_sums(float (&v)[K], float &mine) {
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16;
    if constexpr (K == 4) {
        const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
        float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1];
        a = __fadd_rn(a, __shfl_xor_sync(kFull, s0, 16));
        b = __fadd_rn(b, __shfl_xor_sync(kFull, s1, 16));
        const bool h2 = lane & 8;
        const float s = h2 ? a : b;
        mine = __fadd_rn(h2 ? b : a, __shfl_xor_sync(kFull, s, 8));
    } else {
        const float s = hi ? v[0] : v[1];
        mine = __fadd_rn(hi ? v[1] : v[0], __shfl_xor_sync(kFull, s, 16));
        mine = __fadd_rn(mine, __shfl_xor_sync(kFull, mine, 8));
    }
    mine = __fadd_rn(mine, __shfl_xor_sync(kFull, mine, 4));
    mine = __fadd_rn(mine, __shfl_xor_sync(kFull, mine, 2));
    mine = __fadd_rn(mine, __shfl_xor_sync(kFull, mine, 1));
}

template <int K, int DIRECT>
__device__ __forceinline__ void cta_sums(float (&v)[K], float *red) {
    const int lane = threadIdx.x & 31;
    float m;
    lane_sums(v, m);
    constexpr int kLanes = 32 / K;                       // lanes that hold the same value
    if constexpr (DIRECT > 0) {
        static_assert(K == 2, "pairs of two values");
        if (lane % kLanes == 0) red[(threadIdx.x >> 5) * K + lane / kLanes] = m;
        __syncthreads();
        ulonglong2 q[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) q[w] = 2 * w < DIRECT ? reinterpret_cast<const ulonglong2 *>(red)[w] : make_ulonglong2(0, 0);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
            for (int w = 0; w < o; ++w) q[w] = make_ulonglong2(f2_add(q[w].x, q[w + o].x), f2_add(q[w].y, q[w + o].y));
        q[0].x = f2_add(q[0].x, q[0].y);
        v[0] = f2_lo(q[0].x);
        v[1] = f2_hi(q[0].x);
        return;
    }
    if (lane % kLanes == 0) red[(lane / kLanes) * 16 + (threadIdx.x >> 5)] = m;
    __syncthreads();
    if constexpr (K == 4) {
        m = __fadd_rn(red[(lane >> 3) * 16 + (lane & 7)], red[(lane >> 3) * 16 + (lane & 7) + 8]);
    } else {
        m = red[(lane >> 4) * 16 + (lane & 15)];
        m = __fadd_rn(m, __shfl_xor_sync(kFull, m, 8));
    }
    m = __fadd_rn(m, __shfl_xor_sync(kFull, m, 4));
    m = __fadd_rn(m, __shfl_xor_sync(kFull, m, 2));
    m = __fadd_rn(m, __shfl_xor_sync(kFull, m, 1));
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(kFull, m, k * (32 / K));
}

template <int P>
__device__ __forceinline__ float pair_total(const f2_t (&s)[P]) {
    f2_t t = s[0];
#pragma unroll
    for (int i = 1; i < P; ++i) t = f2_add(t, s[i]);
    return __fadd_rn(f2_lo(t), f2_hi(t));
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// Asks for global memory to be in the L2 (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_prefetch_l2(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ LnEntry lds_entry(uint32_t addr) {
    LnEntry e;
    asm volatile("{\n\t.reg .b32 a, b;\n\tld.shared.v4.u32 {a,b,%1,%2}, [%3];\n\tmov.b64 %0, {a,b};\n\t}"
                 : "=l"(e.off), "=r"(e.lrow), "=r"(e.tag)
                 : "r"(addr));
    return e;
}
// P pairs to consecutive floats, 16 bytes at a time.
template <int P>
__device__ __forceinline__ void pairs_store(float *p, const f2_t (&f)[P]) {
#pragma unroll
    for (int j = 0; j < P; j += 2) *reinterpret_cast<ulonglong2 *>(p + 2 * j) = make_ulonglong2(f[j], f[j + 1]);
}

// The sums of one vector (dweight, then dbias) in tensor memory at `at`, read or
// written by the whole warp.
template <int P>
__device__ __forceinline__ void sums_load(uint32_t at, f2_t (&w)[P], f2_t (&b)[P]) {
    uint32_t u[4 * P];
    if constexpr (P == 4) umma::ld_32x32_x16(at, u);
    else umma::ld_32x32_x8(at, u);
    umma::wait_ld(u);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        w[i] = f2_make(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        b[i] = f2_make(__uint_as_float(u[2 * P + 2 * i]), __uint_as_float(u[2 * P + 2 * i + 1]));
    }
}
template <int P>
__device__ __forceinline__ void sums_store(uint32_t at, const f2_t (&w)[P], const f2_t (&b)[P]) {
    uint32_t u[4 * P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        u[2 * i] = __float_as_uint(f2_lo(w[i]));
        u[2 * i + 1] = __float_as_uint(f2_hi(w[i]));
        u[2 * P + 2 * i] = __float_as_uint(f2_lo(b[i]));
        u[2 * P + 2 * i + 1] = __float_as_uint(f2_hi(b[i]));
    }
    if constexpr (P == 4) umma::st_32x32_x16(at, u);
    else umma::st_32x32_x8(at, u);
}

// Writes the CTA's list number `turn` and returns its length, -1 behind the last
// one.  The CTA's share of positions: with parameter gradients consecutive slots
// of the plan (blocks stay together); else position q is slot q gridDim + blockIdx,
// so that padding, which comes in long runs, falls on every CTA alike.
template <class E, bool GRADS>
__device__ __forceinline__ int ln_list(const LnParams &p, uint8_t *smem, int turn) {
    volatile int *count = reinterpret_cast<volatile int *>(smem + kCountOff);
    LnEntry *list = reinterpret_cast<LnEntry *>(smem + kListOff);
    const int tid = threadIdx.x, T = blockDim.x, warps = T >> 5;
    const int64_t cta = blockIdx.x, more = cta < p.share_rest ? 1 : 0;
    const int64_t share_lo = GRADS ? cta * p.share + (more ? cta : int64_t(p.share_rest)) : 0, share_hi = share_lo + p.share + more;
    const int64_t lo = GRADS ? share_lo * kGroupRows : 0, end = GRADS ? share_hi * kGroupRows : share_hi;
    // whole items after the first list
    const int64_t base = (GRADS ? lo - lo % kBlockRows : 0) + int64_t(turn) * kListRows;
    if (base >= end) return -1;
    const int64_t pos = base < lo ? lo : base, stop = base + kListRows < end ? base + kListRows : end;
    __syncthreads();                                     // the last list is read, its stages are free
    int n = 0;
    for (int64_t q0 = pos; q0 < stop; q0 += T) {
        const int64_t q = q0 + tid;
        LnEntry e = {0, 0, 0};
        bool valid = false;
        if (q < stop) {
            if constexpr (GRADS) {
                const int64_t item = q >> 6;
                const int slot = int(q & 63);
                const PlanItem &it = p.items[item];
                const int kind = it.kind, blk = it.block;
                const int32_t prow = it.prow[slot], lrow = it.lrow[slot];
                if (prow >= 0) {
                    // whole blocks and quarters hold each row at its place, so a
                    // group ends at its last row
                    valid = prow < p.n_rows && lrow >= 0 && lrow < p.ws.n_rows &&
                            (kind == kItemSpill ||
                             ((kind == kItemWhole || kind == kItemQuarters) && lrow == int64_t(blk) * kBlockRows + slot));
                    if (!valid) set_status(p.ws.hdr, kStPlan);
                    const bool block_end = slot == kBlockRows - 1 || lrow == p.ws.n_rows - 1;
                    if (kind == kItemSpill) {
                        e.tag = kTagSpill;
                    } else if (slot % kGroupRows == kGroupRows - 1 || block_end) {
                        e.tag = kTagClose | kTagStore;
                        if (kind == kItemWhole && item * kGroups >= share_lo) {
                            e.tag = kTagClose | kTagFold;
                            if (block_end || (q >> 3) == share_hi - 1) e.tag |= kTagStore;
                        }
                    }
                }
                const uint32_t tok = uint32_t(prow) / uint32_t(p.rpt), head = uint32_t(prow) - tok * uint32_t(p.rpt);
                e.off = int64_t(tok) * p.token_stride + int64_t(head) * p.hidden;
                e.lrow = uint32_t(lrow);
            } else {
                const int64_t slot = q * gridDim.x + blockIdx.x;
                const uint32_t tok = uint32_t(slot) / uint32_t(p.rpt), head = uint32_t(slot) - tok * uint32_t(p.rpt);
                const int32_t id = p.tok_id[tok];
                valid = id >= 0;
                e.off = int64_t(tok) * p.token_stride + int64_t(head) * p.hidden;
                e.lrow = uint32_t(id) * uint32_t(p.rpt) + head;
                e.tag = uint32_t(slot);
            }
        }
        const uint32_t bits = __ballot_sync(kFull, valid);
        if ((tid & 31) == 0) count[tid >> 5] = __popc(bits);
        __syncthreads();
        int at = n;
        for (int i = 0; i < warps; ++i) {
            const int c = count[i];
            if (i < (tid >> 5)) at += c;
            n += c;
        }
        if (valid) list[at + __popc(bits & ((1u << (tid & 31)) - 1u))] = e;
        __syncthreads();
    }
    return n;
}

// With parameter gradients the rare parts are functions of their own, called:
// inlined, their registers would count in the row loop's.
template <class E>
__device__ __noinline__ int ln_list_called(const LnParams &p, uint8_t *smem, int turn) {
    return ln_list<E, true>(p, smem, turn);
}

// Ends a group (its sums are in tensor memory at `sums`, the block's fold behind
// them), or stores a row of a cut one (xhat and dy; the sums held that row alone
// and are dropped).  st: this thread's vectors of the row in its stage.
template <class E, int NV>
__device__ __noinline__ void ln_close(const LnParams &p, uint32_t sums, uint32_t st, uint32_t pitch, float neg_mean, float rstd,
                                      uint32_t lrow, uint32_t tag) {
    constexpr int kE = Lane<E>::kE, P = Lane<E>::kP, kSumCols = 2 * NV * kE;
    const int tid = threadIdx.x, T = blockDim.x, V = p.hidden / kE;
    const bool spill = tag & kTagSpill, fold = tag & kTagFold, store = tag & kTagStore;
    const uint32_t group = lrow / kGroupRows, place = group % kGroups;
    const int64_t slot = fold ? int64_t(group - place) : int64_t(group);
    float *dst = spill ? p.ws.spill + int64_t(lrow) * 2 * p.hidden : p.ws.partial + slot * 2 * p.hidden;
    umma::wait_st();
#pragma unroll 1
    for (int k = 0; k < NV; ++k) {
        const int v = tid + k * T;
        f2_t w[P], b[P];
        if (spill) {
            up<E>(lds_v4(st + k * T * 16), w);
            up<E>(lds_v4(st + pitch + k * T * 16), b);
#pragma unroll
            for (int j = 0; j < P; ++j) w[j] = f2_mul(f2_add(w[j], f2_both(neg_mean)), f2_both(rstd));
        } else {
            sums_load(sums + k * 2 * kE, w, b);
            if (fold && place != 0) {
                f2_t fw[P], fb[P];
                sums_load(sums + kSumCols + k * 2 * kE, fw, fb);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    w[j] = f2_add(fw[j], w[j]);
                    b[j] = f2_add(fb[j], b[j]);
                }
            }
        }
        if (spill || store) {
            if (v < V) {
                pairs_store(dst + v * kE, w);
                pairs_store(dst + p.hidden + v * kE, b);
            }
        } else {
            sums_store(sums + kSumCols + k * 2 * kE, w, b);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) w[j] = 0;            // the next group begins
        sums_store(sums + k * 2 * kE, w, w);
    }
    if (tid == 0) {
        if (p.ws.state[group] != 0 || (spill && p.ws.flag[lrow])) set_status(p.ws.hdr, kStDouble);
        if (spill) p.ws.flag[lrow] = 1;
        else if (!fold) p.ws.state[group] = 1;
        else if (store) p.ws.state[group - place] = uint8_t(place + 1);
    }
}

enum LnMode : int { kLnFwd = 0, kLnAdd = 1, kLnBwd = 2 };

// p.res in kLnBwd: dres, staged as the third tensor when nt is 3.  Rows too wide for
// three stages of three tensors read it directly; it is asked into the L2 when the
// row's copies are issued (with dropout, hidden 16384 bf16, 64 M elements: 241 -> 216
// us; FP32 8192, 32 M: 202 -> 182).
//
// A staged tensor takes NV * T vectors; those past the row's end are zeroed
// once and never written again, and their weights and the mean taken off them
// are zero, so that the passes need no bounds checks, only the stores do.
template <class E, int NV, int MODE, bool DROP, bool GRADS, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) ln_stream_kernel(const __grid_constant__ LnParams p, int S, int nt,
                                                               int tmem_cols) {
    constexpr int kE = Lane<E>::kE, P = Lane<E>::kP;
    constexpr bool kFwd = MODE != kLnBwd;
    constexpr bool kWide = NV == 4 && MAXT == 512;       // instances that hold the rows with nt 2 and dres
    // d and dy stay in registers between the two passes (else they are read from the
    // stage again), where the registers hold them without spills
    constexpr bool kHold = NV * kE <= 16 && !(GRADS && MAXT == 320);
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);
    float *red = reinterpret_cast<float *>(smem + kRedOff);
    volatile int *count = reinterpret_cast<volatile int *>(smem + kCountOff);   // [0..15] warps; [16, 17] a copy
                                                         // did not arrive (alternating like red)
    LnEntry *list = reinterpret_cast<LnEntry *>(smem + kListOff);
    const int tid = threadIdx.x, T = blockDim.x;
    const int V = p.hidden / kE;
    const uint32_t row_bytes = uint32_t(p.hidden) * uint32_t(sizeof(E));
    const uint32_t pitch = uint32_t(NV * T) * 16u, stage_pitch = pitch * uint32_t(nt);
    constexpr uint32_t stage0 = kFixedBytes;
    const uint32_t my0 = smem_addr(smem) + stage0 + uint32_t(tid) * 16u;        // this thread's vectors of stage 0
    const uint32_t list0 = smem_addr(list);
    const uint32_t step = uint32_t(T) * 16u;

    bool header = true;
    if constexpr (GRADS) header = ln_header_ok(p.ws);    // used behind the loads of the parameters
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        count[16] = count[17] = 0;
    }
    for (int i = tid; i < 128; i += T) red[i] = 0.f;
    const DropKey key = DROP ? drop_key(p.drop) : DropKey{0, 0, 0, 0};

    // Forward with four vectors of 16-bit elements a thread: weight and bias as pairs
    // would take 128 registers; they are kept packed (FP32 ones are read per row).
    // Residual add of 64 M elements, hidden 12288: 138 us spilled, 98 packed.
    constexpr bool kPacked = kFwd && NV * kE > 16;
    f2_t w[kPacked ? 1 : NV][P], b[kFwd && !kPacked ? NV : 1][P], in_row[NV];   // in_row: 1 inside the row, 0 past its end
    uint4 wq[kPacked ? NV : 1], bq[kPacked ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = tid + k * T;
        in_row[k] = v < V ? f2_both(1.f) : 0;
        if constexpr (kPacked) {
            f2_t none[P];
#pragma unroll
            for (int i = 0; i < P; ++i) none[i] = f2_both(1.f);
            const bool own = v < V && !p.params_f32;
            wq[k] = own && p.w ? static_cast<const uint4 *>(p.w)[v] : down<E>(none);
            bq[k] = own && p.b ? static_cast<const uint4 *>(p.b)[v] : make_uint4(0, 0, 0, 0);
        } else if (v < V) {
            param_pairs<E>(p.w, p.params_f32, v, 1.f, w[k]);
            if constexpr (kFwd) param_pairs<E>(p.b, p.params_f32, v, 0.f, b[k]);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                w[k][i] = 0;
                if constexpr (kFwd) b[k][i] = 0;
            }
        }
        if (v >= V) {
            for (int s = 0; s < S; ++s)
                for (int t = 0; t < nt; ++t)
                    *reinterpret_cast<uint4 *>(smem + stage0 + s * stage_pitch + t * pitch + v * 16) = make_uint4(0, 0, 0, 0);
        }
    }
    if constexpr (GRADS) {
        if (!header) {
            if (tid == 0) set_status(p.ws.hdr, kStHeader);
            return;
        }
    }
    // Tensor memory: kSumCols columns of a warp's 32 lanes for the group's sums and as
    // many for the block's fold; warps w, w + 4, ... share a quarter of the lanes.
    constexpr int kSumCols = 2 * NV * kE;
    uint32_t sums = 0;
    if constexpr (GRADS) {
        uint32_t *slot = reinterpret_cast<uint32_t *>(smem + kCountOff + 80);
        if (tid < 32) {
            umma::tmem_alloc(slot, uint32_t(tmem_cols));
            umma::tmem_relinquish();
        }
        umma::fence_before();
        __syncthreads();
        umma::fence_after();
        sums = *slot + (uint32_t((tid >> 5) & 3) << 21) + uint32_t(tid >> 7) * uint32_t(2 * kSumCols);
        f2_t zero[P];
#pragma unroll
        for (int i = 0; i < P; ++i) zero[i] = 0;
#pragma unroll 1
        for (int k = 0; k < NV; ++k) sums_store(sums + k * 2 * kE, zero, zero);
    }

    uint32_t done = 0;                                   // rows through the ring so far
    int turn = 0;
    bool dead = false;

#pragma unroll 1
    for (int lists = 0; !dead; ++lists) {
        int n;
        if constexpr (GRADS) n = ln_list_called<E>(p, smem, lists);
        else n = ln_list<E, false>(p, smem, lists);
        if (n < 0) break;
        if (n == 0) continue;

        auto issue = [&](int i) {                        // thread 0
            const uint32_t r = done + uint32_t(i), s = r % uint32_t(S);
            const int64_t off = list[i].off;
            uint8_t *dst = smem + stage0 + s * stage_pitch;
            mbar_arrive_expect_tx(&bars[s], row_bytes * uint32_t(nt));
            bulk_copy_g2s(dst, static_cast<const E *>(p.x) + off, row_bytes, &bars[s]);
            if constexpr (MODE == kLnAdd) bulk_copy_g2s(dst + pitch, static_cast<const E *>(p.res) + off, row_bytes, &bars[s]);
            if constexpr (MODE == kLnBwd) {
                bulk_copy_g2s(dst + pitch, static_cast<const E *>(p.dy) + off, row_bytes, &bars[s]);
                if (nt == 3) bulk_copy_g2s(dst + 2 * pitch, static_cast<const E *>(p.res) + off, row_bytes, &bars[s]);
                else if (kWide && p.res) bulk_prefetch_l2(static_cast<const E *>(p.res) + off, row_bytes);
            }
        };
        int issued = 0;
        if (tid == 0)
            for (; issued < S && issued < n; ++issued) issue(issued);

        uint4 cur[kFwd ? NV : 1], nxt[kFwd ? NV : 1];
        uint32_t s_nxt = done % uint32_t(S), par_nxt = (done / uint32_t(S)) & 1u;
        uint32_t st_nxt = my0 + s_nxt * stage_pitch, st_cur = st_nxt;

        // Sum of row i (the next one), which has to have arrived; forward: the
        // row moves into registers (residual add: it is formed and stored here).
        auto first_pass = [&](int i) -> float {
            int h_end = V;                               // nothing goes into h of a row that did not arrive
            if (!mbar_wait_spin_bounded(&bars[s_nxt], par_nxt)) {
                count[16 + (turn & 1)] = 1;
                h_end = 0;
            }
            f2_t acc[P];
            LnEntry en;
            if constexpr (MODE == kLnAdd) en = lds_entry(list0 + uint32_t(i) * 16u);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                uint4 u = lds_v4(st_nxt + k * step);
                f2_t f[P];
                if constexpr (MODE == kLnAdd) {
                    const int v = tid + k * T;
                    f2_t r[P];
                    up<E>(lds_v4(st_nxt + pitch + k * step), r);
                    up<E>(u, f);
                    if constexpr (DROP) {
                        uint32_t words[P];
                        lane_words<E>(v, en.lrow, key, words);
                        drop_add_pairs(f, r, words, drop_rule(p.drop));
                    } else {
#pragma unroll
                        for (int j = 0; j < P; ++j) f[j] = f2_add(f[j], r[j]);
                    }
                    u = down<E>(f);
                    if (v < h_end) st_global_v4(static_cast<E *>(p.out2) + en.off + v * kE, u);
                }
                up<E>(u, f);
                if constexpr (kFwd) nxt[k] = u;
#pragma unroll
                for (int j = 0; j < P; ++j) acc[j] = k == 0 ? f[j] : f2_add(acc[j], f[j]);
            }
            st_cur = st_nxt;
            st_nxt += stage_pitch;
            if (++s_nxt == uint32_t(S)) {
                s_nxt = 0;
                st_nxt = my0;
                par_nxt ^= 1u;
            }
            return pair_total(acc);
        };

        constexpr int K = kFwd ? 2 : 4;
        float mean;
        {
            float v[K] = {};
            v[0] = first_pass(0);
            cta_sums<K, MODE == kLnAdd && MAXT == 320 ? MAXT / 32 : 0>(v, red + (turn & 1) * 64);
            dead = count[16 + (turn & 1)] != 0;          // the same for every thread
            ++turn;
            mean = __fmul_rn(v[0], p.inv_h);
        }
        for (int i = 0; i < n && !dead; ++i) {
            const uint32_t st = st_cur;
            if constexpr (kFwd) {
#pragma unroll
                for (int k = 0; k < NV; ++k) cur[k] = nxt[k];
            }
            float v[K] = {};
            if (i + 1 < n) v[0] = first_pass(i + 1);
            // ------------------------------------------------ second pass: deviations
            const f2_t neg = f2_both(-mean);
            f2_t d[kHold ? NV : 1][P], g[kHold && !kFwd ? NV : 1][P];
            f2_t m2[P], sa[P], sc[P];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int kk = kHold ? k : 0;
                if constexpr (kFwd) up<E>(cur[k], d[kk]);
                else up<E>(lds_v4(st + k * step), d[kk]);
                if constexpr (!kFwd) up<E>(lds_v4(st + pitch + k * step), g[kk]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    // (a thread's first vector is always inside the row)
                    d[kk][j] = k == 0 ? f2_add(d[kk][j], neg) : f2_fma(in_row[k], neg, d[kk][j]);
                    m2[j] = k == 0 ? f2_mul(d[kk][j], d[kk][j]) : f2_fma(d[kk][j], d[kk][j], m2[j]);
                    if constexpr (!kFwd) {
                        const f2_t a = f2_mul(g[kk][j], w[k][j]);
                        sa[j] = k == 0 ? a : f2_add(sa[j], a);
                        sc[j] = k == 0 ? f2_mul(a, d[kk][j]) : f2_fma(a, d[kk][j], sc[j]);
                    }
                }
            }
            v[1] = pair_total(m2);
            if constexpr (!kFwd) {
                v[2] = pair_total(sa);
                v[3] = pair_total(sc);
            }
            cta_sums<K, MODE == kLnAdd && MAXT == 320 ? MAXT / 32 : 0>(v, red + (turn & 1) * 64);
            dead = count[16 + (turn & 1)] != 0;
            ++turn;
            if (dead) break;
            // every thread has read the stage of row i + 1 (forward) or i - 1 (backward)
            // (a test-only build defines RBI_TEST_WITHHOLD_EMPTY: no stage is refilled, so
            // the wait for row S runs out; see the timeout test)
#ifndef RBI_TEST_WITHHOLD_EMPTY
            if (tid == 0 && issued < n && (kFwd || i >= 1)) issue(issued++);
#endif
            const LnEntry e = lds_entry(list0 + uint32_t(i) * 16u);
            const float rstd = rsqrtf(__fmaf_rn(v[1], p.inv_h, p.eps));
            const f2_t r2 = f2_both(rstd);
            if constexpr (kFwd) {
                if (tid == 0) {
                    if (p.mean) p.mean[e.tag] = mean;
                    if (p.rstd) p.rstd[e.tag] = rstd;
                }
                E *out = static_cast<E *>(p.out) + e.off + tid * kE;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int kk = kHold ? k : 0;
                    if constexpr (!kHold) {
                        up<E>(cur[k], d[0]);
#pragma unroll
                        for (int j = 0; j < P; ++j) d[0][j] = f2_add(d[0][j], neg);
                    }
                    const int kw = kPacked ? 0 : k;
                    if constexpr (kPacked) {
                        if (p.params_f32) {
                            const int v = tid + k * T < V ? tid + k * T : 0;
                            param_pairs<E>(p.w, 1, v, 1.f, w[0]);
                            param_pairs<E>(p.b, 1, v, 0.f, b[0]);
                        } else {
                            up<E>(wq[k], w[0]);
                            up<E>(bq[k], b[0]);
                        }
                    }
                    f2_t o[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) o[j] = f2_fma(f2_mul(d[kk][j], r2), w[kw][j], b[kw][j]);
                    const uint4 u = down<E>(o);
                    if (tid + k * T < V) st_global_v4(out + k * T * kE, u);
                }
            } else {
                // o = s (a - mean(a) - xhat mean(a xhat)) as a s + (d c1 + c0)
                const float s1 = __fmul_rn(rstd, p.grad_scale), ma = __fmul_rn(v[2], p.inv_h);
                const float mc = __fmul_rn(__fmul_rn(v[3], p.inv_h), rstd);
                const f2_t s2 = f2_both(s1), c0 = f2_both(-__fmul_rn(s1, ma));
                const f2_t c1 = f2_both(-__fmul_rn(s1, __fmul_rn(mc, rstd)));
                const bool write = !GRADS || p.out;
                if constexpr (GRADS) umma::wait_st();
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int kk = kHold ? k : 0;
                    if constexpr (!kHold) {
                        up<E>(lds_v4(st + k * step), d[0]);
                        up<E>(lds_v4(st + pitch + k * step), g[0]);
#pragma unroll
                        for (int j = 0; j < P; ++j) d[0][j] = f2_add(d[0][j], neg);
                    }
                    f2_t o[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        o[j] = f2_fma(f2_mul(g[kk][j], w[k][j]), s2, f2_fma(d[kk][j], c1, c0));
                    }
                    if constexpr (GRADS) {
                        f2_t dw[P], db[P];
                        sums_load(sums + k * 2 * kE, dw, db);
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            d[kk][j] = f2_mul(d[kk][j], r2);
                            dw[j] = f2_fma(g[kk][j], d[kk][j], dw[j]);
                            db[j] = f2_add(db[j], g[kk][j]);
                        }
                        sums_store(sums + k * 2 * kE, dw, db);
                    }
                    if (write) {
                        const int64_t at = e.off + (tid + k * T) * kE;
                        const bool in = tid + k * T < V;
                        if (p.res) {
                            f2_t q[P];
                            if (nt == 3) up<E>(lds_v4(st + 2 * pitch + k * step), q);
                            else up<E>(in ? *reinterpret_cast<const uint4 *>(static_cast<const E *>(p.res) + at) : make_uint4(0, 0, 0, 0), q);
#pragma unroll
                            for (int j = 0; j < P; ++j) o[j] = f2_add(o[j], q[j]);
                        }
                        const uint4 u = down<E>(o);
                        if (in) st_global_v4(static_cast<E *>(p.out) + at, u);
                        if constexpr (DROP) {
                            uint32_t words[P];
                            lane_words<E>(tid + k * T, e.lrow, key, words);
                            drop_pairs(o, words, drop_rule(p.drop));
                            const uint4 u2 = down<E>(o);
                            if (in) st_global_v4(static_cast<E *>(p.out2) + at, u2);
                        }
                    }
                }
                if constexpr (GRADS) {
                    if (e.tag) ln_close<E, NV>(p, sums, st, pitch, -mean, rstd, e.lrow, e.tag);
                }
            }
            mean = __fmul_rn(v[0], p.inv_h);
        }
        if (dead) {
            // a copy did not arrive within the limit: report, wait (again with a
            // limit) for what is still in flight, and leave
            if constexpr (GRADS) {
                if (tid == 0) set_status(p.ws.hdr, kStTimeout);
            }
            if (tid == 0) {
                for (int i = issued < S ? 0 : issued - S; i < issued; ++i) {
                    const uint32_t r = done + uint32_t(i);
                    mbar_wait_spin_bounded(&bars[r % uint32_t(S)], (r / uint32_t(S)) & 1u);
                }
            }
            __syncthreads();
        }
        done += uint32_t(n);
    }
    if constexpr (GRADS) {
        umma::wait_st();                                 // this warp's last stores (cleared sums) have landed: the
                                                         // columns may go to another CTA now
        umma::fence_before();
        __syncthreads();
        umma::fence_after();
        if (tid < 32) umma::tmem_dealloc(sums, uint32_t(tmem_cols));
    }
}

}  // namespace rbi
