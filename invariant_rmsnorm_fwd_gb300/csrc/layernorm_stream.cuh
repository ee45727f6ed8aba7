// Streaming row kernel of the layer norm for rows of more than 256 columns.
//
// A CTA owns a contiguous share of the call (rows, or 8-row groups of plan
// items) and keeps all columns of a row: thread i holds the 16-byte vectors
// i, i + T, ... (NV of them).  Rows arrive in a ring of S shared-memory stages
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
// Parameter gradients: a thread's columns accumulate in registers over the 8
// rows of a group (in logical order), and over the groups of a block in shared
// memory where the CTA holds the whole block.
#pragma once
#include "layernorm_kernels.cuh"

namespace rbi {

constexpr int kListRows = 256;                           // rows of one list of a CTA (a multiple of 64)
constexpr int kRedOff = 128, kCountOff = 640, kListOff = 768, kFixedBytes = kListOff + kListRows * 16;
constexpr int kMaxStages = 16;

struct LnEntry {                     // one row of a CTA's list
    int64_t off;                     // element offset of the row
    uint32_t lrow;                   // logical row; bit 31: its group goes into a whole-block partial
    uint32_t prow;                   // physical row; bit 31: a row of a cut group (spilled)
};
static_assert(sizeof(LnEntry) == 16, "one 16-byte shared-memory load");

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

// Keep bits of the elements of 16-byte vector v of logical row g.
template <class E>
__device__ __forceinline__ uint32_t lane_keep(int v, uint32_t g, const DropKey &key, uint32_t t) {
    if constexpr (Lane<E>::kE == 8) return keep_bits(uint32_t(v), g, key, t);
    return keep_bits(uint32_t(v) >> 1, g, key, t) >> (4 * (v & 1));
}

// Pairs times the factor where kept, +0 elsewhere.
template <int P>
__device__ __forceinline__ void drop_pairs(f2_t (&f)[P], uint32_t keep, float scale) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float a = (keep >> (2 * i)) & 1 ? __fmul_rn(f2_lo(f[i]), scale) : 0.f;
        const float b = (keep >> (2 * i + 1)) & 1 ? __fmul_rn(f2_hi(f[i]), scale) : 0.f;
        f[i] = f2_make(a, b);
    }
}

// Sums K values over the CTA: lanes by a butterfly that hands each value to
// its own lanes on the way (K = 4: 6 shuffles instead of 20), warps through
// shared memory.  The order of the additions is the same for K = 2 and 4 and
// depends on the thread count only.  `red` is one of two alternating buffers.
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

template <int K>
__device__ __forceinline__ void cta_sums(float (&v)[K], float *red, int warps) {
    const int lane = threadIdx.x & 31;
    float m;
    lane_sums(v, m);
    if (warps > 1) {
        constexpr int kLanes = 32 / K;                   // lanes that hold the same value
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
    } else {
        __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(kFull, m, k * (32 / K));
}

template <int P, int NV>
__device__ __forceinline__ float pair_total(const f2_t (&s)[P][NV]) {
    f2_t t = s[0][0];
#pragma unroll
    for (int i = 1; i < P * NV; ++i) t = f2_add(t, s[i / NV][i % NV]);
    return __fadd_rn(f2_lo(t), f2_hi(t));
}

enum LnMode : int { kLnFwd = 0, kLnAdd = 1, kLnBwd = 2 };

// p.res in kLnBwd: dres, staged as the third tensor when nt is 3 (rows too wide
// for three stages of three tensors read it directly).
template <class E, int NV, int MODE, bool DROP, bool GRADS, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) ln_stream_kernel(const __grid_constant__ LnParams p, int S, int nt,
                                                               int use_block) {
    constexpr int kE = Lane<E>::kE, P = Lane<E>::kP;
    constexpr bool kFwd = MODE != kLnBwd;
    constexpr bool kHold = NV * kE <= 16;                // d and dy stay in registers between the two passes
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);
    float *red = reinterpret_cast<float *>(smem + kRedOff);
    int *count = reinterpret_cast<int *>(smem + kCountOff);      // [0..15] warps, [16, 17] a copy did not arrive (alternating like red)
    LnEntry *list = reinterpret_cast<LnEntry *>(smem + kListOff);
    const int tid = threadIdx.x, T = blockDim.x, warps = T >> 5;
    const int V = p.hidden / kE;
    const uint32_t row_bytes = uint32_t(p.hidden) * uint32_t(sizeof(E));
    const uint32_t stage_bytes = row_bytes * uint32_t(nt);
    float *block_acc = reinterpret_cast<float *>(smem + kFixedBytes);
    uint8_t *stages = smem + kFixedBytes + (use_block ? uint32_t(align256(int64_t(p.hidden) * 8)) : 0u);

    if constexpr (GRADS) {
        if (!ln_header_ok(p.ws)) {
            if (tid == 0) set_status(p.ws.hdr, kStHeader);
            return;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        count[16] = count[17] = 0;
    }
    for (int i = tid; i < 128; i += T) red[i] = 0.f;
    const DropKey key = DROP ? drop_key(p.drop) : DropKey{0, 0, 0, 0};

    f2_t w[NV][P], b[kFwd ? NV : 1][P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = tid + k * T;
        if (v < V) {
            param_pairs<E>(p.w, p.params_f32, v, 1.f, w[k]);
            if constexpr (kFwd) param_pairs<E>(p.b, p.params_f32, v, 0.f, b[k]);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                w[k][i] = 0;
                if constexpr (kFwd) b[k][i] = 0;
            }
        }
    }
    f2_t dw[GRADS ? NV : 1][P], db[GRADS ? NV : 1][P];
    if constexpr (GRADS) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) dw[k][i] = db[k][i] = 0;
    }

    // this CTA's share: slots [pos, end)
    const int64_t units = GRADS ? p.n_items * kGroups : p.n_rows;
    int64_t pos = units * blockIdx.x / gridDim.x, end = units * (blockIdx.x + 1) / gridDim.x;
    const int64_t share_lo = pos, share_hi = end;        // in groups (GRADS)
    if constexpr (GRADS) {
        pos *= kGroupRows;
        end *= kGroupRows;
    }
    uint32_t done = 0;                                   // rows through the ring so far
    int turn = 0;
    bool dead = false;

    while (pos < end && !dead) {
        // ------------------------------------------------ the list of the next rows
        int64_t stop = pos + kListRows;
        if constexpr (GRADS) stop -= pos % kBlockRows;   // whole items after the first list
        if (stop > end) stop = end;
        __syncthreads();                                 // the last list is read, its stages are free
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
                        valid = prow < p.n_rows && lrow >= 0 && lrow < p.ws.n_rows &&
                                (kind == kItemSpill ||
                                 ((kind == kItemWhole || kind == kItemQuarters) && lrow == int64_t(blk) * kBlockRows + slot));
                        if (!valid) set_status(p.ws.hdr, kStPlan);
                    }
                    const int64_t rows = p.ws.n_rows - int64_t(blk) * kBlockRows;
                    const int groups = rows >= kBlockRows ? kGroups : int((rows + kGroupRows - 1) / kGroupRows);
                    const bool whole = use_block && kind == kItemWhole && item * kGroups >= share_lo &&
                                       item * kGroups + groups <= share_hi;
                    const uint32_t tok = uint32_t(prow) / uint32_t(p.rpt), head = uint32_t(prow) - tok * uint32_t(p.rpt);
                    e.off = int64_t(tok) * p.token_stride + int64_t(head) * p.hidden;
                    e.lrow = uint32_t(lrow) | (whole ? 0x80000000u : 0u);
                    e.prow = uint32_t(prow) | (kind == kItemSpill ? 0x80000000u : 0u);
                } else {
                    const uint32_t tok = uint32_t(q) / uint32_t(p.rpt), head = uint32_t(q) - tok * uint32_t(p.rpt);
                    const int32_t id = p.tok_id[tok];
                    valid = id >= 0;
                    e.off = int64_t(tok) * p.token_stride + int64_t(head) * p.hidden;
                    e.lrow = uint32_t(id) * uint32_t(p.rpt) + head;
                    e.prow = uint32_t(q);
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
        pos = stop;
        if (n == 0) continue;

        auto issue = [&](int i) {                        // thread 0
            const uint32_t r = done + uint32_t(i), s = r % uint32_t(S);
            const int64_t off = list[i].off;
            uint8_t *dst = stages + s * stage_bytes;
            mbar_arrive_expect_tx(&bars[s], stage_bytes);
            bulk_copy_g2s(dst, static_cast<const E *>(p.x) + off, row_bytes, &bars[s]);
            if constexpr (MODE == kLnAdd) bulk_copy_g2s(dst + row_bytes, static_cast<const E *>(p.res) + off, row_bytes, &bars[s]);
            if constexpr (MODE == kLnBwd) {
                bulk_copy_g2s(dst + row_bytes, static_cast<const E *>(p.dy) + off, row_bytes, &bars[s]);
                if (nt == 3) bulk_copy_g2s(dst + 2 * row_bytes, static_cast<const E *>(p.res) + off, row_bytes, &bars[s]);
            }
        };
        int issued = 0;
        if (tid == 0)
            for (; issued < S && issued < n; ++issued) issue(issued);

        uint4 cur[kFwd ? NV : 1], nxt[kFwd ? NV : 1];
        uint32_t s_cur = done % uint32_t(S), s_nxt = s_cur, par_nxt = (done / uint32_t(S)) & 1u;

        // Sum of row i (the next one), which has to have arrived; forward: the
        // row moves into registers (residual add: it is formed and stored here).
        auto first_pass = [&](int i, float &sum) {
            if (!mbar_wait_spin_bounded(&bars[s_nxt], par_nxt)) count[16 + (turn & 1)] = 1;
            const uint8_t *st = stages + s_nxt * stage_bytes;
            f2_t acc[P][1];
#pragma unroll
            for (int j = 0; j < P; ++j) acc[j][0] = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = tid + k * T;
                if (v < V) {
                    uint4 u = ld_shared_v4(st + v * 16);
                    f2_t f[P];
                    if constexpr (MODE == kLnAdd) {
                        f2_t r[P];
                        up<E>(ld_shared_v4(st + row_bytes + v * 16), r);
                        up<E>(u, f);
                        if constexpr (DROP) {
                            const uint32_t keep = lane_keep<E>(v, list[i].lrow, key, p.drop.t);
#pragma unroll
                            for (int j = 0; j < P; ++j) {
                                const float lo = __fmaf_rn(f2_lo(f[j]), p.drop.scale, f2_lo(r[j]));
                                const float hi = __fmaf_rn(f2_hi(f[j]), p.drop.scale, f2_hi(r[j]));
                                f[j] = f2_make((keep >> (2 * j)) & 1 ? lo : f2_lo(r[j]),
                                               (keep >> (2 * j + 1)) & 1 ? hi : f2_hi(r[j]));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < P; ++j) f[j] = f2_add(f[j], r[j]);
                        }
                        u = down<E>(f);
                        st_global_v4(static_cast<E *>(p.out2) + list[i].off + v * kE, u);
                    }
                    up<E>(u, f);
                    if constexpr (kFwd) nxt[k] = u;
#pragma unroll
                    for (int j = 0; j < P; ++j) acc[j][0] = f2_add(acc[j][0], f[j]);
                }
            }
            sum = pair_total(acc);
            s_cur = s_nxt;
            if (++s_nxt == uint32_t(S)) {
                s_nxt = 0;
                par_nxt ^= 1u;
            }
        };

        constexpr int K = kFwd ? 2 : 4;
        float mean;
        {
            float v[K] = {};
            first_pass(0, v[0]);
            cta_sums<K>(v, red + (turn & 1) * 64, warps);
            dead = count[16 + (turn & 1)] != 0;          // the same for every thread
            ++turn;
            mean = __fmul_rn(v[0], p.inv_h);
        }
        for (int i = 0; i < n && !dead; ++i) {
            const uint32_t s_row = s_cur;
            if constexpr (kFwd) {
#pragma unroll
                for (int k = 0; k < NV; ++k) cur[k] = nxt[k];
            }
            float v[K] = {};
            if (i + 1 < n) first_pass(i + 1, v[0]);
            // ------------------------------------------------ second pass: deviations
            const uint8_t *st = stages + s_row * stage_bytes;
            const f2_t neg = f2_both(-mean);
            const LnEntry e = list[i];
            f2_t d[kHold ? NV : 1][P], g[kHold && !kFwd ? NV : 1][P];
            f2_t m2[P][1], sa[P][1], sc[P][1];
#pragma unroll
            for (int j = 0; j < P; ++j) m2[j][0] = sa[j][0] = sc[j][0] = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int vec = tid + k * T;
                const int kk = kHold ? k : 0;
                if (vec < V) {
                    if constexpr (kFwd) up<E>(cur[k], d[kk]);
                    else up<E>(ld_shared_v4(st + vec * 16), d[kk]);
                    if constexpr (!kFwd) up<E>(ld_shared_v4(st + row_bytes + vec * 16), g[kk]);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        d[kk][j] = f2_add(d[kk][j], neg);
                        m2[j][0] = f2_fma(d[kk][j], d[kk][j], m2[j][0]);
                        if constexpr (!kFwd) {
                            const f2_t a = f2_mul(g[kk][j], w[k][j]);
                            sa[j][0] = f2_add(sa[j][0], a);
                            sc[j][0] = f2_fma(a, d[kk][j], sc[j][0]);
                        }
                    }
                }
            }
            v[1] = pair_total(m2);
            if constexpr (!kFwd) {
                v[2] = pair_total(sa);
                v[3] = pair_total(sc);
            }
            cta_sums<K>(v, red + (turn & 1) * 64, warps);
            dead = count[16 + (turn & 1)] != 0;
            ++turn;
            if (dead) break;
            // every thread has read the stage of row i + 1 (forward) or i - 1 (backward)
            if (tid == 0 && issued < n && (kFwd || i >= 1)) issue(issued++);
            const float rstd = rsqrtf(__fmaf_rn(v[1], p.inv_h, p.eps));
            if constexpr (kFwd) {
                if (tid == 0) {
                    if (p.mean) p.mean[e.prow] = mean;
                    if (p.rstd) p.rstd[e.prow] = rstd;
                }
                const f2_t r2 = f2_both(rstd);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int vec = tid + k * T;
                    const int kk = kHold ? k : 0;
                    if (vec < V) {
                        if constexpr (!kHold) {
                            up<E>(cur[k], d[0]);
#pragma unroll
                            for (int j = 0; j < P; ++j) d[0][j] = f2_add(d[0][j], neg);
                        }
                        f2_t o[P];
#pragma unroll
                        for (int j = 0; j < P; ++j) o[j] = f2_fma(f2_mul(d[kk][j], r2), w[k][j], b[k][j]);
                        st_global_v4(static_cast<E *>(p.out) + e.off + vec * kE, down<E>(o));
                    }
                }
            } else {
                const float ma = __fmul_rn(v[2], p.inv_h), mc = __fmul_rn(__fmul_rn(v[3], p.inv_h), rstd);
                const f2_t r2 = f2_both(rstd), nma = f2_both(-ma), nmc = f2_both(-mc);
                const f2_t s2 = f2_both(__fmul_rn(rstd, p.grad_scale));
                const bool spill = GRADS && (e.prow >> 31);
                const uint32_t lrow = e.lrow & 0x7fffffffu;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int vec = tid + k * T;
                    const int kk = kHold ? k : 0;
                    if (vec < V) {
                        if constexpr (!kHold) {
                            up<E>(ld_shared_v4(st + vec * 16), d[0]);
                            up<E>(ld_shared_v4(st + row_bytes + vec * 16), g[0]);
#pragma unroll
                            for (int j = 0; j < P; ++j) d[0][j] = f2_add(d[0][j], neg);
                        }
                        f2_t xh[P], o[P];
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            xh[j] = f2_mul(d[kk][j], r2);
                            o[j] = f2_add(f2_fma(xh[j], nmc, f2_mul(g[kk][j], w[k][j])), nma);
                        }
                        if constexpr (GRADS) {
                            if (!spill) {
#pragma unroll
                                for (int j = 0; j < P; ++j) {
                                    dw[k][j] = f2_fma(g[kk][j], xh[j], dw[k][j]);
                                    db[k][j] = f2_add(db[k][j], g[kk][j]);
                                }
                            } else {
                                float *sp = p.ws.spill + int64_t(lrow) * 2 * p.hidden + vec * kE;
#pragma unroll
                                for (int j = 0; j < P; ++j) {
                                    *reinterpret_cast<f2_t *>(sp + 2 * j) = xh[j];
                                    *reinterpret_cast<f2_t *>(sp + p.hidden + 2 * j) = g[kk][j];
                                }
                            }
                        }
                        if (!GRADS || p.out) {
                            if (p.res) {
                                f2_t q[P];
                                if (nt == 3) up<E>(ld_shared_v4(st + 2 * row_bytes + vec * 16), q);
                                else up<E>(*reinterpret_cast<const uint4 *>(static_cast<const E *>(p.res) + e.off + vec * kE), q);
#pragma unroll
                                for (int j = 0; j < P; ++j) o[j] = f2_fma(o[j], s2, q[j]);
                            } else {
#pragma unroll
                                for (int j = 0; j < P; ++j) o[j] = f2_mul(o[j], s2);
                            }
                            st_global_v4(static_cast<E *>(p.out) + e.off + vec * kE, down<E>(o));
                            if constexpr (DROP) {
                                drop_pairs(o, lane_keep<E>(vec, lrow, key, p.drop.t), p.drop.scale);
                                st_global_v4(static_cast<E *>(p.out2) + e.off + vec * kE, down<E>(o));
                            }
                        }
                    }
                }
                if constexpr (GRADS) {
                    const LnEntry nx = i + 1 < n ? list[i + 1] : LnEntry{0, 0xffffffffu, 0x80000000u};
                    const uint32_t nx_row = nx.prow >> 31 ? 0xffffffffu : nx.lrow & 0x7fffffffu;
                    if (spill) {
                        if (tid == 0) {
                            if (p.ws.flag[lrow] || p.ws.state[lrow / kGroupRows] != kGroupNone) set_status(p.ws.hdr, kStDouble);
                            p.ws.flag[lrow] = 1;
                        }
                    } else if (nx_row / kGroupRows != lrow / kGroupRows) {
                        // the group is complete
                        const bool whole = e.lrow >> 31;
                        const bool first = lrow % kBlockRows < kGroupRows, last = nx_row / kBlockRows != lrow / kBlockRows;
                        const int64_t slot = whole ? int64_t(lrow / kBlockRows) * kGroups : int64_t(lrow / kGroupRows);
                        float *dst = p.ws.partial + slot * 2 * p.hidden;
#pragma unroll
                        for (int k = 0; k < NV; ++k) {
                            const int vec = tid + k * T;
                            if (vec < V) {
                                float *a = whole && !last ? block_acc : dst;
                                f2_t *aw = reinterpret_cast<f2_t *>(a + vec * kE), *ab = reinterpret_cast<f2_t *>(a + p.hidden + vec * kE);
                                const f2_t *pw = reinterpret_cast<const f2_t *>(block_acc + vec * kE);
                                const f2_t *pb = reinterpret_cast<const f2_t *>(block_acc + p.hidden + vec * kE);
#pragma unroll
                                for (int j = 0; j < P; ++j) {
                                    if (whole && !first) {
                                        dw[k][j] = f2_add(pw[j], dw[k][j]);
                                        db[k][j] = f2_add(pb[j], db[k][j]);
                                    }
                                    aw[j] = dw[k][j];
                                    ab[j] = db[k][j];
                                    dw[k][j] = db[k][j] = 0;
                                }
                            }
                        }
                        if (tid == 0 && (last || !whole)) {
                            if (whole) {
                                uint64_t *state = reinterpret_cast<uint64_t *>(p.ws.state) + lrow / kBlockRows;
                                if (*state != 0) set_status(p.ws.hdr, kStDouble);
                                *state = 0x0101010101010101ull * kGroupWhole;
                            } else {
                                uint8_t *state = p.ws.state + lrow / kGroupRows;
                                if (*state != kGroupNone) set_status(p.ws.hdr, kStDouble);
                                *state = kGroupPartial;
                            }
                        }
                    }
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
}

}  // namespace rbi
