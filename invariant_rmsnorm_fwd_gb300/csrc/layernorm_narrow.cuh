// Row kernel of the layer norm for rows of at most 512 columns (per-head norms).
//
// A row is held by a team of P lanes, 8 columns a lane (16 above 256 columns), so a
// warp works on 32 / P rows at once and a row's sums need only shuffles.  A team
// takes the 8 slots of one group one after the other (in logical order where
// parameter gradients are wanted) and goes on to its next group; each lane keeps
// the next kDepth rows' pieces on their way into shared-memory places of its own
// (cp.async), across groups, and reads the slots of a group while it works on the
// one before, so memory does not wait for a group's end.  Empty slots are computed
// as zeros and store nothing, so the shuffles of a warp stay together.
//
// Parameter gradients: a lane's columns add up over the group; the groups of a
// block are in one CTA, which folds them through shared memory (from the first to
// the last) and writes one partial per block.
//
// Forward, memory bounds it (hidden 128, 64 M bf16 elements: 46 us, 0.87 of the copy
// rate); backward, issue does: a row's 16-byte piece costs a lane its share of up to five
// shuffles for each of four sums next to the arithmetic (102 us, 0.58), and nearly all
// instances with parameter gradients spill a few registers at the 80 that three CTAs
// leave (8 to 108 bytes of local stores and loads in bf16).  A call's last round of
// groups may be half empty (264,960 rows of 128: 4.5 rounds).  Widths between powers of
// two leave lanes idle (hidden 72: 0.6 and 0.37).
#pragma once
#include "host.cuh"
#include "layernorm_host.cuh"
#include "layernorm_stream.cuh"

namespace rbi {

template <class E>
struct Oct {                         // 8 packed elements
    static constexpr int kQ = int(sizeof(E)) / 2;        // 16-byte words
    uint4 q[kQ];
};
template <class E>
__device__ __forceinline__ Oct<E> oct_load(const void *base, int64_t elem) {
    Oct<E> v;
#pragma unroll
    for (int i = 0; i < Oct<E>::kQ; ++i) v.q[i] = reinterpret_cast<const uint4 *>(static_cast<const E *>(base) + elem)[i];
    return v;
}
template <class E>
__device__ __forceinline__ void oct_store(void *base, int64_t elem, const f2_t (&f)[4]) {
    E *p = static_cast<E *>(base) + elem;
    if constexpr (sizeof(E) == 4) {
        st_global_f2x4(reinterpret_cast<float *>(p), f);
    } else {
        st_global_v4(p, down<E>(f));
    }
}
template <class E>
__device__ __forceinline__ void oct_up(const Oct<E> &v, f2_t (&f)[4]) {
    if constexpr (sizeof(E) == 4) {
        f2_t a[2], b[2];
        up<E>(v.q[0], a);
        up<E>(v.q[1], b);
        f[0] = a[0];
        f[1] = a[1];
        f[2] = b[0];
        f[3] = b[1];
    } else {
        up<E>(v.q[0], f);
    }
}
template <class E>
__device__ __forceinline__ void oct_param(const void *p, int f32, int v, float none, f2_t (&f)[4]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2_both(none);
    } else if (f32) {
        oct_up<float>(oct_load<float>(p, v * 8), f);
    } else {
        oct_up<E>(oct_load<E>(p, v * 8), f);
    }
}

// Sum over a team of P lanes; every lane gets it.
template <int P>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int o = P / 2; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

constexpr int kNarrowThreads = 256;

// NO: octets of columns a lane holds (l, l + P).
template <class E, int NO, int MODE, bool RES>
constexpr int kNarrowPieces = (MODE == kLnFwd ? 1 : 2 + (RES ? 1 : 0)) * Oct<E>::kQ * NO;   // 16-byte pieces of a lane's row
template <int NO>
constexpr int kNarrowDepth = 4 / NO;                     // rows of a team on their way

// The slots of a team's group: slot j belongs to lane j % P.
template <int P>
struct TeamSlots {
    static constexpr int kOwn = P >= kGroupRows ? 1 : kGroupRows / P;
    int64_t off[kOwn];               // element offset of the row
    uint32_t row[kOwn];              // logical row
    uint32_t on;                     // the team's slots that hold a row
    int32_t kind, block;             // of the plan item
    int32_t slot0;
    bool partial;                    // the group holds all its rows
};

// What is read of a group before its slots are worked out.
template <int P>
struct TeamRaw {
    int32_t prow[TeamSlots<P>::kOwn], lrow[TeamSlots<P>::kOwn];   // without a plan: lrow is the token's id
    int32_t kind, block, quarters;
};

template <int P, bool GRADS>
__device__ __forceinline__ void team_read(const LnParams &p, int64_t group, TeamRaw<P> &raw) {
    const int l = threadIdx.x % P;
    if constexpr (GRADS) {
        raw.kind = raw.block = -1;
        raw.quarters = 0;
        const bool have = group < p.n_items * kGroups;
        const PlanItem *it = p.items + (have ? group / kGroups : 0);
        if (have) {
            raw.kind = it->kind;
            raw.block = it->block;
            raw.quarters = it->quarters;
        }
#pragma unroll
        for (int o = 0; o < TeamSlots<P>::kOwn; ++o) {
            const int j = l + o * P;
            raw.prow[o] = raw.lrow[o] = -1;
            if (have && j < kGroupRows) {
                raw.prow[o] = it->prow[int(group % kGroups) * kGroupRows + j];
                raw.lrow[o] = it->lrow[int(group % kGroups) * kGroupRows + j];
            }
        }
    } else {
#pragma unroll
        for (int o = 0; o < TeamSlots<P>::kOwn; ++o) {
            const int j = l + o * P;
            const int64_t prow = group * kGroupRows + j;
            raw.prow[o] = raw.lrow[o] = -1;
            if (j < kGroupRows && prow < p.n_rows) {
                raw.prow[o] = int32_t(prow);
                raw.lrow[o] = p.tok_id[p.rpt == 1 ? uint32_t(prow) : uint32_t(prow) / uint32_t(p.rpt)];
            }
        }
    }
}

template <int P, bool GRADS>
__device__ __forceinline__ void team_slots(const LnParams &p, int64_t group, const TeamRaw<P> &raw, TeamSlots<P> &s) {
    const int l = threadIdx.x % P;
    s.on = 0;
    s.slot0 = int(group % kGroups) * kGroupRows;
    if constexpr (GRADS) {
        s.kind = raw.kind;
        s.block = raw.block;
        // an item of a block that the workspace does not have contributes nothing
        const bool blocked = raw.kind == kItemWhole || raw.kind == kItemQuarters;
        const bool known = uint32_t(raw.block) < uint32_t(p.ws.n_blocks);
        s.partial = known && (raw.kind == kItemWhole || (raw.kind == kItemQuarters && ((raw.quarters >> (s.slot0 / 16)) & 1)));
        if (blocked && !known) set_status(p.ws.hdr, kStPlan);
    }
#pragma unroll
    for (int o = 0; o < TeamSlots<P>::kOwn; ++o) {
        const int64_t prow = raw.prow[o], lr = raw.lrow[o];
        bool valid = prow >= 0;
        if constexpr (GRADS) {
            if (valid) {
                valid = prow < p.n_rows && lr >= 0 && lr < p.ws.n_rows &&
                        (raw.kind == kItemSpill || ((raw.kind == kItemWhole || raw.kind == kItemQuarters) &&
                                                    lr == int64_t(raw.block) * kBlockRows + s.slot0 + l + o * P));
                if (!valid) set_status(p.ws.hdr, kStPlan);
            }
        } else {
            valid = valid && lr >= 0;
        }
        s.off[o] = 0;
        s.row[o] = 0;
        if (valid) {
            const uint32_t t = p.rpt == 1 ? uint32_t(prow) : uint32_t(prow) / uint32_t(p.rpt), head = uint32_t(prow) - t * uint32_t(p.rpt);
            s.off[o] = int64_t(t) * p.token_stride + int64_t(head) * p.hidden;
            s.row[o] = GRADS ? uint32_t(lr) : uint32_t(lr) * uint32_t(p.rpt) + head;
        }
        const uint32_t all = __ballot_sync(kFull, valid) >> ((threadIdx.x & 31) - l);
        s.on |= (all & ((1u << (P < kGroupRows ? P : kGroupRows)) - 1u)) << (o * P);
    }
}

// RES: dres is added (kLnBwd).
template <class E, int P, int NO, int MODE, bool DROP, bool GRADS, bool RES>
__global__ void __launch_bounds__(kNarrowThreads, NO == 1 ? 3 : 2) ln_narrow_kernel(const __grid_constant__ LnParams p) {
    constexpr bool kFwd = MODE != kLnBwd, kRes = MODE == kLnAdd || RES;
    constexpr int kPieces = kNarrowPieces<E, NO, MODE, RES>, kDepth = kNarrowDepth<NO>, kQ = Oct<E>::kQ;
    constexpr int kTeams = kNarrowThreads / P, kCols = 8 * P * NO, kPiece = kNarrowThreads * 16;
    constexpr int kOwn = TeamSlots<P>::kOwn;
    extern __shared__ __align__(128) uint8_t smem[];     // [kDepth][kPieces][256 threads], then the block sums
    float *sums = reinterpret_cast<float *>(smem + kDepth * kPieces * kPiece);   // [team][dweight, dbias][kCols]
    const int tid = threadIdx.x, team = tid / P, l = tid % P, V = p.hidden >> 3;
    const uint32_t mine = smem_addr(smem) + uint32_t(tid) * 16u;
    bool col[NO];                                        // this lane has the columns of octet l + k P
    bool header = true;
    if constexpr (GRADS) header = ln_header_ok(p.ws);    // used behind the loads of the parameters
    const DropKey key = DROP ? drop_key(p.drop) : DropKey{0, 0, 0, 0};
    const int64_t groups = GRADS ? p.n_items * kGroups : (p.n_rows + kGroupRows - 1) / kGroupRows;
    const int64_t stride = int64_t(gridDim.x) * kTeams;
    f2_t w[NO][4], b[kFwd ? NO : 1][4];
#pragma unroll
    for (int k = 0; k < NO; ++k) {
        col[k] = l + k * P < V;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[k][j] = 0;
            if constexpr (kFwd) b[k][j] = 0;
        }
        if (col[k]) {
            oct_param<E>(p.w, p.params_f32, l + k * P, 1.f, w[k]);
            if constexpr (kFwd) oct_param<E>(p.b, p.params_f32, l + k * P, 0.f, b[k]);
        }
    }
    if constexpr (GRADS) {
        if (!header) {
            if (tid == 0) set_status(p.ws.hdr, kStHeader);
            return;
        }
    }
    // The sums of a lane's columns over its group: in registers, or in tensor memory
    // (16 columns an octet; warps w and w + 4 share a quarter of the lanes) where
    // dropout or dres need the registers (64 M bf16 elements, registers / tensor
    // memory: hidden 128 backward 103 / 108 us, with both 168 / 144; hidden 512
    // 98 / 102, with both 189 / 160).
    constexpr bool kTmem = GRADS && (DROP || RES), kRegs = GRADS && !kTmem;
    constexpr uint32_t kTmemCols = 32 * NO;
    uint32_t acc = 0;
    f2_t rw[kRegs ? NO : 1][4] = {}, rb[kRegs ? NO : 1][4] = {};
    if constexpr (kTmem) {
        __shared__ uint32_t tmem;
        if (tid < 32) {
            umma::tmem_alloc(&tmem, kTmemCols);
            umma::tmem_relinquish();
        }
        umma::fence_before();
        __syncthreads();
        umma::fence_after();
        acc = tmem + (uint32_t((tid >> 5) & 3) << 21) + uint32_t(tid >> 7) * (16 * NO);
        const f2_t zero[4] = {};
#pragma unroll
        for (int k = 0; k < NO; ++k) sums_store(acc + k * 16, zero, zero);
    }
    TeamSlots<P> cur, nxt;
    // Requests row j of the group into place j % kDepth.
    auto request = [&](const TeamSlots<P> &s, int j) {
        const int64_t at = __shfl_sync(kFull, s.off[j / P], j % P, P) + l * 8;
#pragma unroll
        for (int k = 0; k < NO; ++k) {
            const uint32_t bytes = ((s.on >> j) & 1) && col[k] ? 16u : 0u;
            const uint32_t to = mine + uint32_t((j % kDepth) * kPieces + k) * uint32_t(kPiece);
            const int64_t from = bytes ? at + k * P * 8 : 0;
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                cp_async_zfill(to + q * NO * kPiece, static_cast<const E *>(p.x) + from + q * 4, bytes);
                if constexpr (!kFwd) cp_async_zfill(to + (kQ + q) * NO * kPiece, static_cast<const E *>(p.dy) + from + q * 4, bytes);
                if constexpr (kRes)
                    cp_async_zfill(to + ((kFwd ? 1 : 2) * kQ + q) * NO * kPiece, static_cast<const E *>(p.res) + from + q * 4, bytes);
            }
        }
        cp_async_commit();
    };
    // A lane's octet k of tensor t (0 x, 1 dy, last the residual) of the row in place j % kDepth.
    auto fetch = [&](int j, int t, int k) {
        const uint32_t at = mine + uint32_t((j % kDepth) * kPieces + t * kQ * NO + k) * uint32_t(kPiece);
        Oct<E> v;
#pragma unroll
        for (int q = 0; q < kQ; ++q) ld_shared_vec(at + q * NO * kPiece, v.q[q]);
        return v;
    };
    int64_t unit = int64_t(blockIdx.x) * kTeams;         // first group of this CTA's teams
    {
        TeamRaw<P> raw;
        team_read<P, GRADS>(p, unit + team, raw);
        team_slots<P, GRADS>(p, unit + team, raw, cur);
    }
#pragma unroll
    for (int j = 0; j < kDepth; ++j) request(cur, j);
#pragma unroll 1
    for (; unit < groups; unit += stride) {
        const int64_t group = unit + team;
        TeamRaw<P> raw;
        team_read<P, GRADS>(p, group + stride, raw);
        float own_mean[kFwd ? kOwn : 1], own_rstd[kFwd ? kOwn : 1];
#pragma unroll
        for (int j0 = 0; j0 < kGroupRows; ++j0) {
            cp_async_wait<kDepth - 1>();                 // row j0 has arrived (in this lane's own places)
            Oct<E> xo[NO], go[NO];
#pragma unroll
            for (int k = 0; k < NO; ++k) {
                xo[k] = fetch(j0, 0, k);
                if constexpr (!kFwd) go[k] = fetch(j0, 1, k);
            }
            const int64_t here = __shfl_sync(kFull, cur.off[j0 / P], j0 % P, P) + l * 8;
            const bool row = (cur.on >> j0) & 1;
            uint32_t lrow = 0;
            if constexpr (DROP || GRADS) lrow = __shfl_sync(kFull, cur.row[j0 / P], j0 % P, P);
            f2_t x[NO][4], g[NO][4], t;
#pragma unroll
            for (int k = 0; k < NO; ++k) {
                oct_up<E>(xo[k], x[k]);
                if constexpr (MODE == kLnAdd) {
                    f2_t q[4];
                    oct_up<E>(fetch(j0, 1, k), q);
                    if constexpr (DROP) {
                        const uint4 u = philox4x32(uint32_t(l + k * P), lrow, key);
                        const uint32_t words[4] = {u.x, u.y, u.z, u.w};
                        drop_add_pairs(x[k], q, words, drop_rule(p.drop));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[k][j] = f2_add(x[k][j], q[j]);
                    }
                    if (row && col[k]) oct_store<E>(p.out2, here + k * P * 8, x[k]);
                    if constexpr (sizeof(E) == 2) {      // the norm takes the stored h
                        const uint4 h = down<E>(x[k]);
                        up<E>(h, x[k]);
                    }
                }
                const f2_t s = f2_add(f2_add(x[k][0], x[k][1]), f2_add(x[k][2], x[k][3]));
                t = k == 0 ? s : f2_add(t, s);
            }
            const float mean = __fmul_rn(team_sum<P>(__fadd_rn(f2_lo(t), f2_hi(t))), p.inv_h);
            f2_t m2, sa, sc;
#pragma unroll
            for (int k = 0; k < NO; ++k) {
                const f2_t neg = col[k] ? f2_both(-mean) : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = f2_add(x[k][j], neg);
                    m2 = k + j == 0 ? f2_mul(x[0][0], x[0][0]) : f2_fma(x[k][j], x[k][j], m2);
                }
            }
            if constexpr (kFwd) {
                const float var = __fmul_rn(team_sum<P>(__fadd_rn(f2_lo(m2), f2_hi(m2))), p.inv_h);
                const float rstd = rsqrtf(__fadd_rn(var, p.eps));
                if (l == j0 % P) {
                    own_mean[j0 / P] = mean;
                    own_rstd[j0 / P] = rstd;
                }
                const f2_t r2 = f2_both(rstd);
#pragma unroll
                for (int k = 0; k < NO; ++k) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[k][j] = f2_fma(f2_mul(x[k][j], r2), w[k][j], b[k][j]);
                    if (row && col[k]) oct_store<E>(p.out, here + k * P * 8, x[k]);
                }
            } else {
                // the three sums of the row side by side (independent shuffles)
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    oct_up<E>(go[k], g[k]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f2_t a = f2_mul(g[k][j], w[k][j]);
                        sa = k + j == 0 ? a : f2_add(sa, a);
                        sc = k + j == 0 ? f2_mul(a, x[0][0]) : f2_fma(a, x[k][j], sc);
                    }
                }
                const float var = __fmul_rn(team_sum<P>(__fadd_rn(f2_lo(m2), f2_hi(m2))), p.inv_h);
                const float ma = __fmul_rn(team_sum<P>(__fadd_rn(f2_lo(sa), f2_hi(sa))), p.inv_h);
                const float md = __fmul_rn(team_sum<P>(__fadd_rn(f2_lo(sc), f2_hi(sc))), p.inv_h);
                // (an empty slot adds zeros, also where eps is 0)
                const float rstd = row ? rsqrtf(__fadd_rn(var, p.eps)) : 0.f;
                const f2_t r2 = f2_both(rstd);
                // s (a - mean(a) - xhat mean(a xhat)) as a s + (d c1 + c0)
                if constexpr (kTmem) umma::wait_st();
                const float s1 = __fmul_rn(rstd, p.grad_scale), mc = __fmul_rn(md, rstd);
                const f2_t s2 = f2_both(s1), c0 = f2_both(-__fmul_rn(s1, ma)), c1 = f2_both(-__fmul_rn(s1, __fmul_rn(mc, rstd)));
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    f2_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[j] = f2_fma(f2_mul(g[k][j], w[k][j]), s2, f2_fma(x[k][j], c1, c0));
                    }
                    if constexpr (GRADS) {
                        f2_t (&dw)[4] = rw[kRegs ? k : 0], (&db)[4] = rb[kRegs ? k : 0];
                        if constexpr (kTmem) sums_load(acc + k * 16, dw, db);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[k][j] = f2_mul(x[k][j], r2);
                            dw[j] = f2_fma(g[k][j], x[k][j], dw[j]);
                            db[j] = f2_add(db[j], g[k][j]);
                        }
                        if constexpr (kTmem) sums_store(acc + k * 16, dw, db);
                        if (row && !cur.partial && col[k]) {   // a row of a cut group
                            float *sp = p.ws.spill + int64_t(lrow) * 2 * p.hidden + (l + k * P) * 8;
                            st_global_f2x4(sp, x[k]);
                            st_global_f2x4(sp + p.hidden, g[k]);
                        }
                    }
                    if constexpr (RES) {
                        f2_t q[4];
                        oct_up<E>(fetch(j0, 2, k), q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[j] = f2_add(o[j], q[j]);
                    }
                    if (row && col[k] && (!GRADS || p.out)) {
                        oct_store<E>(p.out, here + k * P * 8, o);
                        if constexpr (DROP) {
                            const uint4 u = philox4x32(uint32_t(l + k * P), lrow, key);
                            const uint32_t words[4] = {u.x, u.y, u.z, u.w};
                            drop_pairs(o, words, drop_rule(p.drop));
                            oct_store<E>(p.out2, here + k * P * 8, o);
                        }
                    }
                }
                if constexpr (GRADS) {
                    if (row && !cur.partial && l == 0) {
                        if (p.ws.flag[lrow] || p.ws.state[lrow / kGroupRows] != 0) set_status(p.ws.hdr, kStDouble);
                        p.ws.flag[lrow] = 1;
                    }
                }
            }
            // the row's place is free again: the next row but kDepth - 1 goes there
            if (j0 + kDepth < kGroupRows) {
                request(cur, j0 + kDepth);
            } else {
                if (j0 + kDepth == kGroupRows) team_slots<P, GRADS>(p, group + stride, raw, nxt);
                request(nxt, j0 + kDepth - kGroupRows);
            }
        }
        if constexpr (kFwd) {
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
                const int j = l + o * P;
                if (j < kGroupRows && ((cur.on >> j) & 1)) {
                    const int64_t prow = group * kGroupRows + j;
                    if (p.mean) p.mean[prow] = own_mean[o];
                    if (p.rstd) p.rstd[prow] = own_rstd[o];
                }
            }
        }
        if constexpr (GRADS) {
            if constexpr (kTmem) umma::wait_st();
#pragma unroll
            for (int k = 0; k < NO; ++k) {
                f2_t (&dw)[4] = rw[kRegs ? k : 0], (&db)[4] = rb[kRegs ? k : 0];
                if constexpr (kTmem) sums_load(acc + k * 16, dw, db);
                float *to = sums + team * 2 * kCols + (l + k * P) * 8;
                pairs_store(to, dw);
                pairs_store(to + kCols, db);
                if (cur.kind == kItemQuarters && cur.partial && col[k]) {   // groups of a cut block stand alone
                    float *dst = p.ws.partial + (int64_t(cur.block) * kGroups + cur.slot0 / kGroupRows) * 2 * p.hidden + (l + k * P) * 8;
                    st_global_f2x4(dst, dw);
                    st_global_f2x4(dst + p.hidden, db);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) dw[j] = db[j] = 0;
                if constexpr (kTmem) sums_store(acc + k * 16, dw, db);
            }
            const int64_t rows = p.ws.n_rows - int64_t(cur.block) * kBlockRows;
            const int n_groups = rows >= kBlockRows ? kGroups : int((rows + kGroupRows - 1) / kGroupRows);
            if (cur.partial && l == 0 && cur.slot0 < rows) {
                uint8_t *state = p.ws.state + int64_t(cur.block) * kGroups + cur.slot0 / kGroupRows;
                if (*state != 0) set_status(p.ws.hdr, kStDouble);
                if (cur.kind == kItemQuarters) *state = 1;
                else if (cur.slot0 == 0) *state = uint8_t(n_groups);
            }
            __syncthreads();
            if (cur.kind == kItemWhole && cur.partial) {
                // lane (team of the block, l): NO pairs of the block's 2 kCols sums
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    const int at = ((k * kGroups + cur.slot0 / kGroupRows) * P + l) * 2, half = at / kCols, c = at - half * kCols;
                    const f2_t *from = reinterpret_cast<const f2_t *>(sums + (team / kGroups) * kGroups * 2 * kCols + at);
                    f2_t v[kGroups];
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) v[j] = from[j * kCols];
#pragma unroll
                    for (int j = 1; j < kGroups; ++j)
                        if (j < n_groups) v[0] = f2_add(v[0], v[j]);
                    if (c < p.hidden)
                        *reinterpret_cast<f2_t *>(p.ws.partial + int64_t(cur.block) * kGroups * 2 * p.hidden + half * p.hidden + c) = v[0];
                }
            }
            __syncthreads();                             // the sums are read
        }
        cur = nxt;
    }
    cp_async_wait<0>();
    if constexpr (kTmem) {
        umma::wait_st();                                 // this warp's last stores have landed before the columns are freed
        umma::fence_before();
        __syncthreads();
        umma::fence_after();
        if (tid < 32) umma::tmem_dealloc(acc, kTmemCols);
    }
}

template <class E, int P, int NO, int MODE, bool DROP, bool GRADS, bool RES>
static int ln_launch_narrow_t(const LnParams &p, cudaStream_t stream) {
    auto kern = ln_narrow_kernel<E, P, NO, MODE, DROP, GRADS, RES>;
    constexpr int smem = kNarrowDepth<NO> * kNarrowPieces<E, NO, MODE, RES> * kNarrowThreads * 16 + (GRADS ? kNarrowThreads * 64 * NO : 0);
    DeviceInfo *d = nullptr;
    if (int rc = device_info(&d)) return rc;
    const int64_t groups = GRADS ? p.n_items * kGroups : (p.n_rows + kGroupRows - 1) / kGroupRows;
    constexpr int kTeams = kNarrowThreads / P;
    static KernelInfo info;
    int regs = 0;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), smem, &regs)) return rc;
    int ctas = resident_ctas(regs, kNarrowThreads);
    if (ctas > kSmemPerSm / (smem + kSmemPerCta)) ctas = kSmemPerSm / (smem + kSmemPerCta);
    if (ctas < 1) return RMSNORM_ERR_HIDDEN;
    int64_t grid = (groups + kTeams - 1) / kTeams;
    if (grid == 0) return RMSNORM_OK;
    if (grid > int64_t(ctas) * d->sms) grid = int64_t(ctas) * d->sms;
    kern<<<unsigned(grid), kNarrowThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

// Lanes per row: the next power of two of hidden / 8, at least 4; rows of 257 to 512
// columns take 32 lanes with two octets each.
template <class E, int MODE, bool DROP, bool GRADS, bool RES>
int ln_launch_narrow(const LnParams &p, cudaStream_t s) {
    if (p.hidden <= 32) return ln_launch_narrow_t<E, 4, 1, MODE, DROP, GRADS, RES>(p, s);
    if (p.hidden <= 64) return ln_launch_narrow_t<E, 8, 1, MODE, DROP, GRADS, RES>(p, s);
    if (p.hidden <= 128) return ln_launch_narrow_t<E, 16, 1, MODE, DROP, GRADS, RES>(p, s);
    if (p.hidden <= 256) return ln_launch_narrow_t<E, 32, 1, MODE, DROP, GRADS, RES>(p, s);
    return ln_launch_narrow_t<E, 32, 2, MODE, DROP, GRADS, RES>(p, s);
}

template <class E>
int ln_run_narrow(const LnParams &p, bool bwd, bool grads, cudaStream_t s) {
    const bool drop = p.drop.state != nullptr;
    if (!bwd) {
        if (!p.res) return ln_launch_narrow<E, kLnFwd, false, false, false>(p, s);
        return drop ? ln_launch_narrow<E, kLnAdd, true, false, false>(p, s)
                    : ln_launch_narrow<E, kLnAdd, false, false, false>(p, s);
    }
    if (p.res) {
        if (grads) return drop ? ln_launch_narrow<E, kLnBwd, true, true, true>(p, s) : ln_launch_narrow<E, kLnBwd, false, true, true>(p, s);
        return drop ? ln_launch_narrow<E, kLnBwd, true, false, true>(p, s) : ln_launch_narrow<E, kLnBwd, false, false, true>(p, s);
    }
    if (grads) return drop ? ln_launch_narrow<E, kLnBwd, true, true, false>(p, s) : ln_launch_narrow<E, kLnBwd, false, true, false>(p, s);
    return drop ? ln_launch_narrow<E, kLnBwd, true, false, false>(p, s) : ln_launch_narrow<E, kLnBwd, false, false, false>(p, s);
}

}  // namespace rbi
