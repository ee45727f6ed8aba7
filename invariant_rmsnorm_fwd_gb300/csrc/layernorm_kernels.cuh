// Row kernels of the batch-invariant layer norm (sm_103a): one CTA per row
// (forward, input gradient) or per 8-row group of a plan item (parameter
// gradients), a row held in registers.
#pragma once
#include <cuda_fp16.h>

#include "philox.cuh"
#include "rbi_device.cuh"

namespace rbi {

constexpr int kGroupRows = 8;                            // rows of one group of the parameter-gradient order
constexpr int kGroups = kBlockRows / kGroupRows;         // groups of a logical block
constexpr uint64_t kLnMagic = 0x3149422d4e4c3352ull;

// State byte of a group: 0 nothing, c > 0 a partial in its slot that covers the
// group and the c - 1 behind it (a fold from the block's first group on, c up
// to 8; other groups are stored alone).

struct LnWs {
    WsHeader *hdr;
    uint8_t *state;                  // [nb][8], see above
    uint8_t *flag;                   // [N] 1 = row spilled
    float *partial;                  // [nb][8][2][H]: dweight and dbias of a group, or of the fold that
                                     //   starts there
    float *scratch_a, *scratch_b;    // [ceil(nb/32)][2][H]
    float *spill;                    // [N][2][H]: xhat and dy of spilled rows
    int64_t n_rows, hidden, n_blocks;
};

struct LnWsLayout {
    int64_t off_state, off_flag, off_partial, off_sa, off_sb, off_spill, total;
    LnWsLayout(int64_t N, int64_t H) {
        const int64_t nb = (N + kBlockRows - 1) / kBlockRows, ng = (nb + 31) / 32;
        off_state = 256;
        off_flag = align256(off_state + nb * kGroups);
        off_partial = align256(off_flag + N);
        off_sa = align256(off_partial + nb * kGroups * 2 * H * 4);
        off_sb = align256(off_sa + ng * 2 * H * 4);
        off_spill = align256(off_sb + ng * 2 * H * 4);
        total = align256(off_spill + N * 2 * H * 4);
    }
};

inline LnWs ln_ws(void *base, int64_t N, int64_t H) {
    const LnWsLayout L(N, H);
    uint8_t *b = static_cast<uint8_t *>(base);
    LnWs w;
    w.hdr = reinterpret_cast<WsHeader *>(b);
    w.state = b + L.off_state;
    w.flag = b + L.off_flag;
    w.partial = reinterpret_cast<float *>(b + L.off_partial);
    w.scratch_a = reinterpret_cast<float *>(b + L.off_sa);
    w.scratch_b = reinterpret_cast<float *>(b + L.off_sb);
    w.spill = reinterpret_cast<float *>(b + L.off_spill);
    w.n_rows = N;
    w.hidden = H;
    w.n_blocks = (N + kBlockRows - 1) / kBlockRows;
    return w;
}

__device__ __forceinline__ bool ln_header_ok(const LnWs &ws) {
    const WsHeader *h = ws.hdr;
    return h->magic == kLnMagic && h->n_rows == ws.n_rows && h->hidden == ws.hidden;
}

struct LnParams {
    const void *x;                   // x, or h in the backward of the residual add
    const void *dy;
    const void *res;                 // residual input (forward) or dres (backward); null = none
    const void *w, *b;               // null = 1 / 0
    void *out;                       // y (forward); dx or dh (backward, may be null)
    void *out2;                      // h (forward of the residual add); dropped dx (backward)
    float *mean, *rstd;              // forward, optional
    DropParams drop;
    float grad_scale, eps, inv_h;
    int32_t params_f32;              // weight and bias are FP32 (else the rows' type)
    int32_t hidden, rpt;
    const int32_t *tok_id;
    int64_t n_rows, token_stride;
    const PlanItem *items;
    int64_t n_items;
    LnWs ws;
};

// ----------------------------------------------------------------- vectors of 8 elements

template <class E>
struct Vec;                          // packed vector of 8 elements of E
template <>
struct Vec<__nv_bfloat16> { uint4 q; };
template <>
struct Vec<__half> { uint4 q; };
template <>
struct Vec<float> { uint4 q, r; };

template <class E>
__device__ __forceinline__ Vec<E> vload(const void *base, int64_t elem) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const E *>(base) + elem);
    Vec<E> v;
    v.q = p[0];
    if constexpr (sizeof(E) == 4) v.r = p[1];
    return v;
}
template <class E>
__device__ __forceinline__ void vstore(void *base, int64_t elem, const Vec<E> &v) {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<E *>(base) + elem);
    p[0] = v.q;
    if constexpr (sizeof(E) == 4) p[1] = v.r;
}

__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16> &v, float (&f)[8]) {
    const uint32_t w[4] = {v.q.x, v.q.y, v.q.z, v.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Vec<__half> &v, float (&f)[8]) {
    const uint32_t w[4] = {v.q.x, v.q.y, v.q.z, v.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
__device__ __forceinline__ void unpack(const Vec<float> &v, float (&f)[8]) {
    f[0] = __uint_as_float(v.q.x); f[1] = __uint_as_float(v.q.y); f[2] = __uint_as_float(v.q.z); f[3] = __uint_as_float(v.q.w);
    f[4] = __uint_as_float(v.r.x); f[5] = __uint_as_float(v.r.y); f[6] = __uint_as_float(v.r.z); f[7] = __uint_as_float(v.r.w);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec<__nv_bfloat16> &v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_to_bf16x2(f2_make(f[2 * i], f[2 * i + 1]));
    v.q = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec<__half> &v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    v.q = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec<float> &v) {
    v.q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    v.r = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
}

// 8 parameters of type E, or FP32 when f32 is set, from column 8v; `none` where the pointer is null.
template <class E>
__device__ __forceinline__ void load_param(const void *p, int f32, int v, float none, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = none;
    } else if (f32) {
        unpack(vload<float>(p, int64_t(v) * 8), f);
    } else {
        unpack(vload<E>(p, int64_t(v) * 8), f);
    }
}

// ----------------------------------------------------------------- block sum

// Sum over the CTA in a fixed order (warp butterfly, then the warps from the
// first to the last); every thread gets the same value.  `red` has two
// alternating halves, so one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float *red, int &turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    const int nw = blockDim.x >> 5;
    float *r = red + (turn & 1) * 32;
    ++turn;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = r[0];
    for (int i = 1; i < nw; ++i) s = __fadd_rn(s, r[i]);
    return s;
}

// Offset of a physical row's first element.
__device__ __forceinline__ int64_t ln_row(const LnParams &p, int64_t prow) {
    const int64_t t = prow / p.rpt;
    return t * p.token_stride + (prow - t * p.rpt) * int64_t(p.hidden);
}

// NV vectors of 8 columns per thread: vector k of thread i is i + k * blockDim.
// BWD: backward; GRADS: plan items with parameter gradients.
template <class E, int NV, bool BWD, bool GRADS>
__global__ void __launch_bounds__(512) ln_rows_kernel(const __grid_constant__ LnParams p) {
    __shared__ float red[64];
    int turn = 0;
    const int V = p.hidden >> 3;
    const DropKey key = p.drop.state ? drop_key(p.drop) : DropKey{0, 0, 0, 0};
    float dw[GRADS ? NV : 1][8], db[GRADS ? NV : 1][8];
    const PlanItem *it = nullptr;
    int slot0 = 0;
    bool partial = false;
    if constexpr (GRADS) {
        it = p.items + blockIdx.x / kGroups;
        slot0 = int(blockIdx.x % kGroups) * kGroupRows;
        if (!ln_header_ok(p.ws)) {
            if (threadIdx.x == 0) set_status(p.ws.hdr, kStHeader);
            return;
        }
        partial = it->kind == kItemWhole || (it->kind == kItemQuarters && ((it->quarters >> (slot0 / 16)) & 1));
        if (it->kind == kItemQuarters && !partial) return;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.f;
    }
    bool any = false;
    const int n_slots = GRADS ? kGroupRows : 1;
#pragma unroll 1
    for (int s = 0; s < n_slots; ++s) {
        int64_t prow = blockIdx.x, g;
        if constexpr (GRADS) {
            prow = it->prow[slot0 + s];
            g = it->lrow[slot0 + s];
            if (prow < 0) continue;
            if (prow >= p.n_rows || g < 0 || g >= p.ws.n_rows) {
                if (threadIdx.x == 0) set_status(p.ws.hdr, kStPlan);
                continue;
            }
        } else {
            const int64_t t = prow / p.rpt;
            const int32_t id = p.tok_id[t];
            if (id < 0) return;
            g = int64_t(id) * p.rpt + (prow - t * p.rpt);
        }
        any = true;
        const int64_t off = ln_row(p, prow);
        float x[NV][8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < V) {
                unpack(vload<E>(p.x, off + 8 * v), x[k]);
                if constexpr (!BWD) {
                    if (p.res) {
                        float r[8];
                        unpack(vload<E>(p.res, off + 8 * v), r);
                        const uint32_t keep = p.drop.state ? keep_bits(v, uint32_t(g), key, p.drop.t) : 0xffu;
                        const float sc = p.drop.state ? p.drop.scale : 1.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = (keep >> e) & 1 ? __fmaf_rn(x[k][e], sc, r[e]) : r[e];
                        Vec<E> h;
                        pack(r, h);
                        vstore<E>(p.out2, off + 8 * v, h);
                        unpack(h, x[k]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __fadd_rn(sum, x[k][e]);
            }
        }
        const float mean = __fmul_rn(block_sum(sum, red, turn), p.inv_h);
        float m2 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (int(threadIdx.x + k * blockDim.x) < V) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[k][e] = __fsub_rn(x[k][e], mean);
                    m2 = __fmaf_rn(x[k][e], x[k][e], m2);
                }
            }
        }
        const float var = __fmul_rn(block_sum(m2, red, turn), p.inv_h);
        const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(var, p.eps)));
        if constexpr (!BWD) {
            if (threadIdx.x == 0) {
                if (p.mean) p.mean[prow] = mean;
                if (p.rstd) p.rstd[prow] = rstd;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                if (v < V) {
                    float w[8], b[8];
                    load_param<E>(p.w, p.params_f32, v, 1.f, w);
                    load_param<E>(p.b, p.params_f32, v, 0.f, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[k][e] = __fmaf_rn(__fmul_rn(x[k][e], rstd), w[e], b[e]);
                    Vec<E> o;
                    pack(x[k], o);
                    vstore<E>(p.out, off + 8 * v, o);
                }
            }
        } else {
            float a[NV][8];
            float sa = 0.f, sc = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                if (v < V) {
                    float w[8];
                    load_param<E>(p.w, p.params_f32, v, 1.f, w);
                    unpack(vload<E>(p.dy, off + 8 * v), a[k]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[k][e] = __fmul_rn(x[k][e], rstd);
                        if constexpr (GRADS) {
                            dw[k][e] = __fmaf_rn(a[k][e], x[k][e], dw[k][e]);
                            db[k][e] = __fadd_rn(db[k][e], a[k][e]);
                        }
                    }
                    if constexpr (GRADS) {
                        if (!partial) {
                            float *sp = p.ws.spill + g * 2 * p.hidden + 8 * v;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                sp[e] = x[k][e];
                                sp[p.hidden + e] = a[k][e];
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        a[k][e] = __fmul_rn(a[k][e], w[e]);
                        sa = __fadd_rn(sa, a[k][e]);
                        sc = __fmaf_rn(a[k][e], x[k][e], sc);
                    }
                }
            }
            if constexpr (GRADS) {
                if (!partial && threadIdx.x == 0) {
                    if (p.ws.flag[g] || p.ws.state[g / kGroupRows] != 0) set_status(p.ws.hdr, kStDouble);
                    p.ws.flag[g] = 1;
                }
            }
            const float ma = __fmul_rn(block_sum(sa, red, turn), p.inv_h);
            const float mc = __fmul_rn(block_sum(sc, red, turn), p.inv_h);
            const float r = __fmul_rn(rstd, p.grad_scale);
            if (p.out) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int v = threadIdx.x + k * blockDim.x;
                    if (v < V) {
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = __fmul_rn(r, __fsub_rn(__fsub_rn(a[k][e], ma), __fmul_rn(x[k][e], mc)));
                        if (p.res) {
                            float q[8];
                            unpack(vload<E>(p.res, off + 8 * v), q);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __fadd_rn(o[e], q[e]);
                        }
                        Vec<E> t;
                        pack(o, t);
                        vstore<E>(p.out, off + 8 * v, t);
                        if (p.drop.state) {
                            const uint32_t keep = keep_bits(v, uint32_t(g), key, p.drop.t);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = (keep >> e) & 1 ? __fmul_rn(o[e], p.drop.scale) : 0.f;
                            pack(o, t);
                            vstore<E>(p.out2, off + 8 * v, t);
                        }
                    }
                }
            }
        }
    }
    if constexpr (GRADS) {
        if (partial && any) {
            const int64_t grp = int64_t(it->block) * kGroups + slot0 / kGroupRows;
            if (it->block < 0 || it->block >= p.ws.n_blocks) {
                if (threadIdx.x == 0) set_status(p.ws.hdr, kStPlan);
                return;
            }
            float *dst = p.ws.partial + grp * 2 * p.hidden;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                if (v < V) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dst[8 * v + e] = dw[k][e];
                        dst[p.hidden + 8 * v + e] = db[k][e];
                    }
                }
            }
            if (threadIdx.x == 0) {
                if (p.ws.state[grp] != 0) set_status(p.ws.hdr, kStDouble);
                p.ws.state[grp] = 1;
            }
        }
    }
}

}  // namespace rbi
