// C-ABI entry points of the rotary operators (sm_103a), the workspace of the
// weight gradients of the norms in front of them, and its final reduction.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "rotary_kernels.cuh"

using namespace rbi;

namespace {

constexpr int64_t kMaxHeadDim = 512, kMaxHeads = 65535;

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) != 0; }
bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// A tensor's strides.  A stride that is never taken (one slot, one head) is set to 0.
struct Strides {
    int64_t token, head;
};
Strides taken(int64_t token, int64_t head, int64_t n, int32_t heads) { return {n > 1 ? token : 0, heads > 1 ? head : 0}; }

int stride_check(const Strides &s) {
    if (s.token % 8 != 0 || s.head % 8 != 0) return RMSNORM_ERR_ALIGN;
    return s.token < 0 || s.head < 0 ? RMSNORM_ERR_STRIDE : RMSNORM_OK;
}

// Rows of an output must not overlap: heads inside token slots or slots inside heads.
int output_check(const Strides &s, int64_t n, int32_t heads, int64_t D) {
    const bool heads_inside = (heads == 1 || s.head >= D) && (n == 1 || s.token >= (heads - 1) * s.head + D);
    const bool slots_inside = (n == 1 || s.token >= D) && (heads == 1 || s.head >= (n - 1) * s.token + D);
    return heads_inside || slots_inside ? RMSNORM_OK : RMSNORM_ERR_STRIDE;
}

bool same(const Strides &a, const Strides &b) { return a.token == b.token && a.head == b.head; }

// Data pointers start on whole vectors of 8 elements.
bool off_data(const void *p, int32_t dtype) { return dtype == LAYERNORM_FP32 ? off32(p) : off16(p); }

int side_check(const rmsnorm_heads_t *h, int64_t n, int64_t D, int32_t dtype, bool norm, bool bwd) {
    if (h->heads < 1 || h->heads > kMaxHeads || h->reserved0 != 0) return RMSNORM_ERR_LAYOUT;
    if (n == 0) return RMSNORM_OK;
    if (!h->in || !h->out || (bwd && !h->dy)) return RMSNORM_ERR_NULL;
    if (off_data(h->in, dtype) || off_data(h->out, dtype) || (bwd && off_data(h->dy, dtype)) || (norm && off16(h->weight)))
        return RMSNORM_ERR_ALIGN;
    const Strides in = taken(h->in_token, h->in_head, n, h->heads), out = taken(h->out_token, h->out_head, n, h->heads),
                  dy = taken(h->dy_token, h->dy_head, n, h->heads);
    int rc;
    if ((rc = stride_check(in)) || (rc = stride_check(out)) || (rc = output_check(out, n, h->heads, D))) return rc;
    if (bwd && (rc = stride_check(dy))) return rc;
    if (h->out == h->in && !same(in, out)) return RMSNORM_ERR_STRIDE;
    if (bwd && h->out == h->dy && !same(dy, out)) return RMSNORM_ERR_STRIDE;
    return RMSNORM_OK;
}

HeadsParams side_params(const rmsnorm_heads_t *h, int64_t n) {
    HeadsParams s = {};
    const Strides in = taken(h->in_token, h->in_head, n, h->heads), out = taken(h->out_token, h->out_head, n, h->heads),
                  dy = taken(h->dy_token, h->dy_head, n, h->heads);
    s.in = h->in;
    s.dy = h->dy;
    s.w = h->weight;
    s.out = h->out;
    s.in_t = in.token;
    s.in_h = in.head;
    s.dy_t = dy.token;
    s.dy_h = dy.head;
    s.out_t = out.token;
    s.out_h = out.head;
    return s;
}

int ws_sizes_check(int64_t N, int32_t hq, int32_t hk, int64_t D) {
    if (D < 8 || D % 8 != 0 || D > kMaxHeadDim) return RMSNORM_ERR_HIDDEN;
    if (N < 0 || N >= (int64_t(1) << 31) || hq < 1 || hk < 0 || hq > kMaxHeads || hk > kMaxHeads) return RMSNORM_ERR_LAYOUT;
    return RMSNORM_OK;
}
int ws_check(const void *ws, int64_t N, int32_t hq, int32_t hk, int64_t D) {
    if (!ws) return RMSNORM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RMSNORM_ERR_ALIGN;
    return ws_sizes_check(N, hq, hk, D);
}

template <class E>
int run(const RotaryParams &p, int mode, bool interleaved, cudaStream_t s) {
    if (interleaved) return rotary_run_pairs<E, kNear>(p, mode, s);
    // halves of whole vectors, of whole pieces of 4 columns, or of 2
    if (p.first % 8 == 0 && p.rot % 16 == 0) return rotary_run_pairs<E, kHalf>(p, mode, s);
    return p.first % 4 == 0 && p.rot % 8 == 0 ? rotary_run_pairs<E, kQuad>(p, mode, s) : rotary_run_pairs<E, kSplit>(p, mode, s);
}

// mode as in rotary_run_pairs; back: turn the other way.
int call(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t D, float eps, int32_t dtype, int32_t param_dtype,
         const rmsnorm_layout_t *L, const rmsnorm_rotary_t *r, void *workspace, int mode, bool back, rmsnorm_stream_t stream) {
    if (dtype < LAYERNORM_BF16 || dtype > LAYERNORM_FP32 || (param_dtype != dtype && param_dtype != LAYERNORM_FP32))
        return RMSNORM_ERR_DTYPE;
    if (D < 8 || D % 8 != 0 || D > kMaxHeadDim) return RMSNORM_ERR_HIDDEN;
    if (!q || !L || !r) return RMSNORM_ERR_NULL;
    if (L->n_tokens < 0 || L->rows_per_token != 1 || L->reserved0 != 0 || L->n_logical_tokens < 0 ||
        L->n_logical_tokens >= (int64_t(1) << 31))
        return RMSNORM_ERR_LAYOUT;
    if (r->rotary_dim < 4 || r->rotary_dim % 4 != 0 || r->rotary_dim > D || r->first < 0 || r->first % 2 != 0 ||
        r->first > D - r->rotary_dim)
        return RMSNORM_ERR_HIDDEN;
    if (r->interleaved != 0 && r->interleaved != 1) return RMSNORM_ERR_LAYOUT;
    if (!std::isfinite(r->scale) || !(std::isfinite(eps) && eps >= 0.f)) return RMSNORM_ERR_VALUE;
    const int64_t n = L->n_tokens, lim = int64_t(1) << 31;
    const bool norm = mode > 0, bwd = mode > 1;
    int rc;
    if ((rc = side_check(q, n, D, dtype, norm, bwd)) || (k && (rc = side_check(k, n, D, dtype, norm, bwd)))) return rc;
    if (n >= lim || n * (q->heads + (k ? k->heads : 0)) >= lim) return RMSNORM_ERR_LAYOUT;
    if (workspace && (rc = ws_check(workspace, L->n_logical_tokens, q->heads, k ? k->heads : 0, D))) return rc;
    if (n == 0) return RMSNORM_OK;
    if (!L->tok_id || !r->position || !r->turns) return RMSNORM_ERR_NULL;
    if (off4(L->tok_id) || off4(r->position) || off16(r->turns)) return RMSNORM_ERR_ALIGN;
    // no tensor of one side is written while the other side may still read or write it
    if (k && (k->out == q->out || k->out == q->in || q->out == k->in || (bwd && (k->out == q->dy || q->out == k->dy))))
        return RMSNORM_ERR_LAYOUT;
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;

    RotaryParams p = {};
    p.side[0] = side_params(q, n);
    if (k) p.side[1] = side_params(k, n);
    p.hq = q->heads;
    p.heads = q->heads + (k ? k->heads : 0);
    p.tok_id = L->tok_id;
    p.position = r->position;
    p.turns = r->turns;
    p.n_tokens = n;
    p.active = L->n_logical_tokens < 1 ? 1 : L->n_logical_tokens < n ? L->n_logical_tokens : n;
    p.D = int32_t(D);
    p.rot = r->rotary_dim;
    p.first = r->first;
    p.params_f32 = param_dtype == LAYERNORM_FP32 ? 1 : 0;
    p.in_place = mode == 0 && q->out == q->in && (!k || k->out == k->in) ? 1 : 0;
    p.scale = r->scale;
    p.scale_sin = back ? -r->scale : r->scale;
    p.eps = eps;
    p.inv_d = float(1.0 / double(D));
    if (workspace) p.ws = qk_ws(workspace, L->n_logical_tokens, q->heads, k ? k->heads : 0, D);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
        case LAYERNORM_BF16: return run<__nv_bfloat16>(p, mode, r->interleaved, s);
        case LAYERNORM_FP16: return run<__half>(p, mode, r->interleaved, s);
        default: return run<float>(p, mode, r->interleaved, s);
    }
}

// ----------------------------------------------------------------- workspace kernels

__global__ void qk_begin_kernel(QkWs ws) {
    const int64_t tid = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, n = int64_t(gridDim.x) * blockDim.x;
    const int64_t n16 = (reinterpret_cast<uint8_t *>(ws.partial) - reinterpret_cast<uint8_t *>(ws.flag)) / 16;
    uint4 *f = reinterpret_cast<uint4 *>(ws.flag);
    for (int64_t i = tid; i < n16; i += n) f[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        ws.hdr->n_rows = ws.n;
        ws.hdr->hidden = ws.sizes;
        ws.hdr->n_blocks = ws.groups;
        ws.hdr->status = 0;
        ws.hdr->magic = kQkMagic;
    }
}

constexpr int kFinalCtas = 8, kFinalWarps = 16;
// Whether one CTA for 32 columns does without a cluster.
bool final_alone(const QkWs &ws) { return ws.groups <= 256 && ws.cut.slots <= 8; }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 plus(const float4 &a, const float4 &b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

// A group's sum of four columns (col on, `have`: there are any) over the partial sums `slots` from
// its tokens' own, in the order in which a warp of the backward pass adds up a whole
// group.  The whole warp does it for one group: quarter q takes the partial sums q, q + 4, ..., all loads of
// one at once, and everyone adds the quarters' sums up in order.
__device__ __noinline__ float4 qk_loose_group(const QkWs &ws, int64_t g, int slot0, int slots, int col, bool have, bool check) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = g * ws.group;
    const int n = ws.n - t0 < ws.group ? int(ws.n - t0) : ws.group;
    const uint32_t there = __ballot_sync(kFull, lane < n && ws.flag[t0 + (lane < n ? lane : 0)] == 2);
    if (check && lane == 0 && there != (1u << n) - 1u) qk_report(ws, kStMissing);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v = zero;
    for (int c0 = 0; c0 < slots; c0 += 4) {
        const int c = c0 + (lane >> 3);
        const float *src = ws.spill + ((slot0 + c) * ws.n + t0) * ws.D + col;
        float4 x[kMostGroup];
#pragma unroll
        for (int i = 0; i < kMostGroup; ++i) x[i] = have && c < slots && i < n ? *reinterpret_cast<const float4 *>(src + i * ws.D) : zero;
        float4 u = zero, s = zero;
        bool any = false;                                // of the share
        int left = ws.share;
#pragma unroll
        for (int i = 0; i < kMostGroup; ++i) {
            if (i < n) {
                if ((there >> i) & 1) {
                    s = any ? plus(s, x[i]) : x[i];
                    any = true;
                }
                if (--left == 0 || i + 1 == n) {
                    if (!any) s = zero;
                    u = i < ws.share ? s : plus(u, s);
                    any = false;
                    left = ws.share;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int from = 8 * k + (lane & 7);
            const float4 w = make_float4(__shfl_sync(kFull, u.x, from), __shfl_sync(kFull, u.y, from), __shfl_sync(kFull, u.z, from),
                                         __shfl_sync(kFull, u.w, from));
            if (c0 + k < slots) v = c0 + k ? plus(v, w) : w;
        }
    }
    return v;
}

// Adds the groups [g, g1) of a quarter-warp's share, at most GROUPS of them, to acc; the loads of SLOTS
// partial sums of each go out together.
template <int GROUPS, int SLOTS>
__device__ __forceinline__ float4 qk_add_groups(const QkWs &ws, float4 acc, int64_t g, int64_t g1, int slot0, int slots, int col, bool have,
                                                bool check) {
    const int lane = threadIdx.x & 31;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *src = ws.partial + (slot0 * ws.groups + g) * ws.D + col;
    bool in[GROUPS], loose[GROUPS];
    float4 v[GROUPS];
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        in[j] = have && g + j < g1;
        loose[j] = g + j < g1 && !ws.whole[g + j];
    }
    // (a partial that is not there is read all the same: its memory is)
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) v[j] = in[j] ? *reinterpret_cast<const float4 *>(src + j * ws.D) : zero;
    for (int c = 1; c < slots; c += SLOTS) {
        float4 x[SLOTS][GROUPS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int j = 0; j < GROUPS; ++j)
                x[i][j] = in[j] && c + i < slots ? *reinterpret_cast<const float4 *>(src + ((c + i) * ws.groups + j) * ws.D) : zero;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
#pragma unroll
            for (int j = 0; j < GROUPS; ++j)
                if (c + i < slots) v[j] = plus(v[j], x[i][j]);
    }
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        uint32_t left = __ballot_sync(kFull, loose[j]) & 0x01010101u;
        while (left) {
            const int from = __ffs(left) - 1;
            left &= left - 1;
            const int64_t its = int64_t(__shfl_sync(kFull, (unsigned long long)(g + j), from));
            const float4 u = qk_loose_group(ws, its, slot0, slots, col, have, check);
            if (lane >> 3 == from >> 3) v[j] = u;
        }
        if (in[j]) acc = plus(acc, v[j]);
    }
    return acc;
}

// Both weight gradients in one launch: a cluster of CTAS takes 32 columns of one of them,
// its CTAs x 16 warps x 4 quarter-warps consecutive shares of the groups, first all first quarters.  The partial sums
// of a group from the first chunk to the last, the groups of a share likewise, then the
// four shares of a warp in pairs, the warps, the CTAs: an order that depends on the sizes
// alone.  What bounds it: latency (a launch, the header, a share's 1 to 3 rounds of loads,
// the cluster's exchange).  33,384 tokens, 5 partial sums of 128 columns a group, 12.8 MB: 7.3 us; up
// to 256 groups of 8 partial sums one CTA does without the exchange (46 tokens: 3.9 us; before loads went out
// eight at once 5.1, 5.7 in a cluster).
template <int CTAS>
__device__ __forceinline__ void qk_finalize(const QkWs &ws, float scale, float *dq, float *dk, int slices) {
    __shared__ float4 part[kFinalWarps][8];
    __shared__ float whole[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!qk_header_ok(ws)) {                             // the same for the whole cluster
        if (threadIdx.x == 0) qk_report(ws, kStHeader);
        return;
    }
    const bool keys = int(blockIdx.x) >= slices;
    const int col0 = (int(blockIdx.x) - (keys ? slices : 0)) * 32, col = col0 + (lane & 7) * 4;
    const int slot0 = keys ? ws.cut.q_slots : 0, slots = keys ? ws.cut.slots - ws.cut.q_slots : ws.cut.q_slots;
    constexpr int kShares = CTAS * kFinalWarps * 4;
    const int64_t per = (ws.groups + kShares - 1) / kShares;
    // (few groups: one a warp, so that cut ones are not added up one after the other; all groups cut, this way and four a
    // warp: 200 tokens of 59+7 heads of 128 12 and 20 us, 504 of 60+3 of 8 18 and 55; above 128 groups it loses a little,
    // 1,140 of 59+7 of 128 10.8 and 8.4)
    const int64_t g0 = ((lane >> 3) * (CTAS * kFinalWarps) + int(blockIdx.y) * kFinalWarps + warp) * per;
    const int64_t g1 = g0 + per < ws.groups ? g0 + per : ws.groups;
    const bool check = blockIdx.x == 0, have = col < ws.D;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // (the warp's quarters go together)
    if (per < 3)
        for (int64_t i = 0; i < per; ++i) acc = qk_add_groups<1, 8>(ws, acc, g0 + i, g1, slot0, slots, col, have, check);
    else
        for (int64_t i = 0; i < per; i += 4) acc = qk_add_groups<4, 4>(ws, acc, g0 + i, g1, slot0, slots, col, have, check);
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1)
        acc = plus(acc, make_float4(__shfl_xor_sync(kFull, acc.x, o), __shfl_xor_sync(kFull, acc.y, o),
                                    __shfl_xor_sync(kFull, acc.z, o), __shfl_xor_sync(kFull, acc.w, o)));
    if (lane < 8) part[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
        const float *f = reinterpret_cast<const float *>(part);
        float v = f[lane];
#pragma unroll
        for (int i = 1; i < kFinalWarps; ++i) v = __fadd_rn(v, f[i * 32 + lane]);
        whole[lane] = v;
    }
    if constexpr (CTAS > 1) cluster_barrier();
    if (blockIdx.y == 0 && warp == 0) {
        float v = whole[lane];
        if constexpr (CTAS > 1) {
            const uint32_t at = smem_addr(&whole[lane]);
#pragma unroll
            for (int i = 1; i < CTAS; ++i) v = __fadd_rn(v, ld_cluster_f32(map_to_rank(at, uint32_t(i))));
        }
        float *dst = keys ? dk : dq;
        if (dst && col0 + lane < ws.D) dst[col0 + lane] = scale != 1.f ? __fmul_rn(v, scale) : v;
    }
    if constexpr (CTAS > 1) cluster_barrier();           // the sums stay until they are read
}
__global__ void __cluster_dims__(1, kFinalCtas, 1) __launch_bounds__(kFinalWarps * 32)
    qk_finalize_kernel(const __grid_constant__ QkWs ws, float scale, float *dq, float *dk, int slices) {
    qk_finalize<kFinalCtas>(ws, scale, dq, dk, slices);
}
__global__ void __launch_bounds__(kFinalWarps * 32)
    qk_finalize_small_kernel(const __grid_constant__ QkWs ws, float scale, float *dq, float *dk, int slices) {
    qk_finalize<1>(ws, scale, dq, dk, slices);
}

}  // namespace

extern "C" int rotary_fwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, int32_t dtype,
                          const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary, rmsnorm_stream_t stream) {
    return call(q, k, head_dim, 0.f, dtype, dtype, layout, rotary, nullptr, 0, false, stream);
}

extern "C" int rotary_bwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, int32_t dtype,
                          const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary, rmsnorm_stream_t stream) {
    return call(q, k, head_dim, 0.f, dtype, dtype, layout, rotary, nullptr, 0, true, stream);
}

extern "C" int qk_norm_rotary_fwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, float eps,
                                  int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout,
                                  const rmsnorm_rotary_t *rotary, rmsnorm_stream_t stream) {
    return call(q, k, head_dim, eps, dtype, param_dtype, layout, rotary, nullptr, 1, false, stream);
}

extern "C" int qk_norm_rotary_bwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, float eps,
                                  int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout,
                                  const rmsnorm_rotary_t *rotary, void *workspace, rmsnorm_stream_t stream) {
    return call(q, k, head_dim, eps, dtype, param_dtype, layout, rotary, workspace, 2, true, stream);
}

extern "C" size_t qk_norm_workspace_bytes(int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads, int64_t head_dim) {
    if (ws_sizes_check(n_logical_tokens, q_heads, k_heads, head_dim)) return 0;
    return size_t(QkWsLayout(n_logical_tokens, q_heads, k_heads, head_dim).total);
}

extern "C" int qk_norm_begin(void *workspace, size_t bytes, int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads,
                             int64_t head_dim, rmsnorm_stream_t stream) {
    int rc = ws_check(workspace, n_logical_tokens, q_heads, k_heads, head_dim);
    if (rc) return rc;
    if (bytes < qk_norm_workspace_bytes(n_logical_tokens, q_heads, k_heads, head_dim)) return RMSNORM_ERR_WORKSPACE;
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;
    int64_t blocks = (n_logical_tokens / 4 + 255) / 256;
    if (blocks > int64_t(d->sms) * 4) blocks = int64_t(d->sms) * 4;
    if (blocks < 1) blocks = 1;
    qk_begin_kernel<<<unsigned(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        qk_ws(workspace, n_logical_tokens, q_heads, k_heads, head_dim));
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

extern "C" int qk_norm_finalize(void *workspace, int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads,
                                int64_t head_dim, float grad_scale, float *dq_weight, float *dk_weight,
                                rmsnorm_stream_t stream) {
    if (!std::isfinite(grad_scale)) return RMSNORM_ERR_VALUE;
    int rc = ws_check(workspace, n_logical_tokens, q_heads, k_heads, head_dim);
    if (rc) return rc;
    if (!dq_weight && !dk_weight) return RMSNORM_ERR_NULL;
    if (dk_weight && k_heads == 0) return RMSNORM_ERR_LAYOUT;
    if (off4(dq_weight) || off4(dk_weight)) return RMSNORM_ERR_ALIGN;
    // both are written at once
    if (dq_weight && dk_weight) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(dq_weight), b = reinterpret_cast<uintptr_t>(dk_weight);
        if ((a < b ? b - a : a - b) < uintptr_t(head_dim) * 4) return RMSNORM_ERR_LAYOUT;
    }
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;
    const int slices = int(head_dim + 31) / 32;
    const unsigned gx = unsigned(slices * (k_heads ? 2 : 1));
    const QkWs ws = qk_ws(workspace, n_logical_tokens, q_heads, k_heads, head_dim);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!final_alone(ws))
        qk_finalize_kernel<<<dim3(gx, kFinalCtas), kFinalWarps * 32, 0, s>>>(ws, grad_scale, dq_weight, dk_weight, slices);
    else
        qk_finalize_small_kernel<<<gx, kFinalWarps * 32, 0, s>>>(ws, grad_scale, dq_weight, dk_weight, slices);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

extern "C" int qk_norm_status(const void *workspace, rmsnorm_stream_t stream, int32_t *status) {
    return rmsnorm_dweight_status(workspace, stream, status);
}
