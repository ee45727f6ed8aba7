// Workspace set-up and the final reduction of the layer norm's parameter
// gradients.  Included by the C-ABI translation unit only.
#pragma once
#include "layernorm_kernels.cuh"

namespace rbi {

__global__ void ln_begin_kernel(LnWs ws) {
    const int64_t tid = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, n = int64_t(gridDim.x) * blockDim.x;
    uint4 *b4 = reinterpret_cast<uint4 *>(ws.state);
    const int64_t n16 = (reinterpret_cast<uint8_t *>(ws.partial) - ws.state) / 16;
    for (int64_t i = tid; i < n16; i += n) b4[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        ws.hdr->n_rows = ws.n_rows;
        ws.hdr->hidden = ws.hidden;
        ws.hdr->n_blocks = ws.n_blocks;
        ws.hdr->status = 0;
        ws.hdr->magic = kLnMagic;
    }
}

constexpr int kLnTreeCols = 32;                          // columns of [dweight | dbias] per CTA: 8 lanes of 4
constexpr int kLnTreeBlocks = 32;                        // inputs per CTA

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

// Four columns of block b from column col of [dweight | dbias]: the groups from
// the first to the last, each from a stored partial or folded from its spilled
// rows.  All stored partials are requested before any is used.  check: report
// rows that are missing or arrived twice (one CTA per block does).
__device__ __forceinline__ float4 ln_block_value(const LnWs &ws, int64_t b, int64_t col, uint64_t state, bool check,
                                                 int &bad) {
    const int64_t H2 = 2 * ws.hidden;
    const float *part = ws.partial + b * kGroups * H2 + col;
    const int64_t left = ws.n_rows - b * kBlockRows;
    const int rows = left < kBlockRows ? int(left) : kBlockRows, groups = (rows + kGroupRows - 1) / kGroupRows;
    float4 v[kGroups];
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
        if ((state >> (8 * j)) & 0xff) v[j] = *reinterpret_cast<const float4 *>(part + j * H2);
    const uint64_t *flags = reinterpret_cast<const uint64_t *>(ws.flag) + b * kGroups;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int next = 0;                                        // first group not yet taken
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const int c = int((state >> (8 * j)) & 0xff);
        if (j < next) {                                  // inside the fold of the block's first groups
            if (check && (c || flags[j])) bad |= kStDouble;
            continue;
        }
        if (j >= groups) continue;
        float4 g;
        if (c) {
            g = v[j];
            next = j + c;
            if (check && flags[j]) bad |= kStDouble;
        } else {
            next = j + 1;
            g = make_float4(0.f, 0.f, 0.f, 0.f);
            const bool is_w = col < ws.hidden;
            const int64_t c0 = is_w ? col : col - ws.hidden;
            for (int r = j * kGroupRows; r < (j + 1) * kGroupRows && r < rows; ++r) {
                const int64_t row = b * kBlockRows + r;
                if (!ws.flag[row]) {
                    bad |= kStMissing;
                    continue;
                }
                const float4 dy = *reinterpret_cast<const float4 *>(ws.spill + row * H2 + ws.hidden + c0);
                if (is_w) {
                    const float4 xh = *reinterpret_cast<const float4 *>(ws.spill + row * H2 + c0);
                    g = make_float4(__fmaf_rn(dy.x, xh.x, g.x), __fmaf_rn(dy.y, xh.y, g.y), __fmaf_rn(dy.z, xh.z, g.z),
                                    __fmaf_rn(dy.w, xh.w, g.w));
                } else {
                    g = add4(g, dy);
                }
            }
        }
        acc = j == 0 ? g : add4(acc, g);
    }
    return acc;
}

// One pass of the pairwise tree with odd carry over n_in inputs (block values in
// the first pass, then the results of the one before): CTA (g, c) reduces inputs
// [32 g, 32 g + 32) of 32 columns to one node.  Eight lanes hold the columns of
// an input, a warp four inputs, which meet by shuffles; the eight warps through
// shared memory.  All loads of a pass are in flight at once; what bounds the
// first pass is reading the partials (mostly from L2), the others are latency.
__global__ void __launch_bounds__(256) ln_tree_kernel(LnWs ws, const float *in, float *out_w, float *out_b,
                                                      int64_t out_stride, int64_t n_in, float scale) {
    __shared__ float4 val[8][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = tid & 7, i = tid >> 3;
    const int64_t H2 = 2 * ws.hidden, col = int64_t(blockIdx.y) * kLnTreeCols + part * 4;
    const int64_t first = int64_t(blockIdx.x) * kLnTreeBlocks;
    if (!in && !ln_header_ok(ws)) {
        if (tid == 0) set_status(ws.hdr, kStHeader);
        return;
    }
    const int m = n_in - first < kLnTreeBlocks ? int(n_in - first) : kLnTreeBlocks;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    int bad = 0;
    if (i < m && col < H2) {
        if (in) v = *reinterpret_cast<const float4 *>(in + (first + i) * H2 + col);
        else v = ln_block_value(ws, first + i, col, reinterpret_cast<const uint64_t *>(ws.state)[first + i],
                                blockIdx.y == 0, bad);
    }
    if (bad) set_status(ws.hdr, bad);
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {                  // inputs 1, then 2 apart
        float4 u;
        u.x = __shfl_down_sync(kFull, v.x, o);
        u.y = __shfl_down_sync(kFull, v.y, o);
        u.z = __shfl_down_sync(kFull, v.z, o);
        u.w = __shfl_down_sync(kFull, v.w, o);
        if (i + (o >> 3) < m) v = add4(v, u);
    }
    if (lane < 8) val[warp][part] = v;
    __syncthreads();
    if (warp == 0) {                                     // one column per lane: the warps' quadruples
        float x[8];
        const float *f = reinterpret_cast<const float *>(val);
        const int n = (m + 3) / 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = f[k * kLnTreeCols + lane];
#pragma unroll
        for (int s = 1; s < 8; s <<= 1)
#pragma unroll
            for (int k = 0; k + s < 8; k += 2 * s)
                if (k + s < n) x[k] = __fadd_rn(x[k], x[k + s]);
        const int64_t c = int64_t(blockIdx.y) * kLnTreeCols + lane;
        const float r = scale != 1.f ? __fmul_rn(x[0], scale) : x[0];   // scaled only at the root
        if (c < H2) {
            float *dst = c < ws.hidden ? out_w : out_b;
            if (dst) dst[blockIdx.x * out_stride + (c < ws.hidden ? c : c - ws.hidden)] = r;
        }
    }
}

}  // namespace rbi
