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

constexpr int kLnTreeCols = 32;                          // columns of [dweight | dbias] per CTA
constexpr int kLnTreeBlocks = 128;                       // blocks per round: 8 lanes (4 columns each) per block

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

// Four columns of block b from column col of [dweight | dbias]: the groups from
// the first to the last, each from a stored partial or folded from its spilled
// rows.  All stored partials are requested before any is used.
__device__ __forceinline__ float4 ln_block_value(const LnWs &ws, int64_t b, int64_t col, uint64_t state, int &bad) {
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
            if (c || flags[j]) bad |= kStDouble;
            continue;
        }
        if (j >= groups) continue;
        float4 g;
        if (c) {
            g = v[j];
            next = j + c;
            if (flags[j]) bad |= kStDouble;
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

// Pairwise tree with odd carry over n_in inputs (block values, or the results
// of an earlier pass): CTA (g, c) reduces inputs [g m, (g + 1) m), m = rounds *
// 128 a power of two, so each result is one node of the tree over all inputs.
// Eight lanes hold the 32 columns of a block; the four blocks of a warp meet by
// shuffles, the warps and the rounds through shared memory.
__global__ void __launch_bounds__(1024) ln_tree_kernel(LnWs ws, const float *in, float *out_w, float *out_b,
                                                       int64_t out_stride, int64_t n_in, int rounds, float scale) {
    __shared__ float4 val[32][8];
    __shared__ float node[4][kLnTreeCols];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = tid & 7;
    const int64_t H2 = 2 * ws.hidden, col = int64_t(blockIdx.y) * kLnTreeCols + part * 4;
    const int64_t base = int64_t(blockIdx.x) * rounds * kLnTreeBlocks;
    if (!in && !ln_header_ok(ws)) {
        if (tid == 0) set_status(ws.hdr, kStHeader);
        return;
    }
    int used = 0;
    for (int r = 0; r < rounds; ++r) {
        const int64_t first = base + r * kLnTreeBlocks;
        if (first >= n_in) break;
        used = r + 1;
        const int m = n_in - first < kLnTreeBlocks ? int(n_in - first) : kLnTreeBlocks;
        const int i = tid >> 3;                          // input of this thread within the round
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        int bad = 0;
        if (i < m && col < H2) {
            if (in) v = *reinterpret_cast<const float4 *>(in + (first + i) * H2 + col);
            else v = ln_block_value(ws, first + i, col, reinterpret_cast<const uint64_t *>(ws.state)[first + i], bad);
        }
        if (bad) set_status(ws.hdr, bad);
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) {              // inputs 1, then 2 apart
            float4 u;
            u.x = __shfl_down_sync(kFull, v.x, o);
            u.y = __shfl_down_sync(kFull, v.y, o);
            u.z = __shfl_down_sync(kFull, v.z, o);
            u.w = __shfl_down_sync(kFull, v.w, o);
            if (i + (o >> 3) < m) v = add4(v, u);
        }
        if (lane < 8) val[warp][part] = v;
        __syncthreads();
        if (warp == 0) {                                 // one column per lane: the warps' quadruples
            float x[32];
            const float *f = reinterpret_cast<const float *>(val);
            const int n = (m + 3) / 4;
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = f[k * kLnTreeCols + lane];
#pragma unroll
            for (int s = 1; s < 32; s <<= 1)
#pragma unroll
                for (int k = 0; k + s < 32; k += 2 * s)
                    if (k + s < n) x[k] = __fadd_rn(x[k], x[k + s]);
            node[r][lane] = x[0];
        }
        __syncthreads();
    }
    if (warp == 0) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = k < used ? node[k][lane] : 0.f;
        if (used > 1) x[0] = __fadd_rn(x[0], x[1]);
        if (used > 3) x[2] = __fadd_rn(x[2], x[3]);
        if (used > 2) x[0] = __fadd_rn(x[0], x[2]);
        const int64_t c = int64_t(blockIdx.y) * kLnTreeCols + lane;
        const float v = scale != 1.f ? __fmul_rn(x[0], scale) : x[0];   // scaled only at the root
        if (c < H2) {
            float *dst = c < ws.hidden ? out_w : out_b;
            if (dst) dst[blockIdx.x * out_stride + (c < ws.hidden ? c : c - ws.hidden)] = v;
        }
    }
}

}  // namespace rbi
