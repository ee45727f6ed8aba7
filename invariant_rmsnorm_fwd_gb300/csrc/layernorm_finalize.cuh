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

// One column's value of block b: the groups from the first to the last, each a
// stored partial or the fold of its spilled rows.
__device__ __forceinline__ float ln_block_value(const LnWs &ws, int64_t b, int64_t col, bool &missing, bool &twice) {
    const int64_t H2 = 2 * ws.hidden;
    const bool is_w = col < ws.hidden;
    const int64_t c = is_w ? col : col - ws.hidden;
    const float *part = ws.partial + b * kGroups * H2 + col;
    float acc = 0.f;
    // a group that arrived as a partial has no spilled rows
    const uint64_t *flags = reinterpret_cast<const uint64_t *>(ws.flag) + b * kGroups;
    if (ws.state[b * kGroups] == kGroupWhole) return part[0];
    const int64_t rows = ws.n_rows - b * kBlockRows < kBlockRows ? ws.n_rows - b * kBlockRows : kBlockRows;
    for (int j = 0; j * kGroupRows < rows; ++j) {
        float v = 0.f;
        const uint8_t st = ws.state[b * kGroups + j];
        if (st == kGroupPartial) {
            v = part[j * H2];
            if (flags[j] != 0) twice = true;
        } else {
            if (st != kGroupNone) missing = true;
            for (int r = j * kGroupRows; r < (j + 1) * kGroupRows && r < rows; ++r) {
                const int64_t g = b * kBlockRows + r;
                if (!ws.flag[g]) missing = true;
                const float xh = ws.spill[g * H2 + c], dy = ws.spill[g * H2 + ws.hidden + c];
                v = is_w ? __fmaf_rn(dy, xh, v) : __fadd_rn(v, dy);
            }
        }
        acc = j == 0 ? v : __fadd_rn(acc, v);
    }
    return acc;
}

// One pass of the pairwise tree with odd carry over groups of 32 inputs (block
// values in the first pass): CTA (g, c) reduces inputs [32g, 32g + 32) of 32
// columns, warp w forming input w.
__global__ void __launch_bounds__(1024) ln_tree_kernel(LnWs ws, const float *in, float *out_w, float *out_b,
                                                       int64_t out_stride, int64_t n_in, float scale) {
    __shared__ float val[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t col = int64_t(blockIdx.y) * 32 + lane, H2 = 2 * ws.hidden, i = int64_t(blockIdx.x) * 32 + w;
    const int m = n_in - int64_t(blockIdx.x) * 32 < 32 ? int(n_in - int64_t(blockIdx.x) * 32) : 32;
    if (!in && !ln_header_ok(ws)) {
        if (threadIdx.x == 0) set_status(ws.hdr, kStHeader);
        return;
    }
    bool missing = false, twice = false;
    if (w < m && col < H2) val[w][lane] = in ? in[i * H2 + col] : ln_block_value(ws, i, col, missing, twice);
    if (missing) set_status(ws.hdr, kStMissing);
    if (twice) set_status(ws.hdr, kStDouble);
    for (int n = m; n > 1; n = (n + 1) / 2) {
        __syncthreads();
        float a = 0.f;
        const bool act = w < (n + 1) / 2;
        if (act) a = 2 * w + 1 < n ? __fadd_rn(val[2 * w][lane], val[2 * w + 1][lane]) : val[2 * w][lane];
        __syncthreads();
        if (act) val[w][lane] = a;
    }
    if (w == 0 && col < H2) {
        const float r = scale != 1.f ? __fmul_rn(val[0][lane], scale) : val[0][lane];
        float *dst = col < ws.hidden ? out_w : out_b;
        if (dst) dst[blockIdx.x * out_stride + (col < ws.hidden ? col : col - ws.hidden)] = r;
    }
}

}  // namespace rbi
