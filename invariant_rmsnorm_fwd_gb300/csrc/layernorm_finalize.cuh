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

constexpr int kLnTreeCols = 64;                          // columns of [dweight | dbias] per CTA: 8 lanes, twice 4 each
constexpr int kLnTreeBlocks = 32;                        // blocks per CTA in the first pass
constexpr int kLnTreeNodes = 256;                        // inputs per CTA in the others: 8 per 8 lanes

struct Cols {                        // a lane's columns: c .. c + 3 and c + 32 .. c + 35
    float4 a, b;
};
__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ float4 fma4(const float4 &a, const float4 &b, const float4 &c) {
    return make_float4(__fmaf_rn(a.x, b.x, c.x), __fmaf_rn(a.y, b.y, c.y), __fmaf_rn(a.z, b.z, c.z), __fmaf_rn(a.w, b.w, c.w));
}
__device__ __forceinline__ Cols add_cols(const Cols &x, const Cols &y) { return {add4(x.a, y.a), add4(x.b, y.b)}; }
__device__ __forceinline__ float4 down4(const float4 &v, int o) {
    return make_float4(__shfl_down_sync(kFull, v.x, o), __shfl_down_sync(kFull, v.y, o), __shfl_down_sync(kFull, v.z, o),
                       __shfl_down_sync(kFull, v.w, o));
}
// two: the second four columns are inside [dweight | dbias]
__device__ __forceinline__ Cols load_cols(const float *p, bool two) {
    Cols v;
    v.a = *reinterpret_cast<const float4 *>(p);
    v.b = two ? *reinterpret_cast<const float4 *>(p + 32) : make_float4(0.f, 0.f, 0.f, 0.f);
    return v;
}

// A group's sums for four columns from its spilled rows.  A function of its own:
// inlined for each of a block's groups it would be most of the kernel's code, and
// fetching that code what the tree waits for.
__device__ __noinline__ float4 spilled4(const LnWs &ws, int64_t row0, int rows, int64_t col) {
    const int64_t H2 = 2 * ws.hidden;
    const bool is_w = col < ws.hidden;
    const int64_t c = is_w ? col : col - ws.hidden;
    float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < rows; ++r) {
        const int64_t row = row0 + r;
        if (!ws.flag[row]) {
            set_status(ws.hdr, kStMissing);
            continue;
        }
        const float4 dy = *reinterpret_cast<const float4 *>(ws.spill + row * H2 + ws.hidden + c);
        if (is_w) g = fma4(dy, *reinterpret_cast<const float4 *>(ws.spill + row * H2 + c), g);
        else g = add4(g, dy);
    }
    return g;
}

// Eight columns of block b: the groups from the first to the last, each from a
// stored partial or folded from its spilled rows.  All stored partials are
// requested before any is used.  check: report rows that are missing or arrived
// twice (one CTA per block does).
__device__ __forceinline__ Cols ln_block_value(const LnWs &ws, int64_t b, int64_t col, bool two, uint64_t state, bool check,
                                               int &bad) {
    const int64_t H2 = 2 * ws.hidden;
    const float *part = ws.partial + b * kGroups * H2 + col;
    const int64_t left = ws.n_rows - b * kBlockRows;
    const int rows = left < kBlockRows ? int(left) : kBlockRows, groups = (rows + kGroupRows - 1) / kGroupRows;
    Cols v[kGroups];
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
        if ((state >> (8 * j)) & 0xff) v[j] = load_cols(part + j * H2, two);
    const uint64_t *flags = reinterpret_cast<const uint64_t *>(ws.flag) + b * kGroups;
    Cols acc = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    int next = 0;                                        // first group not yet taken
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const int c = int((state >> (8 * j)) & 0xff);
        if (check && c && flags[j]) bad |= kStDouble;    // a group that arrived as a partial has no spilled rows
        if (j < next) {                                  // inside the fold of the block's first groups
            if (check && (c || flags[j])) bad |= kStDouble;
            continue;
        }
        if (j >= groups) continue;
        if (c) {
            next = j + c;
        } else {
            next = j + 1;
            const int n = rows - j * kGroupRows < kGroupRows ? rows - j * kGroupRows : kGroupRows;
            v[j].a = spilled4(ws, b * kBlockRows + j * kGroupRows, n, col);
            v[j].b = two ? spilled4(ws, b * kBlockRows + j * kGroupRows, n, col + 32) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        acc = j == 0 ? v[j] : add_cols(acc, v[j]);
    }
    return acc;
}

// One pass of the pairwise tree with odd carry over n_in inputs (block values in
// the first pass, then the results of the one before): CTA (g, c) reduces inputs
// [m g, m (g + 1)) of 64 columns to one node, m = 32 in the first pass, 256 in the
// others.  Eight lanes hold the columns of a block (of 8 consecutive inputs), the
// four of a warp meet by shuffles, the eight warps through shared memory.  All
// loads of a pass are in flight at once.
//
// What bounds it: latency.  Hidden 4096, 276 blocks, 1,055 partials of 304 shares, 35 MB
// (most of them still in the L2): 13 us, hidden 8192 25 us, in 4 and 8 rounds of CTAs of
// about 3 us each, a few dependent loads long; a later pass 2 us.  32 inputs in the
// later passes too: three launches instead of two at hidden 4096; 32 columns a CTA,
// 4 groups in flight at twice the CTAs, CTAs that walk over the columns: equal or
// slower.
template <bool FIRST>
__global__ void __launch_bounds__(256) ln_tree_kernel(const __grid_constant__ LnWs ws, const float *in, float *out_w, float *out_b,
                                                      int64_t out_stride, int64_t n_in, float scale) {
    __shared__ float4 val[8][16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = tid & 7, i = tid >> 3;
    const int64_t H2 = 2 * ws.hidden, col = int64_t(blockIdx.y) * kLnTreeCols + part * 4;
    const int64_t first = int64_t(blockIdx.x) * (FIRST ? kLnTreeBlocks : kLnTreeNodes);
    // m teams of eight lanes have something; in the first pass one block each
    const int64_t left = FIRST ? n_in - first : (n_in - first + 7) / 8;
    const int m = left < 32 ? int(left) : 32;
    uint64_t state = 0;
    if constexpr (FIRST) {
        if (i < m) state = reinterpret_cast<const uint64_t *>(ws.state)[first + i];
        if (!ln_header_ok(ws)) {
            if (tid == 0) set_status(ws.hdr, kStHeader);
            return;
        }
    }
    Cols v = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    int bad = 0;
    if (i < m && col < H2) {
        const bool two = col + 32 < H2;
        if constexpr (!FIRST) {
            const int64_t n = n_in - first - i * 8;
            Cols x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) x[k] = load_cols(in + (first + i * 8 + k) * H2 + col, two);
#pragma unroll
            for (int s = 1; s < 8; s <<= 1)
#pragma unroll
                for (int k = 0; k + s < 8; k += 2 * s)
                    if (k + s < n) x[k] = add_cols(x[k], x[k + s]);
            v = x[0];
        } else {
            v = ln_block_value(ws, first + i, col, two, state,
                               blockIdx.y == 0, bad);
        }
    }
    if (bad) set_status(ws.hdr, bad);
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {                  // inputs 1, then 2 apart
        const Cols u = {down4(v.a, o), down4(v.b, o)};
        if (i + (o >> 3) < m) v = add_cols(v, u);
    }
    if (lane < 8) {
        val[warp][part] = v.a;
        val[warp][8 + part] = v.b;
    }
    __syncthreads();
    if (warp < 2) {                                      // one column per lane: the warps' quadruples
        float x[8];
        const float *f = reinterpret_cast<const float *>(val);
        const int n = (m + 3) / 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = f[k * kLnTreeCols + warp * 32 + lane];
#pragma unroll
        for (int s = 1; s < 8; s <<= 1)
#pragma unroll
            for (int k = 0; k + s < 8; k += 2 * s)
                if (k + s < n) x[k] = __fadd_rn(x[k], x[k + s]);
        const int64_t c = int64_t(blockIdx.y) * kLnTreeCols + warp * 32 + lane;
        const float r = scale != 1.f ? __fmul_rn(x[0], scale) : x[0];   // scaled only at the root
        if (c < H2) {
            float *dst = c < ws.hidden ? out_w : out_b;
            if (dst) dst[blockIdx.x * out_stride + (c < ws.hidden ? c : c - ws.hidden)] = r;
        }
    }
}

}  // namespace rbi
