// Dropout alone (sm_103a): an elementwise pass over the active rows, four vectors
// of 8 columns a thread, whose loads are issued together and whose generator
// rounds are interleaved.  What bounds it is the issue rate next to memory: a
// vector's 16 + 16 bytes leave 174 issue slots of an SM at the memory's pace, of
// which the generator's ten rounds take about 45, selection and rounding 40.
// So rows of 1024 columns and more get CTAs of their own (a row, its offset and
// its part of the generator's counter are then the same for the whole CTA);
// shorter rows are cut into tiles of 1024 vectors that may hold many of them.
#pragma once
#include <cuda_runtime.h>

#include "host.cuh"
#include "layernorm_narrow.cuh"

namespace rbi {

struct DropoutParams {
    const void *x;
    void *y;
    DropParams drop;
    const int32_t *tok_id;
    int64_t n_rows, token_stride;
    int32_t rpt, hidden;
};

constexpr int kDropThreads = 256, kDropPer = 4, kDropTile = kDropThreads * kDropPer;

// ROWS: CTA (row, chunk of at most 1024 vectors).
template <class E, bool ROWS>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutParams p, int chunks) {
    const int tid = threadIdx.x;
    const uint32_t V = uint32_t(p.hidden) >> 3;
    Oct<E> x[kDropPer];
    int64_t off[kDropPer];
    uint32_t lrow[kDropPer], vec[kDropPer];
    bool on[kDropPer];
    if constexpr (ROWS) {
        const uint32_t row = chunks == 1 ? blockIdx.x : blockIdx.x / uint32_t(chunks), chunk = blockIdx.x - row * uint32_t(chunks);
        const uint32_t t = p.rpt == 1 ? row : row / uint32_t(p.rpt), head = row - t * uint32_t(p.rpt);
        const int32_t id = p.tok_id[t];
        if (id < 0) return;
        const int64_t at = int64_t(t) * p.token_stride + int64_t(head) * p.hidden;
#pragma unroll
        for (int k = 0; k < kDropPer; ++k) {
            vec[k] = chunk * (blockDim.x * kDropPer) + tid + k * blockDim.x;
            on[k] = vec[k] < V;
            off[k] = at + int64_t(vec[k] * 8u);
            lrow[k] = uint32_t(id) * uint32_t(p.rpt) + head;
        }
    } else {
        const int64_t first = int64_t(blockIdx.x) * kDropTile, n = p.n_rows * V;
        // the tile's first vector is number v0 of row row0
        const int64_t row0 = first / V;
        const uint32_t v0 = uint32_t(first - row0 * V);
#pragma unroll
        for (int k = 0; k < kDropPer; ++k) {
            const uint32_t i = uint32_t(tid + k * kDropThreads), r = (v0 + i) / V;
            vec[k] = v0 + i - r * V;
            const int64_t row = row0 + r;
            on[k] = first + i < n;
            off[k] = 0;
            lrow[k] = 0;
            if (on[k]) {
                const uint32_t t = p.rpt == 1 ? uint32_t(row) : uint32_t(row) / uint32_t(p.rpt), head = uint32_t(row) - t * uint32_t(p.rpt);
                const int32_t id = p.tok_id[t];
                on[k] = id >= 0;
                lrow[k] = uint32_t(id) * uint32_t(p.rpt) + head;
                off[k] = int64_t(t) * p.token_stride + int64_t(head) * p.hidden + int64_t(vec[k]) * 8;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kDropPer; ++k)
        if (on[k]) x[k] = oct_load<E>(p.x, off[k]);
    const DropKey key = drop_key(p.drop);
    const DropRule rule = drop_rule(p.drop);
#pragma unroll
    for (int k = 0; k < kDropPer; ++k) {
        const uint4 u = philox4x32(vec[k], lrow[k], key);
        const uint32_t words[4] = {u.x, u.y, u.z, u.w};
        if (on[k]) {
            f2_t f[4];
            oct_up<E>(x[k], f);
            drop_pairs(f, words, rule);
            oct_store<E>(p.y, off[k], f);
        }
    }
}

template <class E>
int dropout_launch(const DropoutParams &p, cudaStream_t stream) {
    const int64_t V = p.hidden / 8;
    const bool rows = V >= 128;
    const int64_t chunks = rows ? (V + kDropTile - 1) / kDropTile : 1, per = (V + chunks - 1) / chunks;
    const int64_t grid = rows ? p.n_rows * chunks : (p.n_rows * V + kDropTile - 1) / kDropTile;
    if (grid >= (int64_t(1) << 31)) return RMSNORM_ERR_LAYOUT;
    const unsigned threads = unsigned((per + 32 * kDropPer - 1) / (32 * kDropPer) * 32);
    if (rows) dropout_kernel<E, true><<<unsigned(grid), threads, 0, stream>>>(p, int(chunks));
    else dropout_kernel<E, false><<<unsigned(grid), kDropThreads, 0, stream>>>(p, 1);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

}  // namespace rbi
