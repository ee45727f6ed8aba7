// Dropout alone (sm_103a): an elementwise pass over the active rows, four vectors
// of 8 columns a thread, whose loads are issued together and whose generator
// rounds are interleaved.  What bounds it is the issue rate next to memory: a
// vector's 16 + 16 bytes leave 174 issue slots of an SM at the memory's pace, of
// which the generator's ten rounds take about 45, selection and rounding 40.
// So rows of 1024 columns and more get CTAs of their own (a row, its offset and
// its part of the generator's counter are then the same for the whole CTA);
// shorter rows are taken in tiles of as many whole rows as 1024 vectors hold.
// 33,384 rows of 5120 bf16: 110 us, 6.2 TB/s of 6.8 (154 us in tiles); 64 M bf16
// elements in rows of 1024: 48 us, of 1000: 58, of 128: 56 (64 with tiles cut
// anywhere and hardware divisions), FP32 44 (floor 40).
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

// ROWS: CTA (row, one of its `chunks` chunks of at most 1024 vectors); else a CTA
// takes `chunks` whole rows.
template <class E, bool ROWS>
__global__ void __launch_bounds__(kDropThreads, sizeof(E) == 2 ? 5 : 3) dropout_kernel(const __grid_constant__ DropoutParams p, int chunks, Divisor by_v,
                                                               Divisor by_rpt) {
    const int tid = threadIdx.x;
    const uint32_t V = uint32_t(p.hidden) >> 3;
    Oct<E> x[kDropPer];
    int64_t off[kDropPer];
    uint32_t lrow[kDropPer], vec[kDropPer];
    bool on[kDropPer];
    if constexpr (ROWS) {
        const uint32_t row = chunks == 1 ? blockIdx.x : blockIdx.x / uint32_t(chunks), chunk = blockIdx.x - row * uint32_t(chunks);
        const uint32_t t = by_rpt.quotient(row), head = row - t * uint32_t(p.rpt);
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
        const uint32_t row0 = blockIdx.x * uint32_t(chunks), rows = uint32_t(p.n_rows) - row0;   // chunks: rows of a CTA
#pragma unroll
        for (int k = 0; k < kDropPer; ++k) {
            const uint32_t i = uint32_t(tid + k * kDropThreads), r = by_v.quotient(i), row = row0 + r;
            vec[k] = i - r * V;
            on[k] = r < uint32_t(chunks) && r < rows;
            off[k] = 0;
            lrow[k] = 0;
            if (on[k]) {
                const uint32_t t = by_rpt.quotient(row), head = row - t * uint32_t(p.rpt);
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
    const int64_t tile = rows ? 1 : kDropTile / V;       // rows of a CTA
    const int64_t grid = rows ? p.n_rows * chunks : (p.n_rows + tile - 1) / tile;
    if (grid >= (int64_t(1) << 31)) return RMSNORM_ERR_LAYOUT;
    const unsigned threads = unsigned((per + 32 * kDropPer - 1) / (32 * kDropPer) * 32);
    const Divisor by_v{uint32_t(V)}, by_rpt{uint32_t(p.rpt)};
    if (rows) dropout_kernel<E, true><<<unsigned(grid), threads, 0, stream>>>(p, int(chunks), by_v, by_rpt);
    else dropout_kernel<E, false><<<unsigned(grid), kDropThreads, 0, stream>>>(p, int(tile), by_v, by_rpt);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

}  // namespace rbi
