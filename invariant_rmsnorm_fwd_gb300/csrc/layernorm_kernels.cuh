// What the kernels of the batch-invariant layer norm (sm_103a) share: the
// workspace and the parameters of a call.
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

// (all three fields are loaded at once: small calls wait for each round trip)
__device__ __forceinline__ bool ln_header_ok(const LnWs &ws) {
    const WsHeader *h = ws.hdr;
    const auto magic = h->magic;
    const int64_t n_rows = h->n_rows, hidden = h->hidden;
    return (magic == kLnMagic) & (n_rows == ws.n_rows) & (hidden == ws.hidden);
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
    int32_t share, share_rest;       // streaming kernel: units of a CTA; the first share_rest CTAs have one more
    LnWs ws;
};

}  // namespace rbi
