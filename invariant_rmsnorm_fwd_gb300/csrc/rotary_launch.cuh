// Launcher of the rotary kernels, instantiated per element type and kind of pairs.
#pragma once
#include "rotary_kernels.cuh"

namespace rbi {

// element: bytes; pairs: register pairs of a piece.
inline void set_teams(RotaryParams &p, int element, int pairs) {
    p.by_team = Divisor(uint32_t(p.team));
    p.teams = 32 / p.team;
    p.by_teams = Divisor(uint32_t(p.teams));
    p.pitch = pieces_pitch(p.vectors, 2 * element, p.team, p.teams, pairs * element / 2);
    p.turning = (p.rot / (4 * pairs) + p.team - 1) / p.team;
}

// Heads of a warp of the forward pass: those, up to `most`, with which the warps' rounds take
// least if a warp's start and a token's angles take as long as `start` rows.  A call of a
// few tokens gets many warps of few heads (one token of 40 heads of 128: rotation 4.0 -> 2.6 us,
// norm and rotation 5.7 -> 3.1), but not just more than run at once (3,902 of 2+1 of 192: 7.3 -> 5.6).
// Halves and neighbours alone, which memory bounds, have at most 8 heads (32+8 of 128, 33,384 tokens:
// 100.3 us, 102.5 with 20); others up to 24 (16+16 of 72, 17,620 tokens, with the norm: 43 -> 37, 8+8 of 40
// 19 -> 15, 32+8 of 144 78 -> 72, of 128 104 -> 105).  5 rows for 16 bits, 3 for FP32 (80 columns, 20 turning: 90 us for 96).
inline int forward_heads(int64_t windows, int32_t heads, int most, int start, int64_t at_once) {
    int64_t best = INT64_MAX;
    int per = most;
    for (const int n : {24, 16, 12, 8, 6, 4, 3, 2, 1}) {
        if (n > most) continue;
        const int64_t chunks = (heads + n - 1) / n, rows = (heads + chunks - 1) / chunks;
        const int64_t time = (windows * chunks + at_once - 1) / at_once * (rows + start);
        if (time < best) {
            best = time;
            per = n;
        }
    }
    return per;
}

template <class E, int PAIRS, bool NORM, int TEAM>
static int rotary_launch_fwd(RotaryParams &p, cudaStream_t stream) {
    auto kern = rotary_kernel<E, PAIRS, NORM, TEAM>;
    static KernelInfo info;
    DeviceInfo *d = nullptr;
    int regs = 0;
    if (int rc = device_info(&d)) return rc;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
    set_teams(p, int(sizeof(E)), piece_pairs(PAIRS));
    const int64_t windows = (p.active + p.teams - 1) / p.teams;
    const int most = forward_heads(windows, p.heads, NORM || in_pieces(PAIRS) ? 24 : kChunkHeads, sizeof(E) == 4 ? 3 : 5,
                                   int64_t(kFwdCtas<E, PAIRS, NORM>) * kQkWarps * d->sms);
    p.chunks = (p.heads + most - 1) / most;
    p.per = (p.heads + p.chunks - 1) / p.chunks;
    p.by_chunks = Divisor(uint32_t(p.chunks));
    // Steps of a warp: until its teams have 16 rows each (8 without the norm, whose rows are
    // quicker), so that its start is paid for, while every SM has 64 warps to choose from
    // (one step, two, four: rotation of 17,620 tokens of 40 heads of 128 55, 57, 60 us, norm and
    // rotation of 33,384 106, 105, 110; 1+1 heads, 270,100 tokens 79, 72, 70).
    int steps = 1;
    while (steps * p.per < (NORM ? 16 : 8) && 2 * steps * p.teams <= 32 &&
           p.n_tokens * p.chunks >= int64_t(2) * steps * p.teams * 64 * d->sms)
        steps *= 2;
    const int slots = steps * p.teams;
    p.units = uint32_t((p.n_tokens + slots - 1) / slots * p.chunks);
    kern<<<(p.units + kQkWarps - 1) / kQkWarps, kQkWarps * 32,
           (NORM ? kWeightBytes : 0) + kQkWarps * Ring<E, 1, PAIRS>::kBytes, stream>>>(p, slots);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS, int TEAM>
static int rotary_launch_bwd(RotaryParams &p, cudaStream_t stream) {
    auto kern = qk_bwd_kernel<E, PAIRS, TEAM>;
    static KernelInfo info;
    DeviceInfo *d = nullptr;
    int regs = 0;
    if (int rc = device_info(&d)) return rc;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
    set_teams(p, int(sizeof(E)), piece_pairs(PAIRS));
    const QkGroups t(p.D, p.heads, p.ws.hdr ? p.ws.n : p.n_tokens);
    p.group = t.group;
    p.share = t.share;
    p.by_group = Divisor(uint32_t(t.group));
    const int64_t windows = (p.n_tokens + t.group - 1) / t.group;
    const QkChunks cut = p.ws.hdr ? p.ws.cut : QkChunks(p.hq, p.heads - p.hq, windows, t.share);
    p.chunks = cut.chunks;
    p.per = cut.per;
    p.by_chunks = Divisor(uint32_t(p.chunks));
    p.units = uint32_t(windows * p.chunks);
    const bool straddles = p.hq % p.per != 0 && p.heads > p.hq;
    kern<<<(p.units + kQkWarps - 1) / kQkWarps, kQkWarps * 32,
           qk_bwd_smem(Ring<E, 2, PAIRS>::kBytes, p.ws.hdr != nullptr, straddles), stream>>>(p, straddles);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS>
static int rotary_launch(RotaryParams &p, int mode, cudaStream_t stream) {
    if (mode == 0) {
        // (heads of 80 with 24 columns turning, 33,384 tokens: 76 us, in teams of a power of two 92; else equal)
        p.team = p.in_place && PAIRS != kNear ? PAIRS == kHalf ? p.rot / 16 : (p.vectors + 1) / 2 : p.lanes;
        return rotary_launch_fwd<E, PAIRS, false, 0>(p, stream);
    }
    // Teams of just the lanes that a head needs where a warp then holds more of them (5 lanes for 80 columns, 6
    // for 96, 10 for 160).  Forward, bf16, 32+8 heads of 80, 33,384 tokens: 95 -> 75 us; of 160, 17,620 tokens,
    // 101 -> 75; of 96 54 -> 48; of 48 31.6 -> 32.2; FP32 heads of 72 33 -> 27.  Backward, heads of 80: 166 -> 138;
    // of 160 170 -> 147; of 96, 17,620 tokens, 97 -> 87; of 48 62 -> 60.
    p.team = QkTeams(p.D).size;
    const bool fwd = mode == 1;
    switch (p.team) {
        case 4: return fwd ? rotary_launch_fwd<E, PAIRS, true, 4>(p, stream) : rotary_launch_bwd<E, PAIRS, 4>(p, stream);
        case 5: return fwd ? rotary_launch_fwd<E, PAIRS, true, 5>(p, stream) : rotary_launch_bwd<E, PAIRS, 5>(p, stream);
        case 6: return fwd ? rotary_launch_fwd<E, PAIRS, true, 6>(p, stream) : rotary_launch_bwd<E, PAIRS, 6>(p, stream);
        case 8: return fwd ? rotary_launch_fwd<E, PAIRS, true, 8>(p, stream) : rotary_launch_bwd<E, PAIRS, 8>(p, stream);
        case 16: return fwd ? rotary_launch_fwd<E, PAIRS, true, 16>(p, stream) : rotary_launch_bwd<E, PAIRS, 16>(p, stream);
        default: return fwd ? rotary_launch_fwd<E, PAIRS, true, 0>(p, stream) : rotary_launch_bwd<E, PAIRS, 0>(p, stream);
    }
}

// One translation unit per element type and kind of pairs (rotary_*.cu).
template <class E, int PAIRS>
int rotary_run_pairs(RotaryParams p, int mode, cudaStream_t stream) {
    p.lanes = (p.D + 15) / 16;
    p.vector0 = p.in_place ? p.first / 8 : 0;
    p.all_pieces = mode > 0;
    p.vectors = p.in_place ? (p.first + p.rot + 7) / 8 - p.vector0 : p.D / 8;
    return rotary_launch<E, PAIRS>(p, mode, stream);
}

}  // namespace rbi
