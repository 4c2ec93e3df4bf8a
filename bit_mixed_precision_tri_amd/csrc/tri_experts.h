// tri_experts.h -- how a workgroup finds its rows in a ragged launch over experts.
#pragma once
#include "tri_device.h"
#include "tri_internal.h"

namespace tri {

// The places r0 .. r0 + rows - 1 of one expert; e < 0: none.
struct ExpertTile {
    int e, r0, rows;
};

// Tile `slot` of the list that cuts every expert's places into tiles of `height` (the last of an expert may be shorter;
// experts without places have none), in the experts' order.  Called by whole waves with wave-uniform arguments: lane l
// counts the tiles of experts 4 l .. 4 l + 3 (at most 256), a scan over the lanes finds the lane that owns the slot.
// Offsets are clamped to 0 .. R, so no tile reaches outside whatever they hold.
__device__ __forceinline__ ExpertTile expert_tile(const int32_t *__restrict__ offsets, int E, int R, int slot, int height)
{
    static_assert(TRI_MAX_EXPERTS <= 256, "four experts per lane");
    const int lane = threadIdx.x & 63;
    int at[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        const int e = 4 * lane + i;
        at[i] = e <= E ? min(max(offsets[e], 0), R) : 0;
    }
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rows = 4 * lane + i < E ? max(at[i + 1] - at[i], 0) : 0;
        n[i] = (rows + height - 1) / height;
        sum += n[i];
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d, 64);
        if (lane >= d) run += o;
    }
    const unsigned long long past = __ballot(run > slot);
    if (past == 0) return ExpertTile{-1, 0, 0};
    const int src = __ffsll(past) - 1;           // (wave-uniform)
    int left = slot - (run - sum), e = 4 * lane, r0 = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (left >= 0 && left < n[i]) {
            e = 4 * lane + i;
            r0 = at[i] + left * height;
            hi = at[i + 1];
        }
        left -= n[i];
    }
    e = __builtin_amdgcn_readlane(e, src);
    r0 = __builtin_amdgcn_readlane(r0, src);
    hi = __builtin_amdgcn_readlane(hi, src);
    return ExpertTile{e, r0, min(height, hi - r0)};
}

// Tiles of that height that R places in E experts make at most.
inline int64_t expert_slots(int64_t R, int E, int height) { return R / height + (R < E ? R : E); }

}  // namespace tri
