// tri_experts.h -- how a workgroup finds its rows in a ragged launch over experts.
#pragma once
#include "tri_device.h"
#include "tri_internal.h"

namespace tri {

// Inclusive prefix sums over the 64 lanes: inside rows of 16 lanes by row shifts, then row 0's and 2's last lane into
// the next row, and lane 31 into the upper half.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
    return v;
}

// The places r0 .. r0 + rows - 1 of one expert; e < 0: none.
struct ExpertTile {
    int e, r0, rows;
};

// One tile of the list that cuts every expert's places into tiles of `height` (the last of an expert may be shorter;
// experts without places have none), in the experts' order: tile slot(n), n the length of the list.  Called by whole waves
// with wave-uniform arguments: lane l counts the tiles of expert l (of four experts where there are more than 64), a scan
// over the lanes gives n and finds the lane that owns the tile.  Offsets are clamped to 0 .. R, so no tile reaches outside
// whatever they hold.
template <int PER, typename Slot>
__device__ __forceinline__ ExpertTile expert_tile_of(const int32_t *__restrict__ offsets, int E, int R, int height,
                                                     Slot slot_of)
{
    const int lane = threadIdx.x & 63;
    int at[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) {
        const int e = PER * lane + i;
        at[i] = e <= E ? min(max(offsets[e], 0), R) : 0;
    }
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int rows = PER * lane + i < E ? max(at[i + 1] - at[i], 0) : 0;
        n[i] = (int)(((unsigned)rows + height - 1) / height);   // (unsigned: rows up to 2^31 - 1)
        sum += n[i];
    }
    const int run = wave_scan(sum);
    const int slot = slot_of(__builtin_amdgcn_readlane(run, 63));
    const unsigned long long past = __ballot(run > slot);
    if (past == 0) return ExpertTile{-1, 0, 0};
    const int src = __ffsll(past) - 1;           // (wave-uniform)
    int left = slot - (run - sum), e = PER * lane, r0 = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (left >= 0 && left < n[i]) {
            e = PER * lane + i;
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

template <typename Slot>
__device__ __forceinline__ ExpertTile expert_tile(const int32_t *__restrict__ offsets, int E, int R, int height, Slot slot_of)
{
    static_assert(TRI_MAX_EXPERTS <= 256, "at most four experts per lane");
    return E <= 64 ? expert_tile_of<1>(offsets, E, R, height, slot_of) : expert_tile_of<4>(offsets, E, R, height, slot_of);
}

// Tiles of that height that R places in E experts make at most: an expert with places wastes less than one tile.
inline int64_t expert_slots(int64_t R, int E, int height)
{
    return (R + (int64_t)(height - 1) * (R < E ? R : E)) / height;
}

}  // namespace tri
