// What the kernels that stream an expert's weights for a few rows share (4-bit products, the bf16 expert layer for
// few tokens): loads through buffers, and an expert's list of pairs.
#pragma once

#include "moe_vec.h"

namespace moe {

// Weights and x are read through buffers, whose loads return 0 past the end: an offset of kNoRow or
// kNoK or more (also of both added) lies past every buffer, none of which exceeds 2^30 bytes.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kNoRow = 0x80000000u, kNoK = 0x40000000u;
__device__ __forceinline__ rsrc_t buffer_of(const void* p, int64_t bytes) {   // the same for the whole wave
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(bytes)), 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(rsrc_t r, uint32_t at) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

// The pairs of expert id, ascending, and their number; 0 if `first` >= 0 and an earlier pair has it.  Every
// wave writes the whole list (the same values), so none waits for another.
__device__ __forceinline__ int expert_pairs(const int32_t* topk_idx, int pairs, int id, int first, int* list) {
    const int lane = threadIdx.x & 63;
    int count = 0, earliest = pairs;
    constexpr int AHEAD = 8;   // loads in flight
    for (int p0 = 0; p0 < pairs; p0 += 64 * AHEAD) {
        int ids[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ids[i] = topk_idx[min(p0 + 64 * i + lane, pairs - 1)];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int p = p0 + 64 * i + lane;
            const bool mine = p < pairs && ids[i] == id;
            const uint64_t m = __ballot(mine);
            if (mine) list[count + __popcll(m & ((uint64_t(1) << lane) - 1))] = p;
            if (m != 0 && count == 0) earliest = p0 + 64 * i + __ffsll(static_cast<unsigned long long>(m)) - 1;
            count += __popcll(m);
        }
    }
    wave_sync();   // the list is read by other lanes than those that wrote it
    return earliest < first ? 0 : count;
}

}  // namespace moe
