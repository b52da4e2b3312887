// What the products that stage an operand in LDS share (moe_linear.hip, moe_linear_few.hip).
#pragma once

#include "moe_linear.h"

namespace moe {

struct Plan {
    bool dma;
    int tile, splits;
    double us;   // estimated
};

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) void g_void;
typedef __attribute__((address_space(3))) void l_void;
typedef __attribute__((address_space(3))) s16x4 l_s16x4;

// One operand of a workgroup's tile: W virtual rows (A) or columns (B) from `first`, `count` of which exist.
// For swiglu the virtual columns alternate G gate columns and the G up columns of the same outputs, so that a
// wave holds both halves of its outputs.
struct Side {
    const uint16_t* p;
    int64_t ld;
    int first, count;   // real index of the first, and of one past the last
    int g, up;          // G, and the offset of an up column; g = 0: not paired
    __device__ __forceinline__ int real(int v) const {   // may be >= the bound, which limit() gives
        return g ? first + v / (2 * g) * g + v % g + (v / g & 1) * up : first + v;
    }
    __device__ __forceinline__ int limit(int v) const { return g ? count + (v / g & 1) * up : count; }
};

// A chunk of zeros, read in place of chunks past the end of the reduction.
__device__ __align__(16) const uint32_t kZeroChunk[4] = {0, 0, 0, 0};

// s_waitcnt with these counts (vmcnt up to 63; lgkmcnt 0 or any).
template <int VM, bool LGKM> __device__ __forceinline__ void wait_counts() {
    __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | (LGKM ? 0 : 15 << 8) | ((VM >> 4) << 14));
}

// Whether an operand's 16-byte chunks are aligned and whole (extent: what it has along its contiguous dimension).
bool whole_chunks(const void* p, int64_t ld, int64_t extent) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && extent % 8 == 0; }

}  // namespace
}  // namespace moe
