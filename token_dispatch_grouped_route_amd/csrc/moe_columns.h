// Sums over the partial rows that the workgroups of a backward leave: out[g][c] = the sum over s of
// part[g][s][c], in a fixed order (no atomics: the same bits on every run).
#pragma once

#include "moe_vec.h"

namespace moe {

struct ColumnSum {
    const float* part;   // [groups, slots, cols], NULL: no such sum
    void* out;           // [groups, cols]
};
constexpr int kColumnSums = 5;
struct ColumnSums {
    ColumnSum sum[kColumnSums];
    int64_t groups[kColumnSums], slots[kColumnSums];
    int32_t cols;
};

// 64 columns a workgroup: 16 lanes of four columns by 16 groups of rows (group i takes rows i, i + 16, ...),
// then the groups are added in order.
constexpr int kColumnLanes = 16, kColumnParts = 16;
template <typename WT>
__global__ __launch_bounds__(kColumnLanes * kColumnParts) void column_sums_kernel(ColumnSums a) {
    __shared__ __align__(16) float lds[kColumnParts][64 + 4];
    const int job = blockIdx.z;
    const int64_t slots = a.slots[job], cols = a.cols;
    if (!a.sum[job].part) return;
    const int lane = threadIdx.x % kColumnLanes, from = threadIdx.x / kColumnLanes, c = blockIdx.x * 64 + 4 * lane;
    for (int64_t group = blockIdx.y; group < a.groups[job]; group += gridDim.y) {
        const float* part = a.sum[job].part + group * slots * cols;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int64_t t = from; t < slots; t += kColumnParts) {
            float f[4];
            unpack_chunk<float>(load_chunk<float>(part + t * cols + c, static_cast<int>(cols) - c), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += f[i];
        }
        __syncthreads();   // the last group's sums are no longer read
        *reinterpret_cast<u32x4_t*>(&lds[from][4 * lane]) = pack_chunk<float>(s);
        __syncthreads();
        if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < static_cast<unsigned>(cols)) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < kColumnParts; ++k) t += lds[k][threadIdx.x];
            static_cast<WT*>(a.sum[job].out)[group * cols + blockIdx.x * 64 + threadIdx.x] = from_f32<WT>(t);
        }
    }
}

// One launch for all of them.
template <typename WT> void launch_column_sums(const ColumnSums& a, hipStream_t s) {
    int64_t groups = 1;
    for (int i = 0; i < kColumnSums; ++i)
        if (a.sum[i].part && a.groups[i] > groups) groups = a.groups[i];
    column_sums_kernel<WT><<<dim3((a.cols + 63) / 64, static_cast<unsigned>(groups < 1024 ? groups : 1024), kColumnSums), kColumnLanes * kColumnParts, 0, s>>>(a);
}

}  // namespace moe
