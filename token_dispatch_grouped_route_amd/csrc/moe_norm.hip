// Row norm, forward (layer norm and RMS norm): moe_norm.h has the formulas and the plan.  The variance is
// a sum of centred squares, at no extra read since the row is in registers.
// Layer norm of 8192 x 7168 bf16: 41 us (5.8 TB/s); rms norm of 65536 x 7168: 370 us (5.1 TB/s), one row: 4 us.
#include "moe_norm.h"

namespace moe {

template <typename T, typename WT, int TPR, int NV>
__global__ __launch_bounds__(norm_block(TPR)) void norm_fwd_kernel(NormArgs a, bool layer) {
    constexpr int N = Chunk<T>::N, BLOCK = norm_block(TPR), W = norm_waves(TPR);
    __shared__ float lds[4 * W];   // two sums per row (mean, variance), each in two buffers
    const int tid = threadIdx.x % TPR, cols = a.cols;
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (BLOCK / TPR);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR);   // of the workgroup's first team
    int64_t row = row0 + threadIdx.x / TPR;
    // teams past the last row run along with it (the exchanges need every lane) and store nothing
    auto at = [&](int64_t r) { return (r < a.rows ? r : a.rows - 1) * a.ldx; };

    u32x4_t next[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tid) * N;
        next[j] = load_chunk<T>(x + at(row) + c, cols - c);
    }
    NormWeights<WT, N, NV, TPR> w, b;
    w.load(a.weight, tid, cols, 1.0f);
    b.load(a.bias, tid, cols, 0.0f);
    int slot = 0;
    for (int64_t base = row0; base < a.rows; base += step, row += step) {
        float v[NV][N];
#pragma unroll
        for (int j = 0; j < NV; ++j) unpack_chunk<T>(next[j], v[j]);
        if (base + step < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                next[j] = load_chunk<T>(x + at(row + step) + c, cols - c);
            }
        }
        float mean = 0.0f;
        if (layer) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) s[0] += v[j][i];
            team_sum<TPR, 1>(s, lds, slot);
            mean = s[0] / static_cast<float>(cols);   // divided: the mean of equal elements is theirs
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int valid = cols - (j * TPR + tid) * N;
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] -= mean;
            if (valid < N) {   // the chunk of the row's end, and those past it
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] = i < valid ? v[j][i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) q[0] += v[j][i] * v[j][i];
        }
        team_sum<TPR, 1>(q, lds + 2 * W, slot);
        slot ^= 1;
        // squares whose sum is not finite (an infinity, or elements too large for fp32's range) would give rstd 0 and a
        // row of zeros that nothing shows: NaN instead, here and so in the backward
        const float rstd = q[0] < __builtin_inff() ? 1.0f / sqrtf(q[0] / static_cast<float>(cols) + a.eps) : __builtin_nanf("");
        if (row < a.rows) {
            if (tid == 0) {
                if (layer && a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                float fw[N], fb[N], o[N];
                w.get(j, fw);
                b.get(j, fb);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = v[j][i] * rstd * fw[i] + fb[i];
                store_chunk<T>(y + row * a.ldy + c, pack_chunk<T>(o), cols - c);
            }
        }
    }
}

// Chunks per thread.  With 2, teams of twice the threads: 4000 x 12000 bf16 44 against 34 us, 20000 x 4001 76
// against 69; 65536 x 7168 366 against 371, 1003 x 5001 fp32 10.9 against 11.8.
constexpr int kMost = 4;
constexpr Geometry fwd_geometry(int64_t chunks) { return norm_geometry(chunks, kMost); }
static_assert(every_width<kMost, 2, false>(fwd_geometry) && every_width<kMost, 4, false>(fwd_geometry), "a width without a kernel");

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, int wdtype, bool layer, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    bool done = false;
    with_types(dtype, wdtype, [&](auto t, auto wt) {
        using T = decltype(t);
        done = with_geometry<kMost, sizeof(T), false>(fwd_geometry(norm_chunks(a.cols, sizeof(T))), [&](auto geo) {
            using G = decltype(geo);
            constexpr int block = norm_block(G::tpr), teams = block / G::tpr;
            const int64_t want = (a.rows + teams - 1) / teams, cap = static_cast<int64_t>(device_cu_count()) * (2048 / block);
            norm_fwd_kernel<T, decltype(wt), G::tpr, G::nv><<<static_cast<int>(want < cap ? want : cap), block, 0, s>>>(a, layer);
        });
    });
    return done ? hipGetLastError() : hipErrorInvalidConfiguration;
}

}  // namespace moe
