// Row norm, backward, with the reduction of the weight's and the bias's gradient: moe_norm.h has the
// formulas and the plan.  A thread sums its columns' dy xh and dy over its team's rows in fp32; the teams
// of a workgroup are joined in LDS, a workgroup leaves one partial row of dw and db, and a second launch
// sums those, all in a fixed order: no atomics, the same bits on every run.
// RMS norm of 65536 x 7168 bf16: 546 + 6 us (5.2 TB/s); layer norm of 1003 x 5001 fp32: 14 + 4 us, of 8192 x
// 7168 bf16: 74 us.
#include "moe_norm.h"

namespace moe {

template <typename T, typename WT, bool LAYER, int TPR, int NV>
__global__ __launch_bounds__(norm_block(TPR)) void norm_bwd_kernel(NormArgs a) {
    constexpr int N = Chunk<T>::N, BLOCK = norm_block(TPR), TEAMS = BLOCK / TPR, NS = LAYER ? 2 : 1, W = norm_waves(TPR);
    __shared__ float lds[2 * NS * W];
    __shared__ __align__(16) float join[TEAMS > 1 ? TEAMS * TPR * NV * N : 1];
    const int tid = threadIdx.x % TPR, team = threadIdx.x / TPR, cols = a.cols;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.y);
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS, row0 = static_cast<int64_t>(blockIdx.x) * TEAMS;
    int64_t row = row0 + team;

    NormWeights<WT, N, NV, TPR> w;
    float dw[NV][N], db[NV][N];
    u32x4_t nx[NV], ny[NV];   // the next row
    auto fetch = [&](int64_t r) {   // a team past the last row runs along with that one
        r = r < a.rows ? r : a.rows - 1;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx[j] = load_ahead<T, TPR == 8>(x + r * a.ldx, (j * TPR + tid) * N, cols);
            ny[j] = load_ahead<T, TPR == 8>(dy + r * a.lddy, (j * TPR + tid) * N, cols);
        }
    };
    fetch(row);
    float nmean = LAYER && row < a.rows ? a.mean[row] : 0.0f, nrstd = row < a.rows ? a.rstd[row] : 0.0f;
    w.load(a.weight, tid, cols, 1.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[j][i] = db[j][i] = 0.0f;
    const float inv = 1.0f / static_cast<float>(cols);
    int slot = 0;
    for (int64_t base = row0; base < a.rows; base += step, row += step) {
        u32x4_t rx[NV], ry[NV];
        const float mean = nmean, rstd = nrstd;
        // elements past the row's end, and rows past the last, get dy = 0 and x = 0: they add nothing to any sum
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j] = settle<T, TPR == 8>(nx[j], (j * TPR + tid) * N, cols);
            ry[j] = settle<T, TPR == 8>(ny[j], (j * TPR + tid) * N, cols);
            if (TEAMS > 1 && row >= a.rows) rx[j] = ry[j] = u32x4_t{0, 0, 0, 0};
        }
        if (base + step < a.rows) fetch(row + step);
        nmean = nrstd = 0.0f;
        if (row + step < a.rows) {
            if (LAYER) nmean = a.mean[row + step];
            nrstd = a.rstd[row + step];
        }
        float s[NS] = {};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float fx[N], fy[N], fw[N];
            unpack_chunk<T>(rx[j], fx);
            unpack_chunk<T>(ry[j], fy);
            w.get(j, fw);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float xh = (fx[i] - mean) * rstd, g = fy[i] * fw[i];
                dw[j][i] += fy[i] * xh;
                if constexpr (LAYER) {
                    db[j][i] += fy[i];
                    s[1] += g;
                }
                s[0] += g * xh;
            }
        }
        team_sum<TPR, NS>(s, lds, slot);
        slot ^= 1;
        const float c0 = s[0] * inv, c1 = LAYER ? s[NS - 1] * inv : 0.0f;
        if (dx && row < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                float fx[N], fy[N], fw[N], o[N];
                unpack_chunk<T>(rx[j], fx);
                unpack_chunk<T>(ry[j], fy);
                w.get(j, fw);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float xh = (fx[i] - mean) * rstd;
                    o[i] = rstd * (fy[i] * fw[i] - c1 - xh * c0);
                }
                store_chunk<T>(dx + row * a.lddx + c, pack_chunk<T>(o), cols - c);
            }
        }
    }
    // the workgroup's partial row of one gradient
    auto leave = [&](float* part, const float (&sum)[NV][N]) {
        if (!part) return;   // the same for the whole launch
        part += static_cast<int64_t>(blockIdx.x) * cols;
        if constexpr (TEAMS == 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int h = 0; h < N / 4; ++h) {
                    const int c = (j * TPR + tid) * N + 4 * h;
                    const float o[4] = {sum[j][4 * h], sum[j][4 * h + 1], sum[j][4 * h + 2], sum[j][4 * h + 3]};
                    store_chunk<float>(part + c, pack_chunk<float>(o), cols - c);
                }
        } else {
            constexpr int WIDE = TPR * NV * N;
            lds_barrier();   // the other gradient's sums are no longer read
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) join[team * WIDE + (j * TPR + tid) * N + i] = sum[j][i];
            lds_barrier();
            for (int c = threadIdx.x; c < cols; c += BLOCK) {
                float t = 0.0f;
#pragma unroll
                for (int k = 0; k < TEAMS; ++k) t += join[k * WIDE + c];
                part[c] = t;
            }
        }
    };
    leave(a.part_w, dw);
    if (LAYER) leave(a.part_b, db);
}

// dw and db: the sum over the partial rows, 64 columns a workgroup: 16 lanes of four columns by 64 groups
// of rows (group i takes rows i, i + 64, ...), then the groups are added in order.  No rows: zeros.
// 512 rows of 7168: 6.4 us, most of it the latency of eight loads in flight and a launch.
constexpr int kReduceGroups = 64;
template <typename WT>
__global__ __launch_bounds__(16 * kReduceGroups) void norm_reduce_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b,
                                                                         int64_t slots, int cols, WT* __restrict__ dw, WT* __restrict__ db) {
    __shared__ __align__(16) float lds[kReduceGroups][64 + 4];
    const float* part = blockIdx.y ? part_b : part_w;
    WT* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, c = blockIdx.x * 64 + 4 * lane;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int64_t t = group; t < slots; t += kReduceGroups) {
        float f[4];
        unpack_chunk<float>(load_chunk<float>(part + t * cols + c, cols - c), f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += f[i];
    }
    *reinterpret_cast<u32x4_t*>(&lds[group][4 * lane]) = pack_chunk<float>(s);
    __syncthreads();
    if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < static_cast<unsigned>(cols)) {
        float t = 0.0f;
#pragma unroll 16
        for (int k = 0; k < kReduceGroups; ++k) t += lds[k][threadIdx.x];
        out[blockIdx.x * 64 + threadIdx.x] = from_f32<WT>(t);
    }
}

// A thread takes at most 16 elements of a row where it can: its two sums per element, the row, the next row
// and the weights then leave three (layer norm) or four waves a SIMD (rms backward of 65536 x 7168 bf16: 545
// to 555 us; with 32 elements, 588 to 630 us).  Layer norm rows of more than 512 x 16 elements take up to 32
// in the same 512 threads (12000-wide: 72 us for 4000 rows; 1024 threads of 16 spill, 136 us).
// Rows of more than 12288 elements spill registers (the layer norm's, and fp32 RMS): 2000 x 14000 fp32 151 us for
// layer norm, 92 for RMS, 4000 x 14000 bf16 96 and 70, with 69 us of bytes to move.  Above 16384 elements, where 1024
// threads with 128 registers each hold the row, the next row and the sums, scratch traffic is most of the time:
// 1000 x 32768 fp32 690 and 540 us for 80 us of bytes, 2000 x 20000 bf16 layer norm 290 for 49.
constexpr int bwd_most(int elem_bytes) { return elem_bytes == 4 ? 4 : 2; }
constexpr Geometry bwd_geometry(int64_t chunks, int elem_bytes, bool layer) {
    const int most = bwd_most(elem_bytes);
    Geometry g = norm_geometry(chunks, most);
    if (layer && g.tpr == 1024 && chunks <= 512 * 2 * most) g = {512, static_cast<int>((chunks + 511) / 512)};
    if (elem_bytes == 4 && g.tpr == 512 && g.nv > 4) g.nv = g.nv <= 6 ? 6 : 8;
    return g;
}
template <int BYTES, bool LAYER> constexpr bool every_bwd_width() {
    return every_width<bwd_most(BYTES), BYTES, LAYER>([](int64_t chunks) { return bwd_geometry(chunks, BYTES, LAYER); });
}
static_assert(every_bwd_width<2, true>() && every_bwd_width<2, false>() && every_bwd_width<4, true>() && every_bwd_width<4, false>(), "a width without a kernel");
// Workgroups a CU holds.
constexpr int bwd_per_cu(const Geometry& g, bool layer) { return layer ? (g.tpr <= 256 ? 3 : 1) : g.tpr <= 256 ? 4 : g.tpr == 512 ? 2 : 1; }

// Workgroups of the backward (each leaves one partial row of dw and db): what fills the chip, and at least
// two rows a team, which halves the partial rows of a short batch.
constexpr int kCus = 256;   // MI355X: a constant, so that the workspace's size follows from the sizes alone
int64_t norm_bwd_slots(int64_t rows, int cols, int elem_bytes, bool layer) {
    const Geometry g = bwd_geometry(norm_chunks(cols, elem_bytes), elem_bytes, layer);
    const int64_t cap = kCus * bwd_per_cu(g, layer);
    const int teams = norm_block(g.tpr) / g.tpr;
    const int64_t want = (rows + 2 * teams - 1) / (2 * teams);
    return want < cap ? want : cap;
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, int wdtype, bool layer, hipStream_t s) {
    bool done = true;
    with_types(dtype, wdtype, [&](auto t, auto wt) {
        using T = decltype(t);
        using WT = decltype(wt);
        constexpr int bytes = sizeof(T), most = bwd_most(bytes);
        const int64_t slots = norm_bwd_slots(a.rows, a.cols, bytes, layer);
        const Geometry g = bwd_geometry(norm_chunks(a.cols, bytes), bytes, layer);
        if (slots > 0 && layer) {
            done = with_geometry<most, bytes, true>(g, [&](auto geo) {
                using G = decltype(geo);
                norm_bwd_kernel<T, WT, true, G::tpr, G::nv><<<static_cast<int>(slots), norm_block(G::tpr), 0, s>>>(a);
            });
        } else if (slots > 0) {
            done = with_geometry<most, bytes, false>(g, [&](auto geo) {
                using G = decltype(geo);
                norm_bwd_kernel<T, WT, false, G::tpr, G::nv><<<static_cast<int>(slots), norm_block(G::tpr), 0, s>>>(a);
            });
        }
        if (done && (a.dweight || a.dbias))
            norm_reduce_kernel<WT><<<dim3((a.cols + 63) / 64, a.dbias ? 2 : 1), 16 * kReduceGroups, 0, s>>>(
                a.part_w, a.part_b, slots, a.cols, static_cast<WT*>(a.dweight), static_cast<WT*>(a.dbias));
    });
    return done ? hipGetLastError() : hipErrorInvalidConfiguration;
}

}  // namespace moe
