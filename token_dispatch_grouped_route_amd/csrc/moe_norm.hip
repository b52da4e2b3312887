// Row norm, forward and backward (layer norm and RMS norm), with the reduction of the weight's and
// the bias's gradient.
//
//   forward   mean = sum x / C (layer norm; 0 for RMS), s = 1 / sqrt(sum (x - mean)^2 / C + eps),
//             xh = (x - mean) s,  y = xh w + b
//   backward  g = dy w;  dx = s (g - [layer] sum g / C - xh sum (g xh) / C);
//             dw = sum over rows of dy xh;  db = sum over rows of dy
//
// Both are bound by memory: each element is read once and written once, every statistic is formed
// from registers.  A row is held by TPR threads (a wave for short rows, a workgroup for long ones),
// NV 16-byte chunks each, so the variance is a sum of centred squares at no extra read.  A team of
// TPR threads walks rows at a fixed stride with the next row's loads in flight while this row is
// reduced, and keeps the weights (backward: its columns' share of dw and db, in fp32) in registers
// from row to row.  Each team of the backward then writes one partial row of dw and db, and a second
// launch sums them in a fixed order: no atomics, the same bits on every run.
#include <type_traits>

#include "moe_vec.h"

namespace moe {

// The sums over a row's TPR threads of NS values, in every thread.  `slot` alternates between two
// LDS buffers from one call to the next, so one barrier per call is enough.
template <int TPR, int NS>
__device__ __forceinline__ void team_sum(float (&v)[NS], float* lds, int slot) {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        float* buf = lds + slot * W * NS;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NS; ++i) buf[wave * NS + i] = v[i];
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) t += buf[w * NS + i];
            v[i] = t;
        }
    }
}

template <typename WT, int N> __device__ __forceinline__ void load_weights(const WT* w, int64_t c, int valid, float none, float (&f)[N]) {
    constexpr int WN = Chunk<WT>::N;
#pragma unroll
    for (int h = 0; h < N / WN; ++h) {
        float part[WN];
        if (w) {
            unpack_chunk<WT>(load_chunk<WT>(w + c + h * WN, valid - h * WN), part);
        } else {
#pragma unroll
            for (int i = 0; i < WN; ++i) part[i] = none;
        }
#pragma unroll
        for (int i = 0; i < WN; ++i) f[h * WN + i] = part[i];
    }
}

template <typename T, typename WT, bool LAYER, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(NormArgs a) {
    constexpr int N = Chunk<T>::N, BLOCK = TPR < 256 ? 256 : TPR;
    __shared__ float lds[4 * (TPR / 64)];   // two sums per row (mean, variance), each in two buffers
    const int tid = threadIdx.x % TPR, cols = a.cols;
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (BLOCK / TPR);
    int64_t row = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR) + threadIdx.x / TPR;
    if (row >= a.rows) return;   // a whole team (TPR > 64: the whole workgroup)

    float w[NV][N], b[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tid) * N;
        load_weights<WT, N>(static_cast<const WT*>(a.weight), c, cols - c, 1.0f, w[j]);
        load_weights<WT, N>(static_cast<const WT*>(a.bias), c, cols - c, 0.0f, b[j]);
    }
    u32x4_t next[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tid) * N;
        next[j] = load_chunk<T>(x + row * a.ldx + c, cols - c);
    }
    int slot = 0;
    for (; row < a.rows; row += step) {
        float v[NV][N];
#pragma unroll
        for (int j = 0; j < NV; ++j) unpack_chunk<T>(next[j], v[j]);
        if (row + step < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                next[j] = load_chunk<T>(x + (row + step) * a.ldx + c, cols - c);
            }
        }
        float mean = 0.0f;
        if constexpr (LAYER) {
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
            if (valid >= N) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    v[j][i] -= mean;
                    q[0] += v[j][i] * v[j][i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    v[j][i] = i < valid ? v[j][i] - mean : 0.0f;
                    q[0] += v[j][i] * v[j][i];
                }
            }
        }
        team_sum<TPR, 1>(q, lds + 2 * (TPR / 64), slot);
        slot ^= 1;
        const float rstd = 1.0f / sqrtf(q[0] / static_cast<float>(cols) + a.eps);
        if (tid == 0) {
            if (LAYER && a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + tid) * N;
            float o[N];
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = v[j][i] * rstd * w[j][i] + b[j][i];
            store_chunk<T>(y + row * a.ldy + c, pack_chunk<T>(o), cols - c);
        }
    }
}

template <typename T, typename WT, bool LAYER, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(NormArgs a, int64_t slots) {
    constexpr int N = Chunk<T>::N, BLOCK = TPR < 256 ? 256 : TPR, NS = LAYER ? 2 : 1;
    __shared__ float lds[2 * NS * (TPR / 64)];
    const int tid = threadIdx.x % TPR, cols = a.cols;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.y);
    const int64_t team = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR) + threadIdx.x / TPR;
    if (team >= slots) return;

    float w[NV][N], dw[NV][N], db[NV][N];
    u32x4_t nx[NV], ny[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + tid) * N;
        load_weights<WT, N>(static_cast<const WT*>(a.weight), c, cols - c, 1.0f, w[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) dw[j][i] = db[j][i] = 0.0f;
        nx[j] = load_chunk<T>(x + team * a.ldx + c, cols - c);       // slots <= rows
        ny[j] = load_chunk<T>(dy + team * a.lddy + c, cols - c);
    }
    float nmean = LAYER ? a.mean[team] : 0.0f, nrstd = a.rstd[team];
    const float inv = 1.0f / static_cast<float>(cols);
    int slot = 0;
    for (int64_t row = team; row < a.rows; row += slots) {
        u32x4_t rx[NV], ry[NV];
        const float mean = nmean, rstd = nrstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) rx[j] = nx[j], ry[j] = ny[j];
        if (row + slots < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                nx[j] = load_chunk<T>(x + (row + slots) * a.ldx + c, cols - c);
                ny[j] = load_chunk<T>(dy + (row + slots) * a.lddy + c, cols - c);
            }
            if (LAYER) nmean = a.mean[row + slots];
            nrstd = a.rstd[row + slots];
        }
        // elements past the row's end have dy = 0 and w = 0, so they add nothing to any sum
        float s[NS] = {};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float fx[N], fy[N];
            unpack_chunk<T>(rx[j], fx);
            unpack_chunk<T>(ry[j], fy);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float xh = (fx[i] - mean) * rstd, g = fy[i] * w[j][i];
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
        if (dx) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * TPR + tid) * N;
                float fx[N], fy[N], o[N];
                unpack_chunk<T>(rx[j], fx);
                unpack_chunk<T>(ry[j], fy);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float xh = (fx[i] - mean) * rstd;
                    o[i] = rstd * (fy[i] * w[j][i] - c1 - xh * c0);
                }
                store_chunk<T>(dx + row * a.lddx + c, pack_chunk<T>(o), cols - c);
            }
        }
    }
    if (a.part_w) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + tid) * N;
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const float o[4] = {dw[j][4 * h], dw[j][4 * h + 1], dw[j][4 * h + 2], dw[j][4 * h + 3]};
                store_chunk<float>(a.part_w + team * cols + c + 4 * h, pack_chunk<float>(o), cols - c - 4 * h);
            }
        }
    }
    if (LAYER && a.part_b) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + tid) * N;
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const float o[4] = {db[j][4 * h], db[j][4 * h + 1], db[j][4 * h + 2], db[j][4 * h + 3]};
                store_chunk<float>(a.part_b + team * cols + c + 4 * h, pack_chunk<float>(o), cols - c - 4 * h);
            }
        }
    }
}

// dw and db: the sum over the teams' partial rows, 64 columns a workgroup; wave i takes the teams
// i, i + 16, ..., then the sixteen sums are added in wave order.  No team (no rows): zeros.
constexpr int kReduceWaves = 16;
template <typename WT>
__global__ __launch_bounds__(64 * kReduceWaves) void norm_reduce_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b,
                                                                        int64_t slots, int cols, WT* __restrict__ dw, WT* __restrict__ db) {
    __shared__ float lds[kReduceWaves][64];
    const float* part = blockIdx.y ? part_b : part_w;
    WT* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t t = wave; t < slots; t += kReduceWaves) s += part[t * cols + c];
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < cols) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kReduceWaves; ++w) s += lds[w][lane];
        out[c] = from_f32<WT>(s);
    }
}

namespace {

// Threads per row and chunks per thread of a row of `chunks` 16-byte chunks: a wave (no barrier) up
// to 256 chunks, then workgroups of 256, 512 and 1024.
struct Geometry { int tpr, nv; };
Geometry geometry(int64_t chunks) {
    if (chunks <= 64) return {64, 1};
    if (chunks <= 128) return {64, 2};
    if (chunks <= 256) return {64, 4};
    if (chunks <= 512) return {256, 2};
    if (chunks <= 1024) return {256, 4};
    if (chunks <= 2048) return {512, 4};
    if (chunks <= 4096) return {1024, 4};
    return {1024, 8};
}

template <typename T, typename WT, bool LAYER, typename F> void with_geometry(const Geometry& g, F&& f) {
    if (g.tpr == 64 && g.nv == 1) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (g.tpr == 64 && g.nv == 2) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else if (g.tpr == 64) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    else if (g.tpr == 256 && g.nv == 2) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (g.tpr == 256) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    else if (g.tpr == 512) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
    else if (g.nv == 4) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    else if constexpr (sizeof(T) == 4) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

constexpr int kCus = 256;   // MI355X; the partial rows of the backward are sized from it

int64_t chunks_of(int cols, int elem_bytes) { return (static_cast<int64_t>(cols) * elem_bytes + 15) / 16; }

template <typename T, typename WT, bool LAYER> void run_fwd(const NormArgs& a, hipStream_t s) {
    const Geometry g = geometry(chunks_of(a.cols, sizeof(T)));
    const int per = g.tpr < 256 ? 256 / g.tpr : 1;   // rows a workgroup works on at once
    const int64_t want = (a.rows + per - 1) / per, cap = static_cast<int64_t>(device_cu_count()) * (2048 / (g.tpr < 256 ? 256 : g.tpr));
    const int grid = static_cast<int>(want < cap ? want : cap);
    with_geometry<T, WT, LAYER>(g, [&](auto tpr, auto nv) {
        norm_fwd_kernel<T, WT, LAYER, tpr(), nv()><<<grid, g.tpr < 256 ? 256 : g.tpr, 0, s>>>(a);
    });
}

template <typename T, typename WT, bool LAYER> void run_bwd(const NormArgs& a, hipStream_t s) {
    const Geometry g = geometry(chunks_of(a.cols, sizeof(T)));
    const int64_t slots = norm_bwd_slots(a.rows, a.cols, sizeof(T));
    const int per = g.tpr < 256 ? 256 / g.tpr : 1;
    if (slots > 0) {
        const int grid = static_cast<int>((slots + per - 1) / per);
        with_geometry<T, WT, LAYER>(g, [&](auto tpr, auto nv) {
            norm_bwd_kernel<T, WT, LAYER, tpr(), nv()><<<grid, g.tpr < 256 ? 256 : g.tpr, 0, s>>>(a, slots);
        });
    }
    if (a.dweight || a.dbias)
        norm_reduce_kernel<WT><<<dim3((a.cols + 63) / 64, a.dbias ? 2 : 1), 64 * kReduceWaves, 0, s>>>(
            a.part_w, a.part_b, slots, a.cols, static_cast<WT*>(a.dweight), static_cast<WT*>(a.dbias));
}

template <typename F> void with_types(int dtype, int wdtype, bool layer, F&& f) {
    auto kind = [&](auto t, auto w) {
        if (layer) f(t, w, std::true_type{});
        else f(t, w, std::false_type{});
    };
    if (dtype == MOE_FP32) kind(float{}, float{});
    else if (dtype == MOE_BF16 && wdtype == MOE_BF16) kind(bf16_t{}, bf16_t{});
    else if (dtype == MOE_BF16) kind(bf16_t{}, float{});
    else if (wdtype == MOE_FP16) kind(fp16_t{}, fp16_t{});
    else kind(fp16_t{}, float{});
}

}  // namespace

// Teams of the backward (each leaves one partial row of dw and db): what fills the chip, and no more
// than one per 8 rows, so that the partial rows stay small next to x and dy.
int64_t norm_bwd_slots(int64_t rows, int cols, int elem_bytes) {
    const Geometry g = geometry(chunks_of(cols, elem_bytes));
    const int64_t cap = static_cast<int64_t>(kCus) * (g.tpr == 64 ? 8 : g.tpr == 256 ? 3 : 1), want = (rows + 7) / 8;
    return want < cap ? want : cap;
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, int wdtype, bool layer, hipStream_t s) {
    if (a.rows > 0)
        with_types(dtype, wdtype, layer, [&](auto t, auto w, auto l) { run_fwd<decltype(t), decltype(w), l()>(a, s); });
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, int wdtype, bool layer, hipStream_t s) {
    with_types(dtype, wdtype, layer, [&](auto t, auto w, auto l) { run_bwd<decltype(t), decltype(w), l()>(a, s); });
    return hipGetLastError();
}

}  // namespace moe
