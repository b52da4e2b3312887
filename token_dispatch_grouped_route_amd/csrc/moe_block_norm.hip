// Block norm, forward: moe_block_norm.h has the formulas.  Bound by memory: x and b are read once, r and n
// written once; a row is held in registers by a team of TPR threads, NV chunks of 16 bytes of b each, which forms
// every statistic from there (centred squares) and walks rows with the next row's loads in flight.  n is formed
// from r before its rounding.  8192 x 7168 bf16 with a stream in fp32, both norms and a gate: 137 us, 5.1 TB/s.
#include "moe_block_norm.h"

namespace moe {
namespace {

// A vector of a team's columns: held in registers, or, where a thread has many chunks, read from the caches row by row.
template <typename WT, int N, int NV, int TPR, bool HELD> struct FwdVector {
    NormWeights<WT, N, HELD ? NV : 1, TPR> v;
    const WT* p;
    float none;
    __device__ __forceinline__ void load(const void* w, int tid, int cols, float fill) {
        p = static_cast<const WT*>(w);
        none = fill;
        if constexpr (HELD) v.load(w, tid, cols, fill);
    }
    __device__ __forceinline__ void get(int j, int c, int cols, float (&f)[N]) {
        if constexpr (HELD) {
#pragma unroll
            for (int h = 0; h < NormWeights<WT, N, 1, TPR>::P; ++h) renew(v.raw[j][h]);
            v.get(j, f);
        } else if (p) {
            Pieces<WT, N> q;
            q.load(p + c, cols - c);
            q.get(f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = none;
        }
    }
};
// Waves a SIMD that the registers are cut down to: four where a thread has two chunks and everything is 16-bit, which leaves
// two workgroups of 512 a CU instead of one (with a stream in fp32 that spills: 8192 x 7168 140 to 155 us).
template <typename D, typename R, typename WT, int TPR, int NV> constexpr int fwd_waves() { return TPR == 1024 || (NV <= 2 && sizeof(WT) == sizeof(D) && sizeof(R) == sizeof(D)) ? 4 : 2; }

template <typename D, typename R, typename WT, int TPR, int NV>
__global__ __launch_bounds__(norm_block(TPR), (fwd_waves<D, R, WT, TPR, NV>())) void block_norm_fwd_kernel(BlockNorm a) {
    constexpr int N = Chunk<D>::N, BLOCK = norm_block(TPR), W = norm_waves(TPR);
    static_assert(sizeof(R) >= sizeof(D), "a stream at least as wide as the block's output");
    __shared__ float lds[8 * W];   // four sums per row, each in two buffers
    const int tid = threadIdx.x % TPR, cols = a.cols;
    const R* x = static_cast<const R*>(a.x);
    const D* b = static_cast<const D*>(a.b);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (BLOCK / TPR), row0 = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR);
    int64_t row = row0 + threadIdx.x / TPR;
    // teams past the last row run along with it (the exchanges need every lane) and store nothing
    auto in = [&](int64_t r) { return r < a.rows ? r : a.rows - 1; };
    Pieces<R, N> nx[NV];
    u32x4_t nb[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + tid) * N;
            nb[j] = load_chunk<D>(b + in(r) * a.ldb + c, cols - c);
            nx[j].load(x + in(r) * a.ldx + c, cols - c);
        }
    };
    fetch(row);
    FwdVector<WT, N, NV, TPR, (NV <= 2)> w1, c1, w2, c2, gate;
    w1.load(a.post_weight, tid, cols, 1.0f);
    c1.load(a.post_bias, tid, cols, 0.0f);
    w2.load(a.pre_weight, tid, cols, 1.0f);
    c2.load(a.pre_bias, tid, cols, 0.0f);
    const WT* gates = static_cast<const WT*>(a.gate);
    int64_t held = -1;   // the row of the gate in registers
    int slot = 0;
    // mean and rstd of v, which is centred; elements past the row's end become 0
    auto normalise = [&](float (&v)[NV][N], int area, float& mean, float& rstd) {
        mean = 0.0f;
        if (a.layer) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) s[0] += v[j][i];
            team_sum<TPR, 1>(s, lds + 2 * W * area, slot);
            mean = s[0] / static_cast<float>(cols);
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int valid = cols - (j * TPR + tid) * N;
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] -= mean;
            if (valid < N) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] = i < valid ? v[j][i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) q[0] += v[j][i] * v[j][i];
        }
        team_sum<TPR, 1>(q, lds + 2 * W * (area + 1), slot);
        rstd = q[0] < __builtin_inff() ? 1.0f / sqrtf(q[0] / static_cast<float>(cols) + a.eps) : __builtin_nanf("");   // as the row norm
    };
    for (int64_t base = row0; base < a.rows; base += step, row += step) {
        float v[NV][N], mean, rstd;
        Pieces<R, N> x_now[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack_chunk<D>(nb[j], v[j]);
            x_now[j] = nx[j];
        }
        if (base + step < a.rows) fetch(row + step);
        if (gates && in(row) / a.gate_share != held) {
            held = in(row) / a.gate_share;
            gate.load(gates + held * cols, tid, cols, 1.0f);
        }
        if (a.post) {
            normalise(v, 0, mean, rstd);
            if (row < a.rows && tid == 0) {
                if (a.layer && a.post_mean) a.post_mean[row] = mean;
                if (a.post_rstd) a.post_rstd[row] = rstd;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float w[N], c[N];
                w1.get(j, (j * TPR + tid) * N, cols, w);
                c1.get(j, (j * TPR + tid) * N, cols, c);
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] = v[j][i] * rstd * w[i] + c[i];
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (gates) {
                float g[N];
                gate.get(j, (j * TPR + tid) * N, cols, g);
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] *= g[i];
            }
            float fx[N];
#pragma unroll
            for (int h = 0; h < Pieces<R, N>::P; ++h) renew(x_now[j].raw[h]);
            x_now[j].get(fx);
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] = a.x_scale * fx[i] + a.scale * v[j][i];
            const int c = (j * TPR + tid) * N;
            if (row < a.rows) Pieces<R, N>::put(static_cast<R*>(a.r) + row * a.ldr + c, v[j], cols - c);
        }
        if (a.pre) {
            // past the row's end: b and x are 0 there, but not the weights' biases
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (cols - (j * TPR + tid) * N < N) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[j][i] = i < cols - (j * TPR + tid) * N ? v[j][i] : 0.0f;
                }
            normalise(v, 2, mean, rstd);
            if (row < a.rows) {
                if (tid == 0) {
                    if (a.layer && a.pre_mean) a.pre_mean[row] = mean;
                    if (a.pre_rstd) a.pre_rstd[row] = rstd;
                }
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int at = (j * TPR + tid) * N;
                    float w[N], c[N], o[N];
                    w2.get(j, at, cols, w);
                    c2.get(j, at, cols, c);
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = v[j][i] * rstd * w[i] + c[i];
                    store_chunk<D>(static_cast<D*>(a.n) + row * a.ldn + at, pack_chunk<D>(o), cols - at);
                }
            }
        }
        slot ^= 1;
    }
}

// Calls f with a team for rows of `chunks` 16-byte chunks of b; false if they are too long for any.
template <typename D, typename F> bool with_team(int64_t chunks, F&& f) {
    if (chunks <= 16) f(Geo<16, 1>{});
    else if (chunks <= 64) f(Geo<64, 1>{});
    else if (chunks <= 128) f(Geo<128, 1>{});
    else if (chunks <= 256) f(Geo<256, 1>{});
    else if (chunks <= 512) f(Geo<256, 2>{});
    else if (chunks <= 1024) f(Geo<512, 2>{});
    else if (sizeof(D) == 4 && chunks <= 2048) f(Geo<1024, 2>{});
    else if (chunks <= 2048) f(Geo<512, 4>{});
    else if (chunks <= 4096) f(Geo<512, 8>{});
    else if (chunks <= 8192) f(Geo<1024, 8>{});
    else return false;
    return true;
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNorm& a, int dtype, int sdtype, int wdtype, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    bool done = false;
    with_types(dtype, wdtype, [&](auto t, auto wt) {
        using D = decltype(t);
        using WT = decltype(wt);
        auto go = [&](auto stream) {
            using R = decltype(stream);
            done = with_team<D>(norm_chunks(a.cols, sizeof(D)), [&](auto geo) {
                using G = decltype(geo);
                if constexpr (sizeof(D) == 4 ? G::nv != 4 : G::tpr < 1024) {   // the teams of this type
                    constexpr int block = norm_block(G::tpr), teams = block / G::tpr;
                    const int64_t want = (a.rows + teams - 1) / teams, cap = static_cast<int64_t>(device_cu_count()) * (2048 / block);
                    block_norm_fwd_kernel<D, R, WT, G::tpr, G::nv><<<static_cast<int>(want < cap ? want : cap), block, 0, s>>>(a);
                }
            });
        };
        if (sdtype == dtype) go(t);
        else go(float{});
    });
    return done ? hipGetLastError() : hipErrorInvalidConfiguration;
}

}  // namespace moe
