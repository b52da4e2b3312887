// The linear map for one to four rows: a token or a few of a decode step.  Bound by the weight, which is read once, in one
// launch: the vector unit multiplies each 16-byte chunk of it, as it comes, by the x of up to four rows in fp32, and the
// partial sums of a column meet in its workgroup, through lane exchanges and LDS in a fixed order.  The matrix core would
// need 16 rows or columns side by side, so more columns per workgroup, and then the reduction split over workgroups and a second launch.
#include <type_traits>

#include "moe_linear.h"

namespace moe {
namespace {

template <typename T> __device__ __forceinline__ u32x4_t chunk_of(const uint16_t* p, bool whole, int valid) {   // whole: the same for the launch
    return whole ? *reinterpret_cast<const u32x4_any_t*>(p) : load_chunk<T>(reinterpret_cast<const T*>(p), valid);
}

// What is done with one element of the product (for swiglu, of the gate's and the up's).
template <typename T> __device__ __forceinline__ void linear_out1(const Product& g, int m, int n, float v, float up) {
    auto load = [&](const void* p, int64_t i, bool f32) { return f32 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const T*>(p)[i]); };
    const bool pair = g.act == MOE_ACT_SWIGLU;
    if (g.bias) {
        v += load(g.bias, n, g.bias_f32);
        if (pair) up += load(g.bias, g.out_cols + n, g.bias_f32);
    }
    if (g.z) {
        T* z = static_cast<T*>(g.z) + m * g.ldz + n;
        z[0] = from_f32<T>(v);
        if (pair) z[g.out_cols] = from_f32<T>(up);
    }
    v = pair ? v * sigmoid_f32(v) * up : act_f32(g.act, v);
    if (g.residual) v += load(g.residual, m * g.ldr + n, g.y_f32);
    if (g.y_f32) static_cast<float*>(g.y)[m * g.ldy + n] = v;
    else static_cast<T*>(g.y)[m * g.ldy + n] = from_f32<T>(v);
}

// Weight by row (columns contiguous).  A workgroup of 16 waves takes 8 LANES columns (of the gate, and as many of the up where
// SETS is 2); a wave's load covers 64 / LANES rows of k in groups of 8 a lane, and the waves split K.
constexpr int kRowWaves = 16;
template <typename T, int ROWS, int SETS, int LANES>
__global__ __launch_bounds__(64 * kRowWaves) void linear_rows_kernel(Product g, bool whole) {
    constexpr int GROUPS = 64 / LANES, DEPTH = 8 * GROUPS, COLS = 8 * LANES;   // k of a wave's load
    __shared__ float part[kRowWaves][ROWS][SETS][COLS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane % LANES, group = lane / LANES;
    // neighbours in columns, which share cache lines, on one XCD (workgroup b is on XCD b mod 8)
    const int per = (gridDim.x + 7) / 8, block = (blockIdx.x & 7) * per + (blockIdx.x >> 3), n0 = block * COLS, n = n0 + 8 * c;
    if (n0 >= g.out_cols) return;
    const int valid = g.out_cols - n;
    float acc[ROWS][SETS][8] = {};
    const uint16_t* w = g.b + (whole && valid < 8 ? g.out_cols - 8 : n);   // past the last column: read again, not stored
    for (int k0 = wave * DEPTH + 8 * group; k0 < g.K; k0 += kRowWaves * DEPTH) {
        const int rows = min(8, g.K - k0);
        u32x4_t wt[8][SETS], xt[ROWS];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int s = 0; s < SETS; ++s) {   // past K: row K - 1 again, which is not multiplied
                const uint16_t* p = w + (k0 + min(i, rows - 1)) * g.ldb + s * g.out_cols;
                wt[i][s] = chunk_of<T>(p, whole, valid);
            }
#pragma unroll
        for (int m = 0; m < ROWS; ++m) xt[m] = load_chunk<T>(reinterpret_cast<const T*>(g.a) + min(m, g.M - 1) * g.lda + k0, rows);
        float fx[ROWS][8];
#pragma unroll
        for (int m = 0; m < ROWS; ++m) unpack_chunk<T>(xt[m], fx[m]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= rows) break;
#pragma unroll
            for (int s = 0; s < SETS; ++s) {
                float f[8];
                unpack_chunk<T>(wt[i][s], f);
#pragma unroll
                for (int m = 0; m < ROWS; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[m][s][j] += fx[m][i] * f[j];
            }
        }
    }
    // over the lanes of a column: three steps that halve the columns a lane holds (4, 2, 1), then whole sums
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int s = 0; s < SETS; ++s) {
            float(&v)[8] = acc[m][s];
            int col = 0;
#pragma unroll
            for (int half = 4, d = 32; half > 0; half >>= 1, d >>= 1) {
                const bool up = lane & d;
#pragma unroll
                for (int j = 0; j < half; ++j) {
                    const float send = up ? v[j] : v[j + half], keep = up ? v[j + half] : v[j];
                    v[j] = keep + __shfl_xor(send, d, 64);
                }
                col += up ? half : 0;
            }
#pragma unroll
            for (int d = 4; d >= LANES; d >>= 1) v[0] += __shfl_xor(v[0], d, 64);
            if ((lane & 7) < LANES) part[wave][m][s][8 * c + col] = v[0];   // lanes that differ in the other bits hold the same
        }
    lds_barrier();
    for (int at = threadIdx.x; at < ROWS * COLS; at += 64 * kRowWaves) {
        const int m = at / COLS, j = at % COLS;
        if (m >= g.M || n0 + j >= g.out_cols) continue;
        float v[SETS] = {};
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int i = 0; i < kRowWaves; ++i) v[s] += part[i][m][s][j];
        linear_out1<T>(g, m, n0 + j, v[0], v[SETS - 1]);
    }
}

// Weight by column (k contiguous): a wave takes two columns, the gate's and the up's of one output or two neighbours, and
// walks K with 512 k a load.
template <typename T, int ROWS>
__global__ __launch_bounds__(256) void linear_columns_kernel(Product g) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool pair = g.act == MOE_ACT_SWIGLU;
    const int n = (static_cast<int>(blockIdx.x) * 4 + wave) * (pair ? 1 : 2);
    if (n >= g.out_cols) return;
    const int second = pair ? g.out_cols + n : min(n + 1, g.out_cols - 1);
    const uint16_t *w0 = g.b + n * g.ldb, *w1 = g.b + second * g.ldb;
    float acc[ROWS][2] = {};
    auto add = [&](int k, int valid) {
        float f0[8], f1[8];
        unpack_chunk<T>(chunk_of<T>(w0 + k, valid >= 8, valid), f0);
        unpack_chunk<T>(chunk_of<T>(w1 + k, valid >= 8, valid), f1);
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            float fx[8];
            unpack_chunk<T>(chunk_of<T>(g.a + min(m, g.M - 1) * g.lda + k, valid >= 8, valid), fx);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[m][0] += fx[j] * f0[j], acc[m][1] += fx[j] * f1[j];
        }
    };
    int k = 8 * lane;
    const int end = g.K / 512 * 512;   // the same for the whole wave: no branch within these loads
#pragma unroll 4
    for (; k < end; k += 512) add(k, 8);
    if (k < g.K) add(k, g.K - k);
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
        acc[m][0] = wave_sum(acc[m][0]);
        acc[m][1] = wave_sum(acc[m][1]);
    }
    // lane 2 m + i writes column n + i of row m
    const int row = pair ? lane : lane >> 1, i = pair ? 0 : lane & 1;
    float v = acc[0][0], u = acc[0][1];
#pragma unroll
    for (int m = 1; m < ROWS; ++m) v = row == m ? acc[m][0] : v, u = row == m ? acc[m][1] : u;
    if (row < g.M && row < ROWS && n + i < g.out_cols) linear_out1<T>(g, row, n + i, pair || i == 0 ? v : u, u);
}

template <typename T, int ROWS> hipError_t run_rows(const Product& g, hipStream_t s) {
    if (!g.b_strided) {
        const int per = g.act == MOE_ACT_SWIGLU ? 4 : 8;
        linear_columns_kernel<T, ROWS><<<(g.out_cols + per - 1) / per, 256, 0, s>>>(g);
        return hipGetLastError();
    }
    const bool whole = g.out_cols % 8 == 0;
    auto go = [&](auto sets, auto lanes) {
        const int blocks = (g.out_cols + 8 * lanes() - 1) / (8 * lanes());
        linear_rows_kernel<T, ROWS, sets(), lanes()><<<(blocks + 7) / 8 * 8, 64 * kRowWaves, 0, s>>>(g, whole);
    };
    auto sets = [&](auto lanes) {
        if (g.act == MOE_ACT_SWIGLU) go(std::integral_constant<int, 2>{}, lanes);
        else go(std::integral_constant<int, 1>{}, lanes);
    };
    // 16 columns a workgroup, 32 once that makes two workgroups a CU
    if (g.out_cols >= 32 * 512) sets(std::integral_constant<int, 4>{});
    else sets(std::integral_constant<int, 2>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product_rows(const Product& g, int dtype, hipStream_t s) {
    auto types = [&](auto t) {
        using T = decltype(t);
        return g.M == 1 ? run_rows<T, 1>(g, s) : g.M == 2 ? run_rows<T, 2>(g, s) : run_rows<T, 4>(g, s);
    };
    return dtype == MOE_BF16 ? types(bf16_t{}) : types(fp16_t{});
}

}  // namespace moe
