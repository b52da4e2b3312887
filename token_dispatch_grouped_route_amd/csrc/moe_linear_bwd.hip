// The linear map's backward around its two products: dz = dy act'(z), rounded to the operands' type since the
// matrix instruction takes it as a 16-bit operand, and db = the sum of the unrounded dz over the rows.
// Memory bound: dy and z are read once, dz written once (8192 x 4096 bf16, swiglu: 38 us, 4.4 TB/s).
#include "moe_columns.h"
#include "moe_linear.h"

namespace moe {
namespace {

// 512 columns of y by a run of rows a workgroup: a lane holds 8 columns, the four waves take every fourth row.
constexpr int kSlopeColumns = 512;

// As load8, in two steps.
template <typename T> struct Raw8 {
    u32x4_t lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    __device__ __forceinline__ void load(const void* base, int64_t at, bool f32, int valid) {
        if (f32) {
            lo = load_chunk<float>(static_cast<const float*>(base) + at, valid);
            hi = load_chunk<float>(static_cast<const float*>(base) + at + 4, valid - 4);
        } else {
            lo = load_chunk<T>(static_cast<const T*>(base) + at, valid);
        }
    }
    __device__ __forceinline__ void get(bool f32, float (&f)[8]) const {
        if (f32) {
            float a[4], b[4];
            unpack_chunk<float>(lo, a);
            unpack_chunk<float>(hi, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
        } else {
            unpack_chunk<T>(lo, f);
        }
    }
};

template <typename T> __global__ __launch_bounds__(256) void linear_slope_kernel(LinearSlope a) {
    __shared__ __align__(16) float join[4][2 * kSlopeColumns];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * kSlopeColumns + 8 * lane, valid = a.N - n;
    const bool pair = a.act == MOE_ACT_SWIGLU;
    float sum[8] = {}, sum_up[8] = {};
    const int64_t cols = pair ? 2 * static_cast<int64_t>(a.N) : a.N, per = (a.M + gridDim.y - 1) / gridDim.y, m1 = min(static_cast<int64_t>(a.M), (blockIdx.y + 1) * per);
    if (valid > 0) {
        // two rows at a time, whose loads are all in flight before the first is used: 8192 x 4096 bf16, swiglu, 42 to 38 us
        for (int64_t m0 = blockIdx.y * per + wave; m0 < m1; m0 += 8) {
            Raw8<T> rdy[2], rz[2], rup[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t m = min(m0 + 4 * r, m1 - 1);
                rdy[r].load(a.dy, m * a.lddy + n, a.dy_f32, valid);
                if (a.act != MOE_ACT_NONE) rz[r].load(a.z, m * a.ldz + n, false, valid);
                if (pair) rup[r].load(a.z, m * a.ldz + a.N + n, false, valid);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t m = m0 + 4 * r;
                if (m >= m1) break;
                float dy[8], z[8];
                rdy[r].get(a.dy_f32, dy);
                if (a.act != MOE_ACT_NONE) rz[r].get(false, z);
                if (pair) {
                    float up[8], dup[8];
                    rup[r].get(false, up);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dup[i] = dy[i] * __builtin_amdgcn_fmed3f(z[i], -128.0f, __builtin_inff()) * sigmoid_f32(z[i]);   // silu(-inf) = 0
                        dy[i] = dy[i] * up[i] * act_slope_f32(MOE_ACT_SILU, z[i]);
                        sum_up[i] += dup[i];
                    }
                    if (a.dz) store8<T>(a.dz, m * a.lddz + a.N + n, false, valid, dup);
                } else if (a.act != MOE_ACT_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dy[i] *= act_slope_f32(a.act, z[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += dy[i];
                if (a.dz) {
                    store8<T>(a.dz, m * a.lddz + n, false, valid, dy);
                    // zeros up to the row's end, a multiple of 8
                    for (int64_t c = cols; valid <= 8 && c < a.lddz; ++c) static_cast<T*>(a.dz)[m * a.lddz + c] = from_f32<T>(0.0f);
                }
            }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) join[wave][8 * lane + i] = sum[i], join[wave][kSlopeColumns + 8 * lane + i] = sum_up[i];
    __syncthreads();
    for (int c = threadIdx.x; c < (pair ? 2 : 1) * kSlopeColumns; c += 256) {
        const int at = blockIdx.x * kSlopeColumns + c % kSlopeColumns;
        if (at < a.N) a.part[blockIdx.y * cols + c / kSlopeColumns * a.N + at] = join[0][c] + join[1][c] + join[2][c] + join[3][c];
    }
}

}  // namespace

// Runs of rows: what fills the chip four workgroups a CU, and at least 8 rows, two a wave, each.
int64_t slope_slots(int64_t M, int64_t N) {
    const int64_t cap = 1024 / ((N + kSlopeColumns - 1) / kSlopeColumns), want = (M + 7) / 8;
    const int64_t n = want < cap ? want : cap;
    return n > 0 ? n : 1;
}

hipError_t launch_linear_slope(const LinearSlope& a, int dtype, int bdtype, void* db, hipStream_t s) {
    const int64_t slots = slope_slots(a.M, a.N), cols = (a.N + kSlopeColumns - 1) / kSlopeColumns;
    if (a.M > 0) {
        const dim3 grid(static_cast<unsigned>(cols), static_cast<unsigned>(slots));
        if (dtype == MOE_BF16) linear_slope_kernel<bf16_t><<<grid, 256, 0, s>>>(a);
        else linear_slope_kernel<fp16_t><<<grid, 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (db) {
        ColumnSums c = {};
        c.sum[0] = {a.part, db};
        c.groups[0] = 1;
        c.slots[0] = a.M > 0 ? slots : 0;
        c.cols = a.act == MOE_ACT_SWIGLU ? 2 * a.N : a.N;
        if (bdtype == MOE_FP32) launch_column_sums<float>(c, s);
        else if (bdtype == MOE_BF16) launch_column_sums<bf16_t>(c, s);
        else launch_column_sums<fp16_t>(c, s);
    }
    return hipGetLastError();
}

}  // namespace moe
