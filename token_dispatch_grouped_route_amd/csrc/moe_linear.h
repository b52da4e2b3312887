// The linear map: what its product kernels (moe_linear.hip) and its backward (moe_linear_bwd.hip) share.
//
//   forward   z = x W + b;  y = act(z) + residual  (swiglu: W has [gate | up] columns, act = silu(gate) up)
//   backward  dz = dy act'(z);  dx = dz W^T;  dW = x^T dz;  db = sum over the rows of dz
#pragma once

#include "moe_vec.h"

namespace moe {

// C [M, N] = A B over a reduction of length K.  An operand is stored with the reduction contiguous (element
// (i, k) at i ld + k) or strided (k ld + i), i a row of A or a column of B; 16-bit floats.
struct Product {
    int32_t M, N, K;
    bool a_strided, b_strided;
    const uint16_t *a, *b;
    int64_t lda, ldb;
    bool a_padded, b_padded; // its rows are followed by zeros up to a multiple of 8
    // what is done with C
    int32_t act, out_cols;   // moe_act; columns of y: N, or N / 2 for swiglu
    const void *bias, *residual;
    void *y, *z;
    int64_t ldr, ldy, ldz;
    bool bias_f32, y_f32;    // z is in the operands' type, residual in y's
    // the reduction split over workgroups: fp32 partial sums [splits, M, N], joined by a second launch
    float* part;
    int32_t splits, slots;   // 64-deep steps of the reduction per split
};

constexpr int kLinearDepth = 64;   // reduction elements per step

// dz and db.
struct LinearSlope {
    int32_t M, N, act;   // N: columns of y
    const void *dy, *z;
    int64_t lddy, ldz, lddz;
    bool dy_f32;
    void* dz;      // NULL: db alone
    float* part;   // [slope_slots, columns of z] partial rows of db, NULL: none
};
int64_t slope_slots(int64_t M, int64_t N);
hipError_t launch_linear_slope(const LinearSlope& a, int dtype, int bdtype, void* db, hipStream_t s);

// Bytes that launch_product may write at `part` for a product of these sizes.
size_t product_part_bytes(int64_t M, int64_t N, int64_t K);
// Bytes of the padded copies of operands of a and b elements (0: none is wanted) that it makes at `pad` where that pays.
int64_t padded_elements(int64_t rows, int64_t extent);   // 0 where extent is a multiple of 8
size_t product_pad_bytes(int64_t M, int64_t N, int64_t K, int64_t a, int64_t b);
// pad_bytes: room at `pad`; with less than a product's copies need it makes none.
hipError_t launch_product(Product g, int dtype, void* part, void* pad, size_t pad_bytes, hipStream_t s);
// The products of 1 to kLinearRows rows whose A has the reduction contiguous (moe_linear_rows.hip), without workspace.
constexpr int kLinearRows = 4;
hipError_t launch_product_rows(const Product& g, int dtype, hipStream_t s);
// Those of 1 to kLinearFew rows whose operands' 16-byte chunks are whole (moe_linear_few.hip).  Beyond, x costs more than the tiles'
// idle rows: 4096 x 7168, weight by row, 16 rows 21.8 against 23.6 us, 32 rows 24.4 and 24.9, 48 rows 27.5 and 25.8.
constexpr int kLinearFew = 32;
int few_splits(int64_t M, int64_t N, int64_t K, bool strided);
hipError_t launch_product_few(Product g, int dtype, void* part, hipStream_t s);
// Adds the partial sums of g.splits and finishes y.
hipError_t launch_product_join(const Product& g, int dtype, hipStream_t s);

__device__ __forceinline__ float sigmoid_f32(float z) { return 1.0f / (1.0f + expf(-z)); }
__device__ __forceinline__ float gelu_cdf(float z) { return 0.5f * (1.0f + erff(z * 0.70710678118654752f)); }
__device__ __forceinline__ float act_f32(int act, float z) {   // not swiglu
    switch (act) {
        case MOE_ACT_RELU: return z <= 0.0f ? 0.0f : z;   // NaN stays
        case MOE_ACT_GELU: return z * gelu_cdf(z);
        case MOE_ACT_SILU: return z * sigmoid_f32(z);
        default: return z;
    }
}
// The factor z beside a term that is 0 (or a sum that has reached its limit) in fp32 from 128 on: an infinite z, as fp16 keeps a finite
// one beyond 65504, then gives the slope's limit and not infinity times 0.  NaN comes through the other factor, formed from z itself.
__device__ __forceinline__ float at_most_128(float z) { return __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f); }
__device__ __forceinline__ float act_slope_f32(int act, float z) {   // silu also for swiglu's gate
    switch (act) {
        case MOE_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case MOE_ACT_GELU: return gelu_cdf(z) + at_most_128(z) * 0.39894228040143268f * expf(-0.5f * z * z);
        case MOE_ACT_NONE: return 1.0f;
        default: {
            const float s = sigmoid_f32(z);
            return s * (1.0f + at_most_128(z) * (1.0f - s));
        }
    }
}

// Eight consecutive elements at p of which `valid` exist, T or fp32.
template <typename T> __device__ __forceinline__ void load8(const void* base, int64_t at, bool f32, int valid, float (&f)[8]) {
    if (f32) {
        const float* p = static_cast<const float*>(base) + at;
        float lo[4], hi[4];
        unpack_chunk<float>(load_chunk<float>(p, valid), lo);
        unpack_chunk<float>(load_chunk<float>(p + 4, valid - 4), hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = lo[i], f[4 + i] = hi[i];
    } else {
        unpack_chunk<T>(load_chunk<T>(static_cast<const T*>(base) + at, valid), f);
    }
}
template <typename T> __device__ __forceinline__ void store8(void* base, int64_t at, bool f32, int valid, const float (&f)[8]) {
    if (f32) {
        float* p = static_cast<float*>(base) + at;
        const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
        store_chunk<float>(p, pack_chunk<float>(lo), valid);
        store_chunk<float>(p + 4, pack_chunk<float>(hi), valid - 4);
    } else {
        store_chunk<T>(static_cast<T*>(base) + at, pack_chunk<T>(f), valid);
    }
}

// Eight columns n .. n + 7 of C (for swiglu of the gate's and of the up's) on their way to y, in fp32 up to the last
// rounding: what is added to every row, and a row's part.
template <typename T> struct OutColumns {
    float bias[8], bias_up[8];
    int n, valid;
    bool pair;
    __device__ __forceinline__ void load(const Product& g, int n_) {
        n = n_;
        valid = g.out_cols - n;
        pair = g.act == MOE_ACT_SWIGLU;
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = bias_up[i] = 0.0f;
        if (g.bias) {
            load8<T>(g.bias, n, g.bias_f32, valid, bias);
            if (pair) load8<T>(g.bias, g.out_cols + n, g.bias_f32, valid, bias_up);
        }
    }
    // Each element of the residual is read before its place in y is written, by the same thread, so y may be the residual.
    __device__ __forceinline__ void residual(const Product& g, int64_t m, float (&r)[8]) const {
        if (g.residual) load8<T>(g.residual, m * g.ldr + n, g.y_f32, valid, r);
    }
    __device__ __forceinline__ void store(const Product& g, int64_t m, float (&v)[8], float (&up)[8], const float (&r)[8]) const {
        if (g.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += bias[i], up[i] += bias_up[i];
        }
        if (g.z) {
            store8<T>(g.z, m * g.ldz + n, false, valid, v);
            if (pair) store8<T>(g.z, m * g.ldz + g.out_cols + n, false, valid, up);
        }
        if (pair) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid_f32(v[i]) * up[i];
        } else if (g.act != MOE_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = act_f32(g.act, v[i]);
        }
        if (g.residual) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        store8<T>(g.y, m * g.ldy + n, g.y_f32, valid, v);
    }
};
template <typename T> __device__ __forceinline__ void linear_out(const Product& g, int64_t m, int n, float (&v)[8], float (&up)[8]) {
    OutColumns<T> out;
    float r[8] = {};
    out.load(g, n);
    out.residual(g, m, r);
    out.store(g, m, v, up, r);
}

}  // namespace moe
