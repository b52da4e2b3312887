// Block norm, the seam between two blocks: what the forward (moe_block_norm.hip) and the backward
// (moe_block_norm_bwd.hip) share.  Per row of C columns, with N(v) = (v - mean) rstd (mean 0 for rms):
//
//   forward   p = N(b) w1 + c1 (post norm; else p = b);  r = x_scale x + scale gate p;  n = N(r) w2 + c2 (pre norm)
//   backward  t = dr + N'(dn w2);  dx = x_scale t;  dp = scale gate t;  dgate = sum scale t p;  db = N'(dp w1) (else dp)
//             dw2 = sum dn N(r), dc2 = sum dn, dw1 = sum dp N(b), dc1 = sum dp over the rows
//             with N'(g) = rstd (g - [layer] sum g / C - N sum (g N) / C)
#pragma once

#include "moe_norm.h"

namespace moe {

// Makes the compiler take v for a new value: what was unpacked from it is unpacked again instead of being held in
// registers from one use to the next (without this the widest teams spill).
__device__ __forceinline__ void renew(u32x4_t& v) { asm("" : "+v"(v)); }

// N elements of type X (N that of a 16-byte chunk of another type) in 16-byte pieces.
template <typename X, int N> struct Pieces {
    static constexpr int P = N / Chunk<X>::N;
    u32x4_t raw[P];
    __device__ __forceinline__ void load(const X* p, int valid) {
#pragma unroll
        for (int h = 0; h < P; ++h) raw[h] = load_chunk<X>(p + h * Chunk<X>::N, valid - h * Chunk<X>::N);
    }
    // element c of a row: a base that is the same for a workgroup of one team and a 32-bit offset, for which the hardware has an
    // address form (64-bit addresses of every chunk and tensor cost some 12 registers a chunk)
    template <typename U, typename Row> static __device__ __forceinline__ std::conditional_t<std::is_const<Row>::value, const U, U>* at(Row* row, int c) {
        using byte = std::conditional_t<std::is_const<Row>::value, const char, char>;
        return reinterpret_cast<std::conditional_t<std::is_const<Row>::value, const U, U>*>(reinterpret_cast<byte*>(row) + static_cast<uint32_t>(c) * static_cast<uint32_t>(sizeof(X)));
    }
    // the same in two steps for rows of at least N elements: one load per piece whatever the row's end, put right later
    __device__ __forceinline__ void load_ahead(const X* row, int c, int cols) {
#pragma unroll
        for (int h = 0; h < P; ++h) raw[h] = *at<u32x4_any_t>(row, min(c + h * Chunk<X>::N, cols - Chunk<X>::N));
    }
    __device__ __forceinline__ void settle(int c, int cols) {
#pragma unroll
        for (int h = 0; h < P; ++h) raw[h] = moe::settle<X, false>(raw[h], c + h * Chunk<X>::N, cols);
    }
    __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            float part[Chunk<X>::N];
            unpack_chunk<X>(raw[h], part);
#pragma unroll
            for (int i = 0; i < Chunk<X>::N; ++i) f[h * Chunk<X>::N + i] = part[i];
        }
    }
    static __device__ __forceinline__ void put(X* p, const float (&f)[N], int valid) {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            float part[Chunk<X>::N];
#pragma unroll
            for (int i = 0; i < Chunk<X>::N; ++i) part[i] = f[h * Chunk<X>::N + i];
            store_chunk<X>(p + h * Chunk<X>::N, pack_chunk<X>(part), valid - h * Chunk<X>::N);
        }
    }
};

struct BlockNorm {
    int64_t rows, gate_share;   // gate_share: rows per row of the gate
    int32_t cols;
    bool layer, post, pre;
    bool b_f32, s_f32, w_f32;   // types: of b, n and their gradients; of the stream (x, r, dr, dx); of the vectors
    float eps, x_scale, scale;
    const void *x, *b, *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
    int64_t ldx, ldb, ldr, ldn;
    void *r, *n;
    float *post_mean, *post_rstd, *pre_mean, *pre_rstd;
    // backward (r is read)
    const void *dr, *dn;
    int64_t lddr, lddn, lddx, lddb;
    void *dx, *db, *dgate, *dpost_weight, *dpost_bias, *dpre_weight, *dpre_bias;
    float* ws;
};

// How the rows are cut into runs of a workgroup.  Runs stay inside one row of the gate, or hold whole ones, so that
// the gate's sums are over rows of one run (per_gate = 1: complete), or over per_gate runs.
struct Runs {
    int64_t runs, length, per_gate;   // length: rows of a run, the last of a gate's may be shorter
    int64_t share;                    // rows per row of the gate
    __host__ __device__ void range(int64_t run, int64_t rows, int64_t& r0, int64_t& r1) const {
        const int64_t first = run / per_gate * (per_gate > 1 ? share : length), end = per_gate > 1 ? first + share : rows;
        r0 = first + run % per_gate * length;
        r1 = r0 + length < end ? r0 + length : end;
    }
};
// About `target` runs of at least `least` rows each.
Runs runs_of(int64_t rows, int64_t gate_rows, int64_t target, int64_t least);

// Partial sums, a row of columns per run each; the gate's [gate rows, per_gate, cols], or, where per_gate is 1, final.
struct Partials {
    float *gate, *post_weight, *post_bias, *pre_weight, *pre_bias;
};

// The backward of rows that fit a team's registers, in one launch (moe_block_norm_row.h).  block_norm_row_runs: its runs,
// 0 runs where it does not take such rows.
Runs block_norm_row_runs(int64_t rows, int cols, int64_t gate_rows, int elem_bytes);
hipError_t launch_block_norm_row_bf16(const BlockNorm& a, const Runs& runs, const Partials& part, hipStream_t s);
hipError_t launch_block_norm_row_fp16(const BlockNorm& a, const Runs& runs, const Partials& part, hipStream_t s);
hipError_t launch_block_norm_row_fp32(const BlockNorm& a, const Runs& runs, const Partials& part, hipStream_t s);

size_t block_norm_bwd_bytes(int64_t rows, int cols, int64_t gate_rows, int elem_bytes);
hipError_t launch_block_norm_fwd(const BlockNorm& a, int dtype, int sdtype, int wdtype, hipStream_t s);
hipError_t launch_block_norm_bwd(const BlockNorm& a, int dtype, int wdtype, hipStream_t s);

}  // namespace moe
