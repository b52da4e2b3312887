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

size_t block_norm_bwd_bytes(int64_t rows, int cols, int64_t gate_rows);
hipError_t launch_block_norm_fwd(const BlockNorm& a, int dtype, int sdtype, int wdtype, hipStream_t s);
hipError_t launch_block_norm_bwd(const BlockNorm& a, int dtype, int wdtype, hipStream_t s);

}  // namespace moe
