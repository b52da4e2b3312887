// Row norm: what the forward (moe_norm.hip) and the backward (moe_norm_bwd.hip) share.
//
//   forward   mean = sum x / C (layer norm; 0 for RMS), s = 1 / sqrt(sum (x - mean)^2 / C + eps),
//             xh = (x - mean) s,  y = xh w + b
//   backward  g = dy w;  dx = s (g - [layer] sum g / C - xh sum (g xh) / C);
//             dw = sum over rows of dy xh;  db = sum over rows of dy
//
// Both are bound by memory: each element is read once and written once, every statistic is formed
// from registers.  A row is held by a team of TPR threads (a part of a wave for the shortest rows, a
// workgroup for long ones), NV 16-byte chunks each.  A team walks rows at a fixed stride with the next
// row's loads in flight while this row is reduced, and keeps the weights in registers from row to row.
#pragma once

#include <type_traits>

#include "moe_vec.h"

namespace moe {

constexpr int norm_block(int tpr) { return tpr < 256 ? 256 : tpr; }   // threads of a workgroup

constexpr int norm_waves(int tpr) { return norm_block(tpr) / 64; }

// The sums over a row's TPR threads of NS values, in every thread.  lds: 2 * NS * norm_waves(TPR) floats.  `slot` alternates between two
// LDS buffers from one call to the next, so one barrier per call is enough.
template <int TPR, int NS> __device__ __forceinline__ void team_sum(float (&v)[NS], float* lds, int slot) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if constexpr (TPR >= 64) {
            v[i] = wave_sum(v[i]);
        } else {   // 8, 16 or 32 lanes
            v[i] += dpp<kDppXor1>(v[i]);
            v[i] += dpp<kDppXor2>(v[i]);
            v[i] += dpp<kDppHalfMirror>(v[i]);
            if constexpr (TPR > 8) v[i] += dpp<kDppMirror>(v[i]);
            if constexpr (TPR > 16) {
                const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i]), false, false);
                v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            }
        }
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64, TEAMS = norm_block(TPR) / TPR;
        float* buf = lds + (slot * TEAMS + threadIdx.x / TPR) * W * NS;
        const int wave = threadIdx.x % TPR >> 6;
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

// Weights of NV chunks of N elements in their own type; `none` stands in where there are none.
template <typename WT, int N, int NV, int TPR> struct NormWeights {
    static constexpr int P = N / Chunk<WT>::N;   // 16-byte pieces per chunk
    u32x4_t raw[NV][P];
    __device__ __forceinline__ void load(const void* w, int tid, int cols, float none) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int h = 0; h < P; ++h) {
                const int c = (j * TPR + tid) * N + h * Chunk<WT>::N;
                if (w) {
                    raw[j][h] = load_chunk<WT>(static_cast<const WT*>(w) + c, cols - c);
                } else {
                    float f[Chunk<WT>::N];
#pragma unroll
                    for (int i = 0; i < Chunk<WT>::N; ++i) f[i] = none;
                    raw[j][h] = pack_chunk<WT>(f);
                }
            }
    }
    __device__ __forceinline__ void get(int j, float (&f)[N]) const {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            float part[Chunk<WT>::N];
            unpack_chunk<WT>(raw[j][h], part);
#pragma unroll
            for (int i = 0; i < Chunk<WT>::N; ++i) f[h * Chunk<WT>::N + i] = part[i];
        }
    }
};

// Threads per row and chunks per thread: the smallest team of a power of two (8 to 1024) whose threads take
// at most `most` chunks each; rows beyond 1024 x most, up to 32768 elements, take more.
struct Geometry { int tpr, nv; };
constexpr Geometry norm_geometry(int64_t chunks, int most) {
    for (int tpr = 8; tpr <= 1024; tpr *= 2)
        if (chunks <= static_cast<int64_t>(tpr) * most) return {tpr, static_cast<int>((chunks + tpr - 1) / tpr)};
    const int nv = static_cast<int>((chunks + 1023) / 1024);
    return {1024, nv <= 4 ? nv : 8};
}
constexpr int64_t norm_chunks(int cols, int elem_bytes) { return (static_cast<int64_t>(cols) * elem_bytes + 15) / 16; }

template <int TPR, int NV> struct Geo {
    static constexpr int tpr = TPR, nv = NV;
};
template <int TPR, int NV, typename F> constexpr bool is_geometry(const Geometry& g, F&& f) {
    if (g.tpr != TPR || g.nv != NV) return false;
    f(Geo<TPR, NV>{});
    return true;
}
// A team of TPR threads has over MOST / 2 chunks a thread, the smallest any number.
template <int TPR, int MOST, typename F> constexpr bool is_team(const Geometry& g, F&& f) {
    if constexpr (MOST == 2) return is_geometry<TPR, 2>(g, f);
    else return is_geometry<TPR, 3>(g, f) || is_geometry<TPR, 4>(g, f);
}
// Calls f with the compiled geometry; false if there is none.  LONG512: rows beyond 512 x MOST chunks stay with
// 512 threads up to twice that (the layer norm's backward).
template <int MOST, int BYTES, bool LONG512, typename F> constexpr bool with_geometry(const Geometry& g, F&& f) {
    if (is_geometry<8, 1>(g, f) || (MOST > 2 && is_geometry<8, 2>(g, f)) || is_team<8, MOST>(g, f) || is_team<16, MOST>(g, f) || is_team<32, MOST>(g, f) ||
        is_team<64, MOST>(g, f) || is_team<128, MOST>(g, f) || is_team<256, MOST>(g, f) || is_team<512, MOST>(g, f))
        return true;
    if constexpr (!LONG512) {
        if (is_team<1024, MOST>(g, f)) return true;
    } else if constexpr (MOST == 2) {
        if (is_geometry<512, 3>(g, f) || is_geometry<512, 4>(g, f)) return true;
    } else {
        if (is_geometry<512, 6>(g, f) || is_geometry<512, 8>(g, f)) return true;
    }
    if constexpr (MOST == 2) {
        if (is_geometry<1024, 3>(g, f) || is_geometry<1024, 4>(g, f)) return true;
    }
    if constexpr (BYTES == 4) return is_geometry<1024, 8>(g, f);
    return false;
}
// Whether `pick` (chunks of a row to its geometry) finds a compiled one for every width of BYTES-byte elements.
// A geometry holds for runs of 8 and more chunks that begin after a multiple of 8, so one of each is tried.
template <int MOST, int BYTES, bool LONG512, typename P> constexpr bool every_width(P pick) {
    for (int64_t c = 1; c <= norm_chunks(kNormMaxCols, BYTES); c += 8)
        if (!with_geometry<MOST, BYTES, LONG512>(pick(c), [](auto) {})) return false;
    return true;
}

template <typename F> void with_types(int dtype, int wdtype, F&& f) {
    if (dtype == MOE_FP32) f(float{}, float{});
    else if (dtype == MOE_BF16 && wdtype == MOE_BF16) f(bf16_t{}, bf16_t{});
    else if (dtype == MOE_BF16) f(bf16_t{}, float{});
    else if (wdtype == MOE_FP16) f(fp16_t{}, fp16_t{});
    else f(fp16_t{}, float{});
}

}  // namespace moe
