// The expert layer on packed bf16 weights for the few tokens of a decode step: L1 with SwiGLU, L2 with the routing
// weight, combine.
//
// Bound by the weights, which are streamed once per 32 pairs of an expert.  A packed 1 KB block (32 columns x 16 k) is
// one MFMA operand, so a wave reads it with one 16-byte load per lane, contiguous, and multiplies it with up to 32
// token rows as the other operand, which come from the caches.  The waves of a workgroup split K; their sums are added
// through LDS in wave order: no atomics, the same bits on every run.  64 tokens on 32 of 256 experts, 7168 / 2048: L1 266 us, L2 138 (6.1 TB/s);
// one token on 6 experts, 2048 / 1408: 14.8 and 7.8 us (4.5 TB/s), of which the launches' ramps are some 5.  An
// expert of n pairs has its weights streamed ceil(n / 32) times, one pass after the other: 8 experts of 7168 / 2048 at 32, 64 and 128 pairs
// each 154, 274 and 502 us (moe_forward 200, 220, 248).
#include <type_traits>

#include "moe_stream.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFewDepth = 64;   // k per wave and step: four blocks of each column group
constexpr int kFewAhead = 2;    // steps in flight per wave

__device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// What a wave multiplies: NB column groups (a buffer each, K * 64 bytes) by 32 rows of x (this lane's offset in row
// lane % 32; kNoRow: no row).
template <int NB> struct FewOperands {
    rsrc_t w[NB], x;
    uint32_t row;
    int K;
};

// The sums over this wave's steps slice, slice + KS, ...
template <int NB, int KS> __device__ __forceinline__ void few_sums(const FewOperands<NB>& o, int slice, f32x16_t (&acc)[NB]) {
    const int steps = o.K / kFewDepth, lane = threadIdx.x & 63;
    u32x4_t w[kFewAhead][NB][4], x[kFewAhead][4];
    auto fetch = [&](int c, u32x4_t (&wt)[NB][4], u32x4_t (&xt)[4]) {   // past K: zeros
        const uint32_t at = (c < steps ? static_cast<uint32_t>(c) * 4096 : kNoRow) + 16 * lane, k = c < steps ? static_cast<uint32_t>(c) * (2 * kFewDepth) : kNoK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int n = 0; n < NB; ++n) wt[n][i] = load16(o.w[n], at + 1024 * i);
            xt[i] = load16(o.x, o.row + k + 32 * i);
        }
    };
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) fetch(slice + u * KS, w[u], x[u]);
    for (int c0 = slice; c0 < steps; c0 += kFewAhead * KS) {
#pragma unroll
        for (int u = 0; u < kFewAhead; ++u) {
            const int c = c0 + u * KS;
            if (c >= steps) break;   // the same for the whole wave
            u32x4_t wc[NB][4], xc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int n = 0; n < NB; ++n) wc[n][i] = w[u][n][i];
                xc[i] = x[u][i];
            }
            fetch(c + kFewAhead * KS, w[u], x[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n) acc[n] = mfma(xc[i], wc[n][i], acc[n]);
        }
    }
}

template <int NB, int KS> constexpr int few_lds() { return KS * NB * 4096; }   // the waves' sums

// Grid y: with at most EL pairs, one workgroup row per pair, of which the first pair of each expert works and the
// others leave; with more, one per local expert.  Grid x: column groups.  A workgroup lists its expert's pairs in
// ascending order itself (the ids are a few KB).
// L1: the gate and the up group of 32 intermediate columns; act[pair] = silu(gate) up, formed in fp32 and rounded to
// bf16, the matrix instruction's operand type, as in the layer's other forms.  L2: NB groups of output columns; stage[pair] = w o in fp32.
template <bool L1, int NB, int KS> __global__ __launch_bounds__(64 * KS) void few_kernel(FewExperts a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    static_assert(!L1 || NB == 2, "gate and up");
    const int lane = threadIdx.x & 63, slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pairs = a.T * a.k;
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds_raw);
    int* list = reinterpret_cast<int*>(lds_raw + few_lds<NB, KS>());
    const bool by_pair = pairs <= a.EL;
    const int id = by_pair ? __builtin_amdgcn_readfirstlane(a.topk_idx[blockIdx.y]) : a.e_lo + static_cast<int>(blockIdx.y), e = id - a.e_lo;
    if (e < 0 || e >= a.EL) return;
    const int count = expert_pairs(a.topk_idx, pairs, id, by_pair ? static_cast<int>(blockIdx.y) : -1, list);
    if (count == 0) return;

    const int K = L1 ? a.H : a.I, columns = L1 ? 2 * a.I : a.H, group0 = blockIdx.x * NB;
    FewOperands<NB> o;
    o.K = K;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int64_t group = static_cast<int64_t>(e) * (columns / 32) + group0 + n;
        o.w[n] = buffer_of((L1 ? a.w1 : a.w2) + group * 32 * K, 64 * K);
    }
    o.x = buffer_of(L1 ? a.x : a.act, static_cast<int64_t>(L1 ? a.T : pairs) * (2 * K));
    for (int m0 = 0; m0 < count; m0 += 32) {
        const int mine = m0 + (lane & 31);
        o.row = (mine < count ? static_cast<uint32_t>(L1 ? list[mine] / a.k : list[mine]) * (2 * K) : kNoRow) + 16 * (lane >> 5);
        f32x16_t acc[NB] = {};
        few_sums<NB, KS>(o, slice, acc);
        const int quads = (min(32, count - m0) + 7) / 8;   // of 8 rows: registers 4 q .. + 3
        lds_barrier();   // the last rows' sums have been read
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < quads) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const f32x16_t& v = acc[n];
                    sums[((slice * 4 + q) * NB + n) * 64 + lane] = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
            }
        lds_barrier();
        for (int at = threadIdx.x; at < quads * 64; at += 64 * KS) {
            const int q = at >> 6, l = at & 63;
            f32x4_t v[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                v[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KS; ++s) v[n] += sums[((s * 4 + q) * NB + n) * 64 + l];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + 8 * q + 4 * (l >> 5) + i;
                if (m >= count) break;
                const int pair = list[m];
                if constexpr (L1) {
                    a.act[static_cast<int64_t>(pair) * a.I + group0 * 16 + (l & 31)] = f32_to_bf16(silu_f32(v[0][i]) * v[1][i]);
                } else {
                    const float w = a.topk_w[pair];
#pragma unroll
                    for (int n = 0; n < NB; ++n) a.stage[static_cast<int64_t>(pair) * a.H + (group0 + n) * 32 + (l & 31)] = w * v[n][i];
                }
            }
        }
    }
}

// y[t] = the sum of the token's local pairs' rows, in slot order (0 with none).
__global__ __launch_bounds__(256) void few_finish_kernel(FewExperts a) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (c >= a.H) return;
    f32x4_t s = {0, 0, 0, 0};
    for (int j = 0; j < a.k; ++j) {
        const int64_t pair = static_cast<int64_t>(t) * a.k + j;
        const int id = a.topk_idx[pair];
        if (id >= a.e_lo && id < a.e_lo + a.EL) s += *reinterpret_cast<const f32x4_t*>(a.stage + pair * a.H + c);
    }
    bf16_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f32<bf16_t>(s[i]);
    *reinterpret_cast<uint2*>(a.y + static_cast<int64_t>(t) * a.H + c) = __builtin_bit_cast(uint2, o);
}

template <bool L1, int NB, int KS> hipError_t run_few(const FewExperts& a, hipStream_t s) {
    static_assert(few_lds<NB, KS>() + 4 * kFewMaxPairs <= 65536, "dynamic LDS within the default limit");
    const int pairs = a.T * a.k, groups = (L1 ? 2 * a.I : a.H) / 32;   // H and I are multiples of 128, so NB divides them
    few_kernel<L1, NB, KS><<<dim3(groups / NB, pairs < a.EL ? pairs : a.EL), 64 * KS, few_lds<NB, KS>() + 4 * pairs, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewExperts& a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    // Waves a workgroup: four, or two for a short reduction, of which a wave of four has only a few steps, in L1 while its grid is
    // resident at once.  Whole layer in us, four against two waves: 1 token of 6 experts, 2048 / 1408, 29.5 and 26.7; 128 tokens of 4 of 32, 2048 / 768,
    // 67 and 62; but 16 tokens of 6 of 64, 2048 / 1408, L1 152 and 157; 1 token of one expert, 7168 / 2048, L1 27.8 and 34; I of 8192, L2 29 and 35.
    constexpr int kShort = 2048, kResident = 1024;
    const int64_t rows = static_cast<int64_t>(a.T) * a.k < a.EL ? a.T * a.k : a.EL;
    hipError_t e = a.H <= kShort && rows * (a.I / 32) <= kResident ? run_few<true, 2, 2>(a, s) : run_few<true, 2, 4>(a, s);
    if (e == hipSuccess) e = a.I <= kShort ? run_few<false, 1, 2>(a, s) : run_few<false, 1, 4>(a, s);
    if (e != hipSuccess) return e;
    few_finish_kernel<<<dim3((a.H / 4 + 255) / 256, a.T), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
