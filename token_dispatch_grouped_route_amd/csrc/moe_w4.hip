// Products with 4-bit weights and group scales, for the few rows of a decode step: a plain linear
// map, and the expert layer (L1 with SwiGLU, L2 with the routing weight, combine).
//
//   w[n][k] = (q[n][k] - z[n][g]) s[n][g],  g = k / group,  q and z in 0 .. 15 (z = 8 when not stored)
//   y[m][n] = sum over g of s[n][g] (sum over k in g of (16 + q) x[m][k]  -  (16 + z[n][g]) Sx[m][g])
//
// The weights are streamed once and bound the call, so the work per weight is kept small: a code
// becomes the 16-bit float 16 + q (exact in bf16 and fp16: the nibble is the top of the mantissa of
// 16.0) with one shift and one and-or per two codes, and goes through v_mfma_f32_16x16x32 with the
// rows x as the A operand; Sx comes from the same instruction with a B operand of ones.  The scale
// enters in fp32 after each group, so no product is rounded before it.
//
// A wave reads 16 weight rows x 128 k at a time, 16 bytes (32 codes of one row) per lane: 64
// contiguous bytes per row and instruction.  Two half-wave swaps and two 16-lane swaps transpose the
// 4 x 4 dwords of the four lane groups, so MFMA i of the chunk takes k = 32 i .. 32 i + 31 (any group
// size that is a multiple of 32 then ends between two MFMAs).  The waves of a workgroup split K and
// their sums are added through LDS in wave order: no atomics, the same bits on every run.
#include <type_traits>

#include "moe_vec.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 b16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h16x8_t __attribute__((ext_vector_type(8)));

template <typename T> struct W4Type;
template <> struct W4Type<bf16_t> {   // 16.0 = 0x4180, 7 mantissa bits: the nibble at bits 3 .. 6
    static constexpr uint32_t kBase = 0x41804180u, kMask = 0x00780078u, kOnes = 0x3f803f80u;
    static constexpr int kBit = 3;
    __device__ static f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8_t, a), __builtin_bit_cast(b16x8_t, b), c, 0, 0, 0);
    }
};
template <> struct W4Type<fp16_t> {   // 16.0 = 0x4c00, 10 mantissa bits: the nibble at bits 6 .. 9
    static constexpr uint32_t kBase = 0x4c004c00u, kMask = 0x03c003c0u, kOnes = 0x3c003c00u;
    static constexpr int kBit = 6;
    __device__ static f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8_t, a), __builtin_bit_cast(h16x8_t, b), c, 0, 0, 0);
    }
};

// Eight codes (one dword, low nibble first) as 16 + q, in the order 0 4 1 5 2 6 3 7.
template <typename T> __device__ __forceinline__ u32x4_t expand8(uint32_t w) {
    using W = W4Type<T>;
    u32x4_t r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int up = W::kBit - 4 * p;   // nibble p (and p + 4, 16 bits higher) to bit kBit
        r[p] = ((up >= 0 ? w << up : w >> -up) & W::kMask) | W::kBase;
    }
    return r;
}
// Eight consecutive 16-bit values in that order.
__device__ __forceinline__ u32x4_t order8(u32x4_t v) {
    u32x4_t r;
    r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
    return r;
}
// d[i] of lane group c -> d[c] of lane group i (lane groups of 16).
__device__ __forceinline__ void transpose_groups(u32x4_t& d) {
    auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = lo[0];
    d[1] = lo[1];
    d[2] = hi[0];
    d[3] = hi[1];
}

constexpr int kW4Chunk = 128;   // k per wave and step
constexpr int kW4Ahead = 4;     // chunks of weights in flight per wave

// The sums of this wave's K chunks (wave, wave + WAVES, ...): sum[t][n][i] of x row 16 t + 4 (lane / 16) + i
// and weight row lane % 16 of tile n.  wrow[n]: this lane's weight row (lane % 16) of tile n; xrow[t]: its x
// row (lane % 16) of row tile t, or null; scales, zeros: LDS, this lane's row of tile n at n * 16 * groups.
// FLUSH: MFMAs per scale (min(group, 128) / 32); gshift: log2 of the group.
template <typename T, int MT, int NT, int FLUSH, bool ZEROS, int WAVES>
__device__ __forceinline__ void w4_sums(const uint8_t* const (&wrow)[NT], const T* const (&xrow)[MT], const T* scales,
                                        const uint8_t* zeros, int K, int gshift, f32x4_t (&sum)[MT][NT]) {
    using W = W4Type<T>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = lane >> 4;
    const int groups = K >> gshift, chunks = (K + kW4Chunk - 1) / kW4Chunk;
    const u32x4_t ones = {W::kOnes, W::kOnes, W::kOnes, W::kOnes};
    u32x4_t code[kW4Ahead][NT] = {};   // a lane group past K multiplies zero rows with whatever codes it holds
    auto fetch = [&](int c, u32x4_t (&to)[NT]) {
        const int k = c * kW4Chunk + 32 * part;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (k < K) to[n] = *reinterpret_cast<const u32x4_t*>(wrow[n] + (k >> 1));
    };
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u) fetch(wave + u * WAVES, code[u]);

    for (int c0 = wave; c0 < chunks; c0 += kW4Ahead * WAVES) {
#pragma unroll
        for (int u = 0; u < kW4Ahead; ++u) {
            const int c = c0 + u * WAVES, k0 = c * kW4Chunk;
            if (c < chunks) {   // the same for the whole wave
                u32x4_t xa[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        xa[t][i] = u32x4_t{0, 0, 0, 0};
                        if (xrow[t] && k0 + 32 * i < K) xa[t][i] = *reinterpret_cast<const u32x4_t*>(xrow[t] + k0 + 32 * i + 8 * part);
                    }
                u32x4_t q[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) q[n] = code[u][n];
                fetch(c + kW4Ahead * WAVES, code[u]);
#pragma unroll
                for (int n = 0; n < NT; ++n) transpose_groups(q[n]);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) xa[t][i] = order8(xa[t][i]);
#pragma unroll
                for (int f = 0; f < 4 / FLUSH; ++f) {
                    if (k0 + 32 * f * FLUSH >= K) break;
                    f32x4_t sx[MT] = {}, acc[MT][NT] = {};
#pragma unroll
                    for (int h = 0; h < FLUSH; ++h) {   // MFMAs past K multiply zero rows
                        const int i = f * FLUSH + h;
#pragma unroll
                        for (int t = 0; t < MT; ++t) sx[t] = W::mfma(xa[t][i], ones, sx[t]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const u32x4_t b = expand8<T>(q[n][i]);
#pragma unroll
                            for (int t = 0; t < MT; ++t) acc[t][n] = W::mfma(xa[t][i], b, acc[t][n]);
                        }
                    }
                    const int g = (k0 + 32 * f * FLUSH) >> gshift;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float s = to_f32(scales[n * 16 * groups + g]);
                        const float z = 16.0f + (ZEROS ? static_cast<float>(zeros[n * 16 * groups + g]) : 8.0f);
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[t][n][i] += s * (acc[t][n][i] - z * sx[t][i]);
                    }
                }
            }
        }
    }
}

// Copies `count` contiguous elements to LDS; src 16-byte aligned.
template <typename E> __device__ __forceinline__ void stage(E* dst, const E* src, int count) {
    constexpr int N = 16 / static_cast<int>(sizeof(E));
    const int full = count / N;
    for (int i = threadIdx.x; i < full; i += blockDim.x)
        reinterpret_cast<u32x4_t*>(dst)[i] = reinterpret_cast<const u32x4_t*>(src)[i];
    for (int i = full * N + threadIdx.x; i < count; i += blockDim.x) dst[i] = src[i];
}

// LDS of a workgroup: scales and zero points of its NT tiles, and the waves' sums over them.
template <int MT, int NT, int WAVES> size_t w4_lds_bytes(int groups, bool zeros) {
    const size_t meta = static_cast<size_t>(16 * NT) * groups * (zeros ? 3 : 2), sums = static_cast<size_t>(WAVES) * MT * NT * 1024;
    return (meta > sums ? meta : sums) + 16;
}

// Puts the waves' sums into LDS as [wave][t][n][lane][4] and calls f on them.
template <int MT, int NT, int WAVES, typename F>
__device__ __forceinline__ void w4_join(float* lds, const f32x4_t (&sum)[MT][NT], F&& f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();   // the scales are no longer read
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<f32x4_t*>(lds + ((wave * MT + t) * NT + n) * 256 + lane * 4) = sum[t][n];
    __syncthreads();
    f(lds);
}
// Element (row m, column n) of the tile (t, n) in a wave's sums.
__device__ __forceinline__ int w4_at(int m, int n) { return ((m >> 2) * 16 + n) * 4 + (m & 3); }

template <typename T, int MT, int NT, int FLUSH, bool ZEROS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4_linear_kernel(W4Linear a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    const int lane = threadIdx.x & 63, groups = a.K >> a.gshift;
    const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT, rows = min(16 * NT, a.N - n0);
    T* scales = reinterpret_cast<T*>(lds_raw);
    uint8_t* zeros = lds_raw + static_cast<size_t>(16 * NT) * groups * 2;
    stage<uint16_t>(reinterpret_cast<uint16_t*>(scales), static_cast<const uint16_t*>(a.scales) + static_cast<int64_t>(n0) * groups, rows * groups);
    if (ZEROS) stage<uint8_t>(zeros, a.zeros + static_cast<int64_t>(n0) * groups, rows * groups);
    __syncthreads();

    const uint8_t* wrow[NT];
    const T* xrow[MT];
#pragma unroll
    for (int n = 0; n < NT; ++n)   // rows past N repeat the last one and are not stored
        wrow[n] = a.codes + static_cast<int64_t>(min(n0 + 16 * n + (lane & 15), a.N - 1)) * (a.K >> 1);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + (lane & 15);
        xrow[t] = m < a.M ? static_cast<const T*>(a.x) + m * a.ldx : nullptr;
    }
    f32x4_t sum[MT][NT] = {};
    w4_sums<T, MT, NT, FLUSH, ZEROS, WAVES>(wrow, xrow, scales + (lane & 15) * groups, zeros + (lane & 15) * groups, a.K, a.gshift, sum);
    w4_join<MT, NT, WAVES>(reinterpret_cast<float*>(lds_raw), sum, [&](const float* part) {
        for (int v = threadIdx.x; v < MT * NT * 256; v += 64 * WAVES) {
            const int m = v / (16 * NT), n = v % (16 * NT);   // m in the row tiles, n in the columns of this workgroup
            if (m0 + m >= a.M || n0 + n >= a.N) continue;
            const float* p = part + ((m >> 4) * NT + (n >> 4)) * 256 + w4_at(m & 15, n & 15);
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += p[w * MT * NT * 256];
            static_cast<T*>(a.y)[(m0 + m) * a.ldy + n0 + n] = from_f32<T>(s);
        }
    });
}

// ---------------------------------------------------------------------------------------------
// Expert layer.  Grid y: with at most EL pairs, one workgroup row per pair, of which the first pair
// of each expert works and the others leave; with more, one per local expert.  A workgroup lists its
// expert's pairs in ascending order itself (the ids are a few KB), so no table is built beforehand.
// ---------------------------------------------------------------------------------------------
// The local expert of this workgroup row and its pairs (LDS list, count); false: nothing to do.
__device__ __forceinline__ bool w4_pairs(const W4Experts& a, int* list, int* counts, int& expert, int& count) {
    const int pairs = a.T * a.k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int first = 0, id;
    if (pairs <= a.EL) {
        first = blockIdx.y;
        id = a.topk_idx[first];
        if (id < a.e_lo || id >= a.e_lo + a.EL) return false;
    } else {
        id = a.e_lo + blockIdx.y;
    }
    expert = id - a.e_lo;
    count = 0;
    bool earlier = false;
    for (int p0 = 0; p0 < pairs; p0 += blockDim.x) {
        const int p = p0 + threadIdx.x;
        const bool mine = p < pairs && a.topk_idx[p] == id;
        const uint64_t m = __ballot(mine);
        if (lane == 0) counts[wave] = __popcll(m);
        __syncthreads();
        int at = count;
        for (int w = 0; w < waves; ++w) {
            if (w == wave && mine) list[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = p;
            at += counts[w];
        }
        __syncthreads();
        count = at;
    }
    if (pairs <= a.EL && count > 0) earlier = list[0] < first;
    return count > 0 && !earlier;
}

// L1: NT = 2, tile 0 the gate columns 16 b .. and tile 1 the up columns of the same 16 intermediate
// columns; act[pair] = silu(gate) up in T.  L2: NT tiles of output columns; stage[pair] = w o in fp32.
template <typename T, bool L1, int NT, int FLUSH, bool ZEROS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4_experts_kernel(W4Experts a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    __shared__ int counts[WAVES];
    const int lane = threadIdx.x & 63;
    int* list = reinterpret_cast<int*>(lds_raw + a.list_at);
    int e, count;
    if (!w4_pairs(a, list, counts, e, count)) return;

    const int K = L1 ? a.H : a.I, N = L1 ? 2 * a.I : a.H, groups = K >> a.gshift;
    const int64_t wbase = static_cast<int64_t>(e) * N;   // rows of the expert
    const uint8_t* codes = L1 ? a.w1 : a.w2;
    const uint16_t* scale_g = static_cast<const uint16_t*>(L1 ? a.s1 : a.s2);
    const uint8_t* zero_g = L1 ? a.z1 : a.z2;
    T* scales = reinterpret_cast<T*>(lds_raw);
    uint8_t* zeros = lds_raw + static_cast<size_t>(16 * NT) * groups * 2;
    const uint8_t* wrow[NT];
    for (int m0 = 0; m0 < count; m0 += 16) {
        __syncthreads();   // the sums of the last rows are no longer read
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t row0 = wbase + (L1 ? n * a.I + 16 * blockIdx.x : 16 * (NT * blockIdx.x + n));
            stage<uint16_t>(reinterpret_cast<uint16_t*>(scales) + n * 16 * groups, scale_g + row0 * groups, 16 * groups);
            if (ZEROS) stage<uint8_t>(zeros + n * 16 * groups, zero_g + row0 * groups, 16 * groups);
            wrow[n] = codes + (row0 + (lane & 15)) * (K >> 1);
        }
        __syncthreads();
        const int m = m0 + (lane & 15);
        const T* xrow[1] = {nullptr};
        if (m < count) {
            const int pair = list[m];
            xrow[0] = L1 ? static_cast<const T*>(a.x) + static_cast<int64_t>(pair / a.k) * K : static_cast<const T*>(a.act) + static_cast<int64_t>(pair) * K;
        }
        f32x4_t sum[1][NT] = {};
        w4_sums<T, 1, NT, FLUSH, ZEROS, WAVES>(wrow, xrow, scales + (lane & 15) * groups, zeros + (lane & 15) * groups, K, a.gshift, sum);
        w4_join<1, NT, WAVES>(reinterpret_cast<float*>(lds_raw), sum, [&](const float* part) {
            constexpr int OUT = L1 ? 16 : 16 * NT;   // output columns of the workgroup
            for (int v = threadIdx.x; v < 16 * OUT; v += 64 * WAVES) {
                const int r = v / OUT, n = v % OUT;
                if (m0 + r >= count) continue;
                const int pair = list[m0 + r];
                const float* p = part + (L1 ? 0 : (n >> 4) * 256) + w4_at(r, n & 15);
                float s = 0.0f, u = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    s += p[w * NT * 256];
                    if (L1) u += p[w * NT * 256 + 256];
                }
                if (L1) static_cast<T*>(a.act)[static_cast<int64_t>(pair) * a.I + 16 * blockIdx.x + n] = from_f32<T>(silu_f32(s) * u);
                else a.stage[static_cast<int64_t>(pair) * a.H + 16 * NT * blockIdx.x + n] = a.topk_w[pair] * s;
            }
        });
    }
}

// y[t] = the sum of the token's local pairs' rows, in slot order (0 with none).
template <typename T>
__global__ __launch_bounds__(256) void w4_finish_kernel(W4Experts a) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (c >= a.H) return;
    f32x4_t s = {0, 0, 0, 0};
    for (int j = 0; j < a.k; ++j) {
        const int64_t pair = static_cast<int64_t>(t) * a.k + j;
        const int id = a.topk_idx[pair];
        if (id >= a.e_lo && id < a.e_lo + a.EL) s += *reinterpret_cast<const f32x4_t*>(a.stage + pair * a.H + c);
    }
    T o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(s[i]);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.y) + static_cast<int64_t>(t) * a.H + c) = __builtin_bit_cast(uint2, o);
}

// ---------------------------------------------------------------------------------------------
// Quantisation of [E, K, N] weights (x @ W layout), one thread per (column, group): the scale is
// rounded to its type first, then the codes are the nearest to w / s.
// ---------------------------------------------------------------------------------------------
template <typename T, typename S, bool ZEROS>
__global__ __launch_bounds__(64) void w4_quantize_kernel(const T* __restrict__ w, int K, int N, int group, uint8_t* __restrict__ codes,
                                                         S* __restrict__ scales, uint8_t* __restrict__ zeros) {
    const int n = blockIdx.x * 64 + threadIdx.x, g = blockIdx.y;
    if (n >= N) return;
    const int64_t e = blockIdx.z, groups = K / group, row = e * N + n;
    const T* src = w + (e * K + static_cast<int64_t>(g) * group) * N + n;
    float lo = 0.0f, hi = 0.0f;
    for (int i = 0; i < group; ++i) {
        const float v = to_f32(src[static_cast<int64_t>(i) * N]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    const S st = from_f32<S>(ZEROS ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    const float s = to_f32(st);
    const float z = ZEROS ? (s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f) : 8.0f;
    scales[row * groups + g] = st;
    if (ZEROS) zeros[row * groups + g] = static_cast<uint8_t>(z);
    uint8_t* out = codes + row * (K / 2) + static_cast<int64_t>(g) * (group / 2);
    for (int i = 0; i < group; i += 8) {
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = to_f32(src[static_cast<int64_t>(i + j) * N]);
            const float q = s > 0.0f ? fminf(fmaxf(rintf(v / s) + z, 0.0f), 15.0f) : z;
            word |= static_cast<uint32_t>(q) << (4 * j);
        }
        *reinterpret_cast<uint32_t*>(out + i / 2) = word;
    }
}

namespace {

template <typename F> void with_group(int group, bool zeros, F&& f) {
    auto z = [&](auto flush) {
        if (zeros) f(flush, std::true_type{});
        else f(flush, std::false_type{});
    };
    if (group == 32) z(std::integral_constant<int, 1>{});
    else if (group == 64) z(std::integral_constant<int, 2>{});
    else z(std::integral_constant<int, 4>{});
}

constexpr int kW4Waves = 8;

template <typename T, int MT, int NT> hipError_t run_linear(const W4Linear& a, hipStream_t s) {
    hipError_t err = hipSuccess;
    with_group(1 << a.gshift, a.zeros != nullptr, [&](auto flush, auto zeros) {
        const size_t lds = w4_lds_bytes<MT, NT, kW4Waves>(a.K >> a.gshift, zeros());
        auto* kernel = &w4_linear_kernel<T, MT, NT, flush(), zeros(), kW4Waves>;
        if (lds > 65536) err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (err != hipSuccess) return;
        const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
        kernel<<<grid, 64 * kW4Waves, lds, s>>>(a);
    });
    return err == hipSuccess ? hipGetLastError() : err;
}

template <typename T, bool L1, int NT> hipError_t run_experts(W4Experts a, hipStream_t s) {
    hipError_t err = hipSuccess;
    const int K = L1 ? a.H : a.I, columns = L1 ? a.I : a.H;
    const int64_t pairs = static_cast<int64_t>(a.T) * a.k;
    with_group(1 << a.gshift, (L1 ? a.z1 : a.z2) != nullptr, [&](auto flush, auto zeros) {
        const size_t tiles = (w4_lds_bytes<1, NT, kW4Waves>(K >> a.gshift, zeros()) + 15) / 16 * 16, lds = tiles + 4 * static_cast<size_t>(pairs);
        a.list_at = static_cast<int>(tiles);
        auto* kernel = &w4_experts_kernel<T, L1, NT, flush(), zeros(), kW4Waves>;
        if (lds > 65536) err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (err != hipSuccess) return;
        const dim3 grid(columns / (L1 ? 16 : 16 * NT), static_cast<unsigned>(pairs < a.EL ? pairs : a.EL));
        kernel<<<grid, 64 * kW4Waves, lds, s>>>(a);
    });
    return err == hipSuccess ? hipGetLastError() : err;
}

template <typename T> hipError_t run_forward(const W4Experts& a, hipStream_t s) {
    hipError_t e = run_experts<T, true, 2>(a, s);
    if (e == hipSuccess) e = run_experts<T, false, 1>(a, s);
    if (e != hipSuccess) return e;
    w4_finish_kernel<T><<<dim3((a.H / 4 + 255) / 256, a.T), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_linear(const W4Linear& a, int dtype, hipStream_t s) {
    if (a.M <= 0) return hipSuccess;
    if (dtype == MOE_BF16) return a.M <= 16 ? run_linear<bf16_t, 1, 1>(a, s) : a.M <= 32 ? run_linear<bf16_t, 2, 1>(a, s) : run_linear<bf16_t, 4, 1>(a, s);
    return a.M <= 16 ? run_linear<fp16_t, 1, 1>(a, s) : a.M <= 32 ? run_linear<fp16_t, 2, 1>(a, s) : run_linear<fp16_t, 4, 1>(a, s);
}

hipError_t launch_w4_forward(const W4Experts& a, int dtype, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    return dtype == MOE_BF16 ? run_forward<bf16_t>(a, s) : run_forward<fp16_t>(a, s);
}

hipError_t launch_w4_quantize(int wdtype, int dtype, int E, int K, int N, int group, const void* w, uint8_t* codes, void* scales,
                              uint8_t* zeros, hipStream_t s) {
    const dim3 grid((N + 63) / 64, K / group, E);
    auto go = [&](auto t, auto st) {
        using T = decltype(t);
        using S = decltype(st);
        if (zeros) w4_quantize_kernel<T, S, true><<<grid, 64, 0, s>>>(static_cast<const T*>(w), K, N, group, codes, static_cast<S*>(scales), zeros);
        else w4_quantize_kernel<T, S, false><<<grid, 64, 0, s>>>(static_cast<const T*>(w), K, N, group, codes, static_cast<S*>(scales), nullptr);
    };
    auto types = [&](auto t) {
        if (dtype == MOE_BF16) go(t, bf16_t{});
        else go(t, fp16_t{});
    };
    if (wdtype == MOE_BF16) types(bf16_t{});
    else if (wdtype == MOE_FP16) types(fp16_t{});
    else types(float{});
    return hipGetLastError();
}

}  // namespace moe
