// The linear map for up to 32 rows (a decode batch).  Bound by the weight, which is read once, or, where columns are few,
// by what one compute unit takes in (about 31 GB/s from memory): then the reduction is split over workgroups too and joined by a second launch.
//
// A workgroup takes a few columns and its waves split the reduction.  A wave streams its own slices of the weight through its own two 4 KB LDS slots (no barrier), rows of 128
// bytes as they are in memory: 64 columns x 32 k where columns are contiguous, read transposed (ds_read_b64_tr_b16), or
// 32 columns x 64 k where k is.  They meet x, whose rows come from the caches, in the 16 x 16 x 32 MFMA; the waves' sums are
// added through LDS in wave order.  One row, 7168 x 4096 bf16 by row: 15.3 us (3.8 TB/s), and 3.9 for the join of four splits.
#include <type_traits>

#include "moe_linear_tile.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ f32x4 mfma16(u32x4_t a, u32x4_t b, f32x4 c);
template <> __device__ __forceinline__ f32x4 mfma16<bf16_t>(u32x4_t a, u32x4_t b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mfma16<fp16_t>(u32x4_t a, u32x4_t b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
}

constexpr int kFewSlot = 4096;
typedef __attribute__((address_space(1))) const u32x4_t g_chunk;

// What a wave streams and multiplies.  S: columns of the weight contiguous.  MT: tiles of 16 rows of x.
template <typename T, bool S, int MT> struct FewStream {
    static constexpr int WAVES = 16, SLOTS = 2, COLS = S ? 64 : 32, DEPTH = S ? 32 : 64, BLOCKS = COLS / 16, PARTS = DEPTH / 32;
    static constexpr int LOADS = 4 + MT * PARTS;   // of a step
    const char* src[4];          // this lane's 16 bytes of each instruction at step 0
    int k_of[4];                 // and their k in a step
    const uint16_t* xrow[MT];    // this lane's chunk of its rows of x at k 0
    int64_t step_bytes;
    int K, first, steps, lane;   // steps first .. steps - 1 of the reduction are this workgroup's

    __device__ __forceinline__ void setup(const Product& g, const Side& o, int split, int lane_) {
        lane = lane_;
        K = g.K;
        first = split * g.slots;
        steps = min((K + DEPTH - 1) / DEPTH, first + g.slots);
        step_bytes = S ? 2 * DEPTH * o.ld : 2 * DEPTH;
        // instruction i of a step fills rows 8 i + lane / 8 of a slot; at position lane % 8 lies chunk position ^ swizzle(row).  Past
        // the last column the last one is read again (and not stored).
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 3);
            if constexpr (S) {
                const int c = (lane & 7) ^ ((row >> 1 & 1) << 1) ^ ((row >> 3 & 1) << 2);
                k_of[i] = row;
                src[i] = reinterpret_cast<const char*>(o.p + row * o.ld + min(o.real(8 * c), o.limit(8 * c) - 8));
            } else {
                const int c = (lane & 7) ^ (row >> 1 & 7);
                k_of[i] = 8 * c;
                src[i] = reinterpret_cast<const char*>(o.p + min(o.real(row), o.limit(row) - 1) * o.ld + 8 * c);
            }
        }
        // rows past the last are row M - 1 again (their sums are not stored)
#pragma unroll
        for (int m = 0; m < MT; ++m) xrow[m] = g.a + min(16 * m + (lane & 15), g.M - 1) * g.lda + 8 * (lane >> 4);
    }
    // always LOADS loads, whatever the step: chunks past K are zeros, in the weight and in x
    __device__ __forceinline__ void fetch_weight(int step, char* __restrict__ slot) const {
        const char* zeros = reinterpret_cast<const char*>(kZeroChunk);
        step = min(step, steps - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t p = reinterpret_cast<uint64_t>(step * DEPTH + k_of[i] < K ? src[i] + step * step_bytes : zeros);
            asm("" : "+v"(p));   // a selected address, not two loads under a branch
            __builtin_amdgcn_global_load_lds((g_void*)p, (l_void*)(slot + 1024 * i), 16, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void fetch_x(int step, u32x4_t (&x)[MT][PARTS]) const {
        const char* zeros = reinterpret_cast<const char*>(kZeroChunk);
        step = min(step, steps - 1);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                const int k = step * DEPTH + 32 * h;
                const char* p = k + 8 * (lane >> 4) < K ? reinterpret_cast<const char*>(xrow[m] + k) : zeros;
                x[m][h] = *(g_chunk*)p;   // said to be global memory: the compiler does not see it of a selected address
            }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void fragments(const char* __restrict__ slot, u32x4_t (&w)[BLOCKS][PARTS]) const {
        const int col = lane & 15, group = lane >> 4;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                if constexpr (S) {
                    // a 16-lane group reads 4 rows of 16 columns: lane j 4 columns of row j / 4, and receives column j's four k
                    const int k = 8 * group + (col >> 2), c = 2 * b + ((col & 3) >> 1);
                    const char* p = slot + k * 128 + ((c ^ ((k >> 1 & 1) << 1) ^ ((k >> 3 & 1) << 2)) << 4) + 8 * (col & 1);
                    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s16x4*)p);
                    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s16x4*)(p + 4 * 128));   // k + 4: the same swizzle
                    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    w[b][h] = __builtin_bit_cast(u32x4_t, v);
                } else {
                    const int row = 16 * b + col, c = 4 * h + group;
                    w[b][h] = *reinterpret_cast<const u32x4_t*>(slot + row * 128 + ((c ^ (row >> 1 & 7)) << 4));
                }
            }
    }
    // The sums over the steps first + wave, first + wave + WAVES, ...  The slots are distinct, so that reading one does not wait for the loads into
    // the other.
    __device__ __forceinline__ void run(int wave, char* __restrict__ s0, char* __restrict__ s1, f32x4 (&acc)[MT][BLOCKS]) const {
        char* const slots[SLOTS] = {s0, s1};
        u32x4_t x[SLOTS][MT][PARTS];
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            fetch_weight(first + wave + u * WAVES, slots[u]);
            fetch_x(first + wave + u * WAVES, x[u]);
        }
        for (int j = first + wave; j < steps; j += SLOTS * WAVES) {
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                const int step = j + u * WAVES;
                if (step >= steps) break;   // the same for the whole wave
                wait_counts<LOADS, false>();   // the other slot's loads may be in flight
                __builtin_amdgcn_sched_barrier(0);
                u32x4_t w[BLOCKS][PARTS];
                fragments(slots[u], w);
                wait_counts<63, true>();   // the fragments are in registers: the slot may be filled again
                __builtin_amdgcn_sched_barrier(0);
                fetch_weight(step + SLOTS * WAVES, slots[u]);
#pragma unroll
                for (int h = 0; h < PARTS; ++h)
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                        for (int m = 0; m < MT; ++m) acc[m][b] = mfma16<T>(x[u][m][h], w[b][h], acc[m][b]);
                __builtin_amdgcn_sched_barrier(0);
                fetch_x(step + SLOTS * WAVES, x[u]);
            }
        }
    }
};

template <typename T, bool S, int MT> __global__ __launch_bounds__((64 * FewStream<T, S, MT>::WAVES)) void linear_few_kernel(Product g) {
    extern __shared__ __align__(16) char lds[];   // the waves' slots; then their sums of 16 rows, and those of the workgroup
    using Stream = FewStream<T, S, MT>;
    constexpr int WAVES = Stream::WAVES, COLS = Stream::COLS, BLOCKS = Stream::BLOCKS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool pair = g.act == MOE_ACT_SWIGLU;
    // neighbouring workgroups' columns on one XCD (workgroup b is on XCD b mod 8)
    const int per = (gridDim.x + 7) / 8, block = static_cast<int>((blockIdx.x & 7) * per + (blockIdx.x >> 3)), n0 = block * (pair ? COLS / 2 : COLS);
    if (n0 >= g.out_cols) return;
    Stream stream;
    stream.setup(g, pair ? Side{g.b, g.ldb, n0, g.out_cols, COLS / 2, g.out_cols} : Side{g.b, g.ldb, n0, g.N, 0, 0}, blockIdx.y, lane);
    f32x4 acc[MT][BLOCKS] = {};
    char* slots = lds + wave * (Stream::SLOTS * kFewSlot);
    if (stream.first + wave < stream.steps) stream.run(wave, slots, slots + kFewSlot, acc);
    wait_counts<0, true>();   // nothing is on its way into LDS any more
    __builtin_amdgcn_sched_barrier(0);
    // element (row 4 (l / 16) + r, column l % 16) of block b: sums[(wave * BLOCKS + b) * 256 + 4 l + r]
    float* sums = reinterpret_cast<float*>(lds);
    constexpr int PITCH = COLS + 4;
    float* total = sums + WAVES * BLOCKS * 256;   // [16][PITCH]
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= g.M) break;
        lds_barrier();   // the slots, or the last rows, are no longer read
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) *reinterpret_cast<f32x4*>(sums + (wave * BLOCKS + b) * 256 + 4 * lane) = acc[m][b];
        lds_barrier();
        for (int at = threadIdx.x; at < BLOCKS * 256; at += 64 * WAVES) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v += sums[w * BLOCKS * 256 + at];
            const int l = (at & 255) >> 2;
            total[(4 * (l >> 4) + (at & 3)) * PITCH + 16 * (at >> 8) + (l & 15)] = v;
        }
        lds_barrier();
        const int chunks = pair ? COLS / 16 : COLS / 8, row = threadIdx.x / chunks, c = threadIdx.x % chunks, n = n0 + 8 * c;
        if (row < 16 && 16 * m + row < g.M && n < g.out_cols) {
            const float* p = total + row * PITCH + 8 * c;
            float v[8], up[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i], up[i] = pair ? p[COLS / 2 + i] : 0.0f;
            if (g.part) {
                float* to = g.part + (static_cast<int64_t>(blockIdx.y) * g.M + 16 * m + row) * g.N + n;
                store8<T>(to, 0, true, g.out_cols - n, v);
                if (pair) store8<T>(to, g.out_cols, true, g.out_cols - n, up);
            } else {
                linear_out<T>(g, 16 * m + row, n, v, up);
            }
        }
    }
}

template <typename T, bool S> hipError_t run_few(const Product& g, hipStream_t s) {
    auto go = [&](auto mt) {
        using Stream = FewStream<T, S, mt()>;
        constexpr int lds = Stream::WAVES * Stream::SLOTS * kFewSlot;
        static_assert(Stream::WAVES * Stream::BLOCKS * 1024 + 16 * (Stream::COLS + 4) * 4 <= lds, "sums in the slots' place");
        const int width = g.act == MOE_ACT_SWIGLU ? Stream::COLS / 2 : Stream::COLS, blocks = (g.out_cols + width - 1) / width;
        auto* kernel = &linear_few_kernel<T, S, mt()>;
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        kernel<<<dim3((blocks + 7) / 8 * 8, g.splits), 64 * Stream::WAVES, lds, s>>>(g);
        return hipGetLastError();
    };
    return g.M <= 16 ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
}

hipError_t launch_few_splits(const Product& g, int dtype, hipStream_t s) {
    if (dtype == MOE_BF16) return g.b_strided ? run_few<bf16_t, true>(g, s) : run_few<bf16_t, false>(g, s);
    return g.b_strided ? run_few<fp16_t, true>(g, s) : run_few<fp16_t, false>(g, s);
}

}  // namespace

// The splits of least estimated time, in us: the weight from memory at 4.8 TB/s, or a workgroup's part of the weight into its
// compute unit at 31 GB/s (the requests that one keeps in flight) and of x at 1.7 ns per 64 bytes of a row (from L2); and for a
// split the second launch and the partial sums.
int few_splits(int64_t M, int64_t N, int64_t K, bool strided) {
    const int64_t cols = strided ? 64 : 32, depth = strided ? 32 : 64, blocks = (N + cols - 1) / cols, steps = (K + depth - 1) / depth;
    if (steps == 0) return 1;
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 16; s *= 2) {
        if (s > 1 && (steps < 16 * s || blocks * s > 512)) break;
        const double rounds = static_cast<double>((blocks * s + 255) / 256), unit = rounds * K / s * (2.0 * cols / 31e3 + M / 32.0 * 1.7e-3), memory = 2.0 * N * K / 4.8e6;
        const double us = (unit > memory ? unit : memory) + (s > 1 ? 4.0 + 8.0 * s * M * N / 4.8e6 : 0.0);
        if (s == 1 || us < least) best = s, least = us;
    }
    const int64_t per = (steps + best - 1) / best;
    return static_cast<int>((steps + per - 1) / per);   // none is empty
}

hipError_t launch_product_few(Product g, int dtype, void* part, hipStream_t s) {
    const int depth = g.b_strided ? 32 : 64, steps = (g.K + depth - 1) / depth;
    g.splits = few_splits(g.M, g.N, g.K, g.b_strided);
    g.slots = (steps + g.splits - 1) / g.splits;
    g.part = g.splits > 1 ? static_cast<float*>(part) : nullptr;
    const hipError_t e = launch_few_splits(g, dtype, s);
    return e == hipSuccess && g.part ? launch_product_join(g, dtype, s) : e;
}

}  // namespace moe
