// 16-byte chunks of a row in any of the element types, and wave reductions, for the row kernels
// (norm, router).  A chunk is loaded and stored with the element's own alignment (the hardware
// takes dwordx4 accesses at any address), so rows may start anywhere and have any length; only the
// chunk that holds a row's end is moved element by element.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));

struct bf16_t { uint16_t bits; };
typedef _Float16 fp16_t;

__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(fp16_t v) { return static_cast<float>(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);   // round to nearest even
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) { return bf16_t{f32_to_bf16(v)}; }
template <> __device__ __forceinline__ fp16_t from_f32<fp16_t>(float v) { return static_cast<fp16_t>(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

template <typename T> struct Chunk {
    static constexpr int N = 16 / static_cast<int>(sizeof(T));
    T v[N];
};

// The chunk at p of which `valid` elements lie in the row (<= 0: none, nothing is read); the rest are 0.
template <typename T> __device__ __forceinline__ u32x4_t load_chunk(const T* p, int valid) {
    constexpr int N = Chunk<T>::N;
    if (valid >= N) return *reinterpret_cast<const u32x4_any_t*>(p);
    Chunk<T> c = __builtin_bit_cast(Chunk<T>, u32x4_t{0, 0, 0, 0});
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
        if (i < valid) c.v[i] = p[i];
    return __builtin_bit_cast(u32x4_t, c);
}

// The same in two steps for kernels that load ahead: load_ahead() is one unconditional load (the last 16
// bytes of the row for a chunk that reaches past its end), settle() shifts what it brought into place, under
// a branch that only the last chunks' waves take.  Branches around the loads themselves kept them from being
// issued together and cost registers at every merge.  Rows shorter than a chunk (SHORT) are read by element.
template <typename T, bool SHORT> __device__ __forceinline__ u32x4_t load_ahead(const T* row, int c, int cols) {
    constexpr int N = Chunk<T>::N;
    if (SHORT && cols < N) return load_chunk<T>(row, c == 0 ? cols : 0);
    return *reinterpret_cast<const u32x4_any_t*>(row + min(c, cols - N));
}
template <typename T, bool SHORT> __device__ __forceinline__ u32x4_t settle(u32x4_t v, int c, int cols) {
    constexpr int N = Chunk<T>::N;
    if ((SHORT && cols < N) || c <= cols - N) return v;
    const int past = c - (cols - N);   // elements to drop at the front: the chunk begins there
    if (past >= N) return u32x4_t{0, 0, 0, 0};
    const int bytes = past * static_cast<int>(sizeof(T));
    if (bytes & 8) v = u32x4_t{v[2], v[3], 0, 0};
    if (bytes & 4) v = u32x4_t{v[1], v[2], v[3], 0};
    if (bytes & 2) {
        v[0] = __builtin_amdgcn_alignbyte(v[1], v[0], 2);
        v[1] = __builtin_amdgcn_alignbyte(v[2], v[1], 2);
        v[2] = __builtin_amdgcn_alignbyte(v[3], v[2], 2);
        v[3] >>= 16;
    }
    return v;
}

template <typename T> __device__ __forceinline__ void store_chunk(T* p, u32x4_t raw, int valid) {
    constexpr int N = Chunk<T>::N;
    if (valid >= N) {
        *reinterpret_cast<u32x4_any_t*>(p) = raw;
        return;
    }
    const Chunk<T> c = __builtin_bit_cast(Chunk<T>, raw);
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
        if (i < valid) p[i] = c.v[i];
}

template <typename T> __device__ __forceinline__ void unpack_chunk(u32x4_t raw, float (&f)[Chunk<T>::N]) {
    const Chunk<T> c = __builtin_bit_cast(Chunk<T>, raw);
#pragma unroll
    for (int i = 0; i < Chunk<T>::N; ++i) f[i] = to_f32(c.v[i]);
}

template <typename T> __device__ __forceinline__ u32x4_t pack_chunk(const float (&f)[Chunk<T>::N]) {
    Chunk<T> c;
#pragma unroll
    for (int i = 0; i < Chunk<T>::N; ++i) c.v[i] = from_f32<T>(f[i]);
    return __builtin_bit_cast(u32x4_t, c);
}

// v of the lane that a DPP pattern names (every lane has one: xor inside a quad, mirrors)
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// The wave's sum in every lane: four DPP steps inside each row of 16 lanes, then the two swaps of
// rows and of half-waves (with both operands the same value they pair lanes L and L^16, L and L^32).
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kDppXor1>(v);
    v += dpp<kDppXor2>(v);
    v += dpp<kDppHalfMirror>(v);
    v += dpp<kDppMirror>(v);
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Orders a wave's LDS accesses where its lanes read what others of them wrote: the hardware keeps a wave's
// order, this keeps the compiler to it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

}  // namespace moe
