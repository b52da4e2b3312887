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
// contiguous bytes per row and instruction, two such steps in flight (three and four measured the same
// at best, and 15% slower where more waves hide the latency).  Two half-wave swaps and two 16-lane swaps
// transpose the 4 x 4 dwords of the four lane groups, so MFMA i of the chunk takes k = 32 i .. 32 i + 31
// (any group size that is a multiple of 32 then ends between two MFMAs).  A team of waves splits K, and
// its sums are added through LDS in wave order: no atomics, the same bits on every run.
//
// Reached: 64 tokens through 32 experts of 7168 x 4096 and back, groups of 32: 170 to 190 us for 730 MB
// of codes, scales and zero points; one token through 6 of 2048 x 2816 and back: 18 us for 27 MB.  A small
// call is bound by its steps in turn: in that one's L1 (9.8 us) the ids take 0.9 us, the first codes 2.1,
// the other steps 4.3, joining and SwiGLU 0.5, and the slowest workgroup ends 2 later.
#include <type_traits>

#include "moe_stream.h"

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

// Eight codes (one dword, low nibble first) as 16 + q, in the order 0 4 1 5 2 6 3 7: one shift and one
// bit-field insert per two codes.  mask and base are W4Type's constants, held in registers (the
// insert takes no literals).
template <typename T> __device__ __forceinline__ u32x4_t expand8(uint32_t w, uint32_t mask, uint32_t base) {
    u32x4_t r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int up = W4Type<T>::kBit - 4 * p;   // nibble p (and p + 4, 16 bits higher) to bit kBit
        const uint32_t v = up >= 0 ? w << up : w >> -up;
        r[p] = (v & mask) | (base & ~mask);
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
constexpr int kW4Ahead = 2;     // steps in flight per wave

// Scales and zero points of a workgroup's NT tiles in LDS: a row per weight row, of `stride` elements, an
// odd multiple of 8, so that the 16 rows a wave reads at once start in different banks.
__host__ __device__ inline int w4_stride(int groups) { return ((groups + 7) / 8 | 1) * 8; }
template <int NT, bool ZEROS> __host__ __device__ inline int w4_meta_bytes(int groups) { return 16 * NT * w4_stride(groups) * (ZEROS ? 3 : 2); }

// What a wave multiplies: the weight rows of its NT tiles (codes: a buffer of one tile's rows each; wrow:
// this lane's offset, row lane % 16 and K part lane / 16), and up to 16 rows of x (this lane's offset in
// row w4_row(); kNoRow: no row).
template <int NT> struct W4Operands {
    rsrc_t codes[NT], x;
    uint32_t wrow, xrow;
    int K, gshift;
};
// The x row of a lane: row r is the MFMA's row 4 (r % 4) + r / 4, so that up to four rows all come out in
// the first accumulator register of the lanes.
__device__ __forceinline__ int w4_row() { return (threadIdx.x & 3) * 4 + ((threadIdx.x >> 2) & 3); }

// The sums of this wave's K chunks (slice, slice + KS, ...): sum[n][i] of x row 4 i + lane / 16 and weight
// row lane % 16 of tile n; with FEW (at most four rows) only i = 0.  kW4Ahead chunks are in flight; ready()
// is called once the first are: it fills the LDS rows that scales and zeros (16 + z) point into, this
// lane's row of tile 0.  FLUSH: MFMAs per scale (min(group, 128) / 32).  ORDERED: x is stored in expand8's
// order within every 8 elements.
template <typename T, int NT, int FLUSH, bool ZEROS, int KS, bool ORDERED, bool FEW, typename F>
__device__ __forceinline__ void w4_sums(const W4Operands<NT>& o, int slice, const uint16_t* scales, const uint8_t* zeros, f32x4_t (&sum)[NT], F&& ready) {
    using W = W4Type<T>;
    const int K = o.K, tile = 16 * w4_stride(K >> o.gshift), chunks = (K + kW4Chunk - 1) / kW4Chunk;
    const u32x4_t ones = {W::kOnes, W::kOnes, W::kOnes, W::kOnes};
    uint32_t mask = W::kMask, base = W::kBase;
    asm("" : "+s"(mask));
    asm("" : "+v"(base));
    u32x4_t code[kW4Ahead][NT], xs[kW4Ahead][4];
    auto fetch = [&](int c, u32x4_t (&to)[NT], u32x4_t (&x)[4]) {
        // k past K: zero rows of x (times the codes of whatever row lies there)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = c * kW4Chunk + 32 * i;
            x[i] = load16(o.x, o.xrow + (k < K ? 2 * static_cast<uint32_t>(k) : kNoK));
        }
        const uint32_t at = o.wrow + (c < chunks ? static_cast<uint32_t>(c) * (kW4Chunk / 2) : kNoRow);
#pragma unroll
        for (int n = 0; n < NT; ++n) to[n] = load16(o.codes[n], at);
    };
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u) fetch(slice + u * KS, code[u], xs[u]);
    ready();
    for (int c0 = slice; c0 < chunks; c0 += kW4Ahead * KS) {
#pragma unroll
        for (int u = 0; u < kW4Ahead; ++u) {
            const int c = c0 + u * KS;
            if (c >= chunks) break;   // the same for the whole wave
            u32x4_t q[NT], xa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) xa[i] = ORDERED ? xs[u][i] : order8(xs[u][i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) q[n] = code[u][n];
            fetch(c + kW4Ahead * KS, code[u], xs[u]);
#pragma unroll
            for (int n = 0; n < NT; ++n) transpose_groups(q[n]);
            const int g = c * kW4Chunk >> o.gshift;
#pragma unroll
            for (int f = 0; f < 4 / FLUSH; ++f) {   // groups past K multiply zero rows
                f32x4_t sx = {}, acc[NT] = {};
#pragma unroll
                for (int h = 0; h < FLUSH; ++h) {
                    const int i = f * FLUSH + h;
                    sx = W::mfma(xa[i], ones, sx);
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n] = W::mfma(xa[i], expand8<T>(q[n][i], mask, base), acc[n]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float s = to_f32(__builtin_bit_cast(T, scales[n * tile + g + f]));
                    const float z = ZEROS ? static_cast<float>(zeros[n * tile + g + f]) : 24.0f;
#pragma unroll
                    for (int i = 0; i < (FEW ? 1 : 4); ++i) sum[n][i] += s * (acc[n][i] - z * sx[i]);
                }
            }
        }
    }
}

// The scales and zero points of NT tiles on their way to LDS, for the KS waves that share the tiles: thread
// i of them takes 8 groups, from group 8 (i / 16), of row i % 16 of every tile.  The loads are issued before the codes', so that the store
// waits for them alone.  Groups beyond what one round of the waves covers follow in store().
template <int NT, bool ZEROS, int KS> struct W4Meta {
    static constexpr int kRound = 8 * 4 * KS;   // groups per round
    static __device__ __forceinline__ int first() { return threadIdx.x % (64 * KS) >> 4 << 3; }
    u32x4_t s[NT];
    uint64_t z[NT];
    const uint16_t* src[NT];    // first row of each tile
    const uint8_t* zsrc[NT];
    int rows[NT], groups;

    __device__ __forceinline__ void load(int g) {
        const int r = threadIdx.x & 15;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int valid = r < rows[n] ? groups - g : 0;   // past the rows and groups: 0 (a NaN times a zero sum would stay)
            s[n] = load_chunk<bf16_t>(reinterpret_cast<const bf16_t*>(src[n] + static_cast<int64_t>(r) * groups + g), valid);
            z[n] = 0;
            if constexpr (ZEROS) {
                const uint8_t* p = zsrc[n] + static_cast<int64_t>(r) * groups + g;
                typedef uint64_t u64_any __attribute__((aligned(1)));
                if (valid >= 8) {
                    z[n] = *reinterpret_cast<const u64_any*>(p);
                } else {
                    for (int i = 0; i < valid; ++i) z[n] |= static_cast<uint64_t>(p[i]) << (8 * i);
                }
            }
        }
    }
    __device__ __forceinline__ void load() { load(first()); }
    __device__ __forceinline__ void store(uint16_t* scales, uint8_t* zeros) {
        const int stride = w4_stride(groups), r = threadIdx.x & 15;
        for (int g = first();;) {
            if (g < stride) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    *reinterpret_cast<u32x4_t*>(scales + (16 * n + r) * stride + g) = s[n];
                    if (ZEROS) *reinterpret_cast<uint64_t*>(zeros + (16 * n + r) * stride + g) = z[n] + 0x1010101010101010u;   // 16 + z
                }
            }
            g += kRound;
            if (g - first() >= stride) break;   // the same for all of them
            load(g);
        }
    }
};

// A workgroup is TEAMS teams of KS waves; a team shares NT tiles and splits K.  LDS of a team: its scales and
// zero points, then (in their place) its waves' sums.
template <int NT, int KS, bool ZEROS> __host__ __device__ inline int w4_team_bytes(int groups) {
    const int meta = w4_meta_bytes<NT, ZEROS>(groups), sums = KS > 1 ? KS * NT * 1024 : 0;
    return ((meta > sums ? meta : sums) + 15) / 16 * 16;
}

// Orders a team's LDS accesses.
template <int KS> __device__ __forceinline__ void team_barrier() {
    if constexpr (KS > 1) lds_barrier();
    else wave_sync();
}

// f(m, col, values) for the elements of a team's tiles: row m, column col of each tile (values[n]).  The
// waves' sums are added in wave order.
template <int NT, int KS, typename F>
__device__ __forceinline__ void w4_outputs(float* lds, int slice, const f32x4_t (&sum)[NT], F&& f) {
    const int lane = threadIdx.x & 63;
    if constexpr (KS == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) v[n] = sum[n][i];
            f(4 * i + (lane >> 4), lane & 15, v);
        }
    } else {
        lds_barrier();   // the scales are no longer read
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4_t*>(lds + (slice * NT + n) * 256 + lane * 4) = sum[n];
        lds_barrier();
        for (int at = threadIdx.x % (64 * KS); at < 256; at += 64 * KS) {
            const int m = at >> 4, col = at & 15;
            float v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float* p = lds + n * 256 + ((m & 3) * 16 + col) * 4 + (m >> 2);
                v[n] = 0.0f;
#pragma unroll
                for (int w = 0; w < KS; ++w) v[n] += p[w * NT * 256];
            }
            f(m, col, v);
        }
    }
}

// Grid: the 16-row tiles of x that share a workgroup's weights run on one XCD (workgroup b is on XCD b mod
// 8), one after the other, so that all but the first read them from its L2.
template <typename T, int NT, int FLUSH, bool ZEROS, int TEAMS, int KS, bool FEW>
__global__ __launch_bounds__(64 * TEAMS * KS, 2) void w4_linear_kernel(W4Linear a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / KS, slice = wave % KS;
    const int groups = a.K >> a.gshift, stride = w4_stride(groups);
    const uint32_t row_tiles = (a.M + 15) / 16, b = blockIdx.x >> 3;
    const int64_t col0 = (static_cast<int64_t>(b / row_tiles) * 8 + (blockIdx.x & 7)) * (16 * NT * TEAMS) + team * 16 * NT;
    if (col0 - team * 16 * NT >= a.N) return;   // the whole workgroup
    const int n0 = static_cast<int>(col0), m0 = static_cast<int>(b % row_tiles) * 16;
    unsigned char* lds = lds_raw + team * w4_team_bytes<NT, KS, ZEROS>(groups);
    uint16_t* scales = reinterpret_cast<uint16_t*>(lds);
    uint8_t* zeros = lds + 16 * NT * stride * 2;

    W4Operands<NT> o;
    W4Meta<NT, ZEROS, KS> meta;
    o.K = a.K;
    o.gshift = a.gshift;
    meta.groups = groups;
#pragma unroll
    for (int n = 0; n < NT; ++n) {   // rows past N read nothing
        const int64_t row = n0 + 16 * n;
        const int rows = max(0, min(16, a.N - static_cast<int>(row)));
        meta.rows[n] = rows;
        meta.src[n] = static_cast<const uint16_t*>(a.scales) + row * groups;
        meta.zsrc[n] = ZEROS ? a.zeros + row * groups : nullptr;
        o.codes[n] = buffer_of(a.codes + row * (a.K >> 1), rows * (a.K >> 1));
    }
    meta.load();
    o.wrow = (lane & 15) * (a.K >> 1) + 16 * (lane >> 4);
    o.x = buffer_of(static_cast<const T*>(a.x) + m0 * a.ldx, 2 * ((min(a.M - m0, 16) - 1) * a.ldx + a.K));
    const int m = w4_row();
    o.xrow = (m0 + m < a.M ? static_cast<uint32_t>(m * a.ldx * 2) : kNoRow) + 16 * (lane >> 4);
    f32x4_t sum[NT] = {};
    w4_sums<T, NT, FLUSH, ZEROS, KS, false, FEW>(o, slice, scales + (lane & 15) * stride, zeros + (lane & 15) * stride, sum, [&] {
        meta.store(scales, zeros);
        team_barrier<KS>();
    });
    w4_outputs<NT, KS>(reinterpret_cast<float*>(lds), slice, sum, [&](int r, int col, const float (&v)[NT]) {
        if (m0 + r >= a.M) return;
        T* y = static_cast<T*>(a.y) + (m0 + r) * a.ldy + n0 + col;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n0 + 16 * n + col < a.N) y[16 * n] = from_f32<T>(v[n]);
    });
}

// ---------------------------------------------------------------------------------------------
// Expert layer.  Grid y: with at most EL pairs, one workgroup row per pair, of which the first pair
// of each expert works and the others leave; with more, one per local expert.  Grid x: tiles of columns, and
// for each (on one XCD, as above) the workgroups that share an expert's passes of 16 rows.  A workgroup lists its
// expert's pairs in ascending order itself (the ids are a few KB), so no table is built beforehand.
// ---------------------------------------------------------------------------------------------
// L1: NT / 2 tiles of gate columns and as many of the up columns of the same intermediate columns;
// act[pair] = silu(gate) up, formed in fp32 and rounded to T, the matrix instruction's operand type, in expand8's
// order.  L2: NT tiles of output columns; stage[pair] = w o in fp32.
template <typename T, bool L1, int NT, int FLUSH, bool ZEROS, int TEAMS, int KS>
__global__ __launch_bounds__(64 * TEAMS * KS, 2) void w4_experts_kernel(W4Experts a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / KS, slice = wave % KS;
    const int pairs = a.T * a.k;
    int* list = reinterpret_cast<int*>(lds_raw + a.list_at);
    const bool by_pair = pairs <= a.EL;
    const int id = by_pair ? __builtin_amdgcn_readfirstlane(a.topk_idx[blockIdx.y]) : a.e_lo + static_cast<int>(blockIdx.y), e = id - a.e_lo;
    constexpr int OUT = L1 ? 8 * NT : 16 * NT;   // output columns of a team: L1's first NT / 2 tiles are the gate's, the others the up's
    const uint32_t passes = a.passes, b = blockIdx.x >> 3, pass = b % passes, block = b / passes * 8 + (blockIdx.x & 7);
    const int col0 = (block * TEAMS + team) * OUT, columns = L1 ? a.I : a.H;
    if (e < 0 || e >= a.EL || static_cast<int>(block * TEAMS) * OUT >= columns) return;
    const int count = expert_pairs(a.topk_idx, pairs, id, by_pair ? static_cast<int>(blockIdx.y) : -1, list), m_first = 16 * pass;
    if (m_first >= count) return;

    const int K = L1 ? a.H : a.I, groups = K >> a.gshift, stride = w4_stride(groups);
    const int64_t wbase = static_cast<int64_t>(e) * (L1 ? 2 * a.I : a.H);   // first row of the expert
    unsigned char* lds = lds_raw + team * w4_team_bytes<NT, KS, ZEROS>(groups);
    uint16_t* scales = reinterpret_cast<uint16_t*>(lds);
    uint8_t* zeros = lds + 16 * NT * stride * 2;
    W4Operands<NT> o;
    W4Meta<NT, ZEROS, KS> meta;
    o.K = K;
    o.gshift = a.gshift;
    meta.groups = groups;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = col0 + 16 * (L1 ? n % (NT / 2) : n);
        const int64_t row = wbase + col + (L1 && n >= NT / 2 ? a.I : 0);
        const int rows = col < columns ? 16 : 0;   // the last team may hold tiles past the end (columns is a multiple of 16)
        meta.rows[n] = rows;
        meta.src[n] = static_cast<const uint16_t*>(L1 ? a.s1 : a.s2) + row * groups;
        meta.zsrc[n] = ZEROS ? (L1 ? a.z1 : a.z2) + row * groups : nullptr;
        o.codes[n] = buffer_of((L1 ? a.w1 : a.w2) + row * (K >> 1), rows * (K >> 1));
    }
    o.wrow = (lane & 15) * (K >> 1) + 16 * (lane >> 4);
    o.x = buffer_of(L1 ? a.x : a.act, static_cast<int64_t>(L1 ? a.T : pairs) * (2 * K));
    for (int m0 = m_first; m0 < count; m0 += 16 * passes) {
        meta.load();
        const int m = m0 + w4_row();
        o.xrow = (m < count ? static_cast<uint32_t>(L1 ? list[m] / a.k : list[m]) * (2 * K) : kNoRow) + 16 * (lane >> 4);
        f32x4_t sum[NT] = {};
        auto ready = [&] {
            team_barrier<KS>();   // the sums of the last rows are no longer read
            meta.store(scales, zeros);
            team_barrier<KS>();
        };
        if (count - m0 <= 4) w4_sums<T, NT, FLUSH, ZEROS, KS, !L1, true>(o, slice, scales + (lane & 15) * stride, zeros + (lane & 15) * stride, sum, ready);
        else w4_sums<T, NT, FLUSH, ZEROS, KS, !L1, false>(o, slice, scales + (lane & 15) * stride, zeros + (lane & 15) * stride, sum, ready);
        w4_outputs<NT, KS>(reinterpret_cast<float*>(lds), slice, sum, [&](int r, int c, const float (&v)[NT]) {
            if (m0 + r >= count) return;
            const int pair = list[m0 + r];
            if constexpr (L1) {
                // column c goes where expand8's order has it: 0 4 1 5 2 6 3 7 -> c = 4 h + q at 2 q + h
                T* act = static_cast<T*>(a.act) + static_cast<int64_t>(pair) * a.I + col0 + (c & 8) + 2 * (c & 3) + ((c >> 2) & 1);
#pragma unroll
                for (int n = 0; n < NT / 2; ++n)
                    if (col0 + 16 * n < columns) act[16 * n] = from_f32<T>(silu_f32(v[n]) * v[n + NT / 2]);
            } else {
                const float w = a.topk_w[pair];
                float* out = a.stage + static_cast<int64_t>(pair) * a.H + col0 + c;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (col0 + 16 * n < columns) out[16 * n] = w * v[n];
            }
        });
    }
}

// L2 and the combine of one token (grid y) in one launch: a wave per slot, TEAMS slots at a time, one tile of
// output columns; y = the sum of w o over the token's local slots, in slot order.  Tokens share no weights
// here: an expert's W2 is read once per pair, from the caches but for the first.
template <typename T, int FLUSH, bool ZEROS, int TEAMS>
__global__ __launch_bounds__(64 * TEAMS, 2) void w4_token_kernel(W4Experts a) {
    extern __shared__ __align__(16) unsigned char lds_raw[];
    __shared__ float part[TEAMS][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = a.I, groups = K >> a.gshift, stride = w4_stride(groups), col0 = blockIdx.x * 16;
    unsigned char* lds = lds_raw + wave * w4_team_bytes<1, 1, ZEROS>(groups);
    uint16_t* scales = reinterpret_cast<uint16_t*>(lds);
    uint8_t* zeros = lds + 16 * stride * 2;
    float y = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += TEAMS) {
        const int slots = min(TEAMS, a.k - j0);
        const int64_t pair = static_cast<int64_t>(blockIdx.y) * a.k + j0 + min(wave, slots - 1);
        const int e = __builtin_amdgcn_readfirstlane(a.topk_idx[pair]) - a.e_lo;
        float v = 0.0f;
        if (wave < slots && e >= 0 && e < a.EL) {
            const int64_t row = static_cast<int64_t>(e) * a.H + col0;
            W4Operands<1> o;
            W4Meta<1, ZEROS, 1> meta;
            o.K = K;
            o.gshift = a.gshift;
            o.wrow = (lane & 15) * (K >> 1) + 16 * (lane >> 4);
            o.xrow = (w4_row() == 0 ? 0 : kNoRow) + 16 * (lane >> 4);
            o.codes[0] = buffer_of(a.w2 + row * (K >> 1), 16 * (K >> 1));
            o.x = buffer_of(static_cast<const T*>(a.act) + pair * K, 2 * K);
            meta.groups = groups;
            meta.rows[0] = 16;
            meta.src[0] = static_cast<const uint16_t*>(a.s2) + row * groups;
            meta.zsrc[0] = ZEROS ? a.z2 + row * groups : nullptr;
            meta.load();
            f32x4_t sum[1] = {};
            w4_sums<T, 1, FLUSH, ZEROS, 1, true, true>(o, 0, scales + (lane & 15) * stride, zeros + (lane & 15) * stride, sum, [&] {
                meta.store(scales, zeros);
                wave_sync();
            });
            v = a.topk_w[pair] * sum[0][0];
        }
        if (lane < 16) part[wave][lane] = v;
        lds_barrier();
        if (threadIdx.x < 16)
            for (int j = 0; j < slots; ++j) y += part[j][threadIdx.x];
        lds_barrier();   // the next slots write part
    }
    if (threadIdx.x < 16) static_cast<T*>(a.y)[static_cast<int64_t>(blockIdx.y) * a.H + col0 + threadIdx.x] = from_f32<T>(y);
}

// y[t] = the sum of the token's local pairs' rows, in slot order (0 with none).  Latency: 64 x 7168, 8 slots: 4.9 us.
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
// rounded to its type first, then the codes are the nearest to w / s.  Weights are quantised once, so
// the second read of a group is left to the caches.
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

constexpr int kLdsBytes = 160 * 1024;

// Launches `kernel` with lds bytes of dynamic LDS, which the caller has found to fit.
template <typename K, typename A> hipError_t launch_w4(K* kernel, dim3 grid, int threads, int lds, const A& a, hipStream_t s) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<grid, threads, lds, s>>>(a);
    return hipGetLastError();
}

template <typename T, int NT, int TEAMS, int KS> hipError_t run_linear(const W4Linear& a, hipStream_t s) {
    hipError_t err = hipSuccess;
    with_group(1 << a.gshift, a.zeros != nullptr, [&](auto flush, auto zeros) {
        const int lds = TEAMS * w4_team_bytes<NT, KS, zeros()>(a.K >> a.gshift);
        constexpr int columns = 16 * NT * TEAMS;
        const int64_t grid = ((static_cast<int64_t>(a.N) + columns - 1) / columns + 7) / 8 * 8 * ((a.M + 15) / 16);
        if (lds > kLdsBytes) {
            err = hipErrorInvalidValue;
            return;
        }
        if (a.M <= 4) err = launch_w4(&w4_linear_kernel<T, NT, flush(), zeros(), TEAMS, KS, true>, dim3(static_cast<unsigned>(grid)), 64 * TEAMS * KS, lds, a, s);
        else err = launch_w4(&w4_linear_kernel<T, NT, flush(), zeros(), TEAMS, KS, false>, dim3(static_cast<unsigned>(grid)), 64 * TEAMS * KS, lds, a, s);
    });
    return err;
}

// LDS bytes of a workgroup's teams.
template <int NT, int TEAMS, int KS> int w4_lds(int groups, bool zeros) {
    return TEAMS * (zeros ? w4_team_bytes<NT, KS, true>(groups) : w4_team_bytes<NT, KS, false>(groups));
}
// Passes of 16 rows that an expert of mean load makes.
inline int w4_passes(const W4Experts& a) { return (a.T * a.k + 16 * a.EL - 1) / (16 * a.EL); }
constexpr int kPassGroups = 512;   // two a CU; 1024 and 2048 measured within 5%, but 300 tokens through 16 of 4096 x 4096 217 against 188 us
template <typename T, bool L1, int NT, int TEAMS, int KS> hipError_t run_experts(W4Experts a, hipStream_t s) {
    hipError_t err = hipSuccess;
    const int K = L1 ? a.H : a.I, columns = L1 ? a.I : a.H, pairs = a.T * a.k;
    with_group(1 << a.gshift, (L1 ? a.z1 : a.z2) != nullptr, [&](auto flush, auto zeros) {
        a.list_at = w4_lds<NT, TEAMS, KS>(K >> a.gshift, zeros());
        constexpr int per = (L1 ? 8 * NT : 16 * NT) * TEAMS;
        const int lds = a.list_at + 4 * pairs;
        if (lds > kLdsBytes) {
            err = hipErrorInvalidValue;
            return;
        }
        // An expert's passes go to workgroups of their own while these are few (101 tokens, 6 of 8 experts of 1408
        // x 1280 and back: 91 to 61 us; 256 tokens, 32 of 256 experts of 7168 x 4096, where most would only look
        // for pairs: 270 to 771 us).
        int blocks = (columns + per - 1) / per;
        const int even = (blocks + 7) / 8 * 8, room = kPassGroups / (even * a.EL);
        a.passes = w4_passes(a) < room ? w4_passes(a) : room;
        if (a.passes > 1) blocks = even * a.passes;
        else a.passes = 1;
        err = launch_w4(&w4_experts_kernel<T, L1, NT, flush(), zeros(), TEAMS, KS>, dim3(blocks, pairs < a.EL ? pairs : a.EL), 64 * TEAMS * KS, lds, a, s);
    });
    return err;
}

constexpr int kTokenSlots = 8;   // waves of a workgroup of w4_token_kernel
template <typename T> hipError_t run_token(const W4Experts& a, hipStream_t s) {
    hipError_t err = hipSuccess;
    with_group(1 << a.gshift, a.z2 != nullptr, [&](auto flush, auto zeros) {
        err = launch_w4(&w4_token_kernel<T, flush(), zeros(), kTokenSlots>, dim3(a.H / 16, a.T), 64 * kTokenSlots,
                        w4_lds<1, kTokenSlots, 1>(a.I >> a.gshift, zeros()), a, s);
    });
    return err;
}
template <typename T> hipError_t run_forward(const W4Experts& a, hipStream_t s) {
    const int pairs = a.T * a.k, slots = pairs < a.EL ? pairs : a.EL;
    // L1.  One row or so per expert: 2 + 2 tiles a workgroup (8 experts of 7168 x 4096 and back: 57 us; four
    // tiles a wave 59 to 65 us).  More rows per expert: four tiles a wave, which then reads x half as often
    // (128 tokens, 64 experts of 2048 x 2816 and back: 146 against 154 us), by two teams while three such
    // workgroups fit a CU's LDS, else by one (64 tokens, 32 experts of 7168 x 4096, groups of 32: 179
    // against 204 us).  Scales too many for those (K beyond any in use): one team of two tiles.
    const int g1 = a.H >> a.gshift, list = 4 * pairs;
    const bool z1 = a.z1 != nullptr, z2 = a.z2 != nullptr;
    hipError_t e;
    if (pairs > a.EL && w4_lds<4, 2, 2>(g1, z1) + list <= kLdsBytes / 3) e = run_experts<T, true, 4, 2, 2>(a, s);
    else if (pairs > a.EL && w4_lds<4, 1, 4>(g1, z1) + list <= kLdsBytes / 2) e = run_experts<T, true, 4, 1, 4>(a, s);
    else if (w4_lds<2, 2, 2>(g1, z1) + list <= kLdsBytes / 2) e = run_experts<T, true, 2, 2, 2>(a, s);
    else e = run_experts<T, true, 2, 1, 4>(a, s);
    if (e != hipSuccess) return e;
    if (w4_by_token(a.T, a.H, a.I)) return run_token<T>(a, s);
    // L2.  Independent waves of two tiles, which need no joining, once there are enough of them (8 experts:
    // 57 us against 64 us with one tile split over four waves; 6 experts of 1408 x 2048: 25 against 22 us).
    const int g2 = a.I >> a.gshift;
    if (static_cast<int64_t>(slots) * w4_passes(a) * (a.H / 16) >= 2048 && w4_lds<2, 4, 1>(g2, z2) + list <= kLdsBytes / 2) e = run_experts<T, false, 2, 4, 1>(a, s);
    else e = run_experts<T, false, 1, 1, 4>(a, s);
    if (e != hipSuccess) return e;
    w4_finish_kernel<T><<<dim3((a.H / 4 + 255) / 256, a.T), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Few tiles of 16 columns: one tile a workgroup, K over as many waves as it feeds (7168 x 4096, one row: 7.2
// us over 8 waves, 8.6 over 4; 1024 x 7168: 5.5 and 4.9 us).  More: two tiles a wave (8192 x 16384, one row:
// 18.5 against 22.6 us), four where several row tiles share the weights or tiles abound (64 rows: 39
// against 51 us).
template <typename T> static hipError_t linear_rows(const W4Linear& a, hipStream_t s) {
    const int64_t row_tiles = (a.M + 15) / 16, tiles = (static_cast<int64_t>(a.N) + 15) / 16 * row_tiles;
    const int groups = a.K >> a.gshift;
    if (tiles >= 1024 && (row_tiles >= 3 || tiles >= 2048) && w4_lds<4, 1, 4>(groups, a.zeros != nullptr) <= kLdsBytes / 2) return run_linear<T, 4, 1, 4>(a, s);
    if (tiles >= 640 && w4_lds<2, 1, 4>(groups, a.zeros != nullptr) <= kLdsBytes / 2) return run_linear<T, 2, 1, 4>(a, s);
    if (tiles > 320 || a.K < 2048) return run_linear<T, 1, 1, 4>(a, s);
    return run_linear<T, 1, 1, 8>(a, s);
}

hipError_t launch_w4_linear(const W4Linear& a, int dtype, hipStream_t s) {
    if (a.M <= 0) return hipSuccess;
    return dtype == MOE_BF16 ? linear_rows<bf16_t>(a, s) : linear_rows<fp16_t>(a, s);
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
