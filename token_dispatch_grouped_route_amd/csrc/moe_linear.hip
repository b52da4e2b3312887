// Products of the linear map on the 32 x 32 x 16 MFMA, fp32 accumulators, 16-bit operands in LDS.
//
// A workgroup of four waves (2 x 2) makes a TILE x TILE block of C, in 64-deep steps of the reduction from two
// LDS slots.  An operand whose reduction is contiguous lies in a slot as rows of 64 (128 bytes), its 16-byte
// chunks XOR-swizzled by row so that a fragment read spreads over the banks, and one ds_read_b128 is a lane's
// fragment: 8 consecutive k of a row.  One whose reduction is strided (W in x W, and both operands of x^T dz)
// lies as 64 rows of TILE elements, as it is in memory, chunks swizzled by k, and two transposed reads
// (ds_read_b64_tr_b16) make the same fragment: no copy of a transposed operand is ever written.
#include <type_traits>

#include "moe_linear_tile.h"

namespace moe {

namespace {

template <typename T> __device__ __forceinline__ f32x16 mfma(u32x4_t a, u32x4_t b, f32x16 c);
template <> __device__ __forceinline__ f32x16 mfma<bf16_t>(u32x4_t a, u32x4_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x16 mfma<fp16_t>(u32x4_t a, u32x4_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
}

constexpr int kThreads = 256;   // four waves


// Moves the operand's 64-deep steps into an LDS slot through registers: instruction i of wave w covers the 1 KB
// at 1024 (w + 4 i), lane l its 16 bytes at 16 l; the swizzle is applied to what the lane fetches.  For operands of any
// alignment and size: a load is unconditional, where a chunk would reach past its row's end the row's last 16 bytes,
// which are shifted into place on the way to LDS.  Only the reduction's end needs zeros: rows and columns of the tile past
// the operand's make sums that are not stored.  Rows of less than a chunk are read by element.
template <bool S, int W> struct Loader {
    static constexpr int NI = W / 32;   // instructions per wave and step
    Side o;
    int red, wave, lane;
    bool tiny, edge;   // rows shorter than a chunk; strided: the tile reaches past the last whole chunk of a row

    __device__ __forceinline__ void setup(const Side& side, int reduction, int w, int l) {
        o = side;
        red = reduction;
        wave = w;
        lane = l;
        const int length = S ? o.count : red;
        tiny = length < 8;
        edge = S && o.first + (o.g ? W / 2 : W) > o.count;
    }
    // row and first element (k and column where strided) of this lane's chunk
    __device__ __forceinline__ int row_of(int i) const { return S ? (wave + 4 * i) * (64 / (W / 8)) + lane / (W / 8) : 8 * (wave + 4 * i) + (lane >> 3); }
    __device__ __forceinline__ int chunk_at(int row) const { return S ? 8 * (lane % (W / 8) ^ ((row & 3) << 2)) : 8 * ((lane & 7) ^ ((row >> 1) & 7)); }

    __device__ __forceinline__ void load(int step, u32x4_t (&r)[NI]) const {
        const bf16_t* p = reinterpret_cast<const bf16_t*>(o.p);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int row = row_of(i), at = chunk_at(row);
            if constexpr (!S) {
                const bf16_t* from = p + min(o.real(row), o.limit(row) - 1) * o.ld;
                const int k = step * kLinearDepth + at;
                r[i] = tiny ? load_chunk<bf16_t>(from + k, red - k) : *reinterpret_cast<const u32x4_any_t*>(from + min(k, red - 8));
            } else {
                const int c = o.real(at), end = o.limit(at);
                const bf16_t* from = p + min(step * kLinearDepth + row, red - 1) * o.ld;
                r[i] = tiny ? load_chunk<bf16_t>(from + c, end - c) : *reinterpret_cast<const u32x4_any_t*>(from + min(c, end - 8));
            }
        }
    }
    __device__ __forceinline__ void store(int step, char* slot, u32x4_t (&r)[NI]) const {
        if (!tiny && (edge || (step + 1) * kLinearDepth > red)) {   // the same for the workgroup
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int row = row_of(i), at = chunk_at(row);
                if constexpr (!S) {
                    r[i] = settle<bf16_t, false>(r[i], step * kLinearDepth + at, red);
                } else {
                    r[i] = settle<bf16_t, false>(r[i], o.real(at), o.limit(at));
                    if (step * kLinearDepth + row >= red) r[i] = u32x4_t{0, 0, 0, 0};
                }
            }
        } else if (S && tiny) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (step * kLinearDepth + row_of(i) >= red) r[i] = u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) *reinterpret_cast<u32x4_t*>(slot + 1024 * (wave + 4 * i) + 16 * lane) = r[i];
    }
};

// The same straight from memory into LDS, without registers, for operands whose 16-byte chunks are aligned and whole (or
// padded with zeros): past the last row (column) the last one is read again (its products are not stored), and past the end of the
// reduction, a chunk of zeros.
template <bool S, int W> struct DmaLoader {
    static constexpr int NI = W / 32;
    const char* src[NI];   // this lane's 16 bytes of step 0
    int64_t step_bytes;
    int k0, red, wave;     // k0: this lane's first k of instruction 0 in a step

    __device__ __forceinline__ void setup(const Side& o, int reduction, int w, int lane) {
        red = reduction;
        wave = w;
        const char* p = reinterpret_cast<const char*>(o.p);
        step_bytes = S ? 2 * kLinearDepth * o.ld : 2 * kLinearDepth;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if constexpr (!S) {
                const int v = 8 * (wave + 4 * i) + (lane >> 3), c = (lane & 7) ^ ((v >> 1) & 7);
                src[i] = p + 2 * (min(o.real(v), o.limit(v) - 1) * o.ld + 8 * c);
            } else {
                constexpr int CH = W / 8;
                const int kr = (wave + 4 * i) * (64 / CH) + lane / CH, c = lane % CH ^ ((kr & 3) << 2);
                src[i] = p + 2 * (kr * o.ld + min(o.real(8 * c), (o.limit(8 * c) + 7) / 8 * 8 - 8));   // rows are whole or padded
            }
        }
        // (v >> 1) & 7 and kr & 3 repeat with the instruction: a lane's k of instruction i is k0 (+ 4 i (64 / CH) where strided)
        k0 = S ? wave * (64 / (W / 8)) + lane / (W / 8) : 8 * ((lane & 7) ^ ((8 * wave + (lane >> 3)) >> 1 & 7));
    }
    // LAST: the step may reach past the reduction's end
    template <bool LAST> __device__ __forceinline__ void issue(int step, char* __restrict__ slot, int i) const {
        if constexpr (LAST) {
            const int k = step * kLinearDepth + k0 + (S ? 4 * i * (64 / (W / 8)) : 0);
            uint64_t p = reinterpret_cast<uint64_t>(src[i] + step * step_bytes);
            asm("" : "+v"(p));   // both addresses at hand: one of them is selected, not a load under a branch each
            p = k < red ? p : reinterpret_cast<uint64_t>(kZeroChunk);
            asm("" : "+v"(p));
            __builtin_amdgcn_global_load_lds((g_void*)p, (l_void*)(slot + 1024 * (wave + 4 * i)), 16, 0, 0);
        } else {
            __builtin_amdgcn_global_load_lds((g_void*)(src[i] + step * step_bytes), (l_void*)(slot + 1024 * (wave + 4 * i)), 16, 0, 0);
        }
    }
};

// The MFMA fragments of a wave's 32-wide blocks: lane l holds 8 consecutive k, from 8 (l / 32), of row l % 32.
template <bool S, int W> struct Fragments {
    uint32_t at[4];   // contiguous: per 16-deep part of a step; strided: per block
    __device__ __forceinline__ void setup(int base, int lane) {   // base: first row of the wave's blocks, a multiple of 64
        if constexpr (!S) {
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
                at[kb] = static_cast<uint32_t>((base + (lane & 31)) * 128 + (((2 * kb + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4));
        } else {
            // lane j of a 16-lane group reads 4 consecutive columns 4 (j % 4) of k row j / 4; it receives the four k of column j
            const int g = lane >> 4, j = lane & 15, k = 8 * (g >> 1) + (j >> 2);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int c = base / 8 + 4 * b + 2 * (g & 1) + ((j & 3) >> 1);
                at[b] = static_cast<uint32_t>(k * (2 * W) + ((c ^ ((k & 3) << 2)) << 4) + 8 * (j & 1));
            }
        }
    }
    __device__ __forceinline__ u32x4_t read(const char* __restrict__ slot, int block, int kb) const {
        if constexpr (!S) {
            return *reinterpret_cast<const u32x4_t*>(slot + at[kb] + block * 4096);
        } else {
            const char* p = slot + at[block] + kb * (16 * 2 * W);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s16x4*)(p + 4 * 2 * W));
            const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(u32x4_t, v);
        }
    }
};

template <int TILE> constexpr int lds_slot() { return 2 * TILE * 2 * kLinearDepth; }   // both operands of a step
template <int TILE> constexpr int lds_bytes() {
    const int out = 4 * 32 * (TILE / 2 + 4) * 4;   // 32 rows of each wave's block in fp32
    return 2 * lds_slot<TILE>() > out ? 2 * lds_slot<TILE>() : out;
}

// Workgroup b runs on XCD b mod 8: each XCD takes a run of tiles, in blocks of eight rows of tiles, so that the
// tiles that run together on one XCD share the slices of both operands in its L2.
__device__ __forceinline__ bool tile_of(const Product& g, int tile, int& tm, int& tn, int& split) {
    const int rows = (g.M + tile - 1) / tile, cols = (g.N + tile - 1) / tile;
    const int64_t total = static_cast<int64_t>(rows) * cols * g.splits, per = (total + 7) / 8;
    int64_t t = static_cast<int64_t>(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || t >= total) return false;
    split = static_cast<int>(t / (static_cast<int64_t>(rows) * cols));
    t -= static_cast<int64_t>(split) * rows * cols;
    const int band = static_cast<int>(t / (8 * static_cast<int64_t>(cols))), in = static_cast<int>(t - band * (8 * static_cast<int64_t>(cols)));
    const int high = min(8, rows - 8 * band);
    tm = 8 * band + in % high;
    tn = in / high;
    return true;
}

// The wave's blocks on their way out, 32 rows at a time through LDS (region: 32 rows of WIDE + 4 floats), so
// that every lane ends up with 8 consecutive columns of a row.  For swiglu the first half of the block's columns are
// the gate's.  A lane reads several of its rows, of the residual too, before the first is finished: with one wave a SIMD nothing
// else hides those reads (a 256-wide tile's way out took as long as eight steps of its reduction).
template <typename T, bool PAIR, int NB, int MB>
__device__ __forceinline__ void write_blocks(const Product& g, float* region, const f32x16 (&acc)[MB][NB], int64_t m0, int n0, int split, int lane) {
    constexpr int WIDE = 32 * NB, PITCH = WIDE + 4, CHUNKS = PAIR ? WIDE / 16 : WIDE / 8, STEP = 64 / CHUNKS, ROWS = 32 / STEP, BATCH = ROWS < 4 ? ROWS : 4;
    const int n = n0 + 8 * (lane % CHUNKS);   // an output column
    OutColumns<T> out;
    if (n < g.out_cols && !g.part) out.load(g, n);
    const float* mine = region + lane / CHUNKS * PITCH + 8 * (lane % CHUNKS);
    // one copy of the rows' code for all blocks, and the accumulators still at fixed registers
#pragma unroll 1
    for (int mi = 0; mi < MB; ++mi) {
        wave_sync();   // the last rows have been read
#pragma unroll
        for (int b = 0; b < MB; ++b)
            if (mi == b) {
#pragma unroll
                for (int ni = 0; ni < NB; ++ni)
#pragma unroll
                    for (int r = 0; r < 16; ++r) region[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * PITCH + 32 * ni + (lane & 31)] = acc[b][ni][r];
            }
        wave_sync();
        const int64_t m1 = m0 + 32 * mi + lane / CHUNKS;   // this lane's rows: m1, m1 + STEP, ...
        if (n >= g.out_cols) continue;
#pragma unroll 1
        for (int i0 = 0; i0 < ROWS; i0 += BATCH) {
            float v[BATCH][8], up[BATCH][8], res[BATCH][8];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const float4* p = reinterpret_cast<const float4*>(mine + (i0 + i) * STEP * PITCH);
                auto get = [&](int at, float* to) {
                    const float4 q = p[at];
                    to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                };
                get(0, v[i]);
                get(1, v[i] + 4);
                if (PAIR) {
                    get(WIDE / 8, up[i]);
                    get(WIDE / 8 + 1, up[i] + 4);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) up[i][e] = 0.0f;
                }
            }
            if (g.part) {
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int64_t m = m1 + (i0 + i) * STEP;
                    if (m >= g.M) break;
                    float* to = g.part + (static_cast<int64_t>(split) * g.M + m) * g.N + n;
                    store8<T>(to, 0, true, g.out_cols - n, v[i]);
                    if (PAIR) store8<T>(to, g.out_cols, true, g.out_cols - n, up[i]);
                }
            } else {
                if (g.residual) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (m1 + (i0 + i) * STEP < g.M) out.residual(g, m1 + (i0 + i) * STEP, res[i]);
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (m1 + (i0 + i) * STEP < g.M) out.store(g, m1 + (i0 + i) * STEP, v[i], up[i], res[i]);
            }
        }
    }
}
template <typename T, int NB, int MB>
__device__ __forceinline__ void write_out(const Product& g, float* region, const f32x16 (&acc)[MB][NB], int64_t m0, int n0, int split, int lane) {
    if (g.act == MOE_ACT_SWIGLU) write_blocks<T, true>(g, region, acc, m0, n0, split, lane);
    else write_blocks<T, false>(g, region, acc, m0, n0, split, lane);
}

template <typename T, bool AS, bool BS, int TILE>
__global__ __launch_bounds__(kThreads, 2) void linear_kernel(Product g) {
    extern __shared__ __align__(16) char lds[];
    constexpr int NB = TILE / 64, SLOT = lds_slot<TILE>(), HALF = TILE * 2 * kLinearDepth;
    int tm, tn, split;
    if (!tile_of(g, TILE, tm, tn, split)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
    const bool pair = g.act == MOE_ACT_SWIGLU;
    Loader<AS, TILE> a;
    Loader<BS, TILE> b;
    a.setup(Side{g.a, g.lda, tm * TILE, g.M, 0, 0}, g.K, wave, lane);
    b.setup(pair ? Side{g.b, g.ldb, tn * (TILE / 2), g.out_cols, TILE / 4, g.out_cols} : Side{g.b, g.ldb, tn * TILE, g.N, 0, 0}, g.K, wave, lane);
    Fragments<AS, TILE> fa;
    Fragments<BS, TILE> fb;
    fa.setup(wm * (TILE / 2), lane);
    fb.setup(wn * (TILE / 2), lane);
    const int steps = (g.K + kLinearDepth - 1) / kLinearDepth, j0 = split * g.slots, j1 = min(steps, j0 + g.slots);

    f32x16 acc[NB][NB];
#pragma unroll
    for (int mi = 0; mi < NB; ++mi)
#pragma unroll
        for (int ni = 0; ni < NB; ++ni) acc[mi][ni] = f32x16{};
    // two steps of loads in flight, in registers; two slots
    u32x4_t ra[2][Loader<AS, TILE>::NI], rb[2][Loader<BS, TILE>::NI];
    auto load = [&](int j, int u) {
        a.load(j, ra[u]);
        b.load(j, rb[u]);
    };
    auto store = [&](int j, int u) {
        char* slot = lds + u * SLOT;
        a.store(j, slot, ra[u]);
        b.store(j, slot + HALF, rb[u]);
    };
    if (j0 < j1) {
        load(j0, 0);
        if (j0 + 1 < j1) load(j0 + 1, 1);
        store(j0, 0);
    }
    for (int j = j0; j < j1; j += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (j + u >= j1) break;   // the same for the workgroup
            const char* cur = lds + u * SLOT;
            lds_barrier();   // the step's operands are in LDS, and the last step's no longer read
            if (j + u + 2 < j1) load(j + u + 2, u);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                u32x4_t af[NB], bf[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) af[i] = fa.read(cur, i, kb), bf[i] = fb.read(cur + HALF, i, kb);
#pragma unroll
                for (int mi = 0; mi < NB; ++mi)
#pragma unroll
                    for (int ni = 0; ni < NB; ++ni) acc[mi][ni] = mfma<T>(af[mi], bf[ni], acc[mi][ni]);
            }
            if (j + u + 1 < j1) store(j + u + 1, 1 - u);
        }
    }
    lds_barrier();
    constexpr int REGION = 32 * (32 * NB + 4);
    write_out<T, NB, NB>(g, reinterpret_cast<float*>(lds) + wave * REGION, acc, static_cast<int64_t>(tm) * TILE + wm * (TILE / 2),
                         pair ? tn * (TILE / 2) + wn * (TILE / 4) : tn * TILE + wn * (TILE / 2), split, lane);
}

// The K loop on DMA loads, two slots.  Per step, 16-deep parts 0 .. 3, whose fragments are read two parts ahead (two of the next
// step's during part 3).  So this step's slot has been read by the end of part 1: one barrier, and the loads of the step
// after the next go into it during parts 2 and 3 and part 0 of the next step, spread out, since a compute unit takes in
// 64 bytes a cycle and the waves stall where more are asked for at once (all of them within one part cost 4 to 9% of the
// whole product).  A second barrier, with the next step's loads landed, stands before part 3.
// 8192 x 8192 x 8192 bf16 824 us with W by row (1335 TFLOP/s), 806 by column (1365), 860 for x^T dz (1278).  At 8192 rows, 7168 and 4096 the matrix
// core is busy 64% of the forward, 59% of dx and 54% of dW: 2, 3.5 and 1.75 rounds of tiles on 256 CUs, each with its own ramp and way out.
template <typename T, bool AS, bool BS, int TILE> struct DmaLoop {
    static constexpr int NB = TILE / 64, HALF = TILE * 2 * kLinearDepth, LOADS = 2 * (TILE / 32);
    static constexpr int P2 = LOADS * 3 / 8, P3 = P2, P0 = LOADS - P2 - P3;   // loads in parts 2, 3 and 0
    DmaLoader<AS, TILE> a;
    DmaLoader<BS, TILE> b;
    Fragments<AS, TILE> fa;
    Fragments<BS, TILE> fb;
    typedef u32x4_t Frags[4][NB];

    __device__ __forceinline__ void fragments(const char* __restrict__ slot, int kb, u32x4_t (&af)[NB], u32x4_t (&bf)[NB]) const {
#pragma unroll
        for (int i = 0; i < NB; ++i) af[i] = fa.read(slot, i, kb), bf[i] = fb.read(slot + HALF, i, kb);
    }
    static __device__ __forceinline__ void multiply(const u32x4_t (&af)[NB], const u32x4_t (&bf)[NB], f32x16 (&acc)[NB][NB]) {
#pragma unroll
        for (int mi = 0; mi < NB; ++mi)
#pragma unroll
            for (int ni = 0; ni < NB; ++ni) acc[mi][ni] = mfma<T>(af[mi], bf[ni], acc[mi][ni]);
    }
    // loads FROM .. FROM + N - 1 of a step, of the two operands in turn
    template <bool LAST, int FROM, int N> __device__ __forceinline__ void issue(int step, char* __restrict__ slot) const {
#pragma unroll
        for (int i = FROM; i < FROM + N; ++i) {
            if (i % 2 == 0) a.template issue<LAST>(step, slot, i / 2);
            else b.template issue<LAST>(step, slot + HALF, i / 2);
        }
    }
    // order: an MFMA, fragment reads, a load, in turn
    template <int READS, int LOADS_HERE> static __device__ __forceinline__ void interleave() {
        constexpr int NM = NB * NB, NR = READS * NB * ((AS ? 2 : 1) + (BS ? 2 : 1)), RPM = (NR + NM - 1) / NM, LPM = (LOADS_HERE + NM - 1) / NM;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
            for (int x = 0; x < RPM; ++x)
                if (i * RPM + x < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int x = 0; x < LPM; ++x)
                if (i * LPM + x < LOADS_HERE) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    template <int VM> static __device__ __forceinline__ void barrier() {   // with all but the last VM loads landed, and all reads
        wait_counts<VM, true>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }
    // LAST: steps j + 1 and j + 2 may reach past the end.  Loads past the last step read that one again.
    template <bool LAST> __device__ __forceinline__ void step(int j, int last, char* __restrict__ cur, char* __restrict__ other, Frags& af, Frags& bf, f32x16 (&acc)[NB][NB]) const {
        issue<LAST, P2 + P3, P0>(min(j + 1, last), other);
        fragments(cur, 2, af[2], bf[2]);
        multiply(af[0], bf[0], acc);
        interleave<1, P0>();
        fragments(cur, 3, af[3], bf[3]);
        multiply(af[1], bf[1], acc);
        interleave<1, 0>();
        barrier<63>();   // this slot has been read
        issue<LAST, 0, P2>(min(j + 2, last), cur);
        multiply(af[2], bf[2], acc);
        interleave<0, P2>();
        barrier<P2>();   // the next step has landed
        issue<LAST, P2, P3>(min(j + 2, last), cur);
        fragments(other, 0, af[0], bf[0]);
        fragments(other, 1, af[1], bf[1]);
        multiply(af[3], bf[3], acc);
        interleave<2, P3>();
    }
    __device__ __forceinline__ void run(int j0, int j1, char* __restrict__ s0, char* __restrict__ s1, f32x16 (&acc)[NB][NB]) const {
        const int last = j1 - 1;
        issue<true, 0, LOADS>(j0, s0);
        __builtin_amdgcn_sched_barrier(0);
        issue<true, 0, P2 + P3>(min(j0 + 1, last), s1);
        barrier<P2 + P3>();
        Frags af, bf;
        fragments(s0, 0, af[0], bf[0]);
        fragments(s0, 1, af[1], bf[1]);
        const int main = a.red >= j1 * kLinearDepth ? j1 : last - 2;   // steps before it load whole ones only
        int j = j0;
        for (; j + 1 < main; j += 2) {
            step<false>(j, last, s0, s1, af, bf, acc);
            step<false>(j + 1, last, s1, s0, af, bf, acc);
        }
        // one copy of the code for the rest: with more, the accumulators, which fill their registers, are moved through memory where
        // the paths meet
        for (; j < j1; ++j) step<true>(j, last, (j - j0) & 1 ? s1 : s0, (j - j0) & 1 ? s0 : s1, af, bf, acc);
    }
};

template <typename T, bool AS, bool BS, int TILE>
__global__ __launch_bounds__(kThreads, TILE == 256 ? 1 : 2) void linear_dma_kernel(Product g) {
    extern __shared__ __align__(16) char lds[];
    constexpr int NB = TILE / 64;
    int tm, tn, split;
    if (!tile_of(g, TILE, tm, tn, split)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
    const bool pair = g.act == MOE_ACT_SWIGLU;
    DmaLoop<T, AS, BS, TILE> loop;
    loop.a.setup(Side{g.a, g.lda, tm * TILE, g.M, 0, 0}, g.K, wave, lane);
    loop.b.setup(pair ? Side{g.b, g.ldb, tn * (TILE / 2), g.out_cols, TILE / 4, g.out_cols} : Side{g.b, g.ldb, tn * TILE, g.N, 0, 0}, g.K, wave, lane);
    loop.fa.setup(wm * (TILE / 2), lane);
    loop.fb.setup(wn * (TILE / 2), lane);
    const int steps = (g.K + kLinearDepth - 1) / kLinearDepth, j0 = split * g.slots, j1 = min(steps, j0 + g.slots);
    f32x16 acc[NB][NB];
#pragma unroll
    for (int mi = 0; mi < NB; ++mi)
#pragma unroll
        for (int ni = 0; ni < NB; ++ni) acc[mi][ni] = f32x16{};
    if (j0 < j1) loop.run(j0, j1, lds, lds + lds_slot<TILE>(), acc);
    DmaLoop<T, AS, BS, TILE>::template barrier<0>();   // no load is on its way into LDS, and all has been read
    constexpr int REGION = 32 * (32 * NB + 4);
    write_out<T, NB, NB>(g, reinterpret_cast<float*>(lds) + wave * REGION, acc, static_cast<int64_t>(tm) * TILE + wm * (TILE / 2),
                         pair ? tn * (TILE / 2) + wn * (TILE / 4) : tn * TILE + wn * (TILE / 2), split, lane);
}

// Joins the splits: eight columns of y a thread.
template <typename T> __global__ __launch_bounds__(256) void linear_join_kernel(Product g) {
    const int chunks = (g.out_cols + 7) / 8;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, m = at / chunks;
    if (m >= g.M) return;
    const int n = static_cast<int>(at - m * chunks) * 8, valid = g.out_cols - n;
    float v[8] = {}, up[8] = {};
    for (int s = 0; s < g.splits; ++s) {
        const float* p = g.part + (static_cast<int64_t>(s) * g.M + m) * g.N + n;
        float f[8];
        load8<T>(p, 0, true, valid, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
        if (g.act == MOE_ACT_SWIGLU) {
            load8<T>(p, g.out_cols, true, valid, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) up[i] += f[i];
        }
    }
    linear_out<T>(g, m, n, v, up);
}

// Copies an operand's rows with zeros up to a multiple of 8 elements, 8 a thread.
struct PadCopy {
    const uint16_t* from;
    uint16_t* to;
    int64_t rows, ld;
    int32_t extent;
};
__global__ __launch_bounds__(256) void linear_pad_kernel(PadCopy a, PadCopy b) {
    const PadCopy c = blockIdx.y ? b : a;
    const int chunks = (c.extent + 7) / 8;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = at / chunks;
    if (row >= c.rows) return;
    const int i = static_cast<int>(at - row * chunks) * 8;
    *reinterpret_cast<u32x4_t*>(c.to + at * 8) = load_chunk<bf16_t>(reinterpret_cast<const bf16_t*>(c.from) + row * c.ld + i, c.extent - i);
}

template <typename T, bool AS, bool BS, int TILE, bool DMA> hipError_t run_product(const Product& g, hipStream_t s) {
    void (*kernel)(Product);
    if constexpr (DMA) kernel = &linear_dma_kernel<T, AS, BS, TILE>;
    else kernel = &linear_kernel<T, AS, BS, TILE>;
    constexpr int lds = lds_bytes<TILE>();
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const int64_t total = static_cast<int64_t>((g.M + TILE - 1) / TILE) * ((g.N + TILE - 1) / TILE) * g.splits;
    kernel<<<static_cast<unsigned>((total + 7) / 8 * 8), kThreads, lds, s>>>(g);
    return hipGetLastError();
}

template <typename T, bool AS, bool BS> hipError_t run_tiles(const Product& g, const Plan& plan, hipStream_t s) {
    if (plan.dma && plan.tile == 256) return run_product<T, AS, BS, 256, true>(g, s);
    if (plan.dma) return run_product<T, AS, BS, 128, true>(g, s);
    return run_product<T, AS, BS, 128, false>(g, s);
}
template <typename T> hipError_t run_layouts(const Product& g, const Plan& plan, hipStream_t s) {
    if (g.a_strided) return run_tiles<T, true, true>(g, plan, s);
    if (g.b_strided) return run_tiles<T, false, true>(g, plan, s);
    return run_tiles<T, false, false>(g, plan, s);
}

}  // namespace

// Tile and splits of the reduction: of all, the one of least estimated time.  A step of the reduction takes a workgroup 0.68 us alone on
// its CU and 1.03 us beside another (128 wide), 1.75 us (256 wide, less in a last round that leaves CUs idle); without whole
// chunks 1.3 and 1.9 us; a round of workgroups costs 3 us more, a split the join's launch and its sums' way to memory and back.  Measured: 2048 x 2048 x 2048 27.8 us in 256 tiles,
// 35.4 with two splits; 512 x 4096 x 7168 44 us with four splits, 48 with two; 8192 x 2048 x 2048 71 us 256 wide, 76 us 128 wide.
Plan product_plan(int64_t M, int64_t N, int64_t K, bool dma) {
    const int64_t steps = (K + kLinearDepth - 1) / kLinearDepth;
    Plan best{dma, 128, 1, 0.0};
    if (M <= 0 || steps == 0) return best;
    double least = 0.0;
    for (int tile = 128; tile <= (dma ? 256 : 128); tile *= 2) {
        const int64_t tiles = (M + tile - 1) / tile * ((N + tile - 1) / tile), room = tile == 256 ? 256 : 512;
        for (int n = 1; n <= 16; ++n) {
            if (n > 1 && (steps < 4 * n || tiles * n > room)) break;
            const int64_t per = (steps + n - 1) / n, splits = (steps + per - 1) / per, rest = tiles * splits % room, full = tiles * splits / room;   // none is empty
            const double alone = dma ? 0.68 : 1.3, both = tile == 256 ? 1.75 : dma ? 1.03 : 1.9;
            const double last = rest == 0 ? 0.0 : tile == 256 ? both * (0.4 + 0.6 * rest / 256) : rest <= 256 ? alone : both;
            double us = per * (full * both + last) + 3.0 * (full + (rest > 0)) + 3.0;
            if (splits > 1) us += 4.0 + 5.2 * splits * M * N / 4.5e6;
            if (least == 0.0 || us < least) least = us, best.tile = tile, best.splits = static_cast<int>(splits);
        }
    }
    best.us = least;
    return best;
}

size_t product_part_bytes(int64_t M, int64_t N, int64_t K) {   // whatever the alignment
    int splits = 1;
    auto at_least = [&](int n) { splits = n > splits ? n : splits; };
    at_least(product_plan(M, N, K, true).splits);
    at_least(product_plan(M, N, K, false).splits);
    if (M > 0 && M <= kLinearFew) at_least(few_splits(M, N, K, true)), at_least(few_splits(M, N, K, false));
    return splits > 1 ? static_cast<size_t>(splits) * M * N * 4 : 0;
}

int64_t padded_elements(int64_t rows, int64_t extent) { return extent % 8 == 0 ? 0 : rows * ((extent + 7) / 8 * 8); }
namespace {
size_t pad_bytes_of(int64_t elements) { return (static_cast<size_t>(elements) * 2 + 255) / 256 * 256; }
}  // namespace

// Where the sizes divide into no chunks, the operands are copied with whole ones if that and the faster loop are estimated to
// take less: a launch, and the copy at 4.5 TB/s.  8192 x 4095 x 7167 bf16 847 -> 497 us, 2047 x 2047 x 2047 50 -> 34 us.
size_t product_pad_bytes(int64_t M, int64_t N, int64_t K, int64_t a, int64_t b) {
    constexpr int64_t kMost = int64_t(1) << 33;   // the copy's grid stays below 2^32 threads
    if (M <= 0 || a + b == 0 || a > kMost || b > kMost) return 0;
    const double copy = 4.0 + 4.0 * static_cast<double>(a + b) / 4.5e6;
    return product_plan(M, N, K, true).us + copy < product_plan(M, N, K, false).us ? pad_bytes_of(a) + pad_bytes_of(b) : 0;
}

hipError_t launch_product(Product g, int dtype, void* part, void* pad, size_t pad_bytes, hipStream_t s) {
    if (g.M <= 0) return hipSuccess;
    const bool paired = g.b_strided && g.act == MOE_ACT_SWIGLU;   // a row of the weight is two
    const int64_t a_rows = g.a_strided ? g.K : g.M, b_rows = g.b_strided ? g.K : g.N, a_extent = g.a_strided ? g.M : g.K, b_extent = g.b_strided ? (paired ? g.out_cols : g.N) : g.K;
    auto ready = [](const void* p, int64_t ld, int64_t extent, bool padded) { return whole_chunks(p, ld, padded ? 0 : extent); };
    const bool a_ready = ready(g.a, g.lda, a_extent, g.a_padded), b_ready = ready(g.b, g.ldb, b_extent, g.b_padded);
    bool whole = a_ready && b_ready;
    if (!g.a_strided && whole && g.M <= kLinearFew && (g.M > 1 || g.b_strided)) return launch_product_few(g, dtype, part, s);
    if (!g.a_strided && g.M <= kLinearRows) return launch_product_rows(g, dtype, s);
    if (!whole) {
        const int64_t a = a_ready ? 0 : padded_elements(a_rows, a_extent), b = b_ready || paired ? 0 : padded_elements(b_rows, b_extent);
        const size_t need = (a_ready || a) && (b_ready || b) ? product_pad_bytes(g.M, g.N, g.K, a, b) : 0;
        if (need > 0 && need <= pad_bytes) {
            PadCopy ca = {}, cb = {};
            if (a) ca = {g.a, static_cast<uint16_t*>(pad), a_rows, g.lda, static_cast<int32_t>(a_extent)}, g.a = ca.to, g.lda = a / a_rows;
            if (b) cb = {g.b, reinterpret_cast<uint16_t*>(static_cast<char*>(pad) + pad_bytes_of(a)), b_rows, g.ldb, static_cast<int32_t>(b_extent)}, g.b = cb.to, g.ldb = b / b_rows;
            const int64_t chunks = (a > b ? a : b) / 8;
            linear_pad_kernel<<<dim3(static_cast<unsigned>((chunks + 255) / 256), a && b ? 2 : 1), 256, 0, s>>>(a ? ca : cb, cb);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            whole = true;
        }
    }
    const Plan plan = product_plan(g.M, g.N, g.K, whole);
    g.splits = plan.splits;
    const int steps = (g.K + kLinearDepth - 1) / kLinearDepth;
    g.slots = (steps + g.splits - 1) / g.splits;
    g.part = g.splits > 1 ? static_cast<float*>(part) : nullptr;
    const hipError_t e = dtype == MOE_BF16 ? run_layouts<bf16_t>(g, plan, s) : run_layouts<fp16_t>(g, plan, s);
    return e == hipSuccess && g.part ? launch_product_join(g, dtype, s) : e;
}

hipError_t launch_product_join(const Product& g, int dtype, hipStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(g.M) * ((g.out_cols + 7) / 8) + 255) / 256;
    if (dtype == MOE_BF16) linear_join_kernel<bf16_t><<<static_cast<unsigned>(blocks), 256, 0, s>>>(g);
    else linear_join_kernel<fp16_t><<<static_cast<unsigned>(blocks), 256, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace moe
