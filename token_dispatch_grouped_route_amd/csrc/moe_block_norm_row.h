// Block norm, backward of rows that a team of TPR threads holds in registers (NV 16-byte chunks of b a thread), in one launch
// over a run of rows per workgroup.  Every sum over the row that the gradients need is formed in one exchange: the post norm's
// means follow from sums that do not wait for the pre norm's (as in moe_block_norm_bwd.hip).  The sums over the run's rows
// stay in registers: dn N(r) and dn for the pre norm; over the rows of one row of the gate A = sum t N(b) and B = sum t, of which the rest
// are multiples, dgate = scale (w1 A + c1 B), dw1 = scale gate A and dc1 = scale gate B.  Where the registers suffice
// (AHEAD), the next row's loads are in flight while a row is worked on, else they are issued right after it.
//
// Bound by memory: dr, dn, r and b are read once, dx and db written once (8192 x 7168 bf16, RMS, both norms and a gate: 148 us, 4.8 TB/s).  Included by one source per type of b, which share the
// work of compiling it.
#pragma once

#include "moe_block_norm.h"

namespace moe {
namespace {

// A vector of a team's columns in LDS, in fp32, times `scale`, 0 past the row's end; each thread's own elements (so none waits for another).  In
// registers the vectors would take 48 to 64 of them, and 16-bit ones an instruction per element and use.
template <int N, int NV, int TPR> struct RowVector {
    static constexpr int P = N / 4, BYTES = norm_block(TPR) * NV * P * 16;
    float4* at;   // this thread's first piece
    template <typename D> __device__ __forceinline__ void load(const void* w, int64_t from, bool f32, int tid, int cols, float none, float scale) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + tid) * N;
            float f[N];
            if (!w) {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = i < cols - c ? none : 0.0f;
            } else if (f32) {
                Pieces<float, N> v;
                v.load(static_cast<const float*>(w) + from + c, cols - c);
                v.get(f);
            } else {
                Pieces<D, N> v;
                v.load(static_cast<const D*>(w) + from + c, cols - c);
                v.get(f);
            }
#pragma unroll
            for (int h = 0; h < P; ++h) at[(j * P + h) * norm_block(TPR)] = float4{scale * f[4 * h], scale * f[4 * h + 1], scale * f[4 * h + 2], scale * f[4 * h + 3]};
        }
    }
    __device__ __forceinline__ void get(int j, float (&f)[N]) const {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const float4 v = at[(j * P + h) * norm_block(TPR)];
            f[4 * h] = v.x, f[4 * h + 1] = v.y, f[4 * h + 2] = v.z, f[4 * h + 3] = v.w;
        }
    }
};

// As team_sum, for many sums: the waves' parts are read a wave at a time.
template <int TPR, int NS> __device__ __forceinline__ void team_sums(float (&v)[NS], float* lds, int slot) {
    if constexpr (TPR <= 64) {
        team_sum<TPR, NS>(v, lds, slot);
    } else {
        constexpr int W = TPR / 64, TEAMS = norm_block(TPR) / TPR;
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] = wave_sum(v[i]);
        float* buf = lds + (slot * TEAMS + threadIdx.x / TPR) * W * NS;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NS; ++i) buf[(threadIdx.x % TPR >> 6) * NS + i] = v[i];
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] = 0.0f;
#pragma unroll 1
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < NS; ++i) v[i] += buf[w * NS + i];
    }
}

template <typename D, typename R, bool LAYER, int TPR, int NV, bool AHEAD>
__global__ __launch_bounds__(norm_block(TPR)) void block_norm_row_kernel(BlockNorm a, Runs runs, Partials part) {
    constexpr int N = Chunk<D>::N, BLOCK = norm_block(TPR), TEAMS = BLOCK / TPR, NS = LAYER ? 10 : 4, W = norm_waves(TPR), WIDE = TPR * NV * N;
    extern __shared__ __align__(16) unsigned char vectors[];   // four RowVectors
    __shared__ float lds[2 * NS * W];
    __shared__ __align__(16) float join[TEAMS > 1 ? TEAMS * WIDE : 1];
    // (written out where the workgroup is one team, so that rows and their addresses are known to be the same for all of it)
    const int tid = TEAMS == 1 ? threadIdx.x : threadIdx.x % TPR, team = TEAMS == 1 ? 0 : threadIdx.x / TPR, cols = a.cols;
    auto column = [&](int j) { return (j * TPR + tid) * N; };
    int64_t r0, r1;
    runs.range(blockIdx.x, a.rows, r0, r1);

    struct Row {
        Pieces<R, N> dr[NV], r[NV];
        Pieces<D, N> dn[NV], b[NV];
        float stat[4];   // post mean and rstd, pre mean and rstd
    } next;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (a.dr) next.dr[j].load_ahead(static_cast<const R*>(a.dr) + row * a.lddr, column(j), cols);
            if (a.dn) {
                next.dn[j].load_ahead(static_cast<const D*>(a.dn) + row * a.lddn, column(j), cols);
                next.r[j].load_ahead(static_cast<const R*>(a.r) + row * a.ldr, column(j), cols);
            }
            if (a.b) next.b[j].load_ahead(static_cast<const D*>(a.b) + row * a.ldb, column(j), cols);
        }
        next.stat[0] = LAYER && a.post ? a.post_mean[row] : 0.0f;
        next.stat[1] = a.post ? a.post_rstd[row] : 1.0f;
        next.stat[2] = LAYER && a.dn ? a.pre_mean[row] : 0.0f;
        next.stat[3] = a.dn ? a.pre_rstd[row] : 1.0f;
    };
    next = Row{};   // what is not read is 0
    const int64_t first_gate = r0 / runs.share;
    int64_t gate = first_gate, gate_end = min(r1, (gate + 1) * runs.share);
    fetch(min(r0 + team, gate_end - 1));   // a team without a row of its own runs along with another
    using Vector = RowVector<N, NV, TPR>;
    auto vector = [&](int i) { return Vector{reinterpret_cast<float4*>(vectors + i * Vector::BYTES) + threadIdx.x}; };
    Vector w2 = vector(0), w1 = vector(1), gt = vector(2), c1 = vector(3);
    w2.template load<D>(a.pre_weight, 0, a.w_f32, tid, cols, 1.0f, 1.0f);
    w1.template load<D>(a.post_weight, 0, a.w_f32, tid, cols, 1.0f, 1.0f);
    if (LAYER) c1.template load<D>(a.post_bias, 0, a.w_f32, tid, cols, 0.0f, 1.0f);
    gt.template load<D>(a.gate, gate * cols, a.w_f32, tid, cols, 1.0f, a.scale);   // scale gate

    float s_w2[NV][N] = {}, s_c2[LAYER ? NV : 1][N] = {}, s_a[NV][N] = {}, s_b[LAYER ? NV : 1][N] = {};
    // the sum over the teams of a chunk's columns, in the threads of the first team (elsewhere something else)
    auto joined = [&](const float (&sum)[N], float (&t)[N]) {
        if constexpr (TEAMS == 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = sum[i];
        } else {
            static_assert(TEAMS == 1 || NV == 1, "one chunk a thread");
            lds_barrier();   // the last sums have been read
#pragma unroll
            for (int i = 0; i < N; ++i) join[team * WIDE + tid * N + i] = sum[i];
            lds_barrier();
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < TEAMS; ++k)
#pragma unroll
                for (int i = 0; i < N; ++i) t[i] += join[k * WIDE + tid * N + i];
        }
    };
    auto run_row = [&](float* p, int j) { return p + static_cast<int64_t>(blockIdx.x) * cols + column(j); };
    // A and B of the gate's row on to what they are part of
    auto flush = [&](bool first) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float ta[N], tb[N] = {}, g[N], w[N], c[N] = {}, o[N];
            joined(s_a[j], ta);
            if constexpr (LAYER) joined(s_b[j], tb);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s_a[j][i] = 0.0f;
                if constexpr (LAYER) s_b[j][i] = 0.0f;
            }
            const int valid = team == 0 ? cols - column(j) : 0;
            gt.get(j, g);
            if (a.dgate) {
                w1.get(j, w);
                if constexpr (LAYER) c1.get(j, c);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = a.scale * (a.post ? w[i] * ta[i] + c[i] * tb[i] : ta[i]);
                if (part.gate) Pieces<float, N>::put(part.gate + (gate * runs.per_gate + blockIdx.x % runs.per_gate) * cols + column(j), o, valid);
                else if (a.w_f32) Pieces<float, N>::put(static_cast<float*>(a.dgate) + gate * cols + column(j), o, valid);
                else Pieces<D, N>::put(static_cast<D*>(a.dgate) + gate * cols + column(j), o, valid);
            }
            auto add = [&](float* p, const float (&t)[N]) {   // this thread's own columns: what it wrote at the last flush
                if (!p) return;
                float was[N] = {};
                if (!first) {
                    Pieces<float, N> v;
                    v.load(p, valid);
                    v.get(was);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = was[i] + g[i] * t[i];
                Pieces<float, N>::put(p, o, valid);
            };
            add(part.post_weight ? run_row(part.post_weight, j) : nullptr, ta);
            if constexpr (LAYER) add(part.post_bias ? run_row(part.post_bias, j) : nullptr, tb);
        }
    };
    const float inv = 1.0f / static_cast<float>(cols);
    int slot = 0;
    for (int64_t base = r0; base < r1;) {
        const int here = static_cast<int>(min(static_cast<int64_t>(TEAMS), gate_end - base));   // teams with a row of this gate
        const int64_t row = base + team, next_base = base + here;
        const bool last_of_gate = next_base == gate_end;
        Row cur = next;   // (the same registers where not AHEAD)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            cur.dr[j].settle(column(j), cols);
            cur.r[j].settle(column(j), cols);
            cur.dn[j].settle(column(j), cols);
            cur.b[j].settle(column(j), cols);
        }
        auto fetch_next = [&] {
            if (next_base < r1) fetch(min(next_base + team, (last_of_gate ? min(r1, gate_end + runs.share) : gate_end) - 1));
        };
        if (AHEAD) fetch_next();
        // the elements of a chunk: h2 = N(r), h1 = N(b) (or b), g = dn w2, q = scale gate w1; w1 and w2 are 0 past the row's end
        auto elements = [&](int j, float (&dr)[N], float (&dn)[N], float (&h2)[N], float (&h1)[N], float (&fw2)[N], float (&fw1)[N], float (&fg)[N]) {
            cur.dr[j].get(dr);
            cur.dn[j].get(dn);
            cur.r[j].get(h2);
            cur.b[j].get(h1);
            w2.get(j, fw2);
            w1.get(j, fw1);
            gt.get(j, fg);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                h2[i] = (LAYER ? h2[i] - cur.stat[2] : h2[i]) * cur.stat[3];
                h1[i] = (LAYER ? h1[i] - cur.stat[0] : h1[i]) * cur.stat[1];
            }
        };
        auto renew_all = [&](int j) {
            if (NV > 1) __builtin_amdgcn_sched_barrier(0);   // a chunk at a time: several together need more registers than there are
            renew(cur.dn[j].raw[0]);
            renew(cur.b[j].raw[0]);
#pragma unroll
            for (int h = 0; h < Pieces<R, N>::P; ++h) renew(cur.dr[j].raw[h]), renew(cur.r[j].raw[h]);
        };
        float s[NS] = {};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float dr[N], dn[N], h2[N], h1[N], fw2[N], fw1[N], fg[N];
            renew_all(j);
            elements(j, dr, dn, h2, h1, fw2, fw1, fg);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = dn[i] * fw2[i], q = fg[i] * fw1[i], qh = q * h1[i];
                s[0] += g * h2[i];
                s[1] += qh * dr[i];
                s[2] += qh * g;
                s[3] += qh * h2[i];
                if constexpr (LAYER) {
                    s[4] += g;
                    s[5] += qh;
                    s[6] += q * dr[i];
                    s[7] += q * g;
                    s[8] += q;
                    s[9] += q * h2[i];
                }
            }
        }
        team_sums<TPR, NS>(s, lds, slot);
        slot ^= 1;
        const float m1 = s[0] * inv, m0 = LAYER ? s[NS - 6] * inv : 0.0f, rstd2 = cur.stat[3], rstd1 = cur.stat[1];
        float p1 = s[1] + rstd2 * (s[2] - m1 * s[3]), p0 = 0.0f;
        if constexpr (LAYER) {
            p1 -= rstd2 * m0 * s[5];
            p0 = inv * (s[6] + rstd2 * (s[7] - m0 * s[8] - m1 * s[9]));
        }
        p1 *= inv;
        if (team < here) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float dr[N], dn[N], h2[N], h1[N], fw2[N], fw1[N], fg[N], t[N], o[N];
                renew_all(j);
                elements(j, dr, dn, h2, h1, fw2, fw1, fg);
                const int valid = cols - column(j);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    t[i] = dr[i];
                    if (a.dn) t[i] += rstd2 * (dn[i] * fw2[i] - m0 - h2[i] * m1);
                    s_w2[j][i] += dn[i] * h2[i];
                    if constexpr (LAYER) s_c2[j][i] += dn[i];
                    o[i] = a.x_scale * t[i];
                }
                if (a.dx) Pieces<R, N>::put(Pieces<R, N>::template at<R>(static_cast<R*>(a.dx) + row * a.lddx, column(j)), o, valid);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float dp = t[i] * fg[i];
                    s_a[j][i] += t[i] * h1[i];
                    if constexpr (LAYER) s_b[j][i] += t[i];
                    o[i] = a.post ? rstd1 * (dp * fw1[i] - p0 - h1[i] * p1) : dp;
                }
                if (a.db) Pieces<D, N>::put(Pieces<D, N>::template at<D>(static_cast<D*>(a.db) + row * a.lddb, column(j)), o, valid);
            }
        }
        if (!AHEAD) fetch_next();
        if (last_of_gate) {
            if (a.dgate || part.post_weight || part.post_bias) flush(gate == first_gate);
            if (next_base < r1) {
                ++gate;
                gate_end = min(r1, gate_end + runs.share);
                gt.template load<D>(a.gate, gate * cols, a.w_f32, tid, cols, 1.0f, a.scale);
            }
        }
        base = next_base;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float t[N];
        const int valid = team == 0 ? cols - column(j) : 0;
        if (part.pre_weight) {   // the same for the whole launch
            joined(s_w2[j], t);
            Pieces<float, N>::put(run_row(part.pre_weight, j), t, valid);
        }
        if constexpr (LAYER) {
            if (part.pre_bias) {
                joined(s_c2[j], t);
                Pieces<float, N>::put(run_row(part.pre_bias, j), t, valid);
            }
        }
    }
}

template <typename D, typename F> void with_row_team(int64_t chunks, F&& f) {   // up to 8192 elements
    if (chunks <= 16) f(Geo<16, 1>{});
    else if (chunks <= 64) f(Geo<64, 1>{});
    else if (chunks <= 128) f(Geo<128, 1>{});
    else if (chunks <= 256) f(Geo<256, 1>{});
    else if (chunks <= 512) f(Geo<512, 1>{});
    else if (chunks <= 1024) f(Geo<512, 2>{});
    else if constexpr (sizeof(D) == 4) {
        if (chunks <= 1536) f(Geo<512, 3>{});
        else f(Geo<512, 4>{});
    }
}

constexpr int kRowRegisters = 150;

template <typename D> hipError_t launch_row(const BlockNorm& a, const Runs& runs, const Partials& part, hipStream_t s) {
    hipError_t err = hipSuccess;
    auto go = [&](auto stream, auto layer) {
        using R = decltype(stream);
        with_row_team<D>(norm_chunks(a.cols, sizeof(D)), [&](auto geo) {
            using G = decltype(geo);
            // the registers of a row of inputs, 16 bytes of b a chunk: two rows of them fit beside the sums up to these
            constexpr int row = G::nv * (2 + 2 * static_cast<int>(sizeof(R) / sizeof(D))) * 4, sums = G::nv * static_cast<int>(16 / sizeof(D)) * (decltype(layer)::value ? 4 : 2);
            constexpr bool ahead = 2 * row + sums <= kRowRegisters;
            auto* kernel = &block_norm_row_kernel<D, R, decltype(layer)::value, G::tpr, G::nv, ahead>;
            constexpr int lds = (decltype(layer)::value ? 4 : 3) * RowVector<Chunk<D>::N, G::nv, G::tpr>::BYTES;
            if (lds > 49152) err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (err == hipSuccess) kernel<<<static_cast<unsigned>(runs.runs), norm_block(G::tpr), lds, s>>>(a, runs, part);
        });
    };
    auto kind = [&](auto stream) {
        if (a.layer) go(stream, std::true_type{});
        else go(stream, std::false_type{});
    };
    if (a.s_f32) kind(float{});
    else kind(D{});
    return err == hipSuccess ? hipGetLastError() : err;
}

}  // namespace
}  // namespace moe
