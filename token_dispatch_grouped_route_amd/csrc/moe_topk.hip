// Top-k router: expert ids and weights from router logits, and the gradient back to the logits.
//
//   l = min(logit, largest finite); an expert whose logit is NaN or -inf is out of service
//   s = v + bias, with v = l, or (SCORES) v = the score that follows from l, the p over all in service below;
//   with expert groups, the groups of the largest (best + second best s) stay
//   ids = the k largest s, descending, ties to the lower id; -1 (weight 0) where none is left
//   softmax:  p_j = exp(l_j - m) / sum over the chosen (renormalised) or over all in service
//   sigmoid:  p_j = 1 / (1 + exp(-l_j)), over the sum of the chosen (renormalised) or as it is
//   weight = scale p;  backward, with g = scale dweight and q = sum over the chosen of p g:
//   softmax:  dl_j = p_j (g_j - q) renormalised, else dl_e = p_e ([e chosen] g_e - q) for every e
//   sigmoid:  dl_j = p_j (1 - sigmoid(l_j)) (g_j - [renormalised] q)
//
// A row belongs to LPR lanes, each with NC 16-byte chunks of its logits in registers: 16 lanes (four
// rows a wave; every exchange between the lanes of a row is a DPP step) or 64.
//
// The choice costs more than the memory traffic if it is done on (score, id) pairs: k rounds of finding
// and removing a row's best took 33 us for 65536 x 384 bf16 logits (top 6), whose bytes move in 11 us.
// So a score and its id become one 32-bit key, the score's order-preserving bits with the id (inverted:
// ties go to the lower) in the low bits, and a lane keeps its four largest keys sorted: a compare and
// exchange is a min and a max, and a round is a maximum over the heads of the row's lanes and a pop:
// 17 us for those logits; 65536 x 256, top 8: bf16 with a bias 20 us, fp32 with 8 groups 31 us.  A lane whose four keys were all
// taken makes its list anew from what is below the last one.
// The key drops score bits where the id needs them.  16-bit logits without a bias have none there; else
// the rounds go on while two neighbours agree in all bits kept, and the keys taken are then ranked by
// their scores and ids (exact rounds on pairs only where there are more of them than lanes).
#include <type_traits>

#include "moe_vec.h"

namespace moe {

constexpr float kNegInf = -__builtin_inff();
constexpr float kF32Max = 3.402823466e38f;

// l of a logit: NaN and -inf -> -inf, +inf -> the largest finite number.
// (The larger of a NaN and a number is the number.)
__device__ __forceinline__ float usable_logit(float v) { return fminf(fmaxf(v, kNegInf), kF32Max); }

// The other lanes' (value, id) pairs of a row, step by step: after all steps every lane holds the
// best of the row's lanes, for any combine that is commutative, associative and idempotent or a sum
// over disjoint sets (each step joins two disjoint halves).
template <int LPR, typename F> __device__ __forceinline__ void row_exchange(float& v, int& id, F&& join) {
    join(v, id, dpp<kDppXor1>(v), static_cast<int>(dpp<kDppXor1>(static_cast<uint32_t>(id))));
    join(v, id, dpp<kDppXor2>(v), static_cast<int>(dpp<kDppXor2>(static_cast<uint32_t>(id))));
    join(v, id, dpp<kDppHalfMirror>(v), static_cast<int>(dpp<kDppHalfMirror>(static_cast<uint32_t>(id))));
    join(v, id, dpp<kDppMirror>(v), static_cast<int>(dpp<kDppMirror>(static_cast<uint32_t>(id))));
    if constexpr (LPR == 64) {
        auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        auto b = __builtin_amdgcn_permlane16_swap(static_cast<uint32_t>(id), static_cast<uint32_t>(id), false, false);
        v = __uint_as_float(a[0]);
        id = static_cast<int>(b[0]);
        join(v, id, __uint_as_float(a[1]), static_cast<int>(b[1]));
        a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        b = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(id), static_cast<uint32_t>(id), false, false);
        v = __uint_as_float(a[0]);
        id = static_cast<int>(b[0]);
        join(v, id, __uint_as_float(a[1]), static_cast<int>(b[1]));
    }
}
template <int LPR> __device__ __forceinline__ float row_sum(float v) {
    int none = 0;
    row_exchange<LPR>(v, none, [](float& a, int&, float b, int) { a += b; });
    return v;
}
template <int LPR> __device__ __forceinline__ float row_max(float v) {
    int none = 0;
    row_exchange<LPR>(v, none, [](float& a, int&, float b, int) { a = fmaxf(a, b); });
    return v;
}

__device__ __forceinline__ void better(float& v, int& id, float ov, int oid) {
    if (ov > v || (ov == v && oid < id)) v = ov, id = oid;
}

// The weights are ratios of fast exponentials, off by (2.5 |a| + 4) 2^-24 relative at an argument a: 2^-20 for a
// weight that is e^-5 of its row's largest, less than the products they scale are rounded by.
__device__ __forceinline__ float sigmoid_f32(float l) {   // no overflow on either side
    const float e = __expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}
__device__ __forceinline__ float log_sigmoid_f32(float l) { return fminf(l, 0.0f) - log1pf(__expf(-fabsf(l))); }

// The weight p of each chosen expert before scaling; l: lane j's chosen logit, there: slot j holds one.
template <int LPR>
__device__ __forceinline__ float chosen_weight(const RouteArgs& a, float l, bool there, float all_max, float all_sum) {
    if (a.renorm) {
        const float v = there ? (a.sigmoid ? log_sigmoid_f32(l) : l) : kNegInf;
        const float m = row_max<LPR>(v);
        const float e = there ? __expf(v - m) : 0.0f;
        const float sum = row_sum<LPR>(e);
        return there ? e / sum : 0.0f;
    }
    if (!there) return 0.0f;
    return a.sigmoid ? sigmoid_f32(l) : __expf(l - all_max) / all_sum;
}

// What the choice by scores goes by, for an expert in service.
__device__ __forceinline__ float choice_score(const RouteArgs& a, float l, float all_max, float all_sum) {
    return a.sigmoid ? sigmoid_f32(l) : __expf(l - all_max) / all_sum;
}

template <int LPR> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, dpp<kDppXor1>(v));
    v = max(v, dpp<kDppXor2>(v));
    v = max(v, dpp<kDppHalfMirror>(v));
    v = max(v, dpp<kDppMirror>(v));
    if constexpr (LPR == 64) {
        auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(r[0], r[1]);
        r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(r[0], r[1]);
    }
    return v;
}

// Bits of a float in the order of unsigned integers (-0 below +0: the caller adds +0 first).  -inf and all
// below its place come out under kLeastKey.
__device__ __forceinline__ uint32_t ordered_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// What the kernel is compiled for: any row; rows of whole chunks; those without a bias and groups.  The
// checks of the general form made the plain one's code larger than the instruction cache (65536 x 384
// bf16: 42 us, against 33 us of the exact rounds).
enum RouteMode { kAnyRow, kWholeChunks, kPlain };

// The chunk at p of which `valid` elements lie in the row; the others are -inf.
template <typename T, RouteMode MODE> __device__ __forceinline__ u32x4_t load_logits(const T* p, int valid) {
    constexpr int N = Chunk<T>::N;
    constexpr uint32_t none = std::is_same<T, bf16_t>::value ? 0xff80ff80u : std::is_same<T, fp16_t>::value ? 0xfc00fc00u : 0xff800000u;
    u32x4_t raw = {none, none, none, none};
    if (valid >= N) {
        raw = *reinterpret_cast<const u32x4_any_t*>(p);
    } else if (MODE == kAnyRow && valid > 0) {
        Chunk<T> c = __builtin_bit_cast(Chunk<T>, raw);
#pragma unroll
        for (int i = 0; i < N - 1; ++i)
            if (i < valid) c.v[i] = p[i];
        raw = __builtin_bit_cast(u32x4_t, c);
    }
    return raw;
}
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {   // a >= b
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// The four largest of the sorted list `best` and the four values q, sorted.
__device__ __forceinline__ void merge4(uint32_t (&best)[4], uint32_t (&q)[4]) {
    order2(q[0], q[1]);
    order2(q[2], q[3]);
    order2(q[0], q[2]);
    order2(q[1], q[3]);
    order2(q[1], q[2]);
#pragma unroll
    for (int i = 0; i < 4; ++i) best[i] = max(best[i], q[3 - i]);   // the larger four of both, rising then falling
    order2(best[0], best[2]);
    order2(best[1], best[3]);
    order2(best[0], best[1]);
    order2(best[2], best[3]);
}

// Group-limited choice: which groups of the row stay (bit g for group g).  s: the scores of this lane's
// chunks of N elements.
template <int N, int LPR, int NC>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const float (&s)[NC * N], int lane) {
    const int base = (threadIdx.x & 63) / LPR * LPR;
    float mine = kNegInf;   // lane g: the score of group g
    auto join = [](float& p, int& q, float op, int oq) {
        q = __float_as_int(fmaxf(fmaxf(__int_as_float(q), __int_as_float(oq)), fminf(p, op)));
        p = fmaxf(p, op);
    };
    auto score = [](float v1, float v2) { return v2 > kNegInf ? v1 + v2 : v1; };
    const int shift = a.group_shift;
    if (shift >= 0) {   // a group is 2^shift (1 to 16) lanes of one chunk row
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float v1 = kNegInf, v2 = kNegInf;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v2 = fmaxf(v2, fminf(v1, s[j * N + i]));
                v1 = fmaxf(v1, s[j * N + i]);
            }
            int second = __float_as_int(v2);
            if (shift > 0) join(v1, second, dpp<kDppXor1>(v1), static_cast<int>(dpp<kDppXor1>(static_cast<uint32_t>(second))));
            if (shift > 1) join(v1, second, dpp<kDppXor2>(v1), static_cast<int>(dpp<kDppXor2>(static_cast<uint32_t>(second))));
            if (shift > 2) join(v1, second, dpp<kDppHalfMirror>(v1), static_cast<int>(dpp<kDppHalfMirror>(static_cast<uint32_t>(second))));
            if (shift > 3) join(v1, second, dpp<kDppMirror>(v1), static_cast<int>(dpp<kDppMirror>(static_cast<uint32_t>(second))));
            const int first = lane << shift;   // chunk where group `lane` begins
            const float t = __shfl(score(v1, __int_as_float(second)), first & (LPR - 1), LPR);
            if (first / LPR == j && lane < a.n_group) mine = t;
        }
    } else {
        const int size = a.E / a.n_group;
        for (int g = 0; g < a.n_group; ++g) {
            float v1 = kNegInf, v2 = kNegInf;   // best and second best of the group's elements here
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int e = (j * LPR + lane) * N + i;
                    const float v = e >= g * size && e < (g + 1) * size ? s[j * N + i] : kNegInf;
                    v2 = fmaxf(v2, fminf(v1, v));
                    v1 = fmaxf(v1, v);
                }
            int second = __float_as_int(v2);
            row_exchange<LPR>(v1, second, join);
            if (lane == g) mine = score(v1, __int_as_float(second));
        }
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const float o = __shfl(mine, g, LPR);
        rank += o > mine || (o == mine && g < lane);
    }
    return static_cast<uint32_t>(__ballot(lane < a.n_group && rank < a.topk_group) >> base);
}
// Which elements of the chunk at e0 are in groups that stay (bit i for element i).
template <int N> __device__ __forceinline__ uint32_t chunk_bits(const RouteArgs& a, uint32_t keep, int e0) {
    if (a.group_shift >= 0) return (keep >> (e0 / N >> a.group_shift)) & 1 ? ~0u : 0u;   // past E: no score, no matter
    const int size = a.E / a.n_group;
    uint32_t bits = 0;
    for (int i = 0; i < N; ++i) bits |= (e0 + i < a.E ? (keep >> ((e0 + i) / size)) & 1 : 0) << i;
    return bits;
}

// The exact rounds: k times over, the best (score, id) of the row that comes after the last one chosen.
// Lane n gets the id of slot n.
template <int N, int LPR, int NC> __device__ __forceinline__ int choose_exact(const RouteArgs& a, const float (&s)[NC * N], int lane) {
    float last = __builtin_inff();
    int last_id = -1, pick = -1;
#pragma unroll 1
    for (int n = 0; n < a.k; ++n) {
        float v = kNegInf;
        int id = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = s[j * N + i];
                const int e = (j * LPR + lane) * N + i;
                if ((f < last || (f == last && e > last_id)) && f > v) v = f, id = e;
            }
        row_exchange<LPR>(v, id, better);
        if (lane == n && v > kNegInf) pick = id;
        last = v;
        last_id = id;
    }
    return pick;
}

// A key below this is of an expert out of service (its score -inf), or none.
constexpr uint32_t kLeastKey = 0x00800000u;

// SCORES: bias and group sums are formed on the scores, not on the logits.  (Without bias and groups the order
// is the logits', which keep more of it apart.)  The scores cost one exponential and one division an element:
// 256 experts, top 8, 8 groups and a bias, fp32: 8192 rows 9.0 us (choice by logit 7.4), 65536 rows 34 (28).
template <typename T, int LPR, int NC, RouteMode MODE, bool SCORES>
__global__ __launch_bounds__(256) void route_topk_kernel(RouteArgs a) {
    constexpr int N = Chunk<T>::N, V = NC * N;
    const int lane = threadIdx.x % LPR, E = a.E;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
    const bool live = row < a.T;   // rows past the end run along (the exchanges need every lane) and store nothing
    const T* x = static_cast<const T*>(a.logits) + (live ? row : 0) * a.ld;
    float s[V];   // logits, then what the choice goes by
    {
        u32x4_t raw[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) raw[j] = load_logits<T, MODE>(x + (j * LPR + lane) * N, E - (j * LPR + lane) * N);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float f[N];
            unpack_chunk<T>(raw[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) s[j * N + i] = usable_logit(f[i]) + 0.0f;   // -0 is +0
        }
    }
    float all_max = 0.0f, all_sum = 1.0f;
    if ((SCORES || !a.renorm) && !a.sigmoid) {   // softmax over every expert in service
        float top = kNegInf, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, s[i]);
        all_max = row_max<LPR>(top);
        const float at = all_max > kNegInf ? all_max : 0.0f;   // exp(-inf) = 0 takes care of the rest
#pragma unroll
        for (int i = 0; i < V; ++i) sum += __expf(s[i] - at);
        all_sum = row_sum<LPR>(sum);
    }
    if constexpr (SCORES) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = s[i] > kNegInf ? choice_score(a, s[i], all_max, all_sum) : kNegInf;
    }
    const bool biased = MODE != kPlain && a.bias;
    if (biased) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const int at = (j * LPR + lane) * N + 4 * h;
                float b[4] = {0, 0, 0, 0};
                if (MODE == kWholeChunks) {
                    if (at < E) unpack_chunk<float>(*reinterpret_cast<const u32x4_any_t*>(a.bias + at), b);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i] = at + i < E ? a.bias[at + i] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // -inf stays (plus +inf: NaN); a NaN or -inf score is out of service
                    float& t = s[j * N + 4 * h + i];
                    const float v = t + b[i];
                    t = t > kNegInf && v > kNegInf ? v + 0.0f : kNegInf;
                }
            }
    }
    if (MODE != kPlain && a.n_group > 1) {
        const uint32_t keep = keep_groups<N, LPR, NC>(a, s, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const uint32_t bits = chunk_bits<N>(a, keep, (j * LPR + lane) * N);
#pragma unroll
            for (int i = 0; i < N; ++i) s[j * N + i] = (bits >> i) & 1 ? s[j * N + i] : kNegInf;
        }
    }

    constexpr bool kWide = SCORES || sizeof(T) == 4;   // values with bits where the id goes (16-bit logits: if biased)
    const uint32_t id_mask = a.id_mask;      // 2^b - 1, b bits for an id
    const uint32_t first = id_mask - lane * N;   // the id field of this lane's first element
    uint32_t chosen = 0, last = ~0u;   // lane n: the n-th largest key
    int n = 0;
    for (;;) {   // once, or again with the keys below the last one when a lane's list has run out
        uint32_t best[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = (ordered_bits(s[j + i]) & ~id_mask) | ((first - (j / N * LPR * N + j % N + i)) & id_mask);
            if (n > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = q[i] < last ? q[i] : 0u;
            }
            merge4(best, q);
        }
        const bool full = V > 4 && best[3] >= kLeastKey;   // this lane may hold more than its list
        bool more;
        do {   // with dropped bits one round more than there are slots, and on while the last two agree in the rest
            const uint32_t g = row_max<LPR>(best[0]);
            if (lane == n) chosen = g;
            const bool tied = ((g ^ last) & ~id_mask) == 0 && g >= kLeastKey;
            last = g;
            const bool pop = best[0] == g;   // keys differ, so one lane's
            best[0] = pop ? best[1] : best[0];
            best[1] = pop ? best[2] : best[1];
            best[2] = pop ? best[3] : best[2];
            best[3] = pop ? 0 : best[3];
            ++n;
            more = n < a.k || ((kWide || biased) && (n == a.k || (n < LPR && __ballot(tied) != 0)));
        } while (more && (n < 4 || __ballot(full && best[0] == 0) == 0));
        if (!more) break;
    }
    int pick = lane < a.k && chosen >= kLeastKey ? static_cast<int>(id_mask - (chosen & id_mask)) : -1;
    if (kWide || biased) {   // two neighbours that differ in dropped bits alone
        const uint32_t before = __shfl_up(chosen, 1, LPR);
        const bool tied = lane > 0 && lane < n && chosen >= kLeastKey && ((chosen ^ before) & ~id_mask) == 0;
        if (__ballot(tied) != 0) {
            uint32_t low = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) low |= __float_as_uint(s[i]);
            if (__ballot((low & id_mask) != 0) != 0) {   // else they are equal, and in the right order
                if (n == LPR && __ballot(tied && lane == LPR - 1) != 0) {
                    pick = choose_exact<N, LPR, NC>(a, s, lane);   // more of them than lanes
                } else {   // the n keys hold every candidate: rank them by their scores and ids
                    const bool there = lane < n && chosen >= kLeastKey;
                    const int id = there ? static_cast<int>(id_mask - (chosen & id_mask)) : 0x7fffffff;
                    float v = kNegInf;
                    if (there) {
                        v = usable_logit(to_f32(x[id]));
                        if constexpr (SCORES) v = choice_score(a, v, all_max, all_sum);
                        v = v + (biased ? a.bias[id] : 0.0f) + 0.0f;
                    }
                    int rank = 0;
                    for (int i = 0; i < n; ++i) {
                        const float o = __shfl(v, i, LPR);
                        const int oid = __shfl(id, i, LPR);
                        rank += o > v || (o == v && oid < id);
                    }
                    const int to = (threadIdx.x & 63) / LPR * LPR + (there ? rank : LPR - 1);   // lanes without one push a 0 that says so
                    const int got = __builtin_amdgcn_ds_permute(4 * to, there ? id + 1 : 0);
                    pick = lane < a.k ? got - 1 : -1;
                }
            }
        }
    }
    const bool there = pick >= 0;
    const float l = there ? usable_logit(to_f32(x[pick])) : kNegInf;
    const float p = chosen_weight<LPR>(a, l, there, all_max, all_sum);
    if (live && lane < a.k) {
        a.idx_out[row * a.k + lane] = pick;
        a.w_out[row * a.k + lane] = p * a.scale;
    }
}

// The gradients of the chosen go through a row of LDS, where lane j puts slot j's and every lane then
// reads its chunks' (comparing each element's id with each slot's took 270 instructions a wave, and 65536
// x 250 bf16 logits 22 us, against 13; bound by memory where it is dense: 65536 x 256 fp32 25 us, 5.5 TB/s).
// DENSE: softmax over all, where every expert in service has one.
template <typename T, int LPR, int NC, bool DENSE>
__global__ __launch_bounds__(256) void route_topk_bwd_kernel(RouteArgs a) {
    constexpr int N = Chunk<T>::N, V = NC * N;
    __shared__ __align__(16) float rows[256 / LPR][NC * LPR * N];
    const int lane = threadIdx.x % LPR, E = a.E;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
    const bool live = row < a.T;
    const int64_t r = live ? row : 0;
    const T* x = static_cast<const T*>(a.logits) + r * a.ld;
    float* mine = rows[threadIdx.x / LPR];
    const bool slot = lane < a.k;
    int pick = slot ? a.idx[r * a.k + lane] : -1;
    if (pick < 0 || pick >= E) pick = -1;   // an empty slot, or an id the forward never gives
    const float g0 = slot ? a.dw[r * a.k + lane] * a.scale : 0.0f;
    u32x4_t raw[NC];
    if constexpr (DENSE) {
#pragma unroll
        for (int j = 0; j < NC; ++j) raw[j] = load_logits<T, kAnyRow>(x + (j * LPR + lane) * N, E - (j * LPR + lane) * N);
    }
    const float l = pick >= 0 ? usable_logit(to_f32(x[pick])) : kNegInf;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) *reinterpret_cast<u32x4_t*>(mine + (i * LPR + lane) * 4) = u32x4_t{0, 0, 0, 0};
    const bool there = l > kNegInf;
    const float g = there ? g0 : 0.0f;

    float e[V], all_max = 0.0f, all_sum = 1.0f;
    if constexpr (DENSE) {
        float top = kNegInf, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float f[N];
            unpack_chunk<T>(raw[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                e[j * N + i] = usable_logit(f[i]);
                top = fmaxf(top, e[j * N + i]);
            }
        }
        all_max = row_max<LPR>(top);
        const float at = all_max > kNegInf ? all_max : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = __expf(e[i] - at);
            sum += e[i];
        }
        all_sum = row_sum<LPR>(sum);
    }
    const float p = chosen_weight<LPR>(a, l, there, all_max, all_sum);
    const float q = a.renorm || DENSE ? row_sum<LPR>(p * g) : 0.0f;
    float d = a.renorm ? p * (g - q) : p * g;
    if (a.sigmoid) d *= sigmoid_f32(-l);   // 1 - sigmoid(l)
    wave_sync();   // a row's LDS is its wave's alone
    // Slots that name one expert (the router's never do) are added in slot order: a slot sees from what its place
    // holds whether another one claimed it too, and only then do the slots take turns.
    auto claim = [&](float v) { __hip_atomic_store(mine + pick, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT); };
    if (there) claim(__int_as_float(lane));
    wave_sync();
    const bool shared = there && __float_as_int(__hip_atomic_load(mine + pick, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT)) != lane;
    wave_sync();
    if (__ballot(shared) == 0) {
        if (there) mine[pick] = d;
    } else {
        if (there) claim(0.0f);
        wave_sync();
#pragma unroll 1
        for (int n = 0; n < a.k; ++n) {
            if (there && lane == n) mine[pick] += d;
            wave_sync();
        }
    }
    wave_sync();
    const float share = DENSE && all_sum > 0.0f ? q / all_sum : 0.0f;
    T* dx = static_cast<T*>(a.dlogits) + r * a.ldd;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int e0 = (j * LPR + lane) * N;
        float o[N];
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
            float f[4];
            unpack_chunk<float>(*reinterpret_cast<const u32x4_t*>(mine + e0 + 4 * h), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * h + i] = DENSE ? f[i] - e[j * N + 4 * h + i] * share : f[i];
        }
        if (live) store_chunk<T>(dx + e0, pack_chunk<T>(o), E - e0);
    }
}

namespace {

// Lanes per row and chunks per lane: 16 lanes while the logits fit 32 (fp32) or 64 (16-bit) registers
// and the slots fit the lanes, else a wave.
template <typename T, typename F> void with_row_geometry(int E, int k, F&& f) {
    constexpr int N = Chunk<T>::N;
    const int chunks = (E + N - 1) / N, lanes = k < 16 && chunks <= 128 * 4 / N ? 16 : 64;
    const int per = (chunks + lanes - 1) / lanes;
    auto go = [&](auto lpr) {
        if (per <= 1) f(lpr, std::integral_constant<int, 1>{});
        else if (per <= 2) f(lpr, std::integral_constant<int, 2>{});
        else if constexpr (N == 4) {
            if (per <= 4) f(lpr, std::integral_constant<int, 4>{});
            else if constexpr (lpr() == 16) {
                if (per <= 6) f(lpr, std::integral_constant<int, 6>{});
                else f(lpr, std::integral_constant<int, 8>{});
            }
        } else if constexpr (lpr() == 16) {   // 16-bit rows of up to 512; a wave takes 1024 in two chunks a lane
            if (per <= 3) f(lpr, std::integral_constant<int, 3>{});
            else f(lpr, std::integral_constant<int, 4>{});
        }
    };
    if (lanes == 16) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 64>{});
}

template <typename T, bool BWD> void run_route(const RouteArgs& a, hipStream_t s) {
    with_row_geometry<T>(a.E, a.k, [&](auto lpr, auto nc) {
        constexpr int rows = 256 / decltype(lpr)::value;
        const int grid = static_cast<int>((static_cast<int64_t>(a.T) + rows - 1) / rows);
        if constexpr (BWD) {
            if (!a.renorm && !a.sigmoid) route_topk_bwd_kernel<T, lpr(), nc(), true><<<grid, 256, 0, s>>>(a);
            else route_topk_bwd_kernel<T, lpr(), nc(), false><<<grid, 256, 0, s>>>(a);
        } else if (a.by_score && a.E % Chunk<T>::N != 0) route_topk_kernel<T, lpr(), nc(), kAnyRow, true><<<grid, 256, 0, s>>>(a);
        else if (a.by_score) route_topk_kernel<T, lpr(), nc(), kWholeChunks, true><<<grid, 256, 0, s>>>(a);
        else if (a.E % Chunk<T>::N != 0) route_topk_kernel<T, lpr(), nc(), kAnyRow, false><<<grid, 256, 0, s>>>(a);
        else if (a.bias || a.n_group > 1) route_topk_kernel<T, lpr(), nc(), kWholeChunks, false><<<grid, 256, 0, s>>>(a);
        else route_topk_kernel<T, lpr(), nc(), kPlain, false><<<grid, 256, 0, s>>>(a);
    });
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs& a, int dtype, bool backward, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    auto go = [&](auto t) {
        if (backward) run_route<decltype(t), true>(a, s);
        else run_route<decltype(t), false>(a, s);
    };
    if (dtype == MOE_BF16) go(bf16_t{});
    else if (dtype == MOE_FP16) go(fp16_t{});
    else go(float{});
    return hipGetLastError();
}

}  // namespace moe
