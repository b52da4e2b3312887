// Top-k router: expert ids and weights from router logits, and the gradient back to the logits.
//
//   l = min(logit, largest finite); an expert whose logit is NaN or -inf is out of service
//   s = l + bias; with expert groups, the groups of the largest (best + second best s) stay
//   ids = the k largest s, descending, ties to the lower id; -1 (weight 0) where none is left
//   softmax:  p_j = exp(l_j - m) / sum over the chosen (renormalised) or over all in service
//   sigmoid:  p_j = 1 / (1 + exp(-l_j)), over the sum of the chosen (renormalised) or as it is
//   weight = scale p;  backward, with g = scale dweight and q = sum over the chosen of p g:
//   softmax:  dl_j = p_j (g_j - q) renormalised, else dl_e = p_e ([e chosen] g_e - q) for every e
//   sigmoid:  dl_j = p_j (1 - sigmoid(l_j)) (g_j - [renormalised] q)
//
// A row belongs to LPR lanes, each with V = 16-byte chunks of its logits in registers: 16 lanes
// (four rows a wave; every exchange between the lanes of a row is a DPP step) or 64.
#include <type_traits>

#include "moe_vec.h"

namespace moe {

constexpr float kNegInf = -__builtin_inff();
constexpr float kF32Max = 3.402823466e38f;

// l of a logit: NaN and -inf -> -inf, +inf -> the largest finite number.
__device__ __forceinline__ float usable_logit(float v) { return v > kNegInf ? fminf(v, kF32Max) : kNegInf; }

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

template <typename T, int LPR, int NC>
__global__ __launch_bounds__(256) void route_topk_kernel(RouteArgs a) {
    constexpr int N = Chunk<T>::N, V = NC * N;
    const int lane = threadIdx.x % LPR, E = a.E;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
    const bool live = row < a.T;   // rows past the end run along (the exchanges need every lane) and store nothing
    const T* x = static_cast<const T*>(a.logits) + (live ? row : 0) * a.ld;

    float s[V];
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int e0 = (j * LPR + lane) * N, valid = E - e0;
        float f[N];
        unpack_chunk<T>(load_chunk<T>(x + e0, valid), f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float l = i < valid ? usable_logit(f[i]) : kNegInf;
            top = fmaxf(top, l);
            if (a.bias && i < valid) {
                const float b = l + a.bias[e0 + i];
                l = l > kNegInf && b > kNegInf ? b : kNegInf;
            }
            s[j * N + i] = l;
        }
    }
    float all_max = 0.0f, all_sum = 1.0f;
    if (!a.renorm && !a.sigmoid) {   // softmax over every expert in service
        all_max = row_max<LPR>(top);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int e0 = (j * LPR + lane) * N, valid = E - e0;
            float f[N];
            if (a.bias) unpack_chunk<T>(load_chunk<T>(x + e0, valid), f);   // the scores carry the bias: read again
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float l = a.bias ? (i < valid ? usable_logit(f[i]) : kNegInf) : s[j * N + i];
                sum += l > kNegInf ? __expf(l - all_max) : 0.0f;
            }
        }
        all_sum = row_sum<LPR>(sum);
    }
    if (a.n_group > 1) {
        const int size = E / a.n_group;
        float mine = kNegInf;   // lane g: the score of group g
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
            row_exchange<LPR>(v1, second, [](float& p, int& q, float op, int oq) {
                q = __float_as_int(fmaxf(fmaxf(__int_as_float(q), __int_as_float(oq)), fminf(p, op)));
                p = fmaxf(p, op);
            });
            v2 = __int_as_float(second);
            if (lane == g) mine = v2 > kNegInf ? v1 + v2 : v1;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const float o = __shfl(mine, g, LPR);
            rank += o > mine || (o == mine && g < lane);
        }
        const uint64_t keep = __ballot(lane < a.n_group && rank < a.topk_group) >> ((threadIdx.x & 63) / LPR * LPR);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = (j * LPR + lane) * N + i;
                if (e < E && !((keep >> (e / size)) & 1)) s[j * N + i] = kNegInf;
            }
    }
    int pick = -1;   // lane j: the id of slot j
    for (int n = 0; n < a.k; ++n) {
        float v = kNegInf;
        int id = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (s[j * N + i] > v) v = s[j * N + i], id = (j * LPR + lane) * N + i;
        row_exchange<LPR>(v, id, better);
        if (lane == n && v > kNegInf) pick = id;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (id == (j * LPR + lane) * N + i) s[j * N + i] = kNegInf;
    }
    const bool there = pick >= 0;
    const float l = there ? usable_logit(to_f32(x[pick])) : kNegInf;
    const float p = chosen_weight<LPR>(a, l, there, all_max, all_sum);
    if (live && lane < a.k) {
        a.idx_out[row * a.k + lane] = pick;
        a.w_out[row * a.k + lane] = p * a.scale;
    }
}

template <typename T, int LPR, int NC>
__global__ __launch_bounds__(256) void route_topk_bwd_kernel(RouteArgs a) {
    constexpr int N = Chunk<T>::N;
    const int lane = threadIdx.x % LPR, E = a.E;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
    const bool live = row < a.T;
    const int64_t r = live ? row : 0;
    const T* x = static_cast<const T*>(a.logits) + r * a.ld;
    const bool slot = lane < a.k;
    int pick = slot ? a.idx[r * a.k + lane] : -1;
    if (pick < 0 || pick >= E) pick = -1;   // an empty slot, or an id the forward never gives
    const float l = pick >= 0 ? usable_logit(to_f32(x[pick])) : kNegInf;
    const bool there = l > kNegInf;
    const float g = there ? a.dw[r * a.k + lane] * a.scale : 0.0f;

    float out[NC][N];
    float all_max = 0.0f, all_sum = 1.0f;
    const bool dense = !a.renorm && !a.sigmoid;
    if (dense) {
        float top = kNegInf;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int e0 = (j * LPR + lane) * N, valid = E - e0;
            unpack_chunk<T>(load_chunk<T>(x + e0, valid), out[j]);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                out[j][i] = i < valid ? usable_logit(out[j][i]) : kNegInf;
                top = fmaxf(top, out[j][i]);
            }
        }
        all_max = row_max<LPR>(top);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                out[j][i] = out[j][i] > kNegInf ? __expf(out[j][i] - all_max) : 0.0f;
                sum += out[j][i];
            }
        all_sum = row_sum<LPR>(sum);
    }
    const float p = chosen_weight<LPR>(a, l, there, all_max, all_sum);
    const float q = a.renorm || dense ? row_sum<LPR>(p * g) : 0.0f;
    float d = a.renorm ? p * (g - q) : p * g;
    if (a.sigmoid) d *= sigmoid_f32(-l);   // 1 - sigmoid(l)
    if (!there) d = 0.0f;
    const float share = dense && all_sum > 0.0f ? q / all_sum : 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) out[j][i] = dense ? -out[j][i] * share : 0.0f;
    for (int n = 0; n < a.k; ++n) {
        const int id = __shfl(pick, n, LPR);
        const float dn = __shfl(d, n, LPR);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (id == (j * LPR + lane) * N + i) out[j][i] += dn;
    }
    if (!live) return;
    T* dx = static_cast<T*>(a.dlogits) + row * a.ldd;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int e0 = (j * LPR + lane) * N;
        store_chunk<T>(dx + e0, pack_chunk<T>(out[j]), E - e0);
    }
}

namespace {

// Lanes per row and chunks per lane: 16 lanes while the logits fit 32 (fp32) or 64 (16-bit) registers
// and the slots fit the lanes, else a wave.
template <typename T, typename F> void with_row_geometry(int E, int k, F&& f) {
    constexpr int N = Chunk<T>::N;
    const int chunks = (E + N - 1) / N, lanes = k <= 16 && chunks <= 128 * 4 / N ? 16 : 64;
    const int per = (chunks + lanes - 1) / lanes;
    auto go = [&](auto lpr) {
        if (per <= 1) f(lpr, std::integral_constant<int, 1>{});
        else if (per <= 2) f(lpr, std::integral_constant<int, 2>{});
        else if (per <= 3) f(lpr, std::integral_constant<int, 3>{});
        else if constexpr (N == 4) {   // 16-bit rows end at 3 or 4 chunks per lane
            if (per <= 4) f(lpr, std::integral_constant<int, 4>{});
            else if constexpr (lpr() == 16) {
                if (per <= 6) f(lpr, std::integral_constant<int, 6>{});
                else f(lpr, std::integral_constant<int, 8>{});
            }
        } else {
            f(lpr, std::integral_constant<int, 4>{});
        }
    };
    if (lanes == 16) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 64>{});
}

template <typename T, bool BWD> void run_route(const RouteArgs& a, hipStream_t s) {
    with_row_geometry<T>(a.E, a.k, [&](auto lpr, auto nc) {
        constexpr int rows = 256 / decltype(lpr)::value;
        const int grid = static_cast<int>((static_cast<int64_t>(a.T) + rows - 1) / rows);
        if constexpr (BWD) route_topk_bwd_kernel<T, lpr(), nc()><<<grid, 256, 0, s>>>(a);
        else route_topk_kernel<T, lpr(), nc()><<<grid, 256, 0, s>>>(a);
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
