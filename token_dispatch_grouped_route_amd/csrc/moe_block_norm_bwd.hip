// Block norm, backward: moe_block_norm.h has the formulas.  Rows of 8 to 8192 elements are held in registers, in one
// launch (moe_block_norm_row.h); others in two launches over the rows:
//
//   rows      the four means that N' takes for the two norms, from one pass over each row.  The post norm's follow from sums
//             that do not wait for the pre norm's: with g = dn w2, q = gate w1, t = dr + rstd2 (g - m0 - N(r) m1),
//             sum q t u = sum q u dr + rstd2 (sum q u g - m0 sum q u - m1 sum q u N(r))  for u = 1 and u = N(b).
//   columns   with those, every gradient is a function of its element: dx and db are written, and the vectors' gradients
//             summed over a run of rows in registers, joined in LDS; a last launch adds the runs in a fixed order.
#include "moe_block_norm.h"
#include "moe_columns.h"
#include "moe_linear.h"

namespace moe {
namespace {

// Eight columns of one row, past the row's end 0.
template <typename T> struct RowIn {
    float dr[8], dn[8], h2[8], h1[8];   // h2 = N(r), h1 = N(b) or b
};
template <typename T>
__device__ __forceinline__ void read_row(const BlockNorm& a, int64_t row, int c, RowIn<T>& in, const float (&stat)[4]) {
    const int valid = a.cols - c;
#pragma unroll
    for (int i = 0; i < 8; ++i) in.dr[i] = in.dn[i] = in.h2[i] = in.h1[i] = 0.0f;
    if (a.dr) load8<T>(a.dr, row * a.lddr + c, a.s_f32, valid, in.dr);
    if (a.dn) {
        load8<T>(a.dn, row * a.lddn + c, a.b_f32, valid, in.dn);
        load8<T>(a.r, row * a.ldr + c, a.s_f32, valid, in.h2);
#pragma unroll
        for (int i = 0; i < 8; ++i) in.h2[i] = i < valid ? (in.h2[i] - stat[2]) * stat[3] : 0.0f;
    }
    if (a.b) {
        load8<T>(a.b, row * a.ldb + c, a.b_f32, valid, in.h1);
        if (a.post) {
#pragma unroll
            for (int i = 0; i < 8; ++i) in.h1[i] = i < valid ? (in.h1[i] - stat[0]) * stat[1] : 0.0f;
        }
    }
}
template <typename T> __device__ __forceinline__ void read_vector(const void* p, int64_t at, bool f32, int valid, float none, float (&f)[8]) {
    if (p) {
        load8<T>(p, at, f32, valid, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = none;
    }
}
__device__ __forceinline__ void read_stats(const BlockNorm& a, int64_t row, float (&stat)[4]) {
    stat[0] = a.post && a.layer ? a.post_mean[row] : 0.0f;
    stat[1] = a.post ? a.post_rstd[row] : 1.0f;
    stat[2] = a.dn && a.layer ? a.pre_mean[row] : 0.0f;
    stat[3] = a.dn ? a.pre_rstd[row] : 1.0f;
}

// means[row] = the pre norm's sum g / C (layer) and sum (g N(r)) / C, the post norm's alike.
template <typename T> __global__ __launch_bounds__(256) void block_norm_rows_kernel(BlockNorm a, float4* means) {
    __shared__ float lds[10 * 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float stat[4], sum[10] = {};
        read_stats(a, row, stat);
        const int64_t gate = a.gate ? row / a.gate_share * a.cols : 0;
        for (int c = threadIdx.x * 8; c < a.cols; c += 256 * 8) {
            RowIn<T> in;
            float w2[8], w1[8], gt[8];
            read_row(a, row, c, in, stat);
            read_vector<T>(a.pre_weight, c, a.w_f32, a.cols - c, 1.0f, w2);
            read_vector<T>(a.post_weight, c, a.w_f32, a.cols - c, 1.0f, w1);
            read_vector<T>(a.gate, gate + c, a.w_f32, a.cols - c, 1.0f, gt);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float g = in.dn[i] * w2[i], q = c + i < a.cols ? gt[i] * w1[i] : 0.0f, qh = q * in.h1[i];
                sum[0] += g;
                sum[1] += g * in.h2[i];
                sum[2] += qh * in.dr[i];
                sum[3] += qh * g;
                sum[4] += qh;
                sum[5] += qh * in.h2[i];
                sum[6] += q * in.dr[i];
                sum[7] += q * g;
                sum[8] += q;
                sum[9] += q * in.h2[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) sum[i] = wave_sum(sum[i]);
        __syncthreads();   // the last row's sums have been read
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 10; ++i) lds[i * 4 + wave] = sum[i];
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const float inv = 1.0f / static_cast<float>(a.cols);
            float t[10];
#pragma unroll
            for (int i = 0; i < 10; ++i) t[i] = lds[i * 4] + lds[i * 4 + 1] + lds[i * 4 + 2] + lds[i * 4 + 3];
            const float m0 = a.layer ? t[0] * inv : 0.0f, m1 = t[1] * inv;
            const float p1 = t[2] + stat[3] * (t[3] - m0 * t[4] - m1 * t[5]), p0 = t[6] + stat[3] * (t[7] - m0 * t[8] - m1 * t[9]);
            means[row] = float4{m0, m1, a.layer ? a.scale * p0 * inv : 0.0f, a.scale * p1 * inv};
        }
    }
}

template <typename T> __global__ __launch_bounds__(256) void block_norm_columns_kernel(BlockNorm a, const float4* means, Runs runs, Partials part) {
    __shared__ __align__(16) float join[4][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 512 + 8 * lane, valid = a.cols - c;
    int64_t r0, r1;
    runs.range(blockIdx.y, a.rows, r0, r1);
    float w2[8], w1[8], c1[8], gt[8];
    read_vector<T>(a.pre_weight, c, a.w_f32, valid, 1.0f, w2);
    read_vector<T>(a.post_weight, c, a.w_f32, valid, 1.0f, w1);
    read_vector<T>(a.post_bias, c, a.w_f32, valid, 0.0f, c1);
    float s_w2[8] = {}, s_c2[8] = {}, s_w1[8] = {}, s_c1[8] = {}, s_g[8] = {};
    // adds the waves' sums of these columns and writes them to a row of `to`, or in the vectors' type to row `row` of the gate's gradient
    auto leave = [&](float* to, const float (&sum)[8], int64_t row = -1) {
        if (!to && row < 0) return;   // the same for the whole launch
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) join[wave][8 * lane + i] = sum[i];
        __syncthreads();
        for (int i = threadIdx.x; i < 512; i += 256)
            if (const int at = static_cast<int>(blockIdx.x) * 512 + i; at < a.cols) {
                const float v = join[0][i] + join[1][i] + join[2][i] + join[3][i];
                if (to) to[at] = v;
                else if (a.w_f32) static_cast<float*>(a.dgate)[row * a.cols + at] = v;
                else static_cast<T*>(a.dgate)[row * a.cols + at] = from_f32<T>(v);
            }
    };
    for (int64_t g0 = r0; g0 < r1;) {   // the rows of one row of the gate
        const int64_t gate = g0 / runs.share, g1 = min(r1, (gate + 1) * runs.share);
        read_vector<T>(a.gate, gate * a.cols + c, a.w_f32, valid, 1.0f, gt);
        if (valid > 0) {
            for (int64_t row = g0 + wave; row < g1; row += 4) {
                float stat[4], o[8];
                read_stats(a, row, stat);
                const float4 m = means[row];
                RowIn<T> in;
                read_row(a, row, c, in, stat);
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t[i] = in.dr[i];
                    if (a.dn) {
                        t[i] += stat[3] * (in.dn[i] * w2[i] - m.x - in.h2[i] * m.y);
                        s_w2[i] += in.dn[i] * in.h2[i];
                        s_c2[i] += in.dn[i];
                    }
                    o[i] = a.x_scale * t[i];
                }
                if (a.dx) store8<T>(a.dx, row * a.lddx + c, a.s_f32, valid, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = a.post ? in.h1[i] * w1[i] + c1[i] : in.h1[i], u = a.scale * t[i], dp = u * gt[i];
                    s_g[i] += u * p;
                    s_w1[i] += dp * in.h1[i];
                    s_c1[i] += dp;
                    o[i] = a.post ? stat[1] * (dp * w1[i] - m.z - in.h1[i] * m.w) : dp;
                }
                if (a.db) store8<T>(a.db, row * a.lddb + c, a.b_f32, valid, o);
            }
        }
        leave(part.gate ? part.gate + (gate * runs.per_gate + blockIdx.y % runs.per_gate) * a.cols : nullptr, s_g, a.dgate && !part.gate ? gate : -1);
#pragma unroll
        for (int i = 0; i < 8; ++i) s_g[i] = 0.0f;
        g0 = g1;
    }
    auto row_of = [&](float* p) { return p ? p + static_cast<int64_t>(blockIdx.y) * a.cols : nullptr; };
    leave(row_of(part.pre_weight), s_w2);
    leave(row_of(part.pre_bias), s_c2);
    leave(row_of(part.post_weight), s_w1);
    leave(row_of(part.post_bias), s_c1);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
Runs columns_runs(int64_t rows, int cols, int64_t gate_rows) { return runs_of(rows, gate_rows, 1024 / ((cols + 511) / 512), 16); }   // four workgroups a CU

}  // namespace

Runs runs_of(int64_t rows, int64_t gate_rows, int64_t target, int64_t least) {
    const int64_t even = (rows + target - 1) / target, length = even < least ? least : even, share = gate_rows > 0 ? rows / gate_rows : rows;
    Runs r;
    r.share = share;
    if (share >= length) {   // a gate row's rows in per_gate runs
        r.per_gate = (share + length - 1) / length;
        r.length = (share + r.per_gate - 1) / r.per_gate;
        r.per_gate = (share + r.length - 1) / r.length;
        if (r.per_gate == 1) r.runs = (rows + r.length - 1) / r.length;
        else r.runs = rows / share * r.per_gate;
    } else {   // whole gate rows
        r.per_gate = 1;
        r.length = length / share * share;
        r.runs = (rows + r.length - 1) / r.length;
    }
    return r;
}


// Rows that a team holds in registers, 8 to 8192 elements: two workgroups of 256 threads a CU or one of 512, at least four
// rows each.
Runs block_norm_row_runs(int64_t rows, int cols, int64_t gate_rows, int elem_bytes) {
    if (cols < 8 || cols > 8192 || rows == 0) return Runs{};
    return runs_of(rows, gate_rows, norm_chunks(cols, elem_bytes) > 256 ? 256 : 512, norm_chunks(cols, elem_bytes) > 64 ? 4 : 16);
}

// The rows' means where two launches share the work, then five sets of partial sums.
static size_t bytes_of(const Runs& r, bool means, int64_t rows, int cols, int64_t gate_rows) {
    return (means ? align256(rows * 16) : 0) + 4 * align256(r.runs * cols * 4) + align256((gate_rows > 0 && r.per_gate > 1 ? gate_rows * r.per_gate : 0) * cols * 4);
}
size_t block_norm_bwd_bytes(int64_t rows, int cols, int64_t gate_rows, int elem_bytes) {
    if (rows == 0) return 256;
    const Runs row = block_norm_row_runs(rows, cols, gate_rows, elem_bytes);
    return row.runs ? bytes_of(row, false, rows, cols, gate_rows) : bytes_of(columns_runs(rows, cols, gate_rows), true, rows, cols, gate_rows);
}

hipError_t launch_block_norm_bwd(const BlockNorm& a, int dtype, int wdtype, hipStream_t s) {
    const int64_t gate_rows = a.gate && a.rows > 0 ? a.rows / a.gate_share : 0;
    char* at = reinterpret_cast<char*>(a.ws);
    auto take = [&](bool wanted, size_t bytes) {
        float* p = wanted ? reinterpret_cast<float*>(at) : nullptr;
        if (wanted) at += align256(bytes);
        return p;
    };
    ColumnSums sums = {};
    sums.cols = a.cols;
    Partials part = {};
    auto job = [&](int i, float* p, void* out, int64_t groups, int64_t slots) { sums.sum[i] = {p, out}, sums.groups[i] = groups, sums.slots[i] = slots; };
    if (a.rows > 0) {
        Runs runs = block_norm_row_runs(a.rows, a.cols, gate_rows, dtype == MOE_FP32 ? 4 : 2);
        const bool row = runs.runs > 0;
        if (!row) runs = columns_runs(a.rows, a.cols, gate_rows);
        float4* means = reinterpret_cast<float4*>(take(!row, a.rows * 16));
        const size_t bytes = static_cast<size_t>(runs.runs) * a.cols * 4;
        part.pre_weight = take(a.dpre_weight, bytes);
        part.pre_bias = take(a.dpre_bias, bytes);
        part.post_weight = take(a.dpost_weight, bytes);
        part.post_bias = take(a.dpost_bias, bytes);
        part.gate = take(a.dgate && runs.per_gate > 1, static_cast<size_t>(gate_rows) * runs.per_gate * a.cols * 4);
        hipError_t e;
        if (row) {
            e = dtype == MOE_BF16 ? launch_block_norm_row_bf16(a, runs, part, s) : dtype == MOE_FP16 ? launch_block_norm_row_fp16(a, runs, part, s) : launch_block_norm_row_fp32(a, runs, part, s);
        } else {
            auto go = [&](auto t) {
                using T = decltype(t);
                block_norm_rows_kernel<T><<<static_cast<unsigned>(a.rows < 4096 ? a.rows : 4096), 256, 0, s>>>(a, means);
                block_norm_columns_kernel<T><<<dim3((a.cols + 511) / 512, static_cast<unsigned>(runs.runs)), 256, 0, s>>>(a, means, runs, part);
            };
            if (dtype == MOE_FP16) go(fp16_t{});
            else go(bf16_t{});   // also for fp32, whose vectors are fp32: no element has the 16-bit type
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
        job(0, part.pre_weight, a.dpre_weight, 1, runs.runs);
        job(1, part.pre_bias, a.dpre_bias, 1, runs.runs);
        job(2, part.post_weight, a.dpost_weight, 1, runs.runs);
        job(3, part.post_bias, a.dpost_bias, 1, runs.runs);
        job(4, part.gate, a.dgate, gate_rows, runs.per_gate);
    } else {   // no rows: zeros
        float* any = a.ws;
        job(0, a.dpre_weight ? any : nullptr, a.dpre_weight, 1, 0);
        job(1, a.dpre_bias ? any : nullptr, a.dpre_bias, 1, 0);
        job(2, a.dpost_weight ? any : nullptr, a.dpost_weight, 1, 0);
        job(3, a.dpost_bias ? any : nullptr, a.dpost_bias, 1, 0);
        job(4, a.dgate ? any : nullptr, a.dgate, a.gate_share, 0);   // gate_share holds the gate's rows here
    }
    bool any = false;
    for (const ColumnSum& c : sums.sum) any = any || c.part;
    if (any) {
        if (wdtype == MOE_FP32) launch_column_sums<float>(sums, s);
        else if (wdtype == MOE_BF16) launch_column_sums<bf16_t>(sums, s);
        else launch_column_sums<fp16_t>(sums, s);
    }
    return hipGetLastError();
}

}  // namespace moe
