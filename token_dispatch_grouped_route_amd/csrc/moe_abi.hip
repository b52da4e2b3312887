// C ABI of the gfx950 MoE expert-layer library: argument checks, workspace layout and stage
// launches on the caller's stream.  Declarations and the meaning of every argument are in
// include/moe.h.  No entry point allocates, frees, copies to or from the host, or waits.
#include <string.h>

#include <mutex>

#include "moe_block_norm.h"
#include "moe_internal.h"
#include "moe_linear.h"

using namespace moe;

namespace {

constexpr size_t kWsAlign = 256;
constexpr int kMxSlotK = 256;   // K advances 256 per slot in the MX GEMMs (and the FP4 scale layout groups four 64-deep steps)

size_t align_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int32_t check_shape(const moe_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (s->block_m != 32 && s->block_m != 64 && s->block_m != 128 && s->block_m != 256) return MOE_ERR_BLOCK_M;
    if (s->T < 0 || s->H <= 0 || s->I <= 0 || s->E <= 0 || s->EL < 1 || s->EL > 1024 || s->e_lo < 0 ||
        s->k < 1 || s->k > 32)
        return MOE_ERR_SHAPE;
    if (static_cast<int64_t>(s->e_lo) + s->EL > s->E) return MOE_ERR_SHAPE;
    if (s->H % 128 != 0 || s->I % 128 != 0) return MOE_ERR_SHAPE;
    // row and element indices stay far inside int32 / int64 ranges
    const int64_t rows = static_cast<int64_t>(s->T) * s->k + static_cast<int64_t>(s->EL) * s->block_m;
    if (rows > (int64_t(1) << 28) || s->H > (1 << 20) || s->I > (1 << 20)) return MOE_ERR_SHAPE;
    // byte offsets inside one expert's packed weights are 32-bit in the GEMM tile loaders
    if (4 * static_cast<int64_t>(s->I) * s->H >= (int64_t(1) << 31)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int32_t layout_of(const moe_shape* s, moe_ws_layout* L) {
    const int32_t st = check_shape(s);
    if (st != MOE_OK) return st;
    memset(L, 0, sizeof(*L));
    const int64_t BM = s->block_m;
    const int64_t pairs = static_cast<int64_t>(s->T) * s->k;
    const int64_t R = (pairs + static_cast<int64_t>(s->EL) * (BM - 1) + BM - 1) / BM * BM;
    const int64_t rc = route_chunk_for(pairs, s->EL);
    const int64_t chunks = pairs > 0 ? (pairs + rc - 1) / rc : 1;
    const size_t H = s->H, I = s->I, EL = s->EL;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes);
        return o;
    };
    L->rows_capacity = R;
    L->num_blocks = R / BM;
    L->counts = take(4 * EL);
    L->padded_offsets = take(4 * (EL + 1));
    L->row_pair = take(4 * static_cast<size_t>(R));
    L->pair_row = take(4 * static_cast<size_t>(pairs));
    L->tile_expert = take(4 * static_cast<size_t>(R / BM));
    L->tok_nloc = take(4 * static_cast<size_t>(s->T));
    L->meta = take(16);
    L->act = take(2 * static_cast<size_t>(R) * I);
    L->stage = take(4 * static_cast<size_t>(R) * H);
    if (s->train) {
        L->hgu = take(4 * static_cast<size_t>(R) * 2 * I);
        L->dact = take(4 * static_cast<size_t>(R) * I);
        L->dhgu = take(2 * static_cast<size_t>(R) * 2 * I);
        L->dhgu_lo = take(2 * static_cast<size_t>(R) * 2 * I);
        L->wact = take(2 * static_cast<size_t>(R) * I);
        L->wact_lo = take(2 * static_cast<size_t>(R) * I);
    }
    L->zeros = take(2 * (H > 2 * I ? H : 2 * I));
    L->tile_sync = take(4 * static_cast<size_t>(kMaxGrid));
    L->scratch = take(4 * static_cast<size_t>(chunks) * (EL + 1));
    if (s->train) L->dtw_part = take(4 * static_cast<size_t>(R) * (I / 128));
    L->total_bytes = off;
    return MOE_OK;
}

bool is_gfx950() {
    static int cached[64] = {0};   // 0 unknown, 1 yes, 2 no
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return false;
    if (!cached[dev]) {
        hipDeviceProp_t prop;
        bool ok = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
                  strncmp(prop.gcnArchName, "gfx950", 6) == 0;
        cached[dev] = ok ? 1 : 2;
    }
    return cached[dev] == 1;
}

// Shared preamble of every device entry point: shape, workspace size/alignment, device.
int32_t prepare(const moe_shape* s, const void* ws, size_t ws_bytes, bool need_train, Dims* d, Ws* w,
                moe_ws_layout* L) {
    const int32_t st = layout_of(s, L);
    if (st != MOE_OK) return st;
    if (!ws) return MOE_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0) return MOE_ERR_ALIGN;
    if (ws_bytes < L->total_bytes) return MOE_ERR_WORKSPACE;
    if (need_train && !s->train) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    *d = Dims{s->T, s->H, s->I, s->E, s->e_lo, s->EL, s->k, s->block_m};
    char* b = static_cast<char*>(const_cast<void*>(ws));
    w->counts = reinterpret_cast<int32_t*>(b + L->counts);
    w->offsets = reinterpret_cast<int32_t*>(b + L->padded_offsets);
    w->row_pair = reinterpret_cast<int32_t*>(b + L->row_pair);
    w->pair_row = reinterpret_cast<int32_t*>(b + L->pair_row);
    w->tile_expert = reinterpret_cast<int32_t*>(b + L->tile_expert);
    w->tok_nloc = reinterpret_cast<int32_t*>(b + L->tok_nloc);
    w->meta = reinterpret_cast<int32_t*>(b + L->meta);
    w->act = reinterpret_cast<uint16_t*>(b + L->act);
    w->stage = reinterpret_cast<float*>(b + L->stage);
    w->hgu = s->train ? reinterpret_cast<float*>(b + L->hgu) : nullptr;
    w->dact = s->train ? reinterpret_cast<float*>(b + L->dact) : nullptr;
    w->dhgu = s->train ? reinterpret_cast<uint16_t*>(b + L->dhgu) : nullptr;
    w->dhgu_lo = s->train ? reinterpret_cast<uint16_t*>(b + L->dhgu_lo) : nullptr;
    w->wact = s->train ? reinterpret_cast<uint16_t*>(b + L->wact) : nullptr;
    w->wact_lo = s->train ? reinterpret_cast<uint16_t*>(b + L->wact_lo) : nullptr;
    w->dtw_part = s->train ? reinterpret_cast<float*>(b + L->dtw_part) : nullptr;
    w->dtw_cols = s->I / 128;
    const int64_t pairs = static_cast<int64_t>(s->T) * s->k;
    w->route_chunk = route_chunk_for(pairs, s->EL);
    w->num_chunks = static_cast<int32_t>(pairs > 0 ? (pairs + w->route_chunk - 1) / w->route_chunk : 1);
    w->chunk_hist = reinterpret_cast<int32_t*>(b + L->scratch);
    w->chunk_dropped = w->chunk_hist + static_cast<int64_t>(w->num_chunks) * s->EL;
    w->zeros = reinterpret_cast<uint16_t*>(b + L->zeros);
    w->tile_sync = reinterpret_cast<int32_t*>(b + L->tile_sync);
    w->zero_len = s->H > 2 * s->I ? s->H : 2 * s->I;
    w->rows_cap = L->rows_capacity;
    w->num_blocks = static_cast<int32_t>(L->num_blocks);
    return MOE_OK;
}

int32_t launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

}  // namespace

extern "C" {

const char* moe_status_string(int32_t status) {
    switch (status) {
        case MOE_OK: return "ok";
        case MOE_ERR_NULL: return "a required pointer is NULL";
        case MOE_ERR_SHAPE: return "a size is out of the supported range";
        case MOE_ERR_BLOCK_M: return "block_m must be 32, 64, 128 or 256";
        case MOE_ERR_WORKSPACE: return "workspace too small or without the train buffers";
        case MOE_ERR_ALIGN: return "misaligned pointer (16 bytes; workspace 256 bytes)";
        case MOE_ERR_LAUNCH: return "kernel launch failed";
        case MOE_ERR_DEVICE: return "current device is not gfx950 or HIP failed";
        case MOE_ERR_SCRATCH: return "the shape needs more workspace than the fixed scratch of moe_forward_noalloc";
        default: return "unknown status";
    }
}

size_t moe_workspace_bytes(const moe_shape* shape) {
    moe_ws_layout L;
    return layout_of(shape, &L) == MOE_OK ? L.total_bytes : 0;
}

int32_t moe_workspace_layout(const moe_shape* shape, moe_ws_layout* out) {
    if (!out) return MOE_ERR_NULL;
    return layout_of(shape, out);
}

int32_t moe_preferred_block_m(const moe_shape* s) {
    if (!s || s->E <= 0 || s->T < 0 || s->k < 1) return 64;
    // mean rows per expert under uniform routing; a block at most half that keeps the expected
    // padding of each segment (half a block) under about a quarter of its rows
    const double mean = static_cast<double>(s->T) * s->k / s->E;
    if (mean >= 512) return 256;
    if (mean >= 256) return 128;
    return 64;
}

int32_t moe_pack_weights(const moe_shape* shape, const uint16_t* w1, const uint16_t* w2, uint16_t* w1p,
                         uint16_t* w2p, void* stream) {
    const int32_t st = check_shape(shape);
    if (st != MOE_OK) return st;
    if ((w1 == nullptr) != (w1p == nullptr) || (w2 == nullptr) != (w2p == nullptr)) return MOE_ERR_NULL;
    if ((w1 && w1 == w1p) || (w2 && w2 == w2p)) return MOE_ERR_SHAPE;   // not in place
    if (!aligned16(w1) || !aligned16(w2) || !aligned16(w1p) || !aligned16(w2p)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    const Dims d{shape->T, shape->H, shape->I, shape->E, shape->e_lo, shape->EL, shape->k, shape->block_m};
    return launched(launch_pack(d, w1, w2, w1p, w2p, static_cast<hipStream_t>(stream)));
}

int32_t moe_unpack_weights(const moe_shape* shape, const uint16_t* w1p, const uint16_t* w2p, uint16_t* w1,
                           uint16_t* w2, void* stream) {
    const int32_t st = check_shape(shape);
    if (st != MOE_OK) return st;
    if ((w1 == nullptr) != (w1p == nullptr) || (w2 == nullptr) != (w2p == nullptr)) return MOE_ERR_NULL;
    if ((w1 && w1 == w1p) || (w2 && w2 == w2p)) return MOE_ERR_SHAPE;   // not in place
    if (!aligned16(w1) || !aligned16(w2) || !aligned16(w1p) || !aligned16(w2p)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    const Dims d{shape->T, shape->H, shape->I, shape->E, shape->e_lo, shape->EL, shape->k, shape->block_m};
    return launched(launch_unpack(d, w1p, w2p, w1, w2, static_cast<hipStream_t>(stream)));
}

int32_t moe_route_prologue(const moe_shape* shape, const int32_t* topk_idx, void* ws, size_t ws_bytes,
                           void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!topk_idx && shape->T > 0) return MOE_ERR_NULL;
    if (!aligned4(topk_idx)) return MOE_ERR_ALIGN;
    return launched(launch_route(d, topk_idx, w, static_cast<hipStream_t>(stream)));
}

int32_t moe_dispatch_gemm1(const moe_shape* shape, const uint16_t* x, const uint16_t* w1p, void* ws,
                           size_t ws_bytes, uint16_t* act_out, float* hgu_out, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if ((!x && shape->T > 0) || !w1p || (!act_out && !hgu_out)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1p) || !aligned16(act_out) || !aligned16(hgu_out)) return MOE_ERR_ALIGN;
    return launched(launch_gemm1(d, x, w1p, w, act_out, hgu_out, static_cast<hipStream_t>(stream)));
}

int32_t moe_swiglu(const moe_shape* shape, const float* hgu, const void* ws, size_t ws_bytes, uint16_t* act,
                   void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!hgu || !act) return MOE_ERR_NULL;
    if (!aligned16(hgu) || !aligned16(act)) return MOE_ERR_ALIGN;
    return launched(launch_swiglu(d, hgu, w, act, static_cast<hipStream_t>(stream)));
}

int32_t moe_gemm2_combine(const moe_shape* shape, const uint16_t* act, const uint16_t* w2p, const float* topk_w,
                          void* ws, size_t ws_bytes, uint16_t* y, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!act || !w2p || ((!topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(act) || !aligned16(w2p) || !aligned4(topk_w) || !aligned16(y)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_gemm2_combine(d, act, w2p, topk_w, w, y, s);
    if (e == hipSuccess) e = launch_combine_finish(d, w, y, s);
    return launched(e);
}

int32_t moe_forward(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx, const float* topk_w,
                    const uint16_t* w1p, const uint16_t* w2p, void* ws, size_t ws_bytes, uint16_t* y,
                    void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!w1p || !w2p || ((!x || !topk_idx || !topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned4(topk_idx) || !aligned4(topk_w) || !aligned16(w1p) || !aligned16(w2p) ||
        !aligned16(y))
        return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_route(d, topk_idx, w, s);
    if (e == hipSuccess) e = launch_gemm1(d, x, w1p, w, w.act, w.hgu, s);
    if (e == hipSuccess) e = launch_gemm2_combine(d, w.act, w2p, topk_w, w, y, s);
    if (e == hipSuccess) e = launch_combine_finish(d, w, y, s);
    return launched(e);
}

// ---------------------------------------------------------------------------------------------
// Allocation-free forward: the workspace is a fixed device array of this file
// ---------------------------------------------------------------------------------------------
// The array itself.  In host code its name is only a stand-in for the device symbol: the device
// address of each GPU's copy comes from hipGetSymbolAddress, once per device, and only that
// address is passed to kernels.
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's scratch array (looked up on the first call per device).
int32_t scratch_of_current_device(void** out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return MOE_ERR_DEVICE;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return MOE_OK;
}
}  // namespace

int32_t moe_forward_noalloc(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx, const float* topk_w,
                            const uint16_t* w1p, const uint16_t* w2p, uint16_t* y, void* stream) {
    moe_ws_layout L;
    int32_t st = layout_of(shape, &L);
    if (st != MOE_OK) return st;
    if (shape->train) return MOE_ERR_SHAPE;
    if (L.total_bytes > MOE_NOALLOC_SCRATCH_BYTES) return MOE_ERR_SCRATCH;
    if (!w1p || !w2p || ((!x || !topk_idx || !topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned4(topk_idx) || !aligned4(topk_w) || !aligned16(w1p) || !aligned16(w2p) ||
        !aligned16(y))
        return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    void* ws = nullptr;
    st = scratch_of_current_device(&ws);
    if (st != MOE_OK) return st;
    Dims d;
    Ws w;
    st = prepare(shape, ws, MOE_NOALLOC_SCRATCH_BYTES, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    // the same stages as moe_forward; the prologue rewrites every table, the tile counters and the
    // zero row, and the GEMMs write every row they later read, so stale contents of the array
    // from an earlier call do not matter
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_route(d, topk_idx, w, s);
    if (e == hipSuccess) e = launch_gemm1(d, x, w1p, w, w.act, nullptr, s);
    if (e == hipSuccess) e = launch_gemm2_combine(d, w.act, w2p, topk_w, w, y, s);
    if (e == hipSuccess) e = launch_combine_finish(d, w, y, s);
    return launched(e);
}

int32_t moe_bwd_gemm2_dgrad(const moe_shape* shape, const uint16_t* dy, const float* topk_w, const uint16_t* w2p,
                            void* ws, size_t ws_bytes, int32_t fuse_swiglu_bwd, float* dtopk_w, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!w2p || ((!dy || !topk_w) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(dy) || !aligned4(topk_w) || !aligned16(w2p) || !aligned4(dtopk_w)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_dgrad(d, dy, topk_w, w2p, w, fuse_swiglu_bwd != 0, dtopk_w != nullptr, s);
    if (e == hipSuccess && dtopk_w) e = launch_dtopk_w_finish(d, w, dtopk_w, s);
    return launched(e);
}

int32_t moe_bwd_gemm1_dgrad_combine(const moe_shape* shape, const uint16_t* w1p, void* ws, size_t ws_bytes,
                                    uint16_t* dx, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!w1p || (!dx && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(w1p) || !aligned16(dx)) return MOE_ERR_ALIGN;
    return launched(launch_dgrad1(d, w1p, w, dx, static_cast<hipStream_t>(stream)));
}

int32_t moe_swiglu_bwd(const moe_shape* shape, void* ws, size_t ws_bytes, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    return launched(launch_swiglu_bwd(d, w, static_cast<hipStream_t>(stream)));
}

int32_t moe_wgrad2(const moe_shape* shape, const uint16_t* dy, void* ws, size_t ws_bytes, uint16_t* dw2p,
                   void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!dw2p || (!dy && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(dy) || !aligned16(dw2p)) return MOE_ERR_ALIGN;
    return launched(launch_wgrad2(d, dy, w, dw2p, static_cast<hipStream_t>(stream)));
}

int32_t moe_wgrad1(const moe_shape* shape, const uint16_t* x, void* ws, size_t ws_bytes, uint16_t* dw1p,
                   void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!dw1p || (!x && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(dw1p)) return MOE_ERR_ALIGN;
    return launched(launch_wgrad1(d, x, w, dw1p, static_cast<hipStream_t>(stream)));
}

int32_t moe_backward(const moe_shape* shape, const uint16_t* x, const uint16_t* dy, const float* topk_w,
                     const uint16_t* w1p, const uint16_t* w2p, void* ws, size_t ws_bytes, uint16_t* dw1p,
                     uint16_t* dw2p, uint16_t* dx, float* dtopk_w, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, true, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!w2p || !dw1p || !dw2p || ((!x || !dy || !topk_w) && shape->T > 0)) return MOE_ERR_NULL;
    if (dx && !w1p) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(dy) || !aligned4(topk_w) || !aligned16(w1p) || !aligned16(w2p) ||
        !aligned16(dw1p) || !aligned16(dw2p) || !aligned16(dx) || !aligned4(dtopk_w))
        return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_dgrad(d, dy, topk_w, w2p, w, 1, dtopk_w != nullptr, s);
    if (e == hipSuccess && dtopk_w) e = launch_dtopk_w_finish(d, w, dtopk_w, s);
    if (e == hipSuccess) e = launch_wgrad2(d, dy, w, dw2p, s);
    if (e == hipSuccess) e = launch_wgrad1(d, x, w, dw1p, s);
    if (e == hipSuccess && dx) e = launch_dgrad1(d, w1p, w, dx, s);
    return launched(e);
}

int32_t moe_mx_cast_fp8(int64_t rows, int32_t cols, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                        void* stream) {
    if (rows < 0 || cols <= 0 || cols % 32 != 0) return MOE_ERR_SHAPE;
    if (rows > 0 && (!x || !codes || !scales)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(codes)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    return launched(launch_mx_cast_fp8(rows, cols, x, codes, scales, static_cast<hipStream_t>(stream)));
}

static bool mx_shape_ok(const moe_shape* shape) {
    return shape->H % kMxSlotK == 0 && shape->I % kMxSlotK == 0;
}

int32_t moe_mx_pack_weights(const moe_shape* shape, const uint16_t* w1, const uint16_t* w2, uint8_t* w1q,
                            uint8_t* w1s, uint8_t* w2q, uint8_t* w2s, void* stream) {
    const int32_t st = check_shape(shape);
    if (st != MOE_OK) return st;
    if (!mx_shape_ok(shape)) return MOE_ERR_SHAPE;
    if ((w1 == nullptr) != (w1q == nullptr) || (w1 == nullptr) != (w1s == nullptr) ||
        (w2 == nullptr) != (w2q == nullptr) || (w2 == nullptr) != (w2s == nullptr))
        return MOE_ERR_NULL;
    if (!aligned16(w1) || !aligned16(w2) || !aligned16(w1q) || !aligned16(w2q)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    const Dims d{shape->T, shape->H, shape->I, shape->E, shape->e_lo, shape->EL, shape->k, shape->block_m};
    return launched(launch_mx_pack(d, w1, w2, w1q, w1s, w2q, w2s, static_cast<hipStream_t>(stream)));
}

int32_t moe_mx_dispatch_gemm1(const moe_shape* shape, const uint8_t* xq, const uint8_t* xs, const uint8_t* w1q,
                              const uint8_t* w1s, float clamp, void* ws, size_t ws_bytes, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!mx_shape_ok(shape)) return MOE_ERR_SHAPE;
    if (!w1q || !w1s || ((!xq || !xs) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(xq) || !aligned4(xs) || !aligned16(w1q)) return MOE_ERR_ALIGN;
    return launched(launch_mx_gemm1(d, xq, xs, w1q, w1s, w, clamp, static_cast<hipStream_t>(stream)));
}

int32_t moe_mx_gemm2_combine(const moe_shape* shape, const uint8_t* w2q, const uint8_t* w2s, const float* topk_w,
                             void* ws, size_t ws_bytes, uint16_t* y, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!mx_shape_ok(shape)) return MOE_ERR_SHAPE;
    if (!w2q || !w2s || ((!topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(w2q) || !aligned4(topk_w) || !aligned16(y)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_mx_gemm2(d, w2q, w2s, topk_w, w, y, s);
    if (e == hipSuccess) e = launch_combine_finish(d, w, y, s);
    return launched(e);
}

int32_t moe_forward_mx(const moe_shape* shape, const uint8_t* xq, const uint8_t* xs, const int32_t* topk_idx,
                       const float* topk_w, const uint8_t* w1q, const uint8_t* w1s, const uint8_t* w2q,
                       const uint8_t* w2s, float clamp, void* ws, size_t ws_bytes, uint16_t* y, void* stream) {
    Dims d;
    Ws w;
    moe_ws_layout L;
    int32_t st = prepare(shape, ws, ws_bytes, false, &d, &w, &L);
    if (st != MOE_OK) return st;
    if (!mx_shape_ok(shape)) return MOE_ERR_SHAPE;
    if (!w1q || !w1s || !w2q || !w2s || ((!xq || !xs || !topk_idx || !topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(xq) || !aligned4(xs) || !aligned4(topk_idx) || !aligned4(topk_w) || !aligned16(w1q) ||
        !aligned16(w2q) || !aligned16(y))
        return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = launch_route(d, topk_idx, w, s);
    if (e == hipSuccess) e = launch_mx_gemm1(d, xq, xs, w1q, w1s, w, clamp, s);
    if (e == hipSuccess) e = launch_mx_gemm2(d, w2q, w2s, topk_w, w, y, s);
    if (e == hipSuccess) e = launch_combine_finish(d, w, y, s);
    return launched(e);
}

// ---------------------------------------------------------------------------------------------
// Operators around the expert layer: row norm, router, 4-bit products
// ---------------------------------------------------------------------------------------------
namespace {
constexpr int kW4MaxK = 32768;
constexpr int64_t kW4MaxLd = 1 << 23;   // 16 rows of x stay within 32-bit byte offsets
constexpr int kRouteMaxT = 1 << 25;        // a grid has fewer than 2^32 threads: 64 per token,
constexpr int64_t kW4MaxTiles = 1 << 23;   // and 256 per 16 x 16 tile of moe_w4_linear's y
bool is_dtype(int32_t t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
bool is_16bit(int32_t t) { return t == MOE_BF16 || t == MOE_FP16; }
int elem_bytes(int32_t t) { return t == MOE_FP32 ? 4 : 2; }
bool aligned_to(const void* p, int32_t t) { return (reinterpret_cast<uintptr_t>(p) & (elem_bytes(t) - 1u)) == 0; }

int32_t check_norm(int32_t kind, int32_t dtype, int32_t wdtype, int64_t rows, int32_t cols) {
    if ((kind != MOE_LAYER_NORM && kind != MOE_RMS_NORM) || !is_dtype(dtype) || (wdtype != dtype && wdtype != MOE_FP32)) return MOE_ERR_SHAPE;
    if (rows < 0 || rows > (int64_t(1) << 40) || cols < 1 || cols > kNormMaxCols) return MOE_ERR_SHAPE;
    return MOE_OK;
}
// A leading dimension: at least the row, and row offsets that stay inside int64.
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) { return ld < cols || (rows > 1 && ld > (int64_t(1) << 61) / rows); }
}  // namespace

size_t moe_norm_workspace_bytes(int32_t dtype, int64_t rows, int32_t cols) {
    if (check_norm(MOE_LAYER_NORM, dtype, dtype, rows, cols) != MOE_OK) return 0;
    const int64_t rms = norm_bwd_slots(rows, cols, elem_bytes(dtype), false), layer = norm_bwd_slots(rows, cols, elem_bytes(dtype), true);
    const size_t part = align_up(static_cast<size_t>(rms > layer ? rms : layer) * cols * 4);
    return 2 * (part > 0 ? part : kWsAlign);
}

int32_t moe_norm_forward(int32_t kind, int32_t dtype, int32_t wdtype, int64_t rows, int32_t cols, const void* x, int64_t ldx,
                         const void* weight, const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                         void* stream) {
    const int32_t st = check_norm(kind, dtype, wdtype, rows, cols);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f) || bad_ld(ldx, rows, cols) || bad_ld(ldy, rows, cols) || (kind == MOE_RMS_NORM && bias)) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !y) return MOE_ERR_NULL;
    if (x == y) return MOE_ERR_SHAPE;   // not in place
    if (!aligned_to(x, dtype) || !aligned_to(y, dtype) || !aligned_to(weight, wdtype) || !aligned_to(bias, wdtype) || !aligned4(mean) || !aligned4(rstd))
        return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    NormArgs a = {};
    a.rows = rows, a.cols = cols, a.x = x, a.ldx = ldx, a.weight = weight, a.bias = bias, a.eps = eps, a.y = y, a.ldy = ldy;
    a.mean = mean, a.rstd = rstd;
    return launched(launch_norm_fwd(a, dtype, wdtype, kind == MOE_LAYER_NORM, static_cast<hipStream_t>(stream)));
}

int32_t moe_norm_backward(int32_t kind, int32_t dtype, int32_t wdtype, int64_t rows, int32_t cols, const void* dy, int64_t lddy,
                          const void* x, int64_t ldx, const void* weight, const float* mean, const float* rstd, void* dx,
                          int64_t lddx, void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream) {
    const int32_t st = check_norm(kind, dtype, wdtype, rows, cols);
    if (st != MOE_OK) return st;
    const bool layer = kind == MOE_LAYER_NORM;
    if (bad_ld(ldx, rows, cols) || bad_ld(lddy, rows, cols) || (dx && bad_ld(lddx, rows, cols)) || (!layer && dbias)) return MOE_ERR_SHAPE;
    if (rows > 0 && !dx && !dweight && !dbias) return MOE_ERR_NULL;   // an empty dx may be NULL
    if (rows > 0 && (!x || !dy || !rstd || (layer && !mean))) return MOE_ERR_NULL;
    if (rows > 0 && (dx == x || dx == dy)) return MOE_ERR_SHAPE;   // not in place
    if (!aligned_to(x, dtype) || !aligned_to(dy, dtype) || !aligned_to(dx, dtype) || !aligned_to(weight, wdtype) || !aligned_to(dweight, wdtype) ||
        !aligned_to(dbias, wdtype) || !aligned4(mean) || !aligned4(rstd))
        return MOE_ERR_ALIGN;
    NormArgs a = {};
    if (dweight || dbias) {
        if (!ws) return MOE_ERR_NULL;
        if ((reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0) return MOE_ERR_ALIGN;
        const size_t need = moe_norm_workspace_bytes(dtype, rows, cols);
        if (ws_bytes < need) return MOE_ERR_WORKSPACE;
        if (dweight) a.part_w = static_cast<float*>(ws);
        if (dbias) a.part_b = reinterpret_cast<float*>(static_cast<char*>(ws) + need / 2);
    } else if (rows == 0) {
        return MOE_OK;
    }
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    a.rows = rows, a.cols = cols, a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.weight = weight, a.y = dx, a.lddx = lddx;
    a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd), a.dweight = dweight, a.dbias = dbias;
    return launched(launch_norm_bwd(a, dtype, wdtype, layer, static_cast<hipStream_t>(stream)));
}

namespace {
int32_t check_route(int32_t dtype, int32_t T, int32_t E, int32_t k, int64_t ld, int32_t score) {
    if (!is_dtype(dtype) || T < 0 || T > kRouteMaxT || E < 1 || E > 1024 || k < 1 || k > 32 || k > E || bad_ld(ld, T, E)) return MOE_ERR_SHAPE;
    const int32_t kind = score & ~MOE_CHOOSE_BY_SCORE;
    return kind == MOE_SOFTMAX || kind == MOE_SIGMOID ? MOE_OK : MOE_ERR_SHAPE;
}
}  // namespace

int32_t moe_route_topk(int32_t dtype, int32_t T, int32_t E, int32_t k, const void* logits, int64_t ld, const float* bias,
                       int32_t score, int32_t renormalize, int32_t n_group, int32_t topk_group, float scale,
                       int32_t* topk_idx, float* topk_w, void* stream) {
    const int32_t st = check_route(dtype, T, E, k, ld, score);
    if (st != MOE_OK) return st;
    if (n_group < 1 || n_group > 16 || E % n_group != 0 || topk_group < 1 || topk_group > n_group) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w) return MOE_ERR_NULL;
    if (!aligned_to(logits, dtype) || !aligned4(bias) || !aligned4(topk_idx) || !aligned4(topk_w)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    RouteArgs a = {};
    a.T = T, a.E = E, a.k = k, a.n_group = n_group, a.topk_group = topk_group, a.sigmoid = (score & ~MOE_CHOOSE_BY_SCORE) == MOE_SIGMOID;
    a.by_score = (score & MOE_CHOOSE_BY_SCORE) != 0 && (bias || n_group > 1);
    const int per_chunk = 16 / elem_bytes(dtype), chunks = E / n_group / per_chunk;
    a.group_shift = E / n_group % per_chunk == 0 && chunks <= 16 && (chunks & (chunks - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(chunks)) : -1;
    a.id_mask = 1;
    while (a.id_mask + 1 < static_cast<uint32_t>(E)) a.id_mask = 2 * a.id_mask + 1;
    a.renorm = renormalize != 0, a.scale = scale, a.logits = logits, a.ld = ld, a.bias = bias, a.idx_out = topk_idx, a.w_out = topk_w;
    return launched(launch_route_topk(a, dtype, false, static_cast<hipStream_t>(stream)));
}

int32_t moe_route_topk_backward(int32_t dtype, int32_t T, int32_t E, int32_t k, const void* logits, int64_t ld,
                                const int32_t* topk_idx, const float* dtopk_w, int32_t score, int32_t renormalize, float scale,
                                void* dlogits, int64_t ldd, void* stream) {
    const int32_t st = check_route(dtype, T, E, k, ld, score);
    if (st != MOE_OK) return st;
    if (bad_ld(ldd, T, E)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !dtopk_w || !dlogits) return MOE_ERR_NULL;
    if (logits == dlogits) return MOE_ERR_SHAPE;   // not in place
    if (!aligned_to(logits, dtype) || !aligned_to(dlogits, dtype) || !aligned4(topk_idx) || !aligned4(dtopk_w)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    RouteArgs a = {};
    a.T = T, a.E = E, a.k = k, a.sigmoid = (score & ~MOE_CHOOSE_BY_SCORE) == MOE_SIGMOID, a.renorm = renormalize != 0, a.scale = scale;
    a.logits = logits, a.ld = ld, a.idx = topk_idx, a.dw = dtopk_w, a.dlogits = dlogits, a.ldd = ldd;
    return launched(launch_route_topk(a, dtype, true, static_cast<hipStream_t>(stream)));
}

namespace {
// log2 of a group size that divides K, or -1.
int group_shift(int32_t group, int32_t K) {
    if (group < 32 || (group & (group - 1)) != 0 || K <= 0 || K > kW4MaxK || K % group != 0) return -1;
    return __builtin_ctz(static_cast<unsigned>(group));
}
// Byte offsets of the act and stage rows of moe_forward_w4, and the total; false for a bad shape.
bool w4_layout(const moe_shape* s, size_t* stage, size_t* total) {
    if (check_shape(s) != MOE_OK || s->train || static_cast<int64_t>(s->T) * s->k > kW4MaxPairs) return false;
    const size_t pairs = static_cast<size_t>(s->T) * s->k;
    *stage = align_up(pairs * s->I * 2);
    *total = *stage + align_up(pairs * s->H * 4) + kWsAlign;
    return true;
}
}  // namespace

int32_t moe_w4_quantize(int32_t wdtype, int32_t dtype, int32_t E, int32_t K, int32_t N, int32_t group, const void* w,
                        uint8_t* codes, void* scales, uint8_t* zeros, void* stream) {
    if (!is_dtype(wdtype) || !is_16bit(dtype) || E < 1 || E > 65535 || N < 1 || N > (1 << 28) || group_shift(group, K) < 0) return MOE_ERR_SHAPE;
    if (!w || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned_to(w, wdtype) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    return launched(launch_w4_quantize(wdtype, dtype, E, K, N, group, w, codes, scales, zeros, static_cast<hipStream_t>(stream)));
}

int32_t moe_w4_linear(int32_t dtype, int32_t M, int32_t N, int32_t K, int32_t group, const void* x, int64_t ldx,
                      const uint8_t* codes, const void* scales, const uint8_t* zeros, void* y, int64_t ldy, void* stream) {
    const int gshift = group_shift(group, K);
    if (!is_16bit(dtype) || M < 0 || M > (1 << 20) || N < 1 || N > (1 << 28) || gshift < 0 || bad_ld(ldx, M, K) || bad_ld(ldy, M, N)) return MOE_ERR_SHAPE;
    if (ldx > kW4MaxLd || (static_cast<int64_t>(M) + 15) / 16 * ((static_cast<int64_t>(N) + 15) / 16) > kW4MaxTiles) return MOE_ERR_SHAPE;
    if (M == 0) return MOE_OK;
    if (!x || !codes || !scales || !y) return MOE_ERR_NULL;
    if (!aligned16(x) || ldx % 8 != 0 || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned_to(y, dtype)) return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    const W4Linear a{M, N, K, gshift, x, ldx, ldy, codes, scales, zeros, y};
    return launched(launch_w4_linear(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t moe_w4_workspace_bytes(const moe_shape* shape) {
    size_t stage, total;
    return w4_layout(shape, &stage, &total) ? total : 0;
}

int32_t moe_forward_w4(const moe_shape* shape, int32_t dtype, int32_t group, const void* x, const int32_t* topk_idx,
                       const float* topk_w, const uint8_t* w1, const void* s1, const uint8_t* z1, const uint8_t* w2,
                       const void* s2, const uint8_t* z2, void* ws, size_t ws_bytes, void* y, void* stream) {
    const int32_t st = check_shape(shape);
    if (st != MOE_OK) return st;
    size_t stage, total;
    if (!w4_layout(shape, &stage, &total) || !is_16bit(dtype) || group_shift(group, shape->H) < 0 || group_shift(group, shape->I) < 0)
        return MOE_ERR_SHAPE;
    if (!w1 || !s1 || !w2 || !s2 || !ws || ((!x || !topk_idx || !topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1) || !aligned16(s1) || !aligned16(z1) || !aligned16(w2) || !aligned16(s2) || !aligned16(z2) ||
        !aligned16(y) || !aligned4(topk_idx) || !aligned4(topk_w) || (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0)
        return MOE_ERR_ALIGN;
    if (ws_bytes < total) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    W4Experts a = {};
    a.T = shape->T, a.H = shape->H, a.I = shape->I, a.e_lo = shape->e_lo, a.EL = shape->EL, a.k = shape->k;
    a.gshift = group_shift(group, shape->H), a.x = x, a.topk_idx = topk_idx, a.topk_w = topk_w;
    a.w1 = w1, a.s1 = s1, a.z1 = z1, a.w2 = w2, a.s2 = s2, a.z2 = z2;
    a.act = ws, a.stage = reinterpret_cast<float*>(static_cast<char*>(ws) + stage), a.y = y;
    return launched(launch_w4_forward(a, dtype, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------------------------
// Dense operators of a block: linear map
// ---------------------------------------------------------------------------------------------
namespace {
constexpr int64_t kLinearMaxTiles = 1 << 23;   // of 128 x 128, 256 threads each: grids stay below 2^32 threads
int64_t tiles128(int64_t m, int64_t n) { return (m + 127) / 128 * ((n + 127) / 128); }
struct LinearSizes {
    int64_t M, N, K, C;   // C: columns of the weight and of z
    bool ok;
};
LinearSizes linear_sizes(int32_t act, int32_t M, int32_t N, int32_t K, bool backward) {
    LinearSizes s{M, N, K, act == MOE_ACT_SWIGLU ? 2 * static_cast<int64_t>(N) : N, false};
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU || M < 0 || M > (1 << 24) || N < 1 || N > (1 << 20) || K < 1 || K > (1 << 20)) return s;
    s.ok = tiles128(s.M, s.C) <= kLinearMaxTiles && (!backward || (tiles128(s.M, s.K) <= kLinearMaxTiles && tiles128(s.K, s.C) <= kLinearMaxTiles));
    return s;
}
int64_t dz_row(int64_t C) { return (C + 7) / 8 * 8; }
// The backward's workspace: dz, then the partial rows of db, then the products' partial sums and padded copies.
size_t dz_bytes(const LinearSizes& s) { return align_up(static_cast<size_t>(s.M) * dz_row(s.C) * 2); }
size_t db_bytes(const LinearSizes& s) { return align_up(static_cast<size_t>(slope_slots(s.M, s.N)) * s.C * 4); }
size_t larger(size_t a, size_t b) { return a > b ? a : b; }
// Room for the products' padded copies, whatever the weight's layout: of x and w in the forward (not of paired rows), of w for dx and x for dw.
size_t forward_pad_bytes(const LinearSizes& s) {
    const int64_t x = padded_elements(s.M, s.K), by_row = s.C != s.N ? 0 : padded_elements(s.K, s.C), by_column = padded_elements(s.C, s.K);
    return larger(product_pad_bytes(s.M, s.C, s.K, x, by_row), product_pad_bytes(s.M, s.C, s.K, x, by_column));
}
size_t backward_pad_bytes(const LinearSizes& s) {
    const size_t dx = larger(product_pad_bytes(s.M, s.K, s.C, 0, padded_elements(s.K, s.C)), product_pad_bytes(s.M, s.K, s.C, 0, padded_elements(s.C, s.K)));
    return larger(dx, larger(product_pad_bytes(s.K, s.C, s.M, padded_elements(s.M, s.K), 0), product_pad_bytes(s.C, s.K, s.M, 0, padded_elements(s.M, s.K))));
}
size_t forward_part_bytes(const LinearSizes& s) { return align_up(product_part_bytes(s.M, s.C, s.K)); }
size_t backward_part_bytes(const LinearSizes& s) { return align_up(larger(product_part_bytes(s.M, s.K, s.C), product_part_bytes(s.K, s.C, s.M))); }
}  // namespace

size_t moe_linear_workspace_bytes(int32_t act, int32_t M, int32_t N, int32_t K, int32_t backward) {
    const LinearSizes s = linear_sizes(act, M, N, K, backward != 0);
    if (!s.ok) return 0;
    if (!backward) return forward_part_bytes(s) + forward_pad_bytes(s) + kWsAlign;
    return dz_bytes(s) + db_bytes(s) + backward_part_bytes(s) + backward_pad_bytes(s) + kWsAlign;
}

int32_t moe_linear_forward(int32_t dtype, int32_t bdtype, int32_t odtype, int32_t act, int32_t M, int32_t N, int32_t K,
                           const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t w_by_column, const void* bias,
                           const void* residual, int64_t ldr, void* y, int64_t ldy, void* z, int64_t ldz, void* ws,
                           size_t ws_bytes, void* stream) {
    const LinearSizes s = linear_sizes(act, M, N, K, false);
    if (!s.ok || !is_16bit(dtype) || (bdtype != dtype && bdtype != MOE_FP32) || (odtype != dtype && odtype != MOE_FP32)) return MOE_ERR_SHAPE;
    if (bad_ld(ldx, M, K) || bad_ld(ldw, w_by_column ? s.C : K, w_by_column ? K : s.C) || bad_ld(ldy, M, N) || (residual && bad_ld(ldr, M, N)) ||
        (z && bad_ld(ldz, M, s.C)))
        return MOE_ERR_SHAPE;
    if (M == 0) return MOE_OK;
    const size_t part = forward_part_bytes(s), pad = forward_pad_bytes(s), need = part + pad + kWsAlign;
    if (!x || !w || !y || (!ws && need > kWsAlign)) return MOE_ERR_NULL;
    if (y == x || y == w || z == x || z == w || z == y || (residual == y && ldr != ldy) || (residual && residual == z)) return MOE_ERR_SHAPE;
    if (!aligned_to(x, dtype) || !aligned_to(w, dtype) || !aligned_to(bias, bdtype) || !aligned_to(residual, odtype) || !aligned_to(y, odtype) ||
        !aligned_to(z, dtype) || (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0)
        return MOE_ERR_ALIGN;
    if (need > kWsAlign && ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    Product g = {};
    g.M = M, g.N = static_cast<int32_t>(s.C), g.K = K, g.b_strided = !w_by_column;
    g.a = static_cast<const uint16_t*>(x), g.lda = ldx, g.b = static_cast<const uint16_t*>(w), g.ldb = ldw;
    g.act = act, g.out_cols = N, g.bias = bias, g.residual = residual, g.ldr = ldr, g.y = y, g.ldy = ldy, g.z = z, g.ldz = ldz;
    g.bias_f32 = bdtype == MOE_FP32, g.y_f32 = odtype == MOE_FP32;
    return launched(launch_product(g, dtype, ws, static_cast<char*>(ws) + part, pad, static_cast<hipStream_t>(stream)));
}

int32_t moe_linear_backward(int32_t dtype, int32_t bdtype, int32_t odtype, int32_t act, int32_t M, int32_t N, int32_t K,
                            const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                            int32_t w_by_column, const void* z, int64_t ldz, void* dx, int64_t lddx, void* dw, int64_t lddw,
                            void* dbias, void* ws, size_t ws_bytes, void* stream) {
    const LinearSizes s = linear_sizes(act, M, N, K, true);
    if (!s.ok || !is_16bit(dtype) || (bdtype != dtype && bdtype != MOE_FP32) || (odtype != dtype && odtype != MOE_FP32)) return MOE_ERR_SHAPE;
    const int64_t wr = w_by_column ? s.C : K, wc = w_by_column ? K : s.C;
    if (bad_ld(lddy, M, N) || (dw && (bad_ld(ldx, M, K) || bad_ld(lddw, wr, wc))) || (dx && (bad_ld(ldw, wr, wc) || bad_ld(lddx, M, K))) ||
        (act != MOE_ACT_NONE && bad_ld(ldz, M, s.C)))
        return MOE_ERR_SHAPE;
    if (M == 0 && !dw && !dbias) return MOE_OK;   // an empty dx may be NULL
    if (!dx && !dw && !dbias) return MOE_ERR_NULL;
    if (!ws || (M > 0 && (!dy || (dw && !x) || (dx && !w) || (act != MOE_ACT_NONE && !z)))) return MOE_ERR_NULL;
    const void* in[4] = {dy, x, w, z};
    for (const void* p : in)
        if (p && (p == dx || p == dw || p == dbias)) return MOE_ERR_SHAPE;   // not in place
    if (!aligned_to(dy, odtype) || !aligned_to(x, dtype) || !aligned_to(w, dtype) || !aligned_to(z, dtype) || !aligned_to(dx, dtype) || !aligned_to(dw, dtype) ||
        !aligned_to(dbias, bdtype) || (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0)
        return MOE_ERR_ALIGN;
    const size_t part_bytes = backward_part_bytes(s), pad_room = backward_pad_bytes(s);
    if (ws_bytes < dz_bytes(s) + db_bytes(s) + part_bytes + pad_room + kWsAlign) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* at = static_cast<char*>(ws);
    // else dy is dz; rows that are not whole chunks are copied where that pays for a product
    const int64_t dz_copy = padded_elements(s.M, s.C);
    const bool own_dz = ((dx || dw) && (act != MOE_ACT_NONE || odtype == MOE_FP32)) ||
                        (dx && dz_copy && product_pad_bytes(s.M, s.K, s.C, dz_copy, w_by_column ? padded_elements(s.C, s.K) : padded_elements(s.K, s.C)) > 0) ||
                        (dw && dz_copy && product_pad_bytes(s.K, s.C, s.M, padded_elements(s.M, s.K), dz_copy) > 0);
    LinearSlope l = {};
    l.M = M, l.N = N, l.act = act, l.dy = dy, l.lddy = lddy, l.z = z, l.ldz = ldz, l.dy_f32 = odtype == MOE_FP32;
    l.dz = own_dz ? at : nullptr, l.lddz = dz_row(s.C);
    if (dbias) l.part = reinterpret_cast<float*>(at + dz_bytes(s));
    if (own_dz || dbias) {
        const int32_t e = launched(launch_linear_slope(l, dtype, bdtype, dbias, st));
        if (e != MOE_OK) return e;
    }
    char *part = at + dz_bytes(s) + db_bytes(s), *pad = part + part_bytes;
    const uint16_t* dz = static_cast<const uint16_t*>(own_dz ? at : dy);
    const int64_t lddz = own_dz ? l.lddz : lddy;
    Product g = {};
    if (dx) {
        g.M = M, g.N = K, g.K = static_cast<int32_t>(s.C), g.a = dz, g.lda = lddz, g.b = static_cast<const uint16_t*>(w), g.ldb = ldw;
        g.a_padded = own_dz, g.b_strided = w_by_column != 0, g.out_cols = K, g.y = dx, g.ldy = lddx;
        const int32_t e = launched(launch_product(g, dtype, part, pad, pad_room, st));
        if (e != MOE_OK) return e;
    }
    if (dw) {   // by column: the product's transpose, dz^T x
        const uint16_t* xs = static_cast<const uint16_t*>(x);
        g = {};
        g.a_strided = g.b_strided = true, g.K = M, g.y = dw, g.ldy = lddw;
        g.M = static_cast<int32_t>(wr), g.N = g.out_cols = static_cast<int32_t>(wc);
        g.a = w_by_column ? dz : xs, g.lda = w_by_column ? lddz : ldx;
        g.a_padded = own_dz && w_by_column, g.b_padded = own_dz && !w_by_column;
        g.b = w_by_column ? xs : dz, g.ldb = w_by_column ? ldx : lddz;
        const int32_t e = launched(launch_product(g, dtype, part, pad, pad_room, st));
        if (e != MOE_OK) return e;
    }
    return MOE_OK;
}

// ---------------------------------------------------------------------------------------------
// Block norm
// ---------------------------------------------------------------------------------------------
namespace {
// The checks that both directions share; fills the formula's part of `a`.
int32_t check_block_norm(BlockNorm* a, int32_t kind, int32_t parts, int32_t dtype, int32_t sdtype, int32_t wdtype, int64_t rows, int32_t cols, int64_t ldb,
                         float x_scale, float scale, const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows,
                         const void* pre_weight, const void* pre_bias) {
    const int32_t st = check_norm(kind, dtype, wdtype, rows, cols);
    if (st != MOE_OK) return st;
    if ((sdtype != dtype && sdtype != MOE_FP32) || (parts & ~(MOE_POST_NORM | MOE_PRE_NORM)) != 0) return MOE_ERR_SHAPE;
    const bool post = (parts & MOE_POST_NORM) != 0, pre = (parts & MOE_PRE_NORM) != 0, layer = kind == MOE_LAYER_NORM;
    if ((!post && (post_weight || post_bias)) || (!pre && (pre_weight || pre_bias)) || (!layer && (post_bias || pre_bias))) return MOE_ERR_SHAPE;
    if ((gate != nullptr) != (gate_rows > 0) || gate_rows < 0 || (gate_rows > 0 && rows % gate_rows != 0)) return MOE_ERR_SHAPE;
    if (!aligned_to(post_weight, wdtype) || !aligned_to(post_bias, wdtype) || !aligned_to(gate, wdtype) || !aligned_to(pre_weight, wdtype) ||
        !aligned_to(pre_bias, wdtype))
        return MOE_ERR_ALIGN;
    *a = {};
    a->rows = rows, a->cols = cols, a->layer = layer, a->post = post, a->pre = pre, a->x_scale = x_scale, a->scale = scale;
    a->b_f32 = dtype == MOE_FP32, a->s_f32 = sdtype == MOE_FP32, a->w_f32 = wdtype == MOE_FP32;
    a->post_weight = post_weight, a->post_bias = post_bias, a->gate = gate, a->pre_weight = pre_weight, a->pre_bias = pre_bias, a->ldb = ldb;
    a->gate_share = gate_rows > 0 ? rows / gate_rows : rows;
    return MOE_OK;
}
}  // namespace

int32_t moe_block_norm_forward(int32_t kind, int32_t parts, int32_t dtype, int32_t sdtype, int32_t wdtype, int64_t rows, int32_t cols,
                               const void* x, int64_t ldx, const void* b, int64_t ldb, float x_scale, float scale,
                               const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows,
                               const void* pre_weight, const void* pre_bias, float eps, void* r, int64_t ldr, void* n, int64_t ldn,
                               float* post_mean, float* post_rstd, float* pre_mean, float* pre_rstd, void* stream) {
    BlockNorm a;
    const int32_t st = check_block_norm(&a, kind, parts, dtype, sdtype, wdtype, rows, cols, ldb, x_scale, scale, post_weight, post_bias, gate, gate_rows,
                                        pre_weight, pre_bias);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f) || bad_ld(ldx, rows, cols) || bad_ld(ldb, rows, cols) || bad_ld(ldr, rows, cols) || (a.pre ? bad_ld(ldn, rows, cols) : n != nullptr))
        return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !b || !r || (a.pre && !n)) return MOE_ERR_NULL;
    if (r == b || n == b || n == x || n == r || (r == x && ldr != ldx)) return MOE_ERR_SHAPE;
    if (!aligned_to(x, sdtype) || !aligned_to(r, sdtype) || !aligned_to(b, dtype) || !aligned_to(n, dtype) || !aligned4(post_mean) || !aligned4(post_rstd) ||
        !aligned4(pre_mean) || !aligned4(pre_rstd))
        return MOE_ERR_ALIGN;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    a.eps = eps, a.x = x, a.ldx = ldx, a.b = b, a.r = r, a.ldr = ldr, a.n = n, a.ldn = ldn;
    a.post_mean = post_mean, a.post_rstd = post_rstd, a.pre_mean = pre_mean, a.pre_rstd = pre_rstd;
    return launched(launch_block_norm_fwd(a, dtype, sdtype, wdtype, static_cast<hipStream_t>(stream)));
}

size_t moe_block_norm_workspace_bytes(int32_t dtype, int64_t rows, int32_t cols, int64_t gate_rows) {
    if (check_norm(MOE_LAYER_NORM, dtype, dtype, rows, cols) != MOE_OK || gate_rows < 0 || (gate_rows > 0 && rows % gate_rows != 0)) return 0;
    return block_norm_bwd_bytes(rows, cols, gate_rows, elem_bytes(dtype));
}

int32_t moe_block_norm_backward(int32_t kind, int32_t parts, int32_t dtype, int32_t sdtype, int32_t wdtype, int64_t rows, int32_t cols,
                                const void* dr, int64_t lddr, const void* dn, int64_t lddn, const void* r, int64_t ldr, const void* b,
                                int64_t ldb, float x_scale, float scale, const void* post_weight, const void* post_bias, const void* gate,
                                int64_t gate_rows, const void* pre_weight, const float* post_mean, const float* post_rstd,
                                const float* pre_mean, const float* pre_rstd, void* dx, int64_t lddx, void* db, int64_t lddb, void* dgate,
                                void* dpost_weight, void* dpost_bias, void* dpre_weight, void* dpre_bias, void* ws, size_t ws_bytes,
                                void* stream) {
    BlockNorm a;
    const int32_t st = check_block_norm(&a, kind, parts, dtype, sdtype, wdtype, rows, cols, ldb, x_scale, scale, post_weight, post_bias, gate, gate_rows,
                                        pre_weight, nullptr);
    if (st != MOE_OK) return st;
    const bool needs_b = a.post || dgate;
    if ((dr && bad_ld(lddr, rows, cols)) || (dn && (bad_ld(lddn, rows, cols) || bad_ld(ldr, rows, cols))) || (needs_b && bad_ld(ldb, rows, cols)) ||
        (dx && bad_ld(lddx, rows, cols)) || (db && bad_ld(lddb, rows, cols)))
        return MOE_ERR_SHAPE;
    if ((!a.pre && (dn || dpre_weight || dpre_bias)) || (!a.post && (dpost_weight || dpost_bias)) || (!a.layer && (dpre_bias || dpost_bias)) || (dgate && !gate))
        return MOE_ERR_SHAPE;
    const bool vectors = dgate || dpost_weight || dpost_bias || dpre_weight || dpre_bias;
    if (rows == 0 && !vectors) return MOE_OK;   // empty dx and db may be NULL
    if (!dx && !db && !vectors) return MOE_ERR_NULL;
    if (!ws || (rows > 0 && ((!dr && !dn) || (dn && (!r || !pre_rstd || (a.layer && !pre_mean))) || (needs_b && !b) ||
                             (a.post && (!post_rstd || (a.layer && !post_mean))))))
        return MOE_ERR_NULL;
    const void* in[4] = {dr, dn, r, b};
    for (const void* p : in)
        if (p && (p == dx || p == db)) return MOE_ERR_SHAPE;   // not in place
    if (dx && dx == db) return MOE_ERR_SHAPE;
    if (!aligned_to(dr, sdtype) || !aligned_to(dx, sdtype) || !aligned_to(r, sdtype) || !aligned_to(dn, dtype) || !aligned_to(b, dtype) || !aligned_to(db, dtype) ||
        !aligned_to(dgate, wdtype) || !aligned_to(dpost_weight, wdtype) || !aligned_to(dpost_bias, wdtype) || !aligned_to(dpre_weight, wdtype) ||
        !aligned_to(dpre_bias, wdtype) || !aligned4(post_mean) || !aligned4(post_rstd) || !aligned4(pre_mean) || !aligned4(pre_rstd) ||
        (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0)
        return MOE_ERR_ALIGN;
    if (ws_bytes < moe_block_norm_workspace_bytes(dtype, rows, cols, gate_rows)) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    if (rows == 0) a.gate_share = gate_rows;
    a.dr = dr, a.lddr = lddr, a.dn = dn, a.lddn = lddn, a.r = const_cast<void*>(dn ? r : nullptr), a.ldr = ldr, a.b = needs_b ? b : nullptr;
    a.post_mean = const_cast<float*>(post_mean), a.post_rstd = const_cast<float*>(post_rstd);
    a.pre_mean = const_cast<float*>(pre_mean), a.pre_rstd = const_cast<float*>(pre_rstd);
    a.dx = dx, a.lddx = lddx, a.db = db, a.lddb = lddb, a.dgate = dgate, a.dpost_weight = dpost_weight, a.dpost_bias = dpost_bias;
    a.dpre_weight = dpre_weight, a.dpre_bias = dpre_bias, a.ws = static_cast<float*>(ws);
    return launched(launch_block_norm_bwd(a, dtype, wdtype, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------------------------
// Expert layer for few tokens
// ---------------------------------------------------------------------------------------------
namespace {
// Byte offset of the stage rows and the total; false for a bad shape.
bool few_layout(const moe_shape* s, size_t* stage, size_t* total) {
    if (check_shape(s) != MOE_OK || s->train || static_cast<int64_t>(s->T) * s->k > kFewMaxPairs || s->H > kFewMaxK || s->I > kFewMaxK) return false;
    const size_t pairs = static_cast<size_t>(s->T) * s->k;
    *stage = align_up(pairs * s->I * 2);
    *total = *stage + align_up(pairs * s->H * 4) + kWsAlign;
    return true;
}
}  // namespace

size_t moe_few_workspace_bytes(const moe_shape* shape) {
    size_t stage, total;
    return few_layout(shape, &stage, &total) ? total : 0;
}

int32_t moe_forward_few(const moe_shape* shape, const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint16_t* w1p,
                        const uint16_t* w2p, void* ws, size_t ws_bytes, uint16_t* y, void* stream) {
    const int32_t st = check_shape(shape);
    if (st != MOE_OK) return st;
    size_t stage, total;
    if (!few_layout(shape, &stage, &total)) return MOE_ERR_SHAPE;
    if (!w1p || !w2p || !ws || ((!x || !topk_idx || !topk_w || !y) && shape->T > 0)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(w1p) || !aligned16(w2p) || !aligned16(y) || !aligned4(topk_idx) || !aligned4(topk_w) ||
        (reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0)
        return MOE_ERR_ALIGN;
    if (ws_bytes < total) return MOE_ERR_WORKSPACE;
    if (!is_gfx950()) return MOE_ERR_DEVICE;
    FewExperts a = {};
    a.T = shape->T, a.H = shape->H, a.I = shape->I, a.e_lo = shape->e_lo, a.EL = shape->EL, a.k = shape->k;
    a.x = x, a.topk_idx = topk_idx, a.topk_w = topk_w, a.w1 = w1p, a.w2 = w2p, a.y = y;
    a.act = static_cast<uint16_t*>(ws), a.stage = reinterpret_cast<float*>(static_cast<char*>(ws) + stage);
    return launched(launch_few(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
