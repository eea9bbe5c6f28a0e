// C ABI of the MoE expert layer: argument validation, device check, dispatch.
// Validation runs before any HIP call, so argument errors are reported (and nothing is
// enqueued) even on a machine without a GPU.
#include <atomic>
#include <mutex>

#include "common.hpp"
#include "launch.hpp"

namespace {

constexpr int32_t kVersion = 100;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// gfx950 check, cached per device id (immutable once written).
std::atomic<int> g_dev_state[64];   // 0 unknown, 1 usable, 2 unusable

int32_t check_device() {
    int count = 0;
    if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
        (void)hipGetLastError();
        return MOE_ERR_NO_DEVICE;
    }
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return MOE_ERR_NO_DEVICE;
    if (dev < 0 || dev >= 64) return MOE_ERR_NO_DEVICE;
    int st = g_dev_state[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_NO_DEVICE;
        const char* a = prop.gcnArchName;
        st = (a[0] == 'g' && a[1] == 'f' && a[2] == 'x' && a[3] == '9' && a[4] == '5' &&
              a[5] == '0') ? 1 : 2;
        g_dev_state[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? MOE_OK : MOE_ERR_NO_DEVICE;
}

inline int32_t hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

struct GemmPlan {
    int path;
    int split;
    size_t ws;
};

GemmPlan plan_gemm(int32_t R, int32_t E, int32_t K, int32_t N, int32_t wtype, int32_t act,
                   const moe_gemm_opts* opts) {
    GemmPlan pl;
    const int forced_path = opts ? opts->path : MOE_PATH_AUTO;
    const int forced_split = opts ? opts->split_k : 0;
    pl.path = moe::gemm_choose_path(R, E, K, N, wtype, act, forced_path);
    pl.split = 1;
    if (pl.path == MOE_PATH_STREAM) pl.split = moe::gemm_choose_split(R, E, K, N, wtype, act, forced_split);
    pl.ws = 0;                                   // no kernel of either path needs one
    return pl;
}

int32_t validate_gemm(const uint16_t* a, const int32_t* offsets, int32_t R, int32_t E, int32_t K,
                      int32_t N, const void* w, const uint16_t* scales, int32_t wtype,
                      int32_t group, int32_t act, uint16_t* out, const moe_gemm_opts* opts) {
    if (R < 0 || E < 1 || E > MOE_MAX_EXPERTS || K <= 0 || N <= 0) return MOE_ERR_INVALID;
    if (wtype < MOE_W_INT4 || wtype > MOE_W_FP16) return MOE_ERR_INVALID;
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID;
    if (group != 0 && group != 128) return MOE_ERR_UNSUPPORTED;
    if (wtype == MOE_W_FP16 && group != 0) return MOE_ERR_UNSUPPORTED;
    if (K % 128 != 0 || N % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (act == MOE_ACT_SWIGLU && N % 32 != 0) return MOE_ERR_UNSUPPORTED;
    if (opts) {
        if (opts->path < MOE_PATH_AUTO || opts->path > MOE_PATH_TILE) return MOE_ERR_INVALID;
        if (opts->split_k < 0 || opts->split_k > MOE_MAX_SPLIT_K) return MOE_ERR_INVALID;
        if (opts->tile < MOE_TILE_AUTO || opts->tile > MOE_TILE_48x128) return MOE_ERR_INVALID;
        if (opts->i2f != MOE_I2F_TRICK && opts->i2f != MOE_I2F_NATIVE) return MOE_ERR_INVALID;
        if (opts->i2f == MOE_I2F_NATIVE) {
            // built for the tile path of the MT encoder shapes only
            const int path = moe::gemm_choose_path(R, E, K, N, wtype, act, opts->path);
            const int tile = moe::gemm_choose_tile(R, E, N, act, wtype, group != 0, opts->tile);
            if (path != MOE_PATH_TILE || !moe::gemm_native_supported(wtype, act, group, tile))
                return MOE_ERR_UNSUPPORTED;
        }
    }
    if ((int64_t)R * K >= (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!a || !offsets || !w || !out) return MOE_ERR_INVALID;
    if (wtype != MOE_W_FP16 && !scales) return MOE_ERR_INVALID;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(offsets, 4))
        return MOE_ERR_INVALID;
    if (scales && !aligned(scales, 16)) return MOE_ERR_INVALID;
    return MOE_OK;
}

}  // namespace

// Scratch memory of moe_decode_layer_noalloc: a workspace that lives in the code object, so the
// call needs no allocation.  Each device that loads the library holds its own copy until the
// process ends; host code reaches it only through the address hipGetSymbolAddress returns for
// the current device (the array's name is a host-side stand-in, not a device address).
static __device__ __align__(256) uint8_t scratch[MOE_DECODE_SCRATCH_BYTES];

namespace {

std::atomic<void*> g_scratch_ptr[64];   // device address of `scratch`, per device id
std::mutex g_scratch_mu;

// Address of this device's `scratch`, looked up once per device (with that device current).
void* scratch_address(int dev) {
    void* ptr = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (ptr) return ptr;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    ptr = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (!ptr) {
        if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) {
            (void)hipGetLastError();
            return nullptr;
        }
        g_scratch_ptr[dev].store(ptr, std::memory_order_release);
    }
    return ptr;
}

}  // namespace

namespace moe {
int32_t device_status() { return check_device(); }
}  // namespace moe

extern "C" {

int32_t moe_version(void) { return kVersion; }

const char* moe_status_str(int32_t s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_INVALID: return "MOE_ERR_INVALID: invalid argument";
        case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED: shape or option not supported";
        case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace missing or too small";
        case MOE_ERR_NO_DEVICE: return "MOE_ERR_NO_DEVICE: no usable gfx950 device";
        case MOE_ERR_HIP: return "MOE_ERR_HIP: HIP runtime error";
        default: return "unknown status";
    }
}

int32_t moe_route_topk_active(const float* logits, const uint8_t* active, int32_t T, int32_t E,
                              int32_t k, int32_t gate_mode, int32_t* topk_ids, float* topk_w,
                              void* stream) {
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || k > E)
        return MOE_ERR_INVALID;
    if (gate_mode != MOE_GATE_SOFTMAX_TOPK && gate_mode != MOE_GATE_SOFTMAX_ALL)
        return MOE_ERR_INVALID;
    if ((int64_t)T * E >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4)) return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_route_topk(logits, active, T, E, k,
                                             gate_mode == MOE_GATE_SOFTMAX_ALL, topk_ids, topk_w,
                                             (hipStream_t)stream));
}

int32_t moe_route_topk(const float* logits, int32_t T, int32_t E, int32_t k, int32_t gate_mode,
                       int32_t* topk_ids, float* topk_w, void* stream) {
    return moe_route_topk_active(logits, nullptr, T, E, k, gate_mode, topk_ids, topk_w, stream);
}

size_t moe_permute_workspace_size(int32_t T, int32_t k, int32_t E) {
    if (T <= 0 || k < 1 || k > MOE_MAX_TOPK || E < 1 || E > MOE_MAX_EXPERTS) return 0;
    if ((int64_t)T * k >= (int64_t)1 << 31) return 0;
    return moe::sort_workspace_bytes(T * k, E);
}

int32_t moe_permute(const int32_t* topk_ids, const float* topk_w, const uint16_t* x, int32_t T,
                    int32_t k, int32_t E, int32_t d, int32_t* perm, int32_t* inv_perm,
                    int32_t* expert_offsets, uint16_t* x_perm, float* w_perm, void* ws,
                    size_t ws_bytes, void* stream) {
    if (T < 0 || k < 1 || k > MOE_MAX_TOPK || E < 1 || E > MOE_MAX_EXPERTS || d <= 0)
        return MOE_ERR_INVALID;
    if (d % 8 != 0) return MOE_ERR_UNSUPPORTED;
    const int64_t R = (int64_t)T * k;
    if (R >= (int64_t)1 << 31 || R * (d / 8) >= (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!topk_ids || !perm || !inv_perm || !expert_offsets) return MOE_ERR_INVALID;
    if (x_perm && !x) return MOE_ERR_INVALID;
    if (w_perm && !topk_w) return MOE_ERR_INVALID;
    if ((x_perm && (!aligned(x, 16) || !aligned(x_perm, 16))) || !aligned(topk_ids, 4) ||
        !aligned(perm, 4) || !aligned(inv_perm, 4) || !aligned(expert_offsets, 4))
        return MOE_ERR_INVALID;
    if ((topk_w && !aligned(topk_w, 4)) || (w_perm && !aligned(w_perm, 4))) return MOE_ERR_INVALID;
    const size_t need = moe::sort_workspace_bytes((int)R, E);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 4))) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = moe::launch_sort(topk_ids, topk_w, (int)R, E, perm, inv_perm, expert_offsets,
                                    w_perm, ws, s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    if (!x_perm) return MOE_OK;               // the caller gathers inside the first GEMM
    return hip_status(moe::launch_gather(x, perm, (int)R, k, d, x_perm, s));
}

size_t moe_gemm_workspace_size(int32_t R, int32_t E, int32_t K, int32_t N, int32_t wtype,
                               int32_t act, const moe_gemm_opts* opts) {
    if (R <= 0 || E < 1 || K <= 0 || N <= 0) return 0;
    return plan_gemm(R, E, K, N, wtype, act, opts).ws;
}

static int32_t grouped_gemm(const uint16_t* a, int32_t a_nrows, const int32_t* a_rows,
                            int32_t a_div, const int32_t* expert_offsets, int32_t R, int32_t E,
                            int32_t K, int32_t N, const void* w_packed, const uint16_t* scales,
                            int32_t wtype, int32_t group_size, int32_t act,
                            const float* row_scale, uint16_t* out, int32_t out_nrows,
                            const int32_t* out_rows, const moe_gemm_opts* opts, void* ws,
                            size_t ws_bytes, void* stream) {
    if (int32_t st = validate_gemm(a, expert_offsets, R, E, K, N, w_packed, scales, wtype,
                                   group_size, act, out, opts))
        return st;
    if (a_rows && (a_div < 1 || a_nrows < 1)) return MOE_ERR_INVALID;
    if (out_rows && out_nrows < 0) return MOE_ERR_INVALID;
    if ((int64_t)a_nrows * K >= (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (row_scale && !aligned(row_scale, 4)) return MOE_ERR_INVALID;
    if ((a_rows && !aligned(a_rows, 4)) || (out_rows && !aligned(out_rows, 4)))
        return MOE_ERR_INVALID;
    const GemmPlan pl = plan_gemm(R, E, K, N, wtype, act, opts);
    if (pl.ws > 0 && (!ws || ws_bytes < pl.ws || !aligned(ws, 16))) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;

    moe::GemmParams p;
    p.a = a;
    p.a_rows = a_rows;
    p.a_div = a_rows ? a_div : 1;
    p.a_nrows = a_rows ? a_nrows : R;
    p.out_rows = out_rows;
    p.out_nrows = out_rows ? out_nrows : R;
    p.offsets = expert_offsets;
    p.w = w_packed;
    p.scales = scales;
    p.row_scale = row_scale;
    p.out = out;
    p.R = R;
    p.E = E;
    p.K = K;
    p.N = N;
    p.wtype = wtype;
    p.group = group_size;
    p.act = act;
    p.split = pl.split;
    p.tile = opts ? opts->tile : MOE_TILE_AUTO;
    p.i2f = opts ? opts->i2f : MOE_I2F_TRICK;
    p.tiles16 = nullptr;
    hipStream_t s = (hipStream_t)stream;
    return hip_status(pl.path == MOE_PATH_TILE ? moe::launch_gemm_tile(p, s)
                                               : moe::launch_gemm_stream(p, s));
}

int32_t moe_grouped_gemm_wq(const uint16_t* a, const int32_t* expert_offsets, int32_t R,
                            int32_t E, int32_t K, int32_t N, const void* w_packed,
                            const uint16_t* scales, int32_t wtype, int32_t group_size,
                            int32_t act, const float* row_scale, uint16_t* out,
                            const moe_gemm_opts* opts, void* ws, size_t ws_bytes, void* stream) {
    return grouped_gemm(a, R, nullptr, 1, expert_offsets, R, E, K, N, w_packed, scales, wtype,
                        group_size, act, row_scale, out, R, nullptr, opts, ws, ws_bytes, stream);
}

int32_t moe_grouped_gemm_wq_rows(const uint16_t* a, int32_t a_nrows, const int32_t* a_rows,
                                 int32_t a_row_div, const int32_t* expert_offsets, int32_t R,
                                 int32_t E, int32_t K, int32_t N, const void* w_packed,
                                 const uint16_t* scales, int32_t wtype, int32_t group_size,
                                 int32_t act, const float* row_scale, uint16_t* out,
                                 int32_t out_nrows, const int32_t* out_rows,
                                 const moe_gemm_opts* opts, void* ws, size_t ws_bytes,
                                 void* stream) {
    if (a_nrows < 0 || out_nrows < 0) return MOE_ERR_INVALID;
    return grouped_gemm(a, a_rows ? a_nrows : R, a_rows, a_row_div, expert_offsets, R, E, K, N,
                        w_packed, scales, wtype, group_size, act, row_scale, out,
                        out_rows ? out_nrows : R, out_rows, opts, ws, ws_bytes, stream);
}

static int32_t validate_decode(int32_t T, int32_t E, int32_t k, int32_t gate_mode, int32_t d,
                               int32_t inter, int32_t act, int32_t wtype, int32_t group) {
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || k > E)
        return MOE_ERR_INVALID;
    if (gate_mode != MOE_GATE_SOFTMAX_TOPK && gate_mode != MOE_GATE_SOFTMAX_ALL)
        return MOE_ERR_INVALID;
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID;
    if (wtype < MOE_W_INT4 || wtype > MOE_W_FP16) return MOE_ERR_INVALID;
    if (d <= 0 || inter <= 0) return MOE_ERR_INVALID;
    if (group != 0 && group != 128) return MOE_ERR_UNSUPPORTED;
    if (wtype == MOE_W_FP16 && group != 0) return MOE_ERR_UNSUPPORTED;
    if (d % 128 != 0 || inter % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (T > MOE_DECODE_MAX_TOKENS || T * k > MOE_DECODE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)inter * MOE_DECODE_MAX_ROWS >= (int64_t)1 << 31 ||
        (int64_t)d * MOE_DECODE_MAX_ROWS >= (int64_t)1 << 31)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_decode_workspace_size(int32_t T, int32_t k, int32_t E, int32_t d, int32_t inter,
                                 int32_t wtype) {
    if (validate_decode(T, E, k, MOE_GATE_SOFTMAX_TOPK, d, inter, MOE_ACT_NONE, wtype, 0) !=
        MOE_OK)
        return 0;
    return moe::decode_workspace_layout(T, k, E, d, inter, wtype, 0, nullptr, nullptr);
}

// The shared experts of moe_decode_layer_shared: fp16 weights beside integer-coded routed ones.
static int32_t validate_shared(int32_t wtype, int32_t shared_inter) {
    if (shared_inter <= 0) return MOE_ERR_INVALID;
    if (wtype == MOE_W_FP16 || shared_inter % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)shared_inter * 2 * MOE_DECODE_MAX_TOKENS >= (int64_t)1 << 31)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_decode_shared_workspace_size(int32_t T, int32_t k, int32_t E, int32_t d,
                                        int32_t inter, int32_t wtype, int32_t shared_inter) {
    if (validate_decode(T, E, k, MOE_GATE_SOFTMAX_TOPK, d, inter, MOE_ACT_NONE, wtype, 0) !=
            MOE_OK ||
        validate_shared(wtype, shared_inter) != MOE_OK)
        return 0;
    return moe::decode_workspace_layout(T, k, E, d, inter, wtype, shared_inter, nullptr, nullptr);
}

// moe_decode_layer and moe_decode_layer_shared: sw1 == NULL for no shared experts.
static int32_t decode_layer(const float* logits, const uint8_t* active, const uint16_t* x,
                            int32_t T, int32_t E, int32_t k, int32_t gate_mode, int32_t d,
                            int32_t inter, int32_t act, const void* w1, const uint16_t* s1,
                            const void* w2, const uint16_t* s2, int32_t wtype, int32_t group_size,
                            const void* sw1, const void* sw2, int32_t shared_inter,
                            const uint16_t* addend, void* addend_ready, int32_t* topk_ids,
                            float* topk_w, uint16_t* out, void* ws, size_t ws_bytes,
                            void* stream) {
    if (int32_t st = validate_decode(T, E, k, gate_mode, d, inter, act, wtype, group_size))
        return st;
    const bool shared = sw1 != nullptr;
    if (shared) {
        if (int32_t st = validate_shared(wtype, shared_inter)) return st;
    }
    if (T == 0) return MOE_OK;
    if (!logits || !x || !w1 || !w2 || !topk_ids || !topk_w || !out) return MOE_ERR_INVALID;
    if (wtype != MOE_W_FP16 && (!s1 || !s2)) return MOE_ERR_INVALID;
    if (shared && !sw2) return MOE_ERR_INVALID;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
        !aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(out, 16))
        return MOE_ERR_INVALID;
    if ((s1 && !aligned(s1, 16)) || (s2 && !aligned(s2, 16)) || (addend && !aligned(addend, 16)))
        return MOE_ERR_INVALID;
    if (shared && (!aligned(sw1, 16) || !aligned(sw2, 16))) return MOE_ERR_INVALID;
    const size_t need = moe::decode_workspace_layout(T, k, E, d, inter, wtype,
                                                     shared ? shared_inter : 0, nullptr, nullptr);
    if (!ws || ws_bytes < need || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;
    moe::DecodeArgs a;
    a.logits = logits;
    a.active = active;
    a.x = x;
    a.T = T;
    a.E = E;
    a.k = k;
    a.gate_all = gate_mode == MOE_GATE_SOFTMAX_ALL;
    a.d = d;
    a.inter = inter;
    a.act = act;
    a.w1 = w1;
    a.s1 = s1;
    a.w2 = w2;
    a.s2 = s2;
    a.wtype = wtype;
    a.group = group_size;
    a.sw1 = shared ? sw1 : nullptr;
    a.sw2 = shared ? sw2 : nullptr;
    a.shared_inter = shared ? shared_inter : 0;
    a.addend = shared ? nullptr : addend;
    a.addend_ready = shared ? nullptr : addend_ready;
    a.ids = topk_ids;
    a.wts = topk_w;
    a.out = out;
    a.ws = ws;
    return hip_status(moe::launch_decode(a, (hipStream_t)stream));
}

int32_t moe_decode_layer(const float* logits, const uint8_t* active, const uint16_t* x,
                         int32_t T, int32_t E, int32_t k, int32_t gate_mode, int32_t d,
                         int32_t inter, int32_t act,
                         const void* w1, const uint16_t* s1, const void* w2,
                         const uint16_t* s2, int32_t wtype, int32_t group_size,
                         const uint16_t* addend, void* addend_ready, int32_t* topk_ids,
                         float* topk_w, uint16_t* out, void* ws, size_t ws_bytes,
                         void* stream) {
    return decode_layer(logits, active, x, T, E, k, gate_mode, d, inter, act, w1, s1, w2, s2,
                        wtype, group_size, nullptr, nullptr, 0, addend, addend_ready, topk_ids,
                        topk_w, out, ws, ws_bytes, stream);
}

int32_t moe_decode_layer_shared(const float* logits, const uint8_t* active, const uint16_t* x,
                                int32_t T, int32_t E, int32_t k, int32_t gate_mode, int32_t d,
                                int32_t inter, int32_t act, const void* w1, const uint16_t* s1,
                                const void* w2, const uint16_t* s2, int32_t wtype,
                                int32_t group_size, const void* shared_w1,
                                const void* shared_w2, int32_t shared_inter, int32_t* topk_ids,
                                float* topk_w, uint16_t* out, void* ws, size_t ws_bytes,
                                void* stream) {
    if (!shared_w1) return MOE_ERR_INVALID;
    return decode_layer(logits, active, x, T, E, k, gate_mode, d, inter, act, w1, s1, w2, s2,
                        wtype, group_size, shared_w1, shared_w2, shared_inter, nullptr, nullptr,
                        topk_ids, topk_w, out, ws, ws_bytes, stream);
}

int32_t moe_decode_layer_noalloc(const float* logits, const uint8_t* active, const uint16_t* x,
                                 int32_t T, int32_t E, int32_t k, int32_t gate_mode, int32_t d,
                                 int32_t inter, int32_t act, const void* w1, const uint16_t* s1,
                                 const void* w2, const uint16_t* s2, int32_t wtype,
                                 int32_t group_size, const uint16_t* addend, void* addend_ready,
                                 int32_t* topk_ids, float* topk_w, uint16_t* out, void* stream) {
    if (int32_t st = validate_decode(T, E, k, gate_mode, d, inter, act, wtype, group_size))
        return st;
    if (T == 0) return MOE_OK;
    const size_t need = moe::decode_workspace_layout(T, k, E, d, inter, wtype, 0, nullptr, nullptr);
    if (need > (size_t)MOE_DECODE_SCRATCH_BYTES) return MOE_ERR_UNSUPPORTED;
    if (int32_t st = check_device()) return st;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MOE_ERR_NO_DEVICE;
    void* ws = scratch_address(dev);
    if (!ws) return MOE_ERR_HIP;
    // the rest is moe_decode_layer's validation and launch, on the scratch workspace
    return moe_decode_layer(logits, active, x, T, E, k, gate_mode, d, inter, act, w1, s1, w2, s2,
                            wtype, group_size, addend, addend_ready, topk_ids, topk_w, out, ws,
                            (size_t)MOE_DECODE_SCRATCH_BYTES, stream);
}

int32_t moe_unpermute_combine(const uint16_t* y_perm, const int32_t* inv_perm, const float* topk_w,
                              const uint16_t* addend, int32_t T, int32_t k, int32_t d,
                              uint16_t* out, void* stream) {
    if (T < 0 || k < 1 || k > MOE_MAX_TOPK || d <= 0) return MOE_ERR_INVALID;
    if (d % 8 != 0) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)T * k >= (int64_t)1 << 31 || (int64_t)T * (d / 8) >= (int64_t)1 << 32)
        return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!y_perm || !inv_perm || !out) return MOE_ERR_INVALID;
    if (!aligned(y_perm, 16) || !aligned(out, 16) || !aligned(inv_perm, 4)) return MOE_ERR_INVALID;
    if ((addend && !aligned(addend, 16)) || (topk_w && !aligned(topk_w, 4))) return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_combine(y_perm, inv_perm, topk_w, addend, T, k, d, out,
                                          (hipStream_t)stream));
}

int32_t moe_elb_accumulate(const int32_t* ids, int32_t L, int32_t T, int32_t k, int32_t E,
                           int32_t* counts, void* stream) {
    if (L < 0 || T < 0 || k < 1 || E < 1 || E > MOE_MAX_EXPERTS) return MOE_ERR_INVALID;
    if ((int64_t)L * T * k >= (int64_t)1 << 31 || (int64_t)L * E >= (int64_t)1 << 31)
        return MOE_ERR_UNSUPPORTED;
    if (L == 0) return MOE_OK;
    if (!counts || (T > 0 && !ids)) return MOE_ERR_INVALID;
    if (!aligned(counts, 4) || (ids && !aligned(ids, 4))) return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_elb_accumulate(ids, L, T * k, E, counts, (hipStream_t)stream));
}

int32_t moe_elb_top_m(const int32_t* counts, int32_t L, int32_t E, int32_t M, int32_t* experts,
                      int32_t* top_counts, void* stream) {
    if (L < 0 || E < 1 || E > MOE_MAX_EXPERTS || M < 1 || M > E) return MOE_ERR_INVALID;
    if ((int64_t)L * E >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
    if (L == 0) return MOE_OK;
    if (!counts || !experts) return MOE_ERR_INVALID;
    if (!aligned(counts, 4) || !aligned(experts, 4) || (top_counts && !aligned(top_counts, 4)))
        return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_elb_top_m(counts, L, E, M, experts, top_counts,
                                            (hipStream_t)stream));
}

int32_t moe_bf16_recombine(const uint8_t* exponents, const uint8_t* sign_mantissa, size_t n,
                           uint16_t* out, void* stream) {
    if (n == 0) return MOE_OK;
    if (n >= (size_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    if (!exponents || !sign_mantissa || !out) return MOE_ERR_INVALID;
    if (!aligned(exponents, 16) || !aligned(sign_mantissa, 16) || !aligned(out, 16))
        return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_bf16_recombine(exponents, sign_mantissa, n, out,
                                                 (hipStream_t)stream));
}

// ---- balance loss and the router's gradients ----
static int32_t validate_segments(int32_t S, int32_t T, int32_t E, int32_t k,
                                 const int32_t* seq_offsets) {
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || S < 1)
        return MOE_ERR_INVALID;
    if (!seq_offsets && S != 1) return MOE_ERR_INVALID;
    if (!aligned(seq_offsets, 4)) return MOE_ERR_INVALID;
    if (T >= 1 << 28 || S > 1 << 20 || (int64_t)T * E >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_balance_workspace_size(int32_t T, int32_t E, int32_t S) {
    static const int32_t any = 0;
    if (validate_segments(S, T, E, 1, &any) != MOE_OK) return 0;
    return moe::balance_workspace_layout(T, E, S, nullptr, nullptr);
}

int32_t moe_balance_loss(const float* logits, const int32_t* topk_ids, const uint8_t* active,
                         const int32_t* seq_offsets, int32_t S, int32_t T, int32_t E, int32_t k,
                         float coef, float* loss, int32_t* counts, float* probs, int32_t* tokens,
                         void* ws, size_t ws_bytes, void* stream) {
    if (int32_t st = validate_segments(S, T, E, k, seq_offsets)) return st;
    if (!loss || !counts || !probs || !tokens || (T > 0 && (!logits || !topk_ids)))
        return MOE_ERR_INVALID;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
        !aligned(probs, 4) || !aligned(tokens, 4))
        return MOE_ERR_INVALID;
    const size_t need = moe::balance_workspace_layout(T, E, S, nullptr, nullptr);
    if (!ws || ws_bytes < need || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;
    moe::BalanceParams p;
    p.logits = logits;
    p.ids = topk_ids;
    p.active = active;
    p.offsets = seq_offsets;
    p.S = S;
    p.T = T;
    p.E = E;
    p.k = k;
    p.coef = coef;
    p.loss = loss;
    p.counts = counts;
    p.probs = probs;
    p.tokens = tokens;
    moe::balance_workspace_layout(T, E, S, &p, (char*)ws);
    return hip_status(moe::launch_balance(p, (hipStream_t)stream));
}

int32_t moe_route_backward(const float* logits, const int32_t* topk_ids, const float* topk_w,
                           const float* grad_w, const uint8_t* active, const int32_t* seq_offsets,
                           int32_t S, int32_t T, int32_t E, int32_t k, int32_t gate_mode,
                           const int32_t* counts, const int32_t* tokens, float coef,
                           const float* grad_loss, float* grad_logits, void* stream) {
    if (int32_t st = validate_segments(S, T, E, k, seq_offsets)) return st;
    if (gate_mode != MOE_GATE_SOFTMAX_TOPK && gate_mode != MOE_GATE_SOFTMAX_ALL)
        return MOE_ERR_INVALID;
    if (!grad_w && !counts) return MOE_ERR_INVALID;
    if ((counts != nullptr) != (tokens != nullptr)) return MOE_ERR_INVALID;
    if (T == 0) return MOE_OK;
    if (!logits || !grad_logits || (grad_w && (!topk_ids || !topk_w))) return MOE_ERR_INVALID;
    if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(grad_w, 4) ||
        !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(grad_loss, 4) ||
        !aligned(grad_logits, 4))
        return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    moe::RouteGradParams p;
    p.logits = logits;
    p.ids = topk_ids;
    p.topk_w = topk_w;
    p.grad_w = grad_w;
    p.active = active;
    p.offsets = seq_offsets;
    p.S = S;
    p.T = T;
    p.E = E;
    p.k = k;
    p.gate_all = gate_mode == MOE_GATE_SOFTMAX_ALL;
    p.counts = counts;
    p.tokens = tokens;
    p.coef = coef;
    p.grad_loss = grad_loss;
    p.grad = grad_logits;
    return hip_status(moe::launch_route_backward(p, (hipStream_t)stream));
}

int32_t moe_combine_backward(const uint16_t* grad_out, const uint16_t* y_perm,
                             const int32_t* inv_perm, const float* topk_w, int32_t T, int32_t k,
                             int32_t d, float* grad_w, uint16_t* grad_y, void* stream) {
    if (T < 0 || k < 1 || k > MOE_MAX_TOPK || d <= 0) return MOE_ERR_INVALID;
    if (!grad_w && !grad_y) return MOE_ERR_INVALID;
    if (d % 8 != 0 || T >= 1 << 24) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!grad_out || !inv_perm || (grad_w && !y_perm) || (grad_y && !topk_w)) return MOE_ERR_INVALID;
    if (!aligned(grad_out, 16) || !aligned(y_perm, 16) || !aligned(inv_perm, 4) ||
        !aligned(topk_w, 4) || !aligned(grad_w, 4) || !aligned(grad_y, 16))
        return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    moe::CombineGradParams p;
    p.grad_out = grad_out;
    p.y = y_perm;
    p.inv_perm = inv_perm;
    p.topk_w = topk_w;
    p.T = T;
    p.k = k;
    p.d = d;
    p.grad_w = grad_w;
    p.grad_y = grad_y;
    return hip_status(moe::launch_combine_backward(p, (hipStream_t)stream));
}

// ---- dense linear layer and its gradients ----
namespace {

constexpr int64_t kLinearMaxStride = (int64_t)1 << 22;   // a tile's byte offsets stay below 2^31

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int up8(int n) { return (n + 7) / 8 * 8; }

// Rows that 16-byte pieces can read in place.
bool in_pieces(int cols, int64_t ld) { return cols % 8 == 0 && ld % 8 == 0; }

int32_t validate_linear_sizes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t act) {
    if (M < 0 || N < 0 || K < 1) return MOE_ERR_INVALID;
    if (dtype != MOE_DT_FP16 && dtype != MOE_DT_BF16) return MOE_ERR_INVALID;
    if (act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_ERR_INVALID;
    if (act == MOE_ACT_SWIGLU) return MOE_ERR_UNSUPPORTED;
    if (K > kLinearMaxStride || N > kLinearMaxStride || M > 1 << 28) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)M * N >= (int64_t)1 << 36 || (int64_t)M * K >= (int64_t)1 << 36 ||
        (int64_t)N * K >= (int64_t)1 << 36)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int32_t validate_stride(int64_t ld, int32_t cols) {
    if (ld < cols) return MOE_ERR_INVALID;
    return ld > kLinearMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Hands out 256-byte aligned pieces of a workspace (base NULL: only counts).
struct Carver {
    char* base;
    size_t used = 0;
    void* take(size_t bytes) {
        void* p = base ? base + used : nullptr;
        used += up256(bytes);
        return p;
    }
};

struct LinearForward {
    moe::LinearProduct p;
    uint16_t *pack_a, *pack_w;
};

// Sizes and workspace of moe_linear (pointers are filled in by the caller).
LinearForward linear_forward(int32_t M, int32_t N, int32_t K, int64_t lda, int64_t ldw, Carver& c) {
    LinearForward f{};
    moe::LinearProduct& p = f.p;
    p.lda = lda;
    p.ldb = ldw;
    p.M = p.a_outs = M;
    p.N = p.b_outs = N;
    p.red = p.b_red = up8(K);
    p.parts = 1;
    if (!in_pieces(K, lda)) {
        f.pack_a = (uint16_t*)c.take((size_t)M * up8(K) * 2);
        p.lda = up8(K);
    }
    if (!in_pieces(K, ldw)) {
        f.pack_w = (uint16_t*)c.take((size_t)N * up8(K) * 2);
        p.ldb = up8(K);
    }
    moe::linear_plan(p);
    if (p.split > 1) p.part = (float*)c.take(moe::linear_part_bytes(p));
    return f;
}

struct LinearBackward {
    moe::LinearProduct da, dw;
    moe::LinearDz dz;
    uint16_t *pack_a, *pack_w;
    bool need_dz;             // the products read a copy of the gradient
    bool narrow;              // both gradients in one pass, where both are wanted
    float* part;
};

LinearBackward linear_backward(int32_t M, int32_t N, int32_t K, int64_t lda, int64_t ldw, int64_t ldg,
                               int32_t grad_dtype, int32_t act, Carver& c) {
    LinearBackward f{};
    const int N8 = up8(N), K8 = up8(K);
    f.need_dz = grad_dtype == MOE_DT_FP32 || act != MOE_ACT_NONE || !in_pieces(N, ldg);
    // Through SILU or GELU dz is a product with no 16-bit form.  Rounded once it costs the gradients
    // as much as their own rounding does (1.4 times the error in all); below 256 rows, where the
    // products wait for memory, it is kept in two parts like an fp32 gradient.
    const bool curved = act == MOE_ACT_SILU || act == MOE_ACT_GELU;
    const int parts = grad_dtype == MOE_DT_FP32 || (curved && M < 256) ? 2 : 1;
    f.dz.cols8 = N8;
    f.dz.parts = parts;
    const int64_t ldz = f.need_dz ? N8 : ldg;
    if (f.need_dz) f.dz.dz = (uint16_t*)c.take((size_t)parts * M * N8 * 2);
    f.dz.sums = (float*)c.take((size_t)moe::linear_dz_blocks(M, N) * N * 4);
    if (!in_pieces(K, ldw)) {
        f.pack_w = (uint16_t*)c.take((size_t)N * K8 * 2);
        ldw = K8;
    }
    if (!in_pieces(K, lda)) {
        f.pack_a = (uint16_t*)c.take((size_t)M * K8 * 2);
        lda = K8;
    }
    // da[m, k] = sum_n dz[m][n] w[n][k]
    f.da.lda = ldz;
    f.da.ldb = ldw;
    f.da.b_cols = 1;
    f.da.M = f.da.a_outs = M;
    f.da.N = K;
    f.da.b_outs = K8;
    f.da.red = N8;
    f.da.b_red = N;
    f.da.parts = parts;
    f.da.a_part = (int64_t)M * N8;
    moe::linear_plan(f.da);
    // dw[n, k] = sum_m dz[m][n] a[m][k]
    f.dw.lda = ldz;
    f.dw.ldb = lda;
    f.dw.a_cols = f.dw.b_cols = 1;
    f.dw.M = N;
    f.dw.a_outs = N8;
    f.dw.N = K;
    f.dw.b_outs = K8;
    f.dw.red = f.dw.b_red = M;
    f.dw.parts = parts;
    f.dw.a_part = (int64_t)M * N8;
    moe::linear_plan(f.dw);
    const size_t pa = moe::linear_part_bytes(f.da), pw = moe::linear_part_bytes(f.dw);
    const size_t pn = moe::linear_narrow_bytes(f.da, f.dw);
    const size_t most = pa > pw ? pa : pw;                 // the products run one after the other
    f.part = (float*)c.take(most > pn ? most : pn);
    f.narrow = pn > 0;
    f.da.part = f.da.split > 1 ? f.part : nullptr;
    f.dw.part = f.dw.split > 1 ? f.part : nullptr;
    return f;
}

// A matrix to copy into `dst` (NULL: none).
moe::LinearPack packed(const uint16_t* src, int64_t ld, int32_t rows, int32_t cols, uint16_t* dst) {
    return moe::LinearPack{src, ld, dst ? rows : 0, cols, up8(cols), dst};
}

void grad_out_epilogue(moe::LinearEpilogue& e, uint16_t* out, int32_t K) {
    e.out = out;
    e.ldo = K;
    e.vec = K % 8 == 0;
}

}  // namespace

size_t moe_linear_workspace_size(int32_t M, int32_t N, int32_t K, int64_t lda, int64_t ldw) {
    if (validate_linear_sizes(M, N, K, MOE_DT_FP16, MOE_ACT_NONE) != MOE_OK || M == 0 || N == 0)
        return 0;
    Carver c{nullptr};
    linear_forward(M, N, K, lda, ldw, c);
    return c.used;
}

int32_t moe_linear(const uint16_t* a, int64_t lda, const uint16_t* w, int64_t ldw,
                   const uint16_t* bias, const uint16_t* residual, int64_t ldr, int32_t M,
                   int32_t N, int32_t K, int32_t dtype, int32_t act, void* out, int64_t ldo,
                   int32_t out_dtype, uint16_t* preact, int64_t ldp, void* ws, size_t ws_bytes,
                   void* stream) {
    if (int32_t st = validate_linear_sizes(M, N, K, dtype, act)) return st;
    if (out_dtype < MOE_DT_FP16 || out_dtype > MOE_DT_FP32) return MOE_ERR_INVALID;
    if (out_dtype != dtype && out_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
    if (int32_t st = validate_stride(lda, K)) return st;
    if (int32_t st = validate_stride(ldw, K)) return st;
    if (int32_t st = validate_stride(ldo, N)) return st;
    if (residual)
        if (int32_t st = validate_stride(ldr, N)) return st;
    if (preact)
        if (int32_t st = validate_stride(ldp, N)) return st;
    if (M == 0 || N == 0) return MOE_OK;
    if (!a || !w || !out) return MOE_ERR_INVALID;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(residual, 16) ||
        !aligned(preact, 16) || !aligned(bias, 2))
        return MOE_ERR_INVALID;
    if (preact && (void*)preact == out) return MOE_ERR_INVALID;
    if (residual && (const void*)residual == out && (ldr != ldo || out_dtype != dtype))
        return MOE_ERR_INVALID;
    Carver c{(char*)ws};
    LinearForward f = linear_forward(M, N, K, lda, ldw, c);
    if (c.used && (!ws || ws_bytes < c.used || !aligned(ws, 16))) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;
    hipStream_t s = (hipStream_t)stream;
    moe::LinearProduct& p = f.p;
    p.a = f.pack_a ? f.pack_a : a;
    p.b = f.pack_w ? f.pack_w : w;
    if (moe::launch_linear_pack(packed(a, lda, M, K, f.pack_a), packed(w, ldw, N, K, f.pack_w), s) !=
        hipSuccess)
        return MOE_ERR_HIP;
    moe::LinearEpilogue& e = p.epi;
    e.bias = bias;
    e.residual = residual;
    e.ldr = ldr;
    e.preact = preact;
    e.ldp = ldp;
    e.out = out;
    e.ldo = ldo;
    e.out_f32 = out_dtype == MOE_DT_FP32;
    e.act = act;
    e.vec = ldo % 8 == 0 && (!residual || ldr % 8 == 0) && (!preact || ldp % 8 == 0);
    return hip_status(moe::launch_linear_product(p, dtype, s));
}

size_t moe_linear_backward_workspace_size(int32_t M, int32_t N, int32_t K, int64_t lda, int64_t ldw,
                                          int64_t ldg, int32_t grad_dtype, int32_t act) {
    if (validate_linear_sizes(M, N, K, MOE_DT_FP16, act) != MOE_OK) return 0;
    Carver c{nullptr};
    linear_backward(M, N, K, lda, ldw, ldg, grad_dtype, act, c);
    return c.used;
}

int32_t moe_linear_backward(const void* grad_out, int64_t ldg, int32_t grad_dtype,
                            const uint16_t* preact, int64_t ldp, const uint16_t* a, int64_t lda,
                            const uint16_t* w, int64_t ldw, int32_t M, int32_t N, int32_t K,
                            int32_t dtype, int32_t act, uint16_t* grad_a, uint16_t* grad_w,
                            uint16_t* grad_bias, void* ws, size_t ws_bytes, void* stream) {
    if (int32_t st = validate_linear_sizes(M, N, K, dtype, act)) return st;
    if (grad_dtype < MOE_DT_FP16 || grad_dtype > MOE_DT_FP32) return MOE_ERR_INVALID;
    if (grad_dtype != dtype && grad_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
    if (!grad_a && !grad_w && !grad_bias) return MOE_ERR_INVALID;
    if (int32_t st = validate_stride(ldg, N)) return st;
    if (act != MOE_ACT_NONE)
        if (int32_t st = validate_stride(ldp, N)) return st;
    if (int32_t st = validate_stride(lda, K)) return st;
    if (int32_t st = validate_stride(ldw, K)) return st;
    if (M > 0 && N > 0) {
        if (!grad_out || (act != MOE_ACT_NONE && !preact)) return MOE_ERR_INVALID;
        if ((grad_a && !w) || (grad_w && !a)) return MOE_ERR_INVALID;
    }
    if (!aligned(grad_out, 16) || !aligned(preact, 16) || !aligned(a, 16) || !aligned(w, 16) ||
        !aligned(grad_a, 16) || !aligned(grad_w, 16) || !aligned(grad_bias, 2))
        return MOE_ERR_INVALID;
    if ((M == 0 || !grad_a) && (N == 0 || (!grad_w && !grad_bias))) return MOE_OK;
    Carver c{(char*)ws};
    LinearBackward f = linear_backward(M, N, K, lda, ldw, ldg, grad_dtype, act, c);
    if (c.used && (!ws || ws_bytes < c.used || !aligned(ws, 16))) return MOE_ERR_WORKSPACE;
    if (int32_t st = check_device()) return st;
    hipStream_t s = (hipStream_t)stream;
    moe::LinearBias bias{};
    if (N > 0 && (f.need_dz || grad_bias)) {
        moe::LinearDz& z = f.dz;
        z.grad = grad_out;
        z.ldg = ldg;
        z.grad_f32 = grad_dtype == MOE_DT_FP32;
        z.preact = preact;
        z.ldp = ldp;
        z.act = act;
        z.M = M;
        z.N = N;
        if (!grad_a && !grad_w) z.dz = nullptr;
        if (!grad_bias) z.sums = nullptr;
        if (moe::launch_linear_dz(z, dtype, grad_bias, bias, s) != hipSuccess) return MOE_ERR_HIP;
    }
    const uint16_t* dz = f.need_dz ? f.dz.dz : (const uint16_t*)grad_out;
    const bool want_a = grad_a && M > 0, want_w = grad_w && N > 0;
    if (moe::launch_linear_pack(packed(w, ldw, N, K, want_a ? f.pack_w : nullptr),
                                packed(a, lda, M, K, want_w ? f.pack_a : nullptr), s) != hipSuccess)
        return MOE_ERR_HIP;
    f.da.a = f.dw.a = dz;
    f.da.b = f.pack_w ? f.pack_w : w;
    f.dw.b = f.pack_a ? f.pack_a : a;
    grad_out_epilogue(f.da.epi, grad_a, K);
    grad_out_epilogue(f.dw.epi, grad_w, K);
    if (want_a && want_w && f.narrow) {
        f.dw.part = f.part;
        return hip_status(moe::launch_linear_narrow(f.da, f.dw, bias, dtype, s));
    }
    if (want_a && want_w && moe::linear_pair(f.da, f.dw))
        return hip_status(moe::launch_linear_pair(f.da, f.dw, bias, dtype, s));
    if (moe::launch_linear_bias(bias, dtype, s) != hipSuccess) return MOE_ERR_HIP;
    if (want_a && moe::launch_linear_product(f.da, dtype, s) != hipSuccess) return MOE_ERR_HIP;
    if (want_w && moe::launch_linear_product(f.dw, dtype, s) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
}

int32_t moe_dequant(const void* w_packed, const uint16_t* scales, int32_t wtype, int32_t group_size,
                    int32_t E, int32_t K, int32_t N, uint16_t* w_out, void* stream) {
    if (E < 1 || E > MOE_MAX_EXPERTS || K <= 0 || N <= 0) return MOE_ERR_INVALID;
    if (wtype != MOE_W_INT4 && wtype != MOE_W_INT8) return MOE_ERR_INVALID;
    if (group_size != 0 && group_size != 128) return MOE_ERR_UNSUPPORTED;
    if (K % 128 != 0 || N % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (!w_packed || !scales || !w_out) return MOE_ERR_INVALID;
    if (!aligned(w_packed, 16) || !aligned(scales, 16) || !aligned(w_out, 16)) return MOE_ERR_INVALID;
    if (int32_t st = check_device()) return st;
    return hip_status(moe::launch_dequant(w_packed, scales, wtype, group_size, E, K, N, w_out,
                                          (hipStream_t)stream));
}

}  // extern "C"
