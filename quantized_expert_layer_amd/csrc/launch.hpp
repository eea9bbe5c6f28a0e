// Internal launchers (one per kernel family).  Arguments are validated by the C ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// MOE_OK when the current device is a usable gfx950, else MOE_ERR_NO_DEVICE (cached per device).
int32_t device_status();

hipError_t launch_route_topk(const float* logits, const uint8_t* active, int T, int E, int k,
                             int gate_all, int32_t* ids, float* wts, hipStream_t stream);

// ws: sort_workspace_bytes(R, E) bytes (none up to 1024 slots)
size_t sort_workspace_bytes(int R, int E);
hipError_t launch_sort(const int32_t* ids, const float* wts, int R, int E,
                       int32_t* perm, int32_t* inv_perm, int32_t* offsets, float* w_perm,
                       void* ws, hipStream_t stream);

hipError_t launch_gather(const uint16_t* x, const int32_t* perm, int R, int k, int d,
                         uint16_t* x_perm, hipStream_t stream);

hipError_t launch_combine(const uint16_t* y, const int32_t* inv_perm, const float* w,
                          const uint16_t* addend, int T, int k, int d, uint16_t* out,
                          hipStream_t stream);

hipError_t launch_elb_accumulate(const int32_t* ids, int L, int n, int E, int32_t* counts,
                                 hipStream_t stream);
hipError_t launch_elb_top_m(const int32_t* counts, int L, int E, int M, int32_t* experts,
                            int32_t* top_counts, hipStream_t stream);

hipError_t launch_bf16_recombine(const uint8_t* e, const uint8_t* sm, size_t n, uint16_t* out,
                                 hipStream_t stream);

hipError_t launch_dequant(const void* w, const uint16_t* scales, int wtype, int group,
                          int E, int K, int N, uint16_t* out, hipStream_t stream);

struct GemmParams {
    const uint16_t* a;
    const int32_t* a_rows;   // NULL: GEMM row p reads a[p]; else a[a_rows[p] / a_div]
    int a_div, a_nrows;      // divisor of a_rows, rows of a (source rows are clamped into it)
    const int32_t* out_rows; // NULL: GEMM row p writes out[p]; else out[out_rows[p]]
    int out_nrows;           // rows of out (other destinations are not written)
    const int32_t* offsets;
    const void* w;
    const uint16_t* scales;
    const float* row_scale;
    uint16_t* out;
    int R, E, K, N;
    int wtype, group, act;
    int split;           // stream path: waves per block splitting K (1..MOE_MAX_SPLIT_K)
    int tile;            // enum moe_tile (0 = automatic)
    int i2f;             // enum moe_i2f
    const int32_t* tiles16;  // stream path: NULL, or the decode tile table (16-row m-tiles)
};

// Path/split decisions (host-only, deterministic in the arguments).
int gemm_choose_path(int R, int E, int K, int N, int wtype, int act, int forced);
int gemm_choose_split(int R, int E, int K, int N, int wtype, int act, int forced);
int gemm_choose_tile(int R, int E, int N, int act, int wtype, bool grouped, int forced);
// Whether the native int-to-float conversion is built for this call (tile path).
bool gemm_native_supported(int wtype, int act, int group, int tile);

hipError_t launch_gemm_stream(const GemmParams& p, hipStream_t stream);
// The stream launch of a decode step's first GEMM (integer codes, at most 128 rows) with a
// dense fp16 SwiGLU GEMM over all rows of `side` in the same launch (offsets, row maps and tile
// table NULL; side.split is not read: its K is split over the launch's waves per workgroup,
// p.split, or 4 when p is unsplit).
hipError_t launch_gemm_stream_side(const GemmParams& p, const GemmParams& side,
                                   hipStream_t stream);
hipError_t launch_gemm_tile(const GemmParams& p, hipStream_t stream);

// ---- decode step (few tokens): gating + sort, GEMM 1, GEMM 2 with the combine ----
// Workspace of one decode call, carved from the caller's buffer (256-byte aligned parts).
struct DecodeWs {
    int32_t* perm;           // [R]
    int32_t* inv_perm;       // [R]
    int32_t* offsets;        // [E + 1]
    float* w_perm;           // [R]
    int32_t* tiles;          // [1 + kDecodeMaxTiles] tile table (count, then packed tiles)
    uint16_t* h;             // fp16 [R, inter] GEMM 1 output, sorted rows
    float* part;             // fp32 [nsplit, T, d] partial token sums of GEMM 2 (nsplit > 1)
    uint16_t* sh_h;          // fp16 [T, shared_inter] shared experts' hidden rows (or NULL)
    uint16_t* sh_y;          // fp16 [T, d] shared experts' output (or NULL)
};

struct CombineParams {
    const uint16_t* h;       // fp16 [R, K] rows sorted by expert
    const int32_t* tiles;    // tile table of the sorted rows
    const int32_t* perm;     // [R] flat slot t*k + j of sorted row p
    const float* w_perm;     // [R] gate weight of sorted row p
    const void* w;           // packed weights [E, K, N]
    const uint16_t* scales;  // [E, G, N], NULL for fp16 weights
    const uint16_t* addend;  // fp16 [T, N] or NULL
    uint16_t* out;           // fp16 [T, N]
    float* part;             // fp32 [nsplit, T, N] when nsplit > 1
    int R, E, K, N, T, k;
    int nsplit;              // blocks sharing the units of one 16-column block
};

struct DecodeArgs {
    const float* logits;
    const uint8_t* active;   // [T] or NULL: tokens with 0 take no expert
    const uint16_t* x;
    int T, E, k, gate_all, d, inter, act;
    const void* w1;
    const uint16_t* s1;
    const void* w2;
    const uint16_t* s2;
    int wtype, group;
    const void* sw1;         // shared experts, fp16 packed [d, 2 shared_inter] (gate | up), or NULL
    const void* sw2;         //   and [shared_inter, d]; SwiGLU, weight 1, every token
    int shared_inter;
    const uint16_t* addend;
    void* addend_ready;      // hipEvent_t or NULL: waited for before the launch that adds addend
    int32_t* ids;
    float* wts;
    uint16_t* out;
    void* ws;
};

// Blocks sharing one column group of the decode step's second GEMM (a power of two; at least
// two with shared experts, whose output the reduction launch adds).
int decode_combine_split(int d, bool shared);
// Bytes of the decode workspace (shared_inter 0: no shared experts); with ws and base given,
// also the part addresses.
size_t decode_workspace_layout(int T, int k, int E, int d, int inter, int wtype, int shared_inter,
                               DecodeWs* ws, char* base);
hipError_t launch_decode(const DecodeArgs& a, hipStream_t stream);

// ---- dense linear layer and its gradients ----

struct LinearEpilogue {      // out = act(sum + bias) + residual; preact = sum + bias
    const uint16_t* bias;    // [N] or NULL
    const uint16_t* residual;
    int64_t ldr;
    uint16_t* preact;        // [M, N] or NULL
    int64_t ldp;
    void* out;               // 16-bit of the operands' type, or fp32
    int64_t ldo;
    int out_f32, act;
    int vec;                 // eight columns of a row are 16-byte aligned in every matrix here
};

struct LinearProduct {       // C[i, j] = sum over parts and r < red of A[i, r] B[j, r]
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb;
    int64_t a_part;          // elements from A's first part of the summed index to its second
    int a_cols, b_cols;      // operand stored with its output index contiguous
    int a_outs, b_outs;      // output indices the operands hold (>= M, N: padded copies)
    int red, b_red, parts;   // summed indices per part (b_red: rows B really has); 1 or 2 parts
    int M, N;
    LinearEpilogue epi;
    float* part;             // fp32 [split, M, ldpart] when split > 1
    int ldpart, split, cfg, tiles_m, tiles_n;
    int whole;               // tiles computed whole; the rest in quarters (256 x 256 tiles)
    double us;               // what the plan expects
};

struct LinearPack {          // a matrix copied into rows of cols8 (rows 0: none)
    const uint16_t* src;
    int64_t ld;
    int rows, cols, cols8;
    uint16_t* dst;
};

struct LinearDz {
    const void* grad;        // [M, N], 16-bit or fp32
    int64_t ldg;
    int grad_f32;
    const uint16_t* preact;
    int64_t ldp;
    int act, M, N, cols8;
    uint16_t* dz;            // [parts, M, cols8] or NULL
    int parts;
    float* sums;             // [linear_dz_blocks(M, N), N] or NULL
    int lc;                  // log2 of a block's threads across the columns (set by the launch)
    uint16_t* bias;          // grad_bias where one block sums all rows, else NULL (set by the launch)
};

struct LinearBias {          // what is left to do for grad_bias after linear_dz (out NULL: nothing)
    const float* sums;       // [blocks, N]
    int blocks, N;
    uint16_t* out;
};

// Chooses tile, split and the partial layout from the sizes (host-only, deterministic).
void linear_plan(LinearProduct& p);
size_t linear_part_bytes(const LinearProduct& p);
hipError_t launch_linear_product(const LinearProduct& p, int dtype, hipStream_t stream);
// Both gradients in one launch, if that is the better plan for them (which it then becomes).
bool linear_pair(LinearProduct& da, LinearProduct& dw);
hipError_t launch_linear_pair(const LinearProduct& da, const LinearProduct& dw, const LinearBias& b,
                              int dtype, hipStream_t stream);
// Both gradients of a narrow layer (its input gradient's plan is the narrow one) in one pass;
// dw.part holds linear_narrow_bytes.
size_t linear_narrow_bytes(const LinearProduct& da, const LinearProduct& dw);
hipError_t launch_linear_narrow(const LinearProduct& da, LinearProduct dw, const LinearBias& b,
                                int dtype, hipStream_t stream);
hipError_t launch_linear_pack(const LinearPack& a, const LinearPack& b, hipStream_t stream);
int linear_dz_blocks(int M, int N);
// grad_bias is written here, or what is left of it goes to `rest`, for a later launch.
hipError_t launch_linear_dz(const LinearDz& p, int dtype, uint16_t* grad_bias, LinearBias& rest,
                            hipStream_t stream);
hipError_t launch_linear_bias(const LinearBias& b, int dtype, hipStream_t stream);

// ---- balance loss and the router's gradients ----
struct BalanceParams {
    const float* logits;     // [T, E]
    const int32_t* ids;      // [T, k]
    const uint8_t* active;   // [T] or NULL
    const int32_t* offsets;  // [S + 1] or NULL (S == 1: all tokens)
    int S, T, E, k;
    float coef;
    float* loss;
    int32_t* counts;
    float* probs;
    int32_t* tokens;
    int cell, pieces;        // tokens per cell; pieces of the batch (blocks)
    int* arrived;            // workspace: segments done
    float* part_sums;        // [pieces, E] probability sums
    int32_t* part_counts;    // [pieces, E]
    int32_t* part_tokens;    // [pieces]
    float* terms;            // [S]
    int vec;                 // rows of logits in 16-byte pieces (set by the launch)
    int count_in;            // the segment that is done last writes the loss (set by the launch)
};
size_t balance_workspace_layout(int T, int E, int S, BalanceParams* p, char* base);
hipError_t launch_balance(const BalanceParams& p, hipStream_t stream);

struct RouteGradParams {
    const float* logits;
    const int32_t* ids;
    const float* topk_w;
    const float* grad_w;     // or NULL: no gate term
    const uint8_t* active;
    const int32_t* offsets;
    int S, T, E, k, gate_all;
    const int32_t* counts;   // or NULL: no balance term
    const int32_t* tokens;
    float coef;
    const float* grad_loss;  // or NULL: 1
    float* grad;
    int vec;                 // rows in 16-byte pieces (set by the launch)
};
hipError_t launch_route_backward(const RouteGradParams& p, hipStream_t stream);

struct CombineGradParams {
    const uint16_t* grad_out;
    const uint16_t* y;
    const int32_t* inv_perm;
    const float* topk_w;
    int T, k, d;
    float* grad_w;           // or NULL
    uint16_t* grad_y;        // or NULL
};
hipError_t launch_combine_backward(const CombineGradParams& p, hipStream_t stream);

}  // namespace moe
