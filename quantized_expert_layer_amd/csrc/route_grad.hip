// The router's balance loss with its counts, the gradient of the router logits, and the gradients
// of the combine (of the gate weights and of the expert rows).
//
// Softmax rows are held as in the gating: one token per 16-lane row of a wave, lane j of the row
// with experts j, j + 16, ... (PER_LANE of them), so a row's maximum and sum are DPP reductions.
#include "common.hpp"
#include "launch.hpp"
#include "route.hpp"

namespace moe {

// Sum over the 16 lanes of each row, in every lane, in one fixed order.
__device__ __forceinline__ float row_total(float v) {
    return __builtin_bit_cast(float, row_allreduce_bits(__builtin_bit_cast(int, v), [](int a, int b) {
        return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}

// Probabilities of one token's experts: softmax over its E logits; -inf and NaN have none, and a
// row with nothing else has none at all.
template <int PER_LANE>
__device__ __forceinline__ void softmax_row(const float* row, int E, int j16, float (&p)[PER_LANE]) {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const int e = j16 + 16 * i;
        float x = (row && e < E) ? row[e] : -__builtin_inff();
        if (x != x) x = -__builtin_inff();
        p[i] = x;
        m = fmaxf(m, x);
    }
    m = row_max_f32(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        p[i] = p[i] == -__builtin_inff() ? 0.0f : expf(p[i] - m);
        sum += p[i];
    }
    sum = row_total(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) p[i] *= inv;
}

__device__ __forceinline__ int clamp_offset(const int32_t* offsets, int s, int T) {
    return min(max(offsets[s], 0), T);
}

// ------------------------------------------------------------------------------------
// Pieces.  The batch is cut at every segment's start and at every multiple of `cell` tokens, so a
// piece lies in one segment s and one cell c.  Walking along the tokens each cut raises s or c, so
// s + c is a number of its own for every piece, below S + number of cells: piece b belongs to the
// last segment with start / cell + s <= b, found by a 64-way search of the offsets, without a
// table.  (A number no piece has gives an empty range.)
// ------------------------------------------------------------------------------------
__device__ __forceinline__ void piece_of(const BalanceParams& p, int b, int lane, int& s, int& lo,
                                         int& hi) {
    s = 0;
    if (!p.offsets) {
        lo = b * p.cell;
        hi = min(lo + p.cell, p.T);
        return;
    }
    for (int n = p.S; n > 1;) {                                // s is in [s, s + n)
        const int step = (n + kWave - 1) / kWave;
        const int at = s + lane * step;
        const bool hit = lane * step < n && at < p.S && clamp_offset(p.offsets, at, p.T) / p.cell + at <= b;
        const int hits = __popcll(__ballot(hit));
        s += max(hits - 1, 0) * step;
        n = step;
    }
    s = min(s, p.S - 1);
    const int c = max(b - s, 0);
    lo = max(clamp_offset(p.offsets, s, p.T), (int)min((int64_t)c * p.cell, (int64_t)p.T));
    hi = min(clamp_offset(p.offsets, s + 1, p.T), (int)min((int64_t)(c + 1) * p.cell, (int64_t)p.T));
}

// One piece per block: sums of its live tokens' probabilities (fp32, each lane over its own tokens
// in order, then rows and waves in a fixed order), counts of their slots (integers, so the order
// of the LDS atomics does not matter) and their number.
template <int PER_LANE>
__global__ __launch_bounds__(256) void balance_piece_kernel(BalanceParams p) {
    __shared__ float sums[4][16 * PER_LANE];
    __shared__ int counts[16 * PER_LANE];
    __shared__ int live_tokens;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int j16 = lane & 15, row = lane >> 4;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0;
    for (int e = threadIdx.x; e < 16 * PER_LANE; e += 256) counts[e] = 0;
    if (threadIdx.x == 0) live_tokens = 0;
    __syncthreads();
    int s, lo, hi;
    piece_of(p, blockIdx.x, lane, s, lo, hi);
    float acc[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) acc[i] = 0.0f;
    int seen = 0;
    for (int t0 = lo + wave * 4; t0 < hi; t0 += 16) {
        const int t = t0 + row;
        const bool live = t < hi && (!p.active || p.active[t]);
        float pr[PER_LANE];
        softmax_row<PER_LANE>(live ? p.logits + (size_t)t * p.E : nullptr, p.E, j16, pr);
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) acc[i] += pr[i];
        if (live) {
            seen += j16 == 0;
            if (j16 < p.k) {
                const int id = p.ids[(size_t)t * p.k + j16];
                if ((unsigned)id < (unsigned)p.E) atomicAdd(&counts[id], 1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        acc[i] += __shfl_xor(acc[i], 16);
        acc[i] += __shfl_xor(acc[i], 32);
        if (row == 0) sums[wave][j16 + 16 * i] = acc[i];
    }
    if (seen) atomicAdd(&live_tokens, seen);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += 256) {
        p.part_sums[(size_t)blockIdx.x * p.E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
        p.part_counts[(size_t)blockIdx.x * p.E + e] = counts[e];
    }
    if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = live_tokens;
}

// Fixed-order sum over the block's 1024 threads (in thread 0).
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* scratch) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_down(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x / 64] = v;
    __syncthreads();
    T r = 0;
    if (threadIdx.x == 0)
        for (int w = 0; w < 16; ++w) r += scratch[w];
    return r;
}

// One segment per block: adds its pieces (group g of threads takes pieces g, g + groups, ...; the
// groups are then added in order), writes counts, probs and tokens, and leaves the segment's term.
// The block that arrives last adds the terms in segment order.
__global__ __launch_bounds__(1024) void balance_segment_kernel(BalanceParams p) {
    __shared__ float fsum[1024];
    __shared__ int isum[1024];
    __shared__ float fs[16];
    __shared__ int is[16], is2[16];
    __shared__ int n_live, last;
    const int s = blockIdx.x, tid = threadIdx.x;
    int first = 0, end = p.pieces;
    if (p.offsets) {
        const int lo = clamp_offset(p.offsets, s, p.T), hi = clamp_offset(p.offsets, s + 1, p.T);
        first = min(lo / p.cell + s, p.pieces);
        end = hi > lo ? min((hi - 1) / p.cell + s + 1, p.pieces) : first;
    }
    int n = 0;
    for (int b = first + tid; b < end; b += 1024) n += p.part_tokens[b];
    n = block_sum(n, is);
    if (tid == 0) n_live = n;
    const int ep = p.E <= 16 ? 16 : p.E <= 64 ? 64 : p.E <= 128 ? 128 : 256;
    const int groups = 1024 / ep, g = tid / ep, e = tid % ep;
    float f = 0.0f;
    int c = 0;
    if (e < p.E) {
        for (int b = first + g; b < end; b += groups) {
            f += p.part_sums[(size_t)b * p.E + e];
            c += p.part_counts[(size_t)b * p.E + e];
        }
    }
    fsum[tid] = f;
    isum[tid] = c;
    __syncthreads();
    n = n_live;
    float term = 0.0f;
    if (g == 0 && e < p.E) {
        for (int i = 1; i < groups; ++i) {
            f += fsum[i * ep + e];
            c += isum[i * ep + e];
        }
        const float prob = n ? f / (float)n : 0.0f;
        p.counts[(size_t)s * p.E + e] = c;
        p.probs[(size_t)s * p.E + e] = prob;
        term = n ? (float)c * prob : 0.0f;
    }
    term = block_sum(term, fs);
    if (tid == 0) {
        p.tokens[s] = n;
        term = n ? term * ((float)p.E / ((float)p.k * (float)n)) : 0.0f;
        if (p.S == 1) {
            *p.loss = p.coef * term;
        } else {
            p.terms[s] = term;
            __threadfence();
            last = atomicAdd(p.arrived, 1) == p.S - 1;
        }
    }
    if (p.S == 1) return;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float total = 0.0f;
    int used = 0;
    for (int i = tid; i < p.S; i += 1024) {
        total += __hip_atomic_load(&p.terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        used += __hip_atomic_load(&p.tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
    }
    total = block_sum(total, fs);
    used = block_sum(used, is2);
    if (tid == 0) *p.loss = used ? p.coef * (total / (float)used) : 0.0f;
}

// Gradient of the logits, one token per 16-lane row.
template <int PER_LANE>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradParams p) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int j16 = lane & 15, row = lane >> 4;
    int used = 1;
    if (p.counts && p.S > 1) {                     // segments with tokens
        used = 0;
        for (int i = 0; i < p.S; i += kWave)
            used += __popcll(__ballot(i + lane < p.S && p.tokens[i + lane] > 0));
        used = max(used, 1);
    }
    const float scale = p.counts ? p.coef * (p.grad_loss ? *p.grad_loss : 1.0f) / (float)used : 0.0f;
    const int t = (blockIdx.x * 4 + wave) * 4 + row;
    const bool live = t < p.T && (!p.active || p.active[t]);
    float pr[PER_LANE], g[PER_LANE];
    softmax_row<PER_LANE>(live ? p.logits + (size_t)t * p.E : nullptr, p.E, j16, pr);
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) g[i] = 0.0f;
    if (p.counts) {
        int s = 0;
        if (p.offsets) {
            // last segment that starts at or before t: a 16-way search by the token's row
            int none = 0;
            for (int n = p.S + 1; n > 1;) {
                const int step = (n + 15) / 16;
                const int at = s + j16 * step;
                const bool hit = j16 * step < n && at <= p.S && p.offsets[at] <= t;
                const int hits = __popc((unsigned)(__ballot(hit) >> (row * 16)) & 0xffffu);
                none |= hits == 0;
                s += max(hits - 1, 0) * step;
                n = step;
            }
            if (none || s >= p.S) s = -1;
        }
        const int n = (live && s >= 0) ? p.tokens[s] : 0;
        float f[PER_LANE], dot = 0.0f;
        const float fe = n > 0 ? (float)p.E / ((float)p.k * (float)n) : 0.0f;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const int e = j16 + 16 * i;
            f[i] = (n > 0 && e < p.E) ? (float)p.counts[(size_t)s * p.E + e] * fe : 0.0f;
            dot += f[i] * pr[i];
        }
        dot = row_total(dot);
        const float c = n > 0 ? scale / (float)n : 0.0f;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) g[i] = n > 0 ? c * pr[i] * (f[i] - dot) : 0.0f;
    }
    if (p.grad_w) {
        int id = -1;
        float w = 0.0f, gw = 0.0f;
        if (live && j16 < p.k) {
            id = p.ids[(size_t)t * p.k + j16];
            if ((unsigned)id < (unsigned)p.E) {
                w = p.topk_w[(size_t)t * p.k + j16];
                gw = p.grad_w[(size_t)t * p.k + j16];
            } else {
                id = -1;
            }
        }
        const float u = row_total(w * gw);
        const float mine = p.gate_all ? w * gw : w * (gw - u);
        for (int j = 0; j < p.k; ++j) {
            const int idj = __shfl(id, row * 16 + j);
            const float v = __shfl(mine, row * 16 + j);
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i)
                if (j16 + 16 * i == idj) g[i] += v;
        }
        if (p.gate_all) {
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) g[i] -= pr[i] * u;
        }
    }
    if (t < p.T) {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const int e = j16 + 16 * i;
            if (e < p.E) p.grad[(size_t)t * p.E + e] = g[i];
        }
    }
}

// Gradients of the combine, one token per block: each thread takes 8 columns at a time, reads the
// token's gradient once for its k rows.
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineGradParams p) {
    __shared__ float red[4][MOE_MAX_TOPK];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint32_t R = (uint32_t)p.T * (uint32_t)p.k;
    const int d8 = p.d / 8;
    const int t = blockIdx.x;
    uint32_t pos[MOE_MAX_TOPK];
    float w[MOE_MAX_TOPK], sum[MOE_MAX_TOPK];
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
        sum[j] = 0.0f;
        w[j] = 0.0f;
        pos[j] = 0xffffffffu;
        if (j < p.k) {
            pos[j] = (uint32_t)p.inv_perm[(size_t)t * p.k + j];
            if (p.grad_y) w[j] = p.topk_w[(size_t)t * p.k + j];
        }
    }
    for (int c = threadIdx.x; c < d8; c += 256) {
        const u32x4 gv = ((const u32x4*)p.grad_out)[(size_t)t * d8 + c];
        float g[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const f16x2 v = as_f16x2(gv[h]);
            g[2 * h] = (float)v[0];
            g[2 * h + 1] = (float)v[1];
        }
#pragma unroll
        for (int j = 0; j < MOE_MAX_TOPK; ++j) {
            if (j >= p.k || pos[j] >= R) continue;
            const size_t at = (size_t)pos[j] * d8 + c;
            if (p.grad_w) {
                const u32x4 yv = ((const u32x4*)p.y)[at];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const f16x2 v = as_f16x2(yv[h]);
                    sum[j] += g[2 * h] * (float)v[0];
                    sum[j] += g[2 * h + 1] * (float)v[1];
                }
            }
            if (p.grad_y) {
                u32x4 o;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const f16x2 v = {(f16)(w[j] * g[2 * h]), (f16)(w[j] * g[2 * h + 1])};
                    o[h] = __builtin_bit_cast(uint32_t, v);
                }
                ((u32x4*)p.grad_y)[at] = o;
            }
        }
    }
    if (!p.grad_w) return;
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
        if (j >= p.k) break;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum[j] += __shfl_xor(sum[j], o);
        if (lane == 0) red[wave][j] = sum[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < p.k)
        p.grad_w[(size_t)t * p.k + threadIdx.x] =
            (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
}

// ------------------------------------------------------------------------------------ host

// Tokens per cell: about 512 pieces at most (beside one per segment), at least 16 tokens each.
int balance_cell(int T) { return T <= 8192 ? 16 : (int)(((int64_t)T + 8191) / 8192) * 16; }

size_t balance_workspace_layout(int T, int E, int S, BalanceParams* p, char* base) {
    const int cell = balance_cell(T);
    const int64_t pieces = (int64_t)((int64_t)T + cell - 1) / cell + S;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    size_t at = 0;
    auto take = [&](size_t bytes) {
        void* r = base ? base + at : nullptr;
        at += up(bytes);
        return r;
    };
    void* arrived = take(4);
    void* sums = take((size_t)pieces * E * 4);
    void* counts = take((size_t)pieces * E * 4);
    void* tokens = take((size_t)pieces * 4);
    void* terms = take((size_t)S * 4);
    if (p) {
        p->cell = cell;
        p->pieces = (int)pieces;
        p->arrived = (int*)arrived;
        p->part_sums = (float*)sums;
        p->part_counts = (int32_t*)counts;
        p->part_tokens = (int32_t*)tokens;
        p->terms = (float*)terms;
    }
    return at;
}

hipError_t launch_balance(const BalanceParams& p, hipStream_t s) {
    if (p.E <= 16) balance_piece_kernel<1><<<p.pieces, 256, 0, s>>>(p);
    else if (p.E <= 64) balance_piece_kernel<4><<<p.pieces, 256, 0, s>>>(p);
    else if (p.E <= 128) balance_piece_kernel<8><<<p.pieces, 256, 0, s>>>(p);
    else balance_piece_kernel<16><<<p.pieces, 256, 0, s>>>(p);
    balance_segment_kernel<<<p.S, 1024, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteGradParams& p, hipStream_t s) {
    const int grid = (int)(((int64_t)p.T + 15) / 16);
    if (p.E <= 16) route_backward_kernel<1><<<grid, 256, 0, s>>>(p);
    else if (p.E <= 64) route_backward_kernel<4><<<grid, 256, 0, s>>>(p);
    else if (p.E <= 128) route_backward_kernel<8><<<grid, 256, 0, s>>>(p);
    else route_backward_kernel<16><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineGradParams& p, hipStream_t s) {
    combine_backward_kernel<<<p.T, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace moe
