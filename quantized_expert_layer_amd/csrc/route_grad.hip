// The router's balance loss with its counts, the gradient of the router logits, and the gradients
// of the combine (of the gate weights and of the expert rows).
//
// One token per 16-lane row of a wave, as in the gating, but lane j of the row holds the PER_LANE
// consecutive experts from j PER_LANE on: a row's maximum and sum are DPP reductions, and its loads
// and stores go in 16-byte pieces where E is a multiple of 4.
#include <type_traits>

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

// e^x for x <= 0: the product with log2 e is taken in two parts, so its rounding (|x| 2^-24 of the
// result otherwise) is kept.  A third of expf's instructions, which bound these kernels.  Below
// -120 the result is 0 (and the product of a masked logit's lowest value would overflow).
__device__ __forceinline__ float exp_near(float x) {
    x = x < -120.0f ? -120.0f : x;
    const float hi = x * 1.44269504f, lo = fmaf(x, 1.44269504f, -hi);
    const float e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e, lo * 0.69314718f, e);
}
// Lane j of each 16-lane row, in all lanes of the row.
template <int J> __device__ __forceinline__ int row_lane(int v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x150 + J, 0xF, 0xF, false);   // row_newbcast
}

// This lane's part of a row of E values (experts past E read as some other).  Rows without a live
// token are loaded all the same, from a valid place: a load that waits for a flag costs a memory
// latency.
template <int PER_LANE, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, int j16, bool vec, T (&x)[PER_LANE]) {
    if constexpr (PER_LANE >= 4) {
        if (vec) {
            typedef T T4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int i = 0; i < PER_LANE; i += 4) {
                const T4 v = *(const T4*)(row + min(j16 * PER_LANE + i, E - 4));
#pragma unroll
                for (int c = 0; c < 4; ++c) x[i + c] = v[c];
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) x[i] = row[min(j16 * PER_LANE + i, E - 1)];
}
// Probabilities of the token's experts: softmax over its E logits; -inf and NaN have none, and a
// row with nothing else (or no live token) has none at all.
template <int PER_LANE>
__device__ __forceinline__ void softmax_row(const float (&x)[PER_LANE], bool live, int E, int j16,
                                            float (&p)[PER_LANE]) {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        p[i] = (live && j16 * PER_LANE + i < E && x[i] == x[i]) ? x[i] : -__builtin_inff();
        m = fmaxf(m, p[i]);
    }
    m = row_max_f32(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        p[i] = p[i] == -__builtin_inff() ? 0.0f : exp_near(p[i] - m);
        sum += p[i];
    }
    sum = row_total(sum);
    const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
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
    // the next 16 tokens' logits, ids and flags are on their way while these are summed
    float x[PER_LANE], nx[PER_LANE];
    int id = -1, nid = -1;
    bool live = false, nlive = false;
    auto fetch = [&](int t0, float (&v)[PER_LANE], int& vid, bool& vlive) {
        const int t = t0 + row, tc = min(t, p.T - 1);
        load_row<PER_LANE>(p.logits + (size_t)tc * p.E, p.E, j16, p.vec, v);
        vid = p.ids[(size_t)tc * p.k + min(j16, p.k - 1)];
        vlive = t < hi && (!p.active || p.active[tc]);
    };
    const int first = lo + wave * 4;
    if (first < hi) fetch(first, x, id, live);
    for (int t0 = first; t0 < hi; t0 += 16) {
        const bool more = t0 + 16 < hi;                            // wave-uniform
        if (more) fetch(t0 + 16, nx, nid, nlive);
        float pr[PER_LANE];
        softmax_row<PER_LANE>(x, live, p.E, j16, pr);
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) acc[i] += pr[i];
        if (live) {
            seen += j16 == 0;
            if (j16 < p.k && (unsigned)id < (unsigned)p.E) atomicAdd(&counts[id], 1);
        }
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) x[i] = nx[i];
        id = nid;
        live = nlive;
    }
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        acc[i] += __shfl_xor(acc[i], 16);
        acc[i] += __shfl_xor(acc[i], 32);
        if (row == 0) sums[wave][j16 * PER_LANE + i] = acc[i];
    }
    if (seen) atomicAdd(&live_tokens, seen);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += 256) {
        p.part_sums[(size_t)blockIdx.x * p.E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
        p.part_counts[(size_t)blockIdx.x * p.E + e] = counts[e];
    }
    if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = live_tokens;
}

// Fixed-order sum over the block's threads (in thread 0).
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* scratch) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_down(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x / 64] = v;
    __syncthreads();
    T r = 0;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)blockDim.x / 64; ++w) r += scratch[w];
    return r;
}

// The loss from the segments' terms, in one fixed order (`load` reads them; result in thread 0).
template <typename F, typename G>
__device__ __forceinline__ void balance_total(const BalanceParams& p, F load_term, G load_tokens,
                                              float* fs, int* is) {
    float total = 0.0f;
    int used = 0;
    for (int i = threadIdx.x; i < p.S; i += blockDim.x) {
        total += load_term(i);
        used += load_tokens(i) > 0;
    }
    total = block_sum(total, fs);
    used = block_sum(used, is);
    if (threadIdx.x == 0) *p.loss = used ? p.coef * (total / (float)used) : 0.0f;
}
__global__ __launch_bounds__(1024) void balance_total_kernel(BalanceParams p) {
    __shared__ float fs[16];
    __shared__ int is[16];
    balance_total(p, [&](int i) { return p.terms[i]; }, [&](int i) { return p.tokens[i]; }, fs, is);
}

// One segment per block: adds its pieces (group g of threads takes pieces g, g + groups, ...; the
// groups are then added in order), writes counts, probs and tokens, and leaves the segment's term.
// The block that arrives last adds the terms in segment order; with many segments a launch of its
// own does (the arrivals, one after the other at one address, would take 14 ns each).
__global__ __launch_bounds__(1024) void balance_segment_kernel(BalanceParams p) {
    __shared__ float fsum[1024];
    __shared__ int isum[1024];
    __shared__ float fs[16];
    __shared__ int is[16];
    __shared__ int n_part[16], last;
    const int s = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    int first = 0, end = p.pieces;
    if (p.offsets) {
        const int lo = clamp_offset(p.offsets, s, p.T), hi = clamp_offset(p.offsets, s + 1, p.T);
        first = min(lo / p.cell + s, p.pieces);
        end = hi > lo ? min((hi - 1) / p.cell + s + 1, p.pieces) : first;
    }
    const int ep = p.E <= 16 ? 16 : p.E <= 64 ? 64 : p.E <= 128 ? 128 : 256;
    const int groups = threads / ep, g = tid / ep, e = tid % ep, ec = min(e, p.E - 1);
    float f = 0.0f;
    int c = 0, n = 0;
#pragma unroll 8
    for (int b = first + g; b < end; b += groups) {
        f += p.part_sums[(size_t)b * p.E + ec];
        c += p.part_counts[(size_t)b * p.E + ec];
    }
    for (int b = first + tid; b < end; b += threads) n += p.part_tokens[b];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
    if ((tid & 63) == 0) n_part[tid / 64] = n;
    fsum[tid] = f;
    isum[tid] = c;
    __syncthreads();
    n = 0;
    for (int w = 0; w < threads / 64; ++w) n += n_part[w];
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
        term = n ? term * ((float)p.E / ((float)p.k * (float)n)) : 0.0f;
        if (!p.count_in) {
            p.tokens[s] = n;
            if (p.S == 1) *p.loss = p.coef * term;
            else p.terms[s] = term;
        } else {
            // What the last block reads is written through to memory, and has been before this
            // block counts itself: the wait stands in for a release of the whole L2.
            __hip_atomic_store(&p.tokens[s], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&p.terms[s], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            last = __hip_atomic_fetch_add(p.arrived, 1, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT) == p.S - 1;
        }
    }
    if (!p.count_in) return;
    __syncthreads();
    if (!last) return;
    balance_total(
        p, [&](int i) { return __hip_atomic_load(&p.terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); },
        [&](int i) { return __hip_atomic_load(&p.tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); },
        fs, is);
}

// Gradient of the logits, four consecutive tokens per wave.  All rows, choices and offsets are asked
// for before the first is used.  A slot's term meets its expert's lane through LDS: one add of a
// wave, whose lanes LDS serves in a fixed order (comparing every slot's id with every expert of a
// lane took 10.8 us instead of 9.5).  Bound by its arithmetic (some 200 instructions per wave): 65536 x
// 64, 38 MB, 9.5 us with both terms, 7.3 us through the gate alone (a copy of 17 MB takes 4.6 us);
// waves of 2, 4 and 8 groups with the next group's loads in flight took longer.
template <int PER_LANE, bool GATE, bool BALANCE, bool MANY>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradParams p) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int j16 = lane & 15, row = lane >> 4;
    __shared__ float slots[GATE ? 16 : 1][16 * PER_LANE + 4];
    int used = 1;
    if constexpr (BALANCE && MANY) {              // segments with tokens, counted by the block
        __shared__ int share[4];
        int n = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < p.S; i += 256) n += p.tokens[i] > 0;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o);
        if (lane == 0) share[wave] = n;
        __syncthreads();
        used = max(share[0] + share[1] + share[2] + share[3], 1);
    } else if (BALANCE && p.S > 1) {
        used = 0;
        for (int i = 0; i < p.S; i += kWave)
            used += __popcll(__ballot(i + lane < p.S && p.tokens[i + lane] > 0));
        used = max(used, 1);
    }
    const float scale = BALANCE ? p.coef * (p.grad_loss ? *p.grad_loss : 1.0f) / (float)used : 0.0f;
    // up to 63 segments: their offsets stay in the lanes
    const bool few = p.S < kWave;
    const int my_offset = (BALANCE && p.offsets && few) ? p.offsets[min(lane, p.S)] : 0;

    struct Group {
        float x[PER_LANE], w, gw;
        int count[PER_LANE], id, n;
        bool live;
    };
    auto fetch = [&](int t0, Group& g) {
        const int t = t0 + row, tc = min(t, p.T - 1);
        load_row<PER_LANE>(p.logits + (size_t)tc * p.E, p.E, j16, p.vec, g.x);
        if constexpr (GATE) {
            const size_t slot = (size_t)tc * p.k + min(j16, p.k - 1);
            g.id = p.ids[slot];
            g.w = p.topk_w[slot];
            g.gw = p.grad_w[slot];
        }
        g.live = t < p.T && (!p.active || p.active[tc]);
        if constexpr (!BALANCE) return;
        int s = 0;
        if (p.offsets) {
            // last segment that starts at or before the token (-1: none), for the wave's four
            // tokens: a 64-way search each
            int at[4] = {0, 0, 0, 0};
            bool none[4] = {false, false, false, false};
            if (few) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int hits = __popcll(__ballot(lane <= p.S && my_offset <= t0 + r));
                    none[r] = hits == 0;
                    at[r] = hits - 1;
                }
            } else {
                for (int n = p.S + 1; n > 1;) {
                    const int step = (n + kWave - 1) / kWave;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int o = at[r] + lane * step;
                        const bool in = lane * step < n && o <= p.S;
                        const int hits = __popcll(__ballot(in && p.offsets[min(o, p.S)] <= t0 + r));
                        none[r] |= hits == 0;
                        at[r] += max(hits - 1, 0) * step;
                    }
                    n = step;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (row == r) s = none[r] || at[r] >= p.S ? -1 : at[r];
        }
        const int sc = max(s, 0);
        g.n = p.tokens[sc];
        if (s < 0) g.n = 0;
        load_row<PER_LANE>(p.counts + (size_t)sc * p.E, p.E, j16, p.vec, g.count);
    };
    auto compute = [&](int t0, Group& in) {
        const int t = t0 + row;
        float pr[PER_LANE], g[PER_LANE];
        softmax_row<PER_LANE>(in.x, in.live, p.E, j16, pr);
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) g[i] = 0.0f;
        if constexpr (BALANCE) {
            const int n = in.live ? in.n : 0;
            const float fe = n > 0 ? (float)p.E / ((float)p.k * (float)n) : 0.0f;
            float f[PER_LANE], dot = 0.0f;
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) {
                f[i] = (n > 0 && j16 * PER_LANE + i < p.E) ? (float)in.count[i] * fe : 0.0f;
                dot += f[i] * pr[i];
            }
            dot = row_total(dot);
            const float c = n > 0 ? scale / (float)n : 0.0f;
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) g[i] = n > 0 ? c * pr[i] * (f[i] - dot) : 0.0f;
        }
        if constexpr (GATE) {
            int id = in.id;
            float w = in.w, gw = in.gw;
            if (!in.live || j16 >= p.k || (unsigned)id >= (unsigned)p.E) {
                id = -1;
                w = gw = 0.0f;
            }
            const float u = row_total(w * gw);
            const float mine = p.gate_all ? w * gw : w * (gw - u);
            // the slots' values meet their experts' lanes through LDS
            float* at = slots[wave * 4 + row];
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) at[j16 * PER_LANE + i] = g[i];
            lds_wave_fence();
            if (id >= 0) atomicAdd(&at[id], mine);
            lds_wave_fence();
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) g[i] = at[j16 * PER_LANE + i];
            lds_wave_fence();
            if (p.gate_all) {
#pragma unroll
                for (int i = 0; i < PER_LANE; ++i) g[i] -= pr[i] * u;
            }
        }
        if (t >= p.T) return;
        float* dst = p.grad + (size_t)t * p.E + j16 * PER_LANE;
        if constexpr (PER_LANE >= 4) {
            if (p.vec) {
#pragma unroll
                for (int i = 0; i < PER_LANE; i += 4)
                    if (j16 * PER_LANE + i < p.E)
                        *(f32x4*)(dst + i) = f32x4{g[i], g[i + 1], g[i + 2], g[i + 3]};
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            if (j16 * PER_LANE + i < p.E) dst[i] = g[i];
    };

    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4; t0 < p.T; t0 += (int64_t)gridDim.x * 16) {
        Group g;
        fetch((int)t0, g);
        compute((int)t0, g);
        if (!MANY) return;
    }
}

// Gradients of the combine, one token per block: each thread takes 8 columns at a time, reads the
// token's gradient once for its k rows.  Bound by memory: 8192 x 4096, k = 2, both gradients, 335 MB,
// 66 us (5.1 TB/s).
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

// Tokens per cell: about 1024 pieces at most (beside one per segment), 512 where few segments' blocks
// add them up (65536 x 64: one segment 13.3 against 15.1 us, 48 segments 15.4 against 14.5); at least
// 16 tokens each.
static int balance_cell(int T, int S) {
    const int64_t turns = S < 8 ? 8192 : 16384;
    return (int)(((int64_t)T + turns - 1) / turns) * 16 + (T == 0 ? 16 : 0);
}

size_t balance_workspace_layout(int T, int E, int S, BalanceParams* p, char* base) {
    const int cell = balance_cell(T, S);
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

static bool in_pieces(int E, const void* a, const void* b) {
    return E % 4 == 0 && (((uintptr_t)a | (uintptr_t)b) & 15) == 0;
}

constexpr int kTotalLaunch = 128;

hipError_t launch_balance(const BalanceParams& args, hipStream_t s) {
    BalanceParams p = args;
    p.vec = in_pieces(p.E, p.logits, nullptr);
    if (p.E <= 16) balance_piece_kernel<1><<<p.pieces, 256, 0, s>>>(p);
    else if (p.E <= 64) balance_piece_kernel<4><<<p.pieces, 256, 0, s>>>(p);
    else if (p.E <= 128) balance_piece_kernel<8><<<p.pieces, 256, 0, s>>>(p);
    else balance_piece_kernel<16><<<p.pieces, 256, 0, s>>>(p);
    const bool launch_total = p.S > kTotalLaunch;
    p.count_in = p.S > 1 && !launch_total;
    balance_segment_kernel<<<p.S, p.pieces / p.S > 64 ? 1024 : 256, 0, s>>>(p);
    if (launch_total) balance_total_kernel<<<1, 1024, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteGradParams& args, hipStream_t s) {
    RouteGradParams p = args;
    p.vec = in_pieces(p.E, p.logits, p.grad) && ((uintptr_t)p.counts & 15) == 0;
    // Every wave counts the segments that have tokens.  From some hundred on (512: 18.7 us either way)
    // the block does, and from 2048 blocks on the blocks take several groups of tokens each: 65536 x
    // 64 of 4096 segments 22.6 against 41.3 us, of 65536 segments 52 against 412.
    const bool many = p.counts && p.S > 512;
    int grid = (int)(((int64_t)p.T + 15) / 16);
    if (many && grid > 2048) grid = 2048;
    auto run = [&](auto gate, auto balance, auto mn) {
        constexpr bool G = decltype(gate)::value, B = decltype(balance)::value, M = decltype(mn)::value;
        if (p.E <= 16) route_backward_kernel<1, G, B, M><<<grid, 256, 0, s>>>(p);
        else if (p.E <= 64) route_backward_kernel<4, G, B, M><<<grid, 256, 0, s>>>(p);
        else if (p.E <= 128) route_backward_kernel<8, G, B, M><<<grid, 256, 0, s>>>(p);
        else route_backward_kernel<16, G, B, M><<<grid, 256, 0, s>>>(p);
    };
    auto go = [&](auto gate, auto balance) {
        if constexpr (decltype(balance)::value) {
            if (many) return run(gate, balance, std::true_type{});
        }
        run(gate, balance, std::false_type{});
    };
    if (p.grad_w && p.counts) go(std::true_type{}, std::true_type{});
    else if (p.grad_w) go(std::true_type{}, std::false_type{});
    else go(std::false_type{}, std::true_type{});
    return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineGradParams& p, hipStream_t s) {
    combine_backward_kernel<<<p.T, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace moe
