// Dense linear layer beside the experts: out = act(a w^T + bias) + residual, and its gradients.
#include <type_traits>

#include "linear.hpp"

namespace moe {

// ------------------------------------------------------------------------------------
// Tile product.  A block computes BM x BN outputs with WM x WN waves, 64 summed indices (a stage)
// at a time.  A stage's two halves of 32 alternate between two fragment sets: while one half is
// multiplied the next one is read from LDS, across the stages too, so the matrix cores wait for no
// LDS read.  The barrier therefore sits in the middle of a stage: behind it the next stage has
// landed, and this stage's buffer, its second half read by then, takes the stage after the next.
// ------------------------------------------------------------------------------------
template <int DT, bool ACOLS, bool BCOLS, int BM, int BN, int WM, int WN, int NBUF>
__device__ __forceinline__ void tile_body(const LinearProduct& p, char* lds, int z, int m0, int n0) {
#ifdef __HIP_DEVICE_COMPILE__                  // the host pass has no buffer resources
    constexpr int W = WM * WN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;        // 16x16 subtiles per wave
    using OA = Operand<BM, ACOLS, W>;
    using OB = Operand<BN, BCOLS, W>;
    constexpr int kStage = OA::kBytes + OB::kBytes;

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;

    OA oa;
    OB ob;
    oa.init(p.a, p.lda, m0, p.a_outs, p.red, wave, lane);
    ob.init(p.b, p.ldb, n0, p.b_outs, p.b_red, wave, lane);

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // stages [s0, s1) of parts * per_part
    const int per = (p.red + kBK - 1) / kBK;
    const int total = per * p.parts;
    const int s0 = (int)((int64_t)total * z / p.split), s1 = (int)((int64_t)total * (z + 1) / p.split);
    constexpr int NL = OA::kLoads + OB::kLoads;
    struct Stage {
        __amdgpu_buffer_rsrc_t a, b;
        int left, left_b;
    };
    // The stages in order, each block of an XCD starting an eighth further on and wrapping round:
    // at any moment the XCDs then read different parts of the rows, which spreads their requests
    // over the memory channels (rows a power of two apart share few of them); blocks of one XCD stay
    // together and share its L2.  Stages past the last read as zeros, so that the loop below has
    // no branch and runs a whole number of rounds through the buffers.
    int remain = s1 - s0, cur = s0 + (int)((int64_t)(blockIdx.x % 8) * remain / 8);
    auto next_stage = [&]() {
        const int part = cur >= per ? 1 : 0;
        const int k = cur - part * per;
        const int left = p.red - k * kBK, left_b = p.b_red - k * kBK;
        const Stage st{oa.stage(oa.base + part * p.a_part + k * oa.step(), left, remain > 0),
                       ob.stage(ob.base + k * ob.step(), left_b, remain > 0), left, left_b};
        --remain;
        cur = cur + 1 < s1 ? cur + 1 : s0;
        return st;
    };
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;
    auto load = [&](const Stage& st, int i, int buf) {
        const uint32_t dst = lds0 + buf * kStage;
        if (i < OA::kLoads) oa.load(st.a, i, st.left, dst, wave);
        else ob.load(st.b, i - OA::kLoads, st.left_b, dst + OA::kBytes, wave);
    };
    typename OA::template Reader<TM> ra;
    typename OB::template Reader<TN> rb;
    ra.init(wm * TM * 16, lane);
    rb.init(wn * TN * 16, lane);
    // fragment f (0 .. TN-1: of B, then of A) of half ks of the stage in buffer buf
    auto read = [&](s16x8 (&fa)[TM], s16x8 (&fb)[TN], int f, int buf, int ks) {
        if (f < TN) fb[f] = rb.read(lds + buf * kStage + OA::kBytes, f, ks);
        else fa[f - TN] = ra.read(lds + buf * kStage, f - TN, ks);
    };
    // Multiplies the half in (ca, cb) in TM groups of TN products and reads half ks of buffer buf
    // into (na, nb); `more`: also loads stage st into buffer `into`.  Loads and reads are spread
    // over the groups: issued in one go they fill the memory and LDS queues and stall the wave
    // behind them (1000 cycles a stage in which nothing multiplied).
    auto half = [&](const s16x8 (&ca)[TM], const s16x8 (&cb)[TN], s16x8 (&na)[TM], s16x8 (&nb)[TN],
                    int buf, int ks, bool more, const Stage& st, int into) {
        constexpr int GR = TM - TM / 4;                        // groups with reads
#pragma unroll
        for (int g = 0; g < TM; ++g) {
            if (more) {
#pragma unroll
                for (int i = g * NL / TM; i < (g + 1) * NL / TM; ++i) load(st, i, into);
            }
            if (g < GR) {
#pragma unroll
                for (int f = g * (TM + TN) / GR; f < (g + 1) * (TM + TN) / GR; ++f)
                    read(na, nb, f, buf, ks);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[g][j] = mfma_dt<DT>(cb[j], ca[g], acc[g][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Behind the barrier all but the last `keep` stages that any wave has begun to load have landed,
    // and all LDS reads have been served.
    auto wait_loads = [](auto keep) {
        constexpr int n = decltype(keep)::value * NL;
        static_assert(n < 64, "vmcnt");
        __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);   // vmcnt(n) lgkmcnt(0)
    };
    auto land = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        wait_loads(std::integral_constant<int, NBUF - 2>{});
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    if (s0 < s1) {
        s16x8 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
        Stage st;
#pragma unroll
        for (int b = 0; b < NBUF; ++b) {
            st = next_stage();
#pragma unroll
            for (int i = 0; i < NL; ++i) load(st, i, b);
        }
        wait_loads(std::integral_constant<int, NBUF - 1>{});
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < TM + TN; ++f) read(fa0, fb0, f, 0, 0);
        for (int s = s0; s < s1; s += NBUF) {
#pragma unroll
            for (int b = 0; b < NBUF; ++b) {
                half(fa0, fb0, fa1, fb1, b, 1, false, st, 0);
                st = next_stage();
                land();
                half(fa1, fb1, fa0, fb0, (b + 1) % NBUF, 0, true, st, b);
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0070);                    // nothing may land in LDS any more
    }

    // The accumulators (lane: row lane & 15 of a subtile, columns 4 (lane >> 4) .. + 3) leave
    // through the wave's own piece of LDS, two subtile rows at a time, so that a row's stores are
    // whole cache lines and the epilogue's code stands once.
    constexpr int LPR = TN * 2, RPI = kWave / LPR;             // lanes per row, rows at a time
    constexpr int R = 32 / RPI, RB = R < 2 ? R : 2;            // a lane's rows, as many at once
    constexpr int RS = TN * 16 + 4;                            // fp32 row stride, padded
    static_assert(W * 32 * RS * 4 <= NBUF * kStage && TM % 2 == 0, "epilogue staging");
    __syncthreads();
    float* region = (float*)lds + wave * 32 * RS;
    const int lr = lane / LPR, lc = (lane % LPR) * 8;
    const int col = n0 + wn * TN * 16 + lc;
    float bias[8];
    load_bias<DT>(p.epi, col, p.N, bias);
    for (int h = 0; h < TM; h += 2) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            if (i - h == 0 || i - h == 1)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    *(f32x4*)(region + ((i & 1) * 16 + (lane & 15)) * RS + j * 16 + 4 * (lane >> 4)) =
                        acc[i][j];
        lds_wave_fence();
        for (int r0 = 0; r0 < R; r0 += RB) {
            float v[RB][8];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const float* src = region + ((r0 + r) * RPI + lr) * RS + lc;
                const f32x4 lo = *(const f32x4*)src, hi = *(const f32x4*)(src + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[r][i] = lo[i];
                    v[r][i + 4] = hi[i];
                }
            }
            const int row0 = m0 + (wm * TM + h) * 16 + r0 * RPI + lr;
            if (p.part) {                                      // their rows hold ldpart columns
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const int row = row0 + r * RPI;
                    if (row < p.M && col < p.N) {
                        float* dst = p.part + ((int64_t)z * p.M + row) * p.ldpart + col;
                        *(f32x4*)dst = f32x4{v[r][0], v[r][1], v[r][2], v[r][3]};
                        *(f32x4*)(dst + 4) = f32x4{v[r][4], v[r][5], v[r][6], v[r][7]};
                    }
                }
            } else {
                linear_epilogue<DT, RB>(p.epi, v, bias, row0, RPI, p.M, col, p.N);
            }
        }
        lds_wave_fence();
    }
#endif
}

template <int DT, bool ACOLS, bool BCOLS, int BM, int BN, int WM, int WN, int NBUF>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile_kernel(LinearProduct p) {
    __shared__ __attribute__((aligned(1024))) char lds[(BM + BN) * kBK * 2 * NBUF];
    const int tiles = p.tiles_m * p.tiles_n;
    int tm, tn;
    if constexpr (BM == 256) {
        const int b = blockIdx.x;
        if (p.split == 1 && b >= p.whole) {                    // a quarter of one of the last tiles
            const int q = b - p.whole;
            tile_at(p, p.whole + q / 4, tm, tn);
            const int m0 = tm * BM + (q & 1) * (BM / 2), n0 = tn * BN + (q >> 1 & 1) * (BN / 2);
            if (m0 < p.M && n0 < p.N)
                tile_body<DT, ACOLS, BCOLS, BM / 2, BN / 2, WM, WN, 4>(p, lds, 0, m0, n0);
            return;
        }
    }
    const int z = blockIdx.x / tiles;                          // split of the summed index
    tile_of(p, blockIdx.x - z * tiles, p.split == 1 ? p.whole : tiles, tm, tn);
    tile_body<DT, ACOLS, BCOLS, BM, BN, WM, WN, NBUF>(p, lds, z, tm * BM, tn * BN);
}

// grad_bias of 64 columns from the dz blocks' column sums: a block's G groups of 64 threads take
// every G-th of them, and are then added in order.
template <int DT, int G>
__device__ __forceinline__ void bias_body(const LinearBias& b, int block, float (*red)[64]) {
    const int lane = threadIdx.x & 63, g = threadIdx.x / 64;
    const int col = block * 64 + lane;
    float v = 0.0f;
    if (col < b.N) {
#pragma unroll 8
        for (int i = g; i < b.blocks; i += G) v += b.sums[(int64_t)i * b.N + col];
    }
    red[g][lane] = v;
    __syncthreads();
    if (g == 0 && col < b.N) {
#pragma unroll
        for (int i = 1; i < G; ++i) v += red[i][lane];
        b.out[col] = f32_to_dt<DT>(v);
    }
}
template <int DT>
__global__ __launch_bounds__(1024) void linear_bias_kernel(LinearBias b) {
    __shared__ float red[16][64];
    bias_body<DT, 16>(b, blockIdx.x, red);
}

// Both gradients' products in one launch, 128 x 128 tiles, two blocks per CU: each alone leaves the
// chip half empty where neither fills it (3777 x 1024 x 4096 fp16: 39 + 41 us one after the other, 68
// together).  The last blocks finish the bias gradient.
template <int DT>
__global__ __launch_bounds__(512) void linear_pair_kernel(LinearProduct da, LinearProduct dw, LinearBias b) {
    __shared__ __attribute__((aligned(1024))) char lds[(128 + 128) * kBK * 2 * 2];
    const int na = (da.whole + 7) / 8 * 8;                     // keeps dw's blocks on their XCDs
    int tm, tn;
    if ((int)blockIdx.x < na) {
        if ((int)blockIdx.x >= da.whole) return;
        tile_of(da, blockIdx.x, da.whole, tm, tn);
        tile_body<DT, false, true, 128, 128, 2, 4, 2>(da, lds, 0, tm * 128, tn * 128);
    } else if ((int)blockIdx.x < na + dw.whole) {
        tile_of(dw, blockIdx.x - na, dw.whole, tm, tn);
        tile_body<DT, true, true, 128, 128, 2, 4, 2>(dw, lds, 0, tm * 128, tn * 128);
    } else {
        bias_body<DT, 8>(b, blockIdx.x - na - dw.whole, (float(*)[64])lds);
    }
}

// ------------------------------------------------------------------------------------
// Input gradient of a narrow layer (N <= 64, a router): da = dz w is a write of M x K with next to no
// arithmetic.  A block holds its 256 columns of w in registers (through one LDS stage and the
// transposing reads) and walks down `rows` rows, 16 at a time, the next rows' dz on its way.  The
// four products of a 16 x 64 piece take columns 32 (j / 2) + 8 g + 4 (j % 2) + i (g the lane's
// quarter, j the product, i its result), so a lane ends up with two runs of eight columns and a row's
// four lanes store 64 bytes in a run.  Bound by the write: 8192 x 4096 from 16-bit gradients of 16
// experts, 67 MB, 18.7 us (20.0 us with 16 columns per lane; 30 us in tiles; a fill takes 11.8).
// ------------------------------------------------------------------------------------
#ifdef __HIP_DEVICE_COMPILE__
using ThinW = Operand<256, true, 4>;                           // 256 columns of w, or of a
// w's columns n0 .. n0 + 255 on their way to LDS, and from there as this wave's fragments of them.
__device__ __forceinline__ void thin_load(const LinearProduct& p, int n0, uint32_t lds, int wave, int lane) {
    ThinW ob;
    ob.init(p.b, p.ldb, n0, p.b_outs, p.b_red, wave, lane);
    const auto wb = ob.stage(ob.base, p.b_red, p.b_red > 0);
#pragma unroll
    for (int i = 0; i < ThinW::kLoads; ++i) ob.load(wb, i, p.b_red, lds, wave);
}
template <int H>
__device__ __forceinline__ void thin_weights(const char* lds, int wave, int lane, s16x8 (&w)[H][4]) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 32 * h + 8 * (lane >> 4) + ((lane >> 2) & 3);
            const uint32_t s = (((lane >> 2) & 3) | ((lane >> 4) << 2)) & ThinW::kPairMask;
            const char* q = lds + r * 512 +
                (((uint32_t)(wave * 4 + 2 * (j >> 1) + ((lane >> 1) & 1)) ^ s) << 5) +
                (lane & 1) * 16 + (j & 1) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 4 * 512));
            w[h][j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
}
// The lane's columns of a row: eight from `col` on and eight from col + 32 on.
template <int DT>
__device__ __forceinline__ void thin_store(const LinearProduct& p, const f32x4 (&acc)[4], int64_t row,
                                           int col) {
    uint16_t* dst = (uint16_t*)p.epi.out + row * p.epi.ldo + col;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float v[8] = {acc[2 * c][0], acc[2 * c][1], acc[2 * c][2], acc[2 * c][3],
                            acc[2 * c + 1][0], acc[2 * c + 1][1], acc[2 * c + 1][2], acc[2 * c + 1][3]};
        if (p.epi.vec && col + 32 * c + 8 <= p.N) {
            *(u32x4*)(dst + 32 * c) = pack16<DT>(v);
        } else if (col + 32 * c + 8 <= p.N) {
            store_piece(dst + 32 * c, pack16<DT>(v));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + 32 * c + i < p.N) dst[32 * c + i] = f32_to_dt<DT>(v[i]);
        }
    }
}
#endif

template <int DT>
__global__ __launch_bounds__(256) void linear_thin_kernel(LinearProduct p, int rows) {
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __attribute__((aligned(1024))) char lds[ThinW::kBytes];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = blockIdx.x * 256;
    thin_load(p, n0, (uint32_t)(uintptr_t)(lds_void*)lds, wave, lane);
    // dz: row lane & 15, summed indices 8 (lane >> 4) .. + 7 of each half; past the end zeros
    const int64_t m0 = (int64_t)blockIdx.y * rows;
    const int left = (int)min((int64_t)rows, p.M - m0);
    const int ld = (int)p.lda, kl = 8 * (lane >> 4);
    const uint32_t bytes = ((uint32_t)(left - 1) * ld + p.red) * 2u;
    const auto z0 = buffer_of(p.a + m0 * ld, bytes), z1 = buffer_of(p.a + p.a_part + m0 * ld, bytes);
    auto fetch = [&](int r, s16x8 (&z)[2][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = r + (lane & 15) < left && 32 * h + kl < p.red
                ? (uint32_t)((r + (lane & 15)) * ld + 32 * h + kl) * 2u : kOutside;
            z[0][h] = __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(z0, at, 0, 0));
            z[1][h] = __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(
                z1, p.parts == 2 ? at : kOutside, 0, 0));
        }
    };
    s16x8 z[2][2], nz[2][2];
    fetch(0, z);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    s16x8 w[2][4];
    thin_weights(lds, wave, lane, w);
    const int col = n0 + wave * 64 + (lane >> 4) * 8;
    for (int r = 0; r < left; r += 16) {
        fetch(r + 16, nz);                                     // past the end: nothing is read
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) acc[j] = mfma_dt<DT>(w[h][j], z[0][h], acc[j]);
            if (p.parts == 2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[j] = mfma_dt<DT>(w[h][j], z[1][h], acc[j]);
            }
        }
        const int row = r + (lane & 15);
        if (row < left) thin_store<DT>(p, acc, m0 + row, col);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) z[i][h] = nz[i][h];
    }
#endif
}

// Both gradients of a narrow layer in one pass over the rows: da is written and a is read at the same
// time.  A block has 256 columns (64 a wave) and a share of the rows, 64 at a time through two
// buffers: the stage's dz (both parts) and columns of a land in LDS, da = dz w leaves from
// registers as in the kernel above, and dw += dz^T a stays in registers until the end, one partial sum
// per share.  NO: N rounded up to 32 or 64.  Bound by memory: 8192 x 4096 from 16-bit gradients of 16
// experts, 134 MB, 34 us (the two kernels one after the other 38), of which about 8 us are the first
// loads and the last sums; a third buffer changed nothing.
template <int DT, int NO>
__global__ __launch_bounds__(256) void linear_narrow_kernel(LinearProduct da, LinearProduct dw) {
#ifdef __HIP_DEVICE_COMPILE__
    using OZ = Operand<NO, true, 4>;
    constexpr int kStage = ThinW::kBytes + 2 * OZ::kBytes, NL = ThinW::kLoads + 2 * OZ::kLoads;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = blockIdx.x * 256, z = blockIdx.y;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;
    auto sync = [](auto keep) {                    // all but the last `keep` stages have landed
        constexpr int n = decltype(keep)::value * NL;
        static_assert(n < 64, "vmcnt");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);   // vmcnt(n) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    ThinW oa;
    OZ oz;
    oa.init(dw.b, dw.ldb, n0, dw.b_outs, dw.b_red, wave, lane);
    oz.init(dw.a, dw.lda, 0, dw.a_outs, dw.red, wave, lane);
    const int stages = (dw.red + kBK - 1) / kBK;
    const int s0 = (int)((int64_t)stages * z / dw.split), s1 = (int)((int64_t)stages * (z + 1) / dw.split);
    auto issue = [&](int s, int buf) {             // past the share: nothing is read, zeros
        const bool live = s < s1;
        const int left = live ? dw.red - s * kBK : 0;
        const uint32_t dst = lds0 + buf * kStage;
        const uint16_t* from = oz.base + s * oz.step();
        const auto zh = oz.stage(from, left, live), zl = oz.stage(from + dw.a_part, left, live && dw.parts == 2);
        const auto aa = oa.stage(oa.base + s * oa.step(), left, live);
#pragma unroll
        for (int i = 0; i < OZ::kLoads; ++i) {
            oz.load(zh, i, left, dst + ThinW::kBytes, wave);
            oz.load(zl, i, left, dst + ThinW::kBytes + OZ::kBytes, wave);
        }
#pragma unroll
        for (int i = 0; i < ThinW::kLoads; ++i) oa.load(aa, i, left, dst, wave);
    };
    constexpr int TN = NO / 16;
    typename ThinW::template Reader<4> ra;
    typename OZ::template Reader<TN> rz;
    ra.init(wave * 64, lane);
    rz.init(0, lane);
    f32x4 sum[TN][4];
#pragma unroll
    for (int f = 0; f < TN; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int col = n0 + wave * 64 + (lane >> 4) * 8;
    issue(s0, 0);
    thin_load(da, n0, lds0 + kStage, wave, lane);              // w passes through the other buffer
    sync(std::integral_constant<int, 0>{});
    s16x8 w[NO / 32][4];
    thin_weights(lds + kStage, wave, lane, w);
    sync(std::integral_constant<int, 0>{});
    issue(s0 + 1, 1);
    for (int s = s0; s < s1; ++s) {
        const int buf = (s - s0) & 1;
        const char* base = lds + buf * kStage;
        const char* zbase = base + ThinW::kBytes;
        sync(std::integral_constant<int, 1>{});
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            s16x8 fa[4], fz[2][TN];
#pragma unroll
            for (int f = 0; f < TN; ++f) {
                fz[0][f] = rz.read(zbase, f, ks);
                fz[1][f] = rz.read(zbase + OZ::kBytes, f, ks);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) fa[j] = ra.read(base, j, ks);
#pragma unroll
            for (int f = 0; f < TN; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[f][j] = mfma_dt<DT>(fa[j], fz[0][f], sum[f][j]);
                    if (dw.parts == 2) sum[f][j] = mfma_dt<DT>(fa[j], fz[1][f], sum[f][j]);
                }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {                          // 16 rows of da
            const int r = g * 16 + (lane & 15);
            const uint32_t sw = ((r & 3) | (((r >> 3) & 3) << 2)) & OZ::kPairMask;
            s16x8 zr[2][NO / 32];
#pragma unroll
            for (int h = 0; h < NO / 32; ++h) {
                const uint32_t c = h * 4 + (lane >> 4);
                const char* q = zbase + r * (NO * 2) + (((c >> 1) ^ sw) << 5) + (c & 1) * 16;
                zr[0][h] = *(const s16x8*)q;
                zr[1][h] = *(const s16x8*)(q + OZ::kBytes);
            }
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < NO / 32; ++h) acc[j] = mfma_dt<DT>(w[h][j], zr[0][h], acc[j]);
                if (dw.parts == 2) {
#pragma unroll
                    for (int h = 0; h < NO / 32; ++h) acc[j] = mfma_dt<DT>(w[h][j], zr[1][h], acc[j]);
                }
            }
            const int64_t row = (int64_t)s * kBK + r;
            if (row < da.M) thin_store<DT>(da, acc, row, col);
        }
        // every wave is done with the buffer; the stores count as older than the loads to come
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xc07f);                    // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue(s + 2, buf);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);                        // nothing may land in LDS any more
#pragma unroll
    for (int f = 0; f < TN; ++f) {
        const int n = f * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = n0 + wave * 64 + j * 16 + 4 * (lane >> 4);
            if (n < dw.M && c < dw.ldpart)
                *(f32x4*)(dw.part + ((int64_t)z * dw.M + n) * dw.ldpart + c) = sum[f][j];
        }
    }
#endif
}

// Sums the splits' partial products in their order and applies the epilogue; the blocks past the
// first `blocks` finish a bias gradient.
template <int DT>
__global__ __launch_bounds__(256) void linear_reduce_kernel(LinearProduct p, int blocks, LinearBias b) {
    __shared__ float red[4][64];
    if ((int)blockIdx.x >= blocks) {
        bias_body<DT, 4>(b, blockIdx.x - blocks, red);
        return;
    }
    const int n8 = p.ldpart / 8;
    const int64_t total = (int64_t)p.M * n8;
    for (int64_t i = blockIdx.x * 256 + (int64_t)threadIdx.x; i < total; i += (int64_t)blocks * 256) {
        const int64_t row = i / n8;
        const int col = (int)(i - row * n8) * 8;
        const float* src = p.part + row * p.ldpart + col;
        f32x4 lo = *(const f32x4*)src, hi = *(const f32x4*)(src + 4);
        const int64_t part = (int64_t)p.M * p.ldpart;
        int z = 1;
        for (; z + 15 <= p.split; z += 15) {                   // as many on their way at once
            f32x4 l[15], h[15];
#pragma unroll
            for (int i = 0; i < 15; ++i) {
                l[i] = *(const f32x4*)(src + (z + i) * part);
                h[i] = *(const f32x4*)(src + (z + i) * part + 4);
            }
#pragma unroll
            for (int i = 0; i < 15; ++i) {
                lo += l[i];
                hi += h[i];
            }
        }
#pragma unroll 4
        for (; z < p.split; ++z) {
            lo += *(const f32x4*)(src + z * part);
            hi += *(const f32x4*)(src + z * part + 4);
        }
        float v[1][8], bias[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[0][c] = lo[c];
            v[0][c + 4] = hi[c];
        }
        load_bias<DT>(p.epi, col, p.N, bias);
        linear_epilogue<DT, 1>(p.epi, v, bias, row, 0, p.M, col, p.N);
    }
}

// ------------------------------------------------------------------------------------
// Few rows (M <= 32, decode and verify steps): out = a w^T is one pass over the weights.  A block
// takes 16 weight rows, its waves an even share of K each, straight from memory to registers, four
// stages (8 KB of weights a wave) in flight; the waves' sums meet in LDS in wave order, where the
// epilogue runs, so the product is one launch without a workspace.  Bound by the weights' read and
// its latency: 1 x 4096 x 4096 bf16, 34 MB, 8.8 us (6.5 us at a copy's rate).  Six stages in flight in
// a ring took longer (12.2 us): a wave's share is four stages or fewer here.
// ------------------------------------------------------------------------------------
template <int DT, int MT>
__global__ __launch_bounds__(1024) void linear_stream_kernel(LinearProduct p) {
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ f32x4 sums[16][MT][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
    const int n0 = blockIdx.x * 16;
    const int stages = (p.red + kBK - 1) / kBK;
    const int s0 = (int)((int64_t)stages * wave / waves), s1 = (int)((int64_t)stages * (wave + 1) / waves);
    // rows past the matrices and summed indices past K read as zeros
    const int ld_b = (int)p.ldb, ld_a = (int)p.lda;
    const auto wb = buffer_of(p.b + (int64_t)n0 * ld_b,
                              ((uint32_t)(min(16, p.b_outs - n0) - 1) * ld_b + p.red) * 2u);
    const auto ab = buffer_of(p.a, ((uint32_t)(p.a_outs - 1) * ld_a + p.red) * 2u);
    const int kl = 8 * (lane >> 4);
    const uint32_t wo = (uint32_t)((lane & 15) * ld_b + kl) * 2u;
    const uint32_t ao = (uint32_t)((lane & 15) * ld_a + kl) * 2u;
    const bool w_row = n0 + (lane & 15) < p.b_outs;
    // the epilogue's thread: row t / 2, eight columns
    const int t = threadIdx.x, row = t / 2, c8 = (t & 1) * 8;
    const int col = n0 + c8;
    const bool out = row < p.M && row < 16 * MT && col < p.N;
    float v[1][8] = {}, bias[8] = {};
    if (out) load_bias<DT>(p.epi, col, p.N, bias);
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;                                       // stages in flight
    for (int s = s0; s < s1; s += U) {
        s16x8 w[U][2], a[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + u) * kBK + 32 * h;
                const bool in = s + u < s1 && k + kl < p.red;
                w[u][h] = __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(
                    wb, in && w_row ? wo + k * 2u : kOutside, 0, 0));
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    a[u][h][m] = __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(
                        ab, in && 16 * m + (lane & 15) < p.a_outs ? ao + (uint32_t)(16 * m * ld_a + k) * 2u
                                                                  : kOutside, 0, 0));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m] = mfma_dt<DT>(w[u][h], a[u][h][m], acc[m]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[wave][m][lane] = acc[m];
    __syncthreads();
    if (!out) return;
    // eight columns sit in lanes row + 16 (column / 4)
    const int at = (row & 15) + 16 * (c8 / 4);
#pragma unroll 4
    for (int i = 0; i < waves; ++i) {
        const f32x4 lo = sums[i][row >> 4][at], hi = sums[i][row >> 4][at + 16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[0][c] += lo[c];
            v[0][c + 4] += hi[c];
        }
    }
    linear_epilogue<DT, 1>(p.epi, v, bias, row, 0, p.M, col, p.N);
#endif
}

// Copies up to two 16-bit matrices whose rows cannot be read in 16-byte pieces in place (row length or
// stride not a multiple of 8) into rows of cols8 = cols rounded up to 8, zeros behind; eight values
// per thread.
__global__ __launch_bounds__(256) void linear_pack_kernel(LinearPack a, LinearPack b) {
    const int64_t na = (int64_t)a.rows * (a.cols8 / 8), nb = (int64_t)b.rows * (b.cols8 / 8);
    for (int64_t j = blockIdx.x * 256 + (int64_t)threadIdx.x; j < na + nb; j += (int64_t)gridDim.x * 256) {
        const LinearPack& m = j < na ? a : b;
        const int64_t i = j < na ? j : j - na;
        const int64_t r = i / (m.cols8 / 8);
        const int c = (int)(i - r * (m.cols8 / 8)) * 8;
        const uint16_t* s = m.src + r * m.ld + c;
        u32x4 o;
        if (c + 8 <= m.cols) {
            o = *(const u32x4_on2*)s;
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t lo = c + 2 * h < m.cols ? s[2 * h] : 0;
                const uint32_t hi = c + 2 * h + 1 < m.cols ? s[2 * h + 1] : 0;
                o[h] = lo | hi << 16;
            }
        }
        ((u32x4*)m.dst)[i] = o;
    }
}

// dz = grad * act'(preact) as the 16-bit operand of the gradients' products, and this block's
// column sums of it (fp32, unrounded).  An fp32 gradient is held as two 16-bit parts, dz = hi + lo
// (lo = the rounding error of hi, itself rounded): 16 (bf16) or 22 (fp16) bits of it reach the
// products, which then run over both parts.  A 16-bit gradient through a curved activation is held
// the same way, or with many rows rounded once to its own type (the products take nothing wider):
// each term's error is then at most half a step, and averages to about the output's own rounding.
// A thread takes 8 columns of a row; the block's 256 threads stand 2^lc across the columns and the
// rest down the rows.  Bound by memory: 3840 x 4096 fp16 through ReLU, 94 MB, 17 us (34 us
// with one value per thread at a time).
template <int DT, int ACT>
__device__ __forceinline__ void dz_rows(const LinearDz& p, int col, int64_t row, int64_t step,
                                        float (&sum)[8]) {
    const int live = min(8, p.N - col);
    const bool full = live == 8;                       // 16-byte pieces, on 2 (fp32: on 4) bytes
    for (; row < p.M; row += step) {
        float v[8];
        if (p.grad_f32) {
            const float* src = (const float*)p.grad + row * p.ldg + col;
            if (full) {
                const f32x4_on4 a = *(const f32x4_on4*)src, b = *(const f32x4_on4*)(src + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = a[i];
                    v[i + 4] = b[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = i < live ? src[i] : 0.0f;
            }
        } else {
            const uint16_t* src = (const uint16_t*)p.grad + row * p.ldg + col;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
            if (full) {
                const u32x4 piece = *(const u32x4_on2*)src;
                add16<DT>(v, piece);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) v[i] = dt_to_f32<DT>(src[i]);
            }
        }
        if constexpr (ACT != MOE_ACT_NONE) {
            const uint16_t* src = p.preact + row * p.ldp + col;
            float z[8] = {};
            if (full) {
                const u32x4 piece = *(const u32x4_on2*)src;
                add16<DT>(z, piece);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) z[i] = dt_to_f32<DT>(src[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= act_slope<ACT>(z[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= live) v[i] = 0.0f;
            sum[i] += v[i];
        }
        if (p.dz) {
            uint16_t* dst = p.dz + row * p.cols8 + col;
            const u32x4 hi = pack16<DT>(v);
            *(u32x4*)dst = hi;
            if (p.parts == 2) {
                float h[8] = {}, lo[8];
                add16<DT>(h, hi);
#pragma unroll
                for (int i = 0; i < 8; ++i)          // infinite or NaN: no rounding error to keep
                    lo[i] = h[i] - h[i] == 0.0f ? v[i] - h[i] : 0.0f;
                *(u32x4*)(dst + (int64_t)p.M * p.cols8) = pack16<DT>(lo);
            }
        }
    }
}

template <int DT>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearDz p) {
    __shared__ float red[256][9], red8[256];
    const int across = 1 << p.lc, down = 256 >> p.lc;
    const int tc = threadIdx.x & (across - 1), tr = threadIdx.x >> p.lc;
    const int col = (blockIdx.x * across + tc) * 8;
    const int64_t row = (int64_t)blockIdx.y * down + tr, step = (int64_t)gridDim.y * down;
    float sum[8] = {};
    if (col < p.cols8) {
        if (p.act == MOE_ACT_RELU) dz_rows<DT, MOE_ACT_RELU>(p, col, row, step, sum);
        else if (p.act == MOE_ACT_SILU) dz_rows<DT, MOE_ACT_SILU>(p, col, row, step, sum);
        else if (p.act == MOE_ACT_GELU) dz_rows<DT, MOE_ACT_GELU>(p, col, row, step, sum);
        else dz_rows<DT, MOE_ACT_NONE>(p, col, row, step, sum);
    }
    if (!p.sums && !p.bias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x][i] = sum[i];
    __syncthreads();
    // eight rows of a column per thread, in order, then these sums in order
    const int cols = across * 8, c = threadIdx.x & (cols - 1), g = threadIdx.x / cols;
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) t += red[((g * 8 + r) << p.lc) + (c >> 3)][c & 7];
    red8[threadIdx.x] = t;
    __syncthreads();
    if (g) return;
    for (int i = 1; i < down / 8; ++i) t += red8[i * cols + c];
    const int n = blockIdx.x * cols + c;
    if (n >= p.N) return;
    if (p.bias) p.bias[n] = f32_to_dt<DT>(t);                      // one block down the rows
    else p.sums[(int64_t)blockIdx.y * p.N + n] = t;
}

// ------------------------------------------------------------------------------------ host
namespace {

int grid_for(int64_t items, int per_block) {
    const int64_t want = (items + per_block - 1) / per_block;
    return (int)(want < 1 ? 1 : want > 16384 ? 16384 : want);
}

// The tiles, and what a block of each was measured to take (us): `base` outside the loop over the
// stages (first loads, epilogue), `stage` per 64 summed indices, alone on its CU or with a second
// block on it.  Larger tiles move fewer bytes per product, smaller ones fill the chip with less
// work.  Four stages in LDS instead of two cover the memory's latency where the stage is short and
// the block alone (128 x 128, 2048 x 2048 x 2048: 20.0 against 24.8 us); two blocks of two stages
// do it as well where there are tiles enough (2048 x 4096 x 4096: 65 against 70 us).
struct TileCost {
    int bm, bn, buffers, per_cu;
    double base, stage, base2, stage2;
};
constexpr TileCost kTiles[] = {
    {256, 256, 2, 1, 7.0, 1.15, 0.0, 0.0},
    {128, 128, 4, 1, 2.5, 0.50, 0.0, 0.0},
    {128, 128, 2, 2, 3.0, 0.60, 3.5, 0.92},
    {64, 128, 4, 1, 1.5, 0.34, 0.0, 0.0},
    {64, 64, 4, 2, 1.0, 0.245, 1.3, 0.38},
};
constexpr int kCus = 256;
// linear_stream_kernel instead of a tile, for products of up to 32 rows and kStreamMost terms.  On
// the device (bf16, us, stream against tile): 1 x 4096 x 4096 8.8 / 12.0, 17 x 2048 x 2048 8.7 / 8.7,
// 16 x 4096 x 4096 11.4 / 12.5, 16 x 4096 x 6400 20.0 / 15.6 -- and one launch less on the host.
constexpr int kStream = 100, kThin = 101;            // kThin: linear_thin_kernel
constexpr int64_t kStreamMost = (int64_t)1 << 28;
constexpr int kNarrowBlocks = 256;

// Waves per block: about 4096 in all, 4 to 16 a block, at most one per stage of K.
template <int DT>
void launch_stream(const LinearProduct& p, hipStream_t s) {
    const int stages = (p.red + kBK - 1) / kBK, grid = (p.N + 15) / 16;
    int waves = 4096 / grid;
    waves = waves < 4 ? 4 : waves > 16 ? 16 : waves;
    if (waves > stages) waves = stages;
    if (p.M <= 16) linear_stream_kernel<DT, 1><<<grid, waves * kWave, 0, s>>>(p);
    else linear_stream_kernel<DT, 2><<<grid, waves * kWave, 0, s>>>(p);
}

// About 1024 blocks of at least 64 rows, and at most 2^15 (a block's byte offsets stay below 2^31).
template <int DT>
void launch_thin(const LinearProduct& p, hipStream_t s) {
    const int wide = (p.N + 255) / 256;
    int64_t rows = ((int64_t)p.M * wide / 1024 + 63) / 64 * 64;
    rows = rows < 64 ? 64 : rows > 1 << 15 ? 1 << 15 : rows;
    linear_thin_kernel<DT><<<dim3(wide, (unsigned)((p.M + rows - 1) / rows)), 256, 0, s>>>(p, (int)rows);
}

int bias_blocks(const LinearBias& b) { return b.out ? (b.N + 63) / 64 : 0; }

template <int DT>
void launch_reduce(const LinearProduct& p, const LinearBias& b, hipStream_t s) {
    const int blocks = grid_for((int64_t)p.M * (p.ldpart / 8), 256);
    linear_reduce_kernel<DT><<<blocks + bias_blocks(b), 256, 0, s>>>(p, blocks, b);
}

template <int DT, bool AC, bool BC>
void launch_tiles(const LinearProduct& p, hipStream_t s) {
    const int tiles = p.tiles_m * p.tiles_n;
    const dim3 grid(p.split > 1 ? tiles * p.split : p.whole + 4 * (tiles - p.whole));
    switch (p.cfg) {
        case 0: linear_tile_kernel<DT, AC, BC, 256, 256, 2, 4, 2><<<grid, 512, 0, s>>>(p); break;
        case 1: linear_tile_kernel<DT, AC, BC, 128, 128, 2, 4, 4><<<grid, 512, 0, s>>>(p); break;
        case 2: linear_tile_kernel<DT, AC, BC, 128, 128, 2, 4, 2><<<grid, 512, 0, s>>>(p); break;
        case 3: linear_tile_kernel<DT, AC, BC, 64, 128, 2, 4, 4><<<grid, 512, 0, s>>>(p); break;
        default: linear_tile_kernel<DT, AC, BC, 64, 64, 2, 2, 4><<<grid, 256, 0, s>>>(p); break;
    }
}

}  // namespace

void linear_plan(LinearProduct& p) {
    if (!p.a_cols && !p.b_cols && p.M <= 32 && (int64_t)p.M * p.N * p.red <= kStreamMost) {
        p.cfg = kStream;
        p.split = 1;
        return;
    }
    if (!p.a_cols && p.b_cols && p.red <= kBK && p.lda <= 1 << 14 && (int64_t)p.M * p.N >= 1 << 22) {
        p.cfg = kThin;                       // a write of M x N; a tile's loads and epilogue would not
        p.split = 1;                         // overlap (8192 x 4096 from 16: 30 us in 256 x 256 tiles)
        p.us = 4.0 + 2.0 * p.M * p.N / 4.4e6;
        return;
    }
    const int stages = ((p.red + kBK - 1) / kBK) * p.parts;
    p.ldpart = (p.N + 7) / 8 * 8;
    double best = 1e30;
    for (int c = 0; c < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++c) {
        const TileCost& t = kTiles[c];
        const int tm = (p.M + t.bm - 1) / t.bm, tn = (p.N + t.bn - 1) / t.bn;
        for (int split : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (split > 1 && stages < 2 * split) break;
            int64_t blocks = (int64_t)tm * tn * split;
            if (split > 1 && blocks > 4 * kCus) break;
            const int st = ((stages + split - 1) / split + t.buffers - 1) / t.buffers * t.buffers;
            // rounds of one block, or two, per CU; a split's sums are written and read once more
            // by a launch of their own (4.4 TB/s)
            double us = split > 1 ? 4.5 + 8.0 * split * p.M * (double)p.ldpart / 4.4e6 : 0.0;
            int64_t whole = blocks;
            const int64_t last = blocks % kCus;
            if (c == 0 && split == 1 && blocks > kCus && last <= kCus / 2) {
                whole -= last;                     // the last round in quarters
                us += (double)((4 * last + kCus - 1) / kCus) * (2.5 + 0.55 * st);
            }
            if (t.per_cu == 2) {
                us += (double)(whole / (2 * kCus)) * (t.base2 + t.stage2 * st);
                whole %= 2 * kCus;
                if (whole > kCus) {
                    us += t.base2 + t.stage2 * st;
                    whole = 0;
                }
            }
            us += (double)((whole + kCus - 1) / kCus) * (t.base + t.stage * st);
            if (us < best) {
                best = us;
                p.us = us;
                p.cfg = c;
                p.split = split;
                p.tiles_m = tm;
                p.tiles_n = tn;
                p.whole = tm * tn - (int)(c == 0 && split == 1 && blocks > kCus && last <= kCus / 2 ? last : 0);
            }
        }
    }
}

size_t linear_part_bytes(const LinearProduct& p) {
    return p.split > 1 ? (size_t)p.split * p.M * p.ldpart * 4 : 0;
}

hipError_t launch_linear_product(const LinearProduct& p, int dtype, hipStream_t s) {
    auto go = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.cfg == kStream) launch_stream<DT>(p, s);
        else if (p.cfg == kThin) launch_thin<DT>(p, s);
        else if (!p.a_cols && !p.b_cols) launch_tiles<DT, false, false>(p, s);
        else if (!p.a_cols) launch_tiles<DT, false, true>(p, s);
        else launch_tiles<DT, true, true>(p, s);
        if (p.split > 1) launch_reduce<DT>(p, LinearBias{}, s);
    };
    if (dtype == MOE_DT_BF16) go(std::integral_constant<int, MOE_DT_BF16>{});
    else go(std::integral_constant<int, MOE_DT_FP16>{});
    return hipGetLastError();
}

// Whether the gradients' two products (neither split) run as one launch: all tiles at once on the
// chip, and sooner than one after the other.
bool linear_pair(LinearProduct& da, LinearProduct& dw) {
    const TileCost& t = kTiles[2];
    auto tiles = [&](const LinearProduct& p) {
        return (int64_t)((p.M + t.bm - 1) / t.bm) * ((p.N + t.bn - 1) / t.bn);
    };
    auto stages = [](const LinearProduct& p) { return (p.red + kBK - 1) / kBK * p.parts; };
    const int64_t n = tiles(da) + tiles(dw);
    if (n > 2 * kCus - 8) return false;
    const int st = stages(da) > stages(dw) ? stages(da) : stages(dw);
    const double us = n > kCus ? t.base2 + t.stage2 * st : t.base + t.stage * st;
    if (us > da.us + dw.us) return false;
    for (LinearProduct* p : {&da, &dw}) {
        p->tiles_m = (p->M + t.bm - 1) / t.bm;
        p->tiles_n = (p->N + t.bn - 1) / t.bn;
        p->whole = p->tiles_m * p->tiles_n;
        p->split = 1;
        p->part = nullptr;
    }
    return true;
}

hipError_t launch_linear_pair(const LinearProduct& da, const LinearProduct& dw, const LinearBias& b,
                              int dtype, hipStream_t s) {
    const int grid = (da.whole + 7) / 8 * 8 + dw.whole + bias_blocks(b);
    if (dtype == MOE_DT_BF16) linear_pair_kernel<MOE_DT_BF16><<<grid, 512, 0, s>>>(da, dw, b);
    else linear_pair_kernel<MOE_DT_FP16><<<grid, 512, 0, s>>>(da, dw, b);
    return hipGetLastError();
}

// The gradients of a narrow layer as one pass: up to 256 blocks (512 blocks: 8192 x 4096 x 64 50
// against 43 us), a share of at least two stages each.  Not for small layers, whose two launches are as
// soon done (both gradients, us, one pass against two launches: 4096 x 2048 x 60 28.6 / 27.0, 8192 x 2048 x
// 16 26.7 / 25.8, 2048 x 4096 x 16 from fp32 20.2 / 22.8, 65536 x 2048 x 64 137 / 195).
int linear_narrow_split(int M, int K) {
    const int stages = (M + kBK - 1) / kBK, wide = (K + 255) / 256;
    const int want = kNarrowBlocks / wide, most = stages / 2;
    const int split = want < most ? want : most;
    return split > 1 ? split : 1;
}
size_t linear_narrow_bytes(const LinearProduct& da, const LinearProduct& dw) {
    if (da.cfg != kThin || (int64_t)da.M * da.N < (dw.M <= 32 ? 1 << 23 : 1 << 24)) return 0;
    return (size_t)linear_narrow_split(da.M, da.N) * dw.M * ((dw.N + 7) / 8 * 8) * 4;
}
hipError_t launch_linear_narrow(const LinearProduct& da, LinearProduct dw, const LinearBias& b,
                                int dtype, hipStream_t s) {
    dw.split = linear_narrow_split(da.M, da.N);
    dw.ldpart = (dw.N + 7) / 8 * 8;
    const dim3 grid((da.N + 255) / 256, dw.split);
    auto go = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (dw.M <= 32) linear_narrow_kernel<DT, 32><<<grid, 256, 0, s>>>(da, dw);
        else linear_narrow_kernel<DT, 64><<<grid, 256, 0, s>>>(da, dw);
        launch_reduce<DT>(dw, b, s);
    };
    if (dtype == MOE_DT_BF16) go(std::integral_constant<int, MOE_DT_BF16>{});
    else go(std::integral_constant<int, MOE_DT_FP16>{});
    return hipGetLastError();
}

hipError_t launch_linear_pack(const LinearPack& a, const LinearPack& b, hipStream_t s) {
    const int64_t n = (int64_t)a.rows * (a.cols8 / 8) + (int64_t)b.rows * (b.cols8 / 8);
    if (n == 0) return hipSuccess;
    linear_pack_kernel<<<grid_for(n, 256), 256, 0, s>>>(a, b);
    return hipGetLastError();
}

// Threads of a block across the columns (log 2) and blocks down the rows, about eight blocks per
// CU in all.
static int dz_across(int N) {
    int lc = 0;
    while (lc < 5 && (8 << lc) < N) ++lc;
    return lc;
}
int linear_dz_blocks(int M, int N) {
    const int lc = dz_across(N), down = 256 >> lc;
    const int64_t wide = ((int64_t)N + (8 << lc) - 1) / (8 << lc);
    const int64_t rows = ((int64_t)M + down - 1) / down;
    int64_t want = (2048 + wide - 1) / (wide < 1 ? 1 : wide);
    if (want > 256) want = 256;
    // few rows per thread: one block, which writes the bias gradient itself (a launch less)
    return (int)(rows <= 4 ? 1 : rows < want ? rows : want);
}

hipError_t launch_linear_bias(const LinearBias& b, int dtype, hipStream_t s) {
    if (!b.out) return hipSuccess;
    if (dtype == MOE_DT_BF16) linear_bias_kernel<MOE_DT_BF16><<<bias_blocks(b), 1024, 0, s>>>(b);
    else linear_bias_kernel<MOE_DT_FP16><<<bias_blocks(b), 1024, 0, s>>>(b);
    return hipGetLastError();
}

hipError_t launch_linear_dz(const LinearDz& args, int dtype, uint16_t* grad_bias, LinearBias& rest,
                            hipStream_t s) {
    LinearDz p = args;
    p.lc = dz_across(p.N);
    const int blocks = linear_dz_blocks(p.M, p.N);
    p.bias = blocks == 1 ? grad_bias : nullptr;
    const dim3 grid((p.cols8 / 8 + (1 << p.lc) - 1) >> p.lc, blocks);
    if (grad_bias && blocks > 1) rest = LinearBias{p.sums, blocks, p.N, grad_bias};
    if (dtype == MOE_DT_BF16) linear_dz_kernel<MOE_DT_BF16><<<grid, 256, 0, s>>>(p);
    else linear_dz_kernel<MOE_DT_FP16><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace moe
