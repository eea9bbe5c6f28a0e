// Tile product of the dense linear layer and of its gradients: C[i, j] = sum_r A[i, r] B[j, r]
// over 16-bit operands, fp32 accumulators.  Each operand is stored either with the summed index
// contiguous ("rows": A[i][r]) or with the output index contiguous ("cols": A[r][i]); the three
// products of a linear layer are
//   out[m, n] = sum_k a[m][k] w[n][k]      rows, rows
//   da[m, k]  = sum_n dz[m][n] w[n][k]     rows, cols
//   dw[n, k]  = sum_m dz[m][n] a[m][k]     cols, cols
// so no operand is ever transposed in memory: the matrix core's operand layout (8 consecutive
// summed indices per lane) comes from plain 16-byte LDS reads for "rows" and from the transposing
// LDS read (ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block and receive its columns) for "cols".
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

typedef uint32_t u32x4_on2 __attribute__((ext_vector_type(4), aligned(2)));   // rows of any length
typedef float f32x4_on4 __attribute__((ext_vector_type(4), aligned(4)));

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <int DT>
__device__ __forceinline__ f32x4 mfma_dt(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (DT == MOE_DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int DT> __device__ __forceinline__ float dt_to_f32(uint16_t v) {
    if constexpr (DT == MOE_DT_BF16) return __builtin_bit_cast(float, (uint32_t)v << 16);
    else return (float)__builtin_bit_cast(f16, v);
}
template <int DT> __device__ __forceinline__ uint16_t f32_to_dt(float v) {   // nearest even
    if constexpr (DT == MOE_DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    else return __builtin_bit_cast(uint16_t, (f16)v);
}

// Activations on the fp32 sum and their slopes on the stored argument.  A NaN stays a NaN
// (a maximum with 0 would drop it).
//
// The normal distribution function from erfc(x) = e^(-x^2) P(t), t = 1 / (1 + 0.42 x), x = |z| / sqrt 2:
// P is a least-maximum fit of e^(x^2) erfc(x) in t over 0 <= x <= 9.6 (beyond, e^(-x^2) is 0 in
// fp32), relative error 4e-8; in fp32 the result is within 2.3e-7, and within 2.2e-6 of itself in
// the lower tail.  Half the instructions of erff, which at 8192 x 6400 outputs cost 60 us of
// arithmetic between the products.
__device__ __forceinline__ float gauss_cdf(float z, float& bell) {       // bell = e^(-z^2 / 2)
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.29698485f * fabsf(z));
    float h = 0.078389115f;
    h = h * t - 0.35694963f;
    h = h * t + 0.51032633f;
    h = h * t - 0.20320329f;
    h = h * t + 0.31420779f;
    h = h * t + 0.17730533f;
    h = h * t + 0.24357177f;
    h = h * t + 0.23632675f;
    h = h * t + 2.5940517e-5f;
    bell = __expf(-0.5f * z * z);
    const float q = 0.5f * h * bell;
    return z < 0.0f ? q : 1.0f - q;
}
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
template <int ACT> __device__ __forceinline__ float act_value(float z) {
    float bell;
    if constexpr (ACT == MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;
    else if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid(z);
    else if constexpr (ACT == MOE_ACT_GELU) return z * gauss_cdf(z, bell);
    else return z;
}
template <int ACT> __device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == MOE_ACT_RELU) {
        return z <= 0.0f ? 0.0f : 1.0f;
    } else if constexpr (ACT == MOE_ACT_SILU) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    } else if constexpr (ACT == MOE_ACT_GELU) {
        float bell;
        const float c = gauss_cdf(z, bell);
        return c + z * 0.39894228f * bell;
    } else {
        return 1.0f;
    }
}

constexpr int kBK = 64;                         // summed indices per stage: a 128-byte line of a row

// Tile t in the order the blocks take them: bands of 8 tile rows, column by column, so that the
// tiles in flight share operand rows.
__device__ __forceinline__ void tile_at(const LinearProduct& p, int t, int& tm, int& tn) {
    const int band = t / (8 * p.tiles_n);
    const int high = min(8, p.tiles_m - band * 8);
    const int in = t - band * 8 * p.tiles_n;
    tn = in / high;
    tm = band * 8 + in % high;
}
// Tile of block b of `tiles`.  Hardware block b runs on XCD b % 8, each with its own L2: the tiles
// are cut into 8 contiguous ranges, one per XCD.
__device__ __forceinline__ void tile_of(const LinearProduct& p, int b, int tiles, int& tm, int& tn) {
    const int q = tiles / 8, rem = tiles % 8, x = b % 8;
    tile_at(p, x * q + min(x, rem) + b / 8, tm, tn);
}

// Address past every buffer resource: such a lane's load delivers zeros.
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000);
}

// 16 bytes per lane from memory straight into LDS: lane i's to lds + 16 i.  Issued as an instruction
// of its own: with the builtin the compiler waits for every such load in flight (vmcnt 0) before
// each transposing LDS read, which it cannot tell apart from them.  It has no register result; the
// kernel's own wait and barrier order it before the reads of its buffer.  (The no-op is the wait
// state an LDS load needs after M0 is written; nothing else in these kernels uses M0.)
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 : : "v"(off), "s"(rsrc), "s"(lds) : "memory");
}

// One operand's stage in LDS: OUT output indices x kBK summed indices.
//   rows: row i (128 bytes, 8 chunks of 16) has its chunk c at position c ^ (i & 7), so the rows of
//         a fragment read spread over all banks.
//   cols: row r (2 OUT bytes) has its 32-byte pair p at position p ^ s(r), s(r) made of bits 0-1
//         and 3-4 of r, the bits in which the rows of one transposing read differ.
// The stage is filled by LDS-DMA, whose lanes write consecutive places, so the swizzle is applied
// to the address each lane reads from memory.  Rows and chunks past the matrix read as zeros (the
// buffer resource ends at the last valid element).
template <int OUT, bool COLS, int WAVES>
struct Operand {
    static constexpr int kBytes = OUT * kBK * 2;
    static constexpr int kLoads = kBytes / (1024 * WAVES);     // wave-wide loads per wave
    static_assert(kLoads * 1024 * WAVES == kBytes, "a stage is a whole number of loads");
    static constexpr int CR = COLS ? OUT / 8 : kBK / 8;        // chunks per LDS row
    static constexpr uint32_t kPairMask = COLS ? CR / 2 - 1 : 0;

    const uint16_t* base;    // first element of the tile's first stage
    int64_t ld;
    int outs;                // valid output indices of the tile (1..OUT)
    int red;                 // summed indices in all
    uint32_t off[kLoads];    // byte offset of each load within a stage
    int kchunk[kLoads];      // rows: first summed index of the chunk within the stage

    __device__ __forceinline__ void init(const uint16_t* m, int64_t ld_, int out0, int outs_total,
                                         int red_, int wave, int lane) {
        ld = ld_;
        red = red_;
        outs = min(OUT, outs_total - out0);
        base = COLS ? m + out0 : m + (int64_t)out0 * ld;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (wave * kLoads + i) * kWave + lane;
            const int r = q / CR, pos = q % CR;
            if constexpr (COLS) {
                const uint32_t s = ((r & 3) | (((r >> 3) & 3) << 2)) & kPairMask;
                const int c = pos ^ (int)(s << 1);
                off[i] = c * 8 < outs ? (uint32_t)(r * (uint32_t)ld + c * 8) * 2u : kOutside;
                kchunk[i] = 0;
            } else {
                const int c = pos ^ (r & 7);
                off[i] = (uint32_t)(r * (uint32_t)ld + c * 8) * 2u;
                kchunk[i] = c * 8;
            }
        }
    }

    // The loads of the stage that starts at `from` with `left` summed indices still to come: the
    // buffer resource (empty unless `live`: zeros, and nothing is read), then load i of kLoads into
    // the operand's buffer at LDS address dst.
    __device__ __forceinline__ int64_t step() const { return COLS ? kBK * ld : kBK; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t stage(const uint16_t* from, int left,
                                                            bool live) const {
        const uint32_t n = COLS ? (uint32_t)(min(left, kBK) - 1) * (uint32_t)ld + (uint32_t)outs
                                : (uint32_t)(outs - 1) * (uint32_t)ld + (uint32_t)left;
        return buffer_of(from, live ? n * 2u : 0u);
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, int i, int left, uint32_t dst,
                                         int wave) const {
        load_lds16(rsrc, COLS || kchunk[i] < left ? off[i] : kOutside, dst + (wave * kLoads + i) * 1024);
    }

    // A wave's FR fragments of 16 output indices from `first` (a multiple of 16 FR) on: the offsets
    // of this lane's pieces within a stage's buffer.
    template <int FR>
    struct Reader {
        uint32_t at[COLS ? FR : 2];
        __device__ __forceinline__ void init(int first, int lane) {
            if constexpr (COLS) {
                const int r = 8 * (lane >> 4) + ((lane >> 2) & 3);
                const uint32_t s = (((lane >> 2) & 3) | ((lane >> 4) << 2)) & kPairMask;
#pragma unroll
                for (int f = 0; f < FR; ++f)
                    at[f] = r * (OUT * 2) + (((uint32_t)((first >> 4) + f) ^ s) << 5) + (lane & 3) * 8;
            } else {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    at[ks] = (first + (lane & 15)) * (kBK * 2) +
                             (((ks * 4 + (lane >> 4)) ^ (lane & 7)) * 16);
            }
        }
        // Fragment f, summed indices 32 ks .. 32 ks + 31.
        __device__ __forceinline__ s16x8 read(const char* buf, int f, int ks) const {
            if constexpr (COLS) {
                const char* p = buf + at[f] + ks * (32 * OUT * 2);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * OUT * 2));
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                return *(const s16x8*)(buf + at[ks] + f * (16 * kBK * 2));
            }
        }
    };
};

// ------------------------------------------------------------------------------------
// The linear layer's epilogue on R rows x 8 consecutive columns per lane: row i of the lane is
// row0 + i * step.  Uniform flags are tested once for all of the lane's values, and all residual
// loads are issued before the first is used.
// ------------------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void add16(float (&v)[8], const u32x4& r) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        v[2 * h] += dt_to_f32<DT>((uint16_t)r[h]);
        v[2 * h + 1] += dt_to_f32<DT>((uint16_t)(r[h] >> 16));
    }
}
template <int DT>
__device__ __forceinline__ u32x4 pack16(const float (&v)[8]) {
    u32x4 o;
#pragma unroll
    for (int h = 0; h < 4; ++h)
        o[h] = f32_to_dt<DT>(v[2 * h]) | (uint32_t)f32_to_dt<DT>(v[2 * h + 1]) << 16;
    return o;
}
// 16 bytes of a row that starts on 2 (an odd row length).
__device__ __forceinline__ void store_piece(uint16_t* dst, const u32x4& v) { *(u32x4_on2*)dst = v; }

template <int DT>
__device__ __forceinline__ void load_bias(const LinearEpilogue& e, int col, int n, float (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (e.bias && col + i < n) ? dt_to_f32<DT>(e.bias[col + i]) : 0.0f;
}
template <int ACT, int R>
__device__ __forceinline__ void apply_act(float (&v)[R][8]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[r][i] = act_value<ACT>(v[r][i]);
}

template <int DT, int R>
__device__ __forceinline__ void linear_epilogue(const LinearEpilogue& e, float (&v)[R][8],
                                                const float (&bias)[8], int64_t row0, int step,
                                                int m, int col, int n) {
    const int live = min(8, n - col);                   // columns of this lane, may be <= 0
    const bool vec = live == 8 && e.vec;                // 16-byte aligned pieces throughout
    bool ok[R];
    u32x4 res[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        ok[r] = row0 + r * step < m && live > 0;
        if (e.residual && vec && ok[r])
            res[r] = *(const u32x4*)(e.residual + (row0 + r * step) * e.ldr + col);
    }
    if (e.bias) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] += bias[i];
    }
    if (e.preact) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!ok[r]) continue;
            uint16_t* dst = e.preact + (row0 + r * step) * e.ldp + col;
            if (vec) {
                *(u32x4*)dst = pack16<DT>(v[r]);
            } else if (live == 8) {
                store_piece(dst, pack16<DT>(v[r]));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) dst[i] = f32_to_dt<DT>(v[r][i]);
            }
        }
    }
    if (e.act == MOE_ACT_RELU) apply_act<MOE_ACT_RELU>(v);
    else if (e.act == MOE_ACT_SILU) apply_act<MOE_ACT_SILU>(v);
    else if (e.act == MOE_ACT_GELU) apply_act<MOE_ACT_GELU>(v);
    if (e.residual) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (vec) {
                if (ok[r]) add16<DT>(v[r], res[r]);
            } else if (ok[r]) {
                const uint16_t* src = e.residual + (row0 + r * step) * e.ldr + col;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) v[r][i] += dt_to_f32<DT>(src[i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (!ok[r]) continue;
        if (e.out_f32) {
            float* dst = (float*)e.out + (row0 + r * step) * e.ldo + col;
            if (vec) {
                *(f32x4*)dst = f32x4{v[r][0], v[r][1], v[r][2], v[r][3]};
                *(f32x4*)(dst + 4) = f32x4{v[r][4], v[r][5], v[r][6], v[r][7]};
            } else if (live == 8) {
                *(f32x4_on4*)dst = f32x4{v[r][0], v[r][1], v[r][2], v[r][3]};
                *(f32x4_on4*)(dst + 4) = f32x4{v[r][4], v[r][5], v[r][6], v[r][7]};
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) dst[i] = v[r][i];
            }
        } else {
            uint16_t* dst = (uint16_t*)e.out + (row0 + r * step) * e.ldo + col;
            if (vec) {
                *(u32x4*)dst = pack16<DT>(v[r]);
            } else if (live == 8) {
                store_piece(dst, pack16<DT>(v[r]));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) dst[i] = f32_to_dt<DT>(v[r][i]);
            }
        }
    }
}

}  // namespace moe
