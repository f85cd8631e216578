// gdn_chunk.h -- the key side of a 64-token chunk of the gated delta rule (gfx950): staging,
// decays, the causal Gram tiles and the triangular inverses, built by four producer waves for
// the waves that step the state.
//
// Per chunk (rows t; G_t = sum of the log-decays up to t, inclusive; D_ts = e^{G_t - G_s}):
//   A_ts = beta_t D_ts k_t.k_s  (t > s),  P_ts = D_ts q_t.k_s  (t >= s)
// With ONE decay per token the decays stay off the operands: q and k enter every product as
// they are, and D <= 1 multiplies the accumulators in fp32.  (A decay per key channel has to be
// folded into q and k, which bounds its chunks by the range of e^G; here a chunk can be 64 long
// whatever the decays.)  A chunk of 64 halves both the number of dependent state steps and the
// conversions of the state per token against 32; at 128 its tiles no longer fit LDS twice.
//
// (I + A) is inverted in two 32x32 halves; the block below them stays a product (the state step
// substitutes through it), which costs the state step nothing in matrix operations (6 tiles of
// 32 either way) and saves the producers the third level.  Each 16x16 diagonal block is
// inverted by forward substitution in fp32, one column per lane: the powers of A of a product
// form grow like binomials when keys repeat (A = the all-ones triangle), substitution does not.
// The 32x32 halves are joined by fp32 matrix products.
//
// Sums of log-decays are fp64 (64 values per chunk and head: free) and kept as two floats, so
// that G_t - G_s of near tokens keeps its accuracy behind a strong decay earlier in the chunk.
//
// Fragment conventions: kda_mfma.h.  Column order of the staged key and query rows, and of
// every matrix that contracts over tokens: position 32p + 8g + 4h + i holds column
// 32p + 16h + 4g + i, so one 16-byte read is the operand of a 32-deep step against two stacked
// 16-row accumulator tiles.
#pragma once

#include "gdn_launch.h"
#include "kda_mfma.h"

namespace kda {

constexpr int kGC = 64;  // tokens per chunk

template <int DK>
struct KeyTile {
    static constexpr int RS = 2 * DK + 32;      // row stride, bytes (conflict-free row and transposed reads)
    static constexpr int SIZE = kGC * RS;
    static constexpr int PPT = kGC * DK / 8 / 256;  // 16-byte pieces per producer thread
};
template <int NV>
struct ValueTile {
    static constexpr int RS = 2 * NV + 32;
    static constexpr int SIZE = kGC * RS;
    static constexpr int PIECES = kGC * NV / 8;
    static constexpr int PPT = (PIECES + 255) / 256;
};

// byte of the 4-element group of columns 4c4 .. +3 in a permuted row
__device__ __forceinline__ int perm4(int c4) { return 64 * (c4 >> 3) + 16 * (c4 & 3) + 8 * ((c4 >> 2) & 1); }

// eight bf16 -> the two 8-byte groups of fp16 (or bf16 as they are)
template <bool HALF>
__device__ __forceinline__ void groups8(u32x4 w, u32x2& a, u32x2& b) {
    if constexpr (HALF) {
        a = __builtin_bit_cast(u32x2, to_h4(unpack_bf4(u32x2{w[0], w[1]})));
        b = __builtin_bit_cast(u32x2, to_h4(unpack_bf4(u32x2{w[2], w[3]})));
    } else {
        a = u32x2{w[0], w[1]};
        b = u32x2{w[2], w[3]};
    }
}

// Rows [0, rows) of a chunk of one head: 16-byte pieces, `pieces` per row, zeros behind the
// last row (the buffer's range ends there, so nothing is read).
template <int PPT, int PER_ROW>
__device__ __forceinline__ void load_rows(u32x4 (&dst)[PPT], const bf16* base, int64_t stride, int rows, int tid) {
    const int bytes = rows > 0 ? (int)((rows - 1) * stride) * 2 + PER_ROW * 16 : 0;
    const __amdgpu_buffer_rsrc_t rs = rsrc(base, bytes);
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int e = tid + 256 * i;
        dst[i] = bload16(rs, (uint32_t)((e / PER_ROW) * (int)stride * 2 + (e % PER_ROW) * 16));
    }
}

// [64][DK] rows to LDS, columns permuted
template <int DK, bool HALF>
__device__ __forceinline__ void store_key(unsigned char* tile, const u32x4 (&src)[KeyTile<DK>::PPT], int tid) {
#pragma unroll
    for (int i = 0; i < KeyTile<DK>::PPT; ++i) {
        const int e = tid + 256 * i, row = e / (DK / 8), m = e % (DK / 8);
        u32x2 a, b;
        groups8<HALF>(src[i], a, b);
        lds_st(tile + row * KeyTile<DK>::RS + perm4(2 * m), a);
        lds_st(tile + row * KeyTile<DK>::RS + perm4(2 * m + 1), b);
    }
}

// The decays of a chunk, all in units of log2: lane t of one wave holds token t.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const uint64_t w = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan_f64(double x) {
    x += dpp_f64<0x111, 0xF>(x);  // within rows of 16
    x += dpp_f64<0x112, 0xF>(x);
    x += dpp_f64<0x114, 0xF>(x);
    x += dpp_f64<0x118, 0xF>(x);
    x += dpp_f64<0x142, 0xA>(x);  // lane 15 -> row 1, 47 -> row 3
    x += dpp_f64<0x143, 0xC>(x);  // lane 31 -> rows 2, 3
    return x;
}
// A log-decay below -1000 (its factor is 0 in any case) is taken as -1000, so that sums behind
// it keep their accuracy and -inf - -inf does not arise; NaN stays.
__device__ __forceinline__ double log2_decay(float la) { return (la < -1000.f ? -1000.0 : (double)la) * 1.4426950408889634074; }

// Inverse of the unit lower triangular 16x16 block I + A by forward substitution: lane column
// `col` of the block whose rows start at A (row stride 16 floats); x[i] = row i of that column.
__device__ __forceinline__ void invert16(const float* A, int col, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == col ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(A + 16 * i + 4 * j4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * j4 + j < i) {
                    if (j & 1) s1 = fmaf(-a[j], x[4 * j4 + j], s1);
                    else s = fmaf(-a[j], x[4 * j4 + j], s);
                }
        }
        x[i] = s + s1;
    }
}

// LDS scratch of one half's inverse: A's two diagonal blocks and the block below them (fp32,
// row-major), then the two inverses column by column.
struct InvScratch {
    static constexpr int BLK = 16 * 16 * 4 + 16;
    static constexpr int DIAG = 0, SUB = 2 * BLK, COL = 3 * BLK, SIZE = 5 * BLK;
};

// The 32x32 inverse of one half by one wave: rows[0] = row tile 0's columns 0..15, rows[1] and
// rows[2] = row tile 1's columns 0..15 and 16..31; lane (r, g) gets row r, columns 4g .. 4g+3.
__device__ __forceinline__ void invert32(unsigned char* sc, int lane, f32x4 (&rows)[3]) {
    typedef InvScratch I;
    const int r = lane & 15, g = lane >> 4, b = (lane >> 4) & 1;
    float x[16];
    invert16(reinterpret_cast<const float*>(sc + I::DIAG + b * I::BLK), r, x);
    float* col = reinterpret_cast<float*>(sc + I::COL + b * I::BLK) + 16 * r;
    if (lane < 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(col + 4 * i) = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    const float* ca = reinterpret_cast<const float*>(sc + I::COL);
    const float* cb = reinterpret_cast<const float*>(sc + I::COL + I::BLK);
    f32x4 tb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        rows[0][i] = ca[16 * (4 * g + i) + r];
        tb[i] = cb[16 * (4 * g + i) + r];
    }
    // M = A_10 T_a, then the transpose of -T_b M (its accumulator is a row fragment)
    const f32x4 sub = *reinterpret_cast<const f32x4*>(sc + I::SUB + 64 * r + 16 * g);
    const f32x4 m = Mma<float>::run(sub, *reinterpret_cast<const f32x4*>(ca + 16 * r + 4 * g), zero4());
    rows[1] = -Mma<float>::run(m, tb, zero4());
    rows[2] = tb;
}

// Tiles (it, jt), jt <= it, of the lower triangle of a 4x4 grid of 16x16 tiles, spread over the
// four producer waves (3, 3, 2, 2 tiles)
__device__ __forceinline__ int tri_tiles(int wave) { return wave < 2 ? 3 : 2; }
__device__ __forceinline__ void tri_tile(int wave, int n, int& it, int& jt) {
    const int idx = wave + 4 * n;  // 0..9: (0,0) (1,0) (1,1) (2,0) (2,1) (2,2) (3,0) ..
    it = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
    jt = idx - it * (it + 1) / 2;
}

}  // namespace kda
