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
// Fragment conventions: kda_mfma.h.  A 32-deep operand holds eight consecutive key channels per
// lane group, as they lie in memory: lane (r, g) of step p takes channels 32p + 8g .. +7.  The
// state's accumulator tiles follow: tile 2p + h, row 4g + i is channel 32p + 8g + 4h + i.  Over
// tokens (whose order the triangles fix) a step of 32 stacks two 16-row tiles instead: element
// 4h + i of lane group g is token 16h + 4g + i of the 32.
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

// eight bf16 -> eight fp16 (or bf16 as they are)
template <bool HALF>
__device__ __forceinline__ u32x4 staged8(u32x4 w) {
    if constexpr (!HALF) return w;
    return __builtin_bit_cast(u32x4, to_h8(unpack_bf4(u32x2{w[0], w[1]}), unpack_bf4(u32x2{w[2], w[3]})));
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

__device__ __forceinline__ float bload4f(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
}

// [64][DK] rows to LDS
template <int DK, bool HALF>
__device__ __forceinline__ void store_key(unsigned char* tile, const u32x4 (&src)[KeyTile<DK>::PPT], int tid) {
#pragma unroll
    for (int i = 0; i < KeyTile<DK>::PPT; ++i) {
        const int e = tid + 256 * i;
        lds_st(tile + (e / (DK / 8)) * KeyTile<DK>::RS + (e % (DK / 8)) * 16, staged8<HALF>(src[i]));
    }
}

// The decays of a chunk, all in units of log2: lane t of one wave holds token t.  A log-decay below -1000 (its factor is 0 in any case) is taken as -1000, so that sums behind
// it keep their accuracy and -inf - -inf does not arise; NaN stays.
__device__ __forceinline__ double log2_decay(float la) { return (la < -1000.f ? -1000.0 : (double)la) * 1.4426950408889634074; }

// x[i] += na[i] of lane J of the row of 16 times xj, four rows at once.  The compiler keeps the
// broadcast and the FMA apart (twice the instructions of what bounds the inverse); the two wait
// states cover a DPP read of a register that a VALU instruction has just written.
template <int J>
__device__ __forceinline__ void fma_bcast4(float& x0, float& x1, float& x2, float& x3, float a0, float a1, float a2, float a3,
                                           float xj) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %5, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %7, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "+v"(x0), "+v"(x1), "+v"(x2), "+v"(x3)
        : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "v"(xj), "n"(J));
}

// Inverse of the unit lower triangular 16x16 blocks I + A by forward substitution, one block per
// 16 lanes: lane c holds -A's column c (na[i] = -A[i][c], 0 for i <= c) and gets the inverse's
// column c (x starts as the identity's).  Rows are taken in whole groups of four: above the
// step's row they add 0.
template <int J0, int J1>
__device__ __forceinline__ void invert16(const float (&na)[16], float (&x)[16]) {  // steps J0 .. J1-1 of 15
    unroll<J0, J1>([&](auto J) {
        constexpr int j = decltype(J)::value;
        const float xj = x[j];
#pragma unroll
        for (int i = (j + 1) / 4 * 4; i < 16; i += 4)
            fma_bcast4<j>(x[i], x[i + 1], x[i + 2], x[i + 3], na[i], na[i + 1], na[i + 2], na[i + 3], xj);
    });
}

// LDS scratch of one half's inverse: two 16x16 blocks, column by column
struct InvScratch {
    static constexpr int COL = 80;  // bytes of a column: 16 floats, padded
    static constexpr int BLK = 16 * COL, SIZE = 2 * BLK;
};

__device__ __forceinline__ void wave_lds_sync() {  // this wave's LDS writes before its reads
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Decays and write strengths of the chunk's tokens in LDS: G (log2) as hi and lo floats, beta
struct GateVec {
    static constexpr int HI = 0, LO = 256, BE = 512, SIZE = 768;
};

// D_ts for one row t and the four columns s .. s+3, and for four rows and one column
__device__ __forceinline__ f32x4 decay_row(const unsigned char* gv, int t, int s) {
    const float th = lds_ld<float>(gv + GateVec::HI + 4 * t), tl = lds_ld<float>(gv + GateVec::LO + 4 * t);
    const f32x4 sh = lds_ld<f32x4>(gv + GateVec::HI + 4 * s), sl = lds_ld<f32x4>(gv + GateVec::LO + 4 * s);
    f32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_exp2f((th - sh[i]) + (tl - sl[i]));
    return d;
}
__device__ __forceinline__ f32x4 decay_col(const unsigned char* gv, int t, int s) {
    const float sh = lds_ld<float>(gv + GateVec::HI + 4 * s), sl = lds_ld<float>(gv + GateVec::LO + 4 * s);
    const f32x4 th = lds_ld<f32x4>(gv + GateVec::HI + 4 * t), tl = lds_ld<f32x4>(gv + GateVec::LO + 4 * t);
    f32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_exp2f((th[i] - sh) + (tl[i] - sl));
    return d;
}

// Row fragments of one 16-token tile of a staged tensor (fp16, or bf16 as given), and the
// product of two of them: lane (r, g) of tile_dot(X, Y) holds X_{4g+i} . Y_r
template <int DK, bool HALF = true>
struct TileRows {
    typedef std::conditional_t<HALF, f16x8, bf16x8> E8;
    E8 v[DK / 32];
    __device__ __forceinline__ void load(const unsigned char* tile, int t, int r, int g) {
#pragma unroll
        for (int p = 0; p < DK / 32; ++p) v[p] = lds_ld<E8>(tile + (16 * t + r) * KeyTile<DK>::RS + 64 * p + 16 * g);
    }
};
__device__ __forceinline__ f32x4 mma32(f16x8 a, f16x8 b, f32x4 c) { return mfma32h(a, b, c); }
__device__ __forceinline__ f32x4 mma32(bf16x8 a, bf16x8 b, f32x4 c) { return mfma32(a, b, c); }
template <int DK, bool HALF>
__device__ __forceinline__ f32x4 tile_dot(const TileRows<DK, HALF>& x, const TileRows<DK, HALF>& y) {
    f32x4 c = zero4();
#pragma unroll
    for (int p = 0; p < DK / 32; ++p) c = mma32(x.v[p], y.v[p], c);
    return c;
}

// The 32x32 inverse of one half (rows and columns 32 half .. +31 of A) by one wave, in two
// steps that a barrier may separate.  First A's tiles and the substitution's beginning in its
// diagonal blocks (one per 16 lanes); `sub` is the block below them, lane (r, g): row r,
// columns 4g .. 4g+3.
struct HalfState {
    f32x4 sub;
    float na[16], x[16];
};
constexpr int kHalfSteps = 6;  // of 15 in the first step: the phases it is split over come out even
template <int DK, bool HALF>
__device__ __forceinline__ HalfState half_columns(const unsigned char* Kt, const unsigned char* gv, unsigned char* sc, int half, int lane) {
    typedef InvScratch I;
    const int r = lane & 15, g = lane >> 4, t0 = 32 * half;
    TileRows<DK, HALF> k0, k1;
    k0.load(Kt, 2 * half, r, g);
    k1.load(Kt, 2 * half + 1, r, g);
    f32x4 da = tile_dot(k0, k0), db = tile_dot(k1, k1), sub = tile_dot(k0, k1);
    const f32x4 ba = lds_ld<f32x4>(gv + GateVec::BE + 4 * (t0 + 4 * g));
    const f32x4 bb = lds_ld<f32x4>(gv + GateVec::BE + 4 * (t0 + 16 + 4 * g));
    const float bs = lds_ld<float>(gv + GateVec::BE + 4 * (t0 + 16 + r));
    const f32x4 ea = decay_col(gv, t0 + 4 * g, t0 + r), eb = decay_col(gv, t0 + 16 + 4 * g, t0 + 16 + r);
    const f32x4 es = decay_row(gv, t0 + 16 + r, t0 + 4 * g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // selected, not multiplied: D above the diagonal may be inf
        da[i] = 4 * g + i > r ? -ba[i] * (ea[i] * da[i]) : 0.f;
        db[i] = 4 * g + i > r ? -bb[i] * (eb[i] * db[i]) : 0.f;
        sub[i] = bs * (es[i] * sub[i]);
    }
    lds_st(sc + I::COL * r + 16 * g, da);
    lds_st(sc + I::BLK + I::COL * r + 16 * g, db);
    wave_lds_sync();
    HalfState h;
    h.sub = sub;
    const unsigned char* mine = sc + (g & 1) * I::BLK + I::COL * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 v = lds_ld<f32x4>(mine + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h.na[4 * i + j] = v[j];
            h.x[4 * i + j] = 4 * i + j == r ? 1.f : 0.f;
        }
    }
    invert16<0, kHalfSteps>(h.na, h.x);
    return h;
}
// Then the rest of it and the join.  T: the fragments of the inverse's rows, rows[0]: row tile
// 0, columns 0..15; rows[1], rows[2]: row tile 1, columns 0..15 and 16..31; lane (r, g) gets
// row r, columns 4g .. 4g+3.  TRANSPOSED: those of its transpose, [0] and [1]: row tile 0,
// columns 0..15 and 16..31; [2]: row tile 1, columns 16..31.
template <bool TRANSPOSED>
__device__ __forceinline__ void half_join(unsigned char* sc, HalfState& h, int lane, f32x4 (&T)[3]) {
    typedef InvScratch I;
    const int r = lane & 15, g = lane >> 4;
    invert16<kHalfSteps, 15>(h.na, h.x);
    unsigned char* mine = sc + (g & 1) * I::BLK + I::COL * r;
    if (lane < 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds_st(mine + 16 * i, f32x4{h.x[4 * i], h.x[4 * i + 1], h.x[4 * i + 2], h.x[4 * i + 3]});
    }
    wave_lds_sync();
    f32x4 tb;
#pragma unroll
    for (int i = 0; i < 4; ++i) tb[i] = lds_ld<float>(sc + I::BLK + I::COL * (4 * g + i) + 4 * r);
    // M = A_10 T_a (ta: its column fragment), then -T_b M, transposed by swapping the operands
    const f32x4 ta = lds_ld<f32x4>(sc + I::COL * r + 16 * g);
    const f32x4 m = Mma<float>::run(h.sub, ta, zero4());
    if constexpr (TRANSPOSED) {
        T[0] = ta;
        T[1] = -Mma<float>::run(tb, m, zero4());
        T[2] = lds_ld<f32x4>(sc + I::BLK + I::COL * r + 16 * g);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) T[0][i] = lds_ld<float>(sc + I::COL * (4 * g + i) + 4 * r);
        T[1] = -Mma<float>::run(m, tb, zero4());
        T[2] = tb;
    }
}

// What the backward's launches pass on, per (chunk, value head), as pairs of bf16 (hi plane,
// then lo plane), each plane [dv][*]: the state before the chunk and the gradient of the state
// behind it over key channels, U and dX over the chunk's tokens (order: position 32s + 8g + 4h
// + i holds token 32s + 16h + 4g + i, which is how a wave's registers hold them).
struct BwdSlot {
    __device__ static __forceinline__ int64_t index(int64_t start, int id, int len, int hv, int h, int c) {
        return (start / kGC + id) * hv + (int64_t)h * ((len + kGC - 1) / kGC) + c;
    }
    static constexpr int64_t state(int dk, int dv) { return 2ll * dk * dv; }    // elements
    static constexpr int64_t tokens(int dv) { return 2ll * kGC * dv; }
};

}  // namespace kda
