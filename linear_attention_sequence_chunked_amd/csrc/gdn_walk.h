// gdn_walk.h -- the walk over a sequence's chunks of the gated delta rule, bf16 inputs, fp32
// state (gfx950): all of the prefill (gdn_prefill.hip), and what the gradients' launches need
// of the forward (gdn_backward.hip).
//
// Per 64-token chunk (gdn_chunk.h for G, D, A, P; S the state before the chunk):
//   Y = K S;  X = beta (V - e^G Y);  (I + A) U = X;
//   O = scale (e^G (Q S) + P U);  S <- e^{G_C} S + K^T (e^{G_C - G} U)
// which is the token recurrence exactly in exact arithmetic.
//
// Workgroup = one (sequence, value head, slice of NV value columns); the slices of a state are
// independent.  Chain waves hold 16 or 32 columns of S each in fp32 accumulators for the whole
// sequence.  An accumulator tile is, register for register, the B operand (and, transposed,
// the A operand) of the next product over the same rows, so S, X and U never leave the
// registers: a chain wave takes only the key side from LDS and never waits for another chain
// wave.  The key side of the chunks to come is built by other waves meanwhile (gdn_chunk.h).
//
// The loop's passes have two phases, each ended by a workgroup barrier (LDS only: loads and
// stores stay in flight).  Pass c:
//              phase A                             phase B
//   stage      K, Q, V of chunk c                  (loads of c+1 in flight)
//   gates      its decays
//   inverse    (I + A)'s halves: join of c-1       tiles and substitution of c
//   gram       P of c-1 within the halves          A and P below the halves of c
//   chain      K S of c-1                          X, U of c-1, the state behind it
//   out        P U of c-2, its rows stored         Q S of c-1
// K, Q, V, the decays and the matrices are double-buffered; S and U reach the out wave as the
// fp16 operands they are, through LDS.  Two forms:
//  * narrow (16 or 32 columns, few chains: the step's latency is the launch's time): every row
//    above has waves of its own (4, 1, 2, 2, one per 16 columns, 1).  The decays' wave is apart
//    from the staging ones, the phase's longest: one sequence of 131072 tokens with 32 heads of
//    128 x 128, 16 columns per workgroup, 3.54 ms (1.73 us a chunk) against 3.73; four of 4096
//    with 16 heads, 32 columns, 153 to 157 us (2.4 us a chunk) either way;
//  * wide (64 or 128 columns): the chain waves (two column blocks each at 128) do the out
//    wave's work on their own registers, and four producer waves stage in phase A and invert
//    or form Gram tiles, two and two, in phase B; more waves would not have the registers.
// SAVE (for the gradients, narrow): no outputs; in the out wave's place a save wave stores each
// chunk's S and U as bf16 pairs.
//
// Precision.  Operands are fp16.  The products that make the state (K S, the solve, K^T U)
// take their fp32 side as a pair hi + lo (22 bits): single operands would leave the fp32 state
// only 3e-4 of its size accurate, bf16 pairs 4e-6; these measure 2e-7.  The readout's operands
// (S, P, U) are single (11 bits), an eighth of the rounding of the bf16 output.  bf16 q, k and
// v are exact in fp16 inside its range.  The rule is linear in (v, S): both run multiplied by
// eight, which keeps the low halves above fp16's subnormals for values down to about 1e-2 and
// the high ones finite up to 8000.
#pragma once

#include "gdn_chunk.h"
#include "gdn_launch.h"

namespace kda {
namespace {

constexpr float kPre = 8.f;  // v and the state are carried times this

template <int DK, int NCB, bool SAVE = false>
struct GCfg {
    static constexpr int KB = DK / 16, KP = DK / 32, NV = 16 * NCB;
    static constexpr bool NARROW = NCB <= 2, OUT = !SAVE;
    static_assert(NARROW || OUT, "states are saved by the narrow form");
    // two column blocks per chain wave at full width, so that an operand read from LDS serves
    // 32 columns; one otherwise (the shortest step)
    static constexpr int CPW = NCB >= 8 ? 2 : 1;
    static constexpr int NCHAIN = NCB / CPW;
    // wave numbers: chain, stage (the wide form's producers), inverse, gram, out, gates
    static constexpr int W_STAGE = NCHAIN, W_INV = NARROW ? W_STAGE + 4 : W_STAGE, W_GRAM = W_INV + 2,
                         W_OUT = W_GRAM + 2, W_GATE = NARROW ? W_OUT + 1 : W_STAGE, WAVES = W_OUT + (NARROW ? 2 : 0),
                         THREADS = 64 * WAVES;
    typedef KeyTile<DK> K;
    typedef ValueTile<NV> V;
    // matrices, as operand fragments (16 bytes per lane): row tiles 0 and 1 of T's upper half,
    // of its lower half, of -A's block below them, hi then lo; P's three blocks
    static constexpr int FR = 1024;
    static constexpr int M_T0 = 0, M_T1 = 4 * FR, M_A = 8 * FR, M_P = 12 * FR, M_SIZE = 18 * FR;
    // vectors over the chunk's tokens: e^G, beta e^G, kPre beta, e^{G_C - G}; e^{G_C}
    static constexpr int V_EG = 0, V_BE = 256, V_B = 512, V_ER = 768, V_GC = 1024, V_SIZE = 1040;
    // operands for the out (save) wave, per column block: S, then U; behind each its low half
    static constexpr int XN = SAVE ? 2 : 1;
    static constexpr int X_S = 0, X_U = XN * KP * FR, X_SIZE = X_U + XN * 2 * FR;
    static constexpr int O_K = 0, O_Q = O_K + 2 * K::SIZE, O_V = O_Q + (OUT ? 2 * K::SIZE : 0), O_M = O_V + 2 * V::SIZE,
                         O_VEC = O_M + 2 * M_SIZE, O_G = O_VEC + 2 * V_SIZE, O_INV = O_G + 2 * GateVec::SIZE,
                         O_X = O_INV + 2 * InvScratch::SIZE, LDS_BYTES = O_X + (NARROW ? NCB * X_SIZE : 0);
    static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
};

struct PArgs {
    const bf16 *q, *k, *v;
    const float *la, *be;
    const float* S0;
    float* Sf;
    bf16* out;
    int64_t qs, ks, vs;
    int hk, hv, dv, slices, groups;
    float scale;
    bf16 *save_s, *save_u;
};

// x = hi + lo in fp16, 22 bits.  `m1` is -1 where the compiler cannot see it: fma(hi, m1, x)
// rounded to fp16 is then one v_fma_mixlo/hi_f16 per element, against a conversion, a
// subtraction and half a conversion if it is written as x - hi.
__device__ __forceinline__ void split4h(f32x4 a, f16x4& hi, f16x4& lo, float m1) {
    hi = to_h4(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = (_Float16)__builtin_fmaf((float)hi[i], m1, a[i]);
}
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, f16x8& hi, f16x8& lo, float m1) {
    f16x4 h0, h1, l0, l1;
    split4h(a, h0, l0, m1);
    split4h(b, h1, l1, m1);
    hi = cat8h(h0, h1);
    lo = cat8h(l0, l1);
}

template <int DK, int NCB, bool SAVE>
__device__ __forceinline__ void gdn_walk(const PArgs& a, const GdnTable& tab, int block) {
    typedef GCfg<DK, NCB, SAVE> C;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    // the slices of one state on one XCD (workgroups go round-robin over eight): they share
    // its keys and queries in that XCD's L2
    const int kk = block >> 3;
    const int group = (kk / a.slices) * 8 + (block & 7), slice = kk % a.slices;
    if (group >= a.groups) return;
    const int si = group / a.hv, h = group % a.hv, hk = h / (a.hv / a.hk);
    const int len = tab.len[si], col0 = slice * C::NV;
    const int64_t start = tab.start[si];
    const int64_t sbase = ((int64_t)tab.id[si] * a.hv + h) * (int64_t)DK * a.dv;
    const int nch = (len + kGC - 1) / kGC;

    auto buf = [&](int off, int size, int c) { return smem + off + (c & 1) * size; };
    // zero the fragments' halves that lie above the diagonal; nothing else writes them
    for (int i = tid; i < 2 * C::M_SIZE / 16; i += C::THREADS)
        lds_st(smem + C::O_M + 16 * i, u32x4{0u, 0u, 0u, 0u});
    lds_barrier();

    constexpr int KB = C::KB, KP = C::KP, CPW = C::CPW;
    const float oscale = a.scale / kPre;
    float m1 = -1.f;
    asm("" : "+s"(m1));
    const int os = a.hv * a.dv;  // output stride (the host bounds 64 rows of it to 32 bits)

    using std::integral_constant;
    // the narrow form's passes come in rounds of the staging ring; those behind the last chunk's
    // only keep the barriers
    constexpr int R = C::NARROW ? 3 : 1;
    const int passes = (nch + R) / R * R;
    auto drain = [&]() {
        for (int c = nch + 1; c < passes; ++c) {
            lds_barrier();
            lds_barrier();
        }
    };
    // ------------------------------------------------------------------ parts of the key side
    struct Staged {
        u32x4 k[C::K::PPT], q[C::K::PPT], v[C::V::PPT];
        float la, be;
    };
    const int st = tid - 64 * C::W_STAGE;  // thread among the staging waves
    // No branch may lie between a load and its use: the compiler would wait for every load in
    // flight there.  So chunks behind the last, and the gates in all waves but one, are loaded over
    // an empty range (nothing is read, the registers get zeros).
    // Each call loads the next chunk (addresses are added up, not multiplied out).
    int rows_left = len, gates_left = len;
    const bf16 *kp = a.k + start * a.ks + (int64_t)hk * DK, *qp = a.q + start * a.qs + (int64_t)hk * DK,
               *vp = a.v + start * a.vs + (int64_t)h * a.dv + col0;
    const float *lap = a.la + start * a.hv + h, *bep = a.be + start * a.hv + h;
    auto load_gates = [&](float& la, float& be) {
        const int rows = min(kGC, gates_left);
        const int gates = wave == C::W_GATE && rows > 0 ? ((rows - 1) * a.hv + 1) * 4 : 0;
        la = bload4f(rsrc(lap, gates), (uint32_t)(lane * a.hv * 4));
        be = bload4f(rsrc(bep, gates), (uint32_t)(lane * a.hv * 4));
        gates_left -= kGC;
        lap += (int64_t)kGC * a.hv;
        bep += (int64_t)kGC * a.hv;
    };
    auto put_gates = [&](float la, float be, int c) {
        const double G = wave_scan_f64(log2_decay(la)), GC = __shfl(G, 63);
        const float hi = (float)G, eg = __builtin_amdgcn_exp2f(hi);
        unsigned char* gv = buf(C::O_G, GateVec::SIZE, c);
        lds_st(gv + GateVec::HI + 4 * lane, hi);
        lds_st(gv + GateVec::LO + 4 * lane, (float)(G - (double)hi));
        lds_st(gv + GateVec::BE + 4 * lane, be);
        unsigned char* vec = buf(C::O_VEC, C::V_SIZE, c);
        lds_st(vec + C::V_EG + 4 * lane, eg);
        lds_st(vec + C::V_BE + 4 * lane, be * eg);
        lds_st(vec + C::V_B + 4 * lane, kPre * be);
        lds_st(vec + C::V_ER + 4 * lane, __builtin_amdgcn_exp2f((float)(GC - G)));
        if (lane == 0) lds_st(vec + C::V_GC, __builtin_amdgcn_exp2f((float)GC));
    };
    auto load = [&](Staged& x) {
        const int rows = min(kGC, rows_left);
        load_rows<C::K::PPT, DK / 8>(x.k, kp, a.ks, rows, st);
        if constexpr (C::OUT) load_rows<C::K::PPT, DK / 8>(x.q, qp, a.qs, rows, st);
        load_rows<C::V::PPT, C::NV / 8>(x.v, vp, a.vs, rows, st);
        if constexpr (!C::NARROW) load_gates(x.la, x.be);
        rows_left -= kGC;
        kp += kGC * a.ks;
        qp += kGC * a.qs;
        vp += kGC * a.vs;
    };
    auto stage = [&](const Staged& x, int c) {
        unsigned char* Vt = buf(C::O_V, C::V::SIZE, c);
        store_key<DK, true>(buf(C::O_K, C::K::SIZE, c), x.k, st);
        if constexpr (C::OUT) store_key<DK, true>(buf(C::O_Q, C::K::SIZE, c), x.q, st);
#pragma unroll
        for (int i = 0; i < C::V::PPT; ++i) {
            const int e = st + 256 * i;
            if (e < C::V::PIECES) lds_st(Vt + (e / (C::NV / 8)) * C::V::RS + (e % (C::NV / 8)) * 16, x.v[i]);
        }
        if constexpr (!C::NARROW) {
            if (wave == C::W_GATE) put_gates(x.la, x.be, c);
        }
    };
    unsigned char* isc = smem + C::O_INV + (wave - C::W_INV) * InvScratch::SIZE;  // inverse waves
    auto columns = [&](int c) {
        return half_columns<DK, true>(buf(C::O_K, C::K::SIZE, c), buf(C::O_G, GateVec::SIZE, c), isc, wave - C::W_INV, lane);
    };
    auto join = [&](HalfState& x, int c) {
        f32x4 rows[3];
        half_join<false>(isc, x, lane, rows);
        unsigned char* d = buf(C::O_M, C::M_SIZE, c) + (wave == C::W_INV ? C::M_T0 : C::M_T1) + 16 * lane;
        const int at[3] = {0, C::FR, C::FR + 8};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            f16x4 hi, lo;
            split4h(rows[i], hi, lo, m1);
            lds_st(d + at[i], hi);
            lds_st(d + at[i] + 2 * C::FR, lo);
        }
    };
    // P's tiles (it, J0 .. J1-1), and -A's where they lie below the halves: lane (r, g) holds
    // row 16 it + r, columns 16 jt + 4g ..  A gram wave keeps the rows of K it needs.
    typedef TileRows<DK> KeyRows[4];
    auto gram_row = [&](const KeyRows& k, auto IT, auto J0, auto J1, int c) {
        constexpr int it = decltype(IT)::value;
        const unsigned char* gv = buf(C::O_G, GateVec::SIZE, c);
        unsigned char* M = buf(C::O_M, C::M_SIZE, c);
        TileRows<DK> qt;
        if constexpr (C::OUT) qt.load(buf(C::O_Q, C::K::SIZE, c), it, r, g);
        unroll<decltype(J0)::value, decltype(J1)::value>([&](auto JT) {
            constexpr int jt = decltype(JT)::value;
            const f32x4 d = decay_row(gv, 16 * it + r, 16 * jt + 4 * g);
            if constexpr (C::OUT) {
                f32x4 p = tile_dot(k[jt], qt);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = it > jt || 4 * g + i <= r ? d[i] * p[i] : 0.f;
                // P: block (rows 32 (it / 2), columns 32 (jt / 2)), row tile it % 2
                lds_st(M + C::M_P + (2 * (it / 2 + jt / 2) + it % 2) * C::FR + 16 * lane + 8 * (jt % 2), to_h4(p));
            }
            if constexpr (it / 2 != jt / 2) {
                const f32x4 x = tile_dot(k[jt], k[it]);
                const float nb = -lds_ld<float>(gv + GateVec::BE + 4 * (16 * it + r));
                f16x4 hi, lo;
                split4h(nb * (d * x), hi, lo, m1);
                unsigned char* m = M + C::M_A + (it % 2) * C::FR + 16 * lane + 8 * (jt % 2);
                lds_st(m, hi);
                lds_st(m + 2 * C::FR, lo);
            }
        });
    };
    constexpr integral_constant<int, 0> i0;
    constexpr integral_constant<int, 1> i1;
    constexpr integral_constant<int, 2> i2;
    constexpr integral_constant<int, 3> i3;
    constexpr integral_constant<int, 4> i4;
    // one chunk's Gram work of gram wave n: the block of A below the halves with P's tiles
    // there, then P's other tiles (needed a phase later)
    auto gram_first = [&](KeyRows& k, auto N, int c) {
        constexpr int it = 2 + decltype(N)::value;
        const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
        k[it].load(Kt, it, r, g);
        k[0].load(Kt, 0, r, g);
        k[1].load(Kt, 1, r, g);
        if constexpr (it == 3 && C::OUT) k[2].load(Kt, 2, r, g);
        gram_row(k, integral_constant<int, it>{}, i0, i2, c);
    };
    auto gram_second = [&](const KeyRows& k, auto N, int c) {
        if constexpr (!C::OUT) return;
        if constexpr (decltype(N)::value == 0) {
            gram_row(k, i2, i2, i3, c);
            gram_row(k, i1, i0, i2, c);
        } else {
            gram_row(k, i3, i2, i4, c);
            gram_row(k, i0, i0, i1, c);
        }
    };

    if (!C::NARROW && wave >= C::W_STAGE) {
        // ---------------------------------------------------------------- wide: producers
        Staged x;
        load(x);
        for (int c = 0; c <= nch; ++c) {
            if (c < nch) {
                stage(x, c);
                load(x);
            }
            lds_barrier();
            if (c < nch) {
                if (wave < C::W_GRAM) {
                    HalfState x = columns(c);
                    join(x, c);
                } else {
                    KeyRows k;
                    if (wave == C::W_GRAM) {
                        gram_first(k, i0, c);
                        gram_second(k, i0, c);
                    } else {
                        gram_first(k, i1, c);
                        gram_second(k, i1, c);
                    }
                }
            }
            lds_barrier();
        }
        return;
    }
    if (C::NARROW && wave >= C::W_STAGE && wave < C::W_INV) {
        // Three chunks of loads in flight.  (Chunks behind the last are staged too: nothing reads
        // them.)
        Staged x[R];
        unroll<0, R>([&](auto J) {
            load(x[decltype(J)::value]);
            __builtin_amdgcn_sched_barrier(0);  // in this order
        });
        for (int c = 0; c < passes; c += R) {
            unroll<0, R>([&](auto J) {
                constexpr int j = decltype(J)::value;
                stage(x[j], c + j);
                load(x[j]);
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
                lds_barrier();
            });
        }
        return;
    }
    if (C::NARROW && wave == C::W_GATE) {
        float la[R], be[R];
        unroll<0, R>([&](auto J) { load_gates(la[decltype(J)::value], be[decltype(J)::value]); });
        for (int c = 0; c < passes; c += R) {
            unroll<0, R>([&](auto J) {
                constexpr int j = decltype(J)::value;
                put_gates(la[j], be[j], c + j);
                load_gates(la[j], be[j]);
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
                lds_barrier();
            });
        }
        return;
    }
    if (C::NARROW && wave >= C::W_INV && wave < C::W_GRAM) {
        HalfState x = {};
        for (int c = 0; c <= nch; ++c) {
            if (c > 0) join(x, c - 1);
            lds_barrier();
            if (c < nch) x = columns(c);
            lds_barrier();
        }
        drain();
        return;
    }
    if (C::NARROW && wave >= C::W_GRAM && wave < C::W_OUT) {
        auto run = [&](auto N) {
            KeyRows k;
            for (int c = 0; c <= nch; ++c) {
                if (c > 0) gram_second(k, N, c - 1);
                lds_barrier();
                if (c < nch) gram_first(k, N, c);
                lds_barrier();
            }
        };
        if (wave == C::W_GRAM) run(i0);
        else run(i1);
        drain();
        return;
    }
    // rows of O^T + (P U)^T of chunk c, scaled and stored: lane (r, g) holds token r of the
    // tile, columns 4g .. 4g+3
    auto finish = [&](f32x4 o, f16x8 u0, f16x8 u1, auto T, int c, int col) {
        constexpr int t = decltype(T)::value;
        const unsigned char* P = buf(C::O_M, C::M_SIZE, c) + C::M_P + 16 * lane;
        o = mfma32h(u0, lds_ld<f16x8>(P + t * C::FR), o);
        if constexpr (t >= 2) o = mfma32h(u1, lds_ld<f16x8>(P + (2 + t) * C::FR), o);
        // rows behind the sequence's last lie outside the buffer's range: not written
        const int rows = min(kGC, len - kGC * c);
        const __amdgpu_buffer_rsrc_t rs = rsrc(a.out + (start + (int64_t)kGC * c) * os + (int64_t)h * a.dv + col0,
                                               ((rows - 1) * os + C::NV) * 2);
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, to_bf4(oscale * o)), rs, 2 * (r * os + 4 * g) + 2 * col,
                                              32 * t * os, 0);
    };
    if constexpr (SAVE) {
        if (wave == C::W_OUT) {
            // eight fp16 pairs (times kPre) of lane's column and channels or tokens -> bf16 pairs
            auto put = [&](bf16* hi, int64_t plane, const unsigned char* x, int lo_off) {
                const f16x8 h = lds_ld<f16x8>(x), l = lds_ld<f16x8>(x + lo_off);
                f32x4 v[2];
                bf16x4 bh[2], bl[2];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = ((float)h[i] + (float)l[i]) * (1.f / kPre);
                split4(v[0], bh[0], bl[0]);
                split4(v[1], bh[1], bl[1]);
                *reinterpret_cast<bf16x8*>(hi) = cat8(bh[0], bh[1]);
                *reinterpret_cast<bf16x8*>(hi + plane) = cat8(bl[0], bl[1]);
            };
            const int64_t slot = BwdSlot::index(start, tab.id[si], len, a.hv, h, 0);
            auto save_u = [&](int c) {
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        put(a.save_u + (slot + c) * BwdSlot::tokens(a.dv) + (int64_t)(col0 + 16 * cb + r) * kGC + 32 * s + 8 * g,
                            (int64_t)kGC * a.dv, smem + C::O_X + cb * C::X_SIZE + C::X_U + s * C::FR + 16 * lane, 2 * C::FR);
            };
            for (int c = 0; c <= nch; ++c) {
                if (c > 1) save_u(c - 2);
                lds_barrier();
                if (c > 0) {
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                        for (int p = 0; p < KP; ++p)
                            put(a.save_s + (slot + c - 1) * BwdSlot::state(DK, a.dv) + (int64_t)(col0 + 16 * cb + r) * DK + 32 * p + 8 * g,
                                (int64_t)DK * a.dv, smem + C::O_X + cb * C::X_SIZE + C::X_S + p * C::FR + 16 * lane, KP * C::FR);
                }
                lds_barrier();
            }
            if (nch > 0) save_u(nch - 1);
            drain();
            return;
        }
    }
    if (C::NARROW && wave == C::W_OUT) {
        f32x4 O[NCB][4];
        auto done = [&](int c) {
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                const unsigned char* x = smem + C::O_X + cb * C::X_SIZE + C::X_U + 16 * lane;
                const f16x8 u0 = lds_ld<f16x8>(x), u1 = lds_ld<f16x8>(x + C::FR);
                unroll<0, 4>([&](auto T) { finish(O[cb][decltype(T)::value], u0, u1, T, c, 16 * cb); });
            }
        };
        for (int c = 0; c <= nch; ++c) {
            if (c > 1) done(c - 2);
            lds_barrier();
            if (c > 0) {
                const unsigned char* Qt = buf(C::O_Q, C::K::SIZE, c - 1);
                const unsigned char* vec = buf(C::O_VEC, C::V_SIZE, c - 1);
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                    for (int t = 0; t < 4; ++t) O[cb][t] = zero4();
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    f16x8 sh[NCB];
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) sh[cb] = lds_ld<f16x8>(smem + C::O_X + cb * C::X_SIZE + p * C::FR + 16 * lane);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const f16x8 qf = lds_ld<f16x8>(Qt + (16 * t + r) * C::K::RS + 64 * p + 16 * g);
#pragma unroll
                        for (int cb = 0; cb < NCB; ++cb) O[cb][t] = mfma32h(sh[cb], qf, O[cb][t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float eg = lds_ld<float>(vec + C::V_EG + 4 * (16 * t + r));
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) O[cb][t] *= eg;
                }
            }
            lds_barrier();
        }
        if (nch > 0) done(nch - 1);
        drain();
        return;
    }

    // ==================================================================== chain waves
    f32x4 S[CPW][KB];
    int ccol[CPW];
    auto channel = [&](int b) { return 32 * (b >> 1) + 8 * g + 4 * (b & 1); };  // of a tile's first row
#pragma unroll
    for (int cb = 0; cb < CPW; ++cb) {
        ccol[cb] = col0 + 16 * (CPW * wave + cb) + r;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[cb][b][i] = a.S0 ? kPre * a.S0[sbase + (int64_t)(channel(b) + i) * a.dv + ccol[cb]] : 0.f;
    }
    const int trj = (lane & 15) >> 2, trq = lane & 3;
    const int tr_k = (4 * g + trj) * C::K::RS + 16 * trq;
    const int tr_v = (4 * g + trj) * C::V::RS + 8 * trq;
    unsigned char* xw = smem + C::O_X + wave * C::X_SIZE + 16 * lane;  // narrow: to the out wave

    // Rows of K (and Q) of step p as operands.  They are read a step ahead, the
    // first before the barrier that starts the chunk's step (they were staged a phase earlier),
    // so LDS latency stays off the chain.
    typedef f16x8 Rows[4];
    auto load_k = [&](Rows& x, int c, int p) {
        const unsigned char* at = buf(C::O_K, C::K::SIZE, c) + r * C::K::RS + 64 * p + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = lds_ld<f16x8>(at + 16 * t * C::K::RS);
    };
    auto load_q = [&](Rows& x, int c, int p) {
        const unsigned char* at = buf(C::O_Q, C::K::SIZE, c) + r * C::K::RS + 64 * p + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = lds_ld<f16x8>(at + 16 * t * C::K::RS);
    };
    Rows kf[2], qf[2];

    __builtin_amdgcn_s_setprio(3);  // the chain's instructions before the others' on its SIMD
    lds_barrier();  // pass 0: chunk 0 is staged
    if (nch > 0) {
        load_k(kf[0], 0, 0);
        if constexpr (!C::NARROW) load_q(qf[0], 0, 0);
    }
    lds_barrier();
    for (int c = 0; c < nch; ++c) {
        const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
        const unsigned char* Vt = buf(C::O_V, C::V::SIZE, c);
        const unsigned char* M = buf(C::O_M, C::M_SIZE, c);
        const unsigned char* vec = buf(C::O_VEC, C::V_SIZE, c);
        auto frag = [&](int off) { return lds_ld<f16x8>(M + off + 16 * lane); };
        auto tokens = [&](int v, int t) { return lds_ld<f32x4>(vec + v + 4 * (t + 4 * g)); };
        // Y = K S (rows of tokens) and (Q S)^T (rows of value columns)
        f32x4 Y[CPW][4], O[CPW][4];
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb)
#pragma unroll
            for (int t = 0; t < 4; ++t) Y[cb][t] = O[cb][t] = zero4();
        // The conversions of step p + 1 are issued between the products of step p: the vector unit works under the matrix
        // unit's time (one sequence of 131072 tokens, 32 heads: 3% less than in front of the products).
        f16x8 sh[2][CPW], sl[2][CPW];
        auto split_state = [&](auto PI) {
            constexpr int p = decltype(PI)::value;
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) split8(S[cb][2 * p], S[cb][2 * p + 1], sh[p % 2][cb], sl[p % 2][cb], m1);
        };
        split_state(i0);
        unroll<0, KP>([&](auto PI) {
            constexpr int p = decltype(PI)::value, k = p % 2;
            if constexpr (p + 1 < KP) {
                load_k(kf[1 - k], c, p + 1);
                if constexpr (!C::NARROW) load_q(qf[1 - k], c, p + 1);
            }
            if constexpr (C::NARROW) lds_st(xw + C::X_S + p * C::FR, sh[k][0]);
            if constexpr (SAVE) lds_st(xw + C::X_S + (KP + p) * C::FR, sl[k][0]);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (p + 1 < KP) split_state(integral_constant<int, p + 1>{});
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) Y[cb][t] = mfma32h(kf[k][t], sh[k][cb], Y[cb][t]);
            if constexpr (!C::NARROW) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int cb = 0; cb < CPW; ++cb) O[cb][t] = mfma32h(sh[k][cb], qf[k][t], O[cb][t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) Y[cb][t] = mfma32h(kf[k][t], sl[k][cb], Y[cb][t]);
            if constexpr (p + 1 < KP) {
#pragma unroll
                for (int n = 0; n < CPW * (C::NARROW ? 8 : 12); ++n) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // a product
                    __builtin_amdgcn_sched_group_barrier(0x002, C::NARROW ? 2 : 1, 0);  // a conversion or two
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        __builtin_amdgcn_sched_barrier(0);  // the products stay in this phase
        lds_barrier();
        // U: the upper half's solve, its substitution into the lower half's rows, that solve.
        // Operands are read before the products they wait for; the upper half's part of the
        // state's update fills the wait for the lower half's.
        struct Half {
            f16x8 h[2], l[2];
        };
        auto load_half = [&](int off) {
            return Half{{frag(off), frag(off + C::FR)}, {frag(off + 2 * C::FR), frag(off + 3 * C::FR)}};
        };
        // X = kPre beta V - beta e^G Y of half s, in place of Y
        struct ValueRows {
            f32x4 b[2], e[2];
            bf16x4 v[CPW][2];
        };
        auto load_values = [&](int s) {
            ValueRows x;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                x.b[t] = tokens(C::V_B, 32 * s + 16 * t);
                x.e[t] = tokens(C::V_BE, 32 * s + 16 * t);
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb)
                    x.v[cb][t] = lds_tr(Vt + tr_v + (32 * s + 16 * t) * C::V::RS + 32 * (CPW * wave + cb));
            }
            return x;
        };
        auto right_side = [&](const ValueRows& x, int s) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb)
                    Y[cb][2 * s + t] = x.b[t] * to_f4(x.v[cb][t]) - x.e[t] * Y[cb][2 * s + t];
        };
        const ValueRows v0 = load_values(0);
        const Half T0 = load_half(C::M_T0);
        const float gc = lds_ld<float>(vec + C::V_GC);
        __builtin_amdgcn_sched_barrier(0);
        const Half A = load_half(C::M_A);
        const ValueRows v1 = load_values(1);
        right_side(v0, 0);
        f32x4 U[CPW][4];
        f16x8 uh[CPW][2], ul[CPW];
        auto solve = [&](const Half& T, int s) {
            f16x8 xh[CPW], xl[CPW];
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) split8(Y[cb][2 * s], Y[cb][2 * s + 1], xh[cb], xl[cb], m1);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) U[cb][2 * s + t] = mfma32h(T.l[t], xh[cb], zero4());
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) U[cb][2 * s + t] = mfma32h(T.h[t], xl[cb], U[cb][2 * s + t]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) U[cb][2 * s + t] = mfma32h(T.h[t], xh[cb], U[cb][2 * s + t]);
        };
        // S += K_s^T (e^{G_C - G} U_s) over the tokens of half s, four tiles of S at a time, the
        // next four's columns of K read meanwhile
        typedef f16x8 Cols[4];
        auto load_cols = [&](Cols& x, int s, int b0) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const unsigned char* at = Kt + tr_k + 32 * s * C::K::RS + 64 * ((b0 + b) >> 1) + 8 * (b & 1);
                x[b] = cat8h(lds_trh(at), lds_trh(at + 16 * C::K::RS));
            }
        };
        Cols kt[2];
        auto update = [&](f32x4 e0, f32x4 e1, auto SI) {
            constexpr int s = decltype(SI)::value;
            f16x8 wh[CPW], wl[CPW];
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) split8(e0 * U[cb][2 * s], e1 * U[cb][2 * s + 1], wh[cb], wl[cb], m1);
            unroll<0, KB / 4>([&](auto GI) {
                constexpr int n = decltype(GI)::value;
                if constexpr (n + 1 < KB / 4) load_cols(kt[1 - n % 2], s, 4 * (n + 1));
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int cb = 0; cb < CPW; ++cb) S[cb][4 * n + b] = mfma32h(kt[n % 2][b], wh[cb], S[cb][4 * n + b]);
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int cb = 0; cb < CPW; ++cb) S[cb][4 * n + b] = mfma32h(kt[n % 2][b], wl[cb], S[cb][4 * n + b]);
            });
        };
        solve(T0, 0);
        __builtin_amdgcn_sched_barrier(0);
        right_side(v1, 1);
        load_cols(kt[0], 0, 0);
        f32x4 e0 = tokens(C::V_ER, 0), e1 = tokens(C::V_ER, 16);
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb)
#pragma unroll
            for (int b = 0; b < KB; ++b) S[cb][b] *= gc;
        __builtin_amdgcn_sched_barrier(0);
        const Half T1 = load_half(C::M_T1);
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb) split8(U[cb][0], U[cb][1], uh[cb][0], ul[cb], m1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) Y[cb][2 + t] = mfma32h(A.h[t], uh[cb][0], Y[cb][2 + t]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) Y[cb][2 + t] = mfma32h(A.h[t], ul[cb], Y[cb][2 + t]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) Y[cb][2 + t] = mfma32h(A.l[t], uh[cb][0], Y[cb][2 + t]);
        update(e0, e1, i0);
        solve(T1, 1);
        __builtin_amdgcn_sched_barrier(0);
        load_cols(kt[0], 1, 0);
        e0 = tokens(C::V_ER, 32);
        e1 = tokens(C::V_ER, 48);
        if constexpr (SAVE) {
            f16x8 l1;
            split8(U[0][2], U[0][3], uh[0][1], l1, m1);
            lds_st(xw + C::X_U + 2 * C::FR, ul[0]);
            lds_st(xw + C::X_U + 3 * C::FR, l1);
        } else {
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) uh[cb][1] = to_h8(U[cb][2], U[cb][3]);
        }
        if constexpr (C::NARROW) {
            lds_st(xw + C::X_U, uh[0][0]);
            lds_st(xw + C::X_U + C::FR, uh[0][1]);
        } else {
            unroll<0, 4>([&](auto T) {
                constexpr int t = decltype(T)::value;
                const float eg = lds_ld<float>(vec + C::V_EG + 4 * (16 * t + r));
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) finish(eg * O[cb][t], uh[cb][0], uh[cb][1], T, c, 16 * (CPW * wave + cb));
            });
        }
        update(e0, e1, i1);
        __builtin_amdgcn_sched_barrier(0);
        if (c + 1 < nch) {
            load_k(kf[0], c + 1, 0);
            if constexpr (!C::NARROW) load_q(qf[0], c + 1, 0);
        }
        lds_barrier();
    }
    drain();
    if (a.Sf) {
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb)
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a.Sf[sbase + (int64_t)(channel(b) + i) * a.dv + ccol[cb]] = S[cb][b][i] * (1.f / kPre);
    }
}

// arguments of a walk over one table's sequences, `nv` columns per workgroup
PArgs walk_args(const GdnPrefillArgs& p) {
    PArgs a = {};
    a.q = (const bf16*)p.q; a.k = (const bf16*)p.k; a.v = (const bf16*)p.v;
    a.la = p.log_alpha; a.be = p.beta; a.S0 = p.initial_state; a.Sf = p.final_state; a.out = (bf16*)p.out;
    a.qs = p.d.qs; a.ks = p.d.ks; a.vs = p.d.vs; a.hk = p.d.hk; a.hv = p.d.hv; a.dv = p.d.dv;
    a.slices = p.d.dv / p.nv; a.groups = p.num_seqs * p.d.hv; a.scale = p.d.scale;
    return a;
}
// (sequence, head) pairs in eights (one per XCD) times their slices
inline int64_t walk_blocks(const GdnPrefillArgs& p) { return ((int64_t)p.num_seqs * p.d.hv + 7) / 8 * 8 * (p.d.dv / p.nv); }

}  // namespace
}  // namespace kda
