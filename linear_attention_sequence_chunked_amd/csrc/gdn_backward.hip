// gdn_backward.hip -- gradients of the chunked gated delta rule, bf16 inputs (gfx950).
//
// Notation of gdn_chunk.h and gdn_prefill.hip, per 64-token chunk; dO carries `scale`.  With
// dS' the gradient of the state behind the chunk:
//   dU = P^T dO + e^{G_C - G} (K dS'),   dX = (I + A)^-T dU,
//   dS = e^{G_C} dS' + Q^T (e^G dO) - K^T (beta e^G dX)
// and, E = D o (dO U^T) (t >= s), F = -beta D o (dX U^T) (t > s), o the elementwise product:
//   dQ = e^G (dO S^T) + E K,   dV = beta dX,
//   dK = -beta e^G (dX S^T) + e^{G_C - G} (U dS'^T) + E^T Q + (F + F^T) K,
//   dbeta_t = dX_t . (V_t - e^G (K S)_t) + sum_s F_ts k_t.k_s / beta_t,
//   dG_t = e^G (dO S^T)_t.q_t - beta e^G (dX S^T)_t.k_t - e^{G_C - G} (U dS'^T)_t.k_t
//          + sum_{s<t} (E_ts q_t.k_s + F_ts k_t.k_s) - sum_{s>t} (E_st q_s.k_t + F_st k_s.k_t),
//   dG_C = e^{G_C} <S, dS'> + sum_t e^{G_C - G} (U dS'^T)_t.k_t,
//   dlog_alpha_t = dG_C + sum over the chunk's s >= t of dG_s.
//
// Two launches.  The first holds two walks, each a latency-bound chain over slices of value
// columns: the forward one (gdn_walk.h, SAVE) stores every chunk's S and U, the one below goes
// backwards over the chunks with dS in registers and stores dS' and dX.  Neither needs the
// other's results, so they run side by side, workgroup by workgroup.  The gradient kernel then
// takes every (chunk, value head) on its own: products over the value columns, then over the
// chunk's tokens.
//
// Precision.  Gradients come at any scale, so their side cannot take fp16 operands: here the
// computed operands are pairs of bf16 (16 bits, 4e-6 of a result's size in all; single ones
// would leave the fp32 gradients 2e-3), q, k, v and dO single ones, which they are.
#include <algorithm>

#include "gdn_walk.h"

namespace kda {
namespace {

__device__ __forceinline__ void pair8(f32x4 a, f32x4 b, bf16x8& hi, bf16x8& lo) {
    bf16x4 h0, h1, l0, l1;
    split4(a, h0, l0);
    split4(b, h1, l1);
    hi = cat8(h0, h1);
    lo = cat8(l0, l1);
}

// ------------------------------------------------------------------------- the walk back

// Column blocks of 16 per workgroup, of both walks.  One block spreads few states over more
// compute units but stages the keys as often: 2048 tokens, 4 heads of 128 x 128: 128 us with one,
// 132 with two; 32 heads: 242 and 192.
constexpr int NCB = 2;

template <int DK>
struct WCfg {
    static constexpr int KB = DK / 16, KP = DK / 32, NV = 16 * NCB;
    // wave numbers: chain (one per 16 columns), stage (4), inverse (2), gram (2), gates
    static constexpr int W_STAGE = NCB, W_INV = W_STAGE + 4, W_GRAM = W_INV + 2, W_GATE = W_GRAM + 2, THREADS = 64 * (W_GATE + 1);
    typedef KeyTile<DK> K;
    typedef ValueTile<NV> V;
    // fragments (a pair: hi, lo): T^T's halves, -A^T's block, P^T's three blocks, two row tiles each
    static constexpr int FR = 1024, PAIR = 2 * FR;
    static constexpr int M_T0 = 0, M_T1 = 2 * PAIR, M_A = 4 * PAIR, M_P = 6 * PAIR, M_SIZE = 12 * PAIR;
    // vectors over the tokens: e^{G_C - G}, -beta e^G, scale e^G; e^{G_C}
    static constexpr int V_ER = 0, V_BG = 256, V_EG = 512, V_GC = 768, V_SIZE = 784;
    static constexpr int O_K = 0, O_Q = O_K + 2 * K::SIZE, O_O = O_Q + 2 * K::SIZE, O_M = O_O + 2 * V::SIZE,
                         O_VEC = O_M + 2 * M_SIZE, O_G = O_VEC + 2 * V_SIZE, O_INV = O_G + 2 * GateVec::SIZE,
                         LDS_BYTES = O_INV + 2 * InvScratch::SIZE;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
};

struct WArgs {
    const bf16 *q, *k, *d_out;
    const float *la, *be, *dSf;
    float* dS0;
    bf16 *sgrads, *dx;
    int64_t qs, ks;
    int hk, hv, dv, slices, groups;
    float scale;
};

// Passes and phases as in the prefill's narrow form, the chunks in reverse order: pass c stages
// chunk nch-1-c; the chain's phase A takes K dS' of the chunk staged a pass before, phase B the
// rest of its step.  P^T is needed a phase earlier than there.
template <int DK>
__device__ __forceinline__ void gdn_walk_back(const WArgs& a, const GdnTable& tab, int block) {
    typedef WCfg<DK> C;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int kk = block >> 3;
    const int group = (kk / a.slices) * 8 + (block & 7), slice = kk % a.slices;
    if (group >= a.groups) return;
    const int si = group / a.hv, h = group % a.hv, hk = h / (a.hv / a.hk);
    const int len = tab.len[si], id = tab.id[si], col0 = slice * C::NV;
    const int64_t start = tab.start[si];
    const int64_t sbase = ((int64_t)id * a.hv + h) * (int64_t)DK * a.dv;
    const int nch = (len + kGC - 1) / kGC;
    const int64_t slot0 = BwdSlot::index(start, id, len, a.hv, h, 0);
    const int os = a.hv * a.dv;

    auto buf = [&](int off, int size, int c) { return smem + off + (c & 1) * size; };
    for (int i = tid; i < 2 * C::M_SIZE / 16; i += C::THREADS)
        lds_st(smem + C::O_M + 16 * i, u32x4{0u, 0u, 0u, 0u});
    lds_barrier();
    auto chunk = [&](int c) { return nch - 1 - c; };

    using std::integral_constant;
    constexpr int R = 3;  // chunks of loads in flight, and the passes' rounds, as in the prefill
    const int passes = (nch + R) / R * R;
    auto drain = [&]() {
        for (int c = nch + 1; c < passes; ++c) {
            lds_barrier();
            lds_barrier();
        }
    };
    if (wave > C::W_GATE) {  // the forward walk has a wave more: this one keeps the barriers
        for (int c = 0; c < passes; ++c) {
            lds_barrier();
            lds_barrier();
        }
        return;
    }
    if (wave >= C::W_STAGE && wave < C::W_INV) {
        struct Staged {
            u32x4 k[C::K::PPT], q[C::K::PPT], o[C::V::PPT];
        };
        Staged x[R];
        const int st = tid - 64 * C::W_STAGE;
        const int64_t at = start + (int64_t)kGC * max(nch - 1, 0);
        const bf16 *kp = a.k + at * a.ks + (int64_t)hk * DK, *qp = a.q + at * a.qs + (int64_t)hk * DK,
                   *op = a.d_out + at * os + (int64_t)h * a.dv + col0;
        // Each call loads the chunk before.  (Those before the first over an empty range: no branch
        // between a load and its use.)
        auto load = [&](Staged& y, int c) {
            const int rows = c < nch ? min(kGC, len - kGC * chunk(c)) : 0;
            load_rows<C::K::PPT, DK / 8>(y.k, kp, a.ks, rows, st);
            load_rows<C::K::PPT, DK / 8>(y.q, qp, a.qs, rows, st);
            load_rows<C::V::PPT, C::NV / 8>(y.o, op, os, rows, st);
            kp -= kGC * a.ks;
            qp -= kGC * a.qs;
            op -= (int64_t)kGC * os;
        };
        auto stage = [&](const Staged& y, int c) {
            unsigned char* Ot = buf(C::O_O, C::V::SIZE, c);
            store_key<DK, false>(buf(C::O_K, C::K::SIZE, c), y.k, st);
            store_key<DK, false>(buf(C::O_Q, C::K::SIZE, c), y.q, st);
#pragma unroll
            for (int i = 0; i < C::V::PPT; ++i) {
                const int e = st + 256 * i;
                if (e < C::V::PIECES) lds_st(Ot + (e / (C::NV / 8)) * C::V::RS + (e % (C::NV / 8)) * 16, y.o[i]);
            }
        };
        unroll<0, R>([&](auto J) {
            load(x[decltype(J)::value], decltype(J)::value);
            __builtin_amdgcn_sched_barrier(0);
        });
        for (int c = 0; c < passes; c += R) {
            unroll<0, R>([&](auto J) {
                constexpr int j = decltype(J)::value;
                stage(x[j], c + j);
                load(x[j], c + j + R);
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
                lds_barrier();
            });
        }
        return;
    }
    if (wave >= C::W_INV && wave < C::W_GRAM) {
        const int n = wave - C::W_INV;
        unsigned char* sc = smem + C::O_INV + n * InvScratch::SIZE;
        HalfState x = {};
        for (int c = 0; c <= nch; ++c) {
            if (c > 0) {
                f32x4 T[3];
                half_join<true>(sc, x, lane, T);
                unsigned char* d = buf(C::O_M, C::M_SIZE, c - 1) + (n ? C::M_T1 : C::M_T0) + 16 * lane;
                const int at[3] = {0, 8, C::PAIR + 8};
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    bf16x4 hi, lo;
                    split4(T[i], hi, lo);
                    lds_st(d + at[i], hi);
                    lds_st(d + at[i] + C::FR, lo);
                }
            }
            lds_barrier();
            if (c < nch) x = half_columns<DK, false>(buf(C::O_K, C::K::SIZE, c), buf(C::O_G, GateVec::SIZE, c), sc, n, lane);
            lds_barrier();
        }
        drain();
        return;
    }
    if (wave == C::W_GATE) {
        float la[R], be[R];
        auto load = [&](float& x, float& y, int c) {
            const int rows = c < nch ? min(kGC, len - kGC * chunk(c)) : 0;
            const int64_t at = start + (int64_t)kGC * max(chunk(c), 0);
            const int gates = rows > 0 ? ((rows - 1) * a.hv + 1) * 4 : 0;
            x = bload4f(rsrc(a.la + at * a.hv + h, gates), (uint32_t)(lane * a.hv * 4));
            y = bload4f(rsrc(a.be + at * a.hv + h, gates), (uint32_t)(lane * a.hv * 4));
        };
        unroll<0, R>([&](auto J) { load(la[decltype(J)::value], be[decltype(J)::value], decltype(J)::value); });
        for (int c = 0; c < passes; c += R) {
            unroll<0, R>([&](auto J) {
                constexpr int j = decltype(J)::value;
                const double G = wave_scan_f64(log2_decay(la[j])), GC = __shfl(G, 63);
                const float hi = (float)G, eg = __builtin_amdgcn_exp2f(hi);
                unsigned char* gv = buf(C::O_G, GateVec::SIZE, c + j);
                lds_st(gv + GateVec::HI + 4 * lane, hi);
                lds_st(gv + GateVec::LO + 4 * lane, (float)(G - (double)hi));
                lds_st(gv + GateVec::BE + 4 * lane, be[j]);
                unsigned char* vec = buf(C::O_VEC, C::V_SIZE, c + j);
                lds_st(vec + C::V_ER + 4 * lane, __builtin_amdgcn_exp2f((float)(GC - G)));
                lds_st(vec + C::V_BG + 4 * lane, -be[j] * eg);
                lds_st(vec + C::V_EG + 4 * lane, a.scale * eg);
                if (lane == 0) lds_st(vec + C::V_GC, __builtin_amdgcn_exp2f((float)GC));
                load(la[j], be[j], c + j + R);
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
                lds_barrier();
            });
        }
        return;
    }
    if (wave >= C::W_GRAM) {
        // P^T's tiles (columns of row tile it of P), and -A^T's below the halves: lane (r, g)
        // holds row 16 jt + r of the transpose, columns 16 it + 4g ..
        auto gram_row = [&](auto IT, auto J0, auto J1, int c) {
            constexpr int it = decltype(IT)::value;
            const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
            const unsigned char* gv = buf(C::O_G, GateVec::SIZE, c);
            unsigned char* M = buf(C::O_M, C::M_SIZE, c) + 16 * lane + 8 * (it % 2);
            TileRows<DK, false> qi, ki;
            qi.load(buf(C::O_Q, C::K::SIZE, c), it, r, g);
            if constexpr (it >= 2 && decltype(J0)::value < 2) ki.load(Kt, it, r, g);
            unroll<decltype(J0)::value, decltype(J1)::value>([&](auto JT) {
                constexpr int jt = decltype(JT)::value;
                TileRows<DK, false> kj;
                kj.load(Kt, jt, r, g);
                const f32x4 d = decay_col(gv, 16 * it + 4 * g, 16 * jt + r);
                f32x4 p = tile_dot(qi, kj);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = it > jt || 4 * g + i >= r ? a.scale * (d[i] * p[i]) : 0.f;
                bf16x4 hi, lo;
                split4(p, hi, lo);
                unsigned char* m = M + C::M_P + (2 * (it / 2 + jt / 2) + jt % 2) * C::PAIR;
                lds_st(m, hi);
                lds_st(m + C::FR, lo);
                if constexpr (it / 2 != jt / 2) {
                    f32x4 x = tile_dot(ki, kj);
                    const f32x4 b = lds_ld<f32x4>(gv + GateVec::BE + 4 * (16 * it + 4 * g));
                    split4(-(b * (d * x)), hi, lo);
                    m = M + C::M_A + (jt % 2) * C::PAIR;
                    lds_st(m, hi);
                    lds_st(m + C::FR, lo);
                }
            });
        };
        constexpr integral_constant<int, 0> i0;
        constexpr integral_constant<int, 1> i1;
        constexpr integral_constant<int, 2> i2;
        constexpr integral_constant<int, 3> i3;
        constexpr integral_constant<int, 4> i4;
        for (int c = 0; c <= nch; ++c) {
            if (c > 0) {
                if (wave == C::W_GRAM) {
                    gram_row(i2, i2, i3, c - 1);
                    gram_row(i1, i0, i2, c - 1);
                } else {
                    gram_row(i3, i2, i4, c - 1);
                    gram_row(i0, i0, i1, c - 1);
                }
            }
            lds_barrier();
            if (c < nch) {
                if (wave == C::W_GRAM) gram_row(i2, i0, i2, c);
                else gram_row(i3, i0, i2, c);
            }
            lds_barrier();
        }
        drain();
        return;
    }

    // ==================================================================== chain waves
    constexpr int KB = C::KB, KP = C::KP;
    const int col = col0 + 16 * wave + r;
    auto channel = [&](int b) { return 32 * (b >> 1) + 8 * g + 4 * (b & 1); };  // of a tile's first row
    f32x4 D[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) D[b][i] = a.dSf ? a.dSf[sbase + (int64_t)(channel(b) + i) * a.dv + col] : 0.f;
    const int trj = (lane & 15) >> 2, trq = lane & 3;
    const int tr_k = (4 * g + trj) * C::K::RS + 16 * trq;
    const int tr_o = (4 * g + trj) * C::V::RS + 8 * trq + 32 * wave;
    const int64_t splane = (int64_t)DK * a.dv, tplane = (int64_t)kGC * a.dv;

    typedef bf16x8 Rows[4];
    auto load_k = [&](Rows& x, int c, int p) {
        const unsigned char* at = buf(C::O_K, C::K::SIZE, c) + r * C::K::RS + 64 * p + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = lds_ld<bf16x8>(at + 16 * t * C::K::RS);
    };
    Rows kf[2];
    __builtin_amdgcn_s_setprio(3);
    lds_barrier();
    if (nch > 0) load_k(kf[0], 0, 0);
    lds_barrier();
    for (int c = 0; c < nch; ++c) {
        const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
        const unsigned char* Qt = buf(C::O_Q, C::K::SIZE, c);
        const unsigned char* Ot = buf(C::O_O, C::V::SIZE, c);
        const unsigned char* M = buf(C::O_M, C::M_SIZE, c);
        const unsigned char* vec = buf(C::O_VEC, C::V_SIZE, c);
        const int64_t slot = slot0 + chunk(c);
        bf16* pd = a.sgrads + slot * BwdSlot::state(DK, a.dv) + (int64_t)col * DK + 8 * g;
        bf16* px = a.dx + slot * BwdSlot::tokens(a.dv) + (int64_t)col * kGC + 8 * g;
        auto frag = [&](int off) { return lds_ld<bf16x8>(M + off + 16 * lane); };
        auto tokens = [&](int v, int t) { return lds_ld<f32x4>(vec + v + 4 * (t + 4 * g)); };
        // Z = K dS', and dS' as it is before the chunk to its slot
        f32x4 Z[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) Z[t] = zero4();
        unroll<0, KP>([&](auto PI) {
            constexpr int p = decltype(PI)::value, k = p % 2;
            if constexpr (p + 1 < KP) {
                load_k(kf[1 - k], c, p + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            bf16x8 dh, dl;
            pair8(D[2 * p], D[2 * p + 1], dh, dl);
            *reinterpret_cast<bf16x8*>(pd + 32 * p) = dh;
            *reinterpret_cast<bf16x8*>(pd + 32 * p + splane) = dl;
#pragma unroll
            for (int t = 0; t < 4; ++t) Z[t] = mfma32(kf[k][t], dh, Z[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t) Z[t] = mfma32(kf[k][t], dl, Z[t]);
        });
        __builtin_amdgcn_sched_barrier(0);  // the products stay in this phase
        lds_barrier();
        struct Pair {
            bf16x8 h, l;
        };
        auto pair = [&](int off) { return Pair{frag(off), frag(off + C::FR)}; };
        // c + (hi + lo)(hi + lo) without lo lo, and c + (hi + lo) x
        auto mul = [&](const Pair& m, bf16x8 xh, bf16x8 xl, f32x4 c) {
            return mfma32(m.h, xh, mfma32(m.h, xl, mfma32(m.l, xh, c)));
        };
        bf16x8 o[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            o[s] = cat8(lds_tr(Ot + tr_o + 32 * s * C::V::RS), lds_tr(Ot + tr_o + (32 * s + 16) * C::V::RS));
        const Pair p2 = pair(C::M_P + 4 * C::PAIR), p3 = pair(C::M_P + 5 * C::PAIR);
        const Pair t2 = pair(C::M_T1), t3 = pair(C::M_T1 + C::PAIR);
        const float gc = lds_ld<float>(vec + C::V_GC);
        f32x4 er[4], bg[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) er[t] = tokens(C::V_ER, 16 * t);
        __builtin_amdgcn_sched_barrier(0);
        // dU of the lower half, its solve
        Z[2] = mfma32(p2.h, o[1], mfma32(p2.l, o[1], er[2] * Z[2]));
        Z[3] = mfma32(p3.h, o[1], mfma32(p3.l, o[1], er[3] * Z[3]));
        const Pair p00 = pair(C::M_P), p01 = pair(C::M_P + C::PAIR), p10 = pair(C::M_P + 2 * C::PAIR), p11 = pair(C::M_P + 3 * C::PAIR);
        bf16x8 zh, zl;
        pair8(Z[2], Z[3], zh, zl);
        f32x4 X[4];
        X[2] = mul(t2, zh, zl, zero4());
        X[3] = mul(t3, zh, zl, zero4());
        // dU of the upper half meanwhile
        Z[0] = mfma32(p00.h, o[0], mfma32(p00.l, o[0], er[0] * Z[0]));
        Z[1] = mfma32(p01.h, o[0], mfma32(p01.l, o[0], er[1] * Z[1]));
        Z[0] = mfma32(p10.h, o[1], mfma32(p10.l, o[1], Z[0]));
        Z[1] = mfma32(p11.h, o[1], mfma32(p11.l, o[1], Z[1]));
        __builtin_amdgcn_sched_barrier(0);
        const Pair a0 = pair(C::M_A), a1 = pair(C::M_A + C::PAIR);
        const Pair t0 = pair(C::M_T0), t1 = pair(C::M_T0 + C::PAIR);
#pragma unroll
        for (int t = 0; t < 4; ++t) bg[t] = tokens(C::V_BG, 16 * t);
        bf16x8 xh, xl;
        pair8(X[2], X[3], xh, xl);
        *reinterpret_cast<bf16x8*>(px + 32) = xh;
        *reinterpret_cast<bf16x8*>(px + 32 + tplane) = xl;
        Z[0] = mul(a0, xh, xl, Z[0]);
        Z[1] = mul(a1, xh, xl, Z[1]);
        // dS <- e^{G_C} dS' + Q_s^T (scale e^G dO)_s + K_s^T (-beta e^G dX)_s, half by half
        typedef bf16x8 Cols[4];
        auto load_cols = [&](Cols& x, const unsigned char* tile, int s, int b0) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const unsigned char* at = tile + tr_k + 32 * s * C::K::RS + 64 * ((b0 + b) >> 1) + 8 * (b & 1);
                x[b] = cat8(lds_tr(at), lds_tr(at + 16 * C::K::RS));
            }
        };
        Cols kt[2];
        auto update = [&](const unsigned char* tile, f32x4 w0, f32x4 w1, int s) {
            bf16x8 wh, wl;
            pair8(w0, w1, wh, wl);
            unroll<0, KB / 4>([&](auto GI) {
                constexpr int n = decltype(GI)::value;
                if constexpr (n + 1 < KB / 4) load_cols(kt[1 - n % 2], tile, s, 4 * (n + 1));
#pragma unroll
                for (int b = 0; b < 4; ++b) D[4 * n + b] = mfma32(kt[n % 2][b], wh, D[4 * n + b]);
#pragma unroll
                for (int b = 0; b < 4; ++b) D[4 * n + b] = mfma32(kt[n % 2][b], wl, D[4 * n + b]);
            });
        };
        auto half = [&](bf16x8 x, int h) {
            return to_f4(h ? bf16x4{x[4], x[5], x[6], x[7]} : bf16x4{x[0], x[1], x[2], x[3]});
        };
#pragma unroll
        for (int b = 0; b < KB; ++b) D[b] *= gc;
        load_cols(kt[0], Qt, 0, 0);
        update(Qt, tokens(C::V_EG, 0) * half(o[0], 0), tokens(C::V_EG, 16) * half(o[0], 1), 0);
        pair8(Z[0], Z[1], zh, zl);
        X[0] = mul(t0, zh, zl, zero4());
        X[1] = mul(t1, zh, zl, zero4());
        __builtin_amdgcn_sched_barrier(0);
        load_cols(kt[0], Qt, 1, 0);
        update(Qt, tokens(C::V_EG, 32) * half(o[1], 0), tokens(C::V_EG, 48) * half(o[1], 1), 1);
        __builtin_amdgcn_sched_barrier(0);
        load_cols(kt[0], Kt, 1, 0);
        update(Kt, bg[2] * X[2], bg[3] * X[3], 1);
        __builtin_amdgcn_sched_barrier(0);
        load_cols(kt[0], Kt, 0, 0);
        pair8(X[0], X[1], xh, xl);
        *reinterpret_cast<bf16x8*>(px) = xh;
        *reinterpret_cast<bf16x8*>(px + tplane) = xl;
        update(Kt, bg[0] * X[0], bg[1] * X[1], 0);
        __builtin_amdgcn_sched_barrier(0);
        if (c + 1 < nch) load_k(kf[0], c + 1, 0);
        lds_barrier();
    }
    drain();
    if (a.dS0) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) a.dS0[sbase + (int64_t)(channel(b) + i) * a.dv + col] = D[b][i];
    }
}

// Both walks: stretches of workgroups, one per compute unit at most, first of the walk back (the
// slower by a sixth), then of the forward one.  Four sequences of 4096 tokens with 16 heads fill
// the card with each walk: 710 us in all, 743 with the walks' workgroups alternating, 711 as
// launches of their own; 517 + 300 + 64 + 1 tokens with 4 heads of 64 x 128 leave it half empty:
// 43 us, 63 as launches of their own.
template <int DK>
struct WalksCfg {
    typedef GCfg<DK, NCB, true> F;
    typedef WCfg<DK> B;
    static constexpr int THREADS = F::THREADS, LDS_BYTES = F::LDS_BYTES > B::LDS_BYTES ? F::LDS_BYTES : B::LDS_BYTES;
    static_assert(THREADS == B::THREADS + 64, "the walk back's spare wave");
};
template <int DK>
__global__ __launch_bounds__((WalksCfg<DK>::THREADS)) void gdn_walks_kernel(const PArgs f, const WArgs b, const GdnTable tab, int stretch) {
    const int s = blockIdx.x / stretch, block = (s >> 1) * stretch + blockIdx.x % stretch;
    if (s & 1) gdn_walk<DK, NCB, true>(f, tab, block);
    else gdn_walk_back<DK>(b, tab, block);
}

// ------------------------------------------------------------------------- the gradients

// Four waves per (chunk, value head).  Products over the value columns in slices of 32: wave
// (wi, wj) has token tiles 2wi, 2wi+1 and half wj of the key channels; the ten tiles of the
// causal triangle are spread 3, 2, 2, 3.
template <int DK>
struct GradCfg {
    static constexpr int KB = DK / 16, KW = KB / 2;        // channel tiles, and per wave
    static constexpr int RSS = 2 * DK + 32, RST = 160, RSO = 80;
    static constexpr int PS = 32 * DK / 8 / 256;           // 16-byte pieces per thread of a slice of S
    // slices (phase 1)
    static constexpr int SH = 0, SL = SH + 32 * RSS, DH = SL + 32 * RSS, DL = DH + 32 * RSS, UH = DL + 32 * RSS,
                         UL = UH + 32 * RST, XH = UL + 32 * RST, XL = XH + 32 * RST, OO = XL + 32 * RST, P1 = OO + kGC * RSO;
    // tiles (phase 2): K, Q, E and F as pairs, row-major
    static constexpr int RSE = 144;
    static constexpr int KT = 0, QT = KeyTile<DK>::SIZE, EH = 2 * KeyTile<DK>::SIZE, EL = EH + kGC * RSE, FH = EL + kGC * RSE,
                         FL = FH + kGC * RSE, P2 = FL + kGC * RSE;
    // vectors: gates; e^G, beta e^G, e^{G_C - G}; sums over rows and columns of tiles (E q.k +
    // F k.k by row tile and column tile, both ways; F k.k / beta by row), per half of the
    // channels the three row dots, dX.V, and <S, dS'> per wave
    static constexpr int VEC = P1 > P2 ? P1 : P2;
    static constexpr int GV = VEC, EG = GV + GateVec::SIZE, BG = EG + 256, ER = BG + 256, ROW = ER + 256, COL = ROW + 1024,
                         BET = COL + 1024, DOT = BET + 1024, XV = DOT + 2 * 3 * 256, TR = XV + 256, LDS_BYTES = TR + 64;
    static_assert(LDS_BYTES <= 80 * 1024, "two workgroups per compute unit");
};

template <int DK, int DV>
__global__ __launch_bounds__(256, 2) void gdn_gradients_kernel(const GdnBackwardArgs A, const GdnTable tab, int from) {
    typedef GradCfg<DK> C;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const GdnDims& d = A.d;
    const int si = from + blockIdx.y, len = tab.len[si], nch = (len + kGC - 1) / kGC;
    const int h = blockIdx.x % d.hv, c = blockIdx.x / d.hv;
    if (c >= nch) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4, wi = wave >> 1, wj = wave & 1;
    const int hk = h / (d.hv / d.hk), rows = min(kGC, len - kGC * c);
    const int64_t t0 = tab.start[si] + (int64_t)kGC * c, slot = BwdSlot::index(tab.start[si], tab.id[si], len, d.hv, h, c);
    const bf16* ps = (const bf16*)A.states + slot * BwdSlot::state(DK, DV);
    const bf16* pd = (const bf16*)A.sgrads + slot * BwdSlot::state(DK, DV);
    const bf16* pu = (const bf16*)A.u + slot * BwdSlot::tokens(DV);
    const bf16* px = (const bf16*)A.dx + slot * BwdSlot::tokens(DV);
    const bf16* po = (const bf16*)A.d_out + t0 * d.hv * DV + (int64_t)h * DV;
    const bf16* pv = (const bf16*)A.v + t0 * d.vs + (int64_t)h * DV;
    const int os = d.hv * DV;
    const int trj = (lane & 15) >> 2, trq = lane & 3;

    if (wave == 0) {
        float la = 0.f, be = 0.f;
        if (lane < rows) {
            la = A.log_alpha[(t0 + lane) * d.hv + h];
            be = A.beta[(t0 + lane) * d.hv + h];
        }
        const double G = wave_scan_f64(log2_decay(la)), GC = __shfl(G, 63);
        const float hi = (float)G, eg = __builtin_amdgcn_exp2f(hi);
        lds_st(smem + C::GV + GateVec::HI + 4 * lane, hi);
        lds_st(smem + C::GV + GateVec::LO + 4 * lane, (float)(G - (double)hi));
        lds_st(smem + C::GV + GateVec::BE + 4 * lane, be);
        lds_st(smem + C::EG + 4 * lane, eg);
        lds_st(smem + C::BG + 4 * lane, be * eg);
        lds_st(smem + C::ER + 4 * lane, __builtin_amdgcn_exp2f((float)(GC - G)));
        if (lane == 0) lds_st(smem + C::TR + 16, __builtin_amdgcn_exp2f((float)GC));
    }
    // ---------------------------------------------------------------- over the value columns
    struct Slice {
        u32x4 s[2][C::PS], d[2][C::PS], u[2], x[2], o[1];
        u32x2 v[2];  // V of token tile `wave`: lane (r, g) has token r, columns 4g .. and 16 + 4g ..
    } y;
    auto load = [&](int n) {
        const int64_t at = (int64_t)32 * n;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
#pragma unroll
            for (int i = 0; i < C::PS; ++i) {
                y.s[pl][i] = *reinterpret_cast<const u32x4*>(ps + pl * (int64_t)DK * DV + at * DK + 8 * (tid + 256 * i));
                y.d[pl][i] = *reinterpret_cast<const u32x4*>(pd + pl * (int64_t)DK * DV + at * DK + 8 * (tid + 256 * i));
            }
            y.u[pl] = *reinterpret_cast<const u32x4*>(pu + pl * (int64_t)kGC * DV + at * kGC + 8 * tid);
            y.x[pl] = *reinterpret_cast<const u32x4*>(px + pl * (int64_t)kGC * DV + at * kGC + 8 * tid);
        }
        load_rows<1, 4>(y.o, po + at, os, rows, tid);
        const __amdgpu_buffer_rsrc_t rv = rsrc(pv + at, ((rows - 1) * (int)d.vs + 32) * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) y.v[i] = bload8(rv, (uint32_t)((16 * wave + r) * (int)d.vs + 16 * i + 4 * g) * 2);
    };
    auto put = [&]() {
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
#pragma unroll
            for (int i = 0; i < C::PS; ++i) {
                const int e = tid + 256 * i, off = (e / (DK / 8)) * C::RSS + (e % (DK / 8)) * 16;
                lds_st(smem + C::SH + pl * 32 * C::RSS + off, y.s[pl][i]);
                lds_st(smem + C::DH + pl * 32 * C::RSS + off, y.d[pl][i]);
            }
            const int off = (tid / 8) * C::RST + (tid % 8) * 16;
            lds_st(smem + C::UH + pl * 32 * C::RST + off, y.u[pl]);
            lds_st(smem + C::XH + pl * 32 * C::RST + off, y.x[pl]);
        }
        lds_st(smem + C::OO + (tid / 4) * C::RSO + (tid % 4) * 16, y.o[0]);
    };
    // operands over a slice's 32 value columns (element 4x + i of lane group g: column 16x + 4g
    // + i): a channel tile of S or dS', a token tile of U, dX or dO
    auto channels = [&](int plane, int b) {
        const unsigned char* at = smem + plane + (4 * g + trj) * C::RSS + 32 * b + 8 * trq;
        return cat8(lds_tr(at), lds_tr(at + 16 * C::RSS));
    };
    auto tokens = [&](int plane, int t) {
        const unsigned char* at = smem + plane + (4 * g + trj) * C::RST + 64 * (t >> 1) + 8 * (t & 1) + 16 * trq;
        return cat8(lds_tr(at), lds_tr(at + 16 * C::RST));
    };
    auto outs = [&](int t) {
        const unsigned char* at = smem + C::OO + (16 * t + r) * C::RSO + 8 * g;
        return cat8(lds_ld<bf16x4>(at), lds_ld<bf16x4>(at + 32));
    };
    auto lower = [](bf16x8 x) { return to_f4(bf16x4{x[0], x[1], x[2], x[3]}); };
    auto upper = [](bf16x8 x) { return to_f4(bf16x4{x[4], x[5], x[6], x[7]}); };
    // this wave's tiles of the triangle
    const int ntile = wave == 0 || wave == 3 ? 3 : 2;
    auto tile = [&](int n, int& it, int& jt) {
        if (wave == 0 || wave == 3) {
            it = (wave ? 2 : 0) + (n > 0);
            jt = (wave ? 2 : 0) + (n > 1);
        } else {
            it = wave + 1;
            jt = n;
        }
    };
    f32x4 OS[2][C::KW], XS[2][C::KW], UD[2][C::KW], OU[3], XU[3], tr[C::KW / 2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int b = 0; b < C::KW; ++b) OS[x][b] = XS[x][b] = UD[x][b] = zero4();
#pragma unroll
    for (int n = 0; n < 3; ++n) OU[n] = XU[n] = zero4();
#pragma unroll
    for (int b = 0; b < C::KW / 2; ++b) tr[b] = zero4();
    float xv = 0.f;
    load(0);
    const int slices = d.dv / 32;  // (as a constant, two of them are unrolled into spilled registers)
#pragma unroll 1
    for (int n = 0; n < slices; ++n) {
        lds_barrier();
        put();
        const u32x2 vcur[2] = {y.v[0], y.v[1]};
        lds_barrier();
        if (n + 1 < slices) load(n + 1);
        // (the scheduling barriers keep operands from being read further ahead than fits the
        // registers)
        bf16x8 xh[2], xl[2];
        {
            bf16x8 o[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                o[x] = outs(2 * wi + x);
                xh[x] = tokens(C::XH, 2 * wi + x);
                xl[x] = tokens(C::XL, 2 * wi + x);
            }
#pragma unroll
            for (int b = 0; b < C::KW; ++b) {
                const bf16x8 sh = channels(C::SH, C::KW * wj + b), sl = channels(C::SL, C::KW * wj + b);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    OS[x][b] = mfma32(sh, o[x], OS[x][b]);
                    XS[x][b] = mfma32(sh, xh[x], XS[x][b]);
                    OS[x][b] = mfma32(sl, o[x], OS[x][b]);
                    XS[x][b] = mfma32(sl, xh[x], XS[x][b]);
                    XS[x][b] = mfma32(sh, xl[x], XS[x][b]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // dV = beta dX and dX . V of token tile `wave`: lane (r, g) has token r, eight columns
        {
            const bf16x8 x1 = wj ? xh[1] : xh[0], x2 = wj ? xl[1] : xl[0];
            const f32x4 a0 = lower(x1) + lower(x2), a1 = upper(x1) + upper(x2);
            const int tok = 16 * wave + r;
            const f32x4 v0 = unpack_bf4(vcur[0]), v1 = unpack_bf4(vcur[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) xv += a0[i] * v0[i] + a1[i] * v1[i];
            if (tok < rows) {
                const float be = lds_ld<float>(smem + C::GV + GateVec::BE + 4 * tok);
                bf16* dst = (bf16*)A.dv + (t0 + tok) * os + (int64_t)h * DV + 32 * n + 4 * g;
                *reinterpret_cast<bf16x4*>(dst) = to_bf4(be * a0);
                *reinterpret_cast<bf16x4*>(dst + 16) = to_bf4(be * a1);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        {
            bf16x8 uh[2], ul[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uh[x] = tokens(C::UH, 2 * wi + x);
                ul[x] = tokens(C::UL, 2 * wi + x);
            }
#pragma unroll
            for (int b = 0; b < C::KW; ++b) {
                const bf16x8 dh = channels(C::DH, C::KW * wj + b), dl = channels(C::DL, C::KW * wj + b);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    UD[x][b] = mfma32(dh, uh[x], UD[x][b]);
                    UD[x][b] = mfma32(dl, uh[x], UD[x][b]);
                    UD[x][b] = mfma32(dh, ul[x], UD[x][b]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the diagonal of S dS'^T, every channel tile by one of the two waves that hold it
#pragma unroll
        for (int b = 0; b < C::KW / 2; ++b) {
            const int ch = C::KW * wj + C::KW / 2 * wi + b;
            const bf16x8 sh = channels(C::SH, ch), dh = channels(C::DH, ch);
            tr[b] = mfma32(sh, dh, tr[b]);
            tr[b] = mfma32(channels(C::SL, ch), dh, tr[b]);
            tr[b] = mfma32(sh, channels(C::DL, ch), tr[b]);
            __builtin_amdgcn_sched_barrier(0);
        }
        unroll<0, 3>([&](auto M) {
            constexpr int m = decltype(M)::value;
            if (m >= ntile) return;
            int it, jt;
            tile(m, it, jt);
            const bf16x8 u1 = tokens(C::UH, jt), u2 = tokens(C::UL, jt), oi = outs(it), x1 = tokens(C::XH, it), x2 = tokens(C::XL, it);
            OU[m] = mfma32(u1, oi, OU[m]);
            XU[m] = mfma32(u1, x1, XU[m]);
            OU[m] = mfma32(u2, oi, OU[m]);
            XU[m] = mfma32(u2, x1, XU[m]);
            XU[m] = mfma32(u1, x2, XU[m]);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    // ---------------------------------------------------------------- over the chunk's tokens
    u32x4 rk[KeyTile<DK>::PPT], rq[KeyTile<DK>::PPT];
    load_rows<KeyTile<DK>::PPT, DK / 8>(rk, (const bf16*)A.k + t0 * d.ks + (int64_t)hk * DK, d.ks, rows, tid);
    load_rows<KeyTile<DK>::PPT, DK / 8>(rq, (const bf16*)A.q + t0 * d.qs + (int64_t)hk * DK, d.qs, rows, tid);
    __syncthreads();
    store_key<DK, false>(smem + C::KT, rk, tid);
    store_key<DK, false>(smem + C::QT, rq, tid);
    xv += __shfl_xor(xv, 16);
    xv += __shfl_xor(xv, 32);
    if (g == 0) lds_st(smem + C::XV + 4 * (16 * wave + r), xv);
    float trace = 0.f;
#pragma unroll
    for (int b = 0; b < C::KW / 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) trace += 4 * g + i == r ? tr[b][i] : 0.f;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) trace += __shfl_xor(trace, off);
    if (lane == 0) lds_st(smem + C::TR + 4 * wave, trace);
    // tiles above the diagonal that the 32-deep products touch, and every partial sum, are zero
    // unless written below
    for (int i = tid; i < 3 * 256; i += 256) lds_st(smem + C::ROW + 4 * i, 0.f);
    if (tid < 128) {
        const int p = tid >> 5, l = tid & 31, row = 32 * (l >> 4) + (l & 15);  // four planes, rows of tiles 0 and 2
        unsigned char* at = smem + C::EH + p * kGC * C::RSE + row * C::RSE + 2 * (32 * (l >> 4) + 16);
        lds_st(at, u32x4{0u, 0u, 0u, 0u});
        lds_st(at + 16, u32x4{0u, 0u, 0u, 0u});
    }
    __syncthreads();
    unroll<0, 3>([&](auto N) {
        constexpr int n = decltype(N)::value;
        if (n >= ntile) return;
        int it, jt;
        tile(n, it, jt);
        TileRows<DK, false> ki, kj, qi;
        ki.load(smem + C::KT, it, r, g);
        kj.load(smem + C::KT, jt, r, g);
        qi.load(smem + C::QT, it, r, g);
        const f32x4 dec = decay_row(smem + C::GV, 16 * it + r, 16 * jt + 4 * g);
        const float be = lds_ld<float>(smem + C::GV + GateVec::BE + 4 * (16 * it + r));
        const f32x4 qk = tile_dot(kj, qi), kk = tile_dot(kj, ki);
        // lane (r, g): row 16 it + r, columns 16 jt + 4g ..
        f32x4 E, F, cs;
        float rs = 0.f, bs = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            E[i] = it > jt || 4 * g + i <= r ? d.scale * (dec[i] * OU[n][i]) : 0.f;
            const float f = it > jt || 4 * g + i < r ? -(dec[i] * XU[n][i]) : 0.f;
            F[i] = be * f;
            // (the diagonal carries no decay: out of both sums, where it would drown what does)
            cs[i] = it > jt || 4 * g + i < r ? E[i] * qk[i] + F[i] * kk[i] : 0.f;
            rs += cs[i];
            bs += f * kk[i];
        }
        bf16x4 hi, lo;
        unsigned char* at = smem + (16 * it + r) * C::RSE + 2 * (16 * jt + 4 * g);
        split4(E, hi, lo);
        lds_st(at + C::EH, hi);
        lds_st(at + C::EL, lo);
        split4(F, hi, lo);
        lds_st(at + C::FH, hi);
        lds_st(at + C::FL, lo);
        rs += __shfl_xor(rs, 16);
        rs += __shfl_xor(rs, 32);
        bs += __shfl_xor(bs, 16);
        bs += __shfl_xor(bs, 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int off = 1; off < 16; off *= 2) cs[i] += __shfl_xor(cs[i], off);
        }
        if (g == 0) {
            lds_st(smem + C::ROW + 4 * (64 * jt + 16 * it + r), rs);
            lds_st(smem + C::BET + 4 * (64 * jt + 16 * it + r), bs);
        }
        if (r == 0) lds_st(smem + C::COL + 4 * (64 * it + 16 * jt + 4 * g), cs);
    });
    __syncthreads();
    // dQ and dK: lane (r, g) has token r of the tile, channels 4g .. 4g+3
    const unsigned char* trk = smem + (4 * g + trj) * KeyTile<DK>::RS + 8 * trq;
    auto cols = [&](int tile_off, int s, int b) {  // a channel tile of K or Q over tokens of half s
        const unsigned char* at = trk + tile_off + 32 * s * KeyTile<DK>::RS + 32 * b;
        return cat8(lds_tr(at), lds_tr(at + 16 * KeyTile<DK>::RS));
    };
    auto row_of = [&](int plane, int t, int s) {  // row tile t of E or F, columns of half s
        const unsigned char* at = smem + plane + (16 * t + r) * C::RSE + 64 * s + 8 * g;
        return cat8(lds_ld<bf16x4>(at), lds_ld<bf16x4>(at + 32));
    };
    auto col_of = [&](int plane, int t, int s) {  // column tile t, rows of half s
        const unsigned char* at = smem + plane + (32 * s + 4 * g + trj) * C::RSE + 32 * t + 8 * trq;
        return cat8(lds_tr(at), lds_tr(at + 16 * C::RSE));
    };
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int t = 2 * wi + x, tok = 16 * t + r;
        const float eg = d.scale * lds_ld<float>(smem + C::EG + 4 * tok), bg = lds_ld<float>(smem + C::BG + 4 * tok),
                    er = lds_ld<float>(smem + C::ER + 4 * tok);
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        f32x4 dq[C::KW], dk[C::KW];
#pragma unroll
        for (int b = 0; b < C::KW; ++b) {
            const int ch = 16 * (C::KW * wj + b) + 4 * g;
            const f32x4 kv = to_f4(lds_ld<bf16x4>(smem + C::KT + tok * KeyTile<DK>::RS + 2 * ch));
            const f32x4 qv = to_f4(lds_ld<bf16x4>(smem + C::QT + tok * KeyTile<DK>::RS + 2 * ch));
            dq[b] = eg * OS[x][b];
            const f32x4 ke = bg * XS[x][b], kw = er * UD[x][b];
            dk[b] = kw - ke;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s1 += dq[b][i] * qv[i];
                s2 += XS[x][b][i] * kv[i];
                s3 += kw[i] * kv[i];
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s <= wi) {  // columns of half s: E K, F K
                const bf16x8 eh = row_of(C::EH, t, s), el = row_of(C::EL, t, s), fh = row_of(C::FH, t, s), fl = row_of(C::FL, t, s);
#pragma unroll
                for (int b = 0; b < C::KW; ++b) {
                    const bf16x8 kc = cols(C::KT, s, C::KW * wj + b);
                    dq[b] = mfma32(kc, eh, dq[b]);
                    dk[b] = mfma32(kc, fh, dk[b]);
                    dq[b] = mfma32(kc, el, dq[b]);
                    dk[b] = mfma32(kc, fl, dk[b]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (s >= wi) {  // rows of half s: E^T Q, F^T K
                const bf16x8 eh = col_of(C::EH, t, s), el = col_of(C::EL, t, s), fh = col_of(C::FH, t, s), fl = col_of(C::FL, t, s);
#pragma unroll
                for (int b = 0; b < C::KW; ++b) {
                    const bf16x8 kc = cols(C::KT, s, C::KW * wj + b), qc = cols(C::QT, s, C::KW * wj + b);
                    dk[b] = mfma32(qc, eh, dk[b]);
                    dk[b] = mfma32(kc, fh, dk[b]);
                    dk[b] = mfma32(qc, el, dk[b]);
                    dk[b] = mfma32(kc, fl, dk[b]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (tok < rows) {
#pragma unroll
            for (int b = 0; b < C::KW; ++b) {
                const int ch = 16 * (C::KW * wj + b) + 4 * g;
                if (A.parts) {
                    const int64_t o = ((t0 + tok) * d.hv + h) * (int64_t)DK + ch;
                    *reinterpret_cast<f32x4*>(A.dq_parts + o) = dq[b];
                    *reinterpret_cast<f32x4*>(A.dk_parts + o) = dk[b];
                } else {
                    const int64_t o = ((t0 + tok) * d.hk + hk) * (int64_t)DK + ch;
                    *reinterpret_cast<bf16x4*>((bf16*)A.dq + o) = to_bf4(dq[b]);
                    *reinterpret_cast<bf16x4*>((bf16*)A.dk + o) = to_bf4(dk[b]);
                }
            }
        }
        s1 += __shfl_xor(s1, 16);
        s2 += __shfl_xor(s2, 16);
        s3 += __shfl_xor(s3, 16);
        s1 += __shfl_xor(s1, 32);
        s2 += __shfl_xor(s2, 32);
        s3 += __shfl_xor(s3, 32);
        if (g == 0) {
            lds_st(smem + C::DOT + 768 * wj + 4 * tok, s1);
            lds_st(smem + C::DOT + 768 * wj + 256 + 4 * tok, s2);
            lds_st(smem + C::DOT + 768 * wj + 512 + 4 * tok, s3);
        }
    }
    __syncthreads();
    if (wave == 0) {  // lane = token: the gates' gradients
        auto at = [&](int off) { return lds_ld<float>(smem + off + 4 * lane); };
        const float s1 = at(C::DOT) + at(C::DOT + 768), s2 = at(C::DOT + 256) + at(C::DOT + 1024), s3 = at(C::DOT + 512) + at(C::DOT + 1280);
        const float rs = (at(C::ROW) + at(C::ROW + 256)) + (at(C::ROW + 512) + at(C::ROW + 768));
        const float cs = (at(C::COL) + at(C::COL + 256)) + (at(C::COL + 512) + at(C::COL + 768));
        const float bs = (at(C::BET) + at(C::BET + 256)) + (at(C::BET + 512) + at(C::BET + 768));
        const float eg = at(C::EG), gc = lds_ld<float>(smem + C::TR + 16);
        const float trace = (lds_ld<float>(smem + C::TR) + lds_ld<float>(smem + C::TR + 4)) +
                            (lds_ld<float>(smem + C::TR + 8) + lds_ld<float>(smem + C::TR + 12));
        // suffix sums over the chunk in fp64 (the terms of a token cancel against its neighbours')
        const double dG = ((double)s1 - (double)(at(C::BG) * s2)) - (double)s3 + ((double)rs - (double)cs);
        const double inc = wave_scan_f64(dG), w3 = wave_scan_f64((double)s3);
        const double total = __shfl(inc, 63), dgc = (double)(gc * trace) + __shfl(w3, 63);
        if (lane < rows) {
            A.dlog_alpha[(t0 + lane) * d.hv + h] = (float)(dgc + (total - inc + dG));
            A.dbeta[(t0 + lane) * d.hv + h] = (at(C::XV) - eg * s2) + bs;
        }
    }
}

template <int DK>
hipError_t walks(const GdnBackwardArgs& p, const GdnTable& tab, hipStream_t st) {
    typedef WalksCfg<DK> C;
    GdnPrefillArgs f = {};
    f.d = p.d; f.num_seqs = p.num_seqs; f.q = p.q; f.k = p.k; f.v = p.v; f.log_alpha = p.log_alpha; f.beta = p.beta;
    f.initial_state = p.initial_state; f.nv = 16 * NCB;
    PArgs fa = walk_args(f);
    fa.save_s = (bf16*)p.states; fa.save_u = (bf16*)p.u;
    WArgs a;
    a.q = (const bf16*)p.q; a.k = (const bf16*)p.k; a.d_out = (const bf16*)p.d_out; a.la = p.log_alpha; a.be = p.beta;
    a.dSf = p.d_final_state; a.dS0 = p.d_initial_state; a.sgrads = (bf16*)p.sgrads; a.dx = (bf16*)p.dx;
    a.qs = p.d.qs; a.ks = p.d.ks; a.hk = p.d.hk; a.hv = p.d.hv; a.dv = p.d.dv; a.slices = fa.slices; a.groups = fa.groups;
    a.scale = p.d.scale;
    hipError_t e = hipFuncSetAttribute((const void*)gdn_walks_kernel<DK>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       C::LDS_BYTES);
    if (e != hipSuccess) return e;
    const int64_t blocks = walk_blocks(f), stretch = std::min<int64_t>(blocks, p.cus), grid = (blocks + stretch - 1) / stretch * 2 * stretch;
    hipLaunchKernelGGL((gdn_walks_kernel<DK>), dim3((unsigned)grid), dim3(C::THREADS), C::LDS_BYTES, st, fa, a, tab, (int)stretch);
    return hipGetLastError();
}

template <int DK, int DV>
hipError_t gradients(const GdnBackwardArgs& p, const GdnTable& tab, hipStream_t st) {
    constexpr int lds = GradCfg<DK>::LDS_BYTES;
    hipError_t e = hipFuncSetAttribute((const void*)gdn_gradients_kernel<DK, DV>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    for (int from = 0; from < p.num_seqs;) {
        const int n = gdn_gradient_group(tab, from, p.num_seqs, p.d.hv);
        if (n == 0) break;
        const int chunks = (tab.len[from] + kGC - 1) / kGC;  // of the group's longest
        hipLaunchKernelGGL((gdn_gradients_kernel<DK, DV>), dim3((unsigned)(chunks * p.d.hv), (unsigned)n), dim3(256), lds, st, p, tab,
                           from);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        from += n;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gdn_backward_chunked(const GdnBackwardArgs& p, const GdnTable& tab, hipStream_t st) {
    const hipError_t e = p.d.dk == 128 ? walks<128>(p, tab, st) : walks<64>(p, tab, st);
    if (e != hipSuccess) return e;
    if (p.d.dk == 128) return p.d.dv == 128 ? gradients<128, 128>(p, tab, st) : gradients<128, 64>(p, tab, st);
    return p.d.dv == 128 ? gradients<64, 128>(p, tab, st) : gradients<64, 64>(p, tab, st);
}

}  // namespace kda
