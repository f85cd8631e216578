// gdn_prefill.hip -- chunked gated delta rule, bf16 inputs, fp32 state (gfx950).
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
// wave.  Four producer waves build the key side of chunk c+1 (gdn_chunk.h) while the chain
// waves step chunk c; K, Q, V and the matrices are double-buffered in LDS, and the loads of
// chunk c+2 are in flight meanwhile.  Two of the producers form and invert A's diagonal halves,
// each its own without a barrier between; the others form P and the block of A below.
//
// Precision.  Operands are fp16.  The products that make the state (K S, the solve, K^T U)
// take their fp32 side as a pair hi + lo (22 bits): single operands would leave the fp32 state
// only 3e-4 of its size accurate, bf16 pairs 4e-6; these measure 2e-7.  The readout's operands
// (S, P, U) are single (11 bits), an eighth of the rounding of the bf16 output.  bf16 q, k and
// v are exact in fp16 inside its range.  The rule is linear in (v, S): both run multiplied by
// eight, which keeps the low halves above fp16's subnormals for values down to about 1e-2 and
// the high ones finite up to 8000.
#include "gdn_chunk.h"
#include "gdn_launch.h"

namespace kda {
namespace {

constexpr float kPre = 8.f;  // v and the state are carried times this

template <int DK, int NCB>
struct GCfg {
    static constexpr int KB = DK / 16, KP = DK / 32, NV = 16 * NCB;
    // two column blocks per chain wave at full width, so that an operand read from LDS serves
    // 32 columns; one otherwise (the shortest step)
    static constexpr int CPW = NCB >= 8 ? 2 : 1;
    static constexpr int NCHAIN = NCB / CPW;
    static constexpr int THREADS = 64 * (NCHAIN + 4);
    typedef KeyTile<DK> K;
    typedef ValueTile<NV> V;
    // matrices, as operand fragments (16 bytes per lane): row tiles 0 and 1 of T's upper half,
    // of its lower half, of -A's block below them, hi then lo; P's three blocks
    static constexpr int FR = 1024;
    static constexpr int M_T0 = 0, M_T1 = 4 * FR, M_A = 8 * FR, M_P = 12 * FR, M_SIZE = 18 * FR;
    // vectors over the chunk's tokens: e^G, beta e^G, kPre beta, e^{G_C - G}; e^{G_C}
    static constexpr int V_EG = 0, V_BE = 256, V_B = 512, V_ER = 768, V_GC = 1024, V_SIZE = 1040;
    static constexpr int O_K = 0, O_Q = O_K + 2 * K::SIZE, O_V = O_Q + 2 * K::SIZE, O_M = O_V + 2 * V::SIZE,
                         O_VEC = O_M + 2 * M_SIZE, O_G = O_VEC + 2 * V_SIZE,
                         O_INV = O_G + GateVec::SIZE, LDS_BYTES = O_INV + 2 * InvScratch::SIZE;
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
    GdnTable tab;
};

__device__ __forceinline__ void split8(f32x4 a, f32x4 b, f16x8& hi, f16x8& lo) {
    hi = to_h8(a, b);
    f32x4 ra, rb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ra[i] = a[i] - (float)hi[i];
        rb[i] = b[i] - (float)hi[4 + i];
    }
    lo = to_h8(ra, rb);
}
__device__ __forceinline__ void split4h(f32x4 a, f16x4& hi, f16x4& lo) {
    hi = to_h4(a);
    f32x4 ra;
#pragma unroll
    for (int i = 0; i < 4; ++i) ra[i] = a[i] - (float)hi[i];
    lo = to_h4(ra);
}

template <int DK, int NCB>
__global__ __launch_bounds__((GCfg<DK, NCB>::THREADS)) void gdn_prefill_kernel(const PArgs a) {
    typedef GCfg<DK, NCB> C;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    // the slices of one state on one XCD (workgroups go round-robin over eight): they share
    // its keys and queries in that XCD's L2
    const int kk = blockIdx.x >> 3;
    const int group = (kk / a.slices) * 8 + (blockIdx.x & 7), slice = kk % a.slices;
    if (group >= a.groups) return;
    const int si = group / a.hv, h = group % a.hv, hk = h / (a.hv / a.hk);
    const int len = a.tab.len[si], col0 = slice * C::NV;
    const int64_t start = a.tab.start[si];
    const int64_t sbase = ((int64_t)a.tab.id[si] * a.hv + h) * (int64_t)DK * a.dv;
    const int nch = (len + kGC - 1) / kGC;

    auto buf = [&](int off, int size, int c) { return smem + off + (c & 1) * size; };
    // zero the fragments' halves that lie above the diagonal; nothing else writes them
    for (int i = tid; i < 2 * C::M_SIZE / 16; i += C::THREADS)
        lds_st(smem + C::O_M + 16 * i, u32x4{0u, 0u, 0u, 0u});
    lds_barrier();

    if (wave >= C::NCHAIN) {
        // ================================================================ producers
        const int pw = wave - C::NCHAIN, pt = tid - 64 * C::NCHAIN;
        u32x4 rk[C::K::PPT], rq[C::K::PPT], rv[C::V::PPT];
        float rla = 0.f, rbe = 0.f;
        const bf16* pq = a.q + start * a.qs + (int64_t)hk * DK;
        const bf16* pk = a.k + start * a.ks + (int64_t)hk * DK;
        const bf16* pv = a.v + start * a.vs + (int64_t)h * a.dv + col0;
        auto load = [&](int c) {
            const int rows = min(kGC, len - kGC * c);
            const int64_t at = (int64_t)kGC * c;
            load_rows<C::K::PPT, DK / 8>(rk, pk + at * a.ks, a.ks, rows, pt);
            load_rows<C::K::PPT, DK / 8>(rq, pq + at * a.qs, a.qs, rows, pt);
            load_rows<C::V::PPT, C::NV / 8>(rv, pv + at * a.vs, a.vs, rows, pt);
            if (pw == 0) {
                rla = rbe = 0.f;
                if (lane < rows) {
                    rla = a.la[(start + at + lane) * a.hv + h];
                    rbe = a.be[(start + at + lane) * a.hv + h];
                }
            }
        };
        if (nch > 0) load(0);
        unsigned char* gv = smem + C::O_G;
        for (int c = 0; c <= nch; ++c) {  // builds chunk c; the last pass only keeps the barriers
            if (c < nch) {
                unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
                unsigned char* Qt = buf(C::O_Q, C::K::SIZE, c);
                unsigned char* Vt = buf(C::O_V, C::V::SIZE, c);
                store_key<DK, true>(Kt, rk, pt);
                store_key<DK, true>(Qt, rq, pt);
#pragma unroll
                for (int i = 0; i < C::V::PPT; ++i) {
                    const int e = pt + 256 * i;
                    if (e < C::V::PIECES) lds_st(Vt + (e / (C::NV / 8)) * C::V::RS + (e % (C::NV / 8)) * 16, rv[i]);
                }
                if (pw == 0) {
                    const double G = wave_scan_f64(log2_decay(rla));
                    const double GC = __shfl(G, 63);
                    const float hi = (float)G, eg = __builtin_amdgcn_exp2f(hi);
                    lds_st(gv + GateVec::HI + 4 * lane, hi);
                    lds_st(gv + GateVec::LO + 4 * lane, (float)(G - (double)hi));
                    lds_st(gv + GateVec::BE + 4 * lane, rbe);
                    float* vec = reinterpret_cast<float*>(buf(C::O_VEC, C::V_SIZE, c));
                    vec[C::V_EG / 4 + lane] = eg;
                    vec[C::V_BE / 4 + lane] = rbe * eg;
                    vec[C::V_B / 4 + lane] = kPre * rbe;
                    vec[C::V_ER / 4 + lane] = __builtin_amdgcn_exp2f((float)(GC - G));
                    if (lane == 0) vec[C::V_GC / 4] = __builtin_amdgcn_exp2f((float)GC);
                }
                if (c + 1 < nch) load(c + 1);
            }
            lds_barrier();
            if (c < nch) {
                const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
                const unsigned char* Qt = buf(C::O_Q, C::K::SIZE, c);
                unsigned char* M = buf(C::O_M, C::M_SIZE, c);
                if (pw < 2) {
                    f32x4 rows[3];
                    half_inverse<DK>(Kt, gv, smem + C::O_INV + pw * InvScratch::SIZE, pw, lane, rows);
                    unsigned char* d = M + (pw ? C::M_T1 : C::M_T0) + 16 * lane;
                    const int at[3] = {0, C::FR, C::FR + 8};
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        f16x4 hi, lo;
                        split4h(rows[i], hi, lo);
                        lds_st(d + at[i], hi);
                        lds_st(d + at[i] + 2 * C::FR, lo);
                    }
                } else {
                    TileRows<DK> kt[4], qt;
                    // P's tiles of row tile it, and -A's where they lie below the halves: lane
                    // (r, g) holds row 16 it + r, columns 16 jt + 4g ..
                    auto row_tiles = [&](auto IT) {
                        constexpr int it = decltype(IT)::value;
                        qt.load(Qt, it, r, g);
                        unroll<0, it + 1>([&](auto JT) {
                            constexpr int jt = decltype(JT)::value;
                            const f32x4 d = decay_row(gv, 16 * it + r, 16 * jt + 4 * g);
                            f32x4 p = tile_dot<DK>(kt[jt], qt);
#pragma unroll
                            for (int i = 0; i < 4; ++i) p[i] = it > jt || 4 * g + i <= r ? d[i] * p[i] : 0.f;
                            // P: block (rows 32 (it / 2), columns 32 (jt / 2)), row tile it % 2
                            lds_st(M + C::M_P + (2 * (it / 2 + jt / 2) + it % 2) * C::FR + 16 * lane + 8 * (jt % 2), to_h4(p));
                            if constexpr (it / 2 != jt / 2) {
                                const f32x4 x = tile_dot<DK>(kt[jt], kt[it]);
                                const float nb = -lds_ld<float>(gv + GateVec::BE + 4 * (16 * it + r));
                                f16x4 hi, lo;
                                split4h(nb * (d * x), hi, lo);
                                unsigned char* m = M + C::M_A + (it % 2) * C::FR + 16 * lane + 8 * (jt % 2);
                                lds_st(m, hi);
                                lds_st(m + 2 * C::FR, lo);
                            }
                        });
                    };
                    kt[0].load(Kt, 0, r, g);
                    kt[1].load(Kt, 1, r, g);
                    kt[2].load(Kt, 2, r, g);
                    if (pw == 2) {
                        row_tiles(std::integral_constant<int, 2>{});
                        row_tiles(std::integral_constant<int, 1>{});
                        row_tiles(std::integral_constant<int, 0>{});
                    } else {
                        kt[3].load(Kt, 3, r, g);
                        row_tiles(std::integral_constant<int, 3>{});
                    }
                }
            }
            lds_barrier();
        }
        return;
    }

    // ==================================================================== chain waves
    constexpr int KB = C::KB, KP = C::KP, CPW = C::CPW;
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
    const float oscale = a.scale / kPre;
    bf16* po = a.out + start * a.hv * a.dv + (int64_t)h * a.dv + col0 + 16 * CPW * wave + 4 * g;
    const int64_t os = (int64_t)a.hv * a.dv;

    lds_barrier();  // chunk 0 is built in the producers' first pass
    lds_barrier();
    for (int c = 0; c < nch; ++c) {
        const unsigned char* Kt = buf(C::O_K, C::K::SIZE, c);
        const unsigned char* Qt = buf(C::O_Q, C::K::SIZE, c);
        const unsigned char* Vt = buf(C::O_V, C::V::SIZE, c);
        const unsigned char* M = buf(C::O_M, C::M_SIZE, c);
        const float* vec = reinterpret_cast<const float*>(buf(C::O_VEC, C::V_SIZE, c));
        auto frag = [&](int off) { return lds_ld<f16x8>(M + off + 16 * lane); };
        // Y = K S (rows of tokens) and (Q S)^T (rows of value columns)
        f32x4 Y[CPW][4], O[CPW][4];
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb)
#pragma unroll
            for (int t = 0; t < 4; ++t) Y[cb][t] = O[cb][t] = zero4();
#pragma unroll
        for (int p = 0; p < KP; ++p) {
            f16x8 sh[CPW], sl[CPW];
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) split8(S[cb][2 * p], S[cb][2 * p + 1], sh[cb], sl[cb]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f16x8 kf = lds_ld<f16x8>(Kt + (16 * t + r) * C::K::RS + 64 * p + 16 * g);
                const f16x8 qf = lds_ld<f16x8>(Qt + (16 * t + r) * C::K::RS + 64 * p + 16 * g);
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) {
                    Y[cb][t] = mfma32h(kf, sh[cb], Y[cb][t]);
                    Y[cb][t] = mfma32h(kf, sl[cb], Y[cb][t]);
                    O[cb][t] = mfma32h(sh[cb], qf, O[cb][t]);
                }
            }
        }
        // X = kPre beta V - beta e^G Y, in place of Y
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f32x4 vb = *reinterpret_cast<const f32x4*>(vec + C::V_B / 4 + 16 * t + 4 * g);
            const f32x4 ve = *reinterpret_cast<const f32x4*>(vec + C::V_BE / 4 + 16 * t + 4 * g);
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) {
                const f32x4 vv = to_f4(lds_tr(Vt + tr_v + 16 * t * C::V::RS + 32 * (CPW * wave + cb)));
                Y[cb][t] = vb * vv - ve * Y[cb][t];
            }
        }
        // U: the upper half's solve, its substitution into the lower half's rows, that solve
        f32x4 U[CPW][4];
        f16x8 uh[CPW][2];
#pragma unroll
        for (int cb = 0; cb < CPW; ++cb) {
            f16x8 xh, xl, ul;
            split8(Y[cb][0], Y[cb][1], xh, xl);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f16x8 th = frag(C::M_T0 + t * C::FR), tl = frag(C::M_T0 + (2 + t) * C::FR);
                f32x4 u = mfma32h(tl, xh, zero4());
                u = mfma32h(th, xl, u);
                U[cb][t] = mfma32h(th, xh, u);
            }
            split8(U[cb][0], U[cb][1], uh[cb][0], ul);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f16x8 ah = frag(C::M_A + t * C::FR), al = frag(C::M_A + (2 + t) * C::FR);
                Y[cb][2 + t] = mfma32h(ah, uh[cb][0], Y[cb][2 + t]);
                Y[cb][2 + t] = mfma32h(ah, ul, Y[cb][2 + t]);
                Y[cb][2 + t] = mfma32h(al, uh[cb][0], Y[cb][2 + t]);
            }
            split8(Y[cb][2], Y[cb][3], xh, xl);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f16x8 th = frag(C::M_T1 + t * C::FR), tl = frag(C::M_T1 + (2 + t) * C::FR);
                f32x4 u = mfma32h(tl, xh, zero4());
                u = mfma32h(th, xl, u);
                U[cb][2 + t] = mfma32h(th, xh, u);
            }
            uh[cb][1] = to_h8(U[cb][2], U[cb][3]);
        }
        lds_barrier();
        // O^T = e^G (Q S)^T + (P U)^T: lane (r, g) holds token r, columns 4g .. 4g+3
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float eg = vec[C::V_EG / 4 + 16 * t + r];
            const int row = kGC * c + 16 * t + r;
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) {
                f32x4 o = eg * O[cb][t];
                o = mfma32h(uh[cb][0], frag(C::M_P + t * C::FR), o);
                if (t >= 2) o = mfma32h(uh[cb][1], frag(C::M_P + (2 + t) * C::FR), o);
                if (row < len)
                    *reinterpret_cast<bf16x4*>(po + (int64_t)row * os + 16 * cb) = to_bf4(oscale * o);
            }
        }
        // S <- e^{G_C} S + K^T (e^{G_C - G} U)
        const float gc = vec[C::V_GC / 4];
        f16x8 wh[CPW][2], wl[CPW][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const f32x4 e0 = *reinterpret_cast<const f32x4*>(vec + C::V_ER / 4 + 32 * s + 4 * g);
            const f32x4 e1 = *reinterpret_cast<const f32x4*>(vec + C::V_ER / 4 + 32 * s + 16 + 4 * g);
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) split8(e0 * U[cb][2 * s], e1 * U[cb][2 * s + 1], wh[cb][s], wl[cb][s]);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int cb = 0; cb < CPW; ++cb) S[cb][b] *= gc;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const unsigned char* at = Kt + tr_k + 32 * s * C::K::RS + 64 * (b >> 1) + 8 * (b & 1);
                const f16x8 kt = cat8h(lds_trh(at), lds_trh(at + 16 * C::K::RS));
#pragma unroll
                for (int cb = 0; cb < CPW; ++cb) {
                    S[cb][b] = mfma32h(kt, wl[cb][s], S[cb][b]);
                    S[cb][b] = mfma32h(kt, wh[cb][s], S[cb][b]);
                }
            }
        }
        lds_barrier();
    }
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

template <int DK, int NCB>
hipError_t launch(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    typedef GCfg<DK, NCB> C;
    PArgs a;
    a.q = (const bf16*)p.q; a.k = (const bf16*)p.k; a.v = (const bf16*)p.v;
    a.la = p.log_alpha; a.be = p.beta; a.S0 = p.initial_state; a.Sf = p.final_state; a.out = (bf16*)p.out;
    a.qs = p.d.qs; a.ks = p.d.ks; a.vs = p.d.vs; a.hk = p.d.hk; a.hv = p.d.hv; a.dv = p.d.dv;
    a.slices = p.d.dv / C::NV; a.groups = p.num_seqs * p.d.hv; a.scale = p.d.scale; a.tab = tab;
    const int64_t blocks = ((int64_t)a.groups + 7) / 8 * 8 * a.slices;
    hipError_t e = hipFuncSetAttribute((const void*)gdn_prefill_kernel<DK, NCB>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS_BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdn_prefill_kernel<DK, NCB>), dim3((unsigned)blocks), dim3(C::THREADS), C::LDS_BYTES, st, a);
    return hipGetLastError();
}

template <int DK>
hipError_t launch_nv(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    switch (p.nv) {
        case 16: return launch<DK, 1>(p, tab, st);
        case 32: return launch<DK, 2>(p, tab, st);
        case 64: return launch<DK, 4>(p, tab, st);
        case 128: return launch<DK, 8>(p, tab, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gdn_chunked(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    return p.d.dk == 128 ? launch_nv<128>(p, tab, st) : launch_nv<64>(p, tab, st);
}

}  // namespace kda
