// gdn_recurrent.hip -- the gated delta rule token by token, state in registers (gfx950).
//
// Per (sequence, value head), one log-decay g_t per token:
//   S <- e^{g_t} S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;  o_t = scale S^T q_t
// With w = S^T k and b = S^T (scale q) of the state BEFORE the decay, a = e^{g}:
//   u = beta (v - a w),   o = a b + (k . scale q) u,   S <- a S + k u^T
// so one pass over the state serves the erase, the write and the readout, and both column
// sums share one reduction.
//
// Two uses.  The step (1..16 tokens per sequence, the serving form): the state is the large
// operand, read once and written once whatever the number of tokens; HBM-bound.  The
// sequential prefill (any length, the form of 32-bit inputs): the state stays in registers
// for the whole sequence and the tokens stream through LDS.
//
// The step: a workgroup of four waves owns NV value columns of one state.  Thread t holds columns
// 4 (t % COLG) .. +3 of rows rg + ROWG i (rg = t / COLG): a row of the slice is read and written
// by COLG consecutive threads as one contiguous segment, and the workgroup's accesses of one i
// are one contiguous stretch of the state.  k and q lie in LDS in the order of the threads'
// rows, so a thread reads its own as 16-byte pieces.  TB tokens are staged at a time: four for
// the short steps, whose LDS then lets more workgroups share a compute unit and keep its loads
// in flight.  Everything is fp32; outputs are rounded once to their type.
#include "gdn_launch.h"
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

struct RecArgs {
    const void *q, *k, *v;
    const float *la, *be;
    int64_t qs, ks, vs;
    int hk, hv;
    float scale;
    void* out;
    // step form
    int num_tokens, num_slots;
    const int32_t *steps, *slots;
    float* state;
    bool update;
    // sequential prefill
    const float* S0;
    float* Sf;
};

__device__ inline f32x4 load4f(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ inline f32x4 load4f(const bf16* p) {
    return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(p), f32x4);
}

// a x + c, fused as written: the kernels below form the same bits from the same state and token
__device__ inline f32x4 fma4(float a, f32x4 x, f32x4 c) {
    return f32x4{fmaf(a, x[0], c[0]), fmaf(a, x[1], c[1]), fmaf(a, x[2], c[2]), fmaf(a, x[3], c[3])};
}

template <int DK, int NV, int TB>
struct Tile {
    static constexpr int COLG = NV / 4, ROWG = kThreads / COLG, RPT = DK / ROWG;
    static constexpr int QV = (TB * DK / 4 + kThreads - 1) / kThreads;  // 16-byte pieces of q (and k) per thread
    static constexpr int VV = (TB * NV / 4 + kThreads - 1) / kThreads;
    static_assert(DK % ROWG == 0 && RPT % 2 == 0, "shape");
    // place of a row's k and q in LDS
    static __device__ constexpr int place(int row) { return row % ROWG * RPT + row / ROWG; }
};

// The tokens' rows on their way from memory to LDS.
template <typename T, int DK, int DV, int NV, int TB>
struct Stage {
    using L = Tile<DK, NV, TB>;
    f32x4 q[L::QV], k[L::QV], v[L::VV];
    float g, b;
    __device__ void load(const RecArgs& A, int64_t row0, int n, int hk, int hv, int col0) {
        const int t = threadIdx.x;
#pragma unroll
        for (int i = 0; i < L::QV; ++i) {
            const int e = t + kThreads * i, r = e / (DK / 4), c = 4 * (e % (DK / 4));
            q[i] = k[i] = zero4();
            if (r < n) {
                q[i] = load4f((const T*)A.q + (row0 + r) * A.qs + (int64_t)hk * DK + c);
                k[i] = load4f((const T*)A.k + (row0 + r) * A.ks + (int64_t)hk * DK + c);
            }
        }
#pragma unroll
        for (int i = 0; i < L::VV; ++i) {
            const int e = t + kThreads * i, r = e / (NV / 4), c = 4 * (e % (NV / 4));
            v[i] = zero4();
            if (r < n) v[i] = load4f((const T*)A.v + (row0 + r) * A.vs + (int64_t)hv * DV + col0 + c);
        }
        g = b = 0.f;
        if (t < n) {
            g = A.la[(row0 + t) * A.hv + hv];
            b = A.be[(row0 + t) * A.hv + hv];
        }
    }
};

// one sequence's n <= TB tokens from row0 on; the first `advance` move the stored state (to
// Sout), outputs are written where `out` is given
template <typename T, int DK, int DV, int NV, int TB>
__device__ void walk(const RecArgs& A, const float* Sin, float* Sout, int64_t row0, int n,
                     int advance, T* out, int head, int col0, bool skip_check, int slot_seq) {
    using L = Tile<DK, NV, TB>;
    __shared__ __attribute__((aligned(16))) float s_k[TB][DK], s_q[TB][DK], s_v[TB][NV];
    __shared__ float s_a[TB], s_b[TB], s_kq[TB];
    __shared__ f32x4 s_red[2][4][L::COLG][2];
    const int t = threadIdx.x, cg = t % L::COLG, rg = t / L::COLG, wave = t / 64, lane = t % 64;
    const int hk = head / (A.hv / A.hk);

    // the state's loads first: the long-latency part of a step
    f32x4 s[L::RPT];
    const int64_t at = (int64_t)rg * DV + col0 + 4 * cg;
    constexpr int STEP = L::ROWG * DV;
#pragma unroll
    for (int i = 0; i < L::RPT; ++i)
        s[i] = Sin ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(Sin + at + i * STEP)) : zero4();
    Stage<T, DK, DV, NV, TB> st;
    st.load(A, row0, n, hk, head, col0);
    bool twice = false;  // an earlier row of this call names the same slot
    if (skip_check) {
        for (int j = t; j < slot_seq; j += kThreads) twice |= A.slots[j] == A.slots[slot_seq];
        if (__syncthreads_or(twice)) {
            if (out)
                for (int j = t; j < n * (NV / 4); j += kThreads)
                    store4(out + (row0 + j / (NV / 4)) * (int64_t)A.hv * DV + (int64_t)head * DV +
                               col0 + 4 * (j % (NV / 4)), Mma<T>::pack(zero4()));
            return;
        }
    }
    auto put = [&]() {
        if (!Sout) return;
        // non-temporal: the state is not read again by this call
#pragma unroll
        for (int i = 0; i < L::RPT; ++i)
            __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(Sout + at + i * STEP));
    };
#pragma unroll
    for (int i = 0; i < L::QV; ++i) {
        const int e = t + kThreads * i, r = e / (DK / 4), c = 4 * (e % (DK / 4));
        if (r < TB) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s_k[r][L::place(c + x)] = st.k[i][x];
                s_q[r][L::place(c + x)] = st.q[i][x] * A.scale;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < L::VV; ++i) {
        const int e = t + kThreads * i, r = e / (NV / 4), c = 4 * (e % (NV / 4));
        if (r < TB) *reinterpret_cast<f32x4*>(&s_v[r][c]) = st.v[i];
    }
    if (t < TB) {
        s_a[t] = expf(st.g);
        s_b[t] = st.b;
    }
    __syncthreads();
    if (out) {  // k . (scale q) of every token: 16 lanes each
        float kq = 0.f;
        const int tok = t / 16 % TB;
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) kq = fmaf(s_k[tok][L::place(t % 16 + 16 * c)], s_q[tok][L::place(t % 16 + 16 * c)], kq);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) kq += __shfl_xor(kq, off);
        if (t % 16 == 0 && t / 16 < TB) s_kq[tok] = kq;  // read behind the next barrier
    }
    for (int j = 0; j < n; ++j) {
        f32x4 w = zero4(), b = zero4();
#pragma unroll
        for (int i = 0; i < L::RPT; ++i) {
            w = fma4(s_k[j][rg * L::RPT + i], s[i], w);
            b = fma4(s_q[j][rg * L::RPT + i], s[i], b);
        }
#pragma unroll
        for (int off = L::COLG; off < 64; off <<= 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] += __shfl_xor(w[c], off);
                b[c] += __shfl_xor(b[c], off);
            }
        }
        if (lane < L::COLG) {
            s_red[j & 1][wave][lane][0] = w;
            s_red[j & 1][wave][lane][1] = b;
        }
        __syncthreads();
        w = (s_red[j & 1][0][cg][0] + s_red[j & 1][1][cg][0]) +
            (s_red[j & 1][2][cg][0] + s_red[j & 1][3][cg][0]);
        b = (s_red[j & 1][0][cg][1] + s_red[j & 1][1][cg][1]) +
            (s_red[j & 1][2][cg][1] + s_red[j & 1][3][cg][1]);
        const float a = s_a[j];
        const f32x4 u = s_b[j] * fma4(-a, w, *reinterpret_cast<const f32x4*>(&s_v[j][4 * cg]));
#pragma unroll
        for (int i = 0; i < L::RPT; ++i) s[i] = fma4(s_k[j][rg * L::RPT + i], u, a * s[i]);
        if (out && rg == 0)
            store4(out + (row0 + j) * (int64_t)A.hv * DV + (int64_t)head * DV + col0 + 4 * cg,
                   Mma<T>::pack(fma4(s_kq[j], u, a * b)));
        if (j + 1 == advance) {
            put();
            if (!out) return;  // (the whole workgroup: advance is the same for all)
        }
    }
}

template <typename T, int DK, int DV, int NV, int TB>
__global__ __launch_bounds__(kThreads, TB <= 4 ? 4 : 3) void step_kernel(const RecArgs A) {
    constexpr int SL = DV / NV;
    const int64_t pair = blockIdx.x / SL;
    const int n = (int)(pair / A.hv), head = (int)(pair % A.hv), col0 = NV * (int)(blockIdx.x % SL);
    const int64_t row0 = (int64_t)n * A.num_tokens;
    T* out = (T*)A.out;
    const int slot = A.slots ? A.slots[n] : n;
    if (slot < 0 || slot >= A.num_slots) {  // a padded row: no state, zero outputs
        if (out)
            for (int j = threadIdx.x; j < A.num_tokens * (NV / 4); j += kThreads)
                store4(out + (row0 + j / (NV / 4)) * (int64_t)A.hv * DV + (int64_t)head * DV + col0 +
                           4 * (j % (NV / 4)), Mma<T>::pack(zero4()));
        return;
    }
    int adv = A.update ? A.num_tokens : 0;
    if (A.update && A.steps) adv = min(max(A.steps[n], 0), A.num_tokens);
    if (adv == 0 && !out) return;
    float* S = A.state + ((int64_t)slot * A.hv + head) * (int64_t)(DK * DV);
    walk<T, DK, DV, NV, TB>(A, S, S, row0, A.num_tokens, adv, out, head, col0, A.update && A.slots, n);
}

// One token per sequence, the decode step: the same arithmetic in the same order as walk's, with
// nothing in registers but the state and what a row needs.  The token's loads are issued before
// the state's and the barriers order LDS alone, so k, q and the repeated-slot check are done
// while the state is on its way.  Whole rows: the state is streamed past the caches both ways,
// and no more than 128 KiB of states are in work on a compute unit (unused LDS keeps further
// workgroups out): with more reading and writing at once memory pages change more often.
// 256 x 32 states of 128 x 128 in a pool, slots in random order: 220 us, 195 with streamed
// loads, 193 with three workgroups per unit, 181 with two (5.9 TB/s; a large copy reaches 4.8
// on the same card).
template <int DK, int DV>
constexpr int whole_lds() { return DK * DV * 4 / 8 * 7; }

template <typename T, int DK, int DV, int NV>
__global__ __launch_bounds__(kThreads, DK * NV == 128 * 128 ? 2 : 4) void decode_kernel(const RecArgs A) {
    using L = Tile<DK, NV, 1>;
    constexpr int SL = DV / NV, STEP = L::ROWG * DV;
    __shared__ __attribute__((aligned(16))) float s_k[DK], s_q[DK];
    __shared__ f32x4 s_red[4][L::COLG][2];
    __shared__ int s_twice[4];
    const int t = threadIdx.x, cg = t % L::COLG, rg = t / L::COLG, wave = t / 64, lane = t % 64;
    const int pair = blockIdx.x / SL, n = pair / A.hv, head = pair % A.hv, col0 = NV * (int)(blockIdx.x % SL);
    const int hk = head / (A.hv / A.hk);
    T* out = A.out ? (T*)A.out + (int64_t)pair * DV + col0 : nullptr;
    const int slot = A.slots ? A.slots[n] : n;
    int adv = A.update;
    if (A.update && A.steps) adv = A.steps[n] > 0;
    const bool padded = slot < 0 || slot >= A.num_slots;
    if (padded || (!adv && !out)) {
        if (padded && out && t < L::COLG) store4(out + 4 * t, Mma<T>::pack(zero4()));
        return;
    }
    const bool check = A.update && A.slots;
    const int other = check && t < n ? A.slots[t] : -1;  // (the slot itself is not negative)
    float kv = 0.f, qv = 0.f;
    if (t < DK) {
        kv = to_f32(((const T*)A.k)[n * A.ks + (int64_t)hk * DK + t]);
        qv = A.scale * to_f32(((const T*)A.q)[n * A.qs + (int64_t)hk * DK + t]);
    }
    const f32x4 v = load4f((const T*)A.v + n * A.vs + (int64_t)head * DV + col0 + 4 * cg);
    const float la = A.la[pair], be = A.be[pair];
    float* S = A.state + ((int64_t)slot * A.hv + head) * (int64_t)(DK * DV) + rg * DV + col0 + 4 * cg;
    __builtin_amdgcn_sched_barrier(0);
    f32x4 s[L::RPT];
#pragma unroll
    for (int i = 0; i < L::RPT; ++i) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + i * STEP));
    __builtin_amdgcn_sched_barrier(0);
    if (t < DK) {
        s_k[t] = kv;
        s_q[t] = qv;
    }
    bool twice = other == slot;
    if (check)
        for (int j = t + kThreads; j < n; j += kThreads) twice |= A.slots[j] == slot;
    const bool any = __ballot(twice) != 0;
    if (lane == 0) s_twice[wave] = any;
    lds_barrier();
    if (s_twice[0] | s_twice[1] | s_twice[2] | s_twice[3]) {  // a repeated slot: a padded row
        if (out && rg == 0) store4(out + 4 * cg, Mma<T>::pack(zero4()));
        return;
    }
    const float a = expf(la);
    float kq = 0.f;  // k . (scale q), summed as walk does
    if (wave == 0) {
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) kq = fmaf(s_k[t % 16 + 16 * c], s_q[t % 16 + 16 * c], kq);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) kq += __shfl_xor(kq, off);
    }
    f32x4 w = zero4(), b = zero4();
#pragma unroll
    for (int i = 0; i < L::RPT; ++i) {
        w = fma4(s_k[rg + L::ROWG * i], s[i], w);
        b = fma4(s_q[rg + L::ROWG * i], s[i], b);
    }
#pragma unroll
    for (int off = L::COLG; off < 64; off <<= 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[c] += __shfl_xor(w[c], off);
            b[c] += __shfl_xor(b[c], off);
        }
    }
    if (lane < L::COLG) {
        s_red[wave][lane][0] = w;
        s_red[wave][lane][1] = b;
    }
    lds_barrier();
    w = (s_red[0][cg][0] + s_red[1][cg][0]) + (s_red[2][cg][0] + s_red[3][cg][0]);
    b = (s_red[0][cg][1] + s_red[1][cg][1]) + (s_red[2][cg][1] + s_red[3][cg][1]);
    const f32x4 u = be * fma4(-a, w, v);
    if (adv) {
#pragma unroll
        for (int i = 0; i < L::RPT; ++i)
            __builtin_nontemporal_store(fma4(s_k[rg + L::ROWG * i], u, a * s[i]), reinterpret_cast<f32x4*>(S + i * STEP));
    }
    if (out && rg == 0) store4(out + 4 * cg, Mma<T>::pack(fma4(kq, u, a * b)));  // (wave 0)
}

// The prefill of 32-bit inputs, token by token.  Each wave keeps 4 CW columns of a state for the
// whole sequence: lane (rg, cp) (rg = lane & 15) holds columns CW cp .. of DK / 16 consecutive
// rows, so a column sum is four rotations within the 16 lanes of a DPP row and the waves meet
// only once per 16 staged tokens (with a state's rows spread over four waves, as in the step, the
// barrier and the shuffles through LDS take 0.73 us a token of 64 key channels; this takes 0.12,
// 0.15 with 128).  Bound by the dependent chain of a token (sum, update, next token's sum) and
// its issue: the readout's sum is taken behind the update, off that chain, the next token's
// operands leave LDS a token ahead, and the tokens of a block are unrolled (0.19 in a loop).
template <int DK, int DV, int CW>
__global__ __launch_bounds__(kThreads) void seq_kernel(const RecArgs A, const GdnTable tab) {
    constexpr int TB = 16, NV = 16 * CW, SL = DV / NV, R = DK / 16;
    constexpr int QV = TB * DK / 4 / kThreads;
    typedef float Cols __attribute__((ext_vector_type(CW)));
    __shared__ __attribute__((aligned(16))) float s_k[2][TB][DK], s_q[2][TB][DK], s_v[2][TB][NV], s_o[2][TB][NV];
    __shared__ float s_a[2][TB], s_b[2][TB];
    const int t = threadIdx.x, lane = t & 63, rg = lane & 15, cp = lane >> 4;
    const int64_t pair = blockIdx.x / SL;
    const int i = (int)(pair / A.hv), head = (int)(pair % A.hv), hk = head / (A.hv / A.hk), col0 = NV * (int)(blockIdx.x % SL);
    const int col = 4 * CW * (t / 64) + CW * cp;  // of the slice
    const int64_t start = tab.start[i], ss = ((int64_t)tab.id[i] * A.hv + head) * (int64_t)(DK * DV);
    const int len = tab.len[i];
    const int64_t at = ss + (int64_t)rg * R * DV + col0 + col;
    Cols s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (A.S0) s[r] = *reinterpret_cast<const Cols*>(A.S0 + at + r * DV);
        else s[r] = Cols(0.f);
    }
    // tokens on their way: rows of k and q, CW entries of v, a gate
    f32x4 rk[QV], rq[QV];
    Cols rv;
    float rg_ = 0.f, rb = 0.f;
    const int vr = t / 16, vc = CW * (t % 16);
    auto load = [&](int t0) {
#pragma unroll
        for (int x = 0; x < QV; ++x) {
            const int e = t + kThreads * x, row = e / (DK / 4), c = 4 * (e % (DK / 4));
            rk[x] = rq[x] = zero4();
            if (t0 + row < len) {
                rk[x] = load4f((const float*)A.k + (start + t0 + row) * A.ks + (int64_t)hk * DK + c);
                rq[x] = load4f((const float*)A.q + (start + t0 + row) * A.qs + (int64_t)hk * DK + c);
            }
        }
        rv = Cols(0.f);
        if (t0 + vr < len)
            rv = *reinterpret_cast<const Cols*>((const float*)A.v + (start + t0 + vr) * A.vs + (int64_t)head * DV + col0 + vc);
        rg_ = rb = 0.f;
        if (t < TB && t0 + t < len) {
            rg_ = A.la[(start + t0 + t) * A.hv + head];
            rb = A.be[(start + t0 + t) * A.hv + head];
        }
    };
    auto put = [&](int b) {
#pragma unroll
        for (int x = 0; x < QV; ++x) {
            const int e = t + kThreads * x, row = e / (DK / 4), c = 4 * (e % (DK / 4));
            *reinterpret_cast<f32x4*>(&s_k[b][row][c]) = rk[x];
            *reinterpret_cast<f32x4*>(&s_q[b][row][c]) = rq[x] * A.scale;
        }
        *reinterpret_cast<Cols*>(&s_v[b][vr][vc]) = rv;
        if (t < TB) {
            s_a[b][t] = expf(rg_);
            s_b[b][t] = rb;
        }
    };
    auto sum16 = [](float x) {  // over the row of 16 lanes, in every lane
        x += dpp<0x128>(x);
        x += dpp<0x124>(x);
        x += dpp<0x122>(x);
        x += dpp<0x121>(x);
        return x;
    };
    auto store = [&](int t0) {  // a block's outputs: whole rows of the slice
        if (t0 + vr < len)
            *reinterpret_cast<Cols*>((float*)A.out + ((start + t0 + vr) * A.hv + head) * (int64_t)DV + col0 + vc) =
                *reinterpret_cast<const Cols*>(&s_o[(t0 / TB) & 1][vr][vc]);
    };
    struct Token {
        f32x4 k[R / 4], q[R / 4];
        Cols v;
        float a, b;
    };
    auto fetch = [&](int b, int j) {
        Token x;
#pragma unroll
        for (int r = 0; r < R / 4; ++r) {
            x.k[r] = *reinterpret_cast<const f32x4*>(&s_k[b][j][rg * R + 4 * r]);
            x.q[r] = *reinterpret_cast<const f32x4*>(&s_q[b][j][rg * R + 4 * r]);
        }
        x.v = *reinterpret_cast<const Cols*>(&s_v[b][j][col]);
        x.a = s_a[b][j];
        x.b = s_b[b][j];
        return x;
    };
    load(0);
    for (int t0 = 0; t0 < len; t0 += TB) {
        const int b = (t0 / TB) & 1;
        put(b);
        lds_barrier();
        if (t0 > 0) store(t0 - TB);
        load(t0 + TB);
        // Rows behind the last token are zeros with a = 1 and b = 0 and leave the state as it is,
        // so a block is always whole and its loop unrolled.  Lane rg keeps token rg's outputs.
        Token x = fetch(b, 0);
        Cols mine = Cols(0.f);
        unroll<0, TB>([&](auto J) {
            constexpr int j = decltype(J)::value;
            Token y = x;
            if constexpr (j + 1 < TB) y = fetch(b, j + 1);
            Cols w = Cols(0.f), o = Cols(0.f);
#pragma unroll
            for (int r = 0; r < R; ++r) w += s[r] * x.k[r / 4][r % 4];
#pragma unroll
            for (int c = 0; c < CW; ++c) w[c] = sum16(w[c]);
            const Cols u = x.b * (x.v - x.a * w);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r] = x.a * s[r] + x.k[r / 4][r % 4] * u;
                o += s[r] * x.q[r / 4][r % 4];
            }
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                const float sum = sum16(o[c]);
                mine[c] = rg == j ? sum : mine[c];
            }
            x = y;
            __builtin_amdgcn_sched_barrier(0);  // (operands one token ahead, not more: registers)
        });
        *reinterpret_cast<Cols*>(&s_o[b][rg][col]) = mine;
    }
    lds_barrier();
    if (len > 0) store((len - 1) / TB * TB);
    if (A.Sf) {
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<Cols*>(A.Sf + at + r * DV) = s[r];
    }
}

// f(T, DK, DV, NV) for the call's type and shapes
template <typename F>
hipError_t dispatch(const GdnDims& d, int nv, F&& f) {
    auto nvs = [&](auto t, auto dk, auto dv) {
        if (nv == 32) return f(t, dk, dv, std::integral_constant<int, 32>{});
        return f(t, dk, dv, std::integral_constant<int, 64>{});
    };
    auto dvs = [&](auto t, auto dk) {
        if (d.dv == 128) return nvs(t, dk, std::integral_constant<int, 128>{});
        return nvs(t, dk, std::integral_constant<int, 64>{});
    };
    auto dks = [&](auto t) {
        if (d.dk == 128) return dvs(t, std::integral_constant<int, 128>{});
        return dvs(t, std::integral_constant<int, 64>{});
    };
    return d.dtype == DTYPE_BF16 ? dks(bf16{}) : dks(float{});
}

RecArgs common(const GdnDims& d) {
    RecArgs r = {};
    r.qs = d.qs; r.ks = d.ks; r.vs = d.vs; r.hk = d.hk; r.hv = d.hv; r.scale = d.scale;
    return r;
}

}  // namespace

hipError_t launch_gdn_recurrent(const GdnRecurrentArgs& a, hipStream_t stream) {
    RecArgs r = common(a.d);
    r.q = a.q; r.k = a.k; r.v = a.v; r.la = a.log_alpha; r.be = a.beta; r.out = a.out;
    r.num_tokens = a.num_tokens; r.num_slots = a.num_slots;
    r.steps = a.steps; r.slots = a.state_indices; r.state = a.state; r.update = a.update;
    const int64_t blocks = (int64_t)a.num_seqs * a.d.hv * (a.d.dv / a.nv);
    if (blocks == 0) return hipSuccess;
    return dispatch(a.d, a.nv, [&](auto t, auto dk, auto dv, auto nv) {
        using T = decltype(t);
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, NV = decltype(nv)::value;
        if (a.num_tokens == 1 && a.nv == DV)  // whole rows
            hipLaunchKernelGGL((decode_kernel<T, DK, DV, DV>), dim3((unsigned)blocks), dim3(kThreads), (whole_lds<DK, DV>()), stream, r);
        else if (a.num_tokens == 1)
            hipLaunchKernelGGL((decode_kernel<T, DK, DV, 32>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, r);
        else if (a.num_tokens <= 4)
            hipLaunchKernelGGL((step_kernel<T, DK, DV, NV, 4>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, r);
        else
            hipLaunchKernelGGL((step_kernel<T, DK, DV, NV, 16>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, r);
        return hipGetLastError();
    });
}

hipError_t launch_gdn_sequential(const GdnPrefillArgs& a, const GdnTable& tab, hipStream_t stream) {
    RecArgs r = common(a.d);
    r.q = a.q; r.k = a.k; r.v = a.v; r.la = a.log_alpha; r.be = a.beta; r.out = a.out;
    r.S0 = a.initial_state; r.Sf = a.final_state;
    const int64_t blocks = (int64_t)a.num_seqs * a.d.hv * (a.d.dv / a.nv);
    if (a.d.dtype != DTYPE_F32) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    auto go = [&](auto dk, auto dv, auto cw) {
        hipLaunchKernelGGL((seq_kernel<decltype(dk)::value, decltype(dv)::value, decltype(cw)::value>), dim3((unsigned)blocks),
                           dim3(kThreads), 0, stream, r, tab);
        return hipGetLastError();
    };
    auto widths = [&](auto dk, auto dv) {
        return a.nv == 16 ? go(dk, dv, std::integral_constant<int, 1>{}) : go(dk, dv, std::integral_constant<int, 2>{});
    };
    auto values = [&](auto dk) {
        return a.d.dv == 128 ? widths(dk, std::integral_constant<int, 128>{}) : widths(dk, std::integral_constant<int, 64>{});
    };
    return a.d.dk == 128 ? values(std::integral_constant<int, 128>{}) : values(std::integral_constant<int, 64>{});
}

}  // namespace kda
