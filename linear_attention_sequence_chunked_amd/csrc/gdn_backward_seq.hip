// gdn_backward_seq.hip -- gradients of the gated delta rule token by token (gfx950): the form
// of 32-bit inputs.
//
// Per (sequence, value head), backwards over the tokens, D the gradient of the state behind
// token t (A = e^{g} S the decayed state, err = v - A^T k, u = beta err, S' = A + k u^T):
//   dq = scale S' do            D += scale q do^T           du = D^T k
//   dk = D u - A (beta du)      dbeta = du . err            dv = beta du
//   D -= k (beta du)^T          dg = <D, A>                 D <- e^{g} D
// A walk forwards keeps the state before every 16th token; backwards, each block of 16 is run
// again from there with its decayed states A written to a scratch (1 MiB per workgroup, the next
// token's read during this one's sums), so no state is ever divided by its decay.  Everything is
// fp32.
//
// One workgroup of four waves holds a state, or 32 of its columns: thread t has columns 4 (t % COLG) .. +3 of
// RPT consecutive rows.  Column sums (du) go through LDS, one barrier per token; row sums
// (dq, dk) are reduced among the COLG threads of a row group, halving the rows at each step; the
// gates' sums over the state (dg, dbeta) are kept per thread and added once per block.
// States of 128 x 128: up to 64 of them, in slices, 2.2 to 2.6 us a token, latency of the three
// walks' sums and barriers; whole ones 4.3, of which about 2.5 are the issue of some 1500 vector
// instructions by each of the four SIMDs; 6.6 with a state on each of 256 compute units, where
// the scratch's 128 KiB a token come from beyond L2 at 5 TB/s.
//
// Heads that share a key head, and slices, write their parts of dq and dk apart; a second launch
// adds them in order (and a third the gates' of the slices).
#include <algorithm>

#include "gdn_launch.h"
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int TB = 16;

__device__ inline f32x4 load4f(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// NV columns of a state in one workgroup
template <int DK, int DV, int NV>
struct Shape {
    static constexpr int COLG = NV / 4, ROWG = kThreads / COLG, RPT = DK / ROWG, SL = DV / NV;
    static constexpr int64_t STATE = (int64_t)DK * DV, OWN = (int64_t)DK * NV;
};

// x of the lane whose number differs in bit OFF: one DPP move, or a trip through LDS for 4 and 16
template <int OFF>
__device__ inline float partner(float x) {
    if constexpr (OFF == 1) return dpp<0xB1>(x);
    else if constexpr (OFF == 2) return dpp<0x4E>(x);
    else if constexpr (OFF == 8) return dpp<0x128>(x);
    else return __shfl_xor(x, OFF);
}

// Sums over LANES neighbouring threads of N values each, halving the values at each step: a
// thread returns the sum of value `row`, chosen by the lane bits that the halvings took
// (kTaken<N>).  (A recursion: in a loop whose bound halves the compiler keeps the array's indexes
// dynamic, a select per element and access, which took 8.7 of 13.5 us a token.)
template <int LANES>
constexpr int offset(int step) {  // the moves first
    constexpr int few[3] = {1, 2, 4}, many[5] = {1, 2, 8, 4, 16};
    return LANES == 8 ? few[step] : many[step];
}
template <int N>
constexpr int kTaken = N == 16 ? 15 : N == 8 ? 11 : N - 1;
template <int N, int LANES, int STEP = 0>
__device__ inline float reduce_rows(const float (&v)[N], int c, int& row) {
    if constexpr ((1 << STEP) == LANES) {
        static_assert(N == 1, "no more values than lanes");
        return v[0];
    } else if constexpr (N == 1) {
        const float x[1] = {v[0] + partner<offset<LANES>(STEP)>(v[0])};
        return reduce_rows<1, LANES, STEP + 1>(x, c, row);
    } else {
        constexpr int OFF = offset<LANES>(STEP);
        const bool up = c & OFF;
        float h[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = up ? v[i + N / 2] : v[i], give = up ? v[i] : v[i + N / 2];
            h[i] = keep + partner<OFF>(give);
        }
        row += up ? N / 2 : 0;
        return reduce_rows<N / 2, LANES, STEP + 1>(h, c, row);
    }
}

__device__ inline float sum16(float x) {  // over the row of 16 lanes
    x += dpp<0x128>(x);
    x += dpp<0x124>(x);
    x += dpp<0x122>(x);
    x += dpp<0x121>(x);
    return x;
}

template <int DK, int DV, int NV>
__global__ __launch_bounds__(kThreads) void backward_kernel(const GdnBackwardArgs A, const GdnTable tab, int units) {
    using L = Shape<DK, DV, NV>;
    constexpr int COLG = L::COLG, RPT = L::RPT, SL = L::SL;
    __shared__ __attribute__((aligned(16))) float s_k[TB][DK], s_q[TB][DK], s_v[TB][NV], s_do[TB][NV], s_err[TB][NV];
    __shared__ float s_a[TB], s_b[TB], s_g[TB][kThreads], s_db[TB][COLG];
    __shared__ f32x4 s_red[2][4][COLG];
    const int t = threadIdx.x, cg = t % COLG, rg = t / COLG, wave = t / 64, lane = t % 64;
    float* scratch = A.scratch + (int64_t)blockIdx.x * TB * L::OWN + (rg * RPT) * NV + 4 * cg;
    const GdnDims& d = A.d;

    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int pair = unit / SL, slice = unit % SL, col0 = NV * slice;
        const int64_t at = (int64_t)(rg * RPT) * DV + col0 + 4 * cg;
        const int si = pair / d.hv, h = pair % d.hv, hk = h / (d.hv / d.hk), len = tab.len[si], id = tab.id[si];
        const int64_t start = tab.start[si], ss = ((int64_t)id * d.hv + h) * L::STATE;
        // the state before block b of this sequence and head
        float* keep = A.checkpoints + ((start / TB + id) * d.hv + (int64_t)h * ((len + TB - 1) / TB)) * L::STATE;
        const int blocks = (len + TB - 1) / TB;

        auto stage = [&](int b) {
            const int m = min(TB, len - TB * b);
            const int64_t row0 = start + (int64_t)TB * b;
            lds_barrier();
            for (int e = t; e < TB * DK / 4; e += kThreads) {
                const int r = e / (DK / 4), c = 4 * (e % (DK / 4));
                f32x4 kv = zero4(), qv = zero4();
                if (r < m) {
                    kv = load4f((const float*)A.k + (row0 + r) * d.ks + (int64_t)hk * DK + c);
                    qv = load4f((const float*)A.q + (row0 + r) * d.qs + (int64_t)hk * DK + c);
                }
                *reinterpret_cast<f32x4*>(&s_k[r][c]) = kv;
                *reinterpret_cast<f32x4*>(&s_q[r][c]) = qv * d.scale;
            }
            for (int e = t; e < TB * NV / 4; e += kThreads) {
                const int r = e / (NV / 4), c = 4 * (e % (NV / 4));
                f32x4 vv = zero4(), ov = zero4();
                if (r < m) {
                    vv = load4f((const float*)A.v + (row0 + r) * d.vs + (int64_t)h * DV + col0 + c);
                    ov = load4f((const float*)A.d_out + ((row0 + r) * d.hv + h) * (int64_t)DV + col0 + c);
                }
                *reinterpret_cast<f32x4*>(&s_v[r][c]) = vv;
                *reinterpret_cast<f32x4*>(&s_do[r][c]) = ov;
            }
            if (t < m) {
                s_a[t] = expf(A.log_alpha[(row0 + t) * d.hv + h]);
                s_b[t] = A.beta[(row0 + t) * d.hv + h];
            }
            lds_barrier();
            return m;
        };
        int turn = 0;
        // sum over all rows of this thread's columns
        auto column_sum = [&](f32x4 w) {
#pragma unroll
            for (int off = COLG; off < 64; off <<= 1)
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] += __shfl_xor(w[c], off);
            if (lane < COLG) s_red[turn][wave][lane] = w;
            lds_barrier();
            w = (s_red[turn][0][cg] + s_red[turn][1][cg]) + (s_red[turn][2][cg] + s_red[turn][3][cg]);
            turn ^= 1;
            return w;
        };
        f32x4 S[RPT];
        // tokens 0 .. m-1 of the staged block; SAVE: their decayed states to the scratch, and
        // err over v
        auto forward = [&](int m, bool save) {
            for (int j = 0; j < m; ++j) {
                f32x4 w = zero4();
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    S[i] *= s_a[j];
                    w += S[i] * s_k[j][rg * RPT + i];
                    if (save) *reinterpret_cast<f32x4*>(scratch + j * L::OWN + i * NV) = S[i];
                }
                w = column_sum(w);
                const f32x4 err = *reinterpret_cast<const f32x4*>(&s_v[j][4 * cg]) - w;
#pragma unroll
                for (int i = 0; i < RPT; ++i) S[i] += s_k[j][rg * RPT + i] * (s_b[j] * err);
                if (save && rg == 0) *reinterpret_cast<f32x4*>(&s_err[j][4 * cg]) = err;
            }
        };
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = A.initial_state ? *reinterpret_cast<const f32x4*>(A.initial_state + ss + at + i * DV) : zero4();
        for (int b = 0; b < blocks; ++b) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) *reinterpret_cast<f32x4*>(keep + b * L::STATE + at + i * DV) = S[i];
            if (b + 1 == blocks) break;
            forward(stage(b), false);
        }
        f32x4 D[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) D[i] = A.d_final_state ? *reinterpret_cast<const f32x4*>(A.d_final_state + ss + at + i * DV) : zero4();
        for (int b = blocks - 1; b >= 0; --b) {
            const int m = stage(b);
            const int64_t row0 = start + (int64_t)TB * b;
#pragma unroll
            for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const f32x4*>(keep + b * L::STATE + at + i * DV);
            forward(m, true);
            lds_barrier();
            auto decayed = [&](int j) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const f32x4*>(scratch + j * L::OWN + i * NV);
            };
            decayed(m - 1);
            for (int j = m - 1; j >= 0; --j) {
                const float a = s_a[j], be = s_b[j];
                const f32x4 err = *reinterpret_cast<const f32x4*>(&s_err[j][4 * cg]), u = be * err;
                const f32x4 go = *reinterpret_cast<const f32x4*>(&s_do[j][4 * cg]);
                float pq[RPT], pk[RPT];
                f32x4 w = zero4();
                auto dot = [](f32x4 x, f32x4 y) { return (x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]); };
                const float udo = dot(u, go);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float kr = s_k[j][rg * RPT + i];
                    pq[i] = dot(S[i], go) + kr * udo;  // of S' do
                    D[i] += s_q[j][rg * RPT + i] * go;
                    w += D[i] * kr;
                }
                const f32x4 du = column_sum(w), bdu = be * du;
                float dg = 0.f;
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    pk[i] = dot(D[i], u) - dot(S[i], bdu);
                    D[i] -= s_k[j][rg * RPT + i] * bdu;
                    dg += dot(D[i], S[i]);
                    D[i] *= a;
                }
                if (j > 0) decayed(j - 1);  // on their way during the sums over rows
                int row = 0, same = 0;
                const float rq = reduce_rows<RPT, COLG>(pq, cg, row), rk = reduce_rows<RPT, COLG>(pk, cg, same);
                if ((cg & ~kTaken<RPT>) == 0) {
                    const int64_t o = (A.parts ? ((row0 + j) * d.hv + h) * SL + slice : (row0 + j) * d.hk + hk) * (int64_t)DK + rg * RPT + row;
                    if (A.parts) {
                        A.dq_parts[o] = d.scale * rq;
                        A.dk_parts[o] = rk;
                    } else {
                        ((float*)A.dq)[o] = d.scale * rq;
                        ((float*)A.dk)[o] = rk;
                    }
                }
                s_g[j][t] = dg;  // summed over the threads behind the block
                if (rg == 0) {
                    *reinterpret_cast<f32x4*>((float*)A.dv + ((row0 + j) * d.hv + h) * (int64_t)DV + col0 + 4 * cg) = bdu;
                    s_db[j][cg] = dot(du, err);
                }
            }
            lds_barrier();
            {
                const int j = t / 16, l = t % 16;
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int i = 0; i < kThreads / 16; ++i) x += s_g[j][l + 16 * i];
#pragma unroll
                for (int i = 0; i < COLG; i += 16) y += i + l < COLG ? s_db[j][i + l] : 0.f;
                x = sum16(x);
                y = sum16(y);
                if (l == 0 && j < m) {
                    const int64_t o = ((row0 + j) * d.hv + h) * SL + slice;
                    (SL > 1 ? A.dg_parts : A.dlog_alpha)[o] = x;
                    (SL > 1 ? A.db_parts : A.dbeta)[o] = y;
                }
            }
        }
        if (A.d_initial_state) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) *reinterpret_cast<f32x4*>(A.d_initial_state + ss + at + i * DV) = D[i];
        }
        lds_barrier();
    }
}

// dq and dk of a key head: the sums over the parts of it (the value heads that share it, and the
// slices of their columns), in order
template <typename T>
__global__ __launch_bounds__(256) void sum_parts_kernel(const GdnBackwardArgs A, int64_t total4, int dk4, int parts) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total4) return;
    const int64_t c = i % dk4, th = i / dk4;  // th: token and key head
    const int64_t src = th * parts * dk4 + c;
    f32x4 q = zero4(), k = zero4();
    for (int n = 0; n < parts; ++n) {
        q += reinterpret_cast<const f32x4*>(A.dq_parts)[src + (int64_t)n * dk4];
        k += reinterpret_cast<const f32x4*>(A.dk_parts)[src + (int64_t)n * dk4];
    }
    store4((T*)A.dq + 4 * i, Mma<T>::pack(q));
    store4((T*)A.dk + 4 * i, Mma<T>::pack(k));
}
// the gates' gradients: sums over the slices
__global__ __launch_bounds__(256) void sum_gates_kernel(const GdnBackwardArgs A, int64_t total, int slices) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    float g = 0.f, b = 0.f;
    for (int n = 0; n < slices; ++n) {
        g += A.dg_parts[i * slices + n];
        b += A.db_parts[i * slices + n];
    }
    A.dlog_alpha[i] = g;
    A.dbeta[i] = b;
}

template <typename T>
hipError_t sum_parts(const GdnBackwardArgs& a, hipStream_t st) {
    const int64_t total4 = a.T * a.d.hk * (a.d.dk / 4), gates = a.T * a.d.hv;
    if (total4 == 0) return hipSuccess;
    hipLaunchKernelGGL((sum_parts_kernel<T>), dim3((unsigned)((total4 + 255) / 256)), dim3(256), 0, st, a, total4, a.d.dk / 4,
                       a.d.hv / a.d.hk * a.slices);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.slices == 1) return e;
    hipLaunchKernelGGL(sum_gates_kernel, dim3((unsigned)((gates + 255) / 256)), dim3(256), 0, st, a, gates, a.slices);
    return hipGetLastError();
}

template <int DK, int DV, int NV>
hipError_t launch(const GdnBackwardArgs& a, const GdnTable& tab, hipStream_t st) {
    const int units = a.num_seqs * a.d.hv * (DV / NV);
    if (units == 0) return hipSuccess;
    hipLaunchKernelGGL((backward_kernel<DK, DV, NV>), dim3((unsigned)std::min(units, a.slots)), dim3(kThreads), 0, st, a, tab, units);
    return hipGetLastError();
}
template <int DK, int DV>
hipError_t launch_nv(const GdnBackwardArgs& a, const GdnTable& tab, hipStream_t st) {
    return a.slices > 1 ? launch<DK, DV, 32>(a, tab, st) : launch<DK, DV, DV>(a, tab, st);
}

}  // namespace

hipError_t launch_gdn_backward_seq(const GdnBackwardArgs& a, const GdnTable& tab, hipStream_t st) {
    if (a.d.dtype != DTYPE_F32) return hipErrorInvalidValue;
    if (a.d.dk == 128) return a.d.dv == 128 ? launch_nv<128, 128>(a, tab, st) : launch_nv<128, 64>(a, tab, st);
    return a.d.dv == 128 ? launch_nv<64, 128>(a, tab, st) : launch_nv<64, 64>(a, tab, st);
}

hipError_t launch_gdn_sum_parts(const GdnBackwardArgs& a, hipStream_t st) {
    return a.d.dtype == DTYPE_BF16 ? sum_parts<bf16>(a, st) : sum_parts<float>(a, st);
}

}  // namespace kda
