// spec_accept.hip -- verification of drafted tokens against the target's probabilities
// from given uniform random numbers (gfx950).
//
// Sequence n has K drafts x_j with draft probabilities q_j (or none: a draft is then a
// certain one, q_j(x_j) = 1) and target probabilities p_0 .. p_K.  Draft j is kept while
//   u_j q_j(x_j) < p_j(x_j);
// a = the number kept before the first that is not.  The next token is drawn with u_K from
//   r = max(p_a - q_a, 0)  if a draft was rejected at a (p_a if r is zero everywhere),
//   r = p_a                if all were kept,
// as the smallest i with r_0 + .. + r_i > u_K sum(r).  All products, differences and sums
// are fp64: the products and differences of fp32 values are exact there, and a draw is
// decided by where a sum over the whole vocabulary crosses a border.
//
// Bound by reading one row of p and one of q per sequence; everything else is latency.  A row
// that fits the registers of one workgroup takes one launch (32000 entries of fp32: 8.8 us for one
// sequence, about two of them the launch itself and the rest three dependent loads and the row).
// Longer vocabularies are cut into pieces, so that one sequence also spreads over the card: a
// first launch finds the kept drafts and sums each piece (128 sequences of 151669 entries, 155 MB:
// 23.6 us, 6.6 TB/s with part of it in the last-level cache), a second finds the piece that holds
// the draw from the sums (in piece order: the same result whatever ran first) and scans that piece
// alone (5.1 us; 13.9 with four waves, scans through LDS and atomic minima).
#include "gdn_launch.h"
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// kept drafts of sequence n (every lane of wave 0 returns it); x: the rejected draft, or -1
template <typename T>
__device__ int count_kept(const AcceptArgs& A, int n, int lane, bool* rejected) {
    int m = A.num_draft;
    if (A.num_drafts) m = min(max(A.num_drafts[n], 0), A.num_draft);
    bool keep = false;
    if (lane < m) {
        const int64_t row = (int64_t)n * (A.num_draft + 1) + lane, drow = (int64_t)n * A.num_draft + lane;
        const int64_t x = A.tokens[drow];
        if (x >= 0 && x < A.vocab) {  // a token outside the vocabulary is rejected, never read
            const double px = to_f32(((const T*)A.p)[row * A.vocab + x]);
            const double qx = A.q ? (double)to_f32(((const T*)A.q)[drow * A.vocab + x]) : 1.0;
            keep = (double)A.uniforms[row] * qx < px;
        }
    }
    const unsigned long long miss = ~__ballot(keep);  // lanes >= m miss
    const int a = miss ? (int)__builtin_ctzll(miss) : 64;
    *rejected = a < m;
    return a;
}

// the entry's weight in the draw, and in the fallback (p alone)
struct Weights {
    double r, p;
};
template <typename T>
__device__ inline Weights weights(const T* p, const T* q, int64_t i, int64_t certain) {
    const double pv = to_f32(p[i]);
    Weights w;
    w.p = pv > 0.0 ? pv : 0.0;
    w.r = w.p;
    if (q) {
        const double d = pv - (double)to_f32(q[i]);
        w.r = d > 0.0 ? d : 0.0;  // NaN counts as nothing
    }
    if (i == certain) w.r = 0.0;
    return w;
}

__device__ inline double wave_sum(double x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off);
    return x;
}

struct Row {
    int kept;
    bool rejected;
};

template <typename T>
__device__ Row find_row(const AcceptArgs& A, int n) {
    __shared__ int s_row[2];
    if (threadIdx.x < 64) {
        bool rej;
        const int a = count_kept<T>(A, n, threadIdx.x, &rej);
        if (threadIdx.x == 0) {
            s_row[0] = a;
            s_row[1] = rej;
        }
    }
    __syncthreads();
    return Row{s_row[0], s_row[1] != 0};
}

template <typename T>
__device__ void row_of(const AcceptArgs& A, int n, const Row& R, const T*& p, const T*& q, int64_t& certain) {
    p = (const T*)A.p + ((int64_t)n * (A.num_draft + 1) + R.kept) * A.vocab;
    q = nullptr;
    certain = -1;
    if (R.rejected) {
        const int64_t drow = (int64_t)n * A.num_draft + R.kept;
        if (A.q) q = (const T*)A.q + drow * A.vocab;
        else certain = A.tokens[drow];
    }
}

// Sixteen bytes of a row from entry i on (any alignment of the entries' own size), as fp64
template <typename T>
struct Packed {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
} __attribute__((packed, aligned(sizeof(T))));

// the weights of entries i .. i+N-1, all inside the row: r (and p, where given)
template <typename T>
__device__ inline void weights16(const T* p, const T* q, int64_t i, int64_t certain, double (&r)[Packed<T>::N], double (&pp)[Packed<T>::N]) {
    constexpr int N = Packed<T>::N;
    const Packed<T> a = *reinterpret_cast<const Packed<T>*>(p + i);
    Packed<T> b;
    if (q) b = *reinterpret_cast<const Packed<T>*>(q + i);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const double pv = to_f32(a.v[j]);
        pp[j] = pv > 0.0 ? pv : 0.0;
        r[j] = pp[j];
        if (q) {
            const double d = pv - (double)to_f32(b.v[j]);
            r[j] = d > 0.0 ? d : 0.0;  // NaN counts as nothing
        }
        if (i + j == certain) r[j] = 0.0;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sum_kernel(const AcceptArgs A) {
    constexpr int N = Packed<T>::N;
    __shared__ double s_sum[4][2];
    const int n = blockIdx.x / A.pieces, piece = blockIdx.x % A.pieces;
    const Row R = find_row<T>(A, n);
    const T *p, *q;
    int64_t certain;
    row_of(A, n, R, p, q, certain);
    if (piece == 0 && threadIdx.x == 0) A.accepted[n] = R.kept;
    const int64_t lo = piece * A.piece, hi = min(lo + A.piece, A.vocab);
    double sr = 0.0, sp = 0.0;
    const int64_t whole = (hi - lo) / (N * kThreads) * (N * kThreads);
#pragma unroll 2
    for (int64_t i = lo + N * threadIdx.x; i < lo + whole; i += N * kThreads) {
        double r[N], pp[N];
        weights16(p, q, i, certain, r, pp);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            sr += r[j];
            sp += pp[j];
        }
    }
    for (int64_t i = lo + whole + threadIdx.x; i < hi; i += kThreads) {
        const Weights w = weights(p, q, i, certain);
        sr += w.r;
        sp += w.p;
    }
    sr = wave_sum(sr);
    sp = wave_sum(sp);
    if (threadIdx.x % 64 == 0) {
        s_sum[threadIdx.x / 64][0] = sr;
        s_sum[threadIdx.x / 64][1] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2)
        A.partial[2 * (int64_t)blockIdx.x + threadIdx.x] =
            (s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x]) + (s_sum[2][threadIdx.x] + s_sum[3][threadIdx.x]);
}

constexpr int kOneThreads = 1024;  // of the launches that draw

__device__ inline int first_of(unsigned long long m) { return (int)__builtin_ctzll(m); }
__device__ inline int last_of(unsigned long long m) { return 63 - (int)__builtin_clzll(m); }

// Where the running sum of PL values per lane (x, in lane order, behind `before`) first exceeds
// `target`: that value's place, and the sum in front of it; with none, the last value above 0 and
// found = false.  Every lane returns the same.
template <int PL>
__device__ inline int crossing(const double (&x)[PL], double before, double target, int lane, double& front, bool& found) {
    double mine = 0.0;
#pragma unroll
    for (int e = 0; e < PL; ++e) mine += x[e];
    double c = before + (wave_scan_f64(mine) - mine), at = 0.0;
    int first = -1, last = -1;
#pragma unroll
    for (int e = 0; e < PL; ++e) {
        if (x[e] > 0.0) {
            if (first < 0 && c + x[e] > target) {
                first = PL * lane + e;
                at = c;
            }
            last = PL * lane + e;
        }
        c += x[e];
    }
    const unsigned long long hit = __ballot(first >= 0), any = __ballot(last >= 0);
    found = hit != 0;
    if (!any) return -1;
    const int src = hit ? first_of(hit) : last_of(any);
    front = __shfl(at, src);
    return __builtin_amdgcn_readfirstlane(__shfl(hit ? first : last, src));
}

// The second launch: the piece of the draw from the pieces' sums (every wave by itself), then its
// entry, a round of N per thread at a time (a piece is one round, but of vocabularies above 2^20).
template <typename T>
__global__ __launch_bounds__(kOneThreads) void draw_kernel(const AcceptArgs A) {
    constexpr int N = Packed<T>::N, WAVES = kOneThreads / 64, PL = 4;
    __shared__ double s_seg[2][WAVES];
    __shared__ int s_end;
    const int n = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    Row R;
    R.kept = A.accepted[n];  // the first launch's
    R.rejected = R.kept < (A.num_drafts ? min(max(A.num_drafts[n], 0), A.num_draft) : A.num_draft);
    const T *p, *q;
    int64_t certain;
    row_of(A, n, R, p, q, certain);
    double x[PL], xp[PL], mine = 0.0, mine_p = 0.0;
#pragma unroll
    for (int e = 0; e < PL; ++e) {
        const int piece = PL * lane + e;
        const bool in = piece < A.pieces;
        x[e] = in ? A.partial[2 * ((int64_t)n * A.pieces + piece)] : 0.0;
        xp[e] = in ? A.partial[2 * ((int64_t)n * A.pieces + piece) + 1] : 0.0;
        mine += x[e];
        mine_p += xp[e];
    }
    const double u = (double)A.uniforms[(int64_t)n * (A.num_draft + 1) + A.num_draft];
    int32_t* out = A.out + (int64_t)n * (A.num_draft + 1);
    if (t <= A.num_draft && t != R.kept) out[t] = t < R.kept ? A.tokens[(int64_t)n * A.num_draft + t] : -1;
    if (t == 0) s_end = -1;
    double all = __shfl(wave_scan_f64(mine), 63);
    const bool plain = !(all > 0.0);  // nothing left: draw from p
    if (plain) {
        all = __shfl(wave_scan_f64(mine_p), 63);
#pragma unroll
        for (int e = 0; e < PL; ++e) x[e] = xp[e];
    }
    const double target = u * all;
    double before;
    bool inside;
    const int piece = crossing<PL>(x, 0.0, target, lane, before, inside);
    if (piece < 0) {  // no entry has any weight
        if (t == 0) out[R.kept] = -1;
        return;
    }
    const int64_t lo = piece * A.piece, hi = min(lo + A.piece, A.vocab);
    int turn = 0;
    int64_t last = -1;
    for (int64_t at = lo; at < hi; at += N * kOneThreads) {
        // (entries behind the piece's end: the row's last N again, weighing nothing)
        const int64_t own = at + N * t, from = min(own, A.vocab - N);
        double w[N], sum = 0.0, r[N] = {}, pp[N] = {};
        if (A.vocab >= N) {
            weights16(p, q, from, certain, r, pp);
        } else if (t == 0) {
            for (int e = 0; e < (int)A.vocab; ++e) {
                const Weights y = weights(p, q, e, certain);
                r[e - (int)from] = y.r;
                pp[e - (int)from] = y.p;
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            w[e] = from + e >= own && from + e < hi ? (plain ? pp[e] : r[e]) : 0.0;
            sum += w[e];
        }
        const double inc = wave_scan_f64(sum);
        if (lane == 63) s_seg[turn][wave] = inc;
        __syncthreads();
        const double seg[1] = {lane < WAVES ? s_seg[turn][lane] : 0.0};
        turn ^= 1;
        double front;
        bool found;
        const int s = crossing<1>(seg, before, inside ? target : __builtin_inf(), lane, front, found);
        if (found) {
            if (s != wave) return;
            double c = front + (inc - sum);
            int first = -1, end = -1;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                c += w[e];
                if (w[e] > 0.0) {
                    if (first < 0 && c > target) first = (int)(from + e);
                    end = (int)(from + e);
                }
            }
            const unsigned long long hit = __ballot(first >= 0);
            const int who = hit ? first_of(hit) : last_of(__ballot(end >= 0));
            if (lane == who) out[R.kept] = hit ? first : end;
            return;
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (w[e] > 0.0) last = from + e;
        before += __shfl(wave_scan_f64(seg[0]), 63);
    }
    // u * total not below any sum: the piece's last entry
    if (last >= 0) atomicMax(&s_end, (int)last);
    __syncthreads();
    if (t == 0) out[R.kept] = s_end;
}

// The whole of it in one workgroup per sequence, its two rows in registers: thread t holds
// entries N (1024 j + t) .. +N-1 of every round j, so the order of the vocabulary is that of
// (round, wave, lane).  A segment is a round's share of a wave; the segment of the draw is found
// from all segments' sums by every wave, the entry by the segment's own.
template <typename T, int ROUNDS>
__global__ __launch_bounds__(kOneThreads) void one_kernel(const AcceptArgs A) {
    constexpr int N = Packed<T>::N, WAVES = kOneThreads / 64, SEG = WAVES * ROUNDS, PL = (SEG + 63) / 64;
    __shared__ double s_seg[2][SEG];
    const int n = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    Row R;
    R.kept = count_kept<T>(A, n, lane, &R.rejected);  // (every wave: no wait for another's)
    const T *p, *q;
    int64_t certain;
    row_of(A, n, R, p, q, certain);
    // entries behind the row's end: the last N are loaded again, and weigh nothing where they
    // lie before the thread's own
    const int vocab = (int)A.vocab;
    auto own = [&](int j) { return N * (kOneThreads * j + t); };
    auto from = [&](int j) { return min(own(j), vocab - N); };
    u32x4 a[ROUNDS], b[ROUNDS] = {};
    auto load = [](const T* x) { return __builtin_bit_cast(u32x4, *reinterpret_cast<const Packed<T>*>(x)); };
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) a[j] = load(p + from(j));
    if (q) {
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) b[j] = load(q + from(j));
    }
    const double u = (double)A.uniforms[(int64_t)n * (A.num_draft + 1) + A.num_draft];
    int32_t* out = A.out + (int64_t)n * (A.num_draft + 1);
    if (t == 0) A.accepted[n] = R.kept;
    if (t <= A.num_draft && t != R.kept) out[t] = t < R.kept ? A.tokens[(int64_t)n * A.num_draft + t] : -1;
    // first the draw's weights, then (nothing left of them) p's
#pragma unroll 1
    for (int plain = 0; plain < 2; ++plain) {
        // (opaque, or the compiler keeps every entry's fp64 forms across the loop: twice the registers)
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) asm volatile("" : "+v"(a[j]), "+v"(b[j]));
        auto weight = [&](u32x4 pw, u32x4 qw, int j, int e) {
            const Packed<T> pe = __builtin_bit_cast(Packed<T>, pw), qe = __builtin_bit_cast(Packed<T>, qw);
            const double pv = to_f32(pe.v[e]);
            double w = pv > 0.0 ? pv : 0.0;
            if (!plain) {
                if (q) {
                    const double d = pv - (double)to_f32(qe.v[e]);
                    w = d > 0.0 ? d : 0.0;  // NaN counts as nothing
                }
                if (from(j) + e == certain) w = 0.0;
            }
            return from(j) + e >= own(j) ? w : 0.0;
        };
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
            double sum = 0.0;
#pragma unroll
            for (int e = 0; e < N; ++e) sum += weight(a[j], b[j], j, e);
            sum = wave_scan_f64(sum);
            if (lane == 63) s_seg[plain][WAVES * j + wave] = sum;
            __builtin_amdgcn_sched_barrier(0);  // (one round's fp64 at a time in registers)
        }
        __syncthreads();
        double x[PL], mine = 0.0;
#pragma unroll
        for (int e = 0; e < PL; ++e) {
            x[e] = PL * lane + e < SEG ? s_seg[plain][PL * lane + e] : 0.0;
            mine += x[e];
        }
        const double all = __shfl(wave_scan_f64(mine), 63);
        if (!(all > 0.0)) continue;  // (the same in every wave)
        const double target = u * all;
        double before;
        bool hit;
        const int seg = crossing<PL>(x, 0.0, target, lane, before, hit);
        if (seg % WAVES != wave) return;
        const int round = seg / WAVES;
        u32x4 pe = a[0], qe = b[0];
#pragma unroll
        for (int j = 1; j < ROUNDS; ++j)
            if (j == round) {
                pe = a[j];
                qe = b[j];
            }
        double w[N], sum = 0.0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            w[e] = weight(pe, qe, round, e);
            sum += w[e];
        }
        double s = before + (wave_scan_f64(sum) - sum);
        int at = -1, end = -1;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            s += w[e];
            if (w[e] > 0.0) {
                if (hit && at < 0 && s > target) at = from(round) + e;
                end = from(round) + e;
            }
        }
        const unsigned long long inside = __ballot(at >= 0);
        const int who = inside ? first_of(inside) : last_of(__ballot(end >= 0));
        if (lane == who) out[R.kept] = inside ? at : end;
        return;
    }
    if (t == 0) out[R.kept] = -1;  // no entry has any weight
}

template <typename T>
hipError_t launch_typed(const AcceptArgs& a, hipStream_t stream) {
    if (accept_in_one(a.vocab)) {
        // the fewest rounds (a power of two) that hold a row
        constexpr int64_t round = kOneThreads * Packed<T>::N;
        const dim3 grid((unsigned)a.num_seqs), block(kOneThreads);
        if (a.vocab <= round) hipLaunchKernelGGL((one_kernel<T, 1>), grid, block, 0, stream, a);
        else if (a.vocab <= 2 * round) hipLaunchKernelGGL((one_kernel<T, 2>), grid, block, 0, stream, a);
        else if (a.vocab <= 4 * round) hipLaunchKernelGGL((one_kernel<T, 4>), grid, block, 0, stream, a);
        else if constexpr (sizeof(T) == 4) hipLaunchKernelGGL((one_kernel<T, 8>), grid, block, 0, stream, a);
        static_assert((sizeof(T) == 4 ? 8 : 4) * round == kAcceptOne, "the largest takes every row");
        return hipGetLastError();
    }
    hipLaunchKernelGGL((sum_kernel<T>), dim3((unsigned)(a.num_seqs * (int64_t)a.pieces)), dim3(kThreads), 0,
                       stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((draw_kernel<T>), dim3((unsigned)a.num_seqs), dim3(kOneThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_accept(const AcceptArgs& a, hipStream_t stream) {
    if (a.num_seqs == 0) return hipSuccess;
    return a.dtype == DTYPE_BF16 ? launch_typed<bf16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace kda
