// gdn_api.cpp -- C ABI of the gated delta rule and of draft verification: argument
// validation, scheduling, launch.  As in kda_api.cpp every check runs on the host before any
// HIP call, and a rejected call enqueues nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <numeric>
#include <vector>

#include "../../include/kda.h"
#include "gdn_launch.h"
#include "kda_check.h"

namespace {

using kda::check_ptr;
using kda::fail;
using kda::overlaps;
using kda::Range;
using kda::range;

// Nothing thrown inside crosses the C boundary (only the host tables allocate).
template <typename F>
auto guarded(const char* entry, F&& f) -> decltype(f()) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return static_cast<decltype(f())>(fail(KDA_ERR_HIP, "%s: out of host memory", entry));
    }
}

kda_status check_gdn(const kda_gdn_params* p, kda::GdnDims& d) {
    if (!p) return fail(KDA_ERR_INVALID_ARGUMENT, "params is NULL");
    if (p->dtype != KDA_DTYPE_BF16 && p->dtype != KDA_DTYPE_F32)
        return fail(KDA_ERR_INVALID_ARGUMENT, "dtype %d is not KDA_DTYPE_BF16 or KDA_DTYPE_F32", p->dtype);
    if (p->num_k_heads < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "num_k_heads %d < 1", p->num_k_heads);
    if (p->num_v_heads < 1 || p->num_v_heads % p->num_k_heads)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_v_heads %d is not a multiple of num_k_heads %d",
                    p->num_v_heads, p->num_k_heads);
    if ((p->dk != 64 && p->dk != 128) || (p->dv != 64 && p->dv != 128))
        return fail(KDA_ERR_UNSUPPORTED, "dk=%d dv=%d: each must be 64 or 128", p->dk, p->dv);
    if (!std::isfinite(p->scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale is not finite");
    const int64_t vec = p->dtype == KDA_DTYPE_BF16 ? 8 : 4;
    const int64_t nk = (int64_t)p->num_k_heads * p->dk, nv = (int64_t)p->num_v_heads * p->dv;
    const int64_t given[] = {p->q_stride, p->k_stride, p->v_stride}, dense[] = {nk, nk, nv};
    const char* names[] = {"q_stride", "k_stride", "v_stride"};
    int64_t s[3];
    for (int i = 0; i < 3; ++i) {
        s[i] = given[i] ? given[i] : dense[i];
        if (s[i] < dense[i] || s[i] % vec)
            return fail(KDA_ERR_INVALID_ARGUMENT, "%s %lld: at least %lld and a multiple of %lld is needed",
                        names[i], (long long)given[i], (long long)dense[i], (long long)vec);
        if (s[i] > 1 << 23)  // a chunk's 64 rows stay within 32-bit offsets
            return fail(KDA_ERR_UNSUPPORTED, "%s %lld exceeds 2^23", names[i], (long long)given[i]);
    }
    d = kda::GdnDims{p->dtype, p->num_k_heads, p->num_v_heads, p->dk, p->dv, p->scale, s[0], s[1], s[2]};
    return KDA_OK;
}

size_t element(const kda::GdnDims& d) { return d.dtype == KDA_DTYPE_BF16 ? 2 : 4; }

// bytes from the first token's row to the end of the last one's
uint64_t extent(int64_t tokens, int64_t stride, int64_t row, size_t es) {
    return tokens > 0 ? ((uint64_t)(tokens - 1) * stride + row) * es : 0;
}

// a grid's threads are counted in 32 bits
kda_status check_grid(int64_t blocks, int64_t threads) {
    if (blocks > UINT32_MAX / threads)
        return fail(KDA_ERR_UNSUPPORTED, "%lld workgroups exceed one launch", (long long)blocks);
    return KDA_OK;
}

// the (sequence, head) pairs of one launch, their columns cut finest, at most 1024 threads each
// (768 and two walks in the gradients' first)
kda_status check_pairs(const kda::GdnDims& d, int32_t num_seqs) {
    return check_grid(2 * ((int64_t)std::min(num_seqs, kda::kGdnSeqs) * d.hv * (d.dv / 16) + 64), 1024);
}

kda_status check_cu(const int32_t* cu, int32_t n) {
    if (n < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 1", n);
    if (!cu) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_host is NULL");
    if (cu[0] != 0) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_host[0] = %d, must be 0", cu[0]);
    for (int32_t i = 0; i < n; ++i)
        if (cu[i + 1] < cu[i])
            return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_host decreases at index %d", i + 1);
    return KDA_OK;
}

// the token inputs shared by the prefill and the recurrent form
kda_status check_tokens(const kda::GdnDims& d, int64_t T, const void* q, const void* k, const void* v,
                        const float* la, const float* be, Range (&in)[5]) {
    kda_status st;
    const size_t es = element(d);
    if (T > 0) {
        const void* p[] = {q, k, v};
        const char* names[] = {"q", "k", "v"};
        for (int i = 0; i < 3; ++i)
            if ((st = check_ptr(names[i], p[i], 16)) != KDA_OK) return st;
        if ((st = check_ptr("log_alpha", la, 4)) != KDA_OK) return st;
        if ((st = check_ptr("beta", be, 4)) != KDA_OK) return st;
    }
    in[0] = range("q", q, extent(T, d.qs, (int64_t)d.hk * d.dk, es));
    in[1] = range("k", k, extent(T, d.ks, (int64_t)d.hk * d.dk, es));
    in[2] = range("v", v, extent(T, d.vs, (int64_t)d.hv * d.dv, es));
    in[3] = range("log_alpha", la, (uint64_t)T * d.hv * 4);
    in[4] = range("beta", be, (uint64_t)T * d.hv * 4);
    return KDA_OK;
}

// sequence numbers, longest first: they bound a launch's critical path
std::vector<int32_t> longest_first(const int32_t* cu, int32_t n) {
    std::vector<int32_t> idx(n);
    std::iota(idx.begin(), idx.end(), 0);
    std::stable_sort(idx.begin(), idx.end(), [&](int32_t x, int32_t y) {
        return cu[x + 1] - cu[x] > cu[y + 1] - cu[y];
    });
    return idx;
}

// the next launch's sequences, from place `from` of the order on
int32_t fill_table(kda::GdnTable& t, const int32_t* cu, const std::vector<int32_t>& order, int32_t from) {
    const int32_t n = std::min<int32_t>((int32_t)order.size() - from, kda::kGdnSeqs);
    for (int32_t i = 0; i < n; ++i) {
        const int32_t s = order[from + i];
        t.start[i] = cu[s];
        t.len[i] = cu[s + 1] - cu[s];
        t.id[i] = s;
    }
    return n;
}

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

// Workspace of the backward: parts of dq and dk (shared key heads, or states cut in slices; those
// have parts of the gates' gradients too), then what the form needs.  In chunks (bf16): per chunk and value head the state before it, the gradient of the
// state behind it, U and dX, four bytes an element; at most T/64 + num_seqs chunks per head.
// Token by token: at most T/16 + num_seqs states per value head, and 16 slices of a state for
// each workgroup that runs at once.
struct BwdPlan {
    uint64_t parts = 0, off_k = 0, off_g = 0, off_e = 0, off_a = 0, off_b = 0, off_c = 0, off_d = 0, total = 0;
    int slots = 0, slices = 1;
};
BwdPlan plan_backward(const kda::GdnDims& d, const int32_t* cu, int32_t n) {
    BwdPlan p;
    const uint64_t T = (uint64_t)cu[n], hv = (uint64_t)d.hv, state = 4ull * d.dk * d.dv;
    const int cus = kda::device_cu_count();
    if (d.dtype == KDA_DTYPE_F32) p.slices = kda::gdn_backward_seq_slices(d.dv, (int64_t)n * d.hv, cus);
    if (d.hv != d.hk || p.slices > 1) p.parts = align256(T * hv * p.slices * d.dk * 4);
    const uint64_t gates = p.slices > 1 ? align256(T * hv * p.slices * 4) : 0;
    p.off_k = p.parts;
    p.off_g = 2 * p.parts;
    p.off_e = p.off_g + gates;
    p.off_a = p.off_e + gates;
    if (d.dtype == KDA_DTYPE_BF16) {
        const uint64_t chunks = (T / 64 + n) * hv, rows = 4ull * 64 * d.dv;
        p.off_b = p.off_a + align256(chunks * state);
        p.off_c = p.off_b + align256(chunks * state);
        p.off_d = p.off_c + align256(chunks * rows);
        p.total = p.off_d + align256(chunks * rows);
        return p;
    }
    p.slots = (int)std::min<int64_t>((int64_t)std::min(n, kda::kGdnSeqs) * d.hv * p.slices, 2 * cus);
    p.off_b = p.off_a + align256((T / 16 + n) * hv * state);
    p.total = p.off_b + (uint64_t)p.slots * 16 * (state / p.slices);
    return p;
}

}  // namespace

extern "C" {

int64_t kda_gdn_prefill_backward_workspace(const kda_gdn_params* params, const int32_t* cu_seqlens_host,
                                           int32_t num_seqs) {
    kda::GdnDims d;
    if (check_gdn(params, d) != KDA_OK || check_cu(cu_seqlens_host, num_seqs) != KDA_OK) return -1;
    kda::ok();
    return (int64_t)plan_backward(d, cu_seqlens_host, num_seqs).total;
}

kda_status kda_gdn_prefill_backward(const kda_gdn_params* params, const void* q, const void* k,
                                    const void* v, const float* log_alpha, const float* beta,
                                    const int32_t* cu_seqlens_host, int32_t num_seqs,
                                    const float* initial_state, const void* d_out,
                                    const float* d_final_state, void* dq, void* dk, void* dv,
                                    float* dlog_alpha, float* dbeta, float* d_initial_state,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
    return guarded("kda_gdn_prefill_backward", [&]() -> kda_status {
        kda::GdnBackwardArgs a = {};
        kda_status st = check_gdn(params, a.d);
        if (st != KDA_OK) return st;
        if ((st = check_cu(cu_seqlens_host, num_seqs)) != KDA_OK) return st;
        const kda::GdnDims& d = a.d;
        const int64_t T = cu_seqlens_host[num_seqs];
        const size_t es = element(d);
        Range tok[5];
        if ((st = check_tokens(d, T, q, k, v, log_alpha, beta, tok)) != KDA_OK) return st;
        if (T > 0) {
            const void* p[] = {d_out, dq, dk, dv};
            const char* names[] = {"d_out", "dq", "dk", "dv"};
            for (int i = 0; i < 4; ++i)
                if ((st = check_ptr(names[i], p[i], 16)) != KDA_OK) return st;
            if ((st = check_ptr("dlog_alpha", dlog_alpha, 4)) != KDA_OK) return st;
            if ((st = check_ptr("dbeta", dbeta, 4)) != KDA_OK) return st;
        }
        if (initial_state && (st = check_ptr("initial_state", initial_state, 16)) != KDA_OK) return st;
        if (d_final_state && (st = check_ptr("d_final_state", d_final_state, 16)) != KDA_OK) return st;
        if (d_initial_state && (st = check_ptr("d_initial_state", d_initial_state, 16)) != KDA_OK) return st;
        if ((st = check_ptr("workspace", workspace, 256)) != KDA_OK) return st;
        const BwdPlan plan = plan_backward(d, cu_seqlens_host, num_seqs);
        if (workspace_bytes < (int64_t)plan.total)
            return fail(KDA_ERR_INVALID_ARGUMENT, "workspace_bytes %lld < %llu needed", (long long)workspace_bytes,
                        (unsigned long long)plan.total);
        const uint64_t nk = (uint64_t)T * d.hk * d.dk * es, nv = (uint64_t)T * d.hv * d.dv * es, ng = (uint64_t)T * d.hv * 4;
        const uint64_t ns = (uint64_t)num_seqs * d.hv * d.dk * d.dv * 4;
        const Range ins[] = {tok[0], tok[1], tok[2], tok[3], tok[4], range("d_out", d_out, nv),
                             range("initial_state", initial_state, ns), range("d_final_state", d_final_state, ns)};
        const Range outs[] = {range("dq", dq, nk), range("dk", dk, nk), range("dv", dv, nv),
                              range("dlog_alpha", dlog_alpha, ng), range("dbeta", dbeta, ng),
                              range("d_initial_state", d_initial_state, ns), range("workspace", workspace, plan.total)};
        for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
            for (const Range& r : ins)
                if (overlaps(outs[i], r)) return fail(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, r.name);
            for (size_t j = 0; j < i; ++j)
                if (overlaps(outs[i], outs[j]))
                    return fail(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, outs[j].name);
        }
        if ((st = check_pairs(d, num_seqs)) != KDA_OK) return st;
        if ((st = check_grid(T * d.hk * (d.dk / 4) / 256 + 1, 256)) != KDA_OK) return st;
        if ((st = check_grid((T / 64 + 1) * d.hv, 256)) != KDA_OK) return st;
        a.T = T; a.q = q; a.k = k; a.v = v; a.d_out = d_out; a.log_alpha = log_alpha; a.beta = beta;
        a.initial_state = initial_state; a.d_final_state = d_final_state; a.dq = dq; a.dk = dk; a.dv = dv;
        a.dlog_alpha = dlog_alpha; a.dbeta = dbeta; a.d_initial_state = d_initial_state;
        char* ws = static_cast<char*>(workspace);
        a.parts = plan.parts > 0;
        a.dq_parts = reinterpret_cast<float*>(ws);
        a.dk_parts = reinterpret_cast<float*>(ws + plan.off_k);
        a.dg_parts = reinterpret_cast<float*>(ws + plan.off_g);
        a.db_parts = reinterpret_cast<float*>(ws + plan.off_e);
        a.slices = plan.slices;
        const bool chunked = d.dtype == KDA_DTYPE_BF16;
        if (chunked) {
            a.states = ws + plan.off_a; a.sgrads = ws + plan.off_b; a.u = ws + plan.off_c; a.dx = ws + plan.off_d;
            a.cus = kda::device_cu_count();
        } else {
            a.checkpoints = reinterpret_cast<float*>(ws + plan.off_a);
            a.scratch = reinterpret_cast<float*>(ws + plan.off_b);
            a.slots = plan.slots;
        }
        const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
        const std::vector<int32_t> order = longest_first(cu_seqlens_host, num_seqs);
        kda::GdnTable tab;
        hipError_t e = hipSuccess;
        for (int32_t from = 0; from < num_seqs && e == hipSuccess; from += a.num_seqs) {
            a.num_seqs = fill_table(tab, cu_seqlens_host, order, from);
            e = chunked ? kda::launch_gdn_backward_chunked(a, tab, hs) : kda::launch_gdn_backward_seq(a, tab, hs);
        }
        if (e == hipSuccess && a.parts) e = kda::launch_gdn_sum_parts(a, hs);
        if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_gdn_prefill_backward launch: %s", hipGetErrorString(e));
        return kda::ok();
    });
}

kda_status kda_gdn_chunk_prefill(const kda_gdn_params* params, const void* q, const void* k,
                                 const void* v, const float* log_alpha, const float* beta,
                                 const int32_t* cu_seqlens_host, int32_t num_seqs,
                                 const float* initial_state, float* final_state, void* out,
                                 void* stream) {
    return guarded("kda_gdn_chunk_prefill", [&]() -> kda_status {
        kda::GdnPrefillArgs a = {};
        kda_status st = check_gdn(params, a.d);
        if (st != KDA_OK) return st;
        if ((st = check_cu(cu_seqlens_host, num_seqs)) != KDA_OK) return st;
        const kda::GdnDims& d = a.d;
        const int64_t T = cu_seqlens_host[num_seqs];
        Range in[5];
        if ((st = check_tokens(d, T, q, k, v, log_alpha, beta, in)) != KDA_OK) return st;
        if (T > 0 && (st = check_ptr("out", out, 16)) != KDA_OK) return st;
        if (initial_state && (st = check_ptr("initial_state", initial_state, 16)) != KDA_OK) return st;
        if (final_state && (st = check_ptr("final_state", final_state, 16)) != KDA_OK) return st;
        const uint64_t ns = (uint64_t)num_seqs * d.hv * d.dk * d.dv * 4;
        const Range ro = range("out", out, (uint64_t)T * d.hv * d.dv * element(d));
        const Range r0 = range("initial_state", initial_state, ns), rf = range("final_state", final_state, ns);
        for (const Range& r : in) {
            if (overlaps(ro, r)) return fail(KDA_ERR_INVALID_ARGUMENT, "out overlaps %s", r.name);
            if (overlaps(rf, r)) return fail(KDA_ERR_INVALID_ARGUMENT, "final_state overlaps %s", r.name);
        }
        if (overlaps(ro, r0)) return fail(KDA_ERR_INVALID_ARGUMENT, "out overlaps initial_state");
        if (overlaps(ro, rf)) return fail(KDA_ERR_INVALID_ARGUMENT, "final_state overlaps out");
        if (overlaps(r0, rf) && r0.lo != rf.lo)
            return fail(KDA_ERR_INVALID_ARGUMENT, "final_state overlaps initial_state");
        const int cus = kda::device_cu_count();
        const int64_t pairs = (int64_t)num_seqs * d.hv;
        if ((st = check_pairs(d, num_seqs)) != KDA_OK) return st;
        a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta;
        a.initial_state = initial_state; a.final_state = final_state; a.out = out;
        const bool chunked = d.dtype == KDA_DTYPE_BF16;
        a.nv = chunked ? kda::gdn_prefill_nv(d.dv, pairs, cus) : kda::gdn_sequential_nv(d.dv, pairs, cus);
        const std::vector<int32_t> order = longest_first(cu_seqlens_host, num_seqs);
        kda::GdnTable tab;
        for (int32_t from = 0; from < num_seqs; from += a.num_seqs) {
            a.num_seqs = fill_table(tab, cu_seqlens_host, order, from);
            const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
            const hipError_t e = chunked ? kda::launch_gdn_chunked(a, tab, hs) : kda::launch_gdn_sequential(a, tab, hs);
            if (e != hipSuccess)
                return fail(KDA_ERR_HIP, "kda_gdn_chunk_prefill launch: %s", hipGetErrorString(e));
        }
        return kda::ok();
    });
}

kda_status kda_gdn_recurrent(const kda_gdn_params* params, const void* q, const void* k,
                             const void* v, const float* log_alpha, const float* beta,
                             int32_t num_seqs, int32_t num_tokens, const int32_t* steps,
                             const int32_t* state_indices, int32_t num_slots, float* state,
                             int32_t update_state, void* out, void* stream) {
    kda::GdnRecurrentArgs a = {};
    kda_status st = check_gdn(params, a.d);
    if (st != KDA_OK) return st;
    const kda::GdnDims& d = a.d;
    if (num_seqs < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 0", num_seqs);
    if (num_tokens < 1 || num_tokens > kda::kGdnMaxTokens)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_tokens %d outside [1, %d]", num_tokens, kda::kGdnMaxTokens);
    if (num_slots < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_slots %d < 0", num_slots);
    if (!state_indices && num_slots < num_seqs)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_slots %d < num_seqs %d without state_indices", num_slots, num_seqs);
    if (!out && !update_state) return fail(KDA_ERR_INVALID_ARGUMENT, "out is NULL and update_state is 0");
    if (steps && !update_state) return fail(KDA_ERR_INVALID_ARGUMENT, "steps given but update_state is 0");
    if (num_seqs == 0) return kda::ok();
    const int64_t T = (int64_t)num_seqs * num_tokens;
    Range in[7];
    {
        Range tok[5];
        if ((st = check_tokens(d, T, q, k, v, log_alpha, beta, tok)) != KDA_OK) return st;
        std::copy(tok, tok + 5, in);
    }
    if (num_slots > 0 && (st = check_ptr("state", state, 16)) != KDA_OK) return st;
    if (out && (st = check_ptr("out", out, 16)) != KDA_OK) return st;
    if (steps && (st = check_ptr("steps", steps, 4)) != KDA_OK) return st;
    if (state_indices && (st = check_ptr("state_indices", state_indices, 4)) != KDA_OK) return st;
    in[5] = range("steps", steps, (uint64_t)num_seqs * 4);
    in[6] = range("state_indices", state_indices, (uint64_t)num_seqs * 4);
    const Range rs = range("state", state, (uint64_t)num_slots * d.hv * d.dk * d.dv * 4);
    const Range ro = range("out", out, (uint64_t)T * d.hv * d.dv * element(d));
    if (overlaps(ro, rs)) return fail(KDA_ERR_INVALID_ARGUMENT, "out overlaps state");
    for (const Range& r : in) {
        if (overlaps(ro, r)) return fail(KDA_ERR_INVALID_ARGUMENT, "out overlaps %s", r.name);
        if (update_state && overlaps(rs, r)) return fail(KDA_ERR_INVALID_ARGUMENT, "state overlaps %s", r.name);
    }
    if ((st = check_grid((int64_t)num_seqs * d.hv * (d.dv / 32), 256)) != KDA_OK) return st;
    a.num_seqs = num_seqs; a.num_tokens = num_tokens; a.num_slots = num_slots;
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.steps = steps;
    a.state_indices = state_indices; a.state = state; a.update = update_state != 0; a.out = out;
    a.nv = kda::gdn_recurrent_nv(d.dv, (int64_t)num_seqs * d.hv, num_tokens, kda::device_cu_count());
    const hipError_t e = kda::launch_gdn_recurrent(a, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_gdn_recurrent launch: %s", hipGetErrorString(e));
    return kda::ok();
}

int64_t kda_spec_accept_workspace(int32_t num_seqs, int64_t vocab) {
    if (num_seqs < 0 || vocab < 1) {
        fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 0 or vocab %lld < 1", num_seqs, (long long)vocab);
        return -1;
    }
    kda::ok();
    return (int64_t)num_seqs * kda::accept_pieces(num_seqs, vocab, kda::device_cu_count()) * 16;
}

kda_status kda_spec_accept(int32_t dtype, int32_t num_seqs, int32_t num_draft, int64_t vocab,
                           const void* target_probs, const void* draft_probs,
                           const int32_t* draft_tokens, const float* uniforms,
                           const int32_t* num_drafts, int32_t* accepted, int32_t* tokens,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    kda_status st;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32)
        return fail(KDA_ERR_INVALID_ARGUMENT, "dtype %d is not KDA_DTYPE_BF16 or KDA_DTYPE_F32", dtype);
    if (num_seqs < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 0", num_seqs);
    if (num_draft < 0 || num_draft > 64)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_draft %d outside [0, 64]", num_draft);
    if (vocab < 1 || vocab > INT32_MAX)
        return fail(KDA_ERR_INVALID_ARGUMENT, "vocab %lld outside [1, 2^31 - 1]", (long long)vocab);
    if (num_seqs == 0) return kda::ok();
    const size_t es = dtype == KDA_DTYPE_BF16 ? 2 : 4;
    if ((st = check_ptr("target_probs", target_probs, es)) != KDA_OK) return st;
    if (draft_probs && (st = check_ptr("draft_probs", draft_probs, es)) != KDA_OK) return st;
    if (num_draft > 0 && (st = check_ptr("draft_tokens", draft_tokens, 4)) != KDA_OK) return st;
    if ((st = check_ptr("uniforms", uniforms, 4)) != KDA_OK) return st;
    if (num_drafts && (st = check_ptr("num_drafts", num_drafts, 4)) != KDA_OK) return st;
    if ((st = check_ptr("accepted", accepted, 4)) != KDA_OK) return st;
    if ((st = check_ptr("tokens", tokens, 4)) != KDA_OK) return st;
    if ((st = check_ptr("workspace", workspace, 16)) != KDA_OK) return st;
    const int64_t need = kda_spec_accept_workspace(num_seqs, vocab);
    if (workspace_bytes < need)
        return fail(KDA_ERR_INVALID_ARGUMENT, "workspace_bytes %lld < %lld needed", (long long)workspace_bytes,
                    (long long)need);
    const uint64_t n = (uint64_t)num_seqs, k = (uint64_t)num_draft;
    const Range ins[] = {range("target_probs", target_probs, n * (k + 1) * vocab * es),
                         range("draft_probs", draft_probs, n * k * vocab * es),
                         range("draft_tokens", draft_tokens, n * k * 4), range("uniforms", uniforms, n * (k + 1) * 4),
                         range("num_drafts", num_drafts, n * 4)};
    const Range outs[] = {range("accepted", accepted, n * 4), range("tokens", tokens, n * (k + 1) * 4),
                          range("workspace", workspace, (uint64_t)need)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : ins)
            if (overlaps(outs[i], r)) return fail(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, r.name);
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j]))
                return fail(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    kda::AcceptArgs a = {};
    a.dtype = dtype; a.num_seqs = num_seqs; a.num_draft = num_draft; a.vocab = vocab;
    a.p = target_probs; a.q = draft_probs; a.tokens = draft_tokens; a.uniforms = uniforms;
    a.num_drafts = num_drafts; a.accepted = accepted; a.out = tokens;
    a.partial = static_cast<double*>(workspace);
    a.pieces = kda::accept_pieces(num_seqs, vocab, kda::device_cu_count());
    a.piece = (vocab + a.pieces - 1) / a.pieces;
    if ((st = check_grid((int64_t)num_seqs * a.pieces, 256)) != KDA_OK) return st;
    if ((st = check_grid(num_seqs, 1024)) != KDA_OK) return st;
    const hipError_t e = kda::launch_accept(a, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "kda_spec_accept launch: %s", hipGetErrorString(e));
    return kda::ok();
}

}  // extern "C"
