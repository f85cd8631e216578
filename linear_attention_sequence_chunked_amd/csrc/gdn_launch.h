// gdn_launch.h -- host-side launch descriptors of the gated delta rule and of draft
// verification, shared by the C ABI (gdn_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Shapes every gated-delta-rule kernel takes.  Strides are elements between tokens.
struct GdnDims {
    int dtype, hk, hv, dk, dv;
    float scale;
    int64_t qs, ks, vs;
};

// One launch covers at most this many sequences (their tables travel in the kernel
// arguments, so a call needs no device copy of cu_seqlens); larger batches take several.
constexpr int kGdnSeqs = 256;

struct GdnTable {
    int32_t start[kGdnSeqs];  // first packed token row
    int32_t len[kGdnSeqs];
    int32_t id[kGdnSeqs];     // sequence number (its state's place)
};

struct GdnPrefillArgs {
    GdnDims d;
    int num_seqs;  // entries of the table in use
    const void *q, *k, *v;
    const float *log_alpha, *beta;
    const float* initial_state;  // may be null
    float* final_state;          // may be null
    void* out;
    int nv;                      // value columns per workgroup
};

constexpr int kGdnMaxTokens = 16;  // tokens per sequence of the recurrent form

struct GdnRecurrentArgs {
    GdnDims d;
    int num_seqs, num_tokens, num_slots;
    const void *q, *k, *v;
    const float *log_alpha, *beta;
    const int32_t* steps;          // device [num_seqs] or null
    const int32_t* state_indices;  // device [num_seqs] or null
    float* state;
    bool update;
    void* out;                     // may be null
    int nv;
};

struct GdnBackwardArgs {
    GdnDims d;
    int num_seqs;
    int64_t T;                    // packed tokens
    const void *q, *k, *v, *d_out;
    const float *log_alpha, *beta;
    const float *initial_state, *d_final_state;  // may be null
    void *dq, *dk, *dv;
    float *dlog_alpha, *dbeta;
    float* d_initial_state;       // may be null
    bool parts;                   // dq and dk of each value head (and slice) apart first
    int slices;                   // of a state's columns, over workgroups (token by token; else 1)
    float *dq_parts, *dk_parts;   // [T, hv, slices, dk]
    float *dg_parts, *db_parts;   // [T, hv, slices], several slices alone
    // token by token: states before every 16th token, and a scratch of 16 slices per workgroup
    float *checkpoints, *scratch;
    int slots;                    // workgroups the scratch serves
    // in chunks: per (chunk, value head) the states, their gradients, U and dX (gdn_chunk.h)
    void *states, *sgrads, *u, *dx;
    int cus;  // compute units of the device
};

struct AcceptArgs {
    int dtype, num_seqs, num_draft;
    int64_t vocab;
    const void *p, *q;             // q may be null (drafts without probabilities)
    const int32_t* tokens;
    const float* uniforms;
    const int32_t* num_drafts;     // may be null
    int32_t *accepted, *out;
    double* partial;               // [num_seqs][pieces][2]
    int pieces;
    int64_t piece;                 // vocabulary entries per piece
};

// value columns per workgroup of the token-by-token kernel (gdn_plan.cpp)
int gdn_recurrent_nv(int dv, int64_t pairs, int tokens, int cu_count);
// value columns per workgroup of the chunked prefill (gdn_plan.cpp)
int gdn_prefill_nv(int dv, int64_t pairs, int cu_count);
// value columns per workgroup of the prefill of 32-bit inputs (gdn_plan.cpp)
int gdn_sequential_nv(int dv, int64_t pairs, int cu_count);
// slices of a state's columns in the token-by-token gradients (gdn_plan.cpp)
int gdn_backward_seq_slices(int dv, int64_t pairs, int cu_count);
// sequences from place `from` of a table (longest first) on that share a launch of the chunks'
// gradients; 0: none of them has a token (gdn_plan.cpp)
int gdn_gradient_group(const GdnTable& t, int from, int n, int hv);
// vocabulary that one workgroup holds in registers, and whether this one does (gdn_plan.cpp)
constexpr int64_t kAcceptOne = 32768;
bool accept_in_one(int64_t vocab);
// pieces the vocabulary of one sequence is cut into (gdn_plan.cpp)
int accept_pieces(int64_t num_seqs, int64_t vocab, int cu_count);

hipError_t launch_gdn_recurrent(const GdnRecurrentArgs& a, hipStream_t stream);
hipError_t launch_gdn_sequential(const GdnPrefillArgs& a, const GdnTable& t, hipStream_t stream);
hipError_t launch_gdn_chunked(const GdnPrefillArgs& a, const GdnTable& t, hipStream_t stream);
hipError_t launch_gdn_backward_seq(const GdnBackwardArgs& a, const GdnTable& t, hipStream_t stream);
hipError_t launch_gdn_backward_chunked(const GdnBackwardArgs& a, const GdnTable& t, hipStream_t stream);
hipError_t launch_gdn_sum_parts(const GdnBackwardArgs& a, hipStream_t stream);
hipError_t launch_accept(const AcceptArgs& a, hipStream_t stream);

}  // namespace kda
