// gdn_plan.cpp -- host-side scheduling policy of the gated delta rule and of draft
// verification.  No device code.
#include "gdn_launch.h"

#include <algorithm>

namespace kda {

int gdn_recurrent_nv(int dv, int64_t pairs, int tokens, int cu_count) {
    // Below two (sequence, head) pairs per compute unit, 32 columns (128-byte row segments,
    // still whole cache lines) spread a small batch over more units: one token of one sequence
    // with 32 heads takes 4.4 us, 5.9 us with whole rows.  Above, one token takes whole rows of
    // the state per workgroup (256 x 32 states of 128 x 128: 162 us, 209 us in halves), several
    // tokens, which keep the state in registers for long, halves of them (96 x 32 states, 4
    // tokens: 59 us, 67 us with whole rows).
    if (pairs < 2 * (int64_t)cu_count) return 32;
    return tokens == 1 ? dv : 64;
}

int gdn_prefill_nv(int dv, int64_t pairs, int cu_count) {
    // One workgroup runs per compute unit at a time (its LDS): the columns are split in halves
    // until the (sequence, head) pairs cover every unit once, down to one 16-column block.  A
    // narrower slice has a shorter step: 16384 tokens with 8 heads, 128 columns, 442 us at 16
    // columns per workgroup, 472 at 32.  But every slice stages the keys: 23 sequences of up to
    // 4097 tokens, 32 heads of 128 columns: 309 us at 128 columns, 438 at 64, 655 at 32.
    int nv = dv;
    while (nv > 16 && pairs * (dv / nv) < cu_count) nv /= 2;
    return nv;
}

int gdn_sequential_nv(int dv, int64_t pairs, int cu_count) {
    // One column per lane while two workgroups per compute unit hold every state, else two, which
    // share a token's operands.  1024 tokens, states of 128 x 128: 64 of them 226 us at one and 242
    // at two, 128 of them 399 and 358, four 158 and 227.
    return pairs * (dv / 16) <= 2 * cu_count ? 16 : 32;
}

int gdn_backward_seq_slices(int dv, int64_t pairs, int cu_count) {
    // Slices of 32 columns while two workgroups per compute unit hold every state; whole states
    // else, whose sums over rows need no second launch.  512 tokens, states of 128 x 128: 16 of
    // them 1.18 ms in slices and 2.26 whole, 128 of them 1.94 and 2.56, 256 3.73 and 3.39.
    return pairs * (dv / 32) <= 2 * cu_count ? dv / 32 : 1;
}

int gdn_gradient_group(const GdnTable& t, int from, int n, int hv) {
    // A launch's grid is its longest sequence's chunks by its sequences, so shorter ones leave
    // workgroups without a chunk (0.34 ns each).  A group ends where those would cost as much as a
    // further launch with its tail (13 us: 32768 of them), or half a percent of its work if that is
    // more.  One sequence of 16384 tokens with 255 of 64, 16 heads: 2.12 ms, 2.47 in one launch;
    // 64 sequences of 64, 128, .. 4096 tokens, 8 heads: 2.81 ms in one launch, 2.92 in eight.
    const int64_t longest = (t.len[from] + 63) / 64;
    int64_t work = 0, empty = 0;
    int i = from;
    for (; i < n; ++i) {
        const int64_t chunks = (t.len[i] + 63) / 64;
        if (chunks == 0) break;  // (the rest are empty too)
        work += chunks * hv;
        empty += (longest - chunks) * hv;
        if (empty > 32768 + work) break;
    }
    return i - from;
}

bool accept_in_one(int64_t vocab) {
    // One workgroup per sequence, one launch, against the vocabulary in pieces and a second launch
    // (fp32, replayed from a graph): 32000 entries, 1 / 128 / 512 sequences 8.8 / 10.2 / 27 us and
    // 8.2 / 13.7 / 31; 500 entries, one sequence 3.5 and 6.5; called from the host one by one 10.0
    // and 12.0.  At least the eight entries of a bf16 load.
    return vocab >= 8 && vocab <= kAcceptOne;
}

int accept_pieces(int64_t num_seqs, int64_t vocab, int cu_count) {
    // Pieces of about 4096 entries, which is what the join scans in one go; shorter ones (2048
    // at the least, eight entries per thread) while the batch gives the card too few
    // workgroups; at most 256 (one partial sum per thread of the join).
    const int64_t fill = (4 * (int64_t)cu_count + num_seqs - 1) / std::max<int64_t>(num_seqs, 1);
    const int64_t want = std::max((vocab + 4095) / 4096, std::min(fill, (vocab + 2047) / 2048));
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, 256));
}

}  // namespace kda
