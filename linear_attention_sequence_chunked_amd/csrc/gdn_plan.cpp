// gdn_plan.cpp -- host-side scheduling policy of the gated delta rule and of draft
// verification.  No device code.
#include "gdn_launch.h"

#include <algorithm>

namespace kda {

int gdn_recurrent_nv(int dv, int64_t pairs, int cu_count) {
    // Whole rows of the state per workgroup once the (sequence, head) pairs give every
    // compute unit two of them; 32 columns (128-byte row segments, still whole cache lines)
    // below that, so that a small batch spreads over more compute units.
    return pairs >= 2 * (int64_t)cu_count ? dv : 32;
}

int gdn_prefill_nv(int dv, int64_t pairs, int cu_count) {
    // One workgroup runs per compute unit at a time (its LDS): the columns are split in halves
    // until the (sequence, head) pairs cover every unit once, down to one 16-column block.
    int nv = dv;
    while (nv > 16 && pairs * (dv / nv) < cu_count) nv /= 2;
    return nv;
}

int gdn_backward_nv(int dv, int64_t pairs, int cu_count) {
    // the walks have the narrow form alone
    return pairs * (dv / 32) < cu_count ? 16 : 32;
}

int accept_pieces(int64_t num_seqs, int64_t vocab, int cu_count) {
    // Four workgroups per compute unit over the batch, but no piece below 2048 entries
    // (eight per thread) and at most 256 pieces (one partial sum per thread of the join).
    const int64_t want = (4 * (int64_t)cu_count + num_seqs - 1) / std::max<int64_t>(num_seqs, 1);
    const int64_t most = std::min<int64_t>(256, (vocab + 2047) / 2048);
    return (int)std::max<int64_t>(1, std::min(want, most));
}

}  // namespace kda
