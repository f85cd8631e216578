// Drives the host code of gdn_api.cpp through refusals and through calls that pass every
// check, with the launchers replaced: those end in KDA_ERR_HIP, or check what they are given.
#include <cstdio>
#include <vector>

#include "../../include/kda.h"
#include "gdn_launch.h"

static long long g_seqs = 0, g_tokens = 0;
static int g_longest = 1 << 30;

namespace kda {
hipError_t launch_gdn_sequential(const GdnPrefillArgs& a, const GdnTable& t, hipStream_t) {
    for (int i = 0; i < a.num_seqs; ++i) {
        g_seqs += 1;
        g_tokens += t.len[i];
        if (t.len[i] > g_longest) return hipErrorInvalidValue;  // not longest first
        g_longest = t.len[i];
    }
    return hipSuccess;
}
hipError_t launch_gdn_chunked(const GdnPrefillArgs& a, const GdnTable& t, hipStream_t s) {
    return a.d.dv % a.nv ? hipErrorInvalidValue : launch_gdn_sequential(a, t, s);
}
hipError_t launch_gdn_recurrent(const GdnRecurrentArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_gdn_backward_seq(const GdnBackwardArgs& a, const GdnTable& t, hipStream_t) {
    for (int i = 0; i < a.num_seqs; ++i) g_tokens += t.len[i];
    return a.slots > 0 ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_gdn_backward_chunked(const GdnBackwardArgs& a, const GdnTable& t, hipStream_t) {
    for (int i = 0; i < a.num_seqs; ++i) g_tokens += t.len[i];
    return a.cus > 0 ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_gdn_sum_parts(const GdnBackwardArgs& a, hipStream_t) { return a.parts ? hipSuccess : hipErrorInvalidValue; }
hipError_t launch_accept(const AcceptArgs& a, hipStream_t) {
    return a.piece * a.pieces >= a.vocab && a.pieces <= 256 ? hipErrorNotSupported : hipSuccess;
}
}  // namespace kda

static int bad = 0;
static void expect(int got, int want, const char* what) {
    if (got != want) {
        ++bad;
        std::printf("%s: %d, expected %d\n", what, got, want);
    }
}

int main() {
    char* base = reinterpret_cast<char*>(1ull << 32);
    auto at = [&](int i) { return static_cast<void*>(base + ((long long)i << 32)); };
    auto fl = [&](int i) { return static_cast<float*>(at(i)); };
    auto in = [&](int i) { return static_cast<int32_t*>(at(i)); };
    kda_gdn_params p = {KDA_DTYPE_BF16, 2, 4, 128, 64, 1.f, 0, 0, 0};
    for (int n : {1, 255, 256, 257, 700}) {
        std::vector<int32_t> cu(n + 1, 0);
        for (int i = 0; i < n; ++i) cu[i + 1] = cu[i] + (i * 37) % 91;
        g_seqs = g_tokens = 0;
        g_longest = 1 << 30;
        for (int dt : {KDA_DTYPE_BF16, KDA_DTYPE_F32}) {
            p.dtype = dt;
            g_longest = 1 << 30;
            expect(kda_gdn_chunk_prefill(&p, at(1), at(2), at(3), fl(4), fl(5), cu.data(), n, fl(6), fl(6), at(7), nullptr),
                   KDA_OK, "prefill");
        }
        for (int dt : {KDA_DTYPE_BF16, KDA_DTYPE_F32}) {
            p.dtype = dt;
            const long long ws = kda_gdn_prefill_backward_workspace(&p, cu.data(), n);
            const long long before = g_tokens;
            expect(kda_gdn_prefill_backward(&p, at(1), at(2), at(3), fl(4), fl(5), cu.data(), n, nullptr, at(8), nullptr, at(9),
                                            at(10), at(11), fl(12), fl(13), nullptr, (void*)(1ull << 50), ws, nullptr),
                   KDA_OK, "backward");
            expect(g_tokens - before == cu[n], 1, "every token once");
            g_tokens = before;
            expect(kda_gdn_prefill_backward(&p, at(1), at(2), at(3), fl(4), fl(5), cu.data(), n, nullptr, at(8), nullptr, at(9),
                                            at(10), at(11), fl(12), fl(13), nullptr, (void*)(1ull << 50), ws - 1, nullptr),
                   KDA_ERR_INVALID_ARGUMENT, "a byte short");
        }
        expect(g_seqs == 2 * n && g_tokens == 2 * cu[n], 1, "every sequence once");
    }
    int32_t cu1[] = {0, 4};
    p.dtype = KDA_DTYPE_BF16;
    expect(kda_gdn_chunk_prefill(&p, at(1), at(2), at(3), fl(4), fl(5), cu1, 0, nullptr, nullptr, at(7), nullptr),
           KDA_ERR_INVALID_ARGUMENT, "no sequences");
    expect(kda_gdn_recurrent(&p, at(1), at(2), at(3), fl(4), fl(5), 8, 4, in(8), in(9), 20, fl(6), 1, at(7), nullptr),
           KDA_ERR_HIP, "recurrent");
    expect(kda_gdn_recurrent(&p, at(1), at(2), at(3), fl(4), fl(5), 8, 4, nullptr, nullptr, 7, fl(6), 1, at(7), nullptr),
           KDA_ERR_INVALID_ARGUMENT, "too few slots");
    for (long long v : {1ll, 2047ll, 32000ll, 151669ll, 2147483647ll})
        for (int n : {1, 3, 300}) {
            const long long ws = kda_spec_accept_workspace(n, v);
            expect(kda_spec_accept(KDA_DTYPE_F32, n, n == 300 ? 0 : 4, v, (void*)(1ull << 52), nullptr, in(3), fl(4), nullptr,
                                   in(5), in(6), at(7), ws, nullptr), KDA_ERR_HIP, "accept");
        }
    // groups of a launch: in order, every sequence with tokens once, few workgroups without a chunk
    for (int spread : {1, 7, 900, 100000}) {
        kda::GdnTable t;
        for (int i = 0; i < kda::kGdnSeqs; ++i) t.len[i] = (kda::kGdnSeqs - 10 - i) * spread / 9;
        for (int i = kda::kGdnSeqs - 10; i < kda::kGdnSeqs; ++i) t.len[i] = 0;
        t.len[0] += 50 * spread;
        int from = 0;
        while (from < kda::kGdnSeqs) {
            const int n = kda::gdn_gradient_group(t, from, kda::kGdnSeqs, 4);
            if (n == 0) break;
            long long work = 0;
            for (int i = from; i < from + n; ++i) work += (t.len[i] + 63) / 64 * 4;
            const long long grid = (t.len[from] + 63) / 64 * 4ll * n;
            expect(n > 0 && grid - work <= 32768 + work, 1, "a group's empty workgroups");
            from += n;
        }
        for (int i = from; i < kda::kGdnSeqs; ++i) expect(t.len[i], 0, "no sequence with tokens is left out");
    }
    std::printf("%d unexpected results\n", bad);
    return bad != 0;
}
