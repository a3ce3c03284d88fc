// Which split of the fp32 prefill of the gated delta rule runs (gdr_scan.cu): host only, no CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace wkv7 {

// 8 columns a warp with feeding warps, 16 with them, 16 without.
enum GdrSplit { kGdrNarrow, kGdrWide, kGdrShared };

// A warp of 8 columns takes 0.72 of the time per token of one of 16, but a head then
// has twice the CTAs; with feeders a CTA takes an SM's registers, and without them several
// share one, which costs each less than waiting its turn.  In units of a token of 16 columns with
// feeders (0.17 us at N = 64, 0.24 at 128), the time until the busiest of 152 SMs is done.
// Measured, in us (8 columns, 16 with feeders, 16 without), 1000 tokens a sequence:
//   40 heads of 64,  1 sequence 121 172 191   2 sequences 233 171 189   4 sequences 343 332 283   16 sequences 1019 821 644
//   32 heads of 128, 1 sequence 182 244 264   2 sequences 356 245 264   4 sequences 704 476 437   16 sequences 2448 1650 1456
// and 500, 1000 and 37 tokens with 40 heads of 64: 124 173 192.
inline GdrSplit gdr_choose_split(int num_seqs, int T_total, int Hv, int N, const int32_t *cu_host) {
    constexpr int kSms = 152, kSorted = 32;
    if (static_cast<long long>(num_seqs) * Hv * (N / 32) > (1 << 24)) return kGdrShared;  // far from the grid's limit
    double lens[kSorted], total = T_total, longest = total / num_seqs;  // lens: longest first
    const int n = num_seqs <= kSorted ? num_seqs : 0;
    for (int i = 0; i < num_seqs; ++i) {
        const double len = cu_host ? cu_host[i + 1] - cu_host[i] : total / num_seqs;
        longest = std::max(longest, len);
        if (n == 0) {
            if (!cu_host) break;
            continue;
        }
        int at = i;
        for (; at > 0 && lens[at - 1] < len; --at) lens[at] = lens[at - 1];
        lens[at] = len;
    }
    // With so many CTAs of each sequence, an SM that takes CTA turn * 152 takes turn + 1 of them no shorter
    // than it; no SM can be done before the longest.  The last turn of each sequence is the one that counts.
    auto busiest = [&](long long ctas) {
        double most = std::max(longest, total * ctas / kSms);
        for (int i = 0; i < n; ++i) {
            const long long turn = ((i + 1) * ctas - 1) / kSms;
            if (turn > 0) most = std::max(most, (turn + 1) * lens[turn * kSms / ctas]);
        }
        return most;
    };
    const double wide = busiest(static_cast<long long>(Hv) * (N / 64)), narrow = 0.72 * busiest(static_cast<long long>(Hv) * (N / 32));
    const double shared = 0.3 * longest + 0.75 * wide;
    return narrow <= std::min(wide, shared) ? kGdrNarrow : wide <= shared ? kGdrWide : kGdrShared;
}

}  // namespace wkv7
