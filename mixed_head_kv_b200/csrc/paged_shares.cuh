// paged_shares.cuh — into how many shares the paged decode cuts its list of work. Host
// and device code: a host build is checked against the limit.
//
// Equal shares, one per resident CTA, but none so small that the longest pair is cut into
// more than kPartsPerPair parts (and one, as it need not start where a share does): the
// last CTA of a pair to finish reads G x D floats of every part. Captured, one sequence
// of 131072 tokens with one retrieval head for groups of 1, of 4 (seven streaming heads
// beside it) and of 8; then 500000 tokens of the group of 8 and 16384 of the group of 4:
//   96 parts                  23.1, 29.2, 32.3, 71.5, 14.8 us
//   112                       22.0, 26.5, 33.8, 68.9, 14.9
//   all 296 CTAs              20.2, 33.2, 54.6, 90.9
//   48 per pair on average    33.2, 33.5, 37.2, 91.2, 20.6  (streaming pairs counted too)
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define DUO_SHARE_FN __host__ __device__ __forceinline__
#else
#define DUO_SHARE_FN inline
#endif

namespace duo {

constexpr int kPartsPerPair = 112;

// Shares of `total` units, the longest pair having `longest` of them (<= 2^21 + 1).
DUO_SHARE_FN int share_count(int64_t total, int longest, int ctas) {
    if (longest <= kPartsPerPair) return total < ctas ? static_cast<int>(total) : ctas;
    const int least = (longest + kPartsPerPair - 1) / kPartsPerPair;  // units of a share
    if (total >= static_cast<int64_t>(ctas) * least) return ctas;
    return static_cast<int>(static_cast<uint32_t>(total) / static_cast<uint32_t>(least));
}

}  // namespace duo
