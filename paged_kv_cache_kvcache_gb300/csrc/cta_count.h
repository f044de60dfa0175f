// How many CTAs of a cluster share a (sequence, KV head) in the decodes over a bounded cache (host code, no CUDA).
#pragma once

#include <algorithm>
#include <cstdint>

namespace pa {

constexpr int kMaxClusterCtas = 16;

// CTAs per (sequence, KV head), `units` of them of up to `keys` keys each (whole: contexts of up to keys are seen whole): as
// many as run at once (clusters of a second wave wait for whole ones of the first: 200 sequences of 4 KV heads and 1000 keys
// took 66.8 us with one CTA each, 88.2 with two; 19 of 16384 keys 141 with one, 100 with two).  A cluster stays in one GPC, so
// that fewer fit than there are places (64 clusters of six 6.2 us, of seven, in 456 places, 9.2).
// fit(c, &n): n clusters of c CTAs run at once, 0 if that size does not run at all; returns an error or 0.
template <class Fit>
int count_cluster_ctas(int64_t units, int64_t keys, bool whole, Fit fit, int *ctas)
{
    // No more than four, with 64 keys each (one sequence of 320 keys and 8 KV heads, INT8: 7.0 us with one, 6.0 with two,
    // 5.5 with four to eight), than eight, with 128, or than 16, with 224 (six of 3624 keys 17.1 us with four, 11.4 with
    // eight, 9.5 with 16; ten of 2480 10.5 with eight, 9.5 with twelve, 9.9 with 16).
    const int64_t want = std::max({std::clamp<int64_t>(keys / 64, 1, 4), std::min<int64_t>(8, keys / 128),
                                   std::min<int64_t>(kMaxClusterCtas, keys / 224)});
    int at_once = 0;
    if (int rc = fit(1, &at_once))
        return rc;
    int64_t n = std::clamp<int64_t>(at_once / units, 1, want);
    for (; n > 1; --n) {
        if (int rc = fit((int)n, &at_once))
            return rc;
        if (at_once >= units)
            break;
    }
    // Where contexts are seen whole their lengths differ, and up to eight CTAs of 1024 keys, 1024 CTAs in all, even them
    // out (64 sequences of 4096 to 8192 keys and 4 KV heads: 175 us with one, 153 with four; 18 of up to 13634 and 8: 120
    // with three, 111 with eight; 60 of up to 516 and 8: 12.2 with one, 19.2 with two).
    if (whole)
        for (int64_t more = std::min({(int64_t)8, (1024 + units - 1) / units, keys / 1024}); more > n; --more) {
            if (int rc = fit((int)more, &at_once))
                return rc;
            if (at_once > 0)
                n = more;
        }
    *ctas = (int)n;
    return 0;
}

} // namespace pa
