// Ranges of split launches, for host and device (plain C++).
#pragma once

namespace igc {

// End of the split of `split` elements that starts at `begin`, of `end` in
// all; at or below `begin` where nothing is left.  The sum is formed only
// where it stays below `end`: whole splits may pass 2^31 together (2^31 - 5000
// keys as 1024 splits of 2^21), and a wrapped end would drop the last one.
constexpr int split_end(int begin, int split, int end) {
    return begin < end && split < end - begin ? begin + split : end;
}

}  // namespace igc
