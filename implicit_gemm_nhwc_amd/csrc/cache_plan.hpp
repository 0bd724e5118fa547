// Places in the paged cache and the division of its reading among workgroups,
// for host and device (plain C++).
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define IGC_HD __host__ __device__
#else
#define IGC_HD
#endif

namespace igc {

// Page of position p: its entry of the table, -1 where the position lies
// outside the table or the entry outside the pool.
template <typename Row>
IGC_HD inline int cache_page(Row row, int64_t p, int shift, int entries, int pages) {
    if (p < 0 || (p >> shift) >= entries) return -1;
    const int id = row[p >> shift];
    return id >= 0 && id < pages ? id : -1;
}

// Row of the pool (of all pages, heads and tokens) of a token of a page.
IGC_HD inline int64_t cache_row(int id, int heads, int head, int64_t p, int shift) {
    return (((int64_t)id * heads + head) << shift) + (p & (((int64_t)1 << shift) - 1));
}

// Length of a sequence: within 0 and the table's capacity.
IGC_HD inline int cache_len(int len, int64_t capacity) {
    return len < 0 ? 0 : len < capacity ? len : (int)capacity;
}

// Division of the cache's reading.  A (sequence, key head, row tile) is read by
// k_b = max(1, ceil(n_b / c)) workgroups, n_b the sequence's units of
// kCacheUnit keys; each takes c of them.  The lengths are known on the device
// only, so c comes from them there: with `slots` workgroups a (key head, row
// tile) over all sequences, c = ceil(sum n_b / (slots - B)) leaves at most
// `slots` of them, and a few bisections look for a smaller c that does (16
// sequences of up to 4099 tokens with 5 drafts: 21.8 -> 21.2 us).  slots < 2 B:
// one workgroup each.  With slots up to 512, B is at most 256 where there is
// a division, and sum n_b stays below 2^32.
constexpr int kCacheUnit = 128;   // keys: half a round of a workgroup's waves
constexpr int kCacheLeast = 2;     // units a split at least
constexpr int kCacheMostSlots = 512;
constexpr int kCacheBisect = 4;

IGC_HD inline uint32_t cache_units(int len) {
    return ((uint32_t)len + (kCacheUnit - 1)) / kCacheUnit;
}

IGC_HD inline bool cache_splits(int64_t slots, int64_t batch) { return slots >= 2 * batch; }

// c from the sum of the units: enough for any lengths with per = slots - B, and
// too small with per = slots unless it fits.
IGC_HD inline uint32_t cache_chunk(uint32_t total, uint32_t per) {
    const uint32_t c = total / per + (total % per != 0);
    return c < kCacheLeast ? kCacheLeast : c;
}

IGC_HD inline uint32_t cache_parts(int len, uint32_t chunk) {
    const uint32_t n = (cache_units(len) + (chunk - 1)) / chunk;
    return n < 1 ? 1 : n;
}

// Splits of the smallest size that a sequence as long as the table makes.
IGC_HD inline int64_t cache_most(int64_t capacity) {
    const int64_t units = (capacity + kCacheUnit - 1) / kCacheUnit;
    const int64_t most = (units + kCacheLeast - 1) / kCacheLeast;
    return most < 1 ? 1 : most;
}

// Whether there is room for that many of every sequence: then each has its own
// slots, and no division is needed.
IGC_HD inline bool cache_fixed(int64_t slots, int64_t batch, int64_t capacity) {
    const int64_t most = cache_most(capacity);
    return most < slots / batch + 1 && most * batch <= slots;
}

// Workgroups a (key head, row tile) that a launch needs room for.
IGC_HD inline int64_t cache_slots_bound(int64_t slots, int64_t batch, int64_t capacity) {
    if (!cache_splits(slots, batch)) return batch;
    return cache_fixed(slots, batch, capacity) ? cache_most(capacity) * batch : slots;
}

}  // namespace igc
