// kvslot.h -- where a token of a call lies in a paged cache: the range rules
// that keep every access of the cache kernels in bounds.  Plain C++, so that
// the host tests run the very code the kernels run.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define WLQ_HD __host__ __device__ __forceinline__
#else
#define WLQ_HD inline
#endif

namespace wlq {

enum KvRange : int { KV_OK = 0, KV_NONE = 1, KV_BAD = 2 };

// A sequence's tokens r0 .. r1 of this call (of `tokens` rows), at most max_q
// of them, the last ones of kv_len cached tokens.  KV_BAD: offsets or lengths
// out of range, nothing of the sequence may be read or written.
WLQ_HD KvRange kv_sequence(int64_t r0, int64_t r1, int64_t kv_len, int64_t max_q, int64_t tokens) {
    if (r0 < 0 || r1 < r0 || r1 > tokens || r1 - r0 > max_q || kv_len < r1 - r0) return KV_BAD;
    return r1 > r0 ? KV_OK : KV_NONE;
}

// Table entry and place of cached position `pos` (pages of 2^shift tokens).
WLQ_HD KvRange kv_entry(int64_t pos, int64_t table_width, int shift, int64_t* entry, int* place) {
    *entry = pos >> shift;
    *place = static_cast<int>(pos & ((int64_t(1) << shift) - 1));
    return pos >= 0 && *entry < table_width ? KV_OK : KV_BAD;
}

// How many cached tokens a call looks at: those the table has room for (a
// length beyond it is out of range; nothing is gained by walking it).
WLQ_HD int kv_covered(int64_t kv_len, int64_t table_width, int shift) {
    const int64_t room = table_width >= (int64_t(1) << 31) ? (int64_t(1) << 31) - 1 : table_width << shift;
    const int64_t n = kv_len < room ? kv_len : room;
    return static_cast<int>(n < 0 ? 0 : n);
}

WLQ_HD bool kv_page_ok(int64_t page, int64_t pages) { return page >= 0 && page < pages; }

}  // namespace wlq
