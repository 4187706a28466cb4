// kv_plan.h -- the index arithmetic of the paged key/value cache's kernels, for
// the host and the device: what part of a batch a sequence, a row tile and a
// CTA is.  Every number read from the caller's arrays is brought into range
// here, so that no value in them leads outside a buffer.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KV_HD __host__ __device__ __forceinline__
#else
#define KV_HD inline
#endif

namespace moe {

// New tokens of a batch of B sequences: sequence b's are rows q_start[b] ..
// q_start[b + 1] - 1 of q, k and v, the last of its lengths[b] cached tokens.
struct KvBatch {
    const int32_t* q_start;     // [B + 1]
    const int32_t* lengths;     // [B]
    const int32_t* page_table;  // [B][table_stride], max_pages of a row in use
    int64_t table_stride;
    int B, T, max_pages;
};

KV_HD int kv_clamp(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
KV_HD int kv_min(int a, int b) { return a < b ? a : b; }
KV_HD int kv_max(int a, int b) { return a > b ? a : b; }
KV_HD int64_t kv_min64(int64_t a, int64_t b) { return a < b ? a : b; }

struct KvSeq {
    int q0, n, len;  // first row, new tokens, cached tokens (the new ones included)
};
KV_HD KvSeq kv_seq(const KvBatch& bt, int b, int page) {
    KvSeq s;
    s.q0 = kv_clamp(bt.q_start[b], 0, bt.T);
    s.n = kv_clamp(bt.q_start[b + 1], s.q0, bt.T) - s.q0;
    s.len = kv_clamp(bt.lengths[b], 0, bt.max_pages * page);
    return s;
}

// Pages that hold a sequence's new tokens (those at positions 0 and up): the
// first of them and how many.
KV_HD int kv_first_page(const KvSeq& s, int page) { return kv_max(s.len - s.n, 0) / page; }
KV_HD int kv_run_pages(const KvSeq& s, int page) {
    return s.n == 0 || s.len == 0 ? 0 : (s.len - 1) / page - kv_first_page(s, page) + 1;
}
// The most that all sequences together can have (each touches at most n / page + 2).
KV_HD int64_t kv_most_runs(int64_t B, int64_t T, int64_t page) {
    const int64_t by_pages = T / page + 2 * (B < T ? B : T);
    return by_pages < T ? by_pages : T;
}

// Attention.  The rows of a sequence and key head are its new tokens times the
// `group` query heads that share the key head, row = token * group + head; a row
// tile is `rows` of them.  A unit is `tokens` keys against one row tile.  Row tile
// rt of the sequence sees the units [first, first + count): at least one, which
// may hold no key that it sees.
struct KvShape {
    int group, rows, tokens, window, page;
};
KV_HD int kv_row_tiles(const KvSeq& s, const KvShape& sh) { return (int)(((int64_t)s.n * sh.group + sh.rows - 1) / sh.rows); }
KV_HD void kv_units(const KvSeq& s, const KvShape& sh, int rt, int& first, int& count) {
    const int64_t r0 = (int64_t)rt * sh.rows, all = (int64_t)s.n * sh.group;
    const int64_t r1 = (r0 + sh.rows < all ? r0 + sh.rows : all) - 1;
    const int p0 = s.len - s.n + (int)(r0 / sh.group), p1 = s.len - s.n + (int)(r1 / sh.group);
    const int lo = sh.window > 0 && p0 >= sh.window ? p0 - sh.window + 1 : 0;
    first = lo / sh.tokens;
    count = kv_max(p1 < 0 ? 0 : p1 / sh.tokens + 1 - first, 1);
}
// Units of a sequence and one key head.
KV_HD int64_t kv_seq_units(const KvSeq& s, const KvShape& sh) {
    int64_t sum = 0;
    const int tiles = kv_row_tiles(s, sh);
    for (int rt = 0; rt < tiles; ++rt) {
        int first, count;
        kv_units(s, sh, rt, first, count);
        sum += count;
    }
    return sum;
}

// The batch's U units, in the order (sequence, key head, row tile, unit), are dealt
// to C CTAs in runs that differ by one at most.
KV_HD int64_t kv_deal(int64_t U, int C, int c) { return U * c / C; }
KV_HD int kv_owner(int64_t U, int C, int64_t u) { return (int)(((u + 1) * C - 1) / U); }
KV_HD int kv_ctas(int64_t U, int most, int least_units) {
    const int64_t c = (U + least_units - 1) / least_units;
    return (int)(c < 1 ? 1 : c < most ? c : most);
}

// A place in that order.
struct KvPlace {
    int b, head, rt;     // the row tile
    int unit, end;       // the unit, and the end of its row tile's units
    int64_t base;        // number of the row tile's first unit in the whole order
    int first;           // that unit
    KvSeq s;
};
KV_HD void kv_enter(KvPlace& p, const KvShape& sh) {
    int count;
    kv_units(p.s, sh, p.rt, p.first, count);
    p.unit = p.first;
    p.end = p.first + count;
}
// The unit `u` of sequence b, whose first is number `base` (u - base < heads * its units a head).
KV_HD void kv_locate(KvPlace& p, const KvBatch& bt, const KvShape& sh, int b, int64_t base, int64_t u) {
    p.b = b;
    p.s = kv_seq(bt, b, sh.page);
    const int64_t per = kv_seq_units(p.s, sh);
    p.head = (int)((u - base) / per);
    p.base = base + p.head * per;
    p.rt = 0;
    kv_enter(p, sh);
    while (u - p.base >= p.end - p.first) {
        p.base += p.end - p.first;
        ++p.rt;
        kv_enter(p, sh);
    }
    p.unit = p.first + (int)(u - p.base);
}
// The next unit; there must be one.
KV_HD void kv_next(KvPlace& p, const KvBatch& bt, const KvShape& sh, int heads) {
    if (++p.unit < p.end) return;
    p.base += p.end - p.first;
    ++p.rt;
    if (p.rt >= kv_row_tiles(p.s, sh)) {
        p.rt = 0;
        if (++p.head >= heads) {
            p.head = 0;
            do p.s = kv_seq(bt, ++p.b, sh.page);
            while (p.s.n == 0 && p.b + 1 < bt.B);
        }
    }
    kv_enter(p, sh);
}

}  // namespace moe
