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
// The same for a call that stores the new tokens: those at positions behind the sequence's
// pages are left out (`over` of them), so that the others keep theirs.  Reading alone, as above,
// takes such a sequence as one that ends with its pages.
KV_HD KvSeq kv_seq_stored(const KvBatch& bt, int b, int page, int& over) {
    KvSeq s = kv_seq(bt, b, page);
    over = kv_min(kv_max(bt.lengths[b], 0) - s.len, s.n);
    s.n -= over;
    return s;
}

// Pages that hold a sequence's new tokens (those at positions 0 and up): the
// first of them and how many.
KV_HD int kv_first_page(const KvSeq& s, int page) { return kv_max(s.len - s.n, 0) / page; }
KV_HD int kv_run_pages(const KvSeq& s, int page) {
    return s.n == 0 || s.len == 0 ? 0 : (s.len - 1) / page - kv_first_page(s, page) + 1;
}
// Such a run has a slot: with few tokens a sequence its first token's, else sequence b's runs
// have those from q_start[b] / page + 2 b on (n tokens touch at most n / page + 2 pages, so
// that the next sequence's begin behind them).
KV_HD bool kv_slot_by_token(int64_t B, int64_t T, int64_t page) { return T <= T / page + 2 * B; }
KV_HD int64_t kv_slots(int64_t B, int64_t T, int64_t page) {
    return kv_slot_by_token(B, T, page) ? T : T / page + 2 * B;
}
// The first slot of sequence b: the sequence of a slot is the last one that begins at it or before.
KV_HD int kv_first_slot(const KvBatch& bt, int b, int page, bool by_token) {
    const int q0 = kv_clamp(bt.q_start[b], 0, bt.T);
    return by_token ? q0 : q0 / page + 2 * b;
}
// The page, counted in the sequence, of its i-th slot; -1: none.
KV_HD int kv_slot_page(const KvSeq& s, int i, int page, bool by_token) {
    if (!by_token) return i >= 0 && i < kv_run_pages(s, page) ? kv_first_page(s, page) + i : -1;
    const int p = s.len - s.n + i;
    return i >= 0 && i < s.n && p >= 0 && (i == 0 || p % page == 0) ? p / page : -1;
}

// Attention.  The rows of a sequence and key head are its new tokens times the
// `group` query heads that share the key head, row = token * group + head; a row
// tile is `rows` of them.  A unit is `tokens` keys against one row tile.  Row tile
// rt of the sequence sees the units [first, first + count): at least one, which
// may hold no key that it sees.
// In the deal a row tile counts `extra` units more than it has, before its first: what
// it costs to begin and end one.
struct KvShape {
    int group, rows, tokens, window, page, extra;
};
KV_HD int kv_row_tiles(const KvSeq& s, const KvShape& sh) { return (s.n * sh.group + sh.rows - 1) / sh.rows; }
KV_HD void kv_units(const KvSeq& s, const KvShape& sh, int rt, int& first, int& count) {
    const int c = s.len - s.n, r0 = rt * sh.rows, r1 = kv_min(r0 + sh.rows, s.n * sh.group) - 1;
    const int p0 = c + r0 / sh.group, p1 = c + r1 / sh.group;
    first = sh.window > 0 && p0 >= sh.window ? (p0 - sh.window + 1) / sh.tokens : 0;
    count = p1 < 0 ? 1 : p1 / sh.tokens + 1 - first;
}
// The first key that a row of the row tile sees.  What lies before it may be anything: a serving
// loop takes back pages that nobody sees any more.
KV_HD int kv_first_key(const KvSeq& s, const KvShape& sh, int rt) {
    return sh.window > 0 ? kv_max(s.len - s.n + rt * sh.rows / sh.group - sh.window + 1, 0) : 0;
}

// sum of floor((a i + b) / m) over 0 <= i < n, for a, b >= 0 and m > 0: the points of the
// lattice under a line.  Whole parts of the slope and of b are counted at once; what
// is left is counted along the other axis, where the slope is m / a.
KV_HD int64_t kv_floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (n > 0) {
        sum += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
        a %= m;
        b %= m;
        const int64_t top = a * n + b;  // m times the height at i = n
        if (top < m) break;
        n = top / m;
        b = top % m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}
// Units of a sequence's row tiles before rt as they count, for one key head, 0 <= rt <= its row tiles.
// The last row of a tile but the last is at position c + floor(((rt + 1) rows - 1) / group),
// so that its last unit is the floor of a linear function of rt, as is the first.
KV_HD int64_t kv_units_before(const KvSeq& s, const KvShape& sh, int rt) {
    const int64_t c = s.len - s.n, g = sh.group, R = sh.rows, m = g * sh.tokens;
    int64_t sum = (int64_t)rt * sh.extra;
    int whole = rt;
    if (rt > 0 && rt == kv_row_tiles(s, sh)) {
        int first, count;
        kv_units(s, sh, --whole, first, count);
        sum += count;
    }
    sum += whole;  // one unit each, and those before the last
    int64_t i0 = c < 0 ? -c * g / R : 0;  // the row tiles before see no key
    if (i0 < whole) sum += kv_floor_sum(whole - i0, m, R, c * g + (i0 + 1) * R - 1);
    if (sh.window > 0) {
        const int64_t past = (sh.window - c) * g;  // rows from which on the window cuts
        i0 = past > 0 ? (past + R - 1) / R : 0;
        if (i0 < whole) sum -= kv_floor_sum(whole - i0, m, R, i0 * R + (c - sh.window + 1) * g);
    }
    return sum;
}
// Units of a sequence and one key head, as they count.
KV_HD int64_t kv_seq_units(const KvSeq& s, const KvShape& sh) {
    const int tiles = kv_row_tiles(s, sh);
    if (tiles > 1) return kv_units_before(s, sh, tiles);
    int first = 0, count = 0;
    if (tiles == 0) return 0;
    kv_units(s, sh, 0, first, count);
    return count + sh.extra;
}

// The batch's U units, in the order (sequence, key head, row tile, unit), are dealt
// to C CTAs in runs that differ by one at most.
// (In 32 bits where they are enough: a 64-bit division is a chain of a hundred instructions.)
KV_HD int64_t kv_quotient(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
KV_HD int64_t kv_deal(int64_t U, int C, int c) { return kv_quotient(U * c, C); }
KV_HD int kv_owner(int64_t U, int C, int64_t u) { return (int)kv_quotient((u + 1) * C - 1, U); }
KV_HD int kv_ctas(int64_t U, int most, int least_units) {
    const int64_t c = kv_quotient(U + least_units - 1, least_units);
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
// Whether unit `u`, counted within one key head of p's sequence, is of row tile rt; if so, p is there.
KV_HD bool kv_enter_if(KvPlace& p, const KvShape& sh, int rt, int64_t u, int64_t head_base) {
    const int64_t before = kv_units_before(p.s, sh, rt) + sh.extra;  // of the row tile's first unit
    if (u < before - sh.extra) return false;
    p.rt = rt;
    kv_enter(p, sh);
    if (u >= before + (p.end - p.first)) return false;
    p.base = head_base + before;
    p.unit = u < before ? p.first : p.first + (int)(u - before);
    return true;
}
// The next unit; there must be one in the batch.  (Its number is base + unit - first.)
KV_HD void kv_next(KvPlace& p, const KvBatch& bt, const KvShape& sh, int heads) {
    if (++p.unit < p.end) return;
    p.base += p.end - p.first + sh.extra;
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
