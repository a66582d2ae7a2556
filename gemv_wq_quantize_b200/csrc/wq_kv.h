// wq_kv.h -- index arithmetic of the paged 8-bit key / value cache (kv_append, kv_attention):
// the clamped span of a sequence, the pages an append touches and the offsets of codes and
// scales.  Plain integer functions without CUDA types, so that the same text is checked on
// the CPU over every small case (tests/test_kv_host.py).
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define WQ_HD __host__ __device__ __forceinline__
#else
#define WQ_HD inline
#endif

namespace wq {

constexpr int kKvMaxSeqs = 4096;       // sequences of one call (their unit counts are summed in shared memory)
constexpr int kKvMaxHeadDim = 256;
constexpr int kKvMinPage = 16, kKvMaxPage = 256;
constexpr int kKvMaxTokens = 0x7fffffff - 1023;  // of a block table's row: steps of keys are counted past the last one

WQ_HD int kv_pitch(int head_dim) { return (head_dim + 15) & ~15; }

WQ_HD int kv_clamp(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Tokens q0 .. q0 + n - 1 of the call belong to the sequence; its keys are 0 .. len - 1 and
// token i has position len - n + i (negative: the token has no place and sees no key).
// Offsets outside 0..M and lengths above the block table's capacity are cut to them.
struct KvSpan {
    int q0, n, len;
};
WQ_HD KvSpan kv_span(int cu_lo, int cu_hi, int seq_len, int M, int capacity)
{
    KvSpan s;
    s.q0 = kv_clamp(cu_lo, 0, M);
    s.n = kv_clamp(cu_hi, s.q0, M) - s.q0;
    s.len = kv_clamp(seq_len, 0, capacity);
    return s;
}
// The same for an append, with the length as it is: cut to the capacity, the positions counted from it
// would be those of earlier tokens.  Tokens from the limit (the capacity, or the rope table's
// length) on have no place: kv_placed.
WQ_HD KvSpan kv_append_span(int cu_lo, int cu_hi, int seq_len, int M) { return kv_span(cu_lo, cu_hi, seq_len, M, 0x7fffffff); }

// An append's work: a sequence with up to kKvFewTokens tokens in the call is one item, and the
// others' items are (sequence, page): sequence b with tokens q0 .. q1 - 1 owns those from
// kv_item_start(q0, b) to kv_item_start(q1, b + 1), at least floor(n / page) + 2 of them (floor(n / 4)
// is at least 2), and n tokens touch at most floor((n + page - 2) / page) + 1 pages.  So an item's
// sequence follows from cu_q alone, without a sum over the sequences before it.  by_seq: two items a
// sequence beside the pages, else one for every four tokens: whichever makes fewer.
constexpr int kKvFewTokens = 8;
WQ_HD int64_t kv_item_start(int q0, int b, int page_shift, bool by_seq)
{
    return int64_t(q0 >> page_shift) + (by_seq ? 2 * int64_t(b) : int64_t(q0 >> 2));
}

// Item k of a sequence: the logical page and the call's tokens in it.
struct KvPageSpan {
    int page;    // logical page (block-table column)
    int off;     // first new token's slot in the page: the page holds `off` earlier tokens
    int count;   // new tokens in the page (0: the item is idle)
    int token;   // the call's token at slot `off`
};
WQ_HD KvPageSpan kv_page_span(const KvSpan &s, int64_t k, int page_shift)
{
    KvPageSpan r{0, 0, 0, 0};
    if (k < 0) return r;                           // (sequences that overlap: no item's owner is certain)
    const int i0 = s.n > s.len ? s.n - s.len : 0;  // tokens without a place
    if (i0 >= s.n) return r;
    const int p0 = s.len - s.n + i0;               // first position written, >= 0
    const int64_t page = int64_t(p0 >> page_shift) + k;
    if (page > (s.len - 1) >> page_shift) return r;
    const int lo = int(page) << page_shift;
    const int first = lo > p0 ? lo : p0;
    const int64_t end = int64_t(lo) + (int64_t(1) << page_shift);
    const int last = end < s.len ? int(end) : s.len;  // exclusive
    r.page = int(page);
    r.off = first - lo;
    r.count = last - first;
    r.token = s.q0 + (first - (s.len - s.n));
    return r;
}

// How many of a page's new tokens lie below the limit; not positive: none, and the page may be none of
// the block table's.
WQ_HD int kv_placed(const KvPageSpan &p, int page_shift, int limit)
{
    const int left = limit - ((p.page << page_shift) + p.off);
    return p.count < left ? p.count : left;
}

// A physical page of the cache, or -1 where the block table's entry is out of range.
WQ_HD int64_t kv_page_ok(int entry, int64_t num_pages) { return entry >= 0 && entry < num_pages ? int64_t(entry) : -1; }

// Byte offset of (page, head, slot) in the codes, and index of (page, head) in the scales.
WQ_HD int64_t kv_code_offset(int64_t page, int head, int slot, int heads, int page_shift, int pitch)
{
    return (((page * heads + head) << page_shift) + slot) * int64_t(pitch);
}
WQ_HD int64_t kv_scale_index(int64_t page, int head, int heads) { return page * heads + head; }

// ---- attention: row tiles and units -------------------------------------------------
// The rows of (sequence, key head) are r = i * group + h (token i, query head h of the
// group), in tiles of `rows`; a tile's keys are walked in units of 2^shift tokens.  Every tile
// of a sequence counts the units of the sequence's whole length (at least one, so that tiles
// without keys are written too).
WQ_HD int64_t kv_tiles(int n, int group, int rows) { return (int64_t(n) * group + rows - 1) / rows; }
WQ_HD int kv_units(int len, int shift) { return len > 0 ? int((int64_t(len) + (int64_t(1) << shift) - 1) >> shift) : 1; }

// Which sequences go to the tile kernel: those with more rows per key head than this.  None where all
// rows together are at most `idle` (too few for its blocks), or where sequences bring at most
// kKvFewRows on average and the rows beyond one token a sequence are at most twice `idle`: a decode or
// draft batch.  If those are more, some sequence may be a long one among short ones (the host knows
// their number only): then what has more than `idle` rows by itself.
constexpr int kKvFewRows = 16;
WQ_HD int kv_few_rows(int64_t M, int64_t n_seqs, int q_heads, int kv_heads, int64_t idle)
{
    const int64_t rows = M * (q_heads / kv_heads);  // per key head
    if (M * q_heads <= idle || rows <= kKvFewRows) return 0x7fffffff;
    if (rows > kKvFewRows * n_seqs) return kKvFewRows;
    if ((M - n_seqs) * q_heads <= 2 * idle) return 0x7fffffff;
    return idle / kv_heads > kKvFewRows ? int(idle / kv_heads) : kKvFewRows;
}

// Blocks of `rows` rows for the sequences of a call without a sum over them: sequence b owns
// the items from kv_row_item(q0_b, b) to kv_row_item(q0_{b+1}, b + 1), at least
// floor(n * group / rows) + 1 >= kv_tiles(n, group, rows) of them.  few > 0: that many for sequences
// of more than `few` rows only, beside the multiples of `rows` one item for every few + 1 rows
// instead of one a sequence.
WQ_HD int64_t kv_row_item(int q0, int b, int group, int rows, int few = 0)
{
    const unsigned r = unsigned(q0) * unsigned(group);  // (below 2^31)
    return int64_t(r / unsigned(rows)) + (few ? r / unsigned(few + 1) : unsigned(b));
}

// Block c of `grid` takes the units kv_share(c) .. kv_share(c + 1) - 1 of `total` (grid below 2^16).
WQ_HD int kv_share(int total, int c, int grid)
{
    const unsigned q = unsigned(total) / unsigned(grid), r = unsigned(total) % unsigned(grid);
    return int(q * unsigned(c) + r * unsigned(c) / unsigned(grid));
}

}  // namespace wq
