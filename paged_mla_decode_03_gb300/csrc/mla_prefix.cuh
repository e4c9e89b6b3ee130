// Decode over shared prefixes: what its partitioner, the decode kernel, its join and the plan
// agree on.
//
// The requests of a group hold the same first rows in the cache (a system prompt, a
// document, the prompt of a beam search).  Their query rows, one request after another, are
// cut into row groups of 128, which several requests share where each has fewer.  A row
// group walks a list of segments of whole tiles: first the shared rows, which all of its
// query rows see, then the own rows of each of its requests, which only that request's
// see.  So the shared rows are read and multiplied once for 128 query rows, and nothing has to
// be joined but row groups that are cut between workers.
#pragma once

#include "mla_common.cuh"

namespace mla {

constexpr int kStatusPrefix = 256;  // a bad prefix_indptr, or a negative prefix length

constexpr int kPrefixRows = 128;      // query rows of a row group
constexpr int kPrefixWorkers = 254;   // workers at most (their boundaries are held as bits)
// A row group holds the rows of eight requests at most (H >= 16), and the shared ones.
constexpr int kPrefixSegments = 9;

// The cost model, in tiles (of a worker's time).  An item's fixed part is some 6 us beside
// 0.75 us a tile of bf16, and 1.2 us of the other caches.
__host__ __device__ constexpr int prefix_overhead(int kv_dtype) { return kv_dtype == 0 ? 8 : 5; }

// What sharing has to save, in tiles of the estimate, for its segments and longer joins.
// Measured, a call with sharing and without: bf16, 16 heads, 8 requests behind 4000 rows 30.6 and 29.6 us (6 tiles
// saved), 32 behind 500 26.1 and 26.3 (6), 96 behind 128 45.3 and 50.6 (11), 4 behind 500 24.9 and 21.4
// (0); 4 bits, 16 requests behind 1000 27.0 and 29.4 (3.6), 8 behind 1000 26.5 and 26.1 (2).
__host__ __device__ constexpr int prefix_gain(int kv_dtype) { return kv_dtype == 0 ? 6 : 3; }

struct PrefixArgs {
  int groups;
  const int* lens;    // [groups] rows that the requests of a group share
  const int* indptr;  // [groups + 1] requests of a group, or nullptr: batch / groups each
};

// Tiles of a row group from tile0 on: rows row0, row0 + 64, .. of request b's table, up to
// `end`, seen by query rows [q_lo, q_hi) of the row group, row r by those up to
// mask + (token of r in its owner).
struct PrefixSegment {
  int tile0, b, row0, end;
  int q_lo, q_hi, mask, pad;
};
constexpr int kPrefixNoMask = 1 << 30;  // `mask` of a segment that is seen whole

// Widening.  Over 4 bits and e4m3 a tile's time goes into its conversion to f16 (1.25 and 1.36 us,
// where rows that come by TMA take 0.88).  Where four row groups and more walk the same shared rows
// these are widened once, into the workspace, and walked there, by a list of items of its
// own; the row groups' own rows stay in the first list, and all their query rows are joined.
// Measured without and with, us in a graph, 128 heads, e4m3 (4 bits save less, 0.40 us a tile of a worker
// instead of 0.46): 32 row groups over 65536 rows 591 and 395, over 8192 98 and 89, over 2048 45 and 59; 16
// over 20480 115 and 99, over 8192 62 and 69; 8 over 65536 170 and 150, over 20480 73 and 76; 4 over 65536 104 and
// 111; 12 groups of 8 over 8192 260 and 233, of 4 142 and 153.  So what is saved has to pay for the copy (a row
// read and written: kWideCopy), items and partials of both lists, and kWideFixed: the partitioner weighs
// that, by the lengths it finds.  A plan whose groups have fewer than four row groups has no room for it
// (4 groups of 2, 8 requests of 32 heads each, over 16384 rows: 65 and 95).  One that has, and whose rows are not
// widened, takes some 10 us for the two kernels more.
constexpr int kWideRowGroups = 4;
constexpr int kWideCopy = 75;   // tiles that are widened in the time of one of the first list's
constexpr int kWideFixed = 11;  // of the second list's join and first loads, in the first one's tiles
constexpr long long kWideBytes = 1LL << 30;  // of widened rows at most
constexpr int kWideOverhead = 8;             // of an item over them, in their tiles
constexpr int kWideTenths = 7;               // one of their tiles, in tenths of another's

// A prefix group's widened rows: tiles [base, base + tiles) from request b's table; the entry
// past the last group has the number of all in `base`.
struct PrefixWide {
  int base, tiles, b, pad;
};

// The items of a plan with prefix groups: g is the row group of its owner's q_len tokens from
// q_start on, [kv_begin, kv_end) its tiles times 64, comb its number among all row
// groups and seq_len its segments.

// A row group that is joined: its query rows from row0 of the output on (0: it is not) and its
// partials of either list.
struct PrefixEntry {
  long long row0;
  int rows, pad;
  int slot[2], count[2];
};

// The regions of the workspace beside those that the decode kernel knows (Layout).
struct PrefixLayout {
  size_t entries;   // PrefixEntry[max_groups]
  size_t segments;  // PrefixSegment[max_groups][kPrefixSegments]
  size_t scratch;   // the partitioner's, where shared memory does not hold it
  size_t scratch_bytes;
  int scratch_in_smem;
  // plans that widen (wide_tiles > 0: tiles of widened rows): the second list, its row groups'
  // one segment each (kPrefixSegments apart), PrefixWide[groups + 1], f16 rows of 576
  int wide_tiles;
  size_t wide_items, wide_ranges, wide_segments, wide_groups, wide_rows;
};

// Partials are f16, laid out as part_unit says: over 4 bits and e4m3 times 2^part_shift; over
// bf16, whose values have no bound, 16 dims of a row times a power of two that brings the
// largest of them to [2^14, 2^15), so that each is off by 2^-11 of itself or 2^-39 of the
// largest.  The powers, a byte for each row and 16 dims, follow the LSEs.  (fp32 partials were
// as near and twice the bytes, which bound the join: 6 x 10 requests of 1 to 4 tokens, 64
// heads: 143 us instead of 132.)
__host__ __device__ inline size_t prefix_scale_offset(const Layout& lay) {
  return align_up(lay.part_lse + sizeof(float) * kPrefixRows * (size_t)lay.max_partials, 256);
}
// The power: 0 for zeros, a NaN or an infinity.
__host__ __device__ inline int prefix_scale(unsigned max_bits) {
  const int e = (int)(max_bits >> 23);
  if (max_bits == 0 || e == 255) return 0;
  return 141 - e < 126 ? 141 - e : 126;
}

// Partitioner scratch: by request, prefix group and row group.
__host__ __device__ inline size_t prefix_scratch_bytes(long long batch, long long groups, long long row_groups) {
  return align_up(sizeof(int) * (size_t)(8 * batch + 2 + 5 * groups + 4 * row_groups + 2), 16);
}

// The workspace of a plan with `groups` prefix groups; false: too large a plan.  may_widen: with the room
// that widening wants, where it may pay at all.  Without, it is what every run of the plan needs.
inline bool make_prefix_layout(long long batch, long long heads, long long max_q, bool packed, long long max_total_q,
                               long long max_seq_len, int kv_dtype, long long groups, int n_workers, size_t header,
                               Layout* lay, PrefixLayout* pre, bool may_widen = true) {
  const long long R = kPrefixRows;
  auto ceil_to = [](long long a, long long b) { return (a + b - 1) / b; };
  long long rg = batch * ceil_to(max_q * heads, R);
  if (packed && batch + ceil_to(max_total_q * heads, R) < rg) rg = batch + ceil_to(max_total_q * heads, R);
  rg = rg > 1 ? rg : 1;
  const long long items = rg + n_workers;
  // costs are held in 32 bits (a row group walks kPrefixSegments requests' rows at most)
  const long long cost = rg * (prefix_overhead(0) + kPrefixSegments * (max_seq_len / kKvTile + 1));
  if (items > (1LL << 24) || cost >= (1LL << 31)) return false;
  lay->rows_per_group = (int)R;
  lay->n_workers = n_workers;
  lay->n_ctas = 2 * n_workers;
  lay->max_groups = (int)rg;
  lay->max_items = (int)items;
  // widening pays for four row groups a prefix group on the average, and has its room
  const long long tokens = packed ? max_total_q : batch * max_q;
  const long long tiles = groups * ((max_seq_len + kKvTile - 1) / kKvTile);
  const bool wide = may_widen && kv_dtype != 0 && ceil_to(tokens * heads, R) >= kWideRowGroups * groups &&
                    tiles * kKvTile * 2 * kQkDim <= kWideBytes;
  pre->wide_tiles = wide ? (int)tiles : 0;
  // cut row groups have partials, all of those with widened rows
  lay->max_partials = (int)(wide ? 2 * items : items < 2LL * n_workers ? items : 2LL * n_workers);
  lay->max_combine = 0;
  size_t off = header;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  lay->items = take(sizeof(WorkItem) * (size_t)items);
  lay->worker_ranges = take(sizeof(int) * (size_t)(n_workers + 1));
  pre->entries = take(sizeof(PrefixEntry) * (size_t)rg);
  lay->combine = pre->segments = take(sizeof(PrefixSegment) * (size_t)(kPrefixSegments * rg));
  pre->scratch_bytes = prefix_scratch_bytes(batch, groups, rg);
  pre->scratch_in_smem = pre->scratch_bytes <= kPartitionSmemMax ? 1 : 0;
  pre->scratch = take(pre->scratch_in_smem ? 0 : pre->scratch_bytes);
  lay->req_scratch = lay->group_scratch = pre->scratch;
  lay->scratch_bytes = 0;
  lay->scratch_in_smem = 1;
  lay->part_o = take(kPartBytesPerRow * (size_t)R * (size_t)lay->max_partials);
  lay->part_lse = take(sizeof(float) * (size_t)R * (size_t)lay->max_partials);
  if (kv_dtype == 0) take(32 * (size_t)R * (size_t)lay->max_partials);  // (prefix_scale_offset)
  lay->comb_done = take(sizeof(int));
  pre->wide_items = pre->wide_ranges = pre->wide_segments = pre->wide_groups = pre->wide_rows = off;
  if (wide) {
    pre->wide_items = take(sizeof(WorkItem) * (size_t)items);
    pre->wide_ranges = take(sizeof(int) * (size_t)(n_workers + 1));
    pre->wide_segments = take(sizeof(PrefixSegment) * (size_t)(kPrefixSegments * rg));
    pre->wide_groups = take(sizeof(PrefixWide) * (size_t)(groups + 1));
    pre->wide_rows = take((size_t)tiles * kKvTile * 2 * kQkDim);
  }
  lay->total = off;
  return true;
}

}  // namespace mla
