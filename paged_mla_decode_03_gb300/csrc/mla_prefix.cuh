// Decode over shared prefixes: what its partitioner, its combine and the plan agree on.
//
// The requests of a group hold the same first rows in the cache (a system prompt, a
// document, the prompt of a beam search).  A softmax over a request's rows is the join of
// one over the shared rows and one over its own,
//   l = e^(lse_s) + e^(lse_o),   O = (e^(lse_s) O_s + e^(lse_o) O_o) / l,
// and the first may be taken for the query rows of all requests of the group together: a
// work item's 128 query rows are then full where a request alone has 16, and the shared
// rows are read once for each such item instead of once a request.
#pragma once

#include "mla_common.cuh"

namespace mla {

constexpr int kStatusPrefix = 256;  // a bad prefix_indptr, or a negative prefix length

// Workers of one list at most (their boundaries are held as bits).
constexpr int kPrefixWorkers = 254;

// The cost model, in tiles (of a worker's time).  An item's fixed part is some 6 us beside
// 0.75 us a tile of bf16, and 1.2 us of the other caches.
__host__ __device__ constexpr int prefix_overhead(int kv_dtype) { return kv_dtype == 0 ? 8 : 5; }

struct PrefixArgs {
  int groups;
  const int* lens;    // [groups] rows that the requests of a group share
  const int* indptr;  // [groups + 1] requests of a group, or nullptr: batch / groups each
};

// One row group of a request whose result is joined from partials: `rows` query rows from
// row0 of the output on (0: written by its only item).  Its own partials are in slots
// [own, own + n_own); row r of it is row off + r of the shared rows' partials, in
// slots [pre[0], pre[0] + n_pre[0]) below row 128, else row off + r - 128 of the second.
struct PrefixEntry {
  long long row0;
  int rows, own, n_own, off;
  int pre[2], n_pre[2];
};

// The regions of the workspace beside those that the decode kernel knows (Layout).
struct PrefixLayout {
  size_t entries;   // PrefixEntry[max_entries]
  size_t rg_first;  // int[max_rg]: first slot of each row group
  size_t rg_count;  // int[max_rg]: its items
  size_t owners;    // partitioner scratch, where shared memory does not hold it
  size_t scratch_bytes;
  int max_entries, max_rg;
  int scratch_in_smem;
};

// Partitioner scratch of each owner of row groups (a prefix group or a request), and of
// each request.
__host__ __device__ inline size_t prefix_scratch_bytes(long long owners, long long batch) {
  return align_up(sizeof(long long) * (size_t)(owners + 1), 16) + align_up(sizeof(int) * 3 * (size_t)(owners + 1), 16) +
         align_up(sizeof(int) * 5 * (size_t)batch, 16);
}

// The workspace of a plan with `groups` prefix groups.  Every item has a slot for its
// partial, that of its place in the list.
inline bool make_prefix_layout(long long batch, long long heads, long long max_q, bool packed, long long max_total_q,
                               int kv_dtype, long long groups, int n_workers, size_t header, Layout* lay,
                               PrefixLayout* pre) {
  const long long R = 128;
  auto ceil_to = [](long long a, long long b) { return (a + b - 1) / b; };
  const long long tokens = packed ? max_total_q : batch * max_q;
  long long own = batch * ceil_to(max_q * heads, R);
  if (packed && batch + ceil_to(tokens * heads, R) < own) own = batch + ceil_to(tokens * heads, R);
  const long long shared = groups + ceil_to(tokens * heads, R);
  const long long rg = own + shared > 1 ? own + shared : 1, items = rg + n_workers;
  if (items > (1LL << 24)) return false;
  lay->rows_per_group = (int)R;
  lay->n_workers = n_workers;
  lay->n_ctas = 2 * n_workers;
  lay->max_groups = (int)rg;
  lay->max_items = lay->max_partials = (int)items;
  lay->max_combine = 0;
  size_t off = header;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  lay->items = take(sizeof(WorkItem) * (size_t)items);
  lay->combine = off;
  lay->worker_ranges = take(sizeof(int) * (size_t)(n_workers + 1));
  pre->max_entries = (int)(own > 1 ? own : 1);
  pre->max_rg = (int)rg;
  pre->entries = take(sizeof(PrefixEntry) * (size_t)pre->max_entries);
  pre->rg_first = take(sizeof(int) * (size_t)rg);
  pre->rg_count = take(sizeof(int) * (size_t)rg);
  pre->scratch_bytes = prefix_scratch_bytes(groups + batch, batch);
  pre->scratch_in_smem = pre->scratch_bytes <= kPartitionSmemMax ? 1 : 0;
  pre->owners = take(pre->scratch_in_smem ? 0 : pre->scratch_bytes);
  lay->req_scratch = lay->group_scratch = pre->owners;
  lay->scratch_bytes = 0;
  lay->scratch_in_smem = 1;
  lay->part_o = take(part_row_bytes(kv_dtype, 1) * (size_t)R * (size_t)items);
  lay->part_lse = take(sizeof(float) * (size_t)R * (size_t)items);
  lay->comb_done = take(sizeof(int));
  lay->total = off;
  return true;
}

}  // namespace mla
