// Runs the partitioner of plans with shared prefixes (its source, with host stand-ins) on
// host threads, one problem per text file, and writes the work list and the join's entries.
// Built by tests/test_prefix_partition.py.
#include <cstdio>
#include <deque>
#include <string>

#include "shim.h"

template <typename T, typename F>
T host_reduce(T v, F f) {
  T r = host_exchange(v, 0);
  for (int l = 1; l < 32; ++l) r = f(r, host_exchange(v, l));
  return r;
}
inline int __reduce_min_sync(unsigned, int v) { return host_reduce(v, [](int a, int b) { return min(a, b); }); }
inline int __reduce_max_sync(unsigned, int v) { return host_reduce(v, [](int a, int b) { return max(a, b); }); }
inline unsigned __reduce_add_sync(unsigned, unsigned v) { return host_reduce(v, [](unsigned a, unsigned b) { return a + b; }); }
inline unsigned __reduce_or_sync(unsigned, unsigned v) { return host_reduce(v, [](unsigned a, unsigned b) { return a | b; }); }
inline int __popc(unsigned v) { return __builtin_popcount(v); }
inline int atomicAdd(int* p, int v) { return std::atomic_ref<int>(*p).fetch_add(v); }
inline int atomicMax(int* p, int v) {
  std::atomic_ref<int> a(*p);
  int old = a.load();
  while (old < v && !a.compare_exchange_weak(old, v)) {
  }
  return old;
}
#include "mla_common_host.h"
#include "mla_prefix_host.h"
#include "partition_prefix_host.inc"

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  FILE* f = std::fopen(argv[1], "r");
  if (!f) return 2;
  int B, H, packed, max_q, max_seq_len, n_workers, causal, kv_dtype, G, uniform, global_scratch;
  long long total_q;
  if (std::fscanf(f, "%d %d %d %d %d %d %d %d %d %d %d %lld", &B, &H, &packed, &max_q, &max_seq_len, &n_workers,
                  &causal, &kv_dtype, &G, &uniform, &global_scratch, &total_q) != 12)
    return 2;
  std::vector<int> seq_lens(B), qo(B + 1), lens(G), indptr(G + 1);
  for (auto* v : {&seq_lens, &qo, &lens, &indptr})
    for (auto& x : *v)
      if (std::fscanf(f, "%d", &x) != 1) return 2;
  std::fclose(f);
  mla::Layout lay{};
  mla::PrefixLayout pl{};
  if (!mla::make_prefix_layout(B, H, max_q, packed, total_q, max_seq_len, kv_dtype, G, n_workers, sizeof(int) * mla::kHdrWords, &lay, &pl))
    return 3;
  const size_t starts[] = {lay.items, lay.worker_ranges, pl.entries, pl.segments, lay.part_o, lay.part_lse, lay.comb_done, pl.wide_items,
                           pl.wide_ranges, pl.wide_segments, pl.wide_groups, pl.wide_rows, lay.total};
  for (size_t i = 0; i < sizeof(starts) / sizeof(starts[0]); ++i)
    if (starts[i] % 256 || (i > 0 && starts[i] < starts[i - 1])) return 5;
  if (pl.segments + sizeof(mla::PrefixSegment) * mla::kPrefixSegments * (size_t)lay.max_groups > lay.part_o) return 5;
  if (global_scratch) {  // as a batch that shared memory does not hold: the scratch past the rest
    pl.scratch_in_smem = 0;
    pl.scratch = lay.part_o;
  }
  if (pl.wide_tiles > 0) {
    if (pl.wide_segments + sizeof(mla::PrefixSegment) * mla::kPrefixSegments * (size_t)lay.max_groups > pl.wide_groups ||
        pl.wide_groups + sizeof(mla::PrefixWide) * (size_t)(G + 1) > pl.wide_rows ||
        pl.wide_rows + (size_t)pl.wide_tiles * mla::kKvTile * 1152 > lay.total)
      return 5;
    // (no partial is touched here: the second list right behind the first)
    const size_t back = pl.wide_items - lay.part_o;
    for (size_t* at : {&pl.wide_items, &pl.wide_ranges, &pl.wide_segments, &pl.wide_groups, &pl.wide_rows}) *at -= back;
  }
  const size_t end = pl.wide_tiles > 0 ? pl.wide_rows : lay.part_o;
  if (global_scratch) pl.scratch = end;
  const size_t used = end + (global_scratch ? pl.scratch_bytes : 0);
  std::vector<unsigned char> ws(used, 0xAB);
  std::vector<unsigned char> scratch(pl.scratch_in_smem ? pl.scratch_bytes : 16, 0xCD);
  g_scratch = scratch.data();
  mla::Problem p{};
  p.batch = B;
  p.num_heads = H;
  p.max_q = max_q;
  p.max_seq_len = max_seq_len;
  p.packed = packed;
  p.kv_dtype = kv_dtype;
  p.causal = causal;
  p.cp_world = 1;
  p.total_q = total_q;
  p.seq_lens = seq_lens.data();
  p.qo_indptr = packed ? qo.data() : nullptr;
  const mla::PrefixArgs pa{G, lens.data(), uniform ? nullptr : indptr.data()};
  const int threads = mla::partition_prefix_threads(p, pa, lay);
  blockDim.x = threads;
  std::barrier<> block_bar(threads);
  g_block_barrier = &block_bar;
  std::deque<std::barrier<>> warp_bars;  // constructed in place, never moved
  std::vector<HostWarp> warps(threads / 32);
  for (int w = 0; w < threads / 32; ++w) {
    warp_bars.emplace_back(32);
    warps[w].bar = &warp_bars[w];
    g_warps.push_back(&warps[w]);
  }
  std::vector<std::thread> th;
  for (int t = 0; t < threads; ++t)
    th.emplace_back([&, t] {
      threadIdx.x = t;
      (pl.wide_tiles > 0 ? mla::partition_prefix_kernel<true> : mla::partition_prefix_kernel<false>)(
          p, pa, lay, pl, reinterpret_cast<char*>(ws.data()));
    });
  for (auto& x : th) x.join();
  const int* hdr = reinterpret_cast<const int*>(ws.data());
  FILE* o = std::fopen(argv[2], "w");
  if (!o) return 2;
  std::fprintf(o, "%d %d %d %d %d %d\n", hdr[mla::kHdrStatus], hdr[mla::kHdrNumItems], hdr[mla::kHdrNumCombine],
               lay.max_items, lay.max_groups, lay.max_partials);
  const int* items = reinterpret_cast<const int*>(ws.data() + lay.items);
  for (int i = 0; i < hdr[mla::kHdrNumItems] * 10; ++i) std::fprintf(o, "%d ", items[i]);
  std::fprintf(o, "\n");
  const int* wb = reinterpret_cast<const int*>(ws.data() + lay.worker_ranges);
  for (int i = 0; i <= n_workers; ++i) std::fprintf(o, "%d ", wb[i]);
  std::fprintf(o, "\n");
  const mla::PrefixEntry* e = reinterpret_cast<const mla::PrefixEntry*>(ws.data() + pl.entries);
  for (int i = 0; i < hdr[mla::kHdrNumCombine]; ++i)
    std::fprintf(o, "%lld %d %d %d %d %d ", e[i].row0, e[i].rows, e[i].slot[0], e[i].count[0], e[i].slot[1], e[i].count[1]);
  std::fprintf(o, "\n");
  const mla::PrefixSegment* sg = reinterpret_cast<const mla::PrefixSegment*>(ws.data() + pl.segments);
  for (int i = 0; i < hdr[mla::kHdrNumCombine] * mla::kPrefixSegments; ++i)
    std::fprintf(o, "%d %d %d %d %d %d %d ", sg[i].tile0, sg[i].b, sg[i].row0, sg[i].end, sg[i].q_lo, sg[i].q_hi, sg[i].mask);
  std::fprintf(o, "\n");
  const bool wide = pl.wide_tiles > 0;
  const int* wr = reinterpret_cast<const int*>(ws.data() + pl.wide_ranges);
  const int n_wide = wide ? wr[n_workers] : 0;
  const int* wi = reinterpret_cast<const int*>(ws.data() + pl.wide_items);
  for (int i = 0; i < n_wide * 10; ++i) std::fprintf(o, "%d ", wi[i]);
  std::fprintf(o, "\n");
  for (int i = 0; wide && i <= n_workers; ++i) std::fprintf(o, "%d ", wr[i]);
  std::fprintf(o, "\n");
  const mla::PrefixSegment* wsg = reinterpret_cast<const mla::PrefixSegment*>(ws.data() + pl.wide_segments);
  for (int i = 0; i < n_wide; ++i) {  // by item: its row group's one segment
    const mla::PrefixSegment& z = wsg[(size_t)wi[10 * i + 8] * mla::kPrefixSegments];
    std::fprintf(o, "%d %d %d %d %d %d %d ", z.tile0, z.b, z.row0, z.end, z.q_lo, z.q_hi, z.mask);
  }
  std::fprintf(o, "\n");
  const mla::PrefixWide* wg = reinterpret_cast<const mla::PrefixWide*>(ws.data() + pl.wide_groups);
  for (int i = 0; wide && i <= G; ++i) std::fprintf(o, "%d %d %d ", wg[i].base, wg[i].tiles, wg[i].b);
  std::fprintf(o, "\n%d\n", pl.wide_tiles);
  std::fclose(o);
  return 0;
}
