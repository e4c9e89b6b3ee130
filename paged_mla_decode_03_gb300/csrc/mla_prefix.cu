// The work list and the join of a decode over shared prefixes (mla_prefix.cuh); the items
// run on mla_decode_pair.cu's kernel.
//
// Partition.  Owners of row groups are first the prefix groups, then the requests.  A
// prefix group with P shared rows owns ceil(tokens H / 128) row groups of P / 64 tiles, a
// request ceil(q H / 128) of its rows from P on.  All row groups of an owner cost the same,
// so start units need a scan over the owners alone, and the row group at a unit is a search
// among them and a division.  The rest follows mla_partition_pair.cu: worker boundary p lies
// at unit floor(p W / n'), and with two bits a boundary the place of every item is a
// population count.
//
// Whether a group's rows are shared is decided here, from its lengths.  Sharing saves the
// tiles of the row groups that are left out, and costs the items of the shared ones and the
// round trip of two partials a query row (2 to 4 KB written and read back: for 128 rows some
// 0.2 us of the whole card, 15 us of one worker).  What all groups save together has to shorten a
// worker's share by more than the join's tail.
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_common.cuh"
#include "mla_prefix.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

constexpr int kPartThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowsAJoinTile = 6;       // query rows whose partials take a tile's time
constexpr long long kJoinTailTiles = 4;

// Owners: start unit, first row group, row groups, tiles of each.  Requests: tokens, first
// token, rows, prefix group (-1: none shared), first of all the request's row groups.
struct PrefixScratch {
  long long* start;
  int *base, *count, *tiles;
  int *q, *qs, *len, *group, *entry;
  __device__ PrefixScratch(char* at, int owners, int batch) {
    start = reinterpret_cast<long long*>(at);
    base = reinterpret_cast<int*>(at + align_up(sizeof(long long) * (size_t)(owners + 1), 16));
    count = base + owners + 1;
    tiles = count + owners + 1;
    q = reinterpret_cast<int*>(reinterpret_cast<char*>(base) + align_up(sizeof(int) * 3 * (size_t)(owners + 1), 16));
    qs = q + batch;
    len = qs + batch;
    group = len + batch;
    entry = group + batch;
  }
};

struct PrefixShared {
  long long w_cost[32], carry_cost, saved;
  int w_count[32], carry_count, status, max_tiles, bad;
  long long bound[kPrefixWorkers + 1];
  unsigned cut[8], first[8];
};

template <typename T>
__device__ __forceinline__ T scan_up(T v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// Last index in [0, n) whose value is at most x (values ascending, the first at most x).
template <typename T>
__device__ __forceinline__ int last_upto(const T* v, int n, T x) {
  int lo = 0;
  while (n - lo > 1) {
    const int mid = (lo + n) >> 1;
    if (v[mid] <= x) lo = mid; else n = mid;
  }
  return lo;
}
__device__ __forceinline__ int bits_under(const unsigned* words, int p) {
  int c = 0;
  for (int w = 0; w < (p >> 5); ++w) c += __popc(words[w]);
  return (p & 31) ? c + __popc(words[p >> 5] << (32 - (p & 31))) : c;
}
__device__ __forceinline__ bool bit_at(const unsigned* words, int p) { return (words[p >> 5] >> (p & 31)) & 1u; }

// Exclusive scans over n owners of (cost of all its row groups, their number), carried from
// one pass of the block to the next; the totals end up past the last owner.
__device__ void scan_owners(PrefixShared& sh, const PrefixScratch& s, int n, int overhead) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  if (tid == 0) {
    sh.carry_cost = 0;
    sh.carry_count = 0;
  }
  __syncthreads();
  for (int at = 0; at < n; at += blockDim.x) {
    const int o = at + tid;
    const int c = o < n ? s.count[o] : 0;
    const long long cost = o < n ? (long long)c * (overhead + s.tiles[o]) : 0;
    const long long in_cost = scan_up(cost, lane);
    const int in_count = scan_up(c, lane);
    if (lane == 31) {
      sh.w_cost[warp] = in_cost;
      sh.w_count[warp] = in_count;
    }
    __syncthreads();
    long long before = sh.carry_cost;
    int n_before = sh.carry_count;
    for (int w = 0; w < warp; ++w) {
      before += sh.w_cost[w];
      n_before += sh.w_count[w];
    }
    if (o < n) {
      s.start[o] = before + in_cost - cost;
      s.base[o] = n_before + in_count - c;
    }
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < n_warps; ++w) {
        sh.carry_cost += sh.w_cost[w];
        sh.carry_count += sh.w_count[w];
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    s.start[n] = sh.carry_cost;
    s.base[n] = sh.carry_count;
  }
  __syncthreads();
}

}  // namespace

__global__ void __launch_bounds__(kPartThreads, 1)
partition_prefix_kernel(Problem p, PrefixArgs pa, Layout lay, PrefixLayout pl, char* __restrict__ ws) {
  extern __shared__ __align__(16) unsigned char prefix_smem[];
  __shared__ PrefixShared sh;
  ptx::pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int B = p.batch, G = pa.groups, H = p.num_heads, R = lay.rows_per_group, n = lay.n_workers;
  const int c0 = prefix_overhead(p.kv_dtype);
  int* hdr = reinterpret_cast<int*>(ws);
  WorkItem* items = reinterpret_cast<WorkItem*>(ws + lay.items);
  int* worker_begin = reinterpret_cast<int*>(ws + lay.worker_ranges);
  PrefixEntry* entries = reinterpret_cast<PrefixEntry*>(ws + pl.entries);
  int* rg_first = reinterpret_cast<int*>(ws + pl.rg_first);
  int* rg_count = reinterpret_cast<int*>(ws + pl.rg_count);
  const int owners = G + B;
  const PrefixScratch s(pl.scratch_in_smem ? reinterpret_cast<char*>(prefix_smem) : ws + pl.owners, owners, B);
  auto tiles_of = [](int rows) { return (rows + kKvTile - 1) / kKvTile; };
  auto groups_of = [&](int tokens) { return (int)(((long long)tokens * H + R - 1) / R); };
  if (tid == 0) {
    sh.saved = 0;
    sh.status = sh.max_tiles = 0;
  }
  __syncthreads();

  // 1. Requests: lengths, clamped and flagged as by the other partitioners.
  int status = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    int q, qs, L = p.seq_lens[b];
    if (p.packed) {
      int lo = p.qo_indptr[b], hi = p.qo_indptr[b + 1];
      const int tq = (int)p.total_q;
      if (lo < 0 || hi > tq || hi - lo < 1 || hi - lo > p.max_q) status |= kStatusQLen;
      lo = min(max(lo, 0), tq);
      hi = min(max(hi, lo), tq);
      q = min(hi - lo, p.max_q);
      qs = lo;
    } else {
      q = p.max_q;
      qs = b * p.max_q;
    }
    if (L < 1 || L > p.max_seq_len) status |= kStatusSeqLen;
    L = min(max(L, 0), p.max_seq_len);
    if (p.causal && q > L) status |= kStatusCausal;
    s.q[b] = q;
    s.qs[b] = qs;
    s.len[b] = L;
    s.group[b] = -1;
    s.count[G + b] = L > 0 ? groups_of(q) : 0;
    s.tiles[G + b] = tiles_of(L);
  }
  // 2. Prefix groups: a warp each.  Where the offsets are bad nothing is shared.
  int bad = 0;
  if (pa.indptr)
    for (int g = tid; g < G; g += blockDim.x) {
      const int lo = pa.indptr[g], hi = pa.indptr[g + 1];
      if (lo < 0 || hi < lo || hi > B) bad = 1;
    }
  bad = __syncthreads_or(bad);
  if (bad) status |= kStatusPrefix;
  for (int g = warp; g < G; g += n_warps) {
    const int each = B / G;
    const int lo = bad ? 0 : pa.indptr ? pa.indptr[g] : g * each;
    const int hi = bad ? 0 : pa.indptr ? pa.indptr[g + 1] : lo + each;
    int rows = INT_MAX, tokens = 0, alone = 0, apart = 0;
    for (int b = lo + lane; b < hi; b += 32) {
      if (s.len[b] > 0 && s.q[b] > 0) rows = min(rows, p.causal ? s.len[b] - s.q[b] + 1 : s.len[b]);
      tokens += s.q[b];
      alone += s.count[G + b];
      // (the group's query rows have to follow on one another)
      if (b + 1 < hi && s.qs[b + 1] != s.qs[b] + s.q[b]) apart = 1;
    }
    rows = __reduce_min_sync(kAll, rows);
    tokens = (int)__reduce_add_sync(kAll, (unsigned)tokens);
    alone = (int)__reduce_add_sync(kAll, (unsigned)alone);
    apart = (int)__reduce_or_sync(kAll, (unsigned)apart);
    const int len = pa.lens[g];
    if (len < 0) status |= kStatusPrefix;
    if (lane == 0) {
      const int T = apart || rows == INT_MAX ? 0 : max(0, min(len, rows)) / kKvTile;
      const int together = groups_of(tokens);
      const long long saved =
          (long long)(alone - together) * T - (long long)together * c0 - (long long)tokens * H / kRowsAJoinTile;
      s.count[g] = T > 0 && saved > 0 ? together : 0;
      s.tiles[g] = T;
      if (T > 0 && saved > 0)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.saved), (unsigned long long)saved);
    }
  }
  if (status) atomicOr(&sh.status, status);
  __syncthreads();
  const bool share = sh.saved > kJoinTailTiles * n;
  for (int g = warp; g < G; g += n_warps) {
    const int each = B / G;
    const bool on = share && s.count[g] > 0;
    __syncwarp();
    if (!on) {
      if (lane == 0) s.count[g] = 0;
      continue;
    }
    const int lo = pa.indptr ? pa.indptr[g] : g * each, hi = pa.indptr ? pa.indptr[g + 1] : lo + each;
    for (int b = lo + lane; b < hi; b += 32) {
      s.group[b] = g;
      if (s.len[b] > 0) s.tiles[G + b] -= s.tiles[g];
    }
  }
  __syncthreads();
  // the requests' row groups, all of them, are the join's entries; a request without a
  // row of its own has no item
  {
    int most = 0;
    if (tid == 0) sh.carry_count = 0;
    __syncthreads();
    for (int at = 0; at < B; at += blockDim.x) {
      const int b = at + tid;
      const int c = b < B ? s.count[G + b] : 0;
      const int in = scan_up(c, lane);
      if (lane == 31) sh.w_count[warp] = in;
      __syncthreads();
      int before = sh.carry_count;
      for (int w = 0; w < warp; ++w) before += sh.w_count[w];
      if (b < B) {
        s.entry[b] = before + in - c;
        if (s.tiles[G + b] <= 0) s.count[G + b] = 0;
        if (c > 0) most = max(most, s.tiles[G + b]);
      }
      __syncthreads();
      if (tid == 0)
        for (int w = 0; w < n_warps; ++w) sh.carry_count += sh.w_count[w];
      __syncthreads();
    }
    for (int g = tid; g < G; g += blockDim.x)
      if (s.count[g] > 0) most = max(most, s.tiles[g]);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) atomicMax(&sh.max_tiles, most);
  }
  const int n_entries = sh.carry_count;
  __syncthreads();
  scan_owners(sh, s, owners, c0);
  const long long W = s.start[owners];
  const int n_rg = s.base[owners];
  const int n_eff = (int)max(1LL, min((long long)n, W / kMinUnits));
  const bool uncut = partition_uncut(true, n_rg, n, c0 + sh.max_tiles, W);
  // (malformed offsets may let requests overlap: more row groups than the plan has room for)
  const bool room = n_rg <= lay.max_groups && n_entries <= pl.max_entries;

  // 3. Worker boundaries, and the row group that each falls into.
  struct Group {  // of a row group: owner, number in it, start unit, tiles
    int owner, k, T;
    long long S;
  };
  auto group_at = [&](long long unit) {
    Group g;
    g.owner = last_upto(s.start, owners, unit);
    g.T = s.tiles[g.owner];
    g.k = (int)((unit - s.start[g.owner]) / (c0 + g.T));
    g.S = s.start[g.owner] + (long long)g.k * (c0 + g.T);
    return g;
  };
  auto group_no = [&](int rg) {
    Group g;
    g.owner = last_upto(s.base, owners, rg);
    g.T = s.tiles[g.owner];
    g.k = rg - s.base[g.owner];
    g.S = s.start[g.owner] + (long long)g.k * (c0 + g.T);
    return g;
  };
  for (int w = tid; w <= n; w += blockDim.x) {
    if (uncut)
      sh.bound[w] = room && w < n_rg ? group_no(w).S : W;
    else
      sh.bound[w] = w >= n_eff ? W : w * (W / n_eff) + w * (W % n_eff) / n_eff;
  }
  if (tid < 8) sh.cut[tid] = sh.first[tid] = 0;
  __syncthreads();
  for (int w = tid; w <= n; w += blockDim.x) {
    if (w == 0 || sh.bound[w] >= W) continue;
    const Group g = group_at(sh.bound[w]);
    const long long t = sh.bound[w] - g.S - c0;
    if (t <= 0) continue;
    atomicOr(reinterpret_cast<int*>(&sh.cut[w >> 5]), (int)(1u << (w & 31)));
    if (sh.bound[w - 1] - g.S - c0 <= 0) atomicOr(reinterpret_cast<int*>(&sh.first[w >> 5]), (int)(1u << (w & 31)));
  }
  __syncthreads();

  // 4. Items, row groups' slots, worker ranges.
  const int n_items = n_rg + bits_under(sh.cut, 255);
  const bool fits = room && n_items <= lay.max_items;
  auto emit = [&](int at, const Group& g, long long t0, long long t1, bool partial) {
    WorkItem it;
    it.g = g.k;
    it.slot = partial ? at : -1;
    it.comb = -1;
    if (g.owner < G) {
      const int lo = pa.indptr ? pa.indptr[g.owner] : g.owner * (B / G);
      const int hi = pa.indptr ? pa.indptr[g.owner + 1] : lo + B / G;
      int b = lo;  // the first request that has rows: its table is read
      while (b + 1 < hi && s.len[b] <= 0) ++b;
      const int P = g.T * kKvTile;
      it.b = b;
      it.kv_begin = (int)t0 * kKvTile;
      it.kv_end = (int)t1 * kKvTile;
      it.q_start = s.qs[lo];
      it.q_len = s.qs[hi - 1] + s.q[hi - 1] - it.q_start;
      it.seq_len = P;
      it.mask_base = P - 1;  // every query row sees every shared row
    } else {
      const int b = g.owner - G, P = s.group[b] >= 0 ? s.tiles[s.group[b]] * kKvTile : 0;
      it.b = b;
      it.kv_begin = P + (int)t0 * kKvTile;
      it.kv_end = min(s.len[b], P + (int)t1 * kKvTile);
      it.q_start = s.qs[b];
      it.q_len = s.q[b];
      it.seq_len = s.len[b];
      it.mask_base = s.len[b] - s.q[b];
    }
    items[at] = it;
  };
  auto shared_owner = [&](int owner) { return owner < G || s.group[owner - G] >= 0; };
  if (fits)
    for (int rg = tid; rg < n_rg; rg += blockDim.x) {
      const Group g = group_no(rg);
      // boundaries at or below the unit of the group's first tile
      const int pb = sh.bound[0] > g.S + c0 ? 0 : last_upto(sh.bound, n + 1, g.S + c0) + 1;
      const long long end = g.S + c0 + g.T;
      int last = pb;  // past the group's last cut
      while (last < n && bit_at(sh.cut, last) && sh.bound[last] < end) ++last;
      const int at = rg + bits_under(sh.cut, pb);
      const bool partial = last > pb || shared_owner(g.owner);
      rg_first[rg] = at;
      rg_count[rg] = partial ? 1 + last - pb : 0;
      emit(at, g, 0, last > pb ? sh.bound[pb] - g.S - c0 : g.T, partial);
    }
  if (fits)
    for (int w = tid; w <= n; w += blockDim.x) {
      if (sh.bound[w] >= W) {
        worker_begin[w] = n_items;
        continue;
      }
      const Group g = group_at(sh.bound[w]);
      const bool cuts = bit_at(sh.cut, w);
      const int rg = s.base[g.owner] + g.k;
      // (a boundary inside a group's overhead, or at its start, leaves the group whole)
      worker_begin[w] = rg + bits_under(sh.cut, w) + (cuts ? 1 : 0);
      if (!cuts) continue;
      const long long t = sh.bound[w] - g.S - c0;
      const long long next = w + 1 <= n ? min((long long)g.T, sh.bound[w + 1] - g.S - c0) : g.T;
      emit(rg + 1 + bits_under(sh.cut, w), g, t, next, true);
    }
  if (!fits)
    for (int w = tid; w <= n; w += blockDim.x) worker_begin[w] = 0;
  __syncthreads();

  // 5. The join's entries.
  if (fits)
    for (int b = warp; b < B; b += n_warps) {
      const int all = s.len[b] > 0 ? groups_of(s.q[b]) : 0, own = s.count[G + b], g = s.group[b];
      int token0 = 0;  // of the request, in its prefix group
      if (g >= 0) token0 = s.qs[b] - s.qs[pa.indptr ? pa.indptr[g] : g * (B / G)];
      for (int k = lane; k < all; k += 32) {
        PrefixEntry e = {};
        e.row0 = (long long)s.qs[b] * H + (long long)k * R;
        e.rows = (int)min((long long)R, (long long)s.q[b] * H - (long long)k * R);
        if (own > 0) {
          e.own = rg_first[s.base[G + b] + k];
          e.n_own = rg_count[s.base[G + b] + k];
        }
        if (g >= 0) {
          const long long row = (long long)token0 * H + (long long)k * R;
          const int first = (int)(row / R);
          e.off = (int)(row % R);
          for (int i = 0; i < 2; ++i)
            if (first + i < s.count[g]) {
              e.pre[i] = rg_first[s.base[g] + first + i];
              e.n_pre[i] = rg_count[s.base[g] + first + i];
            }
        } else if (e.n_own == 0) {
          e.rows = 0;
        }
        entries[s.entry[b] + k] = e;
      }
    }
  if (tid == 0) {
    hdr[kHdrStatus] = fits ? sh.status : sh.status | kStatusCapacity;
    hdr[kHdrNumItems] = fits ? n_items : 0;
    hdr[kHdrWorkCounter] = 0;
    hdr[kHdrNumCombine] = fits ? n_entries : 0;
    hdr[kHdrChunkTiles] = (int)min(W, 1LL << 30);
    hdr[kHdrCombineCounter] = 0;
  }
}

// A thread for each request and worker boundary, a warp for each prefix group.
inline int partition_prefix_threads(const Problem& p, const PrefixArgs& pa, const Layout& lay) {
  const long long need = std::max(std::max((long long)p.batch, 32LL * pa.groups), (long long)lay.n_workers + 1);
  return (int)std::min<long long>(kPartThreads, (need + 31) / 32 * 32);
}

// The join: O and the LSE of every row from its own partials and the shared rows'.  A block
// takes eight query rows, its threads a row and 16 dims each: eight neighbouring threads read
// 128 contiguous bytes of a partial.  The decode kernel has ended before anything is read.
constexpr int kJoinThreads = 256, kJoinRows = 8, kJoinBatch = 4;

template <int kFormat>
__global__ void __launch_bounds__(kJoinThreads)
join_prefix_kernel(Problem p, Layout lay, PrefixLayout pl, char* __restrict__ ws) {
  constexpr int kUnits = kFormat == kPartF32 ? kPartUnitsF32 : kPartUnits;
  const PrefixEntry* entries = reinterpret_cast<const PrefixEntry*>(ws + pl.entries);
  const uint4* part_o = reinterpret_cast<const uint4*>(ws + lay.part_o);
  const float* part_lse = reinterpret_cast<const float*>(ws + lay.part_lse);
  const int t = threadIdx.x >> 3, r = blockIdx.x * kJoinRows + (threadIdx.x & 7);
  ptx::pdl_wait();
  const int n_entries = reinterpret_cast<const int*>(ws)[kHdrNumCombine];
  for (int i = blockIdx.y; i < n_entries; i += gridDim.y) {
    const PrefixEntry e = entries[i];
    if (r >= e.rows) continue;
    // (a request starts at a multiple of 16 rows of its group: eight rows share their slots)
    const int at = e.off + r, second = at >= lay.rows_per_group ? 1 : 0;
    const int pr = at - second * lay.rows_per_group;
    const int n_pre = second ? e.n_pre[1] : e.n_pre[0], pre = second ? e.pre[1] : e.pre[0];
    const int n = n_pre + e.n_own;
    float m = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
      uint4 x[kJoinBatch][kUnits];
      float l[kJoinBatch];
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        const int k = k0 + u;
        l[u] = -INFINITY;
#pragma unroll
        for (int v = 0; v < kUnits; ++v) x[u][v] = make_uint4(0, 0, 0, 0);
        if (k < n) {
          const size_t slot = (size_t)(k < n_pre ? pre + k : e.own + k - n_pre);
          const int row = k < n_pre ? pr : r;
#pragma unroll
          for (int v = 0; v < kUnits; ++v)
            x[u][v] = part_o[kFormat == kPartF32 ? part_unit_f32(slot, lay.rows_per_group, t, v, row)
                                                 : part_unit(slot, lay.rows_per_group, t, v, row)];
          l[u] = part_lse[slot * lay.rows_per_group + row];
        }
      }
      float m_new = m;
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) m_new = fmaxf(m_new, l[u]);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float f = expf(m - ref);
      sum *= f;
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[k] *= f;
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        const float w = expf(l[u] - ref);
        sum += w;
#pragma unroll
        for (int v = 0; v < kUnits; ++v) {
          const uint32_t word[4] = {x[u][v].x, x[u][v].y, x[u][v].z, x[u][v].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kFormat == kPartF32) {
              acc[4 * v + k] += w * __uint_as_float(word[k]);
            } else {
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&word[k]));
              acc[8 * v + 2 * k] += w * h.x;
              acc[8 * v + 2 * k + 1] += w * h.y;
            }
          }
        }
      }
      m = m_new;
    }
    const bool any = sum != 0.f;  // (a NaN is no empty sum)
    float s2 = any ? run_bmm2(p) / sum : 0.f;
    if constexpr (kFormat == kPartF16) s2 *= 1.f / (1 << part_shift(p.kv_dtype));
    __nv_bfloat162 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = __floats2bfloat162_rn(acc[2 * k] * s2, acc[2 * k + 1] * s2);
    const size_t row = (size_t)e.row0 + r;
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * kVDim + 16 * t);
    dst[0] = *reinterpret_cast<const uint4*>(o);
    dst[1] = *reinterpret_cast<const uint4*>(o + 4);
    if (p.return_lse && t == 0) p.lse[row] = any ? (m == -INFINITY ? 0.f : m) + logf(sum) : -INFINITY;
  }
}

cudaError_t prefix_setup() {
  return cudaFuncSetAttribute(partition_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kPartitionSmemMax);
}

cudaError_t launch_partition_prefix(const Problem& p, const PrefixArgs& pa, const Layout& lay, const PrefixLayout& pl,
                                    void* ws, cudaStream_t stream) {
  const int threads = partition_prefix_threads(p, pa, lay);
  partition_prefix_kernel<<<1, threads, pl.scratch_in_smem ? pl.scratch_bytes : 0, stream>>>(
      p, pa, lay, pl, static_cast<char*>(ws));
  return cudaGetLastError();
}

cudaError_t launch_join_prefix(const Problem& p, const Layout& lay, const PrefixLayout& pl, void* ws, int sm_count,
                               cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((lay.rows_per_group + kJoinRows - 1) / kJoinRows, std::min(pl.max_entries, 4 * sm_count), 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = p.kv_dtype == kKvFp8 || p.kv_dtype == kKvFp4 ? join_prefix_kernel<kPartF16> : join_prefix_kernel<kPartF32>;
  return cudaLaunchKernelEx(&cfg, kernel, p, lay, pl, static_cast<char*>(ws));
}

}  // namespace mla
