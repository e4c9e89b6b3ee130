// The work list and the join of a decode over shared prefixes (mla_prefix.cuh); the items
// run on mla_decode_pair.cu's kernel.
//
// Partition.  Owners of row groups are the prefix groups that are shared, and the other
// requests.  A prefix group of n tokens with P shared rows owns ceil(n H / 128) row groups, each of
// P / 64 tiles and the own tiles of the requests that it holds rows of; a request on its own
// ceil(q H / 128) row groups of all its tiles.  From the row groups' costs on it is
// mla_partition_pair.cu's way: start units by a scan, worker boundary p at unit floor(p W / n'),
// and with two bits a boundary the place of every item is a population count.
//
// A group's rows are shared where that costs fewer tiles, overheads included (the own tiles
// of a request that straddles one row group more count once more), and groups are shared at all
// where the call's estimate falls: the largest row group where none needs to be cut, else an even
// share and the join (kCutTiles).  So a few beams over a short prompt stay apart: each is
// done on a worker of its own while a common row group would be one worker's work.
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

// By request: tokens, first token, rows, prefix group (-1: on its own), first token in it.
// By prefix group: first and last + 1 request, tokens, shared tiles.  By owner: first row
// group.  By row group: start unit; cost.
struct PrefixScratch {
  long long* start;
  int *cost, *q, *qs, *len, *group, *tok, *lo, *hi, *tokens, *shared, *base;
  __device__ PrefixScratch(char* at, int batch, int groups, int row_groups) {
    start = reinterpret_cast<long long*>(at);
    cost = reinterpret_cast<int*>(at + align_up(sizeof(long long) * (size_t)(row_groups + 1), 16));
    q = cost + row_groups;
    qs = q + batch;
    len = qs + batch;
    group = len + batch;
    tok = group + batch;
    lo = tok + batch;
    hi = lo + groups;
    tokens = hi + groups;
    shared = tokens + groups;
    base = shared + groups;
  }
};

struct PrefixShared {
  long long w_cost[32], carry, alone;
  int w_count[32], count, status, most, alone_most, any;
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

// The time of a list of row groups, in tiles.
__device__ __forceinline__ long long list_estimate(long long total, long long most, long long count, int n) {
  return partition_uncut(true, count, n, most, total) ? most : total / n + kCutTiles;
}

}  // namespace

__global__ void __launch_bounds__(kPartThreads, 1)
partition_prefix_kernel(Problem p, PrefixArgs pa, Layout lay, PrefixLayout pl, char* __restrict__ ws) {
  extern __shared__ __align__(16) unsigned char prefix_smem[];
  __shared__ PrefixShared sh;
  ptx::pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int B = p.batch, G = pa.groups, H = p.num_heads, n = lay.n_workers;
  const int per = kPrefixRows / H;  // tokens of a row group (H is 16, 32, 64 or 128)
  const int c0 = prefix_overhead(p.kv_dtype);
  int* hdr = reinterpret_cast<int*>(ws);
  WorkItem* items = reinterpret_cast<WorkItem*>(ws + lay.items);
  int* worker_begin = reinterpret_cast<int*>(ws + lay.worker_ranges);
  PrefixEntry* entries = reinterpret_cast<PrefixEntry*>(ws + pl.entries);
  PrefixSegment* segments = reinterpret_cast<PrefixSegment*>(ws + pl.segments);
  const int owners = G + B;
  const PrefixScratch s(pl.scratch_in_smem ? reinterpret_cast<char*>(prefix_smem) : ws + pl.scratch, B, G,
                        lay.max_groups);
  auto tiles_of = [](int rows) { return (max(rows, 0) + kKvTile - 1) / kKvTile; };
  auto groups_of = [&](int tokens) { return (tokens + per - 1) / per; };
  if (tid == 0) {
    sh.alone = 0;
    sh.status = sh.alone_most = sh.any = 0;
    sh.count = 0;
  }
  __syncthreads();

  // 1. Requests: lengths, clamped and flagged as by the other partitioners.
  int status = 0;
  {
    long long total = 0;
    int most = 0, count = 0;
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
      s.tok[b] = 0;
      if (L > 0 && q > 0) {
        count += groups_of(q);
        most = max(most, c0 + tiles_of(L));
        total += (long long)groups_of(q) * (c0 + tiles_of(L));
      }
    }
    total = __shfl_sync(kAll, scan_up(total, lane), 31);
    count = (int)__reduce_add_sync(kAll, (unsigned)count);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) {
      atomicAdd(reinterpret_cast<unsigned long long*>(&sh.alone), (unsigned long long)total);
      atomicAdd(&sh.count, count);
      atomicMax(&sh.alone_most, most);
    }
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
  const int alone_count = sh.count;
  for (int g = warp; g < G; g += n_warps) {
    const int each = B / G;
    const int lo = bad ? 0 : pa.indptr ? pa.indptr[g] : g * each;
    const int hi = bad ? 0 : pa.indptr ? pa.indptr[g + 1] : lo + each;
    int rows = INT_MAX, apart = 0;
    for (int b = lo + lane; b < hi; b += 32) {
      if (s.len[b] > 0 && s.q[b] > 0) rows = min(rows, p.causal ? s.len[b] - s.q[b] + 1 : s.len[b]);
      // (the group's query rows have to follow on one another)
      if (b + 1 < hi && s.qs[b + 1] != s.qs[b] + s.q[b]) apart = 1;
    }
    rows = __reduce_min_sync(kAll, rows);
    apart = (int)__reduce_or_sync(kAll, (unsigned)apart);
    const int len = pa.lens[g];
    if (len < 0) status |= kStatusPrefix;
    const int T = apart || rows == INT_MAX ? 0 : max(0, min(len, rows)) / kKvTile;
    const int tokens = hi > lo && T > 0 ? s.qs[hi - 1] + s.q[hi - 1] - s.qs[lo] : 0;
    // fewer tiles and overheads together than each on its own?
    long long saved = 0;
    if (T > 0) {
      for (int b = lo + lane; b < hi; b += 32) {
        const int q = s.q[b], L = s.len[b], tok = s.qs[b] - s.qs[lo];
        if (q <= 0 || L <= 0) continue;
        const int touched = (tok + q - 1) / per - tok / per + 1;
        saved += (long long)groups_of(q) * (c0 + tiles_of(L)) - (long long)touched * tiles_of(L - T * kKvTile);
      }
      saved = __shfl_sync(kAll, scan_up(saved, lane), 31) - (long long)groups_of(tokens) * (c0 + T);
    }
    const bool on = T > 0 && saved > 0;
    if (lane == 0) {
      s.lo[g] = lo;
      s.hi[g] = hi;
      s.tokens[g] = on ? tokens : 0;
      s.shared[g] = T;
      if (on) sh.any = 1;
    }
    if (on)
      for (int b = lo + lane; b < hi; b += 32) {
        s.group[b] = g;
        s.tok[b] = s.qs[b] - s.qs[lo];
      }
  }
  if (status) atomicOr(&sh.status, status);
  __syncthreads();

  // 3. Row groups, their costs and start units; once more with every request on its own where
  // that is the shorter list.
  int n_rg = 0;
  bool room = true;
  auto owned = [&](int o) {  // row groups of an owner
    if (o < G) return groups_of(s.tokens[o]);
    const int b = o - G;
    return s.group[b] >= 0 || s.len[b] <= 0 || s.q[b] <= 0 ? 0 : groups_of(s.q[b]);
  };
  for (int pass = 0; pass < 2; ++pass) {
    if (tid == 0) {
      sh.count = 0;
      sh.most = 0;
      sh.carry = 0;
    }
    __syncthreads();
    for (int at = 0; at < owners; at += blockDim.x) {
      const int o = at + tid, c = o < owners ? owned(o) : 0;
      const int in = scan_up(c, lane);
      if (lane == 31) sh.w_count[warp] = in;
      __syncthreads();
      int before = sh.count;
      for (int w = 0; w < warp; ++w) before += sh.w_count[w];
      if (o < owners) s.base[o] = before + in - c;
      __syncthreads();
      if (tid == 0)
        for (int w = 0; w < n_warps; ++w) sh.count += sh.w_count[w];
      __syncthreads();
    }
    n_rg = sh.count;
    if (tid == 0) s.base[owners] = n_rg;
    // (malformed offsets may let requests overlap: more row groups than the plan has room for)
    room = n_rg <= lay.max_groups;
    if (!room) n_rg = 0;
    for (int r = tid; r < n_rg; r += blockDim.x) s.cost[r] = c0;
    __syncthreads();
    if (n_rg > 0) {
      for (int g = warp; g < G; g += n_warps)
        for (int k = lane; k < groups_of(s.tokens[g]); k += 32) atomicAdd(&s.cost[s.base[g] + k], s.shared[g]);
      for (int b = tid; b < B; b += blockDim.x) {
        const int g = s.group[b], q = s.q[b];
        if (q <= 0 || s.len[b] <= 0) continue;
        const int own = tiles_of(s.len[b] - (g >= 0 ? s.shared[g] * kKvTile : 0));
        const int first = s.base[g >= 0 ? g : G + b] + s.tok[b] / per, last = first - s.tok[b] / per + (s.tok[b] + q - 1) / per;
        if (own > 0)
          for (int r = first; r <= last; ++r) atomicAdd(&s.cost[r], own);
      }
    }
    __syncthreads();
    for (int at = 0; at < n_rg; at += blockDim.x) {
      const int r = at + tid, c = r < n_rg ? s.cost[r] : 0;
      const long long in = scan_up((long long)c, lane);
      const int most = __reduce_max_sync(kAll, c);
      if (lane == 31) {
        sh.w_cost[warp] = in;
        atomicMax(&sh.most, most);
      }
      __syncthreads();
      long long before = sh.carry;
      for (int w = 0; w < warp; ++w) before += sh.w_cost[w];
      if (r < n_rg) s.start[r] = before + in - c;
      __syncthreads();
      if (tid == 0)
        for (int w = 0; w < n_warps; ++w) sh.carry += sh.w_cost[w];
      __syncthreads();
    }
    if (pass == 1 || !sh.any || !room) break;
    if (list_estimate(sh.carry, sh.most, n_rg, n) <= list_estimate(sh.alone, sh.alone_most, alone_count, n)) break;
    __syncthreads();
    for (int b = tid; b < B; b += blockDim.x) {
      s.group[b] = -1;
      s.tok[b] = 0;
    }
    for (int g = tid; g < G; g += blockDim.x) s.tokens[g] = 0;
    __syncthreads();
  }
  const long long W = sh.carry;
  const int n_eff = (int)max(1LL, min((long long)n, W / kMinUnits));
  const bool uncut = partition_uncut(true, n_rg, n, sh.most, W);

  // 4. Worker boundaries, and which of them cut a row group (past its overhead).
  for (int w = tid; w <= n; w += blockDim.x) {
    if (uncut)
      sh.bound[w] = w < n_rg ? s.start[w] : W;
    else
      sh.bound[w] = w >= n_eff ? W : w * (W / n_eff) + w * (W % n_eff) / n_eff;
  }
  if (tid < 8) sh.cut[tid] = sh.first[tid] = 0;
  __syncthreads();
  auto group_at = [&](long long unit) { return last_upto(s.start, n_rg, unit); };
  for (int w = tid; w <= n; w += blockDim.x) {
    if (w == 0 || sh.bound[w] >= W) continue;
    const long long from = s.start[group_at(sh.bound[w])] + c0;  // unit of the row group's first tile
    if (sh.bound[w] <= from) continue;
    atomicOr(reinterpret_cast<int*>(&sh.cut[w >> 5]), (int)(1u << (w & 31)));
    if (sh.bound[w - 1] <= from) atomicOr(reinterpret_cast<int*>(&sh.first[w >> 5]), (int)(1u << (w & 31)));
  }
  __syncthreads();

  // 5. Items, segments, entries of the join, worker ranges.
  const int n_items = n_rg + bits_under(sh.cut, 255);
  const bool fits = room && n_items <= lay.max_items && n_items - n_rg + bits_under(sh.first, 255) <= lay.max_partials;
  auto emit = [&](int at, int rg, int owner, long long t0, long long t1, int slot) {
    WorkItem it;
    const int b = owner < G ? s.lo[owner] : owner - G;
    it.b = b;
    it.g = rg - s.base[owner];
    it.kv_begin = (int)t0 * kKvTile;
    it.kv_end = (int)t1 * kKvTile;
    it.slot = slot;
    it.q_len = owner < G ? s.tokens[owner] : s.q[b];
    it.seq_len = 0;
    it.q_start = s.qs[b];
    it.comb = rg;
    it.mask_base = 0;
    // the row group's segments (each of its items has their number)
    const int first = it.g * per, end = min(first + per, it.q_len);  // tokens
    const int T = owner < G ? s.shared[owner] : 0;
    int count = 0, tile = 0;
    PrefixSegment* seg = segments + (size_t)rg * kPrefixSegments;
    const bool write = t0 == 0;
    if (T > 0) {
      int src = b;  // the first request that has rows: its table is read
      while (src + 1 < s.hi[owner] && (s.len[src] <= 0 || s.q[src] <= 0)) ++src;
      if (write) seg[0] = PrefixSegment{0, src, 0, T * kKvTile, 0, kPrefixRows, kPrefixNoMask, 0};
      count = 1;
      tile = T;
    }
    const int stop = owner < G ? s.hi[owner] : b + 1;
    for (int r = owner < G ? b + last_upto(s.tok + b, stop - b, first) : b; r < stop && s.tok[r] < end; ++r) {
      const int own = tiles_of(s.len[r] - T * kKvTile), q = s.q[r];
      if (q <= 0 || own <= 0 || s.tok[r] + q <= first || count >= kPrefixSegments) continue;
      if (write)
        seg[count] = PrefixSegment{tile, r, T * kKvTile, s.len[r], max(0, s.tok[r] - first) * H,
                                   min(per, s.tok[r] + q - first) * H,
                                   p.causal ? s.len[r] - q - s.tok[r] : kPrefixNoMask, 0};
      ++count;
      tile += own;
    }
    it.seq_len = count;
    items[at] = it;
  };
  if (fits) {
    for (int rg = tid; rg < n_rg; rg += blockDim.x) {
      const int owner = last_upto(s.base, owners, rg);
      const long long from = s.start[rg] + c0, end = s.start[rg] + s.cost[rg];
      const int pb = sh.bound[0] > from ? 0 : last_upto(sh.bound, n + 1, from) + 1;  // boundaries up to the first tile
      int last = pb;  // past the row group's last cut
      while (last < n && bit_at(sh.cut, last) && sh.bound[last] < end) ++last;
      const bool split = last > pb;
      const int before = bits_under(sh.cut, pb), slot = before + bits_under(sh.first, pb);
      emit(rg + before, rg, owner, 0, split ? sh.bound[pb] - from : end - from, split ? slot : -1);
      PrefixEntry e = {};
      const int k = rg - s.base[owner], b = owner < G ? s.lo[owner] : owner - G;
      const int tokens = owner < G ? s.tokens[owner] : s.q[b];
      e.row0 = ((long long)s.qs[b] + (long long)k * per) * H;
      e.rows = split ? min(per, tokens - k * per) * H : 0;
      e.slot = slot;
      e.count = 1 + last - pb;
      entries[rg] = e;
    }
    for (int w = tid; w <= n; w += blockDim.x) {
      if (sh.bound[w] >= W) {
        worker_begin[w] = n_items;
        continue;
      }
      const int rg = group_at(sh.bound[w]);
      const bool cuts = bit_at(sh.cut, w);
      // (a boundary inside a row group's overhead, or at its start, leaves the row group whole)
      worker_begin[w] = rg + bits_under(sh.cut, w) + (cuts ? 1 : 0);
      if (!cuts) continue;
      const long long from = s.start[rg] + c0, tiles = s.cost[rg] - c0;
      const long long next = w + 1 <= n ? min(tiles, sh.bound[w + 1] - from) : tiles;
      const int rank = bits_under(sh.cut, w);
      emit(rg + 1 + rank, rg, last_upto(s.base, owners, rg), sh.bound[w] - from, next,
           rank + bits_under(sh.first, w + 1));
    }
  } else {
    for (int w = tid; w <= n; w += blockDim.x) worker_begin[w] = 0;
  }
  if (tid == 0) {
    hdr[kHdrStatus] = fits ? sh.status : sh.status | kStatusCapacity;
    hdr[kHdrNumItems] = fits ? n_items : 0;
    hdr[kHdrWorkCounter] = 0;
    hdr[kHdrNumCombine] = fits ? n_rg : 0;
    hdr[kHdrChunkTiles] = (int)min(W, 1LL << 30);
    hdr[kHdrCombineCounter] = 0;
  }
}

// A thread for each request, worker boundary and row group, a warp for each prefix group.
inline int partition_prefix_threads(const Problem& p, const PrefixArgs& pa, const Layout& lay) {
  const long long need = std::max(std::max((long long)p.batch, 32LL * pa.groups),
                                  std::max((long long)lay.n_workers + 1, (long long)lay.max_groups));
  return (int)std::min<long long>(kPartThreads, (need + 31) / 32 * 32);
}

// The join: O and the LSE of the rows of cut row groups from their partials.  A block takes eight
// query rows, its threads a row and 16 dims each: eight neighbouring threads read 128
// contiguous bytes of a partial.  A partial of a row that sees none of its tiles has an LSE of
// -inf, and no O.  The decode kernel has ended before anything is read.
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
    float m = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    for (int k0 = 0; k0 < e.count; k0 += kJoinBatch) {
      uint4 x[kJoinBatch][kUnits];
      float l[kJoinBatch];
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        l[u] = -INFINITY;
        if (k0 + u < e.count) l[u] = part_lse[(size_t)(e.slot + k0 + u) * kPrefixRows + r];
      }
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u)
#pragma unroll
        for (int v = 0; v < kUnits; ++v) {
          x[u][v] = make_uint4(0, 0, 0, 0);
          if (l[u] != -INFINITY)
            x[u][v] = part_o[kFormat == kPartF32 ? part_unit_f32(e.slot + k0 + u, kPrefixRows, t, v, r)
                                                 : part_unit(e.slot + k0 + u, kPrefixRows, t, v, r)];
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
  cfg.gridDim = dim3(kPrefixRows / kJoinRows, std::min(lay.max_groups, 4 * sm_count), 1);
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
