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
// where the call's estimate falls by prefix_gain tiles: the largest row group where none needs to
// be cut, else an even share and the join (kCutTiles).  So a few beams over a short prompt stay
// apart.
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_common.cuh"
#include "mla_fp4.cuh"
#include "mla_prefix.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

constexpr int kPartThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;

// By request: tokens, first token, rows, prefix group (-1: on its own), first token in its
// owner, first row group of its owner, own tiles and own segments of the requests before it.  By
// prefix group: first and last + 1 request, tokens (0: not shared), shared tiles, and whether they
// are widened.  By row group: start unit and place in a list, and the requests of its first and last
// token.
struct PrefixScratch {
  int *q, *qs, *len, *group, *tok, *base, *tiles, *count;  // (tiles and count: of all before the end, too)
  int *lo, *hi, *tokens, *shared, *wide;
  int *start, *place, *first, *last;
  __device__ PrefixScratch(char* at, int batch, int groups, int row_groups) {
    q = reinterpret_cast<int*>(at);
    qs = q + batch;
    len = qs + batch;
    group = len + batch;
    tok = group + batch;
    base = tok + batch;
    tiles = base + batch;
    count = tiles + batch + 1;
    lo = count + batch + 1;
    hi = lo + groups;
    tokens = hi + groups;
    shared = tokens + groups;
    wide = shared + groups;
    start = wide + groups;
    place = start + row_groups + 1;
    first = place + row_groups + 1;
    last = first + row_groups;
  }
};

struct PrefixShared {
  int w_scan[3][32], status, most, alone, alone_most, alone_count, any, any_wide, total;
  int bound[kPrefixWorkers + 1];
  unsigned cut[8], first[8];
};

__device__ __forceinline__ int scan_up(int v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// Last index in [0, n) whose value is at most x (values ascending, the first at most x).
__device__ __forceinline__ int last_upto(const int* v, int n, int x) {
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

// Sums of up to three values over all threads before this one, and over all (two barriers).
template <int kN>
__device__ __forceinline__ void block_scan(PrefixShared& sh, int (&v)[kN], int (&before)[kN], int (&total)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  int in[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    in[i] = scan_up(v[i], lane);
    if (lane == 31) sh.w_scan[i][warp] = in[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int w = scan_up(lane < n_warps ? sh.w_scan[i][lane] : 0, lane);
    const int up = __shfl_sync(kAll, w, warp == 0 ? 0 : warp - 1);
    before[i] = (warp == 0 ? 0 : up) + in[i] - v[i];
    total[i] = __shfl_sync(kAll, w, 31);
  }
  __syncthreads();
}

// The time of a list of row groups, in tiles.
__device__ __forceinline__ int list_estimate(int total, int most, int count, int n) {
  return partition_uncut(true, count, n, most, total) ? most : total / n + (int)kCutTiles;
}

}  // namespace

// kWide: plans that widen (a kernel of its own: the others' calls are 1 us shorter without).
template <bool kWide>
__global__ void __launch_bounds__(kPartThreads, 1)
partition_prefix_kernel(Problem p, PrefixArgs pa, Layout lay, PrefixLayout pl, char* __restrict__ ws) {
  extern __shared__ __align__(16) unsigned char prefix_smem[];
  __shared__ PrefixShared sh;
  ptx::pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int B = p.batch, G = pa.groups, H = p.num_heads, n = lay.n_workers;
  // tokens of a row group: 128 / H, a power of two (H is 16, 32, 64 or 128)
  const int per_shift = H == 16 ? 3 : H == 32 ? 2 : H == 64 ? 1 : 0, per = 1 << per_shift;
  const int c0 = prefix_overhead(p.kv_dtype);
  int* hdr = reinterpret_cast<int*>(ws);
  WorkItem* items = reinterpret_cast<WorkItem*>(ws + lay.items);
  int* worker_begin = reinterpret_cast<int*>(ws + lay.worker_ranges);
  PrefixEntry* entries = reinterpret_cast<PrefixEntry*>(ws + pl.entries);
  PrefixSegment* segments = reinterpret_cast<PrefixSegment*>(ws + pl.segments);
  const PrefixScratch s(pl.scratch_in_smem ? reinterpret_cast<char*>(prefix_smem) : ws + pl.scratch, B, G,
                        lay.max_groups);
  auto tiles_of = [](int rows) { return (max(rows, 0) + kKvTile - 1) / kKvTile; };
  auto groups_of = [&](int tokens) { return (tokens + per - 1) >> per_shift; };
  if (tid == 0) {
    sh.status = sh.alone = sh.alone_most = sh.alone_count = sh.any = sh.any_wide = 0;
  }
  // a warp's first prefix group, read beside the lengths
  const int each = B / G;
  int g_lo = 0, g_hi = 0, g_len = 0;
  if (warp < G) {
    g_lo = pa.indptr ? pa.indptr[warp] : warp * each;
    g_hi = pa.indptr ? pa.indptr[warp + 1] : g_lo + each;
    g_len = pa.lens[warp];
  }
  __syncthreads();

  // 1. Requests: lengths, clamped and flagged as by the other partitioners.
  int status = 0, bad = 0;
  {
    int total = 0, most = 0, count = 0;
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
        total += groups_of(q) * (c0 + tiles_of(L));
      }
    }
    total = (int)__reduce_add_sync(kAll, (unsigned)total);
    count = (int)__reduce_add_sync(kAll, (unsigned)count);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0 && count > 0) {
      atomicAdd(&sh.alone, total);
      atomicAdd(&sh.alone_count, count);
      atomicMax(&sh.alone_most, most);
    }
    for (int g = warp; g < G; g += n_warps) {
      const int lo = g == warp ? g_lo : pa.indptr ? pa.indptr[g] : 0, hi = g == warp ? g_hi : pa.indptr ? pa.indptr[g + 1] : 0;
      if (lo < 0 || hi < lo || hi > B) bad = 1;
    }
  }
  bad = __syncthreads_or(bad);  // (offsets that are none: nothing is shared)
  if (bad) status |= kStatusPrefix;

  // 2. Prefix groups: a warp each.
  for (int g = warp; g < G; g += n_warps) {
    const int lo = bad ? 0 : g == warp ? g_lo : pa.indptr ? pa.indptr[g] : g * each;
    const int hi = bad ? 0 : g == warp ? g_hi : pa.indptr ? pa.indptr[g + 1] : lo + each;
    const int len = g == warp ? g_len : pa.lens[g];
    int rows = INT_MAX, apart = 0;
    for (int b = lo + lane; b < hi; b += 32) {
      if (s.len[b] > 0 && s.q[b] > 0) rows = min(rows, p.causal ? s.len[b] - s.q[b] + 1 : s.len[b]);
      // (the group's query rows have to follow on one another)
      if (b + 1 < hi && s.qs[b + 1] != s.qs[b] + s.q[b]) apart = 1;
    }
    rows = __reduce_min_sync(kAll, rows);
    apart = (int)__reduce_or_sync(kAll, (unsigned)apart);
    if (len < 0) status |= kStatusPrefix;
    const int T = apart || rows == INT_MAX ? 0 : max(0, min(len, rows)) / kKvTile;
    const int tokens = hi > lo && T > 0 ? s.qs[hi - 1] + s.q[hi - 1] - s.qs[lo] : 0;
    // fewer tiles and overheads together than each on its own?
    int saved = 0;
    if (T > 0) {
      for (int b = lo + lane; b < hi; b += 32) {
        const int q = s.q[b], L = s.len[b], tok = s.qs[b] - s.qs[lo];
        if (q <= 0 || L <= 0) continue;
        const int touched = ((tok + q - 1) >> per_shift) - (tok >> per_shift) + 1;
        saved += groups_of(q) * (c0 + tiles_of(L)) - touched * tiles_of(L - T * kKvTile);
      }
      saved = (int)__reduce_add_sync(kAll, (unsigned)saved) - groups_of(tokens) * c0;
    }
    const bool wide = kWide && groups_of(tokens) >= kWideRowGroups;
    saved -= groups_of(tokens) * (wide ? min(T, (kWideOverhead + T) * kWideTenths / 10) : T);
    const bool on = T > 0 && saved > 0;
    if (lane == 0) {
      s.lo[g] = lo;
      s.hi[g] = hi;
      s.tokens[g] = on ? tokens : 0;
      s.shared[g] = T;
      s.wide[g] = on && wide;
      if (on) atomicOr(&sh.any, 1);
      if (on && wide) atomicOr(&sh.any_wide, 1);
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
  auto shared_tiles = [&](int b) { return s.group[b] >= 0 ? s.shared[s.group[b]] : 0; };
  auto first_request = [&](int b) { return s.group[b] >= 0 ? s.lo[s.group[b]] : b; };  // of b's owner
  // first of the widened tiles of b's owner, -1: none (before they are placed: 0)
  bool widens = false;
  auto wide_base = [&](int b) { return kWide && widens && s.group[b] >= 0 ? s.wide[s.group[b]] - 1 : -1; };
  // cost of row group r in a list, 0: it is not in it
  auto units = [&](int list, int r) {
    const int b = s.first[r], wide = wide_base(b);
    if (list == 1) return wide >= 0 ? kWideOverhead + shared_tiles(b) : 0;
    const int t = (wide < 0 ? shared_tiles(b) : 0) + s.tiles[s.last[r] + 1] - s.tiles[b];
    return t > 0 ? c0 + t : 0;
  };
  // start units of a list's row groups, and each one's place among them
  int W = 0, members = 0;
  auto scan_list = [&](int list) {
    if (tid == 0) sh.most = sh.total = 0;
    if (tid < 8) sh.cut[tid] = sh.first[tid] = 0;
    W = members = 0;
    __syncthreads();
    for (int at = 0; at < n_rg; at += blockDim.x) {
      const int r = at + tid;
      int v[2] = {r < n_rg ? units(list, r) : 0, 0}, before[2], total[2];
      v[1] = v[0] > 0 ? 1 : 0;
      const int most = __reduce_max_sync(kAll, v[0]);
      if (lane == 0 && most > 0) atomicMax(&sh.most, most);
      block_scan(sh, v, before, total);
      if (r < n_rg) {
        s.start[r] = W + before[0];
        s.place[r] = members + before[1];
      }
      W += total[0];
      members += total[1];
    }
    if (tid == 0) {
      s.start[n_rg] = W;
      s.place[n_rg] = members;
    }
    __syncthreads();
  };
  for (int pass = 0; pass < 2; ++pass) {
    int rg = 0, tiles = 0, count = 0;
    for (int at = 0; at < B; at += blockDim.x) {
      const int b = at + tid;
      int v[3] = {0, 0, 0}, before[3], total[3];
      if (b < B) {
        const int g = s.group[b], q = s.q[b], L = s.len[b];
        if (g >= 0) v[0] = b == s.lo[g] ? groups_of(s.tokens[g]) : 0;
        else v[0] = q > 0 && L > 0 ? groups_of(q) : 0;
        v[1] = q > 0 ? tiles_of(L - shared_tiles(b) * kKvTile) : 0;
        v[2] = v[1] > 0 ? 1 : 0;
      }
      block_scan(sh, v, before, total);
      if (b < B) {
        s.base[b] = rg + before[0];
        s.tiles[b] = tiles + before[1];
        s.count[b] = count + before[2];
      }
      rg += total[0];
      tiles += total[1];
      count += total[2];
    }
    if (tid == 0) {
      s.tiles[B] = tiles;
      s.count[B] = count;
    }
    n_rg = rg;
    // (malformed offsets may let requests overlap: more row groups than the plan has room for)
    room = n_rg <= lay.max_groups;
    if (!room) n_rg = 0;
    __syncthreads();
    // the requests of each row group's first and last token
    if (n_rg > 0)
      for (int b = tid; b < B; b += blockDim.x) {
        const int g = s.group[b], q = s.q[b];
        if (q <= 0 || (g < 0 && s.len[b] <= 0)) continue;
        const int tok = s.tok[b], tokens = g >= 0 ? s.tokens[g] : q, base = s.base[first_request(b)];
        for (int k = (tok + per - 1) >> per_shift; k << per_shift < tok + q; ++k) s.first[base + k] = b;
        for (int k = tok >> per_shift; k <= (tok + q - 1) >> per_shift; ++k)
          if (min((k + 1) << per_shift, tokens) <= tok + q) s.last[base + k] = b;
      }
    __syncthreads();
    scan_list(0);
    if (pass == 1 || !sh.any || !room) break;
    const int alone = list_estimate(sh.alone, sh.alone_most, sh.alone_count, n);
    const int shared = list_estimate(W, sh.most, members, n);
    if (kWide && sh.any_wide) {  // both lists' units, the second one's first tiles, and the copy
      widens = true;
      int other = 0;
      for (int r = tid; r < n_rg; r += blockDim.x) other += units(0, r) + units(1, r) * kWideTenths / 10;
      for (int g = tid; g < G; g += blockDim.x) other += s.wide[g] ? s.shared[g] * n / kWideCopy : 0;
      other = (int)__reduce_add_sync(kAll, (unsigned)other);
      if (lane == 0) atomicAdd(&sh.total, other);
      __syncthreads();
      widens = sh.total / n + kWideFixed < min(alone, shared);
      __syncthreads();  // (every thread has read the sum before a scan clears it)
      if (widens) {
        scan_list(0);
        break;
      }
    }
    if (shared + prefix_gain(p.kv_dtype) <= alone) break;
    __syncthreads();
    for (int b = tid; b < B; b += blockDim.x) {
      s.group[b] = -1;
      s.tok[b] = 0;
    }
    __syncthreads();
  }

  // the groups' widened rows, one after another
  if constexpr (kWide) {
    PrefixWide* of = reinterpret_cast<PrefixWide*>(ws + pl.wide_groups);
    int all = 0;
    for (int at = 0; at < G; at += blockDim.x) {
      const int g = at + tid;
      int v[1] = {widens && g < G && s.wide[g] ? s.shared[g] : 0}, before[1], total[1];
      block_scan(sh, v, before, total);
      if (g < G) {
        int b = s.lo[g];
        while (v[0] > 0 && b + 1 < s.hi[g] && (s.len[b] <= 0 || s.q[b] <= 0)) ++b;
        of[g] = PrefixWide{all + before[0], v[0], b, 0};
        if (widens) s.wide[g] = v[0] > 0 ? 1 + all + before[0] : 0;
      }
      all += total[0];
    }
    if (tid == 0) of[G] = PrefixWide{all, 0, 0, 0};
    __syncthreads();
  }

  // 4. The lists: row groups and what they walk outside widened rows, and these.
  int n_items = 0;
  bool fits = room;
  auto owner_tokens = [&](int b) { return s.group[b] >= 0 ? s.tokens[s.group[b]] : s.q[b]; };
  for (int list = 0; list < (kWide ? 2 : 1); ++list) {
    const int over = list ? kWideOverhead : c0;
    WorkItem* to = list ? reinterpret_cast<WorkItem*>(ws + pl.wide_items) : items;
    int* ranges = list ? reinterpret_cast<int*>(ws + pl.wide_ranges) : worker_begin;
    if (list == 1) scan_list(1);  // (the first one's is there)
    const int n_eff = max(1, min(n, W / (int)kMinUnits));
    const bool uncut = partition_uncut(true, members, n, sh.most, W);
    // worker boundaries, and which of them cut a row group (past its overhead)
    const int quot = W / n_eff, rest = W % n_eff;
    if (uncut) {  // worker w's range starts where row group w of the list does
      for (int r = tid; r < n_rg; r += blockDim.x)
        if (s.place[r + 1] > s.place[r]) sh.bound[s.place[r]] = s.start[r];
      for (int w = members + tid; w <= n; w += blockDim.x) sh.bound[w] = W;
    } else {
      for (int w = tid; w <= n; w += blockDim.x) sh.bound[w] = w >= n_eff ? W : w * quot + w * rest / n_eff;
    }
    __syncthreads();
    // (of row groups that start at the same unit the last is the one that has units)
    for (int w = tid; w <= n; w += blockDim.x) {
      const int at = sh.bound[w];
      if (w == 0 || at >= W) continue;
      const int from = s.start[last_upto(s.start, n_rg, at)] + over;  // unit of the row group's first tile
      if (at <= from) continue;
      atomicOr(reinterpret_cast<int*>(&sh.cut[w >> 5]), (int)(1u << (w & 31)));
      if (sh.bound[w - 1] <= from) atomicOr(reinterpret_cast<int*>(&sh.first[w >> 5]), (int)(1u << (w & 31)));
    }
    __syncthreads();
    const int n_list = members + bits_under(sh.cut, 255);
    // a plan that widens has a slot for every item, another one for those of cut row groups
    const bool enough = n_list <= lay.max_items &&
                        (kWide || n_list - members + bits_under(sh.first, 255) <= lay.max_partials);
    fits = fits && enough;
    if (list == 0) n_items = n_list;
    auto emit = [&](int at, int rg, int t0, int t1, int slot) {
      const int b = s.first[rg], o = first_request(b), shared = shared_tiles(b), wide = wide_base(b);
      WorkItem it;
      it.b = o;
      it.g = rg - s.base[o];
      it.kv_begin = t0 * kKvTile;
      it.kv_end = t1 * kKvTile;
      it.slot = slot;
      it.q_len = owner_tokens(b);
      it.seq_len = list ? 1 : (shared > 0 && wide < 0 ? 1 : 0) + s.count[s.last[rg] + 1] - s.count[b];
      it.q_start = s.qs[o];
      it.comb = rg;
      it.mask_base = 0;
      to[at] = it;
    };
    if (fits) {
      for (int rg = tid; rg < n_rg; rg += blockDim.x) {
        const bool member = s.place[rg + 1] > s.place[rg];
        const int from = s.start[rg] + over, end = s.start[rg + 1];
        const int b = s.first[rg], o = first_request(b), k = rg - s.base[o], T = shared_tiles(b), wide = wide_base(b);
        PrefixEntry* e = entries + rg;
        if (list == 0) {
          e->row0 = ((long long)s.qs[o] + (k << per_shift)) * H;
          e->rows = e->count[0] = e->count[1] = 0;
        }
        if (!member) continue;
        const int pb = sh.bound[0] > from ? 0 : last_upto(sh.bound, n + 1, from) + 1;  // boundaries up to the first tile
        int last = pb;  // past the row group's last cut
        while (last < n && bit_at(sh.cut, last) && sh.bound[last] < end) ++last;
        const bool split = last > pb, partial = split || wide >= 0;
        const int before = bits_under(sh.cut, pb), at = s.place[rg] + before;
        const int slot = kWide ? list * lay.max_items + at : before + bits_under(sh.first, pb);
        emit(at, rg, 0, (split ? sh.bound[pb] : end) - from, partial ? slot : -1);
        if (partial) {
          e->rows = min(per, owner_tokens(b) - (k << per_shift)) * H;
          e->slot[list] = slot;
          e->count[list] = 1 + last - pb;
        }
        if (list == 1) {
          reinterpret_cast<PrefixSegment*>(ws + pl.wide_segments)[(size_t)rg * kPrefixSegments] =
              PrefixSegment{0, 0, wide * kKvTile, (wide + T) * kKvTile, 0, kPrefixRows, kPrefixNoMask, 0};
        } else if (T > 0 && wide < 0) {
          int src = o;  // the owner's first request that has rows: its table is read
          while (src + 1 < s.hi[s.group[b]] && (s.len[src] <= 0 || s.q[src] <= 0)) ++src;
          segments[(size_t)rg * kPrefixSegments] = PrefixSegment{0, src, 0, T * kKvTile, 0, kPrefixRows, kPrefixNoMask, 0};
        }
      }
      // each request's own rows, a segment in every row group that it has query rows in
      if (list == 0)
        for (int b = tid; b < B; b += blockDim.x) {
          const int q = s.q[b], tok = s.tok[b], T = shared_tiles(b), L = s.len[b], in_list = wide_base(b) < 0 ? T : 0;
          if (q <= 0 || L <= T * kKvTile) continue;
          const int base = s.base[first_request(b)];
          for (int k = tok >> per_shift; k <= (tok + q - 1) >> per_shift; ++k) {
            const int f = s.first[base + k], first = k << per_shift, z = (in_list > 0 ? 1 : 0) + s.count[b] - s.count[f];
            if (z >= kPrefixSegments) continue;  // (never)
            segments[(size_t)(base + k) * kPrefixSegments + z] =
                PrefixSegment{in_list + s.tiles[b] - s.tiles[f], b, T * kKvTile, L, max(0, tok - first) * H,
                              min(per, tok + q - first) * H, p.causal ? L - q - tok : kPrefixNoMask, 0};
          }
        }
      for (int w = tid; w <= n; w += blockDim.x) {
        if (sh.bound[w] >= W) {
          ranges[w] = n_list;
          continue;
        }
        const int rg = last_upto(s.start, n_rg, sh.bound[w]);
        const bool cuts = bit_at(sh.cut, w);
        const int rank = bits_under(sh.cut, w), at = s.place[rg] + rank;
        // (a boundary inside a row group's overhead, or at its start, leaves the row group whole)
        ranges[w] = at + (cuts ? 1 : 0);
        if (!cuts) continue;
        const int from = s.start[rg] + over, tiles = s.start[rg + 1] - from;
        emit(at + 1, rg, sh.bound[w] - from, w + 1 <= n ? min(tiles, sh.bound[w + 1] - from) : tiles,
             kWide ? list * lay.max_items + at + 1 : rank + bits_under(sh.first, w + 1));
      }
    } else {
      for (int w = tid; w <= n; w += blockDim.x) worker_begin[w] = ranges[w] = 0;
    }
    __syncthreads();
  }
  if (tid == 0) {
    hdr[kHdrStatus] = fits ? sh.status : sh.status | kStatusCapacity;
    hdr[kHdrNumItems] = fits ? n_items : 0;
    hdr[kHdrWorkCounter] = 0;
    hdr[kHdrNumCombine] = fits ? n_rg : 0;
    hdr[kHdrChunkTiles] = 0;
    hdr[kHdrCombineCounter] = 0;
  }
}

// A thread for each request, worker boundary and row group, a warp for each prefix group.
inline int partition_prefix_threads(const Problem& p, const PrefixArgs& pa, const Layout& lay) {
  const long long need = std::max(std::max((long long)p.batch, std::min(256LL, 32LL * pa.groups)),
                                  std::max((long long)lay.n_workers + 1, (long long)lay.max_groups));
  return (int)std::min<long long>(kPartThreads, (need + 31) / 32 * 32);
}

// The join: O and the LSE of the rows of cut row groups from their partials.  A block takes eight
// query rows, its threads a row and 16 dims each: eight neighbouring threads read 128
// contiguous bytes of a partial.  What bounds it is the partials' bytes: a partial of a row
// that sees none of its tiles has an LSE of -inf and no O, and is not read.  The decode
// kernel has ended before a partial is.
constexpr int kJoinThreads = 256, kJoinRows = 8, kJoinBatch = 4;

__device__ __forceinline__ int slot_of(const PrefixEntry& e, int k) {
  return k < e.count[0] ? e.slot[0] + k : e.slot[1] + k - e.count[0];
}

// kScaled: over bf16 (see prefix_scale_offset).
template <bool kScaled>
__global__ void __launch_bounds__(kJoinThreads)
join_prefix_kernel(Problem p, Layout lay, PrefixLayout pl, char* __restrict__ ws) {
  const PrefixEntry* entries = reinterpret_cast<const PrefixEntry*>(ws + pl.entries);
  const uint4* part_o = reinterpret_cast<const uint4*>(ws + lay.part_o);
  const float* part_lse = reinterpret_cast<const float*>(ws + lay.part_lse);
  const signed char* part_scale = reinterpret_cast<const signed char*>(ws + prefix_scale_offset(lay));
  const int t = threadIdx.x >> 3, r = blockIdx.x * kJoinRows + (threadIdx.x & 7);
  // (before the entries, too: a grid sees what others wrote once it has waited itself)
  ptx::pdl_wait();
  const int n_entries = reinterpret_cast<const int*>(ws)[kHdrNumCombine];
  PrefixEntry e = {};
  if (blockIdx.y < n_entries) e = entries[blockIdx.y];
  for (int i = blockIdx.y; i < n_entries; i += gridDim.y) {
    if (i != blockIdx.y) e = entries[i];
    if (r >= e.rows) continue;
    float m = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    const int count = e.count[0] + e.count[1];
    for (int k0 = 0; k0 < count; k0 += kJoinBatch) {
      uint4 x[kJoinBatch][2];
      float l[kJoinBatch];
      int down[kJoinBatch];
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u)
        l[u] = k0 + u < count ? part_lse[(size_t)slot_of(e, k0 + u) * kPrefixRows + r] : -INFINITY;
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
        down[u] = kScaled ? 0 : part_shift(p.kv_dtype);
        if (l[u] != -INFINITY) {
          const size_t slot = slot_of(e, k0 + u);
          x[u][0] = part_o[part_unit(slot, kPrefixRows, t, 0, r)];
          x[u][1] = part_o[part_unit(slot, kPrefixRows, t, 1, r)];
          if constexpr (kScaled) down[u] = part_scale[(slot * 32 + t) * kPrefixRows + r];
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
        float w = expf(l[u] - ref);  // (0 where there is no partial)
        sum += w;
        w *= __uint_as_float((uint32_t)(127 - down[u]) << 23);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t word[4] = {x[u][v].x, x[u][v].y, x[u][v].z, x[u][v].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&word[k]));
            acc[8 * v + 2 * k] += w * h.x;
            acc[8 * v + 2 * k + 1] += w * h.y;
          }
        }
      }
      m = m_new;
    }
    const bool any = sum != 0.f;  // (a NaN is no empty sum)
    const float s2 = any ? run_bmm2(p) / sum : 0.f;
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
  const cudaError_t e = cudaFuncSetAttribute(partition_prefix_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kPartitionSmemMax);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(partition_prefix_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kPartitionSmemMax);
}

cudaError_t launch_partition_prefix(const Problem& p, const PrefixArgs& pa, const Layout& lay, const PrefixLayout& pl,
                                    void* ws, cudaStream_t stream) {
  const int threads = partition_prefix_threads(p, pa, lay);
  auto kernel = pl.wide_tiles > 0 ? partition_prefix_kernel<true> : partition_prefix_kernel<false>;
  kernel<<<1, threads, pl.scratch_in_smem ? pl.scratch_bytes : 0, stream>>>(p, pa, lay, pl, static_cast<char*>(ws));
  return cudaGetLastError();
}

// The shared rows of groups that are widened, once, to f16 (exact).  A block takes a tile of 64
// rows, four at a time, a thread the same eight dims of every fourth: reads and writes are
// contiguous across a warp, and eight rows are on their way at once.  What bounds it is the
// bytes: 65536 rows of 4 bits, 97 MB read and written.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t h;
  asm("{\n .reg .b16 lo;\n mov.b32 {lo, _}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(codes));
  return h;
}

constexpr int kWidenUnits = kQkDim / 8, kWidenRows = 4, kWidenThreads = kWidenRows * kWidenUnits;

template <bool kFp4>
__global__ void __launch_bounds__(kWidenThreads)
widen_prefix_kernel(Problem p, int groups, PrefixLayout pl, char* __restrict__ ws) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const PrefixWide* of = reinterpret_cast<const PrefixWide*>(ws + pl.wide_groups);
  int* status = reinterpret_cast<int*>(ws) + kHdrStatus;
  const int total = min(of[groups].base, pl.wide_tiles), ps = p.page_size, shift = ps == 64 ? 6 : 5;
  const int u = threadIdx.x % kWidenUnits, r0 = threadIdx.x / kWidenUnits;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    int lo = 0, hi = groups;  // the last group whose tiles start at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (of[mid].base <= t) lo = mid; else hi = mid;
    }
    const int row0 = (t - of[lo].base) * kKvTile;
    const int* table = p.block_tables + (size_t)of[lo].b * p.max_pages;
    uint4* to = reinterpret_cast<uint4*>(ws + pl.wide_rows) + (size_t)t * kKvTile * kWidenUnits + u;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {  // 32 rows, of one page
      const int id = table[(row0 + 32 * half) >> shift], in0 = (32 * half & (ps - 1)) + r0;
      const bool on = id >= 0 && (long long)id < p.num_pages;
      if (!on && threadIdx.x == 0) atomicOr(status, kStatusPage);
      const unsigned char* page =
          static_cast<const unsigned char*>(p.kv_cache) + (on ? (size_t)id * ps * (kFp4 ? kFp4RowBytes : kQkDim) : 0);
      constexpr int kN = 32 / kWidenRows;
      uint32_t code[kN][2], scale[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int in = in0 + kWidenRows * k;
        code[k][0] = code[k][1] = scale[k] = 0;
        if (!on) continue;
        if constexpr (kFp4) {
          code[k][0] = reinterpret_cast<const uint32_t*>(page + in * kFp4CodeBytes)[u];
          scale[k] = page[(size_t)ps * kFp4CodeBytes + in * kFp4ScaleBytes + (u >> 1)];
        } else {
          const uint2 c = reinterpret_cast<const uint2*>(page + in * kQkDim)[u];
          code[k][0] = c.x;
          code[k][1] = c.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        uint32_t h[4];
        if constexpr (kFp4) {
          ptx::e2m1x8_to_f16x2(code[k][0], h);
          const uint32_t two = e4m3x2_to_f16x2(scale[k] | scale[k] << 8);
          const __half2 by = *reinterpret_cast<const __half2*>(&two);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), by);
            h[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = e4m3x2_to_f16x2(code[k][e >> 1] >> (16 * (e & 1)));
        }
        to[(32 * half + r0 + kWidenRows * k) * kWidenUnits] = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  }
}

cudaError_t launch_widen_prefix(const Problem& p, int groups, const PrefixLayout& pl, void* ws, int sm_count,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(pl.wide_tiles, 7 * sm_count), 1, 1);
  cfg.blockDim = dim3(kWidenThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.kv_dtype == kKvFp4 ? widen_prefix_kernel<true> : widen_prefix_kernel<false>, p, groups, pl,
                            static_cast<char*>(ws));
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
  auto kernel = p.kv_dtype == kKvFp8 || p.kv_dtype == kKvFp4 ? join_prefix_kernel<false> : join_prefix_kernel<true>;
  return cudaLaunchKernelEx(&cfg, kernel, p, lay, pl, static_cast<char*>(ws));
}

}  // namespace mla
