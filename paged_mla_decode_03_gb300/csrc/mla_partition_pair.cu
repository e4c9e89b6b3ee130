// The work list of plans on the MMAs across CTA pairs (mla_decode_pair.cu): the
// partition of mla_partition.cu, item for item, for up to kPairMax requests and row
// groups, with a thread for each request, row group and worker boundary.
//
// Every step that the block kernel takes by walking lists is here one thread's
// arithmetic or search, so that five barriers are left, and costs are 32-bit.
// Worker boundary p lies at unit B_p = floor(p W / n'); it cuts the group that starts
// at S <= B_p < S + c0 + T before its tile t = B_p - S - c0 if 0 < t < T.  With two
// bits a boundary, "cuts" (V) and "is its group's first cut" (F), the place of every
// item is a population count: group g's first item follows g groups' first items and
// the cuts before it, and boundary p's item the groups up to its own and the cuts
// before p.  Per call, against the block kernel: 64 requests x 128 heads, window 1024,
// bf16, 48.8 -> 43.1 us; the same over 1-8k rows of 4 bits 112 -> 104; 128 ragged requests,
// window, 86 -> 79; against the one-warp form: 8 x 2 x 64 heads 22.2 -> 20.5.
#include <algorithm>
#include <climits>

#include "mla_common.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

constexpr int kPairMax = 1024;        // requests, and row groups: one thread each
constexpr int kPairWorkers = 255;     // worker boundaries (and their bit words)
constexpr unsigned kWhole = 0xffffffffu;

struct PairShared {
  int q[kPairMax], qs[kPairMax], len[kPairMax], gbase[kPairMax];  // by request
  int start[kPairMax], req[kPairMax], k[kPairMax];                // by row group
  int bound[kPairWorkers + 1];
  unsigned cut[8], first[8];  // V and F
  int w_groups[32], w_min[32], w_max[32], w_tiles[32], w_cost[32], w_status[32], w_start[32];
};

__device__ __forceinline__ int scan32(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kWhole, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// First index in [0, n) whose value is above x, n if none (values ascending).
__device__ __forceinline__ int first_above(const int* v, int n, int x) {
  int lo = 0;
  while (lo < n) {
    const int mid = (lo + n) >> 1;
    if (v[mid] > x) n = mid; else lo = mid + 1;
  }
  return lo;
}
// Bits below p.
__device__ __forceinline__ int bits_below(const unsigned* words, int p) {
  int c = 0;
  for (int w = 0; w < (p >> 5); ++w) c += __popc(words[w]);
  return (p & 31) ? c + __popc(words[p >> 5] << (32 - (p & 31))) : c;
}
__device__ __forceinline__ bool bit(const unsigned* words, int p) { return (words[p >> 5] >> (p & 31)) & 1u; }

}  // namespace

__global__ void __launch_bounds__(kPairMax, 1)
partition_pair_kernel(Problem p, Layout lay, char* __restrict__ ws) {
  __shared__ PairShared sh;
  ptx::pdl_launch_dependents();  // (see partition_kernel)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  int* hdr = reinterpret_cast<int*>(ws);
  WorkItem* items = reinterpret_cast<WorkItem*>(ws + lay.items);
  CombineItem* comb = reinterpret_cast<CombineItem*>(ws + lay.combine);
  int* worker_begin = reinterpret_cast<int*>(ws + lay.worker_ranges);
  int* comb_done = reinterpret_cast<int*>(ws + lay.comb_done);
  const int B = p.batch, R = lay.rows_per_group, H = p.num_heads, n = lay.n_workers;
  const int c0 = (int)kOverheadTilesPair;
  auto kv_rows = [&](int L, int q) { return L - window_skip(p.window, p.sinks, p.causal, L, q); };
  auto tiles_of = [&](int L, int q) { return (kv_rows(L, q) + kKvTile - 1) / kKvTile; };

  // 1. A thread's request: lengths (clamped and flagged as in the block kernel), row groups.
  int status = 0, groups = 0, tiles = 0;
  if (tid < B) {
    int q, qs;
    int L = p.seq_lens[tid];
    if (p.packed) {
      int lo = p.qo_indptr[tid], hi = p.qo_indptr[tid + 1];
      const int tq = (int)p.total_q;
      if (lo < 0 || hi > tq || hi - lo < 1 || hi - lo > p.max_q) status |= kStatusQLen;
      lo = min(max(lo, 0), tq);
      hi = min(max(hi, lo), tq);
      q = min(hi - lo, p.max_q);
      qs = lo;
    } else {
      q = p.max_q;
      qs = tid * p.max_q;
    }
    if (L < 1 || L > p.max_seq_len) status |= kStatusSeqLen;
    L = min(max(L, 0), p.max_seq_len);
    if (p.causal && q > L) status |= kStatusCausal;
    groups = L > 0 ? (q * H + R - 1) / R : 0;
    tiles = tiles_of(L, q);
    sh.q[tid] = q;
    sh.qs[tid] = qs;
    sh.len[tid] = L;
  }
  const int in_warp = scan32(groups, lane);
  {
    const int mn = __reduce_min_sync(kWhole, groups > 0 ? groups : INT_MAX);
    const int mx = __reduce_max_sync(kWhole, groups);
    const int tl = __reduce_max_sync(kWhole, groups > 0 ? tiles : 0);
    const int cost = (int)__reduce_add_sync(kWhole, (unsigned)(groups * (c0 + tiles)));
    const int st = (int)__reduce_or_sync(kWhole, (unsigned)status);
    if (lane == 31) {
      sh.w_groups[warp] = in_warp;
      sh.w_min[warp] = mn;
      sh.w_max[warp] = mx;
      sh.w_tiles[warp] = tl;
      sh.w_cost[warp] = cost;
      sh.w_status[warp] = st;
    }
  }
  __syncthreads();
  const bool w_on = lane < n_warps;
  const int w_scan = scan32(w_on ? sh.w_groups[lane] : 0, lane);
  const int g_min = __reduce_min_sync(kWhole, w_on ? sh.w_min[lane] : INT_MAX);
  const int g_max = __reduce_max_sync(kWhole, w_on ? sh.w_max[lane] : 0);
  const int t_max = __reduce_max_sync(kWhole, w_on ? sh.w_tiles[lane] : 0);
  int W = (int)__reduce_add_sync(kWhole, w_on ? (unsigned)sh.w_cost[lane] : 0u);
  status = (int)__reduce_or_sync(kWhole, w_on ? (unsigned)sh.w_status[lane] : 0u);
  int n_groups = __shfl_sync(kWhole, w_scan, 31);
  {
    const int before = __shfl_sync(kWhole, w_scan, warp == 0 ? 0 : warp - 1);
    if (tid < B) sh.gbase[tid] = (warp == 0 ? 0 : before) + in_warp - groups;
  }
  if (n_groups > lay.max_groups) {  // (overlapping requests of a malformed qo_indptr)
    status |= kStatusCapacity;
    n_groups = 0;
    W = 0;
  }
  const int n_eff = max(1, min(n, W / (int)kMinUnits));
  const int lanes = (g_min == g_max && g_max >= 2 && n_eff / g_max >= 2) ? g_max : 1;
  const int per_lane = lanes > 1 ? n_groups / lanes : 0;  // requests that have groups
  const int nl = n_eff / lanes, WL = W / lanes;
  const bool uncut = partition_uncut(true, n_groups, n, c0 + t_max, W);
  __syncthreads();

  // 2. A thread's row group: its request, cost and start unit.
  int b = 0, k = 0, cost = 0;
  if (tid < n_groups) {
    const int idx = lanes > 1 ? tid % per_lane : tid;
    b = first_above(sh.gbase, B, lanes > 1 ? idx * lanes : tid) - 1;
    k = lanes > 1 ? tid / per_lane : tid - sh.gbase[b];
    cost = c0 + tiles_of(sh.len[b], sh.q[b]);
    sh.req[tid] = b;
    sh.k[tid] = k;
  }
  int start = scan32(cost, lane);
  if (lane == 31) sh.w_start[warp] = start;
  __syncthreads();
  {
    const int s = scan32(w_on ? sh.w_start[lane] : 0, lane);
    const int before = __shfl_sync(kWhole, s, warp == 0 ? 0 : warp - 1);
    start += (warp == 0 ? 0 : before) - cost;
  }
  if (tid < n_groups) sh.start[tid] = start;
  if (uncut) {  // worker p's range starts where group p does
    if (tid <= n) sh.bound[tid] = tid < n_groups ? start : W;
  } else if (tid <= n) {
    const int of = tid / nl, i = tid - of * nl;
    sh.bound[tid] = tid >= lanes * nl ? W : of * WL + i * (WL / nl) + i * (WL % nl) / nl;
  }
  __syncthreads();

  // 3. A thread's worker boundary: the group it falls into, and whether it cuts it.
  int g_of = 0, S = 0, T = 0, t = 0;
  bool cuts = false, leads = false;
  if (tid <= n && sh.bound[tid] < W) {
    const int at = sh.bound[tid];
    g_of = first_above(sh.start, n_groups, at) - 1;
    S = sh.start[g_of];
    T = (g_of + 1 < n_groups ? sh.start[g_of + 1] : W) - S - c0;
    t = at - S - c0;
    cuts = tid > 0 && t > 0;
    leads = cuts && sh.bound[tid - 1] - S - c0 <= 0;
  }
  {
    const unsigned v = __ballot_sync(kWhole, cuts), f = __ballot_sync(kWhole, leads);
    if (lane == 0 && warp < 8) {
      sh.cut[warp] = v;
      sh.first[warp] = f;
    }
  }
  for (int w = n_warps + tid; w < 8; w += blockDim.x) sh.cut[w] = sh.first[w] = 0;
  __syncthreads();

  // 4. Items, combine entries, worker ranges.
  const int n_items = n_groups + bits_below(sh.cut, 255), n_combine = bits_below(sh.first, 255);
  const bool fits = n_items <= lay.max_items && n_items - n_groups + n_combine <= lay.max_partials &&
                    n_combine <= lay.max_combine;  // (always, within the contract)
  auto emit = [&](int at, int g, int t0, int t1, int slot, int entry) {
    const int rb = sh.req[g], L = sh.len[rb], q = sh.q[rb];
    WorkItem it;
    it.b = rb;
    it.g = sh.k[g];
    it.kv_begin = t0 * kKvTile;
    it.kv_end = min(kv_rows(L, q), t1 * kKvTile);
    it.slot = slot;
    it.q_len = q;
    it.seq_len = L;
    it.q_start = sh.qs[rb];
    it.comb = entry;
    it.mask_base = L - q;
    items[at] = it;
  };
  if (fits && tid < n_groups) {
    const int pl = first_above(sh.bound, n + 1, start + c0);  // boundaries below pl: units up to the first tile
    const bool split = pl < n && bit(sh.cut, pl) && sh.bound[pl] < start + cost;
    const int before = bits_below(sh.cut, pl), entry = bits_below(sh.first, pl);
    emit(tid + before, tid, 0, split ? sh.bound[pl] - start - c0 : cost - c0, split ? before + entry : -1,
         split ? entry : -1);
  }
  if (fits && cuts) {
    const int rank = bits_below(sh.cut, tid), entry = bits_below(sh.first, tid + 1) - 1;
    const int next = tid + 1 <= n ? sh.bound[tid + 1] - S - c0 : T;
    emit(g_of + 1 + rank, g_of, t, min(next, T), rank + entry + 1, entry);
    if (leads) {
      int end = tid + 1;  // past the group's last cut
      while (end < n && bit(sh.cut, end) && !bit(sh.first, end)) ++end;
      const int rb = sh.req[g_of];
      CombineItem ci;
      ci.b = rb;
      ci.g = sh.k[g_of];
      ci.first_slot = rank + entry;
      ci.stride = 1;
      ci.n_chunks = 1 + end - tid;
      ci.q_len = sh.q[rb];
      ci.q_start = sh.qs[rb];
      ci.pad = 0;
      comb[entry] = ci;
    }
  }
  if (tid <= n)
    worker_begin[tid] = !fits ? 0 : sh.bound[tid] < W ? g_of + bits_below(sh.cut, tid) + (cuts ? 1 : 0) : n_items;
  for (int e = tid; e < lay.max_combine; e += blockDim.x) comb_done[e] = 0;
  if (tid == 0) {
    hdr[kHdrStatus] = fits ? status : status | kStatusCapacity;
    hdr[kHdrNumItems] = fits ? n_items : 0;
    hdr[kHdrWorkCounter] = 0;
    hdr[kHdrNumCombine] = fits ? n_combine : 0;
    hdr[kHdrChunkTiles] = min(W, 1 << 30);
    hdr[kHdrCombineCounter] = 0;
  }
}

// Whether this form takes a plan: its tables hold it and no cost passes 31 bits.
__host__ __device__ inline bool partition_pair_fits(const Problem& p, const Layout& lay) {
  const long long tiles = ((long long)p.max_seq_len + kKvTile - 1) / kKvTile;
  const long long g_max = ((long long)p.max_q * p.num_heads + lay.rows_per_group - 1) / lay.rows_per_group;
  return pair_mma(p) && p.cp_world <= 1 && p.batch >= 1 && p.batch <= kPairMax && lay.max_groups <= kPairMax &&
         lay.n_workers >= 1 && lay.n_workers < kPairWorkers &&
         (long long)p.batch * g_max * (kOverheadTilesPair + tiles) < (1LL << 31);
}

// One block, a thread for each request, group and boundary.
__host__ __device__ inline int partition_pair_threads(const Problem& p, const Layout& lay) {
  const int need = max(max(p.batch, lay.max_groups), lay.n_workers + 1);
  return (need + 31) / 32 * 32;
}

bool partition_pair_picked(const Problem& p, const Layout& lay) { return partition_pair_fits(p, lay); }

cudaError_t launch_partition_pair(const Problem& p, const Layout& lay, void* ws, cudaStream_t stream) {
  partition_pair_kernel<<<1, partition_pair_threads(p, lay), 0, stream>>>(p, lay, static_cast<char*>(ws));
  return cudaGetLastError();
}

}  // namespace mla
