// Paged MLA decode over a 4-bit cache (mla_fp4.cuh) on sm_103a: a persistent
// kernel of CTA pairs whose tcgen05 MMAs span both CTAs (cta_group::2).
//
// What it computes, for the 128 query rows of a work item and the KV rows
// [kv_begin, kv_end) of its request, in 64-row tiles with an online softmax:
//   S = Q K^T (576 dims),  P = exp2(bmm1 log2(e) S - m),  O = sum P V / sum P
// with K row j = 576 values code * scale and V its first 512.
//
// Numbers.  A cache value has at most six significant bits and lies in
// [2^-10, 2688], so it is exact in f16, and both products run on f16 MMAs with
// fp32 accumulation.  A query row enters times a power of two that brings its
// largest element to [2^14, 2^15): every element down to 2^-31 of it is exact
// in f16, and its scores are multiplied back by 2^-k.  P enters as f16 (2^-11
// relative) times 2^7: the running reference m is raised only when a tile's
// maximum passes it by more than 2^8, so P stays below 2^15, and a P of 2^-31 of
// the row's largest still has a bit.  Row sums are fp32, of the unrounded P.
//
// What bounds it.  At 128 query rows a KV row costs 278 kFLOP against 324
// bytes: the tensor cores and the shared memory that feeds them, not HBM.  A
// pair splits a tile so that nothing but barriers passes between its CTAs:
//  * CTA r holds the item's query rows [64 r, 64 r + 64) whole (Q, S, P, O): a
//    row's softmax needs no other CTA.  O takes 256 columns of TMEM, S two
//    buffers of 32;
//  * S = Q K^T (M = 128, N = 64): CTA r provides tile rows [32 r, 32 r + 32) of
//    K in nine 64-dim chunks, through a ring of twelve 4 KB slots;
//  * O = P V (M = 128, N = 256 twice): CTA r provides V dims [256 r, 256 r +
//    256) of all 64 rows, two stages of 32 KB.
// The codes come by bulk copies into a two-stage staging area (the CTA's own
// rows whole, of the other rows only its V dims), and sixteen warps turn them
// into f16 in the swizzled operand layouts, one row a lane.
//
// Warp roles (896 threads): 0 copies, 1 issues QK (even CTA) and owns TMEM, 2
// issues PV, 4-11 softmax, correction and epilogue, 12-27 conversion and query
// load.  QK runs up to two tiles ahead of PV, so the tensor cores work while a
// softmax runs.  Every wait is bounded; a timeout sets the status word and both
// CTAs unwind.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "mla_common.cuh"
#include "mla_fp4.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

using namespace ptx;

constexpr int kTile = kKvTile;
constexpr int kHalf = kTile / 2;     // KV rows of a tile that one CTA brings for QK
constexpr int kCtaRows = 64;         // query rows of a CTA
constexpr int kRows = 2 * kCtaRows;  // query rows of a work item
constexpr int kChunks = 9;           // 64-dim chunks of a row: 8 latent, 1 RoPE
constexpr int kKSlots = 12;
constexpr int kGroup = 3;            // chunks that share a full and an empty barrier
constexpr int kConvWarps = 16;
constexpr int kSoftWarps = 8;
constexpr int kFirstSoft = 4, kFirstConv = kFirstSoft + kSoftWarps;
constexpr int kThreads = 32 * (kFirstConv + kConvWarps);
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kPShift = 7.0f;            // P is stored times 2^7

// shared memory, from a 1024-aligned base
constexpr uint32_t kQChunk = kCtaRows * 128;  // 64 rows x 64 dims f16, 128B swizzle
constexpr uint32_t kKChunk = kHalf * 128;     // 32 rows x 64 dims
constexpr uint32_t kVChunk = kTile * 128;     // 64 rows x 64 dims
constexpr uint32_t kVStage = 4 * kVChunk;
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = OFF_Q + kChunks * kQChunk;
constexpr uint32_t OFF_V = OFF_K + kKSlots * kKChunk;
constexpr uint32_t OFF_P = OFF_V + 2 * kVStage;
constexpr uint32_t OFF_STG = OFF_P + kCtaRows * 128;
// a staging stage: own rows' codes, other rows' V codes, scales of the tile's two halves
constexpr uint32_t STG_OWN = 0;
constexpr uint32_t STG_OTHER = STG_OWN + kHalf * kFp4CodeBytes;
constexpr uint32_t STG_SCALES = STG_OTHER + kHalf * 128;
constexpr uint32_t kStage = STG_SCALES + kTile * kFp4ScaleBytes;
constexpr uint32_t OFF_BARS = OFF_STG + 2 * kStage;
constexpr uint32_t OFF_XMAX = OFF_BARS + 320;       // float [2][256]: tile maxima by tile parity
constexpr uint32_t OFF_XSUM = OFF_XMAX + 2 * 256 * 4;  // float [256]: row sums, end of an item
constexpr uint32_t OFF_QSCALE = OFF_XSUM + 256 * 4;    // float [4][64]: 2^-k by item
constexpr uint32_t OFF_TMEM = OFF_QSCALE + 4 * kCtaRows * 4;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 16;
constexpr uint32_t OFF_LOADED = OFF_ABORT + 16;        // int [2][2]: staged halves, by stage
constexpr uint32_t kSmemBytes = OFF_LOADED + 16;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_P % 1024 == 0 && kStage % 16 == 0 &&
                  OFF_STG % 16 == 0 && STG_SCALES % 16 == 0 && OFF_BARS % 8 == 0,
              "alignment");

// TMEM columns
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_O = 0;    // lane: query row (mod 64) and V half; 256 V dims
constexpr uint32_t TM_S = 256;  // two 32-column buffers; lane: query row and KV half

enum Bar {
  STG_FULL0, STG_EMPTY0 = STG_FULL0 + 2,
  K_FULL0 = STG_EMPTY0 + 2,            // even CTA: both CTAs' chunks are in a group's slots
  K_EMPTY0 = K_FULL0 + kKSlots / kGroup,
  V_FULL0 = K_EMPTY0 + kKSlots / kGroup,  // even CTA
  PV_DONE0 = V_FULL0 + 2,              // by tile parity: V stage and P free, O stable
  S_FULL0 = PV_DONE0 + 2, S_EMPTY0 = S_FULL0 + 2,  // S_EMPTY: even CTA
  P_FULL = S_EMPTY0 + 2,               // even CTA
  Q_FULL, Q_EMPTY,                     // Q_FULL: even CTA
  QS_FULL0,                            // 4: by item, the query rows' scales are written
  XM0 = QS_FULL0 + 4,                  // 4: [tile parity][pair of warps] maxima exchanged
  XS0 = XM0 + 4,                       // 2: [pair of warps] row sums exchanged
  EPI = XS0 + 2,                       // the partial is written
  DRAIN0,                              // 2: every MMA of an issuing warp has completed
  NUM_BARS = DRAIN0 + 2
};
static_assert(NUM_BARS * 8 <= 320, "barrier area");

struct Ctx {
  uint64_t* bars;
  volatile int* abort;
  uint32_t peer_abort;
  uint32_t leader_bars;  // shared::cluster address of the even CTA's barriers
  int* status;
};

__device__ __forceinline__ void give_up(const Ctx& c) {
  *c.abort = 1;
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(c.peer_abort), "r"(1) : "memory");
  atomicOr(c.status, kStatusTimeout);
}
__device__ __forceinline__ bool wait_bar(const Ctx& c, int bar, uint32_t parity) {
  uint64_t* b = &c.bars[bar];
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 1023) == 1023 && *c.abort) return false;
  }
  give_up(c);
  return false;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit; ++i)
    if (mbar_try_wait(bar, parity)) return;
}
__device__ __forceinline__ void arrive_leader(const Ctx& c, int bar, uint32_t count) {
  mbar_arrive_pair(c.leader_bars + 8u * bar, count);
}

__device__ __forceinline__ int n_tiles_of(const WorkItem& it) {
  return (it.kv_end - it.kv_begin + kTile - 1) / kTile;
}

// The rows that an item's virtual rows stand for (see window_skip), and which of
// them some query row of the request sees: a page without one is not read (a
// sliding window's caller may have given it away), and such rows enter as zeros.
struct Walk {
  int sink_end, skip, sinks, low;  // low: first row of the earliest window
  __device__ Walk(const Problem& p, const WorkItem& it)
      : sink_end(window_sink_rows(p.sinks)),
        skip(window_skip(p.window, p.sinks, p.causal, it.seq_len, it.q_len)),
        sinks(p.sinks),
        low(p.window > 0 ? (p.causal ? it.seq_len - it.q_len : it.seq_len - 1) - p.window + 1 : INT_MIN) {}
  __device__ int row(int v) const { return v < sink_end ? v : v + skip; }
  __device__ bool seen(int first, int last) const { return last >= low || first < sinks; }
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The f16 value of an e4m3 code, in both halves of a word.
__device__ __forceinline__ uint32_t scale_pair(uint32_t code) {
  uint32_t h;
  asm("{\n .reg .b16 lo;\n mov.b32 {lo, _}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(code));
  return __byte_perm(h, h, 0x1010);
}
// Eight codes times their scale, as a 16-byte unit of f16.
__device__ __forceinline__ uint4 convert8(uint32_t codes, uint32_t scale) {
  uint32_t h[4];
  e2m1x8_to_f16x2(codes, h);
  return make_uint4(hmul2(h[0], scale), hmul2(h[1], scale), hmul2(h[2], scale), hmul2(h[3], scale));
}
// Two groups: 32 codes and their two scales.
__device__ __forceinline__ void convert32(const uint4 codes, uint32_t scales, uint4 (&x)[4]) {
  const uint32_t s0 = scale_pair(scales & 0xFFu), s1 = scale_pair(scales >> 8);
  x[0] = convert8(codes.x, s0);
  x[1] = convert8(codes.y, s0);
  x[2] = convert8(codes.z, s1);
  x[3] = convert8(codes.w, s1);
}
__device__ __forceinline__ void put(unsigned char* row, int unit, int r, uint4 v) {
  *reinterpret_cast<uint4*>(row + ((unit ^ (r & 7)) << 4)) = v;
}

// The power of two that brings a query row's largest magnitude (bf16 bits, sign
// cleared) to [2^14, 2^15): its exponent k; 0 for zeros, a NaN or an infinity.
__device__ __forceinline__ int query_exponent(uint32_t mbits) {
  const int e = (int)(mbits >> 7);  // biased exponent
  if (mbits == 0 || e == 255) return 0;
  return min(126, 14 - (e - 127));
}
__device__ __forceinline__ uint32_t max_bits(const uint4 x) {
  return __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                  __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ uint4 bf16x8_to_f16(const uint4 x, float up) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w[e] << 16) * up,
                                        __uint_as_float(w[e] & 0xFFFF0000u) * up);
    o[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 e4m3x8_to_f16(const uint2 x) {
  const uint32_t w[2] = {x.x, x.y};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    asm("{\n .reg .b16 lo;\n mov.b32 {lo, _}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}"
        : "=r"(o[e])
        : "r"(w[e >> 1] >> (16 * (e & 1))));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode_fp4_kernel(const Problem p, const Layout lay, char* __restrict__ ws) {
  // The swizzled tiles need 1024-byte alignment, and there is no room to round
  // up: the block has no other shared memory, so its dynamic part starts at
  // offset 0 of its window.  A block placed otherwise reports and leaves.
  extern __shared__ __align__(1024) unsigned char sm[];
  if ((smem_u32(sm) & 1023) != 0) {
    if (threadIdx.x == 0) atomicOr(reinterpret_cast<int*>(ws) + kHdrStatus, kStatusTimeout);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int worker = (int)cluster_id_x();
  const WorkItem* items = reinterpret_cast<const WorkItem*>(ws + lay.items);
  const int* worker_begin = reinterpret_cast<const int*>(ws + lay.worker_ranges);

  Ctx c;
  c.bars = reinterpret_cast<uint64_t*>(sm + OFF_BARS);
  c.abort = reinterpret_cast<volatile int*>(sm + OFF_ABORT);
  c.peer_abort = map_to_rank(smem_u32(sm + OFF_ABORT), rank ^ 1);
  c.leader_bars = map_to_rank(smem_u32(sm + OFF_BARS), 0);
  c.status = reinterpret_cast<int*>(ws) + kHdrStatus;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
  volatile int* loaded = reinterpret_cast<volatile int*>(sm + OFF_LOADED);

  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      uint32_t n = 1;  // one commit
      if (i >= STG_FULL0 && i < STG_FULL0 + 2) n = 1 + 32;  // bulk copies, each lane's own
      if (i >= STG_EMPTY0 && i < STG_EMPTY0 + 2) n = kConvWarps;
      // a latent chunk's two warps count four times each, as the RoPE chunk has eight
      if (i >= K_FULL0 && i < K_FULL0 + kKSlots / kGroup) n = 2 * 8 * kGroup;
      if (i >= V_FULL0 && i < V_FULL0 + 2) n = 2 * kConvWarps;
      if (i >= S_EMPTY0 && i < S_EMPTY0 + 2) n = 2 * kSoftWarps;
      if (i == P_FULL) n = 2 * kSoftWarps;
      if (i == Q_FULL) n = 2 * kConvWarps;
      if (i >= QS_FULL0 && i < QS_FULL0 + 4) n = kConvWarps;
      if (i >= XM0 && i < XS0 + 2) n = kSoftWarps / 2;
      if (i == EPI) n = kSoftWarps;
      mbar_init(&c.bars[i], n);
    }
    *c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the other CTA's barriers exist before any remote arrival
  // the work list comes from the partitioner; the combine kernel may be
  // scheduled from here on (it waits on counters that the epilogues bump)
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int item_begin = worker_begin[worker], item_end = worker_begin[worker + 1];
  const int H = p.num_heads;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    // Page ids a batch of 32 ahead (one per lane), as virtual page slots of the
    // item.  Lane 0 issues the bulk copies (codes of the own rows, scales); the
    // other rows' V codes, 128 bytes of each 288, go by 16-byte copies of all
    // lanes (one bulk copy a row took 4000 cycles to issue).
    const int ps = p.page_size, npg = kTile / ps;
    const size_t page_bytes = (size_t)ps * kFp4RowBytes;
    const unsigned char* cache = static_cast<const unsigned char*>(p.kv_cache);
    uint32_t g = 0;
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      const Walk walk(p, it);
      const int* bt = p.block_tables + (size_t)it.b * p.max_pages;
      const int n_pages = (it.kv_end - it.kv_begin + ps - 1) / ps;
      auto page_at = [&](int i) {
        const int r = walk.row(it.kv_begin + i * ps);
        return i < n_pages && walk.seen(r, r + ps - 1) ? bt[r / ps] : -1;
      };
      int cur = page_at(lane), nxt = page_at(32 + lane);
      for (int t = 0; t < nt; ++t, ++g) {
        const int slot0 = t * npg;  // never straddles a batch: npg divides 32
        if (slot0 > 0 && (slot0 & 31) == 0) {
          cur = nxt;
          nxt = page_at(slot0 + 32 + lane);
        }
        int pages[2];
        pages[0] = __shfl_sync(0xffffffffu, cur, slot0 & 31);
        pages[1] = __shfl_sync(0xffffffffu, cur, (slot0 + npg - 1) & 31);
        const int s = g & 1;
        const bool ok = lane == 0 ? wait_bar(c, STG_EMPTY0 + s, ((g >> 1) & 1) ^ 1) : false;
        if (!__shfl_sync(0xffffffffu, ok, 0)) goto done_copy;
        const int j0 = it.kv_begin + t * kTile;
        bool on[2];
        const unsigned char* page[2];
        int row[2];
        uint32_t bytes = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = walk.row(j0) + h * kHalf;
          on[h] = j0 + h * kHalf < it.kv_end && walk.seen(r, r + kHalf - 1);
          if (on[h] && (pages[h] < 0 || (long long)pages[h] >= p.num_pages)) {
            if (lane == 0) atomicOr(c.status, kStatusPage);
            on[h] = false;
          }
          page[h] = cache + (size_t)(on[h] ? pages[h] : 0) * page_bytes;
          row[h] = ps == kTile ? h * kHalf : 0;
          if (on[h]) bytes += (h == rank ? kHalf * kFp4CodeBytes : 0) + kHalf * kFp4ScaleBytes;
        }
        unsigned char* stg = sm + OFF_STG + s * kStage;
        uint64_t* full = &c.bars[STG_FULL0 + s];
        if (lane == 0) {
          loaded[2 * s] = on[0];
          loaded[2 * s + 1] = on[1];
          mbar_arrive_expect_tx(full, bytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!on[h]) continue;
            bulk_load(stg + STG_SCALES + h * kHalf * kFp4ScaleBytes,
                      page[h] + (size_t)ps * kFp4CodeBytes + row[h] * kFp4ScaleBytes,
                      kHalf * kFp4ScaleBytes, full);
            if (h == rank)
              bulk_load(stg + STG_OWN, page[h] + row[h] * kFp4CodeBytes, kHalf * kFp4CodeBytes, full);
          }
        }
        __syncwarp();
        // the other rows' V codes, eight 16-byte units of a row: eight lanes a row
        const int o = rank ^ 1;
        if (on[o]) {
          const unsigned char* src = page[o] + row[o] * kFp4CodeBytes + 128 * rank + 16 * (lane & 7);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + (lane >> 3);
            cp_async_16(stg + STG_OTHER + r * 128 + 16 * (lane & 7), src + r * kFp4CodeBytes);
          }
        }
        cp_async_arrive(full);
      }
    }
  done_copy:
    // no copy issued here may still be landing when the CTA leaves
    if (lane == 0)
      for (uint32_t k = 0; k < 2 && k < g; ++k) {
        const uint32_t gi = g - 1 - k;
        drain_wait(&c.bars[STG_FULL0 + (gi & 1)], (gi >> 1) & 1);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issue
    // The whole warp walks the loops and one lane issues (see elect_one).
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_half(kRows, kTile, false, false);
      // operand descriptors; a step along an operand adds its bytes / 16
      const uint64_t q_desc = smem_desc(smem_u32(sm + OFF_Q), 16, 1024, kSwizzle128B);
      const uint64_t k_desc = smem_desc(smem_u32(sm + OFF_K), 16, 1024, kSwizzle128B);
      uint32_t g = 0;
      uint32_t group = 0, round = 0;  // ring place of the next three chunks
      int n_item = 0;
      for (int idx = item_begin; idx < item_end; ++idx) {
        const int nt = __shfl_sync(0xffffffffu, n_tiles_of(items[idx]), 0);
        if (nt <= 0) continue;
        if (!wait_bar(c, Q_FULL, n_item & 1)) goto done_qk;
        ++n_item;
        for (int t = 0; t < nt; ++t, ++g) {
          const uint32_t sb = g & 1;
          if (!wait_bar(c, S_EMPTY0 + sb, ((g >> 1) & 1) ^ 1)) goto done_qk;
#pragma unroll
          for (int k3 = 0; k3 < kChunks / kGroup; ++k3) {
            if (!wait_bar(c, K_FULL0 + group, round & 1)) goto done_qk;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t kd = k_desc + group * (kGroup * kKChunk >> 4);
#pragma unroll
              for (int k = 0; k < kGroup; ++k)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_f16_pair_ss(tmem + TM_S + 32 * sb,
                                  q_desc + ((kGroup * k3 + k) * kQChunk >> 4) + 2 * ks,
                                  kd + (k * kKChunk >> 4) + 2 * ks, idesc,
                                  (k3 | k | ks) != 0 ? 1u : 0u);
              mma_commit_pair(&c.bars[K_EMPTY0 + group]);
              if (k3 == kChunks / kGroup - 1) {
                mma_commit_pair(&c.bars[S_FULL0 + sb]);
                if (t + 1 == nt) mma_commit_pair(&c.bars[Q_EMPTY]);
              }
            }
            __syncwarp();
            if (++group == kKSlots / kGroup) {
              group = 0;
              ++round;
            }
          }
        }
      }
    done_qk:
      __syncwarp();
      if (elect_one()) mma_commit_pair(&c.bars[DRAIN0]);
      drain_wait(&c.bars[DRAIN0], 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ PV issue
    // A warp of its own: its waits for P would hold up the next tile's QK.
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_half(kRows, 256, false, true);
      const uint64_t p_desc = smem_desc(smem_u32(sm + OFF_P), 16, 1024, kSwizzle128B);
      const uint64_t v_desc = smem_desc(smem_u32(sm + OFF_V), kVChunk, 1024, kSwizzle128B);
      uint32_t g = 0;
      for (int idx = item_begin; idx < item_end; ++idx) {
        const int nt = __shfl_sync(0xffffffffu, n_tiles_of(items[idx]), 0);
        for (int t = 0; t < nt; ++t, ++g) {
          const uint32_t s = g & 1;
          if (!wait_bar(c, V_FULL0 + s, (g >> 1) & 1)) goto done_pv;
          if (!wait_bar(c, P_FULL, g & 1)) goto done_pv;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t v = v_desc + s * (kVStage >> 4);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_f16_pair_ss(tmem + TM_O + 128 * j, p_desc + 2 * ks,
                                v + ((j * 2 * kVChunk + ks * 16 * 128) >> 4), idesc,
                                (t == 0 && ks == 0) ? 0u : 1u);
            mma_commit_pair(&c.bars[PV_DONE0 + s]);
          }
          __syncwarp();
        }
      }
    done_pv:
      __syncwarp();
      if (elect_one()) mma_commit_pair(&c.bars[DRAIN0 + 1]);
      drain_wait(&c.bars[DRAIN0 + 1], 0);
    }
  } else if (warp < kFirstSoft) {
    // (warps 4-11 need TMEM lane quarters 0-3 twice)
  } else if (warp < kFirstConv) {
    // ------------------------------------------------------------ softmax, correction, epilogue
    // Thread = TMEM lane l = 32 (warp mod 4) + lane and column part cc: query row
    // l mod 64 of the CTA, KV rows (columns of S) 32 (l / 64) + 16 cc + [0, 16),
    // V dims (columns of O) 256 (l / 64) + 128 cc + [0, 128).  A row's four
    // threads are in four warps that exchange maxima through shared memory.
    const int quad = warp & 3, cc = (warp - kFirstSoft) >> 2;
    const int l = 32 * quad + lane, hh = quad >> 1, row = l & 63;
    const int q = kCtaRows * rank + row;  // row of the work item
    const int pair = quad & 1;
    const uint32_t tm = tmem + ((uint32_t)(32 * quad) << 16);
    const float bmm1 = run_bmm1(p, c.status) * kLog2e;
    const float bmm2 = run_bmm2(p);
    const int W = max(p.cp_world, 1);
    float* xmax = reinterpret_cast<float*>(sm + OFF_XMAX);
    float* xsum = reinterpret_cast<float*>(sm + OFF_XSUM);
    const float* qscale = reinterpret_cast<const float*>(sm + OFF_QSCALE);
    unsigned char* prow = sm + OFF_P + row * 128;
    uint4* part_o = reinterpret_cast<uint4*>(ws + lay.part_o);
    float* part_lse = reinterpret_cast<float*>(ws + lay.part_lse);
    int* comb_done = reinterpret_cast<int*>(ws + lay.comb_done);
    uint32_t g = 0;
    int n_item = 0, n_split = 0;
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      const Walk walk(p, it);
      const int rows_total = it.q_len * H, row0 = it.g * kRows;
      const int n_rows = min(kRows, rows_total - row0);
      const bool row_ok = q < n_rows;
      auto last_of = [&](int r) {
        return p.causal ? causal_last(it.mask_base, (row0 + r) / H, W) : it.seq_len - 1;
      };
      const int last = last_of(min(q, n_rows - 1));
      const int low = p.window > 0 ? last - p.window + 1 : INT_MIN;  // first row of the window
      // tiles inside [clean_lo, clean_hi) need no mask for any row of the item
      const int clean_hi = last_of(0) + 1;
      const int clean_lo = p.window > 0 ? last_of(n_rows - 1) - p.window + 1 : INT_MIN;
      if (!wait_bar(c, QS_FULL0 + (n_item & 3), (n_item >> 2) & 1)) goto done_soft;
      const float scale = bmm1 * qscale[(n_item & 3) * kCtaRows + row];
      float m = -INFINITY, l_part = 0.f;
      for (int t = 0; t < nt; ++t, ++g) {
        const int sb = g & 1;
        if (!wait_bar(c, S_FULL0 + sb, (g >> 1) & 1)) goto done_soft;
        tc_fence_after();
        float sv[16];
        {
          uint32_t v[16];
          tmem_ld_32x32b_x16(tm + TM_S + 32 * sb + 16 * cc, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sv[j] = __uint_as_float(v[j]) * scale;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(c, S_EMPTY0 + sb, 1);
        const int v0 = it.kv_begin + t * kTile;        // virtual row of the tile
        const int r0 = walk.row(v0);                    // its row
        const int valid = it.kv_end - v0;               // rows of the tile inside the item
        const bool clean = valid >= kTile && r0 + kTile <= clean_hi &&
                           (r0 >= clean_lo || r0 + kTile <= p.sinks);
        if (!clean) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int k = 32 * hh + 16 * cc + j, at = r0 + k;
            if (!(at <= last && k < valid && (at >= low || at < p.sinks))) sv[j] = -INFINITY;
          }
        }
        float mt[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int j = 4; j < 16; ++j) mt[j & 3] = fmaxf(mt[j & 3], sv[j]);
        const float m_own = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
        float* xm = xmax + sb * 256;
        xm[128 * cc + l] = m_own;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bars[XM0 + 2 * sb + pair]);
        if (!wait_bar(c, XM0 + 2 * sb + pair, (g >> 1) & 1)) goto done_soft;
        // (all four from shared memory: the same result in the row's four threads)
        const float m_tile = fmaxf(fmaxf(xm[row], xm[row + 64]), fmaxf(xm[row + 128], xm[row + 192]));
        const float m_new = (m_tile > m + kRescaleThreshold || t == 0) ? m_tile : m;
        const bool need = t > 0 && m_new != m;
        const float f = need ? ex2(m - m_new) : 1.f;  // m = -inf: 0
        m = m_new;
        l_part *= f;
        const float ref = (m == -INFINITY ? 0.f : m) - kPShift;
        // (rows past the request's own compute something that nothing reads)
        uint32_t pw[8];
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = ex2(sv[2 * j] - ref), b = ex2(sv[2 * j + 1] - ref);
          rs[j & 3] += a + b;
          const __half2 h = __floats2half2_rn(a, b);
          pw[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        l_part += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        // PV of the previous tile is done: its P may be replaced, and O is stable
        if (g > 0 && !wait_bar(c, PV_DONE0 + ((g - 1) & 1), ((g - 1) >> 1) & 1)) goto done_soft;
        if (__any_sync(0xffffffffu, need)) {
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            uint32_t x[16];
            tmem_ld_32x32b_x16(tm + TM_O + 128 * cc + 16 * k, x);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
            tmem_st_32x32b_x16(tm + TM_O + 128 * cc + 16 * k, x);
          }
          tmem_wait_st();
          tc_fence_before();
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          put(prow, 4 * hh + 2 * cc + u, row,
              make_uint4(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_leader(c, P_FULL, 1);
      }
      // the row's sum: its four threads' shares
      xsum[128 * cc + l] = l_part;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.bars[XS0 + pair]);
      if (!wait_bar(c, XS0 + pair, n_item & 1)) goto done_soft;
      const float l_row = (xsum[row] + xsum[row + 64]) + (xsum[row + 128] + xsum[row + 192]);
      const float lse = l_row > 0.f ? (m - kPShift + log2f(l_row)) * kLn2 : -INFINITY;
      const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
      const size_t grow = (size_t)it.q_start * H + row0 + q;
      if (row_ok && hh == 0 && cc == 0) {
        if (it.slot >= 0)
          part_lse[(size_t)it.slot * kRows + q] = lse;
        else if (p.return_lse)
          p.lse[grow] = lse;
      }
      if (!wait_bar(c, PV_DONE0 + ((g - 1) & 1), ((g - 1) >> 1) & 1)) goto done_soft;
      tc_fence_after();
      const float s2 = it.slot < 0 ? inv * bmm2 : inv;
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        uint32_t x[16];
        tmem_ld_32x32b_x16(tm + TM_O + 128 * cc + 16 * k, x);
        tmem_wait_ld();
        if (!row_ok) continue;
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(x[2 * e]) * s2,
                                                         __uint_as_float(x[2 * e + 1]) * s2);
          o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        const int chunk = 16 * hh + 8 * cc + k;  // of 16 dims
        uint4 *d0, *d1;
        if (it.slot < 0) {
          d0 = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + grow * kVDim + 16 * chunk);
          d1 = d0 + 1;
        } else {
          d0 = part_o + part_unit(it.slot, kRows, chunk, 0, q);
          d1 = part_o + part_unit(it.slot, kRows, chunk, 1, q);
        }
        *d0 = make_uint4(o[0], o[1], o[2], o[3]);
        *d1 = make_uint4(o[4], o[5], o[6], o[7]);
      }
      tc_fence_before();
      if (it.slot >= 0) {
        // the warps' partial is visible GPU-wide, then this CTA counts its chunk
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bars[EPI]);
        if (warp == kFirstSoft) {
          if (!wait_bar(c, EPI, n_split & 1)) goto done_soft;
          if (lane == 0 && it.comb >= 0) {
            __threadfence();
            atomicAdd(comb_done + it.comb, 1);
          }
        }
        ++n_split;
      }
      ++n_item;
    }
  done_soft:;
  } else {
    // ------------------------------------------------------------ conversion and query load
    // Warp w: latent dims [32 w, 32 w + 32) of the own rows, one row a lane, into
    // K; then, if those are V dims of this CTA, the same values into V and eight
    // RoPE dims into K, else 32 V dims of the other rows.
    const int w = warp - kFirstConv;
    const bool in_half = (w >> 3) == rank;
    const int vw = w & 7;  // V part of 32 dims; RoPE part of 8
    float* qscale = reinterpret_cast<float*>(sm + OFF_QSCALE);
    uint32_t g = 0;
    // ring places of this warp's chunk and of the RoPE chunk
    uint32_t kslot = w >> 1, kround = 0, rslot = 8, rround = 0;
    int n_item = 0;
    auto convert_tile = [&](const WorkItem& it, const Walk& walk, int t) -> bool {
      const int s = g & 1;
      if (!wait_bar(c, STG_FULL0 + s, (g >> 1) & 1)) return false;
      const unsigned char* stg = sm + OFF_STG + s * kStage;
      // rows past the item's end, that no query row sees, or on a page that was
      // not loaded, are zeros
      const int v0 = it.kv_begin + t * kTile, r0 = walk.row(v0);
      const int own = kHalf * rank + lane, oth = kHalf * (rank ^ 1) + lane;
      const bool on_own = v0 + own < it.kv_end && loaded[2 * s + rank] && walk.seen(r0 + own, r0 + own);
      const unsigned char* sc_own = stg + STG_SCALES + own * kFp4ScaleBytes;
      const unsigned char* codes = stg + STG_OWN + lane * kFp4CodeBytes;
      const uint32_t sc = on_own ? *reinterpret_cast<const uint16_t*>(sc_own + 2 * w) : 0u;
      uint4 x[4];
      convert32(*reinterpret_cast<const uint4*>(codes + 16 * w), sc, x);
      if (!wait_bar(c, K_EMPTY0 + kslot / kGroup, (kround & 1) ^ 1)) return false;
      {
        unsigned char* kd = sm + OFF_K + kslot * kKChunk + lane * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) put(kd, 4 * (w & 1) + e, lane, x[e]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_leader(c, K_FULL0 + kslot / kGroup, 4);
      if (in_half) {
        const uint32_t rs = on_own ? (uint32_t)sc_own[32 + (vw >> 1)] : 0u;
        const uint4 y = convert8(*reinterpret_cast<const uint32_t*>(codes + 256 + 4 * vw), scale_pair(rs));
        if (!wait_bar(c, K_EMPTY0 + rslot / kGroup, (rround & 1) ^ 1)) return false;
        put(sm + OFF_K + rslot * kKChunk + lane * 128, vw, lane, y);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_leader(c, K_FULL0 + rslot / kGroup, 1);
      } else {
        const bool on_oth = v0 + oth < it.kv_end && loaded[2 * s + (rank ^ 1)] && walk.seen(r0 + oth, r0 + oth);
        const uint32_t so = on_oth ? *reinterpret_cast<const uint16_t*>(stg + STG_SCALES + oth * kFp4ScaleBytes +
                                                                        16 * rank + 2 * vw)
                                   : 0u;
        convert32(*reinterpret_cast<const uint4*>(stg + STG_OTHER + lane * 128 + 16 * vw), so, x);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.bars[STG_EMPTY0 + s]);  // every code is in registers
      if (!wait_bar(c, PV_DONE0 + s, ((g >> 1) & 1) ^ 1)) return false;
      {
        unsigned char* vd = sm + OFF_V + s * kVStage + (vw >> 1) * kVChunk + (in_half ? own : oth) * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) put(vd, 4 * (vw & 1) + e, lane, x[e]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_leader(c, V_FULL0 + s, 1);
      // nine chunks a tile through twelve slots
      kslot += kChunks;
      if (kslot >= kKSlots) {
        kslot -= kKSlots;
        ++kround;
      }
      rslot += kChunks;
      if (rslot >= kKSlots) {
        rslot -= kKSlots;
        ++rround;
      }
      ++g;
      return true;
    };
    // Rows [4 w, 4 w + 4) of the item's query in this CTA: f16 in nine swizzled
    // chunks, and each row's factor 2^-k.  Rows past the query's end are zero.
    auto load_query = [&](const WorkItem& it, int n) -> bool {
      const long long q_rows = p.total_q * H;
      const long long first = (long long)it.q_start * H + (long long)it.g * kRows + kCtaRows * rank + 4 * w;
      const int u2 = 64 + (lane & 7);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint4 x[2][3];
        if (p.q_fp8) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const long long qr = first + 2 * half + r;
            const uint2* src = reinterpret_cast<const uint2*>(p.query) + (qr < q_rows ? qr : 0) * 72;
            const bool in = qr < q_rows;
            uint2 y[3] = {in ? __ldg(src + lane) : make_uint2(0, 0), in ? __ldg(src + 32 + lane) : make_uint2(0, 0),
                          in ? __ldg(src + u2) : make_uint2(0, 0)};
#pragma unroll
            for (int k = 0; k < 3; ++k) x[r][k] = make_uint4(y[k].x, y[k].y, 0, 0);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const long long qr = first + 2 * half + r;
            const uint4* src = reinterpret_cast<const uint4*>(p.query) + (qr < q_rows ? qr : 0) * 72;
            const bool in = qr < q_rows;
            x[r][0] = in ? __ldg(src + lane) : make_uint4(0, 0, 0, 0);
            x[r][1] = in ? __ldg(src + 32 + lane) : make_uint4(0, 0, 0, 0);
            x[r][2] = in ? __ldg(src + u2) : make_uint4(0, 0, 0, 0);
          }
        }
        // every QK of the previous item has read its query
        if (half == 0 && !wait_bar(c, Q_EMPTY, (n & 1) ^ 1)) return false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 4 * w + 2 * half + r;
          int k = 0;
          if (!p.q_fp8) {
            uint32_t mb = __vmaxu2(__vmaxu2(max_bits(x[r][0]), max_bits(x[r][1])), max_bits(x[r][2]));
            mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
            k = query_exponent(mb);
          }
          const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const int unit = e < 2 ? 32 * e + lane : u2;
            const uint4 v = p.q_fp8 ? e4m3x8_to_f16(make_uint2(x[r][e].x, x[r][e].y))
                                    : bf16x8_to_f16(x[r][e], up);
            if (e < 2 || lane < 8)
              put(sm + OFF_Q + (unit >> 3) * kQChunk + row * 128, unit & 7, row, v);
          }
          if (lane == 0) qscale[(n & 3) * kCtaRows + row] = __uint_as_float((uint32_t)(127 - k) << 23);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c.bars[QS_FULL0 + (n & 3)]);
        arrive_leader(c, Q_FULL, 1);
      }
      return true;
    };
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      // the first tile before the query: its conversion needs nothing of the
      // previous item but ring places
      const Walk walk(p, it);
      if (n_item > 0 && !convert_tile(it, walk, 0)) goto done_conv;
      if (!load_query(it, n_item)) goto done_conv;
      for (int t = n_item > 0 ? 1 : 0; t < nt; ++t)
        if (!convert_tile(it, walk, t)) goto done_conv;
      ++n_item;
    }
  done_conv:;
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA touches the other's memory or TMEM any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

namespace {

cudaLaunchConfig_t pair_launch(int grid, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t decode_fp4_setup(int sm_count, int* n_pairs) {
  cudaError_t e = cudaFuncSetAttribute(decode_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  const cudaLaunchConfig_t cfg = pair_launch(2 * (sm_count / 2), nullptr, &attr);
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, decode_fp4_kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (clusters <= 0) return cudaErrorInvalidConfiguration;
  *n_pairs = std::min(clusters, sm_count / 2);
  return cudaSuccess;
}

cudaError_t launch_decode_fp4(const Problem& p, const Layout& lay, void* ws, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  const cudaLaunchConfig_t cfg = pair_launch(lay.n_ctas, stream, &attr);
  return cudaLaunchKernelEx(&cfg, decode_fp4_kernel, p, lay, static_cast<char*>(ws));
}

}  // namespace mla
