// Paged MLA decode over a 4-bit cache (mla_fp4.cuh), and over a cache of any format
// with a sliding window, on sm_103a: a persistent kernel of CTA pairs whose tcgen05
// MMAs span both CTAs (cta_group::2).
//
// What it computes, for the 128 query rows of a work item and the KV rows
// [kv_begin, kv_end) of its request, in 64-row tiles with an online softmax:
//   S = Q K^T (576 dims),  P = exp2(bmm1 log2(e) S - m),  O = sum P V / sum P
// with K row j = 576 values (4 bits: code * scale) and V its first 512.
//
// Numbers.  A 4-bit cache's value has at most six significant bits and lies in
// [2^-10, 2688] (e4m3: four bits, [2^-9, 448]), so it is exact in f16, and both
// products run on f16 MMAs with fp32 accumulation.  A bf16 query row enters times a
// power of two that brings its largest element to [2^14, 2^15): every element down to
// 2^-31 of it is exact in f16, and its scores are multiplied back by 2^-k.  P enters as
// f16 (2^-11 relative) times 2^7: the running reference m is raised only when a tile's
// maximum passes it by more than 2^8, so P stays below 2^15, and a P of 2^-31 of
// the row's largest still has a bit.  A bf16 cache runs on bf16 MMAs, query and cache as
// they are, P rounded to bf16 (by 2^-8 of it at most) and O divided by the sum of
// the rounded P.  Row sums are fp32, of the unrounded P for the LSE and elsewhere for O too.
//
// What bounds it.  At 128 query rows a KV row costs 278 kFLOP against 324 (4 bits) to
// 1152 bytes: the tensor cores and the shared memory that feeds them, not HBM.  A
// pair splits a tile so that nothing but barriers passes between its CTAs:
//  * CTA r holds the item's query rows [64 r, 64 r + 64) whole (Q, S, P, O): a
//    row's softmax needs no other CTA.  TMEM: O 256 columns, S two buffers of 32,
//    six of the query's nine 64-dim chunks 192;
//  * S = Q K^T (M = 128, N = 64): CTA r provides tile rows [32 r, 32 r + 32) of
//    K in nine 64-dim chunks, two stages of 36 KB (bf16: three);
//  * O = P V (M = 128, N = 256 twice): CTA r provides V dims [256 r, 256 r +
//    256) of all 64 rows, two stages of 32 KB.
// 4-bit and e4m3 codes come by bulk copies into a two-stage staging area (the CTA's own
// rows whole, of the other rows only its V dims), and sixteen warps turn them
// into f16 in the swizzled operand layouts, one row a lane.  Shared-memory
// bandwidth is the scarce resource: a tile's MMAs read 24 KB of Q, 68 KB of K and
// V and 16 KB of P, its conversion writes 68 KB and reads 15.  (With all of Q in
// shared memory the MMAs read 48 KB more; with the staged codes read across bank
// conflicts a long call took 476 us instead of 417.)  bf16 rows come by TMA where the
// MMAs read them.
//
// Measured, a call: 8 x 2 x 128 heads over 64-128k rows of 4 bits 377 us, 1.08 PFLOP/s
// (56% of the bf16 rate of a large library product; tensor pipes busy 45% of all cycles,
// shared memory some 90% of a tile's, bank conflicts among them); 64 x 128 heads over 1-8k
// rows 103 us, 779 TFLOP/s; window 4096, e4m3, 32 x 4 x 128 heads 182 us, 801 TFLOP/s;
// window 1024, bf16, 64 x 128 heads 38.8 us, of which some 12 are the launch chain, the
// first loads and the epilogue.
//
// Warp roles (896 threads): 0 and 3 copy, 1 issues QK (even CTA) and owns TMEM, 2
// issues PV, 4-11 softmax, correction and epilogue, 12-27 conversion and query
// load.  Softmax and conversion each run in two groups that take alternate
// tiles: their chains of waits and round trips are longer than a tile's MMAs.
// Every wait is bounded; a timeout sets the status word and both CTAs unwind.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

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
constexpr int kGroup = 3;            // chunks that share a full barrier
constexpr int kTmemChunks = 6;       // the query's chunks that live in TMEM
constexpr int kConvWarps = 16;
constexpr int kSoftWarps = 8;
constexpr int kFirstSoft = 4, kFirstConv = kFirstSoft + kSoftWarps;
constexpr int kThreads = 32 * (kFirstConv + kConvWarps);
constexpr int kAhead = 6;            // tiles prefetched to L2 (under 16: at most one batch of page ids on)
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// shared memory, from a 1024-aligned base
constexpr uint32_t kQChunk = kCtaRows * 128;  // 64 rows x 64 dims f16, 128B swizzle
constexpr uint32_t kKChunk = kHalf * 128;     // 32 rows x 64 dims
constexpr uint32_t kVChunk = kTile * 128;     // 64 rows x 64 dims
constexpr uint32_t kVStage = 4 * kVChunk;
constexpr uint32_t kKStage = kChunks * kKChunk;
constexpr uint32_t kPTile = kCtaRows * 128;
constexpr uint32_t OFF_Q = 0;  // chunks kTmemChunks..8
constexpr uint32_t OFF_K = OFF_Q + (kChunks - kTmemChunks) * kQChunk;
constexpr uint32_t OFF_V = OFF_K + 2 * kKStage;
constexpr uint32_t OFF_P = OFF_V + 2 * kVStage;

// The cache's format: 4 bits; e4m3 (576 bytes a row, values exact in f16); bf16
// (bf16 MMAs, and TMA brings K and V where the MMAs read them: no staging, and
// the conversion warps only load queries and clear unused rows).
enum Cache { kFp4, kE4m3, kBf16 };
template <int kCache> struct Cfg {
  static constexpr bool kTma = kCache == kBf16;
  static constexpr float kPShift = kTma ? 0.f : 7.f;  // P is stored times 2^kPShift (bf16 has the range)
  static constexpr uint32_t kCodeBytes = kCache == kFp4 ? kFp4CodeBytes : kTma ? 2 * kQkDim : kQkDim;  // of a row
  static constexpr uint32_t kScaleBytes = kCache == kFp4 ? kFp4ScaleBytes : 0;
  static constexpr uint32_t kVBytes = kCache == kFp4 ? 128 : 256;  // codes of 256 dims
  static constexpr uint32_t kRowBytes = kCodeBytes + kScaleBytes;
  static constexpr int kPartShift = part_shift(kCache == kFp4 ? kKvFp4 : kKvFp8);
  // V: 64-dim chunks of the tile's 64 rows; TMA brings a half's four chunks together,
  // so there they are of 32 rows, a half after the other
  static constexpr uint32_t kVChunkStep = kTma ? kVChunk / 2 : kVChunk;
  static constexpr uint32_t kVHalfGap = kTma ? kVStage / 2 - kVChunk / 2 : 0;
  // P tiles: the staged e4m3 rows leave room for one
  static constexpr uint32_t kPTiles = kCache == kE4m3 ? 1 : 2;
  static constexpr uint32_t OFF_STG = OFF_P + kPTiles * kPTile;
  // a staging stage: own rows' codes, other rows' V codes, scales of the tile's two halves
  static constexpr uint32_t STG_OWN = 0;
  static constexpr uint32_t STG_OTHER = STG_OWN + kHalf * kCodeBytes;
  static constexpr uint32_t STG_SCALES = STG_OTHER + kHalf * kVBytes;
  static constexpr uint32_t kStage = STG_SCALES + kTile * kScaleBytes;
  // bf16: three stages of K, the third where the others have their staging.  (K of
  // tile g + 2 can go out when QK of g is done, and QK of g + 2 wants it some 500
  // cycles later; a third stage gives its copy a whole tile.)
  static constexpr uint32_t OFF_K2 = OFF_STG;
  static constexpr uint32_t OFF_BARS = OFF_STG + (kTma ? kKStage : 2 * kStage);
  static constexpr uint32_t OFF_XMAX = OFF_BARS + 384;              // float [4][128]: tile maxima by tile mod 4
  static constexpr uint32_t OFF_MREF = OFF_XMAX + 4 * 128 * 4;      // float [2][64]: references by tile parity
  static constexpr uint32_t OFF_XSUM = OFF_MREF + 2 * kCtaRows * 4;  // float [2][3][128]: (sum, reference, sum of the rounded P) by group
  static constexpr uint32_t OFF_QSCALE = OFF_XSUM + 6 * 128 * 4;    // float [4][64]: 2^-k by item
  static constexpr uint32_t OFF_TMEM = OFF_QSCALE + 4 * kCtaRows * 4;
  static constexpr uint32_t OFF_ABORT = OFF_TMEM + 8;
  static constexpr uint32_t OFF_MASK = OFF_ABORT + 8;  // uint32 [2][2]: rows in use, by stage and half
  static constexpr uint32_t kSmemBytes = OFF_MASK + 16;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert((kTma ? OFF_K2 % 1024 == 0 : OFF_STG % 16 == 0) && kStage % 16 == 0 && STG_OTHER % 16 == 0 && STG_SCALES % 16 == 0 &&
                    OFF_BARS % 8 == 0,
                "alignment");
};
static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_P % 1024 == 0, "alignment");

// TMEM columns
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_O = 0;    // lane: query row (mod 64) and V half; 256 V dims
constexpr uint32_t TM_S = 256;  // two 32-column buffers; lane: query row and KV half
constexpr uint32_t TM_Q = 320;  // chunks 0..5 of the query row (mod 64), pairs of f16

enum Bar {
  STG_FULL0, STG_EMPTY0 = STG_FULL0 + 2,  // by tile parity (TMA: unused, V landed)
  K_FULL0 = STG_EMPTY0 + 2,   // even CTA: [tile parity][3], both CTAs' chunks are there
  V_FULL0 = K_FULL0 + 2 * (kChunks / kGroup),  // even CTA
  PV_DONE0 = V_FULL0 + 2,              // by tile parity: V stage and P free, O stable
  S_FULL0 = PV_DONE0 + 2,              // S computed, K stage free
  S_EMPTY0 = S_FULL0 + 2,              // even CTA
  P_FULL0 = S_EMPTY0 + 2,              // even CTA
  Q_FULL = P_FULL0 + 2, Q_EMPTY,       // Q_FULL: even CTA
  QX,                                  // a query's scales (and shared-memory chunks) are written
  QS_FULL0,                            // 4: by item, the same for the softmax
  XM0 = QS_FULL0 + 4,                  // 4: [tile parity][pair of warps] maxima exchanged
  MR0 = XM0 + 4,                       // 4: the same, reference published
  XS0 = MR0 + 4,                       // 2: [pair] row sums exchanged
  EPI = XS0 + 2,                       // the partial is written
  DRAIN0,                              // 2: every MMA of an issuing warp has completed
  QSTG = DRAIN0 + 2, Q_READ,           // the block's first query is staged; has been read
  KE0,                                 // TMA, 3: by tile mod 3, QK has read the K stage
  NUM_BARS = KE0 + 3,
  K_TMA0 = K_FULL0 + 3                 // TMA, 3: by tile mod 3, K landed (K_FULL0: by tile mod 3, too)
};
static_assert(kChunks / kGroup == 3 && NUM_BARS * 8 <= 384, "barrier area");

struct Ctx {
  uint64_t* bars;
  volatile int* abort;
  uint32_t peer_abort;
  uint32_t leader_bars;  // shared::cluster address of the even CTA's barriers
  int* status;
};

// A wait ran out, here or in the other CTA: make both CTAs unwind.
__device__ __forceinline__ void tell_abort(const Ctx& c) {
  *c.abort = 1;
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(c.peer_abort), "r"(1) : "memory");
}
// False after too many polls, or once either CTA has given up; the caller then
// leaves its role, and the block gives up at its end (kept out of the loops: their
// code competes for the instruction cache).
__device__ __forceinline__ bool wait_bar(const Ctx& c, int bar, uint32_t parity) {
  uint64_t* b = &c.bars[bar];
  for (uint32_t i = kWaitLimit; !mbar_try_wait(b, parity); --i)
    if (i == 0 || ((i & 1023) == 0 && *c.abort)) return false;
  return true;
}
// The same on a barrier that both CTAs' threads arrive at (arrive_leader).
__device__ __forceinline__ bool wait_pair(const Ctx& c, int bar, uint32_t parity) {
  uint64_t* b = &c.bars[bar];
  for (uint32_t i = kWaitLimit; !mbar_try_wait_pair(b, parity); --i)
    if (i == 0 || ((i & 1023) == 0 && *c.abort)) return false;
  fence_acquire_pair();
  return true;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit; ++i)
    if (mbar_try_wait(bar, parity)) return;
}
// One lane's arrival for its warp, after __syncwarp (see mbar_arrive_pair).
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
// The f16 values of two e4m3 codes, each in both halves of a word.
__device__ __forceinline__ void scale_pairs(uint32_t codes, uint32_t& s0, uint32_t& s1) {
  uint32_t h;
  asm("{\n .reg .b16 lo;\n mov.b32 {lo, _}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(codes));
  s0 = __byte_perm(h, h, 0x1010);
  s1 = __byte_perm(h, h, 0x3232);
}
// Eight codes times their scale, as a 16-byte unit of f16.
__device__ __forceinline__ uint4 convert8(uint32_t codes, uint32_t scale) {
  uint32_t h[4];
  e2m1x8_to_f16x2(codes, h);
  return make_uint4(hmul2(h[0], scale), hmul2(h[1], scale), hmul2(h[2], scale), hmul2(h[3], scale));
}
// 64 codes and their four scales.
__device__ __forceinline__ void convert64(const uint4 a, const uint4 b, uint32_t scales, uint4 (&x)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t s0, s1;
    scale_pairs(scales >> (16 * e), s0, s1);
    x[4 * e] = convert8(w[4 * e], s0);
    x[4 * e + 1] = convert8(w[4 * e + 1], s0);
    x[4 * e + 2] = convert8(w[4 * e + 2], s1);
    x[4 * e + 3] = convert8(w[4 * e + 3], s1);
  }
}
// Unit `unit` (16 bytes) of a 128-byte row r in the 128B-swizzled layout: at
// unit ^ (r mod 8).  `row` is swizzled_row's address, so a store takes one XOR.
__device__ __forceinline__ uint32_t swizzled_row(uint32_t tile, int r) {
  return tile + 128 * r + ((r & 7) << 4);
}
__device__ __forceinline__ void put(uint32_t row, int unit, uint4 v) {
  st_shared_v4(row ^ (unit << 4), v);
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
__device__ __forceinline__ void exchange(uint4& a, uint4& b, bool on) {
  const uint4 t = a;
  a = on ? b : a;
  b = on ? t : b;
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

__device__ __forceinline__ uint4 e4m3x8_to_bf16(const uint2 x) {
  return make_uint4(e4m3x2_to_bf16x2(x.x & 0xFFFFu), e4m3x2_to_bf16x2(x.x >> 16),
                    e4m3x2_to_bf16x2(x.y & 0xFFFFu), e4m3x2_to_bf16x2(x.y >> 16));
}
// A word whose first n bits are set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}
// 16 e4m3 codes as two 16-byte units of f16.
__device__ __forceinline__ void widen16(const uint4 c, uint4& a, uint4& b) {
  a = e4m3x8_to_f16(make_uint2(c.x, c.y));
  b = e4m3x8_to_f16(make_uint2(c.z, c.w));
}

// A work item's query, rows [64 rank, 64 rank + 64), where it is read from.
struct Query {
  const unsigned char* base;  // row 0, in global or in shared memory
  int pitch, n;               // bytes from row to row; rows (the others are zeros)
  int fp8;
  __device__ uint4 unit(int r, int u) const {  // eight dims, raw
    if (r >= n) return make_uint4(0, 0, 0, 0);
    const unsigned char* at = base + r * pitch;
    if (fp8) {
      const uint2 v = reinterpret_cast<const uint2*>(at)[u];
      return make_uint4(v.x, v.y, 0, 0);
    }
    return reinterpret_cast<const uint4*>(at)[u];
  }
};

// The block's first query, from rows staged in shared memory (see below).  A
// function of its own leaves the conversion loops their registers: inlined, those
// spilled and a long call took 6% more.
template <int kCache>
__device__ __noinline__ bool first_query(Ctx c, unsigned char* sm, uint32_t tmem, Query q, int w) {
  const int lane = threadIdx.x & 31, quad = (kFirstConv + w) & 3;
  float* scales = reinterpret_cast<float*>(sm + Cfg<kCache>::OFF_QSCALE);
  if (!wait_bar(c, QSTG, 0)) return false;
  // the rows' factors 2^-k: four rows a warp, a row's 72 units over its lanes
#pragma unroll 1
  for (int r = 4 * w; r < 4 * w + 4; ++r) {
    int e = 0;
    if (!q.fp8 && kCache != kBf16) {
      const uint4 a = q.unit(r, lane), b = q.unit(r, 32 + lane), d = q.unit(r, 64 + (lane & 7));
      uint32_t mb = __vmaxu2(__vmaxu2(max_bits(a), max_bits(b)), max_bits(d));
      mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
      e = query_exponent(mb);
    }
    if (lane == 0) scales[r] = __uint_as_float((uint32_t)(127 - e) << 23);
  }
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(&c.bars[QX]);
    mbar_arrive(&c.bars[QS_FULL0]);
  }
  if (!wait_bar(c, QX, 0)) return false;
  auto as_operand = [&](const uint4 x, float up) {  // f16, or bf16 for bf16 MMAs
    if constexpr (Cfg<kCache>::kTma) return q.fp8 ? e4m3x8_to_bf16(make_uint2(x.x, x.y)) : x;
    return q.fp8 ? e4m3x8_to_f16(make_uint2(x.x, x.y)) : bf16x8_to_f16(x, up);
  };
  // as in load_query
  const int row = (32 * quad + lane) & 63, part = w >> 2;
  const float up = 1.f / scales[row];
  const uint32_t tq = tmem + ((uint32_t)(32 * quad) << 16) + TM_Q + 48 * part;
  constexpr int kPerRow = 8 * (kChunks - kTmemChunks);
#pragma unroll 1
  for (int j = 0; j < 3; ++j) {
    uint4 f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = as_operand(q.unit(row, 12 * part + 4 * j + u), up);
    tmem_st_32x32b_x16(tq + 16 * j, *reinterpret_cast<const uint32_t(*)[16]>(f));
    const int at = 32 * (kConvWarps * j + w) + lane, r = at / kPerRow, u2 = at - r * kPerRow;
    put(swizzled_row(smem_u32(sm) + OFF_Q + (u2 >> 3) * kQChunk, r), u2 & 7,
        as_operand(q.unit(r, 8 * kTmemChunks + u2), 1.f / scales[r]));
  }
  fence_proxy_async_smem();
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    arrive_leader(c, Q_FULL, 1);
    mbar_arrive(&c.bars[Q_READ]);
  }
  return wait_bar(c, Q_READ, 0);  // K and V may go where it was staged
}

}  // namespace

template <int kCache>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode_pair_kernel(const Problem p, const Layout lay, char* __restrict__ ws,
                   const __grid_constant__ CUtensorMap tm_k,   // (bf16 cache only)
                   const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<kCache>;
  // The swizzled tiles need 1024-byte alignment, and there is no room to round
  // up: the block has no other shared memory, so its dynamic part starts at
  // offset 0 of its window.  A block placed otherwise reports and leaves.
  extern __shared__ __align__(1024) unsigned char sm[];
  if ((smem_u32(sm) & 1023) != 0) {
    pdl_wait();  // the partitioner writes the whole status word
    if (threadIdx.x == 0) atomicOr(reinterpret_cast<int*>(ws) + kHdrStatus, kStatusTimeout);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int worker = (int)cluster_id_x();
  const WorkItem* items = reinterpret_cast<const WorkItem*>(ws + lay.items);
  const int* worker_begin = reinterpret_cast<const int*>(ws + lay.worker_ranges);

  Ctx c;
  c.bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BARS);
  c.abort = reinterpret_cast<volatile int*>(sm + C::OFF_ABORT);
  c.peer_abort = map_to_rank(smem_u32(sm + C::OFF_ABORT), rank ^ 1);
  c.leader_bars = map_to_rank(smem_u32(sm + C::OFF_BARS), 0);
  c.status = reinterpret_cast<int*>(ws) + kHdrStatus;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_TMEM);
  volatile uint32_t* row_mask = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MASK);

  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      uint32_t n = 1;  // one commit, or one warp
      if (i >= STG_FULL0 && i < STG_EMPTY0) n = C::kTma ? 1 : 1 + 32;  // bulk copies, each lane's own
      if (i >= STG_EMPTY0 && i < K_FULL0) n = C::kTma ? 1 : kConvWarps / 2;
      // a latent chunk's warp counts four times, as the RoPE chunk has four warps
      if (i >= K_FULL0 && i < V_FULL0) n = !C::kTma ? 2 * 4 * kGroup : i < K_TMA0 ? 2 : 1;
      if (i >= V_FULL0 && i < V_FULL0 + 2) n = C::kTma ? 2 : kConvWarps;  // half the warps of both CTAs
      if (i >= S_EMPTY0 && i < P_FULL0 + 2) n = kSoftWarps;  // half the warps of both CTAs
      if (i == Q_FULL) n = 2 * kConvWarps;
      if (i == QX || (i >= QS_FULL0 && i < QS_FULL0 + 4)) n = kConvWarps;
      if (i >= XM0 && i < XM0 + 4) n = 2;
      if (i >= XS0 && i < XS0 + 2) n = 4;
      if (i == EPI) n = kSoftWarps;
      if (i == QSTG) n = kCtaRows;
      if (i == Q_READ) n = kConvWarps;
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
  const int h_shift = __ffs(H) - 1;  // a power of two

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ copies
    // Page ids a batch of 32 ahead (one per lane), as virtual page slots of the
    // item.  Warp 0's lane 0 issues the bulk copies: codes of the own rows, scales.
    // Warp 3 fetches the other rows' V codes, 128 bytes of each 288, by 16-byte
    // copies (one bulk copy a row took 4000 cycles to issue), and brings later
    // tiles to L2.
    const bool bulk = warp == 0;
    const int ps = p.page_size, ps_shift = ps == kTile ? 6 : 5, npg = kTile >> ps_shift;
    const size_t page_bytes = (size_t)ps * C::kRowBytes;
    const unsigned char* cache = static_cast<const unsigned char*>(p.kv_cache);
    uint32_t g = 0;
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      const Walk walk(p, it);
      const int* bt = p.block_tables + (size_t)it.b * p.max_pages;
      const int n_pages = (it.kv_end - it.kv_begin + ps - 1) >> ps_shift;
      // a page's id, -1 for one that is not read; a bad id's rows are zeros (TMA:
      // the rows past the cache's end, which the copy fills with zeros)
      auto page_at = [&](int i) -> int {
        const int r = walk.row(it.kv_begin + i * ps);
        if (i >= n_pages || !walk.seen(r, r + ps - 1)) return -1;
        const int id = bt[r >> ps_shift];
        if (id >= 0 && (long long)id < p.num_pages) return id;
        if (bulk) atomicOr(c.status, kStatusPage);
        return C::kTma ? (int)p.num_pages : -1;
      };
      int cur = page_at(lane), nxt = page_at(32 + lane);
      for (int t = 0; t < nt; ++t, ++g) {
        const int slot0 = t * npg;  // never straddles a batch: npg divides 32
        if (slot0 > 0 && (slot0 & 31) == 0) {
          cur = nxt;
          nxt = page_at(slot0 + 32 + lane);
        }
        const int id0 = __shfl_sync(0xffffffffu, cur, slot0 & 31);
        const int id1 = __shfl_sync(0xffffffffu, cur, (slot0 + npg - 1) & 31);
        // a half is read if some query row sees a row of it
        const int j0 = it.kv_begin + t * kTile, r0 = walk.row(j0);
        const bool on0 = id0 >= 0 && walk.seen(r0, r0 + kHalf - 1);
        const bool on1 = id1 >= 0 && j0 + kHalf < it.kv_end && walk.seen(r0 + kHalf, r0 + kTile - 1);
        const uint32_t s = g & 1, use = g >> 1;
        unsigned char* stg = sm + C::OFF_STG + s * C::kStage;
        uint64_t* full = &c.bars[STG_FULL0 + s];
        if constexpr (C::kTma) {
          const int row1 = npg == 1 ? kHalf : 0;  // first row of half 1 in its page
          const int y0 = id0 * ps, y1 = id1 * ps + row1;
          if (bulk) {
            // K: the own rows' nine chunks, once QK of three tiles ago has read the stage
            const uint32_t use3 = g / 3, s3 = g - 3 * use3;
            if (!wait_bar(c, KE0 + s3, (use3 & 1) ^ 1)) goto fail_copy;
            if (lane == 0) {
              const bool own = rank == 0 ? on0 : on1;
              unsigned char* dst = sm + (s3 == 2 ? C::OFF_K2 : OFF_K + s3 * kKStage);
              mbar_arrive_expect_tx(&c.bars[K_TMA0 + s3], own ? kKStage : 0);
              if (own) tma_load_3d(dst, &tm_k, 0, rank == 0 ? y0 : y1, 0, &c.bars[K_TMA0 + s3]);
            }
          } else {
            // V: this CTA's dims of all rows, once PV of two tiles ago has, and the
            // first query, which is staged there
            const uint32_t mask0 = __ballot_sync(0xffffffffu, on0 && j0 + lane < it.kv_end &&
                                                                  walk.seen(r0 + lane, r0 + lane));
            const uint32_t mask1 =
                __ballot_sync(0xffffffffu, on1 && j0 + kHalf + lane < it.kv_end &&
                                               walk.seen(r0 + kHalf + lane, r0 + kHalf + lane));
            if (g == 0 && !wait_bar(c, Q_READ, 0)) goto fail_copy;
            if (!wait_bar(c, PV_DONE0 + s, (use & 1) ^ 1)) goto fail_copy;
            if (lane == 0) {
              uint64_t* v_full = &c.bars[STG_EMPTY0 + s];
              row_mask[2 * s] = mask0;
              row_mask[2 * s + 1] = mask1;
              mbar_arrive_expect_tx(v_full, ((on0 ? 1 : 0) + (on1 ? 1 : 0)) * (kVStage / 2));
              unsigned char* dst = sm + OFF_V + s * kVStage;
              if (on0) tma_load_3d(dst, &tm_v, 0, y0, 4 * rank, v_full);
              if (on1) tma_load_3d(dst + kVStage / 2, &tm_v, 0, y1, 4 * rank, v_full);
            }
            // (not before the block's first tile is there: the prefetches of all blocks
            // would queue in front of it)
            if (g == 1 && !wait_bar(c, STG_EMPTY0, 0)) goto fail_copy;
            for (int a = g == 0 ? kAhead + 1 : g == 1 ? 1 : t == 0 ? 2 : kAhead; a <= kAhead; ++a) {
              const int i = (t + a) * npg + (npg == 2 ? rank : 0);
              const int from = __shfl_sync(0xffffffffu, (i >> 5) == (slot0 >> 5) ? cur : nxt, i & 31);
              if (t + a < nt && lane == 0 && from >= 0 && from < p.num_pages)
                bulk_prefetch_l2(cache + (size_t)from * page_bytes + (npg == 2 ? 0 : kHalf * rank) * C::kCodeBytes,
                                 kHalf * C::kCodeBytes);
            }
          }
          __syncwarp();
        } else if (bulk) {
          // rows past the item's end, that no query row sees, or on a page that is
          // not read, enter as zeros
          const uint32_t mask0 = __ballot_sync(0xffffffffu, on0 && j0 + lane < it.kv_end &&
                                                                walk.seen(r0 + lane, r0 + lane));
          const uint32_t mask1 =
              __ballot_sync(0xffffffffu, on1 && j0 + kHalf + lane < it.kv_end &&
                                             walk.seen(r0 + kHalf + lane, r0 + kHalf + lane));
          if (!wait_bar(c, STG_EMPTY0 + s, (use & 1) ^ 1)) goto fail_copy;
          if (lane == 0) {
            const int row1 = npg == 1 ? kHalf : 0;  // first row of half 1 in its page
            const unsigned char* pg0 = cache + (size_t)(on0 ? id0 : 0) * page_bytes;
            const unsigned char* pg1 = cache + (size_t)(on1 ? id1 : 0) * page_bytes;
            const unsigned char* sc0 = pg0 + (size_t)ps * C::kCodeBytes;
            const unsigned char* sc1 = pg1 + (size_t)ps * C::kCodeBytes + row1 * C::kScaleBytes;
            constexpr uint32_t kScales = kHalf * C::kScaleBytes, kCodes = kHalf * C::kCodeBytes;
            const bool own = rank == 0 ? on0 : on1;
            row_mask[2 * s] = mask0;
            row_mask[2 * s + 1] = mask1;
            mbar_arrive_expect_tx(full, (on0 ? kScales : 0) + (on1 ? kScales : 0) + (own ? kCodes : 0));
            if (own) bulk_load(stg + C::STG_OWN, rank == 0 ? pg0 : pg1 + row1 * C::kCodeBytes, kCodes, full);
            if constexpr (kCache == kE4m3) {
              // (no scales)
            } else if (on0 && on1 && npg == 1) {
              bulk_load(stg + C::STG_SCALES, sc0, 2 * kScales, full);
            } else {
              if (on0) bulk_load(stg + C::STG_SCALES, sc0, kScales, full);
              if (on1) bulk_load(stg + C::STG_SCALES + kScales, sc1, kScales, full);
            }
          }
          __syncwarp();
        } else {
          if (!wait_bar(c, STG_EMPTY0 + s, (use & 1) ^ 1)) goto fail_copy;
          // kUnits 16-byte units of a row: kUnits lanes a row.  Unit u of row r goes to
          // u ^ (r mod 8), so that eight rows' reads of one unit meet eight bank groups
          if (rank == 0 ? on1 : on0) {
            constexpr int kUnits = C::kVBytes / 16, kRowsAStep = 32 / kUnits;
            const int u = lane % kUnits, r0u = lane / kUnits;
            const unsigned char* src = cache + (size_t)(rank == 0 ? id1 : id0) * page_bytes +
                                       (rank == 0 && npg == 1 ? kHalf * C::kCodeBytes : 0) +
                                       C::kVBytes * rank + 16 * u;
            unsigned char* dst = stg + C::STG_OTHER;
#pragma unroll
            for (int i = 0; i < kHalf / kRowsAStep; ++i) {
              const int r = i * kRowsAStep + r0u;
              cp_async_16(dst + r * C::kVBytes + ((u ^ (r & 7)) << 4), src + r * C::kCodeBytes);
            }
          }
          cp_async_arrive(full);
          // this CTA's half of the tiles up to kAhead on, to L2: the staged tiles
          // cover an L2 round trip but not one to HBM
          for (int a = t == 0 ? 2 : kAhead; a <= kAhead; ++a) {
            const int i = (t + a) * npg + (npg == 2 ? rank : 0);
            const int from = __shfl_sync(0xffffffffu, (i >> 5) == (slot0 >> 5) ? cur : nxt, i & 31);
            if (t + a < nt && lane < (kCache == kFp4 ? 2 : 1) && from >= 0) {
              const unsigned char* pg = cache + (size_t)from * page_bytes;
              const int r = npg == 2 ? 0 : kHalf * rank;
              bulk_prefetch_l2(lane == 0 ? pg + r * C::kCodeBytes
                                         : pg + (size_t)ps * C::kCodeBytes + r * C::kScaleBytes,
                               kHalf * (lane == 0 ? C::kCodeBytes : C::kScaleBytes));
            }
          }
        }
      }
    }
    goto done_copy;
  fail_copy:
    tell_abort(c);
  done_copy:
    // no copy issued here may still be landing when the CTA leaves
    for (uint32_t k = 0; k < (C::kTma && bulk ? 3 : 2) && k < g; ++k) {
      const uint32_t gi = g - 1 - k;
      if (C::kTma && bulk)
        drain_wait(&c.bars[K_TMA0 + gi % 3], (gi / 3) & 1);
      else
        drain_wait(&c.bars[(C::kTma ? STG_EMPTY0 : STG_FULL0) + (gi & 1)], (gi >> 1) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issue
    // The whole warp walks the loops and one lane issues (see elect_one).
    if (rank == 0) {
      constexpr uint32_t idesc = C::kTma ? idesc_f16(kRows, kTile, false, false) : idesc_half(kRows, kTile, false, false);
      // operand descriptors; a step along an operand adds its bytes / 16
      const uint64_t q_desc = smem_desc(smem_u32(sm + OFF_Q), 16, 1024, kSwizzle128B);
      const uint64_t k_desc = smem_desc(smem_u32(sm + OFF_K), 16, 1024, kSwizzle128B);
      uint32_t g = 0;
      int n_item = 0;
      for (int idx = item_begin; idx < item_end; ++idx) {
        const int nt = __shfl_sync(0xffffffffu, n_tiles_of(items[idx]), 0);
        if (nt <= 0) continue;
        if (!wait_pair(c, Q_FULL, n_item & 1)) goto fail_qk;
        ++n_item;
        for (int t = 0; t < nt; ++t, ++g) {
          const uint32_t sb = g & 1;
          if (!wait_pair(c, S_EMPTY0 + sb, ((g >> 1) & 1) ^ 1)) goto fail_qk;
          const uint32_t use3 = g / 3, s3 = g - 3 * use3;  // (TMA)
          const uint64_t kd = k_desc + (!C::kTma     ? sb * (kKStage >> 4)
                                        : s3 == 2 ? (C::OFF_K2 - OFF_K) >> 4
                                                  : s3 * (kKStage >> 4));
#pragma unroll
          for (int k3 = 0; k3 < kChunks / kGroup; ++k3) {
            if constexpr (C::kTma) {
              if (k3 == 0 && !wait_pair(c, K_FULL0 + s3, use3 & 1)) goto fail_qk;
            } else {
              if (!wait_pair(c, K_FULL0 + sb * (kChunks / kGroup) + k3, (g >> 1) & 1)) goto fail_qk;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = kGroup * k3; k < kGroup * (k3 + 1); ++k)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                  const uint64_t b_desc = kd + (k * kKChunk >> 4) + 2 * ks;
                  if (k < kTmemChunks)
                    mma_f16_pair_ts(tmem + TM_S + 32 * sb, tmem + TM_Q + 32 * k + 8 * ks, b_desc, idesc,
                                    (k | ks) != 0 ? 1u : 0u);
                  else
                    mma_f16_pair_ss(tmem + TM_S + 32 * sb,
                                    q_desc + ((k - kTmemChunks) * kQChunk >> 4) + 2 * ks, b_desc, idesc, 1u);
                }
              if (k3 == kChunks / kGroup - 1) {
                mma_commit_pair(&c.bars[S_FULL0 + sb]);
                if (C::kTma) mma_commit_pair(&c.bars[KE0 + s3]);
                if (t + 1 == nt) mma_commit_pair(&c.bars[Q_EMPTY]);
              }
            }
            __syncwarp();
          }
        }
      }
      goto done_qk;
    fail_qk:
      tell_abort(c);
    done_qk:
      __syncwarp();
      if (elect_one()) mma_commit_pair(&c.bars[DRAIN0]);
      drain_wait(&c.bars[DRAIN0], 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ PV issue
    // A warp of its own: its waits for P would hold up the next tile's QK.
    if (rank == 0) {
      constexpr uint32_t idesc = C::kTma ? idesc_f16(kRows, 256, false, true) : idesc_half(kRows, 256, false, true);
      const uint64_t p_desc = smem_desc(smem_u32(sm + OFF_P), 16, 1024, kSwizzle128B);
      const uint64_t v_desc = smem_desc(smem_u32(sm + OFF_V), C::kVChunkStep, 1024, kSwizzle128B);
      uint32_t g = 0;
      for (int idx = item_begin; idx < item_end; ++idx) {
        const int nt = __shfl_sync(0xffffffffu, n_tiles_of(items[idx]), 0);
        for (int t = 0; t < nt; ++t, ++g) {
          const uint32_t s = g & 1;
          if (!wait_pair(c, V_FULL0 + s, (g >> 1) & 1)) goto fail_pv;
          if (!wait_pair(c, P_FULL0 + s, (g >> 1) & 1)) goto fail_pv;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t v = v_desc + s * (kVStage >> 4);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_f16_pair_ss(tmem + TM_O + 128 * j, p_desc + (C::kPTiles == 2 ? s * (kPTile >> 4) : 0) + 2 * ks,
                                v + ((j * 2 * C::kVChunkStep + ks * 16 * 128 + (ks >> 1) * C::kVHalfGap) >> 4), idesc,
                                (t == 0 && ks == 0) ? 0u : 1u);
            mma_commit_pair(&c.bars[PV_DONE0 + s]);
          }
          __syncwarp();
        }
      }
      goto done_pv;
    fail_pv:
      tell_abort(c);
    done_pv:
      __syncwarp();
      if (elect_one()) mma_commit_pair(&c.bars[DRAIN0 + 1]);
      drain_wait(&c.bars[DRAIN0 + 1], 0);
    }
  } else if (warp < kFirstConv) {
    // ------------------------------------------------------------ softmax, correction, epilogue
    // Two groups of four warps take alternate tiles.  Thread = TMEM lane l = 32
    // (warp mod 4) + lane: query row l mod 64 of the CTA and KV rows (columns of S)
    // 32 (l / 64) + [0, 32).  The row's other thread is in warp ^ 2 of the group;
    // the running reference passes from tile to tile, and so between the groups,
    // through shared memory.
    const int quad = warp & 3, grp = (warp - kFirstSoft) >> 2;
    const int l = 32 * quad + lane, hh = quad >> 1, row = l & 63;
    const int q = kCtaRows * rank + row;  // row of the work item
    const int pair = quad & 1;
    const uint32_t tm = tmem + ((uint32_t)(32 * quad) << 16);
    const float bmm1 = run_bmm1(p, c.status) * kLog2e;
    const float bmm2 = run_bmm2(p);
    const int W = max(p.cp_world, 1);
    float* mref = reinterpret_cast<float*>(sm + C::OFF_MREF);
    float* xsum = reinterpret_cast<float*>(sm + C::OFF_XSUM);
    const float* qscale = reinterpret_cast<const float*>(sm + C::OFF_QSCALE);
    const uint32_t prow = swizzled_row(smem_u32(sm) + OFF_P + (C::kPTiles == 2 ? kPTile * grp : 0), row);
    uint4* part_o = reinterpret_cast<uint4*>(ws + lay.part_o);
    float* part_lse = reinterpret_cast<float*>(ws + lay.part_lse);
    int* comb_done = reinterpret_cast<int*>(ws + lay.comb_done);
    uint32_t g = 0;
    int n_item = 0;
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      const Walk walk(p, it);
      const int rows_total = it.q_len * H, row0 = it.g * kRows;
      const int n_rows = min(kRows, rows_total - row0);
      const bool row_ok = q < n_rows;
      auto last_of = [&](int r) {
        return p.causal ? causal_last(it.mask_base, (row0 + r) >> h_shift, W) : it.seq_len - 1;
      };
      const int last = last_of(min(q, n_rows - 1));
      const int low = p.window > 0 ? last - p.window + 1 : -1;  // first row of the window
      // tiles inside [clean_lo, clean_hi) need no mask for any row of the item
      const int clean_hi = last_of(0) + 1;
      const int clean_lo = p.window > 0 ? last_of(n_rows - 1) - p.window + 1 : INT_MIN;
      if (!wait_bar(c, QS_FULL0 + (n_item & 3), (n_item >> 2) & 1)) goto fail_soft;
      const float scale = bmm1 * qscale[(n_item & 3) * kCtaRows + row];
      // this group's share of the row sum, relative to its latest reference m
      // (bf16: and the sum of P as it is rounded, by which O is divided: the rounding of a
      // row's large P, 2^-8 of each, then cancels, where the exact sum keeps it whole)
      float m = -INFINITY, l_part = 0.f, r_part = 0.f;
      for (int t = 0; t < nt; ++t, ++g) {
        if ((int)(g & 1) != grp) continue;
        if (!wait_bar(c, S_FULL0 + grp, (g >> 1) & 1)) goto fail_soft;
        tc_fence_after();
        uint32_t v[32];
        tmem_ld_32x32b_x32(tm + TM_S + 32 * grp, v);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        // (relaxed: what was read is in registers)
        if (lane == 0) mbar_arrive_cluster_relaxed(c.leader_bars + 8u * (S_EMPTY0 + grp));
        const int v0 = it.kv_begin + t * kTile;        // virtual row of the tile
        const int r0 = walk.row(v0);                    // its row
        const int valid = it.kv_end - v0;               // rows of the tile inside the item
        const bool clean = valid >= kTile && r0 + kTile <= clean_hi &&
                           (r0 >= clean_lo || r0 + kTile <= p.sinks);
        uint32_t hidden = 0;  // columns that the mask takes out
        if (!clean) {
          // of this thread's columns, rows r0 + 32 hh + [0, 32): those up to `last` and
          // inside the item, from the window's first row on or among the sinks
          const int at = r0 + 32 * hh;
          hidden = ~(first_bits(min(last + 1 - at, valid - 32 * hh)) &
                     (~first_bits(low - at) | first_bits(p.sinks - at)));
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if ((hidden >> j) & 1u) v[j] = 0xFF800000u;  // -inf
        }
        float mt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mt[j] = __uint_as_float(v[j]);
#pragma unroll
        for (int j = 4; j < 32; ++j) mt[j & 3] = fmaxf(mt[j & 3], __uint_as_float(v[j]));
        // (four buffers: a partner that still reads the maxima of tile g has let QK
        // of tile g + 2 into S, but not of g + 4)
        float* xmax = reinterpret_cast<float*>(sm + C::OFF_XMAX) + 128 * (g & 3);
        xmax[l] = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
        // The reference after the previous tile, which the other group had.  Every
        // tile but the very first waits for it, and before its own maximum goes
        // out, so that the barriers' phases stay in step.
        float m_prev = -INFINITY;
        if (g > 0) {
          if (!wait_bar(c, MR0 + 2 * (grp ^ 1) + pair, ((g - 1) >> 1) & 1)) goto fail_soft;
          if (t > 0) m_prev = mref[kCtaRows * (grp ^ 1) + row];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bars[XM0 + 2 * grp + pair]);
        if (!wait_bar(c, XM0 + 2 * grp + pair, (g >> 1) & 1)) goto fail_soft;
        // (both from shared memory: the same result in the row's two threads; the
        // scale is not negative, so it may come after the maximum)
        const float m_raw = fmaxf(xmax[row], xmax[row + 64]);
        const float m_tile = m_raw == -INFINITY ? m_raw : m_raw * scale;
        const float m_new = (m_tile > m_prev + kRescaleThreshold || t == 0) ? m_tile : m_prev;
        if (hh == 0) {
          mref[kCtaRows * grp + row] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.bars[MR0 + 2 * grp + pair]);
        }
        const bool need = t > 0 && m_new != m_prev;
        if (m_new > m) {  // rebase this group's share (0 while m = -inf)
          const float f = ex2(m - m_new);
          l_part *= f;
          r_part *= f;
          m = m_new;
        }
        const float ref = C::kPShift - (m == -INFINITY ? 0.f : m);
        // (rows past the request's own compute something that nothing reads)
        const uint64_t scale2 = pack_f32x2(scale, scale), ref2 = pack_f32x2(ref, ref);
        uint64_t rs[2] = {0, 0}, rr = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float a, b;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), scale2, ref2), a, b);
          a = ex2(a);
          b = ex2(b);
          if (!clean) {  // (-inf times a scale of zero is no zero)
            if ((hidden >> (2 * j)) & 1u) a = 0.f;
            if ((hidden >> (2 * j + 1)) & 1u) b = 0.f;
          }
          rs[j & 1] = add_f32x2(rs[j & 1], pack_f32x2(a, b));
          if constexpr (C::kTma) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            v[j] = *reinterpret_cast<const uint32_t*>(&h);
            rr = add_f32x2(rr, pack_f32x2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xFFFF0000u)));
          } else {
            const __half2 h = __floats2half2_rn(a, b);
            v[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        {
          float a, b;
          unpack_f32x2(add_f32x2(rs[0], rs[1]), a, b);
          l_part += a + b;
          if constexpr (C::kTma) {
            unpack_f32x2(rr, a, b);
            r_part += a + b;
          }
        }
        // this P tile has been read
        if constexpr (C::kPTiles == 2) {
          if (!wait_bar(c, PV_DONE0 + grp, ((g >> 1) & 1) ^ 1)) goto fail_soft;
        } else {
          if (g > 0 && !wait_bar(c, PV_DONE0 + (grp ^ 1), ((g - 1) >> 1) & 1)) goto fail_soft;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          put(prow, 4 * hh + u, make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]));
        if (__any_sync(0xffffffffu, need)) {
          // O, stable once PV of the previous tile is done, to the new reference
          if (!wait_bar(c, PV_DONE0 + (grp ^ 1), ((g - 1) >> 1) & 1)) goto fail_soft;
          tc_fence_after();
          const float f = need ? ex2(m_prev - m_new) : 1.f;  // m_prev = -inf: 0
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            uint32_t x[16];
            tmem_ld_32x32b_x16(tm + TM_O + 16 * k, x);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
            tmem_st_32x32b_x16(tm + TM_O + 16 * k, x);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) arrive_leader(c, P_FULL0 + grp, 1);
      }
      // the row's sum: two threads of each group, each relative to its reference
      xsum[384 * grp + l] = l_part;
      xsum[384 * grp + 128 + l] = m;
      if constexpr (C::kTma) xsum[384 * grp + 256 + l] = r_part;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.bars[XS0 + pair]);
      if (!wait_bar(c, XS0 + pair, n_item & 1)) goto fail_soft;
      float m_fin, l_row = 0.f, r_row = 0.f;
      {
        const float m0 = xsum[128 + row], m1 = xsum[384 + 128 + row];
        m_fin = fmaxf(m0, m1);  // a reference never falls within an item
        const float f0 = m0 != -INFINITY ? ex2(m0 - m_fin) : 0.f, f1 = m1 != -INFINITY ? ex2(m1 - m_fin) : 0.f;
        auto joined = [&](int at) {
          return (xsum[at + row] + xsum[at + row + 64]) * f0 + (xsum[384 + at + row] + xsum[384 + at + row + 64]) * f1;
        };
        l_row = joined(0);
        r_row = C::kTma ? joined(256) : l_row;
      }
      // (0: the row sees nothing; a NaN among its scores stays one)
      const float lse = l_row != 0.f ? (m_fin - C::kPShift + log2f(l_row)) * kLn2 : -INFINITY;
      const float inv = r_row != 0.f ? 1.f / r_row : 0.f;
      const size_t grow = (size_t)it.q_start * H + row0 + q;
      if (row_ok && hh == 0 && grp == 0) {
        if (it.slot >= 0)
          part_lse[(size_t)it.slot * kRows + q] = lse;
        else if (p.return_lse)
          p.lse[grow] = lse;
      }
      if (!wait_bar(c, PV_DONE0 + ((g - 1) & 1), ((g - 1) >> 1) & 1)) goto fail_soft;
      tc_fence_after();
      const float s2 = it.slot < 0 ? inv * bmm2 : C::kTma ? inv : inv * (1 << C::kPartShift);
      // columns of O, V dims 256 hh + 128 grp + [0, 128), 16 at a time
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        uint32_t x[16];
        tmem_ld_32x32b_x16(tm + TM_O + 128 * grp + 16 * k, x);
        tmem_wait_ld();
        if (!row_ok) continue;
        const int chunk = 16 * hh + 8 * grp + k;  // of 16 dims
        if (C::kTma && it.slot >= 0) {  // fp32 (part_format)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            part_o[part_unit_f32(it.slot, kRows, chunk, u, q)] =
                make_uint4(__float_as_uint(__uint_as_float(x[4 * u]) * s2), __float_as_uint(__uint_as_float(x[4 * u + 1]) * s2),
                           __float_as_uint(__uint_as_float(x[4 * u + 2]) * s2), __float_as_uint(__uint_as_float(x[4 * u + 3]) * s2));
          continue;
        }
        uint32_t o[8];
        uint4 *d0, *d1;
        if (it.slot < 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(x[2 * e]) * s2,
                                                           __uint_as_float(x[2 * e + 1]) * s2);
            o[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          d0 = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + grow * kVDim + 16 * chunk);
          d1 = d0 + 1;
        } else {  // f16, times 2^kPartShift
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 h = __floats2half2_rn(__uint_as_float(x[2 * e]) * s2, __uint_as_float(x[2 * e + 1]) * s2);
            o[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          d0 = part_o + part_unit(it.slot, kRows, chunk, 0, q);
          d1 = part_o + part_unit(it.slot, kRows, chunk, 1, q);
        }
        *d0 = make_uint4(o[0], o[1], o[2], o[3]);
        *d1 = make_uint4(o[4], o[5], o[6], o[7]);
      }
      tc_fence_before();
      // both groups have read O before the next item's first PV overwrites it
      if (it.slot >= 0) __threadfence();  // ... and the partial is visible GPU-wide
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.bars[EPI]);
      if (!wait_bar(c, EPI, n_item & 1)) goto fail_soft;
      if (it.slot >= 0 && warp == kFirstSoft && lane == 0 && it.comb >= 0) {
        __threadfence();
        atomicAdd(comb_done + it.comb, 1);
      }
      ++n_item;
    }
    goto done_soft;
  fail_soft:
    tell_abort(c);
  done_soft:;
  } else {
    // ------------------------------------------------------------ conversion and query load
    // Two groups of eight warps take alternate tiles (and staging stages): a
    // tile's conversion is a chain of waits and shared-memory round trips longer
    // than a tile's MMAs.  Warp k of a group: latent dims [64 k, 64 k + 64) of the
    // own rows, one row a lane, into K; then, if those are V dims of this CTA, the
    // same values into V and 16 RoPE dims into K, else 64 V dims of the other rows.
    const int w = warp - kFirstConv;
    const uint32_t grp = (uint32_t)w >> 3;
    const int k = w & 7, vc = k & 3;
    const bool in_half = (k >> 2) == rank;
    float* qscale = reinterpret_cast<float*>(sm + C::OFF_QSCALE);
    uint32_t g = 0;
    int n_item = 0;
    // this lane's rows in the group's stages
    const uint32_t k_row = swizzled_row(smem_u32(sm) + OFF_K + grp * kKStage + k * kKChunk, lane);
    const uint32_t r_row = swizzled_row(smem_u32(sm) + OFF_K + grp * kKStage + 8 * kKChunk, lane);
    const uint32_t v_row = swizzled_row(smem_u32(sm) + OFF_V + grp * kVStage + vc * kVChunk,
                                        kHalf * (in_half ? rank : rank ^ 1) + lane);
    // bf16: warp 0 passes every tile's K on, one warp a group its V (a warp for both
    // held up K of tile g + 2 for V of tile g), after clearing the V rows that are not in
    // use (their K only makes scores that the mask replaces).  (K's stages are by tile
    // mod 3, so a warp of one group would skip phases of their barriers, and a wait for
    // a phase passes while the one before it is still open.)
    auto pass_tile = [&]() -> bool {
      if (w == 0) {
        const uint32_t use3 = g / 3, s3 = g - 3 * use3;
        if (!wait_bar(c, K_TMA0 + s3, use3 & 1)) return false;
        if (lane == 0) arrive_leader(c, K_FULL0 + s3, 1);
      } else if (k == 1 && (g & 1) == grp) {
        if (!wait_bar(c, STG_EMPTY0 + grp, (g >> 1) & 1)) return false;
        const uint32_t m0 = row_mask[2 * grp], m1 = row_mask[2 * grp + 1];
        if ((m0 & m1) != 0xffffffffu) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (((h ? m1 : m0) >> lane) & 1u) continue;
            const uint32_t v = smem_u32(sm) + OFF_V + grp * kVStage + h * (kVStage / 2) + lane * 128;
#pragma unroll 1
            for (int e = 0; e < 32; ++e) st_shared_v4(v + (e >> 3) * C::kVChunkStep + (e & 7) * 16, make_uint4(0, 0, 0, 0));
          }
        }
        __syncwarp();
        if (lane == 0) arrive_leader(c, V_FULL0 + grp, 1);
      }
      return true;
    };
    auto convert_tile = [&]() -> bool {
      if constexpr (C::kTma) return pass_tile();
      const uint32_t s = grp;
      if (!wait_bar(c, STG_FULL0 + s, (g >> 1) & 1)) return false;
      const unsigned char* stg = sm + C::OFF_STG + s * C::kStage;
      const unsigned char* codes = stg + C::STG_OWN + lane * C::kCodeBytes;
      const unsigned char* other = stg + C::STG_OTHER + lane * C::kVBytes;
      // whether this lane's rows are in use (the others are zeros)
      const uint32_t m1 = row_mask[2 * s + rank], m2 = in_half ? m1 : row_mask[2 * s + (rank ^ 1)];
      const bool on1 = (m1 >> lane) & 1u, on2 = (m2 >> lane) & 1u;
      uint4 x[8];
      uint32_t s2 = 0;  // 4 bits: the second part's scales
      if constexpr (kCache == kFp4) {
        const unsigned char* scales = stg + C::STG_SCALES;
        const unsigned char* sc_own = scales + (kHalf * rank + lane) * C::kScaleBytes;
        const unsigned char* sc_oth = scales + (kHalf * (rank ^ 1) + lane) * C::kScaleBytes;
        // (rows are 18 units of 16 bytes apart: rows 4 to 7 of eight take their two
        // units in the other order, and no two rows of a phase share a bank group)
        const int swap = (lane >> 2) & 1;
        const uint4 a = *reinterpret_cast<const uint4*>(codes + 32 * k + 16 * swap);
        const uint4 b = *reinterpret_cast<const uint4*>(codes + 32 * k + 16 * (swap ^ 1));
        uint32_t sc = *reinterpret_cast<const uint32_t*>(sc_own + 4 * k);
        s2 = in_half ? (uint32_t)sc_own[32 + vc]
                     : *reinterpret_cast<const uint32_t*>(sc_oth + 16 * rank + 4 * vc);
        if (!on1) sc = 0u;
        if (!on2) s2 = 0u;
        convert64(swap ? b : a, swap ? a : b, sc, x);
      } else {
        // (rows are 36 units apart: pairs of rows start at four places of the order,
        // and the units are put back by two rounds of exchanges)
        const int r2 = (lane >> 1) & 3;
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = on1 ? *reinterpret_cast<const uint4*>(codes + 64 * k + 16 * (i ^ r2)) : make_uint4(0, 0, 0, 0);
        exchange(u[0], u[1], r2 & 1);
        exchange(u[2], u[3], r2 & 1);
        exchange(u[0], u[2], r2 & 2);
        exchange(u[1], u[3], r2 & 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) widen16(u[i], x[2 * i], x[2 * i + 1]);
      }
      // QK of the group's previous tile has read this K stage
      if (!wait_bar(c, S_FULL0 + grp, ((g >> 1) & 1) ^ 1)) return false;
#pragma unroll
      for (int e = 0; e < 8; ++e) put(k_row, e, x[e]);
      if (in_half) {  // 16 RoPE dims
        uint4 y0, y1;
        if constexpr (kCache == kFp4) {
          const uint2 rc = *reinterpret_cast<const uint2*>(codes + 256 + 8 * vc);
          uint32_t s0, s1;
          scale_pairs(s2, s0, s1);
          y0 = convert8(rc.x, s0);
          y1 = convert8(rc.y, s0);
        } else {
          widen16(on1 ? *reinterpret_cast<const uint4*>(codes + 512 + 16 * vc) : make_uint4(0, 0, 0, 0), y0, y1);
        }
        put(r_row, 2 * vc, y0);
        put(r_row, 2 * vc + 1, y1);
      }
      __syncwarp();
      if (lane == 0) {
        arrive_leader(c, K_FULL0 + 3 * grp + k / kGroup, 4);
        if (in_half) arrive_leader(c, K_FULL0 + 3 * grp + 2, 1);
      }
      if (!in_half) {  // V of the other rows
        if constexpr (kCache == kFp4) {
          convert64(*reinterpret_cast<const uint4*>(other + (((2 * vc) ^ (lane & 7)) << 4)),
                    *reinterpret_cast<const uint4*>(other + (((2 * vc + 1) ^ (lane & 7)) << 4)), s2, x);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            widen16(on2 ? *reinterpret_cast<const uint4*>(other + (((4 * vc + i) ^ (lane & 7)) << 4))
                        : make_uint4(0, 0, 0, 0),
                    x[2 * i], x[2 * i + 1]);
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&c.bars[STG_EMPTY0 + s]);  // every code is in registers
      if (!wait_bar(c, PV_DONE0 + grp, ((g >> 1) & 1) ^ 1)) return false;
#pragma unroll
      for (int e = 0; e < 8; ++e) put(v_row, e, x[e]);
      __syncwarp();
      if (lane == 0) arrive_leader(c, V_FULL0 + grp, 1);
      return true;
    };
    // The item's query, rows [64 rank, 64 rank + 64) (those past the query's end
    // are zero).
    const long long q_rows = p.total_q * H;
    auto unit_of = [&](long long qr, int u) -> uint4 {  // unit u (eight dims) of a row, raw
      if (qr >= q_rows) return make_uint4(0, 0, 0, 0);
      if (p.q_fp8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p.query) + qr * 72 + u);
        return make_uint4(v.x, v.y, 0, 0);
      }
      return __ldg(reinterpret_cast<const uint4*>(p.query) + qr * 72 + u);
    };
    auto first_row = [&](const WorkItem& it) {
      return (long long)it.q_start * H + (long long)it.g * kRows + kCtaRows * rank;
    };
    // The rows' factors 2^-k, while the item before is still running: four rows a
    // warp, a row's 72 units over its lanes.
    auto query_scales = [&](const WorkItem& it, int n) {
      const long long q0 = first_row(it) + 4 * w;
#pragma unroll 2
      for (int r = 0; r < 4; ++r) {
        int e = 0;
        if (!p.q_fp8 && !C::kTma) {
          const uint4 a = unit_of(q0 + r, lane), b = unit_of(q0 + r, 32 + lane),
                      d = unit_of(q0 + r, 64 + (lane & 7));
          uint32_t mb = __vmaxu2(__vmaxu2(max_bits(a), max_bits(b)), max_bits(d));
          mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
          e = query_exponent(mb);
        }
        if (lane == 0)
          qscale[(n & 3) * kCtaRows + 4 * w + r] = __uint_as_float((uint32_t)(127 - e) << 23);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c.bars[QX]);
        mbar_arrive(&c.bars[QS_FULL0 + (n & 3)]);
      }
    };
    // The values: the TMEM chunks by a thread per row and 96 dims (both copies of a
    // row, see mma_f16_pair_ts), loaded before every QK of the previous item has
    // read its query; the shared-memory chunks three units a thread.
    auto load_query = [&](const WorkItem& it, int n) -> bool {
      const long long q0 = first_row(it);
      const float* scales = qscale + (n & 3) * kCtaRows;
      auto as_f16 = [&](const uint4 x, float up) {  // (as bf16 for bf16 MMAs)
        if constexpr (C::kTma) return p.q_fp8 ? e4m3x8_to_bf16(make_uint2(x.x, x.y)) : x;
        return p.q_fp8 ? e4m3x8_to_f16(make_uint2(x.x, x.y)) : bf16x8_to_f16(x, up);
      };
      const int quad = warp & 3, row = (32 * quad + lane) & 63, part = w >> 2;
      uint4 x[4], f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = unit_of(q0 + row, 12 * part + u);
      if (!wait_bar(c, QX, n & 1)) return false;
      const float up = 1.f / scales[row];  // a power of two: exact
      if (!wait_bar(c, Q_EMPTY, (n & 1) ^ 1)) return false;
      const uint32_t tq = tmem + ((uint32_t)(32 * quad) << 16) + TM_Q + 48 * part;
      constexpr int kPerRow = 8 * (kChunks - kTmemChunks);  // shared-memory units of a row
      static_assert(kCtaRows * kPerRow == 3 * 32 * kConvWarps, "three units a thread");
#pragma unroll 1
      for (int j = 0; j < 3; ++j) {  // 32 dims: four units, sixteen columns
#pragma unroll
        for (int u = 0; u < 4; ++u) f[u] = as_f16(x[u], up);
        tmem_st_32x32b_x16(tq + 16 * j, *reinterpret_cast<const uint32_t(*)[16]>(f));
        const int at = 32 * (kConvWarps * j + w) + lane, r = at / kPerRow, u2 = at - r * kPerRow;
        const uint4 y = unit_of(q0 + r, 8 * kTmemChunks + u2);
        if (j < 2) {
#pragma unroll
          for (int u = 0; u < 4; ++u) x[u] = unit_of(q0 + row, 12 * part + 4 * (j + 1) + u);
        }
        put(swizzled_row(smem_u32(sm) + OFF_Q + (u2 >> 3) * kQChunk, r), u2 & 7, as_f16(y, 1.f / scales[r]));
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(c, Q_FULL, 1);
      return true;
    };
    // The block's first query is staged where K or V will be, by copies of whole rows:
    // one round trip.  (By the passes above, in five, it was there 21,000 cycles after
    // the launch, and 15,000 this way.)
    constexpr uint32_t kQPitch = 2 * kQkDim + 16;  // an odd number of units: no bank conflicts
    constexpr uint32_t OFF_QSTG = C::kTma ? OFF_V : OFF_K;  // (TMA writes K as soon as it can)
    static_assert(kCtaRows * kQPitch <= (C::kTma ? 2 * kVStage + 2 * kPTile : 2 * (kKStage + kVStage)), "room");
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      if (n_tiles_of(it) <= 0) continue;
      const long long q0 = first_row(it);
      const int n = (int)min((long long)kCtaRows, q_rows - q0), bytes = p.q_fp8 ? kQkDim : 2 * kQkDim;
      if (lane < 4) {
        const int r = 4 * w + lane;
        mbar_arrive_expect_tx(&c.bars[QSTG], r < n ? bytes : 0);
        if (r < n)
          bulk_load(sm + OFF_QSTG + r * kQPitch, static_cast<const unsigned char*>(p.query) + (q0 + r) * bytes, bytes,
                    &c.bars[QSTG]);
      }
      __syncwarp();
      if (!first_query<kCache>(c, sm, tmem, Query{sm + OFF_QSTG, (int)kQPitch, n, p.q_fp8}, w)) {
        drain_wait(&c.bars[QSTG], 0);  // (rows may still be landing)
        goto fail_conv;
      }
      break;
    }
    for (int idx = item_begin; idx < item_end; ++idx) {
      const WorkItem it = items[idx];
      const int nt = n_tiles_of(it);
      if (nt <= 0) continue;
      // a later item's first tile before its query: its conversion needs nothing of
      // the previous item but free stages
      for (int t = 0; t < nt; ++t, ++g) {
        if ((C::kTma || (g & 1) == grp) && !convert_tile()) goto fail_conv;
        if (t > 0) continue;
        if (n_item > 0 && !load_query(it, n_item)) goto fail_conv;
        for (int nx = idx + 1; nx < item_end; ++nx) {
          const WorkItem itn = items[nx];
          if (n_tiles_of(itn) <= 0) continue;
          query_scales(itn, n_item + 1);
          break;
        }
      }
      ++n_item;
    }
    goto done_conv;
  fail_conv:
    tell_abort(c);
  done_conv:;
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *c.abort) atomicOr(c.status, kStatusTimeout);
  cluster_sync();  // neither CTA touches the other's memory or TMEM any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

namespace {

cudaLaunchConfig_t pair_launch(int grid, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int kCache>
cudaError_t setup_one(int sm_count, int* n_pairs) {
  auto kernel = decode_pair_kernel<kCache>;
  constexpr size_t kSmem = Cfg<kCache>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  const cudaLaunchConfig_t cfg = pair_launch(2 * (sm_count / 2), kSmem, nullptr, &attr);
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (clusters <= 0) return cudaErrorInvalidConfiguration;
  *n_pairs = std::min(clusters, sm_count / 2);
  return cudaSuccess;
}

// The bf16 cache as (64 dims, rows, chunks of 64 dims), boxes of 32 rows and `chunks`
// chunks in the 128B-swizzled layout: an operand's half tile is one copy.  (By boxes of
// one chunk the issue of V's eight took longer than a tile's MMAs.)
bool encode_rows(CUtensorMap* map, const Problem& p, int chunks) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void* ptr = nullptr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                                     &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
  }();
  if (!encode) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)p.num_pages * p.page_size, kChunks};
  cuuint64_t strides[2] = {2 * kQkDim, 128};
  cuuint32_t box[3] = {64, kHalf, (cuuint32_t)chunks}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.kv_cache), dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCache>
cudaError_t launch_one(const Problem& p, const Layout& lay, void* ws, cudaStream_t stream) {
  CUtensorMap tm_k = {}, tm_v = {};
  if (Cfg<kCache>::kTma && !(encode_rows(&tm_k, p, kChunks) && encode_rows(&tm_v, p, 4))) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  const cudaLaunchConfig_t cfg = pair_launch(lay.n_ctas, Cfg<kCache>::kSmemBytes, stream, &attr);
  return cudaLaunchKernelEx(&cfg, decode_pair_kernel<kCache>, p, lay, static_cast<char*>(ws), tm_k, tm_v);
}

}  // namespace

cudaError_t decode_pair_setup(int kv_dtype, int sm_count, int* n_pairs) {
  return kv_dtype == 2   ? setup_one<kFp4>(sm_count, n_pairs)
         : kv_dtype == 1 ? setup_one<kE4m3>(sm_count, n_pairs)
                         : setup_one<kBf16>(sm_count, n_pairs);
}

cudaError_t launch_decode_pair(const Problem& p, const Layout& lay, void* ws, cudaStream_t stream) {
  return p.kv_dtype == 2   ? launch_one<kFp4>(p, lay, ws, stream)
         : p.kv_dtype == 1 ? launch_one<kE4m3>(p, lay, ws, stream)
                           : launch_one<kBf16>(p, lay, ws, stream);
}

}  // namespace mla
