// Beam search over the paged cache: the choice of the next beams and the reordering of the
// cache that follows from it.
//
// Selection.  A request's beams w have scores c_w and rows x_w of logits over a vocabulary of
// V; a continuation (w, v) scores
//   s(w, v) = c_w + x_w[v] - lse_w,   lse_w = ln sum_v exp(x_w[v]),
// and the k best are wanted, the lowest (w, v) first among equals.  The logits are read once.
// Within a beam the order is that of the logits themselves, so each block keeps the k largest
// logits of its part of a row, exactly, beside the part's sum of exponentials; one block a
// request then compares the scores of all parts' candidates.  What decides between nearly equal
// candidates of two beams is lse.  Its sum is of 2^(x log2(e) - n), n whole: the product in two
// parts, sums with their rounding errors, everything else powers of two, which are exact; and
// the largest logit's own term divides it, so that what is wrong with that term, which may
// be all of a sum, leaves lse.  Measured over rows of 100003 tokens, of ordinary, peaked and flat
// shapes: lse off by 2^-25 to 2^-23.4 (root mean square), by 2^-21.7 at most; were all roundings of a sum one
// way it would be 2^-18.  Scores are pairs of floats (48 bits; the card has few units for 64).  Which thread takes a value, and in which order,
// is by its index alone and not by where the row lies in memory: rows with the same logits have the
// same lse, to the bit, and their ties go by index.
//
// What bounds it: the bytes of the logits, where there are many; a chain of two launches, else.
// A thread streams its own values through shared memory, with no barrier, a chunk ahead, four blocks
// to an SM: it keeps their maximum and sum.  (Where rows start off 16 bytes its units are the ends of
// its own copies and the starts of its neighbour's: 24 x 16 beams over 100003 fp32 tokens 41.5 us
// in a graph, and 39.8 when a value's thread hung on where its row starts.)  The k-th
// largest maximum of 64 groups of threads is a threshold that at least k values are at or above,
// and seldom many more; the few stretches of a thread's values whose maximum is not below it are
// read again, and what passes is ranked by counting.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "../../include/mla_decode.h"
#include "mla_common.cuh"
#include "mla_fp4.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocks = 608;            // four on each of 152 SMs, all at once
constexpr int kStages = 2;             // chunks of a block on their way
constexpr int kVectors = 4;             // 16-byte units of a thread in a chunk
constexpr int kGroups = 64;             // groups of a part's values: four threads each
constexpr int kMaxK = 64;
constexpr int kRoom = 1024;             // candidates collected at most (ties may pass it)
constexpr int kMaxLists = 128;          // candidate lists of a request at most
constexpr unsigned kAll = 0xffffffffu;
constexpr int kStretches = 16;          // of a thread's part, each with its maximum
constexpr int kWarpUnits = 33;          // of a warp's 32 units, and the one behind them
constexpr size_t kRing = (size_t)kStages * kVectors * kWarps * kWarpUnits * 16;
constexpr size_t kSmem = kRing + sizeof(float) * kStretches * kThreads;
constexpr float kNone = -INFINITY;

// Order-preserving bits of a float (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
// The largest float below x, and -inf of it.
__device__ __forceinline__ float below(float x) { return x == kNone ? x : -nextafterf(-x, INFINITY); }
__device__ __forceinline__ bool before(float xa, int ia, float xb, int ib) { return xa > xb || (xa == xb && ia < ib); }

struct Logits {
  const void* base;
  long long batch_stride, beam_stride;  // elements
  int beams, vocab;
};

template <typename T>
__device__ __forceinline__ float value_of(uint32_t word, int half) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(word);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return __uint_as_float(half ? word & 0xffff0000u : word << 16);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&word);
    return half ? __high2float(h) : __low2float(h);
  }
}

constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.925963033500e-8f;
// The largest of kCount units' values, two at a time in 16 bits (a NaN is none).
template <typename T, int kCount>
__device__ __forceinline__ float largest(const uint4* w) {
  if constexpr (sizeof(T) == 4) {
    float m = kNone;
#pragma unroll
    for (int v = 0; v < kCount; ++v)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[v].x), __uint_as_float(w[v].y)),
                         fmaxf(__uint_as_float(w[v].z), __uint_as_float(w[v].w))));
    return m;
  } else {
    using Pair = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
    auto pair = [](const uint32_t& x) { return *reinterpret_cast<const Pair*>(&x); };
    Pair m = __hmax2(__hmax2(pair(w[0].x), pair(w[0].y)), __hmax2(pair(w[0].z), pair(w[0].w)));
#pragma unroll
    for (int v = 1; v < kCount; ++v)
      m = __hmax2(m, __hmax2(__hmax2(pair(w[v].x), pair(w[v].y)), __hmax2(pair(w[v].z), pair(w[v].w))));
    const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
    // (two NaN leave one: no maximum)
    return fmaxf(fmaxf(value_of<T>(bits, 0), value_of<T>(bits, 1)), kNone);
  }
}

// e^d for d <= 0: the product by log2(e) in two parts, so that its rounding is not of log2(e).
__device__ __forceinline__ float exp_of(float d) { return ptx::ex2(fmaf(d, kLog2eHi, d * kLog2eLo)); }
// 2^d for a whole d of 0 at most, exact; 0 below 2^-126.
__device__ __forceinline__ float whole_power(float d) {
  return d < -126.f ? 0.f : __uint_as_float((uint32_t)(127 + (int)d) << 23);
}

// A number as the sum of two floats, the second at most half a step of the first.
struct Two {
  float h, l;
};
// (Knuth's sum of two with its rounding error; `settle` is Dekker's, for a larger first.)
__device__ __forceinline__ Two exact_sum(float a, float b) {
  const float s = a + b, z = s - a;
  return {s, (a - (s - z)) + (b - z)};
}
__device__ __forceinline__ Two settle(float h, float l) {  // |h| >= |l|
  const float s = h + l;
  return {s, l - (s - h)};
}
__device__ __forceinline__ Two add(Two a, float b) {
  const Two s = exact_sum(a.h, b);
  return settle(s.h, s.l + a.l);
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = exact_sum(a.h, b.h);
  return settle(s.h, s.l + (a.l + b.l));
}
// e ln 2 for a whole e below 2^23.
__device__ __forceinline__ Two times_ln2(float e) {
  constexpr float kHi = 0.693147182464599609375f, kLo = -1.90465429995776e-9f;
  const float p = e * kHi;
  return settle(p, fmaf(e, kHi, -p) + e * kLo);
}
// ln x for 0 < x < 2^120: x = 2^e f, f in [0.75, 1.5), ln f = 2 atanh z, z = (f - 1) / (f + 1),
// |z| <= 1/5, by its series; only its first term needs more than a float.  Off by some 2^-31.
__device__ __forceinline__ Two log_of(Two x) {
  const uint32_t bits = __float_as_uint(x.h);
  int e = (int)(bits >> 23) - 127;
  if ((bits & 0x7fffffu) >= 0x400000u) ++e;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  const Two f{x.h * down, x.l * down};
  const Two top = add(f, -1.f), bottom = add(f, 1.f);
  const float q = top.h / bottom.h;
  const float rest = (fmaf(-q, bottom.h, top.h) + top.l) - q * bottom.l;
  const Two z = settle(q, rest / bottom.h);
  const float y = z.h * z.h;
  float t = 1.f / 13.f;
  t = fmaf(t, y, 1.f / 11.f);
  t = fmaf(t, y, 1.f / 9.f);
  t = fmaf(t, y, 1.f / 7.f);
  t = fmaf(t, y, 1.f / 5.f);
  t = fmaf(t, y, 1.f / 3.f);
  return add(times_ln2((float)e), add(Two{2.f * z.h, 2.f * z.l}, 2.f * z.h * y * t));
}
// Order-preserving bits of a score; 0: none (one past fp32's range is none, either).
__device__ __forceinline__ unsigned long long key_of_score(Two s) {
  if (!(fabsf(s.h) < INFINITY)) return 0;
  return ((unsigned long long)ordered(s.h) << 32) | ordered(s.l);
}
__device__ __forceinline__ float score_of_key(unsigned long long key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

// x log2(e), and 2^(a - b) for a - b of 0.5 at most: 0 far below (a of -infinity included).
__device__ __forceinline__ Two log2_of(float x) {
  const float h = x * kLog2eHi;
  return {h, fmaf(x, kLog2eHi, -h) + x * kLog2eLo};
}
__device__ __forceinline__ float power_of(Two a, Two b) {
  const float d = a.h - b.h;
  return d < -150.f ? 0.f : ptx::ex2(d + (a.l - b.l));
}

// What a sum of exponentials is relative to: 2^power, the whole number next to its largest
// argument times log2(e); where that is of 2^20 and more, whose powers a float does not hold,
// e^top.  A sum of nothing (top of -infinity) is 0, or a NaN that it has met.
struct Reference {
  float top, power;
};
__device__ __forceinline__ bool is_far(float top) { return !(fabsf(top) < 1048576.f); }
__device__ __forceinline__ Reference reference_of(float top) {
  return {top, is_far(top) ? 0.f : rintf(top * kLog2eHi)};
}
// The factor that takes a sum from a to b, b the higher one.
__device__ __forceinline__ float between(Reference a, Reference b) {
  if (!is_far(a.top) && !is_far(b.top)) return whole_power(a.power - b.power);
  if (b.top == kNone) return 1.f;
  if (is_far(a.top) && is_far(b.top)) return exp_of(a.top - b.top);
  return power_of(is_far(a.top) ? log2_of(a.top) : Two{a.power, 0.f}, is_far(b.top) ? log2_of(b.top) : Two{b.power, 0.f});
}

// A part of a row, as one block found it.
struct Part {
  Reference at;
  Two sum;
};

struct Parts {
  Part* part;    // [rows][parts]
  float* value;  // [rows][parts][k], descending; -inf: none
  int* token;    // [rows][parts][k]
  int parts, share;  // parts of a row, chunks of a part
};

}  // namespace

// The k largest of values [begin, end) of a row, one after another: for parts whose threshold more values
// pass than there is room for.  (Apart, as it is hardly ever called.)
template <typename T>
__device__ __noinline__ void select_slowly(const T* x, int begin, int end, int k, float* out_x, int* out_i,
                                           unsigned long long* best_key) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float last_x = INFINITY;
  int last_i = -1;
  for (int found = 0; found < k; ++found) {
    unsigned long long key = 0;  // (order of the value, lowest index); 0: none
#pragma unroll 1
    for (int i = begin + tid; i < end; i += kThreads) {
      const float y = (float)x[i];
      if (!(y > kNone) || !before(last_x, last_i, y, i)) continue;
      const unsigned long long q = ((unsigned long long)ordered(y) << 32) | (0xffffffffu - (unsigned)i);
      key = q > key ? q : key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long q = __shfl_xor_sync(kAll, key, o);
      key = q > key ? q : key;
    }
    if (lane == 0) best_key[warp] = key;
    __syncthreads();
    key = 0;
    for (int w = 0; w < kWarps; ++w) key = best_key[w] > key ? best_key[w] : key;
    __syncthreads();
    const bool on = key != 0;
    last_x = on ? score_of_key(key) : kNone;
    last_i = on ? (int)(0xffffffffu - (uint32_t)key) : -1;
    if (tid == 0) {
      out_x[found] = last_x;
      out_i[found] = last_i;
    }
  }
}

// kApart: rows that need not start on a 16-byte boundary (a kernel of its own: the others' calls are
// shorter without).
template <typename T, bool kApart>
__global__ void __launch_bounds__(kThreads, 4)
beam_parts_kernel(Logits in, const float* __restrict__ scores, const unsigned char* __restrict__ finished, int k,
                  Parts out) {
  constexpr int kPer = 16 / (int)sizeof(T);  // values of a unit
  constexpr int kHalves = 4 / (int)sizeof(T), kUnits = kThreads * kVectors;
  extern __shared__ __align__(16) uint4 ring[];  // [stage][unit of a thread][thread]
  __shared__ float group_max[kGroups], threshold;
  __shared__ int n_cand, n_hot;
  __shared__ unsigned long long best_key[kWarps];
  __shared__ int equal_sum[kWarps];
  // once the row has gone through it, the ring holds the candidates and the places to look again
  float* cand_x = reinterpret_cast<float*>(ring);
  int* cand_i = reinterpret_cast<int*>(cand_x + kRoom);
  unsigned short* hot = reinterpret_cast<unsigned short*>(cand_i + kRoom);  // thread + 256 stretch
  static_assert(8 * kRoom + 2 * kStretches * kThreads <= kRing && kThreads == 256, "room");
  float* stretch_max = reinterpret_cast<float*>(reinterpret_cast<char*>(ring) + kRing);  // [stretch][thread]
  __shared__ unsigned long long warp_sum[kWarps];
  ptx::pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / out.parts, part = blockIdx.x - row * out.parts;
  // a beam that has ended, or has no score, offers nothing that its logits decide
  if ((finished && finished[row]) || !(fabsf(scores[row]) < INFINITY)) return;
  const T* x = static_cast<const T*>(in.base) + (row / in.beams) * in.batch_stride + (row % in.beams) * in.beam_stride;
  // Units of values [u kPer, (u + 1) kPer).  Copies are of 16 aligned bytes; where the row does not
  // start on one, `off` values before it do, and a unit is the end of one copy and the start of the next.
  const int off = kApart ? (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)) : 0;
  const int units = (in.vocab + kPer - 1) / kPer;
  const int u0 = part * out.share * kUnits, u1 = min(u0 + out.share * kUnits, units);
  const int f0 = off > 0 ? 1 : 0, f1 = (off + in.vocab) / kPer;  // copies [f0, f1) lie inside the row
  constexpr uint32_t kNothing = sizeof(T) == 4 ? 0xff800000u
                                : std::is_same<T, __nv_bfloat16>::value ? 0xff80ff80u : 0xfc00fc00u;  // -inf
  auto copy_at = [&](int u) { return reinterpret_cast<const uint4*>(x + ((long long)u * kPer - off)); };
  // values [first, first + kPer) one by one, -inf where the row has none
  auto pieces = [&](int first) -> uint4 {
    uint32_t e[4] = {kNothing, kNothing, kNothing, kNothing};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = first + j;
      if (i < 0 || i >= in.vocab) continue;
      if constexpr (sizeof(T) == 4) {
        e[j] = reinterpret_cast<const uint32_t*>(x)[i];
      } else {
        const uint32_t bits = reinterpret_cast<const unsigned short*>(x)[i];
        e[j / 2] = j & 1 ? (e[j / 2] & 0xffffu) | bits << 16 : (e[j / 2] & 0xffff0000u) | bits;
      }
    }
    return make_uint4(e[0], e[1], e[2], e[3]);
  };
  // the unit that starts `off` values, `words` whole words, into copy a (b: the next one)
  const int off_words = off * (int)sizeof(T) / 4;
  auto joined = [&](const uint4& a, const uint4& b, int words) -> uint4 {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t y[6], z[5];
#pragma unroll
    for (int j = 0; j < 6; ++j) y[j] = words & 2 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) z[j] = words & 1 ? y[j + 1] : y[j];
    if constexpr (sizeof(T) == 2) {
      const int bits = off & 1 ? 16 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = __funnelshift_r(z[j], z[j + 1], bits);
    }
    return make_uint4(z[0], z[1], z[2], z[3]);
  };
  auto at = [](const uint4& w, int e) {
    const int j = e / kHalves;
    return value_of<T>(j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w, e % kHalves);
  };
  auto slot = [&](int chunk, int v) { return ring + ((chunk % kStages * kVectors + v) * kWarps + warp) * kWarpUnits + lane; };
  const int chunks = u1 > u0 ? (u1 - u0 + kUnits - 1) / kUnits : 0;
  auto bring = [&](int chunk) {
    if (chunk < chunks) {
      const int first = u0 + chunk * kUnits, u = first + tid;
      // the copy behind each of the warp's, one a lane
      const bool behind = kApart && lane < kVectors;
      uint4* to = slot(chunk, lane & (kVectors - 1)) - lane + 32;
      const int next = u - lane + (lane & (kVectors - 1)) * kThreads + 32;
      if (first >= f0 && first + kUnits < f1) {
#pragma unroll
        for (int v = 0; v < kVectors; ++v) ptx::cp_async_16(slot(chunk, v), copy_at(u + v * kThreads));
        if (behind) ptx::cp_async_16(to, copy_at(next));
      } else {
#pragma unroll 1
        for (int v = 0; v < kVectors + 1; ++v) {
          uint4* here = v < kVectors ? slot(chunk, v) : to;
          const int one = v < kVectors ? u + v * kThreads : next;
          if (v == kVectors && !behind) break;
          if (one >= f0 && one < f1) ptx::cp_async_16(here, copy_at(one));
          else *here = pieces(one * kPer - off);
        }
      }
    }
    ptx::cp_async_commit();
  };
  for (int c = 0; c < kStages - 1; ++c) bring(c);
  // a thread's chunks in up to kStretches stretches, whose maxima it writes down
  const int stretch = (chunks + kStretches - 1) / kStretches;
  Reference ref{kNone, 0.f};  // of this thread's maximum,
  float here = kNone;         // the maximum of the stretch,
  Two sum{0.f, 0.f};          // and the sum
  auto take = [&](const uint4* w) {
    const float mine = largest<T, kVectors>(w);
    here = fmaxf(here, mine);
    if (mine > ref.top) {
      const Reference higher = reference_of(mine);
      const float f = between(ref, higher);
      sum.h *= f;
      sum.l *= f;
      ref = higher;
    }
    const float from = is_far(ref.top) && ref.top != kNone ? -ref.top : 0.f;
    const uint64_t minus = ptx::pack_f32x2(from, from), down = ptx::pack_f32x2(-ref.power, -ref.power),
                   hi = ptx::pack_f32x2(kLog2eHi, kLog2eHi), lo = ptx::pack_f32x2(kLog2eLo, kLog2eLo);
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int v = 0; v < kVectors; ++v)
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const uint64_t d = ptx::add_f32x2(ptx::pack_f32x2(at(w[v], e), at(w[v], e + 1)), minus);
        float a, b;
        ptx::unpack_f32x2(ptx::fma_f32x2(d, lo, ptx::fma_f32x2(d, hi, down)), a, b);
        s[(e >> 1) & 1] = ptx::add_f32x2(s[(e >> 1) & 1], ptx::pack_f32x2(ptx::ex2(a), ptx::ex2(b)));
      }
    float a, b;
    ptx::unpack_f32x2(ptx::add_f32x2(s[0], s[1]), a, b);
    const Two t = exact_sum(sum.h, a + b);
    sum = {t.h, t.l + sum.l};
  };
  auto stream = [&](auto shift) {  // (whole words that the row starts past a boundary)
    for (int c = 0; c < chunks; ++c) {
      if (kApart) __syncwarp();  // (its neighbour has read what a lane brings the next chunk to)
      bring(c + kStages - 1);
      ptx::cp_async_wait<kStages - 1>();  // this thread's copies of chunk c are there
      if (kApart) __syncwarp();           // the warp's are
      uint4 w[kVectors];
#pragma unroll
      for (int v = 0; v < kVectors; ++v)
        w[v] = kApart ? joined(slot(c, v)[0], slot(c, v)[1], decltype(shift)::value) : *slot(c, v);
      take(w);
      if ((c + 1) % stretch == 0 || c + 1 == chunks) {
        stretch_max[c / stretch * kThreads + tid] = here;
        here = kNone;
      }
    }
  };
  if (!kApart || off_words == 0) stream(std::integral_constant<int, 0>());
  else if (off_words == 1) stream(std::integral_constant<int, 1>());
  else if (off_words == 2) stream(std::integral_constant<int, 2>());
  else stream(std::integral_constant<int, 3>());
  const float m = ref.top;
  // the maxima of four threads each
  {
    float g = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
    g = fmaxf(g, __shfl_xor_sync(kAll, g, 2));
    if ((lane & 3) == 0) group_max[tid >> 2] = g;
    if (tid == 0) n_hot = n_cand = 0;
  }
  __syncthreads();
  // the rank of a group by its four threads; of two together by their eight, for a small k, in a
  // quarter of the steps
  auto rank_groups = [&](auto wide) {
    constexpr int kPerGroup = decltype(wide)::value, kAll2 = kThreads / kPerGroup;
    auto value = [&](int i) { return kPerGroup == 4 ? group_max[i] : fmaxf(group_max[2 * i], group_max[2 * i + 1]); };
    const int group = tid / kPerGroup;
    const float g = value(group);
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kAll2 / kPerGroup; ++j) {
      const int o = kPerGroup * j + (lane & (kPerGroup - 1));
      rank += before(value(o), o, g, group) ? 1 : 0;
    }
#pragma unroll
    for (int o = 1; o < kPerGroup; o <<= 1) rank += __shfl_xor_sync(kAll, rank, o);
    if (rank == k - 1) threshold = g;
  };
  if (k <= 16) rank_groups(std::integral_constant<int, 8>());
  else rank_groups(std::integral_constant<int, 4>());
  float top = fmaxf(group_max[lane], group_max[lane + 32]);
  {
    const uint32_t u = __reduce_max_sync(kAll, ordered(top));
    top = __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
  }
  // the threads' sums, relative to the part's maximum
  const Reference all_of = reference_of(top);
  {
    // (no value: a sum of 0; a NaN, or an infinity's, stays one)
    const float f = between(ref, all_of);
    // whole multiples of 2^-32 add up without rounding, 22 bits at a time (a thread's sum is
    // below 2^21: of 2^20 values at most, each below 2^0.6)
    const float h = sum.h * f, l = sum.l * f;
    const bool odd = !(h < 2097152.f);  // a NaN, then
    const long long q = odd ? 0 : __float2ll_rn(h * 4294967296.f) + __float2ll_rn(l * 4294967296.f);
    unsigned long long all = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      all += (unsigned long long)__reduce_add_sync(kAll, (unsigned)(q >> (22 * i)) & 0x3fffffu) << (22 * i);
    const bool none = __any_sync(kAll, odd);
    if (lane == 0) warp_sum[warp] = none ? ~0ull : all;
  }
  __syncthreads();
  // the stretches that have a value at or above the threshold
  const float least = threshold;
  const int stretches = chunks > 0 ? (chunks + stretch - 1) / stretch : 0;
  if (m >= least && m > kNone) {
    int mine = 0;
    for (int z = 0; z < stretches; ++z) mine += stretch_max[z * kThreads + tid] >= least;
    int p = atomicAdd(&n_hot, mine);
    for (int z = 0; z < stretches; ++z)
      if (stretch_max[z * kThreads + tid] >= least) hot[p++] = (unsigned short)(tid + kThreads * z);
  }
  __syncthreads();
  auto unit_again = [&](int u) -> uint4 {
    if (u >= u1) return make_uint4(kNothing, kNothing, kNothing, kNothing);
    if (u < f0 || u + f0 >= f1) return pieces(u * kPer);
    return off > 0 ? joined(*copy_at(u), *copy_at(u + 1), off_words) : *copy_at(u);
  };
  // values that are kNone, or `low` and less, are no candidates
  auto offer = [&](const uint4& w, int u, float low) {
    int mine = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) mine += at(w, e) > low;
    if (mine == 0) return;
    int p = atomicAdd(&n_cand, mine);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float y = at(w, e);
      if (y > low) {
        if (p < kRoom) {
          cand_x[p] = y;
          cand_i[p] = u * kPer + e;
        }
        ++p;
      }
    }
  };
  const int each = stretch * kVectors, again = n_hot * each;  // units of a stretch
  // (once there are too many, how many there are does not matter)
  auto collect = [&](float low) {
    constexpr int kAgain = 4;
    for (int q0 = tid; q0 < again && *(volatile int*)&n_cand <= kRoom; q0 += kAgain * kThreads) {
      uint4 w[kAgain];
      int u[kAgain];
#pragma unroll
      for (int j = 0; j < kAgain; ++j) {
        const int q = q0 + j * kThreads, h = q / each;
        u[j] = u1;
        if (q < again) {
          const int z = hot[h];
          u[j] = u0 + (z / kThreads * each + q - h * each) * kThreads + z % kThreads;
        }
        w[j] = unit_again(u[j]);
      }
#pragma unroll
      for (int j = 0; j < kAgain; ++j) offer(w[j], u[j], low);
    }
    __syncthreads();
  };
  collect(below(least));
  const size_t list = (size_t)row * out.parts + part;
  float* out_x = out.value + list * k;
  int* out_i = out.token + list * k;
  // Where too many pass, many equal the threshold (tokens masked by a finite value): the ones above
  // it then, and of its equals the first in the order of their index.  (64 x 4 beams over 131071 tokens
  // of which five are not masked: 51 us, and 495 with all k places found one after another.)
  const bool equals = n_cand > kRoom;
  int first_equal = k;  // places from here on are theirs
  if (equals) {
    __syncthreads();
    if (tid == 0) n_cand = 0;
    __syncthreads();
    collect(least);
    first_equal = min(n_cand, k);
    if (n_cand <= kRoom)
      for (int from = u0, place = first_equal; from < u1 && place < k; from += kThreads) {
        const uint4 w = unit_again(from + tid);
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) mine += at(w, e) == least;
        int up = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kAll, up, o);
          if (lane >= o) up += y;
        }
        __syncthreads();
        if (lane == 31) equal_sum[warp] = up;
        __syncthreads();
        int p = place + up - mine;
        for (int o = 0; o < kWarps; ++o) {
          if (o < warp) p += equal_sum[o];
          place += equal_sum[o];
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (at(w, e) == least) {
            if (p < k) {
              out_x[p] = least;
              out_i[p] = (from + tid) * kPer + e;
            }
            ++p;
          }
      }
  }
  const int n = n_cand;
  if (n <= kRoom) {
    for (int j = tid; j < n; j += kThreads) {
      const float y = cand_x[j];
      const int i = cand_i[j];
      int rank = 0;
      for (int o = 0; o < n; ++o) rank += before(cand_x[o], cand_i[o], y, i) ? 1 : 0;
      if (rank < k) {
        out_x[rank] = y;
        out_i[rank] = i;
      }
    }
    for (int r = n + tid; r < first_equal; r += kThreads) {
      out_x[r] = kNone;
      out_i[r] = -1;
    }
  } else {
    select_slowly(x, u0 * kPer, min(in.vocab, u1 * kPer), k, out_x, out_i, best_key);
  }
  if (tid == 0) {
    unsigned long long s = 0;
    bool odd = false;
    for (int w = 0; w < kWarps; ++w) {
      s += warp_sum[w];
      odd = odd || warp_sum[w] == ~0ull;
    }
    // the sum as two floats: its upper 24 bits and the rest
    const int shift = max(0, 40 - __clzll(s));
    const float h = (float)(s >> shift << shift) * 2.3283064365386963e-10f;
    const float l = (float)(s & ((1ull << shift) - 1)) * 2.3283064365386963e-10f;
    out.part[list] = Part{all_of, odd ? Two{NAN, 0.f} : settle(h, l)};
  }
}

// One block a request: the rows' normalisers, then the k best of all lists.  scores_out may be
// `scores` where k is `beams`: a block reads its request's before a barrier that its results follow.
constexpr int kDepths = 4, kStaged = 2048;

__global__ void __launch_bounds__(kThreads)
beam_join_kernel(const float* scores, const unsigned char* __restrict__ finished, int beams, int k, int end_token, Parts in, float* scores_out, int* __restrict__ tokens_out,
                 int* __restrict__ parents_out) {
  __shared__ Two row_less[kMaxK];                    // what a row's logits are diminished by beside `top`: lse - top - score
  __shared__ float row_top[kMaxK], row_score[kMaxK];  // (beams are 64 at most, too)
  __shared__ float row_least[kMaxK];
  __shared__ int row_lists[kMaxK];  // of a beam; 0: it offers nothing, -1: it has ended
  __shared__ unsigned long long key[kDepths][kMaxLists], cand_s[kRoom], best_s[kWarps], threshold;
  __shared__ long long cand_i[kRoom], best_i[kWarps];
  __shared__ float cand_x[kRoom], best_x[kWarps];
  __shared__ float staged[kStaged];
  __shared__ int staged_token[kStaged];
  __shared__ int n_cand;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lists = beams * in.parts;
  const size_t list0 = (size_t)b * lists;
  ptx::pdl_wait();
  // (beside the normalisers; lists that nobody wrote are not looked at)
  const bool near = lists * k <= kStaged;
  if (near)
    for (int e = tid; e < lists * k; e += kThreads) {
      staged[e] = in.value[list0 * k + e];
      staged_token[e] = in.token[list0 * k + e];
    }
  constexpr int kLanes = 8;  // of a row
  for (int w0 = 0; w0 < beams; w0 += kThreads / kLanes) {
    const int w = w0 + tid / kLanes, part0 = tid % kLanes, row = b * beams + w;
    const float c = w < beams ? scores[row] : kNone;
    const bool scored = fabsf(c) < INFINITY, done = w < beams && finished && finished[row];
    Two sum{0.f, 0.f};
    float top = kNone;
    const int parts = scored && !done ? in.parts : 0;
    const Part* of = in.part + (size_t)row * in.parts;
    for (int p = part0; p < parts; p += kLanes) top = fmaxf(top, of[p].at.top);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const Reference whole = reference_of(top);
    {
      for (int p = part0; p < parts; p += kLanes) {
        const Part q = of[p];
        // (a part without a value adds 0, or a NaN that it holds)
        const float f = between(q.at, whole);
        sum = add(sum, Two{q.sum.h * f, q.sum.l * f});
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        const Two other{__shfl_xor_sync(kAll, sum.h, o), __shfl_xor_sync(kAll, sum.l, o)};
        sum = add(sum, other);
      }
    }
    if (part0 == 0 && w < beams) {
      // an infinity or a NaN among the logits, or nothing above -inf: no continuation
      const bool ok = scored && !done && fabsf(top) < INFINITY && sum.h > 0.f && sum.h < 1e35f;
      row_lists[w] = scored && done ? -1 : ok ? in.parts : 0;
      row_top[w] = top;
      row_score[w] = c;
      Two less{0.f, 0.f};
      if (ok) {
        // beside the largest term, as the sum took it
        const float own = is_far(top) ? 1.f : ptx::ex2(fmaf(top, kLog2eLo, fmaf(top, kLog2eHi, -whole.power)));
        const Two ln_own = log_of(Two{own, 0.f});
        less = add(add(log_of(sum), Two{-ln_own.h, -ln_own.l}), -c);
      }
      row_less[w] = less;
    }
  }
  if (tid == 0) {
    n_cand = 0;
    threshold = 0;
  }
  __syncthreads();
  // candidate j of a list: its key (0: none), and its place (w, token)
  auto logit = [&](int l, int j) { return near ? staged[l * k + j] : in.value[(list0 + l) * k + j]; };
  auto key_of = [&](int l, int j) -> unsigned long long {
    const int w = l / in.parts, lists_of = row_lists[w], p = l - w * in.parts;
    if (lists_of < 0) return j == 0 && p == 0 ? key_of_score(Two{row_score[w], 0.f}) : 0;
    if (p >= lists_of) return 0;
    const float x = logit(l, j);
    if (x == kNone) return 0;
    const Two less = row_less[w];
    return key_of_score(add(exact_sum(x, -row_top[w]), Two{-less.h, -less.l}));
  };
  auto place_of = [&](int l, int j) -> long long {
    const int w = l / in.parts;
    return (long long)w << 32 | (row_lists[w] < 0 ? end_token : near ? staged_token[l * k + j] : in.token[(list0 + l) * k + j]);
  };
  auto value_at = [&](int l, int j) { return row_lists[l / in.parts] < 0 ? 0.f : logit(l, j); };
  // A threshold that at least k candidates are at or above: for some depths d, the
  // ceil(k / d)-th largest of the lists' d-th candidates, and of these the largest.  (With d
  // = 1, 4, 16, 64 fewer than 4 k candidates for each d pass it, ties apart, however the
  // beams' scores lie.)
  for (int t = tid; t < kDepths * lists; t += kThreads) {
    const int e = t / lists, l = t - e * lists, d = min(1 << (2 * e), k);
    key[e][l] = key_of(l, d - 1);
  }
  __syncthreads();
  for (int t = tid; t < kDepths * lists; t += kThreads) {
    const int e = t / lists, l = t - e * lists, d = min(1 << (2 * e), k), want = (k + d - 1) / d;
    if (want > lists || (e > 0 && 1 << (2 * e - 2) >= k)) continue;
    const unsigned long long s = key[e][l];
    int rank = 0;
    for (int o = 0; o < lists; ++o) rank += (key[e][o] > s || (key[e][o] == s && o < l)) ? 1 : 0;
    if (rank == want - 1) atomicMax(&threshold, s);
  }
  __syncthreads();
  const unsigned long long least = max(threshold, 1ull);
  // the same for a beam's logits, a little lower (some 2^-22 of its terms), which spares most
  // candidates their sums
  if (tid < beams) {
    const float s = threshold == 0 ? kNone : score_of_key(threshold), less = row_less[tid].h, top = row_top[tid];
    row_least[tid] = s + less + top - (fabsf(s) + fabsf(less) + fabsf(top) + fabsf(row_score[tid])) * 1e-6f;
  }
  __syncthreads();
  for (int e = tid; e < lists * k; e += kThreads) {
    const int l = e / k, j = e - l * k;
    if (key[0][l] < least) continue;
    if (row_lists[l / in.parts] > 0 && logit(l, j) < row_least[l / in.parts]) continue;
    const unsigned long long s = key_of(l, j);
    if (s < least) continue;
    const int p = atomicAdd(&n_cand, 1);
    if (p < kRoom) {
      cand_s[p] = s;
      cand_i[p] = place_of(l, j);
      cand_x[p] = value_at(l, j);
    }
  }
  __syncthreads();
  const int n = n_cand;
  // By score, beam, logit and token: logits of one beam may be nearer than 48 bits of their scores
  // tell (a beam whose score is -1e9).
  auto ahead = [](unsigned long long sa, long long ia, float xa, unsigned long long sb, long long ib, float xb) {
    if (sa != sb) return sa > sb;
    return ia >> 32 == ib >> 32 && xa != xb ? xa > xb : ia < ib;
  };
  auto write = [&](int rank, unsigned long long s, long long i) {
    scores_out[(size_t)b * k + rank] = s == 0 ? kNone : score_of_key(s);
    tokens_out[(size_t)b * k + rank] = i < 0 ? -1 : (int)i;
    parents_out[(size_t)b * k + rank] = i < 0 ? -1 : (int)(i >> 32);
  };
  if (n <= kRoom) {
    for (int j = tid; j < n; j += kThreads) {
      const unsigned long long mine = cand_s[j];
      int rank = 0;
      for (int o = 0; o < n; ++o) {
        const unsigned long long other = cand_s[o];
        rank += other > mine ? 1 : 0;
        if (other == mine && o != j) rank += ahead(other, cand_i[o], cand_x[o], mine, cand_i[j], cand_x[j]) ? 1 : 0;
      }
      if (rank < k) write(rank, cand_s[j], cand_i[j]);
    }
    for (int r = n + tid; r < k; r += kThreads) write(r, 0, -1);
    return;
  }
  // more ties than there is room for: one after another
  unsigned long long last_s = ~0ull;
  long long last_i = -1;
  float last_x = 0.f;
  for (int r = 0; r < k; ++r) {
    unsigned long long s = 0;
    long long at = -1;
    float x = 0.f;
    for (int e = tid; e < lists * k; e += kThreads) {
      const unsigned long long q = key_of(e / k, e % k);
      if (q == 0 || q < s || q > last_s) continue;
      const long long i = place_of(e / k, e % k);
      const float y = value_at(e / k, e % k);
      if (ahead(last_s, last_i, last_x, q, i, y) && (at < 0 || ahead(q, i, y, s, at, x))) s = q, at = i, x = y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long q = __shfl_xor_sync(kAll, s, o);
      const long long i = __shfl_xor_sync(kAll, at, o);
      const float y = __shfl_xor_sync(kAll, x, o);
      if (i >= 0 && (at < 0 || ahead(q, i, y, s, at, x))) s = q, at = i, x = y;
    }
    if (lane == 0) {
      best_s[warp] = s;
      best_i[warp] = at;
      best_x[warp] = x;
    }
    __syncthreads();
    s = 0;
    at = -1;
    for (int w = 0; w < kWarps; ++w)
      if (best_i[w] >= 0 && (at < 0 || ahead(best_s[w], best_i[w], best_x[w], s, at, x))) s = best_s[w], at = best_i[w], x = best_x[w];
    __syncthreads();
    if (tid == 0) write(r, s, at);
    if (at < 0) {
      for (int q = r + 1 + tid; q < k; q += kThreads) write(q, 0, -1);
      break;
    }
    last_s = s;
    last_i = at;
    last_x = x;
  }
}

// ------------------------------------------------------------------ reordering of the cache
//
// Beam b continues its parent a: its first L rows become a's.  Whole pages are never written
// again, so the table takes a's pages for them.  The page that is still being written, rows
// L mod page_size of it, goes by copy into b's spare page, and the page that b had there is
// its next spare.  Copies read tables, spare pages and parents, and come first; then the
// tables and spare pages change in place, a column by one thread of a block.

constexpr int kMaxLayers = 64;
constexpr int kCopyUnroll = 6;

struct ReorderArgs {
  int batch, beams, page_size, max_pages, kv_dtype, num_layers;
  long long num_pages;
  int* block_tables;       // [batch * beams, max_pages]
  const int* seq_lens;     // [batch * beams]
  const int* parents;      // [batch, beams]
  int* spare;              // [batch * beams]
  int* status;
  void* cache[kMaxLayers];
};

// Length of a request's beams, -1 where it is not one (flagged).
__device__ __forceinline__ int beams_length(const ReorderArgs& a, int request) {
  const int* len = a.seq_lens + (size_t)request * a.beams;
  const int L = len[0];
  bool same = L >= 0 && L <= a.max_pages * (long long)a.page_size;
  for (int w = threadIdx.x & 31; w < a.beams; w += 32) same = same && len[w] == L;
  same = __all_sync(kAll, same);
  if (!same && a.status && threadIdx.x == 0) atomicOr(a.status, kStatusSeqLen);
  return same ? L : -1;
}
__device__ __forceinline__ int parent_of(const ReorderArgs& a, int b, int w) {
  const int p = a.parents[b];
  return p >= 0 && p < a.beams ? p : w;  // none: the beam stays as it is
}
__device__ __forceinline__ bool is_page(const ReorderArgs& a, int id) { return id >= 0 && id < a.num_pages; }

__global__ void __launch_bounds__(kThreads)
reorder_copy_kernel(const __grid_constant__ ReorderArgs a) {
  ptx::pdl_launch_dependents();
  const int b = blockIdx.x, request = b / a.beams, w = b - request * a.beams;
  const int L = beams_length(a, request);
  if (L < 0) return;
  const int p = parent_of(a, b, w), whole = L / a.page_size, rest = L - whole * a.page_size;
  if (threadIdx.x == 0 && a.status && (a.parents[b] < -1 || a.parents[b] >= a.beams)) atomicOr(a.status, kStatusQLen);
  if (p == w || rest == 0) return;
  const int src = a.block_tables[(size_t)(request * a.beams + p) * a.max_pages + whole], dst = a.spare[b];
  if (!is_page(a, src) || !is_page(a, dst)) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusPage);
    return;
  }
  const size_t row = a.kv_dtype == kKvFp4 ? kFp4RowBytes : a.kv_dtype == kKvFp8 ? kQkDim : 2 * kQkDim;
  char* cache = static_cast<char*>(a.cache[blockIdx.y]);
  const char* from = cache + (size_t)src * a.page_size * row;
  char* to = cache + (size_t)dst * a.page_size * row;
  const int units = (int)(rest * (a.kv_dtype == kKvFp4 ? (size_t)kFp4CodeBytes : row) / 16);
  const int each = (units + gridDim.z - 1) / gridDim.z, begin = blockIdx.z * each, end = min(units, begin + each);
  for (int u = begin + threadIdx.x; u < end; u += kThreads * kCopyUnroll) {
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (u + i * kThreads < end) x[i] = reinterpret_cast<const uint4*>(from)[u + i * kThreads];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (u + i * kThreads < end) reinterpret_cast<uint4*>(to)[u + i * kThreads] = x[i];
  }
  if (a.kv_dtype == kKvFp4 && blockIdx.z == 0) {  // the rows' scales, 36 bytes each
    const size_t at = (size_t)a.page_size * kFp4CodeBytes;
    for (int i = threadIdx.x; i < rest * (kFp4ScaleBytes / 4); i += kThreads)
      reinterpret_cast<uint32_t*>(to + at)[i] = reinterpret_cast<const uint32_t*>(from + at)[i];
  }
}

constexpr int kColumns = 32;

__global__ void __launch_bounds__(kThreads)
reorder_tables_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int tile[kMaxK][kColumns];
  const int request = blockIdx.x;
  ptx::pdl_wait();
  const int L = beams_length(a, request);
  if (L < 0) return;
  const int whole = L / a.page_size, rest = L - whole * a.page_size, last = rest > 0 ? whole + 1 : whole;
  int* tables = a.block_tables + (size_t)request * a.beams * a.max_pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c0 = blockIdx.y * kColumns; c0 < last; c0 += gridDim.y * kColumns) {
    const int c = c0 + lane;
    for (int w = warp; w < a.beams; w += kWarps)
      if (c < last) tile[w][lane] = tables[(size_t)w * a.max_pages + c];
    __syncthreads();
    for (int w = warp; w < a.beams; w += kWarps) {
      const int b = request * a.beams + w, p = parent_of(a, b, w);
      if (p == w || c >= last) continue;
      if (c < whole) {
        tables[(size_t)w * a.max_pages + c] = tile[p][lane];
      } else {
        const int src = tile[p][lane], dst = a.spare[b];
        if (!is_page(a, src) || !is_page(a, dst)) continue;  // (nothing was copied, and it is flagged)
        tables[(size_t)w * a.max_pages + c] = dst;
        a.spare[b] = tile[w][lane];
      }
    }
    __syncthreads();
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct BeamPlan {
  int parts, share, blocks;
  size_t value, token, bytes;
};

// Even parts of each row: as many as make up to kBlocks blocks, which run all at once; and no more
// lists a request than the join ranks.  (Shares of all rows' chunks that end inside a row kept every SM as
// busy, but each end of a part costs 4 us: 64 x 4 beams over 131071 tokens took 30 us instead of
// 24.)
BeamPlan beam_plan(const mla_beam_params& p) {
  const int per_chunk = kThreads * kVectors * (p.logits_dtype == MLA_LOGITS_FP32 ? 4 : 8);
  const long long rows = (long long)p.batch * p.beams;
  BeamPlan b;
  const long long chunks = ((long long)p.vocab + per_chunk - 1) / per_chunk;
  const long long want = std::min({chunks, std::max(1LL, kBlocks / std::max(rows, 1LL)), (long long)kMaxLists / p.beams});
  b.share = (int)((chunks + want - 1) / want);
  b.parts = (int)((chunks + b.share - 1) / b.share);
  b.blocks = (int)(rows * b.parts);
  const size_t lists = (size_t)rows * b.parts;
  b.value = align_up(sizeof(Part) * lists, 256);
  b.token = b.value + align_up(sizeof(float) * lists * p.k, 256);
  b.bytes = b.token + align_up(sizeof(int) * lists * p.k, 256);
  return b;
}

int beam_check(const mla_beam_params* p) {
  if (!p) return MLA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->beams < 1 || p->k < 1 || p->vocab < 1) return MLA_ERR_INVALID_ARG;
  if (p->logits_dtype != MLA_LOGITS_FP32 && p->logits_dtype != MLA_LOGITS_BF16 && p->logits_dtype != MLA_LOGITS_FP16)
    return MLA_ERR_INVALID_ARG;
  if (p->beams > kMaxK || p->k > kMaxK || p->vocab > (1 << 28) || p->batch > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

cudaError_t launch_dependent(const void* kernel, dim3 grid, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace
}  // namespace mla

extern "C" {

size_t mla_beam_workspace_size(const mla_beam_params* params) {
  if (mla::beam_check(params) != MLA_OK || params->batch == 0) return 0;
  return mla::beam_plan(*params).bytes;
}

int mla_beam_select(const mla_beam_params* params, const void* logits, int64_t batch_stride, int64_t beam_stride,
                    const float* scores, const uint8_t* finished, float* scores_out, int32_t* tokens_out,
                    int32_t* parents_out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mla;
  const int rc = beam_check(params);
  if (rc != MLA_OK) return rc;
  const mla_beam_params& p = *params;
  if (finished && (p.end_token < 0 || p.end_token >= p.vocab)) return MLA_ERR_INVALID_ARG;
  if (p.batch == 0) return MLA_OK;
  if (!logits || !scores || !scores_out || !tokens_out || !parents_out || !workspace) return MLA_ERR_INVALID_ARG;
  if (batch_stride < 0 || beam_stride < 0) return MLA_ERR_INVALID_ARG;
  const size_t size = p.logits_dtype == MLA_LOGITS_FP32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(scores, 4) || !aligned(scores_out, 4) || !aligned(tokens_out, 4) ||
      !aligned(parents_out, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGNMENT;
  if (workspace_bytes < mla_beam_workspace_size(params)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const BeamPlan plan = beam_plan(p);
  char* ws = static_cast<char*>(workspace);
  Parts parts{reinterpret_cast<Part*>(ws), reinterpret_cast<float*>(ws + plan.value),
              reinterpret_cast<int*>(ws + plan.token), plan.parts, plan.share};
  const Logits in{logits, batch_stride, beam_stride, p.beams, p.vocab};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)plan.blocks);
  const bool whole = aligned(logits, 16) && (p.batch == 1 || batch_stride * size % 16 == 0) &&
                     (p.beams == 1 || beam_stride * size % 16 == 0);
  auto kernel = p.logits_dtype == MLA_LOGITS_FP32 ? (whole ? beam_parts_kernel<float, false> : beam_parts_kernel<float, true>)
                : p.logits_dtype == MLA_LOGITS_BF16
                    ? (whole ? beam_parts_kernel<__nv_bfloat16, false> : beam_parts_kernel<__nv_bfloat16, true>)
                    : (whole ? beam_parts_kernel<__half, false> : beam_parts_kernel<__half, true>);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
    return MLA_ERR_CUDA;
  kernel<<<grid, kThreads, kSmem, s>>>(in, scores, finished, p.k, parts);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  int beams = p.beams, k = p.k, end = p.end_token;
  void* args[] = {&scores, &finished, &beams, &k, &end, &parts, &scores_out, &tokens_out, &parents_out};
  return launch_dependent(reinterpret_cast<const void*>(beam_join_kernel), dim3((unsigned)p.batch), s, args) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

int mla_cache_reorder(const mla_reorder_params* params, void* const* caches, int32_t num_layers, int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* parents, int32_t* spare_pages, int32_t* status,
                      void* stream) {
  using namespace mla;
  if (!params) return MLA_ERR_INVALID_ARG;
  const mla_reorder_params& p = *params;
  if (p.batch < 0 || p.beams < 1 || p.max_pages_per_req < 1 || p.num_pages < 1 || num_layers < 0)
    return MLA_ERR_INVALID_ARG;
  if (p.kv_dtype != MLA_KV_BF16 && p.kv_dtype != MLA_KV_FP8_E4M3 && p.kv_dtype != MLA_KV_FP4_E2M1)
    return MLA_ERR_INVALID_ARG;
  if (p.page_size != 32 && p.page_size != 64) return MLA_ERR_UNSUPPORTED;
  if (p.beams > kMaxK || (long long)p.batch * p.beams > (1 << 24) || p.num_pages > (1LL << 31) / p.page_size)
    return MLA_ERR_UNSUPPORTED;
  if (p.batch == 0) return MLA_OK;
  if (!block_tables || !seq_lens || !parents || !spare_pages || (num_layers > 0 && !caches)) return MLA_ERR_INVALID_ARG;
  if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(parents, 4) || !aligned(spare_pages, 4) ||
      (status && !aligned(status, 4)))
    return MLA_ERR_ALIGNMENT;
  for (int l = 0; l < num_layers; ++l) {
    if (!caches[l]) return MLA_ERR_INVALID_ARG;
    if (!aligned(caches[l], 16)) return MLA_ERR_ALIGNMENT;
  }
  ReorderArgs a = {};
  a.batch = p.batch;
  a.beams = p.beams;
  a.page_size = p.page_size;
  a.max_pages = p.max_pages_per_req;
  a.kv_dtype = p.kv_dtype;
  a.num_pages = p.num_pages;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.spare = spare_pages;
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)p.batch * p.beams;
  for (int l0 = 0; l0 < num_layers; l0 += kMaxLayers) {
    a.num_layers = std::min(kMaxLayers, num_layers - l0);
    for (int l = 0; l < a.num_layers; ++l) a.cache[l] = caches[l0 + l];
    const unsigned parts = (unsigned)std::max(1LL, std::min(8LL, 608 / (rows * a.num_layers)));
    reorder_copy_kernel<<<dim3((unsigned)rows, (unsigned)a.num_layers, parts), kThreads, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  }
  void* args[] = {&a};
  const unsigned columns = (unsigned)((p.max_pages_per_req + kColumns - 1) / kColumns);
  return launch_dependent(reinterpret_cast<const void*>(reorder_tables_kernel),
                          dim3((unsigned)p.batch, std::min(columns, 64u)), s, args) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // extern "C"
