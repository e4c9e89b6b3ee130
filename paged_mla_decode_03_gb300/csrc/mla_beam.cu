// Beam search over the paged cache: the choice of the next beams and the reordering of the
// cache that follows from it.
//
// Selection.  A request's beams w have scores c_w and rows x_w of logits over a vocabulary of
// V; a continuation (w, v) scores
//   s(w, v) = c_w + x_w[v] - lse_w,   lse_w = ln sum_v exp(x_w[v]),
// and the k best are wanted, the lowest (w, v) first among equals.  The logits are read once.
// Within a beam the order is that of the logits themselves, so each block keeps the k largest
// logits of its part of a row, exactly, beside the part's maximum and sum of exponentials; one
// block a request then compares the scores of all parts' candidates in 64 bits.  What decides
// between nearly equal candidates of two beams is lse: exponentials are of differences from the
// maximum, taken with the product by log2(e) in two parts, and their sums leave a thread
// in 64 bits.
//
// What bounds it: the bytes of the logits, where there are many; a chain of two launches, else.
// A row goes through a block in chunks that stay in registers, the next chunk's loads on their
// way.  A thread keeps the maximum and the sum of its own values, so a chunk takes one barrier:
// it asks whether any value passes the k-th largest so far.  Those that do are collected and
// ranked by counting.  The first chunk, and one with very many of them, has a threshold first:
// of the maxima of 64 groups of its values the k-th largest has at least k values at or
// above it, and seldom many more.
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
constexpr int kVectors = 4;             // 16-byte units of a thread in a chunk
constexpr int kGroups = 64;             // groups of a chunk's values: four threads each
constexpr int kMaxK = 64;
constexpr int kRoom = 1024;             // candidates collected at most (ties may pass it)
constexpr int kMaxLists = 128;          // candidate lists of a request at most
constexpr unsigned kAll = 0xffffffffu;
constexpr float kNone = -INFINITY;

// Order-preserving bits of a float (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ bool before(float xa, int ia, float xb, int ib) { return xa > xb || (xa == xb && ia < ib); }

__device__ __forceinline__ unsigned long long ordered64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double from_ordered64(unsigned long long u) {
  return __longlong_as_double((long long)(u ^ ((u >> 63) ? 1ull << 63 : ~0ull)));
}

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
// e^d for d <= 0: the product by log2(e) in two parts, so that its rounding is not of log2(e).
__device__ __forceinline__ float exp_of(float d) { return ptx::ex2(fmaf(d, kLog2eHi, d * kLog2eLo)); }

struct Part {  // of a row, as one block found it
  double sum;  // of exp(x - top)
  float top;
  int pad;
};

struct Parts {
  Part* part;      // [rows][parts]
  float* value;    // [rows][parts][k], descending; -inf: none
  int* token;      // [rows][parts][k]
  int parts, chunks;  // parts of a row, chunks of a part
};

}  // namespace

// The k largest values of a chunk and of the list before it, one after another: for chunks
// with more ties than there is room for.  (Apart, and from memory: it is hardly ever called, and would
// take the other path's registers.)
template <typename T>
__device__ __noinline__ int select_slowly(const T* x, int begin, int end, int k, int n_top, const float* top_x,
                                          const int* top_i, float* next_x, int* next_i, unsigned long long* best_key) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float last_x = INFINITY;
  int last_i = -1, found = 0;
  for (; found < k; ++found) {
    unsigned long long key = 0;  // (order of the value, lowest index); 0: none
    auto look = [&](float y, int i) {
      if (!(y > kNone) || !before(last_x, last_i, y, i)) return;
      const unsigned long long q = ((unsigned long long)ordered(y) << 32) | (0xffffffffu - (unsigned)i);
      key = q > key ? q : key;
    };
#pragma unroll 1
    for (int i = begin + tid; i < end; i += kThreads) look((float)x[i], i);
    if (tid < n_top) look(top_x[tid], top_i[tid]);
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
    if (key == 0) break;
    const uint32_t u = (uint32_t)(key >> 32);
    last_x = __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
    last_i = (int)(0xffffffffu - (uint32_t)key);
    if (tid == 0) {
      next_x[found] = last_x;
      next_i[found] = last_i;
    }
  }
  return found;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
beam_parts_kernel(Logits in, const float* __restrict__ scores, const unsigned char* __restrict__ finished, int k,
                  Parts out) {
  constexpr int kPer = 16 / (int)sizeof(T);  // values of a unit
  constexpr int kHalves = 4 / (int)sizeof(T), kUnits = kThreads * kVectors;
  __shared__ float group_max[kGroups], threshold;
  __shared__ float cand_x[kRoom], top_x[2][kMaxK];
  __shared__ int cand_i[kRoom], top_i[2][kMaxK], n_cand;
  __shared__ unsigned long long best_key[kWarps];
  __shared__ float warp_max[kWarps];
  __shared__ double warp_sum[kWarps];
  ptx::pdl_launch_dependents();
  const int row = blockIdx.x, part = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a beam that has ended, or has no score, offers nothing that its logits decide
  if (finished && finished[row]) return;
  if (!(fabsf(scores[row]) < INFINITY)) return;
  const T* x = static_cast<const T*>(in.base) + (row / in.beams) * in.batch_stride + (row % in.beams) * in.beam_stride;
  // units of 16 aligned bytes; the first and last may hold values outside the row
  const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int units = (off + in.vocab + kPer - 1) / kPer;
  const int c0 = part * out.chunks, c1 = min(c0 + out.chunks, (units + kUnits - 1) / kUnits);
  auto load = [&](int c, uint4 (&w)[kVectors]) {
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      const int u = c * kUnits + v * kThreads + tid, i0 = u * kPer - off;
      if (c < c1 && i0 >= 0 && i0 + kPer <= in.vocab) {
        w[v] = __ldcs(reinterpret_cast<const uint4*>(x + i0));
      } else {  // -inf where there is no value
        constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __nv_bfloat16>::value ? 0xff80u : 0xfc00u;
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = 0;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const int i = i0 + j * kHalves + h;
            uint32_t bits = none;
            if (c < c1 && i >= 0 && i < in.vocab) {
              if constexpr (sizeof(T) == 4) bits = reinterpret_cast<const uint32_t*>(x)[i];
              else bits = reinterpret_cast<const unsigned short*>(x)[i];
            }
            e[j] |= bits << (16 * h);
          }
        }
        w[v] = make_uint4(e[0], e[1], e[2], e[3]);
      }
    }
  };
  auto word_of = [](const uint4& w, int j) { return j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w; };
  uint4 now[kVectors], next_words[kVectors];
  load(c0, now);
  int n_top = 0, cur = 0;
  float so_far = kNone;        // the list's last, once it is full
  float m = kNone, sum = 0.f, low = 0.f;  // this thread's maximum, and sum of exp(x - m) with its rounding
  for (int c = c0; c < c1; ++c) {
    load(c + 1, next_words);
    auto at = [&](int v, int e) { return value_of<T>(word_of(now[v], e / kHalves), e % kHalves); };
    float mine = kNone;
#pragma unroll
    for (int v = 0; v < kVectors; ++v)
#pragma unroll
      for (int e = 0; e < kPer; ++e) mine = fmaxf(mine, at(v, e));
    const bool any = __syncthreads_or(mine > so_far);
    if (mine > m) {
      const float f = exp_of(m - mine);  // m = -inf: 0
      sum *= f;
      low *= f;
      m = mine;
    }
    {
      const float ref = m == kNone ? 0.f : m;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kVectors; ++v)
#pragma unroll
        for (int e = 0; e < kPer; ++e) s[e & 3] += exp_of(at(v, e) - ref);
      const float a = (s[0] + s[1]) + (s[2] + s[3]), t = sum + a, z = t - sum;
      low += (sum - (t - z)) + (a - z);
      sum = t;
    }
    if (any) {
      // values above the list's last; the first chunk's, or of too many, from a threshold on
      bool thin = n_top < k;
      int n = 0;
      for (;;) {
        if (thin) {
          float g = fmaxf(mine, __shfl_xor_sync(kAll, mine, 1));
          g = fmaxf(g, __shfl_xor_sync(kAll, g, 2));
          if ((lane & 3) == 0) group_max[tid >> 2] = g;
        }
        if (tid == 0) n_cand = n_top;
        __syncthreads();
        if (thin && tid < kGroups) {
          const float g = group_max[tid];
          int rank = 0;
#pragma unroll 8
          for (int j = 0; j < kGroups; ++j) rank += before(group_max[j], j, g, tid) ? 1 : 0;
          if (rank == k - 1) threshold = g;
        }
        if (tid < n_top) {  // the k largest so far are candidates again
          cand_x[tid] = top_x[cur][tid];
          cand_i[tid] = top_i[cur][tid];
        }
        if (thin) __syncthreads();
        const float least = thin ? threshold : kNone;
        // (a later token loses a tie against the list: strictly above its last)
        if (mine >= least && mine > so_far) {
#pragma unroll
          for (int v = 0; v < kVectors; ++v)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const float y = at(v, e);
              if (y >= least && y > so_far) {
                const int p = atomicAdd(&n_cand, 1);
                if (p < kRoom) {
                  cand_x[p] = y;
                  cand_i[p] = (c * kUnits + v * kThreads + tid) * kPer + e - off;
                }
              }
            }
        }
        __syncthreads();
        n = n_cand;
        if (thin || n <= kRoom) break;
        thin = true;
        __syncthreads();  // (every thread has read the count)
      }
      const int next = cur ^ 1;
      if (n <= kRoom) {
        for (int j = tid; j < n; j += kThreads) {
          const float y = cand_x[j];
          const int i = cand_i[j];
          int rank = 0;
          for (int o = 0; o < n; ++o) rank += before(cand_x[o], cand_i[o], y, i) ? 1 : 0;
          if (rank < k) {
            top_x[next][rank] = y;
            top_i[next][rank] = i;
          }
        }
        n_top = min(k, n);
      } else {
        n_top = select_slowly(x, max(0, c * kUnits * kPer - off), min(in.vocab, (c + 1) * kUnits * kPer - off), k, n_top,
                              top_x[cur], top_i[cur], top_x[next], top_i[next], best_key);
      }
      cur = next;
      __syncthreads();
      so_far = n_top == k ? top_x[cur][k - 1] : kNone;
    }
#pragma unroll
    for (int v = 0; v < kVectors; ++v) now[v] = next_words[v];
  }
  const size_t list = (size_t)row * out.parts + part;
  if (tid < k) {
    const bool on = tid < n_top;
    out.value[list * k + tid] = on ? top_x[cur][tid] : kNone;
    out.token[list * k + tid] = on ? top_i[cur][tid] : -1;
  }
  // the threads' sums, each relative to its own maximum, to the part's
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  if (lane == 0) warp_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_max[w]);
  // (no value: 0; a NaN, or an infinity's, stays one)
  double s = ((double)sum + (double)low) * (double)exp_of(m - (top == kNone ? 0.f : top));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) s += warp_sum[w];
    out.part[list] = Part{s, top, 0};
  }
}

// One block a request: the rows' normalisers, then the k best of all lists.
constexpr int kDepths = 4, kStaged = 2048;

__global__ void __launch_bounds__(kThreads)
beam_join_kernel(const float* __restrict__ scores, const unsigned char* __restrict__ finished, int beams, int k,
                 int vocab, int end_token, Parts in, float* __restrict__ scores_out, int* __restrict__ tokens_out,
                 int* __restrict__ parents_out) {
  __shared__ double row_log[kMaxK], row_score[kMaxK];  // (beams are 64 at most, too)
  __shared__ float row_top[kMaxK];
  __shared__ int row_kind[kMaxK];  // 0: nothing, 1: lists, 2: has ended
  __shared__ float row_least[kMaxK];
  __shared__ unsigned long long key[kDepths][kMaxLists], cand_s[kRoom], best_s[kWarps], threshold;
  __shared__ long long cand_i[kRoom], best_i[kWarps];
  __shared__ float staged[kStaged];
  __shared__ int n_cand;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lists = beams * in.parts;
  const size_t list0 = (size_t)b * lists;
  ptx::pdl_wait();
  // (beside the normalisers; lists that nobody wrote are not looked at)
  const bool near = lists * k <= kStaged;
  if (near)
    for (int e = tid; e < lists * k; e += kThreads) staged[e] = in.value[list0 * k + e];
  for (int w = warp; w < beams; w += kWarps) {
    const int row = b * beams + w;
    const float c = scores[row];
    const bool scored = fabsf(c) < INFINITY, done = finished && finished[row];
    float top = kNone;
    double sum = 0.0;
    if (scored && !done) {
      for (int p = lane; p < in.parts; p += 32) top = fmaxf(top, in.part[(size_t)row * in.parts + p].top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      for (int p = lane; p < in.parts; p += 32) {
        const Part q = in.part[(size_t)row * in.parts + p];
        sum += q.sum * exp((double)q.top - (top == kNone ? 0.0 : (double)top));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    if (lane == 0) {
      // an infinity or a NaN among the logits, or nothing above -inf: no continuation
      const bool ok = scored && !done && fabsf(top) < INFINITY && sum > 0.0 && sum < 1e300;
      row_kind[w] = scored && done ? 2 : ok ? 1 : 0;
      row_top[w] = top;
      row_log[w] = ok ? log(sum) : 0.0;
      row_score[w] = (double)c;
    }
  }
  if (tid == 0) n_cand = 0;
  __syncthreads();
  constexpr unsigned long long kNothing = 0;  // below the key of any score
  // candidate j of a list: its key, and its place (w, token)
  auto logit = [&](int l, int j) { return near ? staged[l * k + j] : in.value[(list0 + l) * k + j]; };
  auto key_of = [&](int l, int j) -> unsigned long long {
    const int w = l / in.parts, kind = row_kind[w];
    if (kind == 2) return j == 0 && l == w * in.parts ? ordered64(row_score[w]) : kNothing;
    if (kind == 0) return kNothing;
    const float x = logit(l, j);
    return x == kNone ? kNothing : ordered64((((double)x - row_top[w]) - row_log[w]) + row_score[w]);
  };
  auto place_of = [&](int l, int j) -> long long {
    const int w = l / in.parts;
    return (long long)w * vocab + (row_kind[w] == 2 ? end_token : in.token[(list0 + l) * k + j]);
  };
  // A threshold that at least k candidates are at or above: for some depths d, the
  // ceil(k / d)-th largest of the lists' d-th candidates, and of these the largest.  (With d
  // = 1, 4, 16, 64 fewer than 4 k candidates for each d pass it, ties apart, however the
  // beams' scores lie.)
  for (int t = tid; t < kDepths * lists; t += kThreads) {
    const int e = t / lists, l = t - e * lists, d = min(1 << (2 * e), k);
    key[e][l] = key_of(l, d - 1);
  }
  if (tid == 0) threshold = kNothing;
  __syncthreads();
  for (int t = tid; t < kDepths * lists; t += kThreads) {
    const int e = t / lists, l = t - e * lists, d = min(1 << (2 * e), k), want = (k + d - 1) / d;
    if (want > lists) continue;
    const unsigned long long s = key[e][l];
    int rank = 0;
    for (int o = 0; o < lists; ++o) rank += (key[e][o] > s || (key[e][o] == s && o < l)) ? 1 : 0;
    if (rank == want - 1) atomicMax(&threshold, s);
  }
  __syncthreads();
  const unsigned long long least = max(threshold, kNothing + 1);
  // the same for a beam's logits, a little lower, which spares most the sums in 64 bits
  if (tid < beams) {
    // (off by some 2^-23 of the largest term at most)
    const float score = threshold == kNothing ? kNone : (float)from_ordered64(threshold), c = (float)row_score[tid];
    const float log_sum = (float)row_log[tid], top = row_top[tid];
    row_least[tid] = score - c + log_sum + top - (fabsf(score) + fabsf(c) + fabsf(log_sum) + fabsf(top)) * 1e-6f;
  }
  __syncthreads();
  for (int e = tid; e < lists * k; e += kThreads) {
    const int l = e / k, j = e - l * k;
    if (key[0][l] < least) continue;
    if (row_kind[l / in.parts] == 1 && logit(l, j) < row_least[l / in.parts]) continue;
    const unsigned long long s = key_of(l, j);
    if (s < least) continue;
    const int p = atomicAdd(&n_cand, 1);
    if (p < kRoom) {
      cand_s[p] = s;
      cand_i[p] = place_of(l, j);
    }
  }
  __syncthreads();
  const int n = n_cand;
  auto ahead = [](unsigned long long sa, long long ia, unsigned long long sb, long long ib) {
    return sa > sb || (sa == sb && ia < ib);
  };
  auto write = [&](int rank, unsigned long long s, long long i) {
    scores_out[(size_t)b * k + rank] = s == kNothing ? kNone : (float)from_ordered64(s);
    tokens_out[(size_t)b * k + rank] = i < 0 ? -1 : (int)(i % vocab);
    parents_out[(size_t)b * k + rank] = i < 0 ? -1 : (int)(i / vocab);
  };
  if (n <= kRoom) {
    for (int j = tid; j < n; j += kThreads) {
      int rank = 0;
      for (int o = 0; o < n; ++o) rank += ahead(cand_s[o], cand_i[o], cand_s[j], cand_i[j]) ? 1 : 0;
      if (rank < k) write(rank, cand_s[j], cand_i[j]);
    }
    for (int r = n + tid; r < k; r += kThreads) write(r, kNothing, -1);
    return;
  }
  // more ties than there is room for: one after another
  unsigned long long last_s = ~0ull;
  long long last_i = -1;
  for (int r = 0; r < k; ++r) {
    unsigned long long s = kNothing;
    long long at = -1;
    for (int e = tid; e < lists * k; e += kThreads) {
      const unsigned long long q = key_of(e / k, e % k);
      if (q == kNothing || q < s || q > last_s) continue;
      const long long i = place_of(e / k, e % k);
      if (ahead(last_s, last_i, q, i) && (at < 0 || ahead(q, i, s, at))) s = q, at = i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long q = __shfl_xor_sync(kAll, s, o);
      const long long i = __shfl_xor_sync(kAll, at, o);
      if (i >= 0 && (at < 0 || ahead(q, i, s, at))) s = q, at = i;
    }
    if (lane == 0) {
      best_s[warp] = s;
      best_i[warp] = at;
    }
    __syncthreads();
    s = kNothing;
    at = -1;
    for (int w = 0; w < kWarps; ++w)
      if (best_i[w] >= 0 && (at < 0 || ahead(best_s[w], best_i[w], s, at))) s = best_s[w], at = best_i[w];
    __syncthreads();
    if (tid == 0) write(r, s, at);
    if (at < 0) {
      for (int q = r + 1 + tid; q < k; q += kThreads) write(q, kNothing, -1);
      break;
    }
    last_s = s;
    last_i = at;
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
  if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
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
        tables[(size_t)w * a.max_pages + c] = a.spare[b];
        a.spare[b] = tile[w][lane];
      }
    }
    __syncthreads();
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct BeamPlan {
  int parts, chunks;
  size_t value, token, bytes;
};

// Parts of a row.  Enough blocks for some eight on every SM, where there are so many chunks;
// and no more lists a request than the join ranks.
BeamPlan beam_plan(const mla_beam_params& p) {
  const int per_chunk = kThreads * kVectors * (p.logits_dtype == MLA_LOGITS_FP32 ? 4 : 8);
  const long long rows = (long long)p.batch * p.beams;
  // (a row that starts off a 16-byte boundary has a unit more)
  const int chunks = (int)((p.vocab + 8LL + per_chunk - 1) / per_chunk);
  const long long want = std::max(1LL, (1216 + rows - 1) / std::max(rows, 1LL));
  BeamPlan b;
  b.parts = (int)std::min<long long>(std::min<long long>(chunks, want), kMaxLists / p.beams);
  b.chunks = (chunks + b.parts - 1) / b.parts;
  b.parts = (chunks + b.chunks - 1) / b.chunks;
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
  const BeamPlan plan = beam_plan(p);
  if (workspace_bytes < plan.bytes) return MLA_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  Parts parts{reinterpret_cast<Part*>(ws), reinterpret_cast<float*>(ws + plan.value),
              reinterpret_cast<int*>(ws + plan.token), plan.parts, plan.chunks};
  const Logits in{logits, batch_stride, beam_stride, p.beams, p.vocab};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(p.batch * p.beams), (unsigned)plan.parts);
  if (p.logits_dtype == MLA_LOGITS_FP32)
    beam_parts_kernel<float><<<grid, kThreads, 0, s>>>(in, scores, finished, p.k, parts);
  else if (p.logits_dtype == MLA_LOGITS_BF16)
    beam_parts_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(in, scores, finished, p.k, parts);
  else
    beam_parts_kernel<__half><<<grid, kThreads, 0, s>>>(in, scores, finished, p.k, parts);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  int beams = p.beams, k = p.k, vocab = p.vocab, end = p.end_token;
  void* args[] = {&scores, &finished, &beams, &k, &vocab, &end, &parts, &scores_out, &tokens_out, &parents_out};
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
