// Writing and reading rows of the paged latent cache: mla_cache_append,
// mla_cache_gather and mla_rope_table.
//
// append, for new token i of request b at position p = seq_lens[b] - q_len + i:
//   rstd = 1 / sqrt(mean(x^2) + eps)             x: the 512-wide latent
//   y    = [x * rstd * w,  R_p k]                k: the 64 RoPE dims
//   cache row p = quantise(y / kv_scale)
//   query row h = quantise([q_nope_h, R_p q_pe_h] / q_scale)
// R_p turns each pair (a, b) into (a c - b s, b c + a s), with c and s from
// row p of a table.  Every step is a separately rounded fp32 operation and the
// sum of squares carries its rounding error along (two fp32 words), so the mean is
// the rounded exact one and a row does not depend on how the sum is split over
// lanes.  (rstd has two roundings more, of mean + eps and of the root.)
//
// What bounds it: bytes.  A token moves 1152 B in and 324-1152 B out for the
// cache row and, per head, 1152 B in and 576 or 1152 B out for the query, with
// a few operations per value.  One launch does all of it, one warp per work
// unit (a token's cache row, or four heads of a token's query), so that a small
// call is one latency chain and a large one keeps every SM's loads in flight: a
// warp issues its nine 16-byte loads per lane before it looks up the token's
// request, position and rotation.  Measured: 8000 prompt tokens x 128 heads into 4
// bits with their queries (1.84 GB), append and gather together, 276 us: 6.67 TB/s, the
// rate of a plain copy.  128 x 128 heads (38 MB) with the gather 8.6 us in a graph, 4 x 32 x 128
// heads 8.4, 8 x 16 heads 2.8; launched one by one such calls take the host's 20 us.
//
// gather reads the same rows back as bf16 (value * kv_scale), one warp a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/mla_decode.h"
#include "mla_common.cuh"
#include "mla_fp4.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerUnit = 4;
constexpr unsigned kAll = 0xffffffffu;

struct RowMap {  // which cache row each token has
  int batch, q_len, page_size, max_pages;
  long long num_pages, total_q;
  const int* block_tables;
  const int* seq_lens;
  const int* qo_indptr;  // [B + 1], or nullptr: q_len tokens per request
  int* status;           // may be nullptr
};

struct AppendArgs {
  RowMap map;
  const __nv_bfloat16* latent;
  const __nv_bfloat16* k_pe;
  const __nv_bfloat16* norm_weight;  // [512] or nullptr: no norm
  const float* rope_table;           // [max_position][32 cos, 32 sin]
  const int* positions;              // [total_q] or nullptr: the cache position
  unsigned char* cache;
  const __nv_bfloat16* q_nope;  // nullptr: the query's first 512 dims stay as they are
  const __nv_bfloat16* q_pe;    // nullptr: no query
  unsigned char* query;
  long long latent_stride, k_pe_stride, q_nope_token, q_nope_head, q_pe_token, q_pe_head;
  int num_heads, max_position, half_style;
  float eps, inv_kv_scale, inv_q_scale;
};

__device__ __forceinline__ void flag(const RowMap& m, int bit) {
  if (m.status) atomicOr(m.status, bit);
}

struct Place {
  long long pos;   // logical position, or < 0: no row
  long long page;  // physical page
  int row;         // row within the page
};

// The cache row of token t: its request (the last b with qo_indptr[b] <= t,
// found by the warp in 32-way steps), position and page.  Tokens past the last
// request, positions outside the table and page ids outside the pool give
// pos = -1 (the latter two are flagged).  The same for all lanes.
__device__ __forceinline__ Place place_of(const RowMap& m, long long t, int lane) {
  Place pl{-1, 0, 0};
  int b, i, q;
  if (m.qo_indptr) {
    int lo = 0, hi = m.batch + 1;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + lane * step;
      const bool le = at < hi && (long long)__ldg(m.qo_indptr + at) <= t;
      const unsigned ball = __ballot_sync(kAll, le);
      if (!ball) return pl;  // before the first request
      lo = lo + (31 - __clz(ball)) * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    if (b >= m.batch) return pl;  // rows behind the last request
    const int q0 = __ldg(m.qo_indptr + b), q1 = __ldg(m.qo_indptr + b + 1);
    i = (int)(t - q0);
    q = q1 - q0;
    if (q0 < 0 || i < 0 || i >= q) {
      if (lane == 0) flag(m, kStatusQLen);
      return pl;
    }
  } else {
    b = (int)(t / m.q_len);
    i = (int)(t - (long long)b * m.q_len);
    q = m.q_len;
  }
  const long long L = __ldg(m.seq_lens + b);
  const long long pos = L - q + i;
  if (pos < 0 || L > (long long)m.max_pages * m.page_size) {
    if (lane == 0) flag(m, kStatusSeqLen);
    return pl;
  }
  const int pg = __ldg(m.block_tables + (long long)b * m.max_pages + pos / m.page_size);
  if (pg < 0 || pg >= m.num_pages) {
    if (lane == 0) flag(m, kStatusPage);
    return pl;
  }
  pl.pos = pos;
  pl.page = pg;
  pl.row = (int)(pos % m.page_size);
  return pl;
}

__device__ __forceinline__ void widen8(const uint4 x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 to_bf16x8(const float* f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
// Eight values times `s` as e4m3 (saturating; NaN stays NaN).
__device__ __forceinline__ uint2 to_e4m3x8(const float* f, float s) {
  uint32_t w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t a = ptx::f32x2_to_e4m3x2(__fmul_rn(f[4 * e], s), __fmul_rn(f[4 * e + 1], s));
    const uint32_t b = ptx::f32x2_to_e4m3x2(__fmul_rn(f[4 * e + 2], s), __fmul_rn(f[4 * e + 3], s));
    w[e] = a | (b << 16);
  }
  return make_uint2(w[0], w[1]);
}

// (c, s) of the eight RoPE dims [8 u, 8 u + 8) that a lane holds: four pairs
// when pairs are neighbours, eight when dim i goes with dim i + 32.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ Turn load_turn(const float* table, long long pos, int u, int half_style) {
  Turn t;
  const float4* row = reinterpret_cast<const float4*>(table + pos * 64);
  if (half_style) {
    const int k = 2 * (u & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 a = __ldg(row + k + e), b = __ldg(row + 8 + k + e);
      t.c[4 * e] = a.x; t.c[4 * e + 1] = a.y; t.c[4 * e + 2] = a.z; t.c[4 * e + 3] = a.w;
      t.s[4 * e] = b.x; t.s[4 * e + 1] = b.y; t.s[4 * e + 2] = b.z; t.s[4 * e + 3] = b.w;
    }
  } else {
    const float4 a = __ldg(row + u), b = __ldg(row + 8 + u);
    t.c[0] = a.x; t.c[1] = a.y; t.c[2] = a.z; t.c[3] = a.w;
    t.s[0] = b.x; t.s[1] = b.y; t.s[2] = b.z; t.s[3] = b.w;
  }
  return t;
}
// The rotation of unit u (of 8) of one row; the row's other units are in the
// neighbouring lanes (lane ^ 4 holds unit u ^ 4).  Called by whole warps.
__device__ __forceinline__ void turn8(float* f, const Turn& t, int u, int half_style) {
  if (half_style) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_xor_sync(kAll, f[e], 4);
      const float fc = __fmul_rn(f[e], t.c[e]), os = __fmul_rn(o, t.s[e]);
      f[e] = u < 4 ? __fsub_rn(fc, os) : __fadd_rn(fc, os);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = f[2 * e], b = f[2 * e + 1];
      f[2 * e] = __fsub_rn(__fmul_rn(a, t.c[e]), __fmul_rn(b, t.s[e]));
      f[2 * e + 1] = __fadd_rn(__fmul_rn(b, t.c[e]), __fmul_rn(a, t.s[e]));
    }
  }
}

// a + b as a rounded sum and its exact error (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// The warp's sum of y^2 over 16 values a lane.  Squares of bf16 values are exact
// in fp32 and hi + lo is their sum.
__device__ __forceinline__ float sum_of_squares(const float (&y)[16]) {
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float err;
    two_sum(hi, __fmul_rn(y[e], y[e]), hi, err);
    lo = __fadd_rn(lo, err);
  }
  for (int o = 16; o > 0; o >>= 1) {
    float err;
    const float h2 = __shfl_xor_sync(kAll, hi, o), l2 = __shfl_xor_sync(kAll, lo, o);
    two_sum(hi, h2, hi, err);
    lo = __fadd_rn(__fadd_rn(lo, l2), err);
  }
  return hi <= 3.4028235e38f ? __fadd_rn(hi, lo) : hi;  // an infinite sum has no error term
}

// Scale of a 16-dim group: e4m3 of amax / 6, its value and the factor that
// brings the group's values to e2m1's range (0 for a group of zeros).
__device__ __forceinline__ uint32_t group_scale(float amax, float& inv) {
  const uint32_t code = ptx::f32x2_to_e4m3x2(__fmul_rn(amax, 1.f / 6.f), 0.f) & 0xFFu;
  float v, unused;
  ptx::e4m3x2_to_f32x2(code, v, unused);
  inv = v > 0.f ? __frcp_rn(v) : 0.f;
  return code;
}

// The cache row of a token.  Lane l holds latent dims [16 l, 16 l + 16), and
// for l < 8 RoPE dims [8 l, 8 l + 8) (the other lanes repeat lane l % 8's).
template <int kKv>
__device__ __forceinline__ void append_row(const AppendArgs& a, long long t, int lane) {
  const uint4* lat = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
  const uint4* kpe = reinterpret_cast<const uint4*>(a.k_pe + t * a.k_pe_stride);
  const int u = lane & 7;
  const uint4 x0 = __ldg(lat + 2 * lane), x1 = __ldg(lat + 2 * lane + 1), xr = __ldg(kpe + u);
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (a.norm_weight) {
    const uint4* w = reinterpret_cast<const uint4*>(a.norm_weight);
    w0 = __ldg(w + 2 * lane);
    w1 = __ldg(w + 2 * lane + 1);
  }
  const Place pl = place_of(a.map, t, lane);
  if (pl.pos < 0) return;
  const long long rp = a.positions ? (long long)__ldg(a.positions + t) : pl.pos;
  if (rp < 0 || rp >= a.max_position) {
    if (lane == 0) flag(a.map, kStatusPosition);
    return;
  }
  const Turn turn = load_turn(a.rope_table, rp, u, a.half_style);
  float y[16], r[8];
  widen8(x0, y);
  widen8(x1, y + 8);
  widen8(xr, r);
  if (a.norm_weight) {
    float ss = sum_of_squares(y), eps = a.eps, back = 1.f;
    // latents near the top of bf16's range: the mean on a scale of 2^-192, and so rstd
    // on one of 2^96 (no lane diverges: the sum is the warp's; the latents themselves
    // stay as they are, small ones beside them would lose bits)
    if (ss > 3.4028235e38f) {
      float z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = __fmul_rn(y[e], 0x1p-96f);
      ss = sum_of_squares(z);
      back = 0x1p-96f;
      // (exact, or below every rounding of the mean, which is at least 2^-73 here)
      eps = __fmul_rn(__fmul_rn(eps, 0x1p-96f), 0x1p-96f);
    }
    const float rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.f / 512.f), eps));
    float w[16];
    widen8(w0, w);
    widen8(w1, w + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(__fmul_rn(__fmul_rn(y[e], rstd), back), w[e]);
  }
  turn8(r, turn, u, a.half_style);
  if (kKv == MLA_KV_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(a.cache + (pl.page * a.map.page_size + pl.row) * (2 * kQkDim));
    dst[2 * lane] = to_bf16x8(y);
    dst[2 * lane + 1] = to_bf16x8(y + 8);
    if (lane < 8) dst[64 + u] = to_bf16x8(r);
  } else if (kKv == MLA_KV_FP8_E4M3) {
    unsigned char* dst = a.cache + (pl.page * a.map.page_size + pl.row) * kQkDim;
    const uint2 p = to_e4m3x8(y, a.inv_kv_scale), q = to_e4m3x8(y + 8, a.inv_kv_scale);
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(p.x, p.y, q.x, q.y);
    if (lane < 8) reinterpret_cast<uint2*>(dst + kVDim)[u] = to_e4m3x8(r, a.inv_kv_scale);
  } else {
    unsigned char* page = a.cache + pl.page * a.map.page_size * kFp4RowBytes;
    unsigned char* codes = page + pl.row * kFp4CodeBytes;
    unsigned char* scales = page + a.map.page_size * kFp4CodeBytes + pl.row * kFp4ScaleBytes;
    float amax = 0.f, rmax = 0.f, inv, rinv;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      y[e] = __fmul_rn(y[e], a.inv_kv_scale);
      amax = fmaxf(amax, fabsf(y[e]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r[e] = __fmul_rn(r[e], a.inv_kv_scale);
      rmax = fmaxf(rmax, fabsf(r[e]));
    }
    rmax = fmaxf(rmax, __shfl_xor_sync(kAll, rmax, 1));  // two lanes share a group
    const uint32_t sc = group_scale(amax, inv), rsc = group_scale(rmax, rinv);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(y[e], inv);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = __fmul_rn(r[e], rinv);
    reinterpret_cast<uint2*>(codes)[lane] = make_uint2(ptx::f32x8_to_e2m1(y), ptx::f32x8_to_e2m1(y + 8));
    scales[lane] = (unsigned char)sc;
    if (lane < 8) reinterpret_cast<uint32_t*>(codes + 256)[u] = ptx::f32x8_to_e2m1(r);
    if (lane < 8 && (lane & 1) == 0) scales[32 + u / 2] = (unsigned char)rsc;
  }
}

// Four heads of a token's query: 8 loads per lane of the latent part, and one
// of the RoPE part (lane l: head l / 8, unit l % 8).
template <bool kQFp8>
__device__ __forceinline__ void append_query(const AppendArgs& a, long long t, int h0, int lane) {
  const int u = lane & 7, hr = h0 + (lane >> 3);
  uint4 x[2 * kHeadsPerUnit];
  if (a.q_nope) {
#pragma unroll
    for (int k = 0; k < 2 * kHeadsPerUnit; ++k) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q_nope + t * a.q_nope_token + (long long)(h0 + k / 2) * a.q_nope_head);
      x[k] = __ldg(src + 32 * (k & 1) + lane);
    }
  }
  const uint4 xr = __ldg(reinterpret_cast<const uint4*>(a.q_pe + t * a.q_pe_token +
                                                        (long long)hr * a.q_pe_head) + u);
  const Place pl = place_of(a.map, t, lane);
  if (pl.pos < 0) return;
  const long long rp = a.positions ? (long long)__ldg(a.positions + t) : pl.pos;
  if (rp < 0 || rp >= a.max_position) return;  // flagged by the token's cache row
  const Turn turn = load_turn(a.rope_table, rp, u, a.half_style);
  float r[8];
  widen8(xr, r);
  turn8(r, turn, u, a.half_style);
  const long long row0 = t * a.num_heads + h0;
  if (!kQFp8) {
    uint4* dst = reinterpret_cast<uint4*>(a.query) + row0 * 72;
    if (a.q_nope) {
#pragma unroll
      for (int k = 0; k < 2 * kHeadsPerUnit; ++k) dst[(k / 2) * 72 + 32 * (k & 1) + lane] = x[k];
    }
    dst[(lane >> 3) * 72 + 64 + u] = to_bf16x8(r);
  } else {
    uint2* dst = reinterpret_cast<uint2*>(a.query) + row0 * 72;
#pragma unroll
    for (int k = 0; k < 2 * kHeadsPerUnit; ++k) {
      float f[8];
      widen8(x[k], f);
      dst[(k / 2) * 72 + 32 * (k & 1) + lane] = to_e4m3x8(f, a.inv_q_scale);
    }
    dst[(lane >> 3) * 72 + 64 + u] = to_e4m3x8(r, a.inv_q_scale);
  }
}

// Work unit w: the cache rows of all tokens first (they are the longer chains),
// then the query, four heads a unit.
template <int kKv, bool kQFp8>
__global__ void __launch_bounds__(kThreads)
append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w < a.map.total_q) {
    append_row<kKv>(a, w, lane);
    return;
  }
  if (!a.q_pe) return;
  const int per = a.num_heads / kHeadsPerUnit;
  const long long k = w - a.map.total_q;
  const long long t = k / per;
  if (t < a.map.total_q) append_query<kQFp8>(a, t, (int)(k - t * per) * kHeadsPerUnit, lane);
}

template <int kKv>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const RowMap m, const unsigned char* __restrict__ cache, float kv_scale,
              __nv_bfloat16* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= m.total_q) return;
  const Place pl = place_of(m, t, lane);
  if (pl.pos < 0) return;
  uint4* dst = reinterpret_cast<uint4*>(out + t * kQkDim);
  if (kKv == MLA_KV_BF16) {
    const uint4* src = reinterpret_cast<const uint4*>(cache + (pl.page * m.page_size + pl.row) * (2 * kQkDim));
    const uint4 a = src[lane], b = src[32 + lane], c = src[64 + (lane & 7)];
    dst[lane] = a;
    dst[32 + lane] = b;
    if (lane < 8) dst[64 + lane] = c;
    return;
  }
  float y[16], r[8];
  if (kKv == MLA_KV_FP8_E4M3) {
    const unsigned char* src = cache + (pl.page * m.page_size + pl.row) * kQkDim;
    const uint4 a = reinterpret_cast<const uint4*>(src)[lane];
    const uint2 b = reinterpret_cast<const uint2*>(src + kVDim)[lane & 7];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w}, v[2] = {b.x, b.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ptx::e4m3x2_to_f32x2(w[e] & 0xFFFFu, y[4 * e], y[4 * e + 1]);
      ptx::e4m3x2_to_f32x2(w[e] >> 16, y[4 * e + 2], y[4 * e + 3]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ptx::e4m3x2_to_f32x2(v[e] & 0xFFFFu, r[4 * e], r[4 * e + 1]);
      ptx::e4m3x2_to_f32x2(v[e] >> 16, r[4 * e + 2], r[4 * e + 3]);
    }
  } else {
    const unsigned char* page = cache + pl.page * m.page_size * kFp4RowBytes;
    const unsigned char* codes = page + pl.row * kFp4CodeBytes;
    const unsigned char* scales = page + m.page_size * kFp4CodeBytes + pl.row * kFp4ScaleBytes;
    const uint2 a = reinterpret_cast<const uint2*>(codes)[lane];
    const uint32_t b = reinterpret_cast<const uint32_t*>(codes + 256)[lane & 7];
    const uint32_t sc = scales[lane], rsc = scales[32 + (lane & 7) / 2];
    float sv, rv;
    ptx::e4m3x2_to_f32x2(sc | (rsc << 8), sv, rv);
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      ptx::e2m1x8_to_f16x2(e == 0 ? a.x : e == 1 ? a.y : b, h);
      float* d = e == 0 ? y : e == 1 ? y + 8 : r;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        d[2 * k] = f.x * (e < 2 ? sv : rv);
        d[2 * k + 1] = f.y * (e < 2 ? sv : rv);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(y[e], kv_scale);
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = __fmul_rn(r[e], kv_scale);
  dst[2 * lane] = to_bf16x8(y);
  dst[2 * lane + 1] = to_bf16x8(y + 8);
  if (lane < 8) dst[64 + lane] = to_bf16x8(r);
}

// Angles in 64 bits: a far position times a frequency of one has no bits left
// for its fraction in fp32.  Built once, so its speed does not matter.
__global__ void __launch_bounds__(kThreads)
rope_table_kernel(mla_rope_params p, double low, double high, float* __restrict__ table) {
  const long long n = (long long)p.max_position * 32;
  for (long long k = (long long)blockIdx.x * kThreads + threadIdx.x; k < n;
       k += (long long)gridDim.x * kThreads) {
    const int i = (int)(k & 31);
    const long long pos = k >> 5;
    double f = exp2(-(double)i / 32.0 * log2(p.base));
    if (p.scaling == MLA_ROPE_LINEAR) f /= p.factor;
    if (p.scaling == MLA_ROPE_YARN) {
      // the part of the frequency that is interpolated: 0 up to dim pair low,
      // 1 from high on, linear between
      const double ramp = fmin(fmax(((double)i - low) / (high - low), 0.0), 1.0);
      f = f / p.factor * ramp + f * (1.0 - ramp);
    }
    double s, c;
    sincos((double)pos * f, &s, &c);
    table[pos * 64 + i] = (float)(c * p.amplitude);
    table[pos * 64 + 32 + i] = (float)(s * p.amplitude);
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The checks append and gather share; on success *m is filled.
int row_map(const mla_cache_params* p, const void* cache, const int32_t* block_tables,
            const int32_t* seq_lens, const int32_t* qo_indptr, int64_t total_q, int32_t* status,
            RowMap* m) {
  if (!p) return MLA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->max_pages_per_req < 1 || p->num_pages < 1 || total_q < 0 ||
      total_q > (1LL << 31))
    return MLA_ERR_INVALID_ARG;
  if (p->packed != 0 && p->packed != 1) return MLA_ERR_INVALID_ARG;
  if (p->kv_dtype != MLA_KV_BF16 && p->kv_dtype != MLA_KV_FP8_E4M3 && p->kv_dtype != MLA_KV_FP4_E2M1)
    return MLA_ERR_INVALID_ARG;
  if (p->page_size != 32 && p->page_size != 64) return MLA_ERR_UNSUPPORTED;
  if (p->num_pages > (1LL << 31) / p->page_size) return MLA_ERR_UNSUPPORTED;
  if (p->packed ? !qo_indptr : (qo_indptr != nullptr || p->q_len < 1 ||
                                total_q != (int64_t)p->batch * p->q_len))
    return MLA_ERR_INVALID_ARG;
  if (p->batch == 0 || total_q == 0) return MLA_OK;
  if (!cache || !block_tables || !seq_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
      (qo_indptr && !aligned(qo_indptr, 4)) || (status && !aligned(status, 4)))
    return MLA_ERR_ALIGNMENT;
  *m = RowMap{p->batch, p->q_len, p->page_size, p->max_pages_per_req, p->num_pages, total_q,
              block_tables, seq_lens, qo_indptr, status};
  return MLA_OK;
}

// Quantising multiplies by the reciprocal, which a subnormal scale would not have.
bool scale_ok(float v) { return v >= 1.17549435e-38f && v <= 3.0e38f; }

template <int kKv>
void launch_append(const AppendArgs& a, bool q_fp8, unsigned blocks, cudaStream_t s) {
  if (q_fp8)
    append_kernel<kKv, true><<<blocks, kThreads, 0, s>>>(a);
  else
    append_kernel<kKv, false><<<blocks, kThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_cache_append(const mla_cache_params* params, const void* latent, int64_t latent_stride,
                     const void* k_pe, int64_t k_pe_stride, const void* norm_weight, float eps,
                     const float* rope_table, int32_t max_position, int32_t rope_style,
                     const int32_t* positions, const int32_t* block_tables,
                     const int32_t* seq_lens, const int32_t* qo_indptr, int64_t total_q,
                     float kv_scale, void* kv_cache, const void* q_nope,
                     int64_t q_nope_token_stride, int64_t q_nope_head_stride, const void* q_pe,
                     int64_t q_pe_token_stride, int64_t q_pe_head_stride, float q_scale,
                     void* query, int32_t* status, void* stream) {
  using namespace mla;
  AppendArgs a = {};
  const int rc = row_map(params, kv_cache, block_tables, seq_lens, qo_indptr, total_q, status, &a.map);
  if (rc != MLA_OK) return rc;
  const mla_cache_params& p = *params;
  if (rope_style != MLA_ROPE_INTERLEAVED && rope_style != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
  if (max_position < 1 || !scale_ok(kv_scale) || !scale_ok(q_scale))
    return MLA_ERR_INVALID_ARG;
  // below 1e-30 squares that underflow would count beside eps
  if (norm_weight && !(eps >= 1e-30f && eps <= 3.0e38f)) return MLA_ERR_INVALID_ARG;
  if (p.kv_dtype == MLA_KV_BF16 && kv_scale != 1.f) return MLA_ERR_INVALID_ARG;
  const bool with_q = q_pe != nullptr;
  if (with_q != (query != nullptr) || (q_nope && !with_q)) return MLA_ERR_INVALID_ARG;
  if (with_q) {
    if (p.q_dtype != MLA_Q_BF16 && p.q_dtype != MLA_Q_FP8_E4M3) return MLA_ERR_INVALID_ARG;
    if (p.num_heads != 16 && p.num_heads != 32 && p.num_heads != 64 && p.num_heads != 128)
      return MLA_ERR_UNSUPPORTED;
    // an e4m3 query is quantised whole; a bf16 one may keep its latent part
    if (p.q_dtype == MLA_Q_FP8_E4M3 ? !q_nope : q_scale != 1.f) return MLA_ERR_INVALID_ARG;
  }
  if (p.batch == 0 || total_q == 0) return MLA_OK;
  if (!latent || !k_pe || !rope_table) return MLA_ERR_INVALID_ARG;
  // rows are read in 16-byte units
  auto rows_ok = [](const void* q, int64_t s) { return aligned(q, 16) && s >= 0 && s % 8 == 0; };
  if (!rows_ok(latent, latent_stride) || !rows_ok(k_pe, k_pe_stride) || !aligned(rope_table, 16) ||
      (norm_weight && !aligned(norm_weight, 16)) || (positions && !aligned(positions, 4)) ||
      (with_q && (!rows_ok(q_pe, q_pe_token_stride) || !rows_ok(q_pe, q_pe_head_stride) ||
                  !aligned(query, 16))) ||
      (q_nope && (!rows_ok(q_nope, q_nope_token_stride) || !rows_ok(q_nope, q_nope_head_stride))))
    return MLA_ERR_ALIGNMENT;
  a.latent = static_cast<const __nv_bfloat16*>(latent);
  a.k_pe = static_cast<const __nv_bfloat16*>(k_pe);
  a.norm_weight = static_cast<const __nv_bfloat16*>(norm_weight);
  a.rope_table = rope_table;
  a.positions = positions;
  a.cache = static_cast<unsigned char*>(kv_cache);
  a.q_nope = static_cast<const __nv_bfloat16*>(q_nope);
  a.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  a.query = static_cast<unsigned char*>(query);
  a.latent_stride = latent_stride;
  a.k_pe_stride = k_pe_stride;
  a.q_nope_token = q_nope_token_stride;
  a.q_nope_head = q_nope_head_stride;
  a.q_pe_token = q_pe_token_stride;
  a.q_pe_head = q_pe_head_stride;
  a.num_heads = p.num_heads;
  a.max_position = max_position;
  a.half_style = rope_style == MLA_ROPE_HALF;
  a.eps = eps;
  a.inv_kv_scale = (float)(1.0 / (double)kv_scale);
  a.inv_q_scale = (float)(1.0 / (double)q_scale);
  const long long units = total_q + (with_q ? total_q * (p.num_heads / kHeadsPerUnit) : 0);
  const long long blocks = (units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool q_fp8 = with_q && p.q_dtype == MLA_Q_FP8_E4M3;
  if (p.kv_dtype == MLA_KV_BF16)
    launch_append<MLA_KV_BF16>(a, q_fp8, (unsigned)blocks, s);
  else if (p.kv_dtype == MLA_KV_FP8_E4M3)
    launch_append<MLA_KV_FP8_E4M3>(a, q_fp8, (unsigned)blocks, s);
  else
    launch_append<MLA_KV_FP4_E2M1>(a, q_fp8, (unsigned)blocks, s);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_gather(const mla_cache_params* params, const void* kv_cache,
                     const int32_t* block_tables, const int32_t* seq_lens,
                     const int32_t* qo_indptr, int64_t total_q, float kv_scale, void* out,
                     int32_t* status, void* stream) {
  using namespace mla;
  RowMap m = {};
  const int rc = row_map(params, kv_cache, block_tables, seq_lens, qo_indptr, total_q, status, &m);
  if (rc != MLA_OK) return rc;
  const mla_cache_params& p = *params;
  if (!scale_ok(kv_scale) || (p.kv_dtype == MLA_KV_BF16 && kv_scale != 1.f)) return MLA_ERR_INVALID_ARG;
  if (p.batch == 0 || total_q == 0) return MLA_OK;
  if (!out) return MLA_ERR_INVALID_ARG;
  if (!aligned(out, 16)) return MLA_ERR_ALIGNMENT;
  const unsigned blocks = (unsigned)((total_q + kWarps - 1) / kWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned char* c = static_cast<const unsigned char*>(kv_cache);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  if (p.kv_dtype == MLA_KV_BF16)
    gather_kernel<MLA_KV_BF16><<<blocks, kThreads, 0, s>>>(m, c, kv_scale, o);
  else if (p.kv_dtype == MLA_KV_FP8_E4M3)
    gather_kernel<MLA_KV_FP8_E4M3><<<blocks, kThreads, 0, s>>>(m, c, kv_scale, o);
  else
    gather_kernel<MLA_KV_FP4_E2M1><<<blocks, kThreads, 0, s>>>(m, c, kv_scale, o);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_rope_table(const mla_rope_params* params, float* table, void* stream) {
  using namespace mla;
  if (!params || !table) return MLA_ERR_INVALID_ARG;
  const mla_rope_params& p = *params;
  if (p.max_position < 1 || !(p.base > 1.0 && p.base <= 1e300) ||
      !(p.amplitude > 0.0 && p.amplitude <= 1e30))
    return MLA_ERR_INVALID_ARG;
  if (p.scaling != MLA_ROPE_NONE && p.scaling != MLA_ROPE_LINEAR && p.scaling != MLA_ROPE_YARN)
    return MLA_ERR_INVALID_ARG;
  if (p.scaling != MLA_ROPE_NONE && !(p.factor > 0.0 && p.factor <= 1e30)) return MLA_ERR_INVALID_ARG;
  if (!aligned(table, 16)) return MLA_ERR_ALIGNMENT;
  double low = 0, high = 1;
  if (p.scaling == MLA_ROPE_YARN) {
    if (!(p.original_max_position >= 1.0 && p.original_max_position <= 1e15) ||
        !(p.beta_slow > 0.0 && p.beta_fast >= p.beta_slow && p.beta_fast <= 1e15))
      return MLA_ERR_INVALID_ARG;
    // the dim pair whose wavelength fits `turns` times into the original context
    auto pair_of = [&](double turns) {
      return 32.0 * log(p.original_max_position / (turns * 2.0 * 3.14159265358979323846)) / log(p.base);
    };
    low = std::max(0.0, floor(pair_of(p.beta_fast)));
    high = std::min(63.0, ceil(pair_of(p.beta_slow)));
    if (!(high > low)) high = low + 0.001;
  }
  const long long n = (long long)p.max_position * 32;
  const unsigned blocks = (unsigned)std::min<long long>((n + kThreads - 1) / kThreads, 1 << 16);
  rope_table_kernel<<<blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, low, high, table);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
