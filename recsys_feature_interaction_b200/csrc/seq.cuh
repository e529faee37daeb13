// seq.cuh -- attention over behaviour sequences: jagged cross attention and its gradients, the
// paged cache (write, read) and attention over it (WHALE pages, section 2.1 item 3 and section 2.2).
// First form: one warp per row, plain fp32 arithmetic on the CUDA cores.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "seq_index.h"

namespace wk {

struct SeqArgs {
  int32_t batch, q_heads, kv_heads, max_q, max_kv;
  int64_t total_q, total_kv;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  const int32_t *q_off, *kv_off, *kv_lens;
  // cache
  const int32_t* table;
  int32_t table_width, num_pages, page_shift, causal;
  const uint8_t *k_exp, *v_exp;
  unsigned* status;
};

// 2^(e - 127) of a cache row's exponent byte; NaN for 255.
__device__ __forceinline__ float seq_pow(uint8_t e) {
  return __uint_as_float(e == 255 ? 0x7FC00000u : (e == 0 ? 0x00400000u : static_cast<uint32_t>(e) << 23));
}

__device__ __forceinline__ float seq_e4m3(uint8_t v) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
  return __half2float(__half(h));
}

// ---------------------------------------------------------------- cache write

// One warp per (new token, kv head, K or V).
template <int D, typename T, bool Q8>
__global__ void cache_write_kernel(const T* __restrict__ K, const T* __restrict__ V, void* cK, void* cV, uint8_t* eK,
                                   uint8_t* eV, SeqArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t per_seq = static_cast<int64_t>(a.max_q) * a.kv_heads * 2;
  const int64_t b = unit / per_seq;
  if (b >= a.batch) return;
  const int r = static_cast<int>(unit % per_seq);
  const int i = r / (a.kv_heads * 2), h = (r >> 1) % a.kv_heads, which = r & 1;
  const SeqSpan q = seq_span(a.q_off, nullptr, b, a.total_q, a.max_q);
  const SeqSpan kv = seq_cached(a.kv_lens, b, static_cast<int64_t>(a.table_width) << a.page_shift, INT32_MAX);
  if (q.bad || kv.bad || kv.len < q.len) {
    if (lane == 0) flag_error(a.status, kFlagBadShape);
    return;
  }
  if (i >= q.len) return;
  const int64_t pos = static_cast<int64_t>(kv.len) - q.len + i;
  const int page = seq_page(a.table + b * a.table_width, pos, a.page_shift, a.num_pages);
  if (page < 0) {
    if (lane == 0) flag_error(a.status, kFlagBadShape);
    return;
  }
  const int64_t row = ((static_cast<int64_t>(page) * a.kv_heads + h) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  const T* src = (which ? V + (q.begin + i) * a.v_stride : K + (q.begin + i) * a.k_stride) + h * D;
  float x[D / 32], amax = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) x[c] = Half16<T>::to(src[c * 32 + lane]);
  if constexpr (Q8) {
    bool odd = false;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      amax = fmaxf(amax, fabsf(x[c]));
      odd |= !(fabsf(x[c]) < INFINITY);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    odd = __any_sync(~0u, odd);
    int e = 0;  // biased
    if (!odd && amax > 0.f) {
      int p;
      const float f = frexpf(amax, &p);
      e = min(max(p - 9 + (f > 0.875f ? 1 : 0) + 127, 0), 254);
    }
    uint8_t* dst = static_cast<uint8_t*>(which ? cV : cK) + row * D;
    const double inv = odd ? 0. : ldexp(1., 127 - e);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      dst[c * 32 + lane] = __nv_cvt_float_to_fp8(static_cast<float>(x[c] * inv), __NV_SATFINITE, __NV_E4M3);
    if (lane == 0) (which ? eV : eK)[row] = odd ? 255 : e;
  } else {
    T* dst = static_cast<T*>(which ? cV : cK) + row * D;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dst[c * 32 + lane] = src[c * 32 + lane];
  }
}

// ---------------------------------------------------------------- key rows

// Element access to key (or value) row j of sequence b, head h.
template <int D, typename T, int SRC>  // SRC 0: jagged, 1: 16-bit cache, 2: 8-bit cache
struct SeqRows {
  const void* base;
  const uint8_t* ex;
  int64_t stride, begin;
  const int32_t* row;
  int h;
  __device__ __forceinline__ bool load(const SeqArgs& a, int j, int lane, float (&x)[D / 32]) const {
    if constexpr (SRC == 0) {
      const T* p = static_cast<const T*>(base) + (begin + j) * stride + h * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) x[c] = Half16<T>::to(p[c * 32 + lane]);
    } else {
      const int page = seq_page(row, j, a.page_shift, a.num_pages);
      if (page < 0) {
        flag_error(a.status, kFlagBadShape);
        return false;
      }
      const int64_t r = ((static_cast<int64_t>(page) * a.kv_heads + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      if constexpr (SRC == 1) {
        const T* p = static_cast<const T*>(base) + r * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) x[c] = Half16<T>::to(p[c * 32 + lane]);
      } else {
        const uint8_t* p = static_cast<const uint8_t*>(base) + r * D;
        const float s = seq_pow(ex[r]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) x[c] = seq_e4m3(p[c * 32 + lane]) * s;
      }
    }
    return true;
  }
};

template <int D, typename T, int SRC>
__device__ __forceinline__ SeqRows<D, T, SRC> seq_rows(const SeqArgs& a, const void* base, const uint8_t* ex,
                                                       int64_t stride, int64_t b, int64_t begin, int h) {
  return {base, ex, stride, begin, SRC ? a.table + b * a.table_width : nullptr, h};
}

template <int SRC>
__device__ __forceinline__ SeqSpan seq_keys(const SeqArgs& a, int64_t b) {
  if constexpr (SRC == 0) return seq_span(a.kv_off, a.kv_lens, b, a.total_kv, a.max_kv);
  return seq_cached(a.kv_lens, b, static_cast<int64_t>(a.table_width) << a.page_shift, a.max_kv);
}

// ---------------------------------------------------------------- cache read

template <int D, typename T, int SRC>
__global__ void cache_read_kernel(const void* cK, const void* cV, T* __restrict__ K, T* __restrict__ V, SeqArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t per_seq = static_cast<int64_t>(a.max_kv) * a.kv_heads * 2;
  const int64_t b = unit / per_seq;
  if (b >= a.batch) return;
  const int64_t r = unit % per_seq;
  const int j = static_cast<int>(r / (a.kv_heads * 2)), h = static_cast<int>((r >> 1) % a.kv_heads), which = r & 1;
  const SeqSpan kv = seq_keys<SRC>(a, b);
  const SeqSpan out = seq_span(a.kv_off, nullptr, b, a.total_kv, INT32_MAX);
  if (kv.bad || out.bad || out.room < kv.len)
    if (lane == 0) flag_error(a.status, kFlagBadShape);
  if (j >= kv.len || j >= out.room) return;
  float x[D / 32];
  if (!seq_rows<D, T, SRC>(a, which ? cV : cK, which ? a.v_exp : a.k_exp, 0, b, 0, h).load(a, j, lane, x)) return;
  T* dst = (which ? V : K) + ((out.begin + j) * a.kv_heads + h) * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) dst[c * 32 + lane] = Half16<T>::from(x[c]);
}

// ---------------------------------------------------------------- forward

template <int D>
__device__ __forceinline__ float seq_dot(const float (&x)[D / 32], const float (&y)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s = fmaf(x[c], y[c], s);
  return warp_sum(s);
}

// One warp per (query row, query head).
template <int D, typename T, int SRC>
__global__ void xattn_forward_kernel(const T* __restrict__ Q, const void* K, const void* V, T* __restrict__ O,
                                     float* __restrict__ lse, SeqArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t per_seq = static_cast<int64_t>(a.max_q) * a.q_heads;
  const int64_t b = unit / per_seq;
  if (b >= a.batch) return;
  const int i = static_cast<int>(unit % per_seq / a.q_heads), h = static_cast<int>(unit % a.q_heads);
  const SeqSpan q = seq_span(a.q_off, nullptr, b, a.total_q, a.max_q);
  const SeqSpan kv = seq_keys<SRC>(a, b);
  if ((q.bad || kv.bad) && lane == 0) flag_error(a.status, kFlagBadShape);
  if (i >= q.len) return;
  const int hk = h / (a.q_heads / a.kv_heads);
  const auto kr = seq_rows<D, T, SRC>(a, K, a.k_exp, a.k_stride, b, kv.begin, hk);
  const auto vr = seq_rows<D, T, SRC>(a, V, a.v_exp, a.v_stride, b, kv.begin, hk);
  const int seen = seq_seen(kv.len, q.len, i, a.causal);
  float x[D / 32], o[D / 32], y[D / 32], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    x[c] = Half16<T>::to(Q[(q.begin + i) * a.q_stride + h * D + c * 32 + lane]);
    o[c] = 0.f;
  }
  for (int j = 0; j < seen; ++j) {
    if (!kr.load(a, j, lane, y)) continue;
    const float s = seq_dot<D>(x, y) * a.scale;
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), p = expf(s - mn);
    if (!vr.load(a, j, lane, y)) continue;
    l = l * f + p;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = o[c] * f + p * y[c];
    m = mn;
  }
  const float inv = seen > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    O[((q.begin + i) * a.q_heads + h) * D + c * 32 + lane] = Half16<T>::from(o[c] * inv);
  if (lse && lane == 0) lse[(q.begin + i) * a.q_heads + h] = m + logf(l);
}

// ---------------------------------------------------------------- backward

// delta[i, h] = sum_c O dO, per (row, head): the softmax backward's row constant.
template <int D, typename T>
__global__ void xattn_delta_kernel(const T* __restrict__ O, const T* __restrict__ dO, float* __restrict__ delta,
                                   int64_t rows) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (r >= rows) return;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s += Half16<T>::to(O[r * D + c * 32 + lane]) * Half16<T>::to(dO[r * D + c * 32 + lane]);
  s = warp_sum(s);
  if (lane == 0) delta[r] = s;
}

// dQ: one warp per (query row, query head).
template <int D, typename T>
__global__ void xattn_dq_kernel(const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
                                const T* __restrict__ dO, const float* __restrict__ lse,
                                const float* __restrict__ delta, T* __restrict__ dQ, SeqArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t per_seq = static_cast<int64_t>(a.max_q) * a.q_heads;
  const int64_t b = unit / per_seq;
  if (b >= a.batch) return;
  const int i = static_cast<int>(unit % per_seq / a.q_heads), h = static_cast<int>(unit % a.q_heads);
  const SeqSpan q = seq_span(a.q_off, nullptr, b, a.total_q, a.max_q);
  const SeqSpan kv = seq_keys<0>(a, b);
  if ((q.bad || kv.bad) && lane == 0) flag_error(a.status, kFlagBadShape);
  if (i >= q.len) return;
  const int hk = h / (a.q_heads / a.kv_heads);
  const auto kr = seq_rows<D, T, 0>(a, K, nullptr, a.k_stride, b, kv.begin, hk);
  const auto vr = seq_rows<D, T, 0>(a, V, nullptr, a.v_stride, b, kv.begin, hk);
  const int64_t r = (q.begin + i) * a.q_heads + h;
  float x[D / 32], g[D / 32], acc[D / 32], y[D / 32], z[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    x[c] = Half16<T>::to(Q[(q.begin + i) * a.q_stride + h * D + c * 32 + lane]);
    g[c] = Half16<T>::to(dO[r * D + c * 32 + lane]);
    acc[c] = 0.f;
  }
  const float ls = lse[r], dl = delta[r];
  for (int j = 0; j < kv.len; ++j) {
    kr.load(a, j, lane, y);
    vr.load(a, j, lane, z);
    const float p = expf(seq_dot<D>(x, y) * a.scale - ls);
    const float ds = p * (seq_dot<D>(g, z) - dl) * a.scale;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(ds, y[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) dQ[r * D + c * 32 + lane] = Half16<T>::from(acc[c]);
}

// dK, dV: one warp per (key row, key head); also the zeros of a sequence's padding rows.
template <int D, typename T>
__global__ void xattn_dkv_kernel(const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
                                 const T* __restrict__ dO, const float* __restrict__ lse,
                                 const float* __restrict__ delta, T* __restrict__ dK, T* __restrict__ dV, SeqArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t r = unit / a.kv_heads;
  const int h = static_cast<int>(unit % a.kv_heads);
  if (r >= a.total_kv) return;
  int64_t lo = 0, hi = a.batch;  // the last sequence that begins at or before r
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.kv_off[mid] <= r) lo = mid;
    else hi = mid;
  }
  const SeqSpan kv = seq_span(a.kv_off, a.kv_lens, lo, a.total_kv, a.max_kv);
  const SeqSpan q = seq_span(a.q_off, nullptr, lo, a.total_q, a.max_q);
  if ((q.bad || kv.bad) && lane == 0) flag_error(a.status, kFlagBadShape);
  if (r < kv.begin || r >= kv.begin + kv.room) return;
  float y[D / 32], z[D / 32], ak[D / 32], av[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) ak[c] = av[c] = 0.f;
  if (r < kv.begin + kv.len) {
    seq_rows<D, T, 0>(a, K, nullptr, a.k_stride, lo, 0, h).load(a, static_cast<int>(r), lane, y);
    seq_rows<D, T, 0>(a, V, nullptr, a.v_stride, lo, 0, h).load(a, static_cast<int>(r), lane, z);
    const int group = a.q_heads / a.kv_heads;
    for (int i = 0; i < q.len; ++i)
      for (int hq = h * group; hq < (h + 1) * group; ++hq) {
        const int64_t qr = (q.begin + i) * a.q_heads + hq;
        float x[D / 32], g[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          x[c] = Half16<T>::to(Q[(q.begin + i) * a.q_stride + hq * D + c * 32 + lane]);
          g[c] = Half16<T>::to(dO[qr * D + c * 32 + lane]);
        }
        const float p = expf(seq_dot<D>(x, y) * a.scale - lse[qr]);
        const float ds = p * (seq_dot<D>(g, z) - delta[qr]) * a.scale;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          av[c] = fmaf(p, g[c], av[c]);
          ak[c] = fmaf(ds, x[c], ak[c]);
        }
      }
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    dK[(r * a.kv_heads + h) * D + c * 32 + lane] = Half16<T>::from(ak[c]);
    dV[(r * a.kv_heads + h) * D + c * 32 + lane] = Half16<T>::from(av[c]);
  }
}

}  // namespace wk
