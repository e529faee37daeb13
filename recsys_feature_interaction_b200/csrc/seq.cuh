// seq.cuh -- attention over behaviour sequences: jagged cross attention and its gradients, the
// paged cache (write, read) and attention over it (WHALE pages, section 2.1 item 3 and section 2.2).
// First form: one warp per row, plain fp32 arithmetic on the CUDA cores.
#pragma once

#include <cuda_fp8.h>

#include "seq_args.cuh"

namespace wk {

__device__ __forceinline__ float seq_e4m3(uint8_t v) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
  return __half2float(__half(h));
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

template <int D>
__device__ __forceinline__ float seq_dot(const float (&x)[D / 32], const float (&y)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s = fmaf(x[c], y[c], s);
  return warp_sum(s);
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
