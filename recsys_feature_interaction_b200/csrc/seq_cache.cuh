// seq_cache.cuh -- the paged cache's two copies: new tokens into it (quantised with 8-bit caches),
// cached sequences out of it.
//
// Both are bound by the bytes they move. Four lanes share a row (one token, one key head) and take
// it in chunks of 8 elements, 16 bytes on the 16-bit side and 8 on the 8-bit one: every access of a
// warp covers whole 32-byte sectors of 8 rows, all of a row's loads are in flight at once, and the
// row's largest magnitude is two shuffles away. A warp's 8 rows are 8 consecutive tokens of one
// head, which lie next to each other in a page. A block takes 64 tokens of one (sequence, key head,
// K or V); blocks past a short sequence's end leave at once.
#pragma once

#include <cuda_fp8.h>

#include "seq_args.cuh"

namespace wk {

constexpr int SEQ_COPY_THREADS = 256;
constexpr int SEQ_COPY_ROWS = SEQ_COPY_THREADS / 4;  // tokens per block

// blockIdx.x = ((b * chunks + chunk) * kv_heads + h) * 2 + (K or V)
struct SeqCopyPlace {
  int64_t b;
  int32_t chunk, h, which;
  __device__ __forceinline__ SeqCopyPlace(const SeqArgs& a, int32_t chunks) {
    uint32_t x = blockIdx.x;
    which = static_cast<int32_t>(x & 1u);
    x >>= 1;
    h = static_cast<int32_t>(x % static_cast<uint32_t>(a.kv_heads));
    x /= static_cast<uint32_t>(a.kv_heads);
    chunk = static_cast<int32_t>(x % static_cast<uint32_t>(chunks));
    b = x / static_cast<uint32_t>(chunks);
  }
};

// Row of the cache that holds position pos of sequence b, head h; -1 (and the status word set) if
// the table names no page for it.
__device__ __forceinline__ int64_t seq_cache_row(const SeqArgs& a, int64_t b, int h, int64_t pos) {
  const int page = seq_page(a.table + b * a.table_width, pos, a.page_shift, a.num_pages);
  if (page < 0) {
    flag_error(a.status, kFlagBadShape);
    return -1;
  }
  return ((static_cast<int64_t>(page) * a.kv_heads + h) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

template <int D, typename T, bool Q8>
__global__ void __launch_bounds__(SEQ_COPY_THREADS)
    cache_write_kernel(const T* __restrict__ K, const T* __restrict__ V, void* __restrict__ cK, void* __restrict__ cV,
                       uint8_t* __restrict__ eK, uint8_t* __restrict__ eV, SeqArgs a, int32_t chunks) {
  constexpr int CH = D / 32;  // chunks of 8 elements per lane
  const SeqCopyPlace p(a, chunks);
  seq_wait_before();
  const SeqSpan q = seq_queries(a, p.b);
  const SeqSpan kv = seq_cached(a.kv_lens, p.b, static_cast<int64_t>(a.table_width) << a.page_shift, INT32_MAX);
  if (q.bad || kv.bad || kv.len < q.len) {
    if (threadIdx.x == 0) flag_error(a.status, kFlagBadShape);
    return;
  }
  const int i = p.chunk * SEQ_COPY_ROWS + (threadIdx.x >> 2), c = threadIdx.x & 3;
  const bool on = i < q.len;
  if (!__any_sync(0xffffffffu, on)) return;
  uint4 x[CH];
  const T* src = (p.which ? V + (q.begin + i) * a.v_stride : K + (q.begin + i) * a.k_stride) + p.h * D;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    x[j] = make_uint4(0u, 0u, 0u, 0u);
    if (on) x[j] = __ldg(reinterpret_cast<const uint4*>(src) + j * 4 + c);
  }
  const int64_t row = on ? seq_cache_row(a, p.b, p.h, static_cast<int64_t>(kv.len) - q.len + i) : -1;
  if constexpr (Q8) {
    // the largest magnitude as 16-bit integers, two at a time: without their signs floats order as
    // integers do, infinities and NaN behind all others
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) top = __vmaxu2(top, reinterpret_cast<const uint32_t*>(&x[j])[k] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = max(top & 0xFFFFu, top >> 16);
    const bool odd = top >= (Half16<T>::kBF16 ? 0x7F80u : 0x7C00u);
    const float amax = Half16<T>::lo(top);
    // amax = 1.f * 2^(E - 127): the least e with amax <= 448 * 2^(e - 127) = 1.75 * 2^(e + 8 - 127)
    const uint32_t bits = __float_as_uint(amax);
    const int e = odd ? 255 : max(0, static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
    const float f = odd ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e)
    if (row >= 0) {
      uint8_t* dst = static_cast<uint8_t*>(p.which ? cV : cK) + row * D;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t u = reinterpret_cast<const uint32_t*>(&x[j])[2 * k],
                         v = reinterpret_cast<const uint32_t*>(&x[j])[2 * k + 1];
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(Half16<T>::lo(u) * f, Half16<T>::hi(u) * f),
                                                       __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(Half16<T>::lo(v) * f, Half16<T>::hi(v) * f),
                                                       __NV_SATFINITE, __NV_E4M3);
          w[k] = lo | (hi << 16);
        }
        *(reinterpret_cast<uint2*>(dst) + j * 4 + c) = make_uint2(w[0], w[1]);
      }
      if (c == 0) (p.which ? eV : eK)[row] = static_cast<uint8_t>(e);
    }
  } else if (row >= 0) {
    T* dst = static_cast<T*>(p.which ? cV : cK) + row * D;
#pragma unroll
    for (int j = 0; j < CH; ++j) *(reinterpret_cast<uint4*>(dst) + j * 4 + c) = x[j];
  }
}

// Two e4m3 values (a 16-bit word) times f, as a pair of T.
template <typename T>
__device__ __forceinline__ uint32_t seq_e4m3_pair(uint32_t w, float f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const float2 v = __half22float2(__half2(h));
  return Half16<T>::pack2(v.x * f, v.y * f);
}

template <int D, typename T, int SRC>
__global__ void __launch_bounds__(SEQ_COPY_THREADS)
    cache_read_kernel(const void* __restrict__ cK, const void* __restrict__ cV, T* __restrict__ K, T* __restrict__ V,
                      SeqArgs a, int32_t chunks) {
  constexpr int CH = D / 32;
  const SeqCopyPlace p(a, chunks);
  seq_wait_before();
  const SeqSpan kv = seq_keys<SRC>(a, p.b);
  const SeqSpan out = seq_span(a.kv_off, nullptr, p.b, a.total_kv, INT32_MAX);
  if ((kv.bad || out.bad || out.room < kv.len) && threadIdx.x == 0) flag_error(a.status, kFlagBadShape);
  const int i = p.chunk * SEQ_COPY_ROWS + (threadIdx.x >> 2), c = threadIdx.x & 3;
  if (i >= kv.len || i >= out.room) return;
  const int64_t row = seq_cache_row(a, p.b, p.h, i);
  if (row < 0) return;
  T* dst = (p.which ? V : K) + ((out.begin + i) * a.kv_heads + p.h) * D;
  if constexpr (SRC == SEQ_PAGED8) {
    const uint8_t* src = static_cast<const uint8_t*>(p.which ? cV : cK) + row * D;
    uint2 x[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) x[j] = __ldg(reinterpret_cast<const uint2*>(src) + j * 4 + c);
    const float f = seq_pow(__ldg((p.which ? a.v_exp : a.k_exp) + row));
#pragma unroll
    for (int j = 0; j < CH; ++j)
      *(reinterpret_cast<uint4*>(dst) + j * 4 + c) =
          make_uint4(seq_e4m3_pair<T>(x[j].x & 0xFFFFu, f), seq_e4m3_pair<T>(x[j].x >> 16, f),
                     seq_e4m3_pair<T>(x[j].y & 0xFFFFu, f), seq_e4m3_pair<T>(x[j].y >> 16, f));
  } else {
    const T* src = static_cast<const T*>(p.which ? cV : cK) + row * D;
    uint4 x[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) x[j] = __ldg(reinterpret_cast<const uint4*>(src) + j * 4 + c);
#pragma unroll
    for (int j = 0; j < CH; ++j) *(reinterpret_cast<uint4*>(dst) + j * 4 + c) = x[j];
  }
}

}  // namespace wk
