// seq_rows.cuh -- attention of at most 16 packed query rows per (sequence, key head) over jagged or
// cached keys: one new token (or a few) per sequence.
//
// With so few rows every key byte is used for 16 rows at most, far below the ridge: the bytes of K
// and V bound it. So no shared memory stands between HBM and the tensor cores: each warp takes its
// own keys and loads them in the register layout of mma.sync, 16 bytes a thread, and the next step's
// K is in flight while this step's V is used, and the other way round. The contraction index may be
// numbered at will, so a thread's 16 consecutive bytes of a K row are what it holds of several k
// steps, and its bytes of a V row are its rows of several output tiles. Keys are the M side:
//   S^T [16 keys, 8 rows] = K Q^T,   O^T [16 d, 8 rows] += V^T P^T
// so that a step costs D / 4 accumulators per 8 rows (the M = rows form would hold 16 rows' worth
// for 4 real ones), and P^T goes from accumulator to operand layout by two movmatrix. Softmax
// statistics are kept per warp and joined over the block's warps, and over blocks, at the end.
//
// 8-bit rows: e4m3 bits shifted into a 16-bit float's fields are the value times a fixed power of
// two (2^-8 in fp16, 2^-120 in bf16), so a conversion is a shift, a mask and a multiplication by a
// power of two, exact. K's exponent joins the fp32 score; V's joins the conversion, relative to a
// reference that is raised (and O rescaled) when a row is more than 2^7 above it, so that fp16
// holds every row down to 2^-15 of the largest exactly.
#pragma once

#include "seq_args.cuh"

namespace wk {

constexpr int SEQ_ROWS_WARPS = 4;
constexpr int SEQ_ROWS_THREADS = 32 * SEQ_ROWS_WARPS;
// Blocks per SM, and so the registers of a thread: with 16 rows of a wide head the accumulators and
// the rows in flight need more than the 168 that three blocks leave (measured: 250 to 620 bytes
// spilled), elsewhere three keep more loads in flight.
constexpr int seq_rows_occupancy(int d, int nq) { return nq == 2 && d >= 128 ? 2 : 3; }

// 16-byte, 8-byte or 4-byte load of data that is read once.
template <int BYTES>
__device__ __forceinline__ void seq_ldg(const void* p, uint32_t* r) {
  if constexpr (BYTES == 16) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r[0]) : "l"(p));
  }
}

// x * y on a pair of 16-bit values.
template <typename T>
__device__ __forceinline__ uint32_t seq_mul2(uint32_t x, uint32_t y) {
  uint32_t r;
  if constexpr (Half16<T>::kBF16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Two e4m3 values in bytes 1 and 3 as two values of T, times 2^-8 (fp16) or 2^-120 (bf16).
template <typename T>
__device__ __forceinline__ uint32_t seq_raw2(uint32_t w) {
  return Half16<T>::kBF16 ? ((w & 0x80008000u) | ((w >> 4) & 0x07F007F0u))
                          : ((w & 0x80008000u) | ((w >> 1) & 0x3F803F80u));
}
template <typename T>
constexpr int kRawPow = Half16<T>::kBF16 ? 120 : 8;

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t seq_movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D_, int SRC_>
struct SrCfg {
  static constexpr int D = D_, SRC = SRC_;
  static constexpr bool Q8 = SRC == SEQ_PAGED8;
  static constexpr int ES = Q8 ? 1 : 2;                            // bytes per element held
  static constexpr int KS = Q8 && D <= 128 ? 32 : 16;              // keys per step of a warp
  static constexpr int KB = 128;                                   // keys per block step: the unit of sharing out
  static constexpr int SUB = KB / (SEQ_ROWS_WARPS * KS);           // steps of a warp in a block step
  static constexpr int KCB = Q8 ? (D % 64 == 0 ? 16 : 8) : 16;     // bytes per load of a K row
  static constexpr int KCH = D * ES / (4 * KCB);                   // loads of a K row (4 lanes a row)
  static constexpr int VL = D * ES / 8;                            // bytes of a V row per lane (8 lanes a row)
  static constexpr int VCB = VL % 16 == 0 ? 16 : (VL % 8 == 0 ? 8 : 4);
  static constexpr int VCH = VL / VCB;
  static constexpr int VCE = VCB / ES;                             // elements per V load
  static constexpr int KSTEPS = D / 16;
  static constexpr int DT = D / 16;                                // tiles of O^T
  static_assert(KCB * 4 * KCH == D * ES && VCB * 8 * VCH == D * ES, "row split");
  // d of the first of a thread's 4 values of k step s (quarter c of the lanes)
  static __device__ __forceinline__ int kd(int s, int c) {
    if constexpr (Q8 && KCB == 16) return (s / 4) * 64 + c * 16 + (s % 4) * 4;
    return (s / 2) * 32 + c * 8 + (s % 2) * 4;
  }
  // d of row g (half 0) or g + 8 (half 1) of output tile t
  static __device__ __forceinline__ int vd(int t, int half, int g) {
    const int e = 2 * t + half;
    return (e / VCE) * (8 * VCE) + g * VCE + e % VCE;
  }
};

// NQ: blocks of 8 packed rows (1 or 2).
template <int D, typename T, int SRC, int NQ>
__global__ void __launch_bounds__(SEQ_ROWS_THREADS, seq_rows_occupancy(D, NQ))
    seq_rows_kernel(const T* __restrict__ Q, const void* __restrict__ K, const void* __restrict__ V, T* __restrict__ O,
                    float* __restrict__ lse, float* __restrict__ ws, SeqArgs a, int64_t pieces) {
  using C = SrCfg<D, SRC>;
  constexpr int R = 8 * NQ;
  constexpr int PITCH = D + 4;
  __shared__ int64_t sh[SEQ_ROWS_THREADS / 32 + 4];
  __shared__ float sm_m[SEQ_ROWS_WARPS][R], sm_l[SEQ_ROWS_WARPS][R];
  __shared__ __align__(16) float sm_o[SEQ_ROWS_WARPS][R][PITCH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  cudaGridDependencySynchronize();
  const SeqPlace place = seq_place<SeqPlan<R, C::KB, SRC>, SEQ_ROWS_THREADS>(a, blockIdx.x, pieces, sh, blockIdx.x == 0);
  using S = SeqSlots<R, D>;
  bool left = false;  // a unit left unfinished
  SeqWalk<SeqPlan<R, C::KB, SRC>> w;
  w.start(a, place);
  for (; w.next(a); w.advance(a)) {
    const SeqUnit& u = w.u;
    const int group = w.group;
    const int r0 = u.t * R;
    // Q^T as the B operand: column g of block q is packed row r0 + 8 q + g
    uint32_t qf[NQ][C::KSTEPS][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = r0 + 8 * q + g;
      const bool on = r < u.rows;
      const T* src = Q + (u.q_begin + (on ? r / group : 0)) * a.q_stride + (u.h * group + (on ? r % group : 0)) * D;
#pragma unroll
      for (int s = 0; s < C::KSTEPS; ++s) {
        uint2 v = make_uint2(0u, 0u);
        if (on) v = *reinterpret_cast<const uint2*>(src + C::kd(s, c));
        if constexpr (C::Q8) {  // the order of the bytes of a K word: (0, 2), (1, 3)
          qf[q][s][0] = __byte_perm(v.x, v.y, 0x5410);
          qf[q][s][1] = __byte_perm(v.x, v.y, 0x7632);
        } else {
          qf[q][s][0] = v.x;
          qf[q][s][1] = v.y;
        }
      }
    }
    // keys that the thread's rows (r0 + 8 q + 2 c, + 1) see
    int seen[NQ][2], most = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * q + 2 * c + e;
        seen[q][e] = r < u.rows ? seq_seen(u.len, u.n, r / group, a.causal) : 0;
        most = max(most, seen[q][e]);
      }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const int kend = min(most, u.j1 * C::KB);
    float m[NQ][2], l[NQ][2], acc[NQ][C::DT][4];
    int vref = -1000;  // reference exponent of V; set by the first step
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m[q][0] = m[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
#pragma unroll
      for (int t = 0; t < C::DT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][t][i] = 0.f;
    }

    uint32_t kr[C::KS / 8][C::KCH * C::KCB / 4];
    uint32_t vr[C::KS / 4][C::VL / 4];
    uint32_t ke[C::KS / 8], ve[C::KS / 4];
    int32_t page[C::KS / 16], npage[C::KS / 16];
    const int32_t* trow = SRC ? a.table + static_cast<int64_t>(u.b) * a.table_width : nullptr;
    const int pmask = (1 << a.page_shift) - 1;

    auto pages = [&](int k0, int32_t (&p)[C::KS / 16]) {  // the pages of a step's keys
      if constexpr (SRC != SEQ_JAGGED) {
#pragma unroll
        for (int i = 0; i < C::KS / 16; ++i) {
          p[i] = -1;
          if (k0 + 16 * i < kend) {
            p[i] = seq_page(trow, k0 + 16 * i, a.page_shift, a.num_pages);
            if (p[i] < 0) flag_error(a.status, kFlagBadShape);
          }
        }
      }
    };
    // row index (of the tensor or the cache) of key k, whose page is p; -1: nothing to load
    auto row_of = [&](int k, int32_t p) -> int64_t {
      if (k >= kend) return -1;
      if constexpr (SRC == SEQ_JAGGED) return u.kv_begin + k;
      if (p < 0) return -1;
      return ((static_cast<int64_t>(p) * a.kv_heads + u.h) << a.page_shift) + (k & pmask);
    };
    auto load_k = [&](int k0) {
#pragma unroll
      for (int i = 0; i < C::KS / 8; ++i) {
        const int64_t row = row_of(k0 + 8 * i + g, SRC ? page[i / 2] : 0);
        ke[i] = 0;
        if (row >= 0) {
          const char* p = SRC == SEQ_JAGGED
                              ? static_cast<const char*>(K) + (row * a.k_stride + u.h * D) * 2
                              : static_cast<const char*>(K) + row * (D * C::ES);
#pragma unroll
          for (int x = 0; x < C::KCH; ++x)
            seq_ldg<C::KCB>(p + (x * 4 + c) * C::KCB, &kr[i][x * (C::KCB / 4)]);
          if constexpr (C::Q8) ke[i] = __ldg(a.k_exp + row);
        } else {
#pragma unroll
          for (int x = 0; x < C::KCH * C::KCB / 4; ++x) kr[i][x] = 0u;
        }
      }
    };
    // V rows of keys 16 s + 2 c, + 1, + 8, + 9
    auto load_v = [&](int k0) {
#pragma unroll
      for (int i = 0; i < C::KS / 4; ++i) {
        const int k = k0 + 16 * (i / 4) + 2 * c + (i & 1) + 8 * ((i >> 1) & 1);
        const int64_t row = row_of(k, SRC ? page[i / 4] : 0);
        ve[i] = 0;
        if (row >= 0) {
          const char* p = SRC == SEQ_JAGGED
                              ? static_cast<const char*>(V) + (row * a.v_stride + u.h * D) * 2
                              : static_cast<const char*>(V) + row * (D * C::ES);
#pragma unroll
          for (int x = 0; x < C::VCH; ++x)
            seq_ldg<C::VCB>(p + (x * 8 + g) * C::VCB, &vr[i][x * (C::VCB / 4)]);
          if constexpr (C::Q8) ve[i] = __ldg(a.v_exp + row);
        } else {
#pragma unroll
          for (int x = 0; x < C::VL / 4; ++x) vr[i][x] = 0u;
        }
      }
    };
    // steps of this warp: block steps j0 .. j1, SUB each
    const int steps = (u.j1 - u.j0) * C::SUB;
    auto key_of = [&](int i) { return (u.j0 + i / C::SUB) * C::KB + ((i % C::SUB) * SEQ_ROWS_WARPS + warp) * C::KS; };
    pages(key_of(0), page);
    load_k(key_of(0));
    load_v(key_of(0));
    for (int i = 0; i < steps; ++i) {
      const int k0 = key_of(i);
      if (k0 >= kend) break;  // a warp's later steps lie behind the end too
      const int k1 = i + 1 < steps ? key_of(i + 1) : kend;
      pages(k1, npage);
      // S^T
      float s[NQ][C::KS / 16][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[q][t][e] = 0.f;
#pragma unroll
      for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
        for (int ks = 0; ks < C::KSTEPS; ++ks) {
          uint32_t a0, a1, a2, a3;
          if constexpr (C::Q8) {
            const uint32_t x = kr[2 * t][ks], y = kr[2 * t + 1][ks];
            a0 = seq_raw2<T>(x << 8);
            a1 = seq_raw2<T>(y << 8);
            a2 = seq_raw2<T>(x);
            a3 = seq_raw2<T>(y);
            if constexpr (Half16<T>::kBF16) {  // out of the range where products would underflow
              constexpr uint32_t f = 0x7B807B80u;  // 2^120 twice
              a0 = seq_mul2<T>(a0, f);
              a1 = seq_mul2<T>(a1, f);
              a2 = seq_mul2<T>(a2, f);
              a3 = seq_mul2<T>(a3, f);
            }
          } else {
            a0 = kr[2 * t][2 * ks];
            a1 = kr[2 * t + 1][2 * ks];
            a2 = kr[2 * t][2 * ks + 1];
            a3 = kr[2 * t + 1][2 * ks + 1];
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma_16816<T>(s[q][t], a0, a1, a2, a3, qf[q][ks][0], qf[q][ks][1]);
        }
      // factors of the scores: the scale, and the rows' exponents
      float kf[C::KS / 8];
#pragma unroll
      for (int t = 0; t < C::KS / 8; ++t) {
        kf[t] = scale_log2;
        if constexpr (C::Q8) kf[t] *= seq_pow(ke[t]) * (Half16<T>::kBF16 ? 1.f : 256.f);
      }
      // V of this step is in registers: its pages are not needed any more
#pragma unroll
      for (int t = 0; t < C::KS / 16; ++t) page[t] = npage[t];
      if (k1 < kend) load_k(k1);
      // softmax weights
      uint32_t pb[NQ][C::KS / 16][2];
      bool raise = false;
      float fac[NQ][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = k0 + 16 * t + 8 * (e >> 1) + g;
            s[q][t][e] = k < seen[q][e & 1] ? s[q][t][e] * kf[2 * t + (e >> 1)] : -INFINITY;
            mx[e & 1] = fmaxf(mx[e & 1], s[q][t][e]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          const float mn = fmaxf(m[q][e], mx[e]);
          raise |= mn > m[q][e];
          fac[q][e] = m[q][e] == -INFINITY ? 0.f : seq_ex2(m[q][e] - mn);
          m[q][e] = mn;
          l[q][e] *= fac[q][e];
        }
        const float mz[2] = {m[q][0] == -INFINITY ? 0.f : m[q][0], m[q][1] == -INFINITY ? 0.f : m[q][1]};
#pragma unroll
        for (int t = 0; t < C::KS / 16; ++t) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = seq_ex2(s[q][t][e] - mz[e & 1]);
            l[q][e & 1] += p[e];
          }
          pb[q][t][0] = seq_movmatrix(Half16<T>::pack2(p[0], p[1]));
          pb[q][t][1] = seq_movmatrix(Half16<T>::pack2(p[2], p[3]));
        }
      }
      float vf = 1.f;  // change of V's reference
      uint32_t vfac[C::KS / 8];
      if constexpr (C::Q8) {
        int top = -1000;
#pragma unroll
        for (int t = 0; t < C::KS / 4; ++t) top = max(top, ve[t] == 255 ? -1000 : static_cast<int>(ve[t]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (top > vref + 7) {  // uniform over the warp
          vf = vref == -1000 ? 0.f : exp2f(static_cast<float>(vref - top));
          vref = top;
          raise = true;
        }
#pragma unroll
        for (int t = 0; t < C::KS / 8; ++t) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = static_cast<int>(ve[2 * t + e]);
            f[e] = x == 255 ? __uint_as_float(0x7FC00000u)
                            : seq_ex2(static_cast<float>(max(x - vref, -140) + kRawPow<T>));
          }
          vfac[t] = Half16<T>::pack2(f[0], f[1]);
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const float f0 = fac[q][0] * vf, f1 = fac[q][1] * vf;
#pragma unroll
          for (int t = 0; t < C::DT; ++t) {
            acc[q][t][0] *= f0;
            acc[q][t][1] *= f1;
            acc[q][t][2] *= f0;
            acc[q][t][3] *= f1;
          }
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
        for (int dt = 0; dt < C::DT; ++dt) {
          uint32_t f[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // keys 2 c, + 1, then + 8, + 9
            if constexpr (C::Q8) {
              const int e = 2 * dt, wd = e / 4;  // elements e, e + 1: bytes of word wd
              const uint32_t x = vr[4 * t + 2 * h][wd], y = vr[4 * t + 2 * h + 1][wd];
              // bytes 1 and 3 of the result: the same byte of both keys' words
              f[2 * h] = seq_mul2<T>(seq_raw2<T>(__byte_perm(x, y, (e % 4) ? 0x6020 : 0x4000)), vfac[2 * t + h]);
              f[2 * h + 1] = seq_mul2<T>(seq_raw2<T>(__byte_perm(x, y, (e % 4) ? 0x7030 : 0x5010)), vfac[2 * t + h]);
            } else {
              const uint32_t x = vr[4 * t + 2 * h][dt], y = vr[4 * t + 2 * h + 1][dt];
              f[2 * h] = __byte_perm(x, y, 0x5410);
              f[2 * h + 1] = __byte_perm(x, y, 0x7632);
            }
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma_16816<T>(acc[q][dt], f[0], f[1], f[2], f[3], pb[q][t][0], pb[q][t][1]);
        }
      if (k1 < kend) load_v(k1);
    }

    // the row sums over the lanes of a column, then the block's warps together
    const float vscale = C::Q8 ? (vref == -1000 ? 0.f : seq_pow(vref)) : 1.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], o);
        if (g == 0) {
          sm_m[warp][8 * q + 2 * c + e] = m[q][e];
          sm_l[warp][8 * q + 2 * c + e] = l[q][e];
        }
#pragma unroll
        for (int t = 0; t < C::DT; ++t)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            sm_o[warp][8 * q + 2 * c + e][C::vd(t, half, g)] = acc[q][t][2 * half + e] * vscale;
      }
    __syncthreads();
    const bool whole = u.j0 == 0 && u.j1 == u.nb;
    const int rows = min(R, u.rows - r0);
    float* slot = whole ? nullptr : S::slot(ws, pieces, blockIdx.x, u.j0 > 0);
    if (u.j0 == 0 && u.j1 < u.nb) {
      left = true;
      if (threadIdx.x == 0) seq_leave_note<R, D>(ws, blockIdx.x, u, u.q_begin, R, group, place.per, false);
    }
    for (int i = threadIdx.x; i < rows * (D / 4); i += SEQ_ROWS_THREADS) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float mm = sm_m[0][r];
#pragma unroll
      for (int x = 1; x < SEQ_ROWS_WARPS; ++x) mm = fmaxf(mm, sm_m[x][r]);
      const float mz = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < SEQ_ROWS_WARPS; ++x) {
        const float f = seq_ex2(sm_m[x][r] - mz);
        const float4 v = *reinterpret_cast<const float4*>(&sm_o[x][r][d]);
        ll += f * sm_l[x][r];
        o.x += f * v.x;
        o.y += f * v.y;
        o.z += f * v.z;
        o.w += f * v.w;
      }
      if (whole) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int64_t row = (u.q_begin + (r0 + r) / group) * a.q_heads + u.h * group + (r0 + r) % group;
        *reinterpret_cast<uint2*>(O + row * D + d) =
            make_uint2(Half16<T>::pack2(o.x * inv, o.y * inv), Half16<T>::pack2(o.z * inv, o.w * inv));
        if (lse && d == 0) lse[row] = ll == 0.f ? -INFINITY : 0.69314718055994531f * (mz + log2f(ll));
      } else {
        *reinterpret_cast<float4*>(S::o(slot, r, d)) = o;
        if (d == 0) {
          S::m(slot)[r] = mm;
          S::l(slot)[r] = ll;
        }
      }
    }
    __syncthreads();
  }
  if (ws && !left && threadIdx.x == 0) seq_leave_note<R, D>(ws, blockIdx.x, w.u, 0, R, 1, place.per, true);
}

}  // namespace wk
