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
// 8-bit rows are converted to fp16, whatever the type of Q and O: e4m3 values are exact in it, and
// one instruction converts two. The rows' powers of two stay apart: K's joins the fp32 score s, V's
// the exponent of the weight, P = 2^(s + x - w), with w the running maximum of s + x over the keys that
// the row sees, beside the row sum of 2^(s - m). So what a row gives does not depend on the size of
// rows that have no weight. (Multiplied onto the converted values, relative to the largest row met, it
// lost those 2^25 below it, and took two more instructions a pair against one exponential a weight.)
// bf16 queries are scaled by a power of two of their own row into fp16: elements down to 2^-31 of the
// row's largest are exact, smaller ones round to steps of 2^-38 of it. (Shifting e4m3's bits into bf16's
// fields instead, which has no such limit, took four instructions a pair and made the kernel wait for
// the ALU: 86 us at 64 sequences of up to 15,000 keys, where this takes 62.)
#pragma once

#include "seq_args.cuh"

namespace wk {

constexpr int SEQ_ROWS_WARPS = 4;
constexpr int SEQ_ROWS_THREADS = 32 * SEQ_ROWS_WARPS;
// Blocks per SM, and so the registers of a thread. More warps hide more of a step's dependent
// instructions, as long as registers do not spill (more than a few dozen bytes). One new token over 64
// caches of up to 15,000 keys, with 2, 3, 4 blocks (bytes spilled):
//   8 bits   d = 128: 77, 64, 63 us (0, 0, 50)     d = 160: 84, 73, 98 us (0, 0, 290)
//   16 bits  d = 128: 88, 85, 98 us (0, 0, 306)    d = 160: 103, 115, 168 us (0, 226, 646)
// 16 rows of a wide head need the registers of two.
constexpr int seq_rows_occupancy(int d, int nq, bool q8) {
  return nq == 2 ? (d >= 128 ? 2 : 3) : (d <= 64 || (d == 128 && q8) ? 4 : d == 160 && !q8 ? 2 : 3);
}

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

// Two e4m3 values as two fp16 values.
__device__ __forceinline__ uint32_t seq_e4m3_f16(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ uint16_t seq_lo16(uint32_t w) { return static_cast<uint16_t>(w); }
__device__ __forceinline__ uint16_t seq_hi16(uint32_t w) { return static_cast<uint16_t>(w >> 16); }

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
  static constexpr int KS = 16;                                    // keys per step of a warp
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
__global__ void __launch_bounds__(SEQ_ROWS_THREADS, seq_rows_occupancy(D, NQ, SRC == SEQ_PAGED8))
    seq_rows_kernel(const T* __restrict__ Q, const void* __restrict__ K, const void* __restrict__ V, T* __restrict__ O,
                    float* __restrict__ lse, float* __restrict__ ws, SeqArgs a, int64_t pieces) {
  using C = SrCfg<D, SRC>;
  using CT = std::conditional_t<C::Q8, __half, T>;  // the tensor cores' operand type
  constexpr int R = 8 * NQ;
  constexpr int PITCH = D + 4;
  __shared__ int64_t sh[SEQ_ROWS_THREADS / 32 + 4];
  __shared__ float sm_m[SEQ_ROWS_WARPS][R], sm_l[SEQ_ROWS_WARPS][R];
  __shared__ __align__(16) float sm_o[SEQ_ROWS_WARPS][R][PITCH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  seq_wait_before();
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
    float qpow[NQ][2];  // powers of two taken out of the thread's rows (bf16 queries, 8-bit keys)
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = r0 + 8 * q + g;
      const bool on = r < u.rows;
      const T* src = Q + (u.q_begin + (on ? r / group : 0)) * a.q_stride + (u.h * group + (on ? r % group : 0)) * D;
#pragma unroll
      for (int s = 0; s < C::KSTEPS; ++s) {
        uint2 v = make_uint2(0u, 0u);
        if (on) v = *reinterpret_cast<const uint2*>(src + C::kd(s, c));
        qf[q][s][0] = v.x;
        qf[q][s][1] = v.y;
      }
      qpow[q][0] = qpow[q][1] = 1.f;
      if constexpr (C::Q8 && Half16<T>::kBF16) {
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < C::KSTEPS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[q][s][i])), fabsf(bf16_hi(qf[q][s][i]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top = 1.f * 2^(e - 127): times 2^(141 - e) it lies in [2^14, 2^15). The factor stops at 2^127
        // for the smallest; rows that are not finite stay so under any.
        const int e = max(14, min(254, static_cast<int>(__float_as_uint(top) >> 23)));
        const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
        const float back = seq_pow(e - 14);  // 2^(e - 141)
#pragma unroll
        for (int s = 0; s < C::KSTEPS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[q][s][i] = Half16<__half>::pack2(bf16_lo(qf[q][s][i]) * f, bf16_hi(qf[q][s][i]) * f);
#pragma unroll
        for (int x = 0; x < 2; ++x) qpow[q][x] = __shfl_sync(0xffffffffu, back, (2 * c + x) * 4);
      }
    }
    // keys that the thread's rows (r0 + 8 q + 2 c, + 1) see
    int seen[NQ][2], most = 0, least = INT32_MAX;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * q + 2 * c + e;
        seen[q][e] = r < u.rows ? seq_seen(u.len, u.n, r / group, a.causal) : 0;
        most = max(most, seen[q][e]);
        if (r < u.rows) least = min(least, seen[q][e]);
      }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
    least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));
    least = min(least, most);
    const int kend = min(most, u.j1 * C::KB);
    float m[NQ][2], l[NQ][2], acc[NQ][C::DT][4];
    float wm[NQ][2];  // 8-bit: what weights and acc are relative to (else m)
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m[q][0] = m[q][1] = wm[q][0] = wm[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
#pragma unroll
      for (int t = 0; t < C::DT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][t][i] = 0.f;
    }

    uint32_t kr[C::KS / 8][C::KCH * C::KCB / 4];
    uint32_t vr[C::KS / 4][C::VL / 4];
    uint32_t ke[C::KS / 8], ve[C::KS / 8];  // exponents of K rows, and of the V rows of the same keys
    // a step's keys in groups of 16, each within one page: the group's first row (of the tensor or the
    // cache), or -1 where there is nothing to load
    int64_t at[C::KS / 16];
    const int32_t* trow = SRC ? a.table + static_cast<int64_t>(u.b) * a.table_width : nullptr;
    const int pmask = (1 << a.page_shift) - 1;
    auto place_of = [&](int k0, int64_t (&p)[C::KS / 16]) {
#pragma unroll
      for (int i = 0; i < C::KS / 16; ++i) {
        const int k = k0 + 16 * i;
        p[i] = -1;
        if (k < kend) {
          if constexpr (SRC == SEQ_JAGGED) {
            p[i] = u.kv_begin + k;
          } else {
            const int page = seq_page(trow, k, a.page_shift, a.num_pages);
            if (page < 0) flag_error(a.status, kFlagBadShape);
            else p[i] = ((static_cast<int64_t>(page) * a.kv_heads + u.h) << a.page_shift) + (k & pmask);
          }
        }
      }
    };
    const int64_t k_row = SRC == SEQ_JAGGED ? a.k_stride * 2 : D * C::ES, v_row = SRC == SEQ_JAGGED ? a.v_stride * 2 : D * C::ES;
    const char* k_lane = static_cast<const char*>(K) + (SRC == SEQ_JAGGED ? u.h * D * 2 : 0) + g * k_row + c * C::KCB;
    const char* v_lane = static_cast<const char*>(V) + (SRC == SEQ_JAGGED ? u.h * D * 2 : 0) + 2 * c * v_row + g * C::VCB;
    // K rows g and g + 8 of each group; all: the step's keys are all there
    auto load_k = [&](int k0, bool all) {
#pragma unroll
      for (int i = 0; i < C::KS / 8; ++i) {
        const int r = 8 * (i & 1);
        ke[i] = ve[i] = 0;
        if (at[i / 2] >= 0 && (all || k0 + 16 * (i / 2) + r + g < kend)) {
          const char* p = k_lane + (at[i / 2] + r) * k_row;
#pragma unroll
          for (int x = 0; x < C::KCH; ++x) seq_ldg<C::KCB>(p + x * 4 * C::KCB, &kr[i][x * (C::KCB / 4)]);
          if constexpr (C::Q8) {
            ke[i] = __ldg(a.k_exp + at[i / 2] + r + g);
            ve[i] = __ldg(a.v_exp + at[i / 2] + r + g);
          }
        } else {
#pragma unroll
          for (int x = 0; x < C::KCH * C::KCB / 4; ++x) kr[i][x] = 0u;
        }
      }
    };
    // V rows 2 c, + 1, + 8, + 9 of each group
    auto load_v = [&](int k0, bool all) {
#pragma unroll
      for (int i = 0; i < C::KS / 4; ++i) {
        const int r = (i & 1) + 8 * ((i >> 1) & 1);
        if (at[i / 4] >= 0 && (all || k0 + 16 * (i / 4) + r + 2 * c < kend)) {
          const char* p = v_lane + (at[i / 4] + r) * v_row;
#pragma unroll
          for (int x = 0; x < C::VCH; ++x) seq_ldg<C::VCB>(p + x * 8 * C::VCB, &vr[i][x * (C::VCB / 4)]);
        } else {
#pragma unroll
          for (int x = 0; x < C::VL / 4; ++x) vr[i][x] = 0u;
        }
      }
    };
    // steps of this warp: block steps j0 .. j1, SUB each
    const int steps = (u.j1 - u.j0) * C::SUB;
    auto key_of = [&](int i) { return (u.j0 + i / C::SUB) * C::KB + ((i % C::SUB) * SEQ_ROWS_WARPS + warp) * C::KS; };
    place_of(key_of(0), at);
    load_k(key_of(0), false);
    load_v(key_of(0), false);
    for (int i = 0; i < steps; ++i) {
      const int k0 = key_of(i);
      if (k0 >= kend) break;  // a warp's later steps lie behind the end too
      const int k1 = i + 1 < steps ? key_of(i + 1) : kend;
      place_of(k1, at);  // this step's V is in registers already
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
            a0 = seq_e4m3_f16(seq_lo16(x));
            a1 = seq_e4m3_f16(seq_lo16(y));
            a2 = seq_e4m3_f16(seq_hi16(x));
            a3 = seq_e4m3_f16(seq_hi16(y));
          } else {
            a0 = kr[2 * t][2 * ks];
            a1 = kr[2 * t + 1][2 * ks];
            a2 = kr[2 * t][2 * ks + 1];
            a3 = kr[2 * t + 1][2 * ks + 1];
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma_16816<CT>(s[q][t], a0, a1, a2, a3, qf[q][ks][0], qf[q][ks][1]);
        }
      // factors of the scores: the scale, and K's powers of two; V's exponents
      float kf[C::KS / 8], vx[C::KS / 8];
#pragma unroll
      for (int t = 0; t < C::KS / 8; ++t) {
        kf[t] = scale_log2;
        vx[t] = 0.f;
        if constexpr (C::Q8) {
          kf[t] *= seq_pow(ke[t]);
          vx[t] = ve[t] == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(static_cast<int>(ve[t]) - 127);
        }
      }
      const bool all1 = k1 + C::KS <= kend;
      if (all1) load_k(k1, true);
      else if (k1 < kend) load_k(k1, false);
      // scores, the exponents of the weights, and each thread's own maxima of its two columns
      bool up = false;
      float mx[NQ][2], wx[NQ][2];
      float y[NQ][C::KS / 16][4];
      if (k0 + C::KS <= least) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[q][t][e] *= kf[2 * t + (e >> 1)] * qpow[q][e & 1];
              if constexpr (C::Q8) y[q][t][e] = s[q][t][e] + vx[2 * t + (e >> 1)];
            }
      } else {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int t = 0; t < C::KS / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = k0 + 16 * t + 8 * (e >> 1) + g;
              const bool sees = k < seen[q][e & 1];
              s[q][t][e] = sees ? s[q][t][e] * (kf[2 * t + (e >> 1)] * qpow[q][e & 1]) : -INFINITY;
              if constexpr (C::Q8) y[q][t][e] = sees ? s[q][t][e] + vx[2 * t + (e >> 1)] : -INFINITY;
            }
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[q][e] = wx[q][e] = -INFINITY;
#pragma unroll
          for (int t = 0; t < C::KS / 16; ++t) {
            mx[q][e] = fmaxf(mx[q][e], fmaxf(s[q][t][e], s[q][t][e + 2]));
            if constexpr (C::Q8) wx[q][e] = fmaxf(wx[q][e], fmaxf(y[q][t][e], y[q][t][e + 2]));
          }
          up |= mx[q][e] > m[q][e] + 8.f;
          if constexpr (C::Q8) up |= wx[q][e] > wm[q][e] + 8.f;
        }
      // The running maxima move only when a value is more than 2^8 above one: one vote, and a reduction
      // over the lanes only then.
      if (__any_sync(0xffffffffu, up)) {
        // the higher of `high` and the lanes' x in `high`; returns 2^(high before - after)
        auto raise = [&](float& high, float x) -> float {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          const float now = fmaxf(high, x);
          const float f = high == -INFINITY ? 0.f : seq_ex2(high - now);
          high = now;
          return f;
        };
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float fac[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            fac[e] = raise(m[q][e], mx[q][e]);
            l[q][e] *= fac[e];
            if constexpr (C::Q8) fac[e] = raise(wm[q][e], wx[q][e]);
          }
#pragma unroll
          for (int t = 0; t < C::DT; ++t) {
            acc[q][t][0] *= fac[0];
            acc[q][t][1] *= fac[1];
            acc[q][t][2] *= fac[0];
            acc[q][t][3] *= fac[1];
          }
        }
      }
      // row sums and weights
      uint32_t pb[NQ][C::KS / 16][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const float mz[2] = {m[q][0] == -INFINITY ? 0.f : m[q][0], m[q][1] == -INFINITY ? 0.f : m[q][1]};
        const float wz[2] = {wm[q][0] == -INFINITY ? 0.f : wm[q][0], wm[q][1] == -INFINITY ? 0.f : wm[q][1]};
#pragma unroll
        for (int t = 0; t < C::KS / 16; ++t) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = seq_ex2(s[q][t][e] - mz[e & 1]);
            l[q][e & 1] += p[e];
            if constexpr (C::Q8) p[e] = seq_ex2(y[q][t][e] - wz[e & 1]);
          }
          pb[q][t][0] = seq_movmatrix(Half16<CT>::pack2(p[0], p[1]));
          pb[q][t][1] = seq_movmatrix(Half16<CT>::pack2(p[2], p[3]));
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
              // byte e of both keys, then byte e + 1 of both
              const uint32_t w = __byte_perm(vr[4 * t + 2 * h][wd], vr[4 * t + 2 * h + 1][wd], (e % 4) ? 0x7362 : 0x5140);
              f[2 * h] = seq_e4m3_f16(seq_lo16(w));
              f[2 * h + 1] = seq_e4m3_f16(seq_hi16(w));
            } else {
              const uint32_t x = vr[4 * t + 2 * h][dt], y = vr[4 * t + 2 * h + 1][dt];
              f[2 * h] = __byte_perm(x, y, 0x5410);
              f[2 * h + 1] = __byte_perm(x, y, 0x7632);
            }
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) mma_16816<CT>(acc[q][dt], f[0], f[1], f[2], f[3], pb[q][t][0], pb[q][t][1]);
        }
      if (all1) load_v(k1, true);
      else if (k1 < kend) load_v(k1, false);
    }

    // the row sums over the lanes of a column, then the block's warps together
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], o);
        // the square root of 2^(w - m), which fp32 holds whatever V's exponents are
        float between = 1.f;
        if constexpr (C::Q8) between = wm[q][e] == -INFINITY ? 0.f : seq_ex2(0.5f * (wm[q][e] - m[q][e]));
        if (g == 0) {
          sm_m[warp][8 * q + 2 * c + e] = m[q][e];
          sm_l[warp][8 * q + 2 * c + e] = l[q][e];
        }
#pragma unroll
        for (int t = 0; t < C::DT; ++t)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            sm_o[warp][8 * q + 2 * c + e][C::vd(t, half, g)] = acc[q][t][2 * half + e] * between * between;
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
