// seq_back.cuh -- gradients of the jagged cross attention on the 5th-generation tensor cores.
//
// With P = exp(S scale - lse), dP = dO V^T and delta = sum(dO * O) per row,
//   dS = P (dP - delta) scale,   dQ = dS K,   dK = dS^T Q,   dV = P^T dO.
// Two kernels of one shape, so that every sum has one owner and nothing is added with atomics (the
// results do not depend on the order in which blocks run):
//   DQ    128 packed query rows stand (Q, dO), blocks of 128 or 64 keys go by (K, V):
//         T1 = Q K^T, T2 = dO V^T, dQ += dS K
//   DKV   128 keys stand (K, V), blocks of up to 64 packed query rows go by (Q, dO), so that a key
//         head's sum over its query heads is part of the product:
//         T1 = K Q^T, T2 = V dO^T, dV += P^T dO, dK += dS^T Q
// S and dP are computed twice (7 products instead of 5): that costs less than exchanging dQ through
// memory, and needs no zeroed fp32 gradient.
//
// Both operands of T1, T2 come from shared memory, the tiles that go by are read a second time as
// MN-major operands of the accumulating products, whose A operands (P, dS) are written over the
// columns of T1, T2 that the same thread has just read, so the element-wise warps (two per lane
// quarter, half the columns each) need no barrier among themselves. T1 and T2 of the next block are
// computed under this one's element-wise work as far as TMEM has room beside the accumulators.
//
// delta comes from the stored (rounded) O, except where one block holds all keys of a row: there it
// is sum P dP in fp32. With few keys dP - delta cancels almost wholly (with one key it is 0), and
// O's rounding would be most of what is left.
//
// Rows of a tile that goes by and lie behind the sequence's end are zeros in shared memory (0 * NaN
// is NaN); their columns get P = 0 (DQ: by a select; DKV: lse = inf). Rows of a tile that stands and
// lie behind it only give results that are not stored.
#pragma once

#include "seq_tile.cuh"

namespace wk {

template <int D_, bool DKV_>
struct SbCfg {
  static constexpr int D = D_;
  static constexpr bool DKV = DKV_;
  // Rows that go by at a time. An MMA of N = 64 with both operands in shared memory reads 6 KB in its 32
  // cycles, one of N = 128 8 KB in 64: 128 where TMEM holds three results of that width (not beside
  // two accumulators, nor beside one of 160).
  static constexpr int R = 128, YB = !DKV && D <= 128 ? 128 : 64;
  static constexpr int BW = (D % 64 == 0) ? 64 : 32;
  static constexpr int SWB = BW * 2;
  static constexpr uint32_t SWMODE = BW == 64 ? 2u : 4u;
  static constexpr uint32_t DESC_HI = seq_desc_hi(8 * SWB, SWMODE);
  static constexpr int NBOX = D / BW;
  static constexpr int ABOXB = R * SWB, YBOXB = YB * SWB;
  static constexpr int AB = NBOX * ABOXB, YBYTES = NBOX * YBOXB;  // one tile that stands / goes by
  static constexpr int NACC = DKV ? 2 : 1;
  static constexpr int LIMIT = 227 * 1024;
  static constexpr int NU = 4;
  static constexpr int BARB = 512;
  static constexpr int UNITB = NU * static_cast<int>(sizeof(SeqUnit));
  static constexpr int REDB = 8 * 2 * 64 * 4;  // pair exchange of DQ; lse and delta of DKV's columns per warp, twice
  static constexpr int STAGEB = 8 * SEQ_STAGE_BYTES;
  static constexpr int FIXED = BARB + UNITB + REDB + STAGEB;
  // Standing tiles in flight: two where units are short (DKV: as many blocks as query rows ask for),
  // one where they are long and the room is better used for blocks that go by.
  static constexpr int SBUF = DKV && D <= 128 ? 2 : 1;
  static constexpr int STAGES_RAW = (LIMIT - FIXED - 2 * SBUF * AB) / (2 * YBYTES);
  static constexpr int STAGES = STAGES_RAW > 4 ? 4 : STAGES_RAW;
  static constexpr int RAW = FIXED + 2 * SBUF * AB + STAGES * 2 * YBYTES;
  static constexpr int SMEM = RAW > 120 * 1024 ? RAW : 120 * 1024;  // one block per SM: its TMEM is its own
  // TMEM: SLOTS places of YB columns that T1 and T2 of the blocks take in turn, then the accumulators.
  // With four, both of the next block are computed under this one's element-wise work; with three
  // its T1 is.
  static constexpr int SLOTS = 4 * YB + NACC * D <= 512 ? 4 : 3;
  static constexpr int ACOL = SLOTS * YB;
  static __device__ __forceinline__ uint32_t t1(uint32_t g) { return (2u * g) % SLOTS * YB; }
  static __device__ __forceinline__ uint32_t t2(uint32_t g) { return (2u * g + 1u) % SLOTS * YB; }
  static constexpr int THREADS = 384;
  static_assert(ACOL + NACC * D <= 512 && STAGES >= 2 && AB % 1024 == 0 && YBYTES % 1024 == 0, "layout");
  static_assert((2 * SBUF + 2 * STAGES + 7 + 2 * NU) * 8 + 8 <= BARB, "barriers");
};

// How large a unit's dS can be, for fp16. |dP - delta| <= 2 |dO_i| max_j |V_j| (norms of rows), so dS
// enters its product times the power of two that takes this bound to at most 2^12, and dQ and dK are
// scaled back in fp32, with `scale` too: a loss of any size uses fp16's range from the top, with all
// bits down to 2^-26 of the bound. (Times `scale` alone, with dO of 2^-10 over 2048 keys, dQ was off by
// 2 %; with dO V^T beyond 65504 it was infinite.) The norms come from a pass over V and dO before the
// two kernels: the largest of each chunk of 32 tokens, so that a unit reads few, and each dO row's own,
// because the rows' losses differ. A training step at the 2-layer shape takes 140 us in fp16 with it and
// 128 without; bf16 does without.
constexpr int SEQ_CHUNK = 32;
struct SeqRange {
  float* rows;  // [total_q, q_heads] squared norms of dO
  float* g;     // [total_q / SEQ_CHUNK + batch, kv_heads] the largest of a chunk of a sequence's tokens
  float* v;     // [total_kv / SEQ_CHUNK + batch, kv_heads] the same of V
};

// A sequence's chunks: those of sequences before it end below (begin / SEQ_CHUNK + b).
__device__ __forceinline__ int64_t seq_chunk(int64_t begin, int64_t b, int c, int kv_heads, int h) {
  return (begin / SEQ_CHUNK + b + c) * kv_heads + h;
}

// The largest over the chunks of `rows` rows, for the whole warp.
__device__ __forceinline__ float seq_chunks_max(const float* chunks, int64_t begin, int64_t b, int rows, int kv_heads,
                                                int h) {
  float x = 0.f;
  for (int c = threadIdx.x & 31; c < (rows + SEQ_CHUNK - 1) / SEQ_CHUNK; c += 32)
    x = fmaxf(x, __ldg(chunks + seq_chunk(begin, b, c, kv_heads, h)));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// k with 2 sqrt(x) 2^k in (2^10, 2^12]; 0 where there is no such bound (zero, infinite, NaN).
__device__ __forceinline__ int seq_range_log2(float x) {
  const uint32_t e = __float_as_uint(x) >> 23;
  if (e == 0 || e >= 255) return 0;
  return 11 - ((static_cast<int>(e) - 127 + 2) >> 1);
}
__device__ __forceinline__ float seq_exp2i(int k) { return __uint_as_float(static_cast<uint32_t>(127 + k) << 23); }

// The warps of blocks (b, V or dO, z) take the (chunk, key head) of sequence b in turn, four lanes to a
// row and 16 rows' loads at a time; bound by the latency of offsets, rows and the reduction, one after
// the other (33 MB of V at the 2-layer shape: 12.4 us from cold caches; 14.3 with chunks of 128 and a block
// each, 14.1 with two chunks to a warp and 32 rows at a time).
template <int D, typename T>
__global__ void __launch_bounds__(256)
    seq_range_kernel(const T* __restrict__ V, const T* __restrict__ dO, SeqRange out, SeqArgs a) {
  seq_wait_before();
  const int lane = threadIdx.x & 31, group = a.q_heads / a.kv_heads;
  const int64_t b = blockIdx.x;
  const bool is_v = blockIdx.y == 0;
  const SeqSpan span = is_v ? seq_keys<SEQ_JAGGED>(a, b) : seq_queries(a, b);
  const int each = is_v ? 1 : group;  // rows of a token
  const int tasks = (span.len + SEQ_CHUNK - 1) / SEQ_CHUNK * a.kv_heads;
  for (int task = blockIdx.z * 8 + (threadIdx.x >> 5); task < tasks; task += gridDim.z * 8) {
    const int c = task / a.kv_heads, h = task % a.kv_heads;
    const int rows = min(SEQ_CHUNK, span.len - c * SEQ_CHUNK) * each;
    float top = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 16) {
      uint4 y[2][D / 32];
      int64_t row[2];  // of dO
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = r0 + 8 * j + (lane >> 2);
        const int64_t token = span.begin + c * SEQ_CHUNK + r / each;
        row[j] = token * a.q_heads + h * group + r % each;
        const uint4* p =
            reinterpret_cast<const uint4*>(is_v ? V + token * a.v_stride + h * D : dO + row[j] * D) + (lane & 3);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          y[j][i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) y[j][i] = __ldg(p + 4 * i);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&y[j][i])[k];
            x = fmaf(Half16<T>::lo(w), Half16<T>::lo(w), x);
            x = fmaf(Half16<T>::hi(w), Half16<T>::hi(w), x);
          }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (!is_v && r0 + 8 * j + (lane >> 2) < rows && (lane & 3) == 0) out.rows[row[j]] = x;
        top = fmaxf(top, x);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) (is_v ? out.v : out.g)[seq_chunk(span.begin, b, c, a.kv_heads, h)] = top;
  }
}

// What a weight of 1 is held as in DKV's operand P. A key of a long history has weights of 2^-14 and
// far below, where fp16 has few bits left or none, and dV adds up ordinary numbers of them. Times 2^12
// weights from 2^-26 on keep all bits, and 2^4 are left for scores so large that fp32's rounding of
// them (the difference of score and lse) lifts a weight above 1. bf16 has the range of fp32.
template <typename T>
struct SbP {
  static constexpr int LOG2 = Half16<T>::kBF16 ? 0 : 12;
  static constexpr float ONE = static_cast<float>(1 << LOG2);
};

template <int D, typename T, bool DKV>
__global__ void __launch_bounds__(SbCfg<D, DKV>::THREADS, 1)
    seq_back_kernel(const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmA2,
                    const __grid_constant__ CUtensorMap tmY1, const __grid_constant__ CUtensorMap tmY2,
                    const T* __restrict__ O, const T* __restrict__ dO, const float* __restrict__ lse,
                    float* __restrict__ delta, SeqRange range, T* __restrict__ G1, T* __restrict__ G2,
                    float* __restrict__ ws, SeqArgs a, int64_t pieces) {
  using C = SbCfg<D, DKV>;
  using P = SeqPlanBack<DKV>;
  using S = SeqSlots<128, C::NACC * D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0u) {  // the swizzled layout needs 1024-byte alignment
    if (threadIdx.x == 0) flag_error(a.status, kFlagBadShape);
    return;
  }
  uint8_t* sA = smem_raw;                           // [SBUF][A1, A2]
  uint8_t* sY = sA + 2 * C::SBUF * C::AB;           // [STAGES][Y1, Y2]
  uint8_t* rest = sY + C::STAGES * 2 * C::YBYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rest);
  uint64_t* a_full = bars;                          // [SBUF] standing tiles landed
  uint64_t* a_empty = a_full + C::SBUF;             // [SBUF] the unit's last T product has read them
  uint64_t* y_full = a_empty + C::SBUF;             // [STAGES]
  uint64_t* y_empty = y_full + C::STAGES;           // [STAGES]
  uint64_t* t_full = y_empty + C::STAGES;           // [2] T1, T2 in TMEM
  uint64_t* p_full = t_full + 2;                    // [2] P, dS in TMEM
  uint64_t* acc_full = p_full + 2;                  // the unit's accumulators are complete
  uint64_t* acc_empty = acc_full + 1;               // and read
  uint64_t* fin = acc_empty + 1;
  uint64_t* u_full = fin + 1;                       // [NU]
  uint64_t* u_empty = u_full + C::NU;               // [NU]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(u_empty + C::NU);
  SeqUnit* unit = reinterpret_cast<SeqUnit*>(rest + C::BARB);
  float* red = reinterpret_cast<float*>(rest + C::BARB + C::UNITB);
  unsigned* status = a.status;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmA1);
    prefetch_tmap(&tmA2);
    prefetch_tmap(&tmY1);
    prefetch_tmap(&tmY2);
    for (int i = 0; i < C::SBUF; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], 1);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&y_full[i], 1);
      mbar_init(&y_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&p_full[i], 8);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 8);
    mbar_init(fin, 1);
    for (int i = 0; i < C::NU; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 10);  // producer, MMA issuer, 8 element-wise warps
    }
    fence_mbar_init();
  }
  // nothing of the kernels before is read above, and no TMEM is taken that they may still need
  seq_wait_before();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const SeqPlace place =
      seq_place<P, C::THREADS>(a, blockIdx.x, pieces, reinterpret_cast<int64_t*>(red), blockIdx.x == 0);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int group = a.q_heads / a.kv_heads;

  uint32_t ui = 0;
  auto unit_take = [&](SeqUnit& u) -> bool {
    const uint32_t s = ui % C::NU;
    if (!seq_wait(&u_full[s], (ui / C::NU) & 1u, status)) return false;
    u = unit[s];
    return u.b >= 0;
  };
  auto unit_done = [&]() { mbar_arrive(&u_empty[ui % C::NU]); };
  // rows that go by in a unit, and the piece's real blocks of them
  auto passing = [&](const SeqUnit& u) -> int { return DKV ? u.n * group : u.len; };
  auto real_end = [&](const SeqUnit& u) -> int { return min(u.j1, (passing(u) + a.block - 1) / a.block); };

  if (warp == 2) {
    // -------------------------------------------------------------- walker
    if (lane == 0) {
      SeqWalk<P> w;
      w.start(a, place);
      bool left = false;
      for (;;) {
        const bool more = w.next(a);
        const uint32_t s = ui % C::NU;
        if (!seq_wait(&u_empty[s], ((ui / C::NU) & 1u) ^ 1u, status)) break;
        if (!more) w.u.b = -1;
        unit[s] = w.u;
        mbar_arrive(&u_full[s]);
        ++ui;
        if (!more) break;
        if (ws && w.u.j0 == 0 && w.u.j1 < w.u.nb) {
          left = true;
          seq_leave_note<128, C::NACC * D>(ws, blockIdx.x, w.u, DKV ? w.u.kv_begin : w.u.q_begin, a.tile,
                                           DKV ? 1 : group, place.per, false);
        }
        w.advance(a);
      }
      if (ws && !left) seq_leave_note<128, C::NACC * D>(ws, blockIdx.x, w.u, 0, a.tile, 1, place.per, true);
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0, sb = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      SeqUnit u;
      const int per_tile = DKV ? 128 : a.tile / group, per_block = DKV ? a.block / group : a.block;  // tokens
      while (ok && unit_take(u)) {
        const int j1 = real_end(u);
        if (u.j0 < j1) {
          ok = seq_wait(&a_empty[sb], aph ^ 1u, status);
          if (ok) {
            mbar_arrive_expect_tx(&a_full[sb], static_cast<uint32_t>(2 * a.tile * D * 2));
            const int h = DKV ? u.h : u.h * group;
            const int r = static_cast<int>(DKV ? u.kv_begin : u.q_begin) + u.t * per_tile;
#pragma unroll
            for (int bx = 0; bx < C::NBOX; ++bx) {
              tma_load_3d(&tmA1, &a_full[sb], sA + (2 * sb) * C::AB + bx * C::ABOXB, bx * C::BW, h, r);
              tma_load_3d(&tmA2, &a_full[sb], sA + (2 * sb + 1) * C::AB + bx * C::ABOXB, bx * C::BW, h, r);
            }
            if (++sb == C::SBUF) {
              sb = 0;
              aph ^= 1u;
            }
          }
          for (int j = u.j0; ok && j < j1; ++j) {
            ok = seq_wait(&y_empty[s], ph ^ 1u, status);
            if (!ok) break;
            mbar_arrive_expect_tx(&y_full[s], static_cast<uint32_t>(2 * a.block * D * 2));
            const int h = DKV ? u.h * group : u.h;
            const int r = static_cast<int>(DKV ? u.q_begin : u.kv_begin) + j * per_block;
#pragma unroll
            for (int bx = 0; bx < C::NBOX; ++bx) {
              tma_load_3d(&tmY1, &y_full[s], sY + (2 * s) * C::YBYTES + bx * C::YBOXB, bx * C::BW, h, r);
              tma_load_3d(&tmY2, &y_full[s], sY + (2 * s + 1) * C::YBYTES + bx * C::YBOXB, bx * C::BW, h, r);
            }
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        unit_done();
        ++ui;
      }
      // copies already issued must land before the block exits (a failed wait left some behind)
      if (status_set(status)) {
        for (int i = 0; i < C::STAGES; ++i) mbar_drain(&y_full[i], ph ^ (i < s ? 0u : 1u), status);
        for (int i = 0; i < C::SBUF; ++i) mbar_drain(&a_full[i], aph ^ (i < sb ? 0u : 1u), status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // T1 and T2 are written over places that P and dS of earlier blocks were read from; the MMAs of a
    // thread run in issue order, so they only have to be issued after those.
    const bool bf = Half16<T>::kBF16;
    const uint32_t idT = idesc_f16kind_f32(C::R, C::YB, 0, 0, bf);
    const uint32_t idA = idesc_f16kind_f32(C::R, D, 0, 1, bf);
    int ts = 0, as = 0, sb = 0;   // ring places of the next T block, of the next accumulation; standing tiles
    uint32_t tph = 0, aph = 0, g = 0, uc = 0;
    bool ok = true;
    SeqUnit u;
    // the block in ring place ts: T1 (w = 0, the first to need it) and T2 (w = 1, the last)
    auto issue_t = [&](int w, int j, uint32_t gb) -> bool {
      if (w == 0) {
        if (!seq_wait(&y_full[ts], tph, status)) return false;
        const int valid = min(a.block, passing(u) - j * a.block);
        if (valid < C::YB) {
          constexpr int UR = C::SWB / 16;  // 16-byte units of a box row
          for (int i = lane; i < (C::YB - valid) * 2 * C::NBOX * UR; i += 32) {
            const int r = valid + i / (2 * C::NBOX * UR), x = i % (2 * C::NBOX * UR);
            *reinterpret_cast<uint4*>(sY + 2 * ts * C::YBYTES + (x / UR) * C::YBOXB + r * C::SWB + (x % UR) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (elect_one()) {
        tc_fence_after();
        const uint32_t x = seq_desc_lo(smem_u32(sA + (2 * sb + w) * C::AB), 16);
        const uint32_t y = seq_desc_lo(smem_u32(sY + (2 * ts + w) * C::YBYTES), 16);
        const uint32_t t = tmem + (w ? C::t2(gb) : C::t1(gb));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int bx = ks / (C::BW / 16), kin = ks % (C::BW / 16);
          seq_mma_ss<C::DESC_HI>(t, x + ((bx * C::ABOXB + kin * 32) >> 4), y + ((bx * C::YBOXB + kin * 32) >> 4), idT,
                                 ks != 0 ? 1u : 0u);
        }
        if (w) umma_commit(&t_full[gb & 1u]);
      }
      __syncwarp();
      if (w && ++ts == C::STAGES) {
        ts = 0;
        tph ^= 1u;
      }
      return true;
    };
    auto issue_acc = [&](uint32_t gb, bool first) -> bool {
      if (!seq_wait(&p_full[gb & 1u], (gb >> 1) & 1u, status)) return false;
      if (elect_one()) {
        tc_fence_after();
        const uint32_t y = seq_desc_lo(smem_u32(sY + 2 * as * C::YBYTES), C::YBOXB);  // MN-major
        const uint32_t p = tmem + C::t1(gb), ds = tmem + C::t2(gb);
        // columns 16 ks .. + 15 of P (dS): 8 TMEM columns, each 32 behind the first of T's own 32
#pragma unroll
        for (int ks = 0; ks < C::YB / 16; ++ks) {
          const uint32_t at = (ks / 2) * 32 + (ks % 2) * 8, yk = y + ((ks * 16 * C::SWB) >> 4);
          if constexpr (DKV)  // dV += P^T dO
            seq_mma_ts<C::DESC_HI>(tmem + C::ACOL + D, p + at, yk + (C::YBYTES >> 4), idA, (!first || ks) ? 1u : 0u);
          seq_mma_ts<C::DESC_HI>(tmem + C::ACOL, ds + at, yk, idA, (!first || ks) ? 1u : 0u);  // dQ, dK
        }
        umma_commit(&y_empty[as]);
      }
      __syncwarp();
      if (++as == C::STAGES) as = 0;
      return true;
    };
    while (ok && unit_take(u)) {
      const int j1 = real_end(u);
      if (u.j0 < j1) {
        ok = seq_wait(&a_full[sb], aph, status);
        auto t_next = [&](int w, int j, uint32_t gb) {
          if (!issue_t(w, j, gb)) return false;
          if (w && j + 1 == j1 && elect_one()) umma_commit(&a_empty[sb]);
          __syncwarp();
          return true;
        };
        if (ok) ok = t_next(0, u.j0, g);
        if (ok) ok = t_next(1, u.j0, g);
        for (int j = u.j0; ok && j < j1; ++j) {
          if (j + 1 < j1) ok = t_next(0, j + 1, g + 1u);
          if (C::SLOTS == 4 && ok && j + 1 < j1) ok = t_next(1, j + 1, g + 1u);
          if (ok && j == u.j0 && uc > 0) ok = seq_wait(acc_empty, (uc - 1u) & 1u, status);
          if (ok) ok = issue_acc(g, j == u.j0);
          if (C::SLOTS == 3 && ok && j + 1 < j1) ok = t_next(1, j + 1, g + 1u);
          ++g;
        }
        if (ok && elect_one()) umma_commit(acc_full);
        __syncwarp();
        ++uc;
        if (++sb == C::SBUF) {
          sb = 0;
          aph ^= 1u;
        }
      }
      __syncwarp();
      if (lane == 0) unit_done();
      ++ui;
    }
    __syncwarp();
    if (elect_one()) {
      umma_commit(fin);  // no MMA may still write TMEM when it is freed
      mbar_drain(fin, 0u, status);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- element-wise
    const int q = warp & 3;
    const int half = (warp - 4) >> 2;
    const int row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const int bar_id = 1 + q;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    constexpr float UP = SbP<T>::LOG2;
    uint8_t* stage = reinterpret_cast<uint8_t*>(red) + C::REDB + (warp - 4) * SEQ_STAGE_BYTES;
    float* cols = red + (warp - 4) * 128;  // DKV: lse (base 2) [32] and delta [32] of this warp's columns, twice
    uint32_t g = 0, uc = 0;
    bool ok = true;
    int64_t high_at = -1;  // fp16: the (sequence, key head) whose largest norms `high` holds
    float high = 0.f;
    SeqUnit u;
    for (;;) {
      const bool got = ok && unit_take(u);
      if (!named_bar_and(bar_id, 64, got)) break;
      __syncwarp();
      const int j1 = real_end(u);
      const int r = u.t * a.tile + row;
      const bool row_on = row < a.tile && r < u.rows;
      const bool warp_on = q * 32 < a.tile && u.t * a.tile + q * 32 < u.rows;
      const bool whole = u.j0 == 0 && u.j1 == u.nb;
      // the row of the output (and, for DQ, of lse and delta)
      const int64_t orow = !row_on ? 0
                           : DKV   ? (u.kv_begin + r) * a.kv_heads + u.h
                                   : (u.q_begin + r / group) * a.q_heads + u.h * group + r % group;
      if (u.j0 < j1) {
        // dS goes into its product times ds_in, the sums come out times ds_out
        float ds_in = a.scale, ds_out = 1.f;
        float lse2 = 0.f, dl = 0.f;
        if constexpr (!Half16<T>::kBF16) {
          const int64_t at = static_cast<int64_t>(u.b) * a.kv_heads + u.h;
          if (at != high_at) {
            high_at = at;
            high = seq_chunks_max(range.v, u.kv_begin, u.b, u.len, a.kv_heads, u.h);
            if constexpr (DKV) high *= seq_chunks_max(range.g, u.q_begin, u.b, u.n, a.kv_heads, u.h);
          }
          const int k = seq_range_log2(DKV ? high : high * (row_on ? __ldg(range.rows + orow) : 0.f));
          ds_in = seq_exp2i(k - (DKV ? SbP<T>::LOG2 : 0));
          ds_out = a.scale * seq_exp2i(-k);
        }
        const bool one = !DKV && u.nb == 1;  // every key in one block
        if constexpr (!DKV) {
          if (row_on) lse2 = __ldg(lse + orow) * 1.4426950408889634f;
          if (!one) {
            // four lanes to a row, 16 rows to each warp of the pair: 64 bytes of 8 rows per load
#pragma unroll
            for (int it = 0; it < 2; ++it) {
              const int rr = q * 32 + half * 16 + it * 8 + (lane >> 2), r2 = u.t * a.tile + rr;
              const bool on = rr < a.tile && r2 < u.rows;
              const int64_t at = on ? (u.q_begin + r2 / group) * a.q_heads + u.h * group + r2 % group : 0;
              float x = 0.f;
              if (on) {
                const uint4* po = reinterpret_cast<const uint4*>(O + at * D) + (lane & 3);
                const uint4* pg = reinterpret_cast<const uint4*>(dO + at * D) + (lane & 3);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                  const uint4 y = __ldg(po + 4 * i), z = __ldg(pg + 4 * i);
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t yy = reinterpret_cast<const uint32_t*>(&y)[k],
                                   zz = reinterpret_cast<const uint32_t*>(&z)[k];
                    x = fmaf(Half16<T>::lo(yy), Half16<T>::lo(zz), x);
                    x = fmaf(Half16<T>::hi(yy), Half16<T>::hi(zz), x);
                  }
                }
              }
              x += __shfl_xor_sync(0xffffffffu, x, 1);
              x += __shfl_xor_sync(0xffffffffu, x, 2);
              if ((lane & 3) == 0) {
                red[rr] = x;
                if (on) delta[at] = x;
              }
            }
            named_bar(bar_id, 64);
            dl = red[row];
          }
        }
        // DKV: lse and delta of block j's columns, one per lane
        auto fetch = [&](int j, float& cl, float& cd) {
          const int c = half * 32 + lane, pr = j * a.block + c;
          cl = INFINITY;
          cd = 0.f;
          if (c < a.block && pr < u.n * group) {
            const int64_t at = (u.q_begin + pr / group) * a.q_heads + u.h * group + pr % group;
            cl = __ldg(lse + at) * 1.4426950408889634f;
            cd = __ldg(delta + at);
          }
        };
        float cl = 0.f, cd = 0.f;
        if constexpr (DKV) fetch(u.j0, cl, cd);
        for (int j = u.j0; j < j1; ++j, ++g) {
          const uint32_t buf = g & 1u;
          float* cj = cols + (j & 1) * 64;
          if constexpr (DKV) {
            cj[lane] = cl;
            cj[32 + lane] = cd;
            __syncwarp();
            if (j + 1 < j1) fetch(j + 1, cl, cd);
          }
          if (ok) ok = seq_wait(&t_full[buf], (g >> 1) & 1u, status);
          tc_fence_after();
          const uint32_t ta = tmem + lane_base + C::t1(g) + half * (C::YB / 2);
          const uint32_t tb = tmem + lane_base + C::t2(g) + half * (C::YB / 2);
          uint32_t t1[32], t2[32];
          auto load = [&](int at) {
            if (warp_on) {
              tmem_ld32(ta + at, t1);
              tmem_ld32(tb + at, t2);
              tmem_ld_wait();
            }
          };
          if constexpr (DKV) {
            load(0);
            uint32_t pp[16], ds[16];
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
              const float4 l4 = *reinterpret_cast<const float4*>(cj + 4 * c4);
              const float4 d4 = *reinterpret_cast<const float4*>(cj + 32 + 4 * c4);
              const float lv[4] = {l4.x, l4.y, l4.z, l4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w};
              float p[4], s[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                p[e] = seq_ex2(fmaf(__uint_as_float(t1[4 * c4 + e]), scale_log2, UP - lv[e]));
                s[e] = p[e] * ((__uint_as_float(t2[4 * c4 + e]) - dv[e]) * ds_in);
              }
              pp[2 * c4] = Half16<T>::pack2(p[0], p[1]);
              pp[2 * c4 + 1] = Half16<T>::pack2(p[2], p[3]);
              ds[2 * c4] = Half16<T>::pack2(s[0], s[1]);
              ds[2 * c4 + 1] = Half16<T>::pack2(s[2], s[3]);
            }
            if (warp_on) {  // over the columns of T1 and T2 that this thread read
              whale_tmem_st_cols<16>(ta, pp);
              whale_tmem_st_cols<16>(tb, ds);
            }
          } else {
            // P over t1; keys behind the sequence's end count for nothing
            auto weights = [&](int at) {
              const int valid = u.len - j * a.block - half * (C::YB / 2) - at;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                t1[c] = __float_as_uint(seq_ex2(fmaf(__uint_as_float(t1[c]), scale_log2, -lse2)));
              if (valid < 32) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (c >= valid) t1[c] = t2[c] = 0u;
              }
            };
            if (one) {
              float x = 0.f;
#pragma unroll 1
              for (int at = 0; at < C::YB / 2; at += 32) {
                load(at);
                weights(at);
#pragma unroll
                for (int c = 0; c < 32; ++c) x = fmaf(__uint_as_float(t1[c]), __uint_as_float(t2[c]), x);
              }
              red[half * 128 + row] = x;
              named_bar(bar_id, 64);
              dl = x + red[(half ^ 1) * 128 + row];
              if (row_on && half == 0) delta[orow] = dl;
            }
#pragma unroll 1
            for (int at = 0; at < C::YB / 2; at += 32) {
              load(at);
              weights(at);
              uint32_t ds[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float s0 = __uint_as_float(t1[2 * c]) * ((__uint_as_float(t2[2 * c]) - dl) * ds_in);
                const float s1 = __uint_as_float(t1[2 * c + 1]) * ((__uint_as_float(t2[2 * c + 1]) - dl) * ds_in);
                ds[c] = Half16<T>::pack2(s0, s1);
              }
              if (warp_on) whale_tmem_st_cols<16>(tb + at, ds);
            }
          }
          whale_tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        if (ok) ok = seq_wait(acc_full, uc & 1u, status);
        tc_fence_after();
        ++uc;
        if (warp_on) {
          const SeqRowsOut out(orow, row_on && ok);
          float* slot = whole ? nullptr : S::slot(ws, pieces, blockIdx.x, u.j0 > 0);
#pragma unroll 1
          for (int cc = half; cc < C::NACC * (D / 32); cc += 2) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + C::ACOL + cc * 32, o);
            tmem_ld_wait();
            const float f = cc < D / 32 ? ds_out : 1.f / SbP<T>::ONE;
            if (whole) {
              seq_store_rows<D, T>(stage, o, f, cc < D / 32 ? G1 : G2, (cc % (D / 32)) * 32, out);
            } else if (row_on && ok) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(S::o(slot, row, cc * 32 + 4 * i)) =
                    make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      } else if (row_on) {  // nothing goes by: the gradients are 0
        const uint32_t z[32] = {};
#pragma unroll 1
        for (int cc = half; cc < C::NACC * (D / 32); cc += 2)
          whale_st_row32<T>((cc < D / 32 ? G1 : G2) + orow * D + (cc % (D / 32)) * 32, z, 0.f, nullptr);
      }
      __syncwarp();
      if (lane == 0) unit_done();
      ++ui;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the pieces of cut units, in the order of the pieces (as seq_combine_kernel); the first D
// columns go to G1, the others to G2.
template <int CR, int D, int NACC, typename T>
__global__ void __launch_bounds__(CR * NACC * D / 8)
    seq_sum_kernel(float* ws, T* __restrict__ G1, T* __restrict__ G2, int32_t heads, int32_t pieces) {
  using S = SeqSlots<128, NACC * D>;
  const int32_t c = blockIdx.x / (128 / CR);
  const int r = (blockIdx.x % (128 / CR)) * CR + threadIdx.x % CR, d = (threadIdx.x / CR) * 8;
  seq_wait_before();
  const SeqNote n = *S::note(ws, c);
  if (r >= n.rows) return;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < n.pieces; ++k) {
    float* s = S::slot(ws, pieces, c + k, k != 0);
    const float4 x = *reinterpret_cast<const float4*>(S::o(s, r, d));
    const float4 y = *reinterpret_cast<const float4*>(S::o(s, r, d + 4));
    o[0] += x.x;
    o[1] += x.y;
    o[2] += x.z;
    o[3] += x.w;
    o[4] += y.x;
    o[5] += y.y;
    o[6] += y.z;
    o[7] += y.w;
  }
  const int pr = n.r0 + r;
  const int64_t row = (n.begin + pr / n.group) * heads + n.h * n.group + pr % n.group;
  T* dst = (d < D ? G1 : G2) + row * D + d % D;
  *reinterpret_cast<uint4*>(dst) = make_uint4(Half16<T>::pack2(o[0], o[1]), Half16<T>::pack2(o[2], o[3]),
                                              Half16<T>::pack2(o[4], o[5]), Half16<T>::pack2(o[6], o[7]));
}

// Zeros in the rows between a sequence's last key and the next sequence (padded batches). Block
// (b, K or V, z) takes each gridDim.z-th run of the sequence: one block alone is slow (the gradients
// of 4 sequences of up to 1,600 keys padded to 8,192, d = 128, took 92 us with one and take 31 with
// 64; of 64 sequences of up to 2,048, 108 and 103).
template <typename T>
__global__ void seq_zero_padding_kernel(T* __restrict__ dK, T* __restrict__ dV, int64_t row_elems, SeqArgs a) {
  seq_wait_before();
  const SeqSpan kv = seq_keys<SEQ_JAGGED>(a, blockIdx.x);
  const int64_t at = (kv.begin + kv.len) * row_elems / 8;
  const int64_t n = static_cast<int64_t>(kv.room - kv.len) * row_elems / 8;
  uint4* g = reinterpret_cast<uint4*>(blockIdx.y ? dV : dK) + at;
  for (int64_t i = static_cast<int64_t>(blockIdx.z) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.z) * blockDim.x)
    g[i] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace wk
