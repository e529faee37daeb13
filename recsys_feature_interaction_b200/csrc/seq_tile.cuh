// seq_tile.cuh -- attention of more than 16 packed query rows per (sequence, key head) on the
// 5th-generation tensor cores, over jagged tensors or a cache.
//
// A block holds up to 128 packed query rows (whole tokens of the query heads that share a key head)
// and walks 128-key blocks: S = Q K^T from shared memory, softmax weights from TMEM by two groups of
// four warps that take the blocks in turn, P written over S's columns, O += P V with the V tile
// MN-major. S has two or three buffers and runs one or two blocks ahead of P V; K and V tiles arrive
// in one ring in the order in which the products use them (K0, K1, V0, K2, V1, ..).
//
// Roles: warp 0 loads tiles with TMA (jagged: 128 rows from the sequence's first; a 16-bit cache:
// one box per page, each by the lane that holds its number); warp 1 issues the MMAs; warp 2 walks the
// block's units and hands them to the other roles through a ring, so that none of them waits for
// offsets; warps 4 .. 11 run the softmax; for an 8-bit cache warps 12 .. 15 load rows, convert them
// to the 16-bit type and store them in the tiles' swizzled layout, in place of the TMA.
//
// Powers of two of 8-bit rows. bf16 has room for every one, so its tiles hold the rows' values. fp16
// has not: its tiles hold the e4m3 values, K's power is a factor of the fp32 score, and V's is added to
// the exponent of the weight, P = 2^(S + x - w) with w the running maximum of S + x over the keys that
// the row sees, beside the row sum of 2^(S - m). So a row's share does not depend on what other rows
// hold, seen or not. (With rows relative to the largest of the piece, those 2^22 below it lost bits.)
// The second exponential costs less than the simpler conversion saves: chunks of 200 .. 512 tokens over
// up to 4096 keys (d = 128, 8 heads on 2) take 143 us in fp16, 147 in bf16.
//
// Rows behind a sequence's last key belong to someone else: their scores are replaced by a select,
// and their V rows, whose weights are 0, are overwritten with zeros in the tile before P V, because
// 0 * NaN is NaN.
//
// The running maximum is raised only when a block exceeds it by more than 2^8; one weight in four
// comes from a polynomial on the FMA pipe (whale.cuh).
#pragma once

#include "seq_args.cuh"
#include "seq_rows.cuh"
#include "whale.cuh"

namespace wk {

// Barrier over `count` threads that also tells every one of them whether `p` held for all.
__device__ __forceinline__ bool named_bar_and(int id, int count, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0u;
}

// Arrives at a barrier over `count` threads without waiting.
__device__ __forceinline__ void named_bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// 32 TMEM lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// True for one thread of a converged warp, always the same one. The MMAs of a warp that runs as a
// whole are issued under it: with a plain lane == 0 the compiler does not know that one thread is
// left, and the tensor pipe falls behind when the softmax warps keep the issue slots busy (18 MMAs
// of a block next to a softmax loop: 1630 cycles against 2240, 1306 with the SM to themselves).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}

// Shared-memory descriptors (see smem_desc) in two words: the upper one is a constant of the layout,
// the lower one moves with the address by additions. With the whole descriptor rebuilt for each MMA
// the issuing thread, which shares its scheduler with the softmax warps, falls behind the tensor pipe
// (18 MMAs of a block next to a softmax loop: 1680 cycles, so 1424).
constexpr uint32_t seq_desc_hi(uint32_t sbo_bytes, uint32_t swizzle_mode) {
  return (sbo_bytes >> 4) | (1u << 14) | (swizzle_mode << 29);
}
__device__ __forceinline__ uint32_t seq_desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return (saddr >> 4) | ((lbo_bytes >> 4) << 16);
}

// D[tmem] (+)= A B^T, kind::f16, operands in shared memory, or A in TMEM.
template <uint32_t HI>
__device__ __forceinline__ void seq_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "n"(HI)
      : "memory");
}
template <uint32_t HI>
__device__ __forceinline__ void seq_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(add), "n"(HI)
      : "memory");
}

// Two e4m3 values times a power of two as a pair of bf16, which holds every such product; NaN stays NaN.
__device__ __forceinline__ uint32_t seq_e4m3_bf16(uint16_t w, float f) {
  const uint32_t h = seq_e4m3_f16(w);
  return pack_bf16x2(Half16<__half>::lo(h) * f, Half16<__half>::hi(h) * f);
}

// max(a, b, c) and max(a, b) that give NaN if an operand is NaN.
__device__ __forceinline__ float seq_max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float seq_max2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 seq_fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 seq_add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// 2^x of two values on the FMA pipe (see whale_ex2_poly), with a floor whose result rounds to 0 in
// both 16-bit types, so that a masked score (-inf) gets a weight of exactly 0: at x = -126.9997 the
// integer part is -127 and the polynomial just above 1, so that adding -127 to its exponent leaves
// a subnormal below 2^-139.
__device__ __forceinline__ float2 seq_ex2_poly(float2 x) {
  const float2 big = make_float2(12582912.f, 12582912.f), nbig = make_float2(-12582912.f, -12582912.f);
  x = make_float2(fmaxf(x.x, -126.9997f), fmaxf(x.y, -126.9997f));
  const float2 t = seq_add2(x, big);
  const float2 j = seq_add2(t, nbig);
  const float2 f = seq_add2(x, make_float2(-j.x, -j.y));
  float2 p = seq_fma2(make_float2(0.05517158f, 0.05517158f), f, make_float2(0.24261111f, 0.24261111f));
  p = seq_fma2(p, f, make_float2(0.69326103f, 0.69326103f));
  p = seq_fma2(p, f, make_float2(0.99992806f, 0.99992806f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

template <int N>
__device__ __forceinline__ float seq_max(const uint32_t (&v)[N]) {
  float t[(N + 2) / 3];
#pragma unroll
  for (int i = 0; i < N / 3; ++i)
    t[i] = seq_max3(__uint_as_float(v[3 * i]), __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
  if constexpr (N % 3 == 1) t[N / 3] = __uint_as_float(v[N - 1]);
  if constexpr (N % 3 == 2) t[N / 3] = seq_max2(__uint_as_float(v[N - 2]), __uint_as_float(v[N - 1]));
  constexpr int M = (N + 2) / 3;
  float a[4] = {t[0], t[1 % M], t[2 % M], t[3 % M]};
#pragma unroll
  for (int i = 4; i + 1 < M; i += 2) a[(i / 2) & 3] = seq_max3(a[(i / 2) & 3], t[i], t[i + 1]);
  if constexpr (M > 4 && M % 2 == 1) a[0] = seq_max2(a[0], t[M - 1]);
  return seq_max2(seq_max3(a[0], a[1], a[2]), a[3]);
}

// Where a warp's 32 accumulator rows go: a lane stores 16 bytes of rows 8 k + lane / 4, k < 4.
struct SeqRowsOut {
  int64_t at[4];
  bool on[4];
  // row, on: this lane's own row of the output
  __device__ __forceinline__ SeqRowsOut(int64_t row, bool valid) {
    const uint32_t all = __ballot_sync(0xffffffffu, valid);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int from = 8 * k + (lane >> 2);
      at[k] = __shfl_sync(0xffffffffu, row, from);
      on[k] = (all >> from) & 1u;
    }
  }
};
constexpr int SEQ_STAGE_BYTES = 32 * 64;  // per warp

// 32 columns of a warp's 32 rows, times scale, as T into out[row * D + col ..]: through a tile of the
// warp's own in shared memory, so that a store covers 64 bytes of 8 rows and not 16 of 32 (which
// keeps the load/store unit busy four times as long; it bounded the gradients of short sequences).
template <int D, typename T>
__device__ __forceinline__ void seq_store_rows(uint8_t* stage, const uint32_t (&o)[32], float scale, T* out, int col,
                                               const SeqRowsOut& w) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = Half16<T>::pack2(__uint_as_float(o[8 * j + 2 * i]) * scale, __uint_as_float(o[8 * j + 2 * i + 1]) * scale);
    *reinterpret_cast<uint4*>(stage + whale_swz<64>(lane, j)) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 v = *reinterpret_cast<const uint4*>(stage + whale_swz<64>(8 * k + (lane >> 2), lane & 3));
    if (w.on[k]) *reinterpret_cast<uint4*>(out + w.at[k] * D + col + (lane & 3) * 8) = v;
  }
  __syncwarp();
}

template <int D_, int SRC_>
struct StCfg {
  static constexpr int D = D_, SRC = SRC_;
  static constexpr int R = 128, KB = 128;
  static constexpr int BW = (D % 64 == 0) ? 64 : 32;     // columns per box
  static constexpr int SWB = BW * 2;                     // bytes per box row = swizzle span
  static constexpr uint32_t SWMODE = BW == 64 ? 2u : 4u;
  static constexpr uint32_t DESC_HI = seq_desc_hi(8 * SWB, SWMODE);
  static constexpr int NBOX = D / BW;
  static constexpr int BOXB = KB * SWB;
  static constexpr int TILEB = NBOX * BOXB;              // one K or V tile
  static constexpr int LIMIT = 227 * 1024;
  static constexpr int NU = 4;                           // units in flight between the walker and the roles
  static constexpr int BARB = 512;                       // barriers, TMEM address
  static constexpr int UNITB = NU * static_cast<int>(sizeof(SeqUnit));
  static constexpr int REDB = (SRC == SEQ_PAGED8 ? 6 : 4) * R * 4;  // what the softmax groups tell each other, per row
  static constexpr int STAGEB = 8 * SEQ_STAGE_BYTES;     // the softmax warps' output tiles
  // TMEM: NS buffers of S (P over their first 64 columns), then O. With three, S runs two blocks
  // ahead of P V, and a softmax group finds its next block ready; d = 160 has room for two.
  static constexpr int NS = D <= 128 ? 3 : 2;
  static constexpr int AHEAD = NS - 1;
  // Powers of two of a block's key and value rows (fp16 over an 8-bit cache), for NX blocks: written
  // with K's tile, read by the softmax warps. Between the tile of V of block g - NX and that of K of
  // block g the ring takes at least 2 (NX - AHEAD - 1) others, so a loader that has found room for the
  // latter knows that the former's product, and the softmax before it, are done.
  static constexpr int NX = AHEAD == 2 ? 8 : 4;
  static constexpr int COLB = SRC == SEQ_PAGED8 ? NX * 2 * KB * 4 : 0;
  static constexpr int FIXED = BARB + UNITB + REDB + STAGEB + COLB;
  // one Q tile: the next unit's is loaded once this one's last S is done, under its last blocks
  static constexpr int STAGES_RAW = (LIMIT - FIXED - TILEB) / TILEB;
  static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
  // more than half an SM's shared memory: one block per SM, whose 512 TMEM columns are its own
  static constexpr int RAW = FIXED + (1 + STAGES) * TILEB;
  static constexpr int SMEM = RAW > 120 * 1024 ? RAW : 120 * 1024;
  static constexpr int OCOL = NS * KB;
  static constexpr int THREADS = SRC == SEQ_PAGED8 ? 512 : 384;
  static constexpr int LOADERS = 128;
  static_assert(OCOL + D <= 512 && STAGES >= 4 && TILEB % 1024 == 0 && UNITB % 16 == 0, "layout");
  static_assert((2 * STAGES + 4 * NS + 2 + 2 + 2 * NU) * 8 + 16 <= BARB, "barriers");
  static_assert(2 * (NX - AHEAD - 1) + 1 >= STAGES, "powers of two are overwritten only after use");
};

// Key blocks [j0, j1) of a unit that hold keys (a unit without keys has a cost, but no block).
__device__ __forceinline__ int seq_real_end(const SeqArgs& a, const SeqUnit& u, int group, int R, int KB) {
  const int last = (min((u.t + 1) * R, u.rows) - 1) / group;
  return min(u.j1, (seq_seen(u.len, u.n, last, a.causal) + KB - 1) / KB);
}

template <int D, typename T, int SRC>
__global__ void __launch_bounds__(StCfg<D, SRC>::THREADS, 1)
    seq_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const void* __restrict__ K8, const void* __restrict__ V8,
                    T* __restrict__ O, float* __restrict__ lse, float* __restrict__ ws, SeqArgs a, int64_t pieces) {
  using C = StCfg<D, SRC>;
  constexpr int R = C::R, KB = C::KB;
  // fp16 over an 8-bit cache: fp16 cannot hold every power of two, so the tiles hold the e4m3 values
  // and the rows' powers join the fp32 scores (K) and the exponents of the weights (V). bf16 tiles
  // hold the rows' values themselves.
  constexpr bool FAR = SRC == SEQ_PAGED8 && !Half16<T>::kBF16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0u) {  // the swizzled layout needs 1024-byte alignment
    if (threadIdx.x == 0) flag_error(a.status, kFlagBadShape);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* tiles = sQ + C::TILEB;                      // [STAGES]
  uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + C::STAGES * C::TILEB);
  uint64_t* kv_full = bars;                  // [STAGES] tile landed
  uint64_t* kv_empty = bars + C::STAGES;     // [STAGES] its product has read it
  uint64_t* s_full = bars + 2 * C::STAGES;   // [NS] S in TMEM
  uint64_t* p_full = s_full + C::NS;         // [NS][2] the halves of P in TMEM
  uint64_t* p_empty = p_full + 2 * C::NS;    // [NS] P V has read it (so O holds that block)
  uint64_t* o_empty = p_empty + C::NS;       // O read by the softmax warps (per unit)
  uint64_t* fin = o_empty + 1;
  uint64_t* q_full = fin + 1;                // the unit's Q rows landed
  uint64_t* q_empty = q_full + 1;            // its last S has read them
  uint64_t* u_full = q_empty + 1;            // [NU] unit handed over
  uint64_t* u_empty = u_full + C::NU;        // [NU] every role is done with it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(u_empty + C::NU);
  SeqUnit* unit = reinterpret_cast<SeqUnit*>(tiles + C::STAGES * C::TILEB + C::BARB);
  float* red = reinterpret_cast<float*>(tiles + C::STAGES * C::TILEB + C::BARB + C::UNITB);
  float* columns = red + (C::REDB + C::STAGEB) / 4;      // [NX][2][KB] a block's powers of two
  unsigned* status = a.status;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmQ);
    if (SRC != SEQ_PAGED8) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&kv_full[s], SRC == SEQ_PAGED8 ? C::LOADERS / 32 : 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, 8);
    mbar_init(fin, 1);
    for (int i = 0; i < C::NU; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 10 + (SRC == SEQ_PAGED8 ? C::LOADERS / 32 : 0));
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
  const SeqPlace place = seq_place<SeqPlan<0, KB, SRC>, C::THREADS>(a, blockIdx.x, pieces, reinterpret_cast<int64_t*>(red), blockIdx.x == 0);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int group = a.q_heads / a.kv_heads;

  // The roles' side of the unit ring: the next unit, or false behind the last (b < 0).
  uint32_t ui = 0;
  auto unit_take = [&](SeqUnit& u) -> bool {
    const uint32_t s = ui % C::NU;
    if (!seq_wait(&u_full[s], (ui / C::NU) & 1u, status)) return false;
    u = unit[s];
    return u.b >= 0;
  };
  auto unit_done = [&]() {  // by one thread per warp
    mbar_arrive(&u_empty[ui % C::NU]);
  };

  if (warp == 2) {
    // -------------------------------------------------------------- walker
    if (lane == 0) {
      SeqWalk<SeqPlan<0, KB, SRC>> w;
      w.start(a, place);
      bool left = false;  // a unit left unfinished
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
          seq_leave_note<R, D>(ws, blockIdx.x, w.u, w.u.q_begin, a.tile, group, place.per, false);
        }
        w.advance(a);
      }
      if (ws && !left) seq_leave_note<R, D>(ws, blockIdx.x, w.u, 0, a.tile, 1, place.per, true);
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp walks, one thread issues. With a cache each lane holds one page of a window of
    // 32, one for K and one for V (K runs ahead), so that a tile does not wait for its table entries.
    int s = 0;
    uint32_t ph = 0, qph = 0;
    bool ok = true;
    SeqUnit u;
    const int tokens = a.tile / group;  // per Q tile: its rows are (token, head) with the head first
    auto load_q = [&]() -> bool {
      if (!seq_wait(q_empty, qph ^ 1u, status)) return false;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(a.tile * D * 2));
#pragma unroll
        for (int bx = 0; bx < C::NBOX; ++bx)
          tma_load_3d(&tmQ, q_full, sQ + bx * C::BOXB, bx * C::BW, u.h * group,
                      static_cast<int32_t>(u.q_begin) + u.t * tokens);
      }
      __syncwarp();
      qph ^= 1u;
      return true;
    };
    int win[2] = {-1, -1};    // the windows' numbers (page index / 32) and this lane's page of each
    int32_t held[2] = {-1, -1};
    auto load = [&](const CUtensorMap* tm, int which, int j) -> bool {
      const int ps = 1 << a.page_shift, per = KB >> a.page_shift;  // keys of a page, pages of a tile
      int np = 0, first = 0;
      if constexpr (SRC == SEQ_PAGED16) {
        np = (min(KB, u.len - j * KB) + ps - 1) >> a.page_shift;
        first = j * per;  // a tile's pages lie in one window
        if (win[which] != first >> 5) {
          win[which] = first >> 5;
          const int64_t pos = (static_cast<int64_t>(win[which]) * 32 + lane) << a.page_shift;
          held[which] = -1;
          if (pos < u.len) {
            held[which] = seq_page(a.table + static_cast<int64_t>(u.b) * a.table_width, pos, a.page_shift, a.num_pages);
            if (held[which] < 0) flag_error(status, kFlagBadShape);
          }
        }
      }
      if (!seq_wait(&kv_empty[s], ph ^ 1u, status)) return false;
      uint8_t* dst = tiles + s * C::TILEB;
      if constexpr (SRC == SEQ_JAGGED) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&kv_full[s], static_cast<uint32_t>(C::TILEB));
#pragma unroll
          for (int bx = 0; bx < C::NBOX; ++bx)
            tma_load_3d(tm, &kv_full[s], dst + bx * C::BOXB, bx * C::BW, u.h, static_cast<int32_t>(u.kv_begin) + j * KB);
        }
      } else {
        const bool mine = lane >= (first & 31) && lane < (first & 31) + np;
        const int good = __popc(__ballot_sync(0xffffffffu, mine && held[which] >= 0));
        if (elect_one()) mbar_arrive_expect_tx(&kv_full[s], static_cast<uint32_t>(good * ps * D * 2));
        __syncwarp();
        if (mine && held[which] >= 0) {  // the lane that holds a page loads it
          const int32_t r =
              static_cast<int32_t>((static_cast<int64_t>(held[which]) * a.kv_heads + u.h) << a.page_shift);
#pragma unroll
          for (int bx = 0; bx < C::NBOX; ++bx)
            tma_load_2d(tm, &kv_full[s], dst + bx * C::BOXB + (lane - (first & 31)) * ps * C::SWB, bx * C::BW, r);
        }
      }
      __syncwarp();
      if (++s == C::STAGES) {
        s = 0;
        ph ^= 1u;
      }
      return true;
    };
    while (ok && unit_take(u)) {
      const int j1 = seq_real_end(a, u, group, a.tile, KB);
      if (u.j0 < j1) ok = load_q();
      if constexpr (SRC != SEQ_PAGED8) {
        win[0] = win[1] = -1;
        for (int j = u.j0; ok && j < j1; ++j) {
          for (int k = u.j0; ok && j == u.j0 && k < min(j1, u.j0 + C::AHEAD); ++k) ok = load(&tmK, 0, k);
          if (ok && j + C::AHEAD < j1) ok = load(&tmK, 0, j + C::AHEAD);
          if (ok) ok = load(&tmV, 1, j);
        }
      }
      __syncwarp();
      if (lane == 0) unit_done();
      ++ui;
    }
    // copies already issued must land before the block exits (a failed wait left some behind)
    if (lane == 0 && status_set(status)) {
      mbar_drain(q_full, qph ^ 1u, status);
      if (SRC != SEQ_PAGED8)
        for (int i = 0; i < C::STAGES; ++i) mbar_drain(&kv_full[i], ph ^ (i < s ? 0u : 1u), status);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks; one thread issues. The MMAs of a thread run in issue order, so S of block
    // j + NS is written into S_j's columns only after P V_j, issued before it, has read P_j there.
    const bool bf = Half16<T>::kBF16;
    const uint32_t idS = idesc_f16kind_f32(R, KB, 0, 0, bf);
    const uint32_t idO = idesc_f16kind_f32(R, D, 0, 1, bf);
    int s = 0;
    uint32_t ph = 0, g = 0, uc = 0;
    bool ok = true;
    SeqUnit u;
    auto step = [&]() {
      if (++s == C::STAGES) {
        s = 0;
        ph ^= 1u;
      }
    };
    auto issue_s = [&](uint32_t gb, bool last) -> bool {
      if (!seq_wait(&kv_full[s], ph, status)) return false;
      if (elect_one()) {
        tc_fence_after();
        const uint32_t k = seq_desc_lo(smem_u32(tiles + s * C::TILEB), 16);
        const uint32_t qd = seq_desc_lo(smem_u32(sQ), 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = ((ks / (C::BW / 16)) * C::BOXB + (ks % (C::BW / 16)) * 32) >> 4;
          seq_mma_ss<C::DESC_HI>(tmem + (gb % C::NS) * KB, qd + at, k + at, idS, ks != 0 ? 1u : 0u);
        }
        umma_commit(&s_full[gb % C::NS]);
        umma_commit(&kv_empty[s]);
        if (last) umma_commit(q_empty);
      }
      __syncwarp();
      step();
      return true;
    };
    auto issue_pv = [&](int j, bool last, uint32_t gj, bool first) -> bool {
      if (!seq_wait(&kv_full[s], ph, status)) return false;
      // MN-major V: BW-column atoms BOXB apart, 8-key groups 8 * SWB apart
      const uint32_t v = seq_desc_lo(smem_u32(tiles + s * C::TILEB), C::BOXB);
      const int valid = u.len - j * KB;
      if (SRC != SEQ_PAGED8 && last && valid < KB) {  // rows behind the sequence: their weights are 0
        for (int i = lane; i < (KB - valid) * C::NBOX * (C::SWB / 16); i += 32) {
          const int r = valid + i / (C::NBOX * (C::SWB / 16)), x = i % (C::NBOX * (C::SWB / 16));
          uint8_t* p = tiles + s * C::TILEB + (x / (C::SWB / 16)) * C::BOXB + r * C::SWB + (x % (C::SWB / 16)) * 16;
          *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t buf = gj % C::NS;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // the first half's product runs under the second's softmax
        if (!seq_wait(&p_full[2 * buf + half], (gj / C::NS) & 1u, status)) return false;
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int ks = half * KB / 32; ks < (half + 1) * KB / 32; ++ks) {
            seq_mma_ts<C::DESC_HI>(tmem + C::OCOL, tmem + buf * KB + ks * 8, v + ((ks * 16 * C::SWB) >> 4), idO,
                                   (!first || ks) ? 1u : 0u);
          }
        }
        __syncwarp();
      }
      if (elect_one()) {
        umma_commit(&p_empty[buf]);
        umma_commit(&kv_empty[s]);
      }
      __syncwarp();
      step();
      return true;
    };
    while (ok && unit_take(u)) {
      const int j1 = seq_real_end(a, u, group, a.tile, KB);
      if (u.j0 < j1) {
        ok = seq_wait(q_full, uc & 1u, status);
        for (int k = 0; ok && k < min(C::AHEAD, j1 - u.j0); ++k) ok = issue_s(g + k, u.j0 + k + 1 == j1);
        for (int j = u.j0; ok && j < j1; ++j) {
          if (j + C::AHEAD < j1) ok = issue_s(g + C::AHEAD, j + C::AHEAD + 1 == j1);
          // O is free once the softmax warps have read the unit before
          if (ok && j == u.j0 && uc > 0) ok = seq_wait(o_empty, (uc - 1u) & 1u, status);
          if (ok) ok = issue_pv(j, j + 1 == j1, g, j == u.j0);
          ++g;
        }
        ++uc;
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
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------- softmax
    // Two groups of four warps take the blocks in turn; a thread has one row and all 128 keys of a
    // block. So the groups are half a block apart, and one's exponentials
    // run while the other waits for TMEM. What they share per row is the running maximum: a group
    // hands its decision on before it computes its weights (an arrive that does not wait), so the
    // other one finds it there.
    const int q = warp & 3;
    const int grp = (warp - 4) >> 2;
    const int row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const int pair_id = 1 + q, hear_id = 6 + q + 4 * (grp ^ 1), tell_id = 6 + q + 4 * grp;
    float* mrow = red;           // [2][R] running maximum after a group's last block
    float* lrow = red + 2 * R;   // [2][R] row sums at the end of a unit, relative to mrow
    float* wrow = red + 4 * R;   // [2][R] FAR: as mrow, of the scores plus V's exponents
    uint8_t* stage = reinterpret_cast<uint8_t*>(red) + C::REDB + (warp - 4) * SEQ_STAGE_BYTES;
    uint32_t g = 0;
    // After a failed wait a thread stops waiting but walks the unit to its end, so that the
    // warp-collective TMEM accesses and the barriers stay converged; the pair of warps of a lane
    // quarter leaves together.
    bool ok = true;
    SeqUnit u;
    for (;;) {
      const bool got = ok && unit_take(u);
      if (!named_bar_and(pair_id, 64, got)) break;
      __syncwarp();
      const int j1 = seq_real_end(a, u, group, a.tile, KB);
      const int r = u.t * a.tile + row;  // packed row of the sequence
      const bool warp_on = q * 32 < a.tile && u.t * a.tile + q * 32 < u.rows;
      const bool row_on = row < a.tile && r < u.rows;
      const int qi = row_on ? r / group : 0, qh = u.h * group + (row_on ? r % group : 0);
      const int seen = row_on ? seq_seen(u.len, u.n, qi, a.causal) : INT32_MAX;
      const bool whole = u.j0 == 0 && u.j1 == u.nb;
      const int64_t orow = (u.q_begin + qi) * a.q_heads + qh;
      if (u.j0 < j1) {
        float m = -INFINITY, l = 0.f;  // this group's row sum, relative to m
        float wm = -INFINITY;          // FAR: what the weights are relative to
        for (int j = u.j0; j < j1; ++j, ++g) {
          if ((g & 1u) != static_cast<uint32_t>(grp)) continue;
          const uint32_t buf = g % C::NS;
          if (ok) ok = seq_wait(&s_full[buf], (g / C::NS) & 1u, status);
          tc_fence_after();
          const float scale_log2 = FAR ? 1.f : a.scale * 1.4426950408889634f;  // FAR: part of K's factors
          const float* kfac = columns + (g % C::NX) * 2 * KB;
          const float* vexp = kfac + KB;
          // Half of the block's scores at a time: the second half's maximum, the first half's, then the
          // first half's weights, and the second half again (a whole row would not fit the registers).
          uint32_t sr[KB / 2];
          const uint32_t ta = tmem + lane_base + buf * KB;
          const int kvalid = seen - j * KB;  // this row's keys in the block
          const bool full = __all_sync(0xffffffffu, kvalid >= KB);
          auto load_half = [&](int at) {
            if (warp_on) {
              tmem_ld32(ta + at, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
              tmem_ld32(ta + at + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
              tmem_ld_wait();
            }
            if constexpr (FAR) {
#pragma unroll
              for (int c4 = 0; c4 < KB / 8; ++c4) {
                const float4 f = *reinterpret_cast<const float4*>(kfac + at + 4 * c4);
                const float fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  sr[4 * c4 + i] = __float_as_uint(__uint_as_float(sr[4 * c4 + i]) * fv[i]);
              }
            }
            if (!full) {
#pragma unroll
              for (int c = 0; c < KB / 2; ++c)
                if (at + c >= kvalid) sr[c] = 0xFF800000u;  // -inf
            }
          };
          float mh = -INFINITY, wh = -INFINITY;
#pragma unroll 1
          for (int at = KB / 2; at >= 0; at -= KB / 2) {
            load_half(at);
            mh = seq_max2(mh, seq_max<KB / 2>(sr));
            if constexpr (FAR) {
#pragma unroll
              for (int c4 = 0; c4 < KB / 8; ++c4) {
                const float4 x = *reinterpret_cast<const float4*>(vexp + at + 4 * c4);
                wh = seq_max3(wh, __uint_as_float(sr[4 * c4]) + x.x, __uint_as_float(sr[4 * c4 + 1]) + x.y);
                wh = seq_max3(wh, __uint_as_float(sr[4 * c4 + 2]) + x.z, __uint_as_float(sr[4 * c4 + 3]) + x.w);
              }
            }
          }
          float mprev = -INFINITY, wprev = -INFINITY;
          if (j > u.j0) {
            named_bar(hear_id, 64);
            mprev = mrow[(grp ^ 1) * R + row];
            if constexpr (FAR) wprev = wrow[(grp ^ 1) * R + row];
          }
          const float mb2 = mh * scale_log2;
          const bool more = row_on && mb2 > mprev + 8.f;
          const float mnew = more ? mb2 : mprev;
          // what P and O are relative to: the running maximum, or (FAR) that of the weights' exponents
          const bool need = FAR ? row_on && wh > wprev + 8.f : more;
          const float wnew = FAR ? (need ? wh : wprev) : mnew;
          if (j + 1 < j1) {
            mrow[grp * R + row] = mnew;
            if constexpr (FAR) wrow[grp * R + row] = wnew;
            named_bar_arrive(tell_id, 64);
          }
          if (j > u.j0 && __any_sync(0xffffffffu, need)) {
            // the maximum was raised: O must hold every earlier block before it is rescaled
            const uint32_t gp = g - 1u;
            if (ok) ok = seq_wait(&p_empty[gp % C::NS], (gp / C::NS) & 1u, status);
            tc_fence_after();
            const float factor = need ? seq_ex2((FAR ? wprev : mprev) - wnew) : 1.f;
            if (warp_on) {
#pragma unroll 1
              for (int cc = 0; cc < D / 16; ++cc) {
                uint32_t o[16];
                tmem_ld16(tmem + lane_base + C::OCOL + cc * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                whale_tmem_st_cols<16>(tmem + lane_base + C::OCOL + cc * 16, o);
              }
            }
          }
          // P = 2^(S scale_log2 - m), rounded to the operand type over S's first 64 columns; row sum
          // in fp32
          const float nm = mnew == -INFINITY ? 0.f : -mnew;
          const float nw = wnew == -INFINITY ? 0.f : -wnew;
          const float2 sc = make_float2(scale_log2, scale_log2), nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int at = 0; at < KB; at += KB / 2) {
            if (at) load_half(at);
            uint32_t pk[KB / 4];
            if constexpr (FAR) {  // the row sum of 2^(S - m), and P = 2^(S + V's exponent - w)
#pragma unroll
              for (int c4 = 0; c4 < KB / 8; ++c4) {
                const float4 x = *reinterpret_cast<const float4*>(vexp + at + 4 * c4);
                const float s[4] = {__uint_as_float(sr[4 * c4]), __uint_as_float(sr[4 * c4 + 1]),
                                    __uint_as_float(sr[4 * c4 + 2]), __uint_as_float(sr[4 * c4 + 3])};
                sum[0] = seq_add2(sum[0], make_float2(seq_ex2(s[0] + nm), seq_ex2(s[1] + nm)));
                sum[1] = seq_add2(sum[1], make_float2(seq_ex2(s[2] + nm), seq_ex2(s[3] + nm)));
                pk[2 * c4] = Half16<T>::pack2(seq_ex2(s[0] + (x.x + nw)), seq_ex2(s[1] + (x.y + nw)));
                pk[2 * c4 + 1] = Half16<T>::pack2(seq_ex2(s[2] + (x.z + nw)), seq_ex2(s[3] + (x.w + nw)));
              }
            } else {
#pragma unroll
              for (int c2 = 0; c2 < KB / 4; ++c2) {
                const float2 x =
                    seq_fma2(make_float2(__uint_as_float(sr[2 * c2]), __uint_as_float(sr[2 * c2 + 1])), sc, nm2);
                const float2 p = c2 % 4 == 3 ? seq_ex2_poly(x) : make_float2(seq_ex2(x.x), seq_ex2(x.y));
                sum[c2 & 1] = seq_add2(sum[c2 & 1], p);
                pk[c2] = Half16<T>::pack2(p.x, p.y);
              }
            }
            if (warp_on) whale_tmem_st32(ta + at / 2, pk);
            whale_tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * buf + (at ? 1 : 0)]);
          }
          float lsum = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (mnew == -INFINITY) lsum = 0.f;  // no key seen yet
          if (mh != mh) lsum = mh;            // a NaN score: the polynomial would lose it
          l = (m == -INFINITY ? l * 0.f : l * seq_ex2(m - mnew)) + lsum;
          m = mnew;
          wm = wnew;
        }
        // both groups' row sums, relative to the last block's maximum
        const uint32_t gl = g - 1u;
        lrow[grp * R + row] = l;
        mrow[grp * R + row] = m;
        if constexpr (FAR) wrow[grp * R + row] = wm;
        named_bar(pair_id, 64);
        const float mf = mrow[(gl & 1u) * R + row];  // the group of the last block knows the final one
        const float mz = mf == -INFINITY ? 0.f : mf;
        // FAR: O is relative to 2^wf and the row sum to 2^mf; the square root of what lies between them,
        // which fp32 holds whatever V's exponents are
        float between = 1.f;
        if constexpr (FAR) {
          const float wf = wrow[(gl & 1u) * R + row];
          between = wf == -INFINITY ? 0.f : seq_ex2(0.5f * (wf - mz));
        }
        float lt = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) lt += lrow[x * R + row] * seq_ex2(mrow[x * R + row] - mz);
        named_bar(pair_id, 64);  // before the next unit overwrites them
        if (ok) ok = seq_wait(&p_empty[gl % C::NS], (gl / C::NS) & 1u, status);
        tc_fence_after();
        if (warp_on) {
          const float inv = between * (whole ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f);
          const SeqRowsOut out(orow, row_on && ok);
          using S = SeqSlots<R, D>;
          float* slot = whole ? nullptr : S::slot(ws, pieces, blockIdx.x, u.j0 > 0);
#pragma unroll 1
          for (int cc = grp; cc < D / 32; cc += 2) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + C::OCOL + cc * 32, o);
            tmem_ld_wait();
            if constexpr (FAR) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * between);
            }
            if (whole) {
              seq_store_rows<D, T>(stage, o, inv, O, cc * 32, out);
            } else if (row_on && ok) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(S::o(slot, row, cc * 32 + 4 * i)) =
                    make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
            }
          }
          if (row_on && grp == 0) {
            if (!whole) {
              S::m(slot)[row] = mf;
              S::l(slot)[row] = lt;
            } else if (lse) {
              lse[orow] = lt == 0.f ? -INFINITY : 0.69314718055994531f * (mz + log2f(lt));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
      } else if (row_on) {  // no key: nothing to attend to
        const uint32_t z[32] = {};
#pragma unroll 1
        for (int cc = grp; cc < D / 32; cc += 2) whale_st_row32<T>(O + orow * D + cc * 32, z, 0.f, nullptr);
        if (lse && grp == 0) lse[orow] = -INFINITY;
      }
      __syncwarp();
      if (lane == 0) unit_done();
      ++ui;
    }
  } else if (SRC == SEQ_PAGED8 && warp >= 12) {
    // --------------------------------------------- loaders of an 8-bit cache
    constexpr int ITEMS = D / 16;  // 16-byte pieces of the tile per thread
    const int tid = threadIdx.x - 384;
    const int pmask = (1 << a.page_shift) - 1;
    int s = 0;
    uint32_t ph = 0, gk = 0;  // gk: K tiles so far, the numbers that the softmax warps give their blocks
    bool ok = true;
    SeqUnit u;
    auto row_of = [&](const int32_t* trow, int k) -> int64_t {
      const int page = seq_page(trow, k, a.page_shift, a.num_pages);
      if (page < 0) {
        flag_error(status, kFlagBadShape);
        return -1;
      }
      return ((static_cast<int64_t>(page) * a.kv_heads + u.h) << a.page_shift) + (k & pmask);
    };
    for (;;) {
      const bool got = ok && unit_take(u);
      if (!named_bar_and(5, C::LOADERS, got)) break;
      __syncwarp();
      const int j1 = seq_real_end(a, u, group, a.tile, KB);
      const int32_t* trow = a.table + static_cast<int64_t>(u.b) * a.table_width;
      auto load = [&](int which, int j) {
        const uint8_t* base = static_cast<const uint8_t*>(which ? V8 : K8);
        const uint8_t* ex = which ? a.v_exp : a.k_exp;
        uint4 x[ITEMS];
        uint32_t e[ITEMS];
        const int valid = min(KB, u.len - j * KB);
        float kf = 0.f, vx = 0.f;  // FAR: the powers of two of row tid
        if (FAR && which == 0 && tid < valid) {
          const int64_t r = row_of(trow, j * KB + tid);
          if (r >= 0) {
            kf = seq_pow(__ldg(a.k_exp + r)) * (a.scale * 1.4426950408889634f);
            vx = static_cast<float>(static_cast<int>(__ldg(a.v_exp + r)) - 127);
          }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int it = i * C::LOADERS + tid, rr = it / ITEMS, ch = it % ITEMS;
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          e[i] = 0;
          if (rr < valid) {
            const int64_t r = row_of(trow, j * KB + rr);
            if (r >= 0) {
              seq_ldg<16>(base + r * D + ch * 16, reinterpret_cast<uint32_t*>(&x[i]));
              e[i] = __ldg(ex + r);
            }
          }
        }
        if (ok) ok = seq_wait(&kv_empty[s], ph ^ 1u, status);
        if (FAR && which == 0) {
          float* col = columns + (gk++ % C::NX) * 2 * KB;
          col[tid] = kf;
          col[KB + tid] = vx;
        }
        uint8_t* dst = tiles + s * C::TILEB;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int it = i * C::LOADERS + tid, rr = it / ITEMS, ch = it % ITEMS;
          uint32_t v[8];
          if constexpr (FAR) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t b = reinterpret_cast<const uint32_t*>(&x[i])[w];
              v[2 * w] = seq_e4m3_f16(seq_lo16(b));
              v[2 * w + 1] = seq_e4m3_f16(seq_hi16(b));
            }
            if (which == 1 && e[i] == 255) {  // a row that is not finite (K's shows by its factor)
#pragma unroll
              for (int w = 0; w < 8; ++w) v[w] = 0x7FFF7FFFu;
            }
          } else {
            const float f = seq_pow(e[i]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t b = reinterpret_cast<const uint32_t*>(&x[i])[w];
              v[2 * w] = seq_e4m3_bf16(seq_lo16(b), f);
              v[2 * w + 1] = seq_e4m3_bf16(seq_hi16(b), f);
            }
          }
          // 16 elements: units 2 ch and 2 ch + 1 of the row
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int unit16 = 2 * ch + hh, bx = unit16 / (C::SWB / 16), jj = unit16 % (C::SWB / 16);
            *reinterpret_cast<uint4*>(dst + bx * C::BOXB + whale_swz<C::SWB>(rr, jj)) =
                make_uint4(v[4 * hh], v[4 * hh + 1], v[4 * hh + 2], v[4 * hh + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[s]);
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1u;
        }
      };
      for (int j = u.j0; j < j1; ++j) {
        for (int k = u.j0; j == u.j0 && k < min(j1, u.j0 + C::AHEAD); ++k) load(0, k);
        if (j + C::AHEAD < j1) load(0, j + C::AHEAD);
        load(1, j);
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

}  // namespace wk
