// seq_args.cuh -- what every sequence kernel is given, and how the work of a jagged batch is shared
// out among the blocks of a grid.
//
// Units. A unit is R packed query rows of one (sequence, key head): row r of a sequence is query
// row r / group of query head h * group + r % group, so that the query heads that share a key head
// share its loads. Unit (b, h, t) costs max(1, key blocks its last row sees); the units of a batch,
// in the order (b, h, t), make one line of key blocks. The line is cut into equal pieces, one per
// thread block: no block has more than ceil(T / grid) key blocks to do, however ragged the batch and
// however few its rows, and which block does what depends on the lengths alone. A unit that a cut
// goes through is finished by the combine kernel from fp32 partial results: piece c leaves those of
// the unit it enters in the middle in slot 2c, those of the unit it leaves unfinished in slot 2c + 1,
// and a note about the latter. Where sequences are so short that a cut would save less than joining
// the parts costs, the line is made of whole units instead (uncut).
#pragma once

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
  int32_t tile, block;  // rows that stand at a time (whole tokens), and rows that go by (backward)
  int32_t uncut;        // units are not cut: a piece is a number of whole units
  unsigned* status;
};

// Where key rows come from: jagged tensors, a 16-bit cache, an 8-bit cache.
enum { SEQ_JAGGED = 0, SEQ_PAGED16 = 1, SEQ_PAGED8 = 2 };

template <int SRC>
__device__ __forceinline__ SeqSpan seq_keys(const SeqArgs& a, int64_t b) {
  if constexpr (SRC == SEQ_JAGGED) return seq_span(a.kv_off, a.kv_lens, b, a.total_kv, a.max_kv);
  return seq_cached(a.kv_lens, b, static_cast<int64_t>(a.table_width) << a.page_shift, a.max_kv);
}

__device__ __forceinline__ SeqSpan seq_queries(const SeqArgs& a, int64_t b) {
  return seq_span(a.q_off, nullptr, b, a.total_q, a.max_q);
}

// Every kernel here is launched so that its blocks may be set up while the one before it on the
// stream ends. This waits for the results of those before: nothing that they wrote or may still use
// (global memory, TMEM) is touched above it. (Letting the next kernel in before this one's blocks
// end was slower: a training step at the 2-layer shape took 145 us, so 133.)
__device__ __forceinline__ void seq_wait_before() { cudaGridDependencySynchronize(); }

// mbar_wait that gives up early only for a wait that ran out: sequences that are in order keep their
// results in a call (or after one) whose tables set another flag.
__device__ __forceinline__ bool seq_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (*reinterpret_cast<const volatile unsigned*>(status) & kFlagTimeout) return false;
      if (clock64() - start > WK_WAIT_LIMIT) {
        flag_error(status, kFlagTimeout);
        return false;
      }
    }
  }
}

// 2^(e - 127) of a cache row's exponent byte; NaN for 255.
__device__ __forceinline__ float seq_pow(uint32_t e) {
  return __uint_as_float(e == 255 ? 0x7FC00000u : (e == 0 ? 0x00400000u : e << 23));
}

// 2^x (the hardware's approximate base-2 exponential; 2^-inf = +0).
__device__ __forceinline__ float seq_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One (sequence, key head, row tile) and the key blocks [j0, j1) of it that a piece holds.
struct SeqUnit {
  int32_t b, h, t;
  int32_t j0, j1, nb;   // nb: the unit's cost (1 for a unit without keys)
  int32_t n, rows;      // query rows of the sequence; rows that stand (packed rows n * group, or keys)
  int32_t len;          // keys of the sequence
  int64_t q_begin, kv_begin;
};

// What a kernel's units are: R stationary rows, key blocks (or, the other way round, row blocks) of
// KB. The forward's: packed query rows stand, keys go by. R_ = 0: a.tile rows.
template <int R_, int KB_, int SRC_>
struct SeqPlan {
  static constexpr int SRC = SRC_;
  static __device__ __forceinline__ int R(const SeqArgs& a) { return R_ ? R_ : a.tile; }
  static __device__ __forceinline__ int rows(int n, int len, int group) { return n * group; }
  // blocks that tile t sees, at least 1
  static __device__ __forceinline__ int cost(const SeqArgs& a, int n, int len, int group, int t) {
    const int last = (min((t + 1) * R(a), n * group) - 1) / group;
    const int nb = (seq_seen(len, n, last, a.causal) + KB_ - 1) / KB_;
    return nb > 1 ? nb : 1;
  }
  static __device__ __forceinline__ bool uniform(const SeqArgs& a) { return !a.causal; }
};

// The backward's: with SWAP keys stand and packed query rows go by. Tile and block sizes follow the
// number of query heads that share a key head, so that both begin at a token: a.tile, a.block.
template <bool SWAP>
struct SeqPlanBack {
  static constexpr int SRC = SEQ_JAGGED;
  static __device__ __forceinline__ int R(const SeqArgs& a) { return a.tile; }
  static __device__ __forceinline__ int rows(int n, int len, int group) { return SWAP ? len : n * group; }
  static __device__ __forceinline__ int cost(const SeqArgs& a, int n, int len, int group, int t) {
    const int nb = ((SWAP ? n * group : len) + a.block - 1) / a.block;
    return nb > 1 ? nb : 1;
  }
  static __device__ __forceinline__ bool uniform(const SeqArgs&) { return true; }
};

template <class P>
__device__ __forceinline__ int64_t seq_cost(const SeqArgs& a, int64_t b) {
  const SeqSpan q = seq_queries(a, b), kv = seq_keys<P::SRC>(a, b);
  const int group = a.q_heads / a.kv_heads;
  const int tiles = (P::rows(q.len, kv.len, group) + P::R(a) - 1) / P::R(a);
  int64_t s = 0;
  if (a.uncut) {
    s = tiles;
  } else if (!P::uniform(a)) {
    for (int t = 0; t < tiles; ++t) s += P::cost(a, q.len, kv.len, group, t);
  } else if (tiles) {
    s = static_cast<int64_t>(tiles) * P::cost(a, q.len, kv.len, group, 0);
  }
  return s * a.kv_heads;
}

// What the threads of a block find out together at its start: how long the line is, how much of it
// one piece is, and the place on it that this block begins at.
struct SeqPlace {
  int64_t per, begin, end;  // key blocks per piece; this piece's part of the line
  int32_t b;                // sequence that holds `begin`
  int64_t into;             // key blocks from that sequence's start to `begin`
};

// All threads call it (it synchronises the block); sh: NT / 32 + 4 values of shared memory. With
// `tell`, spans out of range set the status word (block 0 only: it sees every sequence).
template <class P, int NT>
__device__ SeqPlace seq_place(const SeqArgs& a, int64_t piece, int64_t pieces, int64_t* sh, bool tell) {
  const int tid = threadIdx.x;
  const int64_t each = (a.batch + NT - 1) / NT;
  const int64_t b0 = min(static_cast<int64_t>(a.batch), tid * each), b1 = min(static_cast<int64_t>(a.batch), b0 + each);
  int64_t sum = 0;
  for (int64_t b = b0; b < b1; ++b) {
    sum += seq_cost<P>(a, b);
    if (tell && (seq_queries(a, b).bad || seq_keys<P::SRC>(a, b).bad)) flag_error(a.status, kFlagBadShape);
  }
  // inclusive scan over the block
  const int lane = tid & 31, warp = tid >> 5;
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  x += before;
  SeqPlace p;
  p.per = total <= INT32_MAX ? (static_cast<uint32_t>(total) + static_cast<uint32_t>(pieces) - 1u) / static_cast<uint32_t>(pieces)
                             : (total + pieces - 1) / pieces;
  if (p.per < 1) p.per = 1;
  p.begin = min(piece * p.per, total);
  p.end = min(p.begin + p.per, total);
  p.b = a.batch;
  p.into = 0;
  if (x - sum <= p.begin && p.begin < x) {  // exactly one thread's sequences hold it
    int64_t at = x - sum;
    for (int64_t b = b0; b < b1; ++b) {
      const int64_t c = seq_cost<P>(a, b);
      if (p.begin < at + c) {
        sh[NT / 32] = b;
        sh[NT / 32 + 1] = p.begin - at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  if (p.begin < p.end) {
    p.b = static_cast<int32_t>(sh[NT / 32]);
    p.into = sh[NT / 32 + 1];
  }
  __syncthreads();
  return p;
}

// Walks the units of a piece.
template <class P>
struct SeqWalk {
  int64_t left;  // key blocks of the piece still to do
  SeqUnit u;
  int32_t tiles, group;

  // Reads sequence u.b (or the next one that has rows); false behind the last.
  __device__ __forceinline__ bool open(const SeqArgs& a) {
    for (; u.b < a.batch; ++u.b) {
      const SeqSpan q = seq_queries(a, u.b);
      const SeqSpan kv = seq_keys<P::SRC>(a, u.b);
      u.rows = P::rows(q.len, kv.len, group);
      if (u.rows == 0) continue;
      u.n = q.len;
      u.q_begin = q.begin;
      u.kv_begin = kv.begin;
      u.len = kv.len;
      tiles = (u.rows + P::R(a) - 1) / P::R(a);
      u.h = u.t = 0;
      return true;
    }
    return false;
  }

  // Puts the walk at the piece's first unit; u.j0 is then where the piece enters it.
  __device__ __forceinline__ void start(const SeqArgs& a, const SeqPlace& p) {
    group = a.q_heads / a.kv_heads;
    left = p.end - p.begin;
    if (left <= 0) return;
    u.b = p.b;
    open(a);
    int64_t into = p.into;
    if (a.uncut || P::uniform(a)) {  // every tile of the sequence costs the same
      const int64_t c = a.uncut ? 1 : P::cost(a, u.n, u.len, group, 0);
      int64_t skip;
      if (into <= UINT32_MAX) {  // 64-bit divisions take long on the way to the first load
        const uint32_t x = static_cast<uint32_t>(into) / static_cast<uint32_t>(c);
        u.h = static_cast<int32_t>(x / static_cast<uint32_t>(tiles));
        u.t = static_cast<int32_t>(x % static_cast<uint32_t>(tiles));
        skip = x;
      } else {
        skip = into / c;
        u.h = static_cast<int32_t>(skip / tiles);
        u.t = static_cast<int32_t>(skip % tiles);
      }
      into -= skip * c;
    } else {
      for (;;) {
        const int64_t c = P::cost(a, u.n, u.len, group, u.t);
        if (into < c) break;
        into -= c;
        if (++u.t == tiles) {
          u.t = 0;
          ++u.h;
        }
      }
    }
    u.j0 = static_cast<int32_t>(into);
  }

  // The next unit of the piece in u; false at its end. Call start() first.
  __device__ __forceinline__ bool next(const SeqArgs& a) {
    if (left <= 0) return false;
    u.nb = P::cost(a, u.n, u.len, group, u.t);
    if (a.uncut) {
      u.j1 = u.nb;
      --left;
      return true;
    }
    u.j1 = static_cast<int32_t>(min(static_cast<int64_t>(u.nb), u.j0 + left));
    left -= u.j1 - u.j0;
    return true;
  }
  // Moves past the unit that next() gave.
  __device__ __forceinline__ void advance(const SeqArgs& a) {
    u.j0 = 0;
    if (left <= 0) return;
    if (++u.t == tiles) {
      u.t = 0;
      if (++u.h == a.kv_heads) {
        ++u.b;
        open(a);
      }
    }
  }
};

// Partial results in the workspace: a note per piece about the unit that it leaves unfinished (its
// last one, if any), then two slots per piece. A slot holds, in fp32, the unit's O [R, D] not
// normalised, in pieces of four columns ([D / 4][R][4], so that the rows of a warp lie next to each
// other), then m [R] (base 2) and l [R].
struct SeqNote {
  int32_t rows, r0;       // packed rows of the unit (0: the piece leaves none unfinished), the first one
  int32_t group, pieces;  // query heads per key head; pieces that the unit is spread over
  int64_t begin;          // the sequence's first row of the tensor
  int32_t h, pad[3];
};

template <int R, int D>
struct SeqSlots {
  static constexpr int64_t kFloats = static_cast<int64_t>(R) * (D + 2);
  static __device__ __forceinline__ SeqNote* note(float* ws, int64_t piece) {
    return reinterpret_cast<SeqNote*>(ws) + piece;
  }
  // the slot of the unit that piece enters in the middle, or of the one that it leaves unfinished
  static __device__ __forceinline__ float* slot(float* ws, int64_t pieces, int64_t piece, bool enters) {
    return reinterpret_cast<float*>(reinterpret_cast<SeqNote*>(ws) + pieces) + (2 * piece + (enters ? 0 : 1)) * kFloats;
  }
  static __device__ __forceinline__ float* o(float* slot, int r, int d) { return slot + (d / 4 * R + r) * 4 + d % 4; }
  static __device__ __forceinline__ float* m(float* slot) { return slot + R * D; }
  static __device__ __forceinline__ float* l(float* slot) { return slot + R * D + R; }
};

// Every piece says what it leaves unfinished; by one thread, for a unit u of which the piece has
// [j0, j1) with j0 == 0 and j1 < nb, or with none = true. begin: the sequence's first row of the
// tensor that the unit's rows are of; tile: rows per unit.
template <int R, int D>
__device__ __forceinline__ void seq_leave_note(float* ws, int64_t piece, const SeqUnit& u, int64_t begin, int tile,
                                               int group, int64_t per, bool none) {
  SeqNote n;
  n.rows = none ? 0 : min(tile, u.rows - u.t * tile);
  n.r0 = u.t * tile;
  n.group = group;
  // the unit's last key block lies nb - j1 blocks behind the piece's end
  n.pieces = none ? 0 : 1 + static_cast<int32_t>((u.nb - u.j1 + per - 1) / per);
  n.begin = begin;
  n.h = u.h;
  n.pad[0] = n.pad[1] = n.pad[2] = 0;
  *SeqSlots<R, D>::note(ws, piece) = n;
}

// Joins the pieces of cut units: a block does CR rows of the unit that piece blockIdx.x / (R / CR)
// leaves unfinished, a thread 8 columns of a row. Bound by the latency of its loads (the note, then
// the maxima, then the rest), so the loads of several pieces are in flight at once. m and l of a row
// that a piece saw no key of are -inf and 0.
template <int R, int CR, int D, typename T>
__global__ void __launch_bounds__(CR * D / 8)
    seq_combine_kernel(float* ws, T* __restrict__ O, float* __restrict__ lse, int32_t q_heads, int32_t pieces) {
  using S = SeqSlots<R, D>;
  const int32_t c = blockIdx.x / (R / CR);
  const int r = (blockIdx.x % (R / CR)) * CR + threadIdx.x % CR, d = (threadIdx.x / CR) * 8;
  seq_wait_before();
  const SeqNote n = *S::note(ws, c);
  if (r >= n.rows) return;
  // piece c left the unit's beginning in its second slot, the others what they entered in their first
  auto slot = [&](int k) { return S::slot(ws, pieces, c + k, k != 0); };
  float m = -INFINITY;
#pragma unroll 4
  for (int k = 0; k < n.pieces; ++k) m = fmaxf(m, S::m(slot(k))[r]);
  const float mz = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < n.pieces; ++k) {
    float* s = slot(k);
    const float f = seq_ex2(S::m(s)[r] - mz);
    const float4 x = *reinterpret_cast<const float4*>(S::o(s, r, d));
    const float4 y = *reinterpret_cast<const float4*>(S::o(s, r, d + 4));
    l += f * S::l(s)[r];
    o[0] += f * x.x;
    o[1] += f * x.y;
    o[2] += f * x.z;
    o[3] += f * x.w;
    o[4] += f * y.x;
    o[5] += f * y.y;
    o[6] += f * y.z;
    o[7] += f * y.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: no piece saw a key
  const int pr = n.r0 + r;
  const int64_t row = (n.begin + pr / n.group) * q_heads + n.h * n.group + pr % n.group;
  *reinterpret_cast<uint4*>(O + row * D + d) =
      make_uint4(Half16<T>::pack2(o[0] * inv, o[1] * inv), Half16<T>::pack2(o[2] * inv, o[3] * inv),
                 Half16<T>::pack2(o[4] * inv, o[5] * inv), Half16<T>::pack2(o[6] * inv, o[7] * inv));
  if (lse && d == 0) lse[row] = l == 0.f ? -INFINITY : 0.69314718055994531f * (mz + log2f(l));
}

}  // namespace wk
