// wk_seq.cu -- the C ABI of attention over behaviour sequences (include/wukong.h): argument
// checks, workspaces and launches of the jagged cross attention, its gradients and the paged cache.
// The kernels are in seq_rows.cuh, seq_tile.cuh, seq_back.cuh and seq_cache.cuh.
#include <algorithm>
#include <cmath>

#include "wukong.h"
#include "common.cuh"
#include "host.cuh"
#include "seq_back.cuh"
#include "seq_cache.cuh"
#include "seq_rows.cuh"
#include "seq_tile.cuh"

using namespace wk;

namespace {

typedef __nv_bfloat16 bf16;
typedef __half f16;

bool seq_d_ok(int d) { return d == 32 || d == 64 || d == 128 || d == 160; }
bool type16(wk_dtype t) { return t == WK_BF16 || t == WK_F16; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The largest number of rows a tensor may have (offsets are int32), and the most rows (times
// heads) or keys of one sequence: the kernels number those in 32 bits.
constexpr int64_t kMaxRows = INT32_MAX, kMostRows = int64_t{1} << 30;

// Stride in elements from token to token: 0 means dense.
int64_t stride_of(int64_t s, int heads, int d) { return s == 0 ? static_cast<int64_t>(heads) * d : s; }

// Bytes from the first to the last element of [rows, heads, d] with a token stride.
int64_t extent(int64_t rows, int64_t stride, int heads, int d) {
  return rows <= 0 ? 0 : ((rows - 1) * stride + static_cast<int64_t>(heads) * d) * 2;
}

struct Bytes {
  const void* p;
  int64_t n;
};

// `n` int32 values of device memory (offsets, lengths, a table).
Bytes ints(const int32_t* p, int64_t n) { return {p, n * 4}; }

// Whether something written lies over something read, or over something else written.
template <int W, int R>
bool overlap(const Bytes (&written)[W], const Bytes (&read)[R]) {
  auto over = [](const Bytes& a, const Bytes& b) {
    const uint8_t *x = static_cast<const uint8_t*>(a.p), *y = static_cast<const uint8_t*>(b.p);
    return a.n > 0 && b.n > 0 && x && y && x < y + b.n && y < x + a.n;
  };
  for (int i = 0; i < W; ++i) {
    for (const Bytes& r : read)
      if (over(written[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (over(written[i], written[j])) return true;
  }
  return false;
}

wk_status check_config(const wk_xattn_config* c) {
  if (!c || c->batch < 0 || c->q_heads < 1 || c->kv_heads < 1 || c->q_heads % c->kv_heads != 0 || c->max_q < 0 ||
      c->max_kv < 0 || c->total_q < 0 || c->total_kv < 0 || c->total_q > kMaxRows || c->total_kv > kMaxRows ||
      c->max_kv > kMostRows || static_cast<int64_t>(c->max_q) * c->q_heads > kMostRows || !(c->scale >= 0.f) ||
      !std::isfinite(c->scale))
    return WK_ERR_INVALID_ARG;
  if (!seq_d_ok(c->d) || !type16(c->dtype) || c->q_heads > 1024 || c->q_heads / c->kv_heads > 64)
    return WK_ERR_UNSUPPORTED;
  const int64_t qs = stride_of(c->q_stride, c->q_heads, c->d), ks = stride_of(c->k_stride, c->kv_heads, c->d),
                vs = stride_of(c->v_stride, c->kv_heads, c->d);
  const int64_t qd = static_cast<int64_t>(c->q_heads) * c->d, kd = static_cast<int64_t>(c->kv_heads) * c->d;
  if (qs < qd || ks < kd || vs < kd || qs > (1 << 30) || ks > (1 << 30) || vs > (1 << 30)) return WK_ERR_INVALID_ARG;
  if (qs % 8 != 0 || ks % 8 != 0 || vs % 8 != 0) return WK_ERR_UNSUPPORTED;
  return WK_OK;
}

wk_status check_cache(const wk_cache* c) {
  if (!c || c->num_pages < 0 || c->kv_heads < 1) return WK_ERR_INVALID_ARG;
  if (!seq_d_ok(c->d) || c->kv_heads > 1024 ||
      (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) ||
      (!type16(c->dtype) && c->dtype != WK_E4M3))
    return WK_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && (!c->K || !c->V || !al16(c->K) || !al16(c->V))) return WK_ERR_INVALID_ARG;
  const bool q8 = c->dtype == WK_E4M3;
  if (c->num_pages > 0 && q8 && (!c->K_exp || !c->V_exp || !al16(c->K_exp) || !al16(c->V_exp)))
    return WK_ERR_INVALID_ARG;
  if (!q8 && (c->K_exp || c->V_exp)) return WK_ERR_INVALID_ARG;
  return WK_OK;
}

// Rows of a cache, and bytes of its K (or V).
int64_t cache_rows(const wk_cache& c) { return static_cast<int64_t>(c.num_pages) * c.kv_heads * c.page_size; }
int64_t cache_bytes(const wk_cache& c) { return cache_rows(c) * c.d * (c.dtype == WK_E4M3 ? 1 : 2); }

int shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

SeqArgs make_args(const wk_xattn_config& c, const int32_t* q_off, const int32_t* kv_off, const int32_t* kv_lens,
                  unsigned* status) {
  SeqArgs a{};
  a.batch = c.batch;
  a.q_heads = c.q_heads;
  a.kv_heads = c.kv_heads;
  a.max_q = c.max_q;
  a.max_kv = c.max_kv;
  a.total_q = c.total_q;
  a.total_kv = c.total_kv;
  a.q_stride = stride_of(c.q_stride, c.q_heads, c.d);
  a.k_stride = stride_of(c.k_stride, c.kv_heads, c.d);
  a.v_stride = stride_of(c.v_stride, c.kv_heads, c.d);
  a.scale = c.scale > 0.f ? c.scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.d)));
  a.q_off = q_off;
  a.kv_off = kv_off;
  a.kv_lens = kv_lens;
  a.status = status;
  return a;
}

void cache_args(SeqArgs* a, const wk_cache& c, const int32_t* table, int32_t width) {
  a->table = table;
  a->table_width = width;
  a->num_pages = c.num_pages;
  a->page_shift = shift_of(c.page_size);
  a->kv_heads = c.kv_heads;
  a->k_exp = c.K_exp;
  a->v_exp = c.V_exp;
}

// ---------------------------------------------------------------- launches

// Launches a kernel that may start while the one before it on the stream ends: every kernel here
// waits for that one's results itself, before its first access to global memory. Its launch and set-up
// (barriers, TMEM) then lie under the end of the kernel before.
template <typename... P, typename... A>
wk_status launch(void (*fn)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return WK_ERR_CUDA;
  }
  return WK_OK;
}

// Up to this many blocks of 128 keys (or 64 rows, twice as many) a unit is not cut: joining its parts
// is one more launch of about 3 us, a block takes a fraction of that.
constexpr int kUncut = 4;

// ---- the few-rows kernel: packed rows per (sequence, key head) up to 16 (seq_rows.cuh)
constexpr int kSMs = 148;  // the grids' unit; results do not depend on it
constexpr int kRowsMost = 16, kRowsKB = 128;

int64_t packed_rows(const SeqArgs& a) { return static_cast<int64_t>(a.max_q) * (a.q_heads / a.kv_heads); }
int rows_nq(const SeqArgs& a) { return packed_rows(a) <= 8 ? 1 : 2; }
int rows_pieces(int d, int nq, bool q8) { return kSMs * seq_rows_occupancy(d, nq, q8); }

// Bytes of the notes and slots of `pieces` pieces of units of r rows.
int64_t slot_bytes(int r, int d, int64_t pieces) {
  return pieces * static_cast<int64_t>(sizeof(SeqNote)) + 2 * pieces * r * (d + 2) * 4;
}

bool rows_cut(const SeqArgs& a) { return a.max_q > 0 && a.max_kv > kUncut * kRowsKB; }
// Bytes of partial results.
int64_t rows_ws(const SeqArgs& a, int d, bool q8) {
  const int nq = rows_nq(a);
  return rows_cut(a) ? slot_bytes(8 * nq, d, rows_pieces(d, nq, q8)) : 0;
}

template <int D, typename T, int SRC, int NQ>
wk_status run_rows(const void* Q, const void* K, const void* V, void* O, float* lse, float* ws, SeqArgs a,
                   cudaStream_t st) {
  const int32_t pieces = rows_pieces(D, NQ, SRC == SEQ_PAGED8);
  a.uncut = !rows_cut(a);
  const wk_status s = launch(seq_rows_kernel<D, T, SRC, NQ>, pieces, SEQ_ROWS_THREADS, 0, st, static_cast<const T*>(Q), K,
                             V, static_cast<T*>(O), lse, a.uncut ? nullptr : ws, a, pieces);
  if (s != WK_OK || a.uncut) return s;
  return launch(seq_combine_kernel<8 * NQ, 8 * NQ, D, T>, pieces, NQ * D, 0, st, ws, static_cast<T*>(O), lse,
                a.q_heads, pieces);
}

// ---- the tile kernel: any number of rows, 128 packed rows per tile (seq_tile.cuh)
bool tile_cut(const SeqArgs& a) { return a.max_kv > kUncut * 128; }
int64_t tile_ws(const SeqArgs& a, int d) { return tile_cut(a) ? slot_bytes(128, d, kSMs) : 0; }

// [tokens, heads, d] as a 3-D map (d, heads, tokens) with boxes (bw, box_heads, box_tokens). Of no
// tokens it is a map over `any`, and not used.
template <typename T>
bool map_tokens(const DevInfo* dv, CUtensorMap* m, const void* base, const void* any, int d, int heads, int64_t tokens,
                int64_t stride, int bw, int box_heads, int box_tokens) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(std::max<int64_t>(tokens, 1))};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(stride) * 2};
  const uint32_t box[3] = {static_cast<uint32_t>(bw), static_cast<uint32_t>(box_heads),
                           static_cast<uint32_t>(box_tokens)};
  return make_map(dv, m, tmap_dtype<T>(), 3, tokens > 0 ? base : any, dims, strides, box,
                  bw == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// The rows of a 16-bit cache as a 2-D map (d, rows) with boxes of one page. Of no pages it is a map
// over `any`, and not used.
template <typename T>
bool map_pages(const DevInfo* dv, CUtensorMap* m, const void* base, const void* any, int d, int64_t rows, int bw,
               int page) {
  const uint64_t dims[2] = {static_cast<uint64_t>(d), static_cast<uint64_t>(std::max<int64_t>(rows, 1))};
  const uint64_t strides[1] = {static_cast<uint64_t>(d) * 2};
  const uint32_t box[2] = {static_cast<uint32_t>(bw), static_cast<uint32_t>(page)};
  return make_map(dv, m, tmap_dtype<T>(), 2, rows > 0 ? base : any, dims, strides, box,
                  bw == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, typename T, int SRC>
wk_status run_tile(const DevInfo* dv, const void* Q, const void* K, const void* V, void* O, float* lse, float* ws,
                   SeqArgs a, cudaStream_t st) {
  using C = StCfg<D, SRC>;
  const int group = a.q_heads / a.kv_heads;
  a.tile = group * (128 / group);
  a.uncut = !tile_cut(a);
  CUtensorMap mq{}, mk{}, mv{};
  if (!map_tokens<T>(dv, &mq, Q, Q, D, a.q_heads, a.total_q, a.q_stride, C::BW, group, 128 / group))
    return WK_ERR_UNSUPPORTED;
  if (SRC == SEQ_JAGGED) {
    if (!map_tokens<T>(dv, &mk, K, Q, D, a.kv_heads, a.total_kv, a.k_stride, C::BW, 1, 128) ||
        !map_tokens<T>(dv, &mv, V, Q, D, a.kv_heads, a.total_kv, a.v_stride, C::BW, 1, 128))
      return WK_ERR_UNSUPPORTED;
  } else if (SRC == SEQ_PAGED16) {
    const int64_t rows = (static_cast<int64_t>(a.num_pages) * a.kv_heads) << a.page_shift;
    if (rows > INT32_MAX || !map_pages<T>(dv, &mk, K, Q, D, rows, C::BW, 1 << a.page_shift) ||
        !map_pages<T>(dv, &mv, V, Q, D, rows, C::BW, 1 << a.page_shift))
      return WK_ERR_UNSUPPORTED;
  }
  auto fn = seq_tile_kernel<D, T, SRC>;
  wk_status s = smem_attr(dv, reinterpret_cast<const void*>(fn), C::SMEM);
  if (s != WK_OK) return s;
  s = launch(fn, kSMs, C::THREADS, C::SMEM, st, mq, mk, mv, K, V, static_cast<T*>(O), lse, a.uncut ? nullptr : ws, a,
             int64_t{kSMs});
  if (s != WK_OK || a.uncut) return s;
  constexpr int CR = 16;
  return launch(seq_combine_kernel<128, CR, D, T>, kSMs * (128 / CR), CR * D / 8, 0, st, ws, static_cast<T*>(O), lse,
                a.q_heads, int32_t{kSMs});
}

int64_t forward_ws(const SeqArgs& a, int d, bool q8) {
  return packed_rows(a) <= kRowsMost ? rows_ws(a, d, q8) : tile_ws(a, d);
}

// Calls f with the head width and the 16-bit type as compile-time values.
template <typename F>
wk_status with_type(int d, wk_dtype t, F f) {
  const bool b = t == WK_BF16;
  switch (d) {
    case 32: return b ? f.template operator()<32, bf16>() : f.template operator()<32, f16>();
    case 64: return b ? f.template operator()<64, bf16>() : f.template operator()<64, f16>();
    case 128: return b ? f.template operator()<128, bf16>() : f.template operator()<128, f16>();
    case 160: return b ? f.template operator()<160, bf16>() : f.template operator()<160, f16>();
  }
  return WK_ERR_UNSUPPORTED;
}

struct RunForward {
  const DevInfo* dv;
  const void *Q, *K, *V;
  void* O;
  float* lse;
  float* ws;
  SeqArgs a;
  int src;
  cudaStream_t st;
  template <int D, typename T, int SRC>
  wk_status run() const {
    if (packed_rows(a) <= kRowsMost)
      return rows_nq(a) == 1
                 ? run_rows<D, T, SRC, 1>(Q, K, V, O, lse, ws, a, st)
                 : run_rows<D, T, SRC, 2>(Q, K, V, O, lse, ws, a, st);
    return run_tile<D, T, SRC>(dv, Q, K, V, O, lse, ws, a, st);
  }
  template <int D, typename T>
  wk_status operator()() const {
    return src == 0 ? run<D, T, 0>() : src == 1 ? run<D, T, 1>() : run<D, T, 2>();
  }
};

// ---- the backward (seq_back.cuh): delta [total_q, q_heads], with fp16 the norms of dO and V, then the
// partial results, which the two kernels use one after the other
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
int64_t delta_bytes(const SeqArgs& a) { return up256(a.total_q * a.q_heads * 4); }
// bytes of the chunks of a jagged tensor (SeqRange)
int64_t chunk_bytes(const SeqArgs& a, int64_t total) { return up256((total / SEQ_CHUNK + a.batch) * a.kv_heads * 4); }
int64_t range_bytes(const SeqArgs& a, wk_dtype t) {
  return t == WK_F16 ? delta_bytes(a) + chunk_bytes(a, a.total_q) + chunk_bytes(a, a.total_kv) : 0;
}
int dkv_block(const SeqArgs& a) { return (a.q_heads / a.kv_heads) * (64 / (a.q_heads / a.kv_heads)); }
bool dq_cut(const SeqArgs& a) { return a.max_kv > 2 * kUncut * 64; }
bool dkv_cut(const SeqArgs& a) { return packed_rows(a) > 2 * kUncut * dkv_block(a); }
int64_t backward_ws(const SeqArgs& a, int d, wk_dtype t) {
  return delta_bytes(a) + range_bytes(a, t) + (dkv_cut(a) ? slot_bytes(128, 2 * d, kSMs) : dq_cut(a) ? slot_bytes(128, d, kSMs) : 0);
}

struct RunBackward {
  const DevInfo* dv;
  const void *Q, *K, *V, *O, *dO;
  const float* lse;
  void *dQ, *dK, *dV;
  void* workspace;
  SeqArgs a;
  cudaStream_t st;

  template <int D, typename T, bool DKV>
  wk_status one(const CUtensorMap (&m)[4], float* delta, const SeqRange& range, float* slots, void* G1, void* G2) const {
    using C = SbCfg<D, DKV>;
    SeqArgs x = a;
    const int group = a.q_heads / a.kv_heads;
    x.tile = DKV ? 128 : group * (128 / group);
    x.block = DKV ? dkv_block(a) : C::YB;
    x.uncut = !(DKV ? dkv_cut(a) : dq_cut(a));
    auto fn = seq_back_kernel<D, T, DKV>;
    wk_status s = smem_attr(dv, reinterpret_cast<const void*>(fn), C::SMEM);
    if (s != WK_OK) return s;
    s = launch(fn, kSMs, C::THREADS, C::SMEM, st, m[0], m[1], m[2], m[3], static_cast<const T*>(O),
               static_cast<const T*>(dO), lse, delta, range, static_cast<T*>(G1), static_cast<T*>(G2),
               x.uncut ? nullptr : slots, x, int64_t{kSMs});
    if (s != WK_OK || x.uncut) return s;
    constexpr int CR = 16 / C::NACC;
    return launch(seq_sum_kernel<CR, D, C::NACC, T>, kSMs * (128 / CR), CR * C::NACC * D / 8, 0, st, slots,
                  static_cast<T*>(G1), static_cast<T*>(G2), DKV ? a.kv_heads : a.q_heads, int32_t{kSMs});
  }

  template <int D, typename T>
  wk_status operator()() const {
    constexpr int BW = SbCfg<D, false>::BW, YB = SbCfg<D, false>::YB;
    const int group = a.q_heads / a.kv_heads;
    // without rows (or without keys) the tensors may be NULL; their maps are then not used
    const void* any = a.total_q > 0 ? Q : K;
    const int64_t od = static_cast<int64_t>(a.q_heads) * D;
    auto rows = [&](CUtensorMap* m, const void* p, int64_t stride, int n) {
      return map_tokens<T>(dv, m, p, any, D, a.q_heads, a.total_q, stride, BW, group, n / group);
    };
    auto keys = [&](CUtensorMap* m, const void* p, int64_t stride, int n) {
      return map_tokens<T>(dv, m, p, any, D, a.kv_heads, a.total_kv, stride, BW, 1, n);
    };
    CUtensorMap q[4], k[4];  // the maps of DQ and of DKV
    if (!rows(&q[0], Q, a.q_stride, 128) || !rows(&q[1], dO, od, 128) || !keys(&q[2], K, a.k_stride, YB) ||
        !keys(&q[3], V, a.v_stride, YB) || !keys(&k[0], K, a.k_stride, 128) || !keys(&k[1], V, a.v_stride, 128) ||
        !rows(&k[2], Q, a.q_stride, 64) || !rows(&k[3], dO, od, 64))
      return WK_ERR_UNSUPPORTED;
    float* delta = static_cast<float*>(workspace);
    uint8_t* rest = static_cast<uint8_t*>(workspace) + delta_bytes(a);
    SeqRange range{};
    if constexpr (!Half16<T>::kBF16) {
      range.rows = reinterpret_cast<float*>(rest);
      range.g = reinterpret_cast<float*>(rest + delta_bytes(a));
      range.v = reinterpret_cast<float*>(rest + delta_bytes(a) + chunk_bytes(a, a.total_q));
      rest += range_bytes(a, WK_F16);
      if (a.total_q > 0 && a.total_kv > 0) {
        // a warp to a chunk, as long as that is not many times the blocks that the SMs hold
        const int64_t chunks = (static_cast<int64_t>(std::max(a.max_q, a.max_kv)) + SEQ_CHUNK - 1) / SEQ_CHUNK * a.kv_heads;
        const unsigned z = static_cast<unsigned>(std::clamp<int64_t>((chunks + 7) / 8, 1, std::max(1, 16 * kSMs / a.batch)));
        const wk_status s = launch(seq_range_kernel<D, T>, dim3(static_cast<unsigned>(a.batch), 2, z), 256, 0, st,
                                   static_cast<const T*>(V), static_cast<const T*>(dO), range, a);
        if (s != WK_OK) return s;
      }
    }
    float* slots = reinterpret_cast<float*>(rest);
    if (a.total_q > 0) {
      const wk_status s = one<D, T, false>(q, delta, range, slots, dQ, nullptr);
      if (s != WK_OK) return s;
    }
    if (a.total_kv > 0) {
      const wk_status s = one<D, T, true>(k, delta, range, slots, dK, dV);
      if (s != WK_OK) return s;
      if (a.kv_lens) {
        // a block for each 16 KB that a sequence would have to clear if it were all padding
        const int64_t each = a.total_kv / a.batch * a.kv_heads * D * 2;
        const unsigned z = static_cast<unsigned>(std::clamp<int64_t>(each >> 14, 1, 64));
        return launch(seq_zero_padding_kernel<T>, dim3(static_cast<unsigned>(a.batch), 2, z), 256, 0, st,
                      static_cast<T*>(dK), static_cast<T*>(dV), static_cast<int64_t>(a.kv_heads) * D, a);
      }
    }
    return WK_OK;
  }
};

// Blocks of the copies per (sequence, key head, K or V); one at least, which sees sequences that are
// longer than a maximum of 0.
int32_t copy_chunks(int32_t most) { return std::max(1, (most + SEQ_COPY_ROWS - 1) / SEQ_COPY_ROWS); }

struct RunWrite {
  const wk_cache& c;
  const void *K, *V;
  SeqArgs a;
  unsigned grid;
  int32_t chunks;
  cudaStream_t st;
  template <int D, typename T>
  wk_status operator()() const {
    const T *k = static_cast<const T*>(K), *v = static_cast<const T*>(V);
    if (c.dtype == WK_E4M3)
      return launch(cache_write_kernel<D, T, true>, grid, SEQ_COPY_THREADS, 0, st, k, v, c.K, c.V, c.K_exp, c.V_exp, a,
                    chunks);
    return launch(cache_write_kernel<D, T, false>, grid, SEQ_COPY_THREADS, 0, st, k, v, c.K, c.V, nullptr, nullptr, a,
                  chunks);
  }
};

struct RunRead {
  const wk_cache& c;
  void *K, *V;
  SeqArgs a;
  unsigned grid;
  int32_t chunks;
  cudaStream_t st;
  template <int D, typename T>
  wk_status operator()() const {
    T *k = static_cast<T*>(K), *v = static_cast<T*>(V);
    if (c.dtype == WK_E4M3)
      return launch(cache_read_kernel<D, T, SEQ_PAGED8>, grid, SEQ_COPY_THREADS, 0, st, c.K, c.V, k, v, a, chunks);
    return launch(cache_read_kernel<D, T, SEQ_PAGED16>, grid, SEQ_COPY_THREADS, 0, st, c.K, c.V, k, v, a, chunks);
  }
};

}  // namespace

extern "C" {

wk_status wk_xattn_workspace(const wk_xattn_config* cfg, int backward, int64_t* bytes) {
  if (!bytes) return WK_ERR_INVALID_ARG;
  const wk_status s = check_config(cfg);
  if (s != WK_OK) return s;
  const int64_t forward = forward_ws(make_args(*cfg, nullptr, nullptr, nullptr, nullptr), cfg->d, false);
  *bytes = backward ? std::max(forward, backward_ws(make_args(*cfg, nullptr, nullptr, nullptr, nullptr), cfg->d, cfg->dtype)) : forward;
  return WK_OK;
}

wk_status wk_xattn_forward(const wk_xattn_config* cfg, const void* Q, const void* K, const void* V,
                           const int32_t* q_off, const int32_t* kv_off, const int32_t* kv_lens, void* O, float* lse,
                           void* workspace, int64_t workspace_bytes, wk_stream_t stream) {
  wk_status s = check_config(cfg);
  if (s != WK_OK) return s;
  if (cfg->batch == 0 || cfg->total_q == 0) return WK_OK;
  const bool keys = cfg->total_kv > 0;
  if (!Q || !O || !q_off || !kv_off || (keys && (!K || !V)) || !al16(Q) || !al16(K) || !al16(V) || !al16(O) ||
      !al4(q_off) || !al4(kv_off) || !al4(kv_lens) || !al4(lse) || !al16(workspace) || workspace_bytes < 0)
    return WK_ERR_INVALID_ARG;
  int64_t need = 0;
  s = wk_xattn_workspace(cfg, 0, &need);
  if (s != WK_OK) return s;
  if (need > workspace_bytes || (need > 0 && !workspace)) return WK_ERR_INVALID_ARG;
  SeqArgs a = make_args(*cfg, q_off, kv_off, kv_lens, nullptr);
  const Bytes written[] = {{O, cfg->total_q * cfg->q_heads * cfg->d * 2},
                           {lse, cfg->total_q * cfg->q_heads * 4},
                           {workspace, need}};
  const Bytes read[] = {{Q, extent(cfg->total_q, a.q_stride, cfg->q_heads, cfg->d)},
                        {K, extent(cfg->total_kv, a.k_stride, cfg->kv_heads, cfg->d)},
                        {V, extent(cfg->total_kv, a.v_stride, cfg->kv_heads, cfg->d)},
                        ints(q_off, cfg->batch + int64_t{1}),
                        ints(kv_off, cfg->batch + int64_t{1}),
                        ints(kv_lens, cfg->batch)};
  if (overlap(written, read)) return WK_ERR_INVALID_ARG;
  DevInfo* dv = nullptr;
  s = dev_info(&dv);
  if (s != WK_OK) return s;
  a.status = dv->standalone_status;
  return with_type(cfg->d, cfg->dtype, RunForward{dv, Q, K, V, O, lse, static_cast<float*>(workspace), a, 0, reinterpret_cast<cudaStream_t>(stream)});
}

wk_status wk_xattn_backward(const wk_xattn_config* cfg, const void* Q, const void* K, const void* V, const void* O,
                            const float* lse, const void* dO, const int32_t* q_off, const int32_t* kv_off,
                            const int32_t* kv_lens, void* dQ, void* dK, void* dV, void* workspace,
                            int64_t workspace_bytes, wk_stream_t stream) {
  wk_status s = check_config(cfg);
  if (s != WK_OK) return s;
  if (cfg->batch == 0) return WK_OK;
  const bool keys = cfg->total_kv > 0, rows = cfg->total_q > 0;
  if (!q_off || !kv_off || (rows && (!Q || !O || !lse || !dO || !dQ)) || (keys && (!K || !V || !dK || !dV)) ||
      !al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(dO) || !al16(dQ) || !al16(dK) || !al16(dV) ||
      !al4(q_off) || !al4(kv_off) || !al4(kv_lens) || !al4(lse) || !al16(workspace) || workspace_bytes < 0)
    return WK_ERR_INVALID_ARG;
  int64_t need = 0;
  s = wk_xattn_workspace(cfg, 1, &need);
  if (s != WK_OK) return s;
  if (need > workspace_bytes || (need > 0 && !workspace)) return WK_ERR_INVALID_ARG;
  SeqArgs a = make_args(*cfg, q_off, kv_off, kv_lens, nullptr);
  const int64_t qb = cfg->total_q * cfg->q_heads * cfg->d * 2, kb = cfg->total_kv * cfg->kv_heads * cfg->d * 2;
  const Bytes written[] = {{dQ, qb}, {dK, kb}, {dV, kb}, {workspace, need}};
  const Bytes read[] = {{Q, extent(cfg->total_q, a.q_stride, cfg->q_heads, cfg->d)},
                        {K, extent(cfg->total_kv, a.k_stride, cfg->kv_heads, cfg->d)},
                        {V, extent(cfg->total_kv, a.v_stride, cfg->kv_heads, cfg->d)},
                        {O, qb},
                        {dO, qb},
                        {lse, cfg->total_q * cfg->q_heads * 4},
                        ints(q_off, cfg->batch + int64_t{1}),
                        ints(kv_off, cfg->batch + int64_t{1}),
                        ints(kv_lens, cfg->batch)};
  if (overlap(written, read)) return WK_ERR_INVALID_ARG;
  if (!rows && !keys) return WK_OK;
  DevInfo* dv = nullptr;
  s = dev_info(&dv);
  if (s != WK_OK) return s;
  a.status = dv->standalone_status;
  return with_type(cfg->d, cfg->dtype,
                   RunBackward{dv, Q, K, V, O, dO, lse, dQ, dK, dV, workspace, a, reinterpret_cast<cudaStream_t>(stream)});
}

wk_status wk_cache_write(const wk_cache* cache, const void* K, const void* V, int64_t k_stride, int64_t v_stride,
                         wk_dtype dtype, const int32_t* new_off, const int32_t* table, int32_t table_width,
                         const int32_t* kv_lens, int32_t batch, int64_t total_new, int32_t max_new,
                         wk_stream_t stream) {
  wk_status s = check_cache(cache);
  if (s != WK_OK) return s;
  if (batch < 0 || total_new < 0 || total_new > kMaxRows || max_new < 0 || table_width < 0) return WK_ERR_INVALID_ARG;
  if (!type16(dtype) || (cache->dtype != WK_E4M3 && cache->dtype != dtype)) return WK_ERR_UNSUPPORTED;
  wk_xattn_config cfg{batch, cache->kv_heads, cache->kv_heads, cache->d, max_new, 0, total_new, total_new, 0, k_stride,
                      v_stride, dtype, 0.f};
  s = check_config(&cfg);
  if (s != WK_OK) return s;
  if (batch == 0 || total_new == 0) return WK_OK;
  if (!K || !V || !new_off || !table || !kv_lens || table_width < 1 || cache->num_pages < 1 || !al16(K) || !al16(V) ||
      !al4(new_off) || !al4(table) || !al4(kv_lens))
    return WK_ERR_INVALID_ARG;
  SeqArgs a = make_args(cfg, new_off, nullptr, kv_lens, nullptr);
  cache_args(&a, *cache, table, table_width);
  const Bytes written[] = {{cache->K, cache_bytes(*cache)},
                           {cache->V, cache_bytes(*cache)},
                           {cache->K_exp, cache_rows(*cache)},
                           {cache->V_exp, cache_rows(*cache)}};
  const Bytes read[] = {{K, extent(total_new, a.k_stride, cfg.kv_heads, cfg.d)},
                        {V, extent(total_new, a.v_stride, cfg.kv_heads, cfg.d)},
                        ints(new_off, batch + int64_t{1}),
                        ints(table, static_cast<int64_t>(batch) * table_width),
                        ints(kv_lens, batch)};
  if (overlap(written, read)) return WK_ERR_INVALID_ARG;
  const int32_t chunks = copy_chunks(max_new);
  const int64_t grid = static_cast<int64_t>(batch) * chunks * cache->kv_heads * 2;
  if (grid > INT32_MAX) return WK_ERR_UNSUPPORTED;
  DevInfo* dv = nullptr;
  s = dev_info(&dv);
  if (s != WK_OK) return s;
  a.status = dv->standalone_status;
  return with_type(cache->d, dtype, RunWrite{*cache, K, V, a, static_cast<unsigned>(grid), chunks,
                                                 reinterpret_cast<cudaStream_t>(stream)});
}

wk_status wk_cache_read(const wk_cache* cache, const int32_t* table, int32_t table_width, const int32_t* kv_lens,
                        const int32_t* out_off, void* K, void* V, wk_dtype dtype, int32_t batch, int64_t total,
                        int32_t max_kv, wk_stream_t stream) {
  wk_status s = check_cache(cache);
  if (s != WK_OK) return s;
  if (batch < 0 || total < 0 || total > kMaxRows || max_kv < 0 || table_width < 0) return WK_ERR_INVALID_ARG;
  if (!type16(dtype) || (cache->dtype != WK_E4M3 && cache->dtype != dtype)) return WK_ERR_UNSUPPORTED;
  if (batch == 0 || total == 0) return WK_OK;
  if (!K || !V || !out_off || (!table && table_width > 0) || !kv_lens || !al16(K) || !al16(V) ||
      !al4(out_off) || !al4(table) || !al4(kv_lens))
    return WK_ERR_INVALID_ARG;
  const Bytes written[] = {{K, total * cache->kv_heads * cache->d * 2}, {V, total * cache->kv_heads * cache->d * 2}};
  const Bytes read[] = {{cache->K, cache_bytes(*cache)},
                        {cache->V, cache_bytes(*cache)},
                        {cache->K_exp, cache_rows(*cache)},
                        {cache->V_exp, cache_rows(*cache)},
                        ints(out_off, batch + int64_t{1}),
                        ints(table, static_cast<int64_t>(batch) * table_width),
                        ints(kv_lens, batch)};
  if (overlap(written, read)) return WK_ERR_INVALID_ARG;
  wk_xattn_config cfg{batch, cache->kv_heads, cache->kv_heads, cache->d, 0, max_kv, 0, total, 0, 0, 0, dtype, 0.f};
  SeqArgs a = make_args(cfg, nullptr, out_off, kv_lens, nullptr);
  cache_args(&a, *cache, table, table_width);
  const int32_t chunks = copy_chunks(max_kv);
  const int64_t grid = static_cast<int64_t>(batch) * chunks * cache->kv_heads * 2;
  if (grid > INT32_MAX) return WK_ERR_UNSUPPORTED;
  DevInfo* dv = nullptr;
  s = dev_info(&dv);
  if (s != WK_OK) return s;
  a.status = dv->standalone_status;
  return with_type(cache->d, dtype, RunRead{*cache, K, V, a, static_cast<unsigned>(grid), chunks,
                                                reinterpret_cast<cudaStream_t>(stream)});
}

wk_status wk_cache_attention_workspace(const wk_cache* cache, const wk_xattn_config* cfg, int64_t* bytes) {
  if (!bytes) return WK_ERR_INVALID_ARG;
  wk_status s = check_cache(cache);
  if (s != WK_OK) return s;
  s = check_config(cfg);
  if (s != WK_OK) return s;
  if (cfg->kv_heads != cache->kv_heads || cfg->d != cache->d) return WK_ERR_INVALID_ARG;
  if (cache->dtype != WK_E4M3 && cache->dtype != cfg->dtype) return WK_ERR_UNSUPPORTED;
  *bytes = forward_ws(make_args(*cfg, nullptr, nullptr, nullptr, nullptr), cfg->d, cache->dtype == WK_E4M3);
  return WK_OK;
}

wk_status wk_cache_attention(const wk_cache* cache, const wk_xattn_config* cfg, const void* Q, const int32_t* q_off,
                             const int32_t* table, int32_t table_width, const int32_t* kv_lens, int causal, void* O,
                             float* lse, void* workspace, int64_t workspace_bytes, wk_stream_t stream) {
  int64_t need = 0;
  wk_status s = wk_cache_attention_workspace(cache, cfg, &need);
  if (s != WK_OK) return s;
  if (table_width < 0) return WK_ERR_INVALID_ARG;
  if (cfg->batch == 0 || cfg->total_q == 0) return WK_OK;
  if (!Q || !O || !q_off || (!table && table_width > 0) || !kv_lens || !al16(Q) || !al16(O) ||
      !al4(q_off) || !al4(table) || !al4(kv_lens) || !al4(lse) || !al16(workspace) || workspace_bytes < 0)
    return WK_ERR_INVALID_ARG;
  if (need > workspace_bytes || (need > 0 && !workspace)) return WK_ERR_INVALID_ARG;
  SeqArgs a = make_args(*cfg, q_off, nullptr, kv_lens, nullptr);
  cache_args(&a, *cache, table, table_width);
  a.causal = causal != 0;
  const Bytes written[] = {{O, cfg->total_q * cfg->q_heads * cfg->d * 2},
                           {lse, cfg->total_q * cfg->q_heads * 4},
                           {workspace, need}};
  const Bytes read[] = {{Q, extent(cfg->total_q, a.q_stride, cfg->q_heads, cfg->d)},
                        {cache->K, cache_bytes(*cache)},
                        {cache->V, cache_bytes(*cache)},
                        {cache->K_exp, cache_rows(*cache)},
                        {cache->V_exp, cache_rows(*cache)},
                        ints(q_off, cfg->batch + int64_t{1}),
                        ints(table, static_cast<int64_t>(cfg->batch) * table_width),
                        ints(kv_lens, cfg->batch)};
  if (overlap(written, read)) return WK_ERR_INVALID_ARG;
  DevInfo* dv = nullptr;
  s = dev_info(&dv);
  if (s != WK_OK) return s;
  a.status = dv->standalone_status;
  return with_type(cfg->d, cfg->dtype, RunForward{dv, Q, cache->K, cache->V, O, lse, static_cast<float*>(workspace), a,
                                                  cache->dtype == WK_E4M3 ? 2 : 1, reinterpret_cast<cudaStream_t>(stream)});
}

}  // extern "C"
