// Host side of the paged-serving entry points (include/fia.h): argument
// validation and launches.  Lengths stay on the device; nothing here waits for
// the GPU or copies to it.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "host.h"
#include "paged.h"

using namespace fia;

namespace {

constexpr int64_t kMaxKeys = int64_t(1) << 30;     // keys of one sequence (tile arithmetic stays in 32 bits)
constexpr int64_t kMaxInt = 2147483647;

// An int32 vector on the device; n < 0: any length.
fia_status check_i32(const fia_tensor* t, int64_t n, const char* name) {
  if (!given(t)) return fail(FIA_ERR_NULL, "%s is required", name);
  if (t->dtype != FIA_DTYPE_I32) return fail(FIA_ERR_DTYPE, "%s must be int32", name);
  if (t->ndim != 1) return fail(FIA_ERR_SHAPE, "%s must be 1-D", name);
  if (n >= 0 && t->shape[0] != n)
    return fail(FIA_ERR_SHAPE, "%s has %lld entries, expected %lld", name, (long long)t->shape[0], (long long)n);
  if (t->shape[0] > kMaxInt) return fail(FIA_ERR_SHAPE, "%s has more than 2^31-1 entries", name);
  if (reinterpret_cast<uintptr_t>(t->data) % 4 != 0) return fail(FIA_ERR_ALIGNMENT, "%s not 4-byte aligned", name);
  return FIA_OK;
}

bool overlap(const void* a, uintptr_t na, const void* b, uintptr_t nb) {   // bytes
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && a0 < b0 + nb && b0 < a0 + na;
}
bool overlap(const fia_tensor* a, const fia_tensor* b) {   // int32 tensors
  return overlap(a->data, uintptr_t(numel(a)) * 4, b->data, uintptr_t(numel(b)) * 4);
}

// The kernels scale scores in log2 units with one fp32 factor, and a hidden
// score is -inf: a factor that is 0 there would make it NaN.
fia_status check_scale(const fia_params* prm) {
  const float f = float(prm->scale_value * 1.4426950408889634);
  if (!(f >= FLT_MIN) || !std::isfinite(f))
    return fail(FIA_ERR_UNSUPPORTED, "scale_value must be > 0 and, times log2(e), a normal fp32 number");
  return FIA_OK;
}

#define FIA_TRY(x)                        \
  do {                                    \
    const fia_status st_ = (x);           \
    if (st_ != FIA_OK) return st_;        \
  } while (0)

int elem_bytes(int32_t dt) { return dt == FIA_DTYPE_F8E4M3 ? 1 : 2; }

// One tensor of fia_cache_write and its pool -> entry y of the launch.
fia_status write_side(const fia_tensor* x, int64_t stride, const fia_tensor* cache, int64_t T, int64_t nblk, int64_t bs,
                      int y, CacheWriteParams& p, const char* name) {
  if (!is_half(x->dtype) && x->dtype != FIA_DTYPE_F8E4M3)
    return fail(FIA_ERR_DTYPE, "%s must be f16, bf16 or e4m3", name);
  if (cache->dtype != x->dtype) return fail(FIA_ERR_DTYPE, "%s and its cache differ in type", name);
  if (x->ndim != 3) return fail(FIA_ERR_SHAPE, "%s must be (T, KV_N, D)", name);
  if (x->shape[0] != T) return fail(FIA_ERR_SHAPE, "%s has %lld tokens, slot_mapping %lld", name, (long long)x->shape[0], (long long)T);
  const int64_t e = elem_bytes(x->dtype), N = x->shape[1], D = x->shape[2];
  if (N <= 0 || D <= 0 || N > kMaxInt / 16 || D > kMaxInt / 16 || N * D * e > kMaxInt)
    return fail(FIA_ERR_SHAPE, "%s: KV_N %lld, D %lld", name, (long long)N, (long long)D);
  if (D * e % 16 != 0) return fail(FIA_ERR_UNSUPPORTED, "%s: rows of a head must be a multiple of 16 bytes", name);
  if (stride == 0) stride = N * D;
  if (stride < 0 || (T > 1 && stride < N * D) || stride * e % 16 != 0)
    return fail(FIA_ERR_ALIGNMENT, "%s: token stride %lld (at least %lld elements, a multiple of 16 bytes)", name,
                (long long)stride, (long long)(N * D));
  const bool bnbd = cache->ndim == 4;
  if (bnbd ? (cache->shape[0] != nblk || cache->shape[1] != N || cache->shape[2] != bs || cache->shape[3] != D)
           : (cache->ndim != 3 || cache->shape[0] != nblk || cache->shape[1] != bs || cache->shape[2] != N * D))
    return fail(FIA_ERR_SHAPE, "%s's cache must be (%lld, KV_N, %lld, D) or (%lld, %lld, KV_N*D) for its heads", name,
                (long long)nblk, (long long)bs, (long long)nblk, (long long)bs);
  if (!aligned16(x->data) || !aligned16(cache->data)) return fail(FIA_ERR_ALIGNMENT, "%s or its cache not 16-byte aligned", name);
  p.src[y] = static_cast<const uint8_t*>(x->data);
  p.dst[y] = static_cast<uint8_t*>(cache->data);
  p.src_row[y] = stride * e;
  p.dst_blk[y] = N * bs * D * e;
  p.dst_row[y] = (bnbd ? D : N * D) * e;
  p.dst_head[y] = (bnbd ? bs * D : D) * e;
  p.vecs[y] = int(N * D * e / 16);
  p.head_vecs[y] = int(D * e / 16);
  return FIA_OK;
}

// Query, cache, length and output arguments shared by the decode entry points.
fia_status span_params(const fia_tensor* q, const fia_tensor* k, const fia_tensor* v, const fia_tensor* table,
                       const fia_tensor* kvlen, const fia_params* prm, const fia_tensor* out, const fia_tensor* lse,
                       SpanParams& p, int64_t& D) {
  memset(&p, 0, sizeof(p));
  if (prm == nullptr) return fail(FIA_ERR_NULL, "params is NULL");
  if (!given(q) || !given(k) || !given(v) || !given(out))
    return fail(FIA_ERR_NULL, "query/key/value/attention_out required");
  const Layout L = parse_layout(prm->input_layout);
  if (L == L_BAD) return fail(FIA_ERR_LAYOUT, "input_layout '%s' not supported", prm->input_layout);
  if (L == L_TND) return fail(FIA_ERR_UNSUPPORTED, "TND decode is not implemented");
  if (!is_half(q->dtype) || k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype)
    return fail(FIA_ERR_DTYPE, "query/key/value/attention_out must share fp16 or bf16");
  if (prm->actual_seq_qlen != nullptr || prm->actual_seq_kvlen != nullptr)
    return fail(FIA_ERR_SEQLEN, "lengths are a device tensor here: params' actual_seq lists must be NULL");
  int64_t N1, N2, B, S;
  FIA_TRY(resolve_heads(prm, N1, N2));
  if (!same_shape(q, out)) return fail(FIA_ERR_SHAPE, "attention_out must have the query's shape");
  FIA_TRY(dense_dims(q, L, N1, B, S, D, "query"));
  if (S < 1 || S > 16) return fail(FIA_ERR_UNSUPPORTED, "decode takes Q_S in 1..16 (got %lld)", (long long)S);
  if (D != 64 && D != 128) return fail(FIA_ERR_UNSUPPORTED, "decode head dim %lld (kernels take 64 or 128)", (long long)D);
  if (N1 / N2 * S > 64)
    return fail(FIA_ERR_UNSUPPORTED, "decode rows per KV head (Q_N / KV_N x Q_S = %lld) above 64", (long long)(N1 / N2 * S));
  FIA_TRY(check_scale(prm));
  if (!same_shape(k, v)) return fail(FIA_ERR_SHAPE, "key and value shapes differ");
  if (!aligned16(q->data) || !aligned16(k->data) || !aligned16(v->data) || !aligned16(out->data))
    return fail(FIA_ERR_ALIGNMENT, "query/key/value/attention_out must be 16-byte aligned");
  if (B > kMaxInt / 16 || N2 > 65535)
    return fail(FIA_ERR_SHAPE, "B = %lld or KV_N = %lld is too large", (long long)B, (long long)N2);
  int64_t S2;
  if (present(table)) {
    if (table->dtype != FIA_DTYPE_I32 || table->ndim != 2 || table->shape[0] != B)
      return fail(FIA_ERR_BLOCK_TABLE, "block_table must be int32 (B, maxBlocksPerSeq)");
    if (reinterpret_cast<uintptr_t>(table->data) % 4 != 0) return fail(FIA_ERR_ALIGNMENT, "block_table not 4-byte aligned");
    const int64_t bs = prm->block_size;
    if (bs <= 0 || bs % 16 != 0 || bs > kMaxKeys)
      return fail(FIA_ERR_BLOCK_TABLE, "block_size %lld: a multiple of 16", (long long)bs);
    const bool bnbd = k->ndim == 4;
    if (bnbd ? (k->shape[1] != N2 || k->shape[2] != bs || k->shape[3] != D)
             : (k->ndim != 3 || k->shape[1] != bs || k->shape[2] != N2 * D))
      return fail(FIA_ERR_SHAPE, "paged key must be (blocknum, KV_N, block_size, D) or (blocknum, block_size, KV_N*D)");
    if (k->shape[0] > kMaxInt) return fail(FIA_ERR_SHAPE, "more than 2^31-1 blocks");
    if (!present(kvlen)) return fail(FIA_ERR_SEQLEN, "page attention needs actual_seq_kvlen");
    S2 = table->shape[1] > kMaxKeys / bs ? kMaxKeys + 1 : table->shape[1] * bs;
    p.block_table = static_cast<const int32_t*>(table->data);
    p.table_stride = table->shape[1];
    p.block_size = int(bs);
    p.n_blocks = int(k->shape[0]);
    p.blk_stride = N2 * bs * D;
    p.head_stride = bnbd ? bs * D : D;
    p.row_stride = bnbd ? D : N2 * D;
  } else {
    if (table != nullptr && table->ndim > 0 && B > 0) {
      // a table without columns: no sequence has a key
      return fail(FIA_ERR_BLOCK_TABLE, "block_table has no entries");
    }
    int64_t Bk, Dk;
    FIA_TRY(dense_dims(k, L, N2, Bk, S2, Dk, "key"));
    if (Bk != B || Dk != D) return fail(FIA_ERR_SHAPE, "key must be (B, ..., D) like the query");
    int64_t st[3];
    bns_strides(L, N2, S2, D, st);
    p.blk_stride = st[0];
    p.head_stride = st[1];
    p.row_stride = st[2];
    p.n_blocks = int(std::min<int64_t>(B, kMaxInt));
    p.block_size = 16;   // not read
  }
  if (S2 > kMaxKeys) return fail(FIA_ERR_SHAPE, "more than 2^30 keys per sequence");
  if (kvlen != nullptr && kvlen->ndim > 0) {
    FIA_TRY(check_i32(kvlen, B, "actual_seq_kvlen"));
    p.kv_len = static_cast<const int32_t*>(kvlen->data);
  }
  FIA_TRY(check_lse(lse, prm, L, B, N1, S, 0));
  int64_t qs[3];
  bns_strides(L, N1, S, D, qs);
  p.q = q->data;
  p.out = out->data;
  p.q_sb = qs[0]; p.q_sn = qs[1]; p.q_ss = qs[2];
  if (prm->softmax_lse_flag != 0) p.lse = static_cast<float*>(lse->data);
  p.lse_sb = N1 * S; p.lse_sn = S; p.lse_ss = 1;
  p.k = k->data;
  p.v = v->data;
  p.kv_max = int(S2);
  p.B = int(B); p.N1 = int(N1); p.N2 = int(N2);
  p.group = int(N1 / N2);
  p.q_tokens = int(S);
  p.rows = int(N1 / N2 * S);
  p.pre = int(std::min<int64_t>(std::max<int64_t>(prm->pre_tokens, 0), kMaxInt));
  p.scale_log2 = float(prm->scale_value * 1.4426950408889634);
  return FIA_OK;
}

// Launches the decode over a visible span.
fia_status run_span(const SpanParams& p, int64_t D, bool bf16, int n_sm, cudaStream_t s) {
  if (span_wide_pays(p, n_sm)) return launch_span_wide(p, int(D), bf16, n_sm, s);
  return cuda_check(launch_span_decode(p, int(D), bf16, n_sm, s), "decode launch");
}

// ... as the call's main kernel (the caller's events around it).
fia_status run_profiled(const SpanParams& p, int64_t D, bool bf16, int n_sm, cudaStream_t s) {
  fia_status st = FIA_OK;
  const cudaError_t e = profiled(s, [&] {
    st = run_span(p, D, bf16, n_sm, s);
    return cudaSuccess;
  });
  return st != FIA_OK ? st : cuda_check(e, "profiling events");
}

// Arguments of fia_prefill_window -> launch parameters without the tensor maps.
struct WindowPrefill {
  PrefillParams p;
  Layout layout;
  int64_t B, N1, N2, S1, S2, D, blocks, bs;
  bool bnbd;
};

fia_status window_prefill(const fia_tensor* q, const fia_tensor* k, const fia_tensor* v, const fia_tensor* table,
                          const fia_tensor* qlen, const fia_tensor* kvlen, const fia_params* prm, int64_t sink,
                          const fia_tensor* out, const fia_tensor* lse, WindowPrefill& w) {
  memset(&w, 0, sizeof(w));
  if (prm == nullptr) return fail(FIA_ERR_NULL, "params is NULL");
  if (!given(q) || !given(k) || !given(v) || !given(out))
    return fail(FIA_ERR_NULL, "query/key/value/attention_out required");
  const Layout L = w.layout = parse_layout(prm->input_layout);
  if (L == L_BAD) return fail(FIA_ERR_LAYOUT, "input_layout '%s' not supported", prm->input_layout);
  if (!is_half(q->dtype) || k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype)
    return fail(FIA_ERR_DTYPE, "query/key/value/attention_out must share fp16 or bf16");
  if (prm->actual_seq_qlen != nullptr || prm->actual_seq_kvlen != nullptr)
    return fail(FIA_ERR_SEQLEN, "lengths are a device tensor here: params' actual_seq lists must be NULL");
  FIA_TRY(resolve_heads(prm, w.N1, w.N2));
  if (!same_shape(q, out)) return fail(FIA_ERR_SHAPE, "attention_out must have the query's shape");
  if (!same_shape(k, v)) return fail(FIA_ERR_SHAPE, "key and value shapes differ");
  FIA_TRY(dense_dims(q, L, w.N1, w.B, w.S1, w.D, "query"));
  if (w.D != 64 && w.D != 128) return fail(FIA_ERR_UNSUPPORTED, "head dim %lld (kernels take 64 or 128)", (long long)w.D);
  FIA_TRY(check_scale(prm));
  if (prm->pre_tokens < 0) return fail(FIA_ERR_UNSUPPORTED, "pre_tokens must be 0 or more");
  if (sink < 0) return fail(FIA_ERR_UNSUPPORTED, "sink_tokens must be 0 or more");
  if (!aligned16(q->data) || !aligned16(k->data) || !aligned16(v->data) || !aligned16(out->data))
    return fail(FIA_ERR_ALIGNMENT, "query/key/value/attention_out must be 16-byte aligned");
  const bool tnd = L == L_TND, lens_q = qlen != nullptr && qlen->ndim > 0, lens_k = kvlen != nullptr && kvlen->ndim > 0;
  if (tnd) {
    if (!lens_q) return fail(FIA_ERR_SEQLEN, "actual_seq_qlen is required for TND");
    FIA_TRY(check_i32(qlen, -1, "actual_seq_qlen"));
    w.B = qlen->shape[0];
    if (w.B > 4096) return fail(FIA_ERR_SEQLEN, "actual_seq_qlen has %lld entries (> 4096)", (long long)w.B);
  } else if (lens_q) {
    FIA_TRY(check_i32(qlen, w.B, "actual_seq_qlen"));
  }
  const bool paged = table != nullptr && table->ndim > 0;
  if (paged) {
    if (table->dtype != FIA_DTYPE_I32 || table->ndim != 2 || table->shape[0] != w.B || !given(table) || table->shape[1] < 1)
      return fail(FIA_ERR_BLOCK_TABLE, "block_table must be int32 (B, maxBlocksPerSeq)");
    if (reinterpret_cast<uintptr_t>(table->data) % 4 != 0) return fail(FIA_ERR_ALIGNMENT, "block_table not 4-byte aligned");
    if (!lens_k) return fail(FIA_ERR_SEQLEN, "page attention needs actual_seq_kvlen");
    w.bs = prm->block_size;
    if (w.bs < 128 || w.bs > 512 || w.bs % 128 != 0)
      return fail(FIA_ERR_BLOCK_TABLE, "block_size %lld: 128..512, a multiple of 128", (long long)w.bs);
    w.bnbd = k->ndim == 4;
    if (w.bnbd ? (k->shape[1] != w.N2 || k->shape[2] != w.bs || k->shape[3] != w.D)
               : (k->ndim != 3 || k->shape[1] != w.bs || k->shape[2] != w.N2 * w.D))
      return fail(FIA_ERR_SHAPE, "paged key must be (blocknum, KV_N, block_size, D) or (blocknum, block_size, KV_N*D)");
    w.blocks = k->shape[0];
    w.S2 = table->shape[1] > kMaxKeys / w.bs ? kMaxKeys + 1 : table->shape[1] * w.bs;
    FIA_TRY(check_i32(kvlen, w.B, "actual_seq_kvlen"));
  } else {
    int64_t Bk, Dk;
    FIA_TRY(dense_dims(k, L, w.N2, Bk, w.S2, Dk, "key"));
    if (Dk != w.D || (!tnd && Bk != w.B)) return fail(FIA_ERR_SHAPE, "key must be (B, ..., D) like the query");
    if (tnd && !lens_k) return fail(FIA_ERR_SEQLEN, "actual_seq_kvlen is required for TND");
    if (lens_k) FIA_TRY(check_i32(kvlen, w.B, "actual_seq_kvlen"));
  }
  if (w.S1 > kMaxKeys || w.S2 > kMaxKeys) return fail(FIA_ERR_SHAPE, "more than 2^30 rows or keys");
  FIA_TRY(check_lse(lse, prm, L, w.B, w.N1, w.S1, w.S1));
  PrefillParams& p = w.p;
  int64_t os[3];
  bns_strides(L, w.N1, w.S1, w.D, os);
  p.out = out->data;
  p.out_sb = os[0]; p.out_sn = os[1]; p.out_ss = os[2];
  if (prm->softmax_lse_flag != 0) p.lse = static_cast<float*>(lse->data);
  p.lse_sb = tnd ? 0 : w.N1 * w.S1;
  p.lse_sn = tnd ? 1 : w.S1;
  p.lse_ss = tnd ? w.N1 : 1;
  // pairs of query tiles: TND has at most one part-filled pair a batch
  const int64_t pairs = tnd ? w.S1 / (2 * kTileM) + std::min(w.B, w.S1) : w.B * ((w.S1 + 2 * kTileM - 1) / (2 * kTileM));
  if (pairs * w.N1 > kMaxKeys) return fail(FIA_ERR_SHAPE, "query is too large");
  p.n_items = int(pairs * w.N1);
  p.num_heads = int(w.N1);
  p.num_kv_heads = int(w.N2);
  p.group = int(w.N1 / w.N2);
  p.is_tnd = tnd;
  p.band_pre = int(std::min<int64_t>(prm->pre_tokens, kMaxKeys));
  p.sink = int(std::min<int64_t>(sink, w.S2));
  p.q_lens = lens_q ? static_cast<const int32_t*>(qlen->data) : nullptr;
  p.kv_lens = lens_k ? static_cast<const int32_t*>(kvlen->data) : nullptr;
  p.n_batch = int(w.B);
  p.s1 = int(w.S1);
  p.s2 = int(w.S2);
  p.scale_log2 = float(prm->scale_value * 1.4426950408889634);
  if (paged) {
    p.block_table = static_cast<const int32_t*>(table->data);
    p.table_stride = table->shape[1];
    p.block_size = int(w.bs);
    p.n_blocks = int(std::min<int64_t>(w.blocks, kMaxInt));
  }
  return FIA_OK;
}

std::atomic<int> g_prefix_path{0};   // fia_debug_set_prefix_path

// Whether the prefix gets a kernel of its own: where reading it for every
// sequence costs more than that kernel's start, partial results (which grow with
// a unit's rows) and join.  (us, apart and by every sequence, by the bytes read
// again: 4 rows, 6 MB 12.8, 7.6; 24 MB 14.4, 12.6; 30 MB 11.9, 10.5; 56 MB 12.2,
// 13.7; 120 MB 13.4, 22.7; 32 rows, 14 MB 18.7, 10.7; 56 MB 20.4, 15.8; 120 MB 25.2,
// 22.6; 248 MB 34.8, 35.5.  Of a long prefix a sequence's few CTAs read too much each:
// 8192 keys, one kv head, 4 MB 10.5, 12.2.)
bool prefix_apart(const SpanParams& p, int64_t prefix, int64_t D) {
  const int path = g_prefix_path.load(std::memory_order_relaxed);
  if (prefix == 0 || p.B < 2) return false;   // one sequence shares with nobody
  if (path != 0) return path == 1;
  return prefix > 4096 || (p.B - 1) * prefix * p.N2 * D * 4 > (int64_t(16 + 4 * p.rows) << 20);
}

// How fia_decode_shared_prefix cuts its work.
struct PrefixPlan {
  bool split_off = false;   // a kernel for the prefix, joined by the decode of the rest
  int tile_batches = 0, n_pairs = 0, n_splits = 0;
  int64_t rows = 0;         // rows of one split's partial results
  size_t off_ml = 0, bytes = kHeader;
};

// The prefix kernel's grid: (pairs of 128-row tiles) x kv heads x splits of
// the prefix's 128-key tiles, one CTA per SM.  The split count is the one
// whose waves of CTAs take the least time, a CTA costing its tiles and about
// three more (start, first loads, partial results).
PrefixPlan prefix_plan(const SpanParams& p, int64_t prefix, int64_t D, int n_sm) {
  PrefixPlan w;
  if (prefix == 0 || p.B < 2 || p.n_blocks == 0) return w;   // (one sequence shares with nobody, and nothing is read)
  w.split_off = true;
  w.tile_batches = kTileM / p.rows;
  const int64_t row_tiles = (p.B + w.tile_batches - 1) / w.tile_batches;
  w.n_pairs = int((row_tiles + 1) / 2);
  const int64_t per = int64_t(w.n_pairs) * p.N2, tiles = (prefix + kTileN - 1) / kTileN;
  constexpr int kStart = 3, kMostSplits = 64;
  int64_t best = 0;
  for (int s = 1; s <= std::min<int64_t>(tiles, kMostSplits); ++s) {
    const int64_t cost = (per * s + n_sm - 1) / n_sm * ((tiles + s - 1) / s + kStart);
    if (w.n_splits == 0 || cost < best) {
      best = cost;
      w.n_splits = s;
    }
  }
  w.rows = int64_t(p.B) * p.N1 * p.q_tokens;
  w.off_ml = kHeader + align_up(size_t(w.n_splits) * size_t(w.rows) * size_t(D) * sizeof(float), 256);
  w.bytes = w.off_ml + align_up(size_t(w.n_splits) * size_t(w.rows) * sizeof(float2), 256);
  return w;
}

fia_status prefix_args(const fia_tensor* q, const fia_tensor* k, const fia_tensor* v, const fia_tensor* table,
                       const fia_tensor* kvlen, const fia_params* prm, int64_t prefix, const fia_tensor* out,
                       const fia_tensor* lse, SpanParams& p, int64_t& D) {
  FIA_TRY(span_params(q, k, v, table, kvlen, prm, out, lse, p, D));
  if (p.block_table == nullptr) return fail(FIA_ERR_BLOCK_TABLE, "a shared prefix needs block_table");
  if (p.block_size % 128 != 0 && 128 % p.block_size != 0)
    return fail(FIA_ERR_BLOCK_TABLE, "block_size %d: a multiple of 16 that divides 128, or a multiple of 128", p.block_size);
  if (prefix < 0 || prefix > p.kv_max || prefix % p.block_size != 0)
    return fail(FIA_ERR_SEQLEN, "shared_prefix_len %lld: a multiple of block_size in [0, %d]", (long long)prefix, p.kv_max);
  p.pre = int(kMaxInt);
  return FIA_OK;
}

}  // namespace

extern "C" {

fia_status fia_block_table_append(const fia_tensor* context_lens, const fia_tensor* new_lens,
                                  const fia_tensor* free_blocks, int64_t block_size, const fia_tensor* block_table,
                                  const fia_tensor* slot_mapping, const fia_tensor* kv_lens,
                                  const fia_tensor* cu_new_lens, const fia_tensor* num_blocks, void* stream) {
  FIA_TRY(check_i32(context_lens, -1, "context_lens"));
  const int64_t B = context_lens->shape[0];
  FIA_TRY(check_i32(new_lens, B, "new_lens"));
  FIA_TRY(check_i32(free_blocks, -1, "free_blocks"));
  FIA_TRY(check_i32(slot_mapping, -1, "slot_mapping"));
  FIA_TRY(check_i32(kv_lens, B, "kv_lens"));
  FIA_TRY(check_i32(cu_new_lens, B, "cu_new_lens"));
  FIA_TRY(check_i32(num_blocks, 1, "num_blocks"));
  if (!given(block_table)) return fail(FIA_ERR_NULL, "block_table is required");
  if (block_table->dtype != FIA_DTYPE_I32) return fail(FIA_ERR_DTYPE, "block_table must be int32");
  if (block_table->ndim != 2 || block_table->shape[0] != B || block_table->shape[1] > kMaxInt)
    return fail(FIA_ERR_BLOCK_TABLE, "block_table must be (B, columns)");
  if (reinterpret_cast<uintptr_t>(block_table->data) % 4 != 0)
    return fail(FIA_ERR_ALIGNMENT, "block_table not 4-byte aligned");
  if (block_size < 1 || block_size > kMaxInt) return fail(FIA_ERR_BLOCK_TABLE, "block_size %lld", (long long)block_size);
  const fia_tensor* ins[] = {context_lens, new_lens, free_blocks};
  const fia_tensor* outs[] = {block_table, slot_mapping, kv_lens, cu_new_lens, num_blocks};
  for (int i = 0; i < 5; ++i) {
    for (const fia_tensor* t : ins)
      if (overlap(outs[i], t)) return fail(FIA_ERR_UNSUPPORTED, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(FIA_ERR_UNSUPPORTED, "two outputs overlap");
  }
  TableParams p;
  memset(&p, 0, sizeof(p));
  p.context_lens = static_cast<const int32_t*>(context_lens->data);
  p.new_lens = static_cast<const int32_t*>(new_lens->data);
  p.free_blocks = static_cast<const int32_t*>(free_blocks->data);
  p.block_table = static_cast<int32_t*>(block_table->data);
  p.slot_mapping = static_cast<int32_t*>(slot_mapping->data);
  p.kv_lens = static_cast<int32_t*>(kv_lens->data);
  p.cu_new_lens = static_cast<int32_t*>(cu_new_lens->data);
  p.num_blocks = static_cast<int32_t*>(num_blocks->data);
  p.B = int(B);
  p.n_free = int(free_blocks->shape[0]);
  p.table_cols = int(block_table->shape[1]);
  p.n_tokens = int(slot_mapping->shape[0]);
  p.block_size = int(block_size);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s, [&] { return launch_block_table(p, s); }), "block table launch");
}

fia_status fia_cache_write(const fia_tensor* key, int64_t key_token_stride, const fia_tensor* value,
                           int64_t value_token_stride, const fia_tensor* key_cache, const fia_tensor* value_cache,
                           const fia_tensor* slot_mapping, void* stream) {
  if (!given(key) || !given(key_cache)) return fail(FIA_ERR_NULL, "key and key_cache are required");
  const bool two = value != nullptr && value->ndim > 0;
  if (two != (value_cache != nullptr && value_cache->ndim > 0))
    return fail(FIA_ERR_NULL, "value and value_cache must be given together");
  if (two && (!given(value) || !given(value_cache))) return fail(FIA_ERR_NULL, "value or value_cache has no data");
  FIA_TRY(check_i32(slot_mapping, -1, "slot_mapping"));
  const int64_t T = slot_mapping->shape[0];
  if (key_cache->ndim != 3 && key_cache->ndim != 4) return fail(FIA_ERR_SHAPE, "key_cache must be 3-D or 4-D");
  const int64_t nblk = key_cache->shape[0], bs = key_cache->ndim == 4 ? key_cache->shape[2] : key_cache->shape[1];
  if (bs < 1 || bs > kMaxInt) return fail(FIA_ERR_BLOCK_TABLE, "block_size %lld", (long long)bs);
  CacheWriteParams p;
  memset(&p, 0, sizeof(p));
  FIA_TRY(write_side(key, key_token_stride, key_cache, T, nblk, bs, 0, p, "key"));
  if (two) FIA_TRY(write_side(value, value_token_stride, value_cache, T, nblk, bs, 1, p, "value"));
  if (T == 0 || nblk == 0) return FIA_OK;
  // (a row read while another token's is written over it would be a mixture)
  for (int y = 0; y < (two ? 2 : 1); ++y) {
    const uintptr_t pool = uintptr_t(nblk) * uintptr_t(p.dst_blk[y]);
    for (int x = 0; x < (two ? 2 : 1); ++x)
      if (overlap(p.src[x], uintptr_t(T - 1) * uintptr_t(p.src_row[x]) + uintptr_t(p.vecs[x]) * 16, p.dst[y], pool))
        return fail(FIA_ERR_UNSUPPORTED, "key or value overlaps a cache");
    if (y == 1 && overlap(p.dst[0], uintptr_t(nblk) * uintptr_t(p.dst_blk[0]), p.dst[1], pool))
      return fail(FIA_ERR_UNSUPPORTED, "key_cache and value_cache overlap");
  }
  p.slots = static_cast<const int32_t*>(slot_mapping->data);
  p.n_slots = nblk > kMaxInt / bs ? kMaxInt : nblk * bs;
  p.n_tokens = int(T);
  p.block_size = int(bs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s, [&] { return launch_cache_write(p, s); }), "cache write launch");
}

fia_status fia_decode_window(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                             const fia_tensor* block_table, const fia_tensor* actual_seq_kvlen,
                             const fia_params* params, int64_t sink_tokens, const fia_tensor* attention_out,
                             const fia_tensor* softmax_lse, void* stream) {
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;   // empty query
  SpanParams p;
  int64_t D;
  FIA_TRY(span_params(query, key, value, block_table, actual_seq_kvlen, params, attention_out, softmax_lse, p, D));
  if (params->pre_tokens < 0) return fail(FIA_ERR_UNSUPPORTED, "pre_tokens must be 0 or more");
  if (sink_tokens < 0) return fail(FIA_ERR_UNSUPPORTED, "sink_tokens must be 0 or more");
  p.sink = int(std::min<int64_t>(sink_tokens, p.kv_max));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return run_profiled(p, D, query->dtype == FIA_DTYPE_BF16, sm_count(), s);
}

fia_status fia_prefill_window_get_workspace_size(const fia_tensor* query, const fia_tensor* key,
                                                 const fia_tensor* value, const fia_tensor* block_table,
                                                 const fia_tensor* actual_seq_qlen,
                                                 const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                                 int64_t sink_tokens, const fia_tensor* attention_out,
                                                 const fia_tensor* softmax_lse, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return fail(FIA_ERR_NULL, "workspace_bytes is NULL");
  *workspace_bytes = kHeader;
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;   // empty query
  WindowPrefill w;
  return window_prefill(query, key, value, block_table, actual_seq_qlen, actual_seq_kvlen, params, sink_tokens,
                        attention_out, softmax_lse, w);
}

fia_status fia_prefill_window(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                              const fia_tensor* block_table, const fia_tensor* actual_seq_qlen,
                              const fia_tensor* actual_seq_kvlen, const fia_params* params, int64_t sink_tokens,
                              const fia_tensor* attention_out, const fia_tensor* softmax_lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;
  WindowPrefill w;
  FIA_TRY(window_prefill(query, key, value, block_table, actual_seq_qlen, actual_seq_kvlen, params, sink_tokens,
                         attention_out, softmax_lse, w));
  FIA_TRY(check_ws(workspace, workspace_bytes, kHeader));
  if (w.p.n_items == 0) return FIA_OK;   // a TND query without sequences
  PrefillParams& p = w.p;
  const int64_t Bmap = w.layout == L_TND ? 1 : w.B;
  FIA_TRY(dense_map(&p.tm_q, query, w.layout, Bmap, w.N1, w.S1, w.D));
  if (numel(key) == 0) {
    // K/V without a row are not read (every id of a pool without a block lies
    // outside it), but a map wants an extent
    p.tm_k = p.tm_v = p.tm_q;
    if (p.block_table == nullptr) {
      p.kv_lens = nullptr;
      p.s2 = 0;
    }
  } else if (p.block_table != nullptr) {
    const Layout pl = w.bnbd ? L_BNSD : L_BSND;
    FIA_TRY(dense_map(&p.tm_k, key, pl, w.blocks, w.N2, w.bs, w.D));
    FIA_TRY(dense_map(&p.tm_v, value, pl, w.blocks, w.N2, w.bs, w.D));
  } else {
    FIA_TRY(dense_map(&p.tm_k, key, w.layout, Bmap, w.N2, w.S2, w.D));
    FIA_TRY(dense_map(&p.tm_v, value, w.layout, Bmap, w.N2, w.S2, w.D));
  }
  p.tm_qr = p.tm_q;
  p.tm_kr = p.tm_k;
  p.rope_col = 128;
  p.status = make_status(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s,
                             [&] {
                               return launch_prefill_window(p, int(w.D), query->dtype == FIA_DTYPE_BF16, sm_count(), s);
                             }),
                    "window prefill launch");
}

void fia_debug_set_prefix_path(int32_t path) { g_prefix_path.store(path, std::memory_order_relaxed); }

fia_status fia_decode_shared_prefix_get_workspace_size(const fia_tensor* query, const fia_tensor* key_cache,
                                                       const fia_tensor* value_cache, const fia_tensor* block_table,
                                                       const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                                       int64_t shared_prefix_len, const fia_tensor* attention_out,
                                                       const fia_tensor* softmax_lse, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return fail(FIA_ERR_NULL, "workspace_bytes is NULL");
  *workspace_bytes = kHeader;
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;   // empty query
  SpanParams p;
  int64_t D;
  FIA_TRY(prefix_args(query, key_cache, value_cache, block_table, actual_seq_kvlen, params, shared_prefix_len,
                      attention_out, softmax_lse, p, D));
  *workspace_bytes = prefix_plan(p, shared_prefix_len, D, sm_count()).bytes;
  return FIA_OK;
}

fia_status fia_decode_shared_prefix(const fia_tensor* query, const fia_tensor* key_cache,
                                    const fia_tensor* value_cache, const fia_tensor* block_table,
                                    const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                    int64_t shared_prefix_len, const fia_tensor* attention_out,
                                    const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;
  SpanParams p;
  int64_t D;
  FIA_TRY(prefix_args(query, key_cache, value_cache, block_table, actual_seq_kvlen, params, shared_prefix_len,
                      attention_out, softmax_lse, p, D));
  const int n_sm = sm_count();
  const PrefixPlan w = prefix_plan(p, shared_prefix_len, D, n_sm);
  FIA_TRY(check_ws(workspace, workspace_bytes, w.bytes));
  const bool bf16 = query->dtype == FIA_DTYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  if (!w.split_off || !prefix_apart(p, shared_prefix_len, D)) {
    p.status = make_status(workspace);
    p.shared = int(shared_prefix_len);
    return run_profiled(p, D, bf16, n_sm, s);
  }
  PrefillParams pp;
  memset(&pp, 0, sizeof(pp));
  {
    // query rows of a (batch, kv head): tokens, and within a token the heads of
    // the group; one box holds tile_batches sequences
    const uint64_t e = 2, g = uint64_t(p.group), Q = uint64_t(p.q_tokens);
    const uint64_t dims[5] = {uint64_t(D), g, Q, uint64_t(p.N2), uint64_t(p.B)};
    const uint64_t st[4] = {uint64_t(p.q_sn) * e, uint64_t(p.q_ss) * e, uint64_t(p.q_sn) * g * e, uint64_t(p.q_sb) * e};
    const uint32_t box[5] = {64, uint32_t(g), uint32_t(Q), 1, uint32_t(w.tile_batches)};
    FIA_TRY(make_map(&pp.tm_q, query->data, 5, dims, st, 0, false, box));
    // the pools as (D, block_size, KV_N, blocknum)
    const uint64_t kd[4] = {uint64_t(D), uint64_t(p.block_size), uint64_t(p.N2), uint64_t(p.n_blocks)};
    const uint64_t ks[3] = {uint64_t(p.row_stride) * e, uint64_t(p.head_stride) * e, uint64_t(p.blk_stride) * e};
    pp.box_rows = std::min(p.block_size, kTileN);
    FIA_TRY(make_map(&pp.tm_k, p.k, 4, kd, ks, uint32_t(pp.box_rows)));
    FIA_TRY(make_map(&pp.tm_v, p.v, 4, kd, ks, uint32_t(pp.box_rows)));
    pp.tm_qr = pp.tm_q;
    pp.tm_kr = pp.tm_k;
  }
  pp.num_heads = p.N1;
  pp.num_kv_heads = p.N2;
  pp.group = p.group;
  pp.block_table = p.block_table;
  pp.table_stride = p.table_stride;
  pp.block_size = p.block_size;
  pp.scale_log2 = p.scale_log2;
  pp.kv_lens = p.kv_len;
  pp.n_batch = p.B;
  pp.s2 = int(shared_prefix_len);
  pp.kv_max = p.kv_max;
  pp.q_tokens = p.q_tokens;
  pp.tile_batches = w.tile_batches;
  pp.n_pairs = w.n_pairs;
  pp.n_splits = w.n_splits;
  pp.part_o = reinterpret_cast<float*>(base + kHeader);
  pp.part_ml = reinterpret_cast<float2*>(base + w.off_ml);
  pp.part_rows = w.rows;
  pp.n_items = w.n_pairs * p.N2 * w.n_splits;
  pp.status = make_status(workspace);
  FIA_TRY(cuda_check(profiled(s, [&] { return launch_prefill_pair(pp, int(D), int(D), bf16, kPrefix, s); }),
                     "prefix launch"));
  p.status = pp.status;
  p.base = int(shared_prefix_len);
  p.part_o = pp.part_o;
  p.part_ml = pp.part_ml;
  p.n_parts = w.n_splits;
  p.part_rows = w.rows;
  return run_span(p, D, bf16, n_sm, s);
}

}  // extern "C"
