// Host side of the 4-bit cache's entry points (include/fia.h): argument
// validation and launches.  As in paged_api.cu nothing here waits for the GPU or
// copies to it.
#include <algorithm>
#include <cstring>

#include "paged_host.h"

using namespace fia;

namespace {

// A pool of the 4-bit cache: codes and (step, low) pairs.
struct Int4Pool {
  int64_t blocks, N, bs, D, groups;
  int32_t dtype;
  bool bnbd;
  int64_t blk, row, head;         // bytes of codes between blocks, slots of a block, heads
  int64_t code_bytes, scale_bytes;
};

fia_status int4_pool(const fia_tensor* codes, const fia_tensor* scales, const char* name, Int4Pool& o) {
  if (!given(codes) || !given(scales)) return fail(FIA_ERR_NULL, "%s's codes and scales are required", name);
  if (codes->dtype != FIA_DTYPE_U8) return fail(FIA_ERR_DTYPE, "%s's codes must be uint8", name);
  if (!is_half(scales->dtype)) return fail(FIA_ERR_DTYPE, "%s's scales must be fp16 or bf16", name);
  if (scales->ndim != 5 || scales->shape[4] != 2)
    return fail(FIA_ERR_SHAPE, "%s's scales must be (blocknum, KV_N, block_size, groups, 2)", name);
  o.blocks = scales->shape[0];
  o.N = scales->shape[1];
  o.bs = scales->shape[2];
  o.groups = scales->shape[3];
  o.dtype = scales->dtype;
  if (o.bs < 1 || o.bs > kMaxInt) return fail(FIA_ERR_BLOCK_TABLE, "%s: block_size %lld", name, (long long)o.bs);
  if (o.N < 1 || o.N > 65535) return fail(FIA_ERR_SHAPE, "%s: KV_N = %lld", name, (long long)o.N);
  if (o.blocks > kMaxInt) return fail(FIA_ERR_SHAPE, "%s: more than 2^31-1 blocks", name);
  o.bnbd = codes->ndim == 4;
  if (codes->ndim != 3 && codes->ndim != 4) return fail(FIA_ERR_SHAPE, "%s's codes must be 3-D or 4-D", name);
  o.D = o.bnbd ? codes->shape[3] * 2 : codes->shape[2] * 2 / o.N;
  if (o.bnbd ? (codes->shape[0] != o.blocks || codes->shape[1] != o.N || codes->shape[2] != o.bs)
             : (codes->shape[0] != o.blocks || codes->shape[1] != o.bs || codes->shape[2] * 2 != o.N * o.D))
    return fail(FIA_ERR_SHAPE, "%s's codes must be (blocknum, KV_N, block_size, D/2) or (blocknum, block_size, KV_N*D/2) of its scales", name);
  if (o.D != 64 && o.D != 128) return fail(FIA_ERR_UNSUPPORTED, "%s: head dim %lld (kernels take 64 or 128)", name, (long long)o.D);
  if (o.groups != 1 && o.groups != 2 && !(o.groups == 4 && o.D == 128))
    return fail(FIA_ERR_UNSUPPORTED, "%s: %lld groups of a row of %lld (groups of 32, 64 or 128 values)", name,
                (long long)o.groups, (long long)o.D);
  if (!aligned16(codes->data) || !aligned16(scales->data))
    return fail(FIA_ERR_ALIGNMENT, "%s's codes and scales must be 16-byte aligned", name);
  o.row = o.bnbd ? o.D / 2 : o.N * o.D / 2;
  o.head = o.bnbd ? o.bs * o.D / 2 : o.D / 2;
  o.blk = o.N * o.bs * o.D / 2;
  o.code_bytes = o.blocks * o.blk;
  o.scale_bytes = o.blocks * o.N * o.bs * o.groups * 4;
  return FIA_OK;
}

bool same_pool(const Int4Pool& a, const Int4Pool& b) {
  return a.blocks == b.blocks && a.N == b.N && a.bs == b.bs && a.D == b.D && a.groups == b.groups && a.dtype == b.dtype &&
         a.bnbd == b.bnbd;
}

// The pools of a call: keys, and values where they are given.
fia_status int4_pools(const fia_tensor* kc, const fia_tensor* vc, const fia_tensor* ks, const fia_tensor* vs, bool two,
                      Int4Pool& o) {
  FIA_TRY(int4_pool(kc, ks, "key_cache", o));
  if (!two) return FIA_OK;
  Int4Pool v;
  FIA_TRY(int4_pool(vc, vs, "value_cache", v));
  if (!same_pool(o, v)) return fail(FIA_ERR_SHAPE, "key_cache and value_cache differ in shape, groups or type");
  return FIA_OK;
}

int log2_of(int64_t x) {   // -1: no power of two
  for (int k = 0; k < 31; ++k)
    if (x == int64_t(1) << k) return k;
  return -1;
}

bool there(const fia_tensor* t) { return t != nullptr && t->ndim > 0; }

struct Range {
  const void* p;
  uintptr_t n;
};

fia_status decode_args(const fia_tensor* query, const fia_tensor* key_cache, const fia_tensor* value_cache,
                       const fia_tensor* key_scales, const fia_tensor* value_scales, const fia_tensor* block_table,
                       const fia_tensor* actual_seq_kvlen, const fia_params* params, int64_t sink_tokens,
                       const fia_tensor* attention_out, const fia_tensor* softmax_lse, Int4SpanParams& p, Int4Pool& o) {
  if (params == nullptr) return fail(FIA_ERR_NULL, "params is NULL");
  if (!given(query) || !given(attention_out)) return fail(FIA_ERR_NULL, "query/attention_out required");
  memset(&p, 0, sizeof(p));
  SpanShape d;
  FIA_TRY(span_query(query, params, attention_out, p.s, d));
  FIA_TRY(int4_pools(key_cache, value_cache, key_scales, value_scales, true, o));
  if (o.dtype != query->dtype) return fail(FIA_ERR_DTYPE, "the scales must have the query's type");
  if (o.N != d.N2 || o.D != d.D || o.bs != params->block_size)
    return fail(FIA_ERR_SHAPE, "the caches hold %lld heads of %lld in blocks of %lld; the call has %lld, %lld, %lld",
                (long long)o.N, (long long)o.D, (long long)o.bs, (long long)d.N2, (long long)d.D, (long long)params->block_size);
  if (o.blocks * o.bs > int64_t(0xfffffffe) / o.N) return fail(FIA_ERR_SHAPE, "more than 2^32-2 rows in the caches");
  if (!present(block_table)) return fail(FIA_ERR_BLOCK_TABLE, "block_table is required");
  int64_t room;
  FIA_TRY(span_pages(block_table, params, o.blocks, actual_seq_kvlen, d, p.s, room));
  FIA_TRY(span_rest(actual_seq_kvlen, params, softmax_lse, d, room, p.s));
  if (params->pre_tokens < 0) return fail(FIA_ERR_UNSUPPORTED, "pre_tokens must be 0 or more");
  if (sink_tokens < 0) return fail(FIA_ERR_UNSUPPORTED, "sink_tokens must be 0 or more");
  p.s.sink = int(std::min<int64_t>(sink_tokens, p.s.kv_max));
  p.s.blk_stride = o.blk;
  p.s.row_stride = o.row;
  p.s.head_stride = o.head;
  p.kc = static_cast<const uint8_t*>(key_cache->data);
  p.vc = static_cast<const uint8_t*>(value_cache->data);
  p.ks = static_cast<const uint8_t*>(key_scales->data);
  p.vs = static_cast<const uint8_t*>(value_scales->data);
  return FIA_OK;
}

// Work shared evenly (int4_decode.cuh), where there is enough of it: bytes 0 for no.
struct SplitPlan {
  int ctas, begin;
  size_t ml, heads, bytes;
};

// A unit to a cluster leaves SMs to wait for the longest one; even shares need a
// scan of the lengths first and a second kernel, which joins what they cut.  (us, clusters
// and shares, by the tiles that a group has with all keys, tables as wide as the longest
// sequence: 4 13.4 21.5; 13 16.5 17.2; 27 20.9 22.6; 54, equal lengths, 73 72; 108, equal
// lengths, 94 95; 215, lengths of 1 to 80, 124 94; 431, 1 to 36, 230 210.)
SplitPlan split_plan(const SpanParams& p, const Int4Pool& o, int n_sm) {
  constexpr int64_t kLeast = 32;   // tiles of 16 keys for a group of warps, with all keys that the tables hold
  const Int4Shape c = int4_shape(p.rows, int(o.groups));
  // What a unit's start costs, in chunks (1, 2, 3, 4, 6, 8, 12 of them, us: 16 units of 64 rows and 100 to 8192 keys, on
  // tcgen05, 105 88 75 70 62 63 65; 64 of 16 rows behind a window 99 94 91 91 92 94 96; 64 of 4 rows and up to 32768 keys
  // 197 194 192 191 192 194 199)
  SplitPlan w = {c.resident * n_sm, p.rows > 32 && o.groups == 1 ? 7 : 4, 0, 0, 0};
  const int64_t span = std::min<int64_t>(p.kv_max, int64_t(p.sink) + p.pre + p.q_tokens);
  if (double(p.B) * p.N2 * double(span / 16) < double(kLeast * w.ctas * c.groups) || p.N2 > w.ctas / 4) return w;
  w.ctas -= w.ctas % p.N2;         // whole shares, a CTA a head
  const size_t slots = size_t(2) * w.ctas * p.rows;
  w.ml = align_up(slots * size_t(o.D) * 4, 256);
  w.heads = w.ml + align_up(slots * 8, 256);
  w.bytes = w.heads + align_up(size_t(w.ctas) * 16, 256);
  return w;
}

}  // namespace

extern "C" {

fia_status fia_cache_write_int4(const fia_tensor* key, int64_t key_token_stride, const fia_tensor* value,
                                int64_t value_token_stride, const fia_tensor* key_cache, const fia_tensor* value_cache,
                                const fia_tensor* key_scales, const fia_tensor* value_scales,
                                const fia_tensor* slot_mapping, void* stream) {
  if (!given(key)) return fail(FIA_ERR_NULL, "key is required");
  const bool two = there(value);
  if (two != there(value_cache) || two != there(value_scales))
    return fail(FIA_ERR_NULL, "value, value_cache and value_scales must be given together");
  if (two && !given(value)) return fail(FIA_ERR_NULL, "value has no data");
  FIA_TRY(check_i32(slot_mapping, -1, "slot_mapping"));
  Int4Pool o;
  FIA_TRY(int4_pools(key_cache, value_cache, key_scales, value_scales, two, o));
  Int4WriteParams p;
  memset(&p, 0, sizeof(p));
  const int64_t T = slot_mapping->shape[0];
  const int n = two ? 2 : 1;
  for (int y = 0; y < n; ++y) {
    const fia_tensor* x = y ? value : key;
    const char* name = y ? "value" : "key";
    int64_t stride = y ? value_token_stride : key_token_stride;
    if (x->dtype != o.dtype) return fail(FIA_ERR_DTYPE, "%s must have its scales' type", name);
    if (x->ndim != 3 || x->shape[0] != T || x->shape[1] != o.N || x->shape[2] != o.D)
      return fail(FIA_ERR_SHAPE, "%s must be (T, KV_N, D) = (%lld, %lld, %lld)", name, (long long)T, (long long)o.N, (long long)o.D);
    if (stride == 0) stride = o.N * o.D;
    if (stride < 0 || (T > 1 && stride < o.N * o.D) || stride % 8 != 0)
      return fail(FIA_ERR_ALIGNMENT, "%s: token stride %lld (at least %lld elements, a multiple of 16 bytes)", name,
                  (long long)stride, (long long)(o.N * o.D));
    if (!aligned16(x->data)) return fail(FIA_ERR_ALIGNMENT, "%s not 16-byte aligned", name);
    p.src[y] = static_cast<const uint8_t*>(x->data);
    p.src_row[y] = stride * 2;
    p.dst[y] = static_cast<uint8_t*>((y ? value_cache : key_cache)->data);
    p.scales[y] = static_cast<uint32_t*>((y ? value_scales : key_scales)->data);
  }
  if (T > kMaxInt - 15) return fail(FIA_ERR_SHAPE, "more than 2^31-16 tokens");   // (the kernel counts them in 32 bits)
  if (T == 0 || o.blocks == 0) return FIA_OK;
  // (a row read while another token's is written over it would be a mixture)
  Range outs[4];
  for (int y = 0; y < n; ++y) {
    outs[2 * y] = {p.dst[y], uintptr_t(o.code_bytes)};
    outs[2 * y + 1] = {p.scales[y], uintptr_t(o.scale_bytes)};
  }
  for (int i = 0; i < 2 * n; ++i) {
    for (int y = 0; y < n; ++y)
      if (overlap(p.src[y], uintptr_t(T - 1) * uintptr_t(p.src_row[y]) + uintptr_t(o.N * o.D) * 2, outs[i].p, outs[i].n))
        return fail(FIA_ERR_UNSUPPORTED, "key or value overlaps a cache or its scales");
    if (overlap(slot_mapping->data, uintptr_t(T) * 4, outs[i].p, outs[i].n))
      return fail(FIA_ERR_UNSUPPORTED, "slot_mapping overlaps a cache or its scales");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[j].p, outs[j].n, outs[i].p, outs[i].n))
        return fail(FIA_ERR_UNSUPPORTED, "two of the caches and their scales overlap");
  }
  p.dst_blk = o.blk;
  p.dst_row = o.row;
  p.dst_head = o.head;
  p.slots = static_cast<const int32_t*>(slot_mapping->data);
  p.n_slots = o.blocks > kMaxInt / o.bs ? kMaxInt : o.blocks * o.bs;
  p.n_tokens = int(T);
  p.n_tensors = n;
  p.heads = int(o.N);
  p.block_size = int(o.bs);
  p.lg_block = log2_of(o.bs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s,
                             [&] {
                               return launch_cache_write_int4(p, int(o.D), int(o.groups), o.dtype == FIA_DTYPE_BF16, s);
                             }),
                    "4-bit cache write launch");
}

fia_status fia_cache_read_int4(const fia_tensor* key_cache, const fia_tensor* value_cache, const fia_tensor* key_scales,
                               const fia_tensor* value_scales, const fia_tensor* block_table,
                               const fia_tensor* cu_kv_lens, const fia_tensor* key, const fia_tensor* value,
                               void* stream) {
  if (!given(key)) return fail(FIA_ERR_NULL, "key is required");
  const bool two = there(value);
  if (two != there(value_cache) || two != there(value_scales))
    return fail(FIA_ERR_NULL, "value, value_cache and value_scales must be given together");
  if (two && !given(value)) return fail(FIA_ERR_NULL, "value has no data");
  Int4Pool o;
  FIA_TRY(int4_pools(key_cache, value_cache, key_scales, value_scales, two, o));
  FIA_TRY(check_i32(cu_kv_lens, -1, "cu_kv_lens"));
  const int64_t B = cu_kv_lens->shape[0];
  if (!given(block_table)) return fail(FIA_ERR_NULL, "block_table is required");
  if (block_table->dtype != FIA_DTYPE_I32 || block_table->ndim != 2 || block_table->shape[0] != B)
    return fail(FIA_ERR_BLOCK_TABLE, "block_table must be int32 (B, maxBlocksPerSeq)");
  if (reinterpret_cast<uintptr_t>(block_table->data) % 4 != 0)
    return fail(FIA_ERR_ALIGNMENT, "block_table not 4-byte aligned");
  Int4ReadParams p;
  memset(&p, 0, sizeof(p));
  const int64_t T = key->shape[0];
  const int n = two ? 2 : 1;
  for (int y = 0; y < n; ++y) {
    const fia_tensor* x = y ? value : key;
    const char* name = y ? "value" : "key";
    if (x->dtype != o.dtype) return fail(FIA_ERR_DTYPE, "%s must have its scales' type", name);
    if (x->ndim != 3 || x->shape[0] != T || x->shape[1] != o.N || x->shape[2] != o.D)
      return fail(FIA_ERR_SHAPE, "%s must be (T, KV_N, D) = (%lld, %lld, %lld)", name, (long long)T, (long long)o.N, (long long)o.D);
    if (!aligned16(x->data)) return fail(FIA_ERR_ALIGNMENT, "%s not 16-byte aligned", name);
    p.codes[y] = static_cast<const uint8_t*>((y ? value_cache : key_cache)->data);
    p.scales[y] = static_cast<const uint32_t*>((y ? value_scales : key_scales)->data);
    p.dst[y] = static_cast<uint8_t*>(x->data);
  }
  if (T > kMaxInt) return fail(FIA_ERR_SHAPE, "more than 2^31-1 tokens");
  if (T == 0 || B == 0) return FIA_OK;
  const uintptr_t bytes = uintptr_t(T) * uintptr_t(o.N * o.D) * 2;
  for (int y = 0; y < n; ++y) {
    const Range ins[] = {{p.codes[0], uintptr_t(o.code_bytes)},
                         {p.scales[0], uintptr_t(o.scale_bytes)},
                         {p.codes[n - 1], uintptr_t(o.code_bytes)},
                         {p.scales[n - 1], uintptr_t(o.scale_bytes)},
                         {cu_kv_lens->data, uintptr_t(B) * 4},
                         {block_table->data, uintptr_t(numel(block_table)) * 4}};
    for (const Range& r : ins)
      if (overlap(p.dst[y], bytes, r.p, r.n)) return fail(FIA_ERR_UNSUPPORTED, "key or value overlaps an input");
    if (y == 1 && overlap(p.dst[0], bytes, p.dst[1], bytes)) return fail(FIA_ERR_UNSUPPORTED, "key and value overlap");
  }
  p.src_blk = o.blk;
  p.src_row = o.row;
  p.src_head = o.head;
  p.cu = static_cast<const int32_t*>(cu_kv_lens->data);
  p.block_table = static_cast<const int32_t*>(block_table->data);
  p.table_cols = block_table->shape[1];
  p.n_tokens = int(T);
  p.n_tensors = n;
  p.heads = int(o.N);
  p.block_size = int(o.bs);
  p.lg_block = log2_of(o.bs);
  p.B = int(B);
  p.n_blocks = int(o.blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s,
                             [&] {
                               return launch_cache_read_int4(p, int(o.D), int(o.groups), o.dtype == FIA_DTYPE_BF16,
                                                             sm_count(), s);
                             }),
                    "4-bit cache read launch");
}

fia_status fia_decode_window_int4_get_workspace_size(const fia_tensor* query, const fia_tensor* key_cache,
                                                     const fia_tensor* value_cache, const fia_tensor* key_scales,
                                                     const fia_tensor* value_scales, const fia_tensor* block_table,
                                                     const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                                     int64_t sink_tokens, const fia_tensor* attention_out,
                                                     const fia_tensor* softmax_lse, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return fail(FIA_ERR_NULL, "workspace_bytes is NULL");
  *workspace_bytes = 0;
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;   // empty query
  Int4SpanParams p;
  Int4Pool o;
  FIA_TRY(decode_args(query, key_cache, value_cache, key_scales, value_scales, block_table, actual_seq_kvlen, params,
                      sink_tokens, attention_out, softmax_lse, p, o));
  *workspace_bytes = split_plan(p.s, o, sm_count()).bytes;
  return FIA_OK;
}

fia_status fia_decode_window_int4(const fia_tensor* query, const fia_tensor* key_cache, const fia_tensor* value_cache,
                                  const fia_tensor* key_scales, const fia_tensor* value_scales,
                                  const fia_tensor* block_table, const fia_tensor* actual_seq_kvlen,
                                  const fia_params* params, int64_t sink_tokens, const fia_tensor* attention_out,
                                  const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (query != nullptr && query->ndim > 0 && numel(query) == 0) return FIA_OK;   // empty query
  Int4SpanParams p;
  Int4Pool o;
  FIA_TRY(decode_args(query, key_cache, value_cache, key_scales, value_scales, block_table, actual_seq_kvlen, params,
                      sink_tokens, attention_out, softmax_lse, p, o));
  const int n_sm = sm_count();
  const SplitPlan w = split_plan(p.s, o, n_sm);
  if (w.bytes > 0) {
    FIA_TRY(check_ws(workspace, workspace_bytes, w.bytes));
    uint8_t* base = static_cast<uint8_t*>(workspace);
    p.part_o = reinterpret_cast<float*>(base);
    p.part_ml = reinterpret_cast<float2*>(base + w.ml);
    p.heads = reinterpret_cast<int4*>(base + w.heads);
    p.n_ctas = w.ctas;
    p.begin = w.begin;
  }
  const bool bf16 = query->dtype == FIA_DTYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_check(profiled(s, [&] { return launch_int4_decode(p, int(o.D), int(o.groups), bf16, n_sm, s); }),
                    "4-bit decode launch");
}

}  // extern "C"
