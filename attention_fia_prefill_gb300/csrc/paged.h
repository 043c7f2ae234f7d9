// Launch-side structures of the paged-serving operators (paged_api.cu, their
// host side): block tables and slot maps, the cache write, decode with a
// window, shared-prefix decode.  Lengths live in device memory, so a captured
// call replays with new lengths.
#pragma once
#include <cstdint>

#include "../../include/fia.h"
#include "internal.h"

namespace fia {

// Block tables grown to the requests' new lengths, a slot for every new token.
struct TableParams {
  const int32_t* context_lens;    // [B] tokens already in the cache
  const int32_t* new_lens;        // [B] tokens to append
  const int32_t* free_blocks;     // [n_free] block ids to hand out, in order
  int32_t* block_table;           // [B, table_cols], rows grown in place
  int32_t* slot_mapping;          // [n_tokens]
  int32_t* kv_lens;               // [B] context + new
  int32_t* cu_new_lens;           // [B] running sum of new, no leading 0
  int32_t* num_blocks;            // [1] blocks asked for
  int B, n_free, table_cols, n_tokens, block_size;
};

// Rows of up to two tensors (keys, values) copied to their slots of the pools.
struct CacheWriteParams {
  const uint8_t* src[2];
  uint8_t* dst[2];
  int64_t src_row[2];             // bytes between tokens
  int64_t dst_blk[2], dst_row[2], dst_head[2];   // bytes between blocks / slots of a block / heads
  int vecs[2];                    // 16-byte vectors of a token (all heads)
  int head_vecs[2];               // of one head
  const int32_t* slots;           // [n_tokens]
  int64_t n_slots;                // slots of a pool: others (and negative ones) are skipped
  int n_tokens, block_size;
};

// Decode over the keys [base, length) of every sequence that the window and
// the sinks leave visible, joined with n_parts partial results per row.
struct SpanParams {
  const void* q;
  void* out;
  float* lse;                     // nullable
  int64_t q_sb, q_sn, q_ss;       // element strides of q and out for (b, n, s)
  int64_t lse_sb, lse_sn, lse_ss;
  const void* k;
  const void* v;
  int64_t blk_stride, head_stride, row_stride;   // elements; contiguous caches: a block is a batch
  const int32_t* block_table;     // nullable (contiguous)
  int64_t table_stride;
  int block_size, n_blocks;
  const int32_t* kv_len;          // nullable: kv_max for every batch
  int kv_max;                     // lengths are clamped to [0, kv_max]
  int B, N1, N2, group, q_tokens, rows;
  int pre, sink, base;
  int shared;                     // keys below come from the table's first row
  float scale_log2;
  DevStatus status;               // word nullable; stamped where n_parts is 0
  // partial results to join (the shared prefix): O (not divided by its sum)
  // [n_parts][B * N1 * q_tokens][D], (max in log2 units, sum) likewise (-inf: no
  // keys; NaN, NaN: a NaN score, or a kernel that gave up), row
  // (b * N1 + head) * q_tokens + token
  const float* part_o;
  const float2* part_ml;
  int n_parts;
  int64_t part_rows;              // rows of one part
  // set by the launch: CTAs of a unit (log2), log2 of block_size (-1: no power
  // of two), 2^16 / q_tokens
  int lg_cs, lg_block;
  uint32_t q_inv;
};

cudaError_t launch_block_table(const TableParams& p, cudaStream_t s);
cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s);
// Window prefill (PrefillParams of an item per pair of tiles and head, lengths
// on the device).
cudaError_t launch_prefill_window(const PrefillParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s);
cudaError_t launch_span_decode(const SpanParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s);
// The same for units of 17..64 rows, on the tcgen05 tensor cores (fia_status: it
// builds tensor maps), and whether it is the faster one.
bool span_wide_pays(const SpanParams& p, int n_sm);
fia_status launch_span_wide(const SpanParams& p, int head_dim, bool bf16, int n_sm, cudaStream_t s);

}  // namespace fia
