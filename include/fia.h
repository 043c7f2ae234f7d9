/*
 * fia.h -- C ABI of the fused inference attention library (sm_103a).
 *
 * The operator, as the FusedInferAttentionScore pages define it
 * (torch_npu.npu_fused_infer_attention_score_v2, "计算公式";
 * torch_npu.npu_prompt_flash_attention, "功能说明"):
 *
 *     attention_out = softmax(scale_value * query . key^T + atten_mask) . value
 *     softmax_lse   = log(sum(exp(s - max(s)))) + max(s)     (fp32, optional)
 *
 * Three entry points cover the pages' cases:
 *   fia_prefill  -- full attention, Q_S >= 1 (PromptFlashAttention)
 *   fia_decode   -- incremental attention, Q_S = 1 (or up to 16 new tokens),
 *                   paged or contiguous KV cache, optionally MLA (query_rope /
 *                   key_rope) (IncreFlashAttention)
 *   bsa_forward  -- block-sparse attention selected by blockSparseMask
 *                   (aclnnBlockSparseAttentionV2)
 * Each has a first phase that validates the arguments and reports the scratch
 * ("workspace") size, mirroring aclnn's two-phase GetWorkspaceSize + execute
 * calls (aclnnFusedInferAttentionScoreV5, "函数原型").
 *
 * Conventions shared by every call:
 *   - Tensors are described by fia_tensor: a data pointer, an element type and a
 *     row-major, contiguous shape (the pages accept contiguous tensors only).
 *     Data pointers of execute calls are DEVICE pointers, 16-byte aligned.
 *   - Host arrays (actual_seq_qlen / actual_seq_kvlen) are read during the call
 *     and not kept.
 *   - Ownership: the caller owns every buffer (inputs, outputs, workspace).  The
 *     library allocates no device memory, keeps no pointer after returning, and
 *     launches its kernels asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).
 *   - The return value covers argument validation and kernel launch only.  Errors
 *     found on the device (a bounded wait that ran out) are recorded in the
 *     workspace and read with fia_device_status().
 *   - Rows with no key to attend to (K/V with S2 = 0, a fully masked row, a
 *     padding row past a batch's actual query length) give attention_out = 0 and
 *     softmax_lse = +inf, extending the pages' empty-tensor rule
 *     (npu_fused_infer_attention_score_v2, "入参为空的处理").
 *   - A query with zero elements returns FIA_OK without launching anything.
 */
#ifndef FIA_H_
#define FIA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FIA_API __attribute__((visibility("default")))
#else
#define FIA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fia_status {
  FIA_OK = 0,
  FIA_ERR_NULL = 1,          /* a required pointer is NULL                                  */
  FIA_ERR_DTYPE = 2,         /* element types disagree or are not supported                 */
  FIA_ERR_SHAPE = 3,         /* ranks/dims inconsistent (e.g. key != value shape)           */
  FIA_ERR_LAYOUT = 4,        /* unknown input_layout                                        */
  FIA_ERR_UNSUPPORTED = 5,   /* valid on the pages but not implemented by this library     */
  FIA_ERR_SEQLEN = 6,        /* actual_seq_* list length or values invalid                  */
  FIA_ERR_BLOCK_TABLE = 7,   /* block_table / block_size invalid                            */
  FIA_ERR_WORKSPACE = 8,     /* workspace NULL or smaller than the reported size            */
  FIA_ERR_CUDA = 9,          /* a CUDA runtime call or kernel launch failed                 */
  FIA_ERR_TIMEOUT = 10,      /* device: a bounded wait inside a kernel ran out              */
  FIA_ERR_HEADS = 11,        /* num_heads / num_key_value_heads invalid (GQA rules)         */
  FIA_ERR_SPARSE_MODE = 12,  /* sparse_mode outside 0..4 or its mask requirements unmet     */
  FIA_ERR_ALIGNMENT = 13     /* a device pointer is not 16-byte aligned                     */
} fia_status;

typedef enum fia_dtype {
  FIA_DTYPE_F16 = 0,
  FIA_DTYPE_BF16 = 1,
  FIA_DTYPE_F32 = 2,
  FIA_DTYPE_I32 = 3,
  FIA_DTYPE_I64 = 4,
  FIA_DTYPE_U8 = 5,
  FIA_DTYPE_BOOL = 6,
  FIA_DTYPE_I8 = 7,
  FIA_DTYPE_F8E4M3 = 8   /* float8 e4m3 (FN: no infinities), the FP8 block-sparse inputs */
} fia_dtype;

/* A contiguous row-major tensor.  ndim == 0 or data == NULL means "absent"
 * for optional arguments. */
typedef struct fia_tensor {
  void* data;
  int32_t dtype;       /* fia_dtype */
  int32_t ndim;        /* 0..5 */
  int64_t shape[5];
} fia_tensor;

/* Keyword arguments of the pages' Python API (npu_fused_infer_attention_score_v2
 * parameter list; npu_prompt_flash_attention prototype).  Fill with
 * fia_params_init() and override what is needed. */
typedef struct fia_params {
  int64_t num_heads;              /* Q_N (num_query_heads / num_heads)                         */
  int64_t num_key_value_heads;    /* KV_N; 0 means equal to num_heads; Q_N % KV_N == 0,
                                     Q_N / KV_N <= 64                                          */
  double scale_value;             /* softmax_scale / scale_value; default 1.0; must be > 0     */
  const char* input_layout;       /* "BSH", "BSND", "BNSD" or "TND"; default "BSH"             */
  int64_t sparse_mode;            /* 0..4; 2 = leftUpCausal, 3 = rightDownCausal, 4 = band     */
  int64_t pre_tokens;             /* band (mode 4) width before the diagonal; default 2^31-1   */
  int64_t next_tokens;            /* band (mode 4) width after the diagonal; default 2^31-1    */
  const int64_t* actual_seq_qlen;   /* host array or NULL; TND: cumulative, no leading 0       */
  int64_t n_actual_seq_qlen;
  const int64_t* actual_seq_kvlen;  /* host array or NULL; TND: cumulative, no leading 0       */
  int64_t n_actual_seq_kvlen;
  int64_t block_size;             /* PageAttention tokens per block (0 = no paging)           */
  int32_t softmax_lse_flag;       /* return_softmax_lse: 1 = write softmax_lse                 */
  int32_t inner_precise;          /* accepted (0..3); the kernels always keep fp32 softmax    */
} fia_params;

/* Fills *p with the pages' defaults. */
FIA_API void fia_params_init(fia_params* p);

/* ------------------------------------------------------------------------
 * fia_prefill: full attention with Q_S >= 1 over contiguous key/value.
 *   query  (B,S1,H) BSH | (B,S1,N1,D) BSND | (B,N1,S1,D) BNSD | (T1,N1,D) TND;
 *          f16 or bf16.  D is 64 or 128.
 *   key, value: same layout and element type, N2 heads, identical shapes.
 *   atten_mask: optional.  sparse_mode 2/3/4 compute their pattern from
 *          indices; a mask given there must be (2048,2048) / (1,2048,2048) /
 *          (1,1,2048,2048) and is not read.  Mode 4 (band): query row i sees
 *          keys i + d - pre_tokens .. i + d + next_tokens, d = S2 - S1 of the
 *          batch (npu_fused_infer_attention_score_v2, sparse_mode; pre/next
 *          clamped to +-2^30).  Mode 0 with a mask, and mode 1 (allMask,
 *          mask required): bool/int8/uint8, device memory, contiguous, shape
 *          (S1m,S2m), (B|1,S1m,S2m) or (B|1,1,S1m,S2m) with S1m / S2m at least
 *          every batch's query / key length; byte [b][i][j] != 0 masks key j of
 *          the batch's query row i (batch-local indices, also for TND).  Mode 0
 *          also keeps only i - pre_tokens <= j <= i + next_tokens.  A mask
 *          whose address and S2m are multiples of 16 bytes is read fastest
 *          (8 and 4 next; otherwise byte by byte).  A row with every key
 *          masked gives out 0 and lse +inf.
 *   attention_out: the query's shape and element type.
 *   softmax_lse: fp32 (B,N1,S1,1), or (T1,N1,1) for TND; used when
 *          params->softmax_lse_flag != 0 (may be absent otherwise).
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_prefill_get_workspace_size(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                                          const fia_tensor* atten_mask, const fia_params* params,
                                          const fia_tensor* attention_out, const fia_tensor* softmax_lse,
                                          size_t* workspace_bytes);
FIA_API fia_status fia_prefill(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                       const fia_tensor* atten_mask, const fia_params* params, const fia_tensor* attention_out,
                       const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * fia_prefill_mla: MLA prefill (npu_fused_infer_attention_score_v2, query D
 * not 512: "query, key, value D 128 with query_rope / key_rope D 64", or
 * "query, key D 192, value D 128").  The score of a pair is
 * scale_value * (q . k + q_rope . k_rope), the product over the 192-column
 * concatenation; value and attention_out have D 128.
 *   query / key: D 192 with query_rope = key_rope = NULL, or D 128 with both
 *          rope tensors given (the query's / key's shape with D 64, same type).
 *   value: key's shape with D 128.  attention_out: query's shape with D 128.
 *   Layouts BSH/BSND/BNSD/TND (the pages list TND), f16 or bf16, GQA allowed.
 *   sparse_mode 0 (with or without atten_mask), 1, 2, 3, 4 and atten_mask as
 *   fia_prefill.  softmax_lse as fia_prefill.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_prefill_mla_get_workspace_size(const fia_tensor* query, const fia_tensor* key,
                                              const fia_tensor* value, const fia_tensor* query_rope,
                                              const fia_tensor* key_rope, const fia_tensor* atten_mask,
                                              const fia_params* params, const fia_tensor* attention_out,
                                              const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status fia_prefill_mla(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                           const fia_tensor* query_rope, const fia_tensor* key_rope, const fia_tensor* atten_mask,
                           const fia_params* params, const fia_tensor* attention_out, const fia_tensor* softmax_lse,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * fia_prefill_paged: fia_prefill with key/value in a paged cache (chunked
 * prefill: a chunk of new query tokens against a sequence's cached keys).
 *   npu_fused_infer_attention_score_v2, page attention: key j of batch b is
 *   row j % block_size of block block_table[b][j / block_size].
 *   query, atten_mask, sparse_mode (0..4), pre/next tokens, attention_out and
 *          softmax_lse as in fia_prefill (BSH/BSND/BNSD/TND query).
 *   key_cache, value_cache: device, same shape, the query's element type,
 *          (blocknum, KV_N, block_size, D) or (blocknum, block_size, KV_N*D).
 *   block_table: device int32 (B, >= maxBlockNumPerSeq); B = the query's batch
 *          (the number of sequences for TND).  Entries are not range-checked
 *          (the pages leave them to the caller); an id outside the pool reads
 *          as zeros.  NULL block_table = fia_prefill.
 *   params->block_size: 128..512, a multiple of 128; params->actual_seq_kvlen
 *          is required and holds each batch's key count (not cumulative,
 *          also for a TND query: the cache is not TND).
 *   blocknum must cover the blocks the lengths need (FIA_ERR_BLOCK_TABLE).
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_prefill_paged_get_workspace_size(const fia_tensor* query, const fia_tensor* key_cache,
                                                const fia_tensor* value_cache, const fia_tensor* block_table,
                                                const fia_tensor* atten_mask, const fia_params* params,
                                                const fia_tensor* attention_out, const fia_tensor* softmax_lse,
                                                size_t* workspace_bytes);
FIA_API fia_status fia_prefill_paged(const fia_tensor* query, const fia_tensor* key_cache, const fia_tensor* value_cache,
                             const fia_tensor* block_table, const fia_tensor* atten_mask, const fia_params* params,
                             const fia_tensor* attention_out, const fia_tensor* softmax_lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * fia_decode: incremental attention, Q_S new query tokens per batch.
 *   query  (B,N1,Q_S,D) BNSD | (B,Q_S,N1,D) BSND | (B,Q_S,H) BSH; f16 or bf16.
 *          Q_S = 1, or 2..16 with (N1 / N2) * Q_S <= 64 (not with MLA); then
 *          sparse_mode masks the Q_S x S_kv block as in the formula
 *          (npu_fused_infer_attention_score_v2, sparse_mode): 0 none, 2 key j
 *          <= token i, 3 key j <= i + S_kv - Q_S (the last token sees the whole
 *          cache); other modes return FIA_ERR_UNSUPPORTED.  With Q_S = 1
 *          sparse_mode is ignored, as on the pages.
 *   key/value, contiguous (block_table absent): the query's layout with N2 heads.
 *   key/value, paged (block_table present, PageAttention):
 *          (blocknum, N2, block_size, D)  or  (blocknum, block_size, N2*D);
 *          block_table int32 (B, >= max blocks per sequence); block ids are not
 *          validated (as on the pages); actual_seq_kvlen is required.
 *          block_size: a multiple of 16 that divides 128 or a multiple of 128.
 *   query_rope / key_rope (MLA): both or neither.  Then D = 512, D_rope = 64,
 *          N2 = 1, N1 in {1..128}, key = value = the 512-d latent cache
 *          (blocknum, block_size, 512), key_rope (blocknum, block_size, 64).
 *          scores = scale * (q . k + q_rope . k_rope).
 *   atten_mask: with Q_S = 1 (not MLA), bool / int8 / uint8 of shape (B, KV_S),
 *          (B, 1, KV_S) or (B, 1, 1, KV_S), batch dim B or 1 (broadcast),
 *          KV_S >= every actual_seq_kvlen, contiguous, device memory; a
 *          nonzero byte masks its key.  A row whose keys are all masked gets
 *          0 and softmax_lse +inf.  With Q_S > 1 or MLA it returns
 *          FIA_ERR_UNSUPPORTED.
 *   attention_out: the query's shape; softmax_lse fp32 (B,N1,Q_S,1) if flagged.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_decode_get_workspace_size(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                                         const fia_tensor* query_rope, const fia_tensor* key_rope,
                                         const fia_tensor* block_table, const fia_tensor* atten_mask,
                                         const fia_params* params, const fia_tensor* attention_out,
                                         const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status fia_decode(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                      const fia_tensor* query_rope, const fia_tensor* key_rope, const fia_tensor* block_table,
                      const fia_tensor* atten_mask, const fia_params* params, const fia_tensor* attention_out,
                      const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * fia_decode_no_alloc: fia_decode for callers that cannot allocate device
 * memory.  The pages have no counterpart: it exists because some callers only
 * hold the input and output buffers they were given (plugin hosts, inference
 * servers that own the memory budget, code where a device allocation is not
 * allowed) and cannot create the workspace fia_decode takes.
 *   Arguments: as fia_decode, without the workspace.
 *   Scratch: a 16 MiB array built into the library (one per GPU that loads it,
 *          held until the process exits).  A call whose workspace need
 *          (fia_decode_get_workspace_size) exceeds 16 MiB returns
 *          FIA_ERR_WORKSPACE before touching the device.
 *   Set-up: every call looks up the array's device address in the calling
 *          thread's current CUDA context (the address belongs to a context:
 *          another context made current through the driver API, or a device
 *          reset, gives another one).  The first call in a context also loads
 *          the library's kernels there; make that first call before any
 *          stream capture.
 *   Sharing: every call uses the same array and leaves its contents behind.
 *          Calls that overlap on the GPU (other streams, other host threads)
 *          race on it; serialise them.  The device status word lives in the
 *          array and is not exposed: a device-side timeout of a call made
 *          through this entry point cannot be read back.
 *   Limit: MLA decode keeps two 256-wide partial outputs per query head and
 *          plan slot, so MLA calls with many query heads do not fit (128 heads
 *          never do, whatever the batch); they return FIA_ERR_WORKSPACE.
 *   Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_decode_no_alloc(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                                       const fia_tensor* query_rope, const fia_tensor* key_rope,
                                       const fia_tensor* block_table, const fia_tensor* atten_mask,
                                       const fia_params* params, const fia_tensor* attention_out,
                                       const fia_tensor* softmax_lse, void* stream);

/* ------------------------------------------------------------------------
 * bsa_forward: block-sparse attention (aclnnBlockSparseAttentionV2).
 *   query/key/value: BNSD, BSND or TND (one layout for all three); f16/bf16;
 *          D in {64, 128}; N1 % N2 == 0.
 *   block_sparse_mask: u8/bool (B, N1, ceil(maxQS/X), ceil(maxKVS/Y));
 *          nonzero keeps the X x Y block.
 *   block_shape: {X, Y}; X > 0, Y a multiple of 128 (this library: X also a
 *          multiple of 128).
 *   actual_seq_qlen / actual_seq_kvlen: both or neither (TND: both).
 *   attention_out, softmax_lse: as for fia_prefill.
 * ------------------------------------------------------------------------ */
FIA_API fia_status bsa_get_workspace_size(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                                  const fia_tensor* block_sparse_mask, const int64_t* block_shape,
                                  const fia_params* params, const fia_tensor* attention_out,
                                  const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status bsa_forward(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                       const fia_tensor* block_sparse_mask, const int64_t* block_shape, const fia_params* params,
                       const fia_tensor* attention_out, const fia_tensor* softmax_lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * bsa_forward_fp8: FP8 block-sparse attention (aclnnBlockSparseAttentionV2,
 * "FP8特性说明").  Row i of query head h is worth query[i] *
 * q_dequant_scale[b][h][i / 128]; key / value row j of kv head n is worth
 * key[j] * k_dequant_scale[b][n][j / Y] (value likewise).
 *   query/key/value: float8 e4m3 (FIA_DTYPE_F8E4M3), D = 128, layouts as
 *          bsa_forward.
 *   block_shape: {128, 256} or {128, 512} (the quantisation blocks).
 *   block_sparse_mask: as bsa_forward, or NULL: every block kept, which is
 *          dense (sparse_mode 0) FP8 prefill attention with the same scales.
 *   q_dequant_scale: fp32 (B, N1, ceil(maxQS/128), 1); k_dequant_scale and
 *          v_dequant_scale: fp32 (B, N2, ceil(maxKVS/Y), 1); device memory;
 *          every scale must be positive.  The scales are read on the device
 *          only: a scale <= 0 (or NaN) makes the kernel record
 *          FIA_ERR_UNSUPPORTED in the call's status word (fia_device_status),
 *          and the output of that call is unspecified.
 *   attention_out: bf16, the query's shape.  softmax_lse as bsa_forward.
 *   The scores run on the fp8 tensor cores (e4m3 x e4m3, fp32 accumulate).
 *   V is first rewritten into the workspace as f16 by a separate pass (one
 *   extra read of V and a write of twice its bytes); P V then runs on the
 *   f16 tensor-core path, with P scaled by the tile's value scale.
 * ------------------------------------------------------------------------ */
FIA_API fia_status bsa_fp8_get_workspace_size(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                                      const fia_tensor* block_sparse_mask, const int64_t* block_shape,
                                      const fia_tensor* q_dequant_scale, const fia_tensor* k_dequant_scale,
                                      const fia_tensor* v_dequant_scale, const fia_params* params,
                                      const fia_tensor* attention_out, const fia_tensor* softmax_lse,
                                      size_t* workspace_bytes);
FIA_API fia_status bsa_forward_fp8(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                           const fia_tensor* block_sparse_mask, const int64_t* block_shape,
                           const fia_tensor* q_dequant_scale, const fia_tensor* k_dequant_scale,
                           const fia_tensor* v_dequant_scale, const fia_params* params,
                           const fia_tensor* attention_out, const fia_tensor* softmax_lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Paged serving.  The operators from here to fia_decode_shared_prefix take
 * every length from DEVICE memory (int32), so their launches depend on sizes
 * alone: a captured step replays with new lengths.  A step runs them in this
 * order: tables and slots from the requests' lengths, the write of the new
 * keys and values, attention over the cache.
 *
 * fia_block_table_append: grows the block tables of B requests and gives every
 * new token its slot.
 *   context_lens, new_lens: int32 (B); tokens the cache holds of a request, and
 *          tokens to append (negative: 0).  Request b holds ceil(context /
 *          block_size) blocks and needs ceil((context + new) / block_size).
 *   free_blocks: int32 (F), ids handed out from the front, in request order.
 *          The list is not changed: the next call takes it without its first
 *          min(num_blocks, F) ids, or it hands the same blocks out again.
 *   block_table: int32 (B, W), in place: the columns of the blocks that a
 *          request lacked are written, every other entry stays as it was.
 *   slot_mapping: int32 (T), out: slot block_id * block_size + offset of every
 *          new token, the requests' tokens one after the other; -1 from the
 *          sum of new_lens on (a padded batch).  Tokens past T get no slot,
 *          and a block whose first token is past T no entry.
 *   kv_lens: int32 (B), out: context + new.   cu_new_lens: int32 (B), out:
 *          running sum of new_lens without a leading 0 (the TND lists' form).
 *   num_blocks: int32 (1), out: blocks the batch asked for.  Above F the list
 *          ran out: the entries of blocks without an id are written as -1
 *          and their tokens' slots are -1, as they are for a token past the
 *          table's last column.
 *   block_size: 1 or more.  Outputs may not overlap the inputs.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_block_table_append(const fia_tensor* context_lens, const fia_tensor* new_lens,
                                  const fia_tensor* free_blocks, int64_t block_size, const fia_tensor* block_table,
                                  const fia_tensor* slot_mapping, const fia_tensor* kv_lens,
                                  const fia_tensor* cu_new_lens, const fia_tensor* num_blocks, void* stream);

/* ------------------------------------------------------------------------
 * fia_cache_write: copies new keys and values to their slots of the pools.
 *   key (T, KV_N, D), value (T, KV_N, Dv): f16, bf16 or e4m3; heads and
 *          columns contiguous, tokens key_token_stride / value_token_stride
 *          elements apart (0: contiguous; slices of a fused projection have
 *          its row length), rows 16-byte aligned.  D * element size is a
 *          multiple of 16.  value and value_cache may both be NULL.
 *   key_cache / value_cache: (blocknum, KV_N, block_size, D) or (blocknum,
 *          block_size, KV_N*D), the same blocknum and block_size, the
 *          tensors' types.  The caches may overlap neither each other nor key
 *          or value.
 *   slot_mapping: int32 (T): token t goes to row slot % block_size of block
 *          slot / block_size.  Slots outside the pool (negative ones among
 *          them) are skipped; every other row of the pools stays as it was.
 *          Slots must differ: of two tokens with one slot either may be left,
 *          or a mixture.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_cache_write(const fia_tensor* key, int64_t key_token_stride, const fia_tensor* value,
                           int64_t value_token_stride, const fia_tensor* key_cache, const fia_tensor* value_cache,
                           const fia_tensor* slot_mapping, void* stream);

/* ------------------------------------------------------------------------
 * fia_decode_window: incremental attention with a sliding window and sink
 * tokens.  Token i of a sequence's Q_S new tokens has position p = L - Q_S + i
 * and sees key j when j <= p and (j >= p - pre_tokens or j < sink_tokens).
 *   query, attention_out, softmax_lse: as fia_decode (BNSD / BSND / BSH, Q_S
 *          1..16, Q_N / KV_N * Q_S <= 64, D 64 or 128).
 *   key/value, contiguous or paged: as fia_decode (block_size a multiple of
 *          16).  Block ids outside the pool read as zeros (of a pool without a
 *          block every id does, here and in the two entries below); entries of blocks
 *          that no token sees are never read, so blocks behind the window may
 *          be freed.  At most 2^30 keys per sequence.
 *   actual_seq_kvlen: device int32 (B), the length L with the new tokens,
 *          clamped to [0, keys the tensors have room for]; NULL: all of them
 *          (contiguous key/value only).  params' own lists must be NULL.
 *   params->pre_tokens >= 0 (default 2^31-1: no window), sink_tokens >= 0.
 *          sparse_mode and next_tokens are not read.  scale_value * log2(e) must
 *          be a normal fp32 number (also of the two entries below).
 *   Rows that see no key (p < 0: a padded batch) give 0 and +inf.  With several
 *          new tokens the values (not scores) of a key that only some of them
 *          see enter the others' sums with a weight of 0: they must be finite.
 *   No workspace, and so no status word: a bounded wait that runs out (units of
 *          more than 16 rows) leaves NaN in its unit's rows.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_decode_window(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                             const fia_tensor* block_table, const fia_tensor* actual_seq_kvlen,
                             const fia_params* params, int64_t sink_tokens, const fia_tensor* attention_out,
                             const fia_tensor* softmax_lse, void* stream);

/* ------------------------------------------------------------------------
 * fia_prefill_window: prefill with a sliding window and sink tokens, over
 * contiguous or paged key/value, with lengths in device memory.  Row i of a
 * batch has position p = i + kv_len - q_len and sees key j when j <= p and
 * (j >= p - pre_tokens or j < sink_tokens).
 *   query, attention_out, softmax_lse: as fia_prefill (BSH / BSND / BNSD /
 *          TND, f16 or bf16, D 64 or 128).
 *   key, value: contiguous in the query's layout, or, with block_table, the
 *          pools of fia_prefill_paged (block_size 128..512, a multiple of 128;
 *          block ids outside the pool read as zeros; entries of blocks that
 *          no row sees are never read).
 *   actual_seq_qlen: device int32 (B); rows of each batch, NULL: S1 for all
 *          (TND: required, running sums without a leading 0, B <= 4096).
 *   actual_seq_kvlen: device int32 (B); keys of each batch, NULL: S2 for all
 *          (paged: required; TND with contiguous keys: required, running sums).
 *          Values outside what the tensors hold are taken to the nearest
 *          value inside.  params' own lists must be NULL.
 *   params->pre_tokens >= 0 (default 2^31-1: causal), sink_tokens >= 0.
 *          sparse_mode and next_tokens are not read.
 *   Padding rows of the padded layouts and rows that see no key give 0 and
 *          +inf; rows of a TND query behind the last sequence stay as they were.
 *   Values (not scores) of keys that a row does not see enter its sums with a
 *          weight of 0: they must be finite where they share a 128-key tile with
 *          a seen key and lie before the batch's length.
 *   Workspace: the status word.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_prefill_window_get_workspace_size(const fia_tensor* query, const fia_tensor* key,
                                                 const fia_tensor* value, const fia_tensor* block_table,
                                                 const fia_tensor* actual_seq_qlen,
                                                 const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                                 int64_t sink_tokens, const fia_tensor* attention_out,
                                                 const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status fia_prefill_window(const fia_tensor* query, const fia_tensor* key, const fia_tensor* value,
                              const fia_tensor* block_table, const fia_tensor* actual_seq_qlen,
                              const fia_tensor* actual_seq_kvlen, const fia_params* params, int64_t sink_tokens,
                              const fia_tensor* attention_out, const fia_tensor* softmax_lse, void* workspace,
                              size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * fia_decode_shared_prefix: incremental attention for a batch whose sequences
 * begin with the same keys.  The result is fia_decode_window's without a
 * window; the prefix's keys and values are read once for the whole batch (by
 * every sequence where they are so few that this is faster).
 *   query, key_cache, value_cache, block_table, actual_seq_kvlen (the whole
 *          lengths, prefix and new tokens among them), attention_out,
 *          softmax_lse: as fia_decode_window with paged key/value;
 *          block_size a multiple of 16 that divides 128, or a multiple of 128.
 *   shared_prefix_len: a multiple of block_size, at most the keys of the
 *          table's columns.  The first shared_prefix_len / block_size entries
 *          of every row of block_table must be the same; the first row's are
 *          read.  A sequence shorter than the prefix sees its own length's keys
 *          of it (values of the others must be finite).
 *   Workspace: the status word and the prefix's partial results.  A bounded
 *          wait that runs out leaves NaN in the rows it held up (and
 *          FIA_ERR_TIMEOUT in the word).
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_decode_shared_prefix_get_workspace_size(const fia_tensor* query, const fia_tensor* key_cache,
                                                       const fia_tensor* value_cache, const fia_tensor* block_table,
                                                       const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                                       int64_t shared_prefix_len, const fia_tensor* attention_out,
                                                       const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status fia_decode_shared_prefix(const fia_tensor* query, const fia_tensor* key_cache,
                                    const fia_tensor* value_cache, const fia_tensor* block_table,
                                    const fia_tensor* actual_seq_kvlen, const fia_params* params,
                                    int64_t shared_prefix_len, const fia_tensor* attention_out,
                                    const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* ------------------------------------------------------------------------
 * The 4-bit cache: fia_cache_write_int4, fia_cache_read_int4,
 * fia_decode_window_int4.  A row (one token, one kv head) of D values (64 or
 * 128) is cut into groups of G = 32, 64 or 128 (at most D).  A group holds
 * (step, low) in the type t of the keys and values (f16 or bf16) and a code
 * 0..15 for each value, which stands for low + step * code:
 *     low  = min x
 *     step = max((max x - min x) / 15, tiny), rounded up to t;  tiny = 2^-60
 *            (bf16) or 2^-24 (f16).  f16: rounded down where low + 15 step
 *            would be above 65504 and max x above min x
 *     code = ceil((x - low) / step - 1/2): the nearest one, and the lower of
 *            two equally near
 *   A group that holds a NaN, an infinity or a value beyond 2^60 in magnitude
 *   reads back as NaN (codes 0, low = NaN).
 *   Codes: uint8 (blocknum, KV_N, block_size, D/2) or (blocknum, block_size,
 *   KV_N*D/2).  The 16-bit unit (D/32) g + j of a row holds columns 32 j + 4 g
 *   .. + 3, the first in its lowest four bits (g in 0..7, j in 0..D/32-1).
 *   Scales: t (blocknum, KV_N, block_size, D/G, 2), (step, low) of every group,
 *   head-major in both layouts of the codes.  Their shape says what G is.
 *   Steps must be within [2^-60, 2^60], or 0 with codes of 0, low values a NaN or at
 *   most 2^60 in magnitude (those written are).
 *   Codes and scales are 16-byte aligned; keys and values agree in all this.
 *
 * fia_cache_write_int4: fia_cache_write into such a cache.
 *   key, value (T, KV_N, D) of type t, token strides and slot_mapping: as
 *          fia_cache_write.  value, value_cache and value_scales may all be
 *          NULL.  Caches and scales may overlap neither one another nor the
 *          inputs.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_cache_write_int4(const fia_tensor* key, int64_t key_token_stride, const fia_tensor* value,
                           int64_t value_token_stride, const fia_tensor* key_cache, const fia_tensor* value_cache,
                           const fia_tensor* key_scales, const fia_tensor* value_scales,
                           const fia_tensor* slot_mapping, void* stream);

/* ------------------------------------------------------------------------
 * fia_cache_read_int4: the rows of a batch's sequences, as the values they
 * stand for (rounded to t), one sequence after the other: what attention over
 * keys in 16 bits takes (fia_prefill_window with TND keys).
 *   block_table: device int32 (B, W); cu_kv_lens: device int32 (B), running sums
 *          of the sequences' lengths without a leading 0 (the TND lists' form).
 *   key, value: out, t (T, KV_N, D): row cu_kv_lens[b - 1] + i is token i of
 *          sequence b.  Rows from cu_kv_lens[B - 1] on stay as they were, tokens
 *          past T are left out.  Block ids outside the pool, and tokens past the
 *          table's columns, give zeros.  value, value_cache and value_scales may
 *          all be NULL.  Outputs may overlap neither each other nor an input.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_cache_read_int4(const fia_tensor* key_cache, const fia_tensor* value_cache, const fia_tensor* key_scales,
                           const fia_tensor* value_scales, const fia_tensor* block_table,
                           const fia_tensor* cu_kv_lens, const fia_tensor* key, const fia_tensor* value, void* stream);

/* ------------------------------------------------------------------------
 * fia_decode_window_int4: fia_decode_window over such a cache (paged only).
 * Query, lengths, window, sinks, outputs and what rows without a key give: as
 * there; scores and sums are those of the values that the codes stand for,
 * unrounded.  scale_value times a query value must be below 2^116 in magnitude
 * (f16) or fit fp32 (bf16).  Block ids outside the pool read as zeros, blocks that
 * no token sees are not read, and what a key that a token does not see holds has
 * no part in that token's result.
 *   Workspace: partial results, of calls with much work; of others the size is 0
 *          and workspace may be NULL.  No status word: a bounded wait that runs out
 *          (units of more than 32 rows) leaves NaN in the rows that it held up.
 * ------------------------------------------------------------------------ */
FIA_API fia_status fia_decode_window_int4_get_workspace_size(const fia_tensor* query, const fia_tensor* key_cache,
                             const fia_tensor* value_cache, const fia_tensor* key_scales,
                             const fia_tensor* value_scales, const fia_tensor* block_table,
                             const fia_tensor* actual_seq_kvlen, const fia_params* params, int64_t sink_tokens,
                             const fia_tensor* attention_out, const fia_tensor* softmax_lse, size_t* workspace_bytes);
FIA_API fia_status fia_decode_window_int4(const fia_tensor* query, const fia_tensor* key_cache, const fia_tensor* value_cache,
                             const fia_tensor* key_scales, const fia_tensor* value_scales,
                             const fia_tensor* block_table, const fia_tensor* actual_seq_kvlen,
                             const fia_params* params, int64_t sink_tokens, const fia_tensor* attention_out,
                             const fia_tensor* softmax_lse, void* workspace, size_t workspace_bytes, void* stream);

/* Waits for `stream`, then returns the device-side status recorded in a
 * workspace by the last call that used it (FIA_OK or FIA_ERR_TIMEOUT).  The
 * replays of a captured call are one call here: a timeout of one is reported
 * until another call uses the workspace. */
FIA_API fia_status fia_device_status(const void* workspace, void* stream);

/* Static description of a status code. */
FIA_API const char* fia_status_string(fia_status s);

/* Human-readable detail of the last error returned on the calling thread. */
FIA_API const char* fia_last_error(void);

/* Profiling aid: the next fia_prefill / fia_decode / bsa_forward call made on
 * this thread records `start_event` just before its main attention kernel and
 * `stop_event` just after it, on that call's stream, so the caller can time the
 * kernel alone with cudaEventElapsedTime.  Both are cudaEvent_t created by the
 * caller (either may be NULL); the request is consumed by that one call. */
FIA_API void fia_profile_next_call(void* start_event, void* stop_event);

/* Testing aid for the device-side failure path (FIA-v2 / FIA-V5 constraints
 * list "aicore timeout or trap" among the operator's failures): every kernel
 * wait that can give up does so after `ns` nanoseconds instead of the default
 * 2 s, records FIA_ERR_TIMEOUT in the call's status word (fia_device_status),
 * lets its in-flight copies and products finish, frees its tensor memory and
 * returns.  Applies to calls launched afterwards from any thread; 0 restores
 * the default.  A limit far below a kernel's run time makes its calls fail:
 * meant only for tests of that path. */
FIA_API void fia_debug_set_wait_limit_ns(uint64_t ns);

/* How fia_decode_shared_prefix reads the prefix: 0 (the default) by the sizes,
 * 1 always by a kernel of its own, 2 never (each sequence reads it).  Applies
 * to calls launched afterwards from any thread.  Meant for tests that compare
 * the two. */
FIA_API void fia_debug_set_prefix_path(int32_t path);

/* Selects the decode kernel for units (batch, kv head) of at most 16 query
 * rows with head_dim 128: 0 (the default) the warp-level kernel (mma.sync per
 * warp), 1 the tcgen05 kernel that serves larger units.  Both compute the
 * same operation; applies to calls launched afterwards from any thread.
 * Meant for tests that compare the two. */
FIA_API void fia_debug_set_decode_path(int path);

/* Test hook, host only (no device work): the plan fia_decode deals for
 * per-batch lengths kv_len[0..B) (host memory) and N2 kv heads over at most
 * n_cta_max CTAs, with the same per-segment charge as fia_decode.  Writes
 * cta_seg[0..n_cta] (the first segment of each CTA, then the total),
 * segs[4 i .. 4 i + 3] = (unit, first 128-key stage, end stage, part) for each
 * segment in CTA order, unit_parts[2 u .. 2 u + 1] = (first part, parts) for
 * each unit u = b * N2 + kv head, and the counts.  Returns FIA_ERR_SHAPE if a
 * capacity is too small, FIA_ERR_NULL for a NULL pointer. */
FIA_API fia_status fia_debug_plan_decode(const int32_t* kv_len, int B, int N2, int n_cta_max, int32_t* cta_seg,
                                         int cta_seg_cap, int32_t* segs, int segs_cap, int32_t* unit_parts,
                                         int unit_parts_cap, int* n_cta, int* n_segs);

#ifdef __cplusplus
}
#endif

#endif /* FIA_H_ */
