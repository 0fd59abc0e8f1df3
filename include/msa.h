/*
 * msa.h -- C ABI of libmsa: the MiniMax Sparse Attention (MSA) decode hot path
 * on one GB300 (sm_103a).
 *
 * What the path computes (vLLM blog "vLLM 实现 MiniMax-M3.1-Flash 的 Day-0 支持",
 * section "MSA 入门" and its Figure 1):
 *   1. a lightweight indexer scores every key of the paged context with one
 *      index query per GQA group against one shared 128-dim index-key head;
 *   2. the per-key scores are max-pooled to one score per 128-token block;
 *   3. per group the top-k blocks (k = 16 in the model) are kept, the most
 *      recent block always among them;
 *   4. exact softmax attention runs for every query head of the group over
 *      only the selected blocks (at most k x 128 keys).
 * The index scale and the softmax scale are both head_dim ** -0.5 in the model
 * (API page "vllm.models.minimax_m3.nvidia.model", MiniMaxM3SparseAttention:
 * the indexer is built with scale=self.scaling).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every pointer inside the structs and every tensor argument is DEVICE
 *   memory of the current CUDA device unless stated otherwise.  The caller
 *   owns every buffer, the workspace included; the library allocates nothing
 *   and keeps no state beyond cached device attributes.
 * - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *   stream) and never synchronise the host, except msa_read_device_status.
 * - Host-checkable problems (null pointers, unsupported sizes or dtypes, a
 *   workspace that is too small) return an error before any launch.
 *   Launch failures return MSA_ERR_CUDA.  Data-dependent faults found on the
 *   device (a block-table entry outside [0, num_blocks), a sequence length
 *   outside [q_per_seq, max_blocks_per_seq * 128], a selected block id the
 *   query cannot see) set a sticky status word in the workspace; the kernels
 *   skip the offending work (outputs for it are left as documented below)
 *   and never trap.  msa_read_device_status reports and clears that word.
 * - Query token i (0-based) of the q_per_seq new tokens of sequence s sits at
 *   position seq_lens[s] - q_per_seq + i; its keys are already in the cache.
 *   Key t is visible to it iff t <= that position.
 * - Rows of per-query tensors are token-major: row = s * q_per_seq + i.
 *
 * Paged-cache layout (one physical block = 128 tokens; all dims = 128):
 *   K, V        BF16 / FP8: [num_blocks][num_kv_heads][128][head_dim] elements
 *               NVFP4: [num_blocks][num_kv_heads][128][head_dim/2] bytes, element
 *               2j in the low nibble of byte j; e4m3 scales k_sf / v_sf
 *               [num_blocks][num_kv_heads][128][head_dim/16] (one per 16
 *               consecutive elements), fp32 per-tensor k_global / v_global.
 *   FP8 scales  k_scale, v_scale: fp32 [num_blocks][num_kv_heads][128]
 *               (value = e4m3 * scale of its token and head).
 *   INT8 / FP8  K, V as for FP8, one byte an element; k_scale, v_scale: fp32
 *   by blocks   [num_blocks][num_kv_heads], positive (value = code * scale of its
 *               block and head).  Their tokens are written by msa_block_insert.
 *   index keys  one shared head: [num_blocks][128][index_dim] (BF16 / FP8) or
 *               [num_blocks][128][index_dim/2] bytes + idx_sf
 *               [num_blocks][128][index_dim/16] (NVFP4); FP8 per-token fp32
 *               idx_scale [num_blocks][128]; NVFP4 per-tensor idx_global.
 *   The index cache is addressed with the same block table as K/V.
 *   Every base pointer must be 16-byte aligned.
 * Formats: FP8 = OCP E4M3 ("FN": bias 7, no inf); NVFP4 = e2m1 values, one
 * e4m3 scale per 16 elements, one fp32 per-tensor scale (Day-0 blog, section
 * "MiniMax-M3.1 架构中的新特性").  The fp32 value of an NVFP4 element is
 * fp32(e2m1 * e4m3_scale) * global (the inner product is exact in fp32).
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_BLOCK_SIZE 128
#define MSA_HEAD_DIM 128

typedef struct CUstream_st* msa_stream_t; /* == cudaStream_t */

typedef enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad size, misaligned base */
  MSA_ERR_UNSUPPORTED = 2,        /* valid but not implemented (dtype, topk, dims) */
  MSA_ERR_WORKSPACE_TOO_SMALL = 3,
  MSA_ERR_CUDA = 4,               /* a CUDA launch or copy failed */
  MSA_ERR_DEVICE_FAULT = 5,       /* a kernel found bad data (see status word) */
  MSA_ERR_TIMEOUT = 6             /* a bounded on-device wait gave up */
} msa_status_t;

typedef enum {
  MSA_DTYPE_BF16 = 0,
  MSA_DTYPE_FP8_E4M3 = 1,
  MSA_DTYPE_NVFP4 = 2,
  /* K / V caches only: bytes with one fp32 scale for a block of 128 tokens and head */
  MSA_DTYPE_INT8_BLOCK = 8, /* two's complement, -127 to 127 as msa_block_insert writes them */
  MSA_DTYPE_FP8_BLOCK = 9   /* E4M3 codes */
} msa_dtype_t;

/* How an NVFP4 element's two factors combine (vLLM Day-0 blog, "NVIDIA
 * Blackwell 优化的 MSA 内核": the Blackwell kernels dequantize NVFP4 to FP8 with
 * mul.e4m3x4.e2m1x4.e4m3x4, i.e. the product is rounded to E4M3).
 *   MSA_NVFP4_EXACT          e2m1 x e4m3 block scale exactly (it has at most six
 *                            significant bits), then x the fp32 per-tensor scale;
 *   MSA_NVFP4_E4M3_PRODUCT   the product rounded to E4M3 (nearest, ties to even,
 *                            saturating at +-448) first, as that dequant does. */
typedef enum {
  MSA_NVFP4_EXACT = 0,
  MSA_NVFP4_E4M3_PRODUCT = 1
} msa_nvfp4_mode_t;

/* The paged K/V cache and the index-key side cache of one attention layer.
 * K/V dtype and index dtype are independent (the model's
 * --kv-cache-dtype and indexer_kv_dtype settings).  Unused pointers (scales of
 * another format) may be NULL. */
typedef struct {
  msa_dtype_t kv_dtype;
  msa_dtype_t index_dtype;
  int32_t num_blocks;   /* physical blocks in the pool */
  int32_t block_size;   /* must be 128 */
  int32_t num_kv_heads; /* = number of GQA groups = number of index queries per token */
  int32_t head_dim;     /* must be 128 */
  int32_t index_dim;    /* must be 128 */
  const void* k;
  const void* v;
  const void* k_sf;     /* NVFP4 only */
  const void* v_sf;     /* NVFP4 only */
  const float* k_scale; /* FP8 (a token and head), INT8 / FP8 by blocks (a block and head) */
  const float* v_scale;
  const void* idx;
  const void* idx_sf;     /* NVFP4 only */
  const float* idx_scale; /* FP8 only */
  float k_global;       /* NVFP4 only */
  float v_global;
  float idx_global;
  int32_t nvfp4_mode;   /* msa_nvfp4_mode_t, for every NVFP4 tensor of the cache (0 = exact) */
} msa_cache_t;

/* The batch: num_seqs sequences with q_per_seq new query tokens each.
 * seq_lens[s] counts every token of sequence s, the new ones included.
 * block_table[s][b] is the physical block holding logical block b of s. */
typedef struct {
  int32_t num_seqs;
  int32_t q_per_seq;
  int32_t max_blocks_per_seq;   /* row stride of block_table */
  const int32_t* seq_lens;      /* device int32 [num_seqs] */
  const int32_t* block_table;   /* device int32 [num_seqs][max_blocks_per_seq] */
} msa_batch_t;

/* How the per-key index scores of a block pool into the block's score: the
 * indexer's score_type argument (API page "vllm.models.minimax_m3.nvidia.model",
 * MiniMaxM3SparseAttention.__init__: score_type=sparse_cfg.get(
 * "sparse_score_type", "max")).  The pages define only "max"; any other value
 * returns MSA_ERR_UNSUPPORTED. */
typedef enum {
  MSA_SCORE_MAX = 0
} msa_score_type_t;

/* Where msa_decode selects the blocks of a prefill chunk over FP8 caches (more
 * than 8 new tokens a sequence, the tcgen05 indexer).  The selection is the same
 * either way, bit for bit; the two differ in time and workspace. */
typedef enum {
  /* the indexer writes every pooled score, a top-k launch reads them back
     (default: the faster of the two on a 64K-token context) */
  MSA_PREFILL_SELECT_TOPK = 0,
  /* the indexer's epilogue keeps each row's 16 best free blocks as candidate
     lists and a merge launch picks from them: no pooled scores, so the
     workspace does not grow with the context length; topk <= 16 (otherwise,
     and in msa_decode_noalloc when the lists do not fit, the top-k launch) */
  MSA_PREFILL_SELECT_INDEXER = 1
} msa_prefill_select_t;

/* Method settings (the indexer's constructor arguments in the model). */
typedef struct {
  int32_t topk;         /* blocks kept per (query, group): 4, 8, 16 or 32 */
  int32_t init_blocks;  /* leading blocks always kept (model default 0) */
  int32_t local_blocks; /* blocks just before the query's own block always kept (default 0) */
  float index_scale;    /* multiplies the index scores; model: index_dim ** -0.5 */
  float sm_scale;       /* softmax scale; model: head_dim ** -0.5 */
  int32_t score_type;   /* msa_score_type_t; 0 (max) in a zero-initialised struct */
  int32_t prefill_select; /* msa_prefill_select_t; 0 (top-k launch) in a zero-initialised struct */
} msa_config_t;

/* A query tensor: BF16, or FP8 E4M3 codes times one fp32 per-tensor scale. */
typedef struct {
  const void* data;
  msa_dtype_t dtype; /* MSA_DTYPE_BF16 or MSA_DTYPE_FP8_E4M3 */
  float scale;       /* FP8 only */
} msa_query_t;

/* Bytes of workspace msa_decode (and each of the other entry points) needs
 * for this problem.  Host-only; returns 0 for an invalid description.  A
 * prefill chunk (more than 8 new tokens a sequence) over an FP8 cache also
 * holds one partial per (token, q head, selected block) -- o / l in fp16 (with
 * a power-of-two scale that keeps it in range), m, l and that scale in fp32:
 * 272 bytes x tokens x q heads x topk, and with a bf16 query its rows as two
 * e4m3 terms and a factor: 260 bytes x tokens x q heads (605 MB in all for
 * 8,192 tokens x 16 heads x 16).  Over a cache with block scales the attend's part
 * does not grow with the batch. */
size_t msa_workspace_size(const msa_cache_t* cache, const msa_batch_t* batch,
                          const msa_config_t* cfg, int32_t num_q_heads);

/* Clear the device status word at the start of a (fresh) workspace.  Call once
 * after allocating a workspace; the word is sticky across calls until read. */
msa_status_t msa_workspace_init(void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* Indexer score + block max-pool (steps 1-2 above).
 * index_q: [num_seqs * q_per_seq][num_kv_heads][index_dim].
 * pooled:  fp32 [num_seqs * q_per_seq][num_kv_heads][max_blocks_per_seq];
 *          pooled[row][g][b] = index_scale * max over the keys t of block b
 *          visible to that query of <index_q[row][g], index_key[t]>, and -inf
 *          for a block with no visible key (and for b >= the sequence's block
 *          count).  Rows of a sequence with a device fault are left -inf. */
msa_status_t msa_indexer_score(const msa_cache_t* cache, const msa_batch_t* batch,
                               const msa_config_t* cfg, const msa_query_t* index_q,
                               float* pooled, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream);

/* Top-k block selection (step 3) from pooled scores laid out as above.
 * The output keeps the token-major layout of the model's shared top-k buffer
 * (API page "vllm.models.minimax_m3.nvidia.model", MiniMaxM3Model: the
 * indexer writes [tokens, index heads, topk] int32 block ids that the attend
 * reads back).
 * topk_idx:   int32 [num_seqs * q_per_seq][num_groups][topk], the query's own
 *             block ⌊pos/128⌋ always included (forced, together with the
 *             init/local blocks), the remaining slots filled with the highest
 *             pooled scores of the earlier blocks (equal scores: smaller block
 *             id first), ascending, padded with -1 when fewer blocks exist.
 * topk_score: optional fp32 [same shape], the pooled score of each entry
 *             (-inf for padding); may be NULL. */
msa_status_t msa_topk_blocks(const msa_batch_t* batch, const msa_config_t* cfg,
                             int32_t num_groups, const float* pooled, int32_t* topk_idx,
                             float* topk_score, void* workspace, size_t workspace_bytes,
                             msa_stream_t stream);

/* Sparse attend (step 4): for query head h of group g = h / (num_q_heads /
 * num_kv_heads), exact softmax attention over the visible keys of the blocks
 * topk_idx[row][g][*] (entries < 0 are skipped), logits scaled by sm_scale.
 * q:   [num_seqs * q_per_seq][num_q_heads][head_dim].
 * out: bf16 [num_seqs * q_per_seq][num_q_heads][head_dim] (caller-allocated).
 * lse: optional fp32 [num_seqs * q_per_seq][num_q_heads], natural-log
 *      log-sum-exp of the scaled logits; may be NULL.
 * A row whose selection holds no visible key gets out = 0, lse = -inf.
 * Entries naming a block the query cannot see, or repeating a block an
 * earlier entry of the same row names, are left out and raise the device
 * fault flag: the softmax runs over the selected key set, each key once.
 * Caches with block scales: num_q_heads / num_kv_heads <= 64, q_per_seq * num_kv_heads *
 * (topk + 1) < 2^32, workspace 16-byte aligned; equal calls give equal bits on one GPU. */
msa_status_t msa_sparse_attend(const msa_cache_t* cache, const msa_batch_t* batch,
                               const msa_config_t* cfg, const msa_query_t* q,
                               int32_t num_q_heads, const int32_t* topk_idx, void* out,
                               float* lse, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream);

/* The whole path in one call on one stream (score -> pool -> top-k -> attend),
 * no host synchronisation.  topk_idx (output, layout as in msa_topk_blocks)
 * receives the selection; out / lse as in msa_sparse_attend. */
msa_status_t msa_decode(const msa_cache_t* cache, const msa_batch_t* batch,
                        const msa_config_t* cfg, const msa_query_t* index_q,
                        const msa_query_t* q, int32_t num_q_heads, int32_t* topk_idx,
                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                        msa_stream_t stream);

/* Cache insert: write the K, V and index key of num_tokens new tokens into
 * the paged caches, quantized to the caches' formats -- the step just before
 * the path (Day-0 blog, section "QKV GEMM + norm + RoPE + KV 插入融合": K, V and
 * the index key are quantized and written straight into their caches; PR
 * "[M3] Enable FP8 sparse GQA", items 1 and 4: FP8 values stored through the
 * slot mapping).
 * slot_mapping: device int32 [num_tokens]; token t goes to physical block
 *   slot / 128, row slot % 128; negative entries are skipped (padding);
 *   entries at or beyond num_blocks * 128 raise the device fault flag
 *   (MSA_ERR_DEVICE_FAULT from msa_read_device_status) and are skipped.
 * k, v: device bf16 [num_tokens][num_kv_heads][head_dim]; index_k: device bf16
 *   [num_tokens][index_dim], or NULL to leave the index cache alone.  16-byte
 *   aligned.
 * Formats (per 128-element row, all arithmetic one fp32 operation each):
 *   BF16   the bits are copied;
 *   FP8    scale = amax / 448 (1 for an all-zero row) into k_scale / v_scale /
 *          idx_scale, codes = E4M3(x / scale), round to nearest even,
 *          saturating at +-448, the sign of a zero kept;
 *   NVFP4  with the cache's per-tensor k_global / v_global / idx_global g
 *          (the caller's calibrated scale), per 16 elements
 *          sf = E4M3(amax16 / (6 g)) into k_sf / v_sf / idx_sf and codes =
 *          E2M1(x / (sf * g)) (0 where sf * g = 0), round to nearest even,
 *          saturating at +-6, a value that rounds to zero stored as +0;
 *          element 2j in the low nibble of byte j.
 * The call writes through the cache struct's data and scale pointers (they are
 * declared const for the read-only entry points).  workspace: at least 256
 * bytes; only its status word is used.  Rows of one token may be written in
 * any order; two tokens mapped to one slot race.
 * A cache with block scales: k and v must be NULL (else MSA_ERR_UNSUPPORTED) and
 * only the index keys are written; K and V go through msa_block_insert. */
msa_status_t msa_cache_insert(const msa_cache_t* cache, int32_t num_tokens, const int32_t* slot_mapping,
                              const void* k, const void* v, const void* index_k, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream);

/* Consecutive tokens of each sequence: those at the positions first[s] to
 * end[s] - 1 of sequence s are rows token_offsets[s], token_offsets[s] + 1, ... of
 * the call's row tensors (none where end[s] <= first[s]).  Beside msa_build_tables
 * first is its cached_lens, end its seq_lens and token_offsets its token_offsets: a
 * request that waits, has ended or was refused has no tokens then. */
typedef struct {
  int32_t num_seqs;
  int32_t max_blocks_per_seq;    /* row stride of block_table */
  const int32_t* first;          /* device int32 [num_seqs] */
  const int32_t* end;            /* device int32 [num_seqs] */
  const int32_t* token_offsets;  /* device int32 [num_seqs] (more are not read) */
  const int32_t* block_table;    /* device int32 [num_seqs][max_blocks_per_seq] */
} msa_spans_t;

/* bf16 rows of a projection: element d of head h of token t at data[t * stride +
 * h * 128 + d] (a slice of a fused projection's output).  data 16-byte aligned,
 * stride a multiple of 8 elements. */
typedef struct {
  const void* data;
  int64_t stride;
} msa_rows_t;

/* Block insert: K and V of the spans' tokens (num_tokens rows of num_kv_heads heads)
 * into a cache with block scales.  For each block and head, K and V each by itself,
 * with Q = 127 (INT8) or 448 (E4M3), every operation one in fp32:
 *   need  = max(amax / Q, 2^-126), amax over the finite new elements;
 *   a block whose first row is among the call's tokens starts anew: scale = need;
 *   another one holds the sequence's tokens up to first[s]: scale = the old one x
 *   2^k, with the least k >= 0 that makes it need or more (an old scale that is not
 *   a positive normal number counts as 2^-126), and where k > 0 the codes of the
 *   tokens held become round(code x 2^-k);
 *   code  = round(x / scale), to nearest even, saturating at +-Q; NaN becomes 0 in
 *   INT8 and NaN in E4M3.
 * So E4M3 codes of a block that grows move exactly down to E4M3's subnormals, and INT8
 * codes are off by less than one step of the present scale however often it grew.
 * A scale does not shrink while its block holds tokens: where tokens are written again
 * (first[s] moved back, as behind a draft that was refused), the scale and the codes that
 * were rounded for it stay as they became, unless the block's first row is written again too.
 * Rows of a block behind end[s] are left as they were.
 * Flagged on the device and skipped: a span with first < 0 or end beyond
 * max_blocks_per_seq * 128, a span whose rows are not all inside num_tokens, and the
 * tokens of a block outside the pool.  num_tokens <= 2^27.  A block may be in the spans of one sequence
 * only (two race).  What the call writes (the cache's K, V and scales) may overlap
 * nothing that it reads, nor itself (MSA_ERR_INVALID_ARGUMENT).
 * The call writes through the cache's pointers.  Deterministic.  workspace: at least
 * 256 bytes; only its status word is used. */
msa_status_t msa_block_insert(const msa_cache_t* cache, const msa_spans_t* spans, int32_t num_tokens,
                              const msa_rows_t* k, const msa_rows_t* v, void* workspace, size_t workspace_bytes,
                              msa_stream_t stream);

/* Cache read: the spans' tokens back as bf16 rows (num_tokens rows of num_kv_heads
 * heads), from a cache of any format: the fp32 value of the element (msa_dequant_debug),
 * rounded to nearest even; a BF16 cache's bits are copied.  k or v may be NULL.
 * The call writes through their data pointers, only rows that are a span's; it
 * flags and skips what msa_block_insert does.  Spans may share blocks, not rows.
 * The rows written may overlap nothing that the call reads, nor each other (slices
 * of one tensor side by side do not): MSA_ERR_INVALID_ARGUMENT.
 * workspace: at least 256 bytes; only its status word is used. */
msa_status_t msa_cache_read(const msa_cache_t* cache, const msa_spans_t* spans, int32_t num_tokens, const msa_rows_t* k,
                            const msa_rows_t* v, void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* Dense attend: the layers of the model that select no blocks.  For query head
 * h of KV head g = h / (num_q_heads / num_kv_heads), exact softmax attention over
 * every visible key of the sequence, logits scaled by cfg->sm_scale (the only
 * field of cfg it reads; the others must be valid).
 * q, out, lse: as in msa_sparse_attend.  q_per_seq <= 8 and num_q_heads /
 * num_kv_heads <= 64, else MSA_ERR_UNSUPPORTED.
 * Lengths: seq_lens[s] from 0 up.  0 is a padding row of the batch: out 0, lse
 * -inf.  With 0 < seq_lens[s] < q_per_seq the first new tokens sit at negative
 * positions, see no key, and get out 0, lse -inf.  A length below 0 or beyond
 * max_blocks_per_seq * 128 raises the device fault flag; its rows get out 0, lse
 * -inf.  A block-table entry outside the pool is flagged and its keys are left
 * out.  Entries past a sequence's last block are not read.
 * What the cache holds past a sequence's end (NaN or infinity among it) and what
 * the tokens after a query's own position hold reaches no output of that query (over
 * a cache with block scales other than through the scale of a block it sees).
 * The result does not depend on timing: equal calls give equal bits on one GPU.
 * workspace: msa_dense_workspace_size bytes, 16-byte aligned, msa_workspace_init
 * as for the other entry points (and it may be shared with them); calls that
 * overlap on the GPU need workspaces of their own. */
size_t msa_dense_workspace_size(const msa_cache_t* cache, const msa_batch_t* batch, int32_t num_q_heads);
msa_status_t msa_dense_attend(const msa_cache_t* cache, const msa_batch_t* batch, const msa_config_t* cfg,
                              const msa_query_t* q, int32_t num_q_heads, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream);

/* Rotary positions (model page, MiniMaxM3SparseAttention: partial rotary
 * positions; with several axes -- time, height, width -- for images and video).
 * Pair i of a row's first rotary_dim elements turns by
 *   2 pi * positions[axis[i]][t] * turns[i] / 2^64
 * (a, b) -> (a cos - b sin, a sin + b cos).  The pair is elements (i, i +
 * rotary_dim / 2) (MSA_ROPE_HALVES) or (2i, 2i + 1) (MSA_ROPE_ADJACENT).
 * msa_rope_init fills the struct on the host: frequencies theta^(-2i /
 * rotary_dim), the pairs given to the axes in consecutive sections (sections[a]
 * pairs for axis a, rotary_dim / 2 in all).  A caller with other frequencies
 * or another order of axes writes `turns` and `axis` itself (turns a position x
 * 2^64, modulo 2^64; a negative frequency is its two's complement). */
#define MSA_ROPE_MAX_AXES 4
typedef enum {
  MSA_ROPE_HALVES = 0,
  MSA_ROPE_ADJACENT = 1
} msa_rope_layout_t;
typedef struct {
  int32_t rotary_dim;  /* 16 to 128, a multiple of 16 */
  int32_t axes;        /* 1 to MSA_ROPE_MAX_AXES */
  int32_t layout;      /* msa_rope_layout_t */
  uint8_t axis[64];
  uint64_t turns[64];
} msa_rope_t;
msa_status_t msa_rope_init(msa_rope_t* rope, int32_t rotary_dim, double theta, int32_t axes, const int32_t* sections,
                           int32_t layout);

/* Per-head RMS norm before the rotation: y = x * rsqrt(mean x^2 + eps) * (offset
 * + w), w bf16 [128], 16-byte aligned, shared by the heads of a kind (offset 1 for
 * weights stored around zero, as the model's Gemma-style norm does, else 0).  A
 * null weight: that kind is not normed. */
typedef struct {
  const void* q;
  const void* k;
  const void* index_q;
  const void* index_k;
  float eps;
  float offset;
} msa_qk_norm_t;

/* Rotary insert: the step between the projections and the path.  Norm (norm may
 * be NULL) and rotation of q, index q, k and index k in fp32, then one rounding:
 *   q_out, index_q_out  [num_tokens][heads][128], bf16, or E4M3 codes of y * (1 /
 *                       scale) (fp32, round to nearest even, saturating);
 *   k, v, index k       into the caches through slot_mapping, by the formats'
 *                       rules of msa_cache_insert (v is neither normed nor turned).
 * positions: device int32 [axes][num_tokens], any values.
 * slot_mapping: as in msa_cache_insert (negative: that token's keys and values
 *   are not stored, its queries are still written; beyond the pool: the same,
 *   and flagged).  Two tokens mapped to one slot race.
 * index_q / index_q_out (num_kv_heads heads) may both be NULL, as may index_k.
 * A cache with block scales: k and v must be NULL (else MSA_ERR_UNSUPPORTED), the
 * queries and index keys are written as ever, and K and V go through msa_block_insert
 * (where there is no index query, the rows of K may take its place: normed with
 * norm->index_q, turned, and written as bf16 rows to index_q_out).  K is rounded to
 * bf16 on that way (2^-8 of an element), before the block's own rounding.
 * q_out may be q's own memory when q is dense (stride = heads * 128) and bf16.
 * The call writes through q_out's, index_q_out's and the cache's pointers.
 * workspace: at least 256 bytes; only its status word is used. */
msa_status_t msa_rope_insert(const msa_cache_t* cache, const msa_rope_t* rope, int32_t num_tokens,
                             const int32_t* positions, const int32_t* slot_mapping, int32_t num_q_heads,
                             const msa_rows_t* q, const msa_query_t* q_out, const msa_rows_t* index_q,
                             const msa_query_t* index_q_out, const msa_rows_t* k, const msa_rows_t* v,
                             const msa_rows_t* index_k, const msa_qk_norm_t* norm, void* workspace,
                             size_t workspace_bytes, msa_stream_t stream);

/* Block tables, lengths, slots and positions of one step, from the requests'
 * lengths, on the GPU.
 * Request s has cached_lens[s] tokens in the cache (its row of block_table names
 * their blocks) and new_lens[s] new ones: 0 for a request that waits, -1 for one
 * that has ended.  free_blocks[0 .. *free_count) is a stack of free blocks.
 *   1. The blocks of the ended requests go on top of the stack, in the order of
 *      the requests; their rows of block_table are left as they are.  Entries
 *      outside [0, num_blocks) are flagged and left out.
 *   2. Each request takes the blocks its new tokens need beyond those it has off
 *      the top of the stack, in the order of the requests, into its row.
 * Outputs:
 *   seq_lens       [num_seqs] cached + new (0 for an ended request): the batch's lengths
 *   token_offsets  [num_seqs + 1] exclusive sums of the new tokens (those of the
 *                  refused ones among them; a sum beyond 2^30 is given as 2^30)
 *   slot_mapping, positions  [max_tokens] for new token i of request s, at
 *                  token_offsets[s] + i: its slot and its position cached + i;
 *                  -1 and 0 behind the last token
 *   free_count_out the stack's new size
 * The call reads its inputs while it writes: no array that it writes may overlap
 * another one or an input (MSA_ERR_INVALID_ARGUMENT).
 * A request whose blocks are not there, or whose tokens end beyond max_tokens,
 * is refused (and so is every later one that wants tokens behind it): its length
 * stays cached_lens[s], its slots are -1, it takes no block, and the device fault
 * flag is raised.  A malformed request (a length below 0, new_lens below -1, more
 * than max_blocks_per_seq * 128 tokens) is flagged and counts as length 0.  Blocks
 * outside [0, num_blocks) are flagged; their slots are -1.  Returned blocks beyond
 * free_capacity are dropped and flagged.
 * num_seqs <= 8192, max_tokens < 2^30.  Deterministic.  workspace: at least 256
 * bytes; only its status word is used. */
msa_status_t msa_build_tables(int32_t num_seqs, int32_t num_blocks, const int32_t* cached_lens, const int32_t* new_lens,
                              int32_t max_blocks_per_seq, int32_t* block_table, int32_t free_capacity,
                              int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
                              int32_t* seq_lens, int32_t* token_offsets, int32_t max_tokens, int32_t* slot_mapping,
                              int32_t* positions, void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* Synchronise `stream`, read and clear the workspace's status word.
 * Returns MSA_OK, MSA_ERR_DEVICE_FAULT or MSA_ERR_TIMEOUT; *detail (optional,
 * host pointer) receives the raw flag bits. */
msa_status_t msa_read_device_status(void* workspace, msa_stream_t stream, int32_t* detail);

/* Static, human-readable name of a status code. */
const char* msa_status_string(msa_status_t status);

/* Test hook: the fp32 value of every element of the given physical blocks.
 * which: 0 = K, 1 = V (out fp32 [n][num_kv_heads][128][head_dim]),
 *        2 = index keys (out fp32 [n][128][index_dim]).
 * phys_blocks: device int32 [n].  Entries outside [0, num_blocks) produce NaN
 * rows.  The values are bit-identical to the definition in the format notes
 * above (one fp32 rounding for FP8 and NVFP4). */
msa_status_t msa_dequant_debug(const msa_cache_t* cache, int32_t which,
                               const int32_t* phys_blocks, int32_t n, float* out,
                               msa_stream_t stream);

/* Allocation-free variant of msa_decode (no counterpart in the paper; a
 * deployment convenience).  Some callers cannot allocate device memory for a
 * workspace: code running inside another framework's memory pool, a plugin
 * that must not call cudaMalloc (or a framework allocator) on its hot path, a
 * process whose device memory is reserved up front.  This entry point uses a
 * fixed scratch array inside the library instead of a caller workspace; it
 * allocates nothing and calls no allocating routine.
 *   - Limit: the problem's msa_workspace_size must be at most
 *     MSA_NOALLOC_SCRATCH_BYTES (8 MiB, held on every GPU that loads the
 *     library until the process exits); larger problems return
 *     MSA_ERR_WORKSPACE_TOO_SMALL before any launch.
 *   - The first call on each device looks up the scratch's device address
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *     The address is kept for the life of the process: resetting the device
 *     (cudaDeviceReset) and calling again is not supported.
 *   - Every call shares the one scratch array, which keeps the last call's
 *     contents; each call clears what must start at zero.  Calls that overlap
 *     on the GPU (other streams, other host threads) race on it: serialise them.
 *   - status_out: optional device int32[2]; receives this call's device status
 *     flags (the same bits msa_read_device_status reports) at the end of the call.
 * Arguments, outputs and errors are otherwise those of msa_decode. */
#define MSA_NOALLOC_SCRATCH_BYTES (8u << 20)
msa_status_t msa_decode_noalloc(const msa_cache_t* cache, const msa_batch_t* batch,
                                const msa_config_t* cfg, const msa_query_t* index_q,
                                const msa_query_t* q, int32_t num_q_heads, int32_t* topk_idx,
                                void* out, float* lse, int32_t* status_out, msa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
