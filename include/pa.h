/*
 * pa.h -- C ABI of the paged-attention forward library (GB300, sm_103a).
 *
 * The library computes attention over a key/value cache that is stored in
 * fixed-size physical blocks and reached through a per-sequence block table.
 * The operations follow these passages:
 *
 *   pa_decode        "Perhatian berhalaman" (HF transformers docs), section
 *                    "Jalur decode": one query token per sequence; the cache
 *                    is indexed through block_table[batch, max_blocks_per_seq]
 *                    and updated in place; cache_seqlens gives each
 *                    sequence's cached length.  "39 · PagedAttention"
 *                    (inference-notes), sections 1-3: score every key of the
 *                    sequence in logical order, one softmax, weighted sum of
 *                    the values; partial results merge with
 *                    m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m).
 *   pa_cache_update  "Perhatian berhalaman", section "Jalur Varlen" ->
 *                    "Perilaku cache": the varlen kernel cannot reach the
 *                    paged cache, so the cache is written and read by a
 *                    separate update step.
 *   pa_varlen        "Perhatian berhalaman", section "Jalur Varlen" ->
 *                    "Mekanisme pengindeksan" / "Contoh": packed requests,
 *                    cumulative lengths cu_seq_lens_q / cu_seq_lens_k,
 *                    maxima max_length_q / max_length_k.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every pointer argument is DEVICE memory owned by the caller, unless a
 *    parameter says otherwise.  The library allocates and frees nothing and
 *    keeps no pointer after a call returns.
 *  - Every call is asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL is the legacy default stream) and never synchronises the host.
 *  - Tensors are dense and row-major (C order), with the shapes given below.
 *    q/k/v/out element type is selected by `dtype` and is the same for all of
 *    them.  Index arrays are int32.
 *      KV pool  k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim]
 *      decode   q, out            [batch, num_heads, head_dim]
 *               k_new, v_new      [batch, num_kv_heads, head_dim]
 *      varlen   q, out            [total_q, num_heads, head_dim]
 *               k, v              [total_k, num_kv_heads, head_dim]
 *  - Query head h reads kv head h / (num_heads / num_kv_heads).
 *  - softmax_scale <= 0 selects 1 / sqrt(head_dim).
 *  - Return value: PA_OK, or a negative PA_ERR_* code for misuse the host can
 *    see (null pointer, unsupported shape or dtype, short workspace).  On a
 *    negative return nothing was launched and no memory was touched.
 *  - Problems only the device can see (a needed block_table entry that is
 *    not a valid block, a length beyond the table, inconsistent cumulative
 *    lengths) set bits PA_DEVERR_* in *dev_err with an atomic OR, if dev_err
 *    is not NULL; the affected outputs are written as zeros and no
 *    out-of-range address is touched.  The kernels never trap and every
 *    wait inside them is bounded (PA_DEVERR_TIMEOUT).  The caller clears
 *    *dev_err when it wants to.
 *
 * Supported: dtype PA_BF16 or PA_F32; head_dim 64 or 128; for PA_BF16
 * decode, block_size 16 or 32 and num_heads / num_kv_heads <= 8.  The bf16
 * varlen calls (pa_varlen, pa_varlen_paged) run the tensor-core kernel, built
 * for head_dim 128 only: head_dim 64 returns PA_ERR_UNSUPPORTED there.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PA_F32 = 0, PA_BF16 = 1 } pa_dtype;

enum {
    PA_OK = 0,
    PA_ERR_NULL = -1,        /* a required pointer is NULL */
    PA_ERR_DTYPE = -2,       /* dtype not PA_F32 / PA_BF16 */
    PA_ERR_SHAPE = -3,       /* inconsistent or negative sizes */
    PA_ERR_UNSUPPORTED = -4, /* valid but not built: head_dim, block_size, group size */
    PA_ERR_WORKSPACE = -5,   /* workspace NULL or smaller than the query says */
    PA_ERR_LAUNCH = -6,      /* the CUDA runtime refused a launch or a setup call */
    PA_ERR_DEVICE = -7       /* no usable CUDA device / not an sm_103 GPU */
};

/* bits of *dev_err */
#define PA_DEVERR_BAD_BLOCK 1 /* a needed block_table entry is < 0 or >= num_blocks, or a slot
                                 lies beyond the pool */
#define PA_DEVERR_OVERFLOW 2  /* a position lies beyond max_blocks_per_seq * block_size,
                                 or a length is negative */
#define PA_DEVERR_BAD_CU 4    /* cu_seq_lens not non-decreasing, or cu_seq_lens_k does not
                                 equal cache_seqlens + q lengths in pa_cache_update */
#define PA_DEVERR_TIMEOUT 8   /* a bounded wait inside a kernel gave up */
#define PA_DEVERR_NO_SPACE 16 /* pa_block_tables: too few free blocks, or slot_map too short */

/* as a length of pa_decode_q4: the sequence takes no part in the call */
#define PA_LEFT_OUT INT32_MIN

/*
 * Bytes of scratch workspace pa_decode needs for these sizes on the current
 * device (split-K partials and per-sequence merge counters).  0 for PA_F32.
 */
size_t pa_decode_workspace_size(int batch, int num_heads, int num_kv_heads, int head_dim,
                                int block_size, pa_dtype dtype);

/*
 * Decode step: one query per sequence ("Jalur decode").
 *
 * For every sequence b, with L = cache_seqlens[b]:
 *  1. append: k_new[b], v_new[b] are copied bit for bit into the pool at
 *     logical position L, i.e. physical block block_table[b][L / block_size],
 *     slot L % block_size (the worked example: 30 -> block 2 slot 30,
 *     32 -> second block slot 0, 70 -> third block slot 6);
 *  2. attend: out[b, h] = softmax(q[b, h] . K_j * scale) V_j over the
 *     L + 1 positions j = 0..L in logical order, the new token included.
 * cache_seqlens is read only: the caller advances it.  Only the append slot
 * of each sequence is written in the pool; the caller must not map an
 * append slot into a block shared with another sequence.
 *
 * block_table   [batch, max_blocks_per_seq]; entries past the needed blocks
 *               may be -1.  The needed blocks are 0 .. L / block_size.
 * workspace     device scratch of at least pa_decode_workspace_size(...)
 *               bytes (ignored for PA_F32), 16-byte aligned.  It must be
 *               zero-filled before its first use; every call leaves it in a
 *               state the next call accepts (its merge counters back at
 *               zero, whatever the sizes of the call), so one zero fill at
 *               allocation is enough.  After a call that reported
 *               PA_DEVERR_TIMEOUT, zero it again.  Calls that share one
 *               workspace must be ordered on the GPU.  batch * num_kv_heads
 *               may not exceed 262144 (PA_ERR_UNSUPPORTED).
 * Result is independent of where the blocks sit in the pool (bitwise).
 *
 * Host buffers: q, block_table, cache_seqlens, k_new, v_new and out may be
 * page-locked host memory (cudaHostAlloc / cudaMallocHost, or
 * cudaHostRegister-ed), passed as the host pointer.  GB300 reaches such
 * memory in place over NVLink-C2C (unified addressing), so the kernel reads
 * the step's inputs and writes its output there during the call, with no
 * separate copy; a caller that keeps its per-step tensors on the host saves
 * two transfers per step.  k_cache, v_cache, workspace and dev_err must be
 * device memory.  The caller reads `out` after the stream reaches the call.
 */
int pa_decode(const void *q, void *k_cache, void *v_cache, const int32_t *block_table,
              const int32_t *cache_seqlens, const void *k_new, const void *v_new, void *out,
              int batch, int num_heads, int num_kv_heads, int head_dim, int num_blocks,
              int block_size, int max_blocks_per_seq, pa_dtype dtype, float softmax_scale,
              void *workspace, size_t workspace_bytes, int32_t *dev_err, void *stream);

/*
 * pa_decode without a workspace argument, for callers that cannot allocate
 * device memory when they call: a runtime with its own fixed memory budget
 * and no allocator at hand, a plugin handed only its input and output
 * buffers, or code on a path where cudaMalloc is not allowed or would
 * stall the device.  The pages have no counterpart to this entry point; it
 * is a deployment convenience.
 *
 * Same arguments and results as pa_decode with dtype PA_BF16 (bf16 only).
 * The split-K scratch is a 16 MiB array inside the library (device memory
 * reserved on every GPU that loads the library, held until the process
 * exits); the caller still passes every input and output.  Sizes whose
 * scratch need (pa_decode_workspace_size) exceeds 16 MiB are rejected with
 * PA_ERR_WORKSPACE before anything is launched.  The call allocates nothing
 * (no cudaMalloc/cudaFree, no allocating library routine); it clears the
 * merge counters it uses with cudaMemsetAsync on `stream`.
 *
 * The first call on each device looks up the array's device address with
 * that device current (cudaGetSymbolAddress); make that first call before
 * any stream capture.  All calls share the one array per device, which keeps
 * the previous call's contents: calls that may overlap on the GPU (different
 * streams without ordering) race on it and must be serialised by the caller.
 */
int pa_decode_static_scratch(const void *q, void *k_cache, void *v_cache,
                             const int32_t *block_table, const int32_t *cache_seqlens,
                             const void *k_new, const void *v_new, void *out, int batch,
                             int num_heads, int num_kv_heads, int head_dim, int num_blocks,
                             int block_size, int max_blocks_per_seq, float softmax_scale,
                             int32_t *dev_err, void *stream);

/*
 * The contiguous-cache twin of pa_decode, for measuring what paging costs:
 * "39 · PagedAttention" (inference-notes), sections "Ghi chú" and
 * "4. Có miễn phí không?", compares a paged attention kernel with one over a
 * contiguous cache.  This call is that contiguous kernel: the same decode
 * kernel with the block table taken out.
 *
 * k_cache, v_cache  [batch, max_seqlen, num_kv_heads, head_dim]: sequence b
 *                   holds its position t at [b, t].  Nothing is shared
 *                   between sequences and no table is read.
 * For every sequence b, with L = cache_seqlens[b] (read only):
 *  1. append: k_new[b], v_new[b] are copied bit for bit to [b, L];
 *  2. attend: out[b, h] = softmax(q[b, h] . K_j * scale) V_j over positions
 *     j = 0..L of row b.
 * L + 1 > max_seqlen (or L < 0) sets PA_DEVERR_OVERFLOW and zeroes the
 * sequence's output.  Positions past L of a row are never used in the
 * result (whatever they hold).  bf16 only (dtype PA_BF16 implied); head_dim
 * 64 or 128; num_heads / num_kv_heads <= 8; batch * max_seqlen < 2^31.
 * workspace: as pa_decode, at least pa_decode_contiguous_workspace_size(...)
 * bytes, zero-filled before first use.  For the same logical cache contents,
 * the result equals pa_decode's with block_size 16 (head_dim 128) or 32
 * (head_dim 64) bit for bit.
 */
size_t pa_decode_contiguous_workspace_size(int batch, int num_heads, int num_kv_heads,
                                           int head_dim);
int pa_decode_contiguous(const void *q, void *k_cache, void *v_cache,
                         const int32_t *cache_seqlens, const void *k_new, const void *v_new,
                         void *out, int batch, int num_heads, int num_kv_heads, int head_dim,
                         int max_seqlen, float softmax_scale, void *workspace,
                         size_t workspace_bytes, int32_t *dev_err, void *stream);

/*
 * Varlen cache update ("Jalur Varlen" -> "Perilaku cache").
 *
 * k_chunk, v_chunk [total_q, num_kv_heads, head_dim]: the new tokens of all
 * requests, packed by cu_seq_lens_q [batch + 1].  Row i of request b is
 * copied bit for bit into the pool at logical position cache_seqlens[b] + i
 * (cache_seqlens = tokens already cached, read only).
 *
 * If k_full, v_full and cu_seq_lens_k are all non-NULL, request b's rows
 * [cu_seq_lens_k[b], cu_seq_lens_k[b+1]) of k_full/v_full [total_k,
 * num_kv_heads, head_dim] also receive its whole key sequence in logical
 * order: the cached prefix read from the pool, then the chunk.  That
 * requires cu_seq_lens_k[b+1] - cu_seq_lens_k[b] == cache_seqlens[b] +
 * (cu_seq_lens_q[b+1] - cu_seq_lens_q[b]) (PA_DEVERR_BAD_CU otherwise).
 * All three NULL: scatter only.  total_k is ignored then.
 */
int pa_cache_update(const void *k_chunk, const void *v_chunk, const int32_t *cu_seq_lens_q,
                    const int32_t *cache_seqlens, const int32_t *block_table, void *k_cache,
                    void *v_cache, void *k_full, void *v_full, const int32_t *cu_seq_lens_k,
                    int batch, int total_q, int total_k, int num_kv_heads, int head_dim,
                    int num_blocks, int block_size, int max_blocks_per_seq, pa_dtype dtype,
                    int32_t *dev_err, void *stream);

/*
 * Varlen attention ("Jalur Varlen").  Request r owns q rows
 * [cu_seq_lens_q[r], cu_seq_lens_q[r+1]) and k/v rows [cu_seq_lens_k[r],
 * cu_seq_lens_k[r+1]); max_length_q / max_length_k must be at least the
 * largest q / k length (they size the launch).  causal != 0 masks
 * bottom-right: query i of a request with lengths (ql, kl) sees key j iff
 * j <= i + kl - ql.  A query that sees no key gets a zero output row.
 * PA_BF16 runs on the tcgen05 tensor cores and needs head_dim 128
 * (head_dim 64 returns PA_ERR_UNSUPPORTED); PA_F32 runs on CUDA cores with
 * head_dim 64 or 128.
 */
int pa_varlen(const void *q, const void *k, const void *v, const int32_t *cu_seq_lens_q,
              const int32_t *cu_seq_lens_k, int max_length_q, int max_length_k, int causal,
              void *out, int batch, int total_q, int total_k, int num_heads, int num_kv_heads,
              int head_dim, pa_dtype dtype, float softmax_scale, int32_t *dev_err, void *stream);

/*
 * Varlen attention that reads each request's keys straight from the paged
 * pool through its block_table row, with no packed copy: "Perhatian
 * berhalaman", section "Jalur Varlen" -> "Perilaku cache" names the manual
 * cache read of the varlen path as a bottleneck at long lengths, and
 * "39 · PagedAttention" (inference-notes), section "Ghi chú", notes that
 * attention kernels can take the block table directly.  Typical use: scatter
 * the new chunk with pa_cache_update (k_full/v_full NULL), then call this.
 *
 * Request r owns q rows [cu_seq_lens_q[r], cu_seq_lens_q[r+1]) of q/out
 * [total_q, num_heads, head_dim]; its keys are logical positions
 * 0 .. seqlens_k[r]-1 of block_table row r in k_cache/v_cache
 * [num_blocks, block_size, num_kv_heads, head_dim].  Masking, scaling, GQA
 * mapping and empty rows as pa_varlen; for equal inputs the result equals
 * pa_varlen on the gathered keys bit for bit.  seqlens_k[r] beyond
 * max_blocks_per_seq * block_size sets PA_DEVERR_OVERFLOW and zeroes the
 * request's rows; a needed entry that is not a valid block sets
 * PA_DEVERR_BAD_BLOCK and zeroes the affected query tiles.
 * Supported: PA_BF16, head_dim 128, block_size 8, 16, 32 or 64.
 */
int pa_varlen_paged(const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_table, const int32_t *cu_seq_lens_q,
                    const int32_t *seqlens_k, int max_length_q, int max_length_k, int causal,
                    void *out, int batch, int total_q, int num_heads, int num_kv_heads,
                    int head_dim, int num_blocks, int block_size, int max_blocks_per_seq,
                    pa_dtype dtype, float softmax_scale, int32_t *dev_err, void *stream);

/*
 * The 4-bit pool
 * --------------
 * kv_cache of the *_q4 calls is bytes [num_blocks, num_kv_heads, record],
 * record = block_size * (head_dim + 8): the keys and the values of one kv
 * head of one block, side by side, so that one bulk copy brings all a head
 * needs of a block and no line holds another head's bytes.  pa_q4_block_bytes
 * is num_kv_heads * record (0 for sizes that are not supported: head_dim 64
 * or 128, block_size 16 or 32).
 *
 * A row x of head_dim values (one token, one kv head, K or V) is held as
 * head_dim codes n of 4 bits, a step s and a low value b, both bf16; it
 * stands for b + n s.  With fl = rounding to fp32 after each operation:
 *   b   = min x, rounded down to bf16
 *   r   = fl(fl(max x / 16 - b / 16) * fl(16 / 15))
 *   s   = r rounded up to bf16; 0 when r < 2^-100.  While fl(b + 15 s) is
 *         larger than every bf16 number (rows with a value near 3.4e38), s is
 *         the next lower bf16 number instead, twice at most
 *   n_i = round-half-even(fl(fl(x_i / 16 - b / 16) * fl(16 / s))), at most 15
 *         (0 when s = 0)
 * so |x_i - (b + n_i s)| <= s / 2 up to the fp32 roundings.  A row that
 * holds an infinity or a NaN (or fp32 values that round to an infinite b) is
 * held as s = b = NaN, n = 0: the whole row reads back as NaN.
 *
 * Inside a record, for token t of the block and D = head_dim:
 *   K codes  bytes [0, bs*D/2): row t at t*D/2, dim 2i in the low half of
 *            byte i, dim 2i + 1 in its high half;
 *   V codes  bytes [bs*D/2, bs*D): 16-bit units of 4 dims (dim 4x + k in bits
 *            4k..4k+3).  Tokens 2p and 2p + 1 share 32-bit words: unit (t, x)
 *            is unit number 2 (p D/4 + 8 u + x % 8) + t % 2 with p = t / 2 and
 *            u = (x / 8) xor (p % 4) for D = 128, (x / 8) xor (p / 2 % 2) for
 *            D = 64.  A word is then an operand of the tensor cores' value
 *            product (dims on the rows, a token pair in a register) after one
 *            mask, and the xor spreads the loads over the memory banks;
 *   scales   bytes [bs*D, bs*(D+8)): 4 bf16 a token: K step, K low, V step,
 *            V low.
 */
size_t pa_q4_block_bytes(int num_kv_heads, int head_dim, int block_size);

/*
 * Quantise and scatter: row i of k_chunk, v_chunk [total_q, num_kv_heads,
 * head_dim] is written to slot slot_map[i] (physical block * block_size +
 * offset, as pa_block_tables gives them).  Rows whose slot is negative are
 * skipped (padding of a captured step); a slot >= num_blocks * block_size
 * sets PA_DEVERR_BAD_BLOCK and is skipped.  A slot may appear once only: two
 * rows in one slot leave a mixture of both.  dtype is that of the chunk.
 * num_blocks * block_size and total_q * num_kv_heads stay below 2^31 - 64.
 */
int pa_cache_update_q4(const void *k_chunk, const void *v_chunk, const int32_t *slot_map,
                       void *kv_cache, int total_q, int num_kv_heads, int head_dim,
                       int num_blocks, int block_size, pa_dtype dtype, int32_t *dev_err,
                       void *stream);

/*
 * Read back: rows [cu_seq_lens_k[r], cu_seq_lens_k[r+1]) of k_full, v_full
 * [total_k, num_kv_heads, head_dim] receive logical positions 0, 1, .. of
 * request r as values (b + n s in fp32, rounded to dtype), which pa_varlen
 * takes as they are (total_k * num_kv_heads < 2^31 - 64, total_k / block_size +
 * batch < 2^31).  Rows behind cu_seq_lens_k[batch] are left as they were.  A
 * needed block_table entry that is no block sets PA_DEVERR_BAD_BLOCK, a position
 * beyond the table PA_DEVERR_OVERFLOW; those rows are zeroed.  cu_seq_lens_k that does not start at 0, decreases or
 * passes total_k sets PA_DEVERR_BAD_CU; nothing behind total_k is written.
 */
int pa_cache_gather_q4(const void *kv_cache, const int32_t *block_table,
                       const int32_t *cu_seq_lens_k, void *k_full, void *v_full, int batch,
                       int total_k, int num_kv_heads, int head_dim, int num_blocks,
                       int block_size, int max_blocks_per_seq, pa_dtype dtype, int32_t *dev_err,
                       void *stream);

/*
 * pa_decode over the 4-bit pool: the new token is quantised into position
 * L = cache_seqlens[b] and the query attends over positions 0..L as the pool
 * holds them, the new token included (so a later step sees the same value).
 *   out[b, h] = sum_j softmax_j(scale q.K_j) V_j,  K_j = bK_j + sK_j nK_j, V_j likewise
 * q, k_new, v_new, out (and k_stored, v_stored) are of `dtype`; PA_BF16 and
 * PA_F32 run the same tensor-core kernel, fp32 operands as sums of two halves.
 * k_stored, v_stored [batch, num_kv_heads, head_dim], each or both NULL: the
 * values the pool now stands for at L, for a caller that uses them again in
 * this step (a later layer that shares these keys) or watches the error.
 * Left as they were where the sequence's append was refused.
 * A sequence with cache_seqlens[b] = PA_LEFT_OUT takes no part: nothing is
 * appended, its output rows are zeros and no error bit is set (other negative
 * lengths are errors).
 * block_table, cache_seqlens, workspace, device errors, placement and the
 * limits num_heads / num_kv_heads <= 8, batch * num_kv_heads <= 262144 as
 * pa_decode, and batch * max_blocks_per_seq * num_kv_heads < 2^31; every
 * pointer is device memory.  Elements of q above 2^115 may overflow.  A key or value row that is NaN
 * makes the outputs it reaches NaN, as the formula does.  Value steps below
 * 2^-76, or below 2^-24 of the low value, are weighed as the others but may lose
 * their codes (the low value stays).
 */
size_t pa_decode_q4_workspace_size(int batch, int num_heads, int num_kv_heads, int head_dim,
                                   int block_size, pa_dtype dtype);
int pa_decode_q4(const void *q, void *kv_cache, const int32_t *block_table,
                 const int32_t *cache_seqlens, const void *k_new, const void *v_new, void *out,
                 void *k_stored, void *v_stored, int batch, int num_heads, int num_kv_heads,
                 int head_dim, int num_blocks, int block_size, int max_blocks_per_seq,
                 pa_dtype dtype, float softmax_scale, void *workspace, size_t workspace_bytes,
                 int32_t *dev_err, void *stream);

/*
 * One serving step's block tables and slot map, built on the GPU from the
 * requests' lengths: the device counterpart of pa_bm_append / pa_bm_free /
 * pa_bm_tables (no reference counts: blocks shared by several requests stay
 * with the host manager).  The step needs no host copy and can be captured.
 *
 * Request b holds L = cache_seqlens[b] tokens in the first ceil(L / bs)
 * entries of its block_table row, and gets n = new_lens[b] new ones:
 *   n >= 0  ceil((L+n)/bs) - ceil(L/bs) blocks are taken and entered in its
 *           row;
 *   n = -1  the request has ended: its blocks go back and its length becomes 0.
 *           Its row is left as it is and names blocks that others may own by
 *           now, so it must not be decoded with its old length: see
 *           pa_block_tables_decode.
 * free_blocks [num_blocks] is a stack of *num_free block ids (top at the
 * end).  Ended requests push their blocks first, in order of (request,
 * logical block); then the taken blocks are popped in the same order.
 *   slot_map [total_slots]     the new tokens' slots, packed by
 *                              cu_seq_lens_q; -1 behind the last token
 *   cu_seq_lens_q [batch+1]    cumulative new tokens
 *   cu_seq_lens_k [batch+1]    cumulative lengths after the step
 *   seqlens_k [batch]          lengths after the step; may be cache_seqlens
 *   num_free_out [1]           may be num_free
 * All or nothing: with a negative length, n < -1 or a length beyond
 * max_blocks_per_seq * block_size (PA_DEVERR_OVERFLOW), too few free blocks
 * or more new tokens than total_slots (PA_DEVERR_NO_SPACE), a free stack that
 * would not fit num_blocks (PA_DEVERR_BAD_BLOCK) or lengths that add up past
 * 2^31 - 1 (PA_DEVERR_BAD_CU), the step changes no table, stack or length:
 * slot_map is all -1, both cu arrays are 0.  A block id outside the pool met
 * on the way sets PA_DEVERR_BAD_BLOCK, is passed on as -1, and tokens in it
 * get slot -1.  batch <= 16384; num_blocks * block_size < 2^31.
 */
int pa_block_tables(const int32_t *cache_seqlens, const int32_t *new_lens, int32_t *block_table,
                    int32_t *free_blocks, const int32_t *num_free, int32_t *slot_map,
                    int32_t *cu_seq_lens_q, int32_t *cu_seq_lens_k, int32_t *seqlens_k,
                    int32_t *num_free_out, int batch, int total_slots, int num_blocks,
                    int block_size, int max_blocks_per_seq, int32_t *dev_err, void *stream);

/*
 * The same step, and the lengths for the pa_decode_q4 call behind it:
 *   decode_lens [batch]   L where n = 1, the position of the request's one new
 *                         token; PA_LEFT_OUT where n is anything else (nothing
 *                         new, ended, or a chunk for pa_cache_update_q4) and for
 *                         all requests of a refused step
 * so that one decode over the whole batch appends and attends for the requests
 * with a new token and leaves the blocks of the others, and of ended requests'
 * old rows, alone.  decode_lens overlaps no other argument; NULL leaves it out
 * (pa_block_tables).  seqlens_k may still be cache_seqlens, and the two calls be
 * captured together.
 */
int pa_block_tables_decode(const int32_t *cache_seqlens, const int32_t *new_lens,
                           int32_t *block_table, int32_t *free_blocks, const int32_t *num_free,
                           int32_t *slot_map, int32_t *cu_seq_lens_q, int32_t *cu_seq_lens_k,
                           int32_t *seqlens_k, int32_t *num_free_out, int32_t *decode_lens,
                           int batch, int total_slots, int num_blocks, int block_size,
                           int max_blocks_per_seq, int32_t *dev_err, void *stream);

/*
 * Rotary positions
 * ----------------
 * A row of head_dim values has rotary_dim / 2 pairs (x, y): dims (i, rotary_dim / 2 + i),
 * or neighbours (2i, 2i + 1) where `interleaved` is not 0.  Dims from rotary_dim on pass
 * through.  Pair i of a token belongs to axis a = pair_axis[i] (time, height, width, ...)
 * and is turned by that axis' position p = positions[a * tokens + token]:
 *   x' = x c - y s,  y' = y c + x s,  c = cos_sin[p][i],  s = cos_sin[p][rotary_dim / 2 + i]
 * in fp32, rounded once to dtype.  The table holds what the model's frequencies (and their
 * scaling) give, and is the same for all calls.
 *   positions  [num_axes, tokens]
 *   cos_sin    fp32 [max_position, rotary_dim], 16-byte aligned
 *   pair_axis  HOST array of rotary_dim / 2 axes below num_axes; NULL with one axis
 *   q, k, q_out, k_out   rows of a token are dense [heads, head_dim]; from token to token
 *              they are *_stride elements apart (a multiple of 16 bytes; outputs at
 *              least heads * head_dim), so that q and k can be parts of one
 *              projection's output.  An output may be its input (same stride), and
 *              overlaps nothing else.  q or k may be NULL with 0 heads.
 * A position outside [0, max_position) sets PA_DEVERR_OVERFLOW; the token's rows are
 * zeros.  rotary_dim is a multiple of 16 up to head_dim, num_axes at most 4.
 */
int pa_rotary(const void *q, const void *k, const int32_t *positions, const float *cos_sin,
              void *q_out, void *k_out, int tokens, int num_heads, int num_kv_heads, int head_dim,
              int rotary_dim, int max_position, int num_axes, const uint8_t *pair_axis,
              int interleaved, long long q_stride, long long k_stride, long long q_out_stride,
              long long k_out_stride, pa_dtype dtype, int32_t *dev_err, void *stream);

/*
 * pa_rotary and the append to the paged cache in one pass: q is turned into q_out, k is
 * turned and written with v (bit for bit) to slot slot_map[token] (physical block *
 * block_size + offset, as pa_block_tables gives them) of k_cache, v_cache.  A row whose
 * slot is negative is padding: nothing of it is read or written, its row of q_out
 * included.  A slot >= num_blocks * block_size sets PA_DEVERR_BAD_BLOCK, a position
 * outside the table PA_DEVERR_OVERFLOW: the token's q_out is zeros and nothing is
 * appended.  A slot may appear once only: two rows in one slot leave a mixture.
 * rotary_dim 0 appends without turning (positions and cos_sin NULL; q is copied).
 *
 * bounds [num_blocks, num_kv_heads, 2, head_dim] of dtype, or NULL: the least
 * ([.., 0, :]) and the largest ([.., 1, :]) value of each channel over the keys of a
 * block, as pa_select_blocks takes them.  A token at offset 0 starts its block's bounds
 * anew, others widen them; NaN wins.  (Tokens that are taken back and written again leave
 * bounds that may be wider than need be, until the block starts anew.)  The rows of one block have to follow one another,
 * in order of their offsets, with no padding between (as pa_block_tables packs them).  Blocks that get no token
 * are left alone.
 */
int pa_cache_append_rotary(const void *q, const void *k, const void *v, const int32_t *slot_map,
                           void *k_cache, void *v_cache, void *bounds, const int32_t *positions,
                           const float *cos_sin, void *q_out, int tokens, int num_heads,
                           int num_kv_heads, int head_dim, int rotary_dim, int max_position,
                           int num_axes, const uint8_t *pair_axis, int interleaved,
                           long long q_stride, long long k_stride, long long v_stride,
                           long long q_out_stride, int num_blocks, int block_size, pa_dtype dtype,
                           int32_t *dev_err, void *stream);

/*
 * Block-sparse attention
 * ----------------------
 * Queries are packed rows [total_q, num_heads, head_dim] located by cu_seq_lens_q
 * [batch + 1], or one of each request where cu_seq_lens_q is NULL (total_q = batch).
 * Request r has seqlens_k[r] keys in the cache, the new tokens' among them; of its ql
 * queries, query i sees positions 0 .. seqlens_k[r] - ql + i (none where that is
 * negative), so blocks 0 .. that position / block_size.  Rows behind
 * cu_seq_lens_q[batch] are left as they were.  A request whose length is PA_LEFT_OUT takes
 * no part: its rows see nothing.
 *
 * pa_select_blocks: for each query and kv head the logical numbers of top_k of the
 * visible blocks, ascending, -1 behind them where fewer are visible:
 *   selected [total_q, num_kv_heads, top_k]
 * The first first_blocks and the last last_blocks visible ones are always among them;
 * the others are those of largest
 *   score = max over the kv head's query heads g of sum_d max(q_gd, 0) hi_d + min(q_gd, 0) lo_d,
 * which no key between the block's bounds lo, hi exceeds in its product with q_g.  The
 * choice is that of the exact scores (ties: the lowest block; scores that differ by less than
 * 2^-56 of a sum of |q| |bound| may count as equal), whatever the order of the
 * sums (as long as the sums of |q| |bound| lie between 1e-30 and 3e38; a score that overflows
 * is an infinity).  A NaN ranks above all numbers.  Bounds of the last block are used only where last_blocks is
 * 0: a chunk's later tokens are in them.
 * dtype is that of q and bounds.  first_blocks + last_blocks <= top_k;
 * max_blocks_per_seq <= 49152; top_k at most 2^20; num_heads / num_kv_heads <= 8; head_dim 64 or 128;
 * total_q * num_kv_heads < 2^27.  How the work is shared out follows max_blocks_per_seq, not the
 * lengths: a table much wider than the longest request takes up to three times as long.
 * A needed block_table entry that is no block sets PA_DEVERR_BAD_BLOCK, a length beyond
 * the table PA_DEVERR_OVERFLOW: the rows are -1.  cu_seq_lens_q that does not start at 0 or
 * decreases sets PA_DEVERR_BAD_CU; rows are then -1, left as they were or another request's.
 */
int pa_select_blocks(const void *q, const void *bounds, const int32_t *block_table,
                     const int32_t *seqlens_k, const int32_t *cu_seq_lens_q, int32_t *selected,
                     int batch, int total_q, int num_heads, int num_kv_heads, int head_dim,
                     int num_blocks, int block_size, int max_blocks_per_seq, int top_k,
                     int first_blocks, int last_blocks, pa_dtype dtype, int32_t *dev_err,
                     void *stream);

/*
 * pa_sparse: out[t, h] = softmax(scale q[t, h] K^T) V over the visible positions of the
 * logical blocks selected[t, kv head, :] (any order; negative entries and blocks behind
 * the query count nothing, a block that appears twice counts twice).  A row that sees no
 * position is zeros; NaN that a row sees makes its outputs NaN, an infinite value those
 * it reaches infinite or NaN.  selected, queries and lengths as above; the caches as pa_decode,
 * whose tokens are all written already (nothing is appended).
 * dtype PA_BF16 or PA_F32; num_heads / num_kv_heads <= 8; head_dim 64 or 128; PA_BF16: block_size
 * a multiple of 16; top_k at most 2^20, top_k * block_size < 2^30,
 * total_q * num_kv_heads < 2^27.  A needed block_table entry that is no block sets PA_DEVERR_BAD_BLOCK, a length
 * beyond the table PA_DEVERR_OVERFLOW: the rows are zeros; a bad cu_seq_lens_q as above.
 * Needs no workspace; calls share nothing.
 */
int pa_sparse(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
              const int32_t *seqlens_k, const int32_t *cu_seq_lens_q, const int32_t *selected,
              void *out, int batch, int total_q, int num_heads, int num_kv_heads, int head_dim,
              int num_blocks, int block_size, int max_blocks_per_seq, int top_k, pa_dtype dtype,
              float softmax_scale, int32_t *dev_err, void *stream);

/* Static description of a status code (never NULL). */
const char *pa_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
