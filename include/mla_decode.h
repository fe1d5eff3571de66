/*
 * mla_decode.h -- C ABI of libmla_decode.so: paged multi-head-latent-attention (MLA)
 * decode with decode-context-parallel (DCP) shards, the LSE merge of shard partials,
 * DCP slot mapping, the 8-bit form of the paged cache (a step's tables from request
 * lengths, the quantising store, the decode over it), and prompt processing (rotary positions,
 * the append with rotation, the heads' keys and values, the attention of chunks of new
 * tokens), for NVIDIA GB300 (sm_103a).
 *
 * Sources (web pages summarising vLLM pull requests):
 *   [#52188] "支持 Kimi-K3 DSpark 推测解码与 DCP 并行组合" (vLLM PR 52188)
 *   [#54012] "带 DCP 的 MLA decode 改用 FlashInfer 原生 CP mask" (vLLM PR 54012)
 *   [#48180] "为 TokenSpeed MLA 后端添加 DCP 与 Eagle 支持" (vLLM PR 48180)
 *
 * Conventions shared by every call:
 *   - Every pointer argument is a DEVICE pointer owned by the caller, unless stated.
 *     The library allocates no memory when called.  Its device state is one status word
 *     per device (see mla_get_device_status) and the fixed scratch array that
 *     mla_decode_noalloc uses; its host state is per-device launch settings, filled on
 *     a device's first call.
 *   - Every call is asynchronous on `stream` (the legacy default stream when NULL) and
 *     returns one of the MLA_* codes.  Argument errors are found on the host before
 *     anything is launched; mla_last_error() then returns a message (thread-local).
 *   - Calls are stream-ordered: a call's kernels see every result issued before it on
 *     the stream.  The split-KV combine of mla_decode, the kernel of lse_merge, both
 *     kernels of mla_decode_q8 and those of mla_rope, cp_rope_store, mla_expand, mla_prefill
 *     and lse_merge_v are programmatic dependent launches: they may be scheduled while the
 *     kernel before them drains, but wait for its completion before they read or write
 *     memory (and let one behind them be scheduled in the same way).
 *   - bf16 means IEEE bfloat16 stored as 16-bit words; results are rounded to nearest
 *     even.  Tensors are dense and row-major unless a stride is given.
 */
#ifndef MLA_DECODE_H_
#define MLA_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, without pulling in the CUDA headers. */
typedef struct CUstream_st* mla_stream_t;

#define MLA_OK 0
#define MLA_ERR_INVALID_ARGUMENT (-1) /* null pointer, bad size, range or alignment    */
#define MLA_ERR_UNSUPPORTED (-2)      /* valid request this build does not implement   */
#define MLA_ERR_CUDA (-3)             /* a CUDA runtime call or kernel launch failed    */
#define MLA_ERR_DEVICE (-4)           /* a kernel flagged bad data (see status word)    */

#define MLA_PAD_SLOT_ID (-1)   /* slot of a position this rank does not own            */
#define MLA_HEAD_DIM_QK 576    /* 512 latent (kv_lora_rank) + 64 rope dims            */
#define MLA_HEAD_DIM_V 512     /* V is the first 512 dims of each latent KV row        */
#define MLA_MAX_Q_LEN 16

/* Bits of the device status word. */
#define MLA_STATUS_BAD_PAGE 1u        /* block_table entry outside [0, num_blocks)      */
#define MLA_STATUS_SEQ_TOO_LONG 2u    /* seq_lens[b] > max_blocks * block_size          */
#define MLA_STATUS_BAD_VBLOCK 4u      /* cp_local_slot: virtual block >= max_blocks     */
#define MLA_STATUS_WAIT_TIMEOUT 8u    /* a bounded on-chip wait gave up                 */
#define MLA_STATUS_BAD_SCALE 16u      /* a scale of the 8-bit cache outside its range   */
#define MLA_STATUS_OUT_OF_PAGES 32u   /* cp_step_tables: too few free pages             */
#define MLA_STATUS_BAD_STEP 64u       /* a length or a ring state outside its range     */

/* (major << 16) | minor: what mla_abi_version() of a library built with this header returns. */
#define MLA_ABI_VERSION ((2 << 16) | 2)

/* The 8-bit cache: e4m3 rows, one float scale for every MLA_Q8_GROUP consecutive slots of
 * a page; a scale is at least MLA_Q8_SCALE_MIN and at most MLA_Q8_SCALE_MAX. */
#define MLA_Q8_GROUP 16
#define MLA_Q8_SCALE_MIN 2.3283064365386963e-10f /* 2^-32 */
#define MLA_Q8_SCALE_MAX 1.8446744073709552e19f  /* 2^64  */

/*
 * Bytes of workspace that mla_decode uses to split one request's KV range over several
 * thread blocks (split-KV) for a batch of B requests, H query heads, q_len query rows
 * and a device with num_sms SMs.  Passing less (or NULL) is allowed: the call then uses
 * fewer splits, down to none.  Pure function of its arguments; no CUDA call.
 */
size_t mla_decode_workspace_size(int B, int H, int q_len, int num_sms);

/*
 * mla_decode -- one shard's partial attention for a batch of multi-token decode blocks.
 *
 * Defines ([#54012] "关键源码片段", the native-DCP call; [#52188] "关键源码片段",
 * _prepare_flattened_decode_metadata; [#48180] "实现拆解" step 1):
 *   global position g lives on rank (g / interleave) % cp_world (round-robin segments of
 *   `interleave` positions); with span = cp_world * interleave a global prefix of G
 *   positions holds local_len(G) = G / span * interleave
 *                                  + clamp(G % span - cp_rank * interleave, 0, interleave)
 *   of this shard's keys.  causal != 0: query row i (0 <= i < q_len) of request b sees the
 *   global prefix G_i = max(0, causal_seqlens_global[b] - (q_len - 1 - i)), i.e.
 *       L_i = min(seq_lens[b], local_len(G_i))
 *   local keys; causal == 0 (a non-causal draft block, the snippet's other branch): every
 *   row reads the shard's whole local sequence, L_i = seq_lens[b].  The local key l < L_i
 *   is row kv_cache[block_table[b*bt_stride + l/block_size]][l % block_size].  With
 *   s_l = scale * <q_row, key_l> over all 576 dims,
 *       out = sum_l softmax(s)_l * key_l[0:512],   lse = log(sum_l exp(s_l)),
 *   lse in natural log when lse_base_e != 0, else in log2.  A row with L_i = 0 gets
 *   out = 0 and lse = -inf.
 *
 * Arguments:
 *   q            bf16 [B, q_len, H, 576], 16-byte aligned.
 *   kv_cache     bf16 [num_blocks, block_size, 576] (this shard's pool), 16-byte aligned;
 *                block_size 16, 32 or a multiple of 64.
 *   block_table  int32 [B, bt_stride]; only the first ceil(L/block_size) entries of a
 *                row are read.  An entry outside [0, num_blocks) is not dereferenced:
 *                its keys are read as zeros and MLA_STATUS_BAD_PAGE is set.
 *   seq_lens     int32 [B], this shard's token count of each request.  A value above
 *                max_blocks*block_size is clamped and MLA_STATUS_SEQ_TOO_LONG is set.
 *   causal_seqlens_global  int32 [B] global lengths; may be NULL when cp_world == 1 (then
 *                seq_lens is used) or causal == 0 (then it is not read).
 *   B >= 0, 1 <= H, 1 <= q_len <= MLA_MAX_Q_LEN, ceil(q_len*H/128) <= SMs/2,
 *   num_blocks >= 1, 1 <= max_blocks <= bt_stride, 1 <= cp_world, 0 <= cp_rank <
 *   cp_world, interleave >= 1 dividing block_size (the pool layout cp_local_slot gives),
 *   finite scale > 0.
 *   out          bf16 [B*q_len, H, 512], 16-byte aligned.
 *   lse          float [B*q_len, H] or NULL.
 *   workspace    device scratch of workspace_bytes (may be NULL / 0), 256-byte aligned.
 * Errors: MLA_ERR_INVALID_ARGUMENT for any violated condition above (nothing launched),
 *   MLA_ERR_UNSUPPORTED for a block size or row count the kernel does not take,
 *   MLA_ERR_CUDA if a launch fails.
 */
int mla_decode(const void* q, const void* kv_cache, const int32_t* block_table,
               int64_t bt_stride, const int32_t* seq_lens,
               const int32_t* causal_seqlens_global, int B, int H, int q_len, int causal,
               int block_size, int num_blocks, int max_blocks, int cp_world, int cp_rank,
               int interleave, float scale, void* out, float* lse, int lse_base_e,
               void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * mla_decode_shards -- every shard of one emulated context-parallel decode step in a
 * single launch (the ranks of the pages' native DCP decode, [#54012] "关键源码片段",
 * run side by side on one GPU instead of one per GPU).  The result is exactly that of
 *     for r in 0 .. n_shards-1:
 *         mla_decode(q, kv_cache, block_table + r*B*bt_stride, bt_stride, seq_lens + r*B,
 *                    causal_seqlens_global, B, H, q_len, causal, block_size, num_blocks,
 *                    max_blocks, n_shards, r, interleave, scale,
 *                    out + r*B*q_len*H*512, lse ? lse + r*B*q_len*H : NULL, lse_base_e, ...)
 * with all shards' pages in one cache.
 *
 * Arguments (as mla_decode unless stated):
 *   kv_cache     bf16 [num_blocks, block_size, 576]: the pages of every shard.
 *   block_table  int32 [n_shards*B, bt_stride], shard-major: row r*B + b holds shard r's
 *                page ids (into kv_cache) for request b.
 *   seq_lens     int32 [n_shards*B], shard-major token counts.
 *   causal_seqlens_global  int32 [B]; may be NULL only if n_shards == 1 or causal == 0.
 *   n_shards     >= 1; shard r is rank r of cp_world = n_shards.
 *   out          bf16 [n_shards, B*q_len, H, 512];  lse  float [n_shards, B*q_len, H] or NULL.
 *   workspace    sized by mla_decode_workspace_size(n_shards*B, H, q_len, num_sms).
 * Errors: as mla_decode; also MLA_ERR_INVALID_ARGUMENT for n_shards < 1 and
 *   MLA_ERR_UNSUPPORTED when n_shards > 1 and n_shards * B * B >= 2^32.
 */
int mla_decode_shards(const void* q, const void* kv_cache, const int32_t* block_table,
                      int64_t bt_stride, const int32_t* seq_lens,
                      const int32_t* causal_seqlens_global, int B, int H, int q_len,
                      int causal, int block_size, int num_blocks, int max_blocks, int n_shards,
                      int interleave, float scale, void* out, float* lse, int lse_base_e,
                      void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * lse_merge -- combine n_shards partial results of the same rows through their LSEs.
 *
 * Defines ([#54012] "实现拆解" step 3: shards are merged across ranks and must agree on
 * the LSE base; [#48180] "实现拆解" step 2: merge when DCP is on): per row (t, h),
 *   M = max_s lses[s,t,h],  w_s = base^(lses[s,t,h] - M),
 *   out[t,h,:] = sum_s w_s partials[s,t,h,:] / sum_s w_s,
 *   out_lse[t,h] = M + log_base(sum_s w_s),
 * base e when lse_base_e != 0, else 2.  A shard with lse = -inf has weight 0 and its
 * partial is not read; if every shard has -inf, out = 0 and out_lse = -inf.  A NaN among the
 * row's LSEs makes both NaN.
 *
 * Arguments:
 *   partials        [n_shards, T, H, 512], bf16 when partials_fp32 == 0 else float,
 *                   16-byte aligned.
 *   lses            float [n_shards, T, H].
 *   n_shards >= 1, T >= 0, H >= 1.
 *   out             bf16 [T, H, 512], 16-byte aligned.
 *   out_lse         float [T, H] or NULL.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_CUDA.
 */
int lse_merge(const void* partials, int partials_fp32, const float* lses, int n_shards,
              int T, int H, void* out, float* out_lse, int lse_base_e,
              mla_stream_t stream);

/*
 * cp_local_slot -- this rank's KV slot of each position, MLA_PAD_SLOT_ID otherwise.
 *
 * Defines ([#52188] "关键源码片段", cp_utils.py cp_local_slot; "实现拆解" step 4): a
 * virtual block spans block_size*cp_size global positions and block_table[b, pos /
 * (block_size*cp_size)] names its page on every rank; with o = pos % (block_size*cp_size),
 * position pos is owned by rank (o / interleave) % cp_size, at local offset
 * (o / (interleave*cp_size)) * interleave + o % interleave, so
 *     slots[b,n] = page * block_size + local offset   if this rank owns it,
 *     slots[b,n] = MLA_PAD_SLOT_ID                     otherwise, or when pos < 0
 * (a negative position marks a rejected draft position).  cp_size == 1 gives
 * page * block_size + pos % block_size.
 *
 * Arguments:
 *   positions    int64 [B, N];  block_table int32 [B, bt_stride] with max_blocks valid
 *                columns;  slots int64 [B, N].
 *   B >= 0, N >= 0, block_size >= 1, cp_size >= 1, 0 <= cp_rank < cp_size,
 *   interleave >= 1 with block_size % interleave == 0, 1 <= max_blocks <= bt_stride.
 * A position whose virtual block is >= max_blocks gets MLA_PAD_SLOT_ID and sets
 * MLA_STATUS_BAD_VBLOCK; its table entry is not read.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_CUDA.
 */
int cp_local_slot(const int64_t* positions, const int32_t* block_table, int64_t bt_stride,
                  int max_blocks, int B, int N, int block_size, int cp_size, int cp_rank,
                  int interleave, int64_t* slots, mla_stream_t stream);

/*
 * cp_local_slot_scatter -- writes new KV rows into this rank's pool at the slots
 * cp_local_slot gives them.
 *
 * Defines ([#52188] "实现拆解" step 4: the draft inputs apply cp_local_slot to the slots
 * they write, with the page of a position taken from block_table[pos / (block_size *
 * cp_size)], so that a rank never writes a slot another rank is responsible for): for
 * every (b, n) with s = cp_local_slot(positions[b, n]) != MLA_PAD_SLOT_ID,
 *     kv_cache[s] = kv_new[b, n]          (576 bf16, copied bit for bit);
 * positions this rank does not own, and negative (rejected) positions, write nothing and
 * their rows are not read.
 *
 * Arguments (as cp_local_slot unless stated):
 *   kv_new       bf16 [B, N, 576], 16-byte aligned.
 *   kv_cache     bf16 [num_blocks, block_size, 576] (this rank's pool), 16-byte aligned.
 *   slots        int64 [B, N] or NULL: receives the slots, as cp_local_slot returns them.
 * A slot outside the cache (a table entry outside [0, num_blocks)) is not written and
 * sets MLA_STATUS_BAD_PAGE; a virtual block past the table sets MLA_STATUS_BAD_VBLOCK.
 * Two positions mapping to the same slot race (the pages' slot mapping never does that
 * for distinct positions of one request).
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED (B*N or block_size*cp_size beyond
 *   2^31-1), MLA_ERR_CUDA.
 */
int cp_local_slot_scatter(const int64_t* positions, const void* kv_new,
                          const int32_t* block_table, int64_t bt_stride, int max_blocks, int B,
                          int N, int block_size, int cp_size, int cp_rank, int interleave,
                          void* kv_cache, int num_blocks, int64_t* slots, mla_stream_t stream);

/*
 * cp_step_tables -- the tables of one serving step, built on the GPU from request lengths:
 * pages taken and given back, global and shard-local lengths, the new tokens' positions and
 * their slots.  Everything cp_store_q8, cp_local_slot_scatter and the decode calls read
 * comes from it, so that a step needs no host round trip and can be captured in a graph.
 *
 * With vbs = block_size * cp_size (a virtual block, see cp_local_slot) and
 * pages(x) = ceil(x / vbs), request b holds pages(prev_lens[b]) pages, has ctx_lens[b]
 * tokens in the cache (fewer than prev_lens[b] after a rejected draft, 0 when it has
 * finished) and brings new_lens[b] new tokens:
 *   take_b  = max(0, pages(ctx + new) - pages(prev));  request b is granted when
 *             pages(ctx + new) <= max_blocks and take_b is 0 or take_0 + .. + take_b is at
 *             most the number of free pages (requests that do not fit the table take none);
 *   total_b = ctx + new if granted, else min(ctx, prev) (then it has no new token);
 *   give_b  = max(0, pages(prev) - pages(total)).
 * free_pages is a ring of free_cap entries; free_state = {head, count}.  Granted requests
 * take their pages from the head in the order of b, the page of virtual block j going to
 * block_table[b, j]; pages given back (virtual blocks pages(total) .. pages(prev) - 1, in
 * the order of b) join the end, and can be taken from the next call on.  Other table entries
 * are left as they were.  free_state_out = {(head + taken) % free_cap, count - taken + given}.
 *   total_lens[b]      = total_b  (causal_seqlens_global of the decode calls);
 *   seq_lens[r, b]     = local_len(total_b) on rank cp_rank + r (see mla_decode);
 *   positions[b, n]    = ctx_lens[b] + n for n < new_lens[b] of a granted request, else -1;
 *   slots[r, b, n]     = the slot cp_local_slot gives that position on rank cp_rank + r.
 * A call reads and writes disjoint entries, so repeating it with the same inputs gives the
 * same result.
 *
 * Arguments:
 *   prev_lens, ctx_lens, new_lens  int32 [B], values in [0, 2^31) with new_lens[b] <= N.
 *   block_table  int32 [B, bt_stride], max_blocks columns in use; updated.
 *   free_pages   int32 [free_cap], free_cap at least the number of pages of the pool; updated.
 *   free_state   int32 [2];  free_state_out  int32 [2].
 *   total_lens   int32 [B].
 *   seq_lens     int32 [n_ranks, B] or NULL;  positions  int64 [B, N] or NULL;
 *   slots        int64 [n_ranks, B, N] or NULL.
 *   B >= 0, N >= 0, n_ranks >= 1, 0 <= cp_rank, cp_rank + n_ranks <= cp_size, free_cap >= 1;
 *   block_size, cp_size, interleave, max_blocks, bt_stride as for cp_local_slot.
 *   The outputs may not overlap the inputs (total_lens and prev_lens are two buffers that a
 *   caller swaps; so are free_state and free_state_out).
 * Bad data is flagged and bounded: a request that does not fit the table sets
 * MLA_STATUS_SEQ_TOO_LONG, one that finds too few free pages MLA_STATUS_OUT_OF_PAGES (both
 * are not granted); a negative length is read as 0, a new_lens above N as N, prev_lens beyond
 * the table as the whole table, a ring state outside the ring as an empty ring, and pages
 * given back to a full ring are dropped, each with MLA_STATUS_BAD_STEP.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED (n_ranks*B*N or block_size*cp_size
 *   beyond 2^31-1), MLA_ERR_CUDA.
 */
int cp_step_tables(const int32_t* prev_lens, const int32_t* ctx_lens, const int32_t* new_lens,
                   int B, int N, int32_t* block_table, int64_t bt_stride, int max_blocks,
                   int32_t* free_pages, int free_cap, const int32_t* free_state,
                   int32_t* free_state_out, int block_size, int cp_size, int cp_rank,
                   int n_ranks, int interleave, int32_t* total_lens, int32_t* seq_lens,
                   int64_t* positions, int64_t* slots, mla_stream_t stream);

/*
 * cp_store_q8 -- writes a step's new KV rows into this rank's 8-bit pool.
 *
 * New token n of request b (0 <= n < total_lens[b] - ctx_lens[b], at most N) has position
 * ctx_lens[b] + n; the rank stores those cp_local_slot gives it a slot for.  The slots of a
 * page are grouped by MLA_Q8_GROUP consecutive ones, which share one scale s; a row x is
 * stored as e4m3(x / s), rounded to nearest even, and stands for s times that.  For each
 * group that gets a new row, with a = the largest finite |x| of its new rows:
 *   s = the smallest power of two with a <= 448 s, within [MLA_Q8_SCALE_MIN,
 *       MLA_Q8_SCALE_MAX] (larger values are stored as +-448);
 *   where the group begins with earlier rows of the request (the first new row is not its
 *   first), s is at least the scale s_old that is there; if s grows, the earlier rows are
 *   stored again as e4m3(v * (s_old / s)).
 * Slots of the group behind the new rows are left as they were (whatever they held before
 * they are no longer scaled by the scale they were stored with).  NaN and infinities are
 * stored as NaN and take no part in a.
 *
 * Arguments (as cp_local_slot unless stated):
 *   kv_new       bf16 [B, N, 576], 16-byte aligned.
 *   ctx_lens, total_lens  int32 [B], as cp_step_tables takes and gives them.
 *   kv_cache     e4m3 [num_blocks, block_size, 576] (this rank's pool), 16-byte aligned.
 *   kv_scales    float [num_blocks, block_size / 16].
 *   block_size   a multiple of 16.
 * Two requests with new rows in one page race (pages that requests share hold whole blocks
 * of common tokens, which no one writes).  A table entry outside [0, num_blocks) writes
 * nothing and sets MLA_STATUS_BAD_PAGE, a virtual block past the table MLA_STATUS_BAD_VBLOCK;
 * an earlier scale outside its range is taken as 1 with MLA_STATUS_BAD_SCALE; a negative
 * ctx_lens (the request is skipped) or more than N new tokens (N are stored) sets
 * MLA_STATUS_BAD_STEP.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED (B*N or block_size*cp_size beyond
 *   2^31-1), MLA_ERR_CUDA.
 */
int cp_store_q8(const void* kv_new, const int32_t* ctx_lens, const int32_t* total_lens,
                const int32_t* block_table, int64_t bt_stride, int max_blocks, int B, int N,
                int block_size, int cp_size, int cp_rank, int interleave, void* kv_cache,
                float* kv_scales, int num_blocks, mla_stream_t stream);

/*
 * mla_decode_q8, mla_decode_shards_q8 -- mla_decode and mla_decode_shards over the 8-bit
 * cache that cp_store_q8 writes: key l of the definition there is the row's 576 e4m3 values
 * times the scale of its group, and everything else is the same (row bounds, empty rows,
 * LSE bases, the outputs' layouts).
 *
 * Arguments (as mla_decode / mla_decode_shards unless stated):
 *   kv_cache     e4m3 [num_blocks, block_size, 576], 16-byte aligned;
 *   kv_scales    float [num_blocks, block_size / 16]; any finite scale within
 *                [MLA_Q8_SCALE_MIN, MLA_Q8_SCALE_MAX], powers of two or not.  A scale outside
 *                that range of a group with a visible key is taken as 1 and sets
 *                MLA_STATUS_BAD_SCALE; scales of other groups are not used.
 *   block_size   a multiple of 16.
 *   q            a row (one head of one token) with a NaN or an infinity gives NaN outputs.
 *   scale        scale * s * |q| must stay below 2^127 for every scale s and element of q in
 *                use (scores beyond float's range give NaN, 0 or -inf as floats do).
 *   Limits (else MLA_ERR_UNSUPPORTED, and mla_last_error() names the one that was passed), with R the
 *   requests of all shards: ceil(q_len*H/64) <= SMs; num_blocks*block_size and
 *   max_blocks*block_size below 2^31 - 65536; R * (max_blocks*block_size/128 + 7) below 2^31 (a
 *   table of 131,072 slots: 2,080,000 requests); R * ceil(q_len*H/64) below 2^28.
 *   workspace    scratch for split-KV, sized by mla_decode_q8_workspace_size (for the shards
 *                call with n_shards*B), or NULL / 0: without all of it no request is split.
 * Accuracy: products and sums are fp32; q is used to within 2^-17 of its row's largest
 * magnitude (exactly, for elements within 2^-9 of it).  A softmax weight meets the values in
 * fewer bits than its sum (the LSE) is made of, where the bf16 cache's decode rounds it to bf16
 * (2^-8 of itself).  With p = weight times scale, P the row's largest p, and p' the largest of 16
 * neighbouring keys: p is used to within 2^-7 of itself (2^-8 in tiles of 128 keys where p' is at least
 * 2^-9 P throughout for all rows of a block and P does not grow) plus 2^-6 p', or 2^-22 P where p' is
 * smaller than 2^-9 P (2^-28 P where P's key stands alone among some 100 around it, 2^9 above the
 * rest).  The second term bounds a single key's: it is rounded up or down evenly over the keys, so
 * that sums over many keep it (n equal weights: 2^-7 of their sum and some times that term, not n
 * times).
 * Errors: as mla_decode / mla_decode_shards.
 */
size_t mla_decode_q8_workspace_size(int B, int H, int q_len, int num_sms);

int mla_decode_q8(const void* q, const void* kv_cache, const float* kv_scales,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* seq_lens,
                  const int32_t* causal_seqlens_global, int B, int H, int q_len, int causal,
                  int block_size, int num_blocks, int max_blocks, int cp_world, int cp_rank,
                  int interleave, float scale, void* out, float* lse, int lse_base_e,
                  void* workspace, size_t workspace_bytes, mla_stream_t stream);

int mla_decode_shards_q8(const void* q, const void* kv_cache, const float* kv_scales,
                         const int32_t* block_table, int64_t bt_stride,
                         const int32_t* seq_lens, const int32_t* causal_seqlens_global, int B,
                         int H, int q_len, int causal, int block_size, int num_blocks,
                         int max_blocks, int n_shards, int interleave, float scale, void* out,
                         float* lse, int lse_base_e, void* workspace, size_t workspace_bytes,
                         mla_stream_t stream);

/*
 * mla_rope -- rotary positions: turns the 32 pairs of each rope part (64 dims) of
 * x [T, H, 64] by the token's position p = positions[t]:
 *     a_i = 2 pi frac(p * freqs[i] * 2^-64),
 *     y0 = mscale (x0 cos a_i - x1 sin a_i),  y1 = mscale (x0 sin a_i + x1 cos a_i),
 * with the pairs (2i, 2i+1) (half == 0) or (i, i+32) (half != 0), rounded to bf16 once.  Tokens
 * at negative positions (rejected or padded ones) are left as they were in out.
 *
 * Arguments:
 *   x            bf16, 64 contiguous dims at x + t*x_stride_t + h*x_stride_h (elements): the last
 *                dims of queries of any width; 16-byte aligned, strides multiples of 8.
 *   positions    int64 [T];  freqs  int64 [32], turns a position in units of 2^-64.
 *   out          as x, with its own strides (so that absorbed queries, 576 wide, take their rope
 *                part where it belongs); may be x itself, may not overlap it otherwise.
 *   T >= 0, H >= 1, finite mscale.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_CUDA.
 */
int mla_rope(const void* x, int64_t x_stride_t, int64_t x_stride_h, const int64_t* positions,
             const int64_t* freqs, int T, int H, int half, float mscale, void* out,
             int64_t out_stride_t, int64_t out_stride_h, mla_stream_t stream);

/*
 * cp_rope_store -- writes new tokens into this rank's pool at the slots cp_local_slot gives them,
 * the rope part of their keys rotated on the way:
 *     kv_cache[s] = [ latent[b, n] (512, bit for bit) | rotated k_rope[b, n] (64, see mla_rope) ];
 * positions this rank does not own, and negative ones, write nothing and are not read.
 *
 * Arguments (as cp_local_slot_scatter and mla_rope unless stated):
 *   latent       bf16, row b*N + n (512 contiguous) at latent + (b*N + n)*latent_stride;
 *   k_rope       bf16, row b*N + n (64 contiguous) at k_rope + (b*N + n)*k_rope_stride: both may
 *                be parts of one tensor; 16-byte aligned, strides multiples of 8 elements.
 * A table entry outside [0, num_blocks) writes nothing and sets MLA_STATUS_BAD_PAGE.  The positions of
 * a request, and the pages of different ones that get rows, are distinct: of two tokens for one slot
 * the row may hold parts of either.
 * Errors: as cp_local_slot_scatter.
 */
int cp_rope_store(const void* latent, int64_t latent_stride, const void* k_rope,
                  int64_t k_rope_stride, const int64_t* positions, const int64_t* freqs,
                  const int32_t* block_table, int64_t bt_stride, int max_blocks, int B, int N,
                  int block_size, int cp_size, int cp_rank, int interleave, int half, float mscale,
                  void* kv_cache, int num_blocks, int64_t* slots, mla_stream_t stream);

/*
 * mla_expand -- keys and values of all heads (the expanded form of latent attention) from the
 * paged cache.  Local key l of request b, with cache row c, becomes row r = kv_starts[b] + l of
 *     kv[h, r, 0:128]   = w_kv[h, 0:128] c[0:512]     (the key's part without position),
 *     kv[h, r, 128:256] = w_kv[h, 128:256] c[0:512]   (the value),
 *     k_rope[r]         = c[512:576],
 * products summed in fp32 and rounded to bf16 once.  Rows of no request are left as they were.
 *
 * Arguments:
 *   kv_cache     bf16 [num_blocks, block_size, 576], or, with kv_scales (not NULL), the 8-bit cache
 *                (see mla_decode_q8; c is exact in the products whatever the scales, and k_rope is rounded
 *                once); 16-byte aligned; any block_size >= 1 (8-bit: multiples of 16).
 *   block_table, seq_lens  as mla_decode (shard-local lengths).
 *   kv_starts    int32 [B]: the requests' first rows, in order and apart
 *                (kv_starts[b] + seq_lens[b] <= kv_starts[b+1]).
 *   w_kv         bf16 [H, 256, 512], 16-byte aligned.
 *   kv           bf16 [H, S, 256];  k_rope  bf16 [S, 64]; 16-byte aligned.  Rows from S on are not
 *                written.
 *   B >= 0, S >= 0, H >= 1, (S/256 + 1) * 2 H below 2^31 - 512, 1 <= max_blocks <= bt_stride, num_blocks >= 1.
 * A page outside [0, num_blocks) reads as zeros with MLA_STATUS_BAD_PAGE, a length beyond the table
 * is cut with MLA_STATUS_SEQ_TOO_LONG, a scale out of range is taken as 1 with
 * MLA_STATUS_BAD_SCALE.  kv_starts out of order leave rows unwritten or give them to another request.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED (max_blocks*block_size beyond 2^31-1, or
 *   too many tiles), MLA_ERR_CUDA.
 */
int mla_expand(const void* kv_cache, const float* kv_scales, const int32_t* block_table,
               int64_t bt_stride, const int32_t* seq_lens, const int32_t* kv_starts, int B,
               int block_size, int num_blocks, int max_blocks, const void* w_kv, int H, int S,
               void* kv, void* k_rope, mla_stream_t stream);

/*
 * mla_prefill -- attention of chunks of new tokens, of any and different lengths, over expanded
 * keys and values (those mla_expand gives, or others of these shapes).
 *
 * Request b brings the query rows cu_q_lens[b] .. cu_q_lens[b+1] - 1, n of them, and has
 * seq_lens[b] local keys, the rows from kv_starts[b] on.  Its row i sees the first L_i of them, as
 * in mla_decode with q_len = n: L_i = min(seq_lens[b], local_len(max(0, G_b - (n-1-i)))), G_b =
 * causal_seqlens_global[b], the new tokens included; all of them when causal == 0.  With
 *     s_l = scale * (<q[0:128], k_nope_l> + <q[128:192], k_rope_l>),
 *     out = sum_l softmax(s)_l v_l,   lse = log(sum_l exp(s_l))   (natural, or log2),
 * a row with L_i = 0 gets out = 0 and lse = -inf.  Rows of no request are left as they were.
 * The results of a shard's keys are partial ones, which lse_merge_v joins.
 *
 * Arguments:
 *   q            bf16, 192 contiguous dims (128 without position, 64 rotated) at
 *                q + t*q_stride_t + h*q_stride_h (elements), T rows.
 *   k_nope, v    bf16, 128 contiguous dims at + s*stride_s + h*stride_h, S rows;
 *   k_rope       bf16, 64 contiguous dims at + s*k_rope_stride, S rows, shared by the heads.
 *                All 16-byte aligned, strides multiples of 8 elements and positive.
 *   cu_q_lens    int32 [B+1];  kv_starts, seq_lens  int32 [B].
 *   causal_seqlens_global  int32 [B]; may be NULL when cp_world == 1 (then seq_lens is used) or
 *                causal == 0 (then it is not read).
 *   out          bf16 [T, H, 128], 16-byte aligned;  lse  float [T, H] or NULL.
 *   workspace    scratch of mla_prefill_workspace_size bytes, 256-byte aligned, or NULL / 0: without
 *                all of it the keys of few rows are not split over the SMs.
 *   T, B, S >= 0 (k_nope, v and k_rope may be NULL for S = 0), H >= 1, (T/256 + min(B, T)) * H below 2^31; cp_world,
 *   cp_rank, interleave, scale as mla_decode (interleave need not divide anything here).
 * Keys and values that a row does not see, and rows behind the last key, may hold anything (where
 * they are NaN or infinite, rows of the same 256 that do not see them are computed again, slowly:
 * 32 of them over 130,000 keys take 0.6 s.  The wait limit does not count that time).
 * A request whose cu_q_lens are out of order (before the largest so far) or beyond T is skipped, and
 * kv_starts or seq_lens beyond S are cut; both set MLA_STATUS_BAD_STEP.
 * Accuracy: scores and sums in fp32; a softmax weight is rounded to bf16 where it meets the values.
 * Errors: MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA.
 */
size_t mla_prefill_workspace_size(int T, int B, int H, int S, int num_sms);

int mla_prefill(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_nope,
                int64_t k_stride_s, int64_t k_stride_h, const void* k_rope, int64_t k_rope_stride,
                const void* v, int64_t v_stride_s, int64_t v_stride_h, const int32_t* cu_q_lens,
                const int32_t* kv_starts, const int32_t* seq_lens,
                const int32_t* causal_seqlens_global, int T, int B, int H, int S, int causal,
                int cp_world, int cp_rank, int interleave, float scale, void* out, float* lse,
                int lse_base_e, void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * lse_merge_v -- lse_merge for partials [n_shards, T, H, dv] and out [T, H, dv], dv 512 or 128 (the
 * outputs of mla_prefill).  Errors: as lse_merge, and MLA_ERR_UNSUPPORTED for another dv.
 */
int lse_merge_v(const void* partials, int partials_fp32, const float* lses, int n_shards, int T,
                int H, int dv, void* out, float* out_lse, int lse_base_e, mla_stream_t stream);

/*
 * mla_decode_noalloc -- mla_decode for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this call.  It computes exactly what mla_decode
 * computes, with the same arguments minus the workspace: some callers cannot call
 * cudaMalloc or any allocating routine on their decode path (a runtime whose memory is
 * planned once at start-up, a host program that links only this C library and owns no
 * allocator), yet split-KV needs scratch for its per-split partial results.  This call
 * takes that scratch from one fixed 64 MiB array that the library declares in device
 * memory; every GPU that loads the library holds the array until the process exits.
 *   - A problem whose split-KV scratch exceeds 64 MiB is rejected with
 *     MLA_ERR_UNSUPPORTED (message in mla_last_error) and nothing is launched; every
 *     other argument is checked first, exactly as mla_decode checks it.
 *   - All calls on a device share the array and it keeps the last call's contents;
 *     calls whose kernels overlap on the GPU (other streams or host threads) race on it
 *     and must be serialised.  Nothing in it needs to start at zero.
 *   - The first call on a device looks up the array's device address (once per device,
 *     with that device current); make that first call before any stream capture.
 *   - It calls no cudaMalloc, cudaFree or allocating library routine.
 * Errors: as mla_decode, plus MLA_ERR_UNSUPPORTED for the size limit.
 */
int mla_decode_noalloc(const void* q, const void* kv_cache, const int32_t* block_table,
                       int64_t bt_stride, const int32_t* seq_lens,
                       const int32_t* causal_seqlens_global, int B, int H, int q_len,
                       int causal, int block_size, int num_blocks, int max_blocks,
                       int cp_world, int cp_rank, int interleave, float scale, void* out,
                       float* lse, int lse_base_e, mla_stream_t stream);

/*
 * Waits for `stream`, then reads and clears the current device's status word.
 * Returns MLA_OK when no kernel flagged anything since the last call, MLA_ERR_DEVICE
 * when one did (mla_last_error() names the bits; *bits_out receives them if non-NULL),
 * MLA_ERR_CUDA if the read itself failed.
 */
int mla_get_device_status(mla_stream_t stream, uint32_t* bits_out);

/*
 * Selects the decode kernel for later mla_decode calls in this process (diagnostics and
 * tests): 0 = automatic (the tcgen05/TMEM/TMA kernel; a layout it does not take is
 * refused with MLA_ERR_UNSUPPORTED), 1 = the warp-level mma.sync kernel (any block size;
 * a second, independent implementation that tests compare with the first), 2 = the
 * tcgen05 kernel.  Returns the previous choice, or MLA_ERR_INVALID_ARGUMENT for any other
 * value.  Not to be changed while other threads call mla_decode.
 */
int mla_set_decode_kernel(int choice);

/*
 * Selects the lazy-rescale budget of the tcgen05 kernel's online softmax for later calls
 * (diagnostics and tests): 0 = chosen per call (the wide budget when max_blocks *
 * block_size * cp_world >= 2^18, i.e. for long contexts), 1 = narrow, 2 = wide.  Both
 * compute the same result; they differ in how often the accumulator is rescaled.
 * Returns the previous choice, or MLA_ERR_INVALID_ARGUMENT for any other value.
 */
int mla_set_rescale_budget(int choice);

/*
 * Sets the time limit of every bounded on-chip wait of later launches, in nanoseconds
 * (0 = the default, 2 s); returns the previous setting (0 = default), or
 * MLA_ERR_INVALID_ARGUMENT for ns < 0.  A wait that runs out makes the kernel stop every
 * role of its thread-block pair, let the copies in flight land, release its tensor
 * memory and return; mla_get_device_status then reports MLA_STATUS_WAIT_TIMEOUT and the
 * outputs of that call are undefined.  Tests use a tiny limit to exercise that path.
 */
int64_t mla_set_wait_limit_ns(int64_t ns);

/*
 * Tests of the timeout path only: with on = 1, later launches of the tcgen05 decode kernel
 * make one role of every thread-block pair first wait for an mbarrier arrival that never
 * comes, so that the wait runs out after the limit of mla_set_wait_limit_ns, the kernel
 * stops and returns (outputs undefined) and mla_get_device_status reports
 * MLA_STATUS_WAIT_TIMEOUT.  on = 0 (the default) turns it off.  Returns the previous
 * setting, or MLA_ERR_INVALID_ARGUMENT.
 */
int mla_set_test_stall(int on);

/* Message of the calling thread's last failed call (empty string if none). */
const char* mla_last_error(void);

/* ABI version of this library: (major << 16) | minor (2.2). */
int mla_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DECODE_H_ */
