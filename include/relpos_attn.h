/*
 * relpos_attn.h -- C ABI of the GB300 (sm_103a) relative-position attention
 * library (librelpos_attn.so): the forward pass (also over right-padded
 * batches), the T5 cached decode and the T5, Shaw, DeBERTa and ALiBi
 * backward passes (relpos_t5_attn_bwd, relpos_shaw_attn_bwd,
 * relpos_deberta_attn_bwd, relpos_alibi_attn_bwd), and what serving from a
 * paged key/value cache takes: rotary positions (relpos_rotary), appending to
 * the cache (relpos_paged_append) and decoding over it (relpos_paged_decode),
 * at the end of this header.
 *
 * One forward call computes multi-head attention whose logits carry a relative-
 * position term that is formed inside the kernel and never written to
 * device memory as an L x L (or L x L x d) tensor:
 *
 *   RELPOS_T5      per-head scalar bias looked up by bucket of the offset
 *                  key - query ("Relative Position Embeddings, in depth",
 *                  section "T5: one scalar per head, looked up by bucket";
 *                  "T5 Relative-Position Bias", bucket definition and the
 *                  cached-decoder example).
 *                  logit = q.k / sqrt(d) + bias[bucket(j - p)][h]
 *   RELPOS_SHAW    clipped relative key and value vectors ("Relative
 *                  Position Embeddings, in depth", section "Shaw et al.").
 *                  logit = q.(k_j + a_K[clip(j - p, -k, k) + k]) / sqrt(d)
 *                  out   = sum_j softmax_j * (v_j + a_V[clip(j - p, -k, k) + k])
 *   RELPOS_DEBERTA disentangled content/position attention ("Relative
 *                  Position Embeddings, in depth", section "DeBERTa:
 *                  disentangled content and position"; "DeBERTa > Relative
 *                  Position Encoding", section "The Relative Position
 *                  Formula" for delta).
 *                  logit = (q_i.k_j + q_i.Pk[delta(p, j)] + k_j.Pq[delta(j, p)])
 *                          / sqrt(3d),  delta(a, b) = clip(a - b, -k, k - 1) + k
 *   RELPOS_ALIBI   a fixed slope per head times the distance, no table and
 *                  no maximum distance ("Relative Position Embeddings, in
 *                  depth", section "ALiBi and RoPE: the two endpoints").
 *                  logit = q.k / sqrt(d) - slope[h] * |j - p|
 *   RELPOS_TXL     Transformer-XL: content and position keys with their own
 *                  projections and two global biases u, v ("Relative
 *                  Position Embeddings, in depth", section "Transformer-XL:
 *                  four terms and two global biases").
 *                  logit = ((q + u[h]).k_j + (q + v[h]).W[h] R(p - j)) / sqrt(d)
 *                  with R(t) the fixed sinusoidal encoding of the offset
 *                  t = query - key position: R[2m] = sin(w_m t),
 *                  R[2m+1] = cos(w_m t), w_m = 10000^(-2m/d).
 *
 * Positions: query row i sits at absolute position p = i + q_offset; key
 * row j at position j. With causal = 1 keys j > p are masked out (and T5
 * uses its causal bucket mapping). A query row with no visible key gets a
 * zero output row.
 *
 * Conventions shared by every entry point:
 *  - Pointers marked "device" are CUDA device pointers owned by the caller;
 *    the library keeps no reference to them after the call returns.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). Calls are
 *    asynchronous on that stream unless stated otherwise.
 *  - Return value: RELPOS_OK (0) or a negative RELPOS_ERR_* code; argument
 *    errors are reported before anything is launched. relpos_strerror()
 *    names a code. No entry point falls back to a CPU path.
 */
#ifndef RELPOS_ATTN_H_
#define RELPOS_ATTN_H_

#ifdef __cplusplus
extern "C" {
#endif

/* modes */
#define RELPOS_T5 0
#define RELPOS_SHAW 1
#define RELPOS_DEBERTA 2
#define RELPOS_ALIBI 3
#define RELPOS_TXL 4

/* element types of Q, K, V and out; of a paged cache: BF16 or E4M3 */
#define RELPOS_BF16 0
#define RELPOS_FP32 1
#define RELPOS_E4M3 2

/* return codes */
#define RELPOS_OK 0
#define RELPOS_ERR_INVALID_ARG (-1)    /* null pointer, bad size or parameter */
#define RELPOS_ERR_UNSUPPORTED (-2)    /* valid request this build does not run (d = 128 Shaw, ...) */
#define RELPOS_ERR_CUDA (-3)           /* a CUDA runtime call or launch failed */
#define RELPOS_ERR_DEVICE_TIMEOUT (-4) /* a kernel gave up on a bounded wait */
#define RELPOS_ERR_SCRATCH_LIMIT (-5)  /* request needs more than the fixed scratch of
                                          relpos_t5_decode_noalloc */
#define RELPOS_ERR_PAGE (-6)           /* a kernel met a length, a row range or a page number
                                          outside the paged cache and skipped it */

/*
 * relpos_attn_fwd -- attention forward with an in-kernel relative term.
 *
 *   mode        RELPOS_T5, RELPOS_SHAW, RELPOS_DEBERTA, RELPOS_ALIBI or RELPOS_TXL.
 *   dtype       RELPOS_BF16 or RELPOS_FP32: element type of Q, K, V and out.
 *               FP32 inputs are rounded to bf16 on the device before the
 *               tensor-core products (fp32 accumulation); out is fp32.
 *   Q           device, [B, H, Lq, d] row-major.
 *   K, V        device, [B, H, Lk, d] row-major.
 *   table0/1    device tables, row-major:
 *                 T5:      table0 = bias [num_buckets, H] fp32; table1 unused.
 *                 Shaw:    table0 = a_K, table1 = a_V, each [2k+1, d] bf16,
 *                          shared by all heads.
 *                 DeBERTa: table0 = Pk, table1 = Pq, each [2k, H, d] bf16
 *                          (already projected per head).
 *                 ALiBi:   table0 = slopes [H] fp32 (any values the caller
 *                          chooses); table1 unused.
 *                 TXL:     table0 = W [H, d, d] fp32, the key projection of
 *                          the sinusoid per head, output index first
 *                          (r[e] = sum_f W[h][e][f] R[f]); table1 = [2, H, d]
 *                          fp32, u then v. Memory (cached keys of the
 *                          previous segment) is ordinary keys at positions
 *                          0 .. mem - 1 with q_offset = mem.
 *   B, H        batch and heads (>= 0; 0 makes the call a no-op).
 *   Lq, Lk      query and key lengths (Lq >= 0, Lk >= 0). Lk == 0 writes
 *               zeros.
 *   d           head dimension: 64 for every mode; also 128 for T5 and
 *               ALiBi with dtype BF16 (other modes and FP32 inputs at
 *               d = 128 return RELPOS_ERR_UNSUPPORTED). At d = 128 a few
 *               query rows take the prefill kernel, not the split-key
 *               decode path, and T5 keeps a single table copy when its
 *               four shifted copies do not fit beside the larger tiles.
 *   num_buckets T5 only: even, 4 <= num_buckets <= 128 (ignored otherwise).
 *   rel_param   T5: max_distance (> num_buckets/4 bidirectional, > num_buckets/2
 *               causal); Shaw: clip k (1 <= k <= 64); DeBERTa: k (1 <= k <= 4096);
 *               ALiBi, TXL: ignored.
 *               Shaw's per-row tables and T5's bias-by-offset table live in
 *               shared memory: this build runs Shaw k <= 27, and T5 as long as
 *               the distance at which the last bucket starts (about
 *               max_distance, or the longest offset of the call if shorter)
 *               is at most about 2500 (beyond about 480 through a slower
 *               single-copy table); beyond, the call returns
 *               RELPOS_ERR_UNSUPPORTED.
 *   causal      0 or 1.
 *   q_offset    absolute position of query row 0 (>= 0), for cached decoding.
 *   out         device, [B, H, Lq, d], element type per dtype; written fully.
 *   stream      cudaStream_t.
 *
 * Scratch: calls with dtype FP32, with DeBERTa or TXL (the rows
 * [q + u | W^T (q + v) rotated by the query's angles], 256 bytes per query
 * row, and the keys' sinusoid table), or that take the split-key
 * decode path (few query rows) draw temporary device memory with
 * cudaMallocAsync on `stream` and release it with cudaFreeAsync before
 * returning. Nothing persists between calls.
 * Errors: RELPOS_ERR_INVALID_ARG / _UNSUPPORTED before launch;
 * RELPOS_ERR_CUDA if a launch or allocation fails. Device-side bounded-wait
 * failures are reported by relpos_check_status().
 */
int relpos_attn_fwd(int mode, int dtype, const void* Q, const void* K, const void* V,
                    const void* table0, const void* table1, int B, int H, int Lq, int Lk,
                    int d, int num_buckets, int rel_param, int causal, int q_offset,
                    void* out, void* stream);

/*
 * relpos_attn_fwd_padded -- relpos_attn_fwd over a right-padded batch of
 * sequences of different lengths. The pages do not treat padding; the
 * reading here: batch element b holds lengths[b] valid query rows and keys
 * (its first rows of Q, K and V), so its output equals that sequence
 * computed alone, and its rows from lengths[b] on are written as zeros.
 * Keys from lengths[b] on are masked for every row of element b; the rows and
 * keys in the padding may hold anything. Positions and q_offset are as for
 * relpos_attn_fwd (the relative offsets are the unpadded ones).
 *
 *   lengths     device, int32 [B], 4-byte aligned: read by the kernels, so
 *               the host does not check its values; a negative length counts
 *               as 0 (all rows zero), one beyond Lq / Lk as no padding.
 *   all other arguments as for relpos_attn_fwd. Calls with T5 and Lq <= 8
 *   run the fused kernel, not the split-key decode.
 * Errors: as relpos_attn_fwd; RELPOS_ERR_INVALID_ARG for a null or
 * misaligned lengths.
 */
int relpos_attn_fwd_padded(int mode, int dtype, const void* Q, const void* K, const void* V,
                           const void* table0, const void* table1, const int* lengths, int B,
                           int H, int Lq, int Lk, int d, int num_buckets, int rel_param, int causal,
                           int q_offset, void* out, void* stream);

/*
 * relpos_index_ids -- test hook: the device index generator the kernels use,
 * run over n consecutive offsets rel_first .. rel_first + n - 1.
 *
 *   T5:      offsets are key - query; ids are buckets ("T5: one scalar per
 *            head, looked up by bucket"); causal selects the causal mapping.
 *   Shaw:    offsets are key - query; ids are clip(rel, -k, k) + k.
 *   DeBERTa: offsets are query - key; ids are delta = clip(rel, -k, k-1) + k.
 *   ALiBi:   offsets are key - query; ids are the distances |rel|.
 *   TXL:     offsets are key - query; ids are t = query - key = -rel, the
 *            argument of the sinusoidal encoding R(t).
 *   out_dev  device int32[n], written asynchronously on `stream`.
 * Parameter checks are those of relpos_attn_fwd.
 */
int relpos_index_ids(int mode, int n, int rel_first, int num_buckets, int rel_param,
                     int causal, int* out_dev, void* stream);

/*
 * relpos_check_status -- synchronize `stream` and report whether any kernel
 * of this library hit a bounded-wait limit since the last check
 * (RELPOS_ERR_DEVICE_TIMEOUT) or met a page number or length outside its paged
 * cache (RELPOS_ERR_PAGE), whichever came first, or a CUDA error
 * (RELPOS_ERR_CUDA). Clears the recorded device status. Blocking.
 */
int relpos_check_status(void* stream);

/* relpos_strerror -- static description of a return code; never NULL. */
const char* relpos_strerror(int code);

/*
 * relpos_selftest_wait_timeout -- runs one tiny kernel that waits, with a
 * limit of `timeout_us` microseconds (1 .. 1000000), on a barrier that
 * nothing completes, exactly as the attention kernels' waits do. It records
 * RELPOS_ERR_DEVICE_TIMEOUT in the device status word and returns; the
 * context stays usable. Used to test the failure path without faulting or
 * hanging the GPU. Asynchronous; read the result with relpos_check_status().
 */
int relpos_selftest_wait_timeout(int timeout_us, void* stream);

/*
 * relpos_t5_decode_noalloc -- T5-bias cached decoding that allocates nothing.
 *
 * The pages have no counterpart to this call: it exists for callers that
 * cannot allocate device memory while they run -- code working inside a
 * memory budget planned ahead, or a serving loop that must keep the
 * allocator (cudaMallocAsync can synchronize or fail once the pool is
 * exhausted) off its hot path. It computes exactly what relpos_attn_fwd
 * computes for mode RELPOS_T5, dtype RELPOS_BF16 and Lq <= 8 (the split-key
 * decode path), but keeps the per-chunk partial results in one static
 * device array of 4 MiB built into the library, which every GPU that loads
 * the library holds until the process exits.
 *
 *   Q, K, V, bias, out, B, H, Lq, Lk, num_buckets, max_distance, causal,
 *   q_offset, stream: as for relpos_attn_fwd (bf16 Q/K/V/out, d = 64, fp32
 *   bias [num_buckets, H]); Lq must be <= 8 (RELPOS_ERR_UNSUPPORTED otherwise).
 * Limit: B * H * Lq * ceil(Lk / 256) * 264 bytes must fit in the 4 MiB array
 *   (for example B * H = 512 single-row queries over 4096 keys take 2.2 MiB);
 *   larger requests return RELPOS_ERR_SCRATCH_LIMIT before anything launches.
 * No cudaMalloc, cudaFree or allocating library routine is called. The first
 * call on each device looks up the array's device address (with that device
 * current); make that first call before any stream capture. Every call
 * shares the one array, so calls whose kernels overlap on the GPU (other
 * streams, other host threads) race and corrupt each other's results; order
 * them on one stream. Each call overwrites every partial it reads, so nothing
 * has to be cleared between calls. Asynchronous on `stream`.
 */
int relpos_t5_decode_noalloc(const void* Q, const void* K, const void* V, const void* bias, int B,
                             int H, int Lq, int Lk, int num_buckets, int max_distance, int causal,
                             int q_offset, void* out, void* stream);

/*
 * relpos_t5_decode_positions -- T5-bias cached decoding over keys at explicit
 * positions: a cache that evicted tokens keeps each remaining key at its
 * original position, and since the bias depends only on the offset nothing
 * stored needs rewriting ("Relative Position Embeddings, in depth", section
 * "Kernels and the KV cache").
 *
 *   key_pos     device, int32 [B, H, Lk]: the position of each key row, in
 *               any order, each in [0, 2^28]. The offset of key j to query
 *               row i is key_pos[b, h, j] - (i + q_offset); with causal = 1 a
 *               key whose position lies after the query's is masked out. A
 *               query row with no visible key gets a zero row.
 *   Q, K, V, bias, out, B, H, Lq, Lk, num_buckets, max_distance, causal,
 *   q_offset, stream: as for relpos_attn_fwd with mode RELPOS_T5 and dtype
 *   RELPOS_BF16 (d = 64), any Lq: up to 8 query rows run the split-key
 *   decode kernels, more rows (a chunk of new tokens against the cache) the
 *   fused prefill kernel, which then visits every key tile (a key's index
 *   says nothing about its position) and takes the bias per element from
 *   the positions on tiles that are neither wholly beyond the saturation
 *   distance nor free of masked keys.
 * Scratch: for Lq <= 8 the per-chunk partials (B * H * Lq * ceil(Lk / 256) *
 * 264 bytes) come from cudaMallocAsync on `stream` and go back with
 * cudaFreeAsync before the call returns; none otherwise. Asynchronous on
 * `stream`.
 */
int relpos_t5_decode_positions(const void* Q, const void* K, const void* V, const void* bias,
                               const int* key_pos, int B, int H, int Lq, int Lk, int num_buckets,
                               int max_distance, int causal, int q_offset, void* out, void* stream);

/*
 * relpos_alibi_decode_positions -- ALiBi cached decoding over keys at
 * explicit positions ("Relative Position Embeddings, in depth", sections
 * "ALiBi and RoPE: the two endpoints" and "Kernels and the KV cache"): the
 * logit of query row i and key j is q_i . k_j / sqrt(64) - slope_h *
 * |key_pos[b, h, j] - (i + q_offset)|.
 *
 *   slopes      device, fp32 [H], 4-byte aligned: the heads' slopes.
 *   key_pos, causal, q_offset, out, B, H, Lk, stream: as for
 *               relpos_t5_decode_positions (bf16 Q, K, V, out; d = 64).
 *   Lq          0 .. 8 query rows (RELPOS_ERR_UNSUPPORTED beyond).
 * The split-key decode kernels, with each key's bias formed from its
 * position. Scratch and asynchrony as relpos_t5_decode_positions for
 * Lq <= 8.
 */
int relpos_alibi_decode_positions(const void* Q, const void* K, const void* V, const void* slopes,
                                  const int* key_pos, int B, int H, int Lq, int Lk, int causal,
                                  int q_offset, void* out, void* stream);

/*
 * relpos_t5_attn_bwd -- gradients of the T5-bias attention forward
 * (relpos_attn_fwd with mode RELPOS_T5, dtype RELPOS_BF16). The bias is a
 * learned table ("Relative Position Embeddings, in depth", section "T5: one
 * scalar per head, looked up by bucket"; "T5 Relative-Position Bias": every
 * offset of a bucket shares the bucket's value), so its gradient gathers the
 * logit gradients dS_ij = P_ij (dP_ij - sum_l P_il dP_il) of every (batch, i, j)
 * whose offset falls in the bucket. The pages print no backward pass; the
 * other gradients follow from the chain rule through the forward:
 * dV = P^T dO, dQ = dS K / sqrt(d), dK = dS^T Q / sqrt(d). The row term
 * sum_j P_ij dP_ij is formed from P and dP themselves (not from the forward's
 * output), so no output of the forward is needed.
 *
 *   Q, K, V, bias, B, H, Lq, Lk, d, num_buckets, max_distance, causal,
 *   q_offset, stream: the forward call's arguments (bf16 Q [B,H,Lq,64], K, V
 *               [B,H,Lk,64]; fp32 bias [num_buckets, H]; d must be 64).
 *   dO          device, bf16 [B,H,Lq,64]: gradient of the loss w.r.t. O.
 *   dQ          device, bf16 [B,H,Lq,64], written.
 *   dK, dV      device, bf16 [B,H,Lk,64], written (rows no query sees: zero).
 *   dbias       device, fp32 [num_buckets, H], overwritten with the sum over
 *               the whole batch (the table is shared by it).
 * All pointers 16-byte aligned and caller-owned; the outputs must not overlap
 * the inputs. Limits: the distance R at which the last bucket starts (or the
 * largest offset present, if smaller) must be <= 1024
 * (RELPOS_ERR_UNSUPPORTED otherwise; max_distance 128 gives R = 91
 * bidirectional, 113 causal). Scratch: about 264 * B * H * Lq bytes (an
 * fp32 dQ accumulator and the row statistics, padded to 128-row tiles) from cudaMallocAsync on `stream`,
 * freed with cudaFreeAsync before the call returns. dQ and dbias are
 * accumulated with floating-point atomics, so their last bits may differ
 * between runs. Asynchronous on `stream`; device timeouts surface through
 * relpos_check_status().
 */
int relpos_t5_attn_bwd(const void* Q, const void* K, const void* V, const void* dO,
                       const void* bias, int B, int H, int Lq, int Lk, int d, int num_buckets,
                       int max_distance, int causal, int q_offset, void* dQ, void* dK, void* dV,
                       void* dbias, void* stream);

/*
 * relpos_alibi_attn_bwd -- gradients of the ALiBi attention forward
 * (relpos_attn_fwd with mode RELPOS_ALIBI, dtype RELPOS_BF16; "Relative
 * Position Embeddings, in depth", section "ALiBi and RoPE: the two
 * endpoints"). The pages treat the slopes as fixed; their gradient is still
 * returned, dslope_h = -sum_{b,i,j} dS_ij |j - p_i|, with dS, dQ, dK, dV as
 * for relpos_t5_attn_bwd.
 *
 *   Q, K, V, dO, B, H, Lq, Lk, d, causal, q_offset, dQ, dK, dV, stream: as for
 *               relpos_t5_attn_bwd.
 *   slopes      device, fp32 [H]: the forward call's slopes.
 *   dslopes     device, fp32 [H], overwritten with the sum over the batch.
 * Scratch, limits and errors as relpos_t5_attn_bwd (no saturation-distance
 * limit). dslopes is accumulated with floating-point atomics.
 */
int relpos_alibi_attn_bwd(const void* Q, const void* K, const void* V, const void* dO,
                          const void* slopes, int B, int H, int Lq, int Lk, int d, int causal,
                          int q_offset, void* dQ, void* dK, void* dV, void* dslopes, void* stream);

/*
 * relpos_shaw_attn_bwd -- gradients of the Shaw attention forward
 * (relpos_attn_fwd with mode RELPOS_SHAW, dtype RELPOS_BF16; "Relative
 * Position Embeddings, in depth", section "Shaw et al."). With r_ij =
 * clip(j - p_i, -k, k) + k the logit is q_i . (k_j + a_K[r_ij]) / sqrt(d) and
 * the value of key j for query i is v_j + a_V[r_ij]. The chain rule gives
 *   dP_ij = dO_i . (v_j + a_V[r_ij]),  dS_ij = P_ij (dP_ij - sum_l P_il dP_il),
 *   dQ_i = sum_j dS_ij (k_j + a_K[r_ij]) / sqrt(d),  dK_j = sum_i dS_ij q_i / sqrt(d),
 *   dV_j = sum_i P_ij dO_i,
 *   da_K[r] = sum of dS_ij q_i / sqrt(d) and da_V[r] = sum of P_ij dO_i over
 *   every (batch, head, i, j) with r_ij = r (the tables are shared by the
 *   batch and the heads).
 *
 *   Q, K, V, dO, B, H, Lq, Lk, d, causal, q_offset, dQ, dK, dV, stream: as for
 *               relpos_t5_attn_bwd.
 *   aK, aV      device, bf16 [2k + 1, 64]: the forward call's tables.
 *   clip_k      k, the forward call's rel_param; 1 <= k <= 16
 *               (RELPOS_ERR_INVALID_ARG below 1, RELPOS_ERR_UNSUPPORTED above 16).
 *   daK, daV    device, fp32 [2k + 1, 64], overwritten with the sums over the
 *               batch and the heads.
 * Scratch: about (264 + 16 (2k + 2) + 4) * B * H * Lq bytes plus
 * 2 (2k + 1) * 256 bytes per 128-row query tile and head, from cudaMallocAsync on `stream`,
 * freed with cudaFreeAsync before the call returns. daK and daV are summed in
 * a fixed order (the same bits every run); dQ, dK and dV as for
 * relpos_t5_attn_bwd. Errors and asynchrony as relpos_t5_attn_bwd.
 */
int relpos_shaw_attn_bwd(const void* Q, const void* K, const void* V, const void* dO,
                         const void* aK, const void* aV, int B, int H, int Lq, int Lk, int d,
                         int clip_k, int causal, int q_offset, void* dQ, void* dK, void* dV,
                         void* daK, void* daV, void* stream);

/*
 * relpos_deberta_attn_bwd -- gradients of the DeBERTa attention forward
 * (relpos_attn_fwd with mode RELPOS_DEBERTA, dtype RELPOS_BF16; "Relative
 * Position Embeddings, in depth", section "DeBERTa: disentangled content and
 * position"; "DeBERTa > Relative Position", the relative-position formula).
 * With delta(i, j) = clip(p_i - j, -k, k - 1) + k and s = 1 / sqrt(3 d) the
 * logit is s (q_i . k_j + q_i . Pk[delta(i, j), h] + k_j . Pq[delta(j, i), h]);
 * the chain rule gives, with dS as for relpos_t5_attn_bwd,
 *   dQ_i = s sum_j dS_ij (k_j + Pk[delta(i, j), h]),
 *   dK_j = s sum_i dS_ij (q_i + Pq[delta(j, i), h]),  dV = P^T dO,
 *   dPk[r, h] = s sum of dS_ij q_i over every (batch, i, j) of head h with
 *   delta(i, j) = r, and dPq[r, h] = s sum of dS_ij k_j over delta(j, i) = r.
 *
 *   Q, K, V, dO, B, H, Lq, Lk, d, causal, q_offset, dQ, dK, dV, stream: as for
 *               relpos_t5_attn_bwd.
 *   Pk, Pq      device, bf16 [2k, H, 64]: the forward call's tables.
 *   k           the forward call's rel_param; 1 <= k <= 4096
 *               (RELPOS_ERR_INVALID_ARG below 1, RELPOS_ERR_UNSUPPORTED above).
 *   dPk, dPq    device, fp32 [2k, H, 64], overwritten with the sums over the
 *               batch.
 * The logits' relative part comes from the forward's band pre-pass (c2p +
 * p2c inside the band, rounded to bf16 as in the forward). Scratch, from
 * cudaMallocAsync on `stream` and freed before the call returns: about
 * (300 + 8k) * B * H * Lq bytes plus (280 + 4k) * B * H * Lk bytes (the
 * band, dS gathered by table row query- and key-major, fp32 dQ and dK).
 * The table products run as cuBLAS GEMMs (bf16 operands, fp32 accumulation;
 * the library is loaded with this one). Errors and asynchrony as
 * relpos_t5_attn_bwd.
 */
int relpos_deberta_attn_bwd(const void* Q, const void* K, const void* V, const void* dO,
                            const void* Pk, const void* Pq, int B, int H, int Lq, int Lk, int d, int k,
                            int causal, int q_offset, void* dQ, void* dK, void* dV, void* dPk, void* dPq,
                            void* stream);

/*
 * ---------------------------------------------------------------------------
 * Rotary positions ("Relative Position Embeddings, in depth", section "ALiBi
 * and RoPE: the two endpoints": queries and keys are turned by their position
 * before attention, so that their product depends on the offset alone). The
 * page names the scheme without formulas; the reading here is the usual one.
 *
 * The first rot_dim dimensions of a head form rot_dim / 2 pairs. Pair m at
 * position p is turned by the angle p w_m and scaled by the plan's amplitude a:
 *   (x1, x2) -> a (x1 cos - x2 sin, x1 sin + x2 cos)
 * RELPOS_ROTARY_HALF         x1 = x[m],  x2 = x[m + rot_dim / 2]
 * RELPOS_ROTARY_INTERLEAVED  x1 = x[2m], x2 = x[2m + 1]
 * The dimensions from rot_dim on pass unchanged.
 *
 * Frequencies: w_m = base^(-2m / rot_dim), a = 1, and for contexts longer than
 * the trained one
 *   RELPOS_ROTARY_LINEAR  w_m / factor (position interpolation)
 *   RELPOS_ROTARY_NTK     the base times factor^(rot_dim / (rot_dim - 2))
 *   RELPOS_ROTARY_YARN    by parts: with r_m = original_len w_m / 2 pi turns
 *                         over the trained length and g = (r_m - slow_turns) /
 *                         (fast_turns - slow_turns) clipped to [0, 1], w_m
 *                         becomes (1 - g) w_m / factor + g w_m; a = 0.1
 *                         ln(factor) + 1 (Peng et al., "YaRN: Efficient Context
 *                         Window Extension of Large Language Models")
 */
#define RELPOS_ROTARY_HALF 0
#define RELPOS_ROTARY_INTERLEAVED 1

#define RELPOS_ROTARY_PLAIN 0
#define RELPOS_ROTARY_LINEAR 1
#define RELPOS_ROTARY_NTK 2
#define RELPOS_ROTARY_YARN 3

#define RELPOS_ROTARY_MAX_DIM 256

/* A host-side plan, filled by relpos_rotary_plan_init and passed to the calls
   below by pointer (its contents are copied into the launch). */
typedef struct RelposRotaryPlan {
  int rot_dim;
  int layout;
  double amplitude;
  unsigned long long turns[RELPOS_ROTARY_MAX_DIM / 2]; /* w_m / 2 pi, in 2^-64 of a turn */
} RelposRotaryPlan;

/* One tensor of a relpos_rotary call: x and out [B, H, L, d] with the given
   strides in elements (the d values of a row are contiguous). */
typedef struct RelposRotaryTensor {
  const void* x;
  void* out;
  long long x_batch, x_head, x_row;
  long long out_batch, out_head, out_row;
  int H;
} RelposRotaryTensor;

/*
 * relpos_rotary_plan_init -- fill a plan (host only, nothing is launched).
 *
 *   rot_dim       even, 2 .. RELPOS_ROTARY_MAX_DIM (NTK: at least 4).
 *   layout        RELPOS_ROTARY_HALF or RELPOS_ROTARY_INTERLEAVED.
 *   base          > 1.
 *   scaling       RELPOS_ROTARY_PLAIN, _LINEAR, _NTK or _YARN.
 *   factor        >= 1 (ignored by PLAIN).
 *   original_len  > 0, fast_turns > slow_turns >= 0: YARN only.
 */
int relpos_rotary_plan_init(RelposRotaryPlan* plan, int rot_dim, int layout, double base, int scaling,
                            double factor, double original_len, double fast_turns, double slow_turns);

/*
 * relpos_rotary -- turn one or two tensors (queries and keys) by position, in
 * one launch.
 *
 *   dtype       RELPOS_BF16 or RELPOS_FP32: element type of every x and out.
 *               Computed in fp32, rounded once.
 *   inverse     0, or 1 to turn by the opposite angle with the same amplitude:
 *               the gradient of the call with inverse = 0 (x the gradient of
 *               its output).
 *   tensors     host array of `ntensors` (1 or 2) descriptions. out may be x
 *               itself (with x's strides); otherwise nothing may overlap:
 *               strides of out below d where there is more than one row are
 *               refused (an x of broadcast rows needs an out of its own).
 *   B, L, d     batch, rows and head dimension (even, >= the plan's rot_dim);
 *               an empty size makes the call a no-op.
 *   positions   device, int32: row l of batch element b is at
 *               positions[b * pos_stride + l] (pos_stride 0: one row of
 *               positions for the whole batch). Any int32 values; angles are
 *               exact modulo a full turn. Null: position offset + l.
 * Sizes and strides that allow 16- or 8-byte accesses (rot_dim and d
 * multiples of 16 or 8, rows that start on such a boundary) run with them,
 * others element by element. Asynchronous on `stream`, no scratch.
 */
int relpos_rotary(const RelposRotaryPlan* plan, int dtype, int inverse, const RelposRotaryTensor* tensors,
                  int ntensors, int B, int L, int d, const int* positions, long long pos_stride, int offset,
                  void* stream);

/*
 * ---------------------------------------------------------------------------
 * Paged key/value cache ("Relative Position Embeddings, in depth", section
 * "Kernels and the KV cache"; the pages treat one contiguous cache, the pages
 * of memory are this library's reading). A pool of num_pages pages holds `page`
 * tokens of every key/value head each; a sequence owns a list of pages (its row
 * of the block table) and the token at position j lies in slot j mod page of
 * its page number j / page.
 *
 *   k, v             device, [num_pages, H, page, d], 16-byte aligned: bf16, or
 *                    e4m3 codes (1 byte).
 *   k_scale, v_scale device, fp32 [num_pages, H] (E4M3 only): a stored value is
 *                    its code times its page's and head's scale. The append
 *                    writes powers of two; pages quantised elsewhere may have
 *                    others.
 *   d                64 or 128; page 32, 64 or 128 (RELPOS_ERR_UNSUPPORTED
 *                    otherwise). Host struct, copied into each launch.
 *
 * Block tables are device int32 [B, max_pages] with table_stride elements
 * between rows; lens is device int32 [B]: the tokens of each sequence, those
 * of the current step included. The kernels check lengths and page numbers
 * against the cache, skip what lies outside it and report it through
 * relpos_check_status() as RELPOS_ERR_PAGE: a sequence longer than its row of
 * the block table (nothing is appended; its rows of a decode are zero), and a
 * page number that is none (its tokens are not written; a decode leaves its
 * keys out). Table entries beyond a sequence's last page are never read. Make the first call on a device before any stream
 * capture (it looks up the device status word and sizes launches).
 */
typedef struct RelposPagedCache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int num_pages, H, page, d;
  int dtype;
} RelposPagedCache;

/* strides in elements of a [B, H, L, d] tensor (batch unused for ragged rows) */
typedef struct RelposRowStrides {
  long long batch, head, row;
} RelposRowStrides;

/*
 * relpos_paged_append -- write each sequence's newest tokens into its pages.
 * Sequence b with n_b new tokens and lens[b] tokens in all gets them at
 * positions lens[b] - n_b .. lens[b] - 1.
 *
 *   plan        null: keys are stored as they are; otherwise turned at their
 *               positions (rot_dim <= d and a multiple of 16,
 *               RELPOS_ERR_UNSUPPORTED otherwise).
 *   K, V        device, bf16 rows of d contiguous values with the given
 *               strides. cu_new null: n new tokens of every sequence, row i of
 *               head h of sequence b at b * batch + h * head + i * row. Else
 *               ragged: cu_new is device int32 [B + 1], ascending from >= 0,
 *               n_b = cu_new[b + 1] - cu_new[b], and row i of sequence b is row
 *               cu_new[b] + i of the `rows` rows. Rows behind the last
 *               sequence are not read.
 *   lens        an entry <= 0, or without new tokens, is skipped (an unused
 *               entry of a padded batch).
 *
 * BF16 caches: the turned keys and the values, rounded once. E4M3 caches: a
 * page's scale for a head becomes the smallest power of two (within 2^-120 ..
 * 2^120) that holds the largest new magnitude in 448 times it, for turned keys
 * sqrt(2) * amplitude times that magnitude, which holds them at any angle; it
 * never becomes smaller than it was while the page is being filled (a page
 * whose first token is written starts afresh), and when it grows the codes
 * already in the page are rounded to it. Codes are the correctly rounded ones
 * (nearest, ties to even; a value next to a border is decided in 64 bits), also
 * in a page whose scale so far is no power of two and is kept. An infinity takes the largest scale and saturates, NaN stays NaN and has no
 * share in the scale.
 *
 * Slots outside the new tokens keep their bytes unless their page's scale
 * grows. Pages written by one call must not be shared by two of its
 * sequences, appear twice in one, nor be written or read by another stream
 * meanwhile. Appending the same tokens again writes the same bytes. Asynchronous on `stream`, no
 * scratch.
 */
int relpos_paged_append(const RelposPagedCache* cache, const RelposRotaryPlan* plan, const void* K, const void* V,
                        const RelposRowStrides* k_strides, const RelposRowStrides* v_strides, const int* cu_new,
                        int rows, int n, int B, const int* block_table, long long table_stride, int max_pages,
                        const int* lens, void* stream);

/*
 * relpos_paged_decode -- attention of each sequence's newest Lq rows over its
 * cached tokens, their own included (append them first).
 *   logit = q . k * scale + bias,  out = softmax(logit) v
 * Query row i of sequence b sits at position lens[b] - Lq + i and sees the
 * keys up to that position; a row before the sequence's start is zero. Head hq
 * of the Hq query heads reads key/value head hq / (Hq / H); Hq must be a
 * multiple of the cache's H.
 *
 *   bias_mode   RELPOS_NO_BIAS; RELPOS_T5: bias device fp32 [num_buckets, Hq],
 *               causal buckets (num_buckets and max_distance as for
 *               relpos_attn_fwd); RELPOS_ALIBI: bias device fp32 [Hq], the
 *               slopes, -slope |offset| is added.
 *   Q, out      device, bf16 [B, Hq, Lq, d] with the given strides in elements
 *               (rows of d contiguous values, 2-byte aligned). Rows of out may
 *               not overlap: strides below d are refused; those of Q may.
 *   Lq          0 .. 8 rows (RELPOS_ERR_UNSUPPORTED beyond).
 *   scale       softmax scale, finite; 0 takes 1 / sqrt(d).
 * Keys and values in masked or unused slots have no effect, whatever they
 * hold, nor has a page's scale on rows that see no key of the page. Sums are
 * fp32, of weights up to 2^13 and values, before the division by the weights'
 * sum: values from about 2^100 on may overflow to infinity. A weight is rounded
 * for its product with the value: to 16 bits in BF16 caches, in E4M3 caches to
 * 11 bits down to 2^-18 of the row's largest weight and to 2^-29 of that below.
 * The cache is read once for up to 8 or 16 rows (query heads of a group
 * times Lq) and again, mostly from L2, for each further 8 or 16. Scratch: up to
 * about 8 MB for partial results of sequences that several blocks share, drawn
 * on `stream` from a memory pool of the library (which keeps up to 64 MB for the
 * calls to come) and given back before the call returns; none where the block
 * table holds at most 16 tiles (256 tokens for bf16 with d = 128, 512
 * otherwise). What a call costs beside its tokens follows the width of the block
 * table (launches, rows read together), so it should be no wider than the
 * longest sequence needs. Results do not depend on what else runs. Asynchronous
 * on `stream`.
 */
#define RELPOS_NO_BIAS (-1)
int relpos_paged_decode(const RelposPagedCache* cache, const void* Q, const RelposRowStrides* q_strides, int B,
                        int Hq, int Lq, const int* block_table, long long table_stride, int max_pages,
                        const int* lens, int bias_mode, const void* bias, int num_buckets, int max_distance,
                        float scale, void* out, const RelposRowStrides* out_strides, void* stream);

/*
 * relpos_selftest_paged_decode_split -- how a relpos_paged_decode of these sizes
 * is cut up on the current device: rows of a unit of work (8 or 16) and kernel
 * launches (1 or 2). Launches nothing. Lets a test make sure which kernels it runs.
 */
int relpos_selftest_paged_decode_split(const RelposPagedCache* cache, int B, int Hq, int Lq, int max_pages, int* rows,
                                       int* launches);

#ifdef __cplusplus
}
#endif

#endif /* RELPOS_ATTN_H_ */
