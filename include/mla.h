/*
 * mla.h - C ABI of libmla.so: absorbed Multi-Head Latent Attention decode over
 * a paged latent KV cache, hand-written CUDA for NVIDIA B200 (sm_100a).
 *
 * The method ("Multi-Head Latent Attention: Scaling LLM Serving Throughput via
 * Low-Rank KV Compression", priorstack.com, sections "Empirical Gains" and
 * "Frequently Asked Questions"): every cached token keeps one shared row
 * [c_kv (d_c = 512) | k_rope (d_h^R = 64)]; the key up-projection W_UK is
 * absorbed into the query and W_UV into the output projection, so the decode
 * step attends directly over the latent rows:
 *
 *     q_abs[b,h,:] = q_nope[b,h,:] . W_UK[h]                        (512)
 *     s[b,h,t]     = scale * (q_abs[b,h,:] . c_kv[t] + q_rope[b,h,:] . k_rope[t])
 *     out[b,h,:]   = sum_t softmax_t(s[b,h,:]) c_kv[t]               (512)
 *     lse[b,h]     = log sum_t exp(s[b,h,t])                         (natural log)
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers unless stated otherwise, owned by
 *     the caller.  No call allocates memory (mla_decode_noalloc's scratch is a
 *     file-scope array that exists from load time), and no call synchronises
 *     the stream except the three *_get_error calls, which say so.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     All work is enqueued on it in order.
 *   - Arguments are validated on the host before anything is launched; a
 *     failed check returns an error status and launches nothing.
 *   - A launch failure returns MLA_ERR_CUDA (cudaGetLastError is consumed).
 *   - Fixed dimensions: d_c = 512, d_h^R = 64, row = 576, 64 tokens per cache
 *     block, 128-wide content query (d_h) for absorption.  H must be a
 *     multiple of 16 in [16, 128].
 *   - bf16 = IEEE binary32 upper half; fp8 = OCP E4M3 (bias 7, max 448, NaN
 *     S.1111.111, no infinities).  Outputs are rounded to nearest even.
 *   - State kept by the library: the wait bound of mla_set_wait_limit
 *     (process-wide), the MLA_SPLITS value (read once per process), per-device
 *     kernel attributes set on first use, the text of each host thread's last
 *     CUDA error (mla_last_error_string) and mla_decode_noalloc's scratch
 *     array (shared by every call on a device).  No other call keeps state
 *     between calls: the caller's workspace carries each decode's scratch and
 *     error word.  Concurrent calls on different streams are safe provided
 *     they use different output and workspace buffers (and, for
 *     mla_decode_noalloc, do not overlap on one device).
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MLA_OK = 0,
    MLA_ERR_INVALID_ARG = 1,         /* null pointer, bad size or alignment */
    MLA_ERR_UNSUPPORTED = 2,         /* valid request this build does not handle */
    MLA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < mla_decode_workspace_bytes(...) */
    MLA_ERR_CUDA = 4,                /* a CUDA runtime/driver call or launch failed */
    MLA_ERR_DEVICE = 5               /* reserved, returned by no call: device-side problems are
                                        MLA_DEVERR_* bits read by the *_get_error calls */
} mla_status_t;

typedef enum {
    MLA_CACHE_BF16 = 0,     /* cache: bf16 [num_blocks, 64, 576] rows [c_kv | k_rope] */
    MLA_CACHE_FP8_E4M3 = 1  /* cache: u8 E4M3 [num_blocks, 64, 512] codes of c_kv / block_scale,
                               k_rope: bf16 [num_blocks, 64, 64], block_scale: f32 [num_blocks] */
} mla_cache_dtype_t;

/* Device-side error bits (read with mla_get_device_error). */
#define MLA_DEVERR_BAD_BLOCK   0x1u  /* a block_table entry needed by seq_lens is < 0 or >= num_blocks */
#define MLA_DEVERR_SEQ_TOO_LONG 0x2u /* seq_lens[b] > 64 * max_blocks_per_seq or < 0 */
#define MLA_DEVERR_TIMEOUT     0x4u  /* a bounded wait inside a kernel gave up; the kernel exited */
#define MLA_DEVERR_BAD_PIECES  0x8u  /* decode: split-KV bookkeeping out of range (internal error);
                                        the affected rows read out = 0, lse = NaN */

/*
 * mla_absorb_q - fold the key up-projection into the query ("Empirical Gains":
 * W^UK is absorbed into the query projection):
 *     q_out[(b*H + h)*ldq + c]       = sum_{d<128} q_nope[b,h,d] * w_uk[h,d,c],  c < 512
 *     q_out[(b*H + h)*ldq + 512 + r] = q_rope[b,h,r],  r < 64   (only if q_rope != NULL)
 * q_nope: bf16 [B,H,128]; w_uk: bf16 [H,128,512]; q_rope: bf16 [B,H,64] or NULL;
 * q_out: bf16 rows of stride ldq elements (ldq >= 512, >= 576 if q_rope != NULL,
 * a multiple of 8; 576 builds the packed [B,H,576] query mla_decode reads).
 * fp32 accumulation (tensor cores), one bf16 rounding.  B >= 1.  All pointers
 * 16-byte aligned; q_nope and w_uk dense in the layouts above.
 */
mla_status_t mla_absorb_q(const void *q_nope, const void *w_uk, const void *q_rope,
                          void *q_out, int ldq, int B, int H, void *stream);

/*
 * mla_absorb_o - the output side of the absorption ("Empirical Gains": W^UV is
 * absorbed into the output projection, so per-head values are never formed):
 *     out[(b*H + h)*ldo + d] = sum_{c<512} w_uv[h,d,c] * o_latent[b,h,c],  d < 128
 * o_latent: bf16 [B,H,512] (e.g. mla_decode's out); w_uv: bf16 [H,128,512];
 * out: bf16 rows of stride ldo elements (ldo >= 128, a multiple of 8).
 * fp32 accumulation (tensor cores), one bf16 rounding.  B >= 1; H in
 * {16,32,...,128}.  All pointers 16-byte aligned; o_latent and w_uv dense.
 */
mla_status_t mla_absorb_o(const void *o_latent, const void *w_uv, void *out, int ldo, int B,
                          int H, void *stream);

/*
 * mla_absorb_get_error - device error bits of the mla_absorb_q / mla_absorb_o launches since
 * the last call (MLA_DEVERR_TIMEOUT when a bounded wait in the kernel gave up;
 * the affected rows are then not written).  Synchronises `stream` and clears
 * the bits.  The error word is one per device and process: absorption calls on
 * different streams (or threads) record into, and this call clears, the same
 * word.  MLA_ERR_INVALID_ARG if err_bits is NULL.
 */
mla_status_t mla_absorb_get_error(void *stream, uint32_t *err_bits);

/*
 * mla_decode_workspace_bytes - bytes of device workspace mla_decode needs for
 * H heads (mla_decode_multi: H = q_len * heads rows, up to 1024, which above
 * 128 need the workspace of one 128-row tile) and `num_splits` split-KV partitions (0 = the automatic count the
 * current device would use).  The workspace holds the device error word and
 * the fp32 partial results of sequences that are cut across partitions.
 * Returns 0 on invalid arguments.
 */
size_t mla_decode_workspace_bytes(int B, int H, int num_splits);

/*
 * mla_decode_fp8_workspace_bytes - workspace bytes that let mla_decode widen
 * the whole batch of an fp8 cache at once: mla_decode_workspace_bytes(B, H, num_splits)
 * rounded up to 256, plus a scratch block table (4 * B * max_blocks_per_seq
 * bytes, rounded up to 256) and a widened bf16 copy of the blocks the batch
 * reads (73,728 bytes per table entry: B * max_blocks_per_seq blocks of
 * 64 x 576 bf16).  Returns 0 on invalid arguments or when
 * B * max_blocks_per_seq exceeds 2^24.
 */
size_t mla_decode_fp8_workspace_bytes(int B, int H, int max_blocks_per_seq, int num_splits);

/*
 * mla_decode - the decode-step attention over the paged latent cache
 * ("Empirical Gains": the cache holds only c^KV and the decoupled RoPE key;
 * "The Memory Wall": the whole cache is streamed from HBM every step).
 *
 * q:           bf16 [B,H,576] = [q_abs | q_rope] per (b,h) (from mla_absorb_q).
 * cache_dtype: MLA_CACHE_BF16 or MLA_CACHE_FP8_E4M3 (see the enum).
 * cache:       bf16 [num_blocks,64,576] or u8 [num_blocks,64,512].
 * k_rope:      fp8 cache only: bf16 [num_blocks,64,64]; must be NULL for bf16.
 * block_scale: fp8 cache only: f32 [num_blocks], c_kv = e4m3(code) * scale;
 *              must be NULL for bf16.
 *              The fp8 cache runs in two kernels: the first writes the rows
 *              a group of sequences reads as bf16
 *              [bf16(e4m3(code) * scale) | k_rope] into the workspace (round
 *              to nearest even: relative error <= 2^-9 per element), the
 *              tensor-core decode then reads them as a bf16 cache.  With
 *              mla_decode_fp8_workspace_bytes(B, H, max_blocks_per_seq,
 *              num_splits) bytes the group is the whole batch; with less,
 *              the call runs the largest groups of consecutive sequences (and
 *              if need be fewer split-KV engines) that fit, one after the
 *              other on `stream`; MLA_ERR_WORKSPACE_TOO_SMALL when not even
 *              one sequence on one engine fits.
 * block_table: int32 [B, max_blocks_per_seq]; logical block j of sequence b is
 *              physical block block_table[b*max_blocks_per_seq + j].  Entries
 *              at j >= ceil(seq_lens[b]/64) are never read (pad with -1).
 * seq_lens:    int32 [B] on the device; 0 <= seq_lens[b] <= 64*max_blocks_per_seq.
 * softmax_scale: multiplies the whole score (both terms) before the softmax.
 * out:         bf16 [B,H,512], the softmax-weighted sum of c_kv per head.
 * lse:         f32 [B,H], natural log of sum_t exp(score); a sequence of
 *              length 0 gives out = 0 and lse = -inf.
 * workspace:   device buffer of >= mla_decode_workspace_bytes(B,H,num_splits)
 *              bytes (fp8 cache: see block_scale), 256-byte aligned, ZERO-FILLED BEFORE ITS FIRST USE; the
 *              library keeps its error word zero except when it records an
 *              error.  One workspace must not be shared by calls that may run
 *              at the same time.
 * num_splits:  number of split-KV partitions (0 = automatic: the environment
 *              variable MLA_SPLITS, read once per process, when it holds an
 *              integer in 1..4096; else chosen from the device's SM count and
 *              B, the same in mla_decode_workspace_bytes).  Results do not
 *              depend on the physical block placement; they may differ in the
 *              last bits between different num_splits.
 *
 * Preconditions checked on the host: non-null pointers, B >= 1, H in
 * {16,32,...,128}, num_blocks >= 1, max_blocks_per_seq >= 1, 16-byte
 * alignment, the fp8-only pointers present exactly for the fp8 cache.
 * Checked on the device (recorded as error bits, the offending rows are
 * skipped): block ids in range, seq_lens in range.  Every internal wait is
 * bounded; on expiry the kernel records MLA_DEVERR_TIMEOUT and exits cleanly.
 * While MLA_DEVERR_TIMEOUT is set in the workspace's error word (it stays set
 * until mla_get_device_error reads it), every row a call writes reads out = 0,
 * lse = NaN, so that no result of an incomplete decode is ever returned.
 */
mla_status_t mla_decode(const void *q, mla_cache_dtype_t cache_dtype, const void *cache,
                        const void *k_rope, const float *block_scale,
                        const int32_t *block_table, const int32_t *seq_lens, int B, int H,
                        int num_blocks, int max_blocks_per_seq, float softmax_scale,
                        void *out, float *lse, void *workspace, size_t workspace_bytes,
                        int num_splits, void *stream);

/*
 * mla_decode_multi - decode q_len query tokens per sequence at once (multi-
 * token prediction / speculative drafts): the q_len * H query rows of a
 * sequence share every cache row they read, so one pass over the cache serves
 * them all.  Token j of sequence b is the (seq_lens[b] - q_len + 1 + j)-th
 * token: it attends to the first seq_lens[b] - (q_len - 1 - j) cached tokens
 * (the drafts' own rows are already in the cache; causal among the drafts).
 * q: bf16 [B, q_len, H, 576]; out: bf16 [B, q_len, H, 512]; lse: f32
 * [B, q_len, H]; bf16 cache only.  q_len * H must be a multiple of 16 and at
 * most 128, or a multiple of 128 up to 1024 with H dividing 128 (e.g. H = 128
 * and q_len = 2..8): such rows are decoded in tiles of 128 rows (whole
 * tokens), one kernel pass over the cache per tile, one tile after the other
 * on `stream`; the tiles read q and write out / lse in place.
 * workspace: mla_decode_workspace_bytes(B, q_len * H, num_splits) bytes.
 * Other arguments and error behaviour as mla_decode; a token that sees no
 * cached token gives out = 0 and lse = -inf.
 */
mla_status_t mla_decode_multi(const void *q, int q_len, const void *cache,
                              const int32_t *block_table, const int32_t *seq_lens, int B, int H,
                              int num_blocks, int max_blocks_per_seq, float softmax_scale,
                              void *out, float *lse, void *workspace, size_t workspace_bytes,
                              int num_splits, void *stream);

/*
 * mla_combine - log-sum-exp merge of S split-KV partial results (the
 * flash-decoding merge that makes split-KV equal the unsplit softmax):
 *     M = max_i lse_part[r,i];  lse[r] = M + log sum_i exp(lse_part[r,i] - M)
 *     out[r,:] = sum_i exp(lse_part[r,i] - lse[r]) * o_part[r,i,:]
 * with r = b*H + h.  o_part: f32 [B,H,S,512] (each piece already normalised by
 * its own softmax sum); lse_part: f32 [B,H,S] (-inf marks an empty piece);
 * out: bf16 [B,H,512]; lse: f32 [B,H].  Rows whose pieces are all -inf give
 * out = 0, lse = -inf.  S >= 1.
 */
mla_status_t mla_combine(const float *o_part, const float *lse_part, int B, int H, int S,
                         void *out, float *lse, void *stream);

/*
 * mla_get_device_error - wait for `stream`, read the MLA_DEVERR_* bits that
 * kernels using `workspace` recorded, and reset them to zero.  *err_bits
 * receives the bits.  Returns MLA_OK, or MLA_ERR_CUDA if the stream or copy
 * failed.  It synchronises the stream (as do mla_absorb_get_error and
 * mla_cache_get_error; no other call does).
 */
mla_status_t mla_get_device_error(void *workspace, void *stream, uint32_t *err_bits);

/*
 * mla_decode_noalloc - mla_decode with its scratch memory built into the
 * library.  The paper has no counterpart: this is a deployment variant for
 * callers that cannot allocate device memory themselves (processes that work
 * inside a fixed budget carved out at start-up and route every later device
 * allocation through their own pool, or latency-critical paths where
 * cudaMalloc/cudaFree may synchronise the device).  Arguments are those of
 * mla_decode without workspace/workspace_bytes; results are the same up to
 * the last bits.
 *
 * Scratch: one file-scope device array of 40 MiB, held on every GPU that
 * loads the library until the process exits.  A request whose scratch need
 * (mla_decode_workspace_bytes(B, H, num_splits)) exceeds 40 MiB returns
 * MLA_ERR_WORKSPACE_TOO_SMALL and launches nothing (at H = 128 the automatic
 * split count of a B200 needs at most about 39 MB).  The first call on a device looks
 * up the array's address on that device; make it before any stream capture.
 * All calls on a device share the array and it keeps the last call's
 * contents: calls that overlap on the GPU race, so serialise them.  Nothing
 * in it needs clearing between calls.  Device-side error bits accumulate in
 * the array's error word; read and clear them with
 * mla_decode_noalloc_get_error (while MLA_DEVERR_TIMEOUT is set there, calls
 * write out = 0, lse = NaN, as mla_decode does).  An fp8 cache is widened in
 * the array: the whole batch when mla_decode_fp8_workspace_bytes(...) fits in
 * the 40 MiB, else in groups of sequences (see mla_decode).  Allocates and
 * frees no device memory.
 */
mla_status_t mla_decode_noalloc(const void *q, mla_cache_dtype_t cache_dtype, const void *cache,
                                const void *k_rope, const float *block_scale,
                                const int32_t *block_table, const int32_t *seq_lens, int B, int H,
                                int num_blocks, int max_blocks_per_seq, float softmax_scale,
                                void *out, float *lse, int num_splits, void *stream);

/*
 * mla_decode_noalloc_get_error - mla_get_device_error for the built-in
 * scratch of mla_decode_noalloc on the current device: waits for `stream`,
 * stores the accumulated MLA_DEVERR_* bits in *err_bits and clears them.
 * MLA_ERR_INVALID_ARG if err_bits is NULL, MLA_ERR_CUDA if the scratch
 * cannot be located or the copy fails.
 */
mla_status_t mla_decode_noalloc_get_error(void *stream, uint32_t *err_bits);

/*
 * mla_cache_append - write the rows of T new tokens into the paged bf16 cache
 * ("Empirical Gains": only c^KV and the decoupled RoPE key are cached; the key
 * is rotated before caching, in fp32 — eeumee.net, FP8/FP32 Mixed Precision):
 *     cache[block_table[b*max_blocks_per_seq + p/64], p%64, :] = [c_kv[t] | RoPE(k_r[t], p)]
 * with b = seq_idx[t], p = pos[t].  RoPE rotates consecutive pairs
 * (x_2i, x_2i+1) by p * 10000^(-2i/64).
 * c_kv: bf16 [T,512] (16-byte aligned); k_r: bf16 [T,64], before rotation;
 * seq_idx, pos: int32 [T] on the device; block_table: int32 [B, max_blocks_per_seq];
 * cache: bf16 [num_blocks,64,576] (16-byte aligned).  Tokens with b or p out
 * of range, or whose block id is out of range, are skipped and recorded as
 * MLA_DEVERR_SEQ_TOO_LONG / MLA_DEVERR_BAD_BLOCK (mla_cache_get_error).  Two
 * tokens must not target the same row.  T = 0 is a no-op.
 */
mla_status_t mla_cache_append(const void *c_kv, const void *k_r, const int32_t *seq_idx,
                              const int32_t *pos, int T, const int32_t *block_table, int B,
                              int max_blocks_per_seq, int num_blocks, void *cache, void *stream);

/*
 * mla_cache_quantize_fp8 - convert n whole blocks of a bf16 cache to the fp8
 * layout mla_decode reads (MLA_CACHE_FP8_E4M3), at the same block ids
 * (eeumee.net, FP8/FP32 Mixed Precision; the per-block scale follows the
 * E4M3 range): for each listed block k,
 *     block_scale[k] = amax_k / 448 (1 if the block's c_kv is all zero),
 *     codes[k, r, c] = E4M3(c_kv[k, r, c] / block_scale[k])  (nearest, saturating),
 *     k_rope[k, r, :] = cache_bf16[k, r, 512:576]  (copied),
 * the divisions in IEEE fp32.  cache_bf16: bf16 [num_blocks,64,576];
 * blocks: int32 [n] on the device; codes: u8 [num_blocks,64,512];
 * k_rope: bf16 [num_blocks,64,64]; block_scale: f32 [num_blocks].  Ids out of
 * range are skipped and recorded as MLA_DEVERR_BAD_BLOCK.  n = 0 is a no-op.
 */
mla_status_t mla_cache_quantize_fp8(const void *cache_bf16, const int32_t *blocks, int n,
                                    int num_blocks, void *codes, void *k_rope, float *block_scale,
                                    void *stream);

/*
 * mla_rope_freqs - angle per position of every rotated pair, for mla_rope and
 * mla_cache_append_rope.  HOST function: writes rot / 2 doubles to the host
 * array `freqs` (copy them to the device for the calls).  With
 * theta_i = base^(-2i/rot), i < rot / 2:
 *   MLA_ROPE_PLAIN   f_i = theta_i
 *   MLA_ROPE_LINEAR  f_i = theta_i / factor               (position interpolation)
 *   MLA_ROPE_NTK     f_i = (base * factor^(rot/(rot-2)))^(-2i/rot): the fastest pair
 *                    keeps its angle, the slowest is slowed by `factor`
 *   MLA_ROPE_YARN    pairs that turn more than beta_fast times over the original
 *                    context orig_len keep theta_i, pairs that turn fewer than
 *                    beta_slow times get theta_i / factor, with a linear ramp between
 *                    (NTK-by-parts of "YaRN: Efficient Context Window Extension of
 *                    Large Language Models", but with the ramp over the pair index
 *                    between whole bounds, as released models have it, where the
 *                    paper's is over the turns): with pair(n) = rot * ln(orig_len /
 *                    (2 pi n)) / (2 ln base), lo = max(0, floor(pair(beta_fast))),
 *                    hi = min(rot - 1, ceil(pair(beta_slow))), r_i = clamp((i - lo) /
 *                    max(hi - lo, 0.001), 0, 1):
 *                    f_i = theta_i (1 - r_i) + theta_i / factor * r_i
 * rot: even, 2..256; base > 1; factor >= 1 and finite; orig_len > 0 and beta_fast >=
 * beta_slow > 0 (MLA_ROPE_YARN only, ignored otherwise).  factor = 1 gives theta_i in
 * every mode.  MLA_ROPE_NTK needs rot >= 4.
 */
typedef enum {
    MLA_ROPE_PLAIN = 0,
    MLA_ROPE_LINEAR = 1,
    MLA_ROPE_NTK = 2,
    MLA_ROPE_YARN = 3
} mla_rope_scaling_t;

mla_status_t mla_rope_freqs(int rot, double base, mla_rope_scaling_t scaling, double factor,
                            double orig_len, double beta_fast, double beta_slow, double *freqs);

/* Layout flags of the rotation (mla_rope, mla_cache_append_rope). */
#define MLA_ROPE_INTERLEAVED 0x0u /* pair i = elements (2i, 2i + 1) */
#define MLA_ROPE_HALF        0x1u /* pair i = elements (i, i + rot/2) */
#define MLA_ROPE_INVERSE     0x2u /* rotate by the negative angle */

/*
 * mla_rope - rotary positions of T tokens with H heads each: every pair (a, b) of the
 * rot rotated elements of x[t,h] becomes, with c = mscale cos(pos[t] f_i) and
 * s = mscale sin(pos[t] f_i) (s negated by MLA_ROPE_INVERSE),
 *     (a c - b s,  a s + b c)
 * so that a score depends on the distance of two positions only.  x, y: bf16; element
 * r of head h of token t is x[t*x_ldt + h*x_ldh + r], r < rot (strides in elements), so
 * the rotated part of a longer head ([nope | rope] rows) is a pointer to its first
 * element, and y can be the last 64 columns of the packed [T,H,576] query that
 * mla_absorb_q writes (pass it q_rope = NULL).  Elements outside the rot rotated ones
 * are not touched.  y = x with equal strides rotates in place; y must not overlap x in
 * any other way, nor two of its own rows each other.
 * pos: int32 [T] (any value); freqs: f64 [rot/2] from mla_rope_freqs, on the device;
 * mscale: finite.  The angle is formed and reduced in double (off by at most 2^-30 turns up
 * to position 2^24 and 2^-23 at 2^31); the rotation is fp32, rounded once.  The inverse rotation with the
 * same mscale is also the gradient of y with respect to x.
 * T >= 0 (0 is a no-op), 1 <= H <= 65535, rot even in 2..256, strides >= 0;
 * x, y 2-byte, pos 4-byte and freqs 8-byte aligned.  Rows whose pointers and strides are
 * multiples of 16 bytes, with rot a multiple of 16, are moved 16 bytes at a time.
 */
mla_status_t mla_rope(const void *x, long long x_ldt, long long x_ldh, const int32_t *pos,
                      const double *freqs, float mscale, unsigned flags, void *y,
                      long long y_ldt, long long y_ldh, int T, int H, int rot, void *stream);

/*
 * mla_cache_append_rope - mla_cache_append for tokens whose position is not their slot
 * (a cache that mla_cache_evict compacted) or whose rotation is scaled or laid out
 * differently:
 *     cache[block_table[b,s/64], s%64, :] = [c_kv[t] | R(k_r[t], pos[t])],  s = slot[t]
 * with b = seq_idx[t] and R the rotation of mla_rope (rot = 64; freqs f64 [32]).
 * c_kv: bf16 rows of stride ckv_ld elements (>= 512, a multiple of 8, 16-byte aligned);
 * k_r: bf16 rows of stride kr_ld elements (>= 64, even, 4-byte aligned): both may be
 * columns of one [T,576] projection.  slot_pos: int32 [B, 64*max_blocks_per_seq] or
 * NULL; if given, slot_pos[b,s] = pos[t] is recorded for mla_cache_evict.  Errors as
 * for mla_cache_append (mla_cache_get_error).  T = 0 is a no-op.
 */
mla_status_t mla_cache_append_rope(const void *c_kv, int ckv_ld, const void *k_r, int kr_ld,
                                   const int32_t *seq_idx, const int32_t *slot,
                                   const int32_t *pos, int T, const double *freqs, float mscale,
                                   unsigned flags, const int32_t *block_table, int B,
                                   int max_blocks_per_seq, int num_blocks, void *cache,
                                   int32_t *slot_pos, void *stream);

/*
 * mla_chunk_workspace_bytes - bytes of device workspace mla_chunk_attend needs for T
 * query tokens of B sequences with H heads and `num_splits` split-KV partitions (0 = the
 * automatic count of the current device).  Returns 0 on invalid arguments.
 */
size_t mla_chunk_workspace_bytes(int T, int B, int H, int num_splits);

/*
 * mla_chunk_fp8_workspace_bytes - the same for an fp8 cache: rounded up to 256, plus the
 * scratch block table and the widened bf16 copy of the blocks the batch reads, as in
 * mla_decode_fp8_workspace_bytes.  Returns 0 on invalid arguments or when
 * B * max_blocks_per_seq exceeds 2^24.
 */
size_t mla_chunk_fp8_workspace_bytes(int T, int B, int H, int max_blocks_per_seq, int num_splits);

/*
 * mla_chunk_attend - attention of ragged chunks of new tokens over the paged latent
 * cache (prefill of a prompt in chunks, mixed batches): mla_decode_multi for any number
 * of tokens per sequence.  The queries of sequence b are tokens q_offsets[b] ..
 * q_offsets[b+1] - 1 of q; their own rows are already in the cache, as its last rows.
 * With n = q_offsets[b+1] - q_offsets[b], token j of them attends to the first
 * seq_lens[b] - (n - 1 - j) cached tokens.
 * q: bf16 [T,H,576]; q_offsets: int32 [B+1] on the device, non-decreasing, in 0..T;
 * out: bf16 [T,H,512]; lse: f32 [T,H].  Tokens before q_offsets[0] or at and past
 * q_offsets[B] are neither read nor written.  A token that sees no cached token gives
 * out = 0 and lse = -inf.  cache_dtype, cache, k_rope, block_scale, block_table,
 * seq_lens, softmax_scale, num_splits, the error bits (mla_get_device_error) and the
 * state after a timeout as for mla_decode; workspace as there too, of
 * mla_chunk_workspace_bytes or, for an fp8 cache, mla_chunk_fp8_workspace_bytes bytes (the
 * cache is widened to bf16 rows for the whole batch first; MLA_ERR_WORKSPACE_TOO_SMALL
 * with less).  A sequence whose offsets decrease or leave 0..T records
 * MLA_DEVERR_SEQ_TOO_LONG and its tokens are not written.  A cached row that is not finite
 * affects the tokens that see it only: where its score is NaN or +inf, out and lse are NaN;
 * where it is -inf, the row has probability 0 and out and lse are those without it, but the
 * columns of out in which the row is infinite may be NaN.
 * T >= 0 (0 is a no-op), T * H <= 2^30.
 */
mla_status_t mla_chunk_attend(const void *q, const int32_t *q_offsets, int T,
                              mla_cache_dtype_t cache_dtype, const void *cache,
                              const void *k_rope, const float *block_scale,
                              const int32_t *block_table, const int32_t *seq_lens, int B, int H,
                              int num_blocks, int max_blocks_per_seq, float softmax_scale,
                              void *out, float *lse, void *workspace, size_t workspace_bytes,
                              int num_splits, void *stream);

/*
 * mla_cache_weigh - the attention weight every cached token received, accumulated over
 * heads and queries (what mla_cache_evict ranks tokens by): for t < seq_lens[b]
 *     weight_out[b,t] = weight_in[b,t] + sum_{j,h} exp(scale q[j,h] . row_t - lse[j,h])
 * over the n tokens j of sequence b (q_offsets as for mla_chunk_attend) that see t, i.e.
 * t < seq_lens[b] - (n - 1 - j); lse is mla_decode's or mla_chunk_attend's for the same
 * queries and cache, so every query adds probabilities that sum to 1 per head.
 * q: bf16 [T,H,576]; lse: f32 [T,H] (+inf: the row adds nothing); bf16 cache;
 * weight_in, weight_out: f32 [B, 64*max_blocks_per_seq], slot order; weight_in may be
 * NULL (zeros) or weight_out itself, and must not overlap it otherwise.  Slots at and
 * past seq_lens[b] are not written.  The sum is fp32 in an order that depends on the
 * shapes alone.  Bad block ids, lengths and offsets are recorded for
 * mla_cache_get_error; a token whose block id is bad keeps its weight_in.  After
 * MLA_DEVERR_TIMEOUT there some slots are not written (in place they hold weight_in).
 * T >= 0, T * H <= 2^30.
 */
mla_status_t mla_cache_weigh(const void *q, const int32_t *q_offsets, int T, const float *lse,
                             const void *cache, const int32_t *block_table,
                             const int32_t *seq_lens, int B, int H, int num_blocks,
                             int max_blocks_per_seq, float softmax_scale, const float *weight_in,
                             float *weight_out, void *stream);

/*
 * mla_evict_workspace_bytes - bytes of device workspace mla_cache_evict needs.  Returns
 * 0 on invalid arguments.
 */
size_t mla_evict_workspace_bytes(int B, int max_blocks_per_seq);

/*
 * mla_cache_evict - cut every sequence of the bf16 cache to its budget and compact it.
 * Sequence b keeps n = min(max(keep[b], 0), seq_lens[b]) tokens: the first ones in the
 * order (protected before others, larger weight first, lower slot first), a slot being
 * protected when slot_pos < n_first or slot_pos > (largest slot_pos of the sequence) -
 * n_recent.  A NaN weight ranks as -inf.  Kept tokens in slots below n stay where they
 * are; the k-th kept token behind them moves into the k-th free slot below n, row,
 * weight and position.  Attention does not depend on the order of cached rows (every
 * key carries its own rotation), so the fewest rows move.
 * weight: f32, slot_pos: int32, both [B, 64*max_blocks_per_seq]; keep, seq_lens: int32
 * [B]; new_weight, new_pos, new_lens: the same shapes, for the compacted sequences:
 * slots n .. seq_lens[b] - 1 get weight 0 and position -1, slots past seq_lens[b] are
 * not written.  new_weight, new_pos and new_lens may each be the corresponding input
 * itself (and must not overlap the inputs otherwise).  The block table is not changed:
 * the blocks from ceil(n / 64) on are free for reuse.  No block may be in two rows of
 * the table, or twice in one, below the sequences' lengths (a shared prefix would be
 * compacted for all its sequences).
 * max_blocks_per_seq: at most 65536 (MLA_ERR_UNSUPPORTED above).
 * workspace: mla_evict_workspace_bytes(...), 256-byte aligned, zero-filled before its
 * first use, one call at a time; error bits by mla_get_device_error.  A token whose row
 * cannot move, because its source or destination slot has a bad block id
 * (MLA_DEVERR_BAD_BLOCK) or a wait gave up (MLA_DEVERR_TIMEOUT), stays where it was: its
 * slot, at or past n, has its row and in new_weight and new_pos its weight and position,
 * and the slot below n that waited for it keeps its old row and has weight 0 and position
 * -1.  All other tokens and new_lens are as in a call without errors.
 */
mla_status_t mla_cache_evict(const float *weight, const int32_t *slot_pos,
                             const int32_t *seq_lens, const int32_t *keep, int n_first,
                             int n_recent, const int32_t *block_table, int B, int num_blocks,
                             int max_blocks_per_seq, void *cache, float *new_weight,
                             int32_t *new_pos, int32_t *new_lens, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * mla_cache_get_error - device error bits of the cache writers and of mla_cache_weigh since the last
 * call; synchronises `stream` and clears them.  As for the absorption, the
 * word is one per device and process, shared by calls on every stream.
 * MLA_ERR_INVALID_ARG if err_bits is NULL.
 */
mla_status_t mla_cache_get_error(void *stream, uint32_t *err_bits);

/*
 * mla_set_wait_limit - bound, in SM clock cycles, of every wait inside the
 * decode, chunk, weight and eviction kernels launched from now on (process-wide; default about two
 * seconds of SM clock; cycles <= 0 restores the default).  Returns the
 * previous bound.  A wait that reaches the bound records MLA_DEVERR_TIMEOUT,
 * makes every role of the kernel leave its loop, lets copies in flight land
 * and exits; the outputs of that launch are then undefined (mla_decode and
 * mla_chunk_attend write them as out = 0, lse = NaN while the bit is set,
 * mla_cache_evict leaves every token whole), the context stays usable.  Meant for tests of that failure path and for diagnosis.
 */
long long mla_set_wait_limit(long long cycles);

/* mla_status_string - a static, human-readable name for a status code. */
const char *mla_status_string(mla_status_t status);

/*
 * mla_last_error_string - a static description of the CUDA failure behind the
 * last MLA_ERR_CUDA that a call made on this host thread returned ("no error"
 * before any).  The pointer stays valid until the library is unloaded.
 */
const char *mla_last_error_string(void);

/* mla_num_sms - streaming multiprocessors of the current device (0 on error). */
int mla_num_sms(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
