/*
 * fa.h -- C ABI of the GB300 (sm_103a) fused exact-attention forward library
 *         libfa_gb300.so.
 *
 * The operation (fa_fwd) is the tiled exact-attention forward pass:
 *
 *   O   = softmax(Q K^T * scale) V          per (batch, head), row-wise softmax
 *   LSE = log(sum_j exp(scale * q_i . k_j)) per query row (natural log)
 *
 * as defined on the pages "llm-infra-atlas / FlashAttention 01: IO awareness
 * and online softmax" (section 1 for the three-operation definition, section 3
 * for the tiled forward loop that emits O and LSE = m + log l, section 5 for
 * LSE's role in the backward pass) and "lumenova research-attention"
 * (section 01 for the shapes, section 03 for the per-row recurrence).  The
 * optional causal mask keeps key j for query row i iff j <= i.
 *
 * All functions have C linkage, never throw, never print and never abort the
 * process.  None of them allocates device memory.
 *
 * The first call on a device records per-device state in the library (the
 * kernels' shared-memory opt-in, the multiprocessor count and L2 size, and
 * for fa_fwd_splitkv_noalloc the device address of its fixed array).
 * Resetting a device (cudaDeviceReset) after this library has used it is not
 * supported: that state would be stale.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
typedef enum {
  FA_OK = 0,
  FA_ERR_NULL = 1,          /* a required pointer is NULL                                  */
  FA_ERR_ALIGN = 2,         /* a tensor base pointer is not 16-byte aligned                */
  FA_ERR_SHAPE = 3,         /* B, H, Nk <= 0, a negative Nq, or a size beyond the limits   */
  FA_ERR_HEADDIM = 4,       /* d is not 64 or 128                                          */
  FA_ERR_CAUSAL_SHAPE = 5,  /* causal = 1 with Nq != Nk                                    */
  FA_ERR_LAUNCH = 6,        /* the CUDA runtime refused the launch or a set-up call        */
  FA_ERR_DEVICE = 7,        /* the current device is not compute capability 10.3 (GB300)  */
  FA_ERR_TIMEOUT = 8,       /* a kernel wait gave up (reported by fa_fwd_status)           */
  FA_ERR_SCALE = 9,         /* scale is not a finite positive number                       */
  FA_ERR_POINTER = 10,      /* a tensor pointer is not device memory of the current device */
  FA_ERR_WORKSPACE = 11,    /* split-KV workspace missing or smaller than required         */
  FA_ERR_PAGE = 12,         /* a page index or sequence length outside the cache (reported by
                               fa_fwd_status: the values are known on the device alone)    */
  FA_ERR_STRIDE = 13        /* a stride is not a positive multiple of 8 elements           */
} fa_status;

/*
 * fa_fwd -- fused attention forward on `stream` (asynchronous; no host sync).
 *
 * q    [B, H, Nq, d] bf16, contiguous row-major (d fastest), device memory.
 * k, v [B, H, Nk, d] bf16, contiguous, device memory.
 * o    [B, H, Nq, d] bf16 output, contiguous, device memory; must not overlap
 *      q, k, v or lse.
 * lse  [B, H, Nq] fp32 output: natural-log log-sum-exp of the scaled logits of
 *      each query row (so that P = exp(scale * q.k - LSE)).
 * d    head dimension, 64 or 128.
 * scale  multiplies q.k before the softmax (1/sqrt(d) for standard attention);
 *        must be finite and > 0.
 * causal 0: every key is visible; 1: key j is visible to row i iff j <= i
 *        (requires Nq == Nk).
 *
 * Arithmetic: bf16 products accumulated in fp32 on the tensor cores, softmax
 * in fp32 (base-2 exponentials with log2(e) folded into the scale), the
 * probabilities rounded to bf16 for the P.V product, fp32 accumulation of O,
 * one division at the end by the row sum with the row's largest probability
 * counted as rounded for P.V (so a row dominated by one key returns that
 * key's V), O rounded to bf16 (nearest even).  LSE uses the exact fp32 sum.
 *
 * Ownership: the caller owns all five buffers; the library keeps no pointer
 * after the call returns and allocates nothing.
 * Errors: argument problems return a code before anything is launched and
 * nothing is written.  Nq == 0 is a successful no-op; q, o and lse may then be
 * NULL (k and v may not).  FA_ERR_LAUNCH is
 * returned if the launch itself fails, and by every call of a build whose
 * forward kernels did not get the register count their warpgroup register
 * split assumes (checked once per device, before any launch); faults during
 * execution surface, as usual for CUDA, at the next synchronising call on
 * the stream.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
           int Nk, int d, float scale, int causal, cudaStream_t stream);

/*
 * fa_fwd_window -- fa_fwd under a sliding-window mask (the "sliding" mask that
 * "llm-infra-atlas / FlashAttention 01", section 3, names beside "causal" in
 * the tiled loop; the window form and its alignment are this library's
 * reading, the pages give no formula).
 *
 * Key j is visible to query row i iff
 *     i + (Nk - Nq) - window_left  <=  j  <=  i + (Nk - Nq) + window_right,
 * i.e. the window is aligned so that its diagonal ends at the last query and
 * the last key (bottom-right alignment); -1 leaves that side unbounded.
 * (-1, 0) is causal attention for any Nq and Nk; (-1, -1) is no mask.  A query
 * row that sees no key gets O = 0 and LSE = -inf.
 * Arguments otherwise as fa_fwd (no causal flag, Nq and Nk independent);
 * window_left or window_right below -1 returns FA_ERR_SHAPE.
 */
int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                  int Nk, int d, float scale, int window_left, int window_right, cudaStream_t stream);

/*
 * fa_fwd_splitkv -- the same operation as fa_fwd, with each query tile's K/V
 * range cut into n_splits slices processed by separate CTAs, for shapes whose
 * B * H * ceil(Nq / 256) CTAs would leave most of the GPU idle.
 *
 * Each slice s produces a partial result for its rows: O_s normalised by its
 * own row sum, and L_s = log2 of that row sum in base-2 scaled-logit units.
 * A second kernel on the same stream merges the slices by the rule under which
 * the online-softmax state (m, l, O) is insensitive to block order ("llm-infra-
 * atlas / FlashAttention 01", section 2).  It is launched as a programmatic
 * dependent of the first (it may be scheduled while the first one's last CTAs
 * run and waits on the device for its completion), so stream order and the
 * results are those of two plain launches:
 *   L = log2 sum_s 2^L_s,   O = sum_s 2^(L_s - L) O_s,   LSE = L * ln 2.
 * At d = 64 a CTA takes one query tile instead of two when the CTAs of tile
 * pairs would fill under half of the multiprocessors or more than all of
 * them; the slices, and so the results, are the same either way.
 *
 * Arguments as in fa_fwd, plus:
 * n_splits   requested slices, 1..64; the call uses ceil(n_kv / ceil(n_kv /
 *            n_splits)) of them, n_kv = ceil(Nk / 128).  With one slice this is
 *            exactly fa_fwd and the workspace is not touched.
 * workspace  device memory of at least fa_splitkv_workspace_bytes() bytes,
 *            16-byte aligned, owned by the caller, not read before it is
 *            written; it must not be used by anything else until the call's
 *            kernels have finished on `stream`.
 * Errors as fa_fwd, plus FA_ERR_SHAPE for n_splits outside 1..64 and
 * FA_ERR_WORKSPACE for a missing or short workspace.
 */
int fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                   int Nk, int d, float scale, int causal, int n_splits, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes fa_fwd_splitkv needs for these sizes (0 for invalid sizes):
 * fp32 partial O [splits, B*H*Nq, d] followed by fp32 partial L [splits, B*H*Nq]. */
size_t fa_splitkv_workspace_bytes(int B, int H, int Nq, int Nk, int d, int n_splits);

/* Suggested n_splits for the current device: 1 when B * H * ceil(Nq / 256)
 * CTAs already cover its multiprocessors, otherwise enough slices (at most 16,
 * each of at least two K/V tiles) to fill them about once. */
int fa_splitkv_heuristic(int B, int H, int Nq, int Nk, int d, int causal);

/*
 * fa_bwd -- attention backward pass by recomputation from the forward's LSE
 * ("llm-infra-atlas / FlashAttention 01", section 5):
 *   P = exp(scale * Q K^T - LSE),  dV = P^T dO,  dP = dO V^T,
 *   D = rowsum(dO * O),  dS = P * (dP - D),  dQ = scale * dS K,  dK = scale * dS^T Q.
 *
 * q, o, dout, dq  [B, H, Nq, d] bf16;  k, v, dk, dv  [B, H, Nk, d] bf16;
 * lse [B, H, Nq] fp32 as written by fa_fwd (natural log).  All contiguous,
 * 16-byte aligned device memory of the current device; outputs must not
 * overlap inputs.  causal as in fa_fwd (Nq == Nk).  Nq and Nk must be > 0.
 * workspace: device memory of at least fa_bwd_workspace_bytes(B, H, Nq)
 * bytes, owned by the caller (fp32 L = LSE * log2(e) and D per query, padded
 * to whole 128-row tiles); not read before it is written.
 * Two kernels run on `stream`: one per 128-row query tile for dQ (and L, D),
 * then one per 128-key tile for dK and dV; no atomics, so the result does not
 * depend on scheduling.  Errors as fa_fwd, plus FA_ERR_WORKSPACE.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
           void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
           void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd_window -- fa_bwd under the sliding-window mask of fa_fwd_window (key j
 * kept for query row i iff i + (Nk - Nq) - window_left <= j <= i + (Nk - Nq) +
 * window_right; -1 leaves that side open, so (-1, 0) is the causal mask aligned
 * bottom-right, for any Nq and Nk).  o and lse must come from fa_fwd_window
 * with the same window: a row that keeps no key has lse = -inf and o = 0 there,
 * and its dQ is written as 0; a key that no row keeps gets dK = dV = 0.
 * Each kernel visits only the tiles its window reaches.
 * Arguments, workspace and errors as fa_bwd (no causal argument); a bound
 * below -1 is FA_ERR_SHAPE.
 */
int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int window_left,
                  int window_right, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes fa_bwd and fa_bwd_window need (0 for invalid sizes). */
size_t fa_bwd_workspace_bytes(int B, int H, int Nq);

/*
 * fa_rope -- rotary positions of queries and keys, and their backward.
 *
 * The pair (x0, x1) number i of a head's first `rot` elements, at position p,
 * becomes
 *     mag * (x0 cos a - x1 sin a,  x1 cos a + x0 sin a),   a = p * inv_freq[i],
 * with x0 = x[i], x1 = x[i + rot / 2] (interleaved = 0) or x0 = x[2i],
 * x1 = x[2i + 1] (interleaved = 1); elements from rot on are copied unscaled.
 * backward = 1 applies the transpose (the gradient of the above: sin negated,
 * the same mag).
 *
 * q, q_out    bf16 [B, H, N, d];  k, k_out bf16 [B, Hk, N, d], Hk = 0: no k.
 *             An output may be its own input (same pointer, same strides);
 *             otherwise it must not overlap an input.
 * inv_freq    fp64 [rot / 2], radians per position (any scaling of long
 *             contexts is in these values and in mag).  A position p multiplies
 *             a 64-bit fraction of a turn: the angle is off by at most
 *             |p| (2^-65 + |inv_freq| 2^-72) turns, then fp32's relative error
 *             (sine and cosine too, near their zeros as elsewhere).  Any 32-bit
 *             position is far below a bf16 rounding, and so are offsets up to
 *             2^48 in size; past that the angle fades out.  A value of NaN or
 *             infinity makes its pair NaN.
 * positions   int32 [B, N] (position_stride, >= N, int32s from one sequence to the
 *             next) or one row for all (position_stride 0); NULL: position
 *             = offset + row.  offset is added in both cases.
 * strides     host array of 12: batch, head and row strides, in elements, of q, k,
 *             q_out and k_out (d is contiguous); multiples of 8, outputs' > 0 (a
 *             dimension of size 1 may name any valid stride).  NULL: all
 *             contiguous.  Read during the call only.
 * d           64 or 128;  rot a multiple of 16, 16..d;  mag finite.
 * Products and sums in fp32, one rounding to bf16 (nearest even).
 * Asynchronous on `stream`; N == 0 is a successful no-op.  Errors as fa_fwd, plus
 * FA_ERR_STRIDE.
 */
int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const int* positions,
            long long position_stride, long long offset, const long long* strides, int B, int H, int Hk, int N, int d,
            int rot, float mag, int interleaved, int backward, cudaStream_t stream);

/*
 * The paged K/V cache of fa_kv_append, fa_fwd_paged and fa_fwd_prefix.
 *
 * k_cache, v_cache  bf16 [n_pages, Hk, page_size, d] views with free page, head
 *                   and token strides (elements, multiples of 8, > 0; d contiguous),
 *                   so token-major pages [n_pages, page_size, Hk, d] are the same
 *                   cache with other strides.  page_size 16, 32, 64, 128 or 256.
 * block_table       int32 [B, max_pages]: entry i of a sequence names the page of
 *                   its tokens [i * page_size, (i + 1) * page_size).  Entries
 *                   past the sequence's length, or wholly below its window, are
 *                   not read.
 * seq_lens          int32 [B]: tokens of each sequence in the cache, the new ones
 *                   of this step INCLUDED (the same values serve the append and
 *                   the attention of a step).  <= 0: an empty entry.
 * new_lens          int32 [B]: how many of the T new rows each sequence has
 *                   (clamped to 0..T), or NULL: T each.  Row t < new_lens[b] is
 *                   the token at own position seq_lens[b] - new_lens[b] + t;
 *                   rows past it are padding, and so are rows whose position
 *                   would be negative.
 * A page index that is needed and lies outside [0, n_pages), or a length past
 * max_pages * page_size, raises bit 1 of the status word (fa_fwd_status:
 * FA_ERR_PAGE): the append skips the token, the attention reads zeros for the
 * page or stops at the table's end; memory outside the cache is never touched.
 */

/*
 * fa_kv_append -- put the new tokens' keys (rotated as by fa_rope) and values
 * into their cache slots, and rotate their queries, in one kernel.
 *
 * q, q_out  bf16 [B, H, T, d] (H = 0: keys and values only);  k, v bf16
 *           [B, Hk, T, d].  Padding rows are neither read nor written.
 * strides   host array of 18: batch, head and row strides of q, k and v, the same
 *           of q_out, then page, head and token strides of k_cache and v_cache.
 * rot       0 (nothing turns; inv_freq may be NULL) or as in fa_rope; position =
 *           offset + own position (a shared prefix's length goes in offset).
 * q_out may be q itself (same pointer, same strides); no other output may overlap
 * an input.  Two tokens of one call must not share a slot.  Cache slots of other
 * tokens stay as they are.  Errors as fa_rope; T == 0 is a successful no-op.
 * The first call on a device looks up the status word's address there: make
 * that first call before any stream capture.
 */
int fa_kv_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                 const double* inv_freq, const int* block_table, const int* seq_lens, const int* new_lens,
                 const long long* strides, int B, int H, int Hk, int T, int d, int rot, int n_pages, int page_size,
                 int max_pages, long long offset, float mag, int interleaved, cudaStream_t stream);

/*
 * fa_fwd_paged -- O and LSE (as fa_fwd) of the new tokens' queries over their
 * sequences' cached keys, grouped heads included: query head h reads K/V head
 * h / (H / Hk).
 *
 * q, o  bf16 [B, H, T, d] contiguous;  lse fp32 [B, H, T].  The outputs must not
 *       overlap each other or any input.
 * The token at own position pos sees own keys j with
 *     pos - window_left <= j <= pos + window_right,   0 <= j < seq_lens[b],
 * -1 leaving a side open: (-1, 0) is causal, (-1, -1) every cached key (an
 * encoder's states of a length per sequence; with more new rows than keys the
 * first rows' positions are negative, and a window open or wide enough to the
 * right still reaches keys from there).  Rows from new_lens[b] on and rows that
 * see no key get O = 0, LSE = -inf.  Slots outside every row's window or past the
 * length may hold anything, NaN included; a key that some rows of a sequence
 * see and others do not must be finite.
 * strides    host array of 6: page, head and token strides of k_cache, v_cache.
 * workspace  fa_paged_workspace_bytes(B, H, Hk, T, d, 0) bytes, 16-byte
 *            aligned, not read before it is written, used by nothing else until
 *            the call's kernels have finished (two calls that may overlap, or two
 *            captured graphs that may, need one each).
 * Lengths are read on the device, so a captured call may be replayed as they
 * grow (within max_pages).  No atomics order the sums: results repeat bit
 * for bit on one GPU.  Errors as fa_fwd, plus FA_ERR_STRIDE and FA_ERR_WORKSPACE;
 * T == 0 is a successful no-op.  First call before any stream capture, as
 * fa_kv_append.
 */
int fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, const int* block_table,
                 const int* seq_lens, const int* new_lens, const long long* strides, int B, int H, int Hk, int T, int d,
                 int n_pages, int page_size, int max_pages, float scale, int window_left, int window_right,
                 void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_fwd_prefix -- fa_fwd_paged (causal) for a batch whose sequences all begin
 * with the same prefix_len tokens: the prefix's K and V are read once for the
 * batch, its part and each sequence's own are joined as in fa_fwd_splitkv.
 *
 * prefix_pages  int32 [ceil(prefix_len / page_size)]: the prefix's pages.
 * prefix_len    > 0, known to the host.
 * block_table and seq_lens describe the sequences' OWN tokens, after the prefix;
 * every row that holds a token sees the whole prefix and its own keys up to
 * itself.  seq_lens[b] <= 0: an empty entry (O = 0, LSE = -inf).
 * workspace     fa_paged_workspace_bytes(B, H, Hk, T, d, prefix_len) bytes.
 * Otherwise as fa_fwd_paged.
 */
int fa_fwd_prefix(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                  const int* prefix_pages, int prefix_len, const int* block_table, const int* seq_lens,
                  const int* new_lens, const long long* strides, int B, int H, int Hk, int T, int d, int n_pages,
                  int page_size, int max_pages, float scale, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/* Workspace bytes of fa_fwd_paged (prefix_len 0) and fa_fwd_prefix on the
 * current device (0 for invalid sizes); it does not depend on the lengths. */
size_t fa_paged_workspace_bytes(int B, int H, int Hk, int T, int d, int prefix_len);

/* Size of the fixed device array fa_fwd_splitkv_noalloc works in. */
#define FA_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * fa_fwd_splitkv_noalloc -- fa_fwd_splitkv without a caller workspace and
 * without any allocation: the slice buffers live in a fixed 16 MiB array
 * (FA_NOALLOC_SCRATCH_BYTES) in the library's own device memory.  The pages
 * describe no counterpart; this entry point exists for callers that cannot
 * allocate device memory themselves, for instance code running inside a host
 * framework that owns the whole device memory pool, or a latency path where a
 * cudaMalloc and the synchronisation it implies are not allowed.
 *
 * Arguments and results as fa_fwd_splitkv.  Sizes whose workspace
 * (fa_splitkv_workspace_bytes) exceeds FA_NOALLOC_SCRATCH_BYTES return
 * FA_ERR_WORKSPACE before anything is launched.  No cudaMalloc, cudaFree or
 * other allocating call is made.
 * Every GPU that loads the library holds the array until the process exits.
 * The first call on a device looks up the array's device address there (with
 * that device current); make that first call before any stream capture.
 * All calls share the one array, which keeps whatever the last call left in
 * it: calls whose kernels overlap on the GPU (other streams, other host
 * threads) race on it and must be serialised by the caller.  Nothing has to
 * be cleared between calls: every value the merge reads is written earlier in
 * the same call.
 */
int fa_fwd_splitkv_noalloc(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                           int Nq, int Nk, int d, float scale, int causal, int n_splits, cudaStream_t stream);

/* Bits of the device status word. */
#define FA_STATUS_TIMEOUT 1u /* a bounded wait gave up; bits 8.. name the role   */
#define FA_STATUS_PAGE 2u    /* a page index or length outside the cache or table */

/* Human-readable text for a status code (static storage, never NULL). */
const char* fa_strerror(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
int fa_version(void);

/*
 * fa_fwd_status -- synchronise `stream`, then report whether any kernel of
 * this library (forward, split-KV, backward, paged and shared-prefix attention)
 * on the current device gave up on a wait (FA_ERR_TIMEOUT) since the last
 * clear.  Every wait inside the kernels is bounded (about 2 s); a wait that
 * runs out records the failing role in the device status word (bit 0, and bits
 * 8.. = 1 softmax/compute, 2 producer, 4 MMA issuer, 8 epilogue, 32 loader of Q;
 * 16: the CTA's shared memory did not begin on a 1024-byte boundary, and it
 * computed nothing), the CTA drains its in-flight copies and MMAs, frees its
 * tensor memory and exits.  *detail (optional) receives the raw
 * status word.  clear != 0 resets the word.  Returns FA_OK, FA_ERR_TIMEOUT,
 * FA_ERR_PAGE (bit 1 alone: a page index or sequence length that the paged
 * calls met lies outside the cache or its table), or FA_ERR_LAUNCH if
 * synchronisation failed.
 */
int fa_fwd_status(cudaStream_t stream, unsigned int* detail, int clear);

/*
 * fa_probe_exp2 -- measure how many 2^x results per SM clock cycle the current
 * device produces (median over the SMs of one CTA per SM running independent
 * exp2 chains).  Not an operation of the pages: method 0 times ex2.approx on
 * the special-function unit, the denominator of the forward kernel's
 * exponential-unit roofline; method 1 times a cubic polynomial on the FMA and
 * integer pipes, the kind of offload that the page "pinghaoyang FlashAttention
 * 1-4 guide" (FA4 section, emulated exponential) describes for Blackwell.
 *
 * method      0 or 1 (anything else: FA_ERR_SHAPE).
 * per_clk_sm  host pointer receiving the rate.
 * stream      the probe runs on it; the call synchronises the stream.
 * Uses no caller memory.  Returns FA_ERR_NULL, FA_ERR_SHAPE, FA_ERR_DEVICE
 * (not compute capability 10.3) or FA_ERR_LAUNCH; the value is written only
 * on FA_OK.
 */
int fa_probe_exp2(int method, double* per_clk_sm, cudaStream_t stream);

/*
 * fa_selftest_wait -- exercise the bounded wait that every kernel of this
 * library uses, without any fault: one CTA waits on an mbarrier phase that
 * nothing completes.  Not an operation of the pages.
 *
 * mode 0: the wait must give up when its time limit (about 2 s) runs out;
 * mode 1: another warp raises the CTA's abort flag after about 1 ms and the
 *         wait must give up on it at once.
 * word     receives the self-test's status word: bit 0 set when the wait gave
 *          up; bits 8.. = 1 (time limit) or 2 (abort flag).
 * wait_ns  receives how long the wait lasted, in nanoseconds.
 * Synchronises `stream`; the device status word of the other kernels is not
 * touched.  Returns FA_ERR_NULL, FA_ERR_SHAPE (mode), FA_ERR_DEVICE or
 * FA_ERR_LAUNCH; the outputs are written only on FA_OK.
 */
int fa_selftest_wait(int mode, unsigned int* word, unsigned long long* wait_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
