/*
 * fattn.h -- C-ABI of libfattn: exact tiled scaled-dot-product attention
 * (FlashAttention forward and backward) for NVIDIA GB300 (sm_103a).
 *
 * The operation, for every (batch b, head h) independently
 * ("FlashAttention tiles exact softmax without materializing the score
 * matrix", opening equations; "tm_flash_attention_math", "What we must
 * compute, and why storage is the problem"):
 *
 *     S = scale * Q K^T            (N x N, never stored)
 *     P = softmax(S) row by row    (causal: key j visible to query i iff j <= i)
 *     O = P V
 *     LSE_i = m_i + ln l_i = ln sum_j exp(S_ij)
 *
 * LSE is the one per-row statistic the backward pass keeps ("Decoding flash
 * attention", "The backward pass"); the backward recomputes P = exp(S - LSE)
 * tile by tile and returns dQ, dK, dV of a loss whose gradient w.r.t. O is dO.
 *
 * Layout.  q, k, v, o, dout, dq, dk, dv are DEVICE pointers to contiguous
 * bf16 tensors [B, H, N, d] (row-major, d innermost).  lse is a DEVICE
 * pointer to fp32 [B, H, N].  Every pointer must be 16-byte aligned.
 * d must be 64 or 128.  N >= 1, B >= 1, H >= 1, B*H*N < 2^31.
 * scale must be finite and > 0 (every workload here uses 1/sqrt(d)).
 *
 * Ownership.  The caller allocates and owns every buffer; the library keeps
 * no per-call state and never frees caller memory.
 *
 * Streams and errors.  Calls are asynchronous on `stream` (a cudaStream_t;
 * NULL is the legacy default stream).  Arguments are validated before
 * anything is launched: a bad argument returns a non-zero status and
 * launches nothing.  A launch failure returns FATTN_ERR_CUDA.  Faults during
 * execution surface at the caller's next synchronisation, as usual in CUDA.
 * Every wait inside a kernel is bounded; a wait that runs out records a code
 * in a device error word and the kernel finishes without hanging.  The word is
 * read with fattn_device_error, which returns FATTN_ERR_TIMEOUT while it is
 * set.  With the environment variable FATTN_DEBUG set to a non-zero value
 * (read once per process), every entry point that launches work also
 * synchronises `stream` after enqueueing (not while the stream is being
 * captured into a graph) and returns FATTN_ERR_TIMEOUT if the word is set.
 *
 * The library remembers a few facts per device on first use (kernel
 * attributes, the SM count and L2 size, the error word's address); the
 * entries are tied to the device's current context and are set up again after
 * cudaDeviceReset.
 *
 * The device must be compute capability 10.3 (sm_103a), else
 * FATTN_ERR_UNSUPPORTED.
 */
#ifndef FATTN_H_
#define FATTN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FATTN_OK = 0,
  FATTN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad scale */
  FATTN_ERR_UNSUPPORTED = 2, /* d not in {64,128}, or the device is not sm_103 */
  FATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call or a launch failed */
  FATTN_ERR_WORKSPACE = 4,   /* workspace missing or too small */
  FATTN_ERR_TIMEOUT = 5      /* a bounded in-kernel wait ran out (fattn_device_error) */
} fattn_status;

/* Forward pass.  Writes o [B,H,N,d] bf16 and lse [B,H,N] fp32 (natural log,
 * in units of scaled scores).  The online-softmax state (running max m,
 * running sum l, unnormalised accumulator o~, rescale alpha = exp(m_old - m_new))
 * is carried across 128-key tiles ("tm_flash_attention_math", "The block-wise
 * update, and the full algorithm"); key tiles wholly above the causal
 * diagonal are skipped and only diagonal-crossing or ragged tiles are masked
 * element by element (page 1, "Causal masking fits inside the tiled
 * computation"). */
int fattn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int N, int d, float scale, int causal, void* stream);

/* fattn_fwd plus tile instrumentation: when tile_counts (DEVICE pointer to 3
 * unsigned 64-bit counters, 8-byte aligned) is not NULL, the kernel ADDS the
 * number of (128-row query tile, 128-key tile) pairs it processed without
 * masks [0], processed with element masks [1], and skipped as wholly above
 * the causal diagonal [2] (page 1, "Causal masking fits inside the tiled
 * computation": tiles beyond the permitted region are skipped, the ones on
 * the boundary masked).  The caller zeroes the counters.  The counters are an
 * argument of the call rather than library state set beforehand, so that
 * calls from several threads or streams, and calls captured into graphs,
 * each count into their own buffer. */
int fattn_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, unsigned long long* tile_counts,
                 void* stream);

/* Bytes of device workspace fattn_bwd needs: an fp32 dQ accumulator
 * [B,H,N,d] and the fp32 row statistic D [B,H,N] (256-byte aligned parts).
 * No passage of the pages: it sizes the scratch of the backward formulas
 * below.  Returns 0 for B, H, N < 1 or d not in {64, 128}. */
size_t fattn_bwd_workspace_bytes(int B, int H, int N, int d);

/* Backward pass.  Inputs q, k, v, o, lse as produced by fattn_fwd and dout
 * = dL/dO; outputs dq, dk, dv [B,H,N,d] bf16.  The pages give no gradient
 * formulas; the calculus of the definition is used: D_i = sum_c dO_ic O_ic,
 * P = exp(S - LSE), dV = P^T dO, dP = dO V^T, dS = P o (dP - D),
 * dQ = scale dS K, dK = scale dS^T Q ("FlashAttention tiles exact softmax
 * without materializing the score matrix", "Backward computation can trade
 * recomputation for stored intermediates").
 * workspace: DEVICE memory of at least fattn_bwd_workspace_bytes(B,H,N,d)
 * bytes, 256-byte aligned, owned by the caller; its contents on entry do not
 * matter and are overwritten.  Too small or misaligned -> FATTN_ERR_WORKSPACE,
 * nothing launched.  NULL -> the call takes the scratch from the CUDA
 * stream-ordered allocator: cudaMallocAsync on `stream` before its kernels and
 * cudaFreeAsync on `stream` after them (workspace_bytes is then ignored); an
 * allocation failure returns FATTN_ERR_CUDA and launches nothing.  The
 * device's default memory pool keeps nothing across synchronisations unless
 * its release threshold is raised, so each such call maps its scratch anew;
 * a program that calls this repeatedly avoids that by passing a workspace. */
int fattn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
              const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
              float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

/* fattn_bwd plus phase timing: when phase_events is not NULL it points to 4
 * cudaEvent_t handles (created by the caller) that are recorded on `stream`
 * before the preprocess kernel, before the main kernel, after the main
 * kernel and after the dQ convert kernel. */
int fattn_bwd_ex(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, void* workspace, size_t workspace_bytes,
                 void* const* phase_events, void* stream);

/* Variable-length batches (padded attention without the padding: "Causal
 * masking fits inside the tiled computation" on page "FlashAttention tiles
 * exact softmax without materializing the score matrix" masks positions
 * inside a tile; here each sequence simply ends where its length says).
 * B sequences of lengths n_b = cu_seqlens[b+1] - cu_seqlens[b] are packed
 * head-major: q, k, v, o, dout, dq, dk, dv are DEVICE pointers to bf16
 * [H, total, d] (sequence b at rows [cu_seqlens[b], cu_seqlens[b+1]) of every
 * head) and lse is fp32 [H, total].  Each sequence is its own attention
 * problem: its queries see only its own keys (and, causal, only keys at or
 * before their own position in the sequence).
 * cu_seqlens: DEVICE int32 array of B+1 non-decreasing offsets, cu_seqlens[0]
 * = 0 and cu_seqlens[B] = total; max_seqlen >= every n_b (the grid is sized by
 * it); total is passed by the caller because the host cannot read device
 * memory without a synchronisation.  Entries are checked on the device: a
 * sequence that is out of range, decreasing or longer than max_seqlen is
 * skipped and reported through the device error word (code 0x140 forward,
 * 0x240 backward).  Empty sequences are allowed; total == 0 launches nothing.
 * Returns as fattn_fwd; tile counters are not available. */
int fattn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                     const int* cu_seqlens, int B, int H, int max_seqlen, int total, int d,
                     float scale, int causal, void* stream);

/* Backward of fattn_fwd_varlen ("Backward computation can trade recomputation
 * for stored intermediates" on page 1, per sequence): the layouts above;
 * workspace of at least fattn_bwd_workspace_bytes(1, H, total, d) bytes, or
 * NULL for stream-ordered scratch as in fattn_bwd.  Returns as fattn_bwd. */
int fattn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                     const float* lse, const void* dout, void* dq, void* dk, void* dv,
                     const int* cu_seqlens, int B, int H, int max_seqlen, int total, int d,
                     float scale, int causal, void* workspace, size_t workspace_bytes,
                     void* stream);

/* Split-KV attention for a few queries against many keys (decoding).
 * q [B,H,Nq,d], k, v [B,H,Nkv,d] bf16, 1 <= Nq <= Nkv; outputs o [B,H,Nq,d]
 * bf16 and lse [B,H,Nq] fp32, all DEVICE pointers, 16-byte aligned.  The
 * queries are the LAST Nq positions of the sequence: with causal, query i
 * sees keys j <= Nkv - Nq + i (Nq == Nkv is fattn_fwd's causal mask).
 * The 128-key tiles are cut into key ranges, one per CTA of the forward
 * kernel, each leaving its range's normalised result and log-sum-exp in the
 * workspace; a merge kernel combines them (fattn_merge_partials).  This is
 * the block-wise recurrence of "tm_flash_attention_math" ("The block-wise
 * update, and the full algorithm"), with whole blocks' states merged, which
 * the page's "Proof of exactness" allows in any order.
 * n_splits: 0 = automatic (about ten waves of CTAs, at least four tiles per
 * range), else the requested number
 * of ranges (capped at one per tile; the count used is fattn_decode_splits).
 * workspace: DEVICE memory of fattn_decode_workspace_bytes(...) bytes,
 * 256-byte aligned, owned by the caller.  Returns FATTN_OK,
 * FATTN_ERR_INVALID_ARG, FATTN_ERR_UNSUPPORTED, FATTN_ERR_WORKSPACE or
 * FATTN_ERR_CUDA; launches nothing on an argument error. */
int fattn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int Nq, int Nkv, int d, float scale, int causal, int n_splits, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Number of key ranges fattn_decode uses for these arguments on the current
 * device (the automatic count follows its SM count); 0 if invalid.  A sizing
 * helper of fattn_decode; no passage of its own. */
int fattn_decode_splits(int B, int H, int Nq, int Nkv, int d, int n_splits);

/* Workspace bytes fattn_decode needs on the current device: S x B*H*Nq x
 * (d + 1) fp32 with S = fattn_decode_splits(...); 0 if invalid.  A sizing
 * helper of fattn_decode; no passage of its own. */
size_t fattn_decode_workspace_bytes(int B, int H, int Nq, int Nkv, int d, int n_splits);

/* Merge of partial results over disjoint key ranges ("tm_flash_attention_math",
 * "Proof of exactness": block states combine in any order): o_part [S, rows, d] and
 * lse_part [S, rows] fp32 (range s's normalised output and log-sum-exp; a
 * range in which a row saw no key has lse = -inf) -> lse = log sum_s
 * exp(lse_s), o = sum_s exp(lse_s - lse) o_s as bf16 [rows, d]; a row with
 * every lse_s = -inf gets o = 0 and lse = -inf.  DEVICE pointers, 16-byte
 * aligned; d in {64, 128}. */
int fattn_merge_partials(const float* o_part, const float* lse_part, int n_splits, long long rows,
                         int d, void* o, float* lse, void* stream);

/* Row-wise softmax with the online normaliser: y[r, :] = exp(x[r, :] - m_r) / l_r
 * with m_r the row maximum and l_r = sum exp(x[r, :] - m_r), formed in one
 * sweep by the (m, l) recurrence of "FlashAttention tiles exact softmax
 * without materializing the score matrix" ("The online softmax recurrence").
 * x, y: DEVICE fp32 [rows, cols], row-major, 16-byte aligned (y may equal x);
 * lse: DEVICE fp32 [rows] receiving m_r + ln l_r, or NULL.  A row whose values
 * are all -inf gets y = 0 and lse = -inf.  Rows of up to 49152 values are read
 * from HBM once; longer rows twice.  Returns FATTN_OK, FATTN_ERR_INVALID_ARG,
 * FATTN_ERR_UNSUPPORTED or FATTN_ERR_CUDA. */
int fattn_softmax_rows(const float* x, float* y, float* lse, long long rows, int cols,
                       void* stream);

/* Size of the device array that fattn_bwd_noalloc uses as its workspace. */
#define FATTN_NOALLOC_SCRATCH_BYTES (64u << 20)

/* fattn_bwd without a caller-provided workspace, for callers that cannot
 * allocate device memory where they run the backward (a plugin inside a host
 * program that owns the CUDA allocator, or a runtime that reserves its whole
 * memory budget up front).  The pages have no counterpart to this entry
 * point; it is a packaging variant of fattn_bwd.
 * The workspace is a fixed device array of FATTN_NOALLOC_SCRATCH_BYTES that
 * every GPU loading the library holds until exit; nothing is allocated or
 * freed.  Problems with fattn_bwd_workspace_bytes(B,H,N,d) larger than that
 * return FATTN_ERR_WORKSPACE and launch nothing.  All calls share the array:
 * calls that overlap on the GPU race on it.  The first call on a device looks
 * up the array's device address, so it should come before any stream capture.
 * Arguments, layouts, results and other errors are those of fattn_bwd. */
int fattn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                      const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                      int H, int N, int d, float scale, int causal, void* stream);

/* Sizing helper of fattn_fwd_bwd_host (no passage of its own).
 * Bytes of DEVICE workspace fattn_fwd_bwd_host needs: three staging slots,
 * each holding Q, K, V, dO, O, dQ, dK, dV and LSE of one chunk of heads plus
 * that chunk's backward workspace.  heads_per_chunk = 0 selects the library's
 * chunk size for the current device (the same one fattn_fwd_bwd_host picks
 * for 0).  Returns 0 for invalid sizes. */
size_t fattn_fwd_bwd_host_workspace_bytes(int B, int H, int N, int d, int heads_per_chunk);

/* Forward and backward of tensors in HOST memory: the same results as
 * fattn_fwd followed by fattn_bwd.  q, k, v, dout are HOST pointers to bf16
 * [B,H,N,d]; o, dq, dk, dv HOST pointers to bf16 [B,H,N,d] and lse to fp32
 * [B,H,N], all written by the call.  Every (b, h) slice is an independent
 * problem ("FlashAttention tiles exact softmax without materializing the score
 * matrix", opening equations), so the slices move through `workspace` (DEVICE,
 * 256-byte aligned, fattn_fwd_bwd_host_workspace_bytes large) in chunks of
 * heads_per_chunk consecutive slices (0 = the library's choice; the first
 * chunk is half as large so that the kernels start sooner), and the copy in of
 * one chunk, the kernels of the previous one and the copy out of the one
 * before run at the same time on three streams the library keeps per device.  Asynchronous on `stream` like the other entry points: the host
 * buffers must stay untouched until `stream` has reached this call's end.
 * The copies overlap only when the host buffers are page-locked
 * (cudaHostAlloc or cudaHostRegister); pageable memory gives the same results
 * with the copies serialised.  Calls from several host threads are
 * serialised while they enqueue.  Errors: those of fattn_fwd and fattn_bwd;
 * FATTN_ERR_WORKSPACE for a missing, misaligned or short workspace. */
int fattn_fwd_bwd_host(const void* q, const void* k, const void* v, const void* dout, void* o,
                       float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                       float scale, int causal, int heads_per_chunk, void* workspace,
                       size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ key/value cache
 *
 * A paged cache of keys and values in 8 or 4 bits, its writer, its reader and the
 * attention over it, for serving: the keys and values of `fattn_decode` kept
 * from step to step at half the bytes or 0.28 of them, with grouped heads.  The
 * pages have no counterpart to the storage; the attention is their recurrence
 * over it.
 *
 * The pool, 8 bits.  k and v hold num_blocks blocks of block_size tokens for each of H
 * key/value heads, [num_blocks, H, block_size, d], one 8-bit floating code per
 * value; k_scale and v_scale hold one fp32 scale per (block, head),
 * [num_blocks, H].  The value that code c of a block stands for is scale * c.
 * All four are DEVICE pointers owned by the caller, contiguous, the codes
 * 16-byte aligned and the scales 4-byte aligned (so one layer's part of a larger
 * array will do).  block_size is 16, 32, 64 or 128, d 64 or 128, num_blocks x H
 * below 2^31.
 * fattn_cache_append writes powers of two as scales; the reader and the
 * attention take any positive normal fp32.  Where value scales of one sequence
 * and head differ by more than 2^60 (a block of zeros has the smallest one,
 * 2^-100), the attention takes the smaller as 2^-60 of the larger.
 *
 * The pool, 4 bits.  k and v hold two codes a byte, [num_blocks, H, block_size,
 * d / 2], the even channel in the low half; k_scale and v_scale hold an e5m2 scale
 * for every 16 neighbouring channels of a token, bytes [num_blocks, H, block_size,
 * d / 16].  The value that code c (0 to 15) stands for is (c - 8) * scale.  All four
 * are 16-byte aligned.  Every token has its own scales, so nothing that is written
 * later changes what is there.  The reader takes any scale; for the attention and
 * the keys' weights its magnitude is at most 7168, the largest that append writes (a
 * row that sees a larger one, an infinity or a NaN gets values of no meaning, and so
 * do the weights that come of it; other heads' and sequences' do not). */
typedef enum {
  FATTN_CACHE_E4M3 = 0, /* 4 exponent, 3 mantissa bits, largest value 448, no infinities */
  FATTN_CACHE_E5M2 = 1, /* 5 exponent, 2 mantissa bits, largest value 57344 */
  FATTN_CACHE_INT4 = 4  /* whole numbers from -8 to 7, a scale for 16 channels of a token */
} fattn_cache_format;

typedef struct {
  void* k;
  void* v;
  void* k_scale; /* float; 4 bits: e5m2 bytes */
  void* v_scale;
  int num_blocks;
  int H; /* key/value heads */
  int block_size;
  int d;
  int format; /* fattn_cache_format */
} fattn_cache;

/* Which tokens a call works on: the LAST n_b = cu_seqlens[b+1] - cu_seqlens[b]
 * tokens of each of B sequences, packed token by token into tensors of `total`
 * rows (sequence b at rows [cu_seqlens[b], cu_seqlens[b+1])).
 * lens[b] is the length of sequence b including those tokens; its token p is
 * row p % block_size of block block_table[b * table_width + p / block_size].
 * The three arrays are DEVICE int32, 4-byte aligned: cu_seqlens B + 1
 * non-decreasing offsets from 0, at most `total`; rows at and behind
 * cu_seqlens[B] are neither read nor written, so a captured graph can be sized
 * for more tokens than a replay has.  max_seqlen >= every n_b and at most
 * `total` (it sizes the grids; 0 launches nothing).  table_width x block_size is
 * at most 2^31 - 65536.  A block may appear in several sequences (a shared
 * prefix) as long as no call appends to it.
 * Entries are checked on the device.  A sequence with offsets out of range or
 * decreasing, n_b > max_seqlen, or a length that is negative, beyond its table
 * row or (append, read) below n_b is skipped (where offsets do not ascend, any
 * sequence of the call may be); a block number outside
 * [0, num_blocks) drops its tokens (they are not written; read gives zeros for
 * them; they are not visible to the attention).  Both are reported through the
 * device error word (0x440 and 0x441 append, 0x450 and 0x451 read, 0x460 and
 * 0x461 attention).  Table entries behind a sequence's length are not looked
 * at.  n_b = 0 is allowed; total = 0 launches nothing. */
typedef struct {
  const int* block_table;
  const int* lens;
  const int* cu_seqlens;
  int B;
  int table_width;
  int total;
  int max_seqlen;
} fattn_cache_batch;

/* Quantise the n_b new tokens of each sequence into its blocks.
 * k, v: DEVICE bf16, 16-byte aligned, element (t, h, c) at t * token stride +
 * h * head stride + c (strides in elements, non-negative multiples of 8; so a
 * slice of a fused projection's output or a head-major tensor is taken as it
 * is).
 * The scale of a block and head is the smallest power of two 2^e, e >= -100,
 * with amax <= largest code * 2^e, amax over the finite values written so far.
 * A block that gets its first token starts anew; one that holds earlier tokens
 * of the sequence keeps its scale unless the new tokens need a larger one, in
 * which case the earlier codes are rewritten for it, rounded to nearest even
 * (the ratio is a power of two, so only codes that become subnormal change
 * their value).  New values are divided by the scale (exact) and rounded to
 * nearest even.  NaN and infinities are stored as NaN and do not enter amax.
 * 4 bits: with a the largest magnitude of 16 neighbouring channels, their scale is
 * a / 8 rounded to the nearest e5m2 value, with a negative sign if one of them is +a,
 * else a positive one, and c - 8 is x / scale rounded to the nearest whole number,
 * ties to even, within [-8, 7].  Where the scale is at least 2^-14, a value that this
 * range cuts is off by at most one scale if it has the largest one's sign, else by at
 * most two, and every other by at most half of one.  Magnitudes beyond 57344 and
 * infinities count as 57344, NaN as zero.
 * A call that is repeated with the same arguments leaves the same cache.
 * No block may be named twice among those that a call appends to (the writes
 * would race; nothing out of range is touched). */
int fattn_cache_append(const fattn_cache* cache, const fattn_cache_batch* batch, const void* k,
                       long long k_token_stride, long long k_head_stride, const void* v,
                       long long v_token_stride, long long v_head_stride, void* stream);

/* The inverse: the last n_b tokens of each sequence as bf16 of their values, into
 * k and v laid out as for fattn_cache_append (strides >= d here).  Exact for
 * the scales that append writes (but for bf16 values next to 2^128, whose code
 * rounds up to it and becomes an infinity here), and always in 4 bits. */
int fattn_cache_read(const fattn_cache* cache, const fattn_cache_batch* batch, void* k,
                     long long k_token_stride, long long k_head_stride, void* v,
                     long long v_token_stride, long long v_head_stride, void* stream);

/* Attention of the last n_b tokens of each sequence over its cache.
 * q, o: DEVICE bf16 [total, Hq, d] by strides as above (o's strides >= d); Hq a
 * multiple of H, query head h reads key/value head h / (Hq / H); o may be q
 * itself, with its strides.  lse: DEVICE
 * fp32 [Hq, total], contiguous (the layout of fattn_fwd_varlen), 16-byte
 * aligned.  Query i of sequence b stands at position lens[b] - n_b + i; with
 * causal it sees keys at or before its position, else every key of the
 * sequence.  A query that sees no key gets o = 0 and lse = -inf.  n_b may
 * exceed lens[b].  Values of keys that a query does not see never reach its
 * row, whatever they are (NaN included); an e5m2 infinity, which append never
 * writes, gives the rows that see it an infinity or NaN.
 * Scores, statistics and sums are fp32, of q exact down to 2^-29 of the largest
 * element of its row.  A weight, times its value scale, is
 * rounded to fp16 relative to the largest of its row among blocks whose scales
 * lie within 2^20 of each other or below: 11 bits down to 2^-22 of that, an
 * error of 2^-33 of it below.  (4 bits: no scales, the weights alone.)
 * workspace: DEVICE memory of fattn_cache_fwd_workspace_bytes(...) bytes,
 * 256-byte aligned, owned by the caller, its contents on entry do not matter;
 * calls that overlap on the GPU need one each.  Returns FATTN_OK,
 * FATTN_ERR_INVALID_ARG, FATTN_ERR_UNSUPPORTED, FATTN_ERR_WORKSPACE or
 * FATTN_ERR_CUDA; launches nothing on an argument error, as the two calls
 * above. */
int fattn_cache_fwd(const fattn_cache* cache, const fattn_cache_batch* batch, const void* q,
                    long long q_token_stride, long long q_head_stride, void* o,
                    long long o_token_stride, long long o_head_stride, float* lse, int Hq,
                    float scale, int causal, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Workspace bytes of fattn_cache_fwd on the current device, from the sizes in
 * the two descriptors (their pointers are not looked at); 0 if invalid. */
size_t fattn_cache_fwd_workspace_bytes(const fattn_cache* cache, const fattn_cache_batch* batch,
                                       int Hq);

/* The attention weight that every cached key receives, for choosing what to keep:
 *     W[b, h, j] = (W_in[b, h, j], or 0) + sum exp(scale q . k_j - lse)
 * over the batch's queries of sequence b that see key j (as in fattn_cache_fwd) and the heads
 * of group h; the batch's own tokens (positions from lens[b] - n_b on) start at 0.  Weights are
 * kept by sequence, not by block, as a shared block's keys have others in every sequence.
 * q as for fattn_cache_fwd, lse DEVICE fp32 [Hq, total] as it wrote it (a row with -inf adds
 * nothing), Hq / H x max_seqlen at most 2^31 - 65536.  weights (NULL: zeros) and weights_out: DEVICE
 * fp32, 4-byte aligned, element (b, h, j) at b * sequence stride + h * head stride + j, strides in
 * elements and not negative, rows of `width` elements, those of weights_out not overlapping; they
 * may be the same, with the same strides, and must not overlap otherwise.  Elements at and behind
 * lens[b], and sequences with n_b = 0, are not touched.
 * A sequence whose entries are bad (as above) or whose length exceeds width is skipped (code
 * 0x470), keys of a bad block number get 0 from the queries (0x471); 0x472 to 0x47b say that a
 * wait inside the kernel ran out.  Every sum is formed in one order: repeated calls agree bit for
 * bit.  Scores, exponentials and sums are fp32.
 * A NaN key makes its weight NaN and, by way of lse, those of the keys whose queries see it. */
int fattn_cache_weights(const fattn_cache* cache, const fattn_cache_batch* batch, const void* q,
                        long long q_token_stride, long long q_head_stride, const float* lse,
                        int Hq, float scale, int causal, const float* weights,
                        long long weights_seq_stride, long long weights_head_stride,
                        float* weights_out, long long out_seq_stride, long long out_head_stride,
                        int width, void* stream);

/* Eviction by weight: for every sequence b longer than `keep` tokens and every key/value head,
 * the last `recent` tokens and, of the others, the keep - recent with the largest weights are
 * copied in their order to positions 0 ... keep - 1 of the blocks of table_out; a sequence of at
 * most keep tokens is copied whole.  Heads keep different tokens.  NaN counts as the largest
 * weight, of equal ones the earlier token is kept; -0 equals 0.
 * batch: block_table, lens, B and table_width are used; cu_seqlens, total and max_seqlen are not
 * looked at.  weights as above (one row of `width` per sequence and head).  table_out: DEVICE int32
 * [B, table_out_width] with room for min(keep, width) tokens.  Its blocks belong to the same
 * pool and must not be among those that the call reads, nor twice among those that it writes,
 * but for a sequence of at most keep tokens, which may be given its own.  The blocks read stay
 * as they are, so prefixes that other sequences share stay whole.
 * Written: lens_out [B] (int32, not lens itself) = min(lens, keep); kept [B, H, keep] (int32) the
 * positions kept, ascending, -1 behind the last; weights_out (as above, not weights itself,
 * rows of out_width >= min(keep, width)) their weights, elements behind the last untouched.
 * 8 bits: the scale of a destination block is the largest of its tokens' scales, and codes that
 * had a smaller one are rounded for it to nearest even (exact but for codes that become
 * subnormal, where the scales are powers of two).  4 bits: codes and scales as they are.
 * A length that is negative or beyond its table row or width counts as 0 (code 0x480); a token
 * whose block number is bad becomes zeros, a bad number in table_out drops its tokens (0x481).
 * 1 <= keep, 0 <= recent <= keep. */
int fattn_cache_evict(const fattn_cache* cache, const fattn_cache_batch* batch,
                      const float* weights, long long weights_seq_stride,
                      long long weights_head_stride, int width, const int* table_out,
                      int table_out_width, int keep, int recent, int* lens_out, int* kept,
                      float* weights_out, long long out_seq_stride, long long out_head_stride,
                      int out_width, void* stream);

/* ------------------------------------------------------------------ rotary positions
 *
 * Pairs of channels of queries and keys are turned by angles that grow with a token's
 * position, before the attention (and before keys go into a cache).  The pages have no
 * counterpart.  Channel pair i of a token at position p turns by the angle p w_i:
 *     a' = m (a cos(p w_i) - b sin(p w_i)),   b' = m (a sin(p w_i) + b cos(p w_i)). */
typedef enum {
  FATTN_ROPE_HALF = 0,       /* pair i: channels i and rot / 2 + i */
  FATTN_ROPE_INTERLEAVED = 1 /* pair i: channels 2 i and 2 i + 1 */
} fattn_rope_layout;

/* How the frequencies w_i = base^(-2 i / rot) are changed for contexts `factor` times as
 * long as the `length` that a model was trained with. */
typedef enum {
  FATTN_ROPE_NONE = 0,
  FATTN_ROPE_LINEAR = 1, /* w_i / factor */
  FATTN_ROPE_BASE = 2,   /* base times factor^(rot / (rot - 2)), so the slowest pair is divided by
                            factor and the fastest is kept */
  FATTN_ROPE_YARN = 3,   /* w_i where the pair makes more than about `fast` turns over `length`,
                            w_i / factor where fewer than `slow`, a ramp over the pairs between
                            (floor and ceiling of the two pairs; pair 0 always has w_0);
                            m = 0.1 ln(factor) + 1 */
  FATTN_ROPE_BANDS = 4   /* the same by turns n_i = length w_i / 2 pi: the share of w_i is
                            (n_i - slow) / (fast - slow), cut to [0, 1]; m = 1 */
} fattn_rope_scaling;

/* The frequencies as fractions of a turn, on the HOST (no device is touched): turns[i] =
 * 2^64 frac(w_i / 2 pi) for i < rot / 2, and *magnitude = m.  rot even, base > 1; factor
 * (finite, > 0, as its inverse) is read unless kind is NONE, length, fast and slow (fast > slow >
 * 0) by YARN and BANDS.  Formed in double precision: an angle at position p is off by about
 * 2^-52 p turns at most (2^-52 p w_i where a factor below 1 makes w_i larger than 1). */
int fattn_rope_turns(unsigned long long* turns, float* magnitude, int rot, double base, int kind,
                     double factor, int length, double fast, double slow);

/* Turns the first rot channels of every row of q [total, Hq, d] and k [total, Hk, d] (bf16,
 * DEVICE, 16-byte aligned, strides in elements as for fattn_cache_append, those of the outputs
 * as for fattn_cache_read) and writes rows of d channels to q_out and k_out; the channels from
 * rot on are copied.  An output may be its input, with the same strides; otherwise they must not
 * overlap.  Hq and Hk are at most 65535; one may be 0 (its pointers are not looked at).  total x
 * (Hq + Hk) is at most 2^31 - 4.  positions: DEVICE int32 [total], of either sign; turns: DEVICE
 * [rot / 2] of 64 bits, 8-byte aligned, as fattn_rope_turns gives them; magnitude m finite and
 * > 0.  d is 64 or 128, rot a multiple of 16 up to d.  The angle is exact in turns (64-bit arithmetic modulo one turn) up to the
 * fractions given; sines, products and sums are fp32, rounded once to bf16.
 * backward != 0: the gradient, i.e. the transposed map (q and k are dL/dq_out and dL/dk_out).
 * Returns FATTN_OK, FATTN_ERR_INVALID_ARG, FATTN_ERR_UNSUPPORTED or FATTN_ERR_CUDA; launches
 * nothing on an argument error or when total = 0. */
int fattn_rope(const void* q, long long q_token_stride, long long q_head_stride, void* q_out,
               long long q_out_token_stride, long long q_out_head_stride, int Hq, const void* k,
               long long k_token_stride, long long k_head_stride, void* k_out,
               long long k_out_token_stride, long long k_out_head_stride, int Hk,
               const int* positions, const unsigned long long* turns, float magnitude, int total,
               int d, int rot, int layout, int backward, void* stream);

/* Tile shape used by a pass (0 = forward, 1 = backward) for head size d:
 * rows of Q per tile and keys per K/V tile; 128 x 128, the tile of "Decoding
 * flash attention" ("The idea: never build the matrix").  block_q and block_k may be NULL.
 * Returns FATTN_OK, FATTN_ERR_UNSUPPORTED (d) or FATTN_ERR_INVALID_ARG (pass). */
int fattn_tile_sizes(int d, int pass, int* block_q, int* block_k);

/* Read (and, if clear != 0, reset) the device error word of the current
 * device: *code = 0 if no in-kernel wait ran out since the last reset, else
 * the code of the first one (low byte: the waiting role; next byte: the
 * kernel).  Synchronises the device.  Returns FATTN_OK when the word was 0,
 * FATTN_ERR_TIMEOUT when it was set (with *code written, and cleared if
 * asked), FATTN_ERR_INVALID_ARG for a NULL code, FATTN_ERR_CUDA.  The pages
 * have no counterpart: it reports this library's bounded waits. */
int fattn_device_error(unsigned int* code, int clear);

/* Human-readable name of a status code (static storage).  No passage: a helper.
 * The library also exports two test and measurement hooks, declared apart in
 * fattn_testing.h; they are not part of this interface. */
const char* fattn_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_H_ */
