/*
 * attn.h -- C ABI of the fused attention forward (online softmax) for GB300 (sm_103a).
 *
 * The operation is the exact attention forward
 *
 *     O = softmax(scale * Q K^T + mask) V,   LSE_i = ln sum_j exp(scale * q_i . k_j)  (visible j)
 *
 * computed block by block with the online-softmax recurrence (running max m,
 * running denominator l, unnormalised accumulator o~, rescale by
 * alpha = exp(m_old - m_new) when the max rises, one division o~/l at the end),
 * never materialising the Nq x Nk score matrix.
 * Sources: "2.2b: FlashAttention -- Online Softmax" (hf-cn0.pages.dev), sections
 * "The Complete Online Softmax Algorithm" and "Extending to Attention";
 * "FlashAttention math" (aicassindra.com), sections "What we must compute" and
 * "The block-wise update, and the full algorithm"; "Tiled attention: running
 * max softmax" (archcrux.com) for masked keys and fully masked rows.
 *
 * Conventions (the pages leave these open; this library fixes them):
 *  - Layout: Q [B,H,Nq,d], K and V [B,H,Nk,d], O [B,H,Nq,d]: row-major, contiguous,
 *    bf16.  LSE [B,H,Nq]: fp32, natural log of the sum over visible keys of
 *    exp(scale * q . k).
 *  - Mask: key j is visible to query i iff j < L_b (key padding; L_b = key_padding_lens[b]
 *    clamped to [0, Nk], or Nk when key_padding_lens is NULL) and, when causal != 0,
 *    j <= i + (Nk - Nq) (bottom-right aligned; j <= i when Nq == Nk).  Masked scores are
 *    -inf before the block maximum is taken.
 *  - A row with no visible key (fully masked, or Nk == 0) gets O = 0 and LSE = -inf,
 *    never 0/0.
 *  - d must be 64 or 128.  scale must be finite and > 0 (1/sqrt(d) is the usual value).
 *  - Q, K, V and O must be 16-byte aligned (TMA), LSE 4-byte aligned; the library does
 *    not check that they are device pointers.
 *
 * Ownership: the caller owns every buffer.  attn_fwd allocates no device memory per
 * call; the library keeps one small device status word per device, created on first use.
 * Streams: every kernel is launched with programmatic stream serialization, so it may be
 * scheduled while the previous kernel in the stream finishes; it touches no global
 * memory before that kernel has completed and its writes are visible, so stream order
 * holds for every buffer as with a plain launch.
 * Errors: every entry point returns an attn_status; no C++ exception crosses this ABI.
 * attn_last_error() gives a message for the calling thread's last failure.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_NULLPTR = -1,        /* a required pointer is NULL */
  ATTN_ERR_BAD_SHAPE = -2,      /* negative or too-large B, H, Nq, Nk */
  ATTN_ERR_UNSUPPORTED_D = -3,  /* d not in {64, 128} */
  ATTN_ERR_MISALIGNED = -4,     /* a pointer is not 16-byte aligned */
  ATTN_ERR_NO_DEVICE = -5,      /* no usable sm_103 device / CUDA runtime error at setup */
  ATTN_ERR_LAUNCH = -6,         /* kernel launch or copy failed (message in attn_last_error) */
  ATTN_ERR_TIMEOUT = -7,        /* a bounded device-side wait ran out (see attn_status_sync) */
  ATTN_ERR_BAD_ARG = -8,        /* scale not finite or not > 0, or another bad scalar */
  ATTN_ERR_BAD_PAGE = -9        /* a cached position without a page (see attn_cache_check) */
} attn_status;

/*
 * attn_fwd -- enqueue the attention forward on `stream`.
 *   Q, K, V   device bf16 inputs (layouts above).  K and V may be NULL when Nk == 0.
 *   O         device bf16 output [B,H,Nq,d];  LSE device fp32 output [B,H,Nq].
 *   B, H, Nq, Nk >= 0; a call with B*H*Nq == 0 does nothing and returns ATTN_OK.
 *   d         64 or 128.     scale   multiplies q . k before the softmax.
 *   causal    0 or nonzero (bottom-right aligned causal mask).
 *   key_padding_lens  device int32[B] or NULL (no padding).
 *   stream    a cudaStream_t, or NULL for the legacy default stream.
 * Asynchronous: returns after the launch.  Argument and launch errors are returned at
 * once; a device-side wait timeout is reported by attn_status_sync.
 * Environment, read at every launch (all entry points):
 *   ATTN_WAIT_LIMIT_MS          limit of each device-side wait in ms (default 2000).
 *   ATTN_TEST_WITHHOLD_K_BLOCK  test hook, honoured only while ATTN_ENABLE_TEST_HOOKS=1 is
 *                               also set: the loader skips key block j (0-based) of every
 *                               tile, so the waits on it run out; the call then reports
 *                               ATTN_ERR_TIMEOUT and O / LSE are not written.
 */
attn_status attn_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Nq,
                     int Nk, int d, float scale, int causal, const int32_t* key_padding_lens, void* stream);

/* Exponential evaluation modes (attn_options.exp2_mode). */
enum {
  ATTN_EXP2_DEFAULT = 0,   /* the library's choice (currently ATTN_EXP2_HARDWARE: measured fastest) */
  ATTN_EXP2_HARDWARE = 1,  /* every exp2 on the MUFU unit (ex2.approx) */
  ATTN_EXP2_MIXED = 2      /* in blocks without a masked key, 1 of every 16 pairs of scores takes
                              a degree-4 polynomial on the FMA pipe (relative error < 3e-6) */
};

/* Per-call choices for attn_fwd_ex.  Set size = sizeof(attn_options); zero the rest for
 * the defaults.  (An addition of this library; the pages fix neither choice.) */
typedef struct attn_options {
  size_t size;
  /* Lazy rescale: the running max m is moved (and l, o~ rescaled) only when a block's max
   * exceeds it by more than tau = this many natural-log units.  0 = the pages' rule
   * (rescale whenever the max rises).  The result is the same in exact arithmetic:
   * softmax is invariant to the reference ("FlashAttention math", "Safe softmax": any
   * constant m).  Range [0, 20].
   * Stability bound ("FlashAttention math", "Proof of numerical stability", restated for
   * a reference that may trail the max by up to tau): every score the recurrence meets
   * is at most m + tau, so every probability p = exp(s - m) <= e^tau (<= 4.9e8 at
   * * tau = 20, well inside the range of bf16 P and of fp32), the running sum
   * l <= Nk * e^tau and |o~| <= Nk * e^tau * max|V| (per column).  The result is finite
   * whenever Nk * e^tau * max|V| < FLT_MAX = 3.4e38 (at tau = 0 this is the plain fp32
   * accumulation bound Nk * max|V|); inputs beyond it may overflow o~ to inf and are
   * excluded.  Example: at tau = 20 and Nk = 2^20 keys, |V| must stay below 6.7e23. */
  float rescale_threshold;
  int exp2_mode;           /* ATTN_EXP2_* */
  /* Keys per block: 0 or 128 (the default), 64 or 192.  64 and 192 are available at
   * d = 128 for the dense layouts (attn_fwd_ex; not packed sequences, not split-KV states)
   * with exp2_mode DEFAULT or HARDWARE: the same recurrence over blocks of another size
   * ("FlashAttention math", "Proof of exactness": blocks of any size give the same result).
   * 192 keeps two score buffers in tensor memory instead of three, 64 three buffers of 64
   * columns and four K/V stages.  Both are measured slower than 128 on GB300; they let a
   * caller check that the result does not depend on the block size.  Any other value is
   * ATTN_ERR_BAD_ARG.  Callers built before this field existed pass a smaller size and get
   * the default. */
  int key_block;
} attn_options;

/*
 * attn_fwd_ex -- attn_fwd with options (opts may be NULL: the defaults, identical to
 * attn_fwd).  Errors: as attn_fwd, plus ATTN_ERR_BAD_ARG for a bad options struct.
 */
attn_status attn_fwd_ex(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Nq,
                        int Nk, int d, float scale, int causal, const int32_t* key_padding_lens,
                        const attn_options* opts, void* stream);

/*
 * attn_fwd_strided -- attn_fwd over tensors with any (batch, head, row) strides, e.g.
 * the [B, N, H, d] ("BSHD") layout: strides {N*H*d, d, H*d}.  (The pages fix no layout;
 * an addition of this library.)
 *   q_strides, k_strides, v_strides, o_strides: host int64[3] each, the element strides
 *   of the batch, head and row dimensions; element (b, h, i, x) of Q is at
 *   Q + b*q_strides[0] + h*q_strides[1] + i*q_strides[2] + x (d is contiguous).
 *   Every stride must be a positive multiple of 8 elements (16 bytes, for TMA) below
 *   2^38; the rows of O must not overlap.  LSE stays contiguous [B, H, Nq].
 *   Everything else as attn_fwd.  Errors: as attn_fwd, plus ATTN_ERR_BAD_ARG for a bad
 *   stride and ATTN_ERR_NULLPTR for a NULL stride array.
 */
attn_status attn_fwd_strided(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Nq,
                             int Nk, int d, float scale, int causal, const int32_t* key_padding_lens,
                             const int64_t* q_strides, const int64_t* k_strides, const int64_t* v_strides,
                             const int64_t* o_strides, void* stream);

/*
 * attn_fwd_varlen -- attention over B packed sequences of different lengths (an addition
 * of this library; the pages treat one sequence).
 *   Q, O  device bf16 [total_q, H, d]: sequence b is rows cu_seqlens_q[b] ..
 *         cu_seqlens_q[b+1] - 1.  K, V device bf16 [total_k, H, d] (Q's H), rows cu_seqlens_k[b] ..
 *   cu_seqlens_q, cu_seqlens_k  device int32[B + 1], non-decreasing from 0 to total_q /
 *         total_k (values are clamped to [0, total] on the device, so a bad array cannot
 *         make the kernel write outside O and LSE).
 *   max_seqlen_q  >= the longest query sequence (the grid covers that many rows; longer
 *         sequences are left partly unwritten).  It, total_q and total_k are at most 2^31 - 256, and
 *         B * H * ceil(max_seqlen_q / 128) at most 2^31 - 2^13 - 1.
 *   LSE   device fp32 [H, total_q].
 *   Masks per sequence: query i of sequence b (Nq_b rows, Nk_b keys) sees key j iff
 *   j < Nk_b and, when causal, j <= i + (Nk_b - Nq_b).  A sequence with no keys gets O = 0
 *   and LSE = -inf.  Asynchronous; timeouts through attn_status_sync.
 */
attn_status attn_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* LSE,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int H, int max_seqlen_q,
                            int total_q, int total_k, int d, float scale, int causal, void* stream);

/*
 * attn_fwd_host -- the same operation on HOST buffers (pinned memory recommended).
 * Copies Q, K, V (and key_padding_lens, a host int32[B] or NULL) to the device, runs the
 * forward, copies O and LSE back and synchronises `stream` before it returns.  The copies
 * run on two streams of the library's own, overlapped with the forward on `stream`: the
 * heads are cut into chunks (runs of heads of one batch, about 32 MB of input each) and
 * chunk i is computed while chunk i + 1 is copied in and chunk i - 1 copied out.  The
 * work starts after what is already queued on `stream`.  Uses a per-device workspace
 * that grows to the largest problem seen and is kept until attn_release_workspace(); it
 * allocates only when a call needs more room (and creates its two streams once).
 */
attn_status attn_fwd_host(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                          int Nq, int Nk, int d, float scale, int causal, const int32_t* key_padding_lens,
                          void* stream);

/* Free the attn_fwd_host workspace of the current device. */
attn_status attn_release_workspace(void);

/* Synchronise `stream`, then read and clear the device status words of the current
 * device (the one the allocating entry points use and, once attn_fwd_noalloc has run
 * on the device, its fixed one): ATTN_ERR_TIMEOUT if a kernel's bounded wait ran out
 * since the last check.  Reads and clears with plain copies; allocates nothing. */
attn_status attn_status_sync(void* stream);

/* Message for the calling thread's last non-OK status ("" if none). */
const char* attn_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int attn_version(void);

/*
 * attn_fwd_noalloc -- attn_fwd for callers that must not allocate device memory.
 * (An addition of this library; the source pages have no counterpart.)
 *
 * Who needs it: code that runs where cudaMalloc is off limits -- a process whose device
 * memory is handed out by someone else's pool or a fixed budget, a real-time or
 * embedded caller that may not allocate after start-up, or a plugin that must not
 * grow the host application's footprint.  attn_fwd itself allocates a 4-byte status
 * word with cudaMalloc on its first call on each device; this entry point never does.
 *
 * Same arguments and semantics as attn_fwd, plus check_status.  The caller still
 * passes every input and output buffer.  The only device scratch the kernel needs
 * (one 32-bit status word for its bounded waits) lives in a fixed array compiled into
 * the library: 256 bytes per device, held by every GPU that loads the library until
 * the process exits.  A call whose scratch need exceeds that size is rejected with
 * ATTN_ERR_BAD_SHAPE (the forward kernel needs 4 bytes, so today no call is).
 *
 *  - The first call on a device does one-time set-up with that device current: it
 *    looks up the array's device address (cudaGetSymbolAddress), sets the shared-memory
 *    attribute of every kernel this entry point can launch (d = 128, d = 64 with one
 *    and with two query tiles per CTA) and caches the SM count.  Make that first call
 *    before any stream capture.
 *  - Every call shares the array and it keeps the last call's contents.  Its status
 *    word is the OR of every bounded wait that ran out since the word was last read; it
 *    starts at zero and is cleared where it is read: by a call with check_status != 0
 *    and by attn_status_sync.  Calls that overlap on the GPU (different streams, or
 *    several host threads) share that word, so a timeout is reported to whichever of
 *    them reads it first; serialise them if you rely on the attribution.
 *  - check_status == 0: asynchronous, like attn_fwd; a device-side wait that runs out
 *    still ends the kernel, and attn_status_sync (on a stream ordered after the call)
 *    reports it later.  check_status != 0: the call synchronises `stream` and returns
 *    ATTN_ERR_TIMEOUT if a wait ran out since the word was last read.
 *  - It calls no cudaMalloc, cudaFree or other allocating routine, and its kernels use no
 *    local memory (which the driver would back on first launch).  Loading the library's
 *    device code onto a device takes device memory once per process, as for any CUDA
 *    library (the module image, which holds the fixed array): under CUDA's default lazy
 *    module loading that happens at the library's first call on the device, whichever
 *    entry point it is.  A caller whose device memory must not move after start-up makes
 *    one call at start-up (attn_status_sync(NULL) is enough) or sets
 *    CUDA_MODULE_LOADING=EAGER.
 */
attn_status attn_fwd_noalloc(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                             int Nq, int Nk, int d, float scale, int causal, const int32_t* key_padding_lens,
                             int check_status, void* stream);

/* ------------------------------------------------------------------------------------
 * Split-KV: the keys of every row are cut into splits, each split is absorbed into its
 * own running state, and the states are merged.
 *
 * A state is the triple the recurrence carries ("FlashAttention math", section "The
 * running state"): m = the largest visible scaled score scale * q . k_j of the split,
 * l = sum exp(s_j - m) and o~ = sum exp(s_j - m) v_j (unnormalised) over the split's
 * visible keys.  A split with no visible key for a row holds the initial state
 * m = -inf, l = 0, o~ = 0.  The pages let keys be absorbed in any order and in blocks of
 * any size (same page, "Proof of exactness"); states of disjoint key sets combine with
 * the rescaling identity (section "The rescaling identity, derived"): with
 * m = max_s m_s, l = sum_s exp(m_s - m) l_s and o~ = sum_s exp(m_s - m) o~_s.
 * This serves shapes with few query tiles and many keys (decoding, short prompts over
 * a long cache), where one CTA per query tile leaves most SMs idle; the same merge is
 * the exchange step of a key-sharded (context-parallel) forward.
 * ------------------------------------------------------------------------------------ */

/*
 * attn_fwd_states -- the partial states of num_splits key splits (1 <= num_splits <= 256).
 *   Split s covers keys [s * C, (s + 1) * C) intersected with [0, Nk), where
 *   C = 128 * ceil(ceil(Nk / 128) / num_splits); masks as for attn_fwd.
 *   Q, K, V, B, H, Nq, Nk, d, scale, causal, key_padding_lens, stream: as attn_fwd.
 *   o_states  device fp32 [num_splits, B, H, Nq, d]: o~.
 *   m_states  device fp32 [num_splits, B, H, Nq]: m (natural-log units; -inf = empty).
 *   l_states  device fp32 [num_splits, B, H, Nq]: l.
 *   All three 16-byte aligned.  Asynchronous; timeouts through attn_status_sync.
 *   Errors: as attn_fwd, plus ATTN_ERR_BAD_ARG for num_splits out of range.
 */
attn_status attn_fwd_states(const void* Q, const void* K, const void* V, float* o_states, float* m_states,
                            float* l_states, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                            const int32_t* key_padding_lens, int num_splits, void* stream);

/*
 * attn_merge_states -- merge num_states >= 1 states per row and finish each row:
 *   O = o~ / l (bf16) and LSE = m + ln l, or O = 0 and LSE = -inf when every state of
 *   the row is empty.  rows = number of rows (B * H * Nq for attn_fwd_states' output).
 *   o_states fp32 [num_states, rows, d] (16-byte aligned), m_states and l_states fp32
 *   [num_states, rows], O bf16 [rows, d] (16-byte aligned), LSE fp32 [rows]; all device.
 *   The states may come from anywhere (another GPU's keys, a previous call).
 *   Asynchronous on `stream`.  Errors: NULLPTR, MISALIGNED, UNSUPPORTED_D, BAD_ARG
 *   (num_states < 1), BAD_SHAPE (rows < 0), LAUNCH.
 */
attn_status attn_merge_states(const float* o_states, const float* m_states, const float* l_states, int num_states,
                              long long rows, int d, void* O, float* LSE, void* stream);

/* Bytes of device workspace attn_fwd_splitkv needs for num_splits splits (0 for
 * invalid arguments): the three state arrays, each rounded up to 256 bytes. */
size_t attn_splitkv_workspace_bytes(int B, int H, int Nq, int d, int num_splits);

/* The split count attn_fwd_splitkv picks when given num_splits <= 0, on the current
 * device: 1 when the query tiles alone fill the SMs, else enough splits to fill them
 * once, at most one split per four key blocks and at most 256. */
int attn_splitkv_splits(int B, int H, int Nq, int Nk);

/*
 * attn_fwd_splitkv -- attn_fwd computed as attn_fwd_states + attn_merge_states.
 *   Same arguments and result as attn_fwd (within the same tolerance, not bitwise),
 *   plus num_splits (<= 0: attn_splitkv_splits' choice) and a caller-owned device
 *   workspace of at least attn_splitkv_workspace_bytes(B, H, Nq, d, splits) bytes,
 *   16-byte aligned.  With one split the call is attn_fwd and the workspace is unused.
 *   No allocation.  Asynchronous; ATTN_ERR_BAD_ARG if the workspace is too small.
 */
attn_status attn_fwd_splitkv(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Nq,
                             int Nk, int d, float scale, int causal, const int32_t* key_padding_lens, int num_splits,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Paged key/value cache, and attention over it.
 * (Additions of this library; the pages treat one sequence whose K and V are at hand.)
 *
 * A cache is a pool of pages of page_size tokens: k and v are [num_pages, Hkv, page_size, d],
 * row-major and contiguous.  A batch's sequences find their pages through a block table,
 * device int32 [B, max_pages]: position p of sequence b is row p % page_size of page
 * block_table[b, p / page_size].  Pages may be shared between sequences that only read them.
 * max_pages * page_size <= 2^31 - 256.
 *
 * Types.  ATTN_CACHE_BF16: rows as they are.  ATTN_CACHE_E4M3: 8-bit codes with one scale per
 * (token, head) row, k_scale and v_scale uint8 [num_pages, Hkv, page_size]; a value is
 * code * 2^(s - 127), s in 1 .. 254 (attn_cache_write makes 1 .. 247).  A scale code of 0
 * stands for a factor of 2^-126 or less, one of 255 for one that is not finite.
 *
 * Bad pages.  A block-table entry outside [0, num_pages), or a position at or past
 * max_pages * page_size, never leads outside the cache: a token without a page is not
 * written, is read back as zeros, and is left out of the attention as a masked key is.  It is
 * reported by attn_cache_check.  Positions that no call needs may have any entry.
 * Lengths (cu_seqlens, start_lens, ctx_lens) are read on the device and clamped to what the
 * buffers hold, so a captured call follows their contents at every replay.  Make one call on
 * a device before a stream capture (the first sets up the device).
 * ------------------------------------------------------------------------------------ */

enum { ATTN_CACHE_BF16 = 0, ATTN_CACHE_E4M3 = 1 };

typedef struct attn_cache {
  size_t size;        /* sizeof(attn_cache) */
  void* k;            /* device [num_pages, num_heads, page_size, d], 16-byte aligned */
  void* v;
  uint8_t* k_scale;   /* device [num_pages, num_heads, page_size], 16-byte aligned; e4m3 only */
  uint8_t* v_scale;
  int type;           /* ATTN_CACHE_* */
  int num_pages;      /* >= 0 */
  int page_size;      /* a multiple of 16, at most 65536 */
  int num_heads;      /* K/V heads, 1 .. 65536 */
  int d;              /* 64 or 128 */
} attn_cache;

/*
 * attn_cache_write -- put the new tokens' K and V into the cache.
 *   K, V  device bf16, `total` packed tokens of num_heads rows: element (t, h, x) of K is at
 *         K + t * k_strides[0] + h * k_strides[1] + x, so slices of a joint projection need no
 *         copy.  Host int64[2] strides in elements, multiples of 8.  16-byte aligned.
 *   cu_seqlens  device int32 [B + 1]: sequence b's tokens are rows cu_seqlens[b] ..
 *         cu_seqlens[b + 1] - 1; they go to positions start_lens[b], start_lens[b] + 1, ...
 *         (start_lens: device int32 [B], or NULL for 0; negative counts as 0).  Rows outside
 *         every sequence are not written.
 *   The positions written must be distinct rows of the pool (two sequences that write share no
 *   page there): with the same row named twice, which token it holds, or a mixture, is not
 *   defined.
 * e4m3: a row x gets e, the least integer >= -126 with max |x_i| <= 448 * 2^e over its finite
 * values, s = e + 127 and codes x_i * 2^-e rounded to nearest even: infinities become
 * +-448 * 2^e, NaN stays NaN.  At e = 120, the largest, magnitudes past 240 * 2^120 become
 * that (2^128 would be no bf16).  Asynchronous.
 */
attn_status attn_cache_write(const attn_cache* cache, const void* K, const void* V, const int64_t* k_strides,
                             const int64_t* v_strides, const int32_t* block_table, int max_pages,
                             const int32_t* cu_seqlens, const int32_t* start_lens, int B, int total, void* stream);

/*
 * attn_cache_read -- cached positions back as packed bf16 K and V [total, num_heads, d], e.g.
 *   for a prompt over a cached prefix through attn_fwd_prompt, which takes them as they are.
 *   (attn_fwd_varlen has one head count: for it, where a group of query heads shares a K/V head, repeat
 *   the rows read here for each of them; passing them as they are with Q's H would read past their end.)
 *   Row cu_seqlens[b] + i is position start_lens[b] + i of sequence b.  Exact: every e4m3 value times its scale that
 *   attn_cache_write makes is a bf16.  Rows outside every sequence are left as they were.
 *   K, V 16-byte aligned.  Asynchronous.
 */
attn_status attn_cache_read(const attn_cache* cache, void* K, void* V, const int32_t* block_table, int max_pages,
                            const int32_t* cu_seqlens, const int32_t* start_lens, int B, int total, void* stream);

/*
 * attn_fwd_tree -- attention of each sequence's new (drafted) tokens over its cache.
 *   Sequence b has ctx_lens[b] cached tokens (device int32 [B], NULL: 0) and the T_b tokens of
 *   rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 of Q, whose K and V are already in the
 *   cache at positions ctx_lens[b] .. ctx_lens[b] + T_b - 1.  T_b = 1 is plain decoding.
 *   Q, O  device bf16 [total_q, Hq, d], LSE fp32 [Hq, total_q].  Hq is a multiple of the
 *         cache's heads and at most 65536: query head h reads K/V head h / (Hq / num_heads).
 *         O may be Q itself (not another part of it).
 *   tree_mask  device int64 [total_q] or NULL.  Token i of a sequence sees every context key,
 *         and its token u when bit u of tree_mask[row of i] is set (bits from T_b on are
 *         ignored; a token sees itself only if its own bit is set).  NULL: a chain, u <= i.
 *         A row that sees nothing gets O = 0 and LSE = -inf.  What K and V hold where a row
 *         does not look, infinities and NaN among it, does not reach the row.
 *   The running maximum may trail by a factor of 2^8 (as attn_options.rescale_threshold
 *   describes), so sums must stay in range with that: keys * 2^8 * max|V| < 3.4e38; and, for an
 *   e4m3 cache, 2^8 * d * max|K| < 3.4e38.  Values of an e4m3 cache near the least normal number
 *   lose digits: what a key adds to O may be off by 2^-125 more.
 *   max_seqlen_q  in [0, 64], >= the most tokens of a sequence (rows past it are left as they
 *         were, as are rows of Q outside every sequence).
 *   workspace  device, attn_tree_workspace_bytes(...) bytes, 16-byte aligned, this call's own
 *         until it has finished: calls that may run at the same time (other streams, graphs)
 *         each need one.  Its contents mean nothing between calls.
 *   Asynchronous, allocates nothing; device-side timeouts through attn_status_sync or
 *   attn_cache_check (the environment variables of attn_fwd hold here too, key blocks of 128).
 *   Errors: as attn_fwd, plus ATTN_ERR_BAD_SHAPE for max_seqlen_q > 64 or an Hq that is no
 *   multiple or too large, ATTN_ERR_BAD_ARG for a small workspace.
 */
attn_status attn_fwd_tree(const void* Q, const attn_cache* cache, void* O, float* LSE, const int32_t* block_table,
                          int max_pages, const int32_t* cu_seqlens_q, const int32_t* ctx_lens,
                          const int64_t* tree_mask, int B, int Hq, int max_seqlen_q, int total_q, float scale,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace attn_fwd_tree needs (0 for invalid arguments). */
size_t attn_tree_workspace_bytes(int Hq, int Hkv, int max_seqlen_q, int d);

/* ------------------------------------------------------------------------------------
 * Prompts of grouped heads, and a cache of bounded length.
 * (Additions of this library, as the paged cache is.)
 * ------------------------------------------------------------------------------------ */

enum { ATTN_WEIGHT_BF16 = 0, ATTN_WEIGHT_FP32 = 1 };

/*
 * attn_qk_rotate -- norms of query and key heads and their rotation by position, in one pass.
 *   Q [total, Hq, d], K [total, Hkv, d]: device bf16, element (t, h, x) at t * strides[0] + h *
 *         strides[1] + x (host int64[2] in elements, multiples of 8), so slices of a joint
 *         projection need no copy.  Q_out and K_out the same with strides of their own; Q_out may
 *         be Q itself and K_out K (same strides), an output overlaps no other input.  16-byte aligned.  Hq or Hkv
 *         may be 0 (its pointers are not used).
 *   q_weight, k_weight  device [d] of weight_type, or NULL: no norm.  With one, a row becomes
 *         x_i * w_i / sqrt(mean(x^2) + eps).
 *   inv_freq  device fp32 [num_freq], num_freq a multiple of 8 up to d / 2 (0: no rotation).
 *         Then column i of the first num_freq and column i + num_freq (interleaved != 0: columns
 *         2 i and 2 i + 1) turn by position * inv_freq[i]: (a, b) -> (a cos - b sin, b cos + a sin).
 *         Columns from 2 * num_freq on keep their places.  The angle's error is 2^-52 of it, and
 *         2^-23 rad.  A frequency that is not finite makes its columns NaN.
 *   Positions.  cu_seqlens (device int32 [B + 1]): row cu_seqlens[b] + i is at position
 *         start_lens[b] + i (device int32 [B] or NULL for 0, negative counts as 0); rows outside
 *         every sequence are left as they were.  NULL: all rows are one sequence (B = 1).
 *         positions (device int32 [total] or NULL) replaces these positions: drafted trees, or
 *         caches whose rows have moved (attn_cache_evict).
 *   All in fp32, rounded to bf16 once; |x| must stay below 2^60 for its square.  Asynchronous.
 */
attn_status attn_qk_rotate(const void* Q, const void* K, void* Q_out, void* K_out, const int64_t* q_strides,
                           const int64_t* k_strides, const int64_t* q_out_strides, const int64_t* k_out_strides,
                           const int32_t* cu_seqlens, const int32_t* start_lens, const int32_t* positions,
                           const float* inv_freq, int num_freq, int interleaved, const void* q_weight,
                           const void* k_weight, int weight_type, float eps, int B, int Hq, int Hkv, int d, int total,
                           void* stream);

/*
 * attn_fwd_prompt -- attn_fwd over packed sequences whose query heads share K/V heads.
 *   Q, O [total_q, Hq, d], K, V [total_k, Hkv, d]: device bf16 with strides (token, head) as in
 *         attn_qk_rotate, positive here.  Hq is a multiple of Hkv: query head h reads K/V head
 *         h / (Hq / Hkv).  LSE fp32 [Hq, total_q].
 *   cu_seqlens_q, cu_seqlens_k, max_seqlen_q, and the most rows and tiles: as attn_fwd_varlen (rows
 *         outside every sequence are left as they were, rows past max_seqlen_q may be; a sequence's keys
 *         are rows cu_seqlens_k[b] .. cu_seqlens_k[b + 1] - 1).  causal: bottom-right aligned, so a
 *         sequence with more keys than queries is a prompt over its prefix.
 *   What K and V hold where a row does not look, infinities and NaN among it, does not reach the row.
 *   workspace  device, attn_prompt_workspace_bytes(...) bytes, 16-byte aligned, this call's own until
 *         it is done: few query tiles over many keys are then split along the keys.  NULL: they are not.
 *   Asynchronous, allocates nothing.  Errors as attn_fwd.
 */
attn_status attn_fwd_prompt(const void* Q, const void* K, const void* V, void* O, float* LSE, const int64_t* q_strides,
                            const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int Hq, int Hkv,
                            int max_seqlen_q, int total_q, int total_k, int d, float scale, int causal, void* workspace,
                            size_t workspace_bytes, void* stream);
/* Workspace with which attn_fwd_prompt splits keys, in bytes; 0: such a call would not (or bad sizes). */
size_t attn_prompt_workspace_bytes(int B, int Hq, int max_seqlen_q, int total_q, int total_k, int d);

/*
 * attn_cache_weigh -- the attention weight that cached keys receive from a call's queries.
 *   Q, cu_seqlens_q, ctx_lens, block_table: as attn_fwd_tree without a mask (token i of a sequence
 *         sees positions up to ctx_lens[b] + i), with any number of tokens a sequence, whose K are in
 *         the cache already; e.g. a prompt's last tokens, or all of them.  LSE fp32 [Hq, total_q]:
 *         what the attention of these queries returned (attn_fwd_tree, attn_fwd_prompt,
 *         attn_fwd_varlen), with the same scale.  The cache's values are not used (v and v_scale may
 *         be NULL).
 *   weights, out  device fp32 [num_pages, num_heads, page_size]:
 *           out[p] = decay * weights[p] + sum exp(scale * q . k_p - LSE)
 *         over the rows of the key's head (all tokens that see p, all heads of the group).  Positions
 *         from ctx_lens[b] on, which the call's tokens brought, start from 0, and with decay = 0
 *         weights is not read (may be NULL).  out may be weights itself, or another pool of the same
 *         layout (drafts that may be taken back).  Only positions of sequences with tokens in the
 *         call are written, and no page may be theirs twice.  A row that saw nothing (LSE = -inf)
 *         adds nothing.
 *   scale must be at least 2^-100, |LSE| / scale below 2^127, and max_pages * page_size at most 2^31 -
 *   2^17.  Nothing is added atomically: the
 *   same call gives the same bits.  Asynchronous, allocates nothing; device-side timeouts through
 *   attn_status_sync or attn_cache_check.
 */
attn_status attn_cache_weigh(const void* Q, const float* LSE, const attn_cache* cache, const float* weights, float* out,
                             const int32_t* block_table, int max_pages, const int32_t* cu_seqlens_q,
                             const int32_t* ctx_lens, int B, int Hq, int total_q, float scale, float decay,
                             void* stream);

/*
 * attn_cache_evict -- cut sequences to `keep` tokens a head by their weights.
 *   lens  device int32 [B]: the sequences' tokens (clamped to [0, max_pages * page_size]).
 *   weights  device fp32 [num_pages, num_heads, page_size] (attn_cache_weigh).  Every (sequence, head)
 *         with more than `keep` tokens keeps its first `sink`, its last `recent` (together at most
 *         keep) and, of those between, the ones with the largest weights; of equal ones the first,
 *         NaN counts as -inf.  Heads choose for themselves.
 *   The rows kept (K, V, scale codes, weights) move, in order, to places 0, 1, ... of the pages that
 *         out_table (device int32 [B, out_max_pages]) names, which must be pages that no sequence
 *         of the call reads and no place names twice; or, out_table NULL, of the sequence's own
 *         pages, which then must be no other sequence's of the call.
 *   kept  device int32 [B, num_heads, keep]: the positions kept, increasing; -1 past the sequence's
 *         tokens.  out_lens device int32 [B]: min(lens, keep); no part of lens.
 *   keep and max_pages * page_size are at most 2^31 - 2^17.
 *   Positions without a page count as weight -inf and are packed as zeros of weight 0, places without
 *         one are not written; both are reported by attn_cache_check.
 *   Asynchronous, allocates nothing.
 */
attn_status attn_cache_evict(const attn_cache* cache, float* weights, const int32_t* block_table, int max_pages,
                             const int32_t* out_table, int out_max_pages, const int32_t* lens, int32_t* kept,
                             int32_t* out_lens, int B, int keep, int sink, int recent, void* stream);

/* attn_status_sync, then ATTN_ERR_BAD_PAGE if a cache call on the current device has met a
 * position without a page since the last check (read and cleared with plain copies). */
attn_status attn_cache_check(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H_ */
