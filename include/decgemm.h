/*
 * decgemm.h -- C ABI of a GB300 (sm_103a) library for the weight-bandwidth-
 * bound decode step of a large MoE transformer at batch 1-64.
 *
 * Conventions for every call below
 * --------------------------------
 *  - Pointers named x, W, y, out, ... are DEVICE pointers owned by the caller.
 *    The library never frees or retains them after the call's kernels end.
 *  - bf16 means IEEE bfloat16 (the upper half of a binary32 word). Matrices
 *    are dense row-major: a [R,C] matrix has element (r,c) at r*C + c.
 *  - Activations, weights and outputs must be 16-byte aligned, and every
 *    reduction length (K, H, I) a multiple of 8, because weights and
 *    activations move as 16-byte vectors and TMA tiles.
 *  - `stream` is a cudaStream_t passed as void*; NULL is the legacy default
 *    stream. Every call only enqueues work: no host synchronisation, no
 *    device-to-host copy. Results are ready once the stream reaches them.
 *  - Return value: DEC_OK (0) or a negative DEC_E* code. Nothing throws
 *    across this boundary. Argument errors are detected on the host before
 *    any launch. A device-side wait that gives up (see dec_sync_check) is
 *    reported as DEC_ETIMEOUT by dec_sync_check or by the next call.
 *  - The library owns a per-device workspace (split-K partials, arrival
 *    counters, routing tables, MoE intermediates), one side stream for the
 *    shared expert, and events. They are created on first use; a larger shape
 *    gets a larger one, and all are released by dec_shutdown only, so that a
 *    captured graph stays valid until then. Calls that may
 *    allocate must not be the first ones issued inside a CUDA graph capture:
 *    make one call of each shape outside capture first (of the paged-cache
 *    calls, one that uses the workspace). Calls that share the
 *    workspace must be ordered on one stream (the library orders its own
 *    side stream).
 *
 * Sources. The method is described, in prose only, by web pages on the Kimi
 * K3 specialised decode path for GB300. The ones cited below:
 *   [tune-shapes]  "vLLM 如何用智能体辅助优化 Kimi K3 解码性能", Part 1 §1
 *                  "针对工作负载调优形状" (small-matrix kernel at batch 1-2,
 *                  split-K kernel at larger batch).
 *   [moe-overlap]  same page, Part 1 §3 "改进 MoE 调度与重叠" (router,
 *                  routed experts, shared expert on its own stream).
 *   [prefetch]     same page, Part 1 §4 "将即将使用的权重预取到缓存"
 *                  (side-stream kernel that warms the cache with upcoming
 *                  weights).
 *   [trace-path]   same page, Part 2 §1 "隔离变更" (the optimised path must be
 *                  traceable at run time: when it is chosen and how execution
 *                  returns to the standard path).
 */
#ifndef DECGEMM_H
#define DECGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Error codes. */
#define DEC_OK            0
#define DEC_EINVAL       -1  /* NULL required pointer, bad size, misaligned pointer, K % 8 != 0 */
#define DEC_EUNSUPPORTED -2  /* outside the decode envelope: M > 64, topk > 32 or > E, E > 1024 (the
                                paged cache's limits: see dec_kv_view and its calls) */
#define DEC_ECUDA        -3  /* a CUDA runtime call or a launch failed */
#define DEC_ETIMEOUT     -4  /* a bounded device-side wait gave up */
#define DEC_ENOMEM       -5  /* the workspace could not be allocated */
#define DEC_ENODEV       -6  /* no sm_103 device is current */
#define DEC_EBOUNDS      -7  /* a device-side index check failed (DEC_DEBUG builds), or a paged-cache
                                call met a length, page or sequence out of range */

/* Kernel regimes reported by dec_last_choice (low 8 bits). */
#define DEC_REGIME_NONE   0
#define DEC_REGIME_SMALLM 1  /* CUDA-core small-matrix kernels, M <= 2 */
#define DEC_REGIME_MMA    2  /* mma.sync: split-K at 3 <= M <= 16, whole-row slabs at M <= 16 */
#define DEC_REGIME_TC     3  /* split-K with tcgen05 tensor cores and TMEM, M >= 17 */

/*
 * dec_linear -- decode projection y = x·Wᵀ. [tune-shapes]
 *
 *   x : [M,K] bf16 activations          W : [N,K] bf16 weights (row n = output n)
 *   y : [M,N] bf16 output               1 <= M <= 64, N >= 1, K >= 8, K % 8 == 0
 *
 * Accumulates in fp32 and rounds once to bf16 (nearest even). The kernel is
 * chosen from M: M <= 2 the small-matrix kernels; 3 <= M <= 16 split-K on
 * mma.sync; M >= 17 split-K on tcgen05 (at exactly 16 tokens mma.sync streams
 * faster). For 1-16 tokens, when K % 64 == 0 and slabs of 16, 32, 48 or 64 whole
 * weight rows per CTA fill between three quarters of the SMs and all of them,
 * no CTA splits K (the sum over K stays inside the CTA; dot products on
 * mma.sync, reported as DEC_REGIME_MMA); for 1-2 tokens where only slabs of 8
 * rows fill the SMs, the same on the CUDA cores; otherwise split-K.
 * Split-K partial sums are reduced in a fixed order (by the last-arriving CTA
 * of each output tile, or -- when N has few 128-row tiles, on every kernel --
 * by the CTAs of one thread-block cluster per tile, in rank order), so the
 * result is identical from run to run. The environment variable
 * DEC_FORCE=smallm|mma|tc overrides the choice (smallm only for M <= 2: the
 * CUDA-core kernels, slabs of 8, 16 or 32 rows included); DEC_FORCE=splitk
 * keeps 1-16 tokens on the split-K kernels.
 * Errors: DEC_EINVAL, DEC_EUNSUPPORTED, DEC_ECUDA, DEC_ENOMEM.
 */
int dec_linear(const void* x, const void* W, void* y, int M, int N, int K, void* stream);

/*
 * dec_linear_residual -- y = bf16(res + x·Wᵀ), the projection with the residual
 * add fused into its epilogue (accumulate in fp32, add res in fp32, round
 * once). res is [M,N] bf16 and may alias y. Same rules as dec_linear.
 */
int dec_linear_residual(const void* x, const void* W, const void* res, void* y,
                        int M, int N, int K, void* stream);

/*
 * dec_linear_ex -- dec_linear with a row stride for x and an optional residual:
 * y = bf16(x·Wᵀ), or bf16(res + x·Wᵀ) when res is not NULL, where row m of x
 * starts ldx elements after row m-1 (ldx >= K, ldx % 8 == 0). A column slice
 * of a wider activation -- the q part of a fused q|kv projection's output,
 * say -- is then read in place. res ([M,N] bf16) may alias y. x must be
 * 16-byte aligned. Errors as dec_linear; DEC_EINVAL also for a bad ldx.
 */
int dec_linear_ex(const void* x, int ldx, const void* W, const void* res, void* y,
                  int M, int N, int K, void* stream);

/*
 * dec_linear_splitk -- dec_linear with the split factor forced to S
 * (1 <= S <= min(256, ceil(K/128))): the grid has S CTAs per 128-row output
 * tile and each takes an equal share of the tile's 128-wide K chunks (shares
 * differ by at most one chunk when S does not divide the chunk count). A test
 * and tuning hook for the split-K regime. [tune-shapes]
 */
int dec_linear_splitk(const void* x, const void* W, void* y, int M, int N, int K,
                      int S, void* stream);

/*
 * moe_decode -- one MoE decode block. [moe-overlap]
 *
 *   x    : [M,H] bf16 token activations, 1 <= M <= 64
 *   Wr   : [E,H] bf16 router weights
 *   W13  : [E,2I,H] bf16; for expert e, rows 0..I-1 are the gate projection W1
 *          and rows I..2I-1 the up projection W3
 *   W2   : [E,H,I] bf16 down projections
 *   Ws13 : [2I,H] bf16 shared-expert gate/up, Ws2 : [H,I] bf16 shared down;
 *          both NULL for a block without a shared expert
 *   out  : [M,H] bf16 output
 *   topk_idx : optional [M,topk] int32 output, topk_w : optional [M,topk] fp32
 *
 * Computes, per token m:
 *   logits = x·Wrᵀ (fp32, not rounded);
 *   idx    = the topk largest logits, ordered by (value desc, index asc);
 *   g_j    = exp(l_j - l_max) / sum_{j' < topk} exp(l_j' - l_max);
 *   h      = silu(x·W1ᵀ) * (x·W3ᵀ) per chosen expert (rounded to bf16);
 *   out    = bf16( sum_{j=0..topk-1} g_j · h_j·W2ᵀ  +  shared(x) ).
 * Only the chosen experts' weights are read: each once per call, or once per
 * group of 32 tokens if more than 32 tokens chose it. Kernels on `stream`:
 * router projection with the top-k (one warp per token, in the router's last
 * cluster), schedule + token gather, expert gate/up with SwiGLU, expert down,
 * combine. The shared expert runs on a library-owned side stream of the
 * lowest priority that waits on `stream` at entry: its kernels take the SMs
 * the router leaves free and stream their weights while routing runs;
 * `stream` joins it before the combine.
 * The number of active experts never returns to the host.
 * Limits: H % 8 == 0, I % 8 == 0, 1 <= topk <= min(E, 32), E <= 1024.
 * Errors: DEC_EINVAL, DEC_EUNSUPPORTED, DEC_ECUDA, DEC_ENOMEM.
 */
int moe_decode(const void* x, const void* Wr, const void* W13, const void* W2,
               const void* Ws13, const void* Ws2, void* out,
               int M, int H, int E, int topk, int I,
               int32_t* topk_idx, float* topk_w, void* stream);

/*
 * moe_decode_residual -- moe_decode whose combine adds a residual:
 * out = bf16(res + sum_j g_j·o_j + shared). res is [M,H] bf16 and may alias x
 * or out (the residual stream of a decode layer is usually the block's own
 * input). out may alias x: x is last read before the combine starts.
 */
int moe_decode_residual(const void* x, const void* Wr, const void* W13, const void* W2,
                        const void* Ws13, const void* Ws2, const void* res, void* out,
                        int M, int H, int E, int topk, int I,
                        int32_t* topk_idx, float* topk_w, void* stream);

/*
 * moe_decode_latent -- an MoE decode block whose routed experts work on a
 * latent width L. [moe-overlap] The router scores and the latent input
 * projection are computed as one product over a stacked weight (the pages
 * merge the two into one matrix multiplication); the steps after it are the
 * library's reading of the block, the pages naming only that product:
 *
 *   x    : [M,H] bf16               Wrl : [E+L,H] bf16, rows 0..E-1 the router,
 *                                         rows E..E+L-1 the latent input projection
 *   W13  : [E,2I,L] bf16 (gate rows 0..I-1, up rows I..2I-1)   W2 : [E,L,I] bf16
 *   Wup  : [H,L] bf16 up-projection     Ws13 [2I,H] / Ws2 [H,I]: shared expert on x
 *   res  : optional [M,H] bf16 residual (may alias x or out)   out : [M,H] bf16
 *
 *   sc     = x·Wrlᵀ (fp32);  logits = sc[:, :E];  lat = bf16(sc[:, E:])
 *   idx, g = top-k of logits, renormalised softmax gates (as moe_decode)
 *   z      = bf16( sum_{j=0..topk-1} g_j · expert_{idx_j}(lat) )   (width L)
 *   out    = bf16( res + (z·Wupᵀ + shared(x)) )   (fp32 sum, one rounding)
 *
 * Kernels on `stream`: the router over E+L rows with the top-k, schedule +
 * gather of the latent rows (rounded to bf16 as they are copied), expert
 * gate/up, expert down, the gate-weighted sum z, the up-projection, and the
 * final sum; the shared expert on the library's side stream as in
 * moe_decode. Limits as moe_decode; L >= 8, L % 8 == 0.
 * Errors: DEC_EINVAL, DEC_EUNSUPPORTED, DEC_ECUDA, DEC_ENOMEM.
 */
int moe_decode_latent(const void* x, const void* Wrl, const void* W13, const void* W2,
                      const void* Wup, const void* Ws13, const void* Ws2, const void* res,
                      void* out, int M, int H, int L, int E, int topk, int I,
                      int32_t* topk_idx, float* topk_w, void* stream);

/*
 * l2_prefetch -- enqueue a light kernel on `stream` that pulls
 * [ptr, ptr + bytes) into L2, so that a later kernel reading the range hits
 * in cache. [prefetch] It has no data dependency and changes no memory;
 * ordering against other streams is the caller's. bytes is rounded down to a
 * multiple of 16 and capped at half the L2 size. ptr must be 16-byte aligned.
 */
int l2_prefetch(const void* ptr, size_t bytes, void* stream);

/*
 * dec_add -- out = bf16(a + b) elementwise over n bf16 values (the residual
 * add of a decode layer when it is not fused). out may alias a or b.
 */
int dec_add(const void* a, const void* b, void* out, size_t n, void* stream);

/*
 * dec_last_choice -- regime and split of this thread's last dec_linear* call.
 * [trace-path] Returns regime | (S << 8) | (C << 16) | (Wd << 17) | (Sl << 18)
 * where regime
 * is a DEC_REGIME_* value, S the number of CTAs that share each output tile's
 * K range (1 = none), rounded up, C is 1 when those S CTAs form one
 * thread-block cluster and sum their partial tiles through distributed shared
 * memory (small projections: few 128-row tiles, M <= 16), 0 when the split is
 * the stream-K one with a last-arriver fixup, and Wd is 1 when the output
 * tiles are 256 rows high (large projections at M <= 16), and Sl is 1 when
 * each CTA owned whole weight rows (1-16 tokens, S = 1). DEC_REGIME_NONE before
 * any call.
 */
int dec_last_choice(void);

/* dec_last_grid -- CTAs launched by this thread's last dec_linear* call. */
int dec_last_grid(void);

/* dec_strerror -- static text for a DEC_* code. */
const char* dec_strerror(int code);

/*
 * dec_sync_check -- synchronise `stream` (and the library's side stream),
 * then read and clear the device status words that kernels set when a bounded
 * wait gives up: the library's own and the one in dec_linear_noalloc's fixed
 * array. Returns DEC_OK, DEC_ETIMEOUT, DEC_EBOUNDS as described there, or
 * DEC_ECUDA if the synchronisation itself failed. Where a wait gave up and a
 * check failed it returns DEC_ETIMEOUT, and the next call DEC_EBOUNDS.
 * Allocates nothing: in a process that has only called dec_linear_noalloc it
 * sets up no workspace, stream or event.
 */
int dec_sync_check(void* stream);

/*
 * dec_set_wait_timeout_ns -- upper bound, in nanoseconds of %globaltimer, on
 * every device-side wait of later launches (default 2e9). A wait that runs
 * out sets the status word, drains its own copies in flight and returns.
 * Returns the previous value.
 */
long long dec_set_wait_timeout_ns(long long ns);

/*
 * dec_selftest_timeout -- launch one CTA that waits, with the bounded wait
 * used by every kernel, on a barrier that nothing will complete, with limit
 * `ns`. The wait must give up; dec_sync_check then returns DEC_ETIMEOUT.
 * Exercises failure detection without faulting or hanging the GPU.
 */
int dec_selftest_timeout(long long ns, void* stream);

/*
 * dec_debug_build -- 1 for the index-checking build of this library
 * (libdecgemm_debug.so, compiled with DEC_DEBUG), 0 otherwise. In that build
 * every index a kernel computes into a global buffer (output rows and
 * columns, split-K slots and counters, expert group tables, pair positions,
 * gathered token rows) is checked against the buffer's extent; an access out
 * of range is skipped, and dec_sync_check returns DEC_EBOUNDS.
 * dec_debug_check_site -- the source line of the first failed check and the
 * offending index, as read by the dec_sync_check that returned DEC_EBOUNDS;
 * returns 1 if there was one, 0 if not.
 */
int dec_debug_build(void);
int dec_debug_check_site(int* line, long long* index);

/*
 * dec_debug_stall -- of the index-checking build: with on != 0 the calls of
 * dec_linear_w4 and dec_linear_w4_mx from then on wait in vain for one more arrival
 * on their tokens, give up after the wait bound, and end without a result;
 * dec_sync_check then returns DEC_ETIMEOUT. Exercises their way out without
 * faulting or hanging the GPU. Returns what was set before (0 or 1), or
 * DEC_EUNSUPPORTED from the other build.
 */
int dec_debug_stall(int on);

/* dec_launch_count -- kernels launched by this library since load (all threads). */
long long dec_launch_count(void);

/*
 * dec_probe_begin / dec_probe_end -- time every launch of one kernel kind with
 * CUDA events recorded on the stream the kernel is launched on.
 * kind: 0 = routed-expert gate/up kernel, 1 = routed-expert down kernel,
 *       2 = projection kernels, 3 = router projection kernel, 4 = combine kernel.
 * dec_probe_begin arms the probe for up to `capacity` launches (0 disarms).
 * dec_probe_end synchronises those events and returns, through the
 * pointers, the summed duration in ms and the number of launches timed.
 */
int dec_probe_begin(int kind, int capacity);
int dec_probe_end(double* total_ms, int* launches);

/*
 * dec_linear_noalloc -- dec_linear for callers that must not allocate device
 * memory. The pages describe no counterpart: this entry point exists for
 * integration, not for the method.
 *
 * Who needs it: code whose device memory is owned by someone else (a
 * framework's caching allocator that has reserved the GPU, an engine with a
 * memory budget fixed before the first request) and latency-critical loops
 * in which cudaMalloc/cudaFree, which may synchronise the device, must never
 * run. dec_linear allocates its split-K workspace on first use and grows it
 * for larger shapes; this variant allocates nothing and calls no allocating
 * routine.
 *
 * Same arguments, layouts and result as dec_linear (fp32 accumulation, one
 * bf16 rounding), computed by the same weight-streaming kernel: CUDA-core for
 * M <= 2, mma.sync for 3 <= M <= 16. Its split-K partial sums and arrival
 * counters live in one 4 MiB array compiled into the library; every GPU that
 * loads the library holds that array until the process exits.
 *
 * Limits (DEC_EUNSUPPORTED beyond them): M <= 16; ceil(N/128) <= 16384 output
 * tiles; the partial tiles of the launch, min(SMs, ceil(N/128)*ceil(K/128))
 * CTAs x 2 x 128 x (8 if M <= 2 else 16) floats, within 4 MiB - 64 KiB - 256 B
 * (a 152-SM GB300 needs at most 2.4 MiB, so every N and K fit there).
 * Argument errors as for dec_linear (DEC_EINVAL); DEC_ENODEV without an sm_103
 * device; DEC_ECUDA if a runtime call fails.
 *
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture. Every call shares the one array, which keeps the
 * last call's contents (each call clears the counters it uses): calls that can
 * overlap on the GPU -- on unordered streams or from several host threads --
 * race and corrupt each other's results. A bounded device-side wait that
 * gives up ends the kernel as in dec_linear (y is then incomplete) and sets a
 * status word in the fixed array; the word is not cleared by later calls, and
 * dec_sync_check reports it as DEC_ETIMEOUT (and clears it) -- call it before
 * trusting y where a give-up must not pass unseen. A first call made while
 * `stream` is being captured returns DEC_EINVAL (the set-up above cannot run
 * inside a capture). Does not update dec_last_choice or dec_launch_count.
 */
int dec_linear_noalloc(const void* x, const void* W, void* y, int M, int N, int K, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The paged key/value cache: what stands between a layer's q|k|v projection
 * and its o projection, and the management of the cache's pages. These calls
 * are the library's own; the pages describe no counterpart (the layer they
 * describe is taken without its attention core).
 *
 * A cache of one layer is pages of page_size positions, each holding
 * [2][heads][page_size][dim] bf16: the keys of every key/value head, then the
 * values. Row s of a page table lists the pages of sequence s in order; -1
 * marks an unused entry. A sequence's positions are 0 .. kv_len-1, and a
 * call's new tokens are always its last ones: kv_len counts them.
 *
 * Lengths, page numbers and sequence numbers are device data, read by the
 * kernels (so that a captured graph follows them from step to step). One that
 * is out of range never makes an access out of range: what it names is left
 * out (or read as zeros), and dec_sync_check reports DEC_EBOUNDS.
 */

/* A layer's cache and the batch of sequences that a call works on. */
typedef struct dec_kv_view {
  void* cache;             /* device; 16-byte aligned */
  int64_t page_stride;     /* elements from one page to the next (a multiple of 8) */
  int32_t pages, heads;    /* pages of the pool; key/value heads */
  int32_t page_size, dim;  /* 16, 32, 64, 128 or 256 positions; 64 or 128 elements of a head */
  const int32_t* table;    /* device [table_rows][table_stride] */
  int64_t table_stride;    /* elements from one row to the next */
  int32_t width;           /* entries of a row; width * page_size at most 2^31 - 256 */
  int32_t table_rows;      /* rows of table, and entries of kv_len */
  const int32_t* rows;     /* device [batch]: the row (and kv_len entry) of each sequence of the
                              batch; NULL: sequence b has row b */
  const int32_t* cu_q;     /* device [batch+1]: sequence b's new tokens are cu_q[b] .. cu_q[b+1]-1 */
  const int32_t* kv_len;   /* device [table_rows]: positions, the new tokens included */
  int32_t batch;           /* 1 .. 1024 sequences; some may have no new token */
  int32_t max_q;           /* the most new tokens of one sequence, as far as the caller knows: it
                              chooses the kernel, not the result. 0: unknown, taken as all of
                              the call's tokens (slower for a batch of short steps) */
} dec_kv_view;

/*
 * kv_append -- norm and rotation of the new tokens' queries and keys, head by
 * head, and the append of their keys and values to the cache, in one pass.
 *
 *   qkv  : [tokens, (q_heads + 2*heads)*dim] bf16, rows ldqkv elements apart: the
 *          query heads, the key heads, the value heads (a fused projection's output)
 *   wq, wk : [dim] bf16 norm weights of queries and keys; both NULL: no norm
 *   rope : [rope_len, rot] fp32, for each position rot/2 cosines, then rot/2 sines
 *   positions : optional [tokens] int32, the row of rope of each token; NULL: its
 *          position in its sequence
 *   q    : [tokens, q_heads*dim] bf16 output, rows ldq elements apart; may be qkv
 *
 * Per query or key head x:  y = x * rsqrt(mean(x^2) + eps) * w;  then on its
 * first rot elements (a multiple of 16, at most dim) each pair (a, c) becomes
 * (a cos - c sin, c cos + a sin), pairs being (i, i + rot/2), or (2i, 2i+1) with
 * interleaved. fp32 throughout, rounded once to bf16. Values are copied. Token
 * t of sequence b goes to position kv_len - (its new tokens) + t. Tokens past
 * cu_q[batch] belong to no sequence and are left alone (a padded batch). A row
 * number outside rope is taken as the nearest one (and DEC_EBOUNDS reported).
 */
int kv_append(const dec_kv_view* kv, const void* qkv, int64_t ldqkv, const void* wq, const void* wk,
              float eps, const float* rope, int rope_len, int rot, int interleaved,
              const int32_t* positions, void* q, int64_t ldq, int tokens, int q_heads, void* stream);

/*
 * kv_attention -- attention of the new tokens over the cache.
 *
 *   q   : [tokens, q_heads*dim] bf16, rows ldq elements apart; q_heads a multiple of
 *         heads, at most 64 query heads per key head; query head h reads key head
 *         h / (q_heads/heads)
 *   out : [tokens, q_heads*dim] bf16, rows ldo elements apart
 *   lse : optional [tokens, q_heads] fp32
 *
 * Per token at position i and head, over the positions j it sees (j <= i, and
 * j > i - window if window > 0):
 *   s_j = scale * q·k_j;  lse = log sum_j exp(s_j);  out = sum_j exp(s_j - lse) v_j
 * Scores, maximum, sum and output are fp32; the weights enter the product with
 * the values as bf16; out is rounded once. A token that sees nothing (its
 * position is negative: kv_len below its chunk) gets out = 0, lse = -inf. What
 * lies past a sequence's end in its last page is never used, whatever it is, and
 * with a window neither are the table's entries of pages before the first token's
 * window (a cache may have dropped them).
 * The result is the same from run to run. Rows of tokens past cu_q[batch] are
 * left alone. Uses the library's workspace: order such calls on one stream.
 */
int kv_attention(const dec_kv_view* kv, const void* q, int64_t ldq, void* out, int64_t ldo, float* lse,
                 int tokens, int q_heads, float scale, int window, void* stream);

/* kv_last_attention -- DEC_REGIME_* of this thread's last kv_attention call. */
int kv_last_attention(void);

/* The pages of all layers of a cache, and the state of its sequences. */
typedef struct dec_kv_pool {
  void* data;              /* device; 16-byte aligned */
  int64_t layer_stride;    /* bytes from one layer's pages to the next's */
  int64_t page_stride;     /* bytes from one page to the next */
  int64_t page_bytes;      /* bytes of a page of one layer; all three multiples of 16 */
  int32_t layers, pages;   /* pages: at most 2^19 */
  int32_t page_size;       /* positions of a page, a power of two */
  int32_t* refs;           /* device [pages]: table entries that hold a page; 0: free */
  int32_t* table;          /* device [seqs][table_stride]: pages of a sequence, -1 past its last */
  int64_t table_stride;
  int32_t width;           /* entries of a table row */
  int32_t* lens;           /* device [seqs]: positions of a sequence */
  int32_t seqs;
  int32_t* info;           /* optional device [3], written by kv_resize, kv_free, kv_fork and
                              kv_compact: pages that were lacking (0: done), pages free after
                              the call, pages copied */
} dec_kv_pool;

/*
 * kv_resize -- set the lengths of n sequences (1 .. 1024, all different): pages
 * past the new length are given back, pages up to it are taken. New pages are
 * the lowest free ones, in the order of the requests. A sequence cut inside a
 * page that others hold too gets a copy of that page. All or nothing: if the
 * free pages do not suffice nothing changes and info[0] says how many are
 * lacking. A request that the table cannot hold or that names no sequence is
 * left out (DEC_EBOUNDS from dec_sync_check).
 *
 * kv_free -- kv_resize to length 0.
 *
 * kv_fork -- sequence dst[i] becomes a copy of src[i] (no sequence both a source
 * and a copy; copies all different): it shares the full pages and gets a copy
 * of the last one if that is partly filled, so that both can be appended to.
 * Pages that dst[i] held are given back. All or nothing, as kv_resize.
 *
 * Pages that a call gives back are free from the next call on. kv_resize, kv_fork
 * and kv_compact use the library's workspace, as kv_attention does: order such
 * calls on one stream, and make a first one before capturing them in a graph.
 * The workspace has one size, whatever the calls (about 50 MB).
 */
int kv_resize(const dec_kv_pool* pool, const int32_t* seqs, const int32_t* lens, int n, void* stream);
int kv_free(const dec_kv_pool* pool, const int32_t* seqs, int n, void* stream);
int kv_fork(const dec_kv_pool* pool, const int32_t* src, const int32_t* dst, int n, void* stream);

/* kv_copy -- copy page src[i] to page dst[i] in every layer, i < n (device lists; no
 * page both read and written, none written twice). */
int kv_copy(const dec_kv_pool* pool, const int32_t* src, const int32_t* dst, int n, void* stream);

/* kv_compact -- move pages so that the n pages in use are pages 0 .. n-1: those at or
 * past n go, in order, to the free places before n; table and refs follow. */
int kv_compact(const dec_kv_pool* pool, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The norm of the residual stream, and projections with 4-bit weights: the
 * library's own calls, as the paged cache's are. Numbers in 4 and 8 bits come in
 * blocks of 32 with a shared power of two (the OCP microscaling formats MXFP4 and
 * MXFP8): a scale byte b stands for 2^(b - 127), 255 for NaN.
 *
 * dec_rmsnorm -- y = h * rsqrt(mean(h^2) + eps) * w over each row, with
 * h = bf16(x + res), or h = x when res is NULL.
 *
 *   x, res, h, y : [rows, H] bf16, rows ldx, ldres, ldh, ldy elements apart (each at
 *          least H and a multiple of 8); h is written with res only
 *   w    : [H] bf16;  H a multiple of 8, at most 65536;  eps >= 0
 *
 * The sum of squares is that of the rounded h, in fp32 (past its range the root is 0,
 * and y of finite h too); y is fp32 rounded once.
 * h may be x or res, and y may be x or res, with the same row stride (y not h).
 * Otherwise outputs overlap nothing (outputs that begin where an operand does are refused). Errors: DEC_EINVAL, DEC_EUNSUPPORTED (H),
 * DEC_ECUDA.
 *
 * dec_rmsnorm_mx -- the same y in 8 bits: q [rows, H] e4m3 (rows ldq apart, a
 * multiple of 16) and scales [rows, H/32] bytes (rows ldscales apart); H a multiple
 * of 32. For each 32 values with largest magnitude a the scale is 2^e with
 * e = ceil(log2(a / 448)), at least -127 (for a = 0 too), and q = e4m3(y / 2^e), to
 * nearest even. A group with a value that is not finite: scale 255, q NaN.
 */
int dec_rmsnorm(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w, float eps,
                void* h, int64_t ldh, void* y, int64_t ldy, int rows, int H, void* stream);
int dec_rmsnorm_mx(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w, float eps,
                   void* h, int64_t ldh, void* q, int64_t ldq, void* scales, int64_t ldscales, int rows,
                   int H, void* stream);

/*
 * 4-bit weights [N, K]: W[n][k] = v(code) * 2^(b - 127), b the scale byte of k's 32
 * (aligned) k; a code has its sign in bit 3 and v = 0, .5, 1, 1.5, 2, 3, 4, 6 by
 * its low bits. They lie in units of 128 rows x 128 k:
 *   q      : [ceil(N/128)][ceil(K/128)][128 rows][64 bytes], 128-byte aligned; element
 *            2i of a row's 128 k in the low half of byte i
 *   scales : [ceil(N/128)][ceil(K/128)][32][4][4], 16-byte aligned: row n, group g of
 *            the unit's four at [n % 32][n % 128 / 32][g]
 * What lies past N is read and has no effect; past K, where the tokens read as 0,
 * neither has what is not a scale of 255.
 *
 * dec_quant_w4 -- bf16 weights W [N, K] (rows ldw elements apart, a multiple of 8;
 * K a multiple of 8) in that form, what lies past N and K included (codes 0). For
 * each 32 with largest magnitude a: 2^e with e = ceil(log2(a / 6)), at least -127 (for
 * a = 0 too), codes to nearest, ties to the even code. A group with a value that is
 * not finite: scale 255, codes 0.
 */
int dec_quant_w4(const void* W, int64_t ldw, void* q, void* scales, int N, int K, void* stream);

/*
 * dec_linear_w4 -- y = bf16(x·Wᵀ), or bf16(res + x·Wᵀ) when res is not NULL.
 *
 *   x    : [M, K] bf16, rows ldx elements apart (at least K, a multiple of 8);
 *          1 <= M <= 64, K a multiple of 8
 *   res, y : [M, N] bf16; y may be res. Otherwise y and work overlap nothing (refused where
 *          they begin where another operand does)
 *   work : dec_linear_w4_work(M, K) bytes of device memory, 16-byte aligned, that the
 *          call may write until its kernels end; NULL where that is 0 (M <= 16, and
 *          what is refused). The
 *          library's own workspace is not used: calls with work spaces of their own
 *          may run at once.
 *
 * The tensor cores take 4-bit weights with 8-bit tokens. A bf16 token value enters
 * as the sum of two e4m3 numbers, each with a scale for 32 k. With 2^e the least power of
 * two that brings the largest magnitude of the 32 to 448 or less (e at least -123), values
 * of at least 2^(e-6) are exact, those below off by at most 2^(e-14): 2^-13.8 and 2^-21.8
 * of the largest magnitude, where it is just above 224 * 2^e.
 * Products are exact, sums fp32, in an order that does not change from run to
 * run; y is rounded once. A token with a value that is not finite gives NaN in
 * all its outputs. W is read while the previous kernel of the stream may still run, as
 * by dec_linear; dec_quant_w4 lets nothing start before it has ended.
 * dec_last_choice, dec_last_grid and the probe say nothing of these calls.
 * Errors: DEC_EINVAL, DEC_EUNSUPPORTED (M > 64, K > 2^29, 2^24 units or more), DEC_ECUDA.
 *
 * dec_linear_w4_mx -- the same for tokens in 8 bits: x [M, K] e4m3, rows ldx bytes
 * apart (a multiple of 16), xscales [M, K/32] bytes, rows ldxscales apart; K a
 * multiple of 32. The tokens' values are taken as they are.
 */
int dec_linear_w4(const void* x, int64_t ldx, const void* wq, const void* wscales, const void* res,
                  void* y, int M, int N, int K, void* work, void* stream);
size_t dec_linear_w4_work(int M, int K);
int dec_linear_w4_mx(const void* x, int64_t ldx, const void* xscales, int64_t ldxscales, const void* wq,
                     const void* wscales, const void* res, void* y, int M, int N, int K, void* stream);

/* dec_shutdown -- free the workspace, side stream and events of the current device. */
void dec_shutdown(void);

/* dec_version -- ABI version of this header (major*100 + minor). */
int dec_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DECGEMM_H */
