/*
 * iq.h -- C ABI of the GB300 (sm_103a) DeepSeek-V4 indexer-Q preparation path.
 *
 * Two operations, each an asynchronous launch sequence on a caller stream:
 *
 *  1. iq_fp8_quant_1x128_ue8m0: the packed-UE8M0 FP8 online activation
 *     quantizer of the TokenSpeed PR "perf(deepseek-v4): accelerate indexer Q
 *     and packed FP8 quantization" (Summary; Risk and fallback: contiguous,
 *     aligned BF16 input, K divisible by 128, the packed-UE8M0 scale contract
 *     and the tiny-scale floor), which the TensorRT-LLM PR "Fuse DeepSeek-V4
 *     Indexer Q projection with CuTe DSL" calls fp8_quantize_1x128 with UE8M0
 *     scales (Walkthrough / sequence diagram).
 *
 *  2. iq_prepare_q: the fused indexer-Q projection of the TensorRT-LLM PR
 *     (sequence diagram: FP8 input and UE8M0 scales, block-scaled GEMM "with
 *     RoPE and FP4 epilogue", packed FP4 Q and scales returned; review comment
 *     on the fused epilogue: MXF8 scale vector 32, one 128-column head per MMA
 *     tile) with the Hadamard transform that the TokenSpeed PR applies to the
 *     indexer Q (Summary; Main-rebase compatibility fix).
 *
 * Numbers used throughout (element formats per the OCP FP8 / MX specs):
 *   E4M3: FP8 with 4 exponent bits (bias 7), 3 mantissa bits, max 448.
 *   E2M1: FP4 with 2 exponent bits (bias 1), 1 mantissa bit, max 6.
 *   UE8M0: unsigned 8-bit exponent; byte b encodes 2^(b - 127).
 *   Block scale exponent of a block with largest magnitude a:
 *       e = smallest integer with qmax * 2^e >= max(a, 1e-4)   (qmax 448 or 6)
 *   Element code = round-to-nearest-even(x * 2^-e) in the element format.
 *
 * Memory: the caller owns every buffer (inputs, outputs, workspace).  No call
 * allocates device memory or falls back to another implementation, and none
 * synchronizes the device or the stream except the diagnostics
 * (iq_device_status, iq_selftest_wait_timeout).  Pointers are device pointers unless stated.
 * All calls are asynchronous on `stream`; errors detected on the host are
 * returned before anything is launched.  A return of IQ_OK means the launches
 * were enqueued; a device-side wait that ran out of time is recorded in the
 * device status word (iq_device_status).
 *
 * Thread safety: calls may be made from several host threads.  Shared host
 * state: the per-device set-up done on the first call on a device
 * (architecture check, kernel attributes), which is guarded, and the
 * internal streams and events of iq_prepare_q_host, whose calls on one device
 * enqueue one at a time under a lock.
 */
#ifndef IQ_H_
#define IQ_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  IQ_OK = 0,
  IQ_ERR_ARG = -1,        /* null pointer, M < 0, bad leading dimension */
  IQ_ERR_ALIGN = -2,      /* a pointer or leading dimension breaks the alignment rule */
  IQ_ERR_SHAPE = -3,      /* K <= 0 or K % 128 != 0; a head dimension, page size or head count the cache calls do not take */
  IQ_ERR_ARCH = -4,       /* current device is not compute capability 10.3 (sm_103) */
  IQ_ERR_CUDA = -5,       /* a CUDA runtime call or launch failed */
  IQ_ERR_WORKSPACE = -6,  /* workspace smaller than iq_prepare_q_workspace(M) */
  IQ_ERR_TIMEOUT = -7     /* a device-side wait gave up (see iq_device_status) */
} iq_status;

/* Human-readable name of a status code (static storage). */
const char* iq_status_str(iq_status s);

/* Device-side status word of the current device: bit i set means a wait of
 * kind i ran out of time in some launch since the last reset.  Reads it into
 * *flags (may be NULL) and clears it when `reset` is nonzero.  This call
 * synchronizes with the device (it copies from device memory); it is a
 * diagnostic, not part of the hot path.  Returns IQ_ERR_TIMEOUT when the word
 * was nonzero, IQ_OK otherwise. */
iq_status iq_device_status(uint32_t* flags, int reset);

/* Overrides the time after which a device-side wait gives up, in nanoseconds
 * (default 2e9).  0 restores the default.  Applies to later launches from any
 * thread. */
void iq_set_wait_timeout_ns(uint64_t ns);

/* Diagnostics of the failure handling (no counterpart on the pages).
 *
 * iq_selftest_wait_timeout runs the fused GEMM kernel once on a 256-token
 * problem with its TMA loads left out: the stage barriers its MMA issuer
 * waits on never complete, no MMA is issued, and the producer's, the MMA
 * issuer's and the epilogue's bounded waits give up after timeout_ns with
 * nothing asynchronous in flight.  The kernel then takes its normal give-up
 * and teardown path.  The call resets the status word, launches on `stream`,
 * synchronizes the stream, stores the status bits the launch set in *flags
 * (may be NULL) and resets the word again.  Returns IQ_ERR_TIMEOUT when some
 * wait gave up (the expected result: bits 0, 1 and 2 -- producer, MMA issuer,
 * epilogue -- set, bit 3 -- teardown -- clear), IQ_OK when none did.
 * workspace: iq_selftest_workspace() bytes of device memory, 256-byte
 * aligned, overwritten.  Errors: IQ_ERR_ARG (NULL workspace, timeout 0),
 * IQ_ERR_ALIGN, IQ_ERR_WORKSPACE, IQ_ERR_CUDA, IQ_ERR_ARCH. */
size_t iq_selftest_workspace(void);
iq_status iq_selftest_wait_timeout(void* workspace, size_t ws_bytes, uint64_t timeout_ns, uint32_t* flags,
                                   cudaStream_t stream);

/* Test hook: the next `count` per-device set-ups (the work of the first call
 * on a device) fail as if a CUDA query had failed and return IQ_ERR_CUDA.  A
 * failed set-up is not cached: the next call on the device tries again. */
void iq_debug_fail_next_setups(int count);

/* The FP4 stage's element conversion alone, for testing it directly:
 * codes[i] (low nibble) = E2M1 code of x[i], round to nearest even,
 * saturating at +-6, sign of zero kept -- the conversion both fused GEMM
 * kernels apply to z * 2^-e.  x: n float32, 16-byte aligned; codes: n bytes,
 * 8-byte aligned; n % 8 == 0 (else IQ_ERR_SHAPE).  One kernel launch. */
iq_status iq_debug_e2m1_codes(const float* x, long long n, uint8_t* codes, cudaStream_t stream);

/* Token-count route of the fused GEMM (operation 2).  Calls with
 * 1 <= M <= threshold run the small-M kernel, which swaps the MMA operands
 * (the weights on the MMA's M side, the tokens on its N side: 64 token
 * columns up to 64 tokens, 128 above), the variant the TensorRT-LLM PR routes
 * small token counts to (dispatch thresholds); larger M runs the persistent
 * CTA-pair kernel.  Both compute the same operation;
 * their float32 sums may round differently, within the error the parity rules
 * of operation 2 allow.  The threshold is clamped to [0, IQ_SMALL_M_MAX]; 0
 * sends every M to the CTA-pair kernel.  The default is IQ_SMALL_M_MAX.
 * Process-wide; applies to later calls from any thread (a CUDA graph keeps
 * the route it was captured with).  Returns the previous threshold. */
#define IQ_SMALL_M_MAX 128
int iq_set_small_m_threshold(int max_tokens);

/* The current threshold (see iq_set_small_m_threshold). */
int iq_small_m_threshold(void);

/* Tuning override of the CTA-pair kernel's tiling, for measurements.  By
 * default the kernel takes one head (128 output features) per pair tile up to
 * 256 tokens and two heads (256) above, and orders the pair tiles token-major
 * (consecutive tiles of a CTA pair share their 256 token rows).  tile_n: 128 (one head per tile, two accumulators
 * in tensor memory) or 256 forces that width, any other value restores the
 * default; order: 1 forces feature-major (consecutive tiles share their
 * heads), 2 token-major, 3 interleaved (token-major tiles dealt round-robin
 * to the pairs: pair p takes tiles p, p + P, ...), any other value restores
 * the default.
 * Results are the same under every setting (the same sums in the same order
 * per output).  Process-wide; applies to later calls. */
void iq_set_gemm_tiling(int tile_n, int order);

/* The quantizer fused into the CTA-pair kernel: off (0, the default: the
 * stand-alone quantizer, then the GEMM kernel) or on (1: one launch, see
 * iq_prepare_q).  Results are the same either way; on GB300 the fused launch
 * measured slower at every token count, so it is off unless asked for.  The
 * fused launch always takes two-head tiles; forcing one-head tiles
 * (iq_set_gemm_tiling) turns it off.  Process-wide; applies to later calls;
 * returns the previous setting. */
int iq_set_quant_fusion(int on);

/* Diagnostics: the fused quantizer's warps wait ns nanoseconds (at most 1 ms)
 * before signalling each wave of token rows, so that the GEMM's loads must
 * wait for them.  0 (the default) turns it off.  Process-wide. */
void iq_debug_delay_quant_ns(uint64_t ns);

/* ------------------------------------------------------------------------
 * 1. FP8 1x128 quantizer with packed UE8M0 scales.
 * ------------------------------------------------------------------------ */

/* Number of int32 scale words the quantizer writes for an M x K input:
 * ceil(K / 512) * align_up(M, 4).  Returns 0 when M <= 0 or K <= 0. */
size_t iq_fp8_scale_words(int M, int K);

/* Quantizes x (BF16, row-major [M, ldx], first K columns used) per row and
 * per 1x128 block:
 *   y[m, k]   = E4M3 code of x[m, k] * 2^-e(m, k/128)        (row-major [M, ldy])
 *   scales    = int32 words [ceil(K/512)][align_up(M, 4)] (M-major, the
 *               TMA-aligned layout a DeepGEMM-style consumer reads):
 *               byte j (little-endian) of word [g][m] is the UE8M0 scale byte
 *               e + 127 of block 4g + j of row m; bytes of blocks past K/128
 *               and words of rows m >= M are written as 0.
 * The sign of zero is kept (-0 and values that round to zero from below give
 * code 0x80).  NaN or infinite inputs are outside the contract.
 * Requirements: M >= 0; K > 0 and K % 128 == 0 (else IQ_ERR_SHAPE);
 *   ldx >= K, ldy >= K; x and y 16-byte aligned, ldx % 8 == 0 and
 *   ldy % 16 == 0, scales 4-byte aligned (else IQ_ERR_ALIGN).
 * M == 0 returns IQ_OK without a launch.  One kernel launch, with programmatic
 * stream serialization: its blocks may be scheduled while the preceding
 * kernel on `stream` runs, and they touch no memory before that kernel has
 * completed. */
iq_status iq_fp8_quant_1x128_ue8m0(const void* x_bf16, int M, int K, int ldx,
                                   void* y_e4m3, int ldy, int32_t* scales,
                                   cudaStream_t stream);

/* ------------------------------------------------------------------------
 * 2. Indexer-Q preparation: FP8 quantize -> block-scaled FP8 GEMM -> RoPE ->
 *    Hadamard-128 -> FP4 (E2M1) with 1x32 UE8M0 scales.
 *
 * Fixed shapes: latent dimension K = 1536; Q has 64 heads of 128 dims
 * (N = 8192).  Per token m and head h (n = 128 h + d):
 *   Y[m, n] = sum_kb 2^(eX[m,kb] + eW[h,kb]) * sum_{k in kb} x[m,k] w[n,k]
 *             over 12 blocks kb of 128, x the E4M3 latent codes (operation 1
 *             applied to the BF16 latent), w the weight codes;
 *   RoPE:     NeoX rotation of dims d = 0..63 in pairs (i, i+32) by the angle
 *             position[m] * 10000^(-i/32); dims 64..127 unchanged;
 *   Hadamard: z = H r / sqrt(128), H[i][j] = (-1)^popcount(i & j);
 *   FP4:      per block of 32 consecutive dims, e from qmax 6, codes
 *             E2M1(z * 2^-e) with the sign of zero kept.
 * The pre-quant Q (z) is kept in float32 and is never rounded to BF16.
 * ------------------------------------------------------------------------ */

#define IQ_LATENT_DIM 1536
#define IQ_NUM_HEADS 64
#define IQ_HEAD_DIM 128
#define IQ_Q_DIM 8192

/* Workspace bytes iq_prepare_q needs for M tokens: the E4M3 latent
 * [M, 1536] at offset 0 followed, at the next 256-byte boundary, by its packed
 * scale words [3][align_up(M, 4)], then, at the next 256-byte boundary, the
 * fused quantizer's flags (513 words of 8 bytes: a call counter and one
 * progress word per CTA).  The flags need no initialisation: a progress word
 * counts only if it carries a 48-bit hash of the current call counter and its
 * CTA, which each call advances.  Returns 0 when M <= 0. */
size_t iq_prepare_q_workspace(int M);

/* Arguments:
 *   latent_bf16  [M, 1536] BF16, contiguous, 16-byte aligned.
 *   wq_e4m3      [8192, 1536] E4M3 codes, row-major (row n = output feature n),
 *                16-byte aligned.
 *   wq_sf        [64][12] UE8M0 bytes, row-major: scale of the 128x128 weight
 *                block (head h, K-block kb).
 *   positions    [M] int32 token positions (any value with |p| < 2^24).
 *   q_fp4        [M, 4096] bytes, 16-byte aligned: byte 64 h + 16 b + i of
 *                row m holds dims 32 b + 2i (low nibble) and 32 b + 2i + 1
 *                (high nibble) of head h.
 *   q_sf         [M, 256] UE8M0 bytes, 4-byte aligned: byte 4 h + b is the
 *                scale of block b of head h.
 *   workspace    caller scratch of at least iq_prepare_q_workspace(M) bytes,
 *                256-byte aligned; its contents on return are the FP8 latent
 *                and its packed scales (operation 1's outputs).
 * M == 0 returns IQ_OK without a launch.
 *
 * Launches.  Two kernel launches, back to back on `stream`: the quantizer,
 * then the GEMM kernel of M's route (see iq_set_small_m_threshold), launched
 * as the quantizer's programmatic dependent so that its set-up (and, on the
 * small-M route, its weight loads) overlap the quantizer.  With the fusion
 * switched on (iq_set_quant_fusion) the CTA-pair route is ONE launch: the
 * GEMM kernel quantizes the token rows itself (operation 1's arithmetic, the
 * same codes and scale words in the workspace) in waves ahead of the tiles
 * that read them, and a tile's loads wait for the progress flags of the CTAs
 * that quantized its rows; that launch is cooperative (all of its CTAs, one
 * per SM, resident at once).
 *
 * Ordering: the GEMM kernels of both routes read wq_e4m3 and wq_sf before the
 * kernel launched just before them on `stream` has completed (that kernel is
 * the quantizer for iq_prepare_q; for iq_gemm_rope_hadamard_fp4 it is
 * whatever the caller launched last, and the overlap happens only if that
 * kernel allows programmatic dependents).  The weights must therefore not be
 * written by the immediately preceding kernel.  Every other input is read
 * after that kernel has completed; the quantizer, itself launched as a
 * programmatic dependent of whatever precedes it, touches no memory before
 * that.  The kernels let the next kernel on `stream` be scheduled while they
 * run (griddepcontrol.launch_dependents): a following kernel launched with
 * programmatic stream serialization must wait for them
 * (griddepcontrol.wait) before it reads this call's outputs or workspace, as
 * that launch mode requires of any kernel.  Calls that run at the same time
 * must not share a workspace; calls enqueued one after another on one stream
 * may. */
iq_status iq_prepare_q(const void* latent_bf16, int M,
                       const void* wq_e4m3, const uint8_t* wq_sf,
                       const int32_t* positions,
                       uint8_t* q_fp4, uint8_t* q_sf,
                       void* workspace, size_t ws_bytes, cudaStream_t stream);

/* iq_prepare_q that also writes the float32 pre-quant Q (z above) to
 * q_prequant [M, 8192] (row-major, 16-byte aligned). */
iq_status iq_prepare_q_debug(const void* latent_bf16, int M,
                             const void* wq_e4m3, const uint8_t* wq_sf,
                             const int32_t* positions,
                             uint8_t* q_fp4, uint8_t* q_sf, float* q_prequant,
                             void* workspace, size_t ws_bytes, cudaStream_t stream);

/* The second stage alone, for callers that already hold the FP8 latent and its
 * packed scales (the outputs of operation 1 with K = 1536):
 *   xq_e4m3      [M, 1536] E4M3 codes, contiguous, 16-byte aligned.
 *   x_scales     [3][align_up(M, 4)] packed UE8M0 words, 4-byte aligned.
 *   q_prequant   may be NULL; otherwise as in iq_prepare_q_debug.
 * One kernel launch. */
iq_status iq_gemm_rope_hadamard_fp4(const void* xq_e4m3, const int32_t* x_scales, int M,
                                    const void* wq_e4m3, const uint8_t* wq_sf,
                                    const int32_t* positions,
                                    uint8_t* q_fp4, uint8_t* q_sf, float* q_prequant,
                                    cudaStream_t stream);

/* ------------------------------------------------------------------------
 * FP4 output variants.  iq_prepare_q writes MXFP4 with the scale rule above
 * (IQ_FP4_MX).  iq_prepare_q_ex selects one of:
 *   IQ_FP4_MX      1x32 blocks, UE8M0 scale 2^e, e the smallest integer with
 *                  6 * 2^e >= max(amax, 1e-4); never saturates.  q_sf [M, 256].
 *   IQ_FP4_MX_OCP  1x32 blocks, UE8M0 scale 2^e with e = floor(log2(max(amax,
 *                  1e-4))) - 2, the shared-scale rule of the OCP Microscaling
 *                  (MX) spec for E2M1; elements saturate at 6.  q_sf [M, 256].
 *   IQ_FP4_NV      1x16 blocks with an E4M3 scale s (NVFP4-style, per-tensor
 *                  scale 1): s = round-to-nearest-even E4M3 of
 *                  float32(max(amax, 1e-4) / 6), or 2^-9 (code 1) when that
 *                  rounds to zero; codes E2M1(float32(z * float32(1 / s))),
 *                  saturating at 6.  q_sf [M, 512] E4M3 bytes, byte 8 h + b the
 *                  scale of block b (dims 16 b .. 16 b + 15) of head h; 8-byte
 *                  aligned.
 * The pages specify only the MXFP4 output; the other two are variants of the
 * same FP4 stage for consumers that expect them.
 * ------------------------------------------------------------------------ */

typedef enum { IQ_FP4_MX = 0, IQ_FP4_MX_OCP = 1, IQ_FP4_NV = 2 } iq_fp4_format;

/* Scale bytes per token of a format (256 or 512); 0 for an unknown format. */
size_t iq_fp4_scale_bytes(int fp4_format);

/* iq_prepare_q with the FP4 output variant `fp4_format` (iq_fp4_format);
 * q_sf holds iq_fp4_scale_bytes(fp4_format) bytes per token; q_prequant may
 * be NULL, else it receives the float32 pre-quant Q as in iq_prepare_q_debug.
 * An unknown format returns IQ_ERR_ARG. */
iq_status iq_prepare_q_ex(const void* latent_bf16, int M,
                          const void* wq_e4m3, const uint8_t* wq_sf,
                          const int32_t* positions, int fp4_format,
                          uint8_t* q_fp4, uint8_t* q_sf, float* q_prequant,
                          void* workspace, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Indexer-Q preparation without any device allocation.  The pages have no
 * counterpart of this call; it exists for callers that cannot obtain device
 * memory at the point where they prepare Q -- for example a plugin whose host
 * program owns every device allocation and offers it no allocator, or a
 * latency-bound loop that must not call cudaMalloc (which can synchronize the
 * device).  Such a caller passes only inputs and outputs.
 *
 * The FP8 latent and its packed scales, which iq_prepare_q keeps in the
 * caller's workspace, live instead in one scratch array built into the
 * library: IQ_STATIC_MAX_TOKENS * 1536 bytes plus the scale words (about
 * 3.2 MB), held on every GPU that loads the library until the process exits.
 *
 * Behaviour:
 *  - M > IQ_STATIC_MAX_TOKENS returns IQ_ERR_WORKSPACE (the built-in scratch
 *    is too small) before anything is launched; M == 0 returns IQ_OK.
 *  - The first call on a device looks up the device address of the scratch
 *    array (cudaGetSymbolAddress) with that device current; make that first
 *    call before any stream capture on the device.
 *  - All calls on a device share the one scratch array, and it keeps what the
 *    previous call left there.  Nothing in it needs clearing: every byte the
 *    GEMM kernel reads is written by the quantizer kernel of the same call.
 *    Calls whose work overlaps on the GPU (for example on two streams without
 *    ordering between them) race on the scratch and give wrong results;
 *    order them on one stream or with events.
 *  - Same arguments, results and errors as iq_prepare_q otherwise; nothing
 *    is allocated, no allocating library routine is called.
 * ------------------------------------------------------------------------ */

#define IQ_STATIC_MAX_TOKENS 2048

iq_status iq_prepare_q_static(const void* latent_bf16, int M,
                              const void* wq_e4m3, const uint8_t* wq_sf,
                              const int32_t* positions,
                              uint8_t* q_fp4, uint8_t* q_sf, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Indexer-Q preparation on host-resident tokens.  The pages have no
 * counterpart of this call; it serves a caller whose token rows and results
 * live in host memory (an offload or batch job), and overlaps their transfer
 * with the computation.  Same operation, arguments and results as
 * iq_prepare_q_ex, except where the buffers live:
 *
 *   latent_bf16 [M, 1536] BF16, positions [M] int32   -- read
 *   q_fp4 [M, 4096] uint8, q_sf [M, iq_fp4_scale_bytes(fp4_format)] uint8
 *                                                     -- written
 *     page-locked host memory (cudaHostAlloc / cudaMallocHost, or
 *     cudaHostRegister), or device memory of the current device; the same
 *     row-major layouts and alignments as iq_prepare_q.
 *   wq_e4m3, wq_sf: device memory, as in iq_prepare_q.
 *   workspace: iq_prepare_q_host_workspace(M, fp4_format) bytes of device
 *     memory, 256-byte aligned, used until the call's work completes.
 *
 * The rows are processed in chunks of iq_host_chunk_rows() rows (fewer
 * chunks when M needs more than 64).  On internal streams of the device the
 * quantizer of chunk c reads the chunk's latent rows and positions directly
 * from host memory, the GEMM of chunk c runs once that is done, and chunk c's
 * FP4 codes and scales are copied to q_fp4 / q_sf once its GEMM is done; so
 * reading chunk c + 1, computing chunk c and returning chunk c - 1 overlap.
 *
 * Ordering: the work starts after everything enqueued on `stream` before the
 * call, and everything enqueued on `stream` after the call starts after all
 * of it, the copies into q_fp4 / q_sf included.  Synchronize `stream` (or an
 * event recorded on it after the call) before reading the results on the
 * host, and leave the inputs unchanged until then.
 *
 * Errors: those of iq_prepare_q_ex, and IQ_ERR_ARG when latent_bf16,
 * positions, q_fp4 or q_sf is pageable host memory or another device's
 * memory, or the workspace is NULL; IQ_ERR_WORKSPACE when ws_bytes is smaller
 * than iq_prepare_q_host_workspace(M, fp4_format).  M == 0 returns IQ_OK.
 *
 * The first call on a device creates three streams and 132 events there
 * (kept until the process exits); make it outside stream capture.  Calls on
 * one device enqueue one at a time (a lock) because they share those streams.
 * ------------------------------------------------------------------------ */

size_t iq_prepare_q_host_workspace(int M, int fp4_format);

iq_status iq_prepare_q_host(const void* latent_bf16, int M,
                            const void* wq_e4m3, const uint8_t* wq_sf,
                            const int32_t* positions, int fp4_format,
                            uint8_t* q_fp4, uint8_t* q_sf,
                            void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Rows per chunk of iq_prepare_q_host, rounded up to a multiple of 256 and
 * clamped to [256, 2^20]; returns the previous value (default 1024). */
int iq_set_host_chunk_rows(int rows);
int iq_host_chunk_rows(void);

/* ------------------------------------------------------------------------
 * 3. The consumer of the prepared Q: the sparse-attention indexer's scores
 *    and top-k key selection (the TokenSpeed PR names the indexer top-k and
 *    writes it straight to its destination -- Summary; Prefill host-sync
 *    cleanup -- but gives neither formula nor layout; these are this
 *    library's readings).
 *
 *   score  I[t, s] = sum over heads h < 64 of w[t, h] * max(0, q(t, h) . k(s))
 *          q(t, h): head h of query token t, decoded from the MXFP4 Q that
 *            iq_prepare_q writes (q_fp4 [M, 4096], q_sf [M, 256]);
 *          k(s): the 128-dim key of cached token s, in the same MXFP4 format
 *            (k_fp4 [N, 64] bytes: element 2i in the low nibble of byte i;
 *            k_sf [N, 4] UE8M0 bytes, byte b for dims 32 b .. 32 b + 31);
 *          w: float32 [M, 64] per-head weights of each query token;
 *          keys s < L[t] are visible to query t (L: int32 [M], clamped to
 *            [0, N]; causal prefill passes position + 1).
 *   The head dot products are accumulated in float32 by the tensor cores;
 *   the ReLU and the weighted head sum are float32.
 * ------------------------------------------------------------------------ */

/* Writes logits[t * ld_logits + s] = I[t, s] for every visible pair (s <
 * L[t]); entries s >= L[t] are not written.  One kernel launch.
 * Requirements: M, N >= 0 (M == 0 or N == 0: IQ_OK, no launch); ld_logits >=
 * N; q_fp4, q_sf, k_fp4, k_sf and weights 16-byte aligned, lengths and
 * logits 4-byte aligned (else IQ_ERR_ALIGN); M * 64 < 2^31 (else IQ_ERR_ARG).
 * Launched as a programmatic dependent of the preceding kernel: nothing is
 * read before that kernel completes. */
iq_status iq_indexer_logits(const uint8_t* q_fp4, const uint8_t* q_sf, int M, const uint8_t* k_fp4,
                            const uint8_t* k_sf, int N, const float* weights, const int32_t* lengths,
                            float* logits, long long ld_logits, cudaStream_t stream);

/* For every query row t: the k visible keys (s < L[t]) with the largest
 * logits[t * ld_logits + s], ties to the smaller index (-0 and +0 tie), as
 * int32 indices in ascending order in indices[t * k .. t * k + k - 1], padded
 * with -1 when fewer than k keys are visible.  Scores must not be NaN.  One
 * kernel launch (one block per row), a programmatic dependent of the
 * preceding kernel (normally iq_indexer_logits).  Requirements: k >= 1,
 * ld_logits >= N, 4-byte aligned pointers. */
iq_status iq_indexer_topk(const float* logits, long long ld_logits, int M, int N, const int32_t* lengths, int k,
                          int32_t* indices, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * 4. The 8-bit paged KV cache and the attention that reads it: what the keys
 *    that iq_indexer_topk selects are selected for.  (The pages have no
 *    counterpart; layouts and rules are this library's own.)
 *
 * Cache.  K and V are kept apart, each as E4M3 codes in pages of page_size
 * consecutive tokens of one sequence and one UE8M0 scale byte per page and KV
 * head:
 *   codes [num_pages][kv_heads][page_size][head_dim]   16-byte aligned
 *   sf    [num_pages][kv_heads]
 * A code c under the scale byte b stands for E4M3(c) * 2^(b - 127), under
 * b = 255 for NaN.  Writing stores bytes from 105 to 247.
 * page_size is 16, 32, 64 or 128, head_dim 64 or 128, kv_heads >= 1 (else
 * IQ_ERR_SHAPE); num_pages * kv_heads * page_size < 2^31 (else IQ_ERR_ARG),
 * while byte offsets may pass 32 bits.
 *
 * Batch.  num_seqs sequences, packed along num_rows rows: row t of sequence b,
 * row_start[b] <= t < row_start[b + 1], is one of the sequence's newest
 * n_b = row_start[b + 1] - row_start[b] tokens, at position
 *   kv_len[b] - row_start[b + 1] + t,
 * kv_len[b] being the length with these tokens.  Position s of sequence b is
 * slot s % page_size of page block_table[b * table_ld + s / page_size].
 * row_start is non-decreasing from 0 to num_rows; a sequence may have no row.
 * All three arrays are read on the device; rows outside [0, num_rows) that
 * row_start names are never touched.  Positions below 0 or past
 * max_pages * page_size, and pages outside [0, num_pages), are never touched:
 * writing skips them, reading gives zeros, attention does not see them.
 *
 * All calls are asynchronous on `stream` as programmatic dependents of the
 * kernel before them: they read and write nothing before it has completed.
 * ------------------------------------------------------------------------ */

typedef struct {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint8_t* k_sf;
  uint8_t* v_sf;
  int num_pages;
  int kv_heads;
  int page_size;
  int head_dim;
} iq_kv_cache;

typedef struct {
  const int32_t* block_table; /* [num_seqs][table_ld], the first max_pages of a row used */
  long long table_ld;
  int max_pages;
  const int32_t* row_start;   /* [num_seqs + 1] */
  const int32_t* kv_len;      /* [num_seqs] */
  int num_seqs;
  int num_rows;
} iq_kv_batch;

/* Quantises the batch's rows into their pages.  k, v: BF16, row t at
 * k + t * ldk elements, its kv_heads * head_dim values contiguous; 16-byte
 * aligned, ldk, ldv >= kv_heads * head_dim and multiples of 8.
 *
 * For every page that receives rows, per KV head, K and V apart:
 *   a = largest |x| of the rows it receives;
 *   e = the smallest integer with 448 * 2^e >= max(a, 1e-4);
 *   if the page also holds older tokens of the sequence (slots before the
 *   first row it receives): e = max(e, the page's present exponent), and where
 *   that raises the exponent by d the older tokens' codes become the E4M3
 *   codes nearest (ties to even) to code * 2^-d;
 *   the rows' codes are the E4M3 codes nearest to x * 2^-e, the scale byte is
 *   e + 127.
 * Slots behind the last row keep their bytes.  Pages that receive rows must
 * belong to one sequence.  NaN and infinite inputs are outside the contract
 * (they spoil the page's scale).  One kernel launch. */
iq_status iq_kv_cache_write(const iq_kv_cache* cache, const iq_kv_batch* batch, const void* k_bf16, long long ldk,
                            const void* v_bf16, long long ldv, cudaStream_t stream);

/* Reads the batch's rows back: k, v rows laid out as in iq_kv_cache_write
 * receive E4M3(c) * 2^(b - 127).  BF16 holds that exactly for 3 <= b <= 246;
 * beyond, it is rounded to nearest, ties to even, and from 2^128 on it is
 * infinite.  With row counts
 * equal to kv_len this is the whole cache of each sequence.  One kernel
 * launch. */
iq_status iq_kv_cache_read(const iq_kv_cache* cache, const iq_kv_batch* batch, void* k_bf16, long long ldk,
                           void* v_bf16, long long ldv, cudaStream_t stream);

/* Causal attention of the batch's rows over the cached keys and values:
 *   out[t, h] = sum_s p_s v_s / sum_s p_s,  p_s = exp(scale * q[t, h] . k_s),
 * over the positions s <= the row's own position; query head h reads KV head
 * h / (q_heads / kv_heads).  A row that sees no key gives zeros.
 *   q    BF16, row t at q + t * ldq elements, [q_heads][head_dim] contiguous,
 *   out  BF16, row t at out + t * ldo elements likewise; both 16-byte aligned,
 *        ldq, ldo >= q_heads * head_dim and multiples of 8;
 *   q_heads a positive multiple of kv_heads (else IQ_ERR_SHAPE);
 *   scale finite (else IQ_ERR_ARG), normally 1 / sqrt(head_dim);
 *   workspace of iq_kv_attention_workspace(...) bytes, 256-byte aligned, free
 *        again once the call's work has completed; nothing in it needs
 *        clearing.  Calls that run at the same time must not share one.
 * The keys and values are multiplied as they are stored, values under a scale
 * byte below 64 (less than 2^-54) with fewer bits or as zeros.  Scores, softmax
 * statistics and sums are float32; a weight enters the second product with 8
 * significant bits (BF16), with 16 where a token's query heads per KV head,
 * times the mean number of tokens per sequence without an index list, are 32
 * at most.  A query row that holds NaN or an infinity gives NaN where it sees a
 * key.  Keys and values that hold NaN inside [0, kv_len) are outside the
 * contract; slots past kv_len may hold any bytes. */
iq_status iq_kv_attention(const iq_kv_cache* cache, const iq_kv_batch* batch, const void* q_bf16, long long ldq,
                          int q_heads, float scale, void* out_bf16, long long ldo, void* workspace, size_t ws_bytes,
                          cudaStream_t stream);

/* The same over a list of keys per row, such as iq_indexer_topk writes it:
 * row t sees the positions indices[t * ld_idx + j], j < k, that are >= 0 and
 * no later than its own position (others, -1 among them, are skipped; a
 * position listed twice counts twice).  indices 4-byte aligned, ld_idx >= k,
 * k >= 1 (else IQ_ERR_ARG). */
iq_status iq_kv_attention_topk(const iq_kv_cache* cache, const iq_kv_batch* batch, const void* q_bf16, long long ldq,
                               int q_heads, const int32_t* indices, long long ld_idx, int k, float scale,
                               void* out_bf16, long long ldo, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes of both attention calls; 0 for arguments they refuse. */
size_t iq_kv_attention_workspace(int num_rows, int q_heads, int kv_heads, int head_dim);

/* ------------------------------------------------------------------------
 * 5. The experts' feed-forward block on operation 1's rows: which experts a
 *    token's row goes to, the experts' products, and the weighted sum of what
 *    comes back.  (The pages have no counterpart; layouts and rules are this
 *    library's own.)  A block with gated experts is
 *
 *      iq_moe_route          logits -> weights, slots, rows, row_start
 *      iq_fp8_quant_1x128_rows   the slots' rows as codes and scales
 *      iq_grouped_gemm       gated: up to the hidden rows [T * k, I]
 *      iq_fp8_quant_1x128_ue8m0  their codes and scales
 *      iq_grouped_gemm       down to [T * k, N]
 *      iq_moe_combine        [T, N]
 *
 * All calls are asynchronous on `stream` as programmatic dependents of the
 * kernel before them: they read and write nothing before it has completed.
 * Workspaces are device memory, 256-byte aligned, free again once the call's
 * work has completed; nothing in them needs clearing.  Calls that run at the
 * same time must not share one.
 * ------------------------------------------------------------------------ */

/* Operation 1 over a list of rows: output row s < M holds the codes and scales
 * of row rows[s] of x (num_src rows), or of a row of zeros where rows[s] is
 * outside [0, num_src) (x may be NULL where num_src is 0).  rows: int32 [M], 4-byte
 * aligned; M and K up to 2^31 - 512 (else IQ_ERR_SHAPE); the other arguments and
 * errors as in iq_fp8_quant_1x128_ue8m0.  One kernel launch. */
iq_status iq_fp8_quant_1x128_rows(const void* x_bf16, int num_src, const int32_t* rows, int M, int K, int ldx,
                                  void* y_e4m3, int ldy, int32_t* scales, cudaStream_t stream);

/* Chooses the experts of each token and lays out the (token, expert) pairs.
 *   logits     [num_tokens][ld_logits], float32 or (logits_bf16 != 0) BF16
 *   experts    int32 [num_tokens][k]: the k largest logits' experts, largest
 *              first, ties (-0 and +0 too) to the lower index
 *   weights    float32 [num_tokens][k]:
 *                IQ_SCORE_SOFTMAX  exp(l - max) / sum of that over all experts
 *                IQ_SCORE_SIGMOID  1 / (1 + exp(-l))
 *              with normalize != 0 the sum is, or a division by it follows,
 *              over the chosen experts alone; times scale
 *   slots      int32 [num_tokens][k]: the pair's place among all pairs ordered
 *              by expert, then by token
 *   rows       int32 [num_tokens * k]: the token of each slot
 *   row_start  int32 [num_experts + 1]: the slots of expert e are
 *              row_start[e] .. row_start[e + 1] - 1
 * A NaN logit counts as -inf.  Experts with -inf are chosen last and get
 * weight 0 (a token with no other logit has weights 0; so it has with
 * IQ_SCORE_SIGMOID and normalize where all logits are below -709.78, which makes
 * the scores 0 in 64 bits too).  num_experts at most
 * 1024, k at most 32 and num_experts (else IQ_ERR_SHAPE); scale finite (else
 * IQ_ERR_ARG); num_tokens * k at most 2^31 - 64 (else IQ_ERR_ARG).  num_tokens == 0 writes row_start
 * alone.  Up to 128 tokens one kernel launch and no workspace, else two
 * or three launches. */
enum { IQ_SCORE_SOFTMAX = 0, IQ_SCORE_SIGMOID = 1 };
iq_status iq_moe_route(const void* logits, int logits_bf16, long long ld_logits, int num_tokens, int num_experts, int k,
                       int score, int normalize, float scale, float* weights, int32_t* experts, int32_t* slots,
                       int32_t* rows, int32_t* row_start, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes of iq_moe_route for num_tokens and for any smaller number of them
 * (0 up to 128 tokens and for arguments it refuses). */
size_t iq_moe_route_workspace(int num_tokens, int num_experts);

/* Products grouped by expert: rows m of group g, row_start[g] <= m <
 * row_start[g + 1], are multiplied with that group's weights,
 *   y[m, n] = sum_kb 2^(ex[m, kb] + ew[g, n / 128, kb]) sum_{k in kb} x[m, k] w[g, n, k].
 *   x_e4m3     E4M3 codes, row m at x + m * ldx bytes, and
 *   x_scales   int32 [ceil(K / 512)][align_up(M, 4)]: operation 1's outputs for M
 *              rows; 16-byte aligned, ldx >= K and a multiple of 16
 *   w_e4m3     [num_groups][N][K] E4M3 codes, 16-byte aligned
 *   w_sf       [num_groups][ceil(N / 128)][K / 128] UE8M0 bytes, one per 128x128
 *              block
 *   row_start  int32 [num_groups + 1], non-decreasing, read on the device; rows
 *              of no group keep their bytes in y
 *   y_bf16     BF16, row m at y + m * ldy elements; 16-byte aligned, ldy a
 *              multiple of 8; overlaps no input
 * gated != 0: the weights hold N / 2 gate rows and then N / 2 up rows, and y has
 * N / 2 columns silu(gate) * up, silu(g) = g / (1 + exp(-g)), rounded once.
 * Sums are float32.  K a positive multiple of 128 up to 2^20, N one of 8 (gated of
 * 256), M and N up to 2^31 - 512, num_groups from 1 to 1024, (M / 256 + 1) *
 * num_groups * N / 256 below 2^30 (else IQ_ERR_SHAPE).  row_start entries outside [0, M] are taken as the nearest
 * bound; a group that ends before it begins is empty, and rows that a falling
 * row_start gives to two groups are undefined.  Scale byte 255 (NaN) and NaN codes
 * are outside the contract, but what stands in rows of no group, or in the weights of
 * an empty one, goes nowhere.  M == 0 returns IQ_OK without a launch, else one kernel
 * launch, and a second one where a workspace is needed. */
iq_status iq_grouped_gemm(const void* x_e4m3, long long ldx, const int32_t* x_scales, int M, int K, const void* w_e4m3,
                          const uint8_t* w_sf, int num_groups, int N, const int32_t* row_start, int gated, void* y_bf16,
                          long long ldy, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes of iq_grouped_gemm for M rows and for any smaller number of them
 * (the size never falls as M or K grow); 0 for a short K (up to 2304), where no
 * product is split, and for arguments it refuses.  A call takes less where its own
 * rows need less, and NULL where they need none: where ceil(K / 256) <= 9 + w / 32,
 * quotient rounded down, w = min(256, align_up(M, 16)). */
size_t iq_grouped_gemm_workspace(int M, int K);

/* The weighted sum of each token's rows:
 *   out[t] = add[t] + sum_j weights[t, j] * y[slots[t, j]],  j < k,
 * in float32 in the order of j, rounded once.  y, add and out are BF16 rows of N
 * values at multiples of ldy, ld_add and ld_out elements; add may be NULL, and
 * out may be add but overlaps no input otherwise.  Slots outside [0, num_rows) are left out.  N a positive
 * multiple of 8, k >= 1 (else IQ_ERR_SHAPE); 16-byte aligned rows, slots and
 * weights 4-byte aligned.  A weight of 0 multiplies its row all the same.  One kernel
 * launch. */
iq_status iq_moe_combine(const void* y_bf16, long long ldy, int num_rows, const int32_t* slots, const float* weights,
                         int num_tokens, int k, int N, const void* add_bf16, long long ld_add, void* out_bf16,
                         long long ld_out, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * 6. Low-rank adapters of many requests beside a shared projection.  (The
 *    pages have no counterpart; the layout is this library's own.)
 * ------------------------------------------------------------------------ */

/* Adds each request's own adapter to a projection's output:
 *   out[t] = base[t] + scale[a] * B[a] (A[a] x[t]),  a = adapter[i],
 * for the rows t of request i, row_start[i] <= t < row_start[i + 1].  Where
 * adapter[i] is outside [0, num_adapters) the request has none: out = base.
 *   x_bf16     BF16 [num_tokens][K] at multiples of ldx elements
 *   a_bf16     BF16 [num_adapters][rank][K]
 *   b_bf16     BF16 [num_adapters][N][rank]
 *   scale      float32 [num_adapters]
 *   row_start  int32 [num_requests + 1], non-decreasing, and adapter int32
 *              [num_requests], both read on the device; rows of no request
 *              keep their bytes in out
 *   base_bf16  BF16 [num_tokens][N] at multiples of ld_base elements, or NULL
 *              for zeros; out may be base
 *   out_bf16   BF16 [num_tokens][N] at multiples of ld_out elements
 * K and N positive multiples of 8, rank a multiple of 8 up to 128 (an adapter of
 * a smaller rank is padded with zeros), at most 1024 requests, num_adapters >= 1,
 * (num_tokens / 128 + 1 + min(num_requests, num_tokens)) * max(K / 64 * (192 +
 * rank), N / 128 * 320), both quotients rounded up, below 2^30 (else IQ_ERR_SHAPE);
 * x, a, b, base, out 16-byte aligned, their strides multiples of 8 (else
 * IQ_ERR_ALIGN); out overlaps no input but base.  row_start entries outside [0,
 * num_tokens] are taken as the nearest bound, and rows that a falling row_start gives
 * to two requests belong to the first.  Requests of one adapter that follow one
 * another are multiplied together, so a batch ordered by adapter reads each adapter
 * once.
 * Sums are float32; scale A x is rounded to float32 and enters the second product
 * with all its bits; out is rounded once.  Infinities in x, a and base give what
 * the definition gives; in rows that meet one in b, NaN may stand for it.
 * The workspace is iq_adapters_workspace(num_tokens, rank) bytes, 256-byte aligned,
 * free again once the call's work has completed; nothing in it needs clearing, and
 * calls that run at the same time must not share one.
 * Two kernel launches, programmatic dependents of the kernel before them that
 * read and write nothing before it has completed; none when there is no token
 * or no request. */
iq_status iq_adapters(const void* x_bf16, long long ldx, int num_tokens, int K, const void* a_bf16, const void* b_bf16,
                      const float* scale, int num_adapters, int rank, int N, const int32_t* row_start,
                      const int32_t* adapter, int num_requests, const void* base_bf16, long long ld_base, void* out_bf16,
                      long long ld_out, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes of iq_adapters; 0 for arguments it refuses. */
size_t iq_adapters_workspace(int num_tokens, int rank);

#ifdef __cplusplus
}
#endif

#endif /* IQ_H_ */
