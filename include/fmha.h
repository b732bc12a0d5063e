/*
 * fmha.h -- C ABI of libfmha_gb300.so, the GB300 (sm_103a) fused attention
 * forward.
 *
 * What is computed (per batch b, query head h, query row t):
 *
 *     O[b,h,t,:] = softmax_j( scale * <Q[b,h,t,:], K[b,kvh,j,:]> + mask ) V[b,kvh,j,:]
 *     LSE[b,h,t] = ln sum_{j attended} exp(scale * <Q[b,h,t,:], K[b,kvh,j,:]>)
 *
 * with kvh = h / (n_h / n_kv_h).  Sources: the commit pages of the
 * nvfp4-megamoe-kernel repository (dsv4 directory) and its CURRENT_ISSUE.md
 * "UMMA FMHA -- Full Pipeline + Production":
 *   - FA2 online softmax over KV tiles with a running max and sum, P kept
 *     un-normalised, one final divide by the running sum: commit e4ee9fd,
 *     multi-tile C API part.
 *   - scores are the unscaled dot product, the scale is applied in the
 *     softmax: CURRENT_ISSUE.md, "Key lessons from this session".
 *   - split-KV partials merged as O = sum_i exp(lse_i) O_i / sum_i exp(lse_i):
 *     CURRENT_ISSUE.md, "Next steps" item 4.
 *   - MQA as a K/V head shared by every query head (head stride 0): commit
 *     e4ee9fd, "Architecture".
 *   - sliding-window ("D3") and causal ("D4") masks: commit 593bc25, scalar
 *     reference kernel part.
 *   - a pure C ABI with no framework types and no host synchronisation on the
 *     hot path: commit e4ee9fd, multihead C API and "Architecture" parts.
 *
 * Readings of points the pages leave open:
 *   - query row t sits at absolute key position p = s_k - T + t (the T new
 *     queries follow the s_k - T cached keys: bottom-right alignment);
 *   - causal: key j is attended iff j <= p;
 *   - window w > 0: key j is attended iff j > p - w (the last w positions up to
 *     and including p); w = 0 disables the window;
 *   - LSE is the natural log of the sum over attended keys of exp(scaled
 *     score); a row that attends no key gets O = 0 and LSE = -inf.
 *
 * Layouts (all contiguous, row-major, device memory owned by the caller):
 *   Q, O        [batch, n_h,    T,   hd]  bf16 (raw bits, round-to-nearest-even on output)
 *   K, V        [batch, n_kv_h, s_k, hd]  bf16
 *   LSE         [batch, n_h,    T]        fp32
 *   o_parts     [n_splits, batch, n_h, T, hd] fp32   (split-KV partial outputs)
 *   lse_parts   [n_splits, batch, n_h, T]     fp32
 *
 * Accepted shapes: hd in {64, 128, 256, 512}; n_h % n_kv_h == 0;
 * batch * n_kv_h <= 65535; batch >= 0, T >= 0 (zero means nothing to do);
 * s_k >= 0; with causal, T <= s_k; window >= 0.  q, k, v, o, o_parts must be
 * 16-byte aligned, lse and lse_parts 4-byte aligned.
 *
 * Errors: every call returns FMHA_OK (0) or a negative FMHA_ERR_* code and
 * never aborts.  On an argument error nothing is launched.  The message of the
 * last failure on the calling thread is available from fmha_get_last_error().
 *
 * Asynchrony: every compute call is ordered on `stream` (NULL = the legacy
 * default stream) and returns without synchronising the host.  Kernels bound
 * every internal wait; a wait that gives up sets a device status word that
 * fmha_check_device_status() reports.
 */
#ifndef FMHA_GB300_H
#define FMHA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* fmha_stream_t;

enum fmha_status {
    FMHA_OK = 0,
    FMHA_ERR_NULL = -1,           /* a required pointer is NULL */
    FMHA_ERR_ALIGN = -2,          /* a pointer is not aligned as required */
    FMHA_ERR_HEADDIM = -3,        /* hd not in {64, 128, 256, 512} */
    FMHA_ERR_HEADS = -4,          /* n_h, n_kv_h < 1 or n_h % n_kv_h != 0 */
    FMHA_ERR_SHAPE = -5,          /* negative size, causal with T > s_k, grid limits, bad window/chunk/scale */
    FMHA_ERR_WORKSPACE = -6,      /* the internal split-KV workspace could not be allocated */
    FMHA_ERR_LAUNCH = -7,         /* a CUDA call failed; the message names it */
    FMHA_ERR_DEVICE_TIMEOUT = -8, /* a kernel's bounded wait gave up (from fmha_check_device_status) */
    FMHA_ERR_UNSUPPORTED = -9,    /* a partial format this shape's kernel does not write */
    FMHA_ERR_DEVICE_BOUNDS = -10  /* checked build: a kernel's index check failed (from fmha_check_device_status) */
};

/*
 * Fused attention forward.  Writes O (bf16) and LSE (fp32).
 *
 * scale: multiplies the raw dot products (usually 1/sqrt(hd)).
 * window: sliding-window length in keys, 0 = none.  causal: 0 or 1.
 *
 * The library chooses whether to split the KV range over several thread
 * blocks.  When it splits, the partials live in a workspace the library
 * allocates on `stream` with cudaMallocAsync the first time a (device,
 * stream) pair needs more than it holds, and keeps until fmha_release().
 * They are fp32, except on the hd-512 tensor-core kernel, where they are fp16
 * scaled by a power of two per row half (so any finite value keeps 11
 * significant bits), which halves their traffic.
 * Callers that must not allocate use fmha_fwd_splitkv + fmha_merge with their
 * own buffers.
 */
int fmha_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
             int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
             float scale, int window, int causal, fmha_stream_t stream);

/*
 * The plan fmha_fwd uses for this shape: returns the number of KV chunks
 * (1 = no split: one kernel writes O and LSE directly; > 1 = a split pass
 * into the workspace followed by the merge), stores the chunk length in
 * *kv_chunk and the kernel family in *kernel (1 = decode kernel, 2 =
 * tensor-core kernel, one 128-row tile per thread block, 3 = tensor-core
 * kernel for hd 512, 4 = tensor-core kernel with two 128-row tiles per thread
 * block, hd 64 and 128; fmha_fwd_nvfp4 runs kernel 2 there, with the same
 * chunks);
 * either pointer may be NULL.  Pure host arithmetic apart from reading the current device's SM
 * count; negative FMHA_ERR_* code on invalid shapes.
 */
int fmha_fwd_plan(int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                  int window, int causal, int* kv_chunk, int* kernel);

/*
 * Split-KV layout for chunks of kv_chunk keys (kv_chunk >= 1): returns the
 * number of chunks n_splits (>= 1) and stores in *first_key the first key of
 * chunk 0, which is the first key that query row t = 0 attends (0 without a
 * window).  Chunk i covers keys [first_key + i*kv_chunk, first_key +
 * (i+1)*kv_chunk) clipped to s_k.  Pure host arithmetic; returns a negative
 * FMHA_ERR_* code for invalid arguments.  first_key may be NULL.
 */
int fmha_split_layout(int T, int s_k, int window, int kv_chunk, int* first_key);

/*
 * Split-KV partial pass (the "D5" split of CURRENT_ISSUE.md, "Next steps"
 * item 4).  For every chunk i of fmha_split_layout(T, s_k, window, kv_chunk)
 * writes the normalised partial output O_i and its log-sum-exp lse_i over the
 * keys of that chunk (O_i = 0, lse_i = -inf where the chunk holds no attended
 * key).  o_parts / lse_parts are caller buffers in the layouts above.
 */
int fmha_fwd_splitkv(const void* q, const void* k, const void* v,
                     float* o_parts, float* lse_parts, int kv_chunk,
                     int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                     float scale, int window, int causal, fmha_stream_t stream);

/*
 * Merge split-KV partials (CURRENT_ISSUE.md, "Next steps" item 4):
 *     LSE = ln sum_i exp(lse_i),   O = sum_i exp(lse_i - LSE) O_i
 * Partials with lse_i = -inf carry no weight; if all do, O = 0, LSE = -inf.
 * Writes bf16 O [batch, n_h, T, hd] and fp32 LSE [batch, n_h, T].
 */
int fmha_merge(const float* o_parts, const float* lse_parts, int n_splits,
               void* o, float* lse, int batch, int n_h, int T, int hd,
               fmha_stream_t stream);

/*
 * Partial formats for fmha_fwd_splitkv_ex / fmha_merge_ex.  The merge formula
 * is the one above; only the storage of O_i differs.
 *   FMHA_PARTS_F32: o_parts fp32 [n_splits, batch, n_h, T, hd] (what
 *     fmha_fwd_splitkv writes); range_parts unused, may be NULL.
 *   FMHA_PARTS_F16: o_parts fp16 [n_splits, batch, n_h, T, hd] holding
 *     O_i * 2^-k, and range_parts fp32 [n_splits, batch, n_h, T, 2] holding
 *     2^k for each 256-column half of each row; k is chosen per half row so
 *     that its largest |O_i| * 2^-k lies in [2^14, 2^15) before rounding (so
 *     in [2^14, 2^15] stored), so every finite partial keeps fp16's 11
 *     significant bits and none overflows.  Half the bytes of
 *     FMHA_PARTS_F32 (for callers that move partials elsewhere before merging;
 *     fmha_fwd uses this format internally at hd 512).  Written only by the
 *     hd-512 tensor-core kernel: hd = 512 and fmha_fwd_plan reporting kernel 3,
 *     else FMHA_ERR_UNSUPPORTED.  range_parts must be 4-byte aligned.
 * This extension has no counterpart on the pages; it is a storage format of
 * the partials whose merge they define.
 */
enum fmha_parts_format { FMHA_PARTS_F32 = 0, FMHA_PARTS_F16 = 1 };

/* fmha_fwd_splitkv writing partials in `parts_format`. */
int fmha_fwd_splitkv_ex(const void* q, const void* k, const void* v,
                        void* o_parts, float* lse_parts, float* range_parts, int parts_format,
                        int kv_chunk, int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                        float scale, int window, int causal, fmha_stream_t stream);

/* fmha_merge of partials in `parts_format` (range_parts as written by
 * fmha_fwd_splitkv_ex; FMHA_PARTS_F16 needs hd = 512), with an optional
 * attention sink (see fmha_fwd_sink): sink is NULL or a device array of n_h
 * fp32 logits, added once to each row's denominator. */
int fmha_merge_ex(const void* o_parts, const float* lse_parts, const float* range_parts, int parts_format,
                  int n_splits, const float* sink, void* o, float* lse, int batch, int n_h, int T, int hd,
                  fmha_stream_t stream);

/*
 * fmha_fwd with an attention sink.  The pages list "D5c sink" as a TODO and
 * define nothing; the reading taken here: query head h has a logit sigma_h
 * (natural-log units, the same units as scale * q.k) that joins the softmax
 * denominator only, as one more key whose value row is zero:
 *     O   = sum_j exp(s_j) v_j / (sum_j exp(s_j) + exp(sigma_h))
 *     LSE = ln(sum_j exp(s_j) + exp(sigma_h))
 * A row with no attended key gets O = 0, LSE = sigma_h; sigma_h = -inf is no
 * sink.  sink: device array of n_h fp32 logits, 4-byte aligned, caller-owned;
 * NULL makes this call fmha_fwd.  Everything else as fmha_fwd.
 */
int fmha_fwd_sink(const void* q, const void* k, const void* v, void* o, float* lse, const float* sink,
                  int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                  float scale, int window, int causal, fmha_stream_t stream);

/*
 * fmha_fwd with the output O quantised to NVFP4 in the epilogue, from the fp32
 * values that would otherwise be rounded to bf16 (commit 593bc25 of the
 * pages, TMEM-epilogue part: "register slot for FP4 pack"; its quantiser part
 * names an E2M1 element nibble, an E4M3 scale and round-to-nearest-even, and
 * gives no block size).  Format taken:
 *   - each O row [hd] is cut into hd / 16 blocks of 16 consecutive elements;
 *   - block scale s = E4M3(amax / (6 g)), amax the block's largest |O|, g =
 *     o_global_scale (finite, > 0); E4M3: 4 exponent bits (bias 7), 3
 *     mantissa bits, subnormals, largest finite value 448;
 *   - element code e = E2M1(O / (g s)): magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *     for codes 0..7, sign in bit 3 (never set on a zero magnitude);
 *   - both roundings go to the nearest representable value, a tie to the even
 *     code, and saturate at the largest finite value; s = 0 gives codes 0;
 *   - amax / (6 g) and O / (g s) are IEEE fp32 divisions;
 *   - O is recovered as g * s * e.
 * o_codes:  [batch, n_h, T, hd / 2] bytes, element 2i in the low nibble of
 *           byte i of its row; 16-byte aligned.
 * o_scales: [batch, n_h, T, hd / 16] E4M3 bytes; 4-byte aligned.
 * lse as fmha_fwd.  No attention sink.  Plan, kernels, workspace, errors and
 * asynchrony are fmha_fwd's; when the plan splits, the merge quantises.
 */
int fmha_fwd_nvfp4(const void* q, const void* k, const void* v, void* o_codes, void* o_scales, float* lse,
                   float o_global_scale, int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                   float scale, int window, int causal, fmha_stream_t stream);

/*
 * The NVFP4 quantisation of fmha_fwd_nvfp4 applied to fp32 rows on their own:
 * x [rows, hd] fp32 (hd a multiple of 16, x 16-byte aligned) -> codes
 * [rows, hd / 2] (8-byte aligned) and scales [rows, hd / 16], with the same
 * block quantiser the fused epilogues run, so its codes can be checked bit
 * for bit.  Stream-ordered; FMHA_ERR_SHAPE for a bad hd, rows or global scale.
 */
int fmha_quantize_nvfp4(const float* x, long long rows, int hd, float global_scale, void* codes, void* scales,
                        fmha_stream_t stream);

/* Bytes of fp32 partial output (o_parts + lse_parts) that fmha_fwd_splitkv
 * writes for n_splits chunks: n_splits * batch * n_h * T * (hd + 1) * 4.
 * Negative arguments give 0. */
size_t fmha_splitkv_workspace_bytes(int batch, int n_h, int T, int hd, int n_splits);

/* The same number under the name the split-KV workspace query is usually
 * given: the caller buffers fmha_fwd_splitkv + fmha_merge need for n_splits
 * chunks (the count fmha_fwd_plan or fmha_split_layout returns). */
size_t fmha_workspace_bytes(int batch, int n_h, int T, int hd, int n_splits);

/* Synchronises `stream`, then reads and clears the current device's status
 * word.  Returns FMHA_ERR_DEVICE_BOUNDS if, in a checked build, a kernel's
 * index check failed since the last check (the message names the check's
 * site), else FMHA_ERR_DEVICE_TIMEOUT if a kernel's bounded wait gave up,
 * FMHA_ERR_LAUNCH if the synchronisation failed, else FMHA_OK. */
int fmha_check_device_status(fmha_stream_t stream);

/*
 * Checked build (no counterpart on the pages; the pages debugged an illegal
 * memory access by hand, CURRENT_ISSUE.md "Key lessons from this session").
 * The same sources compiled with -DFMHA_CHECKED give
 * libfmha_gb300_checked.so, with the same entry points.  Its kernels test
 * every computed shared-memory offset, tensor-memory column, global-memory
 * index and TMA coordinate against the extent of its buffer before the
 * access; a failed check skips the access (a warp-collective instruction is
 * pointed at offset 0 of its buffer instead), and the next
 * fmha_check_device_status() returns FMHA_ERR_DEVICE_BOUNDS naming the site.
 * It is a debugging aid and slower; results are otherwise identical.
 * fmha_build_flags() returns FMHA_BUILD_CHECKED in that library, 0 in the
 * normal one.
 */
#define FMHA_BUILD_CHECKED 1
int fmha_build_flags(void);

/* Message for the last non-zero return on the calling thread ("" if none). */
const char* fmha_get_last_error(void);

/* Frees every workspace fmha_fwd allocated (synchronises each device that
 * holds one first).  Safe to call at any time no fmha call is in flight. */
void fmha_release(void);

/*
 * Failure-detection self-test: launches one thread that waits, through the
 * same bounded mbarrier wait the attention kernels use, on a barrier phase
 * that nothing completes.  After timeout_us microseconds (1 .. 10^7) the wait
 * gives up, sets the device status word and the kernel returns normally, so
 * the next fmha_check_device_status() on this device returns
 * FMHA_ERR_DEVICE_TIMEOUT and the context stays usable.  No fault, trap or
 * hang is involved.
 */
int fmha_selftest_wait_timeout(unsigned timeout_us, fmha_stream_t stream);

/*
 * (This entry point has no counterpart on the pages the method comes from;
 * the computation is fmha_fwd's.)
 * fmha_fwd from host memory: copies Q, K and V (layouts of fmha_fwd) from
 * host memory into device buffers the library owns, runs fmha_fwd on them and
 * copies O (bf16) and LSE (fp32) back into host memory.  Everything is
 * stream-ordered on `stream` (one cudaMemcpyAsync per tensor, no host
 * synchronisation), so the host buffers must stay valid and unmodified until
 * `stream` has passed this call; page-locked host memory gives asynchronous
 * copies.  The device buffers (Q + K + V + O + LSE bytes) are cached per
 * device and stream like fmha_fwd's workspace, grown with cudaMallocAsync and
 * freed by fmha_release(); calls on one stream reuse them in stream order.
 * Calls on two streams use two sets, so the host-to-device copies of one can
 * overlap the kernels and the device-to-host copies of the other.
 * Errors: those of fmha_fwd (host pointers need no alignment), and
 * FMHA_ERR_WORKSPACE if the device buffers cannot be allocated.
 */
int fmha_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* o_host, float* lse_host,
                  int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                  float scale, int window, int causal, fmha_stream_t stream);

/*
 * Index-check self-test: launches one thread that runs an index check whose
 * condition is false, with no memory access behind it.  In the checked build
 * the next fmha_check_device_status() on this device returns
 * FMHA_ERR_DEVICE_BOUNDS and names the self-test site; in the normal build
 * the check is compiled out and nothing is recorded.  Returns FMHA_OK, or
 * FMHA_ERR_LAUNCH if the launch failed.
 */
int fmha_selftest_bounds_check(fmha_stream_t stream);

/*
 * Kernel-family selection for every later call in the process: 0 = automatic
 * (default: the 128-row tensor-core kernels when a KV head has at least 64
 * query rows at hd <= 128, or 32 at hd 256 and 512, else the decode kernel;
 * at hd 64 and 128 with more than 128 rows per KV head, one or two row tiles
 * per thread block, whichever the planner estimates faster), 1 = always the
 * decode kernel, 2 = always the tensor-core kernels, with two row tiles per
 * thread block wherever that kernel applies (hd 64 and 128, more than 128 rows
 * per KV head), 3 = always the tensor-core kernels, one row tile per thread
 * block, and the row-tile kernel (hd <= 256) with its P V product in the "SS"
 * form (P staged in shared memory) instead of the default "TS" form (P
 * written over S in tensor memory and read from there as the MMA's A operand;
 * CURRENT_ISSUE.md "Next steps", TS MMA for PV), 4 = always the tensor-core
 * kernels, one row tile per thread block, TS form.  Meant for tests and
 * measurements that compare kernels on one shape; results agree within the
 * documented tolerance.  For fmha_fwd_kv4 and fmha_fwd_paged, 1 selects
 * their mma.sync kernel and 2 to 4 their tensor-core kernel.  Returns FMHA_ERR_SHAPE for other values.
 */
int fmha_set_kernel_path(int path);

/*
 * fmha_fwd_noalloc -- fmha_fwd for callers that cannot allocate device memory.
 * (This entry point has no counterpart on the pages the method comes from.)
 *
 * Some callers must not allocate: an inference runtime that reserves all of
 * its device memory up front and accounts for every byte, code that runs on a
 * strict memory budget, or a hot loop that must not risk the synchronisation
 * and latency that cudaMalloc/cudaFree (or a pool growing) can bring.  For
 * them this call computes what fmha_fwd computes, with the same plan, the
 * same kernels and the same partial format (fp32, or fp16 with range factors
 * on the hd-512 tensor-core kernel; see fmha_fwd), so its results are
 * fmha_fwd's bit for bit, and it calls no allocating routine: when the plan
 * splits the KV range, the partials go to one fixed scratch array of
 * FMHA_NOALLOC_SCRATCH_BYTES (32 MiB) that is part of the library's device
 * image, so every GPU that loads the library holds it until the process exits.
 *
 * - A shape whose partials (fmha_fwd_plan's chunk count times the rows, in
 *   that format) exceed the scratch is rejected with FMHA_ERR_WORKSPACE and a
 *   message naming both sizes; nothing is launched.  Shapes that fmha_fwd_plan
 *   does not split need no scratch at all.
 * - The first call on each device looks up the scratch's device address
 *   (cudaGetSymbolAddress, with that device current) and keeps it for the
 *   life of the process; make that first call before any stream capture.  The
 *   library (this call, and the status word every call uses) must not be used
 *   on a device after cudaDeviceReset: the addresses it kept belong to the
 *   context that the reset destroyed.
 * - Every call on a device shares the one scratch array, which keeps the last
 *   call's contents.  Nothing in it needs to start at zero: each call writes
 *   every partial before its merge reads it.  Calls whose work overlaps on the
 *   GPU (for example on two streams without ordering between them) race on the
 *   scratch and may return wrong results; order them on one stream or with
 *   events.
 * Arguments, layouts and errors are those of fmha_fwd.
 */
#define FMHA_NOALLOC_SCRATCH_BYTES (32u << 20)
int fmha_fwd_noalloc(const void* q, const void* k, const void* v, void* o, float* lse,
                     int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                     float scale, int window, int causal, fmha_stream_t stream);

/*
 * Serving operators around the forward (no counterpart on the pages the method
 * comes from).  All of them are stream-ordered, allocate nothing and keep
 * nothing between calls; a NULL-able argument says so.  Tensors are contiguous
 * device memory, 16-byte aligned unless said otherwise, and outputs may not
 * overlap inputs.
 */

/*
 * fmha_qk_norm_rope -- the rows of a QKV projection to what the forward takes.
 *
 * qkv: [batch, T] rows of (n_h + 2 n_kv_h) * hd bf16 elements (the query
 *   heads, the key heads, the value heads), row (b, t) at element
 *   b * batch_stride + t * token_stride; both strides multiples of 8,
 *   token_stride at least a row.
 * q_weight, k_weight: [hd] fp32.  With a weight each head row x of that kind
 *   becomes x * rsqrt(mean(x^2) + eps) * weight; NULL leaves it as it is.
 * cos_sin: [max_pos, rot] fp32, row p the rot / 2 cosines and then the rot / 2
 *   sines of position p's angles.  Pair i of a query or key row is columns (i,
 *   rot / 2 + i), or (2 i, 2 i + 1) when interleaved is 1, and becomes
 *   (lo cos_i - hi sin_i, hi cos_i + lo sin_i); columns from rot on stay.  rot is
 *   a multiple of 8 up to hd; 0 is no rotation (cos_sin and positions are not
 *   read then, and no token is padding).
 * positions: [batch, T] int32.  A token whose position is outside
 *   [0, max_pos) is padding: none of its outputs is written.
 * q: [batch, n_h, T, hd]; k, v: [batch, n_kv_h, kv_rows, hd], the token's row at
 *   kv_start[b] + t (kv_start NULL: 0); a row outside [0, kv_rows) is not
 *   written.  (fmha_fwd and fmha_fwd_first take every row of K and V as a key.)
 *   Norm and rotation are computed in fp32 and rounded to bf16 once;
 *   V is copied bit for bit.
 */
int fmha_qk_norm_rope(const void* qkv, long long batch_stride, long long token_stride,
                      const float* q_weight, const float* k_weight, float eps,
                      const float* cos_sin, const int* positions, int max_pos, int rot, int interleaved,
                      void* q, void* k, void* v, const int* kv_start, int kv_rows,
                      int batch, int T, int n_h, int n_kv_h, int hd, fmha_stream_t stream);

/*
 * A KV cache held in 4 bits, in the NVFP4 format of fmha_fwd_nvfp4:
 *   codes  [batch, n_kv_h, cap, hd / 2] bytes, scales [batch, n_kv_h, cap, hd / 16]
 * for K and for V, each with a global scale (k_global, v_global; finite, > 0).
 * cap, the rows per sequence and head, is a multiple of 16.
 *
 * fmha_kv4_append quantises k and v [batch, n_kv_h, T, hd] bf16 as
 * fmha_quantize_nvfp4 does (on the bf16 values widened to fp32) and writes row
 * t of sequence b to cache row start[b] + t (start: [batch] int32); a row
 * outside [0, cap) is left out.  k_out and v_out, both or neither:
 * [batch, n_kv_h, T, hd] bf16, the values that the written rows stand for
 * (global * scale * code, rounded to bf16; rows left out of the cache are left
 * unwritten here too).
 */
int fmha_kv4_append(const void* k, const void* v, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                    const int* start, float k_global, float v_global, void* k_out, void* v_out,
                    int batch, int n_kv_h, int T, int cap, int hd, fmha_stream_t stream);

/*
 * The plan of fmha_fwd_kv4: returns the number of KV chunks for sequences of up
 * to s_k keys; ragged: 1 when the call gives seq_lens, else 0.  *kv_chunk (may
 * be NULL) holds the chunk length asked for, in keys, 0 for the library's choice,
 * and receives the one used (a multiple of the kernel's key tile).
 */
int fmha_fwd_kv4_plan(int batch, int n_h, int n_kv_h, int T, int s_k, int hd, int window, int n_first, int causal,
                      int ragged, int* kv_chunk);

/*
 * The forward over a 4-bit cache: O (bf16) and LSE (fp32) as fmha_fwd_sink, with
 * K and V the values that the cache stands for.
 *
 * seq_lens: [batch] int32, the keys of each sequence (clamped to [0, s_k]), or
 *   NULL: s_k each.  s_k <= cap bounds them on the host and shapes the launch.
 *   Rows of the cache from a sequence's length on, and keys that no row attends,
 *   reach no result; V's scales have to be numbers at keys that some row attends.
 *   A NaN score of an attended key (a NaN in the query row or in a K scale) makes
 *   O and LSE of its row NaN, whatever the number of chunks.
 * Query row t of a sequence with len keys sits at position len - T + t; with
 *   causal, a row at a negative position attends nothing (O = 0, LSE = -inf, or
 *   the sink's).
 * n_first: with a window, the keys j < n_first stay attended as well (still
 *   subject to causal).
 * sink: [n_h] fp32 logits or NULL.
 * kv_chunk: keys per split-KV chunk, 0 for the library's choice.
 * workspace: fmha_workspace_bytes(batch, n_h, T, hd, n_splits) bytes for the
 *   partials when fmha_fwd_kv4_plan (same arguments, same kv_chunk) returns
 *   n_splits > 1, else unused; FMHA_ERR_WORKSPACE if it is smaller.  Two calls
 *   that may run at the same time need two workspaces.
 */
int fmha_fwd_kv4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                 const int* seq_lens, void* o, float* lse, const float* sink, float k_global, float v_global,
                 int batch, int n_h, int n_kv_h, int T, int s_k, int cap, int hd, float scale,
                 int window, int n_first, int causal, int kv_chunk, void* workspace, size_t workspace_bytes,
                 fmha_stream_t stream);

/*
 * fmha_fwd_first -- fmha_fwd_sink with a few first keys that a sliding window
 * does not hide: row t at position p = s_k - T + t attends key j iff
 *     (j <= p with causal)  and  (j > p - window  or  j < n_first).
 * Without a window (0, or one of at least s_k keys) n_first changes nothing.
 * Only the first keys' tiles and the window's keys are read.  Keys that no row
 * of the call attends do not reach any result, whatever memory holds there; V
 * has to be finite at keys that some row of the sequence attends.  A NaN score leaves
 * its row's O and LSE undefined, as in fmha_fwd (fmha_fwd_kv4 makes both NaN).
 * sink: [n_h] fp32 logits or NULL.  Kernels, plan and partial format are those of
 * fmha_fwd; the partials live in `workspace`, of at least
 * fmha_fwd_first_workspace_bytes(same shape) bytes (0: none needed; also 0 for an
 * invalid shape, which the call then refuses), 16-byte aligned.  Two calls that
 * may run at the same time need two workspaces.
 */
size_t fmha_fwd_first_workspace_bytes(int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                                      int window, int n_first, int causal);
int fmha_fwd_first(const void* q, const void* k, const void* v, void* o, float* lse, const float* sink,
                   int batch, int n_h, int n_kv_h, int T, int s_k, int hd,
                   float scale, int window, int n_first, int causal,
                   void* workspace, size_t workspace_bytes, fmha_stream_t stream);

/*
 * The serving operators with their arguments in one struct: the same calls, for
 * bindings in which every argument of a foreign call costs time (from Python's
 * ctypes, 26 arguments took 2.7 us, one takes 0.4; the Python binding packs them in
 * csrc/tensor_args.cpp).  Fields as the arguments of the call of the same name.
 */
struct fmha_qk_norm_rope_args {
    const void* qkv;
    const float *q_weight, *k_weight, *cos_sin;
    const int* positions;
    void *q, *k, *v;
    const int* kv_start;
    fmha_stream_t stream;
    long long batch_stride, token_stride;
    float eps;
    int max_pos, rot, interleaved, kv_rows, batch, T, n_h, n_kv_h, hd;
};
struct fmha_kv4_append_args {
    const void *k, *v;
    void *k_codes, *k_scales, *v_codes, *v_scales;
    const int* start;
    void *k_out, *v_out;
    fmha_stream_t stream;
    float k_global, v_global;
    int batch, n_kv_h, T, cap, hd, reserved;
};
struct fmha_fwd_kv4_args {
    const void *q, *k_codes, *k_scales, *v_codes, *v_scales;
    const int* seq_lens;
    void* o;
    float* lse;
    const float* sink;
    void* workspace;
    size_t workspace_bytes;
    fmha_stream_t stream;
    float k_global, v_global, scale;
    int batch, n_h, n_kv_h, T, s_k, cap, hd, window, n_first, causal, kv_chunk;
};
struct fmha_fwd_first_args {
    const void *q, *k, *v;
    void* o;
    float* lse;
    const float* sink;
    void* workspace;
    size_t workspace_bytes;
    fmha_stream_t stream;
    float scale;
    int batch, n_h, n_kv_h, T, s_k, hd, window, n_first, causal;
};
int fmha_qk_norm_rope_packed(const struct fmha_qk_norm_rope_args* args);
int fmha_kv4_append_packed(const struct fmha_kv4_append_args* args);
int fmha_fwd_kv4_packed(const struct fmha_fwd_kv4_args* args);
int fmha_fwd_first_packed(const struct fmha_fwd_first_args* args);

/*
 * A KV cache in pages.  Sequences share a pool of pages of `page` rows each, a power of
 * two from 16 to 65536:
 *   k_pages, v_pages [n_pages, n_kv_h, page, hd], in one of two forms:
 *     bf16 (k_scales and v_scales NULL), or 8 bits: E4M3 codes and a scale byte for every row,
 *     k_scales, v_scales [n_pages, n_kv_h, page], where byte e stands for 2^(e - 127).  A row's
 *     scale is the smallest power of two, from 2^-127 on, that brings its largest magnitude to 448 or
 *     less; code = E4M3(x / scale), to nearest, ties to even (x / scale is exact, so each value is
 *     rounded once); the row stands for scale * code, which is a bf16 value again (below 2^-133 the
 *     nearest one).  A row with a NaN or an infinity gets the byte 255 and reads as NaN throughout.
 *     The codes 0x7F and 0xFF (E4M3's NaN) are never written; in rows that a caller fills otherwise they
 *     may not stand at keys that are attended.
 *   block_table [batch, table_width] int32: row i of sequence b lies in page
 *     block_table[b, i / page], row i % page.  An entry outside [0, n_pages) is a page that is
 *     not there: its rows are not written, not read back and attended by no query row (so the pages
 *     behind a sliding window can be given back).  Sequences may share pages, as far as no two calls or
 *     sequences write one row at the same time.
 * n_pages * n_kv_h * page is at most 2^31 - 65537; offsets are 64-bit.  Pages and scales are 16-byte
 * aligned.
 *
 * New tokens come in one of two forms: T for each sequence (cu_q NULL), or ragged,
 * `total` token rows of which sequence b has cu_q[b] .. cu_q[b + 1] - 1 (cu_q: [batch + 1] int32, not
 * falling).  Rows outside [cu_q[0], cu_q[batch]) are no tokens and nothing is written for them.  An
 * input's three strides, in elements, are those of the sequence (not used with cu_q), the token
 * and the head: multiples of 8, not negative; hd elements lie next to each other.
 *
 * These calls take their arguments in one struct (see below); the fields have the order given there.  Like the
 * other serving operators they are stream-ordered, allocate nothing and keep nothing between calls.
 */

/*
 * fmha_paged_append -- K and V rows of new tokens into the cache: token t of sequence b to row
 * start[b] + t (start: [batch] int32; negative rows, and rows behind the block table, are left out).
 * Where two tokens of a call go to one row of the pool, what it holds afterwards is undefined.
 */
struct fmha_paged_append_args {
    const void *k, *v; /* bf16, n_kv_h heads */
    void *k_pages, *v_pages;
    void *k_scales, *v_scales; /* both NULL: bf16 pages */
    const int *block_table, *start, *cu_q;
    fmha_stream_t stream;
    long long k_strides[3], v_strides[3]; /* sequence, token, head */
    int batch, T, total, n_kv_h, hd, page, n_pages, table_width;
};
int fmha_paged_append(const struct fmha_paged_append_args* args);

/*
 * fmha_paged_gather -- rows of the cache back as contiguous bf16: k, v [batch, n_kv_h, rows, hd],
 * row i of sequence b being cache row start[b] + i (start NULL: i).  Rows at or behind the sequence's
 * length seq_lens[b], and those whose page is not there, are left as they are.
 */
struct fmha_paged_gather_args {
    const void *k_pages, *v_pages, *k_scales, *v_scales;
    const int *block_table, *seq_lens, *start;
    void *k, *v;
    fmha_stream_t stream;
    int batch, rows, n_kv_h, hd, page, n_pages, table_width, reserved;
};
int fmha_paged_gather(const struct fmha_paged_gather_args* args);

/*
 * fmha_fwd_paged -- the forward for new tokens over the cache, their own rows already appended:
 * O (bf16) and LSE (fp32), [batch, n_h, T, hd] and [batch, n_h, T], or with cu_q [total, n_h, hd]
 * and [total, n_h].
 *
 * seq_lens: [batch] int32, the keys of each sequence, new tokens included (clamped to [0, s_k]); s_k bounds
 *   them on the host and shapes the launch: the chunks divide s_k keys, whatever a sequence has, so a bound far
 *   above the lengths (a block table for the longest context, say) costs time: one user's step over 8191 keys
 *   takes 16 us with s_k = 8192 and 79 with 131072.  Rows of the pages from a sequence's length on reach no
 *   result.
 * T: with cu_q the most tokens that a sequence has, by which the kernel is chosen (a sequence with more
 *   is computed all the same).  A bound far above what the sequences have costs time: 32 sequences of one
 *   token over 8191 keys take 165 us with T = 1 and 184 with T = 32, in 8 bits 117 and 275.
 * Token t of a sequence with len keys and n new tokens sits at position p = len - n + t and attends
 *   key j < len iff j's page is there, j <= p with causal, and with a window (j > p - window or
 *   j < n_first).  A row that attends nothing gets O = 0 and LSE = -inf, or the sink's.
 * sink: [n_h] fp32 logits or NULL (fmha_fwd_sink).
 * K may hold anything at keys that a row does not attend, V at keys that no row of the sequence attends;
 *   V has to be finite at the others, and below 2^120 over the number of keys (O is summed in fp32 before it is
 *   divided, under weights of up to 2^8).  A NaN score of an attended key makes O and LSE of its
 *   row NaN, whatever the number of chunks.
 * Weights are rounded to bf16 before they meet V; scores, sums and O are fp32.  With 8-bit pages and few rows
 *   the operands are fp16 times powers of two: elements of q more than 2^28 below their row's largest
 *   lose bits and those more than 2^39 below it are lost, and a weight times its V row's scale is kept to 2^-37 of the
 *   largest such scale.
 * n_splits: chunks that a sequence's keys are divided into, 0 for the library's choice.
 * workspace: fmha_fwd_paged_plan(same arguments) chunks > 1 need
 *   fmha_workspace_bytes(1, n_h, rows, hd, chunks) bytes, rows being batch * T or total,
 *   else unused; FMHA_ERR_WORKSPACE if it is smaller.  (The call may take fewer chunks than that where the block
 *   table holds fewer than s_k keys, never more.)  Two calls that may run at the same time need two.
 */
struct fmha_fwd_paged_args {
    const void *q, *k_pages, *v_pages, *k_scales, *v_scales;
    const int *block_table, *seq_lens, *cu_q;
    void* o;
    float* lse;
    const float* sink;
    void* workspace;
    size_t workspace_bytes;
    fmha_stream_t stream;
    long long q_strides[3]; /* sequence, token, head */
    float scale;
    int batch, T, total, n_h, n_kv_h, hd, page, n_pages, table_width, s_k, window, n_first, causal, n_splits, reserved;
};
int fmha_fwd_paged(const struct fmha_fwd_paged_args* args);

/* The number of chunks that fmha_fwd_paged uses (ragged: 1 with cu_q; codes: 1 for 8-bit pages); a negative FMHA_ERR_* code for invalid arguments. */
int fmha_fwd_paged_plan(int batch, int T, int total, int n_h, int n_kv_h, int hd, int page, int s_k, int window, int n_first,
                        int causal, int ragged, int codes, int n_splits);

/* ABI version: major * 10000 + minor * 100 + patch. */
int fmha_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FMHA_GB300_H */
