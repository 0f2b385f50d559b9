/*
 * qnt.h -- C ABI of libqnt: round-to-nearest (RTN) group-wise 4-bit weight
 * quantization and decode-time fused-dequant GEMV / small-batch GEMM on one
 * NVIDIA B200 (sm_100a).
 *
 * What the operations are, by source page:
 *  - "Is (Selective) Round-To-Nearest Quantization All You Need?" (Kogan,
 *    arXiv 2505.15909), English abstract: RTN is cheap to apply, its token
 *    generation throughput with fused-dequant kernels can beat advanced
 *    methods, and accuracy improves by raising the precision of selected
 *    layers / modules -> qnt_quantize, qnt_gemv / qnt_gemm, qnt_table_*.
 *  - "Revisiting Block-based Quantisation" (Zhang et al., arXiv 2310.05079),
 *    English abstract: scaling factors shared across a block of packed numbers
 *    -> the `group` (block) size along the input dimension.
 *  - "The Power of Negative Zero: RaZeR" (Chen et al., arXiv 2501.04052),
 *    English abstract and method section: FP4 whose negative-zero code is
 *    remapped to a special value, and a fast fused-dequant GEMV -> QNT_FP4_RAZER.
 *  - "AFPQ: Asymmetric Floating Point Quantization" (Zhang et al., arXiv
 *    2311.01792), English abstract: separate scales for positive and negative
 *    values -> QNT_FP4_AFPQ.
 * The pages give no formulas; the exact arithmetic of each format is stated
 * below with each enum value.
 *
 * Conventions (all entry points):
 *  - W is [N][K] row-major (N = output features, K = input features, the
 *    PyTorch nn.Linear convention).  Groups are runs of `group` consecutive
 *    weights along K inside one row.  x is [K], y is [N]; X is [M][K] and Y
 *    is [M][N], row-major.
 *  - Every buffer argument named d_* or documented "device" is device memory
 *    that the CALLER allocates and owns.  The library never allocates or frees
 *    memory, keeps no state between calls and is safe to call from several
 *    host threads.  Work is enqueued asynchronously on `stream` (a
 *    cudaStream_t passed as void*; NULL = the legacy default stream).
 *  - The return value is the host-side validation result.  On any error
 *    nothing is launched.  Device-detected conditions (non-finite weights,
 *    scale overflow, a bounded wait that expired) are written to the optional
 *    device int *d_status (may be NULL) with an atomic max, never cleared by
 *    the library: zero it before the call, read it after synchronizing.
 *  - Pointers to packed codes, metadata, activations and outputs must be 16-byte
 *    aligned (QNT_ERR_ALIGN otherwise).
 */
#ifndef QNT_H_
#define QNT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QNT_VERSION 3

/* Largest K that qnt_gemv, qnt_gemm and qnt_gemv_seq accept: every GEMV
 * kernel stages the activation vector (2K bytes) in shared memory next to its
 * weight ring, and the CUDA-core kernel (INT8, FP16, batch 2) would not fit at
 * K = 65536.  qnt_quantize accepts K up to 2^20. */
#define QNT_MAX_GEMV_K 32768

/* Weight formats.  h(.) = round-to-nearest-even to fp16; every quotient below
 * is one IEEE binary32 division; rint = round half to even; a scale that
 * rounds to zero is stored as 1.0; a scale that overflows fp16 sets
 * QNT_ERR_RANGE in *d_status. */
typedef enum {
  /* Asymmetric INT4 (asymmetric INT named by the RaZeR and AFPQ abstracts):
   * s = h((max - min) / 15), z = clamp(rint(-min / s), 0, 15),
   * q = clamp(rint(w / s) + z, 0, 15), dequant = (q - z) * s.
   * Metadata 2.5 bytes per group (fp16 scale, 4-bit zero). */
  QNT_INT4_ASYM = 1,
  /* Symmetric FP4 E2M1 (sign-magnitude 4-bit float of the RaZeR page): codes
   * 0..7 = 0, .5, 1, 1.5, 2, 3, 4, 6, bit 3 = sign; s = h(absmax / 6);
   * code = nearest value to w / s (ties to even mantissa, saturating at 6);
   * magnitude 0 is always code 0 (0b1000 is never produced). 2 bytes/group. */
  QNT_FP4_E2M1 = 2,
  /* AFPQ: s+ = h(max(max, 0) / 6), s- = h(max(-min, 0) / 6); positive weights
   * use s+, negative weights s- (sign bit set); dequant = e2m1(code) * s+ or
   * * s-.  4 bytes/group. */
  QNT_FP4_AFPQ = 3,
  /* RaZeR: E2M1 whose code 0b1000 decodes to a special value sv chosen per
   * group from {+5, -5, +8, -8} (2-bit selector 0..3 in that order).  For each
   * candidate: s = h(absmax / max(6, |sv|)), codes = nearest of the 15 regular
   * values and sv (a tie with sv goes to the regular value); the candidate with
   * the smallest binary64 sum of squared errors (summed as a balanced binary
   * tree in index order) wins, ties to the smaller selector.  2.25 bytes/group. */
  QNT_FP4_RAZER = 4,
  /* INT8 symmetric per output channel (selective precision): s = h(absmax_row
   * / 127), q = clamp(rint(w / s), -127, 127).  group must equal K. */
  QNT_INT8_PERCHAN = 5,
  /* FP16 (selective precision, no quantization): code = h(w).  group == K. */
  QNT_FP16 = 6
} qnt_fmt;

/* Activation / output element type.  y and Y use the activation type. */
typedef enum { QNT_F16 = 0, QNT_BF16 = 1 } qnt_dtype;

/* Error codes. */
enum {
  QNT_OK = 0,
  QNT_ERR_ARG = 1,       /* null pointer, unknown format / dtype, M out of range */
  QNT_ERR_SHAPE = 2,     /* N < 1, K % 128 != 0, group not in {32,64,128} (4-bit) or != K,
                            K > QNT_MAX_GEMV_K for a GEMV / GEMM */
  QNT_ERR_ALIGN = 3,     /* a buffer is not 16-byte aligned */
  QNT_ERR_CUDA = 4,      /* the kernel launch failed */
  QNT_ERR_TIMEOUT = 5,   /* (device) a bounded wait for an asynchronous copy expired */
  QNT_ERR_NONFINITE = 6, /* (device) NaN or Inf in W; codes are unspecified */
  QNT_ERR_RANGE = 7,     /* (device) a scale or FP16 code overflowed fp16 */
  QNT_ERR_PAGES = 8      /* (device) the free pages do not cover a request's new tokens */
};

/* Shape and format of one quantized matrix. */
typedef struct {
  int32_t fmt;    /* qnt_fmt */
  int32_t N;      /* output features (rows of W), >= 1 */
  int32_t K;      /* input features, a positive multiple of 128 */
  int32_t group;  /* 32, 64 or 128 for 4-bit formats; K for INT8 / FP16 */
} qnt_desc;

/*
 * Packed storage layout (one layout serves qnt_gemv and qnt_gemm).
 *
 * 4-bit codes: rows are stored in groups of eight.  Row group R = n/8 occupies
 * 4K bytes at byte R*4K (the buffer holds ceil(N/8)*8 rows; the contents of
 * padding rows are unspecified and never reach a result).  Within a group,
 * block b (weights 128b..128b+127 of each of its eight rows) occupies 512
 * bytes at offset 512b; row i = n%8 sits at offset 64i inside the block as four
 * 16-byte chunks, chunk c (weights 128b+32c .. 128b+32c+31 of the row) at byte
 * 64i + 16*(c XOR ((i/2) % 4)).  The 16 bytes of a chunk are four little-endian
 * 32-bit words, and nibble p (bits 4p..4p+3) of word j holds chunk weight
 *   QNT_INT4_ASYM:                 16*(p%2) + 4j + 2*((p/2)%2) + p/4
 *   QNT_FP4_E2M1 / AFPQ / RAZER:   8j + p
 * So 256 consecutive weights of eight rows are one contiguous 1 KB run (one
 * bulk copy), eight threads that read the same chunk of eight rows of a group
 * (or the four chunks of two rows) hit distinct shared-memory bank groups, and
 * the INT4 order turns a word into
 * fp16 pairs with two masks and one shift (low nibbles give chunk weights 0..15
 * in order, high nibbles 16..31).  FP4-family bytes hold two consecutive
 * weights, low nibble first.
 * INT8 codes: row-major int8 [N][K].  FP16 codes: row-major fp16 [N][K].
 *
 * Metadata buffer (byte offsets), G = K/group, P = N*G, group f = n*G + j:
 *   INT4:  fp16 scale[P] at 0; 4-bit zeros from Z0 = round_up(2P, 256):
 *          zero of group f in byte Z0 + f/2, low nibble when f is even;
 *          the zero plane is round_up(ceil(P/2), 16) bytes long.
 *   FP4:   fp16 scale[P] at 0.
 *   AFPQ:  32-bit word[P] at 0: bits 0..15 = fp16 s+, bits 16..31 = fp16 s-.
 *   RaZeR: fp16 scale[P] at 0; 2-bit selectors from Z0 = round_up(2P, 256):
 *          selector of group f in byte Z0 + f/4, bits 2*(f%4)..2*(f%4)+1;
 *          the selector plane is round_up(ceil(P/4), 16) bytes long.
 *   INT8:  fp16 scale[N] at 0.
 *   FP16:  none (qnt_meta_bytes returns 0).
 * Every metadata length is rounded up to a multiple of 16 bytes (the GEMV
 * kernels stage whole 16-byte-aligned metadata ranges with bulk copies).
 */

/* Bytes of packed codes / metadata for a descriptor; 0 if it is invalid. */
size_t qnt_codes_bytes(const qnt_desc* desc);
size_t qnt_meta_bytes(const qnt_desc* desc);

/* Validate a descriptor: QNT_OK or the error code that the calls would return. */
int qnt_check_desc(const qnt_desc* desc);

/*
 * qnt_quantize -- RTN-quantize W into packed codes and metadata (the offline
 * step of the RTN page; data-free, no calibration).
 *   d_W        device, fp32 [N][K] row-major, read only.
 *   d_codes    device, qnt_codes_bytes(desc) bytes, written.
 *   d_meta     device, qnt_meta_bytes(desc) bytes, written (may be NULL for FP16).
 *   d_status   device int or NULL: QNT_ERR_NONFINITE / QNT_ERR_RANGE.
 * Bit-exact with the definitions above.  The call ends with an empty kernel on
 * the stream, so that a GEMV enqueued right after it (which requests its codes
 * and metadata before waiting for the preceding kernel, see qnt_gemv) sees them.
 */
int qnt_quantize(const qnt_desc* desc, const float* d_W, void* d_codes, void* d_meta,
                 int* d_status, void* stream);

/*
 * qnt_gemv -- batch-1 fused-dequant GEMV, y[n] = sum_k dq(n, k) * x[k]
 * (the decode-time GEMV of the RaZeR and RTN pages).
 *   d_codes, d_meta  device, packed as above (from qnt_quantize or the layout).
 *   d_x        device, [K] fp16 or bf16 (xdtype).
 *   d_y        device, [N] in the same type, written.
 *   d_status   device int or NULL: QNT_ERR_TIMEOUT if a staging wait expires.
 * Ordering (programmatic dependent launch): the GEMV kernels of qnt_gemv and
 * qnt_gemm start while the preceding kernel on the stream is still running and
 * request their codes and metadata at once; only the reads of x and the writes
 * of y wait for that kernel to complete.  So the kernel IMMEDIATELY preceding
 * the call on the stream must not write d_codes or d_meta.  qnt_quantize
 * complies (it ends with an empty kernel); after any other kernel that writes
 * the weights, enqueue another kernel or a copy in between, or synchronize.
 * Accuracy: |y - y_exact| <= 4e-3 * sum_k |dq(n,k) x[k]| per element.  Every
 * product is formed from exact fp16 operands and accumulated in fp32 (on the
 * CUDA cores exactly; on the tensor cores, which take batch 1 and larger
 * batches, within about 1e-4 of sum |products| as measured), with one final
 * rounding to the output type.  x is rescaled
 * internally by a power of two so fp16 arithmetic cannot overflow.
 */
int qnt_gemv(const qnt_desc* desc, const void* d_codes, const void* d_meta,
             const void* d_x, void* d_y, int xdtype, int* d_status, void* stream);

/*
 * qnt_gemm -- small-batch fused-dequant GEMM, Y[m][n] = sum_k dq(n, k) X[m][k]
 * for 1 <= M <= 128 activation rows.
 *   d_X        device, [M][K] fp16 or bf16, row-major.
 *   d_Y        device, [M][N] in the same type, written.
 * Same ordering rule (the immediately preceding kernel on the stream must not
 * write d_codes or d_meta) and accuracy statement as qnt_gemv.  Batches of 2 to
 * 8 rows of the 4-bit formats with group 128 and K a multiple of 1024 run on
 * the batch-1 kernel, the rows sharing its tensor-core MMAs, when their
 * activations fit in shared memory next to its weight ring; the other batches
 * of 3 to 128 rows of the 4-bit formats run on the tcgen05 tensor cores in one
 * pass over the weights.  d_status may also receive QNT_ERR_TIMEOUT on both.
 */
int qnt_gemm(const qnt_desc* desc, const void* d_codes, const void* d_meta,
             const void* d_X, void* d_Y, int M, int xdtype, int* d_status, void* stream);

/*
 * Sequences of batch-1 GEMVs in one launch: the linear layers of a decode step
 * (token generation with fused-dequant kernels, RTN and RaZeR pages' English
 * abstracts) run one after another on one activation vector each.  One
 * persistent kernel streams the weights of every step back to back; a step
 * with wait = k reads its x only after step i - k and every step before it
 * have written their y, so x may be (part of) one of those y.  (A decode layer:
 * o waits 1 for qkv, gate 1 for o, up 2 for o, down 1 for up.)
 */
#define QNT_SEQ_MAX_STEPS 256

typedef struct {
  qnt_desc desc;       /* 4-bit format, N, K, group: format and group equal in every step */
  const void* codes;   /* device, this step's packed codes */
  const void* meta;    /* device, its metadata */
  const void* x;       /* device, [K] activations (fp16 or bf16, as xdtype) */
  void* y;             /* device, [N] output, same type; written */
  int32_t wait;        /* k >= 1: read x after step i - k and every step before it
                          have written their y (x may be any of those y); 0: x is
                          not written by any earlier step of this call.  0 <= k <= i. */
  int32_t reserved;    /* 0 */
} qnt_seq_step;

/* Bytes of the workspace qnt_gemv_seq needs for nsteps steps (0 if nsteps is
 * out of range). */
size_t qnt_gemv_seq_work_bytes(int nsteps);

/*
 * qnt_gemv_seq -- y_i = W_i x_i for the steps i = 0 .. nsteps-1, in order.
 *   steps      HOST array of nsteps step descriptors (1 <= nsteps <=
 *              QNT_SEQ_MAX_STEPS); read during the call only.
 *   d_work     device, qnt_gemv_seq_work_bytes(nsteps) bytes, 16-byte aligned,
 *              owned by the caller: per-step completion counters.  The call
 *              clears it on the stream before the kernel; two calls that may
 *              run at the same time need two workspaces.
 *   d_status   device int or NULL: QNT_ERR_TIMEOUT if a wait expires (a step's
 *              dependency, a staging copy).
 * Step 0 starts after the preceding work on the stream has completed.  The y of
 * a step must not overlap any other step's y, x, codes or metadata except as
 * the x of a later step marked `wait`.  Accuracy as qnt_gemv.  The kernel keeps
 * one CTA on every SM for its whole duration (a cooperative launch);
 * QNT_ERR_CUDA if the GPU cannot host it.  QNT_ERR_ARG: nsteps out of range,
 * a null pointer, a format that is not 4-bit, formats / groups that differ
 * between steps, or wait outside 0..i; QNT_ERR_SHAPE / QNT_ERR_ALIGN as for
 * qnt_gemv, and QNT_ERR_SHAPE when a step's activations and staged metadata
 * do not fit in shared memory.
 */
int qnt_gemv_seq(const qnt_seq_step* steps, int nsteps, int xdtype, void* d_work, int* d_status, void* stream);

/*
 * qnt_gemv_seq_noalloc -- qnt_gemv_seq for callers that cannot allocate device
 * memory: for example a host framework whose device memory is entirely handed
 * out by its own pool, or a plug-in that is not allowed to call the CUDA
 * allocator, and so cannot provide d_work.  It computes exactly what
 * qnt_gemv_seq computes (same arguments, ordering, accuracy and errors) and
 * allocates nothing.  (No counterpart in the pages: an interface convenience.)
 *   Workspace: the per-step completion counters live in a small array that the
 *     library itself places in the memory of every GPU that loads it, for the
 *     life of the process ((QNT_SEQ_NOALLOC_MAX_STEPS + 1) * 4 bytes per GPU).
 *     Each call clears the part it uses on `stream` before its kernel; the
 *     array keeps the last call's contents afterwards.
 *   Limit: nsteps <= QNT_SEQ_NOALLOC_MAX_STEPS, else QNT_ERR_ARG.
 *   Every call shares the one array: two calls whose work overlaps on the GPU
 *     (other streams, other host threads) race and may hang until their waits
 *     expire (QNT_ERR_TIMEOUT); serialize them, or use qnt_gemv_seq with one
 *     workspace each.
 *   The first call on each device looks up the array's device address (a
 *     runtime query, no allocation); make that first call before capturing a
 *     stream into a CUDA graph.
 */
#define QNT_SEQ_NOALLOC_MAX_STEPS 256
int qnt_gemv_seq_noalloc(const qnt_seq_step* steps, int nsteps, int xdtype, int* d_status, void* stream);

/*
 * Paged 8-bit key/value cache: what a decode step keeps of its past between the
 * qkv and the o product.  ("The Power of Negative Zero: RaZeR", English
 * abstract: quantization extends from the weights to the key/value cache; the
 * pages give no formulas, so the arithmetic is the plain RTN one stated here.)
 * Three calls make a step: qnt_kv_slots gives the step's new tokens their
 * places, qnt_kv_append quantizes their keys and values into them, qnt_kv_attn
 * lets their queries attend to the cache.
 *
 * A page holds `page` consecutive tokens of one request for every head.  K and
 * V have a codes buffer and a scales buffer each:
 *   codes  uint8 [pages][heads][page][dim]      scales  fp32 [pages][heads]
 * so a scale serves the `page` tokens of a head in a page, and a value is
 * code value * scale.  INT8 byte = q + 128 with q in -127..127 (zero-extended
 * bytes are fp16 subnormals, the operand of the tensor cores); E4M3 byte =
 * the OCP 8-bit float (sign, 4 exponent, 3 mantissa bits, largest value 448).
 * Scales are finite and not negative.
 * A token's slot is page * (tokens in a page) + its place in the page.
 */
typedef enum { QNT_KV_INT8 = 1, QNT_KV_E4M3 = 2 } qnt_kv_fmt;

#define QNT_KV_MAX_ROWS 4096             /* requests in one call */
#define QNT_KV_MAX_TOKENS (1 << 30)      /* token rows in one call, and tokens of a page table (width * page) */

typedef struct {
  int32_t fmt;     /* qnt_kv_fmt */
  int32_t page;    /* tokens in a page: 16, 32, 64 or 128 */
  int32_t pages;   /* pages in the cache, >= 1; pages * page < 2^31 */
  int32_t heads;   /* key/value heads, 1..1024 */
  int32_t dim;     /* values in a head: 64, 128 or 256 */
} qnt_kv_desc;

/* Bytes of the codes buffer (and as many again for V) and of the scales buffer
 * (likewise); 0 if the descriptor is invalid. */
size_t qnt_kv_codes_bytes(const qnt_kv_desc* desc);
size_t qnt_kv_scales_bytes(const qnt_kv_desc* desc);

/* QNT_OK or the error code that the calls would return. */
int qnt_check_kv_desc(const qnt_kv_desc* desc);

/*
 * qnt_kv_slots -- page tables and slots of a step's new tokens (reads page and
 * pages of the descriptor).  All arrays are device int32.
 *   d_len      [rows] tokens that each request has cached, 0 for a new one.
 *   d_add      [rows] new tokens of each request (0: none); -1 releases the
 *              request's pages.
 *   d_table    [rows][width] page of each `page` tokens of a request; entries of
 *              cached tokens are read, those of new pages written, the others left.
 *   d_free     [pages] a stack, its first *d_free_count entries the free pages.
 *   d_len_out  [rows] written: d_len + d_add; 0 for a released request; d_len
 *              for one that got no room.
 *   d_cu       [rows + 1] written: first token row of each request (the requests'
 *              new tokens one after another), at most `tokens`.
 *   d_slots    [tokens] written: slot of each token row; -1 for the tokens of a
 *              request that got no room and for the rows behind the last token.
 *   d_free_count_out  [1] written.
 * First every released request's pages go onto the stack (requests in order,
 * pages in order), then the requests take new pages from its top, in order.
 * The inputs d_len, d_add and d_free_count are not written, entries of d_free
 * below *d_free_count neither, and no output may overlap an input, so a
 * repeated call gives the same outputs.  Requests get no room, and the others
 * are served, (a) from the first one on that the stack does not cover
 * (QNT_ERR_PAGES; those that need no new page are served all the same), (b) when
 * they would pass width * page tokens or their token rows `tokens`, or when
 * d_len is outside 0..width * page (QNT_ERR_ARG in *d_status).  A page number
 * outside the cache is handed on as it is, and its tokens get the slot 2^31 - 1,
 * which qnt_kv_append refuses.  d_add below -1 is taken as -1 (QNT_ERR_ARG).  If more
 * pages are released than the cache has, the stack ends full (QNT_ERR_ARG).
 * The pages of a request are the first ceil(d_len / page) entries of its row, no
 * others.  A caller that lowers d_len between two calls (drafted tokens that were
 * refused) and thereby leaves a page behind the end puts it back itself: its entry
 * goes to d_free[*d_free_count], and *d_free_count up by one, before the next call.
 * 1 <= rows <= QNT_KV_MAX_ROWS, 1 <= width, width * page and tokens at most
 * QNT_KV_MAX_TOKENS, else QNT_ERR_SHAPE (here and below).
 */
int qnt_kv_slots(const qnt_kv_desc* desc, const int32_t* d_len, const int32_t* d_add, int32_t* d_table, int32_t* d_free,
                 const int32_t* d_free_count, int32_t* d_len_out, int32_t* d_cu, int32_t* d_slots,
                 int32_t* d_free_count_out, int rows, int width, int tokens, int* d_status, void* stream);

/*
 * qnt_kv_append -- quantizes the keys and values of token rows into their slots.
 *   d_kcodes, d_vcodes, d_kscales, d_vscales  the cache, updated.
 *   d_k, d_v   device, [tokens] rows of heads * dim fp16 or bf16 (xdtype), rows
 *              `stride` elements apart (a multiple of 8, >= heads * dim): slices
 *              of the qkv product's output will do.
 *   d_slots    device int32 [tokens], as from qnt_kv_slots; rows with a negative
 *              slot are skipped.
 * Token rows with consecutive slots of one page are a run.  For every run, head
 * and of K and V: a = max |x| over the run, s = fp32(a / 127) (E4M3: a / 448); a
 * run that does not begin its page keeps the page's scale if that is larger.
 * The codes are the code values nearest to x / s (the real quotient, ties to
 * even; 0 if s = 0).  If the scale of a page grows from s0 to s, the codes of
 * the tokens before the run become those nearest to (code value * s0) / s.  The
 * page's tokens behind the run are left as they are; their values are
 * unspecified until they are written.  A page must not take part in two runs of
 * one call: where a second one follows the first with nothing or only skipped
 * rows in between it is not written (QNT_ERR_ARG in *d_status); elsewhere the
 * page's content is unspecified.  A slot beyond the cache is
 * skipped (QNT_ERR_ARG).  Non-finite x: QNT_ERR_NONFINITE, the scale is that of
 * the finite values and the codes of the others are finite but unspecified.
 * tokens = 0 does nothing.  Bit-exact with the definition.
 */
int qnt_kv_append(const qnt_kv_desc* desc, void* d_kcodes, void* d_vcodes, float* d_kscales, float* d_vscales,
                  const void* d_k, const void* d_v, int64_t stride, const int32_t* d_slots, int tokens, int xdtype,
                  int* d_status, void* stream);

/*
 * qnt_kv_attn -- attention of the new tokens over the cache.  Query head h uses
 * key/value head h / (heads / desc->heads).  Token t of the n = d_cu[b+1] -
 * d_cu[b] new tokens of request b has position p = d_len[b] - n + t and sees the
 * cached tokens j <= p, with window > 0 only j > p - window:
 *   y = sum_j softmax_j(scale * q . k_j) v_j        (0 if it sees none)
 *   d_q        device, [tokens] rows of heads * dim fp16 or bf16 (xdtype), rows
 *              q_stride elements apart (a multiple of 8, >= heads * dim).
 *   d_y        device, the same with y_stride, written in the same type for the
 *              token rows of requests; other rows are left as they are.
 *   heads      query heads, a multiple of desc->heads, at most 65536; tokens * heads /
 *              desc->heads at most QNT_KV_MAX_TOKENS.
 *   d_cu       device int32 [rows + 1] as from qnt_kv_slots.
 *   d_len      device int32 [rows], cached tokens with the new ones among them
 *              (qnt_kv_slots' d_len_out).
 *   d_table    device int32 [rows][width].
 *   max_new    the largest n as far as the caller knows it (>= 1): it chooses the
 *              kernel, not what is computed.
 *   scale      at most 2^64 in magnitude.   window  0: none.
 *   d_work     device, qnt_kv_attn_work_bytes bytes for these heads and max_new,
 *              16-byte aligned, zeroed by the caller before its first use; every
 *              call leaves it ready for the next, of whatever sizes it is large
 *              enough for.  Two calls that may run at the same time need two.
 * Products are of exact fp16 operands with fp32 accumulation (q is rescaled by a
 * power of two per row where it is bf16), the softmax is fp32, its weights are
 * rounded to fp16 for the second product (relative error 2^-11 or absolute error
 * 2^-32 of the largest), and y once to its type.  (Requests of more than 32 query
 * rows a key/value head may go to the tcgen05 tensor cores.  There a weight also
 * carries its page's V scale: its relative error is 2^-11 or its absolute error 2^-30
 * of the largest weight and of the largest V scale of the 128 tokens around it (or
 * 2^-100), and in pages below 2^-40 of that scale the values count as 0, their weights
 * in full.)
 * All of that is fp32: the terms scale * q_i * k_i of a logit and the logit have to
 * stay below 2^120 and cached values below 2^96 in magnitude.
 * The bytes of tokens that no query sees may be anything; a visible E4M3 byte must
 * not be 0x7F or 0xFF (NaN; qnt_kv_append writes none).
 * A page number outside the cache is read as page 0, and d_len beyond
 * width * page is cut there (QNT_ERR_ARG in *d_status).
 */
size_t qnt_kv_attn_work_bytes(const qnt_kv_desc* desc, int heads, int max_new);   /* 0 on bad arguments */
int qnt_kv_attn(const qnt_kv_desc* desc, const void* d_kcodes, const void* d_vcodes, const float* d_kscales,
                const float* d_vscales, const void* d_q, int64_t q_stride, void* d_y, int64_t y_stride, int heads,
                const int32_t* d_cu, const int32_t* d_len, const int32_t* d_table, int rows, int width, int tokens,
                int max_new, float scale, int window, void* d_work, int xdtype, int* d_status, void* stream);

/*
 * Selective precision (RTN page: raise the precision format of chosen layers
 * and modules).  A host-side table of ordered rules; qnt_table_lookup returns
 * the format and group of the first rule whose pattern matches the module name
 * ('*' matches any run of characters, '?' one character), else the default.
 * The table is a host object owned by the caller; not thread-safe for
 * concurrent modification.
 */
typedef struct qnt_table qnt_table;
qnt_table* qnt_table_create(int default_fmt, int default_group); /* NULL on bad args */
int qnt_table_set(qnt_table* t, const char* module_pattern, int fmt, int group);
int qnt_table_lookup(const qnt_table* t, const char* module_name, int* fmt, int* group);
int qnt_table_size(const qnt_table* t);
void qnt_table_destroy(qnt_table* t);

/* Static description of an error code. */
const char* qnt_strerror(int code);

/* After a call returned QNT_ERR_CUDA: the CUDA runtime's name and description
 * of the error, for the calling host thread ("" if none).  The text stays
 * valid until the thread's next failing call. */
const char* qnt_last_error(void);

/* Library version (QNT_VERSION of the build). */
int qnt_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QNT_H_ */
