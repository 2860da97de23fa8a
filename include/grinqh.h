/*
 * grinqh.h - C ABI of the MI355X (gfx950) decode-phase GEMV of GRINQH.
 *
 * Method source: the page "GRINQH: Graded Input-Based Quantization Hierarchy
 * for Efficient LLM Generation" (papernotes.org note on arXiv 2606.23419),
 * section 方法详解 / 关键设计 (key design) items 1-3, cited below as KD1
 * (bit assignment), KD2 (bit-planar storage) and KD3 (midpoint dequant).
 *
 * What the library computes, for one decode step (batch 1) of one linear:
 *
 *   b_i = 2 * #{k : theta_k <= |x_i|}                  KD1  (P = b_max/2 thresholds)
 *   w_hat_ij = s_j * (((q_ji >> k_i) << k_i) + phi_i) + z_j,
 *              k_i = b_max - b_i, phi_i = 2^(k_i - 1)   KD3  (phi = 1/2 at k_i = 0)
 *   y_j = sum over i with b_i > 0 of x_i * w_hat_ij      (channels with b_i = 0 are
 *                                                         never read, KD1/KD2)
 *
 * Only the top b_i/2 two-bit planes of each loaded channel are read (KD2).
 *
 * Packed layout (KD2).  planes is uint32 [d_in][P][W_row], W_row =
 * ceil(d_out/64)*4 words: for input channel i, plane p (p = 0 holds bits
 * [b_max-2, b_max-1] of the code, the most significant), the d_out fragments
 * are contiguous, 16 per word; the fragment of output 16w+t sits at bits
 * [2t, 2t+1] of word w.  Rows are padded to a multiple of 64 outputs with
 * zero fragments, so every plane row is a multiple of 16 bytes.
 *
 * Conventions shared by every call:
 *  - Every pointer argument is a device pointer unless marked "host".  The
 *    caller allocates and owns all memory; the library allocates nothing and
 *    keeps no state beyond a cached device-property query.
 *  - Calls are asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream) and never synchronise the host.  They are thread-safe; calls
 *    that share a workspace must be ordered on one stream.
 *  - Arguments are checked on the host before anything touches the device;
 *    a failed check returns an error code and launches nothing.  Nothing
 *    throws across the ABI.  Values inside device buffers are not checked:
 *    NaN activations get 0 bits (the channel is skipped), +-Inf gets b_max
 *    bits and makes y non-finite, codes above 2^b_max - 1 are masked by
 *    grinqh_pack, unsorted thresholds are used through the count formula.
 */
#ifndef GRINQH_H
#define GRINQH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GRINQH_OK = 0,
    GRINQH_EINVAL = 1,    /* NULL pointer, bad size, bad b_max, bad dtype, bad layout */
    GRINQH_EALIGN = 2,    /* a pointer is not aligned as documented */
    GRINQH_ENOSPACE = 3,  /* workspace smaller than grinqh_gemv_workspace_bytes() */
    GRINQH_ENODEV = 4,    /* no HIP device is visible */
    GRINQH_EDEVICE = 5    /* the HIP runtime reported an error (query or launch) */
} grinqh_status;

typedef enum {
    GRINQH_BF16 = 0,      /* bfloat16, 2 bytes, 2-byte aligned */
    GRINQH_F32 = 1        /* IEEE binary32, 4 bytes, 4-byte aligned */
} grinqh_dtype;

/* Shape of one packed linear layer (plain data; fill with grinqh_layout_init). */
typedef struct {
    int32_t d_in;         /* input channels (reduction dimension), 1 .. 2^20 */
    int32_t d_out;        /* output channels, 1 .. 2^20 */
    int32_t b_max;        /* 2, 4, 6 or 8: full code width */
    int32_t n_planes;     /* b_max / 2 */
    int32_t row_words;    /* ceil(d_out / 64) * 4 uint32 words per plane row */
} grinqh_layout;

/* Library version as major*10000 + minor*100 + patch. */
int32_t grinqh_version(void);

/* Short constant English text for a status code (host pointer, never NULL). */
const char* grinqh_status_string(grinqh_status status);

/* Fill *out (host pointer) for a layer.  EINVAL if out is NULL, a size is
 * outside 1 .. 2^20 or b_max is not 2, 4, 6 or 8.  Pure host function. */
grinqh_status grinqh_layout_init(int32_t d_in, int32_t d_out, int32_t b_max,
                                 grinqh_layout* out);

/* Bytes of the packed planes: d_in * n_planes * row_words * 4 (KD2: storage
 * stays at b_max bits per weight).  0 if L is NULL or invalid.  Host only. */
size_t grinqh_packed_bytes(const grinqh_layout* L);

/* Bytes of device workspace grinqh_gemv needs for this layout on the current
 * device (0 if L is NULL or invalid, or no device is visible).  Host only. */
size_t grinqh_gemv_workspace_bytes(const grinqh_layout* L);

/* Offline bit-plane packing (KD2).
 *   q       uint8 [d_out][d_in], row-major (nn.Linear orientation: q[j][i]
 *           is the code of output j, input i); codes are masked to b_max bits.
 *   planes  uint32 [d_in][n_planes][row_words], 16-byte aligned,
 *           grinqh_packed_bytes(L) bytes; fully overwritten, padding included.
 * q and planes must not overlap. */
grinqh_status grinqh_pack(const grinqh_layout* L, const uint8_t* q, uint32_t* planes,
                          void* stream);

/* Runtime bit assignment (KD1), on its own (grinqh_gemv does the same work
 * inside its own kernel and does not need this call).
 *   x           [d_in] of x_dtype.
 *   theta       float [n_planes], theta_1 .. theta_P (ascending for the
 *               interval reading; any order is defined by the count formula).
 *   bits        uint8 [d_in] out: b_i in {0, 2, .., b_max}.
 *   active_idx  int32 [d_in] out or NULL: the n_active indices with b_i > 0,
 *               ascending, in entries 0 .. n_active-1; later entries unwritten.
 *   n_active    int32 [1] out or NULL. */
grinqh_status grinqh_assign_bits(const grinqh_layout* L, const void* x, grinqh_dtype x_dtype,
                                 const float* theta, uint8_t* bits, int32_t* active_idx,
                                 int32_t* n_active, void* stream);

/* The decode GEMV: bit assignment, prefix-plane streaming, midpoint dequant
 * and the product, all in the library's kernels (KD1, KD2, KD3).
 *   x          [d_in] of x_dtype (GRINQH_BF16 or GRINQH_F32).
 *   theta      float [n_planes].
 *   planes     as written by grinqh_pack, 16-byte aligned.
 *   s, z       fp16 bit patterns [d_out]: per-output-channel scale and zero point.
 *   y          [d_out] of y_dtype, overwritten (not accumulated); bf16 output
 *              is the fp32 result rounded to nearest even.
 *   workspace  >= grinqh_gemv_workspace_bytes(L) bytes, 256-byte aligned.  It
 *              must be zero-filled before its first use; every call leaves it
 *              ready for the next call (no clearing between calls).  Calls
 *              sharing one workspace must not overlap in time.
 * The packed planes of L must be smaller than 2 GiB (EINVAL otherwise).
 * x and y must not overlap.  Accumulation is fp32; the partial sums of the
 * input-channel slices are combined with fp32 atomic adds, so repeated calls
 * may differ in the last bits of y (b_i, the loaded planes and the codes are
 * always identical).  The workspace must be device memory (hipMalloc). */
grinqh_status grinqh_gemv(const grinqh_layout* L, const void* x, grinqh_dtype x_dtype,
                          const float* theta, const uint32_t* planes, const uint16_t* s,
                          const uint16_t* z, void* y, grinqh_dtype y_dtype, void* workspace,
                          size_t workspace_bytes, void* stream);

/* grinqh_gemv without a workspace argument, for callers that cannot allocate
 * device memory: code under stream capture, tight serving loops, harnesses
 * that forbid allocation.  Same arguments (minus the workspace), checks,
 * kernels and results as grinqh_gemv.  The workspace is a static device
 * array of GRINQH_NOALLOC_SCRATCH_BYTES inside the library: every GPU the
 * library runs on holds its own copy until the process ends, and the call
 * allocates nothing.  The first call on a device also queues a kernel that
 * clears that device's copy, ahead of the GEMV on the same stream; every
 * call leaves it cleared for the next one.
 *   Returns ENOSPACE when this layout needs more workspace than the array
 *   holds (grinqh_gemv_workspace_bytes(L) > GRINQH_NOALLOC_SCRATCH_BYTES;
 *   about 230 thousand outputs), ENODEV beyond 64 devices.
 * All calls on one GPU share its array: calls that can overlap in time on
 * one GPU (other streams, other host threads) race and give wrong results;
 * order them on one stream. */
#define GRINQH_NOALLOC_SCRATCH_BYTES (1u << 20)
grinqh_status grinqh_gemv_noalloc(const grinqh_layout* L, const void* x, grinqh_dtype x_dtype,
                                  const float* theta, const uint32_t* planes, const uint16_t* s,
                                  const uint16_t* z, void* y, grinqh_dtype y_dtype, void* stream);

/* Operands of one GEMV in a group call (all device pointers, same meaning and
 * alignment as the grinqh_gemv arguments of the same names). */
typedef struct {
    const void* x;
    const float* theta;
    const uint32_t* planes;
    const uint16_t* s;
    const uint16_t* z;
    void* y;
} grinqh_gemv_operands;

#define GRINQH_MAX_GROUP 8

/* Workspace bytes for grinqh_gemv_group over these layouts (host arrays of n
 * entries); 0 if an argument is invalid or no device is visible. */
size_t grinqh_gemv_group_workspace_bytes(const grinqh_layout* layouts, int32_t n);

/* n (1 .. GRINQH_MAX_GROUP) independent decode GEMVs in one kernel launch,
 * e.g. the q/k/v or gate/up projections of a decoder layer, or any set of
 * linears whose inputs are ready.  Each member computes exactly what
 * grinqh_gemv computes for its own x, theta, planes, s, z and y (KD1-KD3);
 * one launch lets the members' memory latencies overlap.
 *   layouts    host array [n]; every layout must have the same b_max.
 *   ops        host array [n] of operands.
 *   x_dtype, y_dtype  shared by all members.
 *   workspace  >= grinqh_gemv_group_workspace_bytes(layouts, n) bytes,
 *              256-byte aligned, zero-filled before first use, self-clearing.
 * The members' outputs must not overlap each other or any member's input. */
grinqh_status grinqh_gemv_group(const grinqh_layout* layouts, const grinqh_gemv_operands* ops,
                                int32_t n, grinqh_dtype x_dtype, grinqh_dtype y_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Test and diagnostic call: the truncated codes q_b * 2^(b_max - b_i)
 * (KD3's spliced truncated integer, at full scale) that the GEMV kernel's own
 * plane decoder produces for every loaded channel, 0 for skipped channels.
 *   bits    uint8 [d_in], as written by grinqh_assign_bits.
 *   codes   uint8 [d_in][d_out] out. */
grinqh_status grinqh_debug_codes(const grinqh_layout* L, const uint8_t* bits,
                                 const uint32_t* planes, uint8_t* codes, void* stream);

/* Test and tuning call: force the launch shape of later GEMV and prefill
 * calls in this process (0 = the library's own choice, the default).
 *   lane_groups   0, 1, 2, 4 or 8 lane groups per wave: GEMV output tiles of
 *                 2048, 1024, 512 or 256 outputs.
 *   chunk         0 or 1 .. 256 input channels per GEMV slice.
 *   prefill_tile  0, or 1 (128 x 128), 2 (256 x 128), 3 (256 x 256) tokens
 *                 x outputs per prefill tile.
 * The GEMV workspace size depends on the shape: query it again after a
 * change.  EINVAL for any other value (nothing changes).  Host only. */
grinqh_status grinqh_debug_force_launch(int32_t lane_groups, int32_t chunk, int32_t prefill_tile);

/* ---- Threshold calibration (offline) ----------------------------------
 *
 * KD1 fixes the thresholds offline from the magnitudes of about 128 sample
 * inputs of a layer.  This call computes them as quantiles of the pooled
 * magnitudes: with the count magnitudes |x| sorted ascending (NaN after
 * +Inf), for each level q, h = (count - 1) * q, lo = floor(h),
 * hi = min(lo + 1, count - 1), t = h - lo,
 *   theta = v[lo] + t * (v[hi] - v[lo])      (fp64; v[lo] itself at t = 0),
 * rounded once to fp32.  The result is exact: order statistics by radix
 * selection, no sampling.
 *   x          count values (bf16 or fp32), e.g. n samples x d_in, any order.
 *   count      1 .. 2^32 - 1.
 *   levels     host array [n_levels] of quantile levels in [0, 1]; n_levels
 *              1 .. 4 (one per threshold, ascending levels give ascending
 *              thresholds).
 *   theta      fp32 [n_levels] out.
 *   workspace  >= grinqh_calibrate_workspace_bytes() bytes, 256-byte aligned;
 *              any contents (the call initialises it). */
size_t grinqh_calibrate_workspace_bytes(void);
grinqh_status grinqh_calibrate_thresholds(const void* x, grinqh_dtype x_dtype, int64_t count,
                                          const double* levels, int32_t n_levels, float* theta,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* ---- Offline quantisation front end ("RTN") ----------------------------
 *
 * The note names round-to-nearest (RTN) as a base the method can sit on
 * without defining it.  This call quantises a bf16 weight matrix per output
 * channel onto the b_max-bit grid whose KD3 reconstruction at b = b_max,
 * s_j * (q + 1/2) + z_j, is the midpoint of each interval:
 *   lo_j, hi_j = min and max of row j (NaN ignored);
 *   s_j = fp16((hi_j - lo_j) / 2^b_max), z_j = fp16(lo_j) (zeros stored as +0);
 *   q = min(max(floor((w - z_j) / s_j), 0), 2^b_max - 1), in fp32 with the
 *       stored s_j and z_j (IEEE division; a NaN quotient gives 0, a row
 *       with s_j = 0 gets 0).
 * Every weight is then within s_j / 2 of its reconstruction, up to the fp16
 * rounding of s_j and z_j.  The outputs feed grinqh_pack and grinqh_gemv.
 *   w     bf16 [d_out][d_in]: row j holds output channel j's weights.
 *   q     uint8 [d_out][d_in] out.
 *   s, z  fp16 [d_out] out.
 * 1 <= d_in <= 2^30, 1 <= d_out <= 2^30, b_max in {2, 4, 6, 8}. */
grinqh_status grinqh_quantize_rtn(int32_t d_in, int32_t d_out, int32_t b_max, const uint16_t* w,
                                  uint8_t* q, uint16_t* s, uint16_t* z, void* stream);

/* ---- Prefill stage: dense b_max GEMM ----------------------------------
 *
 * The note's overview keeps the prefill stage dense: every weight at b_max
 * precision in ordinary matrix products, no thresholds.  For a block of M
 * prompt tokens this call computes, with every channel at b = b_max (KD3 at
 * k = 0, phi = 1/2),
 *   Y[m][j] = sum_i X[m][i] * (s_j * (q_ji + 1/2) + z_j)
 * from the same packed planes, s and z as grinqh_gemv.  The products of the
 * bf16 activations and the integer codes are exact; they are summed in fp32
 * on the bf16 matrix cores.
 *   L          layout of the planes (any b_max); d_in must be a multiple of 8.
 *   x          bf16 [M][d_in], row-major, 16-byte aligned (x_dtype must be
 *              GRINQH_BF16: the matrix cores take bf16 operands).
 *   M          1 .. 2^20 tokens.
 *   planes, s, z  as for grinqh_gemv.
 *   y          [M][d_out] of y_dtype, row-major, overwritten; bf16 output is
 *              the fp32 result rounded to nearest even.  A 16-byte aligned y
 *              with d_out a multiple of 8 (bf16) or 4 (fp32) is written in
 *              16-byte row segments, otherwise element by element (slower,
 *              same values).
 *   workspace  >= grinqh_prefill_workspace_bytes(M) bytes (the fp32 row sums
 *              of x), 256-byte aligned, any contents.
 * x and y must not overlap.  The planes must be smaller than 2 GiB. */
size_t grinqh_prefill_workspace_bytes(int32_t M);
grinqh_status grinqh_prefill_gemm(const grinqh_layout* L, const void* x, grinqh_dtype x_dtype, int32_t M,
                                  const uint32_t* planes, const uint16_t* s, const uint16_t* z, void* y,
                                  grinqh_dtype y_dtype, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* ---- Key-value cache ----------------------------------------------------
 *
 * The pages of keys and values that a decoder's attention reads, one cache
 * per layer.  A row is the head_dim values of one token and one key-value
 * head.  At 4 and 8 bits a row is quantised as it is written, onto the grid
 * that grinqh_quantize_rtn uses for a row of weights (KD3 at b = b_max):
 *   lo, hi = min and max of the row (NaN ignored);
 *   s = fp16((hi - lo) / 2^bits), z = fp16(lo) (zeros stored as +0);
 *   c = min(max(floor((w - z) / s), 0), 2^bits - 1) in fp32 with the stored
 *       s and z (a NaN quotient gives 0; a row with s = 0 gets 0),
 * and stands for s * (c + 1/2) + z.  At 16 bits a row is kept as bf16 (fp32
 * input rounded to nearest even).  Values outside fp16's range overflow s
 * and z to Inf, and the row then reads as Inf or NaN.
 *
 * A pool holds n_pages pages of page_size tokens:
 *   codes  uint8 [n_pages][n_kv_heads][page_size][row_bytes], 16-byte
 *          aligned; at 4 bits byte i of a row holds values 2i (low half)
 *          and 2i + 1, at 16 bits the row is head_dim bf16.
 *   grid   fp16 [n_pages][n_kv_heads][page_size][2]: s, z of every row,
 *          16-byte aligned; NULL at 16 bits.
 * Slot page * page_size + t names token t of a page, in every head. */
typedef struct {
    int32_t n_kv_heads;   /* 1 .. 1024 */
    int32_t head_dim;     /* 64, 128 or 256 */
    int32_t page_size;    /* 16, 32, 64, 128 or 256 tokens */
    int32_t n_pages;      /* 1 .. 2^24 */
    int32_t bits;         /* 4, 8 or 16 */
    int32_t row_bytes;    /* head_dim * bits / 8 */
} grinqh_kv_layout;

/* Device pointers of one cache: a pool of keys and one of values. */
typedef struct {
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint16_t* k_grid;
    uint16_t* v_grid;
} grinqh_kv_pools;

/* Fill *out (host pointer); EINVAL for a value outside the ranges above. */
grinqh_status grinqh_kv_layout_init(int32_t n_kv_heads, int32_t head_dim, int32_t page_size, int32_t n_pages,
                                    int32_t bits, grinqh_kv_layout* out);

/* Bytes of one pool's codes and of its grid (0 at 16 bits); 0 if L is NULL or
 * invalid.  Host only. */
size_t grinqh_kv_code_bytes(const grinqh_kv_layout* L);
size_t grinqh_kv_grid_bytes(const grinqh_kv_layout* L);

/* Write the keys and values of n_tokens tokens into their slots.
 *   k, v       [n_tokens][n_kv_heads][head_dim] of dtype, 16-byte aligned; the
 *              tokens lie k_stride and v_stride elements apart (multiples of
 *              16 bytes, from n_kv_heads * head_dim to 2^24 elements), so both can be
 *              slices of a fused projection's output.
 *   n_tokens   0 .. 2^24 (0: nothing is launched).
 *   slots      int64 [n_tokens]; a token whose slot is negative or not below
 *              n_pages * page_size is not written (padding).  The slots
 *              written by one call must differ: a slot named twice is left
 *              holding a mixture of the rows.
 * k, v and slots must not overlap the pools, nor the pools one another (EINVAL; a
 * cache whose keys and values share a pool can only be read). */
grinqh_status grinqh_kv_write(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const void* k,
                              const void* v, grinqh_dtype dtype, int64_t k_stride, int64_t v_stride,
                              int32_t n_tokens, const int64_t* slots, void* stream);

/* Read the values of n_tokens slots back, in any order and any number of
 * times each.
 *   k, v   [n_tokens][n_kv_heads][head_dim] of dtype out, contiguous, 16-byte
 *          aligned: s * (c + 1/2) + z in fp32 (one rounding), bf16 output
 *          rounded to nearest even; zeros for a slot outside the pool.  They
 *          must not overlap each other, the slots or the pools. */
grinqh_status grinqh_kv_read(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const int64_t* slots,
                             int32_t n_tokens, void* k, void* v, grinqh_dtype dtype, void* stream);

/* Test call, host only: the row index (of row_bytes codes, and of one s, z
 * pair) that the kernels use for a slot and head; -1 for a slot outside the
 * pool, a head outside 0 .. n_kv_heads - 1 or an invalid layout. */
int64_t grinqh_debug_kv_row(const grinqh_kv_layout* L, int64_t slot, int32_t head);

/* Test call, host only: the row index that the decode attention reads for
 * token t of a sequence and head from a page table's entry; for an entry that
 * names no page of the pool, -1 minus the row that is read in its stead and not
 * used.  -1 for a negative t, a head outside the layout or an invalid layout. */
int64_t grinqh_debug_page_row(const grinqh_kv_layout* L, int32_t page, int32_t head, int32_t t);

/* ---- Attention -----------------------------------------------------------
 *
 * For every query head h of a query token, with key-value head
 * g = h / (n_q_heads / n_kv_heads),
 *   o_h = sum_t p_t v_gt,  p_t = exp(a_t) / sum_u exp(a_u),  a_t = scale * q_h . k_gt,
 * over the tokens t that the query sees.  A query that sees none gets zeros.
 * lse_h = log(sum_t exp(a_t)) (-Inf where no token is seen).  Scores, softmax
 * statistics and sums are fp32; fp32 queries enter the scores as the sum of two
 * bf16 (2^-16 relative; a value past bf16's range counts as infinite).
 * Infinities and NaN in tokens that are seen go through the formula (where an
 * infinite value makes it infinite, an output may be NaN; a query whose seen
 * scores are all -Inf gets zeros); in tokens that are not seen they have no
 * effect.  Where q . k is finite but a score passes fp32's range, lse is
 * infinite; the prefill stage still gives the formula's output, in the decode
 * stage a score past 2.3e38 counts as infinite.
 *
 * Decode stage: one new token of every sequence attends to its cached
 * tokens (the new one among them, if it was written first).
 *   q           [batch][n_q_heads][head_dim] of q_dtype, 16-byte aligned; the
 *               sequences' tokens lie q_stride elements apart (a multiple of
 *               16 bytes, from n_q_heads * head_dim to 2^24 elements).
 *   n_q_heads   a multiple of L->n_kv_heads, up to 1024.
 *   page_table  int32 [batch][max_pages], rows table_stride entries apart: the
 *               pages of a sequence in order.  A page outside 0 .. n_pages - 1
 *               is absent: its tokens are not seen.
 *   seq_lens    int32 [batch]: cached tokens of each sequence, taken as 0 if
 *               negative and as min(max_len, max_pages * page_size) if above.
 *   batch       0 .. 2^20 (0: nothing is launched), and batch * n_kv_heads *
 *               ceil(n_q_heads / n_kv_heads / 16) at most 2^23; max_len 1 ..
 *               2^28, the host's bound on the lengths: a long cache is cut into
 *               parts by it, so one near the longest length is faster.
 *   scale       -1e30 .. 1e30.
 *   out         [batch][n_q_heads][head_dim] of out_dtype, contiguous, 16-byte
 *               aligned.
 *   lse         fp32 [batch][n_q_heads] or NULL.
 *   workspace   >= grinqh_attention_workspace_bytes(...) bytes, 256-byte
 *               aligned, its first 16384 bytes zero-filled before its first use by
 *               this call; every call leaves it ready for the next, of any layout
 *               and sizes that it is large enough for.  The size never falls as
 *               batch or max_len grow: a workspace for a program's largest call
 *               serves all of its calls with that layout and n_q_heads.
 *               Calls that share it must not overlap in time, and
 *               grinqh_gemv must have its own.
 * The result of a call does not depend on timing: the parts of a long
 * cache are joined in their order.  out, lse and the workspace (as much of it
 * as the call uses) must not overlap one another nor anything that is read. */
size_t grinqh_attention_workspace_bytes(const grinqh_kv_layout* L, int32_t n_q_heads, int32_t batch,
                                        int32_t max_len);
grinqh_status grinqh_decode_attention(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const void* q,
                                      grinqh_dtype q_dtype, int64_t q_stride, int32_t n_q_heads,
                                      const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                      const int32_t* seq_lens, int32_t batch, int32_t max_len, float scale,
                                      void* out, grinqh_dtype out_dtype, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Prefill stage: whole prompts, packed behind one another without padding.
 * Sequence b has the query rows cu_q[b] .. cu_q[b+1] - 1 and the key rows
 * cu_k[b] .. cu_k[b+1] - 1.  With causal nonzero the last query sees every key
 * and each earlier one a key less: query i of n sees the keys 0 .. i + m - n of
 * m (so with more keys than queries the first keys are the cached
 * beginning, and with fewer the first queries see nothing).
 *   q          bf16 [total_q][n_q_heads][head_dim], token rows q_stride elements
 *              apart; k, v bf16 [total_k][n_kv_heads][head_dim], k_stride and
 *              v_stride apart (multiples of 8, up to 2^24; rows may be slices of
 *              a fused projection's output); all 16-byte aligned.
 *   cu_q, cu_k int32 [batch + 1], ascending from 0; entries are clamped to
 *              0 .. total_q (total_k).
 *   total_q, total_k  0 .. 2^24 rows (total_q 0: nothing is launched).
 *   n_q_heads  a multiple of n_kv_heads, up to 1024; head_dim 64, 128 or 256.
 *   scale      -1e30 .. 1e30.
 *   out        [total_q][n_q_heads][head_dim] of out_dtype, contiguous, 16-byte
 *              aligned; rows behind the last sequence are left as they are.
 *   lse        fp32 [total_q][n_q_heads] or NULL.
 *   workspace  NULL, or >= grinqh_prefill_attention_workspace_bytes(args) bytes,
 *              256-byte aligned, any contents: with it the keys of few queries
 *              are worked on in parts and joined by a second kernel.  The size
 *              follows from the sizes in args and causal alone (0: it would not
 *              be used, or a size is invalid).
 * out, lse and a workspace that is used must not overlap one another nor
 * anything that is read.
 * total_q * n_q_heads / 128 + min(batch, total_q) * n_kv_heads is at most 2^23.
 * The weights p_t are rounded to bf16 for the product with the values. */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t batch, total_q, total_k;
    int32_t n_q_heads, n_kv_heads, head_dim;
    int32_t causal;
    float scale;
    void* out;
    grinqh_dtype out_dtype;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
} grinqh_prefill_attention_args;
size_t grinqh_prefill_attention_workspace_bytes(const grinqh_prefill_attention_args* args);
grinqh_status grinqh_prefill_attention(const grinqh_prefill_attention_args* args, void* stream);

/* ---- 4-bit weights with group scales -------------------------------------
 *
 * Matrices whose every `group` neighbouring input channels of an output
 * channel share a scale and a zero point, on the grid of grinqh_quantize_rtn at
 * b_max 4 (KD3 at b = b_max), for products that take every channel:
 *   w_ij = s_jg * (q_ji + 1/2) + z_jg,   g = i / group,
 *   y[t][j] = sum_i x[t][i] * w_ij.
 * n_experts matrices of one shape lie behind one another; a plain layer has one.
 * Codes are stored in the order in which the matrix cores take them: tiles of
 * 16 outputs x 128 inputs, uint32 [n_experts][row_tiles][k_tiles][64][4]; in a
 * tile word m of lane 16 * c + r holds the codes of output r and inputs
 * 32 * m + 8 * c + e, e = 0 .. 7, each in the four bits from bit
 * 3 + 4 * (e / 2) + 16 * (e % 2) on (modulo 32).  The grid is fp16
 * [n_experts][row_tiles][k_tiles * 128 / group][16][2]: s, z.  Outputs and inputs
 * past the ends are zeros. */
typedef struct {
    int32_t d_in;         /* input channels, a multiple of group, up to 2^20 */
    int32_t d_out;        /* output channels, 1 .. 2^20 */
    int32_t group;        /* 32, 64 or 128 */
    int32_t n_experts;    /* 1 .. 1024 */
    int32_t k_tiles;      /* ceil(d_in / 128) */
    int32_t row_tiles;    /* ceil(d_out / 16) */
} grinqh_fourbit_layout;

/* Fill *out (host pointer); EINVAL for a value outside the ranges above, or
 * for more than 2^40 bytes of codes. */
grinqh_status grinqh_fourbit_layout_init(int32_t d_in, int32_t d_out, int32_t group, int32_t n_experts,
                                         grinqh_fourbit_layout* out);

/* Bytes of the packed codes and of the packed grid; 0 if L is NULL or invalid.
 * Host only. */
size_t grinqh_fourbit_code_bytes(const grinqh_fourbit_layout* L);
size_t grinqh_fourbit_grid_bytes(const grinqh_fourbit_layout* L);

/* Offline packing.
 *   q      uint8 [n_experts][d_out][d_in], codes masked to 4 bits; 8-byte aligned.
 *   s, z   fp16 [n_experts][d_out][d_in / group].
 *   codes, grid   out, 16-byte aligned, fully overwritten, padding included.
 * With grinqh_quantize_rtn(group, n_experts * d_out * d_in / group, 4, ...) on
 * the bf16 weights as they lie (in several calls where that is more than 2^30),
 * its q, s and z are this call's.  The outputs must not overlap each other or
 * the inputs. */
grinqh_status grinqh_fourbit_pack(const grinqh_fourbit_layout* L, const uint8_t* q, const uint16_t* s,
                                  const uint16_t* z, uint8_t* codes, uint16_t* grid, void* stream);

/* y = x times the matrix, for n_tokens tokens (one and a few stream the weights
 * once; many go through larger tiles).
 *   L          of one expert.
 *   x          [n_tokens][d_in] of x_dtype, 16-byte aligned, tokens x_stride
 *              elements apart (a multiple of 16 bytes, from d_in to 2^24).
 *   n_tokens   0 .. 2^20 (0: nothing is launched).
 *   codes, grid   as written by grinqh_fourbit_pack, 16-byte aligned.
 *   y          [n_tokens][d_out] of y_dtype, contiguous, overwritten; bf16 output is
 *              the fp32 result rounded to nearest even.
 * Codes enter the products exactly and activations as they are (fp32 ones as
 * the sum of three bf16; many tokens of fp32 are worked on sixteen at a time, so
 * a long prompt is better in bf16); sums are fp32, and the same call gives the
 * same bits.  An infinite or NaN activation makes its token's outputs
 * non-finite and no other's, and so may one past 2^115, or a sum of
 * |x| (s (16 + q) + |z - 15.5 s|) past fp32's range, where y itself would not
 * reach it.  y must not overlap anything that is read. */
grinqh_status grinqh_fourbit_linear(const grinqh_fourbit_layout* L, const void* x, grinqh_dtype x_dtype,
                                    int64_t x_stride, int32_t n_tokens, const uint8_t* codes,
                                    const uint16_t* grid, void* y, grinqh_dtype y_dtype, void* stream);

/* The same for rows grouped by expert: row r of y, for ends[e] <= r < ends[e + 1],
 * is a row of x times expert e's matrix.
 *   x       [n_x][d_in] as above; n_x 1 .. 2^20.
 *   rows    int32 [n_rows]: row r of y takes row rows[r] of x, any row any number
 *           of times; a row outside 0 .. n_x - 1 counts as zeros.  NULL: row r
 *           takes row r (rows from n_x on count as zeros).
 *   ends    int32 [n_experts + 1], ascending; entries are clamped to 0 .. n_rows.
 *           An expert may have no rows; rows before the first end and behind the
 *           last are left as they are.
 *   n_rows  0 .. 2^20 (0: nothing is launched).
 *   y       [n_rows][d_out], as above. */
typedef struct {
    const void* x;
    int64_t x_stride;
    grinqh_dtype x_dtype;
    int32_t n_x;
    const int32_t* rows;
    const int32_t* ends;
    int32_t n_rows;
    const uint8_t* codes;
    const uint16_t* grid;
    void* y;
    grinqh_dtype y_dtype;
} grinqh_expert_args;
grinqh_status grinqh_expert_linear(const grinqh_fourbit_layout* L, const grinqh_expert_args* args, void* stream);

/* ---- Norms of queries and keys, rotation by position ----------------------
 *
 * For every head row x of a token's queries and keys, in one pass:
 *   x_i <- x_i * weight_i / sqrt(mean(x^2) + eps)       (where there is a weight)
 *   (a, b) <- (a cos t - b sin t, b cos t + a sin t),   t = position * freqs[p],
 * for the p-th of rope_dim / 2 pairs of the first rope_dim channels: (p, p +
 * rope_dim / 2), or with neighbours nonzero (2p, 2p + 1).  The other channels
 * are only normed.  Sums are fp32 (a normed row whose squares pass fp32's range
 * comes out as zeros, one of zeros with eps 0 as NaN), angles fp64 up to the
 * last turn; the result is rounded once to dtype.  With a cache, the keys as rounded and the values as
 * they are go into their slots as grinqh_kv_write would put them.
 *   q, k       [n_tokens][heads][head_dim] of dtype, 16-byte aligned, tokens
 *              q_stride and k_stride elements apart (multiples of 16 bytes, from
 *              heads * head_dim to 2^24).  n_q_heads, n_kv_heads 1 .. 1024;
 *              head_dim 64, 128 or 256.
 *   n_tokens   0 .. 2^24 (0: nothing is launched).
 *   q_weight, k_weight   [head_dim] of weight_dtype, 16-byte aligned, or NULL: no norm.
 *   eps        0 or more, finite (not used without weights).
 *   positions  int32 [n_tokens], any sign.
 *   freqs      fp64 [rope_dim / 2], radians per position; NULL only at rope_dim 0.
 *   rope_dim   0 .. head_dim, a multiple of 16.
 *   q_out, k_out   as q and k, with strides of their own; either may be its input
 *              itself (same pointer and stride).  k_out NULL: not wanted (with a
 *              cache only).
 *   cache      NULL, or the layout of a cache with these n_kv_heads and head_dim;
 *              then pools, v (as k, v_stride) and slots (int64 [n_tokens]; a token
 *              whose slot is outside the pool is not written, the slots of one
 *              call must differ) are needed.
 * Outputs must not overlap one another nor, but for the case above, anything
 * that is read; the pools neither. */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;
    int32_t n_tokens, n_q_heads, n_kv_heads, head_dim;
    grinqh_dtype dtype;
    const void* q_weight;
    const void* k_weight;
    grinqh_dtype weight_dtype;
    float eps;
    const int32_t* positions;
    const double* freqs;
    int32_t rope_dim, neighbours;
    void* q_out;
    void* k_out;
    int64_t q_out_stride, k_out_stride;
    const grinqh_kv_layout* cache;
    const grinqh_kv_pools* pools;
    const int64_t* slots;
} grinqh_rope_args;
grinqh_status grinqh_qk_rope(const grinqh_rope_args* args, void* stream);

/* ---- Pages of a batch -----------------------------------------------------
 *
 * The cache's pages are handed out on the GPU from the requests' lengths, so
 * that a step can be captured and needs no copy to the host.  A pool's unused
 * pages are a list: free_pages int32 [n_pages], of which the first n_free[0]
 * count (clamped to 0 .. n_pages) and the last of these is handed out first.
 * The two calls on a pool must be ordered on one stream.
 *
 * grinqh_kv_extend makes room for n_new[b] new tokens behind the seq_lens[b]
 * cached ones of every sequence b (negative counts as 0) and writes what
 * the other calls of the step take.  A sequence that no step could serve, because
 * it would pass max_pages or needs more than n_pages new ones, is refused and its
 * pages count for nobody.  The others are served in order: one whose pages, with
 * those of the sequences before it (served or not), are more than the list holds
 * is refused, and so is one whose tokens do not fit into capacity.  A refused
 * sequence keeps its length and pages, and its new tokens have no slots.  A
 * sequence without new tokens is never refused.
 *   page_table  int32 [batch][max_pages], rows table_stride entries apart: entries
 *               of new pages are written, the others left.
 *   new_lens    int32 [batch] out: lengths with the new tokens (may be seq_lens).
 *   n_free_out  int32 [1] out (may be n_free).
 *   refused     int32 [1] out: how many sequences were refused.
 *   cu_q, cu_k  int32 [batch + 1] out: ends of the packed new tokens (as n_new
 *               says, refused or not; clamped to 2^31 - 1), and of all tokens (of new_lens).
 *   slots       int64 [capacity] out: slot of each new token, packed; -1 for a
 *               refused sequence's, for a token whose page is not of the pool, and
 *               behind the last token.
 *   positions   int32 [capacity] out: place in its sequence; 0 behind the last token.
 *   capacity    0 .. 2^24; batch 0 .. 2^20 (0: the outputs are as for none);
 *               max_pages 1 .. 2^24; page_size as in a layout; n_pages 1 .. 2^24.
 *   workspace   >= grinqh_kv_extend_workspace_bytes(batch) bytes, 16-byte aligned,
 *               any contents.
 * All pointers are aligned to their type.  Nothing that is written may overlap
 * anything else, but for the two cases above. */
typedef struct {
    int32_t* page_table;
    int64_t table_stride;
    const int32_t* seq_lens;
    const int32_t* n_new;
    const int32_t* free_pages;
    const int32_t* n_free;
    int32_t batch, max_pages, page_size, n_pages, capacity;
    int32_t* new_lens;
    int32_t* n_free_out;
    int32_t* refused;
    int32_t* cu_q;
    int32_t* cu_k;
    int64_t* slots;
    int32_t* positions;
    void* workspace;
    size_t workspace_bytes;
} grinqh_extend_args;
size_t grinqh_kv_extend_workspace_bytes(int32_t batch);
grinqh_status grinqh_kv_extend(const grinqh_extend_args* args, void* stream);

/* Give the pages of finished sequences back: for every b with finished[b]
 * nonzero (uint8 [batch]), the pages that seq_lens[b] tokens take are put behind
 * the list in their order (entries that name no page of the pool are passed
 * over, and what would pass n_pages is dropped), the entries become -1 and the
 * length 0.  Nothing counts how often a page is named: one that two sequences share
 * would be listed twice, so all but the last give it back as -1. */
grinqh_status grinqh_kv_release(int32_t* page_table, int64_t table_stride, int32_t* seq_lens,
                                const uint8_t* finished, int32_t batch, int32_t max_pages, int32_t page_size,
                                int32_t* free_pages, int32_t* n_free, int32_t n_pages, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GRINQH_H */
