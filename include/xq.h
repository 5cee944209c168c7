/*
 * xq.h — C ABI of libxq, the quantized decode mat-vec for AMD MI355X (gfx950).
 *
 * Every entry point validates its arguments on the host, enqueues its kernel
 * on the caller's HIP stream and returns without synchronising ("25 — Writing
 * XPU Kernels", section 25.5: chain launches on one stream and wait once on
 * the read side). Faults during execution surface at the caller's next
 * synchronisation.
 *
 * Conventions shared by every entry point:
 *  - Pointers named as device buffers are device memory owned by the caller
 *    ("cajeta.xpu — one kernel, any device", section 2.2: buffers are the
 *    caller's allocations). The library allocates no memory and keeps no
 *    per-call state; it never synchronizes a stream or the device.
 *  - Eight entry points need device scratch beyond their inputs and outputs
 *    (xq_gemm_q4k_small_m's split-K partials and arrival counters,
 *    xq_gemv_q4k_q8k's arrival counters, xq_gemm_q4k_id's expert map,
 *    xq_attn_decode's split partials and arrival counters, the lists of
 *    xq_cache_fork and xq_cache_compact, the logits of xq_moe_route, the hidden
 *    values of xq_moe_q4k). The
 *    caller passes it as `workspace` (device memory, 256-byte aligned) and
 *    `workspace_bytes`; the matching *_workspace_bytes query gives the exact
 *    bytes a call needs (0: none, and then workspace may be NULL). The caller
 *    zeroes a workspace once before its first use; every call that completes
 *    leaves it ready for the next (its arrival counters, which lie in its
 *    first 96 KiB, back at zero), so one workspace serves any sequence of
 *    calls on one stream whose needs it covers; xq_gemm_q4k_id alone needs
 *    one of its own, since its map begins at the first byte. Calls that may
 *    run at the same time (different streams) need
 *    different workspaces. A NULL workspace where one is needed is refused
 *    with XQ_E_NULL, a short one with XQ_E_SHAPE, a misaligned one with
 *    XQ_E_ALIGN.
 *  - `stream` is a hipStream_t passed as void*; NULL means the null stream.
 *  - Outputs are fully overwritten, never accumulated into. Outputs must not
 *    alias inputs (documented, not checked).
 *  - A refused call returns a status other than XQ_OK, launches nothing and
 *    sets the thread-local text returned by xq_last_error() naming the gate
 *    that refused (section 25.6: a refusal answers with the gate that
 *    refused). There is no fallback kernel.
 *  - The gates run before any HIP call in this order: null pointers, shape,
 *    alignment, then the device (it must be gfx950).
 *  - A launch counts its threads in 32 bits. Sizes within an entry point's
 *    bounds that would give a kernel 2^32 and more (a mat-vec of 2^26 rows of
 *    at most 16 blocks, say) are refused with XQ_E_LAUNCH.
 *
 * Byte layouts (all little-endian):
 *  q8_K block, 320 B per 256 activations (section 25.2, the integer-route
 *    bullet, and section 25.2.1): int8 codes at +0, eight int32 sums of 32
 *    consecutive codes at +256, the f32 scale at +288; bytes 292..319 are
 *    written as zero and carry no meaning. A q8_K tensor of R rows and K
 *    columns is [R][K/256] blocks, row-major.
 *  Q4_K super-block, 144 B per 256 weights ("cajeta.xpu — one kernel, any
 *    device", section 2.3, the alignment example: nibble group g at
 *    16 + 32*g): f16 d at +0, f16 dmin at +2, twelve bytes of packed 6-bit
 *    scales and mins at +4, 128 B of nibbles at +16. Group g's 32 bytes hold
 *    sub-block 2g in their low nibbles and sub-block 2g+1 in their high
 *    nibbles. Weight = d*sc_j*q - dmin*m_j. A matrix of N rows and K columns
 *    is [N][K/256] blocks, row-major.
 *  IQ4_NL resident row (section 25.2.1): the row's K/32 f16 block scales,
 *    padded to a multiple of 4 bytes, then K/32 payloads of 16 B; payload
 *    byte t gives weight t (low nibble) and weight t+16 (high nibble); a
 *    nibble selects an int8 from the 16-entry IQ4_NL codebook; weight =
 *    d_c * kv[nibble]. A matrix is N such rows back to back.
 */
#ifndef XQ_H
#define XQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t xq_status;

enum {
    XQ_OK = 0,
    XQ_E_NULL = 1,   /* a required pointer is NULL */
    XQ_E_SHAPE = 2,  /* a size is out of range or not a multiple it must be */
    XQ_E_ALIGN = 3,  /* a buffer base is short of the alignment its loads need */
    XQ_E_DEVICE = 4, /* no HIP device, or the current device is not gfx950 */
    XQ_E_LAUNCH = 5  /* the runtime refused the kernel launch */
};

/*
 * Quantize f32 activations to q8_K ("25 — Writing XPU Kernels", section 25.2,
 * the integer-route bullet: the activation is quantized once to q8_K).
 * Per 256-block: amax = max|x_i|; d = amax/127 as one IEEE f32 division;
 * code_i = x_i/d (IEEE f32 division) rounded to nearest, ties to even (0 when
 * d == 0); sum_j = sum of codes 32j..32j+31.
 *
 *  xq    device, out: rows*(K/256) q8_K blocks, 16-byte aligned.
 *  x     device, in: f32 [rows][K] row-major, 4-byte aligned (a 16-byte
 *        aligned x is read with 16-byte loads, any other with 4-byte loads;
 *        the bytes written are the same).
 *  rows  >= 1.  K >= 256, a multiple of 256.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_quantize_q8k(void *xq, const float *x, int64_t rows, int64_t K, void *stream);

/*
 * Q4_K x q8_K decode mat-vec, batch 1 ("25 — Writing XPU Kernels", section
 * 25.2, and section 25.5 for the Q4_K mat-vec's 16-byte loads):
 *   y[r] = sum_b xs_b * (d_rb * S_rb - dmin_rb * M_rb),
 *   S_rb = sum_j sc_j * sum_{t<32} q * code   (exact int32),
 *   M_rb = sum_j m_j * s_j                    (exact int32; s_j the q8_K's stored
 *                                              sum of sub-block j's 32 codes),
 * which is the dot of the dequantized row with the dequantized activation.
 *
 *  y   device, out: f32 [N], 4-byte aligned.
 *  w   device, in: Q4_K [N][K/256], 16-byte aligned.
 *  xq  device, in: one q8_K row of K/256 blocks, 16-byte aligned.
 *  1 <= N <= 2^30.  K >= 256, a multiple of 256, K <= XQ_MAX_K.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_gemv_q4k(float *y, const void *w, const void *xq, int64_t N, int64_t K, void *stream);

/*
 * Q4_K x q8_K mat-vec with its output quantized in the same launch ("25 —
 * Writing XPU Kernels", section 25.5: the FFN pair's fused tail; the up
 * product hands the down product its q8_K activation):
 *   y  = the result of xq_gemv_q4k(y, w, xq, N, K), bit for bit;
 *   yq = the bytes xq_quantize_q8k(yq, y, 1, N) writes, bytes 0..291 of every
 *        block bit for bit (292..319 zero).
 * The 256/(rows per workgroup) workgroups of each q8_K block of y count
 * their arrival on a counter; the last quantizes the block.
 *
 *  y   device, out: f32 [N], 4-byte aligned.
 *  yq  device, out: q8_K [N/256] blocks (xq_q8k_bytes(1, N)), 16-byte aligned.
 *  w, xq, K as xq_gemv_q4k.
 *  N a multiple of 256, 256 <= N <= 2^22.
 *  workspace  the block counters: xq_gemv_q4k_q8k_workspace_bytes(N) bytes
 *      (one 128-byte line per q8_K block of y, at most 768 lines, which more
 *      blocks share), zeroed before first use; the last arrival at a counter
 *      resets it.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_gemv_q4k_q8k(float *y, void *yq, const void *w, const void *xq, int64_t N, int64_t K,
                          void *workspace, size_t workspace_bytes, void *stream);
size_t xq_gemv_q4k_q8k_workspace_bytes(int64_t N);  /* min(N/256, 768) * 128; 0 if N is invalid */

/*
 * IQ4_NL x q8_K decode mat-vec, batch 1 ("25 — Writing XPU Kernels", section
 * 25.2.1): y[r] = sum_c d_rc * xs_(c/8) * D_rc with D_rc = sum_{t<32}
 * kv[nibble_t] * code_(32c+t) (exact int32).
 *
 *  y   device, out: f32 [N], 4-byte aligned.
 *  w   device, in: N resident IQ4_NL rows (xq_iq4nl_bytes(N, K) bytes),
 *      16-byte aligned.
 *  xq  device, in: one q8_K row of K/256 blocks, 16-byte aligned.
 *  1 <= N <= 2^30.  K >= 256, a multiple of 256 (each 32-block must fall inside a
 *  q8_K block), K <= XQ_MAX_K.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_gemv_iq4nl(float *y, const void *w, const void *xq, int64_t N, int64_t K,
                        void *stream);

/*
 * Q4_K x q8_K small-M product (multi-token prefill; "25 — Writing XPU
 * Kernels", section 25.3): Y[m][n] = sum_b xs_mb * (d_nb * S_mnb - dmin_nb *
 * M_mnb), with S and M the exact int32 block partials of xq_gemv_q4k taken
 * against token m's q8_K row.
 *
 *  y   device, out: f32 [M][N] row-major (token-major), 4-byte aligned.
 *  w   device, in: Q4_K [N][K/256], 16-byte aligned.
 *  xq  device, in: q8_K [M][K/256], 16-byte aligned.
 *  1 <= M <= 2^30.  1 <= N <= 2^30.  K >= 256, a multiple of 256. Each of
 *  xq and w below 2 GiB (the kernel's loads use 32-bit offsets).
 * A very short batch (M = 1; M <= 3; M = 4 when K <= 4096 or N*K <= 2^25,
 * M <= 6 when N*K <= 2^24, M <= 8 when N*K <= 2^23 or when K <= 4096 and
 * N*K <= 2^24, in each while the M q8_K rows fit 64 KB) is a weight stream
 * rather than a dense contraction: it runs on the mat-vec kernels, one pass
 * over the weights for all M tokens, and row m is then bit-identical to
 * xq_gemv_q4k on token m. Larger M runs on int8 MFMA: 5 to 16 tokens on
 * matrices of 8161 to 16384 rows and 8 to 16 super-blocks per row in
 * tiles of 32 rows whose four waves split K and sum their partial tiles in
 * a fixed order (no workspace); otherwise in tiles of 16 tokens up to M = 32
 * (64 when N*K <= 2^25 or N <= 4096, 96 when N*K <= 2^25, 128 when
 * N*K <= 2^24) and of 64 tokens beyond.
 * Shapes with at most 256 tiles of 16 or 64 tokens x 128 rows split K over
 * several workgroups (section 25.3: fill the device first); shapes with more
 * tiles than one round of resident workgroups run whole rounds of whole
 * tiles and may split the last, short round's tiles the same way. Splits
 * are summed in a fixed order, so results are bit-identical from call to
 * call and do not depend on the workspace's address.
 *  workspace  96 KiB of arrival counters (one 128-byte line per split tile,
 *      at the same place for every shape), then the split partials:
 *      xq_gemm_q4k_small_m_workspace_bytes(M, N, K) bytes, 0 when the shape
 *      splits no tile (at most 16 MiB + 96 KiB for any shape), zeroed
 *      before first use.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_gemm_q4k_small_m(float *y, const void *w, const void *xq, int64_t M, int64_t N,
                              int64_t K, void *workspace, size_t workspace_bytes, void *stream);
size_t xq_gemm_q4k_small_m_workspace_bytes(int64_t M, int64_t N, int64_t K);  /* 0 if none, or
                                                                              if the shape is refused */

/*
 * xq_gemm_q4k_small_m without a workspace and without any allocation, for
 * callers that cannot allocate device memory or pass a workspace: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results (bit for bit), gates and errors as
 * xq_gemm_q4k_small_m, except the workspace: the split-K partials and
 * arrival counters live in the library's own device array of
 * XQ_NOALLOC_SCRATCH_BYTES, one per GPU, held until the process ends. A shape
 * whose plan needs more scratch than that (xq_gemm_q4k_small_m_workspace_bytes
 * above it: some 64-token-tile shapes with split K) is refused with
 * XQ_E_SHAPE; every shape of up to 32 tokens fits. The first call on a GPU
 * looks the array up and clears its counters on the caller's stream; every
 * completed call leaves them at zero. All calls on one GPU share the array:
 * calls that overlap in time on one GPU (other streams, other threads) race
 * and must not be issued.
 */
#define XQ_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
xq_status xq_gemm_q4k_small_m_noalloc(float *y, const void *w, const void *xq, int64_t M,
                                      int64_t N, int64_t K, void *stream);

/*
 * Grouped Q4_K x q8_K small-M product over an expert slab (mul_mat_id; "25 —
 * Writing XPU Kernels", section 25.3: a mixture-of-experts prefill is one
 * launch over an expert map, padded only to the finest tile, never one
 * product per expert). Token t's slot k uses expert e = ids[t][k]:
 *   y[t][k][n] = sum_b xs_b * (d_enb * S_b - dmin_enb * M_b)
 * with S, M the exact int32 block partials of expert e's row n against the
 * pair's q8_K row, which is row t of xq (x_per_slot = 0: the slots of a
 * token share its activation, as for up and gate) or row t * n_used + k
 * (x_per_slot = 1: each slot has its own, as for down).
 *
 *  y     device, out: f32 [n_tokens][n_used][rows], 4-byte aligned. The rows
 *        of a pair whose selection lies outside 0..n_experts-1 are NaN.
 *  slab  device, in: n_experts experts of rows x K Q4_K weights back to back
 *        (expert e's row n is row e * rows + n), 16-byte aligned.
 *  xq    device, in: q8_K [n_tokens or n_tokens * n_used][K/256], 16-byte aligned.
 *  ids   device, in: int32 [n_tokens][n_used], 4-byte aligned.
 *  1 <= n_tokens * n_used <= 2^20.  1 <= n_experts <= 1024.  1 <= rows <= 2^30.
 *  K >= 256, a multiple of 256. One expert's weights and all of xq below
 *  2 GiB (32-bit offsets).
 * A first kernel groups the pairs by expert into tiles of at most 64 pairs
 * (an expert's remainder of at most 32 pairs into tiles of at most 16); the
 * product then runs once over both lists. Every output is computed from its
 * own pair alone, so results do not depend on how pairs fall into tiles.
 *  workspace  the expert map (tile descriptors, the pairs grouped by
 *      expert, the tile counts): xq_gemm_q4k_id_workspace_bytes(n_tokens,
 *      n_used, n_experts) bytes (at most 4.3 MB), rewritten by every call
 *      from the first byte: no call that keeps counters may share it.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_gemm_q4k_id(float *y, const void *slab, const void *xq, const int32_t *ids,
                         int64_t n_tokens, int64_t n_used, int64_t n_experts, int64_t rows,
                         int64_t K, int64_t x_per_slot, void *workspace, size_t workspace_bytes,
                         void *stream);
size_t xq_gemm_q4k_id_workspace_bytes(int64_t n_tokens, int64_t n_used, int64_t n_experts);

/* Largest K the mat-vecs accept (the q8_K row is then 1.25 MiB). Rows of up
 * to 49152 columns stage the row in the workgroup's LDS (60 KiB at most);
 * longer rows read it from global memory, where every workgroup finds it in
 * L2. The small-M product (xq_gemm_q4k_small_m) takes any K. */
#define XQ_MAX_K 1048576

/* Byte sizes of the layouts above; 0 when the shape is invalid. */
size_t xq_q8k_bytes(int64_t rows, int64_t K);   /* rows*(K/256)*320 */
size_t xq_q4k_bytes(int64_t N, int64_t K);      /* N*(K/256)*144 */
size_t xq_iq4nl_bytes(int64_t N, int64_t K);    /* N*(ceil4(2*(K/32)) + 16*(K/32)) */

/* Static name of a status code ("XQ_OK", "XQ_E_SHAPE", ...). */
const char *xq_status_name(xq_status s);

/* Thread-local text of the last refusal on this thread ("" after success). */
const char *xq_last_error(void);

/*
 * Q4_0 x q8_K mat-vec: y[n] = sum_k w[n][k] * xhat[k] with w = d_c * (nibble - 8)
 * ("25 — Writing XPU Kernels", section 25.2: the Q4_0 twin of the IQ4_NL
 * kernel; its -8 rides on the activation's sum). The weight rows have the
 * IQ4_NL resident shape (K/32 f16 scales padded to a dword, then K/32 payloads
 * of 16 B; xq_iq4nl_bytes(N, K) bytes; xq_repack_iq4nl converts Q4_0 file
 * blocks too, they share the 18-byte shape); each 32-block's integer dot
 * sum(nibble*code) - 8*s uses the q8_K's stored sum s of its 32 codes.
 *  Same arguments, alignment and limits as xq_gemv_iq4nl.
 */
xq_status xq_gemv_q4_0(float *y, const void *w_q4_0, const void *xq, int64_t N, int64_t K,
                       void *stream);

/*
 * Expert-grouped mat-vecs ("25 — Writing XPU Kernels", section 25.2.2: one
 * launch over a bank of experts, the dot loop of the dense kernel unchanged;
 * the expert is picked on the device through a selection buffer, nothing is
 * read back). For each selection slot kk in 0..used-1 and row r in
 * 0..rows-1:
 *   y[kk*rows + r] = row (sel[kk]*rows + r) of `slab` . activation kk
 * where activation kk is the q8_K row starting x_stride_blocks*kk blocks into
 * `xq` (x_stride_blocks = 0: every slot reads the one token, as in decode;
 * = K/256: slot kk reads row kk of a [used][K/256] q8_K tensor).
 *  slab  [n_experts][rows] rows of the format (Q4_K: [.][K/256] blocks of
 *        144 B; IQ4_NL: resident rows), experts back to back, 16-byte aligned.
 *  sel   device int32[used], 4-byte aligned. A value outside
 *        0..n_experts-1 makes that slot's `rows` outputs NaN (nothing is
 *        read for it); the other slots are unaffected.
 *  y     f32[used][rows], slot-major.
 *  1 <= used <= 65535, 1 <= rows, n_experts*rows <= 2^30, K as for the
 *  dense entry point, x_stride_blocks in {0, K/256}.
 * Each slot's outputs are bit-identical to the dense entry point (xq_gemv_q4k
 * or xq_gemv_iq4nl) on that expert's rows and that activation.
 */
xq_status xq_gemv_q4k_id(float *y, const void *slab, const void *xq, const int32_t *sel,
                         int64_t n_experts, int64_t used, int64_t rows, int64_t K,
                         int64_t x_stride_blocks, void *stream);
xq_status xq_gemv_iq4nl_id(float *y, const void *slab, const void *xq, const int32_t *sel,
                           int64_t n_experts, int64_t used, int64_t rows, int64_t K,
                           int64_t x_stride_blocks, void *stream);

/*
 * Bind-time repack of IQ4_NL file blocks into resident rows ("25 — Writing XPU
 * Kernels", section 25.4: weights are converted once, at upload, into the one
 * resident layout the kernels read; section 25.4.1: each work item moves one
 * payload dword). A file block is 18 bytes: the f16 scale, then the 16 payload bytes
 * (byte t: weight t in the low nibble, weight t+16 in the high nibble).
 *  file_blocks  the chunk: n_blocks blocks back to back, global blocks
 *               block_base .. block_base + n_blocks - 1 of a matrix of bpr
 *               blocks per row (block g is block g % bpr of row g / bpr);
 *               2-byte aligned (16-byte aligned chunks are staged through LDS
 *               with 16-byte loads, the faster route; the bytes written are
 *               the same).
 *  resident     row 0 of the matrix in resident rows (xq_iq4nl_bytes per row
 *               for K = 32*bpr: bpr f16 scales, zero-padded to a multiple of
 *               4 bytes, then bpr payloads of 16 B); 4-byte aligned; must hold
 *               rows 0 .. (block_base + n_blocks - 1) / bpr. Only the bytes of
 *               the chunk's blocks are written (and a row's 2 pad bytes, when
 *               bpr is odd, by the chunk holding the row's last block).
 *  1 <= n_blocks <= 2^29, 0 <= block_base <= 2^40, 1 <= bpr <= 2^24.
 * One pass reads each source byte once. A chunk that starts and ends on row
 * boundaries writes its scale prefix as whole dwords; any other chunk writes
 * each scale as a 16-bit half. xq_repack_dword_prefix_launches() counts the
 * launches of the first route in this process (section 25.7.2: a test that
 * the route fires, and one that it does not).
 */
xq_status xq_repack_iq4nl(void *resident, const void *file_blocks, int64_t n_blocks,
                          int64_t block_base, int64_t bpr, void *stream);
int64_t xq_repack_dword_prefix_launches(void);

/* ---- The paged key-value cache: attention, rotary positions, pages ----
 *
 * The calls below are what a decode step needs beside its mat-vecs. Their
 * conventions are those above, and in addition:
 *  - Strides are in elements of the tensor they belong to; the head dimension
 *    (dim) is always contiguous.
 *  - Lengths, tables, positions, slots and reference counts are device data
 *    that the host never reads. What the kernels find in them they check
 *    against the sizes of the call: a length is clamped to what the table
 *    (and max_len) can hold, a page number outside 0..pages-1 hides that
 *    page's tokens, a slot outside the cache drops its token. No value in
 *    them makes a kernel read or write outside its buffers.
 */

/* Element types. */
enum { XQ_F32 = 0, XQ_BF16 = 1, XQ_F16 = 2, XQ_E4M3 = 3, XQ_E2M1 = 4 };

/*
 * A paged cache, a host struct that describes device memory. Token j of a
 * sequence lies in page table[j / page] at slot j % page. Element
 * (layer l, page p, head h, slot s, d) of k is at
 *   k + l * k_stride[0] + p * k_stride[1] + h * k_stride[2] + s * k_stride[3] + d
 * (v the same with v_stride), so pages stored head by head or token by token
 * are both just strides.
 *  dtype  XQ_BF16, XQ_F16, XQ_E4M3 (8 bits, 4 exponent, 3 mantissa, largest
 *         448, no infinity) or XQ_E2M1 (4 bits, below). What a stored k stands
 *         for is k * k_scale, a stored v is v * v_scale, in every type; both
 *         finite and above 0.
 *  XQ_E2M1: an element is a sign (bit 3) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *  (bits 0..2, in that order), two to a byte, the even dim in the low bits,
 *  times a power of two that 32 consecutive dims of a row share: a byte,
 *  exponent + 127. dim is a multiple of 32; strides still count elements. The
 *  powers of layer l, page p, head h, slot s are dim / 32 bytes at
 *   k_exp + l * k_exp_stride[0] + p * k_exp_stride[1] + h * k_exp_stride[2] + s * k_exp_stride[3]
 *  (bytes; v_exp the same), of a row of 4 bytes up to 128 dims and of 8 beyond,
 *  whose rest has no meaning; bases and strides 4-byte aligned. The append
 *  stores powers 2^-23 .. 2^13 (bytes 104..140), which every call reads exactly,
 *  and 255 for a block that holds a NaN, all of which then are NaN. Of other
 *  bytes those up to 250 are read as what they stand for, but in a chunk's
 *  attention with XQ_F16 as f16 holds it. (Attention's sums are f32's, as with
 *  every type: a row's |q||k| added up over its dims, and the |v| of the tokens
 *  that it sees, have to stay below 2^127.) Other types do not read these fields.
 *  1 <= layers <= 2^24; 1 <= pages, page; 1 <= kv_heads <= 2^20; pages * page <= 2^31 - 1 (a slot is an
 *  int32's worth; byte offsets are 64-bit). dim a multiple of 16, 16..256.
 *  k and v 16-byte aligned; strides >= 0 and multiples of 16 bytes.
 * Attention and the append work on one layer (layers = 1: a layer of a larger
 * cache is the struct with k and v advanced).
 */
typedef struct {
    void *k, *v;
    int64_t layers, pages, kv_heads, page, dim;
    int64_t k_stride[4], v_stride[4];
    int32_t dtype;
    float k_scale, v_scale;
    void *k_exp, *v_exp;
    int64_t k_exp_stride[4], v_exp_stride[4];
} xq_kv;

/*
 * Attention of one new token per sequence over the paged cache. Sequence b
 * has lens[b] tokens in the cache, the new one the last of them. With n =
 * lens[b] and g = h / (heads / kv_heads), token j is visible when j < n and
 * (window = 0, or j >= n - window, or j < sinks), and
 *   out[b][h] = sum_j p_j * v_scale * v_j[g],
 *   p = softmax over the visible j of scale * k_scale * (q[b][h] . k_j[g]).
 * A sequence with no visible token gives zeros; a visible infinity or NaN in v
 * reaches the dims that it is in. In k a NaN makes every dim NaN, and so does an
 * infinity but where it makes the score minus infinity, which weighs nothing.
 * Sums, maxima and products are held in f32; q and the weights p enter the
 * matrix instructions as two or three 16-bit pieces where one would round them
 * below the output's type.
 *
 *  out, q   device [seqs][heads][dim] of type io (XQ_F32, XQ_BF16, XQ_F16),
 *           strides per sequence (row) and head, both a multiple of 16 bytes;
 *           bases 16-byte aligned.
 *  tables   device int32, row b at tables + b * table_stride, table_width
 *           pages per row; lens device int32[seqs].
 *  heads a multiple of kv_heads, heads / kv_heads <= 256, seqs * kv_heads <= 2^20,
 *  seqs * kv_heads * ceil(heads / kv_heads / 16) < 2^24;
 *  k, and v, of one layer within 64 GiB, their exponents within 16.
 *  scale finite, and scale * k_scale * log2(e) too; scores of any size, but that
 *  product times q . k has to be in f32's range.
 *  window in 0..2^30 (0: none), sinks in 0..2^30 (read only with a window).
 *  max_len in 1..2^30: no length is above it (longer ones are clamped); the split of
 *  the work is planned for it, the result of a given plan is the same from
 *  call to call, bit for bit. Fewer than 768 (sequence, kv head, 16 heads) units
 *  (1536 of up to 64 dims, or of up to 128 of an 8-bit cache whose pages'
 *  heads lie apart or of a 4-bit one) share the work
 *  evenly whatever their lengths; from there on a unit is one workgroup's, and a
 *  sequence much longer than the others is the call's time.
 *  workspace  the splits' partial results and arrival counters:
 *      xq_attn_decode_workspace_bytes(...) bytes with the same arguments
 *      (0 when the plan does not split), zeroed before first use.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_attn_decode(void *out, const void *q, int32_t io, int64_t seqs, int64_t heads,
                         int64_t out_row, int64_t out_head, int64_t q_row, int64_t q_head,
                         const xq_kv *kv, const int32_t *tables, int64_t table_width,
                         int64_t table_stride, const int32_t *lens, float scale, int64_t window,
                         int64_t sinks, int64_t max_len, void *workspace, size_t workspace_bytes,
                         void *stream);
size_t xq_attn_decode_workspace_bytes(int64_t seqs, int64_t heads, const xq_kv *kv,
                                      int64_t max_len, int64_t window, int64_t sinks);

/*
 * Attention of a chunk of new tokens per sequence over the paged cache, which
 * already holds them (xq_rope_append). Sequence b's rows of q are
 * starts[b] .. starts[b+1]-1; with c of them and n = lens[b], row i has
 * position p = n - c + i and sees token j when j <= p and (window = 0, or
 * j > p - window, or j < sinks). The sum is xq_attn_decode's. A row that sees
 * nothing (a position below 0, pages that are missing) gives zeros. A token
 * that a row does not see has no influence on it, whatever its bytes are.
 * A tile of a chunk's rows is one workgroup's for all the tokens that it sees:
 * a few new tokens on a long context keep few compute units busy (8 on 131072
 * with 8 kv heads take 1.3 ms, 16 of 256 units).
 * The weights p enter their product with v rounded to 16 bits (io's, or better
 * where the rows are few; f16's 11 bits hold down to 2^-26 of a row's largest
 * weight, and what is below is off by at most 2^-37 of it); sums and maxima are
 * f32.
 *
 *  out, q   device [rows][heads][dim] of type io, XQ_BF16 or XQ_F16; the
 *           cache's type is io, XQ_E4M3 or XQ_E2M1. Strides and alignment as in
 *           xq_attn_decode. Rows of out that no sequence names stay as they are.
 *  starts   device int32[seqs + 1], ascending from >= 0 to <= rows; a
 *           sequence's part outside 0..rows or beyond max_chunk is left out,
 *           and its other rows keep the positions that they have in the whole.
 *  max_chunk in 1..rows: the longest chunk; rows * heads <= 2^31 - 1, seqs <= 2^16,
 *  seqs * kv_heads * ceil(max_chunk * heads / kv_heads / 128) < 2^24. The cache,
 *  heads, scale, window and sinks as xq_attn_decode.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_attn_prefill(void *out, const void *q, int32_t io, int64_t rows, int64_t seqs,
                          int64_t heads, int64_t out_row, int64_t out_head, int64_t q_row,
                          int64_t q_head, const xq_kv *kv, const int32_t *tables,
                          int64_t table_width, int64_t table_stride, const int32_t *lens,
                          const int32_t *starts, int64_t max_chunk, float scale, int64_t window,
                          int64_t sinks, void *stream);

/*
 * Rotary positions with one to four axes (a text has one; an image or a video
 * has time, height and width). The first `rot` elements of each head form
 * rot/2 pairs: (i, i + rot/2), or (2i, 2i + 1) when `adjacent` is 1. Pairs are
 * dealt to the axes in order, sections[0] to axis 0 and so on (their sum is
 * rot/2). Pair i of token t turns by pos[axis][t] * freq[i]:
 *   (a, b) -> (a cos - b sin, a sin + b cos);
 * elements from rot on are copied. inverse = 1 turns the other way, which is
 * the gradient's direction (the rotation's transpose). The angle is formed
 * and reduced in f64, its sine and cosine are f32.
 */
typedef struct {
    const double *freq;   /* device f64[rot/2], 8-byte aligned */
    int64_t rot, axes, adjacent;
    int64_t sections[4];  /* >= 0; those from `axes` on are ignored */
} xq_rope_freqs;

/*
 *  out  device [tokens][heads][dim] of type out_type, x of type x_type (each
 *       XQ_F32, XQ_BF16 or XQ_F16), aligned to their elements. out may be x
 *       where types and strides are the same.
 *  pos  device int32, axis a's positions at pos + a * pos_stride.
 *  tokens, heads >= 1, tokens * heads <= 2^31 - 1; dim a multiple of 8, 8..1024;
 *  rot a multiple of 8, 8..dim.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_rope(void *out, int32_t out_type, int64_t out_row, int64_t out_head, const void *x,
                  int32_t x_type, int64_t x_row, int64_t x_head, int64_t tokens, int64_t heads,
                  int64_t dim, const int32_t *pos, int64_t pos_stride, const xq_rope_freqs *rope,
                  int32_t inverse, void *stream);

/*
 * The same rotation of q and k, fused with the append of k and v to the
 * cache: q_out = rope(q); token t's rope(k) / k_scale and v / v_scale go to
 * slot slots[t] (page slots[t] / page, place slots[t] % page), rounded once to
 * the cache's type (XQ_E4M3: clamped to +-448). XQ_E2M1: a block of 32 takes
 * the smallest power of two 2^e, e in -23..13, by which its largest |x| is
 * below 7 (so that it rounds to 6 at most), and each x / 2^e is rounded to the
 * nearest of the eight values, ties to the even code, above 6 to 6; rotation
 * (by the angle as f64 rounds pos * freq) and division are carried in f64 there,
 * so that a value next to a border between two codes falls on its own side, but
 * one of k within a few 2^-53 of |a| + |b|. A slot outside
 * 0..pages*page-1 writes nothing to the cache. No two tokens may have the same
 * slot.
 *  q, k, v  device [tokens][heads or kv_heads][dim] of one type x_type (XQ_F32,
 *           XQ_BF16, XQ_F16), each with its own strides (slices of one
 *           product's output are fine). slots device int64[tokens].
 * Sizes and errors as xq_rope, dim as the cache's.
 */
xq_status xq_rope_append(void *q_out, int32_t out_type, int64_t out_row, int64_t out_head,
                         const xq_kv *kv, const void *q, int64_t q_row, int64_t q_head,
                         const void *k, int64_t k_row, int64_t k_head, const void *v,
                         int64_t v_row, int64_t v_head, int32_t x_type, int64_t tokens,
                         int64_t heads, const int32_t *pos, int64_t pos_stride,
                         const xq_rope_freqs *rope, const int64_t *slots, void *stream);

/*
 * Tokens of a cache as values, for what looks into it or takes it elsewhere:
 * k_out[t][h] = k * k_scale and v_out[t][h] = v * v_scale of slot slots[t]
 * (page slots[t] / page, place slots[t] % page), in f32 and rounded once to
 * out_type. A slot outside 0..pages*page-1 gives zeros; a slot may be named
 * more than once.
 *  k_out, v_out  device [tokens][kv_heads][dim] of type out_type (XQ_F32,
 *         XQ_BF16, XQ_F16), each with its own strides, aligned to their
 *         elements. slots device int64[tokens].
 *  tokens >= 1, tokens * kv_heads <= 2^31 - 1; one layer.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_cache_read(void *k_out, int64_t k_row, int64_t k_head, void *v_out, int64_t v_row,
                        int64_t v_head, int32_t out_type, const xq_kv *kv, const int64_t *slots,
                        int64_t tokens, void *stream);

/*
 * The pages of a cache, all its layers at once. refs[p] counts the table
 * entries that name page p; 0 is free. A table row holds a sequence's pages
 * in order, then -1.
 *
 * xq_cache_copy: page src[i] -> page dst[i] for i < n. No page is named twice
 *   in dst, nor in both lists (unless src[i] = dst[i]); a pair with a page
 *   outside 0..pages-1 is skipped. n may be 0.
 * xq_cache_free: for i < n, row rows[i] (skipped outside 0..slots-1) gives its
 *   pages back: refs[p] -= 1 for each entry, the entries become -1, lens 0. A
 *   row named twice is freed once. (Where n is 0 the lists may be NULL.)
 * xq_cache_fork: for i < n, row children[i], which must be empty (lens 0),
 *   becomes a copy of row parents[i] as it was before the call: full pages are
 *   shared (refs + 1), a part-filled last page is copied into a fresh one.
 *   Fresh pages are the free ones in ascending order, taken in the order of
 *   i, so the result does not depend on timing. A fork is refused when a row
 *   is out of range, its child is not empty or named before, its parent's row
 *   is shorter than its length or has a bad page; its child stays empty. When
 *   the free pages run out the remaining forks that need one are refused too.
 *   status[0] = refused forks, status[1] = free pages that were lacking.
 * xq_cache_compact: the live pages (refs > 0) move to 0..live-1: those at or
 *   above `live`, ascending, into the free ones below it, ascending. Tables and
 *   refs follow. status[0] = 0, status[1] = live.
 *
 *  refs   device int32[pages]; tables device int32 [slots][width] with a
 *         stride; lens device int32[slots]; status device int32[2].
 *  1 <= slots <= 2^20; n >= 0, at most 2^20 (copy: 2^31 - 1; fork: slots).
 *  workspace  (fork, compact) xq_cache_workspace_bytes(pages, slots) bytes,
 *         rewritten by every call but for the first 96 KiB (other calls' counters).
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_cache_copy(const xq_kv *kv, const int32_t *src, const int32_t *dst, int64_t n,
                        void *stream);
xq_status xq_cache_free(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                        int64_t width, int64_t stride, int32_t *lens, const int32_t *rows,
                        int64_t n, void *stream);
xq_status xq_cache_fork(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                        int64_t width, int64_t stride, int32_t *lens, const int32_t *parents,
                        const int32_t *children, int64_t n, int32_t *status, void *workspace,
                        size_t workspace_bytes, void *stream);
xq_status xq_cache_compact(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                           int64_t width, int64_t stride, int32_t *status, void *workspace,
                           size_t workspace_bytes, void *stream);
size_t xq_cache_workspace_bytes(int64_t pages, int64_t slots);

/* ---- A mixture-of-experts layer for a few tokens ---- */

/* Scores of the experts, from their logits. */
enum { XQ_SOFTMAX = 0, XQ_SIGMOID = 1 };

/*
 * The router: for each token the `used` experts of the highest scores, the
 * highest first, and their weights.
 *   logit[e] = router[e] . x[t] (f32 sums);
 *   score[e] = exp(logit[e]) / sum over all experts, or 1 / (1 + exp(-logit[e]));
 *   ids[t] = those with the largest score[e] + bias[e] (bias may be NULL), the
 *     lowest index among equals, NaN below everything. These are f32 numbers:
 *     scores that round to one are equal (sigmoid's to 1 from logits of 17.4 on,
 *     softmax's to 0 from 104 below the highest). Only softmax without a bias
 *     goes by the logits, whose order its scores have before they are rounded;
 *     a bias of zeros is a bias;
 *   weights[t][k] = score[ids[t][k]] (bias not in it), divided by the sum over
 *     the chosen where normalize = 1 (0 where that sum is 0), times scale.
 *  x       device [tokens][K] of type x_type (XQ_F32, XQ_BF16, XQ_F16), rows
 *          x_row elements apart; router device [experts][K] of type router_type
 *          (the same three), contiguous. Both bases and x's rows 16-byte aligned.
 *  bias    device f32[experts] or NULL; ids device int32[tokens][used], weights
 *          device f32[tokens][used]. 4-byte aligned.
 *  1 <= tokens <= 512; 1 <= used <= 64, used <= experts <= 1024; K a multiple of
 *  8, 8..XQ_MAX_K. scale finite.
 *  workspace  arrival counters in its first 96 KiB, then the logits:
 *          xq_moe_route_workspace_bytes(tokens, experts) bytes, zeroed before
 *          first use.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_moe_route(int32_t *ids, float *weights, const void *x, int32_t x_type, int64_t x_row,
                       const void *router, int32_t router_type, const float *bias, int64_t tokens,
                       int64_t experts, int64_t used, int64_t K, int32_t score, int32_t normalize,
                       float scale, void *workspace, size_t workspace_bytes, void *stream);
size_t xq_moe_route_workspace_bytes(int64_t tokens, int64_t experts);  /* 0 if the sizes are refused */

/*
 * The chosen experts' feed-forward on Q4_K weights, and its weighted sum:
 *   h[t][k] = silu(G_e x^[t]) * (U_e x^[t]), e = ids[t][k], silu(g) = g / (1 + exp(-g)),
 *   y[t] = sum_k weights[t][k] * (D_e h^[t][k]),
 * where x^ and h^ are x[t] and h[t][k] in q8_K (as xq_quantize_q8k, but with
 * d = amax * (1/127), one f32 product with the constant as f32 rounds it) and
 * the products are xq_gemv_q4k's; h is f32, the sum over k in f32, one rounding
 * to y's type. A slot whose id lies outside 0..experts-1 is left out (a token
 * with no other gets zeros); an id may stand in several slots of a token.
 * x is to be finite, as for xq_quantize_q8k.
 *  y, x    device [tokens][hidden] of type io (XQ_F32, XQ_BF16, XQ_F16), rows
 *          y_row and x_row elements apart; x and its rows 16-byte aligned, y
 *          aligned to its elements. y may be x where the strides are the same.
 *  gate, up  device Q4_K, `experts` experts of ffn rows of hidden columns back to
 *          back; down the same of hidden rows of ffn columns. 16-byte aligned.
 *  ids     device int32[tokens][used], weights device f32[tokens][used].
 *  tokens, used >= 1, tokens * used <= 512 (more are xq_gemm_q4k_id's); 1 <=
 *  experts <= 1024; hidden and ffn multiples of 256, 256..32768.
 *  workspace  h, and for several tokens the q8_K rows and the slots' results,
 *          behind the first 96 KiB: xq_moe_q4k_workspace_bytes(...) bytes.
 * Errors: XQ_E_NULL, XQ_E_SHAPE, XQ_E_ALIGN, XQ_E_DEVICE, XQ_E_LAUNCH.
 */
xq_status xq_moe_q4k(void *y, int64_t y_row, const void *x, int64_t x_row, int32_t io,
                     const void *gate, const void *up, const void *down, const int32_t *ids,
                     const float *weights, int64_t tokens, int64_t used, int64_t experts,
                     int64_t hidden, int64_t ffn, void *workspace, size_t workspace_bytes,
                     void *stream);
size_t xq_moe_q4k_workspace_bytes(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn);  /* 0 if refused */

/*
 * Measurement helper, not part of the method: read `bytes` of device memory
 * once with 16-byte loads and fold them into one word per workgroup of
 * `sink` (sink must hold xq_bench_sink_words(bytes) uint32). Its duration
 * gives the streaming-read ceiling the mat-vecs are held against ("25 —
 * Writing XPU Kernels", section 25.1: measure the bandwidth once per device
 * with a streaming pass well past L2).
 *  buf 16-byte aligned, bytes a positive multiple of 16.
 */
xq_status xq_bench_stream_read(const void *buf, int64_t bytes, uint32_t *sink, void *stream);
int64_t xq_bench_sink_words(int64_t bytes);

#ifdef __cplusplus
}
#endif

#endif /* XQ_H */
