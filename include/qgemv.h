/*
 * qgemv.h - C ABI of libqgemv: weight-only low-bit dequantize-and-multiply on MI355X (gfx950).
 *
 * Formats (one byte table per 256 weights, "二三五六位量化" page section 2.3; INT4 from the
 * DBHOO-CIM page sections 2.1, 3.1, 3.2 and 4.1):
 *
 *   QG_Q4G32  INT4 symmetric, groups of 32 consecutive weights of a row, fp32 scale per group:
 *             scale = max(max|w| / 8, 1e-12), q = clamp(rint(w / scale), -8, 7) in fp32,
 *             w_hat = q * scale; 16 B of codes + 4 B of scale per group (5.0 bpw).
 *   QG_Q4G16, QG_Q4G64, QG_Q4G128  the same INT4 code with groups of 16, 64 or 128 weights
 *             (6.0, 4.5, 4.25 bpw; DBHOO-CIM page section 5.1 advises groups of 16 against
 *             outlier weights). k must be a multiple of 64 (of 128 for QG_Q4G128).
 *   QG_Q4A32  INT4 asymmetric, groups of 32, fp32 scale s and uint8 zero point z per group
 *             ("二三五六位量化" page section 2.1's x = s (q - z); DBHOO-CIM page section 5.1
 *             keeps asymmetric quantization for layers the symmetric grid serves badly):
 *             lo = min(0, min w), hi = max(0, max w), s = max((hi - lo) / 15, 1e-12),
 *             z = clamp(rint(-lo / s), 0, 15), c = clamp(rint(w / s) + z, 0, 15) in fp32,
 *             w_hat = s * (c - z); 16 B of codes + 4 B of scale + 1 B of zero point per group
 *             (5.25 bpw). k must be a multiple of 64.
 *   QG_Q4G32H INT4 symmetric, groups of 32, fp16 scale ("二三五六位量化" page section 2.1: a
 *             16-bit scale per group of 32): s = fp16_rn(max|w| / 8 in fp32) (0 raised to
 *             2^-24; past 65504 QG_ERR_RANGE), q = clamp(rint(w / s), -8, 7) in fp32 against
 *             that stored s, w_hat = q * s; 16 B of codes + 2 B of scale per group (4.5 bpw).
 *             k must be a multiple of 64.
 *   QG_Q2SB   256-weight super-block, 16 sub-blocks of 16, 2-bit codes c, 4-bit sub-scale sc
 *             and 4-bit sub-min m, fp16 d and dmin: w_hat = d*sc*c - dmin*m  (84 B, 2.625 bpw).
 *   QG_Q3SB   16 sub-blocks of 16, 3-bit codes, 6-bit sc, fp16 d: w_hat = d*sc*(c - 4)
 *             (110 B, 3.4375 bpw).
 *   QG_Q5SB   8 sub-blocks of 32, 5-bit codes (low-4-bit plane + high-bit plane), 6-bit sc and
 *             m, fp16 d and dmin: w_hat = d*sc*c - dmin*m  (176 B, 5.5 bpw).
 *   QG_Q6SB   16 sub-blocks of 16, 6-bit codes (low-4-bit plane + high-2-bit plane), int8 sc,
 *             fp16 d: w_hat = d*sc*(c - 32)  (210 B, 6.5625 bpw).
 *   QG_Q2SB_BF16, QG_Q3SB_BF16, QG_Q5SB_BF16, QG_Q6SB_BF16  the same four formats with the
 *             super-scales d (and dmin) stored as bf16 instead of fp16 ("二三五六位量化" page
 *             section 2.3: against fp16 overflow of the super-scale); same records and sizes,
 *             bf16_ceil in place of fp16_ceil in the rule below. The GEMM paths for m > 4
 *             multiply fp16 W_hat on the matrix cores: weights beyond the fp16 range (which
 *             only bf16 super-scales can express) need the streaming kernel (qg_gemm with
 *             m <= 4, qg_gemm_grouped or qg_gemm_act_order with m <= 8).
 *   QG_Q3SB_PLANES  q3sb with the record's 96 code bytes stored as a 64-byte plane of the low
 *             2 bits (2-bit stream) and a 32-byte plane of the high bit (1-bit stream)
 *             ("二三五六位量化" page section 2.3: split widths that do not divide a byte into
 *             planes); same fields, rule and device layout as QG_Q3SB (110 B, 3.4375 bpw).
 *   QG_Q3G32, QG_Q5G32  plain group-wise 3- and 5-bit codes c with an fp32 scale s and an fp32
 *             min m per group of 32 (the form of "二三五六位量化" page section 3.3's gemv_q3:
 *             w_hat = s*c + m): m = min w (+0 for a zero minimum), s = max((max w - min w) / (2^b - 1), 1e-12),
 *             c = clamp(rint((w - m) / s), 0, 2^b - 1), difference and quotient in fp32.
 *             12 or 20 B of codes + 8 B per group (5.0 and 7.0 bpw). k a multiple of 64.
 *
 * Super-block scales are chosen by "range-covering round to nearest" (the pages give the
 * layouts, not the rule): with fp16_ceil(v) = smallest fp16 >= v, symmetric formats take
 * t_j = max|w_j| / (o - 0.5), d = fp16_ceil(max_j t_j / Smax), sc_j = min(Smax, ceil(t_j / d));
 * asymmetric formats take dmin = fp16_ceil(max_j(-min(0, min w_j)) / Smax),
 * m_j = min(Smax, ceil(-min(0, min w_j) / dmin)), t_j = (max(0, max w_j) + dmin*m_j) / (2^b - 1)
 * and d, sc_j as above; codes are rint (half to even) of w / (d*sc_j) (+ o), or of
 * (w + dmin*m_j) / (d*sc_j), clamped. All in fp64. Every weight is then within d*sc_j / 2.
 * Smax = 15 (q2sb), 63 (q3sb, q5sb), 127 (q6sb).
 *
 * Two encodings of a quantized matrix W [n][k] (W is out_features x in_features):
 *   canonical  the pages' interchange layout. q4g32: codes [n][k/2] (byte = u[2j] | u[2j+1] << 4
 *              with u = q + 8) followed by fp32 scales [n][k/32] (q4gG: [n][k/G]). q4a32: codes
 *              [n][k/2] (u = c), fp32 scales [n][k/32], uint8 zero points [n][k/32]. q4g32h: codes
 *              as q4g32, then fp16 scales [n][k/32]. q3g32 / q5g32: each row's codes as one
 *              little-endian b-bit stream [n][k*b/8], then fp32 scales [n][k/32], then fp32
 *              mins [n][k/32]. Super-block formats: records
 *              [n][k/256] of 84/110/176/210 bytes; fields in the byte table's column order
 *              (codes [, high-bit plane], sub-scales, d [, dmin]; q3sb_planes: low-2-bit plane,
 *              high-bit plane, sub-scales, d); every bit field is a
 *              little-endian bitstream (code i at bits [b*i, b*i + b), section 2.2's unpack3
 *              and unpack5); q2sb sub-block byte = sc | m << 4; q5sb's 12 bytes hold sixteen
 *              6-bit fields sc0..sc7, m0..m7; fp16 values little-endian.
 *   device     a planar, bit-permuted rearrangement of exactly the same bits, built for
 *              128-bit coalesced lane loads and single-instruction field extraction on CDNA4.
 *              Each plane is [n][row_bytes] row-major and starts 256-byte aligned. The planes
 *              hold the same number of bytes as the canonical encoding (plus < 1 KiB of
 *              inter-plane padding, never read). It is opaque: build it with
 *              qg_to_device_layout and read it back with qg_from_device_layout.
 *
 * Conventions: all sizes are int64_t. fp16 values are passed as uint16_t bit patterns.
 * `stream` is a hipStream_t (NULL = the default stream). Every function returns a qg_status.
 *
 * Ownership: the caller allocates and owns every buffer, host and device. The library never
 * allocates, frees or synchronizes, and keeps no pointer past the call. Host functions are
 * pure and thread-safe. Device functions validate their arguments on the host, return an
 * error without launching anything if they are invalid, and otherwise enqueue kernels on
 * `stream` and return; execution faults surface at the caller's next synchronization.
 */
#ifndef QGEMV_H
#define QGEMV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QG_ABI_VERSION 1

typedef enum qg_format {
  QG_Q2SB = 2,
  QG_Q3SB = 3,
  QG_Q4G32 = 4,
  QG_Q5SB = 5,
  QG_Q6SB = 6,
  QG_Q4G16 = 7,
  QG_Q4G64 = 8,
  QG_Q4G128 = 9,
  QG_Q4A32 = 10,
  QG_Q4G32H = 11,
  QG_Q2SB_BF16 = 12,
  QG_Q3SB_BF16 = 13,
  QG_Q3SB_PLANES = 14,
  QG_Q5SB_BF16 = 15,
  QG_Q6SB_BF16 = 16,
  QG_Q3G32 = 17,
  QG_Q5G32 = 18
} qg_format;

typedef enum qg_status {
  QG_OK = 0,
  QG_ERR_NULL = -1,      /* a required pointer is NULL                                      */
  QG_ERR_SHAPE = -2,     /* n, k or m out of range (k % 256 super-blocks, % 32 q4g32, ...)   */
  QG_ERR_ALIGN = -3,     /* a device pointer or leading dimension is misaligned              */
  QG_ERR_NONFINITE = -4, /* a weight is NaN or infinite                                     */
  QG_ERR_RANGE = -5,     /* d or dmin does not fit fp16 (section 2.3's overflow warning)     */
  QG_ERR_FORMAT = -6,    /* unknown format or bit width                                     */
  QG_ERR_LAUNCH = -7,    /* the HIP runtime refused a launch                                 */
  QG_ERR_DEVICE = -8,    /* no usable gfx950 device / HIP runtime error                       */
  QG_ERR_WORKSPACE = -9  /* the workspace is smaller than the call needs                      */
} qg_status;

#define QG_MAX_PLANES 4

/* Device layout of one n x k matrix. */
typedef struct qg_layout {
  int64_t total_bytes;                        /* bytes to allocate (planes + padding)        */
  int64_t algorithmic_bytes;                  /* bytes one dequant-GEMV must read            */
  int32_t nplanes;
  int32_t reserved;
  int64_t plane_offset[QG_MAX_PLANES];        /* from the buffer start, 256-byte aligned     */
  int64_t plane_row_bytes[QG_MAX_PLANES];     /* bytes per row of each plane                 */
} qg_layout;

int qg_abi_version(void);
const char *qg_strerror(int status);
/* HIP's description of the last launch the library saw fail on this thread (QG_ERR_LAUNCH). */
const char *qg_last_hip_error(void);

/* ---- sizes and layouts (host) ------------------------------------------------------- */

/* Bytes of the canonical encoding of an n x k matrix: n * k / 256 records of 84 / 110 / 176 /
 * 210 bytes for the super-block formats ("二三五六位量化" page section 2.3, byte table), and
 * for INT4 16 bytes of codes plus the scale bytes per group (DBHOO-CIM page sections 3.2, 4.1).
 * Errors: QG_ERR_NULL, QG_ERR_FORMAT, QG_ERR_SHAPE. */
int qg_canonical_bytes(int fmt, int64_t n, int64_t k, int64_t *bytes);
/* Device layout of an n x k matrix: the planes (codes, high-bit planes, sub-scales,
 * super-scales) kept apart, as the pages advise for the scales (DBHOO-CIM page section 4.1,
 * "二三五六位量化" page section 2.3), with their offsets and row strides; algorithmic_bytes
 * equals the canonical size. Errors: QG_ERR_NULL, QG_ERR_FORMAT, QG_ERR_SHAPE. */
int qg_device_layout(int fmt, int64_t n, int64_t k, qg_layout *out);
/* The two sizes a caller needs, in one call: *total = bytes to allocate for the device layout
 * (planes and padding), *algorithmic = the bytes one dequant GEMV reads (the canonical size,
 * which the effective-bandwidth figure of DBHOO-CIM page section 4.4 divides by the time).
 * Either pointer may be NULL. Errors: QG_ERR_FORMAT, QG_ERR_SHAPE. */
int qg_packed_bytes(int fmt, int64_t n, int64_t k, int64_t *total, int64_t *algorithmic);

/* ---- bitstreams (host; "二三五六位量化" page section 2.2) ---------------------------- */

/* Pack count codes of `bits` bits (1..8) into a little-endian bitstream of
 * ceil(count*bits/8) bytes; code i occupies stream bits [bits*i, bits*i + bits).
 * Codes must be < 2^bits (QG_ERR_RANGE otherwise). */
int qg_pack_bits(int bits, const uint8_t *codes, int64_t count, uint8_t *out);
/* Inverse of qg_pack_bits. */
int qg_unpack_bits(int bits, const uint8_t *in, int64_t count, uint8_t *codes);

/* ---- quantizers (host, synchronous) -------------------------------------------------- */

/* Quantize fp32 W [n][ldw] (first k columns used, ldw >= k) into the canonical encoding
 * `canonical` (qg_canonical_bytes(fmt, n, k) bytes). Multi-threaded over rows; the output is
 * independent of the thread count. Errors: QG_ERR_SHAPE, QG_ERR_NONFINITE, QG_ERR_RANGE. */
int qg_quantize(int fmt, const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4g32(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q2sb(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q3sb(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q5sb(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q6sb(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4g16(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4g64(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4g128(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4a32(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q4g32h(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q2sb_bf16(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q3sb_bf16(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q5sb_bf16(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q6sb_bf16(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q3g32(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q5g32(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);
int quantize_q3sb_planes(const float *w, int64_t n, int64_t k, int64_t ldw, uint8_t *canonical);

/* Canonical encoding (host) -> device layout (host buffer of qg_device_layout().total_bytes;
 * padding is zeroed). A pure bit permutation: the scales move to planes of their own
 * (DBHOO-CIM page section 4.1 keeps scales in a separate array) and the codes to planes of
 * whole bit fields ("二三五六位量化" page section 2.3 splits 5- and 6-bit codes into a low
 * plane and a high-bit plane). Errors: QG_ERR_NULL, QG_ERR_FORMAT, QG_ERR_SHAPE. */
int qg_to_device_layout(int fmt, const uint8_t *canonical, int64_t n, int64_t k, uint8_t *device_layout);
/* Device layout (host copy) -> canonical encoding. Inverse of qg_to_device_layout; same
 * errors. */
int qg_from_device_layout(int fmt, const uint8_t *device_layout, int64_t n, int64_t k, uint8_t *canonical);

/* ---- dequant GEMV, batch 1 (device) ------------------------------------------------------
 * y[r] = sum_c W_hat[r][c] * x[c] for r < n, with W in device layout (`w`, 256-byte aligned),
 * x fp16 [k] (16-byte aligned), y fp16 [n]; fp32 accumulation, one fp16 rounding at the end.
 * The packed weights are streamed once with 128-bit loads and decoded in registers; no
 * dequantized weight is ever written to memory (DBHOO-CIM page section 3.3; "二三五六位量化"
 * page section 3.3's gemv_q3 and its Sigma-x rewrite). Limits: k <= 2^20 and every plane
 * of the device layout under 4 GiB. n == 0 is a no-op; k == 0 writes zeros.
 * Errors: QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_FORMAT, QG_ERR_LAUNCH. */
int dequant_gemv_q4g32(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q2sb(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q3sb(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q5sb(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q6sb(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q4g16(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q4g64(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q4g128(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q4a32(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q4g32h(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q2sb_bf16(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q3sb_bf16(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q5sb_bf16(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q6sb_bf16(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q3g32(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q5g32(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);
int dequant_gemv_q3sb_planes(const void *w, const uint16_t *x, uint16_t *y, int64_t n, int64_t k, void *stream);

/* Generic form: y_f32 != 0 writes fp32 y (4-byte aligned) instead of fp16. */
int qg_gemv(int fmt, const void *w, const uint16_t *x, void *y, int y_f32, int64_t n, int64_t k, void *stream);

/* Strided batch of independent GEMVs of one shape in one launch: for b < count,
 * y_b = W_b x_b with W_b at w + b*w_stride (bytes, multiple of 256), x_b at x + b*x_stride
 * and y_b at y + b*y_stride (elements; x_stride a multiple of 8). Same numerics as qg_gemv.
 * This is how a decode step issues several same-shape projections (or experts) without a
 * launch per matrix ("二三五六位量化" page section 1.2: decode reads every weight once per
 * token, one stream bound by bandwidth). count == 0 is a no-op. Errors as qg_gemv, and
 * QG_ERR_SHAPE for count < 0, QG_ERR_ALIGN for a misaligned stride. */
int qg_gemv_batched(int fmt, const void *w, int64_t w_stride, const uint16_t *x, int64_t x_stride,
                    void *y, int64_t y_stride, int y_f32, int64_t count, int64_t n, int64_t k, void *stream);

/* ---- dequant GEMM with a few activation rows (device) ------------------------------------
 * Y[i][r] = sum_c X[i][c] * W_hat[r][c] for i < m, r < n: X fp16 [m][ldx] (16-byte aligned,
 * ldx >= k and a multiple of 8 when m > 1), Y fp16 [m][ldy] (ldy >= n when m > 1). Batched
 * decode: the weights are streamed once per launch and each decoded code meets all the
 * launch's activation rows, up to 16 of them ("二三五六位量化" page section 1.2: decode
 * batches and prefill are the same contraction with more activation rows; DBHOO-CIM page
 * section 5.2: still bandwidth-bound at small batch, compute-bound at large batch). Any m >= 1:
 * m <= 4 runs on the vector units (each decoded code pair meets every activation row in a
 * v_dot2; the kernel of qg_gemv, qg_gemm_grouped and qg_gemm_act_order), 5 <= m <= 16
 * decodes each code once to fp16 and multiplies on the matrix cores in the same single
 * weight stream, and m > 16 (prefill) stages fp16 weight and activation tiles in LDS for
 * 32x32 matrix-core tiles. For 17 <= m <= 128, when a cost estimate says so (the prefill
 * tiles then carry mostly dead rows), the rows run instead as launches of that decode
 * kernel of up to 32 rows each (two 16-row blocks share each decoded fragment; a 32-row
 * launch gives the same bits as two 16-row launches). Limits as dequant_gemv_*; also
 * ldx < 2^26 for 5 <= m <= 16 and
 * ldx < 2^22 for m > 16 (32-bit activation offsets within a 16-row or a 256-row tile).
 * m == 0 or n == 0 is a no-op; k == 0 writes zeros. Errors as dequant_gemv_*.
 * Precision: m <= 4 works on the codes in fp32 (the 2e-3 * sum |W_hat x| bound holds at any
 * weight and activation scale). The matrix-core paths (m > 4) round each decoded weight to
 * fp16, which keeps 11 significant bits down to 2^-14 only: they hold the bound while the
 * quantization steps (an INT4 group scale, a super-block's d * sc) are at least 2^-14 and
 * the weights stay within +-65504; smaller steps lose relative precision (fp16 subnormals)
 * and weights beyond the fp16 range (the _bf16 formats only) are not representable. Such
 * layers take m <= 4 launches, or qg_gemm_grouped / qg_gemm_act_order up to 8 rows. */
int dequant_gemm_q4g32(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                       int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q2sb(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q3sb(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q5sb(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q6sb(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q4g16(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q4g64(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q4g128(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                      int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q4a32(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                       int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q4g32h(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                        int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q2sb_bf16(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                            int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q3sb_bf16(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                            int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q5sb_bf16(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                            int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q6sb_bf16(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                            int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q3g32(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                        int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q5g32(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                        int64_t m, int64_t n, int64_t k, void *stream);
int dequant_gemm_q3sb_planes(const void *w, const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy,
                              int64_t m, int64_t n, int64_t k, void *stream);
/* Generic form; y_f32 != 0 writes fp32 Y (4-byte aligned). */
int qg_gemm(int fmt, const void *w, const uint16_t *X, int64_t ldx, void *Y, int64_t ldy, int y_f32,
            int64_t m, int64_t n, int64_t k, void *stream);

/* Act-order weights ("二三五六位量化" page section 2.4 and section 3.2, stage 3: GPTQ
 * quantizes the columns in an activation-dependent order and stores that permutation, which
 * inference must apply): W was quantized with its columns permuted, stored column c being
 * original column perm[c], so Y[i][r] = sum_c X[i][perm[c]] * W_hat[r][c]. perm: int32 [k] on
 * the device (16-byte aligned), entries in [0, k) (an entry outside that range reads an
 * activation of 0; it never reads outside X). The gather is fused into the streaming
 * kernel's activation load, so the result equals that kernel's on the gathered activations
 * bit for bit (qg_gemm_grouped's for any m, qg_gemm's for m <= 4). Activation rows of more
 * than 128 KB (m * k * 2 bytes) run as several launches of half, a quarter, ... of the rows,
 * the first size that fits; each such chunk equals qg_gemm_grouped's launch on its rows.
 * m: 0..8 activation rows (the streaming kernel); other arguments, limits and errors as
 * qg_gemm. */
int qg_gemm_act_order(int fmt, const void *w, const uint16_t *X, int64_t ldx, const int32_t *perm, void *Y,
                      int64_t ldy, int y_f32, int64_t m, int64_t n, int64_t k, void *stream);

/* Several matrices of any shapes, one activation-row count m (0..8), in one launch: for
 * g < count (at most 8), Y_g [m][ldy[g]] = X_g [m][ldx[g]] * W_hat_g^T with W_g of n[g] x k[g]
 * at w[g]. The arrays are host arrays read during the call; ldx and ldy are read only when
 * m > 1 (else the rows are dense). Each matrix is checked as by qg_gemm (for m <= 8) before
 * anything is launched; a matrix with n[g] == 0 is skipped and one with k[g] == 0 gets
 * zeros. Every matrix runs on the streaming vector-unit kernel of qg_gemv and shares its
 * numerics (qg_gemm's for m <= 4; for 5 <= m <= 8 qg_gemm uses the matrix cores and agrees
 * within the tolerance, not bit for bit). This serves the projections of a decode step that read one activation (q, k and
 * v; gate and up) or simply follow each other, with one launch's start and drain instead
 * of one per matrix ("二三五六位量化" page section 1.2: the decode pass is one weight stream
 * bound by bandwidth). Errors: QG_ERR_SHAPE (count > 8, m > 8, or a matrix's shape),
 * QG_ERR_NULL, QG_ERR_ALIGN, QG_ERR_FORMAT, QG_ERR_LAUNCH. */
int qg_gemm_grouped(int fmt, int count, const void *const *w, const uint16_t *const *X, const int64_t *ldx,
                    void *const *Y, const int64_t *ldy, const int64_t *n, const int64_t *k, int64_t m, int y_f32,
                    void *stream);

/* ---- 8-bit KV-cache group codec (device) --------------------------------------------------
 * "二三五六位量化" page section 4.1: the KV cache quantized to 8 bits, every 32 elements
 * sharing one fp16 scale (about 1.06 bytes per element, half of fp16). Codes are symmetric
 * int8 in [-127, 127]; the scale d of a group is the smallest fp16 >= max|x| / 127, q is
 * rint(x / d) on the exact quotient (halves to even), an all-zero group has d = 0 and q = 0,
 * and every element is within d/2 of d * q.
 *
 * qg_kv_quantize (on append): src fp16 [rows][ld_src] (first cols used; 16-byte aligned,
 * ld_src a multiple of 8 when rows > 1) -> codes int8 [rows][cols] (8-byte aligned) and scales
 * fp16 [rows][cols/32] (2-byte aligned). qg_kv_dequantize (on read): codes and scales ->
 * dst fp16 [rows][ld_dst] (16-byte aligned, ld_dst a multiple of 8 when rows > 1), each value
 * d * q rounded once to fp16 and saturated at +-65504 (d * q exceeds it only for code
 * +-127 at d = 516, the scale of a group whose maximum is above 65469; the saturated value
 * is still within d/2 of the input). cols must be a multiple of 32. Inputs must be finite
 * (a NaN or Inf gives unspecified codes for its group). rows == 0 or cols == 0 is a no-op.
 * Errors: QG_ERR_SHAPE, QG_ERR_NULL, QG_ERR_ALIGN, QG_ERR_LAUNCH. */
int qg_kv_quantize(const uint16_t *src, int64_t ld_src, int64_t rows, int64_t cols, int8_t *codes, uint16_t *scales,
                   void *stream);
int qg_kv_dequantize(const int8_t *codes, const uint16_t *scales, int64_t rows, int64_t cols, uint16_t *dst,
                     int64_t ld_dst, void *stream);

/* ---- paged KV cache (device) ---------------------------------------------------------------
 * A cache of many sequences in pages of page_tokens tokens each, which grow, branch and end
 * without moving each other ("二三五六位量化" page section 4.1 sizes the cache that these pages
 * hold: one K and one V entry of head_dim elements for every token, KV head and layer).
 *
 * A pool is [layers][num_pages] page records, layer l at pages + l * layer_stride bytes (records
 * are dense, layer_stride is read only when layers > 1). A record (qg_kv_page_bytes) holds, for
 * each KV head in turn, page_tokens (T) consecutive tokens of D = head_dim elements:
 *   QG_KV_Q8   K codes int8 [T][D], V codes int8 [T][D], K scales fp16 [T][D/32], V scales fp16
 *              [D/32][T]: the groups of 32, codes and scales of qg_kv_quantize. A cached value is
 *              what qg_kv_dequantize gives: d * q rounded once to fp16, saturated at +-65504.
 *   QG_KV_F16  K fp16 [T][D], V fp16 [T][D].
 * pages and layer_stride are 16-byte aligned; head_dim is 64, 128 or 256; page_tokens is a power
 * of two from 16 to 256; kv_heads is 1 to 1024, layers 1 to 65535, num_pages 1 to 2^31 - 1.
 *
 * Sequences are rows of a page table, int32 [table_rows][ld_table] on the device, of which the
 * first table_pages entries are used: token j of row s lies in page table[s][j / T] at place
 * j % T. An entry outside [0, num_pages) names no page (-1 by convention): nothing is read or
 * written there. lens, int32 [table_rows], holds the sequences' lengths in tokens (below 0
 * counts as 0, past table_pages * T as that), refs, int32 [num_pages], how many rows hold a
 * page (0: the page is free). All of them are device memory, so that every call below can be
 * captured into a graph and replayed while the cache changes. One table serves all layers.
 * Calls that read what another call writes are ordered by the caller (one stream, or events).
 *
 * Errors of all these calls: QG_ERR_NULL, QG_ERR_FORMAT (kind), QG_ERR_SHAPE, QG_ERR_ALIGN,
 * QG_ERR_LAUNCH. A call with nothing to do (count, batch or table_rows 0) is a no-op. */
typedef enum qg_kv_kind { QG_KV_Q8 = 1, QG_KV_F16 = 2 } qg_kv_kind;

typedef struct qg_kv_pool {
  void *pages;
  int64_t num_pages;
  int64_t layers;
  int64_t layer_stride;
  int32_t kind;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_tokens;
} qg_kv_pool;

/* Bytes of one page record (host). Errors: QG_ERR_NULL, QG_ERR_FORMAT, QG_ERR_SHAPE. */
int qg_kv_page_bytes(int kind, int64_t kv_heads, int64_t head_dim, int64_t page_tokens, int64_t *bytes);

/* Append: for i < count, K row k + i * ldk and V row v + i * ldv (fp16 [kv_heads * head_dim],
 * finite) are quantized (QG_KV_Q8) or copied (QG_KV_F16) into `layer` of the pool as token
 * positions[i] of table row seqs[i] (seqs NULL: row i). A row that names no place (a row outside
 * the table, a position below 0 or past table_pages * T, an entry that is no page) is skipped,
 * which is how a padded batch marks its empty rows. The count rows must name distinct places:
 * two rows written to one place leave a mix of both there. Nothing else of a page changes.
 * k, v: 16-byte aligned, ldk and ldv multiples of 8 and at least kv_heads * head_dim when
 * count > 1. count * kv_heads * head_dim / 8 must be below 2^31. */
int qg_kv_append(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                 int64_t table_pages, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                 const int32_t *seqs, const int32_t *positions, int64_t count, void *stream);

/* The way back: row i of k and v becomes the cached K and V of token positions[i] of row
 * seqs[i], zeros where that names no place. Rows may repeat. This gives a cached prefix as the
 * dense matrices that a prefill over it multiplies. Sizes and alignment as qg_kv_append. */
int qg_kv_gather(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                 int64_t table_pages, uint16_t *k, int64_t ldk, uint16_t *v, int64_t ldv, const int32_t *seqs,
                 const int32_t *positions, int64_t count, void *stream);

/* Attention of one new token a sequence over its cache: for b < batch, h < heads, with
 * g = h / (heads / kv_heads) and n = lens[b] clamped to [0, max_len],
 *   s_j = scale * <q[b][h], K[g][j]>   for the tokens max(0, n - window) <= j < n (all j < n
 *                                      when window is 0) that lie in a page of the pool,
 *   out[b][h] = sum_j e^(s_j) V[g][j] / sum_j e^(s_j),   lse[b][h] = ln sum_j e^(s_j).
 * A sequence without such a token gets out = 0 and lse = -inf whatever its q holds; else a head
 * whose q holds a NaN or an infinity gets NaN. What is cached for those tokens is finite, and so are their scores times
 * log2(e) in fp32; what lies elsewhere in a page may be anything. q: fp16, row b at q + b * ldq,
 * heads dense; out: fp16, or fp32 with out_f32 != 0, row b at out + b * ldo, heads dense; lse:
 * fp32 [batch][heads], or NULL. The new token's own K and V are in the cache before the call
 * (qg_kv_append) and counted by lens. Products, the softmax and its sums are fp32; the weights
 * e^(s_j - max) meet V as a pair of fp16 numbers (their rounding and its remainder, 22 bits).
 * Bounds of the error, relative to sum_j w_j |V_j| with w_j the weights' shares for fp32 out and
 * absolute for lse: 2 (head_dim + 8) 2^-24 max_j |scale| sum |q K_j| for the scores' fp32 rounding, 2^-20
 * and 2^-31 a token for the weights' pairs, 2^-24 for each of the sums' roundings: 76 a step of 32
 * tokens of a wave (at most 16 steps, or a wave's share if all head tiles' steps are shared out over
 * 1024 waves) and 520 for the joins; lse also has 2^-22 of its own and the scores' size. 8000 to
 * 131072 tokens of random values measured 4e-7 at most with |scale| sum |q K_j| up to 21, 6e-6 up to
 * 84 (lse 2e-6 and 6e-6). fp16 out adds its one rounding.
 *
 * The cache's length is split over the workgroups, whose partial results go through
 * `workspace` (device, 16-byte aligned, at least qg_paged_attention_bytes, which is 0, and NULL will
 * do, for short lengths; its contents need no preparation, and calls that may run at the same time
 * each need their own). The split follows
 * lens on the device, so a captured call follows lens as it changes; the result depends on the
 * split only by rounding, and equal inputs give equal bits. max_len bounds the lengths (a graph
 * that is replayed while sequences grow passes the longest it will see); the table has at least
 * ceil(max_len / T) entries a row. q and out: 16-byte aligned, ldq a multiple of 8 (ldo of 8, of
 * 4 for fp32) and at least heads * head_dim when batch > 1. heads is a multiple of kv_heads;
 * batch * heads is at most 2^22, max_len at most 2^30, batch * heads * ceil(max_len / 32) below
 * 2^31, window >= 0, scale * log2(e) finite in fp32. out, lse and the workspace overlap nothing
 * that the call reads: one workgroup's q may be loaded after another's out is stored.
 * Errors: also QG_ERR_WORKSPACE, and QG_ERR_RANGE for any other scale. */
int qg_paged_attention_bytes(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t max_len, int64_t *bytes);
int qg_paged_attention(const qg_kv_pool *pool, int64_t layer, const uint16_t *q, int64_t ldq, const int32_t *table,
                       int64_t ld_table, const int32_t *lens, int64_t batch, int64_t heads, int64_t max_len,
                       int64_t window, float scale, void *out, int64_t ldo, int out_f32, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream);

/* Copy whole pages in every layer: page src[i] to page dst[i] for i < count (device arrays). A
 * pair with an index outside [0, num_pages) is skipped. No page may be a destination twice, or
 * both a source and a destination of different pairs. count is at most 2^23 (also of freed
 * rows below). */
int qg_kv_copy_pages(const qg_kv_pool *pool, const int32_t *src, const int32_t *dst, int64_t count, void *stream);

/* Fork: for i < count, table row dst_rows[i] becomes a second holder of row src_rows[i]'s
 * tokens. Its whole pages are shared (refs + 1 each); a last page that is only partly filled is
 * copied in every layer to page new_pages[i], whose refs become 1, so that the two rows grow
 * apart. Where an entry of the source row is no page, the new row's is the same, a last one
 * included: nothing is copied then, and new_pages[i] stays as it is. Further entries of the row
 * become -1 and lens[dst] = lens[src]. What the row held before is overwritten, not released
 * (qg_kv_free releases it). new_pages[i] is a free page, used only when a last page is copied; one
 * that some row holds would be overwritten. A fork is skipped, its row left as it was, when a row
 * is outside the table, when dst_rows[i] is also a source row or an earlier destination row of the
 * call, or when a copy is needed and new_pages[i] is outside the pool or named earlier in the call.
 * count is at most 4096. */
int qg_kv_fork(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *src_rows, const int32_t *dst_rows,
               const int32_t *new_pages, int64_t count, void *stream);

/* Free: for i < count, table row rows[i] gives up its pages (refs - 1 for each page of its
 * lens tokens), its table_pages entries become -1 and its length 0. A row outside the table, or
 * one that is empty already (named twice, for instance), is left as it is. */
int qg_kv_free(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *rows, int64_t count, void *stream);

/* Compact: with L pages held (refs > 0), the held pages at index L and above move, in every
 * layer, to the free pages below L (both in ascending order), after which the pages from L on
 * are free and that end of the pool can be given back. remap, int32 [num_pages], receives each
 * page's new index (-1 for a free page), live, int32 [1], receives L, refs_out the moved counts
 * and table_out the table with its entries replaced (-1 where the page was free or no page).
 * table_out and refs_out may be table and refs themselves; else they must not overlap them.
 * workspace (4-byte aligned): at least qg_kv_compact_bytes, as for qg_paged_attention.
 * num_pages is at most 2^24 here. Errors: also QG_ERR_WORKSPACE. */
int qg_kv_compact_bytes(const qg_kv_pool *pool, int64_t *bytes);
int qg_kv_compact(const qg_kv_pool *pool, const int32_t *table, int64_t ld_table, int32_t *table_out, int64_t ld_out,
                  int64_t table_rows, int64_t table_pages, const int32_t *refs, int32_t *refs_out, int32_t *remap,
                  int32_t *live, void *workspace, int64_t workspace_bytes, void *stream);

/* Attention of one new token a sequence where neighbouring sequences share their first tokens (forks of one
 * prompt, many requests after one long instruction): the shared tokens are read and multiplied once for
 * all of them. Group g < groups is the rows starts[g] to starts[g + 1] - 1 of the batch (int32 [groups + 1] on the
 * device; rows before starts[0] and from starts[groups] on are in no group), and the first prefix[g] tokens
 * (int32 [groups] on the device) of each of its rows are the same, in the same pages or in equal ones: as far as
 * they fill whole pages and row starts[g] has them (a prefix below 0 counts as 0, past lens[starts[g]] as that), they
 * are read once through that row's table entries, or, where a group's few rows make that more work, for each row
 * through its own. Further tokens, and all of a group of one row, are read through each
 * row's own entries. A row that is shorter than the prefix sees its lens tokens.
 * Values of starts outside [0, batch] count as the nearest of these, one below an earlier one as that one.
 * The result is defined as qg_paged_attention's with window 0, its error bounded as there (with 512 in place of 1024
 * waves in the count of a wave's steps, fewer where max_tail does not hold), and by 2^-31 sum |V_j| on top for weights
 * below fp16's normal range.
 *
 * max_tail bounds the tokens that a row does not share and chooses the workspace and with it how far the work on them
 * is spread: where rows have more of them it is slower, no less right. Arguments, alignment, limits and errors otherwise as
 * qg_paged_attention; groups is at most 1023 and at most batch, and the sizes are refused (QG_ERR_SHAPE) where the
 * work could pass 2^31 units. The workspace, at least qg_prefix_attention_bytes, is always needed; what is said of
 * qg_paged_attention's holds for it. */
int qg_prefix_attention_bytes(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len,
                              int64_t max_tail, int64_t *bytes);
int qg_prefix_attention(const qg_kv_pool *pool, int64_t layer, const uint16_t *q, int64_t ldq, const int32_t *table,
                        int64_t ld_table, const int32_t *lens, const int32_t *starts, const int32_t *prefix,
                        int64_t groups, int64_t batch, int64_t heads, int64_t max_len, int64_t max_tail, float scale,
                        void *out, int64_t ldo, int out_f32, float *lse, void *workspace, int64_t workspace_bytes,
                        void *stream);

/* Extend: places for a step's new tokens. Row r of the table asks for add[r] tokens (int32 [table_rows] on the
 * device; 0 or less: none) after its lens[r], and for the pages that it lacks for them. With N_r the tokens asked
 * by rows 0 to r, its tokens are the places N_(r-1) to N_r - 1 of the slot map seqs, positions (int32
 * [slots]), whether it gets them or not: the order in which the caller's batch holds them. A row is served
 * unless
 *   N_r exceeds slots, or lens[r] + add[r] the row's table_pages * T tokens, or
 *   its last page is partly filled and not held by this row alone (refs 1): appending would write into
 *     another row's tokens (qg_kv_fork copies such a page), or
 *   it lacks pages and these, with those lacked by the rows before it that neither of the two refuses, are more
 *     than there are free pages (refs 0 or less). A row that this refuses counts for the rows behind it, too: after one
 *     request for more pages than are free, no later row that lacks a page is served, though pages are left (3 free
 *     pages of 16 tokens, empty rows that ask for 80 and 32: both get none). A caller that wants later rows served asks for
 *     no more than there is, or for such requests behind the others.
 * A served row's new entries name free pages, in ascending order over all rows, whose refs become 1; lens[r] grows
 * by add[r], granted[r] (int32 [table_rows]) is add[r], and slot i of its tokens holds seqs r and
 * positions the token's place in the row: what qg_kv_append takes. A row that is not served stays as it was,
 * granted is 0, its slots hold -1 and -1, and so do the slots past the last row's. starts (int32 [table_rows + 1], or
 * NULL) receives N_(r-1) at r, at most slots. The entries past a row's pages are overwritten whatever they
 * hold (-1 by convention).
 * workspace (4-byte aligned): at least qg_kv_extend_bytes, as for qg_paged_attention. add, granted, starts, the
 * slot map and the workspace overlap nothing else. table_rows is at most 65536, num_pages 2^24, slots
 * 2^26 here. Errors: also QG_ERR_WORKSPACE. */
int qg_kv_extend_bytes(const qg_kv_pool *pool, int64_t table_rows, int64_t *bytes);
int qg_kv_extend(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
                 int32_t *lens, int32_t *refs, const int32_t *add, int32_t *granted, int32_t *starts, int32_t *seqs,
                 int32_t *positions, int64_t slots, void *workspace, int64_t workspace_bytes, void *stream);

/* Trim, the way back: a row r with 0 <= to[r] < lens[r] (int32 [table_rows] on the device) keeps its first to[r]
 * tokens; its entries past their pages give up their page (refs - 1) and become -1. Other rows stay as they
 * are. A last page that is then partly filled and held by other rows too is not copied (qg_kv_extend refuses to
 * add to it). table_rows is at most 65536. */
int qg_kv_trim(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *to, void *stream);

/* ---- norm and rotation of queries and keys ---------------------------------------------------
 * Between the projections and the attention, a head x of D = head_dim elements becomes
 *   y = x / sqrt(mean(x^2) + eps) * w     with q_weight for queries and k_weight for keys (fp16 [D],
 *                                         16-byte aligned), or y = x where that is NULL; then
 *   (y_i, y_k) -> factor * (y_i cos t - y_k sin t, y_k cos t + y_i sin t),  t = position * freqs[j]
 * for the pairs j < rotary_dim / 2: (i, k) = (j, j + rotary_dim / 2), or (2 j, 2 j + 1) with interleaved
 * != 0. Elements from rotary_dim on are not rotated. freqs, fp64 [rotary_dim / 2] on the device (8-byte
 * aligned), are radians a token: qg_rope_freqs makes them, scaled for long contexts if need be, and factor (1 where
 * nothing is to be changed) is the factor of the attention's logits that goes with some scalings. The angle, its
 * cosine and sine are fp64 and right at any position, the rest is fp32 with one rounding to fp16. rotary_dim is a multiple of 16,
 * at most head_dim; head_dim is 64, 128 or 256; eps is at least the smallest normal fp32 (read where there is
 * a weight), factor finite, else QG_ERR_RANGE. */
typedef struct qg_rotary {
  const double *freqs;
  const uint16_t *q_weight;
  const uint16_t *k_weight;
  float eps;
  float factor;
  int32_t rotary_dim;
  int32_t interleaved;
} qg_rotary;

/* Frequencies (host): freqs[j], j < rotary_dim / 2, for the given base (10000 by habit), with f_j = base^(-2 j /
 * rotary_dim) and t_j = context * f_j / (2 pi), the turns of pair j in the `context` tokens of training:
 *   QG_ROPE_PLAIN   f_j
 *   QG_ROPE_LINEAR  f_j / scale: all positions closer together
 *   QG_ROPE_BASE    f_j of the base base * scale^(rotary_dim / (rotary_dim - 2)): the slowest pair
 *                   `scale` times slower, the fastest as it was
 *   QG_ROPE_TURNS   f_j (g + (1 - g) / scale), g = clamp((t_j - low) / (high - low), 0, 1): pairs of less than
 *                   `low` turns in training slowed, of more than `high` as they were
 *   QG_ROPE_PARTS   the same with 1 - g = clamp((j - a) / (b - a), 0, 1), a and b the pairs (as real numbers, rounded
 *                   down and up, at least 0 and at most rotary_dim - 1) that make `high` and `low` turns; b - a at least 0.001
 * scale is read by all but QG_ROPE_PLAIN, context, low and high by the last two; base > 1, scale > 0, context > 0 and
 * 0 < low < high, all finite, as are the raised base and the frequencies, else QG_ERR_RANGE. rotary_dim is a positive even number, above 2 for QG_ROPE_BASE.
 * Errors: QG_ERR_NULL, QG_ERR_FORMAT (kind), QG_ERR_SHAPE, QG_ERR_RANGE. */
typedef enum qg_rope_kind { QG_ROPE_PLAIN = 0, QG_ROPE_LINEAR = 1, QG_ROPE_BASE = 2, QG_ROPE_TURNS = 3, QG_ROPE_PARTS = 4 } qg_rope_kind;
int qg_rope_freqs(int kind, int64_t rotary_dim, double base, double scale, double context, double low, double high,
                  double *freqs);

/* Queries [count][heads * head_dim] and keys [count][kv_heads * head_dim] (fp16, rows at q + i * ldq and k + i *
 * ldk) into q_out and k_out, row i at positions[i] (int32 [count] on the device). A row with a position below 0
 * is skipped: its output stays as it was. q_out may be q with the same leading dimension, and k_out k; else outputs
 * overlap nothing that the call reads. All rows 16-byte aligned, leading dimensions multiples of 8 and at least
 * the row's elements when count > 1. heads or kv_heads may be 0 (its pointers are not read then); both are at
 * most 65536, count is at most 2^23. Errors: QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_RANGE, QG_ERR_LAUNCH. */
int qg_qk_rope(const qg_rotary *rotary, int64_t head_dim, int64_t heads, int64_t kv_heads, const uint16_t *q, int64_t ldq,
               const uint16_t *k, int64_t ldk, const int32_t *positions, int64_t count, uint16_t *q_out, int64_t ld_q_out,
               uint16_t *k_out, int64_t ld_k_out, void *stream);

/* qg_qk_rope and qg_kv_append in one pass: the queries into q_out, the keys (rounded to fp16) and the values v into
 * `layer` of the pool: for fp16 pages the same bytes as by the two calls; for int8 pages keys are computed in fp64 and
 * rounded to fp32, then to fp16, which in one of some 10000 elements is the other way than qg_qk_rope's, and in one of 16384
 * than one rounding. A row with a position below 0 is skipped, one whose
 * place is no page (see qg_kv_append) gives its queries only. What is cached, rotated keys among it, is finite.
 * heads may be 0. q_out may be q as above, and overlaps nothing else that the call reads. Sizes and alignment of
 * qg_qk_rope for q and q_out, of qg_kv_append for k and v; errors of both. */
int qg_kv_append_rope(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                      int64_t table_pages, const qg_rotary *rotary, int64_t heads, const uint16_t *q, int64_t ldq,
                      const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int32_t *seqs,
                      const int32_t *positions, int64_t count, uint16_t *q_out, int64_t ld_q_out, void *stream);

/* ---- decode to memory (device; for verification, not for inference) ----------------------
 * Writes W_hat as fp32 [n][k] to w_out (if non-NULL) and the integer codes as uint8 [n][k]
 * to codes_out (if non-NULL; q4g32 writes the unsigned nibble u = q + 8, q4a32 the code c).
 * fp32 values are single-rounding products (q*scale, (c - z)*s, d*sc*(c - o),
 * fma(d*sc, c, -dmin*m), fma(s, c, m)), hence exactly fp32(W_hat). */
int dequantize_q4g32(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q2sb(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q3sb(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q5sb(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q6sb(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q4g16(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q4g64(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q4g128(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q4a32(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q4g32h(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q2sb_bf16(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q3sb_bf16(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q5sb_bf16(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q6sb_bf16(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q3g32(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q5g32(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int dequantize_q3sb_planes(const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);
int qg_dequantize(int fmt, const void *w, float *w_out, uint8_t *codes_out, int64_t n, int64_t k, void *stream);

/* ---- measurement (device) -----------------------------------------------------------------
 * Streams `bytes` bytes (a multiple of 16; buf 16-byte aligned) through non-temporal 128-bit
 * loads (a grid-stride loop, four loads in flight per thread) and writes nothing except, with
 * negligible probability, one word of `sink`: the achievable HBM
 * read rate the GEMV kernels are measured against (the DBHOO-CIM page, section 5.3,
 * measures the machine's ceiling with STREAM first). */
int qg_read_probe(const void *buf, int64_t bytes, uint32_t *sink, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H */
