/*
 * gemm_mx.h -- C ABI of the 4-bit microscaled (MXFP4) operators of the
 * gemm_f32 library (MI355X, gfx950): quantisation, its inverse, the product
 * of two MX matrices, and the product of 16-bit rows with an MX matrix.
 *
 * An MX matrix has `rows` rows of K values each, in blocks of 32 along K
 * (the published OCP microscaling format with E2M1 elements and E8M0 scales):
 *
 *   value(r, k) = e2m1(code(r, k)) * 2^(scale(r, k / 32) - 127)
 *
 *   codes   4 bits each, sign and magnitude {0, 0.5, 1, 1.5, 2, 3, 4, 6};
 *           row r starts at codes + r * ld; value k is in byte k / 2, the
 *           lower four bits for even k.  A row holds whole blocks:
 *           gemm_mx_code_bytes(K) = 16 ceil(K / 32) bytes; codes past K in
 *           the last block must be 0 (gemm_mx_quantize writes them so).
 *   scales  one byte per block, row r at scales + r * lds; byte 255 makes
 *           every value of its block NaN.  A row holds whole 16-byte groups:
 *           gemm_mx_scale_bytes(K) = 16 ceil(K / 512) bytes, of which those
 *           past the last block may be read but have no effect
 *           (gemm_mx_quantize writes 0).
 *
 * `ld` and `lds` are in bytes, at least those sizes (and at least 16), and
 * multiples of 16; `codes` and `scales` are 16-byte aligned.  The products
 * take the right operand by its columns, B[k][j] = value(j, k): both
 * operands' blocks run along the shared dimension.
 *
 * Memory, streams and errors are as for gemm_f32 (gemm_f32.h): device
 * pointers owned by the caller, nothing allocated, asynchronous on `stream`
 * (hipStream_t as void*, NULL = null stream), argument errors returned
 * before anything is enqueued, status codes GEMM_F32_*.  Outputs must not
 * overlap inputs.  Results do not depend on timing: each output element is
 * summed in one fixed order.
 */
#ifndef GEMM_MX_H
#define GEMM_MX_H

#ifdef __cplusplus
extern "C" {
#endif

/* Formats of unquantised matrices: GEMM_MIXED_BF16 (0) and GEMM_MIXED_F16 (1)
 * of gemm_mixed.h, and fp32. */
#define GEMM_MX_F32 2

/* Which way blocks run through a row-major unquantised matrix X.
 * GEMM_MX_ROWS: X is rows x K, X[r * ldx + k] (a product's left operand).
 * GEMM_MX_COLUMNS: X is K x rows, X[k * ldx + r] (a product's right operand:
 * MX row r is column r of X). */
#define GEMM_MX_ROWS 0
#define GEMM_MX_COLUMNS 1

/* Bytes of one row of codes and of scales. */
long long gemm_mx_code_bytes(int K);
long long gemm_mx_scale_bytes(int K);

/*
 * gemm_mx_quantize -- X to MX.  For each block with largest magnitude m:
 * e = floor(log2 m) - 2, clamped to [-127, 127] (m = 0: -127); the scale byte
 * is e + 127 and each code the nearest element to x / 2^e, ties to the even
 * code, magnitudes above 6 to 6.  A block that holds an infinity or a NaN
 * gets scale byte 255 and codes 0.
 *   rows, K   >= 0; rows == 0 or K == 0: no-op.
 *   X, ldx    in `format`, element-aligned; ldx in elements, >= max(1, K)
 *             (GEMM_MX_ROWS) or >= max(1, rows) (GEMM_MX_COLUMNS).
 *   along     GEMM_MX_ROWS or GEMM_MX_COLUMNS.
 * Writes every byte of the rows' whole blocks and whole scale groups, and
 * nothing else.
 */
int gemm_mx_quantize(int rows, int K, const void *X, int ldx, int format, int along,
                     unsigned char *codes, int ld, unsigned char *scales, int lds,
                     void *stream);

/*
 * gemm_mx_dequantize -- MX to Y, laid out as X above.  A value outside the
 * format's range becomes an infinity or is rounded to nearest even there.
 */
int gemm_mx_dequantize(int rows, int K, const unsigned char *codes, int ld,
                       const unsigned char *scales, int lds, void *Y, int ldy, int format,
                       int along, void *stream);

/*
 * gemm_mx -- C[i][j] = sum_{k<K} A(i, k) B(j, k) with both operands MX,
 * accumulated in fp32 and rounded once to `c_format`.
 *   M, N, K   each >= 0.  M == 0 or N == 0: no-op.  K == 0: C is set to 0.
 *   A, B      codes (M and N rows); SA, SB their scales.
 *   C, ldc    M x N row-major in `c_format`, element-aligned, ldc in elements.
 *   config    -1 picks a launch-table entry for the shape, otherwise an index
 *             below gemm_mx_num_configs() (else GEMM_F32_BAD_CONFIG); an
 *             entry that the sizes or pitches do not fit runs entry 0.
 * Products of two elements and their block sums are formed by the scaled
 * matrix instruction, v_mfma_scale_f32_16x16x128_f8f6f4.
 */
int gemm_mx(int M, int N, int K, const unsigned char *A, int lda, const unsigned char *SA,
            int ldsa, const unsigned char *B, int ldb, const unsigned char *SB, int ldsb,
            void *C, int ldc, int c_format, int config, void *stream);

/* Number of launch-table entries of gemm_mx, and the entry it would use (host
 * only): workgroup tile BM x BN, k step BK, threads and the entry index.  Any
 * output pointer may be NULL. */
int gemm_mx_num_configs(void);
int gemm_mx_tile(int config, int M, int N, int K, int *BM, int *BN, int *BK, int *threads,
                 int *chosen_config);

/*
 * gemm_mx_a16 -- C[i][j] = sum_{k<K} A[i][k] B(j, k) with A in 16 bits
 * (row-major M x K in `a_format`, 2-byte aligned, lda in elements) and B MX:
 * weights in 4 bits, activations as they are.  Every A value and every value of
 * B enters exactly.  Made for few rows (up to 32 read B once, up to 64 where N and
 * K are large; blocks of rows past that read it again, from cache where it holds
 * it); any M is served.
 */
int gemm_mx_a16(int M, int N, int K, const void *A, int lda, int a_format,
                const unsigned char *B, int ldb, const unsigned char *SB, int ldsb, void *C,
                int ldc, int c_format, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MX_H */
