/*
 * boost_ops.h -- C ABI of the layer's operators around the bottleneck block
 * (boost_block.h): rotary positions of q and k, dropout of a residual branch, and the
 * 8-bit floating-point quantiser and matrix product.
 *
 * The conventions of boost_block.h hold here too: row-major tensors (bf16 unless
 * stated) of the current device, 16-byte aligned pointers, caller-owned buffers,
 * asynchronous calls on `stream` that may be captured into CUDA graphs, arguments
 * checked on the host before anything is enqueued. The calls keep nothing between calls.
 */
#ifndef BOOST_OPS_H
#define BOOST_OPS_H

#include "boost_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------- rotary positions
 *
 * Pair i of a head (i < rot / 2; see `interleaved`) of token t turns by the angle
 *     phi = positions[axis[i]][t] * inv_freq[i]        (radians; -phi when inverse)
 *     (u, v) -> (u cos phi - v sin phi, v cos phi + u sin phi)
 * in fp32, rounded once to bf16. The angle is reduced to a fraction of a turn in 64-bit
 * fixed point, so it is as exact at position 2^31 as at position 1 (a position p loses
 * less than 2^-63 |p| turns at any frequency, which begins to show behind 2^37). The inverse is the transpose of the
 * rotation: it takes the gradients of the rotated q and k to those of q and k. Several
 * axes (time, height, width) turn different pairs of the same head.
 *
 *   T        tokens, >= 0
 *   hq, hk   query and key heads (hk may be 0: q alone, k and k_out NULL)
 *   dim      values per head, a multiple of 8, <= 512
 *   rot      values that turn, a multiple of 8, 0 < rot <= dim; the rest are copied
 *   axes     position axes, 1..8
 *   interleaved  0: pair i is (i, i + rot / 2); 1: pair i is (2 i, 2 i + 1)
 *   inverse  0: rotate, 1: rotate back
 *   pos64    0: positions are int32, 1: int64 (any sign)
 *   q_ts, q_hs, ...  token and head strides in elements, multiples of 8, >= 0. In an
 *            output no two elements may coincide.
 *   pos_at   where in `positions` the tokens begin, >= 0 (a decoding step takes one column
 *            of a table, whose address is aligned although the column's is not)
 *   pos_as   positions from one axis to the next, >= T; 0: T
 *   axis     [rot / 2] the axis of each pair, each < axes (the rest of the array unused)
 */
#define BOOST_ROPE_MAX_DIM 512
#define BOOST_ROPE_MAX_AXES 8

typedef struct {
    int64_t T;
    int32_t hq, hk, dim, rot;
    int32_t axes, interleaved, inverse, pos64;
    int64_t q_ts, q_hs, k_ts, k_hs;
    int64_t qo_ts, qo_hs, ko_ts, ko_hs;
    int64_t pos_at, pos_as;
    uint8_t axis[BOOST_ROPE_MAX_DIM / 2];
} boost_rope_desc;

/*
 *   q, k        inputs (strides in the desc)
 *   positions   int32 or int64, that of token t on axis a at pos_at + a pos_as + t: [axes, T]
 *               with both 0
 *   inv_freq    [rot / 2] fp64, radians per position (one that is not finite, or is 2^64 or
 *               more in magnitude, gives NaN)
 *   q_out, k_out  out; an output may be its own input with the same strides (in place),
 *               and operands may lie in one packed buffer: heads side by side in a token's
 *               row ([T, heads, dim]), or with the same strides and no element in common
 *               ([T, heads, 3, dim], [heads, 3, T, dim] and the like). Any other overlap of
 *               an output with a tensor of the call is BOOST_ERR_INVALID_ARG.
 */
boost_status boost_rope(const boost_rope_desc* desc, const void* q, const void* k,
                        const void* positions, const double* inv_freq, void* q_out, void* k_out,
                        void* stream);

/* ----------------------------------------------------------------------- dropout
 *
 *     out[e] = res[e] + (keep(e) ? x[e] * 65536 / (65536 - drop) : 0)
 *
 * over `count` elements, in fp32, rounded once. keep(e) is a pure function of e, seed and
 * offset, so the mask is regenerated wherever it is needed and never stored: element
 * e = 8 g + j is kept when 16-bit half j (low half of word 0 first) of the Philox4x32-10
 * block (Salmon, Moraes, Dror and Shaw, SC 2011) with counter (g low, g high, offset
 * low, offset high) and key (seed low, seed high) is >= drop, with
 * drop = round(65536 p): p is honoured to 2^-17, and the scale uses drop / 65536, so the
 * expectation of out is exact. A dropped value is 0 whatever x holds there (NaN included).
 *
 *   count   elements, any number >= 0; element e is that of the flattened tensor
 *   x       the branch's output
 *   res     the residual, or NULL (then out = dropout(x))
 *   out     out; may be x or res
 *   p       0 <= p < 1; a p that rounds to no drop at all (0 < p < 2^-17) or to 1 is
 *           BOOST_ERR_INVALID_ARG
 *   seed, offset   which mask: calls that share both share the mask
 *   counter device uint64, 8-byte aligned, or NULL: added to offset when the kernel runs,
 *           so that a replayed CUDA graph takes a new mask when the caller advances it
 *
 * The gradient of x is the same call on the gradient of out, with the same seed and
 * offset and without res; the gradient of res is the gradient of out.
 */
boost_status boost_dropout(int64_t count, const void* x, const void* res, void* out, double p,
                           uint64_t seed, uint64_t offset, const uint64_t* counter, void* stream);

/* ------------------------------------------------- 8-bit floating-point operands
 *
 * An operand is a matrix [rows, K] of e4m3 or e5m2 values (K contracted) with one
 * power-of-two scale for each block of 128 along K: value = q * 2^(byte - 127).
 *   values  [G, rows, pitch] bytes, pitch a multiple of 16, >= K
 *   scales  [G] planes of boost_fp8_scale_bytes(rows, K) bytes: tiles of 128 rows x 4
 *           blocks, the byte of row r, block b at
 *           ((r / 128) * ceil(blocks / 4) + b / 4) * 512 + (r % 32) * 16
 *             + (r / 32 % 4) * 4 + b % 4,        blocks = ceil(K / 128)
 *           (the layout the tensor core reads). A byte of 255 stands for NaN.
 */
typedef enum { BOOST_E4M3 = 0, BOOST_E5M2 = 1 } boost_fp8;

/* Bytes of one plane of scales (0 when rows or K is 0). */
size_t boost_fp8_scale_bytes(int64_t rows, int64_t K);

/*
 * Quantise G matrices [rows, cols] of bf16 as they lie (q: K = cols), transposed
 * (qt: [cols, rows], K = rows), or both from one reading of x: the forward product
 * contracts the columns of x, the weight gradient its rows.
 *
 * The scale of a block is the smallest power of two s >= 2^-127 with
 * max |finite x| <= s * fmax (fmax = 448 for e4m3, 57344 for e5m2), 1 for a block of
 * zeros; values are x / s rounded to nearest, ties to even. NaN stays NaN; an infinity
 * becomes NaN in e4m3, which has none, and stays in e5m2.
 *   block_rows  1: each row (of q; each column for qt) has its own scales; 128: a block is
 *               128 x 128, so q and qt hold the same values
 *   ldx, gstride  row and matrix strides of x in elements, multiples of 8
 *   rows        at most 2097120
 *   cols        a multiple of 8
 *   gamma       [rows] or NULL: x is replaced by bf16(gamma[row] * x), the fold of a
 *               norm's weight into a down-projection weight; block_rows 128 or qt only
 *   q, sf       out, or both NULL. pitch = cols rounded up to 16, zeros behind the columns
 *   qt, sft     out, or both NULL. pitch = rows rounded up to 16, zeros behind the rows
 * Scale bytes of rows and blocks outside the operand are 127.
 */
typedef struct {
    int64_t G, rows, cols, ldx, gstride;
    int32_t fmt, block_rows;
} boost_fp8_quant_desc;

boost_status boost_fp8_quantize(const boost_fp8_quant_desc* desc, const void* x,
                                const void* gamma, void* q, void* sf, void* qt, void* sft,
                                void* stream);

/*
 * out[g] = act(row_scale (.) (A[g] @ B[g]^T)), g < G, A [M, K], B [N, K], out [M, N] bf16,
 * products and sums in fp32 on the tensor cores.
 *   G, M, N, K   K >= 0 (K == 0: out = act(0) = 0); a matrix of an operand or of out is
 *                smaller than 2^40 bytes
 *   a_pitch, b_pitch   bytes between rows of the operands, multiples of 16, >= K
 *   a_fmt, b_fmt  boost_fp8
 *   act          boost_act, applied after the row scale
 *   row_scale    [M] fp32 or NULL: the deferred 1/rms of a normed block
 *   out          [G, M, N] bf16; N a multiple of 8, at most 1048560
 *   ws           workspace of boost_fp8_matmul_workspace_bytes(desc) bytes or more,
 *                256-byte aligned, error word cleared by boost_block_ws_init
 * A gradient is the same product on operands quantised the other way: for y = x W^T,
 * dx = dy W contracts the rows of W (qt of W), dW = dy^T x the tokens (qt of dy and x).
 */
typedef struct {
    int64_t G, M, N, K, a_pitch, b_pitch;
    int32_t a_fmt, b_fmt, act;
} boost_fp8_matmul_desc;

size_t boost_fp8_matmul_workspace_bytes(const boost_fp8_matmul_desc* desc);

boost_status boost_fp8_matmul(const boost_fp8_matmul_desc* desc, const void* a, const void* a_sf,
                              const void* b, const void* b_sf, const float* row_scale, void* out,
                              void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BOOST_OPS_H */
