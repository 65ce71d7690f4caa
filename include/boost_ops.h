/*
 * boost_ops.h -- C ABI of the layer's operators around the bottleneck block
 * (boost_block.h): rotary positions of q and k, dropout of a residual branch, the 8-bit
 * floating-point quantiser and matrix product, attention and its gradients, the norm with an
 * 8-bit output, and gradient clipping.
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

/* ------------------------------------------------------------------- attention
 *
 * The layer's attention core over packed sequences:
 *     s_ij = scale q_i . k_j     for the keys j that query i sees
 *     out_i = sum_j exp(s_ij - lse_i) v_j,     lse_i = ln sum_j exp(s_ij)
 * Sequence s has the queries [q_starts[s], q_starts[s + 1]) and the keys [k_starts[s],
 * k_starts[s + 1]); with `causal` its last query sees all its keys, the one before all but the
 * last, and so on, so that new tokens can follow a context, and queries beyond the number of
 * keys, the first ones, see none: their out and gradients are 0, their lse is -infinity. Query
 * head h reads key head h / (hq / hk). Products of bf16 values, sums and the softmax's
 * statistics in fp32; the probabilities and their gradients are rounded to bf16 as the operands
 * of the second products. The backward of a call of few scores (at most 2^18 of all heads, in up to
 * 32 sequences whose rows bound them by 2^24) takes both as two bf16 operands, 2^-16 off in place
 * of 2^-8; so the last bits of a sequence's gradients depend on what else is in the call, as those
 * of its out do on how its keys are cut into parts. Scores and their magnitudes' sums stay within
 * fp32's range (below 2^127): beyond it out, lse and the gradients are not defined.
 *
 *   Tq, Tk    rows of q and of k and v, >= 0
 *   hq, hk    query and key heads, hq a multiple of hk
 *   dim       values per head, a multiple of 8, <= 128
 *   sequences >= 1
 *   causal    0 or 1
 *   scale     > 0, at most 2^127
 *   q_ts, q_hs, ...  token and head strides in elements, multiples of 8, positive where there is
 *             more than one token or head. In an output no two elements may coincide.
 * The strides of dout, dq, dk and dv are the backward's alone.
 */
#define BOOST_ATTENTION_MAX_DIM 128

typedef struct {
    int64_t Tq, Tk;
    int32_t hq, hk, dim, sequences, causal;
    float scale;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    int64_t do_ts, do_hs, dq_ts, dq_hs, dk_ts, dk_hs, dv_ts, dv_hs;
} boost_attention_desc;

/* Bytes of the workspace of either call (0 for a desc that the calls refuse). */
size_t boost_attention_workspace_bytes(const boost_attention_desc* desc);

/*
 *   q, k, v    [T, heads, dim] (strides in the desc)
 *   q_starts, k_starts   device int32 [sequences + 1], ascending, from 0 to at most Tq (Tk).
 *              Either may be NULL with one sequence: then it holds all rows. Rows behind the last
 *              sequence are not read as its keys, and left as they were in the outputs. (Values
 *              outside of 0..T are taken as its bounds; what sequences that overlap give is not
 *              defined.)
 *   out        out; shares no element with an input, but may lie between their heads in one
 *              packed buffer
 *   lse        out, [hq, Tq] fp32, or NULL
 *   ws         workspace, 256-byte aligned, error word cleared by boost_block_ws_init. Calls that
 *              may run at the same time need one each.
 * A NaN or an infinity in k or v may reach every row of its own sequence, and no other's.
 */
boost_status boost_attention(const boost_attention_desc* desc, const void* q, const void* k,
                             const void* v, const int32_t* q_starts, const int32_t* k_starts,
                             void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * Gradients of q, k and v from dout, the gradient of out; out and lse are the forward's. The
 * probabilities are regenerated from q, k and lse. Sums over the query heads that share a key
 * head are in fp32 too, and every sum is taken in a fixed order: two calls give the same bits.
 */
boost_status boost_attention_bwd(const boost_attention_desc* desc, const void* q, const void* k,
                                 const void* v, const void* out, const float* lse,
                                 const void* dout, const int32_t* q_starts,
                                 const int32_t* k_starts, void* dq, void* dk, void* dv, void* ws,
                                 size_t ws_bytes, void* stream);

/* ----------------------------------------------- norm with an 8-bit output
 *
 * The residual's addition and the statistics of the root-mean-square norm behind it, with the
 * sum quantised for the 8-bit product that follows:
 *     h = x + residual (bf16)          rstd[t] = (mean_j h[t][j]^2 + eps)^-1/2
 *     q, sf = 8-bit operand of h, or of bf16(gamma[j] h[t][j]), rows alone (block_rows 1)
 * as boost_fp8_quantize gives it; squares and their sums in fp32. The norm's value is q's times rstd of its row, which the product
 * applies (row_scale). Its gradient is the normed block's (boost_block_bwd).
 *   T, d       d a multiple of 8
 *   fmt        boost_fp8
 *   residual   [T, d] or NULL
 *   gamma      [d] or NULL
 *   h          out, [T, d], or NULL; may be x or residual
 *   rstd       out, [T] fp32
 *   q, sf      out, [T, d rounded up to 16] with zeros behind the columns, and its scales
 */
boost_status boost_norm_quantize(int64_t T, int64_t d, int32_t fmt, float eps, const void* x,
                                 const void* residual, const void* gamma, void* h, float* rstd,
                                 void* q, void* sf, void* stream);

/* --------------------------------------------------------- gradient clipping
 *
 *     norm = sqrt(sum over all tensors of g^2),     out = g min(1, max_norm / (norm + 1e-6))
 * Squares in fp32, where that holds them, their sums in fp64 in a fixed order: two calls give the
 * same bits, and gradients of any size count. Gradients that hold an infinity or NaN give what the
 * formula gives, with any max_norm (all NaN where there is a NaN; 0, and NaN from an infinity).
 *   count      tensors, >= 0
 *   g          16-byte aligned
 *   out        may be g (then nothing is written where nothing is to be scaled); NULL: the tensor
 *              only counts in the norm. Otherwise it shares no byte with any tensor of the call.
 *   n          elements, >= 0
 *   wide       0: bf16, 1: fp32
 *   max_norm   >= 0; infinity: no scaling of finite gradients
 *   norm       out, fp32 [1] (infinity beyond fp32's range; what scales is its fp64 value)
 *   ws         workspace of boost_grad_clip_workspace_bytes() bytes, 256-byte aligned. Calls that
 *              may run at the same time need one each.
 */
typedef struct {
    const void* g;
    void* out;
    int64_t n;
    int32_t wide;
} boost_grad;

size_t boost_grad_clip_workspace_bytes(void);

boost_status boost_grad_clip(int64_t count, const boost_grad* grads, double max_norm, float* norm,
                             void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BOOST_OPS_H */
