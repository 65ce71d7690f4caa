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
 * 2^-63 |p| turns, which begins to show behind 2^37). The inverse is the transpose of the
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
    uint8_t axis[BOOST_ROPE_MAX_DIM / 2];
} boost_rope_desc;

/*
 *   q, k        inputs (strides in the desc)
 *   positions   [axes, T] int32 or int64
 *   inv_freq    [rot / 2] fp64, radians per position (a non-finite value gives NaN)
 *   q_out, k_out  out; an output may be its own input with the same strides (in place),
 *               and slices of one packed buffer [T, heads, dim] may be given side by
 *               side. Any other overlap of an output with a tensor of the call is
 *               BOOST_ERR_INVALID_ARG.
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

#ifdef __cplusplus
}
#endif

#endif /* BOOST_OPS_H */
