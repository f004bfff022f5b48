/*
 * nvfp4mi_layer.h - C ABI of libnvfp4mi_layer.so: what stands around the packed
 * products of nvfp4mi.h in a layer whose tokens each choose their own matrices.
 * Tokens sorted by expert and back with the gradient, the expert layer for any
 * number of tokens, and low-rank adapters beside a W4A16 projection.
 *
 * A library of its own, linked to libnvfp4mi.so, whose functions stay the ones
 * that nvfp4mi.h lists.  The conventions are those of nvfp4mi.h: device pointers
 * owned by the caller, bf16 as uint16_t bit patterns, row strides ("ld") in
 * elements, caller-provided workspaces and no device memory of its own, all work
 * enqueued on `stream`, arguments validated before any HIP call, status codes of
 * enum nvfp4_status (text from nvfp4_status_string).  Results are the same bits on
 * every call.  Calls (or replays of captured ones) that overlap in time need a
 * workspace each.
 */
#ifndef NVFP4MI_LAYER_H
#define NVFP4MI_LAYER_H

#include "nvfp4mi.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Tokens sorted by expert.  A choice is a token and one of its top_k places, c =
 * token * top_k + place; the sorted rows are the choices whose id lies in 0 ..
 * experts-1, by expert, then by choice:
 *   order[row] = choice           (-1 behind the last row)
 *   place[choice] = row           (-1 for a choice whose id names no expert: a place
 *                                 the router left empty, an expert elsewhere)
 *   offsets[e] = first row of expert e, offsets[experts] = number of rows.
 *
 * ids     [tokens][top_k] int32 (from nvfp4_moe_route).
 * order   [tokens * top_k] int32 out;  place [tokens][top_k] int32 out;
 * offsets [experts + 1] int32 out.
 * top_k 1 .. 16, experts 1 .. 1024, tokens * top_k at most 2^30.  With no tokens
 * the offsets are zeros.
 * workspace  4-byte aligned, at least nvfp4_moe_sort_workspace_bytes(tokens, top_k,
 *            experts) bytes (0 for few tokens: workspace may then be NULL).
 * Errors: NULL_ARG, BAD_SHAPE (tokens), BAD_INPUT (top_k, experts), MISALIGNED
 *         (4 bytes), WORKSPACE, HIP.
 */
NVFP4_CHECKED size_t nvfp4_moe_sort_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts);
NVFP4_CHECKED int nvfp4_moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts,
                                 int32_t* order, int32_t* place, int32_t* offsets, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * Rows of any type to their sorted rows: xs[place[t][s]] = x[t], bytes as they
 * are.  Rows of xs to which no choice goes (those behind the last) are left as
 * they were; a place outside 0 .. tokens*top_k-1 gets nothing.
 *
 * x   [tokens] rows of row_bytes bytes, ldx_bytes apart; any alignment (16 bytes
 *     of rows and strides are the quick case).
 * xs  [tokens * top_k] rows, ldxs_bytes apart.  place as nvfp4_moe_sort leaves it
 *     (no row twice).
 * Errors: NULL_ARG, BAD_SHAPE (tokens, row_bytes < 1, ld < row_bytes), BAD_INPUT
 *         (top_k), MISALIGNED (place: 4 bytes), HIP.
 */
NVFP4_CHECKED int nvfp4_moe_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ldx_bytes,
                                     const int32_t* place, int64_t top_k, void* xs, int64_t ldxs_bytes,
                                     void* stream);

/*
 * The way back: y[t] = RN_bf16( sum over s of weights[t][s] ys[place[t][s]] ), s
 * ascending, in fp32.  Places outside 0 .. tokens*top_k-1 add nothing, whatever
 * their weight; a token without any gets zeros.  weights NULL: all 1, which is the
 * gradient of nvfp4_moe_dispatch (dx from the rows' gradients).
 *
 * ys [tokens * top_k][ldys] bf16, y [tokens][ldy] bf16, columns 0..cols-1, cols a
 * multiple of 8, rows 16-byte aligned.  weights [tokens][top_k] float.
 * Errors: NULL_ARG, BAD_SHAPE, BAD_INPUT (top_k), MISALIGNED, HIP.
 */
NVFP4_CHECKED int nvfp4_moe_combine(const uint16_t* ys, int64_t ldys, const int32_t* place, const float* weights,
                                    int64_t tokens, int64_t top_k, int64_t cols, uint16_t* y, int64_t ldy,
                                    void* stream);

/*
 * The gradient of nvfp4_moe_combine: for dy = dL/dy,
 *   dys[place[t][s]]  = RN_bf16( weights[t][s] dy[t] )
 *   dweights[t][s]    = sum over columns of dy[t] ys[place[t][s]], in fp32
 * Rows of dys to which no choice goes are left as they were; dweights of a place
 * outside 0 .. tokens*top_k-1 is 0.
 *
 * dy [tokens][lddy], ys [tokens * top_k][ldys], dys [tokens * top_k][lddys] (no
 * memory of dy or ys): bf16, as in nvfp4_moe_combine.  place: no row twice.
 * dweights [tokens][top_k] float.
 * Errors: as nvfp4_moe_combine.
 */
NVFP4_CHECKED int nvfp4_moe_combine_grad(const uint16_t* dy, int64_t lddy, const uint16_t* ys, int64_t ldys,
                                         const int32_t* place, const float* weights, int64_t tokens, int64_t top_k,
                                         int64_t cols, uint16_t* dys, int64_t lddys, float* dweights, void* stream);

/*
 * nvfp4_moe_forward for any number of tokens: the same layer and arguments,
 *   y[t] = RN_bf16( sum_s weights[t][s] W2_e ( silu(W1_e x[t]) * (W3_e x[t]) ) ).
 * Up to 64 tokens it is that function's streaming kernels; beyond, the tokens are
 * sorted by expert.  Sums are in fp32 (that over s ascending); before y, silu(..)*(..)
 * and an expert's row, weight included, are each rounded to fp16 with a power of two
 * for every 32 columns (11 bits, where y has 8).  x and silu(..)*(..) enter the products
 * as fp16 with a power of two for each token (and expert), which is exact but for
 * values 2^29 and more below the largest of its row (x is off by 2^-39 of that at most,
 * silu(..)*(..), which is rounded before, by 2^-38).  An id outside 0..experts-1 adds
 * nothing; a token without any gets zeros; an expert that a token names twice counts
 * twice.
 *
 * Arguments as nvfp4_moe_forward (rows of x and y 16-byte aligned); tokens * top_k
 * at most 2^30; hidden and inter multiples of 16, at most 2^17, their product below
 * 2^31.
 * workspace  256-byte aligned, at least nvfp4_moe_forward_sorted_workspace_bytes(...)
 *            bytes (more than 131072 choices go pass by pass, which bounds it).
 * Errors: NULL_ARG, BAD_SHAPE, BAD_INPUT (top_k, experts), MISALIGNED, WORKSPACE,
 *         HIP.
 */
NVFP4_CHECKED size_t nvfp4_moe_forward_sorted_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts,
                                                              int64_t hidden, int64_t inter);
NVFP4_CHECKED int nvfp4_moe_forward_sorted(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx,
                                           const int32_t* ids, const float* weights, int64_t top_k, int64_t experts,
                                           int64_t inter, const uint8_t* w13_packed, const uint8_t* w13_codes,
                                           const float* w13_scale2, const uint8_t* w2_packed,
                                           const uint8_t* w2_codes, const float* w2_scale2, uint16_t* y,
                                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nvfp4_matmul_w4a16 with a low-rank adapter for each token, of many resident at
 * once (a = adapter_ids[t]; outside 0 .. adapters-1: none):
 *   y[t][o] = RN_bf16( w_scale2 sum_k x[t][k] v[o][k]
 *                      + scale[a] sum_r ( sum_k x[t][k] A_a[r][k] ) B_a[o][r] ),
 * v the exact NVFP4 value; everything in fp32 up to the rounding.  Tokens may name
 * their adapters in any order; runs of one adapter (prompts) are the quick case.
 * An infinity or NaN in an adapter reaches its own tokens alone.
 *
 * lora_a  [adapters][rank][k] bf16, lora_b [adapters][out_features][rank] bf16,
 *         contiguous, 16-byte aligned;  lora_scale float[adapters].
 * adapter_ids [tokens] int32.  rank: a multiple of 8, 8 .. 256;  adapters >= 0
 * (0: lora_a, lora_b and lora_scale may be NULL), at most 2^31 - 1.
 * The others as nvfp4_matmul_w4a16; workspace 16-byte aligned, at least
 * nvfp4_matmul_w4a16_lora_workspace_bytes(tokens, out_features, k, rank) bytes.
 * Errors: as nvfp4_matmul_w4a16, plus BAD_INPUT (rank, adapters).
 */
NVFP4_CHECKED size_t nvfp4_matmul_w4a16_lora_workspace_bytes(int64_t tokens, int64_t out_features, int64_t k,
                                                             int64_t rank);
NVFP4_CHECKED int nvfp4_matmul_w4a16_lora(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx,
                                          const uint8_t* w_packed, const uint8_t* w_codes, const float* w_scale2,
                                          int64_t out_features, const int32_t* adapter_ids, int64_t adapters,
                                          int64_t rank, const uint16_t* lora_a, const uint16_t* lora_b,
                                          const float* lora_scale, uint16_t* y, int64_t ldy, void* workspace,
                                          size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4MI_LAYER_H */
