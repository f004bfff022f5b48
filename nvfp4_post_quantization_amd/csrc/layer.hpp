// Launchers of libnvfp4mi_layer.so (include/nvfp4mi_layer.h): tokens sorted by
// expert and back, the expert layer for many tokens, low-rank adapters beside a
// W4A16 product.  Arguments are validated by the caller.
#pragma once
#include "common.hpp"
#include "../include/nvfp4mi_layer.h"

namespace nvfp4 {

// Choices (a token and one of its top_k places) of one call: row numbers and
// their byte offsets in int32 tables stay clear of 2^31.
constexpr int64_t kMaxChoices = INT64_C(1) << 30;

// A band of the expert layer: rows first .. first + rows - 1 are expert's.
struct ExpertBand { int expert, first, rows, unused; };
// What the sort also writes for the expert layer (bands NULL: nothing): the bands of
// up to kBandRows rows, those of more kBandUnit rows first, and by row its choice's
// weight and its token's scale.
constexpr int kBandRows = 256, kBandUnit = 32;
struct BandList {
  ExpertBand* bands;
  int* count;
  const float *weights, *scales;
  float *row_weight, *row_scale;
  int top_k;
};

size_t moe_sort_workspace_bytes(int64_t choices, int64_t experts);
int launch_moe_sort(const int32_t* ids, int64_t choices, int64_t experts, int32_t* order, int32_t* place,
                    int32_t* offsets, void* workspace, const BandList& list, hipStream_t s);
int launch_moe_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ldx, const int32_t* place, int top_k,
                        void* xs, int64_t ldxs, hipStream_t s);
int launch_moe_combine(const uint16_t* ys, int64_t ldys, const int32_t* place, const float* weights, int64_t tokens,
                       int top_k, int64_t cols, uint16_t* y, int64_t ldy, hipStream_t s);
// The same without weights of rows in fp16 with an exponent byte for every 32
// columns: value = fp16 * 2^(byte - kHalfBias).
constexpr int kHalfBias = 141;
int launch_moe_combine_half(const uint16_t* ys, const uint8_t* exponents, const int32_t* place, int64_t tokens, int top_k,
                            int64_t cols, uint16_t* y, int64_t ldy, hipStream_t s);
int launch_moe_combine_grad(const uint16_t* dy, int64_t lddy, const uint16_t* ys, int64_t ldys, const int32_t* place,
                            const float* weights, int64_t tokens, int top_k, int64_t cols, uint16_t* dys, int64_t lddys,
                            float* dweights, hipStream_t s);

struct ExpertWeights {
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
};
size_t moe_sorted_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter);
int launch_moe_sorted(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx, const int32_t* ids,
                      const float* weights, int top_k, int64_t experts, int64_t inter, const ExpertWeights& w,
                      uint16_t* y, int64_t ldy, void* workspace, hipStream_t s);

struct Adapters {
  const int32_t* ids;          // of the tokens
  const uint16_t *a, *b;       // bf16 [count][rank][k], [count][out][rank]
  const float* scale;
  int count, rank;
};
size_t lora_workspace_bytes(int64_t tokens, int64_t out, int64_t k, int64_t rank);
int launch_w4a16_lora(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx, const uint8_t* wp, const uint8_t* wc,
                      const float* ws2, int64_t out, const Adapters& ad, uint16_t* y, int64_t ldy, void* workspace,
                      hipStream_t s);

}  // namespace nvfp4
