// C ABI entry points of libnvfp4mi_layer.so (include/nvfp4mi_layer.h): argument
// validation on the host, then the launches.  No HIP call happens before
// validation succeeds.
#include "check.hpp"
#include "layer.hpp"

using namespace nvfp4;

// tokens and their places; `rows` gets their product
static int check_choices(int64_t tokens, int64_t top_k, int64_t& rows) {
  if (top_k < 1 || top_k > kMoeMaxTopK) return NVFP4_ERR_BAD_INPUT;
  if (tokens < 0 || tokens > kMaxChoices / top_k) return NVFP4_ERR_BAD_SHAPE;
  rows = tokens * top_k;
  return NVFP4_OK;
}
static int check_experts(int64_t experts) {
  return experts < 1 || experts > kMoeMaxExperts ? NVFP4_ERR_BAD_INPUT : NVFP4_OK;
}
static bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

extern "C" {

size_t nvfp4_moe_sort_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
  int64_t rows;
  if (check_choices(tokens, top_k, rows) || check_experts(experts)) return 0;
  return moe_sort_workspace_bytes(rows, experts);
}

int nvfp4_moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int32_t* order, int32_t* place,
                   int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t rows;
  int st = check_choices(tokens, top_k, rows);
  if (st || (st = check_experts(experts))) return st;
  if (!offsets || ((!ids || !order || !place) && tokens > 0)) return NVFP4_ERR_NULL_ARG;
  if (!aligned4(ids) || !aligned4(order) || !aligned4(place) || !aligned4(offsets)) return NVFP4_ERR_MISALIGNED;
  const size_t need = moe_sort_workspace_bytes(rows, experts);
  if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (need && !workspace) return NVFP4_ERR_NULL_ARG;
  if (need && !aligned4(workspace)) return NVFP4_ERR_MISALIGNED;
  return launch_moe_sort(ids, rows, experts, order, place, offsets, workspace, BandList{},
                         as_stream(stream));
}

int nvfp4_moe_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ldx_bytes, const int32_t* place,
                       int64_t top_k, void* xs, int64_t ldxs_bytes, void* stream) {
  int64_t rows;
  int st = check_choices(tokens, top_k, rows);
  if (st || (st = check_matrix(tokens, row_bytes, ldx_bytes, 1)) || (st = check_matrix(rows, row_bytes, ldxs_bytes, 1)))
    return st;
  if ((!x || !place || !xs) && tokens > 0) return NVFP4_ERR_NULL_ARG;
  if (tokens == 0) return NVFP4_OK;
  if (!aligned4(place)) return NVFP4_ERR_MISALIGNED;
  return launch_moe_dispatch(x, tokens, row_bytes, ldx_bytes, place, (int)top_k, xs, ldxs_bytes, as_stream(stream));
}

int nvfp4_moe_combine(const uint16_t* ys, int64_t ldys, const int32_t* place, const float* weights, int64_t tokens,
                      int64_t top_k, int64_t cols, uint16_t* y, int64_t ldy, void* stream) {
  int64_t rows;
  int st = check_choices(tokens, top_k, rows);
  if (st || (st = check_matrix(rows, cols, ldys, 2)) || (st = check_matrix(tokens, cols, ldy, 2))) return st;
  if (cols % 8) return NVFP4_ERR_BAD_SHAPE;
  if ((!ys || !place || !y) && tokens > 0) return NVFP4_ERR_NULL_ARG;
  if (tokens == 0) return NVFP4_OK;
  if ((st = check_bf16_rows(ys, ldys)) || (st = check_bf16_rows(y, ldy))) return st;
  if (!aligned4(place) || !aligned4(weights)) return NVFP4_ERR_MISALIGNED;
  return launch_moe_combine(ys, ldys, place, weights, tokens, (int)top_k, cols, y, ldy, as_stream(stream));
}

int nvfp4_moe_combine_grad(const uint16_t* dy, int64_t lddy, const uint16_t* ys, int64_t ldys, const int32_t* place,
                           const float* weights, int64_t tokens, int64_t top_k, int64_t cols, uint16_t* dys,
                           int64_t lddys, float* dweights, void* stream) {
  int64_t rows;
  int st = check_choices(tokens, top_k, rows);
  if (st || (st = check_matrix(tokens, cols, lddy, 2)) || (st = check_matrix(rows, cols, ldys, 2)) ||
      (st = check_matrix(rows, cols, lddys, 2)))
    return st;
  if (cols % 8) return NVFP4_ERR_BAD_SHAPE;
  if ((!dy || !ys || !place || !weights || !dys || !dweights) && tokens > 0) return NVFP4_ERR_NULL_ARG;
  if (tokens == 0) return NVFP4_OK;
  if ((st = check_bf16_rows(dy, lddy)) || (st = check_bf16_rows(ys, ldys)) || (st = check_bf16_rows(dys, lddys))) return st;
  if (!aligned4(place) || !aligned4(weights) || !aligned4(dweights)) return NVFP4_ERR_MISALIGNED;
  return launch_moe_combine_grad(dy, lddy, ys, ldys, place, weights, tokens, (int)top_k, cols, dys, lddys, dweights,
                                 as_stream(stream));
}

// Output rows and channels of an expert: its tiles, the launches over them and the
// offsets within it stay below 2^31.
static int check_expert_sizes(int64_t hidden, int64_t inter) {
  constexpr int64_t most = INT64_C(1) << 17;
  if (hidden <= 0 || inter <= 0 || hidden % 16 || inter % 16 || hidden > most || inter > most) return NVFP4_ERR_BAD_SHAPE;
  return hidden * inter >= INT64_C(1) << 31 ? NVFP4_ERR_BAD_SHAPE : NVFP4_OK;
}
// Up to kMoeMaxTokens tokens it is nvfp4_moe_forward's kernels and its bits: they round
// neither silu(..)*(..) nor an expert's row.  8 of 128 experts of 7168 x 2048, weights
// cold, us, with them and sorted: 1 token 94 and 136, 4 tokens 234 and 249, 16 tokens
// 505 and 520, 32 tokens 647 and 655, 48 tokens 735 and 701, 64 tokens 816 and 721.
static size_t layer_workspace(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  return tokens <= kMoeMaxTokens ? moe_workspace_bytes(tokens, top_k, inter)
                                 : moe_sorted_workspace_bytes(tokens, top_k, experts, hidden, inter);
}

size_t nvfp4_moe_forward_sorted_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden,
                                                int64_t inter) {
  int64_t rows;
  if (check_choices(tokens, top_k, rows) || check_experts(experts) || check_expert_sizes(hidden, inter) || tokens == 0)
    return 0;
  return layer_workspace(tokens, top_k, experts, hidden, inter);
}

int nvfp4_moe_forward_sorted(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx, const int32_t* ids,
                             const float* weights, int64_t top_k, int64_t experts, int64_t inter,
                             const uint8_t* w13_packed, const uint8_t* w13_codes, const float* w13_scale2,
                             const uint8_t* w2_packed, const uint8_t* w2_codes, const float* w2_scale2, uint16_t* y,
                             int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t rows;
  int st = check_choices(tokens, top_k, rows);
  if (st || (st = check_experts(experts)) || (st = check_expert_sizes(hidden, inter)) ||
      (st = check_matrix(tokens, hidden, ldx, 2)) || (st = check_matrix(tokens, hidden, ldy, 2)))
    return st;
  if (!w13_packed || !w13_codes || !w13_scale2 || !w2_packed || !w2_codes || !w2_scale2 ||
      ((!x || !ids || !weights || !y) && tokens > 0))
    return NVFP4_ERR_NULL_ARG;
  if (tokens == 0) return NVFP4_OK;
  if ((st = check_bf16_rows(x, ldx)) || (st = check_bf16_rows(y, ldy))) return st;
  if (!aligned4(ids) || !aligned4(weights) || !aligned16(w13_packed) || !aligned16(w13_codes) || !aligned4(w13_scale2) ||
      !aligned16(w2_packed) || !aligned16(w2_codes) || !aligned4(w2_scale2))
    return NVFP4_ERR_MISALIGNED;
  const size_t need = layer_workspace(tokens, top_k, experts, hidden, inter);
  if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (!workspace) return NVFP4_ERR_NULL_ARG;
  if (!aligned256(workspace)) return NVFP4_ERR_MISALIGNED;
  if (tokens <= kMoeMaxTokens)
    return launch_moe_forward(x, tokens, hidden, ldx, ids, weights, (int)top_k, experts, inter, w13_packed, w13_codes,
                              w13_scale2, w2_packed, w2_codes, w2_scale2, y, ldy, workspace, as_stream(stream));
  const ExpertWeights w{w13_packed, w13_codes, w2_packed, w2_codes, w13_scale2, w2_scale2};
  return launch_moe_sorted(x, tokens, hidden, ldx, ids, weights, (int)top_k, experts, inter, w, y, ldy, workspace,
                           as_stream(stream));
}

static int check_lora(int64_t tokens, int64_t out, int64_t k, int64_t rank, int64_t ldy) {
  const int st = check_product(tokens, out, k, 16, ldy);
  if (st) return st;
  return rank < 8 || rank > kMaxRank || rank % 8 ? NVFP4_ERR_BAD_INPUT : NVFP4_OK;
}

size_t nvfp4_matmul_w4a16_lora_workspace_bytes(int64_t tokens, int64_t out_features, int64_t k, int64_t rank) {
  if (tokens <= 0 || check_lora(tokens, out_features, k, rank, out_features)) return 0;
  return lora_workspace_bytes(tokens, out_features, k, rank);
}

int nvfp4_matmul_w4a16_lora(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx, const uint8_t* w_packed,
                            const uint8_t* w_codes, const float* w_scale2, int64_t out_features,
                            const int32_t* adapter_ids, int64_t adapters, int64_t rank, const uint16_t* lora_a,
                            const uint16_t* lora_b, const float* lora_scale, uint16_t* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int st = check_lora(tokens, out_features, k, rank, ldy);
  if (st || (st = check_matrix(tokens, k, ldx, 2))) return st;
  if (adapters < 0 || adapters > INT32_MAX) return NVFP4_ERR_BAD_INPUT;
  if (!mul_fits(adapters * rank, 2 * k) || !mul_fits(adapters * rank, 2 * out_features)) return NVFP4_ERR_BAD_SHAPE;
  if (!w_packed || !w_codes || !w_scale2 || ((!x || !adapter_ids || !y) && tokens > 0) ||
      ((!lora_a || !lora_b || !lora_scale) && adapters > 0))
    return NVFP4_ERR_NULL_ARG;
  if (tokens == 0) return NVFP4_OK;
  if ((st = check_bf16_rows(x, ldx))) return st;
  if (!aligned16(w_packed) || !aligned16(w_codes) || !aligned4(w_scale2) || !aligned4(adapter_ids) ||
      !aligned16(lora_a) || !aligned16(lora_b) || !aligned4(lora_scale) || !aligned2(y))
    return NVFP4_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, lora_workspace_bytes(tokens, out_features, k, rank)))) return st;
  const Adapters ad{adapter_ids, lora_a, lora_b, lora_scale, (int)adapters, (int)rank};
  return launch_w4a16_lora(x, tokens, k, ldx, w_packed, w_codes, w_scale2, out_features, ad, y, ldy, workspace,
                           as_stream(stream));
}

}  // extern "C"
