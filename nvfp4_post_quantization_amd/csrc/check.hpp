// Argument checks that the entry points share.
#pragma once
#include "common.hpp"

namespace nvfp4 {

// a * b <= INT64_MAX for non-negative a, b
inline bool mul_fits(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }

// [rows][ld] matrix of `elem` bytes with `cols` used columns.
inline int check_matrix(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  if (rows < 0 || cols <= 0 || ld < cols) return NVFP4_ERR_BAD_SHAPE;
  if (!mul_fits(rows, ld) || !mul_fits(rows * ld, elem)) return NVFP4_ERR_BAD_SHAPE;
  return NVFP4_OK;
}

inline int check_bf16_rows(const void* p, int64_t ld) {
  if (!aligned16(p) || (ld % 8) != 0) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Sizes of a product: rows and columns are indexed with 32 bits, up to the end
// of the last tile (256 tokens; 16 output rows, since the tiles that have more
// are not used where they would pass 2^31), and 16 rows of packed channels have
// 32-bit offsets.
constexpr int64_t kMaxChannels = INT64_C(1) << 26;
inline int check_product(int64_t tokens, int64_t out, int64_t k, int64_t block, int64_t ldy) {
  if (tokens < 0 || out <= 0 || k <= 0 || k % block || ldy < out) return NVFP4_ERR_BAD_SHAPE;
  if (tokens > INT32_MAX - 255 || out > INT32_MAX - 15 || k > kMaxChannels) return NVFP4_ERR_BAD_SHAPE;
  return check_matrix(tokens, out, ldy, 2);
}

inline int check_workspace(const void* workspace, size_t have, size_t need) {
  if (have < need) return NVFP4_ERR_WORKSPACE;
  if (need && !workspace) return NVFP4_ERR_NULL_ARG;
  return need && !aligned16(workspace) ? NVFP4_ERR_MISALIGNED : NVFP4_OK;
}

}  // namespace nvfp4
