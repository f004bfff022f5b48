// Products of packed 4-bit matrices: y[t][o] = RN_bf16(sum_k x[t][k] w[o][k])
// for W4A16 and W4A4 NVFP4 ("Coder390 NVFP4 校正（校准）方式" §3, the W4A16 and
// W4A4 tiers) and for MXFP4 on both sides.
//
// Few tokens: the weights are read once and bound the call.  A workgroup
// takes a run of 16-row tiles, as many workgroups as there are CUs; its eight
// waves split the channels, hold their part of the tokens in registers and
// stream the rows' packed weights past them from HBM, expanding them in
// registers for the matrix cores (the rows are the instruction's M side, the
// tokens its N side).  The waves' partial tiles meet in LDS and are added in
// wave order.
#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

struct ProductArgs {
  const uint8_t* xp;      // bf16 rows (kW4A16) or packed nibbles
  const uint8_t* xc;      // block scales of x, or NULL
  const float* xs2;       // tensor scale of x, or NULL
  const uint8_t* wp;
  const uint8_t* wc;
  const float* ws2;       // tensor scale of w, or NULL (MXFP4)
  int64_t ldx;            // row stride of xp in bytes
  int64_t ldy;
  uint16_t* y;
  int tokens, out, k;
};

template <int KIND>
__device__ __forceinline__ float tensor_scaled(float v, const ProductArgs& a) {
  if constexpr (KIND == kW4A16) return v * *a.ws2;
  else if constexpr (KIND == kW4A4) return (v * *a.ws2) * *a.xs2;
  else return v;
}

template <int KIND, int NT, int QW>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void few_tokens_kernel(ProductArgs a) {
  constexpr int RT = 2 / QW, TB = 4 / RT / NT;
  __shared__ f32x4 part[kStreamWaves * TB * RT * NT * 64];
  const int lane = threadIdx.x & 63, r16 = lane & 15;
  const int tiles = (a.out + 15) >> 4;
  const int begin = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  const int tok0 = blockIdx.y * 16 * NT;
  const uint32_t ldw = (uint32_t)a.k >> 1, lds = (uint32_t)a.k >> (KIND == kMX ? 5 : 4);
  TokenRows tokens[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t0 = min(tok0 + 16 * n, a.tokens - 1);             // tokens past the end are not stored
    const int t = min(r16, a.tokens - 1 - t0);
    if constexpr (KIND == kW4A16) {
      tokens[n].x = a.xp + (int64_t)(t0 + t) * a.ldx;
    } else {
      const uint32_t rows = min(16, a.tokens - t0);
      tokens[n].packed = PackedRows{a.xp + (int64_t)t0 * ldw, a.xc + (int64_t)t0 * lds, rows * ldw, rows * lds};
      tokens[n].row_w = t * ldw;
      tokens[n].row_s = t * lds;
    }
  }
  auto rows_of = [&](int t) {
    const int row = t * 16;
    const uint32_t rows = min(min(16 * RT, (end - t) * 16), a.out - row);
    return PackedRows{a.wp + (int64_t)row * ldw, a.wc + (int64_t)row * lds, rows * ldw, rows * lds};
  };
  auto done = [&](int t, int n, int l, auto sum) {
    const int row = t * 16 + 4 * (l >> 4), tok = tok0 + 16 * n + (l & 15);
    if (tok >= a.tokens || row >= a.out) return;
    const f32x4 v = sum(l);
    uint16_t* dst = a.y + (int64_t)tok * a.ldy + row;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (row + e < a.out) dst[e] = to_bf16(tensor_scaled<KIND>(v[e], a));
  };
  stream_tiles<KIND, NT, QW, TB>(begin, end, a.k, r16 * ldw, r16 * lds, 16 * ldw, 16 * lds, tokens, part, rows_of, done);
}

constexpr int kCus = 256;

template <int KIND, int NT, int QW>
int run_few(const ProductArgs& a, hipStream_t s) {
  const int tiles = (a.out + 15) / 16;
  const dim3 grid(tiles < kCus ? tiles : kCus, (a.tokens + 16 * NT - 1) / (16 * NT));
  few_tokens_kernel<KIND, NT, QW><<<grid, 64 * kStreamWaves, 0, s>>>(a);
  return launch_status("few_tokens_kernel");
}

// One quad of the tokens a wave and two row tiles at a time where that covers
// the channels, else two quads and one row tile.
template <int KIND>
int run(const ProductArgs& a, hipStream_t s) {
  const bool one = a.k <= 512 * kStreamWaves;
  if (a.tokens <= 16) return one ? run_few<KIND, 1, 1>(a, s) : run_few<KIND, 1, 2>(a, s);
  return run_few<KIND, 2, 1>(a, s);
}

}  // namespace

// Tokens up to which the streaming kernel is used.
constexpr int64_t kFewTokens = 32;

static bool use_tiles(int64_t tokens, int64_t out, int64_t k, bool mx, int64_t ldx_bytes) {
  return tokens > kFewTokens && tile_product_fits(tokens, out, k, mx, ldx_bytes);
}

size_t product_workspace_bytes(int64_t tokens, int64_t out, int64_t k, bool mx) {
  return use_tiles(tokens, out, k, mx, mx ? k / 2 : k * 2) ? tile_product_workspace(tokens, out, k, mx) : 0;
}

int launch_matmul_w4a16(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx, const uint8_t* wp, const uint8_t* wc,
                        const float* ws2, int64_t out, uint16_t* y, int64_t ldy, void* workspace, hipStream_t s) {
  if (use_tiles(tokens, out, k, false, ldx * 2))
    return launch_tile_nv(x, ldx, nullptr, nullptr, nullptr, tokens, k, wp, wc, ws2, out, y, ldy, workspace, s);
  const ProductArgs a{reinterpret_cast<const uint8_t*>(x), nullptr, nullptr, wp, wc, ws2, ldx * 2, ldy, y, (int)tokens,
                      (int)out, (int)k};
  return run<kW4A16>(a, s);
}

int launch_matmul_w4a4(const uint8_t* xp, const uint8_t* xc, const float* xs2, int64_t tokens, int64_t k,
                       const uint8_t* wp, const uint8_t* wc, const float* ws2, int64_t out, uint16_t* y, int64_t ldy,
                       void* workspace, hipStream_t s) {
  if (use_tiles(tokens, out, k, false, k * 2))
    return launch_tile_nv(nullptr, 0, xp, xc, xs2, tokens, k, wp, wc, ws2, out, y, ldy, workspace, s);
  const ProductArgs a{xp, xc, xs2, wp, wc, ws2, k / 2, ldy, y, (int)tokens, (int)out, (int)k};
  return run<kW4A4>(a, s);
}

int launch_mxfp4_matmul(const uint8_t* xp, const uint8_t* xe, int64_t tokens, int64_t k, const uint8_t* wp,
                        const uint8_t* we, int64_t out, uint16_t* y, int64_t ldy, void* workspace, hipStream_t s) {
  if (use_tiles(tokens, out, k, true, k / 2))
    return launch_tile_mx(xp, xe, tokens, k, wp, we, out, y, ldy, workspace, s);
  const ProductArgs a{xp, xe, nullptr, wp, we, nullptr, k / 2, ldy, y, (int)tokens, (int)out, (int)k};
  return run<kMX>(a, s);
}

}  // namespace nvfp4
