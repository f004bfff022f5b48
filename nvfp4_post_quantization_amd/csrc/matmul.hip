// Products of packed 4-bit matrices: y[t][o] = RN_bf16(sum_k x[t][k] w[o][k])
// for W4A16 and W4A4 NVFP4 ("Coder390 NVFP4 校正（校准）方式" §3, the W4A16 and
// W4A4 tiers) and for MXFP4 on both sides.
//
// Few tokens: the weights are read once and bound the call.  A workgroup
// takes 16 RT output rows and splits the channels over its waves; each wave
// streams its share of the rows straight from HBM into registers, expands it
// there, and multiplies it by up to 16 NT tokens on the matrix cores (the
// rows are the instruction's M side, the tokens its N side).  The waves'
// partial tiles meet in LDS and are added in wave order.
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

// Bytes of a row's block scales.
template <int KIND>
__device__ __forceinline__ int64_t scale_row(int k) { return KIND == kMX ? k >> 5 : k >> 4; }

template <int KIND>
__device__ __forceinline__ float tensor_scaled(float v, const ProductArgs& a) {
  if constexpr (KIND == kW4A16) return v * *a.ws2;
  else if constexpr (KIND == kW4A4) return (v * *a.ws2) * *a.xs2;
  else return v;
}

template <int KIND, int RT, int NT, int NW, bool K32>
__global__ __launch_bounds__(64 * NW) void few_tokens_kernel(ProductArgs a) {
  __shared__ f32x4 part[NW][RT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row0 = blockIdx.x * 16 * RT;
  const int tok0 = blockIdx.y * 16 * NT;
  ProductRows<RT, NT> p;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t row = min(row0 + 16 * r + (lane & 15), a.out - 1);      // rows past the end are not stored
    p.wp[r] = a.wp + row * (a.k >> 1);
    p.wc[r] = a.wc + row * scale_row<KIND>(a.k);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t t = min(tok0 + 16 * n + (lane & 15), a.tokens - 1);
    p.xp[n] = a.xp + t * a.ldx;
    p.xc[n] = a.xc + t * scale_row<KIND>(a.k);
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int units = (a.k + 127) >> 7;
  const int per = (units + NW - 1) / NW;
  product_units<KIND, RT, NT, K32, false, (NT > 1 ? 1 : 2)>(acc, p, min(wave * per, units), min((wave + 1) * per, units),
                                                           lane >> 4, a.k, 0);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) part[wave][r * NT + n][lane] = acc[r][n];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * NT * 64; i += 64 * NW) {
    const int tile = i >> 6, l = i & 63;
    f32x4 s = part[0][tile][l];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += part[w][tile][l];
    const int row = row0 + 16 * (tile / NT) + 4 * (l >> 4);
    const int t = tok0 + 16 * (tile % NT) + (l & 15);
    if (t < a.tokens) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (row + e < a.out) a.y[t * a.ldy + row + e] = to_bf16(tensor_scaled<KIND>(s[e], a));
    }
  }
}

template <int KIND, int RT, int NT, int NW, bool K32>
void run_few(const ProductArgs& a, hipStream_t s) {
  const dim3 grid((a.out + 16 * RT - 1) / (16 * RT), (a.tokens + 16 * NT - 1) / (16 * NT));
  few_tokens_kernel<KIND, RT, NT, NW, K32><<<grid, 64 * NW, 0, s>>>(a);
}

template <int KIND, bool K32>
int run(const ProductArgs& a, hipStream_t s) {
  if (a.tokens <= 16) run_few<KIND, 1, 1, 8, K32>(a, s);
  else run_few<KIND, 2, 2, 8, K32>(a, s);
  return launch_status("few_tokens_kernel");
}

}  // namespace

// Tokens up to which the streaming kernel is used.
constexpr int64_t kFewTokens = 64;

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
  return (k % 32) ? run<kW4A16, false>(a, s) : run<kW4A16, true>(a, s);
}

int launch_matmul_w4a4(const uint8_t* xp, const uint8_t* xc, const float* xs2, int64_t tokens, int64_t k,
                       const uint8_t* wp, const uint8_t* wc, const float* ws2, int64_t out, uint16_t* y, int64_t ldy,
                       void* workspace, hipStream_t s) {
  if (use_tiles(tokens, out, k, false, k * 2))
    return launch_tile_nv(nullptr, 0, xp, xc, xs2, tokens, k, wp, wc, ws2, out, y, ldy, workspace, s);
  const ProductArgs a{xp, xc, xs2, wp, wc, ws2, k / 2, ldy, y, (int)tokens, (int)out, (int)k};
  return (k % 32) ? run<kW4A4, false>(a, s) : run<kW4A4, true>(a, s);
}

int launch_mxfp4_matmul(const uint8_t* xp, const uint8_t* xe, int64_t tokens, int64_t k, const uint8_t* wp,
                        const uint8_t* we, int64_t out, uint16_t* y, int64_t ldy, void* workspace, hipStream_t s) {
  if (use_tiles(tokens, out, k, true, k / 2))
    return launch_tile_mx(xp, xe, tokens, k, wp, we, out, y, ldy, workspace, s);
  const ProductArgs a{xp, xe, nullptr, wp, we, nullptr, k / 2, ldy, y, (int)tokens, (int)out, (int)k};
  return run<kMX, true>(a, s);
}

}  // namespace nvfp4
