// Products of packed 4-bit matrices: y[t][o] = RN_bf16(sum_k x[t][k] w[o][k])
// for W4A16 and W4A4 NVFP4 ("Coder390 NVFP4 校正（校准）方式" §3, the W4A16 and
// W4A4 tiers) and for MXFP4 on both sides.
//
// Few tokens: the weights are read once and bound the call.  A workgroup
// takes a run of row tiles; its waves split the channels, hold their part of
// the tokens in registers and stream the rows' packed weights past them from
// HBM.  The waves' partial sums meet in LDS and are added in wave order.
// A call in a captured graph, with the weights cold (768 MB of others since their
// last use; in brackets: one set, which the 256 MB MALL keeps), us:
//   12288x4096 (28 MB; MXFP4 27)  W4A16, 1, 5, 16 tokens  8.9, 11.2, 14.7  (7.1, 8.8, 12.2)
//                                 W4A4                    9.2, 11.3, 14.3  (7.2, 8.8, 12.1)
//                                 MXFP4                   8.3,  8.4,  8.7  (5.1, 5.2,  5.6)
//   4096x12288                    W4A16                  10.0, 12.4, 17.0  (7.4, 9.4, 14.4)
//   28672x8192 (132 MB; 125)      W4A16, 1, 16 tokens    30, 50 (24, 44);  MXFP4, 16: 27.5 (21)
// that is 3.2 TB/s of cold weights for one token at the small end and 4.4 at the
// large one.  What is left at the small end is a launch, one trip to memory and
// the sum over the waves; at the large end the SIMDs issue something over 90% of
// the time (52 to 55 vector instructions a KiB for up to four tokens).
// Comparisons of variants below that do not say cold are of one set of weights.
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

constexpr int kCus = 256;

// Workgroups: enough to give every CU its waves.
unsigned few_grid(int tiles, int waves, int cu_waves) {
  const int most = kCus * (cu_waves / waves);
  return (unsigned)(tiles < most ? tiles : most);
}

// A workgroup's run of tiles.  Those that share a CU (kCus apart) share a run
// that is as long as any other CU's, also where the tiles per workgroup are not
// whole.
__device__ __forceinline__ void tile_run(int tiles, int& begin, int& end) {
  const int n = gridDim.x, shared = n / kCus;
  int at = blockIdx.x;
  if (shared > 1 && n == shared * kCus) at = at % kCus * shared + at / kCus;
  begin = (int)((int64_t)tiles * at / n);
  end = (int)((int64_t)tiles * (at + 1) / n);
}

template <int KIND>
__device__ __forceinline__ void store_rows(const ProductArgs& a, int row, int tok, f32x4 v) {
  uint16_t* dst = a.y + (int64_t)tok * a.ldy + row;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (row + e < a.out) dst[e] = to_bf16(tensor_scaled<KIND>(v[e], a));
}

// 4 NG tokens (the y coordinate's) against NVFP4 rows.  CU: waves that share a
// CU, MW: waves of a workgroup, both at most.
template <int KIND, bool ODD, int NG, int CU, int MW>
__global__ __launch_bounds__(64 * MW, CU / 4) void few_tokens_kernel(ProductArgs a) {
  constexpr int TB = 4;
  __shared__ f32x4 part[MW * TB * NG * 16];
  constexpr int STAGE = KIND == kW4A16 ? 4096 : 1024;      // of a wave: tokens, then weights, change their order there
  __shared__ __attribute__((aligned(16))) uint8_t stage[MW * STAGE];
  const int lane = threadIdx.x & 63;
  uint8_t* const lds_wave = stage + (threadIdx.x >> 6) * STAGE;
  const int tok0 = blockIdx.y * 4 * NG;
  const uint32_t ldw = (uint32_t)a.k >> 1, lds = (uint32_t)a.k >> 4;
  int begin, end;
  tile_run((a.out + 15) >> 4, begin, end);
  const uint32_t group_row[4] = {0, 4, 8, 12};
  Chunk x[1][NG];
  auto rows_of = [&](int t) {
    const int row = t * 16;
    const uint32_t rows = min(16, a.out - row);
    return PackedRows{a.wp + (int64_t)row * ldw, a.wc + (int64_t)row * lds, rows * ldw, rows * lds};
  };
  RowGroup packed[NG];
  auto load_tokens = [&](int q) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int t0 = min(tok0 + 4 * n, a.tokens - 1), last = a.tokens - 1 - t0;               // others are not stored
      if constexpr (KIND == kW4A16) {
        load_pieces(x[0][n], a.xp + (int64_t)(t0 + min(lane >> 4, last)) * a.ldx, q, a.k);
      } else {
        const uint32_t rows = q * 512 < a.k ? min(4, a.tokens - t0) : 0;
        packed[n].load(PackedRows{a.xp + (int64_t)t0 * ldw, a.xc + (int64_t)t0 * lds, rows * ldw, rows * lds}, 0, q,
                       LaneAt<ODD>(min(lane >> 4, last), q, a.k), a.k);
      }
    }
  };
  auto take_tokens = [&]() {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if constexpr (KIND == kW4A16) pieces_to_chunk(x[0][n], lds_wave);
      else expand_chunk(x[0][n], packed[n].arranged(lds_wave));
    }
  };
  auto done = [&](int t, int n, int q, int tj, f32x4 v) {
    const int row = t * 16 + q * 4, tok = tok0 + 4 * n + tj;
    if (tok < a.tokens && row < a.out) store_rows<KIND>(a, row, tok, v);
  };
  stream_rows<ODD, NG, TB>(begin, end, a.k, quad_plan<1>(a.k, CU), group_row, x, part, lds_wave, rows_of, load_tokens,
                           take_tokens, done);
}

// 16 NT tokens against MXFP4 rows.
template <int NT, int QW, int RT, int CU, int MW>
__global__ __launch_bounds__(64 * MW, CU / 4) void few_mx_tokens_kernel(ProductArgs a) {
  constexpr int TB = 4 / NT;
  __shared__ f32x4 part[MW * TB * NT * 64];
  __shared__ __attribute__((aligned(16))) uint8_t turn[MW][1024];          // operands change their order there
  const int r4 = (threadIdx.x & 63) >> 2;
  const int tok0 = blockIdx.y * 16 * NT;
  const uint32_t ldw = (uint32_t)a.k >> 1, lds = (uint32_t)a.k >> 5;
  int begin, end;
  tile_run((a.out + 15) >> 4, begin, end);
  PackedRows tokens[NT];
  uint32_t token_row[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t0 = min(tok0 + 16 * n, a.tokens - 1);
    const uint32_t rows = min(16, a.tokens - t0);
    tokens[n] = PackedRows{a.xp + (int64_t)t0 * ldw, a.xc + (int64_t)t0 * lds, rows * ldw, rows * lds};
    token_row[n] = min(r4, a.tokens - 1 - t0);                                   // others are not stored
  }
  auto rows_of = [&](int t) {
    const int row = t * 16;
    const uint32_t rows = min(min(16 * RT, (end - t) * 16), a.out - row);
    return PackedRows{a.wp + (int64_t)row * ldw, a.wc + (int64_t)row * lds, rows * ldw, rows * lds};
  };
  auto done = [&](int t, int n, int l, f32x4 v) {
    const int row = t * 16 + 4 * (l >> 4), tok = tok0 + 16 * n + (l & 15);
    if (tok < a.tokens && row < a.out) store_rows<kMX>(a, row, tok, v);
  };
  stream_mx_rows<NT, QW, RT, TB>(begin, end, a.k, quad_plan<QW>(a.k, CU), tokens, token_row, part, turn[threadIdx.x >> 6], rows_of,
                                 done);
}

template <int KIND, bool ODD, int NG, int CU>
int run_few(const ProductArgs& a, hipStream_t s) {
  const int waves = quad_plan<1>(a.k, CU).waves;
  const dim3 grid(few_grid((a.out + 15) / 16, waves, CU), (a.tokens + 4 * NG - 1) / (4 * NG));
  if (waves <= 4) few_tokens_kernel<KIND, ODD, NG, CU, 4><<<grid, 64 * waves, 0, s>>>(a);
  else if (CU == 8 || waves <= 8) few_tokens_kernel<KIND, ODD, NG, CU, 8><<<grid, 64 * waves, 0, s>>>(a);
  else few_tokens_kernel<KIND, ODD, NG, CU, CU><<<grid, 64 * waves, 0, s>>>(a);
  return launch_status("few_tokens_kernel");
}

template <int NT, int QW, int RT, int CU>
int run_few_mx(const ProductArgs& a, hipStream_t s) {
  const int waves = quad_plan<QW>(a.k, CU).waves;
  const dim3 grid(few_grid((a.out + 15) / 16, waves, CU), (a.tokens + 16 * NT - 1) / (16 * NT));
  if (waves <= 4) few_mx_tokens_kernel<NT, QW, RT, CU, 4><<<grid, 64 * waves, 0, s>>>(a);
  else if (CU == 8 || waves <= 8) few_mx_tokens_kernel<NT, QW, RT, CU, 8><<<grid, 64 * waves, 0, s>>>(a);
  else few_mx_tokens_kernel<NT, QW, RT, CU, CU><<<grid, 64 * waves, 0, s>>>(a);
  return launch_status("few_mx_tokens_kernel");
}

template <int KIND>
int run(const ProductArgs& a, hipStream_t s) {
  if constexpr (KIND == kMX) {
    // Two row tiles a step and 8 waves where those hold the channels, else two
    // quads a wave: 12288x4096, one token: 8.2 us against 9.5 with one tile and 16
    // waves (both before lanes shared cache lines, which took the first to 5.1).
    const bool narrow = a.k <= 4096;
    if (a.tokens <= 16) return narrow ? run_few_mx<1, 1, 2, 8>(a, s) : run_few_mx<1, 2, 1, 12>(a, s);
    return narrow ? run_few_mx<2, 1, 2, 8>(a, s) : run_few_mx<2, 2, 1, 12>(a, s);
  } else {
    // Tokens a workgroup: what their registers leave of the waves that share a
    // CU counts.  4096x12288: one token takes 7.4 us with 4 and 16 waves; five 9.4
    // with 8 and 16 (two quads a wave and 12 waves: 1 more); sixteen 14.4 with 16
    // and 8 (as two workgroups of 8: half as much again).  k off 32 has few uses:
    // two sizes.
    if (a.k % 32) return a.tokens <= 4 ? run_few<KIND, true, 1, 16>(a, s) : run_few<KIND, true, 4, 8>(a, s);
    if (a.tokens <= 4) return run_few<KIND, false, 1, 16>(a, s);
    if (a.tokens <= 8) return run_few<KIND, false, 2, 16>(a, s);
    return run_few<KIND, false, 4, 8>(a, s);
  }
}

}  // namespace

// Tokens up to which the streaming kernels are used.  Weights cold, us here and
// in tiles:
//             4096x12288      12288x4096      28672x8192
//   MXFP4 32  11.2 and 15.6   10.2 and 15.2   30 and 38
//         48  17.2 and 16.5
//         64  17.7 and 17.0   15.7 and 17.0   48 and 38
//   W4A16 16  17.8 and 24.2   14.7 and 22.6   50 and 68
//         24  31.5 and 24.9   25.3 and 23.2
//         32  31.6 and 25.2   25.3 and 24.2   96 and 68
//   W4A4  16  16.5 and 26.0   14.3 and 24.1
//         32  29.5 and 27.3   25.3 and 25.8
// (MXFP4 tokens are taken 32 at a time, NVFP4 weights are read again for every 16.)
static bool use_tiles(int64_t tokens, int64_t out, int64_t k, bool mx, int64_t ldx_bytes) {
  return tokens > (mx ? 32 : 16) && tile_product_fits(tokens, out, k, ldx_bytes);
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
