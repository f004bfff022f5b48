// A mixture-of-experts layer over NVFP4 experts for any number of tokens, in the
// layout the MXFP4 -> NVFP4 cast leaves them (w1 and w3 of an expert share a
// tensor scale, "从MXFP4到NVFP4：Model Optimizer混合精度格式转换完全攻略" §3):
//
//   y[t] = sum over the experts e chosen for t of
//          weight(t, e) * W2_e ( silu(W1_e x[t]) * (W3_e x[t]) )
//
// The choices are sorted by expert, so that an expert's tokens are rows of row
// tiles of its own, which the sort lists.  Two launches of the tile kernels that
// multiply 16-bit rows by packed NVFP4 weights go over that list: the first reads
// the tokens where they are and makes h = silu(gate) * up, the second makes
// weight * s2 * W2 h, a row for every choice, and a last launch adds the rows of
// each token.  The number of row tiles is known on the device only; the grids are
// for the most there can be, and workgroups past the last tile end at once.
//
// Rounded on the way: h to bf16, which halves what moves and lets bf16 matrix
// instructions take it (an error the size of the final rounding's); the rows to the
// 11 bits of fp16, with a power of two of their own for every 32 columns, for a third
// error of that size would show.
#include "layer.hpp"
#include "tile_device.hpp"

namespace nvfp4 {

namespace {

struct SortedArgs {
  const uint16_t* x;               // fp16 rows of the tokens, [tokens][hidden]
  const float* xs;                 // their powers of two: value = fp16 * xs
  uint32_t x_bytes;                // of all of them, below 2^31
  const int32_t* order;            // choice of a sorted row
  const ExpertBand* bands;
  const int* count;                // of bands
  int band_tiles;                  // row tiles of a band, at most
  const float* weights;            // by choice
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
  uint16_t* h;                     // [rows][inter]
  uint16_t* ys;                    // fp16 [rows][hidden]
  uint8_t* ye;                     // their exponents, [rows][lde]
  int lde;
  int top_k, hidden, inter;
  int lds13, lds2;                 // bytes of a row of scales
};

// The largest finite magnitude of 8 bf16 values, or `top`.
__device__ __forceinline__ float finite_max(const uint4& v, float top) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = __uint_as_float((e & 1 ? q[e >> 1] & 0x7FFF0000u : q[e >> 1] << 16 & 0x7FFF0000u));
    top = a <= 3.40282347e38f ? fmaxf(top, a) : top;
  }
  return top;
}

// Rows of x in fp16 with a power of two each that puts the largest below 2^15: exact,
// but for values 2^29 and more below that, which are rounded to its 2^-39.  fp16
// weights take half the work of bf16 ones to make, which is most of what a tile of few
// rows has to do: 100 tokens of 128 experts of 7168 x 2048 (first product) 600 us with
// x in bf16.
__global__ __launch_bounds__(256) void half_rows_kernel(const uint16_t* x, int64_t ldx, int64_t tokens, int pieces,
                                                        uint16_t* y, float* scale) {
  __shared__ float part[4];
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(x + t * ldx);
    float top = 0.f;
    for (int i = threadIdx.x; i < pieces; i += 256) top = finite_max(src[i], top);
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const int e = max((int)(__float_as_uint(top) >> 23), 15);
    const float f = __uint_as_float((uint32_t)(127 + kHalfBias - e) << 23);
    for (int i = threadIdx.x; i < pieces; i += 256) {
      const uint4 v = src[i];
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
      f16x8 h;
#pragma unroll
      for (int z = 0; z < 8; ++z)
        h[z] = (_Float16)(__uint_as_float(z & 1 ? q[z >> 1] & 0xFFFF0000u : q[z >> 1] << 16) * f);
      reinterpret_cast<f16x8*>(y + t * (int64_t)pieces * 8)[i] = h;
    }
    if (threadIdx.x == 0) scale[t] = __builtin_amdgcn_ldexpf(1.0f, e - kHalfBias);
    __syncthreads();                                 // before the next token's maximum
  }
}

// A row tile and run of output rows.
struct TileAt { int expert, first, rows, n; };
// Those that a workgroup takes: false past the last.  Consecutive workgroups go to
// the 8 XCDs in turn, and so do bands: what an XCD's CUs work on at one time is the
// row tiles of one expert, up to band_tiles of them, against the same output rows, so
// that its L2 hands each weight to all of them and each row of x to all output rows
// (8192 tokens, 8 of 128 experts of 7168 x 2048: the first product fetches 6 GB so,
// 19 GB with every row tile on another XCD).  The list has the longest bands first:
// the XCDs have as much to do, and what is left at the end is short.
__device__ __forceinline__ bool expert_tile(const SortedArgs& a, int rows, int tiles_n, TileAt& t) {
  const uint32_t xcd = blockIdx.x & 7, i = blockIdx.x >> 3, per = a.band_tiles * tiles_n;
  const uint32_t at = i / per * 8 + xcd, m = i % per / tiles_n;
  if (at >= (uint32_t)*a.count) return false;
  const ExpertBand v = a.bands[at];
  t.expert = __builtin_amdgcn_readfirstlane(v.expert);
  t.first = __builtin_amdgcn_readfirstlane(v.first + m * rows);
  t.rows = __builtin_amdgcn_readfirstlane(min(v.rows - (int)m * rows, rows));
  t.n = __builtin_amdgcn_readfirstlane(i % per % tiles_n);
  return t.rows > 0;
}

// A form of the tile kernels: TN x 32 output rows a wave, WM x WN waves, NL that
// only load, OCC waves a SIMD.  A row tile has up to 32 MOST WM rows; the workgroup
// takes the least multiple of 32 WM that holds it, so that products of rows that are
// not there are left out.  Few rows leave LDS for more stages ahead (A1, A2 of them
// for one and two multiples, else 2), which weights that are used once need.
template <int TN_, int WM_, int WN_, int NL_, int MOST_, int OCC_, int A1, int A2>
struct Form {
  static constexpr int TN = TN_, WM = WM_, WN = WN_, NL = NL_, MOST = MOST_, OCC = OCC_;
  static constexpr int ROWS = 32 * MOST * WM, BN = 32 * TN * WN, THREADS = 64 * (WM * WN + NL);
  static constexpr int ahead(int tm) { return tm == 1 ? A1 : tm == 2 ? A2 : 2; }
  template <int TM, bool PAIRED>
  using Tile = NvTile<TM, TN, WM, WN, NL, ahead(TM), PAIRED>;
  static constexpr int most(int a, int b) { return a > b ? a : b; }
  static constexpr int LDS = most(most(Tile<1, false>::LDS, Tile<2, false>::LDS),
                                  MOST > 2 ? most(Tile<3, false>::LDS, Tile<4, false>::LDS) : 0);
};
template <typename F, typename Body>
__device__ __forceinline__ void with_rows(int rows, Body f) {
  constexpr int UNIT = 32 * F::WM;
  if (rows <= UNIT) return f(std::integral_constant<int, 1>{});
  if (F::MOST == 2 || rows <= 2 * UNIT) return f(std::integral_constant<int, 2>{});
  if constexpr (F::MOST > 2) {
    if (rows <= 3 * UNIT) return f(std::integral_constant<int, 3>{});
    return f(std::integral_constant<int, 4>{});
  }
}

// h of a row tile: of every 32 output rows of a tile, 16 are gate rows and 16 the
// up rows of the same channels, so that a lane holds both.
template <typename F>
__global__ __launch_bounds__(F::THREADS, F::OCC) void moe_up_tile_kernel(SortedArgs a) {
  constexpr int TN = F::TN, CH = F::BN / 2;          // channels of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[F::LDS];
  TileAt t;
  if (!expert_tile(a, F::ROWS, (a.inter + CH - 1) / CH, t)) return;
  const int ch0 = t.n * CH, left = a.inter - ch0;
  const uint32_t ldw = (uint32_t)a.hidden >> 1, ldx = (uint32_t)a.hidden * 2;
  const int64_t row = (int64_t)t.expert * 2 * a.inter + ch0;
  const int rows_w = 2 * a.inter - ch0;              // to the end of the expert's up rows
  const int32_t* order = a.order + t.first;
  const auto bx = make_buffer(a.x, a.x_bytes);
  const auto bw = make_buffer(a.p13 + row * ldw, (uint32_t)rows_w * ldw);
  const float s13 = a.s13[t.expert];
  constexpr int PITCH = 32 * TN + 16, LANES = 2 * TN, ROWS = 64 / LANES;      // of a wave's h in lds
  static_assert(F::WM * F::WN * 32 * PITCH <= F::LDS, "store staging");
  with_rows<F>(t.rows, [&](auto tm) {
    constexpr int TM = decltype(tm)::value;
    using T = typename F::template Tile<TM, true>;
    const typename T::Scales scales(a.c13 + row * a.lds13, rows_w * a.lds13, a.lds13, a.inter * a.lds13,
                                    lds_address(lds) + T::NBUF * T::STAGE, 0, loader_of<T::NW, F::NL>());
    nv_tile<true, TM, TN, F::WM, F::WN, F::NL, F::ahead(TM)>(
        bx, bw, a.hidden, 0, (a.hidden + 63) >> 6,
        [&](int r) { return (uint32_t)(order[min(r, t.rows - 1)] / a.top_k) * ldx; },
        [&](int r) { return (uint32_t)(min((r >> 5) * 16 + (r & 15), left - 1) + ((r >> 4) & 1) * a.inter) * ldw; }, scales,
        lds, [&](const f32x16 (&acc)[TN][TM], int wm, int wn, int wave, bool multiplies) {
          if (!multiplies) return;
          const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
          const int piece = lane % LANES, row0 = lane / LANES, ch = ch0 + wn * TN * 16 + piece * 8;
          uint8_t* mine = lds + wave * 32 * PITCH;
          float s[TM];
#pragma unroll
          for (int m = 0; m < TM; ++m)
            s[m] = a.xs[order[min((wm * TM + m) * 32 + l32, t.rows - 1)] / a.top_k] * s13;
#pragma unroll
          for (int m = 0; m < TM; ++m) {
            const int r0 = (wm * TM + m) * 32;
            if (r0 >= t.rows) break;
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float gate = acc[i][m][4 * g + e] * s[m], up = acc[i][m][8 + 4 * g + e] * s[m];
                  v[e] = to_bf16(gate / (1.0f + expf(-gate)) * up);
                }
                *reinterpret_cast<uint2*>(mine + l32 * PITCH + 32 * i + 16 * g + 2 * sub) =
                    make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
              }
#pragma unroll
            for (int r = 0; r < 32; r += ROWS) {
              const uint4 v = *reinterpret_cast<const uint4*>(mine + (r + row0) * PITCH + piece * 16);
              const int at = r0 + r + row0;
              if (at < t.rows && ch < a.inter)
                *reinterpret_cast<uint4*>(a.h + (int64_t)(t.first + at) * a.inter + ch) = v;
            }
          }
        });
  });
}

// v *= w; the biased exponent to store for the 32 columns of a token that this lane
// and the one 32 on hold: that of the largest finite value, at least 14, so that
// both powers of two are normal floats or, at the end of the range, exact ones.
__device__ __forceinline__ int half_exponent(f32x16& v, float w) {
  float top = 0.f;
#pragma unroll
  for (int z = 0; z < 16; ++z) {
    v[z] *= w;
    top = fmaxf(top, __builtin_fabsf(v[z]));         // (a NaN is passed over)
  }
  if (top > 3.40282347e38f) {
    top = 0.f;
#pragma unroll
    for (int z = 0; z < 16; ++z)
      if (__builtin_fabsf(v[z]) <= 3.40282347e38f) top = fmaxf(top, __builtin_fabsf(v[z]));
  }
  uint32_t p = __float_as_uint(top), q = p;
  swap32(p, q);
  return max((int)(max(p, q) >> 23), 14);
}

// The rows of a row tile, with their weight and the tensor scale.
template <typename F>
__global__ __launch_bounds__(F::THREADS, F::OCC) void moe_down_tile_kernel(SortedArgs a) {
  constexpr int TN = F::TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[F::LDS];
  TileAt t;
  if (!expert_tile(a, F::ROWS, (a.hidden + F::BN - 1) / F::BN, t)) return;
  const int o0 = t.n * F::BN, rows_w = min(F::BN, a.hidden - o0);
  const uint32_t ldw = (uint32_t)a.inter >> 1, ldh = (uint32_t)a.inter * 2;
  const int64_t row = (int64_t)t.expert * a.hidden + o0;
  const auto bx = make_buffer(a.h + (int64_t)t.first * a.inter, (uint32_t)t.rows * ldh);
  const auto bw = make_buffer(a.p2 + row * ldw, (uint32_t)rows_w * ldw);
  const float s2 = a.s2[t.expert];
  constexpr int PITCH = 64 * TN + 16, LANES = 4 * TN, ROWS = 64 / LANES;      // of a wave's rows in lds
  static_assert(F::WM * F::WN * 32 * PITCH <= F::LDS, "store staging");
  with_rows<F>(t.rows, [&](auto tm) {
    constexpr int TM = decltype(tm)::value;
    using T = typename F::template Tile<TM, false>;
    const typename T::Scales scales(a.c2 + row * a.lds2, rows_w * a.lds2, a.lds2, 0, lds_address(lds) + T::NBUF * T::STAGE,
                                    0, loader_of<T::NW, F::NL>());
    nv_tile<false, TM, TN, F::WM, F::WN, F::NL, F::ahead(TM)>(
        bx, bw, a.inter, 0, (a.inter + 63) >> 6, [&](int r) { return (uint32_t)min(r, t.rows - 1) * ldh; },
        [&](int r) { return (uint32_t)min(r, rows_w - 1) * ldw; }, scales, lds,
        [&](f32x16 (&acc)[TN][TM], int wm, int wn, int wave, bool multiplies) {
          if (!multiplies) return;
          const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
          const int piece = lane % LANES, row0 = lane / LANES, ob = o0 + wn * TN * 32, o = ob + piece * 8;
          uint8_t* mine = lds + wave * 32 * PITCH;
          float w[TM];
#pragma unroll
          for (int m = 0; m < TM; ++m)
            w[m] = a.weights[a.order[t.first + min((wm * TM + m) * 32 + l32, t.rows - 1)]] * s2;
#pragma unroll
          for (int m = 0; m < TM; ++m) {
            const int r0 = (wm * TM + m) * 32;
            if (r0 >= t.rows) break;
            const int at = t.first + min(r0 + l32, t.rows - 1);
#pragma unroll
            for (int i = 0; i < TN; ++i) {
              const int e = half_exponent(acc[i][m], w[m]);
              const float f = __uint_as_float((uint32_t)(127 + kHalfBias - e) << 23);      // the block's largest below 2^15
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  v[z] = __builtin_bit_cast(uint16_t, (_Float16)(acc[i][m][4 * g + z] * f));
                *reinterpret_cast<uint2*>(mine + l32 * PITCH + 64 * i + 16 * g + 2 * sub) =
                    make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
              }
              if (sub == 0 && r0 + l32 < t.rows && ob + 32 * i < a.hidden)
                a.ye[(int64_t)at * a.lde + (ob >> 5) + i] = (uint8_t)e;
            }
#pragma unroll
            for (int r = 0; r < 32; r += ROWS) {
              const uint4 v = *reinterpret_cast<const uint4*>(mine + (r + row0) * PITCH + piece * 16);
              const int to = r0 + r + row0;
              if (to < t.rows && o < a.hidden) *reinterpret_cast<uint4*>(a.ys + (int64_t)(t.first + to) * a.hidden + o) = v;
            }
          }
        });
  });
}

// Rows of scales to rows of whole words, zero past nb.
__global__ __launch_bounds__(256) void pad_scales_kernel(const uint8_t* src, int64_t rows, int nb, uint32_t* dst, int words) {
  const int64_t total = rows * words, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t row = i / words;
    const int w = (int)(i - row * words);
    uint32_t v = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (w * 4 + b < nb) v |= (uint32_t)src[row * nb + w * 4 + b] << (8 * b);
    dst[i] = v;
  }
}

template <typename F>
int run_products(const SortedArgs& a, int64_t max_bands, hipStream_t s) {
  const auto grid = [&](int64_t runs) { return (unsigned)((max_bands + 7) / 8 * 8 * a.band_tiles * runs); };
  moe_up_tile_kernel<F><<<grid((a.inter + F::BN / 2 - 1) / (F::BN / 2)), F::THREADS, 0, s>>>(a);
  const int st = launch_status("moe_up_tile_kernel");
  if (st) return st;
  moe_down_tile_kernel<F><<<grid((a.hidden + F::BN - 1) / F::BN), F::THREADS, 0, s>>>(a);
  return launch_status("moe_down_tile_kernel");
}
using Small = Form<1, 1, 4, 4, 4, 4, 6, 4>;
using Large = Form<2, 1, 4, 0, 4, 2, 4, 2>;

constexpr int64_t kPassRows = INT64_C(1) << 17;      // choices of one pass, at most

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Plan {
  int64_t tokens;                                    // of a pass, at most
  bool large;                                        // form of the tiles
  int rows, band_tiles;                              // rows of a tile, row tiles of a band
  int64_t max_bands;                                 // of a pass
  bool pad13, pad2;
  size_t order, place, offsets, sort, bands, count, c13, c2, x, xs, h, ys, ye, bytes;
};

Plan plan_layer(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  Plan p{};
  // a pass's rows of x have 32-bit offsets
  const int64_t most = ((INT64_C(1) << 31) - 1) / (hidden * 2);
  p.tokens = kPassRows / top_k;
  if (p.tokens > most) p.tokens = most;
  if (p.tokens > tokens) p.tokens = tokens;
  const int64_t n = p.tokens * top_k, per = n / experts;
  p.large = per > 32;
  p.rows = p.large ? Large::ROWS : Small::ROWS;
  p.band_tiles = p.large ? 2 : 1;
  // a band is whole, or the last one of an expert that has rows
  p.max_bands = n / (p.rows * p.band_tiles) + (n < experts ? n : experts);
  p.pad13 = hidden % 64 != 0;
  p.pad2 = inter % 64 != 0;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at = align256(at + bytes);
    return here;
  };
  p.order = take(n * 4);
  p.place = take(n * 4);
  p.offsets = take((experts + 1) * 4);
  p.sort = take(moe_sort_workspace_bytes(n, experts));
  p.bands = take(p.max_bands * sizeof(ExpertBand));
  p.count = take(4);
  p.c13 = take(p.pad13 ? experts * 2 * inter * ((hidden + 63) / 64 * 4) : 0);
  p.c2 = take(p.pad2 ? experts * hidden * ((inter + 63) / 64 * 4) : 0);
  p.x = take(p.tokens * hidden * 2);
  p.xs = take(p.tokens * 4);
  p.h = take(n * inter * 2);
  p.ys = take(n * hidden * 2);
  p.ye = take(n * ((hidden + 31) / 32));
  p.bytes = at;
  return p;
}

int pad_scales(const uint8_t* src, int64_t rows, int64_t k, uint8_t* dst, hipStream_t s) {
  const int words = (int)((k + 63) / 64);
  const int64_t want = (rows * words + 255) / 256;
  pad_scales_kernel<<<(unsigned)(want < 8192 ? want : 8192), 256, 0, s>>>(src, rows, (int)(k / 16),
                                                                          reinterpret_cast<uint32_t*>(dst), words);
  return launch_status("pad_scales_kernel");
}

}  // namespace

size_t moe_sorted_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  return plan_layer(tokens, top_k, experts, hidden, inter).bytes;
}

int launch_moe_sorted(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx, const int32_t* ids,
                      const float* weights, int top_k, int64_t experts, int64_t inter, const ExpertWeights& w,
                      uint16_t* y, int64_t ldy, void* workspace, hipStream_t s) {
  const Plan p = plan_layer(tokens, top_k, experts, hidden, inter);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  SortedArgs a{};
  int32_t* const order = reinterpret_cast<int32_t*>(base + p.order);
  int32_t* const place = reinterpret_cast<int32_t*>(base + p.place);
  const BandList list{reinterpret_cast<ExpertBand*>(base + p.bands), reinterpret_cast<int*>(base + p.count),
                      p.rows * p.band_tiles, p.rows};
  a.order = order;
  a.bands = list.bands;
  a.count = list.count;
  a.band_tiles = p.band_tiles;
  a.p13 = w.p13;
  a.p2 = w.p2;
  a.s13 = w.s13;
  a.s2 = w.s2;
  a.c13 = p.pad13 ? base + p.c13 : w.c13;
  a.c2 = p.pad2 ? base + p.c2 : w.c2;
  a.h = reinterpret_cast<uint16_t*>(base + p.h);
  a.ys = reinterpret_cast<uint16_t*>(base + p.ys);
  a.ye = base + p.ye;
  a.lde = (int)((hidden + 31) / 32);
  a.top_k = top_k;
  a.hidden = (int)hidden;
  a.inter = (int)inter;
  a.lds13 = (int)((hidden + 63) / 64 * 4);
  a.lds2 = (int)((inter + 63) / 64 * 4);
  int st;
  if (p.pad13 && (st = pad_scales(w.c13, experts * 2 * inter, hidden, base + p.c13, s))) return st;
  if (p.pad2 && (st = pad_scales(w.c2, experts * hidden, inter, base + p.c2, s))) return st;
  a.x = reinterpret_cast<const uint16_t*>(base + p.x);
  a.xs = reinterpret_cast<const float*>(base + p.xs);
  for (int64_t t = 0; t < tokens; t += p.tokens) {
    const int64_t here = tokens - t < p.tokens ? tokens - t : p.tokens;
    a.x_bytes = (uint32_t)(here * hidden * 2);
    half_rows_kernel<<<(unsigned)here, 256, 0, s>>>(x + t * ldx, ldx, here, (int)(hidden / 8),
                                                    reinterpret_cast<uint16_t*>(base + p.x),
                                                    reinterpret_cast<float*>(base + p.xs));
    if ((st = launch_status("half_rows_kernel"))) return st;
    a.weights = weights + t * top_k;
    if ((st = launch_moe_sort(ids + t * top_k, here * top_k, experts, order, place,
                              reinterpret_cast<int32_t*>(base + p.offsets), base + p.sort, list, s)))
      return st;
    if ((st = p.large ? run_products<Large>(a, p.max_bands, s) : run_products<Small>(a, p.max_bands, s))) return st;
    if ((st = launch_moe_combine_half(a.ys, a.ye, place, here, top_k, hidden, y + t * ldy, ldy, s))) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
