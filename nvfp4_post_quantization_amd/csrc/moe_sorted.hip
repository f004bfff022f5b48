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
  const uint8_t* x;                // bf16 rows of the tokens
  int64_t ldx;                     // bytes
  uint32_t x_bytes;                // of all of them, below 2^31
  const int32_t* order;            // choice of a sorted row
  const ExpertTile* tiles;
  const int* count;                // of tiles
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

// Which row tile and run of output rows a workgroup takes: false past the last.
// Consecutive workgroups go to the 8 XCDs in turn, row tiles do so too; an XCD takes
// all output rows of one before its next.  The list has the longest tiles first, so
// that the XCDs have as much to do and what is left at the end is short.
__device__ __forceinline__ bool expert_tile(const SortedArgs& a, int tiles_n, ExpertTile& t, int& n) {
  const uint32_t xcd = blockIdx.x & 7, i = blockIdx.x >> 3, at = i / tiles_n * 8 + xcd;
  if (at >= (uint32_t)*a.count) return false;
  const ExpertTile v = a.tiles[at];
  t.expert = __builtin_amdgcn_readfirstlane(v.expert);
  t.first = __builtin_amdgcn_readfirstlane(v.first);
  t.rows = __builtin_amdgcn_readfirstlane(v.rows);
  n = __builtin_amdgcn_readfirstlane(i % tiles_n);
  return true;
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
  ExpertTile t;
  int n;
  if (!expert_tile(a, (a.inter + CH - 1) / CH, t, n)) return;
  const int ch0 = n * CH, left = a.inter - ch0;
  const uint32_t ldw = (uint32_t)a.hidden >> 1;
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
    nv_tile<false, TM, TN, F::WM, F::WN, F::NL, F::ahead(TM)>(
        bx, bw, a.hidden, 0, (a.hidden + 63) >> 6,
        [&](int r) { return (uint32_t)(order[min(r, t.rows - 1)] / a.top_k) * (uint32_t)a.ldx; },
        [&](int r) { return (uint32_t)(min((r >> 5) * 16 + (r & 15), left - 1) + ((r >> 4) & 1) * a.inter) * ldw; }, scales,
        lds, [&](const f32x16 (&acc)[TN][TM], int wm, int wn, int wave, bool multiplies) {
          if (!multiplies) return;
          const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
          const int piece = lane % LANES, row0 = lane / LANES, ch = ch0 + wn * TN * 16 + piece * 8;
          uint8_t* mine = lds + wave * 32 * PITCH;
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
                  const float gate = acc[i][m][4 * g + e] * s13, up = acc[i][m][8 + 4 * g + e] * s13;
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
  ExpertTile t;
  int n;
  if (!expert_tile(a, (a.hidden + F::BN - 1) / F::BN, t, n)) return;
  const int o0 = n * F::BN, rows_w = min(F::BN, a.hidden - o0);
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
#pragma unroll
          for (int m = 0; m < TM; ++m) {
            const int r0 = (wm * TM + m) * 32;
            if (r0 >= t.rows) break;
            const int at = t.first + min(r0 + l32, t.rows - 1);
            const float w = a.weights[a.order[at]] * s2;
#pragma unroll
            for (int i = 0; i < TN; ++i) {
              const int e = half_exponent(acc[i][m], w);
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
int run_products(const SortedArgs& a, int64_t max_tiles, hipStream_t s) {
  const auto grid = [&](int64_t runs) { return (unsigned)((max_tiles + 7) / 8 * 8 * runs); };
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
  int bm;                                            // their rows
  int64_t max_tiles;                                 // row tiles of a pass, at most
  bool pad13, pad2;
  size_t order, place, offsets, sort, tiles, count, c13, c2, h, ys, ye, bytes;
};

Plan plan_layer(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  Plan p{};
  p.tokens = kPassRows / top_k;
  if (p.tokens > tokens) p.tokens = tokens;
  const int64_t n = p.tokens * top_k, per = n / experts;
  p.large = per > 32;
  p.bm = p.large ? Large::ROWS : Small::ROWS;
  // a tile is full, or the last one of an expert that has rows
  p.max_tiles = n / p.bm + (n < experts ? n : experts);
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
  p.tiles = take(p.max_tiles * sizeof(ExpertTile));
  p.count = take(4);
  p.c13 = take(p.pad13 ? experts * 2 * inter * ((hidden + 63) / 64 * 4) : 0);
  p.c2 = take(p.pad2 ? experts * hidden * ((inter + 63) / 64 * 4) : 0);
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
  a.ldx = ldx * 2;
  int32_t* const order = reinterpret_cast<int32_t*>(base + p.order);
  int32_t* const place = reinterpret_cast<int32_t*>(base + p.place);
  ExpertTile* const tiles = reinterpret_cast<ExpertTile*>(base + p.tiles);
  int* const count = reinterpret_cast<int*>(base + p.count);
  a.order = order;
  a.tiles = tiles;
  a.count = count;
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
  // a pass's rows of x have 32-bit offsets
  int64_t pass = ((INT64_C(1) << 31) - 1 - hidden * 2) / (ldx * 2) + 1;
  if (pass > p.tokens) pass = p.tokens;
  for (int64_t t = 0; t < tokens; t += pass) {
    const int64_t here = tokens - t < pass ? tokens - t : pass;
    a.x = reinterpret_cast<const uint8_t*>(x + t * ldx);
    a.x_bytes = (uint32_t)((here - 1) * a.ldx + hidden * 2);
    a.weights = weights + t * top_k;
    if ((st = launch_moe_sort(ids + t * top_k, here * top_k, experts, order, place,
                              reinterpret_cast<int32_t*>(base + p.offsets), base + p.sort, TileList{tiles, count, p.bm, p.bm / (p.large ? Large::MOST : Small::MOST)}, s)))
      return st;
    if ((st = p.large ? run_products<Large>(a, p.max_tiles, s) : run_products<Small>(a, p.max_tiles, s))) return st;
    if ((st = launch_moe_combine_half(a.ys, a.ye, place, here, top_k, hidden, y + t * ldy, ldy, s))) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
