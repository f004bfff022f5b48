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
// instructions take it (an error the size of the final rounding's); the rows stay
// in fp32, for a third error of that size would show.
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
  float* ys;                       // [rows][hidden]
  int top_k, hidden, inter;
  int lds13, lds2;                 // bytes of a row of scales
};

// Which row tile and run of output rows a workgroup takes: false past the last.
// Consecutive workgroups go to the 8 XCDs in turn; each XCD gets a contiguous run
// of (row tile, output rows), output rows first, so that an expert's weights are
// read by its row tiles at one time and rows of x by neighbours.
__device__ __forceinline__ bool expert_tile(const SortedArgs& a, int tiles_n, ExpertTile& t, int& n) {
  const uint32_t total = (uint32_t)*a.count * (uint32_t)tiles_n;
  const uint32_t id = blockIdx.x, xcd = id & 7, i = id >> 3, q = total >> 3, r = total & 7;
  if (i >= q + (xcd < r ? 1 : 0)) return false;
  const uint32_t at = xcd * q + min(xcd, r) + i;
  const ExpertTile v = a.tiles[at / tiles_n];
  t.expert = __builtin_amdgcn_readfirstlane(v.expert);
  t.first = __builtin_amdgcn_readfirstlane(v.first);
  t.rows = __builtin_amdgcn_readfirstlane(v.rows);
  n = __builtin_amdgcn_readfirstlane(at % tiles_n);
  return true;
}

// h of a row tile: of every 32 output rows of a tile, 16 are gate rows and 16 the
// up rows of the same channels, so that a lane holds both.
template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
__global__ __launch_bounds__(64 * (WM * WN + NL), NL && AHEAD == 2 ? 4 : 2) void moe_up_tile_kernel(SortedArgs a) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD, true>;
  constexpr int CH = T::BN / 2;                      // channels of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::LDS];
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
  const int loader = loader_of<T::NW, NL>();
  const typename T::Scales scales(a.c13 + row * a.lds13, rows_w * a.lds13, a.lds13, a.inter * a.lds13,
                                  lds_address(lds) + T::NBUF * T::STAGE, 0, loader);
  const float s13 = a.s13[t.expert];
  constexpr int PITCH = 32 * TN + 16, LANES = 2 * TN, ROWS = 64 / LANES;      // of a wave's h in lds
  static_assert(T::NW * 32 * PITCH <= T::LDS, "store staging");
  nv_tile<false, TM, TN, WM, WN, NL, AHEAD>(
      bx, bw, a.hidden, 0, (a.hidden + 63) >> 6,
      [&](int r) { return (uint32_t)(order[min(r, t.rows - 1)] / a.top_k) * (uint32_t)a.ldx; },
      [&](int r) { return (uint32_t)(min((r >> 5) * 16 + (r & 15), left - 1) + ((r >> 4) & 1) * a.inter) * ldw; }, scales,
      lds, [&](const f32x16 (&acc)[TN][TM], int wm, int wn, int wave) {
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
}

// The rows of a row tile, with their weight and the tensor scale.
template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
__global__ __launch_bounds__(64 * (WM * WN + NL), NL && AHEAD == 2 ? 4 : 2) void moe_down_tile_kernel(SortedArgs a) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::LDS];
  ExpertTile t;
  int n;
  if (!expert_tile(a, (a.hidden + T::BN - 1) / T::BN, t, n)) return;
  const int o0 = n * T::BN, rows_w = min(T::BN, a.hidden - o0);
  const uint32_t ldw = (uint32_t)a.inter >> 1, ldh = (uint32_t)a.inter * 2;
  const int64_t row = (int64_t)t.expert * a.hidden + o0;
  const auto bx = make_buffer(a.h + (int64_t)t.first * a.inter, (uint32_t)t.rows * ldh);
  const auto bw = make_buffer(a.p2 + row * ldw, (uint32_t)rows_w * ldw);
  const int loader = loader_of<T::NW, NL>();
  const typename T::Scales scales(a.c2 + row * a.lds2, rows_w * a.lds2, a.lds2, 0, lds_address(lds) + T::NBUF * T::STAGE, 0,
                                  loader);
  const float s2 = a.s2[t.expert];
  nv_tile<false, TM, TN, WM, WN, NL, AHEAD>(
      bx, bw, a.inter, 0, (a.inter + 63) >> 6, [&](int r) { return (uint32_t)min(r, t.rows - 1) * ldh; },
      [&](int r) { return (uint32_t)min(r, rows_w - 1) * ldw; }, scales, lds,
      [&](const f32x16 (&acc)[TN][TM], int wm, int wn, int) {
        const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const int r = (wm * TM + m) * 32 + l32;
          if (r >= t.rows) continue;
          const float w = a.weights[a.order[t.first + r]] * s2;
          float* dst = a.ys + (int64_t)(t.first + r) * a.hidden;
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int o = o0 + (wn * TN + i) * 32 + 8 * g + sub;
              if (o < a.hidden)
                *reinterpret_cast<f32x4*>(dst + o) = f32x4{acc[i][m][4 * g] * w, acc[i][m][4 * g + 1] * w,
                                                           acc[i][m][4 * g + 2] * w, acc[i][m][4 * g + 3] * w};
            }
        }
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

constexpr int64_t kPassRows = INT64_C(1) << 17;      // choices of one pass, at most

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Plan {
  int64_t tokens;                                    // of a pass, at most
  int bm;
  int64_t max_tiles;                                 // row tiles of a pass, at most
  bool pad13, pad2;
  size_t order, place, offsets, sort, tiles, count, c13, c2, h, ys, bytes;
};

Plan plan_layer(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  Plan p{};
  p.tokens = kPassRows / top_k;
  if (p.tokens > tokens) p.tokens = tokens;
  const int64_t n = p.tokens * top_k, per = n / experts;
  p.bm = per <= 32 ? 32 : per <= 64 ? 64 : per <= 256 ? 128 : 256;
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
  p.ys = take(n * hidden * 4);
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

template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
int run_up(const SortedArgs& a, int64_t max_tiles, hipStream_t s) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD>;
  const int64_t grid = max_tiles * ((a.inter + T::BN / 2 - 1) / (T::BN / 2));
  moe_up_tile_kernel<TM, TN, WM, WN, NL, AHEAD><<<(unsigned)((grid + 7) / 8 * 8), T::THREADS, 0, s>>>(a);
  return launch_status("moe_up_tile_kernel");
}
template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
int run_down(const SortedArgs& a, int64_t max_tiles, hipStream_t s) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD>;
  const int64_t grid = max_tiles * ((a.hidden + T::BN - 1) / T::BN);
  moe_down_tile_kernel<TM, TN, WM, WN, NL, AHEAD><<<(unsigned)((grid + 7) / 8 * 8), T::THREADS, 0, s>>>(a);
  return launch_status("moe_down_tile_kernel");
}

int run_products(const SortedArgs& a, const Plan& p, hipStream_t s) {
  int st;
  if (p.bm == 256) return (st = run_up<4, 2, 2, 4, 0, 2>(a, p.max_tiles, s)) ? st : run_down<4, 2, 2, 4, 0, 2>(a, p.max_tiles, s);
  if (p.bm == 128) return (st = run_up<4, 1, 1, 4, 4, 2>(a, p.max_tiles, s)) ? st : run_down<4, 1, 1, 4, 4, 2>(a, p.max_tiles, s);
  if (p.bm == 64) return (st = run_up<2, 1, 1, 4, 4, 2>(a, p.max_tiles, s)) ? st : run_down<2, 1, 1, 4, 4, 2>(a, p.max_tiles, s);
  return (st = run_up<1, 1, 1, 4, 4, 2>(a, p.max_tiles, s)) ? st : run_down<1, 1, 1, 4, 4, 2>(a, p.max_tiles, s);
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
  a.ys = reinterpret_cast<float*>(base + p.ys);
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
                              reinterpret_cast<int32_t*>(base + p.offsets), base + p.sort, TileList{tiles, count, p.bm}, s)))
      return st;
    if ((st = run_products(a, p, s))) return st;
    if ((st = launch_moe_combine(a.ys, hidden, place, nullptr, here, top_k, hidden, y + t * ldy, ldy, s))) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
