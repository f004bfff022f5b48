// Products of packed 4-bit matrices for more tokens than the streaming
// kernels of matmul.hip take: tiles of tokens x output rows on the matrix
// cores, fed through LDS.
//
//   MXFP4       32x32x64 scaled FP4 instructions on the packed operands
//   16 x NVFP4  32x32x16 bf16 / fp16 instructions; the weights stay packed in
//               LDS and are expanded (exactly) in registers by the one wave
//               column that multiplies them; W4A4's activations are expanded
//               to fp16 once, into the workspace
//
// The weights are the instruction's M side, the tokens its N side, so that a
// lane's results are runs of four neighbouring outputs of one token.
//
// Stages of the channel axis (128 channels of MXFP4, 64 of 16-bit
// activations) go from HBM / L2 straight to LDS (buffer loads to LDS, 16 bytes
// a lane), AHEAD stages ahead; waves wait for their own loads by count and
// meet at one barrier per stage, towards its end, so that the first operands
// of the next stage are read while the rest of this one is multiplied.
// LDS addresses are the lanes' in order, so the swizzle that keeps the operand
// reads free of bank conflicts permutes the 16-byte pieces of a row on the
// global side.  Pieces beyond k are given an offset beyond the buffer, which
// reads as zero; rows beyond the matrix repeat its last row and are not
// stored.
//
// A stage has four block scales of a row.  Those of four stages are loaded
// together, 16 bytes of every row, for which rows of scales start at multiples
// of four bytes; where k does not give that, a small launch first copies them
// to such rows in the workspace.
//
// 8192 tokens: MXFP4 12288x4096 243 us (3.4 PFLOP/s) and 12288x16384 826 (4.0),
// W4A16 4096x12288 650 (1.27 PFLOP/s); 4095 tokens: W4A4 12288x4096 327 with the
// expansion (1.26).  With zeros for data they take 213, 687, 472 and 262, the rest
// being a clock that power lowers to 1.6 - 1.8 GHz.  The matrix cores are busy for
// 0.72 (W4A16), 0.70 (W4A4) and 0.46 (MXFP4) of the cycles; in the last, LDS reads
// take 0.39 (0.15 of it conflicts of the scale words), direct loads come on top,
// and neither is full: they do not overlap well enough, and tiles end.
// 333 tokens, 4096x12288: MXFP4 24 us, W4A16 51, W4A4 54 (weights cold: 30, 53 and
// 55).  On the MXFP4 ones' 192 CUs the matrix cores are busy for 0.29 and LDS for
// 0.29 of the time: one multiplying wave a SIMD waits for its operands and meets
// a barrier every eight products.
#include "lora_device.hpp"

namespace nvfp4 {

namespace {

// MXFP4: WM x WN waves of 32 TM tokens x 32 TN outputs, stages of 128 channels.
// NL: waves that do nothing but load, so that the others, one a SIMD in the
// small tiles, need not issue it between their products (W4A16 333x4096x12288
// unsplit: 106 us -> 82); 0: all waves load (the large tiles, two a SIMD).
template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
__global__ __launch_bounds__(64 * (WM * WN + NL), NL ? 4 : 2) void mx_tile_kernel(TileArgs a) {
  constexpr int NW = WM * WN, LW = NL ? NL : NW, BM = 32 * TM * WM, BN = 32 * TN * WN, NBUF = AHEAD + 1;
  static_assert((NBUF & AHEAD) == 0, "a power of two of stages");
  constexpr int XB = BM * 64, WB = BN * 64, STAGE = XB + WB;
  using Scales = ScaleStages<BM, BN, LW, AHEAD, false>;
  constexpr int XL = BM / 16 / LW, WL = BN / 16 / LW, LOADS = XL + WL + Scales::STAGE_LOADS;      // of a wave per stage
  static_assert(BM % (16 * LW) == 0 && BN % (16 * LW) == 0, "tile split");
  __shared__ __attribute__((aligned(16))) uint8_t lds[NBUF * STAGE + Scales::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool loads = NL == 0 || wave >= NW, multiplies = wave < NW;
  const int loader = NL ? wave - NW : wave;                                   // (of those that load)
  const uint32_t lds_base = lds_address(lds);
  const TilePos pos = tile_of(a);
  const int t0 = pos.m * BM, o0 = pos.n * BN;
  const int s_begin = (int)((int64_t)a.steps * pos.split / a.splits);
  const int s_end = (int)((int64_t)a.steps * (pos.split + 1) / a.splits);

  const int rows_x = min(BM, a.tokens - t0), rows_w = min(BN, a.out - o0);
  const auto bx = make_buffer(a.x + (int64_t)t0 * a.ldx, (uint32_t)((int64_t)rows_x * a.ldx));
  const auto bw = make_buffer(a.w + (int64_t)o0 * a.ldw, (uint32_t)((int64_t)rows_w * a.ldw));
  const Scales scales(a, lds_base + NBUF * STAGE, t0, rows_x, o0, rows_w, s_begin, loader);
  // this lane's part of the loads: 4 lanes per 64-byte row
  uint32_t xo[XL], wo[WL];
  const int piece = (lane & 3) ^ swizzle64(lane >> 2);
#pragma unroll
  for (int i = 0; i < XL; ++i)
    xo[i] = (uint32_t)(min((loader + i * LW) * 16 + (lane >> 2), rows_x - 1) * a.ldx + piece * 16);
#pragma unroll
  for (int i = 0; i < WL; ++i)
    wo[i] = (uint32_t)(min((loader + i * LW) * 16 + (lane >> 2), rows_w - 1) * a.ldw + piece * 16);

  const uint32_t lds_wave = lds_base + loader * 1024;
  auto load_stage = [&](int s, auto whole) {
    const uint32_t dst = lds_wave + (s & (NBUF - 1)) * STAGE;
    const bool cut = !whole && s * 128 + piece * 32 >= a.k;                   // this lane's piece lies beyond k
    each<XL>([&](auto i) { load_lds16<i * LW * 1024>(bx, dst, cut ? kBeyond : xo[i], s * 64); });
    each<WL>([&](auto i) { load_lds16<XB + i * LW * 1024>(bw, dst, cut ? kBeyond : wo[i], s * 64); });
    scales.load_with(s);
  };

  const int wm = wave % WM, wn = wave / WM, half = lane >> 5, l32 = lane & 31;
  const int frag = l32 * 64 + ((half ^ swizzle64(l32)) << 4);                 // piece `half`; ^ 32 gives piece 2 + half
  const int xf = wm * TM * 32 * 64 + frag, wf = XB + wn * TN * 32 * 64 + frag;
  const int xsf = NBUF * STAGE + wm * TM * 512, wsf = NBUF * STAGE + (BM + wn * TN * 32) * 16;
  uint4 xr[2][TM], wr[2][TN];
  uint32_t xsr[TM], wsr[TN], xs_next[TM], ws_next[TN];
  auto read_scales = [&](int s) {
    const uint8_t* b = lds + scales.place(s, l32);
#pragma unroll
    for (int i = 0; i < TM; ++i) xs_next[i] = *reinterpret_cast<const uint32_t*>(b + xsf + i * 512);
#pragma unroll
    for (int i = 0; i < TN; ++i) ws_next[i] = *reinterpret_cast<const uint32_t*>(b + wsf + i * 512);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i) xsr[i] = xs_next[i] >> (8 * half);
#pragma unroll
    for (int i = 0; i < TN; ++i) wsr[i] = ws_next[i] >> (8 * half);
  };
  auto read_frags = [&](int set, int s) {
    const uint8_t* b = lds + (s & (NBUF - 1)) * STAGE;
#pragma unroll
    for (int i = 0; i < TM; ++i) xr[set][i] = *reinterpret_cast<const uint4*>(b + ((xf + i * 2048) ^ (set * 32)));
#pragma unroll
    for (int i = 0; i < TN; ++i) wr[set][i] = *reinterpret_cast<const uint4*>(b + ((wf + i * 2048) ^ (set * 32)));
  };

  f32x16 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] = 0.0f;

  auto multiply = [&](int set) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int m = 0; m < TM; ++m)
        acc[n][m] = mfma32_mx(wr[set][n], wsr[n], xr[set][m], xsr[m], acc[n][m], set);
    __builtin_amdgcn_sched_barrier(0);
  };

  if (loads) {
    scales.load_first();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (s_begin + i < s_end) load_stage(s_begin + i, std::false_type{});
    if (s_begin + AHEAD <= s_end) wait_loads<(AHEAD - 1) * LOADS>();
    else wait_loads<0>();
  }
  stage_barrier();
  if (multiplies) {
    read_scales(s_begin);
    read_frags(0, s_begin);
  }
  // on to stage s + 1, in one of the ways below
  auto next_stage = [&](int s, auto way) {
    if constexpr (way == kLast) return;
    if (loads) wait_loads<way == kDrain ? 0 : (AHEAD - 2) * LOADS>();
    stage_barrier();
    if constexpr (way == kWhole || way == kCut)
      if (loads) load_stage(s + AHEAD, std::bool_constant<way == kWhole>{});
  };
  if (NL && loads) {
    run_stages<AHEAD>(s_begin, s_end, a.k >> 7, next_stage);
  } else {
    run_stages<AHEAD>(s_begin, s_end, a.k >> 7, [&](int s, auto way) {
      take_scales();
      read_frags(1, s);
      multiply(0);
      next_stage(s, way);
      if constexpr (way != kLast) {
        read_scales(s + 1);
        read_frags(0, s + 1);
      }
      multiply(1);
    });
  }
  __syncthreads();                                                // the stages are done with
  static_assert(NW * 32 * (64 * TN + 16) <= sizeof(lds), "store staging");
  if (!multiplies) return;
  store_tiles<TN, TM>(a, acc, o0 + wn * TN * 32, t0 + wm * TM * 32, pos.split, lds + wave * 32 * (64 * TN + 16));
}

// 16-bit activations x NVFP4 weights (with an adapter's term).
template <bool F16, int TM, int TN, int WM, int WN, int NL, int AHEAD, typename... Lora>
__global__ __launch_bounds__(64 * (WM * WN + NL), NL && AHEAD == 2 ? 4 : 2) void nv_tile_kernel(TileArgs a, Lora... lora) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::LDS];
  const TilePos pos = tile_of(a);
  const int t0 = pos.m * T::BM, o0 = pos.n * T::BN;
  const int s_begin = (int)((int64_t)a.steps * pos.split / a.splits);
  const int s_end = (int)((int64_t)a.steps * (pos.split + 1) / a.splits);

  const int rows_x = min(T::BM, a.tokens - t0), rows_w = min(T::BN, a.out - o0);
  // the last row ends with its k channels, not with its stride
  const auto bx = make_buffer(a.x + (int64_t)t0 * a.ldx, (uint32_t)((int64_t)(rows_x - 1) * a.ldx + (int64_t)a.k * 2));
  const auto bw = make_buffer(a.w + (int64_t)o0 * a.ldw, (uint32_t)((int64_t)rows_w * a.ldw));
  const int loader = loader_of<T::NW, NL>();
  const typename T::Scales scales(a, lds_address(lds) + T::NBUF * T::STAGE, 0, 0, o0, rows_w, s_begin, loader);
  static_assert(T::NW * 32 * (64 * TN + 16) <= T::LDS, "store staging");
  nv_tile<F16, TM, TN, WM, WN, NL, AHEAD>(
      bx, bw, a.k, s_begin, s_end, [&](int row) { return (uint32_t)(min(row, rows_x - 1) * a.ldx); },
      [&](int row) { return (uint32_t)(min(row, rows_w - 1) * a.ldw); }, scales, lds,
      [&](f32x16 (&acc)[TN][TM], int wm, int wn, int wave, bool multiplies) {
        const int o = o0 + wn * TN * 32, t = t0 + wm * TM * 32;
        (add_lora<TN, TM, T::BM, T::LDS, T::THREADS>(lora, a.tokens, a.out, acc, multiplies, o, t0, wm * TM * 32, pos.split, a.splits,
                                         lds),
         ...);
        if (!multiplies) return;
        store_tiles<TN, TM>(a, acc, o, t, pos.split, lds + wave * 32 * (64 * TN + 16));
      });
}

struct PrepArgs {
  const uint8_t* ws;          // weight scales [out][nb] to go to rows of `steps` words, zero past nb
  uint32_t* wdst;             // (NULL: they stay where they are)
  const uint8_t* xs;          // the same of the tokens (MXFP4)
  uint32_t* xdst;
  const uint8_t* xp;          // W4A4: packed tokens, expanded to fp16 [tokens][k] at xh
  const uint8_t* xc;
  uint16_t* xh;
  int tokens, out, nb, steps, k;
};

// What the tile kernels want laid out differently, one thread a scale word or
// 16-channel block.
__device__ __forceinline__ void scale_word(const uint8_t* src, int nb, uint32_t* dst, int steps, int64_t i) {
  const int64_t row = i / steps;
  const int step = (int)(i - row * steps);
  uint32_t v = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (step * 4 + b < nb) v |= (uint32_t)src[row * nb + step * 4 + b] << (8 * b);
  dst[i] = v;
}

__global__ __launch_bounds__(256) void prep_kernel(PrepArgs a) {
  const int64_t nw = a.wdst ? (int64_t)a.steps * a.out : 0, nx = a.xdst ? (int64_t)a.steps * a.tokens : 0;
  const int64_t nh = a.xh ? (int64_t)a.tokens * (a.k >> 4) : 0;
  const int64_t total = nw + nx + nh, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    if (i < nw) {
      scale_word(a.ws, a.nb, a.wdst, a.steps, i);
    } else if (i < nw + nx) {
      scale_word(a.xs, a.nb, a.xdst, a.steps, i - nw);
    } else {
      const int64_t b = i - nw - nx;
      const uint2 q = *reinterpret_cast<const uint2*>(a.xp + b * 8);
      const f16x2 s = splat_f16(e4m3_f32<0>(a.xc[b]));
      uint4* dst = reinterpret_cast<uint4*>(a.xh + b * 16);
      dst[0] = fp4x8_f16(q.x, s);
      dst[1] = fp4x8_f16(q.y, s);
    }
  }
}

// y = RN_bf16(s0 s1 sum over splits), in split order.
__global__ __launch_bounds__(256) void join_kernel(TileArgs a) {
  const int64_t quads = a.ldp >> 2, total = a.tokens * quads;
  float s0 = 1.0f, s1 = 1.0f;
  if (a.s0) s0 = *a.s0;
  if (a.s1) s1 = *a.s1;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / quads;
    const int o = (int)(i % quads) * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(a.partial + t * a.ldp + o);
    for (int s = 1; s < a.splits; ++s)
      v += *reinterpret_cast<const f32x4*>(a.partial + ((int64_t)s * a.tokens + t) * a.ldp + o);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (o + e < a.out) a.y[t * a.ldy + o + e] = to_bf16(v[e] * s0 * s1);
  }
}

constexpr int kCus = 256;

// How a product is cut.  Large tiles where they fill the card and more than half
// of their rows are tokens (a small tile's time goes by its rows, a large one's
// too: 128 tokens of 151936x4096 take 119 us in large tiles and 94 in small ones
// (MXFP4), 302 and 184 (W4A16), 291 and 184 (W4A4); 129 take 119 and 126, 302 and
// 305, 290 and 299), else tiles of 128 x 128, with the channels split where that
// is quicker: a stage of such a tile takes 0.29 us (MXFP4) or 0.37, 1.4 times that
// where two share a CU, and a split costs a launch and a trip of its fp32 partial
// sums through memory.  MXFP4, 333 tokens: 4096x4096 takes 13.5 us whole and 17.3
// in two, 4096x12288 32.6 and 26.3 (one set of weights, in the MALL).
struct Plan {
  int rows, cols;                        // of a tile: tokens x outputs
  int tiles_m, tiles_n, splits, steps;
  bool pad;                              // the scales' rows are no multiples of 4 bytes
  size_t xs, ws, xh, partial, bytes;     // workspace offsets
};

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

Plan plan_product(int64_t tokens, int64_t out, int64_t k, bool mx) {
  Plan p{};
  const int span = mx ? 128 : 64;        // channels of a stage: four scales
  p.steps = (int)((k + span - 1) / span);
  p.pad = k % span != 0;
  const bool many = out >= INT64_C(1) << 26;                      // more small tiles than a launch has places
  const bool large = (tokens > 128 || many) && (tokens + 255) / 256 * ((out + 255) / 256) >= kCus * 3 / 4;
  p.rows = p.cols = large ? 256 : 128;
  p.tiles_m = (int)((tokens + p.rows - 1) / p.rows);
  p.tiles_n = (int)((out + p.cols - 1) / p.cols);
  p.splits = 1;
  if (!large) {
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    const double stage = mx ? 0.29 : 0.37, launch = 3.0, partial = (double)tokens * out * 8 / 4e6;       // us; 4 TB/s
    double best = 0;
    for (int n = 1; n <= 16 && (n == 1 || n * 8 <= p.steps); ++n) {
      const int64_t all = tiles * n, rounds = (all + 2 * kCus - 1) / (2 * kCus);
      const double us = (all <= kCus ? 1.0 : 1.4 * (double)rounds) * ((p.steps + n - 1) / n) * stage +
                        (n > 1 ? launch + partial * n : 0);
      if (n == 1 || us < best) {
        best = us;
        p.splits = n;
      }
    }
  }
  size_t at = 0;
  p.ws = at;
  if (p.pad) at = align256(at + (size_t)p.steps * out * 4);
  p.xs = at;
  if (p.pad && mx) at = align256(at + (size_t)p.steps * tokens * 4);
  p.xh = at;
  if (!mx) at = align256(at + (size_t)tokens * k * 2);                        // used by W4A4 only
  p.partial = at;
  if (p.splits > 1) at = align256(at + (size_t)p.splits * tokens * ((out + 3) / 4 * 4) * 4);
  p.bytes = at;
  return p;
}

// The launch that follows a tile kernel: joins the channel splits.
int join(const TileArgs& a, hipStream_t s) {
  int st = launch_status("tile kernel");
  if (st || a.splits == 1) return st;
  const int64_t quads = (int64_t)a.tokens * (a.ldp >> 2);
  const int64_t want = (quads + 255) / 256;
  join_kernel<<<(unsigned)(want < 4096 ? want : 4096), 256, 0, s>>>(a);
  return launch_status("join_kernel");
}

unsigned tile_grid(const TileArgs& a) { return (unsigned)(a.tiles_m * a.tiles_n * a.splits); }

template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
int run_mx(const TileArgs& a, hipStream_t s) {
  mx_tile_kernel<TM, TN, WM, WN, NL, AHEAD><<<tile_grid(a), 64 * (WM * WN + NL), 0, s>>>(a);
  return join(a, s);
}

template <bool F16, int TM, int TN, int WM, int WN, int NL, int AHEAD, typename... Lora>
int run_nv(const TileArgs& a, hipStream_t s, const Lora&... lora) {
  nv_tile_kernel<F16, TM, TN, WM, WN, NL, AHEAD, Lora...><<<tile_grid(a), 64 * (WM * WN + NL), 0, s>>>(a, lora...);
  return join(a, s);
}

int launch_prep(const PrepArgs& a, hipStream_t s) {
  const int64_t total = (a.wdst ? (int64_t)a.steps * a.out : 0) + (a.xdst ? (int64_t)a.steps * a.tokens : 0) +
                        (a.xh ? (int64_t)a.tokens * (a.k >> 4) : 0);
  if (total == 0) return NVFP4_OK;
  const int64_t want = (total + 255) / 256;
  prep_kernel<<<(unsigned)(want < 8192 ? want : 8192), 256, 0, s>>>(a);
  return launch_status("prep_kernel");
}

// What is the same for both kinds of product.
TileArgs tile_args(const Plan& p, const PrepArgs& q, int64_t tokens, int64_t out, int64_t k, const uint8_t* wp,
                   uint16_t* y, int64_t ldy, uint8_t* base) {
  TileArgs a{};
  a.w = wp;
  a.xs = q.xdst ? reinterpret_cast<const uint8_t*>(q.xdst) : q.xs;
  a.ws = q.wdst ? reinterpret_cast<const uint8_t*>(q.wdst) : q.ws;
  a.lds = p.steps * 4;
  a.y = y;
  a.partial = reinterpret_cast<float*>(base + p.partial);
  a.ldw = k / 2;
  a.ldy = ldy;
  a.ldp = (out + 3) / 4 * 4;
  a.tokens = (int)tokens;
  a.out = (int)out;
  a.k = (int)k;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.splits = p.splits;
  a.steps = p.steps;
  return a;
}

}  // namespace

// Byte offsets inside a tile's rows stay below 2^31, and the threads of a launch
// below 2^32: a tile, large or small, has at most 512.  Small ones, in up to 16
// parts, are used in place of fewer than 3/4 kCus large ones, or fewer than 2^19
// of them for up to 128 tokens.
bool tile_product_fits(int64_t tokens, int64_t out, int64_t k, int64_t ldx_bytes) {
  const int64_t lim = INT64_C(1) << 31, threads = 512;
  return 256 * ldx_bytes < lim && 256 * k < lim && (out + 255) / 256 * ((tokens + 255) / 256) < 2 * lim / threads;
}

size_t tile_product_workspace(int64_t tokens, int64_t out, int64_t k, bool mx) {
  return plan_product(tokens, out, k, mx).bytes;
}

int launch_tile_mx(const uint8_t* xp, const uint8_t* xe, int64_t tokens, int64_t k, const uint8_t* wp, const uint8_t* we,
                   int64_t out, uint16_t* y, int64_t ldy, void* workspace, hipStream_t s) {
  const Plan p = plan_product(tokens, out, k, true);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  PrepArgs q{};
  q.ws = we;
  q.xs = xe;
  if (p.pad) {
    q.wdst = reinterpret_cast<uint32_t*>(base + p.ws);
    q.xdst = reinterpret_cast<uint32_t*>(base + p.xs);
  }
  q.tokens = (int)tokens;
  q.out = (int)out;
  q.nb = (int)(k / 32);
  q.steps = p.steps;
  q.k = (int)k;
  const int st = launch_prep(q, s);
  if (st) return st;
  TileArgs a = tile_args(p, q, tokens, out, k, wp, y, ldy, base);
  a.x = xp;
  a.ldx = k / 2;
  if (p.rows == 256) return run_mx<4, 2, 2, 4, 0, 3>(a, s);
  return run_mx<2, 2, 2, 2, 4, 3>(a, s);
}

int launch_tile_nv(const uint16_t* x, int64_t ldx, const uint8_t* xp, const uint8_t* xc, const float* xs2, int64_t tokens,
                   int64_t k, const uint8_t* wp, const uint8_t* wc, const float* ws2, int64_t out, uint16_t* y,
                   int64_t ldy, void* workspace, hipStream_t s, const LoraTerm* lora) {
  const Plan p = plan_product(tokens, out, k, false);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const bool f16 = xp != nullptr;
  PrepArgs q{};
  q.ws = wc;
  if (p.pad) q.wdst = reinterpret_cast<uint32_t*>(base + p.ws);
  q.xp = xp;
  q.xc = xc;
  q.xh = f16 ? reinterpret_cast<uint16_t*>(base + p.xh) : nullptr;
  q.tokens = (int)tokens;
  q.out = (int)out;
  q.nb = (int)(k / 16);
  q.steps = p.steps;
  q.k = (int)k;
  const int st = launch_prep(q, s);
  if (st) return st;
  TileArgs a = tile_args(p, q, tokens, out, k, wp, y, ldy, base);
  a.x = reinterpret_cast<const uint8_t*>(f16 ? q.xh : x);
  a.s0 = ws2;
  a.s1 = xs2;
  a.ldx = (f16 ? k : ldx) * 2;
  // one tile a CU: more stages ahead in LDS; more: two share it
  const bool alone = (int64_t)p.tiles_m * p.tiles_n * p.splits <= kCus;
  if (lora) {                                        // (the term comes with the tensor scale applied)
    a.s0 = nullptr;
    if (p.rows == 256) return run_nv<false, 4, 2, 2, 4, 0, 2>(a, s, *lora);
    return alone ? run_nv<false, 4, 1, 1, 4, 4, 6>(a, s, *lora) : run_nv<false, 4, 1, 1, 4, 4, 2>(a, s, *lora);
  }
  if (f16) {
    if (p.rows == 256) return run_nv<true, 4, 2, 2, 4, 0, 2>(a, s);
    return alone ? run_nv<true, 2, 2, 2, 2, 4, 6>(a, s) : run_nv<true, 2, 2, 2, 2, 4, 2>(a, s);
  }
  if (p.rows == 256) return run_nv<false, 4, 2, 2, 4, 0, 2>(a, s);
  return alone ? run_nv<false, 4, 1, 1, 4, 4, 6>(a, s) : run_nv<false, 4, 1, 1, 4, 4, 2>(a, s);
}

}  // namespace nvfp4
