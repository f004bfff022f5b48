// A mixture-of-experts layer over NVFP4 experts for any number of tokens, in the
// layout the MXFP4 -> NVFP4 cast leaves them (w1 and w3 of an expert share a
// tensor scale, "从MXFP4到NVFP4：Model Optimizer混合精度格式转换完全攻略" §3):
//
//   y[t] = sum over the experts e chosen for t of
//          weight(t, e) * W2_e ( silu(W1_e x[t]) * (W3_e x[t]) )
//
// The choices are sorted by expert, so that an expert's tokens are rows of row
// tiles of its own, which the sort lists.  Two launches that multiply fp16 rows by
// packed NVFP4 weights go over that list: the first reads the tokens where they are
// and makes h = silu(gate) * up, the second makes weight * s2 * W2 h, a row for
// every choice, and a last launch adds the rows of each token.  The number of row
// tiles is known on the device only; the grids are for the most there can be, and
// workgroups past the last tile end at once.
//
// Rounded on the way: h and the rows, both to the 11 bits of fp16 with a power of two of
// their own for every 32 columns, which halves what moves; in bf16, of the same size,
// either would be off by as much as y's own rounding.  x and h enter the products as
// fp16 with a power of two a row, exact but for values far below a row's largest.
//
// 8 of 128 experts of 7168 x 2048, by the card (a library's bf16 product of 8192^3 makes
// 1.18 to 1.37 PFLOP/s on them): 100 tokens 0.62 to 0.65 ms (weights that cross memory
// at 5 TB/s), 1023 tokens 1.13 to 1.20 ms (bound by neither memory nor matrix units,
// which are 42% busy: half the experts have more than 64 rows and are multiplied as
// 96), 8192 tokens 5.64 to 5.93 ms (0.97 to 1.02 PFLOP/s; the clocks fall to 1.7 GHz
// under the matrix units' power).  Figures of one comparison below are of one card, and
// of the form that the kernels had when it was made.
#include "layer.hpp"
#include "tile_device.hpp"

namespace nvfp4 {

namespace {

struct SortedArgs {
  const uint16_t* x;               // fp16 rows of the tokens, [tokens][hidden]
  uint32_t x_bytes;                // of all of them, below 2^31
  const int32_t* order;            // choice of a sorted row
  const ExpertBand* bands;
  const int* count;                // of bands
  const float* row_weight;         // by row: the choice's weight,
  const float* row_scale;          // the token's power of two: value = fp16 * scale
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
  uint16_t* h;                     // fp16 [rows][inter]
  uint8_t* he;                     // its exponents, [rows][ldhe], until each row has one (which goes into row_weight)
  uint16_t* ys;                    // fp16 [rows][hidden]
  uint8_t* ye;                     // their exponents, [rows][lde]
  int ldhe, lde;
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

// x: bf16 rows in fp16 with a power of two each that puts the largest below 2^15: exact,
// but for values 2^29 and more below that, which are rounded to its 2^-39.  fp16
// weights take half the work of bf16 ones to make, which is much of what a tile of few
// rows has to do (100 tokens of 128 experts of 7168 x 2048, first product 600 us in
// bf16, 550 so).  Row t goes to y + t cols; scale[t] gets the power.
// The first 2048 HELD columns stay in registers: read once, all on their way at a time
// (rows of 2048 columns, 1023 x 8 of them: 16 us with 1, 23 with 4).
template <int HELD>
__global__ __launch_bounds__(256) void half_rows_kernel(const uint16_t* x, int64_t ldx, int64_t rows, int pieces,
                                                        uint16_t* y, float* scale) {
  __shared__ float part[4];
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(x + t * ldx);
    f16x8* const dst = reinterpret_cast<f16x8*>(y + t * (int64_t)pieces * 8);
    uint4 held[HELD];
#pragma unroll
    for (int z = 0; z < HELD; ++z) {
      const int i = threadIdx.x + 256 * z;
      held[z] = i < pieces ? src[i] : make_uint4(0, 0, 0, 0);
    }
    float top = 0.f;
#pragma unroll
    for (int z = 0; z < HELD; ++z) top = finite_max(held[z], top);
    for (int i = threadIdx.x + 256 * HELD; i < pieces; i += 256) top = finite_max(src[i], top);
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const int e = max((int)(__float_as_uint(top) >> 23), 15);
    const float f = __uint_as_float((uint32_t)(127 + kHalfBias - e) << 23);
    const auto put = [&](int i, const uint4& v) {
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
      f16x8 h;
#pragma unroll
      for (int z = 0; z < 8; ++z)
        h[z] = (_Float16)(__uint_as_float(z & 1 ? q[z >> 1] & 0xFFFF0000u : q[z >> 1] << 16) * f);
      dst[i] = h;
    };
#pragma unroll
    for (int z = 0; z < HELD; ++z)
      if ((int)threadIdx.x + 256 * z < pieces) put(threadIdx.x + 256 * z, held[z]);
    for (int i = threadIdx.x + 256 * HELD; i < pieces; i += 256) put(i, src[i]);
    if (threadIdx.x == 0) scale[t] = __builtin_amdgcn_ldexpf(1.0f, e - kHalfBias);
    __syncthreads();                                 // before the next row's maximum
  }
}

// h: from an exponent for every 32 columns to one a row, their largest, which weight[row]
// is multiplied by; in place, and only the columns that change.  Exact, but for values
// 2^29 and more below the row's largest: with h's own rounding they are off by 2^-38 of
// that at most.  A workgroup a row; those behind the last are left alone.  (8192 x 8 rows
// of 2048: 84 us, 108 with what is to change asked for when the exponents are there.)
__global__ __launch_bounds__(256) void one_exponent_kernel(uint16_t* h, const uint8_t* exponents, int lde, int pieces,
                                                           const int32_t* rows, float* weight) {
  const int64_t t = blockIdx.x;
  if ((int)t >= *rows) return;
  const uint8_t* const of = exponents + t * lde;
  f16x8* const row = reinterpret_cast<f16x8*>(h + t * (int64_t)pieces * 8);
  int i = threadIdx.x, e = of[min(i, pieces - 1) >> 2];
  f16x8 v = row[min(i, pieces - 1)];                 // on its way beside the exponents
  int top = 0;
  for (int z = threadIdx.x & 63; z < lde; z += 64) top = max(top, (int)of[z]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top = max(top, __shfl_xor(top, m));
  while (i < pieces) {
    if (e < top) {                                   // (64 powers below, a finite value is nothing; an infinity stays)
      const float f = __builtin_amdgcn_ldexpf(1.0f, max(e - top, -64));
#pragma unroll
      for (int z = 0; z < 8; ++z) v[z] = (_Float16)((float)v[z] * f);
      row[i] = v;
    }
    i += 256;
    if (i >= pieces) break;
    e = of[i >> 2];
    v = row[i];
  }
  if (threadIdx.x == 0) weight[t] = __builtin_amdgcn_ldexpf(weight[t], top - kHalfBias);
}

// A row tile and run of output rows.
struct TileAt { int expert, first, rows, n; };
// Those that a workgroup of the tile kernels takes: false past the last.  Consecutive
// workgroups go to the 8 XCDs in turn, and so do bands, two row tiles of an expert; of
// a band, all output rows of the first come before those of the second.  What an XCD's
// CUs work on at one time is then one or two experts, whose weights its L2 hands to
// both row tiles (8192 tokens, 8 of 128 experts of 7168 x 2048: the first product
// fetches 8 GB; the layer took 5.80 ms with each row tile on another XCD, 5.59 so).  The
// list has the bands of most rows first, by 32: the XCDs have as much to do, and what
// is left at the end is short (1023 tokens 1.25 ms by 128 rows, 1.20 so).
constexpr int kBandTiles = 2;
__device__ __forceinline__ bool expert_tile(const SortedArgs& a, int tiles_n, TileAt& t) {
  constexpr int ROWS = 128;
  const uint32_t xcd = blockIdx.x & 7, i = blockIdx.x >> 3, per = kBandTiles * tiles_n;
  const uint32_t at = i / per * 8 + xcd, m = i % per / tiles_n;
  if (at >= (uint32_t)*a.count) return false;
  const ExpertBand v = a.bands[at];
  t.expert = __builtin_amdgcn_readfirstlane(v.expert);
  t.first = __builtin_amdgcn_readfirstlane(v.first + m * ROWS);
  t.rows = __builtin_amdgcn_readfirstlane(min(v.rows - (int)m * ROWS, ROWS));
  t.n = __builtin_amdgcn_readfirstlane(i % per % tiles_n);
  return t.rows > 0;
}

// (a conditional on the variables themselves would choose among their addresses,
// which puts them in memory)
__device__ __forceinline__ uint32_t beyond_if(bool cut, uint32_t offset) { return cut ? kBeyond : offset; }

// The tile kernels' form: 4 waves, 64 output rows each; a row tile has up to 128 rows,
// and the workgroup takes the least multiple of 32 that holds it, so that products of
// rows that are not there are left out.  Two workgroups share a CU (one of 256 x 256,
// whose start and end nothing hides: 6.2 ms against 5.9 for 8192 tokens).
//
// A stage is 64 channels.  What bounds the tiles of few rows is how many pieces of
// cache lines are asked for, how many are on their way, and how often a line of scales,
// which serves 32 stages, leaves the L2 between two of them: weights come two stages at
// a time, 64 bytes a row, and scales eight or sixteen, 32 or 64 bytes a row (parts of
// the rows with each pair).  LDS keeps two pairs of weights, two groups of scales and
// two stages of x, three where rows are few; when something takes a place, what was
// there has been read.  (100, 256 and 1023 tokens of 128 experts of 7168 x 2048 in us:
// 670, 765, 1165.  Groups of eight stages and three pairs for 32 rows: 690, 785, 1170.
// A stage of each at a time, 32 and 16 bytes a row: 847, 932, 1350.  A stage of 256
// channels, 128 bytes a row, one workgroup of 16 waves a CU: 692, 878, 1735.)
struct Tiles {
  static constexpr int TN = 2, WAVES = 4, ROWS = 128, BN = 32 * TN * WAVES, THREADS = 64 * WAVES;
  static constexpr int PAIR = BN * 64;                           // weights of two stages
  static constexpr int WL = PAIR / 1024 / WAVES;                 // loads of a wave
  static constexpr int x_kept(int tm) { return tm == 1 ? 3 : 2; }             // stages of x; of weights two pairs
  static constexpr int group(int tm) { return tm <= 2 ? 16 : 8; }             // stages of a group of scales
  static constexpr int LDS = 80 * 1024;
};
static_assert(Tiles::WAVES * 32 * (64 * Tiles::TN + 16) <= Tiles::LDS && 2 * Tiles::LDS <= 160 * 1024,
              "store staging; two workgroups a CU");

// One tile of 32 TM rows: acc[n][m] as store_tiles takes it, to finish(acc, wave).
//   bx, bw, bs     buffers of the rows, the packed weights and their scales (stride bytes
//                  a row, scale_bytes in all)
//   x_at(row), w_at(row)   the bytes in them at which the tile's rows begin
//   PAIRED         of 32 rows of the tile the first 16 and the others are as many rows of
//                  two matrices, whose scales are `pair` bytes apart
// Lane half h of an instruction takes channels 32 h + 8 j .. + 7 of the stage at step
// j, so that a lane's weights of a stage are one 16-byte piece.
template <bool PAIRED, int TM, typename XAt, typename WAt, typename Finish>
__device__ __forceinline__ void run_tile(i32x4 bx, i32x4 bw, i32x4 bs, int k, XAt x_at, WAt w_at, int stride,
                                         uint32_t scale_bytes, int pair, uint8_t* lds, Finish finish) {
  constexpr int TN = Tiles::TN, WAVES = Tiles::WAVES, WL = Tiles::WL;
  constexpr int X = Tiles::x_kept(TM), XB = TM * 4096, W_AT = X * XB, S_AT = W_AT + 2 * Tiles::PAIR;
  constexpr int G = Tiles::group(TM), GROUP = Tiles::BN * 4 * G, GR = 64 / G;  // GR: rows of scales a wave loads at a time
  static_assert(S_AT + 2 * GROUP <= Tiles::LDS && (G == 8 || G == 16), "stages");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31, end = (k + 63) >> 6;
  const uint32_t lds_wave = lds_address(lds) + wave * 1024;
  const int x_bytes = bx[2], w_bytes = bw[2];        // the buffers' sizes, below 2^31
  // loads of x: 8 rows each; of weights: 16 rows
  uint32_t xo[TM], wo[WL];
  const int xpiece = (lane & 7) ^ swizzle128(wave * 8 + (lane >> 3));
  const int wpiece = (lane & 3) ^ swizzle64(lane >> 2);
#pragma unroll
  for (int i = 0; i < TM; ++i) xo[i] = x_at((wave + i * WAVES) * 8 + (lane >> 3)) + xpiece * 16;
#pragma unroll
  for (int i = 0; i < WL; ++i) wo[i] = w_at((wave + i * WAVES) * 16 + (lane >> 2)) + wpiece * 16;
  // Of scales: GR rows, block e WAVES + wave of the tile's; word w of a row lies at place
  // w ^ (row / GR % G), so that 32 rows' words lie in as many banks.
  const int s_row = wave * GR + lane / G;            // of the first WAVES GR
  const uint32_t so = (uint32_t)(s_row & (PAIRED ? 15 : 31)) * stride + (PAIRED ? (s_row >> 4) * pair : 0);

  // Loads run ahead of the last stage: past k a lane's offset is beyond the buffer, which
  // reads as zero, and the scalar offset is held to the buffer's size, without which the
  // bounds check (lane's offset against size less scalar offset) could wrap: a tile of
  // one row has 2 k bytes of x, and a stage that begins behind them is loaded all the same.
  const auto load_x = [&](int s, int buf, auto whole) {
    const bool cut = !whole && s * 64 + xpiece * 8 >= k;
    const uint32_t dst = lds_wave + buf * XB;
    const int base = min(s * 128, x_bytes);
    each<TM>([&](auto i) { load_lds16<i * WAVES * 1024>(bx, dst, beyond_if(cut, xo[i]), base); });
  };
  const auto load_w = [&](int p, int buf) {
    const bool cut = p * 128 + wpiece * 32 >= k;
    const uint32_t dst = lds_wave + buf * Tiles::PAIR;
    const int base = min(p * 64, w_bytes);
    each<WL>([&](auto i) { load_lds16<W_AT + i * WAVES * 1024>(bw, dst, beyond_if(cut, wo[i]), base); });
  };
  // (words past a row's end: read, not used)
  const auto load_scales = [&](int i) {                          // part i % G of group i / G
    const int g = i / G, e = i % G, row = e * WAVES * GR;
    const uint32_t base = (uint32_t)(g * 4 * G + (PAIRED ? (row >> 5) * 16 * stride + (row >> 4 & 1) * pair : row * stride));
    load_lds4<S_AT>(bs, lds_address(lds) + (g & 1) * GROUP + (e * WAVES + wave) * 256,
                    so + (((lane ^ (e * WAVES + wave)) & (G - 1)) << 2),
                    (int)min(base, scale_bytes));
  };

  uint4 xr[2][TM], wr[TN], wr_next[TN];
  uint32_t wsr[TN], wsr_next[TN];
  const int x_row = l32 * 128, w_row = (wave * TN * 32 + l32);
  const auto read_x = [&](int set, int j, int buf) {
    const uint8_t* b = lds + buf * XB + x_row + (((4 * half + j) ^ swizzle128(l32)) << 4);
#pragma unroll
    for (int i = 0; i < TM; ++i) xr[set][i] = *reinterpret_cast<const uint4*>(b + i * 4096);
  };
  const auto read_w = [&](int s, int buf) {
    const uint8_t* b = lds + W_AT + buf * Tiles::PAIR + w_row * 64 + (((2 * (s & 1) + half) ^ swizzle64(l32)) << 4);
    const uint8_t* c = lds + S_AT + (s / G & 1) * GROUP + w_row * 4 * G;
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      wr_next[n] = *reinterpret_cast<const uint4*>(b + n * 2048);
      wsr_next[n] = *reinterpret_cast<const uint32_t*>(c + n * 128 * G + (((s % G) ^ (n * 32 / GR) ^ (l32 / GR)) << 2));
    }
  };
  static_assert(TN == 2, "a wave's rows start at a multiple of 64");

  f32x16 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] = 0.0f;

  // What goes on its way at the end of stage s: x of stage s + X, and where s = 2 p + 1
  // parts s + G + 1 and s + G + 2 of scales and pair p + 2.  A group's last parts are
  // there two stages on, before its first stage is read; its first are loaded when the
  // group in whose place they go has been read.
  const auto load_behind = [&](int s, int xbuf, int wbuf, auto whole) {
    load_x(s + X, xbuf, whole);
    if (s & 1) {
      load_scales(s + G + 1);
      load_scales(s + G + 2);
      load_w((s >> 1) + 2, wbuf);
    }
  };
#pragma unroll
  for (int i = 0; i < G; ++i) load_scales(i);
  load_w(0, 0);
  load_x(0, 0, std::false_type{});
  if (X == 3) load_x(1, 1, std::false_type{});
  wait_loads<(X - 2) * TM>();
  stage_barrier();
  load_behind(-1, X - 1, 1, std::false_type{});
  int xbuf = 0, wbuf = 0;                            // stage s's
  read_w(0, 0);
  read_x(0, 0, 0);
  const auto step = [&](int s, auto whole, auto last) {
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      wr[n] = wr_next[n];
      wsr[n] = wsr_next[n] >> (16 * half);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < 3) {
        read_x((j + 1) & 1, j + 1, xbuf);
      } else if constexpr (!last) {
        // Stage s + 1 is to be there, what comes behind its x may be on its way, and all
        // that is read of stage s is in registers.
        if (s & 1) wait_loads<(X - 2) * TM>();
        else wait_loads<(X - 2) * TM + 2 + WL>();
        lds_barrier();
        load_behind(s, xbuf, wbuf, whole);
        xbuf = xbuf == X - 1 ? 0 : xbuf + 1;
        if (s & 1) wbuf ^= 1;
        read_w(s + 1, wbuf);
        read_x(0, 0, xbuf);
      }
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const uint32_t nib = j == 0 ? wr[n].x : j == 1 ? wr[n].y : j == 2 ? wr[n].z : wr[n].w;
        const uint4 w = fp4x8_f16(nib, splat_f16(j < 2 ? e4m3_f32<0>(wsr[n]) : e4m3_f32<1>(wsr[n])));
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[n][m] = mfma32_16<true>(w, xr[j & 1][m], acc[n][m]);
      }
    }
  };
  int s = 0;
  for (; s + X < k >> 6; ++s) step(s, std::true_type{}, std::false_type{});
  for (; s + 1 < end; ++s) step(s, std::false_type{}, std::false_type{});
  step(s, std::false_type{}, std::true_type{});
  wait_loads<0>();                                               // what is still on its way to LDS
  __syncthreads();                                               // the stages are done with
  finish(acc, wave);
}

template <typename Body>
__device__ __forceinline__ void with_rows(int rows, Body f) {
  if (rows <= 32) f(std::integral_constant<int, 1>{});
  else if (rows <= 64) f(std::integral_constant<int, 2>{});
  else if (rows <= 96) f(std::integral_constant<int, 3>{});
  else f(std::integral_constant<int, 4>{});
}

// by[first row + 32 m + the lane's] * s
template <int TM>
struct RowValues {
  float v[TM];
  __device__ __forceinline__ RowValues(const float* by, const TileAt& t, float s) {
#pragma unroll
    for (int m = 0; m < TM; ++m) v[m] = by[t.first + min(32 * m + (int)(threadIdx.x & 31), t.rows - 1)] * s;
  }
};

// The biased exponent to store for the 32 columns of a token that this lane and the one
// 32 on hold: that of the largest finite value, at least 14, so that both powers of
// two are normal floats or, at the end of the range, exact ones.
__device__ __forceinline__ int half_exponent(const f32x16& v) {
  float top = 0.f;
#pragma unroll
  for (int z = 0; z < 16; ++z) top = fmaxf(top, __builtin_fabsf(v[z]));       // (a NaN is passed over)
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
// What those columns are multiplied by: the largest comes below 2^15.
__device__ __forceinline__ float half_factor(int e) { return __uint_as_float((uint32_t)(127 + kHalfBias - e) << 23); }
__device__ __forceinline__ uint32_t half_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// A wave's part of h: 32 channels from ch0 on of the tile's rows (s: what their sums
// are to be multiplied by), through `mine` in LDS so that whole runs are stored.
// (Channels past the last: their up rows' scales are read as zero, so that they are
// nothing or NaN and do not enter the exponent.)
template <int TN, int TM>
__device__ __forceinline__ void put_h(const SortedArgs& a, const TileAt& t, const f32x16 (&acc)[TN][TM],
                                      const RowValues<TM>& s, int ch0, uint8_t* mine) {
  static_assert(TN == 2, "one exponent's channels");
  constexpr int PITCH = 32 * TN + 16, LANES = 2 * TN, ROWS = 64 / LANES;
  const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
  const int piece = lane % LANES, row0 = lane / LANES, ch = ch0 + piece * 8;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    if (32 * m >= t.rows) break;
    f32x16 h;
#pragma unroll
    for (int z = 0; z < 16; ++z) {
      const int i = z >> 3, g = z >> 2 & 1, e = z & 3;
      const float gate = acc[i][m][4 * g + e] * s.v[m], up = acc[i][m][8 + 4 * g + e] * s.v[m];
      h[z] = gate / (1.0f + expf(-gate)) * up;
    }
    const int exponent = half_exponent(h);
    const float f = half_factor(exponent);
#pragma unroll
    for (int z = 0; z < 16; z += 4)                  // channels 2 z + sub .. + 3
      *reinterpret_cast<uint2*>(mine + l32 * PITCH + 4 * z + 2 * sub) =
          make_uint2(half_bits(h[z] * f) | half_bits(h[z + 1] * f) << 16, half_bits(h[z + 2] * f) | half_bits(h[z + 3] * f) << 16);
    if (sub == 0 && 32 * m + l32 < t.rows && ch0 < a.inter)
      a.he[(int64_t)(t.first + 32 * m + l32) * a.ldhe + (ch0 >> 5)] = (uint8_t)exponent;
#pragma unroll
    for (int r = 0; r < 32; r += ROWS) {
      const uint4 v = *reinterpret_cast<const uint4*>(mine + (r + row0) * PITCH + piece * 16);
      const int at = 32 * m + r + row0;
      if (at < t.rows && ch < a.inter) *reinterpret_cast<uint4*>(a.h + (int64_t)(t.first + at) * a.inter + ch) = v;
    }
  }
}

// A wave's part of the rows: 32 TN outputs from o0 on (w as s).
template <int TN, int TM>
__device__ __forceinline__ void put_rows(const SortedArgs& a, const TileAt& t, f32x16 (&acc)[TN][TM],
                                         const RowValues<TM>& w, int o0, uint8_t* mine) {
  constexpr int PITCH = 64 * TN + 16, LANES = 4 * TN, ROWS = 64 / LANES;
  const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
  const int piece = lane % LANES, row0 = lane / LANES, o = o0 + piece * 8;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    if (32 * m >= t.rows) break;
    const int at = t.first + min(32 * m + l32, t.rows - 1);
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
      for (int z = 0; z < 16; ++z) acc[i][m][z] *= w.v[m];
      const int e = half_exponent(acc[i][m]);
      const float f = half_factor(e);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t v[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] = half_bits(acc[i][m][4 * g + z] * f);
        *reinterpret_cast<uint2*>(mine + l32 * PITCH + 64 * i + 16 * g + 2 * sub) =
            make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
      }
      if (sub == 0 && 32 * m + l32 < t.rows && o0 + 32 * i < a.hidden)
        a.ye[(int64_t)at * a.lde + (o0 >> 5) + i] = (uint8_t)e;
    }
#pragma unroll
    for (int r = 0; r < 32; r += ROWS) {
      const uint4 v = *reinterpret_cast<const uint4*>(mine + (r + row0) * PITCH + piece * 16);
      const int to = 32 * m + r + row0;
      if (to < t.rows && o < a.hidden) *reinterpret_cast<uint4*>(a.ys + (int64_t)(t.first + to) * a.hidden + o) = v;
    }
  }
}

// h of a row tile: of every 32 output rows of a tile, 16 are gate rows and 16 the
// up rows of the same channels, so that a lane holds both.
__global__ __launch_bounds__(Tiles::THREADS, 2) void moe_up_tile_kernel(SortedArgs a) {
  constexpr int TN = Tiles::TN, CH = Tiles::BN / 2;  // channels of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tiles::LDS];
  TileAt t;
  if (!expert_tile(a, (a.inter + CH - 1) / CH, t)) return;
  const int ch0 = t.n * CH, left = a.inter - ch0;
  const uint32_t ldw = (uint32_t)a.hidden >> 1, ldx = (uint32_t)a.hidden * 2;
  const int64_t row = (int64_t)t.expert * 2 * a.inter + ch0;
  const int rows_w = 2 * a.inter - ch0;              // to the end of the expert's up rows
  const auto bx = make_buffer(a.x, a.x_bytes);
  const auto bw = make_buffer(a.p13 + row * ldw, (uint32_t)rows_w * ldw);
  const uint32_t bytes_s = (uint32_t)rows_w * a.lds13;
  const auto bs = make_buffer(a.c13 + row * a.lds13, bytes_s);
  with_rows(t.rows, [&](auto tm) {
    constexpr int TM = decltype(tm)::value;
    run_tile<true, TM>(
        bx, bw, bs, a.hidden, [&](int r) { return (uint32_t)(a.order[t.first + min(r, t.rows - 1)] / a.top_k) * ldx; },
        [&](int r) { return (uint32_t)(min((r >> 5) * 16 + (r & 15), left - 1) + ((r >> 4) & 1) * a.inter) * ldw; },
        a.lds13, bytes_s, a.inter * a.lds13, lds, [&](const f32x16 (&acc)[TN][TM], int wave) {
          put_h<TN, TM>(a, t, acc, RowValues<TM>(a.row_scale, t, a.s13[t.expert]), ch0 + wave * TN * 16,
                        lds + wave * 32 * (32 * TN + 16));
        });
  });
}

// The rows of a row tile.
__global__ __launch_bounds__(Tiles::THREADS, 2) void moe_down_tile_kernel(SortedArgs a) {
  constexpr int TN = Tiles::TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Tiles::LDS];
  TileAt t;
  if (!expert_tile(a, (a.hidden + Tiles::BN - 1) / Tiles::BN, t)) return;
  const int o0 = t.n * Tiles::BN, rows_w = min(Tiles::BN, a.hidden - o0);
  const uint32_t ldw = (uint32_t)a.inter >> 1, ldh = (uint32_t)a.inter * 2;
  const int64_t row = (int64_t)t.expert * a.hidden + o0;
  const auto bx = make_buffer(a.h + (int64_t)t.first * a.inter, (uint32_t)t.rows * ldh);
  const auto bw = make_buffer(a.p2 + row * ldw, (uint32_t)rows_w * ldw);
  const uint32_t bytes_s = (uint32_t)rows_w * a.lds2;
  const auto bs = make_buffer(a.c2 + row * a.lds2, bytes_s);
  with_rows(t.rows, [&](auto tm) {
    constexpr int TM = decltype(tm)::value;
    run_tile<false, TM>(
        bx, bw, bs, a.inter, [&](int r) { return (uint32_t)min(r, t.rows - 1) * ldh; },
        [&](int r) { return (uint32_t)min(r, rows_w - 1) * ldw; }, a.lds2, bytes_s, 0, lds,
        [&](f32x16 (&acc)[TN][TM], int wave) {
          put_rows<TN, TM>(a, t, acc, RowValues<TM>(a.row_weight, t, a.s2[t.expert]), o0 + wave * TN * 32,
                           lds + wave * 32 * (64 * TN + 16));
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

int half_rows(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, uint16_t* y, float* scale, hipStream_t s) {
  if (cols <= 2048) half_rows_kernel<1><<<(unsigned)rows, 256, 0, s>>>(x, ldx, rows, (int)(cols / 8), y, scale);
  else half_rows_kernel<4><<<(unsigned)rows, 256, 0, s>>>(x, ldx, rows, (int)(cols / 8), y, scale);
  return launch_status("half_rows_kernel");
}
constexpr int64_t kPassRows = INT64_C(1) << 17;      // choices of one pass, at most
static_assert(kBandRows == kBandTiles * Tiles::ROWS, "bands");

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Plan {
  int64_t tokens;                                    // of a pass, at most
  int64_t max_bands;                                 // of a pass
  bool pad13, pad2;
  size_t order, place, offsets, sort, bands, count, c13, c2, x, xs, row_weight, row_scale, h, he, ys, ye, bytes;
};

Plan plan_layer(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inter) {
  Plan p{};
  // a pass's rows of x have 32-bit offsets
  const int64_t most = ((INT64_C(1) << 31) - 1) / (hidden * 2);
  p.tokens = kPassRows / top_k;
  if (p.tokens > most) p.tokens = most;
  if (p.tokens > tokens) p.tokens = tokens;
  const int64_t n = p.tokens * top_k;
  // a band is whole, or the last one of an expert that has rows
  p.max_bands = n / kBandRows + (n < experts ? n : experts);
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
  p.row_weight = take(n * 4);
  p.row_scale = take(n * 4);
  p.h = take(n * inter * 2);
  p.he = take(n * ((inter + 31) / 32));
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
  int32_t* const offsets = reinterpret_cast<int32_t*>(base + p.offsets);
  BandList list{};
  list.bands = reinterpret_cast<ExpertBand*>(base + p.bands);
  list.count = reinterpret_cast<int*>(base + p.count);
  list.scales = reinterpret_cast<const float*>(base + p.xs);
  list.row_weight = reinterpret_cast<float*>(base + p.row_weight);
  list.row_scale = reinterpret_cast<float*>(base + p.row_scale);
  list.top_k = top_k;
  a.order = order;
  a.bands = list.bands;
  a.count = list.count;
  a.row_weight = list.row_weight;
  a.row_scale = list.row_scale;
  a.p13 = w.p13;
  a.p2 = w.p2;
  a.s13 = w.s13;
  a.s2 = w.s2;
  a.c13 = p.pad13 ? base + p.c13 : w.c13;
  a.c2 = p.pad2 ? base + p.c2 : w.c2;
  a.h = reinterpret_cast<uint16_t*>(base + p.h);
  a.he = base + p.he;
  a.ldhe = (int)((inter + 31) / 32);
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
  const auto grid = [&](int64_t runs) { return (unsigned)((p.max_bands + 7) / 8 * 8 * kBandTiles * runs); };
  for (int64_t t = 0; t < tokens; t += p.tokens) {
    const int64_t here = tokens - t < p.tokens ? tokens - t : p.tokens;
    a.x_bytes = (uint32_t)(here * hidden * 2);
    if ((st = half_rows(x + t * ldx, ldx, here, hidden, reinterpret_cast<uint16_t*>(base + p.x),
                        reinterpret_cast<float*>(base + p.xs), s)))
      return st;
    list.weights = weights + t * top_k;
    if ((st = launch_moe_sort(ids + t * top_k, here * top_k, experts, order, place, offsets, base + p.sort, list, s)))
      return st;
    moe_up_tile_kernel<<<grid((inter + Tiles::BN / 2 - 1) / (Tiles::BN / 2)), Tiles::THREADS, 0, s>>>(a);
    if ((st = launch_status("moe_up_tile_kernel"))) return st;
    one_exponent_kernel<<<(unsigned)(here * top_k), 256, 0, s>>>(a.h, a.he, a.ldhe, (int)(inter / 8), offsets + experts,
                                                                list.row_weight);
    if ((st = launch_status("one_exponent_kernel"))) return st;
    moe_down_tile_kernel<<<grid((hidden + Tiles::BN - 1) / Tiles::BN), Tiles::THREADS, 0, s>>>(a);
    if ((st = launch_status("moe_down_tile_kernel"))) return st;
    if ((st = launch_moe_combine_half(a.ys, a.ye, place, here, top_k, hidden, y + t * ldy, ldy, s))) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
