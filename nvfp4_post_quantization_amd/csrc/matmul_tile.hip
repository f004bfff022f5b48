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
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

// A raw buffer resource: loads past `bytes` return zero.
__device__ __forceinline__ i32x4 make_buffer(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return i32x4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)bytes, 0x00020000};
}

// 16 (4) bytes a lane from the buffer to LDS at dst + AT + 16 (4) lane; dst is
// uniform over the wave.  In assembly because the compiler, which cannot tell
// the stages apart, waits for every load in flight before the next read of
// LDS; these write no register, and the kernels wait for them by count.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// (m0 is the compiler's to set anew before each of its own uses, of which these
// kernels have none; it only warns that it is named.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int AT>
__device__ __forceinline__ void load_lds16(i32x4 b, uint32_t dst, uint32_t offset, int base) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"(dst), "v"(offset), "s"(b), "s"(base), "n"(AT) : "memory", "m0", "scc");
}
template <int AT>
__device__ __forceinline__ void load_lds4(i32x4 b, uint32_t dst, uint32_t offset, int base) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               ::"s"(dst), "v"(offset), "s"(b), "s"(base), "n"(AT) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
// f(0), f(1) .. f(N - 1), each with a constant
template <int N, typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
template <int N, typename F>
__device__ __forceinline__ void each(F f) { each_of<N>(f, std::make_integer_sequence<int, N>{}); }

template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// Waves meet, and the compiler moves no read of LDS across (the builtin alone
// would let it).  Reads in flight stay so: what they read is overwritten after
// the next meeting at the earliest.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Piece swizzles of LDS rows of 64, 128 and 32 bytes: piece p of a row lies at
// place p ^ swizzle.  A 16-byte read of a wave is served in four groups of 16
// lanes (0-3, 12-15, 20-27; 4-11, 16-19, 28-31; the same + 32) over 64 banks;
// with these, the lanes of a group that read one piece of their 16 rows touch
// every bank once (no conflict counted for operands; the plain row-order ones cost 4
// cycles in 12).
__device__ __forceinline__ int swizzle64(int row) { return (row >> 2) & 3; }
__device__ __forceinline__ int swizzle128(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swizzle32(int row) { return (row >> 3) & 1; }

struct TileArgs {
  const uint8_t* x;           // packed MXFP4 rows, or 16-bit rows
  const uint8_t* w;           // packed rows
  const uint8_t* xs;          // rows of scales (MXFP4), lds bytes each, a multiple of 4
  const uint8_t* ws;
  const float* s0;            // tensor scales, or NULL
  const float* s1;
  uint16_t* y;
  float* partial;             // [splits][tokens][ldp] when splits > 1
  int64_t ldx, ldw, ldy;      // bytes, bytes, elements
  int64_t ldp;
  int tokens, out, k, lds;
  int tiles_m, tiles_n, splits, steps;
};

// Which tile a workgroup takes.  Consecutive workgroups go to the 8 XCDs in
// turn; each XCD gets a contiguous run of tiles, walked in columns of up to 8
// token tiles, so that what its CUs read at one time shares its L2.
struct TilePos { int m, n, split; };
__device__ __forceinline__ TilePos tile_of(const TileArgs& a) {
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int id = blockIdx.x, xcd = id & 7, i = id >> 3;
  const int q = total >> 3, r = total & 7;
  int t = xcd * q + min(xcd, r) + i;
  const int per = a.tiles_m * a.tiles_n;
  TilePos p;
  p.split = t / per;
  t -= p.split * per;
  const int band = t / (8 * a.tiles_n);
  const int rows = min(8, a.tiles_m - band * 8);
  t -= band * 8 * a.tiles_n;
  p.n = t / rows;
  p.m = band * 8 + t % rows;
  return p;
}

// Results of a wave: tile (n, m) covers outputs o0 + 32 n + .., tokens
// t0 + 32 m + (lane & 31).  Register 4 g + e of a lane is output
// 8 g + 4 (lane >> 5) + e of the tile.  Where rows of y are 16-byte aligned
// the bf16 results go through `lds` (32 rows of the wave at a time, nobody
// else's), so that a store instruction writes whole runs of 64 TN bytes.
template <int TN, int TM>
__device__ __forceinline__ void store_tiles(const TileArgs& a, const f32x16 (&acc)[TN][TM], int o0, int t0, int split,
                                            uint8_t* lds) {
  constexpr int PITCH = 64 * TN + 16, LANES = 4 * TN, ROWS = 64 / LANES;       // lanes per row, rows per store
  const int lane = threadIdx.x & 63, l32 = lane & 31, sub = 4 * (lane >> 5);
  if (a.splits > 1) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int t = t0 + 32 * m + l32;
      if (t >= a.tokens) continue;
      float* dst = a.partial + ((int64_t)split * a.tokens + t) * a.ldp;
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int o = o0 + 32 * n + 8 * g + sub;
          if (o < a.out)
            *reinterpret_cast<f32x4*>(dst + o) = f32x4{acc[n][m][4 * g], acc[n][m][4 * g + 1], acc[n][m][4 * g + 2],
                                                       acc[n][m][4 * g + 3]};
        }
    }
    return;
  }
  float s0 = 1.0f, s1 = 1.0f;
  if (a.s0) s0 = *a.s0;
  if (a.s1) s1 = *a.s1;
  auto quad = [&](int n, int m, int g) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_bf16(acc[n][m][4 * g + e] * s0 * s1);
    return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
  };
  if ((a.ldy & 7) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0) {
    const int piece = lane % LANES, row0 = lane / LANES, o = o0 + piece * 8;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<uint2*>(lds + l32 * PITCH + 64 * n + 16 * g + 2 * sub) = quad(n, m, g);
#pragma unroll
      for (int r = 0; r < 32; r += ROWS) {
        const uint4 v = *reinterpret_cast<const uint4*>(lds + (r + row0) * PITCH + piece * 16);
        const int t = t0 + 32 * m + r + row0;
        if (t >= a.tokens) continue;
        uint16_t* dst = a.y + (int64_t)t * a.ldy + o;
        if (o <= a.out - 8) {                        // (o + 8 may be 2^31)
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (o + e < a.out) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
    return;
  }
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int t = t0 + 32 * m + l32;
    if (t >= a.tokens) continue;
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int o = o0 + 32 * n + 8 * g + sub;
        const uint2 v = quad(n, m, g);
        uint16_t* dst = a.y + (int64_t)t * a.ldy + o;
        if (o < a.out) dst[0] = (uint16_t)v.x;
        if (o + 1 < a.out) dst[1] = (uint16_t)(v.x >> 16);
        if (o + 2 < a.out) dst[2] = (uint16_t)v.y;
        if (o + 3 < a.out) dst[3] = (uint16_t)(v.y >> 16);
      }
  }
}

__device__ __forceinline__ f32x16 mfma32_mx(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x16 c, int sel) {
  const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  if (sel == 0) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, 0, (int)sa, 0, (int)sb);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, 2, (int)sa, 2, (int)sb);
}

// The scales of groups of four stages in LDS: RX rows of x (none for 16-bit x)
// and RW of w, 16 bytes each (stages are counted from the first).
//   QUARTERS  stage s brings quarter (s + 3) % 4 of group (s + 3) / 4, 16 rows
//             an instruction and 4 bytes a lane
//   else      stage 4 g + 3 brings group g + 1, 64 rows an instruction
// Either way a group is there with its first stage, and the one that it
// replaces has been read: stages are AHEAD steps ahead, so two groups are kept
// for three steps and four for up to eight.  16-bit x, 8192x4096x12288: 675 us
// with quarters, 706 without; MXFP4, which has scales of x too, 8192x12288x4096:
// 252 and 247 us (without quarters the words of 32 rows lie in 16 of the 64 banks:
// 36 of 99 LDS cycles of a wave and stage of the large tile are their conflicts).
template <int RX, int RW, int NW, int AHEAD, bool QUARTERS>
struct ScaleStages {
  static constexpr int CHUNKS = (RX + RW) / 64, LOADS = (CHUNKS + NW - 1) / NW, GROUP = (RX + RW) * 16;
  static constexpr int GROUPS = AHEAD <= 3 ? 2 : 4, BYTES = GROUPS * GROUP;
  static_assert(AHEAD <= (QUARTERS ? 2 : 3) || (GROUPS == 4 && AHEAD <= 8), "groups kept");
  static constexpr int STAGE_LOADS = QUARTERS ? LOADS : 0;       // of a wave, with every stage
  static_assert(RX % 64 == 0 && RW % 64 == 0, "whole chunks of rows");
  i32x4 b[LOADS];
  uint32_t dst[LOADS];        // where the wave's chunks go
  uint32_t at[LOADS];         // where the lane reads,
  int odd;                    // and how far from there in odd quarters
  int end[LOADS];             // the buffers' sizes
  int stride, first;          // bytes of a row; the first stage

  // Rows past the last one read as zero: their results are not stored.
  __device__ __forceinline__ ScaleStages(const TileArgs& a, uint32_t lds, int t0, int rows_x, int o0, int rows_w, int s,
                                         int loader)
      : stride(a.lds), first(s) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int c = (loader + i * NW) % CHUNKS;                  // more waves than chunks: the same ones again
      const bool x = c < RX / 64;
      const uint8_t* rows = x ? a.xs + (int64_t)t0 * stride : a.ws + (int64_t)o0 * stride;
      end[i] = (x ? rows_x : rows_w) * stride;
      b[i] = make_buffer(rows, (uint32_t)end[i]);
      dst[i] = lds + c * 1024;
      at[i] = (uint32_t)(c * 64 - (x ? 0 : RX) + (QUARTERS ? lane >> 2 : lane)) * stride + (QUARTERS ? (lane & 3) * 4 : 0);
    }
    odd = lane & 1 ? -4 : 4;
  }
  // (words past a row's end: read, not used; a scalar offset is held to the
  // buffer's size, which keeps the bounds check right)
  __device__ __forceinline__ void load_quarter(int g, int q) const {
    const int base = (first + 4 * g) * 4 + q * 16 * stride;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_lds4<0>(b[i], dst[i] + (g & (GROUPS - 1)) * GROUP + q * 256, at[i] + (q & 1 ? odd : 0), min(base, end[i]));
  }
  __device__ __forceinline__ void load_group(int g) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_lds16<0>(b[i], dst[i] + (g & (GROUPS - 1)) * GROUP, at[i], min((first + 4 * g) * 4, end[i]));
  }
  // before the first stage
  __device__ __forceinline__ void load_first() const {
    if constexpr (QUARTERS) {
#pragma unroll
      for (int q = 0; q < 3; ++q) load_quarter(0, q);
    } else {
      load_group(0);
    }
  }
  __device__ __forceinline__ void load_with(int s) const {
    const int n = s - first;
    if constexpr (QUARTERS) load_quarter((n + 3) >> 2, (n + 3) & 3);
    else if ((n & 3) == 3) load_group((n >> 2) + 1);
  }
  // where the words of stage s are, for the lane's row among 32 (odd quarters
  // swap neighbouring words, so that 32 rows' words lie in as many banks)
  __device__ __forceinline__ int place(int s, int l32) const {
    const int n = s - first;
    return (n >> 2 & (GROUPS - 1)) * GROUP + l32 * 16 + (((n & 3) ^ (QUARTERS ? l32 >> 4 : 0)) << 2);
  }
};

// Stages begin .. end - 1, whole the first that may end before its last channel;
// step(s, way) works on one.
enum Way {
  kWhole,                     // stage s + AHEAD, a whole one, is loaded meanwhile
  kCut,                       // it may not be whole
  kDrain,                     // everything that is needed is on its way
  kLast
};
template <int AHEAD, typename Step>
__device__ __forceinline__ void run_stages(int begin, int end, int whole, Step step) {
  int s = begin;
  const int stop = min(end, whole) - AHEAD;
  for (; s < stop; ++s) step(s, std::integral_constant<Way, kWhole>{});
  if (s + AHEAD < end) step(s++, std::integral_constant<Way, kCut>{});
  for (; s + 1 < end; ++s) step(s, std::integral_constant<Way, kDrain>{});
  step(s, std::integral_constant<Way, kLast>{});
}

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

template <bool F16>
__device__ __forceinline__ f32x16 mfma32_16(uint4 a, uint4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// 16-bit activations x NVFP4 weights: WM x WN waves of 32 TM tokens x 32 TN
// outputs, stages of 64 channels.
// Lane half h of an instruction takes channels 32 h + 8 j .. + 7 of the stage
// at step j, so that a lane's weights of a stage are one 16-byte piece.
template <bool F16, int TM, int TN, int WM, int WN, int NL, int AHEAD>
__global__ __launch_bounds__(64 * (WM * WN + NL), NL && AHEAD == 2 ? 4 : 2) void nv_tile_kernel(TileArgs a) {
  constexpr int NW = WM * WN, LW = NL ? NL : NW, BM = 32 * TM * WM, BN = 32 * TN * WN, NBUF = AHEAD + 1;
  constexpr int XB = BM * 128, WB = BN * 32, STAGE = XB + WB;
  using Scales = ScaleStages<0, BN, LW, AHEAD, true>;
  constexpr int XL = BM / 8 / LW, WL = BN / 32 / LW, LOADS = XL + WL + Scales::STAGE_LOADS;
  static_assert(BM % (8 * LW) == 0 && BN % (32 * LW) == 0 && LW % 2 == 0, "tile split");
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
  // the last row ends with its k channels, not with its stride
  const auto bx = make_buffer(a.x + (int64_t)t0 * a.ldx, (uint32_t)((int64_t)(rows_x - 1) * a.ldx + (int64_t)a.k * 2));
  const auto bw = make_buffer(a.w + (int64_t)o0 * a.ldw, (uint32_t)((int64_t)rows_w * a.ldw));
  const Scales scales(a, lds_base + NBUF * STAGE, 0, 0, o0, rows_w, s_begin, loader);
  uint32_t xo[XL], wo[WL];
  const int xpiece = (lane & 7) ^ swizzle128(loader * 8 + (lane >> 3));    // loader + i LW has loader's parity
  const int wpiece = (lane & 1) ^ swizzle32(lane >> 1);
#pragma unroll
  for (int i = 0; i < XL; ++i)
    xo[i] = (uint32_t)(min((loader + i * LW) * 8 + (lane >> 3), rows_x - 1) * a.ldx + xpiece * 16);
#pragma unroll
  for (int i = 0; i < WL; ++i)
    wo[i] = (uint32_t)(min((loader + i * LW) * 32 + (lane >> 1), rows_w - 1) * a.ldw + wpiece * 16);

  const uint32_t lds_wave = lds_base + loader * 1024;
  auto load_stage = [&](int s, int buf, auto whole) {
    const uint32_t dst = lds_wave + buf * STAGE;
    const bool xcut = !whole && s * 64 + xpiece * 8 >= a.k, wcut = !whole && s * 64 + wpiece * 32 >= a.k;
    each<XL>([&](auto i) { load_lds16<i * LW * 1024>(bx, dst, xcut ? kBeyond : xo[i], s * 128); });
    each<WL>([&](auto i) { load_lds16<XB + i * LW * 1024>(bw, dst, wcut ? kBeyond : wo[i], s * 32); });
    scales.load_with(s);
  };

  const int wm = wave % WM, wn = wave / WM, half = lane >> 5, l32 = lane & 31;
  const int xrow = (wm * TM * 32 + l32) * 128;
  const int wf = XB + (wn * TN * 32 + l32) * 32 + ((half ^ swizzle32(l32)) << 4);
  const int wsf = NBUF * STAGE + wn * TN * 512;
  uint4 xr[2][TM], wr[TN];
  uint32_t wsr[TN];
  auto read_x = [&](int set, int j, int buf) {
    const uint8_t* b = lds + buf * STAGE + xrow + (((4 * half + j) ^ swizzle128(l32)) << 4);
#pragma unroll
    for (int i = 0; i < TM; ++i) xr[set][i] = *reinterpret_cast<const uint4*>(b + i * 4096);
  };
  uint4 wr_next[TN];
  uint32_t wsr_next[TN];
  auto read_w = [&](int s, int buf) {
    const uint8_t* b = lds + buf * STAGE;
    const uint8_t* c = lds + wsf + scales.place(s, l32);
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      wr_next[i] = *reinterpret_cast<const uint4*>(b + wf + i * 1024);
      wsr_next[i] = *reinterpret_cast<const uint32_t*>(c + i * 512);
    }
  };
  auto expand = [&](int n, int j) {
    const uint32_t q = j == 0 ? wr[n].x : j == 1 ? wr[n].y : j == 2 ? wr[n].z : wr[n].w;
    const float s = j < 2 ? e4m3_f32<0>(wsr[n]) : e4m3_f32<1>(wsr[n]);
    return F16 ? fp4x8_f16(q, splat_f16(s)) : fp4x8_bf16(q, s);
  };

  f32x16 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] = 0.0f;

  if (loads) {
    scales.load_first();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (s_begin + i < s_end) load_stage(s_begin + i, i, std::false_type{});
    if (s_begin + AHEAD <= s_end) wait_loads<(AHEAD - 1) * LOADS>();
    else wait_loads<0>();
  }
  stage_barrier();
  int buf = 0, free = AHEAD;                                      // stage s, and where stage s + AHEAD goes
  // on to stage s + 1, in one of the ways below
  auto next_stage = [&](int s, auto way) {
    if constexpr (way == kLast) return;
    if (loads) wait_loads<way == kDrain ? 0 : (AHEAD - 2) * LOADS>();
    stage_barrier();
    if constexpr (way == kWhole || way == kCut)
      if (loads) load_stage(s + AHEAD, free, std::bool_constant<way == kWhole>{});
    free = buf;
    buf = buf == AHEAD ? 0 : buf + 1;
  };
  if (NL && loads) {
    run_stages<AHEAD>(s_begin, s_end, a.k >> 6, next_stage);
  } else {
    read_w(s_begin, 0);
    read_x(0, 0, 0);
    run_stages<AHEAD>(s_begin, s_end, a.k >> 6, [&](int s, auto way) {
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        wr[n] = wr_next[n];
        wsr[n] = wsr_next[n] >> (16 * half);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < 3) {
          read_x((j + 1) & 1, j + 1, buf);
        } else {
          next_stage(s, way);
          if constexpr (way != kLast) {
            read_w(s + 1, buf);
            read_x(0, 0, buf);
          }
        }
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          const uint4 w = expand(n, j);
#pragma unroll
          for (int m = 0; m < TM; ++m) acc[n][m] = mfma32_16<F16>(w, xr[j & 1][m], acc[n][m]);
        }
      }
    });
  }
  __syncthreads();                                                // the stages are done with
  static_assert(NW * 32 * (64 * TN + 16) <= sizeof(lds), "store staging");
  if (!multiplies) return;
  store_tiles<TN, TM>(a, acc, o0 + wn * TN * 32, t0 + wm * TM * 32, pos.split, lds + wave * 32 * (64 * TN + 16));
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

template <bool F16, int TM, int TN, int WM, int WN, int NL, int AHEAD>
int run_nv(const TileArgs& a, hipStream_t s) {
  nv_tile_kernel<F16, TM, TN, WM, WN, NL, AHEAD><<<tile_grid(a), 64 * (WM * WN + NL), 0, s>>>(a);
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
                   int64_t ldy, void* workspace, hipStream_t s) {
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
  if (f16) {
    if (p.rows == 256) return run_nv<true, 4, 2, 2, 4, 0, 2>(a, s);
    return alone ? run_nv<true, 2, 2, 2, 2, 4, 6>(a, s) : run_nv<true, 2, 2, 2, 2, 4, 2>(a, s);
  }
  if (p.rows == 256) return run_nv<false, 4, 2, 2, 4, 0, 2>(a, s);
  return alone ? run_nv<false, 4, 1, 1, 4, 4, 6>(a, s) : run_nv<false, 4, 1, 1, 4, 4, 2>(a, s);
}

}  // namespace nvfp4
