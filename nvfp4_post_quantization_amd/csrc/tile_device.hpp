// Tiles of tokens x output rows on the matrix cores, fed through LDS: what the
// kernels that multiply packed 4-bit weights by many tokens share (gfx950).
// matmul_tile.hip says how a tile works and what it reaches.
#pragma once
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

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
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));                     // the places are worked out here, not kept in registers
  const int l32 = lane & 31, sub = 4 * (lane >> 5);
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

template <bool F16>
__device__ __forceinline__ f32x16 mfma32_16(uint4 a, uint4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// 16-bit activations x NVFP4 weights: WM x WN waves of 32 TM tokens x 32 TN
// outputs, stages of 64 channels; NL waves that only load, AHEAD stages ahead.
template <int TM, int TN, int WM, int WN, int NL, int AHEAD>
struct NvTile {
  static constexpr int NW = WM * WN, LW = NL ? NL : NW, BM = 32 * TM * WM, BN = 32 * TN * WN, NBUF = AHEAD + 1;
  static constexpr int XB = BM * 128, WB = BN * 32, STAGE = XB + WB;
  using Scales = ScaleStages<0, BN, LW, AHEAD, true>;
  static constexpr int XL = BM / 8 / LW, WL = BN / 32 / LW, LOADS = XL + WL + Scales::STAGE_LOADS;
  static constexpr int LDS = NBUF * STAGE + Scales::BYTES, THREADS = 64 * (NW + NL);
  static_assert(BM % (8 * LW) == 0 && BN % (32 * LW) == 0 && LW % 2 == 0, "tile split");
};

// Which of the waves that load this one is (0 for one that only multiplies: it works
// out places of rows too, though it loads none).
template <int NW, int NL>
__device__ __forceinline__ int loader_of() {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return NL ? max(wave - NW, 0) : wave;
}

// One tile's stages s_begin .. s_end - 1.
//   bx, bw         buffers of the activations and the packed weights,
//   x_at(row), w_at(row)   the bytes in them at which the tile's rows begin (rows
//                  past the tile's last: any row, their results are not stored),
//   scales         the weights' (made with where they go in lds: NBUF * STAGE)
//   lds            NvTile::LDS bytes
//   finish(acc, wm, wn, wave, multiplies)  called by all waves once the stages are
//                  done with; acc[n][m], of those that multiply, is what store_tiles
//                  takes
// Lane half h of an instruction takes channels 32 h + 8 j .. + 7 of the stage
// at step j, so that a lane's weights of a stage are one 16-byte piece.
template <bool F16, int TM, int TN, int WM, int WN, int NL, int AHEAD, typename Scales, typename XAt, typename WAt,
          typename Finish>
__device__ __forceinline__ void nv_tile(i32x4 bx, i32x4 bw, int k, int s_begin, int s_end, XAt x_at, WAt w_at,
                                        const Scales& scales, uint8_t* lds, Finish finish) {
  using T = NvTile<TM, TN, WM, WN, NL, AHEAD>;
  constexpr int NW = T::NW, LW = T::LW, NBUF = T::NBUF, XB = T::XB, STAGE = T::STAGE, XL = T::XL, WL = T::WL;
  constexpr int LOADS = T::LOADS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool loads = NL == 0 || wave >= NW, multiplies = wave < NW;
  const int loader = loader_of<NW, NL>();
  const uint32_t lds_base = lds_address(lds);
  uint32_t xo[XL], wo[WL];
  const int xpiece = (lane & 7) ^ swizzle128(loader * 8 + (lane >> 3));    // loader + i LW has loader's parity
  const int wpiece = (lane & 1) ^ swizzle32(lane >> 1);
#pragma unroll
  for (int i = 0; i < XL; ++i)
    xo[i] = x_at((loader + i * LW) * 8 + (lane >> 3)) + xpiece * 16;
#pragma unroll
  for (int i = 0; i < WL; ++i)
    wo[i] = w_at((loader + i * LW) * 32 + (lane >> 1)) + wpiece * 16;

  const uint32_t lds_wave = lds_base + loader * 1024;
  auto load_stage = [&](int s, int buf, auto whole) {
    const uint32_t dst = lds_wave + buf * STAGE;
    const bool xcut = !whole && s * 64 + xpiece * 8 >= k, wcut = !whole && s * 64 + wpiece * 32 >= k;
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
    run_stages<AHEAD>(s_begin, s_end, k >> 6, next_stage);
  } else {
    read_w(s_begin, 0);
    read_x(0, 0, 0);
    run_stages<AHEAD>(s_begin, s_end, k >> 6, [&](int s, auto way) {
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
  finish(acc, wm, wn, wave, multiplies);
}

}  // namespace nvfp4
