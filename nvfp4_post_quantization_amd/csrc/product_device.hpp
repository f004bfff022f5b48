// Device code shared by the kernels that multiply packed 4-bit matrices
// (gfx950): exact expansion of E2M1 nibbles to matrix-core operands, and the
// accumulate of a few output rows against a few tokens.
//
// Three products, all y[t][o] = sum_k x[t][k] w[o][k] with w in 4 bits:
//   kW4A16  x bf16,  w NVFP4.  e2m1 * e4m3 has at most 2 + 4 significant bits
//           and lies in [2^-10, 2688], so it is exact in bf16.
//   kW4A4   both NVFP4.  e2m1 * e4m3 is exact in fp16 as well, and fp16 is
//           cheaper to make: one convert and one packed multiply per pair.
//   kMX     both MXFP4: the scaled FP4 matrix instruction takes the packed
//           nibbles and E8M0 bytes as they are.
// The tensor scales (scale_2) stay out of the sum and multiply the fp32
// result, so an operand is never rounded and the products are exact; what
// rounds is the fp32 accumulation and the final conversion.
#pragma once
#include "nvfp4_device.hpp"

namespace nvfp4 {

enum ProductKind { kW4A16 = 0, kW4A4 = 1, kMX = 2 };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __fp16 fp16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// E4M3FN byte SEL of a word as fp32 (exact; NaN for 0x7F).
template <int SEL>
__device__ __forceinline__ float e4m3_f32(uint32_t w) { return __builtin_amdgcn_cvt_f32_fp8((int)w, SEL); }

// Two exact products e2m1 * s as packed bf16: the fp32 products have at most
// 6 significant bits, so their upper halves are the bf16 values.
template <int SEL>
__device__ __forceinline__ uint32_t fp4x2_bf16(uint32_t w, float s) {
  float a, b;
  fp4x2_to_f32<SEL>(w, a, b);
  return __builtin_amdgcn_perm(__float_as_uint(b * s), __float_as_uint(a * s), 0x07060302u);
}
__device__ __forceinline__ uint4 fp4x8_bf16(uint32_t w, float s) {
  return make_uint4(fp4x2_bf16<0>(w, s), fp4x2_bf16<1>(w, s), fp4x2_bf16<2>(w, s), fp4x2_bf16<3>(w, s));
}

// The same in fp16 (exact: 6 significant bits in [2^-10, 2688]).
template <int SEL>
__device__ __forceinline__ uint32_t fp4x2_f16(uint32_t w, f16x2 s) {
  const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL));
  return __builtin_bit_cast(uint32_t, (f16x2)(v * s));
}
__device__ __forceinline__ uint4 fp4x8_f16(uint32_t w, f16x2 s) {
  return make_uint4(fp4x2_f16<0>(w, s), fp4x2_f16<1>(w, s), fp4x2_f16<2>(w, s), fp4x2_f16<3>(w, s));
}
__device__ __forceinline__ f16x2 splat_f16(float s) { return f16x2{(_Float16)s, (_Float16)s}; }

__device__ __forceinline__ f32x4 mfma_bf16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ f32x4 mfma_f16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_mx(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x4 c) {
  const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Two fp32 to bf16, nearest even.
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ---- a few tokens against many rows -----------------------------------------
//
// A unit is 128 channels, a quad four units.  Lane l of a wave works on row
// (token) l % 16 of a tile and, as group g = l / 16, on chunk g of 32
// consecutive channels of a unit.  A matrix instruction sums over the groups,
// so the order of channels within a unit does not matter as long as both
// operands share it, and a lane's weights of a unit are one 16-byte load.
//
// Loads return in order: a wait for one is a wait for all before it.  So the
// tokens stay in registers (QW quads of them a wave) while the rows go by, and
// the loop loads nothing but weights: 8 units of them are always on their way,
// each loaded again as soon as it has been used.

constexpr int kStreamWaves = 8;
constexpr uint32_t kBeyond = 0x80000000u;           // past any buffer (they are below 2^31 bytes): reads as zero

// Eight waves meet; what they wrote to LDS is seen.  Loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A load that is known to be from global memory, also where the compiler has
// lost sight of it (a flat load would be waited for together with LDS).
__device__ __forceinline__ uint4 global_load16(const uint8_t* p) {
  typedef const __attribute__((address_space(1))) ntu32x4* ptr;
  return __builtin_bit_cast(uint4, *(ptr)(uintptr_t)p);
}

// Exchanges between the groups.  swap32: the upper half of a with the lower
// half of b; swap16: groups 1 and 3 of a with groups 0 and 2 of b.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r.x;
  b = r.y;
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r.x;
  b = r.y;
}
// v[j] of group g becomes v[g] of group j.
__device__ __forceinline__ void transpose_groups(uint32_t& v0, uint32_t& v1, uint32_t& v2, uint32_t& v3) {
  swap32(v0, v2);
  swap32(v1, v3);
  swap16(v0, v1);
  swap16(v2, v3);
}

// Rows of a packed matrix: buffers that start at the first of them (loads past
// the end read as zero).
struct PackedRows {
  const uint8_t* w;
  const uint8_t* s;
  uint32_t w_bytes, s_bytes;
};

// The same in scalar registers: a buffer that the compiler does not know to be
// the same for all lanes is loaded from lane by lane.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ PackedRows uniform(const PackedRows& r) {
  return PackedRows{uniform(r.w), uniform(r.s), (uint32_t)__builtin_amdgcn_readfirstlane(r.w_bytes),
                    (uint32_t)__builtin_amdgcn_readfirstlane(r.s_bytes)};
}

// One quad of a lane's packed row.  The block scales of a quad are 32 bytes of
// the row (MXFP4: 16); group g loads those of unit g and the groups exchange
// them afterwards, which asks memory for a quarter of the pieces that every
// lane loading its own scales unit by unit would.
template <int KIND>
struct Quad {
  uint4 w[4];
  u32x2 s;

  // row_w, row_s: byte offsets of the lane's row; q: the quad
  // (the whole offset is in the lane's part, which is what the bounds check
  // looks at)
  __device__ __forceinline__ void load_weights(int u, const PackedRows& t, uint32_t row_w, int q, int g) {
    const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.w), 0, (int)t.w_bytes, 0x00020000);
    const uint32_t at = row_w + q * 256 + g * 16 + u * 64;
    w[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0));
  }
  // Past channel k the weights are the next row's; their scales are zero here
  // (as a power of two: 2^-127), and so is the other operand.
  __device__ __forceinline__ void load_scales(const PackedRows& t, uint32_t row_s, int q, int g, int k) {
    const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.s), 0, (int)t.s_bytes, 0x00020000);
    constexpr int N = KIND == kMX ? 4 : 8;           // bytes of a unit
    const uint32_t at = row_s + q * (4 * N) + g * N;
    if ((q + 1) * 512 <= k) {
      if constexpr (KIND == kMX) s.x = __builtin_amdgcn_raw_buffer_load_b32(b, (int)at, 0, 0);
      else s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, (int)at, 0, 0));
    } else {                                         // byte by byte: the words may reach past the buffer
      uint32_t v[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool in = q * 512 + g * 128 + i * (128 / N) < k;
        v[i >> 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(b, (int)(in ? at + i : kBeyond), 0, 0) << (8 * (i & 3));
      }
      s.x = v[0];
      s.y = v[1];
    }
  }

  // This lane's scales of the four units.  NVFP4: x = units 0 (low half) and
  // 2, y = units 1 and 3, two codes each; MXFP4: x = a byte per unit.
  __device__ __forceinline__ u32x2 scales(int g) const {
    u32x2 r;
    if constexpr (KIND == kMX) {
      uint32_t a = s.x, b = s.x;
      swap32(a, b);                                  // units g % 2 and g % 2 + 2
      uint32_t c = __builtin_amdgcn_perm(b, a, g < 2 ? 0x05040100u : 0x07060302u), d = c;
      swap16(c, d);                                  // units 0 and 2, units 1 and 3
      r.x = __builtin_amdgcn_perm(d, c, (g & 1) ? 0x07030501u : 0x06020400u);
      r.y = 0;
    } else {
      uint32_t a = s.x, b = s.y;
      swap32(a, b);                                  // groups 2 (g / 2), 2 (g / 2) + 1 of units g % 2 and g % 2 + 2
      uint32_t e = __builtin_amdgcn_perm(b, a, 0x05040100u), f = __builtin_amdgcn_perm(b, a, 0x07060302u);
      swap16(e, f);
      r.x = e;
      r.y = f;
    }
    return r;
  }
  // the two NVFP4 codes of unit u, as fp32
  static __device__ __forceinline__ void codes(u32x2 s, int u, float& a, float& b) {
    const uint32_t v = u & 1 ? s.y : s.x;
    if (u < 2) {
      a = e4m3_f32<0>(v);
      b = e4m3_f32<1>(v);
    } else {
      a = e4m3_f32<2>(v);
      b = e4m3_f32<3>(v);
    }
  }
};

// What tokens read past channel k.
static __device__ const uint4 kZeroPiece[1] = {};

// Where 16 tokens are: the lane's row of bf16 values, or its offsets in the
// rows of a packed matrix.
struct TokenRows {
  const uint8_t* x;
  PackedRows packed;
  uint32_t row_w, row_s;
};

// A quad of 16 tokens in registers: 16-bit values, expanded where they were
// packed; channels past k are zero.
template <int KIND>
struct TokenQuad {
  uint4 x[4][4];                                     // [unit][8 channels]

  __device__ __forceinline__ void load(const TokenRows& t, int q, int g, int k) {
    if constexpr (KIND == kW4A16) {
      // four lanes of a token read 64 neighbouring bytes; the groups then
      // exchange pieces, so that each holds 32 consecutive channels of a unit
      const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroPiece);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = q * 512 + u * 128 + j * 32 + g * 8;
          x[u][j] = global_load16(c < k ? t.x + (int64_t)c * 2 : zero);
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        transpose_groups(x[u][0].x, x[u][1].x, x[u][2].x, x[u][3].x);
        transpose_groups(x[u][0].y, x[u][1].y, x[u][2].y, x[u][3].y);
        transpose_groups(x[u][0].z, x[u][1].z, x[u][2].z, x[u][3].z);
        transpose_groups(x[u][0].w, x[u][1].w, x[u][2].w, x[u][3].w);
      }
    } else {
      Quad<KIND> p;
#pragma unroll
      for (int u = 0; u < 4; ++u) p.load_weights(u, t.packed, t.row_w, q, g);
      p.load_scales(t.packed, t.row_s, q, g, k);
      const u32x2 s = p.scales(g);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float a, b;
        Quad<KIND>::codes(s, u, a, b);
        x[u][0] = fp4x8_f16(p.w[u].x, splat_f16(a));
        x[u][1] = fp4x8_f16(p.w[u].y, splat_f16(a));
        x[u][2] = fp4x8_f16(p.w[u].z, splat_f16(b));
        x[u][3] = fp4x8_f16(p.w[u].w, splat_f16(b));
      }
    }
  }
};

template <>
struct TokenQuad<kMX> {
  uint4 x[4];
  uint32_t s;                                        // a byte per unit

  __device__ __forceinline__ void load(const TokenRows& t, int q, int g, int k) {
    Quad<kMX> p;
#pragma unroll
    for (int u = 0; u < 4; ++u) p.load_weights(u, t.packed, t.row_w, q, g);
    p.load_scales(t.packed, t.row_s, q, g, k);
    s = p.scales(g).x;
    const int left = k - q * 512 - g * 32;
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = left > u * 128 ? p.w[u] : make_uint4(0, 0, 0, 0);
  }
};

template <int U>
__device__ __forceinline__ f32x4 mfma_mx_unit(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x4 c) {
  const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, U, (int)sa, U, (int)sb);
}

// acc[n] += unit u of 16 rows x 16 tokens each.  Even and odd pieces add up
// apart (acc[0], acc[1]), so that one product need not wait for the last.
template <int KIND, int NT>
__device__ __forceinline__ void multiply_unit(uint4 w, u32x2 ws, int u, const TokenQuad<KIND> (&x)[NT],
                                              f32x4 (&acc)[2][NT]) {
  if constexpr (KIND == kMX) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4& c = acc[u & 1][n];
      if (u == 0) c = mfma_mx_unit<0>(w, ws.x, x[n].x[u], x[n].s, c);
      else if (u == 1) c = mfma_mx_unit<1>(w, ws.x, x[n].x[u], x[n].s, c);
      else if (u == 2) c = mfma_mx_unit<2>(w, ws.x, x[n].x[u], x[n].s, c);
      else c = mfma_mx_unit<3>(w, ws.x, x[n].x[u], x[n].s, c);
    }
  } else {
    float s0, s1;
    Quad<KIND>::codes(ws, u, s0, s1);
    const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = j < 2 ? s0 : s1;
      const uint4 a = KIND == kW4A16 ? fp4x8_bf16(wv[j], s) : fp4x8_f16(wv[j], splat_f16(s));
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[j & 1][n] = KIND == kW4A16 ? mfma_bf16(a, x[n].x[u][j], acc[j & 1][n])
                                       : mfma_f16(a, x[n].x[u][j], acc[j & 1][n]);
    }
  }
}

// Row tiles begin .. end - 1 against 16 NT tokens, by a workgroup.  A step is RT
// row tiles; a pass, kStreamWaves * QW quads of the channels, QW a wave's; TB
// steps make a batch, whose partial tiles the waves write to `part`
// (kStreamWaves * TB * RT * NT * 64 of them).
//   rows_of(t)       the packed rows from tile t on (at least to the end of the
//                    step's tiles, as far as they exist)
//   row_w, row_s     byte offsets of the lane's row in a tile; tile_w, tile_s:
//                    from a tile to the next
//   done(t, n, l, sum)  called once for every lane l of tile t, token tile n, by
//                    some thread; sum(l) adds up the waves, in order
template <int KIND, int NT, int QW, int TB, typename RowsOf, typename Done>
__device__ __forceinline__ void stream_tiles(int begin, int end, int k, uint32_t row_w, uint32_t row_s, uint32_t tile_w,
                                             uint32_t tile_s, const TokenRows (&tokens)[NT], f32x4* part, RowsOf rows_of,
                                             Done done) {
  constexpr int RT = 2 / QW;
  static_assert(QW * RT == 2, "8 units in flight");
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quads = (k + 511) >> 9, passes = (quads + kStreamWaves * QW - 1) / (kStreamWaves * QW);
  auto quad_of = [&](int pass, int i) { return (pass * kStreamWaves + wave) * QW + i; };

  Quad<KIND> w[2];
  TokenQuad<KIND> x[QW][NT];
  // the step that is loaded: tile at_t of pass at_pass of the batch from
  // at_batch on
  int at_batch = begin, at_pass = 0, at_t = begin;
  PackedRows next = uniform(rows_of(begin));
  auto advance = [&]() {
    at_t += RT;
    if (at_t >= end || at_t >= at_batch + TB * RT) {
      if (++at_pass == passes) {
        at_pass = 0;
        at_batch += TB * RT;
      }
      at_t = at_batch;
    }
    next = rows_of(min(at_t, end - 1));
    if (at_t >= end) next.w_bytes = next.s_bytes = 0;
    next = uniform(next);
  };
  auto load_scales = [&](int i) {                    // i = r * QW + quad of the wave
    w[i].load_scales(next, row_s + (i / QW) * tile_s, quad_of(at_pass, i % QW), g, k);
  };
  auto load_weights = [&](int i, int u) {
    w[i].load_weights(u, next, row_w + (i / QW) * tile_w, quad_of(at_pass, i % QW), g);
  };
  auto load_tokens = [&](int pass) {
#pragma unroll
    for (int i = 0; i < QW; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) x[i][n].load(tokens[n], quad_of(pass, i), g, k);
    __builtin_amdgcn_s_waitcnt(0x0F70);              // vmcnt(0): the loop awaits nothing of the tokens
  };

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    load_scales(i);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_weights(i, u);
  }
  advance();
  if (passes == 1) load_tokens(0);
  for (int batch = begin; batch < end; batch += TB * RT) {
    f32x4 acc[TB][RT][NT];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[b][r][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int pass = 0; pass < passes; ++pass) {
      if (passes > 1) load_tokens(pass);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if (batch + b * RT >= end) break;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 sum[2][NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[0][n] = acc[b][r][n];
            sum[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
          for (int i = 0; i < QW; ++i) {
            const int at = r * QW + i;
            const u32x2 ws = w[at].scales(g);
            load_scales(at);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              multiply_unit<KIND, NT>(w[at].w[u], ws, u, x[i], sum);
              load_weights(at, u);
              __builtin_amdgcn_sched_barrier(0);     // the load goes out here, not where its value is near
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[b][r][n] = sum[0][n] + sum[1][n];
        }
        advance();
      }
    }
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) part[(((wave * TB + b) * RT + r) * NT + n) * 64 + lane] = acc[b][r][n];
    lds_barrier();
    const int count = min(TB * RT, end - batch);
    for (int q = threadIdx.x; q < count * NT * 64; q += 64 * kStreamWaves)
      done(batch + (q >> 6) / NT, (q >> 6) % NT, q & 63, [&](int l) {
        const f32x4* p = part + (q & ~63) + l;
        f32x4 v = *p;
#pragma unroll
        for (int z = 1; z < kStreamWaves; ++z) v += p[z * TB * RT * NT * 64];
        return v;
      });
    lds_barrier();                                   // before the next batch's partial tiles
  }
}

}  // namespace nvfp4
