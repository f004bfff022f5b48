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

// 32 packed nibbles (16 bytes) of chunk c of a row, whatever of them lies
// below k; rows are 16-byte aligned when k % 32 == 0 and 8-byte aligned else.
template <bool K32, bool TAIL>
__device__ __forceinline__ uint4 load_chunk(const uint8_t* row, int c, int k) {
  const uint8_t* p = row + (int64_t)c * 16;
  if constexpr (K32) {
    if (!TAIL || c * 32 < k) return *reinterpret_cast<const uint4*>(p);
    return make_uint4(0, 0, 0, 0);
  } else {
    uint2 a = make_uint2(0, 0), b = make_uint2(0, 0);
    if (!TAIL || c * 32 < k) a = *reinterpret_cast<const uint2*>(p);
    if (!TAIL || c * 32 + 16 < k) b = *reinterpret_cast<const uint2*>(p + 8);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
}

// The two E4M3 codes of chunk c (second in bits 8-15), 0 beyond k.
template <bool K32, bool TAIL>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* row, int c, int k) {
  const uint8_t* p = row + (int64_t)c * 2;
  if constexpr (K32) {
    if (!TAIL || c * 32 < k) return *reinterpret_cast<const uint16_t*>(p);
    return 0;
  } else {
    uint32_t v = 0;
    if (!TAIL || c * 32 < k) v = p[0];
    if (!TAIL || c * 32 + 16 < k) v |= (uint32_t)p[1] << 8;
    return v;
  }
}

// What a lane reads: the row pointers of its output rows (one per row tile)
// and of its tokens (one per token tile).  Lane l works on row / token l % 16
// of each tile.
template <int RT, int NT>
struct ProductRows {
  const uint8_t* wp[RT];      // packed weights of the row
  const uint8_t* wc[RT];      // its block scales
  const uint8_t* xp[NT];      // the token: bf16 values or packed nibbles
  const uint8_t* xc[NT];      // its block scales (kW4A4, kMX)
};

// One unit of 128 channels: lane group g = l / 16 holds chunk 4u + g of 32
// consecutive channels of its row and token.  A matrix instruction sums over
// the groups, so the order of channels within the unit does not matter as
// long as both operands share it.  SPLIT: x is a pair of bf16 planes,
// `lo` bytes apart, whose sum is the operand.
template <int KIND, int RT, int NT, bool K32, bool SPLIT, bool TAIL>
__device__ __forceinline__ void product_unit(f32x4 (&acc)[RT][NT], const ProductRows<RT, NT>& p, int u, int g, int k,
                                             int64_t lo) {
  const int c = 4 * u + g;
  uint4 w[RT];
  uint32_t ws[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    w[r] = load_chunk<K32, TAIL>(p.wp[r], c, k);
    if constexpr (KIND == kMX) ws[r] = (!TAIL || c * 32 < k) ? p.wc[r][c] : 127u;
    else ws[r] = load_codes<K32, TAIL>(p.wc[r], c, k);
  }
  if constexpr (KIND == kMX) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 x = load_chunk<K32, TAIL>(p.xp[n], c, k);
      const uint32_t xs = (!TAIL || c * 32 < k) ? p.xc[n][c] : 127u;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][n] = mfma_mx(w[r], ws[r], x, xs, acc[r][n]);
    }
  } else {
    uint4 x[NT][4], xl[NT][4];
    if constexpr (KIND == kW4A16) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = !TAIL || c * 32 + 8 * j < k;
          const uint4* src = reinterpret_cast<const uint4*>(p.xp[n] + (int64_t)c * 64) + j;
          x[n][j] = in ? *src : make_uint4(0, 0, 0, 0);
          if constexpr (SPLIT)
            xl[n][j] = in ? *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(src) + lo)
                          : make_uint4(0, 0, 0, 0);
        }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 q = load_chunk<K32, TAIL>(p.xp[n], c, k);
        const uint32_t qs = load_codes<K32, TAIL>(p.xc[n], c, k);
        const f16x2 s0 = splat_f16(e4m3_f32<0>(qs)), s1 = splat_f16(e4m3_f32<1>(qs));
        x[n][0] = fp4x8_f16(q.x, s0);
        x[n][1] = fp4x8_f16(q.y, s0);
        x[n][2] = fp4x8_f16(q.z, s1);
        x[n][3] = fp4x8_f16(q.w, s1);
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float s0 = e4m3_f32<0>(ws[r]), s1 = e4m3_f32<1>(ws[r]);
      const uint32_t wv[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 a = KIND == kW4A16 ? fp4x8_bf16(wv[j], j < 2 ? s0 : s1) : fp4x8_f16(wv[j], splat_f16(j < 2 ? s0 : s1));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (KIND == kW4A16) {
            acc[r][n] = mfma_bf16(a, x[n][j], acc[r][n]);
            if constexpr (SPLIT) acc[r][n] = mfma_bf16(a, xl[n][j], acc[r][n]);
          } else {
            acc[r][n] = mfma_f16(a, x[n][j], acc[r][n]);
          }
        }
      }
    }
  }
}

// Units u0 .. u1-1 of the channel axis (all of them: 0 .. ceil(k / 128)).
template <int KIND, int RT, int NT, bool K32, bool SPLIT, int UNROLL>
__device__ __forceinline__ void product_units(f32x4 (&acc)[RT][NT], const ProductRows<RT, NT>& p, int u0, int u1, int g,
                                              int k, int64_t lo) {
  const int full = min(u1, k >> 7);
  int u = u0;
#pragma unroll UNROLL
  for (; u < full; ++u) product_unit<KIND, RT, NT, K32, SPLIT, false>(acc, p, u, g, k, lo);
  if (u < u1) product_unit<KIND, RT, NT, K32, SPLIT, true>(acc, p, u, g, k, lo);
}

}  // namespace nvfp4
