// The term of a low-rank adapter that a product with an NVFP4 weight adds to its
// sums: scale_a * sum_r (sum_k x[t][k] A_a[r][k]) B_a[o][r], a the token's adapter.
#pragma once
#include "tile_device.hpp"

namespace nvfp4 {

// The inner sums u, scaled, come from a launch of their own, in `splits` parts to
// be added up; they are fp32 and enter the matrix instructions as three bf16 parts
// that hold their 24 bits.
struct LoraTerm {
  const int32_t* ids;         // adapter of a token; outside 0 .. count - 1: none (its u is not there)
  const float* u;             // [splits][tokens][rank]
  const uint16_t* b;          // bf16 [count][out][rank]
  const float* ws2;           // tensor scale of the product's weight
  int64_t part;               // floats of a split
  int count, rank, splits;
};

__device__ __forceinline__ bool has_adapter(const LoraTerm& l, int id) { return id >= 0 && id < l.count; }

// Four of a token's u, from r on, of every step-th split from the first on.
__device__ __forceinline__ f32x4 load_u(const LoraTerm& l, int64_t t, int r, int first = 0, int step = 1) {
  const float* src = l.u + t * l.rank + r;
  f32x4 v = *reinterpret_cast<const f32x4*>(src + first * l.part);
#pragma unroll 4
  for (int s = first + step; s < l.splits; s += step) v += *reinterpret_cast<const f32x4*>(src + s * l.part);
  return v;
}

// Whether eight bf16 values are all finite.
__device__ __forceinline__ bool all_finite(const i32x4& v) {
  bool ok = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = (uint32_t)v[e];
    ok &= (x & 0x7F800000u) != 0x7F800000u && (x & 0x7F80u) != 0x7F80u;
  }
  return ok;
}

// Eight bf16 values with zeros for those that are (not) finite.
template <bool FINITE>
__device__ __forceinline__ i32x4 only(const i32x4& v) {
  i32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = (uint32_t)v[e];
    const bool hi = (x & 0x7F800000u) != 0x7F800000u, lo = (x & 0x7F80u) != 0x7F80u;
    r[e] = (int)((hi == FINITE ? x & 0xFFFF0000u : 0) | (lo == FINITE ? x & 0xFFFFu : 0));
  }
  return r;
}
// -1, 0 or 1 by the signs of eight bf16 values.
__device__ __forceinline__ i32x4 signs(const i32x4& v) {
  i32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = (uint32_t)v[e];
    r[e] = (int)((x & 0x80008000u) | (x & 0x7FFF0000u ? 0x3F800000u : 0) | (x & 0x7FFFu ? 0x3F80u : 0));
  }
  return r;
}

// acc (as store_tiles takes it) *= the tensor scale, and the term is added (all waves
// of the workgroup call this).  The u of the tile's BM tokens go to LDS, 64 ranks at a
// time, as the operands that they become.  A wave takes the (adapter, 16 ranks) pairs
// of its tokens one after another, the next two pairs' rows of B on their way; where
// the channels are split, each split takes its share of the pairs.  Tokens of other
// adapters have zeros for u.  Infinities and NaN of B are kept out of that (zero times
// one is NaN, and parts of u are zero, also its tokens' own); sums of their own with
// the signs of u, which its first part has, are then added to those of their tokens.
//
// It runs once a tile, so that its instructions come from memory more often than not:
// loops stay rolled up.  61 tokens of 64 adapters of 4096x12288, rank 16, take 45 us (22
// without adapters), 59 with four pairs at a time unrolled and the splits' shares of the
// channels alone; 8192 tokens of 12288x4096, rank 64, in a graph of such calls 812 us
// and 672 without adapters (on a slower card 856 and 735), 35 of them u.
template <int TN, int TM, int BM, int LDS, int THREADS>
__device__ __forceinline__ void add_lora(const LoraTerm& l, int tokens, int out, f32x16 (&acc)[TN][TM], bool multiplies,
                                         int o0, int tile0, int row0, int split_at, int splits, uint8_t* lds) {
  constexpr int PITCH = 144, PART = BM * PITCH;                  // 64 bf16 and 16 bytes: rows in all banks
  static_assert(3 * PART <= LDS && BM * 8 % THREADS == 0, "u in LDS");
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  int id[TM];
  bool any = false;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int t = tile0 + row0 + 32 * m + l32, v = l.ids[min(t, tokens - 1)];
    id[m] = t >= tokens ? -2 : has_adapter(l, v) ? v : -1;       // -2: no token, whose results nobody takes
    any |= id[m] >= 0;
  }
  const float ws2 = *l.ws2;
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] *= ws2;
  if (!__syncthreads_or(any)) return;
#pragma unroll 1
  for (int c0 = 0; c0 < l.rank; c0 += 64) {
    const int ranks = min(64, l.rank - c0);                      // a multiple of 8
    if (c0) __syncthreads();
    uint64_t live[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) live[m] = __ballot(id[m] >= 0);
    // pairs: adapter a (-1: no more), ranks from r on
    struct Pair { int a, r; i32x4 w[TN]; };
    int a = multiplies ? 0 : -1, r = ranks, count = -1;
    // (past the last rank, and for no pair: some row, which is not used)
    const auto load_b = [&](int a, int r, int n) {
      return *reinterpret_cast<const i32x4*>(l.b + ((int64_t)a * out + min(o0 + 32 * n + l32, out - 1)) * l.rank +
                                             min(c0 + r + 8 * half, l.rank - 8));
    };
    const auto next_pair = [&]() {
      Pair p;
      if (a >= 0) {
        do {
          ++count;
          r += 16;
          if (r >= ranks) {                                      // on to the adapter of the first token that has had none
            r = 0;
            a = -1;
#pragma unroll
            for (int m = TM - 1; m >= 0; --m)
              if (live[m]) a = __builtin_amdgcn_readlane(id[m], __builtin_ctzll(live[m]));
#pragma unroll
            for (int m = 0; m < TM; ++m) live[m] &= ~__ballot(id[m] == a);
          }
        } while (a >= 0 && count % splits != split_at);
      }
      p.a = a;
      p.r = r;
#pragma unroll
      for (int n = 0; n < TN; ++n) p.w[n] = load_b(max(a, 0), r, n);
      return p;
    };
    Pair next = next_pair(), after = next_pair();
    // u, 8 ranks of a token at a time; zeros for a token without an adapter
#pragma unroll 1
    for (int at = threadIdx.x; at < BM * 8; at += THREADS) {
      const int t = tile0 + (at >> 3), k = (at & 7) * 8, row = min(t, tokens - 1);
      const bool have = t < tokens && k < ranks && has_adapter(l, l.ids[row]);
      const float* src = l.u + (int64_t)row * l.rank + c0 + (k < ranks ? k : 0);
      f32x4 u[2] = {*reinterpret_cast<const f32x4*>(src), *reinterpret_cast<const f32x4*>(src + 4)};
#pragma unroll 1
      for (int s = 1; s < l.splits; ++s) {
        src += l.part;
        u[0] += *reinterpret_cast<const f32x4*>(src);
        u[1] += *reinterpret_cast<const f32x4*>(src + 4);
      }
      uint32_t p[3][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) split(have ? u[e >> 2][e & 3] : 0.f, p[0][e], p[1][e], p[2][e]);
#pragma unroll
      for (int z = 0; z < 3; ++z)
        *reinterpret_cast<uint4*>(lds + z * PART + (at >> 3) * PITCH + k * 2) = make_uint4(
            p[z][0] | p[z][1] << 16, p[z][2] | p[z][3] << 16, p[z][4] | p[z][5] << 16, p[z][6] | p[z][7] << 16);
    }
    __syncthreads();
#pragma unroll 1
    while (next.a >= 0) {
      const Pair now = next;
      next = after;
      after = next_pair();
      // past the last rank: zeros, not another rank's values against u's zeros
      const bool in = now.r + 8 * half < ranks;
      i32x4 b[TN];
      bool finite = true;
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        b[n] = in ? now.w[n] : i32x4{0, 0, 0, 0};
        finite &= all_finite(b[n]);
      }
      finite = !__ballot(!finite);
      if (__builtin_expect(!finite, 0))
#pragma unroll
        for (int n = 0; n < TN; ++n) b[n] = only<true>(b[n]);
      const uint8_t* u = lds + (row0 + l32) * PITCH + (now.r + 8 * half) * 2;
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const bool mine = id[m] == now.a;
        if (!__ballot(mine)) continue;
        i32x4 x[3];
#pragma unroll
        for (int z = 0; z < 3; ++z) {
          x[z] = *reinterpret_cast<const i32x4*>(u + z * PART + m * 32 * PITCH);
          x[z] = mine ? x[z] : i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int z = 0; z < 3; ++z)
#pragma unroll
          for (int n = 0; n < TN; ++n)
            acc[n][m] = mfma32_16<false>(__builtin_bit_cast(uint4, b[n]), __builtin_bit_cast(uint4, x[z]), acc[n][m]);
      }
      if (__builtin_expect(finite, 1)) continue;
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        // (its rows of B once more: kept from before, they cost every call registers)
        const i32x4 w = only<false>(in ? load_b(now.a, now.r, n) : i32x4{0, 0, 0, 0});
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const bool mine = id[m] == now.a;
          if (!__ballot(mine)) continue;
          const i32x4 x = signs(*reinterpret_cast<const i32x4*>(u + m * 32 * PITCH));
          f32x16 sum;
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[e] = 0.f;
          sum = mfma32_16<false>(__builtin_bit_cast(uint4, w), __builtin_bit_cast(uint4, x), sum);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[n][m][e] += mine ? sum[e] : 0.f;
        }
      }
    }
  }
  __syncthreads();                                               // the results go through LDS next
}

}  // namespace nvfp4
