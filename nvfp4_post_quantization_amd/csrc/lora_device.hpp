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

// acc (as store_tiles takes it) *= the tensor scale, and the term is added where
// `add` (the same for a workgroup; all its waves call this).  The u of the tile's BM
// tokens go to LDS, 64 ranks at a time, as the operands that they become.  A wave
// then takes the (adapter, 16 ranks) pairs of its tokens, several at a time, so that
// one wait serves their rows of B.  A token takes the sums of its own adapter alone,
// so that another's infinities do not reach it; 32 tokens of one adapter need no
// choice.
template <int TN, int TM, int BM, int LDS>
__device__ __forceinline__ void add_lora(const LoraTerm& l, int tokens, int out, f32x16 (&acc)[TN][TM], bool multiplies,
                                         int o0, int tile0, int row0, bool add, uint8_t* lds) {
  constexpr int PITCH = 144, PART = BM * PITCH, ITEMS = 4;     // 64 bf16 and 16 bytes: rows in all banks
  static_assert(3 * PART <= LDS, "u in LDS");
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const float ws2 = *l.ws2;
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] *= ws2;
  if (!add) return;
  bool any = false;
#pragma unroll
  for (int r = 0; r < BM; r += 64) {
    const int t = tile0 + r + lane;
    any |= r + lane < BM && t < tokens && has_adapter(l, l.ids[t]);
  }
  if (!__ballot(any)) return;                        // (the same for all waves)
  int id[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int t = tile0 + row0 + 32 * m + l32;
    id[m] = t < tokens ? l.ids[t] : -2;              // -2: no token, whose results nobody takes
    if (id[m] != -2 && !has_adapter(l, id[m])) id[m] = -1;
  }
  for (int c0 = 0; c0 < l.rank; c0 += 64) {
    const int ranks = min(64, l.rank - c0);          // a multiple of 8
    if (c0) __syncthreads();
    for (int i = threadIdx.x; i < BM * 8; i += blockDim.x) {
      const int row = i >> 3, r = (i & 7) * 8, t = tile0 + row;
      uint32_t p[3][8] = {};
      if (r < ranks && t < tokens && has_adapter(l, l.ids[t])) {
        const f32x4 a = load_u(l, t, c0 + r), b = load_u(l, t, c0 + r + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          split(a[e], p[0][e], p[1][e], p[2][e]);
          split(b[e], p[0][4 + e], p[1][4 + e], p[2][4 + e]);
        }
      }
#pragma unroll
      for (int z = 0; z < 3; ++z)
        *reinterpret_cast<uint4*>(lds + z * PART + row * PITCH + r * 2) = make_uint4(
            p[z][0] | p[z][1] << 16, p[z][2] | p[z][3] << 16, p[z][4] | p[z][5] << 16, p[z][6] | p[z][7] << 16);
    }
    __syncthreads();
    if (!multiplies) continue;
    uint64_t live[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) live[m] = __ballot(id[m] >= 0);
    int a = -1, r = ranks;                           // the pair that was last
    for (bool more = true; more;) {
      int item_a[ITEMS], item_r[ITEMS];
      uint4 w[ITEMS][TN];
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        r += 16;
        if (r >= ranks) {                            // on to the adapter of the first token that has had none
          r = 0;
          a = -1;
#pragma unroll
          for (int m = TM - 1; m >= 0; --m)
            if (live[m]) a = __builtin_amdgcn_readlane(id[m], __builtin_ctzll(live[m]));
#pragma unroll
          for (int m = 0; m < TM; ++m) live[m] &= ~__ballot(id[m] == a);
        }
        item_a[i] = a;
        item_r[i] = r;
        if (a < 0) r = ranks;                        // there is none any more
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          w[i][n] = make_uint4(0, 0, 0, 0);
          if (a >= 0 && r + 8 * half < ranks)
            w[i][n] = *reinterpret_cast<const uint4*>(
                l.b + ((int64_t)a * out + min(o0 + 32 * n + l32, out - 1)) * l.rank + c0 + r + 8 * half);
        }
      }
      more = a >= 0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (item_a[i] < 0) break;
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const bool mine = id[m] == item_a[i];
          if (!__ballot(mine)) continue;
          uint4 u[3];
#pragma unroll
          for (int z = 0; z < 3; ++z)
            u[z] = *reinterpret_cast<const uint4*>(lds + z * PART + (row0 + 32 * m + l32) * PITCH + (item_r[i] + 8 * half) * 2);
          if (!__ballot(!mine && id[m] != -2)) {
#pragma unroll
            for (int n = 0; n < TN; ++n)
#pragma unroll
              for (int z = 0; z < 3; ++z) acc[n][m] = mfma32_16<false>(w[i][n], u[z], acc[n][m]);
          } else {
#pragma unroll
            for (int n = 0; n < TN; ++n) {
              f32x16 sum;
#pragma unroll
              for (int e = 0; e < 16; ++e) sum[e] = 0.f;
#pragma unroll
              for (int z = 0; z < 3; ++z) sum = mfma32_16<false>(w[i][n], u[z], sum);
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[n][m][e] += mine ? sum[e] : 0.f;
            }
          }
        }
      }
    }
  }
  __syncthreads();                                   // the results go through LDS next
}

}  // namespace nvfp4
