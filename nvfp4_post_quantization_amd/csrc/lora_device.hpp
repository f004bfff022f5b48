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

// Eight of a token's u, from r on.
__device__ __forceinline__ void load_u(const LoraTerm& l, int64_t t, int r, float (&v)[8]) {
  const float* src = l.u + t * l.rank + r;
  f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
  for (int s = 1; s < l.splits; ++s) {
    src += l.part;
    a += *reinterpret_cast<const f32x4*>(src);
    b += *reinterpret_cast<const f32x4*>(src + 4);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}

// acc (as store_tiles takes it) = s0 * acc, + the term where `add`.  One adapter of
// a fragment's 32 tokens after another; a token takes the sums of its own alone, so
// that another's infinities do not reach it.
template <int TN, int TM>
__device__ __forceinline__ void add_lora(const LoraTerm& l, int tokens, int out, f32x16 (&acc)[TN][TM], int o0, int t0,
                                         float s0, bool add) {
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[n][m][e] *= s0;
  if (!add) return;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int t = t0 + 32 * m + l32;
    const int id = t < tokens ? l.ids[t] : -1;
    uint64_t live = __ballot(has_adapter(l, id));
    while (live) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(live));
      const bool mine = id == a;
      live &= ~__ballot(mine);
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const uint16_t* b = l.b + ((int64_t)a * out + min(o0 + 32 * n + l32, out - 1)) * l.rank;
        f32x16 sum;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = 0.f;
        for (int r0 = 0; r0 < l.rank; r0 += 16) {
          const int r = r0 + 8 * half;
          uint4 w = make_uint4(0, 0, 0, 0);
          float u[8] = {};
          if (r < l.rank) {
            w = *reinterpret_cast<const uint4*>(b + r);
            if (mine) load_u(l, t, r, u);
          }
          uint32_t p[3][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split(u[e], p[0][e], p[1][e], p[2][e]);
#pragma unroll
          for (int z = 0; z < 3; ++z)
            sum = mfma32_16<false>(w, make_uint4(p[z][0] | p[z][1] << 16, p[z][2] | p[z][3] << 16, p[z][4] | p[z][5] << 16,
                                                 p[z][6] | p[z][7] << 16), sum);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[n][m][e] += mine ? sum[e] : 0.f;
      }
    }
  }
}

}  // namespace nvfp4
