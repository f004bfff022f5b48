// Device code shared by the kernels that multiply packed 4-bit matrices
// (gfx950): exact expansion of E2M1 nibbles to matrix-core operands, and the
// accumulate of a few output rows against a few tokens.
//
// Three products, all y[t][o] = sum_k x[t][k] w[o][k] with w in 4 bits:
//   kW4A16  x bf16,  w NVFP4.  e2m1 * e4m3 has at most 2 + 4 significant bits
//           and lies in [2^-10, 2688], so it is exact in bf16.
//   kW4A4   both NVFP4.  e2m1 * e4m3 is exact in fp16 as well, and fp16 is
//           cheaper to make: one convert and one packed multiply per pair.
//           (With few tokens the weights enter as e2m1 alone, exact in either,
//           and e4m3 multiplies the fp32 sums of 16.)
//   kMX     both MXFP4: the scaled FP4 matrix instruction takes the packed
//           nibbles and E8M0 bytes as they are.
// The tensor scales (scale_2) stay out of the sum and multiply the fp32
// result, so an operand is never rounded and the products are exact; what
// rounds is the fp32 accumulation and the final conversion.
#pragma once
#include <type_traits>

#include "nvfp4_device.hpp"

namespace nvfp4 {

enum ProductKind { kW4A16 = 0, kW4A4 = 1, kMX = 2 };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
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

// fp32 to bf16, nearest even.
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// v = a + b + c in bf16, 8 bits each, cut off and not rounded: a finite v stays
// finite, and the differences are exact.  An infinity or NaN is in a alone.
__device__ __forceinline__ void split(float v, uint32_t& a, uint32_t& b, uint32_t& c) {
  const uint32_t bits = __float_as_uint(v), top = bits & 0xFFFF0000u;
  const float rest = (bits & 0x7F800000u) == 0x7F800000u ? 0.f : v - __uint_as_float(top);
  const uint32_t middle = __float_as_uint(rest) & 0xFFFF0000u;
  a = top >> 16;
  b = middle >> 16;
  c = __float_as_uint(rest - __uint_as_float(middle)) >> 16;
}

// ---- a few tokens against many rows -----------------------------------------
//
// The weights are read once and everything else is small, so what matters is
// that loads are in flight all the time.  Loads return in order: a wait for one
// is a wait for all before it.  So the tokens, loaded first, stay in registers,
// a quad (512 channels) of them a wave, while the rows go by, and the loop loads
// nothing but weights and their scales, each register again as soon as it has
// been used.  One wave issues a vector instruction every 8 cycles, four waves of a
// SIMD one every 3 to 5 between them, so up to 16 waves share a CU.

constexpr int kCuWaves = 16;
constexpr uint32_t kBeyond = 0x80000000u;           // past any buffer (they are below 2^31 bytes): reads as zero

// A workgroup's waves meet; what they wrote to LDS is seen.  Loads stay in flight.
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

// How k channels are dealt out: `waves` waves a workgroup, of at most `most`,
// QW quads a wave and pass.
struct QuadPlan { int passes, waves; };
template <int QW>
__host__ __device__ inline QuadPlan quad_plan(int64_t k, int most) {
  const int pieces = (int)((k + 512 * QW - 1) / (512 * QW)), passes = (pieces + most - 1) / most;
  return QuadPlan{passes, (pieces + passes - 1) / passes};
}

// NVFP4 weights against 4 NG tokens on the 4x4x4 matrix instruction, whose 16
// blocks are 16 chunks of 32 channels: lane 4 b + i works on chunk b of row i of
// a group of four rows, or of token i of a group of four tokens.  A block of 16
// weights is four instructions; its scale then multiplies their fp32 sum, so
// that the weights enter as plain E2M1 values, one conversion for two of them.
// Per 1 KiB of weights that is 27 vector and 8 matrix instructions for up to
// four tokens, and 52 to 55 vector ones with the exchange, the sums and the
// addresses (counted); the 16x16x32 instruction, which needs the scales in the
// weights, took 132 and held the expert layer to 3.6 TB/s.
//
// Memory is read by lane 16 i + b instead, so that neighbouring lanes read
// neighbouring pieces: a load of 16 bytes a lane looks up a cache line for every
// four lanes that share one, and for every lane that does not (80 lookups a KiB
// the one way, 20 the other, one a cycle).  A trip through a KiB of LDS of the
// wave's own exchanges the two orders.

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Where a lane reads in four rows of a quad, from the first of them on: its
// chunk's weights and its two codes.  Codes past channel k are past the buffer
// and read as zero.  ODD: k is no multiple of 32, so that rows of codes start at
// odd addresses and the last chunk of a row has one code; a kernel of its own,
// because the choice inside the loop cost 25 to 50 registers and let it spill
// (2 quads a wave, 4096x12288, five tokens: 42 us against 15).
template <bool ODD>
struct LaneAt {
  uint32_t w, s, s1;
  // row: the lane's (lane / 16, or the last one there is)
  __device__ __forceinline__ LaneAt(uint32_t row, int q, int k) {
    const int b = threadIdx.x & 15, left = k - q * 512 - b * 32;
    w = row * ((uint32_t)k >> 1) + b * 16;
    s = row * ((uint32_t)k >> 4) + b * 2;
    s1 = ODD && left > 16 ? s + 1 : kBeyond;
    if (left <= 0) s = kBeyond;
  }
};

// Four rows' chunk of one quad, as loaded.
struct RowGroup {
  uint4 w;
  uint32_t s;                                        // two codes

  // row: the first of the four in t.  The scalar offset is held to the buffer's
  // size, which keeps the bounds check (lane's offset against size less scalar
  // offset) right for rows past the end.
  template <bool ODD>
  __device__ __forceinline__ void load(const PackedRows& t, uint32_t row, int q, const LaneAt<ODD>& at, int k) {
    const auto bw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.w), 0, (int)t.w_bytes, 0x00020000);
    const auto bs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.s), 0, (int)t.s_bytes, 0x00020000);
    const uint32_t ow = min(row * ((uint32_t)k >> 1) + q * 256, t.w_bytes);
    const uint32_t os = min(row * ((uint32_t)k >> 4) + q * 32, t.s_bytes);
    w = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(bw, (int)at.w, (int)ow, 0));
    if constexpr (!ODD) {
      s = __builtin_amdgcn_raw_buffer_load_b16(bs, (int)at.s, (int)os, 0);
    } else {
      const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b8(bs, (int)at.s, (int)os, 0);
      const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b8(bs, (int)at.s1, (int)os, 0);
      s = lo | hi << 8;
    }
  }

  // From the order of loading to that of the matrix instruction.  In lds (1 KiB)
  // piece i of chunk b is at 64 b + 16 (i', with bits of b): both sides then
  // touch every bank once.
  __device__ __forceinline__ RowGroup arranged(uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
    auto place = [](int b, int i) { return b * 64 + (((b >> 2) ^ (0x9C >> (2 * i) & 3)) << 4); };
    *reinterpret_cast<uint4*>(lds + place(lane & 15, lane >> 4)) = w;
    __builtin_amdgcn_wave_barrier();
    RowGroup r;
    r.w = *reinterpret_cast<const uint4*>(lds + place(lane >> 2, lane & 3));
    r.s = (uint32_t)__builtin_amdgcn_ds_bpermute(((lane & 3) << 4 | lane >> 2) << 2, (int)s);
    __builtin_amdgcn_wave_barrier();
    return r;
  }
};

// A chunk of 32 channels of one token, bf16, two to a word.
typedef uint32_t Chunk[16];

template <int HALF>
__device__ __forceinline__ s16x4 e2m1x4(uint32_t w) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  u32x2_t v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2 * HALF));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2 * HALF + 1));
  return __builtin_bit_cast(s16x4, v);
}
__device__ __forceinline__ s16x4 pair_of(uint32_t a, uint32_t b) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(s16x4, u32x2_t{a, b});
}
// lane i of each four gives its value to all four
template <int I>
__device__ __forceinline__ float quad_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), I * 0x55, 0xF, 0xF, true));
}

// acc[n] += 4 rows x 4 tokens over the lane's chunk (register i: row i; the
// tokens are x[0][n], and x[1][n] to be added to it where PARTS is 2).
template <int NG, int PARTS>
__device__ __forceinline__ void multiply_group(const RowGroup& r, const Chunk (&x)[PARTS][NG], f32x4 (&acc)[NG]) {
  const float s[2] = {e4m3_f32<0>(r.s), e4m3_f32<1>(r.s)};
  const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {                      // the two blocks of 16
    s16x4 a[4];
    a[0] = e2m1x4<0>(w[2 * h]);
    a[1] = e2m1x4<1>(w[2 * h]);
    a[2] = e2m1x4<0>(w[2 * h + 1]);
    a[3] = e2m1x4<1>(w[2 * h + 1]);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          d = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(a[m], pair_of(x[p][n][8 * h + 2 * m], x[p][n][8 * h + 2 * m + 1]), d,
                                                     0, 0, 0);
      acc[n][0] = __builtin_fmaf(quad_lane<0>(s[h]), d[0], acc[n][0]);
      acc[n][1] = __builtin_fmaf(quad_lane<1>(s[h]), d[1], acc[n][1]);
      acc[n][2] = __builtin_fmaf(quad_lane<2>(s[h]), d[2], acc[n][2]);
      acc[n][3] = __builtin_fmaf(quad_lane<3>(s[h]), d[3], acc[n][3]);
    }
  }
}

// Exchanges between the four 16-lane rows of a wave.  swap32: the upper half of
// a with the lower half of b; swap16: rows 1 and 3 of a with rows 0 and 2 of b.
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
__device__ __forceinline__ float add_swap32(float a, float b) {
  uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  swap32(x, y);
  return __uint_as_float(x) + __uint_as_float(y);
}
__device__ __forceinline__ float add_swap16(float a, float b) {
  uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  swap16(x, y);
  return __uint_as_float(x) + __uint_as_float(y);
}
// + the lane N further on (around) in its row of 16
template <int N>
__device__ __forceinline__ float add_ror(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x120 + N, 0xF, 0xF, true));
}

// The sums over a wave's 16 chunks of four row groups, two at a time: first
// pair(a0, a2) and pair(a1, a3), then rest of the two.  Lanes 16 q + j (and + 4,
// + 8, + 12) get row group q, token j.
__device__ __forceinline__ f32x4 sum_chunks_pair(const f32x4& a, const f32x4& b) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = add_swap32(a[e], b[e]);
  return v;
}
__device__ __forceinline__ f32x4 sum_chunks_rest(const f32x4& a, const f32x4& b) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = add_ror<4>(add_ror<8>(add_swap16(a[e], b[e])));
  return v;
}

// Row tiles begin .. end - 1 (four groups of four rows) against 4 NG tokens, by
// a workgroup dealt out as in plan, a quad a wave and pass.  TB tiles make a
// batch, whose partial sums the waves leave in `part` (per wave TB * NG * 16).
//   group_row[q]     the first row of group q in a tile
//   lds              1 KiB of the wave's
//   rows_of(t)       the packed rows from which tile t's are counted
//   load_tokens(q)   starts the loads of the lane's chunks of quad q,
//   take_tokens()    puts them into x
//   done(t, n, q, j, sum)  called once for every row group q of tile t and token
//                    4 n + j, by some thread, with the sum over the waves, added
//                    in their order
template <bool ODD, int NG, int TB, typename RowsOf, typename LoadTokens, typename TakeTokens, typename Done>
__device__ __forceinline__ void stream_rows(int begin, int end, int k, const QuadPlan& plan, const uint32_t (&group_row)[4],
                                            Chunk (&x)[1][NG], f32x4* part, uint8_t* lds, RowsOf rows_of,
                                            LoadTokens load_tokens, TakeTokens take_tokens, Done done) {
  const int lane = threadIdx.x & 63, i = lane & 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = plan.waves, passes = plan.passes;
  constexpr int SLOTS = NG * 16;                     // partial sums of a wave and tile

  RowGroup r[4];
  // what is loaded: tile at_t of pass at_pass of the batch from at_batch on
  int at_batch = begin, at_pass = 0, at_t = begin;
  PackedRows next;
  LaneAt<ODD> at(lane >> 4, wave, k);
  auto aim = [&]() {
    next = rows_of(min(at_t, end - 1));
    if (at_t >= end || (at_pass * waves + wave) * 512 >= k) next.w_bytes = next.s_bytes = 0;
    next = uniform(next);
    if (passes > 1) at = LaneAt<ODD>(lane >> 4, at_pass * waves + wave, k);
  };
  auto load = [&](int q) { r[q].load(next, group_row[q], at_pass * waves + wave, at, k); };
  auto advance = [&]() {
    if (++at_t >= min(end, at_batch + TB)) {
      if (++at_pass == passes) {
        at_pass = 0;
        at_batch += TB;
      }
      at_t = at_batch;
    }
    aim();
  };
  load_tokens(wave);                                 // first, so that taking them awaits no weights
  aim();
#pragma unroll
  for (int q = 0; q < 4; ++q) load((q & 1) * 2 + (q >> 1));          // in order of use
  advance();
  take_tokens();
  for (int batch = begin; batch < end; batch += TB) {
    const int count = min(TB, end - batch);
    for (int pass = 0; pass < passes; ++pass) {
      if (passes > 1 && (pass || batch > begin)) {
        load_tokens(pass * waves + wave);
        __builtin_amdgcn_s_waitcnt(0x0F70);          // vmcnt(0): the loop awaits nothing of the tokens
        take_tokens();
      }
      f32x4* mine = part + wave * TB * SLOTS;
      for (int t = 0; t < count; ++t) {
        f32x4 half[2][NG];                           // groups 0 and 2, groups 1 and 3
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          f32x4 acc[2][NG];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int q = p + 2 * h;
#pragma unroll
            for (int n = 0; n < NG; ++n) acc[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
            const RowGroup w = r[q].arranged(lds);
            load(q);
            __builtin_amdgcn_sched_barrier(0);       // the load goes out here, not where its value is near
            multiply_group<NG, 1>(w, x, acc[h]);
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) half[p][n] = sum_chunks_pair(acc[0][n], acc[1][n]);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          f32x4 v = sum_chunks_rest(half[0][n], half[1][n]);
          if ((lane & 12) == 0) {
            f32x4& slot = mine[n * 16 + (lane >> 4) * 4 + i];
            if (pass) v += slot;
            slot = v;
          }
        }
        mine += SLOTS;
        advance();
      }
    }
    lds_barrier();
    for (int s = threadIdx.x; s < count * SLOTS; s += 64 * waves) {
      f32x4 v = part[s];
      for (int z = 1; z < waves; ++z) v += part[z * TB * SLOTS + s];
      done(batch + s / SLOTS, s / 16 % NG, s / 4 % 4, s & 3, v);
    }
    lds_barrier();                                   // before the next batch's partial sums
  }
}

// Chunks of bf16 rows, in two steps: the lanes of a token (row: that of token
// lane / 16) read neighbouring pieces, channels past k as zero, and then
// exchange them in LDS (4 KiB, the wave's own; pieces of a chunk are swapped
// with its place and token, so that 16 lanes touch every bank once).  With token
// lane % 4, which looks up a cache line for every lane, 16 tokens of
// 4096x12288, weights in the MALL, took 22.9 us, so 17.3.
static __device__ const uint4 kZeroPiece[1] = {};
__device__ __forceinline__ void load_pieces(Chunk& x, const uint8_t* row, int q, int k) {
  const int b = threadIdx.x & 15;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroPiece);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int c = q * 512 + (16 * m + b) * 8;
    const uint4 v = global_load16(c < k ? row + (int64_t)c * 2 : zero);
    x[4 * m] = v.x;
    x[4 * m + 1] = v.y;
    x[4 * m + 2] = v.z;
    x[4 * m + 3] = v.w;
  }
}
__device__ __forceinline__ void pieces_to_chunk(Chunk& x, uint8_t* lds) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));                     // the places are worked out here, not kept in registers
  auto place = [](int token, int chunk, int piece) {
    return token * 1024 + chunk * 64 + ((piece ^ token ^ (chunk >> 2)) & 3) * 16;
  };
#pragma unroll
  for (int m = 0; m < 4; ++m)
    *reinterpret_cast<uint4*>(lds + place(lane >> 4, 4 * m + (lane >> 2 & 3), lane & 3)) =
        make_uint4(x[4 * m], x[4 * m + 1], x[4 * m + 2], x[4 * m + 3]);
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint4 p = *reinterpret_cast<const uint4*>(lds + place(lane & 3, lane >> 2, m));
    x[4 * m] = p.x;
    x[4 * m + 1] = p.y;
    x[4 * m + 2] = p.z;
    x[4 * m + 3] = p.w;
  }
  __builtin_amdgcn_wave_barrier();
}

// A chunk of packed NVFP4 values, expanded (without their tensor scale).
__device__ __forceinline__ void expand_chunk(Chunk& x, const RowGroup& r) {
  const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
  const float s0 = e4m3_f32<0>(r.s), s1 = e4m3_f32<1>(r.s);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint4 p = fp4x8_bf16(w[m], m < 2 ? s0 : s1);
    x[4 * m] = p.x;
    x[4 * m + 1] = p.y;
    x[4 * m + 2] = p.z;
    x[4 * m + 3] = p.w;
  }
}

// MXFP4 weights against 16 NT MXFP4 tokens on the scaled 16x16x128 instruction,
// which takes nibbles and scales as they are.  A unit is 128 channels; lane l
// works on row (token) l % 16 of a tile and, as group g = l / 16, on chunk g of
// 32 consecutive channels of a unit.  The order of channels within a unit does
// not matter as long as both operands share it, so a lane's weights of a unit
// are one 16-byte piece.  The block scales of a quad are 16 bytes of the row;
// group g takes those of unit g and the groups exchange them, which asks memory
// for a quarter of the pieces that loading them unit by unit would.
//
// Memory is read by lane 4 r + g, so that four lanes share a cache line (see
// above): 32 tokens of 4096x12288, weights in the MALL, took 14.3 us with lanes
// l % 16, 9.5 so.
struct MxQuad {
  uint4 w[4];
  uint32_t s;

  // row, g: the lane's row in t and piece (the whole offset is in the lane's part,
  // which is what the bounds check looks at)
  __device__ __forceinline__ void load_unit(int u, const PackedRows& t, uint32_t row, int q, int g, int k) {
    const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.w), 0, (int)t.w_bytes, 0x00020000);
    const uint32_t at = row * ((uint32_t)k >> 1) + q * 256 + g * 16 + u * 64;
    w[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0));
  }
  // Past channel k the weights are the next row's; their scales are 2^-127
  // there, and the tokens zero.
  __device__ __forceinline__ void load_scales(const PackedRows& t, uint32_t row, int q, int g, int k) {
    const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(t.s), 0, (int)t.s_bytes, 0x00020000);
    const uint32_t at = row * ((uint32_t)k >> 5) + q * 16 + g * 4;
    if ((q + 1) * 512 <= k) {
      s = __builtin_amdgcn_raw_buffer_load_b32(b, (int)at, 0, 0);
    } else {                                         // byte by byte: the word may reach past the buffer
      s = 0;
      int left = k - q * 512 - g * 128;
      asm volatile("" : "+v"(left));                 // worked out here, not kept in registers
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(b, (int)(i * 32 < left ? at + i : kBeyond), 0, 0) << (8 * i);
    }
  }
  // Unit u from the order of loading (lane 4 r + g: piece g of row r, a cache line
  // for four lanes) to the instruction's, through 1 KiB of LDS as RowGroup's.
  __device__ __forceinline__ uint4 arranged(int u, uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
    auto place = [](int r, int g) { return r * 64 + (((r >> 2) ^ (0x9C >> (2 * g) & 3)) << 4); };
    *reinterpret_cast<uint4*>(lds + place(lane >> 2, lane & 3)) = w[u];
    __builtin_amdgcn_wave_barrier();
    const uint4 v = *reinterpret_cast<const uint4*>(lds + place(lane & 15, lane >> 4));
    __builtin_amdgcn_wave_barrier();
    return v;
  }
  // the scales of the lane's chunk in the four units, a byte each
  __device__ __forceinline__ uint32_t scales(int g) const {
    const int lane = threadIdx.x & 63;               // from the order of loading, as arranged
    uint32_t a = (uint32_t)__builtin_amdgcn_ds_bpermute(((lane & 15) << 2 | g) << 2, (int)s), b = a;
    swap32(a, b);                                    // units g % 2 and g % 2 + 2
    uint32_t c = __builtin_amdgcn_perm(b, a, g < 2 ? 0x05040100u : 0x07060302u), d = c;
    swap16(c, d);                                    // units 0 and 2, units 1 and 3
    return __builtin_amdgcn_perm(d, c, (g & 1) ? 0x07030501u : 0x06020400u);
  }
};

template <int U>
__device__ __forceinline__ f32x4 mfma_mx_unit(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x4 c) {
  const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, U, (int)sa, U, (int)sb);
}

// Row tiles begin .. end - 1 of 16 rows; as stream_rows, with per wave
// TB * NT * 64 partial sums and done(t, n, l, sum) for every lane l of an
// instruction's result.
template <int NT, int QW, int RT, int TB, typename RowsOf, typename Done>
__device__ __forceinline__ void stream_mx_rows(int begin, int end, int k, const QuadPlan& plan,
                                               const PackedRows (&tokens)[NT], const uint32_t (&token_row)[NT],
                                               f32x4* part, uint8_t* lds, RowsOf rows_of, Done done) {
  static_assert(TB % RT == 0, "whole steps in a batch");
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = plan.waves, passes = plan.passes;
  MxQuad w[RT][QW], x[QW][NT];
  uint32_t xs[QW][NT];
  int at_batch = begin, at_pass = 0, at_t = begin;
  PackedRows next;
  auto quad = [&](int pass, int z) { return (pass * waves + wave) * QW + z; };
  auto aim = [&]() {
    next = rows_of(min(at_t, end - 1));
    if (at_t >= end) next.w_bytes = next.s_bytes = 0;
    next = uniform(next);
  };
  auto rows = [&](int z) {
    PackedRows v = next;
    if (quad(at_pass, z) * 512 >= k) v.w_bytes = v.s_bytes = 0;
    return v;
  };
  auto load_unit = [&](int t, int z, int u) {
    w[t][z].load_unit(u, rows(z), 16 * t + (lane >> 2), quad(at_pass, z), lane & 3, k);
  };
  auto load_scales = [&](int t, int z) { w[t][z].load_scales(rows(z), 16 * t + (lane >> 2), quad(at_pass, z), lane & 3, k); };
  auto advance = [&]() {
    at_t += RT;
    if (at_t >= min(end, at_batch + TB)) {
      if (++at_pass == passes) {
        at_pass = 0;
        at_batch += TB;
      }
      at_t = at_batch;
    }
    aim();
  };
  auto load_tokens = [&](int pass) {
#pragma unroll
    for (int z = 0; z < QW; ++z)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int q = quad(pass, z);
#pragma unroll
        for (int u = 0; u < 4; ++u) x[z][n].load_unit(u, tokens[n], token_row[n], q, lane & 3, k);
        x[z][n].load_scales(tokens[n], token_row[n], q, lane & 3, k);
      }
  };
  auto take_tokens = [&](int pass) {
#pragma unroll
    for (int z = 0; z < QW; ++z)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        xs[z][n] = x[z][n].scales(g);
        const int left = k - quad(pass, z) * 512 - g * 32;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[z][n].w[u] = x[z][n].arranged(u, lds);
          if (left <= u * 128) x[z][n].w[u] = make_uint4(0, 0, 0, 0);
        }
      }
  };
  load_tokens(0);                                    // first, so that taking them awaits no weights
  aim();
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int z = 0; z < QW; ++z) {
      load_scales(t, z);
#pragma unroll
      for (int u = 0; u < 4; ++u) load_unit(t, z, u);
    }
  advance();
  take_tokens(0);
  for (int batch = begin; batch < end; batch += TB) {
    const int count = min(TB, end - batch);
    for (int pass = 0; pass < passes; ++pass) {
      if (passes > 1 && (pass || batch > begin)) {
        load_tokens(pass);
        __builtin_amdgcn_s_waitcnt(0x0F70);          // vmcnt(0): the loop awaits nothing of the tokens
        take_tokens(pass);
      }
      f32x4* mine = part + wave * TB * NT * 64 + lane;
      for (int t = 0; t < count; t += RT) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 sum[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) sum[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int z = 0; z < QW; ++z) {
            MxQuad& m = w[r][z];
            const uint32_t ws = m.scales(g);
            load_scales(r, z);
            uint4 v[4];
            auto unit = [&](auto u) {
              constexpr int U = decltype(u)::value;
#pragma unroll
              for (int n = 0; n < NT; ++n) sum[n] = mfma_mx_unit<U>(v[U], ws, x[z][n].w[U], xs[z][n], sum[n]);
            };
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              v[u] = m.arranged(u, lds);
              load_unit(r, z, u);
              __builtin_amdgcn_sched_barrier(0);     // the load goes out here, not where its value is near
            }
            unit(std::integral_constant<int, 0>{});
            unit(std::integral_constant<int, 1>{});
            unit(std::integral_constant<int, 2>{});
            unit(std::integral_constant<int, 3>{});
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (pass) sum[n] += mine[n * 64];
            mine[n * 64] = sum[n];
          }
          mine += NT * 64;
        }
        advance();
      }
    }
    lds_barrier();
    for (int s = threadIdx.x; s < count * NT * 64; s += 64 * waves) {
      f32x4 v = part[s];
      for (int z = 1; z < waves; ++z) v += part[z * TB * NT * 64 + s];
      done(batch + (s >> 6) / NT, (s >> 6) % NT, s & 63, v);
    }
    lds_barrier();                                   // before the next batch's partial sums
  }
}

}  // namespace nvfp4
