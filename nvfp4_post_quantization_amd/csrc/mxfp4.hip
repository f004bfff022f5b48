// MXFP4 quantizer and dequantizer: E2M1 elements, one E8M0 scale (a power of
// two, "从MXFP4到NVFP4：Model Optimizer混合精度格式转换完全攻略" §1) per 32.
//
//   code = max(floor(log2 amax) - 2 + 127, 0)      amax = max |x| of the block
//   nib  = E2M1 RNE_sat(x / 2^(code - 127))
//   out  = RN_bf16(e2m1(nib) * 2^(code - 127))
//
// With the largest E2M1 exponent 2 taken off, amax / scale lies in [4, 8);
// what lies above 6 saturates.  On the bf16 pattern the scale is the block
// max's exponent field less 2, and gfx950's FP4 converts take the scale as an
// fp32 whose exponent field alone counts, so `code << 23` is that operand for
// every code (0, an fp32 zero, stands for 2^-127).  The converts round the
// exact quotient to nearest even and saturate, for every bf16 input, subnormal
// ones too, at every scale (checked exhaustively in the tests), so nothing
// else is computed per element.  Both kernels are bound by HBM.
#include "common.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
// 8-element units per lane per batch (loads in flight) and workgroups at most.
// 65536x4096, reads and writes together: quantizing takes 127 us (5.3 TB/s) as
// here and 174 with half the workgroups; dequantizing 115 us (5.9 TB/s), 123
// with the quantizer's numbers.
constexpr int kUnits = 4, kGrid = 2048;
constexpr int kOutUnits = 8, kOutGrid = 1 << 20;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Position of flat unit index u (row-major [rows][n]) advanced by fixed
// strides without a 64-bit division per step.
struct UnitStep { int64_t r, g; };
struct UnitPos {
  int64_t r, g;
  __device__ __forceinline__ void advance(const UnitStep& d, int64_t n) {
    r += d.r;
    g += d.g;
    if (g >= n) { g -= n; ++r; }
  }
};

// max over the four lanes of a quad (quad_perm 1,0,3,2 then 2,3,0,1)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
}

__device__ __forceinline__ uint32_t absmax_word(uint32_t m, uint32_t w) {
  return max(m, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
}

template <int SEL>
__device__ __forceinline__ uint32_t to_fp4(uint32_t old, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale, SEL);
}

// Four lanes per block, 8 elements each: one 16-byte load and one 4-byte
// store per lane (a wave covers 1 KiB in and 256 bytes out), the block max by
// two DPP steps within the quad.  A workgroup's batch is contiguous, so that
// its scale bytes fill whole cache lines.
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                  int64_t k, int64_t ldx,
                                                                  uint8_t* __restrict__ packed,
                                                                  uint8_t* __restrict__ e8m0) {
  const int64_t n = k >> 3;                                   // units per row, a multiple of 4
  const int64_t skip = (int64_t)(gridDim.x - 1) * (kThreads * kUnits);
  const UnitStep near{kThreads / n, kThreads % n}, far{skip / n, skip % n};
  const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  UnitPos pos{u0 / n, u0 % n};
  while (pos.r < rows) {
    uint4 v[kUnits];
    UnitPos p = pos;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (p.r < rows) v[j] = ld_nt4(x + p.r * ldx + p.g * 8);
      p.advance(near, n);
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (pos.r < rows) {
        uint32_t m = absmax_word(absmax_word(absmax_word(absmax_word(0u, v[j].x), v[j].y), v[j].z), v[j].w);
        m = quad_max(m);
        const bool finite = m < 0x7F80u;
        const int code = finite ? max((int)(m >> 7) - 2, 0) : 255;
        const float scale = __uint_as_float((uint32_t)code << 23);
        uint32_t o = to_fp4<0>(0u, v[j].x, scale);
        o = to_fp4<1>(o, v[j].y, scale);
        o = to_fp4<2>(o, v[j].z, scale);
        o = to_fp4<3>(o, v[j].w, scale);
        *reinterpret_cast<uint32_t*>(packed + pos.r * (k >> 1) + pos.g * 4) = finite ? o : 0u;
        if ((threadIdx.x & 3) == 0) e8m0[pos.r * (k >> 5) + (pos.g >> 2)] = (uint8_t)code;
      }
      pos.advance(near, n);
    }
    pos.advance(far, n);
  }
}

template <int SEL>
__device__ __forceinline__ uint32_t from_fp4(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

__global__ __launch_bounds__(kThreads) void mxfp4_dequant_kernel(const uint8_t* __restrict__ packed,
                                                                 const uint8_t* __restrict__ e8m0, int64_t rows,
                                                                 int64_t k, uint16_t* __restrict__ out) {
  const int64_t units = rows * (k >> 3);                      // contiguous on both sides: flat
  constexpr int64_t kBatch = kThreads * kOutUnits;
  for (int64_t u = blockIdx.x * kBatch + threadIdx.x; u < units; u += gridDim.x * kBatch) {
    uint32_t w[kOutUnits], c[kOutUnits];
#pragma unroll
    for (int j = 0; j < kOutUnits; ++j) {
      const int64_t q = u + j * kThreads;
      if (q < units) {
        w[j] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(packed) + q);
        c[j] = e8m0[q >> 2];
      }
    }
#pragma unroll
    for (int j = 0; j < kOutUnits; ++j) {
      const int64_t q = u + j * kThreads;
      if (q < units) {
        const float scale = __uint_as_float(c[j] << 23);
        st_nt4(out + q * 8, make_uint4(from_fp4<0>(w[j], scale), from_fp4<1>(w[j], scale), from_fp4<2>(w[j], scale),
                                       from_fp4<3>(w[j], scale)));
      }
    }
  }
}

unsigned grid_for(int64_t units, int batch, int most) {
  const int64_t want = (units + kThreads * batch - 1) / (kThreads * batch);
  return (unsigned)(want < most ? want : most);
}

}  // namespace

int launch_mxfp4_quantize(const uint16_t* x, int64_t rows, int64_t k, int64_t ldx, uint8_t* packed, uint8_t* e8m0,
                          hipStream_t s) {
  mxfp4_quantize_kernel<<<grid_for(rows * (k >> 3), kUnits, kGrid), kThreads, 0, s>>>(x, rows, k, ldx, packed, e8m0);
  return launch_status("mxfp4_quantize_kernel");
}

int launch_mxfp4_dequant(const uint8_t* packed, const uint8_t* e8m0, int64_t rows, int64_t k, uint16_t* out,
                         hipStream_t s) {
  mxfp4_dequant_kernel<<<grid_for(rows * (k >> 3), kOutUnits, kOutGrid), kThreads, 0, s>>>(packed, e8m0, rows, k, out);
  return launch_status("mxfp4_dequant_kernel");
}

}  // namespace nvfp4
