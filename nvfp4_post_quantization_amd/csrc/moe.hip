// A mixture-of-experts layer over NVFP4 experts for a few tokens, in the
// layout the MXFP4 -> NVFP4 cast leaves them (w1 and w3 of an expert share a
// tensor scale, "从MXFP4到NVFP4：Model Optimizer混合精度格式转换完全攻略" §3):
//
//   y[t] = sum over the experts e chosen for t of
//          weight(t, e) * W2_e ( silu(W1_e x[t]) * (W3_e x[t]) )
//
// The experts' weights, read once each, bound the layer.  Two launches: the
// first makes h = weight * s2 * silu(gate) * up for every (token, expert)
// pair, the second adds W2_e h over the experts of each token inside the
// matrix accumulators, in a fixed order, so the result is reproducible.
// Who goes where is worked out again from the ids by every workgroup (at
// most 1024 of them), which costs less than a launch that writes it down.
#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kMaxIds = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kUpWaves = 8;
constexpr int kDownWaves = 8;

struct MoeArgs {
  const uint8_t* x;               // bf16 rows
  int64_t ldx;                    // in bytes
  const int32_t* ids;
  const float* weights;
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
  uint16_t* y;
  int64_t ldy;
  uint16_t* h;                    // [tokens * top_k][inter] bf16, then the same for the low parts
  int64_t lo;                     // bytes from a value's high part to its low part
  int tokens, hidden, inter, experts, top_k;
};

struct Routing {
  int32_t ids[kMaxIds];
  uint32_t bits[kMoeMaxExperts / 32];
  uint16_t active[kMoeMaxExperts];        // the chosen experts in ascending order
  int count;
};

// Fill r from the ids (all threads; syncs).
__device__ __forceinline__ void read_routing(Routing& r, const MoeArgs& a) {
  const int n = a.tokens * a.top_k;
  for (int i = threadIdx.x; i < kMoeMaxExperts / 32; i += blockDim.x) r.bits[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = a.ids[i];
    const bool ok = e >= 0 && e < a.experts;
    r.ids[i] = ok ? e : -1;
    if (ok) atomicOr(&r.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (threadIdx.x < kMoeMaxExperts / 32) {
    int base = 0;
    for (int i = 0; i < (int)threadIdx.x; ++i) base += __popc(r.bits[i]);
    uint32_t b = r.bits[threadIdx.x];
    while (b) {
      r.active[base++] = (uint16_t)(threadIdx.x * 32 + __ffs(b) - 1);
      b &= b - 1;
    }
    if (threadIdx.x == kMoeMaxExperts / 32 - 1) r.count = base;
  }
  __syncthreads();
}

// First place s of expert e among token t's choices, or -1; *weight adds up
// all of them (an expert named twice counts once, with both weights).
__device__ __forceinline__ int find_choice(const Routing& r, const MoeArgs& a, int t, int e, float* weight) {
  int first = -1;
  float w = 0.f;
  for (int s = a.top_k - 1; s >= 0; --s) {
    if (r.ids[t * a.top_k + s] == e) {
      first = s;
      if (weight) w += a.weights[t * a.top_k + s];
    }
  }
  if (weight) *weight = w;
  return first;
}

// h of 16 channels of one expert for its tokens, 16 NT at a time.
template <int NT, bool K32>
__device__ __forceinline__ void up_tile(const MoeArgs& a, int e, int row0, int first, int count, const uint8_t* tok,
                                        const uint16_t* slot, const float* wt, f32x4* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  ProductRows<2, NT> p;
#pragma unroll
  for (int r = 0; r < 2; ++r) {                                  // gate row and up row
    const int64_t row = ((int64_t)e * 2 + r) * a.inter + min(row0 + (lane & 15), a.inter - 1);
    p.wp[r] = a.p13 + row * (a.hidden >> 1);
    p.wc[r] = a.c13 + row * (a.hidden >> 4);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    p.xp[n] = a.x + tok[min(first + 16 * n + (lane & 15), count - 1)] * a.ldx;
    p.xc[n] = nullptr;
  }
  f32x4 acc[2][NT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int units = (a.hidden + 127) >> 7, per = (units + kUpWaves - 1) / kUpWaves;
  product_units<kW4A16, 2, NT, K32, false, (NT > 1 ? 1 : 2)>(acc, p, min(wave * per, units), min((wave + 1) * per, units),
                                                            lane >> 4, a.hidden, 0);
  __syncthreads();                                               // the last tile's sums are done with
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) part[(wave * 2 * NT + r * NT + n) * 64 + lane] = acc[r][n];
  __syncthreads();
  const float s13 = a.s13[e], s2 = a.s2[e];
  for (int i = threadIdx.x; i < NT * 64; i += 64 * kUpWaves) {
    const int n = i >> 6, l = i & 63;
    f32x4 g = part[n * 64 + l], u = part[(NT + n) * 64 + l];
#pragma unroll
    for (int w = 1; w < kUpWaves; ++w) {
      g += part[(w * 2 * NT + n) * 64 + l];
      u += part[(w * 2 * NT + NT + n) * 64 + l];
    }
    const int c = first + 16 * n + (l & 15), row = row0 + 4 * (l >> 4);
    if (c < count) {
      const float scale = wt[c] * s2;
      uint16_t* dst = a.h + (int64_t)slot[c] * a.inter + row;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (row + q < a.inter) {
          const float gate = g[q] * s13, up = u[q] * s13;
          const float h = gate / (1.0f + expf(-gate)) * up * scale;
          // two bf16 parts keep 16 significant bits of h
          const uint16_t hi = to_bf16(h);
          dst[q] = hi;
          *reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(dst + q) + a.lo) = to_bf16(h - bf16_to_f32(hi));
        }
      }
    }
  }
}

template <bool K32>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ uint8_t tok[kMoeMaxTokens];
  __shared__ uint16_t slot[kMoeMaxTokens];
  __shared__ float wt[kMoeMaxTokens];
  __shared__ int count;
  __shared__ f32x4 part[kUpWaves * 2 * 2 * 64];
  read_routing(r, a);
  const int row0 = blockIdx.x * 16;
  if ((int)blockIdx.y >= r.count) return;
  const int e = r.active[blockIdx.y];
  if (threadIdx.x < 64) {
    const int t = threadIdx.x;
    float w = 0.f;
    const int s = t < a.tokens ? find_choice(r, a, t, e, &w) : -1;
    const uint64_t mask = __ballot(s >= 0);
    if (s >= 0) {
      const int at = __popcll(mask & ((1ull << t) - 1));
      tok[at] = (uint8_t)t;
      slot[at] = (uint16_t)(t * a.top_k + s);
      wt[at] = w;
    }
    if (t == 0) count = __popcll(mask);
  }
  __syncthreads();
  const int n = count;
  if (n <= 16) {
    up_tile<1, K32>(a, e, row0, 0, n, tok, slot, wt, part);
  } else {
    for (int first = 0; first < n; first += 32) up_tile<2, K32>(a, e, row0, first, n, tok, slot, wt, part);
  }
}

// 16 output channels for all tokens.  The workgroup's waves share out
// (expert, channel part) items.  An item's product has a column for every
// token; each wave adds the columns of the tokens that the expert serves to
// its own sums, item after item, and drops the rest (so a NaN in an expert's
// scales reaches its own tokens only).  The waves are added at the end.
template <int NT, bool K32>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ f32x4 part[kDownWaves][NT][64];
  read_routing(r, a);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row0 = blockIdx.x * 16;
  const int units = (a.inter + 127) >> 7;
  int parts = 1;
  while (parts < units && r.count * parts < 4 * kDownWaves) parts *= 2;
  const int per = (units + parts - 1) / parts;
  const int64_t row = min(row0 + (lane & 15), a.hidden - 1);
  const uint8_t* h = reinterpret_cast<const uint8_t*>(a.h);
  f32x4 sum[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) sum[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = wave; i < r.count * parts; i += kDownWaves) {
    const int e = r.active[i / parts], part_i = i % parts;
    const int s = lane < a.tokens ? find_choice(r, a, lane, e, nullptr) : -1;
    const uint64_t mask = __ballot(s >= 0);
    // other tokens' lanes read the first served token's row, whatever comes of it
    const int any = __shfl(lane * a.top_k + s, __ffsll((unsigned long long)mask) - 1);
    const int slot = s >= 0 ? lane * a.top_k + s : any;
    ProductRows<1, NT> p;
    const int64_t er = (int64_t)e * a.hidden + row;
    p.wp[0] = a.p2 + er * (a.inter >> 1);
    p.wc[0] = a.c2 + er * (a.inter >> 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      p.xp[n] = h + (int64_t)__shfl(slot, 16 * n + (lane & 15)) * a.inter * 2;
      p.xc[n] = nullptr;
    }
    f32x4 acc[1][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[0][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    product_units<kW4A16, 1, NT, K32, true, 1>(acc, p, min(part_i * per, units), min((part_i + 1) * per, units),
                                               lane >> 4, a.inter, a.lo);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if ((mask >> (16 * n + (lane & 15))) & 1) sum[n] += acc[0][n];
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) part[wave][n][lane] = sum[n];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 64; i += 64 * kDownWaves) {
    const int n = i >> 6, l = i & 63;
    f32x4 v = part[0][n][l];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) v += part[w][n][l];
    const int t = 16 * n + (l & 15), o = row0 + 4 * (l >> 4);
    if (t < a.tokens) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (o + q < a.hidden) a.y[t * a.ldy + o + q] = to_bf16(v[q]);
    }
  }
}

template <bool K32>
void run_down(const MoeArgs& a, hipStream_t s) {
  const dim3 grid((a.hidden + 15) / 16);
  if (a.tokens <= 16) moe_down_kernel<1, K32><<<grid, 64 * kDownWaves, 0, s>>>(a);
  else if (a.tokens <= 32) moe_down_kernel<2, K32><<<grid, 64 * kDownWaves, 0, s>>>(a);
  else moe_down_kernel<4, K32><<<grid, 64 * kDownWaves, 0, s>>>(a);
}

// One wave per token.  Lane l holds the logits of experts l, l + 64, ...;
// each of the top_k rounds takes the wave's largest remaining one.
template <int PER>
__global__ __launch_bounds__(256) void moe_route_kernel(const float* __restrict__ logits, int64_t tokens, int experts,
                                                        int64_t ldl, int top_k, int normalize,
                                                        int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  const float ninf = -__builtin_inff();
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const float l = e < experts ? logits[t * ldl + e] : ninf;
    v[i] = l > ninf ? fminf(l, 3.40282347e38f) : ninf;           // NaN is out, like -inf
  }
  float top = 0.f, mine = 0.f, sum = 0.f;
  int my_id = -1;
  for (int s = 0; s < top_k; ++s) {
    float bv = v[0];
    int bi = lane;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (v[i] > bv) { bv = v[i]; bi = lane + 64 * i; }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
      const float ov = __shfl_xor(bv, m);
      const int oi = __shfl_xor(bi, m);
      if (ov > bv || (ov == bv && oi < bi)) { bv = ov; bi = oi; }
    }
    if (s == 0) {
      top = bv;
      if (!normalize) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) z += v[i] > ninf ? expf(v[i] - bv) : 0.f;
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) z += __shfl_xor(z, m);
        sum = z;
      }
    }
    const bool some = bv > ninf;
    const float p = some ? expf(bv - top) : 0.f;
    if (normalize) sum += p;
    if (lane == s) { mine = p; my_id = some ? bi : -1; }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i == bi) v[i] = ninf;
  }
  if (lane < top_k) {
    ids[t * top_k + lane] = my_id;
    weights[t * top_k + lane] = my_id >= 0 ? mine / sum : 0.f;
  }
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t inter) {
  const size_t plane = ((size_t)(tokens * top_k) * (size_t)inter * 2 + 255) & ~(size_t)255;
  return 2 * plane;
}

int launch_moe_route(const float* logits, int64_t tokens, int64_t experts, int64_t ldl, int top_k, int normalize,
                     int32_t* ids, float* weights, hipStream_t s) {
  const unsigned grid = (unsigned)((tokens + 3) / 4);
  const int e = (int)experts;
  if (e <= 64) moe_route_kernel<1><<<grid, 256, 0, s>>>(logits, tokens, e, ldl, top_k, normalize, ids, weights);
  else if (e <= 128) moe_route_kernel<2><<<grid, 256, 0, s>>>(logits, tokens, e, ldl, top_k, normalize, ids, weights);
  else if (e <= 256) moe_route_kernel<4><<<grid, 256, 0, s>>>(logits, tokens, e, ldl, top_k, normalize, ids, weights);
  else moe_route_kernel<16><<<grid, 256, 0, s>>>(logits, tokens, e, ldl, top_k, normalize, ids, weights);
  return launch_status("moe_route_kernel");
}

int launch_moe_forward(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx, const int32_t* ids,
                       const float* weights, int top_k, int64_t experts, int64_t inter, const uint8_t* w13_packed,
                       const uint8_t* w13_codes, const float* w13_scale2, const uint8_t* w2_packed,
                       const uint8_t* w2_codes, const float* w2_scale2, uint16_t* y, int64_t ldy, void* workspace,
                       hipStream_t s) {
  MoeArgs a;
  a.x = reinterpret_cast<const uint8_t*>(x);
  a.ldx = ldx * 2;
  a.ids = ids;
  a.weights = weights;
  a.p13 = w13_packed;
  a.c13 = w13_codes;
  a.p2 = w2_packed;
  a.c2 = w2_codes;
  a.s13 = w13_scale2;
  a.s2 = w2_scale2;
  a.y = y;
  a.ldy = ldy;
  a.h = reinterpret_cast<uint16_t*>(workspace);
  a.lo = (int64_t)(moe_workspace_bytes(tokens, top_k, inter) / 2);
  a.tokens = (int)tokens;
  a.hidden = (int)hidden;
  a.inter = (int)inter;
  a.experts = (int)experts;
  a.top_k = top_k;
  const int64_t pairs = tokens * top_k;
  const dim3 grid((unsigned)((inter + 15) / 16), (unsigned)(pairs < experts ? pairs : experts));
  if (hidden % 32) moe_up_kernel<false><<<grid, 64 * kUpWaves, 0, s>>>(a);
  else moe_up_kernel<true><<<grid, 64 * kUpWaves, 0, s>>>(a);
  const int st = launch_status("moe_up_kernel");
  if (st) return st;
  if (inter % 32) run_down<false>(a, s);
  else run_down<true>(a, s);
  return launch_status("moe_down_kernel");
}

}  // namespace nvfp4
