// Low-rank adapters of many requests at once beside a shared W4A16 projection:
//
//   y[t][o] = RN_bf16( w_scale2 sum_k x[t][k] v[o][k] + scale_a sum_r u[t][r] B_a[o][r] )
//   u[t][r] = sum_k x[t][k] A_a[r][k],  a the token's adapter
//
// Two launches (and the product's own third where it splits the channels): u in
// fp32 here, and the product, whose last step adds the term (matmul.hip,
// matmul_tile.hip), so that nothing is rounded but y.
//
// u: a wave takes 16 or 32 tokens and a run of channels, and the adapters of its
// tokens one after another on the 16x16x32 bf16 instruction, whose columns are the
// tokens: each column of the result belongs to one token, which takes that of its
// own adapter.  Where tokens follow in runs of a request that is one pass over x.
// The waves of a workgroup add up their channels in LDS; what other
// workgroups have of the same tokens are the splits that the product adds up.  Bound
// by the wait for x and A: 8192 tokens of 4096 channels, rank 64, 35 us, 1.9 TB/s of
// x (64 tokens and 4 waves a workgroup took half as long again).
#include "layer.hpp"
#include "lora_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kMaxSplits = 4, kFewSplits = 16;      // up to 16 tokens: the most

struct InnerArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const uint16_t* a;          // [count][rank][k]
  const float* scale;
  float* u;                   // [splits][tokens][rank]
  int64_t part;
  int tokens, k, count, rank, splits;
};

__device__ __forceinline__ f32x4 mfma16_bf16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 16 NT tokens (x), a split of the channels (y), every gridDim.z-th of their
// adapters (z).  RT tiles of 16 rows of A at a time, NB steps of 32 channels.
template <int NT, int RT, int NB, int W>
__global__ __launch_bounds__(64 * W) void lora_inner_kernel(InnerArgs p) {
  __shared__ __attribute__((aligned(16))) f32x4 part[W][NT * RT][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 16 * NT;
  // the wave's steps of 32 channels
  const int steps = (p.k + 31) >> 5, parts = p.splits * W, at = blockIdx.y * W + wave;
  const int s0 = (int)((int64_t)steps * at / parts), s1 = (int)((int64_t)steps * (at + 1) / parts);
  int id[NT];
  const uint16_t* x[NT];
  uint64_t live[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = t0 + 16 * n + l16;
    id[n] = t < p.tokens ? p.ids[t] : -1;
    if (id[n] < 0 || id[n] >= p.count) id[n] = -1;
    live[n] = __ballot(id[n] >= 0);
    x[n] = p.x + (int64_t)min(t, p.tokens - 1) * p.ldx + q * 8;
  }
  const i32x4 zero = {0, 0, 0, 0};
  for (int turn = 0;; ++turn) {
    // the next adapter: that of the first token that has had none
    int a = -1;
#pragma unroll
    for (int n = NT - 1; n >= 0; --n)
      if (live[n]) a = __builtin_amdgcn_readlane(id[n], __builtin_ctzll(live[n]));
    if (a < 0) break;
    uint64_t has[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      has[n] = __ballot(id[n] == a);
      live[n] &= ~has[n];
    }
    if (turn % (int)gridDim.z != (int)blockIdx.z) continue;
    for (int r0 = 0; r0 < p.rank; r0 += 16 * RT) {
      const uint16_t* rows[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r)                   // (rows past the last: it again, their results are not stored)
        rows[r] = p.a + ((int64_t)a * p.rank + min(r0 + 16 * r + l16, p.rank - 1)) * p.k + q * 8;
      const float scale = p.scale[a];
      f32x4 acc[NT][RT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[n][r] = f32x4{0.f, 0.f, 0.f, 0.f};
      // NB steps are on their way at a time; the last ones, where k or the wave's steps
      // end, load what there is and take zeros for the rest
      const auto steps_from = [&](int s, auto all) {
        i32x4 w[NB][RT], v[NB][NT];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int c = (s + i) * 32, at = all ? c : min(c, p.k - 8 - q * 8);
#pragma unroll
          for (int r = 0; r < RT; ++r) w[i][r] = *reinterpret_cast<const i32x4*>(rows[r] + at);
#pragma unroll
          for (int n = 0; n < NT; ++n) v[i][n] = *reinterpret_cast<const i32x4*>(x[n] + at);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if (!all) {
            const bool in = s + i < s1 && (s + i) * 32 + q * 8 < p.k;        // (k is a multiple of 16)
#pragma unroll
            for (int r = 0; r < RT; ++r) w[i][r] = in ? w[i][r] : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) v[i][n] = in ? v[i][n] : zero;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (has[n])
#pragma unroll
              for (int r = 0; r < RT; ++r) acc[n][r] = mfma16_bf16(w[i][r], v[i][n], acc[n][r]);
        }
      };
      int s = s0;
      if constexpr (NT > 1)                          // (few steps a wave: one loop, for its code comes from memory too)
        for (; s + NB <= min(s1, p.k >> 5); s += NB) steps_from(s, std::true_type{});
#pragma unroll 1
      for (; s < s1; s += NB) steps_from(s, std::false_type{});
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r) part[wave][n * RT + r][lane] = acc[n][r];
      __syncthreads();
      for (int i = threadIdx.x; i < NT * RT * 64; i += 64 * W) {
        const int l = i & 63, n = (i >> 6) / RT, r = r0 + 16 * ((i >> 6) % RT) + 4 * (l >> 4);
        const int t = t0 + 16 * n + (l & 15);
        if (r >= p.rank || t >= p.tokens || p.ids[t] != a) continue;
        f32x4 v = part[0][i >> 6][l];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][i >> 6][l];
        *reinterpret_cast<f32x4*>(p.u + blockIdx.y * p.part + (int64_t)t * p.rank + r) = v * scale;
      }
      __syncthreads();
    }
  }
}

// Tokens and waves of a workgroup, splits of the channels (each wave has two steps
// or more), slots of a token group's adapters.
struct InnerPlan { int tokens, waves, splits, slots; };
InnerPlan plan_inner(int64_t tokens, int64_t k) {
  InnerPlan p;
  p.tokens = tokens <= 1024 ? 16 : 32;
  p.waves = 8;
  const int64_t groups = (tokens + p.tokens - 1) / p.tokens, want = (2 * kCus + groups - 1) / groups;
  int64_t splits = k / (64 * p.waves);
  if (splits > want) splits = want;
  if (splits > (groups > 1 ? kMaxSplits : kFewSplits)) splits = groups > 1 ? kMaxSplits : kFewSplits;
  p.splits = splits < 1 ? 1 : (int)splits;
  const int64_t slots = want / p.splits, adapters = tokens < 16 ? tokens : 16;
  p.slots = (int)(slots < 1 ? 1 : slots < adapters ? slots : adapters);
  return p;
}

// Tokens of a launch: 512 threads for every 32 of them, of fewer than 2^32 (with more the
// launch takes them modulo 2^32, without an error).
constexpr int64_t kLaunchTokens = INT64_C(1) << 27;

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t lora_workspace_bytes(int64_t tokens, int64_t out, int64_t k, int64_t rank) {
  return align256(product_workspace_bytes(tokens, out, k, false)) + (size_t)plan_inner(tokens, k).splits * tokens * rank * 4;
}

int launch_w4a16_lora(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx, const uint8_t* wp, const uint8_t* wc,
                      const float* ws2, int64_t out, const Adapters& ad, uint16_t* y, int64_t ldy, void* workspace,
                      hipStream_t s) {
  const InnerPlan plan = plan_inner(tokens, k);
  float* u = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                      align256(product_workspace_bytes(tokens, out, k, false)));
  const int64_t part = tokens * ad.rank;
  for (int64_t t = 0; t < tokens; t += kLaunchTokens) {
    const int64_t here = tokens - t < kLaunchTokens ? tokens - t : kLaunchTokens;
    const InnerArgs p{x + t * ldx, ldx, ad.ids + t, ad.a, ad.scale, u + t * ad.rank, part, (int)here, (int)k, ad.count, ad.rank,
                      plan.splits};
    const dim3 grid((unsigned)((here + plan.tokens - 1) / plan.tokens), plan.splits, plan.slots);
    if (plan.tokens == 16) {
      if (ad.rank <= 16) lora_inner_kernel<1, 1, 4, 8><<<grid, 512, 0, s>>>(p);
      else lora_inner_kernel<1, 4, 4, 8><<<grid, 512, 0, s>>>(p);
    } else {
      if (ad.rank <= 16) lora_inner_kernel<2, 1, 4, 8><<<grid, 512, 0, s>>>(p);
      else lora_inner_kernel<2, 4, 2, 8><<<grid, 512, 0, s>>>(p);
    }
    const int st = launch_status("lora_inner_kernel");
    if (st) return st;
  }
  const LoraTerm l{ad.ids, u, ad.b, ws2, part, ad.count, ad.rank, plan.splits};
  return launch_matmul_w4a16(x, tokens, k, ldx, wp, wc, ws2, out, y, ldy, workspace, s, &l);
}

}  // namespace nvfp4
