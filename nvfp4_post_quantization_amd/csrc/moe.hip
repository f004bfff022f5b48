// A mixture-of-experts layer over NVFP4 experts for a few tokens, in the
// layout the MXFP4 -> NVFP4 cast leaves them (w1 and w3 of an expert share a
// tensor scale, "从MXFP4到NVFP4：Model Optimizer混合精度格式转换完全攻略" §3):
//
//   y[t] = sum over the experts e chosen for t of
//          weight(t, e) * W2_e ( silu(W1_e x[t]) * (W3_e x[t]) )
//
// The experts' weights, read once each, bound the layer.  Two launches: the
// first makes h = weight * s2 * silu(gate) * up for every (expert, token)
// pair, the second adds W2_e h over the experts of each token, in a fixed
// order, so the result is reproducible.  Who goes where is worked out again
// from the ids by every workgroup (at most 1024 of them), which costs less
// than a launch that writes it down: a 64-bit token mask per expert, and the
// list of the jobs to do.
#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kMaxJobs = kMoeMaxTokens * kMoeMaxTopK;

struct MoeArgs {
  const uint8_t* x;               // bf16 rows
  int64_t ldx;                    // in bytes
  const int32_t* ids;
  const float* weights;
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
  uint16_t* y;
  int64_t ldy;
  uint16_t* h;                    // [pairs][ldh] bf16, then the same for the low parts
  int64_t ldh;                    // inter rounded up to whole quads, zero past inter
  int64_t lo;                     // bytes from a value's high part to its low part
  int tokens, hidden, inter, experts, top_k;
};

// A job is a chosen expert with up to 16 of its tokens.
struct Routing {
  uint32_t mask[kMoeMaxExperts][2];       // tokens of an expert
  uint16_t expert[kMaxJobs];              // by job: its expert, experts in ascending order,
  uint16_t base[kMaxJobs];                // its first pair (rows of h),
  uint8_t first[kMaxJobs];                // its first token's place among the expert's
  uint32_t part[16];                      // per wave: jobs and pairs (upper half)
  int jobs;
};

__device__ __forceinline__ uint64_t tokens_of(const Routing& r, int e) {
  return (uint64_t)r.mask[e][1] << 32 | r.mask[e][0];
}

// Fill r from the ids (all threads, THREADS of them; syncs).
template <int THREADS>
__device__ __forceinline__ void read_routing(Routing& r, const MoeArgs& a) {
  constexpr int PER = kMoeMaxExperts / THREADS;
  const int n = a.tokens * a.top_k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < 2 * a.experts; i += THREADS) (&r.mask[0][0])[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const int e = a.ids[i], t = i / a.top_k;
    if (e >= 0 && e < a.experts) atomicOr(&r.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // prefix sums over the experts, PER of them a thread: jobs in the lower half
  // of the word, pairs (at most 1024) in the upper
  uint32_t own[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    const uint32_t c = e < a.experts ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0;
    own[i] = (c + 15) >> 4 | c << 16;
    sum += own[i];
  }
  uint32_t scan = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 63) r.part[wave] = scan;
  __syncthreads();
  uint32_t before = scan - sum;
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += r.part[w];
    all += r.part[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    for (int q = 0; q < (int)(own[i] & 0xFFFF); ++q) {
      const int job = (before & 0xFFFF) + q;
      r.expert[job] = (uint16_t)(tid * PER + i);
      r.base[job] = (uint16_t)((before >> 16) + 16 * q);
      r.first[job] = (uint8_t)(16 * q);
    }
    before += own[i];
  }
  if (tid == 0) r.jobs = (int)(all & 0xFFFF);
  __syncthreads();
}

// The place-th set bit of a nonzero mask, for place = first + lane % 16 (the
// last one for places beyond).
__device__ __forceinline__ int token_of_column(uint64_t mask, int first) {
  const int lane = threadIdx.x & 63;
  const int n = __popcll(mask);
  const int rank = __popcll(mask & ((1ull << lane) - 1));
  // lane t sends t to lane rank(t); lanes whose bit is clear send to a lane of
  // their own past the set bits
  const int to = (mask >> lane) & 1 ? rank : n + lane - rank;
  const int t = __builtin_amdgcn_ds_permute(to * 4, lane);
  return __shfl(t, min(first + (lane & 15), n - 1));
}

// What a token gives an expert (all places that name it).
__device__ __forceinline__ float weight_of(const MoeArgs& a, int t, int e) {
  float w = 0.f;
  for (int s = 0; s < a.top_k; ++s)
    if (a.ids[t * a.top_k + s] == e) w += a.weights[t * a.top_k + s];
  return w;
}

// Where channel c of a row of h is kept: within each unit of 128 channels in
// the order in which the second launch's lanes read them, piece j (8 channels)
// of the four chunks of 32 next to each other.
__device__ __forceinline__ int place_of(int c) {
  return (c & ~127) | ((c >> 3) & 3) << 5 | ((c >> 5) & 3) << 3 | (c & 7);
}

// h of a run of (job, 8 channels) tiles, as many runs as there are workgroups.
// A row tile holds the gate rows of the channels in rows 0-7 and their up rows
// in 8-15, so that one pass over the tokens serves both.
template <int QW>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void moe_up_kernel(MoeArgs a) {
  constexpr int RT = 2 / QW, TB = 4 / RT;
  __shared__ Routing r;
  __shared__ f32x4 part[kStreamWaves * TB * RT * 64];
  __shared__ float wt[16];
  read_routing<64 * kStreamWaves>(r, a);
  const int lane = threadIdx.x & 63, r16 = lane & 15;
  const int tiles = a.inter >> 3;
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(r.jobs) * tiles;
  int64_t begin = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  const uint32_t ldw = (uint32_t)a.hidden >> 1, lds = (uint32_t)a.hidden >> 4;
  const uint32_t row = (r16 >> 3) * (uint32_t)a.inter + (r16 & 7);
  while (begin < end) {                              // one job after another
    const int job = __builtin_amdgcn_readfirstlane((int)(begin / tiles));
    const int t0 = __builtin_amdgcn_readfirstlane((int)(begin - (int64_t)job * tiles));
    const int t1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)tiles, t0 + end - begin));
    begin += t1 - t0;
    const int e = __builtin_amdgcn_readfirstlane(r.expert[job]), first = r.first[job], base = r.base[job];
    const uint64_t mask = tokens_of(r, e);
    const int count = min(16, __popcll(mask) - first);
    const int tok = token_of_column(mask, first);
    if (threadIdx.x < 16) wt[threadIdx.x] = weight_of(a, tok, e) * a.s2[e];
    const float s13 = a.s13[e];
    const uint8_t* w = a.p13 + (int64_t)e * 2 * a.inter * ldw;
    const uint8_t* c = a.c13 + (int64_t)e * 2 * a.inter * lds;
    TokenRows tokens[1];
    tokens[0].x = a.x + tok * a.ldx;
    auto rows_of = [&](int t) {
      const uint32_t rows = a.inter + min(8 * RT, (t1 - t) * 8);      // to the end of the step's up rows
      return PackedRows{w + (int64_t)t * 8 * ldw, c + (int64_t)t * 8 * lds, rows * ldw, rows * lds};
    };
    auto done = [&](int t, int, int l, auto sum) {
      if (l >= 32 || (l & 15) >= count) return;
      const f32x4 gate = sum(l), up = sum(l + 32);
      const float scale = wt[l & 15];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v = gate[q] * s13;
        const float h = v / (1.0f + expf(-v)) * (up[q] * s13) * scale;
        hi[q] = to_bf16(h);                          // two bf16 parts keep 16 significant bits of h
        lo[q] = to_bf16(h - bf16_to_f32(hi[q]));
      }
      uint16_t* row_h = a.h + (int64_t)(base + (l & 15)) * a.ldh;
      auto put = [&](int c, uint2 high, uint2 low) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(row_h + place_of(c));
        *reinterpret_cast<uint2*>(dst) = high;
        *reinterpret_cast<uint2*>(dst + a.lo) = low;
      };
      put(t * 8 + 4 * (l >> 4), make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16),
          make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16));
      if (t == tiles - 1)                            // the rest of the row's last quad
        for (int c = a.inter + 4 * (l >> 4); c < a.ldh; c += 8) put(c, make_uint2(0, 0), make_uint2(0, 0));
    };
    stream_tiles<kW4A16, 1, QW, TB>(t0, t1, a.hidden, row * ldw, row * lds, 8 * ldw, 8 * lds, tokens, part, rows_of,
                                    done);
  }
}

// 32 output channels for all tokens.  The (job, quad of its channels) steps are
// dealt to the waves, and a wave loads the next step's weights and h into the
// registers of the current one's as it uses them.  A product has a column for
// each token of the job, added to the token's sums in the wave's own part of
// LDS, step after step.  The waves are added at the end.
constexpr int kDownRows = 2;              // row tiles of 16

__global__ __launch_bounds__(64 * kStreamWaves, 2) void moe_down_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ __attribute__((aligned(16))) float sums[kStreamWaves * kMoeMaxTokens * 16 * kDownRows];   // [wave][tokens][32]
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int each = a.tokens * 16 * kDownRows;
  for (int i = threadIdx.x; i < kStreamWaves * each; i += 64 * kStreamWaves) sums[i] = 0.f;
  read_routing<64 * kStreamWaves>(r, a);
  const int row0 = blockIdx.x * 16 * kDownRows;
  const int quads = (a.inter + 511) >> 9;
  const int steps = __builtin_amdgcn_readfirstlane(r.jobs) * quads;
  const uint32_t ldw = (uint32_t)a.inter >> 1, lds = (uint32_t)a.inter >> 4;
  const uint32_t rows = min(16 * kDownRows, a.hidden - row0);
  float* mine = sums + wave * each;

  Quad<kW4A16> w[kDownRows];
  uint4 h[2][4][4];                       // high and low parts, [unit][8 channels]
  PackedRows next{};
  const uint8_t* next_h = nullptr;
  int next_q = 0;
  auto aim = [&](int i) {                 // at step i, or at nothing past the last one
    const bool there = i < steps;
    i = min(i, steps - 1);
    const int job = i / quads;
    next_q = i - job * quads;
    const int e = __builtin_amdgcn_readfirstlane(r.expert[job]);
    const int count = min(16, __popcll(tokens_of(r, e)) - r.first[job]);
    const int64_t row = (int64_t)e * a.hidden + row0;
    next = PackedRows{a.p2 + row * ldw, a.c2 + row * lds, there ? rows * ldw : 0, there ? rows * lds : 0};
    next_h = reinterpret_cast<const uint8_t*>(a.h) + (int64_t)(r.base[job] + min(r16, count - 1)) * a.ldh * 2 +
             next_q * 1024 + g * 16;
  };
  auto load_scales = [&](int t) { w[t].load_scales(next, (16 * t + r16) * lds, next_q, g, a.inter); };
  auto load_unit = [&](int u) {
#pragma unroll
    for (int t = 0; t < kDownRows; ++t) w[t].load_weights(u, next, (16 * t + r16) * ldw, next_q, g);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) h[p][u][j] = global_load16(next_h + (p ? a.lo : 0) + u * 256 + j * 64);
  };
  if (wave < steps) {
    aim(wave);
#pragma unroll
    for (int t = 0; t < kDownRows; ++t) load_scales(t);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_unit(u);
    for (int i = wave; i < steps; i += kStreamWaves) {
      const int job = i / quads;
      aim(i + kStreamWaves);
      u32x2 ws[kDownRows];
      f32x4 acc[kDownRows][2];
#pragma unroll
      for (int t = 0; t < kDownRows; ++t) {
        ws[t] = w[t].scales(g);
        load_scales(t);
        acc[t][0] = acc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int t = 0; t < kDownRows; ++t) {
          float s0, s1;
          Quad<kW4A16>::codes(ws[t], u, s0, s1);
          const uint32_t wv[4] = {w[t].w[u].x, w[t].w[u].y, w[t].w[u].z, w[t].w[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = fp4x8_bf16(wv[j], j < 2 ? s0 : s1);
            acc[t][0] = mfma_bf16(v, h[0][u][j], acc[t][0]);
            acc[t][1] = mfma_bf16(v, h[1][u][j], acc[t][1]);
          }
        }
        load_unit(u);
        __builtin_amdgcn_sched_barrier(0);         // the loads go out here, not where their values are near
      }
      const int e = __builtin_amdgcn_readfirstlane(r.expert[job]), first = r.first[job];
      const uint64_t mask = tokens_of(r, e);
      const int tok = token_of_column(mask, first);
      if (r16 < min(16, __popcll(mask) - first)) {
#pragma unroll
        for (int t = 0; t < kDownRows; ++t)
          *reinterpret_cast<f32x4*>(mine + (tok * kDownRows + t) * 16 + 4 * g) += acc[t][0] + acc[t][1];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < each; i += 64 * kStreamWaves) {
    const int t = i / (16 * kDownRows), o = row0 + i % (16 * kDownRows);
    float v = sums[i];
#pragma unroll
    for (int z = 1; z < kStreamWaves; ++z) v += sums[z * each + i];
    if (o < a.hidden) a.y[t * a.ldy + o] = to_bf16(v);
  }
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

static int64_t moe_ldh(int64_t inter) { return (inter + 511) / 512 * 512; }

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t inter) {
  return 2 * ((size_t)(tokens * top_k) * (size_t)moe_ldh(inter) * 2);
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
  a.ldh = moe_ldh(inter);
  a.lo = (int64_t)(moe_workspace_bytes(tokens, top_k, inter) / 2);
  a.tokens = (int)tokens;
  a.hidden = (int)hidden;
  a.inter = (int)inter;
  a.experts = (int)experts;
  a.top_k = top_k;
  const int64_t pairs = tokens * top_k;
  const int64_t most = pairs < experts ? pairs : experts;        // experts reached, at least one job each
  const int64_t want = most * (inter / 8);
  const unsigned grid = (unsigned)(want < kCus ? want : kCus);
  if (hidden <= 512 * kStreamWaves) moe_up_kernel<1><<<grid, 64 * kStreamWaves, 0, s>>>(a);
  else moe_up_kernel<2><<<grid, 64 * kStreamWaves, 0, s>>>(a);
  const int st = launch_status("moe_up_kernel");
  if (st) return st;
  const unsigned rows = (unsigned)((hidden + 16 * kDownRows - 1) / (16 * kDownRows));
  moe_down_kernel<<<rows, 64 * kStreamWaves, 0, s>>>(a);
  return launch_status("moe_down_kernel");
}

}  // namespace nvfp4
