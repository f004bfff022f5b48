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
//
// 8 of 128 experts of 7168 x 2048, with the router's launch: 1 token 61 us (198 MB;
// 55 with the same inputs again, whose weights the MALL keeps), 16 tokens 425 to
// 460 as they reach 80 to 87 experts (2.0 to 2.2 GB, 4.6 TB/s), 61 tokens 745 to
// 770 (3.1 GB, 4.1 TB/s).  The first product takes 60% of it and waits for memory
// (it issues something 0.73 of the time); the second issues 0.79 (16 tokens) and
// 0.84 (61) of the time, for it multiplies three parts of h and reads the weights
// of an expert once for every four of its tokens.
#include "common.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kMaxJobs = kMoeMaxTokens * kMoeMaxTopK;
// h is a float32 value, kept as the sum of three bf16 ones, which hold its 24
// bits; bf16 matrix instructions multiply them one after another.  Two parts, 16
// bits, moved 0.25% of 437248 outputs off the rounded exact value, three move
// 0.025% (float32 products in another order 0.1%); the layer took 411 and 696 us
// for 16 and 61 tokens with two, takes 428 and 755 with three.
constexpr int kParts = 3;

struct MoeArgs {
  const uint8_t* x;               // bf16 rows
  int64_t ldx;                    // in bytes
  const int32_t* ids;
  const float* weights;
  const uint8_t *p13, *c13, *p2, *c2;
  const float *s13, *s2;
  uint16_t* y;
  int64_t ldy;
  uint16_t* h;                    // [parts][groups of four tokens][ldh][4] bf16 (see place_of)
  int64_t ldh;                    // inter rounded up to whole quads, zero past inter
  int64_t part;                   // bytes from a part of a value to the next one
  int tokens, hidden, inter, experts, top_k;
};

// A job is a chosen expert with up to JOB of its tokens.
struct Routing {
  uint32_t mask[kMoeMaxExperts][2];       // tokens of an expert
  uint16_t expert[kMaxJobs];              // by job: its expert, experts in ascending order,
  uint16_t base[kMaxJobs];                // its first group of four tokens (of h),
  uint8_t first[kMaxJobs];                // its first token's place among the expert's
  uint32_t part[16];                      // per wave: jobs and groups (upper half)
  int jobs;
};

__device__ __forceinline__ uint64_t tokens_of(const Routing& r, int e) {
  return (uint64_t)r.mask[e][1] << 32 | r.mask[e][0];
}

// Fill r from the ids (all threads, a whole number of waves; syncs).
template <int JOB>
__device__ __forceinline__ void read_routing(Routing& r, const MoeArgs& a) {
  const int threads = blockDim.x, per = (kMoeMaxExperts + threads - 1) / threads;
  const int n = a.tokens * a.top_k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e0 = tid < n ? a.ids[tid] : -1;                // on its way while the masks are cleared
  for (int i = tid; i < 2 * a.experts; i += threads) (&r.mask[0][0])[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += threads) {
    const int e = i == tid ? e0 : a.ids[i], t = i / a.top_k;
    if (e >= 0 && e < a.experts) atomicOr(&r.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // prefix sums over the experts, `per` of them a thread: jobs in the lower half
  // of the word, groups of four tokens (at most 1024) in the upper
  auto own = [&](int i) {
    const int e = tid * per + i;
    const uint32_t c = e < a.experts ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0;
    return (c + JOB - 1) / JOB | (c + 3) / 4 << 16;
  };
  uint32_t sum = 0;
  for (int i = 0; i < per; ++i) sum += own(i);
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
  for (int w = 0; w < threads / 64; ++w) {
    if (w < wave) before += r.part[w];
    all += r.part[w];
  }
  for (int i = 0; i < per; ++i) {
    const uint32_t mine = own(i);
    for (int q = 0; q < (int)(mine & 0xFFFF); ++q) {
      const int job = (before & 0xFFFF) + q;
      r.expert[job] = (uint16_t)(tid * per + i);
      r.base[job] = (uint16_t)((before >> 16) + JOB / 4 * q);
      r.first[job] = (uint8_t)(JOB * q);
    }
    before += mine;
  }
  if (tid == 0) r.jobs = (int)(all & 0xFFFF);
  __syncthreads();
}

// The place-th set bit of a nonzero mask (the last one for places beyond); all
// lanes take part.
__device__ __forceinline__ int token_of_place(uint64_t mask, int place) {
  const int lane = threadIdx.x & 63;
  const int n = __popcll(mask);
  const int rank = __popcll(mask & ((1ull << lane) - 1));
  // lane t sends t to lane rank(t); lanes whose bit is clear send to a lane of
  // their own past the set bits
  const int to = (mask >> lane) & 1 ? rank : n + lane - rank;
  const int t = __builtin_amdgcn_ds_permute(to * 4, lane);
  return __shfl(t, min(place, n - 1));
}

// What a token gives an expert (all places that name it).
__device__ __forceinline__ float weight_of(const MoeArgs& a, int t, int e) {
  float w = 0.f;
  for (int s = 0; s < a.top_k; ++s)
    if (a.ids[t * a.top_k + s] == e) w += a.weights[t * a.top_k + s];
  return w;
}

// Where channel c of token j of a group of four is kept in the group's part of
// h: within each quad (512 channels) in the order in which the second launch's
// lanes read them, 16 bytes a lane: piece m (8 channels) of the 16 chunks of 32
// next to each other, the four tokens' pieces next to each other.
__device__ __forceinline__ int place_of(int c, int j) {
  return (c & ~511) << 2 | ((c >> 3) & 3) << 9 | ((c >> 5) & 15) << 5 | j << 3 | (c & 7);
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

// h of 4 NG tokens (tok: the lane's of each four) of a job, for row tiles
// t0 .. t1 - 1.  A tile's first two row groups are the gate rows of 8 channels,
// the others their up rows, so that one pass over the tokens serves both.
template <bool ODD, int NG>
__device__ __forceinline__ void up_rows(const MoeArgs& a, const QuadPlan& plan, int e, int base, int count, int first_tok,
                                        uint64_t mask, int t0, int t1, const float* wt, f32x4* part, uint8_t* stage) {
  constexpr int CH = 8;                              // channels of a tile
  const int wave = threadIdx.x >> 6, j = (threadIdx.x & 63) >> 4;
  const uint32_t ldw = (uint32_t)a.hidden >> 1, lds = (uint32_t)a.hidden >> 4;
  const uint8_t* w = a.p13 + (int64_t)e * 2 * a.inter * ldw;
  const uint8_t* c = a.c13 + (int64_t)e * 2 * a.inter * lds;
  const float s13 = a.s13[e];
  const uint32_t group_row[4] = {0, 4, (uint32_t)a.inter, (uint32_t)a.inter + 4};
  Chunk x[1][NG];
  auto rows_of = [&](int t) {
    const uint32_t rows = a.inter + CH;              // to the end of the tile's up rows
    return PackedRows{w + (int64_t)t * CH * ldw, c + (int64_t)t * CH * lds, rows * ldw, rows * lds};
  };
  auto load_tokens = [&](int q) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int tok = token_of_place(mask, first_tok + min(4 * n + j, count - 1));
      load_pieces(x[0][n], a.x + tok * a.ldx, q, a.hidden);
    }
  };
  auto take_tokens = [&]() {
#pragma unroll
    for (int n = 0; n < NG; ++n) pieces_to_chunk(x[0][n], stage + wave * 4096);
  };
  // done is called for the up rows by the lanes 8 after those of the gate rows
  auto done = [&](int t, int n, int q, int tj, f32x4 v) {
    f32x4 up;
#pragma unroll
    for (int z = 0; z < 4; ++z) up[z] = __shfl_down(v[z], 8);
    const int col = 4 * n + tj;
    if (q >= 2 || col >= count) return;
    const float scale = wt[col];
    uint32_t h[kParts][4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const float gate = v[z] * s13;
      split(gate / (1.0f + expf(-gate)) * (up[z] * s13) * scale, h[0][z], h[1][z], h[2][z]);
    }
    uint16_t* group_h = a.h + (int64_t)(base + col / 4) * a.ldh * 4;
    auto put = [&](int p, int ch, uint2 value) {
      *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(group_h + place_of(ch, col & 3)) + p * a.part) = value;
    };
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      put(p, t * CH + 4 * q, make_uint2(h[p][0] | h[p][1] << 16, h[p][2] | h[p][3] << 16));
      if ((t + 1) * CH == a.inter && q == 0)         // the rest of the row's last quad
        for (int ch = a.inter; ch < a.ldh; ch += 4) put(p, ch, make_uint2(0, 0));
    }
  };
  stream_rows<ODD, NG, 4>(t0, t1, a.hidden, plan, group_row, x, part, stage + wave * 4096, rows_of, load_tokens, take_tokens,
                           done);
}

// h of a run of (job, 8 channels) pieces of work, as many runs as there are
// workgroups.
template <bool ODD, int MW>
__global__ __launch_bounds__(64 * MW, 4) void moe_up_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ f32x4 part[MW * 4 * 2 * 16];
  __shared__ __attribute__((aligned(16))) uint8_t stage[MW * 4096];
  __shared__ float wt[8];
  read_routing<8>(r, a);
  const int lane = threadIdx.x & 63;
  const QuadPlan plan = quad_plan<1>(a.hidden, kCuWaves);
  const int tiles = a.inter >> 3;
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(r.jobs) * tiles;
  const int64_t begin = total * blockIdx.x / gridDim.x;
  int left = __builtin_amdgcn_readfirstlane((int)(total * (blockIdx.x + 1) / gridDim.x - begin));
  int job = __builtin_amdgcn_readfirstlane((int)(begin / tiles));
  int t0 = __builtin_amdgcn_readfirstlane((int)(begin - (int64_t)job * tiles));
  for (; left > 0; ++job, t0 = 0) {                  // one job after another
    const int t1 = min(tiles, t0 + left);
    left -= t1 - t0;
    const int e = __builtin_amdgcn_readfirstlane(r.expert[job]), base = __builtin_amdgcn_readfirstlane(r.base[job]);
    const int first = __builtin_amdgcn_readfirstlane(r.first[job]);
    const uint64_t mask = tokens_of(r, e);
    const int count = __builtin_amdgcn_readfirstlane(min(8, __popcll(mask) - first));
    if (threadIdx.x < 64) {                          // (what reads wt comes after a barrier)
      const int tok = token_of_place(mask, first + lane);
      if (lane < 8) wt[lane] = weight_of(a, tok, e) * a.s2[e];
    }
    if (count <= 4) up_rows<ODD, 1>(a, plan, e, base, count, first, mask, t0, t1, wt, part, stage);
    else up_rows<ODD, 2>(a, plan, e, base, count, first, mask, t0, t1, wt, part, stage);
  }
}

// ROWS output channels for all tokens.  The (job, quad of its channels) steps, a
// job being up to four tokens of an expert, are dealt to the waves, and a wave
// loads the next step's weights and h as it uses the current one's.  A product
// has a column for each token of the job, added to the token's sums in the
// wave's own part of LDS, step after step.  The waves are added at the end.
// (12 waves: the same within 1%.)
constexpr int kDownWaves = 8;

template <bool ODD, int GROUPS>           // row groups of four
__global__ __launch_bounds__(64 * kDownWaves, 2) void moe_down_kernel(MoeArgs a) {
  constexpr int ROWS = 4 * GROUPS;
  __shared__ Routing r;
  __shared__ __attribute__((aligned(16))) float sums[kDownWaves * kMoeMaxTokens * ROWS];   // [wave][tokens][ROWS]
  __shared__ __attribute__((aligned(16))) uint8_t turn[kDownWaves][1024];          // weights change their order there
  const int lane = threadIdx.x & 63, j = lane & 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int each = a.tokens * ROWS;
  for (int i = threadIdx.x; i < kDownWaves * each; i += 64 * kDownWaves) sums[i] = 0.f;
  read_routing<4>(r, a);
  const int row0 = blockIdx.x * ROWS;
  const int quads = (a.inter + 511) >> 9;
  const int steps = __builtin_amdgcn_readfirstlane(r.jobs) * quads;
  const uint32_t ldw = (uint32_t)a.inter >> 1, lds = (uint32_t)a.inter >> 4;
  const uint32_t rows = min(ROWS, a.hidden - row0);
  float* mine = sums + wave * each;

  RowGroup w[GROUPS];
  Chunk h[kParts][1], h_next[kParts][1];
  PackedRows next{};
  const uint8_t* next_h = nullptr;
  int next_q = 0;
  auto aim = [&](int i) {                 // at step i, or at nothing past the last one
    const bool there = i < steps;
    i = min(i, steps - 1);
    const int job = i / quads;
    next_q = i - job * quads;
    const int e = __builtin_amdgcn_readfirstlane(r.expert[job]);
    const int64_t row = (int64_t)e * a.hidden + row0;
    next = uniform(PackedRows{a.p2 + row * ldw, a.c2 + row * lds, there ? rows * ldw : 0, there ? rows * lds : 0});
    // (a group's tokens past the last one hold anything: their columns are not added)
    next_h = reinterpret_cast<const uint8_t*>(a.h) + (int64_t)job * a.ldh * 8 + next_q * 4096 + lane * 16;
  };
  auto load_h = [&](Chunk (&d)[kParts][1]) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint4 v = global_load16(next_h + p * a.part + m * 1024);
        d[p][0][4 * m] = v.x;
        d[p][0][4 * m + 1] = v.y;
        d[p][0][4 * m + 2] = v.z;
        d[p][0][4 * m + 3] = v.w;
      }
  };
  auto load_w = [&](int q) { w[q].load(next, 4 * q, next_q, LaneAt<ODD>(lane >> 4, next_q, a.inter), a.inter); };
  auto step = [&](int i, const Chunk (&x)[kParts][1], Chunk (&x_next)[kParts][1]) {
    const int job = i / quads;
    aim(i + kDownWaves);
    load_h(x_next);
    f32x4 acc[8][1];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      const RowGroup r = w[q].arranged(turn[wave]);
      load_w(q);
      __builtin_amdgcn_sched_barrier(0);             // the load goes out here, not where its value is near
      multiply_group<1, kParts>(r, x, acc[q]);
    }
    const int e = __builtin_amdgcn_readfirstlane(r.expert[job]), first = r.first[job];
    const uint64_t mask = tokens_of(r, e);
    const int tok = token_of_place(mask, first + j);
    const f32x4 v0 = sum_chunks_rest(sum_chunks_pair(acc[0][0], acc[2][0]), sum_chunks_pair(acc[1][0], acc[3][0]));
    f32x4 v1;
    if constexpr (GROUPS > 4)
      v1 = sum_chunks_rest(sum_chunks_pair(acc[4][0], acc[6][0]), sum_chunks_pair(acc[5][0], acc[7][0]));
    if ((lane & 12) == 0 && j < __popcll(mask) - first) {
      f32x4* dst = reinterpret_cast<f32x4*>(mine + tok * ROWS) + (lane >> 4);
      dst[0] += v0;
      if constexpr (GROUPS > 4)
        if (4 + (lane >> 4) < GROUPS) dst[4] += v1;
    }
  };
  if (wave < steps) {
    aim(wave);
    load_h(h);
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) load_w(q);
    for (int i = wave; i < steps; i += 2 * kDownWaves) {
      step(i, h, h_next);
      if (i + kDownWaves < steps) step(i + kDownWaves, h_next, h);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < each; i += 64 * kDownWaves) {
    const int t = i / ROWS, o = row0 + i % ROWS;
    float v = sums[i];
#pragma unroll
    for (int z = 1; z < kDownWaves; ++z) v += sums[z * each + i];
    if (o < a.hidden) a.y[t * a.ldy + o] = to_bf16(v);
  }
}

template <bool ODD>
void launch_up(const MoeArgs& a, unsigned grid, int waves, hipStream_t s) {
  if (waves <= 4) moe_up_kernel<ODD, 4><<<grid, 64 * waves, 0, s>>>(a);
  else if (waves <= 8) moe_up_kernel<ODD, 8><<<grid, 64 * waves, 0, s>>>(a);
  else moe_up_kernel<ODD, 16><<<grid, 64 * waves, 0, s>>>(a);
}

// Output channels of a workgroup: those with which the busiest CU has the
// fewest to do, among 16 to 32 (more of them read h less often).
template <bool ODD>
int launch_down(const MoeArgs& a, hipStream_t s) {
  int groups = 8, least = 0;
  for (int g = 8; g >= 4; --g) {
    const int n = (a.hidden + 4 * g - 1) / (4 * g), busiest = (n + kCus - 1) / kCus * g;
    if (g == 8 || busiest < least) {
      least = busiest;
      groups = g;
    }
  }
  const unsigned grid = (unsigned)((a.hidden + 4 * groups - 1) / (4 * groups));
  switch (groups) {
    case 4: moe_down_kernel<ODD, 4><<<grid, 64 * kDownWaves, 0, s>>>(a); break;
    case 5: moe_down_kernel<ODD, 5><<<grid, 64 * kDownWaves, 0, s>>>(a); break;
    case 6: moe_down_kernel<ODD, 6><<<grid, 64 * kDownWaves, 0, s>>>(a); break;
    case 7: moe_down_kernel<ODD, 7><<<grid, 64 * kDownWaves, 0, s>>>(a); break;
    default: moe_down_kernel<ODD, 8><<<grid, 64 * kDownWaves, 0, s>>>(a); break;
  }
  return launch_status("moe_down_kernel");
}

// + N lanes around a row of 16
template <int N>
__device__ __forceinline__ float max_ror(float v) {
  return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x120 + N, 0xF, 0xF, true)));
}
// The largest value of a wave, in all lanes.
__device__ __forceinline__ float wave_max(float v) {
  v = max_ror<1>(max_ror<2>(max_ror<4>(max_ror<8>(v))));
  uint32_t a = __float_as_uint(v), b = a;
  swap16(a, b);
  v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  a = b = __float_as_uint(v);
  swap32(a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

// One wave per token.  Lane l holds the logits of experts l, l + 64, ...;
// each of the top_k rounds takes the wave's largest remaining one, the lowest
// expert that has it.  The rounds follow one another, so what counts is their
// length: the maximum by lane permutes and its place by votes, 5.1 us for 16
// tokens and 8 of 128 experts; shuffles of value and place took 6.5.  A launch
// has fewer than 2^32 threads, so that many tokens go round by round.
constexpr unsigned kRouteGrid = 1 << 22;
template <int PER>
__global__ __launch_bounds__(256) void moe_route_kernel(const float* __restrict__ logits, int64_t tokens, int experts,
                                                        int64_t ldl, int top_k, int normalize,
                                                        int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tokens; t += (int64_t)gridDim.x * 4) {
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
#pragma unroll
      for (int i = 1; i < PER; ++i) bv = fmaxf(bv, v[i]);
      bv = wave_max(bv);
      int bi = 0;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) {
        const uint64_t has = __ballot(v[i] == bv);
        if (has) bi = 64 * i + __builtin_ctzll(has);
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
}

}  // namespace

static int64_t moe_ldh(int64_t inter) { return (inter + 511) / 512 * 512; }

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t inter) {
  // groups of four tokens: as many as pairs where no two tokens share an expert
  return kParts * ((size_t)(tokens * top_k) * 4 * (size_t)moe_ldh(inter) * 2);
}

int launch_moe_route(const float* logits, int64_t tokens, int64_t experts, int64_t ldl, int top_k, int normalize,
                     int32_t* ids, float* weights, hipStream_t s) {
  const int64_t want = (tokens + 3) / 4;
  const unsigned grid = want < kRouteGrid ? (unsigned)want : kRouteGrid;
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
  a.part = (int64_t)(moe_workspace_bytes(tokens, top_k, inter) / kParts);
  a.tokens = (int)tokens;
  a.hidden = (int)hidden;
  a.inter = (int)inter;
  a.experts = (int)experts;
  a.top_k = top_k;
  const int64_t pairs = tokens * top_k;
  const int64_t most = pairs < experts ? pairs : experts;        // experts reached, at least one job each
  const int waves = quad_plan<1>(hidden, kCuWaves).waves;
  const int64_t want = most * (inter / 8), all = kCus * (kCuWaves / waves);
  const unsigned grid = (unsigned)(want < all ? want : all);
  if (hidden % 32 == 0) launch_up<false>(a, grid, waves, s);
  else launch_up<true>(a, grid, waves, s);
  const int st = launch_status("moe_up_kernel");
  if (st) return st;
  return inter % 32 == 0 ? launch_down<false>(a, s) : launch_down<true>(a, s);
}

}  // namespace nvfp4
