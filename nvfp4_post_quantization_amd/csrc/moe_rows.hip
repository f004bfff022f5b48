// Tokens sorted by expert and back.  A choice is a token and one of its top_k
// places; the sorted rows are the choices whose id names an expert, by expert,
// then by choice.
//
//   sort      order[row] = choice, place[choice] = row, offsets[expert]
//   dispatch  xs[place[t][s]] = x[t]
//   combine   y[t] = sum over s of w[t][s] ys[place[t][s]], s ascending
//   gradient  dys[place[t][s]] = w[t][s] dy[t],  dw[t][s] = <dy[t], ys[place[t][s]]>;
//             that of dispatch is combine without weights
//
// Rows move by token, not by row: a token is read (written) once and its top_k
// rows are written (read), so that every byte crosses memory once.
#include <type_traits>

#include "layer.hpp"
#include "product_device.hpp"

namespace nvfp4 {

namespace {

// ---- sort --------------------------------------------------------------------
//
// A counting sort.  The choices are cut into as many chunks as workgroups, a
// chunk into 16 runs, one a wave.  First launch: a count per chunk and expert.
// Second: every workgroup adds up the counts (of all chunks for the experts'
// first rows, of those before its own for its place in them), counts its runs,
// and walks them 64 choices at a time; votes over the bits of the ids find the
// lanes with the same expert, whose order gives the rows.  Counts are whole
// numbers, so the result does not depend on who adds first.  One chunk needs no
// first launch.  Bound by latency, not by its bytes: 61 x 8 choices of 128 experts 4
// us, 65536 x 8 12 us (of 6 MB, which cross memory in 1.2), of which a trace gives the
// first launch 4 to 5 and the second 10.
constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
// Choices of a workgroup, at least, where there are several: 1024, and 4 an expert, for
// every workgroup adds up all counts (1023 x 8 of 128 experts 7.6 us, 10.0 with 4096;
// 65536 x 8 of 1024 experts 22 us with 4096, 30 with 2048).
constexpr int kSortChunk = 1024, kSortChunkPerExpert = 4;
constexpr int kSortAlone = 4096;         // up to this many one workgroup does it (4096 choices 7.2 us; 5600 in two launches 7.1)
constexpr int kSortGroups = 256;

struct SortArgs {
  const int32_t* ids;
  int32_t *order, *place, *offsets;
  uint32_t* counts;                      // [groups][experts] where groups > 1
  int64_t n;
  int experts, groups;
  BandList list;
};

__device__ __forceinline__ int64_t chunk_begin(const SortArgs& a, int g) { return a.n * g / a.groups; }

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t count[kMoeMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t end = chunk_begin(a, blockIdx.x + 1);
  for (int64_t i = chunk_begin(a, blockIdx.x) + threadIdx.x; i < end; i += kSortThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// The sum of v over the threads before this one; all of it in `all`.  (part: one
// word a wave; syncs.)
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t scan = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(scan, d);
    if (lane >= d) scan += o;
  }
  __syncthreads();
  if (lane == 63) part[wave] = scan;
  __syncthreads();
  uint32_t before = scan - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  return before;
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ uint32_t next[kSortWaves * kMoeMaxExperts];         // [wave][expert]: counts, then rows
  __shared__ uint32_t sum[2][kMoeMaxExperts];                    // all chunks', and those before this one
  __shared__ uint32_t part[kSortWaves], last[kSortWaves][kBandRows / kBandUnit];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts, g = blockIdx.x;
  for (int i = tid; i < kSortWaves * E; i += kSortThreads) next[i] = 0;
  if (tid < E) sum[0][tid] = sum[1][tid] = 0;
  __syncthreads();
  const int64_t begin = chunk_begin(a, g), end = chunk_begin(a, g + 1);
  const int64_t run = ((end - begin + kSortThreads - 1) / kSortThreads) * 64;
  const int64_t r0 = begin + wave * run, r1 = r0 + run < end ? r0 + run : end;
  uint32_t* mine = next + wave * E;
  for (int64_t i = r0 + lane; i < r1; i += 64) {
    const int e = a.ids[i];
    if (e >= 0 && e < E) atomicAdd(&mine[e], 1u);
  }
  if (a.groups > 1) {
    // thread tid adds up expert tid % span, every (1024 / span)-th chunk
    int span = 1;
    while (span < E) span *= 2;
    const int e = tid & (span - 1), step = kSortThreads / span;
    if (e < E) {
      uint32_t all = 0, before = 0;
#pragma unroll 16
      for (int c = tid / span; c < a.groups; c += step) {
        const uint32_t v = a.counts[(int64_t)c * E + e];
        all += v;
        if (c < g) before += v;
      }
      atomicAdd(&sum[0][e], all);
      atomicAdd(&sum[1][e], before);
    }
  }
  __syncthreads();
  uint32_t total = 0, rows;
  if (tid < E) {
    if (a.groups > 1) total = sum[0][tid];
    else
      for (int w = 0; w < kSortWaves; ++w) total += next[w * E + tid];
  }
  const uint32_t first = block_scan(total, part, rows);
  if (tid < E) {
    if (g == 0) a.offsets[tid] = (int32_t)first;
    uint32_t row = first + sum[1][tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = next[w * E + tid];
      next[w * E + tid] = row;
      row += c;
    }
  }
  if (g == 0 && tid == 0) a.offsets[E] = (int32_t)rows;
  if (a.list.bands && g == 0) {                                  // (the same way for all threads)
    // whole bands first, then the experts' last ones, those of most units first
    constexpr uint32_t most = kBandRows, classes = kBandRows / kBandUnit;
    const uint32_t whole = total / most, rest = total % most, units = (rest + kBandUnit - 1) / kBandUnit;
    uint64_t same = 0;
#pragma unroll
    for (uint32_t u = 1; u <= classes; ++u) {
      const uint64_t of = __ballot(units == u);
      if (units == u) same = of;
      if (lane == 0) last[wave][u - 1] = __popcll(of);
    }
    uint32_t count;
    uint32_t at = block_scan(whole, part, count);                // (syncs)
    for (uint32_t i = 0; i < whole; ++i) a.list.bands[at + i] = ExpertBand{tid, (int)(first + i * most), (int)most, 0};
    at = count + __popcll(same & ((1ull << lane) - 1));
#pragma unroll 1
    for (int w = 0; w * 64 < E; ++w)                             // (a thread an expert)
#pragma unroll
      for (uint32_t u = 1; u <= classes; ++u) {
        const uint32_t c = last[w][u - 1];
        if (u > units || (u == units && w < wave)) at += c;
        count += c;
      }
    if (units) a.list.bands[at] = ExpertBand{tid, (int)(first + whole * most), (int)rest, 0};
    if (tid == 0) *a.list.count = (int)count;
  }
  __syncthreads();
  // what a step needs from memory is on its way during the one before
  struct Choice { int e; float weight, scale; };
  const auto load = [&](int64_t c) {
    Choice v{-1, 0.f, 0.f};
    if (c < r1) {
      v.e = a.ids[c];
      if (a.list.bands) {
        v.weight = a.list.weights[c];
        v.scale = a.list.scales[(uint32_t)c / (uint32_t)a.list.top_k];        // (a pass: 2^17)
      }
    }
    return v;
  };
  Choice ahead = load(r0 + lane);
  for (int64_t i = r0; i < r1; i += 64) {
    const int64_t c = i + lane;
    const Choice v = ahead;
    ahead = load(c + 64);
    const bool in = v.e >= 0 && v.e < E;
    uint64_t same = __ballot(in);
    for (int b = 0; (1 << b) < E; ++b) {
      const uint64_t set = __ballot(v.e >> b & 1);
      same &= v.e >> b & 1 ? set : ~set;
    }
    if (in) {
      const uint32_t row = mine[v.e] + __popcll(same & ((1ull << lane) - 1));
      if (same >> lane == 1) mine[v.e] = row + 1;                // the last of them
      a.order[row] = (int32_t)c;
      a.place[c] = (int32_t)row;
      if (a.list.bands) {
        a.list.row_weight[row] = v.weight;
        a.list.row_scale[row] = v.scale;
      }
    } else if (c < r1) {
      a.place[c] = -1;
    }
  }
  for (int64_t r = rows + (int64_t)g * kSortThreads + tid; r < a.n; r += (int64_t)a.groups * kSortThreads) a.order[r] = -1;
}

// ---- rows --------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr unsigned kRowGrid = 1 << 22;   // workgroups at most; more units go round by round

// A unit: a token and up to `threads` neighbouring pieces of its row, a thread each.
struct Units {
  int64_t count, chunks;                 // of all tokens, of one
  int threads;
};
// Threads of a unit: the most that leave fewer than an eighth of them without a
// piece (7168 bf16 columns, 896 pieces: 128, not 256).
Units units_of(int64_t tokens, int64_t pieces) {
  Units u{0, 0, kRowThreads};
  for (; u.threads > 1; u.threads /= 2) {
    const int64_t given = (pieces + u.threads - 1) / u.threads * u.threads;
    if ((given - pieces) * 8 <= given) break;
  }
  u.chunks = (pieces + u.threads - 1) / u.threads;
  u.count = tokens * u.chunks;
  return u;
}
unsigned unit_grid(const Units& u) {
  const int64_t per = kRowThreads / u.threads, want = (u.count + per - 1) / per;
  return want < kRowGrid ? (unsigned)want : kRowGrid;
}
// f(token, piece) for the thread's units
template <typename F>
__device__ __forceinline__ void each_unit(const Units& u, int64_t pieces, F f) {
  const int per = kRowThreads / u.threads, sub = threadIdx.x / u.threads, l = threadIdx.x % u.threads;
  for (int64_t i = (int64_t)blockIdx.x * per + sub; i < u.count; i += (int64_t)gridDim.x * per) {
    const int64_t t = u.count >> 32 ? i / u.chunks : (int64_t)((uint32_t)i / (uint32_t)u.chunks);
    const int64_t piece = (i - t * u.chunks) * u.threads + l;
    if (piece < pieces) f(t, piece);
  }
}

// A token's rows among the n = tokens * top_k sorted ones; -1: none.
template <int K>
__device__ __forceinline__ void rows_of_token(const int32_t* place, int64_t t, int top_k, int64_t n, int64_t (&row)[K]) {
#pragma unroll
  for (int s = 0; s < K; ++s) {
    const int64_t r = s < top_k ? place[t * top_k + s] : -1;
    row[s] = r < n ? r : -1;
  }
}

// Rows that are more than the 256 MB MALL can hand on are kept out of it.  8192x8x7168
// (940 MB), call after call: dispatch 216 us without that, 193 so, combine 205 and 197,
// one after the other in turn 439 and 391.  (After 768 MB of other data were written:
// dispatch 222 and 253, combine 259 and 212.)  8192x8x2048 (268 MB) took 51 and 54, and
// 51 and 58.
constexpr int64_t kPastMall = INT64_C(1) << 29;
typedef uint32_t Word4 __attribute__((ext_vector_type(4)));

// The token's piece is read once and written to its rows.
template <typename V, int K, bool PAST>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const uint8_t* x, Units u, int64_t pieces, int64_t ldx,
                                                               const int32_t* place, int64_t n, int top_k, uint8_t* xs,
                                                               int64_t ldxs) {
  each_unit(u, pieces, [&](int64_t t, int64_t i) {
    const V v = reinterpret_cast<const V*>(x + t * ldx)[i];
    int64_t row[K];
    rows_of_token(place, t, top_k, n, row);
#pragma unroll
    for (int s = 0; s < K; ++s)
      if (row[s] >= 0) {
        V* const to = reinterpret_cast<V*>(xs + row[s] * ldxs) + i;
        if constexpr (PAST) __builtin_nontemporal_store(v, to);
        else *to = v;
      }
  });
}

// Rows that are added up, 8 columns a piece: bf16, or fp16 with a power of two for
// every 32 columns (biased: value = fp16 * 2^(e - kHalfBias)).
template <bool PAST>
struct Bf16Rows {
  const uint16_t* p;
  int64_t ld;
  struct Piece { Word4 v; };
  __device__ __forceinline__ Piece load(int64_t row, int64_t i) const {
    const Word4* const at = reinterpret_cast<const Word4*>(p + row * ld + i * 8);
    return Piece{PAST ? __builtin_nontemporal_load(at) : *at};
  }
  static __device__ __forceinline__ void add(float (&acc)[8], const Piece& x, float w) {
    const uint32_t q[4] = {x.v.x, x.v.y, x.v.z, x.v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[2 * e] = __builtin_fmaf(w, __uint_as_float(q[e] << 16), acc[2 * e]);
      acc[2 * e + 1] = __builtin_fmaf(w, __uint_as_float(q[e] & 0xFFFF0000u), acc[2 * e + 1]);
    }
  }
};
struct HalfRows {
  const uint16_t* p;
  const uint8_t* e;
  int64_t ld, lde;
  struct Piece { uint4 v; int e; };
  __device__ __forceinline__ Piece load(int64_t row, int64_t i) const {
    return Piece{*reinterpret_cast<const uint4*>(p + row * ld + i * 8), e[row * lde + (i >> 2)]};
  }
  static __device__ __forceinline__ void add(float (&acc)[8], const Piece& x, float w) {
    const float s = __builtin_amdgcn_ldexpf(w, x.e - kHalfBias);
    const f16x8 h = __builtin_bit_cast(f16x8, x.v);
#pragma unroll
    for (int z = 0; z < 8; ++z) acc[z] = __builtin_fmaf(s, (float)h[z], acc[z]);
  }
};

__device__ __forceinline__ uint4 pack_bf16(const float (&v)[8]) {
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = to_bf16(v[2 * e]) | (uint32_t)to_bf16(v[2 * e + 1]) << 16;
  return make_uint4(p[0], p[1], p[2], p[3]);
}

// Sums in fp32, one rounding.  All rows of a token are on their way before the
// first is added.  Bound by memory: 8192 x 8 rows of 7168, 1.06 GB in 197 us.
template <typename Rows, int K>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(Rows ys, Units u, int64_t pieces, const int32_t* place,
                                                              const float* weights, int64_t n, int top_k, uint16_t* y,
                                                              int64_t ldy) {
  each_unit(u, pieces, [&](int64_t t, int64_t i) {
    int64_t row[K];
    float w[K];
    typename Rows::Piece v[K];
    rows_of_token(place, t, top_k, n, row);
#pragma unroll
    for (int s = 0; s < K; ++s) {
      w[s] = weights && s < top_k ? weights[t * top_k + s] : 1.0f;
      v[s] = ys.load(row[s] < 0 ? 0 : row[s], i);    // (there is a row 0; not added where it is not meant)
    }
    float acc[8] = {};
#pragma unroll
    for (int s = 0; s < K; ++s)
      if (row[s] >= 0) Rows::add(acc, v[s], w[s]);
    *reinterpret_cast<uint4*>(y + t * ldy + i * 8) = pack_bf16(acc);
  });
}

// f(K) for the least K of 1, 2, 4, 8, 16 that holds top_k
template <typename F>
int with_places(int top_k, F f) {
  if (top_k <= 1) return f(std::integral_constant<int, 1>{});
  if (top_k <= 2) return f(std::integral_constant<int, 2>{});
  if (top_k <= 4) return f(std::integral_constant<int, 4>{});
  if (top_k <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

// One token a workgroup (WAVES = 4) or, of short rows, a wave; K >= top_k sums of
// products, each a token's own, so that no two meet.  Bound by memory: 8192 x 8 rows
// of 7168, 2.0 GB in 430 us.
template <int K, int WAVES>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* ys,
                                                                   int64_t ldys, const int32_t* place,
                                                                   const float* weights, int64_t tokens, int top_k,
                                                                   int64_t pieces, uint16_t* dys, int64_t lddys,
                                                                   float* dweights) {
  __shared__ float part[4][K];
  constexpr int PER = 4 / WAVES, THREADS = 64 * WAVES;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = threadIdx.x % THREADS;
  const int64_t n = tokens * top_k;
  for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < tokens; t0 += (int64_t)gridDim.x * PER) {
    const int64_t t = t0 + wave / WAVES;
    float dot[K];
    int64_t row[K];
    float w[K];
    rows_of_token(place, min(t, tokens - 1), top_k, n, row);
#pragma unroll
    for (int s = 0; s < K; ++s) {
      dot[s] = 0.f;
      w[s] = s < top_k && t < tokens ? weights[t * top_k + s] : 0.f;
    }
    if (t < tokens)
      for (int64_t i = l; i < pieces; i += THREADS) {
        const uint4 d = *reinterpret_cast<const uint4*>(dy + t * lddy + i * 8);
        const uint32_t dp[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int s = 0; s < K; ++s) {
          if (row[s] < 0) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(ys + row[s] * ldys + i * 8);
          const uint32_t vp[4] = {v.x, v.y, v.z, v.w};
          float g[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(dp[e] << 16), hi = __uint_as_float(dp[e] & 0xFFFF0000u);
            dot[s] = __builtin_fmaf(lo, __uint_as_float(vp[e] << 16), dot[s]);
            dot[s] = __builtin_fmaf(hi, __uint_as_float(vp[e] & 0xFFFF0000u), dot[s]);
            g[2 * e] = w[s] * lo;
            g[2 * e + 1] = w[s] * hi;
          }
          *reinterpret_cast<uint4*>(dys + row[s] * lddys + i * 8) = pack_bf16(g);
        }
      }
#pragma unroll
    for (int s = 0; s < K; ++s) {
      if (s >= top_k) continue;
      float v = dot[s];
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
      if (lane == 0) part[wave][s] = v;
    }
    __syncthreads();
    if (l < top_k && t < tokens) {
      float v = part[wave][l];
#pragma unroll
      for (int z = 1; z < WAVES; ++z) v += part[z][l];
      dweights[t * top_k + l] = v;
    }
    __syncthreads();
  }
}

template <typename Rows>
int run_combine(const Rows& ys, const int32_t* place, const float* weights, int64_t tokens, int top_k, int64_t cols,
                uint16_t* y, int64_t ldy, hipStream_t s) {
  const int64_t pieces = cols / 8;
  const Units u = units_of(tokens, pieces);
  return with_places(top_k, [&](auto k) {
    combine_kernel<Rows, decltype(k)::value><<<unit_grid(u), kRowThreads, 0, s>>>(ys, u, pieces, place, weights,
                                                                                 tokens * top_k, top_k, y, ldy);
    return launch_status("combine_kernel");
  });
}

}  // namespace

static int sort_groups(int64_t n, int64_t experts) {
  if (n <= kSortAlone) return 1;
  const int64_t chunk = experts * kSortChunkPerExpert > kSortChunk ? experts * kSortChunkPerExpert : kSortChunk;
  const int64_t want = (n + chunk - 1) / chunk;
  return (int)(want < kSortGroups ? want : kSortGroups);
}

size_t moe_sort_workspace_bytes(int64_t choices, int64_t experts) {
  const int g = sort_groups(choices, experts);
  return g > 1 ? (size_t)g * experts * 4 : 0;
}

int launch_moe_sort(const int32_t* ids, int64_t choices, int64_t experts, int32_t* order, int32_t* place,
                    int32_t* offsets, void* workspace, const BandList& list, hipStream_t s) {
  const SortArgs a{ids, order, place, offsets, static_cast<uint32_t*>(workspace), choices, (int)experts,
                   sort_groups(choices, experts), list};
  if (a.groups > 1) {
    sort_count_kernel<<<a.groups, kSortThreads, 0, s>>>(a);
    const int st = launch_status("sort_count_kernel");
    if (st) return st;
  }
  sort_place_kernel<<<a.groups, kSortThreads, 0, s>>>(a);
  return launch_status("sort_place_kernel");
}

int launch_moe_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ldx, const int32_t* place, int top_k,
                        void* xs, int64_t ldxs, hipStream_t s) {
  const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs) | (uint64_t)(row_bytes | ldx | ldxs);
  const auto run = [&](auto v) {
    using V = decltype(v);
    const int64_t pieces = row_bytes / (int64_t)sizeof(V);
    const Units u = units_of(tokens, pieces);
    return with_places(top_k, [&](auto k) {
      const auto go = [&](auto kernel) {
        kernel<<<unit_grid(u), kRowThreads, 0, s>>>(static_cast<const uint8_t*>(x), u, pieces, ldx, place, tokens * top_k,
                                                    top_k, static_cast<uint8_t*>(xs), ldxs);
        return launch_status("dispatch_kernel");
      };
      if constexpr (sizeof(V) == 16)
        if (tokens * top_k > kPastMall / row_bytes) return go(dispatch_kernel<V, decltype(k)::value, true>);
      return go(dispatch_kernel<V, decltype(k)::value, false>);
    });
  };
  if (all % 16 == 0) return run(Word4{});
  if (all % 4 == 0) return run(uint32_t{});
  return run(uint8_t{});
}

int launch_moe_combine(const uint16_t* ys, int64_t ldys, const int32_t* place, const float* weights, int64_t tokens,
                       int top_k, int64_t cols, uint16_t* y, int64_t ldy, hipStream_t s) {
  if (tokens * top_k > kPastMall / (cols * 2))
    return run_combine(Bf16Rows<true>{ys, ldys}, place, weights, tokens, top_k, cols, y, ldy, s);
  return run_combine(Bf16Rows<false>{ys, ldys}, place, weights, tokens, top_k, cols, y, ldy, s);
}
int launch_moe_combine_half(const uint16_t* ys, const uint8_t* exponents, const int32_t* place, int64_t tokens, int top_k,
                            int64_t cols, uint16_t* y, int64_t ldy, hipStream_t s) {
  return run_combine(HalfRows{ys, exponents, cols, (cols + 31) / 32}, place, nullptr, tokens, top_k, cols, y, ldy, s);
}

int launch_moe_combine_grad(const uint16_t* dy, int64_t lddy, const uint16_t* ys, int64_t ldys, const int32_t* place,
                            const float* weights, int64_t tokens, int top_k, int64_t cols, uint16_t* dys, int64_t lddys,
                            float* dweights, hipStream_t s) {
  const int64_t pieces = cols / 8;
  return with_places(top_k, [&](auto k) {
    constexpr int K = decltype(k)::value;
    const int per = pieces > 64 ? 1 : 4;             // tokens of a workgroup
    const int64_t want = (tokens + per - 1) / per;
    const unsigned grid = want < kRowGrid ? (unsigned)want : kRowGrid;
    if (per == 1)
      combine_grad_kernel<K, 4><<<grid, kRowThreads, 0, s>>>(dy, lddy, ys, ldys, place, weights, tokens, top_k, pieces, dys,
                                                             lddys, dweights);
    else
      combine_grad_kernel<K, 1><<<grid, kRowThreads, 0, s>>>(dy, lddy, ys, ldys, place, weights, tokens, top_k, pieces, dys,
                                                             lddys, dweights);
    return launch_status("combine_grad_kernel");
  });
}

}  // namespace nvfp4
