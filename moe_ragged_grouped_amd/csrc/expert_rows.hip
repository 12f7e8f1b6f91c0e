// Tokens' rows to their experts and back, for gfx950: the stable sort of the
// choices by expert, the rows moved to their groups, the weighted sum of a
// token's rows, and its gradient.
//
// All of them move bytes. 2048 tokens of 8 choices, rows of 6144 bf16: spread 34 us
// for 226 MB (6.6 TB/s), combine 41 for 227 (5.5), gradient 90 for 428 (4.8, half
// of it writes). The sort moves little and waits: 64 x 8 choices 4 us, 16384 x 8 in
// two launches 8, each launch's start and its round trips to memory.

#include "gg_common.h"
#include "gg_fp8.h"
#include "gg_host.h"
#include "gg_ring.h"
#include "gg_schedule.h"
#include "grouped_gemm.h"

namespace gg {

// -------------------------------------------------------------------- sort
//
// A counting sort. A choice's row is its expert's first row plus the number of
// earlier choices of that expert; a wave counts the latter for 64 choices at
// once by comparing all of them bit by bit (a ballot per bit of the number).

typedef __attribute__((ext_vector_type(4))) int i32x4;

// The choices are split over workgroups, 1024 each while there are no more than
// 256 workgroups. Every workgroup needs the counts of all choices and of those
// before its own. Few choices it counts by itself, in the same launch; of more
// than 8192 one launch counts each part and the next places. Measured (us, 8
// choices a token by rank^-1.2 of 64 experts, launches in a graph; one launch /
// two): 2048 choices 5.2 / 6.8, 8192 7.7 / 7.3, 16384 10.2 / 7.5, 65536 25.7 /
// 7.9. A launch costs the host 3 us besides, which is why 8192 still takes one.
constexpr int kSortRecount = 8192;
constexpr int kSplitThreads = 512, kSplitWaves = kSplitThreads / kWave;
constexpr int kSplitChunk = 1024, kSplitMost = 256;  // choices a workgroup at least; workgroups at most

template <class I>
__device__ __forceinline__ int choice(const I *experts, long long i, long long n, int E) {
  if (i >= n) return E;
  const I e = experts[i];
  return e >= 0 && e < (I)E ? (int)e : E;
}

// The lanes whose v (0 <= v < 2^bits) is this lane's.
__device__ __forceinline__ unsigned long long same_lanes(int v, int bits) {
  unsigned long long m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = v >> b & 1;
    const unsigned long long ones = __ballot(one);
    m &= one ? ones : ~ones;
  }
  return m;
}
__device__ __forceinline__ int lanes_below(unsigned long long m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// This lane's place among the choices of its expert that the wave has seen,
// which `seen` (a wave's own counts, in LDS) holds up to here.
__device__ __forceinline__ int wave_place(int e, int E, int bits, int *seen) {
  const unsigned long long m = same_lanes(e, bits);
  const int below = lanes_below(m);
  int place = 0;
  if (e < E) {
    place = seen[e] + below;
    __builtin_amdgcn_wave_barrier();
    if (below == 0) seen[e] += __builtin_popcountll(m);
  }
  __builtin_amdgcn_wave_barrier();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  return place;
}

// Exclusive sums of one value a thread over the first E threads' values: the
// groups' offsets. All threads call it. Returns this thread's offset; total: all.
template <int WAVES>
__device__ __forceinline__ int group_starts(int mine, int *wave_sums, int &total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int incl = wave_scan(mine, INT32_MAX);
  if (lane == kWave - 1) wave_sums[wave] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wave) before += wave_sums[w];
    total += wave_sums[w];
  }
  return before + incl - mine;
}

struct SortParams {
  const void *experts;
  const float *w;
  int32_t *offsets, *rows, *pos;
  float *row_w;
  int32_t *counts;  // [workgroups][E up to a multiple of 4], of the split sort
  long long n;
  int k, E, bits, chunk;
};

// Choices of each expert in this workgroup's part.
template <class I>
__global__ __launch_bounds__(kSplitThreads) void sort_count_kernel(SortParams p) {
  extern __shared__ __attribute__((aligned(16))) int sort_lds[];
  for (int e = threadIdx.x; e < p.E; e += kSplitThreads) sort_lds[e] = 0;
  __syncthreads();
  const long long i0 = (long long)blockIdx.x * p.chunk, i1 = min(i0 + p.chunk, p.n);
  for (long long i = i0 + threadIdx.x; i < i1; i += kSplitThreads) {
    const int e = choice((const I *)p.experts, i, p.n, p.E);
    if (e < p.E) atomicAdd(&sort_lds[e], 1);
  }
  __syncthreads();
  const int pitch = (p.E + 3) / 4 * 4;
  for (int e = threadIdx.x; e < pitch; e += kSplitThreads)
    p.counts[(size_t)blockIdx.x * pitch + e] = e < p.E ? sort_lds[e] : 0;
}

template <class I, bool COUNTED>
__global__ __launch_bounds__(kSplitThreads) void sort_place_kernel(SortParams p) {
  extern __shared__ __attribute__((aligned(16))) int sort_lds[];
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, E = p.E;
  const int G = gridDim.x, b = blockIdx.x;
  int *const sums = sort_lds;          // [waves]
  int *const all = sums + kSplitWaves;  // [E] choices of an expert
  int *const base = all + E;           // [E] its first row, then the next one of this workgroup
  int *const seen = base + E;          // [waves][E]
  const I *const experts = (const I *)p.experts;
  const long long i0 = (long long)b * p.chunk, i1 = min(i0 + p.chunk, p.n);
  constexpr int kSteps = kSplitChunk / kSplitThreads;
  // this workgroup's first choices and weights, on their way during the counting
  int e[kSteps];
  float w[kSteps];
  auto fetch = [&](long long r0) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const long long i = r0 + (wave * kSteps + s) * kWave + lane;
      e[s] = choice(experts, i, i1, E);
      w[s] = p.w != nullptr && i < i1 ? p.w[i] : 0.0f;
    }
  };
  fetch(i0);
  for (int x = tid; x < 2 * E; x += kSplitThreads) all[x] = 0;
  __syncthreads();
  if constexpr (COUNTED) {
    // the workgroups' counts: a thread takes four experts of every so many
    // workgroups, with eight loads in flight
    const int quads = (E + 3) / 4, beside = kSplitThreads / quads, g0 = tid / quads, q = tid - g0 * quads;
    if (g0 < beside) {
      i32x4 sum = {0, 0, 0, 0}, before = {0, 0, 0, 0};
      for (int g = g0; g < G; g += 8 * beside) {
        i32x4 c[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          c[u] = i32x4{0, 0, 0, 0};
          if (g + u * beside < G) c[u] = ((const i32x4 *)p.counts)[(size_t)(g + u * beside) * quads + q];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          sum += c[u];
          if (g + u * beside < b) before += c[u];
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (4 * q + x < E) {
          if (sum[x] != 0) atomicAdd(&all[4 * q + x], sum[x]);
          if (before[x] != 0) atomicAdd(&base[4 * q + x], before[x]);
        }
    }
  } else {
    // all choices, those before this workgroup's apart, with eight loads in flight
    for (long long r0 = tid; r0 < p.n; r0 += 8 * kSplitThreads) {
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = choice(experts, r0 + u * kSplitThreads, p.n, E);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c[u] < E) atomicAdd((r0 + u * kSplitThreads < i0 ? base : all) + c[u], 1);
    }
    __syncthreads();
    for (int x = tid; x < E; x += kSplitThreads) all[x] += base[x];
  }
  __syncthreads();
  // two experts a thread (E <= 1024)
  const int e0 = 2 * tid, c0 = e0 < E ? all[e0] : 0, c1 = e0 + 1 < E ? all[e0 + 1] : 0;
  int total;
  const int start = group_starts<kSplitWaves>(c0 + c1, sums, total);
  if (e0 < E) base[e0] += start;
  if (e0 + 1 < E) base[e0 + 1] += start + c0;
  if (b == 0) {
    if (e0 < E) p.offsets[e0] = start;
    if (e0 + 1 < E) p.offsets[e0 + 1] = start + c0;
    if (tid == 0) p.offsets[E] = total;
  }
  for (long long r0 = i0; r0 < i1; r0 += kSplitChunk) {
    if (r0 != i0) fetch(r0);
    for (int i = tid; i < kSplitWaves * E; i += kSplitThreads) seen[i] = 0;
    __syncthreads();
    int place[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) place[s] = wave_place(e[s], E, p.bits, seen + wave * E);
    __syncthreads();
    for (int x = tid; x < E; x += kSplitThreads) {
      int at = base[x];
      for (int v = 0; v < kSplitWaves; ++v) {
        const int c = seen[v * E + x];
        seen[v * E + x] = at;
        at += c;
      }
      base[x] = at;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const long long i = r0 + (wave * kSteps + s) * kWave + lane;
      if (i >= i1) continue;
      const int at = e[s] < E ? seen[wave * E + e[s]] + place[s] : -1;
      p.pos[i] = at;
      if (at >= 0) {
        p.rows[at] = (int)i / p.k;
        if (p.w != nullptr) p.row_w[at] = w[s];
      }
    }
    __syncthreads();  // seen is cleared again
  }
  // rows that no choice has
  for (long long r = total + (long long)b * kSplitThreads + tid; r < p.n; r += (long long)G * kSplitThreads) {
    p.rows[r] = -1;
    if (p.w != nullptr) p.row_w[r] = 0.0f;
  }
}

// ------------------------------------------------------------------ spread
//
// A wave reads V KB of a token's row and writes them to each of its rows; the
// places of eight rows are read together. Block scales are moved by workgroups of
// their own, behind those of the rows: 256 tokens, a token to a lane, and four
// slices each, so that the rows of an expert, which lie in the order of their
// tokens, come out of one L2 as runs (scattered by the waves that move the rows,
// the 800,000 scales of 2048 x 8 rows of 6144 took 8 of 25 us).

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / kWave;
constexpr int kJ = 8;  // rows in flight

struct SpreadParams {
  const u32x4 *X;
  u32x4 *out;
  const char *scales;
  char *out_scales;
  const int32_t *pos;
  long long units;  // tokens x segments
  int T, k, pitch, segments, M;  // pitch in 16 bytes
  int scale_bytes, slices;
  unsigned row_groups, slice_groups;  // workgroups of the rows; of the scales of 256 tokens
};

// The places of choices j0 .. j0 + 7 of a token; -1 where there is no row.
__device__ __forceinline__ void places(int (&at)[kJ], const int32_t *pos, int k, int M, int t, int j0) {
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    at[j] = j0 + j < k ? scalar(pos[(size_t)t * k + j0 + j]) : -1;
    if (at[j] >= M) at[j] = -1;
  }
}

constexpr int kScaleSlices = 4;

template <class S>
__device__ __forceinline__ void spread_scales(const SpreadParams &p, unsigned group) {
  const int t = (int)(group / p.slice_groups) * kRowThreads + threadIdx.x;
  const int s0 = (int)(group % p.slice_groups) * kScaleSlices;
  if (t >= p.T || s0 >= p.slices) return;
  S x[kScaleSlices];
#pragma unroll
  for (int i = 0; i < kScaleSlices; ++i)
    if (s0 + i < p.slices) x[i] = ((const S *)p.scales)[(size_t)(s0 + i) * p.T + t];
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    int at[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) at[j] = j0 + j < p.k ? p.pos[(size_t)t * p.k + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (at[j] < 0 || at[j] >= p.M) continue;
#pragma unroll
      for (int i = 0; i < kScaleSlices; ++i)
        if (s0 + i < p.slices) ((S *)p.out_scales)[(size_t)(s0 + i) * p.M + at[j]] = x[i];
    }
  }
}

template <int V>
__global__ __launch_bounds__(kRowThreads) void spread_kernel(SpreadParams p) {
  if (blockIdx.x >= p.row_groups) {
    if (p.scale_bytes == 4) spread_scales<uint32_t>(p, blockIdx.x - p.row_groups);
    else spread_scales<u32x2>(p, blockIdx.x - p.row_groups);
    return;
  }
  const int lane = threadIdx.x % kWave, wave = scalar(threadIdx.x / kWave);
  const long long u = (long long)blockIdx.x * kRowWaves + wave;
  if (u >= p.units) return;
  const int t = (int)(u / p.segments), seg = (int)(u - (long long)t * p.segments);
  const int c0 = seg * V * kWave + lane;
  u32x4 v[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c0 + i * kWave < p.pitch) v[i] = p.X[(size_t)t * p.pitch + c0 + i * kWave];
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    int at[kJ];
    places(at, p.pos, p.k, p.M, t, j0);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (at[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + i * kWave < p.pitch) p.out[(size_t)at[j] * p.pitch + c0 + i * kWave] = v[i];
    }
  }
}

// Pieces a lane takes: as many as leave every CU eight waves, up to four.
static int spread_pieces(long long T, long long row_bytes) {
  int v = row_bytes > 2048 ? 4 : row_bytes > 1024 ? 2 : 1;
  while (v > 1 && T * ((row_bytes + v * 1024 - 1) / (v * 1024)) < 256 * 8) v /= 2;
  return v;
}

// ----------------------------------------------------------------- combine
//
// A lane takes eight columns of one token: its k rows are loaded together and
// summed in fp32 in the order of the choices, the weighted one by one fused
// multiply-add a term. Rounded once.

template <class Y>
struct Eight;  // eight values of a row in fp32
template <>
struct Eight<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *(const u32x4 *)p; }
  __device__ __forceinline__ float get(int i) const { return i % 2 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]); }
};
template <>
struct Eight<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *(const f32x4 *)p;
    b = *(const f32x4 *)(p + 4);
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};

__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8], bool stream) {
  const u32x2 a = pack_bf16(f32x4{v[0], v[1], v[2], v[3]}), b = pack_bf16(f32x4{v[4], v[5], v[6], v[7]});
  st_rows((u32x4 *)p, u32x4{a.x, a.y, b.x, b.y}, stream);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8], bool stream) {
  st_rows((f32x4 *)p, f32x4{v[0], v[1], v[2], v[3]}, stream);
  st_rows((f32x4 *)(p + 4), f32x4{v[4], v[5], v[6], v[7]}, stream);
}

struct CombineParams {
  const void *Y, *dO;
  const int32_t *pos;
  const float *w;
  void *out;   // the combined rows, or the gradient of Y
  float *dw;
  long long units;
  int T, k, N, M, segments;
  bool stream;  // the combined rows
};

template <class Y, class O>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(CombineParams p) {
  const int lane = threadIdx.x % kWave, wave = scalar(threadIdx.x / kWave);
  const long long u = (long long)blockIdx.x * kRowWaves + wave;
  if (u >= p.units) return;
  const int t = (int)(u / p.segments), seg = (int)(u - (long long)t * p.segments);
  const int n = (seg * kWave + lane) * 8;
  if (n >= p.N) return;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    Eight<Y> y[kJ];
    float w[kJ];
    bool in[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      in[j] = false;
      if (j0 + j < p.k) {
        const size_t c = (size_t)t * p.k + j0 + j;
        const int at = scalar(p.pos[c]);
        in[j] = at >= 0 && at < p.M;
        w[j] = p.w != nullptr ? p.w[c] : 1.0f;
        if (in[j]) y[j].load((const Y *)p.Y + (size_t)at * p.N + n);
      }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (in[j])
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], y[j].get(i), sum[i]);
  }
  store8((O *)p.out + (size_t)t * p.N + n, sum, p.stream);
}

// A workgroup a token: the gradient of its rows, and the scalar products with
// them that are the gradient of its weights.
template <class Y>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(CombineParams p) {
  __shared__ float sums[kRowWaves][kJ];
  const int t = blockIdx.x, tid = threadIdx.x;
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    int at[kJ];
    float w[kJ], dot[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      at[j] = -1;
      w[j] = dot[j] = 0.0f;
      if (j0 + j < p.k) {
        const size_t c = (size_t)t * p.k + j0 + j;
        at[j] = scalar(p.pos[c]);
        if (at[j] >= p.M) at[j] = -1;
        w[j] = p.w[c];
      }
    }
    for (int n = tid * 8; n < p.N; n += kRowThreads * 8) {
      Eight<Y> d, y[kJ];
      d.load((const Y *)p.dO + (size_t)t * p.N + n);
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (at[j] >= 0) y[j].load((const Y *)p.Y + (size_t)at[j] * p.N + n);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if (at[j] < 0) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[j] = __builtin_fmaf(d.get(i), y[j].get(i), dot[j]);
          o[i] = w[j] * d.get(i);
        }
        // (not as streaming data: the gradients of the products read it at once. 64 MB 34.6 us
        // so, 27.1 streamed, and with a reader behind 49.1 and 52.6; 192 MB 95.3 and 93.9, 143
        // and 151; into one buffer again and again 128 MB 53.8 and 64.0, 87 and 100)
        store8((Y *)p.out + (size_t)at[j] * p.N + n, o, false);
      }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const float s = sum_of_wave(dot[j]);
      if (tid % kWave == 0) sums[tid / kWave][j] = s;
    }
    __syncthreads();
    if (tid < kJ && j0 + tid < p.k) {
      float s = 0.0f;
#pragma unroll
      for (int w2 = 0; w2 < kRowWaves; ++w2) s += sums[w2][tid];
      p.dw[(size_t)t * p.k + j0 + tid] = s;
    }
    __syncthreads();  // sums is written again
  }
}

// Tokens and choices: T tokens of k choices each, M rows.
static gg_status_t check_choices(const void *pos, int64_t T, int k, int64_t M) {
  if (T < 0 || k < 1 || M < 0) return GG_ERR_INVALID_VALUE;
  if (T > INT32_MAX || M > INT32_MAX || T * k > INT32_MAX) return GG_ERR_UNSUPPORTED;
  if (T > 0 && pos == nullptr) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(pos, 4)) return GG_ERR_MISALIGNED;
  return GG_OK;
}

// Workgroups that the split sort takes, and choices of each.
static int split_sort(long long n, int *chunk) {
  long long c = (n + kSplitMost - 1) / kSplitMost;
  c = (c + kSplitChunk - 1) / kSplitChunk * kSplitChunk;
  if (c < kSplitChunk) c = kSplitChunk;
  *chunk = (int)c;
  return n > c ? (int)((n + c - 1) / c) : 1;  // (no choices: the offsets remain to be written)
}

template <class I>
static gg_status_t expert_sort(SortParams p, void *stream) {
  const int G = split_sort(p.n, &p.chunk);
  if (p.n <= kSortRecount)
    return launch(sort_place_kernel<I, false>, dim3((unsigned)G), kSplitThreads,
                  (kSplitWaves + 2 * p.E + kSplitWaves * p.E) * 4, stream, p);
  gg_status_t st = launch(sort_count_kernel<I>, dim3((unsigned)G), kSplitThreads, p.E * 4, stream, p);
  if (st != GG_OK) return st;
  return launch(sort_place_kernel<I, true>, dim3((unsigned)G), kSplitThreads,
                (kSplitWaves + 2 * p.E + kSplitWaves * p.E) * 4, stream, p);
}

static_assert((kSplitWaves + 2 * kMaxExperts + kSplitWaves * kMaxExperts) * 4 <= 64 * 1024, "LDS");
static_assert(2 * kSplitThreads >= kMaxExperts, "experts of a thread");

}  // namespace gg

using namespace gg;

extern "C" int64_t gg_expert_sort_workspace(int64_t choices, int32_t E) {
  if (choices <= kSortRecount || choices > INT32_MAX || E < 1) return 0;
  int chunk;
  return (int64_t)split_sort(choices, &chunk) * ((E + 3LL) / 4) * 16;
}

extern "C" gg_status_t gg_expert_sort(const void *experts, int32_t wide, const float *weights,
                                      int32_t *offsets, int32_t *rows, int32_t *pos, float *row_weights,
                                      void *workspace, int64_t T, int32_t k, int32_t E, void *stream) {
  gg_status_t st = check_choices(pos, T, k, 0);
  if (st != GG_OK) return st;
  if (E < 1 || offsets == nullptr || (weights == nullptr) != (row_weights == nullptr))
    return GG_ERR_INVALID_VALUE;
  if (E > kMaxExperts) return GG_ERR_UNSUPPORTED;
  const long long n = T * k, need = gg_expert_sort_workspace(n, E);
  if (n > 0 && (experts == nullptr || rows == nullptr)) return GG_ERR_INVALID_VALUE;
  if (need > 0 && workspace == nullptr) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(experts, wide ? 8 : 4) || !is_aligned(weights, 4) || !is_aligned(offsets, 4) ||
      !is_aligned(rows, 4) || !is_aligned(row_weights, 4) || !is_aligned(workspace, 16))
    return GG_ERR_MISALIGNED;
  const Span in = span(experts, n, wide ? 8 : 4, 1), w = span(weights, n, 4, 1),
             o = span(offsets, E + 1, 4, 1), r = span(rows, n, 4, 1), at = span(pos, n, 4, 1),
             rw = span(row_weights, n, 4, 1), ws = span(workspace, need, 1, 1);
  if (!apart(in, o, r, at, rw, ws) || !apart(w, o, r, at, rw, ws) || !apart(o, r, at, rw, ws) ||
      !apart(r, at, rw, ws) || !apart(at, rw, ws) || !apart(rw, ws))
    return GG_ERR_INVALID_VALUE;
  int bits = 0;
  while ((1 << bits) <= E) ++bits;
  const SortParams p{experts, weights, offsets, rows, pos, row_weights, static_cast<int32_t *>(workspace),
                     n, k, E, bits, 0};
  return wide ? expert_sort<int64_t>(p, stream) : expert_sort<int32_t>(p, stream);
}

extern "C" gg_status_t gg_expert_spread(const void *X, const int32_t *pos, void *out, const void *scales,
                                        void *out_scales, int32_t scale_bytes, int64_t T, int32_t k,
                                        int64_t row_bytes, int32_t slices, int64_t M_cap, void *stream) {
  gg_status_t st = check_choices(pos, T, k, M_cap);
  if (st != GG_OK) return st;
  if (row_bytes < 1 || slices < 0 || (scale_bytes != 0 && scale_bytes != 4 && scale_bytes != 8) ||
      (scale_bytes == 0) != (slices == 0))
    return GG_ERR_INVALID_VALUE;
  if (row_bytes % 16 != 0) return GG_ERR_MISALIGNED;
  if (row_bytes > (1LL << 31)) return GG_ERR_UNSUPPORTED;
  const int V = spread_pieces(T, row_bytes);
  const long long segments = (row_bytes + V * 1024 - 1) / (V * 1024), units = T * segments;
  // (a multiple of the XCDs, so that the same slices stay on one)
  const long long row_groups = (units + kRowWaves - 1) / kRowWaves,
                  slice_groups = ((slices + (long long)kScaleSlices - 1) / kScaleSlices + 7) / 8 * 8;
  const long long groups = row_groups + (T + kRowThreads - 1) / kRowThreads * slice_groups;
  if (!launch_fits(groups, kRowThreads)) return GG_ERR_UNSUPPORTED;
  if (T > 0 && (X == nullptr || (M_cap > 0 && out == nullptr))) return GG_ERR_INVALID_VALUE;
  if (T > 0 && slices > 0 && (scales == nullptr || (M_cap > 0 && out_scales == nullptr)))
    return GG_ERR_INVALID_VALUE;
  if (!is_aligned(X, 16) || !is_aligned(out, 16) || !is_aligned(scales, 16) || !is_aligned(out_scales, 16))
    return GG_ERR_MISALIGNED;
  const Span x = span(X, T, row_bytes, 1), o = span(out, M_cap, row_bytes, 1), at = span(pos, T, k, 4),
             s = span(scales, T, slices, scale_bytes), os = span(out_scales, M_cap, slices, scale_bytes);
  if (!apart(o, x, at, s, os) || !apart(os, x, at, s)) return GG_ERR_INVALID_VALUE;
  if (T == 0 || M_cap == 0) return GG_OK;
  const SpreadParams p{static_cast<const u32x4 *>(X), static_cast<u32x4 *>(out),
                       static_cast<const char *>(scales), static_cast<char *>(out_scales), pos, units,
                       (int)T, k, (int)(row_bytes / 16), (int)segments, (int)M_cap, scale_bytes,
                       slices, (unsigned)row_groups, (unsigned)slice_groups};
  return launch(V == 4 ? spread_kernel<4> : V == 2 ? spread_kernel<2> : spread_kernel<1>, dim3((unsigned)groups), kRowThreads, 0,
                stream, p);
}

extern "C" gg_status_t gg_expert_combine(const void *Y, int32_t y_fp32, const int32_t *pos,
                                         const float *weights, void *out, int32_t out_fp32, int64_t T,
                                         int32_t k, int32_t N, int64_t M_cap, void *stream) {
  gg_status_t st = check_choices(pos, T, k, M_cap);
  if (st != GG_OK) return st;
  if (N < 1) return GG_ERR_INVALID_VALUE;
  if (N % 8 != 0) return GG_ERR_MISALIGNED;
  const long long segments = (N + kWave * 8LL - 1) / (kWave * 8), units = T * segments;
  const long long groups = (units + kRowWaves - 1) / kRowWaves;
  if (N > GG_MAX_N || !launch_fits(groups, kRowThreads)) return GG_ERR_UNSUPPORTED;
  if (T > 0 && (out == nullptr || (M_cap > 0 && Y == nullptr))) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(Y, 16) || !is_aligned(out, 16) || !is_aligned(weights, 4)) return GG_ERR_MISALIGNED;
  if (!apart(span(out, T, N, out_fp32 ? 4 : 2), span(Y, M_cap, N, y_fp32 ? 4 : 2), span(pos, T, k, 4),
             span(weights, T, k, 4)))
    return GG_ERR_INVALID_VALUE;
  if (T == 0) return GG_OK;
  const CombineParams p{Y, nullptr, pos, weights, out, nullptr, units, (int)T, k, N, (int)M_cap,
                        (int)segments, streams(T * N * (out_fp32 ? 4 : 2))};
  const dim3 grid((unsigned)groups);
  if (y_fp32 && out_fp32) return launch(combine_kernel<float, float>, grid, kRowThreads, 0, stream, p);
  if (y_fp32) return launch(combine_kernel<float, uint16_t>, grid, kRowThreads, 0, stream, p);
  if (out_fp32) return launch(combine_kernel<uint16_t, float>, grid, kRowThreads, 0, stream, p);
  return launch(combine_kernel<uint16_t, uint16_t>, grid, kRowThreads, 0, stream, p);
}

extern "C" gg_status_t gg_expert_combine_grad(const void *dO, const void *Y, int32_t fp32,
                                              const int32_t *pos, const float *weights, void *dY,
                                              float *dweights, int64_t T, int32_t k, int32_t N,
                                              int64_t M_cap, void *stream) {
  gg_status_t st = check_choices(pos, T, k, M_cap);
  if (st != GG_OK) return st;
  if (N < 1) return GG_ERR_INVALID_VALUE;
  if (N % 8 != 0) return GG_ERR_MISALIGNED;
  if (N > GG_MAX_N || !launch_fits(T, kRowThreads)) return GG_ERR_UNSUPPORTED;
  if (T > 0 && (dO == nullptr || weights == nullptr || dweights == nullptr)) return GG_ERR_INVALID_VALUE;
  if (T > 0 && M_cap > 0 && (Y == nullptr || dY == nullptr)) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(dO, 16) || !is_aligned(Y, 16) || !is_aligned(dY, 16) || !is_aligned(weights, 4) ||
      !is_aligned(dweights, 4))
    return GG_ERR_MISALIGNED;
  const int b = fp32 ? 4 : 2;
  const Span o = span(dO, T, N, b), y = span(Y, M_cap, N, b), at = span(pos, T, k, 4),
             w = span(weights, T, k, 4), dy = span(dY, M_cap, N, b), dw = span(dweights, T, k, 4);
  if (!apart(dy, o, y, at, w, dw) || !apart(dw, o, y, at, w)) return GG_ERR_INVALID_VALUE;
  if (T == 0) return GG_OK;
  const CombineParams p{Y, dO, pos, weights, dY, dweights, T, (int)T, k, N, (int)M_cap, 1, false};
  return launch(fp32 ? combine_grad_kernel<float> : combine_grad_kernel<uint16_t>, dim3((unsigned)T),
                kRowThreads, 0, stream, p);
}
