// Root-mean-square norm for gfx950: of a sum with the residual, quantised to
// 8 bits with a scale for each block of 128 on its way out; and its gradient.
//
//   z = bf16(x + residual),  r = 1 / sqrt(mean z^2 + eps),  y = z * r * g
//
// z is rounded before it is normalised, as the layers behind the residual see
// it. Everything else is held in fp32 or more and rounded once.
//
// Both move bytes, in one pass over the rows: 16384 x 6144 with a residual 124.5 us
// for 708 MB (5.7 TB/s); the gradient of 8191 x 6144 77 us for 403 MB and 5 for the
// shares of dg. 16 x 6144: 5.7 us, a launch and two round trips.

#include <float.h>

#include "gg_common.h"
#include "gg_fp8.h"
#include "gg_host.h"
#include "gg_ring.h"
#include "grouped_gemm.h"

namespace gg {

// A row on kNormWaves waves, eight neighbouring values to a lane and V such
// pieces of a row a lane; a workgroup takes kNormRows rows.
constexpr int kNormWaves = 4, kNormRows = 2;
constexpr int kNormThreads = kNormWaves * kNormRows * kWave;
constexpr int kNormPiece = kNormWaves * kWave * 8;  // values of a row at one time

// e with 2^-2 <= ms 2^-2e < 1, so that 1 / sqrt(ms) is 2^-e times a number in (1, 2]
// (0 where ms is 0, infinite or NaN).
__device__ __forceinline__ int root_exponent(double ms) { return (__builtin_amdgcn_frexp_exp(ms) + 1) >> 1; }

// 1 / sqrt(ms) = m 2^e.
struct InverseRoot {
  float m;
  int e;
};
__device__ __forceinline__ InverseRoot inverse_root(double ms) {
  const int e = root_exponent(ms);
  return {1.0f / sqrtf((float)__builtin_ldexp(ms, -2 * e)), -e};
}

// The multiplier of a block whose largest magnitude is t * r, t an fp32 number
// (z g is exact: 16 bits) and r a 64-bit one. It is cut to 16 bits, so where 448 /
// (t r) is next to such a number the last bits of r decide on a whole block: the
// one found in fp32 is put right by comparing in 64 bits. (With r in fp32 a
// quarter percent of the blocks came out one step off, which made nearly all of
// the codes that differ from the formula's.)
__device__ __forceinline__ float norm_multiplier(uint32_t t, float r, double rd) {
  const float m = fp8_multiplier(__builtin_bit_cast(uint32_t, __builtin_bit_cast(float, t) * r));
  if (m == 0.0f) return m;
  const double top = fmax((double)__builtin_bit_cast(float, t) * rd, 0x1p-100);
  const uint32_t bits = __builtin_bit_cast(uint32_t, m);
  const float up = __builtin_bit_cast(float, bits + 0x100u), down = __builtin_bit_cast(float, bits - 0x100u);
  return (double)m * top > (double)kFp8Max ? down : (double)up * top <= (double)kFp8Max ? up : m;
}

__device__ __forceinline__ bool empty(const u32x4 &v) {  // zeros of either sign
  return ((v.x | v.y | v.z | v.w) & 0x7fff7fffu) == 0;
}
constexpr int kSubnormal = 0x10 | 0x80;  // v_cmp_class: subnormal numbers of either sign

struct NormParams {
  const u32x4 *x, *res, *g;
  u32x2 *q;
  float *scales;
  u32x4 *sum, *y;
  int T, K;
  float eps;
  bool stream;
};

template <int V>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormParams p) {
  __shared__ double sums[kNormRows][kNormWaves];
  const int tid = threadIdx.x, lane = tid % kWave, wave = scalar(tid / kWave);
  const int row = wave / kNormWaves, part = wave % kNormWaves;
  const int t = blockIdx.x * kNormRows + row, pitch = p.K / 8;
  const bool live = t < p.T;
  const size_t base = (size_t)t * pitch;
  u32x4 z[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * kNormWaves + part) * kWave + lane;
    z[i] = live && c < pitch ? p.x[base + c] : u32x4{0, 0, 0, 0};
  }
  if (p.res != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * kNormWaves + part) * kWave + lane;
      if (!live || c >= pitch) continue;
      const u32x4 r = p.res[base + c];
      u32x4 s;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 two = {bf16_lo(z[i][j]) + bf16_lo(r[j]), bf16_hi(z[i][j]) + bf16_hi(r[j])};
        s[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
      }
      z[i] = s;
      if (p.sum != nullptr) st_rows(p.sum + base + c, s, p.stream);
    }
  }
  auto val = [](const u32x4 &v, int j) { return j % 2 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]); };
  // eight squares in fp32, the rest in 64 bits; all in 64 bits where a lane's leave fp32
  double sq = 0.0;
  bool far = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float few = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) few = __builtin_fmaf(val(z[i], j), val(z[i], j), few);
    if (!(few >= 0x1p-100f && few < INFINITY)) far |= !empty(z[i]);
    sq += (double)few;
  }
  if (__ballot(far) != 0) {
    sq = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sq = __builtin_fma((double)val(z[i], j), (double)val(z[i], j), sq);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
  sq = sum_of_wave(sq);
  if (lane == 0) sums[row][part] = sq;
  __syncthreads();
  sq = 0.0;
#pragma unroll
  for (int w = 0; w < kNormWaves; ++w) sq += sums[row][w];
  const double ms = sq / p.K + (double)p.eps;
  const double rd = 1.0 / sqrt(ms);
  if (!live || part * kWave >= pitch) return;  // (no columns for this wave)
  // Piece i. z g is exact in fp32 and then multiplied by r. Where a z g is subnormal or beyond
  // fp32, or r is so large that one that is 0 might have mattered, the piece has to be done
  // again (true is returned) with z g scaled by r's power of two, 2^-e (FAR). (Squares in 64
  // bits and scaled products throughout: 16384 x 1024 28.9 us against 24.0 - 22.9 so.)
  auto piece = [&](auto FAR, int i, double r64, int e) {
    const int c = (i * kNormWaves + part) * kWave + lane;
    const bool in = c < pitch;
    const u32x4 g = in ? p.g[c] : u32x4{0, 0, 0, 0};
    float v[8], least = INFINITY;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float zj = val(z[i], j), gj = val(g, j);
      if constexpr (FAR)
        v[j] = __builtin_ldexpf(zj * __builtin_amdgcn_frexp_mantf(gj), __builtin_amdgcn_frexp_expf(gj) - e);
      else
        v[j] = zj * gj;
      top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
      least = fminf(least, fabsf(v[j]));
    }
    bool leaves = top >= 0x7f800000u;
    if (in && least < FLT_MIN)
#pragma unroll
      for (int j = 0; j < 8; ++j) leaves |= __builtin_amdgcn_classf(v[j], kSubnormal);
    const float r = (float)r64, m = norm_multiplier(row16_max(top), r, r64);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= r;
    if (!in) return false;
    if (p.y != nullptr) {
      const u32x2 a = pack_bf16(f32x4{v[0], v[1], v[2], v[3]}),
                  b = pack_bf16(f32x4{v[4], v[5], v[6], v[7]});
      st_rows(p.y + base + c, u32x4{a.x, a.y, b.x, b.y}, p.stream);
    }
    u32x2 o = {fp8_quad(v[0] * m, v[1] * m, v[2] * m, v[3] * m),
               fp8_quad(v[4] * m, v[5] * m, v[6] * m, v[7] * m)};
    if (m == 0.0f) o = u32x2{0, 0};
    st_rows(p.q + base + c, o, p.stream);
    if (lane % 16 == 0) p.scales[(size_t)(c / 16) * p.T + t] = fp8_scale(m);
    return leaves;
  };
  far = !(ms >= 0x1p-40 && ms <= 0x1p200);
#pragma unroll
  for (int i = 0; i < V; ++i) far |= piece(std::false_type{}, i, rd, 0);
  if (__ballot(far) == 0) return;
  const int e = ms < INFINITY ? root_exponent(ms) : 512;  // (r = 0: anything finite is 0)
  const double rest = 1.0 / sqrt(__builtin_ldexp(ms, -2 * e));
#pragma unroll
  for (int i = 0; i < V; ++i) piece(std::true_type{}, i, rest, e);
}

// The gradient: with u = g dY, z the norm's input, r = 1 / sqrt(mean z^2 + eps) and n = z r,
//   dz = r u - n * (r mean(u n)) + the residual's gradient,  dg = sum over rows of dY n.
// Rows may lie anywhere in bf16's range, and z^2, u z and r^3 then leave fp32 where dz
// does not. The sums are taken in fp32 first, as they are good where mean z^2 + eps is
// within 2^-40 and 2^40, no u is subnormal (one that is 0 would give less than 2^-130)
// and no lane's eight u z add up to less than 2^-90 or more than 2^60. Another row's are
// taken again in 64 bits, and n and r u from r's mantissa and power of two apart; r mean
// (u n) is at most r times u's root mean square. (In 64 bits throughout: 8191 x 6144
// 84.5 us against 81, 16384 x 8192 241 against 204.)
// A workgroup takes every so many rows, as many lanes to a row as it has pieces of
// eight values (two pieces a lane above 8192 values), and holds its share of dg in
// registers; a second launch adds the shares in their order.
constexpr int kGradMost = 1024;  // threads of a workgroup at most
constexpr float kGradFar = 0x1p40f, kGradTop = 0x1p60f, kGradLeast = 0x1p-90f;

__device__ __forceinline__ float bf16_of(const u32x4 *p, size_t i) {
  return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
}

struct NormGradParams {
  const u32x4 *dy, *z, *g, *res;
  u32x4 *dz;
  float *shares;  // [workgroups][K]
  int T, K;
  float eps;
  bool stream;
};

// A far row t: r, and r mean(u n), from sums in 64 bits. All threads call it.
struct NormGradFar {
  InverseRoot r;
  float back;
};
__device__ __forceinline__ NormGradFar norm_grad_far(const NormGradParams &p, int t, double (*sums)[2]) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // (addresses are formed here, not kept from row to row)
  const int lane = tid % kWave, wave = tid / kWave;
  double sq = 0.0, uz = 0.0;
#pragma unroll 1
  for (int c = tid; c < p.K; c += blockDim.x) {
    const size_t at = (size_t)t * p.K + c;
    const double z = bf16_of(p.z, at);
    sq += z * z;  // (64 bits hold any product of three)
    uz += (double)bf16_of(p.dy, at) * bf16_of(p.g, c) * z;
  }
  sq = sum_of_wave(sq);
  uz = sum_of_wave(uz);
  if (lane == 0) {
    sums[wave][0] = sq;
    sums[wave][1] = uz;
  }
  __syncthreads();
  sq = uz = 0.0;
#pragma unroll 1
  for (int w = 0; w < (int)blockDim.x / kWave; ++w) {
    sq += sums[w][0];
    uz += sums[w][1];
  }
  __syncthreads();  // sums is written again
  const InverseRoot r = inverse_root(sq / p.K + (double)p.eps);
  return {r, (float)__builtin_ldexp(uz / p.K * r.m * r.m, 2 * r.e)};
}

// (six waves a SIMD: two workgroups of up to 768 threads, rows of 6144, share a CU)
template <int V>
__global__ __launch_bounds__(kGradMost) __attribute__((amdgpu_waves_per_eu(V == 1 ? 6 : 4)))
void norm_grad_kernel(NormGradParams p) {
  __shared__ float sums[2][kGradMost / kWave][2];
  __shared__ double far_sums[kGradMost / kWave][2];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, pitch = p.K / 8;
  const int threads = blockDim.x, waves = threads / kWave;
  float dg[V][8];
  u32x4 g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * threads + tid;
    g[i] = c < pitch ? p.g[c] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  }
  auto val = [](const u32x4 &v, int j) { return j % 2 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]); };
  int turn = 0;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)t * pitch;
    u32x4 z[V], d[V], res[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * threads + tid;
      z[i] = d[i] = res[i] = u32x4{0, 0, 0, 0};
      if (c < pitch) {
        z[i] = p.z[base + c];
        d[i] = p.dy[base + c];
        if (p.res != nullptr) res[i] = p.res[base + c];
      }
    }
    float zf[V][8], u[V][8], sq = 0.0f, uz = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float part = 0.0f, least = INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        zf[i][j] = val(z[i], j);
        u[i][j] = val(d[i], j) * val(g[i], j);
        least = fminf(least, fabsf(u[i][j]));
        sq = __builtin_fmaf(zf[i][j], zf[i][j], sq);
        part = __builtin_fmaf(u[i][j], zf[i][j], part);
      }
      if (!(fabsf(part) >= kGradLeast && fabsf(part) <= kGradTop && least >= FLT_MIN)) {
        bool far = !(fabsf(part) <= kGradTop) ||
                   (fabsf(part) < kGradLeast && !empty(z[i]) && !empty(d[i]) && !empty(g[i]));
#pragma unroll
        for (int j = 0; j < 8; ++j) far |= __builtin_amdgcn_classf(u[i][j], kSubnormal);
        if (far) part = NAN;  // (zeros are no reason)
      }
      uz += part;
    }
    sq = sum_of_wave(sq);
    uz = sum_of_wave(uz);
    if (lane == 0) {
      sums[turn][wave][0] = sq;
      sums[turn][wave][1] = uz;
    }
    __syncthreads();  // (one a row: the next row's sums go to the other half)
    sq = uz = 0.0f;
    for (int w = 0; w < waves; ++w) {
      sq += sums[turn][w][0];
      uz += sums[turn][w][1];
    }
    const float ms = sq / (float)p.K + p.eps;
    float r = 1.0f / sqrtf(ms), back = r * r * (uz / (float)p.K);
    if (scalar(!(ms >= 1.0f / kGradFar && ms <= kGradFar && uz == uz))) {
      const NormGradFar f = norm_grad_far(p, t, far_sums);
      r = f.r.m;
      back = f.back;
      int tid2 = tid;
      asm volatile("" : "+v"(tid2));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * threads + tid2;
        if (c >= pitch) continue;
        const u32x4 z2 = p.z[base + c], g2 = p.g[c];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          zf[i][j] = __builtin_ldexpf(val(z2, j), f.r.e);
          u[i][j] = __builtin_ldexpf(val(d[i], j) * __builtin_amdgcn_frexp_mantf(val(g2, j)),
                                     __builtin_amdgcn_frexp_expf(val(g2, j)) + f.r.e);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * threads + tid;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = zf[i][j] * r;
        dg[i][j] = __builtin_fmaf(val(d[i], j), n, dg[i][j]);
        o[j] = __builtin_fmaf(-back, n, r * u[i][j]) + val(res[i], j);
      }
      if (c < pitch) {
        const u32x2 a = pack_bf16(f32x4{o[0], o[1], o[2], o[3]}),
                    b = pack_bf16(f32x4{o[4], o[5], o[6], o[7]});
        st_rows(p.dz + base + c, u32x4{a.x, a.y, b.x, b.y}, p.stream);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * threads + tid;
    if (c >= pitch) continue;
    f32x4 *const s = (f32x4 *)(p.shares + (size_t)blockIdx.x * p.K + 8 * c);
    s[0] = f32x4{dg[i][0], dg[i][1], dg[i][2], dg[i][3]};
    s[1] = f32x4{dg[i][4], dg[i][5], dg[i][6], dg[i][7]};
  }
}

// dg: a workgroup takes 32 columns, a half wave every 32nd of the shares, in four
// sums side by side.
constexpr int kShareThreads = 1024, kShareCols = 32, kShareRows = kShareThreads / kShareCols;

__global__ __launch_bounds__(kShareThreads) void norm_shares_kernel(const float *__restrict__ shares,
                                                                    float *__restrict__ dg, int groups,
                                                                    int K) {
  __shared__ float part[kShareRows][kShareCols];
  const int col = threadIdx.x % kShareCols, row = threadIdx.x / kShareCols;
  const int c = blockIdx.x * kShareCols + col;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < K) {
#pragma unroll 2
    for (int w = row; w < groups; w += 4 * kShareRows)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (w + u * kShareRows < groups) sum[u] += shares[(size_t)(w + u * kShareRows) * K + c];
  }
  part[row][col] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  __syncthreads();
  if (row != 0 || c >= K) return;
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < kShareRows; ++w) all += part[w][col];
  dg[c] = all;
}

constexpr int kNormMost = 16384;  // columns
static_assert(kNormMost == 8 * kNormPiece, "pieces of a lane");

// Threads of a row of the gradient, and workgroups: what the card holds at one time.
static int grad_threads(int K) {
  const int pieces = (K / 8 + (K > 8192)) / (K > 8192 ? 2 : 1);
  return (pieces + kWave - 1) / kWave * kWave;
}
static int grad_groups(long long T, int K) {
  const int beside = 2048 / grad_threads(K);
  const long long most = 256LL * (beside < 16 ? beside : 16);
  return (int)(T < most ? T : most);
}

static gg_status_t check_norm(int64_t T, int K, float eps) {
  if (T < 0 || K < 1 || !(eps >= 0.0f)) return GG_ERR_INVALID_VALUE;
  if (K % 16 != 0) return GG_ERR_MISALIGNED;
  // (a launch counts its threads, two rows to 512, in 32 bits)
  if (K > kNormMost || T > INT32_MAX || !launch_fits((T + kNormRows - 1) / kNormRows, kNormThreads))
    return GG_ERR_UNSUPPORTED;
  return GG_OK;
}

}  // namespace gg

using namespace gg;

extern "C" gg_status_t gg_rms_norm_fp8(const void *X, const void *residual, const void *weight, void *q,
                                       float *scales, void *sum, void *norm, int64_t T, int32_t K,
                                       float eps, void *stream) {
  gg_status_t st = check_norm(T, K, eps);
  if (st != GG_OK) return st;
  const long long groups = (T + kNormRows - 1) / kNormRows;
  if (sum != nullptr && residual == nullptr) return GG_ERR_INVALID_VALUE;
  if (T == 0) return GG_OK;
  if (X == nullptr || weight == nullptr || q == nullptr || scales == nullptr) return GG_ERR_INVALID_VALUE;
  for (const void *a : {X, residual, weight, (const void *)q, (const void *)scales, (const void *)sum, (const void *)norm})
    if (!is_aligned(a, 16)) return GG_ERR_MISALIGNED;
  const Span x = span(X, T, K, 2), res = span(residual, T, K, 2), g = span(weight, K, 2, 1),
             c = span(q, T, K, 1), s = span(scales, (K + 127) / 128, T, 4), z = span(sum, T, K, 2),
             y = span(norm, T, K, 2);
  // (a lane reads what it adds before it stores the sum: in place is safe)
  if (!apart(c, x, res, g, s, z, y) || !apart(s, x, res, g, z, y) || !apart(z, g, y) ||
      !apart(y, x, res, g) || !(sum == X || apart(z, x)) || !(sum == residual || apart(z, res)))
    return GG_ERR_INVALID_VALUE;
  const NormParams p{static_cast<const u32x4 *>(X), static_cast<const u32x4 *>(residual),
                     static_cast<const u32x4 *>(weight), static_cast<u32x2 *>(q), scales,
                     static_cast<u32x4 *>(sum), static_cast<u32x4 *>(norm), (int)T, K, eps,
                     streams(T * K * (1 + 2 * (sum != nullptr) + 2 * (norm != nullptr)))};
  const int v = (K + kNormPiece - 1) / kNormPiece;
  void (*const kernel)(NormParams) = v == 1   ? norm_kernel<1>
                                     : v == 2 ? norm_kernel<2>
                                     : v == 3 ? norm_kernel<3>
                                     : v == 4 ? norm_kernel<4>
                                              : norm_kernel<8>;
  return launch(kernel, dim3((unsigned)groups), kNormThreads, 0, stream, p);
}

extern "C" int64_t gg_rms_norm_grad_workspace(int64_t T, int32_t K) {
  return T < 1 || K < 1 || K > kNormMost ? 0 : (int64_t)grad_groups(T, K) * K * 4;
}

extern "C" gg_status_t gg_rms_norm_grad(const void *dY, const void *Z, const void *weight,
                                        const void *d_residual, void *dZ, float *dweight,
                                        void *workspace, int64_t T, int32_t K, float eps, void *stream) {
  gg_status_t st = check_norm(T, K, eps);
  if (st != GG_OK) return st;
  if (weight == nullptr || dweight == nullptr) return GG_ERR_INVALID_VALUE;
  if (T > 0 && (dY == nullptr || Z == nullptr || dZ == nullptr || workspace == nullptr))
    return GG_ERR_INVALID_VALUE;
  for (const void *a : {dY, Z, weight, d_residual, (const void *)dZ, (const void *)dweight, (const void *)workspace})
    if (!is_aligned(a, 16)) return GG_ERR_MISALIGNED;
  const Span dy = span(dY, T, K, 2), z = span(Z, T, K, 2), g = span(weight, K, 2, 1),
             res = span(d_residual, T, K, 2), dz = span(dZ, T, K, 2), dg = span(dweight, K, 4, 1),
             ws = span(workspace, gg_rms_norm_grad_workspace(T, K), 1, 1);
  if (!apart(dz, dy, z, g, res, dg, ws) || !apart(dg, dy, z, g, res, ws) || !apart(ws, dy, z, g, res))
    return GG_ERR_INVALID_VALUE;
  const int groups = grad_groups(T, K);
  if (T > 0) {
    const NormGradParams p{static_cast<const u32x4 *>(dY), static_cast<const u32x4 *>(Z),
                           static_cast<const u32x4 *>(weight), static_cast<const u32x4 *>(d_residual),
                           static_cast<u32x4 *>(dZ), static_cast<float *>(workspace), (int)T, K, eps,
                           streams(T * K * 2)};
    st = launch(K > 8192 ? norm_grad_kernel<2> : norm_grad_kernel<1>, dim3((unsigned)groups), grad_threads(K),
                0, stream, p);
    if (st != GG_OK) return st;
  }
  return launch(norm_shares_kernel, dim3((unsigned)((K + kShareCols - 1) / kShareCols)), kShareThreads, 0, stream,
                static_cast<const float *>(workspace), dweight, groups, K);
}
