// 4-bit microscaled operands for gfx950: quantisation, what the codes stand
// for, and the ragged grouped product of them.
//
// The format is the OCP MX one for 4 bits: blocks of 32 values along K share a
// scale 2^(code - 127) (E8M0, 0xFF = NaN); a value is E2M1, one of 0, .5, 1,
// 1.5, 2, 3, 4, 6 with a sign. Codes lie two to a byte, the even k in the low
// half. Scale bytes lie slice by slice, a slice being 256 k or 8 blocks:
// scales[k / 256][row][(k / 32) % 8], so that the scales of a tile's rows in
// one slice are one run of memory.
//
// What bounds them. Quantisation and its inverse move bytes: 16384 x 6144 to 4
// bits 44 us (5.8 TB/s), back 40 (6.3); weights [64][1024][2688] 73 (6.1), back
// 64 (7.0). The product of 32 experts x 16 rows, K = 6144, N = 4096: 72 us for
// 438 MB (6.0 TB/s), the weights' bytes, a third of the 16-bit product's. 64
// experts, 16384 skewed rows, K = 1024, N = 2688 with SwiGLU: 62 us for 147 MB
// and 90 GFLOP; four slices a tile leave its start, its epilogue and the last
// partly filled round of tiles uncovered. One row on each of 8 experts: 9.4
// us, nearly all of it launch, schedule and the first loads' latency.

#include "gg_common.h"
#include "gg_host.h"
#include "gg_product.h"
#include "gg_ring.h"
#include "gg_schedule.h"
#include "grouped_gemm.h"

namespace gg {

constexpr int kBlockK = 32, kSliceK = 256, kSliceBlocks = kSliceK / kBlockK;
constexpr int kQThreads = 256;

// Scale code of a block whose largest magnitude has the bf16 bits `top`
// (sign cleared): 2^(floor(log2 top) - 2), not below 2^-127; NaN where the
// block holds an infinity or a NaN.
__device__ __forceinline__ int scale_code(uint32_t top) {
  const int e = (int)(top >> 7);  // 127 + floor(log2), 0 for zeros and subnormals
  return e == 255 ? 255 : max(e - 2, 0);
}

// 2^(code - 127) as a float (code 0 is the subnormal 2^-127)
__device__ __forceinline__ float scale_value(int code) {
  return __builtin_bit_cast(float, code == 0 ? 0x00400000u : (uint32_t)code << 23);
}

// Eight bf16 values -> eight codes: v / scale to the nearest E2M1 value, ties
// to even, at most 6 (v_cvt_scalef32_pk_fp4_bf16; checked against the
// definition for every bf16 pattern).
template <int PAIR>
__device__ __forceinline__ uint32_t encode2(uint32_t q, uint32_t two, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, two), scale, PAIR);
}
__device__ __forceinline__ uint32_t encode8(u32x4 v, float scale) {
  return encode2<3>(encode2<2>(encode2<1>(encode2<0>(0, v.x, scale), v.y, scale), v.z, scale), v.w,
                    scale);
}

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t top8(u32x4 v) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return max_u16x2(max_u16x2(v.x & kMag, v.y & kMag), max_u16x2(v.z & kMag, v.w & kMag));
}
__device__ __forceinline__ uint32_t top_of_pair(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// A value of the lane d lanes on within its group of four (d XORed).
template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;  // quad_perm [1,0,3,2] and [2,3,0,1]

// Rows: 64 blocks a wave. A load takes 16 neighbouring blocks, four lanes of 8
// values each; four loads are in flight together. The four lanes of a block
// then trade codes (a 4 x 4 transposition by quad permutations), so that lane
// p of a group keeps the whole of the p-th load's block: one 16-byte store of
// codes and one byte of scale a lane.
constexpr int kChunks = 4;

__global__ __launch_bounds__(kQThreads) void mx4_rows_kernel(const u32x4 *__restrict__ X,
                                                             u32x4 *__restrict__ q,
                                                             uint8_t *__restrict__ scales,
                                                             long long rows, int K) {
  const uint32_t bpr = (uint32_t)K / kBlockK;  // blocks per row
  const long long blocks = rows * bpr;
  // this wave's first block; the workgroup's place in a row is scalar
  const int wave = scalar(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const long long b0 = ((long long)blockIdx.x * (kQThreads / kWave) + wave) * 64;
  const long long row0 = b0 / bpr;
  const uint32_t rem0 = (uint32_t)(b0 - row0 * bpr);
  u32x4 v[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const long long b = b0 + j * 16 + lane / 4;
    v[j] = b < blocks ? X[4 * b + lane % 4] : u32x4{0, 0, 0, 0};
  }
  uint32_t w[kChunks], code[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    uint32_t m = top8(v[j]);
    m = max_u16x2(m, quad<kQuadXor1>(m));
    m = max_u16x2(m, quad<kQuadXor2>(m));
    const int c = scale_code(top_of_pair(m));
    code[j] = (uint32_t)c;
    w[j] = c == 255 ? 0u : encode8(v[j], scale_value(c));
  }
  // w[j] of lane p is part p of block j: transpose, so that w[i] of lane p is
  // part i of block p
  const bool odd = lane & 1, high = lane & 2;
  u32x4 out;
  {
    const uint32_t s0 = odd ? w[0] : w[1], s1 = odd ? w[2] : w[3];
    const uint32_t r0 = quad<kQuadXor1>(s0), r1 = quad<kQuadXor1>(s1);
    const uint32_t x0 = odd ? r0 : w[0], x1 = odd ? w[1] : r0;  // parts (even, odd) of block 0 or 1
    const uint32_t y0 = odd ? r1 : w[2], y1 = odd ? w[3] : r1;  // of block 2 or 3
    const uint32_t t0 = quad<kQuadXor2>(high ? x0 : y0), t1 = quad<kQuadXor2>(high ? x1 : y1);
    out = high ? u32x4{t0, t1, y0, y1} : u32x4{x0, x1, t0, t1};
  }
  const uint32_t mine = high ? (odd ? code[3] : code[2]) : (odd ? code[1] : code[0]);
  const uint32_t at = (uint32_t)(lane % 4) * 16 + lane / 4;
  const long long b = b0 + at;
  if (b >= blocks) return;
  q[b] = out;
  const uint32_t pos = rem0 + at;
  const uint32_t down = pos / bpr;
  int kb = (int)(pos - down * bpr);
  uint8_t *const s = scales + ((long long)(kb / kSliceBlocks) * rows + row0 + down) * kSliceBlocks;
  s[kb % kSliceBlocks] = (uint8_t)mine;
  if (kb == (int)bpr - 1)
    while (++kb % kSliceBlocks != 0) s[kb % kSliceBlocks] = 0;  // no block there
}

// Weights [K][N] of an expert -> [N][K / 2]: blocks run down the columns. A
// workgroup takes 256 k x 256 n; wave w block w of the slice, a lane four
// columns (32 loads of 8 bytes, 512 bytes of a row to a wave). Codes go
// through LDS, so that a column's 128 bytes leave as one run.
constexpr int kWqThreads = 512, kWqCols = 256;

__global__ __launch_bounds__(kWqThreads) void mx4_weights_kernel(const uint16_t *__restrict__ B,
                                                                 uint8_t *__restrict__ q,
                                                                 uint8_t *__restrict__ scales,
                                                                 int K, int N, int slices,
                                                                 int cols) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[kWqCols * 128];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kWqCols * kSliceBlocks];
  // neighbouring workgroups take neighbouring columns
  const uint32_t at = blockIdx.x / (uint32_t)cols;
  const int slice = (int)(at % (uint32_t)slices), e = (int)(at / (uint32_t)slices);
  const int n0 = (int)(blockIdx.x % (uint32_t)cols) * kWqCols;
  const int tid = threadIdx.x, w = tid / kWave, lane = tid % kWave;
  const int k0 = slice * kSliceK + w * kBlockK;
  const int n = n0 + 4 * lane;
  const bool in = k0 < K && n < N;  // K is a multiple of 32, N of 8
  const uint16_t *const src = B + ((size_t)e * K + k0) * N + n;
  u32x2 v[kBlockK];
#pragma unroll
  for (int k = 0; k < kBlockK; ++k)
    v[k] = in ? __builtin_nontemporal_load((const gbl_u32x2 *)(src + (size_t)k * N)) : u32x2{0, 0};
  uint32_t m[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < kBlockK; ++k) {
    m[0] = max_u16x2(m[0], v[k].x & 0x7fff7fffu);
    m[1] = max_u16x2(m[1], v[k].y & 0x7fff7fffu);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t top = j % 2 ? m[j / 2] >> 16 : m[j / 2] & 0xffffu;
    const int code = scale_code(top);
    const float scale = scale_value(code);
    u32x4 out;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      u32x4 in8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = v[8 * d + 2 * i][j / 2], b = v[8 * d + 2 * i + 1][j / 2];
        in8[i] = j % 2 ? (a >> 16) | (b & 0xffff0000u) : (a & 0xffffu) | (b << 16);
      }
      out[d] = code == 255 ? 0u : encode8(in8, scale);
    }
    const int col = 4 * lane + j;
    // chunk w of column col at chunk w ^ (lane % 8): the lanes of a store
    // would otherwise all meet in the same banks
    *(u32x4 *)(codes + col * 128 + 16 * (w ^ (lane % 8))) = out;
    sc[col * kSliceBlocks + w] = k0 < K ? (uint8_t)code : 0;
  }
  __syncthreads();
  const int c = tid % 8;
#pragma unroll
  for (int i = 0; i < kWqCols / (kWqThreads / 8); ++i) {
    const int col = i * (kWqThreads / 8) + tid / 8;
    const int k = slice * kSliceK + c * kBlockK;
    if (k < K && n0 + col < N)
      *(gbl_u32x4 *)(q + ((size_t)e * N + n0 + col) * (K / 2) + k / 2) =
          *(const u32x4 *)(codes + col * 128 + 16 * (c ^ (col / 4 % 8)));
  }
  if (tid < kWqCols && n0 + tid < N)
    *(gbl_u32x2 *)(scales + (((size_t)e * slices + slice) * N + n0 + tid) * kSliceBlocks) =
        *(const u32x2 *)(sc + tid * kSliceBlocks);
}

// The bf16 values that codes and scales stand for, 8 to a lane. Every value
// below 2^128 is a bf16 value; larger ones become infinite.
__global__ __launch_bounds__(kQThreads) void mx4_values_kernel(const uint32_t *__restrict__ q,
                                                               const uint8_t *__restrict__ scales,
                                                               u32x4 *__restrict__ Y,
                                                               long long rows, int K, int slices) {
  const uint32_t per_row = (uint32_t)K / 8;
  const long long total = rows * per_row;
  const long long c0 = (long long)blockIdx.x * (kQThreads * kChunks);
  const long long row0 = c0 / per_row;
  const uint32_t rem0 = (uint32_t)(c0 - row0 * per_row);
  const size_t base = (size_t)blockIdx.y * total;  // this batch
  uint32_t w[kChunks];
  int code[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const long long c = c0 + j * kQThreads + threadIdx.x;
    w[j] = 0;
    code[j] = 0;
    if (c < total) {
      const uint32_t at = rem0 + j * kQThreads + threadIdx.x;
      const long long r = row0 + at / per_row;
      const int b = (int)(at % per_row) / 4;
      w[j] = q[base + c];
      code[j] = scales[(((size_t)blockIdx.y * slices + b / kSliceBlocks) * rows + r) * kSliceBlocks +
                       b % kSliceBlocks];
    }
  }
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const long long c = c0 + j * kQThreads + threadIdx.x;
    if (c >= total) continue;
    u32x4 y = {0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
    if (code[j] != 255) {
      const float s = scale_value(code[j]);
      y.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0));
      y.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1));
      y.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2));
      y.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3));
    }
    // four times what was read, and whole lines: streamed, so that it does not
    // push everything else out of the caches (16384 x 6144 there and back, each
    // time from other inputs: 97.7 -> 85.0 us)
    __builtin_nontemporal_store(y, Y + base + c);
  }
}

// ----------------------------------------------------------------- product

struct Mx4Params {
  const char *A, *As;   // [M_cap][K / 2], [slices][M_cap][8]
  const char *B, *Bs;   // [E][N][K / 2], [E][slices][N][8]
  const int32_t *off;
  void *C;
  int E, K, N, M_cap;
  int bm_fixed, tile_cap;
};

constexpr int kMx4Lds = kRingBytes + (int)sizeof(RingSched);
static_assert(kMx4Lds <= 160 * 1024, "LDS budget");

template <MOut O>
__global__ __launch_bounds__(kThreads, 1) void mx4_product_kernel(Mx4Params p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_dyn[];
  lds_u8 *const lds = (lds_u8 *)lds_dyn;
  RingSched &sched = *(RingSched *)(lds_dyn + kRingBytes);
  const RingGrid grid = build_ring_schedule(sched, p.off, p.E, p.M_cap, p.N, p.bm_fixed, p.tile_cap,
                                            gridDim.x);
  auto make = [&](const Tile &tl) {
    // sizes the compiler cannot see through: what it derives from them is then
    // computed per tile instead of being kept (and spilled) across tiles
    int K = p.K, N = p.N, M = p.M_cap;
    asm volatile("" : "+s"(K), "+s"(N), "+s"(M));
    RingTile t;
    t.pitch = (uint32_t)K / 2;
    t.A = p.A + (size_t)tl.row0 * t.pitch;
    t.B = p.B + ((size_t)tl.expert * N + tl.col0) * t.pitch;
    t.as_step = (uint64_t)M * kSliceBlocks;
    t.bs_step = (uint64_t)N * kSliceBlocks;
    t.As = p.As + (size_t)tl.row0 * kSliceBlocks;
    t.Bs = p.Bs + (size_t)tl.expert * cdiv(K, kSliceK) * t.bs_step + (size_t)tl.col0 * kSliceBlocks;
    t.rows = tl.rows;
    t.ncols = min(tl.bn, N - tl.col0);
    return t;
  };
  auto run = [&](auto cfg, const RingTile &t, const Tile &tl, auto &next) {
    using C = decltype(cfg);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // keep per-tile index arithmetic inside the tile
    const int wave = scalar(tid / kWave);
    ProductEpi<C, O> epi{p.C, p.N, tl.row0, tl.col0, t.rows, t.ncols, (wave / C::WN) * C::WTM,
                         (wave % C::WN) * C::WTN, tid % kWave};
    run_ring_tile<C>(t, lds, tid, p.K / kBlockK, epi, next);
  };
  run_ring_tiles<kRowsMx4>(sched, grid, p.off, p.E, p.M_cap, p.N, p.bm_fixed, lds, make, run);
}

template <MOut O>
static gg_status_t mx4_product(const void *Aq, const void *a_scale, const void *Bq,
                               const void *b_scale, const int32_t *off, void *C, int E, int K,
                               int N, int M_cap, int bm, void *stream) {
  int tile_cap = 0;
  long long tiles = 0;
  gg_status_t st = check_groups(off, E, N, M_cap, bm, kNarrowestN, &tile_cap, &tiles);
  if (st != GG_OK) return st;
  if (Bq == nullptr || b_scale == nullptr || K < 1) return GG_ERR_INVALID_VALUE;
  // arrays of no rows may be null
  if (M_cap > 0 && (Aq == nullptr || a_scale == nullptr || C == nullptr)) return GG_ERR_INVALID_VALUE;
  if (K % kBlockK != 0 || N % 8 != 0) return GG_ERR_MISALIGNED;
  // a tile's weight rows, 256 * K / 2 bytes, stay within 32-bit offsets
  if (K > GG_MAX_K || N > GG_MAX_N) return GG_ERR_UNSUPPORTED;
  if (!is_aligned(Aq, 16) || !is_aligned(a_scale, 16) || !is_aligned(Bq, 16) ||
      !is_aligned(b_scale, 16) || !is_aligned(C, 16))
    return GG_ERR_MISALIGNED;
  const long long slices = (K + (long long)kSliceK - 1) / kSliceK;
  if (!apart(span(C, M_cap, O == MOut::SwiGlu ? N / 2 : N, O == MOut::F32 ? 4 : 2),
             span(Aq, M_cap, K / 2, 1), span(a_scale, slices * M_cap, kSliceBlocks, 1),
             span(Bq, (long long)E * N, K / 2, 1),
             span(b_scale, (long long)E * N, slices * kSliceBlocks, 1), span(off, E + 1, 1, 4)))
    return GG_ERR_INVALID_VALUE;
  if (M_cap == 0) return GG_OK;
  const Mx4Params p{static_cast<const char *>(Aq), static_cast<const char *>(a_scale),
                    static_cast<const char *>(Bq), static_cast<const char *>(b_scale), off, C, E, K,
                    N, M_cap, bm, tile_cap};
  int dev = 0;
  if (!current_device(&dev)) return GG_ERR_LAUNCH;
  const RingLaunch li = ring_launch<mx4_product_kernel<O>>(dev, kMx4Lds);
  if (li.err != hipSuccess) return GG_ERR_LAUNCH;
  return launch(mx4_product_kernel<O>, dim3((unsigned)li.workgroups(tiles)), kThreads, kMx4Lds, stream, p);
}

// Full-width values, codes and scales of `rows` rows, none overlapping another.
static bool rows_apart(const void *values, const void *q, const void *scales, long long rows,
                       long long K) {
  const Span v = span(values, rows, K, 2), c = span(q, rows, K / 2, 1),
             s = span(scales, rows, (K + kSliceK - 1) / kSliceK * kSliceBlocks, 1);
  return apart(v, c, s) && apart(c, s);
}

// Sizes of the row kernels: blocks of a launch, within the grid's limit.
static gg_status_t check_rows(int64_t rows, int K, long long *blocks) {
  if (rows < 0 || K < 1) return GG_ERR_INVALID_VALUE;
  if (K % kBlockK != 0) return GG_ERR_MISALIGNED;
  if (K > GG_MAX_K || rows > INT32_MAX) return GG_ERR_UNSUPPORTED;
  const long long per = kQThreads * kChunks;
  *blocks = (rows * (K / 8) + per - 1) / per;
  return launch_fits(*blocks, kQThreads) ? GG_OK : GG_ERR_UNSUPPORTED;
}

}  // namespace gg

using namespace gg;

extern "C" gg_status_t gg_mx4_quantize(const void *X, void *q, void *scales, int64_t rows,
                                       int32_t K, void *stream) {
  long long blocks = 0;
  const gg_status_t st = check_rows(rows, K, &blocks);
  if (st != GG_OK) return st;
  if (rows == 0) return GG_OK;
  if (X == nullptr || q == nullptr || scales == nullptr) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(X, 16) || !is_aligned(q, 16) || !is_aligned(scales, 16)) return GG_ERR_MISALIGNED;
  if (!rows_apart(X, q, scales, rows, K)) return GG_ERR_INVALID_VALUE;
  return launch(mx4_rows_kernel, dim3((unsigned)blocks), kQThreads, 0, stream,
                static_cast<const u32x4 *>(X), static_cast<u32x4 *>(q),
                static_cast<uint8_t *>(scales), (long long)rows, K);
}

extern "C" gg_status_t gg_mx4_quantize_weights(const void *B, void *q, void *scales, int32_t E,
                                               int32_t K, int32_t N, void *stream) {
  if (B == nullptr || q == nullptr || scales == nullptr || E < 1 || K < 1 || N < 1)
    return GG_ERR_INVALID_VALUE;
  if (!is_aligned(B, 16) || !is_aligned(q, 16) || !is_aligned(scales, 16) || K % kBlockK != 0 ||
      N % 8 != 0)
    return GG_ERR_MISALIGNED;
  const long long slices = (K + (long long)kSliceK - 1) / kSliceK, cols = (N + (long long)kWqCols - 1) / kWqCols;
  if (E > kMaxExperts || K > GG_MAX_K || N > GG_MAX_N ||
      !launch_fits(slices * cols * E, kWqThreads))
    return GG_ERR_UNSUPPORTED;
  if (!rows_apart(B, q, scales, (long long)E * N, K)) return GG_ERR_INVALID_VALUE;
  return launch(mx4_weights_kernel, dim3((unsigned)(slices * cols * E)), kWqThreads, 0, stream,
                static_cast<const uint16_t *>(B), static_cast<uint8_t *>(q),
                static_cast<uint8_t *>(scales), K, N, (int)slices, (int)cols);
}

extern "C" gg_status_t gg_mx4_dequantize(const void *q, const void *scales, void *Y, int32_t batch,
                                         int64_t rows, int32_t K, void *stream) {
  long long blocks = 0;
  const gg_status_t st = check_rows(rows, K, &blocks);
  if (st != GG_OK) return st;
  if (batch < 0) return GG_ERR_INVALID_VALUE;
  if (batch > 65535) return GG_ERR_UNSUPPORTED;
  if (rows == 0 || batch == 0) return GG_OK;
  if (q == nullptr || scales == nullptr || Y == nullptr) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(q, 16) || !is_aligned(scales, 16) || !is_aligned(Y, 16)) return GG_ERR_MISALIGNED;
  if (!rows_apart(Y, q, scales, batch * rows, K)) return GG_ERR_INVALID_VALUE;
  return launch(mx4_values_kernel, dim3((unsigned)blocks, (unsigned)batch), kQThreads, 0, stream,
                static_cast<const uint32_t *>(q), static_cast<const uint8_t *>(scales),
                static_cast<u32x4 *>(Y), (long long)rows, K, (K + kSliceK - 1) / kSliceK);
}

extern "C" gg_status_t gg_grouped_gemm_mx4(const void *Aq, const void *a_scale, const void *Bq,
                                           const void *b_scale, const int32_t *group_offsets,
                                           float *C, int32_t E, int32_t K, int32_t N,
                                           int32_t M_cap, int32_t bm, void *stream) {
  return mx4_product<MOut::F32>(Aq, a_scale, Bq, b_scale, group_offsets, C, E, K, N, M_cap, bm,
                                stream);
}

extern "C" gg_status_t gg_grouped_gemm_mx4_bf16out(const void *Aq, const void *a_scale,
                                                   const void *Bq, const void *b_scale,
                                                   const int32_t *group_offsets, void *C,
                                                   int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                                   int32_t bm, void *stream) {
  return mx4_product<MOut::BF16>(Aq, a_scale, Bq, b_scale, group_offsets, C, E, K, N, M_cap, bm,
                                 stream);
}

extern "C" gg_status_t gg_grouped_gemm_mx4_swiglu(const void *Aq, const void *a_scale,
                                                  const void *Bq, const void *b_scale,
                                                  const int32_t *group_offsets, void *H, int32_t E,
                                                  int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                                  void *stream) {
  return mx4_product<MOut::SwiGlu>(Aq, a_scale, Bq, b_scale, group_offsets, H, E, K, N, M_cap, bm,
                                   stream);
}
