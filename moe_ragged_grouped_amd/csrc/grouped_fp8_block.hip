// 8-bit operands with a scale for each block of 128 for gfx950: quantisation,
// and the ragged grouped product of them.
//
// Rows have a scale for 128 values along K, weights one for 128 x 128 values.
// Row scales lie slice by slice, scales[k / 128][row], so that those of a
// tile's rows in one slice are one run of memory; weights are kept with their
// output columns as rows, codes [E][N][K] and scales [E][N / 128][K / 128].
//
// What bounds them. The quantisers move bytes: rows 16384 x 6144 54 us (5.6 TB/s),
// weights [64][1024][2688] 85 us (6.2), as they lie 92.5. The product of 32 experts x 16 rows, K =
// 6144, N = 4096: 125 us for 813 MB (6.5 TB/s), the weights' bytes. 64 experts,
// 16384 skewed rows, K = 1024, N = 2688 with SwiGLU: 84 us for 237 MB and 90 GFLOP;
// eight slices a tile at 2.0 us each (0.85 of it on the matrix cores), a tile's
// start and its epilogue not covered by products. One row on each of 8 experts: 9.8
// us, 6 of launch, schedule and first loads.

#include "gg_common.h"
#include "gg_fp8.h"
#include "gg_host.h"
#include "gg_product.h"
#include "gg_ring.h"
#include "gg_schedule.h"
#include "grouped_gemm.h"

namespace gg {

constexpr int kF8Threads = 256;
typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;

__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t two) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                          __builtin_bit_cast(u16x2, two & 0x7fff7fffu)));
}
// The larger half of two bf16 magnitudes, as fp32 bits.
__device__ __forceinline__ uint32_t wider(uint32_t two) { return max(two & 0xffffu, two >> 16) << 16; }

// Rows: a wave takes kF8Rows rows x 4 blocks, a block on 16 lanes of 8 values;
// a workgroup's eight waves take rows below each other, so that its scales of one
// block are 32 rows, a line of memory. (16384 x 6144: 8 rows a wave and four waves
// 54.6 us, 16 rows 124.)
constexpr int kF8Rows = 4, kF8Cols = 4, kF8RowThreads = 512;
constexpr int kF8GroupRows = kF8Rows * kF8RowThreads / kWave;

__global__ __launch_bounds__(kF8RowThreads) void fp8_rows_kernel(const u32x4 *__restrict__ X,
                                                              u32x2 *__restrict__ q,
                                                              float *__restrict__ scales,
                                                              long long rows, int K, int cols) {
  const int lane = threadIdx.x % kWave, wave = scalar(threadIdx.x / kWave);
  const uint32_t down = blockIdx.x / (uint32_t)cols;
  const long long row0 = (long long)down * kF8GroupRows + wave * kF8Rows;
  const int chunk = ((int)(blockIdx.x - down * (uint32_t)cols) * kF8Cols) * 16 + lane;  // of 8 values
  const int pitch = K / 8;
  if (row0 >= rows) return;
  const int n = (int)min((long long)kF8Rows, rows - row0);
  const bool in = chunk < pitch;
  u32x4 v[kF8Rows];
#pragma unroll
  for (int i = 0; i < kF8Rows; ++i)
    v[i] = in && i < n ? X[(row0 + i) * pitch + chunk] : u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kF8Rows; ++i) {
    if (i >= n) break;
    const uint32_t top = row16_max(
        wider(mag_max(mag_max(mag_max(mag_max(0, v[i].x), v[i].y), v[i].z), v[i].w)));
    const float m = fp8_multiplier(top);
    if (!in) continue;
    u32x2 c = {fp8_quad(bf16_lo(v[i].x) * m, bf16_hi(v[i].x) * m, bf16_lo(v[i].y) * m,
                        bf16_hi(v[i].y) * m),
               fp8_quad(bf16_lo(v[i].z) * m, bf16_hi(v[i].z) * m, bf16_lo(v[i].w) * m,
                        bf16_hi(v[i].w) * m)};
    if (m == 0.0f) c = u32x2{0, 0};  // (infinity and NaN times 0 are no 0)
    q[(row0 + i) * pitch + chunk] = c;
    if (lane % 16 == 0) scales[(long long)(chunk / 16) * rows + row0 + i] = fp8_scale(m);
  }
}

// Weights [K][N] of an expert, 128 x 128 a workgroup: a thread takes eight k of
// eight columns. Turned (the product's operand, [N][K]) the codes go through
// LDS; as they lie (the data gradient's operand, [K][N]) they are stored at once.
constexpr int kF8Tile = kFp8Block;

template <bool TURN>
__global__ __launch_bounds__(kF8Threads) void fp8_weights_kernel(const uint16_t *__restrict__ B,
                                                                 uint8_t *__restrict__ q,
                                                                 float *__restrict__ scales, int K,
                                                                 int N, int kblocks, int nblocks,
                                                                 bool stream) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[TURN ? kF8Tile * kF8Tile : 16];
  __shared__ uint32_t tops[kF8Threads / kWave];
  const uint32_t at = blockIdx.x / (uint32_t)nblocks;
  const int nb = (int)(blockIdx.x - at * (uint32_t)nblocks);
  const int kb = (int)(at % (uint32_t)kblocks), e = (int)(at / (uint32_t)kblocks);
  const int tid = threadIdx.x, c = tid % 16, g = tid / 16;
  const int n = nb * kF8Tile + 8 * c, k0 = kb * kF8Tile + 8 * g;
  const bool in = n < N && k0 < K;  // K and N are multiples of 8
  const uint16_t *const src = B + ((size_t)e * K + k0) * N + n;
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    // (streamed: [64][1024][2688] 98.4 -> 82.4 us)
    v[i] = in ? __builtin_nontemporal_load((const u32x4 *)(src + (size_t)i * N)) : u32x4{0, 0, 0, 0};
  uint32_t two = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    two = mag_max(mag_max(mag_max(mag_max(two, v[i].x), v[i].y), v[i].z), v[i].w);
  uint32_t top = wave_max((int)wider(two));
  if (tid % kWave == 0) tops[tid / kWave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kF8Threads / kWave; ++w) top = max(top, tops[w]);
  const float m = fp8_multiplier(top);
  if (tid == 0)
    scales[TURN ? ((size_t)e * nblocks + nb) * kblocks + kb : ((size_t)e * kblocks + kb) * nblocks + nb] =
        fp8_scale(m);
  if constexpr (!TURN) {
    if (!in) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u32x2 o = {fp8_quad(bf16_lo(v[i].x) * m, bf16_hi(v[i].x) * m, bf16_lo(v[i].y) * m,
                          bf16_hi(v[i].y) * m),
                 fp8_quad(bf16_lo(v[i].z) * m, bf16_hi(v[i].z) * m, bf16_lo(v[i].w) * m,
                          bf16_hi(v[i].w) * m)};
      if (m == 0.0f) o = u32x2{0, 0};
      st_rows((u32x2 *)(q + ((size_t)e * K + k0 + i) * N + n), o, stream);
    }
  } else {
    // the eight codes of column 8 c + j at 8-byte chunk g ^ c of its row, so that
    // the 16 columns of a store meet in different banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      auto val = [&](int i) { return (j % 2 ? bf16_hi(v[i][j / 2]) : bf16_lo(v[i][j / 2])) * m; };
      u32x2 o = {fp8_quad(val(0), val(1), val(2), val(3)), fp8_quad(val(4), val(5), val(6), val(7))};
      if (m == 0.0f) o = u32x2{0, 0};
      *(u32x2 *)(codes + (8 * c + j) * kF8Tile + 8 * (g ^ c)) = o;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kF8Tile * kF8Tile / 16 / kF8Threads; ++i) {
      const int col = i * (kF8Threads / 8) + tid / 8, piece = tid % 8, x = col / 8;
      const u32x4 w = *(const u32x4 *)(codes + col * kF8Tile + 16 * (piece ^ (x / 2)));
      const int nn = nb * kF8Tile + col, k = kb * kF8Tile + 16 * piece;
      if (nn < N && k < K)  // K is a multiple of 16
        st_rows((u32x4 *)(q + ((size_t)e * N + nn) * K + k), x % 2 ? u32x4{w.z, w.w, w.x, w.y} : w,
                stream);
    }
  }
}

// ----------------------------------------------------------------- product

struct Fp8BlockParams {
  const char *A, *As;  // [M_cap][K], fp32 [slices][M_cap]
  const char *B, *Bs;  // [E][N][K], fp32 [E][N / 128][slices]
  const int32_t *off;
  void *C;
  int E, K, N, M_cap;
  int bm_fixed, tile_cap;
};

constexpr int kFp8Lds = kRingBytes + (int)sizeof(RingSched);
static_assert(kFp8Lds <= 160 * 1024, "LDS budget");

template <MOut O>
__global__ __launch_bounds__(kThreads, 1) void fp8_product_kernel(Fp8BlockParams p) {
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
    const int slices = cdiv(K, kFp8Block);
    RingTile t;
    t.pitch = (uint32_t)K;
    t.A = p.A + (size_t)tl.row0 * t.pitch;
    t.B = p.B + ((size_t)tl.expert * N + tl.col0) * t.pitch;
    t.as_step = (uint64_t)M * 4;
    t.bs_step = (uint64_t)slices * 4;
    t.As = p.As + (size_t)tl.row0 * 4;
    t.Bs = p.Bs + ((size_t)tl.expert * cdiv(N, kFp8Block) + tl.col0 / kFp8Block) * slices * 4;
    t.rows = tl.rows;
    t.ncols = min(tl.bn, N - tl.col0);
    return t;
  };
  bool after = false;  // the tile before was one of 256 x 256, which stores behind the prologue
  auto run = [&](auto cfg, const RingTile &t, const Tile &tl, auto &next) {
    using C = decltype(cfg);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // keep per-tile index arithmetic inside the tile
    const int wave = scalar(tid / kWave);
    ProductEpi<C, O> epi{p.C, p.N, tl.row0, tl.col0, t.rows, t.ncols, (wave / C::WN) * C::WTM,
                         (wave % C::WN) * C::WTN, tid % kWave};
    int expert = tl.expert;
    asm volatile("" : "+v"(expert));  // (scalars are short)
    auto again = [&] {
      Tile same = tl;
      same.expert = scalar(expert);
      return make(same);
    };
    // its stores: 8 row blocks of one, two or four
    run_ring_tile<C, 8 * (O == MOut::F32 ? 4 : O == MOut::BF16 ? 2 : 1)>(t, lds, tid, 0, epi, next, after,
                                                                         again);
    after = C::BM == 256 && C::BN == 256;
  };
  run_ring_tiles<kRowsFp8>(sched, grid, p.off, p.E, p.M_cap, p.N, p.bm_fixed, lds, make, run);
}

template <MOut O>
static gg_status_t fp8_product(const void *Aq, const void *a_scale, const void *Bq,
                               const void *b_scale, const int32_t *off, void *C, int E, int K,
                               int N, int M_cap, int bm, void *stream) {
  int tile_cap = 0;
  long long tiles = 0;
  gg_status_t st = check_groups(off, E, N, M_cap, bm, kNarrowestN, &tile_cap, &tiles);
  if (st != GG_OK) return st;
  if (Bq == nullptr || b_scale == nullptr || K < 1) return GG_ERR_INVALID_VALUE;
  // arrays of no rows may be null
  if (M_cap > 0 && (Aq == nullptr || a_scale == nullptr || C == nullptr)) return GG_ERR_INVALID_VALUE;
  if (K % 16 != 0 || N % 8 != 0) return GG_ERR_MISALIGNED;
  // a tile's weight rows, 256 * K bytes, stay within 32-bit offsets
  if (K > GG_MAX_K || N > GG_MAX_N) return GG_ERR_UNSUPPORTED;
  if (!is_aligned(Aq, 16) || !is_aligned(a_scale, 16) || !is_aligned(Bq, 16) ||
      !is_aligned(b_scale, 16) || !is_aligned(C, 16))
    return GG_ERR_MISALIGNED;
  const long long slices = (K + (long long)kFp8Block - 1) / kFp8Block,
                  bands = (N + (long long)kFp8Block - 1) / kFp8Block;
  if (!apart(span(C, M_cap, O == MOut::SwiGlu ? N / 2 : N, O == MOut::F32 ? 4 : 2),
             span(Aq, M_cap, K, 1), span(a_scale, slices, M_cap, 4), span(Bq, (long long)E * N, K, 1),
             span(b_scale, E * bands, slices, 4), span(off, E + 1, 1, 4)))
    return GG_ERR_INVALID_VALUE;
  if (M_cap == 0) return GG_OK;
  const Fp8BlockParams p{static_cast<const char *>(Aq), static_cast<const char *>(a_scale),
                         static_cast<const char *>(Bq), static_cast<const char *>(b_scale), off, C, E,
                         K, N, M_cap, bm, tile_cap};
  int dev = 0;
  if (!current_device(&dev)) return GG_ERR_LAUNCH;
  const RingLaunch li = ring_launch<fp8_product_kernel<O>>(dev, kFp8Lds);
  if (li.err != hipSuccess) return GG_ERR_LAUNCH;
  return launch(fp8_product_kernel<O>, dim3((unsigned)li.workgroups(tiles)), kThreads, kFp8Lds, stream, p);
}

}  // namespace gg

using namespace gg;

extern "C" gg_status_t gg_fp8_quantize(const void *X, void *q, float *scales, int64_t rows, int32_t K,
                                       void *stream) {
  if (rows < 0 || K < 1) return GG_ERR_INVALID_VALUE;
  if (K % 16 != 0) return GG_ERR_MISALIGNED;
  if (K > GG_MAX_K || rows > INT32_MAX) return GG_ERR_UNSUPPORTED;
  const long long slices = (K + (long long)kFp8Block - 1) / kFp8Block,
                  cols = (slices + kF8Cols - 1) / kF8Cols;
  const long long groups = (rows + kF8GroupRows - 1) / kF8GroupRows;
  if (!launch_fits(groups * cols, kF8RowThreads)) return GG_ERR_UNSUPPORTED;
  if (rows == 0) return GG_OK;
  if (X == nullptr || q == nullptr || scales == nullptr) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(X, 16) || !is_aligned(q, 16) || !is_aligned(scales, 16)) return GG_ERR_MISALIGNED;
  const Span x = span(X, rows, K, 2), c = span(q, rows, K, 1), s = span(scales, slices, rows, 4);
  if (!apart(x, c, s) || !apart(c, s)) return GG_ERR_INVALID_VALUE;
  return launch(fp8_rows_kernel, dim3((unsigned)(groups * cols)), kF8RowThreads, 0, stream,
                static_cast<const u32x4 *>(X), static_cast<u32x2 *>(q), scales, (long long)rows, K,
                (int)cols);
}

extern "C" gg_status_t gg_fp8_quantize_weights(const void *B, void *q, float *scales, int32_t for_grad,
                                               int32_t E, int32_t K, int32_t N, void *stream) {
  if (B == nullptr || q == nullptr || scales == nullptr || E < 1 || K < 1 || N < 1)
    return GG_ERR_INVALID_VALUE;
  // the rows that are multiplied are whole 16-byte pieces
  if (!is_aligned(B, 16) || !is_aligned(q, 16) || !is_aligned(scales, 16) ||
      K % (for_grad ? 8 : 16) != 0 || N % (for_grad ? 16 : 8) != 0)
    return GG_ERR_MISALIGNED;
  const long long kb = (K + (long long)kFp8Block - 1) / kFp8Block,
                  nb = (N + (long long)kFp8Block - 1) / kFp8Block;
  const int most_k = for_grad ? GG_MAX_N : GG_MAX_K, most_n = for_grad ? GG_MAX_K : GG_MAX_N;
  if (E > kMaxExperts || K > most_k || N > most_n || !launch_fits(kb * nb * E, kF8Threads))
    return GG_ERR_UNSUPPORTED;
  const Span b = span(B, (long long)E * N, K, 2), c = span(q, (long long)E * N, K, 1),
             s = span(scales, E * kb, nb, 4);
  if (!apart(b, c, s) || !apart(c, s)) return GG_ERR_INVALID_VALUE;
  return launch(for_grad ? fp8_weights_kernel<false> : fp8_weights_kernel<true>,
                dim3((unsigned)(kb * nb * E)), kF8Threads, 0, stream, static_cast<const uint16_t *>(B),
                static_cast<uint8_t *>(q), scales, K, N, (int)kb, (int)nb,
                streams((long long)E * K * N));
}

extern "C" gg_status_t gg_grouped_gemm_fp8_block(const void *Aq, const float *a_scale, const void *Bq,
                                                 const float *b_scale, const int32_t *group_offsets,
                                                 float *C, int32_t E, int32_t K, int32_t N,
                                                 int32_t M_cap, int32_t bm, void *stream) {
  return fp8_product<MOut::F32>(Aq, a_scale, Bq, b_scale, group_offsets, C, E, K, N, M_cap, bm, stream);
}

extern "C" gg_status_t gg_grouped_gemm_fp8_block_bf16out(const void *Aq, const float *a_scale,
                                                         const void *Bq, const float *b_scale,
                                                         const int32_t *group_offsets, void *C,
                                                         int32_t E, int32_t K, int32_t N,
                                                         int32_t M_cap, int32_t bm, void *stream) {
  return fp8_product<MOut::BF16>(Aq, a_scale, Bq, b_scale, group_offsets, C, E, K, N, M_cap, bm, stream);
}

extern "C" gg_status_t gg_grouped_gemm_fp8_block_swiglu(const void *Aq, const float *a_scale,
                                                        const void *Bq, const float *b_scale,
                                                        const int32_t *group_offsets, void *H,
                                                        int32_t E, int32_t K, int32_t N,
                                                        int32_t M_cap, int32_t bm, void *stream) {
  return fp8_product<MOut::SwiGlu>(Aq, a_scale, Bq, b_scale, group_offsets, H, E, K, N, M_cap, bm,
                                   stream);
}
