// Data gradient of the ragged grouped product, for gfx950:
//
//   dA[r][k] = sum_n dC[r][n] * B[e][k][n]        for the rows r of expert e
//
// and the same sum with the backward of SwiGLU applied to it before it is
// stored. B keeps the forward product's layout [E][K][N]: its row k is
// contiguous along n, the index summed over here, and so is dC's row r. Both
// operands are read as they lie (gg_ring.h); nothing is transposed.
//
// One persistent launch walks the tiles of all experts (the schedule of
// gg_ring.h, K in the place of the output columns).
//
// What bounds it. 64 experts x 256 rows, K = 1024, N = 2688, bf16 out: 91 us,
// 474 MB (5.2 TB/s, above the 4.9 TB/s of a plain copy, as most of it is read)
// and 988 TFLOP/s; the bytes. Skewed routing of the same rows, K = 1344, N =
// 1024, with the SwiGLU gradient and H: 122 us, 430 MB at 3.5 TB/s; rounds of
// 256-row tiles whose epilogue (a third of the bytes) follows their products.
// Few tiles (12 experts, 777 rows, K = 712, N = 1000): 19 us, 16 slices one after
// the other at about 0.6 us, and 5 us of launch and schedule.

#include "gg_common.h"
#include "gg_host.h"
#include "gg_ring.h"
#include "gg_schedule.h"
#include "grouped_gemm.h"

namespace gg {

enum class DOut { F32, BF16, SwiGlu };

struct DgradParams {
  const char *dC;        // [M_cap][N] bf16
  const char *B;         // [E][K][N] bf16
  const int32_t *off;
  void *out;             // dA [M_cap][K], or d(gate, up) [M_cap][2K]
  const uint16_t *C;     // SwiGlu: gate and up columns interleaved [M_cap][2K]
  uint16_t *H;           // SwiGlu: the activation [M_cap][K], or null
  int E, K, N, M_cap;
  int bm_fixed, tile_cap;
};

// sigmoid(x) with the hardware exp2 and reciprocal (each within one ulp); 0
// where it would be subnormal (x below about -87.3).
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float kLog2e = 1.4426950408889634f;
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xffff0000u);
}

// The epilogue of one tile; row0, col0: its first row and output column.
template <class C, DOut O>
struct DgradEpi {
  const DgradParams &p;
  int row0, col0, rows, ncols, wm0, wn0, lane;
  // SwiGlu: the gate and up columns of a row block, loaded one block ahead of
  // their use. The stores of a block go out after the next one's loads, so
  // that waiting on those does not wait on the stores (one counter covers
  // both, in order).
  u32x4 c[2][O == DOut::SwiGlu ? C::NI : 1];

  __device__ __forceinline__ buf_rsrc pairs(const void *base, int mi) const {
    const size_t bytes = 4 * (size_t)p.K;  // a row of interleaved columns
    return row_block((const char *)base + row0 * bytes + 4 * (size_t)col0, wm0 + mi * 16, rows,
                     bytes, 4 * (size_t)col0);
  }
  // Place of this lane's piece of block ni: row s, or (two blocks trading rows,
  // swap_rows) row s % 8 of left and right, 8 rows further down for odd ni.
  static constexpr bool kTrade = C::NI % 2 == 0;
  __device__ __forceinline__ uint32_t pair_off(int ni) const {
    const int g = lane / 16, s = lane % 16;
    const int n = wn0 + (kTrade ? ni / 2 * 2 + s / 8 : ni) * 16 + 4 * g;
    const int row = kTrade ? s % 8 + ni % 2 * 8 : s;
    return n < ncols ? (uint32_t)row * 4u * (uint32_t)p.K + 4u * n : kOob;
  }
  __device__ __forceinline__ void load(int mi) {
    const buf_rsrc r = pairs(p.C, mi);
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) c[mi % 2][ni] = ld_buf16(r, pair_off(ni), 0);
  }
  __device__ __forceinline__ void begin() {
    if constexpr (O == DOut::SwiGlu) load(0);
  }

  __device__ __forceinline__ void block(const f32x4 (&acc)[C::NI][C::MI], int mi) {
    const size_t es = O == DOut::F32 ? 4 : 2;
    if constexpr (O != DOut::SwiGlu) {
      store_block<C, O == DOut::BF16>(acc, mi, (char *)p.out + ((size_t)row0 * p.K + col0) * es, wm0,
                                      wn0, lane, rows, ncols, p.K * es, col0 * es);
    } else {
      // dH = acc; with sg = sigmoid(gate):
      //   d gate = dH * up * sg * (1 + gate * (1 - sg)),  d up = dH * gate * sg,
      //   H = gate * sg * up
      if (mi + 1 < C::MI) load(mi + 1);
      const buf_rsrc r = pairs(p.out, mi);
      f32x4 h[C::NI][C::MI];
      u32x4 d[C::NI];
      if constexpr (kTrade) {
#pragma unroll
        for (int ni = 0; ni < C::NI; ni += 2) swap_rows(c[mi % 2][ni], c[mi % 2][ni + 1]);
      }
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = c[mi % 2][ni][j];
          const float gate = lo_bf16(w), up = hi_bf16(w);
          const float sg = sigmoid(gate), dh = acc[ni][mi][j];
          const float act = gate * sg;
          // sg * (1 + gate * (1 - sg)), the slope of the activation, goes to
          // up first: dh * up alone may leave fp32's range where a small slope
          // brings it back. slope * up does so only where H does too (a slope
          // above 1 is below the activation itself); what subnormal numbers
          // lose of it is at most 2^-149 |dh|.
          const float slope = sg + act * (1.0f - sg);
          const f32x2 dv = {dh * (slope * up), dh * act};
          d[ni][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(dv, bf16x2));
          h[ni][mi][j] = act * up;
        }
      }
      if constexpr (kTrade) {
#pragma unroll
        for (int ni = 0; ni < C::NI; ni += 2) swap_rows(d[ni], d[ni + 1]);
      }
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) st_buf16(r, pair_off(ni), d[ni]);
      if (p.H != nullptr)
        store_block<C, true>(h, mi, p.H + (size_t)row0 * p.K + col0, wm0, wn0, lane, rows, ncols,
                             p.K * es, col0 * es);
    }
  }
};

constexpr int kDgradLds = kRingBytes + (int)sizeof(RingSched);
static_assert(kDgradLds <= 160 * 1024, "LDS budget");

template <DOut O>
__global__ __launch_bounds__(kThreads, 1) void dgrad_kernel(DgradParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_dyn[];
  lds_u8 *const lds = (lds_u8 *)lds_dyn;
  RingSched &sched = *(RingSched *)(lds_dyn + kRingBytes);
  const RingGrid grid = build_ring_schedule(sched, p.off, p.E, p.M_cap, p.K, p.bm_fixed, p.tile_cap,
                                            gridDim.x);
  auto make = [&](const Tile &tl) {
    // sizes the compiler cannot see through: what it derives from them is then
    // computed per tile instead of being kept (and spilled) across tiles
    int K = p.K, N = p.N;
    asm volatile("" : "+s"(K), "+s"(N));
    RingTile t;
    t.pitch = 2u * (uint32_t)N;
    t.A = p.dC + (size_t)tl.row0 * t.pitch;
    t.B = p.B + ((size_t)tl.expert * K + tl.col0) * t.pitch;
    t.As = t.Bs = nullptr;
    t.as_step = t.bs_step = 0;
    t.rows = tl.rows;
    t.ncols = min(tl.bn, K - tl.col0);
    return t;
  };
  auto run = [&](auto cfg, const RingTile &t, const Tile &tl, auto &next) {
    using C = decltype(cfg);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // keep per-tile index arithmetic inside the tile
    const int wave = scalar(tid / kWave);
    DgradEpi<C, O> epi{p, tl.row0, tl.col0, t.rows, t.ncols, (wave / C::WN) * C::WTM,
                       (wave % C::WN) * C::WTN, tid % kWave, {}};
    run_ring_tile<C>(t, lds, tid, 0, epi, next);
  };
  run_ring_tiles<false>(sched, grid, p.off, p.E, p.M_cap, p.K, p.bm_fixed, lds, make, run);
}

template <DOut O>
static gg_status_t dgrad(DgradParams p, void *stream) {
  long long tiles = 0;
  gg_status_t st =
      check_groups(p.off, p.E, p.K, p.M_cap, p.bm_fixed, kNarrowestN, &p.tile_cap, &tiles);
  if (st != GG_OK) return st;
  if (p.B == nullptr || p.N < 1) return GG_ERR_INVALID_VALUE;
  // arrays of no rows may be null
  if (p.M_cap > 0 && (p.dC == nullptr || p.out == nullptr || (O == DOut::SwiGlu && p.C == nullptr)))
    return GG_ERR_INVALID_VALUE;
  if (p.K % 8 != 0 || p.N % 8 != 0) return GG_ERR_MISALIGNED;
  // a tile's weight rows, 256 * N * 2 bytes, stay within 32-bit offsets
  if (p.N > GG_MAX_DGRAD_N || p.K > GG_MAX_N) return GG_ERR_UNSUPPORTED;
  if (!is_aligned(p.dC, 16) || !is_aligned(p.B, 16) || !is_aligned(p.out, 16) ||
      !is_aligned(p.C, 16) || !is_aligned(p.H, 16))
    return GG_ERR_MISALIGNED;
  const int out_bytes = O == DOut::BF16 ? 2 : 4;  // of an element, or a pair of columns
  const Span dC = span(p.dC, p.M_cap, p.N, 2), B = span(p.B, (long long)p.E * p.K, p.N, 2),
             off = span(p.off, p.E + 1, 1, 4), out = span(p.out, p.M_cap, p.K, out_bytes),
             C = span(p.C, p.M_cap, p.K, 4), H = span(p.H, p.M_cap, p.K, 2);
  // (each tile's columns of C are read before it stores them: in place is safe)
  if (!apart(out, dC, B, off, H) || !apart(H, dC, B, off, C) || !(p.out == p.C || apart(out, C)))
    return GG_ERR_INVALID_VALUE;
  if (p.M_cap == 0) return GG_OK;
  int dev = 0;
  if (!current_device(&dev)) return GG_ERR_LAUNCH;
  const RingLaunch li = ring_launch<dgrad_kernel<O>>(dev, kDgradLds);
  if (li.err != hipSuccess) return GG_ERR_LAUNCH;
  return launch(dgrad_kernel<O>, dim3((unsigned)li.workgroups(tiles)), kThreads, kDgradLds, stream, p);
}

static DgradParams dgrad_params(const void *dC, const void *B, const int32_t *off, void *out,
                                int E, int K, int N, int M_cap, int bm) {
  return DgradParams{static_cast<const char *>(dC), static_cast<const char *>(B), off, out, nullptr,
                     nullptr, E, K, N, M_cap, bm, 0};
}

}  // namespace gg

using namespace gg;

extern "C" gg_status_t gg_grouped_gemm_bf16_dgrad(const void *dC, const void *B,
                                                  const int32_t *group_offsets, float *dA,
                                                  int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                                  int32_t bm, void *stream) {
  return dgrad<DOut::F32>(dgrad_params(dC, B, group_offsets, dA, E, K, N, M_cap, bm), stream);
}

extern "C" gg_status_t gg_grouped_gemm_bf16_dgrad_bf16out(const void *dC, const void *B,
                                                          const int32_t *group_offsets, void *dA,
                                                          int32_t E, int32_t K, int32_t N,
                                                          int32_t M_cap, int32_t bm,
                                                          void *stream) {
  return dgrad<DOut::BF16>(dgrad_params(dC, B, group_offsets, dA, E, K, N, M_cap, bm), stream);
}

extern "C" gg_status_t gg_grouped_gemm_bf16_dgrad_swiglu(const void *dY, const void *B,
                                                         const int32_t *group_offsets,
                                                         const void *C, void *dC, void *H,
                                                         int32_t E, int32_t K, int32_t N,
                                                         int32_t M_cap, int32_t bm,
                                                         void *stream) {
  DgradParams p = dgrad_params(dY, B, group_offsets, dC, E, K, N, M_cap, bm);
  p.C = static_cast<const uint16_t *>(C);
  p.H = static_cast<uint16_t *>(H);
  return dgrad<DOut::SwiGlu>(p, stream);
}
