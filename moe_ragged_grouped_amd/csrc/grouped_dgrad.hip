// Data gradient of the ragged grouped product, for gfx950:
//
//   dA[r][k] = sum_n dC[r][n] * B[e][k][n]        for the rows r of expert e
//
// and the same sum with the backward of SwiGLU applied to it before it is
// stored. B keeps the forward product's layout [E][K][N]: its row k is
// contiguous along n, the index summed over here, and so is dC's row r. Both
// operands are read as they lie (gg_ring.h); nothing is transposed.
//
// One persistent launch walks the tiles of all experts in the order of
// gg_schedule.h, K in the place of the output columns.

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

// Tile heights as in gg_mainloop.h, eight waves, and the deepest ring that
// 160 KB of LDS hold.
using D16 = RingCfg<16, 128, 1, 8, 4, false>;
using D16M = RingCfg<16, 256, 1, 8, 4, false>;
using D16W = RingCfg<16, 512, 1, 8, 2, false>;
using D32 = RingCfg<32, 256, 1, 8, 4, false>;
using D64 = RingCfg<64, 256, 1, 8, 3, false>;
using D128 = RingCfg<128, 256, 2, 4, 3, false>;
using D256 = RingCfg<256, 256, 2, 4, 2, false>;

// sigmoid(x) with the hardware exp2 and reciprocal (each within one ulp); 0
// where e^-x overflows.
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float kLog2e = 1.4426950408889634f;
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xffff0000u);
}

template <class C, DOut O>
__device__ __forceinline__ void dgrad_tile(const DgradParams &p, const Tile &tl, lds_u8 *lds) {
  const int row0 = __builtin_amdgcn_readfirstlane(tl.row0);
  const int col0 = __builtin_amdgcn_readfirstlane(tl.col0);
  const int expert = __builtin_amdgcn_readfirstlane(tl.expert);
  RingTile t;
  t.pitch = 2u * (uint32_t)p.N;
  t.A = p.dC + (size_t)row0 * t.pitch;
  t.B = p.B + ((size_t)expert * p.K + col0) * t.pitch;
  t.As = t.Bs = nullptr;
  t.as_step = t.bs_step = 0;
  t.rows = __builtin_amdgcn_readfirstlane(tl.rows);
  t.ncols = min(C::BN, p.K - col0);
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // keep per-tile index arithmetic inside the tile
  t.tid = tid;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int wm0 = (wave / C::WN) * C::WTM, wn0 = (wave % C::WN) * C::WTN;
  const int g = lane / 16, s = lane % 16;
  const size_t K = p.K;
  f32x4 acc[C::NI][C::MI];
  auto epi = [&](int mi) {
    const int m = wm0 + mi * 16 + s;
    const size_t row = (size_t)(row0 + m);
    const bool in = m < t.rows;
    if constexpr (O == DOut::F32) {
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        const int n = wn0 + ni * 16 + 4 * g;
        if (in && n < t.ncols) st_g16((float *)p.out + row * K + col0 + n, acc[ni][mi]);
      }
    } else if constexpr (O == DOut::BF16) {
      if constexpr (C::NI % 2 == 0) {
#pragma unroll
        for (int ni = 0; ni < C::NI; ni += 2) {
          const u32x4 v = swap_pair(pack_bf16(acc[ni][mi]), pack_bf16(acc[ni + 1][mi]));
          const int n = wn0 + (ni + g % 2) * 16 + 8 * (g / 2);
          if (in && n < t.ncols) st_g16u((uint16_t *)p.out + row * K + col0 + n, v);
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni) {
          const int n = wn0 + ni * 16 + 4 * g;
          if (in && n < t.ncols)
            st_g8u((uint16_t *)p.out + row * K + col0 + n, pack_bf16(acc[ni][mi]));
        }
      }
    } else {
      // dH = acc; with sg = sigmoid(gate):
      //   d gate = dH * up * sg * (1 + gate * (1 - sg)),  d up = dH * gate * sg,
      //   H = gate * sg * up
      u32x2 h[C::NI];
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        const int n = wn0 + ni * 16 + 4 * g;
        u32x4 c = {0, 0, 0, 0}, d;
        const size_t at = 2 * (row * K + col0 + n);
        if (in && n < t.ncols) c = *(const gbl_u32x4 *)(p.C + at);
        f32x4 hv;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gate = lo_bf16(c[j]), up = hi_bf16(c[j]);
          const float sg = sigmoid(gate), dh = acc[ni][mi][j];
          const float act = gate * sg;
          const f32x2 dv = {dh * up * (sg * (1.0f + gate * (1.0f - sg))), dh * act};
          d[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(dv, bf16x2));
          hv[j] = act * up;
        }
        if (in && n < t.ncols) st_g16u((uint16_t *)p.out + at, d);
        h[ni] = pack_bf16(hv);
      }
      if (p.H != nullptr) {
        if constexpr (C::NI % 2 == 0) {
#pragma unroll
          for (int ni = 0; ni < C::NI; ni += 2) {
            const u32x4 v = swap_pair(h[ni], h[ni + 1]);
            const int n = wn0 + (ni + g % 2) * 16 + 8 * (g / 2);
            if (in && n < t.ncols) st_g16u(p.H + row * K + col0 + n, v);
          }
        } else {
          const int n = wn0 + 4 * g;
          if (in && n < t.ncols) st_g8u(p.H + row * K + col0 + n, h[0]);
        }
      }
    }
  };
  run_ring_tile<C, kCacheStream>(t, lds, acc, 0, epi);
}

template <int MASK>
constexpr int dgrad_lds() {
  int m = 0;
  const int b[] = {D16::LDS_BYTES, D16M::LDS_BYTES, D16W::LDS_BYTES};
  if (MASK & 1)
    for (int v : b) m = m > v ? m : v;
  if (MASK & 2) m = m > D32::LDS_BYTES ? m : D32::LDS_BYTES;
  if (MASK & 4) m = m > D64::LDS_BYTES ? m : D64::LDS_BYTES;
  if (MASK & 8) m = m > D128::LDS_BYTES ? m : D128::LDS_BYTES;
  if (MASK & 16) m = m > D256::LDS_BYTES ? m : D256::LDS_BYTES;
  return m;
}

// MASK bit c compiles in tile height 16 << c.
template <int MASK, DOut O>
__global__ __launch_bounds__(kThreads, 1) void dgrad_kernel(DgradParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_dyn[];
  lds_u8 *const lds = (lds_u8 *)lds_dyn;
  RingSched &sched = *(RingSched *)(lds_dyn + dgrad_lds<MASK>());
  const int G = gridDim.x, b = blockIdx.x;
  const int total = build_ring_schedule(sched, p.off, p.E, p.M_cap, p.K, p.bm_fixed, p.tile_cap, G);
  // contiguous tiles on one XCD (workgroup ids go round-robin to the XCDs)
  const int slot = (b % kRingXcds) * (G / kRingXcds) + b / kRingXcds;
  for (int base = 0; base < total; base += G) {
    const int t = base + slot;
    if (t >= total) break;
    const Tile tl = decode_ring_tile(sched, p.off, t, p.E, p.M_cap, p.K, p.bm_fixed);
    switch (tl.bm) {
      case 16:
        if constexpr (MASK & 1) {
          if (tl.bn == kWideN) dgrad_tile<D16W, O>(p, tl, lds);
          else if (tl.bn == kTileN) dgrad_tile<D16M, O>(p, tl, lds);
          else dgrad_tile<D16, O>(p, tl, lds);
        }
        break;
      case 32: if constexpr (MASK & 2) dgrad_tile<D32, O>(p, tl, lds); break;
      case 64: if constexpr (MASK & 4) dgrad_tile<D64, O>(p, tl, lds); break;
      case 128: if constexpr (MASK & 8) dgrad_tile<D128, O>(p, tl, lds); break;
      default: if constexpr (MASK & 16) dgrad_tile<D256, O>(p, tl, lds); break;
    }
  }
}

static_assert(dgrad_lds<31>() + sizeof(RingSched) <= 160 * 1024, "LDS budget");

template <int MASK, DOut O>
static gg_status_t launch_dgrad(const DgradParams &p, long long bound, hipStream_t stream) {
  constexpr int lds = dgrad_lds<MASK>() + (int)sizeof(RingSched);
  int dev = 0;
  if (!current_device(&dev)) return GG_ERR_LAUNCH;
  const RingLaunch li = ring_launch<dgrad_kernel<MASK, O>>(dev, lds);
  if (li.err != hipSuccess) return GG_ERR_LAUNCH;
  long long g = bound < li.grid ? bound : li.grid;
  g = (g + kRingXcds - 1) / kRingXcds * kRingXcds;
  hipLaunchKernelGGL((dgrad_kernel<MASK, O>), dim3((unsigned)g), dim3(kThreads), lds, stream, p);
  return hipGetLastError() == hipSuccess ? GG_OK : GG_ERR_LAUNCH;
}

template <DOut O>
static gg_status_t dgrad(DgradParams p, void *stream) {
  long long bound = 0;
  gg_status_t st = check_groups(p.off, p.E, p.K, p.M_cap, p.bm_fixed, kNarrowN, &bound);
  if (st != GG_OK) return st;
  if (p.B == nullptr || p.N < 1) return GG_ERR_INVALID_VALUE;
  // arrays of no rows may be null
  if (p.M_cap > 0 && (p.dC == nullptr || p.out == nullptr || (O == DOut::SwiGlu && p.C == nullptr)))
    return GG_ERR_INVALID_VALUE;
  if (p.K % 8 != 0 || p.N % 8 != 0) return GG_ERR_MISALIGNED;
  // a tile's weight rows, 512 * N * 2 bytes, stay within 32-bit offsets
  if (p.N > GG_MAX_DGRAD_N || p.K > GG_MAX_N) return GG_ERR_UNSUPPORTED;
  if (!is_aligned(p.dC, 16) || !is_aligned(p.B, 16) || !is_aligned(p.out, 16) ||
      !is_aligned(p.C, 16) || !is_aligned(p.H, 16))
    return GG_ERR_MISALIGNED;
  if (p.M_cap == 0) return GG_OK;
  p.tile_cap = (int)bound;
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (p.bm_fixed) {
    case 16: return launch_dgrad<1, O>(p, bound, s);
    case 32: return launch_dgrad<2, O>(p, bound, s);
    case 64: return launch_dgrad<4, O>(p, bound, s);
    case 128: return launch_dgrad<8, O>(p, bound, s);
    case 256: return launch_dgrad<16, O>(p, bound, s);
    default: return launch_dgrad<31, O>(p, bound, s);
  }
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
