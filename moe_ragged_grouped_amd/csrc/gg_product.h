// What the products on packed operands (gg_ring.h) write: fp32, bf16, or the
// bf16 SwiGLU of interleaved gate and up columns.
#pragma once

#include "gg_ring.h"

namespace gg {

enum class MOut { F32, BF16, SwiGlu };

__device__ __forceinline__ uint32_t swiglu_pair(f32x4 v) {
  const f32x2 h = {silu(v.x) * v.y, silu(v.z) * v.w};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(h, bf16x2));
}

// The epilogue of one tile; row0, col0: its first row and output column.
template <class C, MOut O>
struct ProductEpi {
  void *out;  // row 0, column 0
  int N;      // columns of the product
  int row0, col0, rows, ncols, wm0, wn0, lane;
  __device__ __forceinline__ void begin() {}
  __device__ __forceinline__ void block(const f32x4 (&acc)[C::NI][C::MI], int mi) {
    if constexpr (O != MOut::SwiGlu) {
      const size_t es = O == MOut::F32 ? 4 : 2;
      store_block<C, O == MOut::BF16>(acc, mi, (char *)out + ((size_t)row0 * N + col0) * es, wm0,
                                      wn0, lane, rows, ncols, N * es, col0 * es);
    } else {
      // two activations a block and lane (columns n, n + 1 and n + 2, n + 3):
      // one bf16 each, so a byte of output per column of the product
      const int g = lane / 16, s = lane % 16;
      const buf_rsrc r = row_block((char *)out + (size_t)row0 * N + col0, wm0 + mi * 16, rows,
                                   N, col0);
      const uint32_t row = (uint32_t)s * (uint32_t)N;
      if constexpr (C::NI % 4 == 0) {
        // lane groups trade so that group g holds all 8 activations of block g
#pragma unroll
        for (int ni = 0; ni < C::NI; ni += 4) {
          const auto a = __builtin_amdgcn_permlane16_swap(swiglu_pair(acc[ni][mi]),
                                                          swiglu_pair(acc[ni + 1][mi]), false, false);
          const auto b = __builtin_amdgcn_permlane16_swap(swiglu_pair(acc[ni + 2][mi]),
                                                          swiglu_pair(acc[ni + 3][mi]), false, false);
          const auto lo = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
          const int n = wn0 + (ni + g) * 16;
          st_buf16(r, n + 16 <= ncols ? row + n : kOob, u32x4{lo[0], hi[0], lo[1], hi[1]});
          // a last block of 8 columns
          if (ncols % 16 != 0) st_buf8(r, n + 8 == ncols ? row + n : kOob, u32x2{lo[0], hi[0]});
        }
      } else if constexpr (C::NI % 2 == 0) {
#pragma unroll
        for (int ni = 0; ni < C::NI; ni += 2) {
          const auto h = __builtin_amdgcn_permlane16_swap(swiglu_pair(acc[ni][mi]),
                                                          swiglu_pair(acc[ni + 1][mi]), false, false);
          const int n = wn0 + (ni + g % 2) * 16 + 8 * (g / 2);
          st_buf8(r, n < ncols ? row + n : kOob, u32x2{h[0], h[1]});
        }
      } else {
#pragma unroll
        for (int ni = 0; ni < C::NI; ++ni) {
          const int n = wn0 + ni * 16 + 4 * g;
          st_buf4(r, n < ncols ? row + n : kOob, swiglu_pair(acc[ni][mi]));
        }
      }
    }
  }
};

}  // namespace gg
