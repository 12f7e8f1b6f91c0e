// A ring of LDS stages filled straight from global memory, and the products
// of one output tile out of it, for operands whose contraction index is the
// fastest in memory:
//
//   C[m][n] = sum_l A[m][l] * W[n][l]
//
// The data gradient (A = dC, W = B[e] with its K rows, l = the product's
// columns) and the 4-bit and block-scaled 8-bit products (both operands packed
// along K) have this form. Both operands then look alike in bytes: a row of a
// slice is 128 bytes, 64 bf16, 128 8-bit or 256 4-bit values, and one 16-byte
// piece of a row is what a lane feeds to one matrix instruction (two in 8 bits).
//
// MI355X mapping:
//  * buffer_load_dwordx4 ... lds moves 16 bytes a lane from global memory into
//    LDS without passing through registers: no staging registers beside the
//    accumulators, no ds_write (which costs 8 LDS cycles an instruction), and
//    as many slices in flight as LDS has room for. A lane out of the buffer's
//    range writes zeros (checked by an in-bounds probe), which is the zero
//    fill of padding rows, of columns past the end and of the last slice's
//    tail. Measured alone (8 x 1 KB a wave, two 64 KB groups in flight): 148
//    bytes a ns and CU out of L2, 88 streaming on a quarter of the CUs, 6.1
//    TB/s streaming on all; the swizzle below and the row pitch cost nothing,
//    but a pitch that is no multiple of 128 makes every row's piece touch two
//    lines.
//  * The instruction writes lane l's 16 bytes at base + 16 l, so a swizzle has
//    to be put into the global side: lane l of a wave's 8 x 128-byte piece
//    loads row l / 8, chunk (l % 8) ^ (l / 8), and chunk c of row r then sits
//    at chunk c ^ (r % 8). A fragment read (ds_read_b128, 16 rows) touches
//    every bank once.
//  * S stages, one barrier a slice: the barrier that says "slice i has landed"
//    also says "every wave is done with slice i - 1", whose stage is refilled
//    at once with slice i + S - 1.
//  * A persistent workgroup starts the next tile's first slices as soon as its
//    last LDS read is done, before it stores the present tile.
#pragma once

#include "gg_common.h"
#include "gg_schedule.h"

namespace gg {

typedef __attribute__((ext_vector_type(8))) int ring_i32x8;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) u32x4 gbl_u32x4;
typedef __attribute__((address_space(1))) u32x2 gbl_u32x2;

__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// What a slice holds beside its 128-byte rows.
constexpr int kRowsBf16 = 0;  // nothing
constexpr int kRowsMx4 = 1;   // 8 scale bytes a row, one for 32 values
constexpr int kRowsFp8 = 2;   // one fp32 scale a row of A (that of 128 columns is a scalar)

// 16 bytes a lane, global -> LDS at dst + 16 * lane (dst is wave-uniform).
template <int POLICY = kCacheDefault>
__device__ __forceinline__ void dma16(buf_rsrc r, lds_u8 *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, voff, 0, 0, POLICY);
}

// The same with 4 bytes a lane.
__device__ __forceinline__ void dma4(buf_rsrc r, lds_u8 *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 4, voff, 0, 0, kCacheDefault);
}

// This wave's loads have landed up to the N youngest ones, and its LDS reads
// are done. The compiler moves no memory access across it; it does not count
// the loads into LDS itself, as no register waits on them.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt has 6 bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// The same, with the loads of `younger` slices (at most Y) left in flight.
template <class C, int Y = C::S - 2>
__device__ __forceinline__ void wait_slices(int younger) {
  if constexpr (Y == 0) {
    wait_loads<0>();
  } else {
    if (younger >= Y) wait_loads<Y * C::LPS>();
    else wait_slices<C, Y - 1>(younger);
  }
}

__device__ __forceinline__ void wg_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- schedule
//
// Row tiles per expert by adaptive_bm (or the caller's height), as in
// gg_schedule.h, with three changes.
//
// Height: where even the narrowest tiles leave more than half of the G
// workgroups idle, no tile is taller than the tallest halved (to 32 at the
// least) as often as twice as many tiles still fit. (An estimate: one tall
// expert among low ones is counted as if all tiles doubled, and may keep its
// height although lowering it alone would fit.) A tile's slices come one
// after the other, and the fewer bytes each has the sooner it is done.
// Measured (us, without / with): data gradient, one expert of 618 rows, K = 1200,
// N = 216 with SwiGLU, 11.8 / 9.4; of 1000 rows, K = 512, N = 2048, 23.7 / 16.0;
// 4-bit product, one of 8209 rows, K = 5952, N = 88, 26.4 / 22.1. 8-bit product: 618
// rows, K = 1200, N = 216, 14.1 / 11.2; 8209 rows, K = 5952, N = 88, 42.1 / 28.9.
//
// Width: one for the launch. A launch of few tiles leaves CUs idle, and
// narrower tiles then finish sooner although they fetch A more often. With
// T(w) tiles of width w on G workgroups and H the tallest height, the width is
// the one with the smallest
//   ceil(T(w) / G) * (H + w + 96),
// rounds times the bytes of a slice plus a fixed share for what a tile repeats
// whatever its size; the wider one at a tie. (On the 8-bit product, against one
// width for every launch, 22 shapes of 1 to 128 experts and 8 to 16384 rows: the width
// taken is within 4% of the best of the three on 21 and as often far ahead of the other
// two; 32 x 16 rows, K = 1024, N = 2688 takes 25.9 us, with 256 columns 22.8.)
//
// Order: where a workgroup gets several tiles of different heights, experts
// with tall tiles come first (by index among equals), so that the tiles of a
// round cost about the same and the last round holds the small ones. Measured
// on 16,384 rows routed by rank^-1.2 to 64 experts, K = 1344, N = 1024, replayed
// in a graph on one set of inputs (which stays in the caches in part): data
// gradient 90.0 -> 82.7 us in bf16, 134 -> 113 with the SwiGLU gradient, which
// takes 118 - 122 on inputs that change. Launches of one height keep the order
// of the experts, which costs 1.5 us less.
struct RingSched {
  int start[kMaxExperts];  // first row tile of an expert; INT_MAX if it has none
  int wave_tiles[kNumHeights][kThreads / kWave];
  int wave_tallest[kThreads / kWave];
};

constexpr int kNarrowestN = 64;

struct RingGrid {
  int total;  // tiles of the launch
  int width;  // columns of each
  int most;   // rows of one at most
};

// Lanes shifted or broadcast up a wave by DPP (row = 16 lanes), which takes no
// trip through LDS as a shuffle does. Lanes without a source, and rows outside
// ROWS, get `none`.
constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int lanes_up(int v, int none) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}

// Inclusive sum over the lanes of a wave, saturating at `most`.
__device__ __forceinline__ int wave_scan(int v, int most) {
  v = min(v + lanes_up<kRowShr1>(v, 0), most);
  v = min(v + lanes_up<kRowShr2>(v, 0), most);
  v = min(v + lanes_up<kRowShr4>(v, 0), most);
  v = min(v + lanes_up<kRowShr8>(v, 0), most);
  v = min(v + lanes_up<kRowBcast15, 0xa>(v, 0), most);  // lane 15 to row 1, lane 47 to row 3
  return min(v + lanes_up<kRowBcast31, 0xc>(v, 0), most);  // lane 31 to rows 2 and 3
}

// The largest value of a wave, wave-uniform.
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, lanes_up<kRowShr1>(v, v));
  v = max(v, lanes_up<kRowShr2>(v, v));
  v = max(v, lanes_up<kRowShr4>(v, v));
  v = max(v, lanes_up<kRowShr8>(v, v));
  v = max(v, lanes_up<kRowBcast15, 0xa>(v, v));
  v = max(v, lanes_up<kRowBcast31, 0xc>(v, v));
  return __builtin_amdgcn_readlane(v, kWave - 1);
}

// Tiles of a power-of-two height in `rows` rows (at most 2^31 - 257).
__device__ __forceinline__ int row_tiles(int rows, int height) {
  return (rows + height - 1) >> __builtin_ctz(height);
}

// All threads of the workgroup must call this. tile_cap: the host's bound of
// row tiles; overlapping (malformed) groups that exceed it schedule nothing.
__device__ __forceinline__ RingGrid build_ring_schedule(RingSched &s,
                                                        const int32_t *__restrict__ off_g, int E,
                                                        int M_cap, int N, int bm_fixed,
                                                        int tile_cap, int G) {
  const int tid = threadIdx.x;
  constexpr int kRun = kMaxExperts / kThreads, kWaves = kThreads / kWave;
  const int e0 = tid * kRun;
  int rows[kRun], cnt[kRun], height[kRun], tallest = 16;
  int lo = e0 < E ? clamp_off(off_g, e0, M_cap) : 0;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const int e = e0 + j;
    rows[j] = 0;
    height[j] = 16;
    if (e < E) {
      const int hi = clamp_off(off_g, e + 1, M_cap);
      rows[j] = max(hi - lo, 0);
      height[j] = bm_fixed ? bm_fixed : adaptive_bm(rows[j]);
      if (rows[j] > 0) tallest = max(tallest, height[j]);
      lo = hi;
    }
  }
  // A group counts at most 2^27 row tiles and tile_cap is at most 2^28, so
  // sums that saturate at 2^29 (malformed offsets only) are over the cap.
  constexpr int kMost = 1 << 29;
  const int lane = tid % kWave, wave = tid / kWave;
  tallest = wave_max(tallest);
  int local = 0, incl = 0, before = 0, total = 0;
  for (bool again = bm_fixed == 0;; again = false) {
    local = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      height[j] = min(height[j], tallest);  // (the second time; `tallest` is this wave's the first)
      cnt[j] = row_tiles(rows[j], height[j]);
      local += cnt[j];
    }
    incl = wave_scan(local, kMost);
    if (lane == kWave - 1) {
      s.wave_tiles[0][wave] = incl;
      s.wave_tallest[wave] = tallest;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) before = min(before + s.wave_tiles[0][w], kMost);
      total = min(total + s.wave_tiles[0][w], kMost);
      tallest = max(tallest, s.wave_tallest[w]);
    }
    tallest = scalar(tallest);
    total = scalar(total > tile_cap ? 0 : total);
    const int narrow = total * cdiv(N, kNarrowestN);  // (at most 2^30, by the host's bound)
    if (!again || tallest <= 32 || narrow > G / 2) break;
    // a height's half at most doubles the tiles
    for (int n = 2 * narrow; tallest > 32 && n <= G; n *= 2) tallest /= 2;
    __syncthreads();  // wave_tiles is written again
  }
  int width = kTileN;
  unsigned long long best_cost = 0;
#pragma unroll
  for (int w = kTileN; w >= kNarrowestN; w /= 2) {
    if (w < 128 && tallest == 16) break;  // eight waves side by side, 16 columns each
    const uint32_t rounds = ((uint32_t)(total * cdiv(N, w)) + G - 1) / (uint32_t)G;
    const unsigned long long cost = (unsigned long long)rounds * (uint32_t)(tallest + w + 96);
    if (w == kTileN || cost < best_cost) { width = w; best_cost = cost; }
  }
  width = scalar(width);
  const int tiles = total * cdiv(N, width);
  int first[kRun];
  if (tiles <= G || tallest == 16 || bm_fixed != 0) {  // one round or one height: expert order
    int run = min(before + incl, kMost) - local;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      first[j] = run;
      run += cnt[j];
    }
  } else {
    __syncthreads();  // wave_tiles is written again
    int at[kNumHeights];  // this thread's place among the tiles of a height
#pragma unroll
    for (int c = 0; c < kNumHeights; ++c) {
      int mine = 0;
#pragma unroll
      for (int j = 0; j < kRun; ++j) mine += height[j] == height_of(c) ? cnt[j] : 0;
      const int sum = wave_scan(mine, kMost);
      at[c] = sum - mine;
      if (lane == kWave - 1) s.wave_tiles[c][wave] = sum;
    }
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int c = kNumHeights - 1; c >= 0; --c) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w == wave) at[c] += base;
        base += s.wave_tiles[c][w];
      }
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      first[j] = 0;
#pragma unroll
      for (int c = 0; c < kNumHeights; ++c)
        if (height[j] == height_of(c)) {
          first[j] = at[c];
          at[c] += cnt[j];
        }
    }
  }
#pragma unroll
  for (int j = 0; j < kRun; ++j)
    if (e0 + j < E) s.start[e0 + j] = cnt[j] > 0 ? first[j] : INT32_MAX;
  __syncthreads();
  return RingGrid{tiles, width, tallest};
}

// A device offset through the scalar cache: its wait does not count against
// the loads and stores in flight.
typedef __attribute__((address_space(4))) const int32_t cst_i32;
typedef __attribute__((address_space(4))) const float cst_f32;
__device__ __forceinline__ int clamp_off_s(const int32_t *off_g, int e, int M_cap) {
  const int v = ((cst_i32 *)off_g)[e];
  return min(max(v, 0), M_cap);
}

// Tile t of the list (0 <= t < total), wave-uniform.
__device__ __forceinline__ Tile decode_ring_tile(const RingSched &s, const int32_t *off_g, int t,
                                                 int E, int M_cap, int N, int bm_fixed,
                                                 const RingGrid &grid) {
  const int bn = grid.width;
  const int NT = cdiv(N, bn);
  const int m_index = t / NT;  // an expert's row tiles lie together, NT tiles each
  // the expert with the last start at or before m_index
  const int lane = threadIdx.x % kWave;
  int best = -1, mine = 0;
  for (int e = lane; e < E; e += kWave) {
    const int at = s.start[e];
    if (at <= m_index && at > best) { best = at; mine = e; }
  }
  const int top = wave_max(best);
  const unsigned long long has = __ballot(best == top);
  const int lo = __builtin_amdgcn_readlane(mine, __ffsll((long long)has) - 1);
    const int r0 = clamp_off_s(off_g, lo, M_cap);
  const int m = clamp_off_s(off_g, lo + 1, M_cap) - r0;
  const int b = bm_fixed ? bm_fixed : min(adaptive_bm(m), grid.most);
  const int n_mt = row_tiles(m, b);
  const int local = t - top * NT;
  // groups of kGroupM M tiles; N outer, M inner inside a group
  const int per_group = kGroupM * NT;
  const int grp = local / per_group;
  const int r = local - grp * per_group;
  const int gm = min(kGroupM, n_mt - grp * kGroupM);
  const int nt = r / gm;
  const int mt = grp * kGroupM + (r - nt * gm);
  Tile tl;
  tl.expert = lo;
  // eight waves of 16 columns each do not fit 64: 32 rows, half of them padding
  tl.bm = bn == 64 ? max(b, 32) : b;
  tl.bn = bn;
  tl.row0 = r0 + mt * b;
  tl.rows = min(b, m - mt * b);
  tl.col0 = nt * bn;
  return tl;
}

// ------------------------------------------------------------------- tiles

constexpr int kRowBytes = 128;  // bytes of a row in one slice
constexpr int kRingBytes = 155 * 1024;  // LDS for the stages (the schedule takes 4.2 KB more)

// Bytes of a stage: A's rows, B's rows, then the scales: in 4 bits 8 bytes per
// row of A and of B; in 8 bits 4 bytes per row of A, up to a whole row, as stages
// start on one.
__host__ __device__ constexpr int ring_stage(int BM, int BN, int F) {
  return (BM + BN) * (kRowBytes + (F == kRowsMx4 ? 8 : 0)) +
         (F == kRowsFp8 ? (BM * 4 + kRowBytes - 1) / kRowBytes * kRowBytes : 0);
}
// As many stages as fit, up to 6 (96 KB and more in flight).
__host__ __device__ constexpr int ring_stages(int BM, int BN, int F) {
  const int s = kRingBytes / ring_stage(BM, BN, F);
  return s < 6 ? s : 6;
}

template <int BM_, int BN_, int WM_, int WN_, int F_>
struct RingCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, F = F_;
  static constexpr bool MX = F == kRowsMx4, FP8 = F == kRowsFp8;
  static_assert(WM * WN == kThreads / kWave, "one wave per wave tile");
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static_assert(WTM % 16 == 0 && WTN % 16 == 0, "16x16 blocks");
  static constexpr int MI = WTM / 16, NI = WTN / 16;
  static constexpr int A_BYTES = BM * kRowBytes, B_BYTES = BN * kRowBytes;
  static constexpr int STAGE = ring_stage(BM, BN, F), S = ring_stages(BM, BN, F);
  // loads a wave issues per slice: of A (8 bits: and its scales), and of the
  // weights (4 bits: and all scales)
  static constexpr int NA = (BM >= 64 ? BM / 64 : 1) + (FP8 ? 1 : 0), NB = BN / 64 + (MX ? 1 : 0),
                       LPS = NA + NB;
  // Two stages are all that the tallest tile leaves room for, and one slice
  // ahead is too little for weights that come from HBM (measured: 2.3 us a
  // slice against 1.5 for its products alone). But a wave takes all column
  // fragments and scales of a slice into registers before its second row
  // block, so the weights' half of the stage is free almost a slice early and
  // is refilled two slices ahead; A, which the tiles of a row block share, is
  // mostly in L2.
  static constexpr bool EARLY_B = S == 2;
  static_assert(S >= 2 && (S - 2) * LPS < 64, "loads in flight");
  static_assert(S * STAGE <= kRingBytes, "LDS");
};

struct RingTile {
  const char *A;          // row 0 of the tile
  const char *B;          // weight row (output column) 0 of the tile
  const char *As, *Bs;    // scales of the first slice, row 0 / column 0
  // bytes from a slice's scales to the next one's (8 bits: from a column block's to
  // the next one's)
  uint64_t as_step, bs_step;
  uint32_t pitch;         // bytes of a row of A and of B
  int rows, ncols;        // valid rows and columns
};

// Rows of a tile of fewer than 64: BM / 8 of them a wave, on its first BM
// lanes, so that every wave issues the same number of loads and waits on the
// same count. left: bytes of a row from this slice on.
__device__ __forceinline__ void ring_short_rows(buf_rsrc ra, int BM, lds_u8 *stage, uint32_t pitch,
                                                uint32_t left, int wave, int lane) {
  const int r = wave * (BM / 8), lr = lane / 8;
  const uint32_t c = 16u * ((lane % 8) ^ ((r + lr) % 8));
  if (lane < BM)
    dma16(ra, stage + r * kRowBytes, c < left ? (uint32_t)(r + lr) * pitch + c : kOob);
}

// Scale bytes: 16, two rows' worth, a lane; waves 0-3 take A's, waves 4-7 B's.
__device__ __forceinline__ buf_rsrc ring_scales(const RingTile &t, int k, int wave) {
  const uint64_t as = (uint64_t)t.As + (uint64_t)k * t.as_step;
  const uint64_t bs = (uint64_t)t.Bs + (uint64_t)k * t.bs_step;
  const int rows = t.rows, ncols = t.ncols;
  return make_buf((const void *)(wave >= 4 ? bs : as), 8u * (uint32_t)(wave >= 4 ? ncols : rows));
}
__device__ __forceinline__ void ring_scale_rows(buf_rsrc rs, int BM, int BN, lds_u8 *stage, int wave,
                                                int lane) {
  const bool is_b = wave >= 4;
  const int n = is_b ? BN / 8 : BM / 8;  // lanes of this wave
  const int at = 16 * (wave % 4) * n;
  lds_u8 *const dst = stage + (BM + BN) * kRowBytes + (is_b ? BM * 8 : 0) + at;
  if (lane < n) dma16(rs, dst, (uint32_t)(at + 16 * lane));
}

// fp32 scales of A, a row to a lane, BM / 8 rows a wave.
__device__ __forceinline__ void ring_row_scales(const RingTile &t, int BM, int BN, lds_u8 *stage, int k,
                                                int wave, int lane) {
  const buf_rsrc rs = make_buf(t.As + (uint64_t)k * t.as_step, 4u * (uint32_t)t.rows);
  // (a wave's place is worked out where it is used: kept over the loop it would
  // cost a scalar that the loop does not have)
  asm volatile("" : "+s"(wave));
  const int n = BM / 8, at = wave * n;
  if (lane < n) dma4(rs, stage + (BM + BN) * kRowBytes + 4 * at, 4u * (uint32_t)(at + lane));
}

// This wave's loads of slice k of a BM x BN tile into one stage, a group of 8
// rows to a load: of A, and of the weights with all scales.
//
// Weights are loaded as streaming data (nt) where each row's piece is whole
// lines: each weight byte feeds the few tiles of one column slice, which run
// side by side. Measured on 64 x 256 rows, K = 1024, N = 2688: 111 -> 98 us.
// Where pieces straddle lines, nt drops the line whose other half the next
// slice needs: 12 x 65 rows, K = 712, N = 1000: 17.0 us without, 20.4 with.
__device__ __forceinline__ uint32_t ring_row_off(const RingTile &t, int r, int k, int lane) {
  const int lr = lane / 8;
  const uint32_t chunk = 16u * ((lane % 8) ^ lr);
  // a chunk past the row's end is out of range, as are rows past the last
  return chunk < t.pitch - (uint32_t)k * kRowBytes ? (uint32_t)(r + lr) * t.pitch + chunk : kOob;
}
__device__ __forceinline__ buf_rsrc ring_rows(const char *base, int rows, const RingTile &t, int k) {
  const uint32_t k0 = (uint32_t)k * kRowBytes;
  return make_buf(base + k0, (uint32_t)rows * t.pitch - k0);
}
__device__ __forceinline__ void ring_load_a(const RingTile &t, buf_rsrc ra, int BM, lds_u8 *stage,
                                            int i, int k, int wave, int lane) {
  const int r = (i * 8 + wave) * 8;
  if (BM >= 64) dma16(ra, stage + r * kRowBytes, ring_row_off(t, r, k, lane));
  else ring_short_rows(ra, BM, stage, t.pitch, t.pitch - (uint32_t)k * kRowBytes, wave, lane);
}
__device__ __forceinline__ void ring_load_b(const RingTile &t, buf_rsrc rb, int BM, lds_u8 *stage,
                                            int i, int k, int wave, int lane) {
  const int r = (i * 8 + wave) * 8;
  lds_u8 *const dst = stage + (BM + r) * kRowBytes;
  if (t.pitch % kRowBytes == 0) dma16<kCacheStream>(rb, dst, ring_row_off(t, r, k, lane));
  else dma16(rb, dst, ring_row_off(t, r, k, lane));
}
template <int F>
__device__ __forceinline__ void ring_issue_a(const RingTile &t, int BM, int BN, lds_u8 *stage, int k,
                                             int wave, int lane) {
  const buf_rsrc ra = ring_rows(t.A, t.rows, t, k);
  const int n = BM >= 64 ? BM / 64 : 1;
#pragma unroll 1
  for (int i = 0; i < n; ++i) ring_load_a(t, ra, BM, stage, i, k, wave, lane);
  if constexpr (F == kRowsFp8) ring_row_scales(t, BM, BN, stage, k, wave, lane);
}
template <int F>
__device__ __forceinline__ void ring_issue_b(const RingTile &t, int BM, int BN, lds_u8 *stage, int k,
                                             int wave, int lane) {
  const buf_rsrc rb = ring_rows(t.B, t.ncols, t, k);
#pragma unroll 1
  for (int i = 0; i < BN / 64; ++i) ring_load_b(t, rb, BM, stage, i, k, wave, lane);
  if constexpr (F == kRowsMx4) ring_scale_rows(ring_scales(t, k, wave), BM, BN, stage, wave, lane);
}

// The same loads as pieces, to be issued between matrix instructions: a CU's
// memory pipeline stays full, so a wave that issues its loads in a row blocks
// on them before it multiplies. A of slice ka into stage sa (pieces 0 .. NA -
// 1), weights and scales of slice kb into stage sb (the rest).
template <class C>
struct RingPieces {
  const RingTile &t;
  buf_rsrc ra, rb, rs;
  lds_u8 *sa, *sb;
  int ka, kb, KT, wave, lane;

  __device__ __forceinline__ RingPieces(const RingTile &t_, lds_u8 *sa_, int ka_, lds_u8 *sb_, int kb_,
                                        int KT_, int wave_, int lane_)
      : t(t_), sa(sa_), sb(sb_), ka(ka_), kb(kb_), KT(KT_), wave(wave_), lane(lane_) {
    ra = ring_rows(t.A, t.rows, t, ka);
    rb = ring_rows(t.B, t.ncols, t, kb);
    if constexpr (C::MX) rs = ring_scales(t, kb, wave);
  }
  template <int J>
  __device__ __forceinline__ void issue() const {
    if constexpr (C::FP8 && J == C::NA - 1) {
      if (ka < KT) ring_row_scales(t, C::BM, C::BN, sa, ka, wave, lane);
    } else if constexpr (J < C::NA) {
      if (ka < KT) ring_load_a(t, ra, C::BM, sa, J, ka, wave, lane);
    } else if constexpr (J < C::NA + C::BN / 64) {
      if (kb < KT) ring_load_b(t, rb, C::BM, sb, J - C::NA, kb, wave, lane);
    } else {
      if (kb < KT) ring_scale_rows(rs, C::BM, C::BN, sb, wave, lane);
    }
  }
};

__device__ __forceinline__ int ring_slices(const RingTile &t) {
  return (int)((t.pitch + kRowBytes - 1) / kRowBytes);
}

// The first slices of a tile, as many as the ring takes ahead of the products.
template <int F>
__device__ __forceinline__ void ring_prologue(const RingTile &t, int BM, int BN, lds_u8 *lds,
                                              int wave, int lane) {
  const int n = min(ring_stages(BM, BN, F) - 1, ring_slices(t)), bytes = ring_stage(BM, BN, F);
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    ring_issue_a<F>(t, BM, BN, lds + k * bytes, k, wave, lane);
    ring_issue_b<F>(t, BM, BN, lds + k * bytes, k, wave, lane);
  }
  if (ring_stages(BM, BN, F) == 2 && ring_slices(t) > 1)  // EARLY_B
    ring_issue_b<F>(t, BM, BN, lds + bytes, 1, wave, lane);
}

// The products of one slice. Two matrix steps; lane group g takes 16-byte
// chunk 4 ks + g of a row (bf16: l = 32 ks + 8 g ..) or 2 g + ks (4-bit: block
// 2 g + ks of 32 values, so that a lane's two scale bytes are neighbours; the
// matrix cores pair lane group with lane group, so any order that both
// operands share is the same sum). A row block's fragment is read two blocks
// ahead of its products and the second step's column fragments during the
// first step, so that the matrix cores do not wait on LDS inside a slice.
// mid(mi) runs after row block mi of the first step, blk(mi) after row block
// mi's last product.
template <class C, class Mid, class Blk>
__device__ __forceinline__ void ring_mma(f32x4 (&acc)[C::NI][C::MI], const lds_u8 *a_stage,
                                         const lds_u8 *b_stage, int wm0, int wn0, int lane,
                                         int blocks_left, Mid &&mid, Blk &&blk) {
  const int g = lane / 16, s = lane % 16;
  const lds_u8 *const ar = a_stage + (wm0 + s) * kRowBytes;
  const lds_u8 *const br = b_stage + C::A_BYTES + (wn0 + s) * kRowBytes;
  int sa[C::MX ? C::MI : 1], sb[C::MX ? C::NI : 1];
  const int c0 = 16 * ((C::MX ? 2 * g : g) ^ (s & 7));
  const int c1 = 16 * ((C::MX ? 2 * g + 1 : 4 + g) ^ (s & 7));
  u32x4 x[2][C::NI], y[3];
  auto read_x = [&](auto ks) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
      x[ks][ni] = *(const lds_u32x4 *)(br + ni * 16 * kRowBytes + (ks ? c1 : c0));
  };
  auto read_y = [&](auto bc) {  // block b % MI of step b / MI
    constexpr int b = decltype(bc)::value;
    if constexpr (b < 2 * C::MI)
      y[b % 3] = *(const lds_u32x4 *)(ar + b % C::MI * 16 * kRowBytes + (b / C::MI ? c1 : c0));
  };
  read_x(std::integral_constant<int, 0>{});
  read_y(std::integral_constant<int, 0>{});
  if constexpr (C::MX) {
    // scale bytes past the row's last block are whatever memory holds there;
    // a zero byte (2^-127) times the zero values loaded there is zero
    const int v = blocks_left - 2 * g;
    const int mask = v >= 2 ? 0xffff : (v == 1 ? 0xff : 0);
    const lds_u8 *const sc = b_stage + C::A_BYTES + C::B_BYTES + 2 * g;
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
      sb[ni] = mask & *(const lds_u16 *)(sc + C::BM * 8 + 8 * (wn0 + ni * 16 + s));
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
      sa[mi] = mask & *(const lds_u16 *)(sc + 8 * (wm0 + mi * 16 + s));
  }
  read_y(std::integral_constant<int, 1>{});
  static_for<2 * C::MI>([&](auto bc) {
    constexpr int b = decltype(bc)::value, ks = b / C::MI, mi = b % C::MI;
    read_y(std::integral_constant<int, b + 2>{});
    // (early where the weights' half of the stage is to be freed)
    if constexpr (b == (C::EARLY_B || C::MI < 2 ? 0 : C::MI - 2)) read_x(std::integral_constant<int, 1>{});
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) {
      if constexpr (C::MX) {
        // formats 4, 4 = E2M1; a 4-bit operand is the low half of the eight
        // registers, scale byte ks of each lane's scale register
        const ring_i32x8 xv = __builtin_bit_cast(
            ring_i32x8, __builtin_shufflevector(x[ks][ni], x[ks][ni], 0, 1, 2, 3, -1, -1, -1, -1));
        const ring_i32x8 yv = __builtin_bit_cast(
            ring_i32x8, __builtin_shufflevector(y[b % 3], y[b % 3], 0, 1, 2, 3, -1, -1, -1, -1));
        acc[ni][mi] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xv, yv, acc[ni][mi], 4, 4, ks,
                                                                       sb[ni], ks, sa[mi]);
      } else {
        acc[ni][mi] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, x[ks][ni]), __builtin_bit_cast(bf16x8, y[b % 3]),
            acc[ni][mi], 0, 0, 0);
      }
    }
    if constexpr (ks == 0) mid(std::integral_constant<int, mi>{});
    else blk(mi);
    __builtin_amdgcn_sched_barrier(0);
  });
}

// The same for 8-bit operands: one matrix step a slice, which is one block of
// the scales, so each 16 x 16 product is taken by itself and added times its
// scales (4 fused multiply-adds a lane to a matrix instruction, which the other
// wave of the SIMD covers). Lane group g takes chunks g and 4 + g of a row. A
// product is added while the next four are made (two: 1.5% slower at 64 x 256
// rows, K = 1024, N = 2688; the additions take 10% of that launch's time).
template <class C, class Mid, class Blk>
__device__ __forceinline__ void ring_mma_fp8(f32x4 (&acc)[C::NI][C::MI], const lds_u8 *a_stage,
                                             const lds_u8 *b_stage, int wm0, int wn0, int lane,
                                             float column, Mid &&mid, Blk &&blk) {
  const int g = lane / 16, s = lane % 16;
  const lds_u8 *const ar = a_stage + (wm0 + s) * kRowBytes;
  const lds_u8 *const br = b_stage + C::A_BYTES + (wn0 + s) * kRowBytes;
  const lds_u8 *const sc = a_stage + C::A_BYTES + C::B_BYTES + 4 * (wm0 + s);
  const int c0 = 16 * (g ^ (s & 7)), c1 = 16 * ((4 + g) ^ (s & 7));
  // row fragments are read one block ahead, two where registers allow
  constexpr int Y = C::MI > 4 ? 2 : 3;
  ring_i32x8 x[C::NI], y[Y];
  float scale[Y];
  constexpr int D = 4;  // matrix instructions between a product and its addition
  f32x4 d[D + 1];
  auto read = [&](const lds_u8 *row) {
    const u32x4 lo = *(const lds_u32x4 *)(row + c0), hi = *(const lds_u32x4 *)(row + c1);
    return __builtin_bit_cast(ring_i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_y = [&](auto bc) {
    constexpr int b = decltype(bc)::value;
    if constexpr (b < C::MI) {
      y[b % Y] = read(ar + b * 16 * kRowBytes);
      scale[b % Y] = *(const lds_f32 *)(sc + b * 64);
    }
  };
#pragma unroll
  for (int ni = 0; ni < C::NI; ++ni) x[ni] = read(br + ni * 16 * kRowBytes);
  read_y(std::integral_constant<int, 0>{});
  if constexpr (Y > 2) read_y(std::integral_constant<int, 1>{});
  constexpr int P = C::NI * C::MI;
  // the row's scale times the columns', of every row block that is not added yet
  constexpr int R = D / C::NI + 2;
  float both[R];
  auto add = [&](auto ic) {  // the product of block i % NI of row block i / NI
    constexpr int i = decltype(ic)::value, ni = i % C::NI, b = i / C::NI;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[ni][b][j] = __builtin_fmaf(d[i % (D + 1)][j], both[b % R], acc[ni][b][j]);
    // (the compiler would sink the sums past the loads' branches, and keep every
    // product in registers until then)
    asm volatile("" : "+v"(acc[ni][b]));
    if constexpr (ni == C::NI - 1) blk(b);
  };
  static_for<P>([&](auto ic) {
    constexpr int i = decltype(ic)::value, ni = i % C::NI, b = i / C::NI;
    if constexpr (ni == 0) read_y(std::integral_constant<int, b + Y - 1>{});
    // formats 0, 0 = E4M3; constant scales of 0 select the form without scales
    d[i % (D + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        x[ni], y[b % Y], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
    if constexpr (ni == 0) both[b % R] = scale[b % Y] * column;
    if constexpr (i >= D) add(std::integral_constant<int, i - D>{});
    if constexpr (ni == C::NI - 1) mid(std::integral_constant<int, b>{});
    __builtin_amdgcn_sched_barrier(0);
  });
  constexpr int L = P < D ? P : D;
  static_for<L>([&](auto jc) { add(std::integral_constant<int, P - L + decltype(jc)::value>{}); });
}

// An fp32 scale as its power of two (of a subnormal number -127) and the rest.
struct ScaleParts {
  int power;
  float rest;
  __device__ __forceinline__ explicit ScaleParts(float s) {
    power = min((int)(__builtin_bit_cast(uint32_t, s) >> 23 & 255), 254) - 127;  // (infinity, NaN: the rest)
    rest = __builtin_ldexpf(s, -power);
  }
};

// 8 bits: the scale of a wave's columns (they lie in one block of 128) in each slice, to
// be read through the scalar cache. (A wave past the last column takes the last block's.)
template <class C>
__device__ __forceinline__ cst_f32 *ring_columns(const RingTile &t, int wn0) {
  const int band = C::BN > 128 ? min(wn0, t.ncols - 1) / 128 : 0;
  return (cst_f32 *)(t.Bs + (uint64_t)band * t.bs_step);
}

// Sum of 16 products of E4M3 codes.
__device__ __forceinline__ float dot16_fp8(u32x4 a, u32x4 b, float sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    static_for<2>([&](auto high) {
      const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[i], decltype(high)::value),
                  y = __builtin_amdgcn_cvt_pk_f32_fp8((int)b[i], decltype(high)::value);
      sum = __builtin_fmaf(x.y, y.y, __builtin_fmaf(x.x, y.x, sum));
    });
  return sum;
}

// 8 bits: row block mi, where a row of it came out infinite or NaN. If that may be since
// the product of its scale and the columns' passed fp32, the block is computed anew from
// memory, an output at a time, with the scales' powers of two applied apart from their
// product: a block's sum is a multiple of 2^-18 and at most 2^25, so times 2^-100 ..
// 2^100 it is exact. What is left of the power beyond that goes to the product of the
// rests, up to 2^+-120, where the result is infinite or 0 anyway. (Rare, so it is kept
// plain: with every row so, 64 x 256 rows, K = 1024, N = 2688 take 7.5 ms. Matrix
// instructions stay in the slices' loops, which let no load be waited for.)
template <class C>
__device__ __forceinline__ void ring_block_apart(f32x4 (&acc)[C::NI][C::MI], int mi, const RingTile &t,
                                                 int wm0, int wn0, int lane) {
  cst_f32 *const columns = ring_columns<C>(t, wn0);
  const int g = lane / 16, row = wm0 + mi * 16 + lane % 16, KT = ring_slices(t);
  auto row_scale = [&](int k) {
    const buf_rsrc rs = make_buf(t.As + (uint64_t)k * t.as_step, 4u * (uint32_t)t.rows);
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * row, 0, 0));
  };
  bool passed = false;
#pragma unroll 1
  for (int k = 0; k < KT; ++k) {
    const float s = row_scale(k), c = columns[k];
    passed |= fabsf(s * c) == INFINITY && fabsf(s) < INFINITY && fabsf(c) < INFINITY;
  }
  if (__ballot(passed) == 0) return;
#pragma unroll 1
  for (int q = 0; q < 4 * C::NI; ++q) {
    const int col = wn0 + q / 4 * 16 + 4 * g + q % 4;
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < KT; ++k) {
      const ScaleParts r(row_scale(k)), c(columns[k]);
      const int power = r.power + c.power, at_once = min(max(power, -100), 100);
      const buf_rsrc ra = ring_rows(t.A, t.rows, t, k), rb = ring_rows(t.B, t.ncols, t, k);
      float d = 0.0f;
#pragma unroll 1
      for (uint32_t at = 0; at < kRowBytes; at += 16) {
        const bool in = at < t.pitch - (uint32_t)k * kRowBytes;
        d = dot16_fp8(ld_buf16(ra, in ? (uint32_t)row * t.pitch + at : kOob, 0),
                      ld_buf16(rb, in ? (uint32_t)col * t.pitch + at : kOob, 0), d);
      }
      sum = __builtin_fmaf(__builtin_ldexpf(d, at_once),
                           __builtin_ldexpf(r.rest * c.rest, min(max(power - at_once, -120), 120)), sum);
    }
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[ni][mi][j] = q == 4 * ni + j ? sum : acc[ni][mi][j];
  }
}

// One step: multiply slice k out of its stage (a_cur and b_cur, both its
// start) and meanwhile refill the stage that slice k - 1 left: a_nxt is that
// stage, b_nxt too, or with EARLY_B the present one, whose weights are read
// by then. What is read and what is loaded into are passed as distinct memory
// (__restrict__): without that the compiler would hold back every LDS read
// until all loads into LDS have landed. The barrier in mid() keeps the one
// pair that does meet, the reads of b_cur and the loads into b_nxt, in order.
template <class C>
__device__ __forceinline__ void ring_step(f32x4 (&acc)[C::NI][C::MI], const RingTile &t,
                                          const lds_u8 *__restrict__ a_cur,
                                          const lds_u8 *__restrict__ b_cur,
                                          lds_u8 *__restrict__ a_nxt, lds_u8 *__restrict__ b_nxt,
                                          int ka, int kb, int KT, int wave, int lane, int wm0, int wn0,
                                          int blocks_left, float column) {
  const RingPieces<C> loads(t, a_nxt, ka, b_nxt, kb, KT, wave, lane);
  auto mid = [&](auto mc) {
    constexpr int mi = decltype(mc)::value, j0 = mi * C::LPS / C::MI, j1 = (mi + 1) * C::LPS / C::MI;
    static_for<j1 - j0>([&](auto jc) {
      constexpr int j = j0 + decltype(jc)::value;
      if constexpr (C::EARLY_B && j == C::NA) {
        // every wave has its column fragments and scales
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wg_barrier();
      }
      loads.template issue<j>();
    });
  };
  __builtin_amdgcn_s_setprio(1);
  if constexpr (C::FP8) ring_mma_fp8<C>(acc, a_cur, b_cur, wm0, wn0, lane, column, mid, [](int) {});
  else ring_mma<C>(acc, a_cur, b_cur, wm0, wn0, lane, blocks_left, mid, [](int) {});
  __builtin_amdgcn_s_setprio(0);
}

// A whole tile whose prologue has been issued. n_blocks: 32-value blocks of a
// row (MX only). epi.begin() runs before the last slice's products,
// epi.block(acc, mi) stores row block mi. next() runs between the last LDS
// read of the tile and its stores (or, for tiles of at most 4 row blocks a
// wave, which store during the last slice, after them): it issues the next
// tile's prologue.
//
// Loads and stores return in order, so a wait for the first slice would also wait
// for the stores that the tile before issued after it. Where `after` says that it
// was one that stores behind the prologue, STORES times at least a wave, that many
// may stay in flight at the first slice (64 x 256 rows, K = 1024, N = 2688 with
// SwiGLU 70.1 -> 68.7 us).
//
// again() gives t anew (8 bits): kept over the loop for what is rare after it, its parts
// would take scalars that the loop does not have.
struct NoTile {
  __device__ __forceinline__ RingTile operator()() const { return RingTile{}; }
};
template <class C, int STORES = 0, class Epi, class Next, class Again = NoTile>
__device__ __forceinline__ void run_ring_tile(const RingTile &t, lds_u8 *lds, int tid,
                                              int n_blocks, Epi &&epi, Next &&next,
                                              bool after = false, Again &&again = NoTile{}) {
  const int wave = scalar(tid / kWave);
  const int lane = tid % kWave;
  const int wm0 = (wave / C::WN) * C::WTM, wn0 = (wave % C::WN) * C::WTN;
  f32x4 acc[C::NI][C::MI];
#pragma unroll
  for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) acc[ni][mi] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int KT = ring_slices(t);
  int cur = 0, nxt = C::S - 1;  // stages of slice k and of slice k + S - 1
  cst_f32 *columns = nullptr;
  float column = 0.0f;
  if constexpr (C::FP8) {
    columns = ring_columns<C>(t, wn0);
    column = columns[0];
  }
  for (int k = 0; k < KT - 1; ++k) {
    if constexpr (C::EARLY_B) {  // the weights of slice k + 1 stay in flight
      if (STORES > 0 && k == 0 && after) wait_loads<C::NB + STORES>();
      else wait_loads<C::NB>();
    }
    if constexpr (!C::EARLY_B)
      wait_slices<C>(min(C::S - 2, KT - 1 - k));  // slices k + 1 .. min(k + S - 2, KT - 1) do
    wg_barrier();
    lds_u8 *const c = lds + cur * C::STAGE, *const n = lds + nxt * C::STAGE;
    ring_step<C>(acc, t, c, c, n, C::EARLY_B ? c : n, k + C::S - 1, k + C::S - (C::EARLY_B ? 0 : 1), KT,
                 wave, lane, wm0, wn0, n_blocks - 8 * k, column);
    if constexpr (C::FP8) column = columns[k + 1];
    cur = cur + 1 == C::S ? 0 : cur + 1;
    nxt = nxt + 1 == C::S ? 0 : nxt + 1;
  }
  wait_loads<0>();
  wg_barrier();
  epi.begin();
  // 8 bits: where the product of a row's and the columns' scale passed fp32, all that this
  // wave has of the row is infinite or (for sums of 0) NaN, so one value a row is looked at.
  auto store = [&](int mi) {
    if constexpr (C::FP8)
      if (__builtin_expect(__ballot(!(fabsf(acc[0][mi].x) < INFINITY)) != 0, 0))
        ring_block_apart<C>(acc, mi, again(), wm0, wn0, lane);
    epi.block(acc, mi);
  };
  // Row block mi is final. The empty asm keeps its products ahead of the
  // epilogue's branches (the compiler would move them into those).
  auto final_block = [&](int mi) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) asm volatile("" : "+v"(acc[ni][mi]));
    if constexpr (C::MI <= 4) store(mi);
  };
  const lds_u8 *const last = lds + cur * C::STAGE;
  auto none = [](auto) {};
  if constexpr (C::FP8) ring_mma_fp8<C>(acc, last, last, wm0, wn0, lane, column, none, final_block);
  else ring_mma<C>(acc, last, last, wm0, wn0, lane, n_blocks - 8 * (KT - 1), none, final_block);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  next();
  if constexpr (STORES > 0) asm volatile("" ::: "memory");  // the stores come behind the prologue
  if constexpr (C::MI > 4) {
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      store(mi);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

static_assert(kThreads / kWave == 8, "eight waves share a slice's loads");

// The tiles of one workgroup, one after the other. make(tile) gives a
// RingTile, run(cfg, ring tile, tile, next) runs one with the configuration
// cfg, a default-constructed RingCfg. In 8 bits the tiles are dealt out with two
// differences:
//  * A launch of less than a round spreads its tiles over all XCDs, so that they
//    come through eight L2s and not through the first few.
//  * Every other round from the fourth on is dealt out backwards: where heights
//    mix, tall tiles come first, and the workgroups that got more of them would
//    get the taller ones of every later round too (skewed 16k 84.8 -> 83.8 us).
template <int F, class Make, class Run>
__device__ __forceinline__ void run_ring_tiles(const RingSched &sched, const RingGrid &grid,
                                               const int32_t *off, int E, int M_cap, int N,
                                               int bm_fixed, lds_u8 *lds, Make &&make, Run &&run) {
  const int G = gridDim.x, b = blockIdx.x;
  // contiguous tiles on one XCD (workgroup ids go round-robin to the XCDs)
  constexpr bool FP8 = F == kRowsFp8;
  int t = (b % 8) * (G / 8) + b / 8;
  if constexpr (FP8) {
    const int per = grid.total < G ? cdiv(grid.total, 8) : G / 8;
    t = b / 8 < per ? (b % 8) * per + b / 8 : grid.total;
  }
  if (t >= grid.total) return;
  Tile tl = decode_ring_tile(sched, off, t, E, M_cap, N, bm_fixed, grid);
  RingTile rt = make(tl);
  {
    const int tid = threadIdx.x;
    ring_prologue<F>(rt, tl.bm, tl.bn, lds, scalar(tid / kWave), tid % kWave);
  }
  for (;;) {
    int t2 = t + G;
    if constexpr (FP8) {  // (the place in this round follows from t: one scalar less to keep)
      const int round = t / G, at = t - round * G;
      t2 = (round + 1) * G + (round >= 2 ? G - 1 - at : at);
    }
    const bool more = t2 < grid.total;
    Tile ntl = tl;
    if (more) ntl = decode_ring_tile(sched, off, t2, E, M_cap, N, bm_fixed, grid);
    const RingTile nrt = make(ntl);
    auto next = [&] {
      int tid = threadIdx.x;
      asm volatile("" : "+v"(tid));
      if (more) ring_prologue<F>(nrt, ntl.bm, ntl.bn, lds, scalar(tid / kWave), tid % kWave);
    };
    if (tl.bn == 256) {
      switch (tl.bm) {
        case 16: run(RingCfg<16, 256, 1, 8, F>{}, rt, tl, next); break;
        case 32: run(RingCfg<32, 256, 1, 8, F>{}, rt, tl, next); break;
        case 64: run(RingCfg<64, 256, 1, 8, F>{}, rt, tl, next); break;
        case 128: run(RingCfg<128, 256, 2, 4, F>{}, rt, tl, next); break;
        default: run(RingCfg<256, 256, 2, 4, F>{}, rt, tl, next); break;
      }
    } else if (tl.bn == 128) {
      switch (tl.bm) {
        case 16: run(RingCfg<16, 128, 1, 8, F>{}, rt, tl, next); break;
        case 32: run(RingCfg<32, 128, 1, 8, F>{}, rt, tl, next); break;
        case 64: run(RingCfg<64, 128, 2, 4, F>{}, rt, tl, next); break;
        case 128: run(RingCfg<128, 128, 2, 4, F>{}, rt, tl, next); break;
        default: run(RingCfg<256, 128, 4, 2, F>{}, rt, tl, next); break;
      }
    } else {
      switch (tl.bm) {
        case 32: run(RingCfg<32, 64, 2, 4, F>{}, rt, tl, next); break;
        case 64: run(RingCfg<64, 64, 2, 4, F>{}, rt, tl, next); break;
        case 128: run(RingCfg<128, 64, 4, 2, F>{}, rt, tl, next); break;
        default: run(RingCfg<256, 64, 4, 2, F>{}, rt, tl, next); break;
      }
    }
    if (!more) break;
    t = t2;
    tl = ntl;
    rt = nrt;
  }
}

// --------------------------------------------------------------- epilogues
//
// Each 16 x 16 block leaves lane 16 g + s with columns 4 g .. 4 g + 3 of row
// s: 64 bytes of each of 16 rows in one fp32 store instruction. Stores of
// whole 128-byte lines are three times as fast (measured out of one
// workgroup a CU into L2: 117 bytes a ns against 32 - 37; into HBM on the whole chip 5.5 - 6.0 TB/s
// against 5.3 - 5.7), so neighbouring blocks trade halves first:
//  * swap_rows: of two 16-byte pieces a (left) and b (right) of a row, lanes
//    s < 8 keep a of row s and give b to lane s + 8, which gives its a. a then
//    holds rows 0 .. 7, left in lanes s < 8 and right in lanes s >= 8, b rows 8
//    .. 15 likewise: 8 rows x 128 bytes an instruction.
//  * Outputs of 2 bytes first swap lane groups between two neighbouring blocks
//    (v_permlane16_swap), which gives every lane 8 neighbouring columns: group
//    g then holds columns 8 (g / 2) .. + 7 of block (g % 2).
__device__ __forceinline__ void swap_rows(u32x4 &a, u32x4 &b) {
  constexpr int kRor8 = 0x128;  // lane s reads lane (s + 8) % 16 of its 16
  const u32x4 a0 = a, b0 = b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int av = (int)a0[j], bv = (int)b0[j];
    a[j] = (uint32_t)__builtin_amdgcn_update_dpp(av, bv, kRor8, 0xf, 0xc, false);
    b[j] = (uint32_t)__builtin_amdgcn_update_dpp(bv, av, kRor8, 0xf, 0x3, false);
  }
}

__device__ __forceinline__ u32x2 pack_bf16(f32x4 v) {
  return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

__device__ __forceinline__ u32x4 swap_pair(u32x2 a, u32x2 b) {
  const auto p = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
  const auto q = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
  return u32x4{p[0], q[0], p[1], q[1]};
}

// Rows m0 .. m0 + 15 of a row-major array as a buffer from the tile's first
// column on; rows past the tile's valid ones are outside it, so that a store
// there is dropped and a load reads zeros, without a branch. base: row 0 of
// the tile, its first column; col_bytes: that column's place in the row. 16
// rows stay below 2^31 bytes (columns <= 2^24 of 4 bytes).
__device__ __forceinline__ buf_rsrc row_block(const void *base, int m0, int rows, size_t row_bytes,
                                              size_t col_bytes) {
  const int n = min(max(rows - m0, 0), 16);
  return make_buf((const char *)base + (size_t)m0 * row_bytes,
                  n > 0 ? (uint32_t)((size_t)n * row_bytes - col_bytes) : 0u);
}

template <int POLICY = kCacheDefault>
__device__ __forceinline__ void st_buf16(buf_rsrc r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, POLICY);
}
__device__ __forceinline__ void st_buf8(buf_rsrc r, uint32_t off, u32x2 v) {
  __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, 0);
}
__device__ __forceinline__ void st_buf4(buf_rsrc r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, off, 0, 0);
}

// One row block of a wave tile as fp32 or bf16. row_bytes: of a row of the
// output; base: its first row and column of the tile; ncols: valid columns.
template <class C, bool BF16, int POLICY = kCacheDefault>
__device__ __forceinline__ void store_block(const f32x4 (&acc)[C::NI][C::MI], int mi, void *base,
                                            int wm0, int wn0, int lane, int rows, int ncols,
                                            size_t row_bytes, size_t col_bytes) {
  const int g = lane / 16, s = lane % 16;
  const buf_rsrc r = row_block(base, wm0 + mi * 16, rows, row_bytes, col_bytes);
  const uint32_t row = (uint32_t)s * (uint32_t)row_bytes;
  const uint32_t row8 = (uint32_t)(s % 8) * (uint32_t)row_bytes, down8 = 8u * (uint32_t)row_bytes;
  if constexpr (!BF16 && C::NI % 2 == 0) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ni += 2) {
      u32x4 a = __builtin_bit_cast(u32x4, acc[ni][mi]), b = __builtin_bit_cast(u32x4, acc[ni + 1][mi]);
      swap_rows(a, b);
      const int n = wn0 + (ni + s / 8) * 16 + 4 * g;
      const uint32_t at = row8 + 4u * n;
      st_buf16<POLICY>(r, n < ncols ? at : kOob, a);
      st_buf16<POLICY>(r, n < ncols ? at + down8 : kOob, b);
    }
  } else if constexpr (!BF16) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) {
      const int n = wn0 + ni * 16 + 4 * g;
      st_buf16<POLICY>(r, n < ncols ? row + 4u * n : kOob, __builtin_bit_cast(u32x4, acc[ni][mi]));
    }
  } else if constexpr (C::NI % 4 == 0) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ni += 4) {
      u32x4 a = swap_pair(pack_bf16(acc[ni][mi]), pack_bf16(acc[ni + 1][mi]));
      u32x4 b = swap_pair(pack_bf16(acc[ni + 2][mi]), pack_bf16(acc[ni + 3][mi]));
      swap_rows(a, b);
      const int n = wn0 + (ni + 2 * (s / 8) + g % 2) * 16 + 8 * (g / 2);
      const uint32_t at = row8 + 2u * n;
      st_buf16<POLICY>(r, n < ncols ? at : kOob, a);
      st_buf16<POLICY>(r, n < ncols ? at + down8 : kOob, b);
    }
  } else if constexpr (C::NI % 2 == 0) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ni += 2) {
      const int n = wn0 + (ni + g % 2) * 16 + 8 * (g / 2);
      st_buf16<POLICY>(r, n < ncols ? row + 2u * n : kOob,
               swap_pair(pack_bf16(acc[ni][mi]), pack_bf16(acc[ni + 1][mi])));
    }
  } else {
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) {
      const int n = wn0 + ni * 16 + 4 * g;
      st_buf8(r, n < ncols ? row + 2u * n : kOob, pack_bf16(acc[ni][mi]));
    }
  }
}

}  // namespace gg
