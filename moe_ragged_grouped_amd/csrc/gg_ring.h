// A ring of LDS stages filled straight from global memory, and the products
// of one output tile out of it, for operands whose contraction index is the
// fastest in memory:
//
//   C[m][n] = sum_l A[m][l] * W[n][l]
//
// The data gradient (A = dC, W = B[e] with its K rows, l = the product's
// columns) and the 4-bit product (both operands packed along K) have this
// form. Both operands then look alike in bytes: a row of a slice is 128
// bytes, 64 bf16 or 256 4-bit values, and one 16-byte piece of a row is what
// a lane feeds to one matrix instruction.
//
// MI355X mapping:
//  * buffer_load_dwordx4 ... lds moves 16 bytes a lane from global memory into
//    LDS without passing through registers: no staging registers beside the
//    accumulators, no ds_write (which costs 8 LDS cycles an instruction), and
//    as many slices in flight as LDS has room for. A lane out of the buffer's
//    range writes zeros (checked by an in-bounds probe), which is the zero
//    fill of padding rows, of columns past the end and of the last slice's
//    tail.
//  * The instruction writes lane l's 16 bytes at base + 16 l, so a swizzle has
//    to be put into the global side: lane l of a wave's 8 x 128-byte piece
//    loads row l / 8, chunk (l % 8) ^ (l / 8), and chunk c of row r then sits
//    at chunk c ^ (r % 8). A fragment read (ds_read_b128, 16 rows) touches
//    every bank once.
//  * S stages, one barrier a slice: the barrier that says "slice i has landed"
//    also says "every wave is done with slice i - 1", whose stage is refilled
//    at once with slice i + S - 1.
#pragma once

#include "gg_common.h"
#include "gg_schedule.h"

namespace gg {

typedef __attribute__((ext_vector_type(8))) int ring_i32x8;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) u32x4 gbl_u32x4;
typedef __attribute__((address_space(1))) u32x2 gbl_u32x2;

// 16 bytes a lane, global -> LDS at dst + 16 * lane (dst is wave-uniform).
template <int POLICY = kCacheDefault>
__device__ __forceinline__ void dma16(buf_rsrc r, lds_u8 *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, voff, 0, 0, POLICY);
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
// The tile list of gg_schedule.h with one change: where every expert's tiles
// are 16 rows high (the launch only streams weights), the tile width follows
// from the number of tiles. Wide tiles move longer runs per barrier, but a
// launch of a few tokens has too few of them to occupy the chip, so the
// widest of 512, 256 and 128 columns is taken that still gives every
// workgroup of the launch a tile.
struct RingSched {
  int start[kMaxExperts + 1];
  long long wave_sum[kThreads / kWave];
  int wave_tall[kThreads / kWave];
  int width16;
};

constexpr int kNarrowN = 128;

__device__ __forceinline__ int build_ring_schedule(RingSched &s, const int32_t *__restrict__ off_g, int E,
                                          int M_cap, int N, int bm_fixed, int tile_cap, int G) {
  const int tid = threadIdx.x;
  constexpr int kRun = kMaxExperts / kThreads;
  const int e0 = tid * kRun;
  int rows[kRun], height[kRun];
  int tall = 0;
  long long m16 = 0;  // 16-row tiles of this run, a column apart
  int lo = e0 < E ? clamp_off(off_g, e0, M_cap) : 0;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const int e = e0 + j;
    rows[j] = 0;
    height[j] = 16;
    if (e < E) {
      const int hi = clamp_off(off_g, e + 1, M_cap);
      rows[j] = hi > lo ? hi - lo : 0;
      height[j] = bm_fixed ? bm_fixed : adaptive_bm(rows[j]);
      tall |= rows[j] > 0 && height[j] > 16;
      m16 += cdiv(rows[j], 16);
      lo = hi;
    }
  }
  const int lane = tid % kWave, wave = tid / kWave;
  const bool any = __any(tall);
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) m16 += __shfl_xor(m16, d, kWave);
  if (lane == 0) {
    s.wave_tall[wave] = any;
    s.wave_sum[wave] = m16;
  }
  __syncthreads();
  bool any_tall = false;
  long long all16 = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    any_tall |= s.wave_tall[w] != 0;
    all16 += s.wave_sum[w];
  }
  int width16 = kTileN;
  if (!any_tall)
    width16 = all16 * cdiv(N, kWideN) >= G ? kWideN : (all16 * cdiv(N, kTileN) >= G ? kTileN : kNarrowN);
  __syncthreads();  // wave_sum is written again below
  long long cnt[kRun];
  long long local = 0;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    cnt[j] = rows[j] > 0 ? (long long)cdiv(rows[j], height[j]) *
                               cdiv(N, height[j] == 16 ? width16 : kTileN)
                         : 0;
    local += cnt[j];
  }
  long long incl = local;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const long long y = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += y;
  }
  if (lane == kWave - 1) s.wave_sum[wave] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) before += s.wave_sum[w];
    total += s.wave_sum[w];
  }
  if (total > tile_cap) total = 0;  // overlapping malformed segments: no tiles
  long long run = before + incl - local;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const int e = e0 + j;
    if (e < E) s.start[e] = total ? (int)run : 0;
    run += cnt[j];
  }
  if (tid == 0) {
    s.start[E] = (int)total;
    s.width16 = width16;
  }
  __syncthreads();
  return (int)total;
}

// Tile t of the list (0 <= t < total).
__device__ __forceinline__ Tile decode_ring_tile(const RingSched &s,
                                                 const int32_t *__restrict__ off_g, int t, int E,
                                                 int M_cap, int N, int bm_fixed) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.start[mid] <= t) lo = mid; else hi = mid;
  }
  const int r0 = clamp_off(off_g, lo, M_cap);
  const int m = clamp_off(off_g, lo + 1, M_cap) - r0;
  const int b = bm_fixed ? bm_fixed : adaptive_bm(m);
  const int bn = b == 16 ? s.width16 : kTileN;
  const int NT = cdiv(N, bn);
  const int n_mt = cdiv(m, b);
  const int local = t - s.start[lo];
  // groups of kGroupM M tiles; N outer, M inner inside a group
  const int per_group = kGroupM * NT;
  const int grp = local / per_group;
  const int r = local - grp * per_group;
  const int gm = min(kGroupM, n_mt - grp * kGroupM);
  const int nt = r / gm;
  const int mt = grp * kGroupM + (r - nt * gm);
  Tile tl;
  tl.expert = lo;
  tl.bm = b;
  tl.bn = bn;
  tl.row0 = r0 + mt * b;
  tl.rows = min(b, m - mt * b);
  tl.col0 = nt * bn;
  return tl;
}

// ------------------------------------------------------------------- tiles

constexpr int kRowBytes = 128;  // bytes of a row in one slice

// MX: 4-bit operands with a scale byte per 32 values, 8 of them per row and
// slice, kept beside the slice they belong to.
template <int BM_, int BN_, int WM_, int WN_, int S_, bool MX_>
struct RingCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
  static constexpr bool MX = MX_;
  static_assert(WM * WN == kThreads / kWave, "one wave per wave tile");
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static_assert(WTM % 16 == 0 && WTN % 16 == 0, "16x16 blocks");
  static constexpr int MI = WTM / 16, NI = WTN / 16;
  static constexpr int A_BYTES = BM * kRowBytes, B_BYTES = BN * kRowBytes;
  static constexpr int AS_BYTES = MX ? BM * 8 : 0, BS_BYTES = MX ? BN * 8 : 0;
  static constexpr int STAGE = A_BYTES + B_BYTES + AS_BYTES + BS_BYTES;
  // Loads a wave issues per slice. Tiles of fewer than 64 rows use only the
  // first BM lanes of one instruction, so that every wave issues the same
  // number and waits on the same count.
  static constexpr int A_INSTR = BM >= 64 ? BM / 64 : 1;
  static constexpr int A_LANES = BM >= 64 ? 64 : BM;
  static constexpr int B_INSTR = BN / 64;
  static constexpr int LPS = A_INSTR + B_INSTR + (MX ? 1 : 0);
  static constexpr int LDS_BYTES = S * STAGE;
  static_assert(S >= 2 && (S - 2) * LPS < 64, "loads in flight");
};

struct RingTile {
  const char *A;          // row 0 of the tile
  const char *B;          // weight row (output column) 0 of the tile
  const char *As, *Bs;    // MX: scale bytes of the first slice, row 0 / column 0
  size_t as_step, bs_step;  // MX: bytes from a slice's scales to the next one's
  uint32_t pitch;         // bytes of a row of A and of B
  int rows, ncols;        // valid rows and columns
  int tid;
};

// Per-lane constants of a tile's loads. The chunk is the same for all of a
// lane's loads (a row's place in its group of 8 is l / 8 throughout).
template <class C>
struct RingLoads {
  uint32_t a_off[C::A_INSTR], b_off[C::B_INSTR];
  uint32_t chunk;  // byte position of this lane's 16 bytes in a slice row
  // MX: what this wave brings of the scales, waves 0-3 of A's, waves 4-7 of
  // B's: the first slice's, bytes to the next slice's, and their size
  uint64_t s_base, s_step;
  uint32_t s_bytes;
};

template <class C>
__device__ __forceinline__ RingLoads<C> ring_loads(const RingTile &t, int wave) {
  RingLoads<C> L;
  const int l = t.tid % kWave;
  const uint32_t r = l / 8;
  L.chunk = 16u * ((l % 8) ^ r);
#pragma unroll
  for (int i = 0; i < C::A_INSTR; ++i)
    L.a_off[i] = ((i * 8 + wave) * (C::A_LANES / 8) + r) * t.pitch + L.chunk;
#pragma unroll
  for (int i = 0; i < C::B_INSTR; ++i) L.b_off[i] = ((i * 8 + wave) * 8 + r) * t.pitch + L.chunk;
  if constexpr (C::MX) {
    const uint64_t as = (uint64_t)t.As, bs = (uint64_t)t.Bs;
    const uint64_t as_step = t.as_step, bs_step = t.bs_step;
    const int rows = t.rows, ncols = t.ncols;
    L.s_base = wave >= 4 ? bs : as;
    L.s_step = wave >= 4 ? bs_step : as_step;
    L.s_bytes = 8u * (uint32_t)(wave >= 4 ? ncols : rows);
  }
  return L;
}

// Issues this wave's loads of slice k into one stage. Where rows of A take
// fewer than 8 lanes' worth of an instruction, a row's place in its group of
// 8 is not l / 8 alone; 16- and 32-row tiles therefore load 2 or 4 rows a
// wave and swizzle by the row's own place (a_row8 below).
template <class C, int B_POLICY>
__device__ __forceinline__ void ring_issue(const RingTile &t, const RingLoads<C> &L, lds_u8 *stage,
                                           int k, int wave, int lane) {
  const uint32_t k0 = (uint32_t)k * kRowBytes;
  const buf_rsrc ra = make_buf(t.A + k0, (uint32_t)t.rows * t.pitch - k0);
  const buf_rsrc rb = make_buf(t.B + k0, (uint32_t)t.ncols * t.pitch - k0);
  const uint32_t left = t.pitch - k0;  // bytes of a row from this slice on
  const bool b_in = L.chunk < left;
  if constexpr (C::A_LANES == 64) {
#pragma unroll
    for (int i = 0; i < C::A_INSTR; ++i)
      dma16(ra, stage + (i * 8 + wave) * 1024, b_in ? L.a_off[i] : kOob);
  } else {
    // rows wave * (A_LANES / 8) + l / 8; their place in a group of 8
    constexpr int kR = C::A_LANES / 8;
    const uint32_t r8 = (wave * kR + lane / 8) % 8;
    const uint32_t chunk = 16u * ((lane % 8) ^ r8);
    const uint32_t off = (wave * kR + lane / 8) * t.pitch + chunk;
    if (lane < C::A_LANES)
      dma16(ra, stage + wave * (16 * C::A_LANES), chunk < left ? off : kOob);
  }
#pragma unroll
  for (int i = 0; i < C::B_INSTR; ++i)
    dma16<B_POLICY>(rb, stage + C::A_BYTES + (i * 8 + wave) * 1024, b_in ? L.b_off[i] : kOob);
  if constexpr (C::MX) {
    // scale bytes: 16, two rows' worth, a lane
    const bool is_b = wave >= 4;
    const int n = is_b ? C::BN / 8 : C::BM / 8;  // lanes of this wave
    const int at = 16 * (wave % 4) * n;
    const buf_rsrc rs = make_buf((const void *)(L.s_base + (uint64_t)k * L.s_step), L.s_bytes);
    lds_u8 *const dst = stage + C::A_BYTES + C::B_BYTES + (is_b ? C::AS_BYTES : 0) + at;
    if (lane < n) dma16(rs, dst, (uint32_t)(at + 16 * lane));
  }
}

// The products of one slice. Two matrix steps; lane group g takes 16-byte
// chunk 4 ks + g of a row (bf16: l = 32 ks + 8 g ..) or 2 g + ks (4-bit: block
// 2 g + ks of 32 values, so that a lane's two scale bytes are neighbours; the
// matrix cores pair lane group with lane group, so any order that both
// operands share is the same sum). blk(mi) runs after row block mi's last
// product.
template <class C, class Blk>
__device__ __forceinline__ void ring_mma(f32x4 (&acc)[C::NI][C::MI],
                                         const lds_u8 *__restrict__ stage, int wm0, int wn0,
                                         int lane, int blocks_left, Blk &&blk) {
  const int g = lane / 16, s = lane % 16;
  const lds_u8 *const ar = stage + (wm0 + s) * kRowBytes;
  const lds_u8 *const br = stage + C::A_BYTES + (wn0 + s) * kRowBytes;
  int sa[C::MX ? C::MI : 1], sb[C::MX ? C::NI : 1];
  if constexpr (C::MX) {
    // scale bytes past the row's last block are whatever memory holds there;
    // a zero byte (2^-127) times the zero values loaded there is zero
    const int v = blocks_left - 2 * g;
    const int mask = v >= 2 ? 0xffff : (v == 1 ? 0xff : 0);
    const lds_u8 *const sc = stage + C::A_BYTES + C::B_BYTES + 2 * g;
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
      sb[ni] = mask & *(const lds_u16 *)(sc + C::AS_BYTES + 8 * (wn0 + ni * 16 + s));
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
      sa[mi] = mask & *(const lds_u16 *)(sc + 8 * (wm0 + mi * 16 + s));
  }
  static_for<2>([&](auto ksc) {
    constexpr int ks = decltype(ksc)::value;
    const int c = 16 * ((C::MX ? 2 * g + ks : 4 * ks + g) ^ (s & 7));
    u32x4 x[C::NI];
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) x[ni] = *(const lds_u32x4 *)(br + ni * 16 * kRowBytes + c);
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      const u32x4 y = *(const lds_u32x4 *)(ar + mi * 16 * kRowBytes + c);
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        if constexpr (C::MX) {
          // formats 4, 4 = E2M1; a 4-bit operand is the low half of the eight
          // registers, scale byte ks of each lane's scale register
          const ring_i32x8 xv = __builtin_bit_cast(
              ring_i32x8, __builtin_shufflevector(x[ni], x[ni], 0, 1, 2, 3, -1, -1, -1, -1));
          const ring_i32x8 yv = __builtin_bit_cast(
              ring_i32x8, __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1));
          acc[ni][mi] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              xv, yv, acc[ni][mi], 4, 4, ks, sb[ni], ks, sa[mi]);
        } else {
          acc[ni][mi] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, x[ni]), __builtin_bit_cast(bf16x8, y), acc[ni][mi], 0, 0,
              0);
        }
      }
      if constexpr (ks == 1) blk(mi);
    }
    // one step at a time: the next step's fragments, read above this step's
    // products, would need registers on top of the accumulators
    __builtin_amdgcn_sched_barrier(0);
  });
}

// One step: refill the stage that slice k - 1 left, then multiply slice k.
// The two stages are distinct memory (__restrict__): without that the
// compiler would hold back the reads of one until the loads into the other
// have landed.
template <class C, int B_POLICY>
__device__ __forceinline__ void ring_step(f32x4 (&acc)[C::NI][C::MI], const RingTile &t,
                                          const RingLoads<C> &L, const lds_u8 *__restrict__ cur,
                                          lds_u8 *__restrict__ nxt, int k_next, int KT, int wave,
                                          int lane, int wm0, int wn0, int blocks_left) {
  if (k_next < KT) ring_issue<C, B_POLICY>(t, L, nxt, k_next, wave, lane);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_setprio(1);
  ring_mma<C>(acc, cur, wm0, wn0, lane, blocks_left, [](int) {});
  __builtin_amdgcn_s_setprio(0);
  __builtin_amdgcn_sched_barrier(0);
}

// A whole tile. n_blocks: 32-value blocks of a row (MX only). epi(mi) stores
// row block mi of acc. Ends with a barrier after the last LDS read, so that
// the next tile may fill the ring.
template <class C, int B_POLICY, class Epi>
__device__ __forceinline__ void run_ring_tile(const RingTile &t, lds_u8 *lds,
                                              f32x4 (&acc)[C::NI][C::MI], int n_blocks, Epi &&epi) {
  const int wave = __builtin_amdgcn_readfirstlane(t.tid / kWave);
  const int lane = t.tid % kWave;
  const int wm0 = (wave / C::WN) * C::WTM, wn0 = (wave % C::WN) * C::WTN;
#pragma unroll
  for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) acc[ni][mi] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int KT = (int)((t.pitch + kRowBytes - 1) / kRowBytes);
  const RingLoads<C> L = ring_loads<C>(t, wave);
#pragma unroll 1
  for (int k = 0; k < C::S - 1; ++k)
    if (k < KT) ring_issue<C, B_POLICY>(t, L, lds + k * C::STAGE, k, wave, lane);
  int cur = 0, nxt = C::S - 1;  // stages of slice k and of slice k + S - 1
  for (int k = 0; k < KT - 1; ++k) {
    // slices k + 1 .. min(k + S - 2, KT - 1) stay in flight
    wait_slices<C>(min(C::S - 2, KT - 1 - k));
    wg_barrier();
    ring_step<C, B_POLICY>(acc, t, L, lds + cur * C::STAGE, lds + nxt * C::STAGE, k + C::S - 1, KT,
                           wave, lane, wm0, wn0, n_blocks - 8 * k);
    cur = cur + 1 == C::S ? 0 : cur + 1;
    nxt = nxt + 1 == C::S ? 0 : nxt + 1;
  }
  wait_loads<0>();
  wg_barrier();
  // Row block mi is final. The empty asm keeps its products ahead of the
  // epilogue's branches (the compiler would move them into those).
  auto final_block = [&](int mi) {
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni) asm volatile("" : "+v"(acc[ni][mi]));
    if constexpr (C::MI <= 4) epi(mi);
  };
  ring_mma<C>(acc, lds + cur * C::STAGE, wm0, wn0, lane, n_blocks - 8 * (KT - 1), final_block);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  if constexpr (C::MI > 4) {
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      epi(mi);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

static_assert(kThreads / kWave == 8, "eight waves share a slice's loads");

// --------------------------------------------------------------- epilogues
//
// Each 16 x 16 block leaves lane 16 g + s with columns 4 g .. 4 g + 3 of row
// s. Outputs of 2 bytes would make 8-byte stores of that. Swapping lane
// groups between two neighbouring blocks (v_permlane16_swap) instead gives
// every lane 8 neighbouring columns, one 16-byte store: group g then holds
// columns 8 (g / 2) .. + 7 of block (g % 2).
__device__ __forceinline__ u32x2 pack_bf16(f32x4 v) {
  return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

__device__ __forceinline__ u32x4 swap_pair(u32x2 a, u32x2 b) {
  const auto p = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
  const auto q = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
  return u32x4{p[0], q[0], p[1], q[1]};
}

__device__ __forceinline__ void st_g16u(void *p, u32x4 v) { *(gbl_u32x4 *)p = v; }
__device__ __forceinline__ void st_g8u(void *p, u32x2 v) { *(gbl_u32x2 *)p = v; }

}  // namespace gg
