// Weight gradient of the ragged grouped product, for gfx950:
//
//   dB[e][k][n] = sum over the rows r of expert e of A[r][k] * dC[r][n]
//
// The summed index is the row, the slow one of both operands, and its length
// is the expert's row count: ragged, read on the device, possibly zero (that
// expert's gradient is zero). An output tile is BM x BN of one expert's
// weights; its slices are RB rows of A and of dC, brought into a ring of LDS
// stages by buffer_load ... lds (gg_ring.h) and read by the transposing LDS
// read (ds_read_b64_tr_b16), which hands a lane the four rows of one column.
// The buffers end at the group's last row, so the rows of a slice past it
// read as zeros in both operands.
//
// One workgroup per tile, four waves, two workgroups to a CU. The tiles of all
// experts number E * ceil(K / BM) * ceil(N / BN) whatever the routing, so the
// grid is known on the host and the hardware hands the next tile to whichever
// CU is free. A launch ends with its longest tile, so experts come in the
// order of their size class (power of two of the row count), largest first.
//
// What bounds it. 64 experts x 256 rows, K = 1024, N = 2688, fp32 out: 220 us for
// 826 MB (3.8 TB/s); bf16 139; 32 experts, 2048 skewed rows, K = 6144, N = 4096,
// bf16: 362 us for 1.65 GB (4.6 TB/s, a plain copy moves 4.9). The gradient's
// own bytes are most of it: writing it alone takes 118 - 130 us of the 220, the
// loads and products without the stores 110, and the two add up rather than
// overlap. A CU's vector memory path takes loads and stores in one order
// (L1 is stalled on pending loads for 75% of the launch), and neither staggered
// starts, nor stores spread over the next slices, nor more workgroups a CU
// changed that (skewed routing is bounded by its longest group instead: 4,800 of
// 16,384 rows are 150 slices for one workgroup, and bf16 takes 164 us where
// uniform routing takes 139); what helped is fewer and cheaper accesses: whole-line streamed
// stores (store_block) and rows kept in L2.

#include "gg_common.h"
#include "gg_host.h"
#include "gg_ring.h"
#include "grouped_gemm.h"

namespace gg {

enum class WOut { F32, AddF32, BF16 };

struct WgradParams {
  const char *A;    // [M_cap][K] bf16
  const char *dC;   // [M_cap][N] bf16
  const int32_t *off;
  void *dB;         // [E][K][N]
  int E, K, N, M_cap;
  int tiles;        // tiles of one expert
  int per_xcd;      // ceil(tiles / 8)
};

// R > 1: R groups of waves share a tile's rows (slice k to group k % R), each
// with a ring and accumulators of its own, and add up at the end.
template <int BM_, int BN_, int WM_, int WN_, int RB_, int S_, int R_ = 1>
struct WgradCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, RB = RB_, S = S_, R = R_;
  static constexpr int WAVES = WM * WN;  // of a group
  static constexpr int THREADS = kWave * WAVES * R;
  static_assert(R == 1 || WAVES == 1, "groups run at their own pace: no barrier between waves");
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static constexpr int MI = WTM / 16, NI = WTN / 16;
  static_assert(MI * 16 * WM == BM && NI * 16 * WN == BN && RB % 32 == 0, "16x16x32 blocks");
  static constexpr int A_ROW = 2 * BM, B_ROW = 2 * BN;  // bytes of a slice row
  static constexpr int A_BYTES = RB * A_ROW, B_BYTES = RB * B_ROW, STAGE = A_BYTES + B_BYTES;
  static constexpr int A_INSTR = A_BYTES / (1024 * WAVES), B_INSTR = B_BYTES / (1024 * WAVES);
  static_assert(A_INSTR * 1024 * WAVES == A_BYTES && B_INSTR * 1024 * WAVES == B_BYTES, "loads");
  static constexpr int LPS = A_INSTR + B_INSTR;
  static constexpr int RING_BYTES = R * S * STAGE;
  static constexpr int PART_ROW = BN + 4;  // floats of a row of a group's sums (add_groups)
  static constexpr int PART_BYTES = R > 1 ? R * BM * PART_ROW * 4 : 0;
  static constexpr int LDS_BYTES = RING_BYTES > PART_BYTES ? RING_BYTES : PART_BYTES;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

// Chunk (16 bytes) c of slice row r sits at chunk c ^ swz(r). A transposing
// read touches rows 8 g + k' (k' < 4) of every lane group g, 32 bytes each;
// the XOR spreads those over the banks (for 512-byte rows: gg_mainloop.h).
// 128- and 64-byte rows have 8 and 4 chunks, and neighbouring rows lie in
// different parts of the banks already.
template <int ROW>
__device__ __forceinline__ int wg_swz(int r) {
  if constexpr (ROW >= 256) return ((r & 3) << 1) | (((r >> 3) & 1) << 3);
  else if constexpr (ROW == 128) return (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2);
  else return ((r >> 3) & 1) << 1;
}

// Byte offset of this lane's load i inside a slice of an operand of `pitch`
// bytes a row; `col` gets the byte column it starts at.
template <int ROW, int WAVES>
__device__ __forceinline__ uint32_t wg_off(int i, int wave, int lane, uint32_t pitch, uint32_t &col) {
  constexpr int kRows = 1024 / ROW;  // rows of one load instruction
  const int r = (i * WAVES + wave) * kRows + lane / (64 / kRows);
  const int c = (lane % (64 / kRows)) ^ wg_swz<ROW>(r);
  col = 16u * c;
  return (uint32_t)r * pitch + col;
}

template <class C>
struct WgradTile {
  const char *A, *B;        // row 0 of the group, first column of the tile
  uint32_t a_pitch, b_pitch;  // bytes of a row
  uint32_t a_cols, b_cols;    // bytes of a row from the tile's first column on
  int rows;
};

template <class C>
__device__ __forceinline__ void wg_issue(const WgradTile<C> &t, lds_u8 *stage, int k, int wave,
                                         int lane) {
  const int left = min(C::RB, t.rows - k * C::RB);
  const size_t r0 = (size_t)k * C::RB;
  // the resource ends with the last row that belongs to the group; a lane
  // past the row's end is out of range too
  const buf_rsrc ra = make_buf(t.A + r0 * t.a_pitch, (uint32_t)(left - 1) * t.a_pitch + t.a_cols);
  const buf_rsrc rb = make_buf(t.B + r0 * t.b_pitch, (uint32_t)(left - 1) * t.b_pitch + t.b_cols);
#pragma unroll
  for (int i = 0; i < C::A_INSTR; ++i) {
    uint32_t col;
    const uint32_t off = wg_off<C::A_ROW, C::WAVES>(i, wave, lane, t.a_pitch, col);
    dma16(ra, stage + (i * C::WAVES + wave) * 1024, col < t.a_cols ? off : kOob);
  }
#pragma unroll
  for (int i = 0; i < C::B_INSTR; ++i) {
    uint32_t col;
    const uint32_t off = wg_off<C::B_ROW, C::WAVES>(i, wave, lane, t.b_pitch, col);
    dma16(rb, stage + C::A_BYTES + (i * C::WAVES + wave) * 1024, col < t.b_cols ? off : kOob);
  }
}

// A 16-column fragment of 32 slice rows: lane 16 g + s gets column s of rows
// 8 g .. 8 g + 7. p addresses row 8 g + s / 4, four columns of it.
template <int ROW>
__device__ __forceinline__ bf16x8 wg_frag(const lds_u8 *p) {
  const s16x4 lo = lds_read_tr16((const lds_u16 *)p);
  const s16x4 hi = lds_read_tr16((const lds_u16 *)(p + 4 * ROW));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int ROW>
__device__ __forceinline__ int wg_frag_off(int lane, int col0) {
  const int g = lane / 16, s = lane % 16;
  const int r = 8 * g + s / 4, c = col0 + 4 * (s % 4);
  return r * ROW + 16 * ((c / 8) ^ wg_swz<ROW>(r)) + 2 * (c % 8);
}

template <class C>
__device__ __forceinline__ void wg_step(f32x4 (&acc)[C::NI][C::MI], const WgradTile<C> &t,
                                        const lds_u8 *__restrict__ cur, lds_u8 *__restrict__ nxt,
                                        int k_next, int group, int KT, int wave, int lane, int a_off,
                                        int b_off) {
  if (k_next < KT) wg_issue<C>(t, nxt, k_next * C::R + group, wave, lane);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_setprio(1);
  static_for<C::RB / 32>([&](auto ksc) {
    constexpr int ks = decltype(ksc)::value;
    bf16x8 x[C::NI];
    // a block's 32 bytes are bits 5.. of the chunk index, which the swizzle
    // XORs: block i is the first one's address XOR 32 i
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
      x[ni] = wg_frag<C::B_ROW>(cur + C::A_BYTES + 32 * ks * C::B_ROW + (b_off ^ (32 * ni)));
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) {
      const bf16x8 y = wg_frag<C::A_ROW>(cur + 32 * ks * C::A_ROW + (a_off ^ (32 * mi)));
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni)
        acc[ni][mi] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[ni], y, acc[ni][mi], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  });
  __builtin_amdgcn_s_setprio(0);
}

__device__ __forceinline__ int size_class(int rows) { return rows > 0 ? 32 - __builtin_clz(rows) : 0; }

// The expert at position p of the order by size class (power of two of the
// row count), largest class first and by index inside a class; *first and
// *rows are its rows. Every wave finds it for itself, with votes over RUNS x
// 64 experts and no LDS or barrier, as every workgroup pays for it: the first
// form, which ranked all experts through LDS, took 4.5 us a workgroup.
template <int RUNS>
__device__ __forceinline__ int find_expert(const int32_t *__restrict__ off, int E, int M_cap, int p,
                                           int *first, int *rows) {
  const int lane = threadIdx.x % kWave;
  int lo[RUNS], n[RUNS], cls[RUNS];
#pragma unroll
  for (int r = 0; r < RUNS; ++r) {  // all loads in flight together
    const int e = min(r * kWave + lane, E - 1);
    lo[r] = off[e];
    n[r] = off[e + 1];
  }
#pragma unroll
  for (int r = 0; r < RUNS; ++r) {
    lo[r] = min(max(lo[r], 0), M_cap);
    n[r] = max(min(max(n[r], 0), M_cap) - lo[r], 0);
    cls[r] = r * kWave + lane < E ? size_class(n[r]) : -1;
  }
  for (int c = size_class(M_cap); c >= 0; --c) {
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const unsigned long long has = __ballot(cls[r] == c);
      const int count = __popcll(has);
      if (p >= 0 && p < count) {
        // the p-th lane of the vote
        const int before = __popcll(has & ((1ull << lane) - 1));
        const int src = __ffsll((long long)__ballot(cls[r] == c && before == p)) - 1;
        *first = __builtin_amdgcn_readlane(lo[r], src);
        *rows = __builtin_amdgcn_readlane(n[r], src);
        return r * kWave + src;
      }
      p -= count;
    }
  }
  *first = *rows = 0;
  return 0;  // not reached: the classes hold E > p experts
}

__device__ __forceinline__ int wgrad_expert(const int32_t *off, int E, int M_cap, int p, int *first,
                                            int *rows) {
  if (E <= kWave) return find_expert<1>(off, E, M_cap, p, first, rows);
  if (E <= 4 * kWave) return find_expert<4>(off, E, M_cap, p, first, rows);
  return find_expert<kMaxExperts / kWave>(off, E, M_cap, p, first, rows);
}

// The groups' sums of one BM x BN tile, added in the order of the groups:
// element by element, whole rows of the tile side by side.
template <class C, WOut O>
__device__ __forceinline__ void add_groups(const WgradParams &p, const f32x4 (&acc)[C::NI][C::MI],
                                           lds_u8 *lds, int e, int col_k, int col_n, int group,
                                           int lane) {
  constexpr int P = C::PART_ROW;
  static_assert(C::BM * C::BN % C::THREADS == 0, "whole passes");
  lds_f32 *const part = (lds_f32 *)lds;
  __syncthreads();  // every group is done with its ring
  const int g = lane / 16, s = lane % 16;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < C::NI; ++ni)
      *(lds_f32x4 *)(part + (group * C::BM + mi * 16 + s) * P + ni * 16 + 4 * g) = acc[ni][mi];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::BM * C::BN / C::THREADS; ++i) {
    const int el = i * C::THREADS + (int)threadIdx.x, m = el / C::BN, n = el % C::BN;
    if (col_k + m >= p.K || col_n + n >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < C::R; ++r) v += part[(r * C::BM + m) * P + n];
    const size_t at = ((size_t)e * p.K + col_k + m) * p.N + col_n + n;
    if constexpr (O == WOut::BF16) {
      const bf16x2 w = __builtin_convertvector(f32x2{v, v}, bf16x2);
      ((uint16_t *)p.dB)[at] = __builtin_bit_cast(uint16_t, w[0]);
    } else if constexpr (O == WOut::AddF32) {
      ((float *)p.dB)[at] += v;
    } else {
      ((float *)p.dB)[at] = v;
    }
  }
}

template <class C, WOut O>
__global__ __launch_bounds__(C::THREADS, 2) void wgrad_kernel(WgradParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_dyn[];
  lds_u8 *const lds = (lds_u8 *)lds_dyn;
  // tiles of one expert in runs of per_xcd to an XCD (workgroup ids go
  // round-robin to the XCDs), k inner: a run's dC columns stay in one L2
  const int xcd = blockIdx.x % kRingXcds, i = blockIdx.x / kRingXcds;
  const int pos = i / p.per_xcd, local = xcd * p.per_xcd + i % p.per_xcd;
  if (local >= p.tiles) return;
  int r0, rows;
  const int e = scalar(wgrad_expert(p.off, p.E, p.M_cap, scalar(pos), &r0, &rows));
  const int KT_cols = cdiv(p.K, C::BM);
  const int nt = local / KT_cols, kt = local % KT_cols;
  if (O == WOut::AddF32 && rows == 0) return;  // nothing to add

  const int col_k = kt * C::BM, col_n = nt * C::BN;
  WgradTile<C> t;
  t.a_pitch = 2u * (uint32_t)p.K;
  t.b_pitch = 2u * (uint32_t)p.N;
  t.A = p.A + (size_t)r0 * t.a_pitch + 2 * (size_t)col_k;
  t.B = p.dC + (size_t)r0 * t.b_pitch + 2 * (size_t)col_n;
  t.a_cols = t.a_pitch - 2u * (uint32_t)col_k;
  t.b_cols = t.b_pitch - 2u * (uint32_t)col_n;
  t.rows = rows;
  const int tid = threadIdx.x;
  const int lane = tid % kWave, wave = scalar(tid / kWave) % C::WAVES;
  const int group = scalar(tid / kWave) / C::WAVES;  // takes slices group, group + R, ...
  const int wm0 = (wave / C::WN) * C::WTM, wn0 = (wave % C::WN) * C::WTN;
  const int a_off = wg_frag_off<C::A_ROW>(lane, wm0), b_off = wg_frag_off<C::B_ROW>(lane, wn0);

  f32x4 acc[C::NI][C::MI];
#pragma unroll
  for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi) acc[ni][mi] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int KT = max(cdiv(cdiv(rows, C::RB) - group, C::R), 0);  // this group's slices
  lds_u8 *const ring = lds + group * (C::S * C::STAGE);
#pragma unroll
  for (int k = 0; k < C::S - 1; ++k)
    if (k < KT) wg_issue<C>(t, ring + k * C::STAGE, k * C::R + group, wave, lane);
  int cur = 0, nxt = C::S - 1;
  for (int k = 0; k < KT; ++k) {
    // this wave's slices k + 1 .. min(k + S - 2, KT - 1) stay in flight
    wait_slices<C>(min(C::S - 2, KT - 1 - k));
    if constexpr (C::WAVES > 1) wg_barrier();
    wg_step<C>(acc, t, ring + cur * C::STAGE, ring + nxt * C::STAGE, k + C::S - 1, group, KT, wave,
               lane, a_off, b_off);
    cur = cur + 1 == C::S ? 0 : cur + 1;
    nxt = nxt + 1 == C::S ? 0 : nxt + 1;
  }
  if constexpr (C::R > 1) {
    add_groups<C, O>(p, acc, lds, e, col_k, col_n, group, lane);
    return;
  }

  const int n_in = p.N - col_n;
  constexpr size_t es = O == WOut::BF16 ? 2 : 4;
  void *const base = (char *)p.dB + (((size_t)e * p.K + col_k) * p.N + col_n) * es;
  // The gradient is written once and far larger than what was read: stores of
  // whole lines go out as streaming data, so that they do not displace the
  // rows that the tiles of an expert share (64 x 256 rows, K = 1024, N = 2688:
  // 250 -> 211 us in fp32, 167 -> 138 in bf16). Parts of lines are held back
  // in the cache until the rest comes (streamed they halve the write rate).
  constexpr bool kLines = C::NI % (O == WOut::BF16 ? 4 : 2) == 0;  // store_block's whole lines
  const bool whole = kLines && (p.N * es) % 128 == 0 && (uintptr_t)p.dB % 128 == 0;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi) {
    if constexpr (O == WOut::AddF32) {
      const buf_rsrc r = row_block(base, wm0 + mi * 16, p.K - col_k, p.N * es, col_n * es);
#pragma unroll
      for (int ni = 0; ni < C::NI; ++ni) {
        const int n = wn0 + ni * 16 + 4 * (lane / 16);
        const uint32_t at = n < n_in ? (uint32_t)(lane % 16) * (uint32_t)(p.N * es) + 4u * n : kOob;
        acc[ni][mi] += __builtin_bit_cast(f32x4, ld_buf16(r, at, 0));
      }
    }
    if (whole)
      store_block<C, O == WOut::BF16, kCacheStream>(acc, mi, base, wm0, wn0, lane, p.K - col_k, n_in,
                                                    p.N * es, col_n * es);
    else
      store_block<C, O == WOut::BF16>(acc, mi, base, wm0, wn0, lane, p.K - col_k, n_in, p.N * es,
                                      col_n * es);
    __builtin_amdgcn_sched_barrier(0);
  }
}

using W128 = WgradCfg<128, 256, 2, 2, 32, 3>;  // wave tile 64 x 128
using W64 = WgradCfg<64, 64, 2, 2, 32, 4>;     // wave tile 32 x 32
using W64R = WgradCfg<64, 64, 1, 1, 32, 2, 8>;  // 8 waves, each its own slices
using W32 = WgradCfg<32, 32, 1, 1, 32, 2, 16>;  // 16 of them
static_assert(2 * W128::LDS_BYTES <= 160 * 1024, "two workgroups a CU");

template <class C, WOut O>
static gg_status_t launch_wgrad(WgradParams p, hipStream_t stream) {
  constexpr int lds = C::LDS_BYTES;
  const long long tiles = ((p.K + (long long)C::BM - 1) / C::BM) * ((p.N + (long long)C::BN - 1) / C::BN);
  const long long per = (tiles + kRingXcds - 1) / kRingXcds;
  const long long grid = per * kRingXcds * p.E;
  if (!launch_fits(grid, C::THREADS)) return GG_ERR_UNSUPPORTED;
  if (!apart(span(p.dB, (long long)p.E * p.K, p.N, O == WOut::BF16 ? 2 : 4), span(p.A, p.M_cap, p.K, 2),
             span(p.dC, p.M_cap, p.N, 2), span(p.off, p.E + 1, 1, 4)))
    return GG_ERR_INVALID_VALUE;
  int dev = 0;
  if (!current_device(&dev)) return GG_ERR_LAUNCH;
  if (ring_launch<wgrad_kernel<C, O>>(dev, lds).err != hipSuccess) return GG_ERR_LAUNCH;
  p.tiles = (int)tiles;
  p.per_xcd = (int)per;
  return launch(wgrad_kernel<C, O>, dim3((unsigned)grid), C::THREADS, lds, stream, p);
}

template <WOut O>
static gg_status_t wgrad(const void *A, const void *dC, const int32_t *off, void *dB, int E, int K,
                         int N, int M_cap, void *stream) {
  if (off == nullptr || dB == nullptr || E < 1 || K < 1 || N < 1 || M_cap < 0)
    return GG_ERR_INVALID_VALUE;
  if (M_cap > 0 && (A == nullptr || dC == nullptr)) return GG_ERR_INVALID_VALUE;
  if (!is_aligned(off, 4) || !is_aligned(A, 16) || !is_aligned(dC, 16) || !is_aligned(dB, 16) ||
      K % 8 != 0 || N % 8 != 0)
    return GG_ERR_MISALIGNED;
  if (E > kMaxExperts || K > GG_MAX_K || N > GG_MAX_K || M_cap > INT32_MAX - 256)
    return GG_ERR_UNSUPPORTED;
  WgradParams p{static_cast<const char *>(A), static_cast<const char *>(dC), off, dB, E, K, N,
                M_cap, 0, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const long long big = (long long)E * ((K + 127) / 128) * ((N + 255) / 256);
  const long long mid = (long long)E * ((K + 63) / 64) * ((N + 63) / 64);
  // Large tiles where they give every CU one. Of the others, up to 64 tiles of
  // 64 x 64 leave most CUs idle for the length of the rows: smaller tiles whose
  // rows 16 waves share (us, W64 / W32: one expert of 16384 rows, 64 x 64: 100 /
  // 23; 1024 x 256: 104 / 58; four of 2000 rows, 256 x 256: 15.9 / 9.9; beyond
  // them, eight of 1000 rows, 256 x 512: 10.3 / 21). Up to one tile of 64 x 64 a
  // CU, eight waves share long groups, of 3000 rows and more (W64 / W64R: one of
  // 16384, 1024 x 1024: 100 / 64; one of 8000, 2048 x 512: 50.7 / 48.5; two of
  // 3200, 2776 x 104: 28.8 / 23.9; shorter ones, eight of 1000, 256 x 512: 10.3 /
  // 10.8; more tiles, four of 2000, 1024 x 512: 27.2 / 29.2). All of groups of
  // one size: the host knows M_cap only, so that spare rows count and the
  // longest group of a skewed batch does not.
  if (big >= 256) return launch_wgrad<W128, O>(p, s);
  if (mid <= 64) return launch_wgrad<W32, O>(p, s);
  if (mid <= 256 && M_cap / E >= 3000) return launch_wgrad<W64R, O>(p, s);
  return launch_wgrad<W64, O>(p, s);
}

}  // namespace gg

using namespace gg;

extern "C" gg_status_t gg_grouped_gemm_bf16_wgrad(const void *A, const void *dC,
                                                  const int32_t *group_offsets, float *dB,
                                                  int32_t accumulate, int32_t E, int32_t K,
                                                  int32_t N, int32_t M_cap, void *stream) {
  return accumulate ? wgrad<WOut::AddF32>(A, dC, group_offsets, dB, E, K, N, M_cap, stream)
                    : wgrad<WOut::F32>(A, dC, group_offsets, dB, E, K, N, M_cap, stream);
}

extern "C" gg_status_t gg_grouped_gemm_bf16_wgrad_bf16out(const void *A, const void *dC,
                                                          const int32_t *group_offsets, void *dB,
                                                          int32_t E, int32_t K, int32_t N,
                                                          int32_t M_cap, void *stream) {
  return wgrad<WOut::BF16>(A, dC, group_offsets, dB, E, K, N, M_cap, stream);
}
