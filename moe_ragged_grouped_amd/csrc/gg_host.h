// Host-side pieces the gradient and 4-bit entry points share: argument
// checks, and the launch limits of a persistent kernel per device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gg_schedule.h"
#include "grouped_gemm.h"

namespace gg {

constexpr int kRingXcds = 8;
constexpr int kHostMaxDevices = 64;

inline bool is_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A dispatch counts its threads along x in 32 bits.
inline bool launch_fits(long long workgroups, int threads) {
  return workgroups <= UINT32_MAX / (uint32_t)threads;
}

// Enqueues a kernel. The status is this launch's own: the runtime's last error
// may be an earlier call's, anyone's, and is left to whom it belongs.
template <class T>
struct as_declared {
  typedef T type;
};
template <class... P>
inline gg_status_t launch(void (*kernel)(P...), dim3 grid, int threads, int lds, void *stream,
                          typename as_declared<P>::type... args) {
  void *a[] = {(void *)&args...};
  if (hipLaunchKernel((const void *)kernel, grid, dim3((unsigned)threads), a, (size_t)lds,
                      static_cast<hipStream_t>(stream)) == hipSuccess)
    return GG_OK;
  (void)hipGetLastError();  // reported here, not by the next call of someone else
  return GG_ERR_LAUNCH;
}

inline bool valid_bm(int bm) {
  return bm == 0 || bm == 16 || bm == 32 || bm == 64 || bm == 128 || bm == 256;
}

// An array of a call: its memory. Tiles are stored while others still read, so
// an output that shares memory with anything else of the call would race.
struct Span {
  const void *p;
  unsigned long long bytes;
};
inline Span span(const void *p, long long n, long long m, long long bytes) {
  return Span{p, p == nullptr ? 0ull : (unsigned long long)n * (unsigned long long)m * bytes};
}
inline bool apart(Span a, Span b) {
  const unsigned long long x = (uintptr_t)a.p, y = (uintptr_t)b.p;  // sizes are below 2^60
  return a.bytes == 0 || b.bytes == 0 || x + a.bytes <= y || y + b.bytes <= x;
}
template <class... S>
inline bool apart(Span a, Span b, S... others) {
  return apart(a, b) && apart(a, others...);
}

// Groups, rows and tile height; upper bounds of the row tiles and of the tiles
// of a product with `cols` output columns (narrowest tiles: `narrow` columns).
// The limit is the forward products', 2^28 tiles of kTileN columns.
inline gg_status_t check_groups(const int32_t *off, int E, int cols, int M_cap, int bm, int narrow,
                                int *row_tiles, long long *tiles) {
  if (off == nullptr || E < 1 || cols < 1 || M_cap < 0 || !valid_bm(bm)) return GG_ERR_INVALID_VALUE;
  if (E > kMaxExperts) return GG_ERR_UNSUPPORTED;
  if (!is_aligned(off, 4)) return GG_ERR_MISALIGNED;
  const long long hmin = bm ? bm : 16;
  const long long m = (long long)M_cap / hmin + E;
  // tile ids, also of the narrowest tiles (at most kTileN / narrow times as
  // many), and rows + tile height must stay inside int32
  if (m * (((long long)cols + kTileN - 1) / kTileN) > (1LL << 28) || (long long)M_cap + 256 > INT32_MAX)
    return GG_ERR_UNSUPPORTED;
  *row_tiles = (int)m;
  *tiles = m * ((cols + (long long)narrow - 1) / narrow);
  return GG_OK;
}

// One workgroup per CU of the current device. The kernel's dynamic LDS limit
// is raised once per device and kernel.
struct RingLaunch {
  int grid = 0;
  hipError_t err = hipSuccess;
  // workgroups for at most `tiles` tiles: a multiple of the XCD count
  int workgroups(long long tiles) const {
    const long long g = tiles < grid ? tiles : grid;
    return (int)((g + kRingXcds - 1) / kRingXcds * kRingXcds);
  }
};

template <auto Kernel>
inline RingLaunch ring_launch(int dev, int lds) {
  static RingLaunch cache[kHostMaxDevices];
  static std::once_flag once[kHostMaxDevices];
  std::call_once(once[dev], [dev, lds]() {
    RingLaunch li;
    int cus = 0;
    li.err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (li.err == hipSuccess)
      li.err = hipFuncSetAttribute((const void *)Kernel,
                                   hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    li.grid = cus - cus % kRingXcds;
    if (li.grid < kRingXcds) li.grid = kRingXcds;
    cache[dev] = li;
  });
  return cache[dev];
}

inline bool current_device(int *dev) {
  return hipGetDevice(dev) == hipSuccess && *dev >= 0 && *dev < kHostMaxDevices;
}

}  // namespace gg
