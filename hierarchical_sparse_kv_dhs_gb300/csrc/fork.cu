// Copies within the pool: a request's rows into another request slot (fork),
// pages into lower slots (compaction), and emptied hot caches (release).
//
// Pure copies, bound by memory: every row is read and written once, four rows
// at a time by one warp in 16-byte pieces a lane, and loads and stores bypass
// the caches' recency (nothing is read twice).  A fork of 4 x 32768 rows moves
// 302 MB in 51 us, 5.9 TB/s, 0.88 of the measured copy; a compaction that
// moves 1600 pages of 64 rows, 235 MB in 35 us, 6.7 TB/s, the copy's rate.
//
// The page maps change with the copies: the kernels write the entries
// themselves, from slots that travel in their parameters, so that no upload
// of a map precedes them.
#include <algorithm>

#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kForkThreads = 256, kForkWarps = kForkThreads / 32;

template <int SOURCES, int SLOTS>
struct ForkParams {
  ForkCommon c;
  ForkSource s[SOURCES];
  int32_t slots[SLOTS];
};
static_assert(sizeof(ForkParams<kForkSourcesMax, 1>) <= 32764, "fork source table too large");
static_assert(sizeof(ForkParams<kForkSourcesSome, kForkSlotsMax>) <= 32764, "fork slots too many");

constexpr int kMoveRunsMax = 1280;
struct MoveRun {
  int64_t unit0;          // first row of the run among the launch's
  int64_t map;            // first map entry
  int32_t from, to;       // first slots
};
struct MoveParams {
  uint8_t* opt;
  int32_t* map;
  int64_t n_units;
  int32_t row_bytes, page_shift, n_runs, pad;
  MoveRun r[kMoveRunsMax];
};
static_assert(sizeof(MoveParams) <= 32764, "move run table too large");

constexpr int kRows = 4;  // rows of a warp at a time: as many loads in flight a lane

// Row i from from[i] to to[i], nothing where from[i] is null.
__device__ __forceinline__ void copy_rows(uint8_t* const (&to)[kRows],
                                          const uint8_t* const (&from)[kRows], int bytes, int lane) {
  for (int k = lane * 16; k < bytes; k += 512) {
    uint4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (from[i]) v[i] = __ldcs(reinterpret_cast<const uint4*>(from[i] + k));
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (from[i]) __stcs(reinterpret_cast<uint4*>(to[i] + k), v[i]);
  }
}

// One warp per kRows rows; row units of a source: history, tail ring, hot slots.
// SLOTS: the child's page slots are in the parameters and its map entries are
// written here; else they are in the device's map already.
template <int SOURCES, int SLOTS>
__global__ void __launch_bounds__(kForkThreads)
    fork_kernel(const __grid_constant__ ForkParams<SOURCES, SLOTS> P) {
  const ForkCommon& c = P.c;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kForkWarps;
  if constexpr (SLOTS > 1) {
    const int threads = gridDim.x * kForkThreads;
    for (int n = 0; n < c.n_sources; ++n) {
      const ForkSource& s = P.s[n];
      for (int q = blockIdx.x * kForkThreads + threadIdx.x; q < c.Pmax; q += threads)
        c.map[(size_t)s.to * c.Pmax + q] = q < s.complete ? P.slots[s.slot0 + q] : -1;
    }
  }
  int n = 0;
  const size_t rb = c.row_bytes;
  auto row = [&](int64_t u, const uint8_t*& from, uint8_t*& to) {
    from = nullptr;
    if (u >= c.n_units) return;
    while (n + 1 < c.n_sources && P.s[n + 1].unit0 <= u) ++n;
    const ForkSource& s = P.s[n];
    int64_t r = u - s.unit0;
    const int64_t hist = s.host_from ? s.L : 0;
    if (r < hist) {
      const int64_t page = r >> c.page_shift, in = r & ((1 << c.page_shift) - 1);
      int32_t a = -1, b = -1;
      if (page < s.complete) {
        a = c.map[(size_t)s.from * c.Pmax + page];
        b = SLOTS > 1 ? P.slots[s.slot0 + page] : c.map[(size_t)s.to * c.Pmax + page];
      }
      from = a >= 0 ? c.opt + (((size_t)a << c.page_shift) + in) * rb : s.host_from + r * rb;
      to = b >= 0 ? c.opt + (((size_t)b << c.page_shift) + in) * rb : s.host_to + r * rb;
    } else if ((r -= hist) < c.T) {
      if (r >= s.L) return;  // ring slots that hold no row yet
      from = c.tail + ((size_t)s.from * c.T + r) * rb;
      to = c.tail + ((size_t)s.to * c.T + r) * rb;
    } else {
      r -= c.T;
      const int32_t tag = c.tags[(size_t)s.from * c.B + r];
      if (lane == 0) {
        c.tags[(size_t)s.to * c.B + r] = tag;
        c.stamps[(size_t)s.to * c.B + r] = c.stamps[(size_t)s.from * c.B + r];
      }
      if (tag < 0) return;
      from = c.hot + ((size_t)s.from * c.B + r) * rb;
      to = c.hot + ((size_t)s.to * c.B + r) * rb;
    }
  };
  for (int64_t u = ((int64_t)blockIdx.x * kForkWarps + (threadIdx.x >> 5)) * kRows; u < c.n_units;
       u += warps * kRows) {
    const uint8_t* from[kRows];
    uint8_t* to[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) row(u + i, from[i], to[i]);
    copy_rows(to, from, c.row_bytes, lane);
  }
}

// One warp per kRows rows of the moved pages; the warp of a page's first row writes
// its map entry.  Pages move down into slots that no page of the launch
// leaves, so rows never overlap.
__global__ void __launch_bounds__(kForkThreads)
    move_kernel(const __grid_constant__ MoveParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kForkWarps;
  int n = 0;
  for (int64_t u = ((int64_t)blockIdx.x * kForkWarps + (threadIdx.x >> 5)) * kRows; u < P.n_units;
       u += warps * kRows) {
    const uint8_t* from[kRows];
    uint8_t* to[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      from[i] = nullptr;
      if (u + i >= P.n_units) continue;
      while (n + 1 < P.n_runs && P.r[n + 1].unit0 <= u + i) ++n;
      const MoveRun& run = P.r[n];
      const int64_t r = u + i - run.unit0;
      const int64_t page = r >> P.page_shift, in = r & ((1 << P.page_shift) - 1);
      if (in == 0 && lane == 0) P.map[run.map + page] = run.to + (int32_t)page;
      from[i] = P.opt + ((((size_t)run.from + page) << P.page_shift) + in) * P.row_bytes;
      to[i] = P.opt + ((((size_t)run.to + page) << P.page_shift) + in) * P.row_bytes;
    }
    copy_rows(to, from, P.row_bytes, lane);
  }
}

__global__ void clear_hot_kernel(int32_t* tags, uint32_t* stamps, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  tags[i] = -1;
  stamps[i] = 0;
}

template <int SOURCES, int SLOTS>
cudaError_t launch_fork_t(const ForkCommon& c, const ForkSource* sources, int n_sources,
                          const int32_t* slots, int n_slots, int sms, cudaStream_t stream) {
  ForkParams<SOURCES, SLOTS> P;
  P.c = c;
  P.c.n_sources = n_sources;
  int64_t units = 0;
  for (int i = 0; i < n_sources; ++i) {
    P.s[i] = sources[i];
    P.s[i].unit0 = units;
    units += (sources[i].host_from ? sources[i].L : 0) + c.T + c.B;
  }
  P.c.n_units = units;
  if (SLOTS > 1) std::copy(slots, slots + n_slots, P.slots);
  const int64_t blocks =
      std::min<int64_t>(sms * 8, (units + kForkWarps * kRows - 1) / (kForkWarps * kRows));
  fork_kernel<SOURCES, SLOTS><<<(int)blocks, kForkThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_moves(uint8_t* opt, int32_t* map, int row_bytes, int page_shift,
                           const PageRun* runs, int n_runs, int sms, cudaStream_t stream) {
  MoveParams P;
  P.opt = opt;
  P.map = map;
  P.row_bytes = row_bytes;
  P.page_shift = page_shift;
  P.n_runs = n_runs;
  P.n_units = 0;
  for (int i = 0; i < n_runs; ++i) {
    P.r[i] = {P.n_units, runs[i].map, runs[i].from, runs[i].to};
    P.n_units += (int64_t)runs[i].pages << page_shift;
  }
  const int64_t blocks = std::min<int64_t>(sms * 8, (P.n_units + kForkWarps * kRows - 1) / (kForkWarps * kRows));
  move_kernel<<<(int)blocks, kForkThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fork(const ForkCommon& c, const ForkSource* sources, int n_sources,
                        const int32_t* slots, int n_slots, int sms, cudaStream_t stream) {
  if (n_sources <= 0) return cudaSuccess;
  if (n_sources > kForkSourcesMax) return cudaErrorInvalidValue;
  if (!slots) return launch_fork_t<kForkSourcesMax, 1>(c, sources, n_sources, slots, 0, sms, stream);
  if (n_sources > kForkSourcesSome || n_slots > kForkSlotsMax) return cudaErrorInvalidValue;
  // the whole table travels with every launch: a small one for small requests
  // (a request of 4096 rows released and forked anew 21 us, with the large
  // table 24)
  if (n_sources <= 8 && n_slots <= 512)
    return launch_fork_t<8, 512>(c, sources, n_sources, slots, n_slots, sms, stream);
  return launch_fork_t<kForkSourcesSome, kForkSlotsMax>(c, sources, n_sources, slots, n_slots, sms,
                                                        stream);
}

cudaError_t launch_page_runs(uint8_t* opt, int32_t* map, int row_bytes, int page_shift,
                             const PageRun* runs, int64_t n_runs, int sms, cudaStream_t stream) {
  for (int64_t b = 0; b < n_runs; b += kMoveRunsMax) {
    const int n = (int)std::min<int64_t>(kMoveRunsMax, n_runs - b);
    cudaError_t e = launch_moves(opt, map, row_bytes, page_shift, runs + b, n, sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_clear_hot(int32_t* tags, uint32_t* stamps, int64_t n, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  clear_hot_kernel<<<(int)((n + 255) / 256), 256, 0, stream>>>(tags, stamps, n);
  return cudaGetLastError();
}

}  // namespace dhs
