// Attention over rows of the pool: located rows (a location vector) or a
// source's history (tail ring, optional pages, host copy), read in place.
//
// "Adaptive DHiSparse", How it works / Memory split: sparse attention reads
// the selected rows.  With x_j, y_j the key and the value of row j and s_j =
// scale (q . x_j), one pass keeps a reference m, l = sum exp(s_j - m) and
// o = sum exp(s_j - m) y_j.  m follows the running maximum: it moves only
// when a score passes it by more than kSlack (a factor of 2^8, far inside
// float and 16-bit range), and then l and o are scaled by exp(m_old - m_new).
// out = o / l, log-sum = m + ln l.
//
// Both products run on the 5th-generation tensor cores with the rows as the
// M side, because few query heads share a row and M is 64 or 128 there:
//   S^T[128 rows x N] = X[128 x dk] . Q^T      (tile of 128 rows, N columns)
//   O^T[dv x N]      += Y^T[dv x 128] . P^T    (M = 128 value elements)
// A column is one (query, head) pair sharing the rows: up to 64 of them.
// (A product takes 48 cycles for N = 16, 55 for N = 64: narrow blocks cost
// nearly as much each, so columns that share rows share a block.)  The tile
// of rows is staged once in shared memory and feeds both products (as a
// K-major operand first, as an M-major one then); where keys and values are
// the same bytes (one latent row) they are loaded once.  S^T, O^T stay in
// tensor memory; a thread owns one row of S^T, so weights need no shuffles,
// and the maximum is only reduced across rows when m moves.
//
// Roundings: scores, m, l and o are 32-bit; the weights alone are rounded to
// the rows' 16-bit type, as the second product's operand, while l sums them
// unrounded: an error of half a unit of each weight, of the size of the
// output's own rounding.  m being up to 2^8 behind the maximum costs an f16
// weight nothing (2^8 < 65504) and gives small ones 8 bits more above zero.
//
// A block has 8 softmax warps, 4 loading warps, an issuing warp, a warp that
// finds the block's segments ahead and two that find the rows' addresses,
// joined by mbarriers.  Each role's code is kept short, loops rolled: a
// launch starts with cold instruction caches, and a kernel of 167 KB instead
// of 70 spent 10 us there (one query over 256 rows 16.4 us -> 14.4; grouped
// verify blocks, whose loading warps then also found their rows, 78 -> 54).
//
// Rows lie at arbitrary addresses of four memories, so loads are 16-byte
// asynchronous copies into the swizzled layout, at most 27 bytes a cycle and
// SM (7.9 TB/s).  Tensor gathers of four rows reach twice that, but take a
// map for each memory and 65 cycles a warp each; with 64-row tiles, which
// let scores run ahead, they lost everywhere (500K rows 126 -> 150 us, 64
// verify blocks 265 -> 287): less of the ring was left for rows in flight.
//
// The launch is one block per SM (its shared memory is filled by rows in
// flight); all tiles of all jobs (a job: one item, kv head and block of
// columns) are dealt out in order, evenly; a job cut by a block's boundary
// leaves (m, l, o) parts that merge_kernel joins in block order, so that a
// call's bits do not depend on timing.
//
// What bounds it (16 query heads on a 1152-byte latent row unless said):
// 64 verify blocks of 8 queries over 2048 rows each, 234 us: every query's
// rows staged once, 1.21 GB through the loading warps at 5.2 TB/s (DRAM
// reads 409 MB, each distinct row once).  One token over 512K rows, 115 us:
// 590 MB of DRAM reads at 5.8 TB/s between a start of 4 us and a merge of 10.
// 128 heads, 158 us: one tile at a time is resident beside 64 queries, so
// that loads, scores, weights and sums follow each other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kTile = 128;                 // rows per tile
constexpr int kSoftThreads = 256, kLoadThreads = 128;
constexpr int kIssueWarp = (kSoftThreads + kLoadThreads) / 32, kFindWarp = kIssueWarp + 1;
constexpr int kRowWarp = kFindWarp + 1, kRowThreads = 64;
constexpr int kThreads = 32 * kRowWarp + kRowThreads;
constexpr int kChunk = kTile * 128;        // bytes of a 64-element column chunk of a tile
constexpr int kUnit = 2 * kChunk;          // a value unit: 128 elements
constexpr int kMaxK = 12, kMaxV = 8;       // ring slots at most
constexpr int kSegments = 4;               // segments found ahead
constexpr int kRowSlots = 2;               // tiles whose row addresses are found ahead
constexpr float kSlack = 8.f;              // log2 units

// How a launch's row slices are staged.
struct Plan {
  int32_t shared;        // the value is the key's beginning: loaded once
  int32_t key_chunks;    // 64-element chunks of a key
  int32_t only_chunks;   // of them in the key ring (all, unless shared)
  int32_t units;         // value units
  int32_t kslots, vslots;
  int32_t alias;         // the weights take the key ring's only slot (shared only)
  uint32_t off_q, off_p, off_k, off_v;  // from the aligned shared-memory base
  uint32_t smem;
};

template <int MAXI>
struct AttendParams {
  AttendCommon c;
  Plan plan;
  int32_t first[MAXI];   // first tile of each item, past the last one INT32_MAX
  AttendItem items[MAXI];
};
static_assert(sizeof(AttendParams<kAttendItemsLarge>) <= 32764, "attend item table too large");

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait (a poll that fails takes 4 us).  A wait that runs out raises
// *gave_up; every later wait of the block then falls through, so that all its
// warps still reach their end, on wrong data: the launch's status says so.
// What lies behind a wait that fell through may not have been written, so no
// address is taken from there: a segment is used only if gave_up is still
// down after the wait for it, and not replaced after a wait that gave up; the
// table of rows holds nothing but rows and nulls from the start.
struct Patience {
  volatile uint32_t* gave_up;
  uint32_t polls;
};
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, const Patience& until) {
#pragma unroll 1
  for (uint32_t n = 0; !bar_try(bar, parity); ++n) {
    if (*until.gave_up) return;
    if (n >= until.polls) *until.gave_up = 1;
  }
}

// The same by whole warps, together again afterwards: what follows may be an
// instruction that a warp executes as one (block barriers, tcgen05 loads).
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, const Patience& until) {
  bar_wait(bar, parity, until);
  __syncwarp();
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One of the warp's threads, the same one each time.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(p)::"memory");
  return p != 0;
}

// D += A B (D = A B unless add) with operand descriptors given as halves: the
// high one is fixed for a kind of operand, the low one moves with the address.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t ahi, uint32_t b, uint32_t bhi,
                                    uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\n"
      "mov.b64 x, {%1, %2};\nmov.b64 y, {%3, %4};\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}\n" ::"r"(d),
      "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// Arrives on `bar` once every product issued so far is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Eight columns of the warp's 32 lanes.  The values may be used only behind
// tm_wait, which every later use depends on.
__device__ __forceinline__ void tm_load8(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7])
      : "r"(addr)
      : "memory");
}

template <int C>
__device__ __forceinline__ void tm_wait(float (&v)[C]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < C; ++k) asm volatile("" : "+f"(v[k]));
}

template <int C>
__device__ __forceinline__ void tm_load(uint32_t addr, float (&v)[C]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < C; k += 8) tm_load8(addr + k, v + k);
  tm_wait(v);
}

template <int C>
__device__ __forceinline__ void tm_store(uint32_t addr, const float (&v)[C]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < C; k += 8)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(v[k]),
        "f"(v[k + 1]), "f"(v[k + 2]), "f"(v[k + 3]), "f"(v[k + 4]), "f"(v[k + 5]), "f"(v[k + 6]),
        "f"(v[k + 7]), "r"(addr + k)
        : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool named_or(int id, int threads, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\n"
      "bar.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory operand descriptor.  Low half: start and leading stride
// (bytes); high half: 8-row stride, format version, swizzle (2 = 128 B, 4 =
// 64 B, 6 = 32 B rows).
__device__ __forceinline__ uint32_t operand_lo(uint32_t addr, uint32_t lead) {
  return (addr & 0x3FFFF) >> 4 | (lead >> 4) << 16;
}
__host__ __device__ constexpr uint32_t operand_hi(uint32_t eight, uint32_t swizzle) {
  return eight >> 4 | 1u << 14 | swizzle << 29;
}

// Eight values of each lane reduced over the warp: lane i gets the result of
// value i & 7.
template <class F>
__device__ __forceinline__ float fold8(const float* in, int lane, F f) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = in[k];
#pragma unroll
  for (int w = 4; w; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float send = up ? v[k] : v[k + w], keep = up ? v[k + w] : v[k];
      v[k] = f(keep, __shfl_xor_sync(~0u, send, w));
    }
  }
  v[0] = f(v[0], __shfl_xor_sync(~0u, v[0], 8));
  return f(v[0], __shfl_xor_sync(~0u, v[0], 16));
}

// ------------------------------------------------------------------ jobs

// A block's share of one job: tiles [t0, t1) of item `it`, columns [col0,
// col0 + cols) of kv head g (column = query * group + head within the group
// for a history; located items: query qbase, column = head).
struct Segment {
  AttendItem it;     // a copy: the table is indexed constant memory, slow to read
  int32_t tiles;     // of the whole job
  int32_t t0, t1;    // the segment's tiles before clipping to visible rows
  int32_t g, qbase, col0, cols;
  int64_t lo, hi;    // rows any of the columns may see, relative to it->first
  int32_t v0, v1;    // tiles that hold some of them (v0 >= v1: none)
  __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Rows [lo, hi) (relative to it.first) that query i of a history item sees.
__device__ __forceinline__ void query_rows(const AttendItem& it, int i, int64_t& lo, int64_t& hi) {
  const int64_t L = it.first + it.len;
  lo = it.range ? max((int64_t)it.range[2 * i] - it.first, (int64_t)0) : 0;
  hi = (it.range ? min((int64_t)it.range[2 * i + 1], L) : L - it.Q + 1 + i) - it.first;
}

// The last item whose first tile is <= t (an item without jobs has none).
template <int MAXI>
__device__ __forceinline__ int item_at(const AttendParams<MAXI>& P, int32_t t) {
  const int32_t* first = P.first + (threadIdx.x & 31);
  int32_t x[(MAXI + 31) / 32];
#pragma unroll
  for (int k = 0; k < (MAXI + 31) / 32; ++k)
    x[k] = 32 * k + (threadIdx.x & 31) < MAXI ? first[32 * k] : INT32_MAX;
  int n = 0;
#pragma unroll
  for (int k = 0; k < (MAXI + 31) / 32; ++k) n += __popc(__ballot_sync(~0u, x[k] <= t));
  return n - 1;
}

// The segment that begins at tile `t` of the launch and ends before `te`.
// Called by whole warps.
template <int MAXI>
__device__ Segment segment_at(const AttendParams<MAXI>& P, int32_t t, int32_t te) {
  const AttendCommon& c = P.c;
  __syncwarp();
  Segment s;
  s.it = P.items[item_at(P, t)];
  const AttendItem& it = s.it;
  const bool located = it.loc != nullptr;
  s.tiles = it.tiles;
  const int32_t job = (t - it.tile0) / it.tiles;
  s.t0 = (t - it.tile0) - job * it.tiles;
  s.t1 = min(it.tiles, s.t0 + (te - t));
  const int32_t columns = located ? c.group : it.Q * c.group;
  const int32_t query = job / it.blocks;
  s.col0 = (job - query * it.blocks) * it.width;
  s.cols = min(it.width, columns - s.col0);
  s.qbase = query / c.kv;
  s.g = query - s.qbase * c.kv;
  s.lo = 0;
  s.hi = it.len;
  if (!located) {
    const int q0 = s.col0 / c.group, q1 = (s.col0 + s.cols - 1) / c.group;
    int64_t lo = it.len, hi = 0;
#pragma unroll 1
    for (int i = q0 + (threadIdx.x & 31); i <= q1; i += 32) {
      int64_t x, y;
      query_rows(it, i, x, y);
      if (x < y) {
        lo = min(lo, x);
        hi = max(hi, y);
      }
    }
#pragma unroll 1
    for (int w = 16; w; w >>= 1) {
      lo = min(lo, (int64_t)__shfl_xor_sync(~0u, (long long)lo, w));
      hi = max(hi, (int64_t)__shfl_xor_sync(~0u, (long long)hi, w));
    }
    s.lo = lo;
    s.hi = hi;
  }
  s.v0 = max(s.t0, (int32_t)(s.lo / kTile));
  s.v1 = min(s.t1, (int32_t)((s.hi + kTile - 1) / kTile));
  return s;
}

// First tile of block b's share of what the waves leave.
__host__ __device__ __forceinline__ int32_t first_tile(const AttendCommon& c, int32_t b) {
  return c.waved + b * c.share + min(b, c.extra);
}

// A block's segments: first a whole job of each wave (jobs of equal length go
// to the blocks in order, so that blocks running side by side work on
// neighbouring jobs, which read the same rows), then its even share of the
// tiles that are left.
struct Walk {
  int32_t wave, t, te;
};
template <int MAXI>
__device__ __forceinline__ Walk first_of(const AttendParams<MAXI>& P) {
  const AttendCommon& c = P.c;
  return {0, first_tile(c, blockIdx.x), first_tile(c, blockIdx.x + 1)};
}
template <int MAXI>
__device__ bool next_segment(const AttendParams<MAXI>& P, Walk& w, Segment& s) {
  const AttendCommon& c = P.c;
  int32_t t = w.t, te = w.te;
  const bool wave = w.wave < c.waves;
  if (wave) {
    t = (int32_t)((w.wave * gridDim.x + blockIdx.x) * c.job_tiles);
    te = t + c.job_tiles;
    ++w.wave;
  } else if (t >= te) {
    return false;
  }
  s = segment_at(P, t, te);
  if (!wave) w.t += s.t1 - s.t0;
  return true;
}

// Finding row j of a job takes up to two dependent loads: a list position
// (union items), then the location or (histories) the page's slot.  They are
// split so that a row thread can keep them in flight: `row_index` two
// tiles ahead, `row_word` one tile ahead, `row_of` when the tile is loaded.
__device__ __forceinline__ int32_t row_index(const Segment& s, int64_t j) {
  const AttendItem& it = s.it;
  if (!it.index || j < s.lo || j >= s.hi) return -1;
  return __ldg(it.index + (int64_t)s.qbase * it.len + j);
}

__device__ __forceinline__ uint32_t row_word(const AttendCommon& c, const Segment& s, int64_t j,
                                             int32_t index) {
  const AttendItem& it = s.it;
  if (j < s.lo || j >= s.hi) return kNoLoc;
  if (it.loc) {
    if (!it.index) return __ldg(it.loc + (int64_t)s.qbase * it.len + j);
    if (index < 0) return kNoLoc;
    // a position past the list: a location of no tier
    return index < (int64_t)it.Q * it.len ? __ldg(it.loc + index) : 3u << 30;
  }
  const int64_t page = (it.first + j) >> c.page_shift;
  return page < it.complete ? (uint32_t)__ldg(c.map + (size_t)it.pair * c.Pmax + page) : kNoLoc;
}

// Address of row j of the job, or null when there is none.
__device__ __forceinline__ const uint8_t* row_of(const AttendCommon& c, const Segment& s, int64_t j,
                                                 uint32_t word) {
  const AttendItem& it = s.it;
  if (j < s.lo || j >= s.hi) return nullptr;
  if (it.loc) {
    if (word >= kEndLoc) return nullptr;
    const uint32_t tier = word >> 30, x = word & 0x3FFFFFFFu;
    const uint32_t rows = tier == kTierTail ? c.tail_rows : tier == kTierOpt ? c.opt_rows
                          : tier == kTierHot ? c.hot_rows : 0;
    if (x >= rows) {
      atomicOr(c.status, kStatusEloc);
      return nullptr;
    }
    const uint8_t* base = tier == kTierTail ? c.tail : tier == kTierOpt ? c.opt : c.hot;
    return base + (size_t)x * c.row_bytes;
  }
  const int64_t r = it.first + j;
  if (r >= it.first + it.len - c.T)
    return c.tail + ((size_t)it.pair * c.T + (uint32_t)r % (uint32_t)c.T) * c.row_bytes;
  if ((int32_t)word >= 0)
    return c.opt + (((size_t)word << c.page_shift) + (r & ((1 << c.page_shift) - 1))) * c.row_bytes;
  return it.host + (size_t)r * c.row_bytes;
}

// ------------------------------------------------------------------ kernel

constexpr int kUnusedBars = 8 - 2 * kRowSlots;
struct Control {
  uint64_t kfull[kMaxK], kempty[kMaxK], vfull[kMaxV], vempty[kMaxV];
  uint64_t qfull, qempty, sfull[2], pfull, odone, oempty, rfull[kRowSlots], rempty[kRowSlots], drain;
  uint64_t segfull[kSegments], segempty[kSegments];
  uint64_t unused[kUnusedBars];  // to 64: two barriers a lane
  Segment seg[kSegments];  // from the finding warp to the others
  const uint8_t* row[kRowSlots][kTile];
  int64_t out_off[64];
  int32_t lse_at[64];
  int32_t col_lo[64], col_hi[64];
  alignas(16) float m[64], base[64], fac[64];
  float part[4][64];
  uint32_t odd[4];    // rows of the tile whose products are taken by hand
  const uint8_t* odd_row;
  uint32_t o_begun;   // the segment's sums hold such products before the first tile's
  uint32_t tmem;
  volatile uint32_t gave_up;
};
// Places of the single barriers in Control's order
constexpr int kBarQfull = 2 * kMaxK + 2 * kMaxV, kBarPfull = kBarQfull + 4,
              kBarOempty = kBarQfull + 6, kBarRfull = kBarQfull + 7,
              kBarRempty = kBarRfull + kRowSlots, kBarDrain = kBarRempty + kRowSlots,
              kBarSegempty = kBarDrain + 1 + kSegments, kBarriers = 64;
static_assert(kBarSegempty + kSegments + kUnusedBars == kBarriers, "barrier table");
constexpr uint32_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

// Parity bookkeeping of a ring of slots.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Two buffers of scores, then up to four units of sums.
__host__ __device__ constexpr uint32_t tmem_columns(int n) {
  return 6 * n <= 128 ? 128 : 6 * n <= 256 ? 256 : 512;
}
// Bytes of one row of weights, the swizzle of that row width, and its 8-row stride.
__host__ __device__ constexpr int weight_row(int n) { return n <= 16 ? 32 : n <= 32 ? 64 : 128; }
__host__ __device__ constexpr uint32_t weight_swizzle(int n) { return n <= 16 ? 6 : n <= 32 ? 4 : 2; }

// Loading warps: queries once per segment, rows tile by tile.
template <int N, bool SHARED, int MAXI>
__device__ void load_rows(const AttendParams<MAXI>& P, uint8_t* sm, Control& ctl, int tid) {
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const Plan& pl = P.plan;
  const bool alias = SHARED && pl.alias;
  const uint32_t base = smem_u32(sm);
  Ring kr, vr, rr;
  uint32_t qphase = 0;
  auto wait_empty = [&](uint32_t bar, uint32_t parity) { warp_wait(bar, parity, until); };
  // The slot's barrier gets this thread's arrival when its copies so far have
  // landed.  The issuing warp makes them visible to the tensor cores: a proxy
  // fence here would wait for every copy in flight.
  auto launch = [&](uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
  };
  const int piece = tid & 7, r0 = tid >> 3;  // rows r0 + 16 i
  bool first = true;
  Ring seg;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    if (__any_sync(~0u, ctl.gave_up) || !s.cols) break;
    const int32_t v0 = s.v0, v1 = s.v1;
    const AttendItem& it = s.it;
    // Queries: [chunk][column][128 B], zeros past the key and the columns.
    // Loaded behind the first tile's key chunks: the segment before may still
    // hold the buffer, and does so about as long as the slots of its rows.
    auto load_queries = [&] {
      if (!first) {
        warp_wait(smem_u32(&ctl.qempty), qphase, until);
        qphase ^= 1;
      }
      first = false;
      const bool aligned = !(((uintptr_t)it.q | c.q_qs | c.q_hs) & 15);
#pragma unroll 1
      for (int col = tid >> 3; col < N; col += kLoadThreads / 8) {
        const bool on = col < s.cols;
        const int qc = s.col0 + min(col, s.cols - 1);
        const int qi = it.loc ? s.qbase : qc / c.group;
        const int h = s.g * c.group + (it.loc ? qc : qc % c.group);
        const uint8_t* src = it.q + qi * c.q_qs + h * c.q_hs;
        const uint32_t dst = pl.off_q + col * 128 + ((piece ^ (col & 7)) << 4);
#pragma unroll 1
        for (int ch = 0; ch < pl.key_chunks; ++ch) {
          const int el = ch * 64 + piece * 8;
          const bool in = on && el < c.dk;
          if (aligned) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             base + dst + ch * (N * 128)),
                         "l"(in ? src + 2 * el : c.tail), "r"(in ? 16 : 0)
                         : "memory");
          } else {
            const uint16_t* s2 = reinterpret_cast<const uint16_t*>(src + 2 * el);
            uint32_t w[4] = {};
            if (in)
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = s2[2 * k] | (uint32_t)s2[2 * k + 1] << 16;
            *reinterpret_cast<uint4*>(sm + dst + ch * (N * 128)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (aligned) launch(smem_u32(&ctl.qfull));
      else bar_arrive(smem_u32(&ctl.qfull));
    };

    const uint32_t key_at = c.key_off + s.g * c.key_stride;
    const uint32_t val_at = c.val_off + s.g * c.val_stride;
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile) {
      warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
      const uint8_t* row[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = ctl.row[rr.slot][r0 + 16 * i];
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
      rr.next(kRowSlots);
      // one 64-element chunk of the 128 rows: element el.. of a slice of
      // `n` elements at byte `at` of each row
      auto chunk = [&](uint32_t dst, uint32_t at, int el, int n) {
        const int e = el + piece * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 16 * i;
          const bool on = row[i] && e < n;
          const uint8_t* src = on ? row[i] + at + 2 * e : c.tail;
          asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                           dst + r * 128 + ((piece ^ (r & 7)) << 4)),
                       "l"(src), "r"(on ? 16 : 0)
                       : "memory");
        }
      };
      // Key chunks, then value units; where the weights take the key chunk's
      // slot, which is then free last, the units first.
      const int c0 = pl.key_chunks - pl.only_chunks, items = pl.only_chunks + pl.units;
#pragma unroll 1
      for (int i = 0; i < items; ++i) {
        const bool key = alias ? i >= pl.units : i < pl.only_chunks;
        // a slot that this tile itself has to free needs the queries
        if (tile == v0 && i == (alias ? 0 : min(pl.kslots, pl.only_chunks))) load_queries();
        if (key) {
          wait_empty(smem_u32(&ctl.kempty[kr.slot]), kr.phase ^ 1);
          chunk(base + pl.off_k + kr.slot * kChunk, key_at, (c0 + (alias ? 0 : i)) * 64, c.dk);
          launch(smem_u32(&ctl.kfull[kr.slot]));
          kr.next(pl.kslots);
        } else {
          const int el = (alias ? i : i - pl.only_chunks) * 128, n = SHARED ? c.dk : c.dv;
          const uint32_t at = SHARED ? key_at : val_at, dst = base + pl.off_v + vr.slot * kUnit;
          wait_empty(smem_u32(&ctl.vempty[vr.slot]), vr.phase ^ 1);
          chunk(dst, at, el, n);
          if (el + 64 < n) chunk(dst + kChunk, at, el + 64, n);
          launch(smem_u32(&ctl.vfull[vr.slot]));
          vr.next(pl.vslots);
        }
      }
    }
    __syncwarp();
    if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Finding warp: the block's segments, ahead of the others, who read them from
// shared memory.  One without columns ends the walk.  The first one is found
// while the block sets up.
template <int MAXI>
__device__ void find_segments(const AttendParams<MAXI>& P, Control& ctl) {
  const Patience until{&ctl.gave_up, P.c.polls};
  Ring seg;
  Walk w = first_of(P);
  bool more = true;
#pragma unroll 1
  for (bool begin = true; more; begin = false) {
    Segment s;
    more = next_segment(P, w, s);
    if (begin) __syncthreads();
    if (!more) s.cols = 0;
    warp_wait(smem_u32(&ctl.segempty[seg.slot]), seg.phase ^ 1, until);
    if (__any_sync(~0u, ctl.gave_up)) break;  // the slot may still be in use
    if (elected()) {
      ctl.seg[seg.slot] = s;
      bar_arrive(smem_u32(&ctl.segfull[seg.slot]));
    }
    seg.next(kSegments);
  }
}

// Row warps: the addresses of every tile's rows, ahead of the loading warps.
template <int MAXI>
__device__ void find_rows(const AttendParams<MAXI>& P, Control& ctl, int tid) {
  constexpr int R = kTile / kRowThreads;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  Ring seg, rr;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment s = ctl.seg[seg.slot];
    if (__any_sync(~0u, ctl.gave_up) || !s.cols) break;
    int64_t j = (int64_t)s.v0 * kTile + tid;
    uint32_t word[R];
    int32_t index[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t i = j + k * kRowThreads;
      index[k] = row_index(s, i);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t i = j + k * kRowThreads;
      word[k] = row_word(c, s, i, index[k]);
      index[k] = row_index(s, i + kTile);
    }
#pragma unroll 1
    for (int tile = s.v0; tile < s.v1; ++tile, j += kTile) {
      warp_wait(smem_u32(&ctl.rempty[rr.slot]), rr.phase ^ 1, until);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t i = j + k * kRowThreads;
        ctl.row[rr.slot][tid + k * kRowThreads] = row_of(c, s, i, word[k]);
        word[k] = row_word(c, s, i + kTile, index[k]);
        index[k] = row_index(s, i + 2 * kTile);
      }
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.rfull[rr.slot]));
      rr.next(kRowSlots);
    }
    __syncwarp();
    if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
}

// Issuing warp: all its lanes walk the same path, one of them issues.
template <int N, bool SHARED, int MAXI>
__device__ void issue_products(const AttendParams<MAXI>& P, uint8_t* sm, Control& ctl) {
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const Plan& pl = P.plan;
  const bool alias = SHARED && pl.alias;
  const uint32_t base = smem_u32(sm);
  const uint32_t tm_s = ctl.tmem, tm_o = ctl.tmem + 2 * N;
  const uint32_t type = c.f16 ? 0u : 1u;
  // float accumulator, operand types, N, M = 128; the second product's
  // operands are both M/N-major
  const uint32_t id1 = 1u << 4 | type << 7 | type << 10 | (uint32_t)(N >> 3) << 17 | 8u << 24;
  const uint32_t id2 = id1 | 1u << 15 | 1u << 16;
  constexpr uint32_t psbo = 8 * weight_row(N);
  constexpr uint32_t hi = operand_hi(1024, 2), hi_p = operand_hi(psbo, weight_swizzle(N));
  const uint32_t q_lo = operand_lo(base + pl.off_q, 16);
  const uint32_t p_lo = operand_lo(base + (alias ? pl.off_k : pl.off_p), 16);
  const uint32_t k_lo = operand_lo(base + pl.off_k, 16);
  const uint32_t v_lo = operand_lo(base + pl.off_v, 16), vt_lo = operand_lo(base + pl.off_v, kChunk);
  const bool lead = elected();
  const int c0 = pl.key_chunks - pl.only_chunks;
  const int last_steps = (c.dk - (pl.key_chunks - 1) * 64 + 15) / 16;
  Ring kr, vs, vr;  // key slots; value slots of the scores and of the sums
  uint32_t qphase = 0, pphase = 0, ophase = 0, n_scores = 0;
  bool first = true;
  // the products of key chunk `ch` staged at `at`
  auto chunk = [&](uint32_t d, uint32_t at, int ch, bool add) {
    const uint32_t b = q_lo + ch * (N * 128 >> 4);
    const int steps = ch + 1 < pl.key_chunks ? 4 : last_steps;
    if (!lead) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < steps) mma(d, at + 2 * k, hi, b + 2 * k, hi, id1, add || k > 0);
  };
  Ring seg;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    const int32_t v0 = s.v0, v1 = s.v1, cols = s.cols;
    if (__any_sync(~0u, ctl.gave_up) || !cols) break;
    if (lead) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
    if (v0 >= v1) continue;
    warp_wait(smem_u32(&ctl.qfull), qphase, until);
    fence_async();
    qphase ^= 1;
    int next = v0;  // the tile whose scores are next
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile) {
      // Values of their own arrive behind the keys, so that the next tile's
      // scores can be made while the softmax warps have this one's (grouped
      // histories 49 -> 45 us); shared rows hold their slots until the sums
      // are made, and leave none for the next tile.
      const int last = SHARED ? tile : min(tile + 1, v1 - 1);
#pragma unroll 1
      for (; next <= last; ++next) {
        const uint32_t buf = SHARED ? 0 : n_scores & 1, d = tm_s + buf * N;
        auto keys = [&](bool add) {
#pragma unroll 1
          for (int k = 0; k < pl.only_chunks; ++k) {
            warp_wait(smem_u32(&ctl.kfull[kr.slot]), kr.phase, until);
            fence_async();
            tc_after();
            chunk(d, k_lo + kr.slot * (kChunk >> 4), c0 + k, add || k > 0);
            if (lead && !alias) commit(smem_u32(&ctl.kempty[kr.slot]));
            kr.next(pl.kslots);
          }
        };
        if (!alias) keys(false);
        if (SHARED) {
#pragma unroll 1
          for (int u = 0; u < pl.units; ++u) {
            warp_wait(smem_u32(&ctl.vfull[vs.slot]), vs.phase, until);
            fence_async();
            tc_after();
            const uint32_t at = v_lo + vs.slot * (kUnit >> 4);
            chunk(d, at, 2 * u, (pl.only_chunks > 0 && !alias) || u > 0);
            if (2 * u + 1 < pl.key_chunks) chunk(d, at + (kChunk >> 4), 2 * u + 1, true);
            vs.next(pl.vslots);
          }
        }
        if (alias) keys(true);
        if (lead) {
          commit(smem_u32(&ctl.sfull[buf]));
          if (next + 1 == v1) commit(smem_u32(&ctl.qempty));
        }
        ++n_scores;
      }
      warp_wait(smem_u32(&ctl.pfull), pphase, until);
      pphase ^= 1;
      if (tile == v0 && !first) {  // the previous segment's sums are read
        warp_wait(smem_u32(&ctl.oempty), ophase, until);
        ophase ^= 1;
      }
      tc_after();
      const bool begun = tile > v0 || *(volatile uint32_t*)&ctl.o_begun;
#pragma unroll 1
      for (int u = 0; u < pl.units; ++u) {
        if (!SHARED) {
          warp_wait(smem_u32(&ctl.vfull[vr.slot]), vr.phase, until);
          fence_async();
          tc_after();
        }
        if (lead) {
          const uint32_t at = vt_lo + vr.slot * (kUnit >> 4);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma(tm_o + u * N, at + k * (2048 >> 4), hi, p_lo + k * (2 * psbo >> 4), hi_p, id2,
                begun || k > 0);
          commit(smem_u32(&ctl.vempty[vr.slot]));
        }
        vr.next(pl.vslots);
      }
      if (lead) {
        if (alias) commit(smem_u32(&ctl.kempty[0]));
        if (!SHARED || tile + 1 == v1) commit(smem_u32(&ctl.odone));
      }
    }
    first = false;
  }
  // nothing of ours is in flight when tensor memory goes back
  if (lead) commit(smem_u32(&ctl.drain));
#pragma unroll 1
  for (uint32_t n = 0; n < kAttendPolls && !bar_try(smem_u32(&ctl.drain), 0); ++n) {
  }
  __syncwarp();
}

// Whether none of the n elements at `p` is an infinity or NaN.
__device__ bool finite_row(const uint8_t* p, int n, int f16) {
  const uint32_t e = f16 ? 0x7C00u : 0x7F80u;
  bool ok = true;
#pragma unroll 1
  for (int k = 0; k < n; k += 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + 2 * k));
    for (const uint32_t w : {v.x, v.y, v.z, v.w})
      ok &= (w & e) != e && (w >> 16 & e) != e;
  }
  return ok;
}

// The products of the tile's rows marked `odd` (thread = row and half of the
// columns), added to the sums of the columns that see them; their staged
// values become zeros.  Runs while no product is in flight: those of the
// tiles before are complete.
template <int N, int MAXI>
__device__ __noinline__ void odd_rows(const AttendParams<MAXI>& P, uint8_t* sm, Control& ctl,
                                      int tid, bool odd, const uint8_t* value, Ring vr,
                                      int32_t tile0, bool first, uint32_t tm_scores) {
  constexpr int C = N / 2;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const Plan& pl = P.plan;
  const int r = tid & (kTile - 1), k0 = tid / kTile * C;
  const uint32_t tm_o = ctl.tmem + ((uint32_t)(r & ~31) << 16) + k0 + 2 * N;
  const float scale = c.scale * 1.44269504088896341f;
  const uint32_t marked = __ballot_sync(~0u, odd);
  if ((tid & 31) == 0 && tid < kTile) ctl.odd[tid >> 5] = marked;
  float v[8];
  if (first) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u)
#pragma unroll 1
      for (int k = 0; k < C; k += 8) tm_store(tm_o + u * N + k, v);
    if (tid == 0) ctl.o_begun = 1;
  }
  named_sync(1, kSoftThreads);
#pragma unroll 1
  for (int i = 0; i < kTile; ++i) {
    if (!(ctl.odd[i >> 5] >> (i & 31) & 1)) continue;
    if ((r >> 5) == (i >> 5)) {  // the warps that own the row
#pragma unroll 1
      for (int k = 0; k < C; k += 8) {
        tm_load(tm_scores + k, v);
        if (r == i)
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int col = k0 + k + n;
            const bool seen = tile0 + i >= ctl.col_lo[col] && tile0 + i < ctl.col_hi[col];
            ctl.part[0][col] = seen ? exp2_fast(v[n] * scale - ctl.base[col]) : 0.f;
          }
      }
      if (tid == i) ctl.odd_row = value;
    }
    named_sync(1, kSoftThreads);
    const uint8_t* y = ctl.odd_row;
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u) {
      const int d = u * 128 + r;
      float e = 0.f;
      if (d < c.dv)
        e = c.f16 ? __half2float(*reinterpret_cast<const __half*>(y + 2 * d))
                  : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(y + 2 * d));
#pragma unroll 1
      for (int k = 0; k < C; k += 8) {
        tm_load(tm_o + u * N + k, v);
#pragma unroll
        for (int n = 0; n < 8; ++n)
          if (ctl.part[0][k0 + k + n] != 0.f) v[n] += ctl.part[0][k0 + k + n] * e;
        tm_store(tm_o + u * N + k, v);
      }
    }
    named_sync(1, kSoftThreads);
  }
#pragma unroll 1
  for (int u = 0; u < pl.units; ++u) {
    warp_wait(smem_u32(&ctl.vfull[vr.slot]), vr.phase, until);
    if (odd && tid < kTile) {
      uint8_t* at = sm + pl.off_v + vr.slot * kUnit + r * 128;
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        *reinterpret_cast<uint4*>(at + 16 * k) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(at + kChunk + 16 * k) = make_uint4(0, 0, 0, 0);
      }
    }
    vr.next(pl.vslots);
  }
}

// 4 x 4 values of four neighbouring lanes transposed: lane i (mod 4) gets
// value i of lanes 0..3.
__device__ __forceinline__ void transpose4(float* v, int lane) {
  const bool a = lane & 1, b = lane & 2;
  float s0 = a ? v[0] : v[1], s1 = a ? v[2] : v[3];
  s0 = __shfl_xor_sync(~0u, s0, 1);
  s1 = __shfl_xor_sync(~0u, s1, 1);
  if (a) {
    v[0] = s0;
    v[2] = s1;
  } else {
    v[1] = s0;
    v[3] = s1;
  }
  s0 = b ? v[0] : v[2];
  s1 = b ? v[1] : v[3];
  s0 = __shfl_xor_sync(~0u, s0, 2);
  s1 = __shfl_xor_sync(~0u, s1, 2);
  if (b) {
    v[0] = s0;
    v[1] = s1;
  } else {
    v[2] = s0;
    v[3] = s1;
  }
}

// Softmax warps: a thread has one row of the tile and half of the columns;
// then the segment's output.
template <int N, bool SHARED, int MAXI>
__device__ void softmax_rows(const AttendParams<MAXI>& P, uint8_t* sm, Control& ctl, int tid,
                             float* parts) {
  constexpr int C = N / 2;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const Plan& pl = P.plan;
  const bool alias = SHARED && pl.alias;
  const int lane = tid & 31, r = tid & (kTile - 1), quarter = r >> 5, k0 = tid / kTile * C;
  const uint32_t tm_s = ctl.tmem + ((uint32_t)(r & ~31) << 16) + k0, tm_o = tm_s + 2 * N;
  const float scale = c.scale * 1.44269504088896341f;  // log2 e
  uint8_t* const weights = sm + (alias ? pl.off_k : pl.off_p) + r * weight_row(N);
  const bool wide = !(((uintptr_t)c.o_qs | c.o_hs) & 7);  // outputs store four elements at once
  const int turn = weight_row(N) == 32 ? (r >> 2) & 1 : weight_row(N) == 64 ? (r >> 1) & 3 : r & 7;
  Ring rr, vr;
  uint32_t n_scores = 0, ophase = 0;
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto sum = [](float a, float b) { return a + b; };
  Ring seg;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    const AttendItem& it = s.it;
    // the previous segment's column tables are read; all leave together
    if (named_or(1, kSoftThreads, ctl.gave_up) || !s.cols) break;
    if (tid == 0) ctl.o_begun = 0;
    if (tid < N) {
      const bool on = tid < s.cols;
      const int qc = s.col0 + min(tid, s.cols - 1);
      const int qi = it.loc ? s.qbase : qc / c.group;
      const int h = s.g * c.group + (it.loc ? qc : qc % c.group);
      ctl.out_off[tid] = qi * c.o_qs + h * c.o_hs;
      ctl.lse_at[tid] = on ? qi * c.heads + h : -1;
      int64_t lo = 0, hi = it.len;
      if (!it.loc) query_rows(it, qi, lo, hi);
      ctl.col_lo[tid] = (int32_t)min(lo, (int64_t)INT32_MAX);
      ctl.col_hi[tid] = (int32_t)max(hi, (int64_t)INT32_MIN);
      ctl.m[tid] = -INFINITY;
      ctl.base[tid] = 0.f;
    }
    named_sync(1, kSoftThreads);
    // rows [all_lo, all_hi) are visible to every column
    int32_t all_lo = 0, all_hi = INT32_MAX;
    if (!it.loc) {
#pragma unroll 1
      for (int k = 0; k < s.cols; ++k) {
        all_lo = max(all_lo, ctl.col_lo[k]);
        all_hi = min(all_hi, ctl.col_hi[k]);
      }
    }
    float l[C];
#pragma unroll
    for (int k = 0; k < C; ++k) l[k] = 0.f;

#pragma unroll 1
    for (int tile = s.v0; tile < s.v1; ++tile) {
      const int32_t j = tile * kTile + r;
      warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
      const uint8_t* row = ctl.row[rr.slot][r];
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
      rr.next(kRowSlots);
      const bool ragged = tile * kTile < all_lo || tile * kTile + kTile > all_hi;
      const uint32_t buf = SHARED ? 0 : n_scores & 1, tm = tm_s + buf * N;
      warp_wait(smem_u32(&ctl.sfull[buf]), (SHARED ? n_scores : n_scores >> 1) & 1, until);
      ++n_scores;
      tc_after();
      // The products of the tile before: complete, unless these scores were
      // made beside its weights.
      bool pending = !SHARED && tile > s.v0;
      auto settle = [&] {
        if (!pending) return;
        warp_wait(smem_u32(&ctl.odone), ophase, until);
        ophase ^= 1;
        tc_after();
        pending = false;
      };
      float x[C];  // scores in log2 units
      tm_load(tm, x);
#pragma unroll
      for (int k = 0; k < C; ++k) x[k] = row ? x[k] * scale : -INFINITY;
      if (ragged) {
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (j < ctl.col_lo[k0 + k] || j >= ctl.col_hi[k0 + k]) x[k] = -INFINITY;
      }
      bool move = tile == s.v0;
      if (!move) {
        // an unset reference (-inf) gives +inf, or NaN for a score of -inf
        float over = -INFINITY;
#pragma unroll
        for (int k = 0; k < C; k += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&ctl.m[k0 + k]);
          over = fmaxf(fmaxf(fmaxf(over, x[k] - m.x), x[k + 1] - m.y),
                       fmaxf(x[k + 2] - m.z, x[k + 3] - m.w));
        }
        move = named_or(1, kSoftThreads, over > kSlack);
      }
      if (move) {  // new references: the maxima so far
#pragma unroll
        for (int k = 0; k < C; k += 8) {
          const float y = fold8(x + k, lane, larger);
          if (lane < 8) ctl.part[quarter][k0 + k + lane] = y;
        }
        named_sync(1, kSoftThreads);
        if (tid < N) {
          const float old = ctl.m[tid];
          const float m = fmaxf(fmaxf(fmaxf(ctl.part[0][tid], ctl.part[1][tid]),
                                      fmaxf(ctl.part[2][tid], ctl.part[3][tid])), old);
          const float b = m == -INFINITY ? 0.f : m;
          ctl.fac[tid] = old == -INFINITY ? 0.f : exp2_fast(old - b);
          ctl.m[tid] = m;
          ctl.base[tid] = b;
        }
        named_sync(1, kSoftThreads);
        if (tile > s.v0) {
#pragma unroll
          for (int k = 0; k < C; ++k) l[k] *= ctl.fac[k0 + k];
          settle();
#pragma unroll 1
          for (int u = 0; u < pl.units; ++u)
#pragma unroll 1
            for (int k = 0; k < C; k += 8) {
              float v[8];
              tm_load(tm_o + u * N + k, v);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] *= ctl.fac[k0 + k + i];
              tm_store(tm_o + u * N + k, v);
            }
        }
      }
      // A row that only some of the columns see would reach the others too
      // if its value is not finite (0 x inf): such rows leave the tile, and
      // their products are added by hand to the columns that see them.
      bool odd = false;
      if (ragged) {
        const uint8_t* value = row + c.val_off + (int64_t)s.g * c.val_stride;
        if (row && (j < all_lo || j >= all_hi)) odd = !finite_row(value, c.dv, c.f16);
        if (named_or(1, kSoftThreads, odd)) {
          settle();
          odd_rows<N>(P, sm, ctl, tid, odd, value, vr, tile * kTile, tile == s.v0, tm);
        }
      }
#pragma unroll 1
      for (int u = 0; u < pl.units; ++u) vr.next(pl.vslots);
      // weights: half of a row of N in the swizzled layout
      settle();
#pragma unroll
      for (int k = 0; k < C; k += 8) {
        const float4 b0 = *reinterpret_cast<const float4*>(&ctl.base[k0 + k]);
        const float4 b1 = *reinterpret_cast<const float4*>(&ctl.base[k0 + k + 4]);
        const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = exp2_fast(x[k + i] - b[i]);
          l[k + i] += p[i];
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c.f16) {
            const __half2 z = __floats2half2_rn(p[2 * i], p[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&z);
          } else {
            const __nv_bfloat162 z = __floats2bfloat162_rn(p[2 * i], p[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&z);
          }
          if (odd) w[i] = 0;
        }
        *reinterpret_cast<uint4*>(weights + ((((k0 + k) / 8) ^ turn) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_async();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.pfull));
    }

    named_sync(1, kSoftThreads);
#pragma unroll
    for (int k = 0; k < C; k += 8) {
      const float y = fold8(l + k, lane, sum);
      if (lane < 8) ctl.part[quarter][k0 + k + lane] = y;
    }
    named_sync(1, kSoftThreads);
    const bool none = s.v0 >= s.v1, whole = s.whole();
    float* part = nullptr;
    if (!whole) {
      // a block leaves at most two parts: of the job it begins inside of,
      // and of the job that it ends inside of
      const int slot = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
      part = parts + (size_t)slot * N * (c.dv + 2);
    }
    if (tid < N) {
      const float z = ctl.part[0][tid] + ctl.part[1][tid] + ctl.part[2][tid] + ctl.part[3][tid];
      if (whole) {
        ctl.fac[tid] = z == 0.f ? 0.f : 1.f / z;
        if (it.lse && ctl.lse_at[tid] >= 0)
          it.lse[ctl.lse_at[tid]] =
              z == 0.f ? -INFINITY : (ctl.base[tid] + log2f(z)) * 0.693147180559945309f;
      } else {
        ctl.fac[tid] = 1.f;
        part[(size_t)N * c.dv + tid] = z == 0.f ? -INFINITY : ctl.base[tid];
        part[(size_t)N * c.dv + N + tid] = z;
      }
    }
    named_sync(1, kSoftThreads);
    if (!none) {
      warp_wait(smem_u32(&ctl.odone), ophase, until);
      ophase ^= 1;
      tc_after();
    }
    const bool quads = wide && !((uintptr_t)it.out & 7);
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u) {
      // after the exchange lane i of four has column k + i of four elements
      const int d = u * 128 + quarter * 32 + (lane & ~3);
      float v[C];
      if (none) {
#pragma unroll
        for (int k = 0; k < C; ++k) v[k] = 0.f;
      } else {
        tm_load(tm_o + u * N, v);
      }
#pragma unroll
      for (int k = 0; k < C; k += 4) {
        transpose4(v + k, lane);
        const int col = k0 + k + (lane & 3);
        const float f = ctl.fac[col];
        const bool on = d < c.dv && col < s.cols;
        float y[4];
        // a weight sum of zero leaves products of zero: the output is zero
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f == 0.f ? 0.f : v[k + i] * f;
        if (!whole) {
          if (on)
            *reinterpret_cast<float4*>(part + (size_t)col * c.dv + d) =
                make_float4(y[0], y[1], y[2], y[3]);
          continue;
        }
        uint32_t w[2];
        if (c.f16) {
          const __half2 a = __floats2half2_rn(y[0], y[1]), b = __floats2half2_rn(y[2], y[3]);
          w[0] = *reinterpret_cast<const uint32_t*>(&a);
          w[1] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
          const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]);
          const __nv_bfloat162 b = __floats2bfloat162_rn(y[2], y[3]);
          w[0] = *reinterpret_cast<const uint32_t*>(&a);
          w[1] = *reinterpret_cast<const uint32_t*>(&b);
        }
        uint8_t* out = it.out + ctl.out_off[col] + 2 * d;
        if (!on) {
        } else if (quads) {
          *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
        } else {
          uint16_t* o = reinterpret_cast<uint16_t*>(out);
          o[0] = (uint16_t)w[0];
          o[1] = (uint16_t)(w[0] >> 16);
          o[2] = (uint16_t)w[1];
          o[3] = (uint16_t)(w[1] >> 16);
        }
      }
      __syncwarp();
    }
    if (!none) {
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.oempty));
    }
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
}

template <int N, bool SHARED, int MAXI>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams<MAXI> P, float* parts) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  Control& ctl = *reinterpret_cast<Control*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  static_assert(kRowSlots * kTile == kSoftThreads, "one address a softmax thread");
  if (tid < kSoftThreads) (&ctl.row[0][0])[tid] = nullptr;
  if (warp == kIssueWarp) {
#pragma unroll
    for (int k = 0; k < kBarriers; k += 32) {
      const int i = k + (tid & 31);
      const bool full = i < kMaxK || (i >= 2 * kMaxK && i < 2 * kMaxK + kMaxV) || i == kBarQfull;
      const bool soft = i == kBarPfull || i == kBarOempty;
      const bool rows = i >= kBarRfull && i < kBarRempty;
      const bool read = i >= kBarRempty && i < kBarDrain;
      const bool segs = i >= kBarSegempty && i < kBarSegempty + kSegments;
      bar_init(smem_u32(&ctl.kfull[0]) + 8 * i,
               full ? kLoadThreads : soft ? kSoftThreads / 32 : rows ? kRowThreads / 32
               : read ? (kSoftThreads + kLoadThreads) / 32 : segs ? kThreads / 32 - 1 : 1);
    }
    ctl.gave_up = P.c.polls == 0;  // nothing is waited for then
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "r"(tmem_columns(N))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kFindWarp) {
    find_segments(P, ctl);  // meets the others' barrier inside
  } else {
    tc_before();
    __syncthreads();
    tc_after();
    if (warp < kSoftThreads / 32) softmax_rows<N, SHARED>(P, sm, ctl, tid, parts);
    else if (warp < kIssueWarp) load_rows<N, SHARED>(P, sm, ctl, tid - kSoftThreads);
    else if (warp == kIssueWarp) issue_products<N, SHARED>(P, sm, ctl);
    else find_rows(P, ctl, tid - 32 * kRowWarp);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(ctl.tmem),
                 "r"(tmem_columns(N))
                 : "memory");
  if (tid == 0 && ctl.gave_up) atomicOr(P.c.status, kStatusEtimeout);
}

// ------------------------------------------------------------------ merge

constexpr int kMergeWarps = 16;
constexpr int kMergeElems = 128;  // value elements of a warp: a float4 a lane

// A split job: parts of the blocks [b0, b0 + n).
struct Cut {
  uint8_t* out;       // of the job's kv head and, if located, query
  float* lse;         // or null
  int32_t b0, n;
  int32_t col0, cols;
};

struct MergeParams {
  int32_t groups;     // warps that share one column's parts: 1, 4 or 16
  int32_t columns;    // of a part
  int32_t dv, f16, heads, group;
  int64_t o_qs, o_hs;
  Cut cut[kAttendMaxBlocks];
};

// Joins the parts of the split jobs in block order.  A warp has 128 value
// elements of one column and every `groups`-th part; the groups' sums meet in
// shared memory.  Bound by latency: statistics, then weights, then parts, each
// a trip to L2; 104 jobs of 64 columns in 2 to 3 parts, 34 MB, take 23 us, one
// job of 16 columns in 152 parts 13 (each on cold caches).
__global__ void __launch_bounds__(kMergeWarps * 32, 2)
    merge_kernel(const __grid_constant__ MergeParams M, const float* parts) {
  __shared__ float4 sums[kMergeWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cut& cut = M.cut[blockIdx.x];
  const int n = cut.n, b0 = cut.b0;
  const int spans = (M.dv + kMergeElems - 1) / kMergeElems;
  const int pair = blockIdx.y * (kMergeWarps / M.groups) + warp / M.groups;
  const int col = pair / spans, d = pair % spans * kMergeElems + lane * 4;
  const int group = warp % M.groups;
  const bool on = col < cut.cols;
  const size_t stride = (size_t)M.columns * (M.dv + 2);
  auto part = [&](int i) { return parts + (size_t)(2 * (b0 + i) + (i == 0)) * stride; };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float base = 0.f, z = 0.f;
  if (on) {
    const size_t ml = (size_t)M.columns * M.dv + col;
    float m = -INFINITY;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) m = fmaxf(m, part(i)[ml]);
#pragma unroll
    for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, w));
    base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
    for (int i = lane; i < n; i += 32)
      z += exp2_fast(part(i)[ml] - base) * part(i)[ml + M.columns];
#pragma unroll
    for (int w = 16; w; w >>= 1) z += __shfl_xor_sync(~0u, z, w);
    // lane k's weight is that of the group's k-th part, of 32 at a time
#pragma unroll 1
    for (int i0 = group; i0 < n; i0 += 32 * M.groups) {
      const int mine = i0 + lane * M.groups;
      const float weight = mine < n ? exp2_fast(part(mine)[ml] - base) : 0.f;
      const int count = min(32, (n - i0 + M.groups - 1) / M.groups);
#pragma unroll 1
      for (int k = 0; k < count; k += 4) {
        float4 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (k + u < count && d < M.dv)
            y[u] = *reinterpret_cast<const float4*>(part(i0 + (k + u) * M.groups) +
                                                    (size_t)col * M.dv + d);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float w = __shfl_sync(~0u, weight, (k + u) & 31);
          // a part without weight may hold sums that are not finite
          if (k + u < count && w != 0.f && d < M.dv) {
            x.x += w * y[u].x;
            x.y += w * y[u].y;
            x.z += w * y[u].z;
            x.w += w * y[u].w;
          }
        }
      }
    }
  }
  if (M.groups > 1) {
    sums[warp][lane] = x;
    __syncthreads();
    if (group) return;
#pragma unroll 1
    for (int k = 1; k < M.groups; ++k) {
      const float4 y = sums[warp + k][lane];
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
  }
  if (!on) return;
  const int qc = cut.col0 + col, qi = qc / M.group, h = qc - qi * M.group;
  if (cut.lse && lane == 0 && d == 0)
    cut.lse[(size_t)qi * M.heads + h] =
        z == 0.f ? -INFINITY : (base + log2f(z)) * 0.693147180559945309f;
  if (d >= M.dv) return;
  uint8_t* out = cut.out + qi * M.o_qs + h * M.o_hs + 2 * d;
  const float inv = z == 0.f ? 0.f : 1.f / z;
  float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
  uint16_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (inv == 0.f) y[k] = 0.f;
    const __half a = __float2half_rn(y[k]);
    const __nv_bfloat16 b = __float2bfloat16_rn(y[k]);
    w[k] = M.f16 ? __half_as_ushort(a) : __bfloat16_as_ushort(b);
  }
  if ((uintptr_t)out & 7) {
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<uint16_t*>(out)[k] = w[k];
  } else {
    *reinterpret_cast<uint2*>(out) =
        make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
  }
}

// ------------------------------------------------------------------ host

constexpr uint32_t kSmemLimit = 232448;  // opt-in shared memory of a block

uint32_t round_up(uint32_t x, uint32_t to) { return (x + to - 1) / to * to; }

// Ring sizes that fit shared memory: what a tile needs at once, then one
// value unit and one key chunk more in turn while there is room.
Plan make_plan(const AttendCommon& c, int n) {
  Plan p{};
  p.key_chunks = (c.dk + 63) / 64;
  p.units = (c.dv + 127) / 128;
  p.shared = c.val_off == c.key_off && c.dv <= c.dk &&
             (c.heads == c.group || c.val_stride == c.key_stride);
  p.only_chunks = p.shared ? std::max(0, p.key_chunks - 2 * p.units) : p.key_chunks;
  const uint32_t q = round_up((uint32_t)p.key_chunks * n * 128, 1024);
  const uint32_t w = (uint32_t)kTile * weight_row(n);
  p.kslots = p.only_chunks ? 1 : 0;
  p.vslots = p.units;
  auto bytes = [&](int k, int v, bool alias) {
    return 1024 + kControlBytes + q + (alias ? 0 : w) + (uint32_t)k * kChunk + (uint32_t)v * kUnit;
  };
  // the weights can take the place of a key chunk that is done with by then
  p.alias = p.shared && p.only_chunks == 1 && bytes(p.kslots, p.vslots, false) > kSmemLimit;
  for (bool more = true; more;) {
    more = false;
    if (p.vslots < std::min(kMaxV, 2 * p.units) && bytes(p.kslots, p.vslots + 1, p.alias) <= kSmemLimit) {
      ++p.vslots;
      more = true;
    }
    if (!p.alias && p.only_chunks && p.kslots < std::min(kMaxK, 2 * p.only_chunks) &&
        bytes(p.kslots + 1, p.vslots, false) <= kSmemLimit) {
      ++p.kslots;
      more = true;
    }
  }
  p.off_q = kControlBytes;
  p.off_p = p.off_q + q;
  p.off_k = round_up(p.off_p + (p.alias ? 0 : w), 1024);
  p.off_v = p.off_k + (uint32_t)p.kslots * kChunk;
  p.smem = 1024 + p.off_v + (uint32_t)p.vslots * kUnit;
  return p;
}

// The widest block of columns whose queries leave room for a tile: 64, or 48
// for the largest keys and values that are not the same bytes.
int widest_block(const AttendCommon& c) {
  int n = 64;
  while (n > 16 && make_plan(c, n).smem > kSmemLimit) n -= 16;
  return n;
}

struct Shape {
  int n = 0;          // columns of a block
  int64_t tiles = 0;
  int blocks = 0;
  int n_cut = 0;      // jobs cut by a block's boundary
  int groups = 1;     // of the merge
  Cut cut[kAttendMaxBlocks];
};

int columns_of(const AttendCommon& c, const AttendItem& it, int most) {
  const int all = it.loc ? c.group : it.Q * c.group;
  const int blk = (all + most - 1) / most;
  return (all + blk - 1) / blk;
}

// Fills in every item's tiles, and how the blocks share them.
Shape shape_of(AttendCommon& c, AttendItem* items, int n_items, int sms) {
  Shape s;
  const int most = widest_block(c);
  int widest = 1;
  int64_t n_jobs = 0, longest = 0, shortest = INT64_MAX;
  for (int i = 0; i < n_items; ++i) widest = std::max(widest, columns_of(c, items[i], most));
  s.n = (widest + 15) / 16 * 16;
  c.kv = c.heads / c.group;
  for (int i = 0; i < n_items; ++i) {
    AttendItem& it = items[i];
    it.tile0 = (int32_t)std::min<int64_t>(s.tiles, INT32_MAX);
    // an item without rows still has one tile, that writes its empty outputs
    it.tiles = (int32_t)std::max<int64_t>(1, (it.len + kTile - 1) / kTile);
    const int64_t all = it.loc ? c.group : (int64_t)it.Q * c.group;
    it.blocks = (int32_t)((all + s.n - 1) / s.n);
    it.width = it.blocks ? (int32_t)((all + it.blocks - 1) / it.blocks) : 0;
    const int64_t jobs = (it.loc ? it.Q : 1) * (int64_t)c.kv * it.blocks;
    s.tiles += jobs * it.tiles;
    n_jobs += jobs;
    longest = std::max<int64_t>(longest, it.tiles);
    shortest = std::min<int64_t>(shortest, it.tiles);
  }
  sms = std::min(sms, kAttendMaxBlocks);
  s.blocks = (int)std::max<int64_t>(1, std::min<int64_t>(sms, s.tiles));
  c.waves = c.waved = c.job_tiles = c.share = c.extra = 0;
  if (s.tiles > INT32_MAX) return s;  // refused
  // Jobs of equal length: whole ones in waves over the blocks, as neighbours
  // often read the same rows (64 verify blocks of 8 queries with 80 % of their
  // rows in common 267 -> 250 us, 128 heads 191 -> 185; grouped heads on
  // unrelated rows lose, 76 -> 82).  Fewer blocks if that leaves nothing to
  // split and no block with more to do, or with two tiles instead of one,
  // which take no longer than a merge (40 x 256 rows 14.4 us instead of 16.7,
  // 16 x 256 grouped 10.3 instead of 12.4; three tiles: 17.4 instead of 14.4).
  if (longest == shortest) {
    const int64_t each = (n_jobs + sms - 1) / sms;
    const int64_t even = (s.tiles + s.blocks - 1) / s.blocks;
    if (n_jobs % each == 0 && each * longest <= std::max<int64_t>(2, even))
      s.blocks = (int)(n_jobs / each);
    c.waves = (int)(n_jobs / s.blocks);
    c.job_tiles = (int32_t)longest;
    c.waved = (int32_t)(c.waves * s.blocks * longest);
  }
  const int64_t rest = s.tiles - c.waved;  // dealt out evenly, cut where it falls
  c.share = (int32_t)(rest / s.blocks);
  c.extra = (int32_t)(rest % s.blocks);
  const int parts = rest ? (int)std::min<int64_t>(s.blocks, longest * s.blocks / rest + 2) : 0;
  // Warps that share a column: few parts leave too little to each, many wait
  // in line.  8 x 2048 rows in 20 parts: 4 groups 16.4 us, 1 18.5, 16 20.5;
  // 512 K rows in 152 parts: 16 groups 116.5 us, 4 122.3.
  s.groups = parts > 24 ? 16 : parts > 4 ? 4 : 1;
  if (rest) {
    int k = 0;
    int64_t cut_job = -1;  // first tile of the job cut last
    for (int b = 1; b < s.blocks; ++b) {
      const int32_t t = first_tile(c, b);
      if (t >= s.tiles) break;
      while (k + 1 < n_items && items[k + 1].tile0 <= t) ++k;
      const AttendItem& it = items[k];
      const int32_t job = (t - it.tile0) / it.tiles, in = (t - it.tile0) - job * it.tiles;
      if (in == 0 || t - in == cut_job) continue;
      cut_job = t - in;
      Cut& cut = s.cut[s.n_cut++];
      const int32_t query = job / it.blocks, q = query / c.kv, head = (query - q * c.kv) * c.group;
      const int32_t columns = it.loc ? c.group : it.Q * c.group;
      cut.out = it.out + q * c.o_qs + head * c.o_hs;
      cut.lse = it.lse ? it.lse + (size_t)q * c.heads + head : nullptr;
      cut.col0 = (job - query * it.blocks) * it.width;
      cut.cols = std::min(it.width, columns - cut.col0);
      // up to the block that holds the job's last tile
      const int32_t last = (int32_t)cut_job + it.tiles - 1 - c.waved, more = c.extra * (c.share + 1);
      cut.b0 = b - 1;
      cut.n = (last < more ? last / (c.share + 1) : c.extra + (last - more) / c.share) - b + 2;
    }
  }
  return s;
}

cudaError_t launch_merge(const AttendCommon& c, const Shape& s, const float* parts,
                         cudaStream_t stream) {
  MergeParams M;
  M.groups = s.groups;
  M.columns = s.n;
  M.dv = c.dv;
  M.f16 = c.f16;
  M.heads = c.heads;
  M.group = c.group;
  M.o_qs = c.o_qs;
  M.o_hs = c.o_hs;
  std::copy(s.cut, s.cut + s.n_cut, M.cut);
  cudaLaunchConfig_t cfg{};
  const int per = kMergeWarps / s.groups;
  const int pairs = s.n * ((c.dv + kMergeElems - 1) / kMergeElems);
  cfg.gridDim = dim3(s.n_cut, (pairs + per - 1) / per);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel, M, parts);
}

// Lets a kernel's blocks use all of an SM's shared memory: once on each device,
// with its first launch there.  (The driver loads a kernel when it is first
// named.  Pools that named all 16 of these when they were made took 1 ms more
// for that, and their resolve and gather kernels, loaded around them, ran 25.2
// us a step of 8 items with one build of this file and 24.7 with another;
// without them 24.8 with either.)
template <int N, bool SHARED, int MAXI>
cudaError_t use_all_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(attend_kernel<N, SHARED, MAXI>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int N, bool SHARED, int MAXI>
cudaError_t launch_kernel(const AttendParams<MAXI>& P, const Shape& s, float* parts,
                          cudaStream_t stream) {
  cudaError_t e = use_all_smem<N, SHARED, MAXI>();
  if (e != cudaSuccess) return e;
  attend_kernel<N, SHARED><<<s.blocks, kThreads, P.plan.smem, stream>>>(P, parts);
  e = cudaGetLastError();
  if (e != cudaSuccess || !s.n_cut) return e;
  return launch_merge(P.c, s, parts, stream);
}

// A kernel for each kind of layout: with one that asked at run time, both were
// slower (128 heads 172 us instead of 166, grouped heads 55.7 instead of 54.4).
template <int N, int MAXI>
cudaError_t launch_n(const AttendParams<MAXI>& P, const Shape& s, float* parts, cudaStream_t stream) {
  return P.plan.shared ? launch_kernel<N, true, MAXI>(P, s, parts, stream)
                       : launch_kernel<N, false, MAXI>(P, s, parts, stream);
}

template <int MAXI>
cudaError_t launch_t(const AttendCommon& c, const AttendItem* items, int n_items, const Shape& s,
                     float* parts, cudaStream_t stream) {
  AttendParams<MAXI> P;
  P.c = c;
  P.plan = make_plan(c, s.n);
  for (int i = 0; i < MAXI; ++i) P.first[i] = i < n_items ? items[i].tile0 : INT32_MAX;
  for (int i = 0; i < n_items; ++i) P.items[i] = items[i];
  switch (s.n) {
    case 16: return launch_n<16, MAXI>(P, s, parts, stream);
    case 32: return launch_n<32, MAXI>(P, s, parts, stream);
    case 48: return launch_n<48, MAXI>(P, s, parts, stream);
    default: return launch_n<64, MAXI>(P, s, parts, stream);
  }
}

}  // namespace

bool attend_shape(AttendCommon c, AttendItem* items, int n_items, int sms, size_t* bytes) {
  const Shape s = shape_of(c, items, n_items, sms);
  *bytes = s.n_cut ? (size_t)2 * s.blocks * s.n * (c.dv + 2) * sizeof(float) : 0;
  return s.tiles <= INT32_MAX;
}

cudaError_t launch_attend(AttendCommon c, AttendItem* items, int n_items, int sms,
                          void* work, cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kAttendItemsLarge) return cudaErrorInvalidValue;
  const Shape s = shape_of(c, items, n_items, sms);
  if (s.tiles > INT32_MAX) return cudaErrorInvalidValue;
  float* parts = static_cast<float*>(work);
  // The whole table travels with a launch: a small one for few items (12
  // histories 41.7 us instead of 42.5, 8 of 32 K rows 66.3 instead of 67.0).
  return n_items <= kAttendItemsSmall
             ? launch_t<kAttendItemsSmall>(c, items, n_items, s, parts, stream)
             : launch_t<kAttendItemsLarge>(c, items, n_items, s, parts, stream);
}

}  // namespace dhs
