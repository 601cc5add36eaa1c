// What the attention kernels share (attend.cu: 16-bit rows, attend_packed.cu:
// rows in 8 bits): the instructions they use, how a launch's tiles are dealt
// out to blocks, the warps that find segments and row addresses, and the host
// side of splitting jobs and of joining their parts (attend_merge.cu).
#pragma once

#include <cuda_runtime.h>

#include "dhs_internal.h"

namespace dhs {

// ------------------------------------------------------------------ jobs cut by blocks

// A split job: parts of the blocks [b0, b0 + n).
struct Cut {
  uint8_t* out;       // of the job's kv head and, if located, query
  float* lse;         // or null
  int32_t b0, n;
  int32_t col0, cols;
};

struct Shape {
  int n = 0;          // columns of a block
  int64_t tiles = 0;
  int blocks = 0;
  int n_cut = 0;      // jobs cut by a block's boundary
  int groups = 1;     // of the merge
  Cut cut[kAttendMaxBlocks];
};

// Fills in every item's tiles, and how the blocks share them; `most`: the
// widest block of columns that the kernel takes for these heads.
Shape shape_of(AttendCommon& c, AttendItem* items, int n_items, int sms, int most);
// Workspace bytes of such a launch.
size_t parts_bytes(const AttendCommon& c, const Shape& s);
// Joins the parts of the split jobs (s.n_cut > 0) behind the launch.
cudaError_t launch_merge(const AttendCommon& c, const Shape& s, const float* parts,
                         cudaStream_t stream);

// First tile of block b's share of what the waves leave.
__host__ __device__ __forceinline__ int32_t first_tile(const AttendCommon& c, int32_t b) {
  return c.waved + b * c.share + min(b, c.extra);
}

constexpr uint32_t kSmemLimit = 232448;  // opt-in shared memory of a block
constexpr int kTile = 128;               // rows per tile

inline uint32_t round_up(uint32_t x, uint32_t to) { return (x + to - 1) / to * to; }

#ifdef __CUDACC__
namespace {

constexpr int kSegments = 4;               // segments found ahead

// A launch's item table, which travels with it.
template <int MAXI, class Plan>
struct AttendParams {
  static constexpr int kItems = MAXI;
  AttendCommon c;
  Plan plan;
  int32_t first[MAXI];   // first tile of each item, past the last one INT32_MAX
  AttendItem items[MAXI];
};

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
template <class P_>
__device__ __forceinline__ int item_at(const P_& P, int32_t t) {
  constexpr int MAXI = P_::kItems;
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
template <class P_>
__device__ Segment segment_at(const P_& P, int32_t t, int32_t te) {
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

// A block's segments: first a whole job of each wave (jobs of equal length go
// to the blocks in order, so that blocks running side by side work on
// neighbouring jobs, which read the same rows), then its even share of the
// tiles that are left.
struct Walk {
  int32_t wave, t, te;
};
template <class P_>
__device__ __forceinline__ Walk first_of(const P_& P) {
  const AttendCommon& c = P.c;
  return {0, first_tile(c, blockIdx.x), first_tile(c, blockIdx.x + 1)};
}
template <class P_>
__device__ bool next_segment(const P_& P, Walk& w, Segment& s) {
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

// ------------------------------------------------------------------ roles

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

// Finding warp: the block's segments, ahead of the others, who read them from
// shared memory.  One without columns ends the walk.  The first one is found
// while the block sets up.
template <class P_, class C_>
__device__ void find_segments(const P_& P, C_& ctl) {
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
template <class P_, class C_>
__device__ void find_rows(const P_& P, C_& ctl, int tid) {
  constexpr int kRowThreads = C_::kRowThreads, kRowSlots = C_::kRowSlots, R = kTile / kRowThreads;
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

}  // namespace
#endif  // __CUDACC__

}  // namespace dhs
