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
// reads 409 MB, each distinct row once).  One token over 512K rows, 107 us:
// 590 MB of DRAM reads at 5.8 TB/s between a start of 4 us and a merge of 5.
// 128 heads, 158 us: one tile at a time is resident beside 64 queries, so
// that loads, scores, weights and sums follow each other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "attend_core.cuh"

namespace dhs {
namespace {

constexpr int kSoftThreads = 256, kLoadThreads = 128;
constexpr int kIssueWarp = (kSoftThreads + kLoadThreads) / 32, kFindWarp = kIssueWarp + 1;
constexpr int kRowWarp = kFindWarp + 1, kRowThreads = 64;
constexpr int kThreads = 32 * kRowWarp + kRowThreads;
constexpr int kChunk = kTile * 128;        // bytes of a 64-element column chunk of a tile
constexpr int kUnit = 2 * kChunk;          // a value unit: 128 elements
constexpr int kMaxK = 12, kMaxV = 8;       // ring slots at most
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
using Params = AttendParams<MAXI, Plan>;
static_assert(sizeof(Params<kAttendItemsLarge>) <= 32764, "attend item table too large");

// ------------------------------------------------------------------ kernel

constexpr int kUnusedBars = 8 - 2 * kRowSlots;
struct Control {
  static constexpr int kRowSlots = dhs::kRowSlots, kRowThreads = dhs::kRowThreads;
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

// Two buffers of scores, then up to four units of sums.
__host__ __device__ constexpr uint32_t tmem_columns(int n) {
  return 6 * n <= 128 ? 128 : 6 * n <= 256 ? 256 : 512;
}
// Bytes of one row of weights, the swizzle of that row width, and its 8-row stride.
__host__ __device__ constexpr int weight_row(int n) { return n <= 16 ? 32 : n <= 32 ? 64 : 128; }
__host__ __device__ constexpr uint32_t weight_swizzle(int n) { return n <= 16 ? 6 : n <= 32 ? 4 : 2; }

// Loading warps: queries once per segment, rows tile by tile.
template <int N, bool SHARED, int MAXI>
__device__ void load_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid) {
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

// Issuing warp: all its lanes walk the same path, one of them issues.
template <int N, bool SHARED, int MAXI>
__device__ void issue_products(const Params<MAXI>& P, uint8_t* sm, Control& ctl) {
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
__device__ __noinline__ void odd_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl,
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

// Softmax warps: a thread has one row of the tile and half of the columns;
// then the segment's output.
template <int N, bool SHARED, int MAXI>
__device__ void softmax_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid,
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
    attend_kernel(const __grid_constant__ Params<MAXI> P, float* parts) {
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

// ------------------------------------------------------------------ host

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
cudaError_t launch_kernel(const Params<MAXI>& P, const Shape& s, float* parts,
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
cudaError_t launch_n(const Params<MAXI>& P, const Shape& s, float* parts, cudaStream_t stream) {
  return P.plan.shared ? launch_kernel<N, true, MAXI>(P, s, parts, stream)
                       : launch_kernel<N, false, MAXI>(P, s, parts, stream);
}

template <int MAXI>
cudaError_t launch_t(const AttendCommon& c, const AttendItem* items, int n_items, const Shape& s,
                     float* parts, cudaStream_t stream) {
  Params<MAXI> P;
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
  const Shape s = shape_of(c, items, n_items, sms, widest_block(c));
  *bytes = parts_bytes(c, s);
  return s.tiles <= INT32_MAX;
}

cudaError_t launch_attend(AttendCommon c, AttendItem* items, int n_items, int sms,
                          void* work, cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kAttendItemsLarge) return cudaErrorInvalidValue;
  const Shape s = shape_of(c, items, n_items, sms, widest_block(c));
  if (s.tiles > INT32_MAX) return cudaErrorInvalidValue;
  float* parts = static_cast<float*>(work);
  // The whole table travels with a launch: a small one for few items (12
  // histories 41.7 us instead of 42.5, 8 of 32 K rows 66.3 instead of 67.0).
  return n_items <= kAttendItemsSmall
             ? launch_t<kAttendItemsSmall>(c, items, n_items, s, parts, stream)
             : launch_t<kAttendItemsLarge>(c, items, n_items, s, parts, stream);
}

}  // namespace dhs
