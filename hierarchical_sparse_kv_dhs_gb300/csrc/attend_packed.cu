// Attention over packed rows (e4m3 codes with a power-of-two scale for each
// head, and a few 16-bit elements): located rows or a source's history, read in
// 8 bits where they lie.
//
// With codes c_j (keys) and d_j (values), scales 2^k_j and 2^v_j, wide elements
// w_j, and a query's coded part a and wide part b, s_j = scale (2^k_j a . c_j +
// b . w_j), and one pass keeps a reference m, l = sum exp(s_j - m) and o = sum
// exp(s_j - m) 2^v_j d_j; out = o / l, log-sum = m + ln l.
//
// Both products take the codes as they lie in memory as their 8-bit M operand:
// no code is ever converted.
//   S^T[128 rows x N] = C[128 x 128-element chunks] . A^T,  W . B^T in 16 bits
//   O^T[dv x N]      += D^T[dv x 128] . P^T
// What meets them has to be 8 bits wide too, and is split into pieces whose sum
// it is, side by side as further columns (N is small: a product of 64 columns
// takes hardly longer than one of 16) or, where tensor memory does not hold
// their sums apart, one product after the other into the same sums:
//   - the query, brought to 448 or below by a power of two: 2 pieces of e4m3
//     hold bf16's 8 bits, 3 hold f16's 11, exactly (each piece holds 4 and its
//     sign one more), but for elements under 2^-9 of a step's unit, 2^-18 of
//     the largest one;
//   - the weights exp(s_j - m) 2^v_j: e5m2, whose range is f16's.  Taken to f16
//     first (2^-11 of a weight at most), a piece is the upper byte of the number
//     plus half a unit, and what is left is exact in f16.  Three pieces hold every
//     f16 number from 2^-6 up exactly, the smaller ones to 2^-17, half of e5m2's
//     smallest; a fourth, which f16 rows make, holds nothing better.
//     m follows the maximum of s_j + v_j, and moves when one passes it by 2^6: the
//     largest weight is 2^9 to 2^15, so that 2^-17 is 2^-26 of it at most.  That
//     much is lost or added by each row alike where many share a small weight, in
//     the part of a job that holds the large one: 2^-7 of its value in all for
//     half a million rows.  Smaller steps of m would hold more, 2^-28 where it
//     moves at 2^4 and 2^-30 at 2^2, but the sums are rescaled at each (128 heads
//     168 us, then 176 and 185).  (e4m3 would hold 2^-18 at best.)
// l sums the weights unrounded, without 2^v_j, which is divided out exactly (from
// floats, which end at 2^-126 where the largest weight has 2^9 or more).
//
// The rest is the 16-bit attention's (attend.cu): roles, tiles of 128 rows, the
// dealing of jobs and the joining of parts.
//
// What it takes and what bounds it (latent rows of 656 bytes and 16 heads in bf16
// unless said; in parentheses the same call over 16-bit rows of 1152 bytes):
//   - 64 verify blocks of 8 queries over 2048 rows each: 168 us (234), 688 MB of
//     rows staged at 4.1 TB/s.  The copies alone take 90 us, the products 43 (36
//     of 40 to 45 cycles a tile); what a tile waits for is the way from its scores
//     to its weights.  An earlier step of this kernel took 170 us, and 135 without
//     its copies: its softmax warps worked through 200 of 279 thousand cycles, and
//     waited for scores for 66.  Some SMs run a fifth slower than the mean.
//   - 128 heads, 16 blocks of 8: 169 us (158), the same way with 32 columns: a
//     weight is made and written in three pieces instead of one, and a query's 128
//     heads take four passes over the rows instead of two (48 or 64 columns a
//     block, whose pieces' sums tensor memory does not hold apart: 210 us).
//   - a history of 512,000 rows: 72 us (107), its rows at 4.9 TB/s of DRAM reads,
//     then the joining kernel.
//   - one query of 256 rows 12.3 us (14.3), 8 requests of 2048 rows 16.4 (17): once
//     through the pipeline, and the joining kernel.
//   - ragged f16 histories, 4 kv heads with values of their own: 51 us (41): 64 MB,
//     12 tiles a block, of which each weight takes four pieces.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstddef>

#include "attend_core.cuh"
#include "dhs.h"

namespace dhs {
namespace {

constexpr int kChunk = kTile * 128;  // bytes of a ring slot: 128 bytes of each row
constexpr int kMaxSlots = 12;
constexpr float kSlack = 6.f;        // log2 units that a weight may pass the reference by
constexpr float kLift = 9.f;         // log2 of a weight at the reference
// log2 of what a row's key scale is held below itself by, and a query's above: a sum of
// products of codes and pieces, 576 * 448 * 448 < 2^27, times 2^120 stays finite then.
constexpr int kAside = 19;
constexpr int kLoadThreads = 128, kRowThreads = 32;
constexpr int kTmemColumns = 512;

// How a launch's rows are staged.
struct PackedPlan {
  int32_t shared;        // the value is the key's beginning: loaded once
  int32_t key_chunks;    // of 128 codes
  int32_t units;         // value units of 128 codes: tiles of O^T's M side
  int32_t per_tile;      // ring slots of a tile: keys, wide elements, values unless shared
  int32_t slots;
  int32_t bufs;          // buffers of scores: 2: the next tile's are made beside this tile's weights
  int32_t weight_bufs;   // buffers of weights: 2: filled beside the products of the tile before
  int32_t buf_columns;   // tensor memory of one buffer of scores
  int32_t sum_column;    // where the sums begin
  int32_t key8, wide;    // elements of a head
  int32_t off_value, off_wide, off_scale, value_scales;  // within a row
  uint32_t off_q, off_qw, off_p, off_rows;  // from the aligned shared-memory base
  uint32_t smem;
};

template <int MAXI>
using Params = AttendParams<MAXI, PackedPlan>;
static_assert(sizeof(Params<kAttendItemsLarge>) <= 32764, "attend item table too large");

template <int N, bool F16>
struct Pieces {
  static constexpr int kQ = F16 ? 3 : 2, kP = F16 ? 4 : 3;
  static constexpr int kScore = (kQ + 1) * N;  // columns of a buffer of scores, wide ones last
  // pieces of the weights as further columns, where four units of sums leave room
  static constexpr bool kStack = 4 * kP * N + kScore <= kTmemColumns;
  static constexpr int kSum = kStack ? kP * N : N;  // columns of a unit's sums
  static constexpr int kRow = kSum <= 32 ? 32 : kSum <= 64 ? 64 : 128;  // bytes of a row of weights
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kWeights = (kStack ? 1 : kP) * kTileBytes;  // of one buffer
  // Softmax threads: one for each row and group of columns.
  static constexpr int kGroups = 2, kSoft = kTile * kGroups;
  static constexpr int kLoadWarp = kSoft / 32, kKeyWarp = kLoadWarp + kLoadThreads / 32,
                       kSumWarp = kKeyWarp + 1, kFindWarp = kKeyWarp + 2, kRowWarp = kKeyWarp + 3,
                       kThreads = 32 * kRowWarp + kRowThreads;
  static constexpr uint32_t kSwizzle = kRow == 32 ? 6 : kRow == 64 ? 4 : 2;
};

// ------------------------------------------------------------------ PTX

// D += A B (D = A B unless add) of 8-bit operands.  A product of M = 128 takes
// 32 + N/4 cycles in either kind (N 16 to 128, K 16 elements of 16 bits or 32 of
// 8), whichever operand is transposed.
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint32_t ahi, uint32_t b, uint32_t bhi,
                                     uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\n"
      "mov.b64 x, {%1, %2};\nmov.b64 y, {%3, %4};\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n}\n" ::"r"(d),
      "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float2 numbers2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ------------------------------------------------------------------ kernel

// Where rows lie that location vectors name: tail ring, pages, hot cache, and no
// rows for the fourth value that the two bits can have.
struct Tier {
  const uint8_t* base;
  uint32_t rows;
};

struct Control {
  static constexpr int kRowSlots = 3;  // tiles whose row addresses are found ahead
  // Barriers.  Those of buffers that a warp may be a use behind on come in
  // pairs, by the tile's number, so that their phases cannot lap each other.
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t qfull, sfull[2], sread[2], pfull[2], odone[2], oempty, rfull[kRowSlots], rempty[kRowSlots];
  uint64_t drain, segfull[kSegments], segempty[kSegments];
  Segment seg[kSegments];  // from the finding warp to the others
  Tier tier[4];
  const uint8_t* row[kRowSlots][kTile];
  uint32_t all[kRowSlots];  // none of them is null
  uint32_t word[2][kTile];  // the row warp's: entries or page slots, and positions in a list
  int32_t position[2][kTile];
  float scale[kRowSlots][2][kTile];  // the rows' key and value scales, loaded with the rows
  int64_t out_off[64];
  int32_t lse_at[64];
  int32_t col_lo[64], col_hi[64];
  alignas(16) float m[64], base[64], fac[64];
  alignas(16) float qk[2][64];  // what a column's coded scores are multiplied by, by segment
  float part[4][64];
  uint32_t odd[4];    // rows of the tile whose products are taken by hand
  const uint8_t* odd_row;
  uint32_t o_begun;   // the segment's sums hold such products before the first tile's
  uint32_t tmem;
  volatile uint32_t gave_up;
};
enum Bar {  // places in Control's order
  kBarEmpty = kMaxSlots, kBarQfull = 2 * kMaxSlots, kBarSfull, kBarSread = kBarSfull + 2,
  kBarPfull = kBarSread + 2, kBarOdone = kBarPfull + 2, kBarOempty = kBarOdone + 2, kBarRfull,
  kBarRempty = kBarRfull + Control::kRowSlots, kBarDrain = kBarRempty + Control::kRowSlots,
  kBarSegfull, kBarSegempty = kBarSegfull + kSegments, kBarriers = kBarSegempty + kSegments
};
static_assert(offsetof(Control, drain) == 8 * kBarDrain, "barrier table");
constexpr uint32_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;
static_assert(kControlBytes <= 14336, "32 columns of latent rows just have slots for two tiles");

// A value that all lanes have alike, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

// A ring position `k` slots further on.
__device__ __forceinline__ Ring further(Ring r, int k, int n) {
  r.slot += k;
  while (r.slot >= n) {
    r.slot -= n;
    r.phase ^= 1;
  }
  return r;
}

// Queries of a segment in pieces: coded part [chunk][piece][column][128 B], wide
// part [column][128 B], zeros past the elements and the columns; sixteen threads
// have a column.  By the softmax warps, which have nothing else to do then: at
// the first segment, and later between a segment's last weights and its sums.
// Elements wait for their column's largest in the pieces' own places, so that
// what comes after is a short loop: code that runs once a segment is fetched
// anew each time.
template <int N, bool F16, int MAXI>
__device__ __noinline__ void split_queries(const Params<MAXI>& P, uint8_t* sm, Control& ctl,
                                           const Segment& s, int tid, float* qk) {
  using S = Pieces<N, F16>;
  const AttendCommon& c = P.c;
  const PackedPlan& pl = P.plan;
  const AttendItem& it = s.it;
  const bool aligned = !(((uintptr_t)it.q | c.q_qs | c.q_hs) & 15);
  const int piece = tid & 15;
#pragma unroll 1
  for (int col = tid >> 4; col < N; col += S::kSoft / 16) {
    const bool on = col < s.cols;
    const int qc = s.col0 + min(col, s.cols - 1);
    const int qi = it.loc ? s.qbase : qc / c.group;
    const int h = s.g * c.group + (it.loc ? qc : qc % c.group);
    const uint8_t* src = it.q + qi * c.q_qs + h * c.q_hs + 16 * piece;
    uint8_t* const to = sm + pl.off_q + col * 128 + ((piece >> 1 ^ (col & 7)) << 4) + (piece & 1) * 8;
    uint32_t top = 0;  // the largest magnitude's bits
    // six groups of eight elements: the chunks' of the coded part, and the wide one
    uint4 w[6];
#pragma unroll
    for (int ch = 0; ch < 6; ++ch) {
      const int el = (ch < 5 ? ch * 128 : pl.key8) + piece * 8;
      const bool in = on && (ch < 5 ? el < pl.key8 : piece * 8 < pl.wide);
      const uint8_t* p = src + 2 * (el - piece * 8);
      w[ch] = make_uint4(0, 0, 0, 0);
      if (in && aligned) w[ch] = *reinterpret_cast<const uint4*>(p);
      if (in && !aligned)
#pragma unroll 1
        for (int k = 7; k >= 0; --k)  // shifted in from the end
          w[ch] = make_uint4(w[ch].x << 16 | reinterpret_cast<const uint16_t*>(p)[k],
                             w[ch].y << 16 | w[ch].x >> 16, w[ch].z << 16 | w[ch].y >> 16,
                             w[ch].w << 16 | w[ch].z >> 16);
    }
#pragma unroll
    for (int ch = 0; ch < 5; ++ch) {
      if (ch >= pl.key_chunks) continue;
      for (const uint32_t u : {w[ch].x, w[ch].y, w[ch].z, w[ch].w})
        top = max(top, max(u & 0x7FFFu, u >> 16 & 0x7FFFu));
      *reinterpret_cast<uint2*>(to + ch * (S::kQ * N * 128)) = make_uint2(w[ch].x, w[ch].y);
      *reinterpret_cast<uint2*>(to + ch * (S::kQ * N * 128) + N * 128) = make_uint2(w[ch].z, w[ch].w);
    }
    if (pl.wide && piece < 8)
      *reinterpret_cast<uint4*>(sm + pl.off_qw + col * 128 + ((piece ^ (col & 7)) << 4)) = w[5];
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(~0u, top, x));
    // 2^e: the least that brings the largest to 448 = 0.875 * 2^9
    const bool finite = top < (F16 ? 0x7C00u : 0x7F80u);
    const float most = F16 ? __half2float(__ushort_as_half((unsigned short)top))
                           : __uint_as_float(top << 16);
    const uint32_t bits = __float_as_uint(most);
    int e = (int)(bits >> 23) - 126 - ((bits & 0x7FFFFFu) <= 0x600000u ? 9 : 8);
    // (-126: of smaller queries, which are bf16's last bits, 2^126 makes whole codes)
    e = most == 0.f ? 0 : min(max(e, -126), 120);
    const float down = finite ? __int_as_float((127 - e) << 23) : NAN;
    if (piece == 0)
      qk[col] = c.scale * 1.44269504088896341f * __int_as_float((127 + (e >> 1)) << 23) *
                __int_as_float((127 + e - (e >> 1) + kAside) << 23);  // neither half out of range
#pragma unroll 1
    for (int ch = 0; ch < pl.key_chunks; ++ch) {
      uint8_t* const at = to + ch * (S::kQ * N * 128);
      const uint2 x = *reinterpret_cast<const uint2*>(at), y = *reinterpret_cast<const uint2*>(at + N * 128);
      const uint32_t in[4] = {x.x, x.y, y.x, y.y};
      uint32_t out[S::kQ][2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 f;
        if (F16) f = __half22float2(*reinterpret_cast<const __half2*>(&in[k]));
        else f = make_float2(__uint_as_float(in[k] << 16), __uint_as_float(in[k] & 0xFFFF0000u));
        f.x *= down;
        f.y *= down;
#pragma unroll
        for (int p = 0; p < S::kQ; ++p) {
          const uint32_t z = codes2(f.x, f.y);
          const float2 g = numbers2(z);
          f.x -= g.x;
          f.y -= g.y;
          if (k & 1) out[p][k >> 1] |= z << 16;
          else out[p][k >> 1] = z;
        }
      }
#pragma unroll
      for (int p = 0; p < S::kQ; ++p)
        *reinterpret_cast<uint2*>(at + p * (N * 128)) = make_uint2(out[p][0], out[p][1]);
    }
  }
  fence_async();
  __syncwarp();
  if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.qfull));
}

// Loading warps: rows tile by tile, 128 bytes of each row a slot.  A thread has
// 16 bytes of every 128 of eight rows.  Copies alone bring 656-byte rows at 7.7
// TB/s (64 verify blocks' rows, mostly from L2) and 6.2 (a history, from DRAM).
// A row of an odd number of 16-byte pieces begins inside a 32-byte sector every
// other time, and its slices then touch one sector more each; copies shifted to
// sectors move a third fewer, but were slower (7.1 and 5.9 TB/s).
template <int MAXI>
__device__ void load_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid) {
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const PackedPlan& pl = P.plan;
  const int piece = tid & 7, r0 = tid >> 3;  // rows r0 + 16 i
  const uint32_t mine = smem_u32(sm) + pl.off_rows + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
  const int nk = pl.key_chunks, nw = pl.wide ? 1 : 0;
  Ring ring, rr, seg;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    if (__any_sync(~0u, ctl.gave_up) || !s.cols) break;
    const int32_t v0 = s.v0, v1 = s.v1;
    const uint32_t key_at = s.g * pl.key8 + 16 * piece;
    const uint32_t wide_at = pl.off_wide + s.g * pl.wide * 2 + 16 * piece + 128;  // u is -1 there
    const uint32_t val_at = pl.off_value + s.g * c.dv + 16 * piece;
    const uint32_t scale_at = pl.off_scale + 4 * s.g;
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile) {
      warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
      const uint8_t* row[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = ctl.row[rr.slot][r0 + 16 * i];
      const bool all = ctl.all[rr.slot];
      // the scales arrive with the tile's first slot
      const uint8_t* const at = ctl.row[rr.slot][tid];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         smem_u32(&ctl.scale[rr.slot][k][tid])),
                     "l"(at ? at + scale_at + 4 * k * pl.value_scales : c.tail), "r"(at ? 4 : 0)
                     : "memory");
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
      rr.next(Control::kRowSlots);
      // slots: 128 bytes of each row of the keys, the wide elements, the values
#pragma unroll 1
      for (int i = 0; i < pl.per_tile; ++i) {
        const int u = i < nk ? i : i - nk - nw;
        const uint32_t from = (i < nk ? key_at : u < 0 ? wide_at : val_at) + u * 128;
        const int left = u < 0 ? 2 * pl.wide : (i < nk ? pl.key8 : c.dv) - u * 128;
        warp_wait(smem_u32(&ctl.empty[ring.slot]), ring.phase ^ 1, until);
        const uint32_t dst = mine + ring.slot * kChunk;
        if (all && left >= 128) {
          // (a wait that ran out may leave a null beside an old `all`: any row then)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst + k * 2048),
                         "l"((row[k] ? row[k] : c.tail) + from)
                         : "memory");
        } else {  // zeros for rows that are none and past the slice
          const bool in = piece * 16 < left;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst + k * 2048),
                         "l"(in && row[k] ? row[k] + from : c.tail), "r"(in && row[k] ? 16 : 0)
                         : "memory");
        }
        // The slot's barrier gets this thread's arrival when its copies so far
        // have landed; the issuing warps make them visible to the tensor cores.
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&ctl.full[ring.slot]))
                     : "memory");
        ring.next(pl.slots);
      }
    }
    __syncwarp();
    if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Row warp: the addresses of every tile's rows, ahead of the loading warps.
// What a row's address hangs on (its entry, or its page's slot) is asked for a
// tile ahead, the list position that a union entry hangs on two tiles, by copies
// into shared memory, so that the four rows of a lane take one short loop.
template <int MAXI>
__device__ void place_rows(const Params<MAXI>& P, Control& ctl, int lane) {
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const uint32_t rb = c.row_bytes;
  const int shift = c.page_shift, in_page = (1 << shift) - 1;
  const uint32_t words = smem_u32(&ctl.word[0][0]), positions = smem_u32(&ctl.position[0][0]);
  auto fetch = [&](uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  };
  Ring seg, rr;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    if (__any_sync(~0u, ctl.gave_up) || !s.cols) break;
    const AttendItem& it = s.it;
    const bool located = it.loc != nullptr;
    // rows [lo, lo + n) of the job (fewer than 2^31: a source's length is)
    const int32_t lo = (int32_t)s.lo;
    const uint32_t n = (uint32_t)(s.hi - s.lo);
    // located: the query's entries, or its positions in a list of `listed`
    // entries; histories: its first row, and the first one that the ring holds
    const int64_t entries = located ? (int64_t)s.qbase * it.len : 0;
    const int32_t* const index = located && it.index ? it.index + entries : nullptr;
    const uint32_t* const from = located ? it.loc + (index ? 0 : entries)
                                         : (const uint32_t*)c.map + (size_t)it.pair * c.Pmax;
    const uint32_t listed = index ? (uint32_t)min((int64_t)it.Q * it.len, (int64_t)INT32_MAX)
                            : located ? 0x7FFFFFFFu : (uint32_t)it.complete;
    const int32_t first = (int32_t)it.first, ring = (int32_t)(it.first + it.len) - c.T;
#pragma unroll 1
    for (int tile = s.v0 - 2; tile < s.v1; ++tile) {
      asm volatile("cp.async.wait_all;" ::: "memory");  // asked for a tile ago
      if (tile >= s.v0) {
        warp_wait(smem_u32(&ctl.rempty[rr.slot]), rr.phase ^ 1, until);
        bool all = true;
#pragma unroll 1
        for (int k = lane; k < kTile; k += 32) {
          const int32_t i = tile * kTile + k;
          uint32_t w = ctl.word[tile & 1][k];
          const uint8_t* p = nullptr;
          if ((uint32_t)(i - lo) >= n) {
          } else if (located) {
            const uint32_t x = w & 0x3FFFFFFFu;
            const Tier& t = ctl.tier[w >> 30];
            if (x < t.rows) p = t.base + (size_t)x * rb;
            else if (w < kEndLoc) atomicOr(c.status, kStatusEloc);
          } else {
            const uint32_t r = (uint32_t)(first + i);
            if ((int32_t)r >= ring) p = c.tail + ((size_t)it.pair * c.T + r % (uint32_t)c.T) * rb;
            else if ((int32_t)w >= 0) p = c.opt + (((size_t)w << shift) + (r & in_page)) * rb;
            else p = it.host + (size_t)r * rb;
          }
          ctl.row[rr.slot][k] = p;
          all &= p != nullptr;
        }
        // the vote orders no stores: all lanes' addresses have to be behind the arrival
        all = __all_sync(~0u, all);
        if (lane == 0) ctl.all[rr.slot] = all;
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&ctl.rfull[rr.slot]));
        rr.next(Control::kRowSlots);
      }
#pragma unroll 1
      for (int k = lane; k < kTile; k += 32) {
        // a position past the list is a location of no tier; a page that is not
        // complete has no slot
        const int32_t i = (tile + 1) * kTile + k;
        const uint32_t x = index ? (uint32_t)ctl.position[tile & 1][k]
                           : located ? (uint32_t)i : (uint32_t)(first + i) >> shift;
        const bool on = tile >= s.v0 - 1 && (uint32_t)(i - lo) < n;
        if (on && x < listed) fetch(words + ((tile + 1 & 1) * kTile + k) * 4, from + x);
        else ctl.word[tile + 1 & 1][k] = index && (int32_t)x >= 0 ? 3u << 30 : kNoLoc;
        const int32_t next = i + kTile;
        if (index && (uint32_t)(next - lo) < n) fetch(positions + ((tile + 1 & 1) * kTile + k) * 4, index + next);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
}

// Two warps issue the products, one those of the scores and one those of the
// sums: for one alone, waiting for each slot and issuing its four products took
// longer (260 cycles a slot) than making them (160).  All lanes of a warp walk
// the same path, one of them issues.
template <int N, bool F16, int MAXI>
__device__ void issue_scores(const Params<MAXI>& P, uint8_t* sm, Control& ctl) {
  using S = Pieces<N, F16>;
  const Patience until{&ctl.gave_up, P.c.polls};
  const PackedPlan& pl = P.plan;
  const uint32_t base = smem_u32(sm), tm_s = uniform(ctl.tmem);
  // float accumulators, operand types (8 bits: 0 e4m3; 16 bits: 0 f16, 1 bf16),
  // N, M = 128
  constexpr uint32_t common = 1u << 4 | 8u << 24, type = F16 ? 0u : 1u;
  constexpr uint32_t id_key = common | (uint32_t)(S::kQ * N >> 3) << 17;
  constexpr uint32_t id_wide = common | type << 7 | type << 10 | (uint32_t)(N >> 3) << 17;
  constexpr uint32_t hi = operand_hi(1024, 2);
  const uint32_t q_lo = operand_lo(base + pl.off_q, 16), qw_lo = operand_lo(base + pl.off_qw, 16);
  const uint32_t rows_lo = operand_lo(base + pl.off_rows, 16);
  const bool lead = elected(), two = pl.bufs == 2;
  const int nk = pl.key_chunks, parts = nk + (pl.wide ? 1 : 0), held = pl.shared ? pl.units : 0;
  Ring ring, seg;
  uint32_t n = 0, qphase = 0;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    const int32_t v0 = uniform(s.v0), v1 = uniform(s.v1), cols = uniform(s.cols);
    if (__any_sync(~0u, ctl.gave_up) || !cols) break;
    __syncwarp();
    if (lead) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
    if (v0 >= v1) continue;
    warp_wait(smem_u32(&ctl.qfull), qphase, until);
    fence_async();
    qphase ^= 1;
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile, ++n) {
      const uint32_t buf = two ? n & 1 : 0, use = two ? n >> 1 : n, d = tm_s + buf * pl.buf_columns;
      if (use > 0) warp_wait(smem_u32(&ctl.sread[buf]), (use - 1) & 1, until);
      // Each slot's products as soon as it has landed.  Every slot is 128 bytes wide,
      // zeros past its slice.
#pragma unroll 1
      for (int i = 0; i < parts; ++i) {
        warp_wait(smem_u32(&ctl.full[ring.slot]), ring.phase, until);
        fence_async();
        tc_after();
        if (lead) {
          const uint32_t a = rows_lo + ring.slot * (kChunk >> 4);
          if (i < nk) {
            const uint32_t b = q_lo + i * (S::kQ * N * 128 >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma8(d, a + 2 * k, hi, b + 2 * k, hi, id_key, i > 0 || k > 0);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma(d + S::kQ * N, a + 2 * k, hi, qw_lo + 2 * k, hi, id_wide, k > 0);
          }
          if (i >= held) commit(smem_u32(&ctl.empty[ring.slot]));
          if (i + 1 == parts) commit(smem_u32(&ctl.sfull[buf]));
        }
        __syncwarp();
        ring.next(pl.slots);
      }
      ring = further(ring, pl.per_tile - parts, pl.slots);
    }
  }
  if (lead) commit(smem_u32(&ctl.drain));
  __syncwarp();
}

template <int N, bool F16, int MAXI>
__device__ void issue_sums(const Params<MAXI>& P, uint8_t* sm, Control& ctl) {
  using S = Pieces<N, F16>;
  const Patience until{&ctl.gave_up, P.c.polls};
  const PackedPlan& pl = P.plan;
  const uint32_t base = smem_u32(sm), tm_o = uniform(ctl.tmem) + pl.sum_column;
  // float accumulators, A e4m3, B e5m2, both M/N-major, N, M = 128
  constexpr uint32_t id_sum =
      1u << 4 | 8u << 24 | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(S::kSum >> 3) << 17;
  constexpr uint32_t hi = operand_hi(1024, 2), hi_p = operand_hi(8 * S::kRow, S::kSwizzle);
  const uint32_t rows_lo = operand_lo(base + pl.off_rows, 16);
  const bool lead = elected(), two = pl.weight_bufs == 2;
  const int before = pl.shared ? 0 : pl.key_chunks + (pl.wide ? 1 : 0);
  const int after = pl.per_tile - before - pl.units;
  Ring ring, seg;
  uint32_t n = 0, ophase = 0;
  bool first = true;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    const int32_t v0 = uniform(s.v0), v1 = uniform(s.v1), cols = uniform(s.cols);
    if (__any_sync(~0u, ctl.gave_up) || !cols) break;
    __syncwarp();
    if (lead) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile, ++n) {
      const uint32_t p_lo = operand_lo(base + pl.off_p + (two && n & 1 ? S::kWeights : 0), 16);
      ring = further(ring, before, pl.slots);
      warp_wait(smem_u32(&ctl.pfull[n & 1]), n >> 1 & 1, until);
      if (tile == v0 && !first) {  // the previous segment's sums are read
        warp_wait(smem_u32(&ctl.oempty), ophase, until);
        ophase ^= 1;
      }
      first = false;
      tc_after();
      const bool begun = tile > v0 || uniform(*(volatile uint32_t*)&ctl.o_begun);
      if (!pl.shared) {
        const Ring end = further(ring, pl.units - 1, pl.slots);
        warp_wait(smem_u32(&ctl.full[end.slot]), end.phase, until);
        fence_async();
        tc_after();
      }
#pragma unroll 1
      for (int u = 0; u < pl.units; ++u) {
        if (lead) {
          const uint32_t a = rows_lo + ring.slot * (kChunk >> 4), d = tm_o + u * S::kSum;
#pragma unroll
          for (int p = 0; p < (S::kStack ? 1 : S::kP); ++p)
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma8(d, a + k * (4096 >> 4), hi, p_lo + (p * S::kTileBytes + k * 32 * S::kRow >> 4), hi_p,
                   id_sum, begun || k > 0 || p > 0);
          commit(smem_u32(&ctl.empty[ring.slot]));
          if (u + 1 == pl.units) commit(smem_u32(&ctl.odone[n & 1]));
        }
        __syncwarp();
        ring.next(pl.slots);
      }
      ring = further(ring, after, pl.slots);
    }
  }
  // nothing of either warp's is in flight when tensor memory goes back
  if (lead) commit(smem_u32(&ctl.drain));
#pragma unroll 1
  for (uint32_t k = 0; k < kAttendPolls && !bar_try(smem_u32(&ctl.drain), 0); ++k) {
  }
  __syncwarp();
}

// Whether none of the n codes at `p` is a NaN.
__device__ bool finite_codes(const uint8_t* p, int n) {
  bool ok = true;
#pragma unroll 1
  for (int k = 0; k < n; k += 16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + k));
    for (const uint32_t w : {v.x, v.y, v.z, v.w})
      ok &= __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) == 0;
  }
  return ok;
}

// What a thread knows of its row of the tile: its scales.
struct RowScale {
  float key;      // 2^(k - kAside), 0 without a row
  float value;    // v
  float inverse;  // 2^-v, 0 without a row
};

// A row's scores of B columns in log2 units, value scale included.
template <int N, bool F16, int B>
__device__ __forceinline__ void scores(uint32_t tm, const float* qk, float wide, bool has_wide,
                                       const RowScale& z, bool row, float* x) {
  using S = Pieces<N, F16>;
  float v[(S::kQ + 1) * B];
  __syncwarp();
#pragma unroll
  for (int p = 0; p < S::kQ + 1; ++p)
    if (p < S::kQ || has_wide)
#pragma unroll
      for (int k = 0; k < B; k += 8) tm_load8(tm + p * N + k, v + p * B + k);
  tm_wait(v);
#pragma unroll
  for (int k = 0; k < B; k += 4) {
    const float4 q4 = *reinterpret_cast<const float4*>(qk + k);
    const float q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y = v[k + i];
#pragma unroll
      for (int p = 1; p < S::kQ; ++p) y += v[p * B + k + i];
      y = fmaf(y * z.key, q[i], z.value);
      if (has_wide) y = fmaf(v[S::kQ * B + k + i], wide, y);
      x[k + i] = row ? y : -INFINITY;
    }
  }
}

// The products of the tile's rows marked `odd` (thread = row and half of the
// columns), added to the sums of the columns that see them; their staged
// values become zeros.  Runs while no product is in flight: those of the
// tiles before are complete.
template <int N, bool F16, int MAXI>
__device__ __noinline__ void odd_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid,
                                      bool odd, const uint8_t* value, Ring at, int32_t tile0,
                                      bool first, uint32_t tm_scores, const float* qk,
                                      const RowScale& z) {
  using S = Pieces<N, F16>;
  constexpr int C = N / S::kGroups, kSoftThreads = S::kSoft;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const PackedPlan& pl = P.plan;
  const int r = tid & (kTile - 1), k0 = tid / kTile * C;
  const uint32_t tm_o = ctl.tmem + ((uint32_t)(r & ~31) << 16) + k0 + pl.sum_column;
  const float wide = c.scale * 1.44269504088896341f;
  const uint32_t marked = __ballot_sync(~0u, odd);
  if ((tid & 31) == 0 && tid < kTile) ctl.odd[tid >> 5] = marked;
  float v[8];
  if (first) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll 1
    for (int u = 0; u < pl.units * (S::kSum / N); ++u)
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
        scores<N, F16, 8>(tm_scores + k, qk + k0 + k, wide, pl.wide > 0, z, true, v);
        if (r == i)
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int col = k0 + k + n;
            const bool seen = tile0 + i >= ctl.col_lo[col] && tile0 + i < ctl.col_hi[col];
            ctl.part[0][col] = seen ? exp2_fast(v[n] - ctl.base[col]) : 0.f;
          }
      }
      if (tid == i) ctl.odd_row = value;
    }
    named_sync(1, kSoftThreads);
    const uint8_t* y = ctl.odd_row;
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u) {
      const int d = u * 128 + r;
      const float e = d < c.dv ? numbers2(y[d]).x : 0.f;
#pragma unroll 1
      for (int k = 0; k < C; k += 8) {
        tm_load(tm_o + u * S::kSum + k, v);
#pragma unroll
        for (int n = 0; n < 8; ++n)
          if (ctl.part[0][k0 + k + n] != 0.f) v[n] += ctl.part[0][k0 + k + n] * e;
        tm_store(tm_o + u * S::kSum + k, v);
      }
    }
    named_sync(1, kSoftThreads);
  }
#pragma unroll 1
  for (int u = 0; u < pl.units; ++u) {
    warp_wait(smem_u32(&ctl.full[at.slot]), at.phase, until);
    if (odd && tid < kTile) {
      uint8_t* to = sm + pl.off_rows + at.slot * kChunk + r * 128;
#pragma unroll 1
      for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(to + 16 * k) = make_uint4(0, 0, 0, 0);
    }
    at.next(pl.slots);
  }
}

// Softmax warps: a thread has one row of the tile and some of the columns; then
// the segment's output.
template <int N, bool F16, int MAXI>
__device__ void softmax_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid, float* parts) {
  using S = Pieces<N, F16>;
  constexpr int C = N / S::kGroups, kSoftThreads = S::kSoft;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const PackedPlan& pl = P.plan;
  const int lane = tid & 31, r = tid & (kTile - 1), quarter = r >> 5, k0 = tid / kTile * C;
  const uint32_t tm_s = ctl.tmem + ((uint32_t)(r & ~31) << 16) + k0, tm_o = tm_s + pl.sum_column;
  const float wide = c.scale * 1.44269504088896341f;  // log2 e
  const bool quads_ok = !(((uintptr_t)c.o_qs | c.o_hs) & 7);  // outputs store four elements at once
  const int turn = S::kRow == 32 ? (r >> 2) & 1 : S::kRow == 64 ? (r >> 1) & 3 : r & 7;
  const int nk = pl.key_chunks, nw = pl.wide ? 1 : 0;
  const bool two = pl.bufs == 2;
  Ring rr, tr, seg;  // row slots, first ring slot of the tile, segments
  uint32_t n = 0, n_queries = 0;  // tiles and segments with tiles so far
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto sum = [](float a, float b) { return a + b; };
  // waits for tile m's sums
  auto summed = [&](uint32_t m) {
    warp_wait(smem_u32(&ctl.odone[m & 1]), m >> 1 & 1, until);
    tc_after();
  };
#pragma unroll 1
  for (bool begin = true;; begin = false) {  // first for the queries of the first segment alone
    const Segment& s = ctl.seg[seg.slot];
    const AttendItem& it = s.it;
    float l[C];
#pragma unroll
    for (int k = 0; k < C; ++k) l[k] = 0.f;
    bool some = false;
    if (!begin) {
      warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
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
      some = s.v0 < s.v1;
      const float* const qk = ctl.qk[n_queries & 1];
      if (some) ++n_queries;

#pragma unroll 1
      for (int tile = s.v0; tile < s.v1; ++tile, ++n) {
        const int32_t j = tile * kTile + r;
        const bool ragged = tile * kTile < all_lo || tile * kTile + kTile > all_hi;
        const uint32_t buf = two ? n & 1 : 0, tm = tm_s + buf * pl.buf_columns;
        warp_wait(smem_u32(&ctl.sfull[buf]), (two ? n >> 1 : n) & 1, until);
        tc_after();
        // the row and its scales: there since before its scores were made
        warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
        const uint8_t* const row = ctl.row[rr.slot][r];
        const float ks = ctl.scale[rr.slot][0][r];
        const uint32_t vbits = __float_as_uint(ctl.scale[rr.slot][1][r]) >> 23 & 255;
        const RowScale z{ks * __int_as_float((127 - kAside) << 23), (float)((int)vbits - 127),
                         row ? __uint_as_float(max(1u, min(253u, 254u - vbits)) << 23) : 0.f};
        float x[C];  // scores and value scale in log2 units
#pragma unroll
        for (int k = 0; k < C; k += 8)
          scores<N, F16, 8>(tm + k, qk + k0 + k, wide, pl.wide > 0, z, row != nullptr, x + k);
        tc_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
          if (!ragged) bar_arrive(smem_u32(&ctl.sread[buf]));
        }
        rr.next(Control::kRowSlots);
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
        if (n >= (uint32_t)pl.weight_bufs) summed(n - pl.weight_bufs);
        uint8_t* const weights = sm + pl.off_p + r * S::kRow +
                                 (pl.weight_bufs == 2 && n & 1 ? S::kWeights : 0);
        bool odd = false;
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
            ctl.fac[tid] = old == -INFINITY ? 0.f : exp2_fast(old - m);
            ctl.m[tid] = m;
            ctl.base[tid] = m == -INFINITY ? 0.f : m - kLift;
          }
          named_sync(1, kSoftThreads);
          if (tile > s.v0) {
            summed(n - 1);
#pragma unroll
            for (int k = 0; k < C; k += 8) {
              float f[8];
              bool same = true;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                f[i] = ctl.fac[k0 + k + i];
                l[k + i] *= f[i];
                same &= f[i] == 1.f;
              }
              if (same) continue;  // as for all lanes of the warp
#pragma unroll 1
              for (int u = 0; u < pl.units; ++u) {
                constexpr int kSums = S::kSum / N;
                float v[8 * kSums];
                __syncwarp();
#pragma unroll
                for (int p = 0; p < kSums; ++p) tm_load8(tm_o + u * S::kSum + p * N + k, v + 8 * p);
                tm_wait(v);
#pragma unroll
                for (int p = 0; p < kSums; ++p) {
                  float y[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i) y[i] = v[8 * p + i] * f[i];
                  tm_store(tm_o + u * S::kSum + p * N + k, y);
                }
              }
            }
          }
        }
        // A row that only some of the columns see would reach the others too
        // if its value is not finite (0 x NaN): such rows leave the tile, and
        // their products are added by hand to the columns that see them.
        if (ragged) {
          const uint8_t* value = row + (pl.shared ? s.g * pl.key8 : pl.off_value + s.g * c.dv);
          if (row && (j < all_lo || j >= all_hi)) odd = !finite_codes(value, c.dv);
          if (named_or(1, kSoftThreads, odd)) {
            if (tile > s.v0) summed(n - 1);
            odd_rows<N, F16>(P, sm, ctl, tid, odd, value,
                             pl.shared ? tr : further(tr, nk + nw, pl.slots), tile * kTile,
                             tile == s.v0, tm, qk, z);
          }
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(smem_u32(&ctl.sread[buf]));
        }
        // weights in pieces, in the swizzled layout
#pragma unroll
        for (int k = 0; k < C; k += 8) {
          const float4 b0 = *reinterpret_cast<const float4*>(&ctl.base[k0 + k]);
          const float4 b1 = *reinterpret_cast<const float4*>(&ctl.base[k0 + k + 4]);
          const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
          uint32_t w[S::kP][2];
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            __half2 h[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float p0 = exp2_fast(x[k + i + 2 * q] - b[i + 2 * q]);
              const float p1 = exp2_fast(x[k + i + 2 * q + 1] - b[i + 2 * q + 1]);
              l[k + i + 2 * q] = fmaf(p0, z.inverse, l[k + i + 2 * q]);
              l[k + i + 2 * q + 1] = fmaf(p1, z.inverse, l[k + i + 2 * q + 1]);
              h[q] = __floats2half2_rn(p0, p1);
            }
#pragma unroll
            for (int p = 0; p < S::kP; ++p) {
              uint32_t u[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                // the upper byte of each number, rounded to nearest, and the rest
                u[q] = (*reinterpret_cast<uint32_t*>(&h[q]) + 0x00800080u) & 0xFF00FF00u;
                h[q] = __hsub2(h[q], *reinterpret_cast<__half2*>(&u[q]));
              }
              w[p][i / 4] = odd ? 0 : __byte_perm(u[0], u[1], 0x7531);
            }
          }
#pragma unroll
          for (int p = 0; p < S::kP; ++p) {
            const int at = (S::kStack ? p * N : 0) + k0 + k;
            *reinterpret_cast<uint2*>(weights + (S::kStack ? 0 : p * S::kTileBytes) +
                                      ((at >> 4 ^ turn) << 4) + (at & 8)) = make_uint2(w[p][0], w[p][1]);
          }
        }
        tr = further(tr, pl.per_tile, pl.slots);
        fence_async();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&ctl.pfull[n & 1]));
      }
    }

    // the next segment's queries: its scores can be made beside this one's sums
    // and outputs (the queries here are done with: so are their scores)
    {
      Ring next = seg;
      if (!begin) next.next(kSegments);
      warp_wait(smem_u32(&ctl.segfull[next.slot]), next.phase, until);
      const Segment& t = ctl.seg[next.slot];
      const bool split = !ctl.gave_up && t.cols && t.v0 < t.v1;
      if (__all_sync(~0u, split)) split_queries<N, F16>(P, sm, ctl, t, tid, ctl.qk[n_queries & 1]);
    }
    if (begin) continue;

    named_sync(1, kSoftThreads);
#pragma unroll
    for (int k = 0; k < C; k += 8) {
      const float y = fold8(l + k, lane, sum);
      if (lane < 8) ctl.part[quarter][k0 + k + lane] = y;
    }
    named_sync(1, kSoftThreads);
    const bool whole = s.whole();
    float* part = nullptr;
    if (!whole) {
      // a block leaves at most two parts: of the job it begins inside of,
      // and of the job that it ends inside of
      const int slot = 2 * blockIdx.x + (s.t0 == 0 ? 1 : 0);
      part = parts + (size_t)slot * N * (c.dv + 2);
    }
    if (tid < N) {
      const float sums = ctl.part[0][tid] + ctl.part[1][tid] + ctl.part[2][tid] + ctl.part[3][tid];
      if (whole) {
        ctl.fac[tid] = sums == 0.f ? 0.f : 1.f / sums;
        if (it.lse && ctl.lse_at[tid] >= 0)
          it.lse[ctl.lse_at[tid]] =
              sums == 0.f ? -INFINITY : (ctl.base[tid] + log2f(sums)) * 0.693147180559945309f;
      } else {
        ctl.fac[tid] = 1.f;
        part[(size_t)N * c.dv + tid] = sums == 0.f ? -INFINITY : ctl.base[tid];
        part[(size_t)N * c.dv + N + tid] = sums;
      }
    }
    named_sync(1, kSoftThreads);
    if (some) summed(n - 1);
    const bool quads = quads_ok && !((uintptr_t)it.out & 7);
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u) {
      // after the exchange lane i of four has column k + i of four elements
      const int d = u * 128 + quarter * 32 + (lane & ~3);
#pragma unroll
      for (int k = 0; k < C; k += 8) {
        float v[8] = {};
        if (some) {
          constexpr int kSums = S::kSum / N;
          float y[8 * kSums];
          __syncwarp();
#pragma unroll
          for (int p = 0; p < kSums; ++p) tm_load8(tm_o + u * S::kSum + p * N + k, y + 8 * p);
          tm_wait(y);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = y[i];
#pragma unroll
            for (int p = 1; p < kSums; ++p) v[i] += y[8 * p + i];
          }
        }
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          transpose4(v + q, lane);
          const int col = k0 + k + q + (lane & 3);
          const float f = ctl.fac[col];
          const bool on = d < c.dv && col < s.cols;
          float y[4];
          // a weight sum of zero leaves products of zero: the output is zero
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = f == 0.f ? 0.f : v[q + i] * f;
          if (!whole) {
            if (on)
              *reinterpret_cast<float4*>(part + (size_t)col * c.dv + d) =
                  make_float4(y[0], y[1], y[2], y[3]);
            continue;
          }
          uint32_t w[2];
          if (F16) {
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
      }
      __syncwarp();
    }
    if (some) {
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.oempty));
    }
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
}

template <int N, bool F16, int MAXI>
__global__ void __launch_bounds__(Pieces<N, F16>::kThreads, 1)
    attend_packed_kernel(const __grid_constant__ Params<MAXI> P, float* parts) {
  using S = Pieces<N, F16>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  Control& ctl = *reinterpret_cast<Control*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  for (int k = tid; k < Control::kRowSlots * kTile; k += S::kThreads) (&ctl.row[0][0])[k] = nullptr;
  if (tid < Control::kRowSlots) ctl.all[tid] = 0;
  if (warp == S::kRowWarp && (tid & 31) < 4) {
    const int k = tid & 3;
    const AttendCommon& c = P.c;
    ctl.tier[k] = {k == kTierTail ? c.tail : k == kTierOpt ? c.opt : c.hot,
                   k == kTierTail ? c.tail_rows : k == kTierOpt ? c.opt_rows : k == kTierHot ? c.hot_rows : 0};
  }
  if (warp == S::kKeyWarp) {
#pragma unroll
    for (int k = 0; k < kBarriers; k += 32) {
      const int i = k + (tid & 31);
      const bool soft = i == kBarQfull || (i >= kBarSread && i < kBarOdone) || i == kBarOempty;
      const bool rows = i >= kBarRfull && i < kBarRempty, read = i >= kBarRempty && i < kBarDrain;
      if (i < kBarriers)
        bar_init(smem_u32(&ctl.full[0]) + 8 * i,
                 i < kBarEmpty ? kLoadThreads : soft ? S::kSoft / 32 : rows ? kRowThreads / 32
                 : read ? (S::kSoft + kLoadThreads) / 32 : i == kBarDrain ? 2
                 : i >= kBarSegempty ? S::kThreads / 32 - 1 : 1);
    }
    ctl.gave_up = P.c.polls == 0;  // nothing is waited for then
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == S::kFindWarp) {
    find_segments(P, ctl);  // meets the others' barrier inside
  } else {
    tc_before();
    __syncthreads();
    tc_after();
    if (warp < S::kLoadWarp) softmax_rows<N, F16>(P, sm, ctl, tid, parts);
    else if (warp < S::kKeyWarp) load_rows(P, sm, ctl, tid - S::kSoft);
    else if (warp == S::kKeyWarp) issue_scores<N, F16>(P, sm, ctl);
    else if (warp == S::kSumWarp) issue_sums<N, F16>(P, sm, ctl);
    else place_rows(P, ctl, tid - 32 * S::kRowWarp);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == S::kKeyWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(ctl.tmem),
                 "r"(kTmemColumns)
                 : "memory");
  if (tid == 0 && ctl.gave_up) atomicOr(P.c.status, kStatusEtimeout);
}

// ------------------------------------------------------------------ host

template <int N, bool F16>
PackedPlan plan_n(const AttendCommon& c, const PackedLayout& l) {
  using S = Pieces<N, F16>;
  PackedPlan p{};
  p.shared = l.shared;
  p.key8 = l.key8;
  p.wide = l.wide;
  p.key_chunks = (l.key8 + 127) / 128;
  p.units = (c.dv + 127) / 128;
  const int nw = l.wide ? 1 : 0, nv = l.shared ? 0 : p.units;
  p.per_tile = p.key_chunks + nw + nv;
  p.off_value = l.off_value;
  p.off_wide = l.off_wide;
  p.off_scale = l.off_scale;
  p.value_scales = l.shared ? 0 : l.kv;
  p.off_q = kControlBytes;
  p.off_qw = p.off_q + (uint32_t)p.key_chunks * S::kQ * N * 128;
  p.off_p = p.off_qw + (uint32_t)nw * N * 128;
  p.buf_columns = (S::kQ + nw) * N;
  const int sums = p.units * S::kSum;
  auto slots = [&](int weight_bufs) {
    const uint32_t used = 1024 + p.off_p + (uint32_t)weight_bufs * S::kWeights;
    return used < kSmemLimit ? std::min<int>(kMaxSlots, (kSmemLimit - used) / kChunk) : 0;
  };
  // The next tile's keys need slots of their own while this tile holds its
  // values: slots are taken in order, so that the ring has to reach from the
  // first value (shared rows: the first slot) of a tile to the next one's last
  // key.  A second buffer of weights may cost slots beyond that.
  const int two = (l.shared ? 2 : 1) * p.per_tile;
  p.weight_bufs = slots(2) >= two ? 2 : 1;
  p.slots = slots(p.weight_bufs);
  p.bufs = 2 * p.buf_columns + sums <= kTmemColumns && p.slots >= two ? 2 : 1;
  p.sum_column = p.bufs * p.buf_columns;
  p.off_rows = p.off_p + (uint32_t)p.weight_bufs * S::kWeights;
  p.smem = 1024 + p.off_rows + (uint32_t)p.slots * kChunk;
  return p;
}

// Shared rows stay until their sums are made: without slots for two tiles,
// loads, scores, weights and sums would follow each other (128 heads in blocks of
// 64 columns 209 us, of 32 178).  Others need those of a tile's scores, or of its
// sums, at once.
bool plan_fits(const PackedPlan& p) {
  const int values = p.shared ? 0 : p.units;
  return p.slots >= (p.shared ? 2 * p.per_tile : std::max(p.per_tile - values, values));
}

// Sixteen columns are taken whether they fit so or not (shared rows of more than 512
// coded elements and wide ones do not).  All that a plan needs is a tile of shared
// rows, or the scores' part and the values of others, in the ring at once: six slots
// at most, of five chunks of keys and one of wide elements.  Any layout has those:
template <bool F16>
constexpr uint32_t kFewestSlots =
    (kSmemLimit - 1024 - kControlBytes - (5 * Pieces<16, F16>::kQ + 1) * 16 * 128 -
     Pieces<16, F16>::kWeights) / kChunk;
static_assert(kFewestSlots<false> >= 6 && kFewestSlots<true> >= 6, "a tile does not fit");
static_assert((DHS_ATTEND_MAX_KEY + 127) / 128 == 5 && 2 * DHS_PACKED_MAX_WIDE <= 128, "slots of a tile");

PackedPlan make_plan(const AttendCommon& c, const PackedLayout& l, int n) {
  switch (n) {
    case 16: return l.f16 ? plan_n<16, true>(c, l) : plan_n<16, false>(c, l);
    case 32: return l.f16 ? plan_n<32, true>(c, l) : plan_n<32, false>(c, l);
    case 48: return l.f16 ? plan_n<48, true>(c, l) : plan_n<48, false>(c, l);
    default: return l.f16 ? plan_n<64, true>(c, l) : plan_n<64, false>(c, l);
  }
}

// The widest block of columns whose queries leave the slots that it wants, or 16.
int widest_block(const AttendCommon& c, const PackedLayout& l) {
  int n = 64;
  while (n > 16 && !plan_fits(make_plan(c, l, n))) n -= 16;
  return n;
}

// Lets a kernel's blocks use all of an SM's shared memory: once on each device,
// with its first launch there.
template <int N, bool F16, int MAXI>
cudaError_t use_all_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(attend_packed_kernel<N, F16, MAXI>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int N, bool F16, int MAXI>
cudaError_t launch_kernel(const Params<MAXI>& P, const Shape& s, float* parts, cudaStream_t stream) {
  cudaError_t e = use_all_smem<N, F16, MAXI>();
  if (e != cudaSuccess) return e;
  attend_packed_kernel<N, F16><<<s.blocks, Pieces<N, F16>::kThreads, P.plan.smem, stream>>>(P, parts);
  e = cudaGetLastError();
  if (e != cudaSuccess || !s.n_cut) return e;
  return launch_merge(P.c, s, parts, stream);
}

template <int N, int MAXI>
cudaError_t launch_n(const Params<MAXI>& P, const Shape& s, float* parts, cudaStream_t stream) {
  return P.c.f16 ? launch_kernel<N, true, MAXI>(P, s, parts, stream)
                 : launch_kernel<N, false, MAXI>(P, s, parts, stream);
}

template <int MAXI>
cudaError_t launch_t(const AttendCommon& c, const PackedLayout& l, const AttendItem* items,
                     int n_items, const Shape& s, float* parts, cudaStream_t stream) {
  Params<MAXI> P;
  P.c = c;
  P.plan = make_plan(c, l, s.n);
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

bool attend_packed_shape(AttendCommon c, const PackedLayout& l, AttendItem* items, int n_items,
                         int sms, size_t* bytes) {
  const Shape s = shape_of(c, items, n_items, sms, widest_block(c, l));
  *bytes = parts_bytes(c, s);
  return s.tiles <= INT32_MAX;
}

cudaError_t launch_attend_packed(AttendCommon c, const PackedLayout& l, AttendItem* items,
                                 int n_items, int sms, void* work, cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kAttendItemsLarge) return cudaErrorInvalidValue;
  const Shape s = shape_of(c, items, n_items, sms, widest_block(c, l));
  if (s.tiles > INT32_MAX) return cudaErrorInvalidValue;
  float* parts = static_cast<float*>(work);
  return n_items <= kAttendItemsSmall
             ? launch_t<kAttendItemsSmall>(c, l, items, n_items, s, parts, stream)
             : launch_t<kAttendItemsLarge>(c, l, items, n_items, s, parts, stream);
}

}  // namespace dhs
