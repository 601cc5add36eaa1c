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
//     first, a piece is the upper byte of the number plus half a unit, and what
//     is left is exact in f16: 3 pieces hold 9 bits (an error of 2^-9 of a
//     weight and f16's 2^-11: less than bf16's 2^-8), 4 hold all of f16's 11.
//     m follows the maximum of s_j + v_j: weights reach 2^11..2^15, and those
//     down to 2^-17 are held, 2^-28 to 2^-32 of the largest.  (e4m3 would hold
//     2^-18 at best: half a million rows that share the weight of one that
//     stands out would be lost.)
// l sums the weights unrounded, without 2^v_j, which is divided out exactly.
//
// The rest is the 16-bit attention's (attend.cu): roles, tiles of 128 rows, the
// dealing of jobs and the joining of parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "attend_core.cuh"

namespace dhs {
namespace {

constexpr int kChunk = kTile * 128;  // bytes of a ring slot: 128 bytes of each row
constexpr int kMaxSlots = 12;
constexpr float kSlack = 4.f;        // log2 units that a weight may pass the reference by
constexpr float kLift = 11.f;        // log2 of a weight at the reference
constexpr int kTmemColumns = 512;

// How a launch's rows are staged.
struct PackedPlan {
  int32_t shared;        // the value is the key's beginning: loaded once
  int32_t key_chunks;    // of 128 codes
  int32_t units;         // value units of 128 codes: tiles of O^T's M side
  int32_t per_tile;      // ring slots of a tile: keys, wide elements, values unless shared
  int32_t slots;
  int32_t ahead;         // the next tile's scores are made beside this tile's weights
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
  static constexpr int kWeights = (kStack ? 1 : kP) * kTileBytes;
  static constexpr uint32_t kSwizzle = kRow == 32 ? 6 : kRow == 64 ? 4 : 2;
};

// ------------------------------------------------------------------ PTX

// D += A B (D = A B unless add) of 8-bit operands.
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

struct Control {
  static constexpr int kRowSlots = 4;  // tiles whose row addresses are found ahead
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t qfull[2], qempty, sfull[2], pfull, odone, oempty, rfull[kRowSlots], rempty[kRowSlots], drain;
  uint64_t segfull[kSegments], segempty[kSegments];
  Segment seg[kSegments];  // from the finding warp to the others
  const uint8_t* row[kRowSlots][kTile];
  int64_t out_off[64];
  int32_t lse_at[64];
  int32_t col_lo[64], col_hi[64];
  alignas(16) float m[64], base[64], fac[64];
  // What a column's coded scores are multiplied by.  Two tables in turn: queries
  // are loaded up to a segment ahead (never two: the products of a segment wait
  // for the weights of the one before).
  alignas(16) float qk[2][64];
  float part[4][64];
  uint32_t odd[4];    // rows of the tile whose products are taken by hand
  const uint8_t* odd_row;
  uint32_t o_begun;   // the segment's sums hold such products before the first tile's
  uint32_t tmem;
  volatile uint32_t gave_up;
};
constexpr int kBarQfull = 2 * kMaxSlots, kBarPfull = kBarQfull + 5, kBarOempty = kBarQfull + 7,
              kBarRfull = kBarQfull + 8, kBarRempty = kBarRfull + Control::kRowSlots,
              kBarDrain = kBarRempty + Control::kRowSlots, kBarSegempty = kBarDrain + 1 + kSegments,
              kBarriers = kBarSegempty + kSegments;
constexpr uint32_t kControlBytes = (sizeof(Control) + 1023) / 1024 * 1024;

// A ring position `k` slots further on.
__device__ __forceinline__ Ring further(Ring r, int k, int n) {
  r.slot += k;
  while (r.slot >= n) {
    r.slot -= n;
    r.phase ^= 1;
  }
  return r;
}

// Sixteen or eight 16-bit elements at `p`, zeros if !on.
__device__ __forceinline__ uint4 eight(const uint8_t* p, bool on, bool aligned) {
  if (!on) return make_uint4(0, 0, 0, 0);
  if (aligned) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
  return make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16,
                    s[4] | (uint32_t)s[5] << 16, s[6] | (uint32_t)s[7] << 16);
}

// Loading warps: queries once per segment, rows tile by tile.
template <int N, bool F16, int MAXI>
__device__ void load_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid) {
  using S = Pieces<N, F16>;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const PackedPlan& pl = P.plan;
  const uint32_t base = smem_u32(sm);
  Ring ring, rr, seg;
  uint32_t n_queries = 0;
  const int piece = tid & 7, r0 = tid >> 3;  // rows r0 + 16 i
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    if (__any_sync(~0u, ctl.gave_up) || !s.cols) break;
    const int32_t v0 = s.v0, v1 = s.v1;
    const AttendItem& it = s.it;
    // Queries: coded part [chunk][piece][column][128 B], wide part [column][128
    // B], zeros past the elements and the columns.  Eight threads have a column.
    auto load_queries = [&] {
      if (n_queries) warp_wait(smem_u32(&ctl.qempty), (n_queries - 1) & 1, until);
      const bool aligned = !(((uintptr_t)it.q | c.q_qs | c.q_hs) & 15);
      float* const qk = ctl.qk[n_queries & 1];
#pragma unroll 1
      for (int col = r0; col < N; col += kLoadThreads / 8) {
        const bool on = col < s.cols;
        const int qc = s.col0 + min(col, s.cols - 1);
        const int qi = it.loc ? s.qbase : qc / c.group;
        const int h = s.g * c.group + (it.loc ? qc : qc % c.group);
        const uint8_t* src = it.q + qi * c.q_qs + h * c.q_hs;
        constexpr int kChunks = 5;
        uint4 w[kChunks][2];
        uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int el = ch * 128 + piece * 16 + z * 8;
            w[ch][z] = eight(src + 2 * el, on && el < pl.key8, aligned);
            for (const uint32_t u : {w[ch][z].x, w[ch][z].y, w[ch][z].z, w[ch][z].w})
              top = max(top, max(u & 0x7FFFu, u >> 16 & 0x7FFFu));
          }
        const uint4 wide = eight(src + 2 * (pl.key8 + piece * 8), on && piece * 8 < pl.wide, aligned);
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) top = max(top, __shfl_xor_sync(~0u, top, x));
        // 2^e: the least that brings the largest to 448 = 0.875 * 2^9
        const bool finite = top < (F16 ? 0x7C00u : 0x7F80u);
        const float most = F16 ? __half2float(__ushort_as_half((unsigned short)top))
                               : __uint_as_float(top << 16);
        const uint32_t bits = __float_as_uint(most);
        int e = (int)(bits >> 23) - 126 - ((bits & 0x7FFFFFu) <= 0x600000u ? 9 : 8);
        e = most == 0.f ? 0 : min(max(e, -110), 120);
        const float down = __int_as_float((127 - e) << 23);
        if (piece == 0) qk[col] = __int_as_float((127 + e) << 23) * (c.scale * 1.44269504088896341f);
        uint8_t* const to = sm + pl.off_q + col * 128 + ((piece ^ (col & 7)) << 4);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          if (ch >= pl.key_chunks) continue;
          const uint32_t in[8] = {w[ch][0].x, w[ch][0].y, w[ch][0].z, w[ch][0].w,
                                  w[ch][1].x, w[ch][1].y, w[ch][1].z, w[ch][1].w};
          uint32_t out[S::kQ][4];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float2 f;
            if (F16) f = __half22float2(*reinterpret_cast<const __half2*>(&in[k]));
            else f = make_float2(__uint_as_float(in[k] << 16), __uint_as_float(in[k] & 0xFFFF0000u));
            f.x = finite ? f.x * down : NAN;
            f.y = finite ? f.y * down : NAN;
#pragma unroll
            for (int p = 0; p < S::kQ; ++p) {
              const uint32_t z = codes2(f.x, f.y);
              const float2 y = numbers2(z);
              f.x -= y.x;
              f.y -= y.y;
              if (k & 1) out[p][k >> 1] |= z << 16;
              else out[p][k >> 1] = z;
            }
          }
#pragma unroll
          for (int p = 0; p < S::kQ; ++p)
            *reinterpret_cast<uint4*>(to + (ch * S::kQ + p) * (N * 128)) =
                make_uint4(out[p][0], out[p][1], out[p][2], out[p][3]);
        }
        if (pl.wide)
          *reinterpret_cast<uint4*>(sm + pl.off_qw + col * 128 + ((piece ^ (col & 7)) << 4)) = wide;
      }
      fence_async();
      bar_arrive(smem_u32(&ctl.qfull[n_queries & 1]));
      ++n_queries;
    };

    const int nk = pl.key_chunks, nw = pl.wide ? 1 : 0;
    const uint32_t key_at = s.g * pl.key8, wide_at = pl.off_wide + s.g * pl.wide * 2;
    const uint32_t val_at = pl.off_value + s.g * c.dv;
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile) {
      warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
      const uint8_t* row[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = ctl.row[rr.slot][r0 + 16 * i];
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
      rr.next(Control::kRowSlots);
#pragma unroll 1
      for (int i = 0; i < pl.per_tile; ++i) {
        // loaded behind the rows that need no slot of this tile's own
        if (tile == v0 && i == pl.slots) load_queries();
        uint32_t at, n;  // the slice of the row that this slot takes
        if (i < nk) at = key_at + i * 128, n = pl.key8 - i * 128;
        else if (i < nk + nw) at = wide_at, n = 2 * pl.wide;
        else at = val_at + (i - nk - nw) * 128, n = c.dv - (i - nk - nw) * 128;
        warp_wait(smem_u32(&ctl.empty[ring.slot]), ring.phase ^ 1, until);
        const uint32_t dst = base + pl.off_rows + ring.slot * kChunk;
        const bool in = (uint32_t)piece * 16 < n;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + 16 * k;
          const bool on = row[k] && in;
          const uint8_t* src = on ? row[k] + at + 16 * piece : c.tail;
          asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                           dst + r * 128 + ((piece ^ (r & 7)) << 4)),
                       "l"(src), "r"(on ? 16 : 0)
                       : "memory");
        }
        // The slot's barrier gets this thread's arrival when its copies so far
        // have landed; the issuing warp makes them visible to the tensor cores.
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&ctl.full[ring.slot]))
                     : "memory");
        ring.next(pl.slots);
      }
      if (tile == v0 && pl.per_tile <= pl.slots) load_queries();
    }
    __syncwarp();
    if ((tid & 31) == 0) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Issuing warp: all its lanes walk the same path, one of them issues.
template <int N, bool F16, int MAXI>
__device__ void issue_products(const Params<MAXI>& P, uint8_t* sm, Control& ctl) {
  using S = Pieces<N, F16>;
  const Patience until{&ctl.gave_up, P.c.polls};
  const PackedPlan& pl = P.plan;
  const uint32_t base = smem_u32(sm);
  const uint32_t tm_s = ctl.tmem, tm_o = ctl.tmem + pl.sum_column;
  // float accumulators, operand types (8 bits: 0 e4m3, 1 e5m2; 16 bits: 0 f16,
  // 1 bf16), N, M = 128; the weights' product takes both operands M/N-major
  constexpr uint32_t common = 1u << 4 | 8u << 24;
  constexpr uint32_t id_key = common | (uint32_t)(S::kQ * N >> 3) << 17;
  constexpr uint32_t type = F16 ? 0u : 1u;
  constexpr uint32_t id_wide = common | type << 7 | type << 10 | (uint32_t)(N >> 3) << 17;
  constexpr uint32_t id_sum = common | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(S::kSum >> 3) << 17;
  constexpr uint32_t hi = operand_hi(1024, 2), hi_p = operand_hi(8 * S::kRow, S::kSwizzle);
  const uint32_t q_lo = operand_lo(base + pl.off_q, 16), qw_lo = operand_lo(base + pl.off_qw, 16);
  const uint32_t p_lo = operand_lo(base + pl.off_p, 16);
  const uint32_t rows_lo = operand_lo(base + pl.off_rows, 16);
  const bool lead = elected();
  const int nk = pl.key_chunks, nw = pl.wide ? 1 : 0, held = pl.shared ? pl.units : 0;
  Ring qr, seg;  // first slot of the tile whose scores are next
  uint32_t n_queries = 0, pphase = 0, ophase = 0, n_scores = 0;
  bool first = true;
#pragma unroll 1
  for (;;) {
    warp_wait(smem_u32(&ctl.segfull[seg.slot]), seg.phase, until);
    const Segment& s = ctl.seg[seg.slot];
    const int32_t v0 = s.v0, v1 = s.v1, cols = s.cols;
    if (__any_sync(~0u, ctl.gave_up) || !cols) break;
    if (lead) bar_arrive(smem_u32(&ctl.segempty[seg.slot]));
    seg.next(kSegments);
    if (v0 >= v1) continue;
    warp_wait(smem_u32(&ctl.qfull[n_queries & 1]), n_queries >> 1 & 1, until);
    fence_async();
    ++n_queries;
    int next = v0;   // the tile whose scores are next
    Ring vr = qr;    // first slot of the tile whose sums are next
#pragma unroll 1
    for (int tile = v0; tile < v1; ++tile) {
      const int last = pl.ahead ? min(tile + 1, v1 - 1) : tile;
#pragma unroll 1
      for (; next <= last; ++next) {
        const uint32_t buf = pl.ahead ? n_scores & 1 : 0, d = tm_s + buf * pl.buf_columns;
        Ring at = qr;
#pragma unroll 1
        for (int i = 0; i < nk + nw; ++i) {
          warp_wait(smem_u32(&ctl.full[at.slot]), at.phase, until);
          fence_async();
          tc_after();
          if (lead) {
            const uint32_t a = rows_lo + at.slot * (kChunk >> 4);
            if (i < nk) {
              const uint32_t b = q_lo + i * (S::kQ * N * 128 >> 4);
              const int steps = min(4, (pl.key8 - i * 128 + 31) / 32);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < steps) mma8(d, a + 2 * k, hi, b + 2 * k, hi, id_key, i > 0 || k > 0);
            } else {
              const int steps = (pl.wide + 15) / 16;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < steps) mma(d + S::kQ * N, a + 2 * k, hi, qw_lo + 2 * k, hi, id_wide, k > 0);
            }
            if (i >= held) commit(smem_u32(&ctl.empty[at.slot]));
          }
          at.next(pl.slots);
        }
        if (lead) {
          commit(smem_u32(&ctl.sfull[buf]));
          if (next + 1 == v1) commit(smem_u32(&ctl.qempty));
        }
        ++n_scores;
        qr = further(qr, pl.per_tile, pl.slots);
      }
      warp_wait(smem_u32(&ctl.pfull), pphase, until);
      pphase ^= 1;
      if (tile == v0 && !first) {  // the previous segment's sums are read
        warp_wait(smem_u32(&ctl.oempty), ophase, until);
        ophase ^= 1;
      }
      tc_after();
      const bool begun = tile > v0 || *(volatile uint32_t*)&ctl.o_begun;
      Ring at = pl.shared ? vr : further(vr, nk + nw, pl.slots);
#pragma unroll 1
      for (int u = 0; u < pl.units; ++u) {
        if (!pl.shared) {
          warp_wait(smem_u32(&ctl.full[at.slot]), at.phase, until);
          fence_async();
          tc_after();
        }
        if (lead) {
          const uint32_t a = rows_lo + at.slot * (kChunk >> 4), d = tm_o + u * S::kSum;
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
#pragma unroll
            for (int p = 0; p < (S::kStack ? 1 : S::kP); ++p)
              mma8(d, a + k * (4096 >> 4), hi,
                   p_lo + (p * S::kTileBytes + k * 32 * S::kRow >> 4), hi_p, id_sum,
                   begun || k > 0 || p > 0);
          commit(smem_u32(&ctl.empty[at.slot]));
        }
        at.next(pl.slots);
      }
      if (lead && (pl.ahead || tile + 1 == v1)) commit(smem_u32(&ctl.odone));
      vr = further(vr, pl.per_tile, pl.slots);
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
  float key;      // 2^k, 0 without a row
  float value;    // v
  float inverse;  // 2^-v, 0 without a row
};

// A row's scores of eight columns in log2 units, value scale included.
template <int N, bool F16>
__device__ __forceinline__ void scores8(uint32_t tm, const float* qk, float wide, bool has_wide,
                                        const RowScale& z, bool row, float (&x)[8]) {
  using S = Pieces<N, F16>;
  float v[S::kQ + 1][8];
  __syncwarp();
#pragma unroll
  for (int p = 0; p < S::kQ; ++p) tm_load8(tm + p * N, v[p]);
  if (has_wide) tm_load8(tm + S::kQ * N, v[S::kQ]);
#pragma unroll
  for (int p = 0; p < S::kQ + 1; ++p) tm_wait(v[p]);
  const float4 q0 = *reinterpret_cast<const float4*>(qk), q1 = *reinterpret_cast<const float4*>(qk + 4);
  const float q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float y = v[0][k];
#pragma unroll
    for (int p = 1; p < S::kQ; ++p) y += v[p][k];
    y = fmaf(y * z.key, q[k], z.value);
    if (has_wide) y = fmaf(v[S::kQ][k], wide, y);
    x[k] = row ? y : -INFINITY;
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
  constexpr int C = N / 2;
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
        scores8<N, F16>(tm_scores + k, qk + k0 + k, wide, pl.wide > 0, z, true, v);
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

// Softmax warps: a thread has one row of the tile and half of the columns;
// then the segment's output.
template <int N, bool F16, int MAXI>
__device__ void softmax_rows(const Params<MAXI>& P, uint8_t* sm, Control& ctl, int tid, float* parts) {
  using S = Pieces<N, F16>;
  constexpr int C = N / 2;
  const AttendCommon& c = P.c;
  const Patience until{&ctl.gave_up, c.polls};
  const PackedPlan& pl = P.plan;
  const int lane = tid & 31, r = tid & (kTile - 1), quarter = r >> 5, k0 = tid / kTile * C;
  const uint32_t tm_s = ctl.tmem + ((uint32_t)(r & ~31) << 16) + k0, tm_o = tm_s + pl.sum_column;
  const float wide = c.scale * 1.44269504088896341f;  // log2 e
  uint8_t* const weights = sm + pl.off_p + r * S::kRow;
  const bool quads_ok = !(((uintptr_t)c.o_qs | c.o_hs) & 7);  // outputs store four elements at once
  const int turn = S::kRow == 32 ? (r >> 2) & 1 : S::kRow == 64 ? (r >> 1) & 3 : r & 7;
  const int nk = pl.key_chunks, nw = pl.wide ? 1 : 0;
  Ring rr, tr, seg;  // row slots, first ring slot of the tile, segments
  uint32_t n_scores = 0, ophase = 0, n_queries = 0;
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto sum = [](float a, float b) { return a + b; };
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
    const bool some = s.v0 < s.v1;
    const float* const qk = ctl.qk[n_queries & 1];
    const uint32_t scale_at = pl.off_scale + 4 * s.g;
    // The next tile's row and scales, asked for a tile ahead.
    const uint8_t* row = nullptr;
    float ks = 0.f, vs = 1.f;
    auto find = [&](const uint8_t*& p, float& a, float& b) {
      warp_wait(smem_u32(&ctl.rfull[rr.slot]), rr.phase, until);
      p = ctl.row[rr.slot][r];
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.rempty[rr.slot]));
      rr.next(Control::kRowSlots);
      a = p ? __ldg(reinterpret_cast<const float*>(p + scale_at)) : 0.f;
      b = p ? __ldg(reinterpret_cast<const float*>(p + scale_at) + pl.value_scales) : 1.f;
    };
    if (some) {
      find(row, ks, vs);
      warp_wait(smem_u32(&ctl.qfull[n_queries & 1]), n_queries >> 1 & 1, until);
      ++n_queries;
    }

#pragma unroll 1
    for (int tile = s.v0; tile < s.v1; ++tile) {
      const int32_t j = tile * kTile + r;
      const bool ragged = tile * kTile < all_lo || tile * kTile + kTile > all_hi;
      const uint32_t buf = pl.ahead ? n_scores & 1 : 0, tm = tm_s + buf * pl.buf_columns;
      const uint8_t* next_row = nullptr;
      float next_ks = 0.f, next_vs = 1.f;
      if (tile + 1 < s.v1) find(next_row, next_ks, next_vs);
      const uint32_t vbits = __float_as_uint(vs) >> 23 & 255;
      const RowScale z{ks, (float)((int)vbits - 127),
                       row ? __uint_as_float(max(1u, min(253u, 254u - vbits)) << 23) : 0.f};
      warp_wait(smem_u32(&ctl.sfull[buf]), (pl.ahead ? n_scores >> 1 : n_scores) & 1, until);
      ++n_scores;
      tc_after();
      // The products of the tile before: complete, unless these scores were
      // made beside its weights.
      bool pending = pl.ahead && tile > s.v0;
      auto settle = [&] {
        if (!pending) return;
        warp_wait(smem_u32(&ctl.odone), ophase, until);
        ophase ^= 1;
        tc_after();
        pending = false;
      };
      float x[C];  // scores and value scale in log2 units
#pragma unroll
      for (int k = 0; k < C; k += 8) {
        float y[8];
        scores8<N, F16>(tm + k, qk + k0 + k, wide, pl.wide > 0, z, row != nullptr, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k + i] = y[i];
      }
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
          ctl.fac[tid] = old == -INFINITY ? 0.f : exp2_fast(old - m);
          ctl.m[tid] = m;
          ctl.base[tid] = m == -INFINITY ? 0.f : m - kLift;
        }
        named_sync(1, kSoftThreads);
        if (tile > s.v0) {
#pragma unroll
          for (int k = 0; k < C; ++k) l[k] *= ctl.fac[k0 + k];
          settle();
#pragma unroll 1
          for (int u = 0; u < pl.units * (S::kSum / N); ++u)
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
      // if its value is not finite (0 x NaN): such rows leave the tile, and
      // their products are added by hand to the columns that see them.
      bool odd = false;
      if (ragged) {
        const uint8_t* value = row + (pl.shared ? s.g * pl.key8 : pl.off_value + s.g * c.dv);
        if (row && (j < all_lo || j >= all_hi)) odd = !finite_codes(value, c.dv);
        if (named_or(1, kSoftThreads, odd)) {
          settle();
          odd_rows<N, F16>(P, sm, ctl, tid, odd, value,
                           pl.shared ? tr : further(tr, nk + nw, pl.slots), tile * kTile,
                           tile == s.v0, tm, qk, z);
        }
      }
      tr = further(tr, pl.per_tile, pl.slots);
      // weights in pieces, in the swizzled layout
      settle();
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
          for (int n = 0; n < 2; ++n) {
            const float p0 = exp2_fast(x[k + i + 2 * n] - b[i + 2 * n]);
            const float p1 = exp2_fast(x[k + i + 2 * n + 1] - b[i + 2 * n + 1]);
            l[k + i + 2 * n] = fmaf(p0, z.inverse, l[k + i + 2 * n]);
            l[k + i + 2 * n + 1] = fmaf(p1, z.inverse, l[k + i + 2 * n + 1]);
            h[n] = __floats2half2_rn(p0, p1);
          }
#pragma unroll
          for (int p = 0; p < S::kP; ++p) {
            uint32_t u[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              // the upper byte of each number, rounded to nearest, and the rest
              u[n] = (*reinterpret_cast<uint32_t*>(&h[n]) + 0x00800080u) & 0xFF00FF00u;
              h[n] = __hsub2(h[n], *reinterpret_cast<__half2*>(&u[n]));
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
      fence_async();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&ctl.pfull));
      row = next_row;
      ks = next_ks;
      vs = next_vs;
    }

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
    if (some) {
      warp_wait(smem_u32(&ctl.odone), ophase, until);
      ophase ^= 1;
      tc_after();
    }
    const bool quads = quads_ok && !((uintptr_t)it.out & 7);
#pragma unroll 1
    for (int u = 0; u < pl.units; ++u) {
      // after the exchange lane i of four has column k + i of four elements
      const int d = u * 128 + quarter * 32 + (lane & ~3);
#pragma unroll
      for (int k = 0; k < C; k += 8) {
        float v[8] = {};
        if (some) {
          tm_load(tm_o + u * S::kSum + k, v);
#pragma unroll
          for (int p = 1; p < (S::kStack ? S::kP : 1); ++p) {
            float y[8];
            tm_load(tm_o + u * S::kSum + p * N + k, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += y[i];
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
__global__ void __launch_bounds__(kThreads, 1)
    attend_packed_kernel(const __grid_constant__ Params<MAXI> P, float* parts) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  Control& ctl = *reinterpret_cast<Control*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  for (int k = tid; k < Control::kRowSlots * kTile; k += kThreads) (&ctl.row[0][0])[k] = nullptr;
  if (warp == kIssueWarp) {
#pragma unroll
    for (int k = 0; k < kBarriers; k += 32) {
      const int i = k + (tid & 31);
      const bool full = i < kMaxSlots || i == kBarQfull || i == kBarQfull + 1;
      const bool soft = i == kBarPfull || i == kBarOempty;
      const bool rows = i >= kBarRfull && i < kBarRempty;
      const bool read = i >= kBarRempty && i < kBarDrain;
      const bool segs = i >= kBarSegempty;
      if (i < kBarriers)
        bar_init(smem_u32(&ctl.full[0]) + 8 * i,
                 full ? kLoadThreads : soft ? kSoftThreads / 32 : rows ? kRowThreads / 32
                 : read ? (kSoftThreads + kLoadThreads) / 32 : segs ? kThreads / 32 - 1 : 1);
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
  if (warp == kFindWarp) {
    find_segments(P, ctl);  // meets the others' barrier inside
  } else {
    tc_before();
    __syncthreads();
    tc_after();
    if (warp < kSoftThreads / 32) softmax_rows<N, F16>(P, sm, ctl, tid, parts);
    else if (warp < kIssueWarp) load_rows<N, F16>(P, sm, ctl, tid - kSoftThreads);
    else if (warp == kIssueWarp) issue_products<N, F16>(P, sm, ctl);
    else find_rows(P, ctl, tid - 32 * kRowWarp);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kIssueWarp)
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
  p.off_rows = p.off_p + S::kWeights;
  const uint32_t room = kSmemLimit - 1024 > p.off_rows ? kSmemLimit - 1024 - p.off_rows : 0;
  p.slots = std::min<int>(kMaxSlots, room / kChunk);
  p.smem = 1024 + p.off_rows + (uint32_t)p.slots * kChunk;
  p.buf_columns = (S::kQ + nw) * N;
  const int sums = p.units * S::kSum;
  // The next tile's keys need slots of their own while this tile holds its
  // values: slots are taken in order, so that the ring has to reach from the
  // first value (shared rows: the first slot) of a tile to the next one's last key.
  p.ahead = 2 * p.buf_columns + sums <= kTmemColumns &&
            p.slots >= (l.shared ? 2 : 1) * p.per_tile;
  p.sum_column = (p.ahead ? 2 : 1) * p.buf_columns;
  return p;
}

// Slots without which a tile cannot be worked on: shared rows stay until their
// sums are made.
bool plan_fits(const PackedPlan& p) {
  return p.slots >= (p.shared ? p.per_tile : std::min(p.per_tile, 2));
}

PackedPlan make_plan(const AttendCommon& c, const PackedLayout& l, int n) {
  switch (n) {
    case 16: return l.f16 ? plan_n<16, true>(c, l) : plan_n<16, false>(c, l);
    case 32: return l.f16 ? plan_n<32, true>(c, l) : plan_n<32, false>(c, l);
    case 48: return l.f16 ? plan_n<48, true>(c, l) : plan_n<48, false>(c, l);
    default: return l.f16 ? plan_n<64, true>(c, l) : plan_n<64, false>(c, l);
  }
}

// The widest block of columns whose queries leave room for a tile.
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
  attend_packed_kernel<N, F16><<<s.blocks, kThreads, P.plan.smem, stream>>>(P, parts);
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
