// Rotary positions, and rows in 8 bits written and read back.
//
// Rotation.  Pair i of a head turns by an angle proportional to the position.
// The table holds each pair's turn a position as a 64-bit fraction of a whole
// turn, so that position * turns mod 2^64 is the angle, exactly, at any
// position: one integer product.  Its top 32 bits are reduced to an eighth of a
// turn around the nearest quarter before they become a float, which leaves the
// angle 2^-28 + 2^-32 turns off at most, under 2^-25 radians.  A block makes the sines of its tokens once, in
// shared memory, for all their heads.
//
// Packing.  A group of lanes has a head (16 elements a lane): its largest
// magnitude goes round by shuffles, the scale's exponent comes from that
// number's own exponent field, and the codes leave as 16-byte stores.  The
// elements are read once and turned in registers (half pairs read the partner's
// element too, which another lane of the group reads at the same time: an L1
// hit).  Sines and products aside, one rounding: to a code.
//
// Reading back.  Eight to 32 lanes have a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kItemsSmall = 16;  // items of a launch whose table is small
constexpr int kSinesMax = kRotaryMax / 2;  // sines and cosines a block holds: 16 KB

// ------------------------------------------------------------------ numbers

template <bool F16>
__device__ __forceinline__ float2 wide2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight 16-bit elements at `p`, 16-byte aligned or not.  CONST: of memory that the
// kernel does not write, which the read-only path is for.
template <bool CONST>
__device__ __forceinline__ uint4 raw8(const uint8_t* p, bool aligned) {
  if (CONST && aligned) return __ldg(reinterpret_cast<const uint4*>(p));
  if (aligned) return *reinterpret_cast<const uint4*>(p);
  const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
  return make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16,
                    s[4] | (uint32_t)s[5] << 16, s[6] | (uint32_t)s[7] << 16);
}

template <bool F16>
__device__ __forceinline__ void floats8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = wide2<F16>(u[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ void put8(uint8_t* p, bool aligned, const uint4& w) {
  if (aligned) {
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint16_t* s = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = (uint16_t)(u[k >> 1] >> (16 * (k & 1)));
  }
}

template <bool F16>
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(narrow2<F16>(v[0], v[1]), narrow2<F16>(v[2], v[3]), narrow2<F16>(v[4], v[5]),
                    narrow2<F16>(v[6], v[7]));
}

// n / d for n < 2^31, by one product: where a thread finds its place by division,
// that costs more than what it then does.
struct Div {
  uint32_t mul, shift, d;
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};
Div div_by(uint32_t d) {
  Div x{0, 0, d};
  while ((1u << x.shift) < d) ++x.shift;
  x.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << x.shift) - d)) / d + 1);
  return x;
}

__device__ __forceinline__ uint16_t codes2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two codes times their scale.
__device__ __forceinline__ float2 numbers2(uint16_t codes, float scale) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return make_float2(f.x * scale, f.y * scale);
}

// The smallest e in [-64, 120] with top <= 448 * 2^e (448 = 0.875 * 2^9).
__device__ __forceinline__ int exponent_of(float top) {
  const uint32_t b = __float_as_uint(top);
  const int x = (int)(b >> 23) - 126;  // top = m * 2^x, m in [0.5, 1)
  const int e = x - ((b & 0x7FFFFFu) <= 0x600000u ? 9 : 8);
  return top == 0.f ? -64 : min(max(e, -64), 120);
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// ------------------------------------------------------------------ rotation

// (cos, sin) of position * turns, times the amplitude.
__device__ __forceinline__ float2 sine_of(uint64_t turns, int32_t position, const Rotation& r) {
  const uint32_t t = (uint32_t)((uint64_t)(int64_t)position * turns >> 32);  // 2^-32 turns
  const uint32_t quarter = (t + (1u << 29)) >> 30;
  float s, c;
  sincospif((float)(int32_t)(t - (quarter << 30)) * 0x1p-31f, &s, &c);
  const float y = quarter & 1 ? c : s, x = quarter & 1 ? s : c;
  const float cosine = (quarter + 1) & 2 ? -x : x, sine = quarter & 2 ? -y : y;
  return make_float2(cosine * r.amplitude, sine * (r.amplitude * r.sign));
}

// Sines lie so that the threads of a warp, which have neighbouring groups of eight
// elements, read neighbouring 16 bytes: a group's (half pairs: of its lower half)
// pairs two by two, the first two of all groups, the next two, and so on.
struct SineTable {
  int half, groups, shift;  // pairs, groups of them, log2 of pairs in a group
  __device__ __forceinline__ SineTable(const Rotation& r) {
    half = r.rotary / 2;
    shift = r.interleaved ? 2 : 3;
    groups = half >> shift;
  }
  __device__ __forceinline__ int place(int pair) const {
    const int k = (pair >> 1) & ((1 << (shift - 1)) - 1);
    return 2 * (k * groups + (pair >> shift)) + (pair & 1);
  }
};

// Four pairs (a, b) next to each other; their sines begin at s.
__device__ __forceinline__ void turn_pairs(float (&v)[8], const float4* s, int groups) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 z = s[k * groups];
    const float a = v[4 * k], b = v[4 * k + 1], c = v[4 * k + 2], d = v[4 * k + 3];
    v[4 * k] = a * z.x - b * z.y;
    v[4 * k + 1] = b * z.x + a * z.y;
    v[4 * k + 2] = c * z.z - d * z.w;
    v[4 * k + 3] = d * z.z + c * z.w;
  }
}

// Eight elements whose partners are `u`: the lower ones of their pairs, or
// (sign -1) the upper ones.
__device__ __forceinline__ void turn_half(float (&v)[8], const float (&u)[8], float sign,
                                          const float4* s, int groups) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 z = s[k * groups];
    v[2 * k] = v[2 * k] * z.x - sign * u[2 * k] * z.y;
    v[2 * k + 1] = v[2 * k + 1] * z.z - sign * u[2 * k + 1] * z.w;
  }
}

struct RotateGrid {
  Div groups, heads, half;
  int32_t tokens_each;
};

// Rotates or copies groups of eight elements; a thread that has the lower half
// of eight half pairs writes both halves.  Its first group is asked for ahead of
// the sines.  Bound by memory once it runs: 8192 tokens of 32 heads of 128, 134 MB
// in 25 us, 5.5 TB/s (37 with the sines in pairs' order, where a warp's reads met in
// the same banks); 512 tokens of 16 heads of 576 6.2 us, most of it a launch, the
// sines and one trip to memory.
template <bool F16>
__global__ void __launch_bounds__(kThreads)
    rotate_kernel(const __grid_constant__ RotateParams P, const __grid_constant__ RotateGrid G) {
  __shared__ alignas(16) float2 sines[kSinesMax];
  const Rotation& r = P.r;
  const SineTable table(r);
  const int half = table.half;
  const int64_t t0 = (int64_t)blockIdx.x * G.tokens_each;
  const int n = (int)min((int64_t)G.tokens_each, P.tokens - t0);
  const bool aligned_x = !(((uintptr_t)P.x | P.x_ts | P.x_hs) & 15);
  const bool aligned_y = !(((uintptr_t)P.y | P.y_ts | P.y_hs) & 15);
  const uint8_t* const x0 = P.x + t0 * P.x_ts;
  uint8_t* const y0 = P.y + t0 * P.y_ts;
  // of a head: groups that turn (half pairs: two groups each), then the rest
  const int turning = (r.interleaved ? r.rotary : half) / 8;
  const int all = n * P.heads * (int)G.groups.d;
  uint4 a, b;
  int t, g, h;
  auto element = [&] {
    if (g < turning) return r.offset + g * 8;
    const int el = (g - turning) * 8;
    return el >= r.offset ? el + r.rotary : el;
  };
  auto ask = [&](int k) {
    const int th = G.groups.of(k);
    t = G.heads.of(th);
    h = th - t * P.heads;
    g = k - th * (int)G.groups.d;
    const uint8_t* x = x0 + t * P.x_ts + h * P.x_hs + 2 * element();
    a = raw8<false>(x, aligned_x);  // y may be the same memory
    if (!r.interleaved && g < turning) b = raw8<false>(x + 2 * half, aligned_x);
  };
  if ((int)threadIdx.x < all) ask(threadIdx.x);
  for (int k = threadIdx.x; k < n * half; k += kThreads) {
    const int i = G.half.of(k);
    sines[i * half + table.place(k - i * half)] =
        sine_of(__ldg(r.turns + (k - i * half)), __ldg(P.position + t0 + i), r);
  }
  __syncthreads();
#pragma unroll 1
  for (int k = threadIdx.x; k < all; k += kThreads) {
    if (k >= kThreads) ask(k);
    uint8_t* to = y0 + t * P.y_ts + h * P.y_hs + 2 * element();
    if (g < turning) {
      const float4* s = reinterpret_cast<const float4*>(sines + t * half) + g;
      float v[8];
      floats8<F16>(a, v);
      if (r.interleaved) {
        turn_pairs(v, s, table.groups);
      } else {
        float w[8];
        floats8<F16>(b, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 z = s[i * table.groups];
          const float v0 = v[2 * i], v1 = v[2 * i + 1], w0 = w[2 * i], w1 = w[2 * i + 1];
          v[2 * i] = v0 * z.x - w0 * z.y;
          v[2 * i + 1] = v1 * z.z - w1 * z.w;
          w[2 * i] = w0 * z.x + v0 * z.y;
          w[2 * i + 1] = w1 * z.z + v1 * z.w;
        }
        put8(to + 2 * half, aligned_y, narrow8<F16>(w));
      }
      a = narrow8<F16>(v);
    }
    put8(to, aligned_y, a);
  }
}

// ------------------------------------------------------------------ packing

template <int MAXI>
struct PackParams {
  PackCommon c;
  int32_t lanes;         // of a head of codes: a power of two
  int32_t key_passes, value_passes;  // of a warp over a token's heads; then the wide ones
  int32_t keys_each;     // passes over keys of a block; of the others it has one
  int32_t tokens_each;   // tokens of a block
  Div half, wide;
  int32_t first[MAXI];  // first block of each item, past the last one INT32_MAX
  PackItem items[MAXI];
};
static_assert(sizeof(PackParams<kPackItemsMax>) <= 32764, "pack item table too large");

// The last of the entries that is <= x; called by whole warps.
template <class T, int MAX>
__device__ __forceinline__ int item_of(const T (&first)[MAX], int n, T x) {
  int found = 0;
  for (int k = 0; k < n; k += 32) {
    const int i = k + (threadIdx.x & 31);
    found += __popc(__ballot_sync(~0u, i < n && first[i] <= x));
  }
  return found - 1;
}

// Where the bytes of one packed row go: the caller's row, or the tail ring and
// the host copy.
struct RowOut {
  uint8_t* a;
  uint8_t* b;
};

template <class T>
__device__ __forceinline__ void put(const RowOut& to, int at, T v) {
  *reinterpret_cast<T*>(to.a + at) = v;
  if (to.b) *reinterpret_cast<T*>(to.b + at) = v;
}

// A block has some tokens of an item and one pass over their heads: as many heads
// of keys, or of values, as the warp has groups of lanes for, or 256 wide
// elements.  So a thread's heads and elements are the same for all its tokens, and
// finding them costs it nothing per token.  Where there are blocks enough, one has
// all passes over its tokens' keys instead, and makes their sines once.  A token's
// elements are asked for a token ahead.  The conversions bound it: 67 MB in, 35 MB out
// in 30 us where a copy takes 15.  LONG: heads of more than 512 elements, 32 a lane.
template <bool F16, bool LONG, int MAXI>
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const __grid_constant__ PackParams<MAXI> P) {
  __shared__ alignas(16) float2 sines[kSinesMax];
  constexpr int Z = LONG ? 2 : 1;
  const PackCommon& c = P.c;
  const PackedLayout& l = c.l;
  const Rotation& r = c.r;
  const SineTable table(r);
  const int half = table.half, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = c.n_items > 1 ? item_of(P.first, c.n_items, (int32_t)blockIdx.x) : 0;
  const PackItem& it = P.items[item];
  const int t0 = (blockIdx.x - P.first[item]) * P.tokens_each, n = min(P.tokens_each, it.count - t0);
  // what this thread has of every token
  const int key_blocks = (P.key_passes + P.keys_each - 1) / P.keys_each;
  const bool wide = (int)blockIdx.y >= key_blocks + P.value_passes;
  const bool value = !wide && (int)blockIdx.y >= key_blocks;
  int pass = (int)blockIdx.y - (wide ? key_blocks + P.value_passes : value ? key_blocks : 0);
  int passes = 1;
  if (!wide && !value) {
    pass *= P.keys_each;
    passes = min(P.keys_each, P.key_passes - pass);
  }
  const int at = lane & (P.lanes - 1);
  int g = wide ? (int)P.wide.of(pass * 32 + lane) : pass * (32 / P.lanes) + lane / P.lanes;
  bool on = g < l.kv;
  const int elems = wide ? l.wide : value ? l.value : l.key8;
  const int el0 = wide ? (pass * 32 + lane - g * (int)P.wide.d) * 8 : at * 16;
  const uint8_t* const base = wide ? it.wide : value ? it.value : it.key;
  const int64_t ts = wide ? c.w_ts : value ? c.v_ts : c.k_ts, hs = wide ? c.w_hs : value ? c.v_hs : c.k_hs;
  const bool aligned = !(((uintptr_t)base | ts | hs) & 15);
  const int from = r.offset - (wide ? l.key8 : 0);  // the rotary range among these elements
  const bool turned = r.rotary && !value && from >= 0 && from < elems;
  const uint8_t* const x0 = base + (int64_t)(t0 + warp) * ts + 2 * el0;
  const uint8_t* x = x0 + (on ? g : 0) * hs;
  uint4 a[Z][2], b[Z][2];  // elements, and the partners of half pairs
  auto each = [&](auto f) {  // f(z, q, element) for the groups of eight of this thread
#pragma unroll
    for (int z = 0; z < Z; ++z)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = el0 + z * P.lanes * 16 + 8 * q;
        if (on && e < elems && !(wide && (z || q))) f(z, q, e);
      }
  };
  auto in_range = [&](int e) { return turned && e >= from && e < from + r.rotary; };
  auto ask = [&] {
    each([&](int z, int q, int e) {
      const uint8_t* p = x + 2 * (e - el0);
      a[z][q] = raw8<true>(p, aligned);
      if (!r.interleaved && in_range(e))
        b[z][q] = raw8<true>(p + (e - from < half ? 2 * half : -2 * half), aligned);
    });
    x += kWarps * ts;
  };
  if (warp < n) ask();
  if (turned) {  // for all threads of the block
    for (int k = threadIdx.x; k < n * half; k += kThreads) {
      const int i = P.half.of(k);
      sines[i * half + table.place(k - i * half)] =
          sine_of(__ldg(r.turns + (k - i * half)), __ldg(it.position + t0 + i), r);
    }
    __syncthreads();
  }
  int t = warp;
#pragma unroll 1
  for (;;) {
    if (t >= n) {  // the block's next heads
      if (!--passes || warp >= n) break;
      g += 32 / P.lanes;
      on = g < l.kv;
      x = x0 + (on ? g : 0) * hs;
      t = warp;
      ask();
    }
    const int now = t;
    t += kWarps;
    float v[Z][2][8];
    float top = 0.f;
    uint4 raw = a[0][0];
    each([&](int z, int q, int e) {
      floats8<F16>(a[z][q], v[z][q]);
      if (in_range(e)) {
        const int j = e - from;
        const float4* s = reinterpret_cast<const float4*>(sines + now * half);
        if (r.interleaved) {
          turn_pairs(v[z][q], s + j / 8, table.groups);
        } else {
          float u[8];
          floats8<F16>(b[z][q], u);
          turn_half(v[z][q], u, j < half ? 1.f : -1.f, s + (j < half ? j : j - half) / 8, table.groups);
        }
        if (wide) raw = narrow8<F16>(v[0][0]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[z][q][k]));
    });
    if (t < n) ask();
    RowOut to;
    if (it.rows) {
      to = {it.rows + (int64_t)(t0 + now) * l.row_bytes, nullptr};
    } else {
      const uint32_t row = (uint32_t)(it.L0 + t0 + now);
      to = {c.tail + ((size_t)it.pair * c.T + row % (uint32_t)c.T) * l.row_bytes,
            it.host ? it.host + (size_t)row * l.row_bytes : nullptr};
    }
    if (wide) {
      if (on) put(to, l.off_wide + 2 * (g * l.wide + el0), raw);
      continue;
    }
    // Infinities, which are rare, make NaN codes and leave the scale to the rest;
    // a NaN is passed over by the maximum and is a NaN code by itself.
    if (top == INFINITY) {
      top = 0.f;
      each([&](int z, int q, int) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (fabsf(v[z][q][k]) == INFINITY) v[z][q][k] = NAN;
          top = fmaxf(top, fabsf(v[z][q][k]));
        }
      });
    }
    __syncwarp();
#pragma unroll
    for (int w = 16; w; w >>= 1)
      if (w < P.lanes) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (!on) continue;
    const int e = exponent_of(top);
    const float inverse = power_of_two(-e);
    const int head = (value ? l.off_value : 0) + g * elems;
#pragma unroll
    for (int z = 0; z < Z; ++z) {
      const int el = el0 + z * P.lanes * 16;
      if (el >= elems) continue;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* f = &v[z][k >> 1][(k & 1) * 4];
        w[k] = codes2(f[0] * inverse, f[1] * inverse) |
               (uint32_t)codes2(f[2] * inverse, f[3] * inverse) << 16;
      }
      put(to, head + el, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (at == 0) {
      put(to, l.off_scale + 4 * (value ? l.kv + g : g), power_of_two(e));
      if (!value && g == 0)  // what is left of the last 16 bytes
        for (int k = l.off_scale + 4 * l.kv * (l.shared ? 1 : 2); k < l.row_bytes; k += 4) put(to, k, 0.f);
    }
  }
}

// ------------------------------------------------------------------ reading back

template <int MAXI>
struct UnpackParams {
  UnpackCommon c;
  int32_t coded, values, wides;  // pieces of a row, of 8 elements
  int32_t lanes, lanes_log;      // of a row
  Div key, value, wide;          // of a head
  int32_t first[MAXI];  // first block of each item, past the last one INT32_MAX
  UnpackItem items[MAXI];
};
static_assert(sizeof(UnpackParams<kUnpackItemsMax>) <= 32764, "unpack item table too large");

// Where entry j of an item lies: 0: zeros, 1: untouched.  `first`: the one thread
// that says so where a location is outside its arena.
__device__ __forceinline__ uintptr_t entry_of(const UnpackCommon& c, const UnpackItem& it, int64_t j,
                                              bool first) {
  const size_t rb = (size_t)c.l.row_bytes;
  if (it.rows) return (uintptr_t)(it.rows + j * rb);
  if (it.loc) {
    const uint32_t w = __ldg(it.loc + j);
    if (w == kNoLoc) return 0;
    if (w == kEndLoc) return 1;
    const uint32_t tier = w >> 30, x = w & 0x3FFFFFFFu;
    const uint32_t rows = tier == kTierTail ? c.tail_rows : tier == kTierOpt ? c.opt_rows
                          : tier == kTierHot ? c.hot_rows : 0;
    if (x >= rows) {
      if (first) atomicOr(c.status, kStatusEloc);
      return 0;
    }
    return (uintptr_t)((tier == kTierTail ? c.tail : tier == kTierOpt ? c.opt : c.hot) + x * rb);
  }
  const int64_t row = it.first + j;
  if (row >= it.L - c.T)  // (rows are numbered in 31 bits)
    return (uintptr_t)(c.tail + ((size_t)it.pair * c.T + (uint32_t)row % (uint32_t)c.T) * rb);
  const int64_t page = row >> c.page_shift;
  const int32_t slot = page < it.complete ? __ldg(c.map + (size_t)it.pair * c.Pmax + page) : -1;
  if (slot >= 0)
    return (uintptr_t)(c.opt + (((size_t)slot << c.page_shift) + (row & ((1 << c.page_shift) - 1))) * rb);
  return (uintptr_t)(it.host + row * rb);
}

// Eight lanes have a row (16 or 32 where each still has 16 elements or more), each
// eight of its elements at a time, so that their stores are whole lines; they ask
// for those of four turns at once.  What belongs to the row (its address, where
// its numbers go) is found once, for four rows of a warp together: the instructions
// bound it.  262,144 located rows of 656 bytes, whose 16-bit numbers are 4/5 of the
// bytes: 86 us, 4.1 TB/s (each lane finding row, item and head of each piece: 158; a
// warp's rows in turn 125; a row a warp 123).
template <bool F16, int MAXI>
__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const __grid_constant__ UnpackParams<MAXI> P) {
  const UnpackCommon& c = P.c;
  const PackedLayout& l = c.l;
  const int lanes = P.lanes, lane = threadIdx.x & (lanes - 1);
  const int item = c.n_items > 1 ? item_of(P.first, c.n_items, (int32_t)blockIdx.x) : 0;
  const UnpackItem& it = P.items[item];
  const int64_t j = ((int64_t)(blockIdx.x - P.first[item]) * kThreads + threadIdx.x) >> P.lanes_log;
  if (j >= it.count) return;
  const uintptr_t from = entry_of(c, it, j, lane == 0);
  if (from == 1) return;
  const uint8_t* const src = reinterpret_cast<const uint8_t*>(from);
  uint8_t* const key = it.key ? it.key + j * c.k_rs : nullptr;
  uint8_t* const value = it.value ? it.value + j * c.v_rs : nullptr;
  const float* const scales = reinterpret_cast<const float*>(src + l.off_scale);
  const bool plain = l.kv == 1, too = l.shared && value;
  const bool aligned = !(((uintptr_t)it.key | c.k_rs | c.k_hs | (uintptr_t)it.value | c.v_rs | c.v_hs) & 15);
  const float only = src && plain ? __ldg(scales) : 0.f;
  // key codes, then value codes, which follow them in the row
  const int q0 = key || too ? 0 : P.coded, q1 = P.coded + (value ? P.values : 0);
#pragma unroll 4
  for (int q = q0 + lane; q < q1; q += lanes) {
    const bool v = q >= P.coded;
    const int i = v ? q - P.coded : q;
    const int g = plain ? 0 : (int)(v ? P.value.of(i) : P.key.of(i));
    const int el = (i - g * (int)(v ? P.value.d : P.key.d)) * 8;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (src) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(src) + q);
      const float z = plain && !v ? only : __ldg(scales + (v ? l.kv + g : g));
      const float2 a = numbers2((uint16_t)w.x, z), b = numbers2((uint16_t)(w.x >> 16), z);
      const float2 d = numbers2((uint16_t)w.y, z), e = numbers2((uint16_t)(w.y >> 16), z);
      y = make_uint4(narrow2<F16>(a.x, a.y), narrow2<F16>(b.x, b.y), narrow2<F16>(d.x, d.y),
                     narrow2<F16>(e.x, e.y));
    }
    if (v) {
      put8(value + g * c.v_hs + 2 * el, aligned, y);
    } else {
      if (key) put8(key + g * c.k_hs + 2 * el, aligned, y);
      if (too && el < l.value) put8(value + g * c.v_hs + 2 * el, aligned, y);
    }
  }
  if (!key) return;
#pragma unroll 1
  for (int q = lane; q < P.wides; q += lanes) {
    const int g = plain ? 0 : (int)P.wide.of(q);
    const uint4 y = src ? __ldg(reinterpret_cast<const uint4*>(src + l.off_wide) + q) : make_uint4(0, 0, 0, 0);
    put8(key + g * c.k_hs + 2 * (l.key8 + (q - g * (int)P.wide.d) * 8), aligned, y);
  }
}

// Tokens of a block of which each has `units` of work: enough for its threads,
// no more than the sines hold or than leave every SM a block.
int tokens_of_block(int64_t tokens, int rotary, int units, int want, int sms) {
  int64_t n = std::max<int64_t>(1, want / std::max(1, units));
  if (rotary) n = std::min<int64_t>(n, kSinesMax / (rotary / 2));
  return (int)std::max<int64_t>(1, std::min<int64_t>(n, (tokens + sms - 1) / sms));
}

template <int MAXI>
cudaError_t launch_pack_t(const PackCommon& c, const PackItem* items, int n_items, int sms,
                          cudaStream_t stream) {
  PackParams<MAXI> P;
  P.c = c;
  P.c.n_items = n_items;
  const PackedLayout& l = c.l;
  const int longest = std::max(l.key8, l.shared ? 0 : l.value);
  P.lanes = 1;
  while (P.lanes < 32 && P.lanes * 16 < longest) P.lanes *= 2;
  const int heads = 32 / P.lanes;  // of a pass
  P.key_passes = (l.kv + heads - 1) / heads;
  P.value_passes = l.shared ? 0 : P.key_passes;
  const int wide_passes = (l.kv * (l.wide / 8) + 31) / 32;
  int64_t tokens = 0, blocks = 0;
  for (int i = 0; i < n_items; ++i) tokens += items[i].count;
  const int64_t passes = P.key_passes + P.value_passes + wide_passes;
  P.tokens_each = tokens_of_block(tokens * passes, c.r.rotary, 1, 4 * kWarps, sms);
  for (int i = 0; i < MAXI; ++i) {
    P.first[i] = i < n_items ? (int32_t)std::min<int64_t>(blocks, INT32_MAX) : INT32_MAX;
    if (i >= n_items) continue;
    P.items[i] = items[i];
    blocks += ((int64_t)items[i].count + P.tokens_each - 1) / P.tokens_each;
  }
  if (!blocks) return cudaSuccess;
  P.keys_each = blocks >= 2 * sms ? P.key_passes : 1;
  const int64_t rows = (P.key_passes + P.keys_each - 1) / P.keys_each + P.value_passes + wide_passes;
  if (blocks > INT32_MAX || rows > 65535) return cudaErrorInvalidValue;
  P.half = div_by(std::max(1, c.r.rotary / 2));
  P.wide = div_by(std::max(1, l.wide / 8));
  const bool wider = P.lanes * 16 < longest;
  auto kernel = l.f16
                    ? (wider ? pack_kernel<true, true, MAXI> : pack_kernel<true, false, MAXI>)
                    : (wider ? pack_kernel<false, true, MAXI> : pack_kernel<false, false, MAXI>);
  kernel<<<dim3((unsigned)blocks, (unsigned)rows), kThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

template <int MAXI>
cudaError_t launch_unpack_t(const UnpackCommon& c, const UnpackItem* items, int n_items,
                            cudaStream_t stream) {
  UnpackParams<MAXI> P;
  P.c = c;
  P.c.n_items = n_items;
  const PackedLayout& l = c.l;
  P.coded = l.kv * l.key8 / 8;
  P.values = l.shared ? 0 : l.kv * l.value / 8;
  P.wides = l.kv * l.wide / 8;
  P.lanes_log = 3;
  while (P.lanes_log < 5 && P.coded + P.values >= 16 << P.lanes_log) ++P.lanes_log;
  P.lanes = 1 << P.lanes_log;
  const int rows = kThreads / P.lanes;  // of a block
  int64_t blocks = 0;
  for (int i = 0; i < MAXI; ++i) {
    P.first[i] = i < n_items ? (int32_t)std::min<int64_t>(blocks, INT32_MAX) : INT32_MAX;
    if (i >= n_items) continue;
    P.items[i] = items[i];
    blocks += ((int64_t)items[i].count + rows - 1) / rows;
  }
  if (!blocks) return cudaSuccess;
  P.key = div_by(l.key8 / 8);
  P.value = div_by(l.value / 8);
  P.wide = div_by(std::max(1, l.wide / 8));
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (l.f16) unpack_kernel<true, MAXI><<<(int)blocks, kThreads, 0, stream>>>(P);
  else unpack_kernel<false, MAXI><<<(int)blocks, kThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int sms, cudaStream_t stream) {
  if (p.tokens <= 0 || p.heads <= 0) return cudaSuccess;
  const int groups = p.elems / 8;
  const int each = tokens_of_block(p.tokens, p.r.rotary, p.heads * groups, 4 * kThreads, sms);
  const int blocks = (int)(((int64_t)p.tokens + each - 1) / each);
  const int turning = (p.r.interleaved ? p.r.rotary : p.r.rotary / 2) / 8;
  const int rest = p.x == p.y ? 0 : (p.elems - p.r.rotary) / 8;  // in place: nothing is copied
  const RotateGrid g{div_by(turning + rest), div_by(p.heads), div_by(p.r.rotary / 2), each};
  if (p.f16) rotate_kernel<true><<<blocks, kThreads, 0, stream>>>(p, g);
  else rotate_kernel<false><<<blocks, kThreads, 0, stream>>>(p, g);
  return cudaGetLastError();
}

// A launch carries its table of items, 20 KB for 256; few items have a small one
// (8 items: 2.9 us of the host's time a call instead of 3.8).
cudaError_t launch_pack(const PackCommon& c, const PackItem* items, int n_items, int sms,
                        cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kPackItemsMax) return cudaErrorInvalidValue;
  return n_items <= kItemsSmall ? launch_pack_t<kItemsSmall>(c, items, n_items, sms, stream)
                                : launch_pack_t<kPackItemsMax>(c, items, n_items, sms, stream);
}

cudaError_t launch_unpack(const UnpackCommon& c, const UnpackItem* items, int n_items,
                          cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kUnpackItemsMax) return cudaErrorInvalidValue;
  return n_items <= kItemsSmall ? launch_unpack_t<kItemsSmall>(c, items, n_items, stream)
                                : launch_unpack_t<kUnpackItemsMax>(c, items, n_items, stream);
}

}  // namespace dhs
