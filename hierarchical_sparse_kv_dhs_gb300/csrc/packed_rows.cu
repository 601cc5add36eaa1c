// Rotary positions, and rows in 8 bits written and read back.
//
// Rotation.  Pair i of a head turns by an angle proportional to the position.
// The table holds each pair's turn a position as a 64-bit fraction of a whole
// turn, so that position * turns mod 2^64 is the angle, exactly, at any
// position: one integer product.  Its top 32 bits are reduced to an eighth of a
// turn around the nearest quarter before they become a float, which leaves the
// angle 2^-26 off at most.  A block makes the sines of its tokens once, in
// shared memory, for all their heads.
//
// Packing.  A group of lanes has a head (16 elements a lane): its largest
// magnitude goes round by shuffles, the scale's exponent comes from that
// number's own exponent field, and the codes leave as 16-byte stores.  The
// elements are read once and turned in registers (half pairs read the partner's
// element too, which another lane of the group reads at the same time: an L1
// hit).  Two roundings in all: to a code, and nothing else.
//
// Reading back.  A warp has four rows, whose addresses it finds at once; a lane
// takes 16 codes (or 8 wide elements) at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

// Eight 16-bit elements at `p`, 16-byte aligned or not.
template <bool F16>
__device__ __forceinline__ void load8(const uint8_t* p, bool aligned, float (&v)[8]) {
  uint4 w;
  if (aligned) {
    w = __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
    w.x = s[0] | (uint32_t)s[1] << 16;
    w.y = s[2] | (uint32_t)s[3] << 16;
    w.z = s[4] | (uint32_t)s[5] << 16;
    w.w = s[6] | (uint32_t)s[7] << 16;
  }
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = wide2<F16>(u[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}

template <bool F16>
__device__ __forceinline__ void store8(uint8_t* p, bool aligned, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = narrow2<F16>(v[2 * k], v[2 * k + 1]);
  if (aligned) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t* s = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
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

// The group of eight elements that begins at rotary element j, turned; `other`
// has the eight partners of half pairs.
__device__ __forceinline__ void turn8(float (&v)[8], const float (&other)[8], int j,
                                      const Rotation& r, const float2* sines) {
  if (r.interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 s = sines[j / 2 + k];
      const float a = v[2 * k], b = v[2 * k + 1];
      v[2 * k] = a * s.x - b * s.y;
      v[2 * k + 1] = b * s.x + a * s.y;
    }
  } else {
    const int half = r.rotary / 2;
    const bool up = j >= half;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 s = sines[(up ? j - half : j) + k];
      v[k] = up ? v[k] * s.x + other[k] * s.y : v[k] * s.x - other[k] * s.y;
    }
  }
}

// Rotates or copies groups of eight elements; a thread that has the lower half
// of eight half pairs writes both halves.  Bound by memory: what it reads and
// writes once.
template <bool F16>
__global__ void __launch_bounds__(kThreads)
    rotate_kernel(const __grid_constant__ RotateParams P, int tokens_each) {
  __shared__ float2 sines[kSinesMax];
  const Rotation& r = P.r;
  const int half = r.rotary / 2;
  const int64_t t0 = (int64_t)blockIdx.x * tokens_each;
  const int n = (int)min((int64_t)tokens_each, P.tokens - t0);
  for (int k = threadIdx.x; k < n * half; k += kThreads) {
    const int t = k / half;
    sines[k] = sine_of(__ldg(r.turns + (k - t * half)), __ldg(P.position + t0 + t), r);
  }
  __syncthreads();
  const bool in_place = P.x == P.y;
  const bool aligned_x = !(((uintptr_t)P.x | P.x_ts | P.x_hs) & 15);
  const bool aligned_y = !(((uintptr_t)P.y | P.y_ts | P.y_hs) & 15);
  // of a head: groups that turn (half pairs: two groups each), then the rest
  const int turning = (r.interleaved ? r.rotary : half) / 8;
  const int groups = turning + (in_place ? 0 : (P.elems - r.rotary) / 8);
  const int all = n * P.heads * groups;
#pragma unroll 2
  for (int k = threadIdx.x; k < all; k += kThreads) {
    const int th = k / groups, g = k - th * groups;
    const int t = th / P.heads, h = th - t * P.heads;
    const uint8_t* x = P.x + (t0 + t) * P.x_ts + h * P.x_hs;
    uint8_t* y = P.y + (t0 + t) * P.y_ts + h * P.y_hs;
    float v[8];
    if (g >= turning) {
      int el = (g - turning) * 8;
      if (el >= r.offset) el += r.rotary;
      if (aligned_x && aligned_y)
        *reinterpret_cast<uint4*>(y + 2 * el) = __ldg(reinterpret_cast<const uint4*>(x + 2 * el));
      else
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<uint16_t*>(y)[el + i] = reinterpret_cast<const uint16_t*>(x)[el + i];
      continue;
    }
    const int el = r.offset + g * 8;
    float u[8];
    load8<F16>(x + 2 * el, aligned_x, v);
    if (!r.interleaved) load8<F16>(x + 2 * (el + half), aligned_x, u);
    const float2* s = sines + t * half;
    if (!r.interleaved) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = s[g * 8 + i];
        w[i] = u[i] * z.x + v[i] * z.y;
        v[i] = v[i] * z.x - u[i] * z.y;
      }
      store8<F16>(y + 2 * (el + half), aligned_y, w);
    } else {
      turn8(v, v, g * 8, r, s);
    }
    store8<F16>(y + 2 * el, aligned_y, v);
  }
}

// ------------------------------------------------------------------ packing

struct PackParams {
  PackCommon c;
  int32_t lanes;         // of a head of codes: a power of two
  int32_t key_passes, value_passes, wide_passes;  // of a warp over a token's heads
  int32_t tokens_each;   // tokens of a block
  int64_t first[kPackItemsMax];  // first token of each item, past the last one INT64_MAX
  PackItem items[kPackItemsMax];
};
static_assert(sizeof(PackParams) <= 32764, "pack item table too large");

// The last of n entries that is <= x.
__device__ __forceinline__ int item_of(const int64_t* first, int n, int64_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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

template <bool F16>
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const __grid_constant__ PackParams P) {
  __shared__ float2 sines[kSinesMax];
  const PackCommon& c = P.c;
  const PackedLayout& l = c.l;
  const Rotation& r = c.r;
  const int half = r.rotary / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * P.tokens_each;
  const int n = (int)min((int64_t)P.tokens_each, c.tokens - t0);
  if (r.rotary) {
    for (int k = threadIdx.x; k < n * half; k += kThreads) {
      const int t = k / half;
      const int i = item_of(P.first, c.n_items, t0 + t);
      sines[k] = sine_of(__ldg(r.turns + (k - t * half)),
                         __ldg(P.items[i].position + (t0 + t - P.first[i])), r);
    }
    __syncthreads();
  }
  const int passes = P.key_passes + P.value_passes + P.wide_passes;
#pragma unroll 1
  for (int unit = warp; unit < n * passes; unit += kWarps) {
    const int t = unit / passes;
    int pass = unit - t * passes;
    const int i = item_of(P.first, c.n_items, t0 + t);
    const PackItem& it = P.items[i];
    const int64_t j = t0 + t - P.first[i];
    RowOut to;
    if (it.rows) {
      to = {it.rows + j * l.row_bytes, nullptr};
    } else {
      const int64_t row = it.L0 + j;
      to = {c.tail + ((size_t)it.pair * c.T + (size_t)(row % c.T)) * l.row_bytes,
            it.host ? it.host + row * l.row_bytes : nullptr};
    }
    const float2* s = sines + t * half;
    if (pass >= P.key_passes + P.value_passes) {  // wide elements, 8 a lane
      const int per = l.wide / 8, k = (pass - P.key_passes - P.value_passes) * 32 + lane;
      const int g = k / per, el = (k - g * per) * 8;
      if (g >= l.kv) continue;
      const uint8_t* x = it.wide + j * c.w_ts + g * c.w_hs;
      const bool aligned = !(((uintptr_t)it.wide | c.w_ts | c.w_hs) & 15);
      const int from = r.offset - l.key8;  // rotary range within the wide elements
      float v[8], u[8];
      load8<F16>(x + 2 * el, aligned, v);
      if (r.rotary && el >= from && el < from + r.rotary) {
        const int e = el - from;
        if (!r.interleaved) load8<F16>(x + 2 * (e < half ? el + half : el - half), aligned, u);
        turn8(v, u, e, r, s);
      }
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = narrow2<F16>(v[2 * q], v[2 * q + 1]);
      put(to, l.off_wide + 2 * (g * l.wide + el), make_uint4(w[0], w[1], w[2], w[3]));
      continue;
    }
    const bool value = pass >= P.key_passes;
    if (value) pass -= P.key_passes;
    const int elems = value ? l.value : l.key8;
    const int g = pass * (32 / P.lanes) + lane / P.lanes, at = lane % P.lanes;
    const bool on = g < l.kv;
    const uint8_t* base = value ? it.value : it.key;
    const int64_t ts = value ? c.v_ts : c.k_ts, hs = value ? c.v_hs : c.k_hs;
    const bool aligned = !(((uintptr_t)base | ts | hs) & 15);
    const uint8_t* x = base + j * ts + (on ? g : 0) * hs;
    // 16 elements a lane; heads of more than 512 have lanes with 16 more
    float v[2][2][8];
    float top = 0.f;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int el = (at + z * P.lanes) * 16;
      if (!on || el >= elems) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = el + 8 * q;
        load8<F16>(x + 2 * e, aligned, v[z][q]);
        if (!value && r.rotary && e >= r.offset && e < r.offset + r.rotary && r.offset < l.key8) {
          float u[8];
          const int k = e - r.offset;
          if (!r.interleaved) load8<F16>(x + 2 * (k < half ? e + half : e - half), aligned, u);
          turn8(v[z][q], u, k, r, s);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float m = fabsf(v[z][q][k]);
          if (m < INFINITY) top = fmaxf(top, m);
        }
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1)
      if (w < P.lanes) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (!on) continue;
    const int e = exponent_of(top);
    const float inverse = power_of_two(-e);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int el = (at + z * P.lanes) * 16;
      if (el >= elems) continue;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float a = v[z][k >> 1][(k & 1) * 4 + q];
          f[q] = fabsf(a) < INFINITY ? a * inverse : NAN;
        }
        w[k] = codes2(f[0], f[1]) | (uint32_t)codes2(f[2], f[3]) << 16;
      }
      put(to, (value ? l.off_value : 0) + g * elems + el, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (at == 0) {
      put(to, l.off_scale + 4 * (value ? l.kv + g : g), power_of_two(e));
      if (!value && g == 0)  // what is left of the last 16 bytes
        for (int b = l.off_scale + 4 * l.kv * (l.shared ? 1 : 2); b < l.row_bytes; b += 4)
          put(to, b, 0.f);
    }
  }
}

// ------------------------------------------------------------------ reading back

struct UnpackParams {
  UnpackCommon c;
  int32_t pieces;        // of a row: 16 codes or 8 wide elements each
  int64_t first[kUnpackItemsMax];
  UnpackItem items[kUnpackItemsMax];
};
static_assert(sizeof(UnpackParams) <= 32764, "unpack item table too large");

constexpr int kWarpRows = 4;

// Where entry j of an item lies: 0: zeros, 1: untouched.
__device__ __forceinline__ uintptr_t entry_of(const UnpackCommon& c, const UnpackItem& it, int64_t j) {
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
      atomicOr(c.status, kStatusEloc);
      return 0;
    }
    return (uintptr_t)((tier == kTierTail ? c.tail : tier == kTierOpt ? c.opt : c.hot) + x * rb);
  }
  const int64_t row = it.first + j;
  if (row >= it.L - c.T)
    return (uintptr_t)(c.tail + ((size_t)it.pair * c.T + (size_t)(row % c.T)) * rb);
  const int64_t page = row >> c.page_shift;
  const int32_t slot = page < it.complete ? __ldg(c.map + (size_t)it.pair * c.Pmax + page) : -1;
  if (slot >= 0)
    return (uintptr_t)(c.opt + (((size_t)slot << c.page_shift) + (row & ((1 << c.page_shift) - 1))) * rb);
  return (uintptr_t)(it.host + row * rb);
}

template <bool F16>
__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const __grid_constant__ UnpackParams P) {
  const UnpackCommon& c = P.c;
  const PackedLayout& l = c.l;
  const int lane = threadIdx.x & 31;
  const int64_t e0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kWarpRows;
  if (e0 >= c.count) return;
  // lane r finds the address of row r
  uintptr_t mine = 1;
  int item = 0;
  int64_t entry = 0;
  if (lane < kWarpRows && e0 + lane < c.count) {
    item = item_of(P.first, c.n_items, e0 + lane);
    entry = e0 + lane - P.first[item];
    mine = entry_of(c, P.items[item], entry);
  }
  const int coded = l.kv * l.key8 / 16, values = l.shared ? 0 : l.kv * l.value / 16;
#pragma unroll 2
  for (int k0 = 0; k0 < kWarpRows * P.pieces; k0 += 32) {
    const int k = k0 + lane, row = min(k / P.pieces, kWarpRows - 1), p = k - row * P.pieces;
    const uintptr_t from = __shfl_sync(~0u, (unsigned long long)mine, row);
    const int64_t j = __shfl_sync(~0u, (long long)entry, row);
    const UnpackItem& it = P.items[__shfl_sync(~0u, item, row)];
    if (from == 1 || p >= P.pieces) continue;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(from);
    uint8_t* key = it.key ? it.key + j * c.k_rs : nullptr;
    uint8_t* value = it.value ? it.value + j * c.v_rs : nullptr;
    if (p >= coded + values) {
      const int per = l.wide / 8, q = p - coded - values, g = q / per, el = (q - g * per) * 8;
      if (!key) continue;
      float v[8] = {};
      if (src) load8<F16>(src + l.off_wide + 16 * q, true, v);
      uint8_t* to = key + g * c.k_hs + 2 * (l.key8 + el);
      store8<F16>(to, !((uintptr_t)to & 15), v);
      continue;
    }
    const bool is_value = p >= coded;
    const int n = is_value ? l.value : l.key8, at = (is_value ? p - coded : p) * 16;
    const int g = at / n, el = at - g * n;
    float v[2][8] = {};
    if (src) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + (is_value ? l.off_value : 0) + at));
      const float scale = __ldg(reinterpret_cast<const float*>(src + l.off_scale) +
                                (is_value ? l.kv + g : g));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 f = numbers2((uint16_t)(u[q >> 1] >> (16 * (q & 1))), scale);
        v[q >> 2][2 * (q & 3)] = f.x;
        v[q >> 2][2 * (q & 3) + 1] = f.y;
      }
    }
    auto out = [&](uint8_t* to) {
      const bool aligned = !((uintptr_t)to & 15);
      store8<F16>(to, aligned, v[0]);
      store8<F16>(to + 16, aligned, v[1]);
    };
    if (is_value) {
      if (value) out(value + g * c.v_hs + 2 * el);
    } else {
      if (key) out(key + g * c.k_hs + 2 * el);
      if (l.shared && value && el < l.value) out(value + g * c.v_hs + 2 * el);
    }
  }
}

// Tokens of a block of which each has `units` of work: enough for its warps,
// no more than the sines hold or than leave every SM a block.
int tokens_of_block(int64_t tokens, int rotary, int units, int want, int sms) {
  int64_t n = std::max<int64_t>(1, want / std::max(1, units));
  if (rotary) n = std::min<int64_t>(n, kSinesMax / (rotary / 2));
  return (int)std::max<int64_t>(1, std::min<int64_t>(n, (tokens + sms - 1) / sms));
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int sms, cudaStream_t stream) {
  if (p.tokens <= 0 || p.heads <= 0) return cudaSuccess;
  const int groups = p.elems / 8;
  const int each = tokens_of_block(p.tokens, p.r.rotary, p.heads * groups, 4 * kThreads, sms);
  const int blocks = (p.tokens + each - 1) / each;
  if (p.f16) rotate_kernel<true><<<blocks, kThreads, 0, stream>>>(p, each);
  else rotate_kernel<false><<<blocks, kThreads, 0, stream>>>(p, each);
  return cudaGetLastError();
}

cudaError_t launch_pack(const PackCommon& c, const PackItem* items, int n_items, int sms,
                        cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kPackItemsMax) return cudaErrorInvalidValue;
  PackParams P;
  P.c = c;
  P.c.n_items = n_items;
  int64_t tokens = 0;
  for (int i = 0; i < kPackItemsMax; ++i) {
    P.first[i] = i < n_items ? tokens : INT64_MAX;
    if (i >= n_items) continue;
    P.items[i] = items[i];
    tokens += items[i].count;
  }
  P.c.tokens = tokens;
  if (!tokens) return cudaSuccess;
  const PackedLayout& l = c.l;
  const int longest = std::max(l.key8, l.shared ? 0 : l.value);
  P.lanes = 1;
  while (P.lanes < 32 && P.lanes * 16 < longest) P.lanes *= 2;
  const int heads = 32 / P.lanes;  // of a pass
  P.key_passes = (l.kv + heads - 1) / heads;
  P.value_passes = l.shared ? 0 : P.key_passes;
  P.wide_passes = (l.kv * (l.wide / 8) + 31) / 32;
  const int passes = P.key_passes + P.value_passes + P.wide_passes;
  P.tokens_each = tokens_of_block(tokens, c.r.rotary, passes, 2 * kWarps, sms);
  const int64_t blocks = (tokens + P.tokens_each - 1) / P.tokens_each;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (l.f16) pack_kernel<true><<<(int)blocks, kThreads, 0, stream>>>(P);
  else pack_kernel<false><<<(int)blocks, kThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_unpack(const UnpackCommon& c, const UnpackItem* items, int n_items, int sms,
                          cudaStream_t stream) {
  (void)sms;
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kUnpackItemsMax) return cudaErrorInvalidValue;
  UnpackParams P;
  P.c = c;
  P.c.n_items = n_items;
  int64_t count = 0;
  for (int i = 0; i < kUnpackItemsMax; ++i) {
    P.first[i] = i < n_items ? count : INT64_MAX;
    if (i >= n_items) continue;
    P.items[i] = items[i];
    count += items[i].count;
  }
  P.c.count = count;
  if (!count) return cudaSuccess;
  const PackedLayout& l = c.l;
  P.pieces = l.kv * (l.key8 / 16 + (l.shared ? 0 : l.value / 16) + l.wide / 8);
  const int64_t blocks = (count + kWarps * kWarpRows - 1) / (kWarps * kWarpRows);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (l.f16) unpack_kernel<true><<<(int)blocks, kThreads, 0, stream>>>(P);
  else unpack_kernel<false><<<(int)blocks, kThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace dhs
