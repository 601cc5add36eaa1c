// Attention over rows of the pool: located rows (a location vector) or a
// source's history (tail ring, optional pages, host copy), read in place.
//
// "Adaptive DHiSparse", How it works / Memory split: sparse attention reads
// the selected rows.  With x_j, y_j the key and the value of row j and s_j =
// scale (q . x_j), one pass keeps m = max s_j, l = sum exp(s_j - m) and
// o = sum exp(s_j - m) y_j; when m grows, l and o are scaled by
// exp(m_old - m_new).  out = o / l, log-sum = m + ln l.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kThreads = 128;

template <int MAXI>
struct AttendParams {
  AttendCommon c;
  AttendItem items[MAXI];
};
static_assert(sizeof(AttendParams<kAttendItemsLarge>) <= 32764, "attend item table too large");

__device__ __forceinline__ float to_float(const uint8_t* p, int f16) {
  return f16 ? __half2float(*reinterpret_cast<const __half*>(p))
             : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}

// Row j of the item for query i: its address, or null when there is none.
__device__ const uint8_t* row_of(const AttendCommon& c, const AttendItem& it, int i, int64_t j) {
  if (it.loc) {
    const int64_t e = (int64_t)i * it.len + j;
    uint32_t loc;
    if (it.index) {
      const int32_t u = it.index[e];
      if (u < 0) return nullptr;
      if (u >= (int64_t)it.Q * it.len) {
        atomicOr(c.status, kStatusEloc);
        return nullptr;
      }
      loc = it.loc[u];
    } else {
      loc = it.loc[e];
    }
    if (loc >= kEndLoc) return nullptr;
    const uint32_t tier = loc >> 30, x = loc & 0x3FFFFFFFu;
    const uint32_t rows = tier == kTierTail ? c.tail_rows : tier == kTierOpt ? c.opt_rows
                          : tier == kTierHot ? c.hot_rows : 0;
    if (x >= rows) {
      atomicOr(c.status, kStatusEloc);
      return nullptr;
    }
    const uint8_t* base = tier == kTierTail ? c.tail : tier == kTierOpt ? c.opt : c.hot;
    return base + (size_t)x * c.row_bytes;
  }
  const int64_t r = it.first + j, L = it.first + it.len;
  if (r >= L - c.T) return c.tail + ((size_t)it.pair * c.T + (size_t)(r % c.T)) * c.row_bytes;
  const int64_t page = r >> c.page_shift;
  if (page < it.complete) {
    const int32_t slot = c.map[(size_t)it.pair * c.Pmax + page];
    if (slot >= 0)
      return c.opt + (((size_t)slot << c.page_shift) + (r & ((1 << c.page_shift) - 1))) * c.row_bytes;
  }
  return it.host + (size_t)r * c.row_bytes;
}

// One CTA per (item, query, head): warps take 32 rows in turn for the
// scores, then every thread adds the rows to its output elements.
template <int MAXI>
__global__ void __launch_bounds__(kThreads)
    attend_kernel(const __grid_constant__ AttendParams<MAXI> P) {
  const AttendCommon& c = P.c;
  __shared__ float sq[kAttendMaxKey];
  __shared__ float sp[32];
  __shared__ const uint8_t* srow[32];
  const int job = blockIdx.x;
  int n = 0;
  while (n + 1 < c.n_items && P.items[n + 1].job0 <= job) ++n;
  const AttendItem& it = P.items[n];
  const int i = (job - it.job0) / c.heads, h = (job - it.job0) - i * c.heads;
  const int g = h / c.group;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int d = tid; d < c.dk; d += kThreads)
    sq[d] = to_float(it.q + i * c.q_qs + h * c.q_hs + 2 * d, c.f16);
  int64_t lo = 0, hi = it.len;
  if (!it.loc) {
    const int64_t L = it.first + it.len;
    const int64_t a = it.range ? it.range[2 * i] : 0;
    const int64_t b = it.range ? it.range[2 * i + 1] : L - it.Q + 1 + i;
    lo = max(a - it.first, (int64_t)0);
    hi = min(b, L) - it.first;
  }
  float m = -INFINITY, l = 0.f, o[kAttendMaxValue / kThreads] = {};
  for (int64_t j0 = lo; j0 < hi; j0 += 32) {
    __syncthreads();
    if (tid < 32) srow[tid] = j0 + tid < hi ? row_of(c, it, i, j0 + tid) : nullptr;
    __syncthreads();
    for (int j = warp; j < 32; j += kThreads / 32) {
      const uint8_t* row = srow[j];
      float s = 0.f;
      if (row)
        for (int d = lane; d < c.dk; d += 32)
          s += sq[d] * to_float(row + c.key_off + (int64_t)g * c.key_stride + 2 * d, c.f16);
      for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
      if (lane == 0) sp[j] = row ? s * c.scale : -INFINITY;
    }
    __syncthreads();
    float mn = m;
    for (int j = 0; j < 32; ++j) mn = fmaxf(mn, sp[j]);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - base);
    l *= f;
#pragma unroll
    for (int u = 0; u < kAttendMaxValue / kThreads; ++u) o[u] *= f;
    for (int j = 0; j < 32; ++j) {
      if (!srow[j]) continue;
      const float p = expf(sp[j] - base);
      l += p;
      const uint8_t* v = srow[j] + c.val_off + (int64_t)g * c.val_stride;
#pragma unroll
      for (int u = 0; u < kAttendMaxValue / kThreads; ++u)
        if (tid + u * kThreads < c.dv) o[u] += p * to_float(v + 2 * (tid + u * kThreads), c.f16);
    }
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int u = 0; u < kAttendMaxValue / kThreads; ++u) {
    const int d = tid + u * kThreads;
    if (d >= c.dv) continue;
    uint8_t* out = it.out + i * c.o_qs + h * c.o_hs + 2 * d;
    if (c.f16) *reinterpret_cast<__half*>(out) = __float2half_rn(o[u] * inv);
    else *reinterpret_cast<__nv_bfloat16*>(out) = __float2bfloat16_rn(o[u] * inv);
  }
  if (it.lse && tid == 0) it.lse[(size_t)i * c.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int MAXI>
cudaError_t launch_t(const AttendCommon& c, const AttendItem* items, int n_items,
                     cudaStream_t stream) {
  AttendParams<MAXI> P;
  P.c = c;
  P.c.n_items = n_items;
  int64_t jobs = 0;
  for (int i = 0; i < n_items; ++i) {
    P.items[i] = items[i];
    P.items[i].job0 = (int32_t)jobs;
    jobs += (int64_t)items[i].Q * c.heads;
    if (jobs > INT32_MAX) return cudaErrorInvalidValue;
  }
  P.c.n_jobs = (int32_t)jobs;
  attend_kernel<MAXI><<<(int)jobs, kThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const AttendCommon& c, const AttendItem* items, int n_items,
                          cudaStream_t stream) {
  if (n_items <= 0) return cudaSuccess;
  if (n_items > kAttendItemsLarge) return cudaErrorInvalidValue;
  return n_items <= kAttendItemsSmall ? launch_t<kAttendItemsSmall>(c, items, n_items, stream)
                                      : launch_t<kAttendItemsLarge>(c, items, n_items, stream);
}

}  // namespace dhs
