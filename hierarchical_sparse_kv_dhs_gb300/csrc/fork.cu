// Fork kernel: one request's rows into another request slot.
//
// Every row moves once, from where the parent's step-1 place or host copy
// holds it to where the child keeps it: complete pages (either side optional
// page or host rows, by the two page maps), rows past them (host to host),
// the tail ring and the filled hot-cache slots with their tags and stamps.
#include "dhs_internal.h"

namespace dhs {
namespace {

constexpr int kForkThreads = 256;

struct ForkParams {
  ForkCommon c;
  ForkSource s[kForkSourcesMax];
};
static_assert(sizeof(ForkParams) <= 32764, "fork source table too large");

// One warp per row; row units of a source: history rows, tail rows, hot slots.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkParams P) {
  const ForkCommon& c = P.c;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kForkThreads / 32);
  int n = 0;
  for (int u = blockIdx.x * (kForkThreads / 32) + (threadIdx.x >> 5); u < c.n_units; u += warps) {
    while (n + 1 < c.n_sources && P.s[n + 1].unit0 <= u) ++n;
    const ForkSource& s = P.s[n];
    int64_t r = u - s.unit0;
    const int64_t hist = s.host_from ? s.L : 0;
    const uint8_t* from;
    uint8_t* to;
    const size_t rb = c.row_bytes;
    if (r < hist) {
      const int64_t page = r >> c.page_shift, in = r & ((1 << c.page_shift) - 1);
      int32_t a = -1, b = -1;
      if (page < s.complete) {
        a = c.map[(size_t)s.from * c.Pmax + page];
        b = c.map[(size_t)s.to * c.Pmax + page];
      }
      from = a >= 0 ? c.opt + (((size_t)a << c.page_shift) + in) * rb : s.host_from + r * rb;
      to = b >= 0 ? c.opt + (((size_t)b << c.page_shift) + in) * rb : s.host_to + r * rb;
    } else if ((r -= hist) < c.T) {
      if (r >= s.L) continue;  // ring slots that hold no row yet
      from = c.tail + ((size_t)s.from * c.T + r) * rb;
      to = c.tail + ((size_t)s.to * c.T + r) * rb;
    } else {
      r -= c.T;
      const int32_t tag = c.tags[(size_t)s.from * c.B + r];
      if (lane == 0) {
        c.tags[(size_t)s.to * c.B + r] = tag;
        c.stamps[(size_t)s.to * c.B + r] = c.stamps[(size_t)s.from * c.B + r];
      }
      if (tag < 0) continue;
      from = c.hot + ((size_t)s.from * c.B + r) * rb;
      to = c.hot + ((size_t)s.to * c.B + r) * rb;
    }
    for (int k = lane * 16; k < (int)rb; k += 512)
      __stcs(reinterpret_cast<uint4*>(to + k), __ldcs(reinterpret_cast<const uint4*>(from + k)));
  }
}

}  // namespace

cudaError_t launch_fork(const ForkCommon& c, const ForkSource* sources, int n_sources, int sms,
                        cudaStream_t stream) {
  if (n_sources <= 0) return cudaSuccess;
  if (n_sources > kForkSourcesMax) return cudaErrorInvalidValue;
  ForkParams P;
  P.c = c;
  P.c.n_sources = n_sources;
  int64_t units = 0;
  for (int i = 0; i < n_sources; ++i) {
    P.s[i] = sources[i];
    P.s[i].unit0 = (int32_t)units;
    units += (sources[i].host_from ? sources[i].L : 0) + c.T + c.B;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
  }
  P.c.n_units = (int32_t)units;
  fork_kernel<<<sms * 8, kForkThreads, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace dhs
