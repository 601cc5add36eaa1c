// Attention jobs over blocks: how a launch's tiles are shared, and the kernel
// that joins the parts of jobs cut by a block's boundary.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attend_core.cuh"

namespace dhs {
namespace {

// ------------------------------------------------------------------ merge

constexpr int kMergeWarps = 16;
constexpr int kMergeElems = 128;  // value elements of a warp: a float4 a lane

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
// a trip to L2; 104 jobs of 64 columns in 2 to 3 parts, 34 MB, take 23 us.
// MANY (16 groups): a warp asks for all of its parts and statistics at once, in
// 128 registers; the sums are the same (one token over 512 K rows in 152 parts:
// 16-bit rows 113 -> 107 us, packed rows 77.5 -> 71.9).  With few parts to a warp
// there is nothing to ask for ahead, and two blocks to an SM are worth more.
template <bool MANY>
__global__ void __launch_bounds__(kMergeWarps * 32, MANY ? 1 : 2)
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
  if (on && MANY) {
    constexpr int kStats = (kAttendMaxBlocks + 31) / 32;
    constexpr int kParts = (kAttendMaxBlocks + kMergeWarps - 1) / kMergeWarps;
    const size_t ml = (size_t)M.columns * M.dv + col;
    float m[kStats], l[kStats];
    float4 y[kParts];
#pragma unroll
    for (int k = 0; k < kStats; ++k) {
      const int i = lane + 32 * k;
      m[k] = i < n ? part(i)[ml] : -INFINITY;
      l[k] = i < n ? part(i)[ml + M.columns] : 0.f;
    }
    const int mine = group + lane * kMergeWarps;
    const float my = mine < n ? part(mine)[ml] : -INFINITY;
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (group + k * kMergeWarps < n && d < M.dv)
        y[k] = *reinterpret_cast<const float4*>(part(group + k * kMergeWarps) + (size_t)col * M.dv + d);
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kStats; ++k) top = fmaxf(top, m[k]);
#pragma unroll
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int k = 0; k < kStats; ++k)
      if (lane + 32 * k < n) z += exp2_fast(m[k] - base) * l[k];
#pragma unroll
    for (int w = 16; w; w >>= 1) z += __shfl_xor_sync(~0u, z, w);
    const float weight = mine < n ? exp2_fast(my - base) : 0.f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float w = __shfl_sync(~0u, weight, k);
      // a part without weight may hold sums that are not finite
      if (group + k * kMergeWarps < n && w != 0.f && d < M.dv) {
        x.x += w * y[k].x;
        x.y += w * y[k].y;
        x.z += w * y[k].z;
        x.w += w * y[k].w;
      }
    }
  } else if (on) {
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

int columns_of(const AttendCommon& c, const AttendItem& it, int most) {
  const int all = it.loc ? c.group : it.Q * c.group;
  const int blk = (all + most - 1) / most;
  return (all + blk - 1) / blk;
}

}  // namespace

Shape shape_of(AttendCommon& c, AttendItem* items, int n_items, int sms, int most) {
  Shape s;
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
  // 512 K rows in 152 parts: 16 groups 116.5 us, 4 122.3 (107 since 16 groups
  // have a kernel of their own).
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

size_t parts_bytes(const AttendCommon& c, const Shape& s) {
  return s.n_cut ? (size_t)2 * s.blocks * s.n * (c.dv + 2) * sizeof(float) : 0;
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
  return cudaLaunchKernelEx(&cfg, s.groups == kMergeWarps ? merge_kernel<true> : merge_kernel<false>, M,
                            parts);
}

}  // namespace dhs
