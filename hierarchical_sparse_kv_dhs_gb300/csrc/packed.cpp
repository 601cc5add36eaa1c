// C ABI of rotary positions and of rows in 8 bits (see include/dhs.h): checks
// of arguments, the launches' tables, and their order among the pool's work.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "pool_state.h"

using dhs::cuda_rc;
using dhs::kAlign;
using dhs::on_stream;
using dhs::PairState;
using dhs::room;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements: offsets stay far inside 64 bits

bool stride_ok(int64_t s) { return s > -kMaxStride && s < kMaxStride; }

bool type_ok(int32_t dtype) { return dtype == DHS_BF16 || dtype == DHS_F16; }

// The layout's parts; false for one that is refused.
bool layout_of(const dhs_packed_rows& r, dhs::PackedLayout* out) {
  if (!type_ok(r.dtype) || r.kv_heads < 1 || r.kv_heads > 65536) return false;
  if (r.wide_elems < 0 || r.wide_elems > DHS_PACKED_MAX_WIDE || r.wide_elems & 7) return false;
  if (r.key_elems < 16 || r.key_elems > DHS_ATTEND_MAX_KEY) return false;
  const int32_t key8 = r.key_elems - r.wide_elems;
  if (key8 < 16 || key8 & 15) return false;
  if (r.value_elems < 16 || r.value_elems > DHS_ATTEND_MAX_VALUE || r.value_elems & 15) return false;
  if (r.shared != 0 && r.shared != 1) return false;
  if (r.shared && r.value_elems > key8) return false;
  const int64_t kv = r.kv_heads;
  const int64_t off_value = kv * key8, off_wide = off_value + (r.shared ? 0 : kv * r.value_elems);
  const int64_t off_scale = off_wide + 2 * kv * r.wide_elems;
  const int64_t bytes = (off_scale + 4 * kv * (r.shared ? 1 : 2) + 15) / 16 * 16;
  if (bytes > 65536) return false;
  out->kv = r.kv_heads;
  out->key8 = key8;
  out->wide = r.wide_elems;
  out->value = r.value_elems;
  out->shared = r.shared;
  out->off_value = (int32_t)off_value;
  out->off_wide = (int32_t)off_wide;
  out->off_scale = (int32_t)off_scale;
  out->row_bytes = (int32_t)bytes;
  out->f16 = r.dtype == DHS_F16;
  return true;
}

// Select the pool's device for a call that touches nothing of the pool.
int on_device(dhs_pool* p) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return DHS_ECUDA;
  return cur == p->device ? DHS_OK : cuda_rc(cudaSetDevice(p->device));
}

bool rotation_ok(int32_t rotary, int32_t offset, int32_t pairs, float amplitude, const void* turns) {
  return rotary > 0 && rotary % 16 == 0 && offset >= 0 && offset % 8 == 0 &&
         (pairs == DHS_ROPE_HALF || pairs == DHS_ROPE_INTERLEAVED) &&
         amplitude - amplitude == 0.f && turns && (uintptr_t)turns % 8 == 0;
}

int check_pair(const dhs_pool* p, int32_t req, int32_t src) {
  const dhs_pool_config& c = p->cfg;
  if (req < 0 || req >= c.max_requests || src < 0 || src >= c.sources) return DHS_EINVAL;
  return p->ps[(int64_t)req * c.sources + src].admitted ? DHS_OK : DHS_ESTATE;
}

int check_rotate(dhs_pool* p, const dhs_rotate_step* st, dhs::RotateParams* out) {
  if (!p || !st || !type_ok(st->dtype) || st->tokens < 0 || st->heads < 0 || st->heads > 65536)
    return DHS_EINVAL;
  if (st->head_elems < 8 || st->head_elems > 65536 || st->head_elems & 7) return DHS_EINVAL;
  if (!rotation_ok(st->rotary_elems, st->rotary_offset, st->pairs, st->amplitude, st->turns_dev) ||
      st->rotary_elems > dhs::kRotaryMax ||
      (int64_t)st->rotary_offset + st->rotary_elems > st->head_elems)
    return DHS_EINVAL;
  if (st->flags & ~DHS_ROPE_INVERSE) return DHS_EINVAL;
  if (!stride_ok(st->x_token_stride) || !stride_ok(st->x_head_stride) ||
      !stride_ok(st->y_token_stride) || !stride_ok(st->y_head_stride))
    return DHS_EINVAL;
  if (st->tokens > 0 && st->heads > 0) {
    if (!st->x_dev || !st->y_dev || !st->position_dev) return DHS_EINVAL;
    if (((uintptr_t)st->x_dev | (uintptr_t)st->y_dev) & 1 || (uintptr_t)st->position_dev & 3)
      return DHS_EINVAL;
    if (st->x_dev == st->y_dev && (st->x_token_stride != st->y_token_stride ||
                                   st->x_head_stride != st->y_head_stride))
      return DHS_EINVAL;
  }
  dhs::RotateParams r{};
  r.x = (const uint8_t*)st->x_dev;
  r.y = (uint8_t*)st->y_dev;
  r.position = st->position_dev;
  r.r.turns = st->turns_dev;
  r.r.offset = st->rotary_offset;
  r.r.rotary = st->rotary_elems;
  r.r.interleaved = st->pairs == DHS_ROPE_INTERLEAVED;
  r.r.amplitude = st->amplitude;
  r.r.sign = st->flags & DHS_ROPE_INVERSE ? -1.f : 1.f;
  r.tokens = st->tokens;
  r.heads = st->heads;
  r.elems = st->head_elems;
  r.f16 = st->dtype == DHS_F16;
  r.x_ts = st->x_token_stride * 2;
  r.x_hs = st->x_head_stride * 2;
  r.y_ts = st->y_token_stride * 2;
  r.y_hs = st->y_head_stride * 2;
  *out = r;
  return DHS_OK;
}

// Checks a pack step and fills in the kernel's common parameters and the items
// that have tokens (in `items`).  appended: rows go to sources of the pool.
int pack_tables(dhs_pool* p, const dhs_pack_step* st, bool appended, dhs::PackCommon* out,
                std::vector<dhs::PackItem>* items) {
  if (!p || !st || st->n_items < 0 || (st->n_items > 0 && !st->items)) return DHS_EINVAL;
  const dhs_pool_config& cfg = p->cfg;
  dhs::PackCommon c{};
  if (!layout_of(st->rows, &c.l)) return DHS_EINVAL;
  if (appended && c.l.row_bytes != cfg.row_bytes) return DHS_EINVAL;
  if (st->rotary_elems != 0) {
    if (!rotation_ok(st->rotary_elems, st->rotary_offset, st->pairs, st->amplitude, st->turns_dev))
      return DHS_EINVAL;
    const int64_t end = (int64_t)st->rotary_offset + st->rotary_elems;
    if (end > st->rows.key_elems || (st->rotary_offset < c.l.key8 && end > c.l.key8))
      return DHS_EINVAL;
  }
  if (!stride_ok(st->key_token_stride) || !stride_ok(st->key_head_stride) ||
      !stride_ok(st->wide_token_stride) || !stride_ok(st->wide_head_stride) ||
      !stride_ok(st->value_token_stride) || !stride_ok(st->value_head_stride))
    return DHS_EINVAL;
  if (appended) std::fill(p->seen.begin(), p->seen.end(), 0);
  for (int32_t i = 0; i < st->n_items; ++i) {
    const dhs_pack_item& it = st->items[i];
    if (it.count < 0) return DHS_EINVAL;
    if (appended) {
      const int rc = check_pair(p, it.req, it.src);
      if (rc) return rc;
      const int64_t pair = (int64_t)it.req * cfg.sources + it.src;
      if (p->seen[pair] || it.count > cfg.tail_rows) return DHS_EINVAL;
      p->seen[pair] = 1;
      if (p->ps[pair].L + it.count > cfg.max_rows_per_request) return DHS_EINVAL;
    }
    if (it.count == 0) continue;
    if (!it.key_dev || (c.l.wide && !it.wide_dev) || (!c.l.shared && !it.value_dev)) return DHS_EINVAL;
    if (((uintptr_t)it.key_dev | (uintptr_t)it.wide_dev | (uintptr_t)it.value_dev) & 1)
      return DHS_EINVAL;
    if (st->rotary_elems && (!it.position_dev || (uintptr_t)it.position_dev & 3)) return DHS_EINVAL;
    if (!appended && (!it.rows_dev || (uintptr_t)it.rows_dev & 15)) return DHS_EINVAL;
  }
  c.r.turns = st->turns_dev;
  c.r.offset = st->rotary_offset;
  c.r.rotary = st->rotary_elems;
  c.r.interleaved = st->pairs == DHS_ROPE_INTERLEAVED;
  c.r.amplitude = st->amplitude;
  c.r.sign = 1.f;
  c.tail = (uint8_t*)cfg.tail_dev;
  c.T = cfg.tail_rows;
  c.k_ts = st->key_token_stride * 2;
  c.k_hs = st->key_head_stride * 2;
  c.w_ts = st->wide_token_stride * 2;
  c.w_hs = st->wide_head_stride * 2;
  c.v_ts = st->value_token_stride * 2;
  c.v_hs = st->value_head_stride * 2;
  if (!room(*items, (size_t)st->n_items)) return DHS_ENOMEM;
  for (int32_t i = 0; i < st->n_items; ++i) {
    const dhs_pack_item& it = st->items[i];
    if (it.count == 0) continue;
    dhs::PackItem t{};
    t.key = (const uint8_t*)it.key_dev;
    t.wide = (const uint8_t*)it.wide_dev;
    t.value = (const uint8_t*)it.value_dev;
    t.position = it.position_dev;
    t.count = it.count;
    if (appended) {
      const int64_t pair = (int64_t)it.req * cfg.sources + it.src;
      t.pair = (int32_t)pair;
      t.L0 = p->ps[pair].L;
      t.host = p->ps[pair].host_dev;
    } else {
      t.rows = (uint8_t*)it.rows_dev;
    }
    items->push_back(t);
  }
  *out = c;
  return DHS_OK;
}

int launch_packs(dhs_pool* p, const dhs::PackCommon& c, const std::vector<dhs::PackItem>& items) {
  for (size_t b = 0; b < items.size(); b += dhs::kPackItemsMax) {
    const int n = (int)std::min<size_t>(dhs::kPackItemsMax, items.size() - b);
    if (dhs::launch_pack(c, items.data() + b, n, std::max(1, p->sm_count), p->stream) != cudaSuccess)
      return DHS_ECUDA;
  }
  return DHS_OK;
}

// Checks an unpack step and fills in the kernel's parameters; *pool_rows: an
// item reads rows of the pool, *histories: by number.
int unpack_tables(dhs_pool* p, const dhs_unpack_step* st, dhs::UnpackCommon* out,
                  std::vector<dhs::UnpackItem>* items, bool* pool_rows, bool* histories) {
  *pool_rows = *histories = false;
  if (!p || !st || st->n_items < 0 || (st->n_items > 0 && !st->items)) return DHS_EINVAL;
  const dhs_pool_config& cfg = p->cfg;
  dhs::UnpackCommon c{};
  if (!layout_of(st->rows, &c.l)) return DHS_EINVAL;
  if (!stride_ok(st->key_row_stride) || !stride_ok(st->key_head_stride) ||
      !stride_ok(st->value_row_stride) || !stride_ok(st->value_head_stride))
    return DHS_EINVAL;
  if (!room(*items, (size_t)st->n_items)) return DHS_ENOMEM;
  for (int32_t i = 0; i < st->n_items; ++i) {
    const dhs_unpack_item& it = st->items[i];
    if (it.count < 0 || (it.flags & ~DHS_UNPACK_HISTORY)) return DHS_EINVAL;
    if (((uintptr_t)it.key_dev | (uintptr_t)it.value_dev) & 1) return DHS_EINVAL;
    dhs::UnpackItem t{};
    t.key = (uint8_t*)it.key_dev;
    t.value = (uint8_t*)it.value_dev;
    t.count = it.count;
    if (it.flags & DHS_UNPACK_HISTORY) {
      const int rc = check_pair(p, it.req, it.src);
      if (rc) return rc;
      const int64_t pair = (int64_t)it.req * cfg.sources + it.src;
      const PairState& s = p->ps[pair];
      const int64_t lo = s.window ? std::max<int64_t>(0, s.L - cfg.tail_rows) : 0;
      if (it.first < lo || it.first > s.L || it.count > s.L - it.first) return DHS_EINVAL;
      t.host = s.host_dev;
      t.first = it.first;
      t.L = s.L;
      t.pair = (int32_t)pair;
      t.complete = (int32_t)(s.N >> p->page_shift);
      *pool_rows = *histories = true;
    } else if (it.rows_dev) {
      if ((uintptr_t)it.rows_dev & 15) return DHS_EINVAL;
      t.rows = (const uint8_t*)it.rows_dev;
    } else {
      if (it.count > 0 && (!it.loc_dev || (uintptr_t)it.loc_dev & 3)) return DHS_EINVAL;
      t.loc = it.loc_dev;
      *pool_rows = true;
    }
    if (it.count > 0 && (t.key || t.value)) items->push_back(t);
  }
  if (*pool_rows && c.l.row_bytes != cfg.row_bytes) return DHS_EINVAL;
  c.tail = (const uint8_t*)cfg.tail_dev;
  c.opt = (const uint8_t*)cfg.opt_dev;
  c.hot = (const uint8_t*)cfg.hot_dev;
  c.map = p->map;
  c.tail_rows = (uint32_t)(p->pairs * cfg.tail_rows);
  c.opt_rows = (uint32_t)(p->capacity * cfg.page_rows);
  c.hot_rows = (uint32_t)(p->pairs * cfg.hot_rows);
  c.T = cfg.tail_rows;
  c.Pmax = (int32_t)p->pmax;
  c.page_shift = p->page_shift;
  c.status = p->status;
  c.k_rs = st->key_row_stride * 2;
  c.k_hs = st->key_head_stride * 2;
  c.v_rs = st->value_row_stride * 2;
  c.v_hs = st->value_head_stride * 2;
  *out = c;
  return DHS_OK;
}

int launch_unpacks(dhs_pool* p, const dhs::UnpackCommon& c, const std::vector<dhs::UnpackItem>& items) {
  for (size_t b = 0; b < items.size(); b += dhs::kUnpackItemsMax) {
    const int n = (int)std::min<size_t>(dhs::kUnpackItemsMax, items.size() - b);
    if (dhs::launch_unpack(c, items.data() + b, n, p->stream) != cudaSuccess)
      return DHS_ECUDA;
  }
  return DHS_OK;
}

// Checks and tables of a packed attention step, its workspace aside.
int attend_tables(dhs_pool* p, const dhs_attend_packed_step* st, dhs::AttendCommon* out,
                  dhs::PackedLayout* l) {
  if (!p || !st || st->n_items < 0 || (st->n_items > 0 && !st->items)) return DHS_EINVAL;
  if (!layout_of(st->rows, l) || l->row_bytes != p->cfg.row_bytes) return DHS_EINVAL;
  if (st->heads < 1 || st->heads % l->kv) return DHS_EINVAL;
  if (!(st->scale - st->scale == 0.f)) return DHS_EINVAL;  // finite
  int rc = dhs::check_attend_items(p, st->items, st->n_items, st->heads);
  if (rc) return rc;
  rc = dhs::fill_attend_items(p, st->items, st->n_items, out);
  dhs::AttendCommon& a = *out;
  a.f16 = l->f16;
  a.heads = st->heads;
  a.group = st->heads / l->kv;
  a.dv = l->value;
  a.scale = st->scale;
  a.q_qs = st->q_query_stride * 2;
  a.q_hs = st->q_head_stride * 2;
  a.o_qs = st->out_query_stride * 2;
  a.o_hs = st->out_head_stride * 2;
  return rc;
}

int attend_work(dhs_pool* p, const dhs::AttendCommon& a, const dhs::PackedLayout& l, size_t* bytes) {
  *bytes = 0;
  return dhs::each_attend_launch(p, [&](dhs::AttendItem* items, int n) {
    size_t need = 0;
    if (!dhs::attend_packed_shape(a, l, items, n, std::max(1, p->sm_count), &need)) return DHS_EINVAL;
    *bytes = std::max(*bytes, need);
    return DHS_OK;
  });
}

int prepare_attend(dhs_pool* p, const dhs_attend_packed_step* st, dhs::AttendCommon* a,
                   dhs::PackedLayout* l) {
  int rc = attend_tables(p, st, a, l);
  if (rc) return rc;
  size_t need = 0;
  if ((rc = attend_work(p, *a, *l, &need))) return rc;
  if (need && (!st->work_dev || (uintptr_t)st->work_dev % kAlign || st->work_bytes < need))
    return DHS_EINVAL;
  return dhs::enter_reads(p);
}

int launch_attends(dhs_pool* p, const dhs_attend_packed_step* st, const dhs::AttendCommon& a,
                   const dhs::PackedLayout& l) {
  return dhs::each_attend_launch(p, [&](dhs::AttendItem* items, int n) {
    return cuda_rc(dhs::launch_attend_packed(a, l, items, n, std::max(1, p->sm_count), st->work_dev,
                                             p->stream));
  });
}

}  // namespace

extern "C" {

int dhs_rope_table(const dhs_rope_config* cfg, uint64_t* turns) {
  if (!cfg || !turns) return DHS_EINVAL;
  const int32_t n = cfg->rotary_elems;
  if (n < 16 || n % 16 || n > 65536) return DHS_EINVAL;
  if (cfg->scaling < DHS_ROPE_PLAIN || cfg->scaling > DHS_ROPE_PARTS) return DHS_EINVAL;
  const bool plain = cfg->scaling == DHS_ROPE_PLAIN, parts = cfg->scaling == DHS_ROPE_PARTS;
  if (!(cfg->base > 1) || !std::isfinite(cfg->base)) return DHS_EINVAL;
  if (!plain && (!(cfg->factor >= 1) || !std::isfinite(cfg->factor))) return DHS_EINVAL;
  if (parts && (!(cfg->original > 0) || !std::isfinite(cfg->original) || !(cfg->slow >= 0) ||
                !(cfg->fast > cfg->slow) || !std::isfinite(cfg->fast)))
    return DHS_EINVAL;
  double base = cfg->base;
  if (cfg->scaling == DHS_ROPE_BASE) base *= std::pow(cfg->factor, n / (n - 2.0));
  if (!std::isfinite(base)) return DHS_EINVAL;
  const double circle = 6.283185307179586476925;
  for (int32_t i = 0; i < n / 2; ++i) {
    double f = std::pow(base, -2.0 * i / n);  // radians a position, at most 1
    if (cfg->scaling == DHS_ROPE_LINEAR) f /= cfg->factor;
    if (parts) {
      const double t = cfg->original * f / circle;
      const double keep = std::min(1.0, std::max(0.0, (t - cfg->slow) / (cfg->fast - cfg->slow)));
      f = f * keep + f / cfg->factor * (1 - keep);
    }
    turns[i] = (uint64_t)std::ldexp(f / circle, 64);
  }
  return DHS_OK;
}

int dhs_rotate(dhs_pool* p, const dhs_rotate_step* st) {
  dhs::RotateParams r;
  int rc = check_rotate(p, st, &r);
  if (rc) return rc;
  if ((rc = on_device(p))) return rc;
  return cuda_rc(dhs::launch_rotate(r, std::max(1, p->sm_count), p->stream));
}

int dhs_rotate_on(dhs_pool* p, const dhs_rotate_step* st, void* stream) {
  if (!stream) return DHS_EINVAL;
  dhs::RotateParams r;
  int rc = check_rotate(p, st, &r);
  if (rc) return rc;
  if ((rc = on_device(p))) return rc;
  return cuda_rc(dhs::launch_rotate(r, std::max(1, p->sm_count), (cudaStream_t)stream));
}

int dhs_packed_bytes(const dhs_packed_rows* rows, int32_t* row_bytes) {
  if (row_bytes) *row_bytes = 0;
  dhs::PackedLayout l;
  if (!rows || !row_bytes || !layout_of(*rows, &l)) return DHS_EINVAL;
  *row_bytes = l.row_bytes;
  return DHS_OK;
}

int dhs_pack(dhs_pool* p, const dhs_pack_step* st) {
  dhs::PackCommon c;
  std::vector<dhs::PackItem> items;
  int rc = pack_tables(p, st, false, &c, &items);
  if (rc) return rc;
  if ((rc = on_device(p))) return rc;
  return launch_packs(p, c, items);
}

int dhs_append_packed(dhs_pool* p, const dhs_pack_step* st) {
  dhs::PackCommon c;
  std::vector<dhs::PackItem> items;
  int rc = pack_tables(p, st, true, &c, &items);
  if (rc) return rc;
  if ((rc = dhs::enter_writes(p))) return rc;
  for (const dhs::PackItem& it : items) p->ps[it.pair].L += it.count;
  return launch_packs(p, c, items);
}

int dhs_unpack(dhs_pool* p, const dhs_unpack_step* st) {
  dhs::UnpackCommon c;
  std::vector<dhs::UnpackItem> items;
  bool pool_rows, histories;
  int rc = unpack_tables(p, st, &c, &items, &pool_rows, &histories);
  if (rc) return rc;
  if ((rc = pool_rows ? dhs::enter_reads(p) : on_device(p))) return rc;
  return launch_unpacks(p, c, items);
}

int dhs_unpack_on(dhs_pool* p, const dhs_unpack_step* st, void* stream) {
  if (!stream) return DHS_EINVAL;
  dhs::UnpackCommon c;
  std::vector<dhs::UnpackItem> items;
  bool pool_rows, histories;
  int rc = unpack_tables(p, st, &c, &items, &pool_rows, &histories);
  if (rc) return rc;
  if ((rc = dhs::enter_reads(p))) return rc;
  p->map_readers |= histories;
  return on_stream(p, stream, [&] { return launch_unpacks(p, c, items); });
}

int dhs_attend_packed_bytes(dhs_pool* p, const dhs_attend_packed_step* st, size_t* bytes) {
  if (bytes) *bytes = 0;
  if (!bytes) return DHS_EINVAL;
  dhs::AttendCommon a;
  dhs::PackedLayout l;
  const int rc = attend_tables(p, st, &a, &l);
  return rc ? rc : attend_work(p, a, l, bytes);
}

int dhs_attend_packed(dhs_pool* p, const dhs_attend_packed_step* st) {
  dhs::AttendCommon a;
  dhs::PackedLayout l;
  const int rc = prepare_attend(p, st, &a, &l);
  return rc ? rc : launch_attends(p, st, a, l);
}

int dhs_attend_packed_on(dhs_pool* p, const dhs_attend_packed_step* st, void* stream) {
  if (!stream) return DHS_EINVAL;
  dhs::AttendCommon a;
  dhs::PackedLayout l;
  const int rc = prepare_attend(p, st, &a, &l);
  if (rc) return rc;
  for (const dhs::AttendItem& it : p->titems) p->map_readers |= !it.loc;
  return on_stream(p, stream, [&] { return launch_attends(p, st, a, l); });
}

}  // extern "C"
