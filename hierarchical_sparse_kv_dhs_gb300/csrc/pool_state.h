// The pool's host state, for the C ABI's two files: pool.cpp (the pool, its
// steps, attention, forks) and packed.cpp (rows in 8 bits).  Not part of the
// C ABI.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "dhs.h"
#include "dhs_internal.h"

namespace dhs {

constexpr size_t kAlign = 256;

struct MetaLayout {
  size_t tags, stamps, map, miss_rows, miss_slots, miss_count, copy_cursor, pair_status;
  size_t loc_ready, copy_ready, fill, later_count, status, later, miss_off, miss_ent;
  size_t total;
};

struct PairState {
  bool admitted = false;
  bool window = false;          // window source: the tail ring is its only storage
  int64_t N = 0, L = 0;
  uint8_t* host = nullptr;      // caller's pinned host rows
  uint8_t* host_dev = nullptr;  // device-visible address of the same rows
  std::vector<int32_t> pending;  // resident pages whose bytes are not yet copied
  std::vector<uint64_t> backup;  // per page: backup order while the host copy is
                                 // deferred, 0 = backed (empty: all backed)
};

struct BackupRun {
  uint64_t order;  // of the first page
  int32_t pair, page, pages;
};

}  // namespace dhs

struct dhs_pool {
  dhs_pool_config cfg{};
  cudaStream_t stream = nullptr;
  int device = 0;
  int64_t pairs = 0, pmax = 0, mcap = 0;
  int page_shift = 0;
  dhs::MetaLayout layout{};
  int32_t* tags = nullptr;
  uint32_t* stamps = nullptr;
  int32_t* map = nullptr;
  int32_t* miss_rows = nullptr;
  int32_t* miss_slots = nullptr;
  uint32_t* miss_count = nullptr;
  uint32_t* copy_cursor = nullptr;
  int32_t* pair_status = nullptr;
  uint32_t* status = nullptr;
  std::vector<dhs::PairState> ps;
  std::vector<int32_t> map_host;  // [pairs][pmax] mirror of the device map
  std::vector<int32_t> slot_pair, slot_page;
  int64_t first_free = 0, used = 0;
  int64_t capacity = 0;  // optional page slots in use or free (dhs_compact lowers it)
  int64_t dirty_lo = INT64_MAX, dirty_hi = -1;  // pairs whose map changed
  bool any_pending = false;
  int copy_ctas = 0;
  bool union_ok = false;  // the union staging plan fits in shared memory
  int gather_impl = dhs::kGatherTma;
  bool tma_ok = true;  // the TMA gather's tile fits the row size
  int gather_tpc = 1;   // DHS_OPT_GATHER_TPC
  int early = 1;        // fused gathers copy step-1 rows before the resolve ends
  uint32_t seq = 0;             // resolve launches so far
  uint32_t* loc_ready = nullptr;  // [pairs] per-item "locations written" marks
  uint32_t* copy_ready = nullptr; // [pairs] per-item "miss lists written" marks
  uint32_t* fill = nullptr;       // [pairs][fill_words] slots the step's copy fills
  uint32_t* later_count = nullptr;
  dhs::LaterEntry* later = nullptr;
  int64_t later_cap = 0;
  int fill_words = 0;
  uint32_t gen = 0;             // fused steps that launched a resolve
  bool fused_resolved = false;  // the current fused step launched one
  int fresh_list = -1;          // DHS_OPT_FRESH_LIST: -1 auto, 0 off, 1 on
  int64_t complete_pages = 0;   // complete imported pages of admitted pairs
  uint64_t bseq = 0;            // pages put in backup order so far
  // Pages whose host backup is deferred, in order, as runs of consecutive
  // pages and orders (a fork or an admission queues thousands at a time).  A
  // page of a run counts while its PairState::backup holds its order; the
  // others are skipped, and runs without any swept out now and then.
  std::vector<dhs::BackupRun> backup_queue;
  size_t backup_head = 0;       // runs before it are done with
  int64_t backup_live = 0;
  int32_t rr = 0;               // refill cursor: the next request visited
  int sm_count = 0;
  int smem_optin = 0;           // opt-in shared memory per block
  int32_t* miss_off = nullptr;  // [pairs][Mcap + 1] staging entries of each miss
  int32_t* miss_ent = nullptr;  // [pairs][ent_cap]
  int64_t ent_cap = 0;
  int stage_misses = 1;         // DHS_OPT_STAGE_MISSES
  uint32_t mark_polls = dhs::kMarkPolls;  // DHS_OPT_MARK_POLLS
  uint32_t attend_polls = dhs::kAttendPolls;  // DHS_OPT_ATTEND_POLLS
  int copy_pdl = -1;            // DHS_OPT_COPY_PDL: -1 auto, 0 off, 1 on
  int resolve_paired = -1;      // DHS_OPT_RESOLVE_PAIRED: -1 auto, 0 off, 1 whenever it fits
  int copy_steal = -1;          // DHS_OPT_COPY_STEAL: -1 auto, 0 off, 1 on
  int resolve_ctas = 0;         // DHS_OPT_RESOLVE_CTAS: 0 auto, > 0 at most that many
  int smem_per_sm = 0;          // shared memory per SM
  std::vector<uint8_t> staged_pair;  // the host copy stages this pair's misses this step
  std::vector<uint8_t> staged_item;  // per item of the step: a gather-only item whose
                                     // staging the host copy writes too
  unsigned long long* trace = nullptr;  // DHS_OPT_TRACE buffer, null = off
  // reusable launch tables
  std::vector<dhs::ResolveItem> ritems;
  std::vector<dhs::CopyItem> citems;
  std::vector<dhs::GatherItem> gitems;
  // gathers of a fused step: the resolved items' location vectors, sorted,
  // to find which pair (if any) published a gather item's locations
  struct LocKey {
    const void* loc;
    int32_t order;  // item index: of equal vectors the last one counts
    int64_t pair;
    bool operator<(const LocKey& o) const {
      return loc != o.loc ? std::less<const void*>()(loc, o.loc) : order < o.order;
    }
  };
  std::vector<LocKey> loc_keys;
  std::vector<dhs::AppendItem> aitems;
  std::vector<dhs::AttendItem> titems;
  std::vector<dhs::PageRun> runs;      // page runs of a compaction
  std::vector<uint8_t> seen;
  std::vector<int32_t> app_of_pair;  // decode step: append item of each pair, -1 = none
  std::vector<int64_t> l0_of_pair;   // length of each resolved pair before this step's append
  std::vector<const uint8_t*> app_of_pair_rows;  // its appended rows' source, or null
  std::vector<uint32_t> seq_of_pair; // resolve launch that last resolved each pair
  std::vector<dhs::PageMove> moves;  // page list of the next page-move launch
  // dhs_prefetch: resolves enqueued on a caller's side stream; the pool's
  // stream waits for them before its next device work
  cudaEvent_t ev_main = nullptr, ev_prefetch = nullptr;
  // dhs_decode_step_host_async on callers' copy streams: the step waits for
  // the inputs (ev_in), the outputs' copies wait for the step (ev_step)
  cudaEvent_t ev_in = nullptr, ev_step = nullptr;
  bool prefetch_pending = false;
  bool join_gathers = true;  // enter(): also join gathers on other streams
  std::vector<uint8_t> pf_pair;  // pairs resolved by the outstanding prefetch
  // dhs_gather_on: gathers on callers' streams read rows the pool's next
  // resolve / append / admission may change; one event per such call,
  // joined (and recycled) by the pool's next call that can change rows
  std::vector<cudaEvent_t> ev_free, ev_gathers;
  bool map_readers = false;  // some of them read the page maps (histories)
  ~dhs_pool() {
    if (ev_main) cudaEventDestroy(ev_main);
    if (ev_prefetch) cudaEventDestroy(ev_prefetch);
    if (ev_in) cudaEventDestroy(ev_in);
    if (ev_step) cudaEventDestroy(ev_step);
    for (cudaEvent_t e : ev_free) cudaEventDestroy(e);
    for (cudaEvent_t e : ev_gathers) cudaEventDestroy(e);
  }
};

namespace dhs {

inline int cuda_rc(cudaError_t e) { return e == cudaSuccess ? DHS_OK : DHS_ECUDA; }

// For a call that only reads rows: the pool's device, its stream behind an
// outstanding prefetch, pending page copies and map uploads enqueued.
int enter_reads(dhs_pool* p);
// For a call that changes rows: reads on other streams are joined too, and
// nothing else is enqueued.
int enter_writes(dhs_pool* p);

// Items of an attention step: refused or not, and as the kernels' table
// (p->titems, with the pool's part of the common parameters).
int check_attend_items(dhs_pool* p, const dhs_attend_item* items, int32_t n, int32_t heads);
int fill_attend_items(dhs_pool* p, const dhs_attend_item* items, int32_t n, AttendCommon* out);

// Calls f(items, n) for every launch's share of the item table.
template <class F>
int each_attend_launch(dhs_pool* p, F f) {
  for (size_t b = 0; b < p->titems.size(); b += dhs::kAttendItemsLarge) {
    const int n = (int)std::min<size_t>(dhs::kAttendItemsLarge, p->titems.size() - b);
    const int rc = f(p->titems.data() + b, n);
    if (rc) return rc;
  }
  return DHS_OK;
}

// Room for n elements in all, so that adding them cannot throw.
template <class T>
bool room(std::vector<T>& v, size_t n) {
  try {
    v.reserve(n);
  } catch (...) {
    return false;
  }
  return true;
}

// Run `launch` on a caller's stream: after everything the pool's stream holds,
// and joined by the pool's next call that can change rows.
template <class Launch>
int on_stream(dhs_pool* p, void* stream, Launch launch) {
  cudaStream_t other = (cudaStream_t)stream;
  cudaEvent_t done = nullptr;
  // the events come back to ev_free when they are joined
  const size_t gathers = p->ev_gathers.size() + 1;
  if (!room(p->ev_gathers, gathers) || !room(p->ev_free, p->ev_free.size() + gathers))
    return DHS_ENOMEM;
  if (!p->ev_free.empty()) {
    done = p->ev_free.back();
    p->ev_free.pop_back();
  } else if (cudaEventCreateWithFlags(&done, cudaEventDisableTiming) != cudaSuccess) {
    return DHS_ECUDA;
  }
  // after everything the pool's stream holds (resolves, copies, appends)
  if (cudaEventRecord(p->ev_main, p->stream) != cudaSuccess ||
      cudaStreamWaitEvent(other, p->ev_main, 0) != cudaSuccess) {
    p->ev_free.push_back(done);
    return DHS_ECUDA;
  }
  cudaStream_t main = p->stream;
  p->stream = other;
  const int rc = launch();
  p->stream = main;
  // joined before the pool's next call that can change rows, even if the
  // launch failed part way
  if (cudaEventRecord(done, other) != cudaSuccess) {
    p->ev_free.push_back(done);
    return DHS_ECUDA;
  }
  p->ev_gathers.push_back(done);
  return rc;
}

}  // namespace dhs
