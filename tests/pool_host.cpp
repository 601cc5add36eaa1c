// The pool's host side (pool.cpp) run without a GPU: the CUDA calls and the
// kernels' launchers are stand-ins on plain memory, every one of them logged.
// A scenario (argv[1]) drives the C ABI and checks what would reach the device.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "dhs.h"
#include "dhs_internal.h"

// ------------------------------------------------------------ allocations
// Allocation number `g_fail` from now on (0: the next one) fails, once.
static long g_fail = -1;
static bool g_failed = false;
void* operator new(size_t n) {
  if (g_fail >= 0 && g_fail-- == 0) {
    g_failed = true;
    throw std::bad_alloc();
  }
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

// ------------------------------------------------------------ CUDA
static std::vector<std::string>* g_log = nullptr;
static void note(const char* fmt, ...) {
  const long keep = g_fail;  // the log's own allocations never fail
  g_fail = -1;
  char s[160];
  va_list a;
  va_start(a, fmt);
  vsnprintf(s, sizeof s, fmt, a);
  va_end(a);
  g_log->push_back(s);
  g_fail = keep;
}

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : 232448;
  return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
  static uintptr_t next = 0x1000;
  *e = (cudaEvent_t)(next += 16);
  return cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) {
  note("record %p on %p", (void*)e, (void*)s);
  return cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned) {
  note("wait %p on %p", (void*)e, (void*)s);
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaHostGetDevicePointer(void** d, void* h, unsigned) { *d = h; return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t st) {
  note("copy %zu on %p", n, (void*)st);
  std::memcpy(d, s, n);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) {
  std::memset(d, v, n);
  return cudaSuccess;
}
}

// ------------------------------------------------------------ launchers
static const int32_t* g_map = nullptr;  // the page map that an attention was handed last
namespace dhs {
size_t resolve_smem_bytes(int, int, int, bool, int) { return 1024; }
cudaError_t resolve_set_smem_limit(size_t) { return cudaSuccess; }
cudaError_t resolve_set_carveout() { return cudaSuccess; }
cudaError_t hostcopy_set_carveout(size_t) { return cudaSuccess; }
cudaError_t gather_set_carveout() { return cudaSuccess; }
cudaError_t append_set_carveout() { return cudaSuccess; }
cudaError_t gather_set_smem_limit(int, int, bool* ok) { *ok = true; return cudaSuccess; }
cudaError_t noalloc_scratch(NoallocScratch*) { return cudaErrorInvalidValue; }
cudaError_t launch_resolve(const ResolveCommon&, const ResolveItem*, int, int, size_t, bool,
                           cudaStream_t) { return cudaSuccess; }
cudaError_t launch_hostcopy(const CopyCommon&, const CopyItem*, int, int, int, bool, size_t,
                            cudaStream_t) { return cudaSuccess; }
cudaError_t launch_gather(const GatherCommon&, const GatherItem*, int, bool, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_gather_later(const GatherCommon&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_append(const AppendCommon&, const AppendItem*, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_page_moves(const PageMove* m, int n, int bytes, int, cudaStream_t s) {
  note("moves %d on %p", n, (void*)s);
  for (int i = 0; i < n; ++i) std::memcpy(m[i].dst, m[i].src, bytes);
  return cudaSuccess;
}
bool attend_shape(AttendCommon, AttendItem*, int, int, size_t* bytes) {
  *bytes = 0;
  return true;
}
cudaError_t launch_attend(AttendCommon c, AttendItem*, int, int, void*, cudaStream_t s) {
  note("attend on %p", (void*)s);
  g_map = c.map;
  return cudaSuccess;
}
// The launch's limits, and the child's maps as the kernel writes them.
cudaError_t launch_fork(const ForkCommon& c, const ForkSource* src, int n, const int32_t* slots,
                        int n_slots, int, cudaStream_t) {
  if (n > kForkSourcesMax) return cudaErrorInvalidValue;
  if (!slots) return cudaSuccess;
  if (n > kForkSourcesSome || n_slots > kForkSlotsMax) return cudaErrorInvalidValue;
  for (int i = 0; i < n; ++i)
    for (int q = 0; q < c.Pmax; ++q)
      c.map[(size_t)src[i].to * c.Pmax + q] = q < src[i].complete ? slots[src[i].slot0 + q] : -1;
  return cudaSuccess;
}
cudaError_t launch_page_runs(uint8_t*, int32_t* map, int, int, const PageRun* r, int64_t n, int,
                             cudaStream_t) {
  for (int64_t i = 0; i < n; ++i)
    for (int k = 0; k < r[i].pages; ++k) map[r[i].map + k] = r[i].to + k;
  return cudaSuccess;
}
cudaError_t launch_clear_hot(int32_t*, uint32_t*, int64_t, cudaStream_t) { return cudaSuccess; }
}  // namespace dhs

// ------------------------------------------------------------ scenarios
#define CHECK(x)                                                        \
  do {                                                                  \
    if (!(x)) {                                                         \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);               \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

static void* zeros(size_t n) {
  void* p = std::aligned_alloc(256, (n + 256) / 256 * 256);
  std::memset(p, 0, (n + 256) / 256 * 256);
  return p;
}

constexpr int kRow = 16, kPage = 4;

struct Host {
  dhs_pool* p = nullptr;
  dhs_pool_config c{};
  int64_t pmax;
  std::map<int, uint8_t*> rows;  // host rows of each pair
  std::vector<uint8_t> dev, mask[2];  // prefilled rows; no page resident, every page

  Host(int requests, int sources, int64_t max_rows, int64_t pages) {
    c.max_requests = requests;
    c.sources = sources;
    c.row_bytes = kRow;
    c.page_rows = kPage;
    c.tail_rows = 4;
    c.hot_rows = 8;
    c.max_queries = 1;
    c.max_topk = 4;
    c.max_rows_per_request = max_rows;
    c.optional_pages = pages;
    size_t n[DHS_NUM_BUFS];
    CHECK(dhs_pool_bytes(&c, n) == DHS_OK);
    c.hot_dev = zeros(n[0]);
    c.tail_dev = zeros(n[1]);
    c.opt_dev = zeros(n[2]);
    c.meta_dev = zeros(n[3]);
    c.stream = (void*)0x100;
    CHECK(dhs_pool_create(&c, &p) == DHS_OK);
    pmax = (max_rows + kPage - 1) / kPage;
    for (int i = 0; i < requests * sources; ++i) rows[i] = (uint8_t*)zeros(max_rows * kRow);
    dev.assign(max_rows * kRow, 1);
    for (int i = 0; i < 2; ++i) mask[i].assign(pmax, i);
  }
  ~Host() { dhs_pool_destroy(p); }
  int admit(int req, int src, int64_t n, bool resident) {
    return dhs_admit_device(p, req, src, dev.data(), rows[req * c.sources + src], n,
                            mask[resident].data(), nullptr);
  }
  int fork(int req, int child) {
    std::vector<void*> h;
    for (int s = 0; s < c.sources; ++s) h.push_back(rows[child * c.sources + s]);
    return dhs_fork(p, req, child, h.data(), nullptr, nullptr);
  }
  // The page map of a pair: the host's, and the device's as an attention to
  // the pair's history is handed it.
  std::vector<int32_t> slots(int req, int src) {
    std::vector<int32_t> m(pmax);
    CHECK(dhs_read_state(p, req, src, nullptr, nullptr, m.data(), nullptr) == DHS_OK);
    return m;
  }
  std::vector<int32_t> device_slots(int req, int src) {
    CHECK(attend(req, src) == DHS_OK);
    const int32_t* m = g_map + (size_t)(req * c.sources + src) * pmax;
    return std::vector<int32_t>(m, m + pmax);
  }
  int attend(int req, int src, void* stream = nullptr) {
    dhs_attend_item it{};
    it.req = req;
    it.src = src;
    it.queries = 1;
    it.flags = DHS_ATTEND_HISTORY;
    it.q_dev = it.out_dev = c.tail_dev;
    dhs_attend_step st{};
    st.n_items = st.heads = st.kv_heads = 1;
    st.key_elems = st.value_elems = 8;
    st.scale = 1.f;
    st.items = &it;
    return stream ? dhs_attend_on(p, &st, stream) : dhs_attend(p, &st);
  }
};

// The child's slot held a request with two sources, the parent has one: the
// second source's old pages are gone from the device's map too.
static void fork_of_fewer_sources() {
  for (int parent_src = 0; parent_src < 2; ++parent_src) {
    Host h(3, 2, 64, 64);
    CHECK(h.admit(0, parent_src, 40, true) == DHS_OK);
    CHECK(h.admit(1, 0, 32, true) == DHS_OK && h.admit(1, 1, 32, true) == DHS_OK);
    CHECK(dhs_flush(h.p) == DHS_OK);
    CHECK(dhs_release(h.p, 1) == DHS_OK);
    CHECK(h.fork(0, 1) == DHS_OK);
    CHECK(h.admit(1, 1 - parent_src, 32, false) == DHS_OK);
    for (int s = 0; s < 2; ++s) CHECK(h.device_slots(1, s) == h.slots(1, s));
  }
}

// A fork that runs out of host memory at any of its allocations leaves the
// child empty, on the device too, and the pool as it was.
static void fork_without_memory() {
  bool done = false;
  for (int n = 0; !done; ++n) {
    Host h(3, 2, 64, 64);
    for (int s = 0; s < 2; ++s) CHECK(h.admit(0, s, 40, true) == DHS_OK);
    for (int s = 0; s < 2; ++s) CHECK(h.admit(1, s, 24, true) == DHS_OK);
    CHECK(dhs_flush(h.p) == DHS_OK);
    CHECK(dhs_release(h.p, 1) == DHS_OK);
    const int64_t used = dhs_pool_used(h.p), pending = dhs_pending_backup(h.p);
    std::vector<void*> hosts{h.rows[2], h.rows[3]};
    g_failed = false;
    g_fail = n;
    const int rc = dhs_fork(h.p, 0, 1, hosts.data(), nullptr, nullptr);
    g_fail = -1;
    done = !g_failed;
    CHECK(rc == (done ? DHS_OK : DHS_ENOMEM));
    if (done) break;
    CHECK(dhs_pool_used(h.p) == used && dhs_pending_backup(h.p) == pending);
    for (int s = 0; s < 2; ++s) {
      CHECK(h.admit(1, s, 24, false) == DHS_OK);
      CHECK(h.device_slots(1, s) == h.slots(1, s));
    }
  }
}

// Forks around the sizes of the launch's tables of page slots, spread over
// one source or several.
static void fork_table_limits() {
  for (int sources : {1, 4})
    for (int64_t pages : {511, 512, 513, dhs::kForkSlotsMax - 1, dhs::kForkSlotsMax,
                          dhs::kForkSlotsMax + 1}) {
      Host h(2, sources, pages * kPage, 2 * pages);
      for (int s = 0; s < sources; ++s) {
        const int64_t mine = pages / sources + (s < pages % sources);
        CHECK(h.admit(0, s, mine * kPage, true) == DHS_OK);
      }
      CHECK(h.fork(0, 1) == DHS_OK);
      CHECK(dhs_pool_used(h.p) == 2 * pages);
      for (int s = 0; s < sources; ++s) CHECK(h.device_slots(1, s) == h.slots(1, s));
    }
}

// Everything of a pool's state that calls change, the device's maps included.
static std::vector<int64_t> state(Host& h) {
  CHECK(dhs_flush(h.p) == DHS_OK);
  std::vector<int64_t> all{dhs_pool_used(h.p), dhs_pending_backup(h.p), dhs_pool_capacity(h.p)};
  for (int r = 0; r < h.c.max_requests; ++r)
    for (int s = 0; s < h.c.sources; ++s) {
      int64_t info[4];
      CHECK(dhs_read_state(h.p, r, s, nullptr, nullptr, nullptr, info) == DHS_OK);
      all.insert(all.end(), info, info + 3);
      for (int32_t x : h.slots(r, s)) all.push_back(x);
      if (info[2]) CHECK(h.device_slots(r, s) == h.slots(r, s));
    }
  return all;
}

// Each call with its allocations failing one after the other: DHS_ENOMEM and
// no exception, and the same call then leaves what it would have left.
static void calls_without_memory() {
  const int kCalls = 18;
  for (int k = 0; k < kCalls; ++k) {
    std::vector<int64_t> want;
    for (int n = -1;; ++n) {  // -1: nothing fails
      Host h(4, 2, 64, 40);
      for (int s = 0; s < 2; ++s) CHECK(h.admit(0, s, 40, true) == DHS_OK);
      CHECK(h.admit(1, 0, 40, false) == DHS_OK);
      CHECK(dhs_flush(h.p) == DHS_OK);
      // pages still to be copied, and some whose backup is deferred
      const auto admit_host = [&](int req) {
        return dhs_admit(h.p, req, 0, h.rows[req * 2], 20, nullptr, nullptr);
      };
      CHECK(admit_host(2) == DHS_OK);
      int32_t sel[4] = {0, 1, 2, 3};
      uint32_t loc[4] = {};
      alignas(16) uint8_t row[kRow] = {};
      dhs_item it[3]{};
      for (int i = 0; i < 3; ++i) {
        it[i].req = i;
        it[i].queries = 1;
        it[i].topk = 4;
        it[i].sel_dev = sel;
        it[i].loc_dev = loc;
        it[i].staging_dev = h.c.tail_dev;
      }
      const dhs_step st{1, 3, it};
      dhs_append_item ap[3]{};
      for (int i = 0; i < 3; ++i) {
        ap[i].req = i;
        ap[i].count = 1;
        ap[i].rows_dev = row;
      }
      const int32_t order[2] = {0, 1};
      int64_t x = 0, filled = 0;
      const auto call = [&]() -> int {
        switch (k) {
          case 0: return admit_host(3);
          case 1: return h.admit(3, 1, 40, true);
          case 2: return dhs_admit_window(h.p, 3, 0, h.c.tail_dev, 9);
          case 3: return dhs_backup(h.p, 7, &x);
          case 4:
            for (int rc; filled < 5; filled += x)
              if ((rc = dhs_refill(h.p, 5 - filled, &x))) return rc;
            return DHS_OK;
          case 5: return dhs_reclaim(h.p, order, 2, 12, &x);
          case 6: return dhs_release(h.p, 0);
          case 7: return dhs_flush(h.p);
          case 8: return dhs_append(h.p, ap, 3);
          case 9: return dhs_resolve(h.p, &st);
          case 10: return dhs_gather(h.p, &st);
          case 11: return dhs_gather_on(h.p, &st, (void*)0x200);
          case 12: return dhs_resolve_gather(h.p, &st);
          case 13: return dhs_decode_step(h.p, ap, 3, &st);
          case 14: return dhs_prefetch(h.p, &st, (void*)0x200);
          case 15: return h.attend(0, 1);
          case 16: return h.attend(0, 1, (void*)0x200);
          default: return dhs_compact(h.p, dhs_pool_used(h.p), &x);
        }
      };
      if (n < 0) {
        CHECK(call() == DHS_OK);
        want = state(h);
        continue;
      }
      g_failed = false;
      g_fail = n;
      int rc = 1;
      try {
        rc = call();
      } catch (...) {
      }
      g_fail = -1;
      if (k == 4 && g_failed && rc == DHS_OK) rc = DHS_ENOMEM;  // filled in two calls
      if (rc != (g_failed ? DHS_ENOMEM : DHS_OK)) std::printf("call %d, allocation %d: %d\n", k, n, rc);
      CHECK(rc == (g_failed ? DHS_ENOMEM : DHS_OK));
      if (g_failed) CHECK(call() == DHS_OK);
      CHECK(state(h) == want);
      if (!g_failed) break;
    }
  }
}

// A refill flushed while an attention to a history runs on another stream: the
// map that it reads is replaced behind it, and nothing else waits for it.
static void flush_behind_side_attention() {
  Host h(2, 1, 64, 40);
  CHECK(h.admit(0, 0, 40, false) == DHS_OK);
  CHECK(dhs_flush(h.p) == DHS_OK);
  int64_t n = 0;
  const auto waits = [] {
    int k = 0;
    for (const std::string& s : *g_log)
      k += s.compare(0, 4, "wait") == 0 && s.find("on 0x100") != std::string::npos;
    return k;
  };
  for (int flushed = 0; flushed < 2; ++flushed) {
    CHECK(h.attend(0, 0, (void*)0x200) == DHS_OK);
    if (flushed) CHECK(dhs_refill(h.p, 3, &n) == DHS_OK && n == 3);
    g_log->clear();
    CHECK(h.attend(0, 0) == DHS_OK);
    CHECK((waits() > 0) == flushed);
    const auto first = [](const char* what) {
      size_t i = 0;
      while (i < g_log->size() && (*g_log)[i].compare(0, strlen(what), what)) ++i;
      return i;
    };
    if (flushed) CHECK(first("wait") < first("moves") && first("wait") < first("copy"));
  }
  CHECK(h.device_slots(0, 0) == h.slots(0, 0));
}

int main(int argc, char** argv) {
  std::vector<std::string> log;
  g_log = &log;
  const std::map<std::string, void (*)()> all = {
      {"fork_of_fewer_sources", fork_of_fewer_sources},
      {"fork_without_memory", fork_without_memory},
      {"fork_table_limits", fork_table_limits},
      {"calls_without_memory", calls_without_memory},
      {"flush_behind_side_attention", flush_behind_side_attention},
  };
  const auto f = all.find(argc > 1 ? argv[1] : "");
  if (f == all.end()) return 2;
  f->second();
  std::printf("ok\n");
  return 0;
}
