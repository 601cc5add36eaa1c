// The host side of rotations and of packed rows (packed.cpp) run without a GPU, on
// pool_host.cpp's stand-ins.
#define main pool_host_main
#include "pool_host.cpp"
#undef main

namespace dhs {
cudaError_t launch_rotate(const RotateParams& p, int, cudaStream_t s) {
  note("rotate %d on %p", p.tokens, (void*)s);
  return cudaSuccess;
}
cudaError_t launch_pack(const PackCommon&, const PackItem*, int n, int, cudaStream_t s) {
  note("pack %d on %p", n, (void*)s);
  return n <= kPackItemsMax ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t launch_unpack(const UnpackCommon&, const UnpackItem*, int n, cudaStream_t s) {
  note("unpack %d on %p", n, (void*)s);
  return n <= kUnpackItemsMax ? cudaSuccess : cudaErrorInvalidValue;
}
bool attend_packed_shape(AttendCommon, const PackedLayout&, AttendItem*, int, int, size_t* bytes) {
  *bytes = 0;
  return true;
}
cudaError_t launch_attend_packed(AttendCommon c, const PackedLayout&, AttendItem*, int n, int, void*,
                                 cudaStream_t s) {
  note("attend_packed %d on %p", n, (void*)s);
  g_map = c.map;
  return cudaSuccess;
}
}  // namespace dhs

constexpr int kBytes = 32;  // the smallest packed row: 16 codes, a scale, padding
static const dhs_packed_rows kLayout{DHS_BF16, 1, 16, 0, 16, 1};

struct Packed {
  dhs_pool* p = nullptr;
  dhs_pool_config c{};
  std::map<int, uint8_t*> rows;
  std::vector<uint8_t> dev;
  alignas(256) uint8_t data[4096] = {};

  Packed(int requests = 3, int64_t max_rows = 64) {
    c.max_requests = requests;
    c.sources = 1;
    c.row_bytes = kBytes;
    c.page_rows = kPage;
    c.tail_rows = 4;
    c.hot_rows = 8;
    c.max_queries = 1;
    c.max_topk = 4;
    c.max_rows_per_request = max_rows;
    c.optional_pages = 40;
    size_t n[DHS_NUM_BUFS];
    CHECK(dhs_pool_bytes(&c, n) == DHS_OK);
    c.hot_dev = zeros(n[0]);
    c.tail_dev = zeros(n[1]);
    c.opt_dev = zeros(n[2]);
    c.meta_dev = zeros(n[3]);
    c.stream = (void*)0x100;
    CHECK(dhs_pool_create(&c, &p) == DHS_OK);
    for (int i = 0; i < requests; ++i) rows[i] = (uint8_t*)zeros(max_rows * kBytes);
    dev.assign(max_rows * kBytes, 1);
    for (int i = 0; i < requests; ++i)
      CHECK(dhs_admit_device(p, i, 0, dev.data(), rows[i], 20, nullptr, nullptr) == DHS_OK);
    CHECK(dhs_flush(p) == DHS_OK);
  }
  ~Packed() { dhs_pool_destroy(p); }

  dhs_attend_item history(int req) {
    dhs_attend_item it{};
    it.req = req;
    it.queries = 1;
    it.flags = DHS_ATTEND_HISTORY;
    it.q_dev = it.out_dev = data;
    return it;
  }
  dhs_attend_item located() {
    dhs_attend_item it{};
    it.queries = 1;
    it.topk = 4;
    it.q_dev = it.out_dev = data;
    it.loc_dev = (const uint32_t*)data;
    return it;
  }
  int attend(const dhs_attend_item* items, int n, void* stream = nullptr) {
    dhs_attend_packed_step st{};
    st.rows = kLayout;
    st.n_items = n;
    st.heads = 1;
    st.scale = 1.f;
    st.items = items;
    return stream ? dhs_attend_packed_on(p, &st, stream) : dhs_attend_packed(p, &st);
  }
  int attend16(const dhs_attend_item* items, int n) {
    dhs_attend_step st{};
    st.n_items = n;
    st.heads = st.kv_heads = 1;
    st.key_elems = st.value_elems = 8;
    st.scale = 1.f;
    st.items = items;
    return dhs_attend(p, &st);
  }
  int unpack(const std::vector<dhs_unpack_item>& items, void* stream = nullptr) {
    dhs_unpack_step st{};
    st.rows = kLayout;
    st.n_items = (int32_t)items.size();
    st.items = items.data();
    return stream ? dhs_unpack_on(p, &st, stream) : dhs_unpack(p, &st);
  }
  int pack(const std::vector<dhs_pack_item>& items, bool append) {
    dhs_pack_step st{};
    st.rows = kLayout;
    st.n_items = (int32_t)items.size();
    st.items = items.data();
    return append ? dhs_append_packed(p, &st) : dhs_pack(p, &st);
  }
  std::vector<dhs_pack_item> new_rows(int n, int count) {
    std::vector<dhs_pack_item> v((size_t)n);
    for (int i = 0; i < n; ++i) {
      v[(size_t)i].req = i;
      v[(size_t)i].count = count;
      v[(size_t)i].key_dev = v[(size_t)i].rows_dev = data;
    }
    return v;
  }
  std::vector<dhs_unpack_item> reads(int n) {
    std::vector<dhs_unpack_item> v((size_t)n);
    for (dhs_unpack_item& it : v) {
      it.count = 5;
      it.flags = DHS_UNPACK_HISTORY;
      it.key_dev = data;
    }
    return v;
  }
  int64_t length(int req) {
    int64_t info[8] = {};
    CHECK(dhs_read_state(p, req, 0, nullptr, nullptr, nullptr, info) == DHS_OK);
    return info[1];
  }
};

// Lists that the kernels read 4 bytes at a time, at addresses between those.
static void lists_out_of_line() {
  Packed h;
  for (int which = 0; which < 3; ++which)
    for (int off = 0; off < 8; ++off) {
      dhs_attend_item it = which == 2 ? h.history(0) : h.located();
      const void* at = h.data + off;
      if (which == 0) it.loc_dev = (const uint32_t*)at;
      if (which == 1) it.index_dev = (const int32_t*)at;
      if (which == 2) it.range_dev = (const int32_t*)at;
      g_log->clear();
      const int want = off % 4 ? DHS_EINVAL : DHS_OK;
      CHECK(h.attend(&it, 1) == want);
      CHECK(h.attend(&it, 1, (void*)0x200) == want);
      CHECK(h.attend16(&it, 1) == want);
      if (want) CHECK(g_log->empty());
    }
}

// Every host allocation of every call fails once: the call says so, nothing has
// reached a stream, lengths are as they were, and the same call works afterwards.
static void packed_calls_without_memory() {
  for (int k = 0; k < 7; ++k)
    for (int n = 0;; ++n) {
      Packed h;
      const dhs_attend_item its[2] = {h.history(0), h.located()};
      const auto fresh = h.new_rows(3, 2);
      const auto reads = h.reads(3);
      const auto call = [&] {
        switch (k) {
          case 0: return h.pack(fresh, false);
          case 1: return h.pack(fresh, true);
          case 2: return h.unpack(reads);
          case 3: return h.unpack(reads, (void*)0x200);
          case 4: return h.attend(its, 2);
          case 5: return h.attend(its, 2, (void*)0x200);
          default: return dhs_compact(h.p, dhs_pool_used(h.p), nullptr);  // (behind reads on 0x200)
        }
      };
      if (k == 6) CHECK(h.unpack(reads, (void*)0x200) == DHS_OK);
      g_log->clear();
      g_failed = false;
      g_fail = n;
      int rc = 1;
      try {
        rc = call();
      } catch (...) {
      }
      g_fail = -1;
      CHECK(rc == (g_failed ? DHS_ENOMEM : DHS_OK));
      if (g_failed) {
        for (const std::string& s : *g_log) CHECK(s.find("pack") == std::string::npos);
        CHECK(h.length(0) == 20);
        CHECK(call() == DHS_OK);
      }
      CHECK(h.length(0) == (k == 1 ? 22 : 20));
      if (!g_failed) break;
    }
}

// More items than a launch's table has room for, and items without rows.
static void packed_tables() {
  Packed h;
  for (int n : {0, 1, 16, 17, 256, 257, 700}) {
    std::vector<dhs_pack_item> v = h.new_rows(n, 3);
    for (dhs_pack_item& it : v) it.req = 0;
    g_log->clear();
    CHECK(h.pack(v, false) == DHS_OK);
    size_t rows = 0;
    for (const std::string& s : *g_log) rows += (size_t)std::atoi(s.c_str() + 5);
    CHECK((int)rows == n && (int)g_log->size() == (n + 255) / 256);
    for (size_t i = 0; i < v.size(); i += 2) v[i].count = 0;
    g_log->clear();
    CHECK(h.pack(v, false) == DHS_OK);
    CHECK((int)g_log->size() == (n / 2 + 255) / 256);
    g_log->clear();
    CHECK(h.unpack(h.reads(n)) == DHS_OK);
    CHECK((int)g_log->size() == (n + 255) / 256);
  }
}

int main(int argc, char** argv) {
  std::vector<std::string> log;
  g_log = &log;
  const std::map<std::string, void (*)()> all = {
      {"lists_out_of_line", lists_out_of_line},
      {"packed_calls_without_memory", packed_calls_without_memory},
      {"packed_tables", packed_tables},
  };
  const auto f = all.find(argc > 1 ? argv[1] : "");
  if (f == all.end()) return 2;
  f->second();
  std::printf("ok\n");
  return 0;
}
