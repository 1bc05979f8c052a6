// sdpa_serving_api.cu — C entry points of the rotary positions, the paged cache, its pages, the attention
// over it and the verification of drafts: argument checks on the host, then one or two launches.  As everywhere in this library
// nothing is allocated or synchronised, and what is not supported is refused with a message.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/sdpa.h"
#include "sdpa_internal.h"

namespace {

using sdpa::api_fail;

#define SDPA_REFUSE(st, ...) return static_cast<sdpa_status_t>(api_fail(st, __VA_ARGS__))
#define SDPA_TRY(call)                                        \
  do {                                                        \
    const sdpa_status_t st_ = (call);                         \
    if (st_ != SDPA_OK) return st_;                           \
  } while (0)

constexpr int64_t kMaxLen = int64_t(1) << 30;   // tokens of a sequence: positions stay well inside 32 bits

bool is16(int dt) { return dt == SDPA_DTYPE_F16 || dt == SDPA_DTYPE_BF16; }

sdpa_status_t view(const char* name, const void* ptr, const sdpa_strides_t& st, int b, int h, int s, int d, int es) {
  return static_cast<sdpa_status_t>(sdpa::api_check_view(name, ptr, {st.b, st.h, st.s, st.d}, b, h, s, d, es));
}

void strides3(int64_t (&to)[3], const sdpa_strides_t& st, int es = 1) {
  to[0] = st.b * es;
  to[1] = st.h * es;
  to[2] = st.s * es;
}

bool same_strides(const sdpa_strides_t& a, const sdpa_strides_t& b) { return a.b == b.b && a.h == b.h && a.s == b.s; }

// What a rotation needs besides its rows (shared by sdpa_rope_* and sdpa_cache_write).
sdpa_status_t check_turn(const sdpa_rope_t* p, int d) {
  if (p->rot < 2 || p->rot > d || p->rot % 2 != 0)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rot must be even and in 2..%d, got %d", d, p->rot);
  if (p->interleaved != 0 && p->interleaved != 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "interleaved must be 0 or 1, got %d", p->interleaved);
  if (!std::isfinite(p->attn_factor)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "attn_factor must be finite");
  if (p->table == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "table: null pointer");
  if (reinterpret_cast<uintptr_t>(p->table) % 8) SDPA_REFUSE(SDPA_ERR_LAYOUT, "table must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(p->positions) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "positions must be 4-byte aligned");
  if (p->positions_stride < 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "positions_stride must not be negative");
  return SDPA_OK;
}

// The axes of a rotation's pairs, for one that has several.
sdpa_status_t check_axes(const sdpa_rope_t* p, const sdpa_rope_axes_t* a) {
  if (a == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "axes descriptor is NULL");
  if (a->axes < 1 || a->axes > sdpa::kMaxAxes)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "%d axes not supported (1..%d)", a->axes, sdpa::kMaxAxes);
  if (a->axis_stride < 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "axis_stride must not be negative");
  if (p->positions == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "axes need positions");
  for (int i = 0; i < p->rot / 2; ++i)
    if (a->axis[i] >= a->axes)
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "axis[%d] must be below axes (%d), got %d", i, a->axes, a->axis[i]);
  return SDPA_OK;
}

// `a`: checked, or NULL: one position a token.
sdpa::RopeArgs turn_of(const sdpa_rope_t* p, const sdpa_rope_axes_t* a, int sign) {
  sdpa::RopeArgs r;
  memset(&r, 0, sizeof(r));
  if (a) {
    r.axes = a->axes;
    r.axis_stride = a->axis_stride;
    for (int i = 0; i < p->rot / 2; ++i) r.axis_of[i / 16] |= static_cast<uint32_t>(a->axis[i]) << (2 * (i % 16));
  }
  r.table = p->table;
  r.positions = p->positions;
  r.positions_stride = p->positions_stride;
  r.rot = p->rot;
  r.interleaved = p->interleaved;
  r.sign = sign;
  r.factor = p->attn_factor;
  return r;
}

sdpa_status_t rope(const sdpa_rope_t* p, bool several, const sdpa_rope_axes_t* a, const void* q, const void* k, void* q_out,
                   void* k_out, int sign, void* stream_, const char* what) {
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rope descriptor is NULL");
  if (p->b < 1 || p->h_q < 1 || p->h_k < 0 || p->s < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (b=%d h_q=%d h_k=%d s=%d)", p->b, p->h_q, p->h_k, p->s);
  if (p->d < 8 || p->d > 512 || p->d % 8 != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "head dim %d not supported (a multiple of 8, 8..512)", p->d);
  if (!is16(p->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "rotary positions take F16 or BF16 (dtype %d)", p->dtype);
  SDPA_TRY(check_turn(p, p->d));
  if (several) SDPA_TRY(check_axes(p, a));
  SDPA_TRY(view("q", q, p->q, p->b, p->h_q, p->s, p->d, 2));
  SDPA_TRY(view("q_out", q_out, p->q_out, p->b, p->h_q, p->s, p->d, 2));
  if (p->h_k > 0) {
    SDPA_TRY(view("k", k, p->k, p->b, p->h_k, p->s, p->d, 2));
    SDPA_TRY(view("k_out", k_out, p->k_out, p->b, p->h_k, p->s, p->d, 2));
  }
  if ((q == q_out && !same_strides(p->q, p->q_out)) || (p->h_k > 0 && k == k_out && !same_strides(p->k, p->k_out)))
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "an output that is its input must have its strides");
  sdpa::RopeParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.r = turn_of(p, several ? a : nullptr, sign);
  prm.in[0] = q;
  prm.in[1] = k;
  prm.out[0] = q_out;
  prm.out[1] = k_out;
  strides3(prm.in_st[0], p->q);
  strides3(prm.in_st[1], p->k);
  strides3(prm.out_st[0], p->q_out);
  strides3(prm.out_st[1], p->k_out);
  prm.in_place[0] = q == q_out;
  prm.in_place[1] = k == k_out;
  prm.b = p->b;
  prm.s = p->s;
  prm.d = p->d;
  prm.h_q = p->h_q;
  prm.h_all = p->h_q + p->h_k;
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] %s b=%d h_q=%d h_k=%d s=%d d=%d rot=%d dt=%d axes=%d\n", what, p->b, p->h_q, p->h_k, p->s, p->d,
            p->rot, p->dtype, prm.r.axes);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_rope(prm, p->dtype, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, what));
}

// What a cache holds: its pages, without the table of a batch.
sdpa_status_t check_stored(const sdpa_cache_t* c) {
  if (c == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cache descriptor is NULL");
  if (c->num_pages < 1 || c->h_kv < 1 || c->page_size < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cache sizes must be >= 1 (num_pages=%d page_size=%d h_kv=%d)", c->num_pages, c->page_size,
                c->h_kv);
  if (c->page_size % 16 != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "page_size %d not supported (a multiple of 16)", c->page_size);
  if (c->d != 64 && c->d != 128 && c->d != 256)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "head dim %d not supported (64, 128 or 256)", c->d);
  if (!is16(c->dtype) && c->dtype != SDPA_DTYPE_E4M3)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a cache holds F16, BF16 or E4M3 (dtype %d)", c->dtype);
  const int es = c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2;
  SDPA_TRY(view("k cache", c->k, c->k_strides, c->num_pages, c->h_kv, c->page_size, c->d, es));
  SDPA_TRY(view("v cache", c->v, c->v_strides, c->num_pages, c->h_kv, c->page_size, c->d, es));
  if (c->dtype == SDPA_DTYPE_E4M3) {
    if (!c->k_scale || !c->v_scale) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "an E4M3 cache needs k_scale and v_scale");
    if (reinterpret_cast<uintptr_t>(c->k_scale) % 16 || reinterpret_cast<uintptr_t>(c->v_scale) % 16)
      SDPA_REFUSE(SDPA_ERR_LAYOUT, "k_scale and v_scale must be 16-byte aligned");
  } else if (c->k_scale || c->v_scale) {
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "a 16-bit cache takes no k_scale and v_scale");
  }
  return SDPA_OK;
}

sdpa_status_t check_cache(const sdpa_cache_t* c) {
  if (c != nullptr && (c->num_pages < 1 || c->h_kv < 1 || c->b < 1 || c->max_pages < 1 || c->page_size < 1))
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cache sizes must be >= 1 (num_pages=%d page_size=%d h_kv=%d b=%d max_pages=%d)",
                c->num_pages, c->page_size, c->h_kv, c->b, c->max_pages);
  SDPA_TRY(check_stored(c));
  if (!c->page_table || !c->seq_lens_kv)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "page_table and seq_lens_kv must not be NULL");
  if (reinterpret_cast<uintptr_t>(c->page_table) % 4 || reinterpret_cast<uintptr_t>(c->seq_lens_kv) % 4)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "page_table and seq_lens_kv must be 4-byte aligned");
  if (c->b > 1 && c->page_table_stride < c->max_pages)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "page_table_stride below max_pages");
  return SDPA_OK;
}

int max_tokens(int max_pages, int page_size) {
  const int64_t cap = static_cast<int64_t>(max_pages) * page_size;
  return static_cast<int>(cap < kMaxLen ? cap : kMaxLen);
}

sdpa::CacheArgs cache_args(const sdpa_cache_t* c) {
  const int es = c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2;
  sdpa::CacheArgs a;
  memset(&a, 0, sizeof(a));
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  strides3(a.k_st, c->k_strides, es);
  strides3(a.v_st, c->v_strides, es);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_table = c->page_table;
  a.page_table_stride = c->page_table_stride;
  a.seq_lens_kv = c->seq_lens_kv;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.h_kv = c->h_kv;
  a.b = c->b;
  a.max_pages = c->max_pages;
  a.max_len = max_tokens(c->max_pages, c->page_size);
  return a;
}

// 32-bit words on the device that a call needs.
sdpa_status_t words(const char* name, const void* ptr) {
  if (ptr == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (reinterpret_cast<uintptr_t>(ptr) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "%s must be 4-byte aligned", name);
  return SDPA_OK;
}

// Whether n words at a and m at b have any in common.
bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * static_cast<uintptr_t>(m) && y < x + 4 * static_cast<uintptr_t>(n);
}

// Words that a call reads or writes (none where `at` is NULL).
struct Words {
  const char* name;
  const void* at;
  int64_t n;
};

// What is written lies apart from what is read, and from what else is written: the CTAs of a call read and write in no order.
sdpa_status_t apart(std::initializer_list<Words> written, std::initializer_list<Words> read) {
  auto clear = [](const Words& w, const Words& x) {
    return x.at == nullptr || !overlap(static_cast<const int32_t*>(w.at), w.n, static_cast<const int32_t*>(x.at), x.n);
  };
  for (const Words& w : written) {
    for (const Words& x : read)
      if (!clear(w, x)) SDPA_REFUSE(SDPA_ERR_LAYOUT, "%s must lie apart from %s", w.name, x.name);
    for (const Words& x : written)
      if (&x != &w && !clear(w, x)) SDPA_REFUSE(SDPA_ERR_LAYOUT, "%s must lie apart from %s", w.name, x.name);
  }
  return SDPA_OK;
}

// Words from the first to the last entry of a page table.
int64_t table_words(int rows, int columns, int64_t stride) { return (rows - 1) * stride + columns; }

// `rows_out`: rows of the table that is written; `in_place`: it may be the one that is read.
sdpa_status_t check_pages(const sdpa_pages_t* p, int rows_out, bool in_place) {
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "pages descriptor is NULL");
  if (p->num_pages < 1 || p->page_size < 1 || p->b < 1 || p->max_pages < 1 || rows_out < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (num_pages=%d page_size=%d b=%d max_pages=%d, %d rows out)", p->num_pages,
                p->page_size, p->b, p->max_pages, rows_out);
  if (p->page_size % 16 != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "page_size %d not supported (a multiple of 16)", p->page_size);
  if (p->num_pages > (1 << 30) || p->max_pages > (1 << 30)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "num_pages or max_pages too large (1..2^30)");
  if (p->b > (1 << 24) || rows_out > (1 << 24) || (static_cast<int64_t>(p->b) + rows_out) * p->max_pages >= (int64_t(1) << 38))
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "b*max_pages too large");
  SDPA_TRY(words("page_table", p->page_table));
  SDPA_TRY(words("seq_lens", p->seq_lens));
  SDPA_TRY(words("ref_counts", p->ref_counts));
  SDPA_TRY(words("page_table_out", p->page_table_out));
  SDPA_TRY(words("ref_counts_out", p->ref_counts_out));
  if ((p->b > 1 && p->page_table_stride < p->max_pages) || (rows_out > 1 && p->page_table_out_stride < p->max_pages))
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "page_table_stride below max_pages");
  const bool same = p->page_table_out == p->page_table;
  if (same ? !in_place || (p->b > 1 && p->page_table_out_stride != p->page_table_stride)
           : overlap(p->page_table, table_words(p->b, p->max_pages, p->page_table_stride), p->page_table_out,
                     table_words(rows_out, p->max_pages, p->page_table_out_stride)))
    SDPA_REFUSE(SDPA_ERR_LAYOUT, in_place ? "page_table_out must be page_table with its stride, or lie apart from it"
                                          : "page_table_out must lie apart from page_table");
  if (p->ref_counts_out != p->ref_counts && overlap(p->ref_counts, p->num_pages, p->ref_counts_out, p->num_pages))
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "ref_counts_out must be ref_counts or lie apart from it");
  return SDPA_OK;
}

// What a call for pages writes (its own lists, and the tables behind them) lies apart from what it reads, but for a table or counts
// that are changed in place (check_pages).
sdpa_status_t check_lists(const sdpa_pages_t* p, int rows_out, std::initializer_list<Words> lists, Words lens) {
  const Words table = {"page_table", p->page_table, table_words(p->b, p->max_pages, p->page_table_stride)};
  const Words table_out = {"page_table_out", p->page_table_out, table_words(rows_out, p->max_pages, p->page_table_out_stride)};
  const Words counts = {"ref_counts", p->ref_counts, p->num_pages}, counts_out = {"ref_counts_out", p->ref_counts_out, p->num_pages};
  const Words seq_lens = {"seq_lens", p->seq_lens, p->b};
  SDPA_TRY(apart(lists, {table, table_out, counts, counts_out, seq_lens, lens}));
  SDPA_TRY(apart({table_out}, {counts, counts_out, seq_lens, lens}));
  return apart({counts_out}, {table, seq_lens, lens});
}

sdpa::PagesParams pages_params(const sdpa_pages_t* p) {
  sdpa::PagesParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.page_table = p->page_table;
  prm.table_stride = p->page_table_stride;
  prm.seq_lens = p->seq_lens;
  prm.ref_counts = p->ref_counts;
  prm.page_table_out = p->page_table_out;
  prm.table_out_stride = p->page_table_out_stride;
  prm.ref_counts_out = p->ref_counts_out;
  prm.num_pages = p->num_pages;
  prm.page_size = p->page_size;
  prm.b = p->b;
  prm.max_pages = p->max_pages;
  prm.max_len = max_tokens(p->max_pages, p->page_size);
  return prm;
}

void log_pages(const char* what, const sdpa_pages_t* p, int n) {
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] %s b=%d max_pages=%d num_pages=%d page=%d n=%d\n", what, p->b, p->max_pages, p->num_pages, p->page_size, n);
}

// A cache's K or V as units of 16 bytes, in the order of memory: the dimension of the smaller stride is the inner one.
sdpa::CopyTensor copy_tensor(void* base, const sdpa_strides_t& st, const sdpa_cache_t* c, int es) {
  sdpa::CopyTensor t;
  memset(&t, 0, sizeof(t));
  const bool slots_inside = st.s <= st.h;
  t.base = static_cast<uint8_t*>(base);
  t.page = st.b * es;
  t.inner = (slots_inside ? st.s : st.h) * es;
  t.outer = (slots_inside ? st.h : st.s) * es;
  t.inner_n = slots_inside ? c->page_size : c->h_kv;
  t.row_units = c->d * es / 16;
  t.units = c->h_kv * c->page_size * t.row_units;
  return t;
}

sdpa::CopyTensor copy_scales(float* base, const sdpa_cache_t* c) {
  sdpa::CopyTensor t;
  memset(&t, 0, sizeof(t));
  if (base == nullptr) return t;
  t.base = reinterpret_cast<uint8_t*>(base);
  t.page = t.inner = t.outer = static_cast<int64_t>(c->h_kv) * c->page_size * 4;
  t.inner_n = 1;
  t.row_units = t.units = c->h_kv * c->page_size / 4;
  return t;
}

sdpa_status_t check_rows(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v) {
  SDPA_TRY(check_cache(c));
  if (r == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rows descriptor is NULL");
  if (r->s < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (s=%d)", r->s);
  if (!is16(r->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "rows are F16 or BF16 (dtype %d)", r->dtype);
  if (c->dtype != SDPA_DTYPE_E4M3 && r->dtype != c->dtype)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a 16-bit cache takes and gives rows of its own dtype (%d, rows %d)", c->dtype, r->dtype);
  SDPA_TRY(view("k", k, r->k, c->b, c->h_kv, r->s, c->d, 2));
  SDPA_TRY(view("v", v, r->v, c->b, c->h_kv, r->s, c->d, 2));
  return SDPA_OK;
}

sdpa::CacheRowsParams rows_params(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v) {
  sdpa::CacheRowsParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.c = cache_args(c);
  prm.k = const_cast<void*>(k);
  prm.v = const_cast<void*>(v);
  strides3(prm.k_st, r->k);
  strides3(prm.v_st, r->v);
  prm.s = r->s;
  prm.d = c->d;
  return prm;
}

sdpa_status_t write(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, bool several, const sdpa_rope_axes_t* a, const void* k,
                    const void* v, void* stream_, const char* what) {
  SDPA_TRY(check_rows(c, r, k, v));
  if (reinterpret_cast<uintptr_t>(r->seq_lens_q) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "seq_lens_q must be 4-byte aligned");
  if (r->rope) SDPA_TRY(check_turn(r->rope, c->d));
  if (several) {
    if (!r->rope) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "axes need a rope descriptor");
    SDPA_TRY(check_axes(r->rope, a));
  }
  sdpa::CacheRowsParams prm = rows_params(c, r, k, v);
  prm.seq_lens_q = r->seq_lens_q;
  prm.rope = r->rope != nullptr;
  if (r->rope) prm.r = turn_of(r->rope, several ? a : nullptr, 1);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] cache_write b=%d h_kv=%d s=%d d=%d dt=%d cache=%d rot=%d axes=%d\n", c->b, c->h_kv, r->s, c->d,
            r->dtype, c->dtype, r->rope ? r->rope->rot : 0, prm.r.axes);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_cache_write(prm, r->dtype, c->dtype, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, what));
}

// Sizes and options of an attention call (all that its workspace depends on).
sdpa_status_t check_decode_sizes(const sdpa_cache_t* c, const sdpa_decode_t* p) {
  SDPA_TRY(check_cache(c));
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "decode descriptor is NULL");
  if (p->h_q < 1 || p->s_q < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (h_q=%d s_q=%d)", p->h_q, p->s_q);
  if (p->h_q % c->h_kv != 0)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "h_q (%d) must be a multiple of h_kv (%d)", p->h_q, c->h_kv);
  if (!is16(p->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "Q and O are F16 or BF16 (dtype %d)", p->dtype);
  if (c->dtype != SDPA_DTYPE_E4M3 && p->dtype != c->dtype)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "over a 16-bit cache Q and O have its dtype (%d, Q %d)", c->dtype, p->dtype);
  if (p->causal == 1)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "attention over a cache takes causal = 0 or 2 (bottom-right), not top-left");
  if (p->causal != 0 && p->causal != 2)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "causal must be 0 (none) or 2 (bottom-right), got %d", p->causal);
  if (p->tree_mask && p->causal != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a tree mask says itself what a row sees: causal must be 0");
  if (reinterpret_cast<uintptr_t>(p->tree_mask) % 4 || reinterpret_cast<uintptr_t>(p->seq_lens_q) % 4)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "tree_mask and seq_lens_q must be 4-byte aligned");
  if (p->tree_mask_stride < 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "tree_mask_stride must not be negative");
  if (!std::isfinite(p->attn_scale)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "attn_scale must be finite");
  const int64_t rows = static_cast<int64_t>(p->s_q) * (p->h_q / c->h_kv);
  if (rows * c->b * c->h_kv >= (int64_t(1) << 31)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "b*h_q*s_q too large");
  return SDPA_OK;
}

sdpa::DecodeParams decode_params(const sdpa_cache_t* c, const sdpa_decode_t* p) {
  sdpa::DecodeParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.c = cache_args(c);
  strides3(prm.q_st, p->q);
  strides3(prm.o_st, p->o);
  prm.seq_lens_q = p->seq_lens_q;
  prm.tree_mask = p->tree_mask;
  prm.tree_mask_stride = p->tree_mask_stride;
  prm.tree_words = (p->s_q + 31) / 32;
  prm.causal = p->causal;
  prm.h_q = p->h_q;
  prm.s_q = p->s_q;
  prm.group = p->h_q / c->h_kv;
  prm.rows = p->s_q * prm.group;
  prm.scale_log2 = p->attn_scale * 1.4426950408889634f;
  sdpa::decode_plan(&prm, c->d, c->dtype, sdpa::api_num_sms());
  return prm;
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_rope_table(const sdpa_rope_table_t* cfg, int64_t* table, float* attn_factor) {
  if (cfg == nullptr || table == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cfg and table must not be NULL");
  if (cfg->rot < 2 || cfg->rot % 2 != 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rot must be even and >= 2, got %d", cfg->rot);
  const int n = cfg->rot / 2;
  double base = cfg->base;
  if (cfg->inv_freq == nullptr) {
    if (cfg->scaling < 0 || cfg->scaling > 3)
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "scaling must be 0 (none), 1 (linear), 2 (NTK) or 3 (by parts), got %d", cfg->scaling);
    if (!(base > 0) || !std::isfinite(base)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "base must be positive and finite");
    if (cfg->scaling != 0 && !(cfg->factor >= 1 && std::isfinite(cfg->factor)))
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "factor must be >= 1 and finite");
    if (cfg->scaling == 2) {
      if (cfg->rot == 2) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "NTK scaling needs rot > 2");
      base *= std::pow(cfg->factor, cfg->rot / (cfg->rot - 2.0));
    }
    if (cfg->scaling == 3 &&
        !(cfg->original_context > 0 && cfg->beta_fast > cfg->beta_slow && std::isfinite(cfg->original_context) &&
          std::isfinite(cfg->beta_fast) && std::isfinite(cfg->beta_slow)))
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "scaling by parts needs original_context > 0 and beta_fast > beta_slow");
  } else {
    for (int i = 0; i < n; ++i)
      if (!std::isfinite(cfg->inv_freq[i])) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "inv_freq[%d] must be finite", i);
  }
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < n; ++i) {
    double f = 0;
    if (cfg->inv_freq) {
      f = cfg->inv_freq[i];
    } else {
      f = std::pow(base, -2.0 * i / cfg->rot);
      if (cfg->scaling == 1) f /= cfg->factor;
      if (cfg->scaling == 3) {
        const double r = cfg->original_context * f / kTwoPi;
        double g = (r - cfg->beta_slow) / (cfg->beta_fast - cfg->beta_slow);
        g = g < 0 ? 0 : g > 1 ? 1 : g;
        f = f * g + f / cfg->factor * (1 - g);
      }
    }
    double turns = f / kTwoPi;
    turns -= std::floor(turns);                        // [0, 1], 1 where a tiny negative was rounded
    const double hi = std::floor(turns * 4294967296.0);
    const double lo = std::nearbyint((turns * 4294967296.0 - hi) * 4294967296.0);   // 2^32 carries
    table[i] = static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo));
  }
  if (attn_factor)
    *attn_factor = cfg->inv_freq == nullptr && cfg->scaling == 3 ? static_cast<float>(0.1 * std::log(cfg->factor) + 1.0) : 1.f;
  return static_cast<sdpa_status_t>(sdpa::api_ok());
}

sdpa_status_t sdpa_rope_fwd(const sdpa_rope_t* p, const void* q, const void* k, void* q_out, void* k_out, void* stream) {
  return rope(p, false, nullptr, q, k, q_out, k_out, 1, stream, "sdpa_rope_fwd");
}

sdpa_status_t sdpa_rope_bwd(const sdpa_rope_t* p, const void* dq_out, const void* dk_out, void* dq, void* dk, void* stream) {
  return rope(p, false, nullptr, dq_out, dk_out, dq, dk, -1, stream, "sdpa_rope_bwd");
}

sdpa_status_t sdpa_rope_axes_fwd(const sdpa_rope_t* p, const sdpa_rope_axes_t* a, const void* q, const void* k, void* q_out,
                                 void* k_out, void* stream) {
  return rope(p, true, a, q, k, q_out, k_out, 1, stream, "sdpa_rope_axes_fwd");
}

sdpa_status_t sdpa_rope_axes_bwd(const sdpa_rope_t* p, const sdpa_rope_axes_t* a, const void* dq_out, const void* dk_out,
                                 void* dq, void* dk, void* stream) {
  return rope(p, true, a, dq_out, dk_out, dq, dk, -1, stream, "sdpa_rope_axes_bwd");
}

sdpa_status_t sdpa_cache_write(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v,
                               void* stream) {
  return write(c, r, false, nullptr, k, v, stream, "sdpa_cache_write");
}

sdpa_status_t sdpa_cache_write_axes(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const sdpa_rope_axes_t* a,
                                    const void* k, const void* v, void* stream) {
  return write(c, r, true, a, k, v, stream, "sdpa_cache_write_axes");
}

sdpa_status_t sdpa_cache_read(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, void* k, void* v, void* stream_) {
  SDPA_TRY(check_rows(c, r, k, v));
  sdpa::CacheRowsParams prm = rows_params(c, r, k, v);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] cache_read b=%d h_kv=%d s=%d d=%d dt=%d cache=%d\n", c->b, c->h_kv, r->s, c->d, r->dtype, c->dtype);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_cache_read(prm, r->dtype, c->dtype, stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_read"));
}

sdpa_status_t sdpa_decode_workspace_size(const sdpa_cache_t* c, const sdpa_decode_t* p, size_t* bytes) {
  if (bytes == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "bytes is NULL");
  SDPA_TRY(check_decode_sizes(c, p));
  *bytes = sdpa::decode_workspace_bytes(decode_params(c, p), c->d, nullptr);
  return static_cast<sdpa_status_t>(sdpa::api_ok());
}

sdpa_status_t sdpa_decode(const sdpa_cache_t* c, const sdpa_decode_t* p, const void* q, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream_) {
  SDPA_TRY(check_decode_sizes(c, p));
  SDPA_TRY(view("q", q, p->q, c->b, p->h_q, p->s_q, c->d, 2));
  SDPA_TRY(view("o", o, p->o, c->b, p->h_q, p->s_q, c->d, 2));
  if (reinterpret_cast<uintptr_t>(lse) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "lse must be 4-byte aligned");
  sdpa::DecodeParams prm = decode_params(c, p);
  size_t ml = 0;
  const size_t need = sdpa::decode_workspace_bytes(prm, c->d, &ml);
  if (workspace == nullptr || workspace_bytes < need)
    SDPA_REFUSE(SDPA_ERR_WORKSPACE, "workspace of %zu bytes required, %zu given%s", need, workspace_bytes,
                workspace ? "" : " (NULL)");
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    SDPA_REFUSE(SDPA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  prm.q = q;
  prm.o = o;
  prm.lse = lse;
  prm.part_o = static_cast<float*>(workspace);
  prm.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ml);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] decode b=%d h_q=%d h_kv=%d s_q=%d d=%d dt=%d cache=%d page=%d block=%d ctas=%d ws=%zu\n", c->b, p->h_q,
            c->h_kv, p->s_q, c->d, p->dtype, c->dtype, c->page_size, prm.tile_rows, prm.ctas, need);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (prm.wide) {
    CUtensorMap tm_k, tm_v;
    const int box = sdpa::decode_wide_box(c->page_size);
    const sdpa_strides_t &ks = c->k_strides, &vs = c->v_strides;
    SDPA_TRY(static_cast<sdpa_status_t>(sdpa::api_make_map(&tm_k, "k cache", c->k, {ks.b, ks.h, ks.s, ks.d}, c->num_pages,
                                                           c->h_kv, c->page_size, c->d, c->dtype, box)));
    SDPA_TRY(static_cast<sdpa_status_t>(sdpa::api_make_map(&tm_v, "v cache", c->v, {vs.b, vs.h, vs.s, vs.d}, c->num_pages,
                                                           c->h_kv, c->page_size, c->d, c->dtype, box)));
    e = sdpa::launch_decode_wide(prm, tm_k, tm_v, sdpa::api_wait_limit(), c->d, p->dtype, c->dtype, stream);
  } else {
    e = sdpa::launch_decode(prm, c->d, p->dtype, c->dtype, stream);
  }
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_decode"));
}

sdpa_status_t sdpa_cache_fork(const sdpa_pages_t* p, const int32_t* parents, int32_t b_out, int32_t* seq_lens_out, void* stream_) {
  SDPA_TRY(check_pages(p, b_out, false));
  SDPA_TRY(words("parents", parents));
  SDPA_TRY(words("seq_lens_out", seq_lens_out));
  SDPA_TRY(check_lists(p, b_out, {{"seq_lens_out", seq_lens_out, b_out}}, {"parents", parents, b_out}));
  log_pages("fork", p, b_out);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_fork(pages_params(p), parents, b_out, seq_lens_out, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_fork"));
}

sdpa_status_t sdpa_cache_grow(const sdpa_pages_t* p, const int32_t* new_lens, int32_t* src, int32_t* dst, int32_t* missing,
                              void* stream_) {
  SDPA_TRY(check_pages(p, p ? p->b : 1, true));
  if (p->b > sdpa::kMaxPageRows) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "%d rows not supported (1..%d)", p->b, sdpa::kMaxPageRows);
  if (static_cast<int64_t>(p->b) * p->max_pages >= (int64_t(1) << 31))     // (pages that one call may want are counted in 32 bits)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "b*max_pages too large (below 2^31)");
  SDPA_TRY(words("new_lens", new_lens));
  SDPA_TRY(words("src", src));
  SDPA_TRY(words("dst", dst));
  SDPA_TRY(words("missing", missing));
  SDPA_TRY(check_lists(p, p->b, {{"src", src, p->b}, {"dst", dst, p->b}, {"missing", missing, 1}}, {"new_lens", new_lens, p->b}));
  log_pages("grow", p, 0);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_grow(pages_params(p), new_lens, src, dst, missing, stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_grow"));
}

sdpa_status_t sdpa_cache_free(const sdpa_pages_t* p, const int32_t* keep_lens, void* stream_) {
  SDPA_TRY(check_pages(p, p ? p->b : 1, true));
  SDPA_TRY(words("keep_lens", keep_lens));
  SDPA_TRY(check_lists(p, p->b, {}, {"keep_lens", keep_lens, p->b}));
  log_pages("free", p, 0);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_free(pages_params(p), keep_lens, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_free"));
}

sdpa_status_t sdpa_cache_compact(const sdpa_pages_t* p, int32_t* src, int32_t* dst, int32_t pairs, void* stream_) {
  SDPA_TRY(check_pages(p, p ? p->b : 1, true));
  if (pairs < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (pairs=%d)", pairs);
  SDPA_TRY(words("src", src));
  SDPA_TRY(words("dst", dst));
  SDPA_TRY(check_lists(p, p->b, {{"src", src, pairs}, {"dst", dst, pairs}}, {"", nullptr, 0}));
  log_pages("compact", p, pairs);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_compact(pages_params(p), src, dst, pairs, stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_compact"));
}

sdpa_status_t sdpa_cache_copy(const sdpa_cache_t* c, const int32_t* src, const int32_t* dst, int32_t pairs, void* stream_) {
  SDPA_TRY(check_stored(c));
  if (pairs < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (pairs=%d)", pairs);
  SDPA_TRY(words("src", src));
  SDPA_TRY(words("dst", dst));
  const int es = c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2;
  if (static_cast<int64_t>(c->h_kv) * c->page_size * c->d >= (int64_t(1) << 31)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "h_kv*page_size*d too large");
  sdpa::CopyParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.t[0] = copy_tensor(c->k, c->k_strides, c, es);
  prm.t[1] = copy_tensor(c->v, c->v_strides, c, es);
  prm.t[2] = copy_scales(c->k_scale, c);
  prm.t[3] = copy_scales(c->v_scale, c);
  prm.num_pages = c->num_pages;
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] copy pairs=%d h_kv=%d d=%d cache=%d page=%d\n", pairs, c->h_kv, c->d, c->dtype, c->page_size);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_copy(prm, src, dst, pairs, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_copy"));
}

sdpa_status_t sdpa_cache_keep(const sdpa_cache_t* c, const int32_t* path, const int32_t* accepted, int32_t s,
                              const int32_t* seq_lens_q, void* stream_) {
  SDPA_TRY(check_cache(c));
  if (s < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (s=%d)", s);
  SDPA_TRY(words("path", path));
  SDPA_TRY(words("accepted", accepted));
  if (reinterpret_cast<uintptr_t>(seq_lens_q) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "seq_lens_q must be 4-byte aligned");
  sdpa::KeepParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.c = cache_args(c);
  prm.seq_lens_q = seq_lens_q;
  prm.path = path;
  prm.accepted = accepted;
  prm.s = s;
  prm.row_units = c->d * (c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2) / 16;
  if (static_cast<int64_t>(c->h_kv) * (prm.row_units + 1) >= (int64_t(1) << 30)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "h_kv too large");
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] keep b=%d s=%d h_kv=%d d=%d cache=%d page=%d\n", c->b, s, c->h_kv, c->d, c->dtype, c->page_size);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_keep(prm, stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_keep"));
}

sdpa_status_t sdpa_verify(const sdpa_verify_t* p, void* stream_) {
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "verify descriptor is NULL");
  if (p->b < 1 || p->s < 1 || p->vocab < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (b=%d s=%d vocab=%d)", p->b, p->s, p->vocab);
  if (p->s > sdpa::kVerifyRows) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "%d rows not supported (1..%d)", p->s, sdpa::kVerifyRows);
  if (p->vocab > (1 << 20)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "vocabulary of %d not supported (1..2^20)", p->vocab);
  if (p->b > (1 << 24)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "b too large");
  if (!is16(p->dtype) && p->dtype != SDPA_DTYPE_F32)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "probabilities are F16, BF16 or F32 (dtype %d)", p->dtype);
  if (p->parents && p->draft_probs)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "draft_probs are those of a chain: parents must be NULL");
  const int es = p->dtype == SDPA_DTYPE_F32 ? 4 : 2;
  SDPA_TRY(words("tokens", p->tokens));
  SDPA_TRY(words("uniform", p->uniform));
  SDPA_TRY(words("accepted", p->accepted));
  SDPA_TRY(words("path", p->path));
  SDPA_TRY(words("new_tokens", p->new_tokens));
  if (reinterpret_cast<uintptr_t>(p->parents) % 4 || reinterpret_cast<uintptr_t>(p->seq_lens_q) % 4)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "parents and seq_lens_q must be 4-byte aligned");
  if (p->probs == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "probs: null pointer");
  if (reinterpret_cast<uintptr_t>(p->probs) % es || reinterpret_cast<uintptr_t>(p->draft_probs) % es)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "probs and draft_probs must be aligned to their elements");
  if (p->probs_b < 0 || p->probs_s < 0 || p->draft_b < 0 || p->draft_s < 0)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "strides of probs and draft_probs must not be negative");
  const int64_t rows = static_cast<int64_t>(p->b) * p->s;
  SDPA_TRY(apart({{"accepted", p->accepted, p->b}, {"path", p->path, rows}, {"new_tokens", p->new_tokens, rows}},
                 {{"tokens", p->tokens, rows}, {"parents", p->parents, rows}, {"seq_lens_q", p->seq_lens_q, p->b}, {"uniform", p->uniform, rows}}));
  sdpa::VerifyParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.tokens = p->tokens;
  prm.parents = p->parents;
  prm.seq_lens_q = p->seq_lens_q;
  prm.uniform = p->uniform;
  prm.probs = p->probs;
  prm.probs_b = p->probs_b;
  prm.probs_s = p->probs_s;
  prm.draft = p->draft_probs;
  prm.draft_b = p->draft_b;
  prm.draft_s = p->draft_s;
  prm.accepted = p->accepted;
  prm.path = p->path;
  prm.new_tokens = p->new_tokens;
  prm.b = p->b;
  prm.s = p->s;
  prm.vocab = p->vocab;
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] verify b=%d s=%d vocab=%d dt=%d tree=%d draft=%d\n", p->b, p->s, p->vocab, p->dtype, p->parents != nullptr,
            p->draft_probs != nullptr);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_verify(prm, p->dtype, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_verify"));
}

size_t sdpa_serving_struct_size(int which) {
  switch (which) {
    case 0: return sizeof(sdpa_rope_table_t);
    case 1: return sizeof(sdpa_rope_t);
    case 2: return sizeof(sdpa_cache_t);
    case 3: return sizeof(sdpa_cache_rows_t);
    case 4: return sizeof(sdpa_decode_t);
    case 5: return sizeof(sdpa_rope_axes_t);
    case 6: return sizeof(sdpa_pages_t);
    case 7: return sizeof(sdpa_verify_t);
    default: return 0;
  }
}

}  // extern "C"
